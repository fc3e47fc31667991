"""The modality-specific layer norm with weights and its backward on the GPU,
through the C ABI, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
import resolution_packed_diffusion_b200 as mf
from mlp_util import _f64, bf16, check_bf16, dev, dev32, guarded, host, modalities

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

EPS = 1e-6
MIXED = ((1, 3, 5, 2), (0, 0, 0, 4), (1, 1, 1, 0), (1, 2, 9, 7))
# (pack, width): one token, every way rows are shared, widths that end inside a
# thread group, modalities that change inside a step, one modality only
CASES = [(((0, 0, 0, 1),), 8), (((1, 1, 1, 0),), 64), (MIXED, 56), (MIXED, 72), (MIXED, 128),
         (MIXED, 136), (MIXED, 256), (MIXED, 264), (((1, 20, 41, 77), (1, 9, 9, 3)), 512),
         (((0, 0, 0, 301),), 768), (((1, 17, 31, 0),), 1000), (MIXED, 2048), (MIXED, 3000),
         (((1, 40, 41, 60), (1, 13, 7, 1)), 4096), (MIXED, 4104), (MIXED, 8192)]


def _data(descs, hid, seed):
    rng = np.random.default_rng(seed)
    mod = modalities(descs)
    T = len(mod)
    x = bf16(rng.standard_normal((T, hid)) + 0.3 * rng.standard_normal((T, 1)))
    gamma = np.float32(1 + 0.1 * rng.standard_normal((2, hid)))
    beta = np.float32(0.1 * rng.standard_normal((2, hid)))
    dy, resid = bf16(rng.standard_normal((T, hid))), bf16(rng.standard_normal((T, hid)))
    return mod, x, gamma, beta, dy, resid


def _fwd(x, gamma, beta, mod, with_stats=True, eps=EPS):
    T, hid = x.shape
    y, yc = guarded((T, hid), torch.bfloat16)
    st, sc = guarded((T, 2), torch.float32)
    mf.mf_layer_norm(dev(x), dev32(gamma), dev32(beta), torch.from_numpy(mod).cuda(), T, hid, eps, y,
                     st if with_stats else None)
    assert mf.mf_get_error() == mf.MF_OK
    yc()
    sc()
    return host(y), host(st)


def _norm_slack(x, mean, rstd, gamma, beta, mod):
    """fp32 error of a normalised row: the mean and the variance are sums of n terms
    reduced in at most 8 + 5 + 32 additions a path, each off by 2^-24 of the sum of
    magnitudes; xhat and y add a few units more."""
    ax = np.abs(x).mean(1, keepdims=True) * rstd[:, None]
    xhat = np.abs((x - mean[:, None]) * rstd[:, None])
    return 2.0 ** -24 * (64 * ax * np.abs(gamma)[mod] + 64 * xhat * np.abs(gamma)[mod] + 4 * np.abs(beta)[mod])


@pytest.mark.parametrize("k", range(len(CASES)))
def test_forward(k):
    descs, hid = CASES[k]
    mod, x, gamma, beta, _, _ = _data(descs, hid, 100 + k)
    y, st = _fwd(x, gamma, beta, mod)
    ref, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    check_bf16(y, ref, _norm_slack(x, mean, rstd, gamma, beta, mod), "y")
    np.testing.assert_allclose(st[:, 0], mean, rtol=0, atol=64 * 2.0 ** -24 * np.abs(x).mean(1).max())
    np.testing.assert_allclose(st[:, 1], rstd, rtol=128 * 2.0 ** -24)
    again, _ = _fwd(x, gamma, beta, mod, with_stats=False)
    assert np.array_equal(again, y)


def test_forward_keeps_precision_with_an_outlier_and_a_large_mean():
    """A massive channel and a mean far from 0: the variance is taken about the mean."""
    mod, x, gamma, beta, _, _ = _data(MIXED, 1024, 7)
    x[:, 0] = bf16(3e4)
    x[3] = bf16(x[3] + 500)
    y, st = _fwd(x, gamma, beta, mod)
    ref, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    check_bf16(y, ref, _norm_slack(x, mean, rstd, gamma, beta, mod), "y")
    np.testing.assert_allclose(st[:, 1], rstd, rtol=1e-4)


def test_constant_rows():
    mod = modalities(MIXED)
    x = bf16(np.full((len(mod), 128), 5.0))
    gamma, beta = np.ones((2, 128), np.float32), np.full((2, 128), 0.25, np.float32)
    y, st = _fwd(x, gamma, beta, mod)
    assert (y == 0.25).all() and np.allclose(st[:, 1], 1e3)


def _bwd(dy, x, gamma, stats, mod, resid=None, in_place=False, ckpt=False):
    T, hid = dy.shape
    dx, dc = guarded((T, hid), torch.bfloat16)
    r = dev(resid) if resid is not None else None
    if in_place:
        dx, dc = r, lambda: None
    dg = torch.full((2, hid), float("nan"), device="cuda")
    db = torch.full((2, hid), float("nan"), device="cuda")
    x8 = xs = None
    if ckpt:
        q, s = oracle.act8_quantize(x)
        x8, xs = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mf.mf_layer_norm_bwd(dev(dy), None if ckpt else dev(x), x8, xs, dev32(gamma), dev32(stats),
                         torch.from_numpy(mod).cuda(), r, T, hid, dx, dg, db, ws, n)
    assert mf.mf_get_error() == mf.MF_OK
    dc()
    return host(dx), host(dg), host(db)


@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "act8"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_backward(k, ckpt):
    descs, hid = CASES[k]
    mod, x, gamma, beta, dy, resid = _data(descs, hid, 300 + k)
    xv = oracle.act8_values(*oracle.act8_quantize(x)) if ckpt else _f64(x)
    _, mean, rstd = oracle.layer_norm_affine(xv, gamma, beta, mod, EPS)
    stats = np.float32(np.stack([mean, rstd], 1))
    resid = resid if k % 2 else None
    dx, dg, db = _bwd(dy, x, gamma, stats, mod, resid, in_place=k % 4 == 1, ckpt=ckpt)
    rdx, rdg, rdb = oracle.layer_norm_affine_bwd(dy, xv, gamma, stats, mod, resid)
    s64 = _f64(stats)
    xhat = np.abs((xv - s64[:, :1]) * s64[:, 1:])
    g = np.abs(dy * _f64(gamma)[mod])
    # x - mean loses 2^-24 of |x| + |mean|; the two row sums are off by at most 64
    # units of their sums of magnitudes, then a few units for the expression
    lose = (np.abs(xv) + np.abs(s64[:, :1])) * s64[:, 1:]
    m1, m2 = g.mean(1, keepdims=True), (g * (xhat + lose)).mean(1, keepdims=True)
    slack = 2.0 ** -24 * s64[:, 1:] * (8 * g + 72 * m1 + (72 * xhat + 8 * lose) * m2)
    if resid is not None:
        slack = slack + 2.0 ** -24 * np.abs(resid)
    check_bf16(dx, rdx, slack, "dx")
    # column sums: at most T additions deep, each 2^-24 of the sum of magnitudes
    for got, ref, terms, name in ((dg, rdg, np.abs(dy) * (xhat + 4 * lose), "dgamma"),
                                  (db, rdb, np.abs(dy), "dbeta")):
        mags = np.stack([terms[mod == m].sum(0) for m in (0, 1)])
        assert (np.abs(got - ref) <= (len(mod) + 8) * 2.0 ** -24 * mags).all(), name


def test_backward_repeats_bit_for_bit_and_from_a_graph():
    descs, hid = ((1, 40, 41, 60), (1, 30, 7, 900)), 1536
    mod, x, gamma, beta, dy, resid = _data(descs, hid, 55)
    _, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    st = np.float32(np.stack([mean, rstd], 1))
    first = _bwd(dy, x, gamma, st, mod, resid)
    for got, want in zip(_bwd(dy, x, gamma, st, mod, resid), first):
        assert np.array_equal(got, want)
    T = len(mod)
    args = [dev(dy), dev(x), None, None, dev32(gamma), dev32(st), torch.from_numpy(mod).cuda(), dev(resid)]
    out = [torch.empty((T, hid), dtype=torch.bfloat16, device="cuda"),
           torch.empty((2, hid), device="cuda"), torch.empty((2, hid), device="cuda")]
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mf.mf_layer_norm_bwd(*args, T, hid, *out, ws, n)
    for _ in range(2):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, first):
            assert np.array_equal(host(got), want)


def test_bad_modality_rows_are_reported_and_left_alone():
    descs, hid = MIXED, 264
    mod, x, gamma, beta, dy, _ = _data(descs, hid, 77)
    bad = mod.copy()
    bad[5] = 9
    T = len(mod)
    y = torch.full((T, hid), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((T, 2), 3.0, device="cuda")
    tm = torch.from_numpy(bad).cuda()
    mf.mf_layer_norm(dev(x), dev32(gamma), dev32(beta), tm, T, hid, EPS, y, st)
    assert mf.mf_get_error() == mf.MF_ERR_INVALID
    assert (y[5] == 3.0).all() and (st[5] == 3.0).all()
    ref, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    rest = np.arange(T) != 5
    check_bf16(host(y)[rest], ref[rest], _norm_slack(x, mean, rstd, gamma, beta, mod)[rest], "y")
    y.fill_(3.0)
    dg, db = torch.empty((2, hid), device="cuda"), torch.empty((2, hid), device="cuda")
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    stats = np.float32(np.stack([mean, rstd], 1))
    mf.mf_layer_norm_bwd(dev(dy), dev(x), None, None, dev32(gamma), dev32(stats), tm, None, T, hid, y,
                         dg, db, ws, n)
    assert mf.mf_get_error() == mf.MF_ERR_INVALID
    assert (y[5] == 3.0).all()
    _, rdg, rdb = oracle.layer_norm_affine_bwd(dy[rest], x[rest], gamma, stats[rest], mod[rest])
    np.testing.assert_allclose(host(dg), rdg, atol=1e-4)
    np.testing.assert_allclose(host(db), rdb, atol=1e-4)


def test_nothing_to_normalise():
    mf.mf_layer_norm(None, None, None, None, 0, 256, EPS, None)
    dg, db = torch.full((2, 256), 5.0, device="cuda"), torch.full((2, 256), 5.0, device="cuda")
    mf.mf_layer_norm_bwd(None, None, None, None, None, None, None, None, 0, 256, None, dg, db, None, 0)
    assert (dg == 0).all() and (db == 0).all()


def test_foreign_rows_do_not_leak():
    """NaN in the text rows leaves image rows and image gradients as they were."""
    mod, x, gamma, beta, dy, _ = _data(MIXED, 520, 91)
    _, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    st = np.float32(np.stack([mean, rstd], 1))
    clean = _bwd(dy, x, gamma, st, mod)
    T = len(mod)
    xt, dt = dev(x), dev(dy)
    text = torch.from_numpy(mod == 1).cuda()
    xt[text] = float("nan")
    dt[text] = float("inf")
    dx = torch.empty((T, 520), dtype=torch.bfloat16, device="cuda")
    dg, db = torch.empty((2, 520), device="cuda"), torch.empty((2, 520), device="cuda")
    n = mf.mf_layer_norm_bwd_workspace_size(T, 520)
    mf.mf_layer_norm_bwd(dt, xt, None, None, dev32(gamma), dev32(st), torch.from_numpy(mod).cuda(), None,
                         T, 520, dx, dg, db, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert np.array_equal(host(dx)[mod == 0], clean[0][mod == 0])
    assert np.array_equal(host(dg)[0], clean[1][0]) and np.array_equal(host(db)[0], clean[2][0])


def test_offsets_past_32_bits():
    """2^31 + values: the last rows forward and backward, the sums theirs alone."""
    hid = 8192
    T = (1 << 31) // hid + 5
    rng = np.random.default_rng(17)
    tail, dtail = bf16(rng.standard_normal((6, hid))), bf16(rng.standard_normal((6, hid)))
    gamma, beta = (np.float32(a + 0.1 * rng.standard_normal((2, hid))) for a in (1, 0))
    mod = np.zeros(T, np.uint8)
    mod[-3:] = 1
    x = torch.zeros((T, hid), dtype=torch.bfloat16, device="cuda")
    x[-6:] = dev(tail)
    y = torch.empty_like(x)
    st = torch.empty((T, 2), device="cuda")
    tm = torch.from_numpy(mod).cuda()
    mf.mf_layer_norm(x, dev32(gamma), dev32(beta), tm, T, hid, EPS, y, st)
    ref, mean, rstd = oracle.layer_norm_affine(tail, gamma, beta, mod[-6:], EPS)
    check_bf16(host(y[-6:]), ref, _norm_slack(tail, mean, rstd, gamma, beta, mod[-6:]), "tail")
    y.zero_()
    y[-6:] = dev(dtail)
    dx = torch.empty_like(x)
    dg, db = torch.empty((2, hid), device="cuda"), torch.empty((2, hid), device="cuda")
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    mf.mf_layer_norm_bwd(y, x, None, None, dev32(gamma), st, tm, None, T, hid, dx, dg, db,
                         torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert mf.mf_get_error() == mf.MF_OK
    s6 = host(st[-6:])
    rdx, rdg, rdb = oracle.layer_norm_affine_bwd(dtail, tail, gamma, s6, mod[-6:])
    # fp32 units of the row's terms as in test_backward, |xhat| <= 6, |g| <= 6 here
    check_bf16(host(dx[-6:]), rdx, 2.0 ** -24 * 512 * np.abs(s6[:, 1:]), "dx tail")
    np.testing.assert_allclose(host(dg), rdg, atol=16 * 2.0 ** -24 * 150)
    np.testing.assert_allclose(host(db), rdb, atol=16 * 2.0 ** -24 * 30)
    assert (dx[:-6] == 0).all()


def test_tensors_on_16_byte_boundaries():
    """The least alignment the library asks for."""
    mod, x, gamma, beta, dy, resid = _data(MIXED, 1032, 23)
    T, hid = x.shape

    def off(t):
        whole = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = whole[16 // t.element_size():][: t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    want_y, want_st = _fwd(x, gamma, beta, mod)
    y, st = off(torch.zeros((T, hid), dtype=torch.bfloat16)), torch.empty((T, 2), device="cuda")
    tm = torch.from_numpy(mod).cuda()
    mf.mf_layer_norm(off(dev(x)), off(dev32(gamma)), off(dev32(beta)), tm, T, hid, EPS, y, st)
    assert np.array_equal(host(y), want_y) and np.array_equal(host(st), want_st)
    want = _bwd(dy, x, gamma, want_st, mod, resid)
    dx = off(torch.zeros((T, hid), dtype=torch.bfloat16))
    dg, db = off(torch.zeros((2, hid))), off(torch.zeros((2, hid)))
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    mf.mf_layer_norm_bwd(off(dev(dy)), off(dev(x)), None, None, off(dev32(gamma)), st, tm,
                         off(dev(resid)), T, hid, dx, dg, db,
                         torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    for got, ref in zip((dx, dg, db), want):
        assert np.array_equal(host(got), ref)


def test_forward_replayed_on_another_stream():
    mod, x, gamma, beta, _, _ = _data(MIXED, 768, 31)
    T, hid = x.shape
    other = bf16(x[::-1])
    xt, y, st = dev(x), torch.empty((T, hid), dtype=torch.bfloat16, device="cuda"), torch.empty((T, 2), device="cuda")
    args = [dev32(gamma), dev32(beta), torch.from_numpy(mod).cuda()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mf.mf_layer_norm(xt, *args, T, hid, EPS, y, st)
    xt.copy_(dev(other))
    graph.replay()
    torch.cuda.synchronize()
    want_y, want_st = _fwd(other, gamma, beta, mod)
    assert np.array_equal(host(y), want_y) and np.array_equal(host(st), want_st)


@pytest.mark.parametrize("hid,ckpt", [(264, False), (1536, False), (3000, True)])
def test_a_backward_whose_waits_run_out_leaves_nothing_behind(hid, ckpt):
    """With a limit of 1 ns a wait for the first copies may run out: the call then
    reports it, having started no further copies and waited for those under way, and
    the next call under the usual limit is as good as ever."""
    descs = ((1, 40, 41, 60), (1, 30, 7, 900))
    mod, x, gamma, beta, dy, resid = _data(descs, hid, 61)
    xv = oracle.act8_values(*oracle.act8_quantize(x)) if ckpt else x
    _, mean, rstd = oracle.layer_norm_affine(xv, gamma, beta, mod, EPS)
    st = np.float32(np.stack([mean, rstd], 1))
    want = _bwd(dy, x, gamma, st, mod, resid, ckpt=ckpt)
    T = len(mod)
    x8, xs = (torch.from_numpy(a).cuda() for a in oracle.act8_quantize(x))
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    args = [dev(dy), *((None, x8, xs) if ckpt else (dev(x), None, None)), dev32(gamma), dev32(st),
            torch.from_numpy(mod).cuda(), dev(resid), T, hid]
    dx, dxc = guarded((T, hid), torch.bfloat16)
    out = [dx, torch.empty((2, hid), device="cuda"), torch.empty((2, hid), device="cuda"),
           torch.empty(n, dtype=torch.uint8, device="cuda"), n]
    try:
        mf.mf_set_wait_limit_ns(1)
        for _ in range(4):
            mf.mf_layer_norm_bwd(*args, *out)
            status = mf.mf_get_error()
            assert status in (mf.MF_OK, mf.MF_ERR_TIMEOUT)
            if status == mf.MF_OK:
                assert np.array_equal(host(dx), want[0])
            dxc()
    finally:
        mf.mf_set_wait_limit_ns(2_000_000_000)
    for got, ref in zip(_bwd(dy, x, gamma, st, mod, resid, ckpt=ckpt), want):
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "act8"])
@pytest.mark.parametrize("hid", [136, 1000, 2048, 3000])
def test_backward_of_constant_rows(hid, ckpt):
    """Rows that hold one value: xhat is what x and the mean leave, 0 from bf16, and not the
    rounding of mean * rstd (up to 0.016 at 300 with an rstd near 1000)."""
    mod = modalities(MIXED)
    T = len(mod)
    rng = np.random.default_rng(hid)
    x = bf16(np.repeat(rng.choice([300.0, -299.0, 87.5, 0.0], (T, 1)), hid, 1))
    xv = oracle.act8_values(*oracle.act8_quantize(x)) if ckpt else _f64(x)
    dy = bf16(rng.standard_normal((T, hid)))
    gamma = np.float32(1 + 0.1 * rng.standard_normal((2, hid)))
    st = np.float32(np.stack([xv[:, 0], np.full(T, 999.4321)], 1))
    dx, dg, db = _bwd(dy, x, gamma, st, mod, ckpt=ckpt)
    rdx, rdg, rdb = oracle.layer_norm_affine_bwd(dy, xv, gamma, st, mod)
    s64 = _f64(st)
    xhat, g = np.abs((xv - s64[:, :1]) * s64[:, 1:]), np.abs(dy * _f64(gamma)[mod])
    # x - mean is exact here, xhat one rounding of it; the row sums are off by at most 64
    # units of their sums of magnitudes, then a few roundings
    m1, m2 = g.mean(1, keepdims=True), (g * xhat).mean(1, keepdims=True)
    check_bf16(dx, rdx, 2.0 ** -24 * s64[:, 1:] * (8 * g + 72 * m1 + 72 * xhat * m2), "dx")
    for got, ref, terms in ((dg, rdg, np.abs(dy) * xhat), (db, rdb, np.abs(dy))):
        mags = np.stack([terms[mod == m].sum(0) for m in (0, 1)])
        assert (np.abs(got - ref) <= (T + 8) * 2.0 ** -24 * mags).all()
    if not ckpt:
        assert (dg == 0).all()

"""The fused modality-specific linear layer and its backward on the GPU (tcgen05),
through the C ABI, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
import resolution_packed_diffusion_b200 as mf
from mlp_util import (ACTS, _f64, bf16, check_bf16, check_rms, dev, dev32, guarded, host, modalities)

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

MIXED = ((1, 9, 14, 5), (0, 0, 0, 33), (1, 14, 9, 2), (1, 3, 3, 1), (1, 1, 9, 60))
# (pack, K, N): single tokens, widths below a tile and past its edge, tiles that hold
# both modalities, runs that end inside a step of 64 tokens, one modality only
CASES = [(((0, 0, 0, 1),), 8, 8), (((1, 1, 1, 0),), 64, 256), (((1, 1, 1, 1),), 72, 264),
         (((0, 0, 0, 16),), 256, 1024), (MIXED, 24, 40), (MIXED, 128, 256), (MIXED, 136, 520),
         (MIXED, 200, 248), (((1, 8, 16, 128), (1, 16, 8, 128)), 128, 256),
         (((0, 0, 0, 300), (1, 11, 13, 0)), 320, 256), (((0, 0, 0, 65),), 1000, 136),
         (((1, 25, 41, 0),), 264, 328), (((1, 16, 16, 20), (1, 8, 32, 12)), 512, 128),
         (tuple((1, 1, 3, 2) for _ in range(60)), 96, 304), (((1, 5, 13, 2), (1, 31, 9, 70)), 1040, 776),
         # few rows: both modalities, every padding of the tokens, inner dimensions that
         # are cut over 1 to 8 CTAs and end inside a step, outputs that end inside a tile
         (((1, 3, 5, 2), (0, 0, 0, 7)), 1032, 392), (((1, 8, 8, 64),), 2048, 136),
         (((0, 0, 0, 33), (1, 3, 9, 1)), 4096, 1000), (((0, 0, 0, 1),), 4096, 2048),
         (((1, 2, 2, 4), (1, 1, 1, 1)), 328, 5128), (((1, 7, 17, 8),), 64, 1024),
         (((0, 0, 0, 129),), 512, 256),
         # dW's tokens in parts: of one modality, of both, of many runs; dW in narrow
         # tiles beside dx's
         (((1, 47, 55, 3), (0, 0, 0, 5)), 264, 520),
         (((1, 37, 53, 1901), (1, 11, 13, 77)), 200, 328),
         (tuple((1, 7, 9, 31) for _ in range(40)), 520, 264),
         (((1, 25, 40, 300),), 136, 72)]


def _data(descs, K, N, seed):
    rng = np.random.default_rng(seed)
    mod = modalities(descs)
    T = len(mod)
    return dict(mod=mod, T=T, x=bf16(rng.standard_normal((T, K))),
                W=bf16(rng.standard_normal((2, N, K)) / np.sqrt(K)),
                bias=np.float32(0.3 * rng.standard_normal((2, N))), resid=bf16(rng.standard_normal((T, N))),
                dout=bf16(rng.standard_normal((T, N))), z=bf16(rng.standard_normal((T, N))))


def _sum_slack(x, W, mod, K):
    """fp32 slack of z: K + 2 additions of at most one unit of 2^-23 of sum|terms|."""
    z = oracle.linear_fused(np.abs(x), np.abs(W), None, None, mod, "none")[0]
    return (K + 2) * 2.0 ** -23 * z


def _fwd(descs, d, K, N, act, bias=True, resid=True, keep=(), in_place=False):
    T = d["T"]
    out, oc = guarded((T, N), torch.bfloat16)
    r = dev(d["resid"]) if resid else None
    if in_place:
        out, oc = r, lambda: None
    z, zc = guarded((T, N), torch.bfloat16) if "bf16" in keep else (None, lambda: None)
    z8, z8c = guarded((T, N), torch.int8) if "8bit" in keep else (None, lambda: None)
    zs, zsc = guarded((T, -(-N // 128)), torch.float32) if "8bit" in keep else (None, lambda: None)
    mf.mf_linear_fused(dev(d["x"]), dev(d["W"]), dev32(d["bias"]) if bias else None, r,
                       torch.from_numpy(d["mod"]).cuda(), descs, K, N, ACTS[act], z, z8, zs, out)
    assert mf.mf_get_error() == mf.MF_OK
    for c in (oc, zc, z8c, zsc):
        c()
    return out, z, z8, zs


@pytest.mark.parametrize("k", range(len(CASES)))
def test_forward_every_row(k):
    descs, K, N = CASES[k]
    d = _data(descs, K, N, 40 + k)
    act = ("none", "gelu", "silu")[k % 3]
    bias, resid = k % 2 == 0, k % 4 < 2
    out, z, z8, zs = _fwd(descs, d, K, N, act, bias, resid, keep=("bf16", "8bit"),
                          in_place=resid and k % 8 == 1)
    ref, rz = oracle.linear_fused(d["x"], d["W"], d["bias"] if bias else None,
                                  d["resid"] if resid else None, d["mod"], act)
    slack = _sum_slack(d["x"], d["W"], d["mod"], K) + 2.0 ** -23 * np.abs(rz)
    # |act'| <= 1.13; sigma's own error as in its argument's exponent
    aslack = 1.13 * slack + np.abs(rz) * (np.abs(rz) * (1.6 + 0.0714 * rz * rz) + 8) * 2.0 ** -22
    check_bf16(host(out), ref, aslack + 2.0 ** -23 * np.abs(ref), "out")
    check_bf16(host(z), rz, slack, "z")
    # the checkpoint: the fp32 z within half a step of a code, whichever way slack goes
    got = oracle.act8_values(z8.cpu().numpy(), zs.cpu().numpy())
    step = _f64(zs.cpu().numpy())[:, np.arange(N) // 128]
    assert (np.abs(got - rz) <= 0.5 * step * (1 + 2.0 ** -14) + slack).all()
    blocks = [np.abs(rz[:, b:b + 128]).max(1) for b in range(0, N, 128)]
    tol = [slack[:, b:b + 128].max(1) / 127 for b in range(0, N, 128)]
    assert (np.abs(zs.cpu().numpy() - np.stack(blocks, 1) / 127) <=
            np.stack(tol, 1) + 2.0 ** -22 * np.stack(blocks, 1)).all()


# Widths of the column tiles from 144 to 240, and 256 in four rounds, over a pack whose row
# blocks hold both modalities (14 jobs for the 74 pairs of SMs): (K, N, columns of a tile)
WIDTHS = [(72, 1328, 144), (136, 1488, 160), (64, 2640, 176), (200, 2648, 192), (1000, 2056, 208),
          (136, 3128, 224), (520, 1128, 240), (40, 3848, 256)]


@pytest.mark.parametrize("keep", [(), ("bf16",)], ids=["out", "z"])
@pytest.mark.parametrize("k", range(len(WIDTHS)))
def test_forward_column_widths(k, keep):
    """One to four rounds of tiles whose width is no power of two: bias, residual and
    every row, with and without the pre-activation."""
    descs, (K, N, _) = ((1, 31, 33, 7), (1, 17, 91, 45), (0, 0, 0, 129)), WIDTHS[k]
    d = _data(descs, K, N, 200 + k)
    act = ("silu", "none", "gelu")[k % 3]
    out, z, _, _ = _fwd(descs, d, K, N, act, keep=keep, in_place=k % 2 == 1)
    ref, rz = oracle.linear_fused(d["x"], d["W"], d["bias"], d["resid"], d["mod"], act)
    slack = _sum_slack(d["x"], d["W"], d["mod"], K) + 2.0 ** -23 * np.abs(rz)
    aslack = 1.13 * slack + np.abs(rz) * (np.abs(rz) * (1.6 + 0.0714 * rz * rz) + 8) * 2.0 ** -22
    check_bf16(host(out), ref, aslack + 2.0 ** -23 * np.abs(ref), "out")
    if keep:
        check_bf16(host(z), rz, slack, "z")


def test_forward_variants_agree():
    """What is kept beside the output does not change it, and calls repeat bit for bit."""
    descs, K, N = MIXED, 192, 392
    d = _data(descs, K, N, 3)
    outs = [_fwd(descs, d, K, N, "gelu", keep=k)[0] for k in ((), ("bf16",), ("8bit",), ("bf16", "8bit"))]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert torch.equal(_fwd(descs, d, K, N, "gelu", in_place=True)[0], outs[0])


def test_forward_matches_the_plain_linear_layer():
    """Without an epilogue: the layer the framework had, to its rounding."""
    descs, K, N = ((1, 16, 16, 20), (1, 8, 32, 12)), 192, 512
    d = _data(descs, K, N, 4)
    out = _fwd(descs, d, K, N, "none", bias=False, resid=False)[0]
    old = torch.empty_like(out)
    mf.mf_modality_linear(dev(d["x"]), dev(d["W"]), torch.from_numpy(d["mod"]).cuda(), descs, K, N, old)
    ref = oracle.linear_fused(d["x"], d["W"], None, None, d["mod"], "none")[0]
    slack = _sum_slack(d["x"], d["W"], d["mod"], K)
    check_bf16(host(out), ref, slack, "fused")
    check_bf16(host(old), ref, slack, "plain")


def _code(a):
    q, s = oracle.act8_quantize(a)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), oracle.act8_values(q, s)


def _bwd(descs, d, K, N, act, x8=False, z8=False, want=("dx", "dW", "db"), x=None, dout=None, z=None):
    T = d["T"]
    xt, zt = dev(d["x"]) if x is None else x, dev(d["z"]) if z is None else z
    gt = dev(d["dout"]) if dout is None else dout
    xq = xs = zq = zs = None
    if x8:
        xq, xs, _ = _code(d["x"])
        xt = None
    if act == "none":
        zt = None
    elif z8:
        zq, zs, _ = _code(d["z"])
        zt = None
    dx, dxc = guarded((T, K), torch.bfloat16)
    dW = torch.full((2, N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    db = torch.full((2, N), float("nan"), device="cuda")
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    mf.mf_linear_fused_bwd(gt, xt, xq, xs, dev(d["W"]), zt, zq, zs, torch.from_numpy(d["mod"]).cuda(),
                           descs, K, N, ACTS[act], dx if "dx" in want else None,
                           dW if "dW" in want else None, db if "db" in want else None, ws, n)
    assert mf.mf_get_error() == mf.MF_OK
    dxc()
    return dx, dW, db


@pytest.mark.parametrize("x8", [False, True], ids=["x", "x8"])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_backward(k, x8):
    descs, K, N = CASES[k]
    d = _data(descs, K, N, 70 + k)
    act = ("gelu", "none", "silu")[k % 3]
    z8 = k % 2 == 1
    dx, dW, db = _bwd(descs, d, K, N, act, x8, z8)
    xv = _code(d["x"])[2] if x8 else _f64(d["x"])
    zv = _code(d["z"])[2] if z8 else _f64(d["z"])
    rdx, rdW, rdb, dz = oracle.linear_fused_bwd(d["dout"], xv, d["W"], zv, d["mod"], act)
    # act' is off by a few units plus the exponent's, relative to |dout| (1 + |w|)
    w = np.abs(zv) * (1.6 + 0.0714 * zv * zv)
    dz_slack = 0 if act == "none" else np.abs(d["dout"]) * (2 + w) * (w + 8) * 2.0 ** -22
    adz = np.abs(dz) + dz_slack
    # the operands' roundings: dz to bf16 (2^-8; exact without an activation), an
    # 8-bit x to bf16; then a sum of n terms in fp32
    op = 0.0 if act == "none" else 2.0 ** -8
    ox = 2.0 ** -8 if x8 else 0.0
    adx, adW, _, _ = oracle.linear_fused_bwd(adz, np.abs(xv), np.abs(d["W"]), None, d["mod"], "none")
    sdx, sdW, sdb, _ = oracle.linear_fused_bwd(dz_slack + 0 * adz, np.abs(xv), np.abs(d["W"]), None,
                                               d["mod"], "none")
    T = d["T"]
    check_bf16(host(dx), rdx, adx * (op + (N + 2) * 2.0 ** -23) + sdx, "dx")
    check_bf16(host(dW), rdW, adW * (op + ox + op * ox + (T + 64) * 2.0 ** -23) + sdW, "dW")
    mags = np.stack([adz[d["mod"] == m].sum(0) for m in (0, 1)])
    assert (np.abs(host(db) - rdb) <= (T + 8) * 2.0 ** -24 * mags + sdb).all()
    if T * N > 1000:
        check_rms(host(dx), rdx, 1 + (act != "none"), "dx")
        check_rms(host(dW), rdW, 1 + (act != "none") + x8, "dW")
    for m in (0, 1):
        if not (d["mod"] == m).any():
            assert (dW[m] == 0).all() and (db[m] == 0).all()


@pytest.mark.parametrize("want", [("dx",), ("dW",), ("db",), ("dx", "db"), ("dW", "db")])
def test_backward_parts_agree_with_the_whole(want):
    descs, K, N = MIXED, 160, 264
    d = _data(descs, K, N, 9)
    whole = dict(zip(("dx", "dW", "db"), _bwd(descs, d, K, N, "gelu", x8=True)))
    part = dict(zip(("dx", "dW", "db"), _bwd(descs, d, K, N, "gelu", x8=True, want=want)))
    for name in want:
        assert torch.equal(part[name], whole[name]), name


@pytest.mark.parametrize("x8", [False, True], ids=["x", "x8"])
def test_foreign_rows_do_not_leak(x8):
    """Infinities and NaN in the text rows: image outputs and gradients unchanged."""
    descs, K, N = MIXED, 144, 264
    d = _data(descs, K, N, 13)
    image = torch.from_numpy(d["mod"] == 0).cuda()
    clean = _bwd(descs, d, K, N, "silu", x8)
    dirty = dict(d)
    for name, bad in (("x", np.nan), ("dout", np.inf), ("z", np.nan)):
        a = d[name].copy()
        a[d["mod"] == 1] = bad
        dirty[name] = a
    xt, gt, zt = (torch.from_numpy(dirty[n]).cuda().to(torch.bfloat16) for n in ("x", "dout", "z"))
    if x8:
        got = _bwd(descs, dirty, K, N, "silu", x8, dout=gt, z=zt)
    else:
        got = _bwd(descs, d, K, N, "silu", x=xt, dout=gt, z=zt)
    assert torch.equal(got[0][image], clean[0][image])
    assert torch.equal(got[1][0], clean[1][0]) and torch.equal(got[2][0], clean[2][0])
    out = _fwd(descs, d, K, N, "silu", resid=False)[0]
    bad = torch.empty_like(out)
    mf.mf_linear_fused(xt, dev(d["W"]), dev32(d["bias"]), None, torch.from_numpy(d["mod"]).cuda(), descs,
                       K, N, mf.MF_ACT_SILU, None, None, None, bad)
    assert torch.equal(bad[image], out[image]) and not torch.isfinite(bad[~image].float()).any()


def test_foreign_weights_do_not_leak():
    """NaN in the text weights: image rows unchanged, at widths that end inside a tile."""
    descs, K, N = MIXED, 72, 136
    d = _data(descs, K, N, 14)
    image = torch.from_numpy(d["mod"] == 0).cuda()
    out, dx = _fwd(descs, d, K, N, "none")[0], _bwd(descs, d, K, N, "none")[0]
    W = dev(d["W"])
    W[1] = float("nan")
    T = d["T"]
    o2, g2 = torch.empty_like(out), torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    tm = torch.from_numpy(d["mod"]).cuda()
    mf.mf_linear_fused(dev(d["x"]), W, dev32(d["bias"]), dev(d["resid"]), tm, descs, K, N, 0, None, None,
                       None, o2)
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    mf.mf_linear_fused_bwd(dev(d["dout"]), None, None, None, W, None, None, None, tm, descs, K, N, 0, g2,
                           None, None, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert torch.equal(o2[image], out[image]) and torch.equal(g2[image], dx[image])


def test_nan_pre_activation_marks_its_block():
    descs, K, N = ((0, 0, 0, 5),), 64, 264
    d = _data(descs, K, N, 15)
    x = dev(d["x"])
    x[2, 3] = float("nan")
    tm = torch.from_numpy(d["mod"]).cuda()
    out = torch.empty((5, N), dtype=torch.bfloat16, device="cuda")
    z8 = torch.empty((5, N), dtype=torch.int8, device="cuda")
    zs = torch.empty((5, 3), device="cuda")
    mf.mf_linear_fused(x, dev(d["W"]), None, None, tm, descs, K, N, 1, None, z8, zs, out)
    assert torch.isnan(zs[2]).all() and torch.isfinite(zs[[0, 1, 3, 4]]).all()
    assert (z8[2] == 0).all() and torch.isnan(out[2].float()).all()
    assert torch.isfinite(out[[0, 1, 3, 4]].float()).all()


def test_no_tokens():
    descs = ((0, 0, 0, 0),)
    mf.mf_linear_fused(None, None, None, None, None, descs, 64, 64, 0, None, None, None, None)
    dW = torch.full((2, 64, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    db = torch.full((2, 64), 3.0, device="cuda")
    mf.mf_linear_fused_bwd(None, None, None, None, None, None, None, None, None, descs, 64, 64, 0, None,
                           dW, db, None, 0)
    assert (dW == 0).all() and (db == 0).all()


def test_graph_replay_and_two_streams():
    """A captured forward and backward replayed on new inputs, and two streams with
    their own buffers at once."""
    descs, K, N = MIXED, 256, 520
    a, b = _data(descs, K, N, 21), _data(descs, K, N, 22)
    T = a["T"]
    tm = torch.from_numpy(a["mod"]).cuda()
    arr = mf.make_descs(descs)
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)

    def buffers(d):
        e = dict(x=dev(d["x"]), W=dev(d["W"]), b=dev32(d["bias"]), g=dev(d["dout"]),
                 out=torch.zeros((T, N), dtype=torch.bfloat16, device="cuda"),
                 z8=torch.zeros((T, N), dtype=torch.int8, device="cuda"),
                 zs=torch.zeros((T, 5), device="cuda"),
                 dx=torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"),
                 dW=torch.zeros((2, N, K), dtype=torch.bfloat16, device="cuda"),
                 db=torch.zeros((2, N), device="cuda"), ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
        return e

    def step(e):
        mf.mf_linear_fused(e["x"], e["W"], e["b"], None, tm, arr, K, N, 1, None, e["z8"], e["zs"], e["out"])
        mf.mf_linear_fused_bwd(e["g"], e["x"], None, None, e["W"], None, e["z8"], e["zs"], tm, arr, K, N, 1,
                               e["dx"], e["dW"], e["db"], e["ws"], n)

    names = ("out", "z8", "zs", "dx", "dW", "db")
    ea, eb = buffers(a), buffers(b)
    step(ea)
    step(eb)
    torch.cuda.synchronize()
    want_a, want_b = ([e[k].clone() for k in names] for e in (ea, eb))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, e in zip(streams, (ea, eb)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step(e)
    torch.cuda.synchronize()
    for k, w in zip(names, want_a):
        assert torch.equal(ea[k], w), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        step(ea)
    for k in ("x", "W", "b", "g"):
        ea[k].copy_(eb[k])
    graph.replay()
    torch.cuda.synchronize()
    for k, w in zip(names, want_b):
        assert torch.equal(ea[k], w), k
    assert mf.mf_get_error() == mf.MF_OK


def test_offsets_past_32_bits():
    """2^31 + output elements: the last rows against the oracle."""
    T, K, N = 131072, 16, 16400
    rng = np.random.default_rng(31)
    descs = ((1, 256, 511, 256),)
    mod = modalities(descs)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    tail = bf16(rng.standard_normal((300, K)))
    x[-300:] = dev(tail)
    W = bf16(rng.standard_normal((2, N, K)) / 4)
    out = torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda")
    z8 = torch.empty((T, N), dtype=torch.int8, device="cuda")
    zs = torch.empty((T, -(-N // 128)), device="cuda")
    tm = torch.from_numpy(mod).cuda()
    mf.mf_linear_fused(x, dev(W), None, None, tm, descs, K, N, 0, None, z8, zs, out)
    ref = oracle.linear_fused(tail, W, None, None, mod[-300:], "none")[0]
    check_bf16(host(out[-300:]), ref, _sum_slack(tail, W, mod[-300:], K), "tail")
    assert (out[: T - 300] == 0).all() and (zs[: T - 300] == 0).all()
    # backward: dout is zero but for the last rows, so dW is theirs alone
    out.zero_()
    dtail = bf16(rng.standard_normal((300, N)))
    out[-300:] = dev(dtail)
    del z8, zs
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dW = torch.empty((2, N, K), dtype=torch.bfloat16, device="cuda")
    db = torch.empty((2, N), device="cuda")
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    mf.mf_linear_fused_bwd(out, x, None, None, dev(W), None, None, None, tm, descs, K, N, 0, dx, dW, db,
                           torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert mf.mf_get_error() == mf.MF_OK
    rdx, rdW, rdb, _ = oracle.linear_fused_bwd(dtail, tail, W, None, mod[-300:], "none")
    adx, adW, adb, _ = oracle.linear_fused_bwd(np.abs(dtail), np.abs(tail), np.abs(W), None, mod[-300:], "none")
    check_bf16(host(dx[-300:]), rdx, adx * (N + 2) * 2.0 ** -23, "dx")
    check_bf16(host(dW), rdW, adW * 400 * 2.0 ** -23, "dW")
    assert (np.abs(host(db) - rdb) <= 400 * 2.0 ** -24 * adb).all()


@pytest.mark.parametrize("descs,K,N", [(MIXED, 256, 512), (((0, 0, 0, 40),), 256, 512)])
def test_tensors_on_16_byte_boundaries(descs, K, N):
    """The least alignment the library asks for gives the same bits."""
    d = _data(descs, K, N, 51)
    T = d["T"]
    want = _fwd(descs, d, K, N, "gelu", keep=("bf16", "8bit"))
    grads = _bwd(descs, d, K, N, "gelu", x8=True)

    def off(t):
        size = t.element_size()
        v = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")[16 // size:][: t.numel()].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    got = [off(torch.zeros_like(t)) for t in want]
    tm = torch.from_numpy(d["mod"]).cuda()
    W = off(dev(d["W"]))
    mf.mf_linear_fused(off(dev(d["x"])), W, off(dev32(d["bias"])), off(dev(d["resid"])), tm, descs, K, N,
                       mf.MF_ACT_GELU, got[1], got[2], got[3], got[0])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    xq, xs, _ = _code(d["x"])
    dx, dW, db = (off(torch.zeros_like(t)) for t in grads)
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    mf.mf_linear_fused_bwd(off(dev(d["dout"])), None, off(xq), off(xs), W, off(dev(d["z"])), None, None, tm,
                           descs, K, N, mf.MF_ACT_GELU, dx, dW, db,
                           torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    for a, b in zip((dx, dW, db), grads):
        assert torch.equal(a, b)


def test_two_calls_in_a_row_into_the_same_buffers():
    """The second call of a stream overwrites what the first wrote, few rows and many."""
    for descs, K, N in ((((0, 0, 0, 24),), 512, 1024), (MIXED, 128, 264)):
        a, b = _data(descs, K, N, 61), _data(descs, K, N, 62)
        tm = torch.from_numpy(a["mod"]).cuda()
        out = torch.empty((a["T"], N), dtype=torch.bfloat16, device="cuda")
        xs = [dev(a["x"]), dev(b["x"])]
        W = dev(a["W"])
        want = torch.empty_like(out)
        mf.mf_linear_fused(xs[1], W, None, None, tm, descs, K, N, 2, None, None, None, want)
        torch.cuda.synchronize()
        for _ in range(10):
            for x in xs:
                mf.mf_linear_fused(x, W, None, None, tm, descs, K, N, 2, None, None, None, out)
        assert torch.equal(out, want)


def test_weight_sums_cut_over_the_tokens():
    """A narrow layer over many tokens: the token axis in parts, joined in order."""
    descs, K, N = ((1, 64, 80, 333), (1, 37, 41, 2001)), 72, 136
    d = _data(descs, K, N, 71)
    dx, dW, db = _bwd(descs, d, K, N, "none")
    _, rdW, rdb, dz = oracle.linear_fused_bwd(d["dout"], d["x"], d["W"], None, d["mod"], "none")
    _, adW, _, _ = oracle.linear_fused_bwd(np.abs(dz), np.abs(d["x"]), np.abs(d["W"]), None, d["mod"], "none")
    check_bf16(host(dW), rdW, adW * (d["T"] + 64) * 2.0 ** -23, "dW")
    mags = np.stack([np.abs(dz)[d["mod"] == m].sum(0) for m in (0, 1)])
    assert (np.abs(host(db) - rdb) <= (d["T"] + 8) * 2.0 ** -24 * mags).all()
    again = _bwd(descs, d, K, N, "none")
    assert torch.equal(again[1], dW) and torch.equal(again[2], db)


NAN_PACKS = {"few rows": ((1, 3, 5, 2), (0, 0, 0, 23)), "many rows": MIXED}


@pytest.mark.parametrize("n0", [6, 133])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("pack", list(NAN_PACKS))
def test_a_nan_channel_stays_alone(pack, act, n0):
    """A NaN in one channel's bias, weights or pre-activation: every other channel, the
    one beside it too, as it would be."""
    descs, K, N = NAN_PACKS[pack], 72, 264
    d = _data(descs, K, N, 81)
    T, mod = d["T"], d["mod"]
    others = np.arange(N) != n0
    ref, rz = oracle.linear_fused(d["x"], d["W"], d["bias"], d["resid"], mod, act)
    slack = _sum_slack(d["x"], d["W"], mod, K) + 2.0 ** -23 * np.abs(rz)
    aslack = 1.13 * slack + np.abs(rz) * (np.abs(rz) * (1.6 + 0.0714 * rz * rz) + 8) * 2.0 ** -22
    aslack += 2.0 ** -23 * np.abs(ref)
    text, tm = mod == 1, torch.from_numpy(mod).cuda()
    for where in ("bias", "weights"):
        W, bias = dev(d["W"]), dev32(d["bias"])
        if where == "bias":
            bias[1, n0] = float("nan")
        else:
            W[1, n0, 3] = float("nan")
        out, z = (torch.empty((T, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mf.mf_linear_fused(dev(d["x"]), W, bias, dev(d["resid"]), tm, descs, K, N, ACTS[act], z, None, None, out)
        got = host(out)
        assert np.isnan(got[text, n0]).all() and np.isnan(host(z)[text, n0]).all(), where
        check_bf16(got[:, others], ref[:, others], aslack[:, others], f"out, {where}")
        check_bf16(got[~text, n0], ref[~text, n0], aslack[~text, n0], f"image rows, {where}")

    # backward: one NaN pre-activation in a text row
    t0 = int(np.flatnonzero(text)[-1])
    rdx, rdW, rdb, dz = oracle.linear_fused_bwd(d["dout"], d["x"], d["W"], d["z"], mod, act)
    zt = dev(d["z"])
    zt[t0, n0] = float("nan")
    dx, dW, db = (host(t) for t in _bwd(descs, d, K, N, act, z=zt))
    assert np.isnan(dx[t0]).all() and np.isnan(dW[1, n0]).all() and np.isnan(db[1, n0])
    w = np.abs(d["z"]) * (1.6 + 0.0714 * d["z"] ** 2)
    dz_slack = np.abs(d["dout"]) * (2 + w) * (w + 8) * 2.0 ** -22
    adz = np.abs(dz) + dz_slack
    adx, adW, adb, _ = oracle.linear_fused_bwd(adz, np.abs(d["x"]), np.abs(d["W"]), None, mod, "none")
    sdx, sdW, sdb, _ = oracle.linear_fused_bwd(dz_slack, np.abs(d["x"]), np.abs(d["W"]), None, mod, "none")
    rows = np.arange(T) != t0
    check_bf16(dx[rows], rdx[rows], (adx * (2.0 ** -8 + (N + 2) * 2.0 ** -23) + sdx)[rows], "dx")
    tol = adW * (2.0 ** -8 + (T + 64) * 2.0 ** -23) + sdW
    check_bf16(dW[0], rdW[0], tol[0], "dW of the image")
    check_bf16(dW[1, others], rdW[1, others], tol[1, others], "dW of the text")
    tol = (T + 8) * 2.0 ** -24 * adb + sdb
    assert (np.abs(db - rdb)[0] <= tol[0]).all() and (np.abs(db - rdb)[1, others] <= tol[1, others]).all()


@pytest.mark.parametrize("mixed", [False, True], ids=["in_order", "mixed"])
@pytest.mark.parametrize("z8", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activation_gradient_to_fp32_at_every_magnitude(act, z8, mixed):
    """db of one token with dout = 1 is act'(z) in fp32, from -100 to 100. In units u =
    2^-24, with sigma = 1 / (1 + e), e = 2^v, act' = sigma + z w' e sigma^2: v is a
    product of four roundings (4u), 2^v is good to 4u (its instruction) and 4u |v| ln 2,
    1 + e to u beside e's, its reciprocal, shared by two values, to 4u. Beyond the ends
    of the range where act' is held it is within 1e-15 of its limits."""
    z = np.concatenate([np.linspace(-100, 100, 1024), np.linspace(-10, 10, 1536), np.linspace(6, 45, 384)])
    if mixed:  # small and large ones side by side
        z = np.random.default_rng(11).permutation(z)
    z = bf16(z.astype(np.float32))[None, :]
    N, u = z.shape[1], 2.0 ** -24
    tm = torch.zeros(1, dtype=torch.uint8, device="cuda")
    ones = torch.ones((1, N), dtype=torch.bfloat16, device="cuda")
    zt = zq = zs = None
    zv = _f64(z)
    if z8:
        zq, zs, zv = _code(z)
    else:
        zt = dev(z)
    db = torch.empty((2, N), device="cuda")
    n = mf.mf_linear_fused_bwd_workspace_size(1, 8, N)
    mf.mf_linear_fused_bwd(ones, None, None, None, None, zt, zq, zs, tm, ((1, 1, 1, 0),), 8, N, ACTS[act],
                           None, None, db, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert mf.mf_get_error() == mf.MF_OK and (db[1] == 0).all()
    c1, c3 = (2 * np.sqrt(2 / np.pi), 2 * np.sqrt(2 / np.pi) * 0.044715) if act == "gelu" else (1.0, 0.0)
    w = zv * (c1 + c3 * zv * zv)
    s = 1 / (1 + np.exp(-np.clip(w, -700, 700)))
    e = 4 * u * np.abs(w) + 4 * u
    es = (1 - s) * e + 5 * u
    ref = oracle.mlp_act_grad(zv, act)
    zw = np.abs(zv * (c1 + 3 * c3 * zv * zv))
    turn = zw * s * (1 - s)
    tol = 1.01 * (s * es + turn * (e + 2 * es + 6 * u) + u * np.abs(ref)) + 1e-15
    # the oracle's own: tanh is rounded by 2^-54 just below 1, 1 - tanh^2 so by 2^-53
    # beside its own rounding, and it enters times z w' / 2
    tol = tol + 2.0 ** -53 * zw
    err = np.abs(host(db)[0] - ref[0])
    i = int(np.argmax(err - tol[0]))
    assert err[i] <= tol[0, i], f"z {zv[0, i]}: off by {err[i]:.3g}, tolerance {tol[0, i]:.3g}"


@pytest.mark.parametrize("descs", [tuple((1, 1, 1, 1) for _ in range(n)) for n in (23, 24, 25, 48, 49, 130, 512)]
                         + [tuple((1, 1, 65, 66) for _ in range(256)), ((1, 12, 64, 769),), ((0, 0, 0, 1537),)])
def test_backward_stays_in_its_workspace(descs):
    """Packs with the most steps for their tokens, around the first that has dW in parts:
    exactly the bytes asked for, with a pattern behind them."""
    K, N = 8, 264
    d = _data(descs, K, N, 91)
    T, n = d["T"], mf.mf_linear_fused_bwd_workspace_size(d["T"], K, N)
    ws = torch.full((n + (48 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    dx = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    dW = torch.empty((2, N, K), dtype=torch.bfloat16, device="cuda")
    db = torch.empty((2, N), device="cuda")
    xq, xs, xv = _code(d["x"])
    mf.mf_linear_fused_bwd(dev(d["dout"]), None, xq, xs, dev(d["W"]), None, None, None,
                           torch.from_numpy(d["mod"]).cuda(), descs, K, N, 0, dx, dW, db, ws, n)
    assert mf.mf_get_error() == mf.MF_OK
    assert (ws[n:] == 0x5A).all(), "bytes behind the workspace were written"
    rdx, rdW, rdb, dz = oracle.linear_fused_bwd(d["dout"], xv, d["W"], None, d["mod"], "none")
    adx, adW, adb, _ = oracle.linear_fused_bwd(np.abs(dz), np.abs(xv), np.abs(d["W"]), None, d["mod"], "none")
    check_bf16(host(dx), rdx, adx * (N + 2) * 2.0 ** -23, "dx")
    check_bf16(host(dW), rdW, adW * (2.0 ** -8 + (T + 64) * 2.0 ** -23), "dW")
    assert (np.abs(host(db) - rdb) <= (T + 8) * 2.0 ** -24 * adb).all()

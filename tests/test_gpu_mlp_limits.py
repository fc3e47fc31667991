"""The MLP-branch operators at the ends of what their documentation allows: the widest
layers, a single wide row, gradients asked for one by one over few rows, rows without a
valid modality, and a first call inside a capture."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import resolution_packed_diffusion_b200 as mf
from mlp_util import bf16, check_bf16, check_rms, dev, dev32, guarded, host, modalities

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


@pytest.mark.parametrize("descs", [((1, 1, 1, 2),), ((1, 9, 13, 20),)], ids=["few_rows", "many_rows"])
@pytest.mark.parametrize("K,N", [(1 << 20, 8), (8, 1 << 20)])
def test_widest_layers(K, N, descs):
    """2^20 channels on either side, against torch in 64 bits."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K + len(descs))
    mod = modalities(descs)
    T = len(mod)
    x, W, g = _randn(gen, T, K), _randn(gen, 2, N, K, scale=K ** -0.5), _randn(gen, T, N)
    tm = torch.from_numpy(mod).cuda()
    out, dx, dW = torch.empty_like(g), torch.empty_like(x), torch.empty_like(W)
    db = torch.empty((2, N), device="cuda")
    mf.mf_linear_fused(x, W, None, None, tm, descs, K, N, mf.MF_ACT_NONE, None, None, None, out)
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    mf.mf_linear_fused_bwd(g, x, None, None, W, None, None, None, tm, descs, K, N, mf.MF_ACT_NONE, dx, dW,
                           db, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert mf.mf_get_error() == mf.MF_OK
    for m in (0, 1):
        rows = tm == m
        xm, gm, Wm = x[rows].double(), g[rows].double(), W[m].double()
        for got, ref, name in ((out[rows], xm @ Wm.T, "out"), (dx[rows], gm @ Wm, "dx"), (dW[m], gm.T @ xm, "dW")):
            got, ref = host(got), ref.cpu().numpy()
            if got.size > 1000:
                check_rms(got, ref, 1, name)
            else:
                # too few outputs for a mean of roundings: each is off by at most 2^-8 of
                # its value, and the 2^17 / 16 additions of one part by 2^-23 each of a sum
                # about as large as the result: 2^-10
                assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2.0 ** -10) * np.linalg.norm(ref), name
        mags = gm.abs().sum(0).cpu().numpy()
        assert (np.abs(host(db[m]) - gm.sum(0).cpu().numpy()) <= (T + 8) * 2.0 ** -24 * mags).all()


@pytest.mark.parametrize("T", [1, 2, 3, 5])
@pytest.mark.parametrize("hid", [1032, 2056, 4096, 8192])
@pytest.mark.parametrize("ckpt", [False, True], ids=["bf16", "act8"])
def test_layer_norm_backward_of_a_few_wide_rows(T, hid, ckpt):
    rng = np.random.default_rng(T + hid)
    mod = (np.arange(T) % 2).astype(np.uint8)
    x, dy, resid = (bf16(rng.standard_normal((T, hid))) for _ in range(3))
    gamma = np.float32(1 + 0.1 * rng.standard_normal((2, hid)))
    q, s = oracle.act8_quantize(x)
    xv = oracle.act8_values(q, s) if ckpt else np.float64(x)
    _, mean, rstd = oracle.layer_norm_affine(xv, gamma, gamma, mod, 1e-6)
    st = np.float32(np.stack([mean, rstd], 1))
    dx, check = guarded((T, hid), torch.bfloat16)
    dg, db = torch.empty((2, hid), device="cuda"), torch.empty((2, hid), device="cuda")
    n = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    form = (None, torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()) if ckpt else (dev(x), None, None)
    mf.mf_layer_norm_bwd(dev(dy), *form, dev32(gamma), dev32(st), torch.from_numpy(mod).cuda(), dev(resid),
                         T, hid, dx, dg, db, torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    assert mf.mf_get_error() == mf.MF_OK
    check()
    rdx, rdg, rdb = oracle.layer_norm_affine_bwd(dy, xv, gamma, st, mod, resid)
    # |x|, |xhat|, |dy gamma| <= 8 here: the units of a row's terms and sums stay below 2^-14
    check_bf16(host(dx), rdx, 2.0 ** -14, "dx")
    np.testing.assert_allclose(host(dg), rdg, rtol=0, atol=2.0 ** -16)
    np.testing.assert_allclose(host(db), rdb, rtol=0, atol=2.0 ** -18)
    if T == 1:
        assert (dg[1] == 0).all() and (db[1] == 0).all()


@pytest.mark.parametrize("want", [("dx",), ("dW",), ("db",), ("dx", "db"), ("dx", "dW"), ("dW", "db")])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_gradients_one_by_one_over_few_rows(act, want):
    """100 tokens: dx has a kernel of its own here, and db one where no product follows."""
    descs, K, N = ((1, 5, 9, 11), (0, 0, 0, 44)), 136, 264
    mod = modalities(descs)
    T = len(mod)
    rng = np.random.default_rng(5)
    x, g, z = (dev(bf16(rng.standard_normal((T, c)))) for c in (K, N, N))
    W, tm = dev(bf16(rng.standard_normal((2, N, K)) / 12)), torch.from_numpy(mod).cuda()
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    code = {"none": mf.MF_ACT_NONE, "silu": mf.MF_ACT_SILU}[act]

    def call(names):
        o = dict(dx=torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda"),
                 dW=torch.full((2, N, K), 7.0, dtype=torch.bfloat16, device="cuda"),
                 db=torch.full((2, N), 7.0, device="cuda"))
        mf.mf_linear_fused_bwd(g, x if "dW" in names else None, None, None, W if "dx" in names else None,
                               None if act == "none" else z, None, None, tm, descs, K, N, code,
                               *(o[k] if k in names else None for k in ("dx", "dW", "db")),
                               torch.empty(n, dtype=torch.uint8, device="cuda"), n)
        assert mf.mf_get_error() == mf.MF_OK
        return o

    whole, part = call(("dx", "dW", "db")), call(want)
    for k in part:
        assert torch.equal(part[k], whole[k]) if k in want else (part[k] == 7.0).all(), k


@pytest.mark.parametrize("descs", [((1, 3, 5, 2), (0, 0, 0, 23)), ((1, 9, 14, 5), (0, 0, 0, 233))],
                         ids=["few_rows", "many_rows"])
def test_rows_without_a_modality_are_left_alone(descs):
    K, N, bad = 72, 264, 4
    mod = modalities(descs)
    T = len(mod)
    rng = np.random.default_rng(6)
    x, g = dev(bf16(rng.standard_normal((T, K)))), dev(bf16(rng.standard_normal((T, N))))
    W, good = dev(bf16(rng.standard_normal((2, N, K)) / 8)), torch.from_numpy(mod).cuda()
    tm = good.clone()
    tm[bad] = 2
    rest = torch.arange(T, device="cuda") != bad

    def fwd(m):
        o = [torch.full((T, N), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        q, s = torch.full((T, N), 9, dtype=torch.int8, device="cuda"), torch.full((T, 3), 9.0, device="cuda")
        mf.mf_linear_fused(x, W, None, None, m, descs, K, N, mf.MF_ACT_GELU, o[1], q, s, o[0])
        return o + [q, s]

    for got, ref in zip(fwd(tm), fwd(good)):
        assert torch.equal(got[rest], ref[rest]) and (got[bad] == 9).all()
    assert mf.mf_get_error() == mf.MF_OK
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    ws, res = torch.empty(n, dtype=torch.uint8, device="cuda"), []
    for m, status in ((good, mf.MF_OK), (tm, mf.MF_ERR_INVALID)):
        dx = torch.full((T, K), 9.0, dtype=torch.bfloat16, device="cuda")
        db = torch.empty((2, N), device="cuda")
        mf.mf_linear_fused_bwd(g, None, None, None, W, None, None, None, m, descs, K, N, 0, dx, None, db, ws, n)
        assert mf.mf_get_error() == status
        res.append(dx)
    assert torch.equal(res[1][rest], res[0][rest]) and (res[1][bad] == 9).all()


FIRST_CALL = """
import torch, resolution_packed_diffusion_b200 as mf
T, K, N = {T}, 264, 520
d, tm = mf.make_descs([(0, 0, 0, T)]), torch.ones(T, dtype=torch.uint8, device="cuda")
B = torch.bfloat16
x, W, g = (torch.randn(s, device="cuda").to(B) for s in ((T, K), (2, N, K), (T, N)))
gamma, st = torch.ones((2, K), device="cuda"), torch.tensor([[0.0, 1.0]], device="cuda").repeat(T, 1)
n = max(mf.mf_linear_fused_bwd_workspace_size(T, K, N), mf.mf_layer_norm_bwd_workspace_size(T, K))
ws = torch.empty(n, dtype=torch.uint8, device="cuda")
o = [torch.zeros_like(g), torch.zeros((T, N), dtype=torch.int8, device="cuda"), torch.zeros((T, 5), device="cuda"),
     torch.zeros_like(x), torch.zeros_like(W), torch.zeros((2, N), device="cuda"), torch.zeros_like(x),
     torch.zeros_like(x), torch.zeros((2, K), device="cuda"), torch.zeros((2, K), device="cuda")]
def step():
    mf.mf_linear_fused(x, W, None, None, tm, d, K, N, 1, None, o[1], o[2], o[0])
    mf.mf_linear_fused_bwd(g, x, None, None, W, None, o[1], o[2], tm, d, K, N, 1, o[3], o[4], o[5], ws, n)
    mf.mf_layer_norm(x, gamma, gamma, tm, T, K, 1e-6, o[6], st)
    mf.mf_layer_norm_bwd(o[3], x, None, None, gamma, st, tm, None, T, K, o[7], o[8], o[9], ws, n)
s = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    step()
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in o]
step()
assert mf.mf_get_error() == mf.MF_OK
assert all(torch.equal(a, b) and bool((a != 0).any()) for a, b in zip(o, first))
print("captured first")
"""


@pytest.mark.parametrize("T", [40, 300])
def test_the_first_call_of_a_process_may_be_captured(T):
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(T=T)], cwd=ROOT, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]

"""The MLP-branch operators as a training step uses them: layer norm, up
projection + GELU (pre-activation kept in 8 bits), down projection + residual, and
the backward from 8-bit checkpoints, over a pack of both modalities. Every stage is
held to the fp64 oracle on the stage's own inputs, and the whole to the oracle's
chain without any rounding or quantisation."""

import numpy as np
import pytest
import torch

import oracle
import resolution_packed_diffusion_b200 as mf
from mlp_util import bf16, check_rms, dev, dev32, host, modalities

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

EPS = 1e-6


def _rel(got, ref):
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("descs,hid,F", [(((1, 16, 16, 20), (1, 8, 32, 12)), 128, 512),
                                         (((1, 13, 17, 9), (0, 0, 0, 41), (1, 3, 50, 0)), 264, 1000)])
def test_training_step_of_an_mlp_branch(descs, hid, F):
    rng = np.random.default_rng(hid + F)
    mod = modalities(descs)
    T = len(mod)
    x = bf16(rng.standard_normal((T, hid)))
    gamma, beta = (np.float32(a + 0.1 * rng.standard_normal((2, hid))) for a in (1, 0))
    W1 = bf16(rng.standard_normal((2, F, hid)) / np.sqrt(hid))
    W2 = bf16(rng.standard_normal((2, hid, F)) / np.sqrt(F))
    b1, b2 = np.float32(0.1 * rng.standard_normal((2, F))), np.float32(0.1 * rng.standard_normal((2, hid)))
    dy = bf16(rng.standard_normal((T, hid)))

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def ckpt(C):
        return buf(T, C, dtype=torch.int8), buf(T, -(-C // 128), dtype=torch.float32)

    arr, tm = mf.make_descs(descs), torch.from_numpy(mod).cuda()
    xd, gd, bd, W1d, W2d, b1d, b2d, dyd = (dev(x), dev32(gamma), dev32(beta), dev(W1), dev(W2), dev32(b1),
                                           dev32(b2), dev(dy))
    n = max(mf.mf_layer_norm_bwd_workspace_size(T, hid), mf.mf_linear_fused_bwd_workspace_size(T, hid, F),
            mf.mf_linear_fused_bwd_workspace_size(T, F, hid))
    ws = buf(n, dtype=torch.uint8)
    # forward: what is kept is 8-bit x, x1 and z, and the row statistics
    x1, h, y = buf(T, hid), buf(T, F), buf(T, hid)
    stats = buf(T, 2, dtype=torch.float32)
    (x8, xs), (x18, x1s), (z8, zs) = ckpt(hid), ckpt(hid), ckpt(F)
    mf.mf_layer_norm(xd, gd, bd, tm, T, hid, EPS, x1, stats)
    mf.mf_act8_quantize(xd, T, hid, x8, xs)
    mf.mf_act8_quantize(x1, T, hid, x18, x1s)
    mf.mf_linear_fused(x1, W1d, b1d, None, tm, arr, hid, F, mf.MF_ACT_GELU, None, z8, zs, h)
    mf.mf_linear_fused(h, W2d, b2d, xd, tm, arr, F, hid, mf.MF_ACT_NONE, None, None, None, y)
    # backward
    h2, dh, dx1, dx = buf(T, F), buf(T, F), buf(T, hid), buf(T, hid)
    dW1, dW2 = buf(2, F, hid), buf(2, hid, F)
    db1, db2, dg, dbeta = (buf(2, c, dtype=torch.float32) for c in (F, hid, hid, hid))
    mf.mf_act8_dequantize(z8, zs, T, F, mf.MF_ACT_GELU, h2)
    mf.mf_linear_fused_bwd(dyd, h2, None, None, W2d, None, None, None, tm, arr, F, hid, mf.MF_ACT_NONE, dh,
                           dW2, db2, ws, n)
    mf.mf_linear_fused_bwd(dh, None, x18, x1s, W1d, None, z8, zs, tm, arr, hid, F, mf.MF_ACT_GELU, dx1, dW1,
                           db1, ws, n)
    mf.mf_layer_norm_bwd(dx1, None, x8, xs, gd, stats, tm, dyd, T, hid, dx, dg, dbeta, ws, n)
    assert mf.mf_get_error() == mf.MF_OK

    # stage by stage, on what each stage was given
    ry, _ = oracle.linear_fused(host(h), W2, b2, x, mod, "none")
    check_rms(host(y), ry, 1, "y")
    zv = oracle.act8_values(z8.cpu().numpy(), zs.cpu().numpy())
    check_rms(host(h2), oracle.mlp_act(zv, "gelu"), 1, "h from the checkpoint")
    rdh, rdW2, rdb2, _ = oracle.linear_fused_bwd(dy, host(h2), W2, None, mod, "none")
    check_rms(host(dh), rdh, 1, "dh")
    check_rms(host(dW2), rdW2, 1, "dW2")
    assert _rel(host(db2), rdb2) < 1e-5
    x1v = oracle.act8_values(x18.cpu().numpy(), x1s.cpu().numpy())
    rdx1, rdW1, rdb1, _ = oracle.linear_fused_bwd(host(dh), x1v, W1, zv, mod, "gelu")
    check_rms(host(dx1), rdx1, 2, "dx1")
    check_rms(host(dW1), rdW1, 3, "dW1")
    assert _rel(host(db1), rdb1) < 1e-5
    xv = oracle.act8_values(x8.cpu().numpy(), xs.cpu().numpy())
    rdx, rdg, rdbeta = oracle.layer_norm_affine_bwd(host(dx1), xv, gamma, host(stats), mod, dy)
    check_rms(host(dx), rdx, 1, "dx")
    assert _rel(host(dg), rdg) < 1e-5 and _rel(host(dbeta), rdbeta) < 1e-5

    # the whole against the chain without roundings. An 8-bit value is off by at most
    # half a step, amax / 254 of its block, uniform: RMS amax / (254 sqrt 3), with
    # amax <= 4.5 RMS in blocks of up to 128 normal values: 1.1%. Four such errors (x,
    # x1, z through GELU' and through h) and eight bf16 roundings (0.23% each) meet
    # in a gradient: sqrt(4 * 1.1^2 + 8 * 0.23^2) = 2.3%.
    f1, mean, rstd = oracle.layer_norm_affine(x, gamma, beta, mod, EPS)
    fh, fz = oracle.linear_fused(f1, W1, b1, None, mod, "gelu")
    fy, _ = oracle.linear_fused(fh, W2, b2, x, mod, "none")
    gdh, gdW2, gdb2, _ = oracle.linear_fused_bwd(dy, fh, W2, None, mod, "none")
    gdx1, gdW1, gdb1, _ = oracle.linear_fused_bwd(gdh, f1, W1, fz, mod, "gelu")
    gdx, gdg, gdbeta = oracle.layer_norm_affine_bwd(gdx1, x, gamma, np.stack([mean, rstd], 1), mod, dy)
    check_rms(host(y), fy, 4, "y of the chain")
    for got, ref, name in ((dx, gdx, "dx"), (dW1, gdW1, "dW1"), (dW2, gdW2, "dW2"), (db1, gdb1, "db1"),
                           (db2, gdb2, "db2"), (dg, gdg, "dgamma"), (dbeta, gdbeta, "dbeta")):
        assert _rel(host(got), ref) < 0.023, name


def test_captured_behind_copies_and_joined_streams():
    """A capture in which the operators follow a memset, a copy and a join of two
    streams, replayed on new inputs: every call waits for all that came before it."""
    descs, hid, F = ((1, 9, 14, 5), (0, 0, 0, 133), (1, 14, 9, 2)), 256, 520
    mod = modalities(descs)
    T = len(mod)
    rng = np.random.default_rng(3)
    tm, arr = torch.from_numpy(mod).cuda(), mf.make_descs(descs)
    gamma, beta = dev32(1 + 0.1 * rng.standard_normal((2, hid))), dev32(0.1 * rng.standard_normal((2, hid)))
    W = dev(rng.standard_normal((2, F, hid)) / 16)
    src = [dev(rng.standard_normal((T, hid))) for _ in range(2)]
    inp, x, x1 = (torch.empty_like(src[0]) for _ in range(3))
    q = torch.empty((T, hid), dtype=torch.int8, device="cuda")
    s = torch.empty((T, 2), device="cuda")
    h = torch.empty((T, F), dtype=torch.bfloat16, device="cuda")
    bias = torch.empty((2, F), device="cuda")
    dW = torch.empty_like(W)
    n = mf.mf_linear_fused_bwd_workspace_size(T, hid, F)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        x.copy_(inp)                       # a copy before a call
        mf.mf_layer_norm(x, gamma, beta, tm, T, hid, EPS, x1)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):      # a branch of its own
            bias.zero_()
            bias.add_(x1[0, 0].float())
            mf.mf_act8_quantize(x1, T, hid, q, s)
        mf.mf_linear_fused(x1, W, None, None, tm, arr, hid, F, mf.MF_ACT_SILU, None, None, None, h)
        torch.cuda.current_stream().wait_stream(side)
        mf.mf_linear_fused(x1, W, bias, None, tm, arr, hid, F, mf.MF_ACT_SILU, None, None, None, h)
        mf.mf_linear_fused_bwd(h, None, q, s, None, None, None, None, tm, arr, hid, F, mf.MF_ACT_NONE,
                               None, dW, None, ws, n)

    want = []
    with torch.cuda.stream(main):
        for a in src:
            inp.copy_(a)
            step()
            main.synchronize()
            want.append([t.clone() for t in (x1, q, s, h, dW)])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            step()
        for k in (0, 1, 1, 0):
            inp.copy_(src[k])
            graph.replay()
            main.synchronize()
            for got, ref in zip((x1, q, s, h, dW), want[k]):
                assert torch.equal(got, ref)
    assert mf.mf_get_error() == mf.MF_OK

"""Activation checkpoints in 8 bits on the GPU: codes and scales equal the fp32
definition bit for bit, values read back within one bf16 rounding."""

import numpy as np
import pytest
import torch

import oracle
import resolution_packed_diffusion_b200 as mf
from mlp_util import ACTS, bf16, check_bf16, dev, guarded, host

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _quantize(x):
    T, C = x.shape
    q, qc = guarded((T, C), torch.int8)
    s, sc = guarded((T, -(-C // 128)), torch.float32)
    mf.mf_act8_quantize(dev(x), T, C, q, s)
    torch.cuda.synchronize()
    qc()
    sc()
    return q, s


SIZES = [(1, 8), (1, 128), (3, 136), (17, 120), (5, 1000), (129, 264), (64, 4096), (2, 12288)]


@pytest.mark.parametrize("T,C", SIZES)
def test_codes_and_scales_are_exact(T, C):
    rng = np.random.default_rng(T * 10007 + C)
    x = bf16(rng.standard_normal((T, C)) * 10.0 ** rng.integers(-6, 6, (T, 1)))
    q, s = _quantize(x)
    rq, rs = oracle.act8_quantize(x)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("T,C", SIZES)
def test_values_read_back(T, C, act):
    rng = np.random.default_rng(T * 31 + C)
    x = bf16(rng.standard_normal((T, C)) * 3)
    q, s = _quantize(x)
    y, yc = guarded((T, C), torch.bfloat16)
    mf.mf_act8_dequantize(q, s, T, C, ACTS[act], y)
    v = oracle.act8_values(*oracle.act8_quantize(x))
    # q s rounds once (2^-24), sigma(w) is good to a few units of |w| 2^-24 (the
    # exponent's rounding) with |w| <= |z| (1.6 + 0.0714 z^2), and |act'| <= 1.13
    w = np.abs(v) * (1.6 + 0.0714 * v * v)
    check_bf16(host(y), oracle.mlp_act(v, act), np.abs(v) * (w + 8) * 2.0 ** -22, f"act8 {act}")
    yc()


def test_special_blocks():
    x = bf16(np.random.default_rng(5).standard_normal((6, 272)))
    x[0, :128] = 0
    x[1, 128:256] = np.float32(2.0 ** -101)         # below the smallest block kept
    x[2, 256:] = np.float32(2.0 ** -100)            # the smallest kept
    x[3, 5] = np.inf
    x[4, 271] = np.nan
    x[5, 130] = -np.inf
    t = torch.from_numpy(x).cuda().to(torch.bfloat16)
    q = torch.empty((6, 272), dtype=torch.int8, device="cuda")
    s = torch.empty((6, 3), dtype=torch.float32, device="cuda")
    mf.mf_act8_quantize(t, 6, 272, q, s)
    rq, rs = oracle.act8_quantize(t.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)
    y = torch.empty((6, 272), dtype=torch.bfloat16, device="cuda")
    mf.mf_act8_dequantize(q, s, 6, 272, mf.MF_ACT_NONE, y)
    y = host(y)
    assert np.isnan(y[3, :128]).all() and np.isnan(y[4, 256:]).all() and np.isnan(y[5, 128:256]).all()
    assert np.isfinite(y[3, 128:]).all() and np.isfinite(y[5, :128]).all()
    assert (y[0, :128] == 0).all() and (y[1, 128:256] == 0).all() and (y[2, 256:] != 0).all()


def test_largest_magnitudes():
    big = float(torch.finfo(torch.bfloat16).max)
    x = np.full((1, 128), big, dtype=np.float32)
    x[0, 1::2] = -big / 2
    q, s = _quantize(x)
    assert int(q[0, 0]) == 127 and np.isfinite(host(s)).all()
    y = torch.empty((1, 128), dtype=torch.bfloat16, device="cuda")
    for act in (mf.MF_ACT_GELU, mf.MF_ACT_SILU):
        mf.mf_act8_dequantize(q, s, 1, 128, act, y)
        y1 = host(y)
        # far below 0 the activation is held where it is within 1e-16 of its limit 0
        assert (np.abs(y1[0, 1::2]) <= 1e-16).all() and (y1[0, ::2] > 1e38).all()


def test_empty():
    mf.mf_act8_quantize(None, 0, 128, None, None)
    mf.mf_act8_dequantize(None, None, 0, 128, 0, None)


def test_offsets_past_32_bits():
    """2^31 + elements: the last rows, checked against the definition."""
    C = 4096
    T = (1 << 31) // C + 3
    x = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda")
    tail = bf16(np.random.default_rng(9).standard_normal((4, C)))
    x[-4:] = dev(tail)
    q = torch.empty((T, C), dtype=torch.int8, device="cuda")
    s = torch.empty((T, C // 128), dtype=torch.float32, device="cuda")
    mf.mf_act8_quantize(x, T, C, q, s)
    rq, rs = oracle.act8_quantize(tail)
    assert np.array_equal(q[-4:].cpu().numpy(), rq) and np.array_equal(s[-4:].cpu().numpy(), rs)
    x.fill_(-1)
    mf.mf_act8_dequantize(q, s, T, C, mf.MF_ACT_NONE, x)
    check_bf16(host(x[-4:]), oracle.act8_values(rq, rs), np.abs(tail) * 2.0 ** -23, "tail")
    assert (x[: T - 4] == 0).all()


def test_other_stream_and_graph_replay():
    T, C = 40, 520
    a, b = (bf16(np.random.default_rng(k).standard_normal((T, C))) for k in (1, 2))
    x = dev(a)
    q = torch.empty((T, C), dtype=torch.int8, device="cuda")
    s = torch.empty((T, 5), dtype=torch.float32, device="cuda")
    y = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        mf.mf_act8_quantize(x, T, C, q, s)
        mf.mf_act8_dequantize(q, s, T, C, mf.MF_ACT_SILU, y)
    x.copy_(dev(b))
    graph.replay()
    torch.cuda.synchronize()
    rq, rs = oracle.act8_quantize(b)
    assert np.array_equal(q.cpu().numpy(), rq)
    v = oracle.act8_values(rq, rs)
    check_bf16(host(y), oracle.mlp_act(v, "silu"), np.abs(v) * (np.abs(v) + 8) * 2.0 ** -22, "replay")


@pytest.mark.parametrize("C", [128, 264, 4096])
def test_tensors_on_16_byte_boundaries(C):
    """The least alignment the library asks for gives the same codes and values."""
    T = 37
    x = bf16(np.random.default_rng(C).standard_normal((T, C)))
    q, s = _quantize(x)
    y = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    mf.mf_act8_dequantize(q, s, T, C, mf.MF_ACT_GELU, y)

    def off(n, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        v = torch.empty(n + 16, dtype=dtype, device="cuda")[16 // size:][:n]
        assert v.data_ptr() % 32 == 16
        return v

    x2, q2 = off(T * C, torch.bfloat16).view(T, C), off(T * C, torch.int8).view(T, C)
    s2, y2 = off(s.numel(), torch.float32).view(s.shape), off(T * C, torch.bfloat16).view(T, C)
    x2.copy_(dev(x))
    mf.mf_act8_quantize(x2, T, C, q2, s2)
    mf.mf_act8_dequantize(q2, s2, T, C, mf.MF_ACT_GELU, y2)
    assert torch.equal(q2, q) and torch.equal(s2, s) and torch.equal(y2, y)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_a_nan_block_ends_where_it_ends(act):
    """The block beside one that reads back as NaN is as it would be."""
    rng = np.random.default_rng(29)
    x = bf16(rng.standard_normal((5, 392)))
    q, s = oracle.act8_quantize(x)
    s[2, 1] = np.nan
    y = torch.empty((5, 392), dtype=torch.bfloat16, device="cuda")
    mf.mf_act8_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), 5, 392, ACTS[act], y)
    bad = torch.isnan(y.float()).cpu().numpy()
    assert bad[2, 128:256].all() and bad.sum() == 128

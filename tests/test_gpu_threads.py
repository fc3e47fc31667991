"""Calls from host threads of the caller's own: a thread's very first CUDA call may be any
entry point, and threads with streams and buffers of their own do not disturb each other."""

import threading

import numpy as np
import pytest
import torch

import resolution_packed_diffusion_b200 as mf
from mlp_util import bf16, dev, dev32, modalities

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _in_a_thread(call):
    """The exception that ``call`` raises as the first CUDA call of a new host thread."""
    errors = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    return errors


def _first_calls():
    T, K, N = 200, 64, 256
    B, s = torch.bfloat16, torch.cuda.current_stream()
    x, W, g = (torch.randn(shape, device="cuda").to(B) for shape in ((T, K), (2, N, K), (T, N)))
    tm = torch.ones(T, dtype=torch.uint8, device="cuda")
    d, few = mf.make_descs([(0, 0, 0, T)]), mf.make_descs([(0, 0, 0, 20)])
    n = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(g)
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    H, D = 2, 128
    q, k, v = (torch.randn((T, H, D), device="cuda").to(B) for _ in range(3))
    cu_h = np.array([0, T], dtype=np.int32)
    cu, o, lse = torch.from_numpy(cu_h).cuda(), torch.empty_like(q), torch.empty((H, T), device="cuda")
    na = mf.mf_workspace_size(T, H, D, 0)
    wa = torch.empty(max(1, na), dtype=torch.uint8, device="cuda")
    img, wt = torch.randn((1, 8, 8, 64), device="cuda").to(B), torch.randn((64, 3, 3, 64), device="cuda").to(B)
    cb, y = torch.zeros(64, device="cuda"), torch.empty((1, 8, 8, 64), dtype=B, device="cuda")
    return {
        "linear_fused": lambda: mf.mf_linear_fused(x, W, None, None, tm, d, K, N, 1, None, None, None, out, stream=s),
        "linear_fused, few rows": lambda: mf.mf_linear_fused(x, W, None, None, tm, few, K, N, 1, None, None, None,
                                                             out, stream=s),
        "linear_fused_bwd": lambda: mf.mf_linear_fused_bwd(g, x, None, None, W, None, None, None, tm, d, K, N, 0, dx,
                                                           dW, None, ws, n, stream=s),
        "modality_linear": lambda: mf.mf_modality_linear(x, W, tm, [(0, 0, 0, T)], K, N, out, stream=s),
        "varlen_attn_fwd": lambda: mf.mf_varlen_attn_fwd(q, k, v, cu, cu_h, 1, H, D, D ** -0.5, None, 2, 1e4, o, lse,
                                                         wa, na, stream=s),
        "conv3x3": lambda: mf.mf_conv3x3(img, wt, cb, None, 1, 8, 8, 64, 64, y, stream=s),
    }


@pytest.mark.parametrize("name", ["linear_fused", "linear_fused, few rows", "linear_fused_bwd", "modality_linear",
                                  "varlen_attn_fwd", "conv3x3"])
def test_a_threads_first_cuda_call(name):
    call = _first_calls()[name]
    call()  # whatever a process sets up once is there: the thread is what is new
    torch.cuda.synchronize()
    assert _in_a_thread(call) == []
    assert mf.mf_get_error() == mf.MF_OK


def test_calls_from_two_threads():
    """Two host threads, each with a stream, buffers and shapes of its own."""
    packs = [(((1, 9, 14, 5), (0, 0, 0, 133)), 264, 520), (((0, 0, 0, 61),), 512, 136)]
    jobs = []
    for descs, K, N in packs:
        mod = modalities(descs)
        T = len(mod)
        rng = np.random.default_rng(K)
        x, W, g = (dev(bf16(rng.standard_normal(s))) for s in ((T, K), (2, N, K), (T, N)))
        n = max(mf.mf_linear_fused_bwd_workspace_size(T, K, N), mf.mf_layer_norm_bwd_workspace_size(T, K))
        jobs.append(dict(d=mf.make_descs(descs), K=K, N=N, T=T, x=x, W=W, g=g, n=n, tm=torch.from_numpy(mod).cuda(),
                         gamma=dev32(np.ones((2, K))), st=dev32(np.tile([[0.0, 1.0]], (T, 1))),
                         out=torch.empty_like(g), dx=torch.empty_like(x), dW=torch.empty_like(W),
                         db=torch.empty((2, N), device="cuda"), dl=torch.empty_like(x),
                         dg=torch.empty((2, K), device="cuda"), dbeta=torch.empty((2, K), device="cuda"),
                         ws=torch.empty(n, dtype=torch.uint8, device="cuda"), stream=torch.cuda.Stream()))

    def step(j):
        mf.mf_linear_fused(j["x"], j["W"], None, None, j["tm"], j["d"], j["K"], j["N"], 1, None, None, None, j["out"],
                           stream=j["stream"])
        mf.mf_linear_fused_bwd(j["g"], j["x"], None, None, j["W"], j["out"], None, None, j["tm"], j["d"], j["K"],
                               j["N"], 1, j["dx"], j["dW"], j["db"], j["ws"], j["n"], stream=j["stream"])
        mf.mf_layer_norm_bwd(j["dx"], j["x"], None, None, j["gamma"], j["st"], j["tm"], None, j["T"], j["K"],
                             j["dl"], j["dg"], j["dbeta"], j["ws"], j["n"], stream=j["stream"])

    names = ("out", "dx", "dW", "db", "dl", "dg", "dbeta")
    torch.cuda.synchronize()
    for j in jobs:
        step(j)
    torch.cuda.synchronize()
    want = [[j[k].clone() for k in names] for j in jobs]
    errors = []

    def work(j):
        try:
            for _ in range(50):
                step(j)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and mf.mf_get_error() == mf.MF_OK
    for j, ref in zip(jobs, want):
        for k, r in zip(names, ref):
            assert torch.equal(j[k], r), k

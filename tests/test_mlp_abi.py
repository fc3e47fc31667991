"""Refusals and size queries of the MLP-branch operators without a GPU: every call
here fails its checks (or has nothing to do) before anything is launched."""

import ctypes

import pytest

mf = pytest.importorskip("resolution_packed_diffusion_b200")

INV, UNS = mf.MF_ERR_INVALID, mf.MF_ERR_UNSUPPORTED
A = [(i + 1) << 32 for i in range(20)]  # far-apart, aligned stand-ins for device pointers


def _descs(*rows):
    arr = mf.make_descs(rows)
    return ctypes.cast(arr, ctypes.c_void_p), len(rows), arr


def _quant(x=A[0], T=4, C=256, q=A[1], s=A[2]):
    return mf.lib.mf_act8_quantize(x, T, C, q, s, None)


def _dequant(q=A[0], s=A[1], T=4, C=256, act=0, y=A[2]):
    return mf.lib.mf_act8_dequantize(q, s, T, C, act, y, None)


def test_act8_refusals():
    assert _quant(T=0, x=None, q=None, s=None) == mf.MF_OK
    assert _dequant(T=0, q=None, s=None, y=None) == mf.MF_OK
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(C=0), dict(C=12), dict(C=(1 << 20) + 8),
                dict(x=None), dict(q=None), dict(s=None), dict(x=A[0] + 8), dict(q=A[1] + 4),
                dict(s=A[2] + 4), dict(q=A[0]), dict(q=A[0] + 16), dict(s=A[1] + 16), dict(s=A[0])):
        assert _quant(**bad) == INV, bad
    for bad in (dict(T=-1), dict(C=4), dict(act=3), dict(act=-1), dict(q=None), dict(s=None),
                dict(y=None), dict(y=A[0]), dict(y=A[1]), dict(y=A[2] + 2)):
        assert _dequant(**bad) == INV, bad


def _ln(x=A[0], g=A[1], b=A[2], m=A[3], T=4, hid=256, eps=1e-6, y=A[4], st=A[5]):
    return mf.lib.mf_layer_norm(x, g, b, m, T, hid, eps, y, st, None)


def _ln_bwd(dy=A[0], x=A[1], x8=None, xs=None, g=A[2], st=A[3], m=A[4], r=None, T=4, hid=256,
            dx=A[5], dg=A[6], db=A[7], ws=A[8], n=1 << 30):
    return mf.lib.mf_layer_norm_bwd(dy, x, x8, xs, g, st, m, r, T, hid, dx, dg, db, ws, n, None)


def test_layer_norm_refusals():
    assert _ln(T=0, x=None, y=None) == mf.MF_OK
    assert _ln(hid=8200) == UNS
    for bad in (dict(T=-1), dict(hid=0), dict(hid=12), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(g=None), dict(b=None), dict(m=None),
                dict(y=None), dict(x=A[0] + 2), dict(st=A[5] + 8), dict(y=A[0]), dict(y=A[0] + 64),
                dict(st=A[4]), dict(st=A[0]), dict(y=A[1]), dict(y=A[3])):
        assert _ln(**bad) == INV, bad


def test_layer_norm_bwd_refusals():
    n = mf.mf_layer_norm_bwd_workspace_size(4, 256)
    assert n > 0 and mf.mf_layer_norm_bwd_workspace_size(4, 12) == 0
    assert mf.mf_layer_norm_bwd_workspace_size(0, 256) == 0
    assert _ln_bwd(hid=8200) == UNS
    for bad in (dict(T=-1), dict(hid=20), dict(x=None), dict(x8=A[9], xs=A[10]),  # none / both forms
                dict(x=None, x8=A[9]), dict(x=None, xs=A[9]), dict(xs=A[9]),
                dict(dy=None), dict(g=None), dict(st=None), dict(m=None), dict(dx=None),
                dict(dg=None), dict(db=None), dict(ws=None), dict(n=n - 1), dict(dx=A[0]),
                dict(dx=A[1]), dict(r=A[5] + 32), dict(dg=A[7]), dict(dg=A[0]), dict(db=A[2]),
                dict(ws=A[1]), dict(ws=A[5]), dict(dx=A[5] + 2), dict(r=A[9] + 8)):
        assert _ln_bwd(**bad) == INV, bad


def _lin(x=A[0], W=A[1], b=A[2], r=None, m=A[3], d=((1, 2, 2, 3),), S=None, K=64, N=128, act=1,
         z=None, z8=None, zs=None, out=A[4]):
    p, n, keep = _descs(*d)
    return mf.lib.mf_linear_fused(x, W, b, r, m, p, n if S is None else S, K, N, act, z, z8, zs, out,
                                  None)


def _lin_bwd(g=A[0], x=A[1], x8=None, xs=None, W=A[2], z=A[3], z8=None, zs=None, m=A[4],
             d=((1, 2, 2, 3),), S=None, K=64, N=128, act=1, dx=A[5], dW=A[6], db=A[7], ws=A[8],
             n=1 << 30):
    p, c, keep = _descs(*d)
    return mf.lib.mf_linear_fused_bwd(g, x, x8, xs, W, z, z8, zs, m, p, c if S is None else S, K, N,
                                      act, dx, dW, db, ws, n, None)


def test_linear_fused_refusals():
    assert _lin(d=((0, 0, 0, 0),), x=None, out=None) == mf.MF_OK
    assert _lin(d=((0, 0, 0, 131073),)) == UNS
    for bad in (dict(S=0), dict(S=513), dict(K=0), dict(K=12), dict(N=4), dict(N=130),
                dict(K=(1 << 20) + 8), dict(act=3), dict(d=((1, -1, 2, 3),)), dict(d=((1, 2, 2, -3),)),
                dict(d=((2000, 4096, 4096, 0),)), dict(d=((1, 65536, 65536, 0),)),
                dict(x=None), dict(W=None), dict(m=None), dict(out=None),
                dict(z8=A[9]), dict(zs=A[9]), dict(x=A[0] + 8), dict(b=A[2] + 4), dict(r=A[9] + 2),
                dict(out=A[0]), dict(out=A[1] + 64), dict(out=A[2]), dict(r=A[4] + 256),
                dict(z=A[4]), dict(z8=A[4], zs=A[9]), dict(z8=A[9], zs=A[9]), dict(z=A[0]),
                dict(r=A[9], z=A[9])):
        assert _lin(**bad) == INV, bad


def test_linear_fused_bwd_refusals():
    n = mf.mf_linear_fused_bwd_workspace_size(7, 64, 128)
    assert n > 0
    for a in ((0, 64, 128), (7, 60, 128), (7, 64, 4), (7, (1 << 20) + 8, 8)):
        assert mf.mf_linear_fused_bwd_workspace_size(*a) == 0
    assert _lin_bwd(d=((0, 0, 0, 131073),)) == UNS
    for bad in (dict(S=0), dict(K=12), dict(N=0), dict(act=-1), dict(dx=None, dW=None, db=None),
                dict(g=None), dict(m=None), dict(ws=None), dict(n=n - 1), dict(x=None),
                dict(x8=A[9], xs=A[10]), dict(x=None, x8=A[9]), dict(xs=A[9]), dict(W=None),
                dict(z=None), dict(z8=A[9], zs=A[10]), dict(z=None, zs=A[9]),
                dict(dx=A[0]), dict(dW=A[1]), dict(db=A[2]), dict(dx=A[3]), dict(ws=A[0]),
                dict(dW=A[5]), dict(db=A[6]), dict(ws=A[7]), dict(dx=A[5] + 8), dict(dW=A[6] + 2),
                dict(d=((1, 2, -2, 3),))):
        assert _lin_bwd(**bad) == INV, bad


def test_binding_takes_a_descriptor_array():
    arr = mf.make_descs([(1, 2, 2, 3), (0, 0, 0, 5)])
    assert mf._descs(arr) == (arr, 2)
    got, n = mf._descs([(1, 2, 2, 3), (0, 0, 0, 5)])
    assert n == 2 and [(d.frames, d.n_text) for d in got] == [(1, 3), (0, 5)]


def test_binding_takes_subclasses_of_int_as_addresses():
    """A pointer may come as any int, an enum's or a library's own type too."""
    class Address(int):
        pass

    assert mf._ptr(Address(A[0])) == A[0] and mf._ptr(A[0]) == A[0] and mf._ptr(None) is None
    mf.mf_layer_norm(Address(A[0]), Address(A[1]), Address(A[2]), Address(A[3]), 0, 256, 1e-6,
                     Address(A[4]), Address(A[5]), stream=Address(0))
    with pytest.raises(mf.MFError) as e:  # reaches the library, which finds x and y the same
        mf.mf_layer_norm(Address(A[0]), Address(A[1]), Address(A[2]), Address(A[3]), 4, 256, 1e-6,
                         Address(A[0]), stream=0)
    assert e.value.status == INV


@pytest.mark.parametrize("a,b", [(8, 8), (128, 512), (1000, 2056), (12288, 3080)])
def test_a_workspace_for_a_long_pack_serves_a_shorter_one(a, b):
    """The sizes never fall as T grows: a buffer taken for the largest pack is enough for
    every other."""
    lengths = sorted({max(1, c + d) for c in (1, 64, 128, 544, 2048, 4096, 8192, 16384, 131072)
                      for d in (-129, -65, -33, -1, 0, 1, 33, 65, 129) if c + d <= 131072})
    sizes = [mf.mf_linear_fused_bwd_workspace_size(t, a, b) for t in lengths]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    for width in (8, 264, 1000, 3000, 8192):
        sizes = [mf.mf_layer_norm_bwd_workspace_size(t, width) for t in lengths]
        assert sizes[0] > 0 and sizes == sorted(sizes)


def test_the_linear_backward_asks_for_the_memory_that_it_can_use():
    """Few tokens cannot have dW's sum cut into parts, whose places are 256 KB each; a long
    pack and one of many short runs can, of a narrow layer."""
    size = mf.mf_linear_fused_bwd_workspace_size
    for t in (1, 16, 40):
        for k, n in ((8, 8), (128, 512), (512, 128)):
            assert size(t, k, n) < 4 * t * (k + n) + 8 * n * t + 2048
    for t in (1024, 16384):  # up to 512 runs, each with a step of its own
        assert size(t, 128, 512) >= 2 * 2 * 37 * 256 * 256 * 4

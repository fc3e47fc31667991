"""Shared by the GPU tests of the MLP-branch operators: device copies, packs, and
tolerances that follow from the arithmetic.

bf16: an output is one rounding of an fp32 value, off by at most half a step,
2^-8 of it; the fp32 value is off by ``slack`` (given per operator). FP32 sums of n
terms on the tensor cores are bounded by n 2^-23 sum|terms| (one unit per addition,
whether it rounds or truncates)."""

from __future__ import annotations

import numpy as np
import torch

import resolution_packed_diffusion_b200 as mf
from gpu_util import dev_bf16
from packgen import bf16_bits_to_f32, f32_to_bf16_bits

HALF_BF16 = 2.0 ** -8
ACTS = {"none": mf.MF_ACT_NONE, "gelu": mf.MF_ACT_GELU, "silu": mf.MF_ACT_SILU}


def bf16(a) -> np.ndarray:
    """The float32 values of a rounded to bf16."""
    return bf16_bits_to_f32(f32_to_bf16_bits(np.asarray(a, dtype=np.float32)))


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


def dev(a) -> torch.Tensor:
    """float32 bf16-valued array -> bf16 device tensor."""
    return dev_bf16(f32_to_bf16_bits(np.asarray(a, dtype=np.float32)))


def dev32(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def host(t) -> np.ndarray:
    return t.float().cpu().numpy().astype(np.float64)


def modalities(descs) -> np.ndarray:
    out = []
    for f, h, w, t in descs:
        out += [0] * (f * h * w) + [1] * t
    return np.array(out, dtype=np.uint8)


def guarded(shape, dtype, guard=64):
    """An output buffer with ``guard`` rows behind it that hold a pattern; returns
    (the output view, a check that the rows behind are as they were)."""
    rows, rest = shape[0], tuple(shape[1:])
    fill = 77 if dtype == torch.int8 else 1234.0
    whole = torch.full((rows + guard, *rest), fill, dtype=dtype, device="cuda")

    def check():
        assert (whole[rows:] == fill).all(), "rows behind the output were written"
    return whole[:rows], check


def check_bf16(got, ref, slack, name):
    """Every element within its bf16 rounding and the fp32 slack."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), f"{name}: non-finite"
    tol = HALF_BF16 * np.abs(ref) + (1 + HALF_BF16) * slack + 1e-38
    err = np.abs(got - ref)
    if err.size:
        i = np.unravel_index(int(np.argmax(err - tol)), err.shape)
        assert err[i] <= tol[i], f"{name}{i}: got {got[i]}, want {ref[i]}, tolerance {tol[i]:.3g}"


def check_rms(got, ref, roundings, name):
    """Relative RMS for ``roundings`` independent bf16 roundings: each is off by at
    most 2^-8 of a value and uniform in that interval at worst, 2^-8 / sqrt(3) RMS."""
    n = float(np.linalg.norm(ref))
    if n == 0:
        return
    rel = float(np.linalg.norm(np.asarray(got, np.float64) - ref)) / n
    assert rel <= np.sqrt(roundings / 3.0) * HALF_BF16, f"{name}: relative RMS {rel:.3g}"

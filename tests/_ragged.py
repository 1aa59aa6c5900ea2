"""Helpers of the int8 and ragged-product tests: pitched operands, references in 64 bits and
the tolerances, which count roundings."""
from __future__ import annotations

import math

import torch

import synth

U32 = 2.0 ** -24  # half a step of FP32


def pitched(t, extra=0):
    """The same values with rows on 16-byte boundaries (`extra` more units of pitch)."""
    unit = 16 // t.element_size()
    n = t.shape[-1]
    pad = (-(-n // unit) + extra) * unit
    buf = torch.zeros(t.shape[:-1] + (pad,), dtype=t.dtype, device=t.device)
    buf[..., :n] = t
    return buf[..., :n]


def normal(seed, i, shape, dtype, std=1.0):
    return torch.from_numpy(synth.normal(seed, i, tuple(shape), std)).to(dtype)


def codes(seed, i, shape, lo=-128, hi=127):
    return torch.from_numpy(synth.integers(seed, i, tuple(shape), lo, hi)).to(torch.int8)


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32)


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act in ("gelu", "gelu_tanh"):
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def check(got, ref, slack, act="none", what=""):
    """|got - ref| <= half a step of the output type (relative to the value, or the spacing of
    its subnormals) + the error `slack` of the FP32 value before it, through the activation
    (slope at most 1.13 for GeLU, 1.1 for SiLU, and its own relative error below 2^-16)."""
    got, ref = got.double().cpu(), ref.double().cpu()
    dt = check.dtype
    fi = torch.finfo(dt)
    tol = ref.abs() * (fi.eps / 2) * 1.001 + fi.smallest_normal * fi.eps / 2
    tol = tol + (slack * 1.13 + (ref.abs() * 2.0 ** -16 if act != "none" else 0.0))
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i]}, "
                             f"ref {ref[i]}, tolerance {tol[i]}")


def check_as(dtype, got, ref, slack, act="none", what=""):
    check.dtype = dtype
    assert got.dtype == dtype
    check(got, ref, slack, act, what)


def products64(x, w):
    """x @ w in 64 bits and the slack of an FP32 accumulation of it: K products summed with an
    error of at most one FP32 step (two half steps, so that truncation counts too) of the
    running sum of magnitudes each."""
    x, w = x.double(), w.double()
    return x @ w, (x.abs() @ w.abs()) * (2 * U32 * (x.shape[-1] + 2))

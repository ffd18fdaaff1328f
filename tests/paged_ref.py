"""The rotation, the paged cache and the paged decode in plain float64 numpy,
from their definitions, with error bounds for the kernels' roundings."""
from __future__ import annotations

import math

import numpy as np

DTYPES = ("f32", "bf16", "f16")


def torch_dtype(name: str):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def half_step(name: str) -> float:
    """Largest relative error of one rounding to the type."""
    import torch
    return torch.finfo(torch_dtype(name)).eps / 2


def f64(t) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def rope(x, positions, rot, interleaved, pair_axis=None, freqs=None, base=10000.0, sign=1.0):
    """x [..., 64] turned by positions [axes, ...]; returns (result, allowance
    before the rounding to the output type).

    The kernel's cosine and sine come from an angle that is rounded once in
    half turns (at most 2^-25 half turns, pi 2^-25 < 2^-23 radians) and a
    sincospif of at most 2 units in the last place (2^-23 near 1); the two
    products and their sum add three half units.  Each result is thus within
    (|x_u| + |x_v|) (2^-23 + 2^-23 + 3 2^-24) < (|x_u| + |x_v|) 2^-21."""
    y, tol = x.copy(), np.zeros_like(x)
    for p in range(rot // 2):
        u, v = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
        f = base ** (-2.0 * p / rot) if freqs is None else freqs[p]
        a = positions[0 if pair_axis is None else pair_axis[p]].astype(np.float64) * f
        c, s = np.cos(a), sign * np.sin(a)
        y[..., u] = x[..., u] * c - x[..., v] * s
        y[..., v] = x[..., v] * c + x[..., u] * s
        tol[..., u] = tol[..., v] = (np.abs(x[..., u]) + np.abs(x[..., v])) * 2.0 ** -21
    return y, tol


def cache_rows(pages, table_row, length, h):
    """Rows 0..length-1 of head h of a sequence: [length, 64]."""
    size = pages.shape[2]
    return np.stack([pages[table_row[j // size], h, j % size] for j in range(length)]) if length else np.zeros((0, 64))


def attended(length, window, d):
    if window < 0:
        return list(range(length))
    return list(range(length - 1, -1, -d))[:window + 1]


def softmax_row(q, k, v, scale, half_p):
    """(o, lse, allowance of o, allowance of lse) of one query over rows k, v
    [n, 64] in float64.

    Relative error of a probability before normalisation: its score, a float32
    sum of 64 products and a few scalings, is off by at most
    e_s = 70 2^-24 sum_c |q_c k_c| scale (natural units; the same again for the
    stored maximum that is taken from it), the exponential by 2^-22 plus the
    rounding of its argument, 2^-24 times the argument's size; float32 sums of
    n terms and their rescalings add (n + 64) 2^-24 each, in the numerator and
    in the denominator; half_p is the rounding of the probabilities that enter
    a 16-bit matrix product."""
    if len(k) == 0:
        return np.zeros(64), -math.inf, np.zeros(64), 0.0
    s = (k @ q) * scale
    size = (np.abs(k) @ np.abs(q)) * scale
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    o = (p / total) @ v
    e = 2 * 70 * 2.0 ** -24 * size.max() + 2.0 ** -22 + 2 * 2.0 ** -24 * np.abs(s).max() * 1.45 \
        + (len(k) + 64) * 2.0 ** -24
    lse = top + math.log(total)
    return o, lse, (p / total) @ np.abs(v) * (2 * e + half_p), e + 2.0 ** -22 * (abs(lse) + 1)


def check(name, got, ref, tol):
    got = np.asarray(got)
    assert np.all(np.isfinite(got) == np.isfinite(ref)), name + ": finite in other places"
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine]), name + ": other infinities"
    over = np.abs(got[fine] - ref[fine]) - np.broadcast_to(tol, ref.shape)[fine]
    assert over.size == 0 or over.max() <= 0, "%s: %.3g over its allowance" % (name, over.max())

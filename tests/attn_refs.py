"""Plain 64-bit forms of the cache formats and of attention, and the error bounds that the
GPU tests hold the kernels to. Nothing here is taken from the kernels.

The bound on an attention output. Write w_t for the softmax weights and
A = sum_t w_t |v_t| per output element.
  * BF16 result: one rounding to nearest, at most u |o| with u = 2^-8.
  * weights rounded to 16 bits before they multiply V: at most u A (BF16, f16 less).
  * scores: products of 16-bit values are exact in fp32; D of them are added in fp32 in some
    order and scaled, so |dz| <= (D + 4) 2^-24 scale sum_d |q_d k_d| =: e; a score off by e moves
    every weight, and their sum, by a factor within e^(+-e): at most 4 e A for e < 1/4.
  * exponentials, fp32 sums over the keys (chained tile by tile, 2^-24 a step), the division:
    under 2^-14 A together, up to the 100k keys tested here.
Scores, weights and bounds below are evaluated in 64 bits.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -8
QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def round_e4m3(y):
    """float64 array -> nearest value of 4 exponent and 3 mantissa bits (ties to even), clamped to +-448."""
    a = np.minimum(np.abs(y), 448.0)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.sign(y) * np.minimum(np.rint(a / step) * step, 448.0)


def quantise(x, fmt):
    """float32 rows [..., D] -> (code values float64, scale float32), as include/gather_lora.h states it:
    the two divisions and the product in float32, the rounding exact."""
    x = np.asarray(x, dtype=np.float32)
    q = np.float32(QMAX[fmt])
    with np.errstate(all="ignore"):
        a = np.max(np.abs(x), axis=-1)                       # NaN if the row has one
        keep = np.isfinite(a) & (a >= np.float32(2.0 ** -100))
        inv = np.where(keep, q / a, np.float32(0)).astype(np.float32)
        scale = np.where(keep, a / q, np.float32(0)).astype(np.float32)
        y = np.where(keep[..., None], x * inv[..., None], np.float32(0)).astype(np.float64)
    code = round_e4m3(y) if fmt == "e4m3" else np.clip(np.rint(y), -127, 127)
    scale = np.where(np.isfinite(a), scale, np.float32(np.nan))
    return code, scale


def attend(q, k, v, scale, seen=None):
    """One head: q [n, D], k and v [m, D] (float64 tensors), seen [n, m] bool. Returns out [n, D],
    lse [n] and the bound [n, D]. Invisible keys take no part, whatever they hold."""
    n, m, D = q.shape[0], k.shape[0], q.shape[1]
    out = torch.zeros(n, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lse = torch.full((n,), -torch.inf, dtype=torch.float64, device=q.device)
    if m == 0 or n == 0:
        return out, lse, bound
    if seen is None:
        seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    used = seen.any(0)          # keys no row sees are dropped before any arithmetic
    k, v, seen = k[used], v[used], seen[:, used]
    if k.shape[0] == 0:
        return out, lse, bound
    z = torch.where(seen, scale * (q @ k.T), -torch.inf)
    some = seen.any(1)
    mag = torch.where(seen, scale * (q.abs() @ k.abs().T), 0.0).amax(1, keepdim=True)
    top = torch.where(some[:, None], z.amax(1, keepdim=True), 0.0)
    w = torch.exp(z - top)
    s = w.sum(1, keepdim=True)
    w = torch.where(some[:, None], w / s, 0.0)
    if torch.isfinite(v).all():
        out = w @ v
        a = w @ v.abs()
    else:                       # a key with weight zero by the mask has no influence even if infinite
        out = torch.stack([w[i][seen[i]] @ v[seen[i]] for i in range(n)])
        a = torch.stack([w[i][seen[i]] @ v[seen[i]].abs() for i in range(n)])
    e = (D + 4) * 2.0 ** -24 * mag
    lse = torch.where(some, (top + s.log())[:, 0], -torch.inf)
    bound = U * out.abs() + (U + 4 * e + 2.0 ** -14) * a + 1e-30
    return out, lse, bound


def check(got, want, bound, what=""):
    """Every element within its bound; NaN where and only where NaN is wanted."""
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN at other places than wanted"
    off = (got - want).abs()[~nan] - bound[~nan]
    assert off.numel() == 0 or off.max().item() <= 0, f"{what}: {(off > 0).sum().item()} of {off.numel()} outside the bound, worst by {off.max().item():.3g}"


def check_lse(got, want, q_abs, what=""):
    """lse in fp32: off by the score error (q_abs: a bound on scale * sum |q k|) and a few ulps."""
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    tol = 2.0 ** -20 * (1 + want.abs()) + 140 * 2.0 ** -24 * q_abs
    assert ((got - want).abs()[~inf] <= (tol.expand_as(want))[~inf]).all(), what

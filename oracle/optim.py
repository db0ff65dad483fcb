"""AdamW with 32- or 8-bit moments, the global gradient clip, and LayerNorm —
TEST INFRASTRUCTURE ONLY, plain numpy, one tensor at a time.

"noeira docs, SmolVLA" §Fine-tuning names the tensors that train and no
optimiser; the update is AdamW (Loshchilov and Hutter, "Decoupled weight decay
regularization") with the readings below. Nothing here shares code with the
CUDA library; the random numbers are ``oracle.philox``'s.

Readings:
  * each product and sum is rounded to float32 by itself (``dtype=float32``);
    with ``dtype=float64`` the same formulas give the exact update;
  * the norm is over all tensors, in float64; the factor c = min(1, max_norm /
    (norm + 1e-6)) is rounded to ``dtype``; a norm that is not finite skips the
    step;
  * 8-bit moments: m in e4m3, v in e5m2, a power-of-two scale for 256
    consecutive elements of a tensor. The scale puts the largest magnitude into
    [2^7, 2^8) or [2^14, 2^15), but its own exponent is at least that of
    2^-120 or 2^-112 (magnitudes near the end of float32's range). A magnitude
    between two codes becomes the upper one if (distance to the lower) /
    (spacing) + u >= 1, u = 16 random bits / 2^16, on a grid of 8 (4) steps an
    octave. What then lies below the smallest normal code (2^-6 or 2^-14 of the
    scale) has none: m becomes 0, v > 0 the smallest normal.
"""
from __future__ import annotations

import numpy as np

from .philox import philox4x32_10

BLOCK = 256
# (mantissa bits, exponent bias, place of the block's largest exponent, NaN code)
E4M3 = (3, 7, 7, 0x7F)
E5M2 = (2, 15, 14, 0x7F)


def decode(code, fmt):
    """Values of the codes of a format, float64 (subnormal codes included)."""
    digits, bias, _, nan = fmt
    c = np.asarray(code).astype(np.int64)
    e, f = (c & 0x7F) >> digits, (c & ((1 << digits) - 1)).astype(np.float64) / (1 << digits)
    v = np.where(e == 0, f * 2.0 ** (1 - bias), (1 + f) * 2.0 ** (e - bias).astype(np.float64))
    v = np.where((c & 0x7F) == nan, np.nan, v)
    return np.where(c & 0x80, -v, v)


def random16(n: int, tensor: int, step: int, seed: int) -> np.ndarray:
    """The 16 random bits of each of a tensor's n elements."""
    q = np.arange((n + 7) // 8, dtype=np.uint64)
    c = (q & np.uint64(0xFFFFFFFF), q >> np.uint64(32), np.full_like(q, step & 0xFFFFFFFF), np.full_like(q, tensor))
    words = np.stack(philox4x32_10(c, (seed & 0xFFFFFFFF, seed >> 32)), axis=1)
    return np.stack([words & 0xFFFF, words >> 16], axis=2).reshape(-1)[:n].astype(np.int64)


def encode(x, u16, fmt, keep_positive: bool):
    """(codes uint8 [n], scales float32 [blocks]) of the values x [n]."""
    digits, bias, top, nan = fmt
    x = np.asarray(x, dtype=np.float64)
    n, blocks = x.size, -(-x.size // BLOCK)
    codes, scales = np.zeros(n, np.uint8), np.zeros(blocks, np.float32)
    least = 2.0 ** (1 - bias)
    for b in range(blocks):
        s = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        a = np.abs(x[s])
        finite = np.isfinite(a)
        most = a[finite].max() if finite.any() else 0.0
        if most > 0:
            e = max(int(np.floor(np.log2(most))) - top, -127 + bias) if most >= 2.0 ** -126 else -127 + bias
            scales[b] = 2.0 ** e
        y = np.where(finite, a, 0.0) / (float(scales[b]) or 1.0)
        # below the smallest normal code the grid goes on octave by octave (down to float32's smallest normal)
        grid = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -126 / (float(scales[b]) or 1.0)))) - digits)
        y = np.floor(y / grid + u16[s] / 65536.0) * grid
        y = np.where(y < least, np.where((a > 0) & keep_positive, least, 0.0), y)
        e = np.floor(np.log2(np.maximum(y, least)))
        code = np.where(y > 0, (e + bias) * 2 ** digits + (y / 2.0 ** e - 1) * 2 ** digits, 0).astype(np.int64)
        code = np.where((x[s] < 0) & (code > 0), code | 0x80, code)
        codes[s] = np.where(finite, code, nan).astype(np.uint8)
    return codes, scales


def grad_norm(grads) -> float:
    return float(np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads)))


def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, decay=True, c=1.0, dtype=np.float64):
    """(p, m, v) after one step of one tensor, in ``dtype`` arithmetic."""
    f = dtype
    p, g, m, v = (np.asarray(x, dtype=f) for x in (p, g, m, v))
    with np.errstate(all="ignore"):
        g = g * f(c)
        m = m * f(beta1) + g * f(1.0 - beta1)
        v = v * f(beta2) + (g * g) * f(1.0 - beta2)
        denom = np.sqrt(v) * f(1.0 / np.sqrt(1.0 - beta2 ** float(step))) + f(eps)
        keep = f(1.0 - lr * weight_decay) if decay else f(1.0)
        p = p * keep - (m / denom) * f(lr / (1.0 - beta1 ** float(step)))
    return p, m, v


def clip_factor(norm: float, max_norm: float) -> float:
    return min(1.0, max_norm / (norm + 1e-6)) if max_norm else 1.0


def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd) of rows, float64."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta), float64, from the statistics given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    w = dy * gamma
    dx = np.asarray(rstd, np.float64)[:, None] * (w - w.mean(1, keepdims=True) - xh * (w * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)

"""CPU oracle of the AdamW step with 32-bit or 8-bit moments, of the global
gradient norm and of the 8-bit codes.

TEST INFRASTRUCTURE ONLY, like :mod:`oracle.muon_oracle`: it shares no code
with the CUDA library and imports nothing from the package.

Two levels.  The formulas in 64 bits (:func:`adamw_step`, :func:`grad_norm`,
:func:`round_to_codes`) say what is meant.  :func:`moments_f32` and
:func:`codes_f32` restate, in NumPy's 32-bit arithmetic (every operation
rounded to the nearest), the chain whose roundings the library fixes, so that
its moments and codes can be compared bit for bit.

The pages name AdamW on embeddings and scalars (PR #1893 "Record:
L_ParallelResiduals_UNetSkips_DepthRecur_Muon_ 1.0901", table "Architecture
and training stack", row "Optimizer") and give no state format; the codes are
defined here: blocks of 256 elements; the first moment as sign, 3 exponent and
4 mantissa bits, the second moment's root as 3 exponent and 5 mantissa bits,
each under a power of two per block, 2^(byte - 127) being the value of the
code with exponent 7 and mantissa 0.
"""

from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

BLOCK = 256
M_BITS, R_BITS = 4, 5
LOW, HIGH, NAN_BYTE = 20, 245, 255


# ---- codes --------------------------------------------------------------------

def code_values(bits: int) -> np.ndarray:
    """Values of the 256 codes for byte 127 (2^0), in 64 bits.  bits: mantissa
    bits; with 4, bit 7 is the sign."""
    c = np.arange(256)
    mag = c & 0x7F if bits == M_BITS else c
    e, f = mag >> bits, (mag & ((1 << bits) - 1)) / 2.0 ** bits
    v = np.where(e == 0, f * 2.0 ** -6, (1 + f) * 2.0 ** (e - 7.0))
    return np.where(c >= 128, -v, v) if bits == M_BITS else v


def decode(codes: np.ndarray, scale_bytes: np.ndarray, bits: int) -> np.ndarray:
    """Values of a tensor's codes (flat), scale_bytes one per block."""
    b = np.repeat(np.asarray(scale_bytes, dtype=np.int64), BLOCK)[:codes.size]
    with np.errstate(over="ignore"):
        v = code_values(bits)[codes] * np.exp2(b - 127.0)
    return np.where(b > HIGH, np.nan, v)


def _blocks(x: np.ndarray) -> np.ndarray:
    n = x.size
    out = np.zeros((-(-n // BLOCK), BLOCK), dtype=x.dtype)
    out.reshape(-1)[:n] = x
    return out


def scale_byte(x: np.ndarray, bits: int) -> np.ndarray:
    """Per block, the least byte whose top code reaches the largest |x|."""
    top = np.max(np.abs(_blocks(np.asarray(x, np.float64))), axis=1)
    out = np.full(top.size, NAN_BYTE)
    fine = np.isfinite(top)
    best = 2.0 - 2.0 ** -bits                  # the top code's value at 2^0
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.ceil(np.log2(np.maximum(top, 1e-300) / best)), -1000)
    # log2 is only near: settle on the least E with best 2^E >= top
    for _ in range(2):
        e = np.where(best * np.exp2(e - 1) >= top, e - 1, e)
    for _ in range(2):
        e = np.where(best * np.exp2(e) < top, e + 1, e)
    b = np.maximum(e + 127, LOW)
    return np.where(fine & (b <= HIGH), b, out).astype(np.int64)


def round_to_codes(x, bits: int, sixteen: Optional[np.ndarray] = None):
    """(codes, bytes) of a flat array from the definition, in 64 bits: to the
    nearest code (ties to the even one), or, with 16 random bits per element,
    up where the place between the two codes plus bits / 2^16 reaches one.
    With bits = 5 a value above zero takes at least code 1."""
    x = np.asarray(x, np.float64)
    b = scale_byte(x, bits)
    unit = np.exp2(np.repeat(b, BLOCK)[:x.size] - 127.0)
    bad = np.repeat(b, BLOCK)[:x.size] == NAN_BYTE
    a = np.where(bad, 0.0, np.abs(x)) / unit
    mag = code_values(bits)[:128 if bits == M_BITS else 256]
    lo = np.clip(np.searchsorted(mag, a, side="right") - 1, 0, mag.size - 1)
    hi = np.minimum(lo + 1, mag.size - 1)
    gap = np.where(hi > lo, mag[hi] - mag[lo], 1.0)
    place = np.where(hi > lo, (a - mag[lo]) / gap, 0.0)
    if sixteen is None:
        up = (place > 0.5) | ((place == 0.5) & (lo % 2 == 1))
    else:
        up = place + np.asarray(sixteen, np.float64) / 65536.0 >= 1.0
    code = np.where(up, hi, lo)
    if bits == R_BITS:
        code = np.where((a > 0) & (code == 0), 1, code)
    else:
        code = code | np.where(np.signbit(x), 128, 0)
    return np.where(bad, 0, code).astype(np.uint8), b


# ---- random bits --------------------------------------------------------------

def mix32(x):
    with np.errstate(over="ignore"):
        x = np.asarray(x, dtype=np.uint32)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x57735285)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x4746E6A3)
        return x ^ (x >> np.uint32(16))


def random_words(seed: int, t: int, tensor: int, numel: int) -> np.ndarray:
    """32 random bits per element: the lower half rounds the first moment, the
    upper half the root."""
    u = np.uint32
    key = mix32(mix32(u(seed & 0xFFFFFFFF)) ^ u((seed >> 32) & 0xFFFFFFFF))
    key = mix32(mix32(key ^ u(t)) ^ u(tensor))
    i = np.arange(numel, dtype=np.int64)
    key = mix32(key ^ (i // BLOCK).astype(np.uint32))
    return mix32(key ^ (i % BLOCK).astype(np.uint32))


# ---- the step -----------------------------------------------------------------

def adamw_step(p, g, m, v, h, t: int, ema=None, ema_decay: float = 0.0,
               coef: float = 1.0, lr_scale: float = 1.0, wd_scale: float = 1.0):
    """(p', m', v', e') in 64 bits; h has lr, beta1, beta2, eps, weight_decay."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = coef * g
    m = h.beta1 * m + (1 - h.beta1) * g
    v = h.beta2 * v + (1 - h.beta2) * g * g
    lr, wd = h.lr * lr_scale, h.weight_decay * wd_scale
    mh, vh = m / (1 - h.beta1 ** t), v / (1 - h.beta2 ** t)
    p = p * (1 - lr * wd) - lr * mh / (np.sqrt(vh) + h.eps)
    e = None if ema is None else ema_decay * np.asarray(ema, np.float64) + (1 - ema_decay) * p
    return p, m, v, e


def moments_f32(g, m, v, h, coef=1.0, root=None):
    """(m', v', r') in 32 bits, each operation rounded in the library's order.
    root: the old second moment's root, in place of v."""
    f = np.float32
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        g = np.asarray(g, f) * f(coef)
        m = np.asarray(m, f) * f(h.beta1) + g * f(1 - h.beta1)
        v = np.asarray(root, f) * np.asarray(root, f) if root is not None else np.asarray(v, f)
        b2, omb2 = f(h.beta2), f(1 - h.beta2)
        v1 = v * b2 + (g * g) * omb2
        r = np.sqrt(v1)
        if root is not None:
            # roots whose squares leave fp32: from inputs scaled by a power of two
            for use, up in ((r < f(2.0 ** -49), f(2.0 ** 70)), (r > f(2.0 ** 63), f(2.0 ** -70))):
                a, b = np.asarray(root, f) * up, g * up
                r = np.where(use, np.sqrt((a * a) * b2 + (b * b) * omb2) * (1 / up), r)
        return m, v1, r


def codes_f32(x, bits: int, sixteen: Optional[np.ndarray] = None):
    """(codes, bytes) of 32-bit values: the top of the pattern of |x| scaled so
    that the codes' least normal value is fp32's, after rounding in it."""
    x = np.asarray(x, np.float32)
    low = 23 - bits
    big = np.max(np.abs(_blocks(x)).view(np.uint32), axis=1).astype(np.int64)
    b = np.maximum((big + (1 << low) - 1) >> 23, LOW)
    b = np.where(b > HIGH, NAN_BYTE, b)
    each = np.repeat(b, BLOCK)[:x.size]
    with np.errstate(under="ignore", over="ignore", invalid="ignore"):
        divisor = np.exp2(np.where(each == NAN_BYTE, 0, 119.0 - each)).astype(np.float32)
        a = np.abs(x) * divisor * np.float32(2.0 ** -112)
    w = a.view(np.uint32).astype(np.int64)
    if sixteen is None:
        w = w + (1 << (low - 1)) - 1 + ((w >> low) & 1)
    else:
        w = w + (np.asarray(sixteen, np.int64) << (low - 16))
    code = w >> low
    if bits == R_BITS:
        code = np.where((x > 0) & (code == 0), 1, code)
    else:
        code = code | np.where(np.signbit(x), 128, 0)
    return np.where(each == NAN_BYTE, 0, code).astype(np.uint8), b


def grad_norm(grads: Sequence[np.ndarray], max_norm: float):
    """(norm, coefficient) of all gradients together, in 64 bits."""
    total = math.fsum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads) \
        if all(np.all(np.isfinite(g)) for g in grads) else math.nan
    if not math.isfinite(total):
        bad = [np.asarray(g, np.float64) for g in grads]
        nan = any(np.any(np.isnan(g)) for g in bad)
        return (math.nan if nan else math.inf), math.nan
    norm = math.sqrt(total)
    return norm, min(1.0, max_norm / (norm + 1e-6))

"""Plain numpy forms of the operators over lists: the update in fp32 (each operation rounded, the order of
include/zero_shard.h) and in 64 bits, and the 8-bit codes from their definition.  Shares nothing with the library."""
from __future__ import annotations

import numpy as np

BLOCK, TILE = 256, 4096
TOP = {"m": 448.0, "v": 1.875}
SMALLEST_PEAK = 2.0**-110
MASK = (1 << 64) - 1
GOLDEN = 0x9E3779B97F4A7C15


def scalars(lr, beta1, beta2, eps, weight_decay, grad_scale, step):
    """The nine scalars in 64 bits."""
    return dict(b1=beta1, omb1=1 - beta1, b2=beta2, omb2=1 - beta2, eps=eps, decay=1 - lr * weight_decay,
                step_size=lr / (1 - beta1**step), bc2_sqrt=(1 - beta2**step) ** 0.5, gscale=grad_scale)


def adamw(g, p, m, v, s, dtype=np.float32):
    """New (p, m, v); every operation rounded to `dtype`."""
    s = {k: dtype(x) for k, x in s.items()}
    g, p, m, v = (np.asarray(x, dtype) for x in (g, p, m, v))
    with np.errstate(all="ignore"):
        g = s["gscale"] * g
        m = s["b1"] * m + s["omb1"] * g
        v = s["b2"] * v + s["omb2"] * (g * g)
        d = np.sqrt(v) / s["bc2_sqrt"] + s["eps"]
        return p * s["decay"] - s["step_size"] * (m / d), m, v


# ---------------------------------------------------------------------- 8-bit moments

def code_values():
    """What codes stand for without their scale, in 64 bits: ('m': 256 signed, NaN at 127 and 255; 'v': 256)."""
    c = np.arange(128)
    e, f = c >> 3, (c & 7).astype(np.float64)
    mag = np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 7), f / 8 * 2.0**-6)
    mag[127] = np.nan
    c = np.arange(256)
    e, f = c >> 3, (c & 7).astype(np.float64)
    return {"m": np.concatenate([mag, -mag]), "v": np.where(e > 0, (1 + f / 8) * 2.0 ** (e - 31), f / 8 * 2.0**-30)}


VALUES = code_values()


def decode(codes, scale, which):
    """fp32 values of whole blocks: codes [blocks, 256], scale [blocks]."""
    with np.errstate(all="ignore"):
        return VALUES[which][codes].astype(np.float32) * scale.astype(np.float32)[:, None]


def position(x, which):
    """Where |x| (fp32, scaled) lies among the codes, in 2^-20 of a step: exact for normal codes, to the nearest
    for subnormal ones."""
    low = -6 if which == "m" else -30  # exponent of the smallest normal code
    a = np.abs(x.astype(np.float64))
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 1, low), low)  # a in [2^e, 2^(e+1)), or subnormal
    steps = a / 2.0 ** (e - 3)               # in steps of this octave: 8 .. 16, or 0 .. 8
    return np.rint((steps + 8 * (e - low)) * 2.0**20).astype(np.int64)


def encode(x, which, dither):
    """(codes, scale) of fp32 blocks [blocks, 256]; dither in 2^-20 of a step."""
    x = np.asarray(x, np.float32)
    peak = np.abs(x).max(axis=1)
    some = ~(peak < np.float32(SMALLEST_PEAK))
    top = np.float32(TOP[which])
    with np.errstate(all="ignore"):
        scale = np.where(some, peak * (np.float32(1) / top), np.float32(0)).astype(np.float32)
        inv = np.where(some, top / peak, np.float32(0)).astype(np.float32)
        scaled = np.abs(x) * inv[:, None]
    most = 126 if which == "m" else 255
    good = np.isfinite(scaled)
    codes = np.where(good, (position(np.where(good, scaled, 0).astype(np.float32), which) + dither) >> 20, most)
    codes = np.minimum(codes, most)
    if which == "m":
        codes = codes | (np.signbit(x).astype(np.int64) << 7)
    else:
        with np.errstate(all="ignore"):
            codes = np.maximum(codes, ((x > 0) & some[:, None]).astype(np.int64))
    return codes.astype(np.uint8), scale


def mix64(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK
    return z ^ (z >> 31)


def dithers(seed, step, block0, blocks):
    """(m, v) dithers [blocks, 256] of the blocks numbered from block0."""
    base = mix64((seed + GOLDEN * step) & MASK)
    keys = np.array([mix64((base + GOLDEN * (block0 + b + 1)) & MASK) & 0xFFFFFFFF for b in range(blocks)], np.int64)
    r = (keys[:, None] + np.arange(BLOCK, dtype=np.int64) * 0x9E3779B9) & 0xFFFFFFFF
    return r >> 12, r & 0xFFFFF


def blocks_of(x):
    """A tensor's elements as whole blocks, zeros past its end."""
    n = x.size
    out = np.zeros((-(-n // BLOCK), BLOCK), x.dtype)
    out.reshape(-1)[:n] = x
    return out


class State8:
    """One tensor's 8-bit state: views into a byte buffer as the library lays it out."""

    def __init__(self, raw, n):
        self.raw, self.n = raw, n
        t = raw.reshape(-1, 6 * TILE + 8 * (TILE // BLOCK))
        a, k = 4 * TILE, TILE // BLOCK

        def floats(lo, cnt):
            return np.ascontiguousarray(t[:, lo:lo + 4 * cnt]).view(np.float32).reshape(-1)
        nb = -(-n // BLOCK)
        self.master = floats(0, TILE)[:n]
        self.m = np.ascontiguousarray(t[:, a:a + TILE]).reshape(-1, BLOCK)[:nb]
        self.v = np.ascontiguousarray(t[:, a + TILE:a + 2 * TILE]).reshape(-1, BLOCK)[:nb]
        self.scale_m = floats(a + 2 * TILE, k)[:nb]
        self.scale_v = floats(a + 2 * TILE + 4 * k, k)[:nb]

    def moments(self):
        """fp32 (m, v), n elements each."""
        return (decode(self.m, self.scale_m, "m").reshape(-1)[:self.n],
                decode(self.v, self.scale_v, "v").reshape(-1)[:self.n])


def adamw8(g, st, s, seed, step, block0):
    """(p, m codes, v codes, m scales, v scales) after one step of a tensor; codes as whole blocks."""
    m0, v0 = st.moments()
    p, m, v = adamw(g, st.master, m0, v0, s)
    dm, dv = dithers(seed, step, block0, len(st.m))
    cm, sm = encode(blocks_of(m), "m", dm)
    cv, sv = encode(blocks_of(v), "v", dv)
    return p, cm, cv, sm, sv

"""Float64 NumPy model of the rotary and paged-cache operators, from their definitions in include/spa.h.
Written apart from the kernels: byte tables and loops, no shared code."""
import math

import numpy as np

D = 128


def frequencies(rot, theta=500000.0, scaling="plain", factor=1.0, low=1.0, high=4.0, orig_ctx=0, **_):
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "bands":
        k = np.clip((orig_ctx * f / (2 * math.pi) - low) / (high - low), 0, 1)
        f = f * (k + (1 - k) / factor)
    if scaling == "ramp":
        n = lambda turns: rot * math.log(orig_ctx / (2 * math.pi * turns)) / (2 * math.log(theta))
        a, b = (min(max(x, 0), rot - 1) for x in (math.floor(n(high)), math.ceil(n(low))))
        b = b if b > a else a + 0.001
        k = np.clip(1 - (np.arange(rot // 2) - a) / (b - a), 0, 1)
        f = f * (k + (1 - k) / factor)
    return f


def rotate(x, pos, rot, layout="half", magnitude=1.0, transpose=False, **freq):
    """x [..., d] float64, pos broadcast over the leading dims."""
    a = np.asarray(pos, np.float64)[..., None] * frequencies(rot, **freq)
    c, s = magnitude * np.cos(a), magnitude * np.sin(a) * (-1 if transpose else 1)
    i = np.arange(rot // 2)
    u, v = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y = np.array(x, np.float64)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def rne_bf16(x):
    """float64 values rounded to 8 significant bits, ties to even (subnormals of bf16 are not met)."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.round(m * 256), e - 8)


GROUP_K, GROUP_V = (np.arange(D) // 8) % 4, (np.arange(D) // 4) % 4
TINY = 2.0 ** -110


def quantise(x, group):
    """x [..., 128] float64 -> codes uint8 [..., 128] (1..15), scales float64 [..., 4] (NaN for non-finite groups)."""
    x = np.asarray(x, np.float64)
    codes = np.full(x.shape, 8, np.uint8)
    scales = np.zeros(x.shape[:-1] + (4,))
    for g in range(4):
        v = x[..., group == g]
        with np.errstate(all="ignore"):
            bad = ~np.isfinite(v).all(-1)
            amax = np.abs(v).max(-1)
            s = np.where(bad, np.nan, np.where(amax < TINY, 0.0, rne_bf16(np.where(bad, 1.0, amax) / 7)))
            ok = (s > 0) & ~bad
            n = np.clip(np.round(np.where(ok[..., None], v, 0.0) / np.where(ok, s, 1.0)[..., None]), -7, 7)
        codes[..., group == g] = (n + 8).astype(np.uint8)
        scales[..., g] = s
    return codes, scales


def bf16_bits(x):
    """bits of values that bf16 holds exactly (NaN: 0x7fc0)."""
    x = np.asarray(x, np.float64)
    b = (np.where(np.isnan(x), 0.0, x).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7fc0), b)


def bf16_values(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def block_bytes(fmt):
    return 2304 if fmt == "int4" else 8192


class Pool:
    """The bytes of a pool, [n_pages][Hkv][blocks][block]."""

    def __init__(self, data, fmt, page):
        self.data, self.fmt, self.page = data, fmt, page

    def block(self, page_id, g, r):
        return self.data[page_id, g, r // 16], r % 16

    def put(self, table, b, g, pos, k, v):
        """Stores one row pair given as float64 (already rotated)."""
        blk, r = self.block(table[b, pos // self.page], g, pos % self.page)
        if self.fmt == "int4":
            for part, x, group in ((0, k, GROUP_K), (1, v, GROUP_V)):
                c, s = quantise(x, group)
                blk[1024 * part + 64 * r:1024 * part + 64 * r + 64] = c[0::2] | (c[1::2] << 4)
                at = 2048 + 16 * r + 8 * part
                blk[at:at + 8] = bf16_bits(s).astype("<u2").view(np.uint8)
        else:
            for part, x in ((0, k), (1, v)):
                bits = bf16_bits(rne_bf16(x)).astype("<u2").view(np.uint8).reshape(16, 16)
                for c in range(16):
                    at = 4096 * part + 256 * r + 16 * (c ^ (r % 8))
                    blk[at:at + 16] = bits[c]

    def get(self, table, b, g, pos):
        """(k, v) float64 of one row pair."""
        blk, r = self.block(table[b, pos // self.page], g, pos % self.page)
        out = []
        for part, group in ((0, GROUP_K), (1, GROUP_V)):
            if self.fmt == "int4":
                w = blk[1024 * part + 64 * r:1024 * part + 64 * r + 64]
                n = np.stack((w & 15, w >> 4), -1).reshape(-1).astype(np.float64) - 8
                at = 2048 + 16 * r + 8 * part
                s = bf16_values(blk[at:at + 8].view("<u2"))
                with np.errstate(all="ignore"):
                    out.append(n * s[group])
            else:
                row = blk[4096 * part + 256 * r:4096 * part + 256 * r + 256].reshape(16, 16)
                out.append(bf16_values(np.concatenate([row[c ^ (r % 8)] for c in range(16)]).view("<u2")))
        return out

    def rows(self, table, b, g, positions):
        kv = [self.get(table, b, g, int(p)) for p in positions]
        return (np.array([k for k, _ in kv]).reshape(-1, D), np.array([v for _, v in kv]).reshape(-1, D))


def attended(L, ret, lists, n_sink, window, masked):
    """Positions one KV head attends (with repetition, in list order)."""
    if not masked or (ret and lists is None):
        return list(range(L))
    n_s = min(n_sink, L)
    rows = list(range(n_s)) + list(range(max(n_s, L - window), L))
    return rows + (list(lists) if ret else [])


def attend(q, k, v):
    """q [G][128], k, v [n][128] -> out [G][128], log2 of the denominator, and a bound of the kernel's error.

    The bound: queries and probabilities are kept as a bf16 and its bf16 residual, each half off by
    at most 2^-9 of it, together 2^-18; float32 sums of 128 products add 2^-24 each in the worst case, 2^-19 with
    room.  So a score is off by at most 2^-17 sum |q k| / sqrt(128) (ln units), a probability's weight by twice
    the largest of those, relative, plus 2^-17 for the exponential, its rounding and the sums."""
    if len(k) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf), np.zeros(q.shape)
    s = q @ k.T / math.sqrt(D)
    off = (np.abs(q) @ np.abs(k).T / math.sqrt(D)).max(-1) * 2.0 ** -17
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    z = p.sum(-1, keepdims=True)
    out = p @ v / z
    bound = (2 * off[:, None] + 2.0 ** -15) * (p @ np.abs(v) / z)
    return out, ((m + np.log(z)) / math.log(2.0))[:, 0], bound

"""Plain references for the 4-bit cache and the rotary positions: numpy, binary32 where the definition says so, binary64
elsewhere.  Nothing here uses the CUDA path."""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
f32 = np.float32


def e4m3_values() -> np.ndarray:
    """The 128 non-negative E4M3 codes' values (0x7F: NaN)."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return v


def _nearest_even(x, grid):
    """Index of the grid value nearest to x >= 0; ties to the even index; beyond the grid, its last."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(grid, x, side="left"), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(x >= grid[-1], len(grid) - 1, pick)


def e4m3_encode(x) -> np.ndarray:
    """Non-negative values (binary32) -> E4M3 codes, saturating at 448 (code 126); NaN -> 127."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    code = _nearest_even(np.where(nan, 0.0, x), e4m3_values()[:127])
    return np.where(nan, 127, code).astype(np.uint8)


def quantize(x, scale):
    """x [..., D] (binary32 values) -> codes [..., D] 0..15, block scale codes [..., D / 16]."""
    scale = f32(scale)
    with np.errstate(all="ignore"):
        x = np.asarray(x, f32)
        blocks = x.reshape(*x.shape[:-1], -1, 16)
        a = np.abs(blocks).max(-1)                       # NaN if any is
        b = e4m3_encode((a / f32(f32(6.0) * scale)).astype(f32))
        d = (e4m3_values()[b].astype(f32) * scale).astype(f32)
        r = np.where(b == 0, f32(0), f32(1) / d).astype(f32)
        y = (blocks * r[..., None]).astype(f32)
    mag = np.where(np.isnan(y), 6.0, np.abs(y))
    code = _nearest_even(mag, E2M1) + 8 * np.signbit(y)
    return code.reshape(x.shape).astype(np.uint8), b


def values(codes, b):
    """codes [..., D], block scale codes [..., D / 16] -> E2M1 * b in binary64 (without the layer's scale)."""
    v = np.where(codes >= 8, -1.0, 1.0) * E2M1[codes & 7]
    full = np.concatenate([e4m3_values(), -e4m3_values()])
    return v * np.repeat(full[b], 16, -1)


def unpack(pool, D):
    """A pool [P, Hkv, 9 D / 4] -> codes [P, Hkv, 4, D], scale codes [P, Hkv, 4, D / 16]."""
    raw = pool[..., :2 * D].reshape(*pool.shape[:2], 4, D // 2)
    codes = np.stack((raw & 15, raw >> 4), -1).reshape(*pool.shape[:2], 4, D)
    b = pool[..., 2 * D:].reshape(*pool.shape[:2], D // 16, 4).swapaxes(-1, -2)
    return codes, b


def append(pool, x, slots, scale):
    """Write rows x [T, Hkv, D] into a copy of the pool."""
    pool = pool.copy()
    D = x.shape[-1]
    codes, b = quantize(x, scale)
    for i, s in enumerate(slots):
        if s < 0 or s // 4 >= pool.shape[0]:
            continue
        page = pool[s // 4]
        page[:, (s % 4) * D // 2:(s % 4 + 1) * D // 2] = codes[i, :, 0::2] | (codes[i, :, 1::2] << 4)
        page[:, 2 * D + (s % 4)::4] = b[i]
    return pool


def pool_values(pool, D):
    codes, b = unpack(pool, D)
    return values(codes, b)


def rope_table(n, rot, base=10000.0, scaling=None, factor=1.0, original=0, fast=32.0, slow=1.0, magnitude=0.0):
    j = np.arange(rot // 2)
    f = base ** (-2.0 * j / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        d = lambda beta: rot * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), rot - 1)
        r = np.clip((j - low) / (high - low if high > low else 0.001), 0, 1)
        f = f * (1 - r) + f / factor * r
        magnitude = magnitude or 0.1 * math.log(factor) + 1
    magnitude = magnitude or 1.0
    angle = np.arange(n)[:, None] * f
    return np.concatenate((np.cos(angle), np.sin(angle)), -1) * magnitude


def rotate(x, table, positions, interleaved):
    """x [T, H, D] fp16, table [N, rot] binary32 -> binary32, every product and sum rounded."""
    rot = table.shape[1]
    c, s = (np.ascontiguousarray(h)[:, None].astype(f32) for h in np.split(table[positions], 2, -1))
    x = np.asarray(x, f32)
    y = x.copy()
    a, b = ((x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot]))
    y1 = ((a * c).astype(f32) - (b * s).astype(f32)).astype(f32)
    y2 = ((b * c).astype(f32) + (a * s).astype(f32)).astype(f32)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = y1, y2
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = y1, y2
    return y


def attend(q, K, V, sm):
    """One query row over keys K [n, D], values V [n, D] in binary64.  Returns the output and how far the kernel's may be
    from it: P rounded to fp16 (half a step, 2^-11, and 2^-25 where it is subnormal) against sum p |V|; the scores'
    binary32 sums of D products (at most 2^-20 of the sum of their magnitudes, which moves p and its sum); the exponentials
    and the binary32 sums over tokens and splits (2^-16); the output's own rounding (2^-11, 2^-25 where subnormal)."""
    n, D = K.shape
    if n == 0:
        return np.zeros(D), np.zeros(D)
    q = np.asarray(q, np.float64)
    s = K @ q * sm
    p = np.exp(s - s.max())
    l = p.sum()
    out = p @ V / l
    e_s = 2.0 ** -20 * (np.abs(K) @ np.abs(q)).max() * sm
    spread = p @ np.abs(V) / l
    tol = spread * (2.0 ** -11 + 2 * e_s + 2.0 ** -16) + np.abs(out) * 2.0 ** -11 + n * 2.0 ** -25 * np.abs(V).max(0) + 2.0 ** -25
    return out, tol


def decode(q, kc, vc, bt, lens, ks, vs, topk_idx=None, topk_lens=None, sm=None):
    """Decode / verify attention over E2M1 pools: out and tolerance [B, n, Hq, D], and the KVQ_DEV_* bits."""
    B, n, Hq, D = q.shape
    P, Hkv = kc.shape[:2]
    K, V = pool_values(kc, D) * float(f32(ks)), pool_values(vc, D) * float(f32(vs))
    sm = 1 / math.sqrt(D) if sm is None else sm
    out, tol, flags = np.zeros(q.shape), np.zeros(q.shape), 0
    for b in range(B):
        L = int(lens[b])
        if L < n or L > 4 * bt.shape[1]:
            flags |= 8
            continue
        for g in range(Hkv):
            if topk_idx is not None and topk_lens[b] > 0:
                pos = topk_idx[b, g, :topk_lens[b]].astype(np.int64)
                if topk_lens[b] > topk_idx.shape[2] or ((pos < 0) | (pos >= L)).any():
                    flags |= 4
                pos = pos[(pos >= 0) & (pos < L)]
            else:
                pos = np.arange(L)
            page = bt[b, pos // 4].astype(np.int64)
            ok = (page >= 0) & (page < P)
            if not ok.all():
                flags |= 1
            pos, page = pos[ok], page[ok]
            k, v = K[page, g, pos % 4], V[page, g, pos % 4]
            for i in range(n):
                see = pos <= L - n + i
                for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
                    out[b, i, h], tol[b, i, h] = attend(q[b, i, h], k[see], v[see], sm)
    return out, tol, flags


def close(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    off = np.abs(got - ref)
    bad = ~(off <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside their tolerance, worst {np.nanmax(off / np.maximum(tol, 1e-30)):.3g} "
                           f"of it, first at {tuple(np.argwhere(bad)[0])}: {got[tuple(np.argwhere(bad)[0])]} for {ref[tuple(np.argwhere(bad)[0])]}")

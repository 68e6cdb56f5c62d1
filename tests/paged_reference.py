"""Plain 64-bit forms of the paged-cache operators, written from their
definitions (numpy only; nothing here imports the package)."""
from __future__ import annotations

import math

import numpy as np

GROUP, TILE = 32, 64


# ------------------------------------------------------------------- bf16
def bf16_bits(x):
    """Round-to-nearest-even bf16 bits of float32 values."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = (u + 0x7FFF + ((u >> 16) & 1)) >> 16
    nan = np.isnan(x)
    return np.where(nan, 0x7FFF, r).astype(np.uint16)


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32)


def bf16_toward(x, up):
    """The bf16 value next to a 64-bit one on the given side (finite, normal)."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    ulp = np.ldexp(1.0, np.maximum(e - 8, -133))
    return (np.ceil(x / ulp) if up else np.floor(x / ulp)) * ulp


# --------------------------------------------------------------- rotation
def frequencies(rot, base, scaling="plain", factor=1.0, slow=1.0, fast=4.0, original=0.0):
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "bands":
        out = []
        for x in f:
            turns = original * x / (2 * math.pi)
            if turns <= slow:
                out.append(x / factor)
            elif turns >= fast:
                out.append(x)
            else:
                s = (turns - slow) / (fast - slow)
                out.append((1 - s) * x / factor + s * x)
        f = out
    if scaling == "yarn":
        dim = lambda n: rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), rot - 1)
        out = []
        for i, x in enumerate(f):
            r = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            out.append(x / factor * r + x * (1 - r))
        f = out
    return f


def angles(pos, turns):
    """Radians in [0, 2 pi) of integer positions and 2^-64-turn frequencies,
    by exact integer arithmetic."""
    a = [[((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64 for t in turns] for p in pos]
    return 2 * math.pi * np.array(a, np.float64).reshape(len(pos), len(turns))


def rotated(x, pos, turns, interleaved, attn=1.0, weight=None, eps=0.0):
    """[T, H, d] -> (norm and rotation in 64 bits, a bound on the sum of the
    magnitudes that enter each value)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    rot = 2 * len(turns)
    if rot:
        a = angles(pos, turns)[:, None, :]
        c, s = attn * np.cos(a), attn * np.sin(a)
        i = np.arange(rot // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ia] * s + x[..., ib] * c
        mag[..., ia] = mag[..., ib] = attn * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    return y, mag


# ------------------------------------------------------------ 4-bit records
def quantise(x):
    """[..., d] 64-bit -> codes, scales, minima ([..., d], [..., d / 32] x 2)."""
    y = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, GROUP)
    mn = bf16_toward(y.min(-1), up=False)
    sc = bf16_toward((y.max(-1) - mn) / 15, up=True)
    sc = np.where(sc > 0, np.maximum(sc, 2.0 ** -126), sc)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.rint((y - mn[..., None]) / sc[..., None])
    n = np.where(sc[..., None] > 0, np.clip(n, 0, 15), 0)
    return n.reshape(x.shape).astype(np.int64), sc, mn


def code_places(d, value):
    """Byte and nibble of each (row, column) code in a 16-row record."""
    r, e = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    if value:
        byte = ((r // 8) * 32 + (e % 32) // 4 * 4 + (r // 2) % 4) * (d // 8) + 4 * (e // 32) + 2 * (r % 2)
        nib = e % 4
    else:
        m, i = e // 8, e % 8
        byte = r * (d // 2) + 4 * ((m % 4) * (d // 32) + m // 4)
        nib = i // 2 + 4 * (i % 2)
    return byte + nib // 2, nib % 2


def unpack(rec, d, value):
    """[..., 10 d] uint8 records -> (codes, scales, minima) [..., 16, ...]."""
    byte, hi = code_places(d, value)
    codes = (rec[..., byte] >> (4 * hi)) & 15
    par = rec[..., 8 * d:].copy().view(np.uint16).reshape(*rec.shape[:-1], 16, d // GROUP, 2)
    return codes.astype(np.int64), bf16_value(par[..., 0]), bf16_value(par[..., 1])


def pack(codes, sc, mn, value):
    """[..., 16, d] codes and their groups' (sc, mn) -> records."""
    d = codes.shape[-1]
    rec = np.zeros((*codes.shape[:-2], 10 * d), np.uint8)
    byte, hi = code_places(d, value)
    for h in (0, 1):  # the two nibbles of a byte never meet in one assignment
        at = hi == h
        np.bitwise_or.at(rec, (..., byte[at]), (codes[..., at] << (4 * h)).astype(np.uint8))
    par = np.stack([bf16_bits(sc), bf16_bits(mn)], -1)
    rec[..., 8 * d:] = np.ascontiguousarray(par).view(np.uint8).reshape(*rec.shape[:-1], -1)
    return rec


def record_values(rec, d, value):
    codes, sc, mn = unpack(rec, d, value)
    rep = lambda x: np.repeat(x.astype(np.float64), GROUP, -1)  # noqa: E731
    return rep(mn) + rep(sc) * codes


def cache_rows(pages, table_row, n, h, d, value):
    """The first n rows of one head of a sequence in 64 bits [n, d]."""
    if pages.dtype == np.uint8:
        P = pages.shape[2] * 16
        ids = table_row[:-(-n // P)]
        return record_values(pages[ids, h], d, value).reshape(-1, d)[:n]
    P = pages.shape[2]
    ids = table_row[:-(-n // P)]
    return pages[ids, h].astype(np.float64).reshape(-1, d)[:n]


# ------------------------------------------------------------------ decode
def decode(q, k_pages, v_pages, table, lens, scale, tsf, splits, tiles=None):
    """The rule, tile after tile, in 64 bits. bf16 pages come as float arrays,
    4-bit ones as uint8 records. `tiles` [B, Hkv, n] replays given decisions
    (1 kept, 2 skipped). Returns o, lse, tile_state, margin (ln t minus the
    decision quantity's largest; the decision flips where it crosses 0),
    the mass sum_k P |v| of each output, and sum |q k| scale of each head."""
    B, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    G = Hq // Hkv
    P = k_pages.shape[2] * (16 if k_pages.dtype == np.uint8 else 1)
    n_tiles = -(-table.shape[1] * P // TILE)
    o, mass = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse, size = np.full((B, Hq), -np.inf), np.zeros((B, Hq))
    state = np.zeros((B, Hkv, n_tiles), np.uint8)
    margin = np.full((B, Hkv, n_tiles), np.nan)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        nk = -(-n // TILE)
        per = -(-nk // splits)
        ln_t = math.log(tsf / n) if tsf > 0 else -math.inf
        for h in range(Hkv):
            K = cache_rows(k_pages, table[b], n, h, d, False)
            V = cache_rows(v_pages, table[b], n, h, d, True)
            Q = q[b, h * G:(h + 1) * G].astype(np.float64)
            s = scale * (Q @ K.T)
            keep = np.zeros(n, bool)
            for j in range(nk):
                if j % per == 0:
                    run = np.full(G, -np.inf)
                local = s[:, j * TILE:(j + 1) * TILE].max(1)
                gap = np.where(run == -np.inf, np.inf, local - run)
                margin[b, h, j] = ln_t - gap.max()
                skip = bool((gap < ln_t).all())
                if tiles is not None:
                    skip = tiles[b, h, j] == 2
                state[b, h, j] = 2 if skip else 1
                if not skip:
                    run = np.maximum(run, local)
                    keep[j * TILE:(j + 1) * TILE] = True
            s = np.where(keep, s, -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p = p / l
            Vk = np.where(keep[:, None], V, 0.0)
            rows = slice(h * G, (h + 1) * G)
            o[b, rows] = p @ Vk
            mass[b, rows] = p @ np.abs(Vk)
            if k_pages.dtype == np.uint8:  # codes and minima are summed apart
                codes, sc, mn = unpack(v_pages[table[b, :-(-n // P)], h], d, True)
                rep = lambda x: np.repeat(np.abs(x.astype(np.float64)), GROUP, -1).reshape(-1, d)[:n]  # noqa: E731
                parts = rep(sc) * 8 + rep(mn + 8 * sc)
                mass[b, rows] = p @ np.where(keep[:, None], parts, 0.0)
            lse[b, rows] = (m + np.log(l))[:, 0]
            size[b, rows] = scale * (np.abs(Q) @ np.abs(K).T).max(1)
            if k_pages.dtype == np.uint8:
                codes, sc, mn = unpack(k_pages[table[b, :-(-n // P)], h], d, False)
                rep = lambda x: np.repeat(np.abs(x.astype(np.float64)), GROUP, -1).reshape(-1, d)[:n]  # noqa: E731
                size[b, rows] = scale * (np.abs(Q) @ (rep(sc) * 8 + rep(mn + 8 * sc)).T).max(1)
    return {"o": o, "lse": lse, "tile_state": state, "margin": margin, "mass": mass, "size": size}


def decode_tolerance(ref, n_max):
    """Bounds on |o - o_ref| [B, Hq, d] and |lse - lse_ref| [B, Hq].

    A score is an fp32 sum of d exact products (in the 4-bit form of at most
    d / 32 + d of them) whose absolute values add up to `size`: with at most
    2^-22 of that size lost in each of the few roundings of a tensor-core chain
    and of the scaling, ds = 2^-19 size bounds its error (d = 128: 8 chained
    products and 8 scale steps, each at most 2^-22 with truncation), plus
    2^-22 of the exponent for exp2's argument and result (|s - m| < 150 where
    P does not vanish: 2^-22 * 150 < 2^-14 only for weights below e^-100, so
    2^-20 covers the weights that count). A weight is then off by 2 (ds +
    2^-20) relative (numerator and denominator), rounded to bf16 by half a step
    2^-8 / (1 - 2^-8), and o itself by another half step. Sums over n keys in
    fp32 and the splits' merge lose at most (n / 64 + 64) 2^-24 of the mass
    (a warp's chain adds one product a tile)."""
    ds = ref["size"] * 2.0 ** -19 + 2.0 ** -20
    chain = (n_max / 64 + 64) * 2.0 ** -24
    half = 2.0 ** -8 * (1 + 2.0 ** -7)
    o = half * np.abs(ref["o"]) + (half + 2 * ds[..., None] + chain) * ref["mass"] + 1e-30
    lse = ds + chain + np.abs(ref["lse"]) * 2.0 ** -22 + 2.0 ** -20
    return o, lse

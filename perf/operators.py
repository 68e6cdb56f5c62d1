"""What the paged key/value cache and the attention over it cost.

The operators: norm + rotation of queries and keys with the append to a paged
cache (bf16 or 4-bit pages), reading rows back out of the cache, and the
split-KV Skip-Softmax decode over the paged cache.  With ``own`` false,
``run`` computes them with elementary torch operations; with ``own`` true it
makes the library's calls.
"""
import math

import torch

own = False

GROUP = 32   # values that share a scale and a minimum in a 4-bit page
TILE = 64    # keys of a decode tile
DEV = "cuda"

#: name, then what a case is: op, sizes, page size, cache format, rotation.
_APPEND = dict(op="append", B=1, T=1, Hq=32, Hkv=8, d=128, page=64, fmt="bf16", pos_hi=16384,
               rot=128, interleaved=False, scaling="none", norm=True, outs=False, pad=0)
_DECODE = dict(op="decode", B=1, Hq=32, Hkv=8, d=128, page=64, fmt="bf16", len_lo=1000,
               len_hi=1000, tsf=0.0, splits=1)


def listed():
    return [
        # One sequence, one new token: the latency of a single-user decode step.
        dict(_APPEND, name="append bf16 1 token"),
        # The batch of the decode workload (64 sequences at 16K to 32K): one token each.
        dict(_APPEND, name="append bf16 64 tokens", B=64, T=64, pos_hi=32768, norm=False,
             scaling="bands"),
        # A whole 16K prompt: rotated q, k, v for the prefill kernel, and the cache filled.
        dict(_APPEND, name="append bf16 16K prompt", T=16384, outs=True, norm=False,
             scaling="bands"),
        # Ragged chunks of a d = 64 model, part of the head rotated in
        # interleaved pairs, short pages, padding tokens behind the last sequence.
        dict(_APPEND, name="append bf16 ragged d64", B=3, T=1237, Hq=16, Hkv=4, d=64, page=16,
             pos_hi=3000, rot=32, interleaved=True, pad=29),
        # One token each of 64 sequences into 4-bit pages, and the rows read back.
        dict(_APPEND, name="append 4bit 64 tokens", B=64, T=64, fmt="q4", pos_hi=32768,
             scaling="yarn"),
        # A chunk of prompts into 4-bit pages, and the rows read back.
        dict(_APPEND, name="append 4bit 1021 tokens", B=2, T=1021, fmt="q4", pos_hi=9000,
             page=32),
        # A short single-user context: latency.
        dict(_DECODE, name="decode bf16 B1 1000", splits=8),
        # The repository's decode workload (64 sequences of 16K to 32K), its factor 500.
        dict(_DECODE, name="decode bf16 B64 16K-32K", B=64, len_lo=16384, len_hi=32768, tsf=500.0,
             splits=16),
        # Ragged batch of a d = 64 model with 8 query heads per kv head and short pages.
        dict(_DECODE, name="decode bf16 ragged d64", B=7, Hq=16, Hkv=2, d=64, page=16, len_lo=1,
             len_hi=5003, splits=16),
        # One sequence of 128K tokens in 4 bits, 64 query heads over 8 kv heads.
        dict(_DECODE, name="decode 4bit B1 128K", Hq=64, fmt="q4", len_lo=131072, len_hi=131072,
             splits=64),
        # The decode workload in 4 bits.
        dict(_DECODE, name="decode 4bit B64 16K-32K", B=64, fmt="q4", len_lo=16384, len_hi=32768,
             tsf=500.0, splits=16),
        # A small ragged batch in 4 bits, d = 64, two query heads per kv head.
        dict(_DECODE, name="decode 4bit ragged d64", B=3, Hq=8, Hkv=4, d=64, fmt="q4", page=32,
             len_lo=17, len_hi=2049, tsf=4.0, splits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 8])
    fmt = rng.choice(["bf16", "q4"])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.5:
        b = _log_int(rng, 1, 64)
        t = b * rng.choice([1, 1, _log_int(rng, 1, max(1, (1000 if fmt == "q4" else 16000) // b))])
        pad = rng.choice([0, rng.randrange(1, 40)])
        return dict(op="append", B=b, T=t + pad, Hq=hkv * g, Hkv=hkv, d=d, page=page, fmt=fmt,
                    pos_hi=max(t, _log_int(rng, 64, 131072)), rot=rng.choice([16, 32, 48, d // 2, d]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                    norm=rng.random() < 0.5, outs=False, pad=pad)
    b = _log_int(rng, 1, 64)
    hi = _log_int(rng, 2, min(131072, 700000 // b))
    return dict(op="decode", B=b, Hq=hkv * g, Hkv=hkv, d=d, page=page, fmt=fmt,
                len_lo=rng.randrange(1, hi + 1), len_hi=hi,
                tsf=rng.choice([0.0, 0.5, 0.01]), splits=_log_int(rng, 1, 64))


# ------------------------------------------------------------------ inputs
def frequencies(rot, scaling, base=500000.0):
    """Radians per position of each pair, in 64 bits, and the factor on cos
    and sin: the four scalings for long contexts the library knows."""
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    attn = 1.0
    if scaling == "linear":
        freq = [f / 4.0 for f in freq]
    elif scaling == "bands":
        # slow pairs by 1 / 8, fast ones kept, a blend between wavelengths
        # of a quarter of the original context and all of it
        def band(f):
            wavelengths = 8192.0 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (wavelengths - 1.0) / (4.0 - 1.0)))
            return f * (keep + (1 - keep) / 8.0)
        freq = [band(f) for f in freq]
    elif scaling == "yarn":
        # the same idea as a ramp over the pair's index between 32 turns and
        # 1 turn over the original context of 4096, and a warmer softmax
        def pair(turns):
            return rot * math.log(4096.0 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(math.floor(pair(32.0)), 0)
        hi = min(math.ceil(pair(1.0)), rot - 1)
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        freq = [f * (1 - r) + f / 8.0 * r for f, r in zip(freq, ramp)]
        attn = 0.1 * math.log(8.0) + 1.0
    return freq, attn


def record(d):
    """Bytes of 16 keys (or values) of one head in a 4-bit page: codes, then
    one bf16 scale and one bf16 minimum for each group."""
    return 16 * (d // 2) + 16 * (d // GROUP) * 4


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tokens(case):
    """How many tokens of the call belong to sequences, as a list for each one."""
    n, b = case["T"] - case["pad"], case["B"]
    return [n // b + (i < n % b) for i in range(b)]


def _lengths(case):
    lo, hi, b = case["len_lo"], case["len_hi"], case["B"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _empty_pages(case, num_pages, g):
    """Pages with what earlier sequences left in them."""
    hkv, page, d = case["Hkv"], case["page"], case["d"]
    if case["fmt"] == "bf16":
        return torch.randn(num_pages, hkv, page, d, device=DEV, generator=g, dtype=torch.bfloat16)
    return _random_q4(num_pages, hkv, page, d, g)


def _random_q4(num_pages, hkv, page, d, g):
    ng = d // GROUP
    rec = torch.empty(num_pages, hkv, page // 16, record(d), dtype=torch.uint8, device=DEV)
    rec[..., :8 * d] = torch.randint(0, 256, (num_pages, hkv, page // 16, 8 * d), device=DEV,
                                     generator=g, dtype=torch.uint8)
    sc = torch.rand(num_pages, hkv, page // 16, 16, ng, device=DEV, generator=g) * 0.1 + 0.15
    sc = sc.bfloat16()
    mn = (-7.5 * sc.float() + 0.2 * torch.randn(sc.shape, device=DEV, generator=g)).bfloat16()
    rec[..., 8 * d:] = torch.stack([sc, mn], -1).flatten(-3).view(torch.uint8)
    return rec


def prepare(case, seed):
    g = _generator(seed)
    return (_prepare_append if case["op"] == "append" else _prepare_decode)(case, g, seed)


def _prepare_append(case, g, seed):
    B, T, Hq, Hkv, d, page = (case[n] for n in ("B", "T", "Hq", "Hkv", "d", "page"))
    counts = _tokens(case)
    r = torch.Generator().manual_seed(seed)
    seq, pos = [], []
    for b, n in enumerate(counts):  # each sequence's new tokens follow what it has already
        start = int(torch.randint(0, case["pos_hi"] - n + 1, (1,), generator=r))
        seq += [b] * n
        pos += range(start, start + n)
    seq += [-1] * case["pad"]
    pos += [0] * case["pad"]
    max_pages = -(-case["pos_hi"] // page)
    used = sorted({(s, p // page) for s, p in zip(seq, pos) if s >= 0})
    num_pages = sum(n // page + 2 for n in counts) + 3  # whatever the starts
    perm = torch.randperm(num_pages, generator=r)
    table = torch.zeros(B, max_pages, dtype=torch.int32)
    for n, (s, j) in enumerate(used):
        table[s, j] = perm[n]
    # the projection's output, one row for each token
    qkv = torch.randn(T, (Hq + 2 * Hkv) * d, device=DEV, generator=g).bfloat16()
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    freq, attn = frequencies(case["rot"], case["scaling"])
    out_len = T if case["outs"] else 1
    heads = lambda h: torch.zeros(T // out_len, h, out_len, d, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    weight = lambda: (1 + 0.1 * torch.randn(d, device=DEV, generator=g)).bfloat16()  # noqa: E731
    st = dict(case=case, q=q, k=k, v=v, out_len=out_len, attn=attn,
              seq=torch.tensor(seq, dtype=torch.int32, device=DEV),
              pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
              table=table.to(DEV),
              freq=torch.tensor(freq, dtype=torch.float64, device=DEV),
              # the same frequencies as the library keeps them: 2^-64 turns
              turns=torch.tensor([int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in freq],
                                 dtype=torch.int64, device=DEV),
              qw=weight() if case["norm"] else None, kw=weight() if case["norm"] else None,
              eps=1e-6, q_out=heads(Hq),
              k_out=heads(Hkv) if case["outs"] else None,
              v_out=heads(Hkv) if case["outs"] else None,
              k_pages=_empty_pages(case, num_pages, g), v_pages=_empty_pages(case, num_pages, g))
    if case["fmt"] == "q4":  # where the rows come back
        st["k_rows"], st["v_rows"] = heads(Hkv), heads(Hkv)
    return st


def _prepare_decode(case, g, seed):
    B, Hq, Hkv, d, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    lens = _lengths(case)
    r = torch.Generator().manual_seed(seed)
    lens = [lens[i] for i in torch.randperm(B, generator=r).tolist()]
    need = [-(-n // page) for n in lens]
    num_pages = sum(need) + 3
    perm = torch.randperm(num_pages, generator=r).int()
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    table = table.to(DEV)
    # One direction that queries and the keys of some tiles share (constant in
    # a group, so that both formats can hold it): attention sinks and hot tiles.
    sign = torch.randint(0, 2, (d // GROUP,), device=DEV, generator=g) * 2.0 - 1
    u = sign.repeat_interleave(GROUP)
    q = (torch.randn(B, Hq, d, device=DEV, generator=g) + 0.5 * u).bfloat16()
    tiles = -(-max(lens) // TILE)
    hot = torch.rand(B, Hkv, tiles, device=DEV, generator=g) < 0.15
    gain = 2.0 * hot.repeat_interleave(TILE, 2).float()  # for each key [B, Hkv, L]
    gain[..., :4] = 3.0
    n_keys = table.shape[1] * page
    gain = torch.nn.functional.pad(gain, (0, max(0, n_keys - gain.shape[2])))[..., :n_keys]
    gain = gain.unflatten(2, (-1, page)).transpose(1, 2)  # [B, max_pages, Hkv, page]
    owner = torch.arange(table.shape[1], device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    by_page = torch.zeros(num_pages, Hkv, page, device=DEV)
    by_page[table[owner].long()] = gain[owner]
    if case["fmt"] == "bf16":
        k_pages = torch.randn(num_pages, Hkv, page, d, device=DEV, generator=g, dtype=torch.bfloat16)
        k_pages.addcmul_(by_page.bfloat16()[..., None], u.bfloat16())
        v_pages = torch.randn(num_pages, Hkv, page, d, device=DEV, generator=g, dtype=torch.bfloat16)
    else:
        k_pages, v_pages = (_random_q4(num_pages, Hkv, page, d, g) for _ in range(2))
        tail = k_pages[..., 8 * d:].contiguous().view(torch.bfloat16)
        mn = tail.unflatten(-1, (16, d // GROUP, 2))[..., 1]
        mn += (by_page.unflatten(2, (-1, 16))[..., None] * sign).bfloat16()
        k_pages[..., 8 * d:] = tail.view(torch.uint8)
    S = case["splits"]
    return dict(case=case, q=q, k_pages=k_pages, v_pages=v_pages, table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), scale=d ** -0.5,
                o=torch.empty_like(q), lse=torch.empty(B, Hq, device=DEV),
                workspace=torch.empty(B * Hq * S * (d + 1) * 4 + 1024, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------ 4-bit records
def unpack_keys(rec, d):
    """[..., page / 16, record] bytes -> the codes' values in 32 bits [..., page, d]."""
    ng, n = d // GROUP, rec.shape[:-1]
    words = rec[..., :8 * d].contiguous().view(torch.int32).reshape(*n, 16, 4, ng)
    words = words.transpose(-1, -2)  # chunk m = 4 group + c
    i = torch.arange(4, device=rec.device) * 4
    shifts = torch.stack([i, i + 16], 1).flatten().int()  # element 2 i, 2 i + 1
    codes = (words[..., None] >> shifts) & 15  # [..., 16, ng, 4, 8]
    return _scaled(codes.reshape(*n, 16, ng, GROUP), rec, d)


def unpack_values(rec, d):
    ng, n = d // GROUP, rec.shape[:-1]
    units = rec[..., :8 * d].contiguous().view(torch.int16).reshape(*n, 2, 8, 4, ng, 2)
    # [half, g, c, group, parity] -> key = 8 half + 2 c + parity, d = 32 group + 4 g + i
    k = len(n)
    units = units.permute(*range(k), k, k + 2, k + 4, k + 3, k + 1)
    codes = (units[..., None].int() >> (torch.arange(4, device=rec.device) * 4).int()) & 15
    return _scaled(codes.reshape(*n, 16, ng, GROUP), rec, d)


def _scaled(codes, rec, d):
    n = rec.shape[:-1]
    par = rec[..., 8 * d:].contiguous().view(torch.bfloat16).float().reshape(*n, 16, d // GROUP, 2, 1)
    x = codes.float() * par[..., 0, :] + par[..., 1, :]
    return x.reshape(*n[:-1], n[-1] * 16, d)


def _bf16_down(x):
    b = x.bfloat16()
    bits = b.view(torch.int16)
    step = torch.where(b > 0, bits - 1, bits + 1)
    step = torch.where(b == 0, torch.full_like(bits, -32767), step)  # below zero: the smallest
    return torch.where(b.float() > x, step.view(torch.bfloat16), b)


def quantised(x):
    """32-bit rows [..., d] -> the values their 4-bit form stands for."""
    y = x.unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    mn = _bf16_down(lo).float()
    sc = -_bf16_down(-torch.div(hi - mn, torch.full_like(hi, 15.0))).float()  # a true quotient
    n = torch.where(sc > 0, torch.round((y - mn) / sc).clamp(0, 15), torch.zeros_like(y))
    return (n * sc + mn).flatten(-2)


# ------------------------------------------------------------------- runs
def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_decode(state) if own else _plain_decode(state)


def _own_append(st):
    import block_sparse_long_tiled_b200 as sk
    case = st["case"]
    sk.sskip_kv_append(st["q"], st["k"], st["v"], st["seq"], st["pos"], q_out=st["q_out"],
                       k_out=st["k_out"], v_out=st["v_out"], k_pages=st["k_pages"],
                       v_pages=st["v_pages"], block_table=st["table"], turns=st["turns"],
                       interleaved=case["interleaved"], attn_factor=st["attn"],
                       q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"])
    if case["fmt"] == "q4":
        sk.sskip_kv_gather(st["k_pages"], st["v_pages"], st["table"], st["seq"], st["pos"],
                           st["k_rows"], st["v_rows"])
        return {"q": st["q_out"], "k_rows": st["k_rows"], "v_rows": st["v_rows"]}
    return {n: st[n] for n in ("q_out", "k_out", "v_out", "k_pages", "v_pages") if st[n] is not None}


def _plain_rows(x, w, cos, sin, st):
    """Norm and rotation of [T, H, d] rows in 32 bits."""
    case = st["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
    rot = case["rot"]
    if rot == 0:
        return x
    y = x[..., :rot]
    a, b = (y[..., 0::2], y[..., 1::2]) if case["interleaved"] else y.chunk(2, -1)
    c, s = cos[:, None, :], sin[:, None, :]
    turned = (a * c - b * s, a * s + b * c)
    y = torch.stack(turned, -1).flatten(-2) if case["interleaved"] else torch.cat(turned, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(st):
    case = st["case"]
    angle = st["pos"].double()[:, None] * st["freq"]
    cos, sin = (angle.cos() * st["attn"]).float(), (angle.sin() * st["attn"]).float()
    q, k = (_plain_rows(st[n], st[w], cos, sin, st) for n, w in (("q", "qw"), ("k", "kw")))
    v = st["v"].float()
    live = st["seq"] >= 0
    L = st["out_len"]

    def laid(x, like):  # [T, H, d] -> [T / L, H, L, d]; padding tokens' rows stay
        x = x.bfloat16().unflatten(0, (-1, L)).transpose(1, 2)
        return torch.where(live.view(-1, 1, L, 1), x, like)

    if case["fmt"] == "q4":
        zero = torch.zeros((), device=q.device, dtype=torch.bfloat16)
        rows = [laid(quantised(x), zero) for x in (k, v)]
        return {"q": laid(q, st["q_out"]), "k_rows": rows[0], "v_rows": rows[1]}
    t = live.nonzero()[:, 0]
    s, p = st["seq"][t].long(), st["pos"][t].long()
    where = st["table"][s, p // case["page"]].long(), p % case["page"]
    out = {"q_out": laid(q, st["q_out"])}
    if case["outs"]:
        out |= {"k_out": laid(k, st["k_out"]), "v_out": laid(v, st["v_out"])}
    for n, x in (("k_pages", k), ("v_pages", v)):
        st[n].transpose(1, 2)[where] = x[t].bfloat16()
        out[n] = st[n]
    return out


def _own_decode(st):
    import block_sparse_long_tiled_b200 as sk
    case = st["case"]
    sk.sskip_attn_decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                               st["o"], st["lse"], sm_scale=st["scale"],
                               threshold_scale_factor=case["tsf"], num_splits=case["splits"],
                               workspace=st["workspace"])
    return {"o": st["o"], "lse": st["lse"]}


def _cache(st, name):
    """A sequence's rows in order, in 32 bits: [B, Hkv, max_pages * page, d]."""
    case, pages = st["case"], st[name][st["table"].long()]
    if case["fmt"] == "bf16":
        x = pages.float()
    else:
        x = (unpack_keys if name == "k_pages" else unpack_values)(pages, case["d"])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_decode(st):
    case = st["case"]
    B, Hq, Hkv, d, S, tsf = (case[n] for n in ("B", "Hq", "Hkv", "d", "splits", "tsf"))
    lens = st["lens"]
    q = st["q"].float().unflatten(1, (Hkv, -1)) * st["scale"]
    s = q @ _cache(st, "k_pages").transpose(2, 3)  # [B, Hkv, G, L]
    L = s.shape[-1]
    dead = torch.arange(L, device=s.device) >= lens.view(-1, 1, 1, 1)
    s = s.masked_fill(dead, -math.inf)
    if tsf > 0:
        # Tiles of 64 keys; the splits are runs of ceil(tiles / S) tiles, each
        # with a running maximum of its own.
        nk = -(-L // TILE)
        tiles = torch.nn.functional.pad(s, (0, nk * TILE - L), value=-math.inf)
        local = tiles.unflatten(-1, (nk, TILE)).amax(-1)  # [B, Hkv, G, nk]
        per = -(-(-(-lens // TILE)) // S).view(-1, 1)
        j = torch.arange(nk, device=s.device)
        start = (j // per) * per  # [B, nk]
        at = (j - start).view(B, 1, 1, nk)
        # the running maximum before tile j: over tiles start .. j - 1
        best, width = torch.full_like(local, -math.inf), 1
        before = torch.nn.functional.pad(local, (1, 0), value=-math.inf)[..., :-1]
        before = before.masked_fill(at < 1, -math.inf)
        while width < nk:  # a prefix maximum in log2(tiles) doublings, cut at the splits
            shifted = torch.nn.functional.pad(before, (width, 0), value=-math.inf)[..., :nk]
            before = torch.maximum(before, shifted.masked_fill(at < width + 1, -math.inf))
            width *= 2
        best = torch.maximum(best, before)
        ln_t = torch.log(tsf / lens.double()).float().view(-1, 1, 1, 1)
        skip = ((local - best) < ln_t).all(2, keepdim=True)
        s = s.masked_fill(skip.repeat_interleave(TILE, -1)[..., :L], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = _cache(st, "v_pages").masked_fill(dead.transpose(2, 3), 0.0)
    o = (p / l) @ v
    return {"o": o.flatten(1, 2).bfloat16(), "lse": (m + torch.log(l)).reshape(B, Hq)}


# ------------------------------------------------------------------ floors
def work(case):
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    row = d * 2 if case["fmt"] == "bf16" else record(d) // 16
    if case["op"] == "append":
        n = case["T"] - case["pad"]
        outs = 2 * Hkv * d * 2 if case["outs"] else 0
        moved = (Hq + 2 * Hkv) * d * 2 + Hq * d * 2 + outs + 2 * Hkv * row
        if case["fmt"] == "q4":  # read back
            moved += 2 * Hkv * row + 2 * Hkv * d * 2
        return {"bytes": n * moved, "flops": n * (Hq + Hkv) * (3 * case["rot"] + 4 * d)}
    keys = sum(_lengths(case))
    return {"bytes": keys * Hkv * 2 * row + case["B"] * Hq * (4 * d + 4),
            "flops": 4 * keys * Hq * d}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_decode)(st)


def _bf16_grid(x, up):
    """The nearest bf16 value not above (or not below) a 64-bit one."""
    _, e = torch.frexp(x)
    ulp = torch.ldexp(torch.ones_like(x), (e - 8).clamp_min(-133))
    return (torch.ceil(x / ulp) if up else torch.floor(x / ulp)) * ulp


def _exact_4bit(x):
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], GROUP):
        y = x[..., a:a + GROUP]
        mn = _bf16_grid(y.min(-1, keepdim=True).values, up=False)
        sc = _bf16_grid((y.max(-1, keepdim=True).values - mn) / 15, up=True)
        n = torch.round((y - mn) / sc.clamp_min(1e-300)).clamp(0, 15)
        out[..., a:a + GROUP] = mn + sc * n
    return out


def _exact_append(st):
    case = st["case"]
    T, d, rot, L = case["T"], case["d"], case["rot"], st["out_len"]
    seq, pos = st["seq"].tolist(), st["pos"].tolist()
    live = [t for t in range(T) if seq[t] >= 0]

    def turned(x, w):
        x = x.double().clone()
        if w is not None:
            x *= w.double() / (x.pow(2).sum(-1, keepdim=True) / d + st["eps"]).sqrt()
        if rot:
            e = st["pos"].double()[:, None] * st["freq"]
            e = torch.polar(torch.full_like(e, st["attn"]), e)[:, None]
            if case["interleaved"]:
                z = torch.view_as_complex(x[..., :rot].reshape(T, -1, rot // 2, 2).contiguous()) * e
                x[..., :rot] = torch.view_as_real(z).reshape(T, -1, rot)
            else:
                z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * e
                x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        return x

    def outs(x):
        y = torch.zeros(T // L, x.shape[1], L, d, dtype=torch.float64, device=x.device)
        t = torch.tensor(live, device=x.device)
        y[t // L, :, t % L] = x[t]
        return y

    q, k, v = turned(st["q"], st["qw"]), turned(st["k"], st["kw"]), st["v"].double()
    if case["fmt"] == "q4":
        return {"q": outs(q), "k_rows": outs(_exact_4bit(k)), "v_rows": outs(_exact_4bit(v))}
    got = {"q_out": outs(q)}
    if case["outs"]:
        got |= {"k_out": outs(k), "v_out": outs(v)}
    table = st["table"].tolist()
    page = torch.tensor([table[seq[t]][pos[t] // case["page"]] for t in live], device=q.device)
    slot = torch.tensor([pos[t] % case["page"] for t in live], device=q.device)
    for n, x in (("k_pages", k), ("v_pages", v)):
        pages = st[n].double()
        pages[page, :, slot] = x[torch.tensor(live, device=x.device)]
        got[n] = pages
    return got


def _exact_unpack(rec, d, values):
    """[n, record] bytes of 16 keys each -> [n * 16, d] in 64 bits, one
    nibble of every record at a time."""
    n, ng = rec.shape[0], d // GROUP
    word = rec.int()
    par = rec[:, 8 * d:].contiguous().view(torch.bfloat16).double().reshape(n, 16, ng, 2)
    key, e = torch.meshgrid(torch.arange(16), torch.arange(d), indexing="ij")
    if values:  # 16-bit units of four
        byte = ((key // 8 * 32 + e % 32 // 4 * 4 + key // 2 % 4) * ng + e // 32) * 4 + key % 2 * 2
        nib = e % 4
    else:       # 32-bit words of eight
        m = e // 8
        byte = key * (d // 2) + ((m % 4) * ng + m // 4) * 4
        nib = e % 8 // 2 + e % 2 * 4
    byte, shift = (byte + nib // 2).to(rec.device), (nib % 2 * 4).to(rec.device)
    code = (word[:, byte.flatten()].reshape(n, 16, d) >> shift) & 15
    sc, mn = (par[..., i].repeat_interleave(GROUP, -1) for i in (0, 1))
    return (mn + sc * code).reshape(n * 16, d)


def _exact_decode(st):
    case = st["case"]
    Hq, Hkv, d, page, S = (case[n] for n in ("Hq", "Hkv", "d", "page", "splits"))
    G = Hq // Hkv
    o = torch.zeros(case["B"], Hq, d, dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros(case["B"], Hq, dtype=torch.float64, device=st["q"].device)
    for b, n in enumerate(st["lens"].tolist()):
        ids = st["table"][b, :-(-n // page)].long()
        for h in range(Hkv):
            rows = []
            for name in ("k_pages", "v_pages"):
                x = st[name][ids, h]
                x = x.reshape(-1, d).double() if case["fmt"] == "bf16" else \
                    _exact_unpack(x.flatten(0, 1), d, name == "v_pages")
                rows.append(x[:n])
            s = st["scale"] * (rows[0] @ st["q"][b, h * G:(h + 1) * G].double().T)  # [n, G]
            keep = list(range(-(-n // TILE)))
            if case["tsf"] > 0:
                top = torch.stack([t.max(0).values for t in s.split(TILE)]).cpu()
                per, keep = -(-len(top) // S), []
                for j in range(len(top)):
                    run_max = top[j] * 0 - math.inf if j % per == 0 else run_max
                    if not bool(((top[j] - run_max) < math.log(case["tsf"] / n)).all()):
                        keep.append(j)
                        run_max = torch.maximum(run_max, top[j])
            at = torch.cat([torch.arange(j * TILE, min(n, (j + 1) * TILE)) for j in keep]).to(s.device)
            s = s[at]
            z = torch.logsumexp(s, 0)
            lse[b, h * G:(h + 1) * G] = z
            o[b, h * G:(h + 1) * G] = torch.exp(s - z).T @ rows[1][at]
    return {"o": o, "lse": lse}

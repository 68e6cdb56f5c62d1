"""The paged operators as they are used together: a layer that prefills
prompts into a paged cache and then decodes token by token."""
import numpy as np
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
import paged_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_long_tiled_b200 import build
    build.build()
    assert torch.cuda.is_available()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host(t):
    return t.cpu().numpy() if t.dtype == torch.uint8 else t.float().cpu().numpy()


class Layer:
    """Hq query heads over Hkv, d, pages of P, B sequences; the projections of
    a step are random rows."""

    def __init__(self, B=3, Hq=8, Hkv=2, d=128, P=16, int4=False, interleaved=False, seed=0):
        self.__dict__.update(B=B, Hq=Hq, Hkv=Hkv, d=d, P=P, scale=d ** -0.5)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        M, N = 300 // P + 1, B * (300 // P + 1) + 2
        self.table = torch.randperm(N, generator=torch.Generator().manual_seed(seed))[:B * M]
        self.table = self.table.reshape(B, M).int().cuda()
        self.k_pages, self.v_pages = sk.paged_cache(N, Hkv, P, d, int4=int4)
        turns, attn = sk.rope_table(d, 10000.0, scaling="yarn", factor=4.0, slow_turns=1.0,
                                    fast_turns=32.0, original_len=128.0)
        w = lambda: (1 + 0.1 * torch.randn(d, device="cuda", generator=self.g)).bfloat16()  # noqa: E731
        self.rope = dict(turns=turns, attn_factor=attn, interleaved=interleaved, q_weight=w(),
                         k_weight=w())

    def qkv(self, T):
        x = torch.randn(T, (self.Hq + 2 * self.Hkv) * self.d, device="cuda", generator=self.g)
        x = x.bfloat16().unflatten(1, (-1, self.d))
        return x.split([self.Hq, self.Hkv, self.Hkv], 1)

    def check_decode(self, q, lens, out, splits, tsf):
        want = ref.decode(host(q), host(self.k_pages), host(self.v_pages), self.table.cpu().numpy(),
                          lens, self.scale, tsf, splits)
        assert np.array_equal(out["counts"].cpu().numpy(),
                              [(want["tile_state"] == 2).sum(), (want["tile_state"] > 0).sum()])
        tol_o, tol_l = ref.decode_tolerance(want, max(lens))
        live = np.array(lens) > 0
        assert np.all(np.abs(host(out["o"]) - want["o"])[live] <= tol_o[live])
        assert np.all(np.abs(out["lse"].cpu().numpy()[live] - want["lse"][live]) <= tol_l[live])
        assert np.all(host(out["o"])[~live] == 0)


def attention(q, k, v, scale):
    """Causal attention in 64 bits, [B, H, L, d] with shared kv heads: o, lse,
    and the mass sum P |v| and sum |q k| scale that its tolerance needs."""
    q, k, v = (x.astype(np.float64) for x in (q, k, v))
    k, v = (np.repeat(x, q.shape[1] // k.shape[1], 1) for x in (k, v))
    s = scale * q @ k.swapaxes(-1, -2)
    L = s.shape[-1]
    s = np.where(np.tril(np.ones((L, L), bool)), s, -np.inf)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    l = p.sum(-1, keepdims=True)
    size = scale * (np.abs(q) @ np.abs(k).swapaxes(-1, -2)).max(-1)
    return {"o": p / l @ v, "lse": (m + np.log(l))[..., 0], "mass": p / l @ np.abs(v), "size": size}


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(d=64, P=64, interleaved=True), dict(Hq=2, Hkv=2, P=32)],
                         ids=str)
def test_prompts_then_tokens(kw, int4):
    y = Layer(int4=int4, **kw)
    L, B = 130, y.B
    q, k, v = y.qkv(B * L)
    seq, pos = np.repeat(np.arange(B), L), np.tile(np.arange(L), B)
    out = sk.prefill_paged(q, k, v, i32(seq), i32(pos), y.k_pages, y.v_pages, y.table, L=L,
                           sm_scale=y.scale, threshold_scale_factor=0.0, **y.rope)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    # What the prefill saw: the rotated rows in bf16, which another call of the
    # append gives again to the bit (they are tested against the definition on
    # their own; two roundings of q and k would move a logit by 2^-7 |q| |k| scale
    # here, far more than the attention's own error).
    qr = torch.empty(B, y.Hq, L, y.d, device="cuda", dtype=torch.bfloat16)
    kr, vr = (torch.empty(B, y.Hkv, L, y.d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sk.sskip_kv_append(q, k, v, None, i32(pos), q_out=qr, k_out=kr, v_out=vr, **y.rope)
    want = attention(host(qr), host(kr), host(vr), y.scale)
    # As in the decode: a bf16 half step of o and of each weight, and the scores' error.
    tol_o, tol_l = ref.decode_tolerance(want, L)
    assert np.all(np.abs(host(out["o"]) - want["o"]) <= tol_o)
    assert np.all(np.abs(out["lse"].cpu().numpy() - want["lse"]) <= tol_l)
    # 4 steps: ragged from the second one on (a sequence ends: a padded entry)
    lens = np.full(B, L)
    for step in range(4):
        live = np.ones(B, bool)
        if step >= 2:
            live[1] = False
        lens = np.where(live, lens + 1, lens)
        q, k, v = y.qkv(B)
        out = sk.decode_step_paged(q, k, v, i32(np.where(live, np.arange(B), -1)), i32(lens - 1),
                                   i32(np.where(live, lens, 0)), y.k_pages, y.v_pages, y.table,
                                   sm_scale=y.scale, threshold_scale_factor=3.0 * (step % 2),
                                   num_splits=1 + step, **y.rope)
        torch.cuda.synchronize()
        assert sk.sskip_get_status() == sk.SSKIP_OK
        qr = torch.zeros(B, y.Hq, y.d, device="cuda", dtype=torch.bfloat16)
        sk.sskip_kv_append(q, None, None, None, i32(lens - 1), q_out=qr, turns=y.rope["turns"],
                           attn_factor=y.rope["attn_factor"], interleaved=y.rope["interleaved"],
                           q_weight=y.rope["q_weight"])
        y.check_decode(qr, list(np.where(live, lens, 0)), out, 1 + step, 3.0 * (step % 2))
    # the whole history read back is what a contiguous cache of it would hold
    n = int(lens[0])
    kr, vr = (torch.empty(1, y.Hkv, n, y.d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sk.sskip_kv_gather(y.k_pages, y.v_pages, y.table, i32([0] * n), i32(range(n)), kr, vr)
    q1 = torch.randn(1, y.Hq, y.d, device="cuda", generator=y.g).bfloat16()
    a = sk.decode(q1, kr, vr, i32([n]), sm_scale=y.scale, threshold_scale_factor=0.0, num_splits=2)
    b = sk.decode_paged(q1, y.k_pages, y.v_pages, y.table[:1].contiguous(), i32([n]),
                        sm_scale=y.scale, threshold_scale_factor=0.0, num_splits=2)
    # read-back rounds 4-bit values to bf16: half a step of each key and value
    assert float((a["lse"] - b["lse"]).abs().max()) < 2.0 ** -8 * float(
        (q1.float().abs().sum(-1) * y.scale).max() * kr.float().abs().max())
    assert float((a["o"].float() - b["o"].float()).abs().max()) < 0.1 * float(vr.float().abs().max())


@pytest.mark.parametrize("int4", [False, True])
def test_a_captured_step_replayed_token_by_token(int4):
    y = Layer(int4=int4, seed=3)
    e = Layer(int4=int4, seed=3)  # the same, run eagerly
    B = y.B
    e.k_pages.copy_(y.k_pages)
    e.v_pages.copy_(y.v_pages)
    q, k, v = (x.contiguous() for x in y.qkv(B))
    seq, pos, lens = i32(range(B)), i32([0] * B), i32([1] * B)
    qr, lse = torch.empty_like(q), torch.empty(B, y.Hq, device="cuda")
    o = torch.empty_like(q)
    ws = torch.empty(sk.sskip_attn_decode_workspace_size(B, y.Hq, y.d, 10), device="cuda",
                     dtype=torch.uint8)

    def step():
        sk.sskip_kv_append(q, k, v, seq, pos, q_out=qr, k_pages=y.k_pages, v_pages=y.v_pages,
                           block_table=y.table, **y.rope)
        sk.sskip_attn_decode_paged(qr, y.k_pages, y.v_pages, y.table, lens, o, lse,
                                   sm_scale=y.scale, threshold_scale_factor=2.0, num_splits=10,
                                   workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(70):
        for x, new in zip((q, k, v), y.qkv(B)):
            x.copy_(new)
        pos.fill_(n)
        lens.fill_(n + 1)
        g.replay()
        want = sk.decode_step_paged(q, k, v, seq, pos, lens, e.k_pages, e.v_pages, y.table,
                                    sm_scale=y.scale, threshold_scale_factor=2.0, num_splits=10,
                                    **y.rope)
        assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"]), n
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    del g


def test_two_streams_at_once_with_a_workspace_each():
    ys = [Layer(int4=i == 1, seed=5 + i, B=6) for i in range(2)]
    calls = []
    for y in ys:
        q, k, v = y.qkv(y.B * 280)
        seq, pos = np.repeat(np.arange(y.B), 280), np.tile(np.arange(280), y.B)
        sk.sskip_kv_append(None, k, v, i32(seq), i32(pos), k_pages=y.k_pages, v_pages=y.v_pages,
                           block_table=y.table, turns=y.rope["turns"])
        lens = i32([280, 17, 0, 64, 100, 256])
        calls.append((q[:y.B].contiguous(), y, lens))
    run = lambda c, st=None: sk.decode_paged(c[0], c[1].k_pages, c[1].v_pages, c[1].table, c[2],  # noqa: E731
                                             sm_scale=c[1].scale, threshold_scale_factor=1.0,
                                             num_splits=9, stream=st)
    want = [run(c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[run(c, st) for c, st in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    for round_ in got:
        for a, b in zip(round_, want):
            assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("tsf", [0.0, 3.0])
def test_debug_build_matches_release(int4, tsf):
    """The debug library's index checks hold and its outputs are the release's."""
    outs = []
    for lib in (sk.lib(), sk.debug_lib()):
        y = Layer(int4=int4, seed=11, P=16)
        y.k_pages.zero_()
        y.v_pages.zero_()
        q, k, v = y.qkv(y.B * 150)
        seq, pos = np.repeat(np.arange(y.B), 150), np.tile(np.arange(150), y.B)
        keep, sk._lib = sk._lib, lib
        try:
            sk.sskip_kv_append(None, k, v, i32(seq), i32(pos), k_pages=y.k_pages,
                               v_pages=y.v_pages, block_table=y.table, turns=y.rope["turns"])
            got = [sk.decode_paged(q[:y.B].contiguous(), y.k_pages, y.v_pages, y.table,
                                   i32([150, 0, 33]), sm_scale=y.scale, threshold_scale_factor=tsf,
                                   num_splits=S) for S in (1, 3, 20)]
            kr, vr = (torch.zeros(y.B * 150, y.Hkv, y.d, device="cuda", dtype=torch.bfloat16)
                      for _ in range(2))
            sk.sskip_kv_gather(y.k_pages, y.v_pages, y.table, i32(seq), i32(pos), kr, vr)
            torch.cuda.synchronize()
            assert lib.sskip_get_status(None) == sk.SSKIP_OK
        finally:
            sk._lib = keep
        outs.append([y.k_pages, y.v_pages, kr, vr] + [x[n] for x in got for n in ("o", "lse", "counts")])
    for a, b in zip(*outs):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("splits", [1, 4, 12])
def test_calls_in_a_row_see_what_the_calls_before_wrote(int4, splits):
    """Each call reads what the one before it wrote, with nothing in between
    (their launches overlap); the same calls, waited for one by one, agree."""
    steps, outs = 60, []
    for wait in (True, False):
        y = Layer(int4=int4, seed=21, B=2)
        y.k_pages.zero_()
        y.v_pages.zero_()
        q, k, v = (x.contiguous() for x in y.qkv(y.B))
        o = [q] + [torch.empty_like(q) for _ in range(steps)]
        ks = [k] + [torch.empty_like(k) for _ in range(steps)]
        vs = [v] + [torch.empty_like(v) for _ in range(steps)]
        qr, lse = torch.empty_like(q), torch.empty(y.B, y.Hq, device="cuda")
        seq = i32(range(y.B))
        pos, lens = ([i32([n + i] * y.B) for n in range(steps)] for i in (0, 1))
        ws = torch.empty(sk.sskip_attn_decode_workspace_size(y.B, y.Hq, y.d, splits), device="cuda",
                         dtype=torch.uint8) if splits > 1 else None
        done = torch.cuda.synchronize if wait else lambda: None
        done()
        for n in range(steps):
            sk.sskip_kv_append(o[n], ks[n], vs[n], seq, pos[n], q_out=qr, k_pages=y.k_pages,
                               v_pages=y.v_pages, block_table=y.table, **y.rope)
            done()
            sk.sskip_kv_gather(y.k_pages, y.v_pages, y.table, seq, pos[n], ks[n + 1], vs[n + 1])
            done()
            sk.sskip_attn_decode_paged(qr, y.k_pages, y.v_pages, y.table, lens[n], o[n + 1], lse,
                                       sm_scale=y.scale, threshold_scale_factor=2.0,
                                       num_splits=splits, workspace=ws)
            done()
        torch.cuda.synchronize()
        outs.append([torch.stack(o), torch.stack(ks), torch.stack(vs), y.k_pages, y.v_pages])
    assert sk.sskip_get_status() == sk.SSKIP_OK
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert bool(torch.isfinite(outs[0][0].float()).all())


@pytest.mark.parametrize("int4", [False, True])
def test_captured_behind_copies_fills_and_joined_streams(int4):
    """The calls as nodes of a graph whose other nodes are no kernels, or
    come from another stream, replayed on new inputs."""
    y = Layer(int4=int4, seed=23, B=3)
    y.k_pages.zero_()
    y.v_pages.zero_()
    B, T = y.B, y.B * 40
    src = [[x.contiguous() for x in y.qkv(T)] for _ in range(3)]
    q, k, v = (torch.zeros_like(x) for x in src[0])
    seq, pos = i32(np.repeat(np.arange(B), 40)), i32(np.tile(np.arange(40), B))
    lens = i32([40] * B)
    fresh = lambda: [torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),  # noqa: E731
                     torch.empty(B, y.Hq, y.d, device="cuda", dtype=torch.bfloat16),
                     torch.empty(B, y.Hq, device="cuda")]
    out, last = fresh(), torch.zeros(B, y.Hq, y.d, device="cuda", dtype=torch.bfloat16)

    def append(st):
        sk.sskip_kv_append(q, k, v, seq, pos, q_out=out[0], k_pages=y.k_pages, v_pages=y.v_pages,
                           block_table=y.table, stream=st, **y.rope)

    def gather(st):
        sk.sskip_kv_gather(y.k_pages, y.v_pages, y.table, seq, pos, out[1], out[2], stream=st)

    def decode(st):
        sk.sskip_attn_decode_paged(last, y.k_pages, y.v_pages, y.table, lens, out[3], out[4],
                                   sm_scale=y.scale, threshold_scale_factor=1.0, num_splits=1,
                                   stream=st)

    def run(new):
        for x, n in zip((q, k, v), new):
            x.copy_(n)
        append(None)
        last.copy_(out[0].view(B, 40, y.Hq, y.d)[:, -1])
        gather(None)
        decode(None)

    inputs = [torch.empty_like(x) for x in src[0]]
    side = torch.cuda.Stream()
    run(src[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        y.k_pages.zero_()                       # a fill
        for x, n in zip((q, k, v), inputs):     # copies
            x.copy_(n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            y.v_pages.zero_()
        main.wait_stream(side)                  # a join, the fill last
        append(None)
        side.wait_stream(main)
        with torch.cuda.stream(side):           # a fork: gather beside the decode
            gather(side)
        last.copy_(out[0].view(B, 40, y.Hq, y.d)[:, -1])
        decode(None)
        main.wait_stream(side)
        out[4].add_(0.0)                        # a kernel behind the join
        decode(None)                            # and a call behind a call
    for new in src:
        for x, n in zip(inputs, new):
            x.copy_(n)
        g.replay()
        got = [x.clone() for x in out]
        y.k_pages.zero_()
        y.v_pages.zero_()
        run(new)
        for a, b in zip(got, out):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    del g


@pytest.mark.parametrize("tsf", [0.0, 2.0])
def test_shorter_prompts_end_in_padding(tsf):
    """What stood in the memory before does not reach the rows of a prompt
    whose last rows are padding."""
    y = Layer(seed=25, B=2)
    L, n = 200, 131
    q, k, v = y.qkv(2 * L)
    seq, pos = np.repeat([0, 1], L), np.tile(np.arange(L), 2)
    seq[L + n:] = -1
    outs = []
    for fill in (float("nan"), 0.0):
        dirt = [torch.full((2, h, L, y.d), fill, device="cuda", dtype=torch.bfloat16)
                for h in (y.Hq, y.Hkv, y.Hkv, y.Hq)]
        del dirt
        out = sk.prefill_paged(q, k, v, i32(seq), i32(pos), y.k_pages, y.v_pages, y.table, L=L,
                               sm_scale=y.scale, threshold_scale_factor=tsf, **y.rope)
        outs.append([out["o"][0], out["o"][1, :, :n], out["lse"][0], out["lse"][1, :, :n]])
    assert sk.sskip_get_status() == sk.SSKIP_OK
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a.float()).all()) and torch.equal(a, b)
    if tsf == 0.0:  # and they are what real tokens behind them would leave them
        seq[L + n:] = 1
        full = sk.prefill_paged(q, k, v, i32(seq), i32(pos), y.k_pages, y.v_pages, y.table, L=L,
                                sm_scale=y.scale, threshold_scale_factor=tsf, **y.rope)
        assert torch.equal(outs[0][1], full["o"][1, :, :n])


@pytest.mark.parametrize("tsf", [0.0, 2.0])
@pytest.mark.parametrize("int4,pages", [(False, 40_000), (True, 110_000)])
def test_pools_of_more_than_4_gib(int4, pages, tsf):
    """Pages on both sides of byte 2^32 of a pool give what a small pool with
    the same rows does."""
    y = Layer(Hq=16, Hkv=8, P=64, B=3, int4=int4, seed=27)
    M = y.table.shape[1]
    assert pages * sk.sskip_kv_page_bytes(sk.SSKIP_KV_INT4 if int4 else sk.SSKIP_KV_BF16, 8, 64,
                                          128) > 2 ** 32
    far = sk.paged_cache(pages, 8, 64, 128, int4=int4)
    far_table = torch.linspace(0, pages - 1, 3 * M).int().reshape(M, 3).t().contiguous().cuda()
    lens = [290, 64, 201]
    seq = np.concatenate([np.full(n, b) for b, n in enumerate(lens)])
    pos = np.concatenate([np.arange(n) for n in lens])
    q, k, v = y.qkv(len(seq))
    q1 = y.qkv(3)[0].contiguous()
    got = []
    for (kp, vp), table in (((y.k_pages, y.v_pages), y.table), (far, far_table)):
        sk.sskip_kv_append(None, k, v, i32(seq), i32(pos), k_pages=kp, v_pages=vp, block_table=table,
                           turns=y.rope["turns"], k_weight=y.rope["k_weight"])
        rows = [torch.empty(len(seq), 8, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
        sk.sskip_kv_gather(kp, vp, table, i32(seq), i32(pos), *rows)
        out = sk.decode_paged(q1, kp, vp, table, i32(lens), sm_scale=y.scale,
                              threshold_scale_factor=tsf, num_splits=3)
        got.append(rows + [out["o"], out["lse"], out["counts"]])
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    for a, b in zip(*got):
        assert torch.equal(a, b)

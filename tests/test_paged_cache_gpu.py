"""Append to and read-back from the paged cache against the 64-bit forms."""
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


def bf16(x):
    """Float array -> (CUDA bf16 tensor, its values)."""
    bits = ref.bf16_bits(np.asarray(x, np.float32))
    t = torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16)
    return t, ref.bf16_value(bits)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.uint8 else t.float().cpu().numpy()


class Case:
    """Inputs of one append: tokens of B ragged sequences in a shuffled order,
    projection slices, pages in a shuffled order, marks in what must not change."""

    def __init__(self, seed=1, counts=(3, 1, 5), starts=(0, 17, 62), pad=2, Hq=4, Hkv=2, d=128, P=16,
                 fmt="bf16", rot=None, interleaved=False, norm=True, eps=1e-6, out_len=1, attn=1.0,
                 base=10000.0, spread=1.0, shuffle=True, outs=True, cache=True):
        r = np.random.default_rng(seed)
        self.__dict__.update(Hq=Hq, Hkv=Hkv, d=d, P=P, fmt=fmt, interleaved=interleaved, eps=eps,
                             attn=attn, out_len=out_len, cache=cache)
        seq = sum(([b] * n for b, n in enumerate(counts)), []) + [-1] * pad
        pos = sum((list(range(s, s + n)) for s, n in zip(starts, counts)), []) + [-5] * pad
        self.T = len(seq)
        order = r.permutation(self.T) if shuffle else np.arange(self.T)
        self.seq, self.pos = np.array(seq)[order], np.array(pos)[order]
        self.B = len(counts)
        M = max(-(-(s + n) // P) for s, n in zip(starts, counts)) + 1
        self.N = self.B * M + 3
        self.table = r.permutation(self.N)[:self.B * M].reshape(self.B, M)
        rot = d if rot is None else rot
        self.turns = (sk.sskip_rope_freqs(rot, base)[0] if rot else np.zeros(0, np.int64))
        H = Hq + 2 * Hkv
        self.qkv_t, qkv = bf16(spread * r.standard_normal((self.T, H, d)))
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        self.q_t, self.k_t, self.v_t = (self.qkv_t[:, :Hq], self.qkv_t[:, Hq:Hq + Hkv],
                                        self.qkv_t[:, Hq + Hkv:])
        self.qw_t, self.qw = bf16(1 + 0.2 * r.standard_normal(d)) if norm else (None, None)
        self.kw_t, self.kw = bf16(1 + 0.2 * r.standard_normal(d)) if norm else (None, None)
        out = lambda h: torch.full((self.T // out_len, h, out_len, d), 7.0, device="cuda",  # noqa: E731
                                   dtype=torch.bfloat16)
        self.q_out = out(Hq)
        self.k_out, self.v_out = (out(Hkv), out(Hkv)) if outs else (None, None)
        if fmt == "bf16":
            shape, fill = (self.N, Hkv, P, d), 5.0
            pages = lambda: torch.full(shape, fill, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        else:
            pages = lambda: torch.full((self.N, Hkv, P // 16, 10 * d), 0xA5, device="cuda",  # noqa: E731
                                       dtype=torch.uint8)
        self.k_pages, self.v_pages = (pages(), pages()) if cache else (None, None)

    def run(self, **kw):
        a = dict(q_out=self.q_out, k_out=self.k_out, v_out=self.v_out, k_pages=self.k_pages,
                 v_pages=self.v_pages, block_table=i32(self.table) if self.cache else None,
                 turns=torch.from_numpy(self.turns).cuda() if len(self.turns) else None,
                 interleaved=self.interleaved, attn_factor=self.attn, q_weight=self.qw_t,
                 k_weight=self.kw_t, eps=self.eps)
        a.update(kw)
        sk.sskip_kv_append(self.q_t, self.k_t, self.v_t, i32(self.seq), i32(self.pos), **a)
        torch.cuda.synchronize()
        assert sk.sskip_get_status() == sk.SSKIP_OK

    def want(self):
        y = lambda x, w: ref.rotated(x, self.pos, self.turns, self.interleaved, self.attn, w,  # noqa: E731
                                     self.eps)
        return y(self.q, self.qw), y(self.k, self.kw), (self.v.astype(np.float64), np.abs(self.v))

    def rows(self, t):
        """[T / L, H, L, d] -> [T, H, d]"""
        x = host(t)
        return x.swapaxes(1, 2).reshape(self.T, x.shape[1], self.d)

    def check(self):
        live = self.seq >= 0
        wants = self.want()
        for t, (y, mag) in zip((self.q_out, self.k_out, self.v_out), wants):
            if t is None:
                continue
            got = self.rows(t)
            assert np.all(got[~live] == 7.0), "rows of padding tokens were touched"
            close(got[live], y[live], mag[live])
        if not self.cache:
            return
        for val, pages, (y, mag) in ((False, self.k_pages, wants[1]), (True, self.v_pages, wants[2])):
            got, touched = host(pages), np.zeros((self.N, self.P), bool)
            for t in np.nonzero(live)[0]:
                page, off = self.table[self.seq[t], self.pos[t] // self.P], self.pos[t] % self.P
                touched[page, off] = True
                if self.fmt == "bf16":
                    close(got[page, :, off], y[t], mag[t])
                else:
                    rec = got[page, :, off // 16]
                    self.check_q4(rec, off % 16, y[t], mag[t], val)
            if self.fmt == "bf16":
                assert np.all(got.swapaxes(1, 2)[~touched] == 5.0), "other rows were touched"
            else:
                codes, sc, mn = ref.unpack(got, self.d, val)  # [N, Hkv, P / 16, 16, ...]
                idle = ~touched.reshape(self.N, 1, self.P // 16, 16).repeat(self.Hkv, 1)
                assert np.all((codes[idle] == 5) | (codes[idle] == 10)), "other rows were touched"
                mark = ref.bf16_value(np.uint16(0xA5A5))
                assert np.all(sc[idle] == mark) and np.all(mn[idle] == mark)

    def check_q4(self, rec, r, y, mag, value):
        codes, sc, mn = (x[:, r] for x in ref.unpack(rec, self.d, value))
        n, want_sc, want_mn = ref.quantise(y)
        if value:  # exact inputs: the same codes, scales and minima to the bit
            assert np.array_equal(sc, want_sc) and np.array_equal(mn, want_mn)
            assert np.array_equal(codes, n)
            return
        # Keys are quantised from fp32: no value is off by more than half a
        # scale and the fp32 error; the minimum lies at most one bf16 step below
        # the group's, the scale at most one above the fifteenth of the spread.
        g = y.reshape(*y.shape[:-1], -1, 32)
        err = fp32_error(mag).reshape(g.shape).max(-1)
        lo, hi = g.min(-1), g.max(-1)
        assert np.all(mn <= lo + err) and np.all(mn >= lo - err - 2.0 ** -7 * (np.abs(lo) + err))
        spread = (hi - mn) / 15
        assert np.all(sc >= spread - err) and np.all(sc <= (spread + err) * (1 + 2.0 ** -7))
        got = np.repeat(mn, 32, -1).astype(np.float64) + np.repeat(sc, 32, -1) * codes
        half = np.repeat(sc * 0.5 * (1 + 2.0 ** -20) + err, 32, -1)
        assert np.all(np.abs(got - y) <= half)


def fp32_error(mag):
    """fp32 between load and store: the norm's 128-term sum and rsqrt (12 steps
    of 2^-24 each, halved by the root), two products, cosine and sine good to
    2^-22 with their angle: under 2^-19 of the magnitudes that meet."""
    return 2.0 ** -19 * mag


def close(got, y, mag):
    """One rounding to bf16: half a step is 2^-8 of the rounded value."""
    err = fp32_error(mag)
    tol = 2.0 ** -8 * (np.abs(y) + err) + err
    bad = np.abs(got - y) > tol
    assert not bad.any(), (got[bad][:4], y[bad][:4])


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("kw", [
    dict(), dict(d=64), dict(interleaved=True), dict(d=64, interleaved=True),
    dict(rot=0), dict(rot=16), dict(rot=48), dict(rot=64), dict(rot=96, interleaved=True),
    dict(rot=32), dict(rot=80), dict(rot=112), dict(d=64, rot=16), dict(rot=80, interleaved=True),
    dict(d=64, rot=32), dict(d=64, rot=48), dict(norm=False), dict(attn=1.3),
    dict(Hq=1, Hkv=1), dict(Hq=7, Hkv=7, d=64), dict(Hq=64, Hkv=8), dict(Hq=3, Hkv=1, d=64),
    dict(P=32), dict(P=64), dict(P=128), dict(P=256), dict(outs=False),
    dict(counts=(1,), starts=(0,), pad=0), dict(counts=(1,), starts=(15,), pad=0),
    dict(counts=(40, 0, 3), starts=(9, 0, 31), pad=5), dict(eps=0.0), dict(eps=10.0),
], ids=str)
def test_append(kw, fmt):
    c = Case(fmt=fmt, **kw)
    c.run()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_layout(d):
    c = Case(counts=(21, 21), starts=(0, 0), pad=0, out_len=21, d=d, shuffle=False)
    c.run()
    c.check()


def test_many_tokens():
    c = Case(counts=(4001, 3, 997), starts=(5, 0, 1000), pad=7, P=64, Hq=8, Hkv=2)
    c.run()
    c.check()


def test_far_positions():
    # Positions whose fp32 angles would be off by radians.
    c = Case(counts=(2, 2), starts=(1, 1), pad=0, cache=False)
    c.pos = np.array([2 ** 31 - 1, 1_000_003, -(2 ** 31), 16_777_217])
    c.seq = np.zeros(4, int)
    c.run()
    c.check()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_token_and_head_strides(fmt):
    # q, k and v in buffers of their own, with gaps behind each token.
    c = Case(fmt=fmt)
    for n in ("q_t", "k_t", "v_t"):
        x = getattr(c, n)
        wide = torch.full((c.T, x.shape[1] * c.d + 24), float("nan"), device="cuda",
                          dtype=torch.bfloat16)
        wide[:, :x.shape[1] * c.d] = x.flatten(1)
        setattr(c, n, wide[:, :x.shape[1] * c.d].unflatten(1, (-1, c.d)))
    c.run()
    c.check()


def test_queries_alone_and_keys_alone():
    c = Case(cache=False, pad=1)
    turns = torch.from_numpy(c.turns).cuda()
    sk.sskip_kv_append(c.q_t, None, None, i32(c.seq), i32(c.pos), q_out=c.q_out, turns=turns,
                       q_weight=c.qw_t, eps=c.eps)
    sk.sskip_kv_append(None, c.k_t, c.v_t, i32(c.seq), i32(c.pos), k_out=c.k_out, v_out=c.v_out,
                       turns=turns, k_weight=c.kw_t, eps=c.eps)
    torch.cuda.synchronize()
    c.check()


def test_without_sequences_nothing_is_padding():
    c = Case(cache=False, pad=0)
    sk.sskip_kv_append(c.q_t, c.k_t, c.v_t, None, i32(c.pos), q_out=c.q_out, k_out=c.k_out,
                       v_out=c.v_out, turns=torch.from_numpy(c.turns).cuda(), q_weight=c.qw_t,
                       k_weight=c.kw_t, eps=c.eps)
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("what", ["sequence", "position", "far position", "page", "negative page"])
def test_bad_indices_are_latched_and_left_out(what, fmt):
    c = Case(fmt=fmt, pad=1, shuffle=False)
    bad, table = 4, c.table.copy()
    seq, pos = c.seq.copy(), c.pos.copy()
    if what == "sequence":
        seq[bad] = c.B
    elif what == "position":
        pos[bad] = -1
    elif what == "far position":
        pos[bad] = c.table.shape[1] * c.P
    else:  # token `bad` is alone on this page of its sequence
        seq[bad], pos[bad] = 1, (c.table.shape[1] - 1) * c.P
        table[1, -1] = c.N if what == "page" else -1
    sk.sskip_kv_append(c.q_t, c.k_t, c.v_t, i32(seq), i32(pos), q_out=c.q_out, k_out=c.k_out,
                       v_out=c.v_out, k_pages=c.k_pages, v_pages=c.v_pages, block_table=i32(table),
                       turns=torch.from_numpy(c.turns).cuda(), q_weight=c.qw_t, k_weight=c.kw_t,
                       eps=c.eps)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_ERR_INVALID_ARG
    c.seq[bad] = -1  # as if it were padding
    c.check()
    k = torch.full((c.T, c.Hkv, c.d), 7.0, device="cuda", dtype=torch.bfloat16)
    v = k.clone()
    sk.sskip_kv_gather(c.k_pages, c.v_pages, i32(table), i32(seq), i32(pos), k, v)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_ERR_INVALID_ARG
    assert bool((k[bad] == 7).all()) and bool((v[bad] == 7).all())
    assert not bool((k[0] == 7).all())


def test_q4_groups_that_are_flat_tiny_or_not_finite():
    c = Case(fmt="q4", counts=(1,), starts=(3,), pad=0, Hq=1, Hkv=1, rot=0, norm=False, outs=False)
    rows = np.random.default_rng(3).standard_normal((1, 1, 128)).astype(np.float32)
    rows[..., :32] = -2.5                      # one value: the scale is 0
    rows[..., 32:64] *= 1e-37                  # close to the smallest normal numbers
    rows[..., 70] = np.inf
    rows[..., 100] = np.nan
    c.v_t, c.v = bf16(rows)
    c.k_t, c.k = bf16(rows)
    c.run()
    k, v = (torch.zeros(1, 1, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sk.sskip_kv_gather(c.k_pages, c.v_pages, i32(c.table), i32(c.seq), i32(c.pos), k, v)
    for t in (k, v):
        got = host(t)[0, 0]
        assert np.all(got[:32] == -2.5)
        x = c.v[0, 0, 32:64].astype(np.float64)
        sc = ref.quantise(x)[1]
        assert np.all(np.abs(got[32:64] - x) <= 0.5 * sc * (1 + 2.0 ** -6) + 2.0 ** -8 * np.abs(x) + 1e-40)
        assert np.all(np.isnan(got[64:]))


@pytest.mark.parametrize("fill", [np.nan, np.inf, -np.inf])
def test_q4_a_value_that_is_not_finite_spoils_its_group_wherever_it_stands(fill):
    """One such value at each place of a group; the other groups keep theirs."""
    c = Case(fmt="q4", counts=(32,), starts=(5,), pad=0, Hq=1, Hkv=2, rot=0, norm=False, outs=False)
    rows = np.random.default_rng(4).standard_normal((32, 2, 128)).astype(np.float32)
    for i in range(32):
        rows[i, i % 2, 32 * (i % 4) + i] = fill
    c.k_t, c.k = bf16(rows)
    c.v_t, c.v = bf16(rows)
    c.run()
    k, v = (torch.zeros(32, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sk.sskip_kv_gather(c.k_pages, c.v_pages, i32(c.table), i32(c.seq), i32(c.pos), k, v)
    bad = ~np.isfinite(c.v.astype(np.float64).reshape(32, 2, 4, 32)).all(-1)
    assert bad.sum() == 32
    for t in (k, v):
        got = host(t).reshape(32, 2, 4, 32)
        assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


@pytest.mark.parametrize("spread", [2.0 ** -133, 2.0 ** -128, 2.0 ** -123, 2.0 ** -122])
def test_q4_spreads_about_the_smallest_scale(spread):
    """A scale is 2^-126 at least: codes, scales and minima as the formula says."""
    c = Case(fmt="q4", counts=(1,), starts=(0,), pad=0, Hq=1, Hkv=1, rot=0, norm=False, outs=False)
    rows = (np.random.default_rng(5).uniform(-1, 1, (1, 1, 128)) * spread).astype(np.float32)
    c.k_t, c.k = bf16(rows)
    c.v_t, c.v = bf16(rows)
    c.run()
    k, v = (torch.zeros(1, 1, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sk.sskip_kv_gather(c.k_pages, c.v_pages, i32(c.table), i32(c.seq), i32(c.pos), k, v)
    x = c.v.astype(np.float64)
    sc = np.repeat(ref.quantise(x)[1], 32, -1)
    assert sc.min() >= 2.0 ** -126
    for t in (k, v):  # half a scale, and half a step of bf16 (2^-134 where it is subnormal)
        got = host(t).astype(np.float64)
        assert np.all(np.abs(got - x) <= 0.5 * sc + np.maximum(2.0 ** -8 * np.abs(got), 2.0 ** -134) + 2.0 ** -149)


@pytest.mark.parametrize("d,P,fmt,out_len", [(128, 16, "bf16", 1), (64, 64, "bf16", 4), (128, 32, "q4", 1),
                                             (64, 16, "q4", 3), (64, 256, "q4", 1)])
def test_gather_reads_what_stands_there(d, P, fmt, out_len):
    r = np.random.default_rng(5)
    N, Hkv, B, M, T = 9, 3, 2, 4, 24
    if fmt == "bf16":
        kp, vp = (torch.randn(N, Hkv, P, d, device="cuda").bfloat16() for _ in range(2))
        kv, vv = host(kp), host(vp)
    else:
        recs = []
        for value in (False, True):
            codes = r.integers(0, 16, (N, Hkv, P // 16, 16, d))
            sc = ref.bf16_value(ref.bf16_bits(r.uniform(0.1, 0.4, (N, Hkv, P // 16, 16, d // 32))))
            recs.append(ref.pack(codes, sc, -8 * sc, value))
        kp, vp = (torch.from_numpy(x).cuda() for x in recs)
        kv, vv = (ref.record_values(x, d, i == 1).reshape(N, Hkv, P, d) for i, x in enumerate(recs))
    table = r.permutation(N)[:B * M].reshape(B, M)
    seq, pos = r.integers(0, B, T), r.integers(0, M * P, T)  # repeats allowed
    seq[5], pos[3] = -1, M * P - 1
    k, v = (torch.full((T // out_len, Hkv, out_len, d), 7.0, device="cuda", dtype=torch.bfloat16)
            for _ in range(2))
    sk.sskip_kv_gather(kp, vp, i32(table), i32(seq), i32(pos), k, v)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    for t, x in ((k, kv), (v, vv)):
        got = host(t).swapaxes(1, 2).reshape(T, Hkv, d)
        for i in range(T):
            if seq[i] < 0:
                assert np.all(got[i] == 7)
                continue
            want = x[table[seq[i], pos[i] // P], :, pos[i] % P]
            # one fp32 multiply-add, then half a bf16 step
            assert np.all(np.abs(got[i] - want) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(want) + 2.0 ** -20)


def test_append_in_two_halves_equals_one_call():
    a, b = Case(fmt="q4", pad=0, P=32), Case(fmt="q4", pad=0, P=32)
    a.run()
    for part in (slice(0, 4), slice(4, None)):
        half = lambda t: t[part]  # noqa: E731
        sk.sskip_kv_append(half(b.q_t), half(b.k_t), half(b.v_t), i32(b.seq[part]), i32(b.pos[part]),
                           q_out=half(b.q_out), k_out=half(b.k_out), v_out=half(b.v_out),
                           k_pages=b.k_pages, v_pages=b.v_pages, block_table=i32(b.table),
                           turns=torch.from_numpy(b.turns).cuda(), q_weight=b.qw_t,
                           k_weight=b.kw_t, eps=b.eps)
    torch.cuda.synchronize()
    for n in ("q_out", "k_out", "v_out", "k_pages", "v_pages"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n

"""The decode over the paged cache, both formats, against the 64-bit rule."""
import numpy as np
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
import paged_reference as ref
from parity_helpers import NEAR_TIE, note_flips

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_long_tiled_b200 import build
    build.build()
    assert torch.cuda.is_available()


def bf16(x):
    bits = ref.bf16_bits(np.asarray(x, np.float32))
    t = torch.from_numpy(bits.view(np.int16).copy()).cuda().view(torch.bfloat16)
    return t, ref.bf16_value(bits)


class Case:
    def __init__(self, lens, seed=1, Hq=8, Hkv=2, d=128, P=64, fmt="bf16", tsf=0.0, splits=4,
                 spare=1, planted=True, garbage=True):
        r = np.random.default_rng(seed)
        self.__dict__.update(lens=np.asarray(lens), Hq=Hq, Hkv=Hkv, d=d, P=P, fmt=fmt, tsf=tsf,
                             splits=splits, scale=d ** -0.5)
        B = len(lens)
        need = [max(1, -(-n // P)) for n in lens]
        M = max(need) + spare
        N = sum(need) + 2
        perm = r.permutation(N)
        # Entries past a sequence's pages are never read: they may be anything.
        self.table = r.integers(-(2 ** 31), 2 ** 31, (B, M))
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        u = np.repeat(r.choice([-1.0, 1.0], d // 32), 32) if planted else np.zeros(d)
        self.q_t, self.q = bf16(r.standard_normal((B, Hq, d)) + 0.5 * u)
        K, V = r.standard_normal((N, Hkv, P, d)), r.standard_normal((N, Hkv, P, d))
        hot = r.random((N, Hkv, max(1, P // 64))) < 0.3
        K += 2.0 * np.repeat(hot, min(P, 64), 2)[..., None] * u
        if fmt == "bf16":
            (k_t, k), (v_t, v) = bf16(K), bf16(V)
        else:
            pages = []
            for x, value in ((K, False), (V, True)):
                codes, sc, mn = ref.quantise(x.reshape(N, Hkv, P // 16, 16, d))
                pages.append(ref.pack(codes, sc, mn, value))
            (k, v), (k_t, v_t) = pages, [torch.from_numpy(x.copy()).cuda() for x in pages]
        self.k, self.v = k, v
        if garbage:  # rows behind the last key: NaN, infinities
            for b, n in enumerate(self.lens):
                page, off = (self.table[b, n // P], n % P) if n < need[b] * P else (None, 0)
                if page is None:
                    continue
                for t, value in ((k_t, False), (v_t, True)):
                    if fmt == "bf16":
                        t[page, :, off:] = float("inf") if value else float("nan")
                        t[page, :, off + 1::2] = float("nan")
                    else:
                        for row in range(off, P):
                            rec = t[page, :, row // 16, 8 * d:].view(Hkv, 16, -1)
                            rec[:, row % 16] = 0xFF  # scales and minima are NaN
        self.k_t, self.v_t = k_t, v_t

    def run(self, splits=None, workspace=None, stream=None, tsf=None):
        B, S = len(self.lens), self.splits if splits is None else splits
        o = torch.full((B, self.Hq, self.d), 9.0, device="cuda", dtype=torch.bfloat16)
        lse = torch.full((B, self.Hq), 9.0, device="cuda")
        ws = torch.full((sk.sskip_attn_decode_workspace_size(B, self.Hq, self.d, S),), 0xFF,
                        device="cuda", dtype=torch.uint8) if workspace is None else workspace
        state = torch.full((B, self.Hkv, -(-self.table.shape[1] * self.P // 64)), 9, device="cuda",
                           dtype=torch.uint8)
        count = torch.full((2,), 77, device="cuda", dtype=torch.int64)
        sk.sskip_attn_decode_paged(
            self.q_t, self.k_t, self.v_t, torch.from_numpy(self.table.astype(np.int32)).cuda(),
            torch.tensor(self.lens, dtype=torch.int32, device="cuda"), o, lse, sm_scale=self.scale,
            threshold_scale_factor=self.tsf if tsf is None else tsf, num_splits=S, workspace=ws,
            skip_count=count, tile_state=state, stream=stream)
        torch.cuda.synchronize()
        assert sk.sskip_get_status() == sk.SSKIP_OK
        return {"o": o.float().cpu().numpy(), "lse": lse.cpu().numpy(),
                "tile_state": state.cpu().numpy(), "count": count.tolist()}

    def check(self, got=None, splits=None):
        got = self.run(splits) if got is None else got
        args = (self.q, self.k, self.v, self.table, self.lens, self.scale, self.tsf,
                self.splits if splits is None else splits)
        want = ref.decode(*args)
        flips = want["tile_state"] != got["tile_state"]
        if flips.any():  # only where the decision quantity sits on the border
            assert np.all((want["tile_state"] > 0) == (got["tile_state"] > 0))
            assert np.abs(want["margin"][flips]).max() < NEAR_TIE
            want = ref.decode(*args, tiles=got["tile_state"])
        note_flips(int((want["tile_state"] > 0).sum()), want["margin"][flips])
        tol_o, tol_l = ref.decode_tolerance(want, max(1, int(self.lens.max())))
        empty = self.lens == 0
        assert np.all(got["o"][empty] == 0) and np.all(got["lse"][empty] == -np.inf)
        full = ~empty
        assert np.all(np.isfinite(got["o"])) and np.all(np.isfinite(got["lse"][full]))
        d_o = np.abs(got["o"] - want["o"])[full]
        d_l = np.abs(got["lse"][full] - want["lse"][full])
        assert np.all(d_o <= tol_o[full]), float((d_o / tol_o[full]).max())
        assert np.all(d_l <= tol_l[full]), float((d_l / tol_l[full]).max())
        st = got["tile_state"]
        assert got["count"] == [int((st == 2).sum()), int((st > 0).sum())]
        return got


FMT = pytest.mark.parametrize("fmt", ["bf16", "q4"])


@FMT
@pytest.mark.parametrize("tsf", [0.0, 4.0, 60.0])
@pytest.mark.parametrize("kw", [
    dict(), dict(d=64), dict(P=16), dict(P=32, d=64), dict(P=128), dict(P=256, d=64),
    dict(Hq=2, Hkv=2), dict(Hq=4, Hkv=2, d=64), dict(Hq=16, Hkv=2), dict(Hq=8, Hkv=1, d=64, P=16),
    dict(splits=1), dict(splits=2), dict(splits=64), dict(splits=1, P=16, d=64),
    dict(splits=3), dict(splits=5, d=64), dict(splits=7, P=16), dict(splits=8), dict(splits=9),
], ids=str)
def test_ragged_batch(kw, tsf, fmt):
    c = Case([700, 0, 1, 65, 333, 64], fmt=fmt, tsf=tsf, **kw)
    got = c.check()
    if tsf == 0:
        assert got["count"][0] == 0


@FMT
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 47, 48, 63, 64, 65, 80, 127, 128, 129, 1023])
@pytest.mark.parametrize("P", [16, 64])
def test_every_kind_of_last_tile(n, P, fmt):
    for splits, tsf in ((1, 0.0), (3, 0.0), (2, 0.3)):
        Case([n], fmt=fmt, P=P, splits=splits, tsf=tsf, seed=n).check()


@FMT
@pytest.mark.parametrize("kw", [dict(), dict(d=64, P=16), dict(splits=1, Hq=16, Hkv=16)], ids=str)
def test_more_ctas_than_two_an_sm(kw, fmt):
    # 320 or more: no clusters, and (4-bit) one slot a warp
    kw = dict(dict(splits=10, Hq=16, Hkv=8), **kw)
    lens = [2100, 0, 1, 65, 700, 64, 1025, 17] if kw["splits"] > 1 else [1025, 0, 1, 65] * 5
    got = Case(lens[:4] if kw["splits"] > 1 else lens, fmt=fmt, **kw).check()
    assert got["count"][0] == 0


@FMT
@pytest.mark.parametrize("tsf", [0.0, 500.0])
def test_long_sequences(tsf, fmt):
    # rings go round many times, splits of uneven length
    got = Case([9001, 4160, 12000], fmt=fmt, tsf=tsf, splits=5, Hq=8, Hkv=1).check()
    if tsf:
        assert got["count"][0] > 0.3 * got["count"][1]


@FMT
def test_a_factor_of_the_length_and_more(fmt):
    # t >= 1: a tile may pass although it raises the maximum; the literal rule
    Case([300, 130], fmt=fmt, tsf=400.0, splits=1).check()


@FMT
@pytest.mark.parametrize("tsf", [0.0, 2.0])
def test_scores_of_large_spread(tsf, fmt):
    # rising scores: the reference of the exponent moves again and again
    c = Case([1500], fmt=fmt, tsf=tsf, splits=2, planted=False, garbage=False)
    c.q_t, c.q = bf16(c.q * 12)
    c.check()


@FMT
def test_equal_scores(fmt):
    c = Case([200], fmt=fmt, planted=False, garbage=False)
    c.q_t, c.q = bf16(c.q * 0)
    c.check()


@FMT
def test_nan_and_infinite_keys_reach_their_rows_alone(fmt):
    c = Case([100, 100], fmt=fmt, garbage=False)
    page = int(c.table[0, 0])
    if fmt == "bf16":
        c.k_t[page, 0, 3] = float("nan")
    else:
        c.k_t[page, 0, 0, 8 * 128:] = 0xFF
    got = c.run()
    assert np.isnan(got["o"][0, :4]).all() and np.isnan(got["lse"][0, :4]).all()
    assert np.isfinite(got["o"][0, 4:]).all() and np.isfinite(got["o"][1]).all()


@FMT
def test_shared_pages(fmt):
    # two sequences with a common prefix read the same pages
    c = Case([128, 300], fmt=fmt, P=64, garbage=False)
    c.table[0, :2] = c.table[1, :2]
    c.check()


@FMT
@pytest.mark.parametrize("bad", [-3, 10 ** 6])
def test_bad_length_is_latched_and_clamped(bad, fmt):
    c = Case([256, 100], fmt=fmt, P=64, spare=0, garbage=False)
    full = c.table.copy()
    full[1] = full[0]  # every page in range
    c.table = full
    lens = torch.tensor([100, bad], dtype=torch.int32, device="cuda")
    o = torch.empty(2, 8, 128, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(2, 8, device="cuda")
    sk.sskip_attn_decode_paged(c.q_t, c.k_t, c.v_t, torch.from_numpy(full.astype(np.int32)).cuda(),
                               lens, o, lse, sm_scale=c.scale, threshold_scale_factor=0.0,
                               num_splits=1)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_ERR_INVALID_ARG
    c.lens = np.array([100, 0 if bad < 0 else 256])
    want = c.run(splits=1)
    assert np.array_equal(o.float().cpu().numpy(), want["o"])
    assert np.array_equal(lse.cpu().numpy(), want["lse"])


@FMT
@pytest.mark.parametrize("tsf", [0.0, 4.0])
@pytest.mark.parametrize("bad", [-1, 99])
def test_bad_page_is_latched(bad, tsf, fmt):
    c = Case([300, 200], fmt=fmt, garbage=False)
    good = c.run(tsf=tsf)
    c.table[0, 1] = bad
    o = torch.empty(2, 8, 128, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(2, 8, device="cuda")
    ws = torch.empty(sk.sskip_attn_decode_workspace_size(2, 8, 128, 4), device="cuda", dtype=torch.uint8)
    sk.sskip_attn_decode_paged(c.q_t, c.k_t, c.v_t, torch.from_numpy(c.table.astype(np.int32)).cuda(),
                               torch.tensor(c.lens, dtype=torch.int32, device="cuda"), o, lse,
                               sm_scale=c.scale, threshold_scale_factor=tsf, num_splits=4, workspace=ws)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_ERR_INVALID_ARG
    assert np.array_equal(o[1].float().cpu().numpy(), good["o"][1])  # the other sequence


@FMT
def test_the_same_call_twice_and_on_another_stream(fmt):
    c = Case([1000, 64, 513], fmt=fmt, tsf=4.0)
    a = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = c.run(stream=s)
    for n in ("o", "lse", "tile_state"):
        assert np.array_equal(a[n], b[n]), n


def test_contiguous_and_paged_decode_take_the_same_decisions():
    c = Case([640, 1000], tsf=20.0, splits=4, garbage=False)
    got = c.check()
    Lmax = c.table.shape[1] * c.P
    rows = lambda t: torch.stack([t[torch.from_numpy(np.where(  # noqa: E731
        (row >= 0) & (row < t.shape[0]), row, 0)).cuda()].transpose(0, 1).flatten(1, 2)
        for row in c.table]).contiguous()
    kc, vc = rows(c.k_t), rows(c.v_t)
    assert kc.shape == (2, c.Hkv, Lmax, c.d)
    out = sk.decode(c.q_t, kc, vc, torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                    sm_scale=c.scale, threshold_scale_factor=20.0, num_splits=4, with_tiles=True)
    assert np.array_equal(out["tile_state"].cpu().numpy(), got["tile_state"])
    # fp32 probabilities there, bf16 here: half a step of each weight and of o
    assert np.abs(out["o"].float().cpu().numpy() - got["o"]).max() < 2.0 ** -6 * np.abs(got["o"]).max()


@FMT
@pytest.mark.parametrize("tsf", [0.0, 4.0])
def test_captured_and_replayed_on_new_inputs(tsf, fmt):
    a, b = Case([500, 77], fmt=fmt, tsf=tsf, seed=4), Case([310, 450], fmt=fmt, tsf=tsf, seed=9)
    want = [x.run() for x in (a, b)]
    M = max(a.table.shape[1], b.table.shape[1])
    N = max(a.k_t.shape[0], b.k_t.shape[0])
    pages = lambda x: torch.cat([x, x.new_zeros(N - x.shape[0], *x.shape[1:])])  # noqa: E731
    wide = lambda x: torch.from_numpy(np.pad(x, ((0, 0), (0, M - x.shape[1]))).astype(np.int32)).cuda()  # noqa: E731
    lens = lambda x: torch.tensor(x.lens, dtype=torch.int32, device="cuda")  # noqa: E731
    st = [a.q_t.clone(), pages(a.k_t), pages(a.v_t), wide(a.table), lens(a)]
    o, lse = torch.empty_like(st[0]), torch.empty(2, 8, device="cuda")
    ws = torch.empty(sk.sskip_attn_decode_workspace_size(2, 8, 128, 4), device="cuda", dtype=torch.uint8)
    call = lambda: sk.sskip_attn_decode_paged(*st, o, lse, sm_scale=a.scale, num_splits=4,  # noqa: E731
                                              threshold_scale_factor=tsf, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x, w in ((a, want[0]), (b, want[1])):
        for dst, src in zip(st, (x.q_t, pages(x.k_t), pages(x.v_t), wide(x.table), lens(x))):
            dst.copy_(src)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(o.float().cpu().numpy(), w["o"])
        assert np.array_equal(lse.cpu().numpy(), w["lse"])
    del g

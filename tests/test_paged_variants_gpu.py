"""The paged calls at the sizes where their dispatch changes: the warps of a
token in the append and the gather, the slots of a warp in the 4-bit decode."""
import numpy as np
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
import paged_reference as ref
import test_paged_cache_gpu as cache
import test_paged_decode_gpu as decode
from test_paged_cache_gpu import _built, host, i32  # noqa: F401  (the fixture builds)

pytestmark = pytest.mark.gpu
FMT = pytest.mark.parametrize("fmt", ["bf16", "q4"])


@FMT
@pytest.mark.parametrize("kw", [
    dict(), dict(d=64), dict(rot=48, interleaved=True), dict(d=64, rot=48), dict(norm=False, rot=0)],
    ids=str)
def test_append_with_a_warp_a_token(kw, fmt):
    """More tokens than 16 an SM, the last CTA of four not full."""
    c = cache.Case(fmt=fmt, counts=(1500, 3, 860), starts=(5, 0, 100), pad=10, P=64, Hq=4, Hkv=1, **kw)
    assert c.T == 2373
    c.run()
    c.check()


def pieces(c, n):
    """The append of c in calls of n tokens."""
    for a in range(0, c.T, n):
        s = slice(a, a + n)
        sk.sskip_kv_append(c.q_t[s], c.k_t[s], c.v_t[s], i32(c.seq[s]), i32(c.pos[s]),
                           q_out=c.q_out[s], k_out=c.k_out[s], v_out=c.v_out[s],
                           k_pages=c.k_pages, v_pages=c.v_pages, block_table=i32(c.table),
                           turns=torch.from_numpy(c.turns).cuda(), interleaved=c.interleaved,
                           attn_factor=c.attn, q_weight=c.qw_t, k_weight=c.kw_t, eps=c.eps)
    torch.cuda.synchronize()


@FMT
@pytest.mark.parametrize("T", [888, 889, 1184, 1185, 2368, 2369, 2371])
@pytest.mark.parametrize("kw", [
    dict(Hq=32, Hkv=8), dict(Hq=32, Hkv=8, d=64), dict(Hq=5, Hkv=3, rot=80),
    dict(Hq=16, Hkv=2, d=64, interleaved=True, rot=32)], ids=str)
def test_a_token_does_not_depend_on_the_size_of_its_call(kw, T, fmt):
    """Every row and record to the bit what calls of 37 tokens make of it (the
    sizes that the 64-bit forms check): 12, 6, 4 and 3 warps a token or one."""
    a, b = (cache.Case(fmt=fmt, counts=(T - 50, 41), starts=(9, 0), pad=9, P=32, **kw) for _ in range(2))
    assert a.T == T
    a.run()
    pieces(b, 37)
    for n in ("q_out", "k_out", "v_out", "k_pages", "v_pages"):
        assert torch.equal(getattr(a, n), getattr(b, n)), n


@FMT
@pytest.mark.parametrize("d,P", [(128, 64), (64, 16)])
@pytest.mark.parametrize("T,out_len", [(600, 1), (2500, 5), (9601, 1)])
def test_gather_with_fewer_warps_than_groups_of_heads(T, out_len, d, P, fmt):
    """8 kv heads: four (d = 64: two) groups for keys and values, walked by
    four warps a token, by three, and by one."""
    r = np.random.default_rng(T)
    B, M, Hkv = 3, 4096 // P, 8
    N = B * M + 1
    k, v = sk.paged_cache(N, Hkv, P, d, int4=fmt == "q4")
    if fmt == "bf16":
        for x in (k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
    else:
        for x in (k, v):
            x.copy_(torch.randint(0, 256, x.shape, device="cuda", dtype=torch.uint8))
            x[..., 8 * d:].view(torch.bfloat16).copy_(torch.randn(*x.shape[:3], d, device="cuda"))
    table = r.permutation(N)[:B * M].reshape(B, M)
    seq, pos = r.integers(0, B, T), r.integers(0, M * P, T)
    seq[::97] = -1
    outs = [torch.full((T // out_len, Hkv, out_len, d), 7.0, device="cuda", dtype=torch.bfloat16)
            for _ in range(2)]
    sk.sskip_kv_gather(k, v, i32(table), i32(seq), i32(pos), *outs)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    live = seq >= 0
    page, off = table[seq, pos // P], pos % P
    for value, pages, out in ((False, k, outs[0]), (True, v, outs[1])):
        got = host(out).swapaxes(1, 2).reshape(T, Hkv, d)
        assert np.all(got[~live] == 7.0)
        if fmt == "bf16":
            want = host(pages[torch.from_numpy(page).cuda(), :, torch.from_numpy(off).cuda()])
            assert np.array_equal(got[live], want[live])
            continue
        rec = pages[torch.from_numpy(page).cuda(), :, torch.from_numpy(off // 16).cuda()]
        codes, sc, mn = ref.unpack(rec.cpu().numpy(), d, value)  # [T, Hkv, 16, ...]
        at = np.arange(T), slice(None), off % 16
        sc, mn = (np.repeat(x[at].astype(np.float64), 32, -1) for x in (sc, mn))
        want = mn + sc * codes[at]
        # one fp32 multiply-add (2^-24 of its result), then half a bf16 step
        tol = 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -23 * np.abs(want) + 2.0 ** -133
        assert np.all(np.abs(got - want)[live] <= tol[live])


@pytest.mark.parametrize("tsf", [0.0, 4.0])
@pytest.mark.parametrize("kw", [dict(d=64, P=16), dict(d=64, P=32), dict(d=128, P=16), dict(d=128, P=128)],
                         ids=str)
def test_4bit_decode_with_a_slot_a_warp_over_many_tiles(kw, tsf):
    """More CTAs than two an SM, splits of nine tiles and more: a slot's copies,
    its phase and the look-up of pages go round, the last tile ragged."""
    lens = [2340, 2304, 2305, 577, 0, 64, 1, 2303, 1500, 2176]
    c = decode.Case(lens, fmt="q4", Hq=16, Hkv=8, splits=4, tsf=tsf, **kw)
    assert len(lens) * c.Hkv * c.splits > 2 * 148 and -(-max(lens) // 64) > 4 * 9
    c.check()


@FMT
@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("spare", [0, 70])
def test_the_default_number_of_splits(spare, tsf, fmt):
    """decode_paged chooses the splits from the block table: the rule with that
    number, a table just long enough and one of many times the longest sequence
    (most splits have no tile)."""
    c = decode.Case([700, 0, 1, 65, 333, 64], fmt=fmt, tsf=tsf, spare=spare)
    S = sk.paged_splits(len(c.lens), c.Hkv, c.table.shape[1] * c.P)
    out = sk.decode_paged(c.q_t, c.k_t, c.v_t, i32(c.table.astype(np.int32)), i32(c.lens),
                          sm_scale=c.scale, threshold_scale_factor=tsf, with_tiles=True)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    c.check({"o": host(out["o"]), "lse": out["lse"].cpu().numpy(),
             "tile_state": out["tile_state"].cpu().numpy(), "count": out["counts"].tolist()}, splits=S)

"""NaN and infinite scores in the prefill and the contiguous decode: a NaN
reaches the rows it belongs to and no other, whatever the threshold; rows whose
scores are all -inf give O = 0 and lse = -inf."""
import pytest
import torch

import block_sparse_long_tiled_b200 as sk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_long_tiled_b200 import build
    build.build()
    assert torch.cuda.is_available()


def inputs(B, Hq, Hkv, L, d, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, h, L, d, device="cuda", generator=g).bfloat16() for h in (Hq, Hkv, Hkv)]


def dirty(*shape):
    """Memory that outputs may be allocated in holds numbers."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full(shape if dtype == torch.bfloat16 else shape[:-1], 3.0, device="cuda", dtype=dtype)
        del x


def call(form, q, k, v, **kw):
    dirty(*q.shape)
    if form == "lens":
        kw["seqlens"] = torch.full((q.shape[0],), q.shape[2], dtype=torch.int32, device="cuda")
    if form == "vote":
        kw["vote_rows"] = 32
    out = sk.prefill(q, k, v, sm_scale=q.shape[3] ** -0.5, **kw)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    return out["o"], out["lse"]


FORM = pytest.mark.parametrize("form", ["plain", "lens", "vote"])
SHAPE = pytest.mark.parametrize("L,d,tile", [(40, 128, 128), (300, 128, 128), (300, 64, 64), (130, 64, 128)])


@FORM
@SHAPE
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tsf", [0.0, 3.0])
def test_prefill_of_queries_of_nan(tsf, causal, L, d, tile, form):
    q, k, v = inputs(2, 2, 1, L, d)
    kw = dict(causal=causal, threshold_scale_factor=tsf, Br=tile, Bc=tile)
    clean = call(form, q, k, v, **kw)
    q[0, 0] = float("nan")       # a whole head
    q[1, 1, 17] = float("nan")   # one row
    o, lse = call(form, q, k, v, **kw)
    assert bool(o[0, 0].isnan().all()) and bool(lse[0, 0].isnan().all())
    assert bool(o[1, 1, 17].isnan().all()) and bool(lse[1, 1, 17].isnan())
    o[0, 0], lse[0, 0] = clean[0][0, 0], clean[1][0, 0]
    o[1, 1, 17], lse[1, 1, 17] = clean[0][1, 1, 17], clean[1][1, 1, 17]
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    if tsf == 0:  # (with a threshold the row keeps tiles for its query tile)
        assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


@FORM
@SHAPE
@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("at", [0, 33])
def test_prefill_of_a_key_of_nan(at, tsf, L, d, tile, form):
    q, k, v = inputs(1, 2, 2, L, d)
    kw = dict(causal=True, threshold_scale_factor=tsf, Br=tile, Bc=tile)
    clean = call(form, q, k, v, **kw)
    k[0, 0, at] = float("nan")
    o, lse = call(form, q, k, v, **kw)
    assert bool(o[0, 0, at:].isnan().all()) and bool(lse[0, 0, at:].isnan().all())
    assert torch.equal(o[0, 1], clean[0][0, 1]) and torch.equal(lse[0, 1], clean[1][0, 1])
    assert bool(torch.isfinite(o[0, 0, :at].float()).all())


@FORM
@SHAPE
@pytest.mark.parametrize("tsf", [0.0, 3.0])
def test_prefill_of_scores_of_minus_infinity(tsf, L, d, tile, form):
    q, k, v = inputs(2, 2, 1, L, d)
    kw = dict(causal=True, threshold_scale_factor=tsf, Br=tile, Bc=tile)
    q[0], k[0] = 1.0, 1.0
    k[0, :, :, 0] = float("-inf")
    clean = call(form, q[1:], k[1:], v[1:], **kw)
    o, lse = call(form, q, k, v, **kw)
    assert bool((o[0] == 0).all()) and bool((lse[0] == -float("inf")).all())
    assert torch.equal(o[1], clean[0][0]) and torch.equal(lse[1], clean[1][0])


@FORM
@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("d,tile", [(128, 128), (64, 64)])
def test_prefill_behind_tiles_of_minus_infinity(d, tile, tsf, form):
    """Keys of -inf scores at the front, a tile and more of them, leave the rows
    what the other keys alone make of them (non-causal: those keys' own call)."""
    q, k, v = inputs(1, 2, 1, 300, d)
    q.clamp_(min=0.125)
    k[:, :, :150] = float("-inf")
    o, lse = call(form, q, k, v, causal=False, threshold_scale_factor=0.0, Br=tile, Bc=tile)
    s = d ** -0.5 * q.double() @ k[:, :, 150:].double().transpose(2, 3)
    want = s.softmax(-1) @ v[:, :, 150:].double()
    # P in bf16 and O's own rounding: half a step each of o and of sum P |v|
    tol = 2.0 ** -7 * (want.abs() + s.softmax(-1) @ v[:, :, 150:].double().abs())
    assert bool(((o.double() - want).abs() <= tol).all())
    assert float((lse.double() - s.logsumexp(-1)).abs().max()) < 1e-3
    o, lse = call(form, q, k, v, causal=True, threshold_scale_factor=tsf, Br=tile, Bc=tile)
    assert bool((o[:, :, :150] == 0).all()) and bool((lse[:, :, :150] == -float("inf")).all())
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse[:, :, 150:]).all())


@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("splits", [1, 4, 12])
@pytest.mark.parametrize("paged", [False, True])
def test_decode_behind_tiles_of_minus_infinity(paged, splits, tsf):
    lens = torch.tensor([700, 130], dtype=torch.int32, device="cuda")
    _, k, v = inputs(2, 4, 2, 704, 128)
    q = torch.rand(2, 4, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    k[:, :, :130] = float("-inf")
    kw = dict(sm_scale=128 ** -0.5, threshold_scale_factor=tsf, num_splits=splits)
    if paged:
        pages = [x.unflatten(2, (11, 64)).transpose(1, 2).flatten(0, 1).contiguous() for x in (k, v)]
        table = torch.arange(22, device="cuda", dtype=torch.int32).view(2, 11)
        got = sk.decode_paged(q, *pages, table, lens, **kw)
    else:
        got = sk.decode(q, k, v, lens, **kw)
    torch.cuda.synchronize()
    assert bool((got["o"][1] == 0).all()) and bool((got["lse"][1] == -float("inf")).all())
    assert bool(torch.isfinite(got["o"][0].float()).all()) and bool(torch.isfinite(got["lse"][0]).all())
    if tsf == 0:
        s = 128 ** -0.5 * torch.einsum("hgd,hnd->hgn", q[0].double().unflatten(0, (2, 2)), k[0, :, 130:700].double())
        want = torch.einsum("hgn,hnd->hgd", s.softmax(-1), v[0, :, 130:700].double()).flatten(0, 1)
        assert float((got["o"][0].double() - want).abs().max()) < 4e-3  # half a step below 1, and more
        assert float((got["lse"][0].double() - s.logsumexp(-1).flatten()).abs().max()) < 1e-3


@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("splits", [1, 4, 12])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [2, 8])
def test_contiguous_decode_of_nan(Hq, d, splits, tsf):
    lens = torch.tensor([50, 700, 64, 1], dtype=torch.int32, device="cuda")
    _, k, v = inputs(4, Hq, 2, 700, d)
    q = torch.randn(4, Hq, d, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    kw = dict(sm_scale=d ** -0.5, threshold_scale_factor=tsf, num_splits=splits, with_tiles=True)
    clean = sk.decode(q, k, v, lens, **kw)
    q[:, 0] = float("nan")
    got = sk.decode(q, k, v, lens, **kw)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    assert bool(got["o"][:, 0].isnan().all()) and bool(got["lse"][:, 0].isnan().all())
    G = Hq // 2
    assert bool(torch.isfinite(got["o"][:, 1:].float()).all()) and bool(torch.isfinite(got["lse"][:, 1:]).all())
    for n in ("o", "lse"):
        assert torch.equal(got[n][:, G:], clean[n][:, G:])
    st = got["tile_state"]
    assert not bool((st[:, 0] == 2).any()) and torch.equal(st[:, 1], clean["tile_state"][:, 1])
    # a key of NaN: its kv head's outputs, the other's unchanged
    k[1, 0, 333] = float("nan")
    q[:, 0] = 1.0
    got = sk.decode(q, k, v, lens, **kw)
    torch.cuda.synchronize()
    assert bool(got["o"][1, :G].isnan().all()) and bool(got["lse"][1, :G].isnan().all())
    assert torch.equal(got["o"][1, G:], clean["o"][1, G:])
    assert bool(torch.isfinite(got["o"][[0, 2, 3]].float()).all())


@pytest.mark.parametrize("tsf", [0.0, 20.0])
def test_no_factor_skips_a_tile_of_nan(tsf):
    """The critical values: +inf for every tile of the rows that a NaN query
    makes its query tile keep, and the call's own decisions follow the record."""
    L = 384
    q, k, v = inputs(1, 2, 1, L, 64)
    q[0, 0, 200] = float("nan")
    o, lse = torch.empty_like(q), torch.empty(1, 2, L, device="cuda")
    crit = torch.empty(1, 2, 3, 3, device="cuda")
    state = torch.empty(1, 2, 3, 3, device="cuda", dtype=torch.uint8)
    sk.sskip_attn_prefill_vote(q, k, v, o, lse, causal=True, sm_scale=0.125, threshold_scale_factor=tsf,
                               vote_rows=128, tile_state=state, tile_crit=crit)
    torch.cuda.synchronize()
    assert crit[0, 0, 1, :2].tolist() == [float("inf")] * 2 and state[0, 0, 1, :2].tolist() == [1, 1]
    assert bool(torch.isfinite(crit[0, 1, 1, 1]))  # the other head's
    if tsf:
        seen = state > 0
        assert torch.equal(state[seen] == 2, crit[seen] < torch.tensor(tsf, device="cuda").log())
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    qd = q[:, :, 200].contiguous()
    crit = torch.empty(1, 1, 6, device="cuda")
    state = torch.empty(1, 1, 6, device="cuda", dtype=torch.uint8)
    ws = torch.empty(sk.sskip_attn_decode_workspace_size(1, 2, 64, 2), device="cuda", dtype=torch.uint8)
    sk.sskip_attn_decode_crit(qd, k, v, lens, torch.empty_like(qd), torch.empty(1, 2, device="cuda"),
                              sm_scale=0.125, threshold_scale_factor=tsf, num_splits=2, workspace=ws,
                              tile_state=state, tile_crit=crit)
    torch.cuda.synchronize()
    assert crit.flatten().tolist() == [float("inf")] * 6 and state.flatten().tolist() == [1] * 6

"""NaN scores in the contiguous decode: a NaN reaches the rows it belongs to
and no other, whatever the threshold."""
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

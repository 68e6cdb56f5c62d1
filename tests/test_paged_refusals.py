"""What the paged calls refuse besides bad shapes: outputs in the memory of
tables, indices and counters, and arguments that are missing altogether."""
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
from test_paged_cache_host import (INVALID, append, append_tensors, at, bf, decode, gather, ints,
                                   lib)  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("kw", [
    dict(qo=at(3)), dict(ko=at(4)), dict(vo=at(3, 16 - 4 * 2 * 128 * 2)), dict(qo=at(5)),
    dict(ko=at(6, 240)), dict(vo=at(7)), dict(qo=at(7, 496)), dict(ko=at(13, 16)), dict(kp=at(13)),
    dict(vp=at(3)),
], ids=str)
def test_append_refuses_outputs_in_its_indices(lib, kw):  # noqa: F811
    assert append(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(ko=at(2)), dict(vo=at(2, 16)), dict(ko=at(3)), dict(vo=at(4)),
    dict(ko=at(4, 16 - 4 * 2 * 64 * 2)),
], ids=str)
def test_gather_refuses_outputs_in_its_indices(lib, kw):  # noqa: F811
    assert gather(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(o=at(3)), dict(o=at(4)), dict(lse=at(3, 28)), dict(lse=at(4, 4)), dict(ws=at(3)),
    dict(ws=at(4)), dict(count=at(0)), dict(count=at(1, 64)), dict(count=at(3, 16)),
    dict(count=at(5)), dict(count=at(6, 56)), dict(count=at(7)), dict(state=at(0, 100)),
    dict(state=at(2)), dict(state=at(3, 31)), dict(state=at(4)), dict(state=at(5, 1)),
    dict(state=at(6)), dict(state=at(7, 8)), dict(count=at(8), state=at(8, 15)),
], ids=str)
def test_decode_refuses_outputs_in_what_it_reads_or_counts(lib, kw):  # noqa: F811
    assert decode(lib, **kw) == INVALID


def test_missing_arguments_are_named(lib):  # noqa: F811
    a = append_tensors(q=None, k=None, v=None)
    with pytest.raises(ValueError, match="q, or k and v, must be given"):
        sk.sskip_kv_append(**a)
    with pytest.raises(TypeError, match="q must be a tensor"):
        sk.sskip_kv_append(**append_tensors(q=3))
    pages, i, o = bf(3, 2, 16, 64), ints(5), bf(5, 2, 64)
    with pytest.raises(ValueError, match="k_pages is missing"):
        sk.sskip_kv_gather(None, pages, ints(2, 4), i, i, o, o)
    with pytest.raises(ValueError, match="q is missing"):
        sk.sskip_attn_decode_paged(None, pages, pages, ints(2, 4), ints(2), o, torch.zeros(2, 8),
                                   sm_scale=0.1, threshold_scale_factor=0.0, num_splits=1)


@pytest.mark.parametrize("B,Hkv,n", [(0, 8, 1000), (1, 8, 0), (1, 1, 1), (64, 8, 32768), (1, 8, 1 << 30)])
def test_default_splits_are_ones_a_call_takes(B, Hkv, n):
    assert 1 <= sk.paged_splits(B, Hkv, n) <= 64

"""A NaN in the queries or keys of a paged decode reaches the rows it belongs
to, whatever the threshold, the splits and the length, and no other."""
import numpy as np
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
import paged_reference as ref
from test_paged_decode_gpu import FMT, Case, _built  # noqa: F401  (the fixture builds)

pytestmark = pytest.mark.gpu

LENS = [50, 700, 64, 0, 1]  # below a tile, several rounds, a whole tile, none, one key


@FMT
@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("splits", [1, 4, 12])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [2, 8])  # G = 1 and 4
def test_a_query_of_nan_gives_nan(Hq, d, splits, tsf, fmt):
    """Of a head whose query is NaN both outputs are, except of a sequence
    without keys; the heads of the other kv head are those of clean queries."""
    c = Case(LENS, fmt=fmt, tsf=tsf, splits=splits, Hq=Hq, d=d)
    clean = c.check()
    c.q_t[:, 0] = float("nan")
    got = c.run()
    full = c.lens > 0
    assert np.isnan(got["o"][full, 0]).all() and np.isnan(got["lse"][full, 0]).all()
    assert np.all(got["o"][~full] == 0) and np.all(got["lse"][~full] == -np.inf)
    G = Hq // 2
    assert np.isfinite(got["o"][:, 1:]).all() and np.isfinite(got["lse"][full, 1:]).all()
    for n in ("o", "lse"):
        assert np.array_equal(got[n][:, G:], clean[n][:, G:])
    # a NaN maximum is below no border: nothing the head looks at is skipped
    st = got["tile_state"]
    assert not np.any(st[:, 0] == 2) and np.array_equal(st > 0, clean["tile_state"] > 0)
    assert np.array_equal(st[:, 1], clean["tile_state"][:, 1])
    # the group's other heads saw every tile of theirs, as without a threshold
    if G > 1:
        c.q[:, 0] = 0.0
        want = ref.decode(c.q, c.k, c.v, c.table, c.lens, c.scale, 0.0, splits)
        tol_o, tol_l = ref.decode_tolerance(want, max(LENS))
        assert np.all(np.abs(got["o"] - want["o"])[full, 1:G] <= tol_o[full, 1:G])
        assert np.all(np.abs(got["lse"] - want["lse"])[full, 1:G] <= tol_l[full, 1:G])


@FMT
@pytest.mark.parametrize("splits", [1, 3, 12])
@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("at", [0, 33])
def test_a_key_of_nan_under_a_threshold(at, n, splits, fmt):
    """One key: its tile's maximum is NaN, and so are the outputs of its kv
    head; the other one's and the other sequence's are those without it."""
    c = Case([n, n], fmt=fmt, tsf=3.0, splits=splits, P=64)
    clean = c.run()
    page = int(c.table[0, 0])
    if fmt == "bf16":
        c.k_t[page, 0, at] = float("nan")
    else:
        c.k_t[page, 0, at // 16, 8 * 128:].view(16, -1)[at % 16] = 0xFF
    got = c.run()
    assert np.isnan(got["o"][0, :4]).all() and np.isnan(got["lse"][0, :4]).all()
    for n_ in ("o", "lse"):
        assert np.array_equal(got[n_][0, 4:], clean[n_][0, 4:])
        assert np.array_equal(got[n_][1], clean[n_][1])


@FMT
@pytest.mark.parametrize("splits", [1, 4, 12])
def test_every_key_of_nan(splits, fmt):
    """All of a sequence's keys: every tile of every split is NaN."""
    c = Case([300, 300], fmt=fmt, tsf=3.0, splits=splits, garbage=False)
    for page in c.table[0, :-(-300 // c.P)]:
        if fmt == "bf16":
            c.k_t[int(page)] = float("nan")
        else:
            c.k_t[int(page), :, :, 8 * 128:] = 0xFF
    got = c.run()
    assert np.isnan(got["o"][0]).all() and np.isnan(got["lse"][0]).all()
    assert np.isfinite(got["o"][1]).all() and np.isfinite(got["lse"][1]).all()
    assert got["count"][0] == int((got["tile_state"][1] == 2).sum())


@pytest.mark.parametrize("tsf", [0.0, 3.0])
@pytest.mark.parametrize("splits", [1, 4, 12])
def test_scores_of_minus_infinity_alone_leave_nothing(splits, tsf):
    """Keys whose scores are all -inf weigh nothing: O = 0 and lse = -inf for
    every number of splits, as of a sequence without keys. (A 4-bit group
    holds no infinity.)"""
    c = Case([200, 130], tsf=tsf, splits=splits, planted=False, garbage=False)
    c.q_t[0] = 1.0
    for page in c.table[0, :-(-200 // c.P)]:
        c.k_t[int(page)] = 1.0
        c.k_t[int(page), :, :, 0] = float("-inf")
    got = c.run()
    assert np.all(got["o"][0] == 0) and np.all(got["lse"][0] == -np.inf)
    assert np.isfinite(got["o"][1]).all() and np.isfinite(got["lse"][1]).all()

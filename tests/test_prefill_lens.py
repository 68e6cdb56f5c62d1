"""Prompts of their own lengths in one padded batch: each is what a call with
that prompt alone would make of it."""
import ctypes

import pytest
import torch

import block_sparse_long_tiled_b200 as sk
from test_paged_run_gpu import Layer, i32

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_long_tiled_b200 import build
    build.build()


# ------------------------------------------------------------- without a GPU
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)


@pytest.mark.parametrize("kw,rc", [
    (dict(lens=None), sk.SSKIP_ERR_INVALID_ARG), (dict(lens=ODD), sk.SSKIP_ERR_INVALID_ARG),
    (dict(q=None), sk.SSKIP_ERR_INVALID_ARG), (dict(L=0), sk.SSKIP_ERR_INVALID_ARG),
    (dict(tsf=-1.0), sk.SSKIP_ERR_INVALID_ARG), (dict(d=96), sk.SSKIP_ERR_UNSUPPORTED),
    (dict(Br=64), sk.SSKIP_ERR_UNSUPPORTED),
], ids=str)
def test_refuses(kw, rc):
    a = dict(q=FAKE, lens=FAKE, L=128, d=128, tsf=10.0, Br=128)
    a.update(kw)
    assert sk.lib().sskip_attn_prefill_lens(
        a["q"], FAKE, FAKE, a["lens"], FAKE, FAKE, 2, 4, 2, a["L"], a["d"], 1, 0.088, a["tsf"],
        a["Br"], 128, None, None, None) == rc


@pytest.mark.parametrize("lens,err", [
    (torch.zeros(2, dtype=torch.int64), TypeError), (torch.zeros(2, dtype=torch.int32), ValueError)])
def test_binding_refuses(lens, err):
    x = torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((err, ValueError)):
        sk.sskip_attn_prefill_lens(x, x, x, lens, x, torch.zeros(2, 2, 4), causal=True, sm_scale=0.1,
                                   threshold_scale_factor=0.0)
    with pytest.raises(ValueError):
        sk.prefill(x, x, x, causal=True, sm_scale=0.1, threshold_scale_factor=0.0, vote_rows=32,
                   seqlens=lens)


# --------------------------------------------------------------------- a GPU
def rows(B, H, L, d, g, hot=None):
    x = torch.randn(B, H, L, d, device="cuda", generator=g)
    if hot is not None:  # stretches of keys along one direction: tiles far below the maximum
        x += 2.0 * hot[:, None, :L, None]
    return x.bfloat16()


@gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tsf", [0.0, 8.0, 120.0])
@pytest.mark.parametrize("tile", [64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_each_entry_is_the_call_on_it_alone(d, tile, tsf, causal):
    lens = [513, 0, 1, 64, 65, 127, 129, 256, 257, 385]
    B, Hq, Hkv, L = len(lens), 4, 2, 513
    g = torch.Generator(device="cuda").manual_seed(d + tile)
    hot = (torch.rand(B, -(-L // 64), device="cuda", generator=g) < 0.3).float()
    hot = hot.repeat_interleave(64, 1)
    q = (torch.randn(B, Hq, L, d, device="cuda", generator=g) + 0.5).bfloat16()
    k, v = rows(B, Hkv, L, d, g, hot), rows(B, Hkv, L, d, g)
    for b, n in enumerate(lens):  # behind the end: anything, v finite
        q[b, :, n:] = float("nan")
        k[b, :, n:] = float("nan")
        k[b, :, n::2] = float("inf")
        v[b, :, n:] = 3e38
    kw = dict(causal=causal, sm_scale=d ** -0.5, threshold_scale_factor=tsf, Br=tile, Bc=tile,
              with_tiles=True)
    o = torch.full((B, Hq, L, d), float("nan"), device="cuda", dtype=torch.bfloat16)
    del o  # what the outputs may be allocated in
    got = sk.prefill(q, k, v, seqlens=i32(lens), **kw)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    counts = torch.zeros(2, dtype=torch.int64, device="cuda")
    for b, n in enumerate(lens):
        assert bool((got["o"][b, :, n:] == 0).all())
        assert bool((got["lse"][b, :, n:] == -float("inf")).all())
        nt = -(-n // tile)
        state = got["tile_state"][b]
        assert not bool(state[:, nt:].any()) and not bool(state[:, :, nt:].any())
        if n == 0:
            continue
        one = sk.prefill(*(x[b:b + 1, :, :n].contiguous() for x in (q, k, v)), **kw)
        assert torch.equal(got["o"][b, :, :n], one["o"][0])
        assert torch.equal(got["lse"][b, :, :n], one["lse"][0])
        assert torch.equal(state[:, :nt, :nt], one["tile_state"][0])
        assert bool(torch.isfinite(one["o"].float()).all())
        counts += one["counts"]
    assert torch.equal(got["counts"], counts)
    if tsf > 100:  # the factor matters here
        assert int(counts[0]) > 0.1 * int(counts[1])


@gpu
def test_full_length_entries_are_the_plain_call():
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (rows(2, h, 700, 128, g) for h in (4, 2, 2))
    kw = dict(causal=True, sm_scale=128 ** -0.5, threshold_scale_factor=300.0, with_tiles=True)
    a, b = sk.prefill(q, k, v, **kw), sk.prefill(q, k, v, seqlens=i32([700, 700]), **kw)
    for n in ("o", "lse", "counts", "tile_state"):
        assert torch.equal(a[n], b[n]), n


@gpu
@pytest.mark.parametrize("bad,clamped", [(-4, 0), (301, 300), (2 ** 31 - 1, 300)])
def test_bad_length_is_latched_and_clamped(bad, clamped):
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (rows(2, h, 300, 64, g) for h in (4, 2, 2))
    kw = dict(causal=True, sm_scale=0.125, threshold_scale_factor=2.0)
    a = sk.prefill(q, k, v, seqlens=i32([100, bad]), **kw)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_ERR_INVALID_ARG
    b = sk.prefill(q, k, v, seqlens=i32([100, clamped]), **kw)
    torch.cuda.synchronize()
    assert sk.sskip_get_status() == sk.SSKIP_OK
    assert torch.equal(a["o"], b["o"]) and torch.equal(a["lse"], b["lse"])


@gpu
def test_debug_build_matches_release():
    outs = []
    for lib in (sk.lib(), sk.debug_lib()):
        g = torch.Generator(device="cuda").manual_seed(7)
        q, k, v = (rows(3, h, 400, 128, g) for h in (4, 2, 2))
        keep, sk._lib = sk._lib, lib
        try:
            outs.append(sk.prefill(q, k, v, seqlens=i32([400, 0, 130]), causal=True, sm_scale=0.09,
                                   threshold_scale_factor=5.0, with_tiles=True))
            torch.cuda.synchronize()
            assert lib.sskip_get_status(None) == sk.SSKIP_OK
        finally:
            sk._lib = keep
    for n in ("o", "lse", "counts", "tile_state"):
        assert torch.equal(outs[0][n], outs[1][n]), n


@gpu
@pytest.mark.parametrize("int4", [False, True])
@pytest.mark.parametrize("tsf", [0.0, 2.0, 60.0])
def test_a_prompt_does_not_depend_on_its_batch(tsf, int4):
    """prefill_paged of a ragged batch against each prompt prefilled alone at
    its own length: outputs and decisions do not see the padding."""
    y = Layer(seed=31, B=3, int4=int4)
    L, lens = 280, [280, 131, 7]
    q, k, v = y.qkv(3 * L)
    k[:, :, :] *= torch.where((torch.arange(3 * L, device="cuda") // 64 % 3 == 0), 3.0, 0.3)[:, None, None]
    seq = torch.arange(3).repeat_interleave(L).int()
    pos = torch.arange(L).repeat(3).int().cuda()
    for b, n in enumerate(lens):
        seq[b * L + n:(b + 1) * L] = -1
    kw = dict(sm_scale=y.scale, threshold_scale_factor=tsf, **y.rope)
    got = sk.prefill_paged(q, k, v, seq.cuda(), pos, y.k_pages, y.v_pages, y.table, L=L, **kw)
    counts = torch.zeros(2, dtype=torch.int64, device="cuda")
    for b, n in enumerate(lens):
        s = slice(b * L, b * L + n)
        one = sk.prefill_paged(q[s], k[s], v[s], i32([b] * n), pos[:n].contiguous(), y.k_pages,
                               y.v_pages, y.table, L=n, **kw)
        assert torch.equal(got["o"][b, :, :n], one["o"][0])
        assert torch.equal(got["lse"][b, :, :n], one["lse"][0])
        assert bool((got["o"][b, :, n:] == 0).all())
        counts += one["counts"]
    assert torch.equal(got["counts"], counts)
    assert sk.sskip_get_status() == sk.SSKIP_OK


@gpu
def test_prefill_paged_makes_its_tensors_device_current(monkeypatch):
    """The prefill runs on the current device's stream: prefill_paged makes that
    of its tensors current, as the append and the decode do by themselves."""
    entered, seen = [], []
    real, prefill = torch.cuda.device, sk.prefill

    class Guard(real):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            entered.pop()
            return super().__exit__(*a)

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(sk, "prefill", lambda *a, **kw: (seen.append(list(entered)), prefill(*a, **kw))[1])
    y = Layer(seed=33, B=1)
    q, k, v = y.qkv(20)
    out = sk.prefill_paged(q, k, v, i32([0] * 20), i32(range(20)), y.k_pages, y.v_pages, y.table, L=20,
                           sm_scale=y.scale, threshold_scale_factor=0.0, **y.rope)
    torch.cuda.synchronize()
    assert seen == [[q.get_device()]] and out["o"].device == q.device


@gpu
def test_prefill_paged_captured_and_replayed_with_other_lengths():
    """A graph of a batch's prefill, replayed with prompts of other lengths, and
    the same call on a stream of its own."""
    y, L, B = Layer(seed=35, B=3), 200, 3
    kw = dict(L=L, sm_scale=y.scale, threshold_scale_factor=40.0, **y.rope)
    pos = torch.arange(L).repeat(B).int().cuda()

    def ids(lens):
        seq = torch.arange(B).repeat_interleave(L).int()
        for b, n in enumerate(lens):
            seq[b * L + n:(b + 1) * L] = -1
        return seq.cuda()

    q, k, v = (x.contiguous() for x in y.qkv(B * L))
    seq = ids([200, 130, 1])
    call = lambda st=None: sk.prefill_paged(q, k, v, seq, pos, y.k_pages, y.v_pages, y.table,  # noqa: E731
                                            stream=st, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for lens in ([200, 130, 1], [0, 64, 65], [129, 200, 128]):
        for x, n in zip((q, k, v), y.qkv(B * L)):
            x.copy_(n)
        seq.copy_(ids(lens))
        g.replay()
        got = {n: out[n].clone() for n in ("o", "lse", "counts")}
        side.wait_stream(torch.cuda.current_stream())
        want = call(side)
        torch.cuda.synchronize()
        assert sk.sskip_get_status() == sk.SSKIP_OK
        for n in got:
            assert torch.equal(got[n], want[n]), n
        for b, n in enumerate(lens):
            assert bool((got["o"][b, :, n:] == 0).all()) and bool(torch.isfinite(got["o"][b].float()).all())
    del g

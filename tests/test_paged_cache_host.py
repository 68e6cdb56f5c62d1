"""The paged cache without a GPU: what the calls refuse, the frequency table,
the sizes, and the reference's own packing."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_sparse_long_tiled_b200 as sk
import paged_reference as ref

INVALID, UNSUPPORTED = sk.SSKIP_ERR_INVALID_ARG, sk.SSKIP_ERR_UNSUPPORTED
GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    from block_sparse_long_tiled_b200 import build
    build.build()
    return sk.lib()


def at(i, off=0):
    """A fake device address, 1 GiB apart from the next, never dereferenced."""
    return ctypes.c_void_p((i + 1) * GB + off)


P, I, F, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong


class Cache(ctypes.Structure):
    _fields_ = [("kp", P), ("vp", P), ("table", P)] + [(n, I) for n in ("fmt", "N", "P", "M", "B")]


class AppendArgs(ctypes.Structure):
    _fields_ = ([("cache", Cache)] +
                [(n, P) for n in ("q", "k", "v", "seq", "pos", "qw", "kw", "turns", "qo", "ko", "vo")] +
                [(n, LL) for n in ("qs", "ks", "vs")] +
                [(n, I) for n in ("T", "Hq", "Hkv", "d", "rot", "inter", "out_len")] +
                [("eps", F), ("attn", F)])


class GatherArgs(ctypes.Structure):
    _fields_ = ([("cache", Cache)] + [(n, P) for n in ("seq", "pos", "ko", "vo")] +
                [(n, I) for n in ("T", "Hkv", "d", "out_len")])


class DecodeArgs(ctypes.Structure):
    _fields_ = ([("cache", Cache)] + [(n, P) for n in ("q", "lens", "o", "lse", "ws")] +
                [("ws_bytes", ctypes.c_size_t), ("count", P), ("state", P)] +
                [(n, I) for n in ("Hq", "Hkv", "d", "S")] + [("scale", F), ("tsf", F)])


def fill(kind, a):
    x = kind()
    for n, v in a.items():
        owner = x if n in dict(kind._fields_) else x.cache
        setattr(owner, n, v.value if isinstance(v, P) else v)
    return bytes(x)


@pytest.mark.parametrize("kind,want", [(AppendArgs, 48 + 11 * 8 + 3 * 8 + 7 * 4 + 2 * 4 + 4),
                                       (GatherArgs, 48 + 4 * 8 + 4 * 4),
                                       (DecodeArgs, 48 + 8 * 8 + 4 * 4 + 2 * 4)])
def test_struct_sizes(kind, want):
    """What a C compiler makes of the header's structs (3 pointers and 5 ints
    of the cache padded to 48 bytes, then each call's own fields)."""
    assert ctypes.sizeof(kind) == want


def append(lib, **kw):
    a = dict(q=at(0), k=at(1), v=at(2), qs=8 * 128, ks=2 * 128, vs=2 * 128, seq=at(3), pos=at(4),
             qw=at(5), kw=at(6), eps=1e-6, turns=at(7), rot=128, inter=0, attn=1.0, qo=at(8),
             ko=at(9), vo=at(10), out_len=1, kp=at(11), vp=at(12), table=at(13), fmt=0, N=10, P=64,
             M=4, T=4, B=2, Hq=8, Hkv=2, d=128)
    a.update(kw)
    return lib.sskip_kv_append(fill(AppendArgs, a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(ko=None), INVALID), (dict(vo=None), INVALID),
    (dict(q=at(0, 8)), INVALID), (dict(kp=at(11, 8)), INVALID), (dict(qw=at(5, 2)), INVALID),
    (dict(turns=at(7, 4)), INVALID), (dict(seq=at(3, 2)), INVALID), (dict(table=None), INVALID),
    (dict(seq=None), INVALID), (dict(pos=None), INVALID), (dict(turns=None), INVALID),
    (dict(T=-1), INVALID), (dict(T=5, out_len=2), INVALID), (dict(out_len=0), INVALID),
    (dict(qs=8 * 128 - 8), INVALID), (dict(ks=2 * 128 + 4), INVALID), (dict(vs=0), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(kp=None), INVALID),
    (dict(rot=130), INVALID), (dict(rot=-16), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(attn=float("inf")), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(P=48), UNSUPPORTED), (dict(P=8), UNSUPPORTED),
    (dict(P=512), UNSUPPORTED), (dict(fmt=2), UNSUPPORTED), (dict(M=0), INVALID),
    (dict(N=0), INVALID), (dict(B=0), INVALID), (dict(M=(1 << 24) + 1), UNSUPPORTED),
    (dict(N=1 << 25), UNSUPPORTED),
    # shared memory between an output and anything else
    (dict(qo=at(0)), INVALID), (dict(ko=at(1, 256)), INVALID), (dict(vo=at(9)), INVALID),
    (dict(kp=at(12)), INVALID), (dict(ko=at(11)), INVALID), (dict(vp=at(11, 2 * 64 * 256)), INVALID),
], ids=str)
def test_append_refuses(lib, kw, rc):
    assert append(lib, **kw) == rc


def test_calls_without_tokens_do_nothing(lib):
    assert append(lib, T=0) == sk.SSKIP_OK
    for f in (lib.sskip_kv_append, lib.sskip_kv_gather, lib.sskip_attn_decode_paged):
        assert f(None, None) == INVALID
    assert append(lib, T=0, q=None, k=None, v=None, qo=None) == sk.SSKIP_OK
    assert gather(lib, T=0) == sk.SSKIP_OK


def gather(lib, **kw):
    a = dict(kp=at(0), vp=at(1), table=at(2), seq=at(3), pos=at(4), ko=at(5), vo=at(6), out_len=1,
             fmt=1, N=10, P=64, M=4, T=4, B=2, Hkv=2, d=64)
    a.update(kw)
    return lib.sskip_kv_gather(fill(GatherArgs, a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(kp=None), INVALID), (dict(vp=at(0)), INVALID), (dict(table=None), INVALID),
    (dict(seq=None), INVALID), (dict(pos=None), INVALID), (dict(ko=None), INVALID),
    (dict(vo=at(5)), INVALID), (dict(ko=at(0, 1024)), INVALID), (dict(ko=at(5, 2)), INVALID),
    (dict(T=5, out_len=2), INVALID), (dict(T=-4), INVALID), (dict(d=32), UNSUPPORTED),
    (dict(P=96), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED),
], ids=str)
def test_gather_refuses(lib, kw, rc):
    assert gather(lib, **kw) == rc


def decode(lib, **kw):
    a = dict(q=at(0), kp=at(1), vp=at(2), table=at(3), lens=at(4), o=at(5), lse=at(6), fmt=0, B=2,
             Hq=8, Hkv=2, N=10, P=64, M=4, d=128, scale=0.1, tsf=5.0, S=4, ws=at(7),
             ws_bytes=1 << 20, count=None, state=None)
    a.update(kw)
    return lib.sskip_attn_decode_paged(fill(DecodeArgs, a), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=at(1)), INVALID),
    (dict(lens=None), INVALID), (dict(o=at(5, 2)), INVALID), (dict(lse=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws=at(7, 16)), INVALID), (dict(ws_bytes=1000), INVALID),
    (dict(count=at(8, 4)), INVALID), (dict(Hq=6, Hkv=4), INVALID), (dict(Hq=24), UNSUPPORTED),
    (dict(Hq=32), UNSUPPORTED), (dict(S=0), INVALID), (dict(S=65), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(tsf=-1.0), INVALID), (dict(tsf=float("nan")), INVALID),
    (dict(B=0), INVALID), (dict(d=80), UNSUPPORTED), (dict(P=80), UNSUPPORTED),
    (dict(fmt=7), UNSUPPORTED), (dict(B=70000), UNSUPPORTED), (dict(fmt=1, scale=1e13), UNSUPPORTED),
    (dict(o=at(0)), INVALID), (dict(o=at(0, 16)), INVALID), (dict(lse=at(0, 4)), INVALID),
    (dict(o=at(2, 1024)), INVALID), (dict(ws=at(1)), INVALID), (dict(ws=at(5)), INVALID),
    (dict(lse=at(5, 2 * 8 * 128 * 2 - 4)), INVALID),
], ids=str)
def test_decode_refuses(lib, kw, rc):
    assert decode(lib, **kw) == rc


def test_page_bytes(lib):
    assert sk.sskip_kv_page_bytes(sk.SSKIP_KV_BF16, 8, 64, 128) == 8 * 64 * 256
    assert sk.sskip_kv_page_bytes(sk.SSKIP_KV_INT4, 8, 64, 128) == 8 * 4 * 1280
    assert sk.sskip_kv_page_bytes(sk.SSKIP_KV_INT4, 3, 16, 64) == 3 * 640
    assert sk.sskip_kv_page_bytes(2, 8, 64, 128) == 0
    assert sk.sskip_kv_page_bytes(0, 8, 24, 128) == 0


SCALINGS = [("plain", {}), ("linear", dict(factor=4.0)),
            ("bands", dict(factor=8.0, slow_turns=1.0, fast_turns=4.0, original_len=8192.0)),
            ("yarn", dict(factor=8.0, slow_turns=1.0, fast_turns=32.0, original_len=4096.0))]


@pytest.mark.parametrize("scaling,kw", SCALINGS, ids=lambda s: s if isinstance(s, str) else "")
@pytest.mark.parametrize("rot,base", [(128, 500000.0), (64, 10000.0), (48, 1e6), (16, 10000.0)])
def test_frequency_table(lib, scaling, kw, rot, base):
    turns, attn = sk.sskip_rope_freqs(rot, base, scaling=scaling, **kw)
    want = ref.frequencies(rot, base, scaling, kw.get("factor", 1.0), kw.get("slow_turns", 1.0),
                           kw.get("fast_turns", 4.0), kw.get("original_len", 0.0))
    got = turns.astype(np.float64) / 2.0 ** 64 * (2 * math.pi)
    # a handful of 64-bit roundings on either side (pow is good to 1 ulp), and
    # the table's own step: rounding to a whole 2^-64 turn moves a frequency by
    # at most half of it, 2 pi 2^-65 radians, whatever its size
    want = np.array(want)
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -53 * want + 2 * math.pi * 2.0 ** -65)
    assert attn == (0.1 * math.log(8.0) + 1.0 if scaling == "yarn" else 1.0)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="bands", factor=8.0),
    dict(scaling="yarn", factor=2.0, original_len=4096.0, slow_turns=4.0, fast_turns=4.0),
    dict(scaling="yarn", factor=float("inf"), original_len=4096.0),
], ids=str)
def test_frequency_table_refuses(lib, kw):
    a = dict(rot_dim=64, base=10000.0)
    a.update(kw)
    with pytest.raises(sk.SSkipError) as e:
        sk.sskip_rope_freqs(a.pop("rot_dim"), a.pop("base"), **a)
    assert e.value.status == INVALID


def test_frequency_table_refuses_an_unknown_scaling(lib):
    with pytest.raises(ValueError):
        sk.sskip_rope_freqs(64, 10000.0, scaling="cubic")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [False, True])
def test_reference_records_are_a_bijection(d, value):
    byte, hi = ref.code_places(d, value)
    places = (byte * 2 + hi).ravel()
    assert sorted(places) == list(range(16 * d))  # every nibble of the codes, once
    r = np.random.default_rng(d)
    codes = r.integers(0, 16, (3, 16, d))
    sc, mn = (ref.bf16_value(ref.bf16_bits(r.standard_normal((3, 16, d // 32)))) for _ in range(2))
    got = ref.unpack(ref.pack(codes, sc, mn, value), d, value)
    assert all(np.array_equal(a, b) for a, b in zip(got, (codes, sc, mn)))


# ------------------------------------------------------------ the binding
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def append_tensors(**kw):
    qkv = bf(5, 8, 64)
    a = dict(q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:], seq_ids=ints(5), positions=ints(5),
             q_out=bf(5, 4, 64), k_out=bf(5, 2, 64), v_out=bf(5, 2, 64), k_pages=bf(3, 2, 16, 64),
             v_pages=bf(3, 2, 16, 64), block_table=ints(2, 4),
             turns=torch.zeros(32, dtype=torch.int64), q_weight=bf(64), k_weight=bf(64))
    a.update(kw)
    return a


HOST = "expected CUDA tensors"


@pytest.mark.parametrize("kw,err,words", [
    (dict(), ValueError, HOST),  # every other check passed
    (dict(k=None, v=None, k_out=None, v_out=None, k_pages=None, v_pages=None), ValueError, HOST),
    (dict(q=None, q_out=None), ValueError, HOST),
    (dict(q=bf(1, 4, 64).expand(1, 4, 64), k=bf(1, 2, 64), v=bf(1, 2, 64), seq_ids=ints(1),
          positions=ints(1), q_out=bf(1, 4, 64), k_out=None, v_out=None), ValueError, HOST),
    (dict(k_pages=torch.zeros(3, 2, 1, 640, dtype=torch.uint8),
          v_pages=torch.zeros(3, 2, 1, 640, dtype=torch.uint8)), ValueError, HOST),
    (dict(q=torch.zeros(5, 4, 64)), TypeError, "q must be BFloat16"),
    (dict(q=3), (TypeError, AttributeError), ""),
    (dict(positions=torch.zeros(5, dtype=torch.int64)), TypeError, "positions must be Int"),
    (dict(positions=ints(4)), ValueError, "positions needs 5"),
    (dict(seq_ids=ints(10)[::2]), ValueError, "contiguous"),
    (dict(q=bf(5, 8, 64)[:, ::2]), ValueError, "packed"),
    (dict(q=bf(5, 4, 128)[..., ::2]), ValueError, "packed"),
    (dict(q=bf(20, 64)), ValueError, "must be [T, H, d]"),
    (dict(k=bf(4, 2, 64), v=bf(4, 2, 64)), ValueError, "one T and d"),
    (dict(v=bf(5, 1, 64)), ValueError, "one shape"),
    (dict(v=None), ValueError, "come together"),
    (dict(q_out=bf(5, 3, 64)), ValueError, "q_out must be"),
    (dict(q_out=bf(5, 4, 128)[..., ::2]), ValueError, "q_out must be contiguous"),
    (dict(q_out=torch.zeros(5, 4, 64)), TypeError, "q_out"),
    (dict(q_out=bf(1, 4, 5, 64)), ValueError, "one layout"),
    (dict(q_weight=bf(32)), ValueError, "q_weight must hold 64"),
    (dict(k_weight=torch.zeros(64)), TypeError, "k_weight"),
    (dict(turns=torch.zeros(32)), TypeError, "turns"),
    (dict(block_table=None), ValueError, "block_table"),
    (dict(v_pages=None), ValueError, "block_table"),
    (dict(block_table=ints(2, 4).long()), TypeError, "block_table"),
    (dict(block_table=ints(8)), ValueError, "2-D"),
    (dict(k_pages=bf(3, 3, 16, 64), v_pages=bf(3, 3, 16, 64)), ValueError, "the pages hold 3 heads"),
    (dict(k_pages=bf(3, 2, 16, 128), v_pages=bf(3, 2, 16, 128)), ValueError, "rows of 128"),
    (dict(k_pages=torch.zeros(3, 2, 1, 1280, dtype=torch.uint8),
          v_pages=torch.zeros(3, 2, 1, 1280, dtype=torch.uint8)), ValueError, "hold 640 bytes"),
    (dict(v_pages=bf(3, 2, 32, 64)), ValueError, "one shape and dtype"),
    (dict(k_pages=torch.zeros(3, 2, 16, 64), v_pages=torch.zeros(3, 2, 16, 64)), TypeError, "pages"),
    (dict(k_pages=bf(3, 16, 2, 64).transpose(1, 2), v_pages=bf(3, 16, 2, 64).transpose(1, 2)),
     ValueError, "contiguous"),
    (dict(eps="small"), TypeError, ""),
], ids=lambda x: x if isinstance(x, str) else "")
def test_append_binding_refuses(lib, kw, err, words):
    with pytest.raises(err) as e:
        sk.sskip_kv_append(**append_tensors(**kw))
    assert words in str(e.value)


@pytest.mark.parametrize("kw,err,words", [
    (dict(), ValueError, HOST),
    (dict(k_out=bf(1, 2, 5, 64), v_out=bf(1, 2, 5, 64)), ValueError, HOST),
    (dict(k_out=bf(1, 2, 5, 64)), ValueError, "one layout"),
    (dict(v_out=bf(5, 2, 128)), ValueError, "v_out must be"),
    (dict(seq_ids=None), (ValueError, AttributeError), ""),
    (dict(positions=ints(6)), ValueError, "positions needs 5"),
    (dict(k_pages=bf(3, 2, 16)), ValueError, "4-D"),
], ids=lambda x: x if isinstance(x, str) else "")
def test_gather_binding_refuses(lib, kw, err, words):
    a = dict(k_pages=bf(3, 2, 16, 64), v_pages=bf(3, 2, 16, 64), block_table=ints(2, 4),
             seq_ids=ints(5), positions=ints(5), k_out=bf(5, 2, 64), v_out=bf(5, 2, 64))
    a.update(kw)
    with pytest.raises(err) as e:
        sk.sskip_kv_gather(**a)
    assert words in str(e.value)


@pytest.mark.parametrize("kw,err,words", [
    (dict(), ValueError, HOST),
    (dict(q=bf(2, 8, 128)[..., ::2]), ValueError, "contiguous"),
    (dict(q=bf(16, 64)), ValueError, "q must be"),
    (dict(o=bf(2, 4, 64)), ValueError, "one batch"),
    (dict(lse=torch.zeros(2, 4)), ValueError, "one batch"),
    (dict(lse=torch.zeros(2, 8, dtype=torch.float64)), TypeError, "lse must be Float"),
    (dict(block_table=ints(3, 4)), ValueError, "one batch"),
    (dict(seqlens=torch.zeros(2, dtype=torch.int64)), TypeError, "seqlens must be Int"),
    (dict(skip_count=torch.zeros(1, dtype=torch.int64)), ValueError, "2 entries"),
    (dict(skip_count=ints(2)), TypeError, "skip_count"),
    (dict(tile_state=torch.zeros(5, dtype=torch.uint8)), ValueError, "tile_state must be"),
    (dict(workspace=torch.zeros(64, dtype=torch.uint8)[::2]), ValueError, "workspace"),
    (dict(num_splits=1.5), TypeError, ""),
], ids=lambda x: x if isinstance(x, str) else "")
def test_decode_binding_refuses(lib, kw, err, words):
    a = dict(q=bf(2, 8, 64), k_pages=bf(3, 2, 16, 64), v_pages=bf(3, 2, 16, 64),
             block_table=ints(2, 4), seqlens=ints(2), o=bf(2, 8, 64), lse=torch.zeros(2, 8),
             sm_scale=0.1, threshold_scale_factor=0.0, num_splits=1, tile_state=None)
    a.update(kw)
    with pytest.raises(err) as e:
        sk.sskip_attn_decode_paged(**a)
    assert words in str(e.value)

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


def test_the_binding_packs_the_structs_of_the_header():
    for kind, packed in ((AppendArgs, sk._APPEND_ARGS), (GatherArgs, sk._GATHER_ARGS),
                         (DecodeArgs, sk._DECODE_ARGS)):
        assert ctypes.sizeof(kind) == packed.size, kind
        # every field at its place: fields filled with 1, 2, 3, ... both ways
        names = [n for n, _ in Cache._fields_] + [n for n, _ in kind._fields_ if n != "cache"]
        assert fill(kind, {n: i + 1 for i, n in enumerate(names)}) == \
            packed.pack(*range(1, len(names) + 1))


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


def test_tensor_checks_of_the_binding():
    z = torch.zeros
    bf = torch.bfloat16
    pages, table = z(4, 2, 16, 64, dtype=bf), z(1, 4, dtype=torch.int32)
    got, heads = sk._pages(pages, pages.clone(), table, 64)
    assert (got[3:], heads) == ((0, 4, 16, 4, 1), 2)
    rec = z(4, 2, 1, 640, dtype=torch.uint8)
    got, heads = sk._pages(rec, rec.clone(), table, 64)
    assert (got[3:], heads) == ((1, 4, 16, 4, 1), 2)
    for a, b, t, d, err in [(pages, pages[:, :1], table, 64, ValueError),
                            (pages, pages.float(), table, 64, ValueError),
                            (pages.float(), pages.float(), table, 64, TypeError), (pages, None, table, 64, ValueError),
                            (pages, pages, table.long(), 64, TypeError),
                            (pages, pages, table, 128, ValueError), (rec, rec, table, 128, ValueError),
                            (pages.transpose(1, 2), pages.transpose(1, 2), table, 64, ValueError)]:
        with pytest.raises(err):
            sk._pages(a, b, t, d)
    qkv = z(5, 6 * 64, dtype=bf).unflatten(1, (6, 64))
    assert sk._token_rows(qkv[:, :4], "q") == 6 * 64
    assert sk._token_rows(qkv[:1, :4], "q") == 4 * 64
    for t, err in [(qkv.float(), TypeError), (qkv[:, ::2], ValueError), (qkv[..., ::2], ValueError)]:
        with pytest.raises(err):
            sk._token_rows(t, "q")
    assert sk._rows_out(z(5, 4, 64, dtype=bf), 5, 4, 64, "o") == 1
    assert sk._rows_out(z(2, 4, 3, 64, dtype=bf), 6, 4, 64, "o") == 3
    for t, err in [(z(5, 4, 64), TypeError), (z(4, 4, 64, dtype=bf), ValueError),
                   (z(5, 2, 128, dtype=bf), ValueError), (z(5, 4, 128, dtype=bf)[..., ::2], TypeError)]:
        with pytest.raises(err):
            sk._rows_out(t, 5, 4, 64, "o")
    with pytest.raises(ValueError):  # host tensors
        sk.sskip_kv_append(qkv[:, :4], None, None, None, z(5, dtype=torch.int32),
                           q_out=z(5, 4, 64, dtype=bf))
    with pytest.raises(TypeError):
        sk._tokens(z(5, dtype=torch.int64), 5, "positions")
    with pytest.raises(ValueError):
        sk._tokens(z(4, dtype=torch.int32), 5, "positions")
    with pytest.raises(ValueError):
        sk._one_device(None, qkv)

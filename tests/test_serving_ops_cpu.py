"""The norm-rope-cache write, the 8-bit cache and attention of drafted tokens
on the CPU: pins of their plain fp64 forms, the host helpers, and the argument
checks, which return before any CUDA call."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from oracle import serving_ops as plain

BAD, UNS, WS = pk.PK_ERR_INVALID_ARG, pk.PK_ERR_UNSUPPORTED, pk.PK_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    pk.build()
    return pk.lib()


# -- pins of the plain forms -------------------------------------------------
def test_e4m3_codes_by_hand():
    v = plain.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0
    assert v[0xB8] == -1.0 and np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    codes, exps = plain.quantize_rows([[448.0, 1.0, 0.0, -2.0]])
    assert exps.tolist() == [127] and codes.tolist() == [[0x7E, 0x38, 0, 0xC0]]
    codes, exps = plain.quantize_rows([[449.0, 1.0, 0.0, -2.0]])      # past 448: the next power of two
    assert exps.tolist() == [128] and codes[0, 1] == 0x30             # 0.5 * 2
    assert plain.quantize_rows([[0.0, 0.0]])[1].tolist() == [127]     # a row of zeros
    codes, _ = plain.quantize_rows([[448.0, 17.0, 19.0, 2.0 ** -10]])  # ties go to the even code
    assert plain.e4m3_values()[codes[0]].tolist() == [448.0, 16.0, 20.0, 0.0]
    codes, exps = plain.quantize_rows([[np.inf, np.nan, 448.0]])
    assert exps[0] == 127 and codes[0].tolist() == [0x7F, 0x7F, 0x7E]


def test_e4m3_round_trip_is_exact():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 32)).astype(np.float32) * np.float32(2.0) ** rng.integers(-60, 60, (64, 1))
    codes, exps = plain.quantize_rows(x)
    y = plain.decode_values(codes, exps)
    assert (np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** (exps - 127.0)[:, None])).all()
    again = plain.quantize_rows(y)
    # Values keep their codes; the exponent can only drop where the largest code rounded down.
    assert np.array_equal(plain.decode_values(*again), y)


def test_norm_rope_by_hand():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    cs = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0]])       # position 1: a quarter turn
    w = np.ones(4)
    y = plain.norm_rope(x, w, 0.0, cs, [0], False)
    assert np.allclose(y, x / 2.5)
    y = plain.norm_rope(x, None, 0.0, cs, [1], False)                 # (0, 2), (1, 3): (a, b) -> (-b, a)
    assert y.tolist() == [[[0.0, 0.0, 3.0, 4.0]]]
    y = plain.norm_rope(x, None, 0.0, cs, [1], True)                  # (0, 1), (2, 3)
    assert y.tolist() == [[[-4.0, 3.0, 0.0, 0.0]]]


def test_tree_attention_by_hand():
    k = np.zeros((2, 2, 1, 2))
    v = np.arange(8.0).reshape(2, 2, 1, 2)
    q = np.ones((2, 1, 2))
    out, _ = plain.tree_attention(q, k, v, [[1, 0]], [3], 1.0, [0, 2], [1, 2])
    # base 1: row 0 sees tokens 0, 1 (block 1), row 1 sees tokens 0 and 2
    assert out[0, 0].tolist() == [5.0, 6.0] and out[1, 0].tolist() == [2.0, 3.0]
    out, _ = plain.tree_attention(q, k, v, [[1, 0]], [2], 1.0, [0, 2], [0, 3])
    assert out[0, 0].tolist() == [0.0, 0.0] and out[1, 0].tolist() == [5.0, 6.0]
    out, _ = plain.tree_attention(q, k, v, [[1, 0]], [3], 1.0, [0, 2], None)
    assert out[0, 0].tolist() == [5.0, 6.0] and np.allclose(out[1, 0], [10 / 3, 13 / 3])


# -- host helpers ------------------------------------------------------------
def test_tree_masks(L):
    masks, depths = pk.pk_tree_masks([-1, 0, 0, 1, 2, -1])
    assert masks.tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100000]
    assert depths.tolist() == [0, 1, 1, 2, 2, 0]
    masks, depths = pk.pk_tree_masks(list(range(-1, 63)))              # a chain of 64
    assert masks[63] == -1 and depths[63] == 63 and masks[62] == 2 ** 63 - 1
    assert len(pk.pk_tree_masks([])[0]) == 0
    for parents in ([0], [-1, 1], [-2], [-1] * 65):
        with pytest.raises(pk.PagedKVError):
            pk.pk_tree_masks(parents)


def test_tree_plan_and_workspace(L):
    d = pk.CacheDesc(20000, 16, 8, 128, pk.PK_BF16)
    part, items = pk.pk_tree_plan([32768] * 8, 16, 64, d)
    assert part > 0 and part % 64 == 0 and len(items) == 8 * -(-32768 // part)
    assert sorted(map(tuple, items.tolist())) == [(s, j) for s in range(8) for j in range(-(-32768 // part))]
    part, items = pk.pk_tree_plan([100, 0, 7], 4, 8, d)                # short: whole, one item each
    assert part == 0 and sorted(items[:, 0].tolist()) == [0, 1, 2]
    assert pk.pk_tree_plan([1000, 40], 4, 8, d, 64)[0] == 64
    assert pk.pk_tree_workspace_size(10, 8, 1000, 64, d) == 10 * 8 * 16 * 130 * 4
    assert pk.pk_tree_workspace_size(10, 8, 64, 64, d) == 0
    assert pk.pk_tree_workspace_size(10, 8, 1000, 0, d) == 0
    for bad in (dict(max_draft_len=0), dict(max_draft_len=65), dict(num_q_heads=12), dict(partition_size=24),
                dict(partition_size=-2), dict(desc=pk.CacheDesc(64, 16, 8, 96, 1)),
                dict(desc=pk.CacheDesc(64, 16, 8, 128, pk.PK_E4M3))):
        with pytest.raises(pk.PagedKVError):
            pk.pk_tree_plan(**{**dict(context_lens=[100], max_draft_len=4, num_q_heads=8, desc=d), **bad})


def test_attention_planner_takes_8_bit_caches(L):
    d = pk.CacheDesc(20000, 16, 8, 128, pk.PK_E4M3)
    part, items = pk.pk_attention_plan([32768] * 8, 64, d, -1)
    assert part > 0 and len(items) == 8 * -(-32768 // part)
    assert pk.pk_paged_attention_workspace_size(8, 64, 32768, 512, d) == 8 * 64 * 64 * 130 * 4
    assert pk.pk_paged_attention_resolve_partition(0, 64, 32768, -1, d) == 0      # an empty batch


def test_other_calls_refuse_8_bit_caches(L):
    d = pk.CacheDesc(64, 16, 8, 128, pk.PK_E4M3)
    buf = np.zeros(1 << 16, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    assert L.pk_reshape_and_cache(p, p, p, 1, p, p, ctypes.byref(d), None) == UNS
    assert L.pk_copy_blocks(p, p, p, 1, ctypes.byref(d), None) == UNS
    assert L.pk_paged_attention_decode_impl(p, p, p, p, p, p, 0.1, 4, 8, 4, 64, 0, None, 0, ctypes.byref(d), None,
                                            0, None) == UNS
    assert L.pk_paged_attention_decode_static(p, p, p, p, p, p, 0.1, 16, 4, 8, 4, 64, 0, ctypes.byref(d),
                                              None) == UNS


# -- argument checks (host buffers stand in; no case reaches a CUDA call) ----
@pytest.fixture(scope="module")
def ptr():
    buf = np.zeros(1 << 16, np.uint8)
    base = (buf.ctypes.data + 255) // 256 * 256
    yield lambda i: base + 2048 * i
    del buf


def test_norm_rope_refusals(L, ptr):
    def call(desc=(64, 16, 2, 128, pk.PK_BF16), **kw):
        a = dict(qo=ptr(0), ko=ptr(1), q=ptr(2), k=ptr(3), v=ptr(4), qs=512, ks=256, vs=256, qw=ptr(5), kw=ptr(6),
                 eps=1e-6, cs=ptr(7), pos=ptr(8), maxp=16, rot=128, inter=0, slots=ptr(9), T=2, hq=4, kc=ptr(10),
                 vc=ptr(11))
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_qk_norm_rope_and_cache(a["qo"], a["ko"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"],
                                           a["qw"], a["kw"], a["eps"], a["cs"], a["pos"], a["maxp"], a["rot"],
                                           a["inter"], a["slots"], a["T"], a["hq"], a["kc"], a["vc"],
                                           ctypes.byref(d), None)

    assert call(T=0) == pk.PK_OK
    for bad in (dict(T=-1), dict(qo=None), dict(q=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None),
                dict(qw=None), dict(kw=None), dict(cs=None), dict(pos=None), dict(maxp=0), dict(hq=0),
                dict(rot=8), dict(rot=-16), dict(rot=144), dict(qs=511), dict(qs=516), dict(ks=128), dict(vs=252),
                dict(eps=-1.0), dict(eps=float("nan")), dict(slots=None, ko=None), dict(q=ptr(2) + 8),
                dict(cs=ptr(7) + 4), dict(kc=ptr(10) + 2), dict(qo=ptr(2), qs=1024), dict(ko=ptr(3), ks=512),
                dict(desc=(0, 16, 2, 128, 1)), dict(desc=(64, 16, 0, 128, 1))):
        assert call(**bad) == BAD, bad
    for uns in (dict(desc=(64, 16, 2, 128, pk.PK_E4M3)), dict(desc=(64, 16, 2, 120, 1)),
                dict(desc=(64, 16, 2, 272, 1))):
        assert call(**uns) == UNS, uns


def test_e4m3_cache_refusals(L, ptr):
    def write(desc=(64, 16, 2, 128, pk.PK_E4M3), **kw):
        a = dict(k=ptr(0), v=ptr(1), dt=pk.PK_BF16, ks=256, vs=256, slots=ptr(2), T=2, kc=ptr(3), vc=ptr(4), ex=ptr(5))
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_reshape_and_cache_e4m3(a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["slots"], a["T"], a["kc"],
                                           a["vc"], a["ex"], ctypes.byref(d), None)

    def read(desc=(64, 16, 2, 128, pk.PK_E4M3), **kw):
        a = dict(k=ptr(0), v=ptr(1), dt=pk.PK_BF16, slots=ptr(2), T=2, kc=ptr(3), vc=ptr(4), ex=ptr(5))
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_gather_cache_e4m3(a["k"], a["v"], a["dt"], a["slots"], a["T"], a["kc"], a["vc"], a["ex"],
                                      ctypes.byref(d), None)

    def copy(desc=(64, 16, 2, 128, pk.PK_E4M3), **kw):
        a = dict(kc=ptr(3), vc=ptr(4), ex=ptr(5), pairs=ptr(2), n=1)
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_copy_blocks_e4m3(a["kc"], a["vc"], a["ex"], a["pairs"], a["n"], ctypes.byref(d), None)

    for call in (write, read):
        assert call(T=0) == pk.PK_OK
        for bad in (dict(T=-1), dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
                    dict(ex=None), dict(k=ptr(0) + 8), dict(kc=ptr(3) + 8), dict(ex=ptr(5) + 2),
                    dict(desc=(64, 0, 2, 128, 2))):
            assert call(**bad) == BAD, (call, bad)
        for uns in (dict(desc=(64, 16, 2, 128, pk.PK_BF16)), dict(desc=(64, 16, 2, 72, 2)),
                    dict(desc=(64, 16, 2, 512, 2)), dict(dt=pk.PK_E4M3)):
            assert call(**uns) == UNS, (call, uns)
    assert write(ks=255) == BAD and write(vs=260) == BAD
    assert copy(n=0) == pk.PK_OK
    for bad in (dict(n=-1), dict(kc=None), dict(ex=None), dict(pairs=None), dict(vc=ptr(4) + 4)):
        assert copy(**bad) == BAD
    assert copy(desc=(64, 16, 2, 128, 1)) == UNS


def test_e4m3_attention_refusals(L, ptr):
    def call(desc=(64, 16, 8, 128, pk.PK_E4M3), **kw):
        a = dict(out=ptr(0), q=ptr(1), dt=pk.PK_BF16, kc=ptr(2), vc=ptr(3), ex=ptr(4), tb=ptr(5), ln=ptr(6), sc=0.1,
                 S=4, hq=32, maxb=8, mc=100, part=0, items=ptr(7), n=4, ws=ptr(8), wsb=1024)
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_paged_attention_decode_e4m3(a["out"], a["q"], a["dt"], a["kc"], a["vc"], a["ex"], a["tb"],
                                                a["ln"], a["sc"], a["S"], a["hq"], a["maxb"], a["mc"], a["part"],
                                                a["items"], a["n"], a["ws"], a["wsb"], ctypes.byref(d), None)

    assert call(S=0) == pk.PK_OK and call(S=0, part=-1, mc=4096) == pk.PK_OK
    for bad in (dict(S=-1), dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(ex=None), dict(tb=None),
                dict(ln=None), dict(maxb=0), dict(mc=0), dict(hq=12), dict(part=40), dict(part=-2),
                dict(sc=float("nan")), dict(q=ptr(1) + 4), dict(ex=ptr(4) + 8)):
        assert call(**bad) == BAD, bad
    for uns in (dict(desc=(64, 16, 8, 128, pk.PK_BF16)), dict(dt=pk.PK_E4M3), dict(desc=(64, 64, 8, 128, 2)),
                dict(n=0), dict(n=70000), dict(items=None), dict(S=70000, items=None, n=0)):
        assert call(**uns) == UNS, uns
    assert call(part=16, ws=None) == WS and call(part=16, wsb=16) == WS and call(ws=ptr(8) + 4) == WS
    # Shapes the planner refuses come back as an invalid argument, as in the bf16 call's partition check.
    assert call(desc=(64, 16, 8, 96, 2)) in (BAD, UNS) and call(hq=128) in (BAD, UNS)


def test_tree_attention_refusals(L, ptr):
    def call(desc=(64, 16, 8, 128, pk.PK_BF16), **kw):
        a = dict(out=ptr(0), q=ptr(1), kc=ptr(2), vc=ptr(3), tb=ptr(4), ln=ptr(5), of=ptr(6), mk=ptr(7), sc=0.1, S=4,
                 R=8, md=4, hq=32, maxb=8, mc=100, part=0, items=ptr(8), n=4, ws=ptr(9), wsb=1024)
        a.update(kw)
        d = pk.CacheDesc(*desc)
        return L.pk_paged_attention_tree(a["out"], a["q"], a["kc"], a["vc"], a["tb"], a["ln"], a["of"], a["mk"],
                                         a["sc"], a["S"], a["R"], a["md"], a["hq"], a["maxb"], a["mc"], a["part"],
                                         a["items"], a["n"], a["ws"], a["wsb"], ctypes.byref(d), None)

    for none in (dict(S=0), dict(R=0), dict(md=0)):
        assert call(**none) == pk.PK_OK
    for bad in (dict(S=-1), dict(R=-1), dict(md=-1), dict(out=None), dict(q=None), dict(kc=None), dict(vc=None),
                dict(tb=None), dict(ln=None), dict(of=None), dict(mk=ptr(7) + 4), dict(maxb=0), dict(mc=0),
                dict(hq=12), dict(hq=0), dict(part=40), dict(part=-1), dict(sc=float("nan")), dict(q=ptr(1) + 4),
                dict(kc=ptr(2) + 2)):
        assert call(**bad) == BAD, bad
    for uns in (dict(md=65), dict(desc=(64, 16, 8, 128, pk.PK_E4M3)), dict(desc=(64, 16, 8, 96, 1)), dict(hq=128),
                dict(n=0), dict(n=70000), dict(items=None), dict(S=70000, items=None, n=0)):
        assert call(**uns) == UNS, uns
    assert call(part=16, ws=None) == WS and call(part=16, wsb=16) == WS and call(ws=ptr(9) + 4) == WS


def test_binding_refuses_cpu_tensors(L):
    torch = pytest.importorskip("torch")
    z = torch.zeros
    kc = z((4, 16, 2, 64), dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        pk.pk_reshape_and_cache_e4m3(z(1, 2, 64), z(1, 2, 64), z(1, dtype=torch.int64), kc, kc,
                                     z((4, 2, 16, 2), dtype=torch.uint8))
    with pytest.raises(ValueError):
        pk.pk_qk_norm_rope_and_cache(z(1, 4, 64), z(1, 2, 64), z(1, 4, 64), z(1, 2, 64), None, None, None)
    with pytest.raises(TypeError):
        pk.pk_gather_cache_e4m3(z(1, 2, 64), z(1, 2, 64), z(1, dtype=torch.int64), kc.float(), kc.float(),
                                z((4, 2, 16, 2), dtype=torch.uint8))
    with pytest.raises(ValueError):
        pk.pk_qk_norm_rope_and_cache(z(1, 4, 64), z(1, 2, 64), z(1, 4, 64), z(1, 2, 64), None, None, None,
                                     slot_mapping=z(1, dtype=torch.int64))

"""The norm-rope-cache write, the 8-bit cache and attention of drafted tokens
on the GPU, element by element against their plain fp64 forms.

Tolerances are bounds, derived from the arithmetic (u = 2^-24, one fp32
rounding; eta = half a step of the output type, 2^-8 for bf16, u for fp32):

* norm and rotation: the sum of d squares as a tree over lanes costs at most 16
  roundings, the square root halves them, and the root, the quotient, two
  products, the rotation's two products and sum add 8: 16 u (|a| + |b|) over a
  pair (a, b), plus eta of the result.
* 8-bit rows: exact (one rounding to e4m3 of an exact product).
* attention: a score's d products and sums are off by at most
  D = (d + 8) v |scale| log2(e) sum_i |q_i k_i|, v one rounding of the sums (u on
  CUDA cores; 2 u on tensor cores, which may truncate); a weight by the factor
  1 + 2 ln2 D + 8 u + rho, rho the rounding of the weights where a product takes
  them in fewer bits (2^-11 in fp16, 2^-17 as a bf16 pair; u otherwise); a sum
  over n tokens adds n v. The output is a ratio of two such sums:
  |error| <= (4 ln2 D + 16 u + 2 rho + 2 n v) sum_t w_t |v_t| + eta |out|.
"""
import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from oracle import serving_ops as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ETA = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pk.build()


@pytest.fixture(autouse=True)
def _no_device_error():
    pk.pk_get_device_error()
    yield
    assert pk.pk_get_device_error() == (0, 0)


def f64(t):
    return t.detach().double().cpu().numpy()


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def values_of(kc, vc, ex):
    """The fp64 values of an 8-bit pool's keys and values."""
    e = np.moveaxis(ex.cpu().numpy(), 1, 2)
    return [plain.decode_values(codes_of(c), e[..., i]) for i, c in enumerate((kc, vc))]


def rand(rng, shape, dtype=torch.float32):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).to(dtype)


def i64(x):
    return torch.from_numpy(np.asarray(x, np.int64)).to(DEV)


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


# ---------------------------------------------------------------------------
# Norm, rotation, cache write
# ---------------------------------------------------------------------------
def rope_table(max_pos, rot):
    ang = np.arange(max_pos)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def check_rope(got, x, w, eps, cs, pos, inter, dtype):
    want = plain.norm_rope(f64(x), None if w is None else f64(w), eps, cs, pos, inter)
    y = np.abs(plain.norm_rope(f64(x), None if w is None else f64(w), eps, None, pos, inter))
    pair = y.copy()
    rot = 0 if cs is None else cs.shape[1]
    for j in range(rot // 2):
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + rot // 2)
        pair[..., a] = pair[..., b] = y[..., a] + y[..., b]
    tol = 16 * U * pair + ETA[dtype] * np.abs(want)
    assert (np.abs(f64(got) - want) <= tol).all(), float((np.abs(f64(got) - want) - tol).max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,rot,inter,norm,T", [
    (4, 2, 128, 128, False, True, 33), (8, 8, 64, 32, True, True, 5), (3, 1, 80, 80, False, True, 1),
    (5, 5, 96, 64, False, False, 7), (2, 1, 256, 256, True, True, 3), (2, 2, 256, 16, False, True, 2),
    (7, 1, 16, 16, False, True, 9), (1, 1, 64, 0, False, True, 4), (32, 8, 128, 128, False, True, 64),
])
def test_norm_rope_and_cache(dtype, hq, hk, d, rot, inter, norm, T):
    dt, B, N = DTYPES[dtype], 16, 11
    rng = np.random.default_rng(hq * 1000 + d + T)
    qkv = rand(rng, (T, hq + 2 * hk, d), dt) * 3
    q, k, v = qkv.split([hq, hk, hk], dim=1)
    w = [(1 + 0.2 * rand(rng, (d,))).to(dt) if norm else None for _ in range(2)]
    cs = rope_table(300, rot) if rot else None
    pos = rng.integers(0, 300, T)
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    if T > 2:
        slots[1] = -1
    kc, vc = torch.full((N, B, hk, d), 7.0, dtype=dt, device=DEV), torch.full((N, B, hk, d), -7.0, dtype=dt, device=DEV)
    qo, ko = torch.empty((T, hq, d), dtype=dt, device=DEV), torch.empty((T, hk, d), dtype=dt, device=DEV)
    pk.pk_qk_norm_rope_and_cache(qo, ko, q, k, v, None if cs is None else torch.from_numpy(cs).to(DEV), i64(pos),
                                 q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=inter, slot_mapping=i64(slots),
                                 k_cache=kc, v_cache=vc)
    check_rope(qo, q, w[0], np.float32(1e-5), cs, pos, inter, dt)
    check_rope(ko, k, w[1], np.float32(1e-5), cs, pos, inter, dt)
    wk, wv = torch.full_like(kc, 7.0).view(-1, hk, d), torch.full_like(vc, -7.0).view(-1, hk, d)
    live = slots >= 0
    wk[slots[live]], wv[slots[live]] = ko[live], v[live]
    assert torch.equal(kc.view(-1, hk, d), wk) and torch.equal(vc.view(-1, hk, d), wv)


def test_norm_rope_without_cache_in_place_and_empty():
    rng = np.random.default_rng(5)
    q, k = rand(rng, (6, 4, 64)), rand(rng, (6, 2, 64))
    w, cs, pos = rand(rng, (64,)), rope_table(50, 64), rng.integers(0, 50, 6)
    q0, k0 = q.clone(), k.clone()
    pk.pk_qk_norm_rope_and_cache(q, k, q, k, None, torch.from_numpy(cs).to(DEV), i64(pos), q_weight=w, k_weight=w)
    check_rope(q, q0, w, np.float32(1e-6), cs, pos, False, torch.float32)
    check_rope(k, k0, w, np.float32(1e-6), cs, pos, False, torch.float32)
    e = q[:0]
    pk.pk_qk_norm_rope_and_cache(e, k[:0], e, k[:0], None, torch.from_numpy(cs).to(DEV), i64([]), q_weight=w,
                                 k_weight=w)


def test_norm_rope_bad_positions_and_slots_are_skipped():
    rng = np.random.default_rng(6)
    T, hq, hk, d, N, B = 5, 2, 1, 64, 2, 8
    q, k, v = rand(rng, (T, hq, d)), rand(rng, (T, hk, d)), rand(rng, (T, hk, d))
    cs = torch.from_numpy(rope_table(10, 64)).to(DEV)
    for pos, slots, kind, at in (([0, 10, 3, 2, 1], [0, 1, 2, 3, 4], 7, 1), ([0, -1, 3, 2, 1], [0, 1, 2, 3, 4], 7, 1),
                                 ([0, 1, 3, 2, 1], [0, 1, 16, 3, 4], 1, 2)):
        kc, vc = torch.zeros((N, B, hk, d), device=DEV), torch.zeros((N, B, hk, d), device=DEV)
        qo, ko = torch.full((T, hq, d), 9.0, device=DEV), torch.full((T, hk, d), 9.0, device=DEV)
        pk.pk_qk_norm_rope_and_cache(qo, ko, q, k, v, cs, i64(pos), slot_mapping=i64(slots), k_cache=kc, v_cache=vc)
        assert pk.pk_get_device_error() == (kind, at)
        skipped = 1 if kind == 7 else -1
        for t in range(T):
            assert (qo[t] == 9.0).all().item() == (t == skipped) and (ko[t] == 9.0).all().item() == (t == skipped)
            written = t != skipped and slots[t] < N * B
            if slots[t] < N * B:
                assert torch.equal(vc.view(-1, hk, d)[slots[t]], v[t] if written else torch.zeros_like(v[t]))


# ---------------------------------------------------------------------------
# 8-bit cache
# ---------------------------------------------------------------------------
def e4m3_pool(N, B, Hk, d, code=0x7F, exp=127):
    kc = torch.full((N, B, Hk, d), code, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ex = torch.full((N, Hk, B, 2), exp, dtype=torch.uint8, device=DEV)
    return kc, kc.clone(), ex


def special_rows(rng, T, Hk, d):
    x = rng.standard_normal((T, Hk, d)).astype(np.float32)
    x *= np.float32(2.0) ** rng.integers(-30, 30, (T, Hk, 1)).astype(np.float32)
    flat = x.reshape(-1, d)
    rows = [np.zeros(d), np.full(d, -0.0), np.r_[448.0, np.linspace(-448, 448, d - 1)],
            np.r_[np.nextafter(np.float32(448), np.float32(1e9)), np.full(d - 1, 17.0)],
            np.r_[np.inf, np.ones(d - 1)], np.r_[np.nan, -np.inf, np.ones(d - 2)], np.full(d, np.nan),
            np.full(d, 1e-38), np.full(d, 2.0 ** -149), np.r_[3.0e38, np.full(d - 1, 1e30)],
            np.r_[448.0, 17.0, 19.0, np.full(d - 3, 2.0 ** -10)], np.r_[2.0 ** -100 * 448, np.full(d - 1, 2.0 ** -109)]]
    for i, r in enumerate(rows[: len(flat)]):
        flat[i] = r.astype(np.float32)
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hk,d,B", [(1, 1, 64, 16), (7, 2, 128, 8), (13, 3, 16, 5), (6, 2, 256, 32), (33, 1, 80, 16)])
def test_e4m3_write_and_read_back(dtype, T, Hk, d, B):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(T + d)
    N = 2 * -(-T // B) + 1
    packed = torch.from_numpy(special_rows(rng, T, 2 * Hk, d)).to(DEV).to(dt)   # k and v as views of one tensor
    k, v = packed[:, :Hk], packed[:, Hk:]
    slots = rng.permutation(N * B)[:T].astype(np.int64)
    if T > 3:
        slots[3] = -1
    kc, vc, ex = e4m3_pool(N, B, Hk, d, 0x11, 3)
    pk.pk_reshape_and_cache_e4m3(k, v, i64(slots), kc, vc, ex)
    wc = [np.full((N * B, Hk, d), 0x11, np.uint8) for _ in range(2)]
    we = np.full((N, Hk, B, 2), 3, np.uint8)
    for t, s in enumerate(slots):
        if s < 0:
            continue
        for side, x in enumerate((k, v)):
            c, e = plain.quantize_rows(f64(x[t]))
            wc[side][s] = c
            we[s // B, :, s % B, side] = e
    got = [codes_of(c).reshape(N * B, Hk, d) for c in (kc, vc)]
    for side in range(2):  # a zero's sign is kept
        assert np.array_equal(got[side], wc[side])
    assert np.array_equal(ex.cpu().numpy(), we)

    for odt in DTYPES.values():
        ko = torch.full((T, Hk, d), 5.0, dtype=odt, device=DEV)
        vo = torch.full_like(ko, 6.0)
        pk.pk_gather_cache_e4m3(ko, vo, i64(slots), kc, vc, ex)
        for side, (o, fill) in enumerate(((ko, 5.0), (vo, 6.0))):
            for t, s in enumerate(slots):
                want = np.full((Hk, d), fill) if s < 0 else plain.decode_values(wc[side][s], we[s // B, :, s % B, side])
                over = np.abs(want) >= 2.0 ** 128   # rounds past the largest finite number
                want = np.where(over, np.sign(want) * np.inf, want)
                assert np.array_equal(f64(o[t]), want, equal_nan=True)   # exact in either type
    # What was read back and is written again stands for the same values.
    live = np.flatnonzero(slots >= 0)
    ko = torch.empty((T, Hk, d), dtype=torch.float32, device=DEV)
    vo = torch.empty_like(ko)
    pk.pk_gather_cache_e4m3(ko, vo, i64(slots), kc, vc, ex)
    pk.pk_reshape_and_cache_e4m3(ko, vo, i64(slots), kc, vc, ex)
    k2, v2 = torch.empty_like(ko), torch.empty_like(vo)
    pk.pk_gather_cache_e4m3(k2, v2, i64(slots), kc, vc, ex)
    fine = np.isfinite(f64(ko[live]))
    assert np.array_equal(f64(k2[live])[fine], f64(ko[live])[fine])


def test_e4m3_bad_slots_and_block_copies():
    rng = np.random.default_rng(1)
    N, B, Hk, d = 6, 8, 3, 64
    kc, vc, ex = e4m3_pool(N, B, Hk, d)
    k, v = rand(rng, (3, Hk, d)), rand(rng, (3, Hk, d))
    before = kc.view(torch.uint8).clone()
    pk.pk_reshape_and_cache_e4m3(k, v, i64([N * B, -5, N * B + 7]), kc, vc, ex)
    assert pk.pk_get_device_error()[0] == 1 and torch.equal(kc.view(torch.uint8), before)
    ko = torch.full((2, Hk, d), 4.0, device=DEV)
    vo = ko.clone()
    pk.pk_gather_cache_e4m3(ko, vo, i64([N * B, -1]), kc, vc, ex)
    assert pk.pk_get_device_error() == (1, 0) and (ko == 4.0).all() and (vo == 4.0).all()

    for B, Hk, d in ((8, 3, 64), (5, 3, 16), (32, 8, 128)):
        kc, vc, ex = e4m3_pool(N, B, Hk, d)
        for t in (kc.view(torch.uint8), vc.view(torch.uint8), ex):
            t.copy_(torch.from_numpy(rng.integers(0, 256, tuple(t.shape)).astype(np.uint8)))
        want = [t.clone() for t in (kc.view(torch.uint8), vc.view(torch.uint8), ex)]
        for t in want:
            t[4], t[0] = t[1].clone(), t[5].clone()
        pk.pk_copy_blocks_e4m3(kc, vc, ex, i64([[1, 4], [5, 0]]))
        for t, w in zip((kc.view(torch.uint8), vc.view(torch.uint8), ex), want):
            assert torch.equal(t, w)
        pk.pk_copy_blocks_e4m3(kc, vc, ex, i64([[1, N], [-1, 0]]))
        assert pk.pk_get_device_error()[0] == 3
        for t, w in zip((kc.view(torch.uint8), vc.view(torch.uint8), ex), want):
            assert torch.equal(t, w)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def check_attention(got, want, terms, d, dtype, rho, live=None):
    wv, mag, cnt = terms
    D = (d + 8) * 2 * U * mag
    tol = (4 * np.log(2) * D + 16 * U + 2 * rho + 2 * cnt * 2 * U)[..., None] * wv + ETA[dtype] * np.abs(want)
    err = np.abs(got - want)
    if live is not None:
        err, tol = err[live], tol[live]
    assert np.isfinite(err).all(), "non-finite output"
    assert (err <= tol).all(), f"{float((err - tol).max())} above the bound, error {float(err.max())}"


def tables_for(rng, lens, B, spare=3):
    nb = [-(-max(int(n), 1) // B) for n in lens]
    order = rng.permutation(sum(nb) + spare)
    t = np.full((len(lens), max(nb) + 1), 10 ** 6, np.int32)   # entries past a context are never read
    at = 0
    for s, n in enumerate(nb):
        t[s, :n] = order[at:at + n]
        at += n
    return t, sum(nb) + spare


def fill_e4m3(rng, tables, lens, N, B, Hk, d, spread=0, exp=127):
    """An 8-bit pool whose unwritten slots hold NaN codes, written through the library."""
    kc, vc, ex = e4m3_pool(N, B, Hk, d, 0x7F, 255)
    for s, n in enumerate(lens):
        n = int(n)
        if n < 1:
            continue
        slots = tables[s][np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B
        k, v = rand(rng, (n, Hk, d)), rand(rng, (n, Hk, d))
        if spread:
            k = k * torch.exp2(torch.from_numpy(rng.integers(-2, 3, (n, Hk, 1)).astype(np.float32)).to(DEV))
            step = rng.integers(-spread, spread + 1, (n, Hk, 1)).astype(np.float32)
            v = v * torch.exp2(torch.from_numpy(step).to(DEV))
        pk.pk_reshape_and_cache_e4m3(k, v, i64(slots), kc, vc, ex)
    vals = values_of(kc, vc, ex)
    return kc, vc, ex, vals


RHO_E4M3 = {torch.bfloat16: 2.0 ** -11, torch.float32: 2.0 ** -20}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,B", [(8, 8, 64, 16), (8, 1, 128, 16), (6, 2, 128, 8), (4, 1, 64, 32),
                                       (10, 2, 128, 32),
                                       (7, 1, 64, 8), (8, 8, 128, 16)])
def test_decode_e4m3(dtype, hq, hk, d, B):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(hq * 100 + d + B)
    lens = np.array([1, B - 1, B, B + 1, 63, 64, 65, 127, 129, 300], np.int32)
    S = len(lens)
    tables, N = tables_for(rng, lens, B)
    kc, vc, ex, (kv, vv) = fill_e4m3(rng, tables, lens, N, B, hk, d, spread=3)
    q = rand(rng, (S, hq, d), dt)
    scale = d ** -0.5
    want, terms = plain.tree_attention(f64(q), kv, vv, tables, lens, scale)
    desc = pk.cache_desc(kc)
    tb, ln = i32(tables), i32(lens)
    for part, planned in ((0, False), (64, False), (64, True), (96 if B <= 32 else 64, False), (-1, True)):
        out = torch.full_like(q, float("nan"))
        items = None
        if planned:
            part, it = pk.pk_attention_plan(lens, hq, desc, part)
            items = torch.from_numpy(it).to(DEV)
        ws = torch.full((max(16, pk.pk_paged_attention_workspace_size(S, hq, 300, part, desc)),), 255,
                        dtype=torch.uint8, device=DEV)
        pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, tb, ln, scale, 300, partition_size=part, workspace=ws,
                                          work_items=items)
        check_attention(f64(out), want, terms, d, dt, RHO_E4M3[dt])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [-60, 0, 100])
def test_decode_e4m3_exponents(dtype, shift):
    """Values of very small, very large and mixed magnitudes, zero rows and equal rows."""
    dt, hq, hk, d, B = DTYPES[dtype], 4, 2, 128, 16
    rng = np.random.default_rng(shift + 200)
    lens = np.array([50, 1, 200], np.int32)
    tables, N = tables_for(rng, lens, B)
    kc, vc, ex, _ = fill_e4m3(rng, tables, lens, N, B, hk, d, spread=6)
    live = ex != 255
    ex[..., 1] = torch.where(live[..., 1], (ex[..., 1].int() + shift).clamp(27, 247).to(torch.uint8), ex[..., 1])
    # a token whose value row is zero (exponent 0) and one whose key row is
    first = int(tables[0][0])
    vc.view(torch.uint8)[first, 3], ex[first, :, 3, 1] = 0, 127
    kc.view(torch.uint8)[first, 5], ex[first, :, 5, 0] = 0, 127
    vals = values_of(kc, vc, ex)
    q = rand(rng, (3, hq, d), dt)
    want, terms = plain.tree_attention(f64(q), *vals, tables, lens, d ** -0.5)
    for part in (0, 64):
        out = torch.full_like(q, float("nan"))
        ws = torch.empty(max(16, pk.pk_paged_attention_workspace_size(3, hq, 200, part, pk.cache_desc(kc))),
                         dtype=torch.uint8, device=DEV)
        pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tables), i32(lens), d ** -0.5, 200,
                                          partition_size=part, workspace=ws)
        check_attention(f64(out), want, terms, d, dt, RHO_E4M3[dt])


def test_decode_e4m3_large_scores():
    """Scores of hundreds: the softmax picks single tokens."""
    hq, hk, d, B = 4, 1, 128, 16
    rng = np.random.default_rng(77)
    lens = np.array([130, 70], np.int32)
    tables, N = tables_for(rng, lens, B)
    kc, vc, ex, vals = fill_e4m3(rng, tables, lens, N, B, hk, d)
    q = rand(rng, (2, hq, d)) * 20
    out = torch.empty_like(q)
    pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tables), i32(lens), 1.0, 130, partition_size=0)
    want, terms = plain.tree_attention(f64(q), *vals, tables, lens, 1.0)
    check_attention(f64(out), want, terms, d, torch.float32, RHO_E4M3[torch.float32])


def test_decode_e4m3_bad_inputs_are_recorded():
    hq, hk, d, B = 4, 2, 64, 16
    rng = np.random.default_rng(9)
    lens = np.array([20, 40], np.int32)
    tables, N = tables_for(rng, lens, B)
    kc, vc, ex, vals = fill_e4m3(rng, tables, lens, N, B, hk, d)
    q = rand(rng, (2, hq, d), torch.bfloat16)

    def call(tb, ln, **kw):
        out = torch.full_like(q, 3.0)
        pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tb), i32(ln), 0.125, 40, partition_size=0, **kw)
        return f64(out), pk.pk_get_device_error()

    good, err = call(tables, lens)
    assert err == (0, 0)
    out, err = call(tables, [20, 0])
    assert err == (4, 1) and (out[1] == 0).all() and np.array_equal(out[0], good[0])
    out, err = call(tables[:, :3], [20, 4000])              # longer than its table: clamped to 48
    assert err == (4, 1) and np.array_equal(out[0], good[0])
    for bad in (-1, N):
        t = tables.copy()
        t[1, 0] = bad
        out, err = call(t, lens)
        assert err == (2, 1) and np.array_equal(out[0], good[0])
    items = i32([[0, 0], [1, 0], [2, 0], [0, 1], [-1, 0]])
    out, err = call(tables, lens, work_items=items)
    assert err[0] == 6 and np.array_equal(out, good)


def random_masks(rng, n, kind):
    if kind == "any":
        bits = rng.integers(0, 2, (n, n))
        return [sum(int(b) << j for j, b in enumerate(r)) for r in bits]
    par = [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
    return [int(m) & (2 ** 64 - 1) for m in pk.pk_tree_masks(par)[0]] if n else []


def tree_case(rng, counts, lens, B, hq, hk, d, dt, kind, pad=3):
    tables, N = tables_for(rng, lens, B)
    k = torch.full((N, B, hk, d), float("nan"), dtype=dt, device=DEV)
    v = k.clone()
    for s, n in enumerate(lens):
        slots = tables[s][np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B
        for t in (k, v):
            t.view(-1, hk, d)[slots] = rand(rng, (int(n), hk, d), dt)
    ofs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    masks = None
    if kind != "chain":
        masks = sum([random_masks(rng, int(c), kind) for c in counts], []) + [0] * pad
    q = rand(rng, (int(ofs[-1]) + pad, hq, d), dt)
    q[int(ofs[-1]):] = float("nan")   # rows of no sequence
    mt = None if masks is None else i64([m - 2 ** 64 if m >= 2 ** 63 else m for m in masks])
    return tables, k, v, ofs, masks, q, mt


RHO_TREE = {torch.bfloat16: 2.0 ** -17, torch.float32: U}


def check_tree(out, q, k, v, tables, lens, scale, ofs, masks, d, dt):
    n = int(ofs[-1])
    want, terms = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, masks)
    check_attention(f64(out)[:n], want[:n], tuple(t[:n] for t in terms), d, dt, RHO_TREE[dt])
    assert (f64(out)[n:] == 5.0).all(), "rows of no sequence were written"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,B,kind", [(8, 8, 64, 16, "tree"), (8, 1, 128, 16, "any"), (6, 2, 128, 8, "tree"),
                                            (4, 1, 64, 32, "chain"), (10, 2, 128, 32, "any"), (7, 1, 64, 8, "tree"),
                                            (4, 4, 128, 5, "any"), (2, 1, 64, 64, "tree"), (4, 2, 128, 16, "chain")])
def test_tree_attention(dtype, hq, hk, d, B, kind):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(hq * 100 + d + B)
    counts = np.array([1, 0, 2, 5, 16, 33, 64, 7, 64, 3], np.int32)
    lens = np.array([1, 9, 2, 64, 65, 33, 64, 200, 200, 131], np.int32)   # several of drafts alone
    S = len(lens)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, kind)
    scale = d ** -0.5
    desc = pk.cache_desc(k)
    p64 = -(-64 // B) * B
    for part, planned in ((0, False), (p64, False), (p64, True), (2 * p64, True), (-1, True)):
        items = None
        if planned:
            part, it = pk.pk_tree_plan(lens, 64, hq, desc, part)
            items = torch.from_numpy(it).to(DEV)
        out = torch.full_like(q, 5.0)
        ws = torch.full((max(16, pk.pk_tree_workspace_size(len(q), hq, 200, part, desc)),), 255, dtype=torch.uint8,
                        device=DEV)
        pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), scale, 64, 200, tree_mask=mt,
                                   partition_size=part, workspace=ws, work_items=items)
        check_tree(out, q, k, v, tables, lens, scale, ofs, masks, d, dt)


@pytest.mark.parametrize("hq,hk,d,B,drafts", [(8, 8, 64, 16, 8), (4, 1, 64, 8, 2), (6, 2, 64, 32, 2), (2, 2, 64, 16, 9),
                                              (8, 1, 128, 16, 1), (4, 4, 128, 8, 8)])
def test_tree_few_rows(hq, hk, d, B, drafts):
    """bf16, one to nine rows of a KV head, on both sides of the rule that picks the kernel."""
    rng = np.random.default_rng(hq + 10 * d + drafts)
    counts = rng.integers(0, drafts + 1, 9).astype(np.int32)
    counts[3] = drafts
    lens = np.maximum(counts, [1, 700, 64, 130, 9, 65, 1031, 16, 17]).astype(np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, "any")
    desc = pk.cache_desc(k)
    for part in (0, 256, -1):
        part, it = pk.pk_tree_plan(lens, drafts, hq, desc, part)
        out = torch.full_like(q, 5.0)
        ws = torch.full((max(16, pk.pk_tree_workspace_size(len(q), hq, 1031, part, desc)),), 255, dtype=torch.uint8,
                        device=DEV)
        pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), d ** -0.5, drafts, 1031,
                                   tree_mask=mt, partition_size=part, workspace=ws,
                                   work_items=torch.from_numpy(it).to(DEV))
        check_tree(out, q, k, v, tables, lens, d ** -0.5, ofs, masks, d, torch.bfloat16)
    assert pk.pk_get_device_error() == (0, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_tree_hidden_tokens_do_not_reach_a_row(dtype):
    """NaN and infinities in the K/V of drafts that a row does not see."""
    dt, hq, hk, d, B = DTYPES[dtype], 4, 2, 128, 16
    rng = np.random.default_rng(12)
    counts, lens = [40, 6], np.array([60, 200], np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "chain")
    scale = d ** -0.5
    bad = 30                                       # draft 30 of sequence 0: rows 30.. see it
    pos = 20 + bad
    for side in (k, v):
        for val in (float("nan"), float("inf"), -float("inf")):
            kk, vv = k.clone(), v.clone()
            t = kk if side is k else vv
            t[int(tables[0][pos // B]), pos % B, 1] = val
            for part in (0, 64, 32):
                out = torch.full_like(q, 5.0)
                ws = torch.empty(max(16, pk.pk_tree_workspace_size(len(q), hq, 200, part, pk.cache_desc(k))),
                                 dtype=torch.uint8, device=DEV)
                pk.pk_paged_attention_tree(out, q, kk, vv, i32(tables), i32(lens), i32(ofs), scale, 40, 200,
                                           partition_size=part, workspace=ws)
                want, terms = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, None)
                see = np.ones((46, hq), bool)
                see[bad:40, 2:] = False
                check_attention(f64(out)[:46], want[:46], tuple(x[:46] for x in terms), d, dt, RHO_TREE[dt], see)
                if side is v:                      # the rows that see it show it
                    hit = f64(out)[bad:40, 2:]
                    assert not np.isfinite(hit).any()
                    if np.isinf(val):
                        assert (hit == val).all()


@pytest.mark.parametrize("dtype,B", [("f32", 16), ("bf16", 16), ("bf16", 5)])
def test_tree_infinities_that_a_row_sees(dtype, B):
    """Infinite context keys are scores of +-inf, infinite values reach the rows as they are."""
    dt, hq, hk, d = DTYPES[dtype], 4, 2, 128
    rng = np.random.default_rng(14)
    counts, lens = [7, 3], np.array([150, 40], np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "tree")
    kf, vf = k.clone(), v.clone()                  # finite twins, for the bounds

    def at(s, pos):
        return int(tables[s][pos // B]), pos % B

    inf, n = float("inf"), int(ofs[-1])
    k[at(0, 70)][1, 5] = -inf                      # -inf for positive query elements, +inf for the others
    k[at(1, 3)][0, 40] = inf
    q[0, 2, 5] = 0.75                              # exact in few bits
    for s, pos, col, val in ((0, 3, 7, inf), (0, 100, 8, -inf), (0, 64, 9, float("nan")), (0, 1, 10, inf),
                             (0, 140, 10, -inf), (1, 20, 127, -inf), (0, 130, 11, inf), (0, 131, 11, inf)):
        v[at(s, pos)][1, col] = val
    scale = d ** -0.5
    with np.errstate(invalid="ignore"):
        want, _ = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, masks)
    _, terms = plain.tree_attention(f64(q), f64(kf), f64(vf), tables, lens, scale, ofs, masks)
    live = np.isfinite(want[:n])
    assert live.any(axis=-1).any() and np.isinf(want[:n]).any() and np.isnan(want[:n]).all(axis=-1).any()
    top = np.nanmax(np.abs(f64(vf)))
    for part in (0, -(-64 // B) * B):
        out = torch.full_like(q, 5.0)
        ws = torch.empty(max(16, pk.pk_tree_workspace_size(len(q), hq, 200, part, pk.cache_desc(k))),
                         dtype=torch.uint8, device=DEV)
        pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), scale, 64, 200, tree_mask=mt,
                                   partition_size=part, workspace=ws)
        got = f64(out)[:n]
        assert np.array_equal(np.isnan(got), np.isnan(want[:n]))
        odd = np.isinf(want[:n])
        assert np.array_equal(odd, np.isinf(got)) and (got[odd] == want[:n][odd]).all()
        # The finite elements; a weighted mean of values is at most the largest.
        wv, mag, cnt = (np.full_like(want[:n], top), terms[1][:n], terms[2][:n])
        check_attention(np.where(live, got, 0.0), np.where(live, want[:n], 0.0), (wv, mag, cnt), d, dt, RHO_TREE[dt])


def test_tree_bad_inputs_are_recorded():
    hq, hk, d, B = 4, 2, 64, 16
    rng = np.random.default_rng(13)
    counts, lens = [3, 5], np.array([20, 40], np.int32)
    for dt in (torch.float32, torch.bfloat16):
        tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "tree")

        def call(tb=tables, ln=lens, of=ofs, md=5, **kw):
            out = torch.full_like(q, 5.0)
            pk.pk_paged_attention_tree(out, q, k, v, i32(tb), i32(ln), i32(of), 0.125, md, 40, tree_mask=mt, **kw)
            return f64(out), pk.pk_get_device_error()

        good, err = call()
        assert err == (0, 0)
        out, err = call(md=4)                                    # five drafts, a bound of four
        assert err == (8, 1) and np.array_equal(out[:3], good[:3]) and (out[3:] == 5.0).all()
        for of in ([0, 3, 2], [0, 3, 12], [-1, 3, 8]):
            out, err = call(of=of)
            assert err[0] == 8
        out, err = call(ln=[20, 4])                              # fewer tokens than drafts
        assert err == (4, 1) and np.array_equal(out[:3], good[:3]) and (out[3:8] == 0).all()
        out, err = call(ln=[20, 4000])
        assert err[0] in (2, 4)
        t = tables.copy()
        t[1, 0] = -7
        out, err = call(tb=t)
        assert err == (2, 1) and np.array_equal(out[:3], good[:3])
        out, err = call(work_items=i32([[0, 0], [1, 0], [7, 0], [0, 3]]))
        assert err[0] == 6 and np.array_equal(out, good)


# ---------------------------------------------------------------------------
# Together, on streams and in graphs
# ---------------------------------------------------------------------------
def serving_step(rng, dt, hq=4, hk=2, d=128, B=16):
    """Inputs of a verification step: contexts in the cache, drafts as a packed projection."""
    ctx, counts = np.array([37, 5, 90]), [6, 1, 11]
    bm = pk.BlockManager(64, B, rng.permutation(64).astype(np.int32))
    slots_ctx, slots_new, pos = [], [], []
    masks = []
    for s in range(3):
        bm.add_seq(s)
        slots_ctx.append(bm.append(s, int(ctx[s]))[0])
        slots_new.append(bm.append(s, counts[s])[0])
        m, depth = pk.pk_tree_masks([-1] + [int(rng.integers(-1, i)) for i in range(1, counts[s])])
        masks.append(m)
        pos.append(ctx[s] + depth)
    tables, lens = bm.export_tables(range(3), 8)
    rows = sum(counts)
    return dict(ctx=ctx, counts=counts, bm=bm, slots_ctx=np.concatenate(slots_ctx), slots_new=np.concatenate(slots_new),
                pos=np.concatenate(pos), masks=np.concatenate(masks), tables=tables, lens=lens,
                ofs=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
                qkv=rand(rng, (rows, hq + 2 * hk, d), dt), w=[(1 + 0.1 * rand(rng, (d,))).to(dt) for _ in range(2)],
                past=[rand(rng, (int(ctx.sum()), hk, d), dt) for _ in range(2)])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verification_step(dtype):
    """Norm, rotation and write of the drafts, attention over the tree; then the
    same tokens kept in 8 bits after a fork and a copied block, one more token
    decoded."""
    dt, hq, hk, d, B = DTYPES[dtype], 4, 2, 128, 16
    rng = np.random.default_rng(21)
    st = serving_step(rng, dt, hq, hk, d, B)
    kc, vc = torch.zeros((64, B, hk, d), dtype=dt, device=DEV), torch.zeros((64, B, hk, d), dtype=dt, device=DEV)
    pk.pk_reshape_and_cache(st["past"][0], st["past"][1], i64(st["slots_ctx"]), kc, vc)
    q, k, v = st["qkv"].split([hq, hk, hk], dim=1)
    qo = torch.empty((len(q), hq, d), dtype=dt, device=DEV)
    cs = rope_table(200, d)
    pk.pk_qk_norm_rope_and_cache(qo, None, q, k, v, torch.from_numpy(cs).to(DEV), i64(st["pos"]), q_weight=st["w"][0],
                                 k_weight=st["w"][1], slot_mapping=i64(st["slots_new"]), k_cache=kc, v_cache=vc)
    check_rope(qo, q, st["w"][0], np.float32(1e-6), cs, st["pos"], False, dt)
    check_rope(kc.view(-1, hk, d)[st["slots_new"]], k, st["w"][1], np.float32(1e-6), cs, st["pos"], False, dt)
    out = torch.full_like(qo, 5.0)
    scale = d ** -0.5
    pk.pk_paged_attention_tree(out, qo, kc, vc, i32(st["tables"]), i32(st["lens"]), i32(st["ofs"]), scale, 11, 101,
                               tree_mask=i64(st["masks"]))
    check_tree(out, qo, kc, vc, st["tables"], st["lens"], scale, st["ofs"], st["masks"], d, dt)

    # The pool in 8 bits; sequence 2 forks, its tail block is copied, and each decodes a token.
    k8, v8, ex = e4m3_pool(64, B, hk, d)
    every = np.concatenate([st["slots_ctx"], st["slots_new"]])
    pk.pk_reshape_and_cache_e4m3(kc.view(-1, hk, d)[every], vc.view(-1, hk, d)[every], i64(every), k8, v8, ex)
    bm = st["bm"]
    bm.fork(2, 3)
    slots, pairs = bm.append_batch(range(4))
    assert len(pairs) == 1
    pk.pk_copy_blocks_e4m3(k8, v8, ex, i64(pairs))
    kn, vn = rand(rng, (4, hk, d), dt), rand(rng, (4, hk, d), dt)
    pk.pk_reshape_and_cache_e4m3(kn, vn, i64(slots), k8, v8, ex)
    tables, lens = bm.export_tables(range(4), 8)
    vals = values_of(k8, v8, ex)
    for s, n in enumerate(lens):   # every token of every context has been written
        p = np.arange(n)
        assert np.isfinite(vals[0][tables[s][p // B], p % B]).all()
    q1 = rand(rng, (4, hq, d), dt)
    o1 = torch.empty_like(q1)
    pk.pk_paged_attention_decode_e4m3(o1, q1, k8, v8, ex, i32(tables), i32(lens), scale, int(lens.max()),
                                      partition_size=0)
    want, terms = plain.tree_attention(f64(q1), *vals, tables, lens, scale)
    check_attention(f64(o1), want, terms, d, dt, RHO_E4M3[dt])


def test_streams_and_graph_replay():
    """The operators on a side stream and as one captured graph, replayed with
    new inputs and longer contexts."""
    dt, hq, hk, d, B, S = torch.bfloat16, 4, 2, 128, 16, 3
    rng = np.random.default_rng(31)
    lens = np.array([100, 200, 17], np.int32)
    tables, N = tables_for(rng, lens + 20, B)
    k8, v8, ex, _ = fill_e4m3(rng, tables, lens + 20, N, B, hk, d)
    kc, vc = rand(rng, (N, B, hk, d), dt), rand(rng, (N, B, hk, d), dt)
    tb, ln, of = i32(tables), i32(lens), i32([0, 4, 5, 12])
    q, k, v = rand(rng, (12, hq, d), dt), rand(rng, (12, hk, d), dt), rand(rng, (12, hk, d), dt)
    qd = rand(rng, (S, hq, d), dt)
    pos, slots = i64(np.arange(12)), i64(np.r_[tables[0][0] * B + np.arange(12)])
    cs = torch.from_numpy(rope_table(64, 128)).to(DEV)
    desc, desc8 = pk.cache_desc(kc), pk.cache_desc(k8)
    qo, ko, o1, o2 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(qd)
    ws1 = torch.empty(pk.pk_tree_workspace_size(12, hq, 220, 64, desc), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(pk.pk_paged_attention_workspace_size(S, hq, 220, 64, desc8), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        pk.pk_qk_norm_rope_and_cache(qo, ko, q, k, v, cs, pos, slot_mapping=slots, k_cache=kc, v_cache=vc,
                                     stream=stream)
        pk.pk_reshape_and_cache_e4m3(ko, v, slots, k8, v8, ex, stream=stream)
        pk.pk_paged_attention_tree(o1, qo, kc, vc, tb, ln, of, 0.09, 7, 220, partition_size=64, workspace=ws1,
                                   stream=stream)
        pk.pk_paged_attention_decode_e4m3(o2, qd, k8, v8, ex, tb, ln, 0.09, 220, partition_size=64, workspace=ws2,
                                          stream=stream)

    def snap():
        torch.cuda.synchronize()
        return [t.clone() for t in (qo, ko, o1, o2, kc, k8.view(torch.uint8), ex)]

    step()
    ref = snap()
    side = torch.cuda.Stream()
    for t in (qo, ko, o1, o2):
        t.fill_(1)
    torch.cuda.synchronize()
    step(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, snap()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (qo, ko, o1, o2):
        t.fill_(1)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(ref, snap()))
    q.copy_(rand(rng, (12, hq, d), dt)), qd.copy_(rand(rng, (S, hq, d), dt))
    ln.add_(20)
    g.replay()
    got = snap()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, snap()))
    vals = values_of(k8, v8, ex)
    want, terms = plain.tree_attention(f64(qd), *vals, tables, lens + 20, 0.09)
    check_attention(f64(o2), want, terms, d, dt, RHO_E4M3[dt])


def test_tree_attention_repeats_bit_for_bit():
    """The same call many times, on one to a few tiles per partition and few
    rows, gives the same bits: nothing depends on when a product ends."""
    hq, hk, d, B = 8, 1, 128, 16
    rng = np.random.default_rng(944)
    counts = np.array([3, 1, 12, 40], np.int32)
    lens = np.array([131, 190, 260, 330], np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, "any")
    for part in (0, 64, 128, 192):
        ws = torch.empty(max(16, pk.pk_tree_workspace_size(len(q), hq, 330, part, pk.cache_desc(k))),
                         dtype=torch.uint8, device=DEV)
        first = None
        for _ in range(60):
            out = torch.full_like(q, 5.0)
            pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), d ** -0.5, 40, 330,
                                       tree_mask=mt, partition_size=part, workspace=ws)
            if first is None:
                first = out
                check_tree(out, q, k, v, tables, lens, d ** -0.5, ofs, masks, d, torch.bfloat16)
            assert torch.equal(out, first)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 4.0])
def test_scales_of_any_sign(scale):
    """Zero weighs every seen token alike; a negative scale reverses the order."""
    hq, hk, d, B = 4, 2, 128, 16
    rng = np.random.default_rng(55)
    counts, lens = np.array([5, 3], np.int32), np.array([70, 150], np.int32)
    for dt in (torch.bfloat16, torch.float32):
        tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "any")
        out = torch.full_like(q, 5.0)
        pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), scale, 5, 150, tree_mask=mt)
        n = int(ofs[-1])
        want, (wv, mag, cnt) = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, masks)
        check_attention(f64(out)[:n], want[:n], (wv[:n], np.abs(mag[:n]), cnt[:n]), d, dt, RHO_TREE[dt])
        tables, N = tables_for(rng, lens, B)
        kc, vc, ex, vals = fill_e4m3(rng, tables, lens, N, B, hk, d)
        q = rand(rng, (2, hq, d), dt)
        out = torch.empty_like(q)
        pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tables), i32(lens), scale, 150, partition_size=0)
        want, (wv, mag, cnt) = plain.tree_attention(f64(q), *vals, tables, lens, scale)
        check_attention(f64(out), want, (wv, np.abs(mag), cnt), d, dt, RHO_E4M3[dt])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_units_than_fit_and_sequences_without_work(dtype):
    """Hundreds of units for the persistent kernels, among them sequences without
    drafts, of invalid length and of one token; with a grid of partitions of which
    most are empty."""
    dt, hq, hk, d, B, S = DTYPES[dtype], 16, 16, 64, 16, 90
    rng = np.random.default_rng(66)
    lens = rng.integers(1, 90, S).astype(np.int32)
    lens[::9] = 1
    counts = np.minimum(rng.integers(0, 4, S), lens).astype(np.int32)
    counts[5::7] = 0
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "tree")
    want, terms = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, 0.125, ofs, masks)
    n = int(ofs[-1])
    for part in (0, 16):
        out = torch.full_like(q, 5.0)
        ws = torch.empty(max(16, pk.pk_tree_workspace_size(len(q), hq, 90, part, pk.cache_desc(k))), dtype=torch.uint8,
                         device=DEV)
        pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), 0.125, 3, 90, tree_mask=mt,
                                   partition_size=part, workspace=ws)
        check_attention(f64(out)[:n], want[:n], tuple(t[:n] for t in terms), d, dt, RHO_TREE[dt])
        assert (out[n:] == 5.0).all()
    # every other sequence shorter than its drafts: zero rows, the others as before
    short = lens.copy()
    bad = (np.arange(S) % 2 == 0) & (counts > 0)
    short[bad] = counts[bad] - 1
    out = torch.full_like(q, 5.0)
    pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(short), i32(ofs), 0.125, 3, 90, tree_mask=mt)
    assert pk.pk_get_device_error()[0] == 4
    row_bad = np.repeat(bad, counts)
    got = f64(out)[:n]
    assert (got[row_bad] == 0).all()
    check_attention(got, want[:n], tuple(t[:n] for t in terms), d, dt, RHO_TREE[dt], ~row_bad)

    kc, vc, ex, vals = fill_e4m3(rng, tables, lens, int(k.shape[0]), B, hk, d)
    q = rand(rng, (S, hq, d), dt)
    want, terms = plain.tree_attention(f64(q), *vals, tables, lens, 0.125)
    for part, bad in ((0, False), (16, False), (0, True)):
        use = lens.copy()
        if bad:
            use[::2] = 0
        out = torch.full_like(q, 5.0)
        ws = torch.empty(max(16, pk.pk_paged_attention_workspace_size(S, hq, 90, part, pk.cache_desc(kc))),
                         dtype=torch.uint8, device=DEV)
        pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tables), i32(use), 0.125, 90, partition_size=part,
                                          workspace=ws)
        if bad:
            assert pk.pk_get_device_error()[0] == 4 and (out[::2] == 0).all()
        live = np.ones(S, bool)
        live[::2] = not bad
        check_attention(f64(out), want, terms, d, dt, RHO_E4M3[dt], live)


def test_fp32_sums_have_no_bias():
    """Long unsplit contexts, fp32: rounding errors have no side, so that their mean over thousands of
    elements stays below 2^-20 of the values. (Each element is some 10^-6 off at most, in either
    direction: 140 roundings of 2^-24 a warp, and those of the scores. Sums that are cut off toward
    zero lose 10^-5.)"""
    hq, hk, d, B, ctx = 8, 2, 128, 16, 9000
    rng = np.random.default_rng(31)
    lens = np.array([ctx, ctx - 7], np.int32)
    tables, N = tables_for(rng, lens, B)
    for kind in ("e4m3", "tree"):
        k, v = rand(rng, (N, B, hk, d)), rand(rng, (N, B, hk, d))
        v += 1.0                                     # sums that only grow
        ofs = np.array([0, 12, 24], np.int32) if kind == "tree" else None
        q = rand(rng, (24 if kind == "tree" else 2, hq, d))
        out = torch.empty_like(q)
        if kind == "e4m3":
            kc, vc, ex = e4m3_pool(N, B, hk, d, 0, 127)
            every = torch.arange(N * B, device=DEV)
            pk.pk_reshape_and_cache_e4m3(k.view(-1, hk, d), v.view(-1, hk, d), every, kc, vc, ex)
            pk.pk_gather_cache_e4m3(k.view(-1, hk, d), v.view(-1, hk, d), every, kc, vc, ex)
            pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, i32(tables), i32(lens), d ** -0.5, ctx,
                                              partition_size=0)
        else:
            pk.pk_paged_attention_tree(out, q, k, v, i32(tables), i32(lens), i32(ofs), d ** -0.5, 12, ctx)
        want, _ = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, d ** -0.5, ofs)
        got = f64(out)
        assert abs((got * want).sum() / (want * want).sum() - 1.0) < 2.0 ** -20, kind
    assert pk.pk_get_device_error() == (0, 0)


def test_offsets_past_32_bits():
    """Blocks at the end of pools of more than 2^31 elements, and 2^32 bytes."""
    hq, hk, d, B = 4, 2, 128, 16
    rng = np.random.default_rng(88)
    N = (2 ** 31) // (B * hk * d) + 64
    lens, counts = np.array([40, 20], np.int32), np.array([3, 1], np.int32)
    tables = np.full((2, 3), -1, np.int32)
    tables[0, :3], tables[1, :2] = [N - 1, N - 7, 3], [N - 2, N - 20]
    use = np.unique(tables[tables >= 0])
    small = np.searchsorted(use, tables).astype(np.int32)          # the same blocks, packed
    kc = torch.empty((N, B, hk, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    blocks = i64(use)
    kc[blocks] = rand(rng, (len(use), B, hk, d), torch.bfloat16)
    vc[blocks] = rand(rng, (len(use), B, hk, d), torch.bfloat16)
    q, ofs = rand(rng, (4, hq, d), torch.bfloat16), [0, 3, 4]
    # new tokens through the fused write, at slots of the last blocks
    qkv = rand(rng, (4, hq + 2 * hk, d), torch.bfloat16)
    slots = np.array([(N - 1) * B + 15, (N - 7) * B + 3, (N - 2) * B, (N - 20) * B + 1])
    qo = torch.empty((4, hq, d), dtype=torch.bfloat16, device=DEV)
    pk.pk_qk_norm_rope_and_cache(qo, None, qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], None, None,
                                 slot_mapping=i64(slots), k_cache=kc, v_cache=vc)
    for s, row in zip(slots, qkv[:, hq:]):
        assert torch.equal(kc[int(s) // B, int(s) % B], row[:hk]) and torch.equal(vc[int(s) // B, int(s) % B], row[hk:])
    out = torch.full_like(q, 5.0)
    pk.pk_paged_attention_tree(out, q, kc, vc, i32(tables), i32(lens), i32(ofs), 0.09, 3, 40)
    want, terms = plain.tree_attention(f64(q), f64(kc[blocks]), f64(vc[blocks]), small, lens, 0.09, ofs, None)
    check_attention(f64(out), want, terms, d, torch.bfloat16, RHO_TREE[torch.bfloat16])
    del kc, vc
    torch.cuda.empty_cache()
    k8 = torch.empty((N, B, hk, d), dtype=torch.float8_e4m3fn, device=DEV)
    v8 = torch.empty_like(k8)
    ex = torch.empty((N, hk, B, 2), dtype=torch.uint8, device=DEV)
    every = (use[:, None].astype(np.int64) * B + np.arange(B)).reshape(-1)
    k, v = rand(rng, (len(every), hk, d)), rand(rng, (len(every), hk, d))
    pk.pk_reshape_and_cache_e4m3(k, v, i64(every), k8, v8, ex)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    pk.pk_gather_cache_e4m3(k2, v2, i64(every), k8, v8, ex)
    assert (k2 - k).abs().max() <= k.abs().max() * 2.0 ** -4 and (v2 - v).abs().max() <= v.abs().max() * 2.0 ** -4
    q = rand(rng, (2, hq, d))
    out = torch.empty_like(q)
    pk.pk_paged_attention_decode_e4m3(out, q, k8, v8, ex, i32(tables), i32(lens), 0.09, 40, partition_size=0)
    want, terms = plain.tree_attention(f64(q), f64(k2).reshape(-1, B, hk, d), f64(v2).reshape(-1, B, hk, d), small,
                                       lens, 0.09)
    check_attention(f64(out), want, terms, d, torch.float32, RHO_E4M3[torch.float32])


def test_two_streams_at_once():
    """Overlapping calls of the attentions on two streams, with a workspace each."""
    hq, hk, d, B, S = 8, 2, 128, 16, 40
    rng = np.random.default_rng(99)
    lens = rng.integers(40, 900, S).astype(np.int32)
    counts = rng.integers(1, 9, S).astype(np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, "tree", pad=0)
    kc, vc, ex, _ = fill_e4m3(rng, tables, lens, int(k.shape[0]), B, hk, d)
    qd = rand(rng, (S, hq, d), torch.bfloat16)
    tb, ln, of = i32(tables), i32(lens), i32(ofs)

    def call(stream=None):
        outs = [torch.zeros_like(q), torch.zeros_like(qd)]
        ws = [torch.empty(pk.pk_tree_workspace_size(len(q), hq, 900, 128, pk.cache_desc(k)), dtype=torch.uint8,
                          device=DEV),
              torch.empty(pk.pk_paged_attention_workspace_size(S, hq, 900, 128, pk.cache_desc(kc)), dtype=torch.uint8,
                          device=DEV)]
        torch.cuda.synchronize()
        return outs, ws, lambda: (
            pk.pk_paged_attention_tree(outs[0], q, k, v, tb, ln, of, 0.09, 8, 900, tree_mask=mt, partition_size=128,
                                       workspace=ws[0], stream=stream),
            pk.pk_paged_attention_decode_e4m3(outs[1], qd, kc, vc, ex, tb, ln, 0.09, 900, partition_size=128,
                                              workspace=ws[1], stream=stream))

    ref, _, f = call()
    f()
    torch.cuda.synchronize()
    sides = [call(torch.cuda.Stream()) for _ in range(3)]
    for _ in range(20):
        for _, _, f in sides:
            f()
    torch.cuda.synchronize()
    for outs, _, _ in sides:
        assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])

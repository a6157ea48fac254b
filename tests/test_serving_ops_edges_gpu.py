"""Attention of drafted tokens and over the 8-bit cache where its parts meet: units
that follow one another on a CTA, states that are merged, values that are not
finite, long partitions. Bounds as in test_serving_ops_gpu."""
import time

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from oracle import serving_ops as plain
from test_serving_ops_gpu import (DEV, DTYPES, RHO_E4M3, RHO_TREE, check_attention, f64, fill_e4m3, i32, rand,
                                  tables_for, tree_case, values_of)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


def tree_call(q, k, v, tables, lens, ofs, drafts, longest, part=0, items=None, masks=None, scale=None):
    """pk_paged_attention_tree with a poisoned workspace; rows of no sequence are 5."""
    out = torch.full_like(q, 5.0)
    size = pk.pk_tree_workspace_size(len(q), q.shape[1], longest, part, pk.cache_desc(k))
    ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device=DEV)
    pk.pk_paged_attention_tree(out, q, k, v, tables, lens, ofs, q.shape[2] ** -0.5 if scale is None else scale, drafts,
                               longest, tree_mask=masks, partition_size=part, workspace=ws, work_items=items)
    return out


def decode_call(q, kc, vc, ex, tables, lens, longest, part=0, items=None, scale=None):
    """pk_paged_attention_decode_e4m3 with a poisoned workspace."""
    out = torch.full_like(q, 5.0)
    size = pk.pk_paged_attention_workspace_size(len(q), q.shape[1], longest, part, pk.cache_desc(kc))
    ws = torch.full((max(16, size),), 255, dtype=torch.uint8, device=DEV)
    pk.pk_paged_attention_decode_e4m3(out, q, kc, vc, ex, tables, lens, q.shape[2] ** -0.5 if scale is None else scale,
                                      longest, partition_size=part, workspace=ws, work_items=items)
    return out


def check_like(got, want, terms, top, d, dtype, rho):
    """NaN and infinities where ``want`` has them; the rest within the bound, a weighted mean of
    values being at most the largest, ``top``."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    odd, live = np.isinf(want), np.isfinite(want)
    assert np.array_equal(odd, np.isinf(got)) and (got[odd] == want[odd]).all()
    wv, mag, cnt = np.full_like(want, top), np.abs(terms[1]), terms[2]
    check_attention(np.where(live, got, 0.0), np.where(live, want, 0.0), (wv, mag, cnt), d, dtype, rho)


def test_infinite_drafts_of_alternating_units():
    """Some 1600 units of one or two tiles, several to a CTA one after another, half of them with an
    infinite value in their first or last draft: the rows that see it are infinite in that column, and
    everything else is what it is without infinities, bit for bit, every time."""
    hq, hk, d, B, S = 4, 4, 128, 16, 400
    rng = np.random.default_rng(431)
    counts = rng.integers(1, 5, S).astype(np.int32)
    lens = (counts + rng.integers(0, 100, S)).astype(np.int32)
    tables, N = tables_for(rng, lens, B)
    k, v = rand(rng, (N, B, hk, d), torch.bfloat16), rand(rng, (N, B, hk, d), torch.bfloat16)
    ofs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = rand(rng, (int(ofs[-1]), hq, d), torch.bfloat16)
    args = i32(tables), i32(lens), i32(ofs), 4, int(lens.max())
    want = f64(tree_call(q, k, v, *args))
    assert np.isfinite(want).all()
    for s in range(S):
        for h in range(hk):
            if rng.integers(2):
                continue
            at = int(rng.choice([0, counts[s] - 1]))        # a chain: rows `at` and later see it
            pos, col, val = int(lens[s] - counts[s]) + at, int(rng.integers(d)), [np.inf, -np.inf][int(rng.integers(2))]
            v[int(tables[s][pos // B]), pos % B, h, col] = val
            want[ofs[s] + at:ofs[s + 1], h, col] = val
    for _ in range(100):
        assert np.array_equal(f64(tree_call(q, k, v, *args)), want)


# (dtype, heads, head_dim, block): drafts on tcgen05 (the first), and on the kernel of fp32 pools, of
# other block sizes and of few rows of 64 values
TREE_KERNELS = [("bf16", 8, 2, 128, 16), ("f32", 8, 2, 128, 16), ("bf16", 4, 2, 128, 5), ("bf16", 4, 2, 64, 16)]


@pytest.mark.parametrize("dtype,hq,hk,d,B", TREE_KERNELS)
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_tree_nan_that_a_row_sees(dtype, hq, hk, d, B, what):
    """A NaN query makes its row and head NaN and no other. A NaN key makes NaN what sees it, and a
    NaN or infinite value its column, also where they are alone in a warp's share of the context or in
    a partition, or have a weight that is 0 in 32 bits. Whole, split, and planned."""
    dt, p64 = DTYPES[dtype], -(-64 // B) * B
    rng = np.random.default_rng(17 + d + B)
    lens = np.array([17, p64 + 1, 2 * p64 + 1, 9, 700, 130], np.int32)
    counts = np.array([1, 2, 2, 1, 2, 0], np.int32)
    tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "chain")
    n, scale = int(ofs[-1]), d ** -0.5

    def at(s, pos):
        return int(tables[s][pos // B]), pos % B

    # Sequence 4: some scores of its second half are above those of its first by hundreds, so that the
    # first half's weights are 0 in 32 bits.
    k[at(4, 600)] = k[at(4, 600)] * 0 + 30.0
    q[int(ofs[4]):int(ofs[5])] = q[int(ofs[4]):int(ofs[5])].abs() + 1.0
    kf, vf, qf = k.clone(), v.clone(), q.clone()
    if what == "query":
        q[0, 1], q[int(ofs[2]), hq - 1], q[int(ofs[4]) + 1, 0, 3] = float("nan"), float("nan"), float("nan")
    elif what == "key":
        k[at(0, 16)][1] = float("nan")               # a draft, alone in a warp's 16 tokens
        k[at(1, p64)][0, 3] = float("nan")           # a draft, alone in the last partition
        k[at(2, 2 * p64 - 1)][0] = float("nan")      # the last draft but one: alone in nothing, seen by both rows
        k[at(3, 0)][1] = float("nan")                # context, with the draft in one tile
    else:
        for s, pos, col, val in ((0, 16, 2, "nan"), (1, p64, 5, "inf"), (2, 2 * p64, 6, "-inf"), (3, 0, 7, "nan"),
                                 (4, 3, 8, "inf"), (4, 70, 9, "nan"), (4, 200, 10, "-inf"), (4, 16, 11, "inf")):
            v[at(s, pos)][1, col] = float(val)
    with np.errstate(invalid="ignore"):
        want, _ = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, masks)
    _, terms = plain.tree_attention(f64(qf), f64(kf), f64(vf), tables, lens, scale, ofs, masks)
    terms, top = tuple(t[:n] for t in terms), np.nanmax(np.abs(f64(vf)))
    assert not np.isfinite(want[:n]).all() and np.isfinite(want[:n]).any()
    for part, planned in ((0, False), (p64, False), (p64, True), (-1, True), (2 * p64, True)):
        items = None
        if planned:
            part, it = pk.pk_tree_plan(lens, 2, hq, pk.cache_desc(k), part)
            items = torch.from_numpy(it).to(DEV)
        got = f64(tree_call(q, k, v, i32(tables), i32(lens), i32(ofs), 2, 700, part, items))
        check_like(got[:n], want[:n], terms, top, d, dt, RHO_TREE[dt])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_decode_e4m3_nan(dtype, what):
    """As above over the 8-bit cache, where infinities are the NaN code too."""
    dt, hq, hk, d, B = DTYPES[dtype], 8, 2, 128, 16
    rng = np.random.default_rng(18)
    lens = np.array([1, 17, 65, 129, 700, 700, 64], np.int32)
    S = len(lens)
    tables, N = tables_for(rng, lens, B)
    kc, vc, ex, (kv, vv) = fill_e4m3(rng, tables, lens, N, B, hk, d)
    q = rand(rng, (S, hq, d), dt)
    q[4] = q[4].abs() + 1.0
    qf = q.clone()
    first = int(tables[4][600 // B])
    kc.view(torch.uint8)[first, 600 % B], ex[first, :, 600 % B, 0] = 0x78, 127   # keys of 256: scores of thousands
    finite = values_of(kc, vc, ex)

    def nan(codes, s, pos, h, col):
        codes.view(torch.uint8)[int(tables[s][pos // B]), pos % B, h, col] = 0x7F

    if what == "query":
        q[0, 1], q[2, 7], q[5, 0, 3] = float("nan"), float("nan"), float("nan")
    elif what == "key":
        nan(kc, 0, 0, 0, 5), nan(kc, 1, 16, 1, 6), nan(kc, 2, 64, 0, 7), nan(kc, 3, 128, 1, 8), nan(kc, 5, 3, 0, 9)
    else:
        nan(vc, 0, 0, 0, 5), nan(vc, 1, 16, 1, 6), nan(vc, 2, 64, 0, 7), nan(vc, 3, 128, 1, 8)
        nan(vc, 4, 3, 0, 9), nan(vc, 4, 100, 1, 10), nan(vc, 5, 699, 1, 11)
    with np.errstate(invalid="ignore"):
        want, _ = plain.tree_attention(f64(q), *values_of(kc, vc, ex), tables, lens, d ** -0.5)
    _, terms = plain.tree_attention(f64(qf), *finite, tables, lens, d ** -0.5)
    top = np.nanmax(np.abs(finite[1]))
    assert np.isnan(want).any() and np.isfinite(want).any()
    for part, planned in ((0, False), (64, False), (64, True), (-1, True), (128, True)):
        items = None
        if planned:
            part, it = pk.pk_attention_plan(lens, hq, pk.cache_desc(kc), part)
            items = torch.from_numpy(it).to(DEV)
        got = f64(decode_call(q, kc, vc, ex, i32(tables), i32(lens), 700, part, items))
        check_like(got, want, terms, top, d, dt, RHO_E4M3[dt])


@pytest.mark.parametrize("dtype,hq,hk,d,B", TREE_KERNELS)
def test_tree_rows_whose_scores_are_all_minus_infinity(dtype, hq, hk, d, B):
    """exp(-inf - -inf) is NaN in the formula; a row that sees nothing stays 0, and a row of one more
    token has that token's value."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(19)
    lens, counts = np.array([4, 3, 90], np.int32), np.array([4, 2, 2], np.int32)
    tables, k, v, ofs, _, q, _ = tree_case(rng, counts, lens, B, hq, hk, d, dt, "chain", pad=0)
    q = q.abs() + 0.5
    masks = [0b0, 0b1, 0b11, 0b100, 0, 1, 0, 3]       # per sequence: 4, 2, 2 drafts
    for s, pos in ((0, 0), (0, 1), (1, 0), (1, 1)):
        k[int(tables[s][pos // B]), pos % B] = -float("inf")
    for pos in range(88):                             # the whole context of the last sequence
        k[int(tables[2][pos // B]), pos % B, 1] = -float("inf")
    with np.errstate(invalid="ignore"):
        want, _ = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, d ** -0.5, ofs, masks)
    assert np.isnan(want[[1, 2, 4, 5]]).all() and (want[0] == 0).all() and np.isfinite(want[[3, 7]]).all()
    assert np.isnan(want[6, hq // hk:]).all()
    words = torch.tensor(masks, dtype=torch.int64, device=DEV)
    p32 = -(-32 // B) * B
    for part in (0, p32):
        got = f64(tree_call(q, k, v, i32(tables), i32(lens), i32(ofs), 4, 90, part, masks=words))
        assert np.array_equal(np.isnan(got), np.isnan(want)) and (got[0] == 0).all()
        assert np.array_equal(got[3], want[3])        # one token, exact


@pytest.mark.parametrize("drafts", [2, 9, 20])
def test_tree_largest_finite_fp32_values(drafts):
    """fp32's largest numbers round to infinity in bf16: they must not reach the rows that do not see
    them, and act as finite ones in those that do."""
    hq, hk, d, B = 2, 1, 128, 16
    rng = np.random.default_rng(20)
    lens, counts = np.array([drafts + 21, 40], np.int32), np.array([drafts, 1], np.int32)
    tables, k, v, ofs, _, q, _ = tree_case(rng, counts, lens, B, hq, hk, d, torch.float32, "chain", pad=0)
    top = torch.finfo(torch.float32).max
    last = int(tables[0][(lens[0] - 1) // B]), int(lens[0] - 1) % B
    n = int(ofs[-1])
    for side in (k, v):
        was = side[last].clone()
        for val in (top, -top):
            side[last] = val
            got = f64(tree_call(q, k, v, i32(tables), i32(lens), i32(ofs), drafts, int(lens.max())))
            with np.errstate(over="ignore"):
                want, terms = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, d ** -0.5, ofs, None)
            live = np.ones((n, hq), bool)
            if side is k:                      # its own row's scores pass 32 bits
                live[drafts - 1] = False
            check_attention(got, want, terms, d, torch.float32, RHO_TREE[torch.float32], live)
        side[last] = was


def test_lengths_above_the_bound_are_clamped_to_it():
    """A length that the table holds but the call's max_context_len does not is recorded and cut to
    it, whether the call splits or not."""
    hq, hk, d, B, most = 4, 2, 128, 16, 100
    rng = np.random.default_rng(23)
    lens, counts = np.array([60, 140], np.int32), np.array([2, 3], np.int32)
    cut = np.minimum(lens, most)
    for dt in DTYPES.values():
        tables, k, v, ofs, _, q, _ = tree_case(rng, counts, lens, B, hq, hk, d, dt, "chain", pad=0)
        n = int(ofs[-1])
        want, terms = plain.tree_attention(f64(q), f64(k), f64(v), tables, cut, d ** -0.5, ofs, None)
        for part in (0, 64):
            out = tree_call(q, k, v, i32(tables), i32(lens), i32(ofs), 3, most, part)
            assert pk.pk_get_device_error() == (4, 1)
            check_attention(f64(out)[:n], want[:n], tuple(t[:n] for t in terms), d, dt, RHO_TREE[dt])
        kc, vc, ex, vals = fill_e4m3(rng, tables, lens, int(k.shape[0]), B, hk, d)
        q = rand(rng, (2, hq, d), dt)
        want, terms = plain.tree_attention(f64(q), *vals, tables, cut, d ** -0.5)
        for part in (0, 64):
            out = decode_call(q, kc, vc, ex, i32(tables), i32(lens), most, part)
            assert pk.pk_get_device_error() == (4, 1)
            check_attention(f64(out), want, terms, d, dt, RHO_E4M3[dt])


def test_device_errors_are_read_at_once():
    """Events of several operators: the first of the documented kinds in the library's order comes back,
    all are cleared, and the read costs a few round trips to the device, however many operators there
    are (six reads one after another took nine times one scalar's)."""
    rng = np.random.default_rng(24)
    q, k = rand(rng, (3, 2, 64)), rand(rng, (3, 1, 64))
    cs = torch.ones((4, 64), device=DEV)
    bad_pos = torch.tensor([0, 9, 1], device=DEV)
    kc = torch.zeros((2, 16, 1, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ex = torch.zeros((2, 1, 16, 2), dtype=torch.uint8, device=DEV)
    out = torch.zeros_like(k)
    pool = torch.zeros((2, 16, 1, 64), device=DEV)
    for only in (False, True):
        pk.pk_paged_attention_tree(torch.empty_like(q), q, pool, pool, i32([[0]]), i32([3]), i32([0, 9]), 0.1, 4, 16)
        pk.pk_gather_cache_e4m3(out, out.clone(), torch.tensor([0, 1, 99], device=DEV), kc, kc.clone(), ex)
        if not only:
            pk.pk_qk_norm_rope_and_cache(torch.empty_like(q), torch.empty_like(k), q, k, None, cs, bad_pos)
        assert pk.pk_get_device_error() == ((1, 2) if only else (7, 1))
        assert pk.pk_get_device_error() == (0, 0)

    word = torch.zeros(1, dtype=torch.int32, device=DEV)

    def median(f):
        times = []
        for _ in range(60):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return sorted(times)[30]

    median(pk.pk_get_device_error)
    one, read = median(word.item), median(pk.pk_get_device_error)
    print(f"a scalar {one * 1e6:.1f} us, the errors {read * 1e6:.1f} us")
    assert read < 4 * one


def fast_attention(q, k, v, lens, scale, ofs=None):
    """As plain.tree_attention over contexts that lie one after another, fp64 on the GPU: k, v
    [sum of lens, Hk, d] on the GPU; a chain with ``ofs``."""
    R, hq, d = q.shape
    qd = q.double()
    out, wv = torch.zeros((R, hq, d), dtype=torch.float64, device=DEV), torch.zeros((R, hq, d), dtype=torch.float64,
                                                                                  device=DEV)
    mag, cnt = torch.zeros((R, hq), dtype=torch.float64, device=DEV), torch.zeros((R, hq), dtype=torch.float64,
                                                                                device=DEV)
    at = 0
    for s, n in enumerate(lens):
        ks, vs = k[at:at + n].double(), v[at:at + n].double()
        at += n
        r0, r1 = (s, s + 1) if ofs is None else (ofs[s], ofs[s + 1])
        for i in range(r0, r1):
            m = n - (r1 - 1 - i)
            for h in range(hq):
                g = h // (hq // k.shape[1])
                x = ks[:m, g] @ qd[i, h] * scale
                w = torch.softmax(x, 0)
                out[i, h], wv[i, h] = w @ vs[:m, g], w @ vs[:m, g].abs()
                mag[i, h] = (ks[:m, g].abs() @ qd[i, h].abs()).max() * scale * plain.LOG2E
                cnt[i, h] = m
    return tuple(f64(t) for t in (out, wv, mag, cnt))


def check_long(got, exact, terms, d, dtype, rel, flips=0.02):
    """Three bounds, the coarse one for every element. Each: the scores' D (see test_serving_ops_gpu),
    and ``rel`` of the weighted magnitudes for all that weights and sums may lose if no two errors
    cancel, beside the result's own rounding. fp32: the mean error over all elements, which roundings to
    the nearest leave near 0 (2^-24 sqrt(n), of which independent rows cancel), is below 2^-19; sums
    that are cut off toward zero lose 2^-15 at 32 768 tokens. bf16: an error of r crosses the border of
    a rounding with a probability of at most 2 r 2^8, so that with r up to 2^-16 fewer than 2% of the
    results differ from the exact one, rounded; weights of one fp16 cross it in 10% (``flips`` None:
    not asked)."""
    wv, mag, _ = terms
    half = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}[dtype]
    bound = (4 * np.log(2) * (d + 8) * 2.0 ** -23 * mag[..., None] + rel) * wv + half * np.abs(exact)
    assert np.isfinite(got).all() and (np.abs(got - exact) <= bound).all(), float((np.abs(got - exact) / bound).max())
    if dtype == torch.float32:
        assert abs(((got - exact) * exact).sum() / (exact * exact).sum()) < 2.0 ** -19
    elif flips is not None:
        assert (got != f64(torch.from_numpy(exact).to(torch.bfloat16))).mean() < flips


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,B", [(128, 8), (128, 16), (64, 16)])
def test_decode_e4m3_long(dtype, d, B):
    """Long contexts element by element: hundreds of stages and table chunks, whole and planned. A warp
    adds up to 2^9 tiles, and a lane 2^10 terms of the denominator, each with a rounding of 2^-24 of what
    is there so far, half the total on average: 2^-16 and 2^-15; weights are good to 2^-22."""
    dt, hq, hk = DTYPES[dtype], 8, 2
    rng = np.random.default_rng(25 + d + B)
    lens = np.array([8191, 32768 + 7, 4097], np.int32)
    tables, N = tables_for(rng, lens, B)
    kc, vc = (torch.zeros((N, B, hk, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    ex = torch.zeros((N, hk, B, 2), dtype=torch.uint8, device=DEV)
    slots = torch.from_numpy(np.concatenate([tables[s][np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B
                                             for s, n in enumerate(lens)])).to(DEV)
    k, v = rand(rng, (len(slots), hk, d)), rand(rng, (len(slots), hk, d))
    if dt == torch.float32:
        v += 1.0                                     # sums that only grow
    pk.pk_reshape_and_cache_e4m3(k, v, slots, kc, vc, ex)
    pk.pk_gather_cache_e4m3(k, v, slots, kc, vc, ex)
    q = rand(rng, (3, hq, d), dt)
    exact, *terms = fast_attention(q, k, v, lens, d ** -0.5)
    for part, planned in ((0, False), (-1, True), (1024, True)):
        items = None
        if planned:
            part, it = pk.pk_attention_plan(lens, hq, pk.cache_desc(kc), part)
            items = torch.from_numpy(it).to(DEV)
        out = decode_call(q, kc, vc, ex, i32(tables), i32(lens), int(lens.max()), part, items)
        check_long(f64(out), exact, terms, d, dt, 2.0 ** -14)


@pytest.mark.parametrize("dtype,hq,hk,d,B,drafts", [("bf16", 8, 2, 128, 8, 3), ("bf16", 8, 2, 128, 16, 40),
                                                    ("bf16", 8, 2, 64, 16, 4), ("bf16", 4, 2, 64, 16, 3),
                                                    ("f32", 8, 2, 128, 16, 3)])
def test_tree_long(dtype, hq, hk, d, B, drafts):
    """Long contexts element by element, on both kernels, one and two tiles of rows, whole and planned.
    fp32 as over the 8-bit cache. bf16: weights good to 2^-17, and sums left to the tensor cores, which
    cut each off by at most 2^-23 of what is there so far, half the total on average: eight products a
    tile of 64 tokens, 4104 of them, 2^-12 at most. 2^-11 holds both."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(26 + d + drafts)
    lens, counts = np.array([8191, 32768 + 7, 4097], np.int32), np.array([drafts, drafts - 1, 1], np.int32)
    tables, N = tables_for(rng, lens, B)
    kc, vc = torch.zeros((N, B, hk, d), dtype=dt, device=DEV), torch.zeros((N, B, hk, d), dtype=dt, device=DEV)
    slots = torch.from_numpy(np.concatenate([tables[s][np.arange(n) // B].astype(np.int64) * B + np.arange(n) % B
                                             for s, n in enumerate(lens)])).to(DEV)
    k, v = rand(rng, (len(slots), hk, d), dt), rand(rng, (len(slots), hk, d), dt) + 1.0   # sums that only grow
    kc.view(-1, hk, d)[slots], vc.view(-1, hk, d)[slots] = k, v
    ofs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = rand(rng, (int(ofs[-1]), hq, d), dt)
    exact, *terms = fast_attention(q, k, v, lens, d ** -0.5, ofs)
    for part, planned in ((0, False), (-1, True), (1024, True)):
        items = None
        if planned:
            part, it = pk.pk_tree_plan(lens, drafts, hq, pk.cache_desc(kc), part)
            items = torch.from_numpy(it).to(DEV)
        out = tree_call(q, kc, vc, i32(tables), i32(lens), i32(ofs), drafts, int(lens.max()), part, items)
        check_long(f64(out), exact, terms, d, dt, 2.0 ** (-14 if dt == torch.float32 else -11), None)


@pytest.mark.parametrize("kind", ["decode", "tree", "few rows"])
def test_fp32_rows_are_close_as_a_whole(kind):
    """The bounds of single elements add every rounding up and let 10^-4 pass. Of a whole row the errors
    are independent: d products of a score leave sqrt(d) 2^-24 of its magnitude (a few 10^-7 of a weight
    at scores of a few units), the weights' errors average out over the tokens, and sums of n terms leave
    sqrt(n) 2^-24: below 2^-18 of the row's norm, all told."""
    dt, hq, hk, B = torch.float32, 8, 2, 16
    d, drafts = (64, 2) if kind == "few rows" else (128, 9)
    rng = np.random.default_rng(27 + d)
    lens = np.array([300, 64, 17, 200, 1], np.int32)
    if kind == "decode":
        tables, N = tables_for(rng, lens, B)
        kc, vc, ex, vals = fill_e4m3(rng, tables, lens, N, B, hk, d, spread=3)
        q = rand(rng, (len(lens), hq, d))
        want, _ = plain.tree_attention(f64(q), *vals, tables, lens, d ** -0.5)
        runs = [decode_call(q, kc, vc, ex, i32(tables), i32(lens), 300, part) for part in (0, 64)]
    else:
        counts = np.minimum(drafts, lens).astype(np.int32)
        tables, k, v, ofs, masks, q, mt = tree_case(rng, counts, lens, B, hq, hk, d, dt, "tree", pad=0)
        want, _ = plain.tree_attention(f64(q), f64(k), f64(v), tables, lens, d ** -0.5, ofs, masks)
        runs = [tree_call(q, k, v, i32(tables), i32(lens), i32(ofs), drafts, 300, part, masks=mt) for part in (0, 64)]
    for out in runs:
        off = np.linalg.norm(f64(out) - want, axis=-1) / np.linalg.norm(want, axis=-1)
        assert off.max() < 2.0 ** -18, float(off.max())

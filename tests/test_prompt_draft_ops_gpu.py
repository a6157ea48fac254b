"""Prompt attention with changed scores, draft verification and cache compaction on the
GPU, element by element against their plain fp64 forms.

Tolerances are bounds from the arithmetic (u = 2^-24, one fp32 rounding; eta = half a
step of the output type: 2^-8 for bf16, u for fp32). Of a score in the exponent's scale:

* its product is off by at most D m_t, m_t = scale log2(e) sum_i |q_i k_i|, D = (d + 8) v,
  v one rounding of the sums (u, 2 u where the tensor cores may cut off);
* the cap's slope is at most 1, so D passes on; the tanh itself is off by at most T times
  cap log2(e), T = 2^-22 for fp32 (tanhf, 2 of its ulp) and 2^-17 for bf16 (an exponential and
  a reciprocal of 2 ulp and the roundings around them, 2^-21, or a polynomial, 2^-17.3 of a
  small score itself); products, bias and subtraction of the maximum round four times:
  together (T + 4 u) a_t, a_t the magnitude of cap, score and bias.

A weight is off by ln 2 times that, by 8 u for the exponential, and by rho, its rounding
where a product takes it in fewer bits (2^-17 as a bf16 pair; 2^-8 as one bf16; u
otherwise); a sum over n tokens adds n v. The output is a ratio of two such sums:
|error| <= 2 ln2 (sum_t w_t e_t |v_t| + |out| sum_t w_t e_t) + (16 u + 2 rho + 2 n v) sum_t w_t |v_t|
           + eta |out|,   e_t = D m_t + (T + 4 u) a_t.
"""
import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from oracle import prompt_draft_ops as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LN2 = float(np.log(2.0))
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


def rand(rng, shape, dtype=torch.float32):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).to(dtype)


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def i64(x):
    return torch.from_numpy(np.asarray(x, np.int64)).to(DEV)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
SCORES = {
    "plain": {},
    "cap": dict(softcap=4.0),
    "slopes": dict(slopes=True),
    "window": dict(window=37),
    "prefix": dict(prefix=True),
    "documents": dict(documents=True),
    "cap window": dict(softcap=2.0, window=150),
    "slopes prefix": dict(slopes=True, prefix=True),
    "all": dict(softcap=5.0, slopes=True, window=90, prefix=True, documents=True),
}


def make_case(rng, counts, lens, B, hq, hk, d, dt, kind, pad=3, spare=2):
    """A shuffled pool with spare blocks, offsets with `pad` rows behind the last sequence, score changes."""
    nb = [-(-n // B) for n in lens]
    order = rng.permutation(sum(nb) + spare)
    tables = np.full((len(lens), max(max(nb), 1)), -1, np.int32)
    at = 0
    for s, n in enumerate(nb):
        tables[s, :n] = order[at:at + n]
        at += n
    ofs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(ofs[-1]) + pad
    k, v = rand(rng, (len(order), B, hk, d), dt), rand(rng, (len(order), B, hk, d), dt)
    q = (rand(rng, (R, hq, d)) * 1.5).to(dt)
    o = SCORES[kind]
    sc = {"softcap": o.get("softcap", 0.0), "window": o.get("window", 0)}
    if o.get("slopes"):
        sc["slopes"] = (2.0 ** rng.uniform(-6, 0.5, hq)).astype(np.float32)
    if o.get("prefix"):
        sc["prefix_lens"] = np.array([rng.integers(0, n + 20) if n else 3 for n in lens], np.int32)
    if o.get("documents"):
        first = np.zeros(R, np.int32)
        for s, (c, n) in enumerate(zip(counts, lens)):
            cuts = np.sort(np.append(rng.integers(0, max(n, 1), 4), 0))
            for i in range(c):
                pos = n - c + i
                first[ofs[s] + i] = cuts[cuts <= pos].max() if rng.random() < 0.9 else pos + 1 + rng.integers(0, 3)
        sc["first_tokens"] = first
    return tables, k, v, ofs, q, sc


def on_device(sc):
    out = dict(sc)
    for name in ("prefix_lens", "first_tokens"):
        if name in sc:
            out[name] = i32(sc[name])
    if "slopes" in sc:
        out["slopes"] = torch.from_numpy(sc["slopes"]).to(DEV)
    return out


def check_extend(out, q, k, v, tables, lens, scale, ofs, sc, before=7.0):
    dt, d, R = q.dtype, q.shape[2], len(q)
    want, (wv, (mv, ms), (av, as_), cnt) = plain.extend_attention(f64(q), f64(k), f64(v), tables, lens, scale, ofs, **sc)
    got = f64(out)
    rows = ~np.isnan(want[:, 0, 0])
    if ofs is not None:
        live = np.zeros(R, bool)
        live[: int(ofs[-1])] = True
        assert (got[~live] == before).all(), "rows of no sequence were written"
    D = (d + 8) * 2 * U
    T = 2.0 ** -17 if dt == torch.bfloat16 else 2.0 ** -22
    rho = 2.0 ** -8 if dt == torch.bfloat16 else U
    e_v, e_s = D * mv + (T + 4 * U) * av, D * ms + (T + 4 * U) * as_
    tol = 2 * LN2 * (e_v + np.abs(want) * e_s) + (16 * U + 2 * rho + 4 * U * cnt) * wv + ETA[dt] * np.abs(want) + 1e-30
    bad = ~(np.abs(got - want) <= tol) & rows[:, None, None]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])


def run_extend(case, lens, counts, scale, part=0, listed=True, most=None, max_len=None, out=None):
    tables, k, v, ofs, q, sc = case
    hq, desc = q.shape[1], pk.cache_desc(k)
    most = most or max(max(counts), 1)
    max_len = max_len or max(lens)
    items = None
    if listed:
        part, items = pk.pk_extend_plan(lens, counts, hq, desc, part, window=sc["window"], max_query_len=most)
        items = torch.from_numpy(items).to(DEV)
    ws = torch.full((max(16, pk.pk_extend_workspace_size(len(q), hq, max_len, part, desc)),), 255, dtype=torch.uint8,
                    device=DEV)
    if out is None:
        out = torch.full_like(q, 7.0)
    pk.pk_paged_attention_extend(out, q, k, v, i32(tables), i32(lens), i32(ofs), scale, most, max_len,
                                 partition_size=part, workspace=ws, work_items=items, **on_device(sc))
    return out


@pytest.mark.parametrize("kind", sorted(SCORES))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,B", [(8, 8, 64, 16), (8, 2, 128, 16), (7, 1, 128, 8), (6, 2, 64, 32), (5, 1, 64, 5)])
def test_extend(kind, dtype, hq, hk, d, B):
    """Prompts, chunks, single tokens and an empty sequence in one batch, whole and split."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(hq * 100 + d + len(kind))
    counts = [1, 130, 0, 37, 5, 64]
    lens = [300, 130, 9, 180, 261, 65]
    case = make_case(rng, counts, lens, B, hq, hk, d, dt, kind)
    for part, listed in ((0, True), (0, False), (16 * B, True), (16 * B, False)):
        out = run_extend(case, lens, counts, d ** -0.5, part, listed)
        check_extend(out, case[4], case[1], case[2], case[0], lens, d ** -0.5, case[3], case[5])


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "window", "documents", "all"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hk,d,B", [(8, 1, 128, 16), (4, 4, 64, 8), (6, 2, 128, 32), (10, 2, 64, 16), (3, 3, 128, 12)])
def test_extend_single_tokens(kind, dtype, hq, hk, d, B):
    """One new token each, without offsets, at lengths around tiles and blocks."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(hq * 10 + d)
    lens = [1, 2, B, B + 1, 63, 64, 65, 127, 128, 129, 500, 1031]
    counts = [1] * len(lens)
    tables, k, v, ofs, q, sc = make_case(rng, counts, lens, B, hq, hk, d, dt, kind, pad=0)
    desc = pk.cache_desc(k)
    for part, listed in ((0, True), (0, False), (16 * B, True), (8 * B, False), (-1, True)):
        items = None
        if listed:
            part, it = pk.pk_extend_plan(lens, None, hq, desc, part, window=sc["window"])
            items = torch.from_numpy(it).to(DEV)
        ws = torch.full((max(16, pk.pk_extend_workspace_size(len(q), hq, 1031, part, desc)),), 255, dtype=torch.uint8,
                        device=DEV)
        out = torch.full_like(q, 7.0)
        pk.pk_paged_attention_extend(out, q, k, v, i32(tables), i32(lens), None, d ** -0.5, 1, 1031, partition_size=part,
                                     workspace=ws, work_items=items, **on_device(sc))
        check_extend(out, q, k, v, tables, lens, d ** -0.5, None, sc)


@pytest.mark.parametrize("hq,hk,d,counts", [(8, 1, 128, [1, 1, 0, 1]), (8, 2, 64, [2, 1, 2, 0]), (2, 2, 128, [8, 3, 1, 7]),
                                            (16, 2, 128, [2, 2, 1, 2]), (4, 1, 128, [40, 64, 63, 3]),
                                            (8, 1, 64, [33, 32, 31, 65])])
def test_extend_few_rows(hq, hk, d, counts):
    """Row counts around the borders between the kernels."""
    rng = np.random.default_rng(sum(counts) + hq)
    lens = [700, 64, 129, 300]
    for kind in ("all", "cap", "plain"):
        case = make_case(rng, counts, lens, 16, hq, hk, d, torch.bfloat16, kind)
        for part in (0, 128):
            out = run_extend(case, lens, counts, d ** -0.5, part)
            check_extend(out, case[4], case[1], case[2], case[0], lens, d ** -0.5, case[3], case[5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extend_negative_and_zero_scale(dtype):
    dt, B = DTYPES[dtype], 16
    for counts, lens in (([70, 20], [90, 40]), ([1, 1], [90, 40])):
        for kind in ("plain", "cap", "slopes"):
            case = make_case(np.random.default_rng(3), counts, lens, B, 4, 2, 128, dt, kind)
            for scale in (-0.11, 0.0):
                out = run_extend(case, lens, counts, scale)
                check_extend(out, case[4], case[1], case[2], case[0], lens, scale, case[3], case[5])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[90, 33, 5], [1, 1, 1], [2, 1, 2]])
def test_extend_hidden_tokens_do_not_reach_a_row(dtype, counts):
    """NaN and infinities in every place that no row of its sequence sees, or only some do: the rows
    that do not see them are as without; those that do are not finite in that element (values) or at
    all (NaN keys)."""
    dt, B, hq, hk, d = DTYPES[dtype], 16, 4, 2, 128
    rng = np.random.default_rng(17)
    lens = [200, 120, 61]
    for kind in ("window", "documents", "prefix", "all"):
        tables, k, v, ofs, q, sc = make_case(rng, counts, lens, B, hq, hk, d, dt, kind)
        for s, n in enumerate(lens):  # what lies behind the context in its last block
            if n % B:
                k[tables[s, n // B], n % B:] = float("nan")
                v[tables[s, n // B], n % B:] = float("inf")
        tok = [int(rng.integers(0, n)) for n in lens]
        for bad, where in ((float("nan"), v), (float("inf"), v), (float("nan"), k)):
            kk, vv = k.clone(), v.clone()
            pool = vv if where is v else kk
            for s, t in enumerate(tok):
                pool[tables[s, t // B], t % B, 0, 3] = bad
            case = (tables, kk, vv, ofs, q, sc)
            for part in (0, 64):
                out = run_extend(case, lens, counts, d ** -0.5, part)
                # Rows that see the token, by the definition.
                sees = np.zeros(len(q), bool)
                for s, (c, n) in enumerate(zip(counts, lens)):
                    for i in range(c):
                        pos = n - c + i
                        ok = tok[s] <= pos or ("prefix_lens" in sc and tok[s] < sc["prefix_lens"][s])
                        ok = ok and not (sc["window"] and tok[s] <= pos - sc["window"])
                        ok = ok and not ("first_tokens" in sc and tok[s] < sc["first_tokens"][ofs[s] + i])
                        sees[ofs[s] + i] = ok
                g = f64(out)
                hit = g[: ofs[-1]][sees[: ofs[-1]]][:, : hq // hk]  # KV head 0's
                if where is v:
                    assert not np.isfinite(hit[..., 3]).any()
                else:
                    assert np.isnan(hit).all()
                clean = out.clone()
                mask = torch.from_numpy(sees).to(DEV)
                heads = clean[mask]
                want = run_extend((tables, k, v, ofs, q, sc), lens, counts, d ** -0.5, part)
                heads[:, : hq // hk] = want[mask][:, : hq // hk]
                clean[mask] = heads
                kc, vc = k.nan_to_num(0, 0, 0), v.nan_to_num(0, 0, 0)
                check_extend(clean, q, kc, vc, tables, lens, d ** -0.5, ofs, sc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts", [[90, 33], [1, 1]])
def test_extend_scores_of_minus_infinity(dtype, counts):
    """A key of -inf is as good as hidden; a row that sees nothing else gets zeros."""
    dt, B, d = DTYPES[dtype], 16, 64
    rng = np.random.default_rng(5)
    lens = [90, 40]
    tables, k, v, ofs, q, sc = make_case(rng, counts, lens, B, 2, 2, d, dt, "plain")
    q = q.abs() + 0.1
    k[tables[0, 0], 0] = float("-inf")
    k[tables[1, 0], 5] = float("-inf")
    for part in (0, 64):
        out = run_extend((tables, k, v, ofs, q, sc), lens, counts, 0.125, part)
        got = f64(out)
        kk, vv = f64(k), f64(v)
        for s, n in enumerate(lens):
            for i in range(counts[s]):
                pos = np.arange(n - counts[s] + i + 1)
                ks, vs = kk[tables[s][pos // B], pos % B], vv[tables[s][pos // B], pos % B]
                for h in range(2):
                    with np.errstate(invalid="ignore"):
                        x = ks[:, h] @ f64(q)[ofs[s] + i, h] * 0.125
                    if np.max(x) == -np.inf:
                        assert (got[ofs[s] + i, h] == 0).all()
                        continue
                    w = np.exp(x - x.max())
                    w = w / w.sum()
                    # As check_extend's, with |q k| of 64 products of about 1.2 at most some 400.
                    e = 2 * LN2 * (72 * 2 * U + 4 * U) * 400
                    rho = 2.0 ** -8 if dt == torch.bfloat16 else U
                    tol = (2 * e + 16 * U + 2 * rho + 4 * U * len(pos)) * (w @ np.abs(vs[:, h])) + ETA[dt] * np.abs(
                        w @ vs[:, h])
                    assert (np.abs(got[ofs[s] + i, h] - w @ vs[:, h]) <= tol).all()


def dense(q, k, v, tables, lens, counts, ofs, scale, sc):
    """extend_attention and check_extend's bound for long prompts: fp64 matrices on the GPU, a sequence
    and head at a time."""
    R, hq, d = q.shape
    B, hk = k.shape[1], k.shape[2]
    out, tol = torch.zeros((R, hq, d), dtype=torch.float64, device=DEV), torch.zeros((R, hq, d), dtype=torch.float64, device=DEV)
    D, T, rho, cap = (d + 8) * 2 * U, 2.0 ** -17, 2.0 ** -8, sc["softcap"]
    log2e = 1 / LN2
    for s, (n, c) in enumerate(zip(lens, counts)):
        blocks = i64(tables[s][: -(-n // B)])
        kk, vv = (x[blocks].reshape(-1, hk, d)[:n].double() for x in (k, v))
        pos, t = torch.arange(n - c, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        see = t <= pos
        if "prefix_lens" in sc:
            see = see | (t < int(sc["prefix_lens"][s]))
        if sc["window"]:
            see = see & (t > pos - sc["window"])
        if "first_tokens" in sc:
            see = see & (t >= i32(sc["first_tokens"])[ofs[s]: ofs[s + 1], None])
        for h in range(hq):
            qh, kh, vh = q[ofs[s]: ofs[s + 1], h].double(), kk[:, h * hk // hq], vv[:, h * hk // hq]
            x, m = qh @ kh.T * scale, qh.abs() @ kh.abs().T * abs(scale) * log2e
            if cap:
                x = torch.tanh(x / cap) * cap
            a = x.abs() + cap
            if "slopes" in sc:
                far = (pos - t).abs() * float(sc["slopes"][h])
                x, a = x - far, a + far
            w = torch.softmax(x.masked_fill(~see, -float("inf")), 1).nan_to_num(0.0)
            o, e = w @ vh, w * (D * m + (T + 4 * U) * a * log2e)
            out[ofs[s]: ofs[s + 1], h] = o
            tol[ofs[s]: ofs[s + 1], h] = 2 * LN2 * (e @ vh.abs() + o.abs() * e.sum(1, keepdim=True)) + (
                16 * U + 2 * rho + 4 * U * n) * (w @ vh.abs()) + 2.0 ** -8 * o.abs() + 1e-30
    return out, tol


@pytest.mark.parametrize("kind,cap", [("plain", 0.0), ("cap", 50.0), ("cap", 3.0), ("all", 20.0), ("documents", 0.0),
                                      ("prefix", 30.0), ("slopes", 0.0)])
@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (24, 8, 64)])
def test_extend_more_units_than_fit_at_once(kind, cap, hq, hk, d):
    """CTAs go on to units of other lengths, halves, heads and sequences; capped scores of every size."""
    rng = np.random.default_rng(hq + d + int(cap))
    counts, lens, B = [1500, 700, 40, 300, 1], [1500, 2100, 3100, 300, 1700], 16
    tables, k, v, ofs, q, sc = make_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, kind, pad=2)
    sc["softcap"] = cap
    if cap == 50.0:  # rows of large scores among small ones
        q[::97] *= 8
    want, tol = dense(q, k, v, tables, lens, counts, ofs, d ** -0.5, sc)
    for part in (0, 1024):
        out = run_extend((tables, k, v, ofs, q, sc), lens, counts, d ** -0.5, part)
        bad = (out.double() - want).abs() > tol
        bad[int(ofs[-1]):] = out[int(ofs[-1]):] != 7
        assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:5].tolist())
        assert torch.equal(run_extend((tables, k, v, ofs, q, sc), lens, counts, d ** -0.5, part), out)


def test_extend_hidden_nan_in_every_unit():
    """A NaN value behind every document's end: rows of other documents are as without."""
    rng = np.random.default_rng(77)
    n, B, hq, hk, d = 2600, 16, 16, 4, 128
    tables, k, v, ofs, q, sc = make_case(rng, [n], [n], B, hq, hk, d, torch.bfloat16, "plain")
    cuts = np.arange(0, n, 130)
    first = cuts[np.searchsorted(cuts, np.arange(n), side="right") - 1]
    sc["first_tokens"] = np.concatenate([first, np.zeros(3)]).astype(np.int32)
    clean = run_extend((tables, k, v, ofs, q, sc), [n], [n], 0.1)
    vv = v.clone()
    last = np.append(cuts[1:], n) - 1  # the last token of each document: seen by itself alone
    vv[i64(tables[0][last // B]), i64(last % B)] = float("nan")
    for part in (0, 512):
        out = run_extend((tables, k, vv, ofs, q, sc), [n], [n], 0.1, part)
        hit = torch.zeros(len(q), dtype=torch.bool, device=DEV)
        hit[i64(last)] = True
        assert bool(out[hit].isnan().all())
        want = run_extend((tables, k, v, ofs, q, sc), [n], [n], 0.1, part)
        assert torch.equal(out[~hit], want[~hit])
    assert bool(torch.isfinite(clean).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extend_many_sequences(dtype):
    """More sequences than a warp's lanes, many without rows, with a list and without; windows and first
    tokens beyond everything; and on a stream of its own."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(123)
    S, B, hq, hk, d = 150, 8, 4, 2, 64
    lens = rng.integers(1, 120, S).tolist()
    counts = [int(rng.integers(0, min(n, 40) + 1)) if rng.random() < 0.7 else 0 for n in lens]
    case = make_case(rng, counts, lens, B, hq, hk, d, dt, "plain")
    tables, k, v, ofs, q, sc = case
    for window, first in ((0, None), (2 ** 31 - 1, None), (3, None), (0, 2 ** 31 - 1)):
        sc["window"] = window
        sc.pop("first_tokens", None)
        if first is not None:
            sc["first_tokens"] = np.where(rng.random(len(q)) < 0.5, first, 0).astype(np.int32)
        for part, listed in ((0, True), (0, False), (64, True), (64, False)):
            out = run_extend(case, lens, counts, 0.125, part, listed)
            check_extend(out, q, k, v, tables, lens, 0.125, ofs, sc)
    st = torch.cuda.Stream()
    want = run_extend(case, lens, counts, 0.125)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        got = run_extend(case, lens, counts, 0.125)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_extend_long_context_in_parts_and_offsets_past_32_bits():
    """A pool of more than 2^31 elements, its last blocks in use, and a plan that splits."""
    B, hk, hq, d = 16, 8, 16, 128
    N = (1 << 31) // (B * hk * d) + 900
    k, v = (torch.empty((N, B, hk, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rng = np.random.default_rng(9)
    lens, counts = [9000, 2100], [40, 3]
    nb = [-(-n // B) for n in lens]
    blocks = N - 1 - rng.permutation(sum(nb))
    tables = np.full((2, max(nb)), -1, np.int32)
    tables[0, : nb[0]], tables[1, : nb[1]] = blocks[: nb[0]], blocks[nb[0]:]
    at = torch.from_numpy(np.sort(blocks)).to(DEV)
    for pool in (k, v):
        pool[at] = rand(rng, (len(blocks), B, hk, d), torch.bfloat16)
    small = {int(b): i for i, b in enumerate(np.sort(blocks))}
    ts = np.vectorize(lambda b: small.get(int(b), -1))(tables)
    ofs = np.array([0, 40, 43], np.int32)
    q = rand(rng, (43, hq, d), torch.bfloat16)
    sc = {"softcap": 30.0, "window": 0}
    for c, off, part in ((counts, ofs, -1), ([1, 1], np.array([0, 1, 2], np.int32), -1)):
        x = q[: off[-1]]
        p, items = pk.pk_extend_plan(lens, c, hq, pk.cache_desc(k), part)
        assert p > 0
        ws = torch.empty(pk.pk_extend_workspace_size(len(x), hq, 9000, p, pk.cache_desc(k)), dtype=torch.uint8, device=DEV)
        out = torch.full_like(x, 7.0)
        pk.pk_paged_attention_extend(out, x, k, v, i32(tables), i32(lens), i32(off), d ** -0.5, max(c), 9000, softcap=30.0,
                                     partition_size=p, workspace=ws, work_items=torch.from_numpy(items).to(DEV))
        check_extend(out, x, k[at], v[at], ts, lens, d ** -0.5, off, sc)


def test_extend_bad_inputs_are_recorded():
    rng = np.random.default_rng(1)
    counts, lens, B = [20, 3, 9], [50, 33, 40], 16
    for dt, cs in ((torch.bfloat16, counts), (torch.float32, counts), (torch.bfloat16, [1, 1, 1])):
        tables, k, v, ofs, q, sc = make_case(rng, cs, lens, B, 4, 2, 64, dt, "cap")
        good = run_extend((tables, k, v, ofs, q, sc), lens, cs, 0.125)

        def call(tb=tables, ln=lens, of=ofs, most=max(cs), max_len=50, items=None, part=0, ws=None):
            out = torch.full_like(q, 7.0)
            pk.pk_paged_attention_extend(out, q, k, v, i32(tb), i32(ln), i32(of), 0.125, most, max_len,
                                         partition_size=part, work_items=items, workspace=ws, **on_device(sc))
            return out, pk.pk_get_device_error()

        bad = tables.copy()
        bad[1, 0] = 1 << 20
        out, err = call(tb=bad)
        assert err == (2, 1) and torch.equal(out[: ofs[1]], good[: ofs[1]])
        for ln in ([50, 400, 40], [50, 33, 50000]):
            out, err = call(ln=ln)
            assert err[0] in (2, 4) and torch.equal(out[: ofs[1]], good[: ofs[1]])
            pk.pk_get_device_error()
        out, err = call(ln=[50, 33, cs[2] - 1])
        assert err == (4, 2) and (out[ofs[2]: ofs[3]] == 0).all() and torch.equal(out[: ofs[2]], good[: ofs[2]])
        for of in ([0, ofs[1], ofs[3] + 9, ofs[3]], [0, ofs[1], ofs[1] - 1, ofs[3]], [-1, ofs[1], ofs[2], ofs[3]]):
            out, err = call(of=of)
            assert err[0] == 8
            pk.pk_get_device_error()
        if max(cs) > 1:
            out, err = call(most=max(cs) - 1)
            assert err == (8, 0) and (out[: ofs[1]] == 7).all() and torch.equal(out[ofs[1]: ofs[3]], good[ofs[1]: ofs[3]])
        p, it = pk.pk_extend_plan(lens, cs, 4, pk.cache_desc(k), 0)
        for col, val in ((0, 3), (0, -1), (1, -4), (2, 0), (2, 10000), (3, 1), (3, -1)):
            wrong = it.copy()
            wrong[0, col] = val
            out, err = call(items=torch.from_numpy(wrong).to(DEV))
            assert err == (6, 0)


def test_extend_two_streams_and_a_replayed_graph():
    """Two calls at once with a workspace each, one captured and replayed with other inputs and lengths."""
    rng = np.random.default_rng(21)
    B, hq, hk, d = 16, 8, 2, 128
    counts, lens = [60, 1, 200], [900, 1200, 200]
    a = make_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, "cap window")
    b = make_case(rng, [1, 1, 1], lens, B, hq, hk, d, torch.bfloat16, "slopes")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    calls = []
    for (tables, k, v, ofs, q, sc), cs in ((a, counts), (b, [1, 1, 1])):
        part, items = pk.pk_extend_plan(lens, cs, hq, pk.cache_desc(k), 256)
        ws = torch.empty(pk.pk_extend_workspace_size(len(q), hq, 1200, part, pk.cache_desc(k)), dtype=torch.uint8,
                         device=DEV)
        out = torch.full_like(q, 7.0)
        args = (out, q, k, v, i32(tables), i32(lens), i32(ofs), d ** -0.5, max(cs), 1200)
        kw = dict(on_device(sc), partition_size=part, workspace=ws, work_items=torch.from_numpy(items).to(DEV))
        calls.append((args, kw))
    torch.cuda.synchronize()
    for _ in range(5):
        for (args, kw), st in zip(calls, (s1, s2)):
            pk.pk_paged_attention_extend(*args, stream=st, **kw)
    torch.cuda.synchronize()
    check_extend(calls[0][0][0], a[4], a[1], a[2], a[0], lens, d ** -0.5, a[3], a[5])
    check_extend(calls[1][0][0], b[4], b[1], b[2], b[0], lens, d ** -0.5, b[3], b[5])
    g = torch.cuda.CUDAGraph()
    args, kw = calls[0]
    with torch.cuda.graph(g):
        pk.pk_paged_attention_extend(*args, **kw)
    new = [850, 1100, 200]
    args[1].copy_(rand(rng, args[1].shape, torch.bfloat16))
    args[5].copy_(i32(new))
    args[0].fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    check_extend(args[0], args[1], a[1], a[2], a[0], new, d ** -0.5, a[3], a[5])


def test_extend_repeats_bit_for_bit():
    rng = np.random.default_rng(8)
    counts, lens = [300, 17, 1], [700, 1300, 900]
    case = make_case(rng, counts, lens, 16, 8, 2, 128, torch.bfloat16, "all")
    for part in (0, 256):
        first = run_extend(case, lens, counts, 0.1, part)
        for _ in range(10):
            assert torch.equal(run_extend(case, lens, counts, 0.1, part), first)


def test_extend_is_the_decode_attention_without_changes():
    """One new token and no changes: what pk_paged_attention_decode computes."""
    rng = np.random.default_rng(30)
    lens, B, hq, hk, d = [77, 1024, 5, 300], 16, 8, 2, 128
    tables, k, v, ofs, q, sc = make_case(rng, [1] * 4, lens, B, hq, hk, d, torch.bfloat16, "plain", pad=0)
    out, want = torch.empty_like(q), torch.empty_like(q)
    pk.pk_paged_attention_extend(out, q, k, v, i32(tables), i32(lens), None, d ** -0.5, 1, 1024)
    pk.pk_paged_attention_decode(want, q, k, v, i32(tables), i32(lens), d ** -0.5, 1024, partition_size=0)
    check_extend(out, q, k, v, tables, lens, d ** -0.5, None, sc)
    check_extend(want, q, k, v, tables, lens, d ** -0.5, None, sc)


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------
def make_drafts(rng, counts, V, dt, mask, pad=2, stride=None):
    ofs = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(ofs[-1]) + pad
    logits = rng.standard_normal((R, V)) * 3.0
    parents = np.zeros(R, np.int32)
    for s, n in enumerate(counts):
        for i in range(1, n):
            parents[ofs[s] + i] = i - 1 if mask != "tree" else rng.integers(max(0, i - 4), i)
    target = np.exp(logits - logits.max(1, keepdims=True))
    target /= target.sum(1, keepdims=True)
    tokens = np.zeros(R, np.int64)
    draft = None
    if mask == "chain":
        draft = np.zeros_like(target)
    for s, n in enumerate(counts):
        for i in range(1, n):
            r, up = ofs[s] + i, ofs[s] + parents[ofs[s] + i]
            if mask == "chain":
                x = logits[up] + rng.standard_normal(V)
                draft[r] = np.exp(x - x.max()) / np.exp(x - x.max()).sum()
                tokens[r] = rng.choice(V, p=draft[r])
            else:
                tokens[r] = rng.choice(np.argsort(-target[up])[:3])

    def device(x):
        t = torch.from_numpy(x.astype(np.float32)).to(DEV).to(dt)
        if stride:
            wide = torch.full((R, stride), 0.5, dtype=dt, device=DEV)
            wide[:, :V] = t
            t = wide[:, :V]
        return t

    u = rng.random(R).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    return ofs, device(target), tokens, u, (parents if mask == "tree" else None), (None if draft is None else device(draft))


def run_verify(ofs, target, tokens, u, parents, draft, most=64, **kw):
    S, R = len(ofs) - 1, len(tokens)
    na, nt = torch.full((S,), -7, dtype=torch.int32, device=DEV), torch.full((S,), -7, dtype=torch.int64, device=DEV)
    ac = torch.full((R,), -7, dtype=torch.int32, device=DEV)
    pk.pk_verify_drafts(na, ac, nt, target, i64(tokens), torch.from_numpy(u).to(DEV), i32(ofs), most,
                        parents=None if parents is None else i32(parents), draft_probs=draft, **kw)
    return na, ac, nt


def check_verify(got, ofs, target, tokens, u, parents, draft):
    na, ac, nt = (x.cpu().numpy() for x in got)
    counts, paths, nexts = plain.verify_drafts(f64(target), tokens, u, ofs, parents, None if draft is None else f64(draft))
    want = np.full(len(tokens), -7)
    for s, path in enumerate(paths):
        want[ofs[s]:ofs[s + 1]] = -1
        want[ofs[s]:ofs[s] + len(path)] = path
    assert na.tolist() == counts and nt.tolist() == nexts and ac.tolist() == want.tolist()
    return counts


@pytest.mark.parametrize("mask", ["chain", "greedy", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,stride", [(1, None), (7, None), (1000, 1024), (32000, None), (50257, None), (50257, 50304),
                                      (4099, 4101)])
def test_verify(mask, dtype, V, stride):
    rng = np.random.default_rng(V)
    counts = [1, 5, 0, 9, 2, 4] if V > 10000 else [1, 5, 0, 64, 2, 33, 17, 3, 3, 3, 3, 3]
    if V < 4 and mask != "chain":
        counts = [min(c, 3) for c in counts]
    for seed in range(3):
        case = make_drafts(rng, counts, V, DTYPES[dtype], mask, stride=stride)
        check_verify(run_verify(*case), *case)


def test_verify_accepts_and_refuses_at_every_place():
    """Random numbers at 0 and next to 1: everything accepted, or (of a chain of unlikely tokens) nothing."""
    rng = np.random.default_rng(2)
    for mask in ("chain", "greedy"):
        ofs, target, tokens, u, parents, draft = make_drafts(rng, [8] * 6, 500, torch.float32, mask)
        zero, one = np.zeros_like(u), np.full_like(u, 1 - 2.0 ** -24)
        assert check_verify(run_verify(ofs, target, tokens, zero, parents, draft), ofs, target, tokens, zero, parents,
                            draft) == [7] * 6
        check_verify(run_verify(ofs, target, tokens, one, parents, draft), ofs, target, tokens, one, parents, draft)
        if draft is not None:  # drafts that are the target's: accepted whatever the numbers
            draft[1:] = target[:-1]
            assert check_verify(run_verify(ofs, target, tokens, one, parents, draft), ofs, target, tokens, one, parents,
                                draft) == [7] * 6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_borders(dtype):
    """Values whose sums and products are exact: numbers on a border, siblings of one token, all of the
    weight refused, rows without weight, and what is not a probability."""
    dt = DTYPES[dtype]
    V = 4096
    p = np.zeros((6, V))
    p[0, [5, 9, 4000]] = [0.25, 0.25, 0.5]
    p[1, 17] = 1.0
    p[2] = 1.0 / V
    p[3, [1, 2]] = [0.5, 0.5]
    ofs = np.array([0, 3, 6], np.int32)
    t = torch.from_numpy(p.astype(np.float32)).to(DEV).to(dt)
    tokens = np.array([0, 9, 9, 0, 17, 1])
    for parents in (np.zeros(6, np.int32), np.array([0, 0, 1, 0, 0, 0], np.int32)):
        for u0 in (0.0, 0.25, 0.5, 0.49999997, 0.75, 0.99999994):
            for u1 in (0.0, 0.25, 0.24999999, 0.9):
                u = np.array([u0, u1, u0, u1, u0, u1], np.float32)
                check_verify(run_verify(ofs, t, tokens, u, parents, None, most=3), ofs, t, tokens, u, parents, None)
    # The draft's distribution above the target's everywhere: the row itself is drawn from.
    q = torch.ones_like(t)
    u = np.array([0.6, 0.9, 0.9, 0.3, 0.9, 0.9], np.float32)
    check_verify(run_verify(ofs, t, tokens, u, None, q, most=3), ofs, t, tokens, u, None, q)
    # NaN, negative and infinite entries count as nothing, a row of them as no weight.
    t[0, :9] = float("nan")
    t[0, 100:200] = -1.0
    t[0, 300] = float("inf")
    t[3] = float("nan")
    q[1, 4000] = float("nan")
    for draft in (None, q):
        got = run_verify(ofs, t, tokens, u, None, draft, most=3)
        check_verify(got, ofs, t, tokens, u, None, draft)
        assert int(got[2][1]) == -1


def test_verify_bad_inputs_are_recorded():
    rng = np.random.default_rng(3)
    ofs, target, tokens, u, parents, _ = make_drafts(rng, [4, 5, 3], 300, torch.float32, "tree")
    good = run_verify(ofs, target, tokens, u, parents, None)
    for bad in (-1, 300, 1 << 40):
        wrong = tokens.copy()
        wrong[5] = bad
        got = run_verify(ofs, target, wrong, u, parents, None)
        assert pk.pk_get_device_error() == (9, 1)
        check_verify(got, ofs, target, wrong, u, parents, None)
    for bad in (-1, 2, 100):
        wrong = parents.copy()
        wrong[5 + 1] = bad
        got = run_verify(ofs, target, tokens, u, wrong, None)
        assert pk.pk_get_device_error() == (9, 1)
        assert torch.equal(got[0][::2], good[0][::2]) and torch.equal(got[2][::2], good[2][::2])
    for of, at in (([0, 4, 99, 12], (1, 2)), ([0, 4, 3, 12], (1,)), ([-1, 4, 9, 12], (0,))):
        got = run_verify(np.array(of), target, tokens, u, parents, None)
        assert pk.pk_get_device_error()[0] == 8
        for s in at:
            assert int(got[0][s]) == 0 and int(got[2][s]) == -1
        pk.pk_get_device_error()
    got = run_verify(ofs, target, tokens, u, parents, None, most=4)
    assert pk.pk_get_device_error() == (8, 1) and int(got[2][1]) == -1 and int(got[2][0]) == int(good[2][0])


def test_verify_distribution():
    """Over many draws the kept and drawn tokens are distributed as the target's: frequencies of the
    first new token within five standard deviations."""
    rng = np.random.default_rng(12)
    V, S = 8, 20000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target = np.tile(p, (2 * S, 1)).astype(np.float32)
    draft = np.tile(q, (2 * S, 1)).astype(np.float32)
    tokens = rng.choice(V, 2 * S, p=q)
    u = np.minimum(rng.random(2 * S).astype(np.float32), np.float32(1 - 2.0 ** -24))
    ofs = np.arange(0, 2 * S + 1, 2).astype(np.int32)
    na, ac, nt = run_verify(ofs, torch.from_numpy(target).to(DEV), tokens, u, None, torch.from_numpy(draft).to(DEV), most=2)
    first = np.where(na.cpu().numpy() == 1, tokens[1::2], nt.cpu().numpy())
    f = np.bincount(first, minlength=V) / S
    assert (np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / S)).all()


# ---------------------------------------------------------------------------
# Compaction
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hk,d,B", [(1, 64, 16), (8, 128, 16), (2, 80, 5), (3, 256, 8), (4, 128, 1)])
def test_compact(dtype, hk, d, B):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(hk * d)
    counts = [1, 64, 0, 17, 2, 33, 5]
    lens = [40, 64, 12, 100, 2, 500, 70]
    tables, k, v, ofs, q, _ = make_case(rng, counts, lens, B, hk, hk, 64, dt, "plain")
    k, v = rand(rng, (len(k), B, hk, d), dt), rand(rng, (len(k), B, hk, d), dt)
    for trial in range(4):
        paths = []
        for n in counts:
            if trial == 0:
                path = list(range(n))
            elif trial == 1:
                path = [0] if n else []
            else:
                path = [0] + sorted((1 + rng.permutation(n - 1)[: int(rng.integers(0, n))]).tolist()) if n else []
            if trial == 3 and n > 1:
                path = sorted(rng.permutation(n)[: int(rng.integers(1, n))].tolist())  # without the root
            paths.append(path)
        accepted = np.full(int(ofs[-1]) + 3, -1, np.int32)
        for s, path in enumerate(paths):
            accepted[ofs[s]:ofs[s] + len(path)] = path
        na = [max(len(x) - 1, 0) for x in paths]
        kk, vv, lo = k.clone(), v.clone(), i32([-5] * len(lens))
        pk.pk_compact_drafts(kk, vv, i32(tables), i32(lens), i32(ofs), i32(accepted), i32(na), 64, context_lens_out=lo)
        wk, wv = f64(k), f64(v)
        left = plain.compact_drafts(wk, tables, lens, ofs, paths)
        plain.compact_drafts(wv, tables, lens, ofs, paths)
        assert (f64(kk) == wk).all() and (f64(vv) == wv).all() and lo.tolist() == left
        k2, v2 = k.clone(), v.clone()
        pk.pk_compact_drafts(k2, v2, i32(tables), i32(lens), i32(ofs), i32(accepted), i32(na), 64)
        assert torch.equal(k2, kk) and torch.equal(v2, vv)


def test_compact_bad_inputs_are_recorded():
    rng = np.random.default_rng(4)
    counts, lens, B = [6, 5, 4], [30, 40, 20], 8
    tables, k, v, ofs, q, _ = make_case(rng, counts, lens, B, 2, 2, 64, torch.float32, "plain")
    good = np.array([0, 2, 5, -1, -1, -1, 0, 3, 4, -1, -1, 1, 3, -1, -1, -1, -1, -1], np.int32)

    def call(ac=good, na=(2, 2, 1), ln=lens, of=ofs, tb=tables, most=6):
        kk, vv, lo = k.clone(), v.clone(), i32([-5] * 3)
        pk.pk_compact_drafts(kk, vv, i32(tb), i32(ln), i32(of), i32(ac), i32(na), most, context_lens_out=lo)
        return kk, lo.tolist(), pk.pk_get_device_error()

    want, left, err = call()
    assert err == (0, 0) and left == [27, 38, 18]

    def others(kk, s):  # the blocks of the other sequences are as they should be
        for o in range(3):
            rows = tables[o][tables[o] >= 0]
            assert torch.equal(kk[rows], (k if o == s else want)[rows])

    for change in ({7: 0}, {7: 5}, {7: -1}, {8: 3}, {8: 2}):
        ac = good.copy()
        for i, x in change.items():
            ac[i] = x
        kk, lo, err = call(ac=ac)
        assert err == (9, 1) and lo == [27, 40, 18]
        others(kk, 1)
    for n in (-2, 5, 1 << 30):
        kk, lo, err = call(na=(2, n, 1))
        assert err == (9, 1) and lo == [27, 40, 18]
        others(kk, 1)
    for n in (4, 100000):
        kk, lo, err = call(ln=[30, n, 20])
        assert err == (4, 1) and lo == [27, n, 18]
        others(kk, 1)
    kk, lo, err = call(of=[0, 6, 99, 15])
    assert err[0] == 8 and lo[0] == 27 and lo[1] == 40
    pk.pk_get_device_error()
    kk, lo, err = call(most=5)
    assert err == (8, 0) and lo == [30, 38, 18]
    others(kk, 0)
    bad = tables.copy()
    bad[1, 4] = -3  # the block of tokens 32 .. 39
    kk, lo, err = call(tb=bad)
    assert err == (2, 1) and lo == [27, 38, 18]
    others(kk, 1)


def test_verification_and_compaction_in_a_replayed_graph():
    """The two captured one after the other and replayed with other numbers, drafts and lengths."""
    rng = np.random.default_rng(50)
    B, hk, d, V, counts, lens = 8, 2, 64, 2000, [6, 9, 1, 4], [30, 40, 20, 55]
    tables, k, v, ofs, q, _ = make_case(rng, counts, lens, B, hk, hk, d, torch.bfloat16, "plain", pad=0)
    _, target, tokens, u, parents, _ = make_drafts(rng, counts, V, torch.float32, "tree", pad=0)
    dev = dict(tokens=i64(tokens), u=torch.from_numpy(u).to(DEV), parents=i32(parents), lens=i32(lens), ofs=i32(ofs),
               tables=i32(tables), na=i32([0] * 4), ac=i32([0] * 20), nt=i64([0] * 4), left=i32([0] * 4))

    def run():
        pk.pk_verify_drafts(dev["na"], dev["ac"], dev["nt"], target, dev["tokens"], dev["u"], dev["ofs"], 9,
                            parents=dev["parents"])
        pk.pk_compact_drafts(k, v, dev["tables"], dev["lens"], dev["ofs"], dev["ac"], dev["na"], 9,
                             context_lens_out=dev["left"])

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for trial in range(3):
        _, t2, tokens, u, parents, _ = make_drafts(rng, counts, V, torch.float32, "tree", pad=0)
        target.copy_(t2)
        lens = [int(n - rng.integers(0, 10)) for n in (30, 40, 20, 55)]
        for name, x in (("tokens", i64(tokens)), ("u", torch.from_numpy(u).to(DEV)), ("parents", i32(parents)), ("lens", i32(lens))):
            dev[name].copy_(x)
        wk, wv = f64(k), f64(v)
        g.replay()
        torch.cuda.synchronize()
        check_verify((dev["na"], dev["ac"], dev["nt"]), ofs, target, tokens, u, parents, None)
        _, paths, _ = plain.verify_drafts(f64(target), tokens, u, ofs, parents)
        left = plain.compact_drafts(wk, tables, lens, ofs, paths)
        plain.compact_drafts(wv, tables, lens, ofs, paths)
        assert dev["left"].tolist() == left and (f64(k) == wk).all() and (f64(v) == wv).all()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def test_prompt_drafts_verification_and_the_next_step():
    """A prompt written and attended to; drafts appended as a tree, attended to, verified, compacted, the
    sequences cut; then a decoded token attends to the cache as if the kept tokens had been all along."""
    rng = np.random.default_rng(40)
    B, hq, hk, d, V, dt = 16, 8, 2, 128, 512, torch.bfloat16
    S, prompt, n = 3, [70, 33, 140], 8
    bm = pk.BlockManager(64, B)
    kc, vc = (torch.zeros((64, B, hk, d), dtype=dt, device=DEV) for _ in range(2))
    scale, cap = d ** -0.5, 20.0
    stored = [([], []) for _ in range(S)]

    def append(counts):
        slots, ks, vs = [], [], []
        for s, c in enumerate(counts):
            sl, pair = bm.append(s, c)
            assert pair is None
            slots.append(sl)
            ks.append(rand(rng, (c, hk, d), dt))
            vs.append(rand(rng, (c, hk, d), dt))
        pk.pk_reshape_and_cache(torch.cat(ks), torch.cat(vs), i64(np.concatenate(slots)), kc, vc)
        for s in range(S):
            stored[s][0].append(ks[s])
            stored[s][1].append(vs[s])

    def attend(counts):
        ofs = np.concatenate([[0], np.cumsum(counts)])
        tables, ln = bm.export_tables(range(S), 16)
        q = rand(rng, (int(ofs[-1]), hq, d), dt)
        out = torch.full_like(q, 7.0)
        part, items = pk.pk_extend_plan(ln, counts, hq, pk.cache_desc(kc), -1)
        pk.pk_paged_attention_extend(out, q, kc, vc, i32(tables), i32(ln), i32(ofs), scale, max(counts), int(ln.max()),
                                     softcap=cap, partition_size=part, work_items=torch.from_numpy(items).to(DEV))
        # The same over a cache of one block per token, laid out from what was stored.
        keys = torch.cat([torch.cat(x[0]) for x in stored])[:, None]
        vals = torch.cat([torch.cat(x[1]) for x in stored])[:, None]
        starts = np.concatenate([[0], np.cumsum(ln)])
        flat = np.full((S, int(ln.max())), -1)
        for s in range(S):
            flat[s, : ln[s]] = np.arange(starts[s], starts[s + 1])
        check_extend(out, q, keys, vals, flat, ln, scale, ofs, {"softcap": cap})

    for s in range(S):
        bm.add_seq(s)
    append(prompt)
    attend(prompt)
    for _ in range(3):
        append([n] * S)  # the root and seven drafts
        tables, ln = bm.export_tables(range(S), 16)
        ofs, target, tokens, u, parents, _ = make_drafts(rng, [n] * S, V, torch.float32, "tree", pad=0)
        masks = np.concatenate([pk.pk_tree_masks([-1] + parents[ofs[s] + 1: ofs[s + 1]].tolist())[0] for s in range(S)])
        q, out = rand(rng, (n * S, hq, d), dt), torch.empty((n * S, hq, d), dtype=dt, device=DEV)
        pk.pk_paged_attention_tree(out, q, kc, vc, i32(tables), i32(ln), i32(ofs), scale, n, int(ln.max()),
                                   tree_mask=i64(masks))
        got = run_verify(ofs, target, tokens, u, parents, None, most=n)
        check_verify(got, ofs, target, tokens, u, parents, None)
        left = torch.empty(S, dtype=torch.int32, device=DEV)
        pk.pk_compact_drafts(kc, vc, i32(tables), i32(ln), i32(ofs), got[1], got[0], n, context_lens_out=left)
        ac = got[1].cpu().numpy()
        for s, m in enumerate(left.tolist()):
            bm.truncate(s, m)
            for side in (0, 1):
                rows = torch.cat(stored[s][side])
                base = len(rows) - n
                path = ac[ofs[s]: ofs[s + 1]]
                keep = base + path[path >= 0]
                stored[s][side][:] = [rows[:base], rows[torch.from_numpy(keep).to(DEV)]]
            assert m == sum(len(x) for x in stored[s][0])
        bm.check_invariants()
        append([1] * S)
        attend([1] * S)
        append([3, 1, 20])  # a chunk
        attend([3, 1, 20])

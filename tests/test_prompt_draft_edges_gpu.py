"""Edges of prompt attention, draft verification and cache compaction on the GPU: what the calls are
followed by, sizes and values at the ends of their ranges, and bounds tighter than those of the general tests."""
import math

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk

torch = pytest.importorskip("torch")
import test_prompt_draft_ops_gpu as ops  # noqa: E402

pytestmark = pytest.mark.gpu
DEV, U = ops.DEV, ops.U


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


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,counts", [("bf16", [600, 150, 1, 40]), ("bf16", [1, 1, 1, 1]), ("f32", [60, 15, 1, 4])])
def test_extend_split_call_is_over_when_what_follows_it_starts(dtype, counts):
    """A split call of which no row lies in two partitions, so that the merge has no row to write, then a copy of
    the result: captured together and replayed, the copy is the result every time."""
    rng = np.random.default_rng(60)
    B, hq, hk, d, dt = 16, 8, 2, 128, ops.DTYPES[dtype]
    lens, part = [2040, 900, 700, 1500], 512
    tables, k, v, ofs, q, sc = ops.make_case(rng, counts, lens, B, hq, hk, d, dt, "plain")
    # Documents that end where partitions do, a new one at every multiple of 128 within them.
    sc["first_tokens"] = np.zeros(len(q), np.int32)
    for s, (c, n) in enumerate(zip(counts, lens)):
        pos = np.arange(n - c, n)
        sc["first_tokens"][ofs[s]: ofs[s + 1]] = pos // 128 * 128
    want = ops.run_extend((tables, k, v, ofs, q, sc), lens, counts, d ** -0.5)
    ops.check_extend(want, q, k, v, tables, lens, d ** -0.5, ofs, sc)
    desc = pk.cache_desc(k)
    part, items = pk.pk_extend_plan(lens, counts, hq, desc, part)
    assert part == 512
    ws = torch.zeros(pk.pk_extend_workspace_size(len(q), hq, max(lens), part, desc), dtype=torch.uint8, device=DEV)
    out, copy = torch.full_like(q, 7.0), torch.empty_like(q)
    args = (out, q, k, v, ops.i32(tables), ops.i32(lens), ops.i32(ofs), d ** -0.5, max(counts), max(lens))
    kw = dict(ops.on_device(sc), partition_size=part, workspace=ws, work_items=torch.from_numpy(items).to(DEV))
    pk.pk_paged_attention_extend(*args, **kw)
    torch.cuda.synchronize()
    split = out.clone()  # (of other tiles than the whole call, so not its bits)
    ops.check_extend(split, q, k, v, tables, lens, d ** -0.5, ofs, sc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.fill_(7.0)
        pk.pk_paged_attention_extend(*args, **kw)
        copy.copy_(out)
        out.fill_(-3.0)
    for _ in range(200):
        copy.zero_()
        g.replay()
        assert torch.equal(copy, split)
    assert bool((out == -3.0).all())


@pytest.mark.parametrize("hq,hk,d,B", [(8, 2, 128, 16), (4, 1, 64, 8), (3, 1, 128, 32)])
def test_extend_few_rows_clear_hidden_values_in_places_that_are_filled_again(hq, hk, d, B):
    """Two new tokens, the first of which sees what the second does not, NaN and infinities in all of it: many
    tiles in turn are cleared and their places filled again. The second one's rows are bit for bit as without."""
    rng = np.random.default_rng(d + B)
    lens, counts = [2500, 1300, 700, 1999], [2, 2, 2, 2]
    tables, k, v, ofs, q, sc = ops.make_case(rng, counts, lens, B, hq, hk, d, torch.bfloat16, "plain", pad=0)
    sc["first_tokens"] = np.stack([np.zeros(4), np.array(lens) - 300], 1).astype(np.int32).reshape(-1)
    bad = v.clone()
    for s, n in enumerate(lens):
        t = np.arange(n - 300)
        at = ops.i64(tables[s][t // B]), ops.i64(t % B)
        x = bad[at]
        x[torch.rand(x.shape, device=DEV) < 0.3] = float("nan")
        x[torch.rand(x.shape, device=DEV) < 0.3] = float("-inf")
        bad[at] = x
    for part in (0, 512):
        want = ops.run_extend((tables, k, v, ofs, q, sc), lens, counts, d ** -0.5, part)
        ops.check_extend(want, q, k, v, tables, lens, d ** -0.5, ofs, sc)
        for _ in range(20):
            out = ops.run_extend((tables, k, bad, ofs, q, sc), lens, counts, d ** -0.5, part)
            assert torch.equal(out[1::2], want[1::2])
            assert not bool(torch.isfinite(out[::2]).any())


def dense(q, k, v, tables, lens, counts, ofs, scale, sc, rho, T, A=0.0):
    """The definition in fp64 on the GPU, a sequence and head at a time, and its bound: the general tests'
    with the cap's error relative to the capped score, not to the cap,
    e_t = D m_t + (T + 6 u) (|x_t| + |capped x_t| + |bias_t|) log2(e) + A cap log2(e),
    T being tanh's own relative error: 2^-22 of tanhf, 2^-17 of bf16's (2^-17.3 of the shortest polynomial,
    2^-20.6 of the longer one; an exponential and a reciprocal are off by 2^-21 where tanh is above 0.6),
    A that of prompts of bf16 with caps of at most 88, 2^-21 (the exponential alone);
    six roundings: the product by its factor, the tanh's argument, by the cap, bias twice, the maximum's.
    Where e_t is above 1/2 for a token seen, exp is no longer close to linear and the bound is the values' range."""
    R, hq, d = q.shape
    B, hk = k.shape[1], k.shape[2]
    out, tol = (torch.zeros((R, hq, d), dtype=torch.float64, device=DEV) for _ in range(2))
    D, cap, log2e, eta = (d + 8) * 2 * U, sc.get("softcap", 0.0), 1 / ops.LN2, ops.ETA[q.dtype]
    for s, (n, c) in enumerate(zip(lens, counts)):
        blocks = ops.i64(tables[s][: -(-n // B)])
        kk, vv = (x[blocks].reshape(-1, hk, d)[:n].double() for x in (k, v))
        pos, t = torch.arange(n - c, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        see = t <= pos
        if sc.get("window"):
            see = see & (t > pos - sc["window"])
        for h in range(hq):
            qh, kh, vh = q[ofs[s]: ofs[s + 1], h].double(), kk[:, h * hk // hq], vv[:, h * hk // hq]
            x, m = qh @ kh.T * scale, qh.abs() @ kh.abs().T * abs(scale) * log2e
            a = x.abs()
            if cap:
                x = torch.tanh(x / cap) * cap
                a = a + x.abs()
            if "slopes" in sc:
                far = (pos - t).abs() * float(sc["slopes"][h])
                x, a = x - far, a + far
            w = torch.softmax(x.masked_fill(~see, -float("inf")), 1).nan_to_num(0.0)
            e = D * m + ((T + 6 * U) * a + A * cap) * log2e
            o, we = w @ vh, w * e
            x = 2 * ops.LN2 * (we @ vh.abs() + o.abs() * we.sum(1, keepdim=True)) + (
                16 * U + 2 * rho + 4 * U * n) * (w @ vh.abs()) + eta * o.abs() + 1e-30
            wild = (e.masked_fill(~see, 0.0).amax(1) > 0.5)[:, None]
            out[ofs[s]: ofs[s + 1], h] = o
            tol[ofs[s]: ofs[s + 1], h] = torch.where(wild, 2.1 * vh.abs().amax(), x)
    return out, tol


def check_dense(out, *args):
    want, tol = dense(*args)
    ofs = args[6]
    bad = ~((out.double() - want).abs() <= tol)
    bad[int(ofs[-1]):] = False
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), out[bad][:4], want[bad][:4], tol[bad][:4])


PATHS = {  # type, block size, new tokens, context lengths
    "few": ("bf16", 16, [1, 1, 2], [300, 1000, 77]),
    "prompt": ("bf16", 16, [300, 40, 1], [300, 700, 90]),
    "other blocks": ("bf16", 12, [60, 3], [60, 200]),
    "f32": ("f32", 16, [60, 1], [60, 300]),
    "f32 few": ("f32", 16, [1, 1], [100, 300]),
}
# A weight as the product takes it: a bf16 pair, one bf16, 24 bits.
RHO = {"few": 2.0 ** -17, "prompt": 2.0 ** -8, "other blocks": 2.0 ** -17, "f32": U, "f32 few": U}


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("scale", [1e7, 1e9, -1e9, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("kind", ["plain", "slopes", "window"])
def test_extend_scores_far_above_one(path, scale, kind):
    """Scores of 10^7 and more, where an fp32 score is known to hundreds or worse: finite results within the
    values' range, and of rows that see one token that token's value."""
    dtype, B, counts, lens = PATHS[path]
    rng = np.random.default_rng(len(path))
    hq, hk, d = 4, 2, 128
    tables, k, v, ofs, q, sc = ops.make_case(rng, counts, lens, B, hq, hk, d, ops.DTYPES[dtype], kind)
    for part in (0, 4 * B):
        out = ops.run_extend((tables, k, v, ofs, q, sc), lens, counts, scale, part)
        check_dense(out, q, k, v, tables, lens, counts, ofs, scale, sc, RHO[path], 2.0 ** -17)


@pytest.mark.parametrize("path", sorted(PATHS))
@pytest.mark.parametrize("cap", [2.0 ** -90, 1e-8, 1e-4, 0.5, 20.0, 80.0, 100.0, 1e3, 1e4, 1e6, 1e20])
@pytest.mark.parametrize("kind", ["plain", "slopes", "window"])
def test_extend_cap_of_every_size(path, cap, kind):
    """A cap far above the scores changes nothing, whatever its size, in rows whose neighbours' scores reach it
    too; one far below them leaves nearly equal weights."""
    dtype, B, counts, lens = PATHS[path]
    hq, hk, d = 4, 2, 128
    rng = np.random.default_rng(len(path) + len(kind))
    tables, k, v, ofs, q, sc = ops.make_case(rng, counts, lens, B, hq, hk, d, ops.DTYPES[dtype], kind)
    sc["softcap"] = cap
    T = 2.0 ** -22 if dtype == "f32" else 2.0 ** -17
    for big in (1.0, max(1.0, cap / 2)):
        x = q.clone()
        x[1::7, 1] *= big  # scores of some rows of a head beyond the cap, among others
        out = ops.run_extend((tables, k, v, ofs, x, sc), lens, counts, d ** -0.5)
        check_dense(out, x, k, v, tables, lens, counts, ofs, d ** -0.5, sc, RHO[path], T,
                    2.0 ** -21 if path == "prompt" and cap <= 88 else 0.0)


@pytest.mark.parametrize("dtype,counts", [("bf16", [20, 3, 0, 9]), ("f32", [20, 3, 0, 9]), ("bf16", [1, 1, 0, 1])])
def test_extend_items_behind_their_sequences_rows_are_recorded(dtype, counts):
    """A first row at or past the sequence's rows, or any of a sequence without rows; the others are done."""
    rng = np.random.default_rng(70)
    lens, B, hq = [50, 33, 12, 40], 16, 4
    tables, k, v, ofs, q, sc = ops.make_case(rng, counts, lens, B, hq, 2, 64, ops.DTYPES[dtype], "plain")
    want = ops.run_extend((tables, k, v, ofs, q, sc), lens, counts, 0.125)
    part, items = pk.pk_extend_plan(lens, counts, hq, pk.cache_desc(k), 0)

    def call(extra, ofs=ofs):
        out = torch.full_like(q, 7.0)
        it = np.concatenate([items, np.array(extra, np.int32).reshape(-1, 4)])
        pk.pk_paged_attention_extend(out, q, k, v, ops.i32(tables), ops.i32(lens), ops.i32(ofs), 0.125, max(counts), 50,
                                     work_items=torch.from_numpy(it).to(DEV))
        return out, pk.pk_get_device_error()

    out, err = call([])
    assert err == (0, 0) and torch.equal(out, want)
    for s, r0 in ((0, 2 * counts[0]), (1, 2 * counts[1] + 5), (3, 2 ** 31 - 1), (2, 0), (2, 4)):
        out, err = call([s, r0, 2, 0])
        assert err == (6, len(items)) and torch.equal(out, want), (s, r0)
    # Bad offsets stay what is recorded.
    bad = ofs.copy()
    bad[1] = 1000
    assert call([], bad)[1][0] == 8


@pytest.mark.parametrize("path", ["few", "few of two tokens", "other blocks", "prompt", "f32"])
@pytest.mark.parametrize("part", [0, 96])
def test_extend_weights_have_the_bits_that_are_promised(path, part):
    """Weights whose roundings to one bf16 are as large as they get and of opposite sign, under values that nearly
    cancel: every 16 tokens hold two of score 0 and value 0, the others in turn weights a little above 0.501953,
    the middle of two bf16 (value 1, rounded up by 2^-8.1), and a little below (value -1, rounded down as much).
    |error| <= (2 rho + 16 u + 4 u T) W + 4 ln2 e + eta |out| as in the general tests, W = sum w |v| / sum w < 1,
    with scores that are exact but for factor and exponential: e <= 6 u |x|, |x| <= 1. One bf16 is off by
    2^-9, a pair must be by less than 2^-12; of prompts of bf16 one bf16 is promised."""
    dtype, B, n = {"few": ("bf16", 16, 1), "few of two tokens": ("bf16", 8, 2), "other blocks": ("bf16", 12, 30),
                   "prompt": ("bf16", 16, 60), "f32": ("f32", 16, 3)}[path]
    rho = {"prompt": 2.0 ** -8, "f32": U}.get(path, 2.0 ** -17)
    dt, d, T = ops.DTYPES[dtype], 64, 480
    x = np.where(np.arange(T) % 2 == 0, -1000.0, -1001.0)
    x[::16] = x[1::16] = 0.0
    scale = 0.9939 * math.log(2.0) / 1000
    keys, vals = np.zeros((T, 1, d)), np.zeros((T, 1, d))
    keys[:, 0, :4], keys[:, 0, 4] = (np.trunc(x / 8) * 2)[:, None], x - np.trunc(x / 8) * 8
    vals[:, 0] = np.where(x == 0.0, 0.0, np.where(x == -1000.0, 1.0, -1.0))[:, None]
    assert (torch.from_numpy(keys).to(dt).double().numpy() == keys).all() and (keys.sum(2)[:, 0] == x).all()
    N = -(-T // B)
    pools = []
    for y in (keys, vals):
        pool = np.zeros((N * B, 1, d))
        pool[:T] = y
        pools.append(torch.from_numpy(pool.reshape(N, B, 1, d)).to(DEV).to(dt))
    q = torch.ones((n, 2, d), dtype=dt, device=DEV)
    tables, ofs = np.arange(N, dtype=np.int32)[None], np.array([0, n], np.int32)
    out = ops.run_extend((tables, *pools, ofs, q, {"softcap": 0.0, "window": 0}), [T], [n], scale, part)
    for i in range(n):
        see = np.arange(T - n + i + 1)
        w = np.exp(x[see] * scale)
        want = w @ vals[see, 0, 0] / w.sum()
        W = w @ np.abs(vals[see, 0, 0]) / w.sum()
        tol = (2 * rho + 16 * U + 4 * U * T) * W + 4 * ops.LN2 * 6 * U + ops.ETA[dt] * abs(want)
        got = ops.f64(out[i])
        assert (np.abs(got - want) <= tol).all(), (i, got[0, 0], want, tol)
        if rho == 2.0 ** -17:  # (weights of one bf16 would not pass)
            short = torch.from_numpy(w).bfloat16().double().numpy()
            assert abs(short @ vals[see, 0, 0] / w.sum() - want) > 4 * tol


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("mask,V", [("chain", 50257), ("greedy", 50257), ("tree", 32000), ("chain", 9000)])
def test_verify_by_several_ctas_a_sequence_again_and_again(mask, V):
    """Few sequences, so that eight (of 9000 values two) CTAs share one, with roots alone, sequences without rows
    and bad ranges between them (whose CTAs leave before they meet): the same result every time."""
    rng = np.random.default_rng(V)
    counts = [1, 1, 6, 0, 3, 1, 2]
    ofs, target, tokens, u, parents, draft = ops.make_drafts(rng, counts, V, torch.float32, mask)
    case = (ofs, target, tokens, u, parents, draft)
    first = ops.run_verify(*case)
    ops.check_verify(first, *case)
    bad = ofs.copy()
    bad[4] = 99  # sequences 3 and 4 have no range
    args = [ops.i64(tokens), torch.from_numpy(u).to(DEV)]
    S, R = len(counts), len(tokens)
    for of in (ofs, bad):
        na, ac, nt = (torch.zeros(n, dtype=t, device=DEV) for n, t in ((S, torch.int32), (R, torch.int32), (S, torch.int64)))
        offsets, par = ops.i32(of), None if parents is None else ops.i32(parents)
        for _ in range(300):
            nt.fill_(-9)
            pk.pk_verify_drafts(na, ac, nt, target, *args, offsets, 64, parents=par, draft_probs=draft)
            good = [0, 1, 2, 5, 6] if of is bad else list(range(S))
            assert torch.equal(nt[good], first[2][good]) and torch.equal(na[good], first[0][good])
            if of is bad:
                assert nt[[3, 4]].tolist() == [-1, -1] and na[[3, 4]].tolist() == [0, 0]
        if of is bad:
            assert pk.pk_get_device_error()[0] == 8
            pk.pk_get_device_error()


def test_verify_draws_by_sums_of_long_rows():
    """Rows of 2^24 values, which a CTA sums alone (of 160 sequences): 32 768 values a thread. The first half are
    2^-24 each, whose sums are exact; in the second half all threads have the same values, of which float pairs
    that are not brought in order as they grow lose 2^-34. The whole is 1 + 2^-39, or 1 - 2^-39, so r times
    the whole lies just above a border of the first half, or below: next to none with an error above 2^-39."""
    V, S, n = 1 << 24, 160, 1 << 15
    y = np.random.default_rng(76).random(n)
    y = y * y
    y = y * y
    x = (y / (math.fsum(y.tolist()) * 512)).astype(np.float32)
    # A thread's values: four neighbours of every 128, of its warp's sixteenth.
    second = torch.from_numpy(x).to(DEV).view(1, n // 4, 1, 4).expand(8, n // 4, 32, 4).reshape(-1)
    first = torch.full((V // 2,), 2.0 ** -24, device=DEV)
    rest = 256 * math.fsum(x.tolist()) - 0.5
    k = np.random.default_rng(1).integers(V // 10, V // 2 - V // 16, S)  # r = k 2^-24
    u = (k * 2.0 ** -24).astype(np.float32)
    ofs, tokens = np.arange(S + 1, dtype=np.int32), np.zeros(S, np.int64)
    target = torch.empty((S, V), device=DEV)
    for more in (2.0 ** -39, -(2.0 ** -39)):
        first[-1] = 2.0 ** -24 - rest + more
        assert abs(math.fsum(x.tolist()) * 256 + (V // 2 - 1) * 2.0 ** -24 + float(first[-1]) - 1 - more) < 2.0 ** -46
        target.copy_(torch.cat([first, second]))
        na, ac, nt = ops.run_verify(ofs, target, tokens, u, None, None, most=1)
        # The tokens up to k - 1 weigh r: more than r times the whole, or the next is needed.
        assert nt.tolist() == (k if more > 0 else k - 1).tolist()
        assert na.tolist() == [0] * S and ac.tolist() == [0] * S


@pytest.mark.parametrize("shift", [-88, -40, 40, 126])
def test_verify_draws_by_weights_of_any_whole(shift):
    """The next token goes by shares: rows scaled by a power of two draw the same ones."""
    rng = np.random.default_rng(shift + 100)
    ofs, target, tokens, u, _, _ = ops.make_drafts(rng, [1] * 40, 5000, torch.float32, "greedy", pad=0)
    want = ops.run_verify(ofs, target, tokens, u, None, None, most=1)[2]
    assert int(want.min()) >= 0
    assert torch.equal(ops.run_verify(ofs, target * 2.0 ** shift, tokens, u, None, None, most=1)[2], want)


@pytest.mark.parametrize("kind", ["siblings", "siblings of one token", "two levels", "chain"])
def test_verify_distribution_of_trees(kind):
    """Over many draws what greedy drafts and the drawn token come to is distributed as the target's samples: the
    first new token, and of those that went on the second, within five standard deviations."""
    rng = np.random.default_rng(len(kind))
    V, S = 6, 30000
    p0, p1, p2 = rng.dirichlet(np.ones(V), 3)
    a, b, c = np.argsort(-p0)[:3]
    # Rows: the root and its nodes; each row's target is the distribution after its token.
    parents, toks, rows = {
        "siblings": ([0, 0, 0, 0], [0, a, b, c], [p0, p1, p2, p1]),
        "siblings of one token": ([0, 0, 0, 0], [0, a, a, b], [p0, p1, p1, p2]),
        "two levels": ([0, 0, 0, 1, 1, 2], [0, a, b, 0, 1, 2], [p0, p1, p2, p1, p2, p0]),
        "chain": (None, [0, a, 3], [p0, p1, p2]),
    }[kind]
    n = len(toks)
    target = torch.from_numpy(np.tile(np.array(rows), (S, 1)).astype(np.float32)).to(DEV)
    u = np.minimum(rng.random(n * S).astype(np.float32), np.float32(1 - 2.0 ** -24))
    ofs = np.arange(0, n * S + 1, n).astype(np.int32)
    na, ac, nt = (x.cpu().numpy() for x in ops.run_verify(ofs, target, np.tile(toks, S).astype(np.int64), u, None if parents is None else np.tile(
        parents, S).astype(np.int32), None, most=n))
    ac = ac.reshape(S, n)
    toks = np.array(toks)

    def close(drawn, p):
        f = np.bincount(drawn, minlength=V) / len(drawn)
        assert (np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / len(drawn)) + 1e-6).all(), (f, p)

    close(np.where(na >= 1, toks[ac[:, 1]], nt), p0)
    for node in range(1, n):  # behind a kept node
        on = (na >= 1) & (ac[:, 1] == node)
        if on.sum() > 1000:
            close(np.where(na[on] >= 2, toks[ac[on, 2 % n]], nt[on]), rows[node])

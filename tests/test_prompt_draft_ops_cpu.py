"""Prompt attention, draft verification and cache compaction on the CPU: the plain fp64
forms by hand, the planner, the block manager's cut, and every refusal before a launch."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from oracle import prompt_draft_ops as plain
from oracle import serving_ops

INV, UNS, WSP = pk.PK_ERR_INVALID_ARG, pk.PK_ERR_UNSUPPORTED, pk.PK_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    pk.build()
    return pk.lib()


@pytest.fixture(scope="module")
def ptr():
    buf = np.zeros(1 << 16, np.uint8)
    yield (buf.ctypes.data + 255) // 256 * 256
    del buf


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def test_extend_attention_by_hand():
    """Two new tokens after one, one head of one element: softmax weights written out."""
    k = np.array([1.0, 2.0, 4.0]).reshape(3, 1, 1, 1)
    v = np.array([10.0, 20.0, 40.0]).reshape(3, 1, 1, 1)
    tables, q = [[0, 1, 2]], np.array([0.5, 0.25]).reshape(2, 1, 1)
    e = np.exp

    def out(**kw):
        return plain.extend_attention(q, k, v, tables, [3], 2.0, [0, 2], **kw)[0][:, 0, 0]

    def mean(x, values):
        return e(np.array(x)) @ values / e(np.array(x)).sum()

    a, b = out()
    assert np.isclose(a, mean([1, 2], [10, 20])) and np.isclose(b, mean([.5, 1, 2], [10, 20, 40]))
    a, b = out(window=1)
    assert (a, b) == (20, 40)
    a, b = out(prefix_lens=[3], first_tokens=[1, 2])
    assert np.isclose(a, mean([2, 4], [20, 40])) and b == 40
    a, b = out(softcap=3.0, slopes=[0.5], window=2)
    x = 3 * np.tanh(np.array([1, 2]) / 3) - [0.5, 0.0]
    assert np.isclose(a, mean(x, [10, 20])) and np.isclose(b, mean(x, [20, 40]))
    a, b = out(first_tokens=[5, 0])
    assert a == 0 and np.isclose(b, mean([.5, 1, 2], [10, 20, 40]))


@pytest.mark.parametrize("seed", range(3))
def test_extend_attention_is_the_tree_form_of_a_chain(seed):
    """Without score changes it is the attention of a chain of drafts (stated separately)."""
    rng = np.random.default_rng(seed)
    k, v = rng.standard_normal((2, 9, 4, 2, 8))
    lens, ofs = [7, 12, 3], [0, 3, 8, 8]
    tables = rng.permutation(9)[:6].reshape(3, 2)
    tables = np.concatenate([tables, [[6], [7], [8]]], 1)
    q = rng.standard_normal((8, 4, 8))
    got = plain.extend_attention(q, k, v, tables, lens, 0.3, ofs)[0]
    want = serving_ops.tree_attention(q, k, v, tables, lens, 0.3, ofs, None)[0]
    np.testing.assert_allclose(got, want, rtol=1e-13, atol=1e-13)


def test_verify_drafts_by_hand():
    p = np.array([[.5, .3, .2], [.1, .9, 0], [0, 0, 1.]])
    # A chain 0 -> token 1 -> token 0: u below and above p.
    assert plain.verify_drafts(p, [0, 1, 0], [.7, .29, .09], [0, 3]) == ([2], [[0, 1, 2]], [2])
    # The first refused: drawn from (.5, 0, .2): .7 (.5 + .2) = .49 < .5
    assert plain.verify_drafts(p, [0, 1, 0], [.7, .31, .09], [0, 3]) == ([0], [[0]], [0])
    assert plain.verify_drafts(p, [0, 1, 0], [.72, .31, .09], [0, 3]) == ([0], [[0]], [2])
    # Siblings: token 1 refused leaves .7; token 0 has .5 / .7.
    assert plain.verify_drafts(p, [0, 1, 0], [.0, .31, .70], [0, 3], parents=[0, 0, 0])[:2] == ([1], [[0, 2]])
    assert plain.verify_drafts(p, [0, 1, 0], [.0, .31, .72], [0, 3], parents=[0, 0, 0]) == ([0], [[0]], [2])
    # With the drafts' own distribution: accepted with p / q, else from max(p - q, 0).
    q = np.array([[1, 0, 0], [.2, .6, .2], [1, 0, 0.]])
    assert plain.verify_drafts(p, [0, 1, 0], [.5, .49, .05], [0, 3], draft=q) == ([2], [[0, 1, 2]], [2])
    assert plain.verify_drafts(p, [0, 1, 0], [.99, .51, .05], [0, 3], draft=q) == ([0], [[0]], [0])
    assert plain.verify_drafts(p, [0, 1, 0], [.5, .49, .1], [0, 3], draft=q) == ([1], [[0, 1]], [1])
    # No rows, and no weight.
    assert plain.verify_drafts(p * 0, [0, 0, 0], [0, 0, 0], [0, 0, 1]) == ([0, 0], [[], [0]], [-1, -1])


def test_compact_drafts_by_hand():
    pool = np.arange(12).reshape(4, 3)
    left = plain.compact_drafts(pool, [[3, 1, 0]], [8], [0, 5], [[0, 2, 4]])  # base 3: slots 1,0 1,1 1,2 0,0 0,1
    assert left == [6]
    assert pool.tolist() == [[0, 1, 2], [3, 5, 1], [6, 7, 8], [9, 10, 11]]


# ---------------------------------------------------------------------------
# Planner
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seed", range(12))
def test_plan_covers_every_row_and_partition_once(L, seed):
    rng = np.random.default_rng(seed)
    S, G, hk = int(rng.integers(1, 9)), int(rng.integers(1, 9)), int(rng.integers(1, 5))
    lens = rng.integers(1, 5000, S).astype(np.int32)
    new = None if seed % 4 == 0 else np.minimum(lens, rng.integers(0, 900, S)).astype(np.int32)
    d = pk.CacheDesc(100000, 16, hk, [64, 128][seed % 2], [pk.PK_F32, pk.PK_BF16][seed // 2 % 2])
    window = int(rng.integers(1, 2000)) if seed % 3 == 0 else 0
    for want in (-1, 0, 512):
        part, items = pk.pk_extend_plan(lens, new, G * hk, d, want, window=window)
        assert part % 16 == 0 and (want == -1 or part in (0, want))
        n = np.ones(S, int) if new is None else new
        seen = set()
        for s, r0, rows, p in items.tolist():
            assert rows >= 1 and r0 + rows <= n[s] * G
            for r in range(r0, r0 + rows):
                assert (s, r, p) not in seen
                seen.add((s, r, p))
        for s in range(S):
            for r in range(n[s] * G):
                pos = lens[s] - n[s] + r // G
                lo = max(0, pos - window + 1) if window else 0
                P = part or 1 << 30
                for p in range(lo // P, (lens[s] - 1) // P + 1):
                    assert (s, r, p) in seen
        ws = pk.pk_extend_workspace_size(int(n.sum()), G * hk, int(lens.max()), part, d)
        P = -(-int(lens.max()) // part) if part else 1
        assert ws == (0 if P <= 1 else int(n.sum()) * G * hk * P * (d.head_dim + 2) * 4)


def test_plan_refusals(L):
    d = pk.CacheDesc(64, 16, 2, 128, pk.PK_BF16)
    ref = ctypes.byref(d)
    lens, new, out = np.array([40, 9], np.int32), np.array([3, 9], np.int32), np.zeros((64, 4), np.int32)
    part, n = ctypes.c_int32(0), ctypes.c_int32(0)

    def plan(a=lens, b=new, S=2, most=9, hq=8, window=0, size=0, dd=ref, po=ctypes.byref(part), io=out, cap=64,
             no=ctypes.byref(n)):
        return L.pk_extend_plan(None if a is None else a.ctypes.data, None if b is None else b.ctypes.data, S, most,
                                hq, window, size, dd, po, None if io is None else io.ctypes.data, cap, no)

    assert plan() == pk.PK_OK and n.value >= 2
    for kw in (dict(a=None), dict(S=0), dict(most=8), dict(most=0), dict(window=-1), dict(size=-2), dict(size=24),
               dict(po=None), dict(no=None), dict(cap=1), dict(cap=-1), dict(io=None), dict(hq=7), dict(dd=None),
               dict(b=np.array([-1, 1], np.int32))):
        assert plan(**kw) == INV, kw
    assert plan(hq=18) == UNS
    bad = pk.CacheDesc(64, 16, 2, 96, pk.PK_BF16)
    assert plan(dd=ctypes.byref(bad)) == UNS
    assert pk.pk_extend_workspace_size(10, 8, 100, 0, d) == 0
    with pytest.raises(ValueError):
        pk.pk_extend_plan(lens, new[:1], 8, d)


# ---------------------------------------------------------------------------
# The block manager's cut
# ---------------------------------------------------------------------------
def test_truncate_frees_pages_behind_and_reuses_them_in_order():
    bm = pk.BlockManager(8, 4)
    bm.add_seq(1)
    bm.append(1, 14)
    assert bm.table(1).tolist() == [0, 1, 2, 3] and bm.num_free() == 4
    bm.truncate(1, 5)
    assert bm.table(1).tolist() == [0, 1] and bm.seq_len(1) == 5 and bm.num_free() == 6
    bm.check_invariants()
    slots, pair = bm.append(1, 9)
    assert pair is None and bm.table(1).tolist() == [0, 1, 2, 3] and slots.tolist() == list(range(5, 14))
    bm.truncate(1, 14)
    bm.truncate(1, 8)
    assert bm.table(1).tolist() == [0, 1]
    bm.truncate(1, 0)
    assert bm.table(1).tolist() == [] and bm.num_free() == 8 and bm.seq_len(1) == 0
    bm.append(1, 1)
    bm.check_invariants()


def test_truncate_refusals(L):
    bm = pk.BlockManager(4, 4)
    bm.add_seq(1)
    bm.append(1, 6)
    assert L.pk_bm_truncate(None, 1, 0) == INV
    assert L.pk_bm_truncate(bm._h, 2, 0) == pk.PK_ERR_UNKNOWN_SEQ
    assert L.pk_bm_truncate(bm._h, 1, 7) == INV and L.pk_bm_truncate(bm._h, 1, -1) == INV
    bm.set_swap_space(4)
    bm.swap_out(1)
    assert L.pk_bm_truncate(bm._h, 1, 2) == INV
    bm.check_invariants()


def test_truncate_keeps_shared_and_cached_blocks_intact():
    """A cut inside a block that another table names, or that the prefix cache knows, leaves the block
    as it is: the next token goes into a copy."""
    bm = pk.BlockManager(8, 4)
    bm.add_seq(1)
    bm.append(1, 8)
    bm.fork(1, 2)
    bm.truncate(2, 6)
    slots, pair = bm.append(2, 1)
    assert pair == (1, 2) and slots.tolist() == [2 * 4 + 2] and bm.table(1).tolist() == [0, 1]
    bm.check_invariants()
    # Cached and named by no other table.
    toks = list(range(8))
    bm = pk.BlockManager(8, 4)
    bm.add_seq(1)
    bm.append(1, 8)
    bm.commit(1, toks)
    bm.truncate(1, 7)
    assert bm.is_cached(1)
    slots, pairs = bm.append_batch([1])
    assert pairs.tolist() == [[1, 2]] and slots.tolist() == [2 * 4 + 3]
    assert bm.is_cached(1) and bm.refcount(1) == 0 and bm.cache_match(toks) == 8
    bm.check_invariants()
    # Cut to a block's end: the next token opens a block, the cached one behind stays findable.
    bm.truncate(1, 4)
    assert bm.append(1, 1)[1] is None and bm.cache_match(toks) == 8
    bm.check_invariants()


def test_truncated_cached_tail_counts_its_copy_before_anything_changes():
    bm = pk.BlockManager(2, 4)
    bm.add_seq(1)
    bm.append(1, 8)
    bm.commit(1, list(range(8)))
    bm.truncate(1, 6)
    for append in (lambda: bm.append(1, 1), lambda: bm.append_batch([1])):
        with pytest.raises(pk.PagedKVError) as e:
            append()
        assert e.value.status == pk.PK_ERR_OUT_OF_BLOCKS and bm.seq_len(1) == 6
    bm.check_invariants()


@pytest.mark.parametrize("seed", range(6))
def test_truncate_among_random_operations(seed):
    """Against a model that keeps each sequence's written tokens by slot: what a live sequence wrote
    is there after any order of appends, forks, cuts, commits and retirements."""
    rng = np.random.default_rng(seed)
    B, N = 4, 24
    bm = pk.BlockManager(N, B)
    cell = {}                       # slot -> token
    seqs, nxt, clock = {}, 0, 0     # id -> list of tokens
    for _ in range(400):
        ids = sorted(seqs)
        op = rng.integers(0, 6)
        if op == 0 or not ids:
            nxt += 1
            bm.add_seq(nxt)
            seqs[nxt] = []
        elif op == 1:
            s, n = int(rng.choice(ids)), int(rng.integers(1, 8))
            try:
                slots, pair = bm.append(s, n)
            except pk.PagedKVError as e:
                assert e.status == pk.PK_ERR_OUT_OF_BLOCKS
                bm.free_seq(s)
                del seqs[s]
                continue
            if pair:
                for j in range(B):
                    cell[pair[1] * B + j] = cell.get(pair[0] * B + j)
            for t in slots.tolist():
                clock += 1
                cell[t] = clock
                seqs[s].append(clock)
        elif op == 2 and len(ids) < 6:
            s = int(rng.choice(ids))
            nxt += 1
            bm.fork(s, nxt)
            seqs[nxt] = list(seqs[s])
        elif op == 3:
            s = int(rng.choice(ids))
            n = int(rng.integers(0, len(seqs[s]) + 1))
            bm.truncate(s, n)
            del seqs[s][n:]
        elif op == 4:
            s = int(rng.choice(ids))
            bm.commit(s, seqs[s])
        else:
            s = int(rng.choice(ids))
            bm.free_seq(s)
            del seqs[s]
        bm.check_invariants()
        for s, toks in seqs.items():
            table = bm.table(s)
            assert len(table) == -(-len(toks) // B) and bm.seq_len(s) == len(toks)
            assert [cell[table[i // B] * B + i % B] for i in range(len(toks))] == toks


# ---------------------------------------------------------------------------
# Refusals before any launch
# ---------------------------------------------------------------------------
def test_extend_refusals(L, ptr):
    p = ptr

    def call(out=p, q=p, kc=p, vc=p, tb=p, ln=p, of=p, scale=0.1, cap=0.0, window=0, scores=True, S=2, R=4, most=3,
             hq=8, mb=4, mc=64, part=0, items=None, ni=0, ws=None, wb=0, d=(64, 16, 2, 128, pk.PK_BF16)):
        sc = pk.ScoreDesc(cap, window, None, None, None)
        return L.pk_paged_attention_extend(out, q, kc, vc, tb, ln, of, scale, ctypes.byref(sc) if scores else None, S, R,
                                           most, hq, mb, mc, part, items, ni, ws, wb,
                                           None if d is None else ctypes.byref(pk.CacheDesc(*d)), None)

    assert call(S=0) == pk.PK_OK and call(R=0) == pk.PK_OK and call(most=0) == pk.PK_OK
    for kw in (dict(out=None), dict(q=None), dict(kc=None), dict(vc=None), dict(tb=None), dict(ln=None), dict(of=None),
               dict(out=p + 4), dict(q=p + 8), dict(kc=p + 2), dict(vc=p + 2), dict(scale=float("nan")),
               dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(window=-1), dict(S=-1), dict(R=-1),
               dict(most=-1), dict(hq=7), dict(mb=0), dict(mc=0), dict(part=-1), dict(part=24), dict(d=None),
               dict(items=p, ni=0), dict(items=None, ni=3), dict(items=p + 4, ni=1), dict(ni=-1),
               dict(of=None, most=1, R=1), dict(of=None, most=2)):
        assert call(**kw) == INV, kw
    for kw in (dict(hq=18), dict(d=(64, 16, 2, 96, pk.PK_BF16)), dict(d=(64, 16, 2, 128, pk.PK_E4M3)),
               dict(S=70000, R=70000), dict(R=1 << 30, S=2, hq=8), dict(mb=1 << 28, mc=64)):
        assert call(**kw) == UNS, kw
    assert call(part=32) == WSP and call(part=32, ws=p, wb=16) == WSP and call(ws=p + 4, wb=1 << 10) == WSP
    assert call(part=32, scores=False) == WSP


def test_verify_refusals(L, ptr):
    p = ptr

    def call(na=p, ac=p, nt=p, tp=p, ts=100, dp=None, ds=0, dt=pk.PK_F32, tok=p, un=p, of=p, par=None, S=2, R=4, most=3,
             V=100):
        return L.pk_verify_drafts(na, ac, nt, tp, ts, dp, ds, dt, tok, un, of, par, S, R, most, V, None)

    assert call(S=0) == pk.PK_OK
    for kw in (dict(na=None), dict(ac=None), dict(nt=None), dict(tp=None), dict(tok=None), dict(un=None), dict(of=None),
               dict(ts=99), dict(dp=p, ds=99), dict(S=-1), dict(R=-1), dict(most=-1), dict(V=0), dict(tp=p + 2),
               dict(dp=p + 1, ds=100), dict(tok=p + 4), dict(nt=p + 4)):
        assert call(**kw) == INV, kw
    for kw in (dict(dt=pk.PK_E4M3), dict(most=65), dict(dp=p, ds=100, par=p), dict(V=(1 << 24) + 1, ts=1 << 25)):
        assert call(**kw) == UNS, kw


def test_compact_refusals(L, ptr):
    p = ptr

    def call(kc=p, vc=p, tb=p, mb=4, ln=p, of=p, ac=p, na=p, lo=None, S=2, R=4, most=3, d=(64, 16, 2, 128, pk.PK_BF16)):
        return L.pk_compact_drafts(kc, vc, tb, mb, ln, of, ac, na, lo, S, R, most,
                                   None if d is None else ctypes.byref(pk.CacheDesc(*d)), None)

    assert call(S=0) == pk.PK_OK
    for kw in (dict(kc=None), dict(vc=None), dict(tb=None), dict(ln=None), dict(of=None), dict(ac=None), dict(na=None),
               dict(kc=p + 8), dict(vc=p + 8), dict(mb=0), dict(lo=p), dict(S=-1), dict(R=-1), dict(most=-1),
               dict(d=None), dict(d=(0, 16, 2, 128, pk.PK_BF16)), dict(d=(64, 16, 1, 4, pk.PK_BF16))):
        assert call(**kw) == INV, kw
    for kw in (dict(most=65), dict(S=65536), dict(d=(64, 16, 2, 128, pk.PK_E4M3)),
               dict(d=(1 << 28, 16, 2, 128, pk.PK_BF16))):
        assert call(**kw) == UNS, kw


def test_binding_refuses_cpu_tensors(L):
    torch = pytest.importorskip("torch")
    kc = torch.zeros((4, 16, 2, 64))
    q, tb, ln = torch.zeros((3, 4, 64)), torch.zeros((2, 4)).int(), torch.ones(2).int()
    of = torch.tensor([0, 1, 3]).int()
    with pytest.raises(ValueError, match="CUDA tensor"):
        pk.pk_paged_attention_extend(q, q, kc, kc, tb, ln, of, 0.1, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pk.pk_compact_drafts(kc, kc, tb, ln, of, torch.zeros(3).int(), ln, 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pk.pk_verify_drafts(ln, torch.zeros(3).int(), ln.long(), torch.zeros((3, 9)), torch.zeros(3).long(),
                            torch.zeros(3), of, 2)

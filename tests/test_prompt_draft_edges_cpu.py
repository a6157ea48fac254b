"""Edges of the block manager's cut on the CPU (batches of appends after cuts and commits), and refusals
before a launch."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk


@pytest.fixture(scope="module", autouse=True)
def _built():
    pk.build()


def committed(bm, seq, n):
    bm.add_seq(seq)
    bm.append(seq, n)
    bm.commit(seq, [100 * seq + i for i in range(n)])


def test_a_batch_of_appends_after_cuts_copies_from_no_block_that_it_copies_to():
    """Two sequences cut inside cached blocks, one block to evict: the first one's old tail must not
    become the second one's new tail."""
    bm = pk.BlockManager(6, 4)
    committed(bm, 1, 8)
    committed(bm, 2, 8)
    committed(bm, 3, 4)
    bm.truncate(1, 7)
    bm.truncate(2, 7)
    bm.free_seq(3)
    free = bm.num_free()
    assert free == 2
    pairs = bm.append_batch([1, 2])[1]
    assert not set(pairs[:, 0].tolist()) & set(pairs[:, 1].tolist()), pairs.tolist()
    assert sorted(pairs[:, 0].tolist()) == [1, 3] and sorted(pairs[:, 1].tolist()) == [4, 5]
    # The copied tails are cached still, and free.
    assert bm.is_cached(1) and bm.is_cached(3) and bm.num_free() == 2
    bm.check_invariants()


def test_a_copied_tail_is_the_youngest_block_of_the_cache():
    """The block released longest ago is evicted first, not the tail that an append has just copied."""
    bm = pk.BlockManager(4, 4)
    committed(bm, 1, 8)             # blocks 0, 1
    committed(bm, 2, 4)             # block 2
    bm.truncate(1, 6)
    bm.free_seq(2)                  # 2 is idle since now
    assert bm.append(1, 1)[1] == (1, 3)
    assert bm.is_cached(1) and bm.refcount(1) == 0
    assert bm.append(1, 2)[0].tolist() == [3 * 4 + 3, 2 * 4]  # evicts 2, the older one
    assert bm.is_cached(1) == 1 and bm.is_cached(2) == 0
    bm.check_invariants()


def test_one_append_does_not_go_on_into_the_tail_that_it_copied():
    """All blocks but the copied tail are taken: the tokens behind the copy find no block, and nothing changes."""
    bm = pk.BlockManager(3, 4)
    committed(bm, 1, 8)
    bm.truncate(1, 6)
    with pytest.raises(pk.PagedKVError) as e:
        bm.append(1, 3)
    assert e.value.status == pk.PK_ERR_OUT_OF_BLOCKS and bm.seq_len(1) == 6
    slots, pair = bm.append(1, 2)
    assert pair == (1, 2) and slots.tolist() == [2 * 4 + 2, 2 * 4 + 3] and bm.num_free() == 1
    assert bm.append(1, 1)[0].tolist() == [4] and bm.is_cached(1) == 0
    bm.check_invariants()


@pytest.mark.parametrize("seed", range(8))
def test_batches_among_cuts_and_commits_in_a_pool_that_evicts(seed):
    """A model that keeps each sequence's written tokens by slot: the pairs of a batch applied from a
    snapshot, first to last and last to first give the same cells, and what a live sequence wrote is there."""
    rng = np.random.default_rng(seed)
    B, N = 4, 14
    bm = pk.BlockManager(N, B)
    cells = np.full(N * B, -1)
    seqs, nxt, clock, copied = {}, 0, 0, 0

    def copies(cells, pairs, order, snapshot):
        out = cells.copy()
        for src, dst in (pairs[i] for i in order):
            out[dst * B: dst * B + B] = (cells if snapshot else out)[src * B: src * B + B]
        return out

    for _ in range(600):
        ids = sorted(seqs)
        op = rng.integers(0, 9)
        if op == 0 and len(ids) < 6 or not ids:
            nxt += 1
            bm.add_seq(nxt)
            seqs[nxt] = []
        elif op <= 4:
            batch = rng.permutation(ids)[: int(rng.integers(1, len(ids) + 1))].tolist()
            try:
                slots, pairs = bm.append_batch(batch)
            except pk.PagedKVError as e:
                assert e.status == pk.PK_ERR_OUT_OF_BLOCKS
                bm.free_seq(batch[0])
                del seqs[batch[0]]
                continue
            pairs = pairs.tolist()
            assert not {a for a, _ in pairs} & {b for _, b in pairs}
            assert len({b for _, b in pairs}) == len(pairs)
            copied += len(pairs)
            k = range(len(pairs))
            after = copies(cells, pairs, k, True)
            assert (after == copies(cells, pairs, k, False)).all()
            assert (after == copies(cells, pairs, reversed(k), False)).all()
            cells = after
            for s, t in zip(batch, slots.tolist()):
                clock += 1
                cells[t] = clock
                seqs[s].append(clock)
        elif op == 5 and len(ids) < 6:
            s = int(rng.choice(ids))
            nxt += 1
            bm.fork(s, nxt)
            seqs[nxt] = list(seqs[s])
        elif op == 6:
            s = int(rng.choice(ids))
            bm.commit(s, seqs[s])
            n = max(0, len(seqs[s]) - int(rng.integers(0, 4)))
            bm.truncate(s, n)
            del seqs[s][n:]
        elif op == 7:
            for s in ids:  # several at once, so that a batch copies several cached tails
                bm.commit(s, seqs[s])
                n = max(0, len(seqs[s]) - 1)
                bm.truncate(s, n)
                del seqs[s][n:]
        elif op == 8 and rng.random() < 0.5:
            s = int(rng.choice(ids))
            bm.free_seq(s)
            del seqs[s]
        bm.check_invariants()
        for s, toks in seqs.items():
            table = bm.table(s)
            assert [cells[table[i // B] * B + i % B] for i in range(len(toks))] == toks
    assert copied > 50


def test_extend_refuses_caps_beyond_what_fp32_can_hold():
    L = pk.lib()
    buf = np.zeros(1 << 16, np.uint8)
    p = (buf.ctypes.data + 255) // 256 * 256
    desc = pk.CacheDesc(64, 16, 2, 128, pk.PK_BF16)

    def call(cap, scale=0.1, R=0):
        sc = pk.ScoreDesc(cap, 0, None, None, None)
        return L.pk_paged_attention_extend(p, p, p, p, p, p, p, scale, ctypes.byref(sc), 2, R, 3, 8, 4, 64, 0, None, 0,
                                           None, 0, ctypes.byref(desc), None)

    for cap, scale in ((2.0 ** 99, 1.0), (2.0 ** 100, 1.0), (2.0 ** -100, 1.0), (1e6, 0.0), (30.0, -0.1), (2.0 ** -50, 2.0 ** 50),
                       (0.0, 1e-38), (-0.0, 0.1)):
        assert call(cap, scale) == pk.PK_OK, (cap, scale)  # (no rows, so nothing is launched)
    for cap, scale in ((2.0 ** 101, 1.0), (3.4e38, 0.1), (2.0 ** -101, 2.0 ** -101), (2.0 ** 60, 2.0 ** -41),
                       (2.0 ** -60, 2.0 ** 41), (1e30, 0.1), (1e-40, 0.1), (-1.0, 0.1), (float("nan"), 0.1),
                       (float("inf"), 0.1), (1.0, float("inf"))):
        for R in (0, 4):
            assert call(cap, scale, R) == pk.PK_ERR_INVALID_ARG, (cap, scale)


NO_MEMORY = r"""
// The block manager where allocations fail on request: no exception leaves an entry point, and
// what a call that needs no memory of its own does is done.
#include <cstdio>
#include <cstdlib>
#include <new>
#include "block_manager.cpp"

static long left = -1;  // allocations that succeed; -1: all
static long refused = 0;
void *operator new(std::size_t n) {
  if (left == 0) { ++refused; throw std::bad_alloc(); }
  if (left > 0) --left;
  if (void *p = std::malloc(n)) return p;
  throw std::bad_alloc();
}
void *operator new(std::size_t n, const std::nothrow_t &) noexcept { return std::malloc(n); }
void operator delete(void *p) noexcept { std::free(p); }
void operator delete(void *p, std::size_t) noexcept { std::free(p); }

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  pk_bm *bm;
  int64_t slots[64], pairs[8];
  int32_t n, tokens[64];
  for (int i = 0; i < 64; ++i) tokens[i] = i;
  for (long allow = 0; allow < 4; ++allow) {
    CHECK(pk_bm_create(16, 4, nullptr, &bm) == PK_OK);
    CHECK(pk_bm_add_seq(bm, 1) == PK_OK && pk_bm_append_slots(bm, 1, 24, slots, pairs, &n) == PK_OK);
    CHECK(pk_bm_commit(bm, 1, tokens, 24) == PK_OK);
    left = allow;
    CHECK(pk_bm_truncate(bm, 1, 6) == PK_OK);             // four cached blocks without a table
    const pk_status st = pk_bm_append_slots(bm, 1, 1, slots, pairs, &n);  // a copied tail
    CHECK(st == PK_OK && n == 1);
    left = -1;
    CHECK(refused > 0 && pk_bm_check_invariants(bm) == PK_OK && pk_bm_num_free(bm) == 14);
    left = 0;
    CHECK(pk_bm_free_seq(bm, 1) == PK_OK);
    left = -1;
    CHECK(pk_bm_check_invariants(bm) == PK_OK && pk_bm_num_free(bm) == 16);
    pk_bm_destroy(bm);
    refused = 0;
  }
  std::puts("ok");
  return 0;
}
"""


def test_cuts_and_copies_without_memory_for_the_cache(tmp_path):
    """A block that no table names any more and for which the cache has no memory leaves the cache instead."""
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    (tmp_path / "main.cpp").write_text(NO_MEMORY)
    exe = str(tmp_path / "main")
    subprocess.run([cxx, "-std=c++17", "-O1", "-w", "-I", os.path.join(root, "include"), "-I",
                    os.path.join(root, "paged_kv_cache_113_gb300", "csrc"), str(tmp_path / "main.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stdout, r.stderr)

"""Attention of drafted tokens and over the 8-bit cache where its parts meet: units
that follow one another on a CTA, states that are merged, values that are not
finite, long partitions. Bounds as in test_serving_ops_gpu."""
import numpy as np
import pytest

import paged_kv_cache_113_gb300 as pk
from test_serving_ops_gpu import DEV, f64, i32, rand, tables_for

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

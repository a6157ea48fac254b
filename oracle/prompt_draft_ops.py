"""Plain fp64 restatements of prompt attention with changed scores and of what
follows the attention of drafts: TEST INFRASTRUCTURE, NumPy only, sharing no code
with the CUDA library.

* :func:`extend_attention`  softmax attention of new tokens over a paged context, with
                            what its rounding errors are bounded by;
* :func:`verify_drafts`     drafts accepted or refused, and the next token;
* :func:`compact_drafts`    the kept tokens' rows moved together.

Pinned by ``tests/test_prompt_draft_ops_cpu.py``.
"""
from __future__ import annotations

import numpy as np

LOG2E = 1.4426950408889634


def extend_attention(q, k, v, tables, ctx_lens, scale, q_offsets=None, softcap=0.0, window=0, slopes=None,
                     prefix_lens=None, first_tokens=None):
    """q [R, Hq, d], k and v [N, B, Hk, d] in fp64; tables [S, max_blocks].

    Returns ``(out, terms)``: fp64 [R, Hq, d] with NaN in rows of no sequence, and
    per row and head: sum_t w_t |v_t| [R, Hq, d]; (sum_t w_t m_t |v_t|, sum_t w_t m_t) with m_t the
    magnitude log2(e) (scale sum_i |q_i k_i|) of the score; the same of the magnitude after the cap
    and the bias; and the tokens seen [R].
    """
    R, Hq, d = q.shape
    B, Hk = k.shape[1], k.shape[2]
    out = np.full((R, Hq, d), np.nan)
    wv, mv, av = np.zeros((R, Hq, d)), np.zeros((R, Hq, d)), np.zeros((R, Hq, d))
    ms, as_, cnt = np.zeros((R, Hq, 1)), np.zeros((R, Hq, 1)), np.zeros((R, 1, 1))
    for s, ctx in enumerate(ctx_lens):
        r0, r1 = (s, s + 1) if q_offsets is None else (int(q_offsets[s]), int(q_offsets[s + 1]))
        n, ctx = r1 - r0, int(ctx)
        if n <= 0:
            continue
        pos = np.arange(ctx)
        blocks = np.asarray(tables[s])[pos // B]
        kk, vv = k[blocks, pos % B], v[blocks, pos % B]  # [ctx, Hk, d]
        for i in range(n):
            at = ctx - n + i
            seen = pos <= at
            if prefix_lens is not None:
                seen |= pos < prefix_lens[s]
            if window:
                seen &= pos > at - window
            if first_tokens is not None:
                seen &= pos >= first_tokens[r0 + i]
            t = pos[seen]
            cnt[r0 + i] = len(t)
            for h in range(Hq):
                g = h // (Hq // Hk)
                ks, vs = kk[seen, g], vv[seen, g]
                if not len(t):
                    out[r0 + i, h] = 0.0
                    continue
                x = ks @ q[r0 + i, h] * scale
                m = np.abs(ks) @ np.abs(q[r0 + i, h]) * abs(scale) * LOG2E
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                a = np.abs(x) + (softcap or 0.0)
                if slopes is not None:
                    far = np.abs(at - t) * float(slopes[h])
                    x = x - far
                    a = a + np.abs(far)
                a = a * LOG2E
                top = x.max()
                if top == -np.inf:
                    out[r0 + i, h] = 0.0
                    continue
                w = np.exp(x - top)
                w /= w.sum()
                out[r0 + i, h] = w @ vs
                wv[r0 + i, h] = w @ np.abs(vs)
                mv[r0 + i, h], ms[r0 + i, h] = (w * m) @ np.abs(vs), w @ m
                av[r0 + i, h], as_[r0 + i, h] = (w * a) @ np.abs(vs), w @ a
    return out, (wv, (mv, ms), (av, as_), cnt)


def _weights(x):
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((x > 0) & np.isfinite(x), x, 0.0)


def verify_drafts(target, tokens, uniforms, q_offsets, parents=None, draft=None):
    """target, draft [R, V]; returns (num_accepted [S], accepted: a list of paths, next_tokens [S])."""
    V = target.shape[1]
    counts, paths, nexts = [], [], []
    for a, b in zip(q_offsets[:-1], q_offsets[1:]):
        if b <= a:
            counts.append(0), paths.append([]), nexts.append(-1)
            continue
        node, path = 0, [0]
        while True:
            p = _weights(target[a + node])
            w, mass, down = p.copy(), 1.0, None
            refused = None
            for i in range(node + 1, b - a):
                up = i - 1 if parents is None else int(parents[a + i])
                if up != node:
                    continue
                t = int(tokens[a + i])
                if not 0 <= t < V:
                    continue
                u = float(uniforms[a + i])
                if draft is None:
                    if u * mass < w[t]:
                        down = i
                        break
                    mass -= w[t]
                    w[t] = 0.0
                else:
                    qd = _weights(draft[a + i])
                    if u * qd[t] < p[t]:
                        down = i
                        break
                    refused = np.maximum(p - qd, 0.0)
            if down is None:
                if refused is not None:
                    w = refused
                break
            node = down
            path.append(down)
        if not w.sum() > 0:
            w = p
        c = np.cumsum(w)
        above = np.nonzero(c > float(uniforms[a]) * c[-1])[0]
        counts.append(len(path) - 1), paths.append(path), nexts.append(int(above[0]) if len(above) else -1)
    return counts, paths, nexts


def compact_drafts(pool, tables, ctx_lens, q_offsets, paths):
    """pool [N, B, ...] (changed in place); returns the lengths that are left."""
    B = pool.shape[1]
    out = []
    for s, path in enumerate(paths):
        n = int(q_offsets[s + 1] - q_offsets[s])
        base = int(ctx_lens[s]) - n
        rows = [pool[tables[s][(base + r) // B], (base + r) % B].copy() for r in path]
        for i, row in enumerate(rows):
            pool[tables[s][(base + i) // B], (base + i) % B] = row
        out.append(base + len(path) if n else int(ctx_lens[s]))
    return out

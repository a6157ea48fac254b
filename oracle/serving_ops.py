"""Plain fp64 restatements of the draft-and-verify operators: TEST
INFRASTRUCTURE, NumPy only, sharing no code with the CUDA library.

* :func:`norm_rope`        per-head RMS norm and rotary positions;
* :func:`quantize_rows`    the 8-bit rows (e4m3 codes and one power of two);
* :func:`decode_values`    what codes and exponents stand for;
* :func:`tree_attention`   softmax attention of query rows over the tokens each
                           of them sees, with the bound of its rounding errors.

Pinned by ``tests/test_serving_ops_cpu.py``.
"""
from __future__ import annotations

import numpy as np

LOG2E = 1.4426950408889634


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, H, d] (fp64) -> fp64; weight [d] or None; cos_sin [max, rot] or None."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if cos_sin is None or cos_sin.shape[1] == 0:
        return y
    rot = cos_sin.shape[1]
    half = rot // 2
    out = y.copy()
    for t, p in enumerate(positions):
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = float(cos_sin[p, j]), float(cos_sin[p, half + j])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for code in range(256):
        sign, e, m = -1.0 if code & 0x80 else 1.0, (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            out[code] = np.nan
        elif e == 0:
            out[code] = sign * m * 2.0 ** -9
        else:
            out[code] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


def _nearest_code(x: float) -> int:
    """The code nearest to a finite |x| <= 448, ties to the even code."""
    vals = e4m3_values()[:127]  # the non-negative finite codes, ascending
    a = abs(x)
    hi = int(np.searchsorted(vals, a))
    lo = max(hi - 1, 0)
    hi = min(hi, 126)
    if a - vals[lo] < vals[hi] - a or (a - vals[lo] == vals[hi] - a and lo % 2 == 0):
        code = lo
    else:
        code = hi
    return code | (0x80 if np.signbit(x) else 0)


def quantize_rows(x):
    """Rows [..., d] (fp64 holding fp32 or bf16 values) -> (codes uint8, biased
    exponents uint8 [...])."""
    x = np.asarray(x, np.float64)
    rows = x.reshape(-1, x.shape[-1])
    codes = np.zeros(rows.shape, np.uint8)
    exps = np.zeros(len(rows), np.uint8)
    for r, row in enumerate(rows):
        fin = np.abs(row[np.isfinite(row)])
        amax = fin.max() if len(fin) else 0.0
        e = 0
        if amax > 0:
            e = -100
            while 448.0 * 2.0 ** e < amax:
                e += 1
        exps[r] = e + 127
        for i, v in enumerate(row):
            codes[r, i] = _nearest_code(v * 2.0 ** -e) if np.isfinite(v) else 0x7F
    return codes.reshape(x.shape), exps.reshape(x.shape[:-1])


def decode_values(codes, exps):
    """fp64 values of codes [..., d] with biased exponents [...]."""
    return e4m3_values()[np.asarray(codes, np.uint8)] * 2.0 ** (np.asarray(exps, np.float64) - 127)[..., None]


def tree_attention(q, k, v, tables, ctx_lens, scale, q_offsets=None, masks=None):
    """q [R, Hq, d], k and v [N, B, Hk, d] in fp64; tables [S, max_blocks].

    Without q_offsets row s is sequence s's only query and sees its whole
    context. masks: Python ints or int64 words per row, or None (a chain).
    Returns ``(out, terms)``: fp64 [R, Hq, d] with NaN in rows of no sequence,
    and per row and head (sum_t w_t |v_t| [R, Hq, d], the largest
    scale * log2(e) * sum_i |q_i k_i| of the seen tokens, tokens seen).
    """
    R, Hq, d = q.shape
    B, Hk = k.shape[1], k.shape[2]
    out = np.full((R, Hq, d), np.nan)
    wv = np.zeros((R, Hq, d))
    mag = np.zeros((R, Hq))
    cnt = np.zeros((R, Hq))
    for s, ctx in enumerate(ctx_lens):
        r0, r1 = (s, s + 1) if q_offsets is None else (int(q_offsets[s]), int(q_offsets[s + 1]))
        n = r1 - r0
        if n <= 0:
            continue
        ctx = int(ctx)
        pos = np.arange(ctx)
        blocks = np.asarray(tables[s])[pos // B] if ctx else np.zeros(0, np.int64)
        kk, vv = k[blocks, pos % B], v[blocks, pos % B]  # [ctx, Hk, d]
        for i in range(n):
            seen = pos < ctx - n
            for j in range(n):
                bit = j <= i if masks is None else (int(masks[r0 + i]) >> j) & 1
                if bit:
                    seen[ctx - n + j] = True
            for h in range(Hq):
                g = h // (Hq // Hk)
                ks, vs = kk[seen, g], vv[seen, g]
                if not len(ks):
                    out[r0 + i, h] = 0.0
                    continue
                x = ks @ q[r0 + i, h] * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[r0 + i, h] = w @ vs
                wv[r0 + i, h] = w @ np.abs(vs)
                mag[r0 + i, h] = (np.abs(ks) @ np.abs(q[r0 + i, h])).max() * scale * LOG2E
                cnt[r0 + i, h] = len(ks)
    return out, (wv, mag, cnt)

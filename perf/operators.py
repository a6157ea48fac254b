"""Measured cases of the library's draft-and-verify operators.

Four operators of a serving step beside the decode path the library had:

* ``rope``    per-head RMS norm of queries and keys, the position rotation and
              the cache write, one pass (``pk_qk_norm_rope_and_cache``);
* ``write`` / ``read``  the 8-bit (e4m3) cache as it is written and read back
              (``pk_reshape_and_cache_e4m3``, ``pk_gather_cache_e4m3``);
* ``decode``  decode attention over the 8-bit cache
              (``pk_paged_attention_decode_e4m3``);
* ``tree``    attention of each sequence's drafted tokens, a tree or a chain,
              over its cached context (``pk_paged_attention_tree``).

With ``own`` false ``run`` computes an operator in its plain form: elementary
torch operations in fp32, rounded once at the end. With ``own`` true it makes
the library's calls. ``exact`` computes the definition in fp64, sequence by
sequence.

The 8-bit cache holds e4m3 codes ``[N, B, Hk, d]`` and one biased power of two
per token, KV head and side, ``kv_exp`` uint8 ``[N, Hk, B, 2]`` (K then V):
value = code * 2^(kv_exp - 127).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases. Head layouts, block sizes, context lengths and batches are those of
# the library's own workloads (tiny, mha7b, gqa8b, long, mixed, prefix).
# ---------------------------------------------------------------------------
def _rope(name, tokens, hq, hk, d, dtype, rot, inter, blk, norm=True, prompt=False):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "dtype": dtype, "rot": rot,
            "inter": inter, "blk": blk, "norm": norm, "prompt": prompt}


def _kv(name, op, tokens, hk, d, dtype, blk):
    return {"name": name, "op": op, "tokens": tokens, "hk": hk, "d": d, "dtype": dtype, "blk": blk}


def _dec(name, seqs, hq, hk, d, dtype, blk, lens, lo, hi):
    return {"name": name, "op": "decode", "seqs": seqs, "hq": hq, "hk": hk, "d": d, "dtype": dtype, "blk": blk,
            "lens": lens, "lo": lo, "hi": hi}


def _tree(name, seqs, hq, hk, d, dtype, blk, lens, lo, hi, draft, mask):
    c = _dec(name, seqs, hq, hk, d, dtype, blk, lens, lo, hi)
    return {**c, "op": "tree", "draft": draft, "mask": mask}


def listed():
    return [
        # One decode step of the 7B-like batch: 64 new tokens, latency counts.
        _rope("rope decode 64", 64, 32, 32, 128, "bf16", 128, False, 16),
        # A chunk of prompts of the 8B-like layer, packed, going into the cache.
        _rope("rope prompt 8192", 8192, 32, 8, 128, "bf16", 128, False, 16, prompt=True),
        # An odd number of fp32 tokens, interleaved pairs, half of the head rotated.
        _rope("rope odd f32 1021", 1021, 8, 8, 64, "f32", 32, True, 16),
        # One decode step of the 8B-like batch written into the 8-bit cache.
        _kv("write 256", "write", 256, 8, 128, "bf16", 16),
        # Eight 2000-token prompts written into the 8-bit cache, 32-token blocks.
        _kv("write 16000", "write", 16000, 8, 128, "bf16", 32),
        # One 32K context read back as bf16.
        _kv("read 32768", "read", 32768, 8, 128, "bf16", 16),
        # The smallest batch: four fp32 sequences of 1..100 tokens.
        _dec("decode tiny f32", 4, 8, 8, 64, "f32", 16, "even", 1, 100),
        # The 8B-like batch: heavy-tailed lengths.
        _dec("decode gqa 256", 256, 32, 8, 128, "bf16", 16, "tail", 33, 4608),
        # Eight 32K contexts.
        _dec("decode long 8x32768", 8, 64, 8, 128, "bf16", 16, "even", 32768, 32768),
        # Four short sequences with small trees, fp32.
        _tree("tree tiny f32", 4, 8, 8, 64, "f32", 16, "even", 9, 100, 8, "tree"),
        # The 8B-like batch with 16 drafted tokens per sequence.
        _tree("tree gqa 256x16", 256, 32, 8, 128, "bf16", 16, "tail", 64, 4608, 16, "tree"),
        # Eight 32K contexts with 32 drafted tokens each.
        _tree("tree long 8x32", 8, 64, 8, 128, "bf16", 16, "even", 32768, 32768, 32, "tree"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["rope", "write", "read", "decode", "decode", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    blk = rng.choice([8, 16, 32])
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8, 32])
        hq = hk * rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8) if g * hk <= 64])
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, 16, (d // 32) * 16])
        most = max(1, min(8192, 40_000_000 // ((hq + 2 * hk) * d)))
        return _rope(None, _log(rng, 1, most), hq, hk, d, dtype, rot, rng.random() < 0.4, blk,
                     norm=rng.random() < 0.8, prompt=rng.random() < 0.5)
    if op in ("write", "read"):
        hk = rng.choice([1, 2, 4, 8, 32])
        d = rng.choice([64, 128, 256])
        most = max(1, min(32768, 30_000_000 // (hk * d)))
        return _kv(op, op, _log(rng, 1, most), hk, d, dtype, blk)
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
    d = rng.choice([64, 128])
    lens = rng.choice(["even", "tail", "one long"])
    # Context tokens of the whole batch stay below those of the largest listed cases.
    cap = 262144 * 8 // hk if dtype == "bf16" else 65536 * 8 // hk
    if op == "tree":
        draft = _log(rng, 1, 64)
        cap = min(cap, 262144 * 256 * 8 // (draft * hq)) // (1 if dtype == "bf16" else 4)
    seqs = _log(rng, 1, 256)
    hi = max(66, min(32768, cap // seqs))
    hi = _log(rng, 66, hi)
    lo = _log(rng, 1, hi)
    if op == "decode":
        return _dec(op, seqs, hq, hk, d, dtype, blk, lens, lo, hi)
    return _tree(op, seqs, hq, hk, d, dtype, blk, lens, lo, hi, draft, rng.choice(["tree", "chain", "any"]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case, g):
    """Context lengths: evenly spread, heavy-tailed, or short with one long."""
    S, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case["lens"] == "even":
        return lo + torch.randint(0, hi - lo + 1, (S,), generator=g)
    if case["lens"] == "tail":
        x = torch.exp(torch.randn(S, generator=g) + math.log(200.0) - 0.5) + 32 + torch.rand(S, generator=g) * 480
        return x.round().long().clamp(lo, hi)
    x = lo + torch.randint(0, max(1, (hi - lo) // 8), (S,), generator=g)
    x[int(torch.randint(0, S, (1,), generator=g))] = hi
    return x


def _rand(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _slots(g, tokens, blk, prompt):
    """Slots of new tokens in a pool twice their size: whole shuffled blocks of
    prompts, or one slot in a block of its own for each decoded token."""
    if prompt:
        nb = -(-tokens // blk)
        blocks = torch.randperm(2 * nb, generator=g)[:nb]
        slots = (blocks[:, None] * blk + torch.arange(blk)[None]).reshape(-1)[:tokens]
        return slots, 2 * nb
    blocks = torch.randperm(2 * tokens, generator=g)[:tokens]
    return blocks * blk + torch.randint(0, blk, (tokens,), generator=g), 2 * tokens


def _tables(g, lens, blk):
    nb = (lens + blk - 1) // blk
    maxb = int(nb.max())
    total = int(nb.sum())
    order = torch.randperm(total, generator=g).int()
    tables = torch.full((len(lens), maxb), -1, dtype=torch.int32)
    at = torch.arange(maxb)[None] < nb[:, None]
    tables[at] = order
    return tables, total


def _e4m3_pool(gen, n, blk, hk, d):
    """Codes and exponents as written from keys and values of unit variance
    (largest scaled magnitude of a row in (224, 448])."""
    codes, exps = [], torch.empty((n, hk, blk, 2), dtype=torch.uint8, device=DEV)
    for side in (0, 1):
        x = _rand(gen, (n, blk, hk, d))
        a = x.abs().amax(-1)
        e = torch.ceil(torch.log2(a / 448.0))
        codes.append((x * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn))
        exps[..., side] = (e + 127).to(torch.uint8).permute(0, 2, 1)
    return codes[0], codes[1], exps


def _i64(x):
    """A Python integer of 64 bits as the signed value with its bit pattern."""
    return x - (1 << 64) if x >= 1 << 63 else x


def _masks(case, g, counts):
    """Visibility of each drafted token (bit j: draft j of its sequence): the
    ancestors in a random tree, or any subset with the token itself. None is a chain."""
    if case["mask"] == "chain":
        return None
    out = []
    for n in counts.tolist():
        if case["mask"] == "any":
            bits = torch.randint(0, 2, (n, n), generator=g) | torch.eye(n, dtype=torch.long)
            out += [_i64(sum(int(b) << j for j, b in enumerate(row))) for row in bits.tolist()]
            continue
        rows = []
        parent = (torch.rand(n, generator=g) * torch.arange(n)).long().tolist()
        for i in range(n):
            rows.append((1 << i) | (rows[parent[i]] if i else 0))
        out += [_i64(r) for r in rows]
    return torch.tensor(out, dtype=torch.int64)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    s = {"case": case, "op": case["op"]}
    dt = DTYPES[case["dtype"]]
    d, hk, blk = case["d"], case["hk"], case["blk"]
    if case["op"] == "rope":
        T, hq, rot = case["tokens"], case["hq"], case["rot"]
        slots, nb = _slots(g, T, blk, case["prompt"])
        qkv = _rand(gen, (T, hq + 2 * hk, d)) * (0.5 + torch.rand((1, hq + 2 * hk, 1), generator=gen, device=DEV))
        s["qkv"] = qkv.to(dt)  # the packed projection; q, k and v are views of it
        s["q"], s["k"], s["v"] = s["qkv"].split([hq, hk, hk], dim=1)
        s["q_weight"] = (1 + 0.1 * _rand(gen, (d,))).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + 0.1 * _rand(gen, (d,))).to(dt) if case["norm"] else None
        ang = torch.arange(32768, dtype=torch.float64, device=DEV)[:, None] * \
            (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot))[None]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        pos = torch.arange(T) % 2000 if case["prompt"] else torch.randint(0, 32768, (T,), generator=g)
        s["positions"], s["slots"] = pos.to(DEV), slots.to(DEV)
        s["k_cache"] = torch.zeros((nb, blk, hk, d), dtype=dt, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["q_out"] = torch.empty((T, hq, d), dtype=dt, device=DEV)
        s["k_out"] = torch.empty((T, hk, d), dtype=dt, device=DEV)
        return s
    if case["op"] in ("write", "read"):
        T = case["tokens"]
        slots, nb = _slots(g, T, blk, T > 512)
        s["slots"] = slots.to(DEV)
        if case["op"] == "write":
            s["k"] = _rand(gen, (T, hk, d), dt)
            s["v"] = (_rand(gen, (T, hk, d)) * torch.exp2(2 * _rand(gen, (T, hk, 1)))).to(dt)
            s["k_cache"] = torch.zeros((nb, blk, hk, d), dtype=torch.float8_e4m3fn, device=DEV)
            s["v_cache"] = torch.zeros_like(s["k_cache"])
            s["kv_exp"] = torch.full((nb, hk, blk, 2), 127, dtype=torch.uint8, device=DEV)
        else:
            s["k_cache"], s["v_cache"], s["kv_exp"] = _e4m3_pool(gen, nb, blk, hk, d)
            s["k_out"] = torch.empty((T, hk, d), dtype=dt, device=DEV)
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    S, hq = case["seqs"], case["hq"]
    lens = _lengths(case, g)
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "tree":
        # Each sequence drafts up to `draft` tokens, the last of its context.
        counts = torch.minimum(1 + (torch.rand(S, generator=g) * case["draft"]).long(), lens)
        counts[0] = min(case["draft"], int(lens[0]))
        if case["lens"] == "even" and case["lo"] == case["hi"]:
            counts = torch.full((S,), min(case["draft"], case["hi"]))
        offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
        masks = _masks(case, g, counts)
        s["tree_mask"] = None
        s["q_offsets"], s["max_draft"] = offsets.int().to(DEV), int(counts.max())
        # A fixed batch buffer: the rows behind the last sequence's are padding.
        rows = S * case["draft"]
        if masks is not None:
            s["tree_mask"] = torch.zeros(rows, dtype=torch.int64, device=DEV)
            s["tree_mask"][:len(masks)] = masks.to(DEV)
    else:
        rows = S
    tables, total = _tables(g, lens, blk)
    s["tables"], s["lens"], s["max_len"] = tables.to(DEV), lens.int().to(DEV), int(lens.max())
    s["q"] = _rand(gen, (rows, hq, d), dt)
    s["out"] = torch.zeros_like(s["q"])
    if case["op"] == "decode":
        s["k_cache"], s["v_cache"], s["kv_exp"] = _e4m3_pool(gen, total, blk, hk, d)
    else:
        s["k_cache"] = _rand(gen, (total, blk, hk, d), dt)
        s["v_cache"] = _rand(gen, (total, blk, hk, d), dt)
    if own:  # the plan and the workspace that a serving loop keeps beside its batch
        import paged_kv_cache_113_gb300 as pk
        desc = pk.cache_desc(s["k_cache"])
        if case["op"] == "decode":
            s["partition"], items = pk.pk_attention_plan(lens.numpy(), hq, desc, -1)
            ws = pk.pk_paged_attention_workspace_size(S, hq, s["max_len"], s["partition"], desc)
        else:
            s["partition"], items = pk.pk_tree_plan(lens.numpy(), s["max_draft"], hq, desc, -1)
            ws = pk.pk_tree_workspace_size(rows, hq, s["max_len"], s["partition"], desc)
        s["items"] = torch.from_numpy(items).to(DEV)
        s["workspace"] = torch.empty(max(ws, 16), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_rope(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_qk_norm_rope_and_cache(s["q_out"], s["k_out"], s["q"], s["k"], s["v"], s["cos_sin"], s["positions"],
                                 q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                 interleaved=s["case"]["inter"], slot_mapping=s["slots"], k_cache=s["k_cache"],
                                 v_cache=s["v_cache"])
    return {"q": s["q_out"], "k": s["k_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_write(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_reshape_and_cache_e4m3(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["kv_exp"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_exp": s["kv_exp"]}


def _own_read(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_gather_cache_e4m3(s["k_out"], s["v_out"], s["slots"], s["k_cache"], s["v_cache"], s["kv_exp"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_decode(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_paged_attention_decode_e4m3(s["out"], s["q"], s["k_cache"], s["v_cache"], s["kv_exp"], s["tables"],
                                      s["lens"], s["scale"], s["max_len"], partition_size=s["partition"],
                                      workspace=s["workspace"], work_items=s["items"])
    return s["out"]


def _own_tree(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_paged_attention_tree(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["q_offsets"],
                               s["scale"], s["max_draft"], s["max_len"], tree_mask=s["tree_mask"],
                               partition_size=s["partition"], workspace=s["workspace"], work_items=s["items"])
    return s["out"]


def _plain_rotate(x, cs, rot, inter):
    """Rotates the first `rot` elements of x [T, H, d] by cs [T, rot] (cos, then sin)."""
    c, n = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"]]
    outs = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        outs.append(_plain_rotate(y, cs, c["rot"], c["inter"]).to(x.dtype))
    s["k_cache"].view(-1, c["hk"], c["d"])[s["slots"]] = outs[1]
    s["v_cache"].view(-1, c["hk"], c["d"])[s["slots"]] = s["v"]
    return {"q": outs[0], "k": outs[1], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_quantize(x):
    """e4m3 codes and biased exponents: the smallest power of two at or above
    amax / 448, at least 2^-100; 1 for a row of zeros."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-100)
    e = torch.where(m == 0, torch.zeros_like(e), e)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_write(s):
    c = s["case"]
    block, at = s["slots"] // c["blk"], s["slots"] % c["blk"]
    for side, name in ((0, "k"), (1, "v")):
        codes, exps = _plain_quantize(s[name])
        s[name + "_cache"].view(torch.uint8).view(-1, c["hk"], c["d"])[s["slots"]] = codes.view(torch.uint8)
        s["kv_exp"][block, :, at, side] = exps
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "kv_exp": s["kv_exp"]}


def _values(codes, exps):
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(exps.float() - 127.0)[..., None]


def _plain_read(s):
    c = s["case"]
    block, at = s["slots"] // c["blk"], s["slots"] % c["blk"]
    out = {}
    for side, name in ((0, "k"), (1, "v")):
        codes = s[name + "_cache"].view(torch.uint8).view(-1, c["hk"], c["d"])[s["slots"]]
        out[name] = _values(codes, s["kv_exp"][block, :, at, side]).to(s["k_out"].dtype)
    return out


def _plain_attend(q, k, v, see, scale):
    """q [S, n, Hq, d], k and v [S, t, Hk, d], see [S, n, t]: softmax attention
    of every row over what it sees; a row that sees nothing gets zeros."""
    S, n, hq, d = q.shape
    hk = k.shape[2]
    q = q.view(S, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(S * hk, -1, d)     # [S*Hk, G*n, d]
    k = k.permute(0, 2, 3, 1).reshape(S * hk, d, -1)
    x = torch.bmm(q, k).view(S, hk, hq // hk, n, -1) * scale
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    v = v.permute(0, 2, 1, 3).reshape(S * hk, -1, d)
    o = torch.bmm(p.view(S * hk, -1, p.shape[-1]), v)
    return o.view(S, hk, hq // hk, n, d).permute(0, 3, 1, 2, 4).reshape(S, n, hq, d)


def _plain_decode(s):
    c = s["case"]
    S, t = s["tables"].shape[0], s["tables"].shape[1] * c["blk"]
    tables = s["tables"].clamp_min(0).long()
    kv = []
    for side, name in ((0, "k_cache"), (1, "v_cache")):
        exps = s["kv_exp"][..., side][tables].transpose(2, 3)                            # [S, nb, B, Hk]
        kv.append(_values(s[name].view(torch.uint8)[tables], exps).view(S, t, c["hk"], c["d"]))
    see = torch.arange(t, device=DEV)[None] < s["lens"][:, None]
    return _plain_attend(s["q"].float()[:, None], kv[0], kv[1], see[:, None], s["scale"])[:, 0].to(s["q"].dtype)


def _plain_tree(s):
    c = s["case"]
    S, t, n = s["tables"].shape[0], s["tables"].shape[1] * c["blk"], s["max_draft"]
    tables = s["tables"].clamp_min(0).long()
    k, v = (s[name][tables].view(S, t, c["hk"], c["d"]).float() for name in ("k_cache", "v_cache"))
    first, count = s["q_offsets"][:-1].long(), s["q_offsets"].diff().long()
    i = torch.arange(n, device=DEV)
    live = i[None] < count[:, None]                                                      # [S, n]
    row = torch.where(live, first[:, None] + i[None], torch.zeros_like(first)[:, None])
    j = torch.arange(t, device=DEV)[None] - (s["lens"] - count)[:, None]                 # draft index, < 0: context
    if s["tree_mask"] is None:
        bit = j[:, None] <= i[None, :, None]
    else:
        bit = (s["tree_mask"][row][:, :, None] >> j.clamp(0, 63)[:, None]) & 1 == 1
    see = ((j < 0)[:, None] | bit) & (j < count[:, None])[:, None]
    o = _plain_attend(s["q"].float()[row], k, v, see, s["scale"])
    s["out"][row[live]] = o[live].to(s["q"].dtype)
    return s["out"]


_PLAIN = {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "decode": _plain_decode, "tree": _plain_tree}
_OWN = {"rope": _own_rope, "write": _own_write, "read": _own_read, "decode": _own_decode, "tree": _own_tree}


# ---------------------------------------------------------------------------
# What the path cannot do without
# ---------------------------------------------------------------------------
def _draw_lengths(case):
    """Expected context lengths of a case (its seed is not known here)."""
    S, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case["lens"] == "even":
        return S * (lo + hi) / 2
    if case["lens"] == "tail":
        return S * min(max(472.0, lo), hi)
    return (S - 1) * (lo + max(0, (hi - lo) // 8 - 1) / 2) + hi


def work(case):
    d, hk = case["d"], case["hk"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        T, hq = case["tokens"], case["hq"]
        # q, k, v read; q, k and the cache's K and V written; table row, position and slot of each token
        return {"bytes": T * d * e * (hq + 2 * hk + hq + 3 * hk) + T * (case["rot"] * 4 + 16),
                "flops": T * (hq + hk) * d * 7}
    if case["op"] in ("write", "read"):
        return {"bytes": case["tokens"] * (2 * hk * (d * (e + 1) + 1) + 8), "flops": case["tokens"] * hk * d * 4}
    tokens, hq = _draw_lengths(case), case["hq"]
    if case["op"] == "decode":
        return {"bytes": tokens * hk * 2 * (d + 1) + 2 * case["seqs"] * hq * d * e, "flops": 4.0 * tokens * hq * d}
    n = case["draft"] if case["lo"] == case["hi"] else (case["draft"] + 1) / 2
    return {"bytes": tokens * hk * 2 * d * e + 2 * case["seqs"] * n * hq * d * e, "flops": 4.0 * tokens * n * hq * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(s):
    c = s["case"]
    T, d, half = c["tokens"], c["d"], c["rot"] // 2
    cs = s["cos_sin"].double()[s["positions"]]
    first = 2 * torch.arange(half, device=DEV) if c["inter"] else torch.arange(half, device=DEV)
    second = first + (1 if c["inter"] else half)

    def one(x, w):
        y = x.double().clone()
        if w is not None:
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        z = torch.complex(y[..., first], y[..., second]) * torch.complex(cs[:, :half], cs[:, half:])[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])
    kc, vc = s["k_cache"].double().reshape(-1, c["hk"], d), s["v_cache"].double().reshape(-1, c["hk"], d)
    kc.index_copy_(0, s["slots"], k)
    vc.index_copy_(0, s["slots"], s["v"].double())
    return {"q": q, "k": k, "k_cache": kc.view(s["k_cache"].shape), "v_cache": vc.view(s["v_cache"].shape)}


def _exact_write(s):
    """The scaled values that the codes are the nearest e4m3 numbers to."""
    c = s["case"]
    out = {"kv_exp": None}
    for name in ("k", "v"):
        x = s[name].double()
        a = x.abs().amax(-1, keepdim=True)
        p = torch.ceil(torch.log2(a / 448.0)).clamp_min(-100)                            # amax = 448 * 2^p stays at p
        codes = s[name + "_cache"].double().reshape(-1, c["hk"], c["d"])
        codes.index_copy_(0, s["slots"], torch.where(a > 0, x / torch.pow(2.0, p), x))
        out[name + "_cache"] = codes.view(s[name + "_cache"].shape)
    return out


def _exact_read(s):
    c = s["case"]
    out = {}
    for side, name in ((0, "k"), (1, "v")):
        values = s[name + "_cache"].double() * torch.pow(2.0, s["kv_exp"][..., side].double() - 127).transpose(1, 2)[..., None]
        out[name] = values.reshape(-1, c["hk"], c["d"]).index_select(0, s["slots"])
    return out


def _exact_attention(s):
    c = s["case"]
    hk, hq, d = c["hk"], c["hq"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    ofs = s["q_offsets"].tolist() if c["op"] == "tree" else list(range(len(lens) + 1))
    for b, n in enumerate(lens):
        blocks = s["tables"][b, :-(-n // c["blk"])].long()
        k, v = s["k_cache"][blocks] if c["op"] == "tree" else s["k_cache"].view(torch.uint8)[blocks], \
            s["v_cache"][blocks] if c["op"] == "tree" else s["v_cache"].view(torch.uint8)[blocks]
        if c["op"] == "decode":
            p = torch.pow(2.0, s["kv_exp"][blocks].double() - 127).transpose(1, 2)       # [nb, B, Hk, 2]
            k, v = k.view(torch.float8_e4m3fn).double() * p[..., :1], v.view(torch.float8_e4m3fn).double() * p[..., 1:]
        k, v = (x.double().reshape(-1, hk, d)[:n].transpose(0, 1) for x in (k, v))       # [Hk, n, d]
        rows = ofs[b + 1] - ofs[b]
        q = s["q"][ofs[b]:ofs[b + 1]].double().view(rows, hk, hq // hk, d)
        q = q.permute(1, 2, 0, 3).reshape(hk, -1, d)
        x = (q @ k.transpose(1, 2) * s["scale"]).view(hk, hq // hk, rows, n)
        if c["op"] == "tree":
            hide = torch.ones((rows, rows), dtype=torch.bool, device=DEV).triu(1)
            if s["tree_mask"] is not None:
                words = s["tree_mask"][ofs[b]:ofs[b + 1]].tolist()
                hide = torch.tensor([[not (w >> j) & 1 for j in range(rows)] for w in words], device=DEV)
            x[..., n - rows:] = x[..., n - rows:].masked_fill(hide, -math.inf)
        w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
        o = (w.view(hk, -1, n) @ v).view(hk, hq // hk, rows, d)
        out[ofs[b]:ofs[b + 1]] = o.permute(2, 0, 1, 3).reshape(rows, hq, d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "read":
        return _exact_read(s)
    if case["op"] == "write":
        return _exact_write(s)
    return _exact_attention(s)

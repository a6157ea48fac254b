"""Measured cases of the library's operators around prompts and drafts.

* ``extend``   attention of each sequence's new tokens (a prompt, a chunk of one,
               or one decoded token) over its paged context, with scores capped
               by a tanh, biased by distance, and limited by a window, a prefix
               or documents (``pk_paged_attention_extend``);
* ``verify``   drafted tokens, a chain or a tree, accepted or rejected against
               the target's probabilities by given random numbers, and the next
               token drawn (``pk_verify_drafts``);
* ``compact``  the cached keys and values of the accepted drafts moved together
               (``pk_compact_drafts``).

With ``own`` false ``run`` computes an operator in its plain form: elementary
torch operations in fp32 (verification in fp64: its sums decide whole numbers),
rounded once at the end. With ``own`` true it makes the library's calls.
``exact`` computes the definition in fp64, sequence by sequence.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases. Head layouts, block sizes, context lengths and batches are those of
# the library's own workloads (tiny, mha7b, gqa8b, long, prefix).
# ---------------------------------------------------------------------------
def _ext(name, seqs, hq, hk, d, dtype, blk, lens, lo, hi, new, cap=0.0, window=0, slopes=False, prefix=0, doc=0):
    """`new` 0: whole prompts of the drawn lengths; else so many new tokens at most."""
    return {"name": name, "op": "extend", "seqs": seqs, "hq": hq, "hk": hk, "d": d, "dtype": dtype, "blk": blk,
            "lens": lens, "lo": lo, "hi": hi, "new": new, "cap": cap, "window": window, "slopes": slopes,
            "prefix": prefix, "doc": doc}


def _ver(name, seqs, draft, vocab, dtype, mask):
    return {"name": name, "op": "verify", "seqs": seqs, "draft": draft, "vocab": vocab, "dtype": dtype, "mask": mask}


def _com(name, seqs, hk, d, dtype, blk, draft, lo, hi):
    return {"name": name, "op": "compact", "seqs": seqs, "hk": hk, "d": d, "dtype": dtype, "blk": blk, "draft": draft,
            "lo": lo, "hi": hi}


def listed():
    return [
        # One decode step of the 8B-like batch, heavy-tailed lengths, capped scores.
        _ext("decode cap 256", 256, 32, 8, 128, "bf16", 16, "tail", 33, 4608, 1, cap=50.0),
        # One decode step of eight 32K contexts with a bias of distance per head.
        _ext("decode slopes 8x32768", 8, 64, 8, 128, "bf16", 16, "even", 32768, 32768, 1, slopes=True),
        # One decode step of a layer that sees the last 1024 tokens, a KV head per query head.
        _ext("decode window 64", 64, 32, 32, 128, "bf16", 16, "even", 1000, 4000, 1, window=1024),
        # Four short fp32 prompts.
        _ext("prompt tiny f32", 4, 8, 8, 64, "f32", 16, "even", 1, 100, 0, slopes=True),
        # Eight prompts of 2000 tokens whose first 500 see one another, capped scores.
        _ext("prompt prefix cap 8x2000", 8, 32, 8, 128, "bf16", 16, "even", 2000, 2000, 0, cap=50.0, prefix=500),
        # 16384 tokens of packed documents of 1000 tokens or so.
        _ext("documents 16384", 1, 32, 8, 128, "bf16", 16, "even", 16384, 16384, 0, doc=1000),
        # The last 512 tokens of two 32K prompts, capped scores.
        _ext("chunk cap 2x512 of 32768", 2, 64, 8, 128, "bf16", 16, "even", 32768, 32768, 512, cap=30.0),
        # Four sequences with four drafts each: latency counts.
        _ver("verify 4x4", 4, 4, 32000, "f32", "chain"),
        # The 8B-like batch with eight sampled drafts each.
        _ver("verify chain 256x8", 256, 8, 32000, "f32", "chain"),
        # 64 sequences with trees of 16 drafts, a vocabulary of 128 000.
        _ver("verify tree 64x16", 64, 16, 128000, "f32", "tree"),
        # Four short fp32 sequences with eight drafts.
        _com("compact tiny f32", 4, 8, 64, "f32", 16, 8, 9, 100),
        # The 8B-like batch, 16 drafts each, half of them kept.
        _com("compact 256x16", 256, 8, 128, "bf16", 16, 16, 33, 160),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["extend", "extend", "extend", "verify", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    blk = rng.choice([8, 16, 32])
    if op == "verify":
        draft, vocab = _log(rng, 1, 63), _log(rng, 1000, 160000)
        seqs = _log(rng, 1, max(1, min(256, 130_000_000 // (vocab * (draft + 1)))))
        return _ver(op, seqs, draft, vocab, rng.choice(["f32", "f32", "bf16"]), rng.choice(["chain", "greedy", "tree"]))
    hk = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    if op == "compact":
        draft = _log(rng, 1, 63)
        return _com(op, _log(rng, 1, 256), hk, d, dtype, blk, draft, draft + 1, draft + 1 + _log(rng, 1, 150))
    hq = hk * rng.choice([1, 2, 3, 4, 5, 7, 8])
    new = rng.choice([1, 1, 0, 0, _log(rng, 2, 700)])
    seqs = _log(rng, 1, 256 if new == 1 else 16)
    # Scores and cached tokens stay below those of the largest listed cases.
    flops = 2.5e11 if dtype == "bf16" else 2e10
    cap = (262144 if dtype == "bf16" else 65536) * 8 // hk // seqs
    if new == 0:
        cap = min(cap, int(math.sqrt(flops / (2.0 * d * hq * seqs))))
    else:
        cap = min(cap, int(flops / (4.0 * d * hq * seqs * new)))
    hi = _log(rng, 33, max(34, min(32768, cap)))
    lo = _log(rng, 1, hi)
    window = _log(rng, 1, 4096) if rng.random() < 0.35 else 0
    doc = _log(rng, 5, 2000) if rng.random() < 0.25 else 0
    prefix = _log(rng, 1, hi) if rng.random() < 0.25 else 0
    return _ext(op, seqs, hq, hk, d, dtype, blk, rng.choice(["even", "tail", "one long"]), lo, hi, new,
                cap=rng.choice([0.0, 30.0, 50.0]), window=window, slopes=rng.random() < 0.35, prefix=prefix, doc=doc)


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


def _tables(g, lens, blk):
    nb = (lens + blk - 1) // blk
    maxb = int(nb.max())
    total = int(nb.sum())
    order = torch.randperm(total, generator=g).int()
    tables = torch.full((len(lens), maxb), -1, dtype=torch.int32)
    at = torch.arange(maxb)[None] < nb[:, None]
    tables[at] = order
    return tables, total


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])


def _prepare_extend(case, g, gen):
    s = {}
    dt, S, hq, d = DTYPES[case["dtype"]], case["seqs"], case["hq"], case["d"]
    lens = _lengths(case, g)
    counts = lens.clone() if case["new"] == 0 else lens.clamp_max(case["new"])
    if case["new"] > 1 and case["lo"] != case["hi"]:  # ragged chunks
        counts = torch.minimum(lens, 1 + (torch.rand(S, generator=g) * case["new"]).long())
    offsets = _offsets(counts)
    # A fixed batch buffer: the rows behind the last sequence's are padding.
    rows = S * (case["hi"] if case["new"] == 0 else min(case["new"], case["hi"]))
    tables, total = _tables(g, lens, case["blk"])
    s["lens_host"], s["counts_host"] = lens.tolist(), counts.tolist()
    s["tables"], s["lens"], s["max_len"] = tables.to(DEV), lens.int().to(DEV), int(lens.max())
    s["q_offsets"], s["max_new"] = (None if case["new"] == 1 else offsets.int().to(DEV)), int(counts.max())
    s["scale"] = 1.0 / math.sqrt(d)
    # Queries somewhat larger than unit: scores reach into the cap's bend.
    s["q"] = (_rand(gen, (rows, hq, d)) * 2.0).to(dt)
    s["k_cache"] = _rand(gen, (total, case["blk"], case["hk"], d), dt)
    s["v_cache"] = _rand(gen, (total, case["blk"], case["hk"], d), dt)
    s["out"] = torch.zeros_like(s["q"])
    s["slopes"] = s["prefix_lens"] = s["first_tokens"] = None
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, dtype=torch.float64) / hq).float().to(DEV)
    if case["prefix"]:
        most = lens.clamp_max(case["prefix"])
        pre = most if case["lo"] == case["hi"] else (torch.rand(S, generator=g) * (most + 1)).long()
        s["prefix_lens"] = pre.int().to(DEV)
    if case["doc"]:
        # Where the document of each new token begins: boundaries about `doc` tokens apart.
        longest = int(lens.max())
        cuts = (0.5 + torch.rand(longest // max(1, case["doc"] // 2) + 2, generator=g)) * case["doc"]
        cuts = torch.cat([torch.zeros(1), cuts.cumsum(0)]).long()
        pos = torch.cat([torch.arange(n - c, n) for n, c in zip(lens.tolist(), counts.tolist())])
        s["first_tokens"] = torch.zeros(rows, dtype=torch.int32, device=DEV)
        s["first_tokens"][:len(pos)] = cuts[torch.searchsorted(cuts, pos, right=True) - 1].int().to(DEV)
    if own:  # the plan and the workspace that a serving loop keeps beside its batch
        import paged_kv_cache_113_gb300 as pk
        desc = pk.cache_desc(s["k_cache"])
        s["partition"], items = pk.pk_extend_plan(lens.numpy(), counts.numpy(), hq, desc, -1, window=case["window"])
        ws = pk.pk_extend_workspace_size(rows, hq, s["max_len"], s["partition"], desc)
        s["items"] = torch.from_numpy(items).to(DEV)
        s["workspace"] = torch.empty(max(ws, 16), dtype=torch.uint8, device=DEV)
    return s


def _prepare_verify(case, g, gen):
    s = {}
    S, V, dt = case["seqs"], case["vocab"], DTYPES[case["dtype"]]
    # Rows: each sequence's root, then its drafts.
    counts = 2 + (torch.rand(S, generator=g) * case["draft"]).long()
    counts[0] = case["draft"] + 1
    offsets = _offsets(counts)
    # A fixed batch buffer: the rows behind the last sequence's are padding, of one more node 0 each.
    rows = S * (case["draft"] + 1)
    used = int(offsets[-1])
    first = torch.cat([offsets[:-1].repeat_interleave(counts), torch.arange(used, rows)])
    node = torch.arange(rows) - first
    if case["mask"] == "tree":
        parents = (torch.rand(rows, generator=g) * node).long().clamp_min(0)
    else:
        parents = (node - 1).clamp_min(0)
    at = (first + parents).to(DEV)                               # the row that a draft's token is judged by
    logits = _rand(gen, (rows, V)) * 4.0
    s["target_probs"] = torch.softmax(logits, -1).to(dt)
    s["draft_probs"] = None
    if case["mask"] == "chain":                                  # drafted by a model near the target's
        near = logits[at] + _rand(gen, (rows, V))
        s["draft_probs"] = torch.softmax(near, -1).to(dt)
        tokens = torch.multinomial(torch.softmax(near, -1), 1, generator=gen)[:, 0]
    else:                                                        # the likely tokens of the parent's row
        rank = torch.zeros(rows, dtype=torch.long)
        seen = {}
        for r, p in enumerate((first + parents).tolist()):
            rank[r] = seen.get(p, 0)
            if int(node[r]):
                seen[p] = int(rank[r]) + 1
        top = torch.topk(logits, min(V, int(rank.max()) + 1), dim=-1).indices
        tokens = top[at, rank.to(DEV)]
    s["tokens"] = tokens
    s["uniforms"] = torch.rand(rows, generator=gen, device=DEV)
    s["parents"] = parents.int().to(DEV) if case["mask"] == "tree" else None
    s["q_offsets"], s["max_rows"], s["rows"] = offsets.int().to(DEV), int(counts.max()), rows
    s["num_accepted"] = torch.zeros(S, dtype=torch.int32, device=DEV)
    s["accepted"] = torch.zeros(rows, dtype=torch.int32, device=DEV)
    s["next_tokens"] = torch.zeros(S, dtype=torch.int64, device=DEV)
    return s


def _prepare_compact(case, g, gen):
    s = {}
    S, dt, blk = case["seqs"], DTYPES[case["dtype"]], case["blk"]
    lens = case["lo"] + torch.randint(0, case["hi"] - case["lo"] + 1, (S,), generator=g)
    counts = torch.full((S,), case["draft"] + 1).clamp_max(case["lo"])   # the root and its drafts
    offsets = _offsets(counts)
    rows = int(offsets[-1])
    accepted = torch.full((rows,), -1, dtype=torch.int32)
    kept = []
    for b, n in enumerate(counts.tolist()):                      # half of the drafts, in order
        a = n // 2
        path = [0] + sorted((1 + torch.randperm(n - 1, generator=g)[:a]).tolist()) if n > 1 else [0]
        accepted[int(offsets[b]):int(offsets[b]) + len(path)] = torch.tensor(path, dtype=torch.int32)
        kept.append(len(path) - 1)
    tables, _ = _tables(g, lens, blk)
    total = S * -(-case["hi"] // blk)
    s["tables"], s["lens"] = tables.to(DEV), lens.int().to(DEV)
    s["q_offsets"], s["max_rows"] = offsets.int().to(DEV), int(counts.max())
    s["accepted"], s["num_accepted"] = accepted.to(DEV), torch.tensor(kept, dtype=torch.int32, device=DEV)
    s["k_cache"] = _rand(gen, (total, blk, case["hk"], case["d"]), dt)
    s["v_cache"] = _rand(gen, (total, blk, case["hk"], case["d"]), dt)
    s["lens_out"] = torch.zeros(S, dtype=torch.int32, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed + 1)
    make = {"extend": _prepare_extend, "verify": _prepare_verify, "compact": _prepare_compact}[case["op"]]
    return {"case": case, "op": case["op"], **make(case, g, gen)}


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _own_extend(s):
    import paged_kv_cache_113_gb300 as pk
    c = s["case"]
    pk.pk_paged_attention_extend(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["q_offsets"],
                                 s["scale"], s["max_new"], s["max_len"], softcap=c["cap"], window=c["window"],
                                 slopes=s["slopes"], prefix_lens=s["prefix_lens"], first_tokens=s["first_tokens"],
                                 partition_size=s["partition"], workspace=s["workspace"], work_items=s["items"])
    return s["out"]


def _own_verify(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_verify_drafts(s["num_accepted"], s["accepted"], s["next_tokens"], s["target_probs"], s["tokens"],
                        s["uniforms"], s["q_offsets"], s["max_rows"], parents=s["parents"],
                        draft_probs=s["draft_probs"])
    return {"num_accepted": s["num_accepted"], "accepted": s["accepted"], "next_tokens": s["next_tokens"]}


def _own_compact(s):
    import paged_kv_cache_113_gb300 as pk
    pk.pk_compact_drafts(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["q_offsets"], s["accepted"],
                         s["num_accepted"], s["max_rows"], context_lens_out=s["lens_out"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens_out"]}


def _plain_scores(s, x, pos, t, slopes):
    """x [..., Hk, G, n, t] products with the scale; pos [..., n], t [t] positions; slopes [Hk, G]."""
    if s["case"]["cap"]:
        x = torch.tanh(x / s["case"]["cap"]) * s["case"]["cap"]
    if slopes is not None:
        away = (pos[..., None] - t).abs().float()[..., None, None, :, :]
        x = x - slopes[:, :, None, None] * away
    return x


def _plain_softmax(x, see):
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p / p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_extend(s):
    c = s["case"]
    hk, hq, d, blk = c["hk"], c["hq"], c["d"], c["blk"]
    G = hq // hk
    slopes = None if s["slopes"] is None else s["slopes"].view(hk, G)
    if c["new"] == 1:  # decode: the whole batch at once, padded to the longest
        S, T = s["tables"].shape[0], s["tables"].shape[1] * blk
        tables = s["tables"].clamp_min(0).long()
        k, v = (s[x][tables].view(S, T, hk, d).float() for x in ("k_cache", "v_cache"))
        pos, t = s["lens"].long() - 1, torch.arange(T, device=DEV)
        hi = pos + 1 if s["prefix_lens"] is None else torch.maximum(pos + 1, torch.minimum(s["prefix_lens"], s["lens"]))
        lo = torch.zeros_like(pos) if s["first_tokens"] is None else s["first_tokens"].long()
        if c["window"]:
            lo = torch.maximum(lo, pos + 1 - c["window"])
        x = torch.matmul(s["q"].float().view(S, hk, G, d), k.permute(0, 2, 3, 1)) * s["scale"]
        x = _plain_scores(s, x[:, :, :, None], pos[:, None], t, slopes)
        see = (t >= lo[:, None]) & (t < hi[:, None])
        p = _plain_softmax(x, see[:, None, None, None])[:, :, :, 0]
        s["out"].copy_(torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(S, hq, d))
        return s["out"]
    row = 0
    for b, (n, new) in enumerate(zip(s["lens_host"], s["counts_host"])):
        blocks = s["tables"][b, :-(-n // blk)].long()
        k, v = (s[x][blocks].view(-1, hk, d)[:n].float().transpose(0, 1) for x in ("k_cache", "v_cache"))
        step = max(1, 200_000_000 // (hq * n))                   # rows at a time: some GB of scores
        for r in range(0, new, step):
            m = min(step, new - r)
            pos, t = torch.arange(n - new + r, n - new + r + m, device=DEV), torch.arange(n, device=DEV)
            hi = pos + 1 if s["prefix_lens"] is None else torch.maximum(pos + 1, s["prefix_lens"][b].clamp_max(n))
            lo = torch.zeros_like(pos) if s["first_tokens"] is None else s["first_tokens"][row + r:row + r + m].long()
            if c["window"]:
                lo = torch.maximum(lo, pos + 1 - c["window"])
            q = s["q"][row + r:row + r + m].float().view(m, hk, G, d).permute(1, 2, 0, 3)
            x = torch.matmul(q.reshape(hk, G * m, d), k.transpose(1, 2)).view(hk, G, m, n) * s["scale"]
            x = _plain_scores(s, x, pos, t, slopes)
            p = _plain_softmax(x, (t >= lo[:, None]) & (t < hi[:, None]))
            o = torch.matmul(p.view(hk, G * m, n), v).view(hk, G, m, d)
            s["out"][row + r:row + r + m] = o.permute(2, 0, 1, 3).reshape(m, hq, d).to(s["out"].dtype)
        row += new
    return s["out"]


def _weight(x):
    """Probabilities in fp64; what is not a positive finite number counts as 0."""
    x = x.double()
    return torch.where((x > 0) & torch.isfinite(x), x, torch.zeros_like(x))


def _plain_verify(s):
    first, count = s["q_offsets"][:-1].long(), s["q_offsets"].diff().long()
    S, V, n = len(first), s["case"]["vocab"], s["max_rows"]
    i = torch.arange(n, device=DEV)
    live = i < count[:, None]                                    # [S, n]
    row = torch.where(live, first[:, None] + i, first[:, None])
    parent = (i - 1).clamp_min(0).expand(S, n) if s["parents"] is None else s["parents"].long()[row]
    parent = torch.where(live, parent, torch.zeros_like(parent))
    token = s["tokens"][row]
    p = _weight(s["target_probs"][first[:, None] + parent, token])
    q = None if s["draft_probs"] is None else _weight(s["draft_probs"][row, token])
    cur = torch.zeros(S, dtype=torch.long, device=DEV)
    mass = torch.ones(S, dtype=torch.float64, device=DEV)
    refused = torch.zeros((S, n), dtype=torch.bool, device=DEV)  # nodes rejected at the node where the walk stands
    path = torch.zeros((S, n), dtype=torch.bool, device=DEV)
    path[:, 0] = True
    u = s["uniforms"][row].double()
    for j in range(1, n):
        here = live[:, j] & (parent[:, j] == cur)
        again = (refused & (token == token[:, j:j + 1])).any(1)
        pj = torch.where(again, torch.zeros_like(mass), p[:, j])
        yes = here & (u[:, j] * (mass if q is None else q[:, j]) < pj)
        no = here & ~yes
        path[:, j] = yes
        refused[yes] = False
        refused[:, j] = no
        mass = torch.where(yes, torch.ones_like(mass), torch.where(no, mass - pj, mass))
        cur = torch.where(yes, j, cur)
    w = _weight(s["target_probs"][first + cur])                  # [S, V]
    full = w
    if q is None:
        rest = torch.zeros_like(w).scatter_reduce_(1, token, refused.double(), "amax")
        w = torch.where(rest > 0, torch.zeros_like(w), w)
    else:
        at = torch.where(refused.any(1), first + refused.double().argmax(1), first)
        w = torch.where(refused.any(1)[:, None], (w - _weight(s["draft_probs"][at])).clamp_min(0), w)
    w = torch.where((w.sum(1) > 0)[:, None], w, full)
    c = w.cumsum(1)
    nxt = torch.searchsorted(c, u[:, :1] * c[:, -1:], right=True)[:, 0].clamp_max(V - 1)
    s["next_tokens"].copy_(torch.where(c[:, -1] > 0, nxt, torch.full_like(nxt, -1)))
    s["num_accepted"].copy_(path.sum(1) - 1)
    order = torch.argsort(torch.where(path, i.expand(S, n), n + i), dim=1)  # the path's nodes first, in order
    kept = torch.where(i < path.sum(1, keepdim=True), order, torch.full_like(order, -1))
    s["accepted"][row[live]] = kept[live].int()
    return {"num_accepted": s["num_accepted"], "accepted": s["accepted"], "next_tokens": s["next_tokens"]}


def _plain_compact(s):
    c = s["case"]
    first, count = s["q_offsets"][:-1].long(), s["q_offsets"].diff().long()
    i = torch.arange(s["max_rows"], device=DEV)
    live = i < torch.minimum(count, s["num_accepted"] + 1)[:, None]
    kept = s["accepted"][torch.where(live, first[:, None] + i, first[:, None])].long().clamp_min(0)
    base = (s["lens"].long() - count)[:, None]

    def slots(t):
        return (s["tables"].long().gather(1, t // c["blk"]) * c["blk"] + t % c["blk"])[live]

    src = slots(torch.where(live, base + kept, base))
    dst = slots(torch.where(live, base + i, base))
    for name in ("k_cache", "v_cache"):
        pool = s[name].view(-1, c["hk"], c["d"])
        pool[dst] = pool[src]
    s["lens_out"].copy_(base[:, 0] + s["num_accepted"] + 1)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens_out"]}


_PLAIN = {"extend": _plain_extend, "verify": _plain_verify, "compact": _plain_compact}
_OWN = {"extend": _own_extend, "verify": _own_verify, "compact": _own_compact}


# ---------------------------------------------------------------------------
# What the path cannot do without
# ---------------------------------------------------------------------------
def _mean_length(case):
    """Expected context length of a case (its seed is not known here)."""
    S, lo, hi = case["seqs"], case["lo"], case["hi"]
    if case["lens"] == "even":
        return (lo + hi) / 2
    if case["lens"] == "tail":
        return min(max(472.0, lo), hi)
    return ((S - 1) * (lo + max(0, (hi - lo) // 8 - 1) / 2) + hi) / S


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "verify":
        S, n, V = case["seqs"], (case["draft"] + 3) / 2, case["vocab"]
        two = 1 if case["mask"] != "chain" else 2
        return {"bytes": S * V * e * two + S * n * (e * two + 20) + S * 12, "flops": S * V * (2.0 + two)}
    if case["op"] == "compact":
        # Of the half that is kept, all but about one draft have a new place.
        moved = case["seqs"] * max(0.0, (min(case["draft"] + 1, case["lo"]) // 2) - 1.0)
        return {"bytes": moved * 4 * case["hk"] * case["d"] * e + case["seqs"] * (16 + 4 * case["draft"]), "flops": 0}
    S, hq, hk, d, n = case["seqs"], case["hq"], case["hk"], case["d"], _mean_length(case)
    new = n if case["new"] == 0 else min(case["new"], n)
    if case["new"] > 1 and case["lo"] != case["hi"]:
        new = min(n, (case["new"] + 1) / 2)
    # Tokens that a row sees on average, and the sequence's that any row sees.
    sees = n - (new - 1) / 2
    if case["prefix"]:
        pre = min(case["prefix"], n) / (1 if case["lo"] == case["hi"] else 2)
        inside = max(0.0, pre - (n - new))                       # new tokens within the prefix
        sees += inside * inside / 2 / new
    union = n
    for most, mean in ((case["window"], 1.0), (case["doc"], 0.54)):
        if most:
            sees, union = min(sees, most * mean), min(union, most + new)
    return {"bytes": S * (union * hk * 2 * d * e + 2 * new * hq * d * e), "flops": 4.0 * S * new * sees * hq * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_extend(s):
    c = s["case"]
    hk, hq, d, blk = c["hk"], c["hq"], c["d"], c["blk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, new) in enumerate(zip(s["lens_host"], s["counts_host"])):
        pool = (s["tables"][b].long()[:, None] * blk + torch.arange(blk, device=DEV)).flatten()[:n]
        k, v = (s[x].view(-1, hk, d).index_select(0, pool).double() for x in ("k_cache", "v_cache"))
        position = torch.arange(n - new, n, device=DEV)
        begin = torch.zeros(new, dtype=torch.long, device=DEV)
        if c["doc"]:
            begin = s["first_tokens"][at:at + new].long()
        if c["window"]:
            begin = torch.stack([begin, position - c["window"] + 1]).amax(0).clamp_min(0)
        stop = position + 1
        if c["prefix"]:
            stop = stop.clamp_min(min(int(s["prefix_lens"][b]), n))
        chunk = 1024
        for r in range(0, new, chunk):
            rows = slice(r, min(new, r + chunk))
            left, right = int(begin[rows].min()), int(stop[rows].max())  # nobody here sees what is outside
            t = torch.arange(left, right, device=DEV)
            hidden = (t < begin[rows, None]) | (t >= stop[rows, None])
            for h in range(hq):
                x = s["q"][at:at + new][rows, h].double() @ k[left:right, h * hk // hq].T
                x = x * s["scale"]
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["slopes"]:
                    x = x - float(s["slopes"][h]) * (position[rows, None] - t).abs()
                w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
                out[at:at + new][rows, h] = torch.nan_to_num(w, nan=0.0) @ v[left:right, h * hk // hq]
        at += new
    return out


def _exact_verify(s):
    """One sequence after the other, walking down from its root."""
    offsets, tokens = s["q_offsets"].tolist(), s["tokens"].tolist()
    uniforms = s["uniforms"].double().tolist()
    accepted, counts, nexts = [0] * s["rows"], [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        children = {}
        for r in range(a + 1, b):
            up = a + int(s["parents"][r]) if s["parents"] is not None else r - 1
            children.setdefault(up, []).append(r)
        node, path = a, [a]
        while True:
            p = s["target_probs"][node].double()
            p = torch.where(torch.isfinite(p) & (p > 0), p, torch.zeros_like(p))
            left, weights, down = 1.0, p.clone(), None
            for r in children.get(node, []):
                pr = float(weights[tokens[r]]) if s["draft_probs"] is None else float(p[tokens[r]])
                limit = left if s["draft_probs"] is None else float(s["draft_probs"][r, tokens[r]].double())
                if uniforms[r] * limit < pr:
                    down = r
                    break
                left -= pr
                if s["draft_probs"] is None:
                    weights[tokens[r]] = 0
                else:
                    weights = (p - s["draft_probs"][r].double()).clamp_min(0)
            if down is None:
                break
            node = down
            path.append(down)
        if float(weights.sum()) == 0:
            weights = p
        total = torch.cumsum(weights, 0)
        above = torch.nonzero(total > uniforms[a] * float(total[-1]))
        nexts.append(int(above[0]) if len(above) else -1)
        counts.append(len(path) - 1)
        accepted[a:b] = [r - a for r in path] + [-1] * (b - a - len(path))
    return {"num_accepted": torch.tensor(counts, device=DEV), "accepted": torch.tensor(accepted, device=DEV),
            "next_tokens": torch.tensor(nexts, device=DEV)}


def _exact_compact(s):
    c = s["case"]
    k, v = s["k_cache"].double().view(-1, c["hk"], c["d"]), s["v_cache"].double().view(-1, c["hk"], c["d"])
    lens, offsets, kept = s["lens"].tolist(), s["q_offsets"].tolist(), s["accepted"].tolist()
    tables, counts, out = s["tables"].tolist(), s["num_accepted"].tolist(), []
    src, dst = [], []
    for b, n in enumerate(lens):
        base = n - (offsets[b + 1] - offsets[b])
        for i in range(counts[b] + 1):
            for where, t in ((src, base + kept[offsets[b] + i]), (dst, base + i)):
                where.append(tables[b][t // c["blk"]] * c["blk"] + t % c["blk"])
        out.append(base + counts[b] + 1)
    src, dst = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
    for pool in (k, v):
        pool.index_copy_(0, dst, pool.index_select(0, src))
    return {"k_cache": k.view(s["k_cache"].shape), "v_cache": v.view(s["v_cache"].shape),
            "lens": torch.tensor(out, device=DEV)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "verify": _exact_verify, "compact": _exact_compact}[case["op"]](s)

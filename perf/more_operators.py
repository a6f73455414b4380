"""Cases, plain forms and exact values of a speculative step's operators.

What a serving step with drafted tokens runs on the paged cache around the
decode, the append and the prefill:

* ``tables``  block tables, row starts, positions and slots of the next step
              from request lengths and a free list of pages (``vt.step_tables``);
* ``masks``   bit masks and positions of trees of drafted tokens from their
              parents (``vt.tree_masks``);
* ``norm``    RMS norm of each query and key head, its rotation and the append
              in one pass (``vt.norm_append``, ``vt.norm_append_fp8``), and norm
              and rotation alone (``vt.norm_rope``);
* ``tree``    attention of trees of drafted tokens over the paged cache
              (``vt.prefill_tree``, ``vt.prefill_tree_fp8``);
* ``keep``    the accepted branch's keys and values moved to consecutive slots,
              all layers at once (``vt.keep_path``).

Rows of a batch are packed: sequence b owns rows q_starts[b] to
q_starts[b + 1], the last n_b of its context_lens[b] tokens; rows behind the
last sequence are padding and stay as they were.
"""
import math
import random

import torch

own = False

PAGE = 32
E4M3_MAX = 448.0
_TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(op, **kw):
    c = dict(op=op, dtype="bf16", q_heads=32, kv_heads=8, head_dim=128, seqs=1, new_lo=1, new_hi=1, ctx_lo=0,
             ctx_hi=0, pad=0)
    if op == "tables":
        c.update(finished=0)            # sequences that end in this step
    if op in ("masks", "tree", "keep"):
        c.update(reach=4)               # a token's parent is among the `reach` before it, or the context
    if op == "tree":
        c.update(window=0, mask="tree")
    if op == "keep":
        c.update(layers=1)
    if op == "norm":
        c.update(append=True, rot=128, interleaved=False, base=1e6, per_head=False)
    c.update(kw)
    return c


def listed():
    return [
        # A decode step's bookkeeping: 256 running sequences, one new token each.
        _case("tables", name="tables_b256_decode", seqs=256, ctx_lo=1, ctx_hi=8000),
        # Prompts admitted (about 33 thousand tokens) while 40 sequences end and give their pages back.
        _case("tables", name="tables_prompts_33k", seqs=72, finished=40, new_lo=200, new_hi=1900, ctx_lo=0,
              ctx_hi=8000, pad=29),
        # Trees of drafted tokens of one batch.
        _case("masks", name="masks_b64_n24_64", seqs=64, new_lo=24, new_hi=64, ctx_lo=512, ctx_hi=8000, reach=6),
        # Many wide trees: 256 tokens each, some branches long.
        _case("masks", name="masks_b256_n200_256", seqs=256, new_lo=200, new_hi=256, ctx_lo=0, ctx_hi=4000, reach=2,
              pad=11),
        # A decode step's queries and keys of a 128-sequence batch: latency.
        _case("norm", name="norm_append_b128_gqa4_d128", seqs=128, ctx_lo=64, ctx_hi=2048),
        # Prompts of odd lengths into a cache of 8-bit codes, 64 query heads: bandwidth.
        _case("norm", name="norm_append_fp8_prompts_gqa8_d128", dtype="e4m3", q_heads=64, seqs=12, new_lo=257,
              new_hi=1700, ctx_lo=0, ctx_hi=700, pad=13),
        # One sequence's tree over a context of some thousand tokens: latency (head_dim 64).
        _case("tree", name="tree_b1_n26_gqa4_d64", q_heads=16, kv_heads=4, head_dim=64, new_lo=26, new_hi=26,
              ctx_lo=3000, ctx_hi=4500),
        # A batch's trees over long contexts (the largest case).
        _case("tree", name="tree_b64_n24_64_gqa4_d128", seqs=64, new_lo=24, new_hi=64, ctx_lo=512, ctx_hi=8000,
              reach=6),
        # Small trees of a large-GQA batch over a cache of 8-bit codes, with padding rows.
        _case("tree", name="tree_fp8_b32_n4_12_gqa8_d128", dtype="e4m3", q_heads=64, seqs=32, new_lo=4, new_hi=12,
              ctx_lo=1000, ctx_hi=16000, pad=5),
        # head_dim 256 with a sliding window.
        _case("tree", name="tree_d256_gqa4_w1024", q_heads=8, kv_heads=2, head_dim=256, seqs=16, new_lo=8, new_hi=40,
              ctx_lo=0, ctx_hi=4096, window=1024),
        # The accepted branches of 8 sequences in one layer's pages: latency.
        _case("keep", name="keep_b8_gqa4_d128", seqs=8, new_lo=12, new_hi=40, ctx_lo=10, ctx_hi=500),
        # The accepted branches of a batch in all of 16 layers at once.
        _case("keep", name="keep_b64_16_layers_d128", seqs=64, new_lo=24, new_hi=64, ctx_lo=10, ctx_hi=200, layers=16,
              reach=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5)))


def draw(rng):
    op = rng.choice(["tables", "masks", "norm", "norm", "tree", "tree", "tree", "keep"])
    dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    head_dim = rng.choice([64, 128, 256] + ([512] if dtype == "bf16" else []))
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    kw = dict(dtype=dtype, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, pad=pad)
    ctx = _log(rng, 1, 12000)
    if op == "tables":
        c = _case(op, pad=pad, seqs=_log(rng, 1, 600), new_hi=_log(rng, 1, 1000), ctx_hi=ctx)
        c["finished"] = rng.randint(0, c["seqs"] - 1) if rng.random() < 0.5 else 0
    elif op == "norm":
        c = _case(op, seqs=_log(rng, 1, 96), new_hi=_log(rng, 1, 3000), ctx_hi=ctx, append=rng.random() < 0.7,
                  interleaved=rng.random() < 0.4, base=rng.choice([1e4, 5e5, 1e6]), per_head=rng.random() < 0.3,
                  rot=rng.choice([head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]), **kw)
        if not c["append"] and dtype == "e4m3":
            c["dtype"] = "bf16"
        while c["seqs"] > 1 and c["seqs"] * c["new_hi"] * (q_heads + 2 * kv_heads) * head_dim > 1 << 25:
            c["seqs"] //= 2
        while c["seqs"] > 1 and c["seqs"] * (c["new_hi"] + ctx) * kv_heads * head_dim > 1 << 27:
            c["seqs"] //= 2
        while c["new_hi"] * (q_heads + 2 * kv_heads) * head_dim > 1 << 25:
            c["new_hi"] = c["new_hi"] * 2 // 3
    elif op == "masks":
        c = _case(op, pad=pad, seqs=_log(rng, 1, 200), new_hi=_log(rng, 1, 300), ctx_hi=ctx, reach=_log(rng, 1, 40))
    else:
        c = _case(op, seqs=_log(rng, 1, 64), new_hi=_log(rng, 1, 150 if op == "tree" else 64), ctx_hi=ctx,
                  reach=_log(rng, 1, 40), **kw)
        if op == "tree":
            if rng.random() < 0.3:
                c["window"] = _log(rng, 1, 4096)
            c["mask"] = rng.choice(["tree", "tree", "any"])
            # No dearer than the largest listed case: the padded score matrix of the plain form, the pages.
            room = {"bf16": 1 << 29, "e4m3": 1 << 29, "f32": 1 << 26}[dtype]
            while c["seqs"] > 1 and (c["seqs"] * q_heads * c["new_hi"] * (c["new_hi"] + ctx) > room
                                     or c["seqs"] * (c["new_hi"] + ctx) * kv_heads * head_dim > 1 << 26):
                c["seqs"] //= 2
        else:
            c["layers"] = rng.choice([1, 1, 2, 5, 12])
            c["ctx_hi"] = min(ctx, 400)
            while c["seqs"] > 1 and c["seqs"] * c["layers"] * (c["ctx_hi"] + 64) * kv_heads * head_dim > 1 << 27:
                c["seqs"] //= 2
    c["new_lo"] = rng.choice([c["new_hi"], 0 if c["seqs"] > 1 else 1, max(1, c["new_hi"] // 2)])
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 2, c["ctx_hi"]])
    return c


def _lengths(case):
    """New tokens and contexts of each sequence: the case's own, whatever the seed of its contents."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    if sum(new) == 0:
        new[0] = max(1, case["new_hi"])
    ctx = [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in new]
    return new, ctx


def _parents(case, new):
    """A drafted token's parent: its index within its sequence, -1 for the context."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "parents")
    out = []
    for n in new:
        out.append([])
        for j in range(n):
            out[-1].append(rng.randint(max(-1, j - case["reach"]), j - 1) if rng.random() < 0.9 else max(-1, j - 1))
    return out


def _branch(parents, j):
    """Token j and those it follows, in ascending order."""
    path = []
    while j >= 0:
        path.append(j)
        j = parents[j]
    return path[::-1]


def _ancestors(case, new):
    """For each sequence the tokens that each drafted token sees, in ascending order."""
    if case.get("mask") == "any":  # masks that are no trees: some rows see nothing, some tokens after their own
        rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "any")
        return [[sorted(rng.sample(range(n), rng.randint(0, n))) if rng.random() < 0.8 else [] for _ in range(n)]
                for n in new]
    return [[_branch(p, j) for j in range(n)] for p, n in zip(_parents(case, new), new)]


def _accepted(case, new):
    """The accepted token of each sequence (-1: none): the end of its longest branch among those whose tokens do not
    lie in slots that the branch is written to, or are in place, so that a pass can be repeated."""
    out = []
    for rows in _ancestors(case, new):
        best = -1
        for j, path in enumerate(rows):
            k = len(path)
            if all(i == r or i >= k for r, i in enumerate(path)) and (best < 0 or k > len(rows[best])):
                best = j
        out.append(best)
    return out


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def _plan(case):
    """tables: tokens kept, tokens new and tokens before this step of each sequence."""
    new, ctx = _lengths(case)
    keep = [L - n for n, L in zip(new, ctx)]
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")) + "plan")
    had = [k + rng.randint(0, 40) for k in keep]  # tokens that the last step drafted and did not accept
    for b in rng.sample(range(case["seqs"]), case["finished"]):
        keep[b] = new[b] = 0
    return keep, new, had


def _words(case):
    return max(1, _pages(case["new_hi"]))


def work(case):
    new, ctx = _lengths(case)
    T, Hq, Hkv, D = sum(new), case["q_heads"], case["kv_heads"], case["head_dim"]
    io = 4 if case["dtype"] == "f32" else 2
    kv = {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    if case["op"] == "tables":
        keep, new, had = _plan(case)
        given = sum(_pages(h) - _pages(k) for h, k in zip(had, keep))
        taken = sum(_pages(k + n) - _pages(k) for k, n in zip(keep, new))
        return {"bytes": 20 * case["seqs"] + 8 * sum(new) + 8 * (given + taken), "flops": 0}
    if case["op"] == "masks":
        return {"bytes": T * (4 + 4 * _words(case) + 4) + 8 * case["seqs"], "flops": 0}
    if case["op"] == "keep":
        rows = _ancestors(case, new)
        moved = sum(sum(i != r for r, i in enumerate(rows[b][j])) for b, j in enumerate(_accepted(case, new)) if j >= 0)
        return {"bytes": 4 * moved * Hkv * D * kv * case["layers"] + 12 * case["seqs"], "flops": 0}
    if case["op"] == "norm":
        flops = T * (Hq + Hkv) * (4 * D + 3 * case["rot"])
        if not case["append"]:
            return {"bytes": 2 * T * Hq * D * io, "flops": T * Hq * (4 * D + 3 * case["rot"])}
        return {"bytes": T * D * (2 * Hq * io + 2 * Hkv * (io + kv)), "flops": flops}
    w = case["window"]
    pairs = keys = 0
    for n, L, rows in zip(new, ctx, _ancestors(case, new)):
        base = L - n
        counts = [len(r) for r in rows]
        if w > 0:
            pairs += sum(min(w, base + c) for c in counts)
            first = min((max(0, base - max(0, w - c)) for c in counts), default=base)  # earliest token that any row sees
        else:
            pairs += sum(base + c for c in counts)
            first = 0
        drafted = len(set().union(*[r[max(0, len(r) - w) if w else 0:] for r in rows])) if rows else 0
        keys += (base - first if n else 0) + drafted
    return {"bytes": 2 * T * Hq * D * io + 2 * keys * Hkv * D * kv + 4 * T * _words(case), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _int32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _packed_masks(rows, words, T):
    """[T][words] int32 whose bit i of a row says that it sees drafted token i of its sequence."""
    flat = [r for seq in rows for r in seq]
    out = []
    for r in flat:
        bits = sum(1 << i for i in r)
        line = [(bits >> (32 * w)) & 0xffffffff for w in range(words)]
        out.append([x - (1 << 32) if x >> 31 else x for x in line])
    out += [[0] * words] * (T - len(out))
    return torch.tensor(out, dtype=torch.int32)


def _starts(new):
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return starts


def _block_table(ctx, pool, perm):
    """Each context's pages, taken from a permutation of the pool, and the number of pages taken."""
    pages = [_pages(L) for L in ctx]
    table = torch.full((len(ctx), max(1, max(pages))), int(perm[-1]), dtype=torch.int32)  # (a page no sequence has)
    spots = [(b, i) for b, p in enumerate(pages) for i in range(p)]
    if spots:
        at = torch.tensor(spots)
        table[at[:, 0], at[:, 1]] = perm[:len(spots)]
    return table, len(spots)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    B, op = case["seqs"], case["op"]
    if op == "tables":
        keep, new, had = _plan(case)
        pool = sum(_pages(max(h, k + n)) for h, k, n in zip(had, keep, new)) + 5
        perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        table, used = _block_table(had, pool, perm.cpu())
        room = max(_pages(max(h, k + n)) for h, k, n in zip(had, keep, new))
        table = torch.nn.functional.pad(table, (0, max(0, room - table.shape[1])))
        T = sum(new) + case["pad"]
        free = torch.zeros(pool, dtype=torch.int32, device=dev)
        free[:pool - used] = perm[used:]
        return dict(case=case, rows=T, keep_lens=_int32(keep), new_lens=_int32(new), context_lens=_int32(had),
                    block_tables=table.to(dev), free_pages=free, counters=_int32([pool - used, 0]),
                    q_starts=torch.zeros(B + 1, dtype=torch.int32, device=dev),
                    positions=torch.full((T,), -7, dtype=torch.int32, device=dev),
                    slots=torch.full((T,), -7, dtype=torch.int32, device=dev))

    new, ctx = _lengths(case)
    live, rows = sum(new), sum(new) + case["pad"]
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    s = dict(case=case, live=live, rows=rows, n_max=max(new), ctx_max=max(ctx), q_starts=_int32(_starts(new)),
             context_lens=_int32(ctx), fp8=case["dtype"] == "e4m3")
    if op == "masks":
        # (which tokens a draft proposes differs from step to step: trees of the seed)
        rng = random.Random(int(seed))
        flat = [rng.randint(max(-1, j - case["reach"]), j - 1) for n in new for j in range(n)]
        s["parents"] = _int32(flat + [-1] * case["pad"])
        s["masks"] = torch.full((rows, _words(case)), -7, dtype=torch.int32, device=dev)
        s["positions"] = torch.full((rows,), -7, dtype=torch.int32, device=dev)
        return s

    io = _TORCH["bf16" if s["fp8"] else case["dtype"]]
    pool = sum(_pages(L) for L in ctx) + 3
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    s["block_tables"] = _block_table(ctx, pool, perm.cpu())[0].to(dev)
    if op in ("tree", "keep"):
        s["masks"] = _packed_masks(_ancestors(case, new), _words(case), rows).to(dev)
    shape = ((case["layers"],) if op == "keep" and case["layers"] > 1 else ()) + (pool, PAGE, Hkv, D)
    if op != "norm" or case["append"]:
        if op == "keep":
            # what the slots hold is copied: any numbers of the type, made quickly
            cache = [torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device=dev, dtype=torch.int16).float() * 2.0 ** -14
                     for _ in range(2)]
        else:
            cache = [torch.randn(shape, generator=g, device=dev, dtype=torch.float32) for _ in range(2)]
        if s["fp8"]:
            # calibrated scales: the largest magnitude of a head, with a little room, meets the largest code
            s["k_scale"], s["v_scale"] = (torch.full((Hkv,), 5.5 / E4M3_MAX, device=dev)
                                          * (0.8 + 0.4 * torch.rand((Hkv,), generator=g, device=dev)) for _ in range(2))
            cache = [(x / sc[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                     for x, sc in zip(cache, (s["k_scale"], s["v_scale"]))]
        else:
            cache = [x.to(io) for x in cache]
        s["k_cache"], s["v_cache"] = cache
    if op == "keep":
        s["accepted"] = _int32(_accepted(case, new))
        s["kept_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
        return s
    s["out"] = torch.zeros((rows, Hq, D), dtype=io, device=dev)
    if op == "tree":
        s["q"] = torch.randn((rows, Hq, D), generator=g, device=dev).to(io)
        s["scale"] = D ** -0.5
        return s
    # queries, keys and values as a fused projection leaves them, heads of different sizes
    qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device=dev)
    qkv = (qkv * (0.5 + 3 * torch.rand((1, Hq + 2 * Hkv, 1), generator=g, device=dev))).to(io)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["q_weight"], s["k_weight"] = (1 + 0.2 * torch.randn((h, D) if case["per_head"] else (D,), generator=g, device=dev)
                                    for h in (Hq, Hkv))
    j = torch.arange(case["rot"] // 2, dtype=torch.float64)
    s["inv_freq"] = (case["base"] ** (-2.0 * j / case["rot"])).to(dev)
    s["eps"] = 1e-6
    s["positions"] = _int32([L - n + j for n, L in zip(new, ctx) for j in range(n)] + [0] * case["pad"])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _row_map(s, rows):
    """Sequence, place within it and live or not of each of `rows` packed rows."""
    t = torch.arange(rows, device=s["q_starts"].device)
    starts = s["q_starts"].long()
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp_max(starts.numel() - 2)
    return seq, t - starts[seq], t < starts[-1]


def _tables_plain(s):
    table, free = s["block_tables"], s["free_pages"]
    B, room = table.shape
    cap, T = free.numel(), s["rows"]
    L, k, n = s["context_lens"].long(), s["keep_lens"].long(), s["new_lens"].long()
    have, kept, want = (L + PAGE - 1) // PAGE, (k + PAGE - 1) // PAGE, (k + n + PAGE - 1) // PAGE
    given, need = have - kept, want - kept
    top = s["counters"][0].long() + given.sum()
    grows = (n > 0) & (want <= room)
    need, rows = need * grows, n * grows
    over = grows & ((need.cumsum(0) > top) | (rows.cumsum(0) > T))
    granted = grows & (over.cumsum(0) == 0)                          # none behind the first that does not fit
    need, rows = need * granted, rows * granted
    p = torch.arange(room, device=table.device)
    # released pages to the stack, the first on top (one place behind it takes what is not released)
    rank = (given.cumsum(0) - given)[:, None] + p - kept[:, None]
    at = torch.where((p >= kept[:, None]) & (p < have[:, None]), top - 1 - rank, cap)
    stack = torch.cat([free, free[:1]])
    stack[at.flatten()] = table.flatten()
    free.copy_(stack[:cap])
    # pages from the top of the stack
    rank = (need.cumsum(0) - need)[:, None] + p - kept[:, None]
    fresh = (p >= kept[:, None]) & (p < (kept + need)[:, None])
    table.copy_(torch.where(fresh, free[(top - 1 - rank).clamp(0, cap - 1)], table))
    s["counters"][0] = top - need.sum()
    s["counters"][1] = ((n > 0) & ~granted).sum()
    s["context_lens"].copy_(k + rows)
    s["q_starts"][0] = 0
    s["q_starts"][1:] = rows.cumsum(0)
    seq, place, live = _row_map(s, T)
    pos = k[seq] + place
    slot = table[seq, (pos // PAGE).clamp_max(room - 1)].long() * PAGE + pos % PAGE
    s["positions"].copy_(torch.where(live, pos, s["positions"]))
    s["slots"].copy_(torch.where(live, slot, s["slots"]))
    return [s[x] for x in ("block_tables", "context_lens", "free_pages", "counters", "q_starts", "positions", "slots")]


def _masks_plain(s):
    masks, rows, words = s["masks"], s["rows"], s["masks"].shape[1]
    seq, place, live = _row_map(s, rows)
    starts = s["q_starts"].long()
    parent = s["parents"].long()
    # squaring: after step i a row holds its 2^i nearest ancestors and knows the next one
    bits = torch.zeros((rows + 1, 32 * words), dtype=torch.bool, device=masks.device)
    t = torch.arange(rows, device=masks.device)
    bits[t, place.clamp(0, 32 * words - 1)] = live
    up = torch.full((rows + 1,), rows, dtype=torch.int64, device=masks.device)  # row `rows` stands for the context
    up[:rows] = torch.where(live & (parent >= 0), starts[seq] + parent, rows)
    for _ in range(max(1, math.ceil(math.log2(s["n_max"] + 1)))):
        bits = bits | bits[up]
        up = up[up]
    weight = 2 ** torch.arange(32, dtype=torch.int64, device=masks.device)
    packed = (bits[:rows].view(rows, words, 32) * weight).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
    new = starts[1:] - starts[:-1]
    pos = s["context_lens"].long()[seq] - new[seq] + bits[:rows].sum(-1) - 1
    masks.copy_(torch.where(live[:, None], packed, masks))
    s["positions"].copy_(torch.where(live, pos, s["positions"]))
    return [masks, s["positions"]]


def _normed(x, weight, eps):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _rotated(x, positions, inv_freq, interleaved):
    """x [T][H][D] in 32 bits; the angles of far positions need 64."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _norm_plain(s):
    live, out = s["live"], s["out"]
    pos = s["positions"][:live]
    turn = (pos, s["inv_freq"], s["case"]["interleaved"])
    out[:live] = _rotated(_normed(s["q"][:live], s["q_weight"], s["eps"]), *turn).to(out.dtype)
    if not s["case"]["append"]:
        return out
    k = _rotated(_normed(s["k"][:live], s["k_weight"], s["eps"]), *turn)
    v = s["v"][:live].float()
    if s["fp8"]:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    pos = pos.long()
    page = s["block_tables"].long()[_row_map(s, live)[0], pos // PAGE]
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        if s["fp8"]:
            cache.view(torch.uint8)[page, pos % PAGE] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            cache[page, pos % PAGE] = x.to(cache.dtype)
    return [out, s["k_cache"], s["v_cache"]]


def _tree_plain(s):
    """Padded to one [seqs][new][context] matrix of scores for each head."""
    case, out, live = s["case"], s["out"], s["live"]
    B, N, L = case["seqs"], s["n_max"], s["ctx_max"]
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    dev = out.device
    seq, place, _ = _row_map(s, live)
    starts, ctx = s["q_starts"].long(), s["context_lens"].long()
    base = ctx - (starts[1:] - starts[:-1])
    q = torch.zeros((B, N, Hq, D), device=dev)
    q[seq, place] = s["q"][:live].float()
    # what each row sees of each token of its context
    words = s["masks"].shape[1]
    bits = (s["masks"][:live].long()[:, :, None] >> torch.arange(32, device=dev)) & 1
    drafted = torch.zeros((B, N, 32 * words + 1), dtype=torch.bool, device=dev)
    drafted[seq, place, :32 * words] = bits.flatten(1).bool()
    t = torch.arange(L, device=dev)
    ahead = t - base[:, None]                                        # [B][L]: which drafted token it is
    which = torch.where((ahead >= 0) & (ahead < 32 * words), ahead, 32 * words)
    seen = drafted.gather(2, which[:, None].expand(B, N, L)) | (ahead < 0)[:, None]
    seen &= (t < ctx[:, None])[:, None]
    if case["window"] > 0:  # the last of them
        later = seen.flip(-1).cumsum(-1, dtype=torch.int32).flip(-1)
        seen &= later <= case["window"]
    page = s["block_tables"].long()[:, t // PAGE]                    # [B][L]
    k, v = s["k_cache"], s["v_cache"]
    if s["fp8"]:
        k = k.view(torch.uint8)[page, t % PAGE].view(torch.float8_e4m3fn).float() * s["k_scale"][:, None]
        v = v.view(torch.uint8)[page, t % PAGE].view(torch.float8_e4m3fn).float() * s["v_scale"][:, None]
    else:
        k, v = k[page, t % PAGE].float(), v[page, t % PAGE].float()
    # [B][Hkv][group * N][D] x [B][Hkv][D][L]
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    score = score.view(B, Hkv, Hq // Hkv, N, L).masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    weight = torch.exp_(score.sub_(top))
    total = weight.sum(-1, keepdim=True)
    o = (weight.view(B, Hkv, -1, L) @ v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, N, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))       # a row that sees nothing
    out[:live] = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[seq, place].to(out.dtype)
    return out


def _keep_plain(s):
    masks, starts = s["masks"], s["q_starts"].long()
    dev = masks.device
    rows, bits_of = masks.shape[0], 32 * masks.shape[1]
    new = starts[1:] - starts[:-1]
    base = s["context_lens"].long() - new
    took = s["accepted"].long()
    line = masks[(starts[:-1] + took).clamp(0, rows - 1)].long()
    bits = ((line[:, :, None] >> torch.arange(32, device=dev)) & 1).flatten(1).bool() & (took >= 0)[:, None]
    rank = bits.cumsum(1) - 1                                        # [B][bits]
    s["kept_lens"].copy_(base + bits.sum(1))
    # places that take no part copy what the branch's first does (without a branch: the first slot to itself)
    i = torch.arange(bits_of, device=dev)
    first = bits.to(torch.int64).argmax(1, keepdim=True)
    from_token = torch.where(bits.any(1, keepdim=True), base[:, None] + first, 0)
    to_token = torch.where(bits.any(1), base, 0)[:, None]
    table = s["block_tables"].long()
    last = table.shape[1] * PAGE - 1

    def slot(token):
        token = token.clamp(0, last)
        return table.gather(1, token // PAGE) * PAGE + token % PAGE

    source = slot(torch.where(bits, base[:, None] + i, from_token))
    target = slot(torch.where(bits, base[:, None] + rank, to_token))
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.view(torch.uint8) if s["fp8"] else cache
        flat = flat.flatten(-4, -3)                                  # slots in a row
        if flat.dim() == 4:
            flat[:, target] = flat[:, source]
        else:
            flat[target] = flat[source]
    return [s["kept_lens"], s["k_cache"], s["v_cache"]]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"tables": _tables_plain, "masks": _masks_plain, "norm": _norm_plain, "tree": _tree_plain,
                "keep": _keep_plain}[op](s)
    import paged_attention_decode_kv_gb300 as vt
    if op == "tables":
        vt.step_tables(s["context_lens"], s["new_lens"], s["block_tables"], s["free_pages"], s["counters"], s["rows"],
                       keep_lens=s["keep_lens"], q_starts=s["q_starts"], positions=s["positions"], slots=s["slots"])
        return [s[x] for x in ("block_tables", "context_lens", "free_pages", "counters", "q_starts", "positions",
                               "slots")]
    if op == "masks":
        vt.tree_masks(s["parents"], s["q_starts"], s["context_lens"], masks=s["masks"], positions=s["positions"])
        return [s["masks"], s["positions"]]
    if op == "keep":
        vt.keep_path(s["accepted"], s["masks"], s["k_cache"], s["v_cache"], s["q_starts"], s["block_tables"],
                     s["context_lens"], kept_lens=s["kept_lens"])
        return [s["kept_lens"], s["k_cache"], s["v_cache"]]
    if op == "norm":
        turn = dict(inv_freq=s["inv_freq"], eps=s["eps"], interleaved=s["case"]["interleaved"])
        if not s["case"]["append"]:
            live = s["live"]
            vt.norm_rope(s["q"][:live], s["q_weight"], s["positions"][:live], out=s["out"][:live], **turn)
            return s["out"]
        turn.update(q=s["q"], q_weight=s["q_weight"], q_out=s["out"])
        where = (s["q_starts"], s["block_tables"], s["context_lens"])
        if s["fp8"]:
            vt.norm_append_fp8(s["k"], s["v"], s["k_weight"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                               *where, **turn)
        else:
            vt.norm_append(s["k"], s["v"], s["k_weight"], s["k_cache"], s["v_cache"], *where, **turn)
        return [s["out"], s["k_cache"], s["v_cache"]]
    where = (s["masks"], s["q_starts"], s["block_tables"], s["context_lens"], s["scale"], s["case"]["window"])
    if s["fp8"]:
        return vt.prefill_tree_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], *where,
                                   out=s["out"])
    return vt.prefill_tree(s["q"], s["k_cache"], s["v_cache"], *where, out=s["out"])


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _turned(x, positions, case):
    """Each pair as a complex number, times exp(i * position * frequency)."""
    rot = case["rot"]
    freq = torch.tensor([case["base"] ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64,
                        device=x.device)
    by = torch.polar(torch.ones_like(freq).expand(len(positions), -1).contiguous(),
                     torch.outer(positions.double(), freq))[:, None]
    y = x.clone()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    z = torch.complex(y[..., first], y[..., second]) * by
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(case, s, new, ctx):
    def normed(x, weight):
        x = x.double()
        return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()

    live, out = s["live"], s["out"].double()
    pos = s["positions"][:live].long()
    out[:live] = _turned(normed(s["q"][:live], s["q_weight"]), pos, case)
    if not case["append"]:
        return out
    k, v = _turned(normed(s["k"][:live], s["k_weight"]), pos, case), s["v"][:live].double()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    if s["fp8"]:
        k = (k / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    table = s["block_tables"].cpu().tolist()
    slot = torch.tensor([table[b][p // PAGE] * PAGE + p % PAGE for b, (n, L) in enumerate(zip(new, ctx))
                         for p in range(L - n, L)], device=out.device)
    kc.flatten(0, 1)[slot] = k
    vc.flatten(0, 1)[slot] = v
    return [out, kc, vc]


def _exact_tree(case, s, new, ctx):
    out = s["out"].double()
    table = s["block_tables"].cpu().tolist()
    starts = _starts(new)
    Hq, Hkv, w = case["q_heads"], case["kv_heads"], case["window"]
    for b, (n, L, rows) in enumerate(zip(new, ctx, _ancestors(case, new))):
        if n == 0:
            continue
        ids = torch.tensor(table[b][:_pages(L)], device=out.device)
        k, v = (s[x][ids].flatten(0, 1)[:L].double() for x in ("k_cache", "v_cache"))
        if s["fp8"]:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        seen = torch.zeros((n, L), dtype=torch.bool)
        for j, r in enumerate(rows):
            tokens = list(range(L - n)) + [L - n + i for i in r]
            seen[j, tokens[-w:] if w > 0 else tokens] = True
        seen = seen.to(out.device)
        q = s["q"][starts[b]:starts[b + 1]].double()
        for h in range(Hkv):
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("ngd,td->gnt", q[:, mine], k[:, h]) * s["scale"]
            p = torch.softmax(x.masked_fill(~seen, float("-inf")), -1).nan_to_num(0.0)  # no token seen: 0
            out[starts[b]:starts[b + 1], mine] = torch.einsum("gnt,td->ngd", p, v[:, h])
    return out


def exact(case, seed):
    if case["op"] in ("tables", "masks"):
        return None  # whole numbers
    s = prepare(case, seed)
    new, ctx = _lengths(case)
    if case["op"] == "norm":
        return _exact_norm(case, s, new, ctx)
    if case["op"] == "tree":
        return _exact_tree(case, s, new, ctx)
    table = s["block_tables"].cpu().tolist()
    kept, pairs = [], []
    for b, (n, L, rows, j) in enumerate(zip(new, ctx, _ancestors(case, new), _accepted(case, new))):
        path = rows[j] if j >= 0 else []
        kept.append(L - n + len(path))
        for r, i in enumerate(path):
            pairs.append([table[b][t // PAGE] * PAGE + t % PAGE for t in (L - n + r, L - n + i)])
    caches = []
    for cache in (s["k_cache"], s["v_cache"]):
        c = cache.float()  # (the types' values are exact in it)
        if pairs:
            to, source = torch.tensor(pairs, device=c.device).T
            flat = c.flatten(-4, -3)
            if flat.dim() == 4:
                flat[:, to] = flat[:, source]
            else:
                flat[to] = flat[source]
        caches.append(c)
    return [None, *caches]

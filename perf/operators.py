"""Cases, plain forms and exact values of the paged-cache serving operators.

Three operators that a serving step runs around the paged decode:

* ``rope``     rotary positions on packed rows of heads (``vt.rope``);
* ``append``   new keys and values written into the paged cache, keys and
               queries rotated on the way (``vt.append``, ``vt.append_fp8``);
* ``prefill``  attention of a ragged batch of chunks of new tokens over the
               paged cache (``vt.prefill``, ``vt.prefill_fp8``).

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
             ctx_hi=0, pad=0, rot=128, interleaved=False, base=1e6, stretch=1.0, window=0)
    c.update(kw)
    return c


def listed():
    return [
        # A decode step's queries, rotated apart from the append: 8 sequences, one token each.
        _case("rope", name="rope_b8_h16_d128", q_heads=16, seqs=8, ctx_lo=1, ctx_hi=1152, base=1e6),
        # A long prompt's queries at far positions, frequencies stretched 4 times, half of each head rotated in
        # adjacent pairs.
        _case("rope", name="rope_8191_h32_d128_part64_far", new_lo=8191, new_hi=8191, ctx_lo=120000, ctx_hi=131072,
              rot=64, interleaved=True, stretch=4.0),
        # The append of one decode step of a 128-sequence batch.
        _case("append", name="append_b128_gqa4_d128", seqs=128, ctx_lo=64, ctx_hi=2048),
        # Prompts of odd lengths in one padded batch of about 16 thousand tokens.
        _case("append", name="append_prompts_16k_gqa4_d128", seqs=12, new_lo=257, new_hi=2600, ctx_lo=0, ctx_hi=700,
              pad=13),
        # Chunks of prompts into a cache of 8-bit codes with a scale for each kv head.
        _case("append", name="append_fp8_chunks_gqa8_d128", dtype="e4m3", q_heads=64, seqs=24, new_lo=1, new_hi=400,
              ctx_lo=0, ctx_hi=3000),
        # Draft tokens to verify: a few new tokens for each sequence over long contexts (memory-bound).
        _case("prefill", name="prefill_verify_b64_gqa4_d128", seqs=64, new_lo=1, new_hi=8, ctx_lo=512, ctx_hi=8000),
        # One whole prompt, causal (tensor-core bound; the largest case).
        _case("prefill", name="prefill_prompt_8192_gqa4_d128", new_lo=8192, new_hi=8192),
        # Chunked prompts of a large-GQA server batch over contexts that are partly cached.
        _case("prefill", name="prefill_chunks_gqa8_d128", q_heads=64, seqs=4, new_lo=300, new_hi=1025, ctx_lo=0,
              ctx_hi=6000, pad=7),
        # head_dim 256 with a sliding window.
        _case("prefill", name="prefill_d256_gqa4_w1024", q_heads=16, kv_heads=4, head_dim=256, seqs=3, new_lo=700,
              new_hi=2050, ctx_lo=0, ctx_hi=2000, window=1024),
        # The chunks over a cache of 8-bit codes.
        _case("prefill", name="prefill_fp8_chunks_gqa4_d128", dtype="e4m3", seqs=4, new_lo=500, new_hi=2000,
              ctx_lo=1000, ctx_hi=6000),
        # head_dim 64, many short prompts of odd lengths.
        _case("prefill", name="prefill_short_prompts_gqa4_d64", q_heads=16, kv_heads=4, head_dim=64, seqs=48,
              new_lo=1, new_hi=401, ctx_lo=0, ctx_hi=300),
        # fp32 storage, checked against rather than served from: a small prompt batch.
        _case("prefill", name="prefill_f32_gqa2_d128", dtype="f32", q_heads=16, seqs=3, new_lo=33, new_hi=700,
              ctx_lo=0, ctx_hi=500),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5)))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "prefill", "prefill", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f32"] if op == "rope" else ["bf16", "bf16", "e4m3", "f32"])
    dims = [64, 128, 256] + ([512] if dtype == "bf16" else [])
    head_dim = rng.choice(dims)
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = _case(op, dtype=dtype, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, seqs=_log(rng, 1, 96),
              pad=rng.choice([0, 0, rng.randint(1, 40)]), interleaved=rng.random() < 0.4,
              rot=rng.choice([head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]),
              base=rng.choice([1e4, 5e5, 1e6]), stretch=rng.choice([1.0, 1.0, 2.0, 8.0]))
    most = _log(rng, 1, 6000 if op != "prefill" else 4000)  # new tokens of the longest sequence
    c["new_hi"] = max(1, most if c["seqs"] == 1 else most // rng.choice([1, 2, 4]))
    c["new_lo"] = rng.choice([c["new_hi"], 0 if c["seqs"] > 1 else 1, max(1, c["new_hi"] // 2)])
    c["ctx_hi"] = _log(rng, 1, 12000)
    c["ctx_lo"] = rng.choice([0, c["ctx_hi"] // 2, c["ctx_hi"]])
    if op == "prefill" and rng.random() < 0.3:
        c["window"] = _log(rng, 1, 4096)
    # No dearer than the largest listed case: the padded score matrix of the plain form, the rows, the pages.
    room = {"bf16": 1 << 29, "e4m3": 1 << 29, "f32": 1 << 27}[dtype] if op == "prefill" else 1 << 62
    while c["seqs"] > 1 and (c["seqs"] * q_heads * c["new_hi"] * (c["new_hi"] + c["ctx_hi"]) > room
                             or c["seqs"] * c["new_hi"] * (q_heads + 2 * kv_heads) * head_dim > 1 << 25
                             or c["seqs"] * (c["new_hi"] + c["ctx_hi"]) * kv_heads * head_dim > 1 << 26):
        c["seqs"] //= 2
    while (q_heads * c["new_hi"] * (c["new_hi"] + c["ctx_hi"]) > room
           or c["new_hi"] * (q_heads + 2 * kv_heads) * head_dim > 1 << 25):
        c["new_hi"] = c["new_hi"] * 2 // 3
        c["ctx_hi"] = c["ctx_hi"] * 2 // 3
    c["new_lo"] = min(c["new_lo"], c["new_hi"])
    c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
    return c


def _lengths(case):
    """New tokens and contexts of each sequence: the case's own, whatever the seed of its contents."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    if sum(new) == 0:
        new[0] = case["new_hi"]
    ctx = [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in new]
    return new, ctx


def work(case):
    new, ctx = _lengths(case)
    T, Hq, Hkv, D = sum(new), case["q_heads"], case["kv_heads"], case["head_dim"]
    io = 4 if case["dtype"] == "f32" else 2
    kv = {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    if case["op"] == "rope":
        return {"bytes": 2 * T * Hq * D * io, "flops": 3 * T * Hq * case["rot"]}
    if case["op"] == "append":
        return {"bytes": T * D * (2 * Hq * io + 2 * Hkv * (io + kv)), "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    w = case["window"]
    pairs = keys = 0
    for n, L in zip(new, ctx):
        first = L - n + 1  # keys that the first new token may see
        if w <= 0:
            pairs += n * first + n * (n - 1) // 2
            keys += L if n else 0
        else:
            full = min(n, max(0, w - first))  # rows whose window is not yet full
            pairs += full * first + full * (full - 1) // 2 + (n - full) * w
            keys += min(L, n - 1 + w) if n else 0
    return {"bytes": 2 * T * Hq * D * io + 2 * keys * Hkv * D * kv, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _frequencies(case):
    """Radians for each token of each rotated pair, stretched by a factor for long contexts."""
    j = torch.arange(case["rot"] // 2, dtype=torch.float64)
    return case["base"] ** (-2.0 * j / case["rot"]) / case["stretch"]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))
    new, ctx = _lengths(case)
    live, rows = sum(new), sum(new) + case["pad"]
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    fp8 = case["dtype"] == "e4m3"
    io = _TORCH["bf16" if fp8 else case["dtype"]]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(case=case, live=live, n_max=max(new), ctx_max=max(ctx), fp8=fp8,
             q_starts=torch.tensor(starts, dtype=torch.int32, device=dev),
             context_lens=torch.tensor(ctx, dtype=torch.int32, device=dev),
             inv_freq=_frequencies(case).to(dev), amplitude=1.0 + 0.1 * math.log(case["stretch"]),
             interleaved=case["interleaved"], scale=D ** -0.5, window=case["window"])

    if case["op"] == "rope":
        pos = [L - n + j for n, L in zip(new, ctx) for j in range(n)] + [0] * case["pad"]
        s["positions"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        # queries lie in rows of a fused projection (queries, keys, values)
        s["x"] = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device=dev).to(io)[:, :Hq]
        s["out"] = torch.zeros((rows, Hq, D), dtype=io, device=dev)
        return s

    pages = [(L + PAGE - 1) // PAGE for L in ctx]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((case["seqs"], max(1, max(pages))), dtype=torch.int32)
    spots = [(b, i) for b, p in enumerate(pages) for i in range(p)]
    if spots:
        at = torch.tensor(spots)
        table[at[:, 0], at[:, 1]] = perm[:len(spots)].cpu()
    s["block_tables"] = table.to(dev)
    shape = (pool, PAGE, Hkv, D)
    cache = [torch.randn(shape, generator=g, device=dev, dtype=torch.float32) for _ in range(2)]
    if fp8:
        # calibrated scales: the largest magnitude of a head, with a little room, meets the largest code
        s["k_scale"], s["v_scale"] = (torch.full((Hkv,), 5.5 / E4M3_MAX, device=dev)
                                      * (0.8 + 0.4 * torch.rand((Hkv,), generator=g, device=dev)) for _ in range(2))
        cache = [(x / sc[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                 for x, sc in zip(cache, (s["k_scale"], s["v_scale"]))]
    else:
        cache = [x.to(io) for x in cache]
    s["k_cache"], s["v_cache"] = cache
    if case["op"] == "append":
        qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g, device=dev).to(io)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        s["out"] = torch.zeros((rows, Hq, D), dtype=io, device=dev)
    else:
        s["q"] = torch.randn((rows, Hq, D), generator=g, device=dev).to(io)
        s["out"] = torch.zeros((rows, Hq, D), dtype=io, device=dev)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _rotated(x, positions, inv_freq, interleaved, amplitude):
    """x [T][H][D] in 32 bits; the angles of far positions need 64."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    cos = (angle.cos() * amplitude).float()[:, None]
    sin = (angle.sin() * amplitude).float()[:, None]
    x = x.float()
    turn, keep = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turn[..., :half], turn[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, keep], dim=-1)


def _row_map(s):
    """Sequence and place within it of each live row, and its position in the context."""
    rows = torch.arange(s["live"], device=s["q_starts"].device)
    starts = s["q_starts"].long()
    seq = torch.searchsorted(starts[1:].contiguous(), rows, right=True)
    place = rows - starts[seq]
    new = starts[1:] - starts[:-1]
    return seq, place, s["context_lens"].long()[seq] - new[seq] + place


def _rope_plain(s):
    live = s["live"]
    out = s["out"]
    out[:live] = _rotated(s["x"][:live], s["positions"][:live], s["inv_freq"], s["interleaved"],
                          s["amplitude"]).to(out.dtype)
    return out


def _append_plain(s):
    live, out = s["live"], s["out"]
    seq, _, pos = _row_map(s)
    turn = (pos, s["inv_freq"], s["interleaved"], s["amplitude"])
    out[:live] = _rotated(s["q"][:live], *turn).to(out.dtype)
    k, v = _rotated(s["k"][:live], *turn), s["v"][:live].float()
    if s["fp8"]:
        k = (k / s["k_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["v_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    page = s["block_tables"].long()[seq, pos // PAGE]
    s["k_cache"].view(torch.uint8 if s["fp8"] else out.dtype)[page, pos % PAGE] = _stored(k, s)
    s["v_cache"].view(torch.uint8 if s["fp8"] else out.dtype)[page, pos % PAGE] = _stored(v, s)
    return [out, s["k_cache"], s["v_cache"]]


def _stored(x, s):
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if s["fp8"] else x.to(s["out"].dtype)


def _prefill_plain(s):
    """Padded to one [seqs][new][context] matrix of scores for each head."""
    case, out, live = s["case"], s["out"], s["live"]
    B, N, L = case["seqs"], s["n_max"], s["ctx_max"]
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    seq, place, pos = _row_map(s)
    q = torch.zeros((B, N, Hq, D), device=out.device)
    q[seq, place] = s["q"][:live].float()
    at = torch.full((B, N), -1, device=out.device, dtype=torch.int64)
    at[seq, place] = pos
    t = torch.arange(L, device=out.device)
    page = s["block_tables"].long()[:, t // PAGE]                    # [B][L]
    if s["fp8"]:
        k = s["k_cache"].view(torch.uint8)[page, t % PAGE].view(torch.float8_e4m3fn).float() * s["k_scale"][:, None]
        v = s["v_cache"].view(torch.uint8)[page, t % PAGE].view(torch.float8_e4m3fn).float() * s["v_scale"][:, None]
    else:
        k, v = s["k_cache"][page, t % PAGE].float(), s["v_cache"][page, t % PAGE].float()
    # [B][Hkv][group * N][D] x [B][Hkv][D][L]
    q = q.view(B, N, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    hidden = t > at[:, :, None]
    if s["window"] > 0:
        hidden |= t <= at[:, :, None] - s["window"]
    score = score.view(B, Hkv, Hq // Hkv, N, L).masked_fill_(hidden[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)              # padding rows see no key
    weight = torch.exp_(score.sub_(top))
    total = weight.sum(-1, keepdim=True)
    o = weight.view(B, Hkv, -1, L) @ v.permute(0, 2, 1, 3)
    o = o.view(B, Hkv, Hq // Hkv, N, D) / total
    out[:live] = o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[seq, place].to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import paged_attention_decode_kv_gb300 as vt
        if op == "rope":
            live = s["live"]
            vt.rope(s["x"][:live], s["positions"][:live], s["inv_freq"], interleaved=s["interleaved"],
                    amplitude=s["amplitude"], out=s["out"][:live])
            return s["out"]
        if op == "append":
            turn = dict(q=s["q"], q_out=s["out"], inv_freq=s["inv_freq"], interleaved=s["interleaved"],
                        amplitude=s["amplitude"])
            if s["fp8"]:
                vt.append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_starts"],
                              s["block_tables"], s["context_lens"], **turn)
            else:
                vt.append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["q_starts"], s["block_tables"],
                          s["context_lens"], **turn)
            return [s["out"], s["k_cache"], s["v_cache"]]
        if s["fp8"]:
            return vt.prefill_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_starts"],
                                  s["block_tables"], s["context_lens"], s["scale"], s["window"], out=s["out"])
        return vt.prefill(s["q"], s["k_cache"], s["v_cache"], s["q_starts"], s["block_tables"], s["context_lens"],
                          s["scale"], s["window"], out=s["out"])
    if op == "rope":
        return _rope_plain(s)
    if op == "append":
        return _append_plain(s)
    return _prefill_plain(s)


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _turned(x, positions, case, amplitude):
    """Each pair as a complex number, times amplitude * exp(i * position * frequency)."""
    rot = case["rot"]
    freq = torch.tensor([case["base"] ** (-2.0 * j / rot) / case["stretch"] for j in range(rot // 2)],
                        dtype=torch.float64, device=x.device)
    by = torch.polar(torch.full_like(freq, amplitude).expand(len(positions), -1).contiguous(),
                     torch.outer(positions.double(), freq))[:, None]
    y = x.double().clone()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    z = torch.complex(y[..., first], y[..., second]) * by
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    new, ctx = _lengths(case)
    out = s["out"].double()
    starts = [sum(new[:b]) for b in range(len(new) + 1)]
    if case["op"] == "rope":
        out[:s["live"]] = _turned(s["x"][:s["live"]], s["positions"][:s["live"]], case, s["amplitude"])
        return out
    dev = out.device
    table = s["block_tables"].cpu().tolist()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    if case["op"] == "append":
        for b, (n, L) in enumerate(zip(new, ctx)):
            if n == 0:
                continue
            r = slice(starts[b], starts[b + 1])
            pos = torch.arange(L - n, L, device=dev)
            out[r] = _turned(s["q"][r], pos, case, s["amplitude"])
            k, v = _turned(s["k"][r], pos, case, s["amplitude"]), s["v"][r].double()
            if s["fp8"]:
                k = (k / s["k_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
                v = (v / s["v_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            slot = torch.tensor([table[b][p // PAGE] * PAGE + p % PAGE for p in range(L - n, L)], device=dev)
            kc.flatten(0, 1)[slot] = k
            vc.flatten(0, 1)[slot] = v
        return [out, kc, vc]
    if s["fp8"]:
        kc *= s["k_scale"].double()[:, None]
        vc *= s["v_scale"].double()[:, None]
    group = case["q_heads"] // case["kv_heads"]
    for b, (n, L) in enumerate(zip(new, ctx)):
        if n == 0:
            continue
        ids = torch.tensor(table[b][:(L + PAGE - 1) // PAGE], device=dev)
        k, v = kc[ids].flatten(0, 1)[:L], vc[ids].flatten(0, 1)[:L]
        ago = torch.arange(L - n, L, device=dev)[:, None] - torch.arange(L, device=dev)[None]
        seen = (ago >= 0) if case["window"] <= 0 else (ago >= 0) & (ago < case["window"])
        for i in range(case["q_heads"]):
            x = s["q"][starts[b]:starts[b + 1], i].double() @ k[:, i // group].T * s["scale"]
            out[starts[b]:starts[b + 1], i] = torch.softmax(x.where(seen, float("-inf")), -1) @ v[:, i // group]
    return out

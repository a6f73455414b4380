"""Ragged batches over a paged cache, and the plain 64-bit forms of the
rotary, append and prefill operators the GPU tests compare against (test
infrastructure; shares no code with the library)."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

PAGE = 32
E4M3_MAX = 448.0
STORE = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.bfloat16}


@dataclass
class Batch:
    new: list
    ctx: list
    dtype: str
    q: torch.Tensor            # [T][Hq][D]
    k_cache: torch.Tensor      # every token of every context, paged; NaN in every slot no sequence owns
    v_cache: torch.Tensor
    block_tables: torch.Tensor
    context_lens: torch.Tensor
    q_starts: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    @property
    def starts(self):
        return self.q_starts.tolist()

    def dense(self, which):
        """[Hkv][L][D] float64 rows of each sequence's context."""
        cache = self.k_cache if which == "k" else self.v_cache
        scale = self.k_scale if which == "k" else self.v_scale
        out = []
        for b, L in enumerate(self.ctx):
            ids = self.block_tables[b, : (L + PAGE - 1) // PAGE].long()
            rows = cache[ids].flatten(0, 1)[:L]
            if self.dtype == "e4m3":
                rows = rows.view(torch.float8_e4m3fn).double() * scale.double()[:, None]
            out.append(rows.double().permute(1, 0, 2))
        return out


def make_batch(new, ctx, q_heads, kv_heads, head_dim, dtype="bf16", seed=0, pad=0, device="cuda", sigma=1.0):
    """Contexts of `ctx` tokens whose last `new` are the chunk; every slot and
    page that no sequence owns holds NaN, padding rows of q too."""
    g = torch.Generator().manual_seed(seed)
    pages = [(L + PAGE - 1) // PAGE for L in ctx]
    pool = sum(pages) + 2
    perm = torch.randperm(pool, generator=g)
    maxb = max(1, max(pages, default=1))
    bt = torch.full((len(ctx), maxb), int(perm[-1]), dtype=torch.int64)
    caches, scales = [], []
    at = 0
    for b, p in enumerate(pages):
        bt[b, :p] = perm[at:at + p]
        at += p
    store = STORE[dtype]
    for _ in range(2):
        x = torch.randn((pool, PAGE, kv_heads, head_dim), generator=g) * sigma
        if dtype == "e4m3":
            scale = x.abs().amax(dim=(0, 1, 3)) / E4M3_MAX
            scales.append(scale)
            c = (x / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            nan = 0x7F
        else:
            c, nan = x.to(store), float("nan")
        owned = torch.zeros((pool, PAGE), dtype=torch.bool)
        for b, L in enumerate(ctx):
            for i in range(pages[b]):
                owned[bt[b, i], : min(PAGE, L - i * PAGE)] = True
        c[~owned] = nan
        caches.append(c.to(device))
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    q = (torch.randn((starts[-1] + pad, q_heads, head_dim), generator=g) * sigma).to(store)
    q[starts[-1]:] = float("nan")
    i32 = dict(dtype=torch.int32, device=device)
    return Batch(list(new), list(ctx), dtype, q.to(device), caches[0], caches[1], bt.to(torch.int32).to(device),
                 torch.tensor(ctx, **i32), torch.tensor(starts, **i32),
                 *(s.to(device) for s in scales))


def attention(batch: Batch, scale, window=0, flat=False):
    """(out, weight) float64 [T][Hq][D]: softmax attention row by row of the
    definition, and sum_t p_t |v_t|, what a relative error in the weights can
    move; with `flat` also max_t p_t sum_t |v_t|, what an absolute one can."""
    T, Hq, D = batch.q.shape
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=batch.q.device)
    reach = out.clone()
    even = out.clone()
    ks, vs, st = batch.dense("k"), batch.dense("v"), batch.starts
    for b, (n, L) in enumerate(zip(batch.new, batch.ctx)):
        if n == 0:
            continue
        group = Hq // ks[b].shape[0]
        pos = torch.arange(L - n, L, device=out.device)[:, None]
        t = torch.arange(L, device=out.device)[None]
        seen = t <= pos
        if window > 0:
            seen &= t > pos - window
        for h in range(Hq):
            k, v = ks[b][h // group], vs[b][h // group]
            x = (batch.q[st[b]:st[b + 1], h].double() @ k.T) * scale
            x = x.masked_fill(~seen, float("-inf"))
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = p / p.sum(-1, keepdim=True)
            out[st[b]:st[b + 1], h] = p @ v
            reach[st[b]:st[b + 1], h] = p @ v.abs()
            if flat:
                even[st[b]:st[b + 1], h] = p.amax(-1, keepdim=True) * (seen.double() @ v.abs())
    return (out, reach, even) if flat else (out, reach)


def rotate(x, positions, inv_freq, interleaved, amplitude):
    """(rotated, |a| + |b| of each element's pair times amplitude), float64."""
    half = inv_freq.numel()
    x = x.double()
    y, mag = x.clone(), torch.zeros_like(x)
    # the angle in turns, its whole turns taken off in exact integers: f / 2 pi as a fraction of 2^52
    for j in range(half):
        f = float(inv_freq[j]) / (2 * math.pi)
        turns = torch.tensor([math.fmod(int(p) * f, 1.0) if abs(int(p)) < 2 ** 20 else _turns(int(p), f)
                              for p in positions.tolist()], dtype=torch.float64, device=x.device)
        c, s = torch.cos(2 * math.pi * turns)[:, None], torch.sin(2 * math.pi * turns)[:, None]
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b = x[..., i0], x[..., i1]
        y[..., i0] = amplitude * (a * c - b * s)
        y[..., i1] = amplitude * (b * c + a * s)
        mag[..., i0] = mag[..., i1] = abs(amplitude) * (a.abs() + b.abs())
    return y, mag


def _turns(p, f):
    from fractions import Fraction
    t = Fraction(f) * p
    return float(t - math.floor(t))

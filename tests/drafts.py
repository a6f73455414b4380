"""Plain forms of the speculative step's operators that the tests compare
against (test infrastructure; shares no code with the library)."""
from __future__ import annotations

import random

import torch

PAGE = 32


def pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def random_parents(n, reach, rng):
    return [rng.randint(max(-1, j - reach), j - 1) for j in range(n)]


def branch(parents, j):
    """Token j and those it follows, ascending."""
    path = []
    while j >= 0:
        path.append(j)
        j = parents[j] if -1 <= parents[j] < j else -1
    return path[::-1]


def tree_rows(new, reach, seed=0):
    rng = random.Random(seed)
    out = []
    for n in new:
        p = random_parents(n, reach, rng)
        out.append([branch(p, j) for j in range(n)])
    return out


def any_rows(new, seed=0):
    """Masks that are no trees: rows that see nothing, rows that see tokens after their own."""
    rng = random.Random(seed)
    return [[sorted(rng.sample(range(n), rng.randint(0, n))) if rng.random() < 0.75 else [] for _ in range(n)]
            for n in new]


def pack(rows, words, T, fill=0, device="cuda"):
    """[T][words] int32 masks of the sequences' rows; rows behind them hold `fill`."""
    out = []
    for r in (r for seq in rows for r in seq):
        bits = sum(1 << i for i in r)
        line = [(bits >> (32 * w)) & 0xffffffff for w in range(words)]
        out.append([x - (1 << 32) if x >> 31 else x for x in line])
    out += [[fill] * words] * (T - len(out))
    return torch.tensor(out, dtype=torch.int32, device=device).view(T, words)


def tree_attention(batch, rows, scale, window=0):
    """(out, weight, even) float64 [T][Hq][D]: softmax attention of each row over what it sees, sum_t p_t |v_t|, and
    max_t p_t sum_t |v_t| (see ragged.attention); a row that sees nothing is 0."""
    T, Hq, D = batch.q.shape
    dev = batch.q.device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    reach, even = out.clone(), out.clone()
    ks, vs, st = batch.dense("k"), batch.dense("v"), batch.starts
    for b, (n, L) in enumerate(zip(batch.new, batch.ctx)):
        if n == 0:
            continue
        seen = torch.zeros((n, L), dtype=torch.bool)
        for j, r in enumerate(rows[b]):
            tokens = list(range(L - n)) + [L - n + i for i in r if i < n]
            seen[j, tokens[-window:] if window > 0 else tokens] = True
        seen = seen.to(dev)
        group = Hq // ks[b].shape[0]
        for h in range(Hq):
            k, v = ks[b][h // group], vs[b][h // group]
            q = batch.q[st[b]:st[b + 1], h].double()
            # (what a row does not see takes no part, whatever it holds)
            x = torch.where(seen, q @ k.T * scale, float("-inf"))
            p = torch.exp(x - x.amax(-1, keepdim=True))
            p = torch.where(seen, p, 0.0)
            p = torch.where(seen.any(-1, keepdim=True), p / p.sum(-1, keepdim=True), 0.0)
            if torch.isfinite(v).all():
                out[st[b]:st[b + 1], h] = p @ v
                reach[st[b]:st[b + 1], h] = p @ v.abs()
                even[st[b]:st[b + 1], h] = p.amax(-1, keepdim=True) * (seen.double() @ v.abs())
            else:
                for j in range(n):
                    at = seen[j].nonzero().flatten()
                    out[st[b] + j, h] = p[j, at] @ v[at]
                    reach[st[b] + j, h] = p[j, at] @ v[at].abs()
                    even[st[b] + j, h] = (p[j, at].amax() if len(at) else 0.0) * v[at].abs().sum(0)
    return out, reach, even


def step(state, keep, new, num_tokens):
    """One step of the page tables, sequence by sequence, on host lists: state has tables [B][room], lens, free (the
    stack, its top last) and room; returns (q_starts, positions, slots, refused)."""
    lens, tables, free, room = state["lens"], state["tables"], state["free"], state["room"]
    refused, given, valid = 0, [], []
    for b, (k, n) in enumerate(zip(keep, new)):
        L = lens[b]
        ok = 0 <= L <= room * PAGE and 0 <= k <= L and n >= 0
        valid.append(ok)
        if not ok:
            refused += 1
            continue
        given += tables[b][pages(k):pages(L)]
        lens[b] = k
    free += given[::-1]
    starts, positions, slots = [0], [], []
    full = False
    for b, (k, n) in enumerate(zip(keep, new)):
        rows = 0
        if valid[b] and n > 0:
            need = pages(k + n) - pages(k)
            if k + n > room * PAGE:
                refused += 1
            elif full or need > len(free) or starts[-1] + n > num_tokens:
                full = True
                refused += 1
            else:
                for p in range(pages(k), pages(k + n)):
                    tables[b][p] = free.pop()
                lens[b] = k + n
                rows = n
        for t in range(k, k + rows):
            positions.append(t)
            slots.append(tables[b][t // PAGE] * PAGE + t % PAGE)
        starts.append(starts[-1] + rows)
    return starts, positions, slots, refused

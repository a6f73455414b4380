"""Rotary positions and the paged append against their 64-bit forms (GPU).

Tolerances, from the operators' arithmetic.  The reduced angle is off by at
most 2^-26 turns (its 32-bit fraction becomes a float), 2 pi 2^-26 < 1e-7
radians; sincospi() by about an ulp, 2^-23; the two products, their sum and
the amplitude's product by 2^-24 each: together below 2^-20 of
amplitude (|a| + |b|).  The rounding to bf16 adds 2^-8 of the value; a code of
E4M3 is within 2^-4 of its value, or 2^-10 below the normal range.
"""
from __future__ import annotations

import pytest
import torch

import paged_attention_decode_kv_gb300 as vt
from ragged import E4M3_MAX, PAGE, STORE, make_batch, rotate

pytestmark = pytest.mark.gpu

ARITH = 2.0 ** -20
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from paged_attention_decode_kv_gb300 import build_lib
    build_lib.build()
    vt.library()
    return torch.device("cuda:0")


def rows(T, H, D, dtype, dev, seed=0, extra=0):
    """[T][H][D], a view into rows of H + extra heads."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, H + extra, D), generator=g).to(dtype).to(dev)[:, :H]


def check_rotated(got, x, positions, inv, interleaved, amplitude):
    ref, mag = rotate(x, positions, inv, interleaved, amplitude)
    tol = mag * ARITH + (ref.abs() + mag * ARITH) * HALF_STEP[got.dtype]
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (7, 3, 128, 128), (33, 5, 128, 64), (5, 2, 256, 34),
                                       (130, 1, 80, 48), (3, 4, 512, 512), (2, 2, 1024, 1024), (9, 1, 8, 2),
                                       (2500, 2, 64, 32),
                                       (2999, 20, 128, 128), (4001, 31, 64, 64), (3001, 9, 256, 128)])
def test_rope(dev, T, H, D, rot, dtype, interleaved):
    inv, _ = vt.rope_frequencies(rot, 10000.0)
    g = torch.Generator().manual_seed(T + D)
    positions = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32).to(dev)
    x = rows(T, H, D, dtype, dev, extra=2)
    got = vt.rope(x, positions, inv, interleaved=interleaved, amplitude=1.25)
    check_rotated(got, x, positions, inv, interleaved, 1.25)
    assert torch.equal(got[..., rot:], x[..., rot:])


def test_rope_extreme_positions(dev):
    inv, _ = vt.rope_frequencies(128, 1e6)
    positions = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, -(1 << 24) + 1], dtype=torch.int32, device=dev)
    x = rows(7, 2, 128, torch.float32, dev)
    # the turn per token is off by 2^-53 of the frequency in fp64; 2^31 tokens make 2^-22 radians of that
    ref, mag = rotate(x, positions, inv, False, 1.0)
    got = vt.rope(x, positions, inv).double()
    assert ((got - ref).abs() <= mag * (ARITH + 2.0 ** -21) + ref.abs() * 2.0 ** -24).all()
    assert torch.equal(got[0], x[0].double())  # position 0 turns nothing


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 20])
def test_rope_in_place_and_back(dev, rot, interleaved):
    """x itself as out; a negative position is the transposed rotation, i.e. the gradient, checked against
    differences of the forward call."""
    inv, _ = vt.rope_frequencies(rot, 10000.0)
    T = 700
    positions = torch.arange(T, dtype=torch.int32, device=dev) * 37
    x = rows(T, 3, 128, torch.float32, dev, extra=1)
    y = vt.rope(x, positions, inv, interleaved=interleaved, amplitude=1.5)
    z = x.clone()
    assert vt.rope(z, positions, inv, interleaved=interleaved, amplitude=1.5, out=z) is z
    assert torch.equal(y, z)
    grad = rows(T, 3, 128, torch.float32, dev, seed=9)
    got = vt.rope(grad, -positions, inv, interleaved=interleaved, amplitude=1.5)
    # <grad, R x> = <R^T grad, x> for every row; each side sums 128 products of size <= |g||x| in float64
    lhs = (grad.double() * y.double()).sum(-1)
    rhs = (got.double() * x.double()).sum(-1)
    bound = 2 * ARITH * 1.5 * 2 * (grad.double().norm(dim=-1) * x.double().norm(dim=-1)) * 2
    assert ((lhs - rhs).abs() <= bound).all()
    # a step along one input moves the outputs by its column of R (linear: differences are exact up to rounding)
    e = torch.zeros_like(x)
    e[..., 5] = 1.0
    column = vt.rope(e.contiguous(), positions, inv, interleaved=interleaved, amplitude=1.5).double()
    dot = (column * grad.double()).sum(-1)
    assert ((dot - got[..., 5].double()).abs() <= 8 * ARITH * grad.double().abs().amax(-1)).all()


def test_rope_padding_of_out_is_kept(dev):
    inv, _ = vt.rope_frequencies(64)
    x = rows(5, 2, 64, torch.bfloat16, dev)
    wide = torch.full((5, 7, 64), 3.0, dtype=torch.bfloat16, device=dev)
    vt.rope(x, torch.arange(5, dtype=torch.int32, device=dev), inv, out=wide[:, 1:3])
    assert (wide[:, 0] == 3).all() and (wide[:, 3:] == 3).all()
    check_rotated(wide[:, 1:3], x, torch.arange(5), inv, False, 1.0)


def test_rope_empty(dev):
    inv, _ = vt.rope_frequencies(64)
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)
    assert vt.rope(x, torch.empty((0,), dtype=torch.int32, device=dev), inv).shape == (0, 2, 64)


# ---------------------------------------------------------------------------
def run_append(batch, kv_heads, head_dim, dev, q_heads, rot, interleaved=False, positions=None, amplitude=1.0,
               with_q=True, seed=5):
    T = batch.q.shape[0]
    io = STORE[batch.dtype]
    qkv = rows(T, q_heads + 2 * kv_heads, head_dim, io, dev, seed)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    inv = vt.rope_frequencies(rot, 10000.0)[0] if rot else None
    kc, vc = batch.k_cache.clone(), batch.v_cache.clone()
    kw = dict(q=q if with_q else None, positions=positions, inv_freq=inv, interleaved=interleaved,
              amplitude=amplitude)
    if with_q:
        kw["q_out"] = torch.full((T, q_heads, head_dim), 7.0, dtype=io, device=dev)
    if batch.dtype == "e4m3":
        out = vt.append_fp8(k, v, kc, vc, batch.k_scale, batch.v_scale, batch.q_starts, batch.block_tables,
                            batch.context_lens, **kw)
    else:
        out = vt.append(k, v, kc, vc, batch.q_starts, batch.block_tables, batch.context_lens, **kw)
    return q, k, v, inv, kc, vc, out


def check_append(batch, q, k, v, inv, kc, vc, out, interleaved=False, positions=None, amplitude=1.0):
    """Every owned new slot holds its row, every other byte of the caches is
    the old one, every padding row of q_out too."""
    live = batch.starts[-1]
    pos = torch.tensor([L - n + j for n, L in zip(batch.new, batch.ctx) for j in range(n)], device=kc.device)
    seq = [b for b, n in enumerate(batch.new) for _ in range(n)]
    angle = pos if positions is None else positions[:live]
    page = torch.stack([batch.block_tables[b, int(p) // PAGE] for b, p in zip(seq, pos)]).long()
    slot = pos % PAGE
    touched = torch.zeros(kc.shape[:2], dtype=torch.bool, device=kc.device)
    touched[page, slot] = True
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[kc.element_size()]
    for new, old in ((kc, batch.k_cache), (vc, batch.v_cache)):
        assert torch.equal(new[~touched].view(bits), old[~touched].view(bits))

    def rotated(x):
        if inv is None:
            return x.double(), torch.zeros_like(x, dtype=torch.float64)
        return rotate(x, angle, inv, interleaved, amplitude)

    for cache, x, scale, (ref, mag) in ((kc, k, batch.k_scale, rotated(k[:live])),
                                        (vc, v, batch.v_scale, (v[:live].double(), torch.zeros_like(
                                            v[:live], dtype=torch.float64)))):
        got = cache[page, slot]
        if batch.dtype == "e4m3":
            y = (ref / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            # the quotient is one more fp32 rounding
            slack = mag * ARITH / scale.double()[:, None] + y.abs() * 2.0 ** -23
            err = (got.view(torch.float8_e4m3fn).double() - y).abs()
            assert (err <= torch.maximum((y.abs() + slack) * 2.0 ** -4, torch.tensor(2.0 ** -10)) + slack).all()
        else:
            err = (got.double() - ref).abs()
            assert (err <= mag * ARITH + (ref.abs() + mag * ARITH) * HALF_STEP[got.dtype]).all()
    if out is not None:
        ref, mag = rotated(q[:live])
        err = (out[:live].double() - ref).abs()
        assert (err <= mag * ARITH + (ref.abs() + mag * ARITH) * HALF_STEP[out.dtype]).all()
        assert (out[live:] == 7).all()


RAGGED = [([1], [1]), ([1, 1, 1, 1], [33, 1, 64, 100]), ([0, 5, 0, 33, 64, 0], [40, 5, 0, 65, 64, 7]),
          ([100, 1, 31], [100, 500, 63])]


@pytest.mark.parametrize("new,ctx", RAGGED)
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 512), ("f32", 128), ("f32", 256),
                                     ("e4m3", 64), ("e4m3", 256)])
def test_append(dev, new, ctx, dtype, D):
    batch = make_batch(new, ctx, 6, 2, D, dtype, seed=len(new), pad=3)
    for interleaved in (False, True):
        got = run_append(batch, 2, D, dev, 6, D, interleaved)
        check_append(batch, *got, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, True), (64, False), (36, True), (36, False)])
def test_append_part_of_the_head(dev, dtype, rot, interleaved):
    batch = make_batch([3, 70], [10, 70], 4, 4, 128, dtype, pad=1)
    got = run_append(batch, 4, 128, dev, 4, rot, interleaved, amplitude=1.2 if rot else 1.0)
    check_append(batch, *got, interleaved=interleaved, amplitude=1.2)


def test_append_given_positions_and_no_queries(dev):
    batch = make_batch([4, 9], [50, 9], 2, 1, 128, "bf16", pad=2)
    positions = torch.arange(15, dtype=torch.int32, device=dev) * -1000 + 3
    got = run_append(batch, 1, 128, dev, 2, 128, positions=positions, with_q=False)
    assert got[-1] is None
    check_append(batch, *got, positions=positions)


def test_append_many_sequences(dev):
    """More sequences than one probe round of the row lookup, empty ones among them, and enough tokens for blocks of
    several tokens."""
    g = torch.Generator().manual_seed(3)
    new = [int(x) if x < 5 else 0 for x in torch.randint(0, 8, (1500,), generator=g)]
    ctx = [n + int(x) for n, x in zip(new, torch.randint(0, 60, (1500,), generator=g))]
    batch = make_batch(new, ctx, 2, 1, 64, "bf16", pad=5)
    check_append(batch, *run_append(batch, 1, 64, dev, 2, 64))


@pytest.mark.parametrize("dtype,heads", [("bf16", 20), ("e4m3", 20), ("f32", 28)])
def test_append_where_shares_cut_tokens(dev, dtype, heads):
    """Enough tokens and heads for warps' shares to begin and end inside tokens, at sequences' ends too."""
    batch = make_batch([1511, 0, 1607, 3], [2000, 10, 1607, 77], heads, 4, 128, dtype, pad=6)
    check_append(batch, *run_append(batch, 4, 128, dev, heads, 128))


def test_append_one_long_prompt(dev):
    batch = make_batch([4097], [4100], 4, 2, 64, "bf16")
    check_append(batch, *run_append(batch, 2, 64, dev, 4, 64))


def test_append_bad_device_data(dev):
    """Contexts and pages out of range: nothing is written for them, the sequence's query rows are NaN, the others
    are as ever."""
    batch = make_batch([2, 2, 2, 2], [40, 40, 40, 40], 2, 1, 64, "bf16")
    batch.context_lens[1] = 1                      # fewer tokens than new ones
    batch.context_lens[2] = 10 ** 6                # past the table row
    batch.block_tables[3, 1] = batch.k_cache.shape[0]  # token 38, 39: past the pool
    q, k, v, inv, kc, vc, out = run_append(batch, 1, 64, dev, 2, 64)
    torch.cuda.synchronize()
    assert torch.isnan(out[2:6]).all() and torch.isfinite(out[:2]).all() and torch.isfinite(out[6:]).all()
    wrote = (kc.view(torch.int16) != batch.k_cache.view(torch.int16)).flatten(2).any(-1)
    assert int(wrote.sum()) == 2 and wrote[batch.block_tables[0, 1].long()].sum() == 2


def test_append_nan_and_large_values_in_codes(dev):
    """NaN stays NaN, magnitudes past the scale's range are held at 448."""
    batch = make_batch([1], [1], 1, 1, 64, "e4m3")
    k = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device=dev)
    k[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -1e30, 1e30])
    kc, vc = batch.k_cache.clone(), batch.v_cache.clone()
    vt.append_fp8(k, k, kc, vc, batch.k_scale, batch.v_scale, batch.q_starts, batch.block_tables, batch.context_lens)
    got = vc[batch.block_tables[0, 0].long(), 0, 0].view(torch.float8_e4m3fn).float()
    assert torch.isnan(got[0]) and got[1:4].tolist() == [448.0, -448.0, 448.0] and (got[4:] == 0).all()


def test_append_captured(dev):
    """Replays of a captured append read the buffers as they then are."""
    batch = make_batch([1, 1], [5, 33], 2, 1, 64, "bf16")
    got = run_append(batch, 1, 64, dev, 2, 64)
    q, k, v, inv, kc, vc, out = got
    kc2, vc2, out2 = batch.k_cache.clone(), batch.v_cache.clone(), torch.full_like(out, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.append(k, v, kc2, vc2, batch.q_starts, batch.block_tables, batch.context_lens, q=q, q_out=out2,
                  inv_freq=inv)
    batch.context_lens.sub_(1)
    graph.replay()
    torch.cuda.synchronize()
    batch.ctx = [4, 32]
    check_append(batch, q, k, v, inv, kc2, vc2, out2)


@pytest.mark.parametrize("rot", [64, 36])          # both kernels
@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("starts,must", [
    ([-2 ** 31, 100, 100, 100], []), ([-2 ** 31, -2 ** 31, 4, 8], [2]), ([-5, 4, 8, 12], [1, 2]),
    ([0, 4, 400, 12], [0]), ([0, 4, 2 ** 31 - 1, 2 ** 31 - 1], [0]), ([0, 8, 4, 12], []),
    ([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31], []),
])
def test_append_bad_row_starts(dev, dtype, rot, starts, must):
    """Starts below 0, that decrease or pass the rows: those sequences have no rows; nothing is written for them and
    nothing is read outside the tables, whatever the contexts.  (Where starts decrease, rows of two sequences overlap,
    and some may be left.)"""
    for lens in ([60, 61, 62], [0, 0, 0], [1, 2 ** 31 - 1, -2 ** 31]):
        batch = make_batch([4, 4, 4], [60, 61, 62], 2, 1, 64, dtype)
        batch.q_starts.copy_(torch.tensor(starts, dtype=torch.int32))
        batch.context_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q, k, v, inv, kc, vc, out = run_append(batch, 1, 64, dev, 2, rot)
        torch.cuda.synchronize()
        rows = torch.zeros(12, dtype=torch.bool, device=dev)
        slots = torch.zeros(kc.shape[:2], dtype=torch.bool, device=dev)
        for b in range(3):
            n = starts[b + 1] - starts[b]
            if starts[b] < 0 or n <= 0 or starts[b + 1] > 12:
                assert b not in must
                continue
            rows[starts[b]:starts[b + 1]] = True
            for p in range(lens[b] - n, lens[b]) if n <= lens[b] <= 64 else ():
                slots[batch.block_tables[b, p // 32].long(), p % 32] = True
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[kc.element_size()]
        for new, old in ((kc, batch.k_cache), (vc, batch.v_cache)):
            assert torch.equal(new[~slots].view(bits), old[~slots].view(bits))
        assert (out[~rows] == 7).all()
        for b in must:
            assert not (out[starts[b]:starts[b + 1]] == 7).all(-1).any()


def test_one_token_has_no_stride(dev):
    """Of one row the distance to the next means nothing: a fused projection's only row is rotated in place by the
    append, and an odd distance is no fault."""
    batch = make_batch([1], [40], 4, 2, 64, "bf16")
    qkv = rows(1, 8, 64, torch.bfloat16, dev)
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    inv, _ = vt.rope_frequencies(64)
    args = (batch.q_starts, batch.block_tables, batch.context_lens)
    caches = [(batch.k_cache.clone(), batch.v_cache.clone()) for _ in range(2)]
    want = vt.append(k, v, *caches[0], *args, q=q, inv_freq=inv)
    assert vt.append(k, v, *caches[1], *args, q=q, q_out=q, inv_freq=inv) is q
    assert torch.equal(q, want)
    for a, b in zip(*caches):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    x = torch.empty_strided((1, 4, 64), (257, 64, 1), dtype=torch.bfloat16, device=dev)
    x.copy_(rows(1, 4, 64, torch.bfloat16, dev, seed=3))
    pos = torch.tensor([77], dtype=torch.int32, device=dev)
    check_rotated(vt.rope(x, pos, inv), x, pos, inv, False, 1.0)

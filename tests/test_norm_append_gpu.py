"""The norm of query and key heads with the rotation and the paged append,
against its 64-bit form (GPU).

Tolerances, from the arithmetic.  A sum of D <= 1024 squares is at most 37 fp32
additions deep (32 a lane, 5 over lanes; 16 elements a lane and 5 in the
vectorised kernel), so with the squares' and the mean's own roundings it is off by
2^-18.5 of itself and its root by half that; rsqrtf() by 2^-22; two products by
2^-24 each: below 2^-18 of an element.  The rotation adds 2^-20 of |a| + |b|
(test_rope_append_gpu.py), the storage type half a step.
"""
from __future__ import annotations

import pytest
import torch

import paged_attention_decode_kv_gb300 as vt
from ragged import E4M3_MAX, PAGE, STORE, make_batch, rotate

pytestmark = pytest.mark.gpu

ARITH = 2.0 ** -20 + 2.0 ** -18
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
    """[T][H][D] of heads of different sizes, a view into rows of H + extra heads."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H + extra, D), generator=g) * torch.logspace(-2, 2, H + extra)[:, None]
    return x.to(dtype).to(dev)[:, :H]


def weights(H, D, per_head, dev, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.5 * torch.randn((H, D) if per_head else (D,), generator=g)).to(dev)


def normed(x, weight, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()


def expected(x, weight, eps, positions, inv, interleaved, amplitude):
    """(value, tolerance before the storage type's rounding)."""
    y = normed(x, weight, eps)
    if inv is None:
        return y, y.abs() * ARITH
    ref, mag = rotate(y, positions, inv, interleaved, amplitude)
    return ref, torch.maximum(mag, ref.abs()) * ARITH


def check_rows(got, ref, tol):
    assert torch.isfinite(got).all()
    bound = tol + (ref.abs() + tol) * HALF_STEP[got.dtype]
    err = (got.double() - ref).abs()
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (7, 3, 128, 128), (33, 5, 128, 64), (5, 2, 256, 34),
                                       (130, 1, 80, 48), (3, 4, 512, 512), (2, 2, 1024, 1024), (9, 1, 8, 2),
                                       (4, 3, 128, 0), (3, 2, 24, 0), (2999, 20, 128, 128), (4001, 31, 64, 64),
                                       (3001, 9, 256, 128)])
def test_norm_rope(dev, T, H, D, rot, dtype, interleaved, per_head):
    inv = vt.rope_frequencies(rot, 10000.0)[0] if rot else None
    g = torch.Generator().manual_seed(T + D)
    positions = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32).to(dev)
    x = rows(T, H, D, dtype, dev, extra=2)
    w = weights(H, D, per_head, dev)
    got = vt.norm_rope(x, w, positions if rot else None, inv, eps=1e-5, interleaved=interleaved, amplitude=1.25)
    ref, tol = expected(x, w, 1e-5, positions, inv, interleaved, 1.25)
    check_rows(got, ref, tol)


@pytest.mark.parametrize("rot,D", [(128, 128), (20, 128), (64, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_and_padding(dev, rot, D, dtype):
    inv, _ = vt.rope_frequencies(rot)
    positions = torch.arange(70, dtype=torch.int32, device=dev) * 37
    wide = rows(70, 5, D, dtype, dev, extra=1)
    before = wide.clone()
    x = wide[:, 1:4]
    w = weights(3, D, True, dev)
    y = vt.norm_rope(x, w, positions, inv)
    assert vt.norm_rope(x, w, positions, inv, out=x) is x
    assert torch.equal(x, y)
    assert torch.equal(wide[:, :1], before[:, :1]) and torch.equal(wide[:, 4:], before[:, 4:])


@pytest.mark.parametrize("D,rot", [(128, 128), (72, 8)])
def test_rows_of_zeros_and_extremes(dev, D, rot):
    """A row of zeros stays 0 (eps > 0); tiny rows are held up by eps, not blown up; NaN and inf stay in their row."""
    inv, _ = vt.rope_frequencies(rot)
    x = torch.zeros((5, 1, D), dtype=torch.float32, device=dev)
    x[1] = 1e-12
    x[2] = 1e8 * torch.linspace(-1, 1, D, device=dev)
    x[3, 0, 3] = float("nan")
    x[4, 0, 5] = float("inf")
    w = torch.ones(D, device=dev)
    positions = torch.zeros(5, dtype=torch.int32, device=dev)
    got = vt.norm_rope(x, w, positions, inv, eps=1e-6)
    assert (got[0] == 0).all()
    ref, tol = expected(x[:3], w, 1e-6, positions[:3], inv, False, 1.0)
    check_rows(got[:3], ref, tol)
    assert torch.isnan(got[3]).all()
    assert not torch.isfinite(got[4, 0, 5])
    zero = vt.norm_rope(x[:1], w, positions[:1], inv, eps=0.0)
    assert torch.isnan(zero).all()                      # 0 / 0


def test_empty(dev):
    x = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)
    inv, _ = vt.rope_frequencies(64)
    assert vt.norm_rope(x, torch.ones(64, device=dev), torch.empty((0,), dtype=torch.int32, device=dev),
                        inv).shape == (0, 2, 64)


# ---------------------------------------------------------------------------
def run_append(batch, kv_heads, head_dim, dev, q_heads, rot, interleaved=False, positions=None, per_head=False,
               with_q=True, seed=5):
    T = batch.q.shape[0]
    io = STORE[batch.dtype]
    qkv = rows(T, q_heads + 2 * kv_heads, head_dim, io, dev, seed)
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    inv = vt.rope_frequencies(rot, 10000.0)[0] if rot else None
    kc, vc = batch.k_cache.clone(), batch.v_cache.clone()
    kw, qw = weights(kv_heads, head_dim, per_head, dev, 2), weights(q_heads, head_dim, per_head, dev, 3)
    args = dict(q=q if with_q else None, q_weight=qw if with_q else None, positions=positions, inv_freq=inv,
                interleaved=interleaved, eps=1e-6)
    if with_q:
        args["q_out"] = torch.full((T, q_heads, head_dim), 7.0, dtype=io, device=dev)
    where = (batch.q_starts, batch.block_tables, batch.context_lens)
    if batch.dtype == "e4m3":
        out = vt.norm_append_fp8(k, v, kw, kc, vc, batch.k_scale, batch.v_scale, *where, **args)
    else:
        out = vt.norm_append(k, v, kw, kc, vc, *where, **args)
    return q, k, v, qw, kw, inv, kc, vc, out


def check_append(batch, q, k, v, qw, kw, inv, kc, vc, out, interleaved=False, positions=None):
    """Every owned new slot holds its row, every other byte of the caches is as it was, padding rows too."""
    live = batch.starts[-1]
    dev = k.device
    pos, slot = [], []
    table = batch.block_tables.tolist()
    for b, (n, L) in enumerate(zip(batch.new, batch.ctx)):
        for p in range(L - n, L):
            pos.append(p)
            slot.append(table[b][p // PAGE] * PAGE + p % PAGE)
    at = torch.tensor(pos, dtype=torch.int32, device=dev) if positions is None else positions[:live]
    slot = torch.tensor(slot, dtype=torch.long, device=dev)
    if out is not None:
        ref, tol = expected(q[:live], qw, 1e-6, at, inv, interleaved, 1.0)
        check_rows(out[:live], ref, tol)
        assert (out[live:] == 7).all()
    ref, tol = expected(k[:live], kw, 1e-6, at, inv, interleaved, 1.0)
    for cache, old, want, bound, scale in ((kc, batch.k_cache, ref, tol, batch.k_scale),
                                           (vc, batch.v_cache, v[:live].double(), torch.zeros_like(ref), batch.v_scale)):
        flat, was = cache.flatten(0, 1), old.flatten(0, 1)
        if batch.dtype == "e4m3":
            s = scale.double()[:, None]
            got = flat[slot].view(torch.float8_e4m3fn).double() * s
            want = want.clamp(-E4M3_MAX * s, E4M3_MAX * s)
            bound = bound + 2.0 ** -22 * want.abs()
            err = (got - want).abs()
            assert (err <= bound + (want.abs() + bound) * 2.0 ** -4 + s * 2.0 ** -10).all()
        else:
            check_rows(flat[slot], want, bound)
        others = torch.ones(flat.shape[0], dtype=torch.bool, device=dev)
        others[slot] = False
        bytes_of = lambda x: x.contiguous().view(torch.uint8)  # noqa: E731 (NaN compares unequal)
        assert torch.equal(bytes_of(flat[others]), bytes_of(was[others]))


KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 512), ("f32", 64), ("f32", 128), ("f32", 256),
         ("e4m3", 64), ("e4m3", 128), ("e4m3", 256)]


@pytest.mark.parametrize("rot", ["all", "half", "some", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_append(dev, dtype, D, interleaved, rot):
    turned = {"all": D, "half": D // 2, "some": 22, "none": 0}[rot]
    batch = make_batch([1, 33, 0, 70], [40, 33, 5, 300], 6, 2, D, dtype, seed=D, pad=3)
    got = run_append(batch, 2, D, dev, 6, turned, interleaved, per_head=interleaved)
    check_append(batch, *got, interleaved=interleaved)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64), ("e4m3", 128)])
@pytest.mark.parametrize("new,ctx,q_heads,kv_heads", [([1], [1], 1, 1), ([1] * 130, list(range(1, 131)), 32, 8),
                                                      ([700, 2900], [900, 2900], 5, 1), ([0, 0, 2], [9, 0, 2], 14, 2)])
def test_append_shapes(dev, dtype, D, new, ctx, q_heads, kv_heads):
    batch = make_batch(new, ctx, q_heads, kv_heads, D, dtype, seed=1)
    check_append(batch, *run_append(batch, kv_heads, D, dev, q_heads, D))


@pytest.mark.parametrize("rot", [128, 30])
def test_append_without_queries_and_with_positions(dev, rot):
    batch = make_batch([4, 9], [40, 9], 4, 2, 128, "bf16", pad=2)
    positions = torch.arange(15, dtype=torch.int32, device=dev) * 1000
    got = run_append(batch, 2, 128, dev, 4, rot, positions=positions, with_q=False)
    assert got[-1] is None
    check_append(batch, *got, positions=positions)


@pytest.mark.parametrize("rot", [128, 30])
def test_append_invalid_device_data(dev, rot):
    """A bad context gives NaN query rows and writes nothing; a bad page id only its tokens' keys and values."""
    batch = make_batch([3, 4, 40], [20, 30, 60], 4, 2, 128, "bf16")
    batch.context_lens[0] = 2             # fewer than its rows
    batch.block_tables[2, 1] = 10 ** 6    # its tokens 32 .. 59
    q, k, v, qw, kw, inv, kc, vc, out = run_append(batch, 2, 128, dev, 4, rot)
    assert torch.isnan(out[:3]).all() and torch.isfinite(out[3:]).all()
    ref, tol = expected(q[3:7], qw, 1e-6, torch.arange(26, 30, device=dev), inv, False, 1.0)
    check_rows(out[3:7], ref, tol)
    fresh = batch.k_cache.clone()
    page = int(batch.block_tables[1, 0])
    ref, tol = expected(k[3:7], kw, 1e-6, torch.arange(26, 30, device=dev), inv, False, 1.0)
    check_rows(kc[page, 26:30], ref, tol)
    fresh[page, 26:30] = kc[page, 26:30]
    page = int(batch.block_tables[2, 0])
    fresh[page, 20:32] = kc[page, 20:32]
    assert torch.equal(fresh.view(torch.int16), kc.view(torch.int16))


# Batches of so many units a warp (152 SMs, 16 warps each, units of four bf16 or two fp32 rounds of 512 elements) that
# rows come through shared memory ahead of their turn; heads that fill neither rounds nor units.
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D,rot", [(6203, 17, 128, 128), (6200, 17, 128, 48), (6211, 33, 64, 64), (6201, 9, 256, 0),
                                       (4203, 9, 512, 32)])
def test_norm_rope_long(dev, T, H, D, rot, dtype, interleaved, per_head):
    inv = vt.rope_frequencies(rot, 10000.0)[0] if rot else None
    g = torch.Generator().manual_seed(T + D)
    positions = torch.randint(-5000, 200000, (T,), generator=g, dtype=torch.int32).to(dev)
    x = rows(T, H, D, dtype, dev, extra=2)
    w = weights(H, D, per_head, dev)
    got = vt.norm_rope(x, w, positions if rot else None, inv, eps=1e-5, interleaved=interleaved, amplitude=1.25)
    check_rows(got, *expected(x, w, 1e-5, positions, inv, interleaved, 1.25))
    assert vt.norm_rope(x, w, positions if rot else None, inv, eps=1e-5, interleaved=interleaved, amplitude=1.25,
                        out=x) is x
    assert torch.equal(x, got)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,q_heads,kv_heads", [
    ("bf16", 64, 25, 4), ("bf16", 128, 9, 4), ("bf16", 256, 5, 2), ("bf16", 512, 3, 1), ("f32", 64, 25, 4),
    ("f32", 128, 9, 4), ("f32", 256, 5, 2), ("e4m3", 64, 25, 4), ("e4m3", 128, 9, 4), ("e4m3", 256, 5, 2)])
def test_append_long(dev, dtype, D, q_heads, kv_heads, interleaved):
    """Long batches, whose last sequence's context is shorter than its rows, with padding rows behind."""
    new, ctx = [4100, 0, 1, 2099, 3], [4100, 5, 77, 2500, 64]
    batch = make_batch(new, ctx, q_heads, kv_heads, D, dtype, seed=D, pad=4)
    batch.context_lens[4] = 2
    live = sum(new[:4])
    q, k, v, qw, kw, inv, kc, vc, out = run_append(batch, kv_heads, D, dev, q_heads, D if interleaved else D // 2,
                                                   interleaved, per_head=interleaved)
    assert torch.isnan(out[live:live + 3]).all() and (out[live + 3:] == 7).all()
    again = q.contiguous()
    scales = (batch.k_scale, batch.v_scale) if dtype == "e4m3" else ()
    (vt.norm_append_fp8 if scales else vt.norm_append)(
        k, v, kw, batch.k_cache.clone(), batch.v_cache.clone(), *scales, batch.q_starts, batch.block_tables,
        batch.context_lens, q=again, q_weight=qw, q_out=again, inv_freq=inv, interleaved=interleaved, eps=1e-6)
    assert torch.equal(again[:live], out[:live])
    batch.new, batch.ctx, batch.q_starts = new[:4], ctx[:4], batch.q_starts[:5]
    check_append(batch, q, k, v, qw, kw, inv, kc, vc, out[:live], interleaved=interleaved)


def test_captured_on_a_stream(dev):
    batch = make_batch([1, 2, 3], [30, 60, 90], 8, 2, 128, "bf16")
    side = torch.cuda.Stream()
    want = run_append(batch, 2, 128, dev, 8, 128)
    q, k, v, qw, kw, inv = want[:6]
    kc, vc, out = batch.k_cache.clone(), batch.v_cache.clone(), torch.zeros_like(want[-1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        vt.norm_append(k, v, kw, kc, vc, batch.q_starts, batch.block_tables, batch.context_lens, q=q, q_weight=qw,
                       q_out=out, inv_freq=inv)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[-1])
    assert torch.equal(kc.view(torch.int16), want[6].view(torch.int16))
    side.wait_stream(torch.cuda.current_stream())
    got = vt.norm_rope(q, qw, torch.zeros(6, dtype=torch.int32, device=dev), inv, stream=side)
    side.synchronize()
    check_rows(got, *expected(q, qw, 1e-6, torch.zeros(6, dtype=torch.int32), inv, False, 1.0))


def test_refusals(dev):
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    pos = torch.zeros(2, dtype=torch.int32, device=dev)
    inv, _ = vt.rope_frequencies(64)
    for bad, error in ((w.bfloat16(), TypeError), (w[:32], ValueError), (torch.ones((3, 64), device=dev), ValueError),
                       (w.cpu(), ValueError), (torch.ones((4, 128), device=dev)[:, ::2], ValueError), (None, ValueError)):
        with pytest.raises(error):
            vt.norm_rope(x, bad, pos, inv)
    with pytest.raises(ValueError):
        vt.norm_rope(x, w, None, inv)
    with pytest.raises(vt.VtError):
        vt.norm_rope(x, w, pos, inv, eps=-1.0)
    with pytest.raises(vt.VtError):
        vt.norm_rope(x, torch.ones(65, device=dev)[1:], pos, inv)      # not on 16 bytes
    batch = make_batch([2], [2], 4, 2, 64, "bf16")
    kv = x[:, :2]
    with pytest.raises(ValueError):
        vt.norm_append(kv, kv, None, batch.k_cache, batch.v_cache, batch.q_starts, batch.block_tables,
                       batch.context_lens)
    with pytest.raises(ValueError):
        vt.norm_append(kv, kv, w, batch.k_cache, batch.v_cache, batch.q_starts, batch.block_tables,
                       batch.context_lens, q=x)                        # queries without their weights

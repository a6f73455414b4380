"""Ragged prefill over the paged cache against its 64-bit form (GPU).

Tolerances, from the kernel's arithmetic, with w = sum_t p_t |v_t| of an
output element: the softmax weights are rounded to bf16 (2^-8 of each, so at
most 2^-8 w), or for codes to f16 (2^-11, and 2^-25 of the largest), the
output to bf16 (2^-8 of it); scores, their exponentials and sums are fp32,
whose errors over D products and a few thousand keys stay below 2^-12 w at
these magnitudes.  Codes: a query is two E4M3 terms, off by at most 2^-17 of
the row's largest magnitude an element, so a score by up to
e = 2^-17 max|q| sum_d |k_d| scale, twice that in weights that are
quotients, 2 e w.  fp32 storage: a score sums D products of magnitude up to
sum |q k| with 2^-24 each, the output up to n of them.
"""
from __future__ import annotations

import pytest
import torch

import paged_attention_decode_kv_gb300 as vt
from ragged import attention, make_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from paged_attention_decode_kv_gb300 import build_lib
    build_lib.build()
    vt.library()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _reset():
    yield
    if vt._lib is not None:
        vt.vt_paged_attn_set_override(0, 0)
        vt.vt_paged_attn_set_test_wait(0, -1, -1)
        vt.vt_paged_attn_set_workspace(0, 0)


def run(batch, scale=None, window=0, out=None, grid=0, blocks=0, stream=None):
    vt.vt_paged_attn_set_override(grid, blocks)
    if batch.dtype == "e4m3":
        out = vt.prefill_fp8(batch.q, batch.k_cache, batch.v_cache, batch.k_scale, batch.v_scale, batch.q_starts,
                             batch.block_tables, batch.context_lens, scale, window, out=out, stream=stream)
    else:
        out = vt.prefill(batch.q, batch.k_cache, batch.v_cache, batch.q_starts, batch.block_tables,
                         batch.context_lens, scale, window, out=out, stream=stream)
    vt.vt_paged_attn_set_override(0, 0)
    return out


def check(batch, got, scale=None, window=0):
    live, D = batch.starts[-1], batch.q.shape[2]
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    plan = vt.vt_paged_attn_last_plan()
    assert plan["tensor_cores"] == (0 if batch.dtype == "f32" else 1)
    ref, reach, even = attention(batch, D ** -0.5 if scale is None else scale, window, flat=True)
    ref, reach, even, got = ref[:live], reach[:live], even[:live], got[:live].double()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    if batch.dtype == "f32":
        n = max(batch.ctx)
        span = float(batch.q[:live].double().norm(dim=-1).max()) * 1.5 * D ** 0.5 * abs(
            D ** -0.5 if scale is None else scale)   # no |q||k| scale is above it (k rows: 1.5 sqrt(D) at most)
        tol = ((2 * D * span + n + 16) * 2.0 ** -24) * reach
    else:
        tol = (2.0 ** -8 + 2.0 ** -12) * reach + 2.0 ** -8 * ref.abs() + 1e-30
        if batch.dtype == "e4m3":
            most = batch.q[:live].double().abs().amax(-1, keepdim=True)
            keys = max(float(k.abs().sum(-1).max()) for k in batch.dense("k") if k.numel())
            e = 2.0 ** -17 * most * keys * abs(D ** -0.5 if scale is None else scale)
            tol = (2.0 ** -11 + 2.0 ** -12 + 2 * e) * reach + 2.0 ** -8 * ref.abs() + 2.0 ** -25 * even
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    if live:
        nmse = float((err ** 2).sum() / (ref ** 2).sum())
        assert nmse <= (1e-10 if batch.dtype == "f32" else 2e-5), nmse


#: (type, head_dim): every kernel
KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 512), ("f32", 64), ("f32", 128), ("f32", 256),
         ("e4m3", 64), ("e4m3", 128), ("e4m3", 256)]
SHAPES = {
    "one_token": ([1], [1]),
    "first_tokens": ([2, 3], [2, 3]),
    "decode_rows": ([1, 1, 1], [33, 100, 257]),
    "page_edges": ([31, 32, 33, 64], [31, 64, 97, 300]),
    "empty_between": ([0, 7, 0, 0, 130, 0], [5, 7, 0, 300, 131, 64]),
    "block_edges": ([127, 128, 129], [128, 256, 385]),
    "long": ([300, 1, 65], [300, 1025, 900]),
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D", KINDS)
def test_shapes(dev, dtype, D, shape):
    new, ctx = SHAPES[shape]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=D)
    check(batch, run(batch))


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (6, 2), (5, 1), (14, 2), (16, 2), (33, 1), (64, 1)])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("e4m3", 128)])
def test_groups(dev, dtype, D, q_heads, kv_heads):
    batch = make_batch([70, 3, 131], [200, 3, 131], q_heads, kv_heads, D, dtype, seed=q_heads)
    check(batch, run(batch))


@pytest.mark.parametrize("window", [1, 2, 31, 33, 128, 200, 1000])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_windows(dev, dtype, D, window):
    batch = make_batch([150, 1, 40], [500, 300, 40], 4, 2, D, dtype, seed=window)
    check(batch, run(batch, window=window), window=window)


@pytest.mark.parametrize("grid", [1, 2, 3, 7, 40, 152, 400])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_forced_partitions(dev, dtype, D, grid):
    """Any number of CTAs, down to shares of two blocks, so that items are cut everywhere."""
    batch = make_batch([100, 260, 5, 1], [1200, 260, 900, 2000], 8, 2, D, dtype, seed=1)
    got = run(batch, grid=grid, blocks=2)
    assert vt.vt_paged_attn_last_plan()["grid_ctas"] == grid
    check(batch, got)
    assert torch.equal(got, run(batch, grid=grid, blocks=2))  # the same bits every time


@pytest.mark.parametrize("grid", [7, 152])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_forced_partitions_with_a_window(dev, dtype, D, grid):
    batch = make_batch([100, 260, 5, 1], [1200, 260, 900, 2000], 8, 2, D, dtype, seed=2)
    check(batch, run(batch, grid=grid, blocks=2, window=333), window=333)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5, 2.0])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 128), ("e4m3", 128)])
def test_scales(dev, dtype, D, scale):
    """Flat, reversed and peaked softmax (peaked: scores up to about 150, so a score error of 2^-20 of that is
    2^-12)."""
    batch = make_batch([200, 9], [300, 70], 4, 2, D, dtype, seed=3)
    check(batch, run(batch, scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_growing_scores(dev, dtype, D):
    """Keys that grow along the context move the running maximum at every block."""
    batch = make_batch([64, 10], [1000, 800], 4, 2, D, dtype, seed=4)
    if dtype == "e4m3":
        batch.k_scale = batch.k_scale * 2
    else:
        for b, L in enumerate(batch.ctx):
            for i in range((L + 31) // 32):
                batch.k_cache[batch.block_tables[b, i].long()] *= 2.0 ** min(3, i // 8)
    check(batch, run(batch, scale=D ** -0.5 / 2), scale=D ** -0.5 / 2)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_padding_rows_are_kept(dev, dtype, D):
    batch = make_batch([5, 0, 140], [5, 9, 200], 4, 2, D, dtype, pad=19)
    out = torch.full_like(batch.q, 3.0)
    check(batch, run(batch, out=out))
    assert (out[145:] == 3).all()


@pytest.mark.parametrize("dtype,D", KINDS)
def test_bad_device_data(dev, dtype, D):
    batch = make_batch([20, 20, 20, 20, 20], [100] * 5, 4, 2, D, dtype)
    good, _ = attention(batch, D ** -0.5)
    batch.context_lens[1] = 19
    batch.context_lens[2] = 10 ** 6
    batch.context_lens[4] = -5
    batch.block_tables[3, 1] = batch.k_cache.shape[0]
    for grid in (0, 11):
        out = run(batch, grid=grid, blocks=2 if grid else 0)
        torch.cuda.synchronize()
        assert vt.vt_paged_attn_device_status() == 0
        assert torch.isnan(out[20:]).all()
        assert (out[:20].double() - good[:20]).abs().max() < 0.02


def test_bad_row_starts(dev):
    """Starts that decrease or pass the rows: those sequences have no rows; nothing faults."""
    batch = make_batch([8, 8, 8], [40, 40, 40], 4, 2, 128, "bf16")
    good, _ = attention(batch, 128 ** -0.5)
    out = torch.full_like(batch.q, 3.0)
    batch.q_starts.copy_(torch.tensor([0, 8, 4, 400], dtype=torch.int32))
    run(batch, out=out)
    torch.cuda.synchronize()
    assert (out[8:] == 3).all() and (out[:8].double() - good[:8]).abs().max() < 0.02


@pytest.mark.parametrize("dtype,D", KINDS)
def test_values_that_are_not_finite_in_masked_places(dev, dtype, D):
    """A value of a later new token that is not finite does not reach the rows before it; rows that attend to it
    are not finite there."""
    batch = make_batch([60], [150], 2, 1, D, dtype)
    ref, _ = attention(batch, D ** -0.5)
    t = 120                                        # position of new token 30
    page = batch.block_tables[0, t // 32].long()
    for col, bits in ((3, float("nan")), (D - 1, float("inf"))):
        if dtype == "e4m3":
            batch.v_cache[page, t % 32, 0, col] = 0x7F
        else:
            batch.v_cache[page, t % 32, 0, col] = bits
    out = run(batch)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:30]).all()
    assert (out[:30].double() - ref[:30]).abs().max() < 0.02
    assert not torch.isfinite(out[30:, :, 3]).any() and not torch.isfinite(out[30:, :, D - 1]).any()
    clean = [c for c in range(D) if c not in (3, D - 1)]
    assert (out[30:][..., clean].double() - ref[30:][..., clean]).abs().max() < 0.02


def test_queries_that_are_not_finite(dev):
    """A row whose query is not finite is NaN, the others are as ever."""
    for dtype, D in (("bf16", 128), ("e4m3", 128), ("e4m3", 256), ("f32", 64)):
        batch = make_batch([40], [150], 2, 1, D, dtype)
        ref, _ = attention(batch, D ** -0.5)
        batch.q[7, 1, 5] = float("inf")
        batch.q[20, 0, 0] = float("nan")
        out = run(batch)
        assert torch.isnan(out[7, 1]).all() and torch.isnan(out[20, 0]).all()
        keep = torch.ones(out.shape[:2], dtype=torch.bool, device=dev)
        keep[7, 1] = keep[20, 0] = False
        assert (out[keep].double() - ref[keep]).abs().max() < 0.02


@pytest.mark.parametrize("dtype,D", KINDS)
def test_bounded_wait_gives_up_and_reports(dev, dtype, D):
    """A withheld block: the waits for it run out, the kernel returns, the status says so, and the next call is
    exact.  (fp32 has no waits: it is not concerned.  CTA 0 has a second block to withhold if shares are of 8.)"""
    if dtype == "f32":
        return
    batch = make_batch([100, 30], [900, 2000], 8, 2, D, dtype)
    run(batch)
    torch.cuda.synchronize()
    vt.vt_paged_attn_set_test_wait(4_000_000, 0, 1)
    run(batch, blocks=8)
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    torch.cuda.synchronize()
    words = vt.vt_paged_attn_device_status_detail()
    assert words[0] != 0 and words[1] == 1
    assert vt.vt_paged_attn_device_status() != 0
    assert vt.vt_paged_attn_device_status() == 0
    check(batch, run(batch, blocks=8))
    check(batch, run(batch))


def test_capture_before_the_first_call_is_refused(dev):
    """The scratch is allocated outside captures only; a refused call leaves the capture usable."""
    batch = make_batch([10], [50], 2, 1, 64, "bf16")
    out = torch.zeros_like(batch.q)
    torch.cuda.synchronize()
    vt.vt_paged_attn_release()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.add_(1)
        with pytest.raises(vt.VtError) as e:
            run(batch, out=out)
    assert e.value.status == vt.VT_ERR_SCRATCH_LIMIT
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 1).all()
    check(batch, run(batch, out=out))


def test_larger_scratch_leaves_a_captured_graph_alone(dev):
    """A call that needs a larger scratch does not take away the one a graph names."""
    batch = make_batch([100, 30], [900, 2000], 8, 2, 64, "bf16")
    out = torch.zeros_like(batch.q)
    torch.cuda.synchronize()
    vt.vt_paged_attn_release()
    run(batch, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(batch, out=out)
    wide = make_batch([100, 30], [900, 2000], 8, 2, 256, "bf16")
    run(wide)
    other = run(wide, grid=400)
    out.zero_()
    graph.replay()
    check(batch, out)
    check(wide, other)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_workspace_of_the_caller(dev, dtype, D):
    batch = make_batch([100, 30], [900, 2000], 8, 2, D, dtype)
    need = vt.vt_paged_attn_prefill_workspace_bytes(D, vt.VT_BF16 if dtype == "bf16" else vt.VT_F32)
    area = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), need)
    got = run(batch)
    assert vt.vt_paged_attn_last_plan()["scratch_source"] == 1
    check(batch, got)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), need - 256)
    with pytest.raises(vt.VtError) as e:
        run(batch)
    assert e.value.status == vt.VT_ERR_SCRATCH_LIMIT


def test_captured_prefill_stays_off_the_decodes_counters(dev):
    """In the caller's area a decode of more sequences extends the counters, which have to stay zero between decodes:
    replays of a prefill captured before it do not write there."""
    batch = make_batch([100, 30], [900, 2000], 8, 2, 64, "bf16")
    area = torch.empty(vt.vt_paged_attn_prefill_workspace_bytes(64, vt.VT_BF16) + (64 << 20), dtype=torch.uint8,
                       device=dev)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), area.numel())
    out = torch.zeros_like(batch.q)
    run(batch, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(batch, out=out)
    seqs = 200000
    table = batch.block_tables[1:2, :4].expand(seqs, 4).contiguous()
    lens = torch.full((seqs,), 100, dtype=torch.int32, device=dev)
    q = torch.randn((seqs, 2, 64), device=dev).to(torch.bfloat16)
    first = vt.decode(q, batch.k_cache, batch.v_cache, table, lens)
    out.zero_()
    graph.replay()
    again = vt.decode(q, batch.k_cache, batch.v_cache, table, lens)
    assert torch.equal(first, again)
    check(batch, out)


def test_captured_and_replayed_with_other_lengths(dev):
    """The plan is made on the device: a replay follows the lengths as they then are."""
    batch = make_batch([100, 30], [900, 2000], 8, 2, 128, "bf16")
    out = torch.zeros_like(batch.q)
    run(batch, out=out)
    other = make_batch([60, 70], [400, 1500], 8, 2, 128, "bf16", seed=8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(batch, out=out)
    graph.replay()
    check(batch, out)
    pages = min(batch.k_cache.shape[0], other.k_cache.shape[0])
    assert other.k_cache.shape[0] <= batch.k_cache.shape[0] and pages == other.k_cache.shape[0]
    batch.k_cache[:pages].copy_(other.k_cache)
    batch.v_cache[:pages].copy_(other.v_cache)
    batch.q.copy_(other.q)
    batch.q_starts.copy_(other.q_starts)
    batch.context_lens.copy_(other.context_lens)
    batch.block_tables[:, : other.block_tables.shape[1]].copy_(other.block_tables)
    batch.new, batch.ctx = other.new, other.ctx
    graph.replay()
    check(batch, out)


def test_other_stream(dev):
    batch = make_batch([64], [700], 8, 2, 128, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(batch, stream=s)
    s.synchronize()
    check(batch, got)


def test_many_sequences(dev):
    """More sequences than threads of a CTA, one to four new tokens each."""
    g = torch.Generator().manual_seed(0)
    new = torch.randint(0, 5, (900,), generator=g).tolist()
    ctx = [n + int(c) for n, c in zip(new, torch.randint(0, 200, (900,), generator=g))]
    batch = make_batch(new, ctx, 4, 1, 64, "bf16")
    check(batch, run(batch))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("e4m3", 128)])
def test_one_chunk_for_all_is_the_multi_token_decode(dev, dtype, D):
    """Uniform chunks, against the decode entry points on the same cache."""
    batch = make_batch([6] * 5, [100, 37, 500, 6, 64], 8, 2, D, dtype)
    got = run(batch)
    q = batch.q.view(5, 6, 8, D)
    args = (batch.block_tables, batch.context_lens)
    if dtype == "e4m3":
        ref = vt.decode_fp8(q, batch.k_cache, batch.v_cache, batch.k_scale, batch.v_scale, *args)
    else:
        ref = vt.decode_multi(q, batch.k_cache, batch.v_cache, *args)
    _, reach = attention(batch, D ** -0.5)
    # both are within their own bounds of the same value
    assert ((got.double() - ref.view_as(got).double()).abs() <= 2.0 ** -5 * reach + 1e-6).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_serving_steps(dev, dtype):
    """Append, prefill, append one token, decode: what a serving loop runs, against dense attention on rotated
    rows."""
    D, Hq, Hkv = 128, 8, 2
    new, ctx = [50, 3, 64], [50, 90, 64]
    batch = make_batch(new, ctx, Hq, Hkv, D, dtype, seed=11)
    io = batch.q.dtype
    inv, amp = vt.rope_frequencies(D, 10000.0, vt.VT_ROPE_YARN, 4.0, 4096)
    g = torch.Generator().manual_seed(2)
    scales = (batch.k_scale, batch.v_scale) if dtype == "e4m3" else ()
    # room for one more token in each sequence
    pool = torch.cat([batch.block_tables, torch.zeros((3, 1), dtype=torch.int32, device=dev)], 1)
    extra = batch.k_cache.shape[0]
    grow = [torch.cat([c, torch.zeros_like(c[:3])]) for c in (batch.k_cache, batch.v_cache)]
    for b, L in enumerate(ctx):
        if L % 32 == 0:
            pool[b, L // 32] = extra + b
    batch.k_cache, batch.v_cache, batch.block_tables = *grow, pool

    def append(rows, starts, lens):
        qkv = torch.randn((rows, Hq + 2 * Hkv, D), generator=g).to(io).to(dev)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        fn = vt.append_fp8 if dtype == "e4m3" else vt.append
        return fn(k, v, batch.k_cache, batch.v_cache, *scales, starts, batch.block_tables, lens, q=q, inv_freq=inv,
                  amplitude=amp)

    batch.q = append(117, batch.q_starts, batch.context_lens)
    check(batch, run(batch))
    lens = batch.context_lens + 1
    q = append(3, torch.arange(4, dtype=torch.int32, device=dev), lens)
    step = batch
    step.q, step.new, step.ctx = q, [1, 1, 1], [L + 1 for L in ctx]
    step.q_starts, step.context_lens = torch.arange(4, dtype=torch.int32, device=dev), lens
    got = run(step)
    check(step, got)
    dec = vt.decode_fp8(q, step.k_cache, step.v_cache, *scales, step.block_tables, lens) if dtype == "e4m3" else \
        vt.decode(q, step.k_cache, step.v_cache, step.block_tables, lens)
    _, reach = attention(step, D ** -0.5)
    assert ((got.double() - dec.double()).abs() <= 2.0 ** -5 * reach + 1e-6).all()


@pytest.mark.parametrize("window", [0, 20000])
@pytest.mark.parametrize("dtype,D", [k for k in KINDS if k[0] != "f32"])
def test_values_that_are_not_finite_over_a_long_context(dev, dtype, D, window):
    """What such a value costs is a matter of the keys that only some rows see, not of the context: two items of one
    CTA over 30000 keys are done within 8 million cycles a wait (128 columns times 30000 keys, a few cycles each,
    are more)."""
    L, n = 30000, 40
    batch = make_batch([n], [L], 4, 2, D, dtype, seed=D)
    spots = [(L - n + 17, 3, "nan"), (L - n + 30, D - 1, "inf")]
    if window:
        spots.append((L - n - window + 12, 5, "nan"))  # at the first rows' window's far end
    rows = torch.arange(L - n, L, device=dev)
    hit = torch.zeros((n, D), dtype=torch.bool, device=dev)
    for t, col, what in spots:
        seen = (rows >= t) & (rows < t + window if window else rows >= t)
        assert 0 < int(seen.sum()) < n
        hit[seen, col] = True
    ref, _ = attention(batch, D ** -0.5, window)
    for t, col, what in spots:
        page = batch.block_tables[0, t // 32].long()
        batch.v_cache[page, t % 32, :, col] = 0x7F if dtype == "e4m3" else float(what)
    vt.vt_paged_attn_set_test_wait(8_000_000, -1, -1)
    out = run(batch, window=window, grid=1)
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    bad = hit[:, None, :].expand_as(out)
    assert not torch.isfinite(out[bad]).any()
    assert (out[~bad].double() - ref[~bad]).abs().max() < 0.02
    check_split = run(batch, window=window)  # the same, in pieces
    torch.cuda.synchronize()
    assert not torch.isfinite(check_split[bad]).any()
    assert (check_split[~bad].double() - ref[~bad]).abs().max() < 0.02


def test_give_up_in_a_scratch_that_a_graph_still_names(dev):
    """A replay whose waits run out reports it although a larger call has meanwhile taken a larger scratch."""
    batch = make_batch([100, 30], [900, 2000], 8, 2, 64, "bf16")
    out = torch.zeros_like(batch.q)
    torch.cuda.synchronize()
    vt.vt_paged_attn_release()
    run(batch, out=out)
    graph = torch.cuda.CUDAGraph()
    vt.vt_paged_attn_set_test_wait(4_000_000, 0, 1)
    with torch.cuda.graph(graph):
        run(batch, out=out, blocks=8)
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    wide = make_batch([100, 30], [900, 2000], 8, 2, 256, "bf16")
    run(wide)
    run(wide, grid=400)                    # larger again: two buffers are kept for graphs
    assert vt.vt_paged_attn_device_status() == 0
    graph.replay()
    torch.cuda.synchronize()
    words = vt.vt_paged_attn_device_status_detail()
    assert words[0] != 0 and words[1] == 1
    assert vt.vt_paged_attn_device_status() == words[0]
    assert vt.vt_paged_attn_device_status() == 0
    check(wide, run(wide))


def test_decode_counters_stay_off_a_captured_prefill(dev):
    """In a caller's area without room for both, a decode whose counters would reach a captured prefill's scratch is
    refused; what fits runs, and replays leave its counters alone."""
    batch = make_batch([100, 30], [900, 2000], 8, 2, 64, "bf16")
    need = vt.vt_paged_attn_prefill_workspace_bytes(64, vt.VT_BF16)
    room = 4096                            # of counters, beside the prefill: 1024 rows of heads
    area = torch.empty(need + room, dtype=torch.uint8, device=dev)

    def decode(seqs):
        table = batch.block_tables[1:2, :4].expand(seqs, 4).contiguous()
        lens = torch.full((seqs,), 100, dtype=torch.int32, device=dev)
        q = torch.randn((seqs, 2, 64), generator=torch.Generator().manual_seed(seqs)).to(torch.bfloat16).to(dev)
        return vt.decode(q, batch.k_cache, batch.v_cache, table, lens)

    free = decode(500)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), area.numel())
    assert area.numel() > vt.vt_paged_attn_workspace_bytes(1000, 2, 2, 64, vt.VT_BF16)
    out = torch.zeros_like(batch.q)
    run(batch, out=out)
    decode(600)                            # 1200 counters, past the prefill's start: nothing names it yet
    vt.vt_paged_attn_set_workspace(area.data_ptr(), area.numel())
    run(batch, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(batch, out=out)
    with pytest.raises(vt.VtError) as e:
        decode(1000)                       # 2000 counters: 8000 bytes
    assert e.value.status == vt.VT_ERR_SCRATCH_LIMIT
    first = decode(500)
    out.zero_()
    graph.replay()
    assert torch.equal(first, decode(500)) and torch.equal(first, free)
    check(batch, out)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), area.numel())
    decode(1000)                           # the caller's area handed over anew: no graph of before counts


#: groups of which a tile holds one token, with rows that nothing fills
@pytest.mark.parametrize("q_heads,kv_heads", [(65, 1), (100, 1), (127, 1), (256, 2)])
@pytest.mark.parametrize("dtype,D", [k for k in KINDS if k[0] != "f32"])
def test_one_token_a_tile(dev, dtype, D, q_heads, kv_heads):
    batch = make_batch([70, 0, 3, 131], [200, 5, 3, 131], q_heads, kv_heads, D, dtype, seed=q_heads, pad=2)
    out = torch.full_like(batch.q, 3.0)
    check(batch, run(batch, out=out))
    assert (out[204:] == 3).all()
    check(batch, run(batch, window=50, grid=11, blocks=2), window=50)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_scores_of_codes(dev, D):
    """Keys that grow along the context, by codes that grow: every few blocks' scores pass the maximum so far by more
    than a weight may hold, and the sums are rescaled."""
    batch = make_batch([64, 10], [1000, 800], 4, 2, D, "e4m3", seed=4)
    for b, L in enumerate(batch.ctx):
        for i in range((L + 31) // 32):
            page = batch.block_tables[b, i].long()
            k = batch.k_cache[page].view(torch.float8_e4m3fn).float()  # (NaN where nobody owns the slot stays)
            batch.k_cache[page] = (k * 2.0 ** (i // 8 - 3)).to(torch.float8_e4m3fn).view(torch.uint8)
    batch.k_scale = batch.k_scale * 8
    scale = 2 * D ** -0.5
    # the last page's scores spread by 2 * 8 standard deviations of 1, those of the first pages by 2
    grow = [(batch.q[:64, 0].double() @ k[0].T * scale).amax(0) for k in batch.dense("k")[:1]][0]
    assert grow[960:1000].max() - grow[:256].max() > 12
    check(batch, run(batch, scale=scale), scale=scale)
    check(batch, run(batch, scale=scale, grid=7, blocks=2), scale=scale)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_prefill_beside_the_decode_within_their_roundings(dev, dtype, D):
    """The same rows by the two entry points.  Each is off from the exact value by no more than its own arithmetic
    allows: prefill by the bounds above; the decode by its weights (two bf16 terms, or f16) and its result's
    rounding, with what is summed in fp32 below 2^-12 w."""
    batch = make_batch([6] * 5, [100, 37, 500, 6, 64], 8, 2, D, dtype, seed=5)
    got = run(batch).double()
    q = batch.q.view(5, 6, 8, D)
    args = (batch.block_tables, batch.context_lens)
    if dtype == "e4m3":
        dec = vt.decode_fp8(q, batch.k_cache, batch.v_cache, batch.k_scale, batch.v_scale, *args)
    else:
        dec = vt.decode_multi(q, batch.k_cache, batch.v_cache, *args)
    dec = dec.view_as(got).double()
    ref, reach, even = attention(batch, D ** -0.5, flat=True)
    if dtype == "f32":
        span = float(batch.q.double().norm(dim=-1).max()) * 1.5
        tol = 2 * ((2 * D * span + 500 + 16) * 2.0 ** -24) * reach
    else:
        own = 2.0 ** -8                    # prefill's weights
        if dtype == "e4m3":
            most = batch.q.double().abs().amax(-1, keepdim=True)
            keys = max(float(k.abs().sum(-1).max()) for k in batch.dense("k"))
            own = 2.0 ** -11 + 2 * 2.0 ** -17 * most * keys * D ** -0.5
        tol = (own + 2.0 ** -11 + 2 * 2.0 ** -12) * reach + 2 * 2.0 ** -8 * ref.abs() + 2 * 2.0 ** -25 * even
    assert ((got - dec).abs() <= tol).all(), float(((got - dec).abs() - tol).max())


@pytest.mark.parametrize("dtype,D", KINDS)
def test_no_rows_at_all(dev, dtype, D):
    """Sequences without new tokens and padding rows only: nothing is written."""
    batch = make_batch([0, 0, 0], [5, 0, 300], 4, 2, D, dtype, pad=9)
    out = torch.full_like(batch.q, 3.0)
    run(batch, out=out)
    run(batch, out=out, window=7)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0 and (out == 3).all()


def spread(batch, gaps):
    """(run arguments' q_starts, block_tables, context_lens) of the batch with gaps[i] sequences without rows in front
    of sequence i, and gaps[-1] behind the last."""
    starts, lens, rows = [0], [], []
    for b in range(len(batch.new) + 1):
        starts += [starts[-1]] * gaps[b]
        lens += [0] * gaps[b]
        rows += [0] * gaps[b]
        if b < len(batch.new):
            starts.append(starts[-1] + batch.new[b])
            lens.append(batch.ctx[b])
            rows.append(b)
    i32 = dict(dtype=torch.int32, device=batch.q.device)
    return (torch.tensor(starts, **i32), batch.block_tables[torch.tensor(rows, device=batch.q.device)].contiguous(),
            torch.tensor(lens, **i32))


@pytest.mark.parametrize("gaps", [(0, 1, 31, 32), (33, 0, 64, 700), (5, 100, 1000, 0)])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_sequences_without_rows_among_others(dev, dtype, D, gaps):
    """A padded batch: sequences without rows in front, between and behind, over any cut."""
    batch = make_batch([40, 1, 150], [500, 300, 150], 4, 2, D, dtype, seed=9)
    q_starts, table, lens = batch.q_starts, batch.block_tables, batch.context_lens
    for grid in (0, 1, 3, 17):
        batch.q_starts, batch.block_tables, batch.context_lens = spread(batch, gaps)
        out = run(batch, grid=grid, blocks=2 if grid else 0)
        batch.q_starts, batch.block_tables, batch.context_lens = q_starts, table, lens
        check(batch, out)


@pytest.mark.parametrize("dtype,D", [k for k in KINDS if k[0] != "f32"])
def test_many_sequences_without_rows(dev, dtype, D):
    """65536 of them between two with rows, and as many behind, keep nobody waiting for 5 million cycles (one after
    the other, at a memory latency each, they would)."""
    batch = make_batch([40, 30], [200, 150], 4, 2, D, dtype, seed=9)
    q_starts, table, lens = batch.q_starts, batch.block_tables, batch.context_lens
    batch.q_starts, batch.block_tables, batch.context_lens = spread(batch, (0, 65536, 65536))
    vt.vt_paged_attn_set_test_wait(5_000_000, -1, -1)
    out = run(batch, grid=1)
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    batch.q_starts, batch.block_tables, batch.context_lens = q_starts, table, lens
    check(batch, out)


@pytest.mark.parametrize("as_handle", [False, True])
def test_results_for_another_stream_are_its_own(dev, as_handle):
    """A result that the call allocates for another stream is that stream's memory: not what the current stream has
    given back and may still be reading."""
    batch = make_batch([256], [256], 8, 2, 64, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    stream = s.cuda_stream if as_handle else s
    inv, _ = vt.rope_frequencies(64)
    pos = torch.arange(256, dtype=torch.int32, device=dev)
    kv = batch.q[:, :2].contiguous()
    args = (batch.q_starts, batch.block_tables, batch.context_lens)
    calls = (lambda: vt.prefill(batch.q, batch.k_cache, batch.v_cache, *args, stream=stream),
             lambda: vt.rope(batch.q, pos, inv, stream=stream),
             lambda: vt.append(kv, kv, batch.k_cache.clone(), batch.v_cache.clone(), *args, q=batch.q, inv_freq=inv,
                               stream=stream))
    for call in calls:
        call()
        torch.cuda.synchronize()
        spare = [torch.empty_like(batch.q) for _ in range(64)]  # more than a call allocates
        given_back = {t.data_ptr() for t in spare}
        del spare
        out = call()
        s.synchronize()
        assert out.data_ptr() not in given_back
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_pages_past_two_billion_elements(dev, dtype):
    """Pages whose offset in the pool passes 32 bits: append and prefill give the bits that they give in a small pool."""
    D, Hq, Hkv, far = 128, 8, 8, 66000     # 66000 x 32 x 8 x 128 = 2.16e9 elements
    batch = make_batch([70, 1, 33], [200, 300, 33], Hq, Hkv, D, dtype, seed=6)
    qkv = torch.randn((104, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(1)).to(batch.q.dtype).to(dev)
    inv, _ = vt.rope_frequencies(D)
    scales = (batch.k_scale, batch.v_scale) if dtype == "e4m3" else ()
    small = batch.k_cache.shape[0]
    results = []
    for base in (0, far):
        pools = [torch.empty((base + small, *c.shape[1:]), dtype=c.dtype, device=dev)
                 for c in (batch.k_cache, batch.v_cache)]
        for pool, c in zip(pools, (batch.k_cache, batch.v_cache)):
            pool[base:] = c
        table = batch.block_tables + base
        args = (batch.q_starts, table, batch.context_lens)
        append, prefill = (vt.append_fp8, vt.prefill_fp8) if dtype == "e4m3" else (vt.append, vt.prefill)
        q = append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], *pools, *scales, *args, q=qkv[:, :Hq], inv_freq=inv)
        out = prefill(q, *pools, *scales, *args)
        results.append((q, out, pools[0][base:].clone(), pools[1][base:].clone()))
        del pools
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.isfinite(results[0][1]).all()


def test_rows_past_two_billion_elements(dev):
    """Half a million single tokens of 32 heads of 128: the last rows lie past 2^31 elements.  A context of one token
    gives its value, a rotation by position 0 its query."""
    T, Hq, Hkv, D = 530000, 32, 8, 128
    cache = torch.randn((2, 2, 32, Hkv, D), device=dev).to(torch.bfloat16)
    k = torch.randn((T, Hkv, D), device=dev).to(torch.bfloat16)
    q = torch.randn((T, Hq, D), device=dev).to(torch.bfloat16)
    starts = torch.arange(T + 1, dtype=torch.int32, device=dev)
    table = torch.randint(0, 2, (T, 1), dtype=torch.int32, device=dev)
    lens = torch.ones(T, dtype=torch.int32, device=dev)
    out = vt.prefill(q, cache[0], cache[1], starts, table, lens)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    first = cache[1, :, 0].repeat_interleave(Hq // Hkv, dim=1)   # [pages][Hq][D]
    for at in range(0, T, 53000):
        assert torch.equal(out[at:at + 53000], first[table[at:at + 53000, 0].long()])
    inv, _ = vt.rope_frequencies(D)
    turned = vt.rope(q, torch.zeros(T, dtype=torch.int32, device=dev), inv)
    assert torch.equal(turned, q)
    out.zero_()
    vt.append(k, k, cache[0], cache[1], starts, table, lens, q=q, q_out=out, inv_freq=inv)
    assert torch.equal(out, q)

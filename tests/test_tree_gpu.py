"""Trees of drafted tokens: masks, attention and accepted branches against
their plain forms, and a whole speculative loop (GPU).

Attention's tolerances are those of test_prefill_gpu.py, whose arithmetic this
is, with w = sum_t p_t |v_t|.  Two tiles that share rows are joined by two more
fp32 products and a sum, 2^-23 of w, within what is left of its 2^-12.
"""
from __future__ import annotations

import math
import random

import pytest
import torch

import paged_attention_decode_kv_gb300 as vt
from drafts import PAGE, any_rows, branch, pack, pages, random_parents, tree_attention, tree_rows
from ragged import E4M3_MAX, make_batch

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


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


# ------------------------------------------------------------------- masks
def starts_of(new):
    out = [0]
    for n in new:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("words,new,reach", [
    (1, [1], 1), (1, [32], 1), (1, [5, 0, 32, 7], 4), (2, [33, 1, 64], 6), (2, [26] * 64, 3), (8, [256, 200, 33], 2),
    (9, [260, 288], 1), (32, [1024, 1000, 3], 5), (32, [1024], 1), (3, [96], 1000)])
def test_masks(dev, words, new, reach):
    rng = random.Random(words)
    parents = [random_parents(n, reach, rng) for n in new]
    T = sum(new) + 4
    flat = [p for seq in parents for p in seq] + [0] * 4
    masks, positions = torch.full((T, words), -77, **I32), torch.full((T,), -5, **I32)
    ctx = [n + rng.randint(0, 900) for n in new]
    got = vt.tree_masks(torch.tensor(flat, **I32), torch.tensor(starts_of(new), **I32), torch.tensor(ctx, **I32),
                        masks=masks, positions=positions)
    assert got[0] is masks and got[1] is positions
    rows = [[branch(p, j) for j in range(n)] for p, n in zip(parents, new)]
    assert torch.equal(masks, pack(rows, words, T, fill=-77))
    want = [L - n + len(r) - 1 for n, L, seq in zip(new, ctx, rows) for r in seq]
    assert positions.tolist() == want + [-5] * 4


def test_masks_of_parents_that_are_none(dev):
    """A parent at or behind its own place, or below -1, is the context."""
    big = 2 ** 31 - 1
    parents = [0, 1, 0, 3, -2, big, -big, 2]
    masks, positions = vt.tree_masks(torch.tensor(parents, **I32), torch.tensor([0, 8], **I32),
                                     torch.tensor([20], **I32), 1)
    rows = [[[0], [1], [0, 2], [3], [4], [5], [6], [0, 2, 7]]]
    assert torch.equal(masks, pack(rows, 1, 8))
    assert positions.tolist() == [12, 12, 13, 12, 12, 12, 12, 14]


def test_masks_leave_what_is_no_tree(dev):
    """More rows than a mask has bits, fewer context tokens than rows, starts that are none."""
    for starts, ctx in (([0, 33, 35], [40, 2]), ([0, 3, 35], [2, 32]), ([-1, 3, 35], [9, 32]), ([0, 40, 35], [40, 2])):
        masks, positions = torch.full((35, 1), 9, **I32), torch.full((35,), 9, **I32)
        vt.tree_masks(torch.full((35,), -1, **I32), torch.tensor(starts, **I32), torch.tensor(ctx, **I32),
                      masks=masks, positions=positions)
        s, e, L = starts[0], starts[1], ctx[0]
        assert (masks[:max(e, 0)][:35] == 9).all() and (positions[:max(e, 0)][:35] == 9).all()
        if starts[2] > starts[1]:
            assert masks[e:, 0].tolist() == [s_ - (1 << 32) if (s_ := 1 << (i % 32)) >> 31 else s_
                                             for i in range(35 - e)]


def test_masks_allocate_and_capture(dev):
    parents, starts, ctx = torch.tensor([-1, 0, 0], **I32), torch.tensor([0, 3], **I32), torch.tensor([9], **I32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    masks, positions = vt.tree_masks(parents, starts, ctx, 2, stream=side)
    side.synchronize()
    assert masks.tolist() == [[1, 0], [3, 0], [5, 0]] and positions.tolist() == [6, 7, 7]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.tree_masks(parents, starts, ctx, masks=masks, positions=positions)
    parents.copy_(torch.tensor([-1, 0, 1], **I32))
    graph.replay()
    assert masks.tolist() == [[1, 0], [3, 0], [7, 0]] and positions.tolist() == [6, 7, 8]
    empty = torch.zeros(0, **I32)
    masks, positions = vt.tree_masks(empty, torch.zeros(1, **I32), empty, 1)
    assert masks.shape == (0, 1) and positions.shape == (0,)


def test_masks_refusals(dev):
    p, s, c = torch.tensor([-1, 0], **I32), torch.tensor([0, 2], **I32), torch.tensor([2], **I32)
    with pytest.raises(ValueError):
        vt.tree_masks(p, s, c)
    with pytest.raises(ValueError):
        vt.tree_masks(p, s, c, 2, masks=torch.zeros((2, 1), **I32))
    with pytest.raises(ValueError):
        vt.tree_masks(p, s[:1], c, 1)
    with pytest.raises(ValueError):
        vt.tree_masks(p, s, c, masks=torch.zeros((3, 1), **I32))
    with pytest.raises(TypeError):
        vt.tree_masks(p.long(), s, c, 1)
    for words in (0, 33):
        with pytest.raises(vt.VtError):
            vt.tree_masks(p, s, c, words)


# ------------------------------------------------------------------- attention
def run(batch, masks, scale=None, window=0, out=None, grid=0, blocks=0, stream=None):
    vt.vt_paged_attn_set_override(grid, blocks)
    where = (masks, batch.q_starts, batch.block_tables, batch.context_lens, scale, window)
    if batch.dtype == "e4m3":
        out = vt.prefill_tree_fp8(batch.q, batch.k_cache, batch.v_cache, batch.k_scale, batch.v_scale, *where, out=out,
                                  stream=stream)
    else:
        out = vt.prefill_tree(batch.q, batch.k_cache, batch.v_cache, *where, out=out, stream=stream)
    vt.vt_paged_attn_set_override(0, 0)
    return out


def check(batch, rows, got, scale=None, window=0, finite=True):
    live, D = batch.starts[-1], batch.q.shape[2]
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    plan = vt.vt_paged_attn_last_plan()
    assert plan["tensor_cores"] == (0 if batch.dtype == "f32" else 1)
    scale = D ** -0.5 if scale is None else scale
    ref, reach, even = (x[:live] for x in tree_attention(batch, rows, scale, window))
    got = got[:live].double()
    if finite:
        assert torch.isfinite(got).all()
    else:
        assert torch.equal(torch.isfinite(got), torch.isfinite(ref))
        keep = torch.isfinite(ref)
        ref, reach, even = (torch.where(keep, x, 0.0) for x in (ref, reach, even))
        got = torch.where(keep, got, 0.0)
    err = (got - ref).abs()
    if batch.dtype == "f32":
        n = max(batch.ctx)
        span = float(batch.q[:live].double().norm(dim=-1).max()) * 1.5 * D ** 0.5 * abs(scale)
        tol = ((2 * D * span + n + 16) * 2.0 ** -24) * reach
    else:
        tol = (2.0 ** -8 + 2.0 ** -12) * reach + 2.0 ** -8 * ref.abs() + 1e-30
        if batch.dtype == "e4m3":
            most = batch.q[:live].double().abs().amax(-1, keepdim=True)
            keys = max(float(k.nan_to_num(0.0).abs().sum(-1).max()) for k in batch.dense("k") if k.numel())
            e = 2.0 ** -17 * most * keys * abs(scale)
            tol = (2.0 ** -11 + 2.0 ** -12 + 2 * e) * reach + 2.0 ** -8 * ref.abs() + 2.0 ** -25 * even
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 512), ("f32", 64), ("f32", 128), ("f32", 256),
         ("e4m3", 64), ("e4m3", 128), ("e4m3", 256)]
#: new tokens, contexts: 4 query heads a kv head, so a tile of 128 rows is 32 tokens and an item of two 64
SHAPES = {
    "one_token": ([1], [1]),
    "first_tokens": ([2, 3, 32], [2, 3, 32]),
    "one_tile": ([1, 31, 32, 7], [33, 100, 257, 1000]),
    "two_tiles": ([33, 64, 40], [33, 64, 700]),
    "many_items": ([65, 130, 200], [65, 500, 900]),
    "empty_between": ([0, 7, 0, 0, 60, 0], [5, 7, 0, 300, 131, 64]),
    "block_edges": ([3, 3, 3, 3], [128, 129, 131, 256]),
    "long": ([26, 1, 12], [1500, 2049, 1023]),
}


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("dtype,D", KINDS)
def test_shapes(dev, dtype, D, shape, kind):
    new, ctx = SHAPES[shape]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=D)
    rows = tree_rows(new, 5, D) if kind == "tree" else any_rows(new, D)
    check(batch, rows, run(batch, pack(rows, pages(max(new)), sum(new))))


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (6, 2), (5, 1), (14, 2), (16, 2), (33, 1), (64, 1)])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("e4m3", 128)])
def test_groups(dev, dtype, D, q_heads, kv_heads):
    new, ctx = [20, 3, 41], [300, 3, 550]
    batch = make_batch(new, ctx, q_heads, kv_heads, D, dtype, seed=q_heads)
    rows = tree_rows(new, 6, q_heads)
    check(batch, rows, run(batch, pack(rows, 2, sum(new))))


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("window", [1, 2, 5, 31, 33, 128, 200, 1000])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_windows(dev, dtype, D, window, kind):
    new, ctx = [40, 1, 50, 17], [500, 300, 50, 145]
    batch = make_batch(new, ctx, 4, 2, D, dtype, seed=window)
    rows = tree_rows(new, 3, window) if kind == "tree" else any_rows(new, window)
    check(batch, rows, run(batch, pack(rows, 2, sum(new)), window=window), window=window)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("grid", [1, 2, 3, 7, 40, 152, 400])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_forced_partitions(dev, dtype, D, grid, window):
    new, ctx = [26, 70, 5, 1], [1200, 260, 900, 2000]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=1)
    rows = tree_rows(new, 4, 1)
    masks = pack(rows, 3, sum(new))
    got = run(batch, masks, window=window, grid=grid, blocks=1)
    assert vt.vt_paged_attn_last_plan()["grid_ctas"] == grid
    check(batch, rows, got, window=window)
    assert torch.equal(got, run(batch, masks, window=window, grid=grid, blocks=1))  # the same bits every time


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5, 2.0])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 128), ("e4m3", 128)])
def test_scales(dev, dtype, D, scale):
    batch = make_batch([20, 3], [250, 9], 8, 2, D, dtype, seed=3, sigma=0.5)
    rows = tree_rows(batch.new, 4, 3)
    check(batch, rows, run(batch, pack(rows, 1, 23), scale=scale), scale=scale)


@pytest.mark.parametrize("dtype,D", KINDS)
def test_rows_that_see_nothing(dev, dtype, D):
    """Without a context, an empty mask leaves nothing: 0, split into pieces or not, whatever the slots hold."""
    new, ctx = [300, 40, 5], [300, 40, 5]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=2)
    rows = [[[] if j % 3 else [j] for j in range(n)] for n in new]
    rows[2] = [[]] * 5
    masks = pack(rows, 10, sum(new))
    for grid in (0, 3, 60):
        got = run(batch, masks, grid=grid, blocks=1 if grid else 0)
        check(batch, rows, got)
        empty = torch.tensor([not r for seq in rows for r in seq])
        assert (got[empty.to(got.device)] == 0).all()


@pytest.mark.parametrize("dtype,D", KINDS)
def test_a_chain_is_a_causal_chunk(dev, dtype, D):
    new, ctx = [60, 7, 33], [500, 7, 160]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=4)
    parents = torch.tensor([j - 1 for n in new for j in range(n)], **I32)
    masks, positions = vt.tree_masks(parents, batch.q_starts, batch.context_lens, 2)
    assert positions.tolist() == [p for n, L in zip(new, ctx) for p in range(L - n, L)]
    rows = [[list(range(j + 1)) for j in range(n)] for n in new]
    for window in (0, 40):
        check(batch, rows, run(batch, masks, window=window), window=window)


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_values_that_are_not_finite_reach_only_rows_that_see_them(dev, dtype, D, value, where):
    if dtype == "e4m3" and value == value:
        pytest.skip("codes hold no infinity")
    new, ctx = [30, 70, 9], [200, 70, 400]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=5)
    rows = tree_rows(new, 4, 5)
    cache = batch.k_cache if where == "k" else batch.v_cache
    for b, i in ((0, 4), (1, 33), (2, 8)):            # drafted tokens that some rows see
        t = ctx[b] - new[b] + i
        cache[int(batch.block_tables[b, t // PAGE]), t % PAGE, 0, 3] = 0x7f if dtype == "e4m3" else value
    for grid in (0, 5):
        got = run(batch, pack(rows, 3, sum(new)), grid=grid, blocks=1 if grid else 0)
        torch.cuda.synchronize()
        hit = torch.tensor([{0: 4, 1: 33, 2: 8}[b] in r for b, seq in enumerate(rows) for r in seq], device=got.device)
        group = got.shape[1] // 2
        if where == "v":
            assert not torch.isfinite(got[hit][:, :group, 3]).any()
            others = got.clone()
            others[hit, :group, 3] = 0
            assert torch.isfinite(others).all()
        else:
            # a key of +-inf makes scores of +-inf or NaN, one of NaN scores of NaN
            if value != value:
                assert torch.isnan(got[hit][:, :group]).all()
            assert torch.isfinite(got[hit][:, group:]).all()
            assert torch.isfinite(got[~hit]).all()
        assert hit.any() and not hit.all()


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 128)])
def test_scores_of_minus_infinity(dev, dtype, D):
    """A row that sees only such scores is NaN (0 / 0), one that sees others too is made of those, and one that sees
    nothing is 0."""
    batch = make_batch([4], [4], 4, 1, D, dtype, seed=6)
    batch.q.abs_().add_(0.1)
    page = int(batch.block_tables[0, 0])
    batch.k_cache[page, 1, 0, 0] = -float("inf")
    rows = [[[0], [1], [0, 1], []]]
    for grid in (0, 1):
        got = run(batch, pack(rows, 1, 4), grid=grid)
        torch.cuda.synchronize()
        v = batch.v_cache[page, 0, 0].expand(4, D)
        assert torch.isnan(got[1]).all() and (got[3] == 0).all()
        assert torch.equal(got[0], v) and torch.equal(got[2], v)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("e4m3", 128)])
def test_values_that_are_not_finite_keep_through_weights_that_underflow(dev, dtype, D):
    """The first key's value is not finite and its weight, over 200 powers of 2 below the last key's, is 0 in 32 bits:
    the rows are not finite, in one piece or in several."""
    batch = make_batch([3], [2000], 8, 2, D, dtype, seed=8)
    batch.q.abs_().add_(0.1)
    table = batch.block_tables[0]
    batch.v_cache[int(table[0]), 0, 0, 3] = 0x7f if dtype == "e4m3" else float("inf")
    batch.k_cache[int(table[1996 // PAGE]), 1996 % PAGE] = 0x7e if dtype == "e4m3" else 8.0
    rows = [[[0], [0, 1], [0, 2]]]
    scale = 8 * D ** -0.5
    k = batch.dense("k")[0]
    scores = torch.einsum("thd,hld->thl", batch.q.double(), k.repeat_interleave(4, 0)) * scale
    assert ((scores[..., 1996] - scores[..., 0]) / math.log(2) > 200).all()
    for grid in (1, 5):
        got = run(batch, pack(rows, 1, 3), scale=scale, grid=grid, blocks=1)
        torch.cuda.synchronize()
        assert not torch.isfinite(got[:, :4, 3]).any()
        got[:, :4, 3] = 0
        assert torch.isfinite(got).all()


def test_bits_past_the_rows_are_not_looked_at(dev):
    batch = make_batch([5, 30], [150, 31], 8, 2, 128, "bf16", seed=7)
    rows = tree_rows(batch.new, 3, 7)
    masks = pack(rows, 3, 35)
    want = run(batch, masks)
    dirty = masks.clone()
    dirty[:, 1:] = -1
    dirty[:5, 0] |= ~31
    dirty[5:, 0] |= -(1 << 30)
    assert torch.equal(want, run(batch, dirty))
    window = run(batch, masks, window=40)
    assert torch.equal(window, run(batch, dirty, window=40))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 64), ("e4m3", 128)])
def test_invalid_device_data(dev, dtype, D):
    new, ctx = [3, 33, 4, 5], [100, 90, 200, 64]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=8, pad=2)
    rows = [[[j] for j in range(n)] for n in new]
    rows[1] = [[0]] * 33
    masks = pack(rows, 1, sum(new) + 2)
    batch.block_tables[2, 3] = -1       # tokens 96 .. 127 of it
    out = torch.full_like(batch.q, 5.0)
    got = run(batch, masks, out=out)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    assert torch.isfinite(got[:3]).all()
    assert torch.isnan(got[3:36]).all()     # more rows than bits
    assert torch.isnan(got[36:40]).all()    # a page out of range
    assert torch.isfinite(got[40:45]).all()
    assert (got[45:] == 5).all()            # padding
    batch.context_lens[0] = 2               # fewer than its rows
    got = run(batch, masks)
    torch.cuda.synchronize()
    assert torch.isnan(got[:3]).all() and torch.isfinite(got[40:45]).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 512), ("f32", 128), ("e4m3", 64)])
def test_captured_on_a_stream(dev, dtype, D):
    batch = make_batch([20, 50], [700, 300], 8, 2, D, dtype, seed=9)
    rows = tree_rows(batch.new, 4, 9)
    masks = pack(rows, 2, 70)
    want = run(batch, masks)
    out, side = torch.zeros_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(batch, masks, out=out)
    others = tree_rows(batch.new, 9, 10)
    masks.copy_(pack(others, 2, 70))
    graph.replay()
    torch.cuda.synchronize()
    check(batch, others, out)
    side.wait_stream(torch.cuda.current_stream())
    got = run(batch, masks, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


def test_callers_workspace(dev):
    batch = make_batch([20, 50], [700, 900], 8, 2, 128, "bf16", seed=11)
    rows = tree_rows(batch.new, 4, 11)
    masks = pack(rows, 2, 70)
    want = run(batch, masks)
    n = vt.vt_paged_attn_prefill_workspace_bytes(128, vt.VT_BF16)
    area = torch.empty(n + 4096, dtype=torch.uint8, device=dev)
    vt.vt_paged_attn_set_workspace(area.data_ptr(), area.numel())
    assert torch.equal(run(batch, masks), want)
    assert vt.vt_paged_attn_last_plan()["scratch_source"] == 1
    vt.vt_paged_attn_set_workspace(area.data_ptr(), n // 2)
    with pytest.raises(vt.VtError):
        run(batch, masks)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (256, "bf16"), (128, "e4m3")])
def test_bounded_wait_gives_up_and_reports(dev, D, dtype):
    batch = make_batch([20, 50], [700, 900], 8, 2, D, dtype, seed=12)
    rows = tree_rows(batch.new, 4, 12)
    masks = pack(rows, 2, 70)
    run(batch, masks)
    torch.cuda.synchronize()
    vt.vt_paged_attn_set_test_wait(2000000, 0, 1)
    run(batch, masks, grid=2, blocks=1)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() != 0
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    check(batch, rows, run(batch, masks))


def test_prefill_tree_refusals(dev):
    batch = make_batch([3], [40], 4, 2, 64, "bf16")
    masks = torch.zeros((3, 1), **I32)
    for bad, error in ((masks[:2], ValueError), (masks.long(), TypeError), (masks.flatten(), ValueError),
                       (masks.cpu(), ValueError), (torch.zeros((3, 2), **I32)[:, ::2], ValueError)):
        with pytest.raises(error):
            run(batch, bad)
    for words in (0, 33):
        with pytest.raises(vt.VtError):
            run(batch, torch.zeros((3, words), **I32))


def test_pages_past_2_31_elements(dev):
    """A pool of more than 2^31 elements, its far pages in use."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs memory")
    pool = (1 << 31) // (PAGE * 2 * 128) + 50
    small = make_batch([12, 40], [90, 333], 8, 2, 128, "bf16", seed=13)
    used = small.k_cache.shape[0]
    k, v = (torch.zeros((pool, PAGE, 2, 128), dtype=torch.bfloat16, device=dev) for _ in range(2))
    k[-used:], v[-used:] = small.k_cache, small.v_cache
    small.k_cache, small.v_cache = k, v
    small.block_tables += pool - used
    rows = tree_rows(small.new, 4, 13)
    masks = pack(rows, 2, 52)
    check(small, rows, run(small, masks))
    accepted = torch.tensor([11, 39], **I32)
    was = {}
    for b, j in enumerate((11, 39)):
        base = small.ctx[b] - small.new[b]
        for r, i in enumerate(rows[b][j]):
            was[b, base + r] = cell(k, small, b, base + i).clone()
    kept = vt.keep_path(accepted, masks, k, v, small.q_starts, small.block_tables, small.context_lens)
    assert kept.tolist() == [L - n + len(r[j]) for L, n, r, j in zip(small.ctx, small.new, rows, (11, 39))]
    for (b, t), x in was.items():
        assert torch.equal(cell(k, small, b, t), x)


# ------------------------------------------------------------------- accepted branches
def cell(cache, batch, b, t):
    return cache[int(batch.block_tables[b, t // PAGE]), t % PAGE]


def kept_by_hand(batch, rows, accepted, caches):
    """Expected caches (copies) and lengths, token by token."""
    out = [c.clone() for c in caches]
    kept = []
    for b, (n, L) in enumerate(zip(batch.new, batch.ctx)):
        j, base = accepted[b], L - n
        path = [i for i in rows[b][j] if i < n] if 0 <= j < n else []
        kept.append(base + len(path) if n else L)
        for c, was in zip(out, caches):
            for r, i in enumerate(path):
                cell(c, batch, b, base + r).copy_(cell(was, batch, b, base + i))
    return kept, out


@pytest.mark.parametrize("dtype,heads,D", [("bf16", 8, 128), ("bf16", 1, 64), ("f32", 2, 256), ("e4m3", 4, 128),
                                           ("e4m3", 1, 64), ("bf16", 3, 512)])
def test_keep_path(dev, dtype, heads, D):
    new, ctx = [40, 1, 0, 64, 33, 7], [40, 100, 9, 300, 95, 33]
    batch = make_batch(new, ctx, heads, heads, D, dtype, seed=D)
    rows = tree_rows(new, 7, D)
    masks = pack(rows, 2, sum(new))
    rng = random.Random(D)
    # a branch's end, all of a long chain, none, out of range
    for accepted in ([39, 0, -1, 63, 32, 6], [rng.randint(-1, max(0, n - 1)) for n in new], [-1] * 6,
                     [40, 5, 0, 2 ** 31 - 1, -9, 3]):
        k, v = batch.k_cache.clone(), batch.v_cache.clone()
        want, (wk, wv) = kept_by_hand(batch, rows, accepted, (k, v))
        got = vt.keep_path(torch.tensor(accepted, **I32), masks, k, v, batch.q_starts, batch.block_tables,
                           batch.context_lens)
        assert got.tolist() == want
        for x, y in ((k, wk), (v, wv)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_keep_path_of_masks_that_are_no_trees(dev):
    """Long branches with every gap, moved over each other, and 1024 bits."""
    new, ctx = [1024, 500, 64], [1100, 500, 65]
    batch = make_batch(new, ctx, 2, 2, 64, "bf16", seed=3)
    rng = random.Random(3)
    rows = [[sorted(rng.sample(range(n), rng.randint(n // 2, n))) for _ in range(n)] for n in new]
    rows[2][5] = list(range(1, 64))
    masks = pack(rows, 32, sum(new))
    accepted = [1023, 17, 5]
    k, v = batch.k_cache.clone(), batch.v_cache.clone()
    want, (wk, wv) = kept_by_hand(batch, rows, accepted, (k, v))
    got = vt.keep_path(torch.tensor(accepted, **I32), masks, k, v, batch.q_starts, batch.block_tables,
                       batch.context_lens)
    assert got.tolist() == want
    assert torch.equal(k.view(torch.uint8), wk.view(torch.uint8))
    assert torch.equal(v.view(torch.uint8), wv.view(torch.uint8))


@pytest.mark.parametrize("layout", ["apart", "together", "none"])
def test_keep_path_of_all_layers(dev, layout):
    new, ctx, layers = [20, 33], [50, 200], 5
    batch = make_batch(new, ctx, 2, 2, 64, "f32", seed=4)
    rows = tree_rows(new, 6, 4)
    masks = pack(rows, 2, sum(new))
    g = torch.Generator(device=dev).manual_seed(4)
    shape = batch.k_cache.shape
    pool = torch.randn((layers, 2, *shape), generator=g, device=dev)
    k, v = (pool[:, 0], pool[:, 1]) if layout == "together" else (pool[:, 0].contiguous(), pool[:, 1].contiguous())
    if layout == "none":
        k, v = k[:0], v[:0]
    expected = [kept_by_hand(batch, rows, [19, 32], (k[i].clone(), v[i].clone()))[1] for i in range(len(k))]
    kept = torch.zeros(2, **I32)
    got = vt.keep_path(torch.tensor([19, 32], **I32), masks, k, v, batch.q_starts, batch.block_tables,
                       batch.context_lens, kept_lens=kept)
    assert got is kept and kept.tolist() == [30 + len(rows[0][19]), 167 + len(rows[1][32])]
    for i, (wk, wv) in enumerate(expected):
        assert torch.equal(k[i], wk) and torch.equal(v[i], wv)


def test_keep_path_invalid_device_data(dev):
    new, ctx = [10, 40, 8, 6], [100, 60, 70, 40]
    batch = make_batch(new, ctx, 2, 2, 64, "bf16", seed=5)
    rows = [[[j] for j in range(n)] for n in new]
    masks = pack([r[:] if len(r) <= 32 else [[0]] * len(r) for r in rows], 1, sum(new))
    batch.context_lens[0] = 5                    # fewer than its rows
    batch.block_tables[2, 2] = 10 ** 6           # tokens 64 .. 69 of 62 .. 69
    k, v = batch.k_cache.clone(), batch.v_cache.clone()
    got = vt.keep_path(torch.tensor([9, 39, 7, 5], **I32), masks, k, v, batch.q_starts, batch.block_tables,
                       batch.context_lens)
    assert got.tolist() == [5, 60, 63, 35]       # the second has more rows than bits
    want = batch.k_cache.clone()
    cell(want, batch, 3, 34).copy_(cell(want, batch, 3, 39))
    assert torch.equal(k.view(torch.int16), want.view(torch.int16))


def test_keep_path_captured_and_refusals(dev):
    batch = make_batch([6], [40], 2, 2, 64, "bf16", seed=6)
    rows = tree_rows([6], 3, 6)
    masks = pack(rows, 1, 6)
    accepted = torch.tensor([-1], **I32)
    k, v, kept = batch.k_cache, batch.v_cache, torch.zeros(1, **I32)
    where = (batch.q_starts, batch.block_tables, batch.context_lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.keep_path(accepted, masks, k, v, *where, kept_lens=kept)
    want, (wk, wv) = kept_by_hand(batch, rows, [5], (k, v))
    accepted.fill_(5)
    graph.replay()
    assert kept.tolist() == want and torch.equal(k.view(torch.int16), wk.view(torch.int16))
    side = torch.cuda.Stream()
    accepted.fill_(-1)
    side.wait_stream(torch.cuda.current_stream())
    got = vt.keep_path(accepted, masks, k, v, *where, stream=side)
    side.synchronize()
    assert got.tolist() == [34]
    with pytest.raises(vt.VtError):
        vt.keep_path(accepted, masks, k, v, *where, kept_lens=batch.context_lens)
    with pytest.raises(ValueError):
        vt.keep_path(accepted, masks, k, v[:1], *where)
    with pytest.raises(ValueError):
        vt.keep_path(accepted, masks, k.transpose(1, 2), v.transpose(1, 2), *where)
    with pytest.raises(TypeError):
        vt.keep_path(accepted, masks, k.half(), v.half(), *where)
    with pytest.raises(TypeError):
        vt.keep_path(accepted, masks, k, v.float(), *where)
    with pytest.raises(ValueError):
        vt.keep_path(accepted[:0], masks, k, v, *where)
    with pytest.raises(vt.VtError):
        vt.keep_path(accepted, torch.zeros((6, 33), **I32), k, v, *where)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,window", [("bf16", 0), ("f32", 0), ("e4m3", 0), ("f32", 20)])
def test_a_speculative_loop(dev, dtype, window):
    """Prompts, then rounds of drafted trees of which a branch is accepted: page tables, masks, normed append, tree
    attention and kept branches, one after the other on the GPU.  In the end the cache holds what an append of the
    accepted tokens in order puts there, and a decode step over it answers as a plain one over those tokens."""
    B, Hq, Hkv, D, room, pool = 5, 8, 2, 64, 8, 48
    rng = random.Random(1)
    g = torch.Generator(device=dev).manual_seed(1)
    io = torch.float32 if dtype == "f32" else torch.bfloat16
    kv = torch.uint8 if dtype == "e4m3" else io
    inv, _ = vt.rope_frequencies(D)
    qw, kw = (1 + 0.3 * torch.randn(D, generator=g, device=dev) for _ in range(2))
    scales = [torch.full((Hkv,), 0.02, device=dev) for _ in range(2)]

    def fresh():
        return [torch.zeros((pool, PAGE, Hkv, D), dtype=kv, device=dev) for _ in range(2)]

    def append(x, cache, starts, tables, lens, positions):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        args = dict(q=q, q_weight=qw, inv_freq=inv, positions=positions)
        if dtype == "e4m3":
            return vt.norm_append_fp8(k, v, kw, *cache, *scales, starts, tables, lens, **args)
        return vt.norm_append(k, v, kw, *cache, starts, tables, lens, **args)

    cache = fresh()
    tables, lens = torch.zeros((B, room), **I32), torch.zeros(B, **I32)
    free, counters = torch.randperm(pool, generator=g, device=dev).to(torch.int32), torch.tensor([pool, 0], **I32)
    token_rows = [[] for _ in range(B)]       # the accepted tokens' projections, in order
    kept = None
    for round_ in range(4):
        new = [rng.randint(1, 60) if round_ == 0 else rng.choice([0, 1, rng.randint(2, 30)]) for _ in range(B)]
        T = sum(new) + 3
        starts, positions, _ = vt.step_tables(lens, torch.tensor(new, **I32), tables, free, counters, T, keep_lens=kept)
        assert counters[1].item() == 0
        x = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=dev).to(io)
        parents = [[j - 1 for j in range(n)] if round_ == 0 else random_parents(n, 4, rng) for n in new]
        flat = torch.tensor([p for seq in parents for p in seq] + [0] * 3, **I32)
        masks, positions = vt.tree_masks(flat, starts, lens, 2, positions=positions)
        q = append(x, cache, starts, tables, lens, positions)
        where = (masks, starts, tables, lens, None, window)
        out = vt.prefill_tree_fp8(q, *cache, *scales, *where) if dtype == "e4m3" else vt.prefill_tree(q, *cache, *where)
        assert torch.isfinite(out[:sum(new)]).all()
        last = [n - 1 if round_ == 0 else rng.randint(-1, n - 1) if n else -1 for n in new]
        at = 0
        for b, n in enumerate(new):
            path = branch(parents[b], last[b]) if last[b] >= 0 else []
            token_rows[b] += [x[at + i] for i in path]
            # what the last accepted token's row answered: plain attention over the accepted tokens
            if path:
                check_row(out[at + path[-1]], q[at + path[-1]], token_rows[b], kw, inv, dtype, scales, window)
            at += n
        kept = vt.keep_path(torch.tensor(last, **I32), masks, *cache, starts, tables, lens)
        assert kept.tolist() == [len(r) for r in token_rows]
    # the accepted tokens appended in order, into pages of their own
    vt.step_tables(lens, torch.zeros(B, **I32), tables, free, counters, 0, keep_lens=kept)
    assert counters[0].item() == pool - sum(pages(len(r)) for r in token_rows)
    plain, starts = fresh(), torch.tensor(starts_of([len(r) for r in token_rows]), **I32)
    append(torch.stack([r for seq in token_rows for r in seq]), plain, starts, tables, lens, None)
    for b, r in enumerate(token_rows):
        for t in range(len(r)):
            page = int(tables[b, t // PAGE])
            for x, y in zip(cache, plain):
                assert torch.equal(x[page, t % PAGE], y[page, t % PAGE])


def check_row(out, q, token_rows, kw, inv, dtype, scales, window):
    """out [Hq][D] of rotated query q over the tokens' projections, in 64 bits but for the cache's rounding."""
    Hq, D = q.shape
    Hkv = scales[0].numel()
    x = torch.stack(token_rows).double()
    k, v = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    k = k / torch.sqrt((k * k).mean(-1, keepdim=True) + 1e-6) * kw.double()
    angle = torch.arange(len(token_rows), device=q.device).double()[:, None] * inv
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    a, b = k[..., :D // 2], k[..., D // 2:]
    k = torch.cat([a * c - b * s, b * c + a * s], -1)
    if dtype == "e4m3":
        k, v = ((y / 0.02).clamp(-E4M3_MAX, E4M3_MAX) for y in (k, v))
        k, v = (y.float().to(torch.float8_e4m3fn).double() * sc.double()[:, None] for y, sc in zip((k, v), scales))
    elif dtype == "bf16":
        k = k.to(torch.bfloat16).double()
    if window:
        k, v = k[-window:], v[-window:]
    group = Hq // Hkv
    for h in range(Hq):
        p = torch.softmax(k[:, h // group] @ q[h].double() * D ** -0.5, 0)
        reach = p @ v[:, h // group].abs()
        # (a key's own rounding may fall to the other side of a tie: one more step of it, 2^-7 or 2^-3 of a term of
        # the score, shows as a part of the weights no larger than this)
        slack = {"f32": 2.0 ** -14, "bf16": 2.0 ** -6, "e4m3": 2.0 ** -4}[dtype]
        assert ((out[h].double() - p @ v[:, h // group]).abs() <= slack * (reach + reach.mean())).all()


# ------------------------------------------------------------------- what calls meet
def test_codes_under_either_name(dev):
    """E4M3 codes as uint8, as float8_e4m3fn, or one of each."""
    batch = make_batch([9, 40], [200, 60], 8, 2, 128, "e4m3", seed=20)
    rows = tree_rows(batch.new, 3, 20)
    masks = pack(rows, 2, 49)
    want = run(batch, masks)
    k8, v8 = batch.k_cache.view(torch.float8_e4m3fn), batch.v_cache.view(torch.float8_e4m3fn)
    where = (masks, batch.q_starts, batch.block_tables, batch.context_lens)
    for k, v in ((k8, v8), (k8, batch.v_cache), (batch.k_cache, v8)):
        assert torch.equal(vt.prefill_tree_fp8(batch.q, k, v, batch.k_scale, batch.v_scale, *where), want)
        was = batch.k_cache.clone()
        kept = vt.keep_path(torch.tensor([0, 0], **I32), masks, k, v, *where[1:])
        assert kept.tolist() == [192, 21] and torch.equal(was, batch.k_cache)
    with pytest.raises(TypeError):
        vt.prefill_tree_fp8(batch.q, k8, batch.v_cache.view(torch.int8), batch.k_scale, batch.v_scale, *where)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 256), ("f32", 64), ("e4m3", 128)])
@pytest.mark.parametrize("window", [7, 40])
def test_windows_pass_over_what_is_not_finite(dev, dtype, D, window):
    """NaN before a row's window, drafted or not, is not its."""
    new, ctx = [20, 20], [300, 45]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=21)
    rows = [[list(range(j + 1)) for j in range(n)] for n in new]
    spots = [(0, ctx[0] - new[0] - window + 2), (1, ctx[1] - new[1] + 1)]  # seen by a chain's first rows only
    for b, t in spots:
        batch.v_cache[int(batch.block_tables[b, t // PAGE]), t % PAGE, 1, 5] = 0x7f if dtype == "e4m3" else float("nan")
    for grid in (0, 3):
        got = run(batch, pack(rows, 1, 40), window=window, grid=grid, blocks=1 if grid else 0)
        torch.cuda.synchronize()
        for b, t in spots:
            base = ctx[b] - new[b]
            for j in range(new[b]):
                seen = (list(range(base)) + [base + i for i in range(j + 1)])[-window:]
                bad = torch.isnan(got[b * 20 + j])
                assert bool(bad[4:, 5].all()) == (t in seen), (b, j)
                bad[4:, 5] = False
                assert not bad.any()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_starts_and_contexts_that_are_none(dev, dtype, D):
    """Row starts that decrease, are below 0 or pass the rows are sequences without rows; contexts past the table NaN."""
    batch = make_batch([4, 5, 6], [40, 70, 64], 8, 2, D, dtype, seed=22, pad=1)
    rows = [[[j] for j in range(n)] for n in batch.new]
    masks = pack(rows, 1, 16)
    out = torch.full_like(batch.q, 3.0)
    for starts in ([0, 4, 9, 40], [-5, 4, 9, 15], [0, 9, 4, 15], [15, 9, 4, 0]):
        q_starts = torch.tensor(starts, **I32)
        vt.prefill_tree(batch.q, batch.k_cache, batch.v_cache, masks, q_starts, batch.block_tables,
                        batch.context_lens, out=out)
        kept = vt.keep_path(torch.zeros(3, **I32), masks, batch.k_cache.clone(), batch.v_cache.clone(), q_starts,
                            batch.block_tables, batch.context_lens)
        assert [k for k, s, e in zip(kept.tolist(), starts, starts[1:]) if not (0 <= s < e <= 16)] == \
            [L for L, s, e in zip(batch.ctx, starts, starts[1:]) if not (0 <= s < e <= 16)]
    assert vt.vt_paged_attn_device_status() == 0
    lens = torch.tensor([40, 10 ** 9, -3], **I32)
    got = vt.prefill_tree(batch.q, batch.k_cache, batch.v_cache, masks, batch.q_starts, batch.block_tables, lens)
    assert torch.isfinite(got[:4]).all() and torch.isnan(got[4:15]).all()
    kept = vt.keep_path(torch.zeros(3, **I32), masks, batch.k_cache.clone(), batch.v_cache.clone(), batch.q_starts,
                        batch.block_tables, lens)
    assert kept.tolist() == [37, 10 ** 9, -3]


def test_batches_without_rows(dev):
    batch = make_batch([0, 0], [40, 33], 4, 2, 64, "bf16")
    masks = torch.zeros((0, 2), **I32)
    assert run(batch, masks).shape == (0, 4, 64)
    k, v = batch.k_cache.clone(), batch.v_cache.clone()
    kept = vt.keep_path(torch.tensor([0, -1], **I32), masks, k, v, batch.q_starts, batch.block_tables,
                        batch.context_lens)
    assert kept.tolist() == [40, 33] and torch.equal(k.view(torch.int16), batch.k_cache.view(torch.int16))
    empty = torch.zeros(0, **I32)
    kept = vt.keep_path(empty, masks, k, v, torch.zeros(1, **I32), torch.zeros((0, 3), **I32), empty)
    assert kept.shape == (0,)


def test_calls_at_once_on_two_streams(dev):
    """Operators without a workspace run side by side."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    new, ctx = [30, 64, 5], [500, 900, 64]
    states = []
    for i in range(2):
        batch = make_batch(new, ctx, 2, 2, 128, "bf16", seed=30 + i)
        parents = [random_parents(n, 5, random.Random(i)) for n in new]
        flat = torch.tensor([p for seq in parents for p in seq], **I32)
        states.append((batch, parents, flat, torch.zeros((99, 2), **I32), torch.zeros(99, **I32)))
    torch.cuda.synchronize()
    kept = []
    for _ in range(5):
        for s, (batch, parents, flat, masks, positions) in zip(sides, states):
            vt.tree_masks(flat, batch.q_starts, batch.context_lens, masks=masks, positions=positions, stream=s)
    for s, (batch, parents, flat, masks, positions) in zip(sides, states):
        with torch.cuda.stream(s):
            k, v, took = batch.k_cache.clone(), batch.v_cache.clone(), torch.tensor([29, 63, 4], **I32)
            kept.append((k, v, vt.keep_path(took, masks, k, v, batch.q_starts, batch.block_tables, batch.context_lens)))
    torch.cuda.synchronize()
    for (batch, parents, flat, masks, positions), (k, v, lens) in zip(states, kept):
        rows = [[branch(p, j) for j in range(n)] for p, n in zip(parents, new)]
        assert torch.equal(masks, pack(rows, 2, 99))
        want, (wk, wv) = kept_by_hand(batch, rows, [29, 63, 4], (batch.k_cache, batch.v_cache))
        assert lens.tolist() == want
        assert torch.equal(k.view(torch.int16), wk.view(torch.int16))
        assert torch.equal(v.view(torch.int16), wv.view(torch.int16))


FIRST = """
import torch, paged_attention_decode_kv_gb300 as vt
i32 = dict(dtype=torch.int32, device="cuda")
lens, new = torch.tensor([5, 0], **i32), torch.tensor([3, 40], **i32)
tables, free, counters = torch.tensor([[4, 0], [0, 0]], **i32), torch.arange(5, **i32), torch.tensor([4, 0], **i32)
parents, starts = torch.tensor([j - 1 for n in (3, 40) for j in range(n)], **i32), torch.tensor([0, 3, 43], **i32)
masks = torch.zeros((43, 32), **i32)
k, v = torch.zeros((2, 5, 32, 2, 64), dtype=torch.bfloat16, device="cuda").unbind()
x = torch.ones((43, 2, 64), dtype=torch.bfloat16, device="cuda")
w = torch.ones(64, device="cuda")
inv, _ = vt.rope_frequencies(64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q_starts, positions, slots = vt.step_tables(lens, new, tables, free, counters, 43)
    vt.tree_masks(parents, q_starts, lens, masks=masks, positions=positions)
    q = vt.norm_append(x, x, w, k, v, q_starts, tables, lens, q=x, q_weight=w, positions=positions, inv_freq=inv)
    kept = vt.keep_path(starts[:2], masks, k, v, q_starts, tables, lens)
    try:
        vt.prefill_tree(q, k, v, masks, q_starts, tables, lens)
        raise SystemExit("a first prefill inside a capture allocates")
    except vt.VtError as e:
        assert e.status == vt.VT_ERR_SCRATCH_LIMIT, e
g.replay()
torch.cuda.synchronize()
assert lens.tolist() == [8, 40] and q_starts.tolist() == [0, 3, 43], (lens, q_starts)
assert positions.tolist() == [5, 6, 7, *range(40)]
assert slots.tolist() == [4 * 32 + 5, 4 * 32 + 6, 4 * 32 + 7] + [3 * 32 + i for i in range(32)] + [2 * 32 + i for i in range(8)]
assert masks[42, 0].item() == -1 and masks[42, 1].item() == 255
assert kept.tolist() == [6, 4], kept
assert torch.isfinite(q).all() and (v[4, 5:8] == 1).all() and (v[3] == 1).all()
print("fine")
"""


def test_first_calls_of_a_process_inside_a_capture(dev):
    """Nothing of the step but the attention allocates, so it can be captured at once; the attention refuses."""
    import subprocess
    import sys
    from pathlib import Path
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=Path(__file__).resolve().parents[1], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr


@pytest.mark.parametrize("dtype,D", KINDS)
def test_many_items_of_both_kinds(dev, dtype, D):
    """Trees of one tile and of two in one batch, in shares that cut them anywhere."""
    rng = random.Random(D)
    new = [rng.randint(1, 64) for _ in range(40)]
    ctx = [n + rng.randint(0, 700) for n in new]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=D)
    rows = tree_rows(new, 4, D)
    masks = pack(rows, 2, sum(new))
    for grid in (0, 11, 97):
        check(batch, rows, run(batch, masks, grid=grid, blocks=1 if grid else 0))


# ------------------------------------------------------------------- values that are not finite, by how work is cut
def not_finite(dtype, value):
    return 0x7f if dtype == "e4m3" else value


@pytest.mark.parametrize("dtype,D", KINDS)
def test_weights_that_underflow_between_pieces_keep_what_is_not_finite(dev, dtype, D):
    """As the test of weights that underflow, with the pieces of every type joined: what a row sees and is not finite
    is so in the result, however the work was cut."""
    batch = make_batch([3], [2000], 8, 2, D, dtype, seed=8)
    batch.q.abs_().add_(0.1)
    table = batch.block_tables[0]
    batch.v_cache[int(table[0]), 0, 0, 3] = not_finite(dtype, float("inf"))
    batch.k_cache[int(table[1990 // PAGE]), 1990 % PAGE] = 0x7e if dtype == "e4m3" else 8.0
    scale = 8 * D ** -0.5
    k = batch.dense("k")[0]
    scores = torch.einsum("thd,hld->thl", batch.q.double(), k.repeat_interleave(4, 0)) * scale
    assert ((scores[..., 1990] - scores[..., 0]) / math.log(2) > 200).all()
    for grid in (1, 2, 5, 16):
        got = run(batch, pack([[[0], [0, 1], [0, 2]]], 1, 3), scale=scale, grid=grid, blocks=1)
        torch.cuda.synchronize()
        assert not torch.isfinite(got[:, :4, 3]).any()
        got[:, :4, 3] = 0
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_weights_that_underflow_within_a_block_keep_what_is_not_finite(dev, dtype, D, window):
    """Among keys that only some rows see, a value that is not finite and whose weight is 0 in 32 bits: the rows that
    see it are not finite, the others are."""
    new, L = 20, 100
    batch = make_batch([new], [L], 8, 2, D, dtype, seed=9)
    batch.q.abs_().add_(0.1)
    rows = [[0], [0, 1], [0, 2], [3]] + [list(range(4, j + 1)) for j in range(4, new)]
    table = batch.block_tables[0]
    base = L - new
    spots = [(base, 3), (base + 6, 7)] + ([(45, 5)] if window else [])
    for t, col in spots:
        batch.v_cache[int(table[t // PAGE]), t % PAGE, 0, col] = not_finite(dtype, float("inf"))
    batch.k_cache[int(table[60 // PAGE]), 60 % PAGE] = 0x7e if dtype == "e4m3" else 8.0   # which every row sees
    scale = 8 * D ** -0.5
    k = batch.dense("k")[0]
    scores = torch.einsum("thd,hld->thl", batch.q.double(), k.repeat_interleave(4, 0)) * scale
    for t, _ in spots:
        assert ((scores[..., 60] - scores[..., t]) / math.log(2) > 200).all()
    seen = [(list(range(base)) + [base + i for i in r])[-window:] for r in rows]
    got = run(batch, pack([rows], 1, new), scale=scale, window=window)
    torch.cuda.synchronize()
    for t, col in spots:
        sees = torch.tensor([t in s for s in seen], device=got.device)
        assert sees.any() and not sees.all()
        assert not torch.isfinite(got[sees][:, :4, col]).any()
        got[sees, :4, col] = 0
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("grid", [0, 1, 2, 5])
@pytest.mark.parametrize("dtype,D", [k for k in KINDS if k[0] != "e4m3"])
def test_infinities_keep_their_sign(dev, dtype, D, grid, window):
    """Infinite values are infinities of their sign in the rows that see them, NaN where a row sees both signs, and
    nothing elsewhere: with items of one tile and of two, rows that see keys in one of two blocks only, and an
    infinity every row sees."""
    new, ctx = [20, 50, 9, 33], [130, 140, 400, 33]
    batch = make_batch(new, ctx, 8, 2, D, dtype, seed=14)
    rows = tree_rows(new, 4, 14)
    inf = float("inf")
    for b, t, col, value in ((0, 114, 3, inf), (0, 114, 4, -inf), (0, 112, 5, inf), (0, 129, 5, -inf), (0, 5, 6, -inf),
                             (0, 108, 7, inf), (0, 109, 7, -inf), (1, 100, 3, inf), (1, 138, 4, inf), (1, 91, 5, -inf), (2, 100, 3, inf),
                             (2, 395, 4, -inf), (2, 398, 5, inf), (3, 4, 3, inf), (3, 4, 4, -inf),
                             (3, 32, 5, -inf)):
        batch.v_cache[int(batch.block_tables[b, t // PAGE]), t % PAGE, 0, col] = value
    got = run(batch, pack(rows, 2, sum(new)), window=window, grid=grid, blocks=1 if grid else 0)
    check(batch, rows, got, window=window, finite=False)
    ref = tree_attention(batch, rows, D ** -0.5, window)[0]
    some = ~torch.isfinite(ref)
    assert torch.equal(got[some].double().nan_to_num(7.0), ref[some].nan_to_num(7.0))
    for what in (ref == inf, ref == -inf, torch.isnan(ref)):
        assert what.any()


@pytest.mark.parametrize("window", [0, 200, 1100])
@pytest.mark.parametrize("dtype,D", [k for k in KINDS if k[0] != "f32"])
def test_a_large_tree_of_values_that_are_not_finite(dev, dtype, D, window):
    """What they cost is a look at each new token's values an item, whatever the number of those that are not finite:
    no wait takes more than 8 million cycles."""
    new, L = 1024, 1400
    batch = make_batch([new], [L], 4, 2, D, dtype, seed=15)
    rows = tree_rows([new], 3, 15)
    rows[0] = [r if j % 5 else [] for j, r in enumerate(rows[0])]   # rows that see the context alone
    base = L - new
    spots = torch.arange(base if not window else base - 100, L, device=dev)
    pages_, at = batch.block_tables[0, spots // PAGE].long(), spots % PAGE
    batch.v_cache[pages_, at] = not_finite(dtype, float("nan"))
    vt.vt_paged_attn_set_test_wait(8_000_000, -1, -1)
    got = run(batch, pack(rows, 32, new), window=window, grid=4, blocks=8)
    vt.vt_paged_attn_set_test_wait(0, -1, -1)
    torch.cuda.synchronize()
    assert vt.vt_paged_attn_device_status() == 0
    first = int(spots[0])
    hit = torch.tensor([max((list(range(base)) + [base + i for i in r])[-window:]) >= first for r in rows[0]], device=dev)
    assert hit.any()
    assert torch.isnan(got[hit]).all() and torch.isfinite(got[~hit]).all()
    if not window:
        assert not hit.all()


@pytest.mark.parametrize("dtype,D", KINDS)
def test_the_workspace_asked_for_holds_a_call(dev, dtype, D):
    """Of trees and of causal chunks, beside what was asked for and not a byte behind it."""
    batch = make_batch([20, 50], [700, 900], 8, 2, D, dtype, seed=16)
    rows = tree_rows(batch.new, 4, 16)
    masks = pack(rows, 2, 70)
    n = vt.vt_paged_attn_prefill_workspace_bytes(D, {"bf16": vt.VT_BF16, "f32": vt.VT_F32, "e4m3": vt.VT_E4M3}[dtype])
    area = torch.full((n + 4096,), 7, dtype=torch.uint8, device=dev)
    area[:n] = 0
    vt.vt_paged_attn_set_workspace(area.data_ptr(), n)
    check(batch, rows, run(batch, masks))
    plan = vt.vt_paged_attn_last_plan()
    assert plan["scratch_source"] == 1 and plan["workspace_bytes"] <= n
    assert (area[n:] == 7).all()


@pytest.mark.parametrize("group", [24, 7, 127, 4])
@pytest.mark.parametrize("dtype,D", KINDS)
def test_a_row_depends_on_its_own_sequence_alone(dev, dtype, D, group):
    """To the bit: not on what an earlier call left in shared memory where groups do not fill a tile's 128 rows, nor on
    other sequences' queries, nor on what lies in rows behind the last one."""
    if dtype == "f32" and group > 64:
        pytest.skip("fp32 has 64 rows")
    new, ctx = [3, 9, 2], [2500, 1800, 900]
    batch = make_batch(new, ctx, group, 1, D, dtype, seed=40, pad=9)
    rows = tree_rows(new, 3, 40)
    masks = pack(rows, 1, sum(new) + 9)
    other = make_batch([64], [700], 16, 2, D, dtype, seed=41)
    chain = pack([[list(range(j + 1)) for j in range(64)]], 2, 64)
    results = []
    for scale in (0.0, 1.0, 6.0, 40.0):
        other.q.mul_(0).add_(1).mul_(scale)
        run(other, chain)
        batch.q[3:12] = torch.randn((9, group, D), generator=torch.Generator().manual_seed(int(scale))) * scale
        batch.q[14:] = scale
        results.append(run(batch, masks)[[0, 1, 2, 12, 13]])
    for got in results[1:]:
        assert torch.equal(got.view(torch.uint8), results[0].view(torch.uint8))

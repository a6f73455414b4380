"""Host-side checks of the speculative step's entry points (page tables, tree
masks, normed append, tree attention, accepted branches) without a GPU."""
import pytest

import paged_attention_decode_kv_gb300 as vt


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_attention_decode_kv_gb300 import build_lib
    build_lib.build()
    return vt.library()


BAD, NOT = vt.VT_ERR_INVALID_ARG, vt.VT_ERR_UNSUPPORTED
TABLES = dict(block_tables=0x1000, context_lens=0x2000, free_pages=0x3000, counters=0x4000, q_starts=0x5000,
              positions=0x6000, slots=0x7000, keep_lens=0x8000, new_lens=0x9000, num_seqs=3, num_tokens=9,
              block_size=32, stream=None, max_blocks_per_seq=4, num_blocks=16)
MASKS = dict(masks=0x1000, positions=0x2000, parents=0x3000, q_starts=0x4000, context_lens=0x5000, num_seqs=2,
             num_tokens=5, mask_words=1, stream=None)
NORM = dict(out=0x1000, x=0x2000, weight=0x5000, positions=0x3000, inv_freq=0x4000, num_tokens=2, num_heads=4,
            head_dim=128, rot_dim=128, interleaved=0, amplitude=1.0, eps=1e-6, x_stride=512, out_stride=512,
            weight_stride=0, stream=None, dtype=vt.VT_BF16)
APPEND = dict(k_cache=0x1000, v_cache=0x2000, q_out=0x3000, k=0x4000, v=0x5000, q=0x6000, k_weight=0xd000,
              q_weight=0xe000, q_starts=0x7000, block_tables=0x8000, context_lens=0x9000, positions=None,
              inv_freq=0xa000, num_seqs=2, num_tokens=5, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=32,
              rot_dim=128, interleaved=0, amplitude=1.0, eps=1e-6, q_stride=1024, k_stride=256, v_stride=256,
              q_weight_stride=0, k_weight_stride=128, stream=None, max_blocks_per_seq=4, num_blocks=16,
              dtype=vt.VT_BF16)
TREE = dict(out=0x1000, q=0x2000, k_cache=0x3000, v_cache=0x4000, masks=0x8000, q_starts=0x5000, block_tables=0x6000,
            context_lens=0x7000, num_seqs=2, num_tokens=5, mask_words=2, num_q_heads=8, num_kv_heads=2, head_dim=128,
            block_size=32, scale=0.1, window=0, stream=None, max_blocks_per_seq=4, num_blocks=16, dtype=vt.VT_BF16)
KEEP = dict(k_cache=0x1000, v_cache=0x2000, kept_lens=0x3000, accepted=0x4000, masks=0x5000, q_starts=0x6000,
            block_tables=0x7000, context_lens=0x8000, num_seqs=2, num_tokens=5, mask_words=1, num_layers=3,
            num_kv_heads=2, head_dim=128, block_size=32, k_layer_stride=16 * 32 * 256, v_layer_stride=16 * 32 * 256,
            stream=None, max_blocks_per_seq=4, num_blocks=16, dtype=vt.VT_BF16)
SCALES = dict(k_scale=0xb000, v_scale=0xc000)


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=-1), BAD), (dict(num_tokens=-1), BAD), (dict(max_blocks_per_seq=0), BAD), (dict(num_blocks=0), BAD),
    (dict(free_pages=None), BAD), (dict(counters=None), BAD), (dict(q_starts=None), BAD),
    (dict(block_tables=None), BAD), (dict(context_lens=None), BAD), (dict(new_lens=None), BAD),
    (dict(keep_lens=0x8002), BAD), (dict(slots=0x7001), BAD), (dict(positions=0x6002), BAD),
    (dict(block_size=16), NOT), (dict(num_seqs=16385), NOT), (dict(num_tokens=0x7ff00000), NOT),
    (dict(num_blocks=1 << 26), NOT), (dict(max_blocks_per_seq=1 << 26), NOT),
])
def test_step_tables_refusals(over, status):
    assert vt.vt_paged_step_tables(**dict(TABLES, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=0, masks=None), vt.VT_OK), (dict(num_tokens=0, masks=None), vt.VT_OK),
    (dict(num_seqs=-1), BAD), (dict(num_tokens=-2), BAD), (dict(masks=None), BAD), (dict(parents=None), BAD),
    (dict(q_starts=None), BAD), (dict(context_lens=None), BAD), (dict(mask_words=0), BAD), (dict(masks=0x1001), BAD),
    (dict(positions=0x2002), BAD), (dict(parents=0x1000), BAD), (dict(parents=0x2000), BAD),
    (dict(mask_words=33), NOT), (dict(num_seqs=0x7ff00000), NOT), (dict(num_tokens=0x7fffffff), NOT),
])
def test_tree_masks_refusals(over, status):
    assert vt.vt_tree_masks(**dict(MASKS, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(num_tokens=0, out=None, x=None), vt.VT_OK), (dict(num_tokens=-1), BAD), (dict(out=None), BAD),
    (dict(weight=None), BAD), (dict(weight=0x5008), BAD), (dict(weight_stride=64), BAD), (dict(weight_stride=130), BAD),
    (dict(weight_stride=-128), BAD), (dict(eps=-1e-9), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(positions=None), BAD), (dict(positions=0x3002), BAD),
    (dict(inv_freq=None), BAD), (dict(rot_dim=0), BAD), (dict(rot_dim=63), BAD), (dict(rot_dim=130), BAD),
    (dict(interleaved=2), BAD), (dict(amplitude=float("nan")), BAD), (dict(x=0x2008), BAD), (dict(x_stride=511), BAD),
    (dict(out_stride=516), BAD), (dict(out=0x2000, out_stride=1024), BAD), (dict(dtype=vt.VT_E4M3), BAD),
    (dict(num_heads=0), BAD), (dict(num_tokens=0x7fffffff), NOT), (dict(head_dim=100, rot_dim=100), NOT),
    (dict(head_dim=1032, x_stride=8256, out_stride=8256), NOT),
])
def test_norm_rope_refusals(over, status):
    assert vt.vt_norm_rope(**dict(NORM, **over)) == status


COMMON_APPEND = [
    (dict(num_seqs=0, k=None), vt.VT_OK), (dict(num_tokens=0, k=None), vt.VT_OK), (dict(num_seqs=-1), BAD),
    (dict(k=None), BAD), (dict(v_cache=None), BAD), (dict(q=None), BAD), (dict(q_out=None), BAD),
    (dict(k_weight=None), BAD), (dict(q_weight=None), BAD), (dict(k_weight=0xd004), BAD), (dict(q_weight=0xe008), BAD),
    (dict(k_weight_stride=100), BAD), (dict(q_weight_stride=129), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("inf")), BAD), (dict(k_stride=252), BAD), (dict(rot_dim=0), BAD), (dict(inv_freq=None), BAD),
    (dict(amplitude=float("inf")), BAD), (dict(q_out=0x6000, q_stride=2048), BAD), (dict(num_kv_heads=0), BAD),
    (dict(num_tokens=0x7ff00000), NOT), (dict(head_dim=96, rot_dim=96), NOT), (dict(block_size=16), NOT),
    (dict(num_blocks=1 << 27), NOT), (dict(num_seqs=0x7fffffff), NOT),
]


@pytest.mark.parametrize("over,status", COMMON_APPEND + [
    (dict(dtype=vt.VT_E4M3), BAD), (dict(dtype=9), BAD),
    (dict(head_dim=512, dtype=vt.VT_F32, k_stride=1024, v_stride=1024, q_stride=4096, k_weight_stride=0), NOT),
])
def test_norm_append_refusals(over, status):
    assert vt.vt_paged_kv_norm_append(**dict(APPEND, **over)) == status


@pytest.mark.parametrize("over,status", COMMON_APPEND + [
    (dict(k_scale=None), BAD), (dict(v_scale=0xc002), BAD),
    (dict(head_dim=512, k_stride=1024, v_stride=1024, q_stride=4096, k_weight_stride=0), NOT),
])
def test_norm_append_fp8_refusals(over, status):
    args = dict(APPEND, **SCALES)
    args.pop("dtype")
    assert vt.vt_paged_kv_norm_append_fp8(**dict(args, **over)) == status


COMMON_TREE = [
    (dict(num_seqs=0, q=None), vt.VT_OK), (dict(num_tokens=0, q=None), vt.VT_OK), (dict(num_tokens=-3), BAD),
    (dict(masks=None), BAD), (dict(masks=0x8002), BAD), (dict(mask_words=0), BAD), (dict(mask_words=-1), BAD),
    (dict(out=None), BAD), (dict(q_starts=None), BAD), (dict(q=0x2004), BAD), (dict(q=0x1000), BAD),
    (dict(num_q_heads=7), BAD), (dict(scale=float("nan")), BAD), (dict(num_blocks=0), BAD), (dict(mask_words=33), NOT),
    (dict(head_dim=96), NOT), (dict(block_size=64), NOT), (dict(num_q_heads=258), NOT),
    (dict(max_blocks_per_seq=1 << 27), NOT), (dict(num_seqs=0x7fffffff), NOT), (dict(num_tokens=0x7ff00000), NOT),
]


@pytest.mark.parametrize("over,status", COMMON_TREE + [
    (dict(dtype=vt.VT_E4M3), BAD), (dict(dtype=vt.VT_F32, head_dim=512), NOT),
    (dict(dtype=vt.VT_F32, num_q_heads=130), NOT),
])
def test_prefill_tree_refusals(over, status):
    assert vt.vt_paged_attn_prefill_tree(**dict(TREE, **over)) == status


@pytest.mark.parametrize("over,status", COMMON_TREE + [(dict(k_scale=None), BAD), (dict(k_scale=0xb001), BAD),
                                                       (dict(head_dim=512), NOT)])
def test_prefill_tree_fp8_refusals(over, status):
    args = dict(TREE, **SCALES)
    args.pop("dtype")
    assert vt.vt_paged_attn_prefill_tree_fp8(**dict(args, **over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(num_seqs=0, k_cache=None), vt.VT_OK), (dict(num_seqs=-1), BAD), (dict(num_layers=-1), BAD),
    (dict(k_cache=None), BAD), (dict(v_cache=None), BAD), (dict(kept_lens=None), BAD), (dict(accepted=None), BAD),
    (dict(masks=None), BAD), (dict(q_starts=None), BAD), (dict(block_tables=None), BAD),
    (dict(context_lens=None), BAD), (dict(kept_lens=0x8000), BAD), (dict(kept_lens=0x4000), BAD),
    (dict(kept_lens=0x6000), BAD), (dict(mask_words=0), BAD), (dict(num_kv_heads=0), BAD), (dict(head_dim=0), BAD),
    (dict(k_cache=0x1008), BAD), (dict(accepted=0x4002), BAD), (dict(dtype=3), BAD),
    (dict(k_layer_stride=16 * 32 * 256 - 8), BAD), (dict(v_layer_stride=16 * 32 * 256 + 4), BAD),
    (dict(mask_words=33), NOT), (dict(block_size=8), NOT), (dict(head_dim=3, num_kv_heads=1), NOT),
    (dict(num_tokens=0x7ff00000), NOT), (dict(num_blocks=1 << 27), NOT), (dict(num_seqs=0x7fffffff), NOT),
])
def test_keep_path_refusals(over, status):
    assert vt.vt_paged_kv_keep_path(**dict(KEEP, **over)) == status


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    i32 = torch.zeros((2,), dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16)
    w = torch.ones((64,))
    codes = cache.to(torch.float8_e4m3fn)
    ones = torch.ones((2,))
    with pytest.raises(ValueError, match="CUDA"):
        vt.step_tables(i32[:1], i32[:1], table, i32, i32, 4)
    with pytest.raises(ValueError, match="CUDA"):
        vt.tree_masks(i32, i32, i32[:1], 1)
    with pytest.raises(ValueError, match="CUDA"):
        vt.norm_rope(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        vt.norm_append(kv, kv, w, cache, cache.clone(), i32, table, i32[:1], q=x, q_weight=w)
    with pytest.raises(ValueError, match="CUDA"):
        vt.prefill_tree(x, cache, cache.clone(), i32[:, None], i32, table, i32[:1])
    with pytest.raises(ValueError, match="CUDA"):
        vt.prefill_tree_fp8(x, codes, codes.clone(), ones, ones, i32[:, None], i32, table, i32[:1])
    with pytest.raises(TypeError):
        vt.norm_append_fp8(kv, kv, w, cache, cache.clone(), ones, ones, i32, table, i32[:1])  # not codes
    with pytest.raises(ValueError, match="CUDA"):
        vt.keep_path(i32[:1], i32[:, None], cache, cache.clone(), i32, table, i32[:1])


def test_wrappers_refuse_trees_without_masks():
    """(which would be a causal chunk's rows)"""
    torch = pytest.importorskip("torch")
    i32 = torch.zeros((2,), dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16)
    codes = torch.zeros((3, 32, 2, 64), dtype=torch.uint8)
    ones = torch.ones((2,))
    with pytest.raises(ValueError, match="masks must be given"):
        vt.prefill_tree(x, cache, cache.clone(), None, i32, table, i32[:1])
    with pytest.raises(ValueError, match="masks must be given"):
        vt.prefill_tree_fp8(x, codes, codes.clone(), ones, ones, None, i32, table, i32[:1])


# ------------------------------------------------------------------- arguments in slots
def packed(op, values, count=None):
    import struct
    slots = [op, len(values) if count is None else count, *values]
    return vt.library().vt_call(struct.pack("".join("d" if isinstance(v, float) else "q" for v in slots), *slots))


CALLS = {1: (vt.vt_paged_step_tables, TABLES), 2: (vt.vt_tree_masks, MASKS), 3: (vt.vt_norm_rope, NORM),
         4: (vt.vt_paged_kv_norm_append, APPEND), 5: (vt.vt_paged_kv_norm_append_fp8, APPEND),
         6: (vt.vt_paged_attn_prefill_tree, TREE), 7: (vt.vt_paged_attn_prefill_tree_fp8, TREE),
         8: (vt.vt_paged_kv_keep_path, KEEP)}


def slots_of(op, **over):
    import inspect
    function, args = CALLS[op]
    args = dict(args, **SCALES, **over)
    return [0 if args[name] is None else args[name] for name in inspect.signature(function).parameters]


@pytest.mark.parametrize("op", sorted(CALLS))
def test_packed_calls(op):
    """Each argument arrives in its place: what is refused for one of them alone is refused here, too."""
    import inspect
    function, args = CALLS[op]
    names = list(inspect.signature(function).parameters)
    number = {1: "num_seqs", 2: "num_seqs", 3: "num_tokens", 4: "num_tokens", 5: "num_tokens", 6: "num_tokens",
              7: "num_tokens", 8: "num_seqs"}[op]
    if op != 1:                                                      # (no tokens, nothing to do, whatever else)
        assert packed(op, slots_of(op, **{number: 0})) == vt.VT_OK
    assert packed(op, slots_of(op, **{number: -1})) == BAD
    assert packed(op, slots_of(op, **{number: 0x7ff00000})) == NOT
    for name in ("block_size", "mask_words", "head_dim"):
        if name in names:
            assert packed(op, slots_of(op, **{name: 1 << 40})) == BAD        # no int
            assert packed(op, slots_of(op, **{name: -(1 << 32) + 32})) == BAD
    for name in ("eps", "scale"):
        if name in names:
            assert packed(op, slots_of(op, **{name: float("nan")})) == BAD
    for name in ("weight_stride", "q_weight_stride", "k_weight_stride"):
        if name in names:
            assert packed(op, slots_of(op, **{name: 130})) == BAD
    for name in names:
        if name in ("q_starts", "context_lens", "new_lens", "free_pages", "masks", "weight", "k_weight", "accepted"):
            assert packed(op, slots_of(op, **{name: args.get(name, 0x1000) + 1})) == BAD
    if names[-1] == "dtype":
        assert packed(op, slots_of(op, dtype=9)) == BAD
    values = slots_of(op)
    assert packed(op, values[:-1]) == BAD and packed(op, values + [0]) == BAD
    assert packed(op, values, count=len(values) + 1) == BAD


def test_packed_calls_of_nothing():
    assert packed(0, []) == BAD and packed(9, [0, 0]) == BAD and packed(-1, []) == BAD
    assert vt.library().vt_call(None) == BAD


@pytest.mark.parametrize("out", ["masks", "positions"])
@pytest.mark.parametrize("other", ["parents", "q_starts", "context_lens", "masks"])
def test_tree_masks_refuse_outputs_that_are_read(out, other):
    if out != other:
        assert vt.vt_tree_masks(**dict(MASKS, **{out: MASKS[other]})) == BAD


@pytest.mark.parametrize("other", ["context_lens", "accepted", "q_starts", "block_tables", "masks"])
def test_keep_path_refuses_lengths_that_are_read(other):
    assert vt.vt_paged_kv_keep_path(**dict(KEEP, kept_lens=KEEP[other])) == BAD

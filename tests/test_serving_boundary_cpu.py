"""Host-side checks of the rotary, append and prefill entry points, and the
frequency tables, on a machine without a GPU."""
import ctypes
import math

import pytest

import paged_attention_decode_kv_gb300 as vt


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_attention_decode_kv_gb300 import build_lib
    build_lib.build()
    return vt.library()


ROPE = dict(out=0x1000, x=0x2000, positions=0x3000, inv_freq=0x4000, num_tokens=2, num_heads=4, head_dim=128,
            rot_dim=128, interleaved=0, amplitude=1.0, x_stride=512, out_stride=512, stream=None, dtype=vt.VT_BF16)
APPEND = dict(k_cache=0x1000, v_cache=0x2000, q_out=0x3000, k=0x4000, v=0x5000, q=0x6000, q_starts=0x7000,
              block_tables=0x8000, context_lens=0x9000, positions=None, inv_freq=0xa000, num_seqs=2, num_tokens=5,
              num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=32, rot_dim=128, interleaved=0, amplitude=1.0,
              q_stride=1024, k_stride=256, v_stride=256, stream=None, max_blocks_per_seq=4, num_blocks=16,
              dtype=vt.VT_BF16)
PREFILL = dict(out=0x1000, q=0x2000, k_cache=0x3000, v_cache=0x4000, q_starts=0x5000, block_tables=0x6000,
               context_lens=0x7000, num_seqs=2, num_tokens=5, num_q_heads=8, num_kv_heads=2, head_dim=128,
               block_size=32, scale=0.1, window=0, stream=None, max_blocks_per_seq=4, num_blocks=16,
               dtype=vt.VT_BF16)
SCALES = dict(k_scale=0xb000, v_scale=0xc000)


@pytest.mark.parametrize("over,status", [
    (dict(num_tokens=0, out=None, x=None), vt.VT_OK),
    (dict(num_tokens=-1), vt.VT_ERR_INVALID_ARG),
    (dict(out=None), vt.VT_ERR_INVALID_ARG),
    (dict(positions=None), vt.VT_ERR_INVALID_ARG),
    (dict(inv_freq=None), vt.VT_ERR_INVALID_ARG),
    (dict(inv_freq=0x4004), vt.VT_ERR_INVALID_ARG),
    (dict(x=0x2008), vt.VT_ERR_INVALID_ARG),
    (dict(positions=0x3002), vt.VT_ERR_INVALID_ARG),
    (dict(rot_dim=0), vt.VT_ERR_INVALID_ARG),
    (dict(rot_dim=63), vt.VT_ERR_INVALID_ARG),
    (dict(rot_dim=130), vt.VT_ERR_INVALID_ARG),
    (dict(interleaved=2), vt.VT_ERR_INVALID_ARG),
    (dict(amplitude=float("nan")), vt.VT_ERR_INVALID_ARG),
    (dict(x_stride=511), vt.VT_ERR_INVALID_ARG),
    (dict(x_stride=516), vt.VT_ERR_INVALID_ARG),        # rows that do not start on 16 bytes
    (dict(out_stride=500), vt.VT_ERR_INVALID_ARG),
    (dict(out=0x2000, out_stride=1024), vt.VT_ERR_INVALID_ARG),
    (dict(dtype=vt.VT_E4M3), vt.VT_ERR_INVALID_ARG),
    (dict(num_heads=0), vt.VT_ERR_INVALID_ARG),
    (dict(num_tokens=0x7fffffff), vt.VT_ERR_UNSUPPORTED),
    (dict(head_dim=100, rot_dim=100), vt.VT_ERR_UNSUPPORTED),
    (dict(head_dim=1032, x_stride=8256, out_stride=8256), vt.VT_ERR_UNSUPPORTED),
])
def test_rope_refusals(over, status):
    assert vt.vt_rope(**dict(ROPE, **over)) == status


COMMON_APPEND = [
    (dict(num_seqs=0, k=None), vt.VT_OK),
    (dict(num_tokens=0, k=None), vt.VT_OK),
    (dict(num_seqs=-1), vt.VT_ERR_INVALID_ARG),
    (dict(k=None), vt.VT_ERR_INVALID_ARG),
    (dict(v_cache=None), vt.VT_ERR_INVALID_ARG),
    (dict(q_starts=None), vt.VT_ERR_INVALID_ARG),
    (dict(q=None), vt.VT_ERR_INVALID_ARG),              # q_out without q
    (dict(q_out=None), vt.VT_ERR_INVALID_ARG),
    (dict(k=0x4008), vt.VT_ERR_INVALID_ARG),
    (dict(positions=0x3002), vt.VT_ERR_INVALID_ARG),
    (dict(k_stride=252), vt.VT_ERR_INVALID_ARG),
    (dict(v_stride=258), vt.VT_ERR_INVALID_ARG),
    (dict(q_stride=8), vt.VT_ERR_INVALID_ARG),
    (dict(rot_dim=0), vt.VT_ERR_INVALID_ARG),           # a table without a rotated part
    (dict(q_out=0x6000, q_stride=2048), vt.VT_ERR_INVALID_ARG),  # in place, but with other strides
    (dict(inv_freq=None), vt.VT_ERR_INVALID_ARG),
    (dict(rot_dim=7), vt.VT_ERR_INVALID_ARG),
    (dict(amplitude=float("inf")), vt.VT_ERR_INVALID_ARG),
    (dict(num_kv_heads=0), vt.VT_ERR_INVALID_ARG),
    (dict(max_blocks_per_seq=0), vt.VT_ERR_INVALID_ARG),
    (dict(num_tokens=0x7ff00000), vt.VT_ERR_UNSUPPORTED),
    (dict(head_dim=96, rot_dim=96), vt.VT_ERR_UNSUPPORTED),
    (dict(block_size=16), vt.VT_ERR_UNSUPPORTED),
    (dict(num_blocks=1 << 27), vt.VT_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", COMMON_APPEND + [
    (dict(dtype=vt.VT_E4M3), vt.VT_ERR_INVALID_ARG),
    (dict(dtype=9), vt.VT_ERR_INVALID_ARG),
    (dict(head_dim=512, dtype=vt.VT_F32, k_stride=1024, v_stride=1024, q_stride=4096), vt.VT_ERR_UNSUPPORTED),
])
def test_append_refusals(over, status):
    assert vt.vt_paged_kv_append(**dict(APPEND, **over)) == status


@pytest.mark.parametrize("over,status", COMMON_APPEND + [
    (dict(k_scale=None), vt.VT_ERR_INVALID_ARG),
    (dict(v_scale=0xc002), vt.VT_ERR_INVALID_ARG),
    (dict(head_dim=512, k_stride=1024, v_stride=1024, q_stride=4096), vt.VT_ERR_UNSUPPORTED),
])
def test_append_fp8_refusals(over, status):
    args = dict(APPEND, **SCALES, **{})
    args.pop("dtype")
    assert vt.vt_paged_kv_append_fp8(**dict(args, **over)) == status


COMMON_PREFILL = [
    (dict(num_seqs=0, q=None), vt.VT_OK),
    (dict(num_tokens=0, q=None), vt.VT_OK),
    (dict(num_tokens=-3), vt.VT_ERR_INVALID_ARG),
    (dict(out=None), vt.VT_ERR_INVALID_ARG),
    (dict(q_starts=None), vt.VT_ERR_INVALID_ARG),
    (dict(context_lens=0x7002), vt.VT_ERR_INVALID_ARG),
    (dict(q=0x2004), vt.VT_ERR_INVALID_ARG),
    (dict(q=0x1000), vt.VT_ERR_INVALID_ARG),            # in place
    (dict(num_q_heads=7), vt.VT_ERR_INVALID_ARG),
    (dict(scale=float("nan")), vt.VT_ERR_INVALID_ARG),
    (dict(num_blocks=0), vt.VT_ERR_INVALID_ARG),
    (dict(head_dim=96), vt.VT_ERR_UNSUPPORTED),
    (dict(block_size=64), vt.VT_ERR_UNSUPPORTED),
    (dict(num_q_heads=258), vt.VT_ERR_UNSUPPORTED),     # 129 query heads for each kv head
    (dict(max_blocks_per_seq=1 << 27), vt.VT_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", COMMON_PREFILL + [
    (dict(dtype=vt.VT_E4M3), vt.VT_ERR_INVALID_ARG),
    (dict(dtype=vt.VT_F32, head_dim=512), vt.VT_ERR_UNSUPPORTED),
    (dict(dtype=vt.VT_F32, num_q_heads=130), vt.VT_ERR_UNSUPPORTED),
])
def test_prefill_refusals(over, status):
    assert vt.vt_paged_attn_prefill(**dict(PREFILL, **over)) == status


@pytest.mark.parametrize("over,status", COMMON_PREFILL + [
    (dict(k_scale=None), vt.VT_ERR_INVALID_ARG),
    (dict(k_scale=0xb001), vt.VT_ERR_INVALID_ARG),
    (dict(head_dim=512), vt.VT_ERR_UNSUPPORTED),
])
def test_prefill_fp8_refusals(over, status):
    args = dict(PREFILL, **SCALES)
    args.pop("dtype")
    assert vt.vt_paged_attn_prefill_fp8(**dict(args, **over)) == status


def test_workspace_bytes_of_what_is_not_taken():
    assert vt.vt_paged_attn_prefill_workspace_bytes(96, vt.VT_BF16) == 0
    assert vt.vt_paged_attn_prefill_workspace_bytes(512, vt.VT_F32) == 0


# ---- frequency tables ------------------------------------------------------------
def freq(rot, base=10000.0, kind=vt.VT_ROPE_PLAIN, factor=1.0, ctx=0.0, fast=32.0, slow=1.0):
    st, inv, amp = vt.vt_rope_frequencies(rot, base, vt.vt_rope_stretch(kind, factor, ctx, fast, slow))
    assert st == vt.VT_OK
    return inv, amp


def test_plain_and_linear_frequencies():
    inv, amp = freq(64)
    assert amp == 1.0
    assert inv == pytest.approx([10000.0 ** (-2 * j / 64) for j in range(32)], rel=1e-15)
    st, same, _ = vt.vt_rope_frequencies(64, 10000.0)
    assert st == vt.VT_OK and same == inv
    lin, amp = freq(64, kind=vt.VT_ROPE_LINEAR, factor=4.0)
    assert amp == 1.0 and lin == pytest.approx([f / 4 for f in inv], rel=1e-15)


def test_ntk_stretches_the_slowest_pair_by_the_factor():
    inv, _ = freq(128)
    ntk, amp = freq(128, kind=vt.VT_ROPE_NTK, factor=8.0)
    assert amp == 1.0 and ntk[0] == 1.0
    assert ntk[-1] == pytest.approx(inv[-1] / 8, rel=1e-12)


def test_yarn_keeps_fast_pairs_and_stretches_slow_ones():
    rot, base, factor, ctx = 128, 10000.0, 16.0, 4096.0
    inv, _ = freq(rot, base)
    got, amp = freq(rot, base, vt.VT_ROPE_YARN, factor, ctx)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-6)
    share = [(f / g - 1) / (factor - 1) for f, g in zip(inv, got)]  # 0: kept, 1: stretched
    for j, (f, s) in enumerate(zip(inv, share)):
        turns = ctx * f / (2 * math.pi)
        if turns > 32 * base ** (2 / rot):      # a whole pair above the bound (the ramp starts at its floor)
            assert s == pytest.approx(0.0, abs=1e-12), j
        if turns < base ** (-2 / rot):
            assert s == pytest.approx(1.0, abs=1e-12), j
    assert share == sorted(share) and 0 < share[30] < 1
    assert freq(rot, base, vt.VT_ROPE_YARN, 0.5, ctx)[1] == 1.0


def test_banded_is_linear_in_the_turns():
    rot, base, factor, ctx = 128, 5e5, 8.0, 8192.0
    inv, _ = freq(rot, base)
    got, amp = freq(rot, base, vt.VT_ROPE_BANDED, factor, ctx, 4.0, 1.0)
    assert amp == 1.0
    for f, g in zip(inv, got):
        turns = ctx * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        assert g == pytest.approx(keep * f + (1 - keep) * f / factor, rel=1e-13)


@pytest.mark.parametrize("rot,base,stretch", [
    (0, 1e4, None), (3, 1e4, None), (-2, 1e4, None), (64, 1.0, None), (64, float("inf"), None),
    (64, 1e4, (7, 1.0, 0, 0, 0)), (64, 1e4, (vt.VT_ROPE_LINEAR, 0.0, 0, 0, 0)),
    (64, 1e4, (vt.VT_ROPE_LINEAR, float("nan"), 0, 0, 0)), (2, 1e4, (vt.VT_ROPE_NTK, 2.0, 0, 0, 0)),
    (64, 1e4, (vt.VT_ROPE_YARN, 2.0, 0.0, 32, 1)), (64, 1e4, (vt.VT_ROPE_YARN, 2.0, 4096, 1, 1)),
    (64, 1e4, (vt.VT_ROPE_BANDED, 2.0, 4096, 4, 0)),
])
def test_frequency_refusals(rot, base, stretch):
    st, _, _ = vt.vt_rope_frequencies(rot, base, vt.vt_rope_stretch(*stretch) if stretch else None)
    assert st == vt.VT_ERR_INVALID_ARG


def test_frequencies_need_their_arrays(lib):
    amp = ctypes.c_float()
    assert lib.vt_rope_frequencies(None, ctypes.byref(amp), 64, 1e4, None) == vt.VT_ERR_INVALID_ARG
    inv = (ctypes.c_double * 32)()
    assert lib.vt_rope_frequencies(inv, None, 64, 1e4, None) == vt.VT_ERR_INVALID_ARG


# ---- the torch wrappers' own checks ----------------------------------------------
def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    kv = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16)
    i32 = torch.zeros((2,), dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    inv, amp = vt.rope_frequencies(64, device="cpu")
    assert inv.dtype == torch.float64 and inv.shape == (32,) and amp == 1.0
    with pytest.raises(ValueError, match="CUDA"):
        vt.rope(x, i32, inv)
    with pytest.raises(ValueError, match="CUDA"):
        vt.append(kv, kv, cache, cache.clone(), i32, table, i32[:1], q=x, inv_freq=inv)
    with pytest.raises(ValueError, match="CUDA"):
        vt.prefill(x, cache, cache.clone(), i32, table, i32[:1])
    codes = cache.to(torch.float8_e4m3fn)
    ones = torch.ones((2,))
    with pytest.raises(ValueError, match="CUDA"):
        vt.prefill_fp8(x, codes, codes.clone(), ones, ones, i32, table, i32[:1])
    with pytest.raises(TypeError):
        vt.append_fp8(kv, kv, cache, cache.clone(), ones, ones, i32, table, i32[:1])  # not codes
    with pytest.raises(vt.VtError):
        vt.rope_frequencies(63, device="cpu")


@pytest.mark.parametrize("over", [dict(num_seqs=0x7fffffff), dict(num_seqs=0x7ff00000), dict(num_tokens=0x7fffffff),
                                  dict(num_tokens=0x7ff00000)])
def test_batches_whose_numbers_would_leave_32_bits(over):
    """The search for a row's sequence probes past the last one; so many of them are refused."""
    for call, args in ((vt.vt_paged_kv_append, APPEND), (vt.vt_paged_attn_prefill, PREFILL)):
        assert call(**dict(args, **over)) == vt.VT_ERR_UNSUPPORTED

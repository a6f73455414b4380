// Rotary positions and the append of new keys and values to the paged cache.
//
// Mathematics.  A pair (a, b) of a head's row at position p becomes
// A (a cos w - b sin w), A (b cos w + a sin w) with w = p f_j.  Positions are
// integers, so only the fraction of a turn that f_j stands for matters: with
// u_j = frac(f_j / 2 pi) held as a 64-bit fixed-point fraction, p u_j modulo
// 2^64 is the reduced angle exactly as the hardware's integer product wraps,
// for either sign of p and at any distance.  Its top 32 bits become a float
// in [-1/2, 1/2) turns, and sincospi() takes it from there.  (In fp32 an
// angle of 10^5 radians would be off by 4e-3.)
//
// What bounds it: every element is read and written once, so HBM for long
// batches and the launch for short ones.  A warp takes tokens one by one (or a
// part of one's heads at either end of its share).  A lane has a fixed place in
// a head's row, 16 elements with 16-byte accesses, and walks over the token's
// heads four rounds at a time; the first rounds' loads are issued before the
// token is looked up (a warp-wide search of the row starts, then the block
// table).  Each angle is formed once for all heads: the lanes share out a
// token's pairs and hand (cos, sin) round by shuffles, so there is no table in
// shared memory and no block-wide wait, and a warp's next token reuses its
// frequencies.
// Measured (bf16, head_dim 128): 16803 tokens of 32 + 8 + 8 heads appended in
// 74 to 77 us, 5.5 TB/s of reads and writes; 5173 tokens of 64 + 8 + 8 into
// E4M3 pages 43 us; a block-wide kernel with a table in shared memory took 86
// and 54.  That one remains for rows the lanes do not divide (rot_dim or
// head_dim not a multiple of 16, head_dim 80 or 1024, say).
#include "rope_append.cuh"

extern "C" {

vt_status vt_rope_frequencies(double* inv_freq, float* amplitude, int rot_dim, double base,
                              const vt_rope_stretch* stretch) {
  if (!inv_freq || !amplitude || rot_dim <= 0 || rot_dim % 2 != 0 || !std::isfinite(base) || !(base > 1.0))
    return VT_ERR_INVALID_ARG;
  vt_rope_stretch s{};
  if (stretch) s = *stretch;
  if (s.kind < VT_ROPE_PLAIN || s.kind > VT_ROPE_BANDED) return VT_ERR_INVALID_ARG;
  if (s.kind != VT_ROPE_PLAIN && (!std::isfinite(s.factor) || !(s.factor > 0.0))) return VT_ERR_INVALID_ARG;
  if (s.kind == VT_ROPE_NTK && rot_dim < 4) return VT_ERR_INVALID_ARG;
  if ((s.kind == VT_ROPE_YARN || s.kind == VT_ROPE_BANDED) &&
      (!std::isfinite(s.original_context) || !(s.original_context > 0.0) || !std::isfinite(s.beta_fast) ||
       !(s.beta_slow > 0.0) || !(s.beta_fast > s.beta_slow)))
    return VT_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925;
  const double b = s.kind == VT_ROPE_NTK ? base * std::pow(s.factor, rot_dim / (rot_dim - 2.0)) : base;
  // YaRN's ramp runs over the pair index, between the (fractional) pairs that make beta_fast and beta_slow turns
  double first = 0.0, last = 0.0;
  if (s.kind == VT_ROPE_YARN) {
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(s.original_context / (turns * kTwoPi)) / (2.0 * std::log(base));
    };
    first = std::fmax(std::floor(pair_of(s.beta_fast)), 0.0);
    last = std::fmin(std::ceil(pair_of(s.beta_slow)), rot_dim - 1.0);
    if (!(last > first)) last = first + 0.001;
  }
  for (int j = 0; j < rot_dim / 2; ++j) {
    const double f = std::pow(b, -2.0 * j / rot_dim);
    double keep = 1.0;  // share of the pair that keeps its frequency
    if (s.kind == VT_ROPE_YARN) {
      keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (j - first) / (last - first)));
    } else if (s.kind == VT_ROPE_BANDED) {
      const double turns = s.original_context * f / kTwoPi;
      keep = std::fmin(1.0, std::fmax(0.0, (turns - s.beta_slow) / (s.beta_fast - s.beta_slow)));
    } else if (s.kind == VT_ROPE_LINEAR) {
      keep = 0.0;
    }
    const bool stretched = s.kind == VT_ROPE_LINEAR || s.kind == VT_ROPE_YARN || s.kind == VT_ROPE_BANDED;
    inv_freq[j] = stretched ? keep * f + (1.0 - keep) * f / s.factor : f;
  }
  *amplitude = s.kind == VT_ROPE_YARN && s.factor > 1.0 ? static_cast<float>(0.1 * std::log(s.factor) + 1.0) : 1.0f;
  return VT_OK;
}

vt_status vt_rope(void* out, const void* x, const int32_t* positions, const double* inv_freq, int num_tokens,
                  int num_heads, int head_dim, int rot_dim, int interleaved, float amplitude, long long x_stride,
                  long long out_stride, vt_stream_t stream, vt_dtype dtype) {
  using namespace vt;
  if (num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (num_tokens == 0) return VT_OK;
  if (!out || !x || !positions || (dtype != VT_BF16 && dtype != VT_F32) || num_heads <= 0 || head_dim <= 0)
    return VT_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(x, 16) || !aligned(positions, 4)) return VT_ERR_INVALID_ARG;
  if (!rotation_ok(inv_freq, rot_dim, head_dim, interleaved, amplitude, false)) return VT_ERR_INVALID_ARG;
  const int es = dtype == VT_F32 ? 4 : 2;
  if (!stride_ok(x_stride, num_heads, head_dim, es) || !stride_ok(out_stride, num_heads, head_dim, es))
    return VT_ERR_INVALID_ARG;
  if (out == x && x_stride != out_stride) return VT_ERR_INVALID_ARG;
  if (num_tokens > kMaxTokens || head_dim % 8 != 0 || head_dim > 1024) return VT_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_heads) * head_dim * kMaxTokensPerBlock > 0x3fffffffLL) return VT_ERR_UNSUPPORTED;
  RopeArgs a{};
  a.q = x;
  a.q_out = out;
  a.q_stride = x_stride;
  a.q_out_stride = out_stride;
  a.q_heads = num_heads;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.num_tokens = num_tokens;
  a.head_dim = head_dim;
  a.rot_dim = rot_dim;
  a.amplitude = amplitude;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return guarded([&] {
    int sms = 0;
    const vt_status st = current_sms(&sms);
    if (st != VT_OK) return st;
    const cudaError_t e = dtype == VT_BF16 ? launch_rope<__nv_bfloat16, __nv_bfloat16, false, false>(a, interleaved, sms, s)
                                           : launch_rope<float, float, false, false>(a, interleaved, sms, s);
    return e == cudaSuccess ? VT_OK : cuda_fail(e, "rope launch");
  });
}

vt_status vt_paged_kv_append(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v, const void* q,
                             const int32_t* q_starts, const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* positions, const double* inv_freq, int num_seqs, int num_tokens,
                             int num_q_heads, int num_kv_heads, int head_dim, int block_size, int rot_dim,
                             int interleaved, float amplitude, long long q_stride, long long k_stride,
                             long long v_stride, vt_stream_t stream, int max_blocks_per_seq, int num_blocks,
                             vt_dtype dtype) {
  if (dtype == VT_E4M3) return VT_ERR_INVALID_ARG;
  return vt::guarded([&] {
    return vt::append<false>(vt::append_args(k_cache, v_cache, q_out, k, v, q, nullptr, nullptr, q_starts, block_tables,
                                      context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                      num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                      max_blocks_per_seq, num_blocks),
                      block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), dtype);
  });
}

vt_status vt_paged_kv_append_fp8(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                 const void* q, const float* k_scale, const float* v_scale, const int32_t* q_starts,
                                 const int32_t* block_tables, const int32_t* context_lens, const int32_t* positions,
                                 const double* inv_freq, int num_seqs, int num_tokens, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size, int rot_dim, int interleaved,
                                 float amplitude, long long q_stride, long long k_stride, long long v_stride,
                                 vt_stream_t stream, int max_blocks_per_seq, int num_blocks) {
  return vt::guarded([&] {
    return vt::append<false>(vt::append_args(k_cache, v_cache, q_out, k, v, q, k_scale, v_scale, q_starts, block_tables,
                                      context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                      num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                      max_blocks_per_seq, num_blocks),
                      block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), VT_E4M3);
  });
}

}  // extern "C"

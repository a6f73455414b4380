// The norm of each query and key head in the pass that rotates it and appends
// keys and values to the paged cache.
//
// Mathematics.  A head's row x of head_dim elements becomes
// x / sqrt(mean(x^2) + eps) * weight and is then turned by its position's angles
// (rope_append.cu).  Everything is fp32 and rounded once, to the storage type
// or the code: between norm and rotation nothing is rounded.
//
// What bounds it: as without the norm, every element is read and written once,
// and here also issue: a lane's 16 elements cost some 170 instructions.  A row's
// elements are in its lanes' registers when its sum of squares is formed, so the
// norm costs log2 of those lanes in shuffles; weights and angles are multiplied
// once a token for all heads that share the weights, and products are taken two
// at a time.  Measured: 11583 tokens of 64 + 8 + 8 heads of 128 into E4M3 pages
// 77.7 us, 0.86 of the copy rate; 128 tokens of 32 + 8 + 8 4.7 us from a graph
// (fp32 5.1); 8191 tokens of 32 + 8 + 8 37.1, in fp32 66.6.  With weights per head
// the products of weights and angles are formed for every round of heads: 44.8 and,
// of the E4M3 batch, 104.  Rows that lanes do not divide (a rotation of 34 of 128)
// take 180: a warp a row, read twice an element at a time, its angles formed for
// every head.  Of the short batches' kernel, held to 128 registers, the variants of
// head_dim 512 spill 36 to 84 bytes and those of 256 up to 28.
#include "rope_append.cuh"

extern "C" {

vt_status vt_norm_rope(void* out, const void* x, const float* weight, const int32_t* positions,
                       const double* inv_freq, int num_tokens, int num_heads, int head_dim, int rot_dim,
                       int interleaved, float amplitude, float eps, long long x_stride, long long out_stride,
                       long long weight_stride, vt_stream_t stream, vt_dtype dtype) {
  using namespace vt;
  if (num_tokens < 0) return VT_ERR_INVALID_ARG;
  if (num_tokens == 0) return VT_OK;
  if (!out || !x || (dtype != VT_BF16 && dtype != VT_F32) || num_heads <= 0 || head_dim <= 0)
    return VT_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(x, 16) || !aligned(positions, 4)) return VT_ERR_INVALID_ARG;
  if (!rotation_ok(inv_freq, rot_dim, head_dim, interleaved, amplitude, true)) return VT_ERR_INVALID_ARG;
  if (rot_dim > 0 && !positions) return VT_ERR_INVALID_ARG;
  if (!weight_ok(weight, weight_stride, head_dim) || !eps_ok(eps)) return VT_ERR_INVALID_ARG;
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
  a.q_weight = weight;
  a.q_weight_stride = weight_stride;
  a.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return guarded([&] {
    int sms = 0;
    const vt_status st = current_sms(&sms);
    if (st != VT_OK) return st;
    const cudaError_t e = dtype == VT_BF16
                              ? launch_rope<__nv_bfloat16, __nv_bfloat16, false, true>(a, interleaved, sms, s)
                              : launch_rope<float, float, false, true>(a, interleaved, sms, s);
    return e == cudaSuccess ? VT_OK : cuda_fail(e, "norm rope launch");
  });
}

vt_status vt_paged_kv_norm_append(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                  const void* q, const float* k_weight, const float* q_weight,
                                  const int32_t* q_starts, const int32_t* block_tables, const int32_t* context_lens,
                                  const int32_t* positions, const double* inv_freq, int num_seqs, int num_tokens,
                                  int num_q_heads, int num_kv_heads, int head_dim, int block_size, int rot_dim,
                                  int interleaved, float amplitude, float eps, long long q_stride,
                                  long long k_stride, long long v_stride, long long q_weight_stride,
                                  long long k_weight_stride, vt_stream_t stream, int max_blocks_per_seq,
                                  int num_blocks, vt_dtype dtype) {
  if (dtype == VT_E4M3) return VT_ERR_INVALID_ARG;
  return vt::guarded([&] {
    vt::RopeArgs a = vt::append_args(k_cache, v_cache, q_out, k, v, q, nullptr, nullptr, q_starts, block_tables,
                                     context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                     max_blocks_per_seq, num_blocks);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_weight_stride = q_weight_stride;
    a.k_weight_stride = k_weight_stride;
    a.eps = eps;
    return vt::append<true>(a, block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), dtype);
  });
}

vt_status vt_paged_kv_norm_append_fp8(void* k_cache, void* v_cache, void* q_out, const void* k, const void* v,
                                      const void* q, const float* k_weight, const float* q_weight,
                                      const float* k_scale, const float* v_scale, const int32_t* q_starts,
                                      const int32_t* block_tables, const int32_t* context_lens,
                                      const int32_t* positions, const double* inv_freq, int num_seqs,
                                      int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                      int block_size, int rot_dim, int interleaved, float amplitude, float eps,
                                      long long q_stride, long long k_stride, long long v_stride,
                                      long long q_weight_stride, long long k_weight_stride, vt_stream_t stream,
                                      int max_blocks_per_seq, int num_blocks) {
  return vt::guarded([&] {
    vt::RopeArgs a = vt::append_args(k_cache, v_cache, q_out, k, v, q, k_scale, v_scale, q_starts, block_tables,
                                     context_lens, positions, inv_freq, num_seqs, num_tokens, num_q_heads,
                                     num_kv_heads, head_dim, rot_dim, amplitude, q_stride, k_stride, v_stride,
                                     max_blocks_per_seq, num_blocks);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.q_weight_stride = q_weight_stride;
    a.k_weight_stride = k_weight_stride;
    a.eps = eps;
    return vt::append<true>(a, block_size, interleaved, reinterpret_cast<cudaStream_t>(stream), VT_E4M3);
  });
}

}  // extern "C"

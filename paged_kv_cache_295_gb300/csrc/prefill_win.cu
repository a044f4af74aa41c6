// paged_attention_prefill_window: argument checks, tensor maps and the launch of
// the tcgen05 prefill kernel with a window, sinks and scales per block.
#include <cmath>

#include "prefill_win.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
int ilog2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status paged_attention_prefill_window(
    const void* q, const int32_t* query_start, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, const int32_t* context_lens, int32_t num_seqs,
    int32_t num_tokens, int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
    int32_t max_context_len, float scale, int32_t causal, int32_t q_dtype, int32_t kv_dtype,
    const float* k_scale, const float* v_scale, int64_t scale_stride, int32_t window,
    int32_t sinks, int32_t out_dtype, void* out, int32_t* device_status, pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
      window < 0 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || (causal != 0 && causal != 1)) return PKV_ERR_INVALID_ARG;
  if ((window > 0 && !causal) || (sinks > 0 && window == 0)) return PKV_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  const int G = num_q_heads / num_kv_heads;
  const bool codes = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_INT8;
  if (head_dim != kPfD || q_dtype != PKV_BF16 || (kv_dtype != PKV_BF16 && !codes) || G > 16)
    return PKV_ERR_UNSUPPORTED;
  if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (!pow2(block_size) || block_size < 8 || block_size > 4096) return PKV_ERR_UNSUPPORTED;
  if (num_blocks > INT32_MAX || num_blocks * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const int64_t by_table = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  if (by_table > INT32_MAX || max_context_len > by_table) return PKV_ERR_INVALID_ARG;
  if (max_context_len > (1 << 30) || num_seqs > 65535 || num_kv_heads > 65535)
    return PKV_ERR_UNSUPPORTED;
  if (max_query_len > num_tokens) return PKV_ERR_INVALID_ARG;
  if (codes && scale_stride != 0 && scale_stride < num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_query_len == 0) return PKV_OK;
  if (!q || !query_start || !k_cache || !v_cache || !block_tables || !context_lens || !out ||
      (codes && (!k_scale || !v_scale)))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      !aligned4(query_start) || !aligned4(block_tables) || !aligned4(context_lens))
    return PKV_ERR_INVALID_ARG;
  if (!encode_fn()) return PKV_ERR_CUDA;

  PrefillWinParams w{};
  PrefillParams& p = w.p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.status = device_status;
  p.num_blocks = num_blocks;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.bs_log2 = ilog2(block_size);
  p.box_rows = block_size < kPfKeys ? block_size : kPfKeys;
  p.tile_tokens = kPfRows / G;
  p.causal = causal;
  p.max_context_len = max_context_len;
  p.num_tokens = num_tokens;
  p.qk_scale_log2 = scale * 1.4426950408889634f;
  p.test_stall_bytes = test_stall_bytes();
  p.k_scale = codes ? k_scale : nullptr;
  p.v_scale = codes ? v_scale : nullptr;
  w.out = out;
  w.scale_stride = codes ? scale_stride : 0;
  w.out_bf16 = out_dtype == PKV_BF16;
  w.window = window;
  w.sinks = sinks;

  CUtensorMap tk, tv;
  const int64_t rows = num_blocks * block_size;
  if (!make_map(&tk, k_cache, kPfD, num_kv_heads, rows, p.box_rows, codes) ||
      !make_map(&tv, v_cache, kPfD, num_kv_heads, rows, p.box_rows, codes))
    return PKV_ERR_CUDA;

  const int pairs = (max_query_len + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
  const dim3 grid(pairs, num_kv_heads, num_seqs);
  auto launch = [&](auto kern, int threads, size_t smem) {
    if (!opt_in_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem)))
      return PKV_ERR_CUDA;
    kern<<<grid, threads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(tk, tv, w);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  };
  const size_t smem8 = PwLayout::bytes(kPfStagesFp8, true);
  // 8-bit caches: two fp16 weight parts for a float32 output, one for a bf16 output
  if (kv_dtype == PKV_FP8_E4M3)
    return w.out_bf16 ? launch(paged_prefill_win_kernel<kPfStagesFp8, 1, false>, kPwThreads8, smem8)
                      : launch(paged_prefill_win_kernel<kPfStagesFp8, 1, true>, kPwThreads8, smem8);
  if (kv_dtype == PKV_INT8)
    return w.out_bf16 ? launch(paged_prefill_win_kernel<kPfStagesFp8, 2, false>, kPwThreads8, smem8)
                      : launch(paged_prefill_win_kernel<kPfStagesFp8, 2, true>, kPwThreads8, smem8);
  return launch(paged_prefill_win_kernel<kPfStages, 0, true>, kPfThreads,
                PwLayout::bytes(kPfStages, false));
}

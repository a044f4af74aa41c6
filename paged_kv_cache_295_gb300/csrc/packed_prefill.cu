// packed_attention_prefill: argument checks, tensor maps and the launch of the tcgen05 kernel over
// packed prompts.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "packed_prefill.cuh"
#include "ranges.cuh"
#include "tmap.cuh"

namespace pkv {
namespace {

constexpr int64_t kMaxStride = int64_t{1} << 38;   // elements; a tensor map takes 2^40 bytes

// 3-D map over rows [rows][heads][dim] of bf16 with these strides (elements): boxes of 64 dims (what lies
// past `dim` reads as 0), box_heads heads and box_rows rows.
bool rows_map(CUtensorMap* m, const void* base, int dim, int heads, int64_t rows, int64_t head_stride,
              int64_t row_stride, int box_heads, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  if (heads == 1) head_stride = (dim + 7) / 8 * 8;   // of a single one the stride says nothing
  if (rows == 1) row_stride = (dim + 7) / 8 * 8;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
  cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}


// A stride between rows or heads, where there is more than one of them.
bool stride_ok(int64_t stride, int64_t count) {
  return count <= 1 || (stride > 0 && stride % 8 == 0 && stride < kMaxStride);
}

// Items of a call at most: a sequence's last pair of query tiles may be short.
int64_t units_of(const pkv_packed_prefill_args& a) {
  const int pair = 2 * (kPkRows / (a.num_q_heads / a.num_kv_heads));
  return ((static_cast<int64_t>(a.num_tokens) + pair - 1) / pair + a.num_seqs) * a.num_kv_heads;
}

// What packed_attention_prefill refuses.
pkv_status refusal(const pkv_packed_prefill_args& a) {
  if (a.num_seqs < 0 || a.num_tokens < 0 || a.num_keys < 0 || a.num_q_heads <= 0 || a.num_kv_heads <= 0 ||
      a.head_dim <= 0 || a.window < 0 || a.sinks < 0 || (a.causal != 0 && a.causal != 1) ||
      a.num_q_heads % a.num_kv_heads != 0 || !std::isfinite(a.scale))
    return PKV_ERR_INVALID_ARG;
  if ((a.window > 0 && !a.causal) || (a.sinks > 0 && a.window == 0)) return PKV_ERR_INVALID_ARG;
  if (a.weight_parts < 0 || a.weight_parts > 2) return PKV_ERR_INVALID_ARG;
  const int G = a.num_q_heads / a.num_kv_heads;
  if (a.q_dtype != PKV_BF16 || a.kv_dtype != PKV_BF16 || (a.out_dtype != PKV_F32 && a.out_dtype != PKV_BF16))
    return PKV_ERR_UNSUPPORTED;
  if (a.weight_parts == 1 && a.out_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (a.head_dim > 128 || a.head_dim % 8 != 0 || G > kPkRows || a.num_seqs > (1 << 24) ||
      a.num_tokens > (1 << 30) || a.num_keys > (1 << 30) || a.num_q_heads > (1 << 16))
    return PKV_ERR_UNSUPPORTED;
  // of no rows the strides say nothing
  if (a.num_tokens > 0 && (!stride_ok(a.q_token_stride, a.num_tokens) || !stride_ok(a.q_head_stride, a.num_q_heads)))
    return PKV_ERR_INVALID_ARG;
  if (a.num_keys > 0 && (!stride_ok(a.k_token_stride, a.num_keys) || !stride_ok(a.k_head_stride, a.num_kv_heads) ||
                         !stride_ok(a.v_token_stride, a.num_keys) || !stride_ok(a.v_head_stride, a.num_kv_heads)))
    return PKV_ERR_INVALID_ARG;
  if (a.num_seqs == 0 || a.num_tokens == 0) return PKV_OK;
  if (!a.q || !a.out || !a.query_start || (a.num_keys > 0 && (!a.k || !a.v))) return PKV_ERR_INVALID_ARG;
  if (!a.key_start && a.num_keys != a.num_tokens) return PKV_ERR_INVALID_ARG;
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.v) || !aligned16(a.out) || !aligned4(a.query_start) ||
      !aligned4(a.key_start) || !aligned4(a.context_lens) || !aligned4(a.device_status))
    return PKV_ERR_INVALID_ARG;

  // from the first element to the last one
  auto range = [&](int64_t rows, int64_t heads, int64_t row_stride, int64_t head_stride) {
    return static_cast<size_t>(2 * ((rows > 1 ? (rows - 1) * row_stride : 0) + (heads > 1 ? (heads - 1) * head_stride : 0) +
                                    a.head_dim));
  };
  const size_t out_bytes = static_cast<size_t>(a.num_tokens) * a.num_q_heads * a.head_dim * elem_bytes(a.out_dtype);
  const size_t starts = 4 * (static_cast<size_t>(a.num_seqs) + 1);
  if (overlap(a.out, out_bytes, a.q, range(a.num_tokens, a.num_q_heads, a.q_token_stride, a.q_head_stride)) ||
      (a.num_keys > 0 &&
       (overlap(a.out, out_bytes, a.k, range(a.num_keys, a.num_kv_heads, a.k_token_stride, a.k_head_stride)) ||
        overlap(a.out, out_bytes, a.v, range(a.num_keys, a.num_kv_heads, a.v_token_stride, a.v_head_stride)))) ||
      overlap(a.out, out_bytes, a.query_start, starts) || overlap(a.out, out_bytes, a.key_start, starts) ||
      overlap(a.out, out_bytes, a.context_lens, starts - 4))
    return PKV_ERR_INVALID_ARG;

  // the items are counted in 32 bits
  if (units_of(a) > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status packed_attention_prefill_check(const pkv_packed_prefill_args* args) {
  return args ? pkv::refusal(*args) : PKV_ERR_INVALID_ARG;
}

extern "C" pkv_status packed_attention_prefill(const pkv_packed_prefill_args* args, pkv_stream_t stream) {
  using namespace pkv;
  const pkv_status refused = packed_attention_prefill_check(args);
  if (refused != PKV_OK) return refused;
  const pkv_packed_prefill_args& a = *args;
  if (a.num_seqs == 0 || a.num_tokens == 0) return PKV_OK;
  const int G = a.num_q_heads / a.num_kv_heads;
  PackedParams p{};
  p.out = a.out;
  p.query_start = a.query_start;
  p.key_start = a.key_start ? a.key_start : a.query_start;
  p.context_lens = a.context_lens;
  p.status = a.device_status;
  p.num_seqs = a.num_seqs, p.num_tokens = a.num_tokens, p.num_keys = a.num_keys;
  p.num_q_heads = a.num_q_heads, p.num_kv_heads = a.num_kv_heads, p.dim = a.head_dim;
  p.tile_tokens = kPkRows / G;
  // A window past all keys hides none, and one of that size does: position - window, of a query before
  // every key too (-2^30 at the least), stays within 32 bits.
  p.causal = a.causal, p.window = std::min(a.window, std::max(a.num_keys, 1)), p.sinks = a.sinks;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.test_stall_bytes = test_stall_bytes();

  CUtensorMap tq, tk, tv;
  auto keys_map = [&](CUtensorMap* m, const void* base, int64_t head_stride, int64_t token_stride) {
    if (a.num_keys == 0)   // no key tile is read: any map will do
      return rows_map(m, a.q, a.head_dim, a.num_kv_heads, 1, a.q_head_stride, 0, 1, kPkKeys);
    return rows_map(m, base, a.head_dim, a.num_kv_heads, a.num_keys, head_stride, token_stride, 1, kPkKeys);
  };
  if (!rows_map(&tq, a.q, a.head_dim, a.num_q_heads, a.num_tokens, a.q_head_stride, a.q_token_stride, G,
                p.tile_tokens) ||
      !keys_map(&tk, a.k, a.k_head_stride, a.k_token_stride) || !keys_map(&tv, a.v, a.v_head_stride, a.v_token_stride))
    return PKV_ERR_CUDA;

  const int64_t units = units_of(a);   // no more CTAs than items
  const int64_t sms = device_sm_count();
  const dim3 grid(static_cast<unsigned>(units < sms ? units : sms));
  auto launch = [&](auto kern, size_t smem) {
    if (!opt_in_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem))) return PKV_ERR_CUDA;
    return cuda_status(launch_pdl(kern, grid, dim3(kPkThreads), smem, reinterpret_cast<cudaStream_t>(stream), tq, tk,
                                  tv, p));
  };
  auto of = [&](auto slabs, auto stages) {
    constexpr int N = decltype(slabs)::value, ST = decltype(stages)::value;
    const size_t smem = PkLayout<N, ST>::bytes();
    return a.out_dtype == PKV_F32 ? launch(packed_prefill_kernel<N, ST, true, true>, smem)
           : a.weight_parts == 1  ? launch(packed_prefill_kernel<N, ST, false, false>, smem)
                                  : launch(packed_prefill_kernel<N, ST, false, true>, smem);
  };
  return a.head_dim > 64 ? of(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{})
                         : of(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
}

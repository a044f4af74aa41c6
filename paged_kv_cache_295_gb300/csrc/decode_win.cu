// paged_attention_decode_window: argument checks, partition choice and the
// launch of the windowed decode kernel (16-bit caches here, 8-bit ones in
// decode_win_8bit.cu).
#include <cmath>

#include "decode_win_launch.cuh"

namespace pkv {
namespace {

bool pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
int ilog2(int64_t x) {
  int l = 0;
  while ((int64_t{1} << l) < x) ++l;
  return l;
}

// Tokens of whole 32-token chunks a query can see: what the partitions are
// sized for (16-token chunks need no more).
int64_t visible_tokens(int32_t max_ctx, int32_t window, int32_t sinks) {
  return 32 * max_visible_chunks(max_ctx, window, sinks, 32);
}

// Most CTAs (heads times partitions) of a launch whose partition is chosen here.  It bounds the
// scratch of every call up to a given size: it grows with both arguments, where the choice itself
// goes up and down.  Twice what the box table's 4,096 tokens a CTA need, and at least eight waves,
// past which shorter partitions gain less than 1.5 % by the estimate below.
int64_t most_ctas(int64_t heads, int64_t tokens) {
  const int64_t waves = 8 * 3LL * device_sm_count(), twice = 2 * heads * ((tokens + 4095) / 4096);
  return twice > waves ? twice : waves;
}

// Tokens per partition.  `tokens` is what the longest query can see; token_bytes the K and V
// bytes of one token and head.  With n partitions a launch has heads * n CTAs of about
// tokens / n tokens, three to an SM, and is estimated (us) as
//   3, and for merging 1.5 more within a cluster, 2 by a second kernel
//   + per full wave of CTA slots: 1 + len * slots * token_bytes / HBM bandwidth
//   + the last, partial wave: 1 + len * the root of the squares of that rate times how full
//     the wave is and of the rate of a CTA alone, which its two-stage rings bound (42 KB/us).
// The n with the least estimate is taken, of those within most_ctas.  Measured (bf16, GQA-8,
// 64 x 8 heads, window 1024): one partition 57.6 us (1.1 waves), two of 576 and 512 57.4, of
// 704 and 384 53.0; 16 x 8 heads, GQA-4: 20.3 with one, 17.1 with three; 4 x 8 heads: 18.6
// with one, 8.7 with six; one sequence, window 4096: 56.9 with two, 10.1 with 33.
int32_t auto_win_partition(int64_t heads, int64_t tokens, int token_bytes) {
  const int64_t most = most_ctas(heads, tokens);
  const double slots = 3.0 * device_sm_count();
  const double full = slots * token_bytes / 6.6e6, alone = token_bytes / 4.2e4;
  int32_t best = 4096;
  double least = 1e30;
  auto consider = [&](int64_t len, double t) {
    if (t < least && heads * ((tokens + len - 1) / len) <= most) {
      least = t;
      best = static_cast<int32_t>(len);
    }
  };
  int32_t before = 0;
  for (int64_t n = 1; n <= 64; ++n) {
    int64_t len = ((tokens + n - 1) / n + 63) / 64 * 64;
    if (len < 64) len = 64;
    if (len > 4096 || len == before) continue;   // 4096: the box table's room
    before = static_cast<int32_t>(len);
    const int64_t parts = (tokens + len - 1) / len;
    const double waves = static_cast<double>(heads) * parts / slots;
    const double whole = static_cast<double>(static_cast<int64_t>(waves)), rest = waves - whole;
    const double merge = parts <= 1 ? 0 : parts <= kWinCluster && heads * parts <= slots ? 1.5 : 2;
    double t = 3.0 + merge + whole * (1.0 + len * full);
    if (rest > 0) t += 1.0 + len * std::sqrt(rest * full * rest * full + alone * alone);
    consider(len, t);
    // The same number of partitions with a last one of about 40 %: past one wave the short
    // ones fill the slots that equal ones would leave empty at the end.
    const int64_t longer = (tokens * 10 / (10 * n - 6) + 63) / 64 * 64, last = tokens - (n - 1) * longer;
    if (n > 1 && waves > 1 && longer <= 4096 && last > 0)
      consider(longer, 5.0 + waves + heads * tokens / slots * full + last * alone);
  }
  return best;
}

int32_t win_partition(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int64_t tokens,
                      int token_bytes, int32_t req) {
  if (req < 0 || req % 64 != 0) return 0;
  if (req > 0) return req;
  const int split = num_q_heads / num_kv_heads > 8 ? 2 : 1;
  return auto_win_partition(static_cast<int64_t>(num_seqs) * num_kv_heads * split, tokens,
                            token_bytes);
}

// Whether the partitions of a sequence and head run as one cluster.  Clusters save the
// scratch and the merging kernel (4 sequences x 8 heads: 8.9 -> 8.3 us, and a launch on the
// host) but a cluster waits for all of its CTA slots at once: where the grid is more than
// one wave of slots they lose (64 x 8 heads, two partitions: 52 us without, 69 with).
bool in_cluster(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int64_t parts) {
  const int split = num_q_heads / num_kv_heads > 8 ? 2 : 1;
  return parts > 1 && parts <= kWinCluster &&
         static_cast<int64_t>(num_seqs) * num_kv_heads * split * parts <= 3LL * device_sm_count();
}

size_t window_scratch(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                      int32_t head_dim, int64_t tokens, int32_t P) {
  const int64_t parts = P > 0 ? (tokens + P - 1) / P : 0;
  if (parts <= 1 || in_cluster(num_seqs, num_q_heads, num_kv_heads, parts)) return 0;
  return static_cast<size_t>(num_seqs) * num_q_heads * parts * (head_dim + 2) * sizeof(float);
}

template <int D>
pkv_status launch16(const WinLaunch& a, const CUtensorMap& tk, const CUtensorMap& tv) {
  constexpr int NW = D == 256 ? 2 : 4, STAGES = D == 64 ? 3 : 2;   // as launch_mma2
  return a.q_f32 ? launch_win_shape<BF16, D, true, true, NW, STAGES, 16>(a, tk, tv)
                 : launch_win_shape<BF16, D, false, true, NW, STAGES, 16>(a, tk, tv);
}

}  // namespace

pkv_status launch_decode_win(const WinLaunch& a) {
  CUtensorMap tk, tv;
  if (!win_maps(a, &tk, &tv)) return PKV_ERR_CUDA;
  switch (a.head_dim) {
    case 64: return launch16<64>(a, tk, tv);
    case 128: return launch16<128>(a, tk, tv);
    default: return launch16<256>(a, tk, tv);
  }
}

}  // namespace pkv

extern "C" size_t paged_attention_window_workspace_bytes(int32_t num_seqs, int32_t num_q_heads,
                                                         int32_t num_kv_heads, int32_t head_dim,
                                                         int32_t max_context_len,
                                                         int32_t partition_tokens, int32_t window,
                                                         int32_t sinks) {
  if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context_len < 0 || window < 0 || sinks < 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  const int64_t tokens = pkv::visible_tokens(max_context_len, window, sinks);
  if (partition_tokens != 0)   // grows with the batch and the context
    return pkv::window_scratch(num_seqs, num_q_heads, num_kv_heads, head_dim, tokens,
                               pkv::win_partition(num_seqs, num_q_heads, num_kv_heads, tokens, 1,
                                                  partition_tokens));
  // an automatic partition has at least 64 tokens and a launch at most most_ctas
  if (tokens <= 64) return 0;
  const int64_t group = num_q_heads / num_kv_heads, split = group > 8 ? 2 : 1;
  const int64_t heads = static_cast<int64_t>(num_seqs) * num_kv_heads * split;
  const int64_t short_ones = heads * ((tokens + 63) / 64), most = pkv::most_ctas(heads, tokens);
  const int64_t ctas = short_ones < most ? short_ones : most;
  return static_cast<size_t>((ctas * group + split - 1) / split) * (head_dim + 2) * sizeof(float);
}

extern "C" size_t paged_attention_window_call_bytes(int32_t num_seqs, int32_t num_q_heads,
                                                    int32_t num_kv_heads, int32_t head_dim,
                                                    int32_t max_context_len,
                                                    int32_t partition_tokens, int32_t window,
                                                    int32_t sinks, int32_t kv_dtype) {
  if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      max_context_len < 0 || window < 0 || sinks < 0 || num_q_heads % num_kv_heads != 0)
    return 0;
  const int64_t tokens = pkv::visible_tokens(max_context_len, window, sinks);
  const int32_t P = pkv::win_partition(num_seqs, num_q_heads, num_kv_heads, tokens,
                                       2 * head_dim * pkv::elem_bytes(kv_dtype), partition_tokens);
  return pkv::window_scratch(num_seqs, num_q_heads, num_kv_heads, head_dim, tokens, P);
}

extern "C" pkv_status paged_attention_decode_window(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* context_lens, int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
    int32_t max_context_len, float scale, int32_t q_dtype, int32_t kv_dtype, const float* k_scale,
    const float* v_scale, int64_t scale_stride, int32_t window, int32_t sinks, int32_t out_dtype,
    void* out, void* workspace, size_t workspace_bytes, int32_t partition_tokens,
    int32_t* device_status, pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_context_len < 0 || window < 0 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_q_heads % num_kv_heads != 0 || partition_tokens < 0 || partition_tokens % 64 != 0)
    return PKV_ERR_INVALID_ARG;
  if (sinks > 0 && window == 0) return PKV_ERR_INVALID_ARG;   // sinks add to a window
  if (!std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
    return PKV_ERR_INVALID_ARG;
  const bool codes = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_INT8;
  if (!codes && kv_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (codes ? head_dim != 128 : (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return PKV_ERR_UNSUPPORTED;
  if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  const int G = num_q_heads / num_kv_heads;
  if (G > 16 || !pow2(block_size) || block_size < 8 || block_size > 4096)
    return PKV_ERR_UNSUPPORTED;
  if (num_blocks > INT32_MAX || num_blocks * block_size > INT32_MAX ||
      max_context_len > (1 << 30) || num_seqs > 65535 || num_kv_heads > 32767 ||
      static_cast<int64_t>(num_seqs) * num_q_heads > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  if (codes && scale_stride != 0 && scale_stride < num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out ||
      (codes && (!k_scale || !v_scale)))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return PKV_ERR_INVALID_ARG;
  if (!encode_fn()) return PKV_ERR_CUDA;

  const int64_t tokens = visible_tokens(max_context_len, window, sinks);
  const int32_t P = win_partition(num_seqs, num_q_heads, num_kv_heads, tokens,
                                  2 * head_dim * (codes ? 1 : 2), partition_tokens);
  if (P <= 0) return PKV_ERR_INVALID_ARG;
  const int64_t parts = tokens > 0 ? (tokens + P - 1) / P : 1;
  if (parts > 65535) return PKV_ERR_UNSUPPORTED;
  const size_t need = window_scratch(num_seqs, num_q_heads, num_kv_heads, head_dim, tokens, P);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return PKV_ERR_INVALID_ARG;

  WinLaunch a{};
  DecodeParams& p = a.w.p;
  p.q = q;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  float* ws = static_cast<float*>(workspace);
  p.part_ml = need > 0 ? ws : nullptr;
  p.part_o = need > 0 ? ws + static_cast<size_t>(num_seqs) * num_q_heads * parts * 2 : nullptr;
  p.status = device_status;
  p.num_kv_heads = num_kv_heads;
  p.num_q_heads = num_q_heads;
  p.bs_log2 = ilog2(block_size);
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.partition_tokens = P;
  p.max_parts = static_cast<int32_t>(parts);
  p.q_is_bf16 = q_dtype == PKV_BF16;
  p.qk_scale_log2 = scale * 1.4426950408889634f;
  p.test_stall_bytes = test_stall_bytes();
  const int chl = codes ? 5 : 4;
  a.w.out = out;
  a.w.scale_stride = codes ? scale_stride : 0;
  a.w.out_bf16 = out_dtype == PKV_BF16;
  a.w.window = window;
  a.w.sinks = sinks;
  a.w.max_context_len = max_context_len;
  a.w.box_log2 = p.bs_log2 < chl ? p.bs_log2 : chl;
  a.w.head_split = G > 8 ? 2 : 1;
  a.w.bits8 = codes;
  a.w.cluster = in_cluster(num_seqs, num_q_heads, num_kv_heads, parts);
  a.num_seqs = num_seqs;
  a.head_dim = head_dim;
  a.kv_dtype = kv_dtype;
  a.num_blocks = num_blocks;
  a.q_f32 = q_dtype == PKV_F32;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  return codes ? launch_decode_win_8bit(a) : launch_decode_win(a);
}

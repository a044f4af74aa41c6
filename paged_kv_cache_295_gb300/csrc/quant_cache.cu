// quantize_and_cache: the new tokens' K and V rows into an 8-bit paged cache
// that holds one scale per (block, KV head), and gather_cache: rows of a paged
// cache back as bf16 or f32 ("LLM inference tutorial" section 3.1 symmetric
// quantisation, 4.2 append_token and get_kv; "ToPG framework" section 3.3).
//
// Scale of one block and head (K and V apart), a = max |x| over the finite new
// values that fall into the block, qmax = 448 (E4M3) or 127 (INT8):
//   the call's first token in the block is at offset 0:
//     s = max(a / qmax, 2^-64)
//   else (the block holds older tokens with scale s0):
//     s = s0 2^k with the least k >= 0 such that a <= qmax s0 2^k
//     older codes c become round(c 2^-k)
//   code = round_half_even(x / s), saturating, the quotient an IEEE float32 one.
// Growth by powers of two keeps the error of repeated growth bounded: an E4M3
// code is rescaled exactly unless it becomes subnormal, and the INT8 rounding
// errors of successive growths are halved by each later one, so a value is
// never more than one step of its final scale off, however often its block grew.
#include "common.cuh"
#include "quant.cuh"

namespace pkv {
namespace {

constexpr int kQThreads = 256;
constexpr float kMinScale = 5.421010862427522e-20f;   // 2^-64

template <typename Q>
struct CodeRange;
template <>
struct CodeRange<FP8> {
  static constexpr float kMax = 448.f;
};
template <>
struct CodeRange<INT8> {
  static constexpr float kMax = 127.f;
};

struct QuantParams {
  const void* k_new;
  const void* v_new;
  const int32_t* query_start;    // [S + 1], or null: one token per sequence, row s
  const int32_t* block_tables;   // [S, max_blocks_per_seq]
  const int32_t* context_lens;   // [S], the new tokens included
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scales;               // [num_blocks, scale_stride]
  float* v_scales;
  int32_t* status;
  int64_t num_blocks;
  int64_t scale_stride;
  int32_t num_tokens;
  int32_t num_kv_heads;
  int32_t segs;                  // 16-element segments per row
  int32_t bs_log2;
  int32_t max_blocks_per_seq;
  int32_t max_query_len;
  int32_t head_groups;           // CTAs per block
};

// The new rows of one sequence: q0 .. q0 + n, at positions ctx - n .. ctx - 1.
struct Chunk {
  int32_t q0, n, ctx;
  bool bad;
};

__device__ __forceinline__ Chunk load_chunk(const QuantParams& p, int s) {
  Chunk c;
  c.ctx = __ldg(p.context_lens + s);
  if (p.query_start) {
    c.q0 = __ldg(p.query_start + s);
    const int32_t q1 = __ldg(p.query_start + s + 1);
    c.bad = c.q0 < 0 || q1 < c.q0 || q1 > p.num_tokens || q1 - c.q0 > p.max_query_len;
    c.n = q1 - c.q0;
  } else {   // a padded row has context 0
    c.q0 = s;
    c.n = c.ctx > 0 ? 1 : 0;
    c.bad = false;
  }
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.bs_log2;
  c.bad = c.bad || c.ctx < c.n || c.ctx > cap;
  return c;
}

// One team of T threads per (sequence, touched block, head, K or V); a CTA holds
// 256 / T teams.  Each thread takes 16-element segments of the new rows.
template <typename Src, typename Q, int T>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const QuantParams p) {
  constexpr int U = kQThreads / T;
  __shared__ float red[kQThreads / 32];
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.y;
  const int i = blockIdx.x / p.head_groups;   // touched block of the sequence
  const int team = threadIdx.x / T, t = threadIdx.x % T;
  const int unit = (blockIdx.x % p.head_groups) * U + team;   // head, then K | V
  const Chunk c = load_chunk(p, s);
  if (c.bad) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    return;
  }
  if (c.n == 0) return;
  const int first = c.ctx - c.n;
  const int lb = (first >> p.bs_log2) + i;
  if ((static_cast<int64_t>(lb) << p.bs_log2) >= c.ctx) return;
  const int bs = 1 << p.bs_log2;
  const int pos0 = max(first, lb << p.bs_log2), pos1 = min(c.ctx, (lb + 1) << p.bs_log2);
  const int off = pos0 & (bs - 1);
  const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + lb);
  if (blk < 0 || blk >= p.num_blocks) {   // the same for the whole CTA
    if (threadIdx.x == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
    return;
  }
  const bool live = unit < 2 * p.num_kv_heads;
  const int head = live ? unit >> 1 : 0;
  const bool is_v = unit & 1;
  const Src* src = static_cast<const Src*>(is_v ? p.v_new : p.k_new) +
                   (static_cast<int64_t>(c.q0 + pos0 - first) * p.num_kv_heads + head) *
                       (p.segs * 16);
  const int64_t src_row = static_cast<int64_t>(p.num_kv_heads) * p.segs * 16;
  const int items = live ? (pos1 - pos0) * p.segs : 0;

  float a = 0.f;
  for (int it = t; it < items; it += T) {
    float x[16];
    load16<Src>(src + (it / p.segs) * src_row + (it % p.segs) * 16, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float v = fabsf(x[e]);
      a = v <= 3.402823466e38f ? fmaxf(a, v) : a;   // finite values only
    }
  }
  float* sp = (is_v ? p.v_scales : p.k_scales) + blk * p.scale_stride + head;
  const float s0 = live && off > 0 ? *sp : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T / 32; ++w) a = fmaxf(a, red[team * (T / 32) + w]);
  } else {
    __syncwarp();
  }
  if (!live) return;
  constexpr float kQ = CodeRange<Q>::kMax;
  float sc, shrink = 1.f;
  if (off == 0 || !(s0 >= kMinScale) || s0 > 3.402823466e38f) {
    sc = fmaxf(__fdiv_rn(a, kQ), kMinScale);
  } else {
    sc = s0;
    while (a > kQ * sc) {
      sc *= 2.f;
      shrink *= 0.5f;
    }
  }
  if (t == 0) *sp = sc;
  uint4* cache = reinterpret_cast<uint4*>(is_v ? p.v_cache : p.k_cache) +
                 ((static_cast<int64_t>(blk) << p.bs_log2) * p.num_kv_heads + head) * p.segs;
  const int64_t row = static_cast<int64_t>(p.num_kv_heads) * p.segs;
  if (shrink < 1.f) {   // the scale grew: the block's older codes move to it
    for (int it = t; it < off * p.segs; it += T) {
      uint4* at = cache + (it / p.segs) * row + it % p.segs;
      float x[16];
      decode16<Q>(*at, x);
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = x[4 * k + e] * shrink;
        w[k] = quant4<Q>(q);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  for (int it = t; it < items; it += T)
    cache[(off + it / p.segs) * row + it % p.segs] =
        quant16<Src, Q>(src + (it / p.segs) * src_row + (it % p.segs) * 16, sc);
}

template <typename Src, typename Q, int T>
cudaError_t launch_quantize(QuantParams& p, int num_seqs, cudaStream_t st) {
  constexpr int U = kQThreads / T;
  p.head_groups = (2 * p.num_kv_heads + U - 1) / U;
  const int bs = 1 << p.bs_log2;
  const int64_t touched = (static_cast<int64_t>(p.max_query_len) + bs - 2) / bs + 1;
  const int64_t x = touched * p.head_groups;
  if (x > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(quantize_kernel<Src, Q, T>, dim3(static_cast<unsigned>(x), num_seqs),
                    dim3(kQThreads), 0, st, p);
}

template <typename Src, typename Q>
cudaError_t pick_team(QuantParams& p, int num_seqs, cudaStream_t st) {
  const int bs = 1 << p.bs_log2;
  const int64_t items = static_cast<int64_t>(p.max_query_len < bs ? p.max_query_len : bs) * p.segs;
  if (items <= 128) return launch_quantize<Src, Q, 32>(p, num_seqs, st);
  if (items <= 256) return launch_quantize<Src, Q, 64>(p, num_seqs, st);
  if (items <= 512) return launch_quantize<Src, Q, 128>(p, num_seqs, st);
  return launch_quantize<Src, Q, 256>(p, num_seqs, st);
}

// ---- read-back ---------------------------------------------------------------
struct GatherParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* row_start;     // [S + 1]
  const int32_t* first_pos;     // [S], or null: 0
  const float* k_scale;         // 8-bit caches
  const float* v_scale;
  void* k_out;                  // [num_rows, num_kv_heads, head_dim]
  void* v_out;
  int32_t* status;
  int64_t num_blocks;
  int64_t scale_stride;         // 0: one scale per head
  int32_t num_rows;
  int32_t max_rows;
  int32_t num_kv_heads;
  int32_t segs;                 // 16-element segments per row
  int32_t bs_log2;
  int32_t max_blocks_per_seq;
  int32_t tile_rows;            // rows per CTA
};

template <typename KV>
__device__ __forceinline__ void load_values16(const uint8_t* row, int seg, float* x) {
  constexpr int V = KV::kBytes;   // 16-byte vectors per segment
  const uint4* v = reinterpret_cast<const uint4*>(row) + seg * V;
#pragma unroll
  for (int i = 0; i < V; ++i) decode16<KV>(__ldg(v + i), x + i * KV::kPerVec);
}

__device__ __forceinline__ void store16(float* out, const float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(out)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* out, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// One CTA per (tile of a sequence's rows, sequence); a thread takes 16-element
// segments, K and V of the same place.
template <typename KV, typename Out>
__global__ void __launch_bounds__(kQThreads) gather_kernel(const GatherParams p) {
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.y;
  const int r0 = __ldg(p.row_start + s), r1 = __ldg(p.row_start + s + 1);
  const int64_t pos0 = p.first_pos ? __ldg(p.first_pos + s) : 0;
  const int n = r1 - r0;
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.bs_log2;
  if (r0 < 0 || n < 0 || r1 > p.num_rows || n > p.max_rows || pos0 < 0 || pos0 + n > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    return;
  }
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.tile_rows;
  if (tile >= n) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.tile_rows), n - tile));
  const int per_row = p.num_kv_heads * p.segs;
  const int32_t* bt = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
  for (int64_t it = threadIdx.x; it < static_cast<int64_t>(rows) * per_row; it += kQThreads) {
    const int r = static_cast<int>(it / per_row), hs = static_cast<int>(it % per_row);
    const int head = hs / p.segs;
    const int64_t pos = pos0 + tile + r;
    const int32_t blk = __ldg(bt + (pos >> p.bs_log2));
    float k[16], v[16];
    if (blk >= 0 && blk < p.num_blocks) {
      const int64_t slot = (static_cast<int64_t>(blk) << p.bs_log2) + (pos & ((1 << p.bs_log2) - 1));
      const int64_t row = slot * per_row * 16 * KV::kBytes;
      load_values16<KV>(p.k_cache + row, hs, k);
      load_values16<KV>(p.v_cache + row, hs, v);
      if (KV::kBytes == 1) {
        const int64_t at = p.scale_stride ? blk * p.scale_stride + head : head;
        const float ks = __ldg(p.k_scale + at), vs = __ldg(p.v_scale + at);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          k[e] *= ks;
          v[e] *= vs;
        }
      }
    } else {
      flag_status(p.status, PKV_DEV_BAD_BLOCK);
#pragma unroll
      for (int e = 0; e < 16; ++e) k[e] = v[e] = 0.f;
    }
    const int64_t o = ((r0 + tile + r) * per_row + hs) * 16;
    store16(static_cast<Out*>(p.k_out) + o, k);
    store16(static_cast<Out*>(p.v_out) + o, v);
  }
}

bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
int ilog2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status quantize_and_cache(
    const void* k_new, const void* v_new, const int32_t* query_start, const int32_t* block_tables,
    const int32_t* context_lens, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
    int32_t num_seqs, int32_t num_tokens, int32_t max_query_len, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int64_t num_blocks, int32_t max_blocks_per_seq,
    int64_t scale_stride, int32_t src_dtype, int32_t cache_dtype, int32_t* device_status,
    pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq <= 0 || scale_stride < num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (cache_dtype != PKV_FP8_E4M3 && cache_dtype != PKV_INT8) return PKV_ERR_UNSUPPORTED;
  if (src_dtype != PKV_F32 && src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (head_dim % 16 != 0 || !pow2(block_size) || block_size > 4096) return PKV_ERR_UNSUPPORTED;
  if (num_blocks > INT32_MAX || num_seqs > 65535 || num_kv_heads > 65535 || head_dim > 65536)
    return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_ERR_INVALID_ARG;
  if (max_query_len > num_tokens) return PKV_ERR_INVALID_ARG;
  if (!query_start && (max_query_len > 1 || num_tokens < num_seqs)) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_query_len == 0) return PKV_OK;
  if (!k_new || !v_new || !block_tables || !context_lens || !k_cache || !v_cache || !k_scales ||
      !v_scales)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(query_start) || !aligned4(block_tables) || !aligned4(context_lens) ||
      !aligned4(k_scales) || !aligned4(v_scales))
    return PKV_ERR_INVALID_ARG;
  QuantParams p{};
  p.k_new = k_new;
  p.v_new = v_new;
  p.query_start = query_start;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.status = device_status;
  p.num_blocks = num_blocks;
  p.scale_stride = scale_stride;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.segs = head_dim / 16;
  p.bs_log2 = ilog2(block_size);
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_query_len = max_query_len;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache_dtype == PKV_FP8_E4M3)
    e = src_dtype == PKV_F32 ? pick_team<float, FP8>(p, num_seqs, st)
                             : pick_team<__nv_bfloat16, FP8>(p, num_seqs, st);
  else
    e = src_dtype == PKV_F32 ? pick_team<float, INT8>(p, num_seqs, st)
                             : pick_team<__nv_bfloat16, INT8>(p, num_seqs, st);
  return cuda_status(e);
}

extern "C" pkv_status gather_cache(
    const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* row_start, const int32_t* first_pos, int32_t num_seqs, int32_t num_rows,
    int32_t max_rows, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int64_t num_blocks, int32_t max_blocks_per_seq, int32_t kv_dtype, const float* k_scale,
    const float* v_scale, int64_t scale_stride, int32_t out_dtype, void* k_out, void* v_out,
    int32_t* device_status, pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_rows < 0 || max_rows < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq <= 0 || max_rows > num_rows)
    return PKV_ERR_INVALID_ARG;
  const bool codes = kv_dtype == PKV_FP8_E4M3 || kv_dtype == PKV_INT8;
  if (!codes && kv_dtype != PKV_F32 && kv_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (head_dim % 16 != 0 || !pow2(block_size) || block_size > 4096) return PKV_ERR_UNSUPPORTED;
  if (num_blocks > INT32_MAX || num_seqs > 65535 || num_kv_heads > 65535 || head_dim > 65536)
    return PKV_ERR_UNSUPPORTED;
  if (codes && scale_stride != 0 && scale_stride < num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_rows == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !row_start || !k_out || !v_out ||
      (codes && (!k_scale || !v_scale)))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) ||
      !aligned4(block_tables) || !aligned4(row_start) || !aligned4(first_pos) ||
      !aligned4(k_scale) || !aligned4(v_scale))
    return PKV_ERR_INVALID_ARG;
  GatherParams p{};
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.row_start = row_start;
  p.first_pos = first_pos;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_out = k_out;
  p.v_out = v_out;
  p.status = device_status;
  p.num_blocks = num_blocks;
  p.scale_stride = codes ? scale_stride : 0;
  p.num_rows = num_rows;
  p.max_rows = max_rows;
  p.num_kv_heads = num_kv_heads;
  p.segs = head_dim / 16;
  p.bs_log2 = ilog2(block_size);
  p.max_blocks_per_seq = max_blocks_per_seq;
  const int per_row = num_kv_heads * p.segs;
  p.tile_rows = per_row >= 4 * kQThreads ? 1 : (4 * kQThreads) / per_row;
  const int64_t tiles = (static_cast<int64_t>(max_rows) + p.tile_rows - 1) / p.tile_rows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto launch = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(tiles), num_seqs), dim3(kQThreads), 0, st, p);
  };
  auto pick = [&](auto tag) {
    using KV = decltype(tag);
    return out_dtype == PKV_F32 ? launch(gather_kernel<KV, float>)
                                : launch(gather_kernel<KV, __nv_bfloat16>);
  };
  const cudaError_t e = kv_dtype == PKV_FP8_E4M3 ? pick(FP8{})
                        : kv_dtype == PKV_INT8   ? pick(INT8{})
                        : kv_dtype == PKV_BF16   ? pick(BF16{})
                                                 : pick(F32{});
  return cuda_status(e);
}

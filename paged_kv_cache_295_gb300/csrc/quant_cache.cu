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
//
// Both are bound by HBM: the new rows read once and their codes written (201 MB for 8,192
// tokens x 32 heads x 128 in bf16: 35.3 us, 29.7 at the copy rate), the codes read and the
// rows written (35.6 us against 31.9 for the same number of rows).  A call with one token
// per sequence is launch latency: 3 us.  Large blocks keep a team of up to 512 threads for one
// head's rows: the same append into blocks of 128 takes 44 us, one of 64 x 128 tokens x 8 heads
// into blocks of 256 18 (7.4 at the copy rate).
#include <type_traits>

#include "common.cuh"
#include "quant.cuh"

// Rows, codes and scales that an earlier kernel may have written are read past L1 (__ldcg):
// with programmatic launches a kernel's CTAs share an SM with the writer's, whose own
// loads may have left older lines there.

namespace pkv {
namespace {

constexpr int kGThreads = 256;
constexpr int kQWarps = 28;   // warps of the append per SM (72 registers; 32 would spill)
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

// 8 consecutive elements of a row, as loaded.  kHeld of them per thread stay in
// registers between the maximum and the codes.
template <typename Src>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  static constexpr int kHeld = 8;
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  // Elements 2i and 2i + 1, negated.
  __device__ __forceinline__ float2 neg2(int i) const {
    const uint32_t n = w[i] ^ 0x80008000u;
    return make_float2(bf16_lo(n), bf16_hi(n));
  }
  // The largest |x| so far as two bf16 halves (NaN stays), and as a float32's bits.
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
    __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162*>(&m);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t = __hmax2_nan(t, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
    return *reinterpret_cast<const uint32_t*>(&t);
  }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t m) {
    m &= 0x7FFF7FFFu;
    return max(m & 0xFFFFu, m >> 16) << 16;
  }
};
template <>
struct Vec8<float> {
  static constexpr int kHeld = 4;
  uint32_t w[8];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldcg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float2 neg2(int i) const {
    return make_float2(-__uint_as_float(w[2 * i]), -__uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t m) { return m; }
};

// x / s rounded to nearest, for two finite x given as -x, without a divide per
// element, by Markstein's theorem ("Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): with r = 1 / s rounded to nearest and q within
// one ulp of x / s, q - (q s - x) r, whose residual one fma gives exactly, is x / s
// rounded to nearest.  x r is within two ulps, so one step makes it faithful and a
// second one exact.  s >= 2^-64 keeps the residuals of every quotient that rounds to
// a non-zero code in the normal range; the sign of a zero x is kept.
__device__ __forceinline__ float2 quotient2(float2 neg_x, float2 s, float2 neg_r) {
  float2 q = __fmul2_rn(neg_x, neg_r);
  q = __ffma2_rn(__ffma2_rn(q, s, neg_x), neg_r, q);
  return __ffma2_rn(__ffma2_rn(q, s, neg_x), neg_r, q);
}

// Codes of 8 elements; FINITE: none is an infinity or NaN.
template <typename Src, typename Q, bool FINITE>
__device__ __forceinline__ uint2 codes8(const Vec8<Src>& v, float s, float r) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 n = v.neg2(2 * k + e);
      const float2 y = FINITE ? quotient2(n, make_float2(s, s), make_float2(-r, -r))
                              : make_float2(__fdiv_rn(-n.x, s), __fdiv_rn(-n.y, s));
      q[2 * e] = y.x;
      q[2 * e + 1] = y.y;
    }
    if constexpr (FINITE && std::is_same<Q, INT8>::value) {
      // |q| < 127.5: adding 1.5 * 2^23 leaves round-half-even(q) in the low byte
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(q[e] + 12582912.f);
      w[k] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    } else {
      w[k] = quant4<Q>(q);
    }
  }
  return make_uint2(w[0], w[1]);
}

// A team of T threads takes one (head, K or V) of one sequence's touched block
// at a time; a CTA (128 threads, or one larger team) walks a share of the block's
// 2 Hkv of them, so the lookups (context, table) are paid once.  Rows are read
// once, unless a block holds more than T * kHeld vectors (T = 512: block_size *
// head_dim above 32,768 for bf16): the rest is then read again, from L2.  Bound by
// HBM: 2 or 4 bytes read and 1 written per element.
template <int T>
constexpr int kQThreads = T > 128 ? T : 128;

template <typename Src, typename Q, int T>
__global__ void __launch_bounds__(kQThreads<T>, (kQWarps * 32) / kQThreads<T>)
    quantize_kernel(const QuantParams p) {
  constexpr int U = kQThreads<T> / T;
  constexpr int kHeld = Vec8<Src>::kHeld;
  __shared__ uint32_t red[2][kQThreads<T> / 32];
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.y;
  const int i = blockIdx.x / p.head_groups;   // touched block of the sequence
  const int team = threadIdx.x / T, t = threadIdx.x % T;
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
  const int pos0 = max(first, lb << p.bs_log2);
  const int pos1 = static_cast<int>(min(static_cast<int64_t>(c.ctx), (static_cast<int64_t>(lb) + 1) << p.bs_log2));
  const int off = pos0 & (bs - 1);
  const int32_t blk = __ldg(p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq + lb);
  const int vecs = p.segs * 2;   // 8-element vectors per row
  const int items = (pos1 - pos0) * vecs;
  const int units = 2 * p.num_kv_heads;
  const int64_t row = static_cast<int64_t>(p.num_kv_heads) * vecs;   // vectors per token
  const int64_t src0 = (static_cast<int64_t>(c.q0) + pos0 - first) * row;
  // this thread's vectors t, t + T, ...: offsets within a head's rows, -1 past the end
  int rel[kHeld];
  {
    int r = t / vecs, v = t - r * vecs;   // row and vector of the row, advanced by T vectors
    const int dr = T / vecs, dv = T - dr * vecs;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      rel[k] = t + k * T < items ? r * static_cast<int>(row) + v : -1;
      r += dr;
      v += dv;
      if (v >= vecs) {
        v -= vecs;
        ++r;
      }
    }
  }
  const bool whole = items >= kHeld * T;   // every thread holds kHeld vectors
  const int step = p.head_groups * U;
  auto head_of = [&](int unit) { return unit >= p.num_kv_heads ? unit - p.num_kv_heads : unit; };
  auto rows_of = [&](int unit) {   // K of every head, then V
    return static_cast<const Src*>(unit >= p.num_kv_heads ? p.v_new : p.k_new) +
           (src0 + head_of(unit) * vecs) * 8;
  };
  auto load = [&](Vec8<Src>(&v)[kHeld], int unit) {
    const Src* src = rows_of(unit < units ? unit : 0);
    if (whole && unit < units) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) v[k].load(src + static_cast<int64_t>(rel[k]) * 8);
    } else {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        v[k].zero();
        if (unit < units && rel[k] >= 0) v[k].load(src + static_cast<int64_t>(rel[k]) * 8);
      }
    }
  };
  Vec8<Src> held[kHeld];
  const int u_first = (blockIdx.x % p.head_groups) * U;
  load(held, u_first + team);
  if (blk < 0 || blk >= p.num_blocks) {   // the same for the whole CTA
    if (threadIdx.x == 0 && blockIdx.x % p.head_groups == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
    return;
  }
  int turn = 0;
  // the team's maximum; buf: one of red's halves, by turns
  auto team_max = [&](uint32_t x, uint32_t* buf) {
    x = __reduce_max_sync(T < 32 ? 0xFFFFu << (threadIdx.x & 16) : 0xffffffffu, x);
    if (T > 32) {
      if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < T / 32; ++w) x = max(x, buf[team * (T / 32) + w]);
    }
    return x;
  };
  auto work = [&](Vec8<Src>(&v)[kHeld], int unit) {
    const bool live = unit < units;
    const bool is_v = unit >= p.num_kv_heads;
    const int head = live ? head_of(unit) : 0;
    const Src* src = rows_of(live ? unit : 0);
    float* sp = (is_v ? p.v_scales : p.k_scales) + blk * p.scale_stride + head;
    const float s0 = live && off > 0 ? __ldcg(sp) : 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) m = v[k].top(m);
    if (live)
      for (int it = t + kHeld * T; it < items; it += T) {
        Vec8<Src> y;
        y.load(src + ((it / vecs) * row + it % vecs) * 8);
        m = y.top(m);
      }
    m = team_max(Vec8<Src>::top_bits(m), red[turn]);
    const bool finite = m < 0x7F800000u;
    // rare: the maximum of the finite values; every team of the CTA takes part
    if (T > 32 && U > 1 ? __syncthreads_or(!finite) : !finite) {
      uint32_t f = 0;
      for (int it = t; live && it < items; it += T) {
        Vec8<Src> y;
        y.load(src + ((it / vecs) * row + it % vecs) * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 n = y.neg2(e);
          const uint32_t b0 = __float_as_uint(n.x) & 0x7FFFFFFFu, b1 = __float_as_uint(n.y) & 0x7FFFFFFFu;
          if (b0 < 0x7F800000u) f = max(f, b0);
          if (b1 < 0x7F800000u) f = max(f, b1);
        }
      }
      m = team_max(f, red[turn ^ 1]);
      if (T > 32) __syncthreads();
    }
    turn ^= 1;
    if (T <= 32) __syncwarp(T < 32 ? 0xFFFFu << (threadIdx.x & 16) : 0xffffffffu);
    if (!live) return;   // (the team's reads of s0 come before its write below)
    const float a = __uint_as_float(m);
    constexpr float kQ = CodeRange<Q>::kMax;
    float sc, shrink = 1.f;
    if (off == 0 || !(s0 >= kMinScale) || s0 > 3.402823466e38f) {
      sc = fmaxf(__fdiv_rn(a, kQ), kMinScale);
    } else {
      sc = s0;
      while (a > kQ * sc) {   // ends: a is finite
        sc *= 2.f;
        shrink *= 0.5f;
      }
    }
    if (t == 0) *sp = sc;
    uint2* cache = reinterpret_cast<uint2*>(is_v ? p.v_cache : p.k_cache) +
                   (static_cast<int64_t>(blk) << p.bs_log2) * row + head * vecs;
    if (shrink < 1.f) {   // the scale grew: the block's older codes move to it
      uint4* old = reinterpret_cast<uint4*>(cache);
      for (int it = t; it < off * p.segs; it += T) {
        uint4* at = old + (it / p.segs) * (row / 2) + it % p.segs;
        float x[16];
        decode16<Q>(__ldcg(at), x);
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
    cache += off * row;
    if (finite) {
      const float r = __frcp_rn(sc);
      if (whole) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) cache[rel[k]] = codes8<Src, Q, true>(v[k], sc, r);
      } else {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
          if (rel[k] >= 0) cache[rel[k]] = codes8<Src, Q, true>(v[k], sc, r);
      }
      for (int it = t + kHeld * T; it < items; it += T) {
        Vec8<Src> y;
        y.load(src + ((it / vecs) * row + it % vecs) * 8);
        cache[(it / vecs) * row + it % vecs] = codes8<Src, Q, true>(y, sc, r);
      }
    } else {
      for (int it = t; it < items; it += T) {
        Vec8<Src> y;
        y.load(src + ((it / vecs) * row + it % vecs) * 8);
        cache[(it / vecs) * row + it % vecs] = codes8<Src, Q, false>(y, sc, 0.f);
      }
    }
  };
  for (int u = u_first; u < units; u += step) {   // uniform over the CTA
    work(held, u + team);
    load(held, u + step + team);
  }
}

template <typename Src, typename Q, int T>
cudaError_t launch_quantize(QuantParams& p, int num_seqs, cudaStream_t st) {
  constexpr int U = kQThreads<T> / T;
  const int bs = 1 << p.bs_log2;
  const int64_t touched = (static_cast<int64_t>(p.max_query_len) + bs - 2) / bs + 1;
  // CTAs per block: as many as make up to two whole waves, at least one.  A partial wave
  // costs its whole length: 8,192 tokens x 32 heads took 38.2 us with three CTAs per block
  // (1.5 waves) and take 34.6 with two or four; 64 x 128 tokens x 8 heads 16.9 with one
  // (half a wave) and 13.3 with two.
  const int64_t most = (2 * p.num_kv_heads + U - 1) / U;
  const int64_t waves =
      2 * (kQWarps * 32 / kQThreads<T>) * static_cast<int64_t>(device_sm_count()) / (touched * num_seqs);
  p.head_groups = static_cast<int32_t>(waves < 1 ? 1 : (waves < most ? waves : most));
  const int64_t x = touched * p.head_groups;
  if (x > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(quantize_kernel<Src, Q, T>, dim3(static_cast<unsigned>(x), num_seqs),
                    dim3(kQThreads<T>), 0, st, p);
}

template <typename Src, typename Q>
cudaError_t pick_team(QuantParams& p, int num_seqs, cudaStream_t st) {
  const int bs = 1 << p.bs_log2;
  const int64_t items = static_cast<int64_t>(p.max_query_len < bs ? p.max_query_len : bs) * p.segs * 2;
  constexpr int kHeld = Vec8<Src>::kHeld;
  if (items <= 16 * kHeld) return launch_quantize<Src, Q, 16>(p, num_seqs, st);
  if (items <= 32 * kHeld) return launch_quantize<Src, Q, 32>(p, num_seqs, st);
  if (items <= 64 * kHeld) return launch_quantize<Src, Q, 64>(p, num_seqs, st);
  if (items <= 128 * kHeld) return launch_quantize<Src, Q, 128>(p, num_seqs, st);
  if (items <= 256 * kHeld) return launch_quantize<Src, Q, 256>(p, num_seqs, st);
  return launch_quantize<Src, Q, 512>(p, num_seqs, st);
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

// E elements of a cache row, as loaded, and as values.
template <typename KV, int E>
struct Piece {
  static constexpr int kWords = E * KV::kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // Past L1, whose lines may be older than what the kernel before this one wrote.
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (kWords == 1) {
      w[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (kWords == 2) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void values(float scale, float* x) const {
    if constexpr (KV::kBytes == 4) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (KV::kBytes == 2) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        if constexpr (std::is_same<KV, FP8>::value) {
          const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w[i] & 0xFFFFu));
          const float2 b = e4m3x2_to_float2(static_cast<uint16_t>(w[i] >> 16));
          x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[4 * i + e] = static_cast<float>(static_cast<int8_t>((w[i] >> (8 * e)) & 0xFFu));
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] *= scale;
    }
  }
};

__device__ __forceinline__ void store_piece(float* out, const float* x) {
  *reinterpret_cast<float4*>(out) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_piece(__nv_bfloat16* out, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per (tile of a sequence's rows, sequence); a thread takes pieces of 16 output
// bytes (so that a warp's stores are whole lines; pieces of 16 elements, stored as two
// halves, took 39.5 us where these take 35), K and V of the same place, kGHeld at a
// time.  Bound by HBM: one byte read and two (bf16) or four written per element.
constexpr int kGHeld = 2;
constexpr int kGTile = 4;

template <typename KV, typename Out>
__global__ void __launch_bounds__(kGThreads) gather_kernel(const GatherParams p) {
  constexpr int E = 16 / sizeof(Out);
  grid_dependency_wait();
  allow_dependents();
  const int s = blockIdx.y;
  const int r0 = __ldg(p.row_start + s), r1 = __ldg(p.row_start + s + 1);
  const int64_t pos0 = p.first_pos ? __ldg(p.first_pos + s) : 0;
  const int64_t n = static_cast<int64_t>(r1) - r0;
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.bs_log2;
  if (r0 < 0 || n < 0 || r1 > p.num_rows || n > p.max_rows || pos0 < 0 || pos0 + n > cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    return;
  }
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * p.tile_rows;
  if (tile >= n) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.tile_rows), n - tile));
  const uint32_t per_head = p.segs * (16 / E), per_row = p.num_kv_heads * per_head;
  const int32_t* bt = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
  // this thread's place, row r and piece c of the row, and its step of kGThreads pieces
  const uint32_t dr = kGThreads / per_row, dc = kGThreads % per_row;
  int r = threadIdx.x / per_row;
  uint32_t c = threadIdx.x % per_row;
  while (r < rows) {
    Piece<KV, E> k[kGHeld], v[kGHeld];
    float ks[kGHeld], vs[kGHeld];
    int64_t out[kGHeld];
#pragma unroll
    for (int i = 0; i < kGHeld; ++i) {
      out[i] = -1;
      ks[i] = vs[i] = 0.f;
      k[i].zero();
      v[i].zero();
      if (r < rows) {
        out[i] = ((r0 + tile + r) * per_row + c) * E;
        const int64_t pos = pos0 + tile + r;
        const int32_t blk = __ldg(bt + (pos >> p.bs_log2));
        if (blk >= 0 && blk < p.num_blocks) {
          const int64_t slot =
              (static_cast<int64_t>(blk) << p.bs_log2) + (pos & ((1 << p.bs_log2) - 1));
          const int64_t at = (slot * per_row + c) * (E * KV::kBytes);
          k[i].load(p.k_cache + at);
          v[i].load(p.v_cache + at);
          if (KV::kBytes == 1) {
            const int64_t sc = blk * p.scale_stride + c / per_head;   // stride 0: per head
            ks[i] = __ldcg(p.k_scale + sc);
            vs[i] = __ldcg(p.v_scale + sc);
          }
        } else {
          flag_status(p.status, PKV_DEV_BAD_BLOCK);
        }
      }
      r += dr;
      c += dc;
      if (c >= per_row) {
        c -= per_row;
        ++r;
      }
    }
#pragma unroll
    for (int i = 0; i < kGHeld; ++i) {
      if (out[i] < 0) continue;
      float x[E];
      k[i].values(ks[i], x);
      store_piece(static_cast<Out*>(p.k_out) + out[i], x);
      v[i].values(vs[i], x);
      store_piece(static_cast<Out*>(p.v_out) + out[i], x);
    }
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
  if (static_cast<int64_t>(block_size) * num_kv_heads * (head_dim / 8) > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;   // places within a block are 32-bit
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (max_query_len > num_tokens) return PKV_ERR_INVALID_ARG;
  if (!query_start && (max_query_len > 1 || num_tokens < num_seqs)) return PKV_ERR_INVALID_ARG;
  if (max_query_len == 0) return PKV_OK;
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
  // a tile of about kGTile pieces per thread
  const int64_t per_row = static_cast<int64_t>(num_kv_heads) * p.segs * (out_dtype == PKV_F32 ? 4 : 2);
  p.tile_rows = per_row >= kGTile * kGThreads ? 1 : static_cast<int32_t>(kGTile * kGThreads / per_row);
  const int64_t tiles = (static_cast<int64_t>(max_rows) + p.tile_rows - 1) / p.tile_rows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto launch = [&](auto kern) {
    return launch_pdl(kern, dim3(static_cast<unsigned>(tiles), num_seqs), dim3(kGThreads), 0, st, p);
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

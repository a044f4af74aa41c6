// rotary_and_cache: rotary position embedding of q and k rows with one position axis or several, and
// the append of the turned k and of v to a paged cache, in one pass over the rows.
//
//   angle_i = pos[axis_i] inv_freq_i,   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin
//
// Angles.  A position times a float32 frequency is off by 2^-24 of the angle: 0.06 at position a
// million.  Here a frequency is what one position is worth in turns, as a 64-bit fraction, so
// position * turns modulo 2^64 is the angle modulo one turn (three integer multiplications, signed
// positions included).  Its cosine and sine are rounded almost correctly: an 8-bit code is that of
// the float32 result, and every unit that this is off by moves values across a border between codes.
//
// What bounds it: HBM.  Every row is read and written once; the angles of a token are computed
// once per CTA, into shared memory, and kept in registers over the rows of the token: a group of 64
// threads works on one token, thread = (pair of 16-byte segments in the row, row), so that the
// same frequencies serve all rows a thread meets.  V rows go through the same loop with no turn.  Three
// rows a thread are in flight, the first of them asked for before the angles are computed, and three CTAs
// an SM fit (two rows and four CTAs: 36.9 us for the first case below; four rows 44; one kind of row
// after another, without a choice per row, 40).
//
// Measured: 8,192 tokens of 32 + 8 heads x 128, bf16, three axes, turned k kept and appended 36.5 us
// (6.0 TB/s, 89 % of the copy rate); 8,191 tokens of 32 + 32 heads into an fp8 cache 63 us (5.3 TB/s,
// 79 %: the codes' arithmetic and its latency; 67 with the cache's type looked at per row and one segment's
// codes after the other's, 75 with a bounds check per element, 107 with a divide per element), into an int8
// one 69, into one of bf16 63 (6.4 TB/s); 8 tokens of 32 + 8 heads 2.0 us in a graph.
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "quant.cuh"
#include "ranges.cuh"

namespace pkv {
namespace {

constexpr int kRoThreads = 256;
constexpr int kRoGroup = 64;                        // threads on one token
constexpr int kRoTokens = kRoThreads / kRoGroup;    // tokens of a CTA
constexpr int kRoBatch = 3;                         // rows in flight per thread
constexpr int kRoCtas = 3;                          // CTAs of an SM: 85 registers

struct RotaryParams {
  const void *q, *k, *v;
  void *q_out, *k_out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  int32_t tokens, hq, hkv, dim, rot, axes;
  const uint64_t* turns;
  const int32_t* axis;
  const int32_t* pos;
  float scale;
  const int64_t* slots;
  void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  int64_t num_slots;
  int32_t kind;       // cache: 0 none, 1 the rows' own type, 2 FP8, 3 INT8
  int32_t adjacent;
  int32_t small_scale; // |scale| <= 2^29
  int32_t units;      // pairs of 16-byte segments in a row
  int32_t rows_per_y; // rows of a token that one CTA takes
  int32_t* status;
};

// cos and sin of a 64-bit fraction of a turn, each within 0.6 units of its last place: the nearest
// quarter turn is taken off exactly, the rest r (at most pi / 4) is a sum of two floats, and so are the
// leading terms, r and 1 - r^2 / 2; the others are the Taylor series' (to 2^-30 of the result).
__device__ __forceinline__ float2 cos_sin(uint64_t part) {
  const uint32_t quarter = static_cast<uint32_t>((part + (1ull << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(part - (static_cast<uint64_t>(quarter) << 62));   // |rest| <= 2^61
  // turns: 24 bits and the 24 below them
  const float hi = static_cast<float>(static_cast<int32_t>(rest >> 40)) * 5.9604644775390625e-8f;   // 2^-24
  const float lo = static_cast<float>(static_cast<int32_t>((rest >> 16) & 0xFFFFFF)) * 3.5527136788005009e-15f;
  const float t = hi + lo, t_lo = lo - (t - hi);
  constexpr float kTwoPi = 6.28318548202514648f, kTwoPiLo = -1.74845553146951715e-7f;   // 2 pi in two floats
  const float r = t * kTwoPi;
  const float r_lo = fmaf(t, kTwoPi, -r) + fmaf(t, kTwoPiLo, t_lo * kTwoPi);
  const float z = r * r;
  // sin r = r + (r_lo (1 - z / 2) + r z (-1/6 + z/120 - z^2/5040 + z^3/362880))
  const float ps = fmaf(fmaf(fmaf(z, 1.f / 362880.f, -1.f / 5040.f), z, 1.f / 120.f), z, -1.f / 6.f);
  const float s = r + fmaf(r * z, ps, fmaf(-0.5f * z, r_lo, r_lo));
  // cos r = 1 - h + (z^2 (1/24 - z/720 + z^2/40320 - z^3/3628800) - r r_lo - the part of z / 2 that h lacks)
  const float h = 0.5f * z, w = 1.f - h;
  const float pc = fmaf(fmaf(fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), z, -1.f / 720.f), z, 1.f / 24.f);
  const float left = ((1.f - w) - h) - fmaf(0.5f * r, r, -h);
  const float c = w + fmaf(z * z, pc, fmaf(-r, r_lo, left));
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

__device__ __forceinline__ float2 turn_of(const RotaryParams& p, int t, int i) {
  const int ax = p.axis ? p.axis[i] : 0;
  const int64_t at = ax >= 0 && ax < p.axes ? p.pos[static_cast<int64_t>(ax) * p.tokens + t] : 0;
  const float2 v = cos_sin(static_cast<uint64_t>(at) * p.turns[i]);
  return make_float2(v.x * p.scale, v.y * p.scale);
}

// 4 N bytes of a row.
template <int N>
struct alignas(4 * N) Words {
  uint32_t w[N];
};

template <typename Src, int N>
struct Seg {
  static constexpr int E = 4 * N / static_cast<int>(sizeof(Src));
  static __device__ __forceinline__ void unpack(const Words<N>& v, float* x) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(Src) == 2) {
        x[2 * i] = __uint_as_float(v.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
      } else {
        x[i] = __uint_as_float(v.w[i]);
      }
    }
  }
  static __device__ __forceinline__ Words<N> pack(const float* x) {
    Words<N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(Src) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        v.w[i] = __float_as_uint(x[i]);
      }
    }
    return v;
  }
};

// Codes of E float32 values x / s.
template <typename Q, int E>
__device__ __forceinline__ void codes(const float* x, float s, float neg_r, bool plain, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < (E + 3) / 4; ++i) {
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4 && 4 * i + e < E; e += 2) {
      float2 v;
      if (plain)
        v = quotient2(make_float2(-x[4 * i + e], -x[4 * i + e + 1]), make_float2(s, s), make_float2(neg_r, neg_r));
      else
        v = make_float2(__fdiv_rn(x[4 * i + e], s), __fdiv_rn(x[4 * i + e + 1], s));
      q[e] = v.x;
      q[e + 1] = v.y;
    }
    w[i] = quant4<Q>(q);
  }
}
template <int E>
__device__ __forceinline__ void put_codes(uint8_t* dst, const uint32_t* w) {
  if constexpr (E == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else if constexpr (E == 4)
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  else
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(w[0]);
}

// The largest |element| of two segments, as a float32's bits, at least; infinities and NaN are larger
// than any.
template <typename Src, int N>
__device__ __forceinline__ uint32_t top_of(const Words<N>& a, const Words<N>& b) {
  if constexpr (sizeof(Src) == 2) {
    __nv_bfloat162 t = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&a.w[0]));
#pragma unroll
    for (int i = 1; i < 2 * N; ++i)
      t = __hmax2_nan(t, __habs2(*reinterpret_cast<const __nv_bfloat162*>(i < N ? &a.w[i] : &b.w[i - N])));
    const uint32_t m = *reinterpret_cast<const uint32_t*>(&t) & 0x7FFF7FFFu;
    return max(m << 16, m & 0x7FFF0000u);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, max(a.w[i] & 0x7FFFFFFFu, b.w[i] & 0x7FFFFFFFu));
    return m;
  }
}

// A pair of segments to the cache, in its type: x at element `at` + a, y (where there is one) at `at` + b.
// `top`: top_of() the source's segments, which the turned ones exceed by |scale| sqrt(2) at most.
// Q: the codes' type; Src: the rows' own.
template <typename Src, typename Q, int N>
__device__ __forceinline__ void to_cache(const RotaryParams& p, void* cache, const float* scales, int head,
                                         int64_t at, int a, int b, bool has_b, uint32_t top, const float* x,
                                         const float* y) {
  using S = Seg<Src, N>;
  constexpr int E = S::E;
  if constexpr (std::is_same_v<Src, Q>) {
    Src* dst = static_cast<Src*>(cache) + at;
    *reinterpret_cast<Words<N>*>(dst + a) = S::pack(x);
    if (has_b) *reinterpret_cast<Words<N>*>(dst + b) = S::pack(y);
  } else {
    const float s = __ldg(scales + head);
    // quotient2's range: scales from 2^-64 to 2^64 and elements below 2^60 (|scale| up to 2^29, elements of
    // the source below 2^30)
    const bool plain = top < 0x4E800000u && p.small_scale && s >= 5.421010862427522e-20f && s <= 18446744073709551616.f;
    uint8_t* dst = static_cast<uint8_t*>(cache) + at;
    uint32_t wx[(E + 3) / 4], wy[(E + 3) / 4];   // both segments' quotients run side by side
    if (__builtin_expect(plain, 1)) {
      const float neg_r = -__frcp_rn(s);
      codes<Q, E>(x, s, neg_r, true, wx);
      codes<Q, E>(y, s, neg_r, true, wy);
    } else {
      codes<Q, E>(x, s, 0.f, false, wx);
      codes<Q, E>(y, s, 0.f, false, wy);
    }
    put_codes<E>(dst + a, wx);
    if (has_b) put_codes<E>(dst + b, wy);
  }
}

// Rows whose halves (or whose whole, with neighbouring pairs) are multiples of 4 N bytes.  Q: the cache's
// type where it is one of codes, else Src (a cache of the rows' own type, or none).
template <typename Src, bool ADJ, typename Q, int N>
__global__ void __launch_bounds__(kRoThreads, kRoCtas) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using S = Seg<Src, N>;
  constexpr int E = S::E;
  extern __shared__ float2 cs[];   // [kRoTokens][E][turned units]: (cos, sin)
  const int half = p.rot / 2, tid = threadIdx.x;
  // pairs of segments that turn
  const int tu = ADJ ? (p.rot + 2 * E - 1) / (2 * E) : half / E;
  const int t0 = blockIdx.x * kRoTokens;
  const int t = t0 + tid / kRoGroup, g = tid % kRoGroup;
  const int lanes = kRoGroup / p.units;   // rows at a time
  const int u = g % p.units, lane = g / p.units;
  // Segments: halves pair dim i with rot / 2 + i; the rest of a row goes in neighbouring segments.
  int a, b;
  if (!ADJ && u < tu) {
    a = u * E;
    b = half + u * E;
  } else {
    a = (ADJ ? 0 : p.rot) + (ADJ ? u : u - tu) * 2 * E;
    b = a + E;
  }
  const bool has_b = b < p.dim;
  const int rows = p.hq + (p.kind ? 2 : 1) * p.hkv;
  const int r1 = min(rows, (static_cast<int>(blockIdx.y) + 1) * p.rows_per_y);
  int r = t < p.tokens && lane < lanes ? blockIdx.y * p.rows_per_y + lane : r1;
  Words<N> va[kRoBatch], vb[kRoBatch];
  auto load = [&] {
#pragma unroll
    for (int n = 0; n < kRoBatch; ++n) {
      const int row = r + n * lanes;
      if (row >= r1) break;
      const Src* src = row < p.hq ? static_cast<const Src*>(p.q) + t * p.q_ts + row * p.q_hs
                       : row < p.hq + p.hkv
                           ? static_cast<const Src*>(p.k) + t * p.k_ts + (row - p.hq) * p.k_hs
                           : static_cast<const Src*>(p.v) + t * p.v_ts + (row - p.hq - p.hkv) * p.v_hs;
      va[n] = *reinterpret_cast<const Words<N>*>(src + a);
      vb[n] = has_b ? *reinterpret_cast<const Words<N>*>(src + b) : Words<N>{};
    }
  };
  grid_dependency_wait();
  allow_dependents();
  load();   // on their way while the angles are computed
  const int64_t slot = p.kind && t < p.tokens ? p.slots[t] : -1;
  // frequency f of a token lies at [f % E][f / E]: a thread's E of them in as many loads, without
  // conflicts between units.  The last unit of neighbouring pairs may be half past rotary_dim.
  for (int i = tid; i < kRoTokens * tu * E; i += kRoThreads) {
    const int tt = i / (tu * E), f = i - tt * (tu * E);
    float2 v = make_float2(1.f, 0.f);
    if (f < half && t0 + tt < p.tokens) v = turn_of(p, t0 + tt, f);
    cs[(tt * E + f % E) * tu + f / E] = v;
  }
  __syncthreads();
  float2 w[E];
#pragma unroll
  for (int e = 0; e < E; ++e)
    w[e] = u < tu ? cs[((tid / kRoGroup) * E + e) * tu + u] : make_float2(1.f, 0.f);
  const bool append = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && p.kind && blockIdx.y == 0 && g == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);

  while (r < r1) {
#pragma unroll
    for (int n = 0; n < kRoBatch; ++n) {
      const int row = r + n * lanes;
      if (row >= r1) break;
      const bool is_q = row < p.hq, is_v = row >= p.hq + p.hkv;
      const int head = is_q ? row : is_v ? row - p.hq - p.hkv : row - p.hq;
      float x[E], y[E];
      S::unpack(va[n], x);
      S::unpack(vb[n], y);
      if (!is_v && !ADJ && u < tu) {   // dims past rotary_dim keep infinities: no product with 0
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float x0 = x[e];
          x[e] = fmaf(x0, w[e].x, -(y[e] * w[e].y));
          y[e] = fmaf(y[e], w[e].x, x0 * w[e].y);
        }
      }
      if (!is_v && ADJ) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 wa = w[e / 2], wb = w[E / 2 + e / 2];
          const float x0 = x[e], y0 = y[e];
          if (a + e < p.rot) {
            x[e] = fmaf(x0, wa.x, -(x[e + 1] * wa.y));
            x[e + 1] = fmaf(x[e + 1], wa.x, x0 * wa.y);
          }
          if (b + e < p.rot) {
            y[e] = fmaf(y0, wb.x, -(y[e + 1] * wb.y));
            y[e + 1] = fmaf(y[e + 1], wb.x, y0 * wb.y);
          }
        }
      }
      Src* dst = nullptr;
      if (is_q)
        dst = static_cast<Src*>(p.q_out) + t * p.qo_ts + head * p.qo_hs;
      else if (!is_v && p.k_out)
        dst = static_cast<Src*>(p.k_out) + t * p.ko_ts + head * p.ko_hs;
      if (dst) {
        *reinterpret_cast<Words<N>*>(dst + a) = S::pack(x);
        if (has_b) *reinterpret_cast<Words<N>*>(dst + b) = S::pack(y);
      }
      if (!is_q && append) {
        const int64_t at = (slot * p.hkv + head) * p.dim;
        to_cache<Src, Q, N>(p, is_v ? p.v_cache : p.k_cache, is_v ? p.v_scale : p.k_scale, head, at, a, b, has_b,
                         std::is_same_v<Src, Q> ? 0u : top_of<Src, N>(va[n], vb[n]), x, y);
      }
    }
    r += lanes * kRoBatch;
    load();
  }
}

template <typename Src>
__device__ __forceinline__ float load1(const Src* x);
template <>
__device__ __forceinline__ float load1<float>(const float* x) { return *x; }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* x) { return __bfloat162float(*x); }
__device__ __forceinline__ void store1(float* d, float x) { *d = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* d, float x) { *d = __float2bfloat16_rn(x); }

template <typename Src>
__device__ __forceinline__ void to_cache1(const RotaryParams& p, bool is_v, int head, int64_t at, float y) {
  void* cache = is_v ? p.v_cache : p.k_cache;
  if (p.kind == 1) {
    store1(static_cast<Src*>(cache) + at, y);
    return;
  }
  const float x[4] = {__fdiv_rn(y, __ldg((is_v ? p.v_scale : p.k_scale) + head)), 0.f, 0.f, 0.f};
  static_cast<uint8_t*>(cache)[at] = static_cast<uint8_t>(p.kind == 2 ? quant4<FP8>(x) : quant4<INT8>(x));
}

// Any strides, alignment and dims: a thread takes one pair of elements, or one element past
// rotary_dim.
template <typename Src>
__global__ void __launch_bounds__(kRoThreads) rotary_any_kernel(const __grid_constant__ RotaryParams p) {
  grid_dependency_wait();
  allow_dependents();
  const int half = p.rot / 2, per_row = p.dim - half;
  const int rows = p.hq + (p.kind ? 2 : 1) * p.hkv;
  const int64_t total = static_cast<int64_t>(p.tokens) * rows * per_row;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kRoThreads) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kRoThreads) {
    const int u = static_cast<int>(i % per_row);
    const int64_t tr = i / per_row;
    const int row = static_cast<int>(tr % rows), t = static_cast<int>(tr / rows);
    const bool is_q = row < p.hq, is_v = row >= p.hq + p.hkv, pair = u < half;
    const int head = is_q ? row : is_v ? row - p.hq - p.hkv : row - p.hq;
    const int a = !pair ? u + half : p.adjacent ? 2 * u : u, b = p.adjacent ? a + 1 : a + half;
    const Src* src = is_q   ? static_cast<const Src*>(p.q) + t * p.q_ts + head * p.q_hs
                     : is_v ? static_cast<const Src*>(p.v) + t * p.v_ts + head * p.v_hs
                            : static_cast<const Src*>(p.k) + t * p.k_ts + head * p.k_hs;
    float x = load1(src + a), y = pair ? load1(src + b) : 0.f;
    if (pair && !is_v) {
      const float2 w = turn_of(p, t, u);
      const float x0 = x;
      x = fmaf(x0, w.x, -(y * w.y));
      y = fmaf(y, w.x, x0 * w.y);
    }
    Src* dst = nullptr;
    if (is_q)
      dst = static_cast<Src*>(p.q_out) + t * p.qo_ts + head * p.qo_hs;
    else if (!is_v && p.k_out)
      dst = static_cast<Src*>(p.k_out) + t * p.ko_ts + head * p.ko_hs;
    if (dst) {
      store1(dst + a, x);
      if (pair) store1(dst + b, y);
    }
    if (!is_q && p.kind) {
      const int64_t slot = p.slots[t];
      if (slot >= p.num_slots) {
        if (head == 0 && !is_v && u == 0) flag_status(p.status, PKV_DEV_BAD_SLOT);
      } else if (slot >= 0) {
        const int64_t at = (slot * p.hkv + head) * p.dim;
        to_cache1<Src>(p, is_v, head, at + a, x);
        if (pair) to_cache1<Src>(p, is_v, head, at + b, y);
      }
    }
  }
}

bool multiple(std::initializer_list<int64_t> xs, int64_t n) {
  for (int64_t x : xs)
    if (x % n != 0) return false;
  return true;
}

// Whether what a call writes overlaps something else that it reads or writes, but for rows turned in place.
bool outputs_overlap(const pkv_rotary_args& a, bool cached, bool codes) {
  const int64_t es = elem_bytes(a.src_dtype), T = a.num_tokens;
  auto rows = [&](const void* base, int32_t heads, int64_t ts, int64_t hs) {
    return Rows(base, T, heads, Wide{ts} * es, Wide{hs} * es, a.head_dim * es);
  };
  const Rows q = rows(a.q, a.num_q_heads, a.q_token_stride, a.q_head_stride);
  const Rows k = rows(a.k, a.num_kv_heads, a.k_token_stride, a.k_head_stride);
  const Rows v = rows(cached ? a.v : nullptr, a.num_kv_heads, a.v_token_stride, a.v_head_stride);
  const Rows qo = rows(a.q_out, a.num_q_heads, a.q_out_token_stride, a.q_out_head_stride);
  const Rows ko = rows(a.k_out, a.num_kv_heads, a.k_out_token_stride, a.k_out_head_stride);
  const int64_t cache = cached ? a.num_blocks * a.block_size * a.num_kv_heads * a.head_dim * elem_bytes(a.cache_dtype) : 0;
  const Rows kc(a.k_cache, cache), vc(a.v_cache, cache);
  if ((meet(qo, q) && !(qo == q)) || (meet(ko, k) && !(ko == k))) return true;
  if (meet(qo, k) || meet(qo, v) || meet(qo, ko) || meet(ko, q) || meet(ko, v) || meet(kc, vc)) return true;
  for (const Rows* c : {&kc, &vc})
    for (const Rows* x : {&q, &k, &v, &qo, &ko})
      if (meet(*c, *x)) return true;
  const int64_t half = a.rotary_dim / 2, scales = codes ? 4 * int64_t{a.num_kv_heads} : 0;
  for (const Rows& x : {Rows(a.turns, 8 * half), Rows(a.axis, 4 * half), Rows(a.positions, 4 * T * a.num_axes),
                        Rows(cached ? a.slot_mapping : nullptr, 8 * T), Rows(a.k_scale, scales),
                        Rows(a.v_scale, scales), Rows(a.device_status, 4)})
    for (const Rows* w : {&qo, &ko, &kc, &vc})
      if (meet(x, *w)) return true;
  return false;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status rotary_turns(const double* inv_freq, int32_t n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!inv_freq || !turns))) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return PKV_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    const double turn = inv_freq[i] / 6.283185307179586476925286766559;
    double part = turn - std::floor(turn);         // [0, 1]; 1 only by rounding
    part = std::ldexp(part, 64);
    turns[i] = part >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(part);
  }
  return PKV_OK;
}

extern "C" pkv_status rotary_and_cache(const pkv_rotary_args* args, pkv_stream_t stream) {
  using namespace pkv;
  if (!args) return PKV_ERR_INVALID_ARG;
  const pkv_rotary_args& a = *args;
  if (a.num_tokens < 0 || a.num_q_heads < 0 || a.num_kv_heads <= 0 || a.head_dim <= 0 ||
      a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 2 != 0 || a.num_axes <= 0 ||
      (a.adjacent != 0 && a.adjacent != 1) || !std::isfinite(a.scale))
    return PKV_ERR_INVALID_ARG;
  if (a.src_dtype != PKV_F32 && a.src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  const bool cached = a.k_cache != nullptr;
  int kind = 0;
  if (cached) {
    if (a.block_size <= 0 || a.num_blocks <= 0) return PKV_ERR_INVALID_ARG;
    kind = a.cache_dtype == a.src_dtype ? 1 : a.cache_dtype == PKV_FP8_E4M3 ? 2 : a.cache_dtype == PKV_INT8 ? 3 : 0;
    if (kind == 0) return PKV_ERR_UNSUPPORTED;
    if (a.num_blocks > INT64_MAX / a.block_size) return PKV_ERR_UNSUPPORTED;
  }
  if (a.num_q_heads > (1 << 20) || a.num_kv_heads > (1 << 20) || a.head_dim > (1 << 20))
    return PKV_ERR_UNSUPPORTED;
  if (cached && a.num_blocks * a.block_size > INT64_MAX / (int64_t{a.num_kv_heads} * a.head_dim * 4))
    return PKV_ERR_UNSUPPORTED;   // a cache's bytes
  if (a.num_tokens == 0) return PKV_OK;
  const unsigned es = static_cast<unsigned>(elem_bytes(a.src_dtype));
  if ((a.num_q_heads > 0 && (!a.q || !a.q_out)) || !a.k || (!cached && !a.k_out) ||
      (a.rotary_dim > 0 && (!a.turns || !a.positions)))
    return PKV_ERR_INVALID_ARG;
  if (cached && (!a.v || !a.v_cache || !a.slot_mapping)) return PKV_ERR_INVALID_ARG;
  if (kind >= 2 && (!a.k_scale || !a.v_scale)) return PKV_ERR_INVALID_ARG;
  for (const void* ptr : {a.q, a.k, a.v, static_cast<const void*>(a.q_out), static_cast<const void*>(a.k_out)})
    if (!aligned_to(ptr, es)) return PKV_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(a.axis), static_cast<const void*>(a.positions),
                          static_cast<const void*>(a.k_scale), static_cast<const void*>(a.v_scale),
                          static_cast<const void*>(a.device_status)})
    if (!aligned4(ptr)) return PKV_ERR_INVALID_ARG;
  if (!aligned_to(a.turns, 8) || !aligned_to(a.slot_mapping, 8)) return PKV_ERR_INVALID_ARG;
  if (cached && (!aligned16(a.k_cache) || !aligned16(a.v_cache))) return PKV_ERR_INVALID_ARG;
  if (outputs_overlap(a, cached, kind >= 2)) return PKV_ERR_INVALID_ARG;

  RotaryParams p{};
  p.q = a.q, p.k = a.k, p.v = a.v, p.q_out = a.q_out, p.k_out = a.k_out;
  p.q_ts = a.q_token_stride, p.q_hs = a.q_head_stride;
  p.k_ts = a.k_token_stride, p.k_hs = a.k_head_stride;
  p.v_ts = a.v_token_stride, p.v_hs = a.v_head_stride;
  p.qo_ts = a.q_out_token_stride, p.qo_hs = a.q_out_head_stride;
  p.ko_ts = a.k_out_token_stride, p.ko_hs = a.k_out_head_stride;
  p.tokens = a.num_tokens, p.hq = a.num_q_heads, p.hkv = a.num_kv_heads;
  p.dim = a.head_dim, p.rot = a.rotary_dim, p.axes = a.num_axes;
  p.turns = a.turns, p.axis = a.axis, p.pos = a.positions, p.scale = a.scale;
  p.slots = a.slot_mapping, p.k_cache = a.k_cache, p.v_cache = a.v_cache;
  p.k_scale = a.k_scale, p.v_scale = a.v_scale;
  p.num_slots = cached ? a.num_blocks * a.block_size : 0;
  p.kind = kind, p.adjacent = a.adjacent, p.status = a.device_status;
  p.small_scale = std::fabs(a.scale) <= 536870912.f;

  const int rows = p.hq + (cached ? 2 : 1) * p.hkv;
  const int half = p.rot / 2;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Loads of 4 n bytes: every segment of every row begins on such a boundary, and pairs of segments
  // turn together.  16 bytes where they will do; halves of 20 dims, as 40 of 80 have, take 8 (8,192 tokens
  // of 32 + 8 heads of 80, bf16: 26 us, 146 element by element, as what is left goes).
  for (int n = 4; n >= 2; n -= 2) {
    const int E = 4 * n / static_cast<int>(es);
    const unsigned bytes = 4u * n;
    const bool wide =
        aligned_to(p.q, bytes) && aligned_to(p.k, bytes) && (!cached || aligned_to(p.v, bytes)) &&
        aligned_to(p.q_out, bytes) && aligned_to(p.k_out, bytes) && p.dim % E == 0 &&
        (p.adjacent || half % E == 0) &&
        (p.hq == 0 || multiple({p.q_ts, p.q_hs, p.qo_ts, p.qo_hs}, E)) && multiple({p.k_ts, p.k_hs}, E) &&
        (!p.k_out || multiple({p.ko_ts, p.ko_hs}, E)) && (!cached || multiple({p.v_ts, p.v_hs}, E));
    p.units = p.adjacent ? (p.dim + 2 * E - 1) / (2 * E) : half / E + (p.dim - p.rot + 2 * E - 1) / (2 * E);
    if (!wide || p.units > kRoGroup) continue;
    const int lanes = kRoGroup / p.units, groups = (p.tokens + kRoTokens - 1) / kRoTokens;
    // few tokens: their rows are shared out among CTAs, no thread taking more than one at a time
    int ys = 1;
    const int most = (rows + lanes - 1) / lanes;
    while (ys < most && static_cast<int64_t>(groups) * ys < device_sm_count()) ++ys;
    p.rows_per_y = (most + ys - 1) / ys * lanes;
    ys = (rows + p.rows_per_y - 1) / p.rows_per_y;
    const int tu = p.adjacent ? (p.rot + 2 * E - 1) / (2 * E) : half / E;
    const size_t smem = sizeof(float2) * kRoTokens * tu * E;
    const dim3 grid(groups, ys);
    auto launch = [&](auto kernel) { return cuda_status(launch_pdl(kernel, grid, dim3(kRoThreads), smem, st, p)); };
    auto of = [&](auto src, auto adj, auto words) {
      using Src = decltype(src);
      constexpr bool A = decltype(adj)::value;
      constexpr int N = decltype(words)::value;
      return kind == 2   ? launch(rotary_kernel<Src, A, FP8, N>)
             : kind == 3 ? launch(rotary_kernel<Src, A, INT8, N>)
                         : launch(rotary_kernel<Src, A, Src, N>);
    };
    auto with = [&](auto words) {
      if (a.src_dtype == PKV_F32)
        return p.adjacent ? of(float{}, std::true_type{}, words) : of(float{}, std::false_type{}, words);
      return p.adjacent ? of(__nv_bfloat16{}, std::true_type{}, words) : of(__nv_bfloat16{}, std::false_type{}, words);
    };
    return n == 4 ? with(std::integral_constant<int, 4>{}) : with(std::integral_constant<int, 2>{});
  }
  const int64_t work = static_cast<int64_t>(p.tokens) * rows * (p.dim - half);
  const int64_t want = (work + kRoThreads - 1) / kRoThreads, cap = static_cast<int64_t>(device_sm_count()) * 16;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  return cuda_status(a.src_dtype == PKV_F32
                         ? launch_pdl(rotary_any_kernel<float>, grid, dim3(kRoThreads), 0, st, p)
                         : launch_pdl(rotary_any_kernel<__nv_bfloat16>, grid, dim3(kRoThreads), 0, st, p));
}

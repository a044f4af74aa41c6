// PagedAttention decode with a sliding window and sinks, and with one dequant
// scale per (block, KV head) on 8-bit caches (mma.sync m16n8k16, transposed).
//
// The query of a sequence of ctx tokens sees token t < ctx when
//   t >= ws = max(ctx - window, 0)  (the window; none given: ws = 0)   or
//   t <  sk = min(sinks, ws)        (the first tokens, which stay visible)
// and with K_t = ks[b(t)] * code_t, V_t = vs[b(t)] * code_t, b(t) the block:
//   out = sum_t p_t V_t / sum_t p_t,  p_t = 2^(c (q . K_t) - m),  c = scale log2(e).
//
// Work split, staging and operand layout are those of decode_mma2.cuh (one CTA
// per sequence x KV head x partition; each warp streams every NW-th chunk of CH
// tokens through its own TMA ring; heads ride in the mma's N = 8 columns).
// What differs:
//  * Only chunks with a visible token are walked: the sinks' chunks, then the
//    window's.  A partition is a run of that list, so hidden blocks are neither
//    read nor looked up (their table entries may be stale).
//  * The partition's boxes (a chunk's rows of one block) are looked up once into
//    shared memory: row of the cache and, for 8-bit caches, {c ks, vs, log2 vs}.
//    A box is at least 8 rows, so the eight token rows a lane group handles
//    share one entry and the scales cost one broadcast load per 8 x 8 scores.
//  * Tokens the query does not see score -inf and their rows are zeroed in
//    shared memory, so whatever those slots hold reaches no product.
//  * 8-bit caches: the running reference m follows max_t(c q.K_t + log2 vs), so
//    the weights w = p vs that enter the PV product stay below 2^15 whatever the
//    scales of the blocks; the sum takes p itself.
//  * The weights enter P V as 16-bit parts: for a float32 output three of bf16
//    (2^-24; the third costs 2 % of the time) or, on 8-bit caches (HL), two of
//    fp16 (2^-22); for a bf16 output two of bf16 (2^-16) or, on FP8 caches, two of
//    fp16.  INT8 caches with a bf16 output take one of fp16 (2^-11 of each weight,
//    where a code is off by half a step, 2^-8 or more of its value) and keep the
//    codes' offset of 1152 (see decode_mma2.cuh), else codes are widened exactly.
//
// Bound by HBM on long contexts, by what a CTA costs before its first tile (context length,
// table entry and scales, each load behind the one before: as long as about 110 tokens) on
// windows of about 1,000.  Measured: 32 sequences x 32 heads, fp8, contexts up to 4,096:
// 103 us (89 at the copy rate); 8 x 8 heads GQA-4, int8, 32K to 128K: 205 (189); 64 x 8
// heads GQA-8, bf16, window 1,024 and 4 sinks: 54 (40), at head_dim 64 36 (20) and at 256
// 105 (80); 4 x 8 heads, window 256: 7.
#pragma once

#include "decode_mma2.cuh"

namespace pkv {

// Smallest V scale (2^-80): keeps log2 vs, and p = w / vs <= 2^95 and its sums, finite.
constexpr float kMinVScale = 8.271806125530277e-25f;

struct WinParams {
  DecodeParams p;         // partition_tokens: a multiple of CH; out: unused
  void* out;              // [S, Hq, D] float32 or bf16
  int64_t scale_stride;   // 8-bit caches: floats between blocks' scales; 0: one scale per head
  int32_t out_bf16;
  int32_t window;         // 0: none
  int32_t sinks;
  int32_t max_context_len;
  int32_t box_log2;       // log2 of the rows per TMA box: min(block_size, CH)
  int32_t head_split;     // CTAs per KV head: 1, or 2 for groups of 9 to 16 heads
  int32_t bits8;          // CH of the cache type: 32 when set, else 16
  int32_t cluster;        // the partitions of a sequence and head are one cluster
};

// Up to 8 partitions of a sequence and KV head run as one thread-block cluster, which
// merges them through distributed shared memory: no scratch in HBM and no second kernel.
constexpr int kWinCluster = 8;

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {   // exited CTAs are not waited for
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// The same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// What one sequence's query sees, in chunks of CH tokens.
struct Visible {
  int ctx, ws, sk;       // see above
  int nsc, wc;           // sink chunks 0 .. nsc - 1; then chunks wc ..
  int nvc;               // chunks in all
};

__device__ __forceinline__ Visible visible_of(const WinParams& w, int ctx, int ch_log2) {
  Visible v;
  v.ctx = ctx;
  v.ws = w.window > 0 && ctx > w.window ? ctx - w.window : 0;
  v.sk = min(w.sinks, v.ws);
  const int ch = 1 << ch_log2;
  v.nsc = static_cast<int>((static_cast<uint32_t>(v.sk) + ch - 1) >> ch_log2);
  v.wc = max(v.ws >> ch_log2, v.nsc);
  v.nvc = v.nsc + static_cast<int>((static_cast<uint32_t>(ctx) + ch - 1) >> ch_log2) - v.wc;
  return v;
}

// The sequence's context, clamped to what the table and the call's bound cover.
__device__ __forceinline__ int win_context(const WinParams& w, int s, bool report) {
  int ctx = __ldg(w.p.context_lens + s);
  const long long by_table = static_cast<long long>(w.p.max_blocks_per_seq) << w.p.bs_log2;
  const int cap = static_cast<int>(min(by_table, static_cast<long long>(w.max_context_len)));
  if (ctx < 0 || ctx > cap) {
    if (report) flag_status(w.p.status, PKV_DEV_BAD_CONTEXT);
    ctx = ctx < 0 ? 0 : cap;
  }
  return ctx;
}

__device__ __forceinline__ void put_out(const WinParams& w, int64_t i, float x) {
  if (w.out_bf16)
    static_cast<__nv_bfloat16*>(w.out)[i] = __float2bfloat16_rn(x);
  else
    static_cast<float*>(w.out)[i] = x;
}

// Chunks of `ch` tokens a query of a context of up to max_ctx can see, at most.
inline int64_t max_visible_chunks(int32_t max_ctx, int32_t window, int32_t sinks, int ch) {
  const int64_t all = (static_cast<int64_t>(max_ctx) + ch - 1) / ch;
  if (window <= 0) return all;
  const int64_t sk = sinks < max_ctx ? sinks : max_ctx;
  const int64_t some = (sk + ch - 1) / ch + (static_cast<int64_t>(window) + ch - 2) / ch + 1;
  return some < all ? some : all;
}

struct WinLaunch {
  WinParams w;
  int num_seqs, head_dim, kv_dtype;
  int64_t num_blocks;
  bool q_f32;
  cudaStream_t stream;
};
pkv_status launch_decode_win(const WinLaunch& a);        // 16-bit caches
pkv_status launch_decode_win_8bit(const WinLaunch& a);   // FP8 and INT8 caches

template <typename KV, int D, int NW, int STAGES, int CH>
struct WinSmem {
  using Base = Mma2Smem<KV, D, NW, STAGES, CH>;
  static constexpr int kScratch = 1024;   // P^T: [64 rows][8 heads] fp16 at most
  static constexpr int kStageBytes = Base::kStageBytes;
  static constexpr int kBoxes = Base::kBoxes;
  static constexpr int kBoxBytes = Base::kBoxBytes;
  static constexpr int kWarpBytes = STAGES * kStageBytes + kScratch;
  static_assert(STAGES * kStageBytes >= 2 * 8 * (D + 3) * 4, "two combine areas fit a warp ring");
  static constexpr int kEntry = KV::kBytes == 1 ? 16 : 4;   // bytes per box entry
  static size_t bytes(int boxes) {
    return 1024 + static_cast<size_t>(NW) * kWarpBytes + static_cast<size_t>(boxes) * kEntry;
  }
};

template <typename KV, int D, bool QF32, bool HL, int NW, int STAGES, int CH>
__global__ void __launch_bounds__(NW * 32)
    paged_decode_win_kernel(const __grid_constant__ CUtensorMap tmap_k,
                            const __grid_constant__ CUtensorMap tmap_v,
                            const __grid_constant__ WinParams wp) {
  using SM = WinSmem<KV, D, NW, STAGES, CH>;
  constexpr bool F8 = KV::kBytes == 1;
  constexpr bool I8 = std::is_same<KV, INT8>::value;
  constexpr bool BIAS = I8 && !HL;   // INT8 codes enter the products as code + 1152
  static_assert(!F8 || D == 128, "the 8-bit path is built for head_dim 128");
  static_assert(I8 || HL, "one weight part only beside INT8 codes");
  constexpr int RT = CH / 16;
  constexpr int CHL = CH == 32 ? 5 : 4;
  static_assert(CH == 16 || (F8 && CH == 32), "16-token chunks, or 32 for 8-bit rows");
  constexpr int H = SM::kBoxes;
  constexpr int KSTEPS = D / 16;
  constexpr int MT = D / 16;
  const DecodeParams& p = wp.p;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[NW][STAGES];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);

  // shuffled, so that the compiler knows it uniform (window 1,024, 64 x 8 heads: 54.5 -> 53.5 us)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int s = blockIdx.z, part = blockIdx.y;
  // Groups of 9 to 16 heads run as two CTAs per KV head, the first with the
  // larger half; adjacent in the grid, so the second finds the rows in L2.
  const int hs = wp.head_split > 1 ? 1 : 0;
  const int g = static_cast<int>(blockIdx.x) >> hs;
  const int gall = p.num_q_heads / p.num_kv_heads;
  const int ghalf = hs ? (gall + 1) >> 1 : gall;
  const int which = hs ? static_cast<int>(blockIdx.x) & 1 : 0;
  const int G = which ? gall - ghalf : ghalf;
  const int hq0 = g * gall + which * ghalf;
  grid_dependency_wait();   // launched with launch_pdl: earlier work on the stream is done
  allow_dependents();

  const int ctx = win_context(wp, s, part == 0 && blockIdx.x == 0 && threadIdx.x == 0);
  const Visible vi = visible_of(wp, ctx, CHL);
  const int PC = p.partition_tokens >> CHL;   // chunks per partition
  const int nparts = (vi.nvc + PC - 1) / PC;
  if (part >= (nparts > 0 ? nparts : 1)) return;
  if (ctx == 0) {   // nothing to attend: output 0
    for (int i = threadIdx.x; i < G * D; i += NW * 32)
      put_out(wp, (static_cast<int64_t>(s) * p.num_q_heads + hq0) * D + i, 0.f);
    return;
  }
  const int c0 = part * PC;
  const int nchunks = min(PC, vi.nvc - c0);
  auto chunk_t0 = [&](int c) {   // first token of visible chunk c0 + c
    const int i = c0 + c;
    return (i < vi.nsc ? i : i - vi.nsc + vi.wc) << CHL;
  };
  auto sees = [&](int t) { return t < ctx && (t < vi.sk || t >= vi.ws); };

  // ---- box table: cache row (-1: nothing to copy) and scales ----------------------
  const int nbox = 1 << (CHL - wp.box_log2), box_rows = 1 << wp.box_log2;
  uint8_t* table = smem + NW * SM::kWarpBytes;
  int32_t* rows16 = reinterpret_cast<int32_t*>(table);
  float4* ents8 = reinterpret_cast<float4*>(table);   // {row bits, c ks, vs, log2 vs}
  {
    const int32_t* bt_row = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;
    for (int i = threadIdx.x; i < nchunks * nbox; i += NW * 32) {
      const int t = chunk_t0(i / nbox) + (i % nbox) * box_rows;
      int32_t row = -1;
      float4 e = make_float4(0.f, 0.f, 1.f, 0.f);
      if (t < ctx && (t < vi.sk || t + box_rows > vi.ws)) {
        const int32_t b = __ldg(bt_row + (t >> p.bs_log2));
        if (b < 0 || b >= p.num_blocks) {
          flag_status(p.status, PKV_DEV_BAD_BLOCK);
        } else {
          row = (b << p.bs_log2) + (t & ((1 << p.bs_log2) - 1));
          if (F8) {
            const int64_t at = static_cast<int64_t>(b) * wp.scale_stride + g;
            // past L1, whose line may be older than the append before this launch
            e.y = fabsf(p.qk_scale_log2) * __ldcg(p.k_scale + at);
            e.z = fmaxf(__ldcg(p.v_scale + at), kMinVScale);
            e.w = __log2f(e.z);
          }
        }
      }
      if (F8) {
        e.x = __int_as_float(row);
        ents8[i] = e;
      } else {
        rows16[i] = row;
      }
    }
  }
  auto box_row = [&](int i) { return F8 ? __float_as_int(ents8[i].x) : rows16[i]; };
  if (lane == 0) {
    for (int st = 0; st < STAGES; ++st) mbar_init(smem_u32(&bars[warp][st]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  fence_proxy_async();
  __syncthreads();

  float o[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
  float ps0 = 0.f, ps1 = 0.f;   // BIAS: sum of the weights as rounded to fp16

  uint8_t* ring = smem + warp * SM::kWarpBytes;
  uint8_t* scratch = ring + STAGES * SM::kStageBytes;
  const uint32_t ring_a = smem_u32(ring);
  const int my_n = warp < nchunks ? (nchunks - warp + NW - 1) / NW : 0;
  bool alive = true;

  // One box per lane: K (even lanes) or V (odd), 128-byte column hh, box bx of the chunk.
  auto issue = [&](int it) {
    if (it >= my_n) return;   // warp-uniform
    const int stage = it % STAGES;
    const uint32_t bar = smem_u32(&bars[warp][stage]);
    const int kv = lane & 1, hh = (lane >> 1) % H, bx = (lane >> 1) / H;
    const int row = bx < nbox ? box_row((warp + it * NW) * nbox + bx) : -1;
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, row >= 0));
    if (lane == 0) mbar_arrive_expect_tx(bar, n * box_rows * 128);
    __syncwarp();
    if (row >= 0)
      tma_load_3d(ring_a + stage * SM::kStageBytes + (kv * H + hh) * SM::kBoxBytes +
                      bx * box_rows * 128,
                  kv ? &tmap_v : &tmap_k, hh * (128 / KV::kBytes), g, row, bar);
  };

  const uint32_t k_swz0 = swz(gid, 2 * tig), k_swz1 = swz(gid, 2 * tig + 1);
  const uint32_t v_swz0 = swz(2 * tig, gid), v_swz1 = swz(2 * tig + 1, gid);
  // Tests of the bounded waits: CTA (0, 0, 0)'s first phase expects bytes that no copy brings.
  if (p.test_stall_bytes != 0 && threadIdx.x == 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0)
    mbar_expect_tx(smem_u32(&bars[0][0]), p.test_stall_bytes);
  __syncwarp();
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) issue(st);

  // ---- q^T as B fragments (decode_mma2.cuh: the dimension map of each cache type) --------
  // A negative logit scale is folded into q and a zero one raised to the smallest normal, so
  // that the factors below are positive and a masked -inf stays -inf under them.
  constexpr float kTiny = 1.17549435e-38f;
  const float qsign = p.qk_scale_log2 < 0.f ? -1.f : 1.f;
  uint32_t qb[KSTEPS][2];
  uint32_t qblo[QF32 ? KSTEPS : 1][2];
  float q_unscale = 1.f;
  float qsum0 = 0.f, qsum1 = 0.f;   // BIAS: 1152 * sum of q of heads 2tig, 2tig+1
  {
    const int64_t row = static_cast<int64_t>(s) * p.num_q_heads + hq0 + gid;
    const bool real = gid < G;
    auto qpair = [&](int ks, int half, float& x0, float& x1) {
      const int col = F8 ? 32 * tig + 4 * ks + 2 * half : 16 * ks + 8 * half + 2 * tig;
      x0 = x1 = 0.f;
      if (real) {
        if (QF32) {
          const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(p.q) + row * D + col);
          x0 = qsign * v.x;
          x1 = qsign * v.y;
        } else {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(
              static_cast<const __nv_bfloat16*>(p.q) + row * D + col);
          x0 = qsign * bf16_lo(v);
          x1 = qsign * bf16_hi(v);
        }
      }
    };
    float qmul = 1.f;
    if constexpr (F8) {
      float mx = 0.f;
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float x0, x1;
          qpair(ks, half, x0, x1);
          mx = fmaxf(mx, fmaxf(fabsf(x0), fabsf(x1)));
        }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      qmul = q_fp16_scale(mx, q_unscale);
    }
    float qs = 0.f;
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x0, x1;
        qpair(ks, half, x0, x1);
        uint32_t hi, lo;
        if (F8) {
          x0 *= qmul;   // exact: a power of two
          x1 *= qmul;
          hi = pack_f16(x0, x1);
          const __half2 hv = *reinterpret_cast<const __half2*>(&hi);
          const float y0 = x0 - __low2float(hv), y1 = x1 - __high2float(hv);
          lo = pack_f16(y0, y1);
          if (BIAS) {   // q as the products see it
            qs += __low2float(hv) + __high2float(hv);
            if (QF32) {
              const __half2 lv = *reinterpret_cast<const __half2*>(&lo);
              qs += __low2float(lv) + __high2float(lv);
            }
          }
        } else {
          hi = pack_bf16(x0, x1);
          lo = pack_bf16(x0 - bf16_lo(hi), x1 - bf16_hi(hi));
        }
        qb[ks][half] = hi;
        if (QF32) qblo[QF32 ? ks : 0][half] = lo;
      }
    }
    if (BIAS) {   // lanes 4 gid + (0 .. 3) hold head gid's quarters
      qs += __shfl_xor_sync(0xffffffffu, qs, 1);
      qs += __shfl_xor_sync(0xffffffffu, qs, 2);
      qsum0 = kI8Bias * __shfl_sync(0xffffffffu, qs, 8 * tig);
      qsum1 = kI8Bias * __shfl_sync(0xffffffffu, qs, 8 * tig + 4);
    }
  }
  const float sl2 = fmaxf(fabsf(p.qk_scale_log2), kTiny);   // 16-bit caches
  const bool third = !F8 && !wp.out_bf16;   // P in three bf16 parts

  for (int it = 0; it < my_n; ++it) {
    issue(it + STAGES - 1);
    const int stage = it % STAGES;
    const bool landed =
        __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][stage]), (it / STAGES) & 1));
    if (!landed) {
      if (lane == 0) flag_status(p.status, PKV_DEV_TIMEOUT);
      alive = false;
      for (int k = it + 1; k < min(my_n, it + STAGES); ++k)
        mbar_wait(smem_u32(&bars[warp][k % STAGES]), (k / STAGES) & 1);
      break;
    }
    const int c = warp + it * NW;
    const int t0 = chunk_t0(c);
    const int e0 = c * nbox;
    uint8_t* kb = ring + stage * SM::kStageBytes;
    uint8_t* vb = kb + H * SM::kBoxBytes;
    const bool partial = t0 + CH > ctx || (t0 < vi.ws && t0 + CH > vi.sk);   // warp-uniform
    const bool hole = __any_sync(0xffffffffu, partial || (lane < nbox && box_row(e0 + lane) < 0));
    if (hole) {   // rows not copied, and rows the query does not see, become zero
      for (int i = lane; i < CH * 8 * H * 2; i += 32) {
        const int r = (i >> 3) % CH;
        const int rest = i / (8 * CH);
        if (!sees(t0 + r) || box_row(e0 + (r >> wp.box_log2)) < 0) {
          uint8_t* base = (rest < H ? kb : vb) + (rest % H) * SM::kBoxBytes;
          *reinterpret_cast<uint4*>(base + r * 128 + ((i & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async();   // these generic writes precede the TMA refill of the stage
      __syncwarp();
    }
    const uint32_t kb_a = smem_u32(kb), vb_a = smem_u32(vb);

    // ---- S^T = K q^T: tokens 16rt + gid, 16rt + gid + 8 x heads 2tig, 2tig+1 --------
    float sacc[RT][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) sacc[rt][0] = sacc[rt][1] = sacc[rt][2] = sacc[rt][3] = 0.f;
    if (F8) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        uint32_t wa[8], wb[8];
        {
          const uint8_t* ka = kb + rt * 2048;
          const uint4 a0 = *reinterpret_cast<const uint4*>(ka + k_swz0);
          const uint4 a1 = *reinterpret_cast<const uint4*>(ka + k_swz1);
          const uint4 b0 = *reinterpret_cast<const uint4*>(ka + 1024 + k_swz0);
          const uint4 b1 = *reinterpret_cast<const uint4*>(ka + 1024 + k_swz1);
          wa[0] = a0.x; wa[1] = a0.y; wa[2] = a0.z; wa[3] = a0.w;
          wa[4] = a1.x; wa[5] = a1.y; wa[6] = a1.z; wa[7] = a1.w;
          wb[0] = b0.x; wb[1] = b0.y; wb[2] = b0.z; wb[3] = b0.w;
          wb[4] = b1.x; wb[5] = b1.y; wb[6] = b1.z; wb[7] = b1.w;
        }
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ++ks) {
          uint32_t a[4];
          if (I8 && HL) {
            s8x4_to_f16x2x2(wa[ks], a[0], a[2]);
            s8x4_to_f16x2x2(wb[ks], a[1], a[3]);
          } else {
            byte4_to_f16x2x2<KV>(wa[ks], a[0], a[2]);
            byte4_to_f16x2x2<KV>(wb[ks], a[1], a[3]);
          }
          mma_f16(sacc[rt], a, qb[ks][0], qb[ks][1]);
          if (QF32) mma_f16(sacc[rt], a, qblo[QF32 ? ks : 0][0], qblo[QF32 ? ks : 0][1]);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        const int i = lane >> 3, r = (i & 1) * 8 + (lane & 7);
        const int hh = (16 * ks) / 64;
        const int u = ((16 * ks) % 64) / 8 + (i >> 1);
        uint32_t a[4];
        ldsm_x4(kb_a + hh * SM::kBoxBytes + swz(r, u), a[0], a[1], a[2], a[3]);
        mma_bf16(sacc[0], a, qb[ks][0], qb[ks][1]);
        if (QF32) mma_bf16(sacc[0], a, qblo[QF32 ? ks : 0][0], qblo[QF32 ? ks : 0][1]);
      }
    }
    // ---- the chunk's largest logit (log2 units; 8-bit caches: + log2 vs) -------------------
    // Tokens the query does not see become -inf.  Rows 16rt + 8hf + gid share one box, hence
    // one logit factor fs and one V scale.
    float fs[RT][2], vsc[RT][2], mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (BIAS) {
          sacc[rt][2 * hf] -= qsum0;
          sacc[rt][2 * hf + 1] -= qsum1;
        }
        if (partial && !sees(t0 + 16 * rt + 8 * hf + gid))
          sacc[rt][2 * hf] = sacc[rt][2 * hf + 1] = -CUDART_INF_F;
        if (F8) {
          const float4 e = ents8[e0 + ((16 * rt + 8 * hf) >> wp.box_log2)];
          fs[rt][hf] = fmaxf(e.y * q_unscale, kTiny);
          vsc[rt][hf] = e.z;
          mx0 = fmaxf(mx0, fmaf(sacc[rt][2 * hf], fs[rt][hf], e.w));
          mx1 = fmaxf(mx1, fmaf(sacc[rt][2 * hf + 1], fs[rt][hf], e.w));
        } else {
          fs[rt][hf] = sl2;
          mx0 = fmaxf(mx0, sacc[rt][2 * hf]);
          mx1 = fmaxf(mx1, sacc[rt][2 * hf + 1]);
        }
      }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    if (!F8) {   // sl2 > 0: the max of the scaled logits
      mx0 *= sl2;
      mx1 *= sl2;
    }
    // Lazy rescale: the reference moves only when a weight would exceed 2^(kUp + kLazyLog2).
    // 8-bit caches set it kUp = 7 below the maximum, so that fp16 weights (at most 2^15) and
    // their lo parts stay clear of its smallest step.
    constexpr float kUp = F8 ? 7.f : 0.f;
    const bool up0 = mx0 > m0 + (kUp + kLazyLog2), up1 = mx1 > m1 + (kUp + kLazyLog2);
    if (__any_sync(0xffffffffu, up0 || up1)) {
      const float mn0 = up0 ? mx0 - kUp : m0, mn1 = up1 ? mx1 - kUp : m1;
      const float a0 = up0 ? fast_ex2(m0 - mn0) : 1.f;
      const float a1 = up1 ? fast_ex2(m1 - mn1) : 1.f;
      l0 *= a0;
      l1 *= a1;
      if (BIAS) {
        ps0 *= a0;
        ps1 *= a1;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= a0;
        o[mt][1] *= a1;
        o[mt][2] *= a0;
        o[mt][3] *= a1;
      }
      m0 = mn0;
      m1 = mn1;
    }
    // ---- weights to B fragments: scratch [token][8 heads], hi rows then lo rows -----------
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float p0 = fast_ex2(fmaf(sacc[rt][2 * hf], fs[rt][hf], -m0));
        float p1 = fast_ex2(fmaf(sacc[rt][2 * hf + 1], fs[rt][hf], -m1));
        l0 += p0;
        l1 += p1;
        if (F8) {
          p0 *= vsc[rt][hf];
          p1 *= vsc[rt][hf];
        }
        uint8_t* at = scratch + (16 * rt + 8 * hf + gid) * 16 + 4 * tig;
        const uint32_t hi = F8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
        *reinterpret_cast<uint32_t*>(at) = hi;
        float h0, h1;
        if (F8) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          h0 = f.x;
          h1 = f.y;
        } else {
          h0 = bf16_lo(hi);
          h1 = bf16_hi(hi);
        }
        if (BIAS) {
          ps0 += h0;
          ps1 += h1;
        }
        if (HL) {
          const uint32_t lo = F8 ? pack_f16(p0 - h0, p1 - h1) : pack_bf16(p0 - h0, p1 - h1);
          *reinterpret_cast<uint32_t*>(at + CH * 16) = lo;
          if (!F8 && third)
            *reinterpret_cast<uint32_t*>(at + 2 * CH * 16) =
                pack_bf16(p0 - h0 - bf16_lo(lo), p1 - h1 - bf16_hi(lo));
        }
      }
    }
    __syncwarp();
    uint32_t pb0[RT], pb1[RT], pl0[RT], pl1[RT];   // k-steps' hi and lo fragments
    uint32_t pt0 = 0, pt1 = 0;                     // 16-bit caches: the third part's
    {
      uint32_t r0, r1, r2, r3;
      ldsm_x4_t(smem_u32(scratch) + lane * 16, r0, r1, r2, r3);
      pb0[0] = r0;
      pb1[0] = r1;
      if constexpr (RT == 2) {
        pb0[RT - 1] = r2;
        pb1[RT - 1] = r3;
        if constexpr (HL) {
          ldsm_x4_t(smem_u32(scratch) + 512 + lane * 16, r0, r1, r2, r3);
          pl0[0] = r0;
          pl1[0] = r1;
          pl0[RT - 1] = r2;
          pl1[RT - 1] = r3;
        }
      } else {
        pl0[0] = r2;
        pl1[0] = r3;
        if (third) {
          ldsm_x4_t(smem_u32(scratch) + 512 + lane * 16, r0, r1, r2, r3);   // rows 32 .. 47
          pt0 = r0;
          pt1 = r1;
        }
      }
    }

    // ---- O^T += V^T w^T -----------------------------------------------------------
    if (F8) {
#pragma unroll
      for (int kk = 0; kk < RT; ++kk) {
        const uint8_t* va_row = vb + kk * 2048;
        const uint4 va = *reinterpret_cast<const uint4*>(va_row + v_swz0);
        const uint4 vv = *reinterpret_cast<const uint4*>(va_row + v_swz1);
        const uint4 vc = *reinterpret_cast<const uint4*>(va_row + 1024 + v_swz0);
        const uint4 vd = *reinterpret_cast<const uint4*>(va_row + 1024 + v_swz1);
        const uint32_t A[4] = {va.x, va.y, va.z, va.w}, B[4] = {vv.x, vv.y, vv.z, vv.w};
        const uint32_t Cw[4] = {vc.x, vc.y, vc.z, vc.w}, Dw[4] = {vd.x, vd.y, vd.z, vd.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t lo01 = __byte_perm(A[w], B[w], 0x5140);
          const uint32_t hi01 = __byte_perm(A[w], B[w], 0x7362);
          const uint32_t lo89 = __byte_perm(Cw[w], Dw[w], 0x5140);
          const uint32_t hi89 = __byte_perm(Cw[w], Dw[w], 0x7362);
          uint32_t aA[4], aB[4];
          if (I8 && HL) {
            s8x4_to_f16x2x2(lo01, aA[0], aA[1]);
            s8x4_to_f16x2x2(lo89, aA[2], aA[3]);
            s8x4_to_f16x2x2(hi01, aB[0], aB[1]);
            s8x4_to_f16x2x2(hi89, aB[2], aB[3]);
          } else {
            byte4_to_f16x2x2<KV>(lo01, aA[0], aA[1]);
            byte4_to_f16x2x2<KV>(lo89, aA[2], aA[3]);
            byte4_to_f16x2x2<KV>(hi01, aB[0], aB[1]);
            byte4_to_f16x2x2<KV>(hi89, aB[2], aB[3]);
          }
          mma_f16(o[2 * w], aA, pb0[kk], pb1[kk]);
          mma_f16(o[2 * w + 1], aB, pb0[kk], pb1[kk]);
          if (HL) {
            mma_f16(o[2 * w], aA, pl0[kk], pl1[kk]);
            mma_f16(o[2 * w + 1], aB, pl0[kk], pl1[kk]);
          }
        }
      }
    } else {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int i = lane >> 3, r = (i >> 1) * 8 + (lane & 7);
        const int hh = (16 * mt) / 64;
        const int u = ((16 * mt) % 64) / 8 + (i & 1);
        uint32_t a[4];
        ldsm_x4_t(vb_a + hh * SM::kBoxBytes + swz(r, u), a[0], a[1], a[2], a[3]);
        mma_bf16(o[mt], a, pb0[0], pb1[0]);
        mma_bf16(o[mt], a, pl0[0], pl1[0]);
        if (third) mma_bf16(o[mt], a, pt0, pt1);
      }
    }
    __syncwarp();   // every lane is done with this stage before it is refilled
  }

  // ---- warp epilogue: l over the 8 token-row lanes; rows into the idle ring ----------------
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, off);
    l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    if (BIAS) {
      ps0 += __shfl_xor_sync(0xffffffffu, ps0, off);
      ps1 += __shfl_xor_sync(0xffffffffu, ps1, off);
    }
  }
  if (!alive) {
    m0 = m1 = -CUDART_INF_F;
    l0 = l1 = 0.f;
  }
  __syncwarp();
  float* wres = reinterpret_cast<float*>(ring);   // [8][D] o, then m[8], l[8], ps[8]
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int h = 2 * tig + e;
    if (h < G) {
      const float back = BIAS ? kI8Bias * (e ? ps1 : ps0) : 0.f;   // the V codes' offset
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int d_lo = F8 ? 16 * gid + 2 * mt : 16 * mt + gid;
        const int d_hi = F8 ? 16 * gid + 2 * mt + 1 : 16 * mt + gid + 8;
        wres[h * D + d_lo] = alive ? o[mt][e] - back : 0.f;
        wres[h * D + d_hi] = alive ? o[mt][2 + e] - back : 0.f;
      }
      if (gid == 0) {
        wres[8 * D + h] = e ? m1 : m0;
        wres[8 * D + 8 + h] = e ? l1 : l0;
      }
    }
  }
  __syncthreads();

  const bool single = nparts == 1;
  // this partition's result for the cluster: [8][D] o, m[8], l[8], behind warp 0's own
  float* cres = reinterpret_cast<float*>(smem) + 8 * (D + 2);
  for (int i = threadIdx.x; i < G * D; i += NW * 32) {
    const int h = i / D, d = i % D;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w)
      M = fmaxf(M, reinterpret_cast<const float*>(smem + w * SM::kWarpBytes)[8 * D + h]);
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* r = reinterpret_cast<const float*>(smem + w * SM::kWarpBytes);
      const float cw = exp2f(r[8 * D + h] - M);
      L = fmaf(r[8 * D + 8 + h], cw, L);
      O = fmaf(r[h * D + d], cw, O);
    }
    const int64_t sh = static_cast<int64_t>(s) * p.num_q_heads + hq0 + h;
    if (single) {
      put_out(wp, sh * D + d, O / L);
    } else if (wp.cluster) {
      cres[i] = O;
      if (d == 0) {
        cres[8 * D + h] = M;
        cres[8 * D + 8 + h] = L;
      }
    } else {
      const int64_t pi = sh * p.max_parts + part;
      p.part_o[pi * D + d] = O;
      if (d == 0) {
        p.part_ml[pi * 2 + 0] = M;
        p.part_ml[pi * 2 + 1] = L;
      }
    }
  }
  if (single || !wp.cluster) return;
  // Every CTA of the cluster that has tokens merges a share of the outputs; the others
  // have left.  None leaves before all have read.
  cluster_arrive();
  cluster_wait();
  const uint32_t cres_a = smem_u32(cres);
  for (int i = part * (NW * 32) + static_cast<int>(threadIdx.x); i < G * D; i += nparts * NW * 32) {
    const int h = i / D;
    float m[kWinCluster], M = -CUDART_INF_F;
#pragma unroll
    for (int r = 0; r < kWinCluster; ++r) {
      m[r] = r < nparts ? cluster_ld(cluster_map(cres_a + 4 * (8 * D + h), r)) : -CUDART_INF_F;
      M = fmaxf(M, m[r]);
    }
    float L = 0.f, O = 0.f;
#pragma unroll
    for (int r = 0; r < kWinCluster; ++r) {
      if (r < nparts) {
        const float c = exp2f(m[r] - M);
        L = fmaf(cluster_ld(cluster_map(cres_a + 4 * (8 * D + 8 + h), r)), c, L);
        O = fmaf(cluster_ld(cluster_map(cres_a + 4 * i, r)), c, O);
      }
    }
    put_out(wp, (static_cast<int64_t>(s) * p.num_q_heads + hq0) * D + i, O / L);
  }
  cluster_arrive();
  cluster_wait();
}

// Merges the partitions' (m, l, o): one warp per (sequence, query head), as
// paged_decode_reduce_kernel, over the partitions that hold visible chunks.
template <int D>
__global__ void __launch_bounds__(32)
    paged_decode_win_reduce_kernel(const __grid_constant__ WinParams wp) {
  grid_dependency_wait();
  allow_dependents();
  const DecodeParams& p = wp.p;
  const int sh = blockIdx.x;
  const int lane = threadIdx.x;
  const int ctx = win_context(wp, sh / p.num_q_heads, false);
  const int chl = wp.bits8 ? 5 : 4;
  const int PC = p.partition_tokens >> chl;
  const int nparts = (visible_of(wp, ctx, chl).nvc + PC - 1) / PC;
  if (nparts <= 1) return;   // written by the main kernel
  const float* ml = p.part_ml + static_cast<int64_t>(sh) * p.max_parts * 2;
  const float* po = p.part_o + static_cast<int64_t>(sh) * p.max_parts * D;
  float M = -CUDART_INF_F;
  for (int i = lane; i < nparts; i += 32) M = fmaxf(M, ml[2 * i]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float L = 0.f;
  for (int i = lane; i < nparts; i += 32) L = fmaf(ml[2 * i + 1], exp2f(ml[2 * i] - M), L);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  const float invL = 1.f / L;
  constexpr int V = D / 32;
  constexpr int U = 8;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int i0 = 0; i0 < nparts; i0 += U) {
    float x[U][V], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      const bool in = i < nparts;
      w[u] = in ? ml[2 * i] : -CUDART_INF_F;
#pragma unroll
      for (int v = 0; v < V; ++v) x[u][v] = in ? po[static_cast<int64_t>(i) * D + lane + 32 * v] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float wu = exp2f(w[u] - M);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(x[u][v], wu, acc[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    put_out(wp, static_cast<int64_t>(sh) * D + lane + 32 * v, acc[v] * invL);
}

}  // namespace pkv

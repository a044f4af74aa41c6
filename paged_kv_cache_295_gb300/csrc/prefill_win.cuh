// Paged prefill attention with a sliding window and sinks, one dequant scale per
// (block, KV head) on 8-bit caches, and f32 or bf16 output (tcgen05 + TMEM; bf16 q,
// bf16, FP8-E4M3 or INT8 caches, head_dim 128).
//
// The query at position p sees key t <= p when t > p - window or t < sinks, and
//   out = sum_t p_t V_t / sum_t p_t,  p_t = 2^(c (q . K_t) - m),  c = scale log2(e),
// K_t = ks[b(t)] code_t and V_t = vs[b(t)] code_t on 8-bit caches.
//
// Work split as in prefill_tc.cuh: one CTA per (pair of query tiles A and B, KV
// head, sequence); a query tile is 128 rows (TQ = 128 / G tokens x G heads); keys
// come in tiles of 64.  Per key tile and query tile
//   S_t  = Q_t K^T   M=128 N=64  K=128   A = Q_t (smem), B = K tile (smem)
//   O_t += P_t V     M=128 N=128 K=64    A = P_t (TMEM), B = V tile (smem)
// TMEM, per query tile: P in 64 columns (hi, then lo; or one value in 32), S in 64, O in
// 128.  With P apart from S, the next key tile's QK runs while this one's softmax is still at
// its exponentials, and with P out of shared memory the softmax stores it in two instructions.
//
// What bounds it (clock64 trace with one weight part, two query tiles of 128 rows, steady
// state): the chain of a key tile in the softmax warps - look at the barriers (over 100 cycles
// each, so two are asked together), S load 110, maximum 260, exponentials 500, P store 200 to
// 600 - next to the MMAs, which hold both issuers for 1,200 cycles a key tile; and, on 8-bit
// caches, instruction fetch: the roles' loops together overrun the instruction cache.  So: the
// issuers' code is uniform (pw_elect); a mask is built only for tiles that cut some row of the
// warp; 8-bit tiles are widened by four warps of their own.  A key tile takes 1,050 ns on bf16
// caches, where its products alone need 1,000, and on 8-bit ones 1,120 to 1,130 with a bf16 output
// (667) and 1,260 to 1,350 with a float32 one (1,000).
//
// bf16 caches carry P as two bf16 parts (2^-16 of each weight) whatever the output's type: a bf16
// output is the float32 one rounded.  One part would be off by 2^-8 of each weight, which is
// relative to sum p |v| and not to the output: 1.4 times the error against 64 bits on normal
// values, without bound where they cancel.  It would take 123 us for the ragged chunks below.
//
// 8-bit caches: the running reference m follows max(logit + log2 vs), so the weights
// w = p vs that enter P V stay below 2^15 whatever the blocks' scales; l sums p itself.
// Each row of q is scaled by a power of two into fp16's range.  A float32 output takes
// the weights as two fp16 parts (2^-22), a bf16 one as one (2^-11 of each weight, where the codes
// themselves are off by up to 2^-4 (E4M3) or half a step (INT8) of their values).  Codes are
// widened to fp16 exactly.
//
// Measured, chunks of 512 tokens at contexts up to 4,096: 16 x 32 heads, bf16, window 1,024,
// f32 output 199 us (607 TFLOP/s); 16 x 8 heads GQA-4, fp8, no window, bf16 output 282 (927
// TFLOP/s), f32 output 336; the same in int8 292 and 349.  Three ragged chunks of up to 700
// tokens, 8 heads GQA-8, window 4,096, bf16 output: 147 (858 TFLOP/s).  Every CTA has about
// 10 us of setup, Q, first copies and epilogue besides its key tiles, of which a window leaves few.
//
// Every wait is bounded (2 s) and gives up when another role has given up; the copies in
// flight are then waited for, and TMEM is released before the CTA exits.
#pragma once

#include "prefill_tc.cuh"

namespace pkv {

constexpr int kPwThreads8 = 512;   // 8-bit caches: four widening warps more

struct PrefillWinParams {
  PrefillParams p;          // out: unused
  void* out;                // [T, Hq, D], f32 or bf16
  int64_t scale_stride;     // 8-bit caches: floats between blocks' scales; 0: one per head
  int32_t out_bf16;
  int32_t window;           // 0: none
  int32_t sinks;
};

// The key tiles a CTA walks: the sinks' tiles, then those from its first query's
// window on.  Tile B skips the entries between the sinks and its own first window.
struct PfList {
  int ns;        // entries 0 .. ns - 1 are key tiles 0 .. ns - 1
  int base;      // entry j >= ns is key tile j - ns + base
  int low;       // first key of tile A's first window: older keys are hidden (but sinks)
  int skip0, nskip;   // tile B leaves out entries skip0 .. skip0 + nskip - 1
  __device__ __forceinline__ int key0(int j) const { return (j < ns ? j : j - ns + base) * kPfKeys; }
  __device__ __forceinline__ bool skips(int t, int j) const {
    return t == 1 && j >= skip0 && j < skip0 + nskip;
  }
  // How many entries query tile t has worked through before entry j.
  __device__ __forceinline__ int count(int t, int j) const {
    return t == 1 && j >= skip0 + nskip ? j - nskip : j;
  }
};

// 8-bit caches: what 8 consecutive keys of a stage share.
struct PfScale {
  float kf;    // K scale * |logit scale| * log2(e)
  float vs;    // V scale
  float lv;    // log2 vs
  float pad;
};
// Smallest V scale (2^-80): keeps log2 vs, and p = w / vs <= 2^95, finite.
constexpr float kPfMinVScale = 8.271806125530277e-25f;

struct PwLayout {
  // [Q_A][Q_B] 32 KB each (two halves of 64 dims); [8-bit only: raw tiles, K x4 then
  // V x4, 8 KB each]; [stages: K 16 KB, V 16 KB]
  static constexpr int kQHalf = kPfRows * 128;
  static constexpr int kQ = 2 * kQHalf;
  __host__ __device__ static constexpr int raw() { return 2 * kQ; }
  __host__ __device__ static constexpr int ring(bool codes) {
    return raw() + (codes ? PfLayout::kRawBytes : 0);
  }
  static constexpr size_t bytes(int stages, bool codes) {
    return 1024 + static_cast<size_t>(ring(codes)) + static_cast<size_t>(stages) * PfLayout::kStage;
  }
};

// Bounded wait that gives up once any role of the CTA has; the timer is read only
// when the phase is not complete at the first look.
__device__ __forceinline__ bool pw_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok = 0;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if ((it & 15u) == 0) {
      const uint64_t now = global_ns();
      if (it == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The same for a whole warp.
__device__ __forceinline__ bool pw_wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, pw_wait(bar, parity, abort_flag));
}

// Whether two phases are complete, asked together: a look at a barrier takes over 100 cycles,
// however long ago its phase completed.
__device__ __forceinline__ bool pw_test2(uint32_t bar_a, uint32_t par_a, uint32_t bar_b, uint32_t par_b) {
  uint32_t a, b;
  asm volatile(
      "{\n .reg .pred p, q;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%2], %3;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 q, [%4], %5;\n"
      " selp.u32 %0, 1, 0, p;\n selp.u32 %1, 1, 0, q;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(bar_a), "r"(par_a), "r"(bar_b), "r"(par_b)
      : "memory");
  return (a & b) != 0;
}

// 32 registers to 32 TMEM columns of this warp's lanes, without the wait.
__device__ __forceinline__ void pw_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void pw_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// One lane of the warp, the same each time; the compiler knows its code uniform, with `warp`,
// the TMEM base and the lengths shuffled, and keeps descriptors and barriers in uniform
// registers: the three measured cases take 196, 146 and 285 us, with `lane == 0` 202, 157 and 302.
__device__ __forceinline__ bool pw_elect() {
  uint32_t e = 0;
  asm volatile("{\n .reg .b32 x;\n .reg .pred p;\n elect.sync x|p, 0xffffffff;\n @p mov.s32 %0, 1;\n}\n"
               : "+r"(e));
  return e != 0;
}
// Bits lo .. of a 64-key mask below key `n` of the tile.
__device__ __forceinline__ uint64_t pw_below(int n) {
  return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1ull);
}

// KIND: 0 bf16 cache; 1 FP8-E4M3 codes; 2 INT8 codes.  LO: the weights are two 16-bit parts.
template <int STAGES, int KIND, bool LO>
__global__ void __launch_bounds__(KIND == 0 ? kPfThreads : kPwThreads8, 1)
    paged_prefill_win_kernel(const __grid_constant__ CUtensorMap tmap_k,
                             const __grid_constant__ CUtensorMap tmap_v,
                             const __grid_constant__ PrefillWinParams wp) {
  using LY = PwLayout;
  constexpr int kKVHalf = PfLayout::kKVHalf, kStage = PfLayout::kStage;
  constexpr int kRawTile = PfLayout::kRawTile;
  constexpr bool C8 = KIND != 0;
  constexpr bool I8 = KIND == 2;
  constexpr int kThreads = C8 ? kPwThreads8 : kPfThreads;
  constexpr int kRing = LY::ring(C8);
  const PrefillParams& p = wp.p;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int TQ = p.tile_tokens;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[STAGES], full_v[STAGES], empty[STAGES];
  __shared__ __align__(8) uint64_t s_full[2], s_free[2], q_ready[2], p_full[2], o_done[2], drain[2];
  __shared__ __align__(8) uint64_t raw_full[2][kPfRawBufs], raw_free[2][kPfRawBufs];   // [K | V]
  __shared__ uint64_t key_mask[STAGES];   // per stage: keys with cache data that some query sees
  __shared__ uint64_t raw_mask[C8 ? kPfRawBufs : 1];
  __shared__ __align__(16) PfScale key_scale[C8 ? STAGES : 1][8];         // per 8 keys of a stage
  __shared__ __align__(16) PfScale raw_scale[C8 ? kPfRawBufs : 1][8];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, seq_sh;
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sma = smem_u32(sm);
  volatile int* abort_flag = &abort_sh;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == kThreads - 1) {   // while the others read the lengths
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(smem_u32(&full[st]), C8 ? 2 : 1);     // K in the stage, key mask and scales
      mbar_init(smem_u32(&full_v[st]), C8 ? 2 : 1);   // V in the stage
      mbar_init(smem_u32(&empty[st]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&s_free[t]), 4);
      mbar_init(smem_u32(&q_ready[t]), 4);
      mbar_init(smem_u32(&p_full[t]), 4);
      mbar_init(smem_u32(&o_done[t]), 1);
      mbar_init(smem_u32(&drain[t]), 1);
    }
    for (int i = 0; i < 2 * kPfRawBufs; ++i) {
      mbar_init(smem_u32(&raw_full[i / kPfRawBufs][i % kPfRawBufs]), 1);
      mbar_init(smem_u32(&raw_free[i / kPfRawBufs][i % kPfRawBufs]), 2);
    }
    if (p.test_stall_bytes != 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0)
      mbar_expect_tx(smem_u32(&full_v[0]), p.test_stall_bytes);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  // Work order (prefill_tc.cuh): KV heads fastest, then the pairs of a sequence, latest
  // first, then the sequences by context length, longest first.  The batch's lengths
  // and starts are read in one round trip.
  const uint64_t lin = blockIdx.x + static_cast<uint64_t>(gridDim.x) *
                                        (blockIdx.y + static_cast<uint64_t>(gridDim.y) * blockIdx.z);
  const int g = static_cast<int>(lin % gridDim.y);
  const uint64_t unit = lin / gridDim.y;
  const int pair = static_cast<int>(gridDim.x - 1 - unit % gridDim.x);
  const int rank = static_cast<int>(unit / gridDim.x);   // < gridDim.z
  int s = rank, q0, q1, ctx;
  if (gridDim.z <= kPfRankSeqs) {
    const int ns = static_cast<int>(gridDim.z);
    int* ctx_sh = reinterpret_cast<int*>(sm);   // Q's room, before Q is there
    int* start_sh = ctx_sh + kPfRankSeqs;
    int c = 0;
    if (tid < ns) ctx_sh[tid] = c = __ldg(p.context_lens + tid);
    if (tid <= ns) start_sh[tid] = __ldg(p.query_start + tid);
    if (tid == 0) seq_sh = rank;   // kept if no sequence claims the rank
    __syncthreads();
    if (tid < ns) {
      int r = 0;
      for (int i = 0; i < ns; ++i) {
        const int ci = ctx_sh[i];
        r += (ci > c || (ci == c && i < tid)) ? 1 : 0;
      }
      if (r == rank) seq_sh = tid;   // ranks are distinct: one writer
    }
    __syncthreads();
    s = seq_sh;
    q0 = start_sh[s];
    q1 = start_sh[s + 1];
    ctx = ctx_sh[s];
  } else {
    q0 = __ldg(p.query_start + s);
    q1 = __ldg(p.query_start + s + 1);
    ctx = __ldg(p.context_lens + s);
  }
  s = __shfl_sync(0xffffffffu, s, 0);
  q0 = __shfl_sync(0xffffffffu, q0, 0);
  q1 = __shfl_sync(0xffffffffu, q1, 0);
  ctx = __shfl_sync(0xffffffffu, ctx, 0);
  if (q0 < 0 || q1 < q0 || q1 > p.num_tokens) {   // rows outside q / out: touch nothing
    if (pair == 0 && g == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    return;
  }
  const int n = q1 - q0;
  if (pair == 0 && tid == 0 && n > 2 * static_cast<int>(gridDim.x) * TQ)
    flag_status(p.status, PKV_DEV_BAD_CONTEXT);   // more queries than max_query_len
  const int tok0 = pair * 2 * TQ;                 // tile A: tok0 .., tile B: tok0 + TQ ..
  if (n <= 0 || tok0 >= n) return;
  const bool has_b = tok0 + TQ < n;
  const int cap = min(p.max_context_len, p.max_blocks_per_seq << p.bs_log2);
  if (ctx < n || ctx > cap) {   // queries must be the last n of a context the table covers
    if (pair == 0 && tid == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    const int ntok = min(2 * TQ, n - tok0);
    for (int i = tid; i < ntok * G * kPfD; i += kThreads) {
      const int t = i / (G * kPfD), r = i % (G * kPfD);
      const int64_t at = (static_cast<int64_t>(q0 + tok0 + t) * p.num_q_heads + g * G) * kPfD + r;
      if (wp.out_bf16)
        static_cast<__nv_bfloat16*>(wp.out)[at] = __float2bfloat16_rn(0.f);
      else
        static_cast<float*>(wp.out)[at] = 0.f;
    }
    return;
  }
  // list entries each query tile needs (causal: up to its last token's position)
  const int end_a = min(tok0 + TQ, n), end_b = min(tok0 + 2 * TQ, n);
  int nt_a = ((p.causal ? ctx - n + end_a : ctx) + kPfKeys - 1) / kPfKeys;
  int nt_b = has_b ? ((p.causal ? ctx - n + end_b : ctx) + kPfKeys - 1) / kPfKeys : 0;
  PfList ls = {0, 0, 0, 0, 0};
  if (wp.window > 0) {
    const int first_a = ctx - n + tok0;
    const int sink_tiles = (min(wp.sinks, ctx) + kPfKeys - 1) / kPfKeys;
    ls.low = max(0, first_a - wp.window + 1);
    ls.base = ls.low / kPfKeys;
    ls.ns = min(sink_tiles, ls.base);
    nt_a += ls.ns - ls.base;
    if (has_b) {
      nt_b += ls.ns - ls.base;
      ls.skip0 = sink_tiles > ls.base ? sink_tiles : ls.ns;   // (then ns = base)
      ls.nskip = max(0, max(0, first_a + TQ - wp.window + 1) / kPfKeys - ls.base + ls.ns - ls.skip0);
    }
  }
  const int ntiles = max(nt_a, nt_b);
  // a box of keys that some query of the CTA may see
  auto box_seen = [&](int kb) { return kb < ctx && (kb < wp.sinks || kb + p.box_rows > ls.low); };
  // the tile's keys with cache data (bit i of valid: box i) that some query sees; nearly
  // every tile has all of them (the general case takes about 1,000 cycles)
  auto tile_mask = [&](int k0, uint32_t valid, int nbox) -> uint64_t {
    if (valid == (1u << nbox) - 1u && k0 + kPfKeys <= ctx &&
        (k0 >= ls.low || k0 + kPfKeys <= wp.sinks))
      return ~0ull;
    uint64_t m = 0;
    for (int i = 0; i < nbox; ++i)
      if ((valid >> i) & 1u)
        m |= pw_below(min(p.box_rows, ctx - (k0 + i * p.box_rows))) << (i * p.box_rows);
    return m & ~(pw_below(ls.low - k0) & ~pw_below(wp.sinks - k0));
  };
  const int32_t* bt_row = p.block_tables + static_cast<int64_t>(s) * p.max_blocks_per_seq;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     smem_u32(&tmem_base_sh))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // TMEM: query tile t's P at columns 256t + [0, 64), S at 256t + 64, O at 256t + 128
  const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base_sh, 0);

  // 8-bit caches launch 512 threads of 128 registers; the softmax warps take 168 and the
  // others 88 (256 x 168 + 256 x 88 = 512 x 128).
  // The issuing roles: one lane's code on bf16 caches (146 us on the three ragged chunks named
  // above, 149 as a whole warp's), a whole warp's on 8-bit ones (285 us on the fp8 chunks, 291
  // as one lane's).
  auto issuer = [&] { return !C8 || pw_elect(); };
  auto issuer_wait = [&](uint32_t bar, uint32_t parity) {
    return C8 ? pw_wait_all(bar, parity, abort_flag) : pw_wait(bar, parity, abort_flag);
  };
  int copied = 0;   // copying warps: key tiles whose copies were started
  if (warp >= 8) {
  if constexpr (C8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
  if (warp == 8 || warp == 11) {
    // --------------------- TMA producers: warp 8 K, warp 11 V -------------------
    const bool is_v = warp == 11;
    const int box_rows = p.box_rows;
    const int nbox = kPfKeys / box_rows;
    bool flagged = false;
    auto lookup = [&](int kb) -> int32_t {   // a block id; -1: nothing to see; -2: out of range
      const int32_t b = __ldg(bt_row + (kb >> p.bs_log2));
      return (b >= 0 && b < p.num_blocks) ? b : -2;
    };
    auto report = [&](int32_t blk) {
      if (!is_v && __ballot_sync(0xffffffffu, blk == -2) && !flagged) {
        if (lane == 0) flag_status(p.status, PKV_DEV_BAD_BLOCK);
        flagged = true;
      }
    };
    if constexpr (!C8) {
      // Per key tile, lanes i and i + 16 look up box i's block (before the wait for the
      // stage) and copy a 64-column half each.
      const int bx = lane & 15, hh = lane >> 4;
      for (int j = 0; j < ntiles; ++j) {
        const int st = j % STAGES;
        const int k0 = ls.key0(j);
        const int kb = k0 + bx * box_rows;
        const int32_t blk = bx < nbox && box_seen(kb) ? lookup(kb) : -1;
        const uint32_t valid = __ballot_sync(0xffffffffu, blk >= 0) & 0xFFFFu;   // bit i: box i
        report(blk);
        if (j >= STAGES) {
          if (!pw_wait_all(smem_u32(&empty[st]), ((j / STAGES) - 1) & 1, abort_flag)) break;
        }
        const uint32_t bar = smem_u32(is_v ? &full_v[st] : &full[st]);
        if (lane == 0) {
          if (!is_v) key_mask[st] = tile_mask(k0, valid, nbox);
          mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(valid)) * 2u * box_rows * 128u);
        }
        __syncwarp();
        if (blk >= 0) {
          const uint32_t dst = sma + kRing + st * kStage + (is_v ? 2 * kKVHalf : 0) + hh * kKVHalf +
                               bx * box_rows * 128;
          const int z = (blk << p.bs_log2) + (kb & ((1 << p.bs_log2) - 1));
          tma_load_3d(dst, is_v ? &tmap_v : &tmap_k, hh * 64, g, z, bar);
        }
        copied = j + 1;
      }
    } else {
      // Lane i looks up box i and copies its codes, [box_rows][128 B], into one of the raw
      // buffers; the K producer leaves the tile's mask and scales beside it.
      const uint32_t raw_a = sma + LY::raw() + (is_v ? kPfRawBufs * kRawTile : 0);
      // The table is read two tiles ahead and the scales one tile ahead of the copy: each
      // is a round trip of its own.
      auto entry = [&](int j) -> int32_t {
        const int kb = ls.key0(j) + lane * box_rows;
        return j < ntiles && lane < nbox && box_seen(kb) ? lookup(kb) : -1;
      };
      float ks_next = 0.f, vs_next = 1.f;
      auto load_scales = [&](int32_t b) {
        ks_next = 0.f;
        vs_next = 1.f;
        if (!is_v && b >= 0) {
          const int64_t at = static_cast<int64_t>(b) * wp.scale_stride + g;
          ks_next = __ldg(p.k_scale + at);
          vs_next = __ldg(p.v_scale + at);
        }
      };
      int32_t blk = -1, blk1 = entry(0), blk2 = entry(1);
      load_scales(blk1);
      for (int j = 0; j < ntiles; ++j) {
        const int rb = j % kPfRawBufs;
        const int k0 = ls.key0(j);
        const int kb = k0 + lane * box_rows;
        blk = blk1;
        blk1 = blk2;
        const float ks = ks_next, vs = fmaxf(vs_next, kPfMinVScale);
        blk2 = entry(j + 2);
        load_scales(blk1);
        const uint32_t valid = __ballot_sync(0xffffffffu, blk >= 0);   // bit i: box i has data
        report(blk);
        const PfScale e = {fabsf(p.qk_scale_log2) * ks, vs, __log2f(vs), 0.f};
        if (j >= kPfRawBufs) {
          if (!pw_wait_all(smem_u32(&raw_free[is_v ? 1 : 0][rb]), ((j / kPfRawBufs) - 1) & 1, abort_flag))
            break;
        }
        if (!is_v && lane < nbox)
          for (int u = 0; u < box_rows / 8; ++u) raw_scale[rb][lane * (box_rows / 8) + u] = e;
        if (!is_v && lane == 0) raw_mask[rb] = tile_mask(k0, valid, nbox);
        __syncwarp();
        const uint32_t rbar = smem_u32(&raw_full[is_v ? 1 : 0][rb]);
        if (lane == 0)
          mbar_arrive_expect_tx(rbar, static_cast<uint32_t>(__popc(valid)) * box_rows * 128u);
        __syncwarp();
        if (blk >= 0) {
          const int z = (blk << p.bs_log2) + (kb & ((1 << p.bs_log2) - 1));
          tma_load_3d(raw_a + rb * kRawTile + lane * box_rows * 128, is_v ? &tmap_v : &tmap_k, 0, g, z,
                      rbar);
        }
        copied = j + 1;
      }
    }
  } else if (warp == 9) {
    // ---------------------------- QK issuer ------------------------------------
    // Key tiles in order, query tile A then B: once the stage has landed and the S
    // columns are free (the softmax has loaded the previous S).
    if (C8 || pw_elect()) {
      const uint32_t idesc_qk = tc_idesc(kPfRows, kPfKeys, false, false, !C8);
      const uint64_t qd[2] = {tc_desc(sma, 0, 1024), tc_desc(sma + LY::kQ, 0, 1024)};
      for (int j = 0; j < ntiles; ++j) {
        if (!issuer_wait(smem_u32(&full[j % STAGES]), (j / STAGES) & 1)) break;
        const uint64_t kd = tc_desc(sma + kRing + (j % STAGES) * kStage, 0, 1024);
        bool ok = true;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= (t == 0 ? nt_a : nt_b) || ls.skips(t, j)) continue;
          const int jt = ls.count(t, j);   // entries this query tile has done
          ok = jt == 0 ? issuer_wait(smem_u32(&q_ready[t]), 0)
                       : issuer_wait(smem_u32(&s_free[t]), (jt - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (issuer()) {
#pragma unroll
            for (int ks = 0; ks < kPfD / 16; ++ks)   // 16 dims: half ks / 4, 32 bytes each
              tc_mma(tm + 256 * t + kPfKeys, qd[t] + (((ks >> 2) * LY::kQHalf + (ks & 3) * 32) >> 4),
                     kd + (((ks >> 2) * kKVHalf + (ks & 3) * 32) >> 4), idesc_qk, ks > 0);
            tc_commit(smem_u32(&s_full[t]));
          }
        }
        if (!ok) break;
      }
      if (issuer()) tc_commit(smem_u32(&drain[0]));   // its MMAs finish before TMEM is released
      volatile int no_abort = 0;
      pw_wait(smem_u32(&drain[0]), 0, &no_abort);
    }
  } else if (warp == 10) {
    // ---------------------------- PV issuer ------------------------------------
    // Query tile A then B of each key tile, once its P is written; then the stage is
    // released (its QK finished before its P could be written).
    if (C8 || pw_elect()) {
      const uint32_t idesc_pv = tc_idesc(kPfRows, kPfD, false, true, !C8);
      for (int j = 0; j < ntiles; ++j) {
        if (!issuer_wait(smem_u32(&full_v[j % STAGES]), (j / STAGES) & 1)) break;
        const uint64_t vd =
            tc_desc(sma + kRing + (j % STAGES) * kStage + 2 * kKVHalf, kKVHalf, 1024);
        bool ok = true;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j >= (t == 0 ? nt_a : nt_b) || ls.skips(t, j)) continue;
          const int jt = ls.count(t, j);
          ok = issuer_wait(smem_u32(&p_full[t]), jt & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t dO = tm + 256 * t + 2 * kPfKeys;
          if (issuer()) {
#pragma unroll
            for (int kk = 0; kk < kPfKeys / 16; ++kk) {
              const uint64_t bdesc = vd + ((kk * 2048) >> 4);
              tc_mma_ts(dO, tm + 256 * t + 8 * kk, bdesc, idesc_pv, (jt > 0 || kk > 0));
              if (LO) tc_mma_ts(dO, tm + 256 * t + 32 + 8 * kk, bdesc, idesc_pv, 1);
            }
            tc_commit(smem_u32(&o_done[t]));
          }
        }
        if (!ok) break;
        if (issuer()) tc_commit(smem_u32(&empty[j % STAGES]));
      }
      if (issuer()) tc_commit(smem_u32(&drain[1]));
      volatile int no_abort = 0;
      pw_wait(smem_u32(&drain[1]), 0, &no_abort);
    }
  } else if (C8 && warp >= 12) {
    // ---------------- widening: warps 12, 13 K; 14, 15 V; 32 rows each ----------------
    // A lane widens one row's 128 codes to fp16 (exactly) into the stage's two swizzled
    // halves.  Lane = row and one 16-byte chunk per step spread each step's loads and stores
    // evenly over the banks; loads precede the stores.
    const bool is_v = warp >= 14;
    const int r0 = (warp & 1) * 32;
    const uint8_t* raw = sm + LY::raw() + (is_v ? kPfRawBufs * kRawTile : 0) + (r0 + lane) * 128;
    // Units per pass.  The roles' loops together overrun the instruction cache, which slows
    // the softmax warps: INT8, whose widening is the longer code, takes 1,349 ns a key tile with
    // two units a pass and 1,411 with all eight at once (float32 output; bf16 1,130 and 1,118).
    constexpr int kStep = 2;
    auto off = [&](int u) { return (u ^ (lane & 7)) << 4; };   // 16-byte unit u in a row = lane (mod 8)
    for (int j = 0; j < ntiles; ++j) {
      const int st = j % STAGES, rb = j % kPfRawBufs;
      bool ok = pw_wait(smem_u32(&raw_full[is_v ? 1 : 0][rb]), (j / kPfRawBufs) & 1, abort_flag);
      if (j >= STAGES)
        ok = ok && pw_wait(smem_u32(&empty[st]), ((j / STAGES) - 1) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* src = raw + rb * kRawTile;
      uint8_t* dst = sm + kRing + st * kStage + (is_v ? 2 * kKVHalf : 0) + (r0 + lane) * 128;
      if (warp == 12) {
        if (lane < 8) key_scale[st][lane] = raw_scale[rb][lane];
        if (lane == 0) key_mask[st] = raw_mask[rb];
      }
#pragma unroll 1
      for (int u0 = 0; u0 < 8; u0 += kStep) {
        uint4 cs[kStep];
#pragma unroll
        for (int v = 0; v < kStep; ++v) cs[v] = *reinterpret_cast<const uint4*>(src + off(u0 + v));
#pragma unroll
        for (int v = 0; v < kStep; ++v) {
          uint32_t h[8];
          const uint32_t w[4] = {cs[v].x, cs[v].y, cs[v].z, cs[v].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (I8)
              s8x4_to_f16x2x2_biased(w[e], h[2 * e], h[2 * e + 1]);
            else
              e4m3x4_to_f16x2x2(w[e], h[2 * e], h[2 * e + 1]);
          }
          if constexpr (I8) {   // code + 1152 - 1152: the code, exactly
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = hsub2_u32(h[e], 0x64806480u);
          }
          uint8_t* half = dst + ((u0 + v) >> 2) * kKVHalf;
          const int uu = 2 * ((u0 + v) & 3);
          *reinterpret_cast<uint4*>(half + off(uu)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(half + off(uu + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
      }
      fence_proxy_async();   // the stage's writes before the MMAs' reads, the raw buffer's
      __syncwarp();          // reads before the next copy into it
      if (lane == 0) {
        mbar_arrive(smem_u32(is_v ? &full_v[st] : &full[st]));
        mbar_arrive(smem_u32(&raw_free[is_v ? 1 : 0][rb]));
      }
    }
  }
  } else {
    if constexpr (C8) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
    // -------------------- softmax warpgroups (A: 0-3, B: 4-7) -----------------
    const int t = warp >> 2;                            // query tile of this warpgroup
    const int w0 = (warp & 3) * 32;                     // this warp's rows w0 .. w0 + 31
    const int r = w0 + lane;                            // accumulator row = TMEM lane
    const int my_nt = t == 0 ? nt_a : nt_b;
    const uint32_t lane_q = static_cast<uint32_t>(w0) << 16;
    const uint32_t tP = tm + 256 * t + lane_q, tS = tP + kPfKeys, tO = tP + 2 * kPfKeys;
    const uint32_t g_inv = (65536u + G - 1) / G;        // r / G for r < 128, G <= 16
    auto row_token = [&](int row) { return static_cast<int>((row * g_inv) >> 16); };
    // this row's offset in q and out (elements), -1 past the chunk
    auto row_at = [&](int row) -> int64_t {
      const int tk = row_token(row), tok = tok0 + t * TQ + tk;
      if (row >= TQ * G || tok >= n) return -1;
      return (static_cast<int64_t>(q0 + tok) * p.num_q_heads + g * G + row - tk * G) * kPfD;
    };
    float q_unscale = 1.f;   // 8-bit caches: the row of q went to fp16 times 1 / q_unscale
    {
      // The warp's 32 rows of Q_t into shared memory (two halves of 64 dims, K-major, 128B
      // swizzle).  Pass i takes rows 2i and 2i + 1, 16 lanes x 16 bytes each, so that every
      // load is of whole rows.
      uint8_t* qb = sm + t * LY::kQ;
      const int ch = lane & 15;
      uint4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int64_t at = row_at(w0 + 2 * i + (lane >> 4));
        v[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + ch) : make_uint4(0, 0, 0, 0);
      }
      // a negative logit scale goes into q, so that a larger product is a larger logit
      const uint32_t flip = p.qk_scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (C8) {
          // fp16, scaled by 2^qsh, which puts the row's largest |q| in [2^14, 2^15): inside
          // fp16's range whatever q's magnitude, and exact for every element within 2^-24
          // of that max (a bf16 has 8 significant bits)
          uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t mb = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) mb = max(mb, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
          const int ex = mb >= 0x0080u ? static_cast<int>(mb >> 7) - 127 : 0;
          const int qsh = min(max(14 - ex, -126), 126);
          const float qmul = __uint_as_float(static_cast<uint32_t>(127 + qsh) << 23);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = pack_f16(qmul * bf16_lo(x[e]), qmul * bf16_hi(x[e]));
          v[i] = make_uint4(x[0], x[1], x[2], x[3]);
          // thread `lane` keeps row w0 + lane's factor: pass lane / 2, half-warp lane % 2
          const int sh = __shfl_sync(0xffffffffu, qsh, (lane & 1) * 16);
          if (i == (lane >> 1)) q_unscale = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
        }
        *reinterpret_cast<uint4*>(qb + (ch >> 3) * LY::kQHalf + swz(w0 + 2 * i + (lane >> 4), ch & 7)) =
            v[i];
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_ready[t]));
    }
    const bool row_ok = row_at(r) >= 0;
    const int qpos = ctx - n + tok0 + t * TQ + row_token(r);   // this row's position
    const int last = p.causal ? qpos : ctx - 1;                // last key it sees
    const int row_low = wp.window > 0 ? qpos - wp.window + 1 : 0;   // first key of its window
    // over the warp's rows; rows past the chunk do not count (their outputs are not stored)
    const int last_min = __reduce_min_sync(0xffffffffu, row_ok ? last : INT32_MAX - 1);
    const int low_max = __reduce_max_sync(0xffffffffu, row_ok ? row_low : INT32_MIN);
    // Logit factors are kept positive (a zero one is raised to the smallest normal), so that
    // a masked -inf stays -inf under them.
    constexpr float kTiny = 1.17549435e-38f;
    const float sl2 = fmaxf(fabsf(p.qk_scale_log2), kTiny);    // 16-bit caches
    float m = -CUDART_INF_F, l = 0.f;                          // m in log2 units
    bool alive = true;
    bool s_there = false;   // warp-uniform: S and the stage's mask were seen to be there
    for (int j = 0; j < my_nt && alive; ++j) {
      if (ls.skips(t, j)) continue;
      const int jt = ls.count(t, j), st = j % STAGES;
      const int k0 = ls.key0(j);
      // S ready implies that the stage's K landed; waiting on the stage's barrier as well
      // makes the producer's key mask and scales for it visible here.
      if (!s_there) {
        if (!pw_wait(smem_u32(&s_full[t]), jt & 1, abort_flag) ||
            !pw_wait(smem_u32(&full[st]), (j / STAGES) & 1, abort_flag))
          alive = false;
        if (!__all_sync(0xffffffffu, alive)) break;
      }
      tc_fence_after();
      // the stage's logit factors and V scales: loads from shared memory take hundreds of
      // cycles beside the MMAs' and the widening warps', so all are asked for here at once
      float fk[C8 ? 8 : 1], vk[C8 ? 8 : 1], lk[C8 ? 8 : 1];
      if constexpr (C8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float4 e = *reinterpret_cast<const float4*>(&key_scale[st][u]);
          fk[u] = fmaxf(e.x * q_unscale, kTiny);
          vk[u] = e.y;
          lk[u] = e.z;
        }
      }
      const uint64_t vmask = key_mask[st];
      float sv[kPfKeys];
      pf_ld64(tS, sv);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_free[t]));
      // keys the row sees: with cache data, up to `last`, in the window or among the sinks
      if (vmask != ~0ull || k0 + kPfKeys > last_min + 1 ||
          (k0 < low_max && k0 + kPfKeys > wp.sinks)) {   // not all of them for all of the warp's rows
        uint64_t rmask = vmask & pw_below(last - k0 + 1) &
                         (~pw_below(row_low - k0) | pw_below(wp.sinks - k0));
        if (!row_ok) rmask = 0ull;
        const uint32_t mlo = static_cast<uint32_t>(rmask), mhi = static_cast<uint32_t>(rmask >> 32);
#pragma unroll
        for (int c = 0; c < kPfKeys; ++c)
          if (!(((c < 32 ? mlo : mhi) >> (c & 31)) & 1u)) sv[c] = -CUDART_INF_F;
      }
      float mt = -CUDART_INF_F;   // the tile's largest logit (8-bit caches: + log2 vs)
      if constexpr (C8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float a = pf_max3(sv[8 * u], sv[8 * u + 1], sv[8 * u + 2]);
          const float b = pf_max3(sv[8 * u + 3], sv[8 * u + 4], sv[8 * u + 5]);
          const float c = fmaxf(sv[8 * u + 6], sv[8 * u + 7]);
          mt = fmaxf(mt, fmaf(pf_max3(a, b, c), fk[u], lk[u]));
        }
      } else {
        float ma = sv[0], mb = sv[1];
#pragma unroll
        for (int c = 2; c + 3 < kPfKeys; c += 4) {
          ma = pf_max3(ma, sv[c], sv[c + 1]);
          mb = pf_max3(mb, sv[c + 2], sv[c + 3]);
        }
        mt = fmaxf(pf_max3(ma, sv[kPfKeys - 2], sv[kPfKeys - 1]), mb) * sl2;
      }
      float alpha = 1.f;
      bool resc = false;
      // The reference moves only when a weight would exceed 2^(kUp + 8).  8-bit caches set it kUp = 7
      // below the maximum: fp16 weights (at most 2^15) then hold what is 2^-21 of the largest with
      // all their bits, and what is 2^-31 of it at all.
      constexpr float kUp = C8 ? 7.f : 0.f;
      if (mt > m + (kUp + 8.f)) {
        if (m != -CUDART_INF_F) {
          alpha = pf_ex2(m - (mt - kUp));
          resc = true;
        }
        m = mt - kUp;
      }
      const float mu = m == -CUDART_INF_F ? 0.f : m;   // rows with nothing seen yet: p = 0
      // p, l and the packed weights; pairs go through the packed fp32 pipe
      uint32_t w[kPfKeys / 2];
      float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float f = C8 ? fk[C8 ? u : 0] : sl2;
        const float vs = C8 ? vk[C8 ? u : 0] : 1.f;
#pragma unroll
        for (int c = 8 * u; c < 8 * u + 8; c += 2) {
          const float2 x = __ffma2_rn(make_float2(sv[c], sv[c + 1]), make_float2(f, f),
                                      make_float2(-mu, -mu));
          float2 y = make_float2(pf_ex2(x.x), pf_ex2(x.y));   // 2^-inf = 0 for masked keys
          ls2[(c >> 1) & 1] = __fadd2_rn(ls2[(c >> 1) & 1], y);
          if constexpr (C8) {
            y = __fmul2_rn(y, make_float2(vs, vs));
            w[c >> 1] = pack_f16(y.x, y.y);
          } else {
            w[c >> 1] = pack_bf16(y.x, y.y);
          }
          if constexpr (LO) {
            sv[c] = y.x;
            sv[c + 1] = y.y;
          }
        }
      }
      l = l * alpha + ((ls2[0].x + ls2[0].y) + (ls2[1].x + ls2[1].y));
      // PV(j-1) must be finished before P is overwritten and before O is scaled
      if (jt >= 1 && !pw_wait(smem_u32(&o_done[t]), (jt - 1) & 1, abort_flag)) alive = false;
      if (!__all_sync(0xffffffffu, alive)) break;
      tc_fence_after();
      pw_st32(tP, w);   // row = lane, column c = keys 2c and 2c + 1
      if constexpr (LO) {   // what the first part left: 2^-16 together in bf16, 2^-22 in fp16
        uint32_t wl[kPfKeys / 2];
#pragma unroll
        for (int c = 0; c < kPfKeys; c += 2) {
          float2 hi;
          if constexpr (C8)
            hi = __half22float2(*reinterpret_cast<const __half2*>(&w[c >> 1]));
          else
            hi = make_float2(bf16_lo(w[c >> 1]), bf16_hi(w[c >> 1]));
          const float2 lo = __ffma2_rn(hi, make_float2(-1.f, -1.f), make_float2(sv[c], sv[c + 1]));
          wl[c >> 1] = C8 ? pack_f16(lo.x, lo.y) : pack_bf16(lo.x, lo.y);
        }
        pw_st32(tP + 32, wl);
      }
      if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int c = 0; c < kPfD; c += 32) {
          float o[32];
          tc_ld32(tO + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tc_st32(tO + c, o);
        }
      }
      // V rows that no query sees or without cache data -> 0, once per key tile: by tile A's
      // group while it needs this tile, else by tile B's; after the V copies landed
      if ((t == 0) == (j < nt_a) && vmask != ~0ull) {
        // a vote: lanes that leave the loop alone would miss the warp-wide instructions below
        if (!pw_wait_all(smem_u32(&full_v[st]), (j / STAGES) & 1, abort_flag)) alive = false;
        if (alive && r < kPfKeys && !((vmask >> r) & 1ull)) {
          uint8_t* vrow = sm + kRing + st * kStage + 2 * kKVHalf + r * 128;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            *reinterpret_cast<uint4*>(vrow + (u << 4)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(vrow + kKVHalf + (u << 4)) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async();
      }
      s_there = __all_sync(0xffffffffu,
                           !ls.skips(t, j + 1) &&
                               pw_test2(smem_u32(&s_full[t]), (jt + 1) & 1,
                                        smem_u32(&full[(j + 1) % STAGES]), ((j + 1) / STAGES) & 1));
      pw_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[t]));
    }
    // Epilogue: 128 bytes of each row at a time through shared memory (the warp's share of
    // Q_t, which every QK has read by now), so that a store is of whole lines.
    const int done = my_nt > 0 ? ls.count(t, my_nt) : 0;
    const bool ok = alive && my_nt > 0 &&
                    pw_wait(smem_u32(&o_done[t]), (done - 1) & 1, abort_flag);
    if (__all_sync(0xffffffffu, ok)) {   // warp-uniform: the TMEM load is warp-wide
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint8_t* stage = sm + t * LY::kQ + (warp & 3) * 4096;
      const int esz = wp.out_bf16 ? 2 : 4;
      uint8_t* dst[8];   // rows 4i + lane / 8, eight lanes each
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t at = row_at(w0 + 4 * i + (lane >> 3));
        dst[i] = at >= 0 ? static_cast<uint8_t*>(wp.out) + at * esz + (lane & 7) * 16 : nullptr;
      }
      const int cols = 128 / esz;
      for (int c = 0; c < kPfD; c += cols) {
        if (wp.out_bf16) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float o[32];
            tc_ld32(tO + c + 32 * hf, o);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(stage + swz(lane, 4 * hf + u)) = make_uint4(
                  pack_bf16(o[8 * u] * inv, o[8 * u + 1] * inv),
                  pack_bf16(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                  pack_bf16(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                  pack_bf16(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
          }
        } else {
          float o[32];
          tc_ld32(tO + c, o);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<float4*>(stage + swz(lane, u)) = make_float4(
                o[4 * u] * inv, o[4 * u + 1] * inv, o[4 * u + 2] * inv, o[4 * u + 3] * inv);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (dst[i])
            *reinterpret_cast<uint4*>(dst[i] + c * esz) =
                *reinterpret_cast<const uint4*>(stage + swz(4 * i + (lane >> 3), lane & 7));
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && (warp == 8 || warp == 11)) {   // copies may be in flight: no role waits for them now
    constexpr int kBufs = C8 ? kPfRawBufs : STAGES;
    const int is_v = warp == 11 ? 1 : 0;
    volatile int no_abort = 0;
    for (int j = max(0, copied - kBufs); j < copied; ++j)
      pw_wait(smem_u32(C8 ? &raw_full[is_v][j % kBufs] : is_v ? &full_v[j % kBufs] : &full[j % kBufs]),
              (j / kBufs) & 1, &no_abort);
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tm) : "memory");
  if (tid == 0 && *abort_flag) flag_status(p.status, PKV_DEV_TIMEOUT);
}

}  // namespace pkv

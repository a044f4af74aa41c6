// Attention over packed prompts on the 5th-generation tensor cores (tcgen05 + TMEM): bf16 q, k and v as
// a projection leaves them, sequences back to back, head_dim up to 128, causal or not, with a window
// and sinks, f32 or bf16 output.
//
//   out_i = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (q_i . k_j) - m),  c = scale log2(e)
//
// Work.  A query tile is 128 accumulator rows: TQ = 128 / G consecutive tokens times the G query heads
// of one KV head (row r = token r / G, head r % G), so that a K/V tile serves all of them.  An item
// is two neighbouring query tiles A and B of one sequence and KV head, and walks the keys that some
// of their rows see in tiles of 128:
//   S_t  = Q_t K^T   M=128 N=128 K=D    both from shared memory
//   O_t += P_t V     M=128 N=D   K=128  P_t from TMEM, V from shared memory
// TMEM: S_A, S_B (128 columns each; P_t takes the place of S_t, two bf16 to a column), O_A, O_B.
//
// A persistent CTA per SM takes items, longest first, so that the roles of one item run into the
// next: while the last products of an item are under way, the next one's first keys are loaded.  Warps:
//   0-7, 8-15  softmax and epilogue of tile A, of tile B: 16 rows a warp, four lanes on a row.  With a row per
//              thread and four warps a tile, a key tile's softmax took 1,750 cycles of a chain of 3,500:
//              one warp on a sub-partition waits for its own loads, exponentials and stores in turn
//   16         issues the MMAs: PV_A(j), QK_A(j+1), PV_B(j), QK_B(j+1), so that one tile's softmax
//              runs under the other's products (P takes S's place: the next scores wait for the product)
//   17         TMA loads (Q_A, Q_B; a ring of K and V tiles)
//   18         finds the items: the u-th unit of the batch, longest first
// Rows of a V tile past its sequence's end belong to another sequence, and a weight of 0 times what is
// not finite would be NaN: the softmax warps clear them before they hand over the tile's weights.
// The running reference m moves only when a weight would exceed 2^kPkLag, so that O is hardly ever
// scaled; S_t(j) being there implies that PV_t(j-1) is done (one thread issues both), so the softmax
// warps scale it themselves.
//
// Precision.  Scores, sums and O are float32, and the weights enter the product as two bf16 parts (2^-17 of
// each at most): a bf16 output is the float32 one rounded.  A caller may ask for one part (2^-9 of each)
// for a bf16 output: 1.2 to 1.4 times the error against 64 bits on normal values (2.0e-3 to 2.4e-3 of
// the norm for 1.6e-3) and half the product's time.  A third part for float32 outputs has no room: the two
// take all 128 columns of S.
//
// What bounds it.  At head_dim 128 with two weight parts the products: a pair of key tiles needs 3,072 cycles of
// them and takes 3,660 (tensor pipe 84 % of active cycles).  With one part the chain of a key tile: softmax
// 1,400 cycles, product and next scores 770 of its 1,024 behind it, and about 450 until each sees that the
// other is done, with the other tile's products in between: 2,600 cycles for a pair whose products need
// 2,048; without the exponentials it would be 6 % faster, without the maxima 4 %.  What it took to get
// there: no mask code in tiles without one; a plain loop for the issuer (its general steps took 3,100
// cycles a pair); references that move only on a vote; both halves' scores asked for together.  Short lists wait for their first rows
// (Q and K of the next item reach shared memory 2 to 3 us after they are asked for, as all CTAs ask at
// once) and a cold CTA for its code.  Tried and left out, with one part: one issuer for each tile (both tiles' phases
// fall together), with and without turns; prefetches of the next item to L2 (16 prompts of 512 tokens 77
// -> 90 us); the order of items kept within sequences whose keys fit L2; lists of equal length for both tiles; the halves as a loop (20 % slower); Q before K.
//
// Measured (bf16 output; with one weight part; float32 output): three prompts of 700 to 8,192 tokens, 32 heads
// on 8, causal 585 to 655 us across GPUs, 460 to 506, 767 (1,100 to 1,230 TFLOP/s of q k and p v, the second part
// of p not counted; 1,430 to 1,570 with one); 16 prompts of 512 tokens, 32 heads 74 us, 66, 81; 11 images of 64 to
// 1,156 patches, 16 heads of 80, not causal 56 us, 47, 62; nine chunks of up to 1,500 tokens behind 333 keys, 16
// heads on 2 of 64, window 1,024 44 us, 37, 48 to 52; four prompts of up to 60 tokens 9.7 us, 9.2, 10.3.
//
// Every wait is bounded (2 s) and gives up when another role has given up; copies in flight are then
// waited for, and TMEM is released before the CTA exits.
#pragma once

#include "prefill_win.cuh"

namespace pkv {

constexpr int kPkRows = 128;      // accumulator rows of a query tile (M)
constexpr int kPkKeys = 128;      // keys of a tile (N of QK, K of PV)
constexpr int kPkThreads = 640;
constexpr int kPkRank = 1024;     // sequences whose items are ordered by length together
constexpr int kPkSlab = 128 * 128;   // 128 rows of 64 bf16 (128-byte swizzle)
// The reference m moves only when a weight would exceed 2^kPkLag: the weights, their sum and O are
// floating-point numbers of float32's range, in which a factor loses nothing, and with a lag of 24
// O is scaled for logits that grow by 16 from one key tile to another, where one of 8 has most
// short prompts' second tiles scale it (a first row of few keys is enough), at 1,500 cycles.
constexpr float kPkLag = 24.f;
// Key tiles after which a float32 output takes O up.  The tensor cores cut their sums towards zero, half a
// step of O's last place each time on average, which adds up with the keys: 8 tiles are 128 sums (8 of 16 keys a
// tile, two weight parts) and 2.9e-6 of an output of one sign; measured 2.2e-6 to 2.8e-6, and 3.2e-6 to 3.6e-6 of
// the norm for normal values, over 3,000 keys as over a million.  16 tiles are off by twice that (5.3e-6 to
// 6.5e-6) and up to 8 % faster (three prompts to 8,192 tokens 706 us for 767).  In between the epilogue adds in float32,
// in the output's own rows.  A bf16 output has no room for that in them and stays in the tensor cores to its end: 3e-4 of
// the norm over 130,000 keys, 2.3e-3 over a million (5.1e-3 for values of one sign; its own rounding: 1.7e-3).
constexpr int kPkPart = 8;

struct PackedParams {
  void* out;                    // [T, Hq, D]
  const int32_t* query_start;   // [S + 1]
  const int32_t* key_start;     // [S + 1]
  const int32_t* context_lens;  // [S] or null
  int32_t* status;
  int32_t num_seqs, num_tokens, num_keys;
  int32_t num_q_heads, num_kv_heads, dim;
  int32_t tile_tokens;          // TQ = 128 / G
  int32_t causal, window, sinks;
  float scale_log2;
  uint32_t test_stall_bytes;    // CTA 0's first V tile waits for these in vain; 0 but in tests
};

struct PkItem {
  int32_t valid;     // 0: no more items
  int32_t row0;      // first row of q and out (tile A's first token)
  int32_t tokens;    // tokens of the sequence from there on
  int32_t key0;      // first row of k and v
  int32_t keys;      // keys of the sequence
  int32_t pos0;      // position of tile A's first token
  int32_t head;      // KV head
  int32_t all_a, all_b;   // key tiles of A and B
  int32_t ns, base;  // entry j of the list is key tile j (j < ns) or j - ns + base
  int32_t j0;        // first entry of this part of the list
  int32_t nt_a, nt_b;   // entries of this part
  int32_t ragged;    // the part's last tile reaches past the sequence's end
  __device__ __forceinline__ int nt(int t) const { return t == 0 ? nt_a : nt_b; }
  __device__ __forceinline__ int most() const { return max(nt_a, nt_b); }
  // whether this part ends tile t's list
  __device__ __forceinline__ bool ends(int t) const { return nt(t) > 0 && j0 + nt(t) == (t == 0 ? all_a : all_b); }
};

template <int SLABS, int STAGES>
struct PkLayout {
  static constexpr int kTile = SLABS * kPkSlab;   // a query or key tile
  static constexpr int kRing = 2 * kTile;         // after Q_A, Q_B
  static constexpr int kRankAt = kRing + STAGES * kTile;
  static constexpr size_t bytes() { return 1024 + kRankAt + kPkRank * 8; }
};

// 16 rows x 64 TMEM columns -> 32 registers a lane, in two steps: they hold the columns after
// pk_ld_wait.  Registers 4g, 4g + 1 are columns 8g + 2c, 8g + 2c + 1 of row lane / 4, c = lane % 4, and
// 4g + 2, 4g + 3 those of row lane / 4 + 8.
__device__ __forceinline__ void pk_ld64(uint32_t taddr, float* v) {
#define PKV_F8(i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), \
                  "=f"(v[i + 5]), "=f"(v[i + 6]), "=f"(v[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : PKV_F8(0), PKV_F8(8), PKV_F8(16), PKV_F8(24)
      : "r"(taddr));
#undef PKV_F8
}
__device__ __forceinline__ void pk_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
  // nothing that reads them moves before the wait
#define PKV_F8(i) "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), \
                  "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7])
  asm volatile("" : PKV_F8(0), PKV_F8(8), PKV_F8(16), PKV_F8(24));
#undef PKV_F8
}

// 16 registers to 16 rows x 32 TMEM columns, without the wait: registers 2g, 2g + 1 are column 4g + c of
// rows lane / 4 and lane / 4 + 8.
__device__ __forceinline__ void pk_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// 16 TMEM columns of 16 rows, times f0 (row lane / 4) and f1 (row lane / 4 + 8), without the wait for the
// stores.
__device__ __forceinline__ void pk_scale16(uint32_t taddr, float f0, float f1) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * ((i & 2) ? f1 : f0));
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 32 bytes to global memory, on a 32-byte boundary: a whole sector.
__device__ __forceinline__ void pk_store32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Waits for the barriers of those lanes that have one, looked at in one instruction.
__device__ __forceinline__ bool pk_wait_lanes(bool any, uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    uint32_t there = 1;
    if (any)
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
          " selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(there)
          : "r"(bar), "r"(parity)
          : "memory");
    if (__all_sync(0xffffffffu, there != 0)) return true;
    if ((n & 63u) == 0) {
      bool stop = *abort_flag != 0;
      const uint64_t now = global_ns();
      if (n == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

// Two phases, looked at together by a whole warp.
__device__ __forceinline__ bool pk_wait2(uint32_t bar_a, uint32_t par_a, uint32_t bar_b, uint32_t par_b,
                                         volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    if (__all_sync(0xffffffffu, pw_test2(bar_a, par_a, bar_b, par_b))) return true;
    if ((n & 63u) == 63u) {
      bool stop = *abort_flag != 0;
      const uint64_t now = global_ns();
      if (n == 63u) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}

// Warp 18: the items of one CTA.  Units (sequence, pair of query tiles, KV head) are ordered by
// the length of their key lists (in pairs of query tiles, cut at the window), longest first and KV heads fastest, within each kPkRank sequences;
// round k of a grid of n CTAs takes units kn .. kn + n - 1, every other round in the opposite
// order.  Order by counting: the units of sequence s that are at least x long are known in closed
// form, so the length of the u-th unit is found by halving.
struct PkOrder {
  const PackedParams& p;
  int32_t* pairs;    // shared, [kPkRank]: pairs of query tiles of a sequence
  int32_t* level;    // shared: length of its first pair, in pairs
  bool flat;         // all pairs of a sequence are alike
  int cap;           // a window lets no list grow past this level
  int first = 0, count = 0, top = 0, lane;   // the sequences at hand; the longest unit
  uint32_t before = 0, total = 0;            // units before them; theirs

  __device__ __forceinline__ int longer(int i, int x) const {   // units of sequence i of level >= x
    if (flat) return level[i] >= x ? pairs[i] : 0;
    return x > cap ? 0 : min(max(level[i] + pairs[i] - x, 0), pairs[i]);
  }
  __device__ __forceinline__ void fill(int s0, bool report) {
    first = s0;
    count = min(kPkRank, p.num_seqs - s0);
    const int per = 2 * p.tile_tokens;
    int hi = 0, sum = 0;
    bool bad = false;
    for (int i = lane; i < count; i += 32) {
      const int s = s0 + i;
      const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
      const int k0 = __ldg(p.key_start + s), k1 = __ldg(p.key_start + s + 1);
      const int ctx = p.context_lens ? __ldg(p.context_lens + s) : k1 - k0;
      int n = 0, lv = 0;
      if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || k0 < 0 || k1 < k0 || k1 > p.num_keys ||
          (q1 > q0 && ctx != k1 - k0)) {
        bad = true;
      } else {
        n = static_cast<int>((static_cast<int64_t>(q1) - q0 + per - 1) / per);
        const int c = k1 - k0;
        lv = flat ? c / per : max(c - (q1 - q0), 0) / per;
      }
      pairs[i] = n;
      level[i] = lv;
      sum += n;
      if (n > 0) hi = max(hi, flat ? lv : min(lv + n - 1, cap));
    }
    __syncwarp();
    if (report && __any_sync(0xffffffffu, bad) && lane == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
    top = __reduce_max_sync(0xffffffffu, hi);
    total = static_cast<uint32_t>(__reduce_add_sync(0xffffffffu, sum)) * p.num_kv_heads;
  }
  __device__ __forceinline__ int sum_longer(int x) const {
    int sum = 0;
    for (int i = lane; i < count; i += 32) sum += longer(i, x);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  // Unit `u` of the batch (u grows from call to call): its sequence, pair and KV head.
  __device__ __forceinline__ bool find(uint32_t u, bool report, int& s, int& pair, int& g) {
    while (u >= before + total) {
      const int next = first + count;
      if (next >= p.num_seqs) return false;
      before += total;
      fill(next, report);
    }
    const uint32_t w = u - before;
    const int r = static_cast<int>(w / p.num_kv_heads);
    g = static_cast<int>(w - r * p.num_kv_heads);
    int lo = 0, hi = top + 1;   // more than r units are of level >= lo, not more of level >= hi
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (sum_longer(mid) > r) lo = mid; else hi = mid;
    }
    int left = r - sum_longer(lo + 1);   // the left-th unit of level lo
    for (int i0 = 0; i0 < count; i0 += 32) {
      const int i = i0 + lane;
      const int mine = i < count ? longer(i, lo) - longer(i, lo + 1) : 0;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, incl > left);
      if (hit != 0) {
        const int at = __ffs(hit) - 1;
        const int offset = left - (__shfl_sync(0xffffffffu, incl, at) - __shfl_sync(0xffffffffu, mine, at));
        s = first + i0 + at;
        pair = offset + (flat ? 0 : max(lo - level[i0 + at], 0));
        return true;
      }
      left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// F32: float32 output, else bf16.  LO: the weights are two bf16 parts, else one.
template <int SLABS, int STAGES, bool F32, bool LO>
__global__ void __launch_bounds__(kPkThreads, 1)
    packed_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                          const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ PackedParams p) {
  using LY = PkLayout<SLABS, STAGES>;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int TQ = p.tile_tokens;

  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t kv_full[STAGES], kv_empty[STAGES];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], o_empty[2],
      item_full[2], item_empty[2], drain;
  __shared__ PkItem items[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sma = smem_u32(sm);
  volatile int* abort_flag = &abort_sh;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  allow_dependents();
  if (tid == kPkThreads - 1) {
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(smem_u32(&kv_full[st]), 1);
      mbar_init(smem_u32(&kv_empty[st]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&q_full[t]), 1);
      mbar_init(smem_u32(&q_empty[t]), 1);
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[t][0]), 8);
      mbar_init(smem_u32(&p_full[t][1]), 8);
      mbar_init(smem_u32(&o_full[t]), 1);
      mbar_init(smem_u32(&o_empty[t]), 8);
      mbar_init(smem_u32(&item_full[t]), 1);
      mbar_init(smem_u32(&item_empty[t]), 18);   // 16 softmax warps, 16, 17
    }
    mbar_init(smem_u32(&drain), 1);
    if (p.test_stall_bytes != 0 && blockIdx.x == 0)
      mbar_expect_tx(smem_u32(&kv_full[1]), p.test_stall_bytes);
    abort_sh = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
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
  // Every role waits for earlier work here: the bounded waits below begin after it.
  grid_dependency_wait();
  const uint32_t tm = __shfl_sync(0xffffffffu, tmem_base_sh, 0);
  // S_t and P_t at columns 128 t, O_t at 256 + 128 t

  auto stage_at = [&](int idx) { return sma + LY::kRing + (idx % STAGES) * LY::kTile; };
  auto kv_bar = [&](int idx) { return smem_u32(&kv_full[idx % STAGES]); };
  auto key_tile = [](const PkItem& it, int j) { return j < it.ns ? j : j - it.ns + it.base; };
  // The i-th item of this CTA, by one lane or a whole warp; false: no more, or another role gave up.
  auto next_item = [&](int i, PkItem& it) {
    if (!pw_wait(smem_u32(&item_full[i & 1]), (i >> 1) & 1, abort_flag)) return false;
    it = items[i & 1];
    return it.valid != 0;
  };
  int loads = 0, copied_q[2] = {0, 0};   // warp 17: copies started, K/V tiles and Q tiles

  // 640 threads of 96 registers; 512 x 104 + 128 x 64 = 640 x 96
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    if (warp == 16) {
      // ------------------------------ MMA issuer ------------------------------
      // The whole warp walks the lists, so that the compiler knows stages and descriptors uniform, and one
      // lane issues.  Barriers are looked at together, a lane each: the tensor cores queue little, and
      // every look (100 to 200 cycles) is time they lie idle.
      // a negative logit scale turns q's sign (bit 13), so that a larger product is a larger logit
      const uint32_t idesc_qk =
          tc_idesc(kPkRows, kPkKeys, false, false, true) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
      const uint32_t idesc_pv = tc_idesc(kPkRows, (p.dim + 15) & ~15, false, true, true);
      const int ksteps = (p.dim + 15) / 16;
      const uint64_t qd0 = tc_desc(sma, 0, 1024), kd0 = tc_desc(sma + LY::kRing, 0, 1024),
                     vd0 = tc_desc(sma + LY::kRing, kPkSlab, 1024);
      // phases gone by, one bit per tile: q_full, p_full, o_empty (nothing to wait for at first)
      uint32_t ph_q = 0, ph_p = 0, ph_o = 3;
      auto qk = [&](int t, int st, bool ends) {   // by one lane; `ends`: Q_t is not needed after this
        const uint64_t qd = qd0 + ((t * LY::kTile) >> 4), kd = kd0 + ((st * LY::kTile) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4 * SLABS; ++ks) {   // 16 dims: slab ks / 4, 32 bytes each
          const int at = ((ks >> 2) * kPkSlab + (ks & 3) * 32) >> 4;
          if (ks < ksteps) tc_mma(tm + 128 * t, qd + at, kd + at, idesc_qk, ks > 0);
        }
        tc_commit(smem_u32(&s_full[t]));
        if (ends) tc_commit(smem_u32(&q_empty[t]));
      };
      auto pv = [&](int t, int st, int half, bool first) {   // by one lane
        const uint64_t vd = vd0 + ((st * LY::kTile) >> 4);
        const uint32_t dO = tm + 256 + 128 * t;
#pragma unroll
        for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {   // 16 keys: 16 rows of 128 bytes
          const uint64_t bd = vd + ((kk * 2048) >> 4);
          tc_mma_ts(dO, tm + 128 * t + 8 * kk, bd, idesc_pv, (!first || kk > 0));
          if (LO) tc_mma_ts(dO, tm + 128 * t + 64 + 8 * kk, bd, idesc_pv, 1);
        }
      };
      // Waits for up to three barriers: lane 0, 1 and 2's.
      auto wait3 = [&](bool a, uint32_t bar_a, uint32_t par_a, bool b, uint32_t bar_b, uint32_t par_b, bool c,
                       uint32_t bar_c, uint32_t par_c) {
        const uint32_t bar = lane == 0 ? bar_a : lane == 1 ? bar_b : bar_c;
        const uint32_t par = lane == 0 ? par_a : lane == 1 ? par_b : par_c;
        const bool any = lane == 0 ? a : lane == 1 ? b : lane == 2 ? c : false;
        return pk_wait_lanes(any, bar, par, abort_flag);
      };
      int nt[2] = {0, 0}, nn[2] = {0, 0}, fl = 0, nfl = 0;   // lists of this item and the next
      constexpr int kFirst = 1, kEnds = 2;   // kEnds << t
      auto lists = [&](int i, int& a, int& b, int& f) {
        if (!pw_wait_all(smem_u32(&item_full[i & 1]), (i >> 1) & 1, abort_flag)) return false;
        const PkItem& it = items[i & 1];
        a = __shfl_sync(0xffffffffu, it.nt_a, 0);
        b = __shfl_sync(0xffffffffu, it.nt_b, 0);
        f = __shfl_sync(0xffffffffu, (it.j0 == 0 ? kFirst : 0) | (it.ends(0) ? kEnds : 0) |
                                         (it.ends(1) ? 2 * kEnds : 0), 0);
        return __shfl_sync(0xffffffffu, it.valid, 0) != 0;
      };
      bool ok = true, more = lists(0, nt[0], nt[1], fl);
      // ring position: stage and its phase, of the next tile to be waited for
      int st = 0;
      uint32_t st_ph = 0;
      auto advance = [&] {
        if (++st == STAGES) {
          st = 0;
          st_ph ^= 1;
        }
      };
      // the first item's first scores
      if (more && max(nt[0], nt[1]) > 0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || nt[t] == 0) continue;
          ok = wait3(true, smem_u32(&kv_full[0]), 0, true, smem_u32(&q_full[t]), 0, false, 0, 0);
          ph_q ^= 1u << t;
          if (!ok) break;
          tc_fence_after();
          if (pw_elect()) qk(t, 0, nt[t] == 1 && (fl & (kEnds << t)));
          __syncwarp();
        }
        if (ok && pw_elect()) tc_commit(smem_u32(&kv_empty[0]));
        __syncwarp();
        advance();
      }
      for (int i = 0; more && ok; ++i) {
        const int most = max(nt[0], nt[1]), steps = max(most, 1);
        bool go_on = false;
        int j = 0;
        // Steps in which both tiles have weights and next scores of this item: nearly all of a long list.
        const int plain = min(nt[0], nt[1]) - 1;
        if (plain > 0) {
          ok = wait3(true, smem_u32(&o_empty[0]), ph_o & 1, true, smem_u32(&o_empty[1]), ph_o >> 1, false, 0, 0);
          ph_o ^= 3u;
        }
        for (; j < plain && ok; ++j) {
          const int vs = st;
          const uint32_t v_ph = st_ph;
          advance();
          const int ks = st;
          const uint32_t k_ph = st_ph;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            ok = pk_wait2(smem_u32(&p_full[t][0]), (ph_p >> t) & 1, smem_u32(&kv_full[vs]), v_ph, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (pw_elect()) pv(t, vs, 0, j == 0);
            __syncwarp();
            ok = pk_wait2(smem_u32(&p_full[t][1]), (ph_p >> t) & 1, smem_u32(&kv_full[ks]), k_ph, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (pw_elect()) {
              pv(t, vs, 1, false);
              qk(t, ks, j + 2 == nt[t] && (fl & (kEnds << t)));
              if (t == 1) {   // both tiles are done with these
                tc_commit(smem_u32(&kv_empty[vs]));
                tc_commit(smem_u32(&kv_empty[ks]));
              }
            }
            __syncwarp();
          }
          ph_p ^= 3u;
          advance();
        }
        for (; j < steps && ok; ++j) {
          const bool last = j == steps - 1;
          if (last) go_on = lists(i + 1, nn[0], nn[1], nfl);
          // V_j, then K_(j+1) or the next item's K_0
          const int vs = st;
          const uint32_t v_ph = st_ph;
          if (most > 0) advance();
          const int ks = st;
          const uint32_t k_ph = st_ph;
          const bool any_k = !last || (go_on && max(nn[0], nn[1]) > 0);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool work = j < nt[t], need = last ? go_on && nn[t] > 0 : j + 1 < nt[t];
            const bool new_q = need && last && (nfl & kFirst);
            if (work) {
              ok = wait3(true, smem_u32(&p_full[t][0]), (ph_p >> t) & 1, true, smem_u32(&kv_full[vs]), v_ph,
                         j == 0, smem_u32(&o_empty[t]), (ph_o >> t) & 1);
              if (j == 0) ph_o ^= 1u << t;
              if (!ok) break;
              tc_fence_after();
              if (pw_elect()) pv(t, vs, 0, j == 0);
              __syncwarp();
            }
            if (work || need) {
              ok = wait3(work, smem_u32(&p_full[t][1]), (ph_p >> t) & 1, need, smem_u32(&kv_full[ks]), k_ph, new_q,
                         smem_u32(&q_full[t]), (ph_q >> t) & 1);
              if (work) ph_p ^= 1u << t;
              if (new_q) ph_q ^= 1u << t;
              if (!ok) break;
              tc_fence_after();
              if (pw_elect()) {
                if (work) {
                  pv(t, vs, 1, false);
                  if (j == nt[t] - 1) tc_commit(smem_u32(&o_full[t]));
                }
                if (need) qk(t, ks, last ? nn[t] == 1 && (nfl & (kEnds << t)) : j + 2 == nt[t] && (fl & (kEnds << t)));
                if (t == 1) {   // both tiles are done with these
                  if (most > 0) tc_commit(smem_u32(&kv_empty[vs]));
                  if (any_k) tc_commit(smem_u32(&kv_empty[ks]));
                }
              }
              __syncwarp();
            } else if (t == 1) {
              if (pw_elect()) {
                if (most > 0) tc_commit(smem_u32(&kv_empty[vs]));
                if (any_k) tc_commit(smem_u32(&kv_empty[ks]));
              }
              __syncwarp();
            }
          }
          if (any_k) advance();
        }
        if (ok && lane == 0) mbar_arrive(smem_u32(&item_empty[i & 1]));
        nt[0] = nn[0];
        nt[1] = nn[1];
        fl = nfl;
        more = go_on;
      }
      if (pw_elect()) tc_commit(smem_u32(&drain));   // its MMAs finish before TMEM is released
      __syncwarp();
      volatile int no_abort = 0;
      pw_wait(smem_u32(&drain), 0, &no_abort);
    } else if (warp == 17) {
      // ------------------------------ TMA loads -------------------------------
      if (pw_elect()) {
        PkItem it;
        bool ok = true;
        for (int i = 0; ok && next_item(i, it); ++i) {
          const int nt = it.most();
          for (int x = 0; x < 2 * nt && ok; ++x) {   // K_0, Q_A, Q_B, V_0, K_1, V_1, ...
            const int st = loads % STAGES;
            if (loads >= STAGES)
              ok = pw_wait(smem_u32(&kv_empty[st]), ((loads / STAGES) - 1) & 1, abort_flag);
            if (!ok) break;
            const uint32_t bar = smem_u32(&kv_full[st]);
            mbar_arrive_expect_tx(bar, LY::kTile);
            const int row = it.key0 + key_tile(it, it.j0 + (x >> 1)) * kPkKeys;
#pragma unroll
            for (int h = 0; h < SLABS; ++h)
              tma_load_3d(stage_at(loads) + h * kPkSlab, (x & 1) ? &tmap_v : &tmap_k, 64 * h, it.head, row,
                          bar);
            ++loads;
            if (x > 0 || it.j0 > 0) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || it.nt(t) == 0) continue;
              if (copied_q[t] > 0) ok = pw_wait(smem_u32(&q_empty[t]), (copied_q[t] - 1) & 1, abort_flag);
              if (!ok) break;
              const uint32_t qbar = smem_u32(&q_full[t]);
              mbar_arrive_expect_tx(qbar, SLABS * G * TQ * 128);
#pragma unroll
              for (int h = 0; h < SLABS; ++h)
                tma_load_3d(sma + t * LY::kTile + h * kPkSlab, &tmap_q, 64 * h, it.head * G, it.row0 + t * TQ,
                            qbar);
              ++copied_q[t];
            }
          }
          if (ok) mbar_arrive(smem_u32(&item_empty[i & 1]));
        }
      }
      loads = __reduce_max_sync(0xffffffffu, loads);
      copied_q[0] = __reduce_max_sync(0xffffffffu, copied_q[0]);
      copied_q[1] = __reduce_max_sync(0xffffffffu, copied_q[1]);
    } else if (warp == 18) {
      // ------------------------------- items ----------------------------------
      int32_t* pairs = reinterpret_cast<int32_t*>(sm + LY::kRankAt);
      PkOrder order{p, pairs, pairs + kPkRank, !p.causal,
                    p.window > 0 ? (p.window - 1) / (2 * TQ) + 2 : INT32_MAX / 4};
      order.lane = lane;
      order.fill(0, blockIdx.x == 0);
      const uint32_t n = gridDim.x;
      constexpr int kPart = F32 ? kPkPart : INT32_MAX / 2;
      PkItem it = {};
      bool found = false;
      int at = 0;      // of the unit at hand: entries handed out, and all of them
      int most = 0;
      uint32_t unit = 0;
      for (uint32_t i = 0;; ++i) {
        if (at >= most) {   // the next unit
          int s = 0, pair = 0, g = 0;
          const uint32_t u = unit * n + ((unit & 1) ? n - 1 - blockIdx.x : blockIdx.x);
          ++unit;
          found = order.find(u, blockIdx.x == 0, s, pair, g);
          it = {};
          at = most = 0;
          if (found) {
            const int q0 = __ldg(p.query_start + s), nq = __ldg(p.query_start + s + 1) - q0;
            it.key0 = __ldg(p.key_start + s);
            it.keys = __ldg(p.key_start + s + 1) - it.key0;
            const int tok0 = pair * 2 * TQ;
            it.valid = 1;
            it.row0 = q0 + tok0;
            it.tokens = nq - tok0;
            it.pos0 = it.keys - nq + tok0;
            it.head = g;
            auto tiles = [&](int t) {   // keys up to the last one that some row of the tile sees
              const int end = min(it.tokens, (t + 1) * TQ);
              const int seen = p.causal ? it.pos0 + end : it.keys;
              return end > t * TQ ? (max(seen, 0) + kPkKeys - 1) / kPkKeys : 0;
            };
            it.all_a = tiles(0);
            it.all_b = tiles(1);
            if (p.window > 0) {
              it.base = max(0, it.pos0 - p.window + 1) / kPkKeys;
              it.ns = min((min(p.sinks, it.keys) + kPkKeys - 1) / kPkKeys, it.base);
              if (it.all_a > 0) it.all_a += it.ns - it.base;
              if (it.all_b > 0) it.all_b += it.ns - it.base;
            }
            most = max(it.all_a, it.all_b);
          }
        }
        it.j0 = at;
        it.nt_a = min(max(it.all_a - at, 0), kPart);
        it.nt_b = min(max(it.all_b - at, 0), kPart);
        at += kPart;
        it.ragged = it.most() > 0 && (key_tile(it, it.j0 + it.most() - 1) + 1) * kPkKeys > it.keys;
        bool ok = true;
        if (i >= 2) ok = pw_wait_all(smem_u32(&item_empty[i & 1]), ((i >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          items[i & 1] = it;
          // its rows of q on their way to L2: there is room for them only when the item before has taken
          // its last scores (16 prompts of 512 tokens 66.1 -> 64.5 us; the other cases keep their times)
          if (i > 0 && it.valid && it.j0 == 0) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (it.nt(t) == 0) continue;
#pragma unroll
              for (int h = 0; h < SLABS; ++h)
                asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n" ::"l"(&tmap_q),
                             "r"(64 * h), "r"(it.head * G), "r"(it.row0 + t * TQ)
                             : "memory");
            }
          }
          mbar_arrive(smem_u32(&item_full[i & 1]));
        }
        __syncwarp();
        if (!found) break;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    // ---------------- softmax and epilogue (A: warps 0-7, B: 8-15) ---------------
    // Softmax: rows w0 + lane / 4 and 8 further, columns 2 (lane % 4) and the next one of every eight.
    const int t = warp >> 3, quad = (warp & 3) * 32, half = (warp >> 2) & 1, w0 = quad + 16 * half;
    const int c2 = 2 * (lane & 3);
    const uint32_t tS = tm + 128 * t + (static_cast<uint32_t>(w0) << 16);
    const uint32_t tO = tS + 256;
    const uint32_t g_inv = (65536u + G - 1) / G;   // row / G for row < 128: exact for G <= 128
    // raised to the smallest normal, so that a masked -inf stays -inf under it
    const float sl2 = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
    constexpr int esz = F32 ? 4 : 2;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};   // references (in log2 units), sums
    float ref[2] = {0.f, 0.f};   // references in the part before
    uint32_t n_s = 0, n_o = 0;   // score tiles and items done
    int entries = 0;         // ring entries of the items before
    PkItem it;
    bool alive = true;
    auto hand_over = [&](int part) {   // the part's weights are in TMEM
      pw_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[t][part]));
    };
    for (int i = 0; alive && __all_sync(0xffffffffu, next_item(i, it)); ++i) {
      const int my_nt = it.nt(t);
      int last[2], low[2], last_min = INT32_MAX - 1, low_max = INT32_MIN;   // keys that the rows see
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = w0 + (lane >> 2) + 8 * e, token = t * TQ + static_cast<int>((row * g_inv) >> 16);
        const int pos = it.pos0 + token;
        last[e] = p.causal ? pos : it.keys - 1;
        low[e] = p.window > 0 ? pos - p.window + 1 : 0;
        if (row < TQ * G && token < it.tokens) {
          last_min = min(last_min, last[e]);
          low_max = max(low_max, low[e]);
        }
        if (it.j0 == 0) {
          m[e] = -CUDART_INF_F;
          l[e] = 0.f;
        }
      }
      last_min = __reduce_min_sync(0xffffffffu, last_min);
      low_max = __reduce_max_sync(0xffffffffu, low_max);
      for (int j = 0; j < my_nt; ++j) {
        if (!pw_wait_all(smem_u32(&s_full[t]), n_s & 1, abort_flag)) {
          alive = false;
          break;
        }
        ++n_s;
        tc_fence_after();
        const int k0 = key_tile(it, it.j0 + j) * kPkKeys;
        float sv[64];
        const bool cut = k0 + kPkKeys > last_min + 1 || (k0 < low_max && k0 + kPkKeys > p.sinks);
        auto look = [&](int h, float (&mt)[2]) {   // 64 keys: those that the row sees, the largest scores
          float* x = sv + 32 * h;
          if (cut) {
            const int k = k0 + 64 * h;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint64_t seen = (pw_below(last[e] + 1 - k) & (~pw_below(low[e] - k) | pw_below(p.sinks - k))) >> c2;
              const uint32_t w[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
#pragma unroll
              for (int g = 0; g < 8; ++g) {
                float* y = x + 4 * g + 2 * e;
                y[0] = ((w[g >> 2] >> (8 * (g & 3))) & 1u) ? y[0] : -CUDART_INF_F;
                y[1] = ((w[g >> 2] >> (8 * (g & 3) + 1)) & 1u) ? y[1] : -CUDART_INF_F;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
            for (int g = 1; g < 7; g += 2) {
              a = pf_max3(a, x[4 * g + 2 * e], x[4 * g + 2 * e + 1]);
              b = pf_max3(b, x[4 * g + 4 + 2 * e], x[4 * g + 5 + 2 * e]);
            }
            mt[e] = pf_max3(a, b, fmaxf(x[28 + 2 * e], x[29 + 2 * e])) * sl2;
          }
        };
        // The references of rows with a score too far above theirs move: what is summed up so far is
        // scaled, `done` registers of this tile's weights among it.
        auto move = [&](float (&mt)[2], int done) {
          float alpha[2];
          bool resc = false;
#pragma unroll
          for (int e = 0; e < 2; ++e) {   // over the row's four lanes
            mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 1));
            mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], 2));
            const bool up = mt[e] > m[e] + kPkLag;
            alpha[e] = up ? pf_ex2(m[e] - mt[e]) : 1.f;
            resc = resc || (up && m[e] != -CUDART_INF_F);
            m[e] = up ? mt[e] : m[e];
            l[e] *= alpha[e];
          }
          if (done) {
#pragma unroll
            for (int n = 0; n < 32; ++n) sv[n] *= alpha[(n >> 1) & 1];
          }
          if (j > 0 && __any_sync(0xffffffffu, resc)) {   // (a part's first products begin a new O)
#pragma unroll 1
            for (int c = 0; c < p.dim; c += 16) pk_scale16(tO + c, alpha[0], alpha[1]);
            pw_st_wait();
          }
        };
        auto exps = [&](int h) {
          float* x = sv + 32 * h;
          const float mu[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
#pragma unroll
          for (int n = 0; n < 16; ++n) {   // register pair n: group n / 2, row n % 2
            const int e = n & 1;
            const float2 z = __ffma2_rn(make_float2(x[2 * n], x[2 * n + 1]), make_float2(sl2, sl2),
                                        make_float2(-mu[e], -mu[e]));
            x[2 * n] = pf_ex2(z.x);   // 2^-inf = 0 for masked keys
            x[2 * n + 1] = pf_ex2(z.y);
          }
        };
        pk_ld64(tS, sv);
        pk_ld64(tS + 64, sv + 32);
        pk_ld_wait(sv);
        float mt0[2], mt1[2];
        look(0, mt0);
        if (__any_sync(0xffffffffu, mt0[0] > m[0] + kPkLag || mt0[1] > m[1] + kPkLag)) move(mt0, 0);
        exps(0);
        pk_ld_wait(sv + 32);
        look(1, mt1);
        if (__any_sync(0xffffffffu, mt1[0] > m[0] + kPkLag || mt1[1] > m[1] + kPkLag)) move(mt1, 32);
        if (it.ragged && j == it.most() - 1) {
          // S is there, so every ring entry before this K tile has been seen to land: the phase waited for
          // is this V tile's
          const int vi = entries + 2 * j + 1, r = quad + lane;
          if (!pw_wait_all(kv_bar(vi), (vi / STAGES) & 1, abort_flag)) {
            alive = false;
            break;
          }
          if (r >= it.keys - k0) {
            uint8_t* v = sm + LY::kRing + (vi % STAGES) * LY::kTile + r * 128 + half * (SLABS == 2 ? kPkSlab : 64);
#pragma unroll
            for (int u = 0; u < 4 * SLABS; ++u) *reinterpret_cast<uint4*>(v + u * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        float2 ls[2][2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[16], wl[LO ? 16 : 1];
          const float* x = sv + 32 * h;
          const float mu[2] = {m[0] == -CUDART_INF_F ? 0.f : m[0], m[1] == -CUDART_INF_F ? 0.f : m[1]};
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            if (h == 0) {   // the second half's exponentials, between the first half's sums and conversions
              const float2 z = __ffma2_rn(make_float2(sv[32 + 2 * n], sv[33 + 2 * n]), make_float2(sl2, sl2),
                                          make_float2(-mu[n & 1], -mu[n & 1]));
              sv[32 + 2 * n] = pf_ex2(z.x);
              sv[33 + 2 * n] = pf_ex2(z.y);
            }
            const float2 y = make_float2(x[2 * n], x[2 * n + 1]);
            ls[n & 1][(n >> 1) & 1] = __fadd2_rn(ls[n & 1][(n >> 1) & 1], y);
            w[n] = pack_bf16(y.x, y.y);
            if constexpr (LO) {   // what the first part left
              const float2 lo = __ffma2_rn(make_float2(bf16_lo(w[n]), bf16_hi(w[n])), make_float2(-1.f, -1.f), y);
              wl[n] = pack_bf16(lo.x, lo.y);
            }
          }
          if (h == 1) hand_over(0);   // its stores are done by now
          pk_st32(tS + 32 * h, w);   // column c = keys 2c and 2c + 1
          if constexpr (LO) pk_st32(tS + 64 + 32 * h, wl);
          if (h == 1) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 all = __fadd2_rn(ls[e][0], ls[e][1]);
              l[e] += all.x + all.y;
            }
          }
        }
        hand_over(1);
      }
      if (!alive) break;
      entries += 2 * it.most();
      // Epilogue: the rows of the softmax, 64 columns at a time.  The four lanes of a row have two columns in
      // every eight each; they exchange them so that a store takes 128 bytes of a row (bf16) or 64 (f32) at a
      // time.  With a row per lane every store met 32 rows' lines: float32 outputs took up to a quarter longer
      // (16 prompts of 512 tokens, 32 heads 101 us for 80); bf16 ones are as fast, 2 % either way.
      if (my_nt > 0 || it.j0 == 0) {
        float inv[2] = {0.f, 0.f}, keep[2] = {0.f, 0.f};   // factors of O and of what earlier parts left
        if (my_nt > 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float sum = l[e] + __shfl_xor_sync(0xffffffffu, l[e], 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            inv[e] = !F32 || it.ends(t) ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
            if constexpr (F32) {   // the parts' references differ where the row's has moved
              keep[e] = ref[e] == m[e] ? inv[e] : pf_ex2(ref[e] - m[e]) * inv[e];
              ref[e] = m[e];
            }
          }
          if (!pw_wait_all(smem_u32(&o_full[t]), n_o & 1, abort_flag)) break;
          ++n_o;
          tc_fence_after();
        }
        uint8_t* dst[2];
        bool valid[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = w0 + (lane >> 2) + 8 * e, tk = static_cast<int>((row * g_inv) >> 16), token = t * TQ + tk;
          valid[e] = row < TQ * G && token < it.tokens;
          dst[e] = static_cast<uint8_t*>(p.out) +
                   ((static_cast<int64_t>(it.row0 + token) * p.num_q_heads + it.head * G + row - tk * G) * p.dim) * esz;
        }
        const bool odd = lane & 1, high = lane & 2;
#pragma unroll
        for (int h = 0; h < SLABS; ++h) {
          float v[32];
          if (my_nt > 0) {
            pk_ld64(tO + 64 * h, v);
            pk_ld_wait(v);
            if (h == SLABS - 1) {   // O has been read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&o_empty[t]));
            }
          } else {
#pragma unroll
            for (int n = 0; n < 32; ++n) v[n] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (!F32) {
              uint32_t w[8], x[8], y[8];   // column group g; then 2 (kept group) + source; then the lane's 32 bytes
#pragma unroll
              for (int g = 0; g < 8; ++g) w[g] = pack_bf16(v[4 * g + 2 * e] * inv[e], v[4 * g + 2 * e + 1] * inv[e]);
#pragma unroll
              for (int g = 0; g < 4; ++g) {   // groups 0 to 3 to the lower two lanes
                const uint32_t mine = high ? w[g + 4] : w[g];
                const uint32_t other = __shfl_xor_sync(0xffffffffu, high ? w[g] : w[g + 4], 2);
                x[2 * g] = high ? other : mine;
                x[2 * g + 1] = high ? mine : other;
              }
#pragma unroll
              for (int n = 0; n < 4; ++n) {   // and of these two the first ones to the even lane
                const uint32_t mine = odd ? x[n + 4] : x[n];
                const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? x[n] : x[n + 4], 1);
                y[2 * n] = odd ? other : mine;
                y[2 * n + 1] = odd ? mine : other;
              }
              const int col = 64 * h + 16 * (lane & 3);
              uint8_t* d = dst[e] + 2 * col;
              if (valid[e]) {
                if (col + 16 <= p.dim && (reinterpret_cast<uintptr_t>(d) & 31) == 0) {
                  pk_store32(d, y);
                } else {
                  if (col < p.dim) *reinterpret_cast<uint4*>(d) = make_uint4(y[0], y[1], y[2], y[3]);
                  if (col + 8 < p.dim) *reinterpret_cast<uint4*>(d + 16) = make_uint4(y[4], y[5], y[6], y[7]);
                }
              }
            } else {
              float4 rows[4], *to[4];
              bool there[4];
#pragma unroll
              for (int n = 0; n < 4; ++n) {   // even groups to the even lanes
                const int g = 2 * n, z = 4 * g + 2 * e;
                const float m0 = odd ? v[z + 4] : v[z], m1 = odd ? v[z + 5] : v[z + 1];
                const float o0 = __shfl_xor_sync(0xffffffffu, odd ? v[z] : v[z + 4], 1),
                            o1 = __shfl_xor_sync(0xffffffffu, odd ? v[z + 1] : v[z + 5], 1);
                float4 r = odd ? make_float4(o0, o1, m0, m1) : make_float4(m0, m1, o0, o1);
                r = make_float4(r.x * inv[e], r.y * inv[e], r.z * inv[e], r.w * inv[e]);
                const int col = 64 * h + 8 * (g + (lane & 1)) + 2 * (lane & 2);
                rows[n] = r;
                there[n] = valid[e] && col < p.dim;
                to[n] = reinterpret_cast<float4*>(dst[e] + 4 * col);
              }
              if (it.j0 > 0) {   // four reads at a time: more spill, fewer wait in turn
                float4 was[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) was[n] = there[n] ? *to[n] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                  rows[n] = make_float4(fmaf(was[n].x, keep[e], rows[n].x), fmaf(was[n].y, keep[e], rows[n].y),
                                        fmaf(was[n].z, keep[e], rows[n].z), fmaf(was[n].w, keep[e], rows[n].w));
              }
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (there[n]) *to[n] = rows[n];
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&item_empty[i & 1]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && warp == 17) {   // copies may be in flight: no role waits for them now
    volatile int no_abort = 0;
    for (int x = max(0, loads - STAGES); x < loads; ++x)
      pw_wait(kv_bar(x), (x / STAGES) & 1, &no_abort);
    for (int t = 0; t < 2; ++t)
      if (copied_q[t] > 0) pw_wait(smem_u32(&q_full[t]), (copied_q[t] - 1) & 1, &no_abort);
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tm) : "memory");
  if (tid == 0 && *abort_flag) flag_status(p.status, PKV_DEV_TIMEOUT);
}

}  // namespace pkv

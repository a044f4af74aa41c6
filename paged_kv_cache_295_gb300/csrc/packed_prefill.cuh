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
// next: while the last products of an item and its epilogue are under way, the next one's Q and first
// keys are loaded and its first scores computed.  Warps:
//   0-3, 4-7  softmax of tile A, of tile B (thread = row)
//   8-11      epilogue: O out of TMEM, divided by the row's sum, to global memory
//   12        issues the MMAs: PV_A(j), QK_A(j+1), PV_B(j), QK_B(j+1), so that one tile's softmax
//             runs under the other's products
//   13        TMA loads (Q_A, Q_B; a ring of K and V tiles)
//   14        finds the items: the u-th unit of the batch, longest first
//   15        clears the rows of a V tile past its sequence's end: they belong to another sequence,
//             and a weight of 0 times what is not finite would be NaN
// The running reference m moves only when a weight would exceed 2^kPkLag, so that O is hardly ever
// scaled; S_t(j) being there implies that PV_t(j-1) is done (one thread issues both), so the softmax
// warps scale it themselves.
//
// Every wait is bounded (2 s) and gives up when another role has given up; copies in flight are then
// waited for, and TMEM is released before the CTA exits.
#pragma once

#include "prefill_win.cuh"

namespace pkv {

constexpr int kPkRows = 128;      // accumulator rows of a query tile (M)
constexpr int kPkKeys = 128;      // keys of a tile (N of QK, K of PV)
constexpr int kPkThreads = 512;
constexpr int kPkRank = 1024;     // sequences whose items are ordered by length together
constexpr int kPkSlab = 128 * 128;   // 128 rows of 64 bf16 (128-byte swizzle)
// The reference m moves only when a weight would exceed 2^kPkLag: the weights, their sum and O are
// floating-point numbers of float32's range, in which a factor loses nothing, and with a lag of 24
// O is scaled for logits that grow by 16 from one key tile to another, where one of 8 has most
// short prompts' second tiles scale it (a first row of few keys is enough), at 1,500 cycles.
constexpr float kPkLag = 24.f;
// Key tiles after which a float32 output takes O up.  The tensor cores cut every sum towards zero:
// up to 2^-23 of O for each 16 keys and weight part, which adds up (20,000 keys in one go: 4.4e-5 of the
// norm); 8 tiles are 128 such sums.  In between the epilogue adds in float32, in the output's own rows.
constexpr int kPkPart = 8;
constexpr int kPkOut = 4 * 4096;     // epilogue: 32 rows of 128 bytes per warp

struct PackedParams {
  void* out;                    // [T, Hq, D]
  const int32_t* query_start;   // [S + 1]
  const int32_t* key_start;     // [S + 1]
  int32_t* status;
  int32_t num_seqs, num_tokens, num_keys;
  int32_t num_q_heads, num_kv_heads, dim;
  int32_t tile_tokens;          // TQ = 128 / G
  int32_t causal, window, sinks;
  int32_t out_bf16;
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
  static constexpr int kStage = kRing + STAGES * kTile;
  static constexpr int kRankAt = kStage + kPkOut;
  static constexpr size_t bytes() { return 1024 + kRankAt + kPkRank * 8; }
};

// 128 consecutive TMEM columns of this warp's 32 lanes -> 128 registers.
__device__ __forceinline__ void pk_ld128(uint32_t taddr, float* v) {
  uint32_t r[128];
#define PKV_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                  "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define PKV_LD32(i) \
  asm volatile( \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14," \
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n" \
      : PKV_R8(i), PKV_R8(i + 8), PKV_R8(i + 16), PKV_R8(i + 24) \
      : "r"(taddr + i))
  PKV_LD32(0);
  PKV_LD32(32);
  PKV_LD32(64);
  PKV_LD32(96);
#undef PKV_LD32
#undef PKV_R8
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 registers to 16 TMEM columns of this warp's lanes, without the wait.
__device__ __forceinline__ void pk_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// 16 TMEM columns of this warp's lanes, times f, without the wait for the stores (few registers: the
// scores are in the others).
__device__ __forceinline__ void pk_scale16(uint32_t taddr, float f) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  pk_st16(taddr, r);
}

// Warp 14: the items of one CTA.  Units (sequence, pair of query tiles, KV head) are ordered by
// the length of their key lists, longest first and KV heads fastest, within each kPkRank sequences;
// round k of a grid of n CTAs takes units kn .. kn + n - 1, every other round in the opposite
// order.  Order by counting: the units of sequence s that are at least x long are known in closed
// form, so the length of the u-th unit is found by halving.
struct PkOrder {
  const PackedParams& p;
  int32_t* pairs;    // shared, [kPkRank]: pairs of query tiles of a sequence
  int32_t* level;    // shared: length of its first pair, in pairs
  bool flat;         // all pairs of a sequence are alike
  int first = 0, count = 0, top = 0, lane;   // the sequences at hand; the longest unit
  uint32_t before = 0, total = 0;            // units before them; theirs

  __device__ __forceinline__ int longer(int i, int x) const {   // units of sequence i of level >= x
    return flat ? (level[i] >= x ? pairs[i] : 0) : min(max(level[i] + pairs[i] - x, 0), pairs[i]);
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
      int n = 0, lv = 0;
      if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || k0 < 0 || k1 < k0 || k1 > p.num_keys) {
        bad = true;
      } else {
        n = static_cast<int>((static_cast<int64_t>(q1) - q0 + per - 1) / per);
        const int c = k1 - k0;
        lv = flat ? (p.window > 0 ? 0 : c / per) : max(c - (q1 - q0), 0) / per;
      }
      pairs[i] = n;
      level[i] = lv;
      sum += n;
      if (n > 0) hi = max(hi, flat ? lv : lv + n - 1);
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
        pair = flat ? offset : lo - level[i0 + at];
        return true;
      }
      left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
};

// LO: the weights are two bf16 parts (float32 output).
template <int SLABS, int STAGES, bool LO>
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
  // by item slot: these roles may be one item ahead of the one that waits
  __shared__ __align__(8) uint64_t l_full[2][2], v_loading[2], v_clean[2];
  __shared__ PkItem items[2];
  __shared__ float row_sum[2][2][kPkRows], row_ref[LO ? 2 : 1][2][kPkRows];   // [item slot][tile]
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sma = smem_u32(sm);
  volatile int* abort_flag = &abort_sh;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == kPkThreads - 1) {
    for (int st = 0; st < STAGES; ++st) {
      mbar_init(smem_u32(&kv_full[st]), 1);
      mbar_init(smem_u32(&kv_empty[st]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&q_full[t]), 1);
      mbar_init(smem_u32(&q_empty[t]), 1);
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_full[t][0]), 4);
      mbar_init(smem_u32(&p_full[t][1]), 4);
      mbar_init(smem_u32(&o_full[t]), 1);
      mbar_init(smem_u32(&o_empty[t]), 4);
      mbar_init(smem_u32(&l_full[t][0]), 4);
      mbar_init(smem_u32(&l_full[t][1]), 4);
      mbar_init(smem_u32(&v_loading[t]), 1);
      mbar_init(smem_u32(&v_clean[t]), 1);
      mbar_init(smem_u32(&item_full[t]), 1);
      mbar_init(smem_u32(&item_empty[t]), 15);   // 8 softmax, 4 epilogue warps, 12, 13, 15
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
  int loads = 0, copied_q[2] = {0, 0};   // warp 13: copies started, K/V tiles and Q tiles

  // 512 threads of 128 registers; 2 x 128 x 184 + 128 x 80 + 128 x 64 = 512 x 128
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    if (warp == 12) {
      // ------------------------------ MMA issuer ------------------------------
      // The whole warp walks the lists, so that the compiler knows stages and descriptors uniform, and one
      // lane issues.
      const uint32_t idesc_qk = tc_idesc(kPkRows, kPkKeys, false, false, true);
      const uint32_t idesc_pv = tc_idesc(kPkRows, (p.dim + 15) & ~15, false, true, true);
      const int ksteps = (p.dim + 15) / 16;
      const uint64_t qd0 = tc_desc(sma, 0, 1024), kd0 = tc_desc(sma + LY::kRing, 0, 1024),
                     vd0 = tc_desc(sma + LY::kRing, kPkSlab, 1024);
      // phases gone by, one bit each: q_full[t], p_full[t], o_empty[t], v_clean[slot]
      uint32_t ph_q = 0, ph_p = 0, ph_o = 3, ph_c = 0;
      auto flip = [](uint32_t& bits, int b) {
        const uint32_t parity = (bits >> b) & 1;
        bits ^= 1u << b;
        return parity;
      };
      auto qk = [&](int t, int st, bool done) {   // `done`: the item's last scores of this tile
        tc_fence_after();
        if (pw_elect()) {
          const uint64_t qd = qd0 + ((t * LY::kTile) >> 4), kd = kd0 + ((st * LY::kTile) >> 4);
#pragma unroll
          for (int ks = 0; ks < 4 * SLABS; ++ks) {   // 16 dims: slab ks / 4, 32 bytes each
            const int at = ((ks >> 2) * kPkSlab + (ks & 3) * 32) >> 4;
            if (ks < ksteps) tc_mma(tm + 128 * t, qd + at, kd + at, idesc_qk, ks > 0);
          }
          tc_commit(smem_u32(&s_full[t]));
          if (done) tc_commit(smem_u32(&q_empty[t]));
        }
        __syncwarp();
      };
      int nt[2] = {0, 0}, nn[2] = {0, 0}, fl = 0, nfl = 0;   // lists of this item and the next
      constexpr int kRagged = 1, kFirst = 2, kEnds = 4;   // kEnds << t
      auto lists = [&](int i, int& a, int& b, int& r) {
        if (!pw_wait_all(smem_u32(&item_full[i & 1]), (i >> 1) & 1, abort_flag)) return false;
        const PkItem& it = items[i & 1];
        a = __shfl_sync(0xffffffffu, it.nt_a, 0);
        b = __shfl_sync(0xffffffffu, it.nt_b, 0);
        r = __shfl_sync(0xffffffffu, (it.ragged ? kRagged : 0) | (it.j0 == 0 ? kFirst : 0) |
                                         (it.ends(0) ? kEnds : 0) | (it.ends(1) ? 2 * kEnds : 0), 0);
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
        ok = pw_wait_all(smem_u32(&kv_full[0]), 0, abort_flag);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || nt[t] == 0) continue;
          ok = pw_wait_all(smem_u32(&q_full[t]), flip(ph_q, t), abort_flag);
          if (ok) qk(t, 0, nt[t] == 1 && (fl & (kEnds << t)));
        }
        if (ok && pw_elect()) tc_commit(smem_u32(&kv_empty[0]));
        __syncwarp();
        advance();
      }
      for (int i = 0; more && ok; ++i) {
        const int most = max(nt[0], nt[1]), steps = max(most, 1);
        bool go_on = false;
        for (int j = 0; j < steps && ok; ++j) {
          const bool last = j == steps - 1;
          if (last) go_on = lists(i + 1, nn[0], nn[1], nfl);
          // V_j, then K_(j+1) or the next item's K_0
          const int vs = st;
          const uint32_t v_ph = st_ph;
          if (most > 0) advance();
          const int ks = st;
          const uint32_t k_ph = st_ph;
          const bool any_k = last ? go_on && max(nn[0], nn[1]) > 0 : true;
          bool v_there = false, k_there = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) break;
            if (j < nt[t]) {
              const uint32_t pp = flip(ph_p, t);
              ok = pw_wait_all(smem_u32(&p_full[t][0]), pp, abort_flag);
              if (ok && !v_there) {
                ok = pw_wait_all(smem_u32(&kv_full[vs]), v_ph, abort_flag);
                if (ok && last && (fl & kRagged))
                  ok = pw_wait_all(smem_u32(&v_clean[i & 1]), flip(ph_c, i & 1), abort_flag);
                v_there = true;
              }
              if (ok && j == 0) ok = pw_wait_all(smem_u32(&o_empty[t]), flip(ph_o, t), abort_flag);
              const uint64_t vd = vd0 + ((vs * LY::kTile) >> 4);
              const uint32_t dO = tm + 256 + 128 * t;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                if (half == 1 && ok) ok = pw_wait_all(smem_u32(&p_full[t][1]), pp, abort_flag);
                if (!ok) break;
                tc_fence_after();
                if (pw_elect()) {
#pragma unroll
                  for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {   // 16 keys: 16 rows of 128 bytes
                    const uint64_t bd = vd + ((kk * 2048) >> 4);
                    tc_mma_ts(dO, tm + 128 * t + 8 * kk, bd, idesc_pv, (j > 0 || kk > 0));
                    if (LO) tc_mma_ts(dO, tm + 128 * t + 64 + 8 * kk, bd, idesc_pv, 1);
                  }
                  if (half == 1 && j == nt[t] - 1) tc_commit(smem_u32(&o_full[t]));
                }
                __syncwarp();
              }
              if (!ok) break;
            }
            const bool need = last ? go_on && nn[t] > 0 : j + 1 < nt[t];
            if (need) {
              if (!k_there) {
                ok = pw_wait_all(smem_u32(&kv_full[ks]), k_ph, abort_flag);
                k_there = true;
              }
              if (ok && last && (nfl & kFirst)) ok = pw_wait_all(smem_u32(&q_full[t]), flip(ph_q, t), abort_flag);
              if (!ok) break;
              qk(t, ks, last ? nn[t] == 1 && (nfl & (kEnds << t)) : j + 2 == nt[t] && (fl & (kEnds << t)));
            }
          }
          if (!ok) break;
          if (pw_elect()) {
            if (v_there) tc_commit(smem_u32(&kv_empty[vs]));
            if (k_there) tc_commit(smem_u32(&kv_empty[ks]));
          }
          __syncwarp();
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
    } else if (warp == 13) {
      // ------------------------------ TMA loads -------------------------------
      if (pw_elect()) {
        PkItem it;
        bool ok = true;
        for (int i = 0; ok && next_item(i, it); ++i) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || it.j0 > 0 || it.nt(t) == 0) continue;
            if (copied_q[t] > 0) ok = pw_wait(smem_u32(&q_empty[t]), (copied_q[t] - 1) & 1, abort_flag);
            if (!ok) break;
            const uint32_t bar = smem_u32(&q_full[t]);
            mbar_arrive_expect_tx(bar, SLABS * G * TQ * 128);
#pragma unroll
            for (int h = 0; h < SLABS; ++h)
              tma_load_3d(sma + t * LY::kTile + h * kPkSlab, &tmap_q, 64 * h, it.head * G,
                          it.row0 + t * TQ, bar);
            ++copied_q[t];
          }
          const int nt = it.most();
          for (int x = 0; x < 2 * nt && ok; ++x) {   // K_0, V_0, K_1, V_1, ...
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
          }
          if (ok && it.ragged) mbar_arrive(smem_u32(&v_loading[i & 1]));
          if (ok) mbar_arrive(smem_u32(&item_empty[i & 1]));
        }
      }
      loads = __reduce_max_sync(0xffffffffu, loads);
      copied_q[0] = __reduce_max_sync(0xffffffffu, copied_q[0]);
      copied_q[1] = __reduce_max_sync(0xffffffffu, copied_q[1]);
    } else if (warp == 14) {
      // ------------------------------- items ----------------------------------
      int32_t* pairs = reinterpret_cast<int32_t*>(sm + LY::kRankAt);
      PkOrder order{p, pairs, pairs + kPkRank, !p.causal || p.window > 0};
      order.lane = lane;
      order.fill(0, blockIdx.x == 0);
      const uint32_t n = gridDim.x;
      constexpr int kPart = LO ? kPkPart : INT32_MAX / 2;
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
          mbar_arrive(smem_u32(&item_full[i & 1]));
        }
        __syncwarp();
        if (!found) break;
      }
    } else {
      // ---------------- V rows past the sequence's end -> 0 --------------------
      // The loader says when the tile's copy is under way: the phase that its barrier then waits for is
      // this copy's, and not an earlier one of the same parity.
      PkItem it;
      int base = 0;
      uint32_t phase = 0;   // bit: of v_loading[slot]
      for (int i = 0; __all_sync(0xffffffffu, next_item(i, it)); ++i) {
        const int nt = it.most();
        if (it.ragged) {
          const int vi = base + 2 * (nt - 1) + 1;
          if (!pw_wait_all(smem_u32(&v_loading[i & 1]), (phase >> (i & 1)) & 1, abort_flag) ||
              !pw_wait_all(kv_bar(vi), (vi / STAGES) & 1, abort_flag))
            break;
          phase ^= 1u << (i & 1);
          const int from = it.keys - key_tile(it, it.j0 + nt - 1) * kPkKeys;
          uint8_t* v = sm + LY::kRing + (vi % STAGES) * LY::kTile;
          for (int u = lane; u < (kPkKeys - from) * 8; u += 32) {
#pragma unroll
            for (int h = 0; h < SLABS; ++h)
              *reinterpret_cast<uint4*>(v + h * kPkSlab + from * 128 + u * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&v_clean[i & 1]));
        }
        base += 2 * nt;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&item_empty[i & 1]));
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
    // ------------------------------ epilogue ----------------------------------
    // 128 bytes of each row at a time through shared memory, so that a store is of whole lines.
    const int w0 = (warp & 3) * 32;
    uint8_t* stage = sm + LY::kStage + (warp & 3) * 4096;
    const int esz = p.out_bf16 ? 2 : 4, cols = 128 / esz;
    const uint32_t g_inv = (65536u + G - 1) / G;   // row / G for row < 128: exact for G <= 128
    uint32_t phase_o = 0, phase_l = 0;   // bits: phases of o_full[t], of l_full[slot][t]
    float ref_a = 0.f, ref_b = 0.f;      // the row's reference in the part before
    PkItem it;
    for (int i = 0; __all_sync(0xffffffffu, next_item(i, it)); ++i) {
      bool ok = true;
#pragma unroll 1
      for (int t = 0; t < 2 && ok; ++t) {
        // rows of the sequence; those of an earlier part that this one adds nothing to are done
        if (t * TQ >= it.tokens || (it.j0 > 0 && it.nt(t) == 0)) continue;
        uint8_t* dst[8];   // rows 4 r + lane / 8, eight lanes each
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int row = w0 + 4 * r + (lane >> 3);
          const int tk = static_cast<int>((row * g_inv) >> 16), tok = t * TQ + tk;
          dst[r] = nullptr;
          if (row < TQ * G && tok < it.tokens)
            dst[r] = static_cast<uint8_t*>(p.out) + (lane & 7) * 16 +
                     (static_cast<int64_t>(it.row0 + tok) * p.num_q_heads + it.head * G + row - tk * G) *
                         (p.dim * esz);
        }
        const bool some = it.nt(t) > 0;
        float inv = 0.f, keep = 0.f;   // of O, of what earlier parts left
        if (some) {
          const int bl = (i & 1) * 2 + t;
          ok = pw_wait_all(smem_u32(&l_full[i & 1][t]), (phase_l >> bl) & 1, abort_flag) &&
               pw_wait_all(smem_u32(&o_full[t]), (phase_o >> t) & 1, abort_flag);
          if (!ok) break;
          phase_l ^= 1u << bl;
          phase_o ^= 1u << t;
          tc_fence_after();
          const float l = row_sum[i & 1][t][w0 + lane];
          inv = !LO || it.ends(t) ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
          if constexpr (LO) {   // the parts' references differ where the row's has moved
            const float ref = row_ref[i & 1][t][w0 + lane], was = t == 0 ? ref_a : ref_b;
            keep = was == ref ? inv : pf_ex2(was - ref) * inv;
            if (t == 0) ref_a = ref; else ref_b = ref;
          }
        }
        const uint32_t tO = tm + 256 + 128 * t + (static_cast<uint32_t>(w0) << 16);
        for (int c = 0; c < p.dim; c += cols) {
          for (int hf = 0; hf < cols; hf += 32) {
            float o[32];
            if (some) {
              tc_ld32(tO + c + hf, o);
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= inv;
            if (p.out_bf16) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(stage + swz(lane, hf / 8 + u)) =
                    make_uint4(pack_bf16(o[8 * u], o[8 * u + 1]), pack_bf16(o[8 * u + 2], o[8 * u + 3]),
                               pack_bf16(o[8 * u + 4], o[8 * u + 5]), pack_bf16(o[8 * u + 6], o[8 * u + 7]));
            } else {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                *reinterpret_cast<float4*>(stage + swz(lane, u)) =
                    make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
          if (some && c + cols >= p.dim) {   // O has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&o_empty[t]));
          }
          __syncwarp();
          const bool inside = c * esz + (lane & 7) * 16 < p.dim * esz;
          if (LO && it.j0 > 0) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const float f = __shfl_sync(0xffffffffu, keep, 4 * r + (lane >> 3));
              if (!dst[r] || !inside) continue;
              float4* d = reinterpret_cast<float4*>(dst[r] + c * esz);
              const float4 a = *d, b = *reinterpret_cast<const float4*>(stage + swz(4 * r + (lane >> 3), lane & 7));
              *d = make_float4(fmaf(a.x, f, b.x), fmaf(a.y, f, b.y), fmaf(a.z, f, b.z), fmaf(a.w, f, b.w));
            }
          } else if (inside) {
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (dst[r])
                *reinterpret_cast<uint4*>(dst[r] + c * esz) =
                    *reinterpret_cast<const uint4*>(stage + swz(4 * r + (lane >> 3), lane & 7));
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&item_empty[i & 1]));
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;\n");
    // -------------------- softmax warpgroups (A: 0-3, B: 4-7) -------------------
    const int t = warp >> 2, w0 = (warp & 3) * 32, r = w0 + lane;
    const uint32_t tS = tm + 128 * t + (static_cast<uint32_t>(w0) << 16);
    const uint32_t tO = tS + 256;
    const int my_token = t * TQ + r / G;
    const bool neg = p.scale_log2 < 0.f;
    // raised to the smallest normal, so that a masked -inf stays -inf under it
    const float sl2 = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
    float m = -CUDART_INF_F, l = 0.f;   // the row's reference (in log2 units) and sum
    int n_s = 0;   // score tiles done
    PkItem it;
    bool alive = true;
    for (int i = 0; alive && __all_sync(0xffffffffu, next_item(i, it)); ++i) {
      const int my_nt = it.nt(t);
      const bool row_ok = r < TQ * G && my_token < it.tokens;
      const int qpos = it.pos0 + my_token;
      const int last = p.causal ? qpos : it.keys - 1;               // last key that the row sees
      const int low = p.window > 0 ? qpos - p.window + 1 : 0;       // first key of its window
      const int last_min = __reduce_min_sync(0xffffffffu, row_ok ? last : INT32_MAX - 1);
      const int low_max = __reduce_max_sync(0xffffffffu, row_ok ? low : INT32_MIN);
      if (it.j0 == 0) {
        m = -CUDART_INF_F;
        l = 0.f;
      }
      for (int j = 0; j < my_nt; ++j) {
        if (!pw_wait_all(smem_u32(&s_full[t]), n_s & 1, abort_flag)) {
          alive = false;
          break;
        }
        ++n_s;
        tc_fence_after();
        const int k0 = key_tile(it, it.j0 + j) * kPkKeys;
        float sv[kPkKeys];
        pk_ld128(tS, sv);
        if (neg) {
#pragma unroll
          for (int c = 0; c < kPkKeys; ++c) sv[c] = -sv[c];
        }
        if (k0 + kPkKeys > last_min + 1 || (k0 < low_max && k0 + kPkKeys > p.sinks)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // bits of the keys that the row sees
            const int k = k0 + 64 * h;
            const uint64_t seen = pw_below(last + 1 - k) & (~pw_below(low - k) | pw_below(p.sinks - k));
            const uint32_t w[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
#pragma unroll
            for (int c = 0; c < 64; ++c)
              sv[64 * h + c] = ((w[c >> 5] >> (c & 31)) & 1u) ? sv[64 * h + c] : -CUDART_INF_F;
          }
        }
        float ma = sv[0], mb = sv[1];
#pragma unroll
        for (int c = 2; c + 3 < kPkKeys; c += 4) {
          ma = pf_max3(ma, sv[c], sv[c + 1]);
          mb = pf_max3(mb, sv[c + 2], sv[c + 3]);
        }
        const float mt = fmaxf(pf_max3(ma, sv[kPkKeys - 2], sv[kPkKeys - 1]), mb) * sl2;
        float alpha = 1.f;
        bool resc = false;
        if (mt > m + kPkLag) {
          if (m != -CUDART_INF_F) {
            alpha = pf_ex2(m - mt);
            resc = j > 0;   // a part's first products begin a new O
          }
          m = mt;
        }
        const float mu = m == -CUDART_INF_F ? 0.f : m;   // rows with nothing seen yet: p = 0
        if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int c = 0; c < p.dim; c += 16) pk_scale16(tO + c, alpha);
          pw_st_wait();
        }
        float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int part = 0; part < 4; ++part) {   // 32 keys at a time: 16 registers of weights
          uint32_t w[16];
          float* x = sv + 32 * part;
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 z = __ffma2_rn(make_float2(x[c], x[c + 1]), make_float2(sl2, sl2),
                                        make_float2(-mu, -mu));
            const float2 y = make_float2(pf_ex2(z.x), pf_ex2(z.y));   // 2^-inf = 0 for masked keys
            ls[(c >> 1) & 1] = __fadd2_rn(ls[(c >> 1) & 1], y);
            w[c >> 1] = pack_bf16(y.x, y.y);
            if constexpr (LO) {
              x[c] = y.x;
              x[c + 1] = y.y;
            }
          }
          pk_st16(tS + 16 * part, w);   // row = lane, column c = keys 2c and 2c + 1
          if constexpr (LO) {   // what the first part left
            uint32_t wl[16];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float2 lo = __ffma2_rn(make_float2(bf16_lo(w[c >> 1]), bf16_hi(w[c >> 1])),
                                           make_float2(-1.f, -1.f), make_float2(x[c], x[c + 1]));
              wl[c >> 1] = pack_bf16(lo.x, lo.y);
            }
            pk_st16(tS + 64 + 16 * part, wl);
          }
          if (part == 3) {
            l = l * alpha + ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y));
            if (j == my_nt - 1) {
              row_sum[i & 1][t][r] = l;
              if constexpr (LO) row_ref[i & 1][t][r] = m;
            }
          }
          if (part & 1) {
            pw_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(&p_full[t][part >> 1]));
              if (part == 3 && j == my_nt - 1) mbar_arrive(smem_u32(&l_full[i & 1][t]));
            }
          }
        }
      }
      if (!alive) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&item_empty[i & 1]));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && warp == 13) {   // copies may be in flight: no role waits for them now
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

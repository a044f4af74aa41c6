// slots_from_lengths: block tables and slots of a step's new tokens from the request lengths, on
// the device ("LLM inference tutorial" section 4.2 append_token: a new block at every multiple of
// block_size, slot = table[p / bs] * bs + p % bs; blocks from the front of the free list, in the
// order of the sequences).
//
// With need_s = blocks that sequence s lacks and n_s its new tokens, two exclusive prefix sums give
// where its blocks begin in the free list and its rows in the outputs; every row is then
// independent of the others: a search in the starts finds its sequence.
//
// What bounds it: latency.  A step's lists are 16 to 800 KB, 0.12 us of HBM's time at the most; the launch,
// two dependent loads (length, then table or free list), the scan and the search are the rest.  So one
// launch does it: every CTA scans all lengths itself (a thousand sequences at a time, one a
// thread), so that nothing waits for another CTA's sums, and fills its share of the rows.  Where the new
// lengths (or the free list's new start) take the old ones' place, the CTAs are one cluster, whose
// barrier stands between the last read and the first write.
//
// Measured: 8 sequences of one token 3.6 us, 512 of them 4.2 us, 64 prompts and chunks of up to 2,047 tokens
// (66,000 rows) 4.9 us, and 11 in place: a barrier spans one cluster, so that eight CTAs write what 32 do.
#include "common.cuh"
#include "ranges.cuh"

namespace pkv {
namespace {

constexpr int kSlThreads = 1024;
constexpr int kSlCluster = 8;          // CTAs of a portable cluster
constexpr int kSlRowsPerCta = 2048;    // below this many rows a CTA more does not pay

struct SlotsParams {
  int32_t* tables;
  const int32_t* ctx;
  const int32_t* new_lens;
  const int32_t* free_blocks;
  const int32_t* free_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* query_start;
  int32_t* ctx_out;
  int32_t* free_next;
  int32_t* status;
  int64_t num_blocks;
  int32_t num_seqs, num_tokens, num_free, block_size, max_blocks, row_per_seq, first_held;
};

struct Request {
  int32_t ctx, held;
  int64_t rows, need;   // rows that it owns; blocks that it lacks
  bool ok;              // gets slots
};

__device__ __forceinline__ Request read_request(const SlotsParams& p, int s) {
  Request r = {0, 0, 0, 0, false};
  if (s >= p.num_seqs) return r;
  r.ctx = p.ctx[s];
  const int32_t n = p.new_lens ? p.new_lens[s] : 1;
  const int64_t bs = p.block_size;
  r.rows = p.row_per_seq ? 1 : max(n, 0);
  r.ok = r.ctx >= 0 && n >= 0 && (!p.row_per_seq || n <= 1) &&
         static_cast<int64_t>(r.ctx) + n <= bs * p.max_blocks;
  if (r.ok) {
    const int64_t held = max((r.ctx + bs - 1) / bs, static_cast<int64_t>(p.first_held));
    r.held = static_cast<int32_t>(held);
    r.need = max((r.ctx + static_cast<int64_t>(n) + bs - 1) / bs - held, static_cast<int64_t>(0));
  }
  return r;
}

// The CTA's barrier, or the cluster's.
template <bool CLUSTER>
__device__ __forceinline__ void all_read() {
  if constexpr (CLUSTER)
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  else
    __syncthreads();
}

// Inclusive sums over the CTA of (rows, need); their totals too.
__device__ __forceinline__ void scan2(int64_t& rows, int64_t& need, int64_t& all_rows,
                                      int64_t& all_need, int64_t (*sh)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, rows, o), b = __shfl_up_sync(0xffffffffu, need, o);
    if (lane >= o) {
      rows += a;
      need += b;
    }
  }
  if (lane == 31) {
    sh[warp][0] = rows;
    sh[warp][1] = need;
  }
  __syncthreads();
  int64_t a = sh[lane][0], b = sh[lane][1];   // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  all_rows = __shfl_sync(0xffffffffu, a, 31);
  all_need = __shfl_sync(0xffffffffu, b, 31);
  const int64_t before_r = __shfl_sync(0xffffffffu, a, max(warp - 1, 0)),
                before_n = __shfl_sync(0xffffffffu, b, max(warp - 1, 0));
  if (warp > 0) {
    rows += before_r;
    need += before_n;
  }
  __syncthreads();   // sh may be written again
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kSlThreads, 1) slots_kernel(const __grid_constant__ SlotsParams p) {
  __shared__ int64_t sh[32][2];
  __shared__ int32_t start_sh[kSlThreads + 1], base_sh[kSlThreads], ctx_sh[kSlThreads],
      held_sh[kSlThreads];   // held -1: no slots
  const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x;
  grid_dependency_wait();
  allow_dependents();

  // totals of the whole batch: all or nothing
  int64_t all_rows = 0, all_need = 0;
  Request mine = {0, 0, 0, 0, false};
  int64_t in_rows = 0, in_need = 0;   // inclusive sums of this tile
  bool bad = false;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kSlThreads) {
    mine = read_request(p, s0 + tid);
    bad = bad || (s0 + tid < p.num_seqs && !mine.ok);
    in_rows = mine.rows;
    in_need = mine.need;
    int64_t r, n;
    scan2(in_rows, in_need, r, n, sh);
    all_rows += r;
    all_need += n;
  }
  if (bad && cta == 0) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  const int64_t first_free = p.free_start ? *p.free_start : 0;
  const bool few_blocks = all_need > 0 && (first_free < 0 || first_free + all_need > p.num_free);
  const bool many_rows = all_rows > p.num_tokens;
  const bool go = !few_blocks && !many_rows;
  if (cta == 0 && tid == 0) {
    if (few_blocks) flag_status(p.status, PKV_DEV_NO_FREE_BLOCK);
    if (many_rows) flag_status(p.status, PKV_DEV_BAD_CONTEXT);
  }

  const int64_t bs = p.block_size;
  int64_t rows0 = 0, need0 = first_free;   // before this tile of sequences
  for (int s0 = 0; s0 < p.num_seqs; s0 += kSlThreads) {
    const int ns = min(kSlThreads, p.num_seqs - s0);
    int64_t tile_rows = all_rows, tile_need = all_need;
    if (p.num_seqs > kSlThreads) {   // one tile: the scan above is this one's
      mine = read_request(p, s0 + tid);
      in_rows = mine.rows;
      in_need = mine.need;
      scan2(in_rows, in_need, tile_rows, tile_need, sh);
    }
    if (go && tid < ns) {
      start_sh[tid] = static_cast<int32_t>(rows0 + in_rows - mine.rows);
      base_sh[tid] = static_cast<int32_t>(need0 + in_need - mine.need);
      ctx_sh[tid] = mine.ctx;
      held_sh[tid] = mine.ok ? mine.held : -1;
    }
    if (go && tid == 0) start_sh[ns] = static_cast<int32_t>(rows0 + tile_rows);
    all_read<CLUSTER>();   // this tile's lengths (and the free list's start)
    if (cta == 0 && tid < ns) {
      const int s = s0 + tid;
      int32_t n = 0;
      if (go && mine.ok)
        n = p.row_per_seq ? (p.new_lens ? p.new_lens[s] : 1) : static_cast<int32_t>(mine.rows);
      if (p.ctx_out) p.ctx_out[s] = mine.ctx + n;
      if (p.query_start && !p.row_per_seq) p.query_start[s] = go ? start_sh[tid] : 0;
    }
    if (go) {
      const int32_t row_end = start_sh[ns];
      for (int64_t row = start_sh[0] + cta * static_cast<int64_t>(kSlThreads) + tid; row < row_end;
           row += static_cast<int64_t>(ctas) * kSlThreads) {
        int lo = 0, hi = ns - 1;   // the last sequence that begins at or before the row
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (start_sh[mid] <= row) lo = mid; else hi = mid - 1;
        }
        const int s = s0 + lo;
        const int32_t held = held_sh[lo];
        const bool there = held >= 0 && (!p.row_per_seq || !p.new_lens || p.new_lens[s] == 1);
        int64_t slot = -1;
        int32_t pos = 0;
        if (there) {
          pos = ctx_sh[lo] + static_cast<int32_t>(row - start_sh[lo]);
          const int32_t lb = pos / p.block_size, off = pos - lb * p.block_size;
          int32_t* entry = p.tables + static_cast<int64_t>(s) * p.max_blocks + lb;
          int32_t blk;
          if (lb < held) {
            blk = *entry;
          } else {
            blk = p.free_blocks[base_sh[lo] + lb - held];
            if (off == 0) *entry = blk;
          }
          if (blk >= 0 && blk < p.num_blocks)
            slot = blk * bs + off;
          else
            flag_status(p.status, PKV_DEV_BAD_BLOCK);
        }
        p.slots[row] = slot;
        if (p.positions) p.positions[row] = pos;
      }
    }
    rows0 += tile_rows;
    need0 += tile_need;
    __syncthreads();   // the tile's arrays are written again
  }
  if (p.num_seqs == 0) all_read<CLUSTER>();
  if (cta == 0 && tid == 0) {
    if (p.free_next) *p.free_next = static_cast<int32_t>(first_free + (go ? all_need : 0));
    if (p.query_start && !p.row_per_seq) p.query_start[p.num_seqs] = go ? static_cast<int32_t>(all_rows) : 0;
  }
  // rows without a token
  for (int64_t row = (go ? all_rows : 0) + cta * static_cast<int64_t>(kSlThreads) + tid;
       row < p.num_tokens; row += static_cast<int64_t>(ctas) * kSlThreads) {
    p.slots[row] = -1;
    if (p.positions) p.positions[row] = 0;
  }
}


}  // namespace
}  // namespace pkv

extern "C" pkv_status slots_from_lengths(
    int32_t* block_tables, const int32_t* context_lens, const int32_t* new_lens,
    const int32_t* free_blocks, const int32_t* free_start, int32_t num_seqs, int32_t num_tokens,
    int32_t num_free, int64_t num_blocks, int32_t block_size, int32_t max_blocks_per_seq,
    int32_t row_per_sequence, int32_t first_block_held, int64_t* slot_mapping, int32_t* positions,
    int32_t* query_start, int32_t* context_out, int32_t* free_next, int32_t* device_status,
    pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || num_free < 0 || num_blocks <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || (row_per_sequence != 0 && row_per_sequence != 1) ||
      (first_block_held != 0 && first_block_held != 1))
    return PKV_ERR_INVALID_ARG;
  if (row_per_sequence && num_tokens < num_seqs) return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size > INT32_MAX) return PKV_ERR_INVALID_ARG;
  if (num_blocks > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 0 && (!block_tables || !context_lens)) return PKV_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_blocks) || (num_tokens > 0 && !slot_mapping)) return PKV_ERR_INVALID_ARG;
  for (const void* ptr : {static_cast<const void*>(block_tables), static_cast<const void*>(context_lens),
                          static_cast<const void*>(new_lens), static_cast<const void*>(free_blocks),
                          static_cast<const void*>(free_start), static_cast<const void*>(positions),
                          static_cast<const void*>(query_start), static_cast<const void*>(context_out),
                          static_cast<const void*>(free_next), static_cast<const void*>(device_status)})
    if (!aligned4(ptr)) return PKV_ERR_INVALID_ARG;
  if (!aligned_to(slot_mapping, 8)) return PKV_ERR_INVALID_ARG;

  SlotsParams p{block_tables, context_lens, new_lens, free_blocks, free_start, slot_mapping,
                positions, query_start, context_out, free_next, device_status, num_blocks,
                num_seqs, num_tokens, num_free, block_size, max_blocks_per_seq, row_per_sequence,
                first_block_held};
  // what is written overlaps nothing else, but for the two pairs that may be the same array
  const size_t len = 4 * static_cast<size_t>(num_seqs);
  struct Range {
    const void* ptr;
    size_t bytes;
  };
  const Range arrays[] = {{context_out, len}, {free_next, 4}, {block_tables, len * max_blocks_per_seq},
                          {slot_mapping, 8 * static_cast<size_t>(num_tokens)},
                          {positions, 4 * static_cast<size_t>(num_tokens)},
                          {row_per_sequence ? nullptr : query_start, len + 4},
                          {device_status, 4},   // the last one that is written
                          {context_lens, len}, {new_lens, len}, {free_start, 4},
                          {free_blocks, 4 * static_cast<size_t>(num_free)}};
  for (int i = 0; i < 7; ++i)
    for (int j = i + 1; j < 11; ++j)
      if (overlap(arrays[i].ptr, arrays[i].bytes, arrays[j].ptr, arrays[j].bytes) &&
          !(arrays[i].ptr == arrays[j].ptr && ((i == 0 && j == 7) || (i == 1 && j == 9))))
        return PKV_ERR_INVALID_ARG;
  const bool in_place = (len > 0 && context_out == context_lens) || (free_next && free_next == free_start);
  int64_t ctas = (static_cast<int64_t>(num_tokens) + kSlRowsPerCta - 1) / kSlRowsPerCta;
  if (ctas > 1 && in_place) {   // 66,000 rows: 10.8 us by eight CTAs, 4.9 by one for each 2,048
    ctas = ctas <= 2 ? 2 : ctas <= 4 ? 4 : kSlCluster;
  } else {
    const int64_t sms = device_sm_count();
    ctas = ctas < 1 ? 1 : ctas > sms ? sms : ctas;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kSlThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = in_place && ctas > 1 ? 2 : 1;
  return cuda_status(in_place && ctas > 1 ? cudaLaunchKernelEx(&cfg, slots_kernel<true>, p)
                                          : cudaLaunchKernelEx(&cfg, slots_kernel<false>, p));
}

// Launch helpers of the windowed decode kernel, shared by the 16-bit and the
// 8-bit translation units.
#pragma once

#include "decode_win.cuh"
#include "tmap.cuh"

namespace pkv {

template <typename KV, int D, bool QF32, bool HL, int NW, int STAGES, int CH>
pkv_status launch_win_shape(const WinLaunch& a, const CUtensorMap& tk, const CUtensorMap& tv) {
  using SM = WinSmem<KV, D, NW, STAGES, CH>;
  const WinParams& w = a.w;
  const int boxes = w.p.partition_tokens >> w.box_log2;
  const size_t smem = SM::bytes(boxes);
  if (smem > 227 * 1024) return PKV_ERR_UNSUPPORTED;
  auto kern = paged_decode_win_kernel<KV, D, QF32, HL, NW, STAGES, CH>;
  if (!opt_in_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem)))
    return PKV_ERR_CUDA;
  const dim3 grid(w.p.num_kv_heads * w.head_split, w.p.max_parts, a.num_seqs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = w.cluster ? w.p.max_parts : 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = w.cluster ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, tk, tv, w) != cudaSuccess) return PKV_ERR_CUDA;
  if (w.p.max_parts > 1 && !w.cluster &&
      launch_pdl(paged_decode_win_reduce_kernel<D>, dim3(a.num_seqs * w.p.num_q_heads), dim3(32), 0,
                 a.stream, w) != cudaSuccess)
    return PKV_ERR_CUDA;
  return PKV_OK;
}

inline bool win_maps(const WinLaunch& a, CUtensorMap* tk, CUtensorMap* tv) {
  const DecodeParams& p = a.w.p;
  const int64_t rows = a.num_blocks << p.bs_log2;
  const bool byte_codes = a.kv_dtype != PKV_BF16;
  return make_map(tk, p.k_cache, a.head_dim, p.num_kv_heads, rows, 1 << a.w.box_log2, byte_codes) &&
         make_map(tv, p.v_cache, a.head_dim, p.num_kv_heads, rows, 1 << a.w.box_log2, byte_codes);
}

}  // namespace pkv

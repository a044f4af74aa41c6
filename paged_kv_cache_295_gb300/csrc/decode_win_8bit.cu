// Windowed decode over FP8-E4M3 and INT8 caches (scales per block or per head).
#include "decode_win_launch.cuh"

namespace pkv {
namespace {

template <typename KV>
pkv_status pick(const WinLaunch& a, const CUtensorMap& tk, const CUtensorMap& tv) {
  // INT8 codes with a bf16 output: one weight part and codes with their offset, 2 to 10 % faster
  // than two parts and exact codes (which cost FP8 under 2 %)
  if constexpr (std::is_same<KV, INT8>::value)
    if (a.w.out_bf16)
      return a.q_f32 ? launch_win_shape<KV, 128, true, false, 4, 2, 32>(a, tk, tv)
                     : launch_win_shape<KV, 128, false, false, 4, 2, 32>(a, tk, tv);
  return a.q_f32 ? launch_win_shape<KV, 128, true, true, 4, 2, 32>(a, tk, tv)
                 : launch_win_shape<KV, 128, false, true, 4, 2, 32>(a, tk, tv);
}

}  // namespace

pkv_status launch_decode_win_8bit(const WinLaunch& a) {
  CUtensorMap tk, tv;
  if (!win_maps(a, &tk, &tv)) return PKV_ERR_CUDA;
  return a.kv_dtype == PKV_FP8_E4M3 ? pick<FP8>(a, tk, tv) : pick<INT8>(a, tk, tv);
}

}  // namespace pkv

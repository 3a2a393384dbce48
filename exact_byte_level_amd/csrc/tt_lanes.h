// tt_lanes.h -- what the lanes of a wavefront do with each other's values without LDS.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

namespace tt {
namespace {

constexpr int WAVE = 64;

typedef unsigned long long u64;

// What the lanes `CTRL` says (of the rows of 16 in ROWS) hold of v, 0 where there are none.
template <int CTRL, int ROWS>
__device__ inline uint32_t from_lanes(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ inline float from_lanes(float v) {
  return __uint_as_float(from_lanes<CTRL, ROWS>(__float_as_uint(v)));
}
template <int CTRL, int ROWS>
__device__ inline u64 from_lanes(u64 v) {
  return (u64)from_lanes<CTRL, ROWS>((uint32_t)(v >> 32)) << 32 | from_lanes<CTRL, ROWS>((uint32_t)v);
}
template <int CTRL, int ROWS>
__device__ inline double from_lanes(double v) {
  return __longlong_as_double((long long)from_lanes<CTRL, ROWS>((u64)__double_as_longlong(v)));
}
__device__ inline uint32_t of_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ inline float of_lane(float v, int lane) { return __uint_as_float(of_lane(__float_as_uint(v), lane)); }
__device__ inline u64 of_lane(u64 v, int lane) { return (u64)of_lane((uint32_t)(v >> 32), lane) << 32 | of_lane((uint32_t)v, lane); }
__device__ inline double of_lane(double v, int lane) { return __longlong_as_double((long long)of_lane((u64)__double_as_longlong(v), lane)); }

// op over the lanes up to each, of values whose op with 0 leaves them: shifts by 1, 2, 4, 8 in rows of 16, then the last lanes of
// rows 0 and 2, then of row 1.
template <class V, class Op>
__device__ inline V upto_lane(V v, Op op) {
  v = op(v, from_lanes<0x111, 0xf>(v));
  v = op(v, from_lanes<0x112, 0xf>(v));
  v = op(v, from_lanes<0x114, 0xf>(v));
  v = op(v, from_lanes<0x118, 0xf>(v));
  v = op(v, from_lanes<0x142, 0xa>(v));
  return op(v, from_lanes<0x143, 0xc>(v));
}
template <class V>
__device__ inline V sums_upto(V v) {
  return upto_lane(v, [](V x, V y) { return x + y; });
}
template <class V>
__device__ inline V sum_of_lanes(V v) {
  return of_lane(sums_upto(v), WAVE - 1);
}
template <class V>
__device__ inline V max_of_lanes(V v) {
  return of_lane(upto_lane(v, [](V x, V y) { return x > y ? x : y; }), WAVE - 1);
}

// What the lane whose number differs in bit APART holds.
template <int APART>
__device__ inline uint32_t across(uint32_t v) {
  const auto dpp = [](uint32_t x, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(ctrl)::value, 0xf, 0xf, false);
  };
  if constexpr (APART == 1) return dpp(v, std::integral_constant<int, 0xB1>());         // within four: 1 0 3 2
  else if constexpr (APART == 2) return dpp(v, std::integral_constant<int, 0x4E>());    // 2 3 0 1
  else if constexpr (APART == 4)
    return dpp(dpp(v, std::integral_constant<int, 0x141>()), std::integral_constant<int, 0x1B>());  // eight mirrored, then four
  else if constexpr (APART == 8) return dpp(v, std::integral_constant<int, 0x128>());   // sixteen turned by eight
  else if constexpr (APART == 16) {  // rows of 16 exchanged between two copies: the even ones twice, the odd ones twice
    const auto both = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? both[0] : both[1];
  } else {
    const auto both = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & 32 ? both[0] : both[1];
  }
}

// One exchange of a bitonic sort: the first of the two takes the larger key, in every second run the smaller.
template <int APART>
__device__ inline u64 exchanged(u64 key, int tid, int run) {
  const u64 other = (u64)across<APART>((uint32_t)(key >> 32)) << 32 | across<APART>((uint32_t)key);
  return (!(tid & APART) == !(tid & run)) == (other > key) ? other : key;
}

// The exchanges of a run between threads of a wavefront.
__device__ inline u64 exchanged_in_wave(u64 key, int tid, int run) {
  if (run > 32) key = exchanged<32>(key, tid, run);
  if (run > 16) key = exchanged<16>(key, tid, run);
  if (run > 8) key = exchanged<8>(key, tid, run);
  if (run > 4) key = exchanged<4>(key, tid, run);
  if (run > 2) key = exchanged<2>(key, tid, run);
  return exchanged<1>(key, tid, run);
}

}  // namespace
}  // namespace tt

// Reading logits of any of the three types, and what else the language-model operators
// share (k_tokens.hip, k_route.hip, k_vocab.hip).
#pragma once

#include "launch.h"
#include "profk_device.h"

namespace profk {

struct Half16 { unsigned short bits; };   // IEEE binary16
struct Brain16 { unsigned short bits; };  // bfloat16

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Half16 v) {
  _Float16 h;
  __builtin_memcpy(&h, &v.bits, 2);
  return (float)h;
}
__device__ __forceinline__ float to_f32(Brain16 v) { return __uint_as_float((u32)v.bits << 16); }

// Rounds to the nearest value of the type, ties to even (what torch's casts do).
__device__ __forceinline__ void from_f32(float v, float& out) { out = v; }
__device__ __forceinline__ void from_f32(float v, Half16& out) {
  const _Float16 h = (_Float16)v;
  __builtin_memcpy(&out.bits, &h, 2);
}
__device__ __forceinline__ void from_f32(float v, Brain16& out) {
  const __bf16 b = (__bf16)v;  // one instruction on gfx950
  __builtin_memcpy(&out.bits, &b, 2);
}

constexpr float kNone = -__builtin_huge_valf();

// The largest of three, as one instruction also where the compiler cannot know that none
// is a signalling NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Entries of -inf in the words of a load.
template <class T> struct NoneWord { static constexpr u32 value = 0xFF800000u; };
template <> struct NoneWord<Half16> { static constexpr u32 value = 0xFC00FC00u; };
template <> struct NoneWord<Brain16> { static constexpr u32 value = 0xFF80FF80u; };

// A barrier that waits for LDS accesses alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Sum / maximum over the G lanes of a group; every lane gets the result.  Within 16 lanes
// the partner is a mirrored one, which holds the same partial result as the one across.
template <int CTRL, class V>
__device__ __forceinline__ V dpp(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int G, class V, class F>
__device__ __forceinline__ V group_reduce(V v, F f) {
  if constexpr (G > 1) v = f(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
  if constexpr (G > 2) v = f(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  if constexpr (G > 4) v = f(v, dpp<0x141>(v));   // row_half_mirror
  if constexpr (G > 8) v = f(v, dpp<0x140>(v));   // row_mirror
  if constexpr (G > 16) v = f(v, __shfl_xor(v, 16));
  if constexpr (G > 32) v = f(v, __shfl_xor(v, 32));
  return v;
}
__device__ __forceinline__ float add_f(float a, float b) { return a + b; }
__device__ __forceinline__ float max_f(float a, float b) { return __builtin_fmaxf(a, b); }

// Blocks of a kernel that the device holds at once.
template <class K>
u32 resident_blocks(K kernel, int threads) {
  int each = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&each, kernel, threads, 0) != hipSuccess || each < 1) each = 1;
  return (u32)each * (u32)device_cu_count();
}

}  // namespace profk

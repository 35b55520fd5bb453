// Reading logits of any of the three types, shared by the language-model operators
// (k_tokens.hip, k_route.hip).
#pragma once

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

}  // namespace profk

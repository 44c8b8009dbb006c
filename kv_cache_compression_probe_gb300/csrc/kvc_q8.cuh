// What the calls on the 8-bit cache share (kvc_q8_append, kvc_q8_pack, kvc_q8_select,
// kvc_q8_attn): the argument block, the checks of a unit, and the e4m3 arithmetic.
//
// Codes are e4m3 (4 significant bits, largest 448).  A page's scale is a power of two, so
// that a code times its scale is exact in bf16 and fp32, codes move to a larger scale
// without loss (but for those that become subnormal), and a scale never rounds.
#pragma once
#include "kvc_chunk.cuh"

namespace kvc {

constexpr int kQ8MinExp = -40, kQ8MaxExp = 40;       // exponents of the scales

struct Q8Args {
  uint8_t* K;
  uint8_t* V;
  float* k_scale;
  float* v_scale;
  int8_t* bounds;                      // null: not kept
  float* logm;                         // null: all 0
  const int32_t* table;
  const int32_t* n_new;                // append: null = T
  const int32_t* len_lh;
  const int32_t* len_new;              // select, attention: entries with the chunk's own
  int32_t* err;
  int64_t units, lh_span, lh_gap, lh_base;
  int T, H, G, per_seq, max_pages, shift, pages;
};

// Argument checks of the calls, and the fields that come from the blocks.
int q8_check(const kvc_params* p, const kvc_chunk* c, const kvc_q8* x);
void q8_fill(Q8Args& a, const kvc_params* p, const kvc_chunk* c, const kvc_q8* x);
// kvc_q8_attn for many rows (kvc_q8_chunk.cu): its workspace and launches.
size_t q8_chunk_bytes(const kvc_params* p, const kvc_chunk* c);
cudaError_t q8_chunk_launch(const kvc_params* p, const kvc_chunk* c, const Q8Args& x, const void* q, void* out,
                            float* lse, void* workspace, cudaStream_t s);
inline bool q8_misaligned(const void* x, int to) { return (reinterpret_cast<uintptr_t>(x) & (to - 1)) != 0; }

}  // namespace kvc

namespace kvcd {

// unit_global of kvc_chunk.cuh for this block.
__device__ __forceinline__ int64_t q8_unit_global(const kvc::Q8Args& a, int64_t u) {
  return a.lh_gap ? u + (uint32_t)u / (uint32_t)a.lh_span * a.lh_gap + a.lh_base : u + a.lh_base;   // units are below 2^24
}

__device__ __forceinline__ float pow2i(int x) { return __int_as_float((x + 127) << 23); }
// Exponent of a stored scale.
__device__ __forceinline__ int scale_exp(float s) {
  return min(max(((__float_as_int(s) >> 23) & 255) - 127, kvc::kQ8MinExp), kvc::kQ8MaxExp);
}
// Least x with a <= 448 2^x (448 = 1.75 2^8), held to the scales there are.
__device__ __forceinline__ int scale_for(float a) {
  const int bits = __float_as_int(a);
  const int x = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  return a > 0.f ? min(max(x, kvc::kQ8MinExp), kvc::kQ8MaxExp) : kvc::kQ8MinExp;
}

// Two e4m3 codes as fp16 (exact), and two floats as codes, rounded to nearest.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint16_t f32_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void f16x2_f32(uint32_t v, float& lo, float& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(v));
}
__device__ __forceinline__ void e4m3_f32(uint16_t c, float& lo, float& hi) { f16x2_f32(e4m3_f16x2(c), lo, hi); }

// Four elements as floats.  (What an earlier call may have written is read by plain loads, or copied by cp.async, in
// these kernels, not through the read-only path: they may be launched before that call has ended.)
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* o) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  o[0] = __uint_as_float(u.x << 16); o[1] = __uint_as_float(u.x & 0xffff0000u);
  o[2] = __uint_as_float(u.y << 16); o[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* o) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
}

// What a page's bounds hold of a code.
__device__ __forceinline__ int bound_of(float code_value) { return __float2int_rn(code_value * 0.25f); }

}  // namespace kvcd

// bsa_q4.cuh -- the 4-bit cache format: quantising a row, and the places of
// its codes.  Shared by the cache kernels (bsa_q4_cache.cu) and the decode
// kernels (bsa_stream_decode.cu).
//
// A row of d channels is cut into groups of 32.  A group holds
//   s = fp16((max - min) / 15), m = fp16(min), code = floor((x - m) / s + 1/2)
// in 0..15 (0 where s is 0 or NaN), and reads back as code * s + m.  The
// places of the codes are those of the operands of the matrix instructions
// that read them (m16n8k16, lane = 4 g + t):
//   keys    word  t * (d/32) + G holds channels 32G + 8t .. +7, lowest nibble
//           first: lane t takes its words of all groups in one wide load;
//   values  piece (16 bits) y * (d/32) + G holds channels 32G + 4y .. +3: lane
//           y = g takes its channels of all groups in one wide load.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace bsa {
namespace q4 {

constexpr int kGroup = 32;
constexpr float kHalfMax = 65504.f;

__device__ __forceinline__ float bf16lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A group's scale and minimum, as stored and as used.
struct Params {
  uint32_t bits;   // fp16 pair: scale in the low half, minimum in the high
  float s, m;      // their values
  float inv;       // 1 / s, a little high
  float half;      // s / 2
};

__device__ __forceinline__ Params group_params(float lo, float hi) {
  Params p;
  float s = hi == lo ? 0.f : __fdiv_rn(hi - lo, 15.f);  // one infinity less another like it is no NaN
  s = s > kHalfMax ? kHalfMax : s;                       // a NaN stays
  float m = lo > kHalfMax ? kHalfMax : lo;
  m = m < -kHalfMax ? -kHalfMax : m;
  const __half2 h = __floats2half2_rn(s, m);
  p.bits = *reinterpret_cast<const uint32_t*>(&h);
  p.s = __low2float(h);
  p.m = __high2float(h);
  p.inv = __fdividef(1.f, p.s) * (1.f + 0x1p-20f);
  p.half = 0.5f * p.s;
  return p;
}

// floor((x - m) / s + 1/2), clamped to 0..15, as a float.  The quotient is taken with
// a reciprocal that is high by 2^-20, so the rounded code c is right or one too high;
// a comparison with the bound (c - 1/2) s, which is exact (5 bits times 11), tells
// which.  The difference t = x - m is rounded down: bounds are fp32 numbers, so x - m
// reaches one if and only if t does.  An infinite or NaN quotient ends at a clamp.
__device__ __forceinline__ float code_of(float x, const Params& p) {
  const float t = __fsub_rd(x, p.m);
  float c = __fadd_rd(fmaf(t, p.inv, 0.5f), 12582912.f) - 12582912.f;  // floor
  if (t < fmaf(c, p.s, -p.half)) c -= 1.f;
  return fminf(fmaxf(c, 0.f), 15.f);
}

// Four neighbouring codes as 16 bits (exact in fp32).
__device__ __forceinline__ uint32_t pack4(float c0, float c1, float c2, float c3, bool live) {
  const float v = fmaf(4096.f, c3, fmaf(256.f, c2, fmaf(16.f, c1, c0)));
  return live ? __float_as_uint(v + 8388608.f) & 0xffffu : 0u;
}

// Quantises one row of a key (is_key) or value by a warp: lane x < D/4 gives
// channels 4x .. 4x+3 in v.  Returns the lane's 16 bits of codes, their place
// in the row (in 16-bit units), and the group's parameters; every lane of a
// group has the same.
template <int D>
__device__ __forceinline__ uint32_t quantise_row(const float (&v)[4], int lane, bool is_key,
                                                 int* place, uint32_t* params) {
  constexpr int GR = D / kGroup;
  float lo = min_nan(min_nan(v[0], v[1]), min_nan(v[2], v[3]));
  float hi = max_nan(max_nan(v[0], v[1]), max_nan(v[2], v[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const Params p = group_params(lo, hi);
  const int G = (lane >> 3) % GR, y = lane & 7;
  *place = is_key ? 2 * ((y >> 1) * GR + G) + (y & 1) : y * GR + G;
  *params = p.bits;
  return pack4(code_of(v[0], p), code_of(v[1], p), code_of(v[2], p), code_of(v[3], p), p.s > 0.f);
}

}  // namespace q4
}  // namespace bsa

// bsa_window.cuh -- what the sliding-window forward and backward share: bounded
// waits, tensor maps over strided [B, H, N, d] tensors, and argument checks.
// Included by one translation unit per kernel file.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "bsa.h"
#include "sm100_ptx_more.cuh"

namespace bsa {
namespace win {

constexpr long long kWaitLimitCycles = 4000000000LL;  // ~2 s at 1.97 GHz
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kTile = 128;                            // queries, and keys, per tile
constexpr int kAtom = kTile * 128;                    // bytes of a 64-channel swizzle column of a tile

// True when the phase of parity `parity` has completed; false once the limit has
// passed (reported in *status) or another warp has given up.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             unsigned int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 1023u) == 0) {
      if (*abort) return false;
      const long long now = clock64();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitCycles) {
        *abort = 1;
        atomicOr(status, BSA_STATUS_TIMEOUT);
        return false;
      }
    }
  }
}

// Teardown: waits (bounded) for what is in flight, whatever the abort flag says.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, unsigned int* status) {
  const long long t0 = clock64();
  for (uint32_t it = 0; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 1023u) == 1023u && clock64() - t0 > kWaitLimitCycles) {
      atomicOr(status, BSA_STATUS_TIMEOUT);
      return;
    }
  }
}

// Sequence length of batch entry b; a bad one is reported and counts as 0.
__device__ __forceinline__ int length_of(const int32_t* lens, int b, int N, unsigned int* status) {
  if (lens == nullptr) return N;
  const int n = lens[b];
  if (n < 0 || n > N) {
    atomicOr(status, BSA_STATUS_BAD_SEQ_LEN);
    return 0;
  }
  return n;
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// [B, H, N, d] bf16 with strides as a 4-D tensor {d, N, H, B}; box = 64 channels
// x 128 rows of one head.  Rows past N read as zeros.
inline bool make_map(CUtensorMap* m, const bsa_view* v, int B, int H, int N, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  // the stride of a dimension of one entry is never used, but must be legal
  const long long sn = N > 1 ? v->stride_n : d, sh = H > 1 ? v->stride_h : d, sb = B > 1 ? v->stride_b : d;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(sn) * 2, static_cast<cuuint64_t>(sh) * 2,
                           static_cast<cuuint64_t>(sb) * 2};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(kTile), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v->data), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A view that a tensor map can describe: aligned, with every stride that is used a
// multiple of 8, at least d and below 2^39.
inline bool view_ok(const bsa_view* v, int B, int H, int N, int d) {
  if (!v || !v->data || (reinterpret_cast<uintptr_t>(v->data) & 15u) != 0) return false;
  const int64_t s[3] = {v->stride_b, v->stride_h, v->stride_n};
  const int n[3] = {B, H, N};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (s[i] < d || s[i] % 8 != 0 || s[i] >= (1LL << 39))) return false;
  return true;
}

// Whether rows of a view may overlap, which one to be written must not: taken from the
// smallest stride to the largest, each must pass all that the ones before it span.
inline bool rows_overlap(const bsa_view* v, int B, int H, int N, int d) {
  const int64_t s[3] = {v->stride_b, v->stride_h, v->stride_n};
  int n[3] = {B, H, N};
  unsigned __int128 span = static_cast<unsigned>(d);  // (2^30 - 1) 2^39 is past 64 bits
  for (int i = 0; i < 3; ++i) {
    int at = -1;
    for (int j = 0; j < 3; ++j)
      if (n[j] > 1 && (at < 0 || s[j] < s[at])) at = j;
    if (at < 0) break;
    if (static_cast<uint64_t>(s[at]) < span) return true;
    span += static_cast<unsigned __int128>(n[at] - 1) * static_cast<uint64_t>(s[at]);
    n[at] = 1;
  }
  return false;
}

inline int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

}  // namespace win
}  // namespace bsa

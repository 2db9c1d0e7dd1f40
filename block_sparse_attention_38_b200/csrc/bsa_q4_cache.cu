// bsa_q4_cache.cu -- the key/value cache held in 4 bits: quantising rows as
// they are written, and reading them back.  The format is bsa_q4.cuh's.
//
// Both are one pass over the data, bound by HBM: writing a row reads 2 d bytes
// and writes d/2 + d/8, reading it back the reverse.  A lane handles 8
// neighbouring channels (16 bytes of bf16, one 32-bit word of codes), so a row
// is 8 or 16 lanes, a group 4 lanes, and a group's minimum and maximum take two
// shuffles.  A warp takes kRows passes over keys and values whose loads are all
// issued before the first is used.
//
// Measured, d = 128: 16 heads x 32000 rows read back in 58 us (5.9 TB/s; with a
// shift and a conversion for each code 63, bound by instructions), 16 x 2048 rows
// written in 12 us; one token of 64 heads 5 us and 3 us, the latency of a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bsa.h"
#include "bsa_q4.cuh"

namespace bsa {
namespace q4 {

constexpr int kThreads = 256;
constexpr int kRows = 2;      // passes per warp, writing
constexpr int kReadRows = 4;  // and reading, which holds fewer registers a pass
constexpr int kMaxRows = 1 << 30;  // of a cache or a call: row numbers and their ends are ints

__device__ unsigned int g_q4_status;

struct CacheArgs {
  uint32_t* codes[2];       // keys, values: [B, H, L, d/8] words
  uint32_t* params[2];      // [B, H, L, d/32] fp16 pairs
  const __nv_bfloat16* src[2];
  long long sb[2], sh[2], sn[2];
  __nv_bfloat16* dst[2];    // [B, H, T, d]
  const int32_t* start;
  const int32_t* lens;      // may be null: T
  int H, L, T;
  int chunks;               // blocks per (b, h)
};

// Rows of this (b, h) that the call covers, and the first of them; reported
// and treated as none where they leave the cache.
__device__ __forceinline__ int row_range(const CacheArgs& a, int b, int* first) {
  const int s = a.start[b], n = a.lens ? a.lens[b] : a.T;
  *first = s;
  if (n == 0) return 0;
  if (n < 0 || n > a.T || s < 0 || s > a.L - n) {
    if (threadIdx.x == 0) atomicOr(&g_q4_status, BSA_STATUS_BAD_SEQ_LEN);
    return 0;
  }
  return n;
}

template <int D>
__global__ void __launch_bounds__(kThreads) write_kernel(const CacheArgs a) {
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPW = 32 / LPR;       // rows per warp and pass
  constexpr int GR = D / kGroup;
  const long long bh = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - bh * a.chunks);
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh - static_cast<long long>(b) * a.H);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = lane % LPR;                       // channels 8x .. 8x+7
  const int G = x >> 2, z = x & 3;                // group, and this lane's place in it
  const int r0 = chunk * (kThreads / 32 * RPW * kRows) + warp * RPW + lane / LPR;
  constexpr int kStep = kThreads / 32 * RPW;

  uint4 raw[kRows][2];
  auto load = [&](int rows) {
#pragma unroll
    for (int p = 0; p < kRows; ++p)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int r = r0 + p * kStep;
        raw[p][w] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows)
          raw[p][w] = __ldcs(reinterpret_cast<const uint4*>(a.src[w] + b * a.sb[w] + h * a.sh[w] +
                                                            r * a.sn[w] + 8 * x));
      }
  };
  // A few rows are loaded before their range is known, which takes a load off the
  // latency; of many, those past a sequence's end would cost bandwidth.
  if (a.chunks == 1) load(a.T);
  int first;
  const int n = row_range(a, b, &first);
  if (chunk * (kThreads / 32 * RPW * kRows) >= n) return;
  if (a.chunks > 1) load(n);
#pragma unroll
  for (int p = 0; p < kRows; ++p) {
    const int r = r0 + p * kStep;
    const long long row = bh * a.L + first + r;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint4 u = raw[p][w];
      float v[8] = {bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y),
                    bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)};
      float lo = v[0], hi = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, v[i]);
        hi = max_nan(hi, v[i]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      const Params pr = group_params(lo, hi);
      const bool live = pr.s > 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = code_of(v[i], pr);
      const uint32_t c0 = pack4(v[0], v[1], v[2], v[3], live);
      const uint32_t c1 = pack4(v[4], v[5], v[6], v[7], live);
      uint32_t word, place;
      if (w == 0) {
        word = c0 | c1 << 16;
        place = z * GR + G;
      } else {
        // pieces 2z and 2z + 1 of group G; a word holds one piece of an even
        // group and the next: lanes of neighbouring groups trade one each
        const bool odd = G & 1;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 4);
        word = odd ? got | c1 << 16 : c0 | got << 16;
        place = (2 * z + (odd ? 1 : 0)) * (GR / 2) + (G >> 1);
      }
      if (r < n) {
        a.codes[w][row * (D / 8) + place] = word;
        if (z == 0) a.params[w][row * GR + G] = pr.bits;
      }
    }
  }
}

// code * s + m of eight codes, each rounded once to bf16.  A code is taken where it
// lies: under the exponent of 2^(23 - 4i) nibble i counts ones, so nibbles 0 to 4
// need one logical operation each and the others one shift before it; taking the
// power off again is exact.  (With a shift and a conversion a code the kernel was
// bound by its instructions.)
__device__ __forceinline__ void values8(uint32_t word, float s, float m, uint32_t (&o)[4]) {
  const uint32_t high = word >> 12;  // nibbles 5, 6, 7 become 2, 3, 4
  auto pair = [&](uint32_t lo, uint32_t lo_mask, uint32_t lo_power, uint32_t hi, uint32_t hi_mask, uint32_t hi_power) {
    float x = __uint_as_float((lo & lo_mask) | lo_power), y = __uint_as_float((hi & hi_mask) | hi_power);
    asm("{\n\t.reg .b64 v, p, t, u;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 p, {%2, %3};\n\t"
        "sub.rn.f32x2 v, v, p;\n\tmov.b64 t, {%4, %4};\n\tmov.b64 u, {%5, %5};\n\t"
        "fma.rn.f32x2 v, v, t, u;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(__uint_as_float(lo_power)), "f"(__uint_as_float(hi_power)), "f"(s), "f"(m));
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  constexpr uint32_t k23 = 0x4b000000u, k19 = 0x49000000u, k15 = 0x47000000u, k11 = 0x45000000u, k7 = 0x43000000u;
  o[0] = pair(word, 0xfu, k23, word, 0xf0u, k19);
  o[1] = pair(word, 0xf00u, k15, word, 0xf000u, k11);
  o[2] = pair(word, 0xf0000u, k7, high, 0xf00u, k15);
  o[3] = pair(high, 0xf000u, k11, high, 0xf0000u, k7);
}

template <int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheArgs a) {
  constexpr int LPR = D / 8;
  constexpr int RPW = 32 / LPR;
  constexpr int GR = D / kGroup;
  const unsigned bh = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - bh * a.chunks);
  const int b = static_cast<int>(bh / a.H);
  int first;
  const int n = row_range(a, b, &first);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int x = lane % LPR, G = x >> 2, z = x & 3;
  const int r0 = chunk * (kThreads / 32 * RPW * kReadRows) + warp * RPW + lane / LPR;
  constexpr int kStep = kThreads / 32 * RPW;
  const long long row = static_cast<long long>(bh) * a.L + first + r0;
  const uint32_t* kc = a.codes[0] + row * (D / 8) + z * GR + G;
  const uint16_t* vc = reinterpret_cast<const uint16_t*>(a.codes[1] + row * (D / 8)) + 2 * z * GR + G;
  const uint32_t* kp = a.params[0] + row * GR + G;
  const uint32_t* vp = a.params[1] + row * GR + G;

  uint32_t code[kReadRows][2], par[kReadRows][2];
#pragma unroll
  for (int p = 0; p < kReadRows; ++p) {
    code[p][0] = code[p][1] = par[p][0] = par[p][1] = 0u;
    if (r0 + p * kStep < n) {
      code[p][0] = __ldcs(kc + p * kStep * (D / 8));
      code[p][1] = vc[p * kStep * (D / 4)] | static_cast<uint32_t>(vc[p * kStep * (D / 4) + GR]) << 16;
      par[p][0] = __ldcs(kp + p * kStep * GR);
      par[p][1] = __ldcs(vp + p * kStep * GR);
    }
  }
  const long long at = (static_cast<long long>(bh) * a.T + r0) * D + 8 * x;
  __nv_bfloat16 *ko = a.dst[0] + at, *vo = a.dst[1] + at;
#pragma unroll
  for (int p = 0; p < kReadRows; ++p) {
    if (r0 + p * kStep >= a.T) break;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const __half2 h = *reinterpret_cast<const __half2*>(&par[p][w]);
      uint32_t o[4];
      values8(code[p][w], __low2float(h), __high2float(h), o);
      __stcs(reinterpret_cast<uint4*>((w == 0 ? ko : vo) + p * kStep * D), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_cache(const bsa_q4_cache* c) {
  if (!c || !c->k_codes || !c->k_params || !c->v_codes || !c->v_params) return BSA_ERR_INVALID_ARG;
  if (c->B < 1 || c->H < 1 || c->L < 1 || c->d < 1) return BSA_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_params) || !aligned16(c->v_codes) ||
      !aligned16(c->v_params))
    return BSA_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || c->L > kMaxRows) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

void fill(CacheArgs* a, const bsa_q4_cache* c, const int32_t* start, const int32_t* lens, int T, int passes) {
  a->codes[0] = static_cast<uint32_t*>(c->k_codes);
  a->codes[1] = static_cast<uint32_t*>(c->v_codes);
  a->params[0] = static_cast<uint32_t*>(c->k_params);
  a->params[1] = static_cast<uint32_t*>(c->v_params);
  a->start = start;
  a->lens = lens;
  a->H = c->H;
  a->L = c->L;
  a->T = T;
  const int rows = kThreads / 32 * (c->d == 128 ? 2 : 4) * passes;
  a->chunks = (T + rows - 1) / rows;
}

}  // namespace q4
}  // namespace bsa

extern "C" int bsa_q4_write(const bsa_q4_cache* cache, const bsa_view* k, const bsa_view* v,
                            const int32_t* start, const int32_t* lens, int T, void* stream) {
  using namespace bsa::q4;
  const int rc = check_cache(cache);
  if (rc != BSA_OK) return rc;
  if (!k || !v || !k->data || !v->data || !start || T < 1) return BSA_ERR_INVALID_ARG;
  if (T > kMaxRows) return BSA_ERR_UNSUPPORTED;
  CacheArgs a = {};
  fill(&a, cache, start, lens, T, kRows);
  const bsa_view* views[2] = {k, v};
  for (int w = 0; w < 2; ++w) {
    const bsa_view* x = views[w];
    if (!aligned16(x->data) || x->stride_b < 0 || x->stride_h < 0 || x->stride_n < 0 ||
        x->stride_b % 8 != 0 || x->stride_h % 8 != 0 || x->stride_n % 8 != 0)
      return BSA_ERR_INVALID_ARG;
    a.src[w] = static_cast<const __nv_bfloat16*>(x->data);
    a.sb[w] = x->stride_b;
    a.sh[w] = x->stride_h;
    a.sn[w] = x->stride_n;
  }
  const long long blocks = static_cast<long long>(cache->B) * cache->H * a.chunks;
  if (blocks > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 64)
    write_kernel<64><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  else
    write_kernel<128><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

extern "C" int bsa_q4_read(const bsa_q4_cache* cache, const int32_t* start, const int32_t* lens,
                           int T, void* k, void* v, void* stream) {
  using namespace bsa::q4;
  const int rc = check_cache(cache);
  if (rc != BSA_OK) return rc;
  if (!k || !v || !start || T < 1 || !aligned16(k) || !aligned16(v)) return BSA_ERR_INVALID_ARG;
  if (T > kMaxRows) return BSA_ERR_UNSUPPORTED;
  CacheArgs a = {};
  fill(&a, cache, start, lens, T, kReadRows);
  a.dst[0] = static_cast<__nv_bfloat16*>(k);
  a.dst[1] = static_cast<__nv_bfloat16*>(v);
  const long long blocks = static_cast<long long>(cache->B) * cache->H * a.chunks;
  if (blocks > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 64)
    read_kernel<64><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  else
    read_kernel<128><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// The status word of this file's kernels, for bsa_stream_status.
namespace bsa {
int take_status(const void* symbol, uint32_t* status, int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, symbol, sizeof(v)) != cudaSuccess) return BSA_ERR_CUDA;
  if (clear && v) {
    const unsigned int z = 0;
    if (cudaMemcpyToSymbol(symbol, &z, sizeof(z)) != cudaSuccess) return BSA_ERR_CUDA;
  }
  *status |= v;
  return BSA_OK;
}
int q4_status(uint32_t* status, int clear) { return take_status(&q4::g_q4_status, status, clear); }
int stream_decode_status(uint32_t* status, int clear);
int window_forward_status(uint32_t* status, int clear);
int window_backward_status(uint32_t* status, int clear);
}  // namespace bsa

extern "C" int bsa_stream_status(uint32_t* status, int clear) {
  if (!status) return BSA_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return BSA_ERR_CUDA;
  uint32_t v = 0;
  int rc = bsa::q4_status(&v, clear);
  if (rc == BSA_OK) rc = bsa::stream_decode_status(&v, clear);
  if (rc == BSA_OK) rc = bsa::window_forward_status(&v, clear);
  if (rc == BSA_OK) rc = bsa::window_backward_status(&v, clear);
  if (rc == BSA_OK) *status = v;
  return rc;
}

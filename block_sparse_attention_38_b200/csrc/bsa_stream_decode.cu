// bsa_stream_decode.cu -- one decode step over a long cache: bf16 or 4 bits,
// shared key/value heads, and as visible tokens either a sliding window with
// first tokens (sinks) or the blocks of a block-CSR row.
//
// For each (b, cached head) the G = H / Hkv query heads of the group read the
// same cached rows.  With x_k = scale q.k, the step gives
// O = sum_k softmax(x)_k v_k and LSE = ln sum_k exp x_k.  It is bound by HBM:
// 2 (d/2 + d/8) bytes a token and cached head (4 bits) or 4 d (bf16), against
// 4 d G flops.  Both products run on the warp matrix instructions
// (m16n8k16, fp32 accumulation) as
//   S^T[key, head] = K Q^T         16 keys a tile, 8 heads a tile
//   O^T[channel, head] += V^T P^T
// so the cached rows, the large operand, fill the 16 rows of a tile and a group
// of up to 8 heads wastes nothing.  tcgen05 would need the codes decoded into
// shared memory or TMEM first; here they go from shared memory to the operand
// registers with a mask and a shift.
//
// 4 bits (bsa_q4.cuh).  Codes enter the matrix instructions as fp16 subnormals:
// the bits of c are the number c 2^-24, and of c << 4 the number 16 c 2^-24, so
// two codes in place cost one AND.  Q is scaled per head by a power of two to
// 2^13..2^14 (exact) and by 1/16 where a code is 16-fold, so the products are
// exact; group G's sum is multiplied by the key's scale in fp32, and the minima
// add m_kG sum_{c in G} q_c by a product of their own, the sum in two fp16 terms
// (2^-22).  For V, P^T is multiplied by the key's scale of
// the group before its rounding to fp16 (2^-11, against 2^-8 of the bf16
// output), and sum_k p_k m_kG is kept in fp32.  fp16's range is centred for each
// group G: scales count in units of 2^E_G, which has been above every scale of the
// group so far (E_G only grows, like a maximum, and is taken off at the join), and
// the running maximum lies 2^6 below the largest weight.  It is raised only by
// more than 2^8, so P times a scale stays below 2^15; and as fp16 goes down to
// 2^-24, a weight is off by 2^-11, or by 2^-30 of the largest weight where that is
// more, in units of the largest scale that the group has among the rows seen.
//
// bf16: operands by ldmatrix; P is split into two bf16 terms (P = hi + lo), so its
// rounding costs 2^-16; the second product is free under the cache's bytes.
//
// Work split: a unit is 32 (16 for bf16) neighbouring cached rows.  Warps take
// units in turn, each with its own ring of cp.async stages: no barrier or wait
// between warps until the end.  A (b, cached head) is given to a cluster of up
// to 16 CTAs when there are few of them; the CTAs' (max, sum, O) are joined over
// distributed shared memory, so one launch does it all, with no workspace and
// the same result in every run.
//
// Measured, 4 bits, d = 128: 16 cached heads of 4 x 131072 rows 90 us (3.5 TB/s,
// clusters of 13), 148 of 4 x 16384 80 us (4.9 TB/s); the copies alone reach 5.1 to
// 6.2, so the arithmetic's latency at 16 warps an SM bounds it.  bf16, 32 heads of 4,
// window 4096: 18 us, of which some 8 are the start and the join.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "bsa.h"
#include "bsa_q4.cuh"

namespace bsa {
namespace sdec {

namespace cg = cooperative_groups;

constexpr int kMaxM = 4096;
constexpr float kRescale = 8.f;  // log2 units by which a maximum must grow to be raised
// Maxima begin at the least finite number: weights are then 0 for scores of -inf, NaN for
// NaN (which no comparison sees, but every sum keeps) and at most 1 for any other.
constexpr float kLeast = -3.402823466e38f;
constexpr float kLift = 6.f;  // 4 bits: the weight of the running maximum, log2

__device__ unsigned int g_sdec_status;

struct Args {
  const __nv_bfloat16* q;       // [B, H, d]
  const __nv_bfloat16* k_new;   // [B, Hkv, d] or null
  const __nv_bfloat16* v_new;
  unsigned char* k;             // bf16 rows, or codes
  unsigned char* v;
  unsigned char* kp;            // 4 bits: parameters
  unsigned char* vp;
  const int32_t* row_ptr;       // block pattern, or null: window
  const int32_t* col_idx;
  const int32_t* seq_len;
  __nv_bfloat16* O;             // [B, H, d]
  float* LSE;                   // [B, H]
  int Hkv, G, L;
  int chunks;                   // 8 NT-head pieces of a group
  int cluster;
  int bs, M;                    // block pattern
  int window, sinks;
  float scale_log2;
};

template <int D, bool Q4, int NT, int NW>
struct Cfg {
  static constexpr int THREADS = 32 * NW;
  static constexpr int GR = D / 32;
  static constexpr int UK = Q4 ? 32 : 16;              // keys per unit
  static constexpr int SUB = UK / 16;
  static constexpr int ROW = Q4 ? D / 2 : 2 * D;       // bytes of a row
  static constexpr int PROW = Q4 ? 4 * GR : 0;         // bytes of a row's parameters
  static constexpr int V_OFF = UK * ROW;
  static constexpr int KP_OFF = 2 * UK * ROW;
  static constexpr int VP_OFF = KP_OFF + UK * PROW;
  static constexpr int STAGE = 2 * UK * (ROW + PROW);  // 5 KB and 2.5 KB (4 bits), 8 and 4 KB (bf16)
  static constexpr int STAGES = Q4 ? (D == 128 ? 2 : 3) : 3;
  static constexpr int RING = NW * STAGES * STAGE;
  static constexpr int HEADS = 8 * NT;
  // overlaid on the ring at the end: each warp's O and (max, sum)
  static constexpr int PART = NW * HEADS * (D + 2) * 4;
  // the CTA's own result, read by its cluster: not overlaid
  static constexpr int OUT = HEADS * (D + 2) * 4;
  static constexpr int SMEM = (RING > PART ? RING : PART) + OUT;
  static constexpr int PER_SM = NW == 8 && NT == 1 && (Q4 || D == 64) ? 2 : 1;  // by registers and shared memory
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros instead of the source's bytes where it is not live.
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp8_if(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// 8 summed entries instead of 16, onto zeros or onto d.
__device__ __forceinline__ void mma_f16_k8_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
}
__device__ __forceinline__ void mma_f16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_of(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// Key (0..7) at row r of a tile's half, for the 4-bit tiles.  With it the eight
// rows that the lanes of one load take fall into different banks, both for keys
// (rows r, r + 1 at a time) and for values (rows 0, 2, 4, 6, then 1, 3, 5, 7).
__device__ __forceinline__ int key_of_row(int r) { return (0x63417250u >> (4 * r)) & 7; }

// Byte offset of 16-byte piece c of row r within a tile.
template <int D, bool Q4>
__device__ __forceinline__ int place(int r, int c) {
  if constexpr (Q4)
    return D == 128 ? r * 64 + ((c ^ (r & 2)) << 4) : r * 32 + (c << 4);
  else
    return r * 2 * D + ((c ^ (r & 7)) << 4);
}

// The rows that one (b, cached head) sees, as a list of units.
struct Span {
  int t;                 // newest token; -1: none
  int units;
  int head_units;        // window: units before the window (sinks)
  int first_unit;        // window: the window's first unit
  int lo, sinks;         // window: first row of the window, rows always visible
};

template <int D, bool Q4, int NT, int NW>
struct Warp {
  using C = Cfg<D, Q4, NT, NW>;
  // S^T columns 2t, 2t + 1 are this lane's heads in S and O
  float o[D / 16][NT][4];
  float top[NT][2];      // running maximum, log2 units (less kLift for 4 bits)
  float sum[NT][2];      // this lane's share of the denominator
  float pm[Q4 ? C::GR : 1][NT][2];  // sum_k p_k m_kG, this lane's keys
  float unit[Q4 ? C::GR : 1];       // 2^-E_G
  uint32_t qf[NT][D / 16][2];
  uint32_t qs[NT][2];    // 2^-4 sum of q over group t, head g: high and low term, behind a 0
  float mul[NT][2];      // from accumulator to x in log2 units
};

// Query operands.  Lane 4 g + t holds head g's channels.
template <int D, bool Q4, int NT, int NW>
__device__ __forceinline__ void load_q(Warp<D, Q4, NT, NW>& w, const Args& a, long long head0, int heads,
                                       int lane) {
  using C = Cfg<D, Q4, NT, NW>;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = nt * 8 + g;
    const __nv_bfloat16* q = a.q + (head0 + head) * D;
    if constexpr (Q4) {
      uint4 raw[C::GR];
      float amax = 0.f;
#pragma unroll
      for (int G = 0; G < C::GR; ++G) {
        raw[G] = head < heads ? *reinterpret_cast<const uint4*>(q + 32 * G + 8 * t) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t r[4] = {raw[G].x, raw[G].y, raw[G].z, raw[G].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          amax = fmaxf(amax, fmaxf(fabsf(q4::bf16lo(r[i])), fabsf(q4::bf16hi(r[i]))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // amax = 1.x 2^ex
      ex = min(max(ex, -100), 116);  // both factors below stay finite
      const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - ex) << 23);  // 2^(13 - ex)
      const float mul = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + 11 + ex) << 23);  // 2^(24 - 13 + ex)
      w.mul[nt][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
      w.mul[nt][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
      float mine = 0.f;  // of group t
#pragma unroll
      for (int G = 0; G < C::GR; ++G) {
        const float v[8] = {q4::bf16lo(raw[G].x) * up, q4::bf16hi(raw[G].x) * up,
                            q4::bf16lo(raw[G].y) * up, q4::bf16hi(raw[G].y) * up,
                            q4::bf16lo(raw[G].z) * up, q4::bf16hi(raw[G].z) * up,
                            q4::bf16lo(raw[G].w) * up, q4::bf16hi(raw[G].w) * up};
        // nibbles (0, 4), (1, 5) x 1/16, (2, 6), (3, 7) x 1/16
        w.qf[nt][2 * G][0] = pack_h(v[0], v[4]);
        w.qf[nt][2 * G][1] = pack_h(v[1] * 0.0625f, v[5] * 0.0625f);
        w.qf[nt][2 * G + 1][0] = pack_h(v[2], v[6]);
        w.qf[nt][2 * G + 1][1] = pack_h(v[3] * 0.0625f, v[7] * 0.0625f);
        float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (G == t) mine = 0.0625f * s;
      }
      const float high = __half2float(__float2half_rn(mine));
      w.qs[nt][0] = pack_h(0.f, high);
      w.qs[nt][1] = pack_h(0.f, mine - high);
    } else {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          w.qf[nt][kk][i] = head < heads
                                ? *reinterpret_cast<const uint32_t*>(q + 16 * kk + 8 * i + 2 * t)
                                : 0u;
      w.mul[nt][0] = w.mul[nt][1] = a.scale_log2;
    }
  }
}

// Issues the copies of the unit that starts at cached row `row0` of the head
// whose rows start at `base`: the unit's rows lie one behind another, so lane l
// copies bytes 16 l + 512 i.  Rows past the cache's end are zero-filled.
template <int D, bool Q4, int NT, int NW>
__device__ __forceinline__ void load_unit(const Args& a, long long base, int row0, uint32_t st,
                                          int lane) {
  using C = Cfg<D, Q4, NT, NW>;
  constexpr int PIECES = C::ROW / 16, RPI = 32 / PIECES;  // 16-byte pieces of a row, rows an iteration
  const int r0 = lane / PIECES, c = lane % PIECES;
  const unsigned char* kp = a.k + (base + row0) * C::ROW + lane * 16;
  const unsigned char* vp = a.v + (base + row0) * C::ROW + lane * 16;
  if (row0 + C::UK <= a.L) {
#pragma unroll
    for (int i = 0; i < C::UK / RPI; ++i) {
      const int at = place<D, Q4>(i * RPI + r0, c);
      cp16(st + at, kp + 512 * i);
      cp16(st + C::V_OFF + at, vp + 512 * i);
    }
  } else {
    for (int i = 0; i < C::UK / RPI; ++i) {
      const bool live = row0 + i * RPI + r0 < a.L;
      const int at = place<D, Q4>(i * RPI + r0, c);
      cp16_if(st + at, live ? kp + 512 * i : a.k, live);
      cp16_if(st + C::V_OFF + at, live ? vp + 512 * i : a.v, live);
    }
  }
  if constexpr (Q4) {
    const bool live = row0 + lane < a.L;
    const long long off = live ? (base + row0 + lane) * C::PROW : 0;
    if constexpr (C::PROW == 16) {
      cp16_if(st + C::KP_OFF + lane * 16, a.kp + off, live);
      cp16_if(st + C::VP_OFF + lane * 16, a.vp + off, live);
    } else {
      cp8_if(st + C::KP_OFF + lane * 8, a.kp + off, live);
      cp8_if(st + C::VP_OFF + lane * 8, a.vp + off, live);
    }
  }
}

// One warp: the new token's key and value as a cached row, for the cache itself
// (row index `row`) or for row r of a stage.
template <int D, bool Q4, int NT, int NW, bool TO_STAGE>
__device__ __forceinline__ void put_new(const Args& a, long long bh, long long row, unsigned char* st,
                                        int r, int lane) {
  using C = Cfg<D, Q4, NT, NW>;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const __nv_bfloat16* src = (w == 0 ? a.k_new : a.v_new) + bh * D;
    if constexpr (Q4) {
      uint2 raw = make_uint2(0u, 0u);
      if (lane < D / 4) raw = *reinterpret_cast<const uint2*>(src + 4 * lane);
      const float v[4] = {q4::bf16lo(raw.x), q4::bf16hi(raw.x), q4::bf16lo(raw.y), q4::bf16hi(raw.y)};
      int at;
      uint32_t par;
      const uint32_t code = q4::quantise_row<D>(v, lane, w == 0, &at, &par);
      const int G = lane >> 3;
      unsigned char* cp;
      unsigned char* pp;
      if constexpr (TO_STAGE) {
        cp = st + (w == 0 ? 0 : C::V_OFF) + place<D, Q4>(r, at >> 3) + (at & 7) * 2;
        pp = st + (w == 0 ? C::KP_OFF : C::VP_OFF) + r * C::PROW + 4 * G;
      } else {
        cp = (w == 0 ? a.k : a.v) + row * C::ROW + at * 2;
        pp = (w == 0 ? a.kp : a.vp) + row * C::PROW + 4 * G;
      }
      if (lane < D / 4) {
        *reinterpret_cast<uint16_t*>(cp) = static_cast<uint16_t>(code);
        if ((lane & 7) == 0) *reinterpret_cast<uint32_t*>(pp) = par;
      }
    } else {
      if (lane < D / 8) {
        const uint4 raw = *reinterpret_cast<const uint4*>(src + 8 * lane);
        unsigned char* cp;
        if constexpr (TO_STAGE)
          cp = st + (w == 0 ? 0 : C::V_OFF) + place<D, Q4>(r, lane);
        else
          cp = (w == 0 ? a.k : a.v) + row * C::ROW + lane * 16;
        *reinterpret_cast<uint4*>(cp) = raw;
      }
    }
  }
}

// Scores of a 16-key tile, S^T[key, head] * nothing yet: accumulator units.
template <int D, bool Q4, int NT, int NW>
__device__ __forceinline__ void score_tile(const Warp<D, Q4, NT, NW>& w, const unsigned char* st, int sub,
                                           int lane, float (&x)[NT][4]) {
  using C = Cfg<D, Q4, NT, NW>;
  const int g = lane >> 2, t = lane & 3;
  if constexpr (Q4) {
    const int r0 = sub * 16 + key_of_row(g);
    // m_kG times the sum of q over group G: a key's parameters (s_0, m_0, s_1, ...) as
    // they lie against (0, q sum of group 0, 0, ...)
    uint32_t m0 = 0u, m1 = 0u;
    if (t < C::GR) {
      m0 = *reinterpret_cast<const uint32_t*>(st + C::KP_OFF + r0 * C::PROW + 4 * t);
      m1 = *reinterpret_cast<const uint32_t*>(st + C::KP_OFF + (r0 + 8) * C::PROW + 4 * t);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mma_f16_k8_zero(x[nt], m0, m1, w.qs[nt][0]);
      mma_f16_k8(x[nt], m0, m1, w.qs[nt][1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] *= 0x1p-20f;
    }
    uint32_t kw[2][C::GR], kp[2][C::GR];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(st + place<D, Q4>(r, t));
        kw[i][0] = u.x; kw[i][1] = u.y; kw[i][2] = u.z; kw[i][3] = u.w;
        const uint4 p = *reinterpret_cast<const uint4*>(st + C::KP_OFF + r * 16);
        kp[i][0] = p.x; kp[i][1] = p.y; kp[i][2] = p.z; kp[i][3] = p.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(st + r * 32 + t * 8);
        kw[i][0] = u.x; kw[i][1] = u.y;
        const uint2 p = *reinterpret_cast<const uint2*>(st + C::KP_OFF + r * 8);
        kp[i][0] = p.x; kp[i][1] = p.y;
      }
    }
#pragma unroll
    for (int G = 0; G < C::GR; ++G) {
      const uint32_t u0 = kw[0][G], u1 = kw[1][G], v0 = u0 >> 8, v1 = u1 >> 8;
      const float s0 = half2_of(kp[0][G]).x, s1 = half2_of(kp[1][G]).x;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float c[4];
        mma_f16_zero(c, u0 & 0x000f000fu, u1 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x00f000f0u,
                w.qf[nt][2 * G][0], w.qf[nt][2 * G][1]);
        mma_f16(c, v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u,
                w.qf[nt][2 * G + 1][0], w.qf[nt][2 * G + 1][1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[nt][j] = fmaf(s0, c[j], x[nt][j]);
          x[nt][2 + j] = fmaf(s1, c[2 + j], x[nt][2 + j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      // matrices: keys 0-7 / 8-15 of channels 16kk.., then of channels 16kk + 8..
      const int r = sub * 16 + (lane & 15);
      uint32_t k[4];
      ldmatrix4<false>(k, smem_addr(st + place<D, Q4>(r, 2 * kk + (lane >> 4))));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(x[nt], k, w.qf[nt][kk][0], w.qf[nt][kk][1]);
    }
  }
}

// O^T += V^T P^T for a 16-key tile; p in the layout of score_tile.
template <int D, bool Q4, int NT, int NW>
__device__ __forceinline__ void value_tile(Warp<D, Q4, NT, NW>& w, const unsigned char* st, int sub, int lane,
                                           const float (&p)[NT][4]) {
  using C = Cfg<D, Q4, NT, NW>;
  const int g = lane >> 2, t = lane & 3;
  if constexpr (Q4) {
    const int r0 = sub * 16 + key_of_row(g);
    const int ra = sub * 16 + key_of_row(2 * t), rb = sub * 16 + key_of_row(2 * t + 1);
    constexpr int VW = D / 64;  // words of a lane's channels
    uint32_t vw[4][VW], vp[2][C::GR];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ((i & 1) ? rb : ra) + 8 * (i >> 1);
      if constexpr (D == 128) {
        const uint2 u = *reinterpret_cast<const uint2*>(st + C::V_OFF + place<D, Q4>(r, g >> 1) + (g & 1) * 8);
        vw[i][0] = u.x;
        vw[i][VW - 1] = u.y;
      } else {
        vw[i][0] = *reinterpret_cast<const uint32_t*>(st + C::V_OFF + r * 32 + g * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(st + C::VP_OFF + r * 16);
        vp[i][0] = u.x; vp[i][1] = u.y; vp[i][2] = u.z; vp[i][3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(st + C::VP_OFF + r * 8);
        vp[i][0] = u.x; vp[i][1] = u.y;
      }
    }
#pragma unroll
    for (int G = 0; G < C::GR; ++G) {
      const uint32_t sel = (G & 1) ? 0x7632u : 0x5410u;
      const uint32_t e = __byte_perm(vw[0][G / 2], vw[1][G / 2], sel), e8 = e >> 8;  // keys of rows 2t, 2t + 1
      const uint32_t f = __byte_perm(vw[2][G / 2], vw[3][G / 2], sel), f8 = f >> 8;  // the same + 8
      const float2 s0 = half2_of(vp[0][G]), s1 = half2_of(vp[1][G]);
      const float u0 = s0.x * w.unit[G], u1 = s1.x * w.unit[G];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t b0 = transpose8x8(pack_h(p[nt][0] * u0, p[nt][1] * u0));
        const uint32_t b1 = transpose8x8(pack_h(p[nt][2] * u1, p[nt][3] * u1));
        mma_f16(w.o[2 * G][nt], e & 0x000f000fu, e8 & 0x000f000fu, f & 0x000f000fu, f8 & 0x000f000fu, b0, b1);
        mma_f16(w.o[2 * G + 1][nt], e & 0x00f000f0u, e8 & 0x00f000f0u, f & 0x00f000f0u, f8 & 0x00f000f0u, b0, b1);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w.pm[G][nt][j] = fmaf(p[nt][j], s0.y, fmaf(p[nt][2 + j], s1.y, w.pm[G][nt][j]));
      }
    }
  } else {
    uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float p0 = p[nt][2 * i], p1 = p[nt][2 * i + 1];
        const uint32_t h = pack_b(p0, p1);
        hi[nt][i] = transpose8x8(h);
        lo[nt][i] = transpose8x8(pack_b(p0 - q4::bf16lo(h), p1 - q4::bf16hi(h)));
      }
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
      // transposed matrices: (channels 16m.., keys 0-7), (16m + 8.., 0-7), (16m.., 8-15), (16m + 8.., 8-15)
      const int r = sub * 16 + (lane & 7) + ((lane >> 4) << 3);
      uint32_t v[4];
      ldmatrix4<true>(v, smem_addr(st + C::V_OFF + place<D, Q4>(r, 2 * m + ((lane >> 3) & 1))));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16(w.o[m][nt], v, hi[nt][0], hi[nt][1]);
        mma_bf16(w.o[m][nt], v, lo[nt][0], lo[nt][1]);
      }
    }
  }
}

// Channel of O^T tile m, row half i (rows g and g + 8) of lane group g.
template <int D, bool Q4>
__device__ __forceinline__ int channel_of(int m, int i, int g) {
  if constexpr (Q4)
    return 32 * (m >> 1) + 4 * g + 2 * i + (m & 1);
  else
    return 16 * m + 8 * i + g;
}

template <int D, bool Q4, int NT, int NW>
__global__ void __launch_bounds__(32 * NW, Cfg<D, Q4, NT, NW>::PER_SM) stream_decode_kernel(const Args a) {
  using C = Cfg<D, Q4, NT, NW>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t bitmap[kMaxM / 32];
  __shared__ uint16_t blocks[kMaxM];
  __shared__ int n_blocks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int rank = static_cast<int>(blockIdx.x % a.cluster);
  const long long grp = blockIdx.x / a.cluster;
  const int chunk = static_cast<int>(grp % a.chunks);
  const long long bh = grp / a.chunks;                    // (b, cached head)
  const int b = static_cast<int>(bh / a.Hkv), hkv = static_cast<int>(bh - static_cast<long long>(b) * a.Hkv);
  const long long base = bh * a.L;                        // cached row 0
  const long long head0 = static_cast<long long>(b) * a.Hkv * a.G + static_cast<long long>(hkv) * a.G + chunk * C::HEADS;
  const int heads = min(C::HEADS, a.G - chunk * C::HEADS);

  int len = a.seq_len[b];
  if (len < 0 || len > a.L) {
    if (tid == 0) atomicOr(&g_sdec_status, BSA_STATUS_BAD_SEQ_LEN);
    len = 0;
  }
  Span sp;
  sp.t = len - 1;
  sp.units = sp.head_units = sp.first_unit = sp.lo = sp.sinks = 0;
  if (len > 0 && a.row_ptr == nullptr) {
    sp.lo = a.window < len ? len - a.window : 0;
    sp.sinks = a.sinks;
    sp.first_unit = sp.lo / C::UK;
    sp.head_units = min((min(a.sinks, sp.lo) + C::UK - 1) / C::UK, sp.first_unit);
    sp.units = sp.head_units + sp.t / C::UK + 1 - sp.first_unit;
  } else if (len > 0) {
    const int i = sp.t / a.bs, W = i / 32 + 1;
    for (int w = tid; w < W; w += C::THREADS) bitmap[w] = 0u;
    __syncthreads();
    int e0 = a.row_ptr[static_cast<long long>(hkv) * a.M + i];
    int e1 = a.row_ptr[static_cast<long long>(hkv) * a.M + i + 1];
    if (e0 < 0 || e1 < e0) {
      if (tid == 0) atomicOr(&g_sdec_status, BSA_STATUS_BAD_ROW_PTR);
      e0 = e1 = 0;
    }
    for (int e = e0 + tid; e < e1; e += C::THREADS) {
      const int j = a.col_idx[e];
      if (j < 0 || j >= a.M)
        atomicOr(&g_sdec_status, BSA_STATUS_BAD_COLUMN);
      else if (j <= i)
        atomicOr(&bitmap[j >> 5], 1u << (j & 31));
    }
    __syncthreads();
    if (warp == 0) {  // the blocks in ascending order
      int n = 0;
      for (int w0 = 0; w0 < W; w0 += 32) {
        uint32_t bits = w0 + lane < W ? bitmap[w0 + lane] : 0u;
        int at = __popc(bits);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, o);
          if (lane >= o) at += y;
        }
        const int total = __shfl_sync(0xffffffffu, at, 31);
        at += n - __popc(bits);
        for (; bits; bits &= bits - 1) blocks[at++] = static_cast<uint16_t>((w0 + lane) * 32 + __ffs(bits) - 1);
        n += total;
      }
      if (lane == 0) n_blocks = n;
    }
    __syncthreads();
    // every block is bs rows; of the newest token's block, the rows up to it
    const int nb = n_blocks;
    sp.units = nb * (a.bs / C::UK);
    if (nb > 0 && blocks[nb - 1] == i) sp.units -= a.bs / C::UK - ((sp.t - i * a.bs) / C::UK + 1);
  }
  const int per = a.row_ptr == nullptr ? 0 : 31 - __clz(a.bs / C::UK);  // log2 of a block's units
  auto row_of = [&](int u) {  // first cached row of unit u
    if (a.row_ptr == nullptr)
      return (u < sp.head_units ? u : sp.first_unit + u - sp.head_units) * C::UK;
    return blocks[u >> per] * a.bs + (u & ((1 << per) - 1)) * C::UK;
  };

  unsigned char* ring = smem + warp * C::STAGES * C::STAGE;
  const uint32_t ring_u = smem_addr(ring);
  const int step = a.cluster * NW;
  const int u0 = warp * a.cluster + rank;
  int rows[C::STAGES];  // first rows of the units in flight
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) {
    const int u = u0 + s * step;
    rows[s] = u < sp.units ? row_of(u) : 0;
    if (u < sp.units) load_unit<D, Q4, NT, NW>(a, base, rows[s], ring_u + s * C::STAGE, lane);
    cp_commit();
  }

  Warp<D, Q4, NT, NW> w;
  load_q<D, Q4, NT, NW>(w, a, head0, heads, lane);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w.top[nt][j] = kLeast;
      w.sum[nt][j] = 0.f;
#pragma unroll
      for (int G = 0; G < (Q4 ? C::GR : 1); ++G) w.pm[G][nt][j] = 0.f;
    }
#pragma unroll
  for (int G = 0; G < (Q4 ? C::GR : 1); ++G) w.unit[G] = 0x1p25f;  // any scale above 0 calls for another
#pragma unroll
  for (int m = 0; m < D / 16; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[m][nt][i] = 0.f;

  // The new token's row goes into the cache once; the warp that attends to it
  // takes it from k_new / v_new again, so no order between the two is needed.
  if (a.k_new != nullptr && len > 0 && rank == 0 && chunk == 0 && warp == NW - 1)
    put_new<D, Q4, NT, NW, false>(a, bh, base + sp.t, nullptr, 0, lane);

  int slot = 0;
  for (int u = u0; u < sp.units; u += step) {
    {
      const int un = u + (C::STAGES - 1) * step;
      int sn = slot + C::STAGES - 1;
      if (sn >= C::STAGES) sn -= C::STAGES;
      if (un < sp.units) {
        rows[C::STAGES - 1] = row_of(un);
        load_unit<D, Q4, NT, NW>(a, base, rows[C::STAGES - 1], ring_u + sn * C::STAGE, lane);
      }
      cp_commit();
    }
    cp_wait<C::STAGES - 1>();
    __syncwarp();
    unsigned char* st = ring + slot * C::STAGE;
    const int row0 = rows[0];
#pragma unroll
    for (int s = 0; s + 1 < C::STAGES; ++s) rows[s] = rows[s + 1];
    bool all;  // every row of the unit is visible
    if (a.row_ptr == nullptr)
      all = row0 + C::UK - 1 <= sp.t && (row0 >= sp.lo || row0 + C::UK <= sp.sinks);
    else
      all = row0 + C::UK - 1 <= sp.t;
    auto visible = [&](int r) {
      const int k = row0 + r;
      return k <= sp.t && (a.row_ptr != nullptr || k >= sp.lo || k < sp.sinks);
    };
    if (!all || (a.k_new != nullptr && row0 + C::UK - 1 == sp.t)) {
      if (a.k_new != nullptr && row0 <= sp.t && sp.t < row0 + C::UK) {
        put_new<D, Q4, NT, NW, true>(a, bh, 0, st, sp.t - row0, lane);
        __syncwarp();
      }
      // Hidden rows take weight 0, but 0 times what they hold (anything, NaN
      // too) must be 0: their values are cleared.
      for (int r = lane; r < C::UK; r += 32)
        if (!visible(r)) {
          if constexpr (Q4) {
#pragma unroll
            for (int G = 0; G < C::GR; ++G)
              *reinterpret_cast<uint32_t*>(st + C::VP_OFF + r * C::PROW + 4 * G) = 0u;
          } else {
            for (int c = 0; c < C::ROW / 16; ++c)
              *reinterpret_cast<uint4*>(st + C::V_OFF + r * C::ROW + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      __syncwarp();
    }

    float x[C::SUB][NT][4];
#pragma unroll
    for (int s = 0; s < C::SUB; ++s) score_tile<D, Q4, NT, NW>(w, st, s, lane, x[s]);
#pragma unroll
    for (int s = 0; s < C::SUB; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[s][nt][i] *= w.mul[nt][i & 1];
    if (!all) {
#pragma unroll
      for (int s = 0; s < C::SUB; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = s * 16 + 8 * i + (Q4 ? key_of_row(g) : g);
          if (!visible(r)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[s][nt][2 * i] = x[s][nt][2 * i + 1] = -INFINITY;
          }
        }
    }
    // The running maximum (and E_G) are raised only where a lane's own scores (or
    // scales) call for it, by more than the threshold: mostly one vote is all.
    bool want = false;
    constexpr float kUp = Q4 ? kLift : 0.f;
    const uint32_t* vp = reinterpret_cast<const uint32_t*>(st + C::VP_OFF + lane * C::PROW);
    if constexpr (Q4) {
#pragma unroll
      for (int G = 0; G < C::GR; ++G) want |= half2_of(vp[G]).x * w.unit[G] >= 2.f;
    }
    float most[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float m = fmaxf(x[0][nt][j], x[0][nt][2 + j]);
#pragma unroll
        for (int s = 1; s < C::SUB; ++s) m = fmaxf(m, fmaxf(x[s][nt][j], x[s][nt][2 + j]));
        most[nt][j] = m;
        want |= m > w.top[nt][j] + (kRescale + kUp);
      }
    if (__any_sync(0xffffffffu, want)) {
      if constexpr (Q4) {
#pragma unroll
        for (int G = 0; G < C::GR; ++G) {
          // E_G is one more than the largest scale's exponent: the next power of two is no cause to raise
          const uint32_t big = min(__reduce_max_sync(0xffffffffu, vp[G] & 0x7fffu), 0x7bffu);
          const float half_of = __half2float(__ushort_as_half(static_cast<unsigned short>(big)));
          const float unit = __uint_as_float((253u << 23) - (__float_as_uint(half_of) & 0x7f800000u));
          if (big != 0u && unit < w.unit[G]) {
            const float f = unit * __uint_as_float((254u << 23) - __float_as_uint(w.unit[G]));
            w.unit[G] = unit;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                w.o[2 * G][nt][i] *= f;
                w.o[2 * G + 1][nt][i] *= f;
              }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = most[nt][j];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float old = w.top[nt][j], now = fmaxf(old, m - kUp);
          const float f = now == old ? 1.f : ex2(old - now);
          w.top[nt][j] = now;
          w.sum[nt][j] *= f;
#pragma unroll
          for (int G = 0; G < (Q4 ? C::GR : 1); ++G) w.pm[G][nt][j] *= f;
#pragma unroll
          for (int m2 = 0; m2 < D / 16; ++m2) {
            w.o[m2][nt][j] *= f;
            w.o[m2][nt][2 + j] *= f;
          }
        }
    }
#pragma unroll
    for (int s = 0; s < C::SUB; ++s) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = ex2(x[s][nt][i] - w.top[nt][i & 1]);
          x[s][nt][i] = p;
          w.sum[nt][i & 1] += p;
        }
      value_tile<D, Q4, NT, NW>(w, st, s, lane, x[s]);
    }
    __syncwarp();  // the stage is free for the next copy
    if (++slot == C::STAGES) slot = 0;
  }
  cp_wait<0>();
  __syncthreads();  // the ring becomes the warps' partial results

  // ------------------------------------------------------------------ join
  float* part = reinterpret_cast<float*>(smem) + warp * C::HEADS * (D + 2);  // O [head][D], then max, sum
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float sum = w.sum[nt][j];
      float pm[Q4 ? C::GR : 1];
#pragma unroll
      for (int G = 0; G < (Q4 ? C::GR : 1); ++G) pm[G] = w.pm[G][nt][j];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (Q4) {
#pragma unroll
          for (int G = 0; G < C::GR; ++G) pm[G] += __shfl_xor_sync(0xffffffffu, pm[G], o);
        }
      }
      const int head = nt * 8 + 2 * t4 + j;
      if (g == 0) {
        part[C::HEADS * D + head] = w.top[nt][j];
        part[C::HEADS * D + C::HEADS + head] = sum;
      }
#pragma unroll
      for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v = w.o[m][nt][2 * i + j];
          if constexpr (Q4)  // 2^24 (or 2^20: the code was 16-fold) 2^E_G
            v = fmaf(v, __uint_as_float(((m & 1) ? 274u << 23 : 278u << 23) - __float_as_uint(w.unit[m >> 1])), pm[m >> 1]);
          part[head * D + channel_of<D, Q4>(m, i, g)] = v;
        }
    }
  __syncthreads();
  const bool none = sp.units == 0;  // no rows are seen
  auto finish = [&](int e, int head, float o, float sum, float top) {
    a.O[head0 * D + e] = __float2bfloat16_rn(none ? 0.f : o / sum);
    if (e % D == 0) a.LSE[head0 + head] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  };
  float* out = reinterpret_cast<float*>(smem + C::SMEM - C::OUT);
  const float* parts = reinterpret_cast<const float*>(smem);
  constexpr int PS = C::HEADS * (D + 2);
  for (int e = tid; e < heads * D; e += C::THREADS) {
    const int head = e / D;
    float top = kLeast;
#pragma unroll
    for (int v = 0; v < NW; ++v) top = fmaxf(top, parts[v * PS + C::HEADS * D + head]);
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const float f = ex2(parts[v * PS + C::HEADS * D + head] - top);
      o = fmaf(parts[v * PS + e], f, o);
      sum = fmaf(parts[v * PS + C::HEADS * D + C::HEADS + head], f, sum);
    }
    if (a.cluster == 1) {
      finish(e, head, o, sum, top);
    } else {
      out[e] = o;
      if (e % D == 0) {
        out[C::HEADS * D + head] = top;
        out[C::HEADS * D + C::HEADS + head] = sum;
      }
    }
  }
  if (a.cluster == 1) return;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int n = a.cluster;
  for (int e = rank * C::THREADS + tid; e < heads * D; e += n * C::THREADS) {
    const int head = e / D;
    float top = kLeast;
    for (int v = 0; v < n; ++v) top = fmaxf(top, cluster.map_shared_rank(out, v)[C::HEADS * D + head]);
    float o = 0.f, sum = 0.f;
    for (int v = 0; v < n; ++v) {
      const float* q = cluster.map_shared_rank(out, v);
      const float f = ex2(q[C::HEADS * D + head] - top);
      o = fmaf(q[e], f, o);
      sum = fmaf(q[C::HEADS * D + C::HEADS + head], f, sum);
    }
    finish(e, head, o, sum, top);
  }
  cluster.sync();  // no CTA leaves while another reads its result
}

inline int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

cudaLaunchConfig_t config(long long blocks, int threads, int smem, int cluster, cudaStream_t s, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// How many clusters of n CTAs of this kernel the current device runs at once, asked
// once each.  A cluster sits in one GPC, so of large ones there are fewer than the
// SMs would hold, and one too many waits for a second wave.
constexpr int kMaxCluster = 16;

template <int D, bool Q4, int NT, int NW>
int clusters_at_once(int n) {
  using C = Cfg<D, Q4, NT, NW>;
  static std::atomic<int> known[64][kMaxCluster + 1];  // answer + 1; 0: not asked
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int k = known[dev][n].load(std::memory_order_relaxed);
  if (k == 0) {
    const auto kernel = stream_decode_kernel<D, Q4, NT, NW>;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config(n, C::THREADS, C::SMEM, n, nullptr, &attr);
    int most = 0;
    const bool ok =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) == cudaSuccess &&
        (n <= 8 || cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) &&
        cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) == cudaSuccess;
    if (!ok) cudaGetLastError();  // a refusal is an answer, not an error
    k = (ok ? most : 0) + 1;
    known[dev][n].store(k, std::memory_order_relaxed);
  }
  return k - 1;
}

// CTAs per (b, cached head): as many as all run at once, while a warp keeps two
// units.
template <int D, bool Q4, int NT, int NW>
int cluster_size(long long groups, long long max_units) {
  int n = kMaxCluster;
  while (n > 1 && (max_units < 2LL * NW * n || groups > clusters_at_once<D, Q4, NT, NW>(n))) --n;
  return n;
}

template <int D, bool Q4, int NT, int NW>
int launch(Args a, long long groups, int cluster, cudaStream_t s) {
  using C = Cfg<D, Q4, NT, NW>;
  const auto kernel = stream_decode_kernel<D, Q4, NT, NW>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return BSA_ERR_CUDA;
  a.cluster = cluster;
  const long long blocks = groups * cluster;
  if (blocks > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(blocks, C::THREADS, C::SMEM, cluster, s, &attr);
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return BSA_ERR_CUDA;
  }
  return BSA_OK;
}

// A lane with one head tile of a 4-bit cache fits sixteen warps on an SM, as two CTAs
// or as one.  Which of them puts more warps on the long axis depends on how clusters
// of the two pack into the GPCs.
template <int D, bool Q4, int NT>
int launch_best(const Args& a, long long groups, long long max_units, cudaStream_t s) {
  const int n = cluster_size<D, Q4, NT, 8>(groups, max_units);
  if constexpr (Q4 && NT == 1) {
    const int m = cluster_size<D, Q4, NT, 16>(groups, max_units);
    if (groups <= sm_count() && 2 * m > n && max_units >= 2LL * 16 * m) return launch<D, Q4, NT, 16>(a, groups, m, s);
  }
  return launch<D, Q4, NT, 8>(a, groups, n, s);
}

template <bool Q4>
int dispatch(Args a, int B, int d, long long max_units, cudaStream_t s) {
  const int nt = a.G > 8 ? 2 : 1;
  a.chunks = (a.G + 8 * nt - 1) / (8 * nt);
  const long long groups = static_cast<long long>(B) * a.Hkv * a.chunks;
  if (d == 64)
    return nt == 1 ? launch_best<64, Q4, 1>(a, groups, max_units, s) : launch_best<64, Q4, 2>(a, groups, max_units, s);
  return nt == 1 ? launch_best<128, Q4, 1>(a, groups, max_units, s) : launch_best<128, Q4, 2>(a, groups, max_units, s);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks that every step shares; fills what they cover.
int common(Args* a, const void* q, const void* k_new, const void* v_new, const int32_t* seq_len, int B,
           int H, int Hkv, int L, int d, float scale, void* O, float* LSE) {
  if (!q || !seq_len || !O || !LSE || (k_new == nullptr) != (v_new == nullptr)) return BSA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 1 || L < 1 || d < 1 || H % Hkv != 0 || !std::isfinite(scale))
    return BSA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(O) || (k_new && (!aligned16(k_new) || !aligned16(v_new))) ||
      (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0)
    return BSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || L > (1 << 30)) return BSA_ERR_UNSUPPORTED;  // row numbers and their ends are ints
  *a = Args{};
  a->q = static_cast<const __nv_bfloat16*>(q);
  a->k_new = static_cast<const __nv_bfloat16*>(k_new);
  a->v_new = static_cast<const __nv_bfloat16*>(v_new);
  a->seq_len = seq_len;
  a->O = static_cast<__nv_bfloat16*>(O);
  a->LSE = LSE;
  a->Hkv = Hkv;
  a->G = H / Hkv;
  a->L = L;
  a->scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  return BSA_OK;
}

int set_cache(Args* a, const bsa_q4_cache* c) {
  if (!c->k_codes || !c->k_params || !c->v_codes || !c->v_params) return BSA_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_params) || !aligned16(c->v_codes) || !aligned16(c->v_params))
    return BSA_ERR_INVALID_ARG;
  a->k = static_cast<unsigned char*>(c->k_codes);
  a->v = static_cast<unsigned char*>(c->v_codes);
  a->kp = static_cast<unsigned char*>(c->k_params);
  a->vp = static_cast<unsigned char*>(c->v_params);
  return BSA_OK;
}

long long window_units(int L, int window, int sinks, int unit) {
  const long long near = window < L ? window : L, far = sinks < L ? sinks : L;
  return (near + far + 2 * unit - 1) / unit;
}

}  // namespace sdec

int take_status(const void* symbol, uint32_t* status, int clear);
int stream_decode_status(uint32_t* status, int clear) {
  return take_status(&sdec::g_sdec_status, status, clear);
}
}  // namespace bsa

extern "C" int bsa_q4_decode(const void* q, const void* k_new, const void* v_new,
                             const bsa_q4_cache* cache, const int32_t* row_ptr,
                             const int32_t* col_idx, const int32_t* seq_len, int H, int block_size,
                             float scale, void* O, float* LSE, void* stream) {
  using namespace bsa::sdec;
  if (!cache || !row_ptr || !col_idx || block_size < 1) return BSA_ERR_INVALID_ARG;
  Args a;
  int rc = common(&a, q, k_new, v_new, seq_len, cache->B, H, cache->H, cache->L, cache->d, scale, O, LSE);
  if (rc == BSA_OK || rc == BSA_ERR_UNSUPPORTED) {
    const int bad = set_cache(&a, cache);
    if (bad != BSA_OK) return bad;
  }
  if (rc != BSA_OK) return rc;
  if (cache->L % block_size != 0) return BSA_ERR_INVALID_ARG;
  if (block_size != 32 && block_size != 64 && block_size != 128) return BSA_ERR_UNSUPPORTED;
  if (cache->L / block_size > kMaxM) return BSA_ERR_UNSUPPORTED;
  a.row_ptr = row_ptr;
  a.col_idx = col_idx;
  a.bs = block_size;
  a.M = cache->L / block_size;
  if (static_cast<long long>(a.Hkv) * a.M + 1 > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  // A row is taken to list an eighth of its blocks, as the CSR is not read on the host; it
  // decides how many CTAs a head is cut into.  Rows of 3 and 10 blocks and of all, 1 head of
  // 4 over 32768 rows: 7.3, 7.8 and 29 us; taken for half of them 9.6, 9.8 and 19, for a
  // 32nd 7.7, 10.4 and 89.  With 32 heads, or 8 of 131072 rows, the choice is that of half.
  return dispatch<true>(a, cache->B, cache->d, cache->L / 32 / 8, static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_q4_window_decode(const void* q, const void* k_new, const void* v_new,
                                    const bsa_q4_cache* cache, const int32_t* seq_len, int H, int window,
                                    int sinks, float scale, void* O, float* LSE, void* stream) {
  using namespace bsa::sdec;
  if (!cache || window < 1 || sinks < 0) return BSA_ERR_INVALID_ARG;
  Args a;
  int rc = common(&a, q, k_new, v_new, seq_len, cache->B, H, cache->H, cache->L, cache->d, scale, O, LSE);
  if (rc == BSA_OK || rc == BSA_ERR_UNSUPPORTED) {
    const int bad = set_cache(&a, cache);
    if (bad != BSA_OK) return bad;
  }
  if (rc != BSA_OK) return rc;
  a.window = window;
  a.sinks = sinks;
  return dispatch<true>(a, cache->B, cache->d, window_units(cache->L, window, sinks, 32),
                        static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_window_decode(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                 void* v_cache, const int32_t* seq_len, int B, int H, int Hkv, int L, int d,
                                 int window, int sinks, float scale, void* O, float* LSE, void* stream) {
  using namespace bsa::sdec;
  if (!k_cache || !v_cache || window < 1 || sinks < 0) return BSA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return BSA_ERR_INVALID_ARG;
  Args a;
  const int rc = common(&a, q, k_new, v_new, seq_len, B, H, Hkv, L, d, scale, O, LSE);
  if (rc != BSA_OK) return rc;
  a.k = static_cast<unsigned char*>(k_cache);
  a.v = static_cast<unsigned char*>(v_cache);
  a.window = window;
  a.sinks = sinks;
  return dispatch<false>(a, B, d, window_units(L, window, sinks, 16), static_cast<cudaStream_t>(stream));
}

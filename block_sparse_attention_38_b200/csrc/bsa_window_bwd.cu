// bsa_window_bwd.cu -- attention with a sliding window and first tokens that stay
// visible (sinks): the gradients of bsa_window_fwd.cu's forward.
//
// With P_qk = exp(scale q.k - LSE_q) over the visible pairs and D_q = dO_q . O_q:
//   dV_k = sum_q P dO_q,  dS = P (dO_q . v_k - D_q),
//   dQ_q = scale sum_k dS k_k,  dK_k = scale sum_q dS q_q,
// the sums for dK and dV over the G query heads that share the key/value head too.
//
// 10 d flops a visible pair, bound by the tensor cores.  Two kinds of tiles, each
// output row produced by one CTA (no atomics, the same bits every run), at the
// price of computing S and dP twice (14 d flops issued):
//   dkdv  one CTA per 128-key tile (or one each for parts of the group's heads, where
//         key tiles are few); a step is one query tile of one head:
//           S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
//   dq    a CTA per run of (head, 128-query tile); a step is one key tile:
//           S = Q K^T, dP = dO V^T;  dQ += dS K
// P and dS go to the second products from TMEM as bf16 (2^-8 at most, like the
// operands they meet); scores, P before that rounding and sums are fp32.  Over a
// query's keys dS adds up to about 0, so an offset that the keys share drops out of
// dQ but not out of dS's rounding errors, which it multiplies.  So their sum is kept
// (fp32), and one more product in each query tile takes it off again, spread evenly
// over the keys of the diagonal tile that the query sees (the diagonal tile's own
// errors over those of the same 32): that is exact for the offset, and leaves of each
// error its product with the key's distance from its neighbours' mean.  The diagonal
// tile comes last, after the sinks' (whose weights are the largest) and the window's.
//
// In both, sixteen warps (four threads a row) turn S into P (phase A), then dP
// into dS (phase B), while the tensor core works on the products of the other
// phase: dkdv issues dP(j) | dV(j), S(j+1) | dK(j), dP(j+1) | ..., so that A(j+1)
// runs beside dK(j) and dP(j+1), and B(j) beside dV(j) and S(j+1).  The order of
// issue by the one MMA thread protects P and dS, which lie over S and dP.
// TMEM, 512 columns at d = 128: S, dP, dV, dK; and S, dP, two dQ (the next tile
// begins while the last one's dQ is stored).
//
// The keys of the sink tiles are seen by every later query.  Their far queries
// (beyond the window) are cut into chunks that run as CTAs of their own and leave
// fp32 partial sums in the workspace, added up in a fixed order by sum_kernel, as are
// those of parts of a group's heads.
//
// Every wait is bounded.
#include "bsa_window.cuh"

namespace bsa {
namespace wbwd {

using namespace bsa::win;

constexpr int kSoftWarps = 16;           // elementwise: four per TMEM lane quadrant, 32 columns each
constexpr int kMmaWarp = 16, kLoadWarp = 17;
constexpr int kThreads = 18 * 32;
constexpr int kMaxChunks = 32;

__device__ unsigned int g_wbwd_status;

struct Args {
  const int32_t* lens;
  const float* LSE;          // [B, H, N]
  const float* Dq;           // [B, H, N]
  __nv_bfloat16* out[2];     // dV, dK, or dQ
  long long sb[2], sh[2], sn[2];
  int wide[2];               // the outputs' rows are 32-byte aligned
  float* part;               // partial sums, fp32: [B * Hkv, part tiles, parts, 2, 128, d]
  float* far_part;           // and of far queries [B * Hkv, sink tiles, chunks, 2, 128, d]
  int B, H, N;
  unsigned Hkv, G, tiles;
  int window, sinks;
  unsigned sink_tiles;       // key tiles with sinks that have far queries
  unsigned chunks;           // far chunks per sink tile, of chunk_tiles query tiles
  unsigned parts;            // near items per key tile, of some of the group's heads each
  unsigned part_tiles;       // key tiles whose items leave partial sums
  int chunk_tiles;
  int alone;                 // every query sees itself only
  unsigned items;
  float scale, scale_log2;
};

template <int D>
struct Cfg {
  static constexpr int TILE = kTile * D * 2;
  static constexpr int ATOMS = D / 64;
};

// Clears rows from `from` on of a tile that TMA has written, by one warp: what
// lies past a sequence's end may be NaN, and its weight 0 does not remove that.
template <int D>
__device__ __forceinline__ void clear_rows(unsigned char* tile, int from, int lane) {
  constexpr int P = D / 8;
  for (int e = lane; e < (kTile - from) * P; e += 32) {
    const int r = from + e / P, c = e % P;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * kAtom + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_shared();
}

// D (+)= A B^T over the d channels, both tiles K-major in shared memory; n columns.
template <int D>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint32_t idesc) {
  const uint64_t ad = sdesc_sw128(a_smem, 16, 1024), bd = sdesc_sw128(b_smem, 16, 1024);
  umma_qk_chain<D / 16>(d_tmem, static_cast<uint32_t>(ad), static_cast<uint32_t>(ad >> 32),
                        static_cast<uint32_t>(bd), static_cast<uint32_t>(bd >> 32), idesc);
}

// C (+)= A B with A in TMEM (bf16 pairs; columns 32 h .. 32 h + 15 hold entries
// 32 h .. 32 h + 31 of the summed index) and B a tile read MN-major.  narrow: the
// first 32 entries only.
template <int D>
__device__ __forceinline__ void mma_ts(uint32_t c_tmem, uint32_t a_tmem, uint32_t b_smem, bool narrow, bool add) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(128, D, false, true);
  const uint64_t bd = sdesc_sw128(b_smem, kAtom, 1024);
  const uint32_t lo = static_cast<uint32_t>(bd), hi = static_cast<uint32_t>(bd >> 32);
  umma_pv_slices2(c_tmem, a_tmem, lo, hi, kIdesc, add ? 1u : 0u);
  if (narrow) return;
  umma_pv_slices2(c_tmem, a_tmem + 32, lo + 256, hi, kIdesc, 1u);
  umma_pv_slices2(c_tmem, a_tmem + 64, lo + 512, hi, kIdesc, 1u);
  umma_pv_slices2(c_tmem, a_tmem + 96, lo + 768, hi, kIdesc, 1u);
}

// The n lowest bits.
__device__ __forceinline__ uint32_t upto(int n) { return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u); }

// Weights of columns that the row does not see become 0.
__device__ __forceinline__ void hide(float (&p)[32], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(seen & (1u << c))) p[c] = 0.f;
}

__device__ __forceinline__ void zero16(uint32_t taddr) {
  uint32_t z[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) z[c] = 0u;
  tmem_st16(taddr, z);
}

// 16 accumulator columns of this thread's row, times mul, to 16 bf16.
__device__ __forceinline__ void store_row16(uint32_t taddr, float mul, bool zero, __nv_bfloat16* dst, bool write,
                                            bool wide) {
  float w[16];
  tmem_ld16f_wait(taddr, w);
  if (!write) return;
  uint32_t x[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = zero ? 0u : pack_bf16x2(w[2 * c] * mul, w[2 * c + 1] * mul);
  if (wide) {
    store_256(dst, x);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// ------------------------------------------------------------ D = dO . O
struct DotArgs {
  const __nv_bfloat16 *o, *g;
  long long osb, osh, osn, gsb, gsh, gsn;
  float* D;
  long long rows;
  unsigned H, N;
};

constexpr int kDotRows = 4;  // rows a lane group, whose loads are all issued before the first is used

template <int D>
__global__ void __launch_bounds__(256) dot_kernel(const DotArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, part = lane % LPR;
  const long long r0 = (static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * RPW * kDotRows + lane / LPR;
  uint4 x[kDotRows], y[kDotRows];
#pragma unroll
  for (int i = 0; i < kDotRows; ++i) {
    const long long r = r0 + i * RPW;
    x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < a.rows) {
      const unsigned bh = static_cast<unsigned>(r / a.N);
      const long long q = r - static_cast<long long>(bh) * a.N;
      const unsigned b = bh / a.H, h = bh - b * a.H;
      x[i] = __ldg(reinterpret_cast<const uint4*>(a.o + b * a.osb + h * a.osh + q * a.osn + 8 * part));
      y[i] = __ldg(reinterpret_cast<const uint4*>(a.g + b * a.gsb + h * a.gsh + q * a.gsn + 8 * part));
    }
  }
#pragma unroll
  for (int i = 0; i < kDotRows; ++i) {
    const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16), acc);
      acc = fmaf(__uint_as_float(xs[e] & 0xffff0000u), __uint_as_float(ys[e] & 0xffff0000u), acc);
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (r0 + i * RPW < a.rows && part == 0) a.D[r0 + i * RPW] = acc;
  }
}

// ------------------------------------------------------------------- dK, dV
struct KvCtl {
  uint64_t kv_full, q_full[2], q_empty[2], do_full[2], do_empty[2];
  uint64_t s_full, p_ready, dp_full, ds_ready, acc_full, fix;
  uint32_t tmem_base;
  volatile int abort;
  alignas(16) float lse2[2][kTile];  // of a stage's queries: LSE log2(e), and D
  alignas(16) float dq[2][kTile];
};

struct KvItem {
  int b, hk, kt, k0, len;
  float* part;                       // the partial result's place (row 0 of dV), or null
  int g0, heads;                     // the group's heads that it takes
  bool far;
  int first, count;                  // query tiles
};

template <int D>
__device__ __forceinline__ KvItem kv_item(const Args& a, unsigned i) {
  KvItem it;
  const unsigned main_items = static_cast<unsigned>(a.B) * a.Hkv * a.tiles * a.parts;
  unsigned bh, part = 0;
  int chunk = -1;
  it.far = i >= main_items;
  if (!it.far) {
    unsigned r = i / a.parts;
    part = i - r * a.parts;
    bh = r / a.tiles;
    it.kt = static_cast<int>(r - bh * a.tiles);
    it.g0 = static_cast<int>(static_cast<unsigned long long>(part) * a.G / a.parts);
    it.heads = static_cast<int>(static_cast<unsigned long long>(part + 1) * a.G / a.parts) - it.g0;
  } else {
    i -= main_items;
    unsigned r = i / a.chunks;
    chunk = static_cast<int>(i - r * a.chunks);
    bh = r / a.sink_tiles;
    it.kt = static_cast<int>(r - bh * a.sink_tiles);
    it.g0 = 0;
    it.heads = static_cast<int>(a.G);
  }
  it.b = static_cast<int>(bh / a.Hkv);
  it.hk = static_cast<int>(bh - it.b * a.Hkv);
  it.k0 = it.kt * kTile;
  it.len = length_of(a.lens, it.b, a.N, &g_wbwd_status);
  const int last = (it.len - 1) / kTile;                       // last query tile with queries
  const int near = static_cast<int>(min(static_cast<long long>(a.tiles) - 1,
                                        (static_cast<long long>(it.k0) + kTile - 1 + a.window - 1) / kTile));
  int end;
  if (!it.far) {
    it.first = it.kt;
    end = min(near, last);
    it.part = it.kt < static_cast<int>(a.part_tiles)
                  ? a.part + ((static_cast<long long>(bh) * a.part_tiles + it.kt) * a.parts + part) * (2 * kTile * D)
                  : nullptr;
  } else {
    it.first = near + 1 + chunk * a.chunk_tiles;
    end = min(it.first + a.chunk_tiles - 1, last);
    it.part = a.far_part + ((static_cast<long long>(bh) * a.sink_tiles + it.kt) * a.chunks + chunk) * (2 * kTile * D);
  }
  it.count = it.k0 < it.len ? max(0, end - it.first + 1) : 0;
  return it;
}

template <int D>
__device__ __forceinline__ void dkdv_item(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                          const CUtensorMap& mo, const Args& a, unsigned item, unsigned char* smem) {
  using C = Cfg<D>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, false, false);
  constexpr int T_S = 0, T_DP = 128, T_DV = 256, T_DK = 256 + D;
  unsigned char *sK = smem, *sV = smem + C::TILE, *sQ = smem + 2 * C::TILE, *sO = smem + 4 * C::TILE;
  KvCtl* ctl = reinterpret_cast<KvCtl*>(smem + 6 * C::TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const KvItem it = kv_item<D>(a, item);
  const int G = it.heads, steps = it.count * G, head0 = it.hk * static_cast<int>(a.G) + it.g0;

  if (tid == 0) {
    mbar_init(&ctl->kv_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_full[s], 2);
      mbar_init(&ctl->q_empty[s], 1);
      mbar_init(&ctl->do_full[s], 1);
      mbar_init(&ctl->do_empty[s], 1);
    }
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->p_ready, kSoftWarps);
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->ds_ready, kSoftWarps);
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->fix, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_bounded(bar, parity, &ctl->abort, &g_wbwd_status);
  };

  if (warp == kLoadWarp && steps > 0) {
    // ------------------------------------------------------------- producer
    bool ok = true;
    uint32_t fixes = 0;
    if (lane == 0) {
      mbar_arrive_expect_tx(&ctl->kv_full, 2 * C::TILE);
      for (int c = 0; c < C::ATOMS; ++c) {
        tma_load_4d(sK + c * kAtom, &mk, &ctl->kv_full, 64 * c, it.k0, it.hk, it.b);
        tma_load_4d(sV + c * kAtom, &mv, &ctl->kv_full, 64 * c, it.k0, it.hk, it.b);
      }
    }
    // LSE and D of a step's queries, loaded a step ahead: four of each a lane
    float lse[4], dd[4];
    auto fetch = [&](int j) {
      const int qt = j / G;
      const long long row = (static_cast<long long>(it.b) * a.H + head0 + j - qt * G) * a.N;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int q = (it.first + qt) * kTile + r * 32 + lane;
        lse[r] = j < steps && q < a.N ? a.LSE[row + q] : 0.f;
        dd[r] = j < steps && q < a.N ? a.Dq[row + q] : 0.f;
      }
    };
    fetch(0);
    int issued = 0;
    for (int j = 0; j < steps && ok; ++j) {
      const int s = j & 1, qt = j / G, q0 = (it.first + qt) * kTile, h = head0 + j - qt * G;
      const bool fix = q0 + kTile > it.len && it.len < a.N;
      for (int w = 0; w < 2 && ok; ++w) {
        unsigned char* dst = (w == 0 ? sQ : sO) + s * C::TILE;
        uint64_t* full = w == 0 ? &ctl->q_full[s] : &ctl->do_full[s];
        if (j >= 2) ok = __all_sync(0xffffffffu, wait(w == 0 ? &ctl->q_empty[s] : &ctl->do_empty[s], ((j >> 1) - 1) & 1));
        if (!ok) break;
        uint64_t* bar = fix ? &ctl->fix : full;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, C::TILE);
          for (int c = 0; c < C::ATOMS; ++c) tma_load_4d(dst + c * kAtom, w == 0 ? &mq : &mo, bar, 64 * c, q0, h, it.b);
        }
        if (w == 0) {  // q_full takes a second arrival, for these
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            ctl->lse2[s][r * 32 + lane] = lse[r] * kLog2e;
            ctl->dq[s][r * 32 + lane] = dd[r];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
          fetch(j + 1);
        }
        if (fix) {
          ok = __all_sync(0xffffffffu, wait(&ctl->fix, fixes & 1));
          ++fixes;
          if (ok) clear_rows<D>(dst, it.len - q0, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
      }
      if (ok) issued = j + 1;
    }
    // copies in flight must land before the block's shared memory goes away
    if (lane == 0) {
      wait_drain(&ctl->kv_full, 0, &g_wbwd_status);
      for (int s = 0; s < 2; ++s)
        if (issued > s) {
          wait_drain(&ctl->q_full[s], ((issued - 1 - s) >> 1) & 1, &g_wbwd_status);
          wait_drain(&ctl->do_full[s], ((issued - 1 - s) >> 1) & 1, &g_wbwd_status);
        }
      if (fixes > 0) wait_drain(&ctl->fix, (fixes - 1) & 1, &g_wbwd_status);
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    // The whole warp walks the steps, so that what the products need stays in
    // uniform registers; one lane issues them.
    const uint32_t k = smem_u32(sK), v = smem_u32(sV), q = smem_u32(sQ), o = smem_u32(sO);
    const uint32_t t = __shfl_sync(0xffffffffu, tmem, 0);
    const bool lead = elect_one();
    auto arrived = [&](uint64_t* bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, wait(bar, parity))) return false;
      tc_fence_after();
      return true;
    };
    bool ok = steps > 0 && arrived(&ctl->kv_full, 0) && arrived(&ctl->q_full[0], 0);
    if (ok && lead) {
      mma_ss<D>(t + T_S, k, q, kIdesc);
      umma_commit(&ctl->s_full);
    }
    for (int j = 0; j < steps && ok; ++j) {
      const int s = j & 1;
      const uint32_t qs = q + s * C::TILE, qn = q + (s ^ 1) * C::TILE, os = o + s * C::TILE;
      if (!(ok = arrived(&ctl->do_full[s], (j >> 1) & 1))) break;
      if (lead) {
        mma_ss<D>(t + T_DP, v, os, kIdesc);
        umma_commit(&ctl->dp_full);
      }
      if (j + 1 < steps && !(ok = arrived(&ctl->q_full[s ^ 1], ((j + 1) >> 1) & 1))) break;
      if (!(ok = arrived(&ctl->p_ready, j & 1))) break;
      if (lead) {
        mma_ts<D>(t + T_DV, t + T_S, os, false, j > 0);
        umma_commit(&ctl->do_empty[s]);
        if (j + 1 < steps) {
          mma_ss<D>(t + T_S, k, qn, kIdesc);
          umma_commit(&ctl->s_full);
        }
      }
      if (!(ok = arrived(&ctl->ds_ready, j & 1))) break;
      if (lead) {
        mma_ts<D>(t + T_DK, t + T_DP, qs, false, j > 0);
        umma_commit(&ctl->q_empty[s]);
      }
    }
    if (lead) {
      umma_commit(&ctl->acc_full);  // every MMA issued must complete before TMEM is released
      wait_drain(&ctl->acc_full, 0, &g_wbwd_status);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------- elementwise
    const int wu = __shfl_sync(0xffffffffu, warp, 0);  // the same for all lanes, and known to be
    const int quad = wu & 3, part = wu >> 2;
    const int row = quad * 32 + lane, k = it.k0 + row, kw = it.k0 + quad * 32;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_s = t_lane + T_S + 32 * part, t_dp = t_lane + T_DP + 32 * part;
    // of a far chunk only the sinks' rows are used: other warps only keep step
    const bool idle = it.far && kw >= a.sinks;
    bool ok = true;
    for (int j = 0; j < steps && ok; ++j) {
      const int s = j & 1, qw = (it.first + j / G) * kTile + 32 * part;  // this thread's first query
      // whether no key of the warp is seen by any of the 32 queries, or every one by all
      const bool none = idle || qw + 31 < kw || qw >= it.len || (qw - (kw + 31) >= a.window && kw >= a.sinks);
      const bool all = qw >= kw + 31 && qw + 32 <= it.len && (qw + 31 - kw < a.window || kw + 32 <= a.sinks);
      float p[32];
      // q_full too: it orders the producer's writes of lse2 and dq before their reads
      ok = __all_sync(0xffffffffu, wait(&ctl->s_full, j & 1) && wait(&ctl->q_full[s], (j >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      if (!none) {
        tmem_ld32f_wait(t_s, p);
        const float4* l4 = reinterpret_cast<const float4*>(ctl->lse2[s] + 32 * part);
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 l = l4[c / 4];
          p[c] = ex2_approx(fmaf(p[c], a.scale_log2, -l.x));
          p[c + 1] = ex2_approx(fmaf(p[c + 1], a.scale_log2, -l.y));
          p[c + 2] = ex2_approx(fmaf(p[c + 2], a.scale_log2, -l.z));
          p[c + 3] = ex2_approx(fmaf(p[c + 3], a.scale_log2, -l.w));
        }
        if (!all) {  // column c is query qw + c
          const int lo = k - qw;
          hide(p, ~upto(lo) & upto(it.len - qw) & (k < a.sinks ? ~0u : upto(lo + a.window)));
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        tmem_st16(t_s, pk);
      } else if (!idle) {
        zero16(t_s);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_ready);
      ok = __all_sync(0xffffffffu, wait(&ctl->dp_full, j & 1));
      if (!ok) break;
      tc_fence_after();
      if (!none) {
        const float4* d4 = reinterpret_cast<const float4*>(ctl->dq[s] + 32 * part);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[16];
          tmem_ld16f_wait(t_dp + 16 * h, x);
          uint32_t pk[8];
#pragma unroll
          for (int c = 0; c < 16; c += 4) {
            const float4 dd = d4[4 * h + c / 4];
            x[c] = p[16 * h + c] * (x[c] - dd.x);
            x[c + 1] = p[16 * h + c + 1] * (x[c + 1] - dd.y);
            x[c + 2] = p[16 * h + c + 2] * (x[c + 2] - dd.z);
            x[c + 3] = p[16 * h + c + 3] * (x[c + 3] - dd.w);
          }
          if (!all) {  // a hidden pair has p = 0, and its dP may be anything
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (p[16 * h + c] == 0.f) x[c] = 0.f;
            if (h == 0 && qw == 0) x[0] = 0.f;  // query 0 sees one key: its P is 1 whatever the score
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) pk[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
          tmem_st8(t_dp + 8 * h, pk);
        }
      } else if (!idle) {
        zero16(t_dp);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->ds_ready);
    }
    if (ok && steps > 0) ok = __all_sync(0xffffffffu, wait(&ctl->acc_full, 0));
    if (ok) {
      tc_fence_after();
      const bool none = steps == 0 || k >= it.len;
      const int c0 = part * (D / 4);
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        const uint32_t t_acc = t_lane + (w == 0 ? T_DV : T_DK) + c0;
        const float mul = w == 0 ? 1.f : a.scale;
        const bool zero = none || (w == 1 && a.alone);
        if (it.part == nullptr) {
          __nv_bfloat16* dst = a.out[w] + it.b * a.sb[w] + it.hk * a.sh[w] + static_cast<long long>(k) * a.sn[w] + c0;
#pragma unroll 1
          for (int c = 0; c < D / 4; c += 16) store_row16(t_acc + c, mul, zero, dst + c, k < a.N, a.wide[w]);
        } else if (!idle) {
          float* dst = it.part + (w * kTile + row) * D + c0;
#pragma unroll 1
          for (int c = 0; c < D / 4; c += 16) {
            float x[16];
            tmem_ld16f_wait(t_acc + c, x);
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(dst + c + e) =
                  zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                       : make_float4(x[e] * mul, x[e + 1] * mul, x[e + 2] * mul, x[e + 3] * mul);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds a key tile's partial sums in a fixed order: the near queries' of each part of
// the group's heads, then each far chunk's (which hold the sinks' rows only).
template <int D>
__global__ void __launch_bounds__(256) sum_kernel(const Args a) {
  const long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;  // (tile, w, row, 4 channels)
  constexpr int Q = D / 4;
  const long long total = static_cast<long long>(a.B) * a.Hkv * a.part_tiles * 2 * kTile * Q;
  if (e >= total) return;
  const int c = static_cast<int>(e % Q);
  long long r = e / Q;
  const int row = static_cast<int>(r % kTile);
  r /= kTile;
  const int w = static_cast<int>(r % 2);
  const long long tile = r / 2;
  const int kt = static_cast<int>(tile % a.part_tiles), k = kt * kTile + row;
  if (k >= a.N) return;
  const long long bh = tile / a.part_tiles;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float* from, unsigned n) {
    from += (w * kTile + row) * D + 4 * c;
    for (unsigned i = 0; i < n; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(from + static_cast<long long>(i) * (2 * kTile * D));
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
  };
  add(a.part + tile * a.parts * (2 * kTile * D), a.parts);
  if (kt < static_cast<int>(a.sink_tiles) && k < a.sinks)
    add(a.far_part + (bh * a.sink_tiles + kt) * a.chunks * (2 * kTile * D), a.chunks);
  const int b = static_cast<int>(bh / a.Hkv), hk = static_cast<int>(bh % a.Hkv);
  *reinterpret_cast<uint2*>(a.out[w] + b * a.sb[w] + hk * a.sh[w] + static_cast<long long>(k) * a.sn[w] + 4 * c) =
      make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// ----------------------------------------------------------------------- dQ
struct QCtl {
  uint64_t q_full[2], q_empty[2], do_full, do_empty;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full, s_free, dp_full, ds_ready;
  uint64_t dq_full[2], dq_free[2], fix, final_bar;
  uint32_t tmem_base;
  volatile int abort;
  float off[4][kTile];       // sums of dS's rounding errors up to the diagonal tile, of a row's four threads
};

struct QItem {
  int b, h, hk, q0, len;
  int sunk, first, steps;  // the sinks' tiles, then the window's, of which the diagonal one is the last
  __device__ __forceinline__ int key0(int j) const {
    return (j < sunk ? j : first + j - sunk) * kTile;
  }
};

__device__ __forceinline__ QItem q_item(const Args& a, unsigned i) {
  QItem it;
  unsigned r = i / a.G;
  const int g = static_cast<int>(i - r * a.G);
  i = r / a.tiles;
  it.q0 = static_cast<int>(r - i * a.tiles) * kTile;
  it.b = static_cast<int>(i / a.Hkv);
  it.hk = static_cast<int>(i - it.b * a.Hkv);
  it.h = it.hk * a.G + g;
  it.len = length_of(a.lens, it.b, a.N, &g_wbwd_status);
  it.first = max(0, it.q0 - a.window + 1) / kTile;
  it.sunk = min((min(a.sinks, it.len) + kTile - 1) / kTile, it.first);
  it.steps = it.q0 < it.len ? it.sunk + (min(it.q0 + kTile, it.len) - 1) / kTile - it.first + 1 : 0;
  return it;
}

// Steps of this CTA's items, one after another.
struct QWalk {
  unsigned i, stride;
  QItem it;
  int j, n;          // step of the item, and the item's number among those with steps
  bool valid;
  __device__ __forceinline__ void seek(const Args& a) {
    for (valid = false; i < a.items; i += stride) {
      it = q_item(a, i);
      if (it.steps > 0) {
        valid = true;
        break;
      }
    }
  }
  __device__ __forceinline__ void begin(const Args& a, unsigned first_item, unsigned step) {
    i = first_item;
    stride = step;
    j = n = 0;
    seek(a);
  }
  __device__ __forceinline__ void next(const Args& a) {
    if (++j < it.steps) return;
    j = 0;
    ++n;
    i += stride;
    seek(a);
  }
  __device__ __forceinline__ bool last() const { return j + 1 == it.steps; }
  // a sink tile outside the window that shows at most 32 keys takes 32 columns
  __device__ __forceinline__ bool narrow(const Args& a) const {
    return j < it.sunk && a.sinks - j * kTile <= 32;
  }
};

template <int D>
__device__ __forceinline__ void dq_items(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                                         const CUtensorMap& mo, const Args& a, unsigned first_item, unsigned stride,
                                         unsigned char* smem) {
  using C = Cfg<D>;
  constexpr int T_S = 0, T_DP = 128, T_DQ = 256;  // two dQ, D columns each
  unsigned char *sQ = smem, *sO = smem + 2 * C::TILE, *sK = smem + 3 * C::TILE, *sV = smem + 5 * C::TILE;
  QCtl* ctl = reinterpret_cast<QCtl*>(smem + 7 * C::TILE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_full[s], 1);
      mbar_init(&ctl->q_empty[s], 1);
      mbar_init(&ctl->k_full[s], 1);
      mbar_init(&ctl->k_empty[s], 1);
      mbar_init(&ctl->v_full[s], 1);
      mbar_init(&ctl->v_empty[s], 1);
      mbar_init(&ctl->dq_full[s], 1);
      mbar_init(&ctl->dq_free[s], kSoftWarps);
    }
    mbar_init(&ctl->do_full, 1);
    mbar_init(&ctl->do_empty, 1);
    mbar_init(&ctl->s_full, 1);
    mbar_init(&ctl->s_free, kSoftWarps);
    mbar_init(&ctl->dp_full, 1);
    mbar_init(&ctl->ds_ready, kSoftWarps);
    mbar_init(&ctl->fix, 1);
    mbar_init(&ctl->final_bar, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return wait_bounded(bar, parity, &ctl->abort, &g_wbwd_status);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------- producer
    QWalk w;
    w.begin(a, first_item, stride);
    bool ok = true;
    uint32_t t = 0, items = 0, fixes = 0;  // steps, items whose tiles were issued
    for (; w.valid && ok; w.next(a)) {
      if (w.j == 0) {
        const int s = w.n & 1;
        if (w.n >= 2) ok = warp_wait(&ctl->q_empty[s], ((w.n >> 1) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl->q_full[s], C::TILE);
          for (int c = 0; c < C::ATOMS; ++c)
            tma_load_4d(sQ + s * C::TILE + c * kAtom, &mq, &ctl->q_full[s], 64 * c, w.it.q0, w.it.h, w.it.b);
        }
      }
      const int k0 = w.it.key0(w.j), s = t & 1;
      const bool fix = k0 + kTile > w.it.len && w.it.len < a.N;  // dS K: key rows past the end must be 0
      if (t >= 2) ok = warp_wait(&ctl->k_empty[s], ((t >> 1) - 1) & 1);
      if (!ok) break;
      {
        uint64_t* bar = fix ? &ctl->fix : &ctl->k_full[s];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, C::TILE);
          for (int c = 0; c < C::ATOMS; ++c)
            tma_load_4d(sK + s * C::TILE + c * kAtom, &mk, bar, 64 * c, k0, w.it.hk, w.it.b);
        }
        if (fix) {
          ok = warp_wait(&ctl->fix, fixes & 1);
          ++fixes;
          if (ok) clear_rows<D>(sK + s * C::TILE, w.it.len - k0, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->k_full[s]);
        }
      }
      if (w.j == 0) {
        if (w.n >= 1) ok = ok && warp_wait(&ctl->do_empty, (w.n - 1) & 1);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&ctl->do_full, C::TILE);
          for (int c = 0; c < C::ATOMS; ++c)
            tma_load_4d(sO + c * kAtom, &mo, &ctl->do_full, 64 * c, w.it.q0, w.it.h, w.it.b);
        }
        if (ok) ++items;
      }
      if (t >= 2) ok = ok && warp_wait(&ctl->v_empty[s], ((t >> 1) - 1) & 1);
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(&ctl->v_full[s], C::TILE);
        for (int c = 0; c < C::ATOMS; ++c)
          tma_load_4d(sV + s * C::TILE + c * kAtom, &mv, &ctl->v_full[s], 64 * c, k0, w.it.hk, w.it.b);
      }
      if (ok) ++t;
    }
    if (lane == 0) {
      for (uint32_t s = 0; s < 2; ++s) {
        if (t > s) {
          wait_drain(&ctl->k_full[s], ((t - 1 - s) >> 1) & 1, &g_wbwd_status);
          wait_drain(&ctl->v_full[s], ((t - 1 - s) >> 1) & 1, &g_wbwd_status);
        }
        if (items > s) wait_drain(&ctl->q_full[s], ((items - 1 - s) >> 1) & 1, &g_wbwd_status);
      }
      if (items > 0) wait_drain(&ctl->do_full, (items - 1) & 1, &g_wbwd_status);
      if (fixes > 0) wait_drain(&ctl->fix, (fixes - 1) & 1, &g_wbwd_status);
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issuer
    const uint32_t k = smem_u32(sK), v = smem_u32(sV), q = smem_u32(sQ), o = smem_u32(sO);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const bool lead = elect_one();
    constexpr uint32_t kWide = idesc_bf16_f32(128, 128, false, false), kNarrow = idesc_bf16_f32(128, 32, false, false);
    auto arrived = [&](uint64_t* bar, uint32_t parity) {
      if (!warp_wait(bar, parity)) return false;
      tc_fence_after();
      return true;
    };
    // S of step t, the j-th of the n-th item
    auto scores = [&](uint32_t t, int n, bool first, bool narrow, bool last) {
      if (first && !arrived(&ctl->q_full[n & 1], (n >> 1) & 1)) return false;
      if (t > 0 && !arrived(&ctl->s_free, (t - 1) & 1)) return false;
      if (!arrived(&ctl->k_full[t & 1], (t >> 1) & 1)) return false;
      if (lead) {
        mma_ss<D>(tm + T_S, q + (n & 1) * C::TILE, k + (t & 1) * C::TILE, narrow ? kNarrow : kWide);
        umma_commit(&ctl->s_full);
        if (last) umma_commit(&ctl->q_empty[n & 1]);
      }
      return true;
    };
    // One step, with the next one's S before its dS is waited for.
    auto step = [&](uint32_t t, int n, bool first, bool narrow, bool last, bool more, int nn, bool nfirst, bool nnarrow,
                    bool nlast) {
      const int s = t & 1, buf = n & 1;
      if (first && !arrived(&ctl->do_full, n & 1)) return false;
      if (!arrived(&ctl->v_full[s], (t >> 1) & 1)) return false;
      if (lead) {
        mma_ss<D>(tm + T_DP, o, v + s * C::TILE, narrow ? kNarrow : kWide);
        umma_commit(&ctl->dp_full);
        umma_commit(&ctl->v_empty[s]);
        if (last) umma_commit(&ctl->do_empty);
      }
      if (more && !scores(t + 1, nn, nfirst, nnarrow, nlast)) return false;
      if (first && n >= 2 && !arrived(&ctl->dq_free[buf], ((n >> 1) - 1) & 1)) return false;
      if (!arrived(&ctl->ds_ready, t & 1)) return false;
      if (lead) {
        mma_ts<D>(tm + T_DQ + buf * D, tm + T_DP, k + s * C::TILE, narrow, !first);
        if (last) mma_ts<D>(tm + T_DQ + buf * D, tm + T_DP + 16, k + s * C::TILE, false, true);
        umma_commit(&ctl->k_empty[s]);
        if (last) umma_commit(&ctl->dq_full[buf]);
      }
      return true;
    };
    QWalk w;
    w.begin(a, first_item, stride);
    bool ok = !w.valid || scores(0, 0, true, w.narrow(a), w.last());
    uint32_t t = 0;
    while (w.valid && ok) {
      const int n = w.n, steps = w.it.steps;
      for (; w.j + 1 < steps && ok; ++w.j, ++t) {
        const bool narrow = w.narrow(a), first = w.j == 0;
        QWalk nx = w;
        ++nx.j;
        ok = step(t, n, first, narrow, false, true, n, false, nx.narrow(a), nx.j + 1 == steps);
      }
      const bool one = steps == 1, narrow = w.narrow(a);
      w.next(a);
      ok = ok && step(t, n, one, narrow, true, w.valid, n + 1, true, w.valid && w.narrow(a), w.valid && w.last());
      ++t;
    }
    if (lead) {
      umma_commit(&ctl->final_bar);
      wait_drain(&ctl->final_bar, 0, &g_wbwd_status);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------- elementwise
    const int wu = __shfl_sync(0xffffffffu, warp, 0);  // the same for all lanes, and known to be
    const int quad = wu & 3, part = wu >> 2, row = quad * 32 + lane, c0 = part * (D / 4);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_s = t_lane + T_S + 32 * part, t_dp = t_lane + T_DP + 32 * part;
    auto place = [&](const QItem& it) {
      return a.out[0] + it.b * a.sb[0] + it.h * a.sh[0] + static_cast<long long>(it.q0 + row) * a.sn[0] + c0;
    };
    // tiles without a visible pair first: nothing in flight depends on them
    if (a.lens != nullptr)
      for (unsigned i = first_item; i < a.items; i += stride) {
        const QItem it = q_item(a, i);
        if (it.steps > 0 || it.q0 + row >= a.N) continue;
        uint4* dst = reinterpret_cast<uint4*>(place(it));
        for (int c = 0; c < D / 32; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    // what is left to do for the item before: its dQ
    __nv_bfloat16* dst = nullptr;
    bool live = false, write = false;
    auto store = [&](int n) {
      const int buf = n & 1;
      if (!warp_wait(&ctl->dq_full[buf], (n >> 1) & 1)) return false;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 4; c += 16)
        store_row16(t_lane + T_DQ + buf * D + c0 + c, a.scale, !live, dst + c, write, a.wide[0]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->dq_free[buf]);
      return true;
    };
    bool ok = true;
    int n = 0;
    uint32_t t = 0;
    for (unsigned i = first_item; i < a.items && ok; i += stride) {
      const QItem it = q_item(a, i);
      if (it.steps == 0) continue;
      const int q = it.q0 + row, qw = it.q0 + 32 * quad;
      const long long at = (static_cast<long long>(it.b) * a.H + it.h) * a.N + q;
      const float lse2 = q < it.len ? a.LSE[at] * kLog2e : 0.f;
      const float dd = q < it.len ? a.Dq[at] : 0.f;
      float off = 0.f;  // sum of dS's rounding errors over this thread's keys, before the diagonal tile and in it
      for (int j = 0; j < it.steps && ok; ++j, ++t) {
        const int kw = it.key0(j) + 32 * part;  // this thread's first key
        const bool narrow = j < it.sunk && a.sinks - j * kTile <= 32;
        // whether no row of the warp sees any of the 32 keys, or every row all of them
        const bool none = (narrow && part > 0) || kw > qw + 31 || (qw - (kw + 31) >= a.window && kw >= a.sinks);
        const bool all = kw + 31 <= qw && qw + 32 <= it.len && (qw + 31 - kw < a.window || kw + 32 <= a.sinks);
        float p[32];
        if (!(ok = warp_wait(&ctl->s_full, t & 1))) break;
        tc_fence_after();
        if (!none) tmem_ld32f_wait(t_s, p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->s_free);
        if (!none) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            fma2(p[c], p[c + 1], a.scale_log2, -lse2);
            p[c] = ex2_approx(p[c]);
            p[c + 1] = ex2_approx(p[c + 1]);
          }
          if (!all)  // column c is key kw + c
            hide(p, q < it.len ? upto(q - kw + 1) & (~upto(q - a.window + 1 - kw) | upto(a.sinks - kw)) : 0u);
        }
        if (!(ok = warp_wait(&ctl->dp_full, t & 1))) break;
        tc_fence_after();
        if (!none) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[16];
            tmem_ld16f_wait(t_dp + 16 * h, x);
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = p[16 * h + c] * (x[c] - dd);
            if (!all) {  // a hidden pair has p = 0, and its dP may be anything
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (p[16 * h + c] == 0.f || q == 0) x[c] = 0.f;  // query 0 sees one key: dS = 0
            }
            uint32_t pk[8];
            float ea = 0.f, eb = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              pk[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
              float ra = __uint_as_float(pk[c] << 16), rb = __uint_as_float(pk[c] & 0xffff0000u);
              sub2v(ra, rb, x[2 * c], x[2 * c + 1]);
              acc2(ea, eb, ra, rb);
            }
            off += ea + eb;
            tmem_st8(t_dp + 8 * h, pk);
          }
        } else if (!narrow) {
          zero16(t_dp);
        }
        if (j >= it.steps - 2) {
          int r = row, c0 = 32 * part;
          asm volatile("" : "+r"(r), "+r"(c0));  // what follows is computed here, not kept from the loop's start
          if (j == it.steps - 2) {  // read at the next step, written again only after that step's ds_ready
            ctl->off[c0 >> 5][r] = off;
            off = 0.f;
          } else {  // the diagonal tile: its key of column c is q - r + c
            const int lo = max(0, r - a.window + 1), below = min(max(a.sinks - q + r, 0), lo);
            const uint32_t seen = upto(r + 1 - c0) & (~upto(lo - c0) | upto(below - c0));
            float share = seen ? __fdividef(-off, static_cast<float>(__popc(seen))) : 0.f;
            if (it.steps > 1) {
              // this step's dP was issued after the last step's ds_ready of all warps: this
              // is true at once, and orders their writes before the reads
              mbar_try_wait(&ctl->ds_ready, (t - 1) & 1);
              const float sum = (ctl->off[0][r] + ctl->off[1][r]) + (ctl->off[2][r] + ctl->off[3][r]);
              share -= __fdividef(sum, static_cast<float>(r + 1 - lo + below));  // the keys that the row sees
            }
            const uint32_t both = pack_bf16x2(share, share);
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c)
              pk[c] = both & ((seen & (1u << 2 * c) ? 0xffffu : 0u) | (seen & (2u << 2 * c) ? 0xffff0000u : 0u));
            tmem_st16(t_dp + 16, pk);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->ds_ready);
        // the last tile's dQ is stored here, beside this tile's products
        if (j == 0 && n > 0) ok = store(n - 1);
      }
      dst = place(it);
      live = q < it.len && !a.alone;
      write = q < a.N;
      ++n;
    }
    if (ok && n > 0) store(n - 1);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One launch for both: the key tiles' blocks first (their lengths differ little, but
// a wave of them is long), then the query tiles' in runs, which fill the SMs
// that the last key tiles leave idle (565 us as two launches, 537 as one: 32 heads x
// 8192 x 128, window 1024).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_backward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                           const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                           const Args kv, const Args qa) {
  extern __shared__ __align__(1024) unsigned char smem[];  // swizzle atoms need 1024 bytes
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_wbwd_status, BSA_STATUS_INTERNAL);
    return;
  }
  if (blockIdx.x < kv.items)
    dkdv_item<D>(mq, mk, mv, mo, kv, blockIdx.x, smem);
  else
    dq_items<D>(mq, mk, mv, mo, qa, blockIdx.x - kv.items, gridDim.x - kv.items, smem);
}

// ------------------------------------------------------------------ host side
// How the far queries of the sinks are cut: into chunks of about a near item's
// length, at most kMaxChunks.  And where key tiles are few, how the heads of a group
// are, so that no long item is what all wait for: into parts until there are 60 items,
// which leaves the rest of the 148 SMs to the query tiles (8 heads over 1, 4096 x 128,
// window 1024, 4 sinks: 139 us whole; 82, 89 and 93 for 60, 85 and 148 items).  Items of
// few steps stay whole, as a part costs a beginning and a pass over fp32 sums.
constexpr int kItemsWanted = 60, kStepsWorthParts = 8;

struct Plan {
  int tiles, sink_tiles, chunks, chunk_tiles, parts, part_tiles;
  size_t d_bytes, part_bytes, far_bytes;
  size_t bytes() const { return d_bytes + part_bytes + far_bytes; }
};

Plan make_plan(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  Plan p;
  const long long w = window < N ? window : N, s = sinks < N ? sinks : N;
  p.tiles = (N + kTile - 1) / kTile;
  // near query tiles of key tile t end at t + (kTile - 1 + w - 1) / kTile
  const long long near = (kTile + w - 2) / kTile;
  const long long far = p.tiles - 1 - near;  // far query tiles of key tile 0
  const long long G = H / Hkv, items = static_cast<long long>(B) * Hkv * p.tiles;
  const long long steps = (near + 1 < p.tiles ? near + 1 : p.tiles) * G;
  p.parts = 1;
  if (items < kItemsWanted && steps >= kStepsWorthParts) {
    const long long n = (kItemsWanted + items - 1) / items;
    p.parts = static_cast<int>(n < G ? n : G);
  }
  p.sink_tiles = p.chunks = p.chunk_tiles = 0;
  if (far > 0 && s > 0) {
    const long long st = (s + kTile - 1) / kTile;
    p.sink_tiles = static_cast<int>(st < far ? st : far);  // tile t has far - t of them
    long long n = (far + near) / (near + 1) * p.parts;
    n = n > kMaxChunks ? kMaxChunks : (n > far ? far : n);
    p.chunk_tiles = static_cast<int>((far + n - 1) / n);
    p.chunks = static_cast<int>((far + p.chunk_tiles - 1) / p.chunk_tiles);
  }
  p.part_tiles = p.parts > 1 ? p.tiles : p.sink_tiles;
  const size_t rows = static_cast<size_t>(B) * H * N;
  p.d_bytes = (rows * 4 + 255) / 256 * 256;
  const size_t sums = static_cast<size_t>(B) * Hkv * 2 * kTile * d * 4;  // dV and dK of a tile for every head
  p.part_bytes = sums * p.part_tiles * p.parts;
  p.far_bytes = sums * p.sink_tiles * p.chunks;
  return p;
}

template <int D>
int launch(const bsa_view* q, const bsa_view* k, const bsa_view* v, const bsa_view* o, const bsa_view* g,
           Args a, float* Dq, const bsa_view* dq, const bsa_view* dk, const bsa_view* dv, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map(&mq, q, a.B, a.H, a.N, D) || !make_map(&mk, k, a.B, a.Hkv, a.N, D) ||
      !make_map(&mv, v, a.B, a.Hkv, a.N, D) || !make_map(&mo, g, a.B, a.H, a.N, D))
    return BSA_ERR_CUDA;
  // One CTA (and its 512 TMEM columns) per SM: more than half an SM's shared memory.
  static_assert(6 * C::TILE + sizeof(KvCtl) <= 232448 && 7 * C::TILE + sizeof(QCtl) <= 232448, "227 KB");
  const int kv_smem = 6 * C::TILE + static_cast<int>(sizeof(KvCtl)), q_smem = 7 * C::TILE + static_cast<int>(sizeof(QCtl));
  int smem = kv_smem > q_smem ? kv_smem : q_smem;
  smem = smem < 120 * 1024 ? 120 * 1024 : smem;
  const auto kernel = window_backward_kernel<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return BSA_ERR_CUDA;
  auto stride = [](int n, long long x) { return n > 1 ? x : 0; };

  DotArgs d;
  d.o = static_cast<const __nv_bfloat16*>(o->data);
  d.g = static_cast<const __nv_bfloat16*>(g->data);
  d.osb = stride(a.B, o->stride_b), d.osh = stride(a.H, o->stride_h), d.osn = stride(a.N, o->stride_n);
  d.gsb = stride(a.B, g->stride_b), d.gsh = stride(a.H, g->stride_h), d.gsn = stride(a.N, g->stride_n);
  d.D = Dq;
  d.rows = static_cast<long long>(a.B) * a.H * a.N;
  d.H = a.H;
  d.N = a.N;
  const long long per = 8 * (32 / (D / 8)) * kDotRows, blocks = (d.rows + per - 1) / per;
  const long long kv_items = static_cast<long long>(a.B) * a.Hkv * (static_cast<long long>(a.tiles) * a.parts + static_cast<long long>(a.sink_tiles) * a.chunks);
  const long long q_items = static_cast<long long>(a.B) * a.H * a.tiles;
  const long long sink_elems = static_cast<long long>(a.B) * a.Hkv * a.part_tiles * 2 * kTile * (D / 4);
  if (blocks > 0x7fffffffLL || kv_items > 0x7fffffffLL || q_items > 0x7fffffffLL || sink_elems / 256 > 0x7ffffff0LL) return BSA_ERR_UNSUPPORTED;
  dot_kernel<D><<<static_cast<unsigned>(blocks), 256, 0, s>>>(d);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;

  Args kv = a;
  const bsa_view* outs[2] = {dv, dk};
  for (int w = 0; w < 2; ++w) {
    kv.out[w] = static_cast<__nv_bfloat16*>(const_cast<void*>(outs[w]->data));
    kv.sb[w] = stride(a.B, outs[w]->stride_b);
    kv.sh[w] = stride(a.Hkv, outs[w]->stride_h);
    kv.sn[w] = stride(a.N, outs[w]->stride_n);
  }
  auto wide = [](const void* p, long long x, long long y, long long z) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ((x | y | z) & 15) == 0;
  };
  for (int w = 0; w < 2; ++w) kv.wide[w] = wide(kv.out[w], kv.sb[w], kv.sh[w], kv.sn[w]);
  kv.items = static_cast<unsigned>(kv_items);
  Args qa = a;
  qa.out[0] = static_cast<__nv_bfloat16*>(const_cast<void*>(dq->data));
  qa.sb[0] = stride(a.B, dq->stride_b);
  qa.sh[0] = stride(a.H, dq->stride_h);
  qa.sn[0] = stride(a.N, dq->stride_n);
  qa.wide[0] = wide(qa.out[0], qa.sb[0], qa.sh[0], qa.sn[0]);
  qa.items = static_cast<unsigned>(q_items);
  // One run of query tiles for each SM: shorter ones balance no better (537, 543 and
  // 544 us for one, two and three at 32 heads x 8192 x 128, window 1024) and pay for
  // more beginnings.
  const long long sms = sm_count(), runs = q_items < sms ? q_items : sms;
  if (kv_items + runs > 0x7fffffffLL) return BSA_ERR_UNSUPPORTED;
  kernel<<<static_cast<unsigned>(kv_items + runs), kThreads, smem, s>>>(mq, mk, mv, mo, kv, qa);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  if (a.part_tiles > 0) {
    sum_kernel<D><<<static_cast<unsigned>((sink_elems + 255) / 256), 256, 0, s>>>(kv);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  }
  return BSA_OK;
}

}  // namespace wbwd

int take_status(const void* symbol, uint32_t* status, int clear);
int window_backward_status(uint32_t* status, int clear) {
  return take_status(&wbwd::g_wbwd_status, status, clear);
}
}  // namespace bsa

extern "C" size_t bsa_window_backward_workspace_bytes(int B, int H, int Hkv, int N, int d, int window, int sinks) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || N < 1 || (d != 64 && d != 128) || window < 1 || sinks < 0) return 0;
  const auto p = bsa::wbwd::make_plan(B, H, Hkv, N, d, window, sinks);
  return p.bytes();
}

extern "C" int bsa_window_backward(const bsa_view* q, const bsa_view* k, const bsa_view* v, const bsa_view* o,
                                   const bsa_view* dO, const float* LSE, const int32_t* lens, int B, int H, int Hkv,
                                   int N, int d, int window, int sinks, float scale, const bsa_view* dq,
                                   const bsa_view* dk, const bsa_view* dv, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  using namespace bsa::wbwd;
  if (B < 1 || H < 1 || Hkv < 1 || N < 1 || d < 1 || H % Hkv != 0 || window < 1 || sinks < 0 ||
      !std::isfinite(scale) || !LSE || (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0 || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0)
    return BSA_ERR_INVALID_ARG;
  if (!view_ok(q, B, H, N, d) || !view_ok(k, B, Hkv, N, d) || !view_ok(v, B, Hkv, N, d) || !view_ok(o, B, H, N, d) ||
      !view_ok(dO, B, H, N, d) || !view_ok(dq, B, H, N, d) || !view_ok(dk, B, Hkv, N, d) || !view_ok(dv, B, Hkv, N, d))
    return BSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (N > (1 << 30)) return BSA_ERR_UNSUPPORTED;
  const Plan p = make_plan(B, H, Hkv, N, d, window, sinks);
  if (workspace_bytes < p.bytes()) return BSA_ERR_BUFFER_TOO_SMALL;
  if (rows_overlap(dq, B, H, N, d) || rows_overlap(dk, B, Hkv, N, d) || rows_overlap(dv, B, Hkv, N, d))
    return BSA_ERR_INVALID_ARG;
  Args a = {};
  a.lens = lens;
  a.LSE = LSE;
  a.Dq = static_cast<float*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.d_bytes);
  a.far_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.d_bytes + p.part_bytes);
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.N = N;
  a.tiles = p.tiles;
  a.window = window < N ? window : N;
  a.sinks = sinks < N ? sinks : N;
  // dQ and dK are 0 where each query sees one key, not what is left of dP - D
  a.alone = window == 1 && sinks == 0;
  a.sink_tiles = p.sink_tiles;
  a.chunks = p.chunks;
  a.chunk_tiles = p.chunk_tiles;
  a.parts = p.parts;
  a.part_tiles = p.part_tiles;
  a.scale = scale;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* D = static_cast<float*>(workspace);
  return d == 64 ? launch<64>(q, k, v, o, dO, a, D, dq, dk, dv, s) : launch<128>(q, k, v, o, dO, a, D, dq, dk, dv, s);
}

// bsa_window_fwd.cu -- attention with a sliding window and first tokens that stay
// visible (sinks): the forward.
//
// Query q of a sequence sees the keys k <= q with k > q - window or k < sinks:
//   O_q = sum_k softmax_k(scale q.k) v_k,   LSE_q = ln sum_k exp(scale q.k).
// H query heads share Hkv key/value heads (G = H / Hkv each).
//
// The work is 4 d flops a visible pair against 4 d bytes a row, so it is bound
// by the tensor cores (and, next to them, by the exponentials: 128 x 128 of a
// tile take 1024 cycles of the SM's 16 a clock, as long as its two products).
//
// One persistent CTA per SM walks items.  An item is two tiles of 128 queries
// ("slots") that see the same keys: the same rows of two heads of a group, or
// two neighbouring tiles of a head where G is odd.  They share every key and
// value tile that TMA brings in, which halves the shared-memory fill and lets
// the tensor core work for one slot while the other's softmax runs:
//   warps 0-7, 8-15  softmax of slot 0, 1: two threads per query row; they store O
//                    too, inside the next item's first step
//   warp 16          tcgen05.mma issuer: the warp walks, one lane issues
//   warp 17          TMA producer
// S = Q K^T lands in TMEM (128 columns a slot); the softmax writes P over it as
// bf16 and O += P V takes P from there.  A slot's next S is issued behind its
// P V, so the order of issue protects P.  TMEM: 2 x 128 columns of S, 2 x d of O.
//
// The walk is the window's tiles, then the sink tiles.  Only tiles that cross the
// diagonal, the window's lower edge or the sequence's end pay for masks, and a
// sink tile of up to 32 visible keys is taken with 32 columns instead of 128.
//
// Softmax: maxima on raw scores, lazy rescale of O (only when the maximum grows by
// more than 2^20), 2^x with the scale folded in.  P is rounded to bf16 (2^-8 at most, like the
// operands it meets); maxima, sums and O are fp32.
//
// Measured, 32 heads over 8, 32768 x 128, window 1024, 4 sinks: 0.71 ms, 760
// TFLOP/s of visible pairs.  Two 128 x 128 tiles with their softmax take 1.93 us on
// an SM (1.58 with the softmax left out), so the hand-over between products and
// exponentials is what bounds it.  One thread per row, with 128 scores, took
// 1.05 ms (spills), with 64 at a time 0.88; two threads a row and products whose
// operands stay in uniform registers 0.81; the next item's first S issued early, sinks
// last and few raises the rest.
//
// Every wait is bounded.
#include "bsa_window.cuh"

namespace bsa {
namespace wfwd {

using namespace bsa::win;

constexpr int kSlots = 2;
constexpr int kSoftWarps = 16;                 // 8 per slot: two per TMEM lane quadrant
constexpr int kMmaWarp = 16, kLoadWarp = 17;
constexpr int kThreads = 18 * 32;
// Log2 units.  P is a floating-point number in every place that holds it, so it may
// be as large as 2^20 without losing anything (sums stay below 2^20 N); what a raise
// costs is a round trip of O.
constexpr float kRescale = 20.f;

__device__ unsigned int g_wfwd_status;

template <int D>
struct Cfg {
  static constexpr int TILE = kTile * D * 2;
  static constexpr int ATOMS = D / 64;
  static constexpr int STAGES = D == 128 ? 5 : 8;     // tiles of K or V in flight
  static constexpr int TMEM_O = 256;                  // slot s: S at 128 s, O at 256 + s D
  static constexpr int TMEM_COLS = 512;
  static constexpr int OFF_KV = kSlots * TILE;
  static constexpr int OFF_CTL = OFF_KV + STAGES * TILE;
};

struct Ctl {
  uint64_t q_full[kSlots], q_empty[kSlots];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[kSlots], p_full[kSlots], p_half[kSlots];
  uint64_t o_full[kSlots], o_free[kSlots];
  uint64_t fix, final_bar;
  uint32_t tmem_base;
  volatile int abort;
  float row[kSlots][2][kTile];  // exchange between the two threads of a row: maxima, sums
};

struct Args {
  const int32_t* lens;
  __nv_bfloat16* O;
  long long o_sb, o_sh, o_sn;
  float* LSE;
  int B, H, G, N;
  unsigned Hkv;
  unsigned pairs;     // items per tile row of a cached head (G even: G / 2; else G)
  unsigned rows;      // tile rows: q tiles (G even) or pairs of them
  int by_head;        // the two slots are two heads
  int rows_first;     // items go through all heads of a tile row before the next row
  int wide;           // O's rows are 32-byte aligned
  int window, sinks;
  unsigned items;
  float scale_log2;
};

struct Item {
  int b, hk, len;
  int h0, dh, q00, dq;  // slot 0's head and first query, and how far slot 1's are on
  int near, first, steps;  // the window's tiles, then the sinks' (few keys: a low first maximum)
  __device__ __forceinline__ int h(int s) const { return h0 + s * dh; }
  __device__ __forceinline__ int q0(int s) const { return q00 + s * dq; }
  __device__ __forceinline__ int key0(int j) const {
    return (j < near ? first + j : j - near) * kTile;
  }
};

// Items run from the last tile row, which sees the most keys, to the first.
__device__ __forceinline__ Item item_of(const Args& a, unsigned i) {
  Item it;
  unsigned r = i / a.pairs;
  const int p = static_cast<int>(i - r * a.pairs);
  const unsigned by = a.rows_first ? a.Hkv * a.B : a.rows;
  i = r / by;
  r -= i * by;
  const int row = static_cast<int>(a.rows - 1 - (a.rows_first ? i : r));
  if (a.rows_first) i = r;
  it.b = static_cast<int>(i / a.Hkv);
  it.hk = static_cast<int>(i - it.b * a.Hkv);
  it.h0 = it.hk * a.G + (a.by_head ? 2 * p : p);
  it.dh = a.by_head ? 1 : 0;
  it.q00 = row * (a.by_head ? kTile : 2 * kTile);
  it.dq = a.by_head ? 0 : kTile;
  it.len = length_of(a.lens, it.b, a.N, &g_wfwd_status);
  const int top = min(it.q0(1) + kTile, it.len) - 1;  // last query with keys
  const int lo = max(0, it.q00 - a.window + 1);
  it.first = lo / kTile;
  it.near = top / kTile - it.first + 1;
  it.steps = it.q00 < it.len ? it.near + min((min(a.sinks, it.len) + kTile - 1) / kTile, it.first) : 0;
  return it;
}

// A block's next item.  Rows first, a wave of the grid takes them in turn and the next
// one backward, so that who had the longest of one wave has the shortest of the next.
__device__ __forceinline__ unsigned after(const Args& a, unsigned i) {
  const unsigned n = gridDim.x;
  if (!a.rows_first) return i + n;
  const unsigned w = i / n;
  return (w + 1) * n + (n - 1 - (i - w * n));
}

// The next item from i on that has steps; false: none.
__device__ __forceinline__ bool seek(const Args& a, unsigned& i, Item& it) {
  for (; i < a.items; i = after(a, i)) {
    it = item_of(a, i);
    if (it.steps > 0) return true;
  }
  return false;
}

// Columns a step takes: 32 where a sink tile outside the window shows no more.
__device__ __forceinline__ bool narrow_step(const Args& a, const Item& it, int j) {
  return j >= it.near && a.sinks - (j - it.near) * kTile <= 32;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctl* ctl) {
  const bool ok = wait_bounded(bar, parity, &ctl->abort, &g_wfwd_status);
  return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ producer
template <int D>
__device__ void load_role(const CUtensorMap* mq, const CUtensorMap* mk, const CUtensorMap* mv,
                          const Args& a, unsigned char* smem, Ctl* ctl) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t n = 0, items = 0, fixes = 0;
  bool ok = true;
  for (unsigned i = blockIdx.x; i < a.items && ok; i = after(a, i)) {
    const Item it = item_of(a, i);
    if (it.steps == 0) continue;
    for (int s = 0; s < kSlots && ok; ++s) {
      if (items > 0) ok = warp_wait(&ctl->q_empty[s], (items - 1) & 1, ctl);
      if (ok && lane == 0) {
        mbar_arrive_expect_tx(&ctl->q_full[s], C::TILE);
        for (int c = 0; c < C::ATOMS; ++c)
          tma_load_4d(smem + s * C::TILE + c * kAtom, mq, &ctl->q_full[s], 64 * c, it.q0(s), it.h(s), it.b);
      }
    }
    ++items;
    for (int j = 0; j < it.steps && ok; ++j) {
      const int k0 = it.key0(j);
      for (int w = 0; w < 2 && ok; ++w) {
        const int st = n % C::STAGES;
        if (n >= C::STAGES) ok = warp_wait(&ctl->kv_empty[st], (n / C::STAGES - 1) & 1, ctl);
        if (!ok) break;
        unsigned char* dst = smem + C::OFF_KV + st * C::TILE;
        // Rows past the sequence's end may hold anything; their weight is 0, but
        // 0 times a NaN is not: they are cleared before the value tile is used.
        const bool fix = w == 1 && k0 + kTile > it.len && it.len < a.N;
        uint64_t* bar = fix ? &ctl->fix : &ctl->kv_full[st];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, C::TILE);
          for (int c = 0; c < C::ATOMS; ++c)
            tma_load_4d(dst + c * kAtom, w == 0 ? mk : mv, bar, 64 * c, k0, it.hk, it.b);
        }
        if (fix) {
          ok = warp_wait(&ctl->fix, fixes & 1, ctl);
          ++fixes;
          if (ok) {
            for (int e = lane; e < (k0 + kTile - it.len) * 8 * C::ATOMS; e += 32) {
              const int r = it.len - k0 + e / (8 * C::ATOMS), c = e % (8 * C::ATOMS);
              *reinterpret_cast<uint4*>(dst + (c >> 3) * kAtom + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->kv_full[st]);
        }
        ++n;
      }
    }
  }
  // Copies in flight must land before the block's shared memory goes away.
  if (lane == 0) {
    for (int s = 0; s < kSlots; ++s)
      if (items > 0) wait_drain(&ctl->q_full[s], (items - 1) & 1, &g_wfwd_status);
    for (uint32_t st = 0; st < static_cast<uint32_t>(C::STAGES); ++st)
      if (n > st) wait_drain(&ctl->kv_full[st], ((n - 1 - st) / C::STAGES) & 1, &g_wfwd_status);
    if (fixes > 0) wait_drain(&ctl->fix, (fixes - 1) & 1, &g_wfwd_status);
  }
}

// ---------------------------------------------------------------- MMA issuer
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tmem, uint32_t sbase, int s, int st, bool narrow) {
  using C = Cfg<D>;
  const uint64_t ad = sdesc_sw128(sbase + s * C::TILE, 16, 1024);
  const uint64_t bd = sdesc_sw128(sbase + C::OFF_KV + st * C::TILE, 16, 1024);
  const uint32_t idesc = narrow ? idesc_bf16_f32(128, 32, false, false) : idesc_bf16_f32(128, 128, false, false);
  umma_qk_chain<D / 16>(tmem + s * 128, static_cast<uint32_t>(ad), static_cast<uint32_t>(ad >> 32),
                        static_cast<uint32_t>(bd), static_cast<uint32_t>(bd >> 32), idesc);
}

// O += P V.  P comes in two parts, the first half of each thread's columns and the
// second (narrow steps: one part of 32), so that the first product runs beside the
// second part's exponentials.
template <int D, int PART, bool NARROW>
__device__ __forceinline__ void issue_pv(uint32_t tmem, uint32_t sbase, int s, int st, bool add) {
  using C = Cfg<D>;
  constexpr uint32_t kIdesc = idesc_bf16_f32(128, D, false, true);
  const uint64_t bd = sdesc_sw128(sbase + C::OFF_KV + st * C::TILE, kAtom, 1024);
  const uint32_t lo = static_cast<uint32_t>(bd), hi = static_cast<uint32_t>(bd >> 32);
  const uint32_t t_o = tmem + C::TMEM_O + s * D, t_p = tmem + s * 128;
  umma_pv_slices2(t_o, t_p + 16 * PART, lo + 256 * PART, hi, kIdesc, add ? 1u : 0u);
  if (!NARROW) umma_pv_slices2(t_o, t_p + 64 + 16 * PART, lo + 512 + 256 * PART, hi, kIdesc, 1u);
}

// The MMA warp's counters: tiles consumed, items begun, steps taken.
struct Issued {
  uint32_t tiles, items, steps;
};

// One step of both slots: O += P V, and behind it the slot's next S, of this item
// (LAST false) or of the next one (LAST; if it exists).  q_done: that S is the last
// to read its Q.
template <int D, bool LAST>
__device__ __forceinline__ bool mma_step(uint32_t tmem, uint32_t sbase, Ctl* ctl, bool lead, Issued& n, bool first,
                                         bool narrow, bool more, bool next_narrow, bool q_done) {
  using C = Cfg<D>;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, ctl); };
  const int vst = n.tiles % C::STAGES;
  const uint32_t vpar = (n.tiles / C::STAGES) & 1;
  ++n.tiles;
  const int kst = n.tiles % C::STAGES;
  const uint32_t kpar = (n.tiles / C::STAGES) & 1;
  if (!LAST || more) ++n.tiles;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if (s == 0) {
      if (!wait(&ctl->kv_full[vst], vpar)) return false;
      if ((!LAST || more) && !wait(&ctl->kv_full[kst], kpar)) return false;
    }
    if (first && n.items > 0 && !wait(&ctl->o_free[s], (n.items - 1) & 1)) return false;
    if (!narrow) {
      if (!wait(&ctl->p_half[s], n.steps & 1)) return false;
      tc_fence_after();
      if (lead) issue_pv<D, 0, false>(tmem, sbase, s, vst, !first);
    }
    if (!wait(&ctl->p_full[s], n.steps & 1)) return false;
    tc_fence_after();
    if (lead) {
      if (narrow)
        issue_pv<D, 0, true>(tmem, sbase, s, vst, !first);
      else
        issue_pv<D, 1, false>(tmem, sbase, s, vst, true);
    }
    if (LAST) {
      if (lead) umma_commit(&ctl->o_full[s]);
      if (more && !wait(&ctl->q_full[s], (n.items + 1) & 1)) return false;
      tc_fence_after();
    }
    if (lead) {
      if (!LAST || more) {
        issue_qk<D>(tmem, sbase, s, kst, next_narrow);
        umma_commit(&ctl->s_full[s]);
        if (q_done) umma_commit(&ctl->q_empty[s]);
      }
      if (s == 1) {
        umma_commit(&ctl->kv_empty[vst]);
        if (!LAST || more) umma_commit(&ctl->kv_empty[kst]);
      }
    }
  }
  ++n.steps;
  return true;
}

// The whole warp walks the steps, so that what the products need stays in uniform
// registers; one lane issues them.  A slot's next S follows its P V at once, the
// next item's first S too, so the slots stay half a step apart.
template <int D>
__device__ void mma_role(const Args& a, unsigned char* smem, Ctl* ctl, uint32_t tmem) {
  const uint32_t sbase = smem_u32(smem);
  const bool lead = elect_one();
  Issued n = {0, 0, 0};
  unsigned i = blockIdx.x;
  Item it;
  bool have = seek(a, i, it), ok = true;
  if (have) {
    ok = warp_wait(&ctl->kv_full[0], 0, ctl);
    for (int s = 0; s < kSlots && ok; ++s) {
      if (!(ok = warp_wait(&ctl->q_full[s], 0, ctl))) break;
      tc_fence_after();
      if (lead) {
        issue_qk<D>(tmem, sbase, s, 0, narrow_step(a, it, 0));
        umma_commit(&ctl->s_full[s]);
        if (it.steps == 1) umma_commit(&ctl->q_empty[s]);
      }
    }
    if (ok && lead) umma_commit(&ctl->kv_empty[0]);
    n.tiles = 1;
  }
  while (have && ok) {
    for (int j = 0; j + 1 < it.steps && ok; ++j)
      ok = mma_step<D, false>(tmem, sbase, ctl, lead, n, j == 0, narrow_step(a, it, j), true,
                              narrow_step(a, it, j + 1), j + 2 == it.steps);
    const bool one = it.steps == 1, narrow = narrow_step(a, it, it.steps - 1);
    i = after(a, i);
    have = seek(a, i, it);
    ok = ok && mma_step<D, true>(tmem, sbase, ctl, lead, n, one, narrow, have, have && narrow_step(a, it, 0),
                                 have && it.steps == 1);
    ++n.items;
  }
  // Every MMA issued must complete before TMEM is released.
  if (lead) {
    umma_commit(&ctl->final_bar);
    wait_drain(&ctl->final_bar, 0, &g_wfwd_status);
  }
  __syncwarp();
}

// ------------------------------------------------------------------- softmax
// Two threads share a query row, 64 of a step's 128 scores each.  They agree on
// the running maximum at a barrier of the slot's 256 threads that also votes
// whether any of them wants it raised: mostly none does, and the barrier is all
// that the agreement costs.  A thread's 64 scores pass through 32 registers: the
// right half for its maximum, the left half for its maximum and its P (which
// lands on scores already taken), then the right half again for its P.  That keeps
// a thread under 96 registers, and so four softmax warps on a scheduler.
__device__ __forceinline__ bool slot_vote(int s, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(mine ? 1u : 0u), "r"(s + 1)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void slot_sync(int s) {
  asm volatile("barrier.cta.sync.aligned %0, 256;" ::"r"(s + 1) : "memory");
}

// Which of 32 columns from c0 on a row sees: those up to hi, from lo on or below
// sink.
__device__ __forceinline__ uint32_t upto(int n) {  // the n lowest bits
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
}
struct Seen {
  int hi, lo, sink;
  __device__ __forceinline__ uint32_t columns(int c0) const {
    return upto(hi + 1 - c0) & (~upto(lo - c0) | upto(sink - c0));
  }
};

// 32 scores of a row from column c0 on, for a positive scale.  The sign is
// compiled in, and a step without hidden scores branches around their masks.
template <bool NEG>
__device__ __forceinline__ void load_scores(float (&x)[32], uint32_t t_s, int c0, bool full, const Seen& seen) {
  tmem_ld32f_wait(t_s + c0, x);
  if constexpr (NEG) {
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = -x[c];
  }
  if (!full) {
    const uint32_t w = seen.columns(c0);
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!(w & (1u << c))) x[c] = -INFINITY;
  }
}

__device__ __forceinline__ float max_of(const float (&x)[32]) {
  float m0 = x[0], m1 = x[1], m2 = x[2], m3 = x[3];
#pragma unroll
  for (int c = 4; c < 28; c += 8) {
    m0 = max3f(m0, x[c], x[c + 1]);
    m1 = max3f(m1, x[c + 2], x[c + 3]);
    m2 = max3f(m2, x[c + 4], x[c + 5]);
    m3 = max3f(m3, x[c + 6], x[c + 7]);
  }
  m0 = max3f(m0, x[28], x[29]);
  m1 = max3f(m1, x[30], x[31]);
  return max3f(fmaxf(m0, m1), m2, m3);
}

// The row's running maximum takes this thread's hm and its partner's in, with O
// and the sums brought to it, where it grows by more than the threshold.
template <int D>
__device__ __forceinline__ void raise_max(int s, float hm, float* mine, const float* other, uint32_t t_o,
                                          bool have_o, float& m, float& l) {
  if (!slot_vote(s, hm > m + kRescale)) return;
  *mine = hm;
  slot_sync(s);
  hm = fmaxf(hm, *other);
  float f = 1.f;
  if (hm > m + kRescale) {
    f = m == -INFINITY ? 1.f : ex2_approx(m - hm);
    m = hm;
  }
  l *= f;
  // this step's S is ready, so the P V of every step before has completed
  if (have_o && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
    for (int c0 = 0; c0 < D / 2; c0 += 8) {
      uint32_t w[8];  // few registers: this is rare, and the scores are live across it
      tmem_ld8_wait(t_o + c0, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = __float_as_uint(__uint_as_float(w[c]) * f);
      tmem_st8_wait(t_o + c0, w);
    }
  }
  slot_sync(s);  // the exchange may be written again
}

// P of 32 scores, to 16 columns from t_p on; their sum.
__device__ __forceinline__ float exponentials(const float (&x)[32], uint32_t t_p, float sl2, float nm) {
  float sa = 0.f, sb = 0.f, sc = 0.f, sd = 0.f;
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    float p0 = x[c], p1 = x[c + 1], p2 = x[c + 2], p3 = x[c + 3];
    fma2(p0, p1, sl2, nm);
    fma2(p2, p3, sl2, nm);
    p0 = ex2_approx(p0);
    p1 = ex2_approx(p1);
    p2 = ex2_approx(p2);
    p3 = ex2_approx(p3);
    acc2(sa, sb, p0, p1);
    acc2(sc, sd, p2, p3);
    pk[c / 2] = pack_bf16x2(p0, p1);
    pk[c / 2 + 1] = pack_bf16x2(p2, p3);
  }
  tmem_st16(t_p, pk);
  return (sa + sb) + (sc + sd);
}

// What is left to do for a thread's half row once its item's last step is taken.
struct Rest {
  __nv_bfloat16* out;
  float* lse;
  float m, l;
  bool pending, live, write;   // live: a row of the sequence; write: a row of the tensor
};

// A half row of O / sum, 32 bytes at a time where the rows are aligned so.
template <int D>
__device__ __forceinline__ void store_half_row(const Rest& r, float inv, uint32_t t_o, bool have_o, bool wide) {
#pragma unroll 1
  for (int c0 = 0; c0 < D / 2; c0 += 16) {
    uint32_t w[16], x[8];
    if (have_o) {
      tmem_ld16(t_o + c0, w);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 16; ++c) asm volatile("" : "+r"(w[c]));  // no use above the wait
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
      x[c] = have_o && r.live ? pack_bf16x2(__uint_as_float(w[2 * c]) * inv, __uint_as_float(w[2 * c + 1]) * inv) : 0u;
    if (!r.write) continue;
    if (wide) {
      store_256(r.out + c0, x);
    } else {
      *reinterpret_cast<uint4*>(r.out + c0) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(r.out + c0 + 8) = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
}

// The barriers that are left of a walk, from step j of item i on, for a warp that gave
// up a wait: the slot's other warps count on it there, and barriers have no limit.
// Its vote is yes, so all take the barriers of a raise.
__device__ __noinline__ void keep_step(int s, const Args& a, unsigned i, int j, bool pending) {
  for (; i < a.items; i = after(a, i), j = 0) {
    const Item it = item_of(a, i);
    for (; j < it.steps; ++j) {
      slot_vote(s, true);
      slot_sync(s);
      slot_sync(s);
      if (pending) slot_sync(s);  // where the others finish the item before
      pending = false;
    }
    pending = pending || it.steps > 0;
  }
  if (pending) slot_sync(s);
}

template <int D, bool NEG>
__device__ void softmax_role(int s, const Args& a, Ctl* ctl, uint32_t tmem) {
  using C = Cfg<D>;
  const int warp = (threadIdx.x >> 5) & 7, wq = warp & 3, half = warp >> 2, lane = threadIdx.x & 31;
  const int row = wq * 32 + lane;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const uint32_t t_s = t_lane + s * 128, t_o = t_lane + C::TMEM_O + s * D + half * (D / 2);
  const float sl2 = fabsf(a.scale_log2);
  float* mine = &ctl->row[s][half][row];
  const float* other = &ctl->row[s][half ^ 1][row];
  uint32_t seen = 0, items = 0;
  Rest rest;
  rest.pending = false;
  // O of the item before: after its last P V, and before the next item's first.
  // The exchange is free again after the next step's vote, before which nothing
  // writes it.
  auto finish = [&]() {
    *mine = rest.l;
    slot_sync(s);
    // added in one order by both, so that they divide by the same sum
    const float l = half == 0 ? rest.l + *other : *other + rest.l;
    if (!warp_wait(&ctl->o_full[s], (items - 1) & 1, ctl)) return false;
    tc_fence_after();
    store_half_row<D>(rest, 1.f / l, t_o, true, a.wide);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl->o_free[s]);
    if (half == 0 && rest.write) *rest.lse = rest.live ? (rest.m + log2f(l)) * kLn2 : -INFINITY;
    rest.pending = false;
    return true;
  };
  for (unsigned i = blockIdx.x; i < a.items; i = after(a, i)) {
    const Item it = item_of(a, i);
    const int q0 = it.q0(s), q = q0 + row;
    float m = -INFINITY, l = 0.f;  // maximum (log2 units) of the row, sum of this thread's columns
    for (int j = 0; j < it.steps; ++j) {
      const int k0 = it.key0(j);
      // all keys of the tile are visible to all of its rows
      const bool full = k0 + kTile - 1 <= q0 && (k0 > q0 + kTile - 1 - a.window || k0 + kTile <= a.sinks);
      if (!warp_wait(&ctl->s_full[s], seen & 1, ctl)) return keep_step(s, a, i, j, rest.pending);
      ++seen;
      tc_fence_after();
      const Seen vis = {q - k0, q - a.window + 1 - k0, a.sinks - k0};
      float x[32];
      if (narrow_step(a, it, j)) {
        float hm = -INFINITY;
        if (half == 0) {
          load_scores<NEG>(x, t_s, 0, false, vis);
          hm = max_of(x) * sl2;
        }
        raise_max<D>(s, hm, mine, other, t_o, j > 0, m, l);
        if (half == 0) l += exponentials(x, t_s, sl2, m == -INFINITY ? 0.f : -m);
        if (lane == 0) mbar_arrive(&ctl->p_half[s]);
      } else {
        const int c0 = 64 * half;
        load_scores<NEG>(x, t_s, c0 + 32, full, vis);
        float hm = max_of(x);
        load_scores<NEG>(x, t_s, c0, full, vis);
        hm = fmaxf(hm, max_of(x)) * sl2;
        raise_max<D>(s, hm, mine, other, t_o, j > 0, m, l);
        const float nm = m == -INFINITY ? 0.f : -m;
        l += exponentials(x, t_s + c0, sl2, nm);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->p_half[s]);
        load_scores<NEG>(x, t_s, c0 + 32, full, vis);
        l += exponentials(x, t_s + c0 + 16, sl2, nm);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[s]);
      // The last item's O is stored here: its last P V ran beside this softmax, and
      // this step's P V is all that waits for it.
      if (rest.pending && !finish()) return keep_step(s, a, i, j + 1, false);
    }

    Rest now;
    now.out = a.O + it.b * a.o_sb + it.h(s) * a.o_sh + static_cast<long long>(q) * a.o_sn + half * (D / 2);
    now.lse = a.LSE + (static_cast<long long>(it.b) * a.H + it.h(s)) * a.N + q;
    now.m = m;
    now.l = l;
    now.live = q < it.len;
    now.write = q < a.N;
    now.pending = it.steps > 0;
    if (now.pending) {
      rest = now;  // the one before was stored in this item's first step
      ++items;
    } else {  // no tile of it was computed: an earlier item may still be pending
      store_half_row<D>(now, 0.f, t_o, false, a.wide);
      if (half == 0 && now.write) *now.lse = -INFINITY;
    }
  }
  if (rest.pending) finish();
}

template <int D, bool NEG>
__global__ void __launch_bounds__(kThreads, 1)
    window_forward_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const __grid_constant__ Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem[];  // swizzle atoms need 1024 bytes
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_wfwd_status, BSA_STATUS_INTERNAL);
    return;
  }
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + C::OFF_CTL);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ctl->q_full[s], 1);
      mbar_init(&ctl->q_empty[s], 1);
      mbar_init(&ctl->s_full[s], 1);
      mbar_init(&ctl->p_full[s], 8);
      mbar_init(&ctl->p_half[s], 8);
      mbar_init(&ctl->o_full[s], 1);
      mbar_init(&ctl->o_free[s], 8);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&ctl->kv_full[i], 1);
      mbar_init(&ctl->kv_empty[i], 1);
    }
    mbar_init(&ctl->fix, 1);
    mbar_init(&ctl->final_bar, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  if (warp < kSoftWarps) {
    softmax_role<D, NEG>(warp >> 3, a, ctl, tmem);
  } else if (warp == kMmaWarp) {
    mma_role<D>(a, smem, ctl, __shfl_sync(0xffffffffu, tmem, 0));
  } else if (warp == kLoadWarp) {
    load_role<D>(&mq, &mk, &mv, a, smem, ctl);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D>
int launch(const bsa_view* q, const bsa_view* k, const bsa_view* v, const Args& a, cudaStream_t s) {
  using C = Cfg<D>;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q, a.B, a.H, a.N, D) || !make_map(&mk, k, a.B, a.Hkv, a.N, D) ||
      !make_map(&mv, v, a.B, a.Hkv, a.N, D))
    return BSA_ERR_CUDA;
  const int smem = C::OFF_CTL + static_cast<int>(sizeof(Ctl));
  static_assert(C::OFF_CTL + sizeof(Ctl) <= 232448, "227 KB of shared memory");
  const auto kernel = a.scale_log2 < 0.f ? window_forward_kernel<D, true> : window_forward_kernel<D, false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return BSA_ERR_CUDA;
  const unsigned sms = static_cast<unsigned>(sm_count());
  kernel<<<a.items < sms ? a.items : sms, kThreads, smem, s>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // namespace wfwd

int take_status(const void* symbol, uint32_t* status, int clear);
int window_forward_status(uint32_t* status, int clear) {
  return take_status(&wfwd::g_wfwd_status, status, clear);
}
}  // namespace bsa

extern "C" int bsa_window_forward(const bsa_view* q, const bsa_view* k, const bsa_view* v,
                                  const int32_t* lens, int B, int H, int Hkv, int N, int d, int window,
                                  int sinks, float scale, const bsa_view* o, float* LSE, void* stream) {
  using namespace bsa::wfwd;
  if (B < 1 || H < 1 || Hkv < 1 || N < 1 || d < 1 || H % Hkv != 0 || window < 1 || sinks < 0 ||
      !std::isfinite(scale) || !LSE || (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0)
    return BSA_ERR_INVALID_ARG;
  if (!view_ok(q, B, H, N, d) || !view_ok(k, B, Hkv, N, d) || !view_ok(v, B, Hkv, N, d) || !view_ok(o, B, H, N, d))
    return BSA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (N > (1 << 30)) return BSA_ERR_UNSUPPORTED;
  if (rows_overlap(o, B, H, N, d)) return BSA_ERR_INVALID_ARG;
  Args a = {};
  a.lens = lens;
  a.O = static_cast<__nv_bfloat16*>(const_cast<void*>(o->data));
  a.o_sb = B > 1 ? o->stride_b : 0;
  a.o_sh = H > 1 ? o->stride_h : 0;
  a.o_sn = N > 1 ? o->stride_n : 0;
  a.wide = (reinterpret_cast<uintptr_t>(o->data) & 31u) == 0 && ((a.o_sb | a.o_sh | a.o_sn) & 15) == 0;
  a.LSE = LSE;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.N = N;
  const int tiles = (N + kTile - 1) / kTile;
  a.by_head = a.G % 2 == 0;
  a.pairs = a.by_head ? a.G / 2 : a.G;
  a.rows = a.by_head ? tiles : (tiles + 1) / 2;
  a.window = window < N ? window : N;
  // Rows first balances the blocks where rows differ (the longest items begin first), as
  // long as what a row of all heads sees stays in half of L2 until the next row.
  a.rows_first = static_cast<long long>(B) * Hkv * (a.window + 2 * kTile) * d * 4 <= (64LL << 20);
  a.sinks = sinks < N ? sinks : N;
  const long long items = static_cast<long long>(B) * Hkv * a.rows * a.pairs;
  if (items >= (1LL << 31)) return BSA_ERR_UNSUPPORTED;
  a.items = static_cast<unsigned>(items);
  // never 0: hidden scores are -inf times it, and must stay -inf
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (std::fabs(a.scale_log2) < 1e-30f) a.scale_log2 = 1e-30f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch<64>(q, k, v, a, s) : launch<128>(q, k, v, a, s);
}

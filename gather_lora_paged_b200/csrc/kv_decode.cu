// kv_decode.cu -- attention of each sequence's newest tokens over its KV pages,
// for few rows per kv head (decode, drafted tokens): a stream of the cache
// through the 5th-generation tensor cores, scores and output transposed.
//
// For query row i of a sequence (position p_i = kv_len - n + i) and query head
// hq reading kv head h = hq / G:
//     o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale * q_i . k_j),
//     j <= p_i and, with a window, j > p_i - window;
//     lse_i = log sum_j w_ij;  a row that sees no key gets 0 and -inf.
//
// HBM bounds this: each cached row is read once per row tile and met by few rows, so
// that instructions spent per cached byte decide.  With the keys on the MMA's M side,
//     S^T [128 keys x rows] = K . Q^T,   O^T [D x rows] += V^T . W^T,
// a tile of 128 keys goes from the pages to shared memory (16-byte cp.async, a page may hold
// one token, so rows are gathered) and from there straight to the tensor cores:
// no thread touches a cached element, and the rows only fill N, a multiple of 16.
// Items, runs, partials and their join: kv_attn.cuh.
//
// One CTA per SM, 20 warps:
//   warps 8..11 copy K and V rows into a ring of slots (K or V of a tile), 32 keys
//               each; the copies signal the slot's barrier when they land;
//   warp 13     the run's items, for all others;
//   warps 14, 15  q of the items ahead, as the N side of S^T, and the rows' positions;
//   warp 12     issues S^T of tile i + 1, then O^T of tile i;
//   warps 0..7  the softmax: a thread owns a key and half of the rows, reads its scores from TMEM
//               and writes its weights to shared memory as the N side of O^T;
//   warps 16..19  an item's end: O^T from TMEM to the output, beside the next item.
//
// Weights are exp(s - m) with m a former maximum of the row: it moves (and O^T is
// scaled) only when a score exceeds it by 2^8, which one vote per tile finds out.
//
// What the tensor cores take is split so that nothing is lost that an output could show:
// 16-bit: weights as hi + lo, two 16-bit columns of N.
// e4m3:   the codes are operands as they are (kind::f8f6f4).  q is a sum of three e4m3 values, each 2^-4 of
//         the one before and a column of its own: 12 bits, so an fp16 q is exact; the
//         largest of a q row lies in [2^7, 2^8) after a power of two, what is lost of any element is under
//         2^-26 of it.  A weight is its fp16 value, as a sum of four e4m3 values, each 2^-5 of the one before.
//         K's row scale multiplies the score, V's the weight, over a unit (a power of two) of
//         each row's own: the largest product of weight and scale that the row has met is 2^3..2^4 units where the
//         unit is set, and 2^8 at most before it moves.  So keys that a row does not see have no part in it, and
//         what is lost of a weight is under 2^-11 of it or 2^-28 of the row's largest with V's scales.
//
// Measured (three inputs in turn): 256 tokens of 32 heads (one row a kv head) over 200..2000 keys, 3.24 GB in
// fp16: 500 to 509 us, 6.4 TB/s; one token, 64 heads on 8, over 130001 keys, bf16: 91 us, 5.8 TB/s (85 in this kernel, at
// 6.2); 64 tokens, 64 heads on 8, over 1000..16000 keys in e4m3, 0.7 GB: 141 us, 5.0 TB/s: at 8 rows the
// copies' issue, the softmax and HBM take about 1370 cycles each for a tile; with 40 rows (5 tokens each: 286 us) the
// softmax takes 3700.
// The copies go at 7.0 TB/s by themselves (16-byte cp.async, four warps); TMA's row gather brings 1.9, a bulk copy
// per 1 KB 3.6.
//
// Values of V that are not finite: kv_attn.cuh.
#include <math.h>

#include "kv_attn.cuh"
#include "kv_tc.cuh"

namespace slora {
namespace {

constexpr int kNT = 640;       // threads
constexpr int kTK = kKvTile;   // keys per tile
constexpr int kMinRun = 1;     // tiles that are worth a CTA of their own
constexpr int kMeta = 8;       // tiles whose scales and masks are kept: what the ring holds, at least
constexpr int kItems = 16;     // items that are known ahead
constexpr float kNoRef = 0x1.fffffep127f;  // (negated) reference of a row that has seen no key: scores are above -2^127

// TM: rows per item.  N is a multiple of 16 rows (e4m3: three columns a row).
template <int DT, int FMT, int D, int TM>
struct Cfg {
  static constexpr bool kF8 = FMT == SLORA_KV_E4M3;
  // log2 by which scores may exceed the row's reference, and in e4m3 of the largest weight (e4m3 ends at 2^8.8)
  static constexpr float kSlack = 8.f;
  // 16-bit: log2 of the weight at a row's maximum.  fp16: weights are up to 2^13 (it ends at 2^16).  bf16: of 2^16
  // keys at 2^8 over the maximum none of V's products and sums overflows, however large V is.
  static constexpr int kLift = kF8 ? 0 : DT == SLORA_F16 ? 5 : -24;
  // e4m3: log2 of the largest weight where a unit is set
  static constexpr float kSet = 4.f;
  static constexpr int kRow = KvRow<FMT, D>::kBytes;                    // a cached row
  static constexpr int kWidth = kRow >= 128 ? 128 : kRow;               // bytes of a row in a panel
  static constexpr int kPanel = kTK * kWidth;
  static constexpr int kSlot = kTK * kRow;                              // K or V of a tile
  static constexpr int kRows16 = (TM + 15) / 16 * 16;
  static constexpr int kQRows = kF8 ? 3 * kRows16 : kRows16;            // columns of S^T
  static constexpr int kPCols = kF8 ? 4 * TM : 2 * TM;                  // columns of O^T
  static constexpr int kQ = kQRows * kRow;                              // one of two buffers
  static constexpr int kP = kPCols * (kF8 ? 1 : 2) * kTK;               // one of two buffers
  static constexpr int kSlots = kF8 ? (D == 64 ? 16 : (TM <= 16 ? 10 : 7)) : (D == 64 ? 10 : (TM <= 16 ? 6 : 5));
  static constexpr int kOffP = kSlots * kSlot;
  static constexpr int kOffQ = kOffP + 2 * kP;
  static constexpr int kOffScale = kOffQ + 2 * kQ;
  static constexpr int kScale = kF8 ? kMeta * 2 * kTK * 4 : 0;
  static constexpr int kOffCtl = kOffScale + kScale;
  static constexpr int kSCols = kQRows;                                 // TMEM: S0, S1, O's
  static constexpr int kOBufs = 2 * (kSCols + kPCols) <= 512 ? 2 : 1;   // items' O^T side by side
  static constexpr int kTmemCols = 2 * kSCols + kOBufs * kPCols;
  static constexpr int kTmem = kTmemCols <= 64 ? 64 : kTmemCols <= 128 ? 128 : kTmemCols <= 256 ? 256 : 512;
  static_assert(kSlots <= 2 * kMeta, "an entry is written again once V's slot of that tile is free");
  static_assert(kTmemCols <= 512, "TMEM");
};

template <int TM, int S>
struct Ctl {
  uint64_t kv_full[S], kv_empty[S], q_full[2], q_empty[2], item_full[kItems], item_empty[kItems], rows_full[kItems];
  uint64_t s_full[2], p_full[2], pv_done[2], o_full[2], o_empty[2], sum_full[2], tmem_full, fin;
  Item item[kItems];
  uint32_t tmem;
  int dead;                                   // a wait gave up: nobody waits any more
  uint32_t mask[kMeta][4];                    // keys of a tile that are there
  alignas(16) float qmul[kItems][(TM + 15) / 16 * 16];    // score multipliers of an item's rows
  int pos[kItems][(TM + 15) / 16 * 16];       // their positions (-1: no such row)
  float red[2][4][TM];                        // warps' maxima, of scores and (e4m3) with V's scales
  alignas(16) float ref[TM];                  // the rows' references, negated
  // e4m3: one over the units of their weights, and the reference (negated) of a score with log2 of V's scale
  alignas(16) float inv[TM];
  alignas(16) float vref[TM];
  float fac[TM], ofac[TM];                    // what a move of these scales sums and products by
  // an item's end, for the epilogue: warps' sums, references, the weights' units, and its own notes
  float sum[2][4][TM], end_ref[2][TM];
  alignas(8) float unit[2][TM];
  alignas(8) float out_fac[TM];
  uint32_t bad[4][2];                         // warps' rows that are not finite
};

__device__ __forceinline__ void st_shared8(uint32_t dst, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void ld8(uint32_t taddr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(taddr));
}
__device__ __forceinline__ void ld4(uint32_t taddr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(taddr));
}
__device__ __forceinline__ void st4(uint32_t taddr, const float* v) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(u[0]), "r"(u[1]), "r"(u[2]),
               "r"(u[3])
               : "memory");
}
__device__ __forceinline__ void st8(uint32_t taddr, const float* v) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}
// tcgen05.wait::ld, tied to the registers that the load fills
__device__ __forceinline__ void wait_ld8(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void wait_ld4(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]) : : "memory");
}
template <int N>
__device__ __forceinline__ void ld_n(uint32_t taddr, float* v) {
  if (N == 8) ld8(taddr, v);
  else ld4(taddr, v);
}
template <int N>
__device__ __forceinline__ void st_n(uint32_t taddr, const float* v) {
  if (N == 8) st8(taddr, v);
  else st4(taddr, v);
}
template <int N>
__device__ __forceinline__ void wait_ld_n(float* v) {
  if (N == 8) wait_ld8(v);
  else wait_ld4(v);
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The softmax warps' and the epilogue warps' barriers, and votes over them.
__device__ __forceinline__ void softmax_sync() { sync_of<1, 256>(); }
__device__ __forceinline__ bool softmax_any(bool p) { return any_of<2, 256>(p); }
__device__ __forceinline__ void epilogue_sync() { sync_of<3, 128>(); }
__device__ __forceinline__ bool epilogue_any(bool p) { return any_of<4, 128>(p); }
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Two weights of up to 2^8 as four e4m3 codes each, every one 2^-5 of the one before: exactly their fp16 values, the
// least ones included (all of them have been tried; three codes at 2^-4 end at 2^-17, at 2^-5 at 2^-19).
__device__ __forceinline__ void split4_weights(uint64_t w, uint32_t& p0, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  float a, b;
  unpair(w, a, b);
  asm("{\n\t.reg .b32 h, c, s;\n\t.reg .b16 k;\n\t"
      "mov.b32 s, 0x50005000;\n\t"                      // 32, 32
      "cvt.rn.f16x2.f32 h, %5, %4;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 k, h;\n\tcvt.u32.u16 %0, k;\n\tcvt.rn.f16x2.e4m3x2 c, k;\n\t"
      "sub.f16x2 h, h, c;\n\tmul.f16x2 h, h, s;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 k, h;\n\tcvt.u32.u16 %1, k;\n\tcvt.rn.f16x2.e4m3x2 c, k;\n\t"
      "sub.f16x2 h, h, c;\n\tmul.f16x2 h, h, s;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 k, h;\n\tcvt.u32.u16 %2, k;\n\tcvt.rn.f16x2.e4m3x2 c, k;\n\t"
      "sub.f16x2 h, h, c;\n\tmul.f16x2 h, h, s;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 k, h;\n\tcvt.u32.u16 %3, k;\n\t}"
      : "=r"(p0), "=r"(p1), "=r"(p2), "=r"(p3) : "f"(a), "f"(b));
}
// Two values as three e4m3 codes each, every one 2^-4 of the one before.
__device__ __forceinline__ void split3(float a, float b, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
  float x, y;
  p0 = e4m3x2(a, b);
  h2x2f(e4m3x2_f16x2(p0), x, y);
  a = (a - x) * 16.f;
  b = (b - y) * 16.f;
  p1 = e4m3x2(a, b);
  h2x2f(e4m3x2_f16x2(p1), x, y);
  p2 = e4m3x2((a - x) * 16.f, (b - y) * 16.f);
}

// Byte offset of 16-byte chunk c of row j, in panels of `rows` rows of W bytes.
template <int W>
__device__ __forceinline__ uint32_t place(int rows, int j, int c) {
  if (W == 128) return (uint32_t)((c >> 3) * rows * 128 + j * 128 + (((c & 7) ^ (j & 7)) << 4));
  return (uint32_t)(j * 64 + ((c ^ ((j >> 1) & 3)) << 4));
}

template <int DT, int FMT, int D, int TM>
__global__ void __launch_bounds__(kNT, 1) k_kv_decode(const __grid_constant__ KvAttnDev A, RowClass cls) {
  using C = Cfg<DT, FMT, D, TM>;
  constexpr int S = C::kSlots, W = C::kWidth;
  constexpr bool F8 = C::kF8;
  using Control = Ctl<TM, S>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = su32(smem);
  Control* const ctl = reinterpret_cast<Control*>(smem + C::kOffCtl);
  const KvDev& P = A.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Split* const split = reinterpret_cast<Split*>(A.workspace) + blockIdx.x;
  float* const parts = reinterpret_cast<float*>(reinterpret_cast<Split*>(A.workspace) + gridDim.x);

  griddep_launch();  // the join's CTAs may take their places (they wait for this grid's end)
  if (tid == 0) split->n = 0;
  if (warp == 12) {
    for (int i = lane; i < S; i += 32) {
      bar_init(&ctl->kv_full[i], 128 + 4);
      bar_init(&ctl->kv_empty[i], 1);
    }
    if (lane < 2) {
      bar_init(&ctl->q_full[lane], 128);
      bar_init(&ctl->q_empty[lane], 1);
      bar_init(&ctl->s_full[lane], 1);
      bar_init(&ctl->p_full[lane], 256);
      bar_init(&ctl->pv_done[lane], 1);
      bar_init(&ctl->o_full[lane], 1);
      bar_init(&ctl->o_empty[lane], 128);
      bar_init(&ctl->sum_full[lane], 256);
    }
    if (lane < kItems) {
      bar_init(&ctl->item_full[lane], 1);
      bar_init(&ctl->item_empty[lane], 1);
      bar_init(&ctl->rows_full[lane], 64);
    }
    if (lane < kItems) {  // what those see who did not wait for an entry (see wait_slow)
      ctl->item[lane].flags = 4;
      ctl->item[lane].n_tiles = 0;
    }
    if (lane == 0) {
      bar_init(&ctl->tmem_full, 32);
      bar_init(&ctl->fin, 1);
      ctl->dead = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();  // the barriers are there
  auto wait = [&](uint64_t* b, uint32_t parity) { wait_for(b, parity, &ctl->dead, P.err); };
  // Nobody walks on through items that may never come once a wait has given up.
  auto over = [&]() -> bool { return *reinterpret_cast<volatile int*>(&ctl->dead); };
  auto tmem_at = [&]() -> uint32_t {  // for those who do not allocate it
    wait(&ctl->tmem_full, 0);
    return ctl->tmem;
  };
  // An item's entry.  It is written again for item it + 16, once the epilogue is through with this
  // one; all others have read it by then.
  auto item_at = [&](uint32_t it) -> const Item& {
    wait(&ctl->item_full[it % kItems], (it / kItems) & 1);
    return ctl->item[it % kItems];
  };

  // 96 registers at launch: the softmax warps, which hold scores and sums of their rows,
  // take from the others (128 + 128 + 72 + 80 + 72 = 5 * 96)
  if (warp >= 8 && warp < 16) {
    if (warp < 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }
    if (warp < 12) {
      // -------------------------------------------------------------- loaders
      constexpr int LPR = C::kRow / 16, RPI = 32 / LPR;  // lanes per row, rows per pass
      const int lw = warp - 8, jl = lane / LPR, cl = lane % LPR, key = lw * 32 + lane;
      const unsigned char* const base = reinterpret_cast<const unsigned char*>(P.pool) + cl * 16;
      const uint32_t vstep = (uint32_t)(P.H * P.pt);
      // places of this lane's chunks: the swizzle has NSW patterns
      constexpr int NSW = RPI >= 8 ? 1 : 8 / RPI;
      uint32_t swz[NSW];
#pragma unroll
      for (int k = 0; k < NSW; ++k) swz[k] = place<W>(kTK, k * RPI + jl, cl) - k * RPI * W;
      uint32_t it = 0;
      int left = 0, j = 0, lo = 0, hi = 0, b = 0, off = 0, last = 0;  // the item whose tiles are looked up
      int todo = 0;  // tiles looked up and not yet copied
      int pg[3], at[3], sq[3];  // page and place in it (-1: no such key) of this lane's key, three tiles
      auto fetch = [&](int i) {
        at[i] = -1;
        pg[i] = 0;
        if (left > 0 || !last) {
          if (left == 0) {
            const Item& x = item_at(it++);
            left = x.n_tiles;
            last = x.flags & 4;
            if (__any_sync(FULL_MASK, over())) left = last = 1;
            if (left == 0) return;  // no work for this CTA
            j = x.tile * kTK + key;
            lo = x.lo;
            hi = x.hi;
            b = x.b;
            off = x.h * P.pt;
          }
          if (j >= lo && j < hi) {
            const int blk = kv_block(P, j);
            pg[i] = __ldg(P.blocks + (int64_t)b * P.ldb + blk);
            at[i] = off + (j - blk * P.pt);
          }
          ++todo;
          sq[i] = b;
          j += kTK;
          --left;
        }
      };
      fetch(0);
      fetch(1);
      uint32_t slot = 0, phase = 1;
#pragma unroll 1
      for (int ti = 0; todo > 0; ++ti, --todo) {
        fetch(2);
        uint32_t row = kNoRow;
        if (at[0] >= 0) {
          if (pg[0] >= 0 && pg[0] < P.n_pages) row = ((uint32_t)pg[0] << P.row_shift) + (uint32_t)at[0];
          else record_error(P.err, kErrKvPage, sq[0]);
        }
        const unsigned have = __ballot_sync(FULL_MASK, row != kNoRow);
        uint32_t rows[32 / RPI];  // of this lane's chunks
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) rows[k] = __shfl_sync(FULL_MASK, row, k * RPI + jl);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          wait(&ctl->kv_empty[slot], phase);
          const uint32_t dst = sb + slot * C::kSlot + lw * 32 * W;
          const unsigned char* const from = base + (part ? (int64_t)vstep * C::kRow : 0);
          if (have == FULL_MASK) {
#pragma unroll
            for (int k = 0; k < 32 / RPI; ++k)
              cp16(dst + k * RPI * W + swz[k % NSW], from + (uint64_t)rows[k] * C::kRow);
          } else {
#pragma unroll 1
            for (int k = 0; k < 32 / RPI; ++k) {  // few tiles: little code rather than fast
              const int x = k * RPI + jl;
              const bool real = (have >> x) & 1;
              const uint32_t r = __shfl_sync(FULL_MASK, row, x);
              cp16(dst + place<W>(kTK, x, cl), real ? from + (uint64_t)r * C::kRow : base, real);
            }
          }
          if (part == 1) {
            if (F8) {
              const uint32_t sc = sb + C::kOffScale + ((ti % kMeta) * 2 * kTK + key) * 4;
              const bool real = row != kNoRow;
              cp4(sc, kv_scale(P, real ? row : 0), real);
              cp4(sc + kTK * 4, kv_scale(P, real ? row + vstep : 0), real);
            }
            if (lane == 0) ctl->mask[ti % kMeta][lw] = have;
          }
          arrive_copies(&ctl->kv_full[slot]);
          if (lane == 0) arrive(&ctl->kv_full[slot]);
          if (++slot == S) {
            slot = 0;
            phase ^= 1;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          pg[i] = pg[i + 1];
          at[i] = at[i + 1];
          sq[i] = sq[i + 1];
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 13) {
      // ------------------------------------------------------ the run's items
      // an item's lead.  0, 1, 2 tiles: 256 tokens (8 rows, 16-bit) 500, 481, 495 us, 64 tokens over an e4m3 cache 130,
      // 123, 124; 2, 3, 4 tiles: a mixed step with items of 40 rows 129, 129, 127.
      constexpr int E = TM <= 16 ? 1 : 3;
      Cursor<TM, kTK, E> c;
      Cut cut;
      const bool any = find_run<TM, kTK, E>(A, cls, kMinRun, c, cut);
      if (lane == 0) {
        if (!any) {
          ctl->item[0].n_tiles = 0;
          arrive(&ctl->item_full[0]);
        } else {
          for (uint32_t it = 0;; ++it) {
            const Item x = item_of(A, c);
            wait(&ctl->item_empty[it % kItems], ((it / kItems) & 1) ^ 1);
            ctl->item[it % kItems] = x;
            arrive(&ctl->item_full[it % kItems]);
            if ((x.flags & 3) == 1) note_split(split, c, cut, 2 * blockIdx.x + (it > 0 ? 1 : 0));
            if ((x.flags & 4) || !c.next(A, cls)) break;
          }
        }
      }
      __syncwarp();
    } else if (warp >= 14) {
      // ----------------------------------------------------- q, positions
      const int qw = warp - 14;
#pragma unroll 1
      for (uint32_t it = 0;; ++it) {
        const Item& x = item_at(it);
        if (x.n_tiles == 0) break;
        const int R = x.R, r_item = x.rt * TM, row0 = x.row0, hq0 = x.h * A.G, last = x.flags & 4;
        const uint32_t dst = sb + C::kOffQ + (it & 1) * C::kQ;
        for (int r = lane + 32 * qw; r < C::kRows16; r += 64)
          ctl->pos[it % kItems][r] = r < R ? x.first + token_of(A, r_item + r) : -1;
        wait(&ctl->q_empty[it & 1], ((it >> 1) & 1) ^ 1);
        auto row_of = [&](int r) -> const uint16_t* {
          const int t = token_of(A, r_item + r);
          return A.q + (int64_t)(row0 + t) * A.ldq + (int64_t)(hq0 + (r_item + r) - t * A.G) * D;
        };
        const int rows = (R + 15) / 16 * 16;
        if (!F8) {
          constexpr int QL = D / 8, QR = 32 / QL;  // lanes per row, rows per pass
          for (int r = qw * QR + lane / QL; r < rows; r += 2 * QR)
            cp16(dst + place<128>(C::kQRows, r, lane % QL), r < R ? row_of(r) + (lane % QL) * 8 : A.q, r < R);
        } else {
          constexpr int QL = D / 16, QR = 32 / QL;  // 16 elements a lane
          const int ch = lane % QL;
          uint4 v[2];
          auto load = [&](int r) {
            v[0] = v[1] = make_uint4(0, 0, 0, 0);
            if (r < R) {
              const uint4* const src = reinterpret_cast<const uint4*>(row_of(r)) + 2 * ch;
              v[0] = __ldg(src);
              v[1] = __ldg(src + 1);
            }
          };
          int r = qw * QR + lane / QL;
          load(r);
#pragma unroll 1
          for (; r - lane / QL < rows; r += 2 * QR) {
            const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
            load(r + 2 * QR);
            float f[16];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              up2<DT>(x[i], f[2 * i], f[2 * i + 1]);
              top = max(top, max(__float_as_uint(f[2 * i]) & 0x7fffffffu, __float_as_uint(f[2 * i + 1]) & 0x7fffffffu));
            }
#pragma unroll
            for (int o = QL / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(FULL_MASK, top, o));
            const int e = min(max((int)(top >> 23) - 127, -100), 127);
            const float up = __int_as_float((134 - e) << 23);  // 2^(7 - e)
            uint32_t p[3][4] = {};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              // an infinity or a NaN becomes a NaN code (satfinite would make the infinity a number)
              const float a = f[i] * up, b = f[i + 1] * up;
              uint32_t h[3];
              split3(a - a == 0.f ? a : NAN, b - b == 0.f ? b : NAN, h[0], h[1], h[2]);
#pragma unroll
              for (int q = 0; q < 3; ++q) p[q][i / 4] |= h[q] << (8 * (i & 2));
            }
            const int col = r / 16 * 48 + r % 16;
            if (r < rows) {
#pragma unroll
              for (int q = 0; q < 3; ++q)
                st_shared16(dst + place<W>(C::kQRows, col + q * 16, ch), p[q][0], p[q][1], p[q][2], p[q][3]);
              if (ch == 0) ctl->qmul[it % kItems][r] = A.c * __int_as_float((120 + e) << 23);
            }
          }
          fence_async_smem();
        }
        arrive_copies(&ctl->q_full[it & 1]);
        arrive(&ctl->q_full[it & 1]);
        arrive(&ctl->rows_full[it % kItems]);
        if (last || __any_sync(FULL_MASK, over())) break;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == 12) {
      // ---------------------------------------------------------- MMA issuer
      tmem_alloc(&ctl->tmem, C::kTmem);
      __syncwarp();
      const uint32_t tmem = ctl->tmem;
      arrive(&ctl->tmem_full);
      {
        const uint32_t fmt = !F8 && DT == SLORA_BF16 ? 1u : 0u;
        // fp32 accumulators; K is K-major, V (bit 15) and the weights (bit 16) are MN-major
        const uint32_t id_s = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 4) << 24);
        const uint32_t id_o = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | (1u << 16) | (((uint32_t)D >> 4) << 24);
        const uint32_t rows_hi = desc_hi(8 * W, W == 128 ? kSwizzle128 : kSwizzle64), weights_hi = desc_hi(kTK * 16, kNoSwizzle);
        const uint32_t k_lo = desc_lo(sb, 16), q_lo = desc_lo(sb + C::kOffQ, 16), v_lo = desc_lo(sb, C::kPanel);
        const uint32_t p_lo = desc_lo(sb + C::kOffP, 128);
        uint32_t qslot = 0, qphase = 0, qit = 0, vslot = 1, vphase = 0, vit = 0, obuf = 0;
        int qleft = 0, vleft = 0, qn = 0, vn = 0, vkey = 0;
        int qlast = 0, vlast = 0;  // the item is the run's last
        int vt = 0, vn0 = 0, vn1 = 0;
        bool first = true;
#pragma unroll 1
        for (int step = 0;; ++step) {
          if (qleft > 0 || !qlast) {  // scores of tile `step`
            const int ti = step;
            if (qleft == 0) {
              const Item& x = item_at(qit);
              qleft = x.n_tiles;
              qlast = x.flags & 4;
              if (qleft == 0 || __any_sync(FULL_MASK, over())) break;
              qn = (x.R + 15) / 16;
              wait(&ctl->q_full[qit & 1], (qit >> 1) & 1);
            }
            wait(&ctl->kv_full[qslot], qphase);
            fence_async_smem();  // the copies were generic writes
            tc_fence_after();
            const uint32_t id = id_s | (uint32_t)(F8 ? qn * 6 : qn * 2) << 17;
            const uint32_t a = k_lo + qslot * (C::kSlot >> 4), b = q_lo + (qit & 1) * (C::kQ >> 4);
            const uint32_t d = tmem + (ti & 1) * C::kSCols;
            --qleft;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < C::kRow / 32; ++k)
                mma<F8>(d, a + (((k >> 2) * C::kPanel + (k & 3) * 32) >> 4), rows_hi,
                        b + (((k >> 2) * (C::kQRows * W) + (k & 3) * 32) >> 4), rows_hi, id, k > 0);
              mma_commit(&ctl->s_full[ti & 1]);
              mma_commit(&ctl->kv_empty[qslot]);
              if (qleft == 0) mma_commit(&ctl->q_empty[qit & 1]);
            }
            __syncwarp();
            if (qleft == 0) ++qit;
            qslot += 2;
            if (qslot >= S) {
              qslot -= S;
              qphase ^= 1;
            }
          }
          if (step > 0) {  // products of tile `step - 1`
            const int ti = step - 1;
            if (vleft == 0) {
              const Item& x = item_at(vit++);
              vleft = x.n_tiles;
              vlast = x.flags & 4;
              vkey = x.tile * kTK;
              vn0 = x.open0;
              vn1 = x.open1;
              vt = 0;
              if (__any_sync(FULL_MASK, over())) break;
              vn = !F8 ? (x.R + 7) / 8 * 2 : TM == 8 ? (x.R + 3) / 4 * 2 : (x.R + 7) / 8 * 4;
              first = true;
              obuf = (vit - 1) % C::kOBufs;
              wait(&ctl->o_empty[obuf], (((vit - 1) / C::kOBufs) & 1) ^ 1);
            }
            wait(&ctl->kv_full[vslot], vphase);
            if (vt < vn0 || vt >= vn1)
              clean_tile<F8, DT, C::kRow / 16>(
                  &ctl->item[(vit - 1) % kItems], vkey + vt * kTK,
                  F8 ? reinterpret_cast<const float*>(smem + C::kOffScale) + ((ti % kMeta) * 2 + 1) * kTK : nullptr,
                  [&](int k, int c) { return sb + vslot * C::kSlot + place<W>(kTK, k, c); });
            ++vt;
            wait(&ctl->p_full[ti & 1], (ti >> 1) & 1);
            fence_async_smem();
            tc_fence_after();
            const uint32_t id = id_o | (uint32_t)vn << 17;
            const uint32_t a = v_lo + vslot * (C::kSlot >> 4), b = p_lo + (ti & 1) * (C::kP >> 4);
            const uint32_t od = tmem + 2 * C::kSCols + obuf * C::kPCols;
            --vleft;
            constexpr int KK = F8 ? 32 : 16;  // keys per MMA
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kTK / KK; ++k)
                mma<F8>(od, a + ((k * KK * W) >> 4), rows_hi, b + ((k * KK * 16) >> 4), weights_hi, id,
                        !(first && k == 0));
              mma_commit(&ctl->pv_done[ti & 1]);
              mma_commit(&ctl->kv_empty[vslot]);
              if (vleft == 0) mma_commit(&ctl->o_full[obuf]);
            }
            __syncwarp();
            first = false;
            vslot += 2;
            if (vslot >= S) {
              vslot -= S;
              vphase ^= 1;
            }
            if (vleft == 0 && vlast) break;
          }
        }
        if (elect_one()) mma_commit(&ctl->fin);  // every product and arrival is done before the block ends
        __syncwarp();
        wait(&ctl->fin, 0);
      }
    }
  } else if (warp < 8) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // A thread owns a key and half of the rows, in units: of 4 rows where there are 8, else every
    // other 8 rows.
    constexpr int UN = TM == 8 ? 4 : 8, NU = TM == 8 ? 1 : TM / 16;
    const int half = warp >> 2, wk = warp & 3, key = tid & 127;
    auto row_of = [&](int u) { return TM == 8 ? half * 4 : (2 * u + half) * 8; };
    auto s_col = [&](int r0) { return F8 ? r0 / 16 * 48 + r0 % 16 : r0; };
    auto o_col = [&](int r0) { return F8 ? r0 * 4 : r0 / 8 * 16 + r0 % 8; };
    constexpr int PS = F8 ? UN : 8, NP = F8 ? 4 : 2;  // columns from piece to piece of O^T, pieces
    const uint32_t tmem = tmem_at(), ts = tmem + ((uint32_t)(wk * 32) << 16);
    const float* const scales = reinterpret_cast<const float*>(smem + C::kOffScale);
    uint32_t ti = 0, vslot = 1, vphase = 0;
    float l[NU * UN];  // this key's sums
    // references and score multipliers: in registers where there are few
    constexpr bool kRegs = NU == 1;
    constexpr float kSlack = C::kSlack, kLift = C::kLift;  // references lie kLift below the maximum
    float mr[kRegs ? UN : 1] = {}, qm[kRegs ? UN : 1] = {}, iu[kRegs ? UN : 1] = {}, mv[kRegs ? UN : 1] = {};
    auto refs = [&](int u, int i) -> uint64_t {  // of rows i, i + 1
      return kRegs ? pair(mr[kRegs ? i : 0], mr[kRegs ? i + 1 : 0]) : *reinterpret_cast<const uint64_t*>(ctl->ref + row_of(u) + i);
    };
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
      const Item& x_ = item_at(it);
      const int n_here = x_.n_tiles, tile0 = x_.tile, R = x_.R, flags = x_.flags;
      if (softmax_any(over() || n_here == 0)) break;
      const uint32_t to = ts + 2 * C::kSCols + it % C::kOBufs * C::kPCols;
      wait(&ctl->rows_full[it % kItems], (it / kItems) & 1);
      const int* const pos = ctl->pos[it % kItems];
      const float* const qmul = ctl->qmul[it % kItems];
      const int pmin = pos[0], pmax = pos[R - 1];
#pragma unroll
      for (int r = 0; r < NU * UN; ++r) l[r] = 0.f;
      if (tid < TM) {
        ctl->ref[tid] = kNoRef;
        ctl->inv[tid] = 0x1p126f;
        ctl->vref[tid] = kNoRef;
      }
      if (kRegs) {
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          mr[kRegs ? i : 0] = kNoRef;
          iu[kRegs ? i : 0] = 0x1p126f;
          mv[kRegs ? i : 0] = kNoRef;
          if (F8) qm[kRegs ? i : 0] = qmul[row_of(0) + i];
        }
      }
      auto muls = [&](int u, int i) -> uint64_t {
        return kRegs ? pair(qm[kRegs ? i : 0], qm[kRegs ? i + 1 : 0]) : *reinterpret_cast<const uint64_t*>(qmul + row_of(u) + i);
      };
      auto invs = [&](int u, int i) -> uint64_t {
        return kRegs ? pair(iu[kRegs ? i : 0], iu[kRegs ? i + 1 : 0]) : *reinterpret_cast<const uint64_t*>(ctl->inv + row_of(u) + i);
      };
      auto vrefs = [&](int u, int i) -> uint64_t {
        return kRegs ? pair(mv[kRegs ? i : 0], mv[kRegs ? i + 1 : 0]) : *reinterpret_cast<const uint64_t*>(ctl->vref + row_of(u) + i);
      };
      softmax_sync();
#pragma unroll 1
      for (int n = 0; n < n_here; ++n, ++ti) {
        const uint32_t sbuf = ts + (ti & 1) * C::kSCols;
        // scales and mask, scores
        wait_for_both(&ctl->kv_full[vslot], vphase, &ctl->s_full[ti & 1], (ti >> 1) & 1, &ctl->dead, P.err);
        vslot += 2;
        if (vslot >= S) {
          vslot -= S;
          vphase ^= 1;
        }
        tc_fence_after();
        const uint32_t have = ctl->mask[ti % kMeta][wk];
        float ks = 1.f, vs = 1.f;
        if (F8) {
          ks = scales[(ti % kMeta) * 2 * kTK + key];
          vs = scales[((ti % kMeta) * 2 + 1) * kTK + key];
          vs = fabsf(vs) < INFINITY ? vs : __uint_as_float(0x7fc00000u);  // (an e4m3 code of an infinity would be a number)
        }
        const int key0 = (tile0 + n) * kTK, j = key0 + key;
        const bool open = have == FULL_MASK && key0 + kTK - 1 <= pmin && (A.window <= 0 || key0 > pmax - A.window);
        const bool mine = (have >> lane) & 1;
        const float lv = F8 ? __log2f(vs) : 0.f;
        float s[NU * UN];
        float most = -INFINITY;  // over the references
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int r0 = row_of(u);
          if (r0 < R) {
            float* const x = s + u * UN;
            const uint32_t col = sbuf + s_col(r0);
            if (!F8) {
              ld_n<UN>(col, x);
              wait_ld_n<UN>(x);
#pragma unroll
              for (int i = 0; i < UN; i += 2) unpair(mul2(pair(x[i], x[i + 1]), pair(A.c, A.c)), x[i], x[i + 1]);
            } else {
              float y[UN], z[UN];
              ld_n<UN>(col, x);
              ld_n<UN>(col + 16, y);
              ld_n<UN>(col + 32, z);
              wait_ld_n<UN>(x);
              wait_ld_n<UN>(y);
              wait_ld_n<UN>(z);
#pragma unroll
              for (int i = 0; i < UN; i += 2) {
                const uint64_t lo = fma2(pair(z[i], z[i + 1]), pair(0x1p-4f, 0x1p-4f), pair(y[i], y[i + 1]));
                const uint64_t all = fma2(lo, pair(0x1p-4f, 0x1p-4f), pair(x[i], x[i + 1]));
                unpair(mul2(all, mul2(pair(ks, ks), muls(u, i))), x[i], x[i + 1]);
              }
            }
            if (!open) {
#pragma unroll
              for (int i = 0; i < UN; ++i) {
                const int p = pos[r0 + i];
                if (!mine || j > p || (A.window > 0 && j <= p - A.window)) x[i] = -INFINITY;
              }
            }
#pragma unroll
            for (int i = 0; i < UN; i += 2) {
              float a, b;
              unpair(add2(pair(x[i], x[i + 1]), refs(u, i)), a, b);
              most = max3(most, a, b);  // (with kLift)
              if (F8) {
                unpair(add2(add2(pair(x[i], x[i + 1]), pair(lv, lv)), vrefs(u, i)), a, b);
                most = max3(most, a, b);
              }
            }
          }
        }
        if (softmax_any(most > kSlack + kLift)) {  // some reference moves to its tile's maximum, or a unit to its tile's largest weight
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            if (row_of(u) < R) {
#pragma unroll
              for (int i = 0; i < UN; ++i) {
                const float x = s[u * UN + i], v = warp_max(x);
                if (lane == 0) ctl->red[0][wk][row_of(u) + i] = v;
                if (F8) {
                  const float w = warp_max(x == -INFINITY ? x : x + lv);
                  if (lane == 0) ctl->red[1][wk][row_of(u) + i] = w;
                }
              }
            }
          }
          softmax_sync();
          if (tid < (R + UN - 1) / UN * UN) {
            const int r = tid;
            auto top_of = [&](int k) {
              return fmaxf(fmaxf(ctl->red[k][0][r], ctl->red[k][1][r]), fmaxf(ctl->red[k][2][r], ctl->red[k][3][r]));
            };
            const float top = top_of(0), m = ctl->ref[r];  // negated
            // e4m3: a whole number, so that a reference moves beside a unit without a rounding of either
            const float m1 = top + m > kSlack + kLift ? (F8 ? -ceilf(top) : kLift - top) : m;
            ctl->fac[r] = m1 == m ? 1.f : ex2(m1 - m);
            ctl->ref[r] = m1;
            if (F8) {
              const bool none = m == kNoRef;
              const float e = (float)(127 - (__float_as_int(ctl->inv[r]) >> 23));  // log2 of the unit
              const float keep = none ? -INFINITY : e + (m1 - m), need = top_of(1) + m1;
              float e1 = need - keep > kSlack ? ceilf(need) - C::kSet : keep;
              e1 = fminf(fmaxf(e1, -126.f), 126.f);
              ctl->ofac[r] = none || e1 == keep ? 1.f : ex2(keep - e1);
              ctl->inv[r] = __int_as_float((127 - (int)e1) << 23);
              ctl->vref[r] = m1 - e1;
            }
          }
          if (n > 0) {  // the products so far
            wait(&ctl->pv_done[(ti - 1) & 1], ((ti - 1) >> 1) & 1);
            tc_fence_after();
          }
          softmax_sync();
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            const int r0 = row_of(u);
            if (r0 < R) {
              float f[UN];
              bool same = true;
#pragma unroll
              for (int i = 0; i < UN; ++i) {
                l[u * UN + i] *= ctl->fac[r0 + i];
                f[i] = F8 ? ctl->ofac[r0 + i] : ctl->fac[r0 + i];
                same &= f[i] == 1.f;
                if (kRegs) mr[kRegs ? i : 0] = ctl->ref[r0 + i];
                if (F8 && kRegs) {
                  iu[kRegs ? i : 0] = ctl->inv[r0 + i];
                  mv[kRegs ? i : 0] = ctl->vref[r0 + i];
                }
              }
              if (n > 0 && !same) {
#pragma unroll 1
                for (int q = 0; q < NP; ++q) {
                  float o[UN];
                  ld_n<UN>(to + o_col(r0) + q * PS, o);
                  wait_ld_n<UN>(o);
#pragma unroll
                  for (int i = 0; i < UN; ++i) o[i] *= f[i];
                  st_n<UN>(to + o_col(r0) + q * PS, o);
                }
              }
            }
          }
          wait_st();
        }
        // the weights of tile ti - 2 have been used: its products were issued before these scores
        const uint32_t pd = sb + C::kOffP + (ti & 1) * C::kP + key * 16;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const int r0 = row_of(u);
          if (r0 < R) {
            uint32_t w[4][UN / 2];
#pragma unroll
            for (int i = 0; i < UN; i += 2) {
              const float* const x = s + u * UN + i;
              float a, b;
              unpair(add2(pair(x[0], x[1]), refs(u, i)), a, b);
              const uint64_t pp = pair(ex2(a), ex2(b));
              if (F8) {  // (p * vs first: no factor of it is out of range where the weight is not)
                unpair(mul2(mul2(pp, pair(vs, vs)), invs(u, i)), a, b);
                if (!open) {  // an infinite or NaN scale of an unseen key stays out
                  a = x[0] == -INFINITY ? 0.f : a;
                  b = x[1] == -INFINITY ? 0.f : b;
                }
                split4_weights(pair(a, b), w[0][i / 2], w[1][i / 2], w[2][i / 2], w[3][i / 2]);
              } else {
                unpair(pp, a, b);
                split2<DT>(a, b, w[0][i / 2], w[1][i / 2]);
              }
              unpair(add2(pair(l[u * UN + i], l[u * UN + i + 1]), pp), l[u * UN + i], l[u * UN + i + 1]);
            }
            if (F8) {  // a unit's columns in 16 bytes (4 rows) or twice 16
              uint32_t c[8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                c[q * (UN / 4)] = w[q][0] | w[q][1] << 16;
                if (UN == 8) c[2 * q + 1] = w[q][UN / 2 - 2] | w[q][UN / 2 - 1] << 16;
              }
              const uint32_t dst = pd + r0 / 4 * (kTK * 16);
              st_shared16(dst, c[0], c[1], c[2], c[3]);
              if (UN == 8) st_shared16(dst + kTK * 16, c[4], c[5], c[6], c[7]);
            } else {
#pragma unroll
              for (int q = 0; q < NP; ++q) {
                const uint32_t dst = pd + (r0 / 8 * 2 + q) * (kTK * 16) + r0 % 8 * 2;
                if (UN == 8) st_shared16(dst, w[q][0], w[q][1], w[q][UN / 2 - 2], w[q][UN / 2 - 1]);
                else st_shared8(dst, w[q][0], w[q][1]);
              }
            }
          }
        }
        fence_async_smem();
        tc_fence_before();
        arrive(&ctl->p_full[ti & 1]);
      }

      // ---- the item's sums, for the epilogue (which is through with those of item it - 2)
      wait(&ctl->o_empty[it % C::kOBufs], ((it / C::kOBufs) & 1) ^ 1);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (row_of(u) < R) {  // over the warp's keys: the lanes end in UN groups, one per row
          float v[UN];
#pragma unroll
          for (int i = 0; i < UN; ++i) v[i] = l[u * UN + i];
#pragma unroll
          for (int o = 16, k = UN / 2; o >= 1; o >>= 1, k >>= 1) {
            if (k >= 1) {
              const bool up = lane & o;
#pragma unroll
              for (int i = 0; i < k; ++i) {
                const float give = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
                v[i] = keep + __shfl_xor_sync(FULL_MASK, give, o);
              }
            } else {
              v[0] += __shfl_xor_sync(FULL_MASK, v[0], o);
            }
          }
          if (lane % (32 / UN) == 0) ctl->sum[it & 1][wk][row_of(u) + lane / (32 / UN)] = v[0];
        }
      }
      if (tid < TM) {
        ctl->end_ref[it & 1][tid] = ctl->ref[tid] == kNoRef ? -INFINITY : kLift - ctl->ref[tid];
        if (F8) ctl->unit[it & 1][tid] = 1.f / ctl->inv[tid];
      }
      arrive(&ctl->sum_full[it & 1]);
      if (flags & 4) break;
    }
  } else {
    // ------------------------------------------- the rows of an item, or their partials
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int wl = warp - 16, tl = tid - 512;
    if (blockIdx.x == 0) kv_record_bad(P, A.max_rows, tl, 128);
    const uint32_t tmem = tmem_at(), ts = tmem + ((uint32_t)(wl * 32) << 16);
    const int d = D == 128 ? tl : wl * 16 + (lane & 15);
    const bool writes = D == 128 || lane < 16;
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
      const Item& x_ = item_at(it);
      const int R = x_.R, flags = x_.flags, r_item = x_.rt * TM, hq0 = x_.h * A.G;
      if (epilogue_any(over() || x_.n_tiles == 0)) break;
      const int NH = (R + 7) / 8;
      const int64_t row0 = x_.row0;
      const bool complete = (flags & 3) == 3;
      float* const part = parts + (size_t)(2 * blockIdx.x + (it > 0 ? 1 : 0)) * slot_floats(TM, D);
      const uint32_t to = ts + 2 * C::kSCols + it % C::kOBufs * C::kPCols;
      wait(&ctl->sum_full[it & 1], (it >> 1) & 1);
      if (tl < R) {
        const int r = tl, t = token_of(A, r_item + r), hq = hq0 + (r_item + r) - t * A.G;
        const float (*const sum)[TM] = ctl->sum[it & 1];
        const float m = ctl->end_ref[it & 1][r], lr = (sum[0][r] + sum[1][r]) + (sum[2][r] + sum[3][r]);
        const float l0 = lr * pow2(-C::kLift);  // of weights of 1 at the maximum
        ctl->out_fac[r] = inverse(lr);
        if (complete) {
          if (A.lse) A.lse[(row0 + t) * A.Hq + hq] = lse_of(m, l0);
        } else {
          part[(size_t)TM * D + r] = m;
          part[(size_t)TM * (D + 1) + r] = l0;
        }
      }
      epilogue_sync();
      wait(&ctl->o_full[it % C::kOBufs], (it / C::kOBufs) & 1);
      tc_fence_after();
      uint32_t bad[2] = {0, 0};
      uint16_t* orow;      // row h * 8 of the output, or of the partial
      float* prow = part + d;
      int hq;
      {
        const int t = token_of(A, r_item);
        hq = r_item - t * A.G;
        orow = A.out + (row0 + t) * A.ldo + (int64_t)(hq0 + hq) * D + d;
      }
      const int64_t step = A.ldo - (int64_t)A.G * D;  // behind a token's last head
#pragma unroll 1
      for (int h = 0; h < NH; ++h) {
        constexpr int NP = F8 ? 4 : 2;
        float v[NP][8], o[8];
        const uint32_t col = to + h * (8 * NP);
#pragma unroll
        for (int q = 0; q < NP; ++q) ld8(col + 8 * q, v[q]);
#pragma unroll
        for (int q = 0; q < NP; ++q) wait_ld8(v[q]);
        auto piece = [&](int q, int i) {  // of rows i, i + 1 (8 rows a unit, or twice 4)
          const int at = F8 && TM == 8 ? i / 4 * 16 + q * 4 + i % 4 : q * 8 + i;
          return pair(v[at / 8][at % 8], v[at / 8][at % 8 + 1]);
        };
        uint64_t zero = 0;  // sum of 0 * output: NaN if one is not finite
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint64_t all;
          if constexpr (F8) {
            const uint64_t s5 = pair(0x1p-5f, 0x1p-5f);
            all = fma2(fma2(fma2(piece(3, i), s5, piece(2, i)), s5, piece(1, i)), s5, piece(0, i));
          } else {
            all = add2(piece(1, i), piece(0, i));
          }
          const uint64_t f2 = *reinterpret_cast<const uint64_t*>(ctl->out_fac + h * 8 + i);
          unpair(f2, f[i], f[i + 1]);
          all = mul2(all, f2);
          if (F8) all = mul2(all, *reinterpret_cast<const uint64_t*>(ctl->unit[it & 1] + h * 8 + i));
          unpair(all, o[i], o[i + 1]);
          o[i] = f[i] == 0.f || h * 8 + i >= R ? 0.f : o[i];  // sees no key, or is no row
          o[i + 1] = f[i + 1] == 0.f || h * 8 + i + 1 >= R ? 0.f : o[i + 1];
          zero = fma2(pair(o[i], o[i + 1]), pair(0.f, 0.f), zero);
        }
        float z0, z1;
        unpair(zero, z0, z1);
        if (writes && z0 + z1 != 0.f) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(fabsf(o[i]) < INFINITY)) bad[h >> 2] |= 1u << ((h & 3) * 8 + i);
        }
        if (complete) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (writes && h * 8 + i < R) *orow = (uint16_t)pk2<DT>(o[i], 0.f);
            orow += D;
            if (++hq == A.G) {
              hq = 0;
              orow += step;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (writes && h * 8 + i < R) prow[i * D] = o[i];
          prow += 8 * D;
        }
      }
      tc_fence_before();
      const bool odd = *reinterpret_cast<const volatile int*>(&x_.odd);
      if (__builtin_expect(epilogue_any((bad[0] | bad[1]) != 0 || odd), 0)) {  // rows that are not finite, or of a marked item
        bad[0] = __reduce_or_sync(FULL_MASK, bad[0]);
        bad[1] = __reduce_or_sync(FULL_MASK, bad[1]);
        if (lane == 0) {
          ctl->bad[wl][0] = bad[0];
          ctl->bad[wl][1] = bad[1];
        }
        epilogue_sync();
        uint32_t any[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) any[k] = ctl->bad[0][k] | ctl->bad[1][k] | ctl->bad[2][k] | ctl->bad[3][k];
        const bool common = __any_sync(FULL_MASK, any[0] | any[1]);
        // a warp's rows: wl, wl + 4, ...; those that see no key, or whose sum is a NaN, are what they should be
        const int r = wl + 4 * lane;
        const bool due = r < R && ctl->end_ref[it & 1][r] != -INFINITY && ctl->out_fac[r] == ctl->out_fac[r] &&
                         (odd || (((r < 32 ? any[0] : any[1]) >> (r & 31)) & 1));
        const uint32_t rows = __ballot_sync(FULL_MASK, due);
        if (rows) settle<DT, FMT, D, TM>(A, x_, rows, wl, 4, common, part);
        epilogue_sync();
      }
      arrive(&ctl->o_empty[it % C::kOBufs]);
      if (tl == 0) arrive(&ctl->item_empty[it % kItems]);
      if (flags & 4) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(ctl->tmem, C::kTmem);
}

template <int DT, int FMT, int D, int TM>
cudaError_t run_decode(const KvAttnDev& A, int sm_count, RowClass cls, cudaStream_t st) {
  using C = Cfg<DT, FMT, D, TM>;
  constexpr int bytes = 1024 + C::kOffCtl + (int)sizeof(Ctl<TM, C::kSlots>);
  static_assert(bytes <= 232448 && C::kOffCtl % 16 == 0, "shared memory");
  static std::atomic<bool> sized[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_decode<DT, FMT, D, TM>), bytes, sized);
  if (e != cudaSuccess) return e;
  k_kv_decode<DT, FMT, D, TM><<<sm_count, kNT, bytes, st>>>(A, cls);
  return cudaGetLastError();
}

template <int DT, int FMT, int D>
cudaError_t run_rows(const KvAttnDev& A, int TM, int sm_count, RowClass cls, cudaStream_t st) {
  if (TM == 8) return run_decode<DT, FMT, D, 8>(A, sm_count, cls, st);
  if (TM == 16) return run_decode<DT, FMT, D, 16>(A, sm_count, cls, st);
  return run_decode<DT, FMT, D, kv_stream_rows(FMT)>(A, sm_count, cls, st);
}

}  // namespace

size_t kv_stream_workspace(int fmt, int D, int sm_count) {
  return (size_t)sm_count * sizeof(Split) + 2 * (size_t)sm_count * slot_floats(kv_stream_rows(fmt), D) * 4;
}

cudaError_t launch_kv_stream(const KvAttnDev& A, int dtype, int fmt, int D, int TM, int sm_count, cudaStream_t s) {
  const RowClass cls = {0, kv_stream_rows(fmt)};
  if (D == 128) {
    if (dtype == SLORA_F16)
      return fmt == SLORA_KV_16 ? run_rows<SLORA_F16, SLORA_KV_16, 128>(A, TM, sm_count, cls, s)
                                : run_rows<SLORA_F16, SLORA_KV_E4M3, 128>(A, TM, sm_count, cls, s);
    return fmt == SLORA_KV_16 ? run_rows<SLORA_BF16, SLORA_KV_16, 128>(A, TM, sm_count, cls, s)
                              : run_rows<SLORA_BF16, SLORA_KV_E4M3, 128>(A, TM, sm_count, cls, s);
  }
  if (dtype == SLORA_F16)
    return fmt == SLORA_KV_16 ? run_rows<SLORA_F16, SLORA_KV_16, 64>(A, TM, sm_count, cls, s)
                              : run_rows<SLORA_F16, SLORA_KV_E4M3, 64>(A, TM, sm_count, cls, s);
  return fmt == SLORA_KV_16 ? run_rows<SLORA_BF16, SLORA_KV_16, 64>(A, TM, sm_count, cls, s)
                            : run_rows<SLORA_BF16, SLORA_KV_E4M3, 64>(A, TM, sm_count, cls, s);
}

}  // namespace slora

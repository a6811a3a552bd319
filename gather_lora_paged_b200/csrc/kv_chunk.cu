// kv_chunk.cu -- attention of prompt chunks (more rows per kv head than kv_decode.cu takes) over
// the KV pages on the 5th-generation tensor cores.  Definition and row order as
// in kv_decode.cu; runs, partials and their join as in kv_attn.cuh.
//
// One CTA per SM, 16 warps; an item is 256 rows (token, head of the group) of
// one kv head as two M = 128 tiles, its keys come 128 at a time:
//   warps 8..11 copy q once per item and K, V of each tile from the pages into a
//               ring of shared-memory slots (128-byte swizzle, K K-major, V as the
//               MN-major operand of P.V; a page may hold one token, so rows are
//               gathered by 16-byte cp.async, whose arrivals fill a slot's barrier).
//               e4m3 codes become their exact fp16 values on the way.
//   warp 12     issues, per q tile i, P_i.V_n as its weights come and S_i = Q_i.K_(n+1)^T behind
//               them (tcgen05.mma, P_i from TMEM), so that the softmax of
//               one q tile runs while the tensor cores work for the other.
//   warp 13     the run's items, for all others.
//   warps 0..3, 4..7   the softmax of q tile 0 and 1: a thread owns a row, reads its
//               scores from TMEM, and writes the weights back over them in 16 bits; at the
//               item's end it writes the row.
// TMEM: S0, S1 (128 columns each, P over S), O0, O1 (D columns each).
// The reference point of a row's weights (its maximum so far, less kLift) moves only when the
// maximum has grown by 2^8, and the accumulator in TMEM is read and scaled on few tiles.  fp16 weights are 2^7
// at the maximum, 2^15 at most, so that what falls below fp16's least step is under 2^-32 of the maximum's.
// Sums and statistics are fp32 and of the unrounded weights; the weights are
// rounded once to the operand type, which puts an error of the size of the output's own
// rounding on it (the two halves of kv_decode.cu would double the P.V
// product, which is half the work here).
// e4m3: K's scale multiplies the score, V's the weight, over a unit (a power of two) of each row's own, so that
// keys that a row does not see have no part in it: the largest product of weight and scale that the row
// has met is 2^7..2^8 units where the unit is set, and 2^15 at most before it moves.
//
// What bounds it: both products of a tile take 2100 cycles (128 columns and 16 elements 64), the
// exponentials of its 256 x 128 weights as long on the special-function units; a tile takes 3300, as
// a q tile's softmax (2200) and its products (1050) follow one another.  2 x 1024..2048 tokens over 8192 keys, 64
// heads on 8 of 128, bf16, three inputs in turn: 1.18 ms, 1000 TFLOP/s at 1.5 to 1.64 GHz (the power
// limit), tensor pipe 58 % of the cycles.  A quarter of the exponentials as polynomials on the FMA pipe did not pay (1234 us for 1184):
// the softmax waits for latencies and issue slots more than for the special-function units.
#include <math.h>

#include <type_traits>

#include "kv_attn.cuh"
#include "kv_tc.cuh"

namespace slora {
namespace {

constexpr int kNT = 512;
constexpr int kTM = 256;      // rows per item
constexpr int kTK = kKvTile;  // keys per tile
constexpr int kHalf = kTK / 2;  // weights are handed over for so many keys
constexpr int kMinRun = 2;
constexpr int kLead = 2;      // an item's lead: q and the outputs cost about two tiles
constexpr int kItems = 4;     // items that are known ahead
constexpr int kMeta = 8;      // tiles whose scales and masks are kept
constexpr float kSlack = 8.f; // log2 by which a maximum may exceed the one that set the reference
// e4m3: log2 of the largest weight where a unit is set, and of what it may grow to (fp16 ends at 2^16)
constexpr int kSet = 7;
constexpr float kMost = 0x1p15f;

template <int FMT, int D>
struct Cfg {
  // Keys of one S, the softmax's step.  With 64, S of the next tile's half is computed while the softmax is at
  // the other half, but an MMA of N = 64 takes 55 cycles, of N = 128 69: 16-bit chunks over 8192 take 1300 us
  // with 64 and 1207 with 128; in e4m3, where the softmax has more to do, a mixed step takes 129 and 138.
  static constexpr int kPart = FMT == SLORA_KV_16 ? 128 : 64;
  static constexpr int kPanel = 128 * 128;                 // 128 rows of 64 16-bit elements
  static constexpr int kSlot = D / 64 * kPanel;            // K or V of a tile
  static constexpr int kSlots = FMT == SLORA_KV_16 ? 5 : 4;
  static constexpr int kQ = 2 * kSlot;                     // two q tiles
  static constexpr int kOffRing = kQ;
  static constexpr int kOffScale = kOffRing + kSlots * kSlot;
  static constexpr int kScale = FMT == SLORA_KV_E4M3 ? kMeta * 2 * kTK * 4 : 0;  // K and V scales of tiles
  static constexpr int kOffQs = kOffScale + kScale;        // score multipliers of items' rows
  static constexpr int kOffCtl = kOffQs + (FMT == SLORA_KV_E4M3 ? kItems * kTM * 4 : 0);
};

template <int S>
struct Ctl {
  uint64_t kv_full[S], kv_empty[S], q_full, q_empty, item_full[kItems], item_empty[kItems], rows_full[kItems];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2], o_full[2], tmem_full, fin;  // [q tile][part, half of the keys]
  Item item[kItems];
  uint32_t tmem;
  int dead;                    // a wait gave up: nobody waits any more
  alignas(16) uint32_t mask[kMeta][4];  // keys of a tile that are there
};

__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
__device__ __forceinline__ void st32(uint32_t taddr, const float* v) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
// tcgen05.wait::ld, tied to the registers that a load fills
__device__ __forceinline__ void wait_ld32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]),
                 "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                 "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of 16-byte chunk c (8 elements) of row j in a slot: panels of 64
// elements, 128-byte rows, chunks swizzled by the row.
__device__ __forceinline__ uint32_t place(int j, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4));
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kNT, 1) k_kv_chunk(const __grid_constant__ KvAttnDev A, RowClass cls) {
  using C = Cfg<FMT, D>;
  constexpr bool F8 = FMT == SLORA_KV_E4M3;
  constexpr int MT = F8 ? SLORA_F16 : DT;  // operand type of the products
  constexpr int S = C::kSlots, kPart = C::kPart, kParts = kTK / kPart;
  // log2 of the weight at a row's maximum.  fp16: weights are up to 2^15 (it ends at 2^16).  bf16: of 2^16
  // keys at 2^8 over the maximum none of V's products and sums overflows, however large V is.
  constexpr int kLift = F8 ? 0 : MT == SLORA_F16 ? 7 : -24;
  using Control = Ctl<S>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = su32(smem);
  Control* const ctl = reinterpret_cast<Control*>(smem + C::kOffCtl);
  float* const scales = reinterpret_cast<float*>(smem + C::kOffScale);
  float* const qscale = reinterpret_cast<float*>(smem + C::kOffQs);
  const KvDev& P = A.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Split* const split = reinterpret_cast<Split*>(A.chunk_workspace) + blockIdx.x;
  float* const parts = reinterpret_cast<float*>(reinterpret_cast<Split*>(A.chunk_workspace) + gridDim.x);

  griddep_launch();  // the join's CTAs may take their places (they wait for this grid's end)
  if (tid == 0) split->n = 0;
  if (warp == 12) {
    for (int i = lane; i < S; i += 32) {
      bar_init(&ctl->kv_full[i], 128 + (F8 ? 128 : 4));
      bar_init(&ctl->kv_empty[i], 1);
    }
    if (lane < kItems) {
      bar_init(&ctl->item_full[lane], 1);
      bar_init(&ctl->item_empty[lane], 2);
      bar_init(&ctl->rows_full[lane], 128);
    }
    if (lane < 2) {
      bar_init(&ctl->s_full[lane][0], 1);
      bar_init(&ctl->s_full[lane][1], 1);
      bar_init(&ctl->pv_done[lane], 1);
      bar_init(&ctl->p_full[lane][0], 128);
      bar_init(&ctl->p_full[lane][1], 128);
      bar_init(&ctl->o_full[lane], 1);
    }
    if (lane < kItems) {  // what those see who did not wait for an entry (see wait_slow)
      ctl->item[lane].flags = 4;
      ctl->item[lane].n_tiles = 0;
    }
    if (lane == 0) {
      bar_init(&ctl->q_full, 256);
      bar_init(&ctl->q_empty, 1);
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
  // An item's entry.  It is written again for item it + 4, once both softmax groups are through with
  // this one; all others have read it by then.
  auto item_at = [&](uint32_t it) -> const Item& {
    wait(&ctl->item_full[it % kItems], (it / kItems) & 1);
    return ctl->item[it % kItems];
  };

  // 128 registers at launch: the softmax warps, which hold a row's scores, take from the
  // others (184 + 184 + 88 + 56 = 4 * 128)
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 13) {
      // ------------------------------------------------------ the run's items
      Cursor<kTM, kTK, kLead> c;
      Cut cut;
      const bool any = find_run<kTM, kTK, kLead>(A, cls, kMinRun, c, cut);
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
    } else if (warp == 12) {
      // ---------------------------------------------------------- MMA issuer
      tmem_alloc(&ctl->tmem, 512);
      __syncwarp();
      const uint32_t tmem = ctl->tmem;
      arrive(&ctl->tmem_full);
      const uint32_t fmt = MT == SLORA_BF16 ? 1u : 0u;
      const uint32_t id0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((128u >> 4) << 24);
      const uint32_t id_s = id0 | ((uint32_t)kPart >> 3) << 17, id_o = id0 | (1u << 16) | ((uint32_t)D >> 3) << 17;  // V: MN-major
      const uint32_t hi = desc_hi(1024, kSwizzle128);
      const uint32_t q_lo = desc_lo(sb, 16), k_lo = desc_lo(sb + C::kOffRing, 16), v_lo = desc_lo(sb + C::kOffRing, C::kPanel);
      uint32_t g = 0, parity = 0;  // slots so far; a bit per q tile, of its weights' barriers
      auto qk = [&](int i, int part, uint32_t slot) {
        const uint32_t a = q_lo + i * (C::kSlot >> 4), b = k_lo + slot * (C::kSlot >> 4) + part * ((kPart * 128) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::kPanel + (k & 3) * 32) >> 4;
          mma<false>(tmem + i * 128 + part * kPart, a + off, hi, b + off, hi, id_s, k > 0);
        }
        mma_commit(&ctl->s_full[i][part]);
      };
      auto pv = [&](int i, int half, uint32_t slot, bool first) {
        const uint32_t b = v_lo + slot * (C::kSlot >> 4) + half * ((kHalf * 128) >> 4), a = tmem + i * 128 + half * (kPart == 128 ? 32 : 64);
#pragma unroll
        for (int k = 0; k < kHalf / 16; ++k)
          mma_ts(tmem + 256 + i * 128, a + k * 8, b + ((k * 2048) >> 4), hi, id_o, !(first && half == 0 && k == 0));
        mma_commit(&ctl->pv_done[i]);
      };
#pragma unroll 1
      for (uint32_t it = 0;; ++it) {
        const Item& x = item_at(it);
        const int n_tiles = x.n_tiles, last = x.flags & 4, q_tiles = x.R > 128 ? 2 : 1, open0 = x.open0, open1 = x.open1;
        if (n_tiles == 0) break;
        wait(&ctl->q_full, it & 1);
        wait(&ctl->kv_full[g % S], (g / S) & 1);
        fence_async_smem();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            qk(0, part, g % S);
            if (q_tiles == 2) qk(1, part, g % S);
          }
          mma_commit(&ctl->kv_empty[g % S]);
          if (n_tiles == 1) mma_commit(&ctl->q_empty);
        }
        __syncwarp();
#pragma unroll 1
        for (int n = 0; n < n_tiles; ++n, g += 2) {
          const bool more = n + 1 < n_tiles;
          const uint32_t v = (g + 1) % S, k = (g + 2) % S;
          wait(&ctl->kv_full[v], ((g + 1) / S) & 1);
          if (n < open0 || n >= open1)
            clean_tile<false, MT, D / 8>(&ctl->item[it % kItems], (x.tile + n) * kTK,
                                         F8 ? scales + (((g >> 1) % kMeta) * 2 + 1) * kTK : nullptr,
                                         [&](int k, int c) { return sb + C::kOffRing + v * C::kSlot + place(k, c); });
          if (more) wait(&ctl->kv_full[k], ((g + 2) / S) & 1);
#pragma unroll 1
          for (int step = 0; step < 2 * q_tiles; ++step) {  // in the order in which the weights come
            const int i = kParts == 1 ? step >> 1 : step & (q_tiles - 1), half = kParts == 1 ? step & 1 : step >> (q_tiles - 1);
            wait(&ctl->p_full[i][half], (parity >> i) & 1);
            fence_async_smem();
            tc_fence_after();
            if (elect_one()) {
              pv(i, half, v, n == 0);
              if (half == 1 && !more) mma_commit(&ctl->o_full[i]);
              if (more && (kParts == 2 || half == 1)) qk(i, kParts == 2 ? half : 0, k);
              if (step + 1 == 2 * q_tiles) {
                mma_commit(&ctl->kv_empty[v]);
                if (more) mma_commit(&ctl->kv_empty[k]);
                if (n + 2 == n_tiles) mma_commit(&ctl->q_empty);
              }
            }
            __syncwarp();
          }
          parity ^= 3u >> (2 - q_tiles);
        }
        if (last || __any_sync(FULL_MASK, over())) break;
      }
      if (elect_one()) mma_commit(&ctl->fin);  // every product and arrival is done before the block ends
      __syncwarp();
      wait(&ctl->fin, 0);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- loaders
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    constexpr int CB = F8 ? D : 2 * D;                         // bytes of a cached row
    constexpr int LPR = CB / 16, RPI = 32 / LPR, KM = 32 / RPI;  // lanes per row, rows per pass, passes
    const int lw = warp - 8, jl = lane / LPR, cl = lane % LPR, key = lw * 32 + lane;
    const unsigned char* const base = reinterpret_cast<const unsigned char*>(P.pool) + cl * 16;
    const uint32_t vstep = (uint32_t)(P.H * P.pt);
    uint32_t g = 0, ti = 0;              // slots and tiles so far
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
      const Item& x = item_at(it);
      const int n_tiles = x.n_tiles, lo = x.lo, hi = x.hi, b = x.b, off = x.h * P.pt, last = x.flags & 4;
      if (n_tiles == 0) break;
      int j = x.tile * kTK + key;
      const int32_t* const table = P.blocks + (int64_t)b * P.ldb;
      int pg = 0, at = -1;                 // page and place in it (-1: no such key) of this lane's key in the next tile
      auto fetch = [&] {
        at = -1;
        if (j >= lo && j < hi) {
          const int blk = kv_block(P, j);
          pg = __ldg(table + blk);
          at = off + (j - blk * P.pt);
        }
        j += kTK;
      };
      fetch();

      // q: rows of both tiles, zeros behind the item's last row
      wait(&ctl->q_empty, (it & 1) ^ 1);
      {
        constexpr int QL = D / 8, QR = 32 / QL;  // lanes per row, rows per pass
        const int R = x.R, r_item = x.rt * kTM, row0 = x.row0, hq0 = x.h * A.G;
        const int rows = R > 128 ? 256 : 128;
#pragma unroll 2
        for (int p = lw; p < rows / QR; p += 4) {
          const int r = p * QR + lane / QL, ch = lane % QL;
          const bool real = r < R;
          const int t = real ? token_of(A, r_item + r) : 0;
          const uint16_t* src = A.q + (real ? (int64_t)(row0 + t) * A.ldq + (int64_t)(hq0 + (r_item + r) - t * A.G) * D + ch * 8 : 0);
          const uint32_t dst = sb + (r >> 7) * C::kSlot + place(r & 127, ch);
          if (!F8 || DT == SLORA_F16) {
            cp16(dst, src, real);
            if (F8 && ch == 0) qscale[(it % kItems) * kTM + r] = A.c;
          } else {  // a bf16 row as fp16 times a power of two: [1, 2) at its largest; what falls below fp16's
                    // range is under 2^-25 of that
            const uint4 v = real ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = QL / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(FULL_MASK, top, o));
            const int e = min(max((int)(top >> 7) - 127, -100), 126);
            const float f = __int_as_float((127 - e) << 23);
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              h[i] = pack2<SLORA_F16>(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xffff0000u) * f);
            st_shared16(dst, h[0], h[1], h[2], h[3]);
            if (ch == 0) qscale[(it % kItems) * kTM + r] = A.c * __int_as_float((127 + e) << 23);
          }
        }
        if (F8) fence_async_smem();
      }
      arrive_copies(&ctl->q_full);
      arrive(&ctl->q_full);
      arrive(&ctl->rows_full[it % kItems]);

      auto resolve = [&](unsigned& have) -> uint32_t {  // the row of this lane's key
        uint32_t row = kNoRow;
        if (at >= 0) {
          if (pg >= 0 && pg < P.n_pages) row = ((uint32_t)pg << P.row_shift) + (uint32_t)at;
          else record_error(P.err, kErrKvPage, b);
        }
        have = __ballot_sync(FULL_MASK, row != kNoRow);
        return row;
      };
      if (!F8) {
#pragma unroll 1
        for (int n = 0; n < n_tiles; ++n, ++ti) {
          unsigned have;
          const uint32_t row = resolve(have);
          if (n + 1 < n_tiles) fetch();
          uint32_t rows[KM];  // of this lane's chunks
#pragma unroll
          for (int k = 0; k < KM; ++k) rows[k] = __shfl_sync(FULL_MASK, row, k * RPI + jl);
#pragma unroll 1
          for (int part = 0; part < 2; ++part, ++g) {
            wait(&ctl->kv_empty[g % S], ((g / S) & 1) ^ 1);
            const uint32_t slot = sb + C::kOffRing + (g % S) * C::kSlot;
            const unsigned char* const from = base + (part ? (int64_t)vstep * CB : 0);
            if (have == FULL_MASK) {
#pragma unroll
              for (int k = 0; k < KM; ++k) cp16(slot + place(lw * 32 + k * RPI + jl, cl), from + (uint64_t)rows[k] * CB);
            } else {
#pragma unroll
              for (int k = 0; k < KM; ++k) {
                const bool real = (have >> (k * RPI + jl)) & 1;
                cp16(slot + place(lw * 32 + k * RPI + jl, cl), real ? from + (uint64_t)rows[k] * CB : base, real);
              }
            }
            if (part == 1 && lane == 0) ctl->mask[ti % kMeta][lw] = have;
            arrive_copies(&ctl->kv_full[g % S]);
            if (lane == 0) arrive(&ctl->kv_full[g % S]);
          }
        }
      } else {
        uint4 code[KM];  // of the next slot
        unsigned have = 0, have_next = 0;
        uint32_t row = resolve(have);
        auto load = [&](int part, uint32_t r0, unsigned hv) {
          const unsigned char* const from = base + (part ? (int64_t)vstep * CB : 0);
#pragma unroll
          for (int k = 0; k < KM; ++k) {
            const uint32_t r = __shfl_sync(FULL_MASK, r0, k * RPI + jl);
            code[k] = make_uint4(0, 0, 0, 0);
            if ((hv >> (k * RPI + jl)) & 1) code[k] = __ldg(reinterpret_cast<const uint4*>(from + (uint64_t)r * CB));
          }
        };
        load(0, row, have);
#pragma unroll 1
        for (int n = 0; n < n_tiles; ++n, ++ti) {
          uint32_t row_next = kNoRow;
#pragma unroll
          for (int part = 0; part < 2; ++part, ++g) {
            wait(&ctl->kv_empty[g % S], ((g / S) & 1) ^ 1);
            const uint32_t slot = sb + C::kOffRing + (g % S) * C::kSlot;
#pragma unroll
            for (int k = 0; k < KM; ++k) {
              const int y = lw * 32 + k * RPI + jl;
              const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
                st_shared16(slot + place(y, 2 * cl + hh), e4m3x2_f16x2(w[2 * hh]), e4m3x2_f16x2(w[2 * hh] >> 16),
                            e4m3x2_f16x2(w[2 * hh + 1]), e4m3x2_f16x2(w[2 * hh + 1] >> 16));
            }
            if (part == 0) {
              load(1, row, have);
              if (n + 1 < n_tiles) fetch();
            } else {
              const uint32_t sc = sb + C::kOffScale + ((ti % kMeta) * 2 * kTK + key) * 4;
              const bool real = row != kNoRow;
              cp4(sc, kv_scale(P, real ? row : 0), real);
              cp4(sc + kTK * 4, kv_scale(P, real ? row + vstep : 0), real);
              if (lane == 0) ctl->mask[ti % kMeta][lw] = have;
              if (n + 1 < n_tiles) {
                row_next = resolve(have_next);
                load(0, row_next, have_next);
              }
            }
            fence_async_smem();
            arrive_copies(&ctl->kv_full[g % S]);
            arrive(&ctl->kv_full[g % S]);
          }
          row = row_next;
          have = have_next;
        }
      }
      if (last || __any_sync(FULL_MASK, over())) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int wg = warp >> 2;
    wait(&ctl->tmem_full, 0);
    const uint32_t tmem = ctl->tmem;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tq = tmem + lanes + wg * 128, to = tmem + lanes + 256 + wg * 128;
    uint32_t sn = 0, on = 0, ti = 0, pv = 0;  // tiles with this q tile, items with it, tiles; weights handed over
#pragma unroll 1
    for (uint32_t it = 0;; ++it) {
      const Item& x = item_at(it);
      const int n_tiles = x.n_tiles;
      const bool none = over() || n_tiles == 0;
      if (wg == 0 ? any_of<1, 128>(none) : any_of<2, 128>(none)) break;
      if (wg == 0 || x.R > 128) {
        const int r = wg * 128 + (warp & 3) * 32 + lane;
        int pos = -1, low = -1, pmin, pmax;  // of this row (keys above `low` are seen), of this q tile's first, the item's last
        {
          const int R = x.R, first = x.first, r_item = x.rt * kTM;
          if (r < R) {
            pos = first + token_of(A, r_item + r);
            if (A.window > 0) low = pos - A.window;
          }
          pmin = first + token_of(A, r_item + wg * 128);
          pmax = first + token_of(A, r_item + R - 1);
        }
        float m = -INFINITY, l = 0.f, cr = A.c;
        float unit = -126.f, inv_unit = 0x1p126f;  // e4m3: log2 of the unit of this row's weights
        if (F8) {
          wait(&ctl->rows_full[it % kItems], (it / kItems) & 1);
          cr = qscale[(it % kItems) * kTM + r];
        }
#pragma unroll 1
        for (int n = 0; n < n_tiles; ++n, ++ti, ++sn) {
          const uint32_t g = 2 * ti + 1;
          // Scales and mask.  The scores first: a group that passed over an item would find V's barrier two
          // phases behind, which looks like done; with these scores issued, the phase before is over.
          wait(&ctl->s_full[wg][0], sn & 1);
          wait(&ctl->kv_full[g % S], (g / S) & 1);
          const float* const ks = scales + (ti % kMeta) * 2 * kTK;
          const int key0 = (x.tile + n) * kTK;
          const uint4 have = *reinterpret_cast<const uint4*>(ctl->mask[ti % kMeta]);
          const bool masked = key0 + kTK - 1 > pmin || (A.window > 0 && key0 <= pmax - A.window) ||
                              (have.x & have.y & have.z & have.w) != FULL_MASK;
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            const uint32_t ts = tq + part * kPart;
            if (part > 0) wait(&ctl->s_full[wg][part], sn & 1);
            tc_fence_after();
            float s[kPart];
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const float* const kh = ks + part * kPart;
#pragma unroll
            for (int h = 0; h < kPart; h += 64) {
              ld32(ts + h, s + h);
              ld32(ts + h + 32, s + h + 32);
              wait_ld32(s + h);
              wait_ld32(s + h + 32);
              if (F8) {
#pragma unroll
                for (int i = h; i < h + 64; i += 4) {
                  const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(kh + i);
                  unpair(mul2(pair(s[i], s[i + 1]), k4.x), s[i], s[i + 1]);
                  unpair(mul2(pair(s[i + 2], s[i + 3]), k4.y), s[i + 2], s[i + 3]);
                }
              }
              if (masked) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {  // bits of the keys low < j <= pos
                  const int word = (part * kPart + h) / 32 + w, base = key0 + 32 * word - 1;
                  const int h2 = min(max(pos - base, 0), 32), l2 = min(max(low - base, 0), 32);
                  const uint32_t below_h = h2 == 32 ? FULL_MASK : (1u << h2) - 1, below_l = l2 == 32 ? FULL_MASK : (1u << l2) - 1;
                  const uint32_t there = ctl->mask[ti % kMeta][word];
                  const uint32_t seen = there & below_h & ~below_l;
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!((seen >> i) & 1)) s[h + w * 32 + i] = -INFINITY;
                }
              }
#pragma unroll
              for (int i = h; i < h + 64; i += 8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) top[q] = max3(top[q], s[i + 2 * q], s[i + 2 * q + 1]);
              }
            }
            float mn = fmaxf(m, fmaf(fmaxf(max3(top[0], top[1], top[2]), top[3]), cr, -(float)kLift));
            auto scale_products = [&](float f) {  // those so far
              wait(&ctl->pv_done[wg], (pv + 1) & 1);
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                float o[32];
                ld32(to + i, o);
                wait_ld32(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= f;
                st32(to + i, o);
              }
            };
            float f = 1.f;  // e4m3: what scales them
            if (__any_sync(FULL_MASK, mn > m + kSlack)) {
              // e4m3: a whole number, so that a reference moves beside the unit without a rounding of either
              if (F8) mn = ceilf(mn);
              const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
              if (F8 && mn != -INFINITY) {
                const float keep = unit + (m - mn);
                unit = fmaxf(keep, -126.f);
                f = unit == keep || m == -INFINITY ? 1.f : ex2(keep - unit);
                inv_unit = __int_as_float((127 - (int)unit) << 23);
              }
              m = mn;
              l *= a;
              if (!F8 && (n > 0 || part > 0)) scale_products(a);
            }
            const float mz = m == -INFINITY ? 0.f : m;
            const uint64_t c2 = pair(cr, cr), m2 = pair(-mz, -mz);
            uint64_t ls[2] = {0, 0};
            if (F8) {  // weights times V's scales, over the scores
              float most[2] = {0.f, 0.f};
              auto scale_v = [&](auto all_seen) {
                constexpr bool kOpen = decltype(all_seen)::value;
#pragma unroll
                for (int i = 0; i < kPart; i += 2) {
                  float p[2], q[2];
                  unpair(fma2(pair(s[i], s[i + 1]), c2, m2), p[0], p[1]);
                  const uint64_t pp = pair(ex2(p[0]), ex2(p[1]));
                  ls[(i >> 1) & 1] = add2(ls[(i >> 1) & 1], pp);
                  unpair(mul2(pp, *reinterpret_cast<const uint64_t*>(kh + kTK + i)), q[0], q[1]);
                  if (!kOpen) {  // an infinite or NaN scale of an unseen key stays out
                    q[0] = s[i] == -INFINITY ? 0.f : q[0];
                    q[1] = s[i + 1] == -INFINITY ? 0.f : q[1];
                  }
                  s[i] = q[0];
                  s[i + 1] = q[1];
                  most[(i >> 1) & 1] = max3(most[(i >> 1) & 1], q[0], q[1]);
                }
              };
              if (masked) scale_v(std::false_type{});
              else scale_v(std::true_type{});
              const float big = fmaxf(most[0], most[1]);
              if (big * inv_unit > kMost) {  // the unit moves: to this row's largest so far
                const float to_unit = fminf((float)((__float_as_int(big) >> 23) - 127 - kSet), 126.f);
                f *= ex2(unit - to_unit);
                unit = to_unit;
                inv_unit = __int_as_float((127 - (int)unit) << 23);
              }
            }
            if (F8 && (n > 0 || part > 0) && __any_sync(FULL_MASK, f != 1.f)) scale_products(f);
            const uint64_t iu2 = pair(inv_unit, inv_unit);
#pragma unroll
            for (int i = 0; i < kPart; i += 32) {  // the weights
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float p[2];
                if (F8) {
                  unpair(mul2(pair(s[i + k], s[i + k + 1]), iu2), p[0], p[1]);
                } else {
                  unpair(fma2(pair(s[i + k], s[i + k + 1]), c2, m2), p[0], p[1]);
                  p[0] = ex2(p[0]);
                  p[1] = ex2(p[1]);
                  ls[(k >> 1) & 1] = add2(ls[(k >> 1) & 1], pair(p[0], p[1]));
                }
                w[k / 2] = pk2<MT>(p[0], p[1]);
              }
              st16(ts + i / 2, w);
              if (i % 64 == 32) {  // the products with these 64 keys may begin
                wait_st();
                tc_fence_before();
                arrive(&ctl->p_full[wg][part + i / 64]);
              }
            }
            pv += kPart / 64;
            float a, b;
            unpair(add2(ls[0], ls[1]), a, b);
            l += a + b;
          }
        }

        // ---- the rows of this item, or their partials
        wait(&ctl->o_full[wg], on++ & 1);
        tc_fence_after();
        // (the entry is read again: what the tiles do not need is not kept through them)
        const bool complete = (x.flags & 3) == 3;
        const int R = x.R, r_item = x.rt * kTM, t = r < R ? token_of(A, r_item + r) : 0;
        const int hq = r < R ? x.h * A.G + (r_item + r) - t * A.G : 0;
        const int64_t tok = x.row0 + t;
        const float inv = inverse(l);
        uint16_t* const orow = A.out + tok * A.ldo + (int64_t)hq * D;
        float* const part = parts + (size_t)(2 * blockIdx.x + (it > 0 ? 1 : 0)) * slot_floats(kTM, D);
        float* const prow = part + (size_t)r * D;
        const float f = F8 ? 1.f / inv_unit : 1.f;
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          ld32(to + i, o);
          wait_ld32(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            o[k] *= inv;
            if (F8) o[k] *= f;
            if (l == 0.f) o[k] = 0.f;  // sees no key
            bad |= !(fabsf(o[k]) < INFINITY);
          }
          if (r < R) {
            if (complete) {
#pragma unroll
              for (int k = 0; k < 32; k += 8)
                *reinterpret_cast<uint4*>(orow + i + k) = make_uint4(pk2<DT>(o[k], o[k + 1]), pk2<DT>(o[k + 2], o[k + 3]),
                                                                     pk2<DT>(o[k + 4], o[k + 5]), pk2<DT>(o[k + 6], o[k + 7]));
            } else {
#pragma unroll
              for (int k = 0; k < 32; k += 4)
                *reinterpret_cast<float4*>(prow + i + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
          }
        }
        tc_fence_before();
        const float m0 = m + kLift, l0 = l * pow2(-kLift);  // the maximum, the sum of weights of 1 there
        if (r < R) {
          if (complete) {
            if (A.lse) A.lse[tok * A.Hq + hq] = lse_of(m0, l0);
          } else {
            part[(size_t)kTM * D + r] = m0;
            part[(size_t)kTM * (D + 1) + r] = l0;
          }
        }
        // rows that are not finite, or of a marked item; those that see no key, or whose sum is a NaN, are what
        // they should be
        const bool odd = *reinterpret_cast<const volatile int*>(&x.odd), common = __any_sync(FULL_MASK, bad && r < R);
        const uint32_t rows = __ballot_sync(FULL_MASK, r < R && m != -INFINITY && l == l && (bad || odd));
        __syncwarp();
        if (__builtin_expect(rows != 0, 0)) settle<DT, FMT, D, kTM>(A, x, rows, wg * 128 + (warp & 3) * 32, 1, common, part);
      } else {
        ti += n_tiles;
      }
      const int last = x.flags & 4;
      // all four warps are through with the entry
      if (wg == 0) sync_of<1, 128>();
      else sync_of<2, 128>();
      if ((tid & 127) == 0) arrive(&ctl->item_empty[it % kItems]);
      if (last) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(ctl->tmem, 512);
  griddep_wait();  // for kv_decode.cu's grid: who waits for this one waits for both
}

// The joins of kv_decode.cu's items (row tiles of TM) and, if there are two grids, of this file's.
template <int DT, int D, int TM>
__global__ void __launch_bounds__(kCombineThreads) k_kv_join(KvAttnDev A, int ctas) {
  griddep_wait();
  if ((int)blockIdx.x < ctas) join_item<DT, D, TM>(A, A.workspace, blockIdx.x, ctas);
  else join_item<DT, D, kTM>(A, A.chunk_workspace, blockIdx.x - ctas, ctas);
}

template <int DT, int FMT, int D>
cudaError_t run_chunk(const KvAttnDev& A, int sm_count, RowClass cls, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  static std::atomic<bool> sized[64];
  constexpr int bytes = 1024 + C::kOffCtl + (int)sizeof(Ctl<C::kSlots>);
  static_assert(bytes <= 232448 && C::kOffCtl % 16 == 0, "shared memory");
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_chunk<DT, FMT, D>), bytes, sized);
  if (e != cudaSuccess) return e;
  return launch_behind(k_kv_chunk<DT, FMT, D>, dim3(sm_count), kNT, bytes, st, A, cls);
}

template <int DT, int D>
cudaError_t run_join(const KvAttnDev& A, int TM, bool chunks, int sm_count, cudaStream_t st) {
  // a row per warp, two where there are row tiles of 256
  const dim3 grid(chunks ? 2 * sm_count : sm_count, chunks ? kTM / 16 : TM / 8);
  if (TM == 8) return launch_behind(k_kv_join<DT, D, 8>, grid, kCombineThreads, 0, st, A, sm_count);
  if (TM == 16) return launch_behind(k_kv_join<DT, D, 16>, grid, kCombineThreads, 0, st, A, sm_count);
  if (TM == 32) return launch_behind(k_kv_join<DT, D, 32>, grid, kCombineThreads, 0, st, A, sm_count);
  return launch_behind(k_kv_join<DT, D, 48>, grid, kCombineThreads, 0, st, A, sm_count);
}

}  // namespace

size_t kv_chunk_workspace(int D, int sm_count) {
  return (size_t)sm_count * sizeof(Split) + 2 * (size_t)sm_count * slot_floats(kTM, D) * 4;
}

cudaError_t launch_kv_join(const KvAttnDev& A, int dtype, int D, int TM, bool chunks, int sm_count, cudaStream_t s) {
  if (D == 128)
    return dtype == SLORA_F16 ? run_join<SLORA_F16, 128>(A, TM, chunks, sm_count, s)
                              : run_join<SLORA_BF16, 128>(A, TM, chunks, sm_count, s);
  return dtype == SLORA_F16 ? run_join<SLORA_F16, 64>(A, TM, chunks, sm_count, s)
                            : run_join<SLORA_BF16, 64>(A, TM, chunks, sm_count, s);
}

cudaError_t launch_kv_chunk(const KvAttnDev& A, int dtype, int fmt, int D, int sm_count, cudaStream_t s) {
  const RowClass cls = {kv_stream_rows(fmt), INT32_MAX};
  if (D == 128) {
    if (dtype == SLORA_F16)
      return fmt == SLORA_KV_16 ? run_chunk<SLORA_F16, SLORA_KV_16, 128>(A, sm_count, cls, s)
                                : run_chunk<SLORA_F16, SLORA_KV_E4M3, 128>(A, sm_count, cls, s);
    return fmt == SLORA_KV_16 ? run_chunk<SLORA_BF16, SLORA_KV_16, 128>(A, sm_count, cls, s)
                              : run_chunk<SLORA_BF16, SLORA_KV_E4M3, 128>(A, sm_count, cls, s);
  }
  if (dtype == SLORA_F16)
    return fmt == SLORA_KV_16 ? run_chunk<SLORA_F16, SLORA_KV_16, 64>(A, sm_count, cls, s)
                              : run_chunk<SLORA_F16, SLORA_KV_E4M3, 64>(A, sm_count, cls, s);
  return fmt == SLORA_KV_16 ? run_chunk<SLORA_BF16, SLORA_KV_16, 64>(A, sm_count, cls, s)
                            : run_chunk<SLORA_BF16, SLORA_KV_E4M3, 64>(A, sm_count, cls, s);
}

}  // namespace slora

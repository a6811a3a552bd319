// kv_chunk.cu -- attention of prompt chunks (more than 64 rows per kv head) over
// the KV pages on the 5th-generation tensor cores.  Definition and row order as
// in kv_decode.cu; runs, partials and their join as in kv_attn.cuh.
//
// One CTA per SM, 12 warps; an item is 256 rows (token, head of the group) of
// one kv head as two M = 128 tiles, its keys come 128 at a time:
//   warps 8..10  copy q once per item and K, V of each tile from the pages into a
//                ring of shared-memory slots (128-byte swizzle, K K-major, V as the
//                MN-major operand of P.V; a page may hold one token, so rows are
//                gathered by 16-byte cp.async).  e4m3 codes become their exact fp16
//                values on the way.
//   warp 11      one thread issues, per tile n and q tile i, P_i.V_n and S_i =
//                Q_i.K_(n+1)^T (tcgen05.mma, P_i from TMEM), so that the softmax of
//                one q tile runs while the tensor cores work for the other.
//   warps 0..3, 4..7   the softmax of q tile 0 and 1: a thread owns a row, reads its 128
//                scores from TMEM, and writes the weights back over them in 16 bits.
// TMEM: S0, S1 (128 columns each, P over S), O0, O1 (D columns each).
// The reference point of a row's weights (its maximum so far) moves only when the
// maximum has grown by 2^8: weights then reach at most 2^8, far inside
// fp16's range, and the accumulator in TMEM is read and scaled on few tiles.
// Sums and statistics are fp32 and of the unrounded weights; the weights are
// rounded once to the operand type, which puts an error of the size of the output's own
// rounding on it (the two halves of kv_decode.cu would double the P.V
// product, which is half the work here).
// e4m3: K's scale multiplies the score, V's the weight, relative to a V scale
// that is raised when a tile's largest is 8 times it.
#include <math.h>

#include "kv_attn.cuh"
#include "tc_common.cuh"

namespace slora {
namespace {

using namespace tc;

constexpr int kNT = 384;
constexpr int kTM = 256;      // rows per item
constexpr int kTK = 128;      // keys per tile
constexpr int kLoadWarps = 3;
constexpr int kLoaders = kLoadWarps * 32;
constexpr int kMinRun = 2;
constexpr int kCtlBytes = 1280;
constexpr float kSlack = 8.f; // log2 of the largest weight

template <int FMT, int D>
struct Cfg {
  static constexpr int kPanel = 128 * 128;                 // 128 rows of 64 16-bit elements
  static constexpr int kSlot = D / 64 * kPanel;            // K or V of a tile
  static constexpr int kSlots = FMT == SLORA_KV_16 ? 5 : 4;
  static constexpr int kQ = 2 * kSlot;                     // two q tiles
  static constexpr int kOffRing = kQ;
  static constexpr int kOffScale = kOffRing + kSlots * kSlot;
  static constexpr int kScale = FMT == SLORA_KV_E4M3 ? 4 * 2 * kTK * 4 : 0;  // 4 tiles of K and V scales
  static constexpr int kOffQs = kOffScale + kScale;        // score multipliers of the 256 rows
  static constexpr int kOffCtl = kOffQs + (FMT == SLORA_KV_E4M3 ? 2 * kTM * 4 : 0);  // of two items
  static constexpr int kSmem = 1024 + kOffCtl + kCtlBytes;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Ctl {
  uint64_t kv_full[5], kv_empty[5], q_full, q_empty, s_full[2], p_full[2], o_full[2], fin;
  uint32_t tmem;
  int dead;                          // a wait gave up: nobody waits any more
  uint32_t any_bad[4][4];            // [tile & 3][loader warp]: keys on bad pages
  uint32_t bad[4][kLoadWarps][4];    // their bits
  float vtop[4][4];                  // [tile & 3][loader warp]: largest V scale
  uint32_t rows[kLoadWarps][64];     // the loader warps' pool rows of a tile
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

__device__ __forceinline__ void arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool ready(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(su32(b)), "r"(parity) : "memory");
  return done;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// Products with the A operand in TMEM.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
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
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of 16-byte chunk c (8 elements) of row j in a slot: panels of 64
// elements, 128-byte rows, chunks swizzled by the row.
__device__ __forceinline__ uint32_t place(int j, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4));
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kNT, 1) k_kv_chunk(const __grid_constant__ KvAttnDev A, RowClass cls) {
  using C = Cfg<FMT, D>;
  constexpr int MT = FMT == SLORA_KV_16 ? DT : SLORA_F16;  // operand type of the products
  constexpr int S = C::kSlots;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const smem = smem_raw + ((1024 - (su32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = su32(smem);
  Ctl* const ctl = reinterpret_cast<Ctl*>(smem + C::kOffCtl);
  float* const scales = reinterpret_cast<float*>(smem + C::kOffScale);
  float* const qscale = reinterpret_cast<float*>(smem + C::kOffQs);
  const KvDev& P = A.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Split* const split = reinterpret_cast<Split*>(A.workspace) + blockIdx.x;
  float* const parts = reinterpret_cast<float*>(reinterpret_cast<Split*>(A.workspace) + gridDim.x);

  if (tid == 0) split->n = 0;
  Cursor<kTM, kTK> c;
  long long total, u1;
  int ctas;
  if (!find_run<kTM, kTK, kNT>(A, cls, kMinRun, reinterpret_cast<long long*>(smem), c, total, ctas, u1)) return;

  if (warp == 11) {
    if (lane == 0) {
      for (int i = 0; i < S; ++i) {
        bar_init(&ctl->kv_full[i], kLoaders);
        bar_init(&ctl->kv_empty[i], 1);
      }
      bar_init(&ctl->q_full, kLoaders);
      bar_init(&ctl->q_empty, 1);
      for (int i = 0; i < 2; ++i) {
        bar_init(&ctl->s_full[i], 1);
        bar_init(&ctl->p_full[i], 128);
        bar_init(&ctl->o_full[i], 1);
      }
      bar_init(&ctl->fin, 1);
      ctl->dead = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    tmem_alloc(&ctl->tmem, 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (*reinterpret_cast<volatile int*>(&ctl->dead)) return;
    if (!bar_wait(b, parity, P.err)) *reinterpret_cast<volatile int*>(&ctl->dead) = 1;
  };

  // 168 registers at launch: the softmax warps, which hold a row's scores, take
  // from the others (104 * 128 + 200 * 256 = 136 * 128 + 184 * 256 = 168 * 384)
  if (warp >= 8) {
    if (FMT == SLORA_KV_16) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
  if (warp < 11) {
    // ---------------------------------------------------------------- loaders
    const int lw = warp - 8;
    constexpr int LPR = C::kSlot ? (FMT == SLORA_KV_16 ? D / 8 : D / 16) : 1;  // lanes per cached row (16 bytes each)
    constexpr int RPI = 32 / LPR;
    constexpr int KW = (kTK + kLoadWarps - 1) / kLoadWarps;                    // keys per warp: lw, lw + 3, ...
    constexpr int KM = (KW + RPI - 1) / RPI;                                   // passes over them
    const int jl = lane / LPR, cl = lane % LPR;
    uint32_t* const rows_of = ctl->rows[lw];
    const unsigned char* const base = reinterpret_cast<const unsigned char*>(P.pool);
    const uint32_t vstep = (uint32_t)(P.H * P.pt);
    uint32_t g = 0, qi = 0, ti = 0;        // slots, items and tiles so far
    uint64_t *pend0 = nullptr, *pend1 = nullptr;  // barriers of copies in flight, oldest first
    auto flush = [&] {
      if (pend0 || pend1) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_async_smem();
        if (pend0) arrive(pend0);
        if (pend1) arrive(pend1);
        pend0 = pend1 = nullptr;
      }
    };
    auto push = [&](uint64_t* b) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (pend0) {
        asm volatile("cp.async.wait_group 2;" ::: "memory");
        fence_async_smem();
        arrive(pend0);
      }
      pend0 = pend1;
      pend1 = b;
    };
    auto acquire = [&](uint64_t* b, uint32_t parity) {  // what is in flight may be what the slot waits for
      if (!ready(b, parity)) {
        flush();
        wait(b, parity);
      }
    };
    for (;;) {
      const int n_tiles = (int)min((long long)(c.x.t1 - c.tile), c.left);
      const int r_item = c.rt * kTM, R = min(c.s.n * A.G - r_item, kTM);
      int pg[2];                              // pages of keys lw + 3 * lane and 32 keys of this warp on
      auto fetch = [&](int tile) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int x = lw + kLoadWarps * (lane + 32 * q), j = tile * kTK + x;
          pg[q] = x < kTK && j >= c.x.lo && j < c.x.hi ? __ldg(P.blocks + (int64_t)c.b * P.ldb + kv_block(P, j)) : 0;
        }
      };
      auto resolve = [&](int tile, uint32_t t) {  // the tile's rows from pg; t: its number
        unsigned bad = 0;
        __syncwarp();                             // the last tile's rows have been read
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int x = lw + kLoadWarps * (lane + 32 * q), j = tile * kTK + x;
          uint32_t r = kNoRow;
          if (x < kTK && j >= c.x.lo && j < c.x.hi) {
            if (pg[q] >= 0 && pg[q] < P.n_pages) r = ((uint32_t)pg[q] << P.row_shift) + (uint32_t)(c.h * P.pt + j - kv_block(P, j) * P.pt);
            else bad |= 1u << q;
          }
          rows_of[lane + 32 * q] = r;
        }
        __syncwarp();
        const bool any = __any_sync(FULL_MASK, bad);
        if (lane == 0) ctl->any_bad[t & 3][lw] = any;
        if (any) {
          if (lane == 0) record_error(P.err, kErrKvPage, c.b);
          if (lane < 4) ctl->bad[t & 3][lw][lane] = 0;
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int x = lw + kLoadWarps * (lane + 32 * q);
            if ((bad >> q) & 1) atomicOr(&ctl->bad[t & 3][lw][x >> 5], 1u << (x & 31));
          }
        }
      };
      fetch(c.tile);

      // q: rows of both tiles, zeros behind the item's last row
      acquire(&ctl->q_empty, (qi & 1) ^ 1);
      {
        constexpr int QL = D / 8, QR = 32 / QL;  // lanes per row, rows per pass
        const int rows = R > 128 ? 256 : 128;
        for (int p = lw; p < rows / QR; p += kLoadWarps) {
          const int r = p * QR + lane / QL, ch = lane % QL;
          const bool real = r < R;
          const int t = real ? (r_item + r) / A.G : 0;
          const uint16_t* src = A.q + (int64_t)(c.s.row0 + t) * A.ldq +
                                (real ? (int64_t)(c.h * A.G + (r_item + r) - t * A.G) * D + ch * 8 : 0);
          const uint32_t dst = sb + (r >> 7) * C::kSlot + place(r & 127, ch);
          if (FMT == SLORA_KV_16 || DT == SLORA_F16) {
            cp16(dst, src, real);
            if (FMT == SLORA_KV_E4M3 && ch == 0) qscale[(qi & 1) * kTM + r] = A.c;
          } else {  // a bf16 row as fp16 times a power of two (see kv_decode.cu)
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
            if (ch == 0) qscale[(qi & 1) * kTM + r] = A.c * __int_as_float((127 + e) << 23);
          }
        }
      }
      push(&ctl->q_full);
      ++qi;

      if (FMT == SLORA_KV_16) {
        for (int n = 0; n < n_tiles; ++n, ++ti) {
          resolve(c.tile + n, ti);
          if (n + 1 < n_tiles) fetch(c.tile + n + 1);
#pragma unroll 1
          for (int part = 0; part < 2; ++part, ++g) {
            acquire(&ctl->kv_empty[g % S], ((g / S) & 1) ^ 1);
            const uint32_t slot = sb + C::kOffRing + (g % S) * C::kSlot;
#pragma unroll 4
            for (int k = 0; k < KM; ++k) {
              const int x = lw + kLoadWarps * (k * RPI + jl);
              const uint32_t r = rows_of[k * RPI + jl];
              const int64_t at = r != kNoRow ? (int64_t)(r + part * vstep) * (2 * D) + cl * 16 : 0;
              if (x < kTK) cp16(slot + place(x, cl), base + at, r != kNoRow);
            }
            push(&ctl->kv_full[g % S]);
          }
        }
      } else {
        uint4 code[2][KM];
        auto load = [&](int part, uint32_t t) {  // codes to registers, scales straight to their place
#pragma unroll
          for (int k = 0; k < KM; ++k) {
            const int x = lw + kLoadWarps * (k * RPI + jl);
            const uint32_t first_row = rows_of[k * RPI + jl];
            const bool real = first_row != kNoRow;
            const uint32_t r = real ? first_row + part * vstep : 0;
            code[part][k] = make_uint4(0, 0, 0, 0);
            if (real) code[part][k] = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)r * D + cl * 16));
            if (cl == 0 && x < kTK)
              cp4(sb + C::kOffScale + (((t & 3) * 2 + part) * kTK + x) * 4, kv_scale(P, r), real);
          }
        };
        flush();
        resolve(c.tile, ti);
        if (n_tiles > 1) fetch(c.tile + 1);
        load(0, ti);
        load(1, ti);
        for (int n = 0; n < n_tiles; ++n, ++ti) {
#pragma unroll
          for (int part = 0; part < 2; ++part, ++g) {
            wait(&ctl->kv_empty[g % S], ((g / S) & 1) ^ 1);
            const uint32_t slot = sb + C::kOffRing + (g % S) * C::kSlot;
            if (part == 0) {  // the tile's scales have arrived: the largest of V's
              asm volatile("cp.async.wait_all;" ::: "memory");
              float top = 0.f;
#pragma unroll
              for (int k = 0; k < KM; ++k) {
                const int x = lw + kLoadWarps * (k * RPI + jl);
                if (cl == 0 && x < kTK) top = fmaxf(top, scales[((ti & 3) * 2 + 1) * kTK + x]);
              }
#pragma unroll
              for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
              if (lane == 0) ctl->vtop[ti & 3][lw] = top;
            }
#pragma unroll
            for (int k = 0; k < KM; ++k) {
              const int x = lw + kLoadWarps * (k * RPI + jl);
              const uint32_t w[4] = {code[part][k].x, code[part][k].y, code[part][k].z, code[part][k].w};
              if (x < kTK) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                  st_shared16(slot + place(x, 2 * cl + hh), e4m3x2_f16x2(w[2 * hh]), e4m3x2_f16x2(w[2 * hh] >> 16),
                              e4m3x2_f16x2(w[2 * hh + 1]), e4m3x2_f16x2(w[2 * hh + 1] >> 16));
              }
            }
            fence_async_smem();
            arrive(&ctl->kv_full[g % S]);
            if (n + 1 < n_tiles) {
              // the next tile: K after this one's K, V after its V.  Its place among the scales and
              // bad-page bits is that of tile ti - 3, which is through: K's slot of this tile was free
              if (part == 0) {
                resolve(c.tile + n + 1, ti + 1);
                if (n + 2 < n_tiles) fetch(c.tile + n + 2);
              }
              load(part, ti + 1);
            }
          }
        }
      }
      c.tile += n_tiles - 1;
      c.left -= n_tiles - 1;
      if (!c.next(A, cls)) break;
    }
    flush();
  } else {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_f16(MT, kTK, 0), id_o = idesc_f16(MT, D, 1);
      const uint32_t ring = sb + C::kOffRing;
      uint32_t g = 0, qi = 0, pn[2] = {0, 0};
      auto qk = [&](int i, uint32_t slot) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * C::kPanel + (k & 3) * 32;
          mma_f16(tmem + i * 128, sdesc(sb + i * C::kSlot + off, 16, 1024), sdesc(ring + slot * C::kSlot + off, 16, 1024), id_s,
                  k > 0);
        }
        mma_commit(&ctl->s_full[i]);
      };
      auto pv = [&](int i, uint32_t slot, bool first) {
        wait(&ctl->p_full[i], pn[i]++ & 1);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTK / 16; ++k)
          mma_f16_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, sdesc(ring + slot * C::kSlot + k * 2048, C::kPanel, 1024),
                     id_o, !(first && k == 0));
      };
      for (;;) {
        const int n_tiles = (int)min((long long)(c.x.t1 - c.tile), c.left);
        const bool two = c.s.n * A.G - c.rt * kTM > 128;
        wait(&ctl->q_full, qi++ & 1);
        wait(&ctl->kv_full[g % S], (g / S) & 1);
        tc_fence_after();
        qk(0, g % S);
        if (two) qk(1, g % S);
        mma_commit(&ctl->kv_empty[g % S]);
        if (n_tiles == 1) mma_commit(&ctl->q_empty);
        for (int n = 0; n < n_tiles; ++n, g += 2) {
          const bool more = n + 1 < n_tiles;
          const uint32_t v = (g + 1) % S, k = (g + 2) % S;
          wait(&ctl->kv_full[v], ((g + 1) / S) & 1);
          pv(0, v, n == 0);
          if (!more) mma_commit(&ctl->o_full[0]);
          if (more) {
            wait(&ctl->kv_full[k], ((g + 2) / S) & 1);
            tc_fence_after();
            qk(0, k);
          }
          if (two) {
            pv(1, v, n == 0);
            if (!more) mma_commit(&ctl->o_full[1]);
          }
          mma_commit(&ctl->kv_empty[v]);
          if (more) {
            if (two) qk(1, k);
            mma_commit(&ctl->kv_empty[k]);
            if (n + 2 == n_tiles) mma_commit(&ctl->q_empty);
          }
        }
        c.tile += n_tiles - 1;
        c.left -= n_tiles - 1;
        if (!c.next(A, cls)) break;
      }
      mma_commit(&ctl->fin);  // every product and every commit's arrival is done before the block ends
      bar_wait(&ctl->fin, 0, P.err);
    }
    __syncwarp();
  }
  } else {
    // -------------------------------------------------------------- softmax
    if (FMT == SLORA_KV_16) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int wg = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + wg * 128, to = tmem + lanes + 256 + wg * 128;
    uint32_t sn = 0, on = 0, ti = 0;
    int segs = 0;
    for (;;) {
      const int n_tiles = (int)min((long long)(c.x.t1 - c.tile), c.left);
      const int r_item = c.rt * kTM, R = min(c.s.n * A.G - r_item, kTM);
      const bool whole_end = c.tile + n_tiles == c.x.t1;
      const bool complete = whole_end && c.tile == c.x.t0;
      const int slot = 2 * blockIdx.x + (segs > 0 ? 1 : 0);
      if (!whole_end && c.tile == c.x.t0 && tid == 0)
        note_split(split, c.b, c.h, c.rt, slot, u1 - c.left + (c.x.t1 - c.tile), total, ctas);
      if (wg == 0 || R > 128) {
        const int r = wg * 128 + (warp & 3) * 32 + lane;
        const int first = c.s.len - c.s.n;
        const int t = r < R ? (r_item + r) / A.G : 0;
        const int pos = r < R ? first + t : -1;
        const int low = A.window > 0 && r < R ? pos - A.window : -1;   // keys above it are seen
        const int pmin = first + (r_item + wg * 128) / A.G;            // of the first row of this q tile
        const int pmax = first + (r_item + R - 1) / A.G;
        float m = -INFINITY, l = 0.f, vn = 0.f, cr = A.c;
        for (int n = 0; n < n_tiles; ++n, ++ti) {
          wait(&ctl->s_full[wg], sn++ & 1);
          tc_fence_after();
          float s[kTK];
#pragma unroll
          for (int i = 0; i < kTK; i += 32) ld32(ts + i, s + i);
          if (FMT == SLORA_KV_E4M3 && n == 0) cr = qscale[(segs & 1) * kTM + r];
          wait_ld();
          if (FMT == SLORA_KV_E4M3) {
            const float* ks = scales + (ti & 3) * 2 * kTK;
#pragma unroll
            for (int i = 0; i < kTK; i += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(ks + i);
              s[i] *= k4.x;
              s[i + 1] *= k4.y;
              s[i + 2] *= k4.z;
              s[i + 3] *= k4.w;
            }
          }
          const int key0 = (c.tile + n) * kTK;
          const uint32_t any = ctl->any_bad[ti & 3][0] | ctl->any_bad[ti & 3][1] | ctl->any_bad[ti & 3][2];
          const bool masked = key0 + kTK - 1 > pmin || (A.window > 0 && key0 <= pmax - A.window) || any;
          if (masked) {
            const int hi = pos - key0, lo = low - key0;
#pragma unroll
            for (int i = 0; i < kTK; ++i)
              if (i > hi || i <= lo) s[i] = -INFINITY;
            if (any) {
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t bits = 0;
                for (int q = 0; q < kLoadWarps; ++q)
                  if (ctl->any_bad[ti & 3][q]) bits |= ctl->bad[ti & 3][q][w];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if ((bits >> i) & 1) s[w * 32 + i] = -INFINITY;
              }
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kTK; i += 4) {
            top[0] = fmaxf(top[0], s[i]);
            top[1] = fmaxf(top[1], s[i + 1]);
            top[2] = fmaxf(top[2], s[i + 2]);
            top[3] = fmaxf(top[3], s[i + 3]);
          }
          const float mn = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cr);
          float ratio = 1.f;
          bool raise = false;
          if (FMT == SLORA_KV_E4M3) {
            const float tv = fmaxf(fmaxf(ctl->vtop[ti & 3][0], ctl->vtop[ti & 3][1]), ctl->vtop[ti & 3][2]);
            if (n == 0) {
              vn = fmaxf(tv, 0x1p-126f);
            } else if (tv > 8.f * vn) {
              ratio = vn / tv;
              vn = tv;
              raise = true;
            }
          }
          if (__any_sync(FULL_MASK, mn > m + kSlack) || raise) {
            const float a = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            l *= a;
            if (n > 0) {
              const float f = a * ratio;
#pragma unroll
              for (int i = 0; i < D; i += 32) {
                float o[32];
                ld32(to + i, o);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= f;
                st32(to + i, o);
              }
            }
          }
          const float mz = m == -INFINITY ? 0.f : m;
          const float vinv = FMT == SLORA_KV_E4M3 ? __frcp_rn(vn) : 1.f;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < kTK; i += 32) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              float p[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                p[q] = ex2(fmaf(s[i + k + q], cr, -mz));
                ls[q] += p[q];
              }
              if (FMT == SLORA_KV_E4M3) {
                const float4 v4 = *reinterpret_cast<const float4*>(scales + (ti & 3) * 2 * kTK + kTK + i + k);
                const float f[4] = {v4.x * vinv, v4.y * vinv, v4.z * vinv, v4.w * vinv};
#pragma unroll
                for (int q = 0; q < 4; ++q) p[q] = masked && p[q] == 0.f ? 0.f : p[q] * f[q];  // a NaN scale of an unseen key stays out
              }
              w[k / 2] = pk2<MT>(p[0], p[1]);
              w[k / 2 + 1] = pk2<MT>(p[2], p[3]);
            }
            st16(ts + i / 2, w);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          wait_st();
          tc_fence_before();
          arrive(&ctl->p_full[wg]);
        }

        // ---- the rows of this item, or their partials
        wait(&ctl->o_full[wg], on++ & 1);
        tc_fence_after();
        const int hq = r < R ? c.h * A.G + (r_item + r) - t * A.G : 0;
        const int64_t tok = c.s.row0 + t;
        const float inv = inverse(l);
        uint16_t* const orow = A.out + tok * A.ldo + (int64_t)hq * D;
        float* const part = parts + (size_t)slot * slot_floats(kTM, D);
        float* const prow = part + (size_t)r * D;
        const float f = complete ? inv : 1.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          float o[32];
          ld32(to + i, o);
          wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (FMT == SLORA_KV_E4M3) o[k] *= vn;
            bad |= !isfinite(o[k]);
            o[k] *= f;
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
        if (r < R) {
          if (complete) {
            if (A.lse) A.lse[tok * A.Hq + hq] = lse_of(m, l);
          } else {
            part[(size_t)kTM * D + r] = m;
            part[(size_t)kTM * (D + 1) + r] = l;
          }
        }
        unsigned again = __ballot_sync(FULL_MASK, bad && r < R && m != -INFINITY);
        while (again) {
          __syncwarp();
          const int src = __ffs(again) - 1;
          again &= again - 1;
          const int r2 = wg * 128 + (warp & 3) * 32 + src;
          const int t2 = (r_item + r2) / A.G, hq2 = c.h * A.G + (r_item + r2) - t2 * A.G;
          const int64_t tok2 = c.s.row0 + t2;
          redo_row<DT, FMT, D>(A, c.b, c.h, A.q + tok2 * A.ldq + (int64_t)hq2 * D, first + t2,
                               max(c.tile * kTK, c.x.lo), min((c.tile + n_tiles) * kTK, c.x.hi),
                               __shfl_sync(FULL_MASK, m, src), __shfl_sync(FULL_MASK, inv, src),
                               complete ? A.out + tok2 * A.ldo + (int64_t)hq2 * D : nullptr, part + (size_t)r2 * D);
        }
      } else {
        ti += n_tiles;
      }
      ++segs;
      c.tile += n_tiles - 1;
      c.left -= n_tiles - 1;
      if (!c.next(A, cls)) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 11) tmem_dealloc(tmem, 512);
}

template <int DT, int FMT, int D>
cudaError_t run_chunk(const KvAttnDev& A, int sm_count, RowClass cls, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  static std::atomic<bool> sized[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_chunk<DT, FMT, D>), C::kSmem, sized);
  if (e != cudaSuccess) return e;
  k_kv_chunk<DT, FMT, D><<<sm_count, kNT, C::kSmem, st>>>(A, cls);
  const cudaError_t e2 = cudaGetLastError();
  return e2 != cudaSuccess ? e2 : launch_combine<DT, D, kTM>(A, sm_count, st);
}

}  // namespace

size_t kv_chunk_workspace(int D, int sm_count) {
  return (size_t)sm_count * sizeof(Split) + 2 * (size_t)sm_count * slot_floats(kTM, D) * 4;
}

cudaError_t launch_kv_chunk(const KvAttnDev& A, int dtype, int fmt, int D, int row_limit, int sm_count, cudaStream_t s) {
  const RowClass cls = {row_limit, INT32_MAX};
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

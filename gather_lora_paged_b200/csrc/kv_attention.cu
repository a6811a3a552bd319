// kv_attention.cu -- attention of each sequence's newest tokens over its KV
// pages, for few rows per kv head (decode, drafted tokens): a stream of the
// cache with the scores of one pass kept in registers.
//
// For query row i of a sequence (position p_i = kv_len - n + i) and query head
// hq reading kv head h = hq / G:
//     o_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = exp(scale * q_i . k_j),
//     j <= p_i and, with a window, j > p_i - window;
//     lse_i = log sum_j w_ij;  a row that sees no key gets 0 and -inf.
//
// The rows of a kv head are the n * G pairs (token, head of the group), in row
// tiles of 64.  A work item is (sequence, kv head, row tile); its keys come in
// tiles of 64, and the tiles of all items, laid out in one line, are cut into
// equal runs, one per CTA, so that ragged lengths and a single long sequence
// keep every SM equally busy.  An item inside one run is finished there; one that
// crosses runs leaves (max, sum, unnormalised row) partials, at most two per
// CTA, and k_kv_combine joins them in key order.  Sums and maxima are fp32.
//
// One CTA: 4 warps, two CTAs per SM.  K and V rows of a tile go to shared
// memory by 16-byte cp.async (the page of a key may be one token long, so a tile
// is gathered row by row), swizzled so that the fragment loads have no bank
// conflicts; kStages tiles are in flight and the page look-ups run one tile further
// ahead, across items.  Items of up to 16 rows give each warp 16 keys of a
// tile, up to 32 rows 32 keys, and beyond that each warp 16 rows and all keys; the warps'
// (max, sum, row) triples are joined at the item's end.  The products run on
// mma.sync m16n8k16: HBM bounds this kernel up to some 64 rows, and tiles this
// small do not fill tcgen05's 128 rows.
//
// e4m3: the fp16 tensor path takes the codes' exact fp16 values for both pool
// types; K's row scale multiplies the score, V's the weight w_ij, relative to the
// largest V scale met so far (the accumulator follows it as it follows the
// maximum).  A bf16 q enters as fp16 after a scaling of the row by a power of two to
// [1, 2): its 8 bits fit, and what falls below fp16's range is under 2^-25 of
// the row's largest element.
//
// Weights w are rounded for the tensor cores as w = hi + lo, two 16-bit
// halves: the second product costs little beside the stream and keeps the
// output within its own rounding.
//
// A key that a row does not see has weight 0, but 0 * inf is NaN: where a
// masked V row holds an infinity or a NaN, the rows that it spoiled are seen to be not
// finite at the end and are summed again key by key, without the masked keys.
#include <math.h>

#include <atomic>

#include "kv_attn.cuh"

namespace slora {
namespace {

constexpr int kNT = 128;      // threads
constexpr int kTK = 64;       // keys per tile
constexpr int kTM = 64;       // rows per row tile
constexpr int kMinRun = 2;    // tiles that are worth a CTA of their own
constexpr int kCtasPerSm = 2;

template <int FMT, int D>
struct Cfg {
  static constexpr int kRow = KvRow<FMT, D>::kBytes;
  static constexpr int kPart = kTK * kRow;                       // K or V rows of a tile
  static constexpr int kScales = FMT == SLORA_KV_E4M3 ? 2 * kTK * 4 : 0;
  static constexpr int kStage = 2 * kPart + kScales;
  static constexpr int kStages = FMT == SLORA_KV_16 ? (D == 128 ? 3 : 5) : (D == 128 ? 5 : 8);
  static constexpr int kMerge = 2 * 16 * D * 4;                  // two warps' rows
  static constexpr int kOffRing = kStages * kStage + kMerge;
  static constexpr int kOffMask = kOffRing + 2 * kTK * 4;
  static constexpr int kOffStat = kOffMask + (kStages + 2) * 8;
  static constexpr int kSmem = kOffStat + 2 * 16 * 2 * 4;
  static_assert(kSmem <= (233472 / kCtasPerSm) - 1024 - 128, "two CTAs per SM");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == SLORA_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, 1));
  return fmaxf(v, __shfl_xor_sync(FULL_MASK, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(FULL_MASK, v, 1);
  return v + __shfl_xor_sync(FULL_MASK, v, 2);
}

// Byte offset of 16-byte chunk c of tile row j (a key).  The rows of an 8-row
// fragment load fall into 8 different 16-byte bank groups.
template <int FMT, int D>
__device__ __forceinline__ uint32_t place(int j, int c) {
  if (FMT == SLORA_KV_16) return j * 2 * D + ((c ^ (j & 7)) << 4);
  if (D == 128) return j * D + ((c ^ (((j & 1) << 2) | ((j >> 1) & 3))) << 4);
  return j * D + ((c ^ ((j >> 1) & 3)) << 4);
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kNT, kCtasPerSm) k_kv_stream(const __grid_constant__ KvAttnDev A, RowClass cls) {
  using C = Cfg<FMT, D>;
  constexpr int MT = FMT == SLORA_KV_16 ? DT : SLORA_F16;  // operand type of the products
  constexpr int NB = D / 8;                                 // 8-column blocks of the output
  constexpr int KS = D / 16;                                // k steps of the score product
  constexpr int S = C::kStages;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* const merge = smem + S * C::kStage;
  uint32_t* const ring = reinterpret_cast<uint32_t*>(smem + C::kOffRing);
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + C::kOffMask);
  float* const stat = reinterpret_cast<float*>(smem + C::kOffStat);
  const KvDev& P = A.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = lane >> 2, ql = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  Split* const split = reinterpret_cast<Split*>(A.workspace) + blockIdx.x;
  float* const parts = reinterpret_cast<float*>(reinterpret_cast<Split*>(A.workspace) + gridDim.x);

  if (tid == 0) split->n = 0;
  if (blockIdx.x == 0) kv_record_bad(P, A.max_rows);

  // ---- this CTA's run of tiles
  Cursor<kTM, kTK> pc;
  long long total, u1;
  int ctas;
  if (!find_run<kTM, kTK, kNT>(A, cls, kMinRun, reinterpret_cast<long long*>(smem), pc, total, ctas, u1)) return;
  Cursor<kTM, kTK> cc = pc;
  const int n_tiles = (int)pc.left;

  // ---- producer side: row numbers of tile i (ring), then its copies
  const int vstep = P.H * P.pt;
  auto fetch = [&](int i) -> int {  // threads 0..63: page id of key `tid` of the tile at pc
    if (i >= n_tiles || tid >= kTK) return -1;
    const int j = pc.tile * kTK + tid;
    return j >= pc.x.lo && j < pc.x.hi ? __ldg(P.blocks + (int64_t)pc.b * P.ldb + j / P.pt) : -1;
  };
  auto resolve = [&](int i, int pg) {
    if (i < n_tiles) {
      if (tid < kTK) {
        const int j = pc.tile * kTK + tid;
        uint32_t r = kNoRow;
        if (j >= pc.x.lo && j < pc.x.hi) {
          if (pg >= 0 && pg < P.n_pages) r = ((uint32_t)pg << P.row_shift) + (uint32_t)(pc.h * P.pt + j % P.pt);
          else record_error(P.err, kErrKvPage, pc.b);
        }
        ring[(i & 1) * kTK + tid] = r;
        const unsigned m = __ballot_sync(FULL_MASK, r != kNoRow);
        if (lane == 0) masks[(i % (S + 2)) * 2 + warp] = m;
      }
      pc.next(A, cls);
    }
  };
  auto copy = [&](int i) {
    if (i < n_tiles) {
      constexpr int CH = C::kRow / 16;            // 16-byte chunks per row
      constexpr int RPP = kNT / CH;               // rows per pass
      const uint32_t st = sbase + (i % S) * C::kStage;
      const unsigned char* base = reinterpret_cast<const unsigned char*>(P.pool);
      const int c = tid % CH;
#pragma unroll
      for (int k = 0; k < kTK / RPP; ++k) {
        const int j = k * RPP + tid / CH;
        const uint32_t r = ring[(i & 1) * kTK + j];
        const bool real = r != kNoRow;
        const unsigned char* src = base + (real ? (int64_t)r * C::kRow + c * 16 : 0);
        cp16(st + place<FMT, D>(j, c), src, real);
        cp16(st + C::kPart + place<FMT, D>(j, c), src + (real ? (int64_t)vstep * C::kRow : 0), real);
      }
      if (FMT == SLORA_KV_E4M3) {
        const uint32_t r = ring[(i & 1) * kTK + (tid & 63)];
        const bool real = r != kNoRow;
        cp4(st + 2 * C::kPart + tid * 4, real ? kv_scale(P, r + (tid < 64 ? 0 : vstep)) : reinterpret_cast<float*>(P.pool),
            real);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  resolve(0, fetch(0));
  __syncthreads();
  for (int i = 0; i < S - 1; ++i) {
    const int pg = fetch(i + 1);
    copy(i);
    resolve(i + 1, pg);
    __syncthreads();
  }

  // ---- consumer side
  uint32_t qf[KS][4];
  float o[NB][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, vn = 0.f, c0 = 0.f, c1 = 0.f;
  int p0 = -1, p1 = -1, MG = 1, KG = 4, rg = 0, kg = warp, R = 0;
  int seg_tile = 0;       // first tile of the item in this run
  int segs = 0;           // items of this run before this one
  bool fresh = true;

  for (int i = 0; i < n_tiles; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
    __syncthreads();
    const int pg_ahead = fetch(i + S);  // arrives during this tile's products
    copy(i + S - 1);

    if (fresh) {  // a new item: its rows, positions and q fragments
      fresh = false;
      seg_tile = cc.tile;
      const int r_item = cc.rt * kTM;
      R = min(cc.s.n * A.G - r_item, kTM);
      MG = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
      KG = 4 / MG;
      rg = warp / KG;
      kg = warp % KG;
      m0 = m1 = -INFINITY;
      l0 = l1 = vn = 0.f;
      c0 = c1 = A.c;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) o[nb][0] = o[nb][1] = o[nb][2] = o[nb][3] = 0.f;
      const int ra = rg * 16 + quad, rb = ra + 8;
      const int ta = (r_item + ra) / A.G, tb = (r_item + rb) / A.G;
      p0 = ra < R ? cc.s.len - cc.s.n + ta : -1;
      p1 = rb < R ? cc.s.len - cc.s.n + tb : -1;
      const uint16_t* qa = A.q + (int64_t)(cc.s.row0 + ta) * A.ldq + (int64_t)(cc.h * A.G + (r_item + ra) - ta * A.G) * D;
      const uint16_t* qb = A.q + (int64_t)(cc.s.row0 + tb) * A.ldq + (int64_t)(cc.h * A.G + (r_item + rb) - tb * A.G) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (FMT == SLORA_KV_16) {
          const int d = ks * 16 + ql * 2;
          qf[ks][0] = ra < R ? __ldg(reinterpret_cast<const uint32_t*>(qa + d)) : 0;
          qf[ks][1] = rb < R ? __ldg(reinterpret_cast<const uint32_t*>(qb + d)) : 0;
          qf[ks][2] = ra < R ? __ldg(reinterpret_cast<const uint32_t*>(qa + d + 8)) : 0;
          qf[ks][3] = rb < R ? __ldg(reinterpret_cast<const uint32_t*>(qb + d + 8)) : 0;
        } else {  // the k order of the code fragments: 16 codes of a lane's chunk in turn
          const int d = (ks >> 2) * 64 + ql * 16 + (ks & 3) * 4;
          const uint2 z = make_uint2(0, 0);
          const uint2 a = ra < R ? __ldg(reinterpret_cast<const uint2*>(qa + d)) : z;
          const uint2 b = rb < R ? __ldg(reinterpret_cast<const uint2*>(qb + d)) : z;
          qf[ks][0] = a.x;
          qf[ks][1] = b.x;
          qf[ks][2] = a.y;
          qf[ks][3] = b.y;
        }
      }
      if (FMT == SLORA_KV_E4M3 && DT == SLORA_BF16) {  // bf16 rows -> fp16 in [1, 2) * 2^e
        uint32_t ta_ = 0, tb_ = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          ta_ = max(max(ta_, qf[ks][0] & 0x7fffu), max((qf[ks][0] >> 16) & 0x7fffu, max(qf[ks][2] & 0x7fffu, (qf[ks][2] >> 16) & 0x7fffu)));
          tb_ = max(max(tb_, qf[ks][1] & 0x7fffu), max((qf[ks][1] >> 16) & 0x7fffu, max(qf[ks][3] & 0x7fffu, (qf[ks][3] >> 16) & 0x7fffu)));
        }
        ta_ = max(ta_, __shfl_xor_sync(FULL_MASK, ta_, 1));
        ta_ = max(ta_, __shfl_xor_sync(FULL_MASK, ta_, 2));
        tb_ = max(tb_, __shfl_xor_sync(FULL_MASK, tb_, 1));
        tb_ = max(tb_, __shfl_xor_sync(FULL_MASK, tb_, 2));
        // exponents in [-100, 126]; an infinite or NaN row stays so
        const int ea = min(max((int)(ta_ >> 7) - 127, -100), 126), eb = min(max((int)(tb_ >> 7) - 127, -100), 126);
        const float fa = __int_as_float((127 - ea) << 23), fb = __int_as_float((127 - eb) << 23);
        c0 = A.c * __int_as_float((127 + ea) << 23);
        c1 = A.c * __int_as_float((127 + eb) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float f = (w & 1) ? fb : fa;
            qf[ks][w] = pack2<SLORA_F16>(__uint_as_float(qf[ks][w] << 16) * f, __uint_as_float(qf[ks][w] & 0xffff0000u) * f);
          }
      }
    }

    const uint32_t st = sbase + (i % S) * C::kStage;
    const uint32_t* mk = masks + (i % (S + 2)) * 2;
    // every row sees every key of the tile
    const int key0 = cc.tile * kTK;
    const int first = cc.s.len - cc.s.n + cc.rt * kTM / A.G;
    const bool open = (mk[0] & mk[1]) == FULL_MASK && key0 + kTK - 1 <= first &&
                      (A.window <= 0 || key0 > cc.s.len - A.window - 1);
    for (int kb = kg; kb < kTK / 16; kb += KG) {
      // scores of 16 keys: s[n][..], n8 blocks of keys kb*16 + 8n
      float s[2][4] = {};
      if (FMT == SLORA_KV_16) {
        const int j = kb * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t r[4];
          ldm4(r, st + place<FMT, D>(j, ks * 2 + ((lane >> 3) & 1)));
          mma<MT>(s[0], qf[ks], r[0], r[1]);
          mma<MT>(s[1], qf[ks], r[2], r[3]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int hh = 0; hh < KS / 4; ++hh) {
            const int j = kb * 16 + n * 8 + quad;
            const uint4 w = *reinterpret_cast<const uint4*>(smem + (st - sbase) + place<FMT, D>(j, hh * 4 + ql));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma<MT>(s[n], qf[hh * 4 + k], e4m3x2_f16x2(ww[k]), e4m3x2_f16x2(ww[k] >> 16));
          }
      }
      float vs[2][2];
      const int jb = kb * 16 + ql * 2;  // this lane's keys: jb, jb + 1, jb + 8, jb + 9
      if (FMT == SLORA_KV_E4M3) {
        const float* sc = reinterpret_cast<const float*>(smem + (st - sbase) + 2 * C::kPart);
        float top = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float2 ksc = *reinterpret_cast<const float2*>(sc + jb + 8 * n);
          const float2 vsc = *reinterpret_cast<const float2*>(sc + kTK + jb + 8 * n);
          vs[n][0] = vsc.x;
          vs[n][1] = vsc.y;
          top = fmaxf(top, fmaxf(vsc.x, vsc.y));  // a NaN scale is passed over here
          s[n][0] *= ksc.x * c0;
          s[n][1] *= ksc.y * c0;
          s[n][2] *= ksc.x * c1;
          s[n][3] *= ksc.y * c1;
        }
        top = quad_max(top);
        if (top > vn) {  // uniform in the warp: the four lanes of a quad hold all 16 keys
          const float r = vn / top;
          vn = top;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            o[nb][0] *= r;
            o[nb][1] *= r;
            o[nb][2] *= r;
            o[nb][3] *= r;
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          s[n][0] *= c0;
          s[n][1] *= c0;
          s[n][2] *= c1;
          s[n][3] *= c1;
        }
      }
      uint32_t vis0 = 0xf, vis1 = 0xf;  // visibility of this lane's four keys for its two rows
      if (!open) {
        const uint32_t word = mk[kb >> 1] >> ((kb & 1) * 16);
        vis0 = vis1 = 0;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = key0 + jb + 8 * n + e;
            const bool have = (word >> (ql * 2 + 8 * n + e)) & 1;
            const bool a = have && j <= p0 && (A.window <= 0 || j > p0 - A.window);
            const bool b = have && j <= p1 && (A.window <= 0 || j > p1 - A.window);
            if (!a) s[n][e] = -INFINITY;
            if (!b) s[n][2 + e] = -INFINITY;
            vis0 |= (uint32_t)a << (2 * n + e);
            vis1 |= (uint32_t)b << (2 * n + e);
          }
      }
      const float x0 = fmaxf(m0, quad_max(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]))));
      const float x1 = fmaxf(m1, quad_max(fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))));
      const float z0 = x0 == -INFINITY ? 0.f : x0, z1 = x1 == -INFINITY ? 0.f : x1;
      if (__any_sync(FULL_MASK, x0 > m0 || x1 > m1)) {
        const float a0 = ex2(m0 - z0), a1 = ex2(m1 - z1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          o[nb][0] *= a0;
          o[nb][1] *= a0;
          o[nb][2] *= a1;
          o[nb][3] *= a1;
        }
        m0 = x0;
        m1 = x1;
      }
      float w[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        w[n][0] = ex2(s[n][0] - z0);
        w[n][1] = ex2(s[n][1] - z0);
        w[n][2] = ex2(s[n][2] - z1);
        w[n][3] = ex2(s[n][3] - z1);
        l0 += w[n][0] + w[n][1];
        l1 += w[n][2] + w[n][3];
      }
      if (FMT == SLORA_KV_E4M3) {
        const float inv = vn > 0.f ? __frcp_rn(fmaxf(vn, 0x1p-126f)) : 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = vs[n][e] * inv;  // NaN scales of unseen keys stay out
            w[n][e] = (vis0 >> (2 * n + e)) & 1 ? w[n][e] * f : 0.f;
            w[n][2 + e] = (vis1 >> (2 * n + e)) & 1 ? w[n][2 + e] * f : 0.f;
          }
      }
      uint32_t hi[4], lo[4];  // A fragments: rows (quad, quad + 8) x keys (2ql, 2ql + 8)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float a = w[n][2 * r], b = w[n][2 * r + 1];
          const uint32_t u = pack2<MT>(a, b);
          float ha, hb;
          if (MT == SLORA_BF16) {
            ha = __uint_as_float(u << 16);
            hb = __uint_as_float(u & 0xffff0000u);
          } else {
            h2x2f(u, ha, hb);
          }
          hi[2 * n + r] = u;
          lo[2 * n + r] = pack2<MT>(a - ha, b - hb);
        }
      const uint32_t sv = st + C::kPart;
      if (FMT == SLORA_KV_16) {
        const int j = kb * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int nb = 0; nb < NB; nb += 2) {
          uint32_t r[4];
          ldm4t(r, sv + place<FMT, D>(j, nb + (lane >> 4)));
          mma<MT>(o[nb], hi, r[0], r[1]);
          mma<MT>(o[nb], lo, r[0], r[1]);
          mma<MT>(o[nb + 1], hi, r[2], r[3]);
          mma<MT>(o[nb + 1], lo, r[2], r[3]);
        }
      } else {
        // 16-bit transposing loads bring pairs of codes (d, d + 1) of a key: blocks
        // nb and nb + 1 take the even and the odd d of 16
        const int j = kb * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int nb = 0; nb < NB; nb += 4) {
          uint32_t r[4];
          ldm4t(r, sv + place<FMT, D>(j, (nb >> 1) + (lane >> 4)));
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint32_t a = __byte_perm(r[2 * g], 0, 0x3120), b = __byte_perm(r[2 * g + 1], 0, 0x3120);
            const uint32_t ea = e4m3x2_f16x2(a), eb = e4m3x2_f16x2(b);
            const uint32_t oa = e4m3x2_f16x2(a >> 16), ob = e4m3x2_f16x2(b >> 16);
            mma<MT>(o[nb + 2 * g], hi, ea, eb);
            mma<MT>(o[nb + 2 * g], lo, ea, eb);
            mma<MT>(o[nb + 2 * g + 1], hi, oa, ob);
            mma<MT>(o[nb + 2 * g + 1], lo, oa, ob);
          }
        }
      }
    }

    resolve(i + S, pg_ahead);

    // ---- the end of the item, or of this run
    const bool whole_end = cc.last_of_item();
    if (whole_end || cc.left == 1) {
      fresh = true;
      if (FMT == SLORA_KV_E4M3) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          o[nb][0] *= vn;
          o[nb][1] *= vn;
          o[nb][2] *= vn;
          o[nb][3] *= vn;
        }
      }
      l0 = quad_sum(l0);
      l1 = quad_sum(l1);
      // join the key groups of a row group: kg 2, 3 into 0, 1, then 1 into 0
      for (int half = KG / 2; half >= 1; half /= 2) {
        const int buf = MG == 1 ? kg & (half - 1) : rg;
        float* const mb = reinterpret_cast<float*>(merge) + buf * 16 * D;
        float* const sb = stat + buf * 32;
        if (kg >= half && kg < 2 * half) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) *reinterpret_cast<float4*>(mb + (nb * 32 + lane) * 4) = make_float4(o[nb][0], o[nb][1], o[nb][2], o[nb][3]);
          if (ql == 0) {
            sb[quad] = m0;
            sb[quad + 8] = m1;
            sb[16 + quad] = l0;
            sb[16 + quad + 8] = l1;
          }
        }
        __syncthreads();
        if (kg < half) {
          const float y0 = sb[quad], y1 = sb[quad + 8], k0 = sb[16 + quad], k1 = sb[16 + quad + 8];
          const float x0 = fmaxf(m0, y0), x1 = fmaxf(m1, y1);
          const float z0 = x0 == -INFINITY ? 0.f : x0, z1 = x1 == -INFINITY ? 0.f : x1;
          const float a0 = ex2(m0 - z0), b0 = ex2(y0 - z0), a1 = ex2(m1 - z1), b1 = ex2(y1 - z1);
          l0 = l0 * a0 + k0 * b0;
          l1 = l1 * a1 + k1 * b1;
          m0 = x0;
          m1 = x1;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const float4 y = *reinterpret_cast<const float4*>(mb + (nb * 32 + lane) * 4);
            o[nb][0] = o[nb][0] * a0 + y.x * b0;
            o[nb][1] = o[nb][1] * a0 + y.y * b0;
            o[nb][2] = o[nb][2] * a1 + y.z * b1;
            o[nb][3] = o[nb][3] * a1 + y.w * b1;
          }
        }
        if (half > 1) __syncthreads();
      }
      const bool complete = whole_end && seg_tile == cc.x.t0;
      const int slot = 2 * blockIdx.x + (segs > 0 ? 1 : 0);
      if (!whole_end && seg_tile == cc.x.t0 && tid == 0) {
        note_split(split, cc.b, cc.h, cc.rt, slot, u1 - cc.left + (cc.x.t1 - cc.tile), total, ctas);
      }
      ++segs;
      if (kg == 0) {
        float* const part = parts + (size_t)slot * slot_floats(kTM, D);
        const float i0 = inverse(l0), i1 = inverse(l1);
        bool bad0 = false, bad1 = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          bad0 |= !isfinite(o[nb][0]) || !isfinite(o[nb][1]);
          bad1 |= !isfinite(o[nb][2]) || !isfinite(o[nb][3]);
        }
        const int r_item = cc.rt * kTM;
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const int r = rg * 16 + quad + 8 * rr;
          if (r < R) {
            const int t = (r_item + r) / A.G, hq = cc.h * A.G + (r_item + r) - t * A.G;
            const int64_t tok = cc.s.row0 + t;
            const float l = rr ? l1 : l0, m = rr ? m1 : m0, inv = rr ? i1 : i0;
            uint16_t* const orow = A.out + tok * A.ldo + (int64_t)hq * D;
            float* const prow = part + (size_t)r * D;
            if (complete) {
              if (FMT == SLORA_KV_16) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  *reinterpret_cast<uint32_t*>(orow + nb * 8 + ql * 2) = pack2<DT>(o[nb][2 * rr] * inv, o[nb][2 * rr + 1] * inv);
              } else {
#pragma unroll
                for (int nb = 0; nb < NB; nb += 2)
                  *reinterpret_cast<uint2*>(orow + nb * 8 + ql * 4) =
                      make_uint2(pack2<DT>(o[nb][2 * rr] * inv, o[nb + 1][2 * rr] * inv),
                                 pack2<DT>(o[nb][2 * rr + 1] * inv, o[nb + 1][2 * rr + 1] * inv));
              }
              if (A.lse && ql == 0) A.lse[tok * A.Hq + hq] = lse_of(m, l);
            } else {
              if (FMT == SLORA_KV_16) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  *reinterpret_cast<float2*>(prow + nb * 8 + ql * 2) = make_float2(o[nb][2 * rr], o[nb][2 * rr + 1]);
              } else {
#pragma unroll
                for (int nb = 0; nb < NB; nb += 2)
                  *reinterpret_cast<float4*>(prow + nb * 8 + ql * 4) =
                      make_float4(o[nb][2 * rr], o[nb + 1][2 * rr], o[nb][2 * rr + 1], o[nb + 1][2 * rr + 1]);
              }
              if (ql == 0) {
                part[(size_t)kTM * D + r] = m;
                part[(size_t)kTM * (D + 1) + r] = l;
              }
            }
          }
        }
        // rows that are not finite: once more without the keys that they do not see
        const unsigned f0 = __ballot_sync(FULL_MASK, bad0), f1 = __ballot_sync(FULL_MASK, bad1);
        if (f0 | f1) {
          __syncwarp();
          for (int r16 = 0; r16 < 16; ++r16) {
            const unsigned f = r16 < 8 ? f0 : f1;
            const float m = __shfl_sync(FULL_MASK, r16 < 8 ? m0 : m1, (r16 & 7) * 4);
            const float inv = __shfl_sync(FULL_MASK, r16 < 8 ? i0 : i1, (r16 & 7) * 4);
            const int r = rg * 16 + r16;
            if (r >= R || !((f >> ((r16 & 7) * 4)) & 0xf) || m == -INFINITY) continue;
            const int t = (r_item + r) / A.G, hq = cc.h * A.G + (r_item + r) - t * A.G;
            const int64_t tok = cc.s.row0 + t;
            redo_row<DT, FMT, D>(A, cc.b, cc.h, A.q + tok * A.ldq + (int64_t)hq * D, cc.s.len - cc.s.n + t,
                                 max(seg_tile * kTK, cc.x.lo), min((cc.tile + 1) * kTK, cc.x.hi), m, inv,
                                 complete ? A.out + tok * A.ldo + (int64_t)hq * D : nullptr, part + (size_t)r * D);
          }
        }
      }
    }
    cc.next(A, cls);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int DT, int FMT, int D>
cudaError_t run_stream(const KvAttnDev& A, int sm_count, RowClass cls, cudaStream_t st) {
  using C = Cfg<FMT, D>;
  const int grid = sm_count * kCtasPerSm;
  static std::atomic<bool> sized[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k_kv_stream<DT, FMT, D>), C::kSmem, sized);
  if (e != cudaSuccess) return e;
  k_kv_stream<DT, FMT, D><<<grid, kNT, C::kSmem, st>>>(A, cls);
  const cudaError_t e2 = cudaGetLastError();
  return e2 != cudaSuccess ? e2 : launch_combine<DT, D, kTM>(A, grid, st);
}

}  // namespace

size_t kv_stream_workspace(int D, int sm_count) {
  const size_t ctas = (size_t)sm_count * kCtasPerSm;
  return ctas * sizeof(Split) + 2 * ctas * slot_floats(kTM, D) * 4;
}

cudaError_t launch_kv_stream(const KvAttnDev& A, int dtype, int fmt, int D, int row_limit, int sm_count, cudaStream_t s) {
  const RowClass cls = {0, row_limit};
  if (D == 128) {
    if (dtype == SLORA_F16)
      return fmt == SLORA_KV_16 ? run_stream<SLORA_F16, SLORA_KV_16, 128>(A, sm_count, cls, s)
                                : run_stream<SLORA_F16, SLORA_KV_E4M3, 128>(A, sm_count, cls, s);
    return fmt == SLORA_KV_16 ? run_stream<SLORA_BF16, SLORA_KV_16, 128>(A, sm_count, cls, s)
                              : run_stream<SLORA_BF16, SLORA_KV_E4M3, 128>(A, sm_count, cls, s);
  }
  if (dtype == SLORA_F16)
    return fmt == SLORA_KV_16 ? run_stream<SLORA_F16, SLORA_KV_16, 64>(A, sm_count, cls, s)
                              : run_stream<SLORA_F16, SLORA_KV_E4M3, 64>(A, sm_count, cls, s);
  return fmt == SLORA_KV_16 ? run_stream<SLORA_BF16, SLORA_KV_16, 64>(A, sm_count, cls, s)
                            : run_stream<SLORA_BF16, SLORA_KV_E4M3, 64>(A, sm_count, cls, s);
}

}  // namespace slora

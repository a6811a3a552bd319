// kv_attn.cuh -- what the attention kernels share (kv_decode.cu,
// kv_chunk.cu): the line of key tiles that is cut into one run per CTA, the
// join of the partials, V's values that are not finite.
//
// The rows of a kv head are the n * G pairs (token, head of the group), in row
// tiles of TM.  A work item is (sequence, kv head, row tile); its keys come in
// tiles of TK.  All items, laid out in one line, are cut into equal runs, one per CTA, so
// that ragged lengths and a single long sequence keep every SM equally busy.  An item is as long there as
// its tiles and a lead of E units, for what it costs beside them (q, the first maximum, its
// outputs).  An item inside one run is finished there; one that
// crosses runs leaves (reference, sum, row) partials, at most two per
// CTA, each row divided by its own sum, so that it is no larger than V; k_kv_join joins them in key order.
//
// The products meet all V rows of a tile, also those that some rows of the item do not see: with weight 0,
// but 0 * inf is NaN.  So in tiles that cross an item's causal or window border the values of such keys that are not
// finite are set to zero in shared memory before the products, and the item is marked (Item::odd).  Whatever
// the values of V and the weights, no finite term overflows (the kernels' references see to that), so a sum that
// is not finite comes from a value that is not: for such rows, and for those of marked items, settle() looks
// up the keys that the row sees, and an output element with infinities of one sign becomes that infinity, one with
// both signs or a NaN a NaN, whatever the products' pieces made of them.  It reads V once per warp and item.
#pragma once

#include <atomic>

#include "kv_common.cuh"

namespace slora {
namespace {

// Lets a kernel have its dynamic shared memory, once per device.
inline cudaError_t allow_smem(const void* kern, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load()) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true);
  return e;
}

constexpr float kLn2 = 0.69314718055994531f;

// Token of a row of a kv head.
__device__ __forceinline__ int token_of(const KvAttnDev& A, int row) {
  return (int)(((uint64_t)(uint32_t)row * A.g_mul) >> A.g_shift);
}

// The sequences a kernel takes: those with row_lo < rows per kv head <= row_hi.
struct RowClass {
  int lo, hi;
};

// A split item, written by the CTA whose run holds its first tile.
struct Split {
  int b, h, rt, slot;  // the first partial; the others are the even slots of the next CTAs
  int n;               // partials (0: none)
  int pad[3];
};

__host__ __device__ inline size_t slot_floats(int TM, int D) { return (size_t)TM * (D + 2); }

struct Span {
  int lo, hi;       // keys some row of the tile sees
  int t0, t1;       // key tiles (at least one)
};

// Keys of rows [rt * TM, ...) of a sequence.
template <int TM, int TK>
__device__ __forceinline__ Span span_of(const KvAttnDev& A, const KvSeq& s, int rt) {
  const int R = s.n * A.G, r0 = rt * TM, r1 = min(R, r0 + TM) - 1;
  const int first = s.len - s.n;
  Span x;
  x.hi = max(0, first + token_of(A, r1) + 1);
  x.lo = A.window > 0 ? max(0, first + token_of(A, r0) - A.window + 1) : 0;
  x.t0 = x.lo / TK;
  x.t1 = max(x.t0 + 1, (x.hi + TK - 1) / TK);
  return x;
}
__device__ __forceinline__ bool takes(const KvAttnDev& A, RowClass cls, int b, KvSeq& s) {
  if (!kv_seq(A.kv, b, A.max_rows, s)) return false;
  const int64_t R = (int64_t)s.n * A.G;
  return R > cls.lo && R <= cls.hi;
}
// Units of all items of sequence b: the lead of an item and its tiles.
template <int TM, int TK, int E>
__device__ __forceinline__ long long seq_units(const KvAttnDev& A, RowClass cls, int b) {
  KvSeq s;
  if (!takes(A, cls, b, s)) return 0;
  const int RT = cdiv_i(s.n * A.G, TM);
  long long u = 0;
  for (int rt = 0; rt < RT; ++rt) {
    const Span x = span_of<TM, TK>(A, s, rt);
    u += E + x.t1 - x.t0;
  }
  return u * A.kv.H;
}

// A place in the line.
template <int TM, int TK, int E>
struct Cursor {
  KvSeq s;
  Span x;
  int b, h, rt, RT, at;  // at: units of the item before this place
  long long left;        // units of this run from here on

  __device__ int size() const { return E + x.t1 - x.t0; }
  __device__ void seek(const KvAttnDev& A, RowClass cls, int b_, long long off) {
    b = b_;
    takes(A, cls, b, s);
    RT = cdiv_i(s.n * A.G, TM);
    long long per = 0;
    for (rt = 0; rt < RT; ++rt) {
      x = span_of<TM, TK>(A, s, rt);
      per += size();
    }
    h = off < (1ll << 31) && per < (1ll << 31) ? (int)((uint32_t)off / (uint32_t)per) : (int)(off / per);
    off -= h * per;
    for (rt = 0;; ++rt) {
      x = span_of<TM, TK>(A, s, rt);
      if (off < size()) break;
      off -= size();
    }
    at = (int)off;
  }
  __device__ bool next(const KvAttnDev& A, RowClass cls) {  // to the next item; false: no tile of it is in the run
    left -= size() - at;
    if (left <= E) return false;
    at = 0;
    if (++rt == RT) {
      rt = 0;
      if (++h == A.kv.H) {
        h = 0;
        do ++b;
        while (b < A.kv.B && !takes(A, cls, b, s));
        if (b >= A.kv.B) return false;  // cannot be: the run ends first
        RT = cdiv_i(s.n * A.G, TM);
      }
    }
    x = span_of<TM, TK>(A, s, rt);
    return true;
  }
};

// The cut of the line: runs of q + 1 units, `rem` of them, then runs of q.
struct Cut {
  long long q, u1;  // u1: the end of this CTA's run
  int rem;
  __device__ long long start(int run) const { return run * q + min(run, rem); }
  __device__ int run_of(long long unit) const {
    const long long edge = rem * (q + 1), x = unit < edge ? unit : unit - edge, d = unit < edge ? q + 1 : q;
    const int i = x < (1ll << 32) && d < (1ll << 32) ? (int)((uint32_t)x / (uint32_t)d) : (int)(x / d);
    return unit < edge ? i : rem + i;
  }
};

// This CTA's run of the line, found by one warp (some 400 instructions: 20 warps of a CTA that all
// went through them spent 4500 cycles), a lane adding up some neighbouring
// sequences.  Runs are at least E + min_tiles units, so that each has a tile.
// False: this CTA has none.
template <int TM, int TK, int E>
__device__ __forceinline__ bool find_run(const KvAttnDev& A, RowClass cls, int min_tiles, Cursor<TM, TK, E>& c, Cut& cut) {
  const int lane = threadIdx.x & 31, B = A.kv.B, per = (B + 31) >> 5, b0 = lane * per;
  long long mine = 0;
#pragma unroll 4
  for (int i = 0; i < per; ++i)
    if (b0 + i < B) mine += seq_units<TM, TK, E>(A, cls, b0 + i);
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(FULL_MASK, inc, o);
    if (lane >= o) inc += y;
  }
  const long long total = __shfl_sync(FULL_MASK, inc, 31);
  const bool small = total < (1ll << 31);
  const long long most = small ? (uint32_t)total / (uint32_t)(E + min_tiles) : total;
  const int ctas = max((int)min((long long)gridDim.x, most), total > 0 ? 1 : 0), run = blockIdx.x;
  if (run >= ctas) return false;
  cut.q = small ? (uint32_t)total / (uint32_t)ctas : total / ctas;
  cut.rem = (int)(total - cut.q * ctas);
  const long long u0 = cut.start(run);
  cut.u1 = cut.start(run + 1);
  // the sequence that holds unit u0 (there is one: u0 < total)
  long long off = u0 - (inc - mine);
  const int src = __ffs(__ballot_sync(FULL_MASK, off >= 0 && off < mine)) - 1;
  int b = b0;
  if (lane == src && per > 1) {
    for (;; ++b) {
      const long long w = seq_units<TM, TK, E>(A, cls, b);
      if (off < w) break;
      off -= w;
    }
  }
  c.seek(A, cls, __shfl_sync(FULL_MASK, b, src), __shfl_sync(FULL_MASK, off, src));
  c.left = cut.u1 - u0;
  return true;
}

// What a run has to do, one entry per item, written by one warp for the others.
struct Item {
  int b, h, rt, R;        // sequence, kv head, row tile, rows
  int row0, first;        // the sequence's first row and that row's position
  int lo, hi;             // keys some row sees
  int tile, n_tiles;      // this run's tiles of the item
  int flags;              // 1: it starts here, 2: it ends here, 4: the run's last
  int odd;                // a V row that some rows see and others do not held values that are not finite
  int shut, late;         // keys above `shut`, or at `late` and below, are not seen by all rows
  int open0, open1;       // which need no looking at: of this run's tiles, those in [open0, open1)
};

constexpr int kNever = -(1 << 30);  // below every position, and that less a position is a number

template <int TM, int TK, int E>
__device__ __forceinline__ Item item_of(const KvAttnDev& A, const Cursor<TM, TK, E>& c) {
  const int end = (int)min((long long)c.size(), c.at + c.left), first = max(c.at - E, 0);
  Item x;
  x.b = c.b;
  x.h = c.h;
  x.rt = c.rt;
  x.R = min(c.s.n * A.G - c.rt * TM, TM);
  x.row0 = c.s.row0;
  x.first = c.s.len - c.s.n;
  x.lo = c.x.lo;
  x.hi = c.x.hi;
  x.tile = c.x.t0 + first;
  x.n_tiles = end - E - first;
  x.flags = (first == 0 ? 1 : 0) | (end == c.size() ? 2 : 0) | (c.left - (end - c.at) <= E ? 4 : 0);
  x.odd = 0;
  x.shut = x.first + token_of(A, x.rt * TM);
  x.late = A.window > 0 ? x.first + token_of(A, x.rt * TM + x.R - 1) - A.window : kNever;
  x.open0 = (x.late >> 7) + 1 - x.tile;
  x.open1 = x.hi - 1 <= x.shut ? INT32_MAX : ((x.shut + 1) >> 7) - x.tile;
  static_assert(TK == 128, "the shifts");
  return x;
}

// Partials of the item at c, whose first tile is in this run (slot: this CTA's).
template <int TM, int TK, int E>
__device__ __forceinline__ void note_split(Split* sp, const Cursor<TM, TK, E>& c, const Cut& cut, int slot) {
  sp->b = c.b;
  sp->h = c.h;
  sp->rt = c.rt;
  sp->slot = slot;
  sp->n = cut.run_of(cut.u1 - c.left + (c.size() - c.at) - 1) - (int)blockIdx.x + 1;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2; }
// 2^e, for a constant e.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((127 + e) << 23); }
// 1 / sum, 0 for a row without keys (a NaN sum stays NaN).
__device__ __forceinline__ float inverse(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }

// ---- values of V that are not finite

// 16-bit values (of type DT), or e4m3 codes, with those that are not finite set to zero.
template <bool CODES, int DT>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if (CODES) return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  constexpr uint32_t kExp = DT == SLORA_BF16 ? 0x7f807f80u : 0x7c007c00u;
  return w & ~__vcmpeq2(w & kExp, kExp);
}
// In a tile that has keys which some rows of the item do not see: their values that are not finite become zero, and
// the item is marked, for a scale that is not finite too.  By the warp that issues the products, while it would wait
// for the weights; chunk c of row k lies at at(k, c).  (In the softmax warps, which know these keys as well, the code alone
// took 3 to 8 % of the calls' time.)
template <bool CODES, int DT, int NC, typename At>
__device__ __forceinline__ void clean_tile(Item* x, int key0, const float* scales, At at) {
  const int lane = threadIdx.x & 31, shut = x->shut - key0, late = x->late - key0;
  const int first = max(x->lo - key0, 0), end = min(x->hi - key0, kKvTile);
  bool odd = false;
#pragma unroll 1
  for (int k = first + lane; k < end; k += 32) {
    if (k <= shut && k > late) continue;
    if (scales != nullptr) odd |= !(fabsf(scales[k]) < INFINITY);
#pragma unroll 1  // (four times the code takes 256 short e4m3 caches from 55 us to 58, though it never runs there)
    for (int c = 0; c < NC; ++c) {
      uint32_t w[4], f[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at(k, c)) : "memory");
      uint32_t diff = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = finite_only<CODES, DT>(w[i]);
        diff |= f[i] ^ w[i];
      }
      if (diff) {
        odd = true;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(k, c)), "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3]) : "memory");
      }
    }
  }
  if (odd) *reinterpret_cast<volatile int*>(&x->odd) = 1;
  __syncwarp();  // (the issuing thread's fence towards the tensor cores follows; all lanes run it)
}

// Which of V's elements lane * E + e (E = D / 32) of keys [ka, kb) are not finite: bits 1 infinity, 2 -infinity,
// 4 NaN, at 4 * e.  One warp.
template <int DT, int FMT, int D>
__device__ __forceinline__ uint32_t odd_values(const KvAttnDev& A, int b, int h, int ka, int kb) {
  constexpr int E = D / 32;
  constexpr bool F8 = FMT == SLORA_KV_E4M3;
  constexpr uint32_t kExp = DT == SLORA_BF16 ? 0x7f80u : 0x7c00u;
  const int lane = threadIdx.x & 31;
  const KvDev& P = A.kv;
  const unsigned char* const base = reinterpret_cast<const unsigned char*>(P.pool) + lane * (F8 ? E : 2 * E);
  uint32_t cls = 0;
#pragma unroll 1
  for (int j0 = ka; j0 < kb; j0 += 32) {
    uint32_t row = j0 + lane < kb ? kv_row(P, b, j0 + lane, h) : kNoRow;
    float scale = 1.f;
    if (row != kNoRow) {
      row += (uint32_t)(P.H * P.pt);
      if (F8) scale = *kv_scale(P, row);
    }
    const unsigned odd_scales = F8 ? __ballot_sync(FULL_MASK, !(fabsf(scale) < INFINITY)) : 0;
#pragma unroll 1
    for (int k0 = 0; k0 < 32; k0 += 8) {  // 8 keys' loads under way at once
      uint32_t w[8][2] = {};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t r = __shfl_sync(FULL_MASK, row, k0 + k);
        const unsigned char* const src = base + (uint64_t)r * KvRow<FMT, D>::kBytes;
        if (r == kNoRow) continue;
        if (!F8 && E == 4) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
          w[k][0] = x.x;
          w[k][1] = x.y;
        } else if (!F8 || E == 4) {
          w[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
        } else {
          w[k][0] = __ldg(reinterpret_cast<const uint16_t*>(src));
        }
      }
      uint32_t diff = odd_scales >> k0 & 0xff;
#pragma unroll
      for (int k = 0; k < 8; ++k) diff |= (w[k][0] ^ finite_only<F8, DT>(w[k][0])) | (w[k][1] ^ finite_only<F8, DT>(w[k][1]));
      if (!__any_sync(FULL_MASK, diff != 0)) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float s = F8 ? __shfl_sync(FULL_MASK, scale, k0 + k) : 1.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t v = F8 ? w[k][0] >> (8 * e) & 0xff : w[k][e >> 1] >> (16 * (e & 1)) & 0xffff;
          uint32_t c = 0;
          if (F8) {
            if ((v & 0x7f) == 0x7f || s != s) c = 4;
            else if (!(fabsf(s) < INFINITY)) c = (v & 0x7f) == 0 ? 4 : ((v >> 7) != 0) != (s < 0.f) ? 2 : 1;
          } else if ((v & kExp) == kExp) {
            c = (v & 0x7fff) != kExp ? 4 : v >> 15 ? 2 : 1;
          }
          cls |= c << (4 * e);
        }
      }
    }
  }
  return cls;
}

// Puts in what V's values that are not finite make of rows r0 + i * step of an item, for the bits i of `rows` (see the top).
// common: among the keys that all rows of the item see there may be some.  One warp.
template <int DT, int FMT, int D, int TM>
__device__ __forceinline__ void settle(const KvAttnDev& A, const Item& x, uint32_t rows, int r0, int step, bool common, float* part) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, r_item = x.rt * TM, b = x.b, h = x.h, W = A.window;
  const int ka = max(x.tile * kKvTile, x.lo), kb = min((x.tile + x.n_tiles) * kKvTile, x.hi);
  const bool odd = *reinterpret_cast<const volatile int*>(&x.odd), complete = (x.flags & 3) == 3;
  const int ac = max(ka, x.late + 1), bc = min(kb, x.shut + 1);  // keys that all rows see
  uint32_t all = 0, later = 0;  // of these keys, of those behind them up to `upto`
  int upto = bc;
  bool first = true;
#pragma unroll 1
  for (; rows; rows &= rows - 1, first = false) {
    const int r = r0 + (__ffs(rows) - 1) * step, t = token_of(A, r_item + r), p = x.first + t;
    const int from = W > 0 ? max(ka, p - W + 1) : ka, to = min(kb, p + 1);
    uint32_t own = 0;
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {  // the three parts of the keys that the row sees (one where no key is seen by all)
      int k0 = ac, k1 = first && common ? bc : ac;
      if (i == 1) {  // (rows in order: their positions do not fall)
        k0 = upto;
        k1 = odd ? to : upto;
      } else if (i == 2) {
        k0 = from;
        k1 = odd ? min(ac, to) : from;
      }
      if (ac >= bc) {
        k0 = from;
        k1 = i == 2 ? to : from;
      }
      if (k0 >= k1) continue;
      const uint32_t c = odd_values<DT, FMT, D>(A, b, h, k0, k1);
      if (i == 0) all |= c;
      else if (i == 1) later |= c;
      else own |= c;
      if (i == 1) upto = k1;
    }
    const uint32_t cls = all | later | own;
    const int hq = x.h * A.G + (r_item + r) - t * A.G;
    uint16_t* const o16 = A.out + (int64_t)(x.row0 + t) * A.ldo + (int64_t)hq * D + lane * E;
    float* const o32 = part + (size_t)r * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = cls >> (4 * e) & 7;
      if (c == 0) continue;
      const float v = c == 1 ? INFINITY : c == 2 ? -INFINITY : __uint_as_float(0x7fc00000u);
      if (complete) o16[e] = (uint16_t)pack2<DT>(v, 0.f);
      else o32[e] = v;
    }
  }
}

// Joins the partials of the item that starts in run `run` of a kernel's `ctas` and ends in a
// later one: weights l_i exp2(m_i - max m), in key order; 2^-40 of that, so that no term overflows where V does
// not.  A warp per row.
constexpr int kCombineThreads = 256;
template <int DT, int D, int TM>
__device__ __forceinline__ void join_item(const KvAttnDev& A, const void* workspace, int run, int ctas) {
  constexpr int E = D / 32;
  const Split sp = reinterpret_cast<const Split*>(workspace)[run];
  if (sp.n == 0) return;
  const float* const parts = reinterpret_cast<const float*>(reinterpret_cast<const Split*>(workspace) + ctas);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  KvSeq s;
  kv_seq(A.kv, sp.b, A.max_rows, s);
  const int r_item = sp.rt * TM, R = min(s.n * A.G - r_item, TM);
  auto at = [&](int i) { return parts + (size_t)(i == 0 ? sp.slot : 2 * (run + i)) * slot_floats(TM, D); };
  for (int r = blockIdx.y * (kCombineThreads / 32) + warp; r < R; r += gridDim.y * (kCombineThreads / 32)) {
    // values of kAhead partials at a time; the first ones' loads are under way beside those of the statistics
    constexpr int kAhead = 8;
    float v[kAhead][E];
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float* const p = at(min(i0 + k, sp.n - 1)) + (size_t)r * D + lane * E;
        if (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          v[k][0] = x.x;
          v[k][1] = x.y;
          v[k][E - 2] = x.z;
          v[k][E - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p);
          v[k][0] = x.x;
          v[k][1] = x.y;
        }
      }
    };
    load(0);
    float m0 = -INFINITY, l0 = 0.f;
    if (lane < sp.n) {
      m0 = at(lane)[(size_t)TM * D + r];
      l0 = at(lane)[(size_t)TM * (D + 1) + r];
    }
    float top = m0;
    for (int i = lane + 32; i < sp.n; i += 32) top = fmaxf(top, at(i)[(size_t)TM * D + r]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULL_MASK, top, o));
    const float z = (top == -INFINITY ? 0.f : top) + 40.f;
    float l = 0.f, o[E] = {};
#pragma unroll 1
    for (int i0 = 0; i0 < sp.n; i0 += 32) {
      if (i0 > 0) {
        m0 = -INFINITY;
        l0 = 0.f;
        if (i0 + lane < sp.n) {
          m0 = at(i0 + lane)[(size_t)TM * D + r];
          l0 = at(i0 + lane)[(size_t)TM * (D + 1) + r];
        }
      }
      const float w = ex2(m0 - z) * l0;
      l += w;
      const int n = min(32, sp.n - i0);
#pragma unroll 1
      for (int j = 0; j < n; j += kAhead) {
        if (i0 + j > 0) load(i0 + j);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float wk = __shfl_sync(FULL_MASK, w, (j + k) & 31);
          if (j + k < n) {
            if (wk != 0.f) {
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] += wk * v[k][e];
            } else {  // no weight in fp32, but some: an infinity stays one
#pragma unroll
              for (int e = 0; e < E; ++e) o[e] += fabsf(v[k][e]) < INFINITY ? 0.f : v[k][e];
            }
          }
        }
      }
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(FULL_MASK, l, k);
    const float inv = inverse(l);
    const int t = token_of(A, r_item + r), hq = sp.h * A.G + (r_item + r) - t * A.G;
    const int64_t tok = s.row0 + t;
    uint16_t* const orow = A.out + tok * A.ldo + (int64_t)hq * D + lane * E;
    if (E == 4)
      *reinterpret_cast<uint2*>(orow) = make_uint2(pack2<DT>(o[0] * inv, o[1] * inv), pack2<DT>(o[E - 2] * inv, o[E - 1] * inv));
    else
      *reinterpret_cast<uint32_t*>(orow) = pack2<DT>(o[0] * inv, o[1] * inv);
    if (A.lse && lane == 0) A.lse[tok * A.Hq + hq] = lse_of(top, l * 0x1p40f);
  }
}

// The kernels of a call follow one another by programmatic dependent launch: kv_chunk.cu's CTAs
// start where those of kv_decode.cu end (it waits for that grid before it ends itself, as
// nothing else would), and the join's are in place when the last of them ends.
template <typename K, typename... Args>
cudaError_t launch_behind(K kern, dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace
}  // namespace slora

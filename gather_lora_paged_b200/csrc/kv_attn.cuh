// kv_attn.cuh -- what the attention kernels share (kv_decode.cu,
// kv_chunk.cu): the line of key tiles that is cut into one run per CTA, the
// join of the partials, the row that is summed again.
//
// The rows of a kv head are the n * G pairs (token, head of the group), in row
// tiles of TM.  A work item is (sequence, kv head, row tile); its keys come in
// tiles of TK.  All items, laid out in one line, are cut into equal runs, one per CTA, so
// that ragged lengths and a single long sequence keep every SM equally busy.  An item is as long there as
// its tiles and a lead of E units, for what it costs beside them (q, the first maximum, its
// outputs).  An item inside one run is finished there; one that
// crosses runs leaves (max, sum, unnormalised row) partials, at most two per
// CTA, and k_kv_join joins them in key order.
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
  int pad;
};

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
  x.pad = 0;
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
// 1 / sum, 0 for a row without keys (a NaN sum stays NaN).
__device__ __forceinline__ float inverse(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }

// One row of an item again, key by key, over keys [ka, kb) with the row's own
// final maximum m: o_d = sum over visible keys of exp2(s_j - m) v_jd.  dst16 (a
// finished row, divided by the sum l) or dst32 (a partial).  One warp; rare.
template <int DT, int FMT, int D>
__device__ __noinline__ void redo_row(const KvAttnDev& A, int b, int h, const uint16_t* qrow, int p, int ka, int kb,
                                      float m, float inv_l, uint16_t* dst16, float* dst32) {
  constexpr int E = D / 32;  // values per lane
  const int lane = threadIdx.x & 31;
  const KvDev& P = A.kv;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t w = __ldg(qrow + lane * E + e);
    float hi;
    if (DT == SLORA_BF16) q[e] = __uint_as_float(w << 16);
    else h2x2f(w, q[e], hi);
    o[e] = 0.f;
  }
  if (A.window > 0) ka = max(ka, p - A.window + 1);
  kb = min(kb, p + 1);
  const unsigned char* base = reinterpret_cast<const unsigned char*>(P.pool);
  for (int j = ka; j < kb; ++j) {
    const uint32_t kr = kv_row(P, b, j, h);
    if (kr == kNoRow) continue;
    const uint32_t vr = kr + (uint32_t)(P.H * P.pt);
    float kv[E], vv[E], dot = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (FMT == SLORA_KV_16) {
        const uint32_t a = reinterpret_cast<const uint16_t*>(base)[(int64_t)kr * D + lane * E + e];
        const uint32_t c = reinterpret_cast<const uint16_t*>(base)[(int64_t)vr * D + lane * E + e];
        float hi;
        if (DT == SLORA_BF16) {
          kv[e] = __uint_as_float(a << 16);
          vv[e] = __uint_as_float(c << 16);
        } else {
          h2x2f(a, kv[e], hi);
          h2x2f(c, vv[e], hi);
        }
      } else {
        const uint32_t a = e4m3x2_f16x2(base[(int64_t)kr * D + lane * E + e]);
        const uint32_t c = e4m3x2_f16x2(base[(int64_t)vr * D + lane * E + e]);
        kv[e] = __low2float(*reinterpret_cast<const __half2*>(&a)) * *kv_scale(P, kr);
        vv[e] = __low2float(*reinterpret_cast<const __half2*>(&c)) * *kv_scale(P, vr);
      }
      dot += q[e] * kv[e];
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) dot += __shfl_xor_sync(FULL_MASK, dot, d);
    const float w = ex2(dot * A.c - m);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += w * vv[e];
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (dst16) dst16[lane * E + e] = (uint16_t)pack2<DT>(o[e] * inv_l, 0.f);
    else dst32[lane * E + e] = o[e];
  }
}

// Joins the partials of the item that starts in run `run` of a kernel's `ctas` and ends in a
// later one: weights exp2(m_i - max m), in key order.  A warp per row.
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
    const float z = top == -INFINITY ? 0.f : top;
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
      const float w = ex2(m0 - z);
      l += w * l0;
      const int n = min(32, sp.n - i0);
#pragma unroll 1
      for (int j = 0; j < n; j += kAhead) {
        if (i0 + j > 0) load(i0 + j);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float wk = __shfl_sync(FULL_MASK, w, (j + k) & 31);
          if (j + k < n) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] += wk * v[k][e];
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
    if (A.lse && lane == 0) A.lse[tok * A.Hq + hq] = lse_of(top, l);
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

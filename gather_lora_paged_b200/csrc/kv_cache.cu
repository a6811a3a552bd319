// kv_cache.cu -- writing new tokens' K and V rows into the KV pages, as they
// are or quantised to e4m3, and reading pages back into dense rows.
//
// Quantisation of one row x (one token, one head, K or V; D values):
//     scale = RN32(max|x| / 448), at least 2^-126; code_d = e4m3(x_d / scale)
// with the exact quotient rounded to nearest, ties to the even code.  An
// all-zero row has scale 0; a row with an infinity or a NaN has scale NaN and
// zero codes, so it reads back as NaN.  Reading: RN16(scale * value(code)).
//
// Both kernels move each byte once and are bound by HBM (small calls: by one
// launch and a chain of three dependent loads).  A warp takes rows of one token,
// kIter * 32 / (D / 8) at a time; the first ones' loads are issued before the token's page is
// looked up, so that the look-up's latency hides behind them.
// Measured: a prefill step's 24,888 tokens of 32 kv heads of 128 into e4m3 pages, 618 MB: 119 us (5.2 TB/s;
// instruction issue, then HBM); 8 heads, 11,935 tokens as they are, 98 MB: 19 us;
// reading 24,273 tokens of 32 heads, 795 MB: 135 us (5.9 TB/s); one token: 4 us.
#include "kv_common.cuh"

namespace slora {
namespace {

constexpr int kWarps = 8;   // per CTA
constexpr int kIter = 4;    // 16-byte loads in flight per lane

// The sequence of row t and its position (the whole warp asks for one t): a
// 32-way search of row_start, after a look at sequence t itself, which is the
// answer when every sequence has one row.  False: no usable sequence owns t, or
// its position lies before the cache's first token.
__device__ __forceinline__ bool kv_locate(const KvDev& P, int t, int& b, int& pos) {
  KvSeq s;
  const int lane = threadIdx.x & 31;
  b = t;
  if (!(t < P.B && __ldg(P.row_start + t) <= t && t < __ldg(P.row_start + t + 1))) {
    int lo = 0, cnt = P.B + 1;  // the last of [lo, lo + cnt) with row_start <= t
    while (cnt > 1) {
      const int step = (cnt + 31) >> 5;
      const bool in = lane * step < cnt && __ldg(P.row_start + lo + lane * step) <= t;
      const unsigned m = __ballot_sync(FULL_MASK, in);
      if (!m) return false;
      const int k = 31 - __clz(m);
      lo += k * step;
      cnt = min(step, cnt - k * step);
    }
    b = lo;
    if (b >= P.B) return false;
  }
  if (!kv_seq(P, b, INT32_MAX, s) || t < s.row0 || t >= s.row0 + s.n) return false;
  pos = s.len - s.n + (t - s.row0);
  return pos >= 0;
}

// Quantisation to the nearest code of the exact quotient q = x / scale, ties to even, with one product
// per value.  With A = max|x| and borders m of two codes (at most 5 significant bits), x * 448 = m * A is an
// equation of integers of at most 16 bits up to powers of two, so either it holds or x / A is off
// m / 448 by 2^-16 (relative) at least.  Where it holds, q = m (A / 448) / scale is on the side of m on
// which A / 448 is of its rounded value, for the whole row.  So x * rinv, rinv within 2^-22 of 1 / scale and
// then moved by 2^-20 to that side, has q's code.  If 448 divides A without a rounding (or scale is the
// least, a power of two), borders are met exactly: x * rinv is corrected by its residual (Markstein),
// which makes it RN(q), the border itself there.
struct RowScale {
  float scale, rinv;
  bool exact;
};
__device__ __forceinline__ float reciprocal(float x) {  // to one ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ RowScale row_scale(float most) {
  // RN(most / 448): the product with RN(1 / 448) corrected by its residual, which is exact (all 16-bit
  // values whose quotient is above 2^-126 have been tried)
  const float c = 1.f / 448.f, q = most * c, s = fmaf(fmaf(-q, 448.f, most), c, q);
  RowScale r;
  r.scale = fmaxf(s, 0x1p-126f);
  const float rest = fmaf(-s, 448.f, most);
  r.exact = rest == 0.f || s < 0x1p-126f;
  r.rinv = reciprocal(r.scale);
  if (!r.exact) r.rinv *= rest > 0.f ? 1.f + 0x1p-20f : 1.f - 0x1p-20f;
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint2 quantise8(const float* f, RowScale s) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 x, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 r, {%4, %4};\n\tmul.rn.f32x2 x, x, r;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(q[i]), "=f"(q[i + 1]) : "f"(f[i]), "f"(f[i + 1]), "f"(s.rinv));
  if (s.exact) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fmaf(-fmaf(q[i], s.scale, -f[i]), s.rinv, q[i]);  // (signs that keep -0)
  }
  return make_uint2(cvt_e4m3x2(q[0], q[1]) | cvt_e4m3x2(q[2], q[3]) << 16, cvt_e4m3x2(q[4], q[5]) | cvt_e4m3x2(q[6], q[7]) << 16);
}
// The larger of two pairs of 15-bit magnitudes.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A token's 2 * H rows come in blocks of kIter * RPI; a warp takes `blocks` of them in a row, the next
// one's loads under way while it deals with one.
template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_write(KvDev P, const uint16_t* k, int64_t ldk, const uint16_t* v,
                                                          int64_t ldv, int blocks, int per_token) {
  constexpr int kRowBytes = KvRow<FMT, D>::kBytes;
  constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes per row, rows per pass
  const int lane = threadIdx.x & 31, col = (lane % LPR) * 8;
  if (blockIdx.x == 0) kv_record_bad(P, INT32_MAX, threadIdx.x, blockDim.x);
  const int units = P.T * per_token;
  for (int u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const int t = u / per_token, first = (u - t * per_token) * blocks * (kIter * RPI);
    const int end = min(2 * P.H, first + blocks * (kIter * RPI));
    const uint16_t* const kt = k + (int64_t)t * ldk + col;
    const uint16_t* const vt = v + (int64_t)t * ldv + col - P.H * D;
    uint4 next[kIter];
    auto load = [&](int r0) {
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = r0 + i * RPI;
        next[i] = make_uint4(0, 0, 0, 0);
        if (r < end) next[i] = __ldg(reinterpret_cast<const uint4*>((r < P.H ? kt : vt) + r * D));
      }
    };
    load(first + lane / LPR);
    int b, pos;
    if (!kv_locate(P, t, b, pos)) continue;
    const uint32_t row = kv_row(P, b, pos, 0);
    if (row == kNoRow) continue;
    unsigned char* const to = reinterpret_cast<unsigned char*>(P.pool) + (int64_t)row * kRowBytes + col * (kRowBytes / D);
    float* const scales = FMT == SLORA_KV_E4M3 ? kv_scale(P, row) : nullptr;
#pragma unroll 1
    for (int r0 = first + lane / LPR; r0 - lane / LPR < end; r0 += kIter * RPI) {
      uint4 x[kIter];
#pragma unroll
      for (int i = 0; i < kIter; ++i) x[i] = next[i];
      if (r0 - lane / LPR + kIter * RPI < end) load(r0 + kIter * RPI);
      uint32_t tops[kIter / 2];  // the rows' largest magnitudes, as 16-bit patterns
      if (FMT == SLORA_KV_E4M3) {
#pragma unroll
        for (int i = 0; i < kIter; i += 2) {
          uint32_t t[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            t[k] = max_u16x2(max_u16x2(x[i + k].x & 0x7fff7fffu, x[i + k].y & 0x7fff7fffu),
                             max_u16x2(x[i + k].z & 0x7fff7fffu, x[i + k].w & 0x7fff7fffu));
          uint32_t top = max_u16x2(__byte_perm(t[0], t[1], 0x5410), __byte_perm(t[0], t[1], 0x7632));
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1) top = max_u16x2(top, __shfl_xor_sync(FULL_MASK, top, o));
          tops[i / 2] = top;
        }
      }
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = r0 + i * RPI;
        const uint32_t off = (uint32_t)r * (uint32_t)P.pt;  // row r = (part, head): of the same page
        if (FMT == SLORA_KV_16) {
          if (r < end) *reinterpret_cast<uint4*>(to + (int64_t)off * kRowBytes) = x[i];
        } else {
          const uint32_t top = i & 1 ? tops[i / 2] >> 16 : tops[i / 2] & 0xffff;
          float scale = 0.f;
          uint2 codes = make_uint2(0, 0);
          if (top >= (DT == SLORA_BF16 ? 0x7f80u : 0x7c00u)) {
            scale = __uint_as_float(0x7fc00000u);
          } else if (top) {
            float f[8], most, zero;
            unpack8<DT>(x[i], f);
            if (DT == SLORA_BF16) most = __uint_as_float(top << 16);
            else h2x2f(top, most, zero);
            const RowScale rs = row_scale(most);
            scale = rs.scale;
            codes = quantise8(f, rs);
          }
          if (r < end) {
            *reinterpret_cast<uint2*>(to + (int64_t)off * kRowBytes) = codes;
            if (col == 0) scales[off] = scale;
          }
        }
      }
    }
  }
}

template <int DT, int FMT, int D>
__global__ void __launch_bounds__(kWarps * 32) k_kv_read(KvDev P, uint16_t* k, int64_t ldk, uint16_t* v, int64_t ldv,
                                                         int per_token) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;
  const int lane = threadIdx.x & 31, col = (lane % LPR) * 8;
  if (blockIdx.x == 0) kv_record_bad(P, INT32_MAX, threadIdx.x, blockDim.x);
  const int units = P.T * per_token;
  for (int u = blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += gridDim.x * kWarps) {
    const int t = u / per_token, r0 = (u - t * per_token) * (kIter * RPI) + lane / LPR;
    int b, pos;
    if (!kv_locate(P, t, b, pos)) continue;
    const uint32_t row = kv_row(P, b, pos, 0);
    if (row == kNoRow) continue;
    uint4 x[kIter];
    float scale[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = r0 + i * RPI;
      const uint32_t src = row + (uint32_t)(r * P.pt);
      x[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 0.f;
      if (r < 2 * P.H) {
        if (FMT == SLORA_KV_16) {
          x[i] = *reinterpret_cast<const uint4*>(P.pool + (int64_t)src * D + col);
        } else {
          const uint2 c = *reinterpret_cast<const uint2*>(reinterpret_cast<const unsigned char*>(P.pool) +
                                                          (int64_t)src * D + col);
          x[i].x = c.x;
          x[i].y = c.y;
          scale[i] = *kv_scale(P, src);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = r0 + i * RPI;
      if (r >= 2 * P.H) break;
      if (FMT == SLORA_KV_E4M3) {
        const uint32_t w[2] = {x[i].x, x[i].y};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h = e4m3x2_f16x2(w[j >> 1] >> (16 * (j & 1)));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          o[j] = pack2<DT>(f.x * scale[i], f.y * scale[i]);
        }
        x[i] = make_uint4(o[0], o[1], o[2], o[3]);
      }
      uint16_t* dst = r < P.H ? k + (int64_t)t * ldk + (int64_t)r * D : v + (int64_t)t * ldv + (int64_t)(r - P.H) * D;
      *reinterpret_cast<uint4*>(dst + col) = x[i];
    }
  }
}

struct Grid {
  int grid, per_token;
};
Grid grid_for(const KvDev& P, int D, int sm_count) {
  const int rows = kIter * 32 / (D / 8);
  Grid g;
  g.per_token = cdiv_i(2 * P.H, rows);
  const int64_t ctas = ((int64_t)P.T * g.per_token + kWarps - 1) / kWarps;
  g.grid = (int)(ctas < (int64_t)sm_count * 8 ? ctas : (int64_t)sm_count * 8);
  return g;
}

}  // namespace

cudaError_t launch_kv_write(const KvDev& P, int dtype, int fmt, int D, const void* k, int64_t ldk, const void* v,
                            int64_t ldv, int sm_count, cudaStream_t s) {
  // a token's rows are spread over warps while there are fewer of these than the GPU holds
  const int all = cdiv_i(2 * P.H, kIter * 32 / (D / 8));
  const int64_t each = (int64_t)P.T * all / ((int64_t)sm_count * 40);
  const int blocks = (int)(each < 1 ? 1 : each > all ? all : each), per_token = cdiv_i(all, blocks);
  const int64_t ctas = ((int64_t)P.T * per_token + kWarps - 1) / kWarps;
  const int grid = (int)(ctas < (int64_t)sm_count * 8 ? ctas : (int64_t)sm_count * 8);
  auto go = [&](auto kern) {
    kern<<<grid, kWarps * 32, 0, s>>>(P, static_cast<const uint16_t*>(k), ldk, static_cast<const uint16_t*>(v), ldv, blocks,
                                      per_token);
    return cudaGetLastError();
  };
  if (fmt == SLORA_KV_16)  // a copy: the element type does not matter
    return D == 64 ? go(k_kv_write<SLORA_F16, SLORA_KV_16, 64>) : go(k_kv_write<SLORA_F16, SLORA_KV_16, 128>);
  if (dtype == SLORA_F16)
    return D == 64 ? go(k_kv_write<SLORA_F16, SLORA_KV_E4M3, 64>) : go(k_kv_write<SLORA_F16, SLORA_KV_E4M3, 128>);
  return D == 64 ? go(k_kv_write<SLORA_BF16, SLORA_KV_E4M3, 64>) : go(k_kv_write<SLORA_BF16, SLORA_KV_E4M3, 128>);
}

cudaError_t launch_kv_read(const KvDev& P, int dtype, int fmt, int D, void* k, int64_t ldk, void* v, int64_t ldv,
                           int sm_count, cudaStream_t s) {
  const Grid g = grid_for(P, D, sm_count);
  auto go = [&](auto kern) {
    kern<<<g.grid, kWarps * 32, 0, s>>>(P, static_cast<uint16_t*>(k), ldk, static_cast<uint16_t*>(v), ldv, g.per_token);
    return cudaGetLastError();
  };
  if (fmt == SLORA_KV_16)
    return D == 64 ? go(k_kv_read<SLORA_F16, SLORA_KV_16, 64>) : go(k_kv_read<SLORA_F16, SLORA_KV_16, 128>);
  if (dtype == SLORA_F16)
    return D == 64 ? go(k_kv_read<SLORA_F16, SLORA_KV_E4M3, 64>) : go(k_kv_read<SLORA_F16, SLORA_KV_E4M3, 128>);
  return D == 64 ? go(k_kv_read<SLORA_BF16, SLORA_KV_E4M3, 64>) : go(k_kv_read<SLORA_BF16, SLORA_KV_E4M3, 128>);
}

}  // namespace slora

// kv_common.cuh -- what the KV-cache kernels share (kv_cache.cu,
// kv_decode.cu, kv_chunk.cu): their parameter blocks, the layout of a KV page, the
// checks of a batch's sequences, e4m3 conversions.
//
// A page of one layer holds page_tokens tokens of H kv heads, as rows of D
// values: [K, V][head][token][D]; in e4m3 the codes are followed by the row
// scales [K, V][head][token] (fp32).  The whole pool is therefore one array of
// rows of D values (a page holds 2^row_shift of them), and the row of (page,
// part, head, slot) is (page << row_shift) + (part * H + head) * pt + slot: an
// unsigned 32-bit number for every pool that fits the device (192 GB / 64 B).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dev_common.cuh"
#include "slora_internal.h"

namespace slora {

// Device error codes of the KV-cache kernels (info: the sequence).
constexpr int kErrKvSeq = 8;    // rows outside [0, T], kv_len outside the table, more rows than max_rows
constexpr int kErrKvPage = 9;   // a page id outside the pool

constexpr uint32_t kNoRow = 0xffffffffu;

template <int FMT, int D>
struct KvRow {
  static constexpr int kBytes = FMT == SLORA_KV_E4M3 ? D : 2 * D;  // one row in the cache
};

struct KvSeq {
  int row0, n, len;  // first row, rows, tokens in the cache (these rows are the newest)
};

// Loads sequence b; false if its numbers are not usable (nothing of it is touched).
__device__ __forceinline__ bool kv_seq(const KvDev& P, int b, int max_rows, KvSeq& s) {
  s.row0 = __ldg(P.row_start + b);
  const int end = __ldg(P.row_start + b + 1);
  s.len = __ldg(P.kv_len + b);
  s.n = end - s.row0;
  return s.row0 >= 0 && end >= s.row0 && end <= P.T && s.len >= 0 && (int64_t)s.len <= P.capacity &&
         s.n <= max_rows;
}

// Records the sequences that kv_seq refuses (n threads of one CTA of a kernel do this).
__device__ __forceinline__ void kv_record_bad(const KvDev& P, int max_rows, int thread, int n) {
  for (int b = thread; b < P.B; b += n) {
    KvSeq s;
    if (!kv_seq(P, b, max_rows, s)) record_error(P.err, kErrKvSeq, b);
  }
}

// Page of a sequence that holds a position.
__device__ __forceinline__ int kv_block(const KvDev& P, int pos) {
  return (int)(((uint64_t)(uint32_t)pos * P.pt_mul) >> P.pt_shift);
}

// Row of (sequence b, position pos, K part, head h) in the pool; kNoRow (and a
// recorded error) if its page id is outside the pool.  The V row is H * pt on.
__device__ __forceinline__ uint32_t kv_row(const KvDev& P, int b, int pos, int h) {
  const int blk = kv_block(P, pos);
  const int pg = __ldg(P.blocks + (int64_t)b * P.ldb + blk);
  if (pg < 0 || pg >= P.n_pages) {
    record_error(P.err, kErrKvPage, b);
    return kNoRow;
  }
  return ((uint32_t)pg << P.row_shift) + (uint32_t)(h * P.pt + (pos - blk * P.pt));
}

// Address of the scale of a row (e4m3): the page's codes end at scale_off floats.
__device__ __forceinline__ float* kv_scale(const KvDev& P, uint32_t row) {
  const uint32_t in_page = row & ((1u << P.row_shift) - 1);
  return reinterpret_cast<float*>(P.pool) + ((int64_t)(row >> P.row_shift) << (P.page_shift - 1)) + P.scale_off +
         in_page;
}

// Two e4m3 codes (low byte first) -> two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;}" : "=r"(r) : "r"(codes));
  return r;
}

}  // namespace slora

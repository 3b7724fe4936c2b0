// The quantized key/value cache as its kernels see it, and the two lookups they share: which
// sequence a row belongs to, and which page a position lies in.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace gptq {

// One of the two halves (K or V) of a cache.
struct CacheHalf {
  uint8_t* codes;     // [pages][heads][page][row_bytes]
  uint16_t* scales;   // [pages][heads][page][groups], bf16 bits
  uint8_t* zeros;     // [pages][heads][page][groups]
};

struct CacheView {
  CacheHalf half[2];  // K, V
  int64_t pages;
  int heads, page_shift, width;   // tokens per page = 1 << page_shift; width: page table columns
};

// Rows starts[b] .. starts[b + 1] - 1 belong to sequence b and are its last positions, the last one
// at lengths[b] - 1. Without starts, row b is the last position of sequence b.
struct CacheRows {
  const int32_t* table;
  int64_t ld_table;
  const int32_t* lengths;
  const int32_t* starts;
  int64_t batch, n;
};

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

// Scale (bf16 bits) of a group whose values are all zero: 2 / (2^bits - 1), rounded up.
template <int BITS>
constexpr uint32_t kEmptyScale = BITS == 4 ? 0x3E09u : 0x3C01u;

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The page of position pos of a sequence, or -1 (recorded in the status word) if the position lies
// past the page table or the table names no page of the cache.
__device__ __forceinline__ int32_t find_page(const CacheView& c, const int32_t* table_row,
                                             int64_t pos, int32_t* info) {
  const int64_t k = pos >> c.page_shift;
  if (pos >= 0 && k < c.width) {
    const int32_t p = __ldg(table_row + k);
    if (p >= 0 && p < c.pages) return p;
  }
  record_info(info, GPTQ_INFO_BAD_PAGE);
  return -1;
}

// Index of row `off` of head `head` on page `page`, in rows of codes (and of grids).
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int32_t page, int head, int off) {
  return ((static_cast<int64_t>(page) * c.heads + head) << c.page_shift) + off;
}

// The sequence of row i, by a whole warp (every lane gets the answer): the number of sequences that
// end at or before row i, found in steps of 32 ends at a time. batch if the row lies behind the
// last sequence. Ends that do not ascend give some sequence, never an index out of range.
__device__ __forceinline__ int64_t find_sequence(const CacheRows& r, int64_t i) {
  if (r.starts == nullptr) return i < r.batch ? i : r.batch;
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, len = r.batch;
  while (len > 0) {
    const int64_t stride = (len + 31) >> 5;
    const int64_t at = min((lane + 1) * stride, len);
    const int k = __popc(__ballot_sync(0xffffffffu, __ldg(r.starts + lo + at) <= i));
    if (k == 32) return lo + len;
    const int64_t skip = min(static_cast<int64_t>(k) * stride, len);
    lo += skip;
    len = min(stride, len - skip) - 1;
  }
  return lo;
}

// Calls f with (dim, bits, group) as compile-time constants.
template <typename F>
gptq_status dispatch_cache(int dim, int bits, int group, F f) {
  auto with = [&](auto d, auto g) {
    return bits == 4 ? f(d, std::integral_constant<int, 4>{}, g)
                     : f(d, std::integral_constant<int, 8>{}, g);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using G32 = std::integral_constant<int, 32>;
  if (dim == 64) return group == 32 ? with(D64{}, G32{}) : with(D64{}, D64{});
  return group == 32 ? with(D128{}, G32{}) : group == 64 ? with(D128{}, D64{}) : with(D128{}, D128{});
}

gptq_status run_cache_append(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const void* K, int64_t ldk, const void* V, int64_t ldv, bool bf16,
                             void* K_hat, void* V_hat, int32_t* info, cudaStream_t stream);
gptq_status run_cache_read(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                           void* K_out, void* V_out, bool bf16, int32_t* info, cudaStream_t stream);

// Attention over the cache. With prefix_len > 0 rows also meet positions 0 .. prefix_len - 1 of the
// common sequence behind prefix_table; 0: plain.
struct CacheQuery {
  const __nv_bfloat16* q;   // [n][ldq], heads * ratio vectors a row
  int64_t ldq;
  int ratio;                // query heads per cache head
  float scale;
  __nv_bfloat16* out;       // [n][ldo]
  int64_t ldo;
  const int32_t* prefix_table;
  int64_t prefix_len;
};
size_t prefix_workspace_bytes(int heads, int dim, int64_t n, int ratio);
// The prefix on the tensor cores, joined with each row's own level (mid, mid_lse) into the output.
gptq_status run_cache_prefix(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const CacheQuery& q, const float* mid, const float* mid_lse, void* ws,
                             int32_t* info, cudaStream_t stream);
size_t cache_workspace_bytes(int heads, int dim, int64_t n, int ratio, bool shared);
gptq_status run_cache_attend(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const CacheQuery& q, void* ws, int32_t* info, cudaStream_t stream);

}  // namespace gptq

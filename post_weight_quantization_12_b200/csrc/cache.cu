// Writing the quantized key/value cache and reading it back.
//
// The grid of a group of g values x of one token and head ("GPTQ second-order quantization" blog,
// "Group-wise quantization": one scale and zero point per group; the layer quantizer's asymmetric
// min/max grid, with one change):
//   lo = min(0, min x), hi = max(0, max x), step = (hi - lo) / (2^bits - 1)   ([-1, 1] if step = 0)
//   s = step rounded up to bf16, z = clamp(rint(-lo / s)), q = clamp(rint(x / s) + z)
// each step rounded once in fp32, half to even; the value the codes stand for is s (q - z). The
// step has 8 significant bits: a scale takes 2 bytes, and rounding it up (by 2^-7 of itself at
// most) keeps both ends of [lo, hi] on the grid. A group with a value that is not finite, or whose
// step is not, gets a NaN scale and zero codes, so it reads back as NaN.
//
// Both kernels move each byte once and are bound by HBM: append reads 2 or 4 bytes a value, writes
// bits / 8 and, where the caller wants the values back, 2 or 4 more; read writes 2 or 4 for
// bits / 8 read.
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace gptq {
namespace {

constexpr int kRowThreads = 256;

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight consecutive values of a row.
template <bool kBf16>
struct Eight {
  uint4 raw[kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (kBf16 ? 1 : 2); ++i) raw[i] = __ldcs(static_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (kBf16) {
      const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(raw[i].x);
        x[4 * i + 1] = __uint_as_float(raw[i].y);
        x[4 * i + 2] = __uint_as_float(raw[i].z);
        x[4 * i + 3] = __uint_as_float(raw[i].w);
      }
    }
  }
};

// Eight values to a row of bf16 (rounded to nearest even) or fp32.
template <bool kBf16>
__device__ __forceinline__ void store8(void* p, const float (&x)[8]) {
  if constexpr (kBf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
    __stcs(static_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(static_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
}

// The small integer that a float holds, as bits: 0 <= v < 2^23.
__device__ __forceinline__ uint32_t int_bits(float v) { return __float_as_uint(v + 8388608.f); }

// The grid of a group and the eight codes of this lane. The lanes of a group are consecutive; all
// of them get the same s and z. Codes come back as small floats.
template <int kBits, int kLanes>
__device__ __forceinline__ void make_grid(const float (&x)[8], float& s, float& z, float (&q)[8]) {
  constexpr float kTop = static_cast<float>((1 << kBits) - 1);
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  float step = __fdiv_rn(__fsub_rn(hi, lo), kTop);
  if (step == 0.f) {
    lo = -1.f;
    step = __fdiv_rn(2.f, kTop);
  }
  s = __uint_as_float((__float_as_uint(step) + 0xFFFFu) & 0xFFFF0000u);
  // a step that is inf or NaN (the only other values the sum of its parts can take) fails here
  if (!(fabsf(lo) <= 3.4028235e38f && hi <= 3.4028235e38f && s <= 3.4028235e38f)) {
    s = __uint_as_float(0x7FC00000u);
    z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = 0.f;
    return;
  }
  z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), kTop);
  // rint(x / s) from x * (1 / s), which is off by at most 255 * 2^-23 < 3.1e-5: if one of the
  // eight quotients lies within 1e-4 of a half-integer (or 1 / s overflows), all are redone with
  // the exact division, so the codes are those of the division always.
  const float inv = __frcp_rn(s);
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = x[i] * inv, k = rintf(r);
    near |= !(fabsf(fabsf(r - k) - 0.5f) > 1e-4f);
    q[i] = k;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = rintf(__fdiv_rn(x[i], s));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(q[i] + z, 0.f), kTop);
}

// A row is one token's vector of one head: kDim / 8 consecutive lanes, eight values each. Every
// warp takes 256 / kDim rows of K and the same of V per step; their loads go out before the page
// lookup, which they do not depend on. At 53,248 tokens x 8 heads x 128, 4-bit, with the stored
// values returned in bf16 (493 MB): see the table of measured times.
template <int kDim, int kBits, int kGroup, bool kXBf16>
__global__ void __launch_bounds__(kRowThreads)
cache_append_kernel(const CacheView c, const CacheRows rows, const void* __restrict__ K,
                    int64_t ldk, const void* __restrict__ V, int64_t ldv, void* K_hat, void* V_hat,
                    int32_t* info) {
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes, kGroups = kDim / kGroup;
  constexpr int kElem = kXBf16 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t total = rows.n * c.heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5)) *
                    kPer;
       r0 < total; r0 += warps * kPer) {
    const int64_t r = min(r0 + sub, total - 1);
    const bool live = r0 + sub < total;
    const int64_t tok = r / c.heads;
    const int head = static_cast<int>(r - tok * c.heads);
    Eight<kXBf16> in[2];
    in[0].load(static_cast<const uint8_t*>(K) + (tok * ldk + head * kDim + 8 * l) * kElem);
    in[1].load(static_cast<const uint8_t*>(V) + (tok * ldv + head * kDim + 8 * l) * kElem);
    // the sequences of this warp's rows (whole-warp searches; one if the rows share their token)
    const int64_t tok0 = r0 / c.heads;
    int64_t b = find_sequence(rows, tok0);
    for (int k = 1; k < kPer; ++k) {
      const int64_t tk = min(r0 + k, total - 1) / c.heads;
      if (tk != tok0) {
        const int64_t bk = find_sequence(rows, tk);
        if (sub == k) b = bk;
      }
    }
    int32_t page = -1;
    int64_t pos = 0;
    if (live && b < rows.batch) {
      const int64_t first = rows.starts ? __ldg(rows.starts + b) : b;
      const int64_t end = rows.starts ? __ldg(rows.starts + b + 1) : b + 1;
      pos = static_cast<int64_t>(__ldg(rows.lengths + b)) - end + tok;
      if (tok >= first) page = find_page(c, rows.table + b * rows.ld_table, pos, info);
    }
    const int64_t at =
        cache_row(c, page < 0 ? 0 : page, head, static_cast<int>(pos) & ((1 << c.page_shift) - 1));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8], q[8], s, z;
      in[h].get(x);
      make_grid<kBits, kGroup / 8>(x, s, z, q);
      if (page < 0) continue;   // behind the last sequence, or no page: left as it was
      uint8_t* codes = c.half[h].codes + at * (kDim * kBits / 8) + l * kBits;
      if constexpr (kBits == 4) {
        // four codes per exact fp32 sum q0 + 16 q1 + 256 q2 + 4096 q3
        const float a = fmaf(4096.f, q[3], fmaf(256.f, q[2], fmaf(16.f, q[1], q[0])));
        const float b4 = fmaf(4096.f, q[7], fmaf(256.f, q[6], fmaf(16.f, q[5], q[4])));
        *reinterpret_cast<uint32_t*>(codes) = __byte_perm(int_bits(a), int_bits(b4), 0x5410);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = int_bits(fmaf(256.f, q[2 * i + 1], q[2 * i]));
        *reinterpret_cast<uint2*>(codes) = make_uint2(__byte_perm(w[0], w[1], 0x5410),
                                                      __byte_perm(w[2], w[3], 0x5410));
      }
      if (l % (kGroup / 8) == 0) {
        const int64_t gi = at * kGroups + l / (kGroup / 8);
        c.half[h].scales[gi] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
        c.half[h].zeros[gi] = static_cast<uint8_t>(int_bits(z));
      }
      uint8_t* hat = static_cast<uint8_t*>(h == 0 ? K_hat : V_hat);
      if (hat != nullptr) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(s, __fsub_rn(q[i], z));
        store8<kXBf16>(hat + ((tok * c.heads + head) * kDim + 8 * l) * kElem, y);
      }
    }
  }
}

// The values of the last positions of every sequence; a position without a page reads as 0.
template <int kDim, int kBits, int kGroup, bool kYBf16>
__global__ void __launch_bounds__(kRowThreads)
cache_read_kernel(const CacheView c, const CacheRows rows, void* __restrict__ K_out,
                  void* __restrict__ V_out, int32_t* info) {
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes, kGroups = kDim / kGroup;
  constexpr int kElem = kYBf16 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int64_t total = rows.n * c.heads;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5)) *
                    kPer;
       r0 < total; r0 += warps * kPer) {
    const int64_t r = min(r0 + sub, total - 1);
    const int64_t tok = r / c.heads;
    const int head = static_cast<int>(r - tok * c.heads);
    const int64_t tok0 = r0 / c.heads;
    int64_t b = find_sequence(rows, tok0);
    for (int k = 1; k < kPer; ++k) {
      const int64_t tk = min(r0 + k, total - 1) / c.heads;
      if (tk != tok0) {
        const int64_t bk = find_sequence(rows, tk);
        if (sub == k) b = bk;
      }
    }
    if (r0 + sub >= total || b >= rows.batch) continue;
    const int64_t first = rows.starts ? __ldg(rows.starts + b) : b;
    const int64_t end = rows.starts ? __ldg(rows.starts + b + 1) : b + 1;
    if (tok < first) continue;
    const int64_t pos = static_cast<int64_t>(__ldg(rows.lengths + b)) - end + tok;
    const int32_t page = find_page(c, rows.table + b * rows.ld_table, pos, info);
    const int64_t at =
        cache_row(c, page < 0 ? 0 : page, head, static_cast<int>(pos) & ((1 << c.page_shift) - 1));
    float y[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint8_t* out = static_cast<uint8_t*>(h == 0 ? K_out : V_out);
      if (out == nullptr) continue;
      const uint8_t* codes = c.half[h].codes + at * (kDim * kBits / 8) + l * kBits;
      const int64_t gi = at * kGroups + l / (kGroup / 8);
      const float s = bf16_bits_to_float(c.half[h].scales[gi]);
      const float z = static_cast<float>(c.half[h].zeros[gi]);
      uint32_t w[2];
      if constexpr (kBits == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(codes);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(codes);
        w[0] = v.x;
        w[1] = v.y;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t q = kBits == 4 ? (w[0] >> (4 * i)) & 15u : (w[i / 4] >> (8 * (i % 4))) & 255u;
        y[h][i] = page < 0 ? 0.f : __fmul_rn(s, __fsub_rn(static_cast<float>(q), z));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint8_t* out = static_cast<uint8_t*>(h == 0 ? K_out : V_out);
      if (out != nullptr) store8<kYBf16>(out + ((tok * c.heads + head) * kDim + 8 * l) * kElem, y[h]);
    }
  }
}

unsigned row_grid(int64_t rows, int per_warp) {
  const int64_t per_cta = (kRowThreads / 32) * per_warp;
  return static_cast<unsigned>(
      std::min<int64_t>((rows + per_cta - 1) / per_cta, static_cast<int64_t>(num_sms()) * 8));
}

template <int kDim, int kBits, int kGroup>
gptq_status append_as(const CacheView& c, const CacheRows& r, const void* K, int64_t ldk,
                      const void* V, int64_t ldv, bool bf16, void* K_hat, void* V_hat,
                      int32_t* info, cudaStream_t stream) {
  const dim3 grid(row_grid(r.n * c.heads, 256 / kDim)), block(kRowThreads);
  return bf16 ? launch_pdl(cache_append_kernel<kDim, kBits, kGroup, true>, grid, block, 0, stream,
                           c, r, K, ldk, V, ldv, K_hat, V_hat, info)
              : launch_pdl(cache_append_kernel<kDim, kBits, kGroup, false>, grid, block, 0, stream,
                           c, r, K, ldk, V, ldv, K_hat, V_hat, info);
}

template <int kDim, int kBits, int kGroup>
gptq_status read_as(const CacheView& c, const CacheRows& r, void* K_out, void* V_out, bool bf16,
                    int32_t* info, cudaStream_t stream) {
  const dim3 grid(row_grid(r.n * c.heads, 256 / kDim)), block(kRowThreads);
  return bf16 ? launch_pdl(cache_read_kernel<kDim, kBits, kGroup, true>, grid, block, 0, stream, c,
                           r, K_out, V_out, info)
              : launch_pdl(cache_read_kernel<kDim, kBits, kGroup, false>, grid, block, 0, stream, c,
                           r, K_out, V_out, info);
}

}  // namespace

gptq_status run_cache_append(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const void* K, int64_t ldk, const void* V, int64_t ldv, bool bf16,
                             void* K_hat, void* V_hat, int32_t* info, cudaStream_t stream) {
  return dispatch_cache(dim, bits, group, [&](auto d, auto b, auto g) {
    return append_as<d.value, b.value, g.value>(c, r, K, ldk, V, ldv, bf16, K_hat, V_hat, info,
                                                stream);
  });
}

gptq_status run_cache_read(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                           void* K_out, void* V_out, bool bf16, int32_t* info,
                           cudaStream_t stream) {
  return dispatch_cache(dim, bits, group, [&](auto d, auto b, auto g) {
    return read_as<d.value, b.value, g.value>(c, r, K_out, V_out, bf16, info, stream);
  });
}

}  // namespace gptq

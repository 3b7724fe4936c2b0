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
// Both kernels move each byte once: append reads 2 or 4 bytes a value, writes bits / 8 and, where the
// caller wants the values back, 2 or 4 more; read writes 2 or 4 for bits / 8 read. What bounds them
// is HBM for read and, for append, the instructions of the grid beside it. Measured (128 dimensions,
// 4-bit codes, one grid a row, bf16, 8 heads, page 128; fractions of the measured copy bandwidth):
//   append of 4 prompts of up to 16,384 tokens with both values back   106 us, 0.70; 69 % of the
//     issue slots, 735 warp instructions per 1024 values. Three CTAs of 256 threads an SM (80
//     registers) took 109 us when the others were tried: bounded to four 111, not bounded 125.
//   read of 16 sequences of up to 8192 tokens  97 us, 0.82. Four CTAs an SM took 100 us when 5, 6
//     and 8, and four heads a warp instead of two, were tried: 107 to 121.
// A single step (one token of 16 sequences) is 3.3 us on the device, of a read of 777 tokens 3.0:
// the launch and one trip to memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"

namespace gptq {
namespace {

constexpr int kRowThreads = 256;

// Minimum that keeps a NaN, of fp32 numbers and of pairs of bf16 numbers.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
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
  // min(0, min x) and max(0, max x) over the values of kLanes lanes; a NaN among them gives NaN.
  // bf16: both in one register, as the minima of (x, -x) pairs.
  template <int kLanes>
  __device__ __forceinline__ void range(float& lo, float& hi) const {
    if constexpr (kBf16) {
      const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
      uint32_t m = 0u, n = 0x80008000u;          // minima of x and of -x
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m = min2_nan(m, w[i]);
        n = min2_nan(n, w[i] ^ 0x80008000u);
      }
      m = min2_nan(__byte_perm(m, n, 0x5410), __byte_perm(m, n, 0x7632));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = min2_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      lo = __uint_as_float(m << 16);
      hi = -__uint_as_float(m & 0xFFFF0000u);
    } else {
      float x[8];
      get(x);
      lo = 0.f;
      float n = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        n = min_nan(n, -x[i]);
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        n = min_nan(n, __shfl_xor_sync(0xffffffffu, n, o));
      }
      hi = -n;
    }
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

// The grid of a group that spans [lo, hi], with 1 / s as the sum of two fp32 numbers: inv = 1 / s
// rounded, rest = inv (1 - s inv), so inv + rest is off by 2^-46 of itself. inv = 0 marks a NaN
// grid, and inv < 0 a scale so large or small that `rest` (or x inv) would leave fp32's range.
struct Grid {
  float s, z, inv, rest;
};
template <int kBits>
__device__ __forceinline__ Grid make_grid(float lo, float hi) {
  constexpr float kTop = static_cast<float>((1 << kBits) - 1);
  float step = __fdiv_rn(__fsub_rn(hi, lo), kTop);
  if (step == 0.f) {
    lo = -1.f;
    step = __fdiv_rn(2.f, kTop);
  }
  Grid g;
  g.s = __uint_as_float((__float_as_uint(step) + 0xFFFFu) & 0xFFFF0000u);
  if (!(fabsf(lo) <= 3.4028235e38f && hi <= 3.4028235e38f && g.s <= 3.4028235e38f))
    return {__uint_as_float(0x7FC00000u), 0.f, 0.f, 0.f};
  g.z = fminf(fmaxf(rintf(__fdiv_rn(-lo, g.s)), 0.f), kTop);
  g.inv = __frcp_rn(g.s);
  g.rest = g.inv * fmaf(-g.s, g.inv, 1.f);
  if (!(g.s > 1e-30f && g.s < 1e30f)) g.inv = -1.f;
  return g;
}

// The codes of eight values on a grid: t[i] = 1.5 2^23 + q (its low bits are the code) and
// d[i] = q - z. r = x inv + x rest, rounded in one fma, is x / s rounded, or its neighbour where
// x / s lies within 2^-44 of itself of the middle between two fp32 numbers; adding 1.5 2^23 rounds
// it to an integer, half to even. The neighbour matters only if r is a border between two codes or
// next to one. For bf16 values it never does: x / s is such a border exactly (then r is, too) or,
// as x has 8 bits and a border times s 16, at least 2^-17 of itself away. fp32 values redo the
// division where r lies within 2^-15 of a border. No code falls below 0: lo itself gives
// rint(lo / s) + rint(-lo / s) = 0.
template <int kBits, bool kBf16>
__device__ __forceinline__ void make_codes(const Grid& g, float (&x)[8], float (&t)[8],
                                           float (&d)[8]) {
  constexpr float kTop = static_cast<float>((1 << kBits) - 1), kMagic = 12582912.f;
  const float bias = kMagic + g.z;
  float near = 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fmaf(x[i], g.inv, x[i] * g.rest);
    const float k = r + kMagic - kMagic;
    if (!kBf16) near = fminf(near, fabsf(fabsf(r - k) - 0.5f));
    d[i] = fminf(k, kTop - g.z);
    t[i] = d[i] + bias;
  }
  if (g.inv <= 0.f || near < 3e-5f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = fminf(fmaxf(rintf(__fdiv_rn(x[i], g.s)) + g.z, 0.f), kTop);
      t[i] = kMagic + (g.inv == 0.f ? 0.f : q);
      d[i] = g.inv == 0.f ? 0.f : q - g.z;
    }
  }
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// The rows of a call, walked by warps. A row's vector of one head takes kDim / 8 consecutive lanes,
// eight values each; a warp takes kUnroll * 256 / kDim heads (blockIdx.y: which) of each token of
// a run of consecutive tokens, so the sequence and the page are looked up where they change, not
// for each token.
constexpr int kUnroll = 2;   // K and V of two heads: four grids a lane, which four lanes share

struct Walk {
  int64_t tok, stop;            // this warp's tokens
  int64_t first = 0, end = -1;  // rows of the current sequence (end - 1 its last)
  int64_t shift = 0;            // position of row i of it: i + shift
  const int32_t* table = nullptr;
  int32_t page = -1;
  bool fresh = true;            // the page must be looked up

  __device__ __forceinline__ Walk(const CacheRows& rows) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    tok = rows.n / warps * w + min(rows.n % warps, w);
    stop = tok + rows.n / warps + (w < rows.n % warps ? 1 : 0);
  }
  // Moves to the sequence and page of row `tok` (the whole warp); false behind the last sequence.
  __device__ __forceinline__ bool at(const CacheView& c, const CacheRows& rows, int32_t* info) {
    if (tok >= end) {
      const int64_t b = find_sequence(rows, tok);
      if (b >= rows.batch) return false;
      first = rows.starts ? __ldg(rows.starts + b) : b;
      end = rows.starts ? __ldg(rows.starts + b + 1) : b + 1;
      shift = static_cast<int64_t>(__ldg(rows.lengths + b)) - end;
      table = rows.table + b * rows.ld_table;
      fresh = true;
    }
    const int64_t pos = tok + shift;
    if (tok < first) {
      page = -1;
    } else if (fresh || page < 0 || (pos & ((1 << c.page_shift) - 1)) == 0) {
      page = find_page(c, table, pos, info);
      fresh = false;
    }
    return true;
  }
  __device__ __forceinline__ int offset(const CacheView& c) const {
    return static_cast<int>(tok + shift) & ((1 << c.page_shift) - 1);
  }
};

template <int kDim, int kBits, int kGroup, bool kXBf16>
__global__ void __launch_bounds__(kRowThreads, 3)
cache_append_kernel(const CacheView c, const CacheRows rows, const void* __restrict__ K,
                    int64_t ldk, const void* __restrict__ V, int64_t ldv, void* K_hat, void* V_hat,
                    int32_t* info) {
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes, kGroups = kDim / kGroup;
  constexpr int kElem = kXBf16 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int head0 = blockIdx.y * (kUnroll * kPer) + sub;
  Walk walk(rows);
  for (; walk.tok < walk.stop; ++walk.tok) {
    // the values first: they do not depend on where they go
    const uint8_t* src[2] = {static_cast<const uint8_t*>(K) + walk.tok * ldk * kElem,
                             static_cast<const uint8_t*>(V) + walk.tok * ldv * kElem};
    Eight<kXBf16> in[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        in[u][h].load(src[h] + (min(head0 + u * kPer, c.heads - 1) * kDim + 8 * l) * kElem);
    if (!walk.at(c, rows, info)) return;      // behind the last sequence: left as it is
    if (walk.page < 0) continue;              // no page: left as it is
    // the four grids of each group: its lanes share the divisions, four lanes one grid each
    float lo[2 * kUnroll], hi[2 * kUnroll];
#pragma unroll
    for (int i = 0; i < 2 * kUnroll; ++i)
      in[i / 2][i % 2].template range<kGroup / 8>(lo[i], hi[i]);
    const bool k1 = lane & 1, k2 = lane & 2;
    const Grid mine = make_grid<kBits>(k2 ? (k1 ? lo[3] : lo[2]) : (k1 ? lo[1] : lo[0]),
                                       k2 ? (k1 ? hi[3] : hi[2]) : (k1 ? hi[1] : hi[0]));
    const int64_t row0 = cache_row(c, walk.page, 0, walk.offset(c));
    uint8_t* hats[2] = {static_cast<uint8_t*>(K_hat), static_cast<uint8_t*>(V_hat)};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint8_t* codes = c.half[h].codes + row0 * (kDim * kBits / 8);
      uint16_t* scales = c.half[h].scales + row0 * kGroups;
      uint8_t* zeros = c.half[h].zeros + row0 * kGroups;
      uint8_t* hat = hats[h] + walk.tok * c.heads * (kDim * kElem);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int head = head0 + u * kPer;
        const int from = (lane & ~3) + 2 * u + h;
        const Grid g{__shfl_sync(0xffffffffu, mine.s, from), __shfl_sync(0xffffffffu, mine.z, from),
                     __shfl_sync(0xffffffffu, mine.inv, from),
                     __shfl_sync(0xffffffffu, mine.rest, from)};
        if (head >= c.heads) continue;
        const uint32_t at = static_cast<uint32_t>(head) << c.page_shift;   // rows after row0
        float x[8], q[8], d[8];
        in[u][h].get(x);
        make_codes<kBits, kXBf16>(g, x, q, d);
        uint8_t* dst = codes + static_cast<uint64_t>(at) * (kDim * kBits / 8) + l * kBits;
        if constexpr (kBits == 4) {
          *reinterpret_cast<uint32_t*>(dst) =
              low_bytes(q[0], q[2], q[4], q[6]) | low_bytes(q[1], q[3], q[5], q[7]) << 4;
        } else {
          *reinterpret_cast<uint2*>(dst) = make_uint2(low_bytes(q[0], q[1], q[2], q[3]),
                                                      low_bytes(q[4], q[5], q[6], q[7]));
        }
        if (l % (kGroup / 8) == 0) {
          const uint64_t gi = static_cast<uint64_t>(at) * kGroups + l / (kGroup / 8);
          scales[gi] = static_cast<uint16_t>(__float_as_uint(g.s) >> 16);
          zeros[gi] = static_cast<uint8_t>(int_bits(g.z));
        }
        if (hats[h] != nullptr) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(g.s, d[i]);
          store8<kXBf16>(hat + (head * kDim + 8 * l) * kElem, y);
        }
      }
    }
  }
}

// The values of the last positions of every sequence; a position without a page reads as 0.
template <int kDim, int kBits, int kGroup, bool kYBf16>
__global__ void __launch_bounds__(kRowThreads, 4)
cache_read_kernel(const CacheView c, const CacheRows rows, void* __restrict__ K_out,
                  void* __restrict__ V_out, int32_t* info) {
  constexpr int kLanes = kDim / 8, kPer = 32 / kLanes, kGroups = kDim / kGroup;
  constexpr int kElem = kYBf16 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
  const int head0 = blockIdx.y * (kUnroll * kPer) + sub;
  Walk walk(rows);
  for (; walk.tok < walk.stop; ++walk.tok) {
    if (!walk.at(c, rows, info)) return;
    if (walk.tok < walk.first) continue;
    uint32_t w[kUnroll][2][kBits / 4];
    uint32_t s[kUnroll][2], z[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = min(head0 + u * kPer, c.heads - 1);
      const int64_t at = cache_row(c, max(walk.page, 0), head, walk.offset(c));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* codes = c.half[h].codes + at * (kDim * kBits / 8) + l * kBits;
        const int64_t gi = at * kGroups + l / (kGroup / 8);
        if constexpr (kBits == 4) {
          w[u][h][0] = __ldg(reinterpret_cast<const uint32_t*>(codes));
        } else {
          *reinterpret_cast<uint2*>(w[u][h]) = __ldg(reinterpret_cast<const uint2*>(codes));
        }
        s[u][h] = __ldg(c.half[h].scales + gi);
        z[u][h] = __ldg(c.half[h].zeros + gi);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* out = static_cast<uint8_t*>(h == 0 ? K_out : V_out);
        const int head = head0 + u * kPer;
        if (out == nullptr || head >= c.heads) continue;
        uint8_t* dst = out + ((walk.tok * c.heads + head) * kDim + 8 * l) * kElem;
        if constexpr (kBits == 4 && kYBf16) {
          // two at a time: 128 + code and 128 + z are bf16 numbers, their difference is exact, and
          // its product with the scale is rounded once, as that of fp32 numbers rounded to bf16
          // would be (8 times 4 bits are exact there)
          const uint32_t s2 = s[u][h] * 0x00010001u, z2 = (0x4300u + z[u][h]) * 0x00010001u;
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)       // values i and i + 4
            v[i] = mul_bf16x2(
                sub_bf16x2(((w[u][h][0] >> (4 * i)) & 0x000F000Fu) | 0x43004300u, z2), s2);
          uint4 y = make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                               __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
          if (walk.page < 0) y = make_uint4(0, 0, 0, 0);
          __stcs(reinterpret_cast<uint4*>(dst), y);
          continue;
        }
        const float sf = bf16_bits_to_float(s[u][h]);
        const float zf = __uint_as_float(0x4B000000u | z[u][h]);     // 2^23 + z
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t q = kBits == 4 ? (w[u][h][0] >> (4 * i)) & 15u
                                        : (w[u][h][i / 4] >> (8 * (i % 4))) & 255u;
          y[i] = __fmul_rn(sf, __fsub_rn(__uint_as_float(0x4B000000u | q), zf));
        }
        if (walk.page < 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = 0.f;
        }
        store8<kYBf16>(dst, y);
      }
  }
}

// CTAs of a kernel that an SM holds at once, cached per device.
template <auto kKernel>
int resident_ctas() {
  static std::atomic<int> cache[64] = {};
  int dev = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  if ((per = cache[dev].load(std::memory_order_relaxed)) == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kKernel, kRowThreads, 0) != cudaSuccess)
      per = 1;
    per = std::max(per, 1);
    cache[dev].store(per, std::memory_order_relaxed);
  }
  return per;
}

// A warp per token and head block while that gives no more CTAs than the device holds at once;
// then as many as it holds, each warp with a longer run.
template <auto kKernel>
dim3 row_grid(const CacheView& c, int64_t n, int per_warp) {
  const int64_t y = (c.heads + per_warp - 1) / per_warp;
  const int64_t x = (n + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t most =
      std::max<int64_t>(static_cast<int64_t>(num_sms()) * resident_ctas<kKernel>() / y, 1);
  return dim3(static_cast<unsigned>(std::min(x, most)), static_cast<unsigned>(y));
}

template <auto kKernel, typename... Args>
gptq_status launch_rows(const CacheView& c, const CacheRows& r, int per_warp, cudaStream_t stream,
                        Args... args) {
  return launch_pdl(kKernel, row_grid<kKernel>(c, r.n, per_warp), dim3(kRowThreads), 0, stream, c,
                    r, args...);
}

template <int kDim, int kBits, int kGroup>
gptq_status append_as(const CacheView& c, const CacheRows& r, const void* K, int64_t ldk,
                      const void* V, int64_t ldv, bool bf16, void* K_hat, void* V_hat,
                      int32_t* info, cudaStream_t stream) {
  constexpr int kPerWarp = kUnroll * 256 / kDim;
  return bf16 ? launch_rows<cache_append_kernel<kDim, kBits, kGroup, true>>(
                    c, r, kPerWarp, stream, K, ldk, V, ldv, K_hat, V_hat, info)
              : launch_rows<cache_append_kernel<kDim, kBits, kGroup, false>>(
                    c, r, kPerWarp, stream, K, ldk, V, ldv, K_hat, V_hat, info);
}

template <int kDim, int kBits, int kGroup>
gptq_status read_as(const CacheView& c, const CacheRows& r, void* K_out, void* V_out, bool bf16,
                    int32_t* info, cudaStream_t stream) {
  constexpr int kPerWarp = kUnroll * 256 / kDim;
  return bf16 ? launch_rows<cache_read_kernel<kDim, kBits, kGroup, true>>(c, r, kPerWarp, stream,
                                                                         K_out, V_out, info)
              : launch_rows<cache_read_kernel<kDim, kBits, kGroup, false>>(c, r, kPerWarp, stream,
                                                                          K_out, V_out, info);
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

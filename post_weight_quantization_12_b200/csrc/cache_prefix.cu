// Attention of many rows over one common sequence of the quantized cache, on the tcgen05 tensor
// cores: the shared prefix of a batch.
//
// All query rows of a cache head (tokens x query heads of it) meet the same keys, so the codes are
// unpacked once per 256 rows, into fp16 images that stay in shared memory:
//   S = Q K^T     128 rows x 128 tokens, Q and the image of K both K-major
//   P = 2^(x + e - M) fp16, written over S in tensor memory, where the second product reads it
//   O += P V      128 rows x D, the image of V with the dimensions contiguous (MN-major)
// K: where a row has one grid, its image is q - z, exact, and the score is x = S times the token's
// scale, which the softmax groups read from shared memory: a rounding of the keys' images would move
// a score by 2^-12 of sum |q k|, which is more than the output's own rounding where a few channels of
// the keys stand out. Where a row has several grids no factor can be taken out: s' (q - z) needs up
// to 16 bits and becomes the sum of two fp16 numbers, the rounded one and what it left, in two images
// and twice the products (one buffer instead of two then: 128 rows x 8 heads x 4 over 32,768 tokens
// of 4-bit codes, group 32, 192 us, and 159 with one image; 96 rows x 32 heads over 8192 tokens 160
// and 153). s' = s 2^(T - E), E the largest exponent among the scales of 32 tokens, so that the
// largest image stays below 65504.
// V: the rounded image alone, throughout; its error stays 2^-12 of the value. Its power of two e goes
// into the exponent of P, per 32 tokens, and per token where scales lie further apart, so a value far
// above the others takes no bits of theirs unless the row gives it weight. Groups whose values are
// all zero, whose grid is [-1, 1], do not count for E.
// M, and m for the sum of 2^(x - m), are kept from tile to tile; the operands are made with the M at
// hand and taken if the sum of 32 stays below 65000 (fp16 ends at 65504). Otherwise, and where m has
// lost touch, the rows find their largest, M is set 2^7 below it, and O is rescaled in tensor memory:
// a few times in all.
//
// A CTA (one per SM) holds two row tiles of 128 and goes over a run of 128-token tiles:
//   warp 0           issues the products: PV(0), QK(0) of the next tile, PV(1), QK(1), so one
//                    tile's softmax runs under the other's products (the oldest warp: an SM's
//                    scheduler lets it go first, and every other role waits for it)
//   warps 4-11, 12-19  softmax of row tile 0 and 1, two threads a row: each takes half of the
//                    tokens, and half of the dimensions when they bring Q in and write the results
//   warps 20-23, 24-27  unpack K and V of the next tiles into two buffers each, loads a tile ahead;
//                    those of V tell the softmax groups what the images lack
// With no more than 128 rows in an item, both softmax groups take the same rows and every other
// token tile. The runs' results (row, fp32, with its log-sum) are joined by cache_merge_kernel.
//
// What bounds it. Two row tiles: the chain of a step. Both products read operands from shared or
// tensor memory (about 840 cycles of S, 700 of O a row tile and token tile), then come the hand-overs
// between them and the softmax: 128 sequences x 8 heads of 4-bit codes x 4 query heads, prefix
// 32,768, 146 us in all, 475 TFLOP/s (0.29 of the measured bf16 rate); this kernel 100 us, tensor pipe
// 37 % busy while an SM works. One row tile: unpacking: 96 sequences x 32 heads of 8-bit codes, prefix
// 8192, 131 us in all, this kernel 52 us. The rest of both is the sequences' own level, the merge
// (about 9 us) and what lies between them. The keys' factors, read by every softmax thread for every
// token, and the second reference cost about 10 us in the first case and 4 in the second, over images
// that carried the scales.
// Tried and slower (first case, while the images carried the scales): S in two halves of the tokens
// (140 to 163 us), the eight unpacking warps on K and V alike (140 to 146 us). Unpackers of K and V
// apart: 144 to 139 us. Copies of codes by half sectors: 207 us in the second case where whole ones
// took 140. V's factor a token's as well as K's, for images of V without scales: 159 us and 128, where
// a power of two per 32 tokens takes 149 and 127.
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace gptq {
namespace {

constexpr int kTok = 128;                  // tokens of a tile
constexpr int kSm0 = 4;                    // the first softmax warp
constexpr int kDq0 = 20, kDqWarps = 4;     // the unpacking warps of K; those of V follow
constexpr int kDqRows = kTok / kDqWarps;   // rows of a tile that one of them takes: one a lane
static_assert(kDqRows == 32, "a lane a row");
constexpr int kMmaWarp = 0;
constexpr int kThreads = 32 * (kDq0 + 2 * kDqWarps);
constexpr float kNegInf = -INFINITY;
// Registers a thread: what the block is launched with (65,536 over its threads), and what the four
// warps in front give to the softmax groups' sixteen, whose 64 products a row and thread do not fit
// otherwise (first case above: 153 us without, 148 with; 88 registers with less for unpacking 151).
constexpr int kLaunchRegs = 72, kMmaRegs = 40, kSoftmaxRegs = 80;
static_assert(kMmaRegs + 4 * kSoftmaxRegs + 2 * kLaunchRegs <= 7 * kLaunchRegs);

enum Image { kPlainImage, kOneImage, kTwoImages };      // see the unpacking

struct Prefix {
  CacheView cache;
  const int32_t* table;
  int64_t len;
  const __nv_bfloat16* q;
  int64_t ldq, n;
  int ratio;
  float scale_log2;
  int row_items;                // items of up to 256 rows of a head
  int tiles, splits;
  int units;                    // heads * row_items * splits
  float* part;                  // [units][2][128][D]
  float* part_lse;              // [units][2][128]
  int32_t* info;
};

// What the warps share beside the tiles.
struct Side {
  uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], g_full[2];
  uint64_t s_full[2], p_full[2], pv_done[2], mma_done;
  // Of step s in slot s % 2. What the images of its tokens lack: K's factor, a token's (with 2^-14 in
  // it), or where a row has several grids 32 tokens'; V's power of two, 32 tokens' (as a number; -inf
  // where they have none in common) and a token's (bf16 bits).
  alignas(16) uint32_t valid[2][4];        // tokens that count
  alignas(16) float k_scale[2][kTok];
  alignas(16) float v_exp[2][4];
  uint16_t v_scale[2][kTok];
  float row_x[2][128];                     // of (row tile, row): what its halves exchange
  uint32_t tmem_base;
  volatile int abort;
};
constexpr float kFirst = -3e38f;           // a reference before the first score
constexpr float kMostSum = 65000.f;        // of 32 operands, each below 65504
constexpr float kMostLog = 15.9882f;       // its logarithm

template <int D, int BITS>
struct Smem {
  static constexpr int kTileBytes = kTok * D * 2;         // an operand tile: D / 64 halves of 16 KB
  static constexpr int kCodeBytes = kTok * D * BITS / 8;  // a tile's codes of K or V
  static constexpr int kAhead = BITS == 4 ? 2 : 1;        // steps whose codes are on the way
  // Q 0, Q 1, K 0, K 1, V 0, V 1, codes, then Side
  static constexpr int kSide = 6 * kTileBytes + kAhead * 2 * kCodeBytes;
  static constexpr int kBytes = kSide + static_cast<int>(sizeof(Side));
  static_assert(kBytes <= 227 * 1024);
};

__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
               ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// All four warps of a group, at the same place.
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Waits for the tensor-memory loads issued so far; the registers are named so that nothing that
// uses them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                 "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                 "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]),
                 "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ float pow2(int e) {          // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// One unit of work: an item (a cache head and up to 256 of its rows) and a run of token tiles.
struct Unit {
  int head, tile0, steps;       // steps: token tiles
  int row0, rows;               // rows of the item
  bool two;                     // two row tiles; else both softmax groups share one
};
__device__ __forceinline__ Unit get_unit(const Prefix& a, int u) {
  Unit w;
  const uint32_t item = static_cast<uint32_t>(u) / static_cast<uint32_t>(a.splits);
  const uint32_t split = static_cast<uint32_t>(u) - item * a.splits;
  w.head = static_cast<int>(item / static_cast<uint32_t>(a.row_items));
  w.row0 = static_cast<int>(item - w.head * static_cast<uint32_t>(a.row_items)) * 256;
  w.rows = min(static_cast<int>(a.n) * a.ratio - w.row0, 256);
  w.two = w.rows > 128;
  // tiles <= 2^23 and splits <= 2 SMs: the products fit in 32 bits
  const uint32_t tiles = static_cast<uint32_t>(a.tiles), splits = static_cast<uint32_t>(a.splits);
  w.tile0 = static_cast<int>(tiles * split / splits);
  w.steps = static_cast<int>(tiles * (split + 1) / splits) - w.tile0;
  return w;
}
// The r-th step of softmax group i, and how many it has.
__device__ __forceinline__ int step_of(const Unit& w, int i, int r) { return w.two ? r : 2 * r + i; }
__device__ __forceinline__ int steps_of(const Unit& w, int i) {
  return w.two ? w.steps : (w.steps + 1 - i) / 2;
}

template <int D, int BITS, int GROUP>
__global__ void __launch_bounds__(kThreads, 1)
cache_prefix_kernel(const Prefix a) {
  constexpr int G = D / GROUP, RB = D * BITS / 8;
  using SM = Smem<D, BITS>;
  constexpr int kTile = SM::kTileBytes;
  // exponent of the largest scale in a token's images: below 2^(kTop + 1) (2^BITS - 1) < 65504
  constexpr int kTop = BITS == 4 ? 11 : 7;
  // K's tiles: two buffers of images, or one of two images that add up to the values
  constexpr bool kPair = G > 1;
  auto k_buffer = [](uint32_t gs) -> int { return kPair ? 0 : gs & 1; };
  auto k_phase = [](uint32_t gs) -> uint32_t { return kPair ? gs & 1u : (gs >> 1) & 1u; };
  extern __shared__ __align__(1024) uint8_t smem[];    // (operand tiles: multiples of 1024 bytes)
  auto q_tile = [&](int i) { return smem + i * kTile; };
  auto k_tile = [&](int b) { return smem + (2 + b) * kTile; };
  auto v_tile = [&](int b) { return smem + (4 + b) * kTile; };
  auto code_slot = [&](int b, int h) { return smem + 6 * kTile + (2 * b + h) * SM::kCodeBytes; };
  Side& sh = *reinterpret_cast<Side*>(smem + SM::kSide);
  uint64_t *q_full = sh.q_full, *k_full = sh.k_full, *k_empty = sh.k_empty, *v_full = sh.v_full;
  uint64_t *v_empty = sh.v_empty, *g_full = sh.g_full, *s_full = sh.s_full, *p_full = sh.p_full;
  uint64_t* pv_done = sh.pv_done;
  volatile int* abort_flag = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 256);
      mbar_init(&k_full[b], 32 * kDqWarps);
      mbar_init(&k_empty[b], 1);
      mbar_init(&v_full[b], 32 * kDqWarps);
      mbar_init(&v_empty[b], 1);
      mbar_init(&g_full[b], 32 * kDqWarps);
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], 256);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  auto tm_s = [&](int i) { return tmem + 128 * i; };   // S; P over the first half of each half
  auto tm_o = [&](int i) { return tmem + 256 + D * i; };
  // What this kernel reads (queries, cache) was complete before the kernel in front of it, which
  // waited for it, let this one start; the results of that kernel are not read here. So the wait for
  // it comes at the end, where it keeps the order for the kernel that follows.
  griddep_launch_dependents();
  int32_t* info = a.info;

  if (warp >= kSm0 && warp < kDq0) {
    registers_up<kSoftmaxRegs>();
    // ---- softmax group i: threads r and r + 128 of it share row r, tokens 64 hf .. of each tile ----
    const int i = (warp - kSm0) >> 3, hf = ((warp - kSm0) >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t pair = 2 + i * 4 + (warp & 3);       // the barrier of the two warps of a row
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    // the other half's value: one place for both, first for the one, then for the other
    auto exchange = [&](float x) -> float {
      if (hf == 0) sh.row_x[i][r] = x;
      pair_sync();
      const float y = sh.row_x[i][r];
      pair_sync();
      if (hf == 1) sh.row_x[i][r] = x;
      pair_sync();
      const float z = sh.row_x[i][r];
      pair_sync();
      return hf == 0 ? z : y;
    };
    uint32_t c_step = 0;        // steps of this group so far
    uint32_t g_base = 0;        // steps of the units before
    bool ok = true;
    for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
      const Unit w = get_unit(a, u);
      const int row = w.two ? i * 128 + r : r;       // of the item
      const bool live = row < w.rows;
      const int my_steps = steps_of(w, i);
      // Q: fp16 after a power of two per row (group 1 writes its own tile only)
      float row_c = 0.f;
      {
        uint4 raw[D / 16];
        float top = 0.f;
        if (live) {
          const int j = w.row0 + row;
          const int tok = static_cast<int>(static_cast<uint32_t>(j) / static_cast<uint32_t>(a.ratio));
          const uint4* src = reinterpret_cast<const uint4*>(
              a.q + tok * a.ldq +
              (static_cast<int64_t>(w.head) * a.ratio + (j - tok * a.ratio)) * D + hf * (D / 2));
#pragma unroll
          for (int c = 0; c < D / 16; ++c) raw[c] = __ldg(src + c);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[k] << 16)),
                                     fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
          }
        } else {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) raw[c] = make_uint4(0, 0, 0, 0);
        }
        top = fmaxf(top, exchange(top));
        const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
        // a negative scale goes into Q, so the largest score is the largest product
        const float up = (e > 127 ? 1.f : pow2(14 - e)) * (a.scale_log2 < 0.f ? -1.f : 1.f);
        // (2^14 makes up for the 2^-14 of the keys' factors; never 0: a token that does not count
        // has a product of -inf)
        row_c = fmaxf((e > 127 ? 16384.f : pow2(e)) * fabsf(a.scale_log2), 1.17549435e-38f);
        if (w.two || i == 0) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              f[2 * k] = __uint_as_float(x[k] << 16) * up;
              f[2 * k + 1] = __uint_as_float(x[k] & 0xFFFF0000u) * up;
            }
            // in the order that 4-bit codes come out of their word; every other one 16 times too
            // large, if its image has no scale
            if (BITS == 4 && G == 1) {
              f[1] *= 0.0625f;
              f[3] *= 0.0625f;
              f[5] *= 0.0625f;
              f[7] *= 0.0625f;
            }
            const uint4 h = BITS == 4 ? make_uint4(half2_bits(f[0], f[4]), half2_bits(f[1], f[5]),
                                                   half2_bits(f[2], f[6]), half2_bits(f[3], f[7]))
                                      : make_uint4(half2_bits(f[0], f[1]), half2_bits(f[2], f[3]),
                                                   half2_bits(f[4], f[5]), half2_bits(f[6], f[7]));
            const int chunk = hf * (D / 16) + c;        // of eight dims
            *reinterpret_cast<uint4*>(q_tile(i) + r * 128 + (chunk >> 3) * (kTok * 128) +
                                      (((chunk & 7) ^ (r & 7)) << 4)) = h;
          }
          fence_proxy_async_smem();
          mbar_arrive(&q_full[i]);
        }
      }
      // references of the row, and this half's share of the sum of 2^(x - m)
      float m = kFirst, M = kFirst, l = 0.f;
      for (int k = 0; k < my_steps; ++k, ++c_step) {
        const uint32_t gs = g_base + step_of(w, i, k);
        const int slot = gs & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&g_full[slot], (gs >> 1) & 1u, abort_flag,
                                                       info) &&
                                     mbar_wait_bounded(&s_full[i], c_step & 1, abort_flag, info));
        tc_fence_after();
        const uint32_t ts = tm_s(i) + lane_base + 64 * hf;
        const float* k_scale = sh.k_scale[slot] + (G == 1 ? 64 : 2) * hf;
        const float2 e_v = *reinterpret_cast<const float2*>(&sh.v_exp[slot][2 * hf]);
        const uint2 vm = *reinterpret_cast<const uint2*>(&sh.valid[slot][2 * hf]);
        if ((vm.x & vm.y) != 0xFFFFFFFFu) {
          // tokens that do not count: their products become -inf
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            const uint32_t mask = (c < 4 ? vm.x : vm.y) >> (8 * (c & 3));
            uint32_t x[8];
            tmem_ld_32x32b_x8(ts + 8 * c, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int t = 0; t < 8; ++t)
              if (!(mask >> t & 1u)) x[t] = __float_as_uint(kNegInf);
            tmem_st_32x32b_x8(ts + 8 * c, x);
          }
          tmem_wait_st();
        }
        // operands 2^(x + e - M) of 32 tokens at a time (e: V's power of two) and their sum
        uint32_t p[2][16];
        float sum[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float c = G == 1 ? row_c : fmaxf(row_c * k_scale[hh], 1.17549435e-38f);
          const float ref = (hh ? e_v.y : e_v.x) - M;
          const float2 c2 = make_float2(c, c), ref2 = make_float2(ref, ref);
          float2 sa = make_float2(0.f, 0.f), sb = sa;
          uint32_t v[32];
          tmem_ld_32x32b_x32(ts + 32 * hh, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int t = 0; t < 32; t += 4) {
            float2 xa = make_float2(__uint_as_float(v[t]), __uint_as_float(v[t + 1]));
            float2 xb = make_float2(__uint_as_float(v[t + 2]), __uint_as_float(v[t + 3]));
            if constexpr (G == 1) {
              const float4 ks = *reinterpret_cast<const float4*>(k_scale + 32 * hh + t);
              xa = mul2(xa, make_float2(ks.x, ks.y));
              xb = mul2(xb, make_float2(ks.z, ks.w));
            }
            const float2 ya = fma2(xa, c2, ref2), yb = fma2(xb, c2, ref2);
            const float2 pa = make_float2(ex2(ya.x), ex2(ya.y));
            const float2 pb = make_float2(ex2(yb.x), ex2(yb.y));
            sa = add2(sa, pa);
            sb = add2(sb, pb);
            p[hh][t / 2] = half2_bits(pa.x, pa.y);
            p[hh][t / 2 + 1] = half2_bits(pb.x, pb.y);
          }
          sa = add2(sa, sb);
          sum[hh] = sa.x + sa.y;
        }
        // Taken as they are if M allows them and the weights are theirs times 2^(M - e - m), a power
        // that neither has lost them (a weight below 2^-62 of the row's unit may be 0) nor is beyond
        // fp32. Both warps of the rows go one way (or out, after an error).
        const bool over = sum[0] > kMostSum || sum[1] > kMostSum;
        const float d0 = M - e_v.x - m, d1 = M - e_v.y - m;
        if (!named_barrier_or(pair, 64, !ok || over || d0 > 64.f || d1 > 64.f)) {
          l += fmaf(sum[0], ex2(d0), sum[1] * ex2(d1));
          // written over the S that they come from: 64 tokens' over the first 32 columns of their
          // half
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) x[t] = p[c / 2][8 * (c & 1) + t];
            tmem_st_32x32b_x8(ts + 8 * c, x);
          }
        } else {
          if (named_barrier_or(pair, 64, !ok)) {
            ok = false;
            break;
          }
          const uint16_t* v_scale = sh.v_scale[slot] + 64 * hf;
          // score and power of two of token t, whose product is v
          auto score = [&](uint32_t v, int t) {
            return G == 1 ? __uint_as_float(v) * k_scale[t] * row_c
                          : __uint_as_float(v) * fmaxf(row_c * k_scale[t >> 5], 1.17549435e-38f);
          };
          auto power = [&](int t) { return static_cast<float>(v_scale[t] >> 7) - 127.f; };
          float top = kNegInf, top_M = kNegInf;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[8];
            tmem_ld_32x32b_x8(ts + 8 * c, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              const float y = score(x[t], 8 * c + t);
              top = fmaxf(top, y);
              top_M = fmaxf(top_M, y + power(8 * c + t));
            }
          }
          top = fmaxf(top, exchange(top));
          top_M = fmaxf(top_M, exchange(top_M));
          const float any_over = over ? 1.f : 0.f;
          const bool raise = fmaxf(any_over, exchange(any_over)) > 0.f || top_M > M + kMostLog;
          if (top > m + 64.f) {
            l *= ex2(m - top);
            m = top;
          }
          // a new reference lies 2^7 below the largest operand
          const float M_new = raise ? fmaxf(M, top_M - 7.f) : M;
          const float f = ex2(M - M_new);
          M = M_new;
          if (k > 0) {
            // O of the steps so far: the products that made it are complete (they were issued
            // before this step's S)
            const uint32_t to = tm_o(i) + lane_base + hf * (D / 2);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t x[8];
              tmem_ld_32x32b_x8(to + 8 * c, x);
              tmem_wait_ld(x);
#pragma unroll
              for (int t = 0; t < 8; ++t) x[t] = __float_as_uint(__uint_as_float(x[t]) * f);
              tmem_st_32x32b_x8(to + 8 * c, x);
            }
          }
          // (16 tokens' operands go over the S of tokens already read)
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[8], y[8], z[8];
            tmem_ld_32x32b_x8(ts + 16 * c, x);
            tmem_ld_32x32b_x8(ts + 16 * c + 8, y);
            tmem_wait_ld(x);
            tmem_wait_ld(y);
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
              const int at = 16 * c + t;
              const float s0 = score(t < 8 ? x[t] : y[t - 8], at);
              const float s1 = score(t < 8 ? x[t + 1] : y[t - 7], at + 1);
              l += ex2(s0 - m) + ex2(s1 - m);
              z[t / 2] = half2_bits(ex2(s0 + (power(at) - M)), ex2(s1 + (power(at + 1) - M)));
            }
            tmem_st_32x32b_x8(ts + 8 * c, z);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[i]);
      }
      g_base += w.steps;
      if (!ok) break;
      // the row's result
      const int64_t slot = 2 * static_cast<int64_t>(u) + i;
      float lse = kNegInf;
      if (my_steps > 0) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&pv_done[i], (c_step - 1) & 1, abort_flag, info));
        if (named_barrier_or(pair, 64, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        l += exchange(l);
        lse = l == 0.f ? kNegInf : m + log2f(l);
        const float f = l == 0.f ? 0.f : 1.f / l;
        // 2^(M - m) as a square: M and m may lie further apart than one factor reaches
        const float f2 = ex2(0.5f * (M - m));
        float* dst = a.part + (slot * 128 + r) * D + hf * (D / 2);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t x[8];
          tmem_ld_32x32b_x8(tm_o(i) + lane_base + hf * (D / 2) + 8 * c, x);
          tmem_wait_ld(x);
#pragma unroll
          for (int t = 0; t < 8; ++t) x[t] = __float_as_uint(__uint_as_float(x[t]) * f * f2 * f2);
          if (live) {
            uint4 lo, hi;
            if constexpr (BITS == 4) {      // columns hold dims 0 4 1 5 2 6 3 7 of each eight
              lo = make_uint4(x[0], x[2], x[4], x[6]);
              hi = make_uint4(x[1], x[3], x[5], x[7]);
            } else {
              lo = make_uint4(x[0], x[1], x[2], x[3]);
              hi = make_uint4(x[4], x[5], x[6], x[7]);
            }
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                         ::"l"(dst + 8 * c), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
                           "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w) : "memory");
          }
        }
        tc_fence_before();
      }
      if (live && hf == 0) a.part_lse[slot * 128 + r] = lse;
    }
  } else if (warp >= kDq0) {
    // ---- unpack: lane t of a row takes 32 dims (8-bit codes: two pieces of 16, half a row apart,
    // so that the lanes of a load meet whole sectors); a warp takes 32 rows of the tile ----
    constexpr int LPR = D / 32, RPI = 32 / LPR;                // lanes a row, rows an access
    constexpr int KI = kDqRows / RPI;
    constexpr int kVec = BITS == 4 ? 1 : 2;                    // 16-byte loads of a lane's codes
    // h: 0 unpacks K, 1 unpacks V; each group keeps its own count of steps
    const int h = warp >= kDq0 + kDqWarps, dw = warp - kDq0 - h * kDqWarps;
    const int t = lane % LPR, g = lane / LPR;
    const CacheHalf half = h ? a.cache.half[1] : a.cache.half[0];
    // first dim of piece v of this lane
    auto dim_of = [&](int v) { return BITS == 4 ? 32 * t : 16 * t + v * (D / 2); };
    constexpr int kS = (G + 1) / 2;      // words of a row's scales
    // The steps, unit by unit. Three things run ahead of the unpacking, so that none waits for
    // another's loads: the page lookup of step gs + kAhead + 1, the codes of step gs + kAhead and
    // the grids of step gs + 1.
    struct At {
      int u, left, tile, head;       // left: steps to come in this unit
    };
    auto enter = [&](At& x, int u) {
      x.u = u;
      if (u < a.units) {
        const Unit w = get_unit(a, u);
        x.left = w.steps;
        x.tile = w.tile0;
        x.head = w.head;
      }
    };
    auto next = [&](At& x) {
      if (x.u >= a.units) return;
      ++x.tile;
      if (--x.left == 0) enter(x, x.u + gridDim.x);
    };
    // page table entry of the warp's row `lane` of a step, -1 past the end; and from it the row's
    // number in the cache, -1 if the token does not count
    int32_t entry = -1, entry_off = 0, entry_head = 0;
    bool entry_in = false;
    auto look = [&](const At& x) {
      const int pos = x.tile * kTok + dw * kDqRows + lane;      // prefix_len <= 2^30
      entry_in = x.u < a.units && pos < static_cast<int>(a.len);
      entry = entry_in ? __ldg(a.table + (pos >> a.cache.page_shift)) : -1;
      entry_off = pos & ((1 << a.cache.page_shift) - 1);
      entry_head = x.head;
    };
    auto resolve = [&]() -> int64_t {
      if (entry >= 0 && entry < a.cache.pages)
        return cache_row(a.cache, entry, entry_head, entry_off);
      if (entry_in) record_info(info, GPTQ_INFO_BAD_PAGE);
      return -1;
    };
    // codes on their way to the slots: each lane copies what it will unpack
    auto copy_codes = [&](int64_t row, int b) {
      uint8_t* dst = code_slot(b, h) + dw * (SM::kCodeBytes / kDqWarps) + lane * 16;
      const uint8_t* base = half.codes + 16 * t;
      const int64_t from = max(row, static_cast<int64_t>(0));
#pragma unroll
      for (int k = 0; k < KI; ++k) {
        const uint8_t* src = base + __shfl_sync(0xffffffffu, from, k * RPI + g) * RB;
#pragma unroll
        for (int v = 0; v < kVec; ++v) cp_async16(dst + (k * kVec + v) * 512, src + v * (RB / 2));
      }
      cp_commit();
    };
    // Of the warp's row `lane`: the zeros (bytes) of this half, its own scales (bf16 pairs) and, for
    // the unpackers of V, K's: they tell the softmax groups what the token's images lack.
    uint32_t sc[kS], sk[kS], zr;
    auto load_scales = [&](const uint16_t* s, uint32_t (&x)[kS]) {
      if constexpr (G == 1) {
        x[0] = __ldg(s);
      } else if constexpr (G == 2) {
        x[0] = __ldg(reinterpret_cast<const uint32_t*>(s));
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
        x[0] = v.x;
        x[kS - 1] = v.y;
      }
    };
    auto load_grids = [&](int64_t row) {
      const int64_t from = max(row, static_cast<int64_t>(0)) * G;
      if (G > 1 || h == 1) load_scales(half.scales + from, sc);
      if (h == 1) load_scales(a.cache.half[0].scales + from, sk);
      const uint8_t* z = half.zeros + from;
      if constexpr (G == 1) zr = __ldg(z);
      else if constexpr (G == 2) zr = __ldg(reinterpret_cast<const uint16_t*>(z));
      else zr = __ldg(reinterpret_cast<const uint32_t*>(z));
    };
    auto scale_of = [&](const uint32_t (&x)[kS], int gr) -> uint32_t {      // as fp32 bits
      return gr & 1 ? x[gr / 2] & 0xFFFF0000u : x[gr / 2] << 16;
    };
    // a token's largest scale, as fp32 bits; not of the ones that are not finite
    auto top_of = [&](const uint32_t (&x)[kS]) -> uint32_t {
      uint32_t top = 0;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const uint32_t y = scale_of(x, gr);
        top = max(top, y < 0x7F800000u ? y : 0u);
      }
      return top;
    };
    bool ok = true;
    uint32_t gs = 0;
    At now;
    enter(now, blockIdx.x);
    At ahead = now;              // the step whose page is looked up next
    int64_t rows[SM::kAhead + 1];    // of steps gs, gs + 1, ..
#pragma unroll
    for (int k = 0; k < SM::kAhead; ++k) {
      look(ahead);
      next(ahead);
      rows[k] = resolve();
      copy_codes(rows[k], k);
    }
    look(ahead);
    next(ahead);
    load_grids(rows[0]);
    for (; now.u < a.units; ++gs) {
      const int b = gs & 1;
      const int cb = SM::kAhead == 1 ? 0 : b;
      const uint32_t ph = (gs >> 1) & 1u;
      const bool counts = rows[0] >= 0;
      const uint32_t counting = __ballot_sync(0xffffffffu, counts);
      // this step's grids move on to make room for the next one's
      uint32_t s_h[kS], k_h[kS];
#pragma unroll
      for (int k = 0; k < kS; ++k) {
        s_h[k] = sc[k];
        k_h[k] = sk[k];
      }
      const uint32_t z_h = zr;
      next(now);
      rows[SM::kAhead] = resolve();
      look(ahead);
      next(ahead);
      load_grids(rows[1]);
      {
        cp_wait<SM::kAhead - 1>();
        __syncwarp();
        ok = __all_sync(0xffffffffu,
                        h == 0 ? mbar_wait_bounded(&k_empty[k_buffer(gs)], k_phase(gs) ^ 1u,
                                                   abort_flag, info)
                               : mbar_wait_bounded(&v_empty[b], ph ^ 1u, abort_flag, info));
        if (!ok) break;
        const uint8_t* warp_codes = code_slot(cb, h) + dw * (SM::kCodeBytes / kDqWarps);
        const uint8_t* src = warp_codes + lane * 16;
        uint8_t* tile = h == 0 ? k_tile(k_buffer(gs)) : v_tile(b);
        // A group of V without values has the grid [-1, 1], a scale that would push the others' out
        // of fp16's range: it counts as 0.
        if (h == 1) {
          bool empty[G], any = false;
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            empty[gr] = counts && scale_of(s_h, gr) == kEmptyScale<BITS> << 16;
            any |= empty[gr];
          }
          if (__any_sync(0xffffffffu, any)) {
            // row `lane`: lane t of row g copied it in access g / RPI
#pragma unroll
            for (int v = 0; v < kVec; ++v)
#pragma unroll
              for (int x = 0; x < LPR; ++x) {
                const int gr = (BITS == 4 ? 32 * x : 16 * x + v * (D / 2)) / GROUP;
                const uint32_t z =
                    (z_h >> (8 * gr) & 0xFFu) * (BITS == 4 ? 0x11111111u : 0x01010101u);
                const uint4 c = *reinterpret_cast<const uint4*>(
                    warp_codes + ((lane / RPI * kVec + v) * 32 + lane % RPI * LPR + x) * 16);
                if ((c.x ^ z) | (c.y ^ z) | (c.z ^ z) | (c.w ^ z)) {
#pragma unroll
                  for (int y = 0; y < G; ++y)
                    if (y == gr) empty[y] = false;
                }
              }
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
              if (empty[gr]) s_h[gr / 2] &= gr & 1 ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
        // a token that does not count has scales of 0
        if (!counts) {
#pragma unroll
          for (int k = 0; k < kS; ++k) s_h[k] = 0;
        }
        // The images carry scales relative to a power of two, the one above the largest scale of the
        // warp's 32 tokens, so that the largest image stays below 65504; K's, where a row has one
        // grid, none at all: codes less their zero points are exact. Where scales of V lie more than
        // 2^12 apart, each token has a power of its own.
        auto exponent = [&](uint32_t top, int least) {
          return max(static_cast<int>(top >> 23) - 127, least);
        };
        const uint32_t top = top_of(s_h);
        int e = 0;
        if (G > 1 || h == 1) e = exponent(__reduce_max_sync(0xffffffffu, top), h == 0 ? -107 : -96);
        if (h == 1) {
          const bool wide = __any_sync(0xffffffffu, top != 0 && exponent(top, -126) < e - 12);
          if (wide) e = exponent(top, -96);
          if constexpr (G == 1) {
            sh.k_scale[b][dw * kDqRows + lane] =
                counts ? __uint_as_float(k_h[0] << 16) * 6.1035156e-5f : 1.f;
          } else {
            const uint32_t k_top = __reduce_max_sync(0xffffffffu, counts ? top_of(k_h) : 0u);
            if (lane == 0) sh.k_scale[b][dw] = pow2(exponent(k_top, -107) - kTop) * 6.1035156e-5f;
          }
          sh.v_scale[b][dw * kDqRows + lane] = static_cast<uint16_t>((e - kTop + 127) << 7);
          if (lane == 0) {
            sh.v_exp[b][dw] = wide ? kNegInf : static_cast<float>(e - kTop);
            sh.valid[b][dw] = counting;
          }
          mbar_arrive(&g_full[b]);
        }
        uint32_t r_h[kS] = {};
        if (G > 1 || h == 1) {
          const float unit = pow2(kTop - e);
#pragma unroll
          for (int k = 0; k < kS; ++k)
            r_h[k] = half2_bits(__uint_as_float(s_h[k] << 16) * unit,
                                __uint_as_float(s_h[k] & 0xFFFF0000u) * unit);
        }
        // images without scales, with them, or with them and a second image of what their rounding
        // left (exact: the residual of a product)
        auto unpack = [&](auto kind) {
          constexpr bool kScaled = kind.value != kPlainImage, kRest = kind.value == kTwoImages;
          uint32_t rest[4];
          auto image = [&](uint32_t x, uint32_t s, int i) -> uint32_t {
            if constexpr (!kScaled) return x;
            const uint32_t y = hmul2(x, s);
            if constexpr (kRest) rest[i] = hfma2(x, s, y ^ 0x80008000u);
            return y;
          };
#pragma unroll
          for (int k = 0; k < KI; ++k) {
            const int rl = k * RPI + g, row = dw * kDqRows + rl;
            uint32_t sw[kS];
#pragma unroll
            for (int x = 0; x < kS; ++x) sw[x] = __shfl_sync(0xffffffffu, r_h[x], rl);
            const uint32_t zw = __shfl_sync(0xffffffffu, z_h, rl);
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
              const int group = dim_of(v) / GROUP;
              const uint32_t s_w = kS == 2 && (group & 2) ? sw[kS - 1] : sw[0];
              const uint32_t z = zw >> (8 * group) & 0xFFu;
              const uint32_t s2 = __byte_perm(s_w, 0, group & 1 ? 0x3232 : 0x1010);
              const uint32_t z2 = (0x6400u + z) * 0x00010001u;            // 1024 + z, exact
              const uint4 w4 = *reinterpret_cast<const uint4*>(src + (k * kVec + v) * 512);
              uint32_t wd[4] = {w4.x, w4.y, w4.z, w4.w};
              // this piece's image: chunks of eight dims from chunk c0 of its 64-dim half
              uint8_t* dst = tile + (dim_of(v) >> 6) * (kTok * 128) + row * 128;
              const uint32_t c0 = (dim_of(v) & 63) >> 3;
              if constexpr (BITS == 4) {
                // lanes t and t + 2 store to different halves, of the same banks: they take their
                // four chunks in another order, so the eight lanes of a store meet all the banks
                const uint32_t flip = D == 128 ? (t & 2) : 0;
                if (D == 128 && flip) {
                  uint32_t x = wd[0]; wd[0] = wd[2]; wd[2] = x;
                  x = wd[1]; wd[1] = wd[3]; wd[3] = x;
                }
                const uint32_t s16 = hmul2(s2, 0x2C002C00u);              // s / 16
                const uint32_t z16 = (0x6400u + 16 * z) * 0x00010001u;    // 1024 + 16 z
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const uint32_t x = wd[c], x8 = x >> 8;
                  const uint4 y = make_uint4(
                      image(sub2((x & 0x000F000Fu) | 0x64006400u, z2), s2, 0),       // codes 0, 4
                      image(sub2((x & 0x00F000F0u) | 0x64006400u, z16), s16, 1),     // 1, 5, times 16
                      image(sub2((x8 & 0x000F000Fu) | 0x64006400u, z2), s2, 2),      // 2, 6
                      image(sub2((x8 & 0x00F000F0u) | 0x64006400u, z16), s16, 3));   // 3, 7
                  uint8_t* at = dst + (((c0 + (c ^ flip)) ^ (row & 7)) << 4);
                  *reinterpret_cast<uint4*>(at) = y;
                  if constexpr (kRest)
                    *reinterpret_cast<uint4*>(at + kTile) =
                        make_uint4(rest[0], rest[1], rest[2], rest[3]);
                }
              } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  uint32_t y[4] = {__byte_perm(wd[2 * c], 0x64646464u, 0x4140),
                                   __byte_perm(wd[2 * c], 0x64646464u, 0x4342),
                                   __byte_perm(wd[2 * c + 1], 0x64646464u, 0x4140),
                                   __byte_perm(wd[2 * c + 1], 0x64646464u, 0x4342)};
#pragma unroll
                  for (int x = 0; x < 4; ++x) y[x] = image(sub2(y[x], z2), s2, x);
                  uint8_t* at = dst + (((c0 + c) ^ (row & 7)) << 4);
                  *reinterpret_cast<uint4*>(at) = make_uint4(y[0], y[1], y[2], y[3]);
                  if constexpr (kRest)
                    *reinterpret_cast<uint4*>(at + kTile) =
                        make_uint4(rest[0], rest[1], rest[2], rest[3]);
                }
              }
            }
          }
        };
        if (h == 0) unpack(std::integral_constant<int, kPair ? kTwoImages : kPlainImage>{});
        else unpack(std::integral_constant<int, kOneImage>{});
        fence_proxy_async_smem();
        mbar_arrive(h == 0 ? &k_full[k_buffer(gs)] : &v_full[b]);
        // the slot is free (its lane has read it): the codes of a step to come
        copy_codes(rows[SM::kAhead], cb);
      }
#pragma unroll
      for (int k = 0; k < SM::kAhead; ++k) rows[k] = rows[k + 1];
    }
    cp_wait<0>();
  } else {
    registers_down<kMmaRegs>();      // (in this branch: code that others reach keeps its registers)
    if (warp == kMmaWarp) {
      // ---- products: the whole warp runs the loop, so that descriptors stay in uniform registers;
      // one lane issues ----
      constexpr uint32_t id_qk = make_idesc(/*f16*/ 0, 0, 0, 128, kTok);
      constexpr uint32_t id_pv = make_idesc(/*f16*/ 0, 0, /*B MN-major*/ 1, 128, D);
      const bool elected = elect_one();
      // operand tiles are 1024-byte aligned: an offset in 16-byte units adds to a descriptor
      const uint64_t q_desc = smem_desc(smem_u32(q_tile(0)), 16, 1024, kSwizzle128B);
      const uint64_t k_desc = smem_desc(smem_u32(k_tile(0)), 16, 1024, kSwizzle128B);
      const uint64_t v_desc = smem_desc(smem_u32(v_tile(0)), kTok * 128, 1024, kSwizzle128B);
      uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0}, n_pv[2] = {0, 0};
      uint32_t g_base = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, info));
        return ok;
      };
      for (int u = blockIdx.x; ok && u < a.units; u += gridDim.x) {
        const Unit w = get_unit(a, u);
        auto qk = [&](int i, int s) {
          const uint32_t gs = g_base + s;
          const int b = k_buffer(gs);
          if (!wait(&k_full[b], k_phase(gs))) return;
          tc_fence_after();
          if (elected) {
            const uint64_t qd = q_desc + (w.two && i ? kTile / 16 : 0);
            const uint64_t kd = k_desc + b * (kTile / 16);
#pragma unroll
            for (int x = 0; x < (kPair ? 2 : 1); ++x)
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t at = ((kk >> 2) * (kTok * 128) + (kk & 3) * 32) / 16;
                tc_mma_f16(tm_s(i), qd + at, kd + x * (kTile / 16) + at, id_qk, x | kk ? 1u : 0u);
              }
            tc_commit(&s_full[i]);
            if (!w.two || i == 1) tc_commit(&k_empty[b]);
          }
          __syncwarp();
        };
        if (!wait(&q_full[0], n_q[0] & 1)) break;
        ++n_q[0];
        if (w.two) {
          if (!wait(&q_full[1], n_q[1] & 1)) break;
          ++n_q[1];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (steps_of(w, i) == 0) continue;
          // S takes the place of the last unit's weights
          if (n_pv[i] > 0 && !wait(&pv_done[i], (n_pv[i] - 1) & 1)) break;
          qk(i, step_of(w, i, 0));
        }
        const int most = steps_of(w, 0);
        for (int r = 0; r < most && ok; ++r) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || r >= steps_of(w, i)) continue;
            const uint32_t gs = g_base + step_of(w, i, r);
            const int b = gs & 1;
            if (!wait(&p_full[i], n_p[i] & 1)) break;
            ++n_p[i];
            if (!wait(&v_full[b], (gs >> 1) & 1u)) break;
            tc_fence_after();
            if (elected) {
              const uint64_t vd = v_desc + b * (kTile / 16);
#pragma unroll
              for (int kk = 0; kk < kTok / 16; ++kk)
                tc_mma_f16_ts(tm_o(i), tm_s(i) + (kk >> 2) * 64 + (kk & 3) * 8, vd + kk * (2048 / 16),
                              id_pv,
                              (r | kk) ? 1u : 0u);
              tc_commit(&pv_done[i]);
              if (!w.two || i == 1) tc_commit(&v_empty[b]);
            }
            __syncwarp();
            ++n_pv[i];
            if (r + 1 < steps_of(w, i)) {
              // the next S takes the place of the weights that this product reads
              if (!wait(&pv_done[i], (n_pv[i] - 1) & 1)) break;
              qk(i, step_of(w, i, r + 1));
            }
          }
        }
        g_base += w.steps;
      }
      if (elected) {
        tc_commit(&sh.mma_done);           // let what was issued finish, after an error too
        mbar_drain_bounded(&sh.mma_done, 0);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  griddep_wait();
}

// out = the results of the prefix's runs and, where a row met own positions, of its own level,
// weighted by their sums. One warp a vector.
struct Merge {
  const float* part;
  const float* part_lse;
  const float* mid;             // own level: [n][heads ratio][D] and log-sums
  const float* mid_lse;
  __nv_bfloat16* out;
  int64_t ldo, n, row_items, batch;
  const int32_t* starts;
  int heads, ratio, splits;
};
template <int D>
__global__ void __launch_bounds__(256) cache_merge_kernel(const Merge a) {
  constexpr int kVec = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int per_row = a.heads * a.ratio;
  // gridDim.y: blocks of eight vectors of a row
  const int qh = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int64_t tok = blockIdx.x, v = tok * per_row + qh;
  if (qh >= per_row) return;
  // (checked where the result is stored: the loads do not wait for it)
  const int64_t first = a.starts ? __ldg(a.starts) : 0;
  const int64_t end = a.starts ? __ldg(a.starts + a.batch) : a.batch;
  const int head = qh / a.ratio;
  const int64_t j = tok * a.ratio + (qh - head * a.ratio);
  const int64_t ri = j >> 8;
  int r = static_cast<int>(j & 255);
  const bool two = a.n * a.ratio - ri * 256 > 128;
  const int64_t u0 = (head * a.row_items + ri) * a.splits;
  const int parts = two ? a.splits : 2 * a.splits;
  const int wg = two ? r >> 7 : 0;
  r &= 127;
  const float mid_lse = __ldcg(a.mid_lse + v);
  float mid[kVec];
  if constexpr (kVec == 4)
    *reinterpret_cast<float4*>(mid) =
        __ldcg(reinterpret_cast<const float4*>(a.mid + v * D + lane * kVec));
  else
    *reinterpret_cast<float2*>(mid) =
        __ldcg(reinterpret_cast<const float2*>(a.mid + v * D + lane * kVec));
  float m = kNegInf, l = 0.f, acc[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
  constexpr int kAhead = 12;
  for (int s0 = 0; s0 < parts; s0 += kAhead) {
    float x[kAhead][kVec], lse[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      lse[k] = kNegInf;
      if (s0 + k >= parts) continue;
      const int64_t slot = two ? 2 * (u0 + s0 + k) + wg : 2 * u0 + s0 + k;
      lse[k] = __ldcg(a.part_lse + slot * 128 + r);
      const float* src = a.part + (slot * 128 + r) * D + lane * kVec;
      if constexpr (kVec == 4)
        *reinterpret_cast<float4*>(x[k]) = __ldcg(reinterpret_cast<const float4*>(src));
      else
        *reinterpret_cast<float2*>(x[k]) = __ldcg(reinterpret_cast<const float2*>(src));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (lse[k] == kNegInf) continue;          // met nothing: its values were not written
      const float top = fmaxf(m, lse[k]), ref = top == kNegInf ? 0.f : top;
      const float f = m == kNegInf ? (l == 0.f ? 0.f : 1.f) : ex2(m - ref), w = ex2(lse[k] - ref);
      m = top;
      l = fmaf(l, f, w);
#pragma unroll
      for (int d = 0; d < kVec; ++d) acc[d] = fmaf(acc[d], f, w * x[k][d]);
    }
  }
  if (mid_lse != kNegInf) {
    const float top = fmaxf(m, mid_lse), ref = top == kNegInf ? 0.f : top;
    const float f = m == kNegInf ? (l == 0.f ? 0.f : 1.f) : ex2(m - ref), w = ex2(mid_lse - ref);
    l = fmaf(l, f, w);
#pragma unroll
    for (int d = 0; d < kVec; ++d) acc[d] = fmaf(acc[d], f, w * mid[d]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t o[kVec / 2];
#pragma unroll
  for (int k = 0; k < kVec / 2; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    o[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (tok < first || tok >= end) return;       // not a row of any sequence: left as it is
  __nv_bfloat16* dst = a.out + tok * a.ldo + static_cast<int64_t>(qh) * D + lane * kVec;
  if constexpr (kVec == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = o[0];
}

int64_t row_items_of(int64_t n, int ratio) { return (n * ratio + 255) / 256; }
// Units never exceed this, so neither do the slots of a workspace.
int64_t most_units(int64_t items) { return std::max<int64_t>(items, 2 * num_sms()); }

}  // namespace

size_t prefix_workspace_bytes(int heads, int dim, int64_t n, int ratio) {
  const size_t slots = 2 * static_cast<size_t>(most_units(heads * row_items_of(n, ratio)));
  return align_up(slots * 128 * 4, 256) + align_up(slots * 128 * dim * 4, 256);
}

gptq_status run_cache_prefix(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const CacheQuery& q, const float* mid, const float* mid_lse, void* ws,
                             int32_t* info, cudaStream_t stream) {
  Prefix a{};
  a.cache = c;
  a.table = q.prefix_table;
  a.len = q.prefix_len;
  a.q = q.q;
  a.ldq = q.ldq;
  a.n = r.n;
  a.ratio = q.ratio;
  a.scale_log2 = q.scale * 1.4426950408889634f;
  a.row_items = static_cast<int>(row_items_of(r.n, q.ratio));
  a.tiles = static_cast<int>((q.prefix_len + kTok - 1) / kTok);
  const int64_t items = static_cast<int64_t>(a.row_items) * c.heads;
  // Runs per item: the fewest rounds of units times the length of one. A unit's start and end
  // (queries in, results out) cost about as much as two tiles.
  const int64_t sms = num_sms();
  int64_t best = INT64_MAX;
  const int64_t most = std::min<int64_t>(a.tiles, std::max<int64_t>(most_units(items) / items, 1));
  a.splits = 1;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t cost = (items * s + sms - 1) / sms * ((a.tiles + s - 1) / s + 2);
    if (cost < best) {
      best = cost;
      a.splits = static_cast<int>(s);
    }
  }
  if (items * a.splits > INT32_MAX / 4) return GPTQ_EUNSUPPORTED;
  a.units = static_cast<int>(items * a.splits);
  const size_t slots = 2 * static_cast<size_t>(most_units(items));
  a.part_lse = static_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align_up(slots * 128 * 4, 256));
  a.info = info;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.units, sms));
  gptq_status st = dispatch_cache(dim, bits, group, [&](auto d, auto b, auto g) {
    const auto kernel = cache_prefix_kernel<d.value, b.value, g.value>;
    const gptq_status s =
        set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), Smem<d.value, b.value>::kBytes);
    return s != GPTQ_OK ? s
                        : launch_pdl(kernel, dim3(grid), dim3(kThreads), Smem<d.value, b.value>::kBytes,
                                     stream, a);
  });
  if (st != GPTQ_OK) return st;
  Merge m{a.part, a.part_lse, mid, mid_lse, q.out, q.ldo, r.n, a.row_items, r.batch,
          r.starts, c.heads, q.ratio, a.splits};
  const dim3 mg(static_cast<unsigned>(r.n), static_cast<unsigned>((c.heads * q.ratio + 7) / 8));
  return dim == 128 ? launch_pdl(cache_merge_kernel<128>, mg, dim3(256), 0, stream, m)
                    : launch_pdl(cache_merge_kernel<64>, mg, dim3(256), 0, stream, m);
}

}  // namespace gptq

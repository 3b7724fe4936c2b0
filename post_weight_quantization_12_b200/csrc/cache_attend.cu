// Attention of a few rows per sequence over the quantized key/value cache.
//
// A row is one query token and head. With x_t = c log2(e) (q . k_t) over the positions t that the
// row meets, k_t and v_t read as s (code - z) per group of head dimensions,
//   o = sum_t 2^(x_t) v_t / sum_t 2^(x_t),
// taken in one pass over the cache. The rows of one cache head (its query heads, and the sequence's
// tokens) form the 8 or 16 columns of tensor-core products whose other operand is the codes:
//   x:  codes of 16 tokens (the product's rows) against the queries,
//   o:  codes of 16 head dimensions against the weights of 16 tokens.
// The codes enter as fp16 numbers without any conversion: an integer below 1024 in the low bits of
// an fp16 word is that integer times 2^-24 exactly (a subnormal), so a mask (and for the odd codes
// a byte permute) makes the operand. Zero points and scales are applied outside the products:
//   q . k_t = s_t ((q . code_t) - z_t sum(q))             scale and zero of token t, per group
// For o each step's products are followed by one whose rows all hold the step's zero points, so the
// running sum stays one of s (code - z): a sum of codes, all positive, would lose 2^-24 of itself
// with each product, the tensor core's sums being cut towards zero, and what is left after the zero
// points' share is a small part of it.
// The queries are fp16 after a power-of-two scale per row (bf16's 8 bits fit in fp16's 11; values
// 2^-38 below the row's largest are lost). The weights w_t s_t become fp16 (rounding 2^-12 of each)
// relative to their own running reference, one per group of dimensions: with u_t = x_t + log2(s_t) and
// M >= max u - 15 the operand is 2^(u_t - M), whatever range the scales have. The denominator has a
// reference of its own and sums 2^(x_t - m): the scales do not enter it. Sums, references and
// denominators are fp32. (The tensor core adds at the exponent of its largest operands, and a
// subnormal counts as 2^-14 there: a step's sums are cut at 2^-14 of a code times its largest weight.)
//
// The work is cut evenly: tiles of 64 tokens (16 where a warp works alone) of all (sequence, head,
// row tile) items are numbered in order and each CTA or warp takes one run of them. A run that
// covers an item writes its output; an item that several runs share is joined from their partial
// results by a second kernel.
// What bounds it: HBM for 8-bit codes in long sequences (bits / 8 + 3 / group bytes a value); every
// warp keeps three steps of 16 tokens (2 to 4 KB each) in flight through its own ring of 16-byte
// copies of whole sectors (89 us for 131,072 tokens of 8-bit codes, 98 with each lane copying what
// it consumes, at that stage of the kernel), four CTAs of four warps an SM. For 4-bit codes the
// integer pipe, which unpacks them, is as busy as the memory: about 346 warp instructions a step of
// 16 tokens, 57 % of the issue slots and of that pipe.
// Measured (128 dimensions, one grid a row, the whole call; fractions of the measured bandwidth):
//   131,072 tokens, 8 heads of 8-bit codes, 4 query heads each    64 us, 0.65 (kernel 56.6); 6.1 TB/s
//     (0.93) in the steady state, the rest is start, last round and join
//   32 sequences of 100 to 16,000 tokens, 8 heads of 4-bit codes  89 us, 0.47 (kernel 89); 4.1 TB/s
//     (0.62) in the steady state; with a second reference less (a denominator of operands over
//     scales, and one reference for all groups, both wrong for scales far apart) 86
//   one sequence of 37 tokens, 32 heads                           7 us on the device
// Tried and slower: the products of the next step issued before this one's weights (4-bit codes 4.0
// to 3.8 TB/s), two steps unrolled (90 to 92 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "cache.cuh"

namespace gptq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStep = 16;                   // tokens of one warp step
constexpr int kStages = 3;                  // ring depth of a warp, in steps
constexpr int kMaxResident = 4;             // CTAs per SM
constexpr float kNegInf = -INFINITY;

// A stage of the ring holds the codes of 16 tokens as they lie in the cache (K, then V, row after
// row) and their grids. In shared memory the 16-byte chunks of a row are permuted: chunk c of row r
// lies at c ^ swizzle(r). A product's row s is token slot_token(s). The two are chosen together so
// that what the lanes of one load read (K: pieces of the rows of slots 0 .. 7; V: a piece of the
// rows of slots 0, 2, 4, 6 or of the odd ones) meets different banks, for every row length and
// group but one (V of 32-byte rows: two rows meet).
__host__ __device__ constexpr int slot_token(int s) { return s ^ ((s >> 1) & 1); }
template <int RB>
__host__ __device__ constexpr int swizzle(int r) {
  return ((r & 1) << 2 | (((r >> 1) ^ (r >> 2)) & 1) << 1 | ((r >> 2) & 1)) & (RB / 16 - 1);
}

// WPI: the warps that work on one item together, 4 (a CTA) or 1. A tile of work is one step of each.
template <int D, int BITS, int GROUP, int NT, int WPI>
struct Cfg {
  static constexpr int kTile = kStep * WPI;
  static constexpr int kWorkers = kWarps / WPI;               // of a CTA
  static constexpr int G = D / GROUP;
  static constexpr int RB = D * BITS / 8;                     // bytes of a row of codes
  static constexpr int NP = G > RB / 64 ? G : RB / 64;        // K pieces a lane takes of a row
  static constexpr int NPS = NP < 1 ? 1 : NP;
  static constexpr int CPB = RB / 4 / NPS;                    // bytes of a K piece: 4, 8 or 16
  static constexpr int VGB = GROUP * BITS / 64;               // bytes of a lane's V share of a group
  static constexpr int VB = VGB < 4 ? 4 : VGB;                // ... and what it reads
  static constexpr int kK = kStep * RB;                       // K (or V) bytes of a stage
  static constexpr int kCopies = kK / 512;                    // 16-byte copies of a lane for them
  static constexpr int kGridBytes = 96 * G;                   // scales and zeros of 16 tokens
  static constexpr int kStage = 2 * kK + kGridBytes;
  static constexpr int kCopied = kStages * kStage;
  static constexpr int R = 8 * NT;                            // rows of a row tile
  static constexpr int kPad = D + 4;
  static constexpr int kResult = R * kPad * 4;                // fp32 results of a warp
  // a warp's ring, which takes its results when it is done
  static constexpr int kRing = kCopied > kResult ? kCopied : kResult;
  static constexpr int kSmem = kWarps * kRing;
};

// One level of attention: the rows meet the positions of their own sequence (causal), or all of
// them the first `fixed_len` positions behind one page table.
struct Level {
  CacheView cache;
  CacheRows rows;
  int64_t fixed_len;            // < 0: lengths and starts of `rows`
  const __nv_bfloat16* q;
  int64_t ldq;
  int ratio;
  float scale_log2;             // c log2(e)
  __nv_bfloat16* out;           // final output, or null: `mid` is written instead
  int64_t ldo;
  float* mid;                   // [n][heads ratio][D] fp32 results of the level before, and its lse
  float* mid_lse;               // read if `out` is set and they are not null
  float* part;                  // [2 runs][R][D], partial results
  float* part_lse;              // [2 runs][R]
  int32_t* join;                // [runs][8]: what the run's last item needs joined
  int32_t* info;
};

struct Sequence {
  int row0, end;                // rows row0 .. row0 + count - 1; end: the nominal end
  int count, len;               // len: positions that the page table reaches
  int row0_pos;                 // position of row row0: by the given length, also past the table
  int row_tiles, tiles_per;     // tiles of one (head, row tile)
  int64_t tiles;                // of the sequence over all heads
};

// (The host admits fewer than 2^31 rows n * ratio, and lengths are int32: an item's own numbers
// fit in 32 bits.)
template <int R, int kTile>
__device__ __forceinline__ Sequence get_sequence(const Level& a, int64_t b) {
  Sequence s;
  const int n = static_cast<int>(a.rows.n);
  if (a.fixed_len >= 0) {
    s.row0 = 0;
    s.end = s.count = n;
    s.len = static_cast<int>(a.fixed_len);
  } else {
    s.row0 = static_cast<int>(b);
    s.end = s.row0 + 1;
    if (a.rows.starts != nullptr) {
      s.row0 = max(__ldg(a.rows.starts + b), 0);
      s.end = __ldg(a.rows.starts + b + 1);
    }
    s.count = max(min(s.end, n) - s.row0, 0);
    s.len = __ldg(a.rows.lengths + b);
  }
  const int64_t cap = static_cast<int64_t>(a.cache.width) << a.cache.page_shift;
  const bool bad = s.len < 0 || s.len > cap;
  if (bad && (threadIdx.x & 31) == 0) record_info(a.info, GPTQ_INFO_BAD_PAGE);
  s.len = max(s.len, 0);
  s.row0_pos = s.len - (s.end - s.row0);
  if (s.len > cap) s.len = static_cast<int>(cap);
  s.row_tiles = (s.count * a.ratio + R - 1) / R;
  s.tiles_per = max(s.len / kTile + (s.len % kTile != 0), 1);
  s.tiles = static_cast<int64_t>(s.tiles_per) * s.row_tiles * a.cache.heads;
  return s;
}

// The cut of the tiles of all sequences into runs, one per worker and none of them empty; and for
// the runs of this CTA's workers the sequence that their first tile lies in, with the number of that
// sequence's first tile.
struct Find {
  int64_t warp_sum[kWarps];
  int64_t b[kWarps], base[kWarps];
};
struct Cut {
  int64_t total, parts;
  int64_t each;                 // tiles of a run, rounded down
  uint32_t more;                // and how many there are besides
  __device__ __forceinline__ Cut(int64_t tiles, uint32_t most) {
    total = tiles;
    const uint32_t n = min(static_cast<uint64_t>(max(tiles, static_cast<int64_t>(1))),
                           static_cast<uint64_t>(most));
    parts = n;
    // (a division of 64-bit numbers takes longer than everything else here)
    each = tiles >> 32 ? tiles / n : static_cast<uint32_t>(tiles) / n;
    more = static_cast<uint32_t>(tiles - each * n);
  }
  // The first `more` runs have one tile more.
  __device__ __forceinline__ int64_t begin(int64_t part) const {
    return each * part + min(part, static_cast<int64_t>(more));
  }
};
template <int R, int kTile, int kWorkers>
__device__ __forceinline__ Cut find_tile(const Level& a, Find& sh) {
  const int64_t batch = a.fixed_len >= 0 ? 1 : a.rows.batch;
  const int64_t per = (batch + kThreads - 1) / kThreads;
  const int64_t b0 = min(threadIdx.x * per, batch), b1 = min(b0 + per, batch);
  int64_t sum = 0;
  for (int64_t b = b0; b < b1; ++b) sum += get_sequence<R, kTile>(a, b).tiles;
  int64_t incl = sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  incl += before;
  const Cut cut(total, gridDim.x * kWorkers);
#pragma unroll
  for (int w = 0; w < kWorkers; ++w) {
    const int64_t part = static_cast<int64_t>(blockIdx.x) * kWorkers + w;
    const int64_t begin = part < cut.parts ? cut.begin(part) : total;
    if (incl - sum <= begin && begin < incl) {
      int64_t base = incl - sum;
      int64_t b = b0;
      for (; b + 1 < b1; ++b) {       // not entered where a thread has one sequence
        const int64_t t = get_sequence<R, kTile>(a, b).tiles;
        if (begin < base + t) break;
        base += t;
      }
      sh.b[w] = b;
      sh.base[w] = base;
    }
  }
  __syncthreads();
  return cut;
}

// Copies 16 bytes where `on` (a predicate of the instruction, not a branch).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(on)
      : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// Byte permute with all four selector bits: 8 | i repeats the sign of byte i, here 0 or 255.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The G scales (bf16, 2 G bytes aligned) of a token, in pairs.
template <int G>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&x)[(G + 1) / 2]) {
  if constexpr (G == 1) x[0] = *reinterpret_cast<const uint16_t*>(p);
  else if constexpr (G == 2) x[0] = *reinterpret_cast<const uint32_t*>(p);
  else *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(p);
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// Where the results of one row go: the final output (joined with the level before, if any), or the
// fp32 results that the next level will join.
template <int D>
__device__ __forceinline__ void finish(const Level& a, int64_t tok, int qhead, int d, float4 o,
                                       float lse) {
  const int heads = a.cache.heads * a.ratio;
  const int64_t mi = tok * heads + qhead;
  if (a.out == nullptr) {
    *reinterpret_cast<float4*>(a.mid + mi * D + d) = o;
    if (d == 0) a.mid_lse[mi] = lse;
    return;
  }
  if (a.mid != nullptr) {
    const float4 p = __ldcg(reinterpret_cast<const float4*>(a.mid + mi * D + d));
    const float pl = __ldcg(a.mid_lse + mi);
    // A level that met nothing (lse = -inf) counts for nothing. fmaxf drops a NaN, which the
    // weights below bring back.
    const float top = fmaxf(lse, pl), ref = top == kNegInf ? 0.f : top;
    float w0 = ex2(pl - ref), w1 = ex2(lse - ref);
    const float inv = top == kNegInf ? 0.f : __frcp_rn(w0 + w1);
    w0 *= inv;
    w1 *= inv;
    // a level of weight 0 keeps its values out (they may be anything if it met nothing)
    o.x = (pl == kNegInf ? 0.f : w0 * p.x) + (lse == kNegInf ? 0.f : w1 * o.x);
    o.y = (pl == kNegInf ? 0.f : w0 * p.y) + (lse == kNegInf ? 0.f : w1 * o.y);
    o.z = (pl == kNegInf ? 0.f : w0 * p.z) + (lse == kNegInf ? 0.f : w1 * o.z);
    o.w = (pl == kNegInf ? 0.f : w0 * p.w) + (lse == kNegInf ? 0.f : w1 * o.w);
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
  uint2 v;
  v.x = *reinterpret_cast<const uint32_t*>(&lo);
  v.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(a.out + tok * a.ldo + static_cast<int64_t>(qhead) * D + d) = v;
}

// The running references of a warp's rows, negated (rows 0 and 1 of each tile side by side):
//   m: l sums 2^(x - m), up to 2^64 a token (fp32 has the range);
//   M: a token's weight with its largest scale S is 2^(x + log2 S - M), up to 2^15 (the operand of the
//      product with V is fp16 and ends at 65504).
template <int NT>
struct Refs {
  float2 m[NT], M[NT];
};
constexpr float kFirst = -3e38f;          // a reference before the first score
constexpr float kMostBoost = 8.507059e37f;    // 2^126

// One step's weights from its products x (score = x rs, in powers of two, per token and row).
// ls: log2 of the largest V scale of its two tokens; share: each group's share of it, times the
// group's power of two. References are kept until a value passes them by far, and then set 2^7 below
// the largest operand, so that the fp16 numbers' range serves the small ones: they are tried first,
// and what came out is checked. (A denominator that summed operands over scales would lose a token
// whose operand is flushed to 0, however much weight its score gives it beside tokens of large
// scales.) special: the shares need a second look, which `look` takes. kEdge: some token does not
// count for some row.
template <int D, int G, int NT, bool kEdge, typename Look>
__device__ __forceinline__ void weigh(const float (&x)[NT][4], const float (&rs)[NT][2],
                                      const float (&ls)[2], const float (&share)[2][G],
                                      uint32_t (&bf)[NT][G][2], Refs<NT>& ref, float (&l)[NT][2],
                                      float (&o)[NT][D / 16][4], const bool (&on)[NT][4],
                                      bool special, Look look) {
  float2 w[NT][2];                        // of token h: rows 0 and 1
  // true if some operand or weight is beyond what the references allow
  auto attempt = [&]() -> bool {
    float most_y = kNegInf, most_z = kNegInf;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 x2 = make_float2(x[nt][2 * h], x[nt][2 * h + 1]);
        const float2 rs2 = make_float2(rs[nt][0], rs[nt][1]);
        float2 y = fma2(x2, rs2, ref.m[nt]);
        float2 z = fma2(x2, rs2, add2(make_float2(ls[h], ls[h]), ref.M[nt]));
        // a token that does not count may have any grid, NaN too: out by selection
        const bool on0 = !kEdge || on[nt][2 * h], on1 = !kEdge || on[nt][2 * h + 1];
        if (kEdge) {
          y = make_float2(on0 ? y.x : kNegInf, on1 ? y.y : kNegInf);
          z = make_float2(on0 ? z.x : kNegInf, on1 ? z.y : kNegInf);
        }
        most_y = fmaxf(fmaxf(most_y, y.x), y.y);
        most_z = fmaxf(fmaxf(most_z, z.x), z.y);
        w[nt][h] = make_float2(ex2(y.x), ex2(y.y));
        const float2 p = make_float2(ex2(z.x), ex2(z.y));
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          float2 q = p;
          if constexpr (G > 1) {
            q = make_float2(p.x * share[h][gr], p.y * share[h][gr]);
            if (kEdge) q = make_float2(on0 ? q.x : 0.f, on1 ? q.y : 0.f);
          }
          bf[nt][gr][h] = half2_bits(q.x, q.y);
        }
      }
    return most_z > 15.f || most_y > 64.f;
  };
  const bool beyond = attempt();
  if (__any_sync(0xffffffffu, beyond || special)) {
    look();
    // only the rows that need a new reference take one: a row's do not depend on the others'
    auto renew = [&](int nt, int k, float& m, float& M) {
      float y[2], z[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        y[h] = kEdge && !on[nt][2 * h + k] ? kNegInf : x[nt][2 * h + k] * rs[nt][k];
        z[h] = kEdge && !on[nt][2 * h + k] ? kNegInf : y[h] + ls[h];
      }
      float top = fmaxf(y[0], y[1]), top_M = fmaxf(z[0], z[1]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top_M = fmaxf(top_M, __shfl_xor_sync(0xffffffffu, top_M, off));
      }
      if (top > 64.f - m) {
        l[nt][k] *= ex2(-m - top);
        m = -top;
      }
      if (top_M > 15.f - M) {
        const float f = ex2(-M - (top_M - 7.f));
        M = 7.f - top_M;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          o[nt][d][k] *= f;
          o[nt][d][2 + k] *= f;
        }
      }
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      renew(nt, 0, ref.m[nt].x, ref.M[nt].x);
      renew(nt, 1, ref.m[nt].y, ref.M[nt].y);
    }
    attempt();
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 sum = add2(make_float2(l[nt][0], l[nt][1]), add2(w[nt][0], w[nt][1]));
    l[nt][0] = sum.x;
    l[nt][1] = sum.y;
  }
}

// CTAs an SM: four, but three where a row of 128 dimensions has several grids: their shares and
// references do not fit in 128 registers (32 sequences of 100 to 16,000 tokens, 8 heads x 4, group 64:
// 4-bit codes 108 us, and 114 with four; 8-bit codes 123 and 133).
template <int D, int BITS, int GROUP, int NT, int WPI>
__global__ void __launch_bounds__(kThreads, NT == 1 ? (D == 128 && GROUP < 128 ? 3 : 4) : 2)
cache_attend_kernel(const Level a) {
  using C = Cfg<D, BITS, GROUP, NT, WPI>;
  constexpr int G = C::G, R = C::R, RB = C::RB, kTile = C::kTile;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Find find;
  __shared__ float row_lse[kWarps][R];
  // (the broadcast tells the compiler that the warp's number is the same in all its lanes)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  // (the trigger stays behind the wait: cache_prefix_kernel may follow, and does not wait itself)
  griddep_wait();
  griddep_launch_dependents();
  const Cut cut = find_tile<R, kTile, C::kWorkers>(a, find);
  // the worker: this CTA or this warp; which of its warps and threads this is
  const int worker = WPI == 1 ? warp : 0, wi = WPI == 1 ? 0 : warp;
  const int tid = WPI == 1 ? lane : threadIdx.x;
  auto worker_sync = [&]() {
    if constexpr (WPI == 1) __syncwarp(); else __syncthreads();
  };
  const int64_t me = static_cast<int64_t>(blockIdx.x) * C::kWorkers + worker;
  if (tid == 0) a.join[me * 8] = 0;
  if (me >= cut.parts || cut.total == 0) return;
  const int64_t end = cut.begin(me + 1);
  int64_t cur = cut.begin(me), b = find.b[worker];
  const int64_t sequences = a.fixed_len >= 0 ? 1 : a.rows.batch;
  Sequence s = get_sequence<R, kTile>(a, b);
  // the item that tile `cur` lies in, its first tile and the tile within it
  int head, rt, tile0;
  int64_t item0;
  {
    const int64_t rel = cur - find.base[worker];
    int64_t item;
    if (rel >> 32) {
      item = rel / s.tiles_per;
      tile0 = static_cast<int>(rel - item * s.tiles_per);
    } else {
      const uint32_t q = static_cast<uint32_t>(rel) / static_cast<uint32_t>(s.tiles_per);
      tile0 = static_cast<int>(static_cast<uint32_t>(rel) - q * s.tiles_per);
      item = q;
    }
    head = static_cast<int>(item >> 32 ? item / s.row_tiles
                                       : static_cast<uint32_t>(item) /
                                             static_cast<uint32_t>(s.row_tiles));
    rt = static_cast<int>(item - static_cast<int64_t>(head) * s.row_tiles);
    item0 = cur - tile0;
  }

  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_addr = smem_u32(ring);
  // this lane copies chunks lane, lane + 32, .. of the 16 tokens' codes
  const uint8_t* k_src = a.cache.half[0].codes + 16 * lane;
  const uint8_t* v_src = a.cache.half[1].codes + 16 * lane;
  uint32_t copy_at[C::kCopies];
#pragma unroll
  for (int j = 0; j < C::kCopies; ++j) {
    const int c = lane + 32 * j, r = c / (RB / 16);
    copy_at[j] = ring_addr + r * RB + ((c % (RB / 16)) ^ swizzle<RB>(r)) * 16;
  }
  // what it reads of a stage: of K, piece p of the row of slot g at k_at ^ (4 CPB p), of slot g + 8
  // 8 rows on; of V, its share of group gr of the row of slot 2t + (h & 1), at v_at[h & 1] ^
  // (bytes of a group gr)
  const int k_tok = slot_token(g);
  const uint32_t k_at = k_tok * RB + ((t * C::CPB / 16) ^ swizzle<RB>(k_tok)) * 16 + t * C::CPB % 16;
  uint32_t v_at[2];
  {
    const int byte = C::VGB < 4 ? (g >> 1) * 4 : g * C::VGB;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = slot_token(2 * t + h);
      v_at[h] = C::kK + r * RB + ((byte / 16) ^ swizzle<RB>(r)) * 16 + byte % 16;
    }
  }
  // slots 2t and 2t + 1 are tokens 2t and 2t + 1, or the other way round
  const uint32_t z_order = t & 1 ? 0x4041u : 0x4140u;
  // scales and zeros of the 16 tokens: 6 G pieces of 16 bytes, a lane a piece
  const bool grid_lane = lane < 6 * G;
  const uint8_t* g_src;
  uint32_t g_row16;             // bytes of 16 tokens
  {
    const int half = lane >= 3 * G, e = lane - half * 3 * G;
    g_row16 = e < 2 * G ? 32 * G : 16 * G;
    g_src = e < 2 * G ? reinterpret_cast<const uint8_t*>(a.cache.half[half].scales) + 16 * e
                      : a.cache.half[half].zeros + 16 * (e - 2 * G);
  }

  while (cur < end) {
    // ---- a run of tiles of one item ----
    const int run = static_cast<int>(min(static_cast<int64_t>(s.tiles_per - tile0), end - cur));
    const int row_first = rt * R;
    const int32_t* table = a.rows.table + (a.fixed_len >= 0 ? 0 : b * a.rows.ld_table);
    const int tok_begin = tile0 * kTile;
    const int n_rows = s.count * a.ratio;
    // row j of the tile is token j / ratio, query head head * ratio + j % ratio; it meets positions
    // below limit_of(j), which ascends with j
    auto limit_of = [&](int j) -> int {
      if (j >= n_rows) return 0;
      if (a.fixed_len >= 0) return s.len;
      return min(max(s.row0_pos + static_cast<int>(static_cast<uint32_t>(j) /
                                                   static_cast<uint32_t>(a.ratio)) + 1, 0), s.len);
    };
    // (a tile's rows past the last one meet whatever the others do; their results are dropped)
    const int limit_lo = limit_of(row_first);
    const int limit_hi = limit_of(min(row_first + R, n_rows) - 1);

    // ---- this warp's steps: tokens first + kTile i, and the pages of 32 of them, one per lane ----
    const int stop = static_cast<int>(
        min(static_cast<int64_t>(limit_hi), (static_cast<int64_t>(tile0) + run) * kTile));
    const int first = tok_begin + kStep * wi;
    const int steps = stop > first ? (stop - first + kTile - 1) / kTile : 0;
    // entries of the page table, checked once they have come in (checked()): the loads that follow
    // need not wait for them
    auto entry_of = [&](int i) -> int32_t {
      const int64_t k = (first + static_cast<int64_t>(i + lane) * kTile) >> a.cache.page_shift;
      return i + lane < steps && k < a.cache.width ? __ldg(table + k) : -1;
    };
    auto checked = [&](int i, int32_t p) -> int32_t {
      const bool ok = p >= 0 && p < a.cache.pages;
      if (!ok && i + lane < steps) record_info(a.info, GPTQ_INFO_BAD_PAGE);
      return ok ? p : -1;
    };
    int32_t entry = entry_of(0);

    // the queries' loads go out while the pages come in
    constexpr int CPD = D / 4 / C::NPS;   // dims of a piece
    uint4 q_raw[NT][D / 32];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int j = row_first + nt * 8 + g;
      const uint32_t tk = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.ratio);
      const __nv_bfloat16* q =
          a.q + (s.row0 + static_cast<int64_t>(tk)) * a.ldq +
          (static_cast<int64_t>(head) * a.ratio + (j - static_cast<int>(tk) * a.ratio)) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        q_raw[nt][i] = j < n_rows ? __ldg(reinterpret_cast<const uint4*>(
                                        q + (i * 8 / CPD * 4 + t) * CPD + i * 8 % CPD))
                                  : make_uint4(0, 0, 0, 0);
    }

    int32_t pages_now = checked(0, entry);        // of steps 0 .. 31 by lane, then of 32 .. 63, ..
    entry = entry_of(32);                         // the next 32, not checked
    uint32_t put = 0;                     // the stage that is filled next
    uint32_t haves = 0;                   // bit k: the k-th last step issued has a page
    const uint32_t g_dst = ring_addr + 2 * C::kK + 16 * lane;
    auto issue = [&](int i) {
      const int32_t page = __shfl_sync(0xffffffffu, pages_now, i & 31);
      const bool have = i < steps && page >= 0;
      // rows / 16 of the cache stay below 2^31
      const uint32_t off = (first + i * kTile) & ((1 << a.cache.page_shift) - 1);
      const uint32_t row16 =
          ((static_cast<uint32_t>(page) * a.cache.heads + head) << (a.cache.page_shift - 4)) +
          (off >> 4);
      const uint8_t* k0 = k_src + static_cast<uint64_t>(row16) * (16 * RB);
      const uint8_t* v0 = v_src + static_cast<uint64_t>(row16) * (16 * RB);
#pragma unroll
      for (int j = 0; j < C::kCopies; ++j) {
        cp_async16(copy_at[j] + put, k0 + 512 * j, have);
        cp_async16(copy_at[j] + put + C::kK, v0 + 512 * j, have);
      }
      cp_async16(g_dst + put, g_src + static_cast<uint64_t>(row16) * g_row16, have && grid_lane);
      haves = haves << 1 | have;
      put = put == (kStages - 1) * C::kStage ? 0 : put + C::kStage;
      if ((i & 31) == 31 && i < steps) {      // the next step's page is in the next batch
        pages_now = checked(i + 1, entry);
        entry = entry_of(i + 33);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- queries: this lane's dims of row g (and g + 8), fp16, scaled by a power of two ----
    uint32_t qf[NT][D / 8];
    float qsum[NT][G][2], row_scale[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[D / 4];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {q_raw[nt][i].x, q_raw[nt][i].y, q_raw[nt][i].z, q_raw[nt][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
          x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^(14 - e), e the exponent of the largest value (bounded so that both powers are normal)
      const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
      const float up = e > 127 ? 1.f : __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      const float down =
          e > 127 ? 1.f : __uint_as_float(static_cast<uint32_t>(max(e - 14 + 127, 1)) << 23);
      float sum[G];
#pragma unroll
      for (int gr = 0; gr < G; ++gr) sum[gr] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 4; i += 8) {
        // in the order that the codes of 32 bits (two words of 8-bit codes) come out of their words
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = x[i + k] * up;
        uint32_t h[4];
        if constexpr (BITS == 4) {
          h[0] = half2_bits(y[0], y[4]);
          h[1] = half2_bits(y[1] * 0.0625f, y[5] * 0.0625f);
          h[2] = half2_bits(y[2], y[6]);
          h[3] = half2_bits(y[3] * 0.0625f, y[7] * 0.0625f);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = half2_bits(y[2 * k], y[2 * k + 1]);
        }
        const int gr = i / CPD / (C::NPS / G);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          qf[nt][i / 2 + k] = h[k];
          const float2 f = half2_floats(h[k]);
          sum[gr] = fmaf(BITS == 4 && (k & 1) ? 16.f : 1.f, f.x + f.y, sum[gr]);
        }
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
        sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
#pragma unroll
        for (int k = 0; k < 2; ++k)   // times the 2^-24 that the codes carry
          qsum[nt][gr][k] = __shfl_sync(0xffffffffu, sum[gr], (2 * t + k) * 4) * 5.9604645e-8f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        row_scale[nt][k] =
            __shfl_sync(0xffffffffu, down, (2 * t + k) * 4) * 4096.f * a.scale_log2;
    }

    float o[NT][D / 16][4], l[NT][2];
    Refs<NT> ref;
    // power of two by which each group's shares are taken to at most 1; only where G > 1
    float boost[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) boost[gr] = kMostBoost;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[nt][k] = 0.f;
      }
      ref.m[nt] = ref.M[nt] = make_float2(-kFirst, -kFirst);
    }

    uint32_t get = 0;                     // the stage that is consumed
    for (int i = 0; i < steps; ++i) {
      cp_wait<kStages - 2>();
      // every lane's copies have landed, and every lane is done with the step before, whose stage
      // the next copies fill
      __syncwarp();
      issue(i + kStages - 1);
      const bool have = haves >> (kStages - 1) & 1u;
      const uint8_t* st = ring + get;
      const int pos = first + i * kTile;

      // grids of slots g and g + 8
      float sk[2][G], nz[2][G];
      const uint8_t* grids = st + 2 * C::kK;
      const uint8_t* zvp = grids + 80 * G;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = k_tok + 8 * h;
        uint32_t k2[(G + 1) / 2], z4;
        load_scales<G>(grids + 2 * G * r, k2);
        if constexpr (G == 1) z4 = grids[32 + r];
        else if constexpr (G == 2) z4 = *reinterpret_cast<const uint16_t*>(grids + 64 + 2 * r);
        else z4 = *reinterpret_cast<const uint32_t*>(grids + 128 + 4 * r);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          // (2^12 of the codes' 2^24 here and 2^12 with the queries' scale: neither leaves fp32)
          sk[h][gr] = 4096.f * __uint_as_float(gr & 1 ? k2[gr / 2] & 0xFFFF0000u : k2[gr / 2] << 16);
          nz[h][gr] = 8388608.f - __uint_as_float(prmt(z4, 0x4B000000u, 0x7540u | gr));
        }
      }
      // V's: log2 of the token's largest scale, and each group's share of it. The shares of a group
      // all carry one power of two, which leaves the largest so far at most 1, so the groups of small
      // values keep their bits. `careful` looks for groups without values: their grid is [-1, 1], a
      // scale that would push the others' operands out of fp16's range, and zero points times it
      // leave the rounding of their sum. Their share is 0.
      float ls[2], share[2][G];
      bool empty = false, over = false;
      auto v_grids = [&](auto careful) {
        float most = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = k_tok + 8 * h;
          uint32_t v2[(G + 1) / 2];
          load_scales<G>(grids + 48 * G + 2 * G * r, v2);
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint32_t sv = gr & 1 ? v2[gr / 2] & 0xFFFF0000u : v2[gr / 2] << 16;
            share[h][gr] = __uint_as_float(sv);
            if constexpr (!careful.value) {
              empty |= sv == kEmptyScale<BITS> << 16;
            } else {
              constexpr int GB = GROUP * BITS / 8;
              const uint32_t z = zvp[r * G + gr] * (BITS == 4 ? 0x11111111u : 0x01010101u);
              uint32_t other = 0;
#pragma unroll
              for (int i = 0; i < GB / 16; ++i) {          // four lanes to a row
                const int byte = gr * GB + 16 * i + 4 * t;
                other |= z ^ *reinterpret_cast<const uint32_t*>(
                                 st + C::kK + r * RB + ((byte / 16) ^ swizzle<RB>(r)) * 16 +
                                 byte % 16);
              }
              other |= __shfl_xor_sync(0xffffffffu, other, 1);
              other |= __shfl_xor_sync(0xffffffffu, other, 2);
              if (other == 0 && sv == kEmptyScale<BITS> << 16) share[h][gr] = 0.f;
            }
          }
          if constexpr (G == 1) {
            ls[h] = lg2(share[h][0]);
          } else {
            float top = 1.1754944e-38f;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) top = fmaxf(top, share[h][gr]);
            ls[h] = lg2(top);
            const float inv = rcp(top);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              share[h][gr] = share[h][gr] * inv * boost[gr];
              most = fmaxf(most, share[h][gr]);
            }
          }
        }
        over = most > 1.f;
      };
      v_grids(std::false_type{});
      auto look = [&]() {
        if (__any_sync(0xffffffffu, empty)) v_grids(std::true_type{});
        if (G > 1 && __any_sync(0xffffffffu, over)) {
          // only tokens that some row meets: what lies behind them must not matter
          const bool met0 = have && pos + k_tok < limit_hi, met1 = have && pos + k_tok + 8 < limit_hi;
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            float top = fmaxf(met0 ? share[0][gr] : 0.f, met1 ? share[1][gr] : 0.f);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if (top > 1.f) {
              // 2^-e, 2^e the power of two above the largest
              const uint32_t e = min((__float_as_uint(top) >> 23) + 1u, 253u);
              const float f = __uint_as_float((254u - e) << 23);
              boost[gr] *= f;
              share[0][gr] *= f;
              share[1][gr] *= f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int d = gr * (D / G / 16); d < (gr + 1) * (D / G / 16); ++d)
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[nt][d][i] *= f;
            }
          }
        }
      };

      // ---- x: 16 tokens x 8 NT rows ----
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        // two chains of products, so that each waits half as long for the last
        float c[NT][4], c2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) c[nt][e] = c2[nt][e] = 0.f;
#pragma unroll
        for (int pp = 0; pp < C::NPS / G; ++pp) {
          const int p = gr * (C::NPS / G) + pp;
          uint32_t wa[C::CPB / 4], wb[C::CPB / 4];
          const uint8_t* pa = st + (k_at ^ (4 * C::CPB * p));
          const uint8_t* pb = pa + 8 * RB;
          if constexpr (C::CPB == 16) {
            *reinterpret_cast<uint4*>(wa) = *reinterpret_cast<const uint4*>(pa);
            *reinterpret_cast<uint4*>(wb) = *reinterpret_cast<const uint4*>(pb);
          } else if constexpr (C::CPB == 8) {
            *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(pa);
            *reinterpret_cast<uint2*>(wb) = *reinterpret_cast<const uint2*>(pb);
          } else {
            wa[0] = *reinterpret_cast<const uint32_t*>(pa);
            wb[0] = *reinterpret_cast<const uint32_t*>(pb);
          }
#pragma unroll
          for (int w = 0; w < C::CPB / 4; ++w) {
            const int wi = p * (C::CPB / 4) + w;     // word of this lane's row
            if constexpr (BITS == 4) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const uint32_t u = hf ? wa[w] >> 8 : wa[w], v = hf ? wb[w] >> 8 : wb[w];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(hf ? c2[nt] : c[nt], u & 0x000F000Fu, v & 0x000F000Fu, u & 0x00F000F0u,
                          v & 0x00F000F0u, qf[nt][4 * wi + 2 * hf], qf[nt][4 * wi + 2 * hf + 1]);
              }
            } else {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(w & 1 ? c2[nt] : c[nt], __byte_perm(wa[w], 0, 0x4140), __byte_perm(wb[w], 0, 0x4140),
                        __byte_perm(wa[w], 0, 0x4342), __byte_perm(wb[w], 0, 0x4342),
                        qf[nt][2 * wi], qf[nt][2 * wi + 1]);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[nt][e] = fmaf(sk[e >> 1][gr], fmaf(nz[e >> 1][gr], qsum[nt][gr][e & 1],
                                                 c[nt][e] + c2[nt][e]), x[nt][e]);
      }

      // ---- weights relative to the running references ----
      bool on[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) on[nt][e] = true;
      uint32_t bf[NT][G][2];
      if (have && pos + kStep <= limit_lo) {
        weigh<D, G, NT, false>(x, row_scale, ls, share, bf, ref, l, o, on, empty || over, look);
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            on[nt][e] = have && pos + k_tok + 8 * (e >> 1) <
                                    limit_of(row_first + nt * 8 + 2 * t + (e & 1));
        weigh<D, G, NT, true>(x, row_scale, ls, share, bf, ref, l, o, on, empty || over, look);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
          for (int h = 0; h < 2; ++h) bf[nt][gr][h] = transpose8x8(bf[nt][gr][h]);

      // ---- o: 16 dims x 8 NT rows per product ----
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        uint32_t w[4][C::VB / 4];
        // minus the zero points of slots 2t and 2t + 1, and of the two eight further on, as fp16
        // codes: rows of an operand whose product with the weights takes the zero points out
        uint32_t zp[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* z = zvp + (2 * t + 8 * h) * G + gr;       // tokens 2t and 2t + 1
          uint32_t zz;
          if constexpr (G == 1) zz = *reinterpret_cast<const uint16_t*>(z);
          else zz = z[0] | static_cast<uint32_t>(z[G]) << 8;
          zp[h] = __byte_perm(zz, 0x80808080u, z_order);           // 0x80 above each: minus z
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint8_t* pv = st + (v_at[h & 1] ^ (gr * (GROUP * BITS / 8))) + (h >> 1) * 8 * RB;
          if constexpr (C::VB == 16)
            *reinterpret_cast<uint4*>(w[h]) = *reinterpret_cast<const uint4*>(pv);
          else if constexpr (C::VB == 8)
            *reinterpret_cast<uint2*>(w[h]) = *reinterpret_cast<const uint2*>(pv);
          else
            w[h][0] = *reinterpret_cast<const uint32_t*>(pv);
          if constexpr (C::VGB < 4) w[h][0] >>= 16 * (g & 1);
        }
        constexpr int kPairs = BITS == 4 ? (C::VGB < 4 ? 2 : 4) : 2;   // dim pairs of a word
#pragma unroll
        for (int wi = 0; wi < C::VB / 4; ++wi) {
          uint32_t ev[4], od[4];       // even and odd codes of the word, 4 bits: in bytes
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            ev[h] = BITS == 4 ? w[h][wi] & 0x0F0F0F0Fu : w[h][wi];
            od[h] = BITS == 4 ? (w[h][wi] >> 4) & 0x0F0F0F0Fu : w[h][wi];
          }
#pragma unroll
          for (int i2 = 0; i2 < kPairs; ++i2) {
            uint32_t a0, a1, a2, a3;
            if constexpr (BITS == 4) {
              const uint32_t sel = i2 | (8 | i2) << 4 | (4 + i2) << 8 | (8 | i2) << 12;
              a0 = prmt(ev[0], ev[1], sel);
              a1 = prmt(od[0], od[1], sel);
              a2 = prmt(ev[2], ev[3], sel);
              a3 = prmt(od[2], od[3], sel);
            } else {
              const uint32_t s0 = (2 * i2) | (4 + 2 * i2) << 8;
              const uint32_t s1 = (2 * i2 + 1) | (5 + 2 * i2) << 8;
              a0 = prmt(ev[0], ev[1], s0) & 0x00FF00FFu;
              a1 = prmt(od[0], od[1], s1) & 0x00FF00FFu;
              a2 = prmt(ev[2], ev[3], s0) & 0x00FF00FFu;
              a3 = prmt(od[2], od[3], s1) & 0x00FF00FFu;
            }
            const int tile = gr * (GROUP / 16) + wi * kPairs + i2;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(o[nt][tile], zp[0], zp[0], zp[1], zp[1], bf[nt][gr][0], bf[nt][gr][1]);
              mma_f16(o[nt][tile], a0, a1, a2, a3, bf[nt][gr][0], bf[nt][gr][1]);
            }
          }
        }
      }
      get = get == (kStages - 1) * C::kStage ? 0 : get + C::kStage;
    }
    cp_wait<0>();

    // ---- join the worker's warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], off);
    worker_sync();         // the rings are idle
    // each warp's own results, divided by their weights (so in the range of the values), and the
    // logarithm of the weights' sum
    float* res = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = nt * 8 + 2 * t + k;
        const float m = k ? ref.m[nt].y : ref.m[nt].x, M = k ? ref.M[nt].y : ref.M[nt].x;
        if (g == 0) row_lse[warp][r] = l[nt][k] == 0.f ? kNegInf : log2f(l[nt][k]) - m;
        const float inv = l[nt][k] == 0.f ? 0.f : 16777216.f * rcp(l[nt][k]);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          // 2^(M - m) / boost as a square: M and m may lie further apart than one factor reaches
          const float f = ex2(0.5f * (m - M - (G == 1 ? 0.f : lg2(boost[gr])))), f1 = inv * f;
#pragma unroll
          for (int i = 0; i < GROUP / 16; ++i) {
            const int tile = gr * (GROUP / 16) + i;
            *reinterpret_cast<float2*>(res + r * C::kPad + gr * GROUP + g * (GROUP / 8) + 2 * i) =
                make_float2(o[nt][tile][k] * f1 * f, o[nt][tile][2 + k] * f1 * f);
          }
        }
      }
    worker_sync();
    const bool whole = run == s.tiles_per;
    const int64_t slot = tile0 == 0 ? 2 * me + 1 : 2 * me;
    const int w0 = WPI == 1 ? warp : 0;          // the worker's first warp
    for (int k = tid; k < R * (D / 4); k += 32 * WPI) {
      const int r = k / (D / 4), d = k % (D / 4) * 4;
      const int j = row_first + r;
      if (j >= n_rows) continue;
      float4 acc;
      float lse;
      if constexpr (WPI == 1) {
        acc = *reinterpret_cast<const float4*>(res + r * C::kPad + d);
        lse = row_lse[warp][r];
      } else {
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < WPI; ++w) top = fmaxf(top, row_lse[w0 + w][r]);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < WPI; ++w) {
          // a warp that met nothing counts for nothing; one that met NaN has NaN weights
          const float lw = row_lse[w0 + w][r];
          const float f = lw == kNegInf ? 0.f : ex2(lw - (top == kNegInf ? 0.f : top));
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + (w0 + w) * C::kRing) + r * C::kPad + d);
          den += f;
          acc.x = fmaf(f, v.x, acc.x);
          acc.y = fmaf(f, v.y, acc.y);
          acc.z = fmaf(f, v.z, acc.z);
          acc.w = fmaf(f, v.w, acc.w);
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        lse = den == 0.f ? kNegInf : (top == kNegInf ? 0.f : top) + log2f(den);
      }
      if (whole) {
        const uint32_t tk = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.ratio);
        finish<D>(a, s.row0 + static_cast<int64_t>(tk),
                  head * a.ratio + j - static_cast<int>(tk) * a.ratio, d, acc, lse);
      } else {
        *reinterpret_cast<float4*>(a.part + (slot * R + r) * D + d) = acc;
        if (d == 0) a.part_lse[slot * R + r] = lse;
      }
    }
    if (!whole && tile0 == 0 && tid == 0) {
      // this run holds the item's beginning: runs me + 1 .. last hold the rest
      const int64_t t_last = item0 + s.tiles_per - 1;
      int64_t last = me + 1;
      while (last + 1 < cut.parts && cut.begin(last + 1) <= t_last) ++last;
      int32_t* join = a.join + me * 8;
      join[1] = min(n_rows - row_first, R);
      join[2] = head;
      join[4] = s.row0;
      join[5] = row_first;
      join[0] = static_cast<int32_t>(last - me);
    }
    // ---- the next item ----
    cur += run;
    if (cur < end) worker_sync();     // its copies overwrite the results just read
    tile0 = 0;
    item0 = cur;
    if (++rt == s.row_tiles) {
      rt = 0;
      if (++head == a.cache.heads && cur < end) {
        head = 0;
        do {
          if (b + 1 >= sequences) return;   // only if the lengths changed under this kernel
          s = get_sequence<R, kTile>(a, ++b);
        } while (s.tiles == 0);
      }
    }
  }
}

// Joins the partial results of the item that starts in run blockIdx.x and ends in a later one: slot
// 2 c + 1 of its first run c, slots 2 c' of the runs after it. The warps share the rows of the item,
// and with more warps than rows the slots of a row.
template <int D, int R, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps)
cache_join_kernel(const Level a) {
  __shared__ float sh[kJoinWarps][D];
  __shared__ float sh_m[kJoinWarps], sh_l[kJoinWarps];
  // (the trigger stays behind the wait: cache_prefix_kernel may follow, and does not wait itself)
  griddep_wait();
  griddep_launch_dependents();
  const int64_t c = blockIdx.x;
  const int32_t* join = a.join + c * 8;
  const int runs = __ldcg(join);
  if (runs == 0) return;
  const int live = __ldcg(join + 1), head = __ldcg(join + 2);
  const int64_t row0 = __ldcg(join + 4);
  const int row_first = __ldcg(join + 5);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int per_row = kJoinWarps / R < 1 ? 1 : kJoinWarps / R;     // warps of a row
  constexpr int kVec = D / 32;                            // dims of a lane: 2 or 4
  for (int r = warp / per_row; r < R; r += kJoinWarps / per_row) {
    const int sub = warp % per_row;
    float m = kNegInf, l = 0.f, acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
    auto add = [&](float lse, const float* v) {
      if (lse == kNegInf) return;
      const float top = fmaxf(m, lse), ref = top == kNegInf ? 0.f : top;
      const float f = m == kNegInf ? (l == 0.f ? 0.f : 1.f) : ex2(m - ref), w = ex2(lse - ref);
      m = top;
      l = fmaf(l, f, w);
#pragma unroll
      for (int k = 0; k < kVec; ++k) acc[k] = fmaf(acc[k], f, w * v[k]);
    };
    constexpr int kAhead = 8;
    if (r < live) {
      for (int s0 = sub; s0 <= runs; s0 += per_row * kAhead) {
        float v[kAhead][kVec], lse[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int si = s0 + u * per_row;
          lse[u] = kNegInf;
          if (si > runs) continue;
          const int64_t slot = si == 0 ? 2 * c + 1 : 2 * (c + si);
          lse[u] = __ldcg(a.part_lse + slot * R + r);
          const float* src = a.part + (slot * R + r) * D + lane * kVec;
          if constexpr (kVec == 4)
            *reinterpret_cast<float4*>(v[u]) = __ldcg(reinterpret_cast<const float4*>(src));
          else
            *reinterpret_cast<float2*>(v[u]) = __ldcg(reinterpret_cast<const float2*>(src));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) add(lse[u], v[u]);
      }
    }
    if (per_row > 1) {
      // the loop runs once for every warp here: R * per_row == kJoinWarps
#pragma unroll
      for (int k = 0; k < kVec; ++k) sh[warp][lane * kVec + k] = acc[k];
      if (lane == 0) {
        sh_m[warp] = m;
        sh_l[warp] = l;
      }
      __syncthreads();
      if (sub == 0) {
        for (int w = 1; w < per_row; ++w) {
          const float wm = sh_m[warp + w], wl = sh_l[warp + w];
          if (wm == kNegInf && wl == 0.f) continue;
          const float top = fmaxf(m, wm), ref = top == kNegInf ? 0.f : top;
          const float f = m == kNegInf ? (l == 0.f ? 0.f : 1.f) : ex2(m - ref);
          const float g = wm == kNegInf ? 1.f : ex2(wm - ref);
          m = top;
          l = l * f + wl * g;
#pragma unroll
          for (int k = 0; k < kVec; ++k)
            acc[k] = acc[k] * f + sh[warp + w][lane * kVec + k] * g;
        }
      }
    }
    if (sub == 0 && r < live) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse = l == 0.f ? kNegInf : (m == kNegInf ? 0.f : m) + log2f(l);
      float x[4];
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = acc[k] * inv;
      const int j = row_first + r;
      const int64_t tok = row0 + j / a.ratio;
      const int qhead = head * a.ratio + j % a.ratio;
      if constexpr (kVec == 4) {
        finish<D>(a, tok, qhead, lane * 4, make_float4(x[0], x[1], x[2], x[3]), lse);
      } else {
        x[2] = __shfl_down_sync(0xffffffffu, x[0], 1);
        x[3] = __shfl_down_sync(0xffffffffu, x[1], 1);
        if ((lane & 1) == 0)
          finish<D>(a, tok, qhead, lane * 2, make_float4(x[0], x[1], x[2], x[3]), lse);
      }
    }
  }
}

// The longest sequence that a level can hold.
int64_t longest_of(const Level& a) {
  return a.fixed_len >= 0 ? a.fixed_len
                          : static_cast<int64_t>(a.cache.width) << a.cache.page_shift;
}

// CTAs of the attention kernel that fit on the device at once, cached per instance and device.
template <int D, int BITS, int GROUP, int NT, int WPI>
int resident_ctas() {
  static std::mutex mu;
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    using C = Cfg<D, BITS, GROUP, NT, WPI>;
    int per = 0;
    const void* k = reinterpret_cast<const void*>(cache_attend_kernel<D, BITS, GROUP, NT, WPI>);
    if (set_max_dynamic_smem(k, C::kSmem) != GPTQ_OK ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, kThreads, C::kSmem) != cudaSuccess ||
        per <= 0)
      return 0;
    cache[dev] = std::min(per, kMaxResident) * num_sms();
  }
  return cache[dev];
}

template <int D, int BITS, int GROUP, int NT, int WPI>
gptq_status attend_level(Level a, cudaStream_t stream) {
  using C = Cfg<D, BITS, GROUP, NT, WPI>;
  const int64_t resident =
      static_cast<int64_t>(resident_ctas<D, BITS, GROUP, NT, WPI>()) * C::kWorkers;
  if (resident <= 0) return GPTQ_ECUDA;
  // no more runs than there can be tiles
  const int64_t seqs = a.fixed_len >= 0 ? 1 : a.rows.batch;
  const int64_t row_tiles = (a.rows.n * a.ratio + C::R - 1) / C::R + seqs;
  const int64_t per = std::max<int64_t>((longest_of(a) + C::kTile - 1) / C::kTile, 1);
  const int64_t items = row_tiles * a.cache.heads;
  int64_t runs = resident;
  if (items < resident && per < resident) runs = std::min<int64_t>(resident, items * per);
  const unsigned grid = static_cast<unsigned>((runs + C::kWorkers - 1) / C::kWorkers);
  runs = static_cast<int64_t>(grid) * C::kWorkers;
  gptq_status st = launch_pdl(cache_attend_kernel<D, BITS, GROUP, NT, WPI>, dim3(grid),
                              dim3(kThreads), C::kSmem, stream, a);
  if (st != GPTQ_OK || per == 1) return st;    // items of one tile are never shared
  // Items of many runs each (few, long sequences): several warps to a row. 131,072 tokens over 8
  // heads are joined from 74 runs a head.
  return runs >= 8 * items ? launch_pdl(cache_join_kernel<D, C::R, 32>,
                                        dim3(static_cast<unsigned>(runs)), dim3(1024), 0, stream, a)
                           : launch_pdl(cache_join_kernel<D, C::R, 8>,
                                        dim3(static_cast<unsigned>(runs)), dim3(256), 0, stream, a);
}

// Runs that a workspace has slots for: of CTAs with up to 16 rows, or of warps with 8.
size_t most_runs() { return static_cast<size_t>(num_sms()) * kMaxResident; }

size_t join_bytes() { return align_up(most_runs() * kWarps * 8 * 4, 256); }
size_t lse_bytes() { return align_up(2 * most_runs() * kWarps * 8 * 4, 256); }
size_t part_bytes(int dim) {
  return align_up(2 * most_runs() * kWarps * 8 * static_cast<size_t>(dim) * 4, 256);
}

}  // namespace

size_t cache_workspace_bytes(int heads, int dim, int64_t n, int ratio, bool shared) {
  size_t b = join_bytes() + lse_bytes() + part_bytes(dim);
  if (shared) {
    const size_t rows = static_cast<size_t>(n) * heads * ratio;
    b += align_up(rows * 4, 256) + align_up(rows * dim * 4, 256) +
         prefix_workspace_bytes(heads, dim, n, ratio);
  }
  return b;
}

gptq_status run_cache_attend(const CacheView& c, const CacheRows& r, int dim, int bits, int group,
                             const CacheQuery& q, void* ws, int32_t* info, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  Level a{};
  a.cache = c;
  a.rows = r;
  a.fixed_len = -1;
  a.q = q.q;
  a.ldq = q.ldq;
  a.ratio = q.ratio;
  a.scale_log2 = q.scale * 1.4426950408889634f;
  a.out = q.out;
  a.ldo = q.ldo;
  a.info = info;
  a.join = reinterpret_cast<int32_t*>(w);
  w += join_bytes();
  a.part_lse = reinterpret_cast<float*>(w);
  w += lse_bytes();
  a.part = reinterpret_cast<float*>(w);
  w += part_bytes(dim);
  // 8 rows a tile where a sequence has no more on average, else 16: a second set of columns costs
  // registers and products, a second pass over the codes costs more. Where sequences of up to 8 rows
  // times heads are enough to give each warp of the device an item, each warp works on its own: no
  // barriers, one conversion of the queries instead of four, no join within the CTA. 128 sequences
  // of 60 to 250 tokens x 32 heads: 51 us, and 88 us with a CTA an item; x 8 heads 27 and 31 us, 32
  // sequences x 8 heads 23 and 16 us.
  auto level = [&](const Level& l, int64_t rows_each) {
    const int64_t items = (l.fixed_len >= 0 ? 1 : l.rows.batch) * c.heads;
    return dispatch_cache(dim, bits, group, [&](auto d, auto b, auto g) {
      return rows_each > 8 ? attend_level<d.value, b.value, g.value, 2, 4>(l, stream)
             : items < static_cast<int64_t>(most_runs()) * kWarps
                 ? attend_level<d.value, b.value, g.value, 1, 4>(l, stream)
                 : attend_level<d.value, b.value, g.value, 1, 1>(l, stream);
    });
  };
  if (q.prefix_len > 0) {
    const size_t rows = static_cast<size_t>(r.n) * c.heads * q.ratio;
    a.mid_lse = reinterpret_cast<float*>(w);
    a.mid = reinterpret_cast<float*>(w + align_up(rows * 4, 256));
    // A second or third row tile of 16 costs a second pass over the codes; the tensor-core kernel
    // costs the same for up to 128 rows. Over 32,768 tokens x 32 heads of 4-bit codes: 32 rows
    // 124 us here and 159 us there, 48 rows 169 and 157, 128 rows 400 and 171; over 1000 tokens
    // the two are within 4 us of each other from 20 to 128 rows.
    if (r.n * q.ratio > 32) {
      w += align_up(rows * 4, 256) + align_up(rows * dim * 4, 256);
      a.out = nullptr;
      const gptq_status st = level(a, (r.n * q.ratio + r.batch - 1) / r.batch);
      if (st != GPTQ_OK) return st;
      return run_cache_prefix(c, r, dim, bits, group, q, a.mid, a.mid_lse, w, info, stream);
    }
    Level p = a;
    p.out = nullptr;
    p.fixed_len = q.prefix_len;
    p.rows.table = q.prefix_table;
    p.cache.width = static_cast<int>((q.prefix_len + (1 << c.page_shift) - 1) >> c.page_shift);
    const gptq_status st = level(p, r.n * q.ratio);
    if (st != GPTQ_OK) return st;
  }
  return level(a, (r.n * q.ratio + r.batch - 1) / r.batch);
}

}  // namespace gptq

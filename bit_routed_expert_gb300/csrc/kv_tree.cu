// Attention over the whole cached context and a tree of drafted tokens behind it, on the 5th-generation tensor cores.
//
// The call's tokens of one sequence, all query heads of one kv head: up to 128 rows of a tile, or 256 in two tiles that
// share the blocks.  Every block of the context is read once for them: (2 D + 2) bytes a token against 4 D operations for
// each row, so DRAM sets the pace up to about 128 rows and the tensor cores beyond.
//
// One CTA an SM, which takes an equal share of the call's work: (rows, kv head) units one after the other, each a run of
// blocks; a share may begin and end inside a unit.  Such parts go to the workspace, and another kernel joins them in the
// order of the context (the same numbers whatever the order in which CTAs finish).  The host knows neither
// lengths nor runs: every CTA adds up the work of all tiles itself and finds its place.  A kernel before forms the queries'
// two terms.
//
// What bounds it: not the tensor cores nor DRAM yet, but the roles' chains of short steps (a wait is some 150 cycles
// even where nothing is to be waited for) and instruction fetch: five roles' loops share a small instruction cache, so that code
// that runs seldom costs some 250 cycles for every 128 bytes of it.  Hence little code: loops that are not unrolled far, what is
// seldom out of line.  A step of 64 tokens takes 1,500 cycles for one tile and 2,100 for two, whose products take 1,260: with two the
// softmax, the conversion and the issue of O's products take 1,700 to 1,800 each, and wait for one another.  More than 16
// warps would leave 96 registers a thread, which costs the softmax more than what other roles gain.
// D = 128, G = 8, four kv heads: 32 sequences of up to 16,384 tokens, 16 drafts each, 115 us (2.5 TB/s); one of
// 131,072, 64 drafts, 157 us (0.87 PFLOP/s, 0.45 of cuBLAS's); a prompt of 4,096 behind 4,096, 466 us (0.88 PFLOP/s).
//
// Sixteen warps:
//   warps 0-3, 4-7  softmax, a thread a row: two tiles' rows of the same block, or, where there is one tile, its
//                   rows of the even and of the odd blocks, each with a running maximum, sum and output of its own
//   warps 8-11      the values' codes into FP16 in 128-byte-swizzled shared memory, two warps for the even and two for the odd
//                   blocks (eight warps: 20% slower)
//   warp 12         walks through the share, looks up pages and starts the copies (TMA: queries and keys swizzled, values as
//                   they lie)
//   warps 13, 14    issue either group's S = Q K^T into tensor memory and tell it of its blocks and of units' ends
//   warp 15         issues O += P V, with P read from tensor memory
//
// The keys' codes are an MMA operand as they lie in the cache.  A BF16 query is q = 2^e (a + b), a and b E4M3: a is
// q's nearest code, b the rest's, so that the two products add up to that of q itself (see bre.h for what is lost).  Two
// products of 8-bit operands take the tensor cores as long as one of 16-bit ones, and the keys need no conversion.  A key's
// scale multiplies its logit.  A value's scale goes into its FP16 value relative to the block's largest, which is exact down to
// 2^-15 of that, and the largest one into the block's weights; where a row is further below, or the scale is above
// EV_LARGE, every token's own goes into its weight (see kv_attend.cu), by slower code.  So do blocks and rows whose logits
// may be too large for FP32's steps (F_LARGE, K_LARGE): to look at every block's product of both instead cost prompts 3%.
#include <atomic>

#include "kv_tc.cuh"
#include "kv_tree.cuh"

namespace bre {

namespace {

constexpr int TT_THREADS = 512;
constexpr int TT_WARPS = TT_THREADS / 32;
constexpr int W_CONV = 8, W_LOAD = 12, W_S = 13, W_O = 15;
// Depths of the rings (powers of 2): keys with what the S warp is told, values with what the converting warps are told;
// converted values; what either softmax group is told; scales.  The last need no barriers: a
// softmax group has one of every two blocks, and lags behind by TT_GROUP of these and by the TT_V that the converting
// warps may be apart.
constexpr int TT_K = 4, TT_V = 4, TT_V16 = 4, TT_GROUP = 4, TT_SC = 16;
constexpr int TT_MAX_CTAS = 160;
constexpr int JOIN_CTAS = 4;             // of the joining kernel, for every one of the other
constexpr int JOIN_FEW = 32;             // parts that half a warp joins
constexpr float P_MOST = 32768.0f;       // a block's sum of weights up to which they are FP16 numbers for sure
// Logits are below 2^24.7 (128 products of codes up to 448) times the row's factor and the key's scale.  Where these are below F_LARGE
// and 2^K_LARGE, that is 2^26.7, an unrounded one is off by 4 at most from a rounded maximum that is as large.
constexpr float F_LARGE = 0.25f;         // |q| of 880 for D = 128 and the usual scale
constexpr int K_LARGE = 4;               // |k| of 7,168
// Costs of the shares: a block for one tile, for two tiles, and what a unit takes beside its blocks.
constexpr int COST_ONE = 2, COST_TWO = 3, COST_UNIT = 16;

enum : int { F_BLOCK = 1, F_FULL = 4, F_END = 8, F_EXIT = 16, F_TWO = 32, F_SOME = 64, F_ODD = 128, F_NEW = 256, F_BEGIN = 512 };

// What the walking warp tells the others: a block (F_ODD: of the second group, where there is one tile; F_BEGIN: the first
// of the unit's part; F_NEW: the first of its group), or the end of a unit's part.
struct Item {
  int t0, n, h, blk;              // tokens, kv head; block (at the end: how many there were)
  int flags, slot, begin, kb;     // slot < 0: the whole unit, its outputs are final; running number of the block
};

constexpr int ITEM_WORDS = sizeof(Item) / sizeof(int);
static_assert(ITEM_WORDS <= 32, "copied by a warp");

// Where the parts of a unit that several CTAs share are to be found (written by the CTA that holds its first block).
struct Join {
  int t0, n, h, parts;   // parts: 0: none; else this CTA's second slot, then the first slots of the next parts - 1 CTAs
};

struct TreeParams {
  const uint8_t* pages;
  int H, G, per;            // per: tokens of a tile
  KvTable tab;
  const uint16_t* q;
  long long q_stride;
  const int32_t* seq;
  const int32_t* pos;
  int T;
  const int32_t* start;
  const uint64_t* mask;
  int words;
  float scale;
  uint16_t* out;
  float* lse;
  int32_t* err;
  long long wait;
  Join* join;               // [CTAs]
  float2* ml;               // [CTAs][2][rows]: maximum and sum
  float* part;              // [CTAs][2][rows][D]
  int rows;                 // rows of a slot
  unsigned char* codes;     // [2 terms][kv heads][q_rows][D]: the queries as E4M3
  float* factors;           // [kv heads][q_rows]: of their logits
  int q_rows;               // tokens times heads of a group, or 128 if that is less
};

template <int D>
struct TreeMem {
  static constexpr int TERM = 128 * D, K = KV_BLOCK * D, V16 = KV_BLOCK * D * 2, V = KV_BLOCK * D + 2 * KV_BLOCK;
  static constexpr int q = 0, k = q + 4 * TERM, v16 = k + TT_K * K, v = v16 + TT_V16 * V16, end = v + TT_V * V;
  static constexpr int bytes = end + 1024;   // the swizzled tiles start on 1024 bytes
};

// Keys and query terms: rows of D bytes, K-major, swizzled by the row's own width.
template <int D>
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)((8 * D) >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)(D == 128 ? 2 : 4) << 61);
}
__device__ __forceinline__ void mma_codes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two FP16 values to E4M3 codes, nearest even, saturating; the difference of two pairs.
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---------------------------------------------------------------------------
// Shares
// ---------------------------------------------------------------------------
// Tiles: the list is cut where the sequence changes, where padding begins or ends, and every `per` tokens of a run.
__device__ __forceinline__ bool other_run(int s, int p, int s2, int p2) {
  return (p < 0) != (p2 < 0) || (p >= 0 && s != s2);
}

// Two counters; which one is not known when the program is compiled, and an array would lie in memory.
struct Pair {
  int a, b;
  __device__ __forceinline__ int operator[](int i) const { return i ? b : a; }
  __device__ __forceinline__ void add(int i) { a += i ^ 1, b += i; }
};

struct Unit {
  int blocks, step;   // of a tile and one kv head: blocks, cost of one
  __device__ __forceinline__ Unit(int n, int top, int N, int per_one) {
    blocks = top < 0 ? 1 : min(top / KV_BLOCK + 1, N);
    step = n > per_one ? COST_TWO : COST_ONE;
  }
  __device__ __forceinline__ long long cost() const { return COST_UNIT + (long long)blocks * step; }
  // block i counts from here on; the first block carries the unit's own cost
  __device__ __forceinline__ long long at(int i) const { return i ? COST_UNIT + (long long)i * step : 0; }
  // the first block that counts from x on or later
  __device__ __forceinline__ int first_from(long long x) const {
    if (x <= 0) return 0;
    if (x > at(blocks - 1)) return blocks;   // (what follows fits 32 bits: a unit has at most 2^25 blocks)
    return max(((int)x - COST_UNIT + step - 1) / step, 1);
  }
};

// a / b; hardly ever of numbers that need the long division
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return a <= 0x7FFFFFFFLL && b <= 0x7FFFFFFFLL ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

constexpr int KEPT = 32;

struct PlanMem {
  int run[TT_WARPS], top[TT_THREADS];
  // of a chunk's last token: first token of its run, largest position of its tile so far (of none, if the tile ends with the chunk:
  // the next chunk's first tile is then another one, whose cost would count the former's position)
  int last_run, last_top;
  int kept_run[KEPT], kept_top[KEPT];   // before chunk i * every
  long long kept_sum[KEPT];
  long long sum[TT_WARPS];
  long long lo, hi, per;   // this CTA's share, costs lo .. hi (none if hi <= lo); length of a share
  long long found_at;      // cost before the tile in which the share begins
  int found;               // that tile's first token
};

// The cost of all tiles, summed up by the whole CTA, a thread a token; and where the CTA's share begins.  Short rather than
// quick: the code runs once, and a line of it takes longer to fetch than to run.
__device__ __noinline__ void make_plan(const TreeParams& a, PlanMem& m) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, per_one = 128 / a.G;
  const int every = (a.T / TT_THREADS / KEPT + 1) * TT_THREADS;
  long long lo = 0, per = 0, total = 0;
  int start = 0, run = -1, top = INT32_MIN;
  long long sum = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {   // a second pass, where the list is longer than the CTA, finds the place of the share
    long long c = 0, at = 0;
    int from = 0;
    int next[6];   // sequence and position of a thread's token, the one before it and the one behind it, of the next chunk
    auto fetch = [&](int base) {
      const int t = base + tid;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int u = i == 0 ? t : i == 1 ? t - 1 : t + 1;
        const bool is = u >= 0 && u < a.T;
        next[2 * i] = is ? __ldg(a.seq + u) : 0, next[2 * i + 1] = is ? __ldg(a.pos + u) : -1;
      }
    };
    fetch(start);
#pragma unroll 1
    for (int base = start; base < a.T && (pass == 0 || sum <= lo); base += TT_THREADS) {
      if (tid == 0 && base % every == 0) m.kept_run[base / every] = run, m.kept_top[base / every] = top, m.kept_sum[base / every] = sum;
      const int t = base + tid;
      const bool in = t < a.T, behind = t + 1 < a.T;
      const int s = next[0], p = next[1], sb = next[2], pb = next[3], sn = next[4], pn = next[5];
      fetch(base + TT_THREADS);
      // first token of the run
      const uint32_t begins = __ballot_sync(0xffffffffu, in && (t == 0 || other_run(s, p, sb, pb)));
      if (lane == 0) m.run[warp] = begins ? base + 32 * warp + 31 - __clz(begins) : -1;
      m.top[tid] = tid == 0 ? top : INT32_MIN;
      __syncthreads();
      const uint32_t upto = begins & (0xFFFFFFFFu >> (31 - lane));
      const int former = max(run, __reduce_max_sync(0xffffffffu, lane < warp ? m.run[lane] : -1));
      const int r = upto ? base + 32 * warp + 31 - __clz(upto) : former;
      const int idx = (t - r) % a.per, slot = max(t - idx - base, 0);
      // the largest position of a tile: of its tokens in this warp, then by the last of these (a lane behind the list has -1 and
      // belongs to the last tile, or to none that counts)
      const uint32_t heads = __ballot_sync(0xffffffffu, idx == 0) | 1u;
      const int behind_head = lane - (31 - __clz(heads & (0xFFFFFFFFu >> (31 - lane))));
      int high = p;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, high, o);
        if (behind_head >= o) high = max(high, x);
      }
      if (lane == 31 || heads >> (lane + 1) & 1u) atomicMax(&m.top[slot], high);
      __syncthreads();
      c = 0;
      const bool last = in && (!behind || other_run(s, p, sn, pn) || idx == a.per - 1);   // a tile's last token
      if (last) c = Unit(idx + 1, m.top[slot], a.tab.N, per_one).cost() * a.H;
      const long long own = c;
#pragma unroll 1
      for (int o = 1; o < 32; o *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c += x;
      }
      if (lane == 31) m.sum[warp] = c;
      if (tid == TT_THREADS - 1) m.last_run = r, m.last_top = last ? INT32_MIN : m.top[slot];
      __syncthreads();
      run = m.last_run, top = m.last_top;
      // the warps' sums, in two parts of 32 bits (a chunk's are below 2^51)
      const long long of = lane < TT_WARPS ? m.sum[lane] : 0, mine = lane < warp ? of : 0;
      auto all = [](long long x) {
        const uint32_t low = __reduce_add_sync(0xffffffffu, (uint32_t)x & 0xFFFFFFu), high = __reduce_add_sync(0xffffffffu, (uint32_t)(x >> 24));
        return ((long long)high << 24) + low;
      };
      at = sum + c - own + all(mine);
      sum += all(of);
      c = own, from = t - idx;
      if (pass && lo >= at && lo < at + c) m.found = from, m.found_at = at;
      __syncthreads();
    }
    if (pass) break;
    // No share is shorter than the step from a unit's first block to its second: every CTA between those of a unit's first
    // and last block then holds a block of it.
    const long long most = quotient(sum, COST_UNIT + COST_TWO);
    per = quotient(sum, most < 1 ? 1 : most < (long long)gridDim.x ? most : (long long)gridDim.x) + 1;
    lo = per * blockIdx.x, total = sum;
    if (a.T <= TT_THREADS) {
      if (lo >= at && lo < at + c) m.found = from, m.found_at = at;
      break;
    }
    // from the last state kept that lies not behind it
    int k = (a.T - 1) / every;
    while (k > 0 && m.kept_sum[k] > lo) --k;
    start = k * every, run = m.kept_run[k], top = m.kept_top[k], sum = m.kept_sum[k];
  }
  if (tid == 0) m.lo = lo, m.hi = min(lo + per, total), m.per = per;
  __syncthreads();
}

// ---------------------------------------------------------------------------
// The queries as two E4M3 terms
// ---------------------------------------------------------------------------
// A lane 16 channels, for all tiles beforehand: CTAs that hold parts of one context read the same queries, and the attention
// kernel is short of instruction cache (four of its warps took 8,500 cycles for 128 rows).  It takes 1 us for few rows; for
// 4,096 tokens of 32 heads 13 us, about as much as the attention kernel gained there.
template <int D>
__global__ void __launch_bounds__(256) kv_tree_queries_kernel(const TreeParams a) {
  constexpr int LR = D / 16;   // lanes a row
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int sub = (int)(i % LR), Hq = a.H * a.G;
  const long long row = i / LR;   // (whole warps stay: 32 is a multiple of LR)
  const bool in = row < (long long)a.T * Hq;
  const int t = in ? (int)(row / Hq) : 0, hq = in ? (int)(row % Hq) : 0, h = hq / a.G;
  pdl_wait();
  pdl_launch_dependents();
  const uint4* src = reinterpret_cast<const uint4*>(a.q + t * a.q_stride + (size_t)hq * D) + 2 * sub;
  const uint4 u = __ldg(src), v = __ldg(src + 1);
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) mx = __vmaxu2(mx, w[k] & 0x7FFF7FFFu);
  mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
  for (int o = 1; o < LR; o *= 2) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // least e with max|q| <= 448 * 2^e
  const int bits = (int)(min(mx, 0x7F7Fu) << 16);
  const int e = max((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0), -118);
  const float down = pow2f(-e);
  const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;   // a row's factor is not negative: see the maximum
  uint32_t hi[4], rest[4];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t y = w[k] ^ flip;
    // (FP16 holds what lies above 2^-23 of the largest exactly; the difference to the nearest code is exact)
    const uint32_t f = pack_f16x2(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xFFFF0000u) * down);
    const uint32_t c = e4m3x2_of_f16x2(f), d = e4m3x2_of_f16x2(sub_f16x2(f, e4m3x2_to_f16x2(c)));
    hi[k / 2] = k & 1 ? hi[k / 2] | c << 16 : c;
    rest[k / 2] = k & 1 ? rest[k / 2] | d << 16 : d;
  }
  if (!in) return;
  const size_t at = (size_t)h * a.q_rows + (size_t)t * a.G + (hq - h * a.G), term = (size_t)a.H * a.q_rows;
  reinterpret_cast<uint4*>(a.codes + at * D)[sub] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  reinterpret_cast<uint4*>(a.codes + (term + at) * D)[sub] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
  if (sub == 0) a.factors[at] = mx > 0x7F7Fu ? __int_as_float(0x7FC00000) : fabsf(a.scale) * LOG2E * pow2f(e);
}

// ---------------------------------------------------------------------------
// The attention kernel
// ---------------------------------------------------------------------------

// A row's part of one block that not every row sees as a whole, or whose values' scales differ too much, or are too large,
// for the ordinary way: every token has an exponent ev of its own in its weight, and the terms of the sum of exponentials
// are formed without it (they may be of any size where the weight has vanished).  By a whole warp.
//
// The largest logit plus ev.  (A key's scale times the row's factor is exact; times S either may pass 2^128.)
__device__ __noinline__ float careful_max(uint32_t S, const float* kf, const float* ev, float f, uint64_t seen) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < KV_BLOCK; c += 16) {
    const uint32_t bits = (uint32_t)(seen >> c);
    uint32_t s[16];
    tmem_ld16(S + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (bits >> x & 1u) mx = fmaxf(mx, fmaf(__uint_as_float(s[x]), kf[c + x] * f, ev[c + x]));
  }
  return mx;
}
// The weights against base; the sum of the terms.
__device__ __noinline__ float careful_weights(uint32_t S, const float* kf, const float* ev, float f, float base, uint64_t seen) {
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < KV_BLOCK; c += 16) {
    const uint32_t bits = (uint32_t)(seen >> c);
    uint32_t s[16], pk[8];
    tmem_ld16(S + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; x += 2) {
      float v0 = fmaf(__uint_as_float(s[x]), kf[c + x] * f, ev[c + x]) - base;
      float v1 = fmaf(__uint_as_float(s[x + 1]), kf[c + x + 1] * f, ev[c + x + 1]) - base;
      if (!(bits >> x & 1u)) v0 = -INFINITY;
      if (!(bits >> (x + 1) & 1u)) v1 = -INFINITY;
      if (bits >> x & 1u) sum += exp2f(v0 - ev[c + x]);
      if (bits >> (x + 1) & 1u) sum += exp2f(v1 - ev[c + x + 1]);
      pk[x / 2] = pack_f16x2(ex2(v0), ex2(v1));
    }
    tmem_st8(S + c / 2, pk);
  }
  return sum;
}

// The largest of half a block's S times the keys' scales.
__device__ __noinline__ float half_max(uint32_t S, const float* kf) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 32; c += 16) {
    uint32_t s[16];
    tmem_ld16(S + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; x += 2) mx = max3(mx, __uint_as_float(s[x]) * kf[c + x], __uint_as_float(s[x + 1]) * kf[c + x + 1]);
  }
  return mx;
}
// 32 weights times sc.
__device__ __noinline__ void rescale_weights(uint32_t P, float sc) {
  uint32_t w[16];
  tmem_ld16(P, w);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    const float2 y = f16x2_to_f32x2(w[x]);
    w[x] = pack_f16x2(y.x * sc, y.y * sc);
  }
  tmem_st16(P, w);
}

// What runs once a unit, or seldom, is out of line: the loops over the blocks shall stay close together.
//
// Slots of a block that token i of the unit sees.
__device__ __noinline__ uint64_t seen_by(const TreeParams& a, const Item& x, int i) {
  return seen_bits(a.mask ? a.mask + (size_t)(x.t0 + i) * a.words : nullptr, a.words, x.begin, __ldg(a.pos + x.t0 + i), x.blk);
}
// Slots that some row of it sees.  By a whole warp.
__device__ __noinline__ uint64_t seen_by_some(const TreeParams& a, const Item& x) {
  uint64_t seen = 0;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < x.n; i += 32)
    seen |= seen_by(a, x, i);
  __syncwarp();
  return (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(seen >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)seen);
}
// Whether a row more than 2^15 below the block's largest scale is not all zeros; c0, c1: scales of tokens lane and lane + 32
// (0: does not count).  By a whole warp.
template <int D>
__device__ __noinline__ bool far_below(const unsigned char* raw, int c0, int c1, int top) {
  bool far = false;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int c = i ? c1 : c0;
    if (c == 0 || top - c <= 15) continue;
#pragma unroll 1
    for (int j = 0; j < D / 16; ++j) {
      const uint4 w = reinterpret_cast<const uint4*>(raw + ((threadIdx.x & 31) + 32 * i) * D)[j];
      far |= ((w.x | w.y | w.z | w.w) & 0x7F7F7F7Fu) != 0;
    }
  }
  __syncwarp();
  return __any_sync(0xffffffffu, far);
}
// The outputs of row r of group w: of two tiles each group has its rows; of one tile (O, O + 128: either group's part of
// every row, times c0 and c1) each joins half of the channels.
// (tr, head: the row's token in its tile and its head.)
template <int D>
__device__ __noinline__ void store_rows(const TreeParams& a, const Item& x, uint32_t O, int r, int per_one, int tr, int head, int w,
                                        float m, float l, float c0, float c1) {
  const bool two = x.flags & F_TWO, some = x.flags & F_SOME, halves = some && !two, both = halves && x.blk > 1;
  const int row = (two ? w * per_one * a.G : 0) + r, tok = (two ? w * per_one : 0) + tr;
  const bool my = tr < per_one && tok < x.n && (two || some || w == 0);
  if (!__any_sync(0xffffffffu, my)) return;
  const size_t at = ((size_t)(x.t0 + tok) * a.H + x.h) * a.G + head, part = (size_t)x.slot * a.rows + row;
  if (my && (two || w == 0)) {
    if (x.slot >= 0) a.ml[part] = make_float2(m, l);
    else if (a.lse) a.lse[at] = l == 0.0f ? -INFINITY : LN2 * ((m > -INFINITY ? m - P_SHIFT : 0.0f) + log2f(l));
  }
  if (two) O += w * 128;
  if (x.slot < 0) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    c0 *= inv, c1 *= inv;
  }
  const int cb = halves ? w * (D / 2) : 0, ce = halves ? cb + D / 2 : D;
  const bool none = !some || (x.slot < 0 && l == 0.0f);
#pragma unroll 1
  for (int c = cb; c < ce; c += 16) {
    uint32_t o[16], o1[16];
    tmem_ld16(O + c, o);
    if (both) tmem_ld16(O + 128 + c, o1);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = none ? 0u : __float_as_uint(__uint_as_float(o[i]) * c0);
    if (both && !none) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(fmaf(__uint_as_float(o1[i]), c1, __uint_as_float(o[i])));
    }
    if (!my) continue;
    if (x.slot >= 0) {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<uint4*>(a.part + part * D + c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    } else {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
      st_v8(a.out + at * D + c, b);
    }
  }
}
// O of a whole warp's rows times sc.
template <int D>
__device__ __noinline__ void rescale(uint32_t O, float sc) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld16(O + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sc);
    tmem_st16(O + c, o);
  }
}

// A warp's waits.  In line and short: five roles' code competes for the SM's instruction cache.  A try suspends the warp for
// up to 2 us (without that time given they poll so often that they cost the others 1 to 2%), so that TRIES take a few
// seconds at most; where a budget is set (PATIENT false) a wait polls.  A wait that runs out makes every later one of the
// warp give up at once; who has waited for a ring's slot must look at `left` before using it.
constexpr int TRIES = 1 << 21;
template <bool PATIENT>
struct Waits {
  int left;   // tries of a wait; 0: some wait has given up
  __device__ __forceinline__ void operator()(uint64_t* bar, int phase) {
#define BRE_WAIT(how, hint)                                                                                                \
  asm volatile(                                                                                                           \
      "{\n\t.reg .pred p;\n\t.reg .s32 n;\n\tmov.s32 n, %0;\n"                                                             \
      "AGAIN:\n\tmbarrier." how ".parity.shared::cta.b64 p, [%1], %2" hint ";\n\tvote.sync.all.pred p, p, 0xffffffff;\n\t"        \
      "@p bra THERE;\n\tsub.s32 n, n, 1;\n\tsetp.gt.s32 p, n, 0;\n\t@p bra AGAIN;\n\tmov.s32 %0, 0;\n"                   \
      "THERE:\n\t}"                                                                                                       \
      : "+r"(left)                                                                                                        \
      : "r"(smem_u32(bar)), "r"((uint32_t)phase & 1u)                                                                     \
      : "memory")
    if (PATIENT) BRE_WAIT("try_wait", ", 2000");
    else BRE_WAIT("test_wait", "");
#undef BRE_WAIT
  }
};

struct TreeBars {
  uint64_t k_full[TT_K], k_empty[TT_K], v_full[TT_V], v_empty[TT_V], v16_full[TT_V16], v16_empty[TT_V16];
  uint64_t gr_full[2][TT_GROUP], gr_empty[2][TT_GROUP], p_full[2][2], o_done[2][2], q_full[2], q_empty[2];
  uint64_t swap_in, swap_out, drain;
};

template <int D, bool PATIENT>
__global__ void __launch_bounds__(TT_THREADS, 1)
    kv_tree_kernel(const __grid_constant__ TreeParams a, const __grid_constant__ CUtensorMap key_map,
                   const __grid_constant__ CUtensorMap query_map) {
  using M = TreeMem<D>;
  constexpr uint32_t COLS = 512;   // tensor memory: S / P of either softmax group twice at 0 .. 255, their O at 256 and 384
  constexpr int PANEL = KV_BLOCK * 128;
  extern __shared__ unsigned char sm_raw[];
  __shared__ TreeBars bar;
  __shared__ Item to_v[TT_V], group[2][TT_GROUP];
  __shared__ int to_s[TT_K], to_o[TT_V16];
  __shared__ __align__(16) float kf[TT_SC][KV_BLOCK], ev_f[TT_SC][KV_BLOCK];   // keys' scales; the values' exponents
  __shared__ float ev_top[TT_SC];                  // the exponent that all weights of a block have; NaN: each has its own, or keys are large
  __shared__ float2 swap[2][128];                  // a row's maximum and sum in either softmax group
  __shared__ PlanMem plan;
  __shared__ uint32_t tmem_s;
  unsigned char* const sm = sm_raw + ((0u - smem_u32(sm_raw)) & 1023u);   // (still known to be shared memory)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  static_assert(TT_K == 4 && TT_V == 4 && TT_V16 == 4 && TT_GROUP == 4, "barriers are set up in one loop");
  if (tid < 4) {
    const int i = tid, g = i & 1, j = i >> 1;
    mbar_init(&bar.k_full[i], 1), mbar_init(&bar.k_empty[i], 2), mbar_init(&bar.v_full[i], 1), mbar_init(&bar.v_empty[i], 4);
    mbar_init(&bar.v16_full[i], 2), mbar_init(&bar.v16_empty[i], 1);
    mbar_init(&bar.gr_full[0][i], 3), mbar_init(&bar.gr_full[1][i], 3), mbar_init(&bar.gr_empty[0][i], 4), mbar_init(&bar.gr_empty[1][i], 4);
    mbar_init(&bar.p_full[g][j], 4), mbar_init(&bar.o_done[g][j], 1);
    if (j == 0) mbar_init(&bar.q_full[g], 1), mbar_init(&bar.q_empty[g], 2);
    if (i == 0) mbar_init(&bar.swap_in, 8), mbar_init(&bar.swap_out, 8), mbar_init(&bar.drain, 3);
    fence_mbar_init();
  }
  if (warp == W_S) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();   // (only now that the CTA holds its tensor memory: see kv_attend_tiles.cu)
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  // What the plan is made from was there before the queries' kernel let this one start; what that kernel writes was not.
  make_plan(a, plan);
  pdl_wait();
  const bool works = plan.lo < plan.hi;
  Waits<PATIENT> wait{PATIENT ? TRIES : (int)min(max(a.wait / 32, 1LL), (long long)INT32_MAX)};

  if (!works) {
    if (tid == 0) a.join[blockIdx.x].parts = 0;
  } else if (warp == W_LOAD) {
    // ---- walk: tiles from plan.found on, kv heads, blocks
    const int per_one = 128 / a.G;
    int it = 0, kb = 0, qb = 0;   // items, blocks; the next one-tile unit's query buffer
    Pair uses{0, 0};              // units of either query buffer so far
    Join join{0, 0, 0, 0};
    // to the S warp and to the converting warps; page < 0: nothing to copy
    auto publish = [&](const Item& x, int page) {
      const int st = it & 3;
      wait(&bar.k_empty[st], (it >> 2) + 1);
      wait(&bar.v_empty[st], (it >> 2) + 1);
      if (wait.left && lane == 0) {
        to_s[st] = x.flags;
        to_v[st] = x;
        if (page >= 0) {
          const long long ph = (long long)page * a.H + x.h;
          mbar_arrive_expect_tx(&bar.k_full[st], M::K);
          tma_load_3d(sm + M::k + st * M::K, &key_map, 0, 0, (int)ph, &bar.k_full[st]);
          mbar_arrive_expect_tx(&bar.v_full[st], M::V);
          bulk_g2s(sm + M::v + st * M::V, a.pages + ph * kv_page_bytes(D) + KV_BLOCK * D, M::V, &bar.v_full[st]);
        } else {
          mbar_arrive(&bar.k_full[st]);
          mbar_arrive(&bar.v_full[st]);
        }
      }
      __syncwarp();
      if (wait.left) ++it;
    };
    const long long lo = plan.lo, hi = plan.hi, share = plan.per;
    long long at = plan.found_at;
#pragma unroll 1
    for (int t0 = plan.found; t0 < a.T && at < hi && wait.left;) {
      // the tile: tokens in a row of one run; their number, largest and smallest position
      const int s = __ldg(a.seq + t0), p0 = __ldg(a.pos + t0);
      int n = 0, top = INT32_MIN, low = INT32_MAX;
#pragma unroll 1
      for (int i = 0; i < a.per; i += 32) {
        const int t = t0 + i + lane;
        const bool in = i + lane < a.per && t < a.T;
        const int p = in ? __ldg(a.pos + t) : -1;
        const uint32_t out = __ballot_sync(0xffffffffu, !in || other_run(s, p0, __ldg(a.seq + (in ? t : t0)), p));
        const int k = out ? __ffs(out) - 1 : 32;
        n += k;
        if (lane < k) top = max(top, p), low = min(low, p);
        if (k < 32) break;
      }
      top = __reduce_max_sync(0xffffffffu, top), low = __reduce_min_sync(0xffffffffu, low);
      const Unit unit(n, top, a.tab.N, per_one);
      const int begin = a.start && (unsigned)s < (unsigned)a.tab.B ? max(__ldg(a.start + s), 0) : 0;
      const int two = n > per_one ? F_TWO : 0;
      // blocks below this one are seen as a whole by all rows
      const int whole = (int)(min((long long)low + 1, a.mask ? (long long)begin : (long long)low + 1) / KV_BLOCK);
#pragma unroll 1
      for (int h = 0; h < a.H && wait.left; ++h, at += unit.cost()) {
        if (at + unit.cost() <= lo) continue;
        if (at >= hi) break;
        const int b0 = unit.first_from(lo - at), b1 = unit.first_from(hi - at);
        if (b0 >= b1) continue;
        int slot = -1;
        if (b0 > 0) {
          slot = 2 * blockIdx.x;
        } else if (b1 < unit.blocks) {
          slot = 2 * blockIdx.x + 1;
          // up to the CTA that holds the unit's last block
          join = Join{t0, n, h, (int)quotient(at + unit.at(unit.blocks - 1), share) - (int)blockIdx.x + 1};
        }
        if (top >= 0 && top / KV_BLOCK >= a.tab.N && b0 == 0 && lane == 0) set_err(a.err, BRE_DEVERR_PAGE);
        int jb = 0;
#pragma unroll 1
        for (int g = b0; g < b1 && top >= 0 && wait.left; g += 32) {
          const int my = g + lane < b1 ? kv_page(a.tab, s, g + lane, a.err) : -1;
#pragma unroll 1
          for (uint32_t todo = __ballot_sync(0xffffffffu, my >= 0); todo && wait.left; todo &= todo - 1) {
            const int src = __ffs(todo) - 1, blk = g + src;
            if (jb == 0) {   // the queries of one or two tiles; the buffers are free when the S of their former unit have been formed
              const int first = two ? 0 : qb, last = two ? 1 : qb;
#pragma unroll 1
              for (int b = first; b <= last; ++b) {
                wait(&bar.q_empty[b], uses[b] + 1);
                if (wait.left) {
                  if (lane == 0) {
                    mbar_arrive_expect_tx(&bar.q_full[b], 2 * M::TERM);
#pragma unroll 1
                    for (int term = 0; term < 2; ++term)
                      tma_load_3d(sm + M::q + (2 * b + term) * M::TERM, &query_map, 0, (t0 + (b - first) * per_one) * a.G,
                                  term * a.H + h, &bar.q_full[b]);
                  }
                  uses.add(b);
                }
              }
              __syncwarp();
              if (!two) qb ^= 1;
            }
            const int flags = F_BLOCK | (blk < whole ? F_FULL : 0) | two | (jb & 1 ? F_ODD : 0) | (jb == 0 ? F_BEGIN : 0) |
                              (jb < (two ? 1 : 2) ? F_NEW : 0);
            publish(Item{t0, n, h, blk, flags, slot, begin, kb}, __shfl_sync(0xffffffffu, my, src));
            ++kb, ++jb;
          }
        }
        publish(Item{t0, n, h, jb, F_END | two | (jb ? F_SOME : 0), slot, begin, kb}, -1);
      }
      t0 += n;
    }
    publish(Item{0, 0, 0, 0, F_EXIT, -1, 0, 0}, -1);
    if (lane == 0) a.join[blockIdx.x] = join;
    if (!wait.left) {   // copies that are on their way still write to this CTA's shared memory
      for (int i = max(0, it - 4); i < it; ++i) {
        mbar_wait_bounded(&bar.k_full[i & 3], i >> 2 & 1, AT_WAIT);
        mbar_wait_bounded(&bar.v_full[i & 3], i >> 2 & 1, AT_WAIT);
      }
      for (int b = 0; b < 2; ++b)
        if (uses[b]) mbar_wait_bounded(&bar.q_full[b], (uses[b] - 1) & 1, AT_WAIT);
    }
  } else if (warp == W_S || warp == W_S + 1) {
    // ---- S = Q K^T: E4M3 operands, FP32 sums, M = 128; a warp either group's
    const uint32_t id_s = (1u << 4) | ((uint32_t)(KV_BLOCK >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t q0 = desc_codes<D>(smem_u32(sm + M::q)), k0 = desc_codes<D>(smem_u32(sm + M::k));
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int w = __shfl_sync(0xffffffffu, warp - W_S, 0);
    int live = 0, qb = 0, c = 0, n = 0;   // the unit's query buffers; the next one-tile unit's; the group's S, messages so far
    Pair uses{0, 0};                      // units of either query buffer so far
#pragma unroll 1
    for (int it = 0;; ++it) {
      const int ks = it & 3;
      wait(&bar.k_full[ks], it >> 2);
      if (!wait.left) break;
      // (a warp reduction: what the MMAs' operands are formed from is then in uniform registers, where they want it)
      const int flags = (int)__reduce_or_sync(0xffffffffu, (uint32_t)to_s[ks]), two = flags & F_TWO ? 1 : 0;
      if (flags & F_BEGIN) {
        live = two ? 3 : 1 << qb;
        if (live & 1) wait(&bar.q_full[0], uses.a);
        if (live & 2) wait(&bar.q_full[1], uses.b);
      }
      const bool block = flags & F_BLOCK, mine = !block || two || (flags & F_ODD ? 1 : 0) == w;
      if (mine) {
        const int buf = c & 1;
        if (block) {
          wait(&bar.o_done[w][buf], (c >> 1) + 1);   // the weights that lay in S's columns have been used
          tc_fence_after();
          if (elect_one()) {
            const uint32_t st = tm + w * 128 + buf * 64;
            const uint64_t qd = q0 + (((two ? w : qb) * 2 * M::TERM) >> 4), kd = k0 + ((ks * M::K) >> 4);
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_codes(st, qd + ((term * M::TERM + kk * 32) >> 4), kd + ((kk * 32) >> 4), id_s, term + kk > 0);
            mma_commit(&bar.gr_full[w][n & 3]);
          }
          __syncwarp();
          ++c;
        }
        // the group's message (of a block two more parts are to come: its S and its scales)
        wait(&bar.gr_empty[w][n & 3], (n >> 2) + 1);
        if (!wait.left) break;
        if (lane < ITEM_WORDS) reinterpret_cast<int*>(&group[w][n & 3])[lane] = reinterpret_cast<const int*>(&to_v[ks])[lane];
        __syncwarp();
        if (lane < (block ? 1 : 3)) mbar_arrive(&bar.gr_full[w][n & 3]);
        ++n;
      }
      if (block && mine) {   // (the message has been copied as well)
        if (elect_one()) mma_commit(&bar.k_empty[ks]);
      } else if (lane == 0) {
        mbar_arrive(&bar.k_empty[ks]);
      }
      __syncwarp();
      if (flags & F_EXIT) break;
      if (!block && live) {
        if (elect_one()) {   // (each warp's commit goes by its own products)
          if (live & 1) mma_commit(&bar.q_empty[0]);
          if (live & 2) mma_commit(&bar.q_empty[1]);
        }
        __syncwarp();
        if (!two) qb ^= 1;
        uses.a += live & 1, uses.b += live >> 1, live = 0;
      }
    }
    // products that are under way still use tensor and shared memory
    if (elect_one()) mma_commit(&bar.drain);
    __syncwarp();
  } else if (warp == W_O) {
    // ---- O += P V: FP16 operands, P from tensor memory, V MN-major
    const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
    const uint64_t v0 = desc_mn_major(smem_u32(sm + M::v16), PANEL);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    Pair cp{0, 0};
#pragma unroll 1
    for (int kb = 0;; ++kb) {
      const int st = kb & 3;
      wait(&bar.v16_full[st], kb >> 2);
      if (!wait.left) break;
      const int flags = (int)__reduce_or_sync(0xffffffffu, (uint32_t)to_o[st]), two = flags & F_TWO ? 1 : 0;
      if (flags & F_EXIT) break;
#pragma unroll 1
      for (int g = 0; g <= two; ++g) {
        const int w = two ? g : flags & F_ODD ? 1 : 0, c = cp[w], buf = c & 1;
        wait(&bar.p_full[w][buf], c >> 1);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t o = tm + 256 + w * 128, pt = tm + w * 128 + buf * 64, more = flags & F_NEW ? 0u : 1u;
          const uint64_t vd = v0 + ((st * M::V16) >> 4);
#pragma unroll
          for (int kk = 0; kk < KV_BLOCK / 16; ++kk) mma_ts(o, pt + kk * 8, vd + ((kk * 2048) >> 4), id_o, kk > 0 ? 1u : more);
          mma_commit(&bar.o_done[w][buf]);
          if (g == two) mma_commit(&bar.v16_empty[st]);
        }
        __syncwarp();
        cp.add(w);
      }
    }
    if (elect_one()) mma_commit(&bar.drain);
    __syncwarp();
  } else if (warp >= W_CONV) {
    // ---- codes of values to FP16
    constexpr int CH = D / 16, NP = KV_BLOCK * CH / 64;   // 16-code pieces of a row, pieces a thread
    const int cw = warp - W_CONV, pair = cw >> 1, dt = (cw & 1) * 32 + lane;
    // where a thread's pieces go: two swizzled ones of 16 bytes each; the lanes of odd panels start with the second, so that
    // eight lanes meet all banks.  (The rows of a thread are whole multiples of 8 apart.)
    const int c = dt % CH, x0 = dt / CH;
    const int second = c & 4 ? 8 : 0;   // byte of the half that comes first
    const int o0 = (c / 4) * PANEL + x0 * 128 + (((2 * (c % 4) + second / 8) ^ (x0 & 7)) << 4), away = (o0 ^ 16) - o0;
    int kb = 0;
    Pair gr{0, 0};
#pragma unroll 1
    for (int it = 0;; ++it) {
      const int vs = it & 3;
      wait(&bar.v_full[vs], it >> 2);
      if (!wait.left) break;
      const int flags = to_v[vs].flags, two = flags & F_TWO;
      // the groups that hear of it
      const int who = !(flags & F_BLOCK) || two ? 3 : flags & F_ODD ? 2 : 1;
      const bool turn = (kb & 1) == pair;
      if (flags & F_BLOCK && !turn) {
        ++kb;   // the other pair's
      } else {
        const int st = kb & 3, sp = kb % TT_SC;
        const unsigned char* const raw = sm + M::v + vs * M::V;
        uint32_t up0 = 0, up1 = 0;   // of rows lane and lane + 32: what their codes are multiplied with; 0: not seen
        if (flags & F_BLOCK) {
          // slots that some row sees (others may never have been written: their values become zeros)
          uint64_t seen = ~0ull;
          if (!(flags & F_FULL)) seen = seen_by_some(a, to_v[vs]);
          const uint8_t* scales = raw + KV_BLOCK * D;
          // the largest scale of the block's values (of a NaN row and of one that no row sees: does not count)
          const int e0 = scales[KV_BLOCK + lane], e1 = scales[KV_BLOCK + 32 + lane];
          const bool s0 = (uint32_t)seen >> lane & 1u, s1 = (uint32_t)(seen >> 32) >> lane & 1u;
          const int c0 = e0 == KV_NAN || !s0 ? 0 : e0, c1 = e1 == KV_NAN || !s1 ? 0 : e1;
          const int top = max(__reduce_max_sync(0xffffffffu, max(c0, c1)), 1);
          const int least = __reduce_min_sync(0xffffffffu, min(c0 ? c0 : 255, c1 ? c1 : 255));
          bool careful = top > EV_LARGE;
          if (top - least > 15) careful |= far_below<D>(raw, c0, c1, top);
          // FP16 pairs of 2^(the row's scale - the largest), at least 2^-15
          auto relative = [&](int e) { return careful ? 0x3C003C00u : (uint32_t)max((15 - min(max(top - e, 0), 15)) << 10, 1 << 9) * 0x10001u; };
          up0 = s0 ? relative(e0) : 0u, up1 = s1 ? relative(e1) : 0u;
          if ((kb >> 1 & 1) == (cw & 1)) {   // this block's scales for the softmax, by one of the two warps
            bool k_large = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int x = lane + 32 * i, ek = scales[x], ev = i ? e1 : e0;
              k_large |= ek > 127 + K_LARGE;
              kf[sp][x] = ek == KV_NAN || ev == KV_NAN ? __int_as_float(0x7FC00000) : pow2f(ek - 127);
              ev_f[sp][x] = (float)((careful ? ev : top) - 127);
            }
            k_large = __any_sync(0xffffffffu, k_large);
            if (lane == 0) ev_top[sp] = careful || k_large ? __int_as_float(0x7FC00000) : (float)(top - 127);
            __syncwarp();
            if (lane < 2 && who >> lane & 1) mbar_arrive(&bar.gr_full[lane][gr[lane] & 3]);
          }
        }
        if (turn && flags & (F_BLOCK | F_EXIT)) {
          wait(&bar.v16_empty[st], (kb >> 2) + 1);
          if (flags & F_BLOCK) {
            const unsigned char* from = raw + dt * 16;
            unsigned char* to = sm + M::v16 + st * M::V16 + o0;
#pragma unroll 4
            for (int j = 0; j < NP; ++j) {
              const uint32_t up = __shfl_sync(0xffffffffu, j < NP / 2 ? up0 : up1, x0 + j * (64 / CH));   // (lane modulo 32)
              uint4 cur = *reinterpret_cast<const uint4*>(from);
              if (up == 0) cur = make_uint4(0, 0, 0, 0);
              const uint32_t u[4] = {second ? cur.z : cur.x, second ? cur.w : cur.y, second ? cur.x : cur.z, second ? cur.y : cur.w};
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                y[2 * i] = mul_f16x2(e4m3x2_to_f16x2(u[i] & 0xFFFFu), up), y[2 * i + 1] = mul_f16x2(e4m3x2_to_f16x2(u[i] >> 16), up);
              *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(to + away) = make_uint4(y[4], y[5], y[6], y[7]);
              from += 64 * 16, to += 64 / CH * 128;
            }
          }
          fence_proxy_async_smem();
          if (dt == 0) to_o[st] = flags;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.v16_full[st]);
          ++kb;
        }
        if (flags & F_EXIT) break;
      }
      gr.a += who & 1, gr.b += who >> 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.v_empty[vs]);
    }
  } else {
    // ---- softmax: row r of group w
    const int w = warp >> 2, r = tid & 127, per_one = 128 / a.G, tr = r / a.G, head = r - tr * a.G;
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);   // lanes 32 (warp % 4) ..
    int swaps = 0, done = 0, mine = 0;              // units of one tile; products of the group, of this unit
    float m = -INFINITY, l = 0.0f, f = 0.0f;        // m: the maximum that the weights are held against
    int tl = 0;
    bool warp_live = false, large = false;
#pragma unroll 1
    for (int it = 0;; ++it) {
      wait(&bar.gr_full[w][it & 3], it >> 2);
      if (!wait.left) break;
      const Item& x = group[w][it & 3];
      const int flags = x.flags;
      if (flags & F_BLOCK) {
        const int buf = done & 1, sp = x.kb % TT_SC;
        const uint32_t S = lane_base + w * 128 + buf * 64;
        if (flags & F_NEW) {
          tl = (flags & F_TWO ? w * per_one : 0) + tr;
          const bool live = tr < per_one && tl < x.n;
          warp_live = __any_sync(0xffffffffu, live);
          f = live ? a.factors[(size_t)x.h * a.q_rows + (size_t)(x.t0 + tl) * a.G + head] : 0.0f;
          large = __any_sync(0xffffffffu, f > F_LARGE);
          if (!live) tl = -1;
        }
        const float top = ev_top[sp];
        tc_fence_after();   // (S is there as well)
        if (warp_live) {
          if (flags & F_FULL && top == top && !large) {
            // The ordinary way: every row sees the whole block, the block's values have one scale, and neither the rows' factors nor
            // the keys' scales are large.  The weights are formed
            // against the maximum so far without looking for the block's own.  Their sum bounds them: while it is below FP16's
            // largest the maximum will do (it lags by 2^7 at most).  Else, and at first, the maximum of the half block is found.
            // (Half a block at a time: a loop of half the code; the SM's instruction cache is short for five roles.)
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              uint32_t pk[16];
              float sum;
#pragma unroll 1
              for (bool again = false;; again = true) {
                uint32_t s[32];
                const float* const kh = &kf[sp][half * 32];
                const float add = top - (m > -INFINITY ? m - P_SHIFT : 0.0f);
                const uint64_t f2 = pack2(f, f), a2 = pack2(add, add);
                float sum0 = 0.0f, sum1 = 0.0f;
                tmem_ld32(S + half * 32, s);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                  const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(kh + c);
                  const float2 v0 = unpack2(fma2(mul2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), k.x), f2, a2));
                  const float2 v1 = unpack2(fma2(mul2(pack2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), k.y), f2, a2));
                  const float p0 = ex2(v0.x), p1 = ex2(v0.y), p2 = ex2(v1.x), p3 = ex2(v1.y);
                  sum0 += p0, sum1 += p1;
                  sum0 += p2, sum1 += p3;
                  pk[c / 2] = pack_f16x2(p0, p1), pk[c / 2 + 1] = pack_f16x2(p2, p3);
                }
                sum = sum0 + sum1;
                if (again || !__any_sync(0xffffffffu, tl >= 0 && (sum > P_MOST || m == -INFINITY))) break;
                // all rows of the warp take their new maximum
                const float mx = fmaf(half_max(S + half * 32, kh), f, top);   // (f is not negative; a query that gives NaN has a NaN maximum)
                if (mine > 0) wait(&bar.o_done[w][buf ^ 1], (done - 1) >> 1);
                tc_fence_after();
                // (by whole steps, so that the weights of the block's first half stay FP16 numbers; of a step that leaves none of
                // them the difference may be rounded)
                const float step = ceilf(mx - m);
                const float then = step < 1024.0f ? m + fmaxf(step, 0.0f) : mx, d = m > -INFINITY ? m - then : 0.0f;
                l = scale_sum(l, d);
                m = then;
                if (mine > 0) rescale<D>(lane_base + 256 + w * 128, ex2(d));
                if (half) rescale_weights(S, ex2(d));
              }
              tmem_st16(S + half * 16, pk);
              l = fmaf(sum, ex2(-top), l);
            }
          } else {
            const uint64_t seen = tl < 0 ? 0ull : flags & F_FULL ? ~0ull : seen_by(a, x, tl);
            const float mx = careful_max(S, kf[sp], ev_f[sp], f, seen);
            if (m == -INFINITY) m = mx;   // nothing has been added for this row yet
            if (__any_sync(0xffffffffu, mx > m)) {
              if (mine > 0) wait(&bar.o_done[w][buf ^ 1], (done - 1) >> 1);
              tc_fence_after();
              const float then = fmaxf(m, mx), d = m > -INFINITY ? m - then : 0.0f;
              l = scale_sum(l, d);
              m = then;
              if (mine > 0) rescale<D>(lane_base + 256 + w * 128, ex2(d));
            }
            l += careful_weights(S, kf[sp], ev_f[sp], f, m > -INFINITY ? weights_base(m) : 0.0f, seen);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[w][buf]), mbar_arrive(&bar.gr_empty[w][it & 3]);
        ++done, ++mine;
        continue;
      }
      if (flags & F_EXIT) break;
      // ---- the end of a unit's part
      const bool some = flags & F_SOME, halves = some && !(flags & F_TWO), both = halves && x.blk > 1;
      if (mine > 0) wait(&bar.o_done[w][(done - 1) & 1], (done - 1) >> 1);
      float c0 = 1.0f, c1 = 0.0f;
      if (halves) {
        swap[w][r] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.swap_in);
        wait(&bar.swap_in, swaps);
        const float2 y0 = swap[0][r], y1 = swap[1][r];
        m = fmaxf(y0.x, y1.x);
        const float ref = m > -INFINITY ? m : 0.0f;
        c0 = ex2(y0.x - ref), c1 = both ? ex2(y1.x - ref) : 0.0f;
        l = scale_sum(y0.y, y0.x - ref) + (both ? scale_sum(y1.y, y1.x - ref) : 0.0f);
      }
      tc_fence_after();
      if (wait.left) store_rows<D>(a, x, lane_base + 256, r, per_one, tr, head, w, m, l, c0, c1);
      if (halves) {   // neither group goes on before both have read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.swap_out);
        wait(&bar.swap_out, swaps);
        ++swaps;
      }
      m = -INFINITY, l = 0.0f, mine = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.gr_empty[w][it & 3]);
    }
  }
  if (!wait.left) set_err(a.err, BRE_DEVERR_TIMEOUT);
  // every MMA has completed before tensor memory is given back
  tc_fence_before();
  __syncthreads();
  if (warp == W_S) {
    if (works) mbar_wait_bounded(&bar.drain, 0, AT_WAIT);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Joining the parts
// ---------------------------------------------------------------------------
// Every CTA finds out which units there are to join, `ctas` at most, and takes its pieces of them (see join_at_once).
template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4) kv_tree_join_kernel(const TreeParams a, int ctas) {
  static_assert(TT_MAX_CTAS <= JOIN_WARPS * 32, "a thread an entry");
  __shared__ Join unit[TT_MAX_CTAS];
  __shared__ int sum[JOIN_WARPS], upto[TT_MAX_CTAS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Join own = tid < ctas ? a.join[tid] : Join{0, 0, 0, 0};
  const int rows = own.n * a.G;
  const int at_once = join_at_once(own.parts, JOIN_FEW);
  int n = own.parts == 0 ? 0 : (rows + at_once - 1) / at_once;   // pieces
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) n += x;
  }
  if (lane == 31) sum[warp] = n;
  __syncthreads();
  for (int w = 0; w < warp; ++w) n += sum[w];
  if (tid < ctas) unit[tid] = own, upto[tid] = n;
  __syncthreads();
  for (int i = blockIdx.x; i < upto[ctas - 1]; i += gridDim.x) {
    int u = 0;   // the first whose pieces end behind i
#pragma unroll
    for (int o = 128; o; o >>= 1)
      if (u + o <= ctas && upto[u + o - 1] <= i) u += o;
    const Join j = unit[u];
    join_rows<D>(a.ml, a.part, j.parts, JOIN_FEW, i - (u ? upto[u - 1] : 0), 1 << 20, j.n * a.G,
                 [&](int p, int r) { return (size_t)(2 * (u + p) + (p == 0)) * a.rows + r; },
                 [&](int r) { return ((size_t)(j.t0 + r / a.G) * a.H + j.h) * a.G + r % a.G; }, a.out, a.lse);
    if (j.parts > JOIN_FEW) __syncthreads();   // (join_rows' shared memory)
  }
}

template <int D, bool PATIENT>
cudaError_t launch(const TreeParams& a, const CUtensorMap& keys, const CUtensorMap& queries, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may have its shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_tree_kernel<D, PATIENT>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeMem<D>::bytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const long long pieces = (long long)a.T * a.H * a.G * (D / 16);
  cudaError_t e = launch_k(kv_tree_queries_kernel<D>, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, a);
  if (e != cudaSuccess) return e;
  e = launch_k(kv_tree_kernel<D, PATIENT>, dim3((unsigned)ctas), dim3(TT_THREADS), TreeMem<D>::bytes, s, a, keys, queries);
  if (e != cudaSuccess) return e;
  return launch_k(kv_tree_join_kernel<D>, dim3((unsigned)(JOIN_CTAS * ctas)), dim3(JOIN_WARPS * 32), 0, s, a, ctas);
}

int slot_rows(int T, int G) {   // rows of a part: those of two tiles, or all that the call has
  const long long most = 2LL * (128 / G) * G, all = (long long)T * G;
  return (int)(all < most ? all : most);
}

// (a copied box is not larger than what it is copied from)
long long query_rows(int T, int G) { return (long long)T * G < 128 ? 128 : (long long)T * G; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
size_t codes_bytes(int T, int H, int G, int D) { return up256((size_t)2 * H * query_rows(T, G) * D); }
size_t factor_bytes(int T, int H, int G) { return up256((size_t)H * query_rows(T, G) * sizeof(float)); }

}  // namespace

size_t kv_tree_ws_bytes(int T, int Hq, int H, int D) {
  const int G = Hq / H;
  if (G < 1 || G > 16) return 0;
  const size_t slots = 2 * TT_MAX_CTAS, rows = slot_rows(T, G);
  const size_t tiles = codes_bytes(T, H, G, D) + factor_bytes(T, H, G) + TT_MAX_CTAS * sizeof(Join) +
                       slots * rows * (sizeof(float2) + D * sizeof(float));
  const size_t single = tree_rows_ws_bytes(H, G, D);
  return tiles > single ? tiles : single;
}

cudaError_t launch_kv_attend_tree(const TreeArgs& t, cudaStream_t s) {
  const bre_kv_cache* c = t.cache;
  const int H = c->n_kv_heads, D = c->head_dim, G = t.Hq / H;
  // A token at a time where that costs less: such a call reads a context once for each of its tokens (mostly from L2), but needs
  // none of the tiles' preparations, worth some 6,000 blocks of a token's (16 bits a key, D = 128), and a tile's block takes as long
  // as two and a half of those.  us, a token at a time / tiles, four kv heads, G = 8, D = 128: 64 sequences of 4,096,
  // 2 tokens each 82 / 113, 3 125 / 114; 8 of 16,384, 3 60 / 66, 4 75 / 66; 32 of 2,048, 3 35 / 46, 4 41 / 47; 16 of 1,024, 8
  // 27 / 29; one of 4,096, 16 22 / 33; one of 65,536, 4 41 / 40.  D = 64: 16 of 4,096, eight kv heads, G = 1, 4 42 / 56, 8
  // 72 / 57; 64 of 200, eight kv heads, G = 4, 4 18 / 43.  G = 16: 16 of 8,192, two kv heads, D = 64, 2 29 / 35, 4 46 / 36.
  // The rule counts the table's rows, as the host does not know how many sequences have tokens in the call.  Those figures are
  // for tables of as many rows; tokens of one sequence behind 16,384 with a table of 256 rows / of one: 64 tokens 120 / 58, 512
  // 860 / 155, 640 1,050 / 190; D = 64, 1,280 1,262 / 308.  (bre.h says what a caller can do; tiles for all of these would
  // cost batches of single tokens, whose tables look the same, twice their time.)
  const long long blocks = (long long)H * t.tk.N, halves = (G > 8 ? 2 : 1) * (D / 64);
  if (t.tk.T * halves * blocks <= 5 * t.tk.B * blocks + 12000) return launch_tree_rows(t, s);
  TreeParams a{};
  a.pages = static_cast<const uint8_t*>(c->pages), a.H = H, a.G = G, a.per = 2 * (128 / G);
  a.tab = KvTable{t.tk.table, t.tk.B, t.tk.N, c->n_pages};
  a.q = t.q, a.q_stride = t.q_stride, a.seq = t.tk.seq, a.pos = t.tk.pos, a.T = t.tk.T;
  a.start = t.start, a.mask = t.mask, a.words = t.words, a.scale = t.scale, a.out = t.out, a.lse = t.lse, a.err = t.err;
  a.wait = ffn_wait_budget(0);   // 0: none set
  a.rows = slot_rows(a.T, G);
  const size_t slots = 2 * TT_MAX_CTAS;
  a.q_rows = (int)query_rows(a.T, G);
  a.codes = static_cast<unsigned char*>(t.ws);
  a.factors = reinterpret_cast<float*>(a.codes + codes_bytes(a.T, H, G, D));
  a.join = reinterpret_cast<Join*>(reinterpret_cast<unsigned char*>(a.factors) + factor_bytes(a.T, H, G));
  a.part = reinterpret_cast<float*>(a.join + TT_MAX_CTAS);
  a.ml = reinterpret_cast<float2*>(a.part + slots * a.rows * D);
  // a head's share of a page as rows of D bytes: 64 keys, 64 values, the scales
  CUtensorMap keys;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)(kv_page_bytes(D) / D), (uint64_t)c->n_pages * H};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)kv_page_bytes(D)};
  const uint32_t box[3] = {(uint32_t)D, (uint32_t)KV_BLOCK, 1};
  const auto swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_tiled(&keys, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c->pages, dims, strides, box, swizzle)) return cudaErrorInvalidValue;
  CUtensorMap queries;
  const uint64_t q_dims[3] = {(uint64_t)D, (uint64_t)a.q_rows, 2ull * H};
  const uint64_t q_strides[2] = {(uint64_t)D, (uint64_t)a.q_rows * D};
  const uint32_t q_box[3] = {(uint32_t)D, 128, 1};
  if (!encode_tiled(&queries, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.codes, q_dims, q_strides, q_box, swizzle)) return cudaErrorInvalidValue;
  const int sms = device_sm_count(), ctas = sms < TT_MAX_CTAS ? sms : TT_MAX_CTAS;
  if (a.wait) return D == 128 ? launch<128, false>(a, keys, queries, ctas, s) : launch<64, false>(a, keys, queries, ctas, s);
  return D == 128 ? launch<128, true>(a, keys, queries, ctas, s) : launch<64, true>(a, keys, queries, ctas, s);
}

}  // namespace bre

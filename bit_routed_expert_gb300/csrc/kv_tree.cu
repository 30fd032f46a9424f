// Attention over the whole cached context and a tree of drafted tokens behind it, on the 5th-generation tensor cores.
//
// The call's tokens of one sequence, all query heads of one kv head: up to 128 rows of a tile, or 256 in two tiles that
// share the blocks.  Every block of the context is read once for them: (2 D + 2) bytes a token against 4 D operations for
// each row, so DRAM sets the pace up to about 128 rows and the tensor cores beyond.
//
// One CTA an SM, which takes an equal share of the call's work: (rows, kv head) units one after the other, each a run of
// blocks; a share may begin and end inside a unit.  Such parts go to the workspace, and a second kernel joins them in the
// order of the context (the same numbers whatever the order in which CTAs finish).  The host knows neither
// lengths nor runs: every CTA adds up the work of all tiles itself and finds its place.
//
// Fourteen warps:
//   warps 0-3, 4-7  softmax, a thread a row: two tiles' rows of the same block, or, where there is one tile, its
//                   rows of the even and of the odd blocks, each with a running maximum, sum and output of its own
//   warps 8-11      queries into two E4M3 terms; the values' codes into FP16 (exact) in 128-byte-swizzled shared memory
//   warp 12         walks through the share, looks up pages and starts the copies (TMA: keys swizzled, values as they lie)
//   warp 13         issues the MMAs: S = Q K^T into tensor memory, O += P V with P read from tensor memory
//
// The keys' codes are an MMA operand as they lie in the cache.  A BF16 query is q = 2^e (a + b), a and b E4M3: a is
// q's nearest code, b the rest's, so that the two products add up to that of q itself (see bre.h for what is lost).  Two
// products of 8-bit operands take the tensor cores as long as one of 16-bit ones, and the keys need no conversion.  A key's
// scale multiplies its logit and a value's scale goes into its weight (see kv_attend.cu), both by token.
#include <atomic>

#include "kv_attend.cuh"
#include "kv_tc.cuh"

namespace bre {

namespace {

constexpr int TT_THREADS = 448;
constexpr int TT_WARPS = TT_THREADS / 32;
constexpr int W_CONV = 8, W_LOAD = 12, W_TREE_MMA = 13;
constexpr int TT_RING = 8;               // descriptors between the walking warp and the others
constexpr int TT_K = 6, TT_V = 6;        // blocks of keys, of values on their way
constexpr int TT_V16 = 3;                // blocks of converted values
constexpr int TT_MAX_CTAS = 160;
constexpr float TT_SLACK = 7.0f;         // growth of a row's maximum (log2) that needs no rescaling
// Costs of the shares: a block for one tile, for two tiles, and what a unit takes beside its blocks.
constexpr int COST_ONE = 2, COST_TWO = 3, COST_UNIT = 6;

enum : int { F_BLOCK = 1, F_FIRST = 2, F_FULL = 4, F_END = 8, F_EXIT = 16, F_TWO = 32, F_SOME = 64 };

// What the walking warp tells the others: a block, or the end of a unit's part.
struct Item {
  int t0, n, h, blk, flags, slot, begin, pad;   // slot < 0: the whole unit, its outputs are final
};

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
// Byte of (row, 16-byte piece) in such a tile.
template <int D>
__device__ __forceinline__ int swizzled(int row, int piece) {
  return row * D + ((piece ^ (D == 128 ? row & 7 : row >> 1 & 3)) << 4);
}

__device__ __forceinline__ void mma_codes(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bit x - 64 blk set: the token sees slot x (of the 64 of a block).
__device__ __forceinline__ uint64_t seen_bits(const uint64_t* __restrict__ mask, int words, int start, int pos, int blk) {
  const long long x0 = (long long)blk * KV_BLOCK;
  uint64_t own = pos >= x0 + 63 ? ~0ull : pos >= x0 ? (2ull << (pos - x0)) - 1ull : 0ull;
  if (!mask || own == 0) return own;
  const long long j = x0 - start;   // bit of the block's first slot
  uint64_t tree = 0;
  if (j < 0) {
    if (j <= -64) return own;
    tree = ((1ull << -j) - 1ull) | __ldg(mask) << -j;
  } else {
    const long long w = j / 64;
    const int r = (int)(j % 64);
    if (w < words) tree = __ldg(mask + w) >> r;
    if (r && w + 1 < words) tree |= __ldg(mask + w + 1) << (64 - r);
  }
  return own & tree;
}

// ---------------------------------------------------------------------------
// Shares
// ---------------------------------------------------------------------------
// Tiles: the list is cut where the sequence changes, where padding begins or ends, and every `per` tokens of a run.
__device__ __forceinline__ bool other_run(int s, int p, int s2, int p2) {
  return (p < 0) != (p2 < 0) || (p >= 0 && s != s2);
}

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
    const long long i = (x - COST_UNIT + step - 1) / step;
    return i < 1 ? 1 : i > blocks ? blocks : (int)i;
  }
};

struct PlanMem {
  int run[TT_WARPS], top[TT_WARPS];
  uint32_t cut[TT_WARPS];
  long long sum[TT_WARPS];
  long long found_at;   // cost before the tile in which the share begins
  int found;            // that tile's first token
};

// Adds up the cost of all tiles; on the second pass (lo >= 0) finds the tile that holds cost lo.  By the whole CTA.
__device__ long long plan_pass(const TreeParams& a, PlanMem& m, long long lo) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, per_one = 128 / a.G;
  int run = -1, top = INT32_MIN;   // of the last token so far: first token of its run; largest position of its tile
  long long sum = 0;
  for (int base = 0; base < a.T; base += TT_THREADS) {
    const int t = base + tid;
    const bool in = t < a.T;
    const int s = in ? __ldg(a.seq + t) : 0, p = in ? __ldg(a.pos + t) : -1;
    const bool begins = in && (t == 0 || other_run(s, p, __ldg(a.seq + t - 1), __ldg(a.pos + t - 1)));
    const bool cut_next = in && (t == a.T - 1 || other_run(s, p, __ldg(a.seq + t + 1), __ldg(a.pos + t + 1)));
    int r = begins ? t : -1;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, r, o);
      if (lane >= o) r = max(r, x);
    }
    if (lane == 31) m.run[warp] = r;
    __syncthreads();
    for (int w = 0; w < TT_WARPS; ++w) {
      if (w < warp) r = max(r, m.run[w]);
    }
    r = max(r, run);
    const int idx = (t - r) % a.per;
    const bool first = in && idx == 0;
    // the largest position since the tile's first token
    int v = p;
    uint32_t cut = first;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, v, o);
      const uint32_t c = __shfl_up_sync(0xffffffffu, cut, o);
      if (lane >= o) {
        if (!cut) v = max(v, x);
        cut |= c;
      }
    }
    if (lane == 31) m.top[warp] = v, m.cut[warp] = cut;
    __syncthreads();
    int before = top;
    for (int w = 0; w < TT_WARPS; ++w)
      if (w < warp) before = m.cut[w] ? m.top[w] : max(before, m.top[w]);
    if (!cut) v = max(v, before);
    long long c = 0;
    if (cut_next || (in && idx == a.per - 1)) c = Unit(idx + 1, v, a.tab.N, per_one).cost() * a.H;
    const long long mine = c;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const long long x = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += x;
    }
    if (lane == 31) m.sum[warp] = c;
    __syncthreads();
    long long all = sum;
    for (int w = 0; w < TT_WARPS; ++w) {
      if (w < warp) c += m.sum[w];
      all += m.sum[w];
    }
    const long long at = sum + c - mine;
    if (lo >= 0 && mine > 0 && lo >= at && lo < at + mine) m.found = t - idx, m.found_at = at;
    // the chunk's last token carries on
    run = max(run, -1);
    for (int w = 0; w < TT_WARPS; ++w) {
      run = max(run, m.run[w]);
      top = m.cut[w] ? m.top[w] : max(top, m.top[w]);
    }
    sum = all;
    __syncthreads();
  }
  return sum;
}

// ---------------------------------------------------------------------------
// The attention kernel
// ---------------------------------------------------------------------------

// The part of a block in a row's sum of exponentials formed without the values' scales: where a value's scale is above
// EV_LARGE the weights, which have it, may vanish although their terms do not.  By a whole warp.
__device__ __noinline__ float careful_sum(uint32_t S, const float* kf, const float* ev, float f, float base, uint64_t seen) {
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < KV_BLOCK; c += 16) {
    uint32_t s[16];
    tmem_ld16(S + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float v = fmaf(__uint_as_float(s[x]) * kf[c + x], f, ev[c + x]);
      if (seen >> (c + x) & 1ull) sum += exp2f(v - base - ev[c + x]);
    }
  }
  return sum;
}

// PATIENT: the waits have the default budget (see kv_attend_tiles.cu).
template <int D, bool PATIENT>
__global__ void __launch_bounds__(TT_THREADS, 1)
    kv_tree_kernel(const TreeParams a, const __grid_constant__ CUtensorMap key_map) {
  using M = TreeMem<D>;
  constexpr uint32_t COLS = 512;   // tensor memory: S / P of either softmax group twice at 0 .. 255, their O at 256 and 384
  constexpr int PANEL = KV_BLOCK * 128;
  extern __shared__ unsigned char sm_raw[];
  __shared__ uint64_t it_full[TT_RING], it_empty[TT_RING], sc_full[TT_RING], k_full[TT_K], k_empty[TT_K], v_full[TT_V], v_empty[TT_V],
      v16_full[TT_V16], v16_empty[TT_V16], s_full[2][2], p_full[2][2], o_done[2], q_full[2], q_empty[2], seg_done, swap_in, swap_out, drain;
  __shared__ Item ring[TT_RING];
  __shared__ __align__(16) float kf[TT_RING][KV_BLOCK], ev_f[TT_RING][KV_BLOCK], ev_inv[TT_RING][KV_BLOCK];
  __shared__ int large[TT_RING];           // some value's scale is above EV_LARGE
  __shared__ float q_factor[2][128];
  __shared__ float2 swap[2][128];          // a row's maximum and sum in either softmax group
  __shared__ PlanMem plan;
  __shared__ uint32_t tmem_s;
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_one = 128 / a.G;           // tokens of one tile of rows

  if (tid == 0) {
    for (int i = 0; i < TT_RING; ++i) mbar_init(&it_full[i], 1), mbar_init(&it_empty[i], 13), mbar_init(&sc_full[i], 1);
    for (int i = 0; i < TT_K; ++i) mbar_init(&k_full[i], 1), mbar_init(&k_empty[i], 1);
    for (int i = 0; i < TT_V; ++i) mbar_init(&v_full[i], 1), mbar_init(&v_empty[i], 4);
    for (int i = 0; i < TT_V16; ++i) mbar_init(&v16_full[i], 4), mbar_init(&v16_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) mbar_init(&s_full[i][j], 1), mbar_init(&p_full[i][j], 4);
      mbar_init(&o_done[i], 1), mbar_init(&q_full[i], 4), mbar_init(&q_empty[i], 1);
    }
    mbar_init(&seg_done, 1), mbar_init(&drain, 1), mbar_init(&swap_in, 8), mbar_init(&swap_out, 8);
  }
  fence_mbar_init();
  if (warp == W_TREE_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();   // (only now that the CTA holds its tensor memory: see kv_attend_tiles.cu)
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();

  // this CTA's share: costs lo .. hi
  const long long total = plan_pass(a, plan, -1);
  // No share is shorter than the step from a unit's first block to its second: every CTA between those of a unit's first and
  // last block then holds a block of it.
  const long long most = total / (COST_UNIT + COST_TWO);
  const long long ctas = most < 1 ? 1 : most < (long long)gridDim.x ? most : (long long)gridDim.x;
  auto share = [&](long long c) { return total * c / ctas; };
  const bool works = blockIdx.x < ctas;
  const long long lo = works ? share(blockIdx.x) : 0, hi = works ? share(blockIdx.x + 1) : 0;
  if (works) plan_pass(a, plan, lo);

  bool ok = true;   // no wait of this thread has given up
  auto wait = [&](uint64_t* bar, int phase) {
    if (ok && (PATIENT ? !try_wait_ms(bar, phase & 1) && !wait_long(bar, phase & 1) : !mbar_wait_bounded(bar, phase & 1, a.wait))) {
      ok = false;
      set_err(a.err, BRE_DEVERR_TIMEOUT);
    }
    return ok;
  };
  auto warp_wait = [&](uint64_t* bar, int phase) { return ok = __all_sync(0xffffffffu, wait(bar, phase)); };

  if (!works) {
    if (tid == 0) a.join[blockIdx.x].parts = 0;
  } else if (warp == W_LOAD) {
    // ---- walk: tiles from plan.found on, kv heads, blocks
    int it = 0, kb = 0;
    Join join{0, 0, 0, 0};
    auto publish = [&](const Item& x) {
      if (!warp_wait(&it_empty[it % TT_RING], it / TT_RING + 1)) return false;
      if (lane == 0) {
        ring[it % TT_RING] = x;
        mbar_arrive(&it_full[it % TT_RING]);
      }
      ++it;
      return true;
    };
    long long at = plan.found_at;
    for (int t0 = plan.found; t0 < a.T && at < hi && ok;) {
      // the tile: tokens in a row of one run; their number, largest and smallest position
      const int s = __ldg(a.seq + t0), p0 = __ldg(a.pos + t0);
      int n = 0, top = INT32_MIN, low = INT32_MAX;
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
      for (int h = 0; h < a.H && ok; ++h, at += unit.cost()) {
        if (at + unit.cost() <= lo) continue;
        if (at >= hi) break;
        const int b0 = unit.first_from(lo - at), b1 = unit.first_from(hi - at);
        if (b0 >= b1) continue;
        int slot = -1;
        if (b0 > 0) {
          slot = 2 * blockIdx.x;
        } else if (b1 < unit.blocks) {
          slot = 2 * blockIdx.x + 1;
          // the CTA that holds the unit's last block
          const long long x = at + unit.at(unit.blocks - 1);
          long long c = x * ctas / total;
          while (c + 1 < ctas && share(c + 1) <= x) ++c;
          while (c > 0 && share(c) > x) --c;
          join = Join{t0, n, h, (int)c - (int)blockIdx.x + 1};
        }
        if (top >= 0 && top / KV_BLOCK >= a.tab.N && b0 == 0 && lane == 0) set_err(a.err, BRE_DEVERR_PAGE);
        int some = 0;
        for (int g = b0; g < b1 && top >= 0 && ok; g += 32) {
          const int my = g + lane < b1 ? kv_page(a.tab, s, g + lane, a.err) : -1;
          for (uint32_t todo = __ballot_sync(0xffffffffu, my >= 0); todo && ok; todo &= todo - 1) {
            const int src = __ffs(todo) - 1, page = __shfl_sync(0xffffffffu, my, src), blk = g + src;
            const long long x1 = (long long)blk * KV_BLOCK + KV_BLOCK - 1;
            const bool full = x1 <= low && (!a.mask || x1 < begin);
            const int ks = kb % TT_K, vs = kb % TT_V;
            if (!warp_wait(&k_empty[ks], kb / TT_K + 1) || !warp_wait(&v_empty[vs], kb / TT_V + 1)) break;
            if (lane == 0) {
              const long long ph = (long long)page * a.H + h;
              mbar_arrive_expect_tx(&k_full[ks], M::K);
              tma_load_3d(sm + M::k + ks * M::K, &key_map, 0, 0, (int)ph, &k_full[ks]);
              mbar_arrive_expect_tx(&v_full[vs], M::V);
              bulk_g2s(sm + M::v + vs * M::V, a.pages + ph * kv_page_bytes(D) + KV_BLOCK * D, M::V, &v_full[vs]);
            }
            ++kb;
            if (!publish(Item{t0, n, h, blk, F_BLOCK | (some ? 0 : F_FIRST) | (full ? F_FULL : 0) | two, slot, begin, 0})) break;
            some = F_SOME;
          }
        }
        if (ok) publish(Item{t0, n, h, 0, F_END | two | some, slot, begin, 0});
      }
      t0 += n;
    }
    if (ok) publish(Item{0, 0, 0, 0, F_EXIT, -1, 0, 0});
    if (lane == 0) a.join[blockIdx.x] = join;
    if (!ok) {   // copies that are on their way still write to this CTA's shared memory
      for (int i = max(0, kb - TT_K); i < kb; ++i) mbar_wait_bounded(&k_full[i % TT_K], i / TT_K & 1, AT_WAIT);
      for (int i = max(0, kb - TT_V); i < kb; ++i) mbar_wait_bounded(&v_full[i % TT_V], i / TT_V & 1, AT_WAIT);
    }
  } else if (warp == W_TREE_MMA) {
    // ---- MMA.  S of a block is formed up to two products ahead of its P V.
    const uint32_t id_s = (1u << 4) | ((uint32_t)(KV_BLOCK >> 3) << 17) | ((128u >> 4) << 24);   // E4M3, FP32 sums, M = 128
    const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);   // FP16; V is MN-major
    const uint64_t q0 = desc_codes<D>(smem_u32(sm + M::q)), k0 = desc_codes<D>(smem_u32(sm + M::k));
    const uint64_t v0 = desc_mn_major(smem_u32(sm + M::v16), PANEL);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    int kb = 0, vb = 0;            // blocks whose S, whose last P V have been issued
    int cs[2] = {0, 0}, cp[2] = {0, 0};   // S and P V of either group so far
    int started[2] = {0, 0};       // products P V of this unit
    int qb = 0, uses[2] = {0, 0};  // the next one-tile unit's query buffer; uses of the buffers
    int queue = 0, queued = 0;     // groups (and whether they are a block's last) that wait for their P V: two bits each
    auto pv = [&]() {
      const int w = queue & 1, last = queue >> 1 & 1;
      queue >>= 2, --queued;
      const int buf = cp[w] & 1, st = vb % TT_V16;
      if (!warp_wait(&v16_full[st], vb / TT_V16) || !warp_wait(&p_full[w][buf], cp[w] >> 1)) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KV_BLOCK / 16; ++kk)
          mma_ts(tm + 256 + w * 128, tm + w * 128 + buf * 64 + kk * 8, v0 + ((st * M::V16 + kk * 2048) >> 4), id_o,
                 kk > 0 ? 1u : started[w] > 0);
        mma_commit(&o_done[w]);
        if (last) mma_commit(&v16_empty[st]);
      }
      __syncwarp();
      ++cp[w], started[w] = 1;
      if (last) ++vb;
    };
    int jb = 0, live = 0;          // blocks of this unit; query buffers that it uses
    int base[2] = {0, 0}, segs = 0;   // S of either group before this unit; units that had blocks
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      if (!warp_wait(&it_full[it % TT_RING], it / TT_RING)) break;
      const int flags = ring[it % TT_RING].flags;
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[it % TT_RING]);
      if (flags & F_EXIT) break;
      if (flags & F_BLOCK) {
        if (flags & F_FIRST) {
          jb = 0, live = flags & F_TWO ? 3 : 1 << qb;
          for (int i = 0; i < 2; ++i)
            if (live >> i & 1) warp_wait(&q_full[i], uses[i]);
        }
        const int ks = kb % TT_K;
        if (!warp_wait(&k_full[ks], kb / TT_K)) break;
        for (int g = 0; g < (flags & F_TWO ? 2 : 1); ++g) {
          const int w = flags & F_TWO ? g : jb & 1, qt = flags & F_TWO ? g : qb, buf = cs[w] & 1;
          // the weights that lay in S's columns must have been used (P V of the group's product before the last)
          if (cs[w] - base[w] > 1 && !warp_wait(&o_done[w], cs[w] - 2)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_codes(tm + w * 128 + buf * 64, q0 + (((qt * 2 + term) * M::TERM + kk * 32) >> 4),
                          k0 + ((ks * M::K + kk * 32) >> 4), id_s, term + kk > 0);
            mma_commit(&s_full[w][buf]);
            if (!(flags & F_TWO) || g) mma_commit(&k_empty[ks]);
          }
          __syncwarp();
          ++cs[w];
          queue |= (w | (!(flags & F_TWO) || g ? 2 : 0)) << (2 * queued++);
          if (queued > 2) pv();
        }
        ++kb, ++jb;
      }
      if (flags & F_END) {
        while (queued && ok) pv();
        started[0] = started[1] = 0;
        if (flags & F_SOME) {
          if (elect_one()) {
            mma_commit(&seg_done);
            for (int i = 0; i < 2; ++i)
              if (live >> i & 1) mma_commit(&q_empty[i]);
          }
          __syncwarp();
          // all of the unit's products have completed before the next one's begin: a wait for a product is then never
          // two phases from its barrier's state
          if (!warp_wait(&seg_done, segs)) break;
          ++segs;
          for (int i = 0; i < 2; ++i) uses[i] += live >> i & 1, base[i] = cs[i];
          if (!(flags & F_TWO)) qb ^= 1;
        }
      }
    }
    if (!ok) {   // products that are under way still use tensor and shared memory
      if (elect_one()) mma_commit(&drain);
      __syncwarp();
      mbar_wait_bounded(&drain, 0, AT_WAIT);
    }
  } else if (warp >= W_CONV && warp < W_LOAD) {
    // ---- queries to two terms; codes of values to FP16
    constexpr int CH = D / 16, NP = KV_BLOCK * CH / 128;   // 16-code pieces of a row, pieces a thread
    const int cw = warp - W_CONV, dt = cw * 32 + lane;
    int kb = 0, qb = 0, uses[2] = {0, 0}, last = 0;
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      const int slot = it % TT_RING;
      if (!warp_wait(&it_full[slot], it / TT_RING)) break;
      const Item x = ring[slot];
      if (x.flags & F_EXIT) break;
      if (x.flags & F_FIRST) {
        // rows of up to two tiles; the buffers are free when the S of their former unit have been formed
        last = x.flags & F_TWO ? 3 : 1 << qb;
        for (int i = 0; i < 2; ++i)
          if (last >> i & 1) warp_wait(&q_empty[i], uses[i] + 1);
        if (!ok) break;
        constexpr int CL = D / 32, UN = 8;   // channels a lane, rows of a warp in flight
        const int rows = x.n * a.G;
#pragma unroll 1
        for (int r0 = cw; r0 < rows; r0 += 4 * UN) {
          uint32_t w[UN][CL / 2];
#pragma unroll
          for (int j = 0; j < UN; ++j) {
            const int r = r0 + 4 * j, tl = r / a.G;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + (long long)(x.t0 + tl) * a.q_stride +
                                                                    (size_t)(x.h * a.G + r - tl * a.G) * D) + lane * (CL / 2);
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) w[j][i] = r < rows ? __ldg(src + i) : 0u;
          }
#pragma unroll
          for (int j = 0; j < UN; ++j) {
            const int r = r0 + 4 * j;
            if (r >= rows) break;
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) mx = __vmaxu2(mx, w[j][i] & 0x7FFF7FFFu);
            mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
            // least e with max|q| <= 448 * 2^e
            const int bits = (int)(min(mx, 0x7F7Fu) << 16);
            const int e = max((bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0), -118);
            const float down = pow2f(-e);
            uint32_t hi = 0, rest = 0;
#pragma unroll
            for (int i = 0; i < CL / 2; ++i) {
              const float u = __uint_as_float(w[j][i] << 16) * down, v = __uint_as_float(w[j][i] & 0xFFFF0000u) * down;
              const uint32_t c = e4m3x2(u, v);
              const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(c));
              hi |= c << (16 * i);
              rest |= e4m3x2(u - f.x, v - f.y) << (16 * i);
            }
            // tile and row in it: a tile holds whole tokens
            const int tile = r >= per_one * a.G, rr = r - tile * per_one * a.G, buf = x.flags & F_TWO ? tile : qb;
            unsigned char* dst = sm + M::q + buf * 2 * M::TERM + swizzled<D>(rr, lane * CL / 16) + lane * CL % 16;
            if constexpr (CL == 4) {
              *reinterpret_cast<uint32_t*>(dst) = hi;
              *reinterpret_cast<uint32_t*>(dst + M::TERM) = rest;
            } else {
              *reinterpret_cast<uint16_t*>(dst) = (uint16_t)hi;
              *reinterpret_cast<uint16_t*>(dst + M::TERM) = (uint16_t)rest;
            }
            if (lane == 0) q_factor[buf][rr] = mx > 0x7F7Fu ? __int_as_float(0x7FC00000) : a.scale * LOG2E * pow2f(e);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          for (int i = 0; i < 2; ++i)
            if (last >> i & 1) mbar_arrive(&q_full[i]);
      }
      if (x.flags & F_BLOCK) {
        const int vs = kb % TT_V, st = kb % TT_V16;
        // slots that some row sees (others may never have been written: their values become zeros)
        uint64_t seen = ~0ull;
        if (!(x.flags & F_FULL)) {
          seen = 0;
          for (int i = lane; i < x.n; i += 32)
            seen |= seen_bits(a.mask ? a.mask + (size_t)(x.t0 + i) * a.words : nullptr, a.words, x.begin, __ldg(a.pos + x.t0 + i), x.blk);
          seen = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(seen >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)seen);
        }
        if (!warp_wait(&v_full[vs], kb / TT_V)) break;
        const unsigned char* raw = sm + M::v + vs * M::V;
        if (kb % 4 == cw) {   // this block's scales
          bool over = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = lane + 32 * i, ek = raw[KV_BLOCK * D + c], ev = raw[KV_BLOCK * D + KV_BLOCK + c];
            kf[slot][c] = pow2f(min(ek, 253) - 127);
            ev_f[slot][c] = ek == KV_NAN || ev == KV_NAN ? __int_as_float(0x7FC00000) : (float)(ev - 127);
            ev_inv[slot][c] = pow2f(127 - min(ev, 253));
            over |= ev > EV_LARGE && (seen >> c & 1ull);
          }
          over = __any_sync(0xffffffffu, over);
          if (lane == 0) large[slot] = over;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[slot]);
        }
        uint4 cur[NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const int x0 = (dt + j * 128) / CH;
          cur[j] = seen >> x0 & 1ull ? reinterpret_cast<const uint4*>(raw)[dt + j * 128] : make_uint4(0, 0, 0, 0);
        }
        if (!warp_wait(&v16_empty[st], kb / TT_V16 + 1)) break;
        // two swizzled pieces of 16 bytes; the lanes of odd panels start with the second, so that eight lanes meet all banks
        const int c = dt % CH;
        const bool second = (c / 4) & 1;
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const int x0 = (dt + j * 128) / CH;
          const int p0 = M::v16 + st * M::V16 + (c / 4) * PANEL + x0 * 128 + (((2 * (c % 4)) ^ (x0 & 7)) << 4);
          const uint32_t u[4] = {second ? cur[j].z : cur[j].x, second ? cur[j].w : cur[j].y, second ? cur[j].x : cur[j].z,
                                 second ? cur[j].y : cur[j].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * k] = e4m3x2_to_f16x2(u[k] & 0xFFFFu);
            o[2 * k + 1] = e4m3x2_to_f16x2(u[k] >> 16);
          }
          *reinterpret_cast<uint4*>(sm + (second ? p0 ^ 16 : p0)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(sm + (second ? p0 : p0 ^ 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v16_full[st]), mbar_arrive(&v_empty[vs]);
        ++kb;
      }
      if (x.flags & F_END && cw == 0 && lane == 0) mbar_arrive(&sc_full[slot]);   // (one arrival for each use of a slot)
      if (x.flags & F_END && x.flags & F_SOME) {
        for (int i = 0; i < 2; ++i) uses[i] += last >> i & 1;
        if (!(x.flags & F_TWO)) qb ^= 1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
    }
  } else if (warp < W_CONV) {
    // ---- softmax: row r of group w
    const int w = warp >> 2, r = tid & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);   // lanes 32 (warp % 4) ..
    const uint32_t O = lane_base + 256 + w * 128;
    int qb = 0, done = 0, segs = 0;   // products of this group; units that had blocks
    float m = -INFINITY, l = 0.0f, f = 0.0f;
    int jb = 0, mine = 0, pos = -1;   // blocks of this unit, those of this group; the row's position
    int tl = 0;
    bool live = false, warp_live = false;
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      const int slot = it % TT_RING;
      if (!warp_wait(&it_full[slot], it / TT_RING)) break;
      const int flags = ring[slot].flags;
      if (flags & F_EXIT) break;
      if (flags & F_FIRST) jb = 0;
      if (flags & F_BLOCK && (flags & F_TWO || (jb & 1) == w)) {
        const int buf = done & 1;
        const uint32_t S = lane_base + w * 128 + buf * 64;
        if (mine == 0) {
          const int tr = r / a.G;
          tl = (flags & F_TWO ? w * per_one : 0) + tr;
          live = tr < per_one && tl < ring[slot].n;
          pos = live ? __ldg(a.pos + ring[slot].t0 + tl) : -1;
          warp_live = __any_sync(0xffffffffu, live);
        }
        if (!warp_wait(&sc_full[slot], it / TT_RING)) break;
        if (!warp_wait(&s_full[w][buf], done >> 1)) break;
        tc_fence_after();
        if (mine == 0) f = q_factor[flags & F_TWO ? w : qb][r];
        if (warp_live) {
          uint32_t s[64];
          tmem_ld32(S, s);
          tmem_ld32(S + 32, s + 32);
          uint64_t seen = live ? ~0ull : 0ull;
          if (!(flags & F_FULL) && live)
            seen = seen_bits(a.mask ? a.mask + (size_t)(ring[slot].t0 + tl) * a.words : nullptr, a.words, ring[slot].begin, pos,
                             ring[slot].blk);
          const uint64_t f2 = pack2(f, f);
          tmem_wait_ld();
          float mx = -INFINITY;
#pragma unroll
          for (int x = 0; x < 64; x += 4) {
            const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(&kf[slot][x]);
            const ulonglong2 ev = *reinterpret_cast<const ulonglong2*>(&ev_f[slot][x]);
            const float2 v0 = unpack2(fma2(mul2(pack2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), kk.x), f2, ev.x));
            const float2 v1 = unpack2(fma2(mul2(pack2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), kk.y), f2, ev.y));
            s[x] = __float_as_uint(v0.x), s[x + 1] = __float_as_uint(v0.y);
            s[x + 2] = __float_as_uint(v1.x), s[x + 3] = __float_as_uint(v1.y);
          }
          if (!(flags & F_FULL)) {
#pragma unroll
            for (int x = 0; x < 64; ++x)
              if (!(seen >> x & 1ull)) s[x] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int x = 0; x < 64; x += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
          if (!live) mx = -INFINITY;
          if (m == -INFINITY) m = mx;   // nothing has been added for this row yet
          if (__any_sync(0xffffffffu, mx > m + TT_SLACK)) {
            // some row's weights would outgrow FP16: all rows of the warp take their new maximum.  (P V of the product
            // before the last has completed: S of this one was formed after it.)
            if (mine > 0 && !warp_wait(&o_done[w], done - 1)) break;
            tc_fence_after();
            const float nm = fmaxf(m, mx), d = m > -INFINITY ? m - nm : 0.0f, sc = ex2(d);
            m = nm;
            l = scale_sum(l, d);
            if (mine > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_ld16(O + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * sc);
                tmem_st16(O + c, o);
              }
            }
          }
          const float base = m > -INFINITY ? m - P_SHIFT : 0.0f;
          if (large[slot]) l += careful_sum(S, kf[slot], ev_f[slot], f, base, seen);
          const uint64_t nb2 = pack2(-base, -base);
          uint64_t add = 0;
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 64; x += 4) {
            const ulonglong2 iv = *reinterpret_cast<const ulonglong2*>(&ev_inv[slot][x]);
            const float2 v0 = unpack2(add2(pack2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), nb2));
            const float2 v1 = unpack2(add2(pack2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), nb2));
            const float p0 = ex2(v0.x), p1 = ex2(v0.y), p2 = ex2(v1.x), p3 = ex2(v1.y);
            add = fma2(pack2(p0, p1), iv.x, fma2(pack2(p2, p3), iv.y, add));
            pk[x / 2] = pack_f16x2(p0, p1), pk[x / 2 + 1] = pack_f16x2(p2, p3);
          }
          const float2 sum = unpack2(add);
          if (!large[slot]) l += sum.x + sum.y;
          tmem_st16(S, pk);
          tmem_st16(S + 16, pk + 16);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w][buf]);
        ++done, ++mine;
      }
      if (flags & F_BLOCK) ++jb;
      if (flags & F_END) {
        const Item x = ring[slot];
        const int count = x.n * a.G;
        if (flags & F_SOME) {
          if (!warp_wait(&seg_done, segs)) break;
          tc_fence_after();
        }
        if (flags & F_TWO || !(flags & F_SOME)) {
          // rows of its own; of a unit without blocks the first group answers for one tile
          const int tr = r / a.G, row = (flags & F_TWO ? w * per_one : 0) * a.G + r;
          const bool my = tr < per_one && row < count && (flags & F_TWO || w == 0);
          const bool any = flags & F_SOME;
          if (my && x.slot >= 0) a.ml[(size_t)x.slot * a.rows + row] = make_float2(any ? m : -INFINITY, any ? l : 0.0f);
          const int tok = row / a.G;
          const size_t at = ((size_t)(x.t0 + tok) * a.H + x.h) * a.G + (row - tok * a.G);
          const float inv = 1.0f / l;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16], b[8];
            if (any) {
              tmem_ld16(O + c, o);
              tmem_wait_ld();
            }
            if (!my) continue;
            if (x.slot >= 0) {
              float* dst = a.part + ((size_t)x.slot * a.rows + row) * D + c;
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<uint4*>(dst + i) = any ? make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]) : make_uint4(0, 0, 0, 0);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                b[i] = !any || l == 0.0f ? 0u : pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
              st_v8(a.out + at * D + c, b);
            }
          }
          if (my && x.slot < 0 && a.lse)
            a.lse[at] = !any || l == 0.0f ? -INFINITY : LN2 * ((m > -INFINITY ? m - P_SHIFT : 0.0f) + log2f(l));
        } else {
          // the two groups have a part of every row each: either joins half of the channels
          swap[w][r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(&swap_in);
          if (!warp_wait(&swap_in, segs)) break;
          const float2 y0 = swap[0][r], y1 = swap[1][r];
          const bool both = jb > 1;   // else the second group has nothing, its O least of all
          const float top = fmaxf(y0.x, y1.x), ref = top > -INFINITY ? top : 0.0f;
          const float c0 = ex2(y0.x - ref), c1 = both ? ex2(y1.x - ref) : 0.0f;
          const float sum = scale_sum(y0.y, y0.x - ref) + (both ? scale_sum(y1.y, y1.x - ref) : 0.0f);
          const bool my = r < count;
          if (my && x.slot >= 0 && w == 0) a.ml[(size_t)x.slot * a.rows + r] = make_float2(top, sum);
          const int tok = r / a.G;
          const size_t at = ((size_t)(x.t0 + tok) * a.H + x.h) * a.G + (r - tok * a.G);
          const float inv = 1.0f / sum;
          const bool warp_my = __any_sync(0xffffffffu, my);
#pragma unroll 1
          for (int c = w * (D / 2); warp_my && c < (w + 1) * (D / 2); c += 16) {
            uint32_t o[16], o1[16], b[8];
            tmem_ld16(lane_base + 256 + c, o);
            if (both) tmem_ld16(lane_base + 384 + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float v = __uint_as_float(o[i]) * c0;
              if (both) v = fmaf(__uint_as_float(o1[i]), c1, v);
              o[i] = __float_as_uint(v);
            }
            if (!my) continue;
            if (x.slot >= 0) {
              float* dst = a.part + ((size_t)x.slot * a.rows + r) * D + c;
#pragma unroll
              for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                b[i] = sum == 0.0f ? 0u : pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
              st_v8(a.out + at * D + c, b);
            }
          }
          if (my && x.slot < 0 && a.lse && w == 0) a.lse[at] = sum == 0.0f ? -INFINITY : LN2 * (ref - (top > -INFINITY ? P_SHIFT : 0.0f) + log2f(sum));
        }
        if (flags & F_SOME) {
          // neither group goes on before both have read (and seen that the unit is done)
          tc_fence_before();
          __syncwarp();
          if (flags & F_TWO) {
            if (lane == 0) mbar_arrive(&swap_in);
            if (!warp_wait(&swap_in, segs)) break;
          }
          if (lane == 0) mbar_arrive(&swap_out);
          if (!warp_wait(&swap_out, segs)) break;
          ++segs;
          if (!(flags & F_TWO)) qb ^= 1;
        }
        m = -INFINITY, l = 0.0f, mine = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[slot]);
    }
  }
  // every MMA has completed before tensor memory is given back: the softmax has waited for the units' ends
  tc_fence_before();
  __syncthreads();
  if (warp == W_TREE_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS) : "memory");
  }
}

// ---------------------------------------------------------------------------
// Joining the parts
// ---------------------------------------------------------------------------
// A warp a row: the parts' maxima and sums by the lanes, then the outputs, part after part.
constexpr int TJ_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(TJ_WARPS * 32) kv_tree_join_kernel(const TreeParams a) {
  constexpr int CL = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const Join j = a.join[blockIdx.x];
  const int lane = threadIdx.x & 31, rows = j.n * a.G;
  if (j.parts == 0) return;
  for (int r = blockIdx.y * TJ_WARPS + (threadIdx.x >> 5); r < rows; r += gridDim.y * TJ_WARPS) {
    auto slot_of = [&](int p) { return (size_t)(2 * (blockIdx.x + p) + (p == 0)); };
    float top = -INFINITY;
    for (int p = lane; p < j.parts; p += 32) top = fmaxf(top, a.ml[slot_of(p) * a.rows + r].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top > -INFINITY ? top : 0.0f;
    float sum = 0.0f, v[CL];
#pragma unroll
    for (int i = 0; i < CL; ++i) v[i] = 0.0f;
    for (int p0 = 0; p0 < j.parts; p0 += 32) {
      const float2 y = p0 + lane < j.parts ? a.ml[slot_of(p0 + lane) * a.rows + r] : make_float2(-INFINITY, 0.0f);
      const float w = ex2(y.x - ref);
      sum += scale_sum(y.y, y.x - ref);
      const int n = min(32, j.parts - p0);
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* src = a.part + (slot_of(p0 + i) * a.rows + r) * D + lane * CL;
        if constexpr (CL == 4) {
          const float4 o = *reinterpret_cast<const float4*>(src);
          v[0] = fmaf(wi, o.x, v[0]), v[1] = fmaf(wi, o.y, v[1]), v[2] = fmaf(wi, o.z, v[2]), v[3] = fmaf(wi, o.w, v[3]);
        } else {
          const float2 o = *reinterpret_cast<const float2*>(src);
          v[0] = fmaf(wi, o.x, v[0]), v[1] = fmaf(wi, o.y, v[1]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int tok = r / a.G;
    const size_t at = ((size_t)(j.t0 + tok) * a.H + j.h) * a.G + (r - tok * a.G);
    const float inv = 1.0f / sum;
    uint32_t b[CL / 2];
#pragma unroll
    for (int i = 0; i < CL / 2; ++i) b[i] = sum == 0.0f ? 0u : pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    if constexpr (CL == 4) *reinterpret_cast<uint2*>(a.out + at * D + lane * CL) = make_uint2(b[0], b[1]);
    else *reinterpret_cast<uint32_t*>(a.out + at * D + lane * CL) = b[0];
    if (lane == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : LN2 * (ref - (top > -INFINITY ? P_SHIFT : 0.0f) + log2f(sum));
  }
}

template <int D, bool PATIENT>
cudaError_t launch(const TreeParams& a, const CUtensorMap& keys, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may have its shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_tree_kernel<D, PATIENT>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeMem<D>::bytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaError_t e = launch_k(kv_tree_kernel<D, PATIENT>, dim3((unsigned)ctas), dim3(TT_THREADS), TreeMem<D>::bytes, s, a, keys);
  if (e != cudaSuccess) return e;
  const int chunks = (a.rows + TJ_WARPS - 1) / TJ_WARPS;
  return launch_k(kv_tree_join_kernel<D>, dim3((unsigned)ctas, (unsigned)(chunks < 32 ? chunks : 32)), dim3(TJ_WARPS * 32), 0, s, a);
}

int slot_rows(int T, int G) {   // rows of a part: those of two tiles, or all that the call has
  const long long most = 2LL * (128 / G) * G, all = (long long)T * G;
  return (int)(all < most ? all : most);
}

}  // namespace

size_t kv_tree_ws_bytes(int T, int Hq, int H, int D) {
  const int G = Hq / H;
  if (G < 1 || G > 16) return 0;
  const size_t slots = 2 * TT_MAX_CTAS, rows = slot_rows(T, G);
  return TT_MAX_CTAS * sizeof(Join) + slots * rows * (sizeof(float2) + D * sizeof(float));
}

cudaError_t launch_kv_attend_tree(const TreeArgs& t, cudaStream_t s) {
  const bre_kv_cache* c = t.cache;
  const int H = c->n_kv_heads, D = c->head_dim, G = t.Hq / H;
  TreeParams a{};
  a.pages = static_cast<const uint8_t*>(c->pages), a.H = H, a.G = G, a.per = 2 * (128 / G);
  a.tab = KvTable{t.tk.table, t.tk.B, t.tk.N, c->n_pages};
  a.q = t.q, a.q_stride = t.q_stride, a.seq = t.tk.seq, a.pos = t.tk.pos, a.T = t.tk.T;
  a.start = t.start, a.mask = t.mask, a.words = t.words, a.scale = t.scale, a.out = t.out, a.lse = t.lse, a.err = t.err;
  a.wait = ffn_wait_budget(0);   // 0: none set
  a.rows = slot_rows(a.T, G);
  const size_t slots = 2 * TT_MAX_CTAS;
  a.join = static_cast<Join*>(t.ws);
  a.part = reinterpret_cast<float*>(a.join + TT_MAX_CTAS);
  a.ml = reinterpret_cast<float2*>(a.part + slots * a.rows * D);
  // a head's share of a page as rows of D bytes: 64 keys, 64 values, the scales
  CUtensorMap keys;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)(kv_page_bytes(D) / D), (uint64_t)c->n_pages * H};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)kv_page_bytes(D)};
  const uint32_t box[3] = {(uint32_t)D, (uint32_t)KV_BLOCK, 1};
  if (!encode_tiled(&keys, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c->pages, dims, strides, box,
                    D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int sms = device_sm_count(), ctas = sms < TT_MAX_CTAS ? sms : TT_MAX_CTAS;
  if (a.wait) return D == 128 ? launch<128, false>(a, keys, ctas, s) : launch<64, false>(a, keys, ctas, s);
  return D == 128 ? launch<128, true>(a, keys, ctas, s) : launch<64, true>(a, keys, ctas, s);
}

}  // namespace bre

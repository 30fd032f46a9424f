// Block selection for sparse attention: every visible block's score against a query's heads, and
// the best blocks in ascending order.
//
// The score is linear in the block's bounds: with the query's whole-number codes c,
//   sum_g sum_ch max(c hi, c lo) = P . hi - M . lo,   P = sum_g max(c, 0), M = sum_g max(-c, 0),
// so a kv head's G query heads fold into one vector of 2 D whole numbers (at most 16 * 127 = 2032:
// exact in FP16) before they meet the blocks, and the sums stay below 2^24: exact in FP32 and in
// 32-bit integers, whatever the order.
#include <cuda_fp16.h>

#include <atomic>

#include "kv_common.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// the best of a list, by one warp
// ---------------------------------------------------------------------------
// Scores are compared as keys: whole numbers in the scores' order, 0 for what cannot be taken.
__device__ __forceinline__ uint32_t key_of_score(float sc) {
  const uint32_t u = __float_as_uint(sc);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float score_of_key(uint32_t key) {
  return __uint_as_float(key ^ (~(uint32_t)((int32_t)key >> 31) | 0x80000000u));
}

// Scores are held as the whole number times 2^(bound_exp - SCORE_DOWN): below 2^24 times 2^122, they would be beyond
// FP32's range for keys near the ends of theirs, and infinities do not compare.
constexpr int SCORE_DOWN = 32;

// Keys lie in shared memory with four unused words after every 16: a lane reads 4, 8 or 16 of them
// in a row by 16-byte loads that meet no bank twice.
__host__ __device__ constexpr int key_at(int i) { return i + 4 * (i >> 4); }
constexpr int SEL_CHUNK = 512;   // entries of one selection

// Of the entries first .. n - 1 (n <= 32 R; lane l holds entries R l ..) the `want` with the largest
// keys, the first ones among equals: put(place, index, key) in ascending order; how many there are.
//
// The threshold comes by bisection of the keys, which ends as soon as a value splits off exactly
// `want` entries.  It starts between the largest key and a lower bound that costs one register a
// lane: the `want`-th largest of the 32 lanes' own largest keys (as many lanes, so as many entries,
// reach it).  Of 512 random keys about 24 lie above that bound for want = 16, so three or four
// steps over all registers are left of about twelve.
template <int R, typename Put>
__device__ __forceinline__ int warp_top(const uint32_t* keys, int first, int n, int want, Put put) {
  const int lane = threadIdx.x & 31;
  uint32_t key[R], top = 0;
#pragma unroll
  for (int j = 0; j < R; j += 4) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (R * lane + j < n) v = *reinterpret_cast<const uint4*>(keys + key_at(R * lane + j));
    key[j] = v.x, key[j + 1] = v.y, key[j + 2] = v.z, key[j + 3] = v.w;
  }
  const int from = first - R * lane, to = n - R * lane;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j >= to || j < from) key[j] = 0u;
    top = max(top, key[j]);
  }
  uint32_t lo = 1, hi = __reduce_max_sync(0xffffffffu, top) + 1u;
  if (want <= 0 || hi == 1u) return 0;
  if (__popc(__ballot_sync(0xffffffffu, top != 0u)) >= want) {
    lo = __reduce_min_sync(0xffffffffu, top != 0u ? top : hi);
    uint32_t h = hi;   // as many lanes reach lo, fewer reach h
    while (h - lo > 1) {
      const uint32_t mid = lo + (h - lo) / 2;
      const int c = __popc(__ballot_sync(0xffffffffu, top >= mid));
      if (c < want)
        h = mid;
      else
        lo = mid;
      if (c == want) break;
    }
  }
  if (lo == 1u) {   // more entries wanted than lanes have: between the smallest key and the largest
    uint32_t least = hi;
#pragma unroll
    for (int j = 0; j < R; ++j) least = min(least, key[j] != 0u ? key[j] : hi);
    lo = __reduce_min_sync(0xffffffffu, least);
  }
  // count(>= lo) >= want unless all entries are fewer; count(>= hi) = above < want
  auto count = [&](uint32_t v) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < R; ++j) c += key[j] >= v;
    return (int)__reduce_add_sync(0xffffffffu, c);
  };
  uint32_t thr = lo;
  int above = 0, got = count(lo);
  const int at_least = got;   // entries that reach lo
  while (got > want && hi - lo > 1) {
    thr = lo + (hi - lo) / 2;
    got = count(thr);
    if (got > want) {
      lo = thr;
    } else if (got < want) {
      hi = thr;
      above = got;
      got = want + 1;
    }
  }
  const bool cut = got > want;   // hi - lo = 1: some of the entries equal to lo are left out
  if (cut) thr = lo;
  got = min(want, at_least);

  int mine = 0, eq = 0;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    mine += key[j] > thr || (key[j] == thr && !cut);
    eq += key[j] == thr;
  }
  int room = eq;   // of this lane's entries equal to thr, the first `room` are taken
  if (cut) {
    int before = eq;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    room = max(0, min(eq, want - above - (before - eq)));
    mine += room;
  }
  int at = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  at -= mine;
  if (mine) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const bool tie = key[j] == thr;
      if (key[j] > thr || (tie && room > 0)) put(at++, R * lane + j, key[j]);
      room -= tie;
    }
  }
  __syncwarp();
  return got;
}

template <typename Put>
__device__ __forceinline__ int warp_top_any(const uint32_t* keys, int first, int n, int want, Put put) {
  return n <= 128 ? warp_top<4>(keys, first, n, want, put) : warp_top<16>(keys, first, n, want, put);
}

// The best `want` of `have` entries held in (ok, ob) and the entries first .. n - 1 (n <= SEL_CHUNK) of a
// further piece, which come after them, block_of(i) their blocks -> (ok, ob); how many are held then.
// (lk, lb): scratch for 2 want entries.
template <typename Block>
__device__ __forceinline__ int warp_top_piece(int have, const uint32_t* keys, int first, int n, Block block_of, int want,
                                              uint32_t* ok, int* ob, uint32_t* lk, int* lb) {
  const bool join = have > 0;
  if (join) {
    for (int i = threadIdx.x & 31; i < have; i += 32) lk[key_at(i)] = ok[key_at(i)], lb[i] = ob[i];
    __syncwarp();   // the second selection reads them in other lanes; the first may find nothing and return at once
  }
  const int got = warp_top_any(keys, first, n, want, [&](int p, int i, uint32_t key) {
    if (join)
      lk[key_at(have + p)] = key, lb[have + p] = block_of(i);
    else
      ok[key_at(p)] = key, ob[p] = block_of(i);
  });
  if (!join) return got;
  return warp_top_any(lk, 0, have + got, want, [&](int p, int i, uint32_t key) { ok[key_at(p)] = key, ob[p] = lb[i]; });
}

// The same for a list of any length.
template <typename Block>
__device__ __forceinline__ int warp_top_list(const uint32_t* keys, int first, int n, Block block_of, int want, uint32_t* ok,
                                             int* ob, uint32_t* lk, int* lb) {
  int have = 0;
  for (int base = 0; base < n; base += SEL_CHUNK)
    have = warp_top_piece(have, keys + key_at(base), first - base, min(SEL_CHUNK, n - base),
                          [&](int i) { return block_of(base + i); }, want, ok, ob, lk, lb);
  return have;
}

// ---------------------------------------------------------------------------
// the query's vector
// ---------------------------------------------------------------------------
// A lane's 2 W channels (W words, word j of head g at qr[g * stride + j]) of one token and kv head:
// P into pl and M into mi; returns the exponent of the codes.  All 32 lanes together hold the G
// heads' D channels.  rint(x 2^-e) is read off the low bits of fma(x, 2^-e, 1.5 * 2^23).  With S the
// sum of the codes, M = P - S.
template <int W>
__device__ __forceinline__ int query_vector(const uint32_t* qr, int stride, int G, int (&pl)[2 * W], int (&mi)[2 * W]) {
  constexpr float MAGIC = 12582912.0f;
  constexpr int MAGIC_BITS = 0x4B400000;
  uint32_t mx = 0;   // magnitudes of BF16 values compare like whole numbers
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < W; ++j) mx = __vmaxu2(mx, __ldg(qr + g * stride + j) & 0x7FFF7FFFu);
  mx = max(mx & 0xFFFFu, mx >> 16);
  mx = __reduce_max_sync(0xffffffffu, mx);
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) pl[i] = mi[i] = 0;
  if (mx <= 0x7F60u) {   // KV_MAX
    const int e = query_exp(bf16_bits_to_f32(mx));
    const float down = pow2f(-e);
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const uint32_t w = __ldg(qr + g * stride + j);
        const float x[2] = {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = __float_as_int(fmaf(x[i], down, MAGIC)) - MAGIC_BITS;
          pl[2 * j + i] += max(b, 0);
          mi[2 * j + i] -= b;
        }
      }
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) mi[i] += pl[i];
    return e;
  }
  // infinities count as the largest value, NaN as 0
  float amax = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    const float down = pow2f(-query_exp(amax));
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < 2 * W; ++j) {
        const uint32_t w = __ldg(qr + g * stride + j / 2);
        const float x = kv_clamp(bf16_bits_to_f32(j & 1 ? w >> 16 : w & 0xFFFFu));
        if (pass == 0) {
          amax = fmaxf(amax, fabsf(x));
        } else {
          const int c = x == x ? __float2int_rn(x * down) : 0;
          pl[j] += max(c, 0);
          mi[j] += max(-c, 0);
        }
      }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  }
  return query_exp(amax);
}

struct SelectArgs {
  const int8_t* bounds;
  const int8_t* bexp;
  int H, G;
  KvTable tab;
  const uint16_t* q;
  long long q_stride;
  const int32_t* seq;
  const int32_t* pos;
  int T, k, n_sink, n_local;
  int32_t* ids;
  float* scores;
  int32_t* err;
};

// ---------------------------------------------------------------------------
// what must be taken
// ---------------------------------------------------------------------------
// The blocks that must be taken are the first n_sink and the last n_local: with the selection
// between them the list is in order, and no entry needs a test of its own.
struct Forced {
  int sinks, local0, nb;   // blocks [0, sinks) and [local0, nb) must be taken; nb visible blocks
  int paged;               // those of them that have pages
  __device__ __forceinline__ int slots() const { return sinks + nb - local0; }
  __device__ __forceinline__ int block(int slot) const { return slot < sinks ? slot : local0 + slot - sinks; }
};
// By one warp.
__device__ __forceinline__ Forced forced_blocks(const SelectArgs& a, int s, int p, int nb) {
  Forced f;
  f.nb = nb;
  f.sinks = min(a.n_sink, nb);
  f.local0 = min(nb, max(f.sinks, p / KV_BLOCK + 1 - a.n_local));
  f.paged = 0;
  for (int i = threadIdx.x & 31; i < f.slots(); i += 32)
    f.paged += (unsigned)__ldg(a.tab.table + (size_t)s * a.tab.N + f.block(i)) < (unsigned)a.tab.n_pages;
  f.paged = __reduce_add_sync(0xffffffffu, f.paged);
  return f;
}

// By one warp: the lists of (token, head) `row` from the forced blocks' keys (by slot; 0: no page)
// and the n_mid best others.
__device__ __forceinline__ void write_lists(const SelectArgs& a, size_t row, const Forced& f, const uint32_t* forced_k,
                                            const uint32_t* mid_k, const int* mid_b, int n_mid, int eq) {
  const int lane = threadIdx.x & 31, slots = f.slots();
  const int e1 = (eq + SCORE_DOWN) / 2;   // in two factors: their product may be beyond FP32 where the score is not
  const float up1 = pow2f(e1), up2 = pow2f(eq + SCORE_DOWN - e1);
  int32_t* ids = a.ids + row * a.k;
  float* scores = a.scores ? a.scores + row * a.k : nullptr;
  auto put = [&](int p, int b, uint32_t key) {
    ids[p] = b;
    if (scores) scores[p] = score_of_key(key) * up1 * up2;
  };
  int at = 0;
  for (int i0 = 0; i0 < slots || i0 == 0; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < slots ? forced_k[i] : 0u;
    const uint32_t all = __ballot_sync(0xffffffffu, key != 0u);
    const uint32_t early = __ballot_sync(0xffffffffu, key != 0u && i < f.sinks);
    const int p = at + __popc(all & ((1u << lane) - 1u));
    if (key != 0u) put(i < f.sinks ? p : p + n_mid, f.block(i), key);
    if (i0 < f.sinks || i0 == 0) {   // the last such step knows where the others start
      if (f.sinks <= i0 + 32)
        for (int j = lane; j < n_mid; j += 32) put(at + __popc(early) + j, mid_b[j], mid_k[key_at(j)]);
    }
    at += __popc(all);
  }
  for (int i = at + n_mid + lane; i < a.k; i += 32) {
    ids[i] = -1;
    if (scores) scores[i] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// a token at a time: decode
// ---------------------------------------------------------------------------
// A cluster per (token, kv head).  Each CTA scores one stretch of the visible blocks, keeps the best
// of it (each warp of a part of it first, where it is long) and writes them into the first CTA's
// shared memory, which selects among them.
constexpr int SR_WARPS = 8, SR_RANKS = 8;

// Shared memory, in words; lists have kk places, k rounded up to whole groups of 16.
struct SelectRowsMem {
  int kk;
  __host__ __device__ explicit SelectRowsMem(int k) : kk((k + 15) / 16 * 16) {}
  __host__ __device__ int all_k() const { return 0; }                                     // every CTA's list
  __host__ __device__ int all_b() const { return all_k() + SR_RANKS * key_at(kk); }
  __host__ __device__ int loc_k() const { return all_b() + SR_RANKS * kk; }               // every warp's list
  __host__ __device__ int loc_b() const { return loc_k() + SR_WARPS * key_at(kk); }
  __host__ __device__ int fin_k() const { return loc_b() + SR_WARPS * kk; }               // the CTA's list
  __host__ __device__ int fin_b() const { return fin_k() + key_at(kk); }
  __host__ __device__ int forced() const { return fin_b() + kk; }
  __host__ __device__ int scratch(int w) const { return forced() + kk + w * (key_at(2 * kk) + 2 * kk); }
  __host__ __device__ int keys() const { return scratch(SR_WARPS); }
  __host__ __device__ int pages(int span) const { return keys() + key_at((span + 15) / 16 * 16); }
  __host__ __device__ size_t bytes(int span) const { return 4 * ((size_t)pages(span) + span); }
};

// Bytes 0, 1 (sel 0x4140) or 2, 3 (0x4342) of four whole numbers that were offset by 128 -> an FP16 pair.
__device__ __forceinline__ uint32_t s8x2_to_f16x2(uint32_t biased, uint32_t sel) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(prmt(biased, 0x64646464u, sel)), "r"(0x64806480u));
  return r;
}

// The `want` best of the entries first .. n - 1 (n <= 2 SR_WARPS 32) by the whole CTA, two entries a thread; else
// as warp_top, without its bound: a step is two barriers that count.  For one token this is what takes least
// time: 2,700 cycles for 16 of 256, against 5,000 for one warp's selection (much code that runs once); counting
// three values a step behind one barrier took longer (8.6 us a call against 8.5).
template <typename Put>
__device__ __forceinline__ int cta_top(const uint32_t* keys, int first, int n, int want, uint32_t (&s_red)[2][SR_WARPS],
                                       Put put) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t key[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (2 * tid + j >= first && 2 * tid + j < n) key[j] = keys[key_at(2 * tid + j)];
  __syncthreads();   // s_red is free
  {
    const uint32_t mx = __reduce_max_sync(0xffffffffu, max(key[0], key[1]));
    const uint32_t mn = __reduce_min_sync(0xffffffffu, min(key[0] - 1u, key[1] - 1u));   // a key of 0 counts as the largest
    if (lane == 0) s_red[0][warp] = mx, s_red[1][warp] = mn;
  }
  __syncthreads();
  uint32_t hi = 0, lo = 0xFFFFFFFFu;
#pragma unroll
  for (int w = 0; w < SR_WARPS; ++w) hi = max(hi, s_red[0][w]), lo = min(lo, s_red[1][w]);
  if (want <= 0 || hi == 0u) return 0;
  lo += 1u, hi += 1u;
  auto count = [&](uint32_t v) { return __syncthreads_count(key[0] >= v) + __syncthreads_count(key[1] >= v); };
  // count(>= lo) = got, count(>= hi) = above < want
  uint32_t thr = lo;
  int above = 0, got = count(lo);
  const int all = got;
  while (got > want && hi - lo > 1) {
    thr = lo + (hi - lo) / 2;
    got = count(thr);
    if (got > want) {
      lo = thr;
    } else if (got < want) {
      hi = thr;
      above = got;
      got = want + 1;
    }
  }
  const bool cut = got > want;   // hi - lo = 1: some of the entries equal to lo are left out
  if (cut) thr = lo;
  const uint32_t before = (1u << lane) - 1u;
  bool take[2] = {key[0] > thr || (!cut && key[0] == thr), key[1] > thr || (!cut && key[1] == thr)};
  if (cut) {
    const uint32_t e0 = __ballot_sync(0xffffffffu, key[0] == thr), e1 = __ballot_sync(0xffffffffu, key[1] == thr);
    __syncthreads();
    if (lane == 0) s_red[0][warp] = __popc(e0) + __popc(e1);
    __syncthreads();
    int rank = __popc(e0 & before) + __popc(e1 & before);
    for (int w = 0; w < warp; ++w) rank += s_red[0][w];
    take[0] |= key[0] == thr && rank < want - above;
    take[1] |= key[1] == thr && rank + (key[0] == thr) < want - above;
  }
  const uint32_t b0 = __ballot_sync(0xffffffffu, take[0]), b1 = __ballot_sync(0xffffffffu, take[1]);
  __syncthreads();
  if (lane == 0) s_red[1][warp] = __popc(b0) + __popc(b1);
  __syncthreads();
  int at = __popc(b0 & before) + __popc(b1 & before);
  for (int w = 0; w < warp; ++w) at += s_red[1][w];
  if (take[0]) put(at, 2 * tid, key[0]);
  if (take[1]) put(at + take[0], 2 * tid + 1, key[1]);
  return min(want, all);
}

template <int D>
__global__ void __launch_bounds__(SR_WARPS * 32, 2) kv_select_rows_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ __align__(16) __half u[2][2 * D];   // the query's vector; zeros
  __shared__ Forced f_s;
  __shared__ int eq_s;
  __shared__ uint32_t s_red[2][SR_WARPS];
  const SelectRowsMem mem(a.k);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kk = mem.kk;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  const int row = blockIdx.x / ranks, t = row / a.H, h = row - t * a.H;
  // the lists' unused places are entries that cannot be taken; the first CTA's are written by the others
  for (int i = tid; i < SR_RANKS * key_at(kk); i += SR_WARPS * 32) sm[mem.all_k() + i] = 0u;
  cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const int p = __ldg(a.pos + t), s = __ldg(a.seq + t);
  const bool ok = p >= 0 && (unsigned)s < (unsigned)a.tab.B;
  if (p >= 0 && (!ok || p / KV_BLOCK >= a.tab.N) && tid == 0) set_err(a.err, BRE_DEVERR_PAGE);
  const int nb = ok ? min(p / KV_BLOCK + 1, a.tab.N) : 0;
  const int span = (nb + ranks - 1) / ranks, b0 = min(rank * span, nb), n = min(span, nb - b0);
  uint32_t* keys = sm + mem.keys();
  int* page = reinterpret_cast<int*>(sm + mem.pages(span));

  // the query's vector by the last warp, what must be taken by the one before, pages by the others
  if (warp == SR_WARPS - 1) {
    constexpr int W = D / 64;
    int pl[2 * W], mi[2 * W];
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q + t * a.q_stride + (size_t)h * a.G * D) + lane * W;
    const int e = query_vector<W>(qr, D / 2, a.G, pl, mi);
    if (lane == 0) eq_s = e;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
      u[0][2 * W * lane + i] = __int2half_rn(pl[i]);
      u[0][D + 2 * W * lane + i] = __int2half_rn(-mi[i]);
    }
  } else if (warp == SR_WARPS - 2) {
    for (int i = lane; i < D; i += 32) reinterpret_cast<uint32_t*>(u[1])[i] = 0u;
    const Forced f = forced_blocks(a, s, p, nb);
    if (lane == 0) f_s = f;
  } else {
    for (int i = tid; i < n; i += (SR_WARPS - 2) * 32) page[i] = kv_page(a.tab, s, b0 + i, a.err);
  }
  __syncthreads();
  const Forced f = f_s;

  // scores, as in the prefill tiles but with the one vector in the first row of the product (the integer dot
  // products dp2a and dp4a are a small fraction of the tensor cores' rate here): eight blocks a product, 32 of a
  // warp in flight
  constexpr int KS = 2 * D / 16, NT = 4;   // k steps, of which four cover 64 channels; products at a time
  const int g = lane >> 2, t4 = lane & 3;
  const __half* ul = u[g ? 1 : 0] + 16 * t4;
  // a warp's part: whole groups of 16, so that parts are lists of their own
  const int part = (n + 16 * SR_WARPS - 1) / (16 * SR_WARPS) * 16, w0 = min(warp * part, n), wn = min(part, n - w0);
#pragma unroll 1
  for (int i0 = 0; i0 < wn; i0 += 8 * NT) {
    uint4 bd[NT][KS / 4];
    int e[NT][2];   // of columns 2 t4, 2 t4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int i = i0 + 8 * nt + g, pg = i < wn ? page[w0 + i] : -1;
      const int8_t* bp = a.bounds + ((size_t)max(pg, 0) * a.H + h) * 2 * D + 16 * t4;
#pragma unroll
      for (int cg = 0; cg < KS / 4; ++cg)
        bd[nt][cg] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(bp + 64 * cg)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ic = i0 + 8 * nt + 2 * t4 + c, pc = g == 0 && ic < wn ? page[w0 + ic] : -1;
        e[nt][c] = pc >= 0 ? (int)__ldg(a.bexp + (size_t)pc * a.H + h) : -128;
      }
    }
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][j] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint2 uf = *reinterpret_cast<const uint2*>(ul + 64 * (ks / 4) + 4 * (ks % 4));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4& q = bd[nt][ks / 4];
        const uint32_t w = (ks % 4 == 0 ? q.x : ks % 4 == 1 ? q.y : ks % 4 == 2 ? q.z : q.w) ^ 0x80808080u;
        mma_f16_16816(acc[nt], uf.x, 0u, uf.y, 0u, s8x2_to_f16x2(w, 0x4140u), s8x2_to_f16x2(w, 0x4342u));
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int ic = i0 + 8 * nt + 2 * t4;
      if (g == 0)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (ic + c < wn) keys[key_at(w0 + ic + c)] = e[nt][c] == -128 ? 0u : key_of_score(acc[nt][c] * pow2f(e[nt][c] - SCORE_DOWN));
    }
  }
  __syncthreads();

  // the stretch's best of the blocks between the forced ones
  const int want = a.k - f.paged, m0 = f.sinks - b0, m1 = min(n, f.local0 - b0);
  uint32_t* fin_k = sm + mem.fin_k();
  int* fin_b = reinterpret_cast<int*>(sm + mem.fin_b());
  uint32_t* lk = sm + mem.scratch(warp);
  int* lb = reinterpret_cast<int*>(lk + key_at(2 * kk));
  auto push = [&](int place, int b, uint32_t key) {   // into the first CTA's lists
    st_cluster_u32(sm + mem.all_k() + key_at(rank * kk + place), 0, key);
    st_cluster_u32(sm + mem.all_b() + rank * kk + place, 0, (uint32_t)b);
  };
  int got = 0;
  uint32_t* loc_k = sm + mem.loc_k();
  int* loc_b = reinterpret_cast<int*>(sm + mem.loc_b());
  if (n > SEL_CHUNK) {
    got = warp_top_list(keys + key_at(w0), m0 - w0, min(wn, m1 - w0), [&](int i) { return b0 + w0 + i; }, want,
                        loc_k + warp * key_at(kk), loc_b + warp * kk, lk, lb);
    for (int i = got + lane; i < kk; i += 32) loc_k[key_at(warp * kk + i)] = 0u;
    __syncthreads();
  }
  cluster_wait();   // the first CTA runs: its shared memory may be written
  if (n <= SEL_CHUNK) {
    got = cta_top(keys, m0, m1, want, s_red, [&](int p, int i, uint32_t key) { push(p, b0 + i, key); });
  } else if (SR_WARPS * kk <= SEL_CHUNK) {
    got = cta_top(loc_k, 0, SR_WARPS * kk, want, s_red, [&](int p, int i, uint32_t key) { push(p, loc_b[i], key); });
  } else if (warp == 0) {
    got = warp_top_list(loc_k, 0, SR_WARPS * kk, [&](int i) { return loc_b[i]; }, want, fin_k, fin_b, lk, lb);
    for (int i = lane; i < got; i += 32) push(i, fin_b[i], fin_k[key_at(i)]);
  }
  if (warp == 1)
    for (int i = lane; i < f.slots(); i += 32) {
      const int b = f.block(i) - b0;
      if (b >= 0 && b < n) st_cluster_u32(sm + mem.forced() + i, 0, keys[key_at(b)]);
    }
  cluster_arrive();
  if (rank != 0) return;
  cluster_wait();
  const uint32_t* all_k = sm + mem.all_k();
  const int* all_b = reinterpret_cast<const int*>(sm + mem.all_b());
  if (ranks == 1) {   // the one list is the result
    if (warp == 0) write_lists(a, row, f, sm + mem.forced(), all_k, all_b, __shfl_sync(0xffffffffu, got, 0), eq_s);
    return;
  }
  if (ranks * kk <= SEL_CHUNK) {
    got = cta_top(all_k, 0, ranks * kk, want, s_red,
                  [&](int p, int i, uint32_t key) { fin_k[key_at(p)] = key, fin_b[p] = all_b[i]; });
    __syncthreads();
  } else if (warp == 0) {
    got = warp_top_list(all_k, 0, ranks * kk, [&](int i) { return all_b[i]; }, want, fin_k, fin_b, lk, lb);
  }
  if (warp == 0) write_lists(a, row, f, sm + mem.forced(), fin_k, fin_b, got, eq_s);
}

// ---------------------------------------------------------------------------
// 32 tokens at a time: prefill
// ---------------------------------------------------------------------------
// A CTA per (32 tokens, kv head).  The tokens' vectors lie in shared memory as FP16 fragments, the
// bounds' bytes become FP16 in registers (1024 + 128 + b in the mantissa, minus 1152: exact), and
// mma.m16n8k16 multiplies them, 512 blocks at a time; each warp then selects for two of the
// tokens, from the scores in shared memory and the best of the blocks before.  Tokens of one
// sequence share the work; a tile that spans sequences goes through each of them in turn.
constexpr int ST_WARPS = 16, ST_ROWS = 32, ST_NT = 2;   // ST_NT: column tiles (of 8 blocks) of a warp at a time
constexpr int ST_LD = key_at(SEL_CHUNK) + 8;   // padded: the fragments' rows fall into different banks

// Shared memory: the fragments, the keys of a piece, its pages and units, the rows' lists (kk places, k
// rounded up to whole groups of 16) and forced blocks' keys, the warps' scratch.
__host__ __device__ constexpr size_t select_tiles_smem(int D, int kk) {
  return (size_t)ST_ROWS * 2 * D * 2 + (size_t)ST_ROWS * ST_LD * 4 + SEL_CHUNK * 8 +
         (size_t)ST_ROWS * (key_at(kk) + 2 * kk) * 4 + (size_t)ST_WARPS * (key_at(2 * kk) + 2 * kk) * 4;
}

template <int D>
__global__ void __launch_bounds__(ST_WARPS * 32, 2) kv_select_tiles_kernel(const SelectArgs a) {
  constexpr int KS = 2 * D / 16;   // k steps; a group of four covers 64 channels
  extern __shared__ __align__(16) unsigned char sm_raw[];
  uint4* af = reinterpret_cast<uint4*>(sm_raw);                        // [2 row tiles][KS][32 lanes]
  uint32_t* keys = reinterpret_cast<uint32_t*>(sm_raw + ST_ROWS * 2 * D * 2);   // [ST_ROWS][ST_LD]
  int* page = reinterpret_cast<int*>(keys + ST_ROWS * ST_LD);          // [SEL_CHUNK]
  float* unit = reinterpret_cast<float*>(page + SEL_CHUNK);            // [SEL_CHUNK] 2^(bound_exp - SCORE_DOWN), 0: no page
  const int kk = (a.k + 15) / 16 * 16;
  uint32_t* best_k = reinterpret_cast<uint32_t*>(unit + SEL_CHUNK);    // [ST_ROWS][key_at(kk)]
  int* best_b = reinterpret_cast<int*>(best_k + ST_ROWS * key_at(kk)); // [ST_ROWS][kk]
  uint32_t* forced_k = reinterpret_cast<uint32_t*>(best_b + ST_ROWS * kk);   // [ST_ROWS][kk]
  uint32_t* scratch = forced_k + ST_ROWS * kk;
  __shared__ int row_seq[ST_ROWS], row_pos[ST_ROWS], row_eq[ST_ROWS], row_have[ST_ROWS];
  __shared__ Forced row_f[ST_ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int t0 = blockIdx.x * ST_ROWS, h = blockIdx.y, rows = min(ST_ROWS, a.T - t0);
  pdl_wait();
  pdl_launch_dependents();
  if (tid < ST_ROWS) {
    const int p = tid < rows ? __ldg(a.pos + t0 + tid) : -1, s = tid < rows ? __ldg(a.seq + t0 + tid) : 0;
    const bool ok = p >= 0 && (unsigned)s < (unsigned)a.tab.B;
    if (p >= 0 && (!ok || p / KV_BLOCK >= a.tab.N)) set_err(a.err, BRE_DEVERR_PAGE);
    row_pos[tid] = ok ? p : -1;
    row_seq[tid] = s;
  }
  // the vectors; a lane takes D / 32 channels of every head
  constexpr int PL = D / 32;
  for (int r = warp; r < ST_ROWS; r += ST_WARPS) {
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q + (long long)(t0 + min(r, rows - 1)) * a.q_stride +
                                                           (size_t)h * a.G * D) + lane * (PL / 2);
    int pl[PL], mi[PL];
    const int eq = query_vector<PL / 2>(qr, D / 2, a.G, pl, mi);
    if (lane == 0) row_eq[r] = eq;
#pragma unroll
    for (int j = 0; j < PL; j += 2)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // channel c of the vector: k step 4 (c / 64) + c % 16 / 4, lane 4 (row % 8) + c % 64 / 16,
        // register row % 16 / 8 + 2 (c % 4 / 2)
        const int c = half * D + lane * PL + j;
        const __half2 v = half ? __floats2half2_rn((float)-mi[j], (float)-mi[j + 1])
                               : __floats2half2_rn((float)pl[j], (float)pl[j + 1]);
        const int at = ((r / 16) * KS + 4 * (c / 64) + c % 16 / 4) * 32 + 4 * (r % 8) + c % 64 / 16;
        reinterpret_cast<__half2*>(af + at)[r % 16 / 8 + 2 * (c % 4 / 2)] = v;
      }
  }
  __syncthreads();

  for (int r0 = 0; r0 < rows;) {   // a stretch of rows of one sequence
    const int s = row_seq[r0];
    int r1 = r0, nb_max = 0;
    while (r1 < rows && row_seq[r1] == s) {
      nb_max = max(nb_max, row_pos[r1] >= 0 ? row_pos[r1] / KV_BLOCK + 1 : 0);
      ++r1;
    }
    nb_max = min(nb_max, a.tab.N);
    for (int r = r0 + warp; r < r1; r += ST_WARPS) {
      const int p = row_pos[r];
      const Forced f = forced_blocks(a, s, p, p >= 0 ? min(p / KV_BLOCK + 1, a.tab.N) : 0);
      if (lane == 0) row_f[r] = f, row_have[r] = 0;
    }
    for (int base = 0; base < nb_max; base += SEL_CHUNK) {
      const int nc = min(SEL_CHUNK, nb_max - base);
      __syncthreads();   // the scores and pages of the piece before are done with
      for (int i = tid; i < SEL_CHUNK; i += ST_WARPS * 32) {
        const int pg = i < nc ? kv_page(a.tab, s, base + i, a.err) : -1;
        page[i] = pg;
        unit[i] = pg >= 0 ? pow2f(__ldg(a.bexp + (size_t)pg * a.H + h) - SCORE_DOWN) : 0.0f;
      }
      __syncthreads();
      for (int c0 = warp * 8 * ST_NT; c0 < nc; c0 += ST_WARPS * 8 * ST_NT) {
        float acc[ST_NT][2][4];
#pragma unroll
        for (int nt = 0; nt < ST_NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[nt][mt][j] = 0.0f;
        const int8_t* bp[ST_NT];
#pragma unroll
        for (int nt = 0; nt < ST_NT; ++nt) {
          const int pg = page[c0 + 8 * nt + g];
          bp[nt] = pg >= 0 ? a.bounds + ((size_t)pg * a.H + h) * 2 * D + 16 * t4 : nullptr;
        }
#pragma unroll
        for (int cg = 0; cg < KS / 4; ++cg) {
          uint4 b[ST_NT];
#pragma unroll
          for (int nt = 0; nt < ST_NT; ++nt)
            b[nt] = bp[nt] ? __ldg(reinterpret_cast<const uint4*>(bp[nt] + cg * 64)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 a0 = af[(cg * 4 + i) * 32 + lane], a1 = af[(KS + cg * 4 + i) * 32 + lane];
#pragma unroll
            for (int nt = 0; nt < ST_NT; ++nt) {
              const uint32_t w = (i == 0 ? b[nt].x : i == 1 ? b[nt].y : i == 2 ? b[nt].z : b[nt].w) ^ 0x80808080u;
              const uint32_t b0 = s8x2_to_f16x2(w, 0x4140u), b1 = s8x2_to_f16x2(w, 0x4342u);
              mma_f16_16816(acc[nt][0], a0.x, a0.y, a0.z, a0.w, b0, b1);
              mma_f16_16816(acc[nt][1], a1.x, a1.y, a1.z, a1.w, b0, b1);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < ST_NT; ++nt) {
          const int col = c0 + 8 * nt + 2 * t4;
          const float u0 = unit[col], u1 = unit[col + 1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              *reinterpret_cast<uint2*>(keys + (16 * mt + 8 * r + g) * ST_LD + key_at(col)) =
                  make_uint2(u0 == 0.0f ? 0u : key_of_score(acc[nt][mt][2 * r] * u0),
                             u1 == 0.0f ? 0u : key_of_score(acc[nt][mt][2 * r + 1] * u1));
        }
      }
      __syncthreads();
      for (int r = r0 + warp; r < r1; r += ST_WARPS) {
        const Forced f = row_f[r];
        const int m = min(f.nb - base, SEL_CHUNK);
        if (m <= 0) continue;
        const uint32_t* kr = keys + r * ST_LD;
        for (int i = lane; i < f.slots(); i += 32) {
          const int b = f.block(i) - base;
          if (b >= 0 && b < m) forced_k[r * kk + i] = kr[key_at(b)];
        }
        uint32_t* lk = scratch + warp * (key_at(2 * kk) + 2 * kk);
        const int have = warp_top_piece(row_have[r], kr, f.sinks - base, min(m, f.local0 - base),
                                        [&](int i) { return base + i; }, a.k - f.paged, best_k + r * key_at(kk),
                                        best_b + r * kk, lk, reinterpret_cast<int*>(lk + key_at(2 * kk)));
        if (lane == 0) row_have[r] = have;
      }
    }
    __syncwarp();
    for (int r = r0 + warp; r < r1; r += ST_WARPS)
      write_lists(a, (size_t)(t0 + r) * a.H + h, row_f[r], forced_k + r * kk, best_k + r * key_at(kk), best_b + r * kk,
                  row_have[r], row_eq[r]);
    r0 = r1;
  }
}

}  // namespace

// Lets a kernel have so much dynamic shared memory; the call is made once a device.
static cudaError_t allow_smem(const void* kern, int which, int bytes) {
  static std::atomic<uint64_t> done[4];
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (done[which].load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[which].fetch_or(bit, std::memory_order_release);
  return e;
}

// Shared memory of the one-token kernel for stretches of `span` blocks.
static size_t select_rows_smem(int span, int k) { return SelectRowsMem(k).bytes(span); }

cudaError_t launch_kv_select(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* q, long long q_stride, int Hq,
                             int k, int n_sink, int n_local, int32_t* ids, float* scores, int32_t* err, cudaStream_t s) {
  const int H = c->n_kv_heads, D = c->head_dim;
  const SelectArgs a{c->bounds, c->bound_exp, H,   Hq / H, KvTable{tk.table, tk.B, tk.N, c->n_pages},
                     q, q_stride, tk.seq, tk.pos, tk.T, k, n_sink, n_local, ids, scores, err};
  // Tiles of 32 tokens: the lists must fit (up to about 170 blocks a token), the tokens mostly be of one sequence
  // (16 on average for each of the table's sequences, whether the call has tokens of all of them or not), and there must be enough of them.  256 blocks, four kv heads, us by token / by tile:
  // 128 tokens of one sequence 17 / 19, 256 31 / 19; 128 tokens of eight 17 / 22, 256 30 / 19; 64 of eight 9 / 34.
  const size_t most = device_max_smem_optin() - 2048;   // less the kernels' static shared memory
  const size_t smem_t = select_tiles_smem(D, (k + 15) / 16 * 16);
  if (tk.T >= 16LL * tk.B && (long long)tk.T * H >= 640 && smem_t <= most) {
    auto kern = D == 128 ? kv_select_tiles_kernel<128> : kv_select_tiles_kernel<64>;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), D == 128, (int)most);
    if (e != cudaSuccess) return e;
    return launch_k(kern, dim3((unsigned)((tk.T + ST_ROWS - 1) / ST_ROWS), (unsigned)H), dim3(ST_WARPS * 32), smem_t, s, a);
  }
  // CTAs of a (token, head): while the GPU has room and a CTA keeps 64 blocks; more where the
  // stretch would not fit its shared memory
  const long long rows = (long long)tk.T * H;
  const size_t room = 200 * 1024;
  int ranks = 1;
  while (ranks < 8 && ((rows * ranks * 2 <= 2LL * device_sm_count() && tk.N / (2 * ranks) >= 64) ||
                       select_rows_smem((tk.N + ranks - 1) / ranks, k) > room))
    ranks *= 2;
  const size_t smem = select_rows_smem((tk.N + ranks - 1) / ranks, k);
  auto kern = D == 128 ? kv_select_rows_kernel<128> : kv_select_rows_kernel<64>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), 2 + (D == 128), (int)most);
  if (e != cudaSuccess) return e;
  return launch_kc(kern, dim3((unsigned)(rows * ranks)), dim3(SR_WARPS * 32), ranks, smem, s, a);
}

}  // namespace bre

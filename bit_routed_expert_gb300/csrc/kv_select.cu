// Block selection for sparse attention: every visible block's score against a query's heads, and
// the best blocks in ascending order.
//
// The score is linear in the block's bounds: with the query's whole-number codes c,
//   sum_g sum_ch max(c hi, c lo) = P . hi - M . lo,   P = sum_g max(c, 0), M = sum_g max(-c, 0),
// so a kv head's G query heads fold into one vector of 2 D whole numbers (at most 16 * 127 = 2032:
// exact in FP16) before they meet the blocks, and the sums stay below 2^24: exact in FP32 and in
// 32-bit integers, whatever the order.
#include <cuda_fp16.h>

#include "kv_common.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// the best of a list, by one warp
// ---------------------------------------------------------------------------
// Order-preserving key of a score; 0 for a block that cannot be taken (score -inf), all ones for
// one that must be.
__device__ __forceinline__ uint32_t select_key(float sc, bool must) {
  const uint32_t u = __float_as_uint(sc);
  const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return sc == -INFINITY ? 0u : must ? 0xFFFFFFFFu : key;
}

// Of n <= 32 R entries in ascending order of block, the `want` with the largest keys (the first ones
// among equals) are passed to put(place, get(index)) in ascending order; returns how many there
// are.  place <= index, and 32 entries at a time are got by all lanes before any is put: put may
// write where get reads.
// Entries live in registers, entry i in lane i % 32.  The threshold comes by bisection of the keys,
// which ends as soon as a value splits off exactly `want` entries.  It starts between the largest
// key and a lower bound that costs one register a lane: the `want`-th largest of the 32 lanes' own
// largest keys (as many lanes, so as many entries, reach it); of 512 random keys about 24 lie
// above the bound for want = 16, so three or four steps over all registers are left of twelve.
struct Entry {
  float sc;
  int id;
};
template <int R, typename Key, typename Get, typename Put>
__device__ __forceinline__ int warp_select(int n, int want, Key key_of, Get get, Put put) {
  const int lane = threadIdx.x & 31;
  uint32_t key[R], lo = 0xFFFFFFFFu, top = 0;   // of the entries that neither must nor cannot be taken
  int valid = 0, must = 0;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int i = 32 * j + lane;
    key[j] = i < n ? key_of(i) : 0u;
    valid += key[j] != 0u;
    must += key[j] == 0xFFFFFFFFu;
    if (key[j] != 0xFFFFFFFFu) top = max(top, key[j]);
    lo = min(lo, key[j] - 1u);   // a key of 0 becomes the largest
  }
  valid = __reduce_add_sync(0xffffffffu, valid);
  must = __reduce_add_sync(0xffffffffu, must);
  uint32_t thr = 1;        // entries with key >= thr are taken, of those equal to thr only the first `ties`
  int ties = 0x7fffffff;
  if (valid > want) {
    // count(>= lo) >= want > count(>= hi) = above, or above == want
    lo = __reduce_min_sync(0xffffffffu, lo) + 1u;
    uint32_t hi = __reduce_max_sync(0xffffffffu, top) + 1u;
    int above = must;
    if (want - must <= 32 && want > must) {
      uint32_t h = hi;
      while (h - lo > 1) {
        const uint32_t mid = lo + (h - lo) / 2;
        const int c = __popc(__ballot_sync(0xffffffffu, top >= mid));
        if (c >= want - must) {
          lo = mid;
          if (c == want - must) break;
        } else {
          h = mid;
        }
      }
    }
    thr = hi;
    for (bool first = true; above < want; first = false) {
      if (hi - lo == 1) {
        thr = lo;
        ties = want - above;
        break;
      }
      const uint32_t mid = first ? lo : lo + (hi - lo) / 2;   // the bound may be the value itself
      int c = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) c += key[j] >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if (c > want) {
        lo = mid;
      } else {
        hi = thr = mid;
        above = c;
      }
    }
  }
  int at = 0;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (32 * j < n) {
      const uint32_t eq = __ballot_sync(0xffffffffu, key[j] == thr);
      const uint32_t before = (1u << lane) - 1u;
      const bool take = key[j] > thr || (key[j] == thr && __popc(eq & before) < ties);
      ties -= min(ties, __popc(eq));
      const uint32_t all = __ballot_sync(0xffffffffu, take);
      const Entry e = take ? get(32 * j + lane) : Entry{0.0f, 0};
      __syncwarp();
      if (take) put(at + __popc(all & before), e);
      at += __popc(all);
    }
  }
  return at;
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

// ---------------------------------------------------------------------------
// a token at a time: decode
// ---------------------------------------------------------------------------
// A cluster per (token, kv head); each CTA scores one stretch of the visible blocks and keeps its
// best k, the first CTA takes the best of those.  Within a CTA each warp selects from its own
// stretch of the scores, the first warp then from the warps' lists; a list that does not fit the
// registers goes through in pieces, the best so far being the head of the next piece.
constexpr int SR_WARPS = 8;
constexpr int SEL_CHUNK = 512, SEL_KMAX = 256;   // entries a piece adds; most blocks taken

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

// One warp: the best k of the `have` entries held in (osc, oid) and m <= SEL_CHUNK more, sc[i] and
// id_of(i), which follow them in order -> (osc, oid); returns how many are held then.
template <typename Id>
__device__ __forceinline__ int select_piece(int have, const float* sc, int m, int k, int n_sink, int first_local, Id id_of,
                                            float* osc, int* oid) {
  auto get = [&](int i) { return i < have ? Entry{osc[i], oid[i]} : Entry{sc[i - have], id_of(i - have)}; };
  auto key = [&](int i) {
    const Entry e = get(i);
    return select_key(e.sc, e.id < n_sink || e.id >= first_local);
  };
  auto put = [&](int p, const Entry& e) { osc[p] = e.sc, oid[p] = e.id; };
  const int total = have + m;
  int got;
  if (total <= 128)
    got = warp_select<4>(total, k, key, get, put);
  else if (total <= 256)
    got = warp_select<8>(total, k, key, get, put);
  else if (total <= 512)
    got = warp_select<16>(total, k, key, get, put);
  else
    got = warp_select<(SEL_CHUNK + SEL_KMAX) / 32>(total, k, key, get, put);
  __syncwarp();
  return got;
}

// The best k of n entries, any number of them.
template <typename Id>
__device__ __forceinline__ int select_list(const float* sc, int n, int k, int n_sink, int first_local, Id id_of,
                                           float* osc, int* oid) {
  int have = 0;
  for (int base = 0; base < n; base += SEL_CHUNK)
    have = select_piece(have, sc + base, min(SEL_CHUNK, n - base), k, n_sink, first_local,
                        [&](int i) { return id_of(base + i); }, osc, oid);
  return have;
}

// Sixteen whole numbers of the query's vector against sixteen bytes of bounds.
__device__ __forceinline__ int dot16(const int (&u)[8], const uint4& b) {
  int acc = 0;
  acc = __dp2a_lo(u[0], (int)b.x, acc);
  acc = __dp2a_hi(u[1], (int)b.x, acc);
  acc = __dp2a_lo(u[2], (int)b.y, acc);
  acc = __dp2a_hi(u[3], (int)b.y, acc);
  acc = __dp2a_lo(u[4], (int)b.z, acc);
  acc = __dp2a_hi(u[5], (int)b.z, acc);
  acc = __dp2a_lo(u[6], (int)b.w, acc);
  return __dp2a_hi(u[7], (int)b.w, acc);
}

template <int D>
__global__ void __launch_bounds__(SR_WARPS * 32, 2) kv_select_rows_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) unsigned char sm_raw[];
  __shared__ __align__(16) short u[2 * D];
  __shared__ float best_sc[SEL_KMAX];
  __shared__ int best_id[SEL_KMAX], n_best, eq_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  const int row = blockIdx.x / ranks, t = row / a.H, h = row - t * a.H;
  if (ranks > 1) cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const int p = __ldg(a.pos + t), s = __ldg(a.seq + t);
  const bool ok = p >= 0 && (unsigned)s < (unsigned)a.tab.B;
  if (p >= 0 && (!ok || p / KV_BLOCK >= a.tab.N) && tid == 0) set_err(a.err, BRE_DEVERR_PAGE);
  const int nb = ok ? min(p / KV_BLOCK + 1, a.tab.N) : 0;
  const int span = (nb + ranks - 1) / ranks, b0 = min(rank * span, nb), n = min(span, nb - b0);
  // shared: the lists (at the same place in every CTA), then pages and scores of this CTA's blocks
  float* list_sc = reinterpret_cast<float*>(sm_raw);
  int* list_id = reinterpret_cast<int*>(list_sc + SR_WARPS * a.k);
  float* all_sc = reinterpret_cast<float*>(list_id + SR_WARPS * a.k);   // every CTA's list, in the first CTA
  int* all_id = reinterpret_cast<int*>(all_sc + 8 * a.k);
  int* page = all_id + 8 * a.k;
  float* sc = reinterpret_cast<float*>(page + span);
  if (warp < SR_WARPS - 1)
    for (int i = tid; i < n; i += (SR_WARPS - 1) * 32) page[i] = kv_page(a.tab, s, b0 + i, a.err);

  // the query's vector, by the last warp (the others look up pages)
  if (warp == SR_WARPS - 1) {
    constexpr int W = D / 64;
    int pl[2 * W], mi[2 * W];
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q + t * a.q_stride + (size_t)h * a.G * D) + lane * W;
    const int e = query_vector<W>(qr, D / 2, a.G, pl, mi);
    if (lane == 0) eq_s = e;
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) u[2 * W * lane + i] = (short)pl[i], u[D + 2 * W * lane + i] = (short)-mi[i];
  }
  __syncthreads();
  const int eq = eq_s;

  // scores: 2 D / 16 lanes a block, eight loads in flight
  constexpr int LB = 2 * D / 16, PW = 32 / LB;   // lanes a block, blocks a load
  int uu[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) uu[j] = reinterpret_cast<const int*>(u)[(lane % LB) * 8 + j];
  const int seg = (n + SR_WARPS - 1) / SR_WARPS, w0 = min(warp * seg, n), wn = min(seg, n - w0);
  for (int i0 = 0; i0 < wn; i0 += 8 * PW) {
    uint4 bd[8];
    int e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * PW + lane / LB;
      const int pg = i < wn ? page[w0 + i] : -1;
      const size_t ph = (size_t)max(pg, 0) * a.H + h;
      bd[j] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.bounds + ph * 2 * D) + lane % LB) : make_uint4(0, 0, 0, 0);
      e[j] = pg >= 0 ? (int)__ldg(a.bexp + ph) : -128;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      int d = dot16(uu, bd[j]);
#pragma unroll
      for (int o = 1; o < LB; o *= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
      const int i = i0 + j * PW + lane / LB;
      if (i < wn && lane % LB == 0) sc[w0 + i] = e[j] == -128 ? -INFINITY : (float)d * pow2f(e[j]);
    }
  }
  __syncthreads();
  const int first_local = p / KV_BLOCK - a.n_local + 1;
  // the lists' unused places are entries that cannot be taken
  auto pad = [&](int got, float* lsc) {
    for (int i = got + lane; i < a.k; i += 32) lsc[i] = -INFINITY;
  };
  if (n > SEL_CHUNK) {
    float* lsc = list_sc + warp * a.k;
    pad(select_list(sc + w0, wn, a.k, a.n_sink, first_local, [&](int i) { return b0 + w0 + i; }, lsc,
                    list_id + warp * a.k), lsc);
    __syncthreads();
  }
  if (warp == 0) {
    const int got = n > SEL_CHUNK
                        ? select_list(list_sc, SR_WARPS * a.k, a.k, a.n_sink, first_local,
                                      [&](int i) { return list_id[i]; }, best_sc, best_id)
                        : select_list(sc, n, a.k, a.n_sink, first_local, [&](int i) { return b0 + i; }, best_sc, best_id);
    if (lane == 0) n_best = got;
  }
  if (ranks > 1) {
    cluster_wait();   // the first CTA runs: its shared memory may be written
    __syncthreads();
    for (int i = tid; i < a.k; i += SR_WARPS * 32) {
      st_cluster_f32(&all_sc[rank * a.k + i], 0, i < n_best ? best_sc[i] : -INFINITY);
      st_cluster_s32(&all_id[rank * a.k + i], 0, i < n_best ? best_id[i] : 0);
    }
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) {
      const int got = select_list(all_sc, ranks * a.k, a.k, a.n_sink, first_local, [&](int i) { return all_id[i]; },
                                  best_sc, best_id);
      if (lane == 0) n_best = got;
    }
  }
  __syncthreads();
  if (rank == 0)
    for (int i = tid; i < a.k; i += SR_WARPS * 32) {
      a.ids[(size_t)row * a.k + i] = i < n_best ? best_id[i] : -1;
      if (a.scores) a.scores[(size_t)row * a.k + i] = i < n_best ? best_sc[i] * pow2f(eq) : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// 32 tokens at a time: prefill
// ---------------------------------------------------------------------------
// A CTA per (32 tokens, kv head).  The tokens' vectors lie in shared memory as FP16 fragments, the
// bounds' bytes become FP16 in registers (1024 + 128 + b in the mantissa, minus 1152: exact), and
// mma.m16n8k16 multiplies them, 512 blocks at a time; each warp then selects for four of the
// tokens, from the scores in shared memory and the best of the blocks before.  Tokens of one
// sequence share the work; a tile that spans sequences goes through each of them in turn.
constexpr int ST_WARPS = 8, ST_ROWS = 32, ST_LD = SEL_CHUNK + 8;   // padded: the fragments' rows fall into different banks

__device__ __forceinline__ uint32_t s8x2_to_f16x2(uint32_t biased, uint32_t sel) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(prmt(biased, 0x64646464u, sel)), "r"(0x64806480u));
  return r;
}

__host__ __device__ constexpr size_t select_tiles_smem(int D, int k) {
  return (size_t)ST_ROWS * 2 * D * 2 + (size_t)ST_ROWS * ST_LD * 4 + SEL_CHUNK * 8 + (size_t)ST_ROWS * k * 8;
}

template <int D>
__global__ void __launch_bounds__(ST_WARPS * 32, 2) kv_select_tiles_kernel(const SelectArgs a) {
  constexpr int KS = 2 * D / 16;   // k steps; a group of four covers 64 channels
  extern __shared__ __align__(16) unsigned char sm_raw[];
  uint4* af = reinterpret_cast<uint4*>(sm_raw);                        // [2 row tiles][KS][32 lanes]
  float* sc = reinterpret_cast<float*>(sm_raw + ST_ROWS * 2 * D * 2);   // [ST_ROWS][ST_LD]
  int* page = reinterpret_cast<int*>(sc + ST_ROWS * ST_LD);            // [SEL_CHUNK]
  float* unit = reinterpret_cast<float*>(page + SEL_CHUNK);            // [SEL_CHUNK] 2^bound_exp, 0: no page
  float* best_sc = unit + SEL_CHUNK;                                   // [ST_ROWS][k]
  int* best_id = reinterpret_cast<int*>(best_sc + ST_ROWS * a.k);
  __shared__ int row_seq[ST_ROWS], row_pos[ST_ROWS], row_eq[ST_ROWS];
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
    int have[ST_ROWS / ST_WARPS] = {};
    for (int base = 0; base < nb_max; base += SEL_CHUNK) {
      const int nc = min(SEL_CHUNK, nb_max - base);
      __syncthreads();   // the scores and pages of the piece before are done with
      for (int i = tid; i < SEL_CHUNK; i += ST_WARPS * 32) {
        const int pg = i < nc ? kv_page(a.tab, s, base + i, a.err) : -1;
        page[i] = pg;
        unit[i] = pg >= 0 ? pow2f(__ldg(a.bexp + (size_t)pg * a.H + h)) : 0.0f;
      }
      __syncthreads();
      // 32 blocks (four column tiles) of a warp at a time
      for (int c0 = warp * 32; c0 < nc; c0 += ST_WARPS * 32) {
        float acc[4][2][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[nt][mt][j] = 0.0f;
        const int8_t* bp[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int pg = page[c0 + 8 * nt + g];
          bp[nt] = pg >= 0 ? a.bounds + ((size_t)pg * a.H + h) * 2 * D + 16 * t4 : nullptr;
        }
#pragma unroll
        for (int cg = 0; cg < KS / 4; ++cg) {
          uint4 b[4];
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
            b[nt] = bp[nt] ? __ldg(reinterpret_cast<const uint4*>(bp[nt] + cg * 64)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 a0 = af[(cg * 4 + i) * 32 + lane], a1 = af[(KS + cg * 4 + i) * 32 + lane];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
              const uint32_t w = (i == 0 ? b[nt].x : i == 1 ? b[nt].y : i == 2 ? b[nt].z : b[nt].w) ^ 0x80808080u;
              const uint32_t b0 = s8x2_to_f16x2(w, 0x4140u), b1 = s8x2_to_f16x2(w, 0x4342u);
              mma_f16_16816(acc[nt][0], a0.x, a0.y, a0.z, a0.w, b0, b1);
              mma_f16_16816(acc[nt][1], a1.x, a1.y, a1.z, a1.w, b0, b1);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int col = c0 + 8 * nt + 2 * t4;
          const float u0 = unit[col], u1 = unit[col + 1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              *reinterpret_cast<float2*>(sc + (16 * mt + 8 * r + g) * ST_LD + col) =
                  make_float2(u0 == 0.0f ? -INFINITY : acc[nt][mt][2 * r] * u0,
                              u1 == 0.0f ? -INFINITY : acc[nt][mt][2 * r + 1] * u1);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < ST_ROWS / ST_WARPS; ++j) {
        const int r = warp + j * ST_WARPS;
        if (r < r0 || r >= r1 || row_pos[r] < 0) continue;
        const int cur = row_pos[r] / KV_BLOCK, m = min(min(cur + 1, a.tab.N) - base, SEL_CHUNK);
        if (m > 0)
          have[j] = select_piece(have[j], sc + r * ST_LD, m, a.k, a.n_sink, cur - a.n_local + 1,
                                 [&](int i) { return base + i; }, best_sc + r * a.k, best_id + r * a.k);
      }
    }
#pragma unroll
    for (int j = 0; j < ST_ROWS / ST_WARPS; ++j) {
      const int r = warp + j * ST_WARPS;
      if (r < r0 || r >= r1) continue;
      const size_t o = ((size_t)(t0 + r) * a.H + h) * a.k;
      const float up = pow2f(row_eq[r]);
      for (int i = lane; i < a.k; i += 32) {
        a.ids[o + i] = i < have[j] ? best_id[r * a.k + i] : -1;
        if (a.scores) a.scores[o + i] = i < have[j] ? best_sc[r * a.k + i] * up : 0.0f;
      }
    }
    r0 = r1;
  }
}

}  // namespace

size_t kv_select_ws_bytes(int T, int Hq, int H, int D, int B, int N, int k) { return 0; }

// Shared memory of the one-token kernel for stretches of `span` blocks.
static size_t select_rows_smem(int span, int k) { return (size_t)span * 8 + (size_t)(SR_WARPS + 8) * k * 8; }

cudaError_t launch_kv_select(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* q, long long q_stride, int Hq,
                             int k, int n_sink, int n_local, int32_t* ids, float* scores, void* ws, int32_t* err,
                             cudaStream_t s) {
  const int H = c->n_kv_heads, D = c->head_dim;
  const SelectArgs a{c->bounds, c->bound_exp, H,   Hq / H, KvTable{tk.table, tk.B, tk.N, c->n_pages},
                     q, q_stride, tk.seq, tk.pos, tk.T, k, n_sink, n_local, ids, scores, err};
  if (tk.T >= 16LL * tk.B) {
    auto kern = D == 128 ? kv_select_tiles_kernel<128> : kv_select_tiles_kernel<64>;
    const size_t smem = select_tiles_smem(D, k);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_k(kern, dim3((unsigned)((tk.T + ST_ROWS - 1) / ST_ROWS), (unsigned)H), dim3(ST_WARPS * 32), smem, s, a);
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
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_kc(kern, dim3((unsigned)(rows * ranks)), dim3(SR_WARPS * 32), ranks, smem, s, a);
}

}  // namespace bre

// Attention over the listed blocks for prefill: 128 rows at a time on the 5th-generation tensor cores.
//
// A CTA takes 128 / G tokens of the call with all G query heads of one kv head: 128 rows.  Each token
// has a block list of its own, but neighbours list mostly the same blocks, so the CTA walks through
// the union of its tokens' lists: every block is brought in and multiplied once for all rows, and
// a row whose token does not list it gets weights of zero.  Per block and 128 rows that is
// 4 * 128 * 64 * D operations whatever the number of rows that use it, against a row-by-row kernel's
// 16 KB from L2 for every (token, block).
//
// Fourteen warps:
//   warps 0-3   softmax: a thread a row; S from tensor memory, weights back over it as FP16
//   warps 4-7   turn the keys' codes into FP16 (exact) in 128-byte-swizzled shared memory
//   warps 8-11  the values'; two warps for the even blocks and two for the odd ones, so that a warp has twice the
//               time for its waits and loads
//   warp 12     merges the tokens' lists: the least next block over all tokens, and which tokens list it
//   warp 13     issues the MMAs: S = Q K^T into tensor memory, O += P V with P read from tensor memory
// K is K-major, V lies as it is in the cache (a token's channels in a row), which is the MN-major
// form of the second product's operand.  S and P share two buffers, K and V have two stages each.
//
// Scales: a key's 2^ek goes into its FP16 values relative to the block's largest as far as that is exact, down
// to 2^-15 (codes are multiples of 2^-9, FP16 values of 2^-24), the rest into the logits' factor: one for the block
// or, where some key is smaller still, one a token.  (The largest key may be one that a row does not even see.)  A
// value's 2^ev goes into its weight (see kv_attend.cu).  O is rescaled only when a
// row's maximum has grown by more than 2^7: the weights then still fit FP16.
#include <atomic>

#include "kv_attend.cuh"

namespace bre {

namespace {

constexpr int AT_CODES = 256;                       // threads that turn codes into FP16: keys, values
constexpr int AT_THREADS = 128 + AT_CODES + 64;
constexpr int W_MERGE = (128 + AT_CODES) / 32, W_MMA = W_MERGE + 1;
constexpr int AT_RING = 4;                          // blocks that the merging warp may be ahead
constexpr float AT_SLACK = 7.0f;                    // growth of a row's maximum (log2) that needs no rescaling
constexpr long long AT_WAIT = 4000000000LL;         // cycles before a wait gives up (~2 s), if no budget is set

struct Block {
  int page, id, n, pad;    // n: tokens that some row sees; page < 0: the end
  uint32_t mask[4];        // tokens of the tile that list it
};

template <int D>
struct TilesMem {
  static constexpr int Q = 128 * D * 2, KV = KV_BLOCK * D * 2;
  static constexpr int q = 0, k = q + Q, v = k + 2 * KV, end = v + 2 * KV;
  static constexpr int bytes = end + 1024;   // the swizzled tiles start on 1024 bytes
};

// Shared-memory descriptors of 128-byte-swizzled tiles: K-major (rows of 64 values, eight rows 1024 bytes
// apart from the next eight), and MN-major (rows of 64 values along M or N; the next 64 of them `panel`
// bytes on, the next eight of K 1024 bytes on).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr, uint32_t panel) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

#define BRE_R8(f, b) f(b), f(b + 1), f(b + 2), f(b + 3), f(b + 4), f(b + 5), f(b + 6), f(b + 7)
// 32 consecutive columns of this thread's tensor-memory lane; the values are there after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
#define BRE_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : BRE_R8(BRE_OUT, 0), BRE_R8(BRE_OUT, 8), BRE_R8(BRE_OUT, 16), BRE_R8(BRE_OUT, 24)
      : "r"(addr));
#undef BRE_OUT
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
#define BRE_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : BRE_R8(BRE_OUT, 0), BRE_R8(BRE_OUT, 8)
      : "r"(addr));
#undef BRE_OUT
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
#define BRE_IN(i) "r"(r[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      BRE_R8(BRE_IN, 0), BRE_R8(BRE_IN, 8)
      : "memory");
#undef BRE_IN
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The first try of a wait is inline, the bounded loop is not: with four roles in one kernel the
// instruction caches are what runs short first.
// A try suspends the warp for up to a millisecond: fourteen warps, half of them waiting, would otherwise take
// the workers' issue slots.
__device__ __forceinline__ bool try_wait_ms(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!try_wait_ms(bar, parity))
    if (clock64() - t0 > AT_WAIT) return false;
  return true;
}

// True in one lane.  The MMA warp stays together and lets one lane issue, so that the compiler keeps descriptors
// and addresses in uniform registers, where the MMA instructions want them.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Two FP32 values at a time.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Whether a key row that is not all zeros lies more than 2^15 below the block's largest scale `top`.  By a whole warp,
// with the scales of tokens lane and lane + 32 (0: not there).  Zero rows, whose scale is the least one, are exact in
// FP16 beside anything.  Out of line, as it is called for few blocks.
__device__ __noinline__ bool far_apart(const uint8_t* keys, int D, int ea, int eb, int top) {
  constexpr int LEAST = KV_EXP_MIN + 127;
  bool far = false;
  for (int half = 0; half < 2; ++half) {
    const int e = half ? eb : ea;
    if (e == 0 || top - e <= 15) continue;
    uint32_t codes = e == LEAST ? 0u : 1u;
    const uint4* row = reinterpret_cast<const uint4*>(keys + ((threadIdx.x & 31) + 32 * half) * D);
    for (int i = 0; codes == 0u && i < D / 16; ++i) {
      const uint4 w = __ldg(row + i);
      codes = (w.x | w.y | w.z | w.w) & 0x7F7F7F7Fu;
    }
    far |= codes != 0u;
  }
  __syncwarp();
  return __any_sync(0xffffffffu, far);
}

// A row's part of one block as in the main loop of the softmax, in steps that are right for scales of any size: the
// logits are S times the query's factor, then times the keys' own; terms of the sum are formed without the values'
// exponents ev.  A tile goes on this way from its first block whose keys are far apart or that has a value scale above
// EV_LARGE, in a loop of its own behind the main one (called in the main loop, where it is never taken, it cost 3 to
// 12 % of the kernel's time).
//
// The logits plus ev in place of S, -inf beyond n; their maximum.  By a whole warp; kt: the factor of the keys of
// tokens 0-31 and 32-63, where it is positive, else it is in ek for each.
__device__ __forceinline__ float careful_logits(uint32_t S, float2 kt, const float* ek, const float* ev, float qf, int n) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < KV_BLOCK; c += 16) {
    uint32_t s[16];
    tmem_ld16(S + c, s);
    tmem_wait_ld();
    const float k = c < 32 ? kt.x : kt.y;
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float v = c + x < n ? fmaf(__uint_as_float(s[x]) * qf, k > 0.0f ? k : ek[c + x], ev[c + x]) : -INFINITY;
      mx = fmaxf(mx, v);
      s[x] = __float_as_uint(v);
    }
    tmem_st16(S + c, s);
  }
  tmem_wait_st();
  return mx;
}
// The weights against the maximum m over those logits; what they add to the row's sum.
__device__ __forceinline__ float careful_weights(uint32_t S, const float* ev, float m, int n) {
  const float base = m > -INFINITY ? m - P_SHIFT : 0.0f;
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < KV_BLOCK; c += 32) {
    uint32_t s[32], pk[16];
    tmem_ld32(S + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const float v0 = __uint_as_float(s[x]) - base, v1 = __uint_as_float(s[x + 1]) - base;
      if (c + x < n) sum += exp2f(v0 - ev[c + x]);
      if (c + x + 1 < n) sum += exp2f(v1 - ev[c + x + 1]);
      pk[x / 2] = pack_f16x2(ex2(v0), ex2(v1));
    }
    tmem_st16(S + c / 2, pk);
  }
  return sum;
}
// O of a whole warp's rows times sc.
template <int D>
__device__ __forceinline__ void rescale(uint32_t O, float sc) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld16(O + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * sc);
    tmem_st16(O + c, o);
  }
  tmem_wait_st();
}

// PATIENT: the waits have the default budget; else the one that was set (a budget that is not a constant costs 5 %
// of the kernel's time, even where only the out-of-line wait knows it).
template <int D, bool PATIENT>
__global__ void __launch_bounds__(AT_THREADS, 2) kv_attend_tiles_kernel(const AttendArgs a) {
  using M = TilesMem<D>;
  constexpr int PANEL_Q = 128 * 128, PANEL = KV_BLOCK * 128;
  constexpr uint32_t COLS = 256;                   // tensor memory: S/P at 0 and 64, O at 128
  extern __shared__ unsigned char sm_raw[];
  __shared__ uint64_t blk_full[AT_RING], blk_empty[AT_RING], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2],
      p_full[2], o_done, drain, sc_full[AT_RING];
  __shared__ Block ring[AT_RING];
  __shared__ __align__(16) float ev_f[AT_RING][KV_BLOCK], ev_inv[AT_RING][KV_BLOCK], ek_f[AT_RING][KV_BLOCK];
  __shared__ float q_factor[128];
  __shared__ float2 ek_top[AT_RING];   // factor of a block's keys, one half by each warp; 0: see careful_logits
  __shared__ uint32_t tmem_s;
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = 128 / a.G;                       // tokens of a tile
  const int t0 = blockIdx.x * per, h = blockIdx.y, nt = min(per, a.T - t0), rows = nt * a.G;

  if (tid == 0) {
    for (int i = 0; i < AT_RING; ++i) mbar_init(&blk_full[i], 1), mbar_init(&sc_full[i], 2), mbar_init(&blk_empty[i], 4 + AT_CODES / 64 + 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 2);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 2);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(&o_done, 1);
    mbar_init(&drain, 1);
  }
  fence_mbar_init();
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();

  // queries: row r = (token r / G, head r % G) scaled by a power of two into FP16; K-major panels
  constexpr int PL = D / 32, QW = AT_THREADS / 32;
#pragma unroll 1
  for (int r0 = warp; r0 < 128; r0 += 10 * QW) {   // ten rows of a warp in flight: one round
    uint32_t w[10][PL / 2];
#pragma unroll
    for (int j = 0; j < 10; ++j) {
      const int r = r0 + j * QW, tl = r / a.G;
      const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q + (long long)(t0 + tl) * a.q_stride +
                                                             (size_t)(h * a.G + r - tl * a.G) * D) + lane * (PL / 2);
#pragma unroll
      for (int i = 0; i < PL / 2; ++i) w[j][i] = r < rows ? __ldg(qr + i) : 0u;
    }
#pragma unroll
    for (int j = 0; j < 10; ++j) {
      const int r = r0 + j * QW;
      if (r >= 128) break;
      uint32_t mx = 0;   // magnitudes of BF16 values compare like whole numbers; NaN and infinities count as 2^127
#pragma unroll
      for (int i = 0; i < PL / 2; ++i) mx = __vmaxu2(mx, w[j][i] & 0x7FFF7FFFu);
      mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
      const int e = query_exp(bf16_bits_to_f32(min(mx, 0x7F00u)));
      const float down = pow2f(-e);
      if (lane == 0) q_factor[r] = a.scale * LOG2E * pow2f(e);
      const int c = lane * PL;
      unsigned char* dst = sm + M::q + (c / 64) * PANEL_Q + r * 128 + ((((c % 64) / 8) ^ (r & 7)) << 4) + (c % 8) * 2;
#pragma unroll
      for (int i = 0; i < PL / 2; ++i)
        reinterpret_cast<uint32_t*>(dst)[i] =
            pack_f16x2(__uint_as_float(w[j][i] << 16) * down, __uint_as_float(w[j][i] & 0xFFFF0000u) * down);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  // Only now, when this CTA has its tensor memory: one thread's signal counts for the CTA, and a following launch of
  // this kernel takes its tensor memory before it waits for this grid.  Signalled earlier, it could take columns that a
  // CTA of this grid still waits for, and each would wait for the other.
  pdl_launch_dependents();
  tc_fence_after();
  const uint32_t tmem = tmem_s;

  bool ok = true;   // no wait of this thread has given up
  auto wait = [&](uint64_t* bar, int phase) {
    if (ok && (PATIENT ? !try_wait_ms(bar, phase & 1) && !wait_long(bar, phase & 1)
                       : !mbar_wait_bounded(bar, phase & 1, a.wait))) {
      ok = false;
      set_err(a.err, BRE_DEVERR_TIMEOUT);
    }
    return ok;
  };
  auto warp_wait = [&](uint64_t* bar, int phase) { return ok = __all_sync(0xffffffffu, wait(bar, phase)); };

  if (warp >= W_MERGE) {
    if (warp == W_MERGE) {
      // ---- merge: token 32 j + lane in slot j
      int pos[4], ptr[4] = {}, sq[4];
      uint32_t cur[4], run[4], starts[4];
      const int32_t* idr[4];
      auto advance = [&](int j) {   // the token's next block that it can see, as run << 25 | block
        cur[j] = 0xFFFFFFFFu;
        while (ptr[j] < a.k) {
          const int b = __ldg(idr[j] + ptr[j]++);
          if (b >= 0 && b <= pos[j] / KV_BLOCK) {
            cur[j] = run[j] | (uint32_t)min(b, (1 << 25) - 2);   // (larger tables are refused: that block is outside)
            break;
          }
        }
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tl = 32 * j + lane;
        const bool live = tl < nt;
        pos[j] = live ? __ldg(a.pos + t0 + tl) : -1;
        sq[j] = live ? __ldg(a.seq + t0 + tl) : -1;
        // tokens of one sequence in a row form a run, which goes by its first token
        int before = __shfl_up_sync(0xffffffffu, sq[j], 1);
        const int last = j ? __shfl_sync(0xffffffffu, sq[j ? j - 1 : 0], 31) : 0;
        if (lane == 0) before = last;
        starts[j] = __ballot_sync(0xffffffffu, tl == 0 || before != sq[j]);
        uint32_t first = 0;
#pragma unroll
        for (int i = 0; i <= j; ++i) {
          const uint32_t upto = i < j ? starts[i] : starts[i] & (0xFFFFFFFFu >> (31 - lane));
          if (upto) first = 32 * i + 31 - __clz(upto);
        }
        run[j] = first << 25;
        ptr[j] = pos[j] >= 0 ? 0 : a.k;
        idr[j] = a.ids + ((size_t)(t0 + (live ? tl : 0)) * a.H + h) * a.k;
        advance(j);
      }
      for (int i = 0, ends = 0;;) {
        const uint32_t key = __reduce_min_sync(0xffffffffu, min(min(cur[0], cur[1]), min(cur[2], cur[3])));
        Block b;
        b.page = -1;
        b.id = (int)(key & 0x1FFFFFFu);
        int top = -1;
        if (key != 0xFFFFFFFFu) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b.mask[j] = 0;
            if (32 * j >= nt) continue;
            b.mask[j] = __ballot_sync(0xffffffffu, cur[j] == key);
            if (cur[j] == key) {
              top = max(top, pos[j]);
              advance(j);
            }
          }
          top = __reduce_max_sync(0xffffffffu, top);
          b.page = kv_page(a.tab, __ldg(a.seq + t0 + (key >> 25)), b.id, lane == 0 ? a.err : nullptr);
          if (b.page < 0) continue;
        }
        b.n = min(KV_BLOCK, top - b.id * KV_BLOCK + 1);
        if (!warp_wait(&blk_empty[i % AT_RING], i / AT_RING + 1)) break;
        if (lane == 0) {
          ring[i % AT_RING] = b;
          mbar_arrive(&blk_full[i % AT_RING]);
        }
        ++i;
        if (key == 0xFFFFFFFFu && ++ends == 2) break;   // one for the even blocks' warps, one for the odd ones'
      }
    } else {
      // ---- MMA: kind::f16, FP32 sums, M = 128; second product with an MN-major B
      const uint32_t id_s = (1u << 4) | ((uint32_t)(KV_BLOCK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint64_t q0 = desc_k_major(smem_u32(sm + M::q)), k0 = desc_k_major(smem_u32(sm + M::k));
      const uint64_t v0 = desc_mn_major(smem_u32(sm + M::v), PANEL);   // offsets count 16 bytes
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      auto pv = [&](int i) {
        const int st = i & 1;
        if (!warp_wait(&v_full[st], i >> 1) || !warp_wait(&p_full[st], i >> 1)) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KV_BLOCK / 16; ++kk)
            mma_ts(tm + 128, tm + st * 64 + kk * 8, v0 + ((st * M::KV + kk * 2048) >> 4), id_o, kk > 0 ? 1u : i > 0);
          mma_commit(&v_empty[st]);
          mma_commit(&o_done);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int i = 0;; ++i) {
        const int st = i & 1;
        if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) break;
        const bool end = ring[i % AT_RING].page < 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
        if (!end) {
          // products into different accumulators may pass one another: the weights that lay in S's
          // columns must have been used
          if (i > 1 && !warp_wait(&o_done, i - 2)) break;
          if (!warp_wait(&k_full[st], i >> 1)) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tm + st * 64, q0 + (((kk / 4) * PANEL_Q + (kk % 4) * 32) >> 4),
                     k0 + ((st * M::KV + (kk / 4) * PANEL + (kk % 4) * 32) >> 4), id_s, kk > 0);
            mma_commit(&s_full[st]);
            mma_commit(&k_empty[st]);
          }
          __syncwarp();
        }
        if (i > 0) pv(i - 1);
        if (end || !ok) break;
      }
      // every MMA has completed before tensor memory is given back
      if (elect_one()) mma_commit(&drain);
      __syncwarp();
      mbar_wait_bounded(&drain, 0, AT_WAIT);
    }
  } else if (warp >= 4) {
    // ---- codes to FP16: 64 threads for the keys (values) of every other block, 16 codes (a 16-byte load) at a
    // time.  A warp works on its own rows; one arrival a warp.
    constexpr int CH = D / 16, NL = KV_BLOCK * CH / 64;   // pieces a row, loads a thread
    const bool values = warp >= 8;
    const int dt = tid & 63, st = (warp >> 1) & 1;        // st: parity of the blocks, and so the stage
    uint64_t* const full = values ? &v_full[st] : &k_full[st];
    uint64_t* const empty = values ? &v_empty[st] : &k_empty[st];
    uint4 cur[NL];
    int e2 = 0, ev = 0;     // key scales of tokens lane and lane + 32; value scale of token dt (keys' threads)
    int n = 0;
    const uint8_t* keys = nullptr;
    // of tokens that no row sees (they may never have been written) neither codes nor scales are read
    auto take_and_load = [&](int i) -> bool {
      if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) return false;
      const int page = ring[i % AT_RING].page;
      n = ring[i % AT_RING].n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
      if (page < 0) return false;
      const uint8_t* pg = a.pages + ((size_t)page * a.H + h) * kv_page_bytes(D);
      if (!values) keys = pg;
      const uint4* src = reinterpret_cast<const uint4*>(pg + (values ? KV_BLOCK * D : 0)) + dt;
      const uint8_t* sc = pg + 2 * KV_BLOCK * D;
#pragma unroll
      for (int j = 0; j < NL; ++j) cur[j] = (dt + j * 64) / CH < n ? __ldg(src + j * 64) : make_uint4(0, 0, 0, 0);
      if (!values) {
        e2 = lane < n ? (int)__ldg(sc + lane) : 0;
        if (lane + 32 < n) e2 |= (int)__ldg(sc + 32 + lane) << 8;
        ev = dt < n ? (int)__ldg(sc + KV_BLOCK + dt) : 127;
      }
      return true;
    };
    // where a thread puts its 16 values (token x0, channels 16 c ..; further loads are whole multiples of 8
    // tokens on): two swizzled pieces of 16 bytes.  The lanes of odd panels start with the second piece, so that
    // eight lanes meet all banks.
    const int x0 = dt / CH, c = dt % CH;
    const bool second = (c / 4) & 1;
    const int p0 = (values ? M::v : M::k) + st * M::KV + (c / 4) * PANEL + x0 * 128 + (((2 * (c % 4)) ^ (x0 & 7)) << 4);
    unsigned char* const put0 = sm + (second ? p0 ^ 16 : p0);
    unsigned char* const put1 = sm + (second ? p0 : p0 ^ 16);
#pragma unroll 1
    for (int i = st; take_and_load(i); i += 2) {
      if (!warp_wait(empty, (i >> 1) + 1)) break;
      int top = 0;
      if (!values) {
        // the block's largest key scale (a NaN row's does not count: its codes are zeros)
        const int ea = e2 & 255, eb = e2 >> 8;
        top = __reduce_max_sync(0xffffffffu, max(ea == KV_NAN ? 0 : ea, eb == KV_NAN ? 0 : eb));
        // the scales go to the softmax first.  Their place is free: S of two blocks ago has been formed, for which
        // the weights of four blocks ago must have been used.  A NaN row makes its token's logit NaN.
        const int sp = i % AT_RING;
        const bool nan = (dt < 32 ? ea : eb) == KV_NAN || ev == KV_NAN;
        ev_f[sp][dt] = nan ? __int_as_float(0x7FC00000) : (float)(ev - 127);
        ev_inv[sp][dt] = pow2f(127 - min(ev, 253));
        // tokens whose own scales reach below what FP16 holds relative to the largest (a byte of 0: not read)
        bool wide = __any_sync(0xffffffffu, (ea && top - ea > 15) || (eb && top - eb > 15));
        if (wide) wide = far_apart(keys, D, ea, eb, top);
        const bool large = __any_sync(0xffffffffu, ev > EV_LARGE);   // (of this warp's half; NaN rows as well)
        if (wide || large) {
          const int ek = dt < 32 ? ea : eb;
          ek_f[sp][dt] = pow2f(ek == KV_NAN ? 0 : ek + min(top - ek, 15) - 127);
        }
        if (lane == 0) reinterpret_cast<float*>(&ek_top[sp])[dt >> 5] = wide || large ? 0.0f : pow2f(max(top, 1) - 127);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[sp]);
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const uint32_t u[4] = {second ? cur[j].z : cur[j].x, second ? cur[j].w : cur[j].y, second ? cur[j].x : cur[j].z,
                               second ? cur[j].y : cur[j].w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] = e4m3x2_to_f16x2(u[k] & 0xFFFFu);
          o[2 * k + 1] = e4m3x2_to_f16x2(u[k] >> 16);
        }
        if (!values) {
          const int x = x0 + j * (64 / CH);
          const int both = __shfl_sync(0xffffffffu, e2, x & 31);
          const int d = max(top - (x < 32 ? both & 255 : both >> 8), 0);
          const uint32_t f = d < 15 ? (uint32_t)(15 - d) << 10 : 1u << 9;   // 2^-min(d, 15)
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = mul_f16x2(o[k], f | f << 16);
        }
        *reinterpret_cast<uint4*>(put0 + j * (64 / CH) * 128) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(put1 + j * (64 / CH) * 128) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
  } else {
    // ---- softmax: row tid
    const int r = tid, tl = r / a.G;
    const bool live = r < rows;
    const int pos = live ? __ldg(a.pos + t0 + tl) : -1;
    const float qf = q_factor[r];
    const uint32_t lane_base = tmem + ((uint32_t)warp << 21);   // lanes 32 warp ..
    float m = -INFINITY, l = 0.0f;   // m: the maximum that the weights are held against
    bool rare = false;               // a block that is not for this loop: see careful_logits
    int i = 0, n = 0;
    for (;; ++i) {
      const int st = i & 1;
      if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) break;
      const Block& b = ring[i % AT_RING];
      const int page = b.page, id = b.id;
      const bool mine = live && (b.mask[tl >> 5] >> (tl & 31) & 1u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
      if (page < 0) break;
      n = mine ? min(KV_BLOCK, pos - id * KV_BLOCK + 1) : 0;   // tokens that the row sees
      const int sp = i % AT_RING;
      if (!warp_wait(&sc_full[sp], i / AT_RING) || !warp_wait(&s_full[st], i >> 1)) break;
      tc_fence_after();
      const bool any = __any_sync(0xffffffffu, n > 0);   // else none of the warp's tokens lists the block
      // two passes over S, 32 columns at a time (as a loop: see wait_long): the maximum, then the weights
      const float2 kt = ek_top[sp];
      if (fminf(kt.x, kt.y) == 0.0f) {
        rare = true;
        break;
      }
      const float f = qf * kt.x;
      const uint64_t f2 = pack2(f, f);
      const bool whole = __all_sync(0xffffffffu, n == 0 || n == KV_BLOCK);
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = any ? 0 : KV_BLOCK; c < KV_BLOCK; c += 32) {
        uint32_t s[32];
        tmem_ld32(lane_base + st * 64 + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const ulonglong2 ev = *reinterpret_cast<const ulonglong2*>(&ev_f[sp][c + x]);
          const float2 v0 = unpack2(fma2(pack2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), f2, ev.x));
          const float2 v1 = unpack2(fma2(pack2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), f2, ev.y));
          s[x] = __float_as_uint(v0.x), s[x + 1] = __float_as_uint(v0.y);
          s[x + 2] = __float_as_uint(v1.x), s[x + 3] = __float_as_uint(v1.y);
        }
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (c + x >= n) s[x] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int x = 0; x < 32; x += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
      }
      if (n == 0) mx = -INFINITY;
      if (m == -INFINITY) m = mx;   // nothing has been added for this row yet
      if (__any_sync(0xffffffffu, mx > m + AT_SLACK)) {
        // some row's weights would outgrow FP16: all rows of the warp take their new maximum
        if (!warp_wait(&o_done, i - 1)) break;
        tc_fence_after();
        const float nm = fmaxf(m, mx), d = m > -INFINITY ? m - nm : 0.0f, sc = ex2(d);
        m = nm;
        l = scale_sum(l, d);
        rescale<D>(lane_base + 128, sc);
      }
      const float base = m > -INFINITY ? m - P_SHIFT : 0.0f;
      const uint64_t nb2 = pack2(-base, -base);
      uint64_t add = 0;
#pragma unroll 1
      for (int c = 0; c < KV_BLOCK; c += 32) {
        uint32_t s[32], pk[16];
        if (!any) {
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[x] = 0u;
          tmem_st16(lane_base + st * 64 + c / 2, pk);
          continue;
        }
        tmem_ld32(lane_base + st * 64 + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const ulonglong2 ev = *reinterpret_cast<const ulonglong2*>(&ev_f[sp][c + x]);
          const float2 v0 = unpack2(add2(fma2(pack2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), f2, ev.x), nb2));
          const float2 v1 =
              unpack2(add2(fma2(pack2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), f2, ev.y), nb2));
          s[x] = __float_as_uint(ex2(v0.x)), s[x + 1] = __float_as_uint(ex2(v0.y));
          s[x + 2] = __float_as_uint(ex2(v1.x)), s[x + 3] = __float_as_uint(ex2(v1.y));
        }
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (c + x >= n) s[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const ulonglong2 iv = *reinterpret_cast<const ulonglong2*>(&ev_inv[sp][c + x]);
          const float p0 = __uint_as_float(s[x]), p1 = __uint_as_float(s[x + 1]);
          const float p2 = __uint_as_float(s[x + 2]), p3 = __uint_as_float(s[x + 3]);
          add = fma2(pack2(p0, p1), iv.x, fma2(pack2(p2, p3), iv.y, add));
          pk[x / 2] = n ? pack_f16x2(p0, p1) : 0u;
          pk[x / 2 + 1] = n ? pack_f16x2(p2, p3) : 0u;
        }
        tmem_st16(lane_base + st * 64 + c / 2, pk);
      }
      const float2 sum = unpack2(add);
      if (n) l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[st]);
    }
    // the rest of the tile's blocks from the first rare one on
    while (rare && ok) {
      const int st = i & 1, sp = i % AT_RING;
      const float mx = careful_logits(lane_base + st * 64, ek_top[sp], ek_f[sp], ev_f[sp], qf, n);
      if (m == -INFINITY) m = mx;
      if (__any_sync(0xffffffffu, mx > m + AT_SLACK)) {
        if (!warp_wait(&o_done, i - 1)) break;
        tc_fence_after();
        const float nm = fmaxf(m, mx), d = m > -INFINITY ? m - nm : 0.0f;
        m = nm;
        l = scale_sum(l, d);
        rescale<D>(lane_base + 128, ex2(d));
      }
      l += careful_weights(lane_base + st * 64, ev_f[sp], m, n);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[st]);
      ++i;
      if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) break;
      const Block& b = ring[i % AT_RING];
      const int page = b.page;
      n = live && (b.mask[tl >> 5] >> (tl & 31) & 1u) ? min(KV_BLOCK, pos - b.id * KV_BLOCK + 1) : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
      if (page < 0 || !warp_wait(&sc_full[i % AT_RING], i / AT_RING) || !warp_wait(&s_full[i & 1], i >> 1)) break;
      tc_fence_after();
    }
    if (i > 0) warp_wait(&drain, 0);   // not o_done: the last two products with V may both be pending
    tc_fence_after();
    // output: a thread its row
    const size_t row = ((size_t)(t0 + tl) * a.H + h) * a.G + (r - tl * a.G);
    const float inv = 1.0f / l;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t o[16], w[8];
      if (i > 0) {
        tmem_ld16(lane_base + 128 + c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
        w[x] = l == 0.0f ? 0u : pack_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
      if (live && ok) st_v8(a.out + row * D + c, w);
    }
    if (live && ok && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : LN2 * ((m > -INFINITY ? m - P_SHIFT : 0.0f) + log2f(l));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS) : "memory");
  }
}

template <int D, bool PATIENT>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};   // devices on which the kernel may have its shared memory
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_attend_tiles_kernel<D, PATIENT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               TilesMem<D>::bytes);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_release);
  }
  const int per = 128 / a.G;
  return launch_k(kv_attend_tiles_kernel<D, PATIENT>, dim3((unsigned)((a.T + per - 1) / per), (unsigned)a.H), dim3(AT_THREADS),
                  TilesMem<D>::bytes, s, a);
}

}  // namespace

cudaError_t launch_kv_attend_tiles(const AttendArgs& args, int D, cudaStream_t s) {
  AttendArgs a = args;
  a.wait = ffn_wait_budget(0);   // 0: none set
  if (a.wait) return D == 128 ? launch<128, false>(a, s) : launch<64, false>(a, s);
  return D == 128 ? launch<128, true>(a, s) : launch<64, true>(a, s);
}

}  // namespace bre

// Attention over the listed blocks for prefill: 128 rows at a time on the 5th-generation tensor cores.
//
// A CTA takes 128 / G tokens of the call with all G query heads of one kv head: 128 rows.  Each token
// has a block list of its own, but neighbours list mostly the same blocks, so the CTA walks through
// the union of its tokens' lists: every block is brought in and multiplied once for all rows, and
// a row whose token does not list it gets weights of zero.  Per block and 128 rows that is
// 4 * 128 * 64 * D operations whatever the number of rows that use it, against a row-by-row kernel's
// 16 KB from L2 for every (token, block).
//
// Ten warps:
//   warps 0-3   softmax: a thread a row; S from tensor memory, weights back over it as FP16
//   warps 4-7   turn the codes into FP16 (exact) in 128-byte-swizzled shared memory; the next block's
//               codes are loaded into the registers that the current block's have left
//   warp 8      merges the tokens' lists: the least next block over all tokens, and which tokens list it
//   warp 9      issues the MMAs: S = Q K^T into tensor memory, O += P V with P read from tensor memory
// K is K-major, V lies as it is in the cache (a token's channels in a row), which is the MN-major
// form of the second product's operand.  S and P share two buffers, K and V have two stages each.
//
// Scales: a key's 2^ek goes into its FP16 values relative to the block's largest (exact unless it
// is 2^15 times smaller, and then off by less than 2^-24 of the block's largest logit), the rest into the
// logits' factor; a value's 2^ev goes into its weight (see kv_attend.cu).  O is rescaled only when a
// row's maximum has grown by more than 2^7: the weights then still fit FP16.
#include "kv_attend.cuh"

namespace bre {

namespace {

constexpr int AT_THREADS = 320;
constexpr int AT_RING = 4;                          // blocks that the merging warp may be ahead
constexpr float AT_SLACK = 7.0f;                    // growth of a row's maximum (log2) that needs no rescaling
constexpr long long AT_WAIT = 4000000000LL;         // cycles before a wait gives up (~2 s)

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

template <int D>
__global__ void __launch_bounds__(AT_THREADS, 2) kv_attend_tiles_kernel(const AttendArgs a) {
  using M = TilesMem<D>;
  constexpr int PANEL_Q = 128 * 128, PANEL = KV_BLOCK * 128;
  constexpr uint32_t COLS = 256;                   // tensor memory: S/P at 0 and 64, O at 128
  extern __shared__ unsigned char sm_raw[];
  __shared__ uint64_t blk_full[AT_RING], blk_empty[AT_RING], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2],
      p_full[2], o_done, drain;
  __shared__ Block ring[AT_RING];
  __shared__ __align__(16) float ev_f[2][KV_BLOCK], ev_inv[2][KV_BLOCK];
  __shared__ float q_factor[128], ek_top[2];
  __shared__ uint32_t tmem_s;
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = 128 / a.G;                       // tokens of a tile
  const int t0 = blockIdx.x * per, h = blockIdx.y, nt = min(per, a.T - t0), rows = nt * a.G;

  if (tid == 0) {
    for (int i = 0; i < AT_RING; ++i) mbar_init(&blk_full[i], 1), mbar_init(&blk_empty[i], 9);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(&o_done, 1);
    mbar_init(&drain, 1);
  }
  fence_mbar_init();
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_s)), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();

  // queries: row r = (token r / G, head r % G) scaled by a power of two into FP16; K-major panels
  {
    constexpr int PL = D / 32;
    for (int r = warp; r < 128; r += AT_THREADS / 32) {
      const int tl = r / a.G;
      uint32_t w[PL / 2] = {};
      if (r < rows) {
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(a.q + (long long)(t0 + tl) * a.q_stride +
                                                               (size_t)(h * a.G + r - tl * a.G) * D) + lane * (PL / 2);
#pragma unroll
        for (int i = 0; i < PL / 2; ++i) w[i] = __ldg(qr + i);
      }
      float x[PL], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        x[i] = bf16_bits_to_f32(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
        amax = fmaxf(amax, fabsf(kv_clamp(x[i])));
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
      const int e = query_exp(amax);
      const float down = pow2f(-e);
      if (lane == 0) q_factor[r] = a.scale * LOG2E * pow2f(e);
      const int c = lane * PL;
      unsigned char* dst = sm + M::q + (c / 64) * PANEL_Q + r * 128 + ((((c % 64) / 8) ^ (r & 7)) << 4) + (c % 8) * 2;
#pragma unroll
      for (int i = 0; i < PL / 2; ++i)
        reinterpret_cast<uint32_t*>(dst)[i] = pack_f16x2(x[2 * i] * down, x[2 * i + 1] * down);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;

  bool ok = true;   // no wait of this thread has given up
  auto wait = [&](uint64_t* bar, int phase) {
    if (ok && !mbar_wait_bounded(bar, phase & 1, AT_WAIT)) {
      ok = false;
      set_err(a.err, BRE_DEVERR_TIMEOUT);
    }
    return ok;
  };
  auto warp_wait = [&](uint64_t* bar, int phase) { return ok = __all_sync(0xffffffffu, wait(bar, phase)); };

  if (warp >= 8) {
    if (warp == 8) {
      // ---- merge: token 32 j + lane in slot j
      int pos[4], ptr[4] = {}, sq[4];
      uint32_t cur[4], run[4], starts[4];
      const int32_t* idr[4];
      auto advance = [&](int j) {   // the token's next block that it can see, as run << 25 | block
        cur[j] = 0xFFFFFFFFu;
        while (ptr[j] < a.k) {
          const int b = __ldg(idr[j] + ptr[j]++);
          if (b >= 0 && b <= pos[j] / KV_BLOCK) {
            cur[j] = run[j] | (uint32_t)min(b, (1 << 25) - 2);
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
      for (int i = 0;;) {
        const uint32_t key = __reduce_min_sync(0xffffffffu, min(min(cur[0], cur[1]), min(cur[2], cur[3])));
        Block b;
        b.page = -1;
        b.id = (int)(key & 0x1FFFFFFu);
        int top = -1;
        if (key != 0xFFFFFFFFu) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
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
        if (key == 0xFFFFFFFFu) break;
      }
    } else {
      if (lane == 0) {
      // ---- MMA: kind::f16, FP32 sums, M = 128; second product with an MN-major B
      const uint32_t id_s = (1u << 4) | ((uint32_t)(KV_BLOCK >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t q0 = smem_u32(sm + M::q), k0 = smem_u32(sm + M::k), v0 = smem_u32(sm + M::v);
      auto pv = [&](int i) {
        const int st = i & 1;
        if (!wait(&v_full[st], i >> 1) || !wait(&p_full[st], i >> 1)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < KV_BLOCK / 16; ++kk)
          mma_ts(tmem + 128, tmem + st * 64 + kk * 8, desc_mn_major(v0 + st * M::KV + kk * 2048, PANEL), id_o,
                 i > 0 || kk > 0);
        mma_commit(&v_empty[st]);
        mma_commit(&o_done);
      };
      int i = 0;
      for (;; ++i) {
        const int st = i & 1;
        if (!wait(&blk_full[i % AT_RING], i / AT_RING)) break;
        const bool end = ring[i % AT_RING].page < 0;
        mbar_arrive(&blk_empty[i % AT_RING]);
        if (!end) {
          // products into different accumulators may pass one another: the weights that lay in S's
          // columns must have been used
          if (i > 1 && !wait(&o_done, i - 2)) break;
          if (!wait(&k_full[st], i >> 1)) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tmem + st * 64, desc_k_major(q0 + (kk / 4) * PANEL_Q + (kk % 4) * 32),
                   desc_k_major(k0 + st * M::KV + (kk / 4) * PANEL + (kk % 4) * 32), id_s, kk > 0);
          mma_commit(&s_full[st]);
          mma_commit(&k_empty[st]);
        }
        if (i > 0) pv(i - 1);
        if (end || !ok) break;
      }
      // every MMA has completed before tensor memory is given back
      mma_commit(&drain);
      mbar_wait_bounded(&drain, 0, AT_WAIT);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---- codes to FP16: 128 threads, 16 codes (one 16-byte load) at a time
    constexpr int CH = D / 16, NL = KV_BLOCK * CH / 128;   // pieces a row, loads a thread
    const int dt = tid - 128;
    uint4 kr[NL], vr[NL];
    int e2 = 0, ek = 0, ev = 0;   // key scales of tokens lane and lane + 32; scales of token dt
    int page = 0, n = 0;  // of the block whose codes are loaded next
    const uint8_t* pg = nullptr;
    auto take = [&](int i) {
      if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) {
        page = -1;
        return;
      }
      page = ring[i % AT_RING].page;
      n = ring[i % AT_RING].n;
      __syncwarp();
      if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
      pg = a.pages + ((size_t)max(page, 0) * a.H + h) * kv_page_bytes(D);
    };
    // of tokens that no row sees (they may never have been written) neither values nor scales are read
    auto load_k = [&] {
#pragma unroll
      for (int j = 0; j < NL; ++j) kr[j] = __ldg(reinterpret_cast<const uint4*>(pg) + dt + j * 128);
      e2 = lane < n ? (int)__ldg(pg + 2 * KV_BLOCK * D + lane) : 0;
      if (lane + 32 < n) e2 |= (int)__ldg(pg + 2 * KV_BLOCK * D + 32 + lane) << 8;
      ek = dt < n ? (int)__ldg(pg + 2 * KV_BLOCK * D + dt % KV_BLOCK) : 0;
    };
    auto load_v = [&] {
#pragma unroll
      for (int j = 0; j < NL; ++j)
        vr[j] = (dt + j * 128) / CH < n ? __ldg(reinterpret_cast<const uint4*>(pg + KV_BLOCK * D) + dt + j * 128)
                                        : make_uint4(0, 0, 0, 0);
      ev = dt < n ? (int)__ldg(pg + 2 * KV_BLOCK * D + KV_BLOCK + dt % KV_BLOCK) : 127;
    };
    // 16 values of token x, channels 16 c ..: two swizzled pieces of 16 bytes; the upper half of a quarter
    // warp's lanes starts with its second piece, so that eight lanes meet all banks
    auto put = [&](unsigned char* tile, int x, int c, const uint4& w, uint32_t f) {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[2 * j] = mul_f16x2(e4m3x2_to_f16x2(u[j] & 0xFFFFu), f);
        o[2 * j + 1] = mul_f16x2(e4m3x2_to_f16x2(u[j] >> 16), f);
      }
      unsigned char* row = tile + (c / 4) * PANEL + x * 128;
      const int c0 = 2 * (c % 4), sw = x & 7;
      const bool second = (c / 4) & 1;
      const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(row + (((c0 + (second ? 1 : 0)) ^ sw) << 4)) = second ? hi : lo;
      *reinterpret_cast<uint4*>(row + (((c0 + (second ? 0 : 1)) ^ sw) << 4)) = second ? lo : hi;
    };
    take(0);
    if (page >= 0) load_k(), load_v();
    for (int i = 0; page >= 0; ++i) {
      const int st = i & 1;
      // the block's largest key scale (a NaN row's does not count: its codes are zeros)
      const int top = __reduce_max_sync(0xffffffffu, max((e2 & 255) == KV_NAN ? 0 : e2 & 255, (e2 >> 8) == KV_NAN ? 0 : e2 >> 8));
      const bool nan_key = ek == KV_NAN;
      if (!warp_wait(&k_empty[st], (i >> 1) + 1)) break;
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int x = (dt + j * 128) / CH, c = (dt + j * 128) % CH;
        const int both = __shfl_sync(0xffffffffu, e2, x & 31);
        const int d = max(top - (x < 32 ? both & 255 : both >> 8), 0);
        const uint32_t f = d < 15 ? (uint32_t)(15 - d) << 10 : d < 25 ? 1u << (24 - d) : 0u;   // 2^-d in FP16
        put(sm + M::k + st * M::KV, x, c, kr[j], f | f << 16);
      }
      fence_proxy_async_smem();
      mbar_arrive(&k_full[st]);
      take(i + 1);
      if (page >= 0) load_k();
      if (!warp_wait(&v_empty[st], (i >> 1) + 1)) break;   // and the softmax is done with the scales before
      if (dt < KV_BLOCK) {
        // a NaN row makes its token's logit NaN
        ev_f[st][dt] = nan_key || ev == KV_NAN ? __int_as_float(0x7FC00000) : (float)(ev - 127);
        ev_inv[st][dt] = pow2f(127 - min(ev, 253));
        if (dt == 0) ek_top[st] = pow2f(max(top, 1) - 127);
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) put(sm + M::v + st * M::KV, (dt + j * 128) / CH, (dt + j * 128) % CH, vr[j], 0x3C003C00u);
      fence_proxy_async_smem();
      mbar_arrive(&v_full[st]);
      if (page >= 0) load_v();
    }
  } else {
    // ---- softmax: row tid
    const int r = tid, tl = r / a.G;
    const bool live = r < rows;
    const int pos = live ? __ldg(a.pos + t0 + tl) : -1;
    const float qf = q_factor[r];
    const uint32_t lane_base = tmem + ((uint32_t)warp << 21);   // lanes 32 warp ..
    float m = -INFINITY, l = 0.0f;   // m: the maximum that the weights are held against
    int i = 0;
    for (;; ++i) {
      const int st = i & 1;
      if (!warp_wait(&blk_full[i % AT_RING], i / AT_RING)) break;
      const Block& b = ring[i % AT_RING];
      const int page = b.page, id = b.id;
      const bool mine = live && (b.mask[tl >> 5] >> (tl & 31) & 1u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&blk_empty[i % AT_RING]);
      if (page < 0) break;
      const int n = mine ? min(KV_BLOCK, pos - id * KV_BLOCK + 1) : 0;   // tokens that the row sees
      if (!warp_wait(&v_full[st], i >> 1) || !warp_wait(&s_full[st], i >> 1)) break;   // the scales, the products
      tc_fence_after();
      uint32_t s[64];
      tmem_ld32(lane_base + st * 64, s);
      tmem_ld32(lane_base + st * 64 + 32, s + 32);
      const float f = qf * ek_top[st];
      const uint64_t f2 = pack2(f, f);
      tmem_wait_ld();
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < 64; x += 4) {
        const ulonglong2 ev = *reinterpret_cast<const ulonglong2*>(&ev_f[st][x]);
        const float2 v0 = unpack2(fma2(pack2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), f2, ev.x));
        const float2 v1 = unpack2(fma2(pack2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), f2, ev.y));
        s[x] = __float_as_uint(v0.x), s[x + 1] = __float_as_uint(v0.y);
        s[x + 2] = __float_as_uint(v1.x), s[x + 3] = __float_as_uint(v1.y);
      }
      if (!__all_sync(0xffffffffu, n == 0 || n == KV_BLOCK)) {
#pragma unroll
        for (int x = 0; x < 64; ++x)
          if (x >= n) s[x] = __float_as_uint(-INFINITY);
      }
#pragma unroll
      for (int x = 0; x < 64; x += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
      if (n == 0) mx = -INFINITY;
      if (m == -INFINITY) m = mx;   // nothing has been added for this row yet
      if (__any_sync(0xffffffffu, mx > m + AT_SLACK)) {
        // some row's weights would outgrow FP16: all rows of the warp take their new maximum
        if (!warp_wait(&o_done, i - 1)) break;
        tc_fence_after();
        const float nm = fmaxf(m, mx), sc = m > -INFINITY ? ex2(m - nm) : 1.0f;
        m = nm;
        l *= sc;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_ld16(lane_base + 128 + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * sc);
          tmem_st16(lane_base + 128 + c, o);
        }
        tmem_wait_st();
      }
      const float base = m > -INFINITY ? m - P_SHIFT : 0.0f;
      const uint64_t nb2 = pack2(-base, -base);
      uint64_t add = 0;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[16];
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const uint32_t* sx = s + hf * 32 + x;
          const ulonglong2 iv = *reinterpret_cast<const ulonglong2*>(&ev_inv[st][hf * 32 + x]);
          const float2 v0 = unpack2(add2(pack2(__uint_as_float(sx[0]), __uint_as_float(sx[1])), nb2));
          const float2 v1 = unpack2(add2(pack2(__uint_as_float(sx[2]), __uint_as_float(sx[3])), nb2));
          const float p0 = ex2(v0.x), p1 = ex2(v0.y), p2 = ex2(v1.x), p3 = ex2(v1.y);
          add = fma2(pack2(p0, p1), iv.x, fma2(pack2(p2, p3), iv.y, add));
          pk[x / 2] = n ? pack_f16x2(p0, p1) : 0u;
          pk[x / 2 + 1] = n ? pack_f16x2(p2, p3) : 0u;
        }
        tmem_st16(lane_base + st * 64 + hf * 16, pk);
      }
      const float2 sum = unpack2(add);
      if (n) l += sum.x + sum.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[st]);
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
        w[x] = l == 0.0f ? 0u
                         : f32_to_bf16_rne(__uint_as_float(o[2 * x]) * inv) |
                               f32_to_bf16_rne(__uint_as_float(o[2 * x + 1]) * inv) << 16;
      if (live && ok) {
        *reinterpret_cast<uint4*>(a.out + row * D + c) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(a.out + row * D + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    if (live && ok && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : LN2 * ((m > -INFINITY ? m - P_SHIFT : 0.0f) + log2f(l));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLS) : "memory");
  }
}

template <int D>
cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kv_attend_tiles_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             TilesMem<D>::bytes);
  if (e != cudaSuccess) return e;
  const int per = 128 / a.G;
  return launch_k(kv_attend_tiles_kernel<D>, dim3((unsigned)((a.T + per - 1) / per), (unsigned)a.H), dim3(AT_THREADS),
                  TilesMem<D>::bytes, s, a);
}

}  // namespace

cudaError_t launch_kv_attend_tiles(const AttendArgs& a, int D, cudaStream_t s) {
  return D == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace bre

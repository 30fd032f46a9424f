// Attention over the listed blocks of the quantised cache.
#include "kv_attend.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// A token's heads at a time: decode and verify batches
// ---------------------------------------------------------------------------
// A cluster of CTAs per (token, kv head); the listed blocks are dealt to its warps in halves of 32
// tokens.  A warp computes S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16 (FP16 operands, FP32
// sums): tokens or channels are the 16 rows, eight query heads the 8 columns, so no tensor-core
// row is padding for G = 8 or 16.  The cache's codes go from memory to the fragments without
// shared memory: the 16 channels (K) or the four tokens' 16 channels (V) that a lane loads are
// the ones its fragment rows need, because the order of a contraction and the numbering of the
// output channels are free.  E4M3 -> FP16 is exact.  A key's scale multiplies its logit.  A
// value's scale 2^ev is put into the weight: with s' = s + ev in the log2 domain and the running
// maximum M taken over s', the weights 2^(s' - M) are at most 1 whatever the values' scales, and
// the sum of exponentials gets back the factor 2^-ev.
constexpr int AR_WARPS = 4;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// CTAs to an SM.  The loads of a half block are all issued before its first product, so warps are what keeps
// memory busy: 64 tokens x 32 blocks take 41 us with three CTAs, 30 with four, 47 with five (spills).  Both halves of 16 heads at D = 128 need the registers of two.
constexpr int ar_ctas(int D, int NT) { return NT == 1 || D == 64 ? 4 : 2; }

// NT: groups of eight query heads.
template <int D, int NT>
__global__ void __launch_bounds__(AR_WARPS * 32, ar_ctas(D, NT)) kv_attend_rows_kernel(const AttendArgs a) {
  constexpr int HB = D / 64;       // 64-channel halves of a key row
  constexpr int MT = D / 16;       // 16-channel row tiles of O^T
  constexpr int VW = D / 32;       // 4-channel words of a value row that a lane holds
  constexpr int PB = kv_page_bytes(D);
  __shared__ float part_o[AR_WARPS][8 * NT][D];
  __shared__ float part_m[AR_WARPS][8 * NT], part_l[AR_WARPS][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  const int row = blockIdx.x / ranks, t = row / a.H, h = row - t * a.H;
  pdl_wait();
  pdl_launch_dependents();
  const int p = __ldg(a.pos + t), s = __ldg(a.seq + t);

  // the query's fragments: B of S^T, head 8 nt + g, channels 64 hb + 16 t4 + 4 i + {0, 1}, {2, 3}
  uint32_t qf[NT][HB][4][2];
  float qs[NT][2];   // logit factors of heads 8 nt + 2 t4, + 1 (the columns of this lane's sums)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float x[HB * 16], amax = 0.0f;
    const bool live = 8 * nt + g < a.G;
    const uint16_t* qr = a.q + t * a.q_stride + (size_t)(h * a.G + 8 * nt + g) * D + 16 * t4;
#pragma unroll
    for (int hb = 0; hb < HB; ++hb)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint4 w = live ? __ldg(reinterpret_cast<const uint4*>(qr + 64 * hb) + v) : make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[hb * 16 + v * 8 + 2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
          x[hb * 16 + v * 8 + 2 * i + 1] = bf16_bits_to_f32(u[i] >> 16);
        }
      }
#pragma unroll
    for (int i = 0; i < HB * 16; ++i) amax = fmaxf(amax, fminf(fabsf(x[i]), KV_MAX));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = query_exp(amax);
    const float down = pow2f(-e);
#pragma unroll
    for (int hb = 0; hb < HB; ++hb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          qf[nt][hb][i][j] = pack_f16x2(x[hb * 16 + 4 * i + 2 * j] * down, x[hb * 16 + 4 * i + 2 * j + 1] * down);
    const float f = a.scale * LOG2E * pow2f(e);
    qs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
    qs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
  }

  float o[NT][MT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.0f;
  }

  bool large = false;   // a value scale above EV_LARGE has been met
  const int step = ranks * AR_WARPS, items = 2 * a.k;
  const int32_t* idr = a.ids + (size_t)row * a.k;
  for (int base = rank * AR_WARPS + warp; base < items; base += 32 * step) {
    // this lane looks up the block of one of the warp's next 32 halves
    const int it = base + lane * step;
    int my_page = -1, my_n = 0;
    if (it < items && p >= 0) {
      const int b = __ldg(idr + (it >> 1));
      if (b >= 0 && b <= p / KV_BLOCK) {
        my_n = min(32, p - b * KV_BLOCK - 32 * (it & 1) + 1);
        if (my_n > 0) my_page = kv_page(a.tab, s, b, a.err);
      }
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, my_page >= 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int page = __shfl_sync(0xffffffffu, my_page, src), n = __shfl_sync(0xffffffffu, my_n, src);
      const int half = (base + src * step) & 1;
      const uint8_t* pg = a.pages + ((size_t)page * a.H + h) * PB + half * 32 * D;
      const uint8_t* ps = a.pages + ((size_t)page * a.H + h) * PB + 2 * KV_BLOCK * D + half * 32;
      // loads: key rows 16 mt + 8 r + g; value rows 16 mt + 8 r + 2 t4 + c; rows past the token's own
      // position are not read (whatever they hold must not reach a product)
      uint4 kf[2][2][HB];
      uint32_t vf[2][2][2][VW];
      int ek[2][2], ev[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int x = 16 * mt + 8 * r + g;
#pragma unroll
          for (int hb = 0; hb < HB; ++hb)
            kf[mt][r][hb] = x < n ? __ldg(reinterpret_cast<const uint4*>(pg + x * D + 64 * hb) + t4)
                                  : make_uint4(0, 0, 0, 0);
          ek[mt][r] = x < n ? (int)__ldg(ps + x) : 127;
          ev[mt][r] = x < n ? (int)__ldg(ps + KV_BLOCK + x) : 127;
        }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int x = 16 * mt + 8 * r + 2 * t4 + c;
            const uint8_t* vr = pg + KV_BLOCK * D + x * D + (D / 8) * g;
            if (D == 128) {
              const uint4 w = x < n ? __ldg(reinterpret_cast<const uint4*>(vr)) : make_uint4(0, 0, 0, 0);
              vf[mt][r][c][0] = w.x, vf[mt][r][c][1] = w.y;
              vf[mt][r][c][VW - 2] = w.z, vf[mt][r][c][VW - 1] = w.w;
            } else {
              const uint2 w = x < n ? __ldg(reinterpret_cast<const uint2*>(vr)) : make_uint2(0, 0);
              vf[mt][r][c][0] = w.x, vf[mt][r][c][1] = w.y;
            }
          }
      // S^T
      float sc[NT][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[nt][mt][j] = 0.0f;
#pragma unroll
      for (int hb = 0; hb < HB; ++hb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint32_t w0 = i == 0 ? kf[mt][0][hb].x : i == 1 ? kf[mt][0][hb].y : i == 2 ? kf[mt][0][hb].z : kf[mt][0][hb].w;
            const uint32_t w1 = i == 0 ? kf[mt][1][hb].x : i == 1 ? kf[mt][1][hb].y : i == 2 ? kf[mt][1][hb].z : kf[mt][1][hb].w;
            const uint32_t a0 = e4m3x2_to_f16x2(w0 & 0xFFFFu), a2 = e4m3x2_to_f16x2(w0 >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(w1 & 0xFFFFu), a3 = e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(sc[nt][mt], a0, a1, a2, a3, qf[nt][hb][i][0], qf[nt][hb][i][1]);
          }
      float kf2[2][2], evf[2][2];   // 2^ek; ev, or NaN where the token's key or value row is NaN
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          kf2[mt][r] = pow2f(ek[mt][r] - 127);
          evf[mt][r] = ek[mt][r] == KV_NAN || ev[mt][r] == KV_NAN ? __int_as_float(0x7FC00000) : (float)(ev[mt][r] - 127);
        }
      bool beyond = false;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) beyond |= ev[mt][r] > EV_LARGE;   // (NaN rows as well; unseen tokens have 127)
      large |= __any_sync(0xffffffffu, beyond);
      // weights; sc[mt][2 r + c] is token 16 mt + 8 r + g, head 2 t4 + c
      uint32_t pb[NT][2][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float& v = sc[nt][mt][2 * r + c];
              v = 16 * mt + 8 * r + g < n ? fmaf(v * qs[nt][c], kf2[mt][r], evf[mt][r]) : -INFINITY;
              mx[c] = fmaxf(mx[c], v);
            }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
          mx[c] = fmaxf(mx[c], m[nt][c]);
          const float base_m = mx[c] > -INFINITY ? mx[c] - P_SHIFT : 0.0f;   // NaN logits have no maximum
          const float r0 = ex2(m[nt][c] - P_SHIFT - base_m);
          l[nt][c] = scale_sum(l[nt][c], m[nt][c] - P_SHIFT - base_m);
          m[nt][c] = mx[c];
          float without = l[nt][c];
          if (large) {
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int r = 0; r < 2; ++r) without += exp2f(sc[nt][mt][2 * r + c] - base_m - evf[mt][r]);
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) o[nt][i][c] *= r0, o[nt][i][2 + c] *= r0;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& v = sc[nt][mt][2 * r + c];
              v = ex2(v - base_m);
              l[nt][c] = fmaf(v, pow2f(127 - ev[mt][r]), l[nt][c]);
            }
          if (large) l[nt][c] = without;
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r) pb[nt][mt][r] = movmatrix_trans(pack_f16x2(sc[nt][mt][2 * r], sc[nt][mt][2 * r + 1]));
      }
      // O^T: row tile i holds channels (D / 8) g + 2 i (rows 0-7) and + 1 (rows 8-15)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t sel = u ? 0x7362u : 0x5140u;
            const uint32_t x0 = prmt(vf[mt][0][0][w], vf[mt][0][1][w], sel);
            const uint32_t x1 = prmt(vf[mt][1][0][w], vf[mt][1][1][w], sel);
            const uint32_t a0 = e4m3x2_to_f16x2(x0 & 0xFFFFu), a1 = e4m3x2_to_f16x2(x0 >> 16);
            const uint32_t a2 = e4m3x2_to_f16x2(x1 & 0xFFFFu), a3 = e4m3x2_to_f16x2(x1 >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16_16816(o[nt][2 * w + u], a0, a1, a2, a3, pb[nt][mt][0], pb[nt][mt][1]);
          }
    }
  }

  // the warps' parts, then the cluster's, joined in a fixed order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float ls = l[nt][c];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      const int head = 8 * nt + 2 * t4 + c;
      if (g == 0) part_m[warp][head] = m[nt][c], part_l[warp][head] = ls;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<float2*>(&part_o[warp][head][(D / 8) * g + 2 * i]) = make_float2(o[nt][i][c], o[nt][i][2 + c]);
    }
  __syncthreads();
  if (ranks > 1) {
    // this CTA's warps into warp 0's place
    float acc[8 * NT * D / (AR_WARPS * 32)];
    float mm = 0.0f, ll = 0.0f;
#pragma unroll
    for (int j = 0; j < 8 * NT * D / (AR_WARPS * 32); ++j) {
      const int i = threadIdx.x + j * AR_WARPS * 32, head = i / D, c = i % D;
      float M = -INFINITY, v = 0.0f;
#pragma unroll
      for (int w = 0; w < AR_WARPS; ++w) M = fmaxf(M, part_m[w][head]);
      const float b = M > -INFINITY ? M : 0.0f;
#pragma unroll
      for (int w = 0; w < AR_WARPS; ++w) v = fmaf(ex2(part_m[w][head] - b), part_o[w][head][c], v);
      acc[j] = v;
    }
    if (threadIdx.x < 8 * NT) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < AR_WARPS; ++w) M = fmaxf(M, part_m[w][threadIdx.x]);
      const float b = M > -INFINITY ? M : 0.0f;
#pragma unroll
      for (int w = 0; w < AR_WARPS; ++w) ll += scale_sum(part_l[w][threadIdx.x], part_m[w][threadIdx.x] - b);
      mm = M;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8 * NT * D / (AR_WARPS * 32); ++j) (&part_o[0][0][0])[threadIdx.x + j * AR_WARPS * 32] = acc[j];
    if (threadIdx.x < 8 * NT) part_m[0][threadIdx.x] = mm, part_l[0][threadIdx.x] = ll;
    cluster_sync_all();
  }
  const int parts = ranks > 1 ? ranks : AR_WARPS;
  for (int i = rank * AR_WARPS * 32 + threadIdx.x; i < a.G * D; i += ranks * AR_WARPS * 32) {
    const int head = i / D, c = i % D;
    float M = -INFINITY, v = 0.0f, z = 0.0f;
    auto at = [&](const float* own, const float* local, int j) { return ranks > 1 ? ld_cluster_f32(local, j) : *own; };
    for (int j = 0; j < parts; ++j) M = fmaxf(M, at(&part_m[j & 3][head], &part_m[0][head], j));
    const float b = M > -INFINITY ? M : 0.0f;
    for (int j = 0; j < parts; ++j) {
      const float d = at(&part_m[j & 3][head], &part_m[0][head], j) - b;
      v = fmaf(ex2(d), at(&part_o[j & 3][head][c], &part_o[0][head][c], j), v);
      z += scale_sum(at(&part_l[j & 3][head], &part_l[0][head], j), d);
    }
    const size_t r = (size_t)row * a.G + head;
    a.out[r * D + c] = (uint16_t)f32_to_bf16_rne(z == 0.0f ? 0.0f : v / z);
    if (c == 0 && a.lse) a.lse[r] = z == 0.0f ? -INFINITY : LN2 * (b - P_SHIFT + log2f(z));
  }
  if (ranks > 1) cluster_sync_all();   // no CTA leaves while another reads its parts
}

}  // namespace

cudaError_t launch_kv_attend(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* q, long long q_stride, int Hq,
                             const int32_t* ids, int k, float scale, uint16_t* out, float* lse, int32_t* err, cudaStream_t s) {
  const int H = c->n_kv_heads, D = c->head_dim, G = Hq / H;
  const AttendArgs a{static_cast<const uint8_t*>(c->pages), H,     G,     KvTable{tk.table, tk.B, tk.N, c->n_pages},
                     q, q_stride, tk.seq, tk.pos, tk.T, ids, k, scale, out, lse, err, 0};
  // Tiles of 128 rows pay where neighbours share their blocks (16 tokens on average for each of the table's sequences,
  // whether the call has tokens of all of them or not) and where there are enough of them: a tile takes its 50 to 70 us
  // (16 blocks a token, G = 8 or 16) however few there are.  Four kv heads, 16 of 256 blocks, us by token / by
  // tile: G = 8, D = 128: 256 tokens 43 / 71, 512 82 / 75, 1,024 154 / 98, 8,192 1,195 / 544; G = 8, D = 64: 512
  // 49 / 68, 1,024 91 / 84; G = 16, D = 64: 256 39 / 48, 512 73 / 58; G = 4, D = 128: 512 72 / 127, 1,024 134 / 137,
  // 2,048 262 / 167; G = 2 (64 tokens a tile, whose lists differ more), D = 64: 1,024 76 / 161, 2,048 147 / 171, 4,096
  // 290 / 194; G = 1, D = 64: 4,096 284 / 239.  At the rule's edges it takes the slower kernel for G = 8, D = 64 (512
  // tokens) and G = 2, D = 64 (2,048).
  const long long pairs = (long long)tk.T * H;
  if (tk.T >= 16LL * tk.B && pairs >= 2048 && pairs * G >= 16384) return launch_kv_attend_tiles(a, D, s);
  // CTAs of a (token, head): halves of blocks for every warp, as long as the GPU has room for them
  const long long rows = (long long)tk.T * H;
  const long long room = (long long)ar_ctas(D, G > 8 ? 2 : 1) * device_sm_count();
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * AR_WARPS <= 2 * k && rows * ranks * 2 <= room) ranks *= 2;
  auto kern = D == 128 ? (G > 8 ? kv_attend_rows_kernel<128, 2> : kv_attend_rows_kernel<128, 1>)
                       : (G > 8 ? kv_attend_rows_kernel<64, 2> : kv_attend_rows_kernel<64, 1>);
  return launch_kc(kern, dim3((unsigned)(rows * ranks)), dim3(AR_WARPS * 32), ranks, 0, s, a);
}

}  // namespace bre

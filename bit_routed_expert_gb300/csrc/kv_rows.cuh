// A token's query heads of one kv head against 32 cached tokens at a time, by a warp: what the attention kernels for single
// tokens share.
//
// S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16 (FP16 operands, FP32 sums): tokens or channels are the 16 rows, eight
// query heads the 8 columns, so no tensor-core row is padding for G = 8 or 16.  The cache's codes go from memory to the
// fragments without shared memory: the 16 channels (K) or the four tokens' 16 channels (V) that a lane loads are the ones
// its fragment rows need, because the order of a contraction and the numbering of the output channels are free.
// E4M3 -> FP16 is exact.  A key's scale multiplies its logit.  A value's scale 2^ev is put into the weight: with s' = s + ev
// in the log2 domain and the running maximum M taken over s', the weights 2^(s' - M) are at most 1 whatever the values'
// scales, and the sum of exponentials gets back the factor 2^-ev.
#pragma once
#include "kv_attend.cuh"

namespace bre {

constexpr int AR_WARPS = 4;

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// CTAs to an SM.  The loads of a half block are all issued before its first product, so warps are what keeps
// memory busy: 64 tokens x 32 blocks take 41 us with three CTAs, 30 with four, 47 with five (spills).  Both halves of 16 heads at D = 128 need the registers of two.
constexpr int ar_ctas(int D, int NT) { return NT == 1 || D == 64 ? 4 : 2; }

// NT: groups of eight query heads.  ODD_IS_NAN: a head whose query holds a NaN or an infinity gives NaN.
template <int D, int NT, bool ODD_IS_NAN>
struct Rows {
  static constexpr int HB = D / 64;   // 64-channel halves of a key row
  static constexpr int MT = D / 16;   // 16-channel row tiles of O^T
  static constexpr int VW = D / 32;   // 4-channel words of a value row that a lane holds

  // the query's fragments: B of S^T, head 8 nt + g, channels 64 hb + 16 t4 + 4 i + {0, 1}, {2, 3}
  uint32_t qf[NT][HB][4][2];
  float qs[NT][2];   // logit factors of heads 8 nt + 2 t4, + 1 (the columns of this lane's sums)
  float o[NT][MT][4], m[NT][2], l[NT][2];
  bool large;        // a value scale above EV_LARGE has been met

  // q: the first of the G heads
  __device__ __forceinline__ Rows(const uint16_t* q, int G, float scale) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[HB * 16], amax = 0.0f;
      const bool live = 8 * nt + g < G;
      const uint16_t* qr = q + (size_t)(8 * nt + g) * D + 16 * t4;
      bool odd = false;   // a value that is no number
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
      for (int i = 0; i < HB * 16; ++i) {
        amax = fmaxf(amax, fminf(fabsf(x[i]), KV_MAX));
        if (ODD_IS_NAN) odd |= !(fabsf(x[i]) < INFINITY);
      }
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
      float f = scale * LOG2E * pow2f(e);
      if (ODD_IS_NAN) {
        const uint32_t any = __ballot_sync(0xffffffffu, odd);
        if (any >> (lane & 28) & 15u) f = __int_as_float(0x7FC00000);
      }
      qs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
      qs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.0f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }
    large = false;
  }

  // 32 tokens: pg their key rows (their values KV_BLOCK rows on), ps their key scales, seen(x) whether token x counts.
  template <typename Seen>
  __device__ __forceinline__ void add(const uint8_t* pg, const uint8_t* ps, Seen seen) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    // loads: key rows 16 mt + 8 r + g; value rows 16 mt + 8 r + 2 t4 + c; rows that are not seen
    // are not read (whatever they hold must not reach a product)
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
          kf[mt][r][hb] = seen(x) ? __ldg(reinterpret_cast<const uint4*>(pg + x * D + 64 * hb) + t4)
                                : make_uint4(0, 0, 0, 0);
        ek[mt][r] = seen(x) ? (int)__ldg(ps + x) : 127;
        ev[mt][r] = seen(x) ? (int)__ldg(ps + KV_BLOCK + x) : 127;
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
            const uint4 w = seen(x) ? __ldg(reinterpret_cast<const uint4*>(vr)) : make_uint4(0, 0, 0, 0);
            vf[mt][r][c][0] = w.x, vf[mt][r][c][1] = w.y;
            vf[mt][r][c][VW - 2] = w.z, vf[mt][r][c][VW - 1] = w.w;
          } else {
            const uint2 w = seen(x) ? __ldg(reinterpret_cast<const uint2*>(vr)) : make_uint2(0, 0);
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
            v = seen(16 * mt + 8 * r + g) ? fmaf(v * qs[nt][c], kf2[mt][r], evf[mt][r]) : -INFINITY;
            mx[c] = fmaxf(mx[c], v);
          }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
        mx[c] = fmaxf(mx[c], m[nt][c]);
        const float base_m = mx[c] > -INFINITY ? weights_base(mx[c]) : 0.0f;   // NaN logits have no maximum
        const float lower = weights_base(m[nt][c]) - base_m;
        const float r0 = ex2(lower);
        l[nt][c] = scale_sum(l[nt][c], lower);
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
};

}  // namespace bre

// Attention over the listed blocks of the quantised cache.
#include "kv_common.cuh"

namespace bre {

namespace {

// One CTA of D threads per (token, kv head): block by block, the G x 64 logits into shared memory,
// then every thread adds its channel's values with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(128)
    kv_attend_kernel(const uint8_t* __restrict__ pages, int H, int G, KvTable tab, const uint16_t* __restrict__ q,
                     long long q_stride, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos,
                     const int32_t* __restrict__ ids, int k, float scale, uint16_t* __restrict__ out,
                     float* __restrict__ lse, int32_t* err) {
  __shared__ float qs[16][D];
  __shared__ float lg[16][KV_BLOCK];
  pdl_wait();
  const int t = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x;
  const int p = __ldg(pos + t), s = __ldg(seq + t);
  for (int i = tid; i < G * D; i += D) qs[i / D][i % D] = bf16_bits_to_f32(q[t * q_stride + (size_t)h * G * D + i]);
  float m[16], l[16], o[16];
#pragma unroll
  for (int g = 0; g < 16; ++g) m[g] = -INFINITY, l[g] = 0.0f, o[g] = 0.0f;
  __syncthreads();
  for (int j = 0; j < k; ++j) {
    const int b = __ldg(ids + ((size_t)t * H + h) * k + j);
    if (b < 0 || p < 0 || (long long)b * KV_BLOCK > p) continue;
    const int page = kv_page(tab, s, b, err);
    if (page < 0) continue;
    const uint8_t* pg = pages + ((size_t)page * H + h) * kv_page_bytes(D);
    const int n = min(KV_BLOCK, p - b * KV_BLOCK + 1);
    for (int i = tid; i < G * KV_BLOCK; i += D) {
      const int g = i / KV_BLOCK, x = i % KV_BLOCK;
      float acc = 0.0f;
      if (x < n)
        for (int c = 0; c < D; c += 2) {
          const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(pg + x * D + c)));
          acc = fmaf(f.x, qs[g][c], fmaf(f.y, qs[g][c + 1], acc));
        }
      lg[g][x] = x < n ? acc * pow2f((int)pg[2 * KV_BLOCK * D + x] - 127) * scale : -INFINITY;
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 16; ++g) {
      if (g >= G) break;
      float nm = m[g];
      for (int x = 0; x < n; ++x) nm = fmaxf(nm, lg[g][x]);
      const float base = nm > -INFINITY ? nm : 0.0f;   // a row of NaN logits has no maximum
      const float r = __expf(m[g] - base);
      l[g] *= r;
      o[g] *= r;
      for (int x = 0; x < n; ++x) {
        const float w = __expf(lg[g][x] - base);
        const float v = f16x2_to_f32x2(e4m3x2_to_f16x2(pg[KV_BLOCK * D + x * D + tid])).x;
        l[g] += w;
        o[g] = fmaf(w, v * pow2f((int)pg[2 * KV_BLOCK * D + KV_BLOCK + x] - 127), o[g]);
      }
      m[g] = nm;
    }
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < 16; ++g) {
    if (g >= G) break;
    const size_t row = ((size_t)t * H + h) * G + g;
    out[row * D + tid] = (uint16_t)f32_to_bf16_rne(l[g] == 0.0f ? 0.0f : o[g] / l[g]);
    if (tid == 0 && lse) lse[row] = l[g] == 0.0f ? -INFINITY : m[g] + logf(l[g]);
  }
}

}  // namespace

size_t kv_attend_ws_bytes(int T, int Hq, int H, int D, int B, int k) { return 0; }

cudaError_t launch_kv_attend(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* q, long long q_stride, int Hq,
                             const int32_t* ids, int k, float scale, uint16_t* out, float* lse, void* ws, int32_t* err,
                             cudaStream_t s) {
  const int H = c->n_kv_heads, D = c->head_dim;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = D == 128 ? kv_attend_kernel<128> : kv_attend_kernel<64>;
  return launch_k(kern, dim3((unsigned)tk.T * H), dim3(D), 0, s, static_cast<const uint8_t*>(c->pages), H, Hq / H, tab,
                  q, q_stride, tk.seq, tk.pos, ids, k, scale, out, lse, err);
}

}  // namespace bre

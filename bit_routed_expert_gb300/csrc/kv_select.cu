// Block selection for sparse attention: every visible block's score against a query's heads, and
// the best blocks in ascending order.
#include "kv_common.cuh"

namespace bre {

namespace {

// One CTA per (token, kv head).  Scores are sums of whole numbers below 2^24 (exact in FP32) times
// powers of two, so any order of the sum gives the same bits.
template <int D>
__global__ void __launch_bounds__(128)
    kv_select_kernel(const int8_t* __restrict__ bounds, const int8_t* __restrict__ bexp, int H, int G, KvTable tab,
                     const uint16_t* __restrict__ q, long long q_stride, const int32_t* __restrict__ seq,
                     const int32_t* __restrict__ pos, int k, int n_sink, int n_local, int32_t* __restrict__ ids,
                     float* __restrict__ scores, float* __restrict__ ws, int32_t* err) {
  __shared__ int u[2 * D];
  __shared__ float red[4];
  __shared__ int redi[4];
  pdl_wait();
  const int t = blockIdx.x / H, h = blockIdx.x % H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int p = __ldg(pos + t), s = __ldg(seq + t);
  int32_t* oid = ids + ((size_t)t * H + h) * k;
  float* osc = scores ? scores + ((size_t)t * H + h) * k : nullptr;
  const bool ok = p >= 0 && (unsigned)s < (unsigned)tab.B;
  if (p >= 0 && !ok && tid == 0) set_err(err, BRE_DEVERR_PAGE);
  const uint16_t* qr = q + t * q_stride + (size_t)h * G * D;
  float a = 0.0f;
  for (int i = tid; i < G * D; i += 128) a = fmaxf(a, fabsf(kv_clamp(bf16_bits_to_f32(qr[i]))));
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (lane == 0) red[warp] = a;
  __syncthreads();
  const int eq = query_exp(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  for (int c = tid; c < D; c += 128) {
    int plus = 0, minus = 0;
    for (int g = 0; g < G; ++g) {
      const float x = kv_clamp(bf16_bits_to_f32(qr[g * D + c]));
      const int code = x == x ? (int)rintf(x * pow2f(-eq)) : 0;
      plus += max(code, 0);
      minus += max(-code, 0);
    }
    u[c] = plus;
    u[D + c] = -minus;
  }
  __syncthreads();
  const int nb = ok ? min(p / KV_BLOCK + 1, tab.N) : 0;
  if (ok && p / KV_BLOCK >= tab.N && tid == 0) set_err(err, BRE_DEVERR_PAGE);
  float* sc = ws + (size_t)blockIdx.x * tab.N * 2;
  float* key = sc + tab.N;
  for (int b = warp; b < nb; b += 4) {
    const int page = kv_page(tab, s, b, err);
    float f = 0.0f;
    if (page >= 0) {
      const size_t ph = (size_t)page * H + h;
      int dot = 0;
      for (int c = lane; c < 2 * D; c += 32) dot += u[c] * (int)bounds[ph * 2 * D + c];
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      f = (float)dot * pow2f(bexp[ph]);
    }
    if (lane == 0) {
      const bool must = b < n_sink || b > p / KV_BLOCK - n_local;
      sc[b] = f;
      key[b] = page < 0 ? -INFINITY : must ? INFINITY : f;
    }
  }
  __syncthreads();
  // the best left, k times; then in ascending order
  __shared__ int sel[256];
  __shared__ int nsel;
  if (tid == 0) nsel = 0;
  for (int j = 0; j < k; ++j) {
    float bf = -INFINITY;
    int bi = 0x7fffffff;
    for (int b = tid; b < nb; b += 128) {
      const float f = key[b];
      if (f > bf) bf = f, bi = b;
    }
    for (int o = 16; o; o >>= 1) {
      const float of = __shfl_xor_sync(0xffffffffu, bf, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (of > bf || (of == bf && oi < bi)) bf = of, bi = oi;
    }
    if (lane == 0) red[warp] = bf, redi[warp] = bi;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < 4; ++w)
        if (red[w] > bf || (red[w] == bf && redi[w] < bi)) bf = red[w], bi = redi[w];
      if (bf > -INFINITY) {
        sel[nsel++] = bi;
        key[bi] = -INFINITY;
      }
    }
    __syncthreads();
  }
  for (int j = tid; j < k; j += 128) {
    if (j >= nsel) {
      oid[j] = -1;
      if (osc) osc[j] = 0.0f;
    } else {
      int rank = 0;
      for (int i = 0; i < nsel; ++i) rank += sel[i] < sel[j];
      oid[rank] = sel[j];
      if (osc) osc[rank] = sc[sel[j]] * pow2f(eq);
    }
  }
}

}  // namespace

size_t kv_select_ws_bytes(int T, int Hq, int H, int D, int B, int N, int k) { return (size_t)T * H * N * 8; }

cudaError_t launch_kv_select(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* q, long long q_stride, int Hq,
                             int k, int n_sink, int n_local, int32_t* ids, float* scores, void* ws, int32_t* err,
                             cudaStream_t s) {
  const int H = c->n_kv_heads;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_select_kernel<128> : kv_select_kernel<64>;
  return launch_k(kern, dim3((unsigned)tk.T * H), dim3(128), 0, s, (const int8_t*)c->bounds,
                  (const int8_t*)c->bound_exp, H, Hq / H, tab, q, q_stride, tk.seq, tk.pos, k, n_sink, n_local, ids,
                  scores, static_cast<float*>(ws), err);
}

}  // namespace bre

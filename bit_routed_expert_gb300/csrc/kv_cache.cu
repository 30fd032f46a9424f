// Writing keys and values into the quantised paged cache, and reading them back.
#include "kv_common.cuh"

namespace bre {

namespace {

// One warp per (token, head).  The warp whose token opens a run (the tokens in a row of one
// block) stores the whole run and, for the keys, the block's channel-wise extremes.
template <int D>
__global__ void __launch_bounds__(128)
    kv_append_kernel(uint8_t* pages, int8_t* bounds, int8_t* bexp, int H, KvTable tab, const uint16_t* __restrict__ k,
                     const uint16_t* __restrict__ v, long long k_stride, long long v_stride,
                     const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, int T, int32_t* err) {
  constexpr int PL = D / 32;   // channels a lane holds
  pdl_wait();
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int t0 = w / H, h = w % H;
  if (t0 >= T) return;
  const int s = __ldg(seq + t0), p0 = __ldg(pos + t0);
  if (p0 < 0) return;
  const int blk = p0 / KV_BLOCK;
  auto in_run = [&](int t) {
    const int p = __ldg(pos + t);
    return __ldg(seq + t) == s && p >= 0 && p / KV_BLOCK == blk;
  };
  if (t0 > 0 && in_run(t0 - 1)) return;
  const int page = kv_page(tab, s, blk, err);
  if (page < 0) {
    set_err(err, BRE_DEVERR_PAGE);   // a token to store needs a page
    return;
  }
  const size_t ph = (size_t)page * H + h;
  uint8_t* pg = pages + ph * kv_page_bytes(D);
  float hi[PL], lo[PL], amax = 0.0f;
  for (int t = t0; t < T && in_run(t); ++t) {
    const int slot = __ldg(pos + t) % KV_BLOCK;
    for (int kv = 0; kv < 2; ++kv) {
      const uint16_t* row = kv ? v + t * v_stride : k + t * k_stride;
      float x[PL], a = 0.0f;
      bool nan = false;
      for (int i = 0; i < PL; ++i) {
        x[i] = kv_clamp(bf16_bits_to_f32(row[h * D + lane * PL + i]));
        nan |= x[i] != x[i];
        a = fmaxf(a, fabsf(x[i]));
      }
      for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      nan = __any_sync(0xffffffffu, nan);
      if (nan)
        for (int i = 0; i < PL; ++i) x[i] = 0.0f;
      const int e = row_exp(a);
      uint8_t* dst = pg + kv * KV_BLOCK * D + slot * D + lane * PL;
      for (int i = 0; i < PL; i += 2) {
        const uint32_t c = e4m3x2(x[i] * pow2f(-e), x[i + 1] * pow2f(-e));
        *reinterpret_cast<uint16_t*>(dst + i) = (uint16_t)c;
        if (kv == 0) {
          const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(c));
          const float y[2] = {f.x * pow2f(e), f.y * pow2f(e)};
          for (int j = 0; j < 2; ++j) {
            hi[i + j] = t == t0 ? y[j] : fmaxf(hi[i + j], y[j]);
            lo[i + j] = t == t0 ? y[j] : fminf(lo[i + j], y[j]);
            amax = fmaxf(amax, fabsf(y[j]));
          }
        }
      }
      if (lane == 0) pg[2 * KV_BLOCK * D + kv * KV_BLOCK + slot] = (uint8_t)(nan ? KV_NAN : e + 127);
    }
  }
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  int e = bound_exp_of(amax);
  int8_t* bd = bounds + ph * 2 * D + lane * PL;
  if (p0 % KV_BLOCK) {   // the block had begun before this call
    const int oe = bexp[ph];
    for (int i = 0; i < PL; ++i) {
      hi[i] = fmaxf(hi[i], bd[i] * pow2f(oe));
      lo[i] = fminf(lo[i], bd[D + i] * pow2f(oe));
    }
    e = max(e, oe);
  }
  __syncwarp();
  for (int i = 0; i < PL; ++i) {
    bd[i] = (int8_t)ceilf(hi[i] * pow2f(-e));
    bd[D + i] = (int8_t)floorf(lo[i] * pow2f(-e));
  }
  if (lane == 0) bexp[ph] = (int8_t)e;
}

// One warp per (token, head): codes times the row's scale, exact in BF16.
template <int D>
__global__ void __launch_bounds__(128)
    kv_read_kernel(const uint8_t* __restrict__ pages, int H, KvTable tab, const int32_t* __restrict__ seq,
                   const int32_t* __restrict__ pos, int T, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                   int32_t* err) {
  constexpr int PL = D / 32;
  pdl_wait();
  const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int t = w / H, h = w % H;
  if (t >= T) return;
  const int p = __ldg(pos + t);
  const int page = p < 0 ? -1 : kv_page(tab, __ldg(seq + t), p / KV_BLOCK, err);
  if (p >= 0 && page < 0) set_err(err, BRE_DEVERR_PAGE);
  const uint8_t* pg = pages + ((size_t)max(page, 0) * H + h) * kv_page_bytes(D);
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? v : k;
    if (!out) continue;
    const int slot = p % KV_BLOCK;
    for (int i = 0; i < PL; ++i) {
      float f = 0.0f;
      if (page >= 0)
        f = f16x2_to_f32x2(e4m3x2_to_f16x2(pg[kv * KV_BLOCK * D + slot * D + lane * PL + i])).x *
            pow2f((int)pg[2 * KV_BLOCK * D + kv * KV_BLOCK + slot] - 127);
      out[((size_t)t * H + h) * D + lane * PL + i] = (uint16_t)f32_to_bf16_rne(f);
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* k, const uint16_t* v,
                             long long k_stride, long long v_stride, int32_t* err, cudaStream_t s) {
  const int H = c->n_kv_heads;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<64>;
  return launch_k(kern, dim3((unsigned)(((long long)tk.T * H + 3) / 4)), dim3(128), 0, s,
                  static_cast<uint8_t*>(c->pages), c->bounds, c->bound_exp, H, tab, k, v, k_stride, v_stride, tk.seq,
                  tk.pos, tk.T, err);
}

cudaError_t launch_kv_read(const bre_kv_cache* c, const KvTokens& tk, uint16_t* k, uint16_t* v, int32_t* err,
                           cudaStream_t s) {
  const int H = c->n_kv_heads;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_read_kernel<128> : kv_read_kernel<64>;
  return launch_k(kern, dim3((unsigned)(((long long)tk.T * H + 3) / 4)), dim3(128), 0, s,
                  static_cast<const uint8_t*>(c->pages), H, tab, tk.seq, tk.pos, tk.T, k, v, err);
}

}  // namespace bre

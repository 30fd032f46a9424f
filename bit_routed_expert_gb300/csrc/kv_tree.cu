// Attention over the whole cached context and a tree of drafted tokens behind it.
#include "kv_attend.cuh"

namespace bre {

namespace {

// Bit x - 64 blk set: the token sees slot x (of the 64 of a block).
__device__ __forceinline__ uint64_t seen_bits(const uint64_t* __restrict__ mask, int words, int start, int pos, int blk) {
  const long long x0 = (long long)blk * KV_BLOCK;
  uint64_t own = pos >= x0 + 63 ? ~0ull : pos >= x0 ? (2ull << (pos - x0)) - 1ull : 0ull;
  if (!mask || own == 0) return own;
  const long long j = x0 - start;   // bit of the block's first slot
  uint64_t tree = 0;
  if (j < 0) {
    if (j <= -64) return own;
    tree = (1ull << -j) - 1ull | __ldg(mask) << -j;
  } else {
    const long long w = j / 64;
    const int r = (int)(j % 64);
    if (w < words) tree = __ldg(mask + w) >> r;
    if (r && w + 1 < words) tree |= __ldg(mask + w + 1) << (64 - r);
  }
  return own & tree;
}

// A warp a query head of a token: the plain order of the formula, one key after the other.
constexpr int TR_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(TR_WARPS * 32)
    kv_tree_rows_kernel(const uint8_t* __restrict__ pages, int H, KvTable tab, const uint16_t* __restrict__ q, long long q_stride,
                        int Hq, const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, int T,
                        const int32_t* __restrict__ start, const uint64_t* __restrict__ mask, int words, float scale,
                        uint16_t* __restrict__ out, float* __restrict__ lse, int32_t* err) {
  constexpr int CL = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * TR_WARPS + (threadIdx.x >> 5);
  if (row >= (long long)T * Hq) return;
  const int t = (int)(row / Hq), head = (int)(row % Hq), h = head / (Hq / H);
  const int p = __ldg(pos + t), s = __ldg(seq + t);
  float x[CL], o[CL], m = -INFINITY, l = 0.0f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < CL; ++i) {
    x[i] = bf16_bits_to_f32(__ldg(q + t * q_stride + (long long)head * D + lane * CL + i));
    odd |= !(fabsf(x[i]) < INFINITY);
    o[i] = 0.0f;
  }
  odd = __any_sync(0xffffffffu, odd);
  const int begin = start && (unsigned)s < (unsigned)tab.B ? max(__ldg(start + s), 0) : 0;
  bool nan = false, some = false;
  if (p >= 0 && p / KV_BLOCK >= tab.N) set_err(err, BRE_DEVERR_PAGE);
  for (int blk = 0; p >= 0 && blk <= p / KV_BLOCK && blk < tab.N; ++blk) {
    const uint64_t bits = seen_bits(mask ? mask + (size_t)t * words : nullptr, words, begin, p, blk);
    const int page = kv_page(tab, s, blk, err);
    if (page < 0) continue;
    const uint8_t* pg = pages + ((size_t)page * H + h) * kv_page_bytes(D);
    some |= bits != 0;
    for (uint64_t todo = bits; todo; todo &= todo - 1) {
      const int at = __ffsll((long long)todo) - 1;
      const int ek = pg[2 * KV_BLOCK * D + at], ev = pg[2 * KV_BLOCK * D + KV_BLOCK + at];
      nan |= ek == KV_NAN || ev == KV_NAN;
      if (nan) break;
      float dot = 0.0f, v[CL];
#pragma unroll
      for (int i = 0; i < CL; i += 2) {
        const uint32_t kc = *reinterpret_cast<const uint16_t*>(pg + at * D + lane * CL + i);
        const uint32_t vc = *reinterpret_cast<const uint16_t*>(pg + KV_BLOCK * D + at * D + lane * CL + i);
        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(kc)), g = f16x2_to_f32x2(e4m3x2_to_f16x2(vc));
        dot = fmaf(x[i], f.x, fmaf(x[i + 1], f.y, dot));
        v[i] = g.x * pow2f(ev - 127 - 24), v[i + 1] = g.y * pow2f(ev - 127 - 24);   // (sums of the largest values fit)
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
      const float logit = dot * pow2f(ek - 127) * scale, nm = fmaxf(m, logit);
      const float keep = expf(m - nm), w = expf(logit - nm);
      m = nm;
      l = fmaf(l, keep, w);
#pragma unroll
      for (int i = 0; i < CL; ++i) o[i] = fmaf(o[i], keep, w * v[i]);
    }
  }
  nan |= odd && some;
#pragma unroll
  for (int i = 0; i < CL; ++i)
    out[row * D + lane * CL + i] = (uint16_t)(nan ? 0x7FC0u : f32_to_bf16_rne(l > 0.0f ? o[i] / l * 0x1p24f : 0.0f));
  if (lane == 0 && lse) lse[row] = nan ? __int_as_float(0x7FC00000) : l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv_tree_ws_bytes(int, int, int, int) { return 0; }

cudaError_t launch_kv_attend_tree(const TreeArgs& a, cudaStream_t s) {
  const bre_kv_cache* c = a.cache;
  const KvTable tab{a.tk.table, a.tk.B, a.tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_tree_rows_kernel<128> : kv_tree_rows_kernel<64>;
  const long long rows = (long long)a.tk.T * a.Hq;
  return launch_k(kern, dim3((unsigned)((rows + TR_WARPS - 1) / TR_WARPS)), dim3(TR_WARPS * 32), 0, s,
                  static_cast<const uint8_t*>(c->pages), c->n_kv_heads, tab, a.q, a.q_stride, a.Hq, a.tk.seq, a.tk.pos, a.tk.T,
                  a.start, a.mask, a.words, a.scale, a.out, a.lse, a.err);
}

}  // namespace bre

// Attention over the listed blocks of the quantised cache.
#include "kv_rows.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// A token's heads at a time: decode and verify batches
// ---------------------------------------------------------------------------
// A cluster of CTAs per (token, kv head); the listed blocks are dealt to its warps in halves of 32
// tokens (kv_rows.cuh).
// NT: groups of eight query heads.
template <int D, int NT>
__global__ void __launch_bounds__(AR_WARPS * 32, ar_ctas(D, NT)) kv_attend_rows_kernel(const AttendArgs a) {
  constexpr int MT = D / 16;       // 16-channel row tiles of O^T
  constexpr int PB = kv_page_bytes(D);
  __shared__ __align__(8) float part_o[AR_WARPS][8 * NT][D];
  __shared__ float part_m[AR_WARPS][8 * NT], part_l[AR_WARPS][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int rank = (int)cluster_ctarank(), ranks = (int)cluster_nctarank();
  const int row = blockIdx.x / ranks, t = row / a.H, h = row - t * a.H;
  pdl_wait();
  pdl_launch_dependents();
  const int p = __ldg(a.pos + t), s = __ldg(a.seq + t);

  Rows<D, NT, false> rows(a.q + t * a.q_stride + (size_t)h * a.G * D, a.G, a.scale);
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
      rows.add(pg, ps, [n](int x) { return x < n; });
    }
  }

  // the warps' parts, then the cluster's, joined in a fixed order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float ls = rows.l[nt][c];
#pragma unroll
      for (int d = 4; d < 32; d *= 2) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      const int head = 8 * nt + 2 * t4 + c;
      if (g == 0) part_m[warp][head] = rows.m[nt][c], part_l[warp][head] = ls;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<float2*>(&part_o[warp][head][(D / 8) * g + 2 * i]) = make_float2(rows.o[nt][i][c], rows.o[nt][i][2 + c]);
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

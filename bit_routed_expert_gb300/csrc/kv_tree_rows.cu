// Attention over the whole cached context for single tokens: a token's heads at a time.
#include "kv_rows.cuh"
#include "kv_tree.cuh"

namespace bre {

namespace {

// A CTA per (token, kv head) and share of the token's context.  The warps take its halves of blocks in turn (kv_rows.cuh); their
// parts are joined in shared memory, and where a context has several shares a second kernel joins these.
// Bound: DRAM where the call is large (64 sequences of 16,384 tokens, four kv heads of 128, 1.08 GB: 181 us, 6.0 TB/s, 0.88 of a
// plain copy's), else two launches and a chain of page lookup, half a block, two joins (one token over 8,192, 8.5 MB: 9.7 us).
struct TreeRows {
  const uint8_t* pages;
  int H, G, shares;
  KvTable tab;
  const uint16_t* q;
  long long q_stride;
  const int32_t* seq;
  const int32_t* pos;
  const int32_t* start;
  const uint64_t* mask;
  int words;
  float scale;
  uint16_t* out;
  float* lse;
  int32_t* err;
  float2* ml;    // [(token, kv head)][shares][G]: maximum and sum
  float* part;   // [(token, kv head)][shares][G][D]
};

template <int D, int NT>
__global__ void __launch_bounds__(AR_WARPS * 32, ar_ctas(D, NT)) kv_tree_rows_kernel(const TreeRows a) {
  constexpr int MT = D / 16, PB = kv_page_bytes(D);
  __shared__ __align__(8) float part_o[AR_WARPS][8 * NT][D];
  __shared__ float part_m[AR_WARPS][8 * NT], part_l[AR_WARPS][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int share = blockIdx.x % a.shares, row = blockIdx.x / a.shares, t = row / a.H, h = row - t * a.H;
  pdl_wait();
  pdl_launch_dependents();
  const int p = __ldg(a.pos + t), s = __ldg(a.seq + t);
  if (p >= 0 && p / KV_BLOCK >= a.tab.N && share == 0 && threadIdx.x == 0) set_err(a.err, BRE_DEVERR_PAGE);
  const int begin = a.start && (unsigned)s < (unsigned)a.tab.B ? max(__ldg(a.start + s), 0) : 0;
  const uint64_t* mask = a.mask ? a.mask + (size_t)t * a.words : nullptr;

  Rows<D, NT, true> rows(a.q + t * a.q_stride + (size_t)h * a.G * D, a.G, a.scale);
  // the share's halves of blocks, dealt to the warps in turn
  const int halves = p < 0 ? 0 : min(p / 32 + 1, 2 * a.tab.N);
  const int first = (int)((long long)halves * share / a.shares), last = (int)((long long)halves * (share + 1) / a.shares);
  for (int base = first + warp; base < last; base += 32 * AR_WARPS) {
    // this lane looks up one of the warp's next 32 halves, and which of its tokens count
    const int it = base + lane * AR_WARPS;
    int my_page = -1;
    uint32_t my_bits = 0;
    if (it < last) {
      my_bits = (uint32_t)(seen_bits(mask, a.words, begin, p, it >> 1) >> (32 * (it & 1)));
      my_page = kv_page(a.tab, s, it >> 1, a.err);
      if (my_bits == 0) my_page = -1;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, my_page >= 0); todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      const int page = __shfl_sync(0xffffffffu, my_page, src), half = (base + src * AR_WARPS) & 1;
      const uint32_t bits = __shfl_sync(0xffffffffu, my_bits, src);
      const uint8_t* pg = a.pages + ((size_t)page * a.H + h) * PB;
      rows.add(pg + half * 32 * D, pg + 2 * KV_BLOCK * D + half * 32, [bits](int x) { return (bits >> x & 1u) != 0; });
    }
  }

  // the warps' parts, joined in a fixed order
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
  for (int i = threadIdx.x; i < a.G * D; i += AR_WARPS * 32) {
    const int head = i / D, c = i % D;
    float M = -INFINITY, v = 0.0f, z = 0.0f;
#pragma unroll
    for (int w = 0; w < AR_WARPS; ++w) M = fmaxf(M, part_m[w][head]);
    const float b = M > -INFINITY ? M : 0.0f;
#pragma unroll
    for (int w = 0; w < AR_WARPS; ++w) {
      const float d = part_m[w][head] - b;
      v = fmaf(ex2(d), part_o[w][head][c], v);
      z += scale_sum(part_l[w][head], d);
    }
    if (a.shares > 1) {
      const size_t r = (size_t)blockIdx.x * a.G + head;
      a.part[r * D + c] = v;
      if (c == 0) a.ml[r] = make_float2(M, z);
    } else {
      const size_t r = (size_t)row * a.G + head;
      a.out[r * D + c] = (uint16_t)f32_to_bf16_rne(z == 0.0f ? 0.0f : v / z);
      if (c == 0 && a.lse) a.lse[r] = z == 0.0f ? -INFINITY : LN2 * (b - (M > -INFINITY ? P_SHIFT : 0.0f) + log2f(z));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kv_tree_rows_join_kernel(const TreeRows a, int rows) {
  pdl_wait();
  pdl_launch_dependents();
  join_rows<D>(a.ml, a.part, a.shares, JOIN_WARPS, blockIdx.x, gridDim.x, rows,
               [&](int p, int r) { return ((size_t)(r / a.G) * a.shares + p) * a.G + r % a.G; }, [](int r) { return (size_t)r; }, a.out, a.lse);
}

// CTAs that a call's contexts are shared out to: a few for every place on the GPU, as contexts differ in length.
constexpr int TREE_ROWS_CTAS = 1216;

int most_shares(long long units) { return units >= TREE_ROWS_CTAS ? 1 : (int)(TREE_ROWS_CTAS / units); }

template <int D>
cudaError_t launch(const TreeRows& a, int T, cudaStream_t s) {
  const long long units = (long long)T * a.H;
  auto kern = a.G > 8 ? kv_tree_rows_kernel<D, 2> : kv_tree_rows_kernel<D, 1>;
  const cudaError_t e = launch_k(kern, dim3((unsigned)(units * a.shares)), dim3(AR_WARPS * 32), 0, s, a);
  if (e != cudaSuccess || a.shares == 1) return e;
  const int rows = (int)(units * a.G);   // (of few units, as there are several shares)
  const int at_once = join_at_once(a.shares, JOIN_WARPS);
  return launch_k(kv_tree_rows_join_kernel<D>, dim3((unsigned)((rows + at_once - 1) / at_once)), dim3(JOIN_WARPS * 32), 0, s, a, rows);
}

}  // namespace

// Enough for every call of as many tokens or fewer: these may have more shares in all (whole numbers for each: three tokens of
// four kv heads have 12 x 101, one has 4 x 304), but never more than TREE_ROWS_CTAS.
size_t tree_rows_ws_bytes(int H, int G, int D) {
  return most_shares(H) == 1 ? 0 : (size_t)TREE_ROWS_CTAS * G * (sizeof(float2) + D * sizeof(float));
}

cudaError_t launch_tree_rows(const TreeArgs& t, cudaStream_t s) {
  const bre_kv_cache* c = t.cache;
  const int H = c->n_kv_heads, D = c->head_dim, G = t.Hq / H;
  TreeRows a{};
  a.pages = static_cast<const uint8_t*>(c->pages), a.H = H, a.G = G;
  a.tab = KvTable{t.tk.table, t.tk.B, t.tk.N, c->n_pages};
  a.q = t.q, a.q_stride = t.q_stride, a.seq = t.tk.seq, a.pos = t.tk.pos;
  a.start = t.start, a.mask = t.mask, a.words = t.words, a.scale = t.scale, a.out = t.out, a.lse = t.lse, a.err = t.err;
  // a share has a half block for each warp at least, if the context is as long as the table allows
  const long long units = (long long)t.tk.T * H, most = (2LL * t.tk.N + AR_WARPS - 1) / AR_WARPS;
  a.shares = (int)(most < most_shares(units) ? most : most_shares(units));
  a.part = static_cast<float*>(t.ws);
  a.ml = reinterpret_cast<float2*>(a.part + (size_t)(units * a.shares) * G * D);
  return D == 128 ? launch<128>(a, t.tk.T, s) : launch<64>(a, t.tk.T, s);
}

}  // namespace bre

// Pages of the quantised cache: kept tokens moved together, sequences that share pages, pages given out and taken back.
#include "kv_common.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// Compaction
// ---------------------------------------------------------------------------
// A CTA moves one head's keys (blockIdx.z = 0) or values (1) of one sequence, one target block after the other: all of a
// block's rows are read before any is written, and a row never moves up, so no later block's source is overwritten.
// What lies in the block below `start` stays where it is.  A lane holds 16 codes of a row, so D / 16 lanes hold a row and
// the CTA 32 or 64 rows at a time; the keys pass through registers anyway, so the block's bounds come from there.
constexpr int KC_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(KC_THREADS)
    kv_compact_kernel(uint8_t* pages, int8_t* __restrict__ bounds, int8_t* __restrict__ bexp, int H, KvTable tab,
                      const int32_t* __restrict__ start, const int32_t* __restrict__ nodes, int A,
                      const int32_t* __restrict__ count, int32_t* __restrict__ length, int32_t* err) {
  constexpr int LR = D / 16, RC = KC_THREADS / LR, UN = KV_BLOCK / RC, WARPS = KC_THREADS / 32;
  __shared__ float s_hi[WARPS][D], s_lo[WARPS][D], s_max[WARPS];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = tid % LR;
  const int b = blockIdx.x, h = blockIdx.y, values = blockIdx.z;
  const int n = __ldg(count + b);
  const long long s0 = __ldg(start + b);
  const int32_t* nd = nodes + (size_t)b * A;
  // nothing is moved unless the list ascends and all of its tokens, and the blocks that they move to, have pages
  bool bad = n > A || (n >= 0 && (s0 < 0 || s0 + n > (long long)tab.N * KV_BLOCK));
  if (n >= 0 && !bad) {
    for (int j = tid; j < n; j += KC_THREADS) {
      const int x = __ldg(nd + j), before = j ? __ldg(nd + j - 1) : -1;
      const long long src = s0 + x;
      if (x <= before || src >= (long long)tab.N * KV_BLOCK || kv_page(tab, b, (int)(src / KV_BLOCK), err) < 0) bad = true;
    }
    const long long last = (s0 + n - 1) / KV_BLOCK;
    for (long long k = s0 / KV_BLOCK + tid; k <= last && s0 + n > 0 && k * KV_BLOCK < s0 + n; k += KC_THREADS)
      if (kv_page(tab, b, (int)k, err) < 0) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && h == 0 && values == 0 && length) length[b] = (int)(n >= 0 && !bad ? s0 + n : s0);
  if (bad && tid == 0) set_err(err, BRE_DEVERR_PAGE);
  if (bad || n < 0) return;
  const int end = (int)(s0 + n);
  const size_t PB = kv_page_bytes(D);
  const int row_at = values ? KV_BLOCK * D : 0, scale_at = 2 * KV_BLOCK * D + (values ? KV_BLOCK : 0);
  for (int blk = (int)(s0 / KV_BLOCK); blk * KV_BLOCK < end; ++blk) {
    const int page = __ldg(tab.table + (size_t)b * tab.N + blk);
    uint8_t* dst = pages + ((size_t)page * H + h) * PB;
    uint4 w[UN];
    int sc[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int x = tid / LR + u * RC, p = blk * KV_BLOCK + x;
      sc[u] = -1;
      if (p >= end) continue;
      const int from = p < s0 ? p : (int)(s0 + __ldg(nd + (p - s0)));
      const uint8_t* src = pages + ((size_t)__ldg(tab.table + (size_t)b * tab.N + from / KV_BLOCK) * H + h) * PB;
      w[u] = *(reinterpret_cast<const uint4*>(src + row_at + (from % KV_BLOCK) * D) + lr);
      sc[u] = src[scale_at + from % KV_BLOCK];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int x = tid / LR + u * RC, p = blk * KV_BLOCK + x;
      if (p < s0 || p >= end) continue;
      *(reinterpret_cast<uint4*>(dst + row_at + x * D) + lr) = w[u];
      if (lr == 0) dst[scale_at + x] = (uint8_t)sc[u];
    }
    if (values) continue;
    // bounds from all keys that the block now has (a NaN row, whose codes are zeros, counts as zeros)
    float hi[16], lo[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) hi[c] = -INFINITY, lo[c] = INFINITY;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      if (sc[u] < 0) continue;
      const float up = pow2f(sc[u] == KV_NAN ? 0 : sc[u] - 127);
      const uint32_t c[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(c[i / 2] >> (16 * (i & 1)) & 0xFFFFu));
        hi[2 * i] = fmaxf(hi[2 * i], f.x * up), hi[2 * i + 1] = fmaxf(hi[2 * i + 1], f.y * up);
        lo[2 * i] = fminf(lo[2 * i], f.x * up), lo[2 * i + 1] = fminf(lo[2 * i + 1], f.y * up);
      }
    }
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int o = LR; o < 32; o *= 2) {
        hi[c] = fmaxf(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], o));
        lo[c] = fminf(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], o));
      }
    if (lane < LR)
#pragma unroll
      for (int c = 0; c < 16; ++c) s_hi[warp][lr * 16 + c] = hi[c], s_lo[warp][lr * 16 + c] = lo[c];
    __syncthreads();
    float ch = -INFINITY, cl = INFINITY, amax = 0.0f;
    if (tid < D) {
#pragma unroll
      for (int i = 0; i < WARPS; ++i) ch = fmaxf(ch, s_hi[i][tid]), cl = fminf(cl, s_lo[i][tid]);
      amax = fmaxf(fabsf(ch), fabsf(cl));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) amax = fmaxf(amax, s_max[i]);
    const int e = bound_exp_of(amax);
    const size_t ph = (size_t)page * H + h;
    if (tid < D) {   // (see kv_append for a channel that vanishes in the unit)
      const float down = pow2f(-e), up = ceilf(ch * down), dn = floorf(cl * down);
      bounds[ph * 2 * D + tid] = (int8_t)(ch > 0.0f ? fmaxf(up, 1.0f) : up);
      bounds[ph * 2 * D + D + tid] = (int8_t)(cl < 0.0f ? fminf(dn, -1.0f) : dn);
    }
    if (tid == 0) bexp[ph] = (int8_t)e;
  }
}

// ---------------------------------------------------------------------------
// Forks
// ---------------------------------------------------------------------------
// A CTA takes some columns (blocks) of the table with all of its rows: what a row gets lies in the same columns of another
// row, so the old entries are brought into shared memory and then replaced in place.  References change by atomic sums
// of whole numbers, whose order does not matter, and only where an entry changes.
constexpr int KF_THREADS = 512;

__global__ void __launch_bounds__(KF_THREADS)
    kv_fork_kernel(int n_pages, int32_t* refs, int32_t* table, int B, int N, int width, const int32_t* __restrict__ parent,
                   const int32_t* __restrict__ length, int32_t* err) {
  extern __shared__ int32_t old[];   // [B][width]
  pdl_wait();
  pdl_launch_dependents();
  const int c0 = blockIdx.x * width, nc = min(width, N - c0);
  const int rows = KF_THREADS / width, col = threadIdx.x % width;
  for (int b = threadIdx.x / width; b < B; b += rows)
    if (col < nc) old[b * width + col] = table[(size_t)b * N + c0 + col];
  __syncthreads();
  if (col >= nc) return;
  for (int b = threadIdx.x / width; b < B; b += rows) {
    const int p = __ldg(parent + b), len = __ldg(length + b);
    if (p >= B) {
      set_err(err, BRE_DEVERR_PAGE);
      continue;
    }
    const int was = old[b * width + col];
    int now = p >= 0 && len > 0 && c0 + col <= (len - 1) / KV_BLOCK ? old[p * width + col] : -1;
    if (now >= n_pages) {
      set_err(err, BRE_DEVERR_PAGE);
      now = -1;
    }
    if (now < 0) now = -1;
    if (now == was) continue;
    table[(size_t)b * N + c0 + col] = now;
    if (now >= 0) atomicAdd(refs + now, 1);
    if (was >= 0 && was < n_pages) atomicSub(refs + was, 1);
  }
}

// ---------------------------------------------------------------------------
// Pages given out and taken back
// ---------------------------------------------------------------------------
// Which blocks need a page, and which pages are free, is settled before anything changes, so that the outcome does not go
// by the order of the CTAs: a first kernel marks the blocks and lists the free pages, a second one hands them out.
struct ResizeWs {
  uint32_t* need;     // [B][words]: a bit for each block of the row
  int32_t* before;    // [B + 1]: needs of the rows before
  int32_t* copy;      // [B]: page whose content the row's first needed block gets, or -1
  int32_t* free;      // the lowest free pages, as many as are needed
  int32_t* n_free;    // how many those are
  int words;
};

__host__ __device__ inline size_t round16(size_t n) { return (n + 15) / 16 * 16; }

__host__ __device__ inline ResizeWs resize_ws(void* ws, int B, int N) {
  ResizeWs w;
  w.words = (N + 31) / 32;
  unsigned char* p = static_cast<unsigned char*>(ws);
  w.need = reinterpret_cast<uint32_t*>(p);
  p += round16((size_t)B * w.words * 4);
  w.before = reinterpret_cast<int32_t*>(p);
  p += round16((size_t)(B + 1) * 4);
  w.copy = reinterpret_cast<int32_t*>(p);
  p += round16((size_t)B * 4);
  w.n_free = reinterpret_cast<int32_t*>(p);
  p += 16;
  w.free = reinterpret_cast<int32_t*>(p);
  return w;
}

struct Span {
  int first, last;   // blocks [first, last) are to be written; last < 0: the row is left alone
};
__device__ __forceinline__ Span span_of(const int32_t* start, const int32_t* end, int b, int N, int32_t* err) {
  const int e = __ldg(end + b), s = max(__ldg(start + b), 0);
  if (e < 0) return {0, -1};
  const int last = e / KV_BLOCK + (e % KV_BLOCK != 0);
  if (last > N) set_err(err, BRE_DEVERR_PAGE);
  return {min(s / KV_BLOCK, N), min(last, N)};
}

constexpr int KZ_THREADS = 1024;

__global__ void __launch_bounds__(KZ_THREADS)
    kv_resize_plan_kernel(const int32_t* __restrict__ refs, int n_pages, const int32_t* __restrict__ table, int B, int N,
                          const int32_t* __restrict__ start, const int32_t* __restrict__ end, ResizeWs w, int32_t* err) {
  __shared__ int s_warp[KZ_THREADS / 32];
  __shared__ int s_total;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a warp a row
  for (int b = warp; b < B; b += KZ_THREADS / 32) {
    const Span sp = span_of(start, end, b, N, lane == 0 ? err : nullptr);
    int n = 0, copy = -1;
    for (int c = sp.first / 32 * 32; c < sp.last; c += 32) {
      const int k = c + lane;
      bool needs = false;
      if (k >= sp.first && k < sp.last) {
        int page = __ldg(table + (size_t)b * N + k);
        if (page >= n_pages) set_err(err, BRE_DEVERR_PAGE), page = -1;
        needs = page < 0 || refs[page] > 1;
        if (needs && page >= 0 && k == sp.first && __ldg(start + b) % KV_BLOCK > 0) copy = page;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, needs);
      if (lane == 0) w.need[(size_t)b * w.words + c / 32] = bits;
      n += __popc(bits);
    }
    copy = __reduce_max_sync(0xffffffffu, copy);
    if (lane == 0) w.before[b + 1] = n, w.copy[b] = copy;
  }
  __syncthreads();
  // running sums over the rows
  if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      int v = b0 + lane < B ? w.before[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
      }
      if (b0 + lane < B) w.before[b0 + lane + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) w.before[0] = 0, s_total = sum;
  }
  __syncthreads();
  const int total = s_total;
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < total; p0 += KZ_THREADS) {
    const bool is = p0 + tid < n_pages && refs[p0 + tid] == 0;
    const uint32_t bits = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_warp[warp] = __popc(bits);
    __syncthreads();
    int at = found;
    for (int i = 0; i < KZ_THREADS / 32; ++i) {
      if (i < warp) at += s_warp[i];
      found += s_warp[i];
    }
    at += __popc(bits & ((1u << lane) - 1u));
    if (is && at < total) w.free[at] = p0 + tid;
    __syncthreads();
  }
  if (tid == 0) {
    *w.n_free = min(found, total);
    if (found < total) set_err(err, BRE_DEVERR_FULL);
  }
}

constexpr int KZ_ROW = 128;

__global__ void __launch_bounds__(KZ_ROW)
    kv_resize_rows_kernel(uint8_t* pages, int8_t* bounds, int8_t* bexp, int n_pages, int H, int D, int32_t* refs, int32_t* table,
                          int N, const int32_t* __restrict__ start, const int32_t* __restrict__ end, ResizeWs w) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int at0 = w.before[b], n_free = *w.n_free;
  if (blockIdx.y) {   // one head's share of the page that the row goes on in
    const int from = w.copy[b], h = blockIdx.y - 1;
    if (from < 0 || at0 >= n_free) return;
    const int to = w.free[at0];
    const size_t PB = kv_page_bytes(D);
    const uint4* src = reinterpret_cast<const uint4*>(pages + ((size_t)from * H + h) * PB);
    uint4* dst = reinterpret_cast<uint4*>(pages + ((size_t)to * H + h) * PB);
    for (int i = tid; i < (int)(PB / 16); i += KZ_ROW) dst[i] = src[i];
    const size_t fh = (size_t)from * H + h, th = (size_t)to * H + h;
    for (int i = tid; i < 2 * D; i += KZ_ROW) bounds[th * 2 * D + i] = bounds[fh * 2 * D + i];
    if (tid == 0) bexp[th] = bexp[fh];
    return;
  }
  const Span sp = span_of(start, end, b, N, nullptr);
  if (sp.last < 0) return;
  int32_t* row = table + (size_t)b * N;
  // every warp walks the whole row, and changes its own 32 blocks of each 128
  int at = at0;
  for (int c = sp.first / 32 * 32; c < sp.last; c += 32) {
    const uint32_t bits = w.need[(size_t)b * w.words + c / 32];
    if (c / 32 % (KZ_ROW / 32) == warp && bits >> lane & 1u) {
      const int i = at + __popc(bits & ((1u << lane) - 1u));
      if (i < n_free) {
        const int old = row[c + lane], page = w.free[i];
        if (old >= 0 && old < n_pages) atomicSub(refs + old, 1);
        row[c + lane] = page;
        refs[page] = 1;
      }
    }
    at += __popc(bits);
  }
  for (int c = sp.last + tid; c < N; c += KZ_ROW) {
    const int old = row[c];
    if (old < 0) continue;
    if (old < n_pages) atomicSub(refs + old, 1);
    row[c] = -1;
  }
}

}  // namespace

cudaError_t launch_kv_compact(const bre_kv_cache* c, const int32_t* table, int B, int N, const int32_t* start,
                              const int32_t* nodes, int A, const int32_t* count, int32_t* length, int32_t* err, cudaStream_t s) {
  const KvTable tab{table, B, N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_compact_kernel<128> : kv_compact_kernel<64>;
  return launch_k(kern, dim3((unsigned)B, (unsigned)c->n_kv_heads, 2), dim3(KC_THREADS), 0, s, static_cast<uint8_t*>(c->pages),
                  c->bounds, c->bound_exp, c->n_kv_heads, tab, start, nodes, A, count, length, err);
}

cudaError_t launch_kv_fork(int n_pages, int32_t* refs, int32_t* table, int B, int N, const int32_t* parent,
                           const int32_t* length, int32_t* err, cudaStream_t s) {
  int width = 32;   // columns of a CTA: whole sectors as long as they fit
  while (width > 1 && (size_t)width * B * 4 > 48 * 1024) width /= 2;
  const size_t smem = (size_t)width * B * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kv_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kv_fork_kernel, dim3((unsigned)((N + width - 1) / width)), dim3(KF_THREADS), smem, s, n_pages, refs, table, B,
                  N, width, parent, length, err);
}

size_t kv_resize_ws_bytes(int n_pages, int B, int N) {
  const size_t blocks = (size_t)B * N, words = ((size_t)N + 31) / 32;
  return round16((size_t)B * words * 4) + round16((size_t)(B + 1) * 4) + round16((size_t)B * 4) + 16 +
         round16(4 * (blocks < (size_t)n_pages ? blocks : (size_t)n_pages));
}

cudaError_t launch_kv_resize(const bre_kv_cache* c, int32_t* refs, int32_t* table, int B, int N, const int32_t* start,
                             const int32_t* end, void* ws, int32_t* err, cudaStream_t s) {
  const ResizeWs w = resize_ws(ws, B, N);
  const cudaError_t e = launch_k(kv_resize_plan_kernel, dim3(1), dim3(KZ_THREADS), 0, s, refs, c->n_pages, table, B, N, start,
                                 end, w, err);
  if (e != cudaSuccess) return e;
  return launch_k(kv_resize_rows_kernel, dim3((unsigned)B, (unsigned)c->n_kv_heads + 1), dim3(KZ_ROW), 0, s,
                  static_cast<uint8_t*>(c->pages), c->bounds, c->bound_exp, c->n_pages, c->n_kv_heads, c->head_dim, refs, table, N,
                  start, end, w);
}

}  // namespace bre

// Pages of the quantised cache: kept tokens moved together, sequences that share pages, pages given out and taken back.
#include "kv_common.cuh"

namespace bre {

namespace {

// ---------------------------------------------------------------------------
// Compaction
// ---------------------------------------------------------------------------
// A cluster of CTAs moves one head's keys (blockIdx.z = 0) or values (1) of one sequence, KC_BLOCKS target blocks a CTA at a
// time: all of them read their blocks' rows into shared memory, a barrier of the cluster, then all write.  A row never
// moves up, so what later rounds read lies behind all that earlier ones write.  What lies in the first block below `start`
// stays where it is.  Keys pass through shared memory anyway, so the blocks' bounds come from there.  (One CTA a head, a block
// after the other: 95 us for 16 sequences of up to 2,000 kept tokens of 6,000, 4 heads of 128; a block's loads ahead: 60; a
// cluster, four blocks ahead: 18, for 67 MB that are read and written, most of it in L2.  Bound: loads, barriers of the cluster
// and stores that follow one another, two or three rounds.  A path of 8 of 32 drafts, 4 sequences: 4.0, a launch and one round.)
constexpr int KC_THREADS = 256, KC_BLOCKS = 4;

template <int D>
struct CompactMem {
  uint4 rows[KC_BLOCKS * KV_BLOCK][D / 16];
  uint8_t scales[KC_BLOCKS * KV_BLOCK];
  float hi[KC_THREADS / 32][D], lo[KC_THREADS / 32][D], top[KC_THREADS / 32];
};

template <int D>
__global__ void __launch_bounds__(KC_THREADS)
    kv_compact_kernel(uint8_t* pages, int8_t* __restrict__ bounds, int8_t* __restrict__ bexp, int H, KvTable tab,
                      const int32_t* __restrict__ start, const int32_t* __restrict__ nodes, int A,
                      const int32_t* __restrict__ count, int32_t* __restrict__ length, int32_t* err) {
  constexpr int LR = D / 16, ROWS = KC_BLOCKS * KV_BLOCK;   // lanes a row
  static_assert(KC_THREADS == 64 * KC_BLOCKS, "two warps a block");
  extern __shared__ __align__(16) unsigned char raw[];
  CompactMem<D>& sh = *reinterpret_cast<CompactMem<D>*>(raw);
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = tid % LR;
  const int ranks = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int b = blockIdx.x / ranks, h = blockIdx.y, values = blockIdx.z;
  const int n = __ldg(count + b);
  const long long s0 = __ldg(start + b);
  const int32_t* nd = nodes + (size_t)b * A;
  const int32_t* row = tab.table + (size_t)b * tab.N;
  // nothing is moved unless the list ascends and all of its tokens, and the blocks that they move to, have pages
  bool bad = n > A || (n >= 0 && (s0 < 0 || s0 + n > (long long)tab.N * KV_BLOCK));
  if (n >= 0 && !bad) {
#pragma unroll 4
    for (int j = tid; j < n; j += KC_THREADS) {
      const int x = __ldg(nd + j), before = j ? __ldg(nd + j - 1) : -1;
      const long long src = s0 + x;
      if (x <= before || src >= (long long)tab.N * KV_BLOCK || kv_page(tab, b, (int)(src / KV_BLOCK), err) < 0) bad = true;
    }
    for (long long k = s0 / KV_BLOCK + tid; k * KV_BLOCK < s0 + n; k += KC_THREADS)
      if (kv_page(tab, b, (int)k, err) < 0) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && rank == 0 && h == 0 && values == 0 && length) length[b] = (int)(n >= 0 && !bad ? s0 + n : s0);
  if (bad && tid == 0) set_err(err, BRE_DEVERR_PAGE);
  if (bad || n < 0) return;   // (all CTAs of the cluster alike)
  const int end = (int)(s0 + n);
  const size_t PB = kv_page_bytes(D);
  const int row_at = values ? KV_BLOCK * D : 0, scale_at = 2 * KV_BLOCK * D + (values ? KV_BLOCK : 0);
  for (long long round = s0 / KV_BLOCK; round * KV_BLOCK < end; round += ranks * KC_BLOCKS) {
    const long long p0 = (round + rank * KC_BLOCKS) * KV_BLOCK;   // this CTA's first token
    const int have = (int)min(max(end - p0, 0LL), (long long)ROWS);
#pragma unroll 4
    for (int i = tid; i < have * LR; i += KC_THREADS) {
      const int x = i / LR, p = (int)(p0 + x), from = p < s0 ? p : (int)(s0 + __ldg(nd + (p - s0)));
      const uint8_t* src = pages + ((size_t)__ldg(row + from / KV_BLOCK) * H + h) * PB + row_at + (from % KV_BLOCK) * D;
      cp_async16(&sh.rows[x][i % LR], src + (i % LR) * 16, 16);
    }
    if (tid < have) {
      const int p = (int)(p0 + tid), from = p < s0 ? p : (int)(s0 + __ldg(nd + (p - s0)));
      sh.scales[tid] = (pages + ((size_t)__ldg(row + from / KV_BLOCK) * H + h) * PB)[scale_at + from % KV_BLOCK];
    }
    static_assert(ROWS <= KC_THREADS, "a thread a scale");
    cp_async_wait_all();
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
    const int kept = (int)min(max(s0 - p0, 0LL), (long long)have);   // rows that stay where they are
#pragma unroll 4
    for (int i = kept * LR + tid; i < have * LR; i += KC_THREADS) {
      const int x = i / LR;
      uint8_t* dst = pages + ((size_t)__ldg(row + (p0 + x) / KV_BLOCK) * H + h) * PB;
      *(reinterpret_cast<uint4*>(dst + row_at + x % KV_BLOCK * D) + i % LR) = sh.rows[x][i % LR];
    }
    if (tid >= kept && tid < have)
      (pages + ((size_t)__ldg(row + (p0 + tid) / KV_BLOCK) * H + h) * PB)[scale_at + tid % KV_BLOCK] = sh.scales[tid];
    if (!values) {
      // bounds from all keys that the blocks now have (a NaN row, whose codes are zeros, counts as zeros): two warps a block
      const int blk = warp / 2, x0 = blk * KV_BLOCK, sub = tid & 63;
      float hi[16], lo[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) hi[c] = -INFINITY, lo[c] = INFINITY;
#pragma unroll 2
      for (int x = x0 + sub / LR; x < min(x0 + KV_BLOCK, have); x += 64 / LR) {
        const uint4 w = sh.rows[x][lr];
        const int sc = sh.scales[x];
        const float up = pow2f(sc == KV_NAN ? 0 : sc - 127);
        const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = f16x2_to_f32x2(e4m3x2_to_f16x2(c[i / 2] >> (16 * (i & 1)) & 0xFFFFu));
          hi[2 * i] = fmaxf(hi[2 * i], f.x * up), hi[2 * i + 1] = fmaxf(hi[2 * i + 1], f.y * up);
          lo[2 * i] = fminf(lo[2 * i], f.x * up), lo[2 * i + 1] = fminf(lo[2 * i + 1], f.y * up);
        }
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < 16; ++c)
#pragma unroll
        for (int o = LR; o < 32; o *= 2) {
          hi[c] = fmaxf(hi[c], __shfl_xor_sync(0xffffffffu, hi[c], o));
          lo[c] = fminf(lo[c], __shfl_xor_sync(0xffffffffu, lo[c], o));
        }
      float amax = 0.0f;
      if (lane < LR)
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          sh.hi[warp][lr * 16 + c] = hi[c], sh.lo[warp][lr * 16 + c] = lo[c];
          if (hi[c] > -INFINITY) amax = fmaxf(amax, fmaxf(fabsf(hi[c]), fabsf(lo[c])));
        }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));   // (not negative)
      if (lane == 0) sh.top[warp] = amax;
      __syncthreads();
      if (x0 < have) {
        const int e = bound_exp_of(fmaxf(sh.top[2 * blk], sh.top[2 * blk + 1]));
        const float down = pow2f(-e);
        const size_t ph = (size_t)__ldg(row + (p0 + x0) / KV_BLOCK) * H + h;
#pragma unroll
        for (int c = sub; c < D; c += 64) {   // (see kv_append for a channel that vanishes in the unit)
          const float ch = fmaxf(sh.hi[2 * blk][c], sh.hi[2 * blk + 1][c]), cl = fminf(sh.lo[2 * blk][c], sh.lo[2 * blk + 1][c]);
          const float up = ceilf(ch * down), dn = floorf(cl * down);
          bounds[ph * 2 * D + c] = (int8_t)(ch > 0.0f ? fmaxf(up, 1.0f) : up);
          bounds[ph * 2 * D + D + c] = (int8_t)(cl < 0.0f ? fminf(dn, -1.0f) : dn);
        }
        if (sub == 0) bexp[ph] = (int8_t)e;
      }
    }
    __syncthreads();   // shared memory is free again
  }
  if (ranks > 1) cluster_sync_all();   // (no CTA of a cluster that shares barriers leaves early)
}

// ---------------------------------------------------------------------------
// Forks
// ---------------------------------------------------------------------------
// A CTA takes some columns (blocks) of the table with all of its rows: what a row gets lies in the same columns of another
// row, so the old entries are brought into shared memory and then replaced in place.  References change by atomic sums
// of whole numbers, whose order does not matter, and only where an entry changes.  Latency: 192 rows of 258 blocks 4 us.
constexpr int KF_THREADS = 512;

__global__ void __launch_bounds__(KF_THREADS)
    kv_fork_kernel(int n_pages, int32_t* refs, int32_t* table, int B, int N, int width, const int32_t* __restrict__ parent,
                   const int32_t* __restrict__ length, int32_t* err) {
  extern __shared__ int32_t old[];   // [B][width]
  pdl_wait();
  pdl_launch_dependents();
  const int c0 = blockIdx.x * width, nc = min(width, N - c0);
  const int rows = KF_THREADS / width, col = threadIdx.x % width;
#pragma unroll 4
  for (int b = threadIdx.x / width; b < B; b += rows)
    if (col < nc) old[b * width + col] = table[(size_t)b * N + c0 + col];
  __syncthreads();
  if (col >= nc) return;
#pragma unroll 2
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
// by the order of the CTAs: a first kernel marks the blocks and lists the free pages, a second one hands them out.  Latency of two
// launches (a grid-wide order cannot be had within one of many CTAs): 4 rows 3.6 us, 192 rows, 13,000 pages 5.4.
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ranks = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  // a warp a row, by all CTAs of the cluster; the first one then has the rest to itself
  for (int b = rank * (KZ_THREADS / 32) + warp; b < B; b += ranks * (KZ_THREADS / 32)) {
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
  cluster_sync_all();
  if (rank) return;
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
  const bool aligned = reinterpret_cast<uintptr_t>(refs) % 16 == 0;
  // 16 pages a thread and round: the loads of a round are in flight together
  constexpr int PT = 16;
  int found = 0;
  for (long long p0 = 0; p0 < n_pages && found < total; p0 += KZ_THREADS * PT) {
    const long long mine = p0 + (long long)tid * PT;
    uint32_t is = 0;
    if (mine + PT <= n_pages && aligned) {
      int4 v[PT / 4];
#pragma unroll
      for (int i = 0; i < PT / 4; ++i) v[i] = reinterpret_cast<const int4*>(refs + mine)[i];
#pragma unroll
      for (int i = 0; i < PT / 4; ++i)
        is |= ((v[i].x == 0) | (v[i].y == 0) << 1 | (v[i].z == 0) << 2 | (v[i].w == 0) << 3) << (4 * i);
    } else {
      for (int i = 0; i < PT; ++i)
        if (mine + i < n_pages && refs[mine + i] == 0) is |= 1u << i;
    }
    int upto = __popc(is);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    const int of = s_warp[lane];   // (32 warps)
    int at = found + upto - __popc(is) + __reduce_add_sync(0xffffffffu, lane < warp ? of : 0);
    found += __reduce_add_sync(0xffffffffu, of);
    for (; is && at < total; is &= is - 1, ++at) w.free[at] = (int)(mine + __ffs(is) - 1);
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
#pragma unroll 5
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
  // CTAs of a head: blocks for all of them in the longest list, as far as the GPU has room for (three an SM fit; 16 sequences of
  // up to 2,000 kept tokens, 4 heads: 1,024 CTAs 24.2 us, 512 18.3, 256 25.9)
  const long long blocks = ((long long)A + 2 * KV_BLOCK - 2) / KV_BLOCK, heads = 2LL * B * c->n_kv_heads;
  int ranks = 1;
  while (ranks < 8 && ranks * KC_BLOCKS < blocks && heads * ranks < 2LL * device_sm_count()) ranks *= 2;
  auto kern = c->head_dim == 128 ? kv_compact_kernel<128> : kv_compact_kernel<64>;
  const size_t smem = c->head_dim == 128 ? sizeof(CompactMem<128>) : sizeof(CompactMem<64>);
  static_assert(sizeof(CompactMem<128>) <= 48 * 1024, "no attribute needed");
  return launch_kc(kern, dim3((unsigned)(B * ranks), (unsigned)c->n_kv_heads, 2), dim3(KC_THREADS), ranks, smem, s,
                   static_cast<uint8_t*>(c->pages), c->bounds, c->bound_exp, c->n_kv_heads, tab, start, nodes, A, count, length, err);
}

cudaError_t launch_kv_fork(int n_pages, int32_t* refs, int32_t* table, int B, int N, const int32_t* parent,
                           const int32_t* length, int32_t* err, cudaStream_t s) {
  int width = 8;   // columns of a CTA: whole sectors as long as they fit
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
  int ranks = 1;
  while (ranks < 8 && ranks * (KZ_THREADS / 32) < B) ranks *= 2;
  const cudaError_t e = launch_kc(kv_resize_plan_kernel, dim3((unsigned)ranks), dim3(KZ_THREADS), ranks, 0, s, refs, c->n_pages, table, B, N, start,
                                  end, w, err);
  if (e != cudaSuccess) return e;
  return launch_k(kv_resize_rows_kernel, dim3((unsigned)B, (unsigned)c->n_kv_heads + 1), dim3(KZ_ROW), 0, s,
                  static_cast<uint8_t*>(c->pages), c->bounds, c->bound_exp, c->n_pages, c->n_kv_heads, c->head_dim, refs, table, N,
                  start, end, w);
}

}  // namespace bre

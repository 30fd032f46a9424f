// Writing keys and values into the quantised paged cache, and reading them back.
#include "kv_common.cuh"

namespace bre {

namespace {

// A chunk of the call's tokens and one head per CTA.  The tokens in a row that belong to one block are
// a run (padding entries among them do not end it); a run is stored by the CTA in whose chunk it starts, which sees all of its keys and so can
// bring the block's bounds up to date without atomics.
//
// A lane holds eight channels, so D / 8 lanes hold a row and a warp two or four rows at a time: 16-byte loads,
// 8-byte stores, a row's maximum by three or four shuffles.  A chunk of 64 tokens gives long calls whole
// blocks; with few tokens the chunks shrink to one token and a call spreads over the GPU.
//
// A call is a chain of loads that wait for one another, and for long calls half of its time is arithmetic
// (4.8 million warp instructions for 8,192 tokens of 4 heads of 128).  So the chain is kept short: positions,
// then the page's number beside the first rows, then two rows a lane in flight, each replaced as it is used; 9.8 us
// for those tokens, against 11.2 us with the rows asked for once the run and its page were known.  Four rows a lane
// take 119 registers: 9.6 us there, but 15.6 against 13.0 us for 6,418 ragged tokens of 8 heads of 64; six CTAs an SM
// instead of five 10.5 us.
constexpr int KA_WARPS = 4;

// A row of eight channels a lane; LR lanes hold the row.
template <int LR>
struct RowCode {
  uint2 codes;
  int e;       // scale exponent
  bool nan;
  __device__ __forceinline__ explicit RowCode(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t mx = 0;   // magnitudes of BF16 values compare like whole numbers
#pragma unroll
    for (int i = 0; i < 4; ++i) mx = __vmaxu2(mx, u[i] & 0x7FFF7FFFu);
    mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
    for (int o = 1; o < LR; o *= 2) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    nan = mx > 0x7F80u;
    e = row_exp(bf16_bits_to_f32(min(mx, 0x7F60u)));   // KV_MAX
    const float down = pow2f(-e);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = __fmul2_rn(make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)),
                                  make_float2(down, down));
      x[2 * i] = y.x, x[2 * i + 1] = y.y;
    }
    // (the conversion saturates what lies above KV_MAX)
    codes = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    if (nan) codes = make_uint2(0u, 0u);
  }
};

// Padding may be long (a graph of a fixed number of tokens): what looks beyond it takes KA_LOOK entries a lane at a time.
constexpr int KA_LOOK = 8;

// By a whole warp: the last index <= i whose entry is no padding, -1 if there is none.
__device__ __forceinline__ int last_real(const int32_t* __restrict__ pos, int i) {
  const int lane = threadIdx.x & 31;
  for (; i >= 0; i -= KA_LOOK * 32) {
    int p[KA_LOOK];
#pragma unroll
    for (int j = 0; j < KA_LOOK; ++j) p[j] = i - 32 * j - lane >= 0 ? __ldg(pos + i - 32 * j - lane) : -1;
#pragma unroll
    for (int j = 0; j < KA_LOOK; ++j) {
      const uint32_t real = __ballot_sync(0xffffffffu, p[j] >= 0);
      if (real) return i - 32 * j - (__ffs(real) - 1);
    }
  }
  return -1;
}

// By a whole warp, of the entries first .. first + 32 KA_LOOK - 1 (< T): the first of another block (else T), and the
// last before it that is of this one, plus 1 (else 0).
__device__ __forceinline__ int2 run_end(const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, int first, int T,
                                        int s, int blk) {
  const int lane = threadIdx.x & 31;
  int p[KA_LOOK], q[KA_LOOK], last = 0;
#pragma unroll
  for (int j = 0; j < KA_LOOK; ++j) {
    const int i = first + 32 * j + lane;
    p[j] = i < T ? __ldg(pos + i) : -1, q[j] = i < T ? __ldg(seq + i) : -1;
  }
#pragma unroll
  for (int j = 0; j < KA_LOOK; ++j) {
    const uint32_t other = __ballot_sync(0xffffffffu, p[j] >= 0 && (q[j] != s || p[j] / KV_BLOCK != blk));
    const uint32_t own = __ballot_sync(0xffffffffu, p[j] >= 0) & ((other & -other) - 1u);   // (all if there is no other)
    if (own) last = first + 32 * j + 32 - __clz(own);
    if (other) return make_int2(first + 32 * j + __ffs(other) - 1, last);
  }
  return make_int2(T, last);
}

template <int D>
__global__ void __launch_bounds__(KA_WARPS * 32, 5)
    kv_append_kernel(uint8_t* __restrict__ pages, int8_t* __restrict__ bounds, int8_t* __restrict__ bexp, int H, KvTable tab,
                     const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, long long k_stride, long long v_stride,
                     const int32_t* __restrict__ seq, const int32_t* __restrict__ pos, int T, int chunk, int32_t* err) {
  constexpr int LR = D / 8, RW = 32 / LR;       // lanes a row, rows a warp
  constexpr int RC = RW * KA_WARPS, UN = 2;     // rows of the CTA at a time, of which UN steps are in flight
  __shared__ float s_hi[KA_WARPS][D], s_lo[KA_WARPS][D], s_max[KA_WARPS];
  __shared__ int2 s_end[2][KA_WARPS];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, lr = lane % LR;
  const int h = blockIdx.y, c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, T);
  int par = 0;   // of s_end: the barrier of one pass also keeps the next but one from overtaking it
  for (int t = c0; t < c1;) {
    // What the run needs is read in two steps, each of loads that do not wait for one another: first the
    // positions, then the page's number, the first rows and (page known) the old bounds.
    const int s = __ldg(seq + t), p = __ldg(pos + t), blk = p / KV_BLOCK;
    const int bs = t ? __ldg(seq + t - 1) : 0, bp = t ? __ldg(pos + t - 1) : 0;
    const int q0 = t + warp * RW + lane / LR;   // this lane's first row
    int slot[UN], sq[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const int r = q0 + j * RC;
      slot[j] = r < T ? __ldg(pos + r) : -1, sq[j] = r < T ? __ldg(seq + r) : -1;
    }
    const int i = t + 1 + tid;
    const int pi = i < T ? __ldg(pos + i) : -1, si = i < T ? __ldg(seq + i) : -1;
    if (p < 0) {   // on to the next entry that is no padding
      const uint32_t real = __ballot_sync(0xffffffffu, t + 1 + lane < c1 && __ldg(pos + t + 1 + lane) >= 0);
      t += real ? __ffs(real) : 33;
      continue;
    }
    // a run that started in a chunk before belongs to it
    bool mine = t == 0 || bp < 0 || bs != s || bp / KV_BLOCK != blk;
    if (t && bp < 0) {
      const int back = last_real(pos, t - 2);
      mine = back < 0 || __ldg(seq + back) != s || __ldg(pos + back) / KV_BLOCK != blk;
    }
    const int page = mine ? kv_page(tab, s, blk, tid == 0 ? err : nullptr) : -1;
    uint4 kw[UN], vw[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {   // (rows of the block behind another block's are of another run: not stored below)
      const int r = q0 + j * RC;
      const bool in = mine && slot[j] >= 0 && sq[j] == s && slot[j] / KV_BLOCK == blk;
      kw[j] = in ? __ldg(reinterpret_cast<const uint4*>(k + r * k_stride + h * D) + lr) : make_uint4(0, 0, 0, 0);
      vw[j] = in ? __ldg(reinterpret_cast<const uint4*>(v + r * v_stride + h * D) + lr) : make_uint4(0, 0, 0, 0);
    }
    // the run's end: the first token of another block; and its last own token, as padding may follow
    int t1 = T, t2 = t + 1;
    {
      const uint32_t other = __ballot_sync(0xffffffffu, pi >= 0 && (si != s || pi / KV_BLOCK != blk));
      const uint32_t own = __ballot_sync(0xffffffffu, pi >= 0) & ((other & -other) - 1u);   // (all if there is no other)
      const int i0 = t + 1 + warp * 32;
      if (lane == 0) s_end[par][warp] = make_int2(other ? i0 + __ffs(other) - 1 : T, own ? i0 + 32 - __clz(own) : 0);
    }
    for (int i0 = t + 1 + KA_WARPS * 32;; i0 += KA_WARPS * KA_LOOK * 32) {
      __syncthreads();
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) {
        const int2 end = s_end[par][w];
        if (t1 == T) t1 = end.x, t2 = max(t2, end.y);
      }
      par ^= 1;
      if (t1 < T || i0 >= T) break;
      const int2 end = run_end(seq, pos, i0 + warp * KA_LOOK * 32, T, s, blk);
      if (lane == 0) s_end[par][warp] = end;
    }
    t = t1;
    if (!mine) continue;
    if (page < 0) {
      if (tid == 0) set_err(err, BRE_DEVERR_PAGE);   // a token to store needs a page
      continue;
    }
    const size_t ph = (size_t)page * H + h;
    uint8_t* pg = pages + ph * kv_page_bytes(D);
    int8_t* bd = bounds + ph * 2 * D + tid;
    const bool begun = p % KV_BLOCK != 0;   // before this call
    int oe = -127, oh = 0, ol = 0;
    if (begun) {
      oe = bexp[ph];
      if (tid < D) oh = bd[0], ol = bd[D];
    }
    float hi[8], lo[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) hi[c] = -INFINITY, lo[c] = INFINITY;
    for (int r0 = q0; r0 - lane / LR < t2; r0 += UN * RC) {
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        const RowCode<LR> kc(kw[j]), vc(vw[j]);
        const int at = r0 + j * RC < t2 ? slot[j] : -1;
        // a later row takes the registers: its loads run while the others are stored
        const int r = r0 + (UN + j) * RC;
        const bool in = r < t2;
        kw[j] = in ? __ldg(reinterpret_cast<const uint4*>(k + r * k_stride + h * D) + lr) : make_uint4(0, 0, 0, 0);
        vw[j] = in ? __ldg(reinterpret_cast<const uint4*>(v + r * v_stride + h * D) + lr) : make_uint4(0, 0, 0, 0);
        slot[j] = in ? __ldg(pos + r) : -1;
        if (at < 0) continue;
        const int sl = at % KV_BLOCK;
        *reinterpret_cast<uint2*>(pg + sl * D + lr * 8) = kc.codes;
        *reinterpret_cast<uint2*>(pg + KV_BLOCK * D + sl * D + lr * 8) = vc.codes;
        if (lr == 0) {
          pg[2 * KV_BLOCK * D + sl] = (uint8_t)(kc.nan ? KV_NAN : kc.e + 127);
          pg[2 * KV_BLOCK * D + KV_BLOCK + sl] = (uint8_t)(vc.nan ? KV_NAN : vc.e + 127);
        }
        const float up = pow2f(kc.e);
        const uint32_t c[2] = {kc.codes.x, kc.codes.y};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f = __fmul2_rn(f16x2_to_f32x2(e4m3x2_to_f16x2(c[x / 2] >> (16 * (x & 1)) & 0xFFFFu)), make_float2(up, up));
          hi[2 * x] = fmaxf(hi[2 * x], f.x), hi[2 * x + 1] = fmaxf(hi[2 * x + 1], f.y);
          lo[2 * x] = fminf(lo[2 * x], f.x), lo[2 * x + 1] = fminf(lo[2 * x + 1], f.y);
        }
      }
    }
    // the warps' extremes, then the block's bounds
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = LR; o < 32; o *= 2) {
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      }
    if (lane < LR)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_hi[warp][lr * 8 + i] = hi[i], s_lo[warp][lr * 8 + i] = lo[i];
    __syncthreads();
    constexpr int ND = D / 128 ? D / 128 : 1;   // channels a thread
    float ch = -INFINITY, cl = INFINITY, amax = 0.0f;
    if (tid < D) {
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) ch = fmaxf(ch, s_hi[w][tid]), cl = fminf(cl, s_lo[w][tid]);
      amax = fmaxf(fabsf(ch), fabsf(cl));
    }
    static_assert(ND == 1 && D <= KA_WARPS * 32, "a thread a channel");
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) amax = fmaxf(amax, s_max[w]);
    int e = bound_exp_of(amax);
    if (begun) {   // (the old exponent was read before the barriers, so it may be overwritten)
      ch = fmaxf(ch, oh * pow2f(oe)), cl = fminf(cl, ol * pow2f(oe));
      e = max(e, oe);
    }
    if (tid < D) {
      // (beside a key 2^115 larger a channel may vanish in the product, yet its bounds lie on their sides of 0)
      const float down = pow2f(-e), hi = ceilf(ch * down), lo = floorf(cl * down);
      bd[0] = (int8_t)(ch > 0.0f ? fmaxf(hi, 1.0f) : hi);
      bd[D] = (int8_t)(cl < 0.0f ? fminf(lo, -1.0f) : lo);
    }
    if (tid == 0) bexp[ph] = (int8_t)e;
  }
}

// Codes times the row's scale, exact in BF16.  A lane takes 16 codes: D / 16 lanes a row, two rows'
// keys and values of a lane in flight (more of them cost registers and so warps: 92 us against 71 for 131,072 tokens).
template <int D>
__global__ void __launch_bounds__(128)
    kv_read_kernel(const uint8_t* __restrict__ pages, int H, KvTable tab, const int32_t* __restrict__ seq,
                   const int32_t* __restrict__ pos, int T, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                   int32_t* err) {
  constexpr int LR = D / 16, UN = 2;
  pdl_wait();
  pdl_launch_dependents();
  // rows run over tokens first: the tokens of a block follow one another in a head's share of its page
  const long long row0 = ((long long)blockIdx.x * 128 + threadIdx.x) / LR;
  const int lr = threadIdx.x % LR, h = blockIdx.y;
  const long long step = (long long)gridDim.x * (128 / LR);
  for (long long r0 = row0; r0 < T; r0 += UN * step) {
    int page[UN], slot[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const long long t = r0 + j * step;
      const int p = t < T ? __ldg(pos + t) : -1;
      page[j] = p < 0 ? -1 : kv_page(tab, __ldg(seq + t), p / KV_BLOCK, err);
      if (p >= 0 && page[j] < 0) set_err(err, BRE_DEVERR_PAGE);
      slot[j] = p % KV_BLOCK;
    }
    uint4 kc[UN], vc[UN];
    int ke[UN], ve[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const uint8_t* pg = pages + ((size_t)max(page[j], 0) * H + h) * kv_page_bytes(D);
      const bool in = page[j] >= 0;
      kc[j] = in && k ? __ldg(reinterpret_cast<const uint4*>(pg + slot[j] * D) + lr) : make_uint4(0, 0, 0, 0);
      vc[j] = in && v ? __ldg(reinterpret_cast<const uint4*>(pg + KV_BLOCK * D + slot[j] * D) + lr) : make_uint4(0, 0, 0, 0);
      ke[j] = in ? (int)__ldg(pg + 2 * KV_BLOCK * D + slot[j]) : 127;
      ve[j] = in ? (int)__ldg(pg + 2 * KV_BLOCK * D + KV_BLOCK + slot[j]) : 127;
    }
#pragma unroll
    for (int j = 0; j < UN; ++j) {
      const long long t = r0 + j * step;
      if (t >= T) break;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint16_t* out = kv ? v : k;
        if (!out) continue;
        const uint4 c = kv ? vc[j] : kc[j];
        const uint32_t u[4] = {c.x, c.y, c.z, c.w};
        const float f = pow2f((kv ? ve[j] : ke[j]) - 127);   // infinite for a NaN row, whose codes are zeros
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2(u[i] & 0xFFFFu)), b = f16x2_to_f32x2(e4m3x2_to_f16x2(u[i] >> 16));
          o[2 * i] = pack_bf16x2(a.x * f, a.y * f), o[2 * i + 1] = pack_bf16x2(b.x * f, b.y * f);
        }
        st_v8(out + ((size_t)t * H + h) * D + 16 * lr, o);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const bre_kv_cache* c, const KvTokens& tk, const uint16_t* k, const uint16_t* v,
                             long long k_stride, long long v_stride, int32_t* err, cudaStream_t s) {
  const int H = c->n_kv_heads;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_append_kernel<128> : kv_append_kernel<64>;
  // tokens a CTA: whole blocks, as long as that leaves four CTAs to an SM
  int chunk = KV_BLOCK;
  while (chunk > 1 && (long long)tk.T * H < 4LL * device_sm_count() * chunk) chunk /= 2;
  return launch_k(kern, dim3((unsigned)((tk.T + chunk - 1) / chunk), (unsigned)H), dim3(KA_WARPS * 32), 0, s,
                  static_cast<uint8_t*>(c->pages), c->bounds, c->bound_exp, H, tab, k, v, k_stride, v_stride, tk.seq,
                  tk.pos, tk.T, chunk, err);
}

cudaError_t launch_kv_read(const bre_kv_cache* c, const KvTokens& tk, uint16_t* k, uint16_t* v, int32_t* err,
                           cudaStream_t s) {
  const int H = c->n_kv_heads;
  const KvTable tab{tk.table, tk.B, tk.N, c->n_pages};
  auto kern = c->head_dim == 128 ? kv_read_kernel<128> : kv_read_kernel<64>;
  // 16 codes a thread; beyond 64 CTAs to an SM they go on to further rows
  const long long ctas = ((long long)tk.T * (c->head_dim / 16) + 127) / 128;
  const long long most = (64LL * device_sm_count() + H - 1) / H;
  return launch_k(kern, dim3((unsigned)(ctas < most ? ctas : most), (unsigned)H), dim3(128), 0, s,
                  static_cast<const uint8_t*>(c->pages), H, tab, tk.seq, tk.pos, tk.T, k, v, err);
}

}  // namespace bre

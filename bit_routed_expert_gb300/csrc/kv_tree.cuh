// What the kernels of the attention over the whole context share: which slots a token sees, and the joining of parts.
#pragma once
#include <type_traits>

#include "kv_attend.cuh"

namespace bre {

// Bit x - 64 blk set: the token sees slot x (of the 64 of a block).
__device__ __forceinline__ uint64_t seen_bits(const uint64_t* __restrict__ mask, int words, int start, int pos, int blk) {
  const long long x0 = (long long)blk * KV_BLOCK;
  uint64_t own = pos >= x0 + 63 ? ~0ull : pos >= x0 ? (2ull << (pos - x0)) - 1ull : 0ull;
  if (!mask || own == 0) return own;
  const long long j = x0 - start;   // bit of the block's first slot
  uint64_t tree = 0;
  if (j < 0) {
    if (j <= -64) return own;
    tree = ((1ull << -j) - 1ull) | __ldg(mask) << -j;
  } else {
    const long long w = j / 64;
    const int r = (int)(j % 64);
    if (w < words) tree = __ldg(mask + w) >> r;
    if (r && w + 1 < words) tree |= __ldg(mask + w + 1) << (64 - r);
  }
  return own & tree;
}

// A row's parts (index(p): where part p's maximum and sum, and its output, lie), those from `from` on in steps of `step`,
// joined in their order by LANES neighbouring lanes of a warp: the maxima and sums by the lanes, then the outputs.
template <int D, int LANES>
struct Joined {
  static constexpr int CL = D / LANES, AHEAD = LANES / 4;   // channels of a lane; parts on their way
  float top, sum, v[CL];   // maximum, sum, output of this lane's channels, relative to the maximum

  template <typename Index>
  __device__ __forceinline__ Joined(const float2* ml, const float* part, int parts, int from, int step, Index index) {
    using Piece = typename std::conditional<CL % 4 == 0, float4, float2>::type;
    constexpr int PIECES = CL * (int)sizeof(float) / (int)sizeof(Piece);
    const int lane = threadIdx.x % LANES, n = (parts - from + step - 1) / step;   // its parts (as many for all of the warp)
    union Loaded {
      Piece x[PIECES];
      float v[CL];
    } o[AHEAD];
    auto fetch = [&](int i0) {   // on their way while the weights are formed
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int k = 0; k < PIECES; ++k) {
          o[i].x[k] = Piece{};
          if (i0 + i < n) o[i].x[k] = reinterpret_cast<const Piece*>(part + index(from + (i0 + i) * step) * D + lane * CL)[k];
        }
    };
    fetch(0);
    top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < n; i += LANES) top = fmaxf(top, ml[index(from + i * step)].x);
    __syncwarp();
#pragma unroll
    for (int j = LANES / 2; j; j >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, j));
    const float ref = top > -INFINITY ? top : 0.0f;
#pragma unroll
    for (int c = 0; c < CL; ++c) v[c] = 0.0f;
    float w = 0.0f;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
      if (i0 % LANES == 0) {
        const float2 y = i0 + lane < n ? ml[index(from + (i0 + lane) * step)] : make_float2(-INFINITY, 0.0f);
        w = ex2(y.x - ref);
        sum += scale_sum(y.y, y.x - ref);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) % LANES, LANES);
        if (i0 + i < n) {
#pragma unroll
          for (int c = 0; c < CL; ++c) v[c] = fmaf(wi, o[i].v[c], v[c]);
        }
      }
      if (i0 + AHEAD < n) fetch(i0 + AHEAD);
    }
#pragma unroll
    for (int j = LANES / 2; j; j >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, j);
  }
  __device__ __forceinline__ void store(uint16_t* out, float* lse) const {
    const int lane = threadIdx.x % LANES;
    const float inv = 1.0f / sum;
    uint32_t b[CL / 2];
#pragma unroll
    for (int i = 0; i < CL / 2; ++i) b[i] = sum == 0.0f ? 0u : pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    if constexpr (CL == 8) *reinterpret_cast<uint4*>(out + lane * CL) = make_uint4(b[0], b[1], b[2], b[3]);
    else if constexpr (CL == 4) *reinterpret_cast<uint2*>(out + lane * CL) = make_uint2(b[0], b[1]);
    else *reinterpret_cast<uint32_t*>(out + lane * CL) = b[0];
    if (lane == 0 && lse) *lse = sum == 0.0f ? -INFINITY : LN2 * (top > -INFINITY ? top - P_SHIFT + log2f(sum) : log2f(sum));
  }
};

// Rows that a CTA of JOIN_WARPS warps joins at a time.  Few parts: half a warp a row (the whole call 2% faster than by whole warps
// for a prompt of 4,096 tokens, 38,912 rows of 2 parts; 2% slower for 2,048 rows of 19 parts).  Many: the CTA a row, its parts dealt to
// the warps, whose results are joined once more (304 parts of 32 rows by warps: 38 us).
constexpr int JOIN_WARPS = 8;
__host__ __device__ constexpr int join_at_once(int parts, int few) { return parts <= few ? 2 * JOIN_WARPS : 1; }
// Pieces first, first + stride, .. of `rows` by a CTA.
template <int D, typename Index, typename Place>
__device__ __forceinline__ void join_rows(const float2* ml, const float* part, int parts, int few, int first, int stride, int rows, Index index,
                                          Place place, uint16_t* out, float* lse) {
  __shared__ float2 sh_ml[2][JOIN_WARPS];
  __shared__ __align__(16) float sh_part[2][JOIN_WARPS * D];   // (read in 16-byte pieces)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int at_once = join_at_once(parts, few);
  if (at_once > 1) {
    for (int r0 = first * at_once + 2 * warp; r0 < rows; r0 += stride * at_once) {
      const int r = min(r0 + lane / 16, rows - 1);   // (both halves of a warp stay together)
      const Joined<D, 16> row(ml, part, parts, 0, 1, [&](int p) { return index(p, r); });
      const size_t at = place(r);
      if (r0 + lane / 16 < rows) row.store(out + at * D, lse ? lse + at : nullptr);
      __syncwarp();
    }
    return;
  }
  int turn = 0;
  for (int r = first; r < rows; r += stride, turn ^= 1) {
    const Joined<D, 32> mine(ml, part, parts, warp, JOIN_WARPS, [&](int p) { return index(p, r); });
    if (lane == 0) sh_ml[turn][warp] = make_float2(mine.top, mine.sum);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) sh_part[turn][warp * D + lane * (D / 32) + i] = mine.v[i];
    __syncthreads();
    if (warp == 0) {
      const size_t at = place(r);
      Joined<D, 32>(sh_ml[turn], sh_part[turn], JOIN_WARPS, 0, 1, [](int p) { return (size_t)p; }).store(out + at * D, lse ? lse + at : nullptr);
    }
  }
}

// A token at a time (kv_tree_rows.cu)
size_t tree_rows_ws_bytes(int H, int G, int D);
cudaError_t launch_tree_rows(const TreeArgs& a, cudaStream_t s);

}  // namespace bre

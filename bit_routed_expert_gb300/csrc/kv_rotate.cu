// Rotary positions of queries and keys, and the host side of their frequencies.
#include <cmath>

#include "kv_common.cuh"

namespace bre {

namespace {

// A pair (a, b) of a head's channels turns by the angle 2 pi * frac(pos * turns / 2^64): the product of whole numbers
// wraps at a full turn by itself, so the angle has no error that grows with the position (a product in FP32 is off by a
// tenth of a radian at position 2^21).  Cosine and sine belong to a token, not to a head: a CTA forms those of its
// tokens once in shared memory; a thread keeps the ones of its pairs in registers for all the heads that it walks.
//
// Bound: HBM, each channel read and written once (4 bytes).  16-byte pieces, a thread's first KR_UNROLL heads on their way
// before the cosines are formed.  8,192 tokens, 36 heads of 128 (151 MB): 28.6 us, 5.3 TB/s, 0.78 of a plain copy's 6.8;
// 5,999 tokens, 16 heads of 64 (24.6 MB, from L2): 8.0 us; one token: 2.6 us, a launch.
constexpr int KR_THREADS = 256;
constexpr int KR_UNROLL = 4;   // heads of a thread in flight

struct RotateArgs {
  const uint16_t* in[2];   // queries, keys
  uint16_t* out[2];
  long long in_stride[2], out_stride[2];
  int heads[2];
  int D, pairs, offset, T;
  const int32_t* pos;
  const uint64_t* turns;
  float gain, sign;
  int items, groups, tokens;   // a head's items; groups of heads and tokens of a CTA
};

template <int V>
struct Vec {
  uint16_t x[V];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (V == 8) *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(x) = *reinterpret_cast<const uint32_t*>(p);
    else x[0] = *p;
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(x);
    else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(x);
    else *p = x[0];
  }
};

// An item is what a thread loads of a head: V channels of either half (HALF), V neighbouring channels (pairs side by
// side; with V = 1 a pair of two single channels), or V channels that only pass through.
template <int V, bool HALF>
__global__ void __launch_bounds__(KR_THREADS) kv_rotate_kernel(const RotateArgs a) {
  constexpr int PAIRS = HALF ? V : (V > 1 ? V / 2 : 1);   // of an item
  constexpr bool TWO = HALF || V == 1;                    // an item is two pieces
  extern __shared__ float2 cs[];                          // [tokens][pairs]
  __shared__ int s_pos[KR_THREADS];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.T - t0);
  const int per = a.items * a.groups, tl = threadIdx.x / per, rest = threadIdx.x - tl * per;
  const int group = rest / a.items, item = rest - group * a.items;
  const int turning = a.pairs / PAIRS;   // items that turn come first
  const bool mine = tl < nt, turns = item < turning;
  int at = 0, at2 = 0;
  if (turns) {
    at = HALF ? a.offset + item * V : a.offset + item * (V > 1 ? V : 2);
    at2 = HALF ? at + a.pairs : at + 1;
  } else {
    at = (item - turning) * V;
    if (at >= a.offset) at += 2 * a.pairs;
  }
  const long long t = t0 + tl;
  const int all = a.heads[0] + a.heads[1], step = a.groups * gridDim.y, first = group + blockIdx.y * a.groups;
  Vec<V> x[KR_UNROLL], y[KR_UNROLL];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < KR_UNROLL; ++u) {
      const int h = h0 + u * step;
      if (!mine || h >= all) continue;
      const uint16_t* p = h < a.heads[0] ? a.in[0] + t * a.in_stride[0] + (long long)h * a.D
                                         : a.in[1] + t * a.in_stride[1] + (long long)(h - a.heads[0]) * a.D;
      x[u].load(p + at);
      if (TWO && turns) y[u].load(p + at2);
    }
  };
  load(first);   // on their way while cosines and sines are formed
  for (int i = threadIdx.x; i < nt; i += blockDim.x) s_pos[i] = __ldg(a.pos + t0 + i);
  for (int i = threadIdx.x; i < nt * a.pairs; i += blockDim.x) {
    const int tt = i / a.pairs, j = i - tt * a.pairs;
    const uint64_t turn = (uint64_t)(uint32_t)max(__ldg(a.pos + t0 + tt), 0) * __ldg(a.turns + j);
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);   // half turns in [-1, 1]
    cs[i] = make_float2(c * a.gain, s * a.gain * a.sign);
  }
  __syncthreads();
  if (!mine) return;
  const bool pad = s_pos[tl] < 0;
  float c[PAIRS], s[PAIRS];
  if (turns) {
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const float2 f = cs[tl * a.pairs + item * PAIRS + i];
      c[i] = f.x, s[i] = f.y;
    }
  }
  for (int h0 = first; h0 < all; h0 += KR_UNROLL * step) {
#pragma unroll
    for (int u = 0; u < KR_UNROLL; ++u) {
      const int h = h0 + u * step;
      if (h >= all) continue;
      uint16_t* p = h < a.heads[0] ? a.out[0] + t * a.out_stride[0] + (long long)h * a.D
                                   : a.out[1] + t * a.out_stride[1] + (long long)(h - a.heads[0]) * a.D;
      if (pad) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[u].x[i] = y[u].x[i] = 0;
      } else if (turns) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          uint16_t &lo = TWO ? x[u].x[i] : x[u].x[2 * i], &hi = TWO ? y[u].x[i] : x[u].x[2 * i + 1];
          const float f = bf16_bits_to_f32(lo), g = bf16_bits_to_f32(hi);
          const uint32_t r = pack_bf16x2(f * c[i] - g * s[i], f * s[i] + g * c[i]);
          lo = (uint16_t)r, hi = (uint16_t)(r >> 16);
        }
      }
      x[u].store(p + at);
      if (TWO && turns) y[u].store(p + at2);
    }
    load(h0 + KR_UNROLL * step);
  }
}

template <int V>
cudaError_t launch(RotateArgs& a, bool half, cudaStream_t s) {
  const int pairs = half ? V : (V > 1 ? V / 2 : 1), all = a.heads[0] + a.heads[1];
  a.items = a.pairs / pairs + (a.D - 2 * a.pairs) / V;
  a.groups = KR_THREADS / a.items < all ? KR_THREADS / a.items : all;
  a.tokens = 1;
  int split = 1;
  // Few tokens: a head a thread, the heads over several CTAs.  Many: as many heads a thread as leave the CTA
  // several tokens, whose cosines and sines are then formed once for all heads.
  const long long ctas = 4LL * device_sm_count();
  if ((long long)a.T >= ctas) {
    while (a.groups > 1 && a.groups * KR_UNROLL * 2 > all) a.groups = (a.groups + 1) / 2;
    const int most = KR_THREADS / (a.items * a.groups);
    while (a.tokens < most && (long long)a.T >= ctas * (a.tokens + 1)) ++a.tokens;
  } else {
    split = (all + a.groups - 1) / a.groups;
    while (split > 1 && (long long)a.T * split > ctas) split = (split + 1) / 2;
  }
  auto kern = half ? kv_rotate_kernel<V, true> : kv_rotate_kernel<V, false>;
  // (no more threads than have work, so that more CTAs find room: 5,999 tokens, 16 heads of 64, 9.5 us with 256, 8.0)
  const int threads = (a.items * a.groups * a.tokens + 31) / 32 * 32;
  return launch_k(kern, dim3((unsigned)((a.T + a.tokens - 1) / a.tokens), (unsigned)split), dim3(threads),
                  (size_t)a.tokens * a.pairs * sizeof(float2), s, a);
}

}  // namespace

cudaError_t launch_kv_rotate(const RotateRows& q, const RotateRows& k, int D, const int32_t* pos, int T, const uint64_t* turns,
                             int pairs, float gain, int offset, bool interleaved, bool backward, cudaStream_t s) {
  RotateArgs a{};
  const RotateRows* r[2] = {&q, &k};
  bool whole = true;   // every row starts on 16 bytes
  for (int i = 0; i < 2; ++i) {
    a.in[i] = r[i]->in, a.out[i] = r[i]->out, a.in_stride[i] = r[i]->in_stride, a.out_stride[i] = r[i]->out_stride;
    a.heads[i] = r[i]->heads;
    if (r[i]->heads)
      whole &= (reinterpret_cast<uintptr_t>(a.in[i]) | reinterpret_cast<uintptr_t>(a.out[i])) % 16 == 0 &&
               (a.in_stride[i] | a.out_stride[i]) % 8 == 0;
  }
  a.D = D, a.pairs = pairs, a.offset = offset, a.T = T, a.pos = pos, a.turns = turns, a.gain = gain;
  a.sign = backward ? -1.0f : 1.0f;
  // the widest pieces into which the turning channels and the others divide
  const int cut = offset | D | (interleaved ? 2 * pairs : pairs);
  if (whole && cut % 8 == 0) return launch<8>(a, !interleaved, s);
  bool even = true;
  for (int i = 0; i < 2; ++i)
    if (a.heads[i])
      even &= (reinterpret_cast<uintptr_t>(a.in[i]) | reinterpret_cast<uintptr_t>(a.out[i])) % 4 == 0 &&
              (a.in_stride[i] | a.out_stride[i]) % 2 == 0;
  if (even && cut % 2 == 0) return launch<2>(a, !interleaved, s);
  return launch<1>(a, !interleaved, s);
}

// Radians a position of each pair in 64 bits, then whole numbers of 2^-64 turns.
bool rope_turns(int rot_dim, double theta, int scaling, double factor, double low, double high, double length,
                uint64_t* turns, float* gain) {
  const double pi2 = 6.283185307179586476925286766559;
  double base = theta;
  if (scaling == BRE_ROPE_BASE && rot_dim > 2) base = theta * std::pow(factor, rot_dim / (rot_dim - 2.0));
  const bool ramp = scaling == BRE_ROPE_RAMP || scaling == BRE_ROPE_RAMP_PAST;
  *gain = ramp && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  auto pair_of = [&](double n) { return rot_dim * std::log(length / (n * pi2)) / (2.0 * std::log(base)); };
  const double first = std::fmax(std::floor(ramp ? pair_of(high) : 0.0), 0.0);
  const double last = std::fmin(std::ceil(ramp ? pair_of(low) : 0.0), scaling == BRE_ROPE_RAMP_PAST ? rot_dim - 1.0 : rot_dim / 2 - 1.0);
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot_dim);
    if (scaling == BRE_ROPE_LINEAR) f /= factor;
    if (ramp) {
      const double r = std::fmin(std::fmax((i - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
      f = f / factor * r + f * (1.0 - r);
    }
    if (scaling == BRE_ROPE_BANDS) {
      const double w = std::fmin(std::fmax((length * f / pi2 - low) / (high - low), 0.0), 1.0);
      f = (1.0 - w) * f / factor + w * f;
    }
    const double t = f / pi2;   // whole turns do not count
    const double x = std::ldexp(t - std::floor(t), 64);
    if (!(x >= 0.0)) return false;   // NaN
    turns[i] = x < 0x1p64 ? (uint64_t)std::nearbyint(x) : 0;
  }
  return true;
}

}  // namespace bre

// What the attention kernels over the quantised cache share.
#pragma once
#include "kv_common.cuh"

namespace bre {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float P_SHIFT = 8.0f;   // weights are held times 2^8: FP16's normal range then reaches 2^-22 of the largest

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 2^x; results below 2^-126 become 0 (without .ftz the compiler adds two scalings to every one).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Weights are 2^(logit + ev) against their own maximum, ev the exponent of the value's scale; the sum of exponentials
// gets the factor 2^-ev back.  A weight that vanishes beside a value of another size still counts in that sum.
// While no value scale is above this byte no term within 2^-40 of the sum is lost (ev is -64 at least, 26 at most: a
// weight is above 2^-126 if its term is); from the first larger one on (values beyond 3 * 10^10; infinities have
// ev = 119) the sum's terms are formed without ev.
constexpr int EV_LARGE = 153;
// l * 2^d for d <= 0, where 2^d alone may vanish although l is large (sums are held relative to the weights' maximum).
__device__ __forceinline__ float scale_sum(float l, float d) {
  const float h = ex2(0.5f * d);
  return l * h * h;
}

struct AttendArgs {
  const uint8_t* pages;
  int H, G;
  KvTable tab;
  const uint16_t* q;
  long long q_stride;
  const int32_t* seq;
  const int32_t* pos;
  int T;
  const int32_t* ids;
  int k;
  float scale;
  uint16_t* out;
  float* lse;
  int32_t* err;
  long long wait;   // budget (cycles) of the tile kernel's waits where one is set
};

// 128 rows (tokens times query heads) at a time (kv_attend_tiles.cu)
cudaError_t launch_kv_attend_tiles(const AttendArgs& a, int D, cudaStream_t s);

}  // namespace bre

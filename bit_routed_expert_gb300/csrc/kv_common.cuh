// What the key/value cache kernels share: the page layout, the row codec and token lookup.
//
// A page holds KV_BLOCK consecutive tokens of one sequence.  For each of its key/value heads, in
// this order and without gaps: KV_BLOCK key rows of D E4M3 codes, KV_BLOCK value rows, KV_BLOCK
// key scales, KV_BLOCK value scales (E8M0, one byte a row).  A head's share of a page is one
// contiguous, 16-byte aligned piece of 128 D + 128 bytes, read and written in 8- and 16-byte pieces.
//
// One power-of-two scale a row, not one for every 32 channels: E4M3 carries an exponent itself,
// and against the row's largest value it keeps four significant bits down to 2^-14 of it, so a
// finer scale would only help values that hardly count in a dot product.  With one scale a row
// the key's scale multiplies a whole logit and the value's scale a whole probability: neither
// ever touches the tensor-core operands, which are the plain codes (exact in FP16).
#pragma once
#include "bre_common.cuh"
#include "kernels.h"

namespace bre {

constexpr int KV_BLOCK = 64;
constexpr int KV_EXP_MIN = -64;   // rows below 2^-56 are stored in steps of 2^-73
// Scale byte of a row that holds a NaN (E8M0's NaN); its codes are zeros and it reads as NaN throughout.
// With one byte to look at, no kernel has to look for NaN among the codes, and a NaN value cannot
// reach a row whose weight for it is zero through a matrix product.
constexpr int KV_NAN = 255;

__host__ __device__ constexpr int kv_page_bytes(int D) { return 2 * KV_BLOCK * D + 2 * KV_BLOCK; }

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// Smallest e >= KV_EXP_MIN with a <= m * 2^(bits + e), where a >= 0 and m = 1 + frac / 2^23.
__device__ __forceinline__ int least_exp(float a, int bits, int frac) {
  const int u = __float_as_int(a);
  const int e = (u >> 23) - 127 - bits + ((u & 0x7FFFFF) > frac ? 1 : 0);
  return max(e, KV_EXP_MIN);
}
__device__ __forceinline__ int row_exp(float amax) { return least_exp(amax, 8, 0x600000); }     // amax <= 448 * 2^e
__device__ __forceinline__ int bound_exp_of(float amax) { return least_exp(amax, 5, 0x7C0000); }   // <= 63 * 2^e
__device__ __forceinline__ int query_exp(float amax) { return least_exp(amax, 6, 0x7E0000); }      // <= 127 * 2^e

constexpr float KV_MAX = 0x1.cp127f;   // 448 * 2^119, the largest storable magnitude: larger values saturate

// Infinities count as the largest storable value; NaN stays.
__device__ __forceinline__ float kv_clamp(float x) { return x != x ? x : fminf(fmaxf(x, -KV_MAX), KV_MAX); }

// Two floats -> two E4M3 codes (low byte first), round to nearest even; |x| <= 448, NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes -> FP16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  return make_float2(f16_bits_to_f32(h & 0xFFFFu), f16_bits_to_f32(h >> 16));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 bytes at a 32-byte aligned address: whole sectors.
__device__ __forceinline__ void st_v8(uint16_t* dst, const uint32_t (&o)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]),
               "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}

// Thread-block clusters and distributed shared memory.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The float at `local`'s place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float ld_cluster_f32(const float* local, uint32_t rank) {
  uint32_t ra;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ra) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u32(const void* local, uint32_t rank, uint32_t v) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ra), "r"(v) : "memory");
}

// Page of block b of sequence s; -1 where there is none (a negative table entry), with the
// error bit where the sequence, the block or the page lies outside what the call was given.
struct KvTable {
  const int32_t* table;
  int B, N, n_pages;
};
__device__ __forceinline__ int kv_page(const KvTable& t, int s, int b, int32_t* err) {
  if ((unsigned)s >= (unsigned)t.B || (unsigned)b >= (unsigned)t.N) {
    set_err(err, BRE_DEVERR_PAGE);
    return -1;
  }
  const int p = __ldg(t.table + (size_t)s * t.N + b);
  if (p >= t.n_pages) {
    set_err(err, BRE_DEVERR_PAGE);
    return -1;
  }
  return p < 0 ? -1 : p;
}

}  // namespace bre

// attn_common.cuh -- parameters and row arithmetic shared by the attention
// kernels (attn_decode.cu, attn_prefill.cu, attn_mass.cu).
//
// Rows are counted as the cache holds them: the query of the i-th of n_new
// new tokens of a sequence sits at row r = n_valid - n_new + i of each of the
// layer's slices, and sees row j when j <= r and (no window, or j < n_sink, or
// j > r - window). The visible rows are therefore two runs, [0, s1) and
// [w0, r], with w0 = max(0, r + 1 - window) and s1 = min(n_sink, w0).
//
// Logits are kept in base 2: x = scale * log2(e) * (q . k), so that a weight is
// one ex2 and the log-sum is ln(2) * (m + log2(l)).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tri_internal.cuh"

namespace tri {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();

// 2^x by the hardware's approximation (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The runs of rows the query at row r sees (none for r < 0).
struct Visible {
  int s1;  // rows [0, s1)
  int w0;  // and [w0, r]
};
__device__ __forceinline__ Visible visible_rows(int r, int n_sink, int window) {
  if (r < 0) return {0, 0};
  if (window == 0) return {0, 0};
  const int w0 = max(0, r - window + 1);
  return {min(n_sink, w0), w0};
}

// Slice index of (seq, layer, head).
__device__ __forceinline__ int64_t slice_of(const AttnParams& p, int seq, int head) {
  return (static_cast<int64_t>(seq) * p.n_layers + p.layer) * p.n_kv_heads + head;
}

// New tokens of a sequence, or -1 (reported) when the count is malformed.
__device__ __forceinline__ int new_tokens(const AttnParams& p, int seq) {
  const int n = p.n_new ? __ldg(p.n_new + seq) : p.n_q;
  if (n < 0 || n > p.n_q) {
    set_status(p.dev_status, TRI_DEV_BAD_QUERY);
    return -1;
  }
  return n;
}

// 16 bytes global -> shared, zeros when not live; groups of a thread's copies.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Barrier over the cluster's CTAs (over the CTA when it is alone).
__device__ __forceinline__ void cluster_sync(int ns) {
  if (ns == 1) {
    __syncthreads();
    return;
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of CTA u of the cluster.
__device__ __forceinline__ float cluster_ld(const float* p, int u, int ns) {
  if (ns == 1) return *p;
  float x;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(x) : "r"(smem_addr(p)), "r"(u) : "memory");
  return x;
}
__device__ __forceinline__ float2 cluster_ld2(const float2* p, int u, int ns) {
  const float* f = reinterpret_cast<const float*>(p);
  return make_float2(cluster_ld(f, u, ns), cluster_ld(f + 1, u, ns));
}
__device__ __forceinline__ float4 cluster_ld4(const float4* p, int u, int ns) {
  if (ns == 1) return *p;
  float4 x;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(smem_addr(p)), "r"(u) : "memory");
  return x;
}

// (lo, hi) rounded to bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace
}  // namespace tri

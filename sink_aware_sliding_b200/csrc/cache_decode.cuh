// What the cluster decode kernels share: asynchronous copies into a warp's own
// ring of stages, the two matrix instructions, and the merge of partial softmax
// states over the warps of a block and the blocks of a cluster.
//
// One cluster of blocks works on one (sequence, KV head).  Its keys are cut into
// tiles of 16; warp w of the cluster takes the tiles w, w + n, w + 2 n, ...  Each
// warp copies its tiles into shared memory several tiles ahead (cp.async, no block
// barrier in the loop) and keeps (reference, sum, O) of its keys for up to eight
// query heads.  The partial states meet in shared memory, first over the warps,
// then over the cluster: no workspace, no second launch, and a sum whose order
// depends on the sizes alone.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace swa {

constexpr int kDecWarps = 4;    // warps per block
constexpr int kDecTile = 16;    // keys per tile
constexpr int kDecHeads = 8;    // query heads per KV head, at most

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool real) {
  const int n = real ? BYTES : 0;  // 0: the destination is filled with zeros, src is not read
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, A row g = head g (rows 8..15 are zero), fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Partial softmax state of the heads of one KV head.  The sums are relative to
// 2^ref: O = sum 2^(z - ref) v, l = sum 2^(z - ref); ref = -inf and l = 0 without keys.
template <int D>
struct Partial {
  float o[kDecHeads][D];
  float ref[kDecHeads];
  float l[kDecHeads];
};

// Weights of n partial states with references r[i] and sums l[i], and the total.
__device__ __forceinline__ float merge_ref(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float merge_weight(float ref, float top) {
  return ref == -INFINITY ? 0.f : exp2f(ref - top);
}

// Combine the warps' states (in shared memory, warp w's at part(w)) into `mine`, then
// the cluster's: rank r of `c` blocks writes its share of the output rows of segment
// `seg_head0` (index of the first query head).  On return lse2[h] (shared memory) is the
// log2 of the segment's sum of 2^z, -inf without keys.
template <int D, typename PartOf>
__device__ __forceinline__ void merge_and_store(PartOf part, Partial<D>* mine, float* lse2, int G, int c, int rank,
                                                size_t seg_head0, void* out, bool out_f32, float* lse) {
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x;
  constexpr int kThreads = kDecWarps * 32;
  __syncthreads();
  for (int i = tid; i < G * D; i += kThreads) {
    const int h = i / D, e = i % D;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, part(w)->ref[h]);
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float a = merge_weight(part(w)->ref[h], top);
      acc += a * part(w)->o[h][e];
      l += a * part(w)->l[h];
    }
    mine->o[h][e] = acc;
    if (e == 0) {
      mine->ref[h] = top;
      mine->l[h] = l;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (c > 1) cluster.sync(); else __syncthreads();
  for (int i = rank * kThreads + tid; i < G * D; i += c * kThreads) {
    const int h = i / D, e = i % D;
    float top = -INFINITY;
    for (int r = 0; r < c; ++r) top = fmaxf(top, cluster.map_shared_rank(mine, r)->ref[h]);
    float acc = 0.f, l = 0.f;
    for (int r = 0; r < c; ++r) {
      const Partial<D>* p = cluster.map_shared_rank(mine, r);
      const float a = merge_weight(p->ref[h], top);
      acc += a * p->o[h][e];
      l += a * p->l[h];
    }
    const float y = l > 0.f ? acc / l : (l == 0.f ? 0.f : l);  // a NaN sum stays one
    const size_t at = (seg_head0 + h) * D + e;
    if (out_f32)
      static_cast<float*>(out)[at] = y;
    else
      static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(y);
  }
  if (tid < G) {
    const int h = tid;
    float top = -INFINITY, l = 0.f;
    for (int r = 0; r < c; ++r) top = fmaxf(top, cluster.map_shared_rank(mine, r)->ref[h]);
    for (int r = 0; r < c; ++r) {
      const Partial<D>* p = cluster.map_shared_rank(mine, r);
      l += merge_weight(p->ref[h], top) * p->l[h];
    }
    const float s = l == 0.f ? -INFINITY : top + log2f(l);
    lse2[h] = s;
    if (rank == 0 && lse != nullptr) lse[seg_head0 + h] = s * 0.69314718055994531f;
  }
  // no block leaves, or reuses its shared memory, while another one reads it
  if (c > 1) cluster.sync(); else __syncthreads();
}

// Blocks per cluster: enough that `segments` fill the GPU about `waves` times over,
// but at least kDecWarps tiles for each block and at most 8 (the portable size).
inline int decode_cluster(long long segments, long long tiles, int sms, int blocks_per_sm, int waves) {
  int c = 1;
  while (c < 8 && segments * c < static_cast<long long>(sms) * blocks_per_sm * waves &&
         tiles >= 2LL * c * kDecWarps)
    c *= 2;
  return c;
}

}  // namespace swa

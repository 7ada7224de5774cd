// What the cluster decode kernels share: asynchronous copies into a warp's own
// ring of stages, the two matrix instructions, and the merge of partial softmax
// states over the warps of a block and the blocks of a cluster.
//
// One cluster of blocks works on one (sequence, KV head).  Its keys are cut into
// tiles; warp w of the cluster takes the tiles w, w + n, w + 2 n, ...  Each
// warp copies its tiles into shared memory one or two tiles ahead (cp.async, no block
// barrier in the loop) and keeps (reference, sum, O) of its keys for up to eight
// query heads.  The partial states meet in shared memory, first over the warps,
// then over the cluster: no workspace, no second launch, and a sum whose order
// depends on the sizes alone.
#pragma once
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fixed_cache.h"
#include "ptx.cuh"

namespace swa {

constexpr int kDecWarps = 4;    // warps per block
constexpr int kDecTile = 16;    // keys per product
constexpr int kDecHeads = 8;    // query heads per KV head, at most

// The caches' rows are read once a step, so they leave the L2 first: what the block
// needs again (positions, scores) stays (evicting cache, B = 64: 96.3 -> 93.0 us).
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool real, uint64_t policy) {
  const int n = real ? BYTES : 0;  // 0: the destination is filled with zeros, src is not read
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
                 "l"(policy)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %4, %2, %3;" ::"r"(dst), "l"(src), "r"(n),
                 "l"(policy), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D += A B, fp32 accumulators.  A's 16 rows are keys, or elements of V, and B's eight columns query heads.
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

// D = A B (no accumulator to clear first).
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Four 8 x 8 matrices of 16-bit elements, the rows of matrix i at the addresses of lanes 8 i .. 8 i + 7: what
// one m16n8k16 product takes as A, or, transposed on the way, what it takes from a tile stored the other way.
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Partial softmax state of the heads of one KV head.  The sums are relative to
// 2^ref: O = sum 2^(z - ref) v, l = sum 2^(z - ref); ref = -inf and l = 0 without keys.
template <int D>
struct alignas(16) Partial {
  float o[kDecHeads][D];
  float ref[kDecHeads];
  float l[kDecHeads];
};

__device__ __forceinline__ float merge_weight(float ref, float top) {
  return ref == -INFINITY ? 0.f : ex2_approx(ref - top);
}
__device__ __forceinline__ float4 axpy4(float a, float4 x, float4 y) {
  return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}

// Combine the warps' states (in shared memory, warp w's at part(w)) into `mine`, then
// the cluster's: rank r of `c` blocks writes its share of the output rows, head0 being
// the index of the segment's first query head.  Four elements a thread throughout, the
// weights once per thread and head.  On return lse2[h] (shared memory) is the log2 of
// the segment's sum of 2^z, -inf without keys; merge_done() has to follow before the end.
template <int D, typename PartOf>
__device__ __forceinline__ void merge_and_store(PartOf part, Partial<D>* mine, float* lse2, int G, int c, int rank,
                                                size_t head0, void* out, bool out_f32, float* lse) {
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x;
  constexpr int kThreads = kDecWarps * 32;
  constexpr int V = D / 4;  // float4s of a row
  __syncthreads();
  for (int i = tid; i < G * V; i += kThreads) {
    const int h = i / V, e = i % V;
    float w[kDecWarps], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kDecWarps; ++k) top = fmaxf(top, w[k] = part(k)->ref[h]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kDecWarps; ++k) {
      const float a = merge_weight(w[k], top);
      acc = axpy4(a, reinterpret_cast<const float4*>(part(k)->o[h])[e], acc);
      l = fmaf(a, part(k)->l[h], l);
    }
    reinterpret_cast<float4*>(mine->o[h])[e] = acc;
    if (e == 0) {
      mine->ref[h] = top;
      mine->l[h] = l;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (c > 1) cluster.sync(); else __syncthreads();
  // this rank's float4s, and every head's log-sum-exp
  const int share = (G * V + c - 1) / c;
  for (int i = tid; i < share + kDecHeads; i += kThreads) {
    const bool row = i < share;
    const int at = rank * share + i;
    const int h = row ? at / V : i - share, e = row ? at % V : 0;
    if (h >= G) continue;
    float top = -INFINITY, l = 0.f;
    for (int r = 0; r < c; ++r) top = fmaxf(top, cluster.map_shared_rank(mine, r)->ref[h]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < c; ++r) {
      const Partial<D>* p = cluster.map_shared_rank(mine, r);
      const float a = merge_weight(p->ref[h], top);
      if (row) acc = axpy4(a, reinterpret_cast<const float4*>(p->o[h])[e], acc);
      l = fmaf(a, p->l[h], l);
    }
    if (row) {
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no keys: zeros; a NaN sum stays one
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      const size_t o = (head0 + h) * D + 4 * e;
      if (out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = acc;
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + o) =
            make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
    } else {
      const float s = l == 0.f ? -INFINITY : top + log2f(l);
      lse2[h] = s;
      if (rank == 0 && lse != nullptr) lse[head0 + h] = s * 0.69314718055994531f;
    }
  }
  // lse2 is there for the whole block; merge_done() is for the other blocks' reads
  if (c > 1) cluster.barrier_arrive();
  __syncthreads();
}

// No block leaves, or reuses the shared memory of its states, while another one reads it.
__device__ __forceinline__ void merge_done(int c) {
  if (c > 1) cooperative_groups::this_cluster().barrier_wait();
}

// Launch with clusters of c blocks that may start while the kernel before them (the step's append, mostly) ends;
// they wait for it before they read anything.
template <typename Kernel, typename Args>
cudaError_t launch_decode_cluster(Kernel kernel, const Args& a, long long segments, int c, size_t smem,
                                  cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(segments * c));
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(c);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = c > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, c);
}

// Blocks per cluster: a power of two, enough that `segments` fill the GPU `waves` times over,
// but with two tiles for each warp and at most 8 (the portable size).  A second wave of few blocks is not looked
// at: 592 segments of the 4-bit decode (window 4096, d = 128) take 76 us and 600 take 94 us; of the evicting one 106
// and 113 us.
inline int decode_cluster(long long segments, long long tiles, int sms, int blocks_per_sm, int waves) {
  int c = 1;
  while (c < 8 && segments * c < static_cast<long long>(sms) * blocks_per_sm * waves &&
         tiles >= 2LL * c * kDecWarps)
    c *= 2;
  return c;
}

}  // namespace swa

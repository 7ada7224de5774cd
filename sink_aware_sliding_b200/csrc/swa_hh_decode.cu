// Decode over the cache that evicts by accumulated attention weight: softmax attention
// over the occupied slots, and each slot's weight added to its score, in one launch.
//
// Bound by HBM like the ring cache's decode: every row is read once.  S = Q K^T and
// O^T += V^T P^T run as mma.sync m16n8k16 on bf16 rows, as they are; P is split into
// two bf16 parts (hi + lo, 2^-17 relative together) at the price of a second product,
// since the weights are a result of their own here.  The scaled scores stay in shared
// memory (4 bytes a slot and query head, spread over the cluster's blocks), so that
// when the cluster has merged its sums, each block turns its slots' scores into
// weights and adds them up without a second pass over K.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_decode.cuh"
#include "fixed_cache.h"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStages = 3;

template <int D>
struct HB {
  static constexpr int UNITS = D / 8;                          // 16-byte units of a row
  static constexpr int HALF = kDecTile * D * 2;                // K's or V's bytes of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int COPIES = kDecTile * UNITS / 32;         // per lane, for K and again for V
  static constexpr int KS = D / 16;                            // k-steps of S
  static constexpr int MT = D / 16;                            // row tiles of O^T
};

// Unit u of row r lies at u ^ swz(r): the K reads of a quarter warp (rows q, q + 4, four
// neighbouring units) and the V reads (rows 0..3 or 4..7, two units) each fall on all
// 32 banks once.
__device__ __forceinline__ int swz(int r) { return ((r & 3) << 1) ^ (r & 4); }

// Blocks per cluster, and the shared memory of its blocks.
template <int D>
struct HhPlan {
  int c;
  size_t smem;
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// bf16 element e of a (low half) and of b
__device__ __forceinline__ uint32_t pair_of(const uint4& a, const uint4& b, int e) {
  return __byte_perm(word_of(a, e >> 1), word_of(b, e >> 1), (e & 1) ? 0x7632 : 0x5410);
}

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32, 2) swa_hh_decode_kernel(const __grid_constant__ HhDecodeArgs a,
                                                                         int c) {
  using C = HB<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Partial<D> s_mine;
  __shared__ float s_lse2[kDecHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % c;
  const size_t seg = blockIdx.x / c;
  const int b = static_cast<int>(seg / a.Hkv), kvh = static_cast<int>(seg % a.Hkv);
  const int G = a.G, cap = a.C;
  const size_t head0 = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(kvh) * G;
  const int tiles = (cap + kDecTile - 1) / kDecTile;
  const uint8_t* kc = static_cast<const uint8_t*>(a.kc) + seg * cap * (D * 2);
  const uint8_t* vc = static_cast<const uint8_t*>(a.vc) + seg * cap * (D * 2);
  const int32_t* sp = a.slot_pos + seg * cap;

  uint8_t* ring = smem + warp * (kStages * C::STAGE);
  const uint32_t ring_u32 = smem_u32(ring);
  float* s_z = reinterpret_cast<float*>(smem + kDecWarps * kStages * C::STAGE);  // [local tile][G][16]
  const int nw = c * kDecWarps;

  // Positions in a tile's slots, one per lane of a half warp, and the occupied ones as bits.
  // They are read a tile before the tile is requested, so that nothing waits for them.
  auto slots_of = [&](int tile) -> int {
    const int i = tile * kDecTile + (lane & 15);
    return tile < tiles && i < cap ? sp[i] : -1;
  };
  auto occupied = [&](int at) -> unsigned { return __ballot_sync(kFull, at >= 0) & 0xffffu; };
  auto issue = [&](int tile, int stage, unsigned mask) {
    if (mask != 0) {
      const uint8_t* ks = kc + static_cast<size_t>(tile) * kDecTile * (D * 2);
      const uint8_t* vs = vc + static_cast<size_t>(tile) * kDecTile * (D * 2);
      const uint32_t dst = ring_u32 + stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < C::COPIES; ++i) {
        const int u = lane + 32 * i;
        const int r = u / C::UNITS, unit = u % C::UNITS;
        const bool real = (mask >> r) & 1;
        const int off = real ? u * 16 : 0;
        const uint32_t at = (r * C::UNITS + (unit ^ swz(r & 7))) * 16;
        cp_async<16>(dst + at, ks + off, real);
        cp_async<16>(dst + C::HALF + at, vs + off, real);
      }
    }
    cp_async_commit();
  };

  int tile = rank * kDecWarps + warp;
  unsigned masks[kStages];  // of the tiles tile, tile + nw, ...
  int ahead;                // slots of the first tile that has no mask yet
  {
    int at[kStages];
#pragma unroll
    for (int s = 0; s < kStages; ++s) at[s] = slots_of(tile + s * nw);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      masks[s] = occupied(at[s]);
      issue(tile + s * nw, s, masks[s]);
    }
    ahead = at[kStages - 1];
  }

  // ---- q: row g of A is head g
  uint32_t qa[C::KS][2];
  {
    const bool real = g < G;
    const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + (head0 + (real ? g : 0)) * D;
#pragma unroll
    for (int s = 0; s < C::KS / 2; ++s) {
      const uint4 w = real ? *reinterpret_cast<const uint4*>(qrow + s * 32 + t * 8) : make_uint4(0, 0, 0, 0);
      qa[2 * s][0] = w.x; qa[2 * s][1] = w.y;
      qa[2 * s + 1][0] = w.z; qa[2 * s + 1][1] = w.w;
    }
  }
  float o[C::MT][4];
#pragma unroll
  for (int i = 0; i < C::MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ref = -INFINITY, l = 0.f;
  const int row_n = (g & 1) ? 4 + (g >> 1) : g >> 1;  // K: this lane's row of a score tile (and + 8)
  const int r0 = t, r1 = t + 4;                       // scores and V: this lane's rows (and + 8)

  int stage = 0, local = warp;
  for (; tile < tiles; tile += nw, local += kDecWarps) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    const unsigned mask = masks[0];
    masks[kStages - 1] = occupied(ahead);
    ahead = slots_of(tile + kStages * nw);
    issue(tile + (kStages - 1) * nw, stage == 0 ? kStages - 1 : stage - 1, masks[kStages - 1]);
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) masks[s] = masks[s + 1];
    if (mask != 0) {
      const uint8_t* kt = ring + stage * C::STAGE;
      const uint8_t* vt = kt + C::HALF;
      float z[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int s = 0; s < C::KS / 2; ++s) {
          const uint4 w = *reinterpret_cast<const uint4*>(
              kt + ((row_n + 8 * nt) * C::UNITS + ((4 * s + t) ^ swz(row_n))) * 16);
          mma_bf16_16816(acc[0], qa[2 * s][0], 0u, qa[2 * s][1], 0u, w.x, w.y);
          mma_bf16_16816(acc[1], qa[2 * s + 1][0], 0u, qa[2 * s + 1][1], 0u, w.z, w.w);
        }
        z[2 * nt] = (acc[0][0] + acc[1][0]) * a.scale_log2;
        z[2 * nt + 1] = (acc[0][1] + acc[1][1]) * a.scale_log2;
      }
      const int rows[4] = {r0, r1, r0 + 8, r1 + 8};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((mask >> rows[i]) & 1)) z[i] = -INFINITY;
      if (g < G) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s_z[(local * G + g) * kDecTile + rows[i]] = z[i];
      }
      float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      if (__any_sync(kFull, mx > ref)) {
        const float next = fmaxf(ref, mx);
        const float alpha = ref == -INFINITY ? 0.f : ex2_approx(ref - next);
        const float a0 = __shfl_sync(kFull, alpha, 8 * t), a1 = __shfl_sync(kFull, alpha, 8 * t + 4);
        ref = next;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          o[i][0] *= a0; o[i][1] *= a1; o[i][2] *= a0; o[i][3] *= a1;
        }
      }
      const float base = ref == -INFINITY ? 0.f : ref;
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(z[i] - base);
      l += (pr[0] + pr[1]) + (pr[2] + pr[3]);
      const uint32_t h0 = pack_bf16x2(pr[0], pr[1]), h1 = pack_bf16x2(pr[2], pr[3]);
      const uint32_t l0 = pack_bf16x2(pr[0] - __uint_as_float(h0 << 16), pr[1] - __uint_as_float(h0 & 0xffff0000u));
      const uint32_t l1 = pack_bf16x2(pr[2] - __uint_as_float(h1 << 16), pr[3] - __uint_as_float(h1 & 0xffff0000u));
      uint4 v[4][C::UNITS / 8];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < C::UNITS / 8; ++u)
          v[i][u] = *reinterpret_cast<const uint4*>(vt + (rows[i] * C::UNITS + ((8 * u + g) ^ swz(rows[i] & 7))) * 16);
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        // row g: element mt of unit g; row g + 8: of unit 8 + g (d = 128) or element 4 + mt (d = 64)
        const int e2 = D == 128 ? mt : 4 + mt;
        constexpr int u2 = D == 128 ? 1 : 0;
        const uint32_t v0 = pair_of(v[0][0], v[1][0], mt), v1 = pair_of(v[0][u2], v[1][u2], e2);
        const uint32_t v2 = pair_of(v[2][0], v[3][0], mt), v3 = pair_of(v[2][u2], v[3][u2], e2);
        mma_bf16_16816(o[mt], v0, v1, v2, v3, h0, h1);
        mma_bf16_16816(o[mt], v0, v1, v2, v3, l0, l1);
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncwarp();

  static_assert(sizeof(Partial<D>) <= kStages * C::STAGE, "a partial state fits a warp's stages");
  auto part = [&](int w) { return reinterpret_cast<Partial<D>*>(smem + w * (kStages * C::STAGE)); };
  Partial<D>* pt = part(warp);
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) {
    const int dA = g * 8 + mt, dB = D == 128 ? 64 + g * 8 + mt : g * 8 + 4 + mt;
    if (2 * t < G) {
      pt->o[2 * t][dA] = o[mt][0];
      pt->o[2 * t][dB] = o[mt][2];
    }
    if (2 * t + 1 < G) {
      pt->o[2 * t + 1][dA] = o[mt][1];
      pt->o[2 * t + 1][dB] = o[mt][3];
    }
  }
  if (t == 0) {
    pt->ref[g] = ref;
    pt->l[g] = l;
  }
  merge_and_store<D>(part, &s_mine, s_lse2, G, c, rank, head0, a.out, a.out_f32 != 0, a.lse);

  // ---- weights of this block's slots: block tile i is tile rank * kDecWarps + (i % kDecWarps) + (i / kDecWarps) * nw
  __syncthreads();
  float* sc = a.score + seg * cap;
  const int mine = tiles > rank * kDecWarps
                       ? (tiles - rank * kDecWarps + nw - 1) / nw * kDecWarps  // upper bound; checked below
                       : 0;
  for (int i = threadIdx.x; i < mine * kDecTile; i += kDecWarps * 32) {
    const int lt = i / kDecTile, r = i % kDecTile;
    const int slot = (rank * kDecWarps + lt % kDecWarps + lt / kDecWarps * nw) * kDecTile + r;
    if (slot < cap && sp[slot] >= 0) {
      float w = 0.f;
      for (int h = 0; h < G; ++h) w += ex2_approx(s_z[(lt * G + h) * kDecTile + r] - s_lse2[h]);
      sc[slot] = fmaf(a.decay, sc[slot], w);
    }
  }
}

template <int D>
cudaError_t launch_impl(const HhDecodeArgs& a, int sms, cudaStream_t stream) {
  using C = HB<D>;
  const long long segments = static_cast<long long>(a.B) * a.Hkv;
  const long long tiles = (a.C + kDecTile - 1) / kDecTile;
  int c = decode_cluster(segments, tiles, sms, 2, 2);
  constexpr size_t kRing = static_cast<size_t>(kDecWarps) * kStages * C::STAGE;
  auto smem_of = [&](int n) {  // the stages, and the scores of a block's tiles
    const long long local = (tiles + n * kDecWarps - 1) / (n * kDecWarps) * kDecWarps;
    return kRing + static_cast<size_t>(local) * a.G * kDecTile * 4;
  };
  constexpr size_t kMost = 220 * 1024;  // of 227 KB; the merge's static part is below 5 KB
  while (c < 8 && smem_of(c) > kMost) c *= 2;
  const size_t smem = smem_of(c);
  if (smem > kMost || segments * c > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(swa_hh_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kMost));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(segments * c));
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(c);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, swa_hh_decode_kernel<D>, a, c);
}

}  // namespace

cudaError_t launch_hh_decode(const HhDecodeArgs& a, int d, int sms, cudaStream_t stream) {
  return d == 128 ? launch_impl<128>(a, sms, stream) : launch_impl<64>(a, sms, stream);
}

}  // namespace swa

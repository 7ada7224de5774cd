// Decode over the cache that evicts by accumulated attention weight: softmax attention
// over the occupied slots, and each slot's weight added to its score, in one launch.
//
// Bound by HBM like the ring cache's decode: every row is read once.  S^T = K Q^T and
// O^T += V^T P^T run as mma.sync m16n8k16 on bf16 rows as they are, the tokens (then the
// elements) as the 16 rows of a product and up to eight query heads as its columns;
// ldmatrix delivers both operands, V's transposed on the way.  P is split into two bf16
// parts (hi + lo, 2^-17 relative together) at the price of a second product, since the
// weights are a result of their own here.  The scaled scores stay in shared memory
// (4 bytes a slot and query head, spread over the cluster's blocks), where they are also
// turned from the first product's layout to the second's; when the cluster has merged
// its sums, each block makes weights of its slots' scores and adds them up, without a
// second pass over K; the scores to add to are read at the block's start.
// B = 64, 8 KV heads, 4 query heads each, d = 128, 2048 slots (550 MB): 94 us, 5.9 TB/s,
// 89% of a copy's rate.  With the heads as rows of the products 180 us (one block on an SM),
// with the scores read after the loop 106 us, without the L2 policy 96 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_decode.cuh"
#include "fixed_cache.h"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStages = 3;  // two tiles on their way: 128 KB on an SM of eight warps

template <int D>
struct HB {
  static constexpr int UNITS = D / 8;                          // 16-byte units of a row
  static constexpr int HALF = kDecTile * D * 2;                // K's or V's bytes of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int COPIES = kDecTile * UNITS / 32;         // per lane, for K and again for V
  static constexpr int KS = D / 16;                            // k-steps of S
  static constexpr int MT = D / 16;                            // row tiles of O^T
};

// In shared memory unit u of row r lies at u ^ (r & 7), so that the eight rows of a matrix
// that ldmatrix reads lie in different banks.
template <int D>
__global__ void __launch_bounds__(kDecWarps * 32, 2) swa_hh_decode_kernel(const __grid_constant__ HhDecodeArgs a,
                                                                         int c) {
  using C = HB<D>;
  extern __shared__ __align__(128) uint8_t smem[];
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
  float* s_z = reinterpret_cast<float*>(smem + kDecWarps * kStages * C::STAGE);  // [local tile][16][G]
  const int nw = c * kDecWarps;

  // Positions in a tile's slots, one per lane of a half warp, and the occupied ones as bits.
  // They are read a tile before the tile is requested, so that nothing waits for them.
  auto slots_of = [&](int tile) -> int {
    const int i = tile * kDecTile + (lane & 15);
    return tile < tiles && i < cap ? sp[i] : -1;
  };
  auto occupied = [&](int at) -> unsigned { return __ballot_sync(kFull, at >= 0) & 0xffffu; };
  const uint64_t policy = stream_policy();
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
        const uint32_t at = (r * C::UNITS + (unit ^ (r & 7))) * 16;
        cp_async<16>(dst + at, ks + off, real, policy);
        cp_async<16>(dst + C::HALF + at, vs + off, real, policy);
      }
    }
    cp_async_commit();
  };

  wait_for_previous_kernel();
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

  // ---- this block's slots: block tile i is tile rank * kDecWarps + i % kDecWarps + i / kDecWarps * nw.  The
  // first ones' positions and scores are read here, long before they are wanted, and stay in registers.
  const int first_tile = rank * kDecWarps;
  const int mine = tiles > first_tile ? (tiles - first_tile + nw - 1) / nw * kDecWarps * kDecTile : 0;  // or fewer
  float* sc = a.score + seg * cap;
  constexpr int kBatch = 8;  // slots a thread has in flight
  constexpr int kThreads = kDecWarps * 32;
  auto slot_at = [&](int i) {
    const int lt = i / kDecTile;
    return (first_tile + lt % kDecWarps + lt / kDecWarps * nw) * kDecTile + i % kDecTile;
  };
  int at_pos[kBatch];
  float old[kBatch];
  auto read_scores = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      const int at = slot_at(i);
      at_pos[k] = -1;
      if (i < mine && at < cap) {
        old[k] = sc[at];
        at_pos[k] = sp[at];
      }
    }
  };
  read_scores(threadIdx.x);

  // ---- q: column g of B is head g
  uint32_t qb[C::KS][2];
  {
    const bool real = g < G;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                             (head0 + (real ? g : 0)) * D);
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      qb[s][0] = real ? qrow[8 * s + t] : 0u;
      qb[s][1] = real ? qrow[8 * s + 4 + t] : 0u;
    }
  }
  float o[C::MT][4];
#pragma unroll
  for (int i = 0; i < C::MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float ref = -INFINITY, l = 0.f;
  // This lane's row of the matrices that ldmatrix reads.  K: matrices (rows 0-7, 8-15) x (unit
  // 2s, 2s + 1); V: (unit 2i, 2i + 1) x (rows 0-7, 8-15), transposed.
  const int km_row = lane & 15, km_unit = lane >> 4;
  const int vm_row = (lane & 7) + ((lane >> 4) << 3), vm_unit = (lane >> 3) & 1;
  const uint32_t km_at = km_row * C::UNITS * 16, vm_at = C::HALF + vm_row * C::UNITS * 16;

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
      const uint32_t tile_u32 = ring_u32 + stage * C::STAGE;
      float acc[2][4];
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint32_t k4[4];
        ldmatrix_x4(k4, tile_u32 + km_at + (((2 * s + km_unit) ^ (km_row & 7)) << 4));
        if (s < 2)
          mma_bf16_zero(acc[s], k4[0], k4[1], k4[2], k4[3], qb[s][0], qb[s][1]);
        else
          mma_bf16_16816(acc[s & 1], k4[0], k4[1], k4[2], k4[3], qb[s][0], qb[s][1]);
      }
      // rows g, g + 8 and heads 2t, 2t + 1, to be read back as head g and rows 2t, 2t + 1 and those + 8
      float* zt = s_z + static_cast<size_t>(local) * kDecTile * G;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * t + (i & 1) < G) zt[(g + (i >> 1) * 8) * G + 2 * t + (i & 1)] = (acc[0][i] + acc[1][i]) * a.scale_log2;
      __syncwarp();
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * t + (i & 1) + (i >> 1) * 8;
        z[i] = g < G && ((mask >> row) & 1) ? zt[row * G + g] : -INFINITY;
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
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        uint32_t v4[4];
        ldmatrix_x4_trans(v4, tile_u32 + vm_at + (((2 * mt + vm_unit) ^ (vm_row & 7)) << 4));
        mma_bf16_16816(o[mt], v4[0], v4[1], v4[2], v4[3], h0, h1);
        mma_bf16_16816(o[mt], v4[0], v4[1], v4[2], v4[3], l0, l1);
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncwarp();

  static_assert(2 * sizeof(Partial<D>) <= kStages * C::STAGE, "a warp's state and the block's fit a warp's stages");
  auto part = [&](int w) { return reinterpret_cast<Partial<D>*>(smem + w * (kStages * C::STAGE)); };
  Partial<D>* pt = part(warp);
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt) {
    const int dA = 16 * mt + g, dB = dA + 8;
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
  merge_and_store<D>(part, part(0) + 1, s_lse2, G, c, rank, head0, a.out, a.out_f32 != 0, a.lse);
  float top[kDecHeads];
#pragma unroll
  for (int h = 0; h < kDecHeads; ++h) top[h] = h < G ? s_lse2[h] : 0.f;
  for (int i0 = threadIdx.x; i0 < mine; i0 += kBatch * kThreads) {
    if (i0 != threadIdx.x) read_scores(i0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (at_pos[k] < 0) continue;
      const float* z = s_z + static_cast<size_t>(i0 + k * kThreads) * G;
      float w = 0.f;
      if ((G & 3) == 0) {
#pragma unroll
        for (int h = 0; h < kDecHeads; h += 4)
          if (h < G) {
            const float4 x = *reinterpret_cast<const float4*>(z + h);
            w += (ex2_approx(x.x - top[h]) + ex2_approx(x.y - top[h + 1])) +
                 (ex2_approx(x.z - top[h + 2]) + ex2_approx(x.w - top[h + 3]));
          }
      } else {
#pragma unroll
        for (int h = 0; h < kDecHeads; ++h)
          if (h < G) w += ex2_approx(z[h] - top[h]);
      }
      sc[slot_at(i0 + k * kThreads)] = fmaf(a.decay, old[k], w);
    }
  }
  merge_done(c);
}

template <int D>
cudaError_t launch_impl(const HhDecodeArgs& a, int sms, cudaStream_t stream) {
  using C = HB<D>;
  const long long segments = static_cast<long long>(a.B) * a.Hkv;
  const long long tiles = (a.C + kDecTile - 1) / kDecTile;
  // 512 segments: 105 us with two blocks each, 118 us with four, whose starts and merges weigh more
  int c = decode_cluster(segments, tiles, sms, 2, 2);
  constexpr size_t kRing = static_cast<size_t>(kDecWarps) * kStages * C::STAGE;
  auto smem_of = [&](int n) {  // the stages, and the scores of a block's tiles
    const long long local = (tiles + n * kDecWarps - 1) / (n * kDecWarps) * kDecWarps;
    return kRing + static_cast<size_t>(local) * a.G * kDecTile * 4;
  };
  constexpr size_t kMost = 226 * 1024, kTwo = 112 * 1024;  // one block's on an SM, and each of two blocks'
  while (c < 8 && smem_of(c) > kTwo) c *= 2;
  const size_t smem = smem_of(c);
  if (smem > kMost || segments * c > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = allow_shared<swa_hh_decode_kernel<D>>(static_cast<int>(kMost));
  if (e != cudaSuccess) return e;
  return launch_decode_cluster(swa_hh_decode_kernel<D>, a, segments, c, smem, stream);
}

}  // namespace

cudaError_t launch_hh_decode(const HhDecodeArgs& a, int d, int sms, cudaStream_t stream) {
  return d == 128 ? launch_impl<128>(a, sms, stream) : launch_impl<64>(a, sms, stream);
}

}  // namespace swa

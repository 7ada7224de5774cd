// Attention weight that the keys of a prompt received from its last queries:
//     score[j] = sum over observing queries t and query heads g of exp(scale q_tg . k_j - lse_tg).
//
// Only column sums are wanted and the rows' log-sum-exps are known, so there is no
// running softmax and no second product: a work unit is one tile of 128 keys of one
// (sequence, KV head), its K tile is loaded once, and the tiles of 128 observing queries
// of each head stream past it.  S^T = K Q^T runs on tcgen05 with the keys as the 128
// TMEM lanes: a thread owns one key and adds up its row of exponentials, without any
// exchange between threads.  Four S tiles in TMEM and four warpgroups that take every
// fourth tile keep the exponentials, which bound the kernel (16 a cycle and SM against
// 4096 multiply-adds: at d = 128 twice the product's time), from waiting for products.
// Sums: float32 over a tile's 128 columns in four chains, float64 over the tiles.
// 512 queries on 32768 keys, 32 heads on 8, d = 128 (136 GFLOP, 5.4e8 exponentials): 162 us at
// 1.96 GHz (2 us of them for the polynomial's upper bound), 185 us at the 1.7 GHz of the power cap.
// The products would take 82 us; with three quarters of the exponentials on it ex2 would take 86 us
// (XU pipe 63% busy, issue slots 58%).  What is left is waiting for long loads, over a third of all
// stalls: tensor memory's, and the next tile's log-sum-exps.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "fixed_cache.h"
#include "hh_scores.h"
#include "prefill_common.cuh"
#include "ptx.cuh"

namespace swa {
namespace {

using prefill::Ctl;
using prefill::wait_bar;

constexpr int kGroups = 4;     // warpgroups of exponentials (2: 182 us, 3: 163, 4: 158)
constexpr int kThreads = 128 * kGroups + 64;  // and a load warp, an MMA warp
constexpr int kLoadWarp = 4 * kGroups, kMmaWarp = kLoadWarp + 1;
constexpr int kBuf = 4;        // S tiles in TMEM
constexpr int kQStages = 3;

template <int D>
struct Cfg {
  static constexpr int TILE = 128 * D * 2;                // bytes of a K or Q tile
  static constexpr int NCHUNK = D / 64;                   // 128-byte columns of a tile
  static constexpr int OFF_K = 0;                         // two K tiles
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_LSE = OFF_Q + kQStages * TILE;   // [4 kGroups warps][128] floats
  static constexpr int OFF_SUM = OFF_LSE + 4 * kGroups * 128 * 4;  // [kGroups - 1][128] doubles
  static constexpr int OFF_BAR = OFF_SUM + (kGroups - 1) * 128 * 8;
  static constexpr int NBAR = 4 + 2 * kQStages + 2 * kBuf + 3;
  static constexpr int SMEM = OFF_BAR + 8 * NBAR + 16 + 1024;
};

// 2^x for two x on the multiply-add pipe: x = n + f with n the nearest integer, a polynomial of degree 5 in f (a
// fit of its own, minimax in relative error on [-1/2, 1/2]: 2.4e-7 with its float32 rounding), times 2^n.  Below
// 2^-126 the result is 2^-126, above 2^127.5 infinity (n = 128 has an infinity's bits); a NaN stays one.
__device__ __forceinline__ float clamp_nan(float x) {
  asm("max.NaN.f32 %0, %0, %1;\n\tmin.NaN.f32 %0, %0, %2;" : "+f"(x) : "f"(-126.f), "f"(128.f));
  return x;
}
__device__ __forceinline__ uint64_t exp2_pair(float x0, float x1) {
  auto both = [](float v) { return f2_pack(v, v); };
  constexpr float kRound = 12582912.f + 127.f;  // 1.5 * 2^23 and the exponent's bias: the sum's low bits are n + 127
  const uint64_t x = f2_pack(clamp_nan(x0), clamp_nan(x1));
  const uint64_t r = f2_add(x, both(kRound));
  const uint64_t f = f2_add(x, f2_mul(f2_add(r, both(-kRound)), both(-1.f)));
  uint64_t p = f2_fma(both(0.0013276472454890609f), f, both(0.009675540961325169f));
  p = f2_fma(p, f, both(0.05550713092088699f));
  p = f2_fma(p, f, both(0.24022120237350464f));
  p = f2_fma(p, f, both(0.6931469440460205f));
  p = f2_fma(p, f, both(1.0000001192092896f));
  float r0, r1;
  f2_unpack(r, r0, r1);
  return f2_mul(p, f2_pack(__uint_as_float(__float_as_uint(r0) << 23), __uint_as_float(__float_as_uint(r1) << 23)));
}
// Of every kPolyOf pairs of columns one goes that way and the others through ex2, so that neither pipe waits
// for the other (512 queries on 32768 keys, d = 128, 32 heads on 8: none 175 us, one of 2 184, of 3 161, of 4 158,
// of 6 158).
constexpr int kPolyOf = 4;

// One tile of keys of (b, kvh) and the observing queries that see any of them.
struct Unit {
  int b, kvh, j0, qt_lo, n_qt;
};

__device__ __forceinline__ Unit get_unit(const HhScoresArgs& a, int u) {
  Unit x;
  const int segs = a.pa.n_seq * a.pa.Hkv;
  const int seg = u % segs;
  x.b = seg / a.pa.Hkv;
  x.kvh = seg % a.pa.Hkv;
  x.j0 = u / segs * 128;
  const int L = a.pa.L, t_first = L - a.n_obs;
  const int j1 = min(x.j0 + 127, L - 1);
  const int lo = max(t_first, x.j0);                                    // first query that sees a key here
  const int hi = x.j0 < a.pa.n_sink ? L - 1 : min(L - 1, j1 + a.pa.window - 1);  // last one; window <= L
  x.qt_lo = (lo - t_first) / 128;
  x.n_qt = hi < lo ? 0 : (hi - t_first) / 128 - x.qt_lo + 1;
  return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    swa_hh_scores_kernel(const __grid_constant__ HhScoresArgs a, const __grid_constant__ CUtensorMap tq,
                         const __grid_constant__ CUtensorMap tk) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint32_t bar = base + C::OFF_BAR;
  const uint32_t k_full = bar, k_empty = bar + 16, q_full = bar + 32, q_empty = q_full + 8 * kQStages,
                 s_full = q_empty + 8 * kQStages, s_empty = s_full + 8 * kBuf, sum_full = s_empty + 8 * kBuf, sum_empty = sum_full + 8, drain = sum_full + 16;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(gbase + C::OFF_BAR + 8 * C::NBAR);
  Ctl ctl{reinterpret_cast<volatile int*>(gbase + C::OFF_BAR + 8 * C::NBAR + 4), &a.pa};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
    }
    for (int i = 0; i < kBuf; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(s_empty + 8 * i, 128);
    }
    mbar_init(sum_full, 128 * (kGroups - 1));
    mbar_init(sum_empty, 128);
    mbar_init(drain, 1);
    *ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base;
  const int G = a.pa.G, L = a.pa.L;
  const int t_first = L - a.n_obs;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      int uc = 0, n = 0;  // units with work, Q tiles
      bool ok = (a.pa.debug_flags & 1) == 0;
      for (int u = blockIdx.x; ok && u < a.n_units; u += gridDim.x) {
        const Unit x = get_unit(a, u);
        if (x.n_qt == 0) continue;
        const int kb = uc & 1;
        if (!(ok = wait_bar(k_empty + 8 * kb, ((uc >> 1) & 1) ^ 1, ctl))) break;
        mbar_expect_tx(k_full + 8 * kb, C::TILE);
        for (int c = 0; c < C::NCHUNK; ++c)
          tma_load_3d(base + C::OFF_K + kb * C::TILE + c * (128 * 128), &tk, k_full + 8 * kb, c * 64, x.kvh,
                      x.b * L + x.j0);
        ++uc;
        for (int h = 0; ok && h < G; ++h)
          for (int i = 0; i < x.n_qt; ++i, ++n) {
            const int st = n % kQStages;
            if (!(ok = wait_bar(q_empty + 8 * st, ((n / kQStages) & 1) ^ 1, ctl))) break;
            mbar_expect_tx(q_full + 8 * st, C::TILE);
            for (int c = 0; c < C::NCHUNK; ++c)
              tma_load_3d(base + C::OFF_Q + st * C::TILE + c * (128 * 128), &tq, q_full + 8 * st, c * 64,
                          x.kvh * G + h, x.b * L + t_first + (x.qt_lo + i) * 128);
          }
      }
      // Copies in flight land before the block ends, whether or not anyone has given up by now: another warp
      // still may, after this one is through with its list.
      for (int i = max(0, uc - 2); i < uc; ++i) wait_bar(k_full + 8 * (i & 1), (i >> 1) & 1, ctl, false);
      for (int i = max(0, n - kQStages); i < n; ++i)
        wait_bar(q_full + 8 * (i % kQStages), (i / kQStages) & 1, ctl, false);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      constexpr uint32_t kIdesc = make_idesc(1u, 128, 128, false);
      int uc = 0, n = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < a.n_units; u += gridDim.x) {
        const Unit x = get_unit(a, u);
        if (x.n_qt == 0) continue;
        const int kb = uc & 1;
        if (!(ok = wait_bar(k_full + 8 * kb, (uc >> 1) & 1, ctl))) break;
        const uint32_t ks = base + C::OFF_K + kb * C::TILE;
        const int count = x.n_qt * G;
        for (int i = 0; i < count; ++i, ++n) {
          const int st = n % kQStages, sb = n & (kBuf - 1);
          if (!(ok = wait_bar(s_empty + 8 * sb, ((n / kBuf) & 1) ^ 1, ctl))) break;
          if (!(ok = wait_bar(q_full + 8 * st, (n / kQStages) & 1, ctl))) break;
          tc_fence_after();
          const uint32_t qs = base + C::OFF_Q + st * C::TILE;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
            umma_ss<false>(tmem + 128 * sb, smem_desc(ks + off, 16, 1024, kLayoutSw128),
                           smem_desc(qs + off, 16, 1024, kLayoutSw128), kIdesc, kk > 0 ? 1u : 0u);
          }
          tc_commit(s_full + 8 * sb);
          tc_commit(q_empty + 8 * st);
        }
        if (ok) tc_commit(k_empty + 8 * kb);
        ++uc;
      }
      tc_commit(drain);  // every product issued is done before TMEM is freed, as above
      wait_bar(drain, 0, ctl, false);
    }
    __syncwarp();
  } else {
    const int wg = warp >> 2, row = tid & 127;
    float* lse = reinterpret_cast<float*>(gbase + C::OFF_LSE) + warp * 128;
    double* s_sum = reinterpret_cast<double*>(gbase + C::OFF_SUM);
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint64_t sl2 = f2_pack(a.pa.scale_log2, a.pa.scale_log2);
    int n = 0, uc = 0;
    bool ok = true;
    // lse of the next tile of this warpgroup, four columns a lane, on its way while the current
    // tile is worked on (tile i of unit x)
    float ahead[4];
    auto fetch = [&](const Unit& x, int i) {
      const int h = i / x.n_qt, t0 = t_first + (x.qt_lo + i - h * x.n_qt) * 128;
      const float* src = a.lse + (static_cast<size_t>(x.b) * a.pa.Hq + x.kvh * G + h) * L + t0;
#pragma unroll
      for (int c = 0; c < 4; ++c) ahead[c] = t0 + lane + 32 * c < L ? src[lane + 32 * c] : 0.f;
    };
    Unit x = get_unit(a, blockIdx.x);  // the grid has no more blocks than units
    if (wg < x.n_qt * G) fetch(x, wg);
    for (int u = blockIdx.x; ok && u < a.n_units; u += gridDim.x, ++uc) {
      const Unit next = get_unit(a, min(u + static_cast<int>(gridDim.x), a.n_units - 1));
      const int j = x.j0 + row;
      // queries that see key j: [j, last]
      const int last = j >= L ? -1 : j < a.pa.n_sink ? L - 1 : min(L - 1, j + a.pa.window - 1);
      const int count = x.n_qt * G;
      double total = 0.0;
      // tiles of all units are numbered through; this warpgroup takes one of kGroups
      const int first = (wg + kGroups - n % kGroups) % kGroups;
      const int first_next = (wg + kGroups - (n + count) % kGroups) % kGroups;
      if (first >= count && first_next < next.n_qt * G) fetch(next, first_next);  // none here
      for (int i = first; i < count; i += kGroups) {
        const int t0 = t_first + (x.qt_lo + i % x.n_qt) * 128;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) lse[lane + 32 * c] = ahead[c] * -1.4426950408889634f;  // this warp's own copy
        __syncwarp();
        if (i + kGroups < count) {
          fetch(x, i + kGroups);
        } else if (first_next < next.n_qt * G) {
          fetch(next, first_next);
        }
        const int sb = (n + i) & (kBuf - 1);
        ok = __all_sync(0xffffffffu, wait_bar(s_full + 8 * sb, ((n + i) / kBuf) & 1, ctl));
        if (!ok) break;
        tc_fence_after();
        // every key here sees every query of the tile?
        const bool whole = x.j0 + 127 <= t0 && t0 + 127 < L &&
                           (t0 + 127 <= x.j0 + a.pa.window - 1 || x.j0 + 127 < a.pa.n_sink);
        const int c_lo = j - t0, c_hi = last - t0;
        uint64_t part0 = 0, part1 = 0;  // two sums each
        // two loops, so that a tile without an edge has no comparisons
        auto add = [&](auto edge) {
#pragma unroll
          for (int c0 = 0; c0 < 128; c0 += 32) {
            uint32_t r[32];
            tmem_ld32_wait(tmem + 128 * sb + lane_off + c0, r);
            if (c0 == 96) {
              tc_fence_before();
              mbar_arrive(s_empty + 8 * sb);
            }
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 w = *reinterpret_cast<const float4*>(lse + c0 + c);
              float e[4];
              f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sl2, f2_pack(w.x, w.y)),
                        e[0], e[1]);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), sl2,
                               f2_pack(w.z, w.w)),
                        e[2], e[3]);
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                if (((c0 + c + q) / 2) % kPolyOf == kPolyOf - 1) {
                  f2_unpack(exp2_pair(e[q], e[q + 1]), e[q], e[q + 1]);
                } else {
                  e[q] = ex2_approx(e[q]);
                  e[q + 1] = ex2_approx(e[q + 1]);
                }
              }
              if constexpr (decltype(edge)::value) {
#pragma unroll
                for (int q = 0; q < 4; ++q) e[q] = (c0 + c + q >= c_lo && c0 + c + q <= c_hi) ? e[q] : 0.f;
              }
              part0 = f2_add(part0, f2_pack(e[0], e[1]));
              part1 = f2_add(part1, f2_pack(e[2], e[3]));
            }
          }
        };
        if (whole)
          add(std::false_type{});
        else
          add(std::true_type{});
        float s0, s1;
        f2_unpack(f2_add(part0, part1), s0, s1);
        total += static_cast<double>(s0 + s1);
      }
      n += count;
      if (!ok) break;
      // the warpgroups' sums; bounded waits, so that an abort ends them too
      if (wg > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(sum_empty, (uc & 1) ^ 1, ctl));
        if (!ok) break;
        s_sum[(wg - 1) * 128 + row] = total;
        mbar_arrive(sum_full);
      } else {
        ok = __all_sync(0xffffffffu, wait_bar(sum_full, uc & 1, ctl));
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < kGroups - 1; ++w) total += s_sum[w * 128 + row];
        mbar_arrive(sum_empty);
        if (j < L) a.score[(static_cast<size_t>(x.b) * a.pa.Hkv + x.kvh) * L + j] = static_cast<float>(total);
      }
      x = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_impl(const HhScoresArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, int grid,
                        cudaStream_t stream) {
  auto kern = swa_hh_scores_kernel<D>;
  static_assert(Cfg<D>::SMEM <= 232448, "shared memory budget");
  cudaError_t e = allow_shared<swa_hh_scores_kernel<D>>(Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, Cfg<D>::SMEM, stream>>>(a, tq, tk);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_hh_scores(const HhScoresArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, int d, int grid,
                             cudaStream_t stream) {
  return d == 128 ? launch_impl<128>(a, tq, tk, grid, stream) : launch_impl<64>(a, tq, tk, grid, stream);
}

}  // namespace swa

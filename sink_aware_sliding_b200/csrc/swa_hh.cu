// Cache of fixed capacity that evicts by accumulated attention weight: filling it from
// a prompt, and appending one token to it.
//
// Both choose by (class, score, index) with a total order on float32 scores: the bits
// of a float, the sign flipped for positive and all bits for negative ones, order like
// the values; -0 counts as 0 and a NaN as the lowest.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fixed_cache.h"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ uint32_t order_bits(float s) {
  if (s != s) return 0u;
  const uint32_t u = __float_as_uint(s + 0.f);  // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// ---------------------------------------------------------------- append
// One block per (b, KV head): the smallest of (class, score, slot) over the slots, where
// class is 0 for the slot of this very position, 1 for an empty one, 2 for one that may
// go and 3 for the others; then the row is written.
constexpr int kAppendThreads = 256;
__global__ void __launch_bounds__(kAppendThreads)
    swa_hh_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, const int32_t* __restrict__ pos,
                         uint4* kc, uint4* vc, int32_t* slot_pos, float* score, int32_t* slot, int Hkv, int vec,
                         int C, int S, int recent) {
  __shared__ unsigned long long s_best[kAppendThreads / 32];
  let_next_kernel_start();
  const size_t seg = blockIdx.x;
  const int p = pos[seg / Hkv];
  if (p < 0) {
    if (threadIdx.x == 0 && slot != nullptr) slot[seg] = -1;
    return;
  }
  const int32_t* sp = slot_pos + seg * C;
  const float* sc = score + seg * C;
  unsigned long long best = ~0ull;
  for (int i = threadIdx.x; i < C; i += kAppendThreads) {
    const int at = sp[i];
    const uint32_t bits = order_bits(sc[i]);
    const bool may = at >= S && at <= p - recent;
    const unsigned cls = at == p ? 0u : at < 0 ? 1u : may ? 2u : 3u;
    // class in 2 bits, score in 32, slot in 30
    const unsigned long long key = (static_cast<unsigned long long>(cls) << 62) |
                                   (static_cast<unsigned long long>(cls < 2 ? 0u : bits) << 30) |
                                   static_cast<unsigned>(i);
    best = min(best, key);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(kFull, best, o));
  if ((threadIdx.x & 31) == 0) s_best[threadIdx.x >> 5] = best;
  __syncthreads();
  best = s_best[0];
#pragma unroll
  for (int w = 1; w < kAppendThreads / 32; ++w) best = min(best, s_best[w]);
  const int i = static_cast<int>(best & 0x3fffffffu);
  const size_t row = (seg * C + i) * vec;
  if (threadIdx.x < vec) kc[row + threadIdx.x] = k[seg * vec + threadIdx.x];
  else if (threadIdx.x < 2 * vec) vc[row + threadIdx.x - vec] = v[seg * vec + threadIdx.x - vec];
  if (threadIdx.x == 0) {
    slot_pos[seg * C + i] = p;
    score[seg * C + i] = 0.f;
    if (slot != nullptr) slot[seg] = i;
  }
}

// ---------------------------------------------------------------- fill
// Select: one block per (b, KV head).  The first S and the last `recent` positions get a key
// above all scores; the largest of the other keys that have room are found by a radix select
// (11, 11 and 10 bits, histograms in shared memory): afterwards `cut` is the smallest kept key
// and `ties` how many positions with exactly that key are kept, the earlier ones first.  Each
// warp then walks one contiguous stretch of positions, so that the kept ones come out in ascending
// order after a prefix over the warps.  The keys are read from global memory once, all loads
// in flight, and stay in shared memory for the five walks over them, four keys a thread and
// step: the walks are what one SM can issue (four prompts of 16384, 8 heads: 28 us with every
// walk in global memory, 13.5 us with a key a step, 11.5 us so; a cluster of blocks per head,
// which has to add up their histograms, 37 us).  Copying the rows takes as long again.  Longer
// prompts go by global memory.
constexpr int kFillThreads = 1024;
constexpr int kFillWarps = kFillThreads / 32;
constexpr int kFillKeys = 49152;  // keys in shared memory (192 KB)

// Sum of `mine` over the threads before this one (all threads take part).
__device__ __forceinline__ unsigned block_prefix(unsigned mine, unsigned* s_warp, int lane, int warp) {
  unsigned incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  return __reduce_add_sync(kFull, lane < warp ? s_warp[lane] : 0u) + incl - mine;
}

// The rows of a cache to fill; `here`: the selecting block copies them itself.
struct FillRows {
  const uint4* k;
  const uint4* v;
  uint4* kc;
  uint4* vc;
  int Hkv, vec, kept;
  bool here;
};

// Copies the 16 bytes number first, first + step, ... of a (b, KV head)'s chosen rows, K's and V's.
__device__ __forceinline__ void copy_rows(const FillRows& f, size_t seg, int L, int C, const int32_t* sp, int first,
                                          int step) {
  const size_t src0 = (seg / f.Hkv * L * f.Hkv + seg % f.Hkv) * f.vec, dst0 = seg * C * f.vec;
  const size_t row = static_cast<size_t>(f.Hkv) * f.vec;
  const int total = f.kept * f.vec;
  const uint4* __restrict__ k = f.k + src0;
  const uint4* __restrict__ v = f.v + src0;
  uint4* __restrict__ kc = f.kc + dst0;
  uint4* __restrict__ vc = f.vc + dst0;
  constexpr int kBatch = 2;  // units in flight
  for (int i0 = first; i0 < total; i0 += kBatch * step) {
    uint4 x[kBatch], y[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * step;
      if (i < total) {
        const int s = i / f.vec, e = i - s * f.vec;
        const size_t src = sp[s] * row + e;
        x[u] = k[src];
        y[u] = v[src];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * step;
      if (i < total) {
        kc[i] = x[u];
        vc[i] = y[u];
      }
    }
  }
}

template <bool SMEM>
__global__ void __launch_bounds__(kFillThreads)
    swa_hh_select_kernel(const float* __restrict__ score_in, int L, int32_t* slot_pos, float* score, int C, int S,
                         int recent, const __grid_constant__ FillRows rows) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ unsigned s_hist[2048];
  __shared__ unsigned s_warp[kFillWarps];
  __shared__ unsigned s_cut, s_left;
  __shared__ int s_kept[kFillWarps], s_ties[kFillWarps];
  let_next_kernel_start();  // the copy of the rows, if there is one: its blocks come when all blocks here have begun
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* in = score_in + static_cast<size_t>(blockIdx.x) * L;
  int32_t* sp = slot_pos + static_cast<size_t>(blockIdx.x) * C;
  float* sc = score + static_cast<size_t>(blockIdx.x) * C;
  if (L <= C) {
    for (int i = tid; i < C; i += kFillThreads) {
      sp[i] = i < L ? i : -1;
      sc[i] = i < L ? in[i] : 0.f;
    }
    if (rows.here) {
      __syncthreads();
      copy_rows(rows, blockIdx.x, L, C, sp, tid, kFillThreads);
    }
    return;
  }
  constexpr uint32_t kAlways = 0xffffffffu;
  const int lo = S, hi = L - recent;  // positions outside stay in any case
  const int quads = (L + 3) / 4;
  auto key_of = [&](int i) -> uint32_t { return i < lo || i >= hi ? kAlways : order_bits(in[i]); };
  if constexpr (SMEM) {
#pragma unroll 8
    for (int i = tid; i < L; i += kFillThreads) s_keys[i] = order_bits(in[i]);
    if (tid < 4 * quads - L) s_keys[L + tid] = 0u;
    __syncthreads();
    for (int i = tid; i < lo + recent; i += kFillThreads) s_keys[i < lo ? i : hi + i - lo] = kAlways;
    __syncthreads();
  }
  // Four neighbouring keys.  Those behind the last position are 0, the lowest: they come after all others, so
  // that no tie is given to them.
  auto keys_at = [&](int q, uint32_t (&k)[4]) {
    if constexpr (SMEM) {
      const uint4 v = reinterpret_cast<const uint4*>(s_keys)[q];
      k[0] = v.x; k[1] = v.y; k[2] = v.z; k[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = 4 * q + e < L ? key_of(4 * q + e) : 0u;
    }
  };
  const unsigned room = C - S - recent;  // fewer than the others, as L > C
  unsigned cut = 0, need = room;         // prefix of the cut so far, keys wanted at or below it
  constexpr int kShift[3] = {21, 10, 0};
  constexpr int kBits[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    if (room == 0) break;
    const int shift = kShift[pass];
    const unsigned bins = 1u << kBits[pass];
    for (unsigned i = tid; i < bins; i += kFillThreads) s_hist[i] = 0;
    __syncthreads();
#pragma unroll 2
    for (int q = tid; q < quads; q += kFillThreads) {
      uint32_t k[4];
      keys_at(q, k);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k[e] != kAlways && (pass == 0 || (k[e] >> (shift + kBits[pass])) == cut))
          atomicAdd(&s_hist[(k[e] >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // from the top bin down, one or two neighbouring bins a thread
    constexpr unsigned kPer[3] = {2, 2, 1};
    unsigned n[2] = {0, 0};
#pragma unroll
    for (unsigned i = 0; i < kPer[pass]; ++i) n[i] = s_hist[bins - 1 - (tid * kPer[pass] + i)];
    unsigned above = block_prefix(n[0] + n[1], s_warp, lane, warp);
#pragma unroll
    for (unsigned i = 0; i < kPer[pass]; ++i) {
      if (above < need && above + n[i] >= need) {  // one bin of one thread
        s_cut = (cut << kBits[pass]) | (bins - 1 - (tid * kPer[pass] + i));
        s_left = need - above;
      }
      above += n[i];
    }
    __syncthreads();
    cut = s_cut;
    need = s_left;
    __syncthreads();
  }
  // no room for others: the cut is the key of those that stay in any case
  if (room == 0) cut = kAlways;
  const int ties = room == 0 ? S + recent : static_cast<int>(need);
  // ---- compaction: stretch of this warp, in quads
  const int per = ((quads + kFillWarps - 1) / kFillWarps + 31) / 32 * 32;
  const int first = min(quads, warp * per), last = min(quads, first + per);
  // this lane's quad: how many lie above the cut (low half) and on it (high half)
  auto count = [&](const uint32_t (&k)[4]) {
    unsigned n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) n += k[e] > cut ? 1u : k[e] == cut ? 0x10000u : 0u;
    return n;
  };
  int n_kept = 0, n_ties = 0;
#pragma unroll 2
  for (int q = first + lane; q < last; q += 32) {
    uint32_t k[4];
    keys_at(q, k);
    const unsigned n = count(k);
    n_kept += n & 0xffffu;
    n_ties += n >> 16;
  }
  n_kept = __reduce_add_sync(kFull, n_kept);
  n_ties = __reduce_add_sync(kFull, n_ties);
  if (lane == 0) {
    s_kept[warp] = n_kept;
    s_ties[warp] = n_ties;
  }
  __syncthreads();
  // kept without ties, and ties, in the stretches before
  int out = __reduce_add_sync(kFull, lane < warp ? s_kept[lane] : 0);
  int tie = __reduce_add_sync(kFull, lane < warp ? s_ties[lane] : 0);
  for (int q0 = first; q0 < last; q0 += 32) {
    const int q = q0 + lane;
    uint32_t k[4] = {0u, 0u, 0u, 0u};
    unsigned n = 0;
    if (q < last) {
      keys_at(q, k);
      n = count(k);
    }
    unsigned incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    int my_tie = tie + static_cast<int>((incl - n) >> 16);
    int slot = out + static_cast<int>((incl - n) & 0xffffu) + min(my_tie, ties);
    if (n != 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool equal = k[e] == cut;
        if (k[e] > cut || (equal && my_tie < ties)) {
          sp[slot++] = 4 * q + e;
        }
        my_tie += equal;
      }
    }
    const unsigned total = __shfl_sync(kFull, incl, 31);
    out += total & 0xffffu;
    tie += total >> 16;
  }
  __syncthreads();
  for (int i = tid; i < C; i += kFillThreads) sc[i] = in[sp[i]];  // all C slots are taken
  if (rows.here) copy_rows(rows, blockIdx.x, L, C, sp, tid, kFillThreads);
}

// Copy the chosen rows, one thread per 16 bytes, `per` blocks a (b, KV head).
__global__ void __launch_bounds__(256)
    swa_hh_gather_kernel(const __grid_constant__ FillRows rows, int L, const int32_t* slot_pos, int C,
                         int per) {
  wait_for_previous_kernel();
  const size_t seg = blockIdx.x / per;
  copy_rows(rows, seg, L, C, slot_pos + seg * C, blockIdx.x % per * 256 + threadIdx.x, per * 256);
}

}  // namespace

cudaError_t launch_hh_append(const void* k, const void* v, const int32_t* pos, void* kc, void* vc,
                             int32_t* slot_pos, float* score, int32_t* slot, int B, int Hkv, int d, int C, int S,
                             int recent, cudaStream_t stream) {
  swa_hh_append_kernel<<<B * Hkv, kAppendThreads, 0, stream>>>(
      static_cast<const uint4*>(k), static_cast<const uint4*>(v), pos, static_cast<uint4*>(kc),
      static_cast<uint4*>(vc), slot_pos, score, slot, Hkv, d / 8, C, S, recent);
  return cudaGetLastError();
}

cudaError_t launch_hh_fill(const void* k, const void* v, const float* score_in, int L, void* kc, void* vc,
                           int32_t* slot_pos, float* score, int B, int Hkv, int d, int C, int S, int recent, int sms,
                           cudaStream_t stream) {
  const int segs = B * Hkv;
  const int kept = std::min(L, C), vec = d / 8;
  // Who copies the rows (K's and V's `bytes` a head): the selecting block itself, which spares the caller a launch,
  // or a kernel of its own, which has all SMs.  Heads x bytes, microseconds of (itself, own kernel):
  //   by call   8 x 128 KB 10.3, 11.1   8 x 192 KB 12.3, 11.1   8 x 512 KB 20.6, 11.1   32 x 128 KB 10.3, 11.1
  //   in a graph 8 x 64 KB 6.8, 6.6     8 x 128 KB 8.3, 6.9    8 x 192 KB 9.9, 7.4     8 x 512 KB 18.6, 9.3
  // so few rows go with the caller's launch, at 1.4 us of a graph's time at most.  With a block for most SMs
  // the block itself copies more (in a graph, and by call alike):
  //   128 x 256 KB 16.6, 17.7   256 x 150 KB 19.3, 21.2   256 x 256 KB 28.7, 29.9   512 x 256 KB 51.3, 56.2
  //   96 x 512 KB 26.2, 26.0    128 x 512 KB 31.2, 31.2   256 x 512 KB 57.3, 54.6   136 x 1 MB 59.5, 54.3
  const long long bytes = static_cast<long long>(kept) * vec * 32;
  const bool here = bytes <= (152 << 10) || (segs >= sms * 7 / 8 && bytes <= (384 << 10));
  const FillRows rows{static_cast<const uint4*>(k), static_cast<const uint4*>(v), static_cast<uint4*>(kc),
                      static_cast<uint4*>(vc), Hkv, vec, kept, here};
  cudaError_t e = cudaSuccess;
  if (L <= kFillKeys) {
    const size_t smem = L > C ? static_cast<size_t>((L + 3) / 4) * 16 : 0;
    e = allow_shared<swa_hh_select_kernel<true>>(kFillKeys * 4);
    if (e != cudaSuccess) return e;
    swa_hh_select_kernel<true><<<segs, kFillThreads, smem, stream>>>(score_in, L, slot_pos, score, C, S, recent, rows);
  } else {
    swa_hh_select_kernel<false><<<segs, kFillThreads, 0, stream>>>(score_in, L, slot_pos, score, C, S, recent, rows);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess || kept == 0 || here) return e;
  const int blocks = (kept * vec + 255) / 256;
  const int per = std::min(blocks, std::max(1, (sms * 32 + segs - 1) / segs));
  return launch_early(swa_hh_gather_kernel, dim3(static_cast<unsigned>(per) * segs), 256, stream, rows, L, slot_pos, C,
                      per);
}

}  // namespace swa

// Rotary positions with several axes, in place, forward or inverse.
//
// Pair i of a head (elements i and i + d/2) turns by positions[axis_i][t] * theta_i.
// The kernel reads and writes every element once and is bound by that; the angles are
// shared by the heads of a token, so a block takes a few tokens, forms their d/2
// cosines and sines once in shared memory (product and reduction in fp64, as far
// positions need), and then streams the tokens' heads with 16-byte loads.
// 16320 tokens of 32 + 8 heads, d = 128, float32 (669 MB): 112 us, 6.0 TB/s, 91% of a copy's
// rate; 64 tokens in bf16: 2.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fixed_cache.h"

namespace swa {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // tokens a block

// cos and sin of p * theta, to float32 accuracy at any int32 position: the product in
// fp64, reduced to [-pi, pi] with 2 pi in two parts.
__device__ __forceinline__ float2 cos_sin(int p, double theta) {
  const double a = static_cast<double>(p) * theta;
  const double k = rint(a * 0.15915494309189533577);
  double r = fma(-k, 6.283185307179586232, a);
  r = fma(-k, 2.4492935982947064e-16, r);
  float s, c;
  sincosf(static_cast<float>(r), &s, &c);
  return make_float2(c, s);
}

// Rotate the pairs (lo[e], hi[e]) of one 16-byte chunk each.
template <bool F32>
__device__ __forceinline__ void rotate(uint4& lo, uint4& hi, const float2* cs) {
  uint32_t* l = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* h = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (F32) {
      const float x = __uint_as_float(l[w]), y = __uint_as_float(h[w]);
      const float2 t = cs[w];
      l[w] = __float_as_uint(fmaf(x, t.x, -y * t.y));
      h[w] = __float_as_uint(fmaf(x, t.y, y * t.x));
    } else {
      const float x0 = __uint_as_float(l[w] << 16), x1 = __uint_as_float(l[w] & 0xffff0000u);
      const float y0 = __uint_as_float(h[w] << 16), y1 = __uint_as_float(h[w] & 0xffff0000u);
      const float2 t0 = cs[2 * w], t1 = cs[2 * w + 1];
      __nv_bfloat162 a = __floats2bfloat162_rn(fmaf(x0, t0.x, -y0 * t0.y), fmaf(x1, t1.x, -y1 * t1.y));
      __nv_bfloat162 b = __floats2bfloat162_rn(fmaf(x0, t0.y, y0 * t0.x), fmaf(x1, t1.y, y1 * t1.x));
      l[w] = *reinterpret_cast<uint32_t*>(&a);
      h[w] = *reinterpret_cast<uint32_t*>(&b);
    }
  }
}

// blockIdx.y takes its share of a token tile's heads (few tokens: more blocks).
template <bool F32, int D>
__global__ void __launch_bounds__(kThreads)
    swa_rope_axes_kernel(const __grid_constant__ RopeAxesArgs a, const __grid_constant__ RopeAxesTable tab) {
  constexpr int EL = F32 ? 4 : 8;         // elements of 16 bytes
  constexpr int HC = D / 2 / EL;          // chunk pairs of a head
  __shared__ float2 cs[kTokens][D / 2];
  const int H = a.Hq + a.Hkv;
  const long long tiles = (a.T + kTokens - 1) / kTokens;
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const long long t0 = tile * kTokens;
    const int n = static_cast<int>(min(static_cast<long long>(kTokens), a.T - t0));
    __syncthreads();
    for (int i = threadIdx.x; i < n * (D / 2); i += kThreads) {
      const int t = i / (D / 2), e = i % (D / 2);
      float2 v = cos_sin(a.positions[tab.axis[e] * a.T + t0 + t], tab.theta[e]);
      v.y *= a.sign;
      cs[t][e] = v;
    }
    __syncthreads();
    const int units = n * H * HC;
    for (int u = blockIdx.y * kThreads + threadIdx.x; u < units; u += gridDim.y * kThreads) {
      const int c = u % HC, th = u / HC;
      const int t = th / H, h = th - t * H;
      char* row = h < a.Hq ? static_cast<char*>(a.q) + ((t0 + t) * a.q_stride + h * D) * (16 / EL)
                           : static_cast<char*>(a.k) + ((t0 + t) * a.k_stride + (h - a.Hq) * D) * (16 / EL);
      uint4* lo = reinterpret_cast<uint4*>(row) + c;
      uint4* hi = lo + HC;
      uint4 x = *lo, y = *hi;
      rotate<F32>(x, y, &cs[t][c * EL]);
      *lo = x;
      *hi = y;
    }
  }
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesArgs& a, const RopeAxesTable& t, bool f32, int sms, cudaStream_t stream) {
  const long long tiles = (a.T + kTokens - 1) / kTokens;
  const long long full = sms * 8LL;
  const long long per_tile = static_cast<long long>(std::min<long long>(a.T, kTokens)) * (a.Hq + a.Hkv) * a.d / 2 / (f32 ? 4 : 8);
  // few tokens: their heads go to several blocks, each with at least one round of work
  const long long split = std::max(1LL, std::min({full / tiles, (per_tile + kThreads - 1) / kThreads, 64LL}));
  const dim3 grid(static_cast<unsigned>(std::min(tiles, full)), static_cast<unsigned>(split));
  if (a.d == 128 && f32)
    swa_rope_axes_kernel<true, 128><<<grid, kThreads, 0, stream>>>(a, t);
  else if (a.d == 128)
    swa_rope_axes_kernel<false, 128><<<grid, kThreads, 0, stream>>>(a, t);
  else if (f32)
    swa_rope_axes_kernel<true, 64><<<grid, kThreads, 0, stream>>>(a, t);
  else
    swa_rope_axes_kernel<false, 64><<<grid, kThreads, 0, stream>>>(a, t);
  return cudaGetLastError();
}

}  // namespace swa

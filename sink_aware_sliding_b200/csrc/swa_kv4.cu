// 4-bit ring cache: quantising fill and append, reading back.
//
// A row of d elements (one token, one KV head) is held by groups of 32:
//   lo   = min of the group                       (exact: the input is bf16)
//   step = bf16((max - lo) * (1/15)),             0 where that is below 2^-126
//   code = rint((x - lo) * (1/step)) in 0..15,    value = code * step + lo.
// Each of these steps rounds once to 32 bits (step to bf16), so that the codes are
// the same wherever they are computed.
// Row layout: d/2 bytes of codes, then d/32 pairs (step, lo) in bf16.  The codes of
// element 32 j + 4 g + i (g < 8, i < 4) are nibble (g * d/32 + j) * 4 + i, low nibble
// first: seen as [d/32, 8, 4] the elements are stored in the order [8, d/32, 4], so
// that 1/8 of the code bytes holds four neighbouring elements of every group, which
// is what one thread of the decode kernel multiplies.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fixed_cache.h"
#include "ptx.cuh"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Quantise eight neighbouring elements x of group j, held by the four lanes t of the
// group (elements 8 t .. 8 t + 7): the 16-bit pieces (four nibbles each) of their two
// quarters, and the group's (step, lo) word.  All 32 lanes take part.
__device__ __forceinline__ void quantise8(const uint4& x, uint32_t& piece0, uint32_t& piece1, uint32_t& param) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // (min, max) of the pairs, then of the lanes; -0 and +0 are the same value
  __nv_bfloat162 mn = __hmin2(__hmin2(as_bf2(w[0]), as_bf2(w[1])), __hmin2(as_bf2(w[2]), as_bf2(w[3])));
  __nv_bfloat162 mx = __hmax2(__hmax2(as_bf2(w[0]), as_bf2(w[1])), __hmax2(as_bf2(w[2]), as_bf2(w[3])));
  // one word (min, -max): both reduce as minima
  __nv_bfloat162 r = __halves2bfloat162(__hmin(__low2bfloat16(mn), __high2bfloat16(mn)),
                                        __hneg(__hmax(__low2bfloat16(mx), __high2bfloat16(mx))));
  r = __hmin2(r, as_bf2(__shfl_xor_sync(kFull, as_u32(r), 1)));
  r = __hmin2(r, as_bf2(__shfl_xor_sync(kFull, as_u32(r), 2)));
  const float lo = __low2float(r), hi = -__high2float(r);
  __nv_bfloat16 step16 = __float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
  float step = __bfloat162float(step16);
  if (!(step >= 1.17549435e-38f)) {  // below 2^-126 (its reciprocal may overflow), or NaN
    step = 0.f;
    step16 = __float2bfloat16_rn(0.f);
  }
  const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
  // (x - lo) * inv + 1.5 * 2^23, each operation rounded: the sum's low bits are the product
  // rounded to nearest even, at most 15 since step is within 2^-9 of (hi - lo) / 15.  Four sums
  // times 1, 16, 256, 4096 add up to four nibbles: the bits above the codes start at bit 22.
  const uint64_t nlo = f2_pack(-lo, -lo);
  uint32_t c[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t x2 = f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    float q0, q1;
    f2_unpack(f2_add(x2, nlo), q0, q1);
    c[2 * e] = __float_as_uint(__fadd_rn(__fmul_rn(q0, inv), 12582912.f));  // packed, the two would become one fma
    c[2 * e + 1] = __float_as_uint(__fadd_rn(__fmul_rn(q1, inv), 12582912.f));
  }
  piece0 = c[0] + c[1] * 16u + c[2] * 256u + c[3] * 4096u;  // only the low 16 bits count
  piece1 = c[4] + c[5] * 16u + c[6] * 256u + c[7] * 4096u;
  param = static_cast<uint32_t>(__bfloat16_as_ushort(step16)) | (__float_as_uint(lo) & 0xffff0000u);
}

// d/8 lanes hold one row; this lane's lane index within the row is rl = 4 j + t.
// Writes the row at dst (and at dst2 when it is not null).
template <int D>
__device__ __forceinline__ void store_row(uint32_t piece0, uint32_t piece1, uint32_t param, int rl, uint8_t* dst,
                                          uint8_t* dst2) {
  constexpr int NG = D / kKv4Group;
  const int j = rl >> 2, t = rl & 3;
  // Neighbouring groups j, j ^ 1 share a word of codes: the even one takes quarter 2 t,
  // the odd one quarter 2 t + 1.
  const bool odd = j & 1;
  const uint32_t other = __shfl_xor_sync(kFull, odd ? piece0 : piece1, 4);
  const uint32_t word = odd ? __byte_perm(other, piece1, 0x5410) : __byte_perm(piece0, other, 0x5410);
  const int at = (2 * t + (odd ? 1 : 0)) * (2 * NG) + (j >> 1) * 4;
  if (dst != nullptr) {
    *reinterpret_cast<uint32_t*>(dst + at) = word;
    if (t == 0) *reinterpret_cast<uint32_t*>(dst + D / 2 + 4 * j) = param;
  }
  if (dst2 != nullptr) {
    *reinterpret_cast<uint32_t*>(dst2 + at) = word;
    if (t == 0) *reinterpret_cast<uint32_t*>(dst2 + D / 2 + 4 * j) = param;
  }
}

// d/8 lanes a row; rows of a sequence in the order (kept position, head), so that the
// reads are consecutive; two rows a thread in flight.  blockIdx.y: 0 for k, 1 for v;
// blockIdx.z: the sequence.
constexpr int kFillRows = 2;
template <int D>
__global__ void __launch_bounds__(256)
    swa_kv4_fill_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, int P, uint8_t* kc, uint8_t* vc,
                        uint8_t* sk, uint8_t* sv, int B, FastDiv hkv, int W, int S) {
  constexpr int LPR = D / 8;  // lanes a row
  constexpr int PER = 256 / LPR;
  constexpr int ROW = kv4_row_bytes(D);
  const int Hkv = static_cast<int>(hkv.d);
  const int n_ring = min(P, W), first = P - n_ring;
  const int n_old = min(min(P, S), first);  // sinks that have left the window
  const int rows = (n_ring + n_old) * Hkv;
  const int slot0 = first % W;              // ring slot of position `first`
  const int rl = threadIdx.x % LPR;
  for (int b = blockIdx.z; b < B; b += gridDim.z) {
    const uint4* src = (blockIdx.y ? v : k) + static_cast<size_t>(b) * P * Hkv * LPR + rl;
    uint8_t* ring = (blockIdx.y ? vc : kc) + static_cast<size_t>(b) * Hkv * W * ROW;
    uint8_t* sink = (blockIdx.y ? sv : sk) + static_cast<size_t>(b) * Hkv * S * ROW;
    // every lane of a warp takes part in each step's shuffles
    for (int r0 = blockIdx.x * (PER * kFillRows); r0 < rows; r0 += gridDim.x * (PER * kFillRows)) {
      uint4 x[kFillRows];
      uint8_t *dst[kFillRows], *dst2[kFillRows];
#pragma unroll
      for (int u = 0; u < kFillRows; ++u) {
        const int r = r0 + u * PER + threadIdx.x / LPR;
        x[u] = make_uint4(0, 0, 0, 0);
        dst[u] = dst2[u] = nullptr;
        if (r < rows) {
          const int i = static_cast<int>(hkv.div(r)), h = r - i * Hkv;
          const int at = i - n_old;  // from the first kept ring position; negative: an old sink
          const int p = at < 0 ? i : first + at;
          x[u] = src[(static_cast<size_t>(p) * Hkv + h) * LPR];
          if (at >= 0) {
            const int slot = slot0 + at < W ? slot0 + at : slot0 + at - W;
            dst[u] = ring + (static_cast<size_t>(h) * W + slot) * ROW;
          }
          if (p < S) dst2[u] = sink + (static_cast<size_t>(h) * S + p) * ROW;
        }
      }
#pragma unroll
      for (int u = 0; u < kFillRows; ++u) {
        uint32_t p0, p1, param;
        quantise8(x[u], p0, p1, param);
        store_row<D>(p0, p1, param, rl, dst[u], dst2[u]);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(128)
    swa_kv4_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v, const int32_t* __restrict__ pos,
                          uint8_t* kc, uint8_t* vc, uint8_t* sk, uint8_t* sv, int B, int Hkv, int W, int S) {
  constexpr int LPR = D / 8;
  constexpr int ROW = kv4_row_bytes(D);
  const long long r = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) / LPR;
  const int rl = threadIdx.x % LPR;
  uint4 x = make_uint4(0, 0, 0, 0);
  uint8_t *dst = nullptr, *dst2 = nullptr;
  if (r < static_cast<long long>(B) * Hkv) {
    const int p = pos[r / Hkv];
    if (p >= 0) {
      x = (blockIdx.y ? v : k)[r * LPR + rl];
      dst = (blockIdx.y ? vc : kc) + (static_cast<size_t>(r) * W + p % W) * ROW;
      if (p < S) dst2 = (blockIdx.y ? sv : sk) + (static_cast<size_t>(r) * S + p) * ROW;
    }
  }
  uint32_t p0, p1, param;
  quantise8(x, p0, p1, param);
  store_row<D>(p0, p1, param, rl, dst, dst2);
}

// One lane per eight elements (group j, elements 8 t .. 8 t + 7: quarters 2 t, 2 t + 1).
// blockIdx.y: 0 for k, 1 for v; blockIdx.z: the sequence.
template <int D, bool F32>
__global__ void __launch_bounds__(256)
    swa_kv4_read_kernel(const int32_t* __restrict__ positions, int n, const uint8_t* __restrict__ kc,
                        const uint8_t* __restrict__ vc, const uint8_t* __restrict__ sk,
                        const uint8_t* __restrict__ sv, void* k_out, void* v_out, int B, FastDiv hkv, FastDiv w, int S) {
  constexpr int LPR = D / 8, NG = D / kKv4Group;
  constexpr int ROW = kv4_row_bytes(D);
  const int Hkv = static_cast<int>(hkv.d), W = static_cast<int>(w.d);
  void* out = blockIdx.y ? v_out : k_out;
  const int rows = n * Hkv;
  const int rl = threadIdx.x % LPR, j = rl >> 2, t = rl & 3;
  for (int b = blockIdx.z; b < B; b += gridDim.z)
#pragma unroll 2
    for (int in_b = (blockIdx.x * 256 + threadIdx.x) / LPR; in_b < rows; in_b += gridDim.x * (256 / LPR)) {
    const int i = static_cast<int>(hkv.div(in_b)), h = in_b - i * Hkv;
    const int p = positions[static_cast<size_t>(b) * n + i];
    const uint8_t* ring = blockIdx.y ? vc : kc;
    const uint8_t* sink = blockIdx.y ? sv : sk;
    const size_t r = static_cast<size_t>(b) * rows + in_b;
    float y[8];
    if (p < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0.f;
    } else {
      const size_t seg = static_cast<size_t>(b) * Hkv + h;
      const uint8_t* row = p < S ? sink + (seg * S + p) * ROW : ring + (seg * W + w.mod(p)) * ROW;
      const uint32_t c0 = *reinterpret_cast<const uint16_t*>(row + (2 * t) * 2 * NG + 2 * j);
      const uint32_t c1 = *reinterpret_cast<const uint16_t*>(row + (2 * t + 1) * 2 * NG + 2 * j);
      const uint32_t param = *reinterpret_cast<const uint32_t*>(row + D / 2 + 4 * j);
      const float step = __uint_as_float(param << 16), lo = __uint_as_float(param & 0xffff0000u);
      const uint32_t c = c0 | (c1 << 16);
      // nibbles to bytes, each byte to the low mantissa bits of 2^23, and off again
      const uint32_t even = c & 0x0f0f0f0fu, odd = (c >> 4) & 0x0f0f0f0fu;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float n0 = __uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 + e)) - 8388608.f;
        const float n1 = __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 + e)) - 8388608.f;
        y[2 * e] = fmaf(n0, step, lo);
        y[2 * e + 1] = fmaf(n1, step, lo);
      }
    }
    if constexpr (F32) {
      float4* o = static_cast<float4*>(out) + (r * LPR + rl) * 2;
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      uint4 o;
      uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
      for (int e = 0; e < 4; ++e) ow[e] = as_u32(__floats2bfloat162_rn(y[2 * e], y[2 * e + 1]));
      static_cast<uint4*>(out)[r * LPR + rl] = o;
    }
  }
}

}  // namespace

namespace {
// Blocks along x for `units` blocks' worth of work of each of B sequences, k and v: as many
// as an SM holds at once (`per_sm`), since a block's start costs as much as two of its rows.
dim3 kv4_grid(long long units, int B, int sms, int per_sm) {
  const int z = std::min(B, 32768);
  const long long x = std::min(units, std::max(1LL, static_cast<long long>(sms) * per_sm / (2LL * z)));
  return dim3(static_cast<unsigned>(x), 2, static_cast<unsigned>(z));
}
}  // namespace

cudaError_t launch_kv4_fill(const void* k, const void* v, int P, void* kc, void* vc, void* sk, void* sv, int B,
                            int Hkv, int d, int W, int S, int sms, cudaStream_t stream) {
  const int n_ring = std::min(P, W);
  const long long rows = static_cast<long long>(Hkv) * (n_ring + std::min(std::min(P, S), P - n_ring));
  const int per = 256 / (d / 8) * kFillRows;
  const dim3 grid = kv4_grid((rows + per - 1) / per, B, sms, 16);
  const FastDiv hkv(Hkv);
  const auto* ks = static_cast<const uint4*>(k);
  const auto* vs = static_cast<const uint4*>(v);
  auto* c0 = static_cast<uint8_t*>(kc);
  auto* c1 = static_cast<uint8_t*>(vc);
  auto* s0 = static_cast<uint8_t*>(sk);
  auto* s1 = static_cast<uint8_t*>(sv);
  if (d == 128)
    swa_kv4_fill_kernel<128><<<grid, 256, 0, stream>>>(ks, vs, P, c0, c1, s0, s1, B, hkv, W, S);
  else
    swa_kv4_fill_kernel<64><<<grid, 256, 0, stream>>>(ks, vs, P, c0, c1, s0, s1, B, hkv, W, S);
  return cudaGetLastError();
}

cudaError_t launch_kv4_append(const void* k, const void* v, const int32_t* pos, void* kc, void* vc, void* sk,
                              void* sv, int B, int Hkv, int d, int W, int S, cudaStream_t stream) {
  const long long rows = static_cast<long long>(B) * Hkv;
  if (rows == 0) return cudaSuccess;
  const int per = 128 / (d / 8);
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per), 2);
  const auto* ks = static_cast<const uint4*>(k);
  const auto* vs = static_cast<const uint4*>(v);
  auto* c0 = static_cast<uint8_t*>(kc);
  auto* c1 = static_cast<uint8_t*>(vc);
  auto* s0 = static_cast<uint8_t*>(sk);
  auto* s1 = static_cast<uint8_t*>(sv);
  if (d == 128)
    swa_kv4_append_kernel<128><<<grid, 128, 0, stream>>>(ks, vs, pos, c0, c1, s0, s1, B, Hkv, W, S);
  else
    swa_kv4_append_kernel<64><<<grid, 128, 0, stream>>>(ks, vs, pos, c0, c1, s0, s1, B, Hkv, W, S);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const int32_t* positions, int n, const void* kc, const void* vc, const void* sk,
                            const void* sv, void* k_out, void* v_out, bool f32, int B, int Hkv, int d, int W, int S,
                            int sms, cudaStream_t stream) {
  const int per = 256 / (d / 8);
  const dim3 grid = kv4_grid((static_cast<long long>(n) * Hkv + per - 1) / per, B, sms, 16);
  const FastDiv hkv(Hkv), w(W);
  const auto* c0 = static_cast<const uint8_t*>(kc);
  const auto* c1 = static_cast<const uint8_t*>(vc);
  const auto* s0 = static_cast<const uint8_t*>(sk);
  const auto* s1 = static_cast<const uint8_t*>(sv);
  if (d == 128 && f32)
    swa_kv4_read_kernel<128, true><<<grid, 256, 0, stream>>>(positions, n, c0, c1, s0, s1, k_out, v_out, B, hkv, w, S);
  else if (d == 128)
    swa_kv4_read_kernel<128, false><<<grid, 256, 0, stream>>>(positions, n, c0, c1, s0, s1, k_out, v_out, B, hkv, w, S);
  else if (f32)
    swa_kv4_read_kernel<64, true><<<grid, 256, 0, stream>>>(positions, n, c0, c1, s0, s1, k_out, v_out, B, hkv, w, S);
  else
    swa_kv4_read_kernel<64, false><<<grid, 256, 0, stream>>>(positions, n, c0, c1, s0, s1, k_out, v_out, B, hkv, w, S);
  return cudaGetLastError();
}

}  // namespace swa

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
//
// The fill is bound by instruction issue (76% of the slots, ALU pipe 59%): 63 instructions a row.
// The read-back waits for loads that depend on each other, position before row (issue 55%, ALU pipe
// 45%, most of the waiting warps on long loads): 38 instructions a row.  Four prompts' last 4096
// positions and 4 sinks, 8 heads, d = 128 (88 MB each way): fill 21 us, 4.2 TB/s, read 20.5 us; with
// 16 lanes a row 27 and 23.5 us, with 64-bit divisions for the row's place 41 and 31 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "fixed_cache.h"
#include "ptx.cuh"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kLanes = 8;  // lanes that share a row: lane g has the elements 32 j + 4 g .. + 3 of every group j

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) { return as_u32(__hmin2(as_bf2(a), as_bf2(b))); }
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return as_u32(__hmax2(as_bf2(a), as_bf2(b))); }

// One row, eight lanes: x[j] are this lane's four elements of group j, and what comes out are its codes (four
// nibbles of each group: 16 bits each) and, in lane g, the (step, lo) word of group g * NG / 8.  All lanes of the warp
// take part.
//   Each group's minimum and negated maximum reduce as one word (both as minima).  The lanes halve the groups among
// them as they go (4 -> 2 -> 1, then the last exchange), so that each group's step is worked out by 8 / NG lanes only,
// which then hand it round.
template <int NG>
__device__ __forceinline__ void quantise_row(const uint2 (&x)[NG], int g, uint32_t (&codes)[NG / 2], uint32_t& param) {
  uint32_t r[NG];
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const uint32_t mn = min2(x[j].x, x[j].y), mx = max2(x[j].x, x[j].y) ^ 0x80008000u;
    r[j] = min2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));  // (min, -max)
  }
  if constexpr (NG == 4) {
    const bool up = g & 4;
    const uint32_t k0 = up ? r[2] : r[0], k1 = up ? r[3] : r[1];
    const uint32_t s0 = up ? r[0] : r[2], s1 = up ? r[1] : r[3];
    r[0] = min2(k0, __shfl_xor_sync(kFull, s0, 4));
    r[1] = min2(k1, __shfl_xor_sync(kFull, s1, 4));
  }
  {
    constexpr int kBit = NG == 4 ? 2 : 4;
    const bool up = g & kBit;
    const uint32_t k0 = up ? r[1] : r[0], s0 = up ? r[0] : r[1];
    r[0] = min2(k0, __shfl_xor_sync(kFull, s0, kBit));
    if constexpr (NG == 2) r[0] = min2(r[0], __shfl_xor_sync(kFull, r[0], 2));
    r[0] = min2(r[0], __shfl_xor_sync(kFull, r[0], 1));
  }
  const float lo = __uint_as_float(r[0] << 16), hi = -__uint_as_float(r[0] & 0xffff0000u);
  __nv_bfloat16 step16 = __float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
  float step = __bfloat162float(step16);
  if (!(step >= 1.17549435e-38f)) {  // below 2^-126 (its reciprocal may overflow), or NaN
    step = 0.f;
    step16 = __float2bfloat16_rn(0.f);
  }
  const float my_inv = step > 0.f ? __frcp_rn(step) : 0.f;
  param = static_cast<uint32_t>(__bfloat16_as_ushort(step16)) | (r[0] << 16);
  // (x - lo) * inv + 1.5 * 2^23, each operation rounded (a packed product and sum would become one fma): the sum's
  // low bits are the product rounded to nearest even, at most 15 since step is within 2^-9 of (hi - lo) / 15.  Four
  // sums times 1, 16, 256, 4096 add up to four nibbles: the bits above the codes start at bit 22.
  uint32_t piece[NG];
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const float inv = __shfl_sync(kFull, my_inv, j * (kLanes / NG), kLanes);
    const float low = __uint_as_float(__shfl_sync(kFull, param, j * (kLanes / NG), kLanes) & 0xffff0000u);
    const uint64_t nlo = f2_pack(-low, -low);
    float d[4];
    f2_unpack(f2_add(f2_pack(__uint_as_float(x[j].x << 16), __uint_as_float(x[j].x & 0xffff0000u)), nlo), d[0], d[1]);
    f2_unpack(f2_add(f2_pack(__uint_as_float(x[j].y << 16), __uint_as_float(x[j].y & 0xffff0000u)), nlo), d[2], d[3]);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = __float_as_uint(__fadd_rn(__fmul_rn(d[e], inv), 12582912.f));
    piece[j] = c[0] + c[1] * 16u + c[2] * 256u + c[3] * 4096u;  // only the low 16 bits count
  }
#pragma unroll
  for (int j = 0; j < NG; j += 2) codes[j / 2] = __byte_perm(piece[j], piece[j + 1], 0x5410);
}

template <int NG>
__device__ __forceinline__ void store_row(const uint32_t (&codes)[NG / 2], uint32_t param, int g, uint8_t* row) {
  if constexpr (NG == 4)
    *reinterpret_cast<uint2*>(row + 8 * g) = make_uint2(codes[0], codes[1]);
  else
    *reinterpret_cast<uint32_t*>(row + 4 * g) = codes[0];
  if (g % (kLanes / NG) == 0) *reinterpret_cast<uint32_t*>(row + 16 * NG + 4 * (g / (kLanes / NG))) = param;
}

template <int NG>
__device__ __forceinline__ void load_row(uint2 (&x)[NG], const void* src, size_t row, int g) {
  const uint2* p = static_cast<const uint2*>(src) + row * (8 * NG) + g;
#pragma unroll
  for (int j = 0; j < NG; ++j) x[j] = p[8 * j];
}

// Eight lanes a row; rows of a sequence in the order (kept position, head), so that the
// reads are consecutive.  blockIdx.y: 0 for k, 1 for v; blockIdx.z: the sequence.
constexpr int kPer = 256 / kLanes;  // rows a block works on at once
template <int D>
__global__ void __launch_bounds__(256)
    swa_kv4_fill_kernel(const void* __restrict__ k, const void* __restrict__ v, int P, uint8_t* kc, uint8_t* vc,
                        uint8_t* sk, uint8_t* sv, int B, FastDiv hkv, int W, int S) {
  constexpr int NG = D / kKv4Group;
  constexpr int ROW = kv4_row_bytes(D);
  let_next_kernel_start();
  const int Hkv = static_cast<int>(hkv.d);
  const int n_ring = min(P, W), first = P - n_ring;
  const int n_old = min(min(P, S), first);  // sinks that have left the window
  const int rows = (n_ring + n_old) * Hkv;
  const int slot0 = first % W;              // ring slot of position `first`
  const int g = threadIdx.x % kLanes;
  for (int b = blockIdx.z; b < B; b += gridDim.z) {
    uint8_t* ring = (blockIdx.y ? vc : kc) + static_cast<size_t>(b) * Hkv * W * ROW;
    uint8_t* sink = (blockIdx.y ? sv : sk) + static_cast<size_t>(b) * Hkv * S * ROW;
    const size_t row0 = static_cast<size_t>(b) * P * Hkv;
    // every lane of a warp takes part in each step's shuffles
#pragma unroll 2
    for (int r0 = blockIdx.x * kPer; r0 < rows; r0 += gridDim.x * kPer) {
      const int r = r0 + threadIdx.x / kLanes;
      uint2 x[NG] = {};
      int p = -1, h = 0, at = 0;
      if (r < rows) {
        const int i = static_cast<int>(hkv.div(r));
        h = r - i * Hkv;
        at = i - n_old;  // from the first kept ring position; negative: an old sink
        p = at < 0 ? i : first + at;
        load_row<NG>(x, blockIdx.y ? v : k, row0 + static_cast<size_t>(p) * Hkv + h, g);
      }
      uint32_t codes[NG / 2], param;
      quantise_row<NG>(x, g, codes, param);
      if (p >= 0) {
        if (at >= 0) {
          const int slot = slot0 + at < W ? slot0 + at : slot0 + at - W;
          store_row<NG>(codes, param, g, ring + (static_cast<size_t>(h) * W + slot) * ROW);
        }
        if (p < S) store_row<NG>(codes, param, g, sink + (static_cast<size_t>(h) * S + p) * ROW);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(128)
    swa_kv4_append_kernel(const void* __restrict__ k, const void* __restrict__ v, const int32_t* __restrict__ pos,
                          uint8_t* kc, uint8_t* vc, uint8_t* sk, uint8_t* sv, int B, int Hkv, int W, int S) {
  constexpr int NG = D / kKv4Group;
  constexpr int ROW = kv4_row_bytes(D);
  let_next_kernel_start();
  const long long r = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) / kLanes;
  const int g = threadIdx.x % kLanes;
  uint2 x[NG] = {};
  int p = -1;
  if (r < static_cast<long long>(B) * Hkv) {
    load_row<NG>(x, blockIdx.y ? v : k, r, g);
    p = pos[r / Hkv];
  }
  uint32_t codes[NG / 2], param;
  quantise_row<NG>(x, g, codes, param);
  if (p >= 0) {
    store_row<NG>(codes, param, g, (blockIdx.y ? vc : kc) + (static_cast<size_t>(r) * W + p % W) * ROW);
    if (p < S) store_row<NG>(codes, param, g, (blockIdx.y ? sv : sk) + (static_cast<size_t>(r) * S + p) * ROW);
  }
}

// Eight lanes a row, four elements of every group each.  blockIdx.y: 0 for k, 1 for v; blockIdx.z: the sequence.
template <int D, bool F32>
__global__ void __launch_bounds__(256)
    swa_kv4_read_kernel(const int32_t* positions, int n, const uint8_t* kc, const uint8_t* vc, const uint8_t* sk,
                        const uint8_t* sv, void* k_out, void* v_out, int B, FastDiv hkv, FastDiv w, int S) {
  constexpr int NG = D / kKv4Group;
  constexpr int ROW = kv4_row_bytes(D);
  wait_for_previous_kernel();
  const int Hkv = static_cast<int>(hkv.d), W = static_cast<int>(w.d);
  const uint8_t* ring = blockIdx.y ? vc : kc;
  const uint8_t* sink = blockIdx.y ? sv : sk;
  void* out = blockIdx.y ? v_out : k_out;
  const int rows = n * Hkv;
  const int g = threadIdx.x % kLanes;
  for (int b = blockIdx.z; b < B; b += gridDim.z) {
#pragma unroll 2
    for (int in_b = blockIdx.x * kPer + threadIdx.x / kLanes; in_b < rows; in_b += gridDim.x * kPer) {
      const int i = static_cast<int>(hkv.div(in_b)), h = in_b - i * Hkv;
      const int p = positions[static_cast<size_t>(b) * n + i];
      uint32_t code[NG / 2] = {}, param[NG] = {};  // p < 0: all zero, and so are the values
      if (p >= 0) {
        const size_t seg = static_cast<size_t>(b) * Hkv + h;
        const uint8_t* row = p < S ? sink + (seg * S + p) * ROW : ring + (seg * W + w.mod(p)) * ROW;
        if constexpr (NG == 4) {
          const uint2 c = *reinterpret_cast<const uint2*>(row + 8 * g);
          const uint4 q = *reinterpret_cast<const uint4*>(row + 64);
          code[0] = c.x; code[1] = c.y;
          param[0] = q.x; param[1] = q.y; param[2] = q.z; param[3] = q.w;
        } else {
          code[0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
          const uint2 q = *reinterpret_cast<const uint2*>(row + 32);
          param[0] = q.x; param[1] = q.y;
        }
      }
      const size_t at = (static_cast<size_t>(b) * rows + in_b) * (D / 4) + g;  // in groups of four elements
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        // nibbles to bytes, each byte to the low mantissa bits of 2^23, and off again
        const uint32_t even = code[j / 2] & 0x0f0f0f0fu, odd = (code[j / 2] >> 4) & 0x0f0f0f0fu;
        const float step = __uint_as_float(param[j] << 16), lo = __uint_as_float(param[j] & 0xffff0000u);
        float y[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t pick = 0x7440 + 2 * (j & 1) + e;
          y[2 * e] = fmaf(__uint_as_float(__byte_perm(even, 0x4b000000u, pick)) - 8388608.f, step, lo);
          y[2 * e + 1] = fmaf(__uint_as_float(__byte_perm(odd, 0x4b000000u, pick)) - 8388608.f, step, lo);
        }
        if constexpr (F32)
          static_cast<float4*>(out)[at + 8 * j] = make_float4(y[0], y[1], y[2], y[3]);
        else
          static_cast<uint2*>(out)[at + 8 * j] = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
      }
    }
  }
}

// Blocks along x for `units` blocks' worth of work of each of B sequences, k and v: 16 blocks of 256 threads for
// an SM, of which it holds 6 at a time at the 39 registers of d = 128, so that blocks that end early make room for
// others.  Four prompts' 4100 rows of 8 heads, fill and read-back in microseconds: 6 blocks 22.1 and 19.4, 8 (a
// second wave of a third) 23.2 and 23.9, 12 21.4 and 19.7, 16 21.1 and 20.3, 24 21.2 and 19.9.
dim3 kv4_grid(long long units, int B, int sms) {
  constexpr int kPerSm = 16;
  const int z = std::min(B, 32768);
  const long long x = std::min(units, std::max(1LL, static_cast<long long>(sms) * kPerSm / (2LL * z)));
  return dim3(static_cast<unsigned>(x), 2, static_cast<unsigned>(z));
}

}  // namespace

cudaError_t launch_kv4_fill(const void* k, const void* v, int P, void* kc, void* vc, void* sk, void* sv, int B,
                            int Hkv, int d, int W, int S, int sms, cudaStream_t stream) {
  const int n_ring = std::min(P, W);
  const long long rows = static_cast<long long>(Hkv) * (n_ring + std::min(std::min(P, S), P - n_ring));
  const dim3 grid = kv4_grid((rows + kPer - 1) / kPer, B, sms);
  const FastDiv hkv(Hkv);
  auto* c0 = static_cast<uint8_t*>(kc);
  auto* c1 = static_cast<uint8_t*>(vc);
  auto* s0 = static_cast<uint8_t*>(sk);
  auto* s1 = static_cast<uint8_t*>(sv);
  if (d == 128)
    swa_kv4_fill_kernel<128><<<grid, 256, 0, stream>>>(k, v, P, c0, c1, s0, s1, B, hkv, W, S);
  else
    swa_kv4_fill_kernel<64><<<grid, 256, 0, stream>>>(k, v, P, c0, c1, s0, s1, B, hkv, W, S);
  return cudaGetLastError();
}

cudaError_t launch_kv4_append(const void* k, const void* v, const int32_t* pos, void* kc, void* vc, void* sk,
                              void* sv, int B, int Hkv, int d, int W, int S, cudaStream_t stream) {
  const long long rows = static_cast<long long>(B) * Hkv;
  if (rows == 0) return cudaSuccess;
  constexpr int per = 128 / kLanes;
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per), 2);
  auto* c0 = static_cast<uint8_t*>(kc);
  auto* c1 = static_cast<uint8_t*>(vc);
  auto* s0 = static_cast<uint8_t*>(sk);
  auto* s1 = static_cast<uint8_t*>(sv);
  if (d == 128)
    swa_kv4_append_kernel<128><<<grid, 128, 0, stream>>>(k, v, pos, c0, c1, s0, s1, B, Hkv, W, S);
  else
    swa_kv4_append_kernel<64><<<grid, 128, 0, stream>>>(k, v, pos, c0, c1, s0, s1, B, Hkv, W, S);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const int32_t* positions, int n, const void* kc, const void* vc, const void* sk,
                            const void* sv, void* k_out, void* v_out, bool f32, int B, int Hkv, int d, int W, int S,
                            int sms, cudaStream_t stream) {
  const dim3 grid = kv4_grid((static_cast<long long>(n) * Hkv + kPer - 1) / kPer, B, sms);
  const FastDiv hkv(Hkv), w(W);
  const auto* c0 = static_cast<const uint8_t*>(kc);
  const auto* c1 = static_cast<const uint8_t*>(vc);
  const auto* s0 = static_cast<const uint8_t*>(sk);
  const auto* s1 = static_cast<const uint8_t*>(sv);
  const auto launch = [&](auto kernel) {
    return launch_early(kernel, grid, 256, stream, positions, n, c0, c1, s0, s1, k_out, v_out, B, hkv, w, S);
  };
  if (d == 128) return f32 ? launch(swa_kv4_read_kernel<128, true>) : launch(swa_kv4_read_kernel<128, false>);
  return f32 ? launch(swa_kv4_read_kernel<64, true>) : launch(swa_kv4_read_kernel<64, false>);
}

}  // namespace swa

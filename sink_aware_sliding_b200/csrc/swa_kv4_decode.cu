// Decode over the 4-bit ring cache (layout: swa_kv4.cu).
//
// With codes n in 0..15, steps a and minima b of the groups j of a row,
//   z_h = scale sum_j [ a_j (n_j . q_hj) + b_j sum(q_hj) ]
//   O_h = sum_keys p_h [ a_j n_j + b_j ].
// The integer part runs on the tensor cores with the codes as they are: a nibble in
// the low bits of a 16-bit word is the subnormal n 2^-24 as fp16 (for K) and n 2^-133 as
// bf16 (for V), one four bits higher is 16 times that, so that "unpacking" is one AND
// per two elements and loses nothing.  q is scaled by a power of two per head into fp16
// (exact for all but elements 2^-28 below the head's largest), and the odd nibbles' factor
// 16 goes into q and, for V, into the final scaling.  K's steps are applied in fp32, its
// minima times the sums of q are a product as well, with the sums in three bf16 parts.
//
// p and p a_j, which multiply V's minima and codes, are each the sum of two bf16 parts
// (1.5 * 2^-17 together), which have the exponents of a float: a key or a group whose
// p a_j is small next to another's keeps its bits down to 2^-73 of the largest step met.
// (In one fp16 part, 11 bits, a group 2^33 below the largest of its tile came out as zeros;
// 67.5 us against 69.3 us.)  Two running references: p and its sum are relative to
// the logits' maximum alone, and O is in units of a power of two that follows V's largest
// step.  (One reference for both loses keys: with V = 0 in one tile and 1e15 in the next it
// moves by 2^137, and the sum of p of the first tile with it.)
//
// Keys are the 16 rows of the products and up to eight query heads their columns: half the
// products of the other orientation, and the codes go into the operand's registers as they
// are masked; the scores are turned through shared memory (one 1 KB tile a warp) to become
// an operand of P V.  Bound by instruction issue, masks and permutes above all (60% of the issue
// slots and of the ALU pipe over a launch with its tail), next to HBM.
// B = 64, 8 KV heads, 4 query heads each, d = 128, window 4096 + 4 sinks (336 MB): 69.3 us,
// 4.8 TB/s (the copies alone take 53 us); 118 us with the heads as rows and 16 keys a step,
// 75 us with the keys as rows, 66 us with 32 keys a step and P in fp16.  With its append
// a step takes 74 us by call, 77 us once a longer load has lowered the clock to 1.85 GHz.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_decode.cuh"
#include "fixed_cache.h"

namespace swa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kStages = 2;       // one tile is worked on while the next one comes: 80 KB in flight on an SM
constexpr int kRows = 32;        // keys per tile: two products of 16 rows share a step of the softmax
constexpr int kBlocksPerSm = 4;  // 16 warps: what 128 registers a thread allow
// p <= 2^kSlack, and V's steps and minima are below 2^(size + 1): their products with p 2^(kTop - size)
// stay below 2^87, which leaves room for sums of 2^40 of them, and a code (2^-133) times a product
// is a normal float as long as p step is above 2^-73 of 2^size.
constexpr int kSlack = 6, kTop = 80, kSizeMin = -40;

template <int D>
struct K4 {
  static constexpr int NG = D / kKv4Group;
  static constexpr int ROW = kv4_row_bytes(D);
  static constexpr int CODES = D / 2;                    // code bytes of a row
  static constexpr int UNIT = D == 128 ? 16 : 8;         // bytes per copy: what a row is aligned to
  static constexpr int UNITS = ROW / UNIT;               // 5: as many copies per lane for 32 rows
  static constexpr int HALF = kRows * ROW;               // K's or V's bytes of a stage, rows as in the cache
  static constexpr int STAGE = 2 * HALF;
  static constexpr int SCORES = kRows * kDecHeads * 4;   // a warp's score tile, turned through shared memory
  static constexpr int WARP = kStages * STAGE + SCORES;
};

__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Two floats in two bf16 parts each: hi + lo is within 2^-17 of them.
__device__ __forceinline__ void split_bf16(uint64_t v, uint32_t& hi, uint32_t& lo) {
  float x, y;
  f2_unpack(v, x, y);
  hi = pack_bf16x2(x, y);
  f2_unpack(f2_fma(f2_pack(step_of(hi), low_of(hi)), f2_pack(-1.f, -1.f), v), x, y);
  lo = pack_bf16x2(x, y);
}

// Numerators (hi + lo) times steps in two bf16 parts again: the product of two 8-bit significands less its own
// rounding fits 8 bits, so that only the last sum rounds, 2^-17 of the whole; together within 1.5 * 2^-17.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// minus_high: -round(hi * step), or with lo = 0 nothing, which gives the high part.
__device__ __forceinline__ uint32_t low_times_step(uint32_t hi, uint32_t lo, uint32_t minus_high, uint32_t step) {
  return fma_bf16x2(lo, step, fma_bf16x2(hi, step, minus_high));
}

template <int NW>
__device__ __forceinline__ void lds_words(uint32_t (&w)[NW], const uint8_t* p) {
  if constexpr (NW == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (NW == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// 2^x, exactly; -126 <= x <= 127.
__device__ __forceinline__ float pow2(int x) { return __uint_as_float(static_cast<uint32_t>(x + 127) << 23); }

// The larger of `most` and of a group's step and |minimum|, in halves: a bf16's bits and 128, infinities and NaN
// below all others (they are their own group's affair).
__device__ __forceinline__ uint32_t larger(uint32_t w, uint32_t most) {
  return __viaddmax_s16x2(w & 0x7fff7fffu, 0x00800080u, most);
}

// FEW: up to four query heads a KV head.  P is the sum of two parts of bf16, and the low part of head h takes
// column h + 4 of the product with V, which would be empty: as many products as P of one part takes.  With more
// heads the low parts are products of their own (B = 64, 8 KV heads of 4: 69.3 us, and 75.3 us that way).
template <int D, bool FEW>
__global__ void __launch_bounds__(kDecWarps * 32, kBlocksPerSm)
    swa_kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs a, int c) {
  using C = K4<D>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_lse2[kDecHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % c;
  const size_t seg = blockIdx.x / c;
  const int b = static_cast<int>(seg / a.Hkv), kvh = static_cast<int>(seg % a.Hkv);
  const int G = a.G, W = a.W, S = a.S;
  const size_t head0 = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(kvh) * G;

  wait_for_previous_kernel();
  const int p = a.pos[b];
  const int n_ring = p < 0 ? 0 : (p < W ? p + 1 : W);
  const int n_sink = p < W ? 0 : min(p - W + 1, S);
  const int ring_tiles = (n_ring + kRows - 1) / kRows;
  const int tiles = ring_tiles + (n_sink + kRows - 1) / kRows;
  // A tile's copies: unit lane + 32 i, i < 5, of K's rows and of V's is this lane's.
  const size_t ring0 = seg * W * C::ROW, sink0 = seg * S * C::ROW;
  uint8_t* mine = smem + warp * C::WARP;
  const uint32_t ring_u32 = smem_u32(mine);
  const int full_tiles = n_ring / kRows;
  const int nw = c * kDecWarps;
  int tile = rank * kDecWarps + warp;
  // where this lane reads the next whole ring tile from
  const uint8_t* ks = a.kc + ring0 + static_cast<size_t>(tile) * C::HALF + lane * C::UNIT;
  const uint8_t* vs = a.vc + ring0 + static_cast<size_t>(tile) * C::HALF + lane * C::UNIT;
  const size_t ks_step = static_cast<size_t>(nw) * C::HALF;
  const uint64_t policy = stream_policy();
  auto issue = [&](int tile, int stage) {
    const uint32_t dst = ring_u32 + stage * C::STAGE + lane * C::UNIT;
    if (tile < full_tiles) {
#pragma unroll
      for (int i = 0; i < C::UNITS; ++i) {
        cp_async<C::UNIT>(dst + 32 * i * C::UNIT, ks + 32 * i * C::UNIT, true, policy);
        cp_async<C::UNIT>(dst + 32 * i * C::UNIT + C::HALF, vs + 32 * i * C::UNIT, true, policy);
      }
      ks += ks_step;
      vs += ks_step;
    } else if (tile < tiles) {  // the ring's last rows, or sinks; rows behind the last one become zeros
      const bool in_ring = tile < ring_tiles;
      const int first = (in_ring ? tile : tile - ring_tiles) * kRows;
      const int n = (in_ring ? n_ring : n_sink) - first;
      const size_t at = (in_ring ? ring0 : sink0) + static_cast<size_t>(first) * C::ROW + lane * C::UNIT;
      const uint8_t* k1 = (in_ring ? a.kc : a.sk) + at;
      const uint8_t* v1 = (in_ring ? a.vc : a.sv) + at;
#pragma unroll
      for (int i = 0; i < C::UNITS; ++i) {
        const bool real = lane + 32 * i < n * C::UNITS;
        cp_async<C::UNIT>(dst + 32 * i * C::UNIT, real ? k1 + 32 * i * C::UNIT : a.kc, real, policy);
        cp_async<C::UNIT>(dst + 32 * i * C::UNIT + C::HALF, real ? v1 + 32 * i * C::UNIT : a.vc, real, policy);
      }
    }
    cp_async_commit();
  };

#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(tile + s * nw, s);

  // ---- q of head g: fp16 fragments scaled by a power of two, and the sums of its groups
  uint32_t qb[NG][4];
  uint32_t qs0, qs1;  // sum of group t in three bf16 parts: what multiplies the minima
  float qscale0, qscale1;
  {
    const bool real = g < G;
    const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + (head0 + (real ? g : 0)) * D;
    float x[NG][8];
    float mx = 0.f, sum_t = 0.f;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const uint4 w = real ? *reinterpret_cast<const uint4*>(qrow + 32 * j + 8 * t) : make_uint4(0, 0, 0, 0);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[j][2 * e] = step_of(ww[e]);
        x[j][2 * e + 1] = low_of(ww[e]);
        sum += x[j][2 * e] + x[j][2 * e + 1];
        mx = fmaxf(mx, fmaxf(fabsf(x[j][2 * e]), fabsf(x[j][2 * e + 1])));
      }
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      if (j == t) sum_t = sum * a.scale_log2;
    }
    const float hi = __bfloat162float(__float2bfloat16_rn(sum_t));
    const float mid = __bfloat162float(__float2bfloat16_rn(sum_t - hi));
    qs0 = pack_bf16x2(hi, mid);
    qs1 = pack_bf16x2(sum_t - hi - mid, 0.f);
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    // largest element to [2^14, 2^15)
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    e = min(max(e, -100), 100) - 14;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e + 12) << 23) * (a.scale_log2 * 4096.f);  // 2^(e + 24)
    qscale0 = __shfl_sync(kFull, up, 8 * t);  // of heads 2t and 2t + 1
    qscale1 = __shfl_sync(kFull, up, 8 * t + 4);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      // k-slots of the two products: nibbles (0, 2), then (1, 3), which carry a factor 16
      qb[j][0] = pack_f16(x[j][0] * down, x[j][4] * down);
      qb[j][1] = pack_f16(x[j][2] * down, x[j][6] * down);
      qb[j][2] = pack_f16(x[j][1] * down * 0.0625f, x[j][5] * down * 0.0625f);
      qb[j][3] = pack_f16(x[j][3] * down * 0.0625f, x[j][7] * down * 0.0625f);
    }
  }

  float o[NG][2][4];
  float om[4] = {0.f, 0.f, 0.f, 0.f};  // minima's part: row g is group g; [0] head 2t, [1] head 2t + 1
#pragma unroll
  for (int j = 0; j < NG; ++j)
#pragma unroll
    for (int x = 0; x < 2; ++x) o[j][x][0] = o[j][x][1] = o[j][x][2] = o[j][x][3] = 0.f;
  float ref = -INFINITY, l = 0.f;  // of this lane's head: the logits' reference, and the sum of p = 2^(z - ref)
  const int head = FEW ? g & 3 : g;
  const uint32_t low_part = FEW && g >= 4 ? 0xffffffffu : 0u;
  int size = kSizeMin;             // O and om are sums of p 2^(kTop - size) V
  // Scores: rows g and g + 8 of the product are the tokens kr and kr + 8; P and V: this
  // lane's tokens are 2t, 2t + 1 and those + 8.  In rows of 80 bytes both orders keep the
  // reads off each other's banks (K: two rows per quarter warp, V: four per half warp).
  const int kr = (g >> 1) + 4 * (g & 1);
  const int kcode = kr * C::ROW + t * (C::CODES / 4), kpar = kr * C::ROW + C::CODES;
  const int vcode = 2 * t * C::ROW + g * 2 * NG, vpar = 2 * t * C::ROW + C::CODES;
  float* scores = reinterpret_cast<float*>(mine + kStages * C::STAGE);

  int stage = 0;
  for (; tile < tiles; tile += nw) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // this tile has arrived for every lane, and every lane is done with the one before
    issue(tile + (kStages - 1) * nw, stage == 0 ? kStages - 1 : stage - 1);
    const uint8_t* kt = mine + stage * C::STAGE;
    const uint8_t* vt = kt + C::HALF;

    // ---- scores of the tokens kr, kr + 8 of each 16 for the heads 2t, 2t + 1
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      uint32_t wa[NG], wb[NG], pa[NG], pb[NG];
      lds_words<NG>(wa, kt + 16 * hf * C::ROW + kcode);
      lds_words<NG>(wb, kt + 16 * hf * C::ROW + kcode + 8 * C::ROW);
      lds_words<NG>(pa, kt + 16 * hf * C::ROW + kpar);
      lds_words<NG>(pb, kt + 16 * hf * C::ROW + kpar + 8 * C::ROW);
      const uint32_t ma = *reinterpret_cast<const uint32_t*>(kt + 16 * hf * C::ROW + kpar + t % NG * 4);
      const uint32_t mb = *reinterpret_cast<const uint32_t*>(kt + 16 * hf * C::ROW + kpar + t % NG * 4 + 8 * C::ROW);
      float low[4];  // minimum of group t in every k-slot, times the sums of q
      const uint32_t a0 = __byte_perm(ma, ma, 0x3232), a1 = __byte_perm(mb, mb, 0x3232);
      mma_bf16_zero(low, a0, a1, a0, a1, qs0, qs1);
      float z0 = 0.f, z1 = 0.f, z2 = 0.f, z3 = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        // elements 8 t + i (low half) and 8 t + 4 + i of group j
        const uint32_t x = __byte_perm(wa[j >> 1], wa[(j >> 1) + NG / 2], (j & 1) ? 0x7632 : 0x5410);
        const uint32_t y = __byte_perm(wb[j >> 1], wb[(j >> 1) + NG / 2], (j & 1) ? 0x7632 : 0x5410);
        const uint32_t xh = x >> 8, yh = y >> 8;
        float acc[4];
        mma_f16_zero(acc, x & 0x000f000fu, y & 0x000f000fu, xh & 0x000f000fu, yh & 0x000f000fu, qb[j][0], qb[j][1]);
        mma_f16_16816(acc, x & 0x00f000f0u, y & 0x00f000f0u, xh & 0x00f000f0u, yh & 0x00f000f0u, qb[j][2], qb[j][3]);
        const float sa = step_of(pa[j]), sb = step_of(pb[j]);
        z0 = fmaf(sa, acc[0], z0);
        z1 = fmaf(sa, acc[1], z1);
        z2 = fmaf(sb, acc[2], z2);
        z3 = fmaf(sb, acc[3], z3);
      }
      *reinterpret_cast<float2*>(scores + (kr + 16 * hf) * kDecHeads + 2 * t) =
          make_float2(fmaf(z0, qscale0, low[0]), fmaf(z1, qscale1, low[1]));
      *reinterpret_cast<float2*>(scores + (kr + 8 + 16 * hf) * kDecHeads + 2 * t) =
          make_float2(fmaf(z2, qscale0, low[2]), fmaf(z3, qscale1, low[3]));
    }
    __syncwarp();
    // ---- turned: this lane's head, tokens 2t, 2t + 1 and those + 8, 16, 24
    float z[8];
    auto token = [&](int i) { return 2 * t + (i & 1) + (i >> 1) * 8; };
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = scores[token(i) * kDecHeads + head];
    if (tile >= full_tiles) {
      const bool in_ring = tile < ring_tiles;
      const int n = (in_ring ? n_ring : n_sink) - (in_ring ? tile : tile - ring_tiles) * kRows;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (token(i) >= n) z[i] = -INFINITY;
    }
    // ---- references
    float mx = max3(max3(z[0], z[1], z[2]), max3(z[3], z[4], z[5]), fmaxf(z[6], z[7]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    int big;
    {
      uint32_t w[NG], most = 0u;
      lds_words<NG>(w, vt + lane * C::ROW + C::CODES);
#pragma unroll
      for (int j = 0; j < NG; ++j) most = larger(w[j], most);
      big = __reduce_max_sync(kFull, static_cast<int>(max(most & 0xffffu, most >> 16)));
    }
    big = max((big >> 7) - 128, kSizeMin);
    if (__any_sync(kFull, mx > ref + static_cast<float>(kSlack)) || big > size) {
      const float next = mx > ref + static_cast<float>(kSlack) ? mx : ref;
      const float alpha = ref == -INFINITY ? 0.f : ex2_approx(ref - next);
      const float a0 = __shfl_sync(kFull, alpha, 8 * t), a1 = __shfl_sync(kFull, alpha, 8 * t + 4);
      const float down = size - big < -126 ? 0.f : pow2(min(size - big, 0));
      ref = next;
      size = max(size, big);
      l *= alpha;
      om[0] *= a0 * down;
      om[1] *= a1 * down;
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[j][x][0] *= a0 * down; o[j][x][1] *= a1 * down; o[j][x][2] *= a0 * down; o[j][x][3] *= a1 * down;
        }
    }
    const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = ex2_approx(z[i] - base);
    l += ((z[0] + z[1]) + (z[2] + z[3])) + ((z[4] + z[5]) + (z[6] + z[7]));
    {
      const float unit = pow2(kTop - size);
#pragma unroll
      for (int i = 0; i < 8; i += 2) f2_unpack(f2_mul(f2_pack(z[i], z[i + 1]), f2_pack(unit, unit)), z[i], z[i + 1]);
    }

    // ---- O += P V, 16 tokens at a time
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint8_t* v0 = vt + 16 * hf * C::ROW;
      uint32_t p0[NG], p1[NG], p2[NG], p3[NG];
      lds_words<NG>(p0, v0 + vpar);
      lds_words<NG>(p1, v0 + vpar + C::ROW);
      lds_words<NG>(p2, v0 + vpar + 8 * C::ROW);
      lds_words<NG>(p3, v0 + vpar + 9 * C::ROW);
      uint32_t ph0, ph1, pl0, pl1;
      split_bf16(f2_pack(z[4 * hf], z[4 * hf + 1]), ph0, pl0);
      split_bf16(f2_pack(z[4 * hf + 2], z[4 * hf + 3]), ph1, pl1);
      {
        // the minima times P in two bf16 parts: row g of the product is group g % NG, and so is row g + 8
        const uint8_t* q = v0 + vpar + g % NG * 4;
        const uint32_t m0 = __byte_perm(*reinterpret_cast<const uint32_t*>(q),
                                        *reinterpret_cast<const uint32_t*>(q + C::ROW), 0x7632);
        const uint32_t m1 = __byte_perm(*reinterpret_cast<const uint32_t*>(q + 8 * C::ROW),
                                        *reinterpret_cast<const uint32_t*>(q + 9 * C::ROW), 0x7632);
        if constexpr (FEW) {
          mma_bf16_16816(om, m0, m0, m1, m1, low_part ? pl0 : ph0, low_part ? pl1 : ph1);
        } else {
          mma_bf16_16816(om, m0, m0, m1, m1, ph0, ph1);
          mma_bf16_16816(om, m0, m0, m1, m1, pl0, pl1);
        }
      }
      // FEW: this lane's column takes the high part less nothing, or the low part, which is less the high one
      const uint32_t less0 = (ph0 ^ 0x80008000u) & low_part, less1 = (ph1 ^ 0x80008000u) & low_part;
      if constexpr (FEW) {
        pl0 &= low_part;
        pl1 &= low_part;
      }
      uint32_t va[NG / 2], vb[NG / 2], vc[NG / 2], vd[NG / 2];
      lds_words<NG / 2>(va, v0 + vcode);
      lds_words<NG / 2>(vb, v0 + vcode + C::ROW);
      lds_words<NG / 2>(vc, v0 + vcode + 8 * C::ROW);
      lds_words<NG / 2>(vd, v0 + vcode + 9 * C::ROW);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const uint32_t a0 = __byte_perm(p0[j], p1[j], 0x5410), a1 = __byte_perm(p2[j], p3[j], 0x5410);
        // elements 4 g + i of group j: tokens 2t (low half) and 2t + 1
        const uint32_t x = __byte_perm(va[j >> 1], vb[j >> 1], (j & 1) ? 0x7632 : 0x5410);
        const uint32_t y = __byte_perm(vc[j >> 1], vd[j >> 1], (j & 1) ? 0x7632 : 0x5410);
        const uint32_t xh = x >> 8, yh = y >> 8;
        const uint32_t e0 = x & 0x000f000fu, e1 = xh & 0x000f000fu, e2 = y & 0x000f000fu, e3 = yh & 0x000f000fu;
        const uint32_t d0 = x & 0x00f000f0u, d1 = xh & 0x00f000f0u, d2 = y & 0x00f000f0u, d3 = yh & 0x00f000f0u;
        if constexpr (FEW) {
          const uint32_t b0 = low_times_step(ph0, pl0, mul_bf16x2(less0, a0), a0);
          const uint32_t b1 = low_times_step(ph1, pl1, mul_bf16x2(less1, a1), a1);
          mma_bf16_16816(o[j][0], e0, e1, e2, e3, b0, b1);
          mma_bf16_16816(o[j][1], d0, d1, d2, d3, b0, b1);
        } else {
          const uint32_t h0 = mul_bf16x2(ph0, a0), h1 = mul_bf16x2(ph1, a1);
          const uint32_t l0 = low_times_step(ph0, pl0, h0 ^ 0x80008000u, a0);
          const uint32_t l1 = low_times_step(ph1, pl1, h1 ^ 0x80008000u, a1);
          mma_bf16_16816(o[j][0], e0, e1, e2, e3, h0, h1);
          mma_bf16_16816(o[j][1], d0, d1, d2, d3, h0, h1);
          mma_bf16_16816(o[j][0], e0, e1, e2, e3, l0, l1);
          mma_bf16_16816(o[j][1], d0, d1, d2, d3, l0, l1);
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- this warp's state, in its own (now idle) stages, relative to its own sum, so that the references
  // of two warps differ by no more than their shares and large V stays finite: l in [2^-9, 2^-8)
  static_assert(2 * sizeof(Partial<D>) <= kStages * C::STAGE, "a warp's state and the block's fit a warp's stages");
  auto part = [&](int w) { return reinterpret_cast<Partial<D>*>(smem + w * C::WARP); };
  Partial<D>* pt = part(warp);
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
  if constexpr (FEW) {  // high and low parts
#pragma unroll
    for (int i = 0; i < 2; ++i) om[i] += __shfl_xor_sync(kFull, om[i], 2);
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][x][i] += __shfl_xor_sync(kFull, o[j][x][i], 2);
  }
  // without keys, or with a NaN or an infinity among them, as it is
  const int shift = l > 0.f && l < INFINITY ? static_cast<int>(__float_as_uint(l) >> 23) - 127 + 9 : 0;
  constexpr int kDown = 64;  // on the way, so that no factor leaves the range of a float
  const float fix = pow2(-shift), unit = pow2(size - kTop + kDown);
  const float f0 = __shfl_sync(kFull, fix, 8 * t), f1 = __shfl_sync(kFull, fix, 8 * t + 4);
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    const float m0 = __shfl_sync(kFull, om[0], 4 * j + t), m1 = __shfl_sync(kFull, om[1], 4 * j + t);
    const float kEven = pow2(133 - kDown), kOdd = pow2(129 - kDown);
    auto value = [&](float x, float code, float m, float f) { return fmaf(x, code, m * pow2(-kDown)) * f * unit; };
    if (2 * t < G)
      *reinterpret_cast<float4*>(&pt->o[2 * t][32 * j + 4 * g]) =
          make_float4(value(o[j][0][0], kEven, m0, f0), value(o[j][1][0], kOdd, m0, f0),
                      value(o[j][0][2], kEven, m0, f0), value(o[j][1][2], kOdd, m0, f0));
    if (2 * t + 1 < G)
      *reinterpret_cast<float4*>(&pt->o[2 * t + 1][32 * j + 4 * g]) =
          make_float4(value(o[j][0][1], kEven, m1, f1), value(o[j][1][1], kOdd, m1, f1),
                      value(o[j][0][3], kEven, m1, f1), value(o[j][1][3], kOdd, m1, f1));
  }
  if (t == 0) {
    pt->ref[g] = ref + static_cast<float>(shift);
    pt->l[g] = l * fix;
  }
  merge_and_store<D>(part, part(0) + 1, s_lse2, G, c, rank, head0, a.out, a.out_f32 != 0, a.lse);
  merge_done(c);
}

template <int D, bool FEW>
cudaError_t launch_impl(const Kv4DecodeArgs& a, int sms, cudaStream_t stream) {
  const size_t smem = kDecWarps * K4<D>::WARP;
  const long long segments = static_cast<long long>(a.B) * a.Hkv;
  const long long tiles = (static_cast<long long>(a.W) + a.S + kRows - 1) / kRows;
  // 512 segments, with P in fp16: 73 us with one block each (3.5 on an SM: some have 4), 66 us with two, 84 us with
  // four, whose starts and merges weigh more
  const int c = decode_cluster(segments, tiles, sms, kBlocksPerSm, 1);
  if (segments * c > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = allow_shared<swa_kv4_decode_kernel<D, FEW>>(static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_decode_cluster(swa_kv4_decode_kernel<D, FEW>, a, segments, c, smem, stream);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int d, int sms, cudaStream_t stream) {
  if (a.G <= 4) return d == 128 ? launch_impl<128, true>(a, sms, stream) : launch_impl<64, true>(a, sms, stream);
  return d == 128 ? launch_impl<128, false>(a, sms, stream) : launch_impl<64, false>(a, sms, stream);
}

}  // namespace swa

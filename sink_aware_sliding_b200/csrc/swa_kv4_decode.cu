// Decode over the 4-bit ring cache (layout: swa_kv4.cu).
//
// With codes n in 0..15, steps a and minima b of the groups j of a row,
//   z_h = scale sum_j [ a_j (n_j . q_hj) + b_j sum(q_hj) ]
//   O_h = sum_keys p_h [ a_j n_j + b_j ].
// The integer part runs on the tensor cores with the codes as they are: a nibble in
// the low bits of an fp16 word is the subnormal n 2^-24, one four bits higher is
// 16 n 2^-24, so that "unpacking" is one AND per two elements and loses nothing.  q is
// scaled by a power of two per head into fp16 (exact for all but elements 2^-28 below
// the head's largest), and the odd nibbles' factor 16 goes into q and, for V, into the
// final scaling.  Scores, steps and minima are applied in fp32.  p a_j is the one value
// that is rounded, to fp16 (relative 2^-12): softmax numerators in 16 bits as in the
// bf16 decode, with the running reference chosen so that p a_j stays below 2^15
// whatever the steps are; the minima's part, sum p b_j, stays in fp32.
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
constexpr int kStages = 4;

template <int D>
struct K4 {
  static constexpr int NG = D / kKv4Group;
  static constexpr int ROW = kv4_row_bytes(D);
  static constexpr int CODES = D / 2;                    // code bytes of a row
  static constexpr int PAR = 4 * NG;                     // parameter bytes of a row
  static constexpr int UNIT = D == 128 ? 16 : 8;         // bytes per copy: what a row is aligned to
  static constexpr int UNITS = ROW / UNIT;               // 5
  static constexpr int COPIES = (kDecTile * UNITS + 31) / 32;  // per lane, for K and again for V
  static constexpr int HALF = kDecTile * ROW;            // K's or V's bytes of a stage
  static constexpr int STAGE = 2 * HALF;
};

// Key rows of a tile that lane (g, t) multiplies: t, 4 + (t ^ X) and those + 8.  X and
// the order of the 16-byte chunks in shared memory (chunk c of row r at c ^ (r & 2) for
// d = 128) keep both the K reads (two rows per quarter warp) and the V reads (four rows)
// off each other's banks.
template <int D>
__device__ __forceinline__ int row_lo(int n) {  // token of column n of a score tile
  constexpr int X = D == 128 ? 1 : 2;
  return (n & 1) ? 4 + ((n >> 1) ^ X) : n >> 1;
}
template <int D>
__device__ __forceinline__ int code_at(int r, int byte) {  // where byte of row r's codes lies in a tile
  if constexpr (D == 128) return r * 64 + ((((byte >> 4) ^ (r & 2)) << 4) | (byte & 15));
  return r * 32 + byte;
}

__device__ __forceinline__ float step_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
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

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32, 4) swa_kv4_decode_kernel(const __grid_constant__ Kv4DecodeArgs a,
                                                                          int c) {
  using C = K4<D>;
  constexpr int NG = C::NG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Partial<D> s_mine;
  __shared__ float s_lse2[kDecHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % c;
  const size_t seg = blockIdx.x / c;
  const int b = static_cast<int>(seg / a.Hkv), kvh = static_cast<int>(seg % a.Hkv);
  const int G = a.G, W = a.W, S = a.S;
  const size_t head0 = static_cast<size_t>(b) * a.Hq + static_cast<size_t>(kvh) * G;

  const int p = a.pos[b];
  const int n_ring = p < 0 ? 0 : (p < W ? p + 1 : W);
  const int n_sink = p < W ? 0 : min(p - W + 1, S);
  const int ring_tiles = (n_ring + kDecTile - 1) / kDecTile;
  const int tiles = ring_tiles + (n_sink + kDecTile - 1) / kDecTile;
  const uint8_t* kc = a.kc + seg * W * C::ROW;
  const uint8_t* vc = a.vc + seg * W * C::ROW;
  const uint8_t* sk = a.sk + seg * S * C::ROW;
  const uint8_t* sv = a.sv + seg * S * C::ROW;

  uint8_t* ring = smem + warp * (kStages * C::STAGE);
  const uint32_t ring_u32 = smem_u32(ring);
  // where this lane's copies go within a half stage
  int copy_row[C::COPIES];
  uint32_t copy_dst[C::COPIES];
#pragma unroll
  for (int i = 0; i < C::COPIES; ++i) {
    const int u = lane + 32 * i;
    const int r = u / C::UNITS, byte = (u % C::UNITS) * C::UNIT;
    copy_row[i] = u < kDecTile * C::UNITS ? r : kDecTile;  // kDecTile: none
    copy_dst[i] = byte < C::CODES ? code_at<D>(r, byte) : kDecTile * C::CODES + r * C::PAR + byte - C::CODES;
  }
  auto issue = [&](int tile, int stage) {
    if (tile < tiles) {
      const bool in_ring = tile < ring_tiles;
      const int first = (in_ring ? tile : tile - ring_tiles) * kDecTile;
      const int n = min(kDecTile, (in_ring ? n_ring : n_sink) - first);
      const uint8_t* ks = (in_ring ? kc : sk) + static_cast<size_t>(first) * C::ROW;
      const uint8_t* vs = (in_ring ? vc : sv) + static_cast<size_t>(first) * C::ROW;
      const uint32_t dst = ring_u32 + stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < C::COPIES; ++i) {
        if (copy_row[i] < kDecTile) {
          const bool real = copy_row[i] < n;
          const int off = real ? (lane + 32 * i) * C::UNIT : 0;
          cp_async<C::UNIT>(dst + copy_dst[i], ks + off, real);
          cp_async<C::UNIT>(dst + C::HALF + copy_dst[i], vs + off, real);
        }
      }
    }
    cp_async_commit();
  };

  const int nw = c * kDecWarps;
  int tile = rank * kDecWarps + warp;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(tile + s * nw, s);

  // ---- q of head g: fp16 fragments scaled by 2^-qe, and the sums of its groups
  uint32_t qa[NG][4];
  float qsum[NG];
  float qscale;
  {
    const bool real = g < G;
    const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) + (head0 + (real ? g : 0)) * D;
    float x[NG][8];
    float mx = 0.f;
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
      qsum[j] = sum * a.scale_log2;
    }
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    // largest element to [2^14, 2^15)
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    e = min(max(e, -100), 100) - 14;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    qscale = __uint_as_float(static_cast<uint32_t>(127 + e + 12) << 23) * (a.scale_log2 * 4096.f);  // 2^(e + 24)
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      // k-slots of the two products: nibbles (0, 2), then (1, 3), which carry a factor 16
      qa[j][0] = pack_f16(x[j][0] * down, x[j][4] * down);
      qa[j][1] = pack_f16(x[j][2] * down, x[j][6] * down);
      qa[j][2] = pack_f16(x[j][1] * down * 0.0625f, x[j][5] * down * 0.0625f);
      qa[j][3] = pack_f16(x[j][3] * down * 0.0625f, x[j][7] * down * 0.0625f);
    }
  }

  float o[NG][2][4];
  float omin[NG];
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    omin[j] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) o[j][x][0] = o[j][x][1] = o[j][x][2] = o[j][x][3] = 0.f;
  }
  float ref = -INFINITY, l = 0.f;
  const int row_n = row_lo<D>(g);                           // K: this lane's token of a score tile (and + 8)
  const int r0 = row_lo<D>(2 * t), r1 = row_lo<D>(2 * t + 1);  // scores and V: this lane's tokens (and + 8)

  int stage = 0;
  for (; tile < tiles; tile += nw) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // this tile has arrived for every lane, and every lane is done with the one before
    issue(tile + (kStages - 1) * nw, stage == 0 ? kStages - 1 : stage - 1);
    const uint8_t* kt = ring + stage * C::STAGE;
    const uint8_t* vt = kt + C::HALF;
    const uint8_t* kp = kt + kDecTile * C::CODES;
    const uint8_t* vp = vt + kDecTile * C::CODES;
    const bool in_ring = tile < ring_tiles;
    const int n = (in_ring ? n_ring : n_sink) - (in_ring ? tile : tile - ring_tiles) * kDecTile;

    // ---- scores of head g for the tokens r0, r1, r0 + 8, r1 + 8
    float z[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      uint32_t w[NG];
      lds_words<NG>(w, kt + code_at<D>(row_n + 8 * nt, t * (C::CODES / 4)));
      uint32_t pa[NG], pb[NG];
      lds_words<NG>(pa, kp + (r0 + 8 * nt) * C::PAR);
      lds_words<NG>(pb, kp + (r1 + 8 * nt) * C::PAR);
      float za = 0.f, zb = 0.f, ma = 0.f, mb = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        // elements 8 t + i (low half) and 8 t + 4 + i of group j
        const uint32_t x = __byte_perm(w[j >> 1], w[(j >> 1) + NG / 2], (j & 1) ? 0x7632 : 0x5410);
        const uint32_t y = x >> 8;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16_16816(acc, qa[j][0], 0u, qa[j][1], 0u, x & 0x000f000fu, y & 0x000f000fu);
        mma_f16_16816(acc, qa[j][2], 0u, qa[j][3], 0u, x & 0x00f000f0u, y & 0x00f000f0u);
        za = fmaf(step_of(pa[j]), acc[0], za);
        zb = fmaf(step_of(pb[j]), acc[1], zb);
        ma = fmaf(low_of(pa[j]), qsum[j], ma);
        mb = fmaf(low_of(pb[j]), qsum[j], mb);
      }
      z[2 * nt] = fmaf(za, qscale, ma);
      z[2 * nt + 1] = fmaf(zb, qscale, mb);
    }
    if (n < kDecTile) {
      if (r0 >= n) z[0] = -INFINITY;
      if (r1 >= n) z[1] = -INFINITY;
      if (r0 + 8 >= n) z[2] = -INFINITY;
      if (r1 + 8 >= n) z[3] = -INFINITY;
    }
    // ---- reference: p times the tile's largest step stays within fp16
    float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    // exponent of the tile's largest step, or of its largest |minimum| less 24 where that is
    // more (groups of one value), as bf16 bits
    auto size_of = [](uint32_t w) {
      return max(static_cast<int>(w & 0x7fffu), static_cast<int>((w >> 16) & 0x7fffu) - (24 << 7));
    };
    int big;
    if constexpr (D == 128) {
      const uint2 w = *reinterpret_cast<const uint2*>(vp + lane * 8);
      big = max(size_of(w.x), size_of(w.y));
    } else {
      big = size_of(*reinterpret_cast<const uint32_t*>(vp + lane * 4));
    }
    big = __reduce_max_sync(kFull, big);
    const int be = min(max((big >> 7) - 127, -90), 100);
    // p a_j < 2^(8 + 1) at the reference, up to 2^15 before it is moved
    const float want = mx + static_cast<float>(be - 8);
    if (__any_sync(kFull, want > ref + 6.f)) {
      const float next = want > ref + 6.f ? want : ref;
      const float alpha = ref == -INFINITY ? 0.f : ex2_approx(ref - next);
      const float a0 = __shfl_sync(kFull, alpha, 8 * t), a1 = __shfl_sync(kFull, alpha, 8 * t + 4);
      ref = next;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        omin[j] *= alpha;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[j][x][0] *= a0; o[j][x][1] *= a1; o[j][x][2] *= a0; o[j][x][3] *= a1;
        }
      }
    }
    const float base = ref == -INFINITY ? 0.f : ref;
    float pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(z[i] - base);
    l += (pr[0] + pr[1]) + (pr[2] + pr[3]);

    // ---- O += P V
    uint32_t va[NG / 2], vb[NG / 2], vc2[NG / 2], vd[NG / 2];
    lds_words<NG / 2>(va, vt + code_at<D>(r0, g * 2 * NG));
    lds_words<NG / 2>(vb, vt + code_at<D>(r1, g * 2 * NG));
    lds_words<NG / 2>(vc2, vt + code_at<D>(r0 + 8, g * 2 * NG));
    lds_words<NG / 2>(vd, vt + code_at<D>(r1 + 8, g * 2 * NG));
    uint32_t p0[NG], p1[NG], p2[NG], p3[NG];
    lds_words<NG>(p0, vp + r0 * C::PAR);
    lds_words<NG>(p1, vp + r1 * C::PAR);
    lds_words<NG>(p2, vp + (r0 + 8) * C::PAR);
    lds_words<NG>(p3, vp + (r1 + 8) * C::PAR);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      omin[j] += (pr[0] * low_of(p0[j]) + pr[1] * low_of(p1[j])) + (pr[2] * low_of(p2[j]) + pr[3] * low_of(p3[j]));
      const uint32_t b0 = pack_f16(pr[0] * step_of(p0[j]), pr[1] * step_of(p1[j]));
      const uint32_t b1 = pack_f16(pr[2] * step_of(p2[j]), pr[3] * step_of(p3[j]));
      // elements 4 g + i of group j: tokens r0 (low half) and r1
      const uint32_t x = __byte_perm(va[j >> 1], vb[j >> 1], (j & 1) ? 0x7632 : 0x5410);
      const uint32_t y = __byte_perm(vc2[j >> 1], vd[j >> 1], (j & 1) ? 0x7632 : 0x5410);
      const uint32_t xh = x >> 8, yh = y >> 8;
      mma_f16_16816(o[j][0], x & 0x000f000fu, xh & 0x000f000fu, y & 0x000f000fu, yh & 0x000f000fu, b0, b1);
      mma_f16_16816(o[j][1], x & 0x00f000f0u, xh & 0x00f000f0u, y & 0x00f000f0u, yh & 0x00f000f0u, b0, b1);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- this warp's state, in its own (now idle) stages
  static_assert(sizeof(Partial<D>) <= kStages * C::STAGE, "a partial state fits a warp's stages");
  auto part = [&](int w) { return reinterpret_cast<Partial<D>*>(smem + w * (kStages * C::STAGE)); };
  Partial<D>* pt = part(warp);
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    float m = omin[j];
    m += __shfl_xor_sync(kFull, m, 1);
    m += __shfl_xor_sync(kFull, m, 2);
    const float m0 = __shfl_sync(kFull, m, 8 * t), m1 = __shfl_sync(kFull, m, 8 * t + 4);
    constexpr float kEven = 16777216.f, kOdd = 1048576.f;  // 2^24, 2^20
    if (2 * t < G)
      *reinterpret_cast<float4*>(&pt->o[2 * t][32 * j + 4 * g]) =
          make_float4(fmaf(o[j][0][0], kEven, m0), fmaf(o[j][1][0], kOdd, m0), fmaf(o[j][0][2], kEven, m0),
                      fmaf(o[j][1][2], kOdd, m0));
    if (2 * t + 1 < G)
      *reinterpret_cast<float4*>(&pt->o[2 * t + 1][32 * j + 4 * g]) =
          make_float4(fmaf(o[j][0][1], kEven, m1), fmaf(o[j][1][1], kOdd, m1), fmaf(o[j][0][3], kEven, m1),
                      fmaf(o[j][1][3], kOdd, m1));
  }
  if (t == 0) {
    pt->ref[g] = ref;
    pt->l[g] = l;
  }
  merge_and_store<D>(part, &s_mine, s_lse2, G, c, rank, head0, a.out, a.out_f32 != 0, a.lse);
}

template <int D>
cudaError_t launch_impl(const Kv4DecodeArgs& a, int sms, cudaStream_t stream) {
  const size_t smem = kDecWarps * kStages * K4<D>::STAGE;
  const long long segments = static_cast<long long>(a.B) * a.Hkv;
  const long long tiles = (static_cast<long long>(a.W) + a.S + kDecTile - 1) / kDecTile;
  const int c = decode_cluster(segments, tiles, sms, 4, 2);
  if (segments * c > INT32_MAX) return cudaErrorInvalidValue;
  static_assert(kDecWarps * kStages * K4<D>::STAGE <= 48 * 1024, "no opt-in shared memory needed");
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
  return cudaLaunchKernelEx(&cfg, swa_kv4_decode_kernel<D>, a, c);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int d, int sms, cudaStream_t stream) {
  return d == 128 ? launch_impl<128>(a, sms, stream) : launch_impl<64>(a, sms, stream);
}

}  // namespace swa

// C ABI of libswa: argument checks, TMA descriptors, launch configuration.
// Declarations and contracts: include/swa.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/swa.h"
#include "based_linear.h"
#include "fixed_cache.h"
#include "hh_scores.h"
#include "swa_internal.h"

namespace {

// Device error word: kernels set it (first writer wins) when a bounded wait expires.
__device__ int g_swa_error;

std::atomic<unsigned long long> g_timeout_ns{2000000000ull};
std::atomic<int> g_debug_flags{0};

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool ready = false;
  int sms = 0;
  int decode_ctas_per_sm[2] = {0, 0};  // d = 64, 128 (for B <= 4096 table)
  int* err = nullptr;
};
std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

int device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SWA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SWA_ERR_CUDA;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_swa_error) != cudaSuccess) return SWA_ERR_CUDA;
    d.err = static_cast<int*>(p);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return SWA_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiled>(fn);
    }
    d.ready = true;
  }
  *out = &d;
  return SWA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// 3-D tiled map over a [rows, heads, d] tensor: box = {128 bytes of d, 1 head, box_rows}.
// atom32: 128-byte swizzle with 32-byte atoms (fp32 operands read in MN-major order).
int make_map(CUtensorMap* m, const void* ptr, bool f32, int d, int heads, long long rows,
             int box_rows, bool atom32 = false) {
  const int elem = f32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * elem,
                           static_cast<cuuint64_t>(d) * elem * heads};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem), 1u, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        atom32 ? CU_TENSOR_MAP_SWIZZLE_128B_ATOM_32B : CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SWA_OK : SWA_ERR_CUDA;
}

int check_heads(int Hq, int Hkv, int d, int window, int n_sink, float scale, int dtype) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return SWA_ERR_INVALID_ARG;
  if (window < 1 || n_sink < 0) return SWA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (dtype != SWA_DTYPE_BF16 && dtype != SWA_DTYPE_F32 && dtype != SWA_DTYPE_BF16_F32OUT)
    return SWA_ERR_INVALID_ARG;
  if (d <= 0) return SWA_ERR_INVALID_ARG;
  if (dtype != SWA_DTYPE_F32 && d != 64 && d != 128) return SWA_ERR_UNSUPPORTED;
  if (dtype == SWA_DTYPE_F32 && d != 64) return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

int run_prefill(const void* q, const void* k, const void* v, void* out, float* lse,
                const int32_t* cu, int n_seq, int L, long long T, int Hq, int Hkv, int d,
                int window, int n_sink, float scale, int dtype, cudaStream_t stream) {
  DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != SWA_OK) return st;
  const bool f32 = dtype == SWA_DTYPE_F32;
  CUtensorMap tq, tk, tv, to;
  std::memset(&to, 0, sizeof(to));
  if ((st = make_map(&tq, q, f32, d, Hq, T, swa::kBM)) != SWA_OK) return st;
  if (dtype == SWA_DTYPE_BF16 && (st = make_map(&to, out, false, d, Hq, T, swa::kBM)) != SWA_OK) return st;
  if ((st = make_map(&tk, k, f32, d, Hkv, T, swa::kBN)) != SWA_OK) return st;
  if ((st = make_map(&tv, v, f32, d, Hkv, T, swa::kBN, f32)) != SWA_OK) return st;
  swa::PrefillArgs a{};
  a.out = out;
  a.lse = lse;
  a.cu_seqlens = cu;
  a.n_seq = n_seq;
  a.L = L;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.window = window;
  a.n_sink = n_sink;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.lse_varlen = cu != nullptr ? 1 : 0;
  a.timeout_ns = g_timeout_ns.load();
  a.debug_flags = g_debug_flags.load();
  a.err = dev->err;
  long long units;
  if (cu == nullptr) {
    const long long tiles = static_cast<long long>(n_seq) * ((L + swa::kBM - 1) / swa::kBM);
    if (tiles * Hq > INT32_MAX) return SWA_ERR_UNSUPPORTED;
    a.total_tiles = static_cast<int>(tiles);
    units = tiles * Hq;
  } else {
    a.total_tiles = -1;
    units = (T / swa::kBM + n_seq) * static_cast<long long>(Hq);  // upper bound
    if (units > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  }
  // Debug flag 4 skips the short-window stream kernel, flag 2 forces the one-tile
  // kernel (so tests can check every kernel on the same inputs).
  if ((a.debug_flags & 6) == 0 && swa::prefill_stream_supported(d, f32, window, n_sink)) {
    const int grid_s = static_cast<int>(std::min<long long>(dev->sms, units));
    cudaError_t es = swa::launch_prefill_stream(a, tq, tk, tv, to, dtype != SWA_DTYPE_BF16, grid_s, stream);
    if (es != cudaErrorNotSupported) return es == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
  }
  const bool pair = (a.debug_flags & 2) == 0 && swa::prefill_pair_supported(Hq, Hq / Hkv, d, f32);
  if (pair) units = (units + 1) / 2;
  const int grid = static_cast<int>(std::min<long long>(dev->sms, units));
  if (grid <= 0) return SWA_OK;
  cudaError_t e = cudaErrorNotSupported;
  if (pair) e = swa::launch_prefill_pair(a, tq, tk, tv, to, d, f32, dtype != SWA_DTYPE_BF16, grid, stream);
  if (e == cudaErrorNotSupported) {  // one-tile kernel (odd Hq, or the two-tile kernel declined)
    const int grid1 = static_cast<int>(std::min<long long>(dev->sms, pair ? 2 * units : units));
    e = swa::launch_prefill(a, tq, tk, tv, d, f32, dtype != SWA_DTYPE_BF16, grid1, stream);
  }
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

// Split-K decode grid: one warp per kDecodeKeysPerWarp keys of the largest
// possible visible set (every segment holds at most window + n_sink keys; the
// positions themselves are on the device), and never more CTAs than fill the GPU.
constexpr long long kDecodeKeysPerWarp = 64;
int decode_grid(DeviceInfo* dev, int d, int B, int Hkv, int window, int n_sink, int* grid) {
  const int idx = d == 128 ? 1 : 0;
  if (dev->decode_ctas_per_sm[idx] == 0) {
    int c = 0;
    if (swa::decode_occupancy(d, 4096, &c) != cudaSuccess || c <= 0) return SWA_ERR_CUDA;
    dev->decode_ctas_per_sm[idx] = c;
  }
  const long long full = static_cast<long long>(dev->sms) * dev->decode_ctas_per_sm[idx];
  const long long max_keys = static_cast<long long>(B) * Hkv * (static_cast<long long>(window) + n_sink);
  const long long warps = (max_keys + kDecodeKeysPerWarp - 1) / kDecodeKeysPerWarp;
  const long long wpc = swa::decode_threads() / 32;
  *grid = static_cast<int>(std::max(1LL, std::min(full, (warps + wpc - 1) / wpc)));
  return SWA_OK;
}

}  // namespace

extern "C" {

int swa_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Hq,
            int Hkv, int L, int d, int window, int n_sink, float scale, int dtype,
            swa_stream_t stream) {
  int st = check_heads(Hq, Hkv, d, window, n_sink, scale, dtype);
  if (st != SWA_OK) return st;
  if (B < 0 || L < 0) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * L == 0) return SWA_OK;
  if (!q || !k || !v || !out) return SWA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return SWA_ERR_INVALID_ARG;
  const long long T = static_cast<long long>(B) * L;
  if (T > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  return run_prefill(q, k, v, out, lse, nullptr, B, L, T, Hq, Hkv, d, window, n_sink, scale, dtype,
                     reinterpret_cast<cudaStream_t>(stream));
}

int swa_fwd_varlen(const void* q, const void* k, const void* v, void* out, float* lse,
                   const int32_t* cu_seqlens, int n_seq, long long T, int Hq, int Hkv, int d,
                   int window, int n_sink, float scale, int dtype, swa_stream_t stream) {
  int st = check_heads(Hq, Hkv, d, window, n_sink, scale, dtype);
  if (st != SWA_OK) return st;
  if (n_seq < 1 || T < 0 || !cu_seqlens) return SWA_ERR_INVALID_ARG;
  if (n_seq > swa::kMaxSeqSmem) return SWA_ERR_UNSUPPORTED;
  if (T > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  if (T == 0) return SWA_OK;
  if (!q || !k || !v || !out) return SWA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) ||
      (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return SWA_ERR_INVALID_ARG;
  return run_prefill(q, k, v, out, lse, cu_seqlens, n_seq, 0, T, Hq, Hkv, d, window, n_sink, scale,
                     dtype, reinterpret_cast<cudaStream_t>(stream));
}

static int check_cache_shape(int B, int Hkv, int d, int window, int n_sink) {
  if (B < 0 || Hkv <= 0 || window < 1 || n_sink < 0) return SWA_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? SWA_OK : SWA_ERR_UNSUPPORTED;
}

static int check_cache(int B, int Hkv, int d, int window, int n_sink, const void* kc,
                       const void* vc, const void* sk, const void* sv) {
  const int st = check_cache_shape(B, Hkv, d, window, n_sink);
  if (st != SWA_OK) return st;
  if (!kc || !vc || !aligned16(kc) || !aligned16(vc)) return SWA_ERR_INVALID_ARG;
  if (n_sink > 0 && (!sk || !sv || !aligned16(sk) || !aligned16(sv))) return SWA_ERR_INVALID_ARG;
  return SWA_OK;
}

int swa_cache_fill(const void* k, const void* v, int P, void* kcache, void* vcache, void* sink_k,
                   void* sink_v, int B, int Hkv, int d, int window, int n_sink,
                   swa_stream_t stream) {
  int st = check_cache(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (P < 0) return SWA_ERR_INVALID_ARG;
  if (P == 0 || B == 0) return SWA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return SWA_ERR_INVALID_ARG;
  cudaError_t e = swa::launch_cache_fill(k, v, P, kcache, vcache, sink_k, sink_v, B, Hkv, d, window,
                                         n_sink, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_cache_append(const void* k_new, const void* v_new, const int32_t* pos, void* kcache,
                     void* vcache, void* sink_k, void* sink_v, int B, int Hkv, int d, int window,
                     int n_sink, swa_stream_t stream) {
  int st = check_cache(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  if (!k_new || !v_new || !pos || !aligned16(k_new) || !aligned16(v_new) ||
      (reinterpret_cast<uintptr_t>(pos) & 3u))
    return SWA_ERR_INVALID_ARG;
  cudaError_t e = swa::launch_cache_append(k_new, v_new, pos, kcache, vcache, sink_k, sink_v, B, Hkv,
                                           d, window, n_sink, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

static int decode_shape_ok(int B, int Hq, int Hkv, int d, int window, int n_sink) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || window < 1 || n_sink < 0)
    return SWA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SWA_ERR_UNSUPPORTED;
  if (Hq / Hkv > 8) return SWA_ERR_UNSUPPORTED;
  if (B > 4096) return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

size_t swa_decode_workspace_bytes(int B, int Hq, int Hkv, int d, int window, int n_sink) {
  if (decode_shape_ok(B, Hq, Hkv, d, window, n_sink) != SWA_OK) return 0;
  DeviceInfo* dev = nullptr;
  if (device_info(&dev) != SWA_OK) return 0;
  int grid = 0;
  if (decode_grid(dev, d, B, Hkv, window, n_sink, &grid) != SWA_OK) return 0;
  const size_t n_warps = static_cast<size_t>(grid) * (swa::decode_threads() / 32);
  const size_t slots = n_warps + static_cast<size_t>(B) * Hkv;
  return slots * swa::decode_partial_floats(Hq / Hkv, d) * sizeof(float);
}

}  // extern "C"

namespace swa {

int decode_args_status(const void* q, const void* kcache, const void* vcache, const void* sink_k,
                       const void* sink_v, const int32_t* pos, const void* out, const float* lse, int B,
                       int Hq, int Hkv, int d, int window, int n_sink, float scale, int out_dtype) {
  int st = decode_shape_ok(B, Hq, Hkv, d, window, n_sink);
  if (st != SWA_OK) return st;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_BF16_F32OUT) return SWA_ERR_INVALID_ARG;
  if (B == 0) return SWA_OK;
  if (!q || !pos || !out || !aligned16(q) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(pos) & 3u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return SWA_ERR_INVALID_ARG;
  return check_cache(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
}

}  // namespace swa

extern "C" {

static int run_decode(const void* q, const void* kcache, const void* vcache, const void* sink_k,
                      const void* sink_v, const int32_t* pos, void* out, float* lse, int B, int Hq,
                      int Hkv, int d, int window, int n_sink, float scale, int out_dtype, void* workspace,
                      size_t workspace_bytes, const swa::RopeTable* rope, swa_stream_t stream) {
  int st = swa::decode_args_status(q, kcache, vcache, sink_k, sink_v, pos, out, lse, B, Hq, Hkv, d, window,
                                   n_sink, scale, out_dtype);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  const size_t need = swa_decode_workspace_bytes(B, Hq, Hkv, d, window, n_sink);
  if (need == 0) return SWA_ERR_CUDA;
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SWA_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  int grid = 0;
  if ((st = decode_grid(dev, d, B, Hkv, window, n_sink, &grid)) != SWA_OK) return st;
  swa::DecodeArgs a{};
  a.q = q;
  a.kcache = kcache;
  a.vcache = vcache;
  a.sink_k = sink_k;
  a.sink_v = sink_v;
  a.pos = pos;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.W = window;
  a.S = n_sink;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.n_warps = grid * (swa::decode_threads() / 32);
  a.out_f32 = out_dtype == SWA_DTYPE_BF16_F32OUT ? 1 : 0;
  cudaError_t e = swa::launch_decode(a, d, grid, swa::decode_threads(),
                                     reinterpret_cast<cudaStream_t>(stream), rope);
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_decode(const void* q, const void* kcache, const void* vcache, const void* sink_k,
               const void* sink_v, const int32_t* pos, void* out, float* lse, int B, int Hq,
               int Hkv, int d, int window, int n_sink, float scale, void* workspace,
               size_t workspace_bytes, swa_stream_t stream) {
  return run_decode(q, kcache, vcache, sink_k, sink_v, pos, out, lse, B, Hq, Hkv, d, window, n_sink,
                    scale, SWA_DTYPE_BF16, workspace, workspace_bytes, nullptr, stream);
}

int swa_decode_ex(const void* q, const void* kcache, const void* vcache, const void* sink_k,
                  const void* sink_v, const int32_t* pos, void* out, float* lse, int B, int Hq, int Hkv,
                  int d, int window, int n_sink, float scale, int out_dtype, void* workspace,
                  size_t workspace_bytes, swa_stream_t stream) {
  return run_decode(q, kcache, vcache, sink_k, sink_v, pos, out, lse, B, Hq, Hkv, d, window, n_sink,
                    scale, out_dtype, workspace, workspace_bytes, nullptr, stream);
}

static bool rope_base_ok(double base) { return base > 0.0 && std::isfinite(base); }

int swa_decode_rope(const void* q, const void* kcache, const void* vcache, const void* sink_k,
                    const void* sink_v, const int32_t* pos, void* out, float* lse, int B, int Hq,
                    int Hkv, int d, int window, int n_sink, float scale, double rope_base,
                    void* workspace, size_t workspace_bytes, swa_stream_t stream) {
  if (!rope_base_ok(rope_base)) return SWA_ERR_INVALID_ARG;
  swa::RopeTable rt;
  swa::make_rope_table(rope_base, d, &rt);
  return run_decode(q, kcache, vcache, sink_k, sink_v, pos, out, lse, B, Hq, Hkv, d, window, n_sink,
                    scale, SWA_DTYPE_BF16, workspace, workspace_bytes, &rt, stream);
}

int swa_rope_qk(void* q, void* k, const int32_t* positions, long long n_tokens, int Hq, int Hkv, int d,
                double rope_base, swa_stream_t stream) {
  if (n_tokens < 0 || Hq < 0 || (k != nullptr && Hkv < 0) || !rope_base_ok(rope_base))
    return SWA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SWA_ERR_UNSUPPORTED;
  if (n_tokens == 0 || (Hq == 0 && (k == nullptr || Hkv == 0))) return SWA_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3u) || (Hq > 0 && (!q || !aligned16(q))) ||
      (k != nullptr && !aligned16(k)))
    return SWA_ERR_INVALID_ARG;
  swa::RopeTable rt;
  swa::make_rope_table(rope_base, d, &rt);
  cudaError_t e = swa::launch_rope_qk(Hq > 0 ? q : nullptr, k, positions, n_tokens, Hq, k ? Hkv : 0, d, rt,
                                      reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_rope_cache_append(const void* k_new, const void* v_new, const int32_t* pos, void* kcache,
                          void* vcache, void* sink_k, void* sink_v, int B, int Hkv, int d, int window,
                          int n_sink, double rope_base, swa_stream_t stream) {
  if (!rope_base_ok(rope_base)) return SWA_ERR_INVALID_ARG;
  int st = check_cache(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  if (!k_new || !v_new || !pos || !aligned16(k_new) || !aligned16(v_new) ||
      (reinterpret_cast<uintptr_t>(pos) & 3u))
    return SWA_ERR_INVALID_ARG;
  swa::RopeTable rt;
  swa::make_rope_table(rope_base, d, &rt);
  cudaError_t e = swa::launch_rope_append(k_new, v_new, pos, kcache, vcache, sink_k, sink_v, B, Hkv, d,
                                          window, n_sink, rt, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_bwd(const void* q, const void* k, const void* v, const void* out, const void* dout, const float* lse,
            float* dq, float* dk, float* dv, int B, int Hq, int Hkv, int L, int d, int window, int n_sink,
            float scale, swa_stream_t stream) {
  int st = check_heads(Hq, Hkv, d, window, n_sink, scale, SWA_DTYPE_BF16);
  if (st != SWA_OK) return st;
  if (B < 0 || L < 0) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * L == 0) return SWA_OK;
  const void* ptrs[9] = {q, k, v, out, dout, dq, dk, dv, nullptr};
  for (int i = 0; i < 8; ++i)
    if (!ptrs[i] || !aligned16(ptrs[i])) return SWA_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u)) return SWA_ERR_INVALID_ARG;
  const long long T = static_cast<long long>(B) * L;
  if (T > INT32_MAX || T * Hq > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  CUtensorMap tq, tk, tv, tdo;
  if ((st = make_map(&tq, q, false, d, Hq, T, swa::kBM)) != SWA_OK) return st;
  if ((st = make_map(&tk, k, false, d, Hkv, T, swa::kBN)) != SWA_OK) return st;
  if ((st = make_map(&tv, v, false, d, Hkv, T, swa::kBN)) != SWA_OK) return st;
  if ((st = make_map(&tdo, dout, false, d, Hq, T, swa::kBM)) != SWA_OK) return st;
  swa::BwdArgs ba{};
  swa::PrefillArgs& a = ba.pa;
  a.n_seq = B;
  a.L = L;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.window = window;
  a.n_sink = n_sink;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.total_tiles = static_cast<int>(static_cast<long long>(B) * ((L + swa::kBM - 1) / swa::kBM));
  a.timeout_ns = g_timeout_ns.load();
  a.debug_flags = g_debug_flags.load();
  a.err = dev->err;
  ba.out = out;
  ba.dout = dout;
  ba.lse = lse;
  ba.dq = dq;
  ba.dk = dk;
  ba.dv = dv;
  cudaError_t e = swa::launch_bwd(ba, tq, tk, tv, tdo, d, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_hybrid_decode(const void* q, const void* k_new, const void* v_new, const int32_t* pos, void* kcache,
                      void* vcache, void* sink_k, void* sink_v, void* out, float* lse, int B, int Hq, int Hkv,
                      int d, int window, int n_sink, float scale, const void* ql, const void* kl, const void* vl,
                      float* state, float* zsum, void* out_l, int H_l, int dk, int dv, float scale_l,
                      swa_stream_t stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || window < 1 || n_sink < 0 || H_l <= 0)
    return SWA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale) || !(scale_l > 0.f) || !std::isfinite(scale_l))
    return SWA_ERR_INVALID_ARG;
  if (!swa::hybrid_window_supported(d, window, n_sink) || dk != 16 || dv != 64) return SWA_ERR_UNSUPPORTED;
  if (B == 0) return SWA_OK;
  const void* ptrs[] = {q, k_new, v_new, kcache, vcache, out, ql, kl, vl, state, zsum, out_l};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return SWA_ERR_INVALID_ARG;
  if (n_sink > 0 && (!sink_k || !sink_v || !aligned16(sink_k) || !aligned16(sink_v))) return SWA_ERR_INVALID_ARG;
  if (!pos || (reinterpret_cast<uintptr_t>(pos) & 3u) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)))
    return SWA_ERR_INVALID_ARG;
  swa::HybridArgs a{};
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.pos = pos;
  a.kcache = kcache;
  a.vcache = vcache;
  a.sink_k = sink_k;
  a.sink_v = sink_v;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.W = window;
  a.S = n_sink;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.ql = ql;
  a.kl = kl;
  a.vl = vl;
  a.state = state;
  a.zsum = zsum;
  a.out_l = out_l;
  a.H_l = H_l;
  a.scale_l = scale_l;
  cudaError_t e = swa::launch_hybrid_decode(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_based_linear_state_features(int dk) { return dk > 0 ? swa::based_linear_features(dk) : 0; }

int swa_based_linear_fwd(const void* q, const void* k, const void* v, void* out, float* state, float* zsum,
                         int B, int L, int H, int dk, int dv, float scale, int out_dtype, swa_stream_t stream) {
  if (B < 0 || L < 0 || H <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_F32) return SWA_ERR_INVALID_ARG;
  if (dk != 16 || dv != 64) return SWA_ERR_UNSUPPORTED;
  if ((state == nullptr) != (zsum == nullptr)) return SWA_ERR_INVALID_ARG;
  // L = 0 still writes the (zero) state when one is asked for
  if (B == 0 || (L == 0 && state == nullptr)) return SWA_OK;
  if (L > 0 && (!q || !k || !v || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)))
    return SWA_ERR_INVALID_ARG;
  if (state != nullptr && !aligned16(state)) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  DeviceInfo* di = nullptr;
  const int st = device_info(&di);
  if (st != SWA_OK) return st;
  swa::BasedLinearArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  a.state = state;
  a.zsum = zsum;
  a.B = B;
  a.L = L;
  a.H = H;
  a.scale = scale;
  a.out_f32 = out_dtype == SWA_DTYPE_F32 ? 1 : 0;
  a.timeout_ns = g_timeout_ns.load();
  a.debug_flags = g_debug_flags.load();
  a.err = di->err;
  cudaError_t e = swa::launch_based_linear_fwd(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_based_linear_decode(const void* q, const void* k, const void* v, float* state, float* zsum, void* out,
                            int B, int H, int dk, int dv, float scale, int out_dtype, swa_stream_t stream) {
  if (B < 0 || H <= 0 || !(scale > 0.f) || !std::isfinite(scale)) return SWA_ERR_INVALID_ARG;
  if (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_F32) return SWA_ERR_INVALID_ARG;
  if (dk != 16 || dv != 64) return SWA_ERR_UNSUPPORTED;
  if (B == 0) return SWA_OK;
  if (!q || !k || !v || !state || !zsum || !out || !aligned16(state)) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  cudaError_t e = swa::launch_based_linear_decode(q, k, v, state, zsum, out, B, H, scale, out_dtype == SWA_DTYPE_F32,
                                                  reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

// An empty batch needs no cache: tensors without elements have no address.
static int check_kv4(int B, int Hkv, int d, int window, int n_sink, const void* kc, const void* vc, const void* sk,
                     const void* sv) {
  return B == 0 ? check_cache_shape(B, Hkv, d, window, n_sink)
                : check_cache(B, Hkv, d, window, n_sink, kc, vc, sk, sv);
}

size_t swa_kv4_row_bytes(int d) { return d == 64 || d == 128 ? swa::kv4_row_bytes(d) : 0; }

int swa_kv4_cache_fill(const void* k, const void* v, int P, void* kcache, void* vcache, void* sink_k, void* sink_v,
                       int B, int Hkv, int d, int window, int n_sink, swa_stream_t stream) {
  int st = check_kv4(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (P < 0) return SWA_ERR_INVALID_ARG;
  if (P == 0 || B == 0) return SWA_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return SWA_ERR_INVALID_ARG;
  if ((static_cast<long long>(std::min(P, window)) + std::min(P, n_sink)) * Hkv > INT32_MAX / 2)
    return SWA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  cudaError_t e = swa::launch_kv4_fill(k, v, P, kcache, vcache, sink_k, sink_v, B, Hkv, d, window, n_sink, dev->sms,
                                       reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_kv4_cache_append(const void* k_new, const void* v_new, const int32_t* pos, void* kcache, void* vcache,
                         void* sink_k, void* sink_v, int B, int Hkv, int d, int window, int n_sink,
                         swa_stream_t stream) {
  int st = check_kv4(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  if (static_cast<long long>(B) * Hkv > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  if (!k_new || !v_new || !pos || !aligned16(k_new) || !aligned16(v_new) || !aligned4(pos)) return SWA_ERR_INVALID_ARG;
  cudaError_t e = swa::launch_kv4_append(k_new, v_new, pos, kcache, vcache, sink_k, sink_v, B, Hkv, d, window, n_sink,
                                         reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_kv4_cache_read(const int32_t* positions, int n, const void* kcache, const void* vcache, const void* sink_k,
                       const void* sink_v, void* k_out, void* v_out, int out_dtype, int B, int Hkv, int d, int window,
                       int n_sink, swa_stream_t stream) {
  int st = check_kv4(B, Hkv, d, window, n_sink, kcache, vcache, sink_k, sink_v);
  if (st != SWA_OK) return st;
  if (n < 0 || (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_F32)) return SWA_ERR_INVALID_ARG;
  if (n == 0 || B == 0) return SWA_OK;
  if (static_cast<long long>(n) * Hkv > INT32_MAX / 2) return SWA_ERR_UNSUPPORTED;
  if (!positions || !aligned4(positions) || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return SWA_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  cudaError_t e = swa::launch_kv4_read(positions, n, kcache, vcache, sink_k, sink_v, k_out, v_out,
                                       out_dtype == SWA_DTYPE_F32, B, Hkv, d, window, n_sink, dev->sms,
                                       reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_kv4_decode(const void* q, const void* kcache, const void* vcache, const void* sink_k, const void* sink_v,
                   const int32_t* pos, void* out, float* lse, int B, int Hq, int Hkv, int d, int window, int n_sink,
                   float scale, int out_dtype, swa_stream_t stream) {
  int st = swa::decode_args_status(q, kcache, vcache, sink_k, sink_v, pos, out, lse, B, Hq, Hkv, d, window, n_sink,
                                   scale, out_dtype);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  if (static_cast<long long>(B) * Hkv > INT32_MAX / 8 || static_cast<long long>(window) + n_sink > INT32_MAX / 2)
    return SWA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  swa::Kv4DecodeArgs a{};
  a.q = q;
  a.kc = static_cast<const uint8_t*>(kcache);
  a.vc = static_cast<const uint8_t*>(vcache);
  a.sk = static_cast<const uint8_t*>(sink_k);
  a.sv = static_cast<const uint8_t*>(sink_v);
  a.pos = pos;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.W = window;
  a.S = n_sink;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out_f32 = out_dtype == SWA_DTYPE_BF16_F32OUT ? 1 : 0;
  cudaError_t e = swa::launch_kv4_decode(a, d, dev->sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_hh_scores(const void* q, const void* k, const float* lse, float* score, int B, int Hq, int Hkv, int L, int d,
                  int n_obs, int window, int n_sink, float scale, swa_stream_t stream) {
  int st = check_heads(Hq, Hkv, d, window, n_sink, scale, SWA_DTYPE_BF16);
  if (st != SWA_OK) return st;
  if (B < 0 || L < 0 || n_obs < 0 || n_obs > L) return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * L == 0) return SWA_OK;
  if (!q || !k || !lse || !score || !aligned16(q) || !aligned16(k) || !aligned4(lse) || !aligned4(score))
    return SWA_ERR_INVALID_ARG;
  const long long T = static_cast<long long>(B) * L;
  const long long units = static_cast<long long>(B) * Hkv * ((L + 127) / 128);
  // the kernel adds a window of up to L to a key's position, and a grid's blocks to a unit's number
  if (T > INT32_MAX - 128 || L >= (1 << 30) - 128 || units > INT32_MAX / 2 ||
      static_cast<long long>(n_obs) * (Hq / Hkv) > INT32_MAX / 2)
    return SWA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  CUtensorMap tq, tk;
  if ((st = make_map(&tq, q, false, d, Hq, T, 128)) != SWA_OK) return st;
  if ((st = make_map(&tk, k, false, d, Hkv, T, 128)) != SWA_OK) return st;
  swa::HhScoresArgs h{};
  swa::PrefillArgs& a = h.pa;
  a.n_seq = B;
  a.L = L;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.window = std::min(window, L);
  a.n_sink = n_sink;
  a.scale = scale;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.timeout_ns = g_timeout_ns.load();
  a.debug_flags = g_debug_flags.load();
  a.err = dev->err;
  h.lse = lse;
  h.score = score;
  h.n_obs = n_obs;
  h.n_units = static_cast<int>(units);
  cudaError_t e = swa::launch_hh_scores(h, tq, tk, d, static_cast<int>(std::min<long long>(dev->sms, units)),
                                        reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

static int check_hh(int B, int Hkv, int d, int capacity, int n_sink, int recent, const void* kc, const void* vc,
                    const int32_t* slot_pos, const float* score) {
  if (B < 0 || Hkv <= 0 || n_sink < 0 || recent < 1 || static_cast<long long>(n_sink) + recent > capacity)
    return SWA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || capacity > swa::kHhMaxCapacity || static_cast<long long>(B) * Hkv > INT32_MAX / 1024)
    return SWA_ERR_UNSUPPORTED;
  if (B == 0) return SWA_OK;
  if (!kc || !vc || !slot_pos || !score || !aligned16(kc) || !aligned16(vc) || !aligned4(slot_pos) || !aligned4(score))
    return SWA_ERR_INVALID_ARG;
  return SWA_OK;
}

int swa_hh_cache_fill(const void* k, const void* v, const float* score_in, int L, void* kcache, void* vcache,
                      int32_t* slot_pos, float* score, int B, int Hkv, int d, int capacity, int n_sink, int recent,
                      swa_stream_t stream) {
  int st = check_hh(B, Hkv, d, capacity, n_sink, recent, kcache, vcache, slot_pos, score);
  if (st != SWA_OK) return st;
  if (L < 0) return SWA_ERR_INVALID_ARG;
  if (B == 0) return SWA_OK;
  if (L > 0 && (!k || !v || !score_in || !aligned16(k) || !aligned16(v) || !aligned4(score_in)))
    return SWA_ERR_INVALID_ARG;
  if (L > INT32_MAX - 4096) return SWA_ERR_UNSUPPORTED;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  cudaError_t e = swa::launch_hh_fill(k, v, score_in, L, kcache, vcache, slot_pos, score, B, Hkv, d, capacity, n_sink,
                                      recent, dev->sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_hh_cache_append(const void* k_new, const void* v_new, const int32_t* pos, void* kcache, void* vcache,
                        int32_t* slot_pos, float* score, int32_t* slot, int B, int Hkv, int d, int capacity,
                        int n_sink, int recent, swa_stream_t stream) {
  int st = check_hh(B, Hkv, d, capacity, n_sink, recent, kcache, vcache, slot_pos, score);
  if (st != SWA_OK) return st;
  if (B == 0) return SWA_OK;
  if (!k_new || !v_new || !pos || !aligned16(k_new) || !aligned16(v_new) || !aligned4(pos) ||
      (slot && !aligned4(slot)))
    return SWA_ERR_INVALID_ARG;
  cudaError_t e = swa::launch_hh_append(k_new, v_new, pos, kcache, vcache, slot_pos, score, slot, B, Hkv, d, capacity,
                                        n_sink, recent, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_hh_decode(const void* q, const void* kcache, const void* vcache, const int32_t* slot_pos, float* score,
                  void* out, float* lse, int B, int Hq, int Hkv, int d, int capacity, float scale, float decay,
                  int out_dtype, swa_stream_t stream) {
  int st = check_hh(B, Hkv, d, capacity, 0, 1, kcache, vcache, slot_pos, score);
  if (st != SWA_OK) return st;
  if (Hq <= 0 || Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale) || !(decay >= 0.f && decay <= 1.f) ||
      (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_BF16_F32OUT))
    return SWA_ERR_INVALID_ARG;
  if (Hq / Hkv > 8) return SWA_ERR_UNSUPPORTED;
  if (B == 0) return SWA_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) || (lse && !aligned4(lse))) return SWA_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != SWA_OK) return st;
  swa::HhDecodeArgs a{};
  a.q = q;
  a.kc = kcache;
  a.vc = vcache;
  a.slot_pos = slot_pos;
  a.score = score;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.C = capacity;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.decay = decay;
  a.out_f32 = out_dtype == SWA_DTYPE_BF16_F32OUT ? 1 : 0;
  cudaError_t e = swa::launch_hh_decode(a, d, dev->sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_rope_axes_qk(void* q, void* k, const int32_t* positions, long long n_tokens, int Hq, int Hkv, int d,
                     long long q_stride, long long k_stride, const int32_t* sections, int n_axes, int layout,
                     double rope_base, int inverse, int dtype, swa_stream_t stream) {
  if (k == nullptr) Hkv = 0;
  if (n_tokens < 0 || Hq < 0 || Hkv < 0 || n_axes < 1 || !sections || !rope_base_ok(rope_base) ||
      (dtype != SWA_DTYPE_BF16 && dtype != SWA_DTYPE_F32) || layout < SWA_ROPE_SECTIONS ||
      layout > SWA_ROPE_INTERLEAVED)
    return SWA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || n_axes > swa::kRopeMaxAxes || Hq > 65536 || Hkv > 65536) return SWA_ERR_UNSUPPORTED;
  const int half = d / 2;
  int sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0 || sections[a] > half) return SWA_ERR_INVALID_ARG;
    sum += sections[a];
    if (layout == SWA_ROPE_INTERLEAVED && a > 0 && sections[a] > 0 && a + n_axes * (sections[a] - 1) >= half)
      return SWA_ERR_INVALID_ARG;
  }
  if (sum != half) return SWA_ERR_INVALID_ARG;
  const long long unit = dtype == SWA_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  if ((Hq > 0 && (q_stride < static_cast<long long>(Hq) * d || q_stride % unit != 0)) ||
      (Hkv > 0 && (k_stride < static_cast<long long>(Hkv) * d || k_stride % unit != 0)))
    return SWA_ERR_INVALID_ARG;
  if (n_tokens == 0 || Hq + Hkv == 0) return SWA_OK;
  if (!positions || !aligned4(positions) || (Hq > 0 && (!q || !aligned16(q))) || (Hkv > 0 && !aligned16(k)))
    return SWA_ERR_INVALID_ARG;
  if (n_tokens > INT64_MAX / 64 / std::max(q_stride, k_stride)) return SWA_ERR_UNSUPPORTED;
  swa::RopeAxesTable t;
  int axis = 0, m = 0;  // sections and per-axis layouts: the current axis and pair within it
  for (int i = 0; i < half; ++i) {
    if (layout == SWA_ROPE_INTERLEAVED) {
      const int a = i % n_axes;
      axis = a > 0 && i / n_axes < sections[a] ? a : 0;
    } else {
      while (m == sections[axis]) {
        ++axis;
        m = 0;
      }
    }
    t.axis[i] = static_cast<unsigned char>(axis);
    t.theta[i] = layout == SWA_ROPE_PER_AXIS ? std::pow(rope_base, -static_cast<double>(m) / sections[axis])
                                             : std::pow(rope_base, -2.0 * i / d);
    ++m;
  }
  for (int i = half; i < 64; ++i) {
    t.axis[i] = 0;
    t.theta[i] = 0.0;
  }
  DeviceInfo* dev = nullptr;
  const int st = device_info(&dev);
  if (st != SWA_OK) return st;
  swa::RopeAxesArgs a{};
  a.q = q;
  a.k = k;
  a.positions = positions;
  a.T = n_tokens;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.sign = inverse ? -1.f : 1.f;
  cudaError_t e = swa::launch_rope_axes(a, t, dtype == SWA_DTYPE_F32, dev->sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

int swa_hadamard_proj(const void* y, const float* alpha, const float* beta, void* z,
                      long long n_rows, int n, int out_dtype, swa_stream_t stream) {
  if (n_rows < 0 || n < 32 || n > 8192 || (n & (n - 1)) != 0) return n_rows < 0 ? SWA_ERR_INVALID_ARG
                                                                      : SWA_ERR_UNSUPPORTED;
  if (out_dtype != SWA_DTYPE_BF16 && out_dtype != SWA_DTYPE_F32) return SWA_ERR_INVALID_ARG;
  if (n_rows == 0) return SWA_OK;
  if (!y || !alpha || !beta || !z || !aligned16(y) || !aligned16(alpha) || !aligned16(beta) ||
      !aligned16(z))
    return SWA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  const int st = device_info(&di);
  if (st != SWA_OK) return st;
  swa::HadamardArgs a;
  a.y = y;
  a.alpha = alpha;
  a.beta = beta;
  a.z = z;
  a.n_rows = n_rows;
  a.timeout_ns = g_timeout_ns.load();
  a.debug_flags = g_debug_flags.load();
  a.err = di->err;
  cudaError_t e = swa::launch_hadamard(a, n, out_dtype == SWA_DTYPE_F32, di->sms,
                                       reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SWA_OK : SWA_ERR_CUDA;
}

const char* swa_status_string(int status) {
  switch (status) {
    case SWA_OK: return "ok";
    case SWA_ERR_INVALID_ARG: return "invalid argument";
    case SWA_ERR_UNSUPPORTED: return "unsupported configuration";
    case SWA_ERR_CUDA: return "CUDA error";
    case SWA_ERR_DEVICE_TIMEOUT: return "device wait timed out";
    case SWA_ERR_WORKSPACE: return "workspace missing or too small";
    default: return "unknown status";
  }
}

int swa_device_error(swa_stream_t stream) {
  DeviceInfo* dev = nullptr;
  int st = device_info(&dev);
  if (st != SWA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return SWA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, dev->err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SWA_ERR_CUDA;
  const int zero = 0;
  if (v != 0 && cudaMemcpy(dev->err, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return SWA_ERR_CUDA;
  return v;
}

int swa_debug_error_word(swa_stream_t stream) { return swa_device_error(stream); }

unsigned long long swa_set_wait_timeout_ns(unsigned long long ns) { return g_timeout_ns.exchange(ns); }

int swa_set_debug_flags(int flags) { return g_debug_flags.exchange(flags); }

int swa_version(void) { return 0x000100; }

}  // extern "C"

// Launch interfaces of the fixed-memory caches: the 4-bit ring cache, the cache
// that evicts by accumulated attention weight, and rotary positions with axes.
#pragma once
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

namespace swa {

// Division of 0 <= n < 2^31 by a divisor known to the host, in three instructions, as Granlund
// and Montgomery describe it ("Division by invariant integers using multiplication"): with 2^l
// the power of two at or above d, q = (n + n * mul / 2^32) / 2^l, mul = 2^32 (2^l - d) / d + 1.
struct FastDiv {
  uint32_t d, mul, shift;
  explicit FastDiv(int divisor) : d(static_cast<uint32_t>(divisor)), shift(0) {
    while (shift < 31 && (1u << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
  __device__ __forceinline__ uint32_t mod(uint32_t n) const { return n - div(n) * d; }
#endif
};

#ifdef __CUDACC__
// A kernel that is launched to start early (cudaLaunchAttributeProgrammaticStreamSerialization)
// waits here for the end and the writes of the kernel before it: its launch and its blocks' start
// are out of the way by then.  The kernels that such a one follows let it go at once.
// What the kernel before may write is no `const __restrict__` parameter of the early one: that
// would promise memory that nobody writes while it runs, and allow loads that are not coherent.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;"); }
#endif

// Launch of a kernel that starts early and waits, as above.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Let a kernel use up to `bytes` of dynamic shared memory: asked of the runtime once per
// device, since the question costs as much as a tenth of a launch.
template <auto Kernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------- 4-bit ring cache
constexpr int kKv4Group = 32;  // elements that share a step and a minimum
__host__ __device__ constexpr int kv4_row_bytes(int d) { return d / 2 + d / kKv4Group * 4; }

cudaError_t launch_kv4_fill(const void* k, const void* v, int P, void* kc, void* vc, void* sk, void* sv, int B,
                            int Hkv, int d, int W, int S, int sms, cudaStream_t stream);
cudaError_t launch_kv4_append(const void* k, const void* v, const int32_t* pos, void* kc, void* vc, void* sk,
                              void* sv, int B, int Hkv, int d, int W, int S, cudaStream_t stream);
cudaError_t launch_kv4_read(const int32_t* positions, int n, const void* kc, const void* vc, const void* sk,
                            const void* sv, void* k_out, void* v_out, bool f32, int B, int Hkv, int d, int W, int S,
                            int sms, cudaStream_t stream);

struct Kv4DecodeArgs {
  const void* q;        // [B, Hq, d] bf16
  const uint8_t* kc;    // [B, Hkv, W, row]
  const uint8_t* vc;
  const uint8_t* sk;    // [B, Hkv, S, row]
  const uint8_t* sv;
  const int32_t* pos;   // [B]
  void* out;            // [B, Hq, d] bf16 or float32
  float* lse;           // [B, Hq] or null
  int B, Hq, Hkv, G, W, S;
  float scale_log2;
  int out_f32;
};
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, int d, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- eviction by weight
struct HhDecodeArgs {
  const void* q;            // [B, Hq, d] bf16
  const void* kc;           // [B, Hkv, C, d] bf16
  const void* vc;
  const int32_t* slot_pos;  // [B, Hkv, C], < 0: empty
  float* score;             // [B, Hkv, C], updated
  void* out;                // [B, Hq, d] bf16 or float32
  float* lse;               // [B, Hq] or null
  int B, Hq, Hkv, G, C;
  float scale_log2, decay;
  int out_f32;
};
constexpr int kHhMaxCapacity = 16384;  // slots whose scores a cluster's shared memory holds (64 KB a block of 8)
cudaError_t launch_hh_decode(const HhDecodeArgs& a, int d, int sms, cudaStream_t stream);
cudaError_t launch_hh_append(const void* k, const void* v, const int32_t* pos, void* kc, void* vc,
                             int32_t* slot_pos, float* score, int32_t* slot, int B, int Hkv, int d, int C, int S,
                             int recent, cudaStream_t stream);
cudaError_t launch_hh_fill(const void* k, const void* v, const float* score_in, int L, void* kc, void* vc,
                           int32_t* slot_pos, float* score, int B, int Hkv, int d, int C, int S, int recent, int sms,
                           cudaStream_t stream);

// ---------------------------------------------------------------- rotary positions with axes
constexpr int kRopeMaxAxes = 4;
struct RopeAxesTable {
  double theta[64];       // per pair
  unsigned char axis[64];
};
struct RopeAxesArgs {
  void* q;
  void* k;                  // may be null
  const int32_t* positions; // [n_axes, T]
  long long T, q_stride, k_stride;  // strides in elements between tokens
  int Hq, Hkv, d;
  float sign;               // +1 forward, -1 inverse
};
cudaError_t launch_rope_axes(const RopeAxesArgs& a, const RopeAxesTable& t, bool f32, int sms, cudaStream_t stream);

}  // namespace swa

// mixer_common.cuh -- what the operators around the chunk core share: host
// checks, the packed-batch offsets, and small device helpers.
#pragma once

#include <atomic>

#include "../carve_internal.cuh"
#include "../sm100_ptx.cuh"

namespace carve {
namespace mix {

// ------------------------------------------------------------------- host
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
inline bool opt_ptr_ok(const void* p) { return p == nullptr || aligned16(p); }
inline bool flag_ok(int v) { return v == 0 || v == 1; }
inline bool dtype_ok(int d) { return d == CARVE_BF16 || d == CARVE_FP32; }

// The status word of a workspace, NULL where there is no room for one (calls
// that need a workspace have refused that before).
inline uint32_t* status_word(void* ws, size_t bytes) {
  return ptr_ok(ws) && bytes >= kHeaderBytes ? static_cast<uint32_t*>(ws) : nullptr;
}

// Token indices (and a tile past the last) stay inside 32 bits; element
// offsets are formed in 64.
constexpr int64_t kMaxTokens = (1LL << 31) - (1 << 16);

// A token pitch: 0 means the width itself.  Offsets within a tile of rows are
// 32 bits wide, which bounds the pitch.
constexpr int64_t kMaxPitch = 1 << 22;
inline bool pitch_ok(int64_t p, int64_t width) {
  return p == 0 || (p >= width && p % 8 == 0);
}

// What is asked of a device once is kept by its number, up to this many.
constexpr int kDevices = 64;
// The number of the current device, -1 if it has none that answers are kept by.
inline int kept_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kDevices ? dev : -1;
}

// The current device's SMs.  They decide how calls are cut up, and so in which
// order partial results are added.
inline int sm_count() {
  static std::atomic<int> kept[kDevices];
  const int at = kept_device();
  int n = at >= 0 ? kept[at].load() : 0, dev = 0;
  if (n > 0) return n;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 148;
  if (at >= 0) kept[at].store(n);
  return n;
}

// Lets the kernel use its shared memory: asked for once a device.
template <auto kernel>
cudaError_t allow_smem(size_t smem) {
  if (smem <= 48 * 1024) return cudaSuccess;
  static std::atomic<uint64_t> asked{0};
  static_assert(kDevices <= 64, "a bit each");
  const int at = kept_device();
  if (at >= 0 && asked.load() >> at & 1) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && at >= 0) asked.fetch_or(1ull << at);
  return e;
}

inline void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* at, dim3 grid,
                           int threads, size_t smem, int ncl) {
  cfg->gridDim = grid;
  cfg->blockDim = dim3(threads);
  cfg->dynamicSmemBytes = smem;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ncl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg->attrs = at;
  cfg->numAttrs = ncl > 1 ? 1 : 0;
}

// Launch of one kernel, in clusters of `ncl` blocks.  Its blocks may take
// their places before the kernel in front of it has ended to the last: each
// begins with after_the_last().
template <auto kernel, typename... Args>
cudaError_t launch_all(dim3 grid, int threads, size_t smem, cudaStream_t st, int ncl,
                       const Args&... args) {
  const cudaError_t e = allow_smem<kernel>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  cluster_config(&cfg, at, grid, threads, smem, ncl);
  at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <auto kernel, typename Args>
cudaError_t launch(const Args& args, dim3 grid, int threads, size_t smem, cudaStream_t st,
                   int ncl = 1) {
  return launch_all<kernel>(grid, threads, smem, st, ncl, args);
}

// ----------------------------------------------------------------- device
// First in every kernel, by every thread: waits until the kernel in front has
// ended and its writes are visible.  Short launches otherwise leave about 1 us
// between them: forward and backward of 3 x 1021 x 1040 fp32 take 25.2 us
// instead of 28.7, the rotation's backward with its sum of dw 9.5 instead of
// 13.0 (1554 tokens).  Blocks take their places as those in front leave; to
// call the next kernel's in at once (launch_dependents) gained nothing more
// and cost large ones 1 % (1 x 65536 x 2048 171.6 us against 169.8).
__device__ __forceinline__ void after_the_last() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// 16 bytes global -> shared, the bytes from `valid` on filled with zeros.
__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src,
                                                 bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(n)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 operations in one instruction (a register pair each): the loops
// here are bound by instruction issue next to the memory traffic.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

// 2 V neighbouring elements as register pairs; four of them also as they lie
// in memory.
template <int V>
struct Vec {
  float2 p[V];
};
using Q = Vec<2>;
template <typename IO>
struct Raw;
template <>
struct Raw<float> {
  using T = float4;
  static __device__ __forceinline__ Q open(const T& v) {
    return Q{{make_float2(v.x, v.y), make_float2(v.z, v.w)}};
  }
  static __device__ __forceinline__ T pack(const Q& q) {
    return make_float4(q.p[0].x, q.p[0].y, q.p[1].x, q.p[1].y);
  }
};
template <>
struct Raw<__nv_bfloat16> {
  using T = uint2;
  static __device__ __forceinline__ float2 wide(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t narrow(float2 f) {
    const __nv_bfloat162 t = __float22bfloat162_rn(f);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
  static __device__ __forceinline__ Q open(const T& v) {
    return Q{{wide(v.x), wide(v.y)}};
  }
  static __device__ __forceinline__ T pack(const Q& q) {
    return make_uint2(narrow(q.p[0]), narrow(q.p[1]));
  }
};
__device__ __forceinline__ Q none() {
  return Q{{make_float2(0.f, 0.f), make_float2(0.f, 0.f)}};
}
template <typename IO>
__device__ __forceinline__ typename Raw<IO>::T ldr(const void* p, int64_t at) {
  return *reinterpret_cast<const typename Raw<IO>::T*>(static_cast<const IO*>(p) + at);
}
template <typename IO>
__device__ __forceinline__ Q ldq(const void* p, int64_t at) {
  return Raw<IO>::open(ldr<IO>(p, at));
}
template <typename IO>
__device__ __forceinline__ void stq(void* p, int64_t at, const Q& q) {
  *reinterpret_cast<typename Raw<IO>::T*>(static_cast<IO*>(p) + at) = Raw<IO>::pack(q);
}
__device__ __forceinline__ Q fma4(const Q& a, const Q& b, const Q& c) {
  return Q{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1])}};
}
__device__ __forceinline__ Q mul4(const Q& a, const Q& b) {
  return Q{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1])}};
}
__device__ __forceinline__ Q add4(const Q& a, const Q& b) {
  return Q{{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1])}};
}
// The hardware's 2^x and 1 / x (relative errors below 2^-22 and 2^-23;
// results below 2^-126 become 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// exp of a pair, x <= 88, for operands of type IO.  The rounding of x log2 e
// makes the hardware's 2^x off by up to |x| 2^-24: for bf16, whose half step is
// 2^-9, that is near enough, but fp32's half step is 2^-24 itself.  fp32
// therefore multiplies by 1 + r, r = x - l ln 2 being what the rounded l =
// x log2 e has left out; ln 2 is taken in two parts, so that r is good to its
// last bits (Cody and Waite's reduction).  That is within 2^-22 + 2^-23, and
// takes 4 x 4096 x 2048 fp32 with the activation from 79 and 120 us, forward and
// backward, to 84 and 129 (with calls of expf: 91 and 133).
__device__ __forceinline__ float at_least(float x, float low) {  // keeps NaN
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(low));
  return y;
}
template <typename IO>
__device__ __forceinline__ float2 exp_of(float2 x) {
  if (sizeof(IO) == 4) x = make_float2(at_least(x.x, -200.f), at_least(x.y, -200.f));  // 0 from there
  const float2 l = mul2(x, both(kLog2e));
  const float2 e = make_float2(ex2(l.x), ex2(l.y));
  if (sizeof(IO) < 4) return e;
  float2 r = fma2(l, both(-0.693147182464599609375f), x);
  r = fma2(l, both(1.9046543e-9f), r);
  return fma2(e, r, e);
}
// 1 / (1 + exp(-z)): relative error below 5 * 2^-23 in fp32 (z >= -87), below
// 2^-21 + |z| 2^-23 for bf16; 0 where exp(-z) overflows.
template <typename IO>
__device__ __forceinline__ float2 sigmoid_of(float2 z) {
  if (sizeof(IO) == 4) z = make_float2(at_least(z.x, -88.f), at_least(z.y, -88.f));
  const float2 e = add2(exp_of<IO>(mul2(z, both(-1.f))), both(1.f));
  return make_float2(rcp(e.x), rcp(e.y));
}

// Two neighbouring elements in the I/O dtype <-> two floats.
__device__ __forceinline__ float2 ld2(const float* p) {
  return *reinterpret_cast<const float2*>(p);
}
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void st2(float* p, float2 v) {
  *reinterpret_cast<float2*>(p) = v;
}
__device__ __forceinline__ void st2(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(v);
}

// Do the offsets of a packed batch rise within [0, T]?  Called by a whole
// block; every block of a grid reaches the same verdict, so all of them
// leave a bad call without touching an output.
__device__ __forceinline__ bool offsets_ok(const int32_t* cu, int B, int T) {
  bool ok = true;
  for (int n = threadIdx.x; n < B; n += blockDim.x)
    ok &= cu[n] >= 0 && cu[n] <= cu[n + 1] && cu[n + 1] <= T;
  return __syncthreads_and(ok);
}

// The same, and a copy of the B + 1 offsets in shared memory (kept[0 .. B]).
__device__ __forceinline__ bool offsets_kept(const int32_t* cu, int B, int T,
                                             int32_t* kept) {
  for (int n = threadIdx.x; n <= B; n += blockDim.x) kept[n] = cu[n];
  return offsets_ok(cu, B, T);  // its barrier publishes the copy
}

// Sequence starts of a batch: the packed offsets, or multiples of T.
struct Bounds {
  const int32_t* cu;
  int T;  // tokens per sequence (cu == NULL)
  int n;  // sequences
  __device__ __forceinline__ int at(int i) const { return cu ? cu[i] : i * T; }
  // First i in [0, n + 1] with at(i) >= t (n + 1: none), by 32 probes at a
  // time: every lane of the warp calls it with the same t.
  __device__ __forceinline__ int first_at_least(int t) const {
    if (!cu) return min((int)(((unsigned)t + (unsigned)T - 1u) / (unsigned)T), n + 1);
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n + 1;
    while (hi - lo > 32) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      const int k = __popc(__ballot_sync(~0u, i < hi && cu[i] < t));
      hi = min(hi, lo + k * step);
      lo = k ? lo + (k - 1) * step + 1 : lo;
      if (!k) hi = lo;
    }
    return lo + __popc(__ballot_sync(~0u, lo + lane < hi && cu[lo + lane] < t));
  }
  // The sequence that token t belongs to (t inside [at(0), at(n))).
  __device__ __forceinline__ int seq_of(int t) const {
    return first_at_least(t + 1) - 1;
  }
};

// The sequence starts and ends among the tokens t0 .. t0 + S - 1 (S <= 32),
// as bit masks, and the tokens that belong to any sequence.
struct Marks {
  unsigned start, end;
  int lo, hi;
};
template <int S>
__device__ __forceinline__ Marks marks_of(const Bounds& b, int t0) {
  Marks m;
  m.lo = b.at(0);
  m.hi = b.at(b.n);
  m.start = m.end = 0;
  const int lane = threadIdx.x & 31;
  for (int i = b.first_at_least(t0); i <= b.n; i += 32) {
    const int v = i + lane <= b.n ? b.at(i + lane) : m.hi + S + 1;
    const int d = v - t0;  // >= 0
    if (v < m.hi && d < S) m.start |= 1u << d;
    if (v > m.lo && v <= m.hi && d >= 1 && d <= S) m.end |= 1u << (d - 1);
    if (__any_sync(~0u, v > t0 + S)) break;
  }
  m.start = __reduce_or_sync(~0u, m.start);
  m.end = __reduce_or_sync(~0u, m.end);
  return m;
}

}  // namespace mix
}  // namespace carve

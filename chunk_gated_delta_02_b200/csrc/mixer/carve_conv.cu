// carve_conv.cu -- short causal convolution over each channel with an
// optional SiLU, forward, backward and one-token form (declared in
// include/carve.h).
//
// A warp takes 128 channels (4 a lane; 64 in small calls) and walks a run of
// consecutive token rows with the last W - 1 inputs in registers, so every
// input is read once;
// runs are long enough that the W - 1 rows before (and in the backward
// behind) them cost little.  Each warp brings its rows in through a ring of
// its own in shared memory, filled by asynchronous copies several chunks
// ahead: what is on its way then does not depend on the registers, which the
// taps, the window and the sums need.  Dense batches are walked as packed
// ones whose sequences start at multiples of T.
//
// What bounds it: 8 x 4096 x 6144 bf16 with W = 4 and SiLU takes 133 us
// forward (6.06 TB/s of x and y, of 6.47 measured for a copy) and 237 us
// backward (5.1 TB/s of x, dy and dx: two streams in and one out, at 54 % of the
// issue slots; twice the warps with half the registers were no faster).
// Without the rings (loads into registers a row ahead) they took 177 and 332.
// Packed sequences are walked one after another by a warp, each with its search
// and its ring's start: 32768 x 6144 in 500 sequences takes 167 and 330 us, in
// 4000 of them 317 and 709, where the bytes take 125 and 187.
#include "mixer_common.cuh"

namespace carve {
namespace mix {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
template <int V>
constexpr int kCh = 64 * V;  // channels of a block: V pairs a lane
// Blocks an SM holds: the forward gets by on 64 registers with 4 channels a
// lane, the backward with its sums of dw does not.
template <int V>
constexpr int kFwdPerSm = V == 2 ? 4 : 6;
template <int V>
constexpr int kBwdPerSm = V == 2 ? 2 : 3;

struct ConvArgs {
  int B, T, C, silu, fill;
  int rows;  // token rows in all
  int run;   // rows of a warp
  int64_t xp;
  const void *x, *w, *bias, *state, *dy, *dstate_T;
  void *y, *state_T, *dx, *dstate;
  const int32_t* cu;
  uint32_t* status;
  float* part;  // [run block][C][W + 1] partial dw | dbias
};

template <int V>
__device__ __forceinline__ Vec<V> zeros() {
  Vec<V> r;
#pragma unroll
  for (int h = 0; h < V; ++h) r.p[h] = both(0.f);
  return r;
}
template <typename IO, int V>
__device__ __forceinline__ Vec<V> ldc(const void* p, int64_t at) {
  if constexpr (V == 2) return ldq<IO>(p, at);
  else return Vec<V>{{ld2(static_cast<const IO*>(p) + at)}};
}
template <typename IO, int V>
__device__ __forceinline__ void stc(void* p, int64_t at, const Vec<V>& v) {
  if constexpr (V == 2) stq<IO>(p, at, v);
  else st2(static_cast<IO*>(p) + at, v.p[0]);
}
template <int V>
__device__ __forceinline__ Vec<V> fmac(const Vec<V>& a, const Vec<V>& b, const Vec<V>& c) {
  Vec<V> r;
#pragma unroll
  for (int h = 0; h < V; ++h) r.p[h] = fma2(a.p[h], b.p[h], c.p[h]);
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> mulc(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> r;
#pragma unroll
  for (int h = 0; h < V; ++h) r.p[h] = mul2(a.p[h], b.p[h]);
  return r;
}
template <int V>
__device__ __forceinline__ Vec<V> addc(const Vec<V>& a, const Vec<V>& b) {
  Vec<V> r;
#pragma unroll
  for (int h = 0; h < V; ++h) r.p[h] = add2(a.p[h], b.p[h]);
  return r;
}
template <typename IO, int V>
__device__ __forceinline__ Vec<V> sigmoids(const Vec<V>& z) {
  Vec<V> r;
#pragma unroll
  for (int h = 0; h < V; ++h) r.p[h] = sigmoid_of<IO>(z.p[h]);
  return r;
}

template <typename IO, int W, int V>
struct Taps {
  Vec<V> w[W], bias;
  __device__ __forceinline__ Taps(const ConvArgs& a, int c) {
    bias = a.bias ? ldc<IO, V>(a.bias, c) : zeros<V>();
    float f[2 * V * W];  // the lane's channels' taps lie in a row
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const Vec<V> q = ldc<IO, V>(a.w, (int64_t)c * W + 2 * V * k);
#pragma unroll
      for (int h = 0; h < V; ++h)
        f[2 * (V * k + h)] = q.p[h].x, f[2 * (V * k + h) + 1] = q.p[h].y;
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int h = 0; h < V; ++h)
        w[j].p[h] = make_float2(f[2 * h * W + j], f[(2 * h + 1) * W + j]);
  }
  // z of the token whose inputs are win[0 .. W - 2] and x
  __device__ __forceinline__ Vec<V> z(const Vec<V> (&win)[W - 1], const Vec<V>& x) const {
    Vec<V> s = bias;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) s = fmac(w[j], win[j], s);
    return fmac(w[W - 1], x, s);
  }
};

// The inputs before row t of the sequence n that starts at row s: from the
// rows themselves as far back as s, then from its state.
template <typename IO, int W, int V>
__device__ __forceinline__ void window_before(const ConvArgs& a, int64_t n, int s,
                                              int t, int c, Vec<V> (&win)[W - 1]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int r = t - (W - 1) + j;
    win[j] = zeros<V>();
    if (r >= s)
      win[j] = ldc<IO, V>(a.x, (int64_t)r * a.xp + c);
    else if (a.state)
      win[j] = ldc<IO, V>(a.state, (n * (W - 1) + (r - s + W - 1)) * a.C + c);
  }
}

template <int W, int V>
__device__ __forceinline__ void push(Vec<V> (&win)[W - 1], const Vec<V>& x) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
  win[W - 2] = x;
}

// dst[n] = src[n] (or zero) for the empty sequences, this block's channels.
template <typename IO, int V>
__device__ __forceinline__ void copy_empty(const ConvArgs& a, int rows, int c,
                                           bool on, const void* src, void* dst) {
  if (!dst || !on) return;
  for (int n = blockIdx.y * kWarps + (threadIdx.x >> 5); n < a.B;
       n += gridDim.y * kWarps) {
    if (a.cu[n] != a.cu[n + 1]) continue;
    for (int j = 0; j < rows; ++j) {
      const int64_t at = ((int64_t)n * rows + j) * a.C + c;
      stc<IO, V>(dst, at, src ? ldc<IO, V>(src, at) : zeros<V>());
    }
  }
}

// Chunks of kN rows x kCh<V> channels of one tensor -> shared memory, by one
// warp; rows from `end` on repeat the last one before it, channels from C on
// the first ones.
template <typename IO, int kN, int V>
struct Fetch {
  static constexpr int E = 16 / sizeof(IO), PER = kCh<V> / E, STEP = 32 / PER;
  const IO* src;
  int64_t pitch;
  int row, at;
  __device__ __forceinline__ Fetch(const void* p, int64_t pitch_, int c0, int C)
      : pitch(pitch_) {
    const int lane = threadIdx.x & 31, c = lane % PER * E;
    row = lane / PER;
    at = row * kCh<V> + c;
    src = static_cast<const IO*>(p) + (c0 + c < C ? c0 + c : 0);
  }
  __device__ __forceinline__ void operator()(IO* dst, int t, int end) const {
    if (t + kN <= end) {
      const IO* s = src + (int64_t)(t + row) * pitch;
#pragma unroll
      for (int i = 0; i < kN / STEP; ++i, s += STEP * pitch)
        ptx::cp_async16(dst + at + i * STEP * kCh<V>, s);
    } else {
#pragma unroll
      for (int i = 0; i < kN / STEP; ++i)
        ptx::cp_async16(dst + at + i * STEP * kCh<V>,
                        src + (int64_t)min(t + row + i * STEP, end - 1) * pitch);
    }
  }
};

__device__ __forceinline__ bool packed_ok(const ConvArgs& a) {
  const bool ok = offsets_ok(a.cu, a.B, a.T);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    *a.status = ok ? CARVE_OK : CARVE_ERR_INVALID_ARG;
  return ok;
}

__device__ __forceinline__ void dense_ok(const ConvArgs& a) {
  if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = CARVE_OK;
}

// Rows [t, end) of a warp that belong to no sequence.
template <typename IO, int V>
__device__ __forceinline__ void fill_rows(const ConvArgs& a, void* out, int t,
                                          int end, int c, bool on) {
  if (a.fill && on)
    for (; t < end; ++t) stc<IO, V>(out, (int64_t)t * a.C + c, zeros<V>());
}

// ---------------------------------------------------------------- forward
template <typename IO, int V>
struct FwdRing {
  static constexpr int kN = sizeof(IO) == 2 ? 8 : 4;  // rows of a chunk
  static constexpr int STAGES = 3;  // 48 KB a block, four blocks an SM
  IO x[kWarps][STAGES][kN * kCh<V>];
};

template <typename IO, int W, int V>
__global__ void __launch_bounds__(kThreads, kFwdPerSm<V>) conv_fwd_kernel(ConvArgs a) {
  after_the_last();
  using R = Raw<IO>;
  using Ring = FwdRing<IO, V>;
  constexpr int kN = Ring::kN, STAGES = Ring::STAGES;
  extern __shared__ __align__(16) unsigned char raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  IO* const ring = reinterpret_cast<Ring*>(raw)->x[warp][0];
  const int col = blockIdx.x * kCh<V> + 2 * V * lane;
  const bool on = col < a.C;
  const int c = on ? col : a.C - 2 * V;  // idle lanes read what others read
  if (a.cu) {
    if (!packed_ok(a)) return;
    copy_empty<IO, V>(a, W - 1, c, on, a.state, a.state_T);
  } else {
    dense_ok(a);
  }
  const Bounds b{a.cu, a.T, a.B};
  const int64_t first = ((int64_t)blockIdx.y * kWarps + warp) * a.run;
  if (first >= a.rows) return;
  const int lo = (int)first, hi = (int)min(first + a.run, (int64_t)a.rows);
  const int begin = min(max(b.at(0), lo), hi), stop = max(min(b.at(b.n), hi), begin);
  fill_rows<IO, V>(a, a.y, lo, begin, c, on);
  fill_rows<IO, V>(a, a.y, stop, hi, c, on);
  if (begin == stop) return;
  const Fetch<IO, kN, V> fetch(a.x, a.xp, blockIdx.x * kCh<V>, a.C);
  const Taps<IO, W, V> taps(a, c);
  // one sequence after the other
  for (int t = begin; t < stop;) {
    const int n = b.seq_of(t), s = b.at(n), e = b.at(n + 1), end = min(e, stop);
    int in = 0, out = 0;  // places in the ring
    auto bring = [&](int row) {
      if (row < end) fetch(ring + in * kN * kCh<V>, row, end);
      ptx::cp_async_commit();
      in = in + 1 < STAGES ? in + 1 : 0;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) bring(t + i * kN);
    Vec<V> win[W - 1];
    window_before<IO, W, V>(a, n, s, t, c, win);
    int64_t at = (int64_t)t * a.C + c;
    for (; t < end; t += kN) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      bring(t + (STAGES - 1) * kN);
      const IO* rows = ring + out * kN * kCh<V> + 2 * V * lane;
      out = out + 1 < STAGES ? out + 1 : 0;
      auto token = [&](int i) {
        const Vec<V> x = ldc<IO, V>(rows, i * kCh<V>);
        Vec<V> z = taps.z(win, x);
        if (a.silu) z = mulc(z, sigmoids<IO>(z));
        push<W, V>(win, x);
        if (on) stc<IO, V>(a.y, at, z);
        at += a.C;
      };
      if (t + kN <= end) {
#pragma unroll
        for (int i = 0; i < kN; ++i) token(i);
      } else {
#pragma unroll 1
        for (int i = 0; t + i < end; ++i) token(i);
      }
    }
    t = end;
    cp_async_wait<0>();
    __syncwarp();
    if (end == e && a.state_T) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        if (on) stc<IO, V>(a.state_T, ((int64_t)n * (W - 1) + j) * a.C + c, win[j]);
    }
  }
}

// --------------------------------------------------------------- backward
// dz_t = dy_t act'(z_t) with z formed again from x; input t - k gets
// w[W - 1 - k] dz_t, so the gradient of input r is complete W - 1 rows later.
// A warp walks its rows of one sequence and the W - 1 rows behind them
// (beyond the sequence's end dz is zero and dstate_T is added instead) and
// stores the gradients of its own rows, and of the state where the sequence
// starts among them.  `acc` holds the gradients not complete yet.  Forming z
// again costs W FMAs an element; to read it back would cost a fourth tensor,
// a third of the traffic.
template <typename IO, int V>
struct BwdRing {
  static constexpr int kN = sizeof(IO) == 2 ? 8 : 4;
  static constexpr int STAGES = 3;
  IO x[kWarps][STAGES][kN * kCh<V>], d[kWarps][STAGES][kN * kCh<V>];
};

template <typename IO, int W, int V>
__global__ void __launch_bounds__(kThreads, kBwdPerSm<V>) conv_bwd_kernel(ConvArgs a) {
  after_the_last();
  using R = Raw<IO>;
  using Ring = BwdRing<IO, V>;
  constexpr int kN = Ring::kN, STAGES = Ring::STAGES;
  extern __shared__ __align__(16) unsigned char raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  IO* const xring = reinterpret_cast<Ring*>(raw)->x[warp][0];
  IO* const dring = reinterpret_cast<Ring*>(raw)->d[warp][0];
  const int col = blockIdx.x * kCh<V> + 2 * V * lane;
  const bool on = col < a.C;
  const int c = on ? col : a.C - 2 * V;
  if (a.cu) {
    if (!packed_ok(a)) return;
    copy_empty<IO, V>(a, W - 1, c, on, a.dstate_T, a.dstate);
  } else {
    dense_ok(a);
  }
  const Bounds b{a.cu, a.T, a.B};
  const int64_t first = ((int64_t)blockIdx.y * kWarps + warp) * a.run;
  const int lo = (int)min(first, (int64_t)a.rows);
  const int hi = (int)min(first + a.run, (int64_t)a.rows);
  const int begin = min(max(b.at(0), lo), hi), stop = max(min(b.at(b.n), hi), begin);
  fill_rows<IO, V>(a, a.dx, lo, begin, c, on);
  fill_rows<IO, V>(a, a.dx, stop, hi, c, on);
  const Fetch<IO, kN, V> fetch_x(a.x, a.xp, blockIdx.x * kCh<V>, a.C);
  const Fetch<IO, kN, V> fetch_d(a.dy, a.C, blockIdx.x * kCh<V>, a.C);
  const Taps<IO, W, V> taps(a, c);
  Vec<V> dw[W], db = zeros<V>();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = zeros<V>();

  for (int at = begin; at < stop;) {
    const int n = b.seq_of(at), s = b.at(n), e = b.at(n + 1), end = min(e, stop);
    const int past = end + W - 1;  // rows walked: dz of [at, past) of [s, e)
    int in = 0, out = 0;
    auto bring = [&](int row) {
      if (row < past) {
        fetch_x(xring + in * kN * kCh<V>, row, e);
        fetch_d(dring + in * kN * kCh<V>, row, e);
      }
      ptx::cp_async_commit();
      in = in + 1 < STAGES ? in + 1 : 0;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) bring(at + i * kN);
    Vec<V> win[W - 1], acc[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) acc[j] = zeros<V>();
    window_before<IO, W, V>(a, n, s, at, c, win);
    int64_t put = (int64_t)(at - (W - 1)) * a.C + c;  // of the row completed next
    for (int t0 = at; t0 < past; t0 += kN) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      bring(t0 + (STAGES - 1) * kN);
      const IO* xs = xring + out * kN * kCh<V> + 2 * V * lane;
      const IO* ds = dring + out * kN * kCh<V> + 2 * V * lane;
      out = out + 1 < STAGES ? out + 1 : 0;
      // own: the row is this warp's, and its gradient adds to dw and dbias;
      // returns the gradient that row t completes, of row t - (W - 1)
      auto token = [&](int i, bool inside, bool own) {
        const Vec<V> x = ldc<IO, V>(xs, i * kCh<V>);
        Vec<V> dz = ldc<IO, V>(ds, i * kCh<V>);
        if (a.silu) {
          const Vec<V> z = taps.z(win, x), g = sigmoids<IO>(z);
#pragma unroll
          for (int h = 0; h < V; ++h)  // g (1 + z (1 - g))
            dz.p[h] = mul2(dz.p[h], mul2(g.p[h], fma2(z.p[h], fma2(both(-1.f), g.p[h], both(1.f)),
                                                       both(1.f))));
        }
        if (!inside) dz = zeros<V>();
        if (own) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j] = fmac(dz, win[j], dw[j]);
          dw[W - 1] = fmac(dz, x, dw[W - 1]);
          db = addc(db, dz);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) acc[j] = fmac(taps.w[j], dz, acc[j]);
        const Vec<V> done = acc[0];
        push<W, V>(acc, mulc(taps.w[W - 1], dz));
        push<W, V>(win, x);
        return done;
      };
      // own rows only, and complete gradients of own rows only
      if (t0 - (W - 1) >= at && t0 + kN <= end && t0 + kN <= e - (W - 1)) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const Vec<V> done = token(i, true, true);
          if (on) stc<IO, V>(a.dx, put, done);
          put += a.C;
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < kN && t0 + i < past; ++i, put += a.C) {
          const int t = t0 + i, r = t - (W - 1);
          Vec<V> done = token(i, t < e, t < end);
          if (r >= at || at == s) {
            const int j = r - (e - (W - 1));
            if (j >= 0 && a.dstate_T)
              done = addc(done, ldc<IO, V>(a.dstate_T, ((int64_t)n * (W - 1) + j) * a.C + c));
            if (r >= s) {
              if (on) stc<IO, V>(a.dx, put, done);
            } else if (on && a.dstate) {
              stc<IO, V>(a.dstate, ((int64_t)n * (W - 1) + r - s + W - 1) * a.C + c, done);
            }
          }
        }
      }
    }
    at = end;
    cp_async_wait<0>();
    __syncwarp();
  }
  // dw and dbias of this block's rows
  auto sum = reinterpret_cast<float(*)[kCh<V>]>(raw);
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    const Vec<V> v = j < W ? dw[j < W ? j : 0] : db;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < V; ++h)
      *reinterpret_cast<float2*>(&sum[warp][2 * (V * lane + h)]) = v.p[h];
    __syncthreads();
    const int i = threadIdx.x;
    if (i < kCh<V> && blockIdx.x * kCh<V> + i < a.C) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t += sum[w][i];
      a.part[((int64_t)blockIdx.y * a.C + blockIdx.x * kCh<V> + i) * (W + 1) + j] = t;
    }
  }
}

// dw, dbias: the blocks' partials, 32 of them a block of threads, summed by
// the warps over every eighth and then over the warps (an order fixed by the
// shape and the number of SMs).  A bad packed call has none.  A call without tokens has no blocks in
// front of this one and gets its status word here.
__global__ void __launch_bounds__(kThreads) conv_dw_kernel(ConvArgs a, int W, int blocks,
                                                           float* dw, float* db) {
  after_the_last();
  __shared__ float sum[kWarps][32];
  if (a.cu && *a.status != CARVE_OK) return;
  if (blocks == 0) dense_ok(a);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = a.C * (W + 1), i = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (i < cols) {
#pragma unroll 4
    for (int k = warp; k < blocks; k += kWarps) t += a.part[(int64_t)k * cols + i];
  }
  sum[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && i < cols) {
    t = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sum[w][lane];
    const int c = i / (W + 1), j = i - c * (W + 1);
    if (j < W) dw[c * W + j] = t;
    else if (db) db[c] = t;
  }
}

// ------------------------------------------------------------------- step
// One token of each sequence, 4 channels a lane, the window shifted in place:
// bound by the launch and one trip to memory (2.3 us in a graph).
template <typename IO, int W>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a) {
  constexpr int V = 2;
  after_the_last();
  const int64_t i = 4 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= (int64_t)a.B * a.C) return;
  const int64_t n = i / a.C;
  const int c = (int)(i - n * a.C);
  const int64_t st = n * (W - 1) * a.C + c;
  const Vec<V> x = ldc<IO, V>(a.x, n * a.xp + c);
  Vec<V> win[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = ldc<IO, V>(a.state_T, st + (int64_t)j * a.C);
  const Taps<IO, W, V> taps(a, c);
  Vec<V> z = taps.z(win, x);
  if (a.silu) z = mulc(z, sigmoids<IO>(z));
  push<W, V>(win, x);
  stc<IO, V>(a.y, i, z);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) stc<IO, V>(a.state_T, st + (int64_t)j * a.C, win[j]);
}

// ------------------------------------------------------------------- host
carve_status check_conv(const carve_conv_shape* s) {
  if (!s) return CARVE_ERR_INVALID_ARG;
  if (s->B < 1 || s->T < 0 || s->C < 1 || s->W < 1 || s->reserved != 0 ||
      !dtype_ok(s->dtype) || !flag_ok(s->silu) || !flag_ok(s->fill_rest) ||
      !pitch_ok(s->x_pitch, s->C))
    return CARVE_ERR_INVALID_ARG;
  if (s->C % 8 || s->C > kMaxPitch || s->x_pitch > kMaxPitch || s->W < 2 ||
      s->W > 4)
    return CARVE_ERR_UNSUPPORTED;
  return CARVE_OK;
}

// Rows a warp walks: within a range, what leaves the last round of blocks the
// fullest, counting a start for each run; fewer where there are too few rows
// to reach every SM; more for very long batches.  The forward
// takes 48 to 96 (8 x 4096 x 6144: 133 us, against 139 with 64 to 256: many
// short runs even out), the backward 64 to 512 at a start's cost of 24 rows
// (237 us, against 252 with 48 to 96: each block ends with its sums of dw,
// and leaves them to be added up).
//
// Where there are too few rows for that, a lane takes 2 channels, so that there
// are more and lighter warps (forward and backward, 2 x 4096 x 1040 bf16 9.4
// and 20.6 us against 10.7 and 24.0, 3 x 1021 x 1040 fp32 6.2 and 14.0 against
// 7.0 and 18.2); with rows enough its rows of 128 bytes are the slower ones
// (8 x 4096 x 6144: 137 and 265 against 130 and 250 on the same device).
struct ConvPlan {
  int rows, run, cols, blocks;
  int pairs;  // V: pairs of channels a lane
};
constexpr int kMaxBlocks = 1024;
bool plan_conv(const carve_conv_shape& s, bool packed, bool backward, ConvPlan* p) {
  const int64_t rows = packed ? s.T : (int64_t)s.B * s.T;
  if (rows > kMaxTokens) return false;
  p->rows = (int)rows;
  const int64_t least = backward ? 64 : 48, most = backward ? 512 : 96;
  const int64_t start = backward ? 24 : 8;
  auto blocks = [&](int64_t run) { return (rows + run * kWarps - 1) / (run * kWarps); };
  int64_t resident = 0;
  auto wide = [&](int V, int per_sm) {
    p->pairs = V;
    p->cols = (s.C + 64 * V - 1) / (64 * V);
    resident = (int64_t)sm_count() * per_sm;
    return blocks(least) * p->cols > resident;
  };
  int64_t run = least;
  if (wide(2, backward ? kBwdPerSm<2> : kFwdPerSm<2>)) {
    int64_t best = 0;
    for (int64_t r = least; r <= most; r += 8) {
      const int64_t rounds = (blocks(r) * p->cols + resident - 1) / resident;
      if (!best || rounds * (r + start) < best) best = rounds * (r + start), run = r;
    }
  } else {
    wide(1, backward ? kBwdPerSm<1> : kFwdPerSm<1>);
    const int64_t room = (resident + p->cols - 1) / p->cols;  // blocks of a column
    run = (rows + room * kWarps - 1) / (room * kWarps);
    run = run < 8 ? (run < 1 ? 1 : run) : (run + 7) / 8 * 8;
  }
  while (blocks(run) > (backward ? kMaxBlocks : 65535)) run *= 2;
  p->run = (int)run;
  p->blocks = blocks(run) > 0 ? (int)blocks(run) : 1;
  return true;
}

size_t conv_ws(const carve_conv_shape& s, const ConvPlan& p, bool backward) {
  return kHeaderBytes +
         (backward ? align256((size_t)p.blocks * s.C * (s.W + 1) * 4) : 0);
}

ConvArgs conv_args(const carve_conv_shape& s, const ConvPlan& p,
                   const int32_t* cu, const void* x, const void* w,
                   const void* bias, void* ws, size_t ws_bytes) {
  ConvArgs a{};
  a.B = s.B; a.T = s.T; a.C = s.C; a.silu = s.silu; a.fill = s.fill_rest;
  a.rows = p.rows; a.run = p.run;
  a.xp = s.x_pitch ? s.x_pitch : s.C;
  a.cu = cu; a.x = x; a.w = w; a.bias = bias;
  a.status = status_word(ws, ws_bytes);
  return a;
}

enum Dir { kFwd, kBwd, kStep };
template <typename IO, int W, int V>
cudaError_t go(Dir d, const ConvArgs& a, dim3 grid, cudaStream_t st) {
  return d == kFwd
             ? launch<conv_fwd_kernel<IO, W, V>>(a, grid, kThreads, sizeof(FwdRing<IO, V>), st)
             : launch<conv_bwd_kernel<IO, W, V>>(a, grid, kThreads, sizeof(BwdRing<IO, V>), st);
}
template <typename IO, int W>
cudaError_t go_v(Dir d, int V, const ConvArgs& a, dim3 grid, cudaStream_t st) {
  if (d == kStep) return launch<conv_step_kernel<IO, W>>(a, grid, 128, 0, st);
  return V == 2 ? go<IO, W, 2>(d, a, grid, st) : go<IO, W, 1>(d, a, grid, st);
}
template <typename IO>
cudaError_t go_w(Dir d, int W, int V, const ConvArgs& a, dim3 grid, cudaStream_t st) {
  return W == 2 ? go_v<IO, 2>(d, V, a, grid, st)
                : W == 3 ? go_v<IO, 3>(d, V, a, grid, st) : go_v<IO, 4>(d, V, a, grid, st);
}
cudaError_t launch_conv(Dir d, const carve_conv_shape& s, int V, const ConvArgs& a, dim3 grid,
                        cudaStream_t st) {
  return s.dtype == CARVE_BF16 ? go_w<__nv_bfloat16>(d, s.W, V, a, grid, st)
                               : go_w<float>(d, s.W, V, a, grid, st);
}

// A batch without tokens: the states pass through.
cudaError_t pass_state(const carve_conv_shape& s, const void* src, void* dst,
                       cudaStream_t st) {
  if (!dst) return cudaSuccess;
  const size_t n = (size_t)s.B * (s.W - 1) * s.C * (s.dtype == CARVE_BF16 ? 2 : 4);
  return src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(dst, 0, n, st);
}

}  // namespace
}  // namespace mix
}  // namespace carve

using namespace carve;
using namespace carve::mix;

extern "C" {

size_t carve_conv_workspace_bytes(const carve_conv_shape* shape, int packed,
                                  int backward) {
  ConvPlan p;
  if (check_conv(shape) != CARVE_OK ||
      !plan_conv(*shape, packed != 0, backward != 0, &p))
    return 0;
  return conv_ws(*shape, p, backward != 0);
}

carve_status carve_conv_fwd(const carve_conv_shape* shape,
                            const int32_t* cu_seqlens, const void* x,
                            const void* w, const void* bias,
                            const void* state, void* y, void* state_T,
                            void* workspace, size_t workspace_bytes,
                            void* stream) {
  carve_status st = check_conv(shape);
  if (st != CARVE_OK) return st;
  const carve_conv_shape& s = *shape;
  ConvPlan p;
  if (!plan_conv(s, cu_seqlens != nullptr, false, &p)) return CARVE_ERR_UNSUPPORTED;
  if (!ptr_ok(w) || (s.T > 0 && (!ptr_ok(x) || !ptr_ok(y))))
    return CARVE_ERR_INVALID_ARG;
  if (!opt_ptr_ok(cu_seqlens) || !opt_ptr_ok(bias) || !opt_ptr_ok(state) ||
      !opt_ptr_ok(state_T))
    return CARVE_ERR_INVALID_ARG;
  if (cu_seqlens && (!workspace || !aligned16(workspace) ||
                     workspace_bytes < conv_ws(s, p, false)))
    return CARVE_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e;
  ConvArgs a = conv_args(s, p, cu_seqlens, x, w, bias, workspace, workspace_bytes);
  if (!cu_seqlens && s.T == 0) {
    static_assert(CARVE_OK == 0, "the status word by memset");
    e = pass_state(s, state, state_T, cs);
    if (e == cudaSuccess && a.status) e = cudaMemsetAsync(a.status, 0, sizeof(*a.status), cs);
  } else {
    a.state = state; a.y = y; a.state_T = state_T;
    e = launch_conv(kFwd, s, p.pairs, a, dim3(p.cols, p.blocks), cs);
  }
  return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA;
}

carve_status carve_conv_bwd(const carve_conv_shape* shape,
                            const int32_t* cu_seqlens, const void* x,
                            const void* w, const void* bias,
                            const void* state, const void* dy,
                            const void* dstate_T, void* workspace,
                            size_t workspace_bytes, void* dx, float* dw,
                            float* dbias, void* dstate, void* stream) {
  carve_status st = check_conv(shape);
  if (st != CARVE_OK) return st;
  const carve_conv_shape& s = *shape;
  ConvPlan p;
  if (!plan_conv(s, cu_seqlens != nullptr, true, &p)) return CARVE_ERR_UNSUPPORTED;
  if (!ptr_ok(w) || !ptr_ok(dw) ||
      (s.T > 0 && (!ptr_ok(x) || !ptr_ok(dy) || !ptr_ok(dx))))
    return CARVE_ERR_INVALID_ARG;
  if (!opt_ptr_ok(cu_seqlens) || !opt_ptr_ok(bias) || !opt_ptr_ok(state) ||
      !opt_ptr_ok(dstate_T) || !opt_ptr_ok(dbias) || !opt_ptr_ok(dstate))
    return CARVE_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < conv_ws(s, p, true))
    return CARVE_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)stream;
  ConvArgs a = conv_args(s, p, cu_seqlens, x, w, bias, workspace, workspace_bytes);
  a.state = state; a.dy = dy; a.dstate_T = dstate_T; a.dx = dx; a.dstate = dstate;
  a.part = (float*)((char*)workspace + kHeaderBytes);
  const bool none = !cu_seqlens && s.T == 0;
  cudaError_t e = none ? pass_state(s, dstate_T, dstate, cs)
                       : launch_conv(kBwd, s, p.pairs, a, dim3(p.cols, p.blocks), cs);
  if (e != cudaSuccess) return CARVE_ERR_CUDA;
  e = launch_all<conv_dw_kernel>((s.C * (s.W + 1) + 31) / 32, kThreads, 0, cs, 1, a, s.W,
                                 none ? 0 : p.blocks, dw, dbias);
  return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA;
}

carve_status carve_conv_step(const carve_conv_shape* shape, const void* x,
                             const void* w, const void* bias, void* state,
                             void* y, void* stream) {
  carve_status st = check_conv(shape);
  if (st != CARVE_OK) return st;
  const carve_conv_shape& s = *shape;
  if (!ptr_ok(x) || !ptr_ok(w) || !ptr_ok(state) || !ptr_ok(y) || !opt_ptr_ok(bias))
    return CARVE_ERR_INVALID_ARG;
  ConvPlan p{};
  ConvArgs a = conv_args(s, p, nullptr, x, w, bias, nullptr, 0);
  a.state_T = state; a.y = y;
  const int64_t blocks = ((int64_t)s.B * s.C / 4 + 127) / 128;
  if (blocks >= (1LL << 31)) return CARVE_ERR_UNSUPPORTED;
  return launch_conv(kStep, s, 2, a, dim3((unsigned)blocks), (cudaStream_t)stream) ==
                 cudaSuccess
             ? CARVE_OK
             : CARVE_ERR_CUDA;
}

}  // extern "C"

// carve_qk_rope.cu -- norms of the queries and keys of each head and the
// position rotation in one pass, forward and backward (declared in
// include/carve.h).
//
// A row (one token, one head) belongs to a group of P lanes, 8 elements a
// lane: two runs of 4, at i and j.  For the half-split rotation the runs are
// the two sides of the same 4 pairs, for the interleaved one they are
// neighbours; either way a lane holds both sides of its pairs and needs the
// angles 4 l .. 4 l + 3 only, which it computes once a token and uses for all
// the heads it takes.  Blocks take rows of q or rows of k, so that a lane has
// one set of weights and one of their gradients.  Rows come in through
// asynchronous copies of each lane's own elements into its own places in
// shared memory, a few rows ahead; no lane reads another's.
//
// What bounds it: 65536 tokens x (16 + 16) heads x 128 bf16 takes 164 us
// forward (6.5 TB/s of the rows in and out, what a plain copy reaches) and 270
// us backward with the weights' gradients (6.0 TB/s of 6 tensors); issue is at
// 74 and 69 %, so both are near its limit too.  With loads into registers in
// place of the rings they took 191 and 332.  Widths that are not 8 times a
// power of two leave lanes of a group without elements, which load and sum all
// the same, and issue is then the bound: 16384 x (12 + 12) x 80 takes 43 and 79
// us where its bytes take 19.5 and 29, x 96 37 and 67 (23 and 35), and (8 + 8)
// x 192 54 and 93 (31 and 47).
#include "mixer_common.cuh"

namespace carve {
namespace mix {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdPerSm = 4, kBwdPerSm = 3;  // blocks an SM holds
// Blocks of the backward, at most so many times that: fewer even out worse,
// more leave more partial sums (65536 x (16 + 16) x 128: 343, 292, 268, 263 us
// with 1, 2, 4, 8; 16384 x (8 + 8) x 256: 104, 94, 91, 93 us).
constexpr int kRounds = 4;

// q or k.
struct Side {
  const void *x, *dy, *w;
  void* out;
  int64_t pitch;
  int heads, slices, per;  // the heads of a token in `slices` parts of `per`
  int blocks;
};
struct RopeArgs {
  Side q, k;
  int64_t N;
  int D, RD, inter;
  float eps, inv_n;  // 1 / D, or 1 for the L2 norm
  const int32_t* pos;
  const double* freqs;
  float* part;  // [block][D] partial weight gradients
};

template <int P>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = P / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// What a lane of a group does in every row.
template <int P>
struct Lane {
  int l, i, j;   // lane of the group, its two runs (element offsets)
  bool on, rot;  // holds elements; holds rotated ones
  __device__ __forceinline__ explicit Lane(const RopeArgs& a) {
    l = threadIdx.x & (P - 1);
    on = l < a.D / 8;
    rot = l < a.RD / 8;
    const bool split = rot && !a.inter;
    // (idle lanes read the first elements and keep nothing)
    i = split ? 4 * l : on ? 8 * l : 0;
    j = split ? 4 * l + a.RD / 2 : i + 4;
  }
};

// cos and sin of the lane's 4 angles: the angle in turns, reduced in fp64
// (off by 2^-52 of the turns: 2^-34 of one at a million positions, 2^-23 at
// 2^31), then fp32.
__device__ __forceinline__ void angles(const RopeArgs& a, int l, int64_t token,
                                       Q& c, Q& s) {
  const double p = (double)a.pos[token] * 0.15915494309189533577;  // 1 / (2 pi)
  float cv[4], sv[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double t = p * a.freqs[4 * l + e];
    sincospif(2.f * (float)(t - rint(t)), &sv[e], &cv[e]);
  }
  c = Q{{make_float2(cv[0], cv[1]), make_float2(cv[2], cv[3])}};
  s = Q{{make_float2(sv[0], sv[1]), make_float2(sv[2], sv[3])}};
}

// (u, v) <- (u c - v s, u s + v c) over the lane's pairs.
__device__ __forceinline__ float2 turned(float2 n, float c, float s) {
  return make_float2(n.x * c - n.y * s, n.x * s + n.y * c);
}
__device__ __forceinline__ void turn(Q& u, Q& v, const Q& c, const Q& s, bool inter) {
  if (!inter) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = u.p[h], y = v.p[h];
      u.p[h] = fma2(x, c.p[h], mul2(y, make_float2(-s.p[h].x, -s.p[h].y)));
      v.p[h] = fma2(x, s.p[h], mul2(y, c.p[h]));
    }
  } else {
    u.p[0] = turned(u.p[0], c.p[0].x, s.p[0].x);
    u.p[1] = turned(u.p[1], c.p[0].y, s.p[0].y);
    v.p[0] = turned(v.p[0], c.p[1].x, s.p[1].x);
    v.p[1] = turned(v.p[1], c.p[1].y, s.p[1].y);
  }
}

__device__ __forceinline__ float inverse_norm(float ss, const RopeArgs& a) {
  const float m = fmaf(ss, a.inv_n, a.eps);
  return m == 0.f ? 0.f : rsqrtf(m);  // NaN stays: the whole row becomes NaN
}
__device__ __forceinline__ Q scaled(const Q& q, float f) {
  return Q{{mul2(q.p[0], both(f)), mul2(q.p[1], both(f))}};
}
// the sum of the 8 products
__device__ __forceinline__ float dot8(const Q& a, const Q& b, const Q& c, const Q& d) {
  const float2 t = fma2(a.p[0], b.p[0], fma2(a.p[1], b.p[1], fma2(c.p[0], d.p[0], mul2(c.p[1], d.p[1]))));
  return t.x + t.y;
}
__device__ __forceinline__ Q all4(float v) { return Q{{both(v), both(v)}}; }
__device__ __forceinline__ Q ones() { return all4(1.f); }

// A lane's ring of rows in shared memory: T tensors, R rows a stage.  The
// runs of one thread lie kThreads places apart.
template <typename IO, int T, int R, int STAGES>
struct Ring {
  using V = typename Raw<IO>::T;
  V* at;
  int in = 0, out = 0;
  __device__ __forceinline__ explicit Ring(void* smem)
      : at(static_cast<V*>(smem) + threadIdx.x) {}
  static constexpr size_t bytes() { return sizeof(V) * kThreads * 2 * T * R * STAGES; }
  template <int P>
  __device__ __forceinline__ void bring(const Lane<P>& ln, int t, const IO* rows, int D, int h,
                                        int h1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const IO* row = rows + min(h + r, h1 - 1) * D;  // past h1 the last head again
      copy(slot(in, t, r, 0), row + ln.i);
      copy(slot(in, t, r, 1), row + ln.j);
    }
  }
  __device__ __forceinline__ void brought() {
    ptx::cp_async_commit();
    in = in + 1 < STAGES ? in + 1 : 0;
  }
  __device__ __forceinline__ Q get(int t, int r, int run) const {
    return Raw<IO>::open(*slot(out, t, r, run));
  }
  __device__ __forceinline__ void next() { out = out + 1 < STAGES ? out + 1 : 0; }
  __device__ __forceinline__ V* slot(int stage, int t, int r, int run) const {
    return at + (((stage * T + t) * R + r) * 2 + run) * kThreads;
  }
  static __device__ __forceinline__ void copy(V* dst, const IO* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ptx::smem_u32(dst)),
                 "l"(src), "n"((int)sizeof(V)) : "memory");
  }
};

// The rows of a block's groups, one (token, part of its heads) at a time.
// The groups of a warp step together; `live` is false for those that are
// through.
template <int P, typename F>
__device__ __forceinline__ void each_item(const Side& sd, int64_t N, int block, F work) {
  constexpr int GROUPS = kThreads / P;
  const int64_t items = N * sd.slices, stride = (int64_t)sd.blocks * GROUPS;
  for (int64_t it = (int64_t)block * GROUPS + threadIdx.x / P; __any_sync(~0u, it < items);
       it += stride) {
    const bool live = it < items;
    const int64_t token = live ? it / sd.slices : 0;
    const int h0 = live ? (int)(it % sd.slices) * sd.per : 0;
    work(token, h0, live ? min(h0 + sd.per, sd.heads) : 0);
  }
}

template <typename IO>
struct FwdCfg {
  static constexpr int R = 2, STAGES = sizeof(IO) == 2 ? 4 : 3;
  using RingT = Ring<IO, 1, R, STAGES>;
};
template <typename IO, int P>
__global__ void __launch_bounds__(kThreads, kFwdPerSm) rope_fwd_kernel(RopeArgs a) {
  after_the_last();
  constexpr int R = FwdCfg<IO>::R, STAGES = FwdCfg<IO>::STAGES;
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<P> ln(a);
  const bool isk = blockIdx.x >= a.q.blocks;
  const Side sd = isk ? a.k : a.q;
  const Q wi = sd.w ? ldq<IO>(sd.w, ln.i) : ones(), wj = sd.w ? ldq<IO>(sd.w, ln.j) : ones();
  typename FwdCfg<IO>::RingT ring(smem);
  each_item<P>(sd, a.N, blockIdx.x - (isk ? a.q.blocks : 0), [&](int64_t token, int h0, int h1) {
    const IO* x = static_cast<const IO*>(sd.x) + token * sd.pitch;
    IO* out = static_cast<IO*>(sd.out) + (token * sd.heads + h0) * a.D;
    auto bring = [&](int h) {
      if (h < h1) ring.bring(ln, 0, x, a.D, h, h1);
      ring.brought();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) bring(h0 + i * R);
    Q c = ones(), s = none();
    if (ln.rot && h0 < h1) angles(a, ln.l, token, c, s);
    for (int h = h0; __any_sync(~0u, h < h1); h += R, out += R * a.D) {
      cp_async_wait<STAGES - 2>();
      bring(h + (STAGES - 1) * R);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Q u = ring.get(0, r, 0), v = ring.get(0, r, 1);
        float ss = dot8(u, u, v, v);
        if (P * 8 != a.D && !ln.on) ss = 0.f;
        const float n = inverse_norm(group_sum<P>(ss), a);
        u = mul4(scaled(u, n), wi);
        v = mul4(scaled(v, n), wj);
        if (ln.rot) turn(u, v, c, s, a.inter);
        if (ln.on && h + r < h1) {
          stq<IO>(out, r * a.D + ln.i, u);
          stq<IO>(out, r * a.D + ln.j, v);
        }
      }
      ring.next();
    }
    cp_async_wait<0>();
    ring.in = ring.out;
  });
}

// --------------------------------------------------------------- backward
// With n = x r (r the inverse norm) and d the gradient turned back:
// dw += d n, and with e = w d: dx = r (e - n (e . n) inv_n).
template <typename IO>
struct BwdCfg {
  static constexpr int R = sizeof(IO) == 2 ? 2 : 1, STAGES = 3;
  using RingT = Ring<IO, 2, R, STAGES>;
};
template <typename IO, int P>
__global__ void __launch_bounds__(kThreads, kBwdPerSm) rope_bwd_kernel(RopeArgs a) {
  after_the_last();
  constexpr int R = BwdCfg<IO>::R, STAGES = BwdCfg<IO>::STAGES, GROUPS = kThreads / P;
  extern __shared__ __align__(16) unsigned char smem[];
  const Lane<P> ln(a);
  const bool isk = blockIdx.x >= a.q.blocks;
  const Side sd = isk ? a.k : a.q;
  const Q wi = sd.w ? ldq<IO>(sd.w, ln.i) : ones(), wj = sd.w ? ldq<IO>(sd.w, ln.j) : ones();
  Q dwi = none(), dwj = none();
  typename BwdCfg<IO>::RingT ring(smem);
  each_item<P>(sd, a.N, blockIdx.x - (isk ? a.q.blocks : 0), [&](int64_t token, int h0, int h1) {
    const IO* x = static_cast<const IO*>(sd.x) + token * sd.pitch;
    const IO* dy = static_cast<const IO*>(sd.dy) + token * sd.heads * a.D;
    IO* out = static_cast<IO*>(sd.out) + (token * sd.heads + h0) * a.D;
    auto bring = [&](int h) {
      if (h < h1) {
        ring.bring(ln, 0, x, a.D, h, h1);
        ring.bring(ln, 1, dy, a.D, h, h1);
      }
      ring.brought();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) bring(h0 + i * R);
    Q c = ones(), s = none();
    if (ln.rot && h0 < h1) angles(a, ln.l, token, c, s);
    s = scaled(s, -1.f);  // turn back
    for (int h = h0; __any_sync(~0u, h < h1); h += R, out += R * a.D) {
      cp_async_wait<STAGES - 2>();
      bring(h + (STAGES - 1) * R);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const Q u = ring.get(0, r, 0), v = ring.get(0, r, 1);
        Q p = ring.get(1, r, 0), q = ring.get(1, r, 1);
        if (ln.rot) turn(p, q, c, s, a.inter);
        const Q ep = mul4(p, wi), eq = mul4(q, wj);
        float ss = dot8(u, u, v, v), dot = dot8(ep, u, eq, v);
        if (P * 8 != a.D && !ln.on) ss = dot = 0.f;
        const float n = inverse_norm(group_sum<P>(ss), a);
        const float along = -group_sum<P>(dot) * n * n * a.inv_n;
        if (h + r < h1) {
          dwi = fma4(p, scaled(u, n), dwi);
          dwj = fma4(q, scaled(v, n), dwj);
          if (ln.on) {
            stq<IO>(out, r * a.D + ln.i, scaled(fma4(u, all4(along), ep), n));
            stq<IO>(out, r * a.D + ln.j, scaled(fma4(v, all4(along), eq), n));
          }
        }
      }
      ring.next();
    }
    cp_async_wait<0>();
    ring.in = ring.out;
  });
  if (!a.part) return;
  __syncthreads();  // the rings are done with
  auto sum = reinterpret_cast<float(*)[8 * P]>(smem);
  const int grp = threadIdx.x / P;
  if (ln.on) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      *reinterpret_cast<float2*>(&sum[grp][ln.i + 2 * h]) = dwi.p[h];
      *reinterpret_cast<float2*>(&sum[grp][ln.j + 2 * h]) = dwj.p[h];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float t = 0.f;
    for (int g = 0; g < GROUPS; ++g) t += sum[g][d];
    a.part[(int64_t)blockIdx.x * a.D + d] = t;
  }
}

// dw[i] = sum over the partials of the blocks of q (blockIdx.y 0) or k, 32
// columns a block: 8 lanes read a row of them, every 128th row each, and the
// sums of the 128 are added in their order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(RopeArgs a, float* dwq, float* dwk,
                                                       uint32_t* status) {
  after_the_last();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *status = CARVE_OK;
  __shared__ float sum[128][33];
  const bool isk = blockIdx.y;
  const int row = threadIdx.x / 8, c = threadIdx.x % 8 * 4;
  const int i = blockIdx.x * 32 + c;
  const int lo = isk ? a.q.blocks : 0, hi = a.q.blocks + (isk ? a.k.blocks : 0);
  Q t = none();
  if (i < a.D) {
#pragma unroll 8
    for (int b = lo + row; b < hi; b += 128) t = add4(t, ldq<float>(a.part, (int64_t)b * a.D + i));
  }
  sum[row][c] = t.p[0].x, sum[row][c + 1] = t.p[0].y;
  sum[row][c + 2] = t.p[1].x, sum[row][c + 3] = t.p[1].y;
  __syncthreads();
  // 32 threads a column, four rows each, then across the warp
  const int col = threadIdx.x / 32, lane = threadIdx.x & 31;
  float v = (sum[lane][col] + sum[lane + 32][col]) + (sum[lane + 64][col] + sum[lane + 96][col]);
  v = group_sum<32>(v);
  float* out = isk ? dwk : dwq;
  const int at = blockIdx.x * 32 + col;
  if (lane == 0 && at < a.D && out) out[at] = v;
}

// ------------------------------------------------------------------- host
carve_status check_rope(const carve_rope_shape* s) {
  if (!s) return CARVE_ERR_INVALID_ARG;
  if (s->N < 0 || s->HQ < 1 || s->HK < 0 || s->D < 1 || s->RD < 0 ||
      s->RD > s->D || !dtype_ok(s->dtype) || !flag_ok(s->l2norm) ||
      !flag_ok(s->interleaved) || !(s->eps >= 0.f) || s->eps > 3.0e38f)
    return CARVE_ERR_INVALID_ARG;
  if (s->D % 16 || s->D > 256 || s->RD % 16 || s->HQ > (1 << 16) ||
      s->HK > (1 << 16) || s->N > kMaxTokens || s->q_pitch > kMaxPitch ||
      s->k_pitch > kMaxPitch)
    return CARVE_ERR_UNSUPPORTED;
  if (!pitch_ok(s->q_pitch, (int64_t)s->HQ * s->D) ||
      !pitch_ok(s->k_pitch, (int64_t)s->HK * s->D))
    return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}

int lanes_of(int D) {
  int p = 2;
  while (p < D / 8) p *= 2;
  return p;
}

// How the heads of a token are dealt out (all of a side's to one group of
// lanes once there are tokens enough for every group of the machine, fewer
// before), and the blocks of each side.  The forward has a group for each
// part; the backward's blocks leave a partial sum each, so they are fewer and
// take several.
void plan_side(const carve_rope_shape& s, int P, int64_t resident, int64_t most, int heads,
               Side* d) {
  const int groups = kThreads / P;
  d->heads = heads;
  d->slices = d->per = d->blocks = 0;
  if (heads == 0) return;
  const int64_t share = resident * groups * heads / (s.HQ + s.HK) + 1;
  int64_t sl = s.N > 0 ? (share + s.N - 1) / s.N : 1;
  sl = sl < heads ? sl : heads;
  d->per = (int)((heads + sl - 1) / sl);
  d->slices = (heads + d->per - 1) / d->per;
  const int64_t need = (s.N * d->slices + groups - 1) / groups;
  const int64_t cap = most * heads / (s.HQ + s.HK) + 1;
  d->blocks = (int)(need < cap ? need : cap);
}
RopeArgs rope_args(const carve_rope_shape& s, bool backward) {
  RopeArgs a{};
  a.N = s.N; a.D = s.D; a.RD = s.RD; a.inter = s.interleaved;
  a.eps = s.eps;
  a.inv_n = s.l2norm ? 1.f : 1.f / (float)s.D;
  a.q.pitch = s.q_pitch ? s.q_pitch : (int64_t)s.HQ * s.D;
  a.k.pitch = s.k_pitch ? s.k_pitch : (int64_t)s.HK * s.D;
  const int64_t resident = (int64_t)sm_count() * (backward ? kBwdPerSm : kFwdPerSm);
  const int64_t most = backward ? resident * kRounds : 1LL << 30;
  plan_side(s, lanes_of(s.D), resident, most, s.HQ, &a.q);
  plan_side(s, lanes_of(s.D), resident, most, s.HK, &a.k);
  return a;
}

template <typename IO, int P>
cudaError_t go(bool bwd, const RopeArgs& a, cudaStream_t st) {
  const dim3 grid(a.q.blocks + a.k.blocks);
  if (!bwd)
    return launch<rope_fwd_kernel<IO, P>>(a, grid, kThreads, FwdCfg<IO>::RingT::bytes(), st);
  constexpr size_t sums = sizeof(float) * 8 * kThreads, ring = BwdCfg<IO>::RingT::bytes();
  return launch<rope_bwd_kernel<IO, P>>(a, grid, kThreads, ring > sums ? ring : sums, st);
}
template <typename IO>
cudaError_t go_p(bool bwd, int P, const RopeArgs& a, cudaStream_t st) {
  switch (P) {
    case 2: return go<IO, 2>(bwd, a, st);
    case 4: return go<IO, 4>(bwd, a, st);
    case 8: return go<IO, 8>(bwd, a, st);
    case 16: return go<IO, 16>(bwd, a, st);
    default: return go<IO, 32>(bwd, a, st);
  }
}
cudaError_t launch_rope(bool bwd, const RopeArgs& a, int dtype, cudaStream_t st) {
  const int P = lanes_of(a.D);
  return dtype == CARVE_BF16 ? go_p<__nv_bfloat16>(bwd, P, a, st) : go_p<float>(bwd, P, a, st);
}

// The pointers both directions take.
bool rope_ptrs_ok(const carve_rope_shape& s, const void* q, const void* k,
                  const void* pos, const void* freqs, const void* w_q,
                  const void* w_k) {
  if (s.N > 0 && (!ptr_ok(q) || (s.HK > 0 && !ptr_ok(k)))) return false;
  if (s.N > 0 && s.RD > 0 && (!ptr_ok(pos) || !ptr_ok(freqs))) return false;
  return opt_ptr_ok(w_q) && opt_ptr_ok(w_k);
}

}  // namespace
}  // namespace mix
}  // namespace carve

using namespace carve;
using namespace carve::mix;

extern "C" {

size_t carve_qk_rope_workspace_bytes(const carve_rope_shape* shape) {
  if (check_rope(shape) != CARVE_OK) return 0;
  const RopeArgs a = rope_args(*shape, true);
  return kHeaderBytes + align256((size_t)(a.q.blocks + a.k.blocks + 1) * shape->D * 4);
}

carve_status carve_qk_rope_fwd(const carve_rope_shape* shape, const void* q,
                               const void* k, const int32_t* pos,
                               const double* freqs, const void* w_q,
                               const void* w_k, void* q_out, void* k_out,
                               void* stream) {
  carve_status st = check_rope(shape);
  if (st != CARVE_OK) return st;
  const carve_rope_shape& s = *shape;
  if (!rope_ptrs_ok(s, q, k, pos, freqs, w_q, w_k)) return CARVE_ERR_INVALID_ARG;
  if (s.N > 0 && (!ptr_ok(q_out) || (s.HK > 0 && !ptr_ok(k_out))))
    return CARVE_ERR_INVALID_ARG;
  if (s.N == 0) return CARVE_OK;
  RopeArgs a = rope_args(s, false);
  a.q.x = q; a.k.x = k; a.pos = pos; a.freqs = freqs; a.q.w = w_q; a.k.w = w_k;
  a.q.out = q_out; a.k.out = k_out;
  return launch_rope(false, a, s.dtype, (cudaStream_t)stream) == cudaSuccess
             ? CARVE_OK
             : CARVE_ERR_CUDA;
}

carve_status carve_qk_rope_bwd(const carve_rope_shape* shape, const void* q,
                               const void* k, const int32_t* pos,
                               const double* freqs, const void* w_q,
                               const void* w_k, const void* dq_out,
                               const void* dk_out, void* workspace,
                               size_t workspace_bytes, void* dq, void* dk,
                               float* dw_q, float* dw_k, void* stream) {
  carve_status st = check_rope(shape);
  if (st != CARVE_OK) return st;
  const carve_rope_shape& s = *shape;
  if (!rope_ptrs_ok(s, q, k, pos, freqs, w_q, w_k)) return CARVE_ERR_INVALID_ARG;
  if (s.N > 0 && (!ptr_ok(dq_out) || !ptr_ok(dq) ||
                  (s.HK > 0 && (!ptr_ok(dk_out) || !ptr_ok(dk)))))
    return CARVE_ERR_INVALID_ARG;
  if ((w_q && !ptr_ok(dw_q)) || (w_k && !ptr_ok(dw_k)))
    return CARVE_ERR_INVALID_ARG;
  const bool sums = w_q || w_k;
  if (sums && (!workspace || !aligned16(workspace) ||
               workspace_bytes < carve_qk_rope_workspace_bytes(shape)))
    return CARVE_ERR_WORKSPACE;
  RopeArgs a = rope_args(s, true);
  a.q.x = q; a.k.x = k; a.pos = pos; a.freqs = freqs; a.q.w = w_q; a.k.w = w_k;
  a.q.dy = dq_out; a.k.dy = dk_out; a.q.out = dq; a.k.out = dk;
  a.part = sums ? (float*)((char*)workspace + kHeaderBytes) : nullptr;
  cudaStream_t cs = (cudaStream_t)stream;
  if (s.N > 0 && launch_rope(true, a, s.dtype, cs) != cudaSuccess)
    return CARVE_ERR_CUDA;
  if (sums) {
    if (launch_all<rope_dw_kernel>(dim3((s.D + 31) / 32, 2), 1024, 0, cs, 1, a,
                                   w_q ? dw_q : nullptr, w_k ? dw_k : nullptr,
                                   static_cast<uint32_t*>(workspace)) != cudaSuccess)
      return CARVE_ERR_CUDA;
  }
  return CARVE_OK;
}

}  // extern "C"

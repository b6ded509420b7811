// carve_scan.cu -- the gated linear scan h_t = exp(g_t) h_{t-1} + u_t,
// forward, backward and one-token form (declared in include/carve.h).
//
// The scan is linear, so the tokens of a segment act on the state before
// them as one pair (A, H): h_after = A h_before + H with A the product of the
// decays and H the segment's own result from zero.  Pairs compose from the
// left, (A1, H1) then (A2, H2) = (A1 A2, A2 H1 + H2).
//
// Layout.  A block takes 64 channels, 2 a lane, so that a row of a tile is one
// or two whole 128-byte lines and the arithmetic is that on packed pairs; its
// 8 warps take a segment of a tile's tokens each (16; 8 in fp32 and in the
// backward, where registers and shared memory hold no more).  Tiles arrive
// through asynchronous copies three stages deep.  Per tile a warp forms its
// segment's pair, the block shares the 8 pairs, and each warp folds those
// before it and walks its segment once more from the state it got: x and g
// are read from memory once, from shared memory twice.  (16 warps of 8 tokens
// were slower, 107 us against 82 forward at 8 x 4096 x 2048: twice the pairs
// to share; so was forming the outputs from the first walk's values and the
// products of the decays, 95 against 76: registers.)
//
// Few chains (ranges x groups of channels) leave SMs idle, so a cluster of up
// to 8 blocks takes a range's tiles in turn and passes the pairs of whole
// tiles through distributed shared memory, one warp of each block sending and
// folding (all 8 doing it took 199 us against 172 at 1 x 65536 x 2048 with
// activation and complement).
//
// What bounds it (bf16, 6.47 TB/s of measured copy bandwidth): 8 x 4096 x 2048
// forward 70 us, 5.7 TB/s of x, g and h, at 19.5 instructions an element and
// 58 % of the issue slots: memory and issue together.  With activation and
// complement 109 us: the polynomials, 33 instructions an element; no unit is
// full (issue 60 %, the heavy half of the FMA pipe 61 %, DRAM 39 %), and the
// warps' first stall is the math pipes.  Backward 117 us, 5.7 TB/s of its 5
// tensors; with activation and complement 195 us, 60 instructions an
// element (62 %, 56 % and 39 %).  Packed rows add the borders, whose
// segments a cluster waits for: 57 us forward, 94 to 104 backward, where one
// sequence of as many tokens takes 47 and 75, and the bytes 31 and 52 (16384
// tokens x 2048 in 33 sequences with states).  With a border every 65 tokens
// nearly every step waits: 239 and 320 us for 500 sequences in 32768 x 2048,
// whose bytes take 62 and 104.  Few channels leave SMs without a block: 110 and
// 199 us for 1 x 65536 x 512, bytes 31 and 52.
#include "mixer_common.cuh"

#include <cooperative_groups.h>
#include <limits.h>
#include <type_traits>

namespace carve {
namespace mix {
namespace {

constexpr int kCh = 64;         // channels of a block: 2 a lane
constexpr int kThreads = 256;   // 8 warps, one segment of tokens each
constexpr int kWarps = kThreads / 32;
constexpr int kKeep = 64;       // tokens between kept states (training)
constexpr int kMaxCluster = 8;
constexpr int kKeepCu = 512;   // packed offsets a block keeps in shared memory

struct ScanArgs {
  int B, T, C, comp, fill;
  float dscale;
  int64_t xp, gp;
  const void *x, *g, *d_h;
  const float *h0, *dh_T;
  void *h, *dx, *dg;
  float *h_T, *dh0;
  const int32_t* cu;
  uint32_t* status;   // NULL without a workspace
  float* keep;        // [range][tiles][C] states before every 64th token
  float* keep_h0;     // [B][C] initial states (segmented calls)
  int ranges;         // independent stretches of tokens
  int seqs;           // sequences of a range (segmented, cu == NULL)
  int groups;         // blocks of kCh channels
  int tiles;          // kept states of a range
  long long spin;     // cycles a wait for a peer's pair spins before it gives up
  int stall;          // test only: step at which block 1 keeps its pair (-1: none)
};

// exp(u), and with REST also 1 - exp(u), of a pair of log-decays.  A decay
// near 1 acts over many tokens, so its error counts as often: the hardware's
// 2^x is low by about 2e-8 there on average, enough to show after a thousand
// tokens.  Close to zero both therefore come from the series of exp(u) - 1:
// four terms within 1/16 (the first one left out is below 2^-27), six within
// 1/4 where 1 - exp(u) needs its own relative accuracy (below 2^-24 of it).
template <typename IO, bool REST>
__device__ __forceinline__ void decays(float2 u, float2& a, float2& rest) {
  constexpr float kNear = REST ? 0.25f : 0.0625f;
  float2 p = both(1.f / 24);
  if (REST) p = fma2(u, fma2(u, both(1.f / 720), both(1.f / 120)), p);
  p = fma2(u, p, both(1.f / 6));
  p = fma2(u, p, both(0.5f));
  p = fma2(u, p, both(1.f));
  const float2 e = exp_of<IO>(u);
  const bool nx = fabsf(u.x) < kNear, ny = fabsf(u.y) < kNear;
  if (REST) {
    const float2 m = mul2(u, p);  // exp(u) - 1
    rest.x = nx ? -m.x : 1.f - e.x;
    rest.y = ny ? -m.y : 1.f - e.y;
    p = add2(m, both(1.f));
  } else {
    p = fma2(u, p, both(1.f));
  }
  a.x = nx ? p.x : e.x;
  a.y = ny ? p.y : e.y;
}

// The fused activation u = -s softplus(g) of a pair, and with SLOPE its
// derivative -s sigmoid(g).  softplus(g) = max(g, 0) + log(1 + e) with e =
// exp(-|g|) <= 1; log(1 + e) / e on [0, 1] is a polynomial of degree 8 fitted
// for the least largest relative error (3e-8; below 1.5e-7 in fp32).
template <typename IO, bool SLOPE>
__device__ __forceinline__ float2 activated(float2 g, float s, float2& slope) {
  const float2 e = exp_of<IO>(make_float2(-fabsf(g.x), -fabsf(g.y)));
  float2 p = fma2(e, both(0.005232689436525106f), both(-0.02950522117316723f));
  p = fma2(e, p, both(0.07822592556476593f));
  p = fma2(e, p, both(-0.13663244247436523f));
  p = fma2(e, p, both(0.19106006622314453f));
  p = fma2(e, p, both(-0.2484298199415207f));
  p = fma2(e, p, both(0.3331909775733948f));
  p = fma2(e, p, both(-0.4999949336051941f));
  p = fma2(e, p, both(0.9999999403953552f));
  if (SLOPE) {
    const float2 o = add2(e, both(1.f));
    const float2 d = mul2(make_float2(rcp(o.x), rcp(o.y)), both(-s));
    slope = make_float2(g.x >= 0.f ? d.x : d.x * e.x, g.y >= 0.f ? d.y : d.y * e.y);
  }
  return mul2(fma2(e, p, make_float2(fmaxf(g.x, 0.f), fmaxf(g.y, 0.f))), both(-s));
}

// The decay of a gate pair, 1 minus it, and the slope of the activation.
template <typename IO, bool ACT, bool REST, bool SLOPE>
__device__ __forceinline__ void gate(float2 g, float s, float2& a, float2& rest,
                                     float2& slope) {
  decays<IO, REST>(ACT ? activated<IO, SLOPE>(g, s, slope) : g, a, rest);
}

// The state after a segment from the one before it.  A segment that starts a
// sequence (`reset`, the same for all lanes) does not depend on what came
// before, which must not meet it in a product: it may be infinite or NaN.
__device__ __forceinline__ void advance(bool reset, float2 A, float2 H, float2& h) {
  h = reset ? H : fma2(A, h, H);
}

// Copies of ROWS x kCh tiles of one tensor into shared memory, 16 bytes a
// thread at a time; rows from `end` on and channels from C on become zero.
// The address is a base that all threads share and a 32-bit offset.
template <typename IO, int ROWS>
struct Loader {
  static constexpr int E = 16 / sizeof(IO), PER = kCh / E, STEP = kThreads / PER;
  static_assert(ROWS % STEP == 0, "whole passes");
  const char* base;      // row 0, channel c0
  int64_t pitch;         // bytes
  uint32_t from, step;   // this thread's offset, and from pass to pass
  int row, at;           // its row, and its place in the tile
  bool ok;
  __device__ __forceinline__ Loader(const IO* p, int64_t pitch_, int c0, int C)
      : base(reinterpret_cast<const char*>(p + c0)), pitch(pitch_ * sizeof(IO)) {
    row = threadIdx.x / PER;
    const int c = threadIdx.x % PER * E;
    at = row * kCh + c;
    ok = c0 + c < C;
    from = row * (uint32_t)pitch + (ok ? c : 0) * sizeof(IO);
    step = STEP * (uint32_t)pitch;
  }
  __device__ __forceinline__ void operator()(IO* dst, int t, int end) const {
    const char* tile = base + t * pitch;
    uint32_t off = from;
    if (t + ROWS <= end) {
#pragma unroll
      for (int i = 0; i < ROWS / STEP; ++i, off += step)
        cp_async16_zfill(dst + at + i * STEP * kCh, tile + off, ok);
    } else {
#pragma unroll
      for (int i = 0; i < ROWS / STEP; ++i, off += step) {
        const bool in = ok && t + row + i * STEP < end;
        cp_async16_zfill(dst + at + i * STEP * kCh, in ? tile + off : base, in);
      }
    }
  }
};

// Everything the two chunk-walking kernels find out first: the range of
// tokens, the channel group and the rank in the cluster.
struct Place {
  int range, c0, rank, ncl;
  int64_t row0;  // first row of the range
  int len;       // its tokens
  int seq0;      // its first sequence
  Bounds b;      // sequence starts within the range
};
template <bool SEG>
__device__ __forceinline__ Place place_of(const ScanArgs& a) {
  Place p;
  p.ncl = cooperative_groups::this_cluster().num_blocks();
  p.rank = cooperative_groups::this_cluster().block_rank();
  const int chain = blockIdx.x / p.ncl;
  p.range = chain / a.groups;
  p.c0 = chain % a.groups * kCh;
  if (SEG && !a.cu) {
    p.seq0 = p.range * a.seqs;
    p.b = Bounds{nullptr, a.T, min(a.seqs, a.B - p.seq0)};
    p.row0 = (int64_t)p.seq0 * a.T;
    p.len = p.b.n * a.T;
  } else {
    p.seq0 = SEG ? 0 : p.range;
    p.b = Bounds{a.cu, a.T, a.B};
    p.row0 = SEG ? 0 : (int64_t)p.range * a.T;
    p.len = a.T;
  }
  return p;
}

// Out of line: borders are rare, and the loops around the calls unrolled.
__device__ __noinline__ int seq_of(const Bounds b, int t) { return b.seq_of(t); }

// What sequence borders make of a warp's segment of S tokens.
enum Kind {
  kPlain,    // S tokens inside one sequence
  kMarked,   // S tokens of sequences, at most one first and one last of them
  kOutside,  // no token of any sequence
  kRagged    // anything else: token by token
};
// What is known of a segment that is not plain lies in shared memory, so that
// plain ones carry nothing along.
struct Edge {
  Marks m;
  int first, last;   // the sequences of the first start and the last end
  float2 start[32];  // the state that start brings in, by lane (kMarked)
};
// 32 neighbouring borders, one a lane: as long as a segment lies among them,
// two votes tell whether any falls into it.
struct Borders {
  int first;  // index of lane 0's
  int mine;
  __device__ __forceinline__ void load(const Bounds& b, int from) {
    const int i = (first = from) + (int)(threadIdx.x & 31);
    mine = i < 0 ? INT_MIN : i > b.n ? INT_MAX : b.at(i);
  }
};

__device__ __forceinline__ float2 ld_state(const float* p, int64_t row, int C,
                                           int c) {
  return p && c < C ? ld2(p + row * C + c) : make_float2(0.f, 0.f);
}

// REV: segments come from the last to the first.
template <bool SEG, int S, bool REV>
__device__ __forceinline__ Kind look(const Place& p, Borders& near, int t0, Edge* e) {
  const bool full = t0 + S <= p.len;
  if (!SEG) return full ? kPlain : kRagged;
  if (t0 >= p.len) return kOutside;
  unsigned below = __ballot_sync(~0u, near.mine < t0);
  unsigned upto = __ballot_sync(~0u, near.mine <= t0 + S);
  if (!below || !~upto) {
    near.load(p.b, p.b.first_at_least(t0) - (REV ? 24 : 1));
    below = __ballot_sync(~0u, near.mine < t0);
    upto = __ballot_sync(~0u, near.mine <= t0 + S);
  }
  const bool clear = below == upto;  // no border in [t0, t0 + S]
  if (clear) {
    const int i = near.first + __popc(below);
    if (i <= 0 || i > p.b.n) return kOutside;
    if (full) return kPlain;
  }
  Marks m{0u, 0u, p.b.at(0), p.b.at(p.b.n)};
  int first = 0, last = 0;
  if (clear) {
    // the end of the batch cuts it short
  } else if (t0 >= m.hi || t0 + S <= m.lo) {
    return kOutside;
  } else if (~upto) {
    const int v = near.mine, d = v - t0;
    if ((upto & ~below) >> (threadIdx.x & 31) & 1) {
      if (v < m.hi && d < S) m.start = 1u << d;
      if (v > m.lo && d >= 1) m.end = 1u << (d - 1);
    }
    m.start = __reduce_or_sync(~0u, m.start);
    m.end = __reduce_or_sync(~0u, m.end);
    // the sequence of a token is the last that starts at it or before it
    first = near.first - 1 +
            __popc(__ballot_sync(~0u, v <= t0 + __ffs(m.start) - 1));
    last = near.first - 1 + __popc(__ballot_sync(~0u, v <= t0 + 31 - __clz(m.end)));
  } else {  // too many borders at one place
    m = marks_of<S>(p.b, t0);
    if (m.start) first = p.b.seq_of(t0 + __ffs(m.start) - 1);
    if (m.end) last = p.b.seq_of(t0 + 31 - __clz(m.end));
  }
  if ((threadIdx.x & 31) == 0) {
    e->m = m;
    e->first = first;
    e->last = last;
  }
  __syncwarp();
  const bool one = !(m.start & m.start - 1) && !(m.end & m.end - 1);
  return full && one && t0 >= m.lo && t0 + S <= m.hi ? kMarked : kRagged;
}

// Asks the L1 for the states that the borders in the segment from t0 on bring
// in, if the borders at hand show any: they are needed a step later.
template <int S>
__device__ __forceinline__ void ask_ahead(const ScanArgs& a, const Place& p, const Borders& near,
                                          int t0, const float* starts, const float* ends, int c) {
  if (!starts && !ends) return;
  const unsigned below = __ballot_sync(~0u, near.mine < t0);
  const unsigned upto = __ballot_sync(~0u, near.mine <= t0 + S);
  if (below == upto || !below || !~upto || c >= a.C) return;
  const int last = near.first - 1 + __popc(below), first = near.first - 1 + __popc(upto);
  if (starts && first < p.b.n)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(starts + (int64_t)(p.seq0 + first) * a.C + c));
  if (ends && last >= 0)
    asm volatile("prefetch.global.L1 [%0];" ::"l"(ends + (int64_t)(p.seq0 + last) * a.C + c));
}

// Asks the L2 for the states that the packed sequences bring in, this block's
// channels of them: a border then costs an L2 access, not one of DRAM.
__device__ __forceinline__ void ask_states(const ScanArgs& a, const Place& p,
                                           const float* states) {
  if (!states) return;
  for (int i = p.rank * kThreads + threadIdx.x; i < 2 * a.B; i += p.ncl * kThreads) {
    const int c = p.c0 + (i & 1) * (kCh / 2);  // 128 bytes
    if (c < a.C)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(states + (int64_t)(i >> 1) * a.C + c));
  }
}

// Copies dst[n] = src[n] (or zero) for the empty sequences of a packed
// batch, this block's channels, the sequences spread over the cluster.
__device__ __forceinline__ void copy_empty(const ScanArgs& a, const Place& p,
                                           const float* src, float* dst) {
  if (!dst) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = p.c0 + 2 * lane;
  for (int n0 = (p.rank * kWarps + warp) * 32; n0 < a.B;
       n0 += p.ncl * kWarps * 32) {
    const int n = n0 + lane;
    unsigned m = __ballot_sync(~0u, n < a.B && a.cu[n] == a.cu[n + 1]);
    for (; m; m &= m - 1) {
      const int64_t row = n0 + __ffs(m) - 1;
      if (c < a.C) st2(dst + row * a.C + c, ld_state(src, row, a.C, c));
    }
  }
}

// One token of a staged tile: its decay and what enters the state.
template <bool ACT, bool COMP, typename IO>
__device__ __forceinline__ void token(const IO* x, const IO* g, int at, float s,
                                      float2& d, float2& v) {
  float2 rest, slope;
  gate<IO, ACT, COMP, false>(ld2(g + at), s, d, rest, slope);
  v = ld2(x + at);
  if (COMP) v = mul2(v, rest);
}

// Exchange of the pairs of a cluster's blocks.  In every step each block
// writes its pair into a slot of every block (its own too), counted on that
// block's barrier in bytes, and waits for all of them.  Two slots by the
// parity of the step are enough: a block sends step s + 2 after it has all of
// s + 1, which the others sent after they had read s.
struct Exchange {
  float4 slot[2][kMaxCluster][32];
  uint64_t bar[2];
};
__device__ __forceinline__ void start_exchange(Exchange& x, int ncl) {
  if (ncl == 1) return;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&x.bar[0], 1);
    ptx::mbar_init(&x.bar[1], 1);
    ptx::mbar_init_fence();
  }
  cooperative_groups::this_cluster().sync();
}
// One warp sends this block's pair to every block.
__device__ __forceinline__ void send_pair(Exchange& x, const ScanArgs& a, int step,
                                          int rank, int ncl, float2 A, float2 H) {
  const int lane = threadIdx.x & 31;
  if (lane == 0)
    ptx::mbar_expect_tx(&x.bar[step & 1], ncl * 32 * (uint32_t)sizeof(float4));
  if (blockIdx.x == 1 && step == a.stall) return;
  const uint32_t slot = ptx::smem_u32(&x.slot[step & 1][rank][lane]);
  const uint32_t mbar = ptx::smem_u32(&x.bar[step & 1]);
  for (int r = 0; r < ncl; ++r) {
    uint32_t to, bar;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(slot), "r"(r));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(mbar), "r"(r));
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 "
        "[%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "f"(A.x), "f"(A.y), "f"(H.x),
        "f"(H.y), "r"(bar) : "memory");
  }
}
// False when the pairs of the step have not come within the limit.
__device__ __forceinline__ bool wait_pairs(Exchange& x, const ScanArgs& a, int step) {
  const uint32_t bar = ptx::smem_u32(&x.bar[step & 1]), parity = step >> 1 & 1;
  const long long began = clock64();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    if (ok) return true;
    if (clock64() - began > a.spin) return false;
  }
}
// The state before this block (through the lower, or with REV the higher,
// ranks) from its own pair and the others'; `carry` moves past the whole
// cluster.  One warp of each block does this.  If it gives up waiting it goes
// on with NaN and sends no more, so that its peers give up as well.
template <bool RST, bool REV>
__device__ __forceinline__ float2 over_cluster(Exchange& x, const ScanArgs& a, int step,
                                               int rank, int ncl, float2 A, float2 H,
                                               float2& carry, bool& dead) {
  const int lane = threadIdx.x & 31;
  if (!dead) {
    send_pair(x, a, step, rank, ncl, A, H);
    dead = !__all_sync(~0u, wait_pairs(x, a, step));
  }
  if (dead) {
    if (a.status && lane == 0) *a.status = CARVE_ERR_TIMEOUT;
    carry = both(__int_as_float(0x7fc00000));
    return carry;
  }
  float2 before = carry;
#pragma unroll 4
  for (int i = 0; i < ncl; ++i) {
    const int r = REV ? ncl - 1 - i : i;
    if (r == rank) before = carry;
    const float4 v = x.slot[step & 1][r][lane];
    advance(RST && v.x < 0.f, make_float2(v.x, v.y), make_float2(v.z, v.w), carry);
  }
  return before;
}

// The pairs of a block's warps.  In the backward each segment has two, with
// the same A: of the states (H) and, backwards, of the gradients (R).
template <bool BWD>
struct Pairs {
  float2 A[kWarps][32], H[kWarps][32], R[BWD ? kWarps : 1][32];
  union {
    uint8_t reset[kWarps];  // bit 0: a sequence starts; bit 1: one ends
    uint64_t resets;        // all of them: usually none, which one load tells
  };
  // Bit 8 w: warp w starts anew (REV: seen from behind).
  template <bool SEG, bool REV>
  __device__ __forceinline__ uint64_t news() const {
    return SEG ? resets >> REV & 0x0101010101010101ull : 0;
  }
  template <bool REV>
  __device__ __forceinline__ void past(int w, bool reset, float2& h) const {
    const int lane = threadIdx.x & 31;
    advance(reset, A[w][lane], REV ? R[w][lane] : H[w][lane], h);
  }
  // Takes the state before the tile to the one before this warp's segment
  // (REV: the gradient after it to the one after the segment).
  template <bool SEG, bool REV>
  __device__ __forceinline__ void fold(int warp, float2& h) const {
    const uint64_t m = news<SEG, REV>();
    if (SEG && m) {
      if (!REV)
        for (int w = 0; w < warp; ++w) past<REV>(w, reset[w] & 1, h);
      else
        for (int w = kWarps - 1; w > warp; --w) past<REV>(w, reset[w] & 2, h);
    } else {
      if (!REV)
        for (int w = 0; w < warp; ++w) past<REV>(w, false, h);
      else
        for (int w = kWarps - 1; w > warp; --w) past<REV>(w, false, h);
    }
  }
};
// All of them as one pair, from the first warp on or, with REV, the last; a
// negative A stands for a reset.
template <bool SEG, bool REV, bool BWD>
__device__ __forceinline__ void total(const Pairs<BWD>& q, float2& A, float2& H) {
  const int lane = threadIdx.x & 31;
  const uint64_t m = q.template news<SEG, REV>();
  A = both(1.f);
  H = both(0.f);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int w = REV ? kWarps - 1 - i : i;
    q.template past<REV>(w, SEG && (q.reset[w] >> REV & 1), H);
    A = mul2(A, q.A[w][lane]);
  }
  if (m) A = both(-1.f);
}

// Two blocks share an SM: 228 KB, less 1 KB a block.
template <typename Smem>
constexpr bool two_fit() {
  return sizeof(Smem) <= 113 * 1024;
}

// No block leaves while a peer may still write to it.
__device__ __forceinline__ void finish_exchange(Exchange& x, const ScanArgs& a,
                                                int steps, int ncl, bool dead) {
  if (ncl == 1) return;
  cooperative_groups::this_cluster().sync();
  // what was on its way to a block that gave up gets the same time again
  if (dead && steps > 0) wait_pairs(x, a, steps - 1);
}

// ---------------------------------------------------------------- forward
template <typename IO, bool SEG>
struct FwdTile {
  static constexpr int S = sizeof(IO) == 2 ? 16 : 8;  // tokens of a warp
  static constexpr int TILE = kWarps * S;
  static constexpr int STAGES = 3;
  // Whether the next tile is asked for after the pairs are formed instead of
  // first of all (4 x 4096 x 2048 fp32: forward 71 us against 73, backward
  // 108 against 124; bf16 at 8 sequences: 72 against 70, and 118 either way).
  static constexpr bool LATE = sizeof(IO) == 4;
  struct Stage {
    IO x[TILE * kCh], g[TILE * kCh];
  };
  struct Smem {
    Stage st[STAGES];
    Pairs<false> pairs;
    float2 last[2][32];  // by the parity of the step
    Exchange ex;
    Edge edge[SEG ? kWarps : 1];
    int32_t cu[SEG ? kKeepCu : 1];
  };
};

template <typename IO, bool SEG, bool ACT, bool COMP>
__global__ void __launch_bounds__(kThreads, 2) scan_fwd_kernel(ScanArgs a) {
  after_the_last();
  using F = FwdTile<IO, SEG>;
  static_assert(two_fit<typename F::Smem>(), "shared memory of two blocks");
  constexpr int S = F::S, TILE = F::TILE, STAGES = F::STAGES;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sm = *reinterpret_cast<typename F::Smem*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Place p = place_of<SEG>(a);
  const int c = p.c0 + 2 * lane;
  const bool ch_ok = c < a.C;
  const Loader<IO, TILE> load_x(static_cast<const IO*>(a.x) + p.row0 * a.xp, a.xp, p.c0, a.C);
  const Loader<IO, TILE> load_g(static_cast<const IO*>(a.g) + p.row0 * a.gp, a.gp, p.c0, a.C);
  IO* h_out = static_cast<IO*>(a.h) + p.row0 * a.C;
  const int64_t row_bytes = (int64_t)a.C * sizeof(IO);
  const uint32_t out_off = warp * S * (uint32_t)row_bytes + c * (uint32_t)sizeof(IO);
  const int at0 = warp * S * kCh + 2 * lane;

  const int steps = (p.len + TILE * p.ncl - 1) / (TILE * p.ncl);
  int in_stage = 0, stage = 0;
  auto fetch = [&](int step) {
    if (step < steps) {
      const int t = (step * p.ncl + p.rank) * TILE;
      auto& st = sm.st[in_stage];
      load_x(st.x, t, p.len);
      load_g(st.g, t, p.len);
    }
    ptx::cp_async_commit();
    in_stage = in_stage + 1 < STAGES ? in_stage + 1 : 0;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  if (SEG && a.cu) {
    const bool small = a.B < kKeepCu;
    const bool ok = small ? offsets_kept(a.cu, a.B, a.T, sm.cu) : offsets_ok(a.cu, a.B, a.T);
    if (small) p.b.cu = sm.cu;
    if (blockIdx.x == 0 && threadIdx.x == 0)
      *a.status = ok ? CARVE_OK : CARVE_ERR_INVALID_ARG;
    if (!ok) {
      cp_async_wait<0>();
      return;
    }
    ask_states(a, p, a.h0);
    copy_empty(a, p, a.h0, a.h_T);
  } else if (a.status && blockIdx.x == 0 && threadIdx.x == 0) {
    *a.status = CARVE_OK;
  }

  start_exchange(sm.ex, p.ncl);
  bool dead = false;
  float2 carry = SEG ? make_float2(0.f, 0.f) : ld_state(a.h0, p.seq0, a.C, c);
  float* keep = a.keep ? a.keep + (int64_t)p.range * a.tiles * a.C : nullptr;
  Borders near{0, INT_MAX};
  Edge* const e = SEG ? &sm.edge[warp] : nullptr;

  for (int step = 0; step < steps; ++step) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();
    if (!F::LATE) fetch(step + STAGES - 1);
    const auto& st = sm.st[stage];
    stage = stage + 1 < STAGES ? stage + 1 : 0;
    const int first = (step * p.ncl + p.rank) * TILE, t0 = first + warp * S;
    const int nv = min(S, p.len - t0);  // tokens of this segment (may be < 0)
    const Kind kind = look<SEG, S, false>(p, near, t0, e);

    // the segment's own pair
    float2 da[S], u[S], A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
    bool reset = false;
    auto own = [&](auto marked) {
      constexpr bool M = decltype(marked)::value;
      const unsigned start = M ? e->m.start : 0u;
      // on its way while the pair is formed, which starts anew there
      const float2 first = M && start ? ld_state(a.h0, p.seq0 + e->first, a.C, c) : both(0.f);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, da[i], u[i]);
        if (M && (start >> i & 1)) A = both(1.f), H = both(0.f);
        H = fma2(da[i], H, u[i]);
        A = mul2(A, da[i]);
      }
      if (M && start) {
        reset = true;
        H = fma2(A, first, H);
        e->start[lane] = first;
        if (a.keep_h0 && ch_ok) st2(a.keep_h0 + (int64_t)(p.seq0 + e->first) * a.C + c, first);
      }
    };
    if (kind == kPlain) {
      own(std::false_type{});
    } else if (SEG && kind == kMarked) {
      own(std::true_type{});
    } else if (!SEG || kind == kRagged) {
#pragma unroll 1
      for (int i = 0; i < nv; ++i) {
        if (SEG && (e->m.start >> i & 1)) {
          const int64_t n = p.seq0 + seq_of(p.b, t0 + i);
          H = ld_state(a.h0, n, a.C, c);
          if (a.keep_h0 && ch_ok) st2(a.keep_h0 + n * a.C + c, H);
        }
        float2 d, v;
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, d, v);
        H = fma2(d, H, v);
        A = mul2(A, d);
      }
      reset = SEG && nv > 0 && e->m.start;
    }
    sm.pairs.A[warp][lane] = A;
    sm.pairs.H[warp][lane] = H;
    if (SEG && lane == 0) sm.pairs.reset[warp] = reset;
    __syncthreads();

    // the state before this segment: from the one before the tile, through
    // the segments before this one
    float2 h;
    if (F::LATE && (p.ncl == 1 || warp < kWarps - 1)) fetch(step + STAGES - 1);
    if (p.ncl > 1) {
      if (warp == kWarps - 1) {
        float2 tA, tH;
        total<SEG, false>(sm.pairs, tA, tH);
        sm.last[0][lane] =
            over_cluster<SEG, false>(sm.ex, a, step, p.rank, p.ncl, tA, tH, carry, dead);
        if (F::LATE) fetch(step + STAGES - 1);
      } else if (SEG) {
        ask_ahead<S>(a, p, near, t0 + p.ncl * TILE, a.h0, nullptr, c);
      }
      __syncthreads();
      h = sm.last[0][lane];
    } else {
      h = step ? sm.last[(step - 1) & 1][lane] : carry;
    }
    sm.pairs.template fold<SEG, false>(warp, h);
    if (keep && t0 % kKeep == 0 && nv > 0 && ch_ok)
      st2(keep + (int64_t)(t0 / kKeep) * a.C + c, h);

    char* tile = reinterpret_cast<char*>(h_out) + first * row_bytes;
    auto finish = [&](auto marked) {
      constexpr bool M = decltype(marked)::value;
      const unsigned start = M ? e->m.start : 0u, end = M ? e->m.end : 0u;
      const float2 s0 = M ? e->start[lane] : both(0.f);
      uint32_t off = out_off;
      float2 last = h;
#pragma unroll
      for (int i = 0; i < S; ++i, off += (uint32_t)row_bytes) {
        if (M && (start >> i & 1)) h = s0;
        h = fma2(da[i], h, u[i]);
        if (M && (end >> i & 1)) last = h;
        st2(reinterpret_cast<IO*>(tile + off), h);
      }
      if (M && end && a.h_T) st2(a.h_T + (int64_t)(p.seq0 + e->last) * a.C + c, last);
    };
    if (kind == kPlain) {
      if (ch_ok) finish(std::false_type{});
    } else if (SEG && kind == kMarked) {
      if (ch_ok) finish(std::true_type{});
    } else if (SEG && kind == kOutside) {
      uint32_t off = out_off;
      if (a.fill && ch_ok)
        for (int i = 0; i < nv; ++i, off += (uint32_t)row_bytes)
          st2(reinterpret_cast<IO*>(tile + off), both(0.f));
    } else {
      uint32_t off = out_off;
#pragma unroll 1
      for (int i = 0; i < nv; ++i, off += (uint32_t)row_bytes) {
        const int t = t0 + i;
        if (SEG && (e->m.start >> i & 1))
          h = ld_state(a.h0, p.seq0 + seq_of(p.b, t), a.C, c);
        float2 d, v;
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, d, v);
        h = fma2(d, h, v);
        const bool live = !SEG || (t >= e->m.lo && t < e->m.hi);
        if (ch_ok && (live || a.fill))
          st2(reinterpret_cast<IO*>(tile + off), live ? h : both(0.f));
        if (SEG && (e->m.end >> i & 1) && a.h_T) {
          const int64_t n = p.seq0 + seq_of(p.b, t);
          if (ch_ok) st2(a.h_T + n * a.C + c, h);
        }
      }
    }
    // the state after the tile (read after the next tile's first barriers)
    if (p.ncl == 1 && warp == kWarps - 1) sm.last[step & 1][lane] = carry = h;
  }
  if (!SEG && a.h_T && p.rank == 0 && warp == kWarps - 1 && ch_ok)
    st2(a.h_T + (int64_t)p.seq0 * a.C + c, carry);
  finish_exchange(sm.ex, a, steps, p.ncl, dead);
}

// --------------------------------------------------------------- backward
template <typename IO, bool SEG>
struct BwdTile {
  static constexpr int S = kKeep / kWarps;  // tokens of a warp
  static constexpr int TILE = kKeep;
  static constexpr int STAGES = sizeof(IO) == 2 ? 3 : 2;
  static constexpr bool LATE = sizeof(IO) == 4;  // as in the forward
  struct Stage {
    IO x[TILE * kCh], g[TILE * kCh], d[TILE * kCh];
    float keep[kCh];
  };
  struct Smem {
    Stage st[STAGES];
    Pairs<true> pairs;
    float2 last[2][32];  // by the parity of the step
    Exchange ex;
    Edge edge[SEG ? kWarps : 1];
    float2 end[SEG ? kWarps : 1][32];
    int32_t cu[SEG ? kKeepCu : 1];
  };
};

// The status word stays what the forward that filled the workspace has made
// it, unless this pass goes wrong too: its gradients come from kept states.
template <typename IO, bool SEG, bool ACT, bool COMP>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs a) {
  after_the_last();
  using F = BwdTile<IO, SEG>;
  static_assert(two_fit<typename F::Smem>() || (SEG && sizeof(IO) == 4),
                "shared memory of two blocks");
  constexpr int S = F::S, TILE = F::TILE, STAGES = F::STAGES;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sm = *reinterpret_cast<typename F::Smem*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Place p = place_of<SEG>(a);
  const int c = p.c0 + 2 * lane;
  const bool ch_ok = c < a.C;
  const Loader<IO, TILE> load_x(static_cast<const IO*>(a.x) + p.row0 * a.xp, a.xp, p.c0, a.C);
  const Loader<IO, TILE> load_g(static_cast<const IO*>(a.g) + p.row0 * a.gp, a.gp, p.c0, a.C);
  const Loader<IO, TILE> load_d(static_cast<const IO*>(a.d_h) + p.row0 * a.C, a.C, p.c0, a.C);
  IO* dx = static_cast<IO*>(a.dx) + p.row0 * a.C;
  IO* dg = static_cast<IO*>(a.dg) + p.row0 * a.C;
  const int64_t row_bytes = (int64_t)a.C * sizeof(IO);
  const uint32_t out_off = warp * S * (uint32_t)row_bytes + c * (uint32_t)sizeof(IO);
  const int tiles = (p.len + TILE - 1) / TILE;
  const float* keep = a.keep + (int64_t)p.range * a.tiles * a.C;

  const int steps = (tiles + p.ncl - 1) / p.ncl;
  int in_stage = 0, stage = 0;
  auto fetch = [&](int step) {  // steps run from the last tokens to the first
    const int tile = (steps - 1 - step) * p.ncl + p.rank;
    if (step < steps && tile < tiles) {
      const int t = tile * TILE;
      auto& st = sm.st[in_stage];
      load_x(st.x, t, p.len);
      load_g(st.g, t, p.len);
      load_d(st.d, t, p.len);
      const int ch = 4 * threadIdx.x;  // the kept state: 16 threads
      if (ch < kCh) {
        const bool ok = p.c0 + ch < a.C;
        cp_async16_zfill(st.keep + ch, ok ? keep + (int64_t)tile * a.C + p.c0 + ch : keep, ok);
      }
    }
    ptx::cp_async_commit();
    in_stage = in_stage + 1 < STAGES ? in_stage + 1 : 0;
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);

  if (SEG && a.cu) {
    const bool small = a.B < kKeepCu;
    const bool ok = small ? offsets_kept(a.cu, a.B, a.T, sm.cu) : offsets_ok(a.cu, a.B, a.T);
    if (small) p.b.cu = sm.cu;
    if (!ok) {
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = CARVE_ERR_INVALID_ARG;
      cp_async_wait<0>();
      return;
    }
    ask_states(a, p, a.keep_h0);
    ask_states(a, p, a.dh_T);
    copy_empty(a, p, a.dh_T, a.dh0);
  }

  start_exchange(sm.ex, p.ncl);
  bool dead = false;
  // the gradient that reaches the token before the tokens seen so far
  float2 carry = SEG ? make_float2(0.f, 0.f) : ld_state(a.dh_T, p.seq0, a.C, c);
  Borders near{0, INT_MAX};
  Edge* const e = SEG ? &sm.edge[warp] : nullptr;
  float2* const ends = SEG ? sm.end[warp] : nullptr;

  for (int step = 0; step < steps; ++step) {
    cp_async_wait<STAGES - 2>();
    __syncthreads();
    if (!F::LATE) fetch(step + STAGES - 1);
    const auto& st = sm.st[stage];
    stage = stage + 1 < STAGES ? stage + 1 : 0;
    const int first = ((steps - 1 - step) * p.ncl + p.rank) * TILE, t0 = first + warp * S;
    const int nv = min(S, p.len - t0);
    const Kind kind = look<SEG, S, true>(p, near, t0, e);
    const int at0 = warp * S * kCh + 2 * lane;

    // the segment's pairs, of the states (forwards) and of the gradients
    // (backwards: c_before = a (d + c_after))
    float2 da[S], rest[S], slope[S];
    float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f), R = H;
    unsigned start = 0, end = 0;
    auto own = [&](auto marked) {
      constexpr bool M = decltype(marked)::value;
      if (M) start = e->m.start, end = e->m.end;
      // on their way while the pairs are formed, which start anew there
      float2 h_in = both(0.f), r_in = both(0.f);
      if (M && start) h_in = ld_state(a.keep_h0, p.seq0 + e->first, a.C, c);
      if (M && end) r_in = ld_state(a.dh_T, p.seq0 + e->last, a.C, c);
#pragma unroll
      for (int i = 0; i < S; ++i) {
        gate<IO, ACT, COMP, ACT>(ld2(st.g + at0 + i * kCh), a.dscale, da[i], rest[i], slope[i]);
        float2 u = ld2(st.x + at0 + i * kCh);
        if (COMP) u = mul2(u, rest[i]);
        if (M && (start >> i & 1)) A = both(1.f), H = both(0.f);
        H = fma2(da[i], H, u);
        A = mul2(A, da[i]);
      }
      float2 back = both(1.f);  // the decays before the end
#pragma unroll
      for (int i = S - 1; i >= 0; --i) {
        if (M && (end >> i & 1)) back = both(1.f), R = both(0.f);
        R = mul2(da[i], add2(ld2(st.d + at0 + i * kCh), R));
        if (M) back = mul2(back, da[i]);
      }
      if (M && start) {
        H = fma2(A, h_in, H);
        e->start[lane] = h_in;
      }
      if (M && end) {
        R = fma2(back, r_in, R);
        ends[lane] = r_in;
      }
    };
    if (kind == kPlain) {
      own(std::false_type{});
    } else if (SEG && kind == kMarked) {
      own(std::true_type{});
    } else if (!SEG || kind == kRagged) {
      if (SEG && nv > 0) start = e->m.start, end = e->m.end;
#pragma unroll 1
      for (int i = 0; i < nv; ++i) {
        if (SEG && (start >> i & 1))
          H = ld_state(a.keep_h0, p.seq0 + seq_of(p.b, t0 + i), a.C, c);
        float2 f, v;
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, f, v);
        H = fma2(f, H, v);
        A = mul2(A, f);
      }
#pragma unroll 1
      for (int i = nv - 1; i >= 0; --i) {
        if (SEG && (end >> i & 1))
          R = ld_state(a.dh_T, p.seq0 + seq_of(p.b, t0 + i), a.C, c);
        float2 f, v;
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, f, v);
        R = mul2(f, add2(ld2(st.d + at0 + i * kCh), R));
      }
    }
    sm.pairs.A[warp][lane] = A;
    sm.pairs.H[warp][lane] = H;
    sm.pairs.R[warp][lane] = R;
    if (SEG && lane == 0) sm.pairs.reset[warp] = (start ? 1u : 0u) | (end ? 2u : 0u);
    __syncthreads();

    // the state before this segment: kept for the tile, folded over the
    // warps before this one
    float2 h = ld2(st.keep + 2 * lane);
    sm.pairs.template fold<SEG, false>(warp, h);
    // the gradient after it, from the one after the tile
    float2 r;
    if (F::LATE && (p.ncl == 1 || warp > 0)) fetch(step + STAGES - 1);
    if (p.ncl > 1) {
      if (warp == 0) {
        float2 tA, tR;
        total<SEG, true>(sm.pairs, tA, tR);
        sm.last[0][lane] =
            over_cluster<SEG, true>(sm.ex, a, step, p.rank, p.ncl, tA, tR, carry, dead);
        if (F::LATE) fetch(step + STAGES - 1);
      } else if (SEG) {
        ask_ahead<S>(a, p, near, t0 - p.ncl * TILE, a.keep_h0, a.dh_T, c);
      }
      __syncthreads();
      r = sm.last[0][lane];
    } else {
      r = step ? sm.last[(step - 1) & 1][lane] : carry;
    }
    sm.pairs.template fold<SEG, true>(warp, r);

    char* dx_tile = reinterpret_cast<char*>(dx) + first * row_bytes;
    char* dg_tile = reinterpret_cast<char*>(dg) + first * row_bytes;
    auto finish = [&](auto marked) {
      constexpr bool M = decltype(marked)::value;
      float2 hp[S];  // the state before each token (less its input: COMP)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const float2 xv = ld2(st.x + at0 + i * kCh);
        if (M && (start >> i & 1)) h = e->start[lane];
        hp[i] = COMP ? fma2(xv, both(-1.f), h) : h;
        h = fma2(da[i], h, COMP ? mul2(xv, rest[i]) : xv);
      }
      uint32_t off = out_off + (S - 1) * (uint32_t)row_bytes;
      float2 before = r;
#pragma unroll
      for (int i = S - 1; i >= 0; --i, off -= (uint32_t)row_bytes) {
        if (M && (end >> i & 1)) r = ends[lane];
        float2 ox = add2(ld2(st.d + at0 + i * kCh), r);
        r = mul2(da[i], ox);
        float2 og = mul2(r, hp[i]);
        if (COMP) ox = mul2(ox, rest[i]);
        if (ACT) og = mul2(og, slope[i]);
        if (M && (start >> i & 1)) before = r;
        st2(reinterpret_cast<IO*>(dx_tile + off), ox);
        st2(reinterpret_cast<IO*>(dg_tile + off), og);
      }
      if (M && start && a.dh0) st2(a.dh0 + (int64_t)(p.seq0 + e->first) * a.C + c, before);
    };
    if (kind == kPlain) {
      if (ch_ok) finish(std::false_type{});
    } else if (SEG && kind == kMarked) {
      if (ch_ok) finish(std::true_type{});
    } else if (SEG && kind == kOutside) {
      uint32_t off = out_off;
      if (a.fill && ch_ok)
        for (int i = 0; i < nv; ++i, off += (uint32_t)row_bytes) {
          st2(reinterpret_cast<IO*>(dx_tile + off), both(0.f));
          st2(reinterpret_cast<IO*>(dg_tile + off), both(0.f));
        }
    } else {
      float2 hp[S];
#pragma unroll 1
      for (int i = 0; i < nv; ++i) {
        if (SEG && (start >> i & 1))
          h = ld_state(a.keep_h0, p.seq0 + seq_of(p.b, t0 + i), a.C, c);
        hp[i] = h;
        float2 f, v;
        token<ACT, COMP>(st.x, st.g, at0 + i * kCh, a.dscale, f, v);
        h = fma2(f, h, v);
      }
#pragma unroll 1
      for (int i = nv - 1; i >= 0; --i) {
        const int t = t0 + i, at = at0 + i * kCh;
        if (SEG && (end >> i & 1))
          r = ld_state(a.dh_T, p.seq0 + seq_of(p.b, t), a.C, c);
        float2 f, k, sl;
        gate<IO, ACT, COMP, ACT>(ld2(st.g + at), a.dscale, f, k, sl);
        float2 ox = add2(ld2(st.d + at), r);
        r = mul2(f, ox);
        float2 og = mul2(r, COMP ? fma2(ld2(st.x + at), both(-1.f), hp[i]) : hp[i]);
        if (COMP) ox = mul2(ox, k);
        if (ACT) og = mul2(og, sl);
        const bool live = !SEG || (t >= e->m.lo && t < e->m.hi);
        if (ch_ok && (live || a.fill)) {
          if (!live) ox = og = both(0.f);
          const uint32_t off = out_off + i * (uint32_t)row_bytes;
          st2(reinterpret_cast<IO*>(dx_tile + off), ox);
          st2(reinterpret_cast<IO*>(dg_tile + off), og);
        }
        if (SEG && (start >> i & 1) && a.dh0) {
          const int64_t n = p.seq0 + seq_of(p.b, t);
          if (ch_ok) st2(a.dh0 + n * a.C + c, r);
        }
      }
    }
    // the gradient before the tile (read after the next tile's first barriers)
    if (p.ncl == 1 && warp == 0) sm.last[step & 1][lane] = carry = r;
  }
  if (!SEG && a.dh0 && p.rank == 0 && warp == 0 && ch_ok)
    st2(a.dh0 + (int64_t)p.seq0 * a.C + c, carry);
  finish_exchange(sm.ex, a, steps, p.ncl, dead);
}

// ------------------------------------------------------------------- step
// One token of each sequence: 2 channels a lane, one round of loads.  Its
// bytes take 0.04 us at 8 x 2048; what is left of 1.3 us in a graph is the
// launch and one trip to memory.
template <typename IO, bool ACT>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs a) {
  after_the_last();
  const int64_t i = 2 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x);
  if (i >= (int64_t)a.B * a.C) return;
  const int64_t b = i / a.C;
  const int c = (int)(i - b * a.C);
  const float2 gv = ld2(static_cast<const IO*>(a.g) + b * a.gp + c);
  float2 u = ld2(static_cast<const IO*>(a.x) + b * a.xp + c);
  float2 h = ld2(a.h_T + i), e, rest, slope;
  gate<IO, ACT, true, false>(gv, a.dscale, e, rest, slope);
  if (a.comp) u = mul2(u, rest);
  h = fma2(e, h, u);
  st2(a.h_T + i, h);
  st2(static_cast<IO*>(a.h) + i, h);
}

// ------------------------------------------------------------------- host
carve_status check_scan(const carve_scan_shape* s) {
  if (!s) return CARVE_ERR_INVALID_ARG;
  if (s->B < 1 || s->T < 0 || s->C < 1 || s->reserved != 0 ||
      !dtype_ok(s->dtype) || !flag_ok(s->complement) || !flag_ok(s->fill_rest))
    return CARVE_ERR_INVALID_ARG;
  if (!(s->decay_scale >= 0.f) || s->decay_scale > 3.0e38f)
    return CARVE_ERR_INVALID_ARG;
  if (!pitch_ok(s->x_pitch, s->C) || !pitch_ok(s->g_pitch, s->C))
    return CARVE_ERR_INVALID_ARG;
  if (s->C % 8 || s->C > kMaxPitch || s->x_pitch > kMaxPitch ||
      s->g_pitch > kMaxPitch)
    return CARVE_ERR_UNSUPPORTED;
  return CARVE_OK;
}

// How a call is cut up: ranges of tokens that do not depend on one another,
// and whether sequences start inside a range.
struct ScanPlan {
  bool seg;
  int ranges, seqs, groups, tiles;  // tiles: kept states of one range
};
bool plan_scan(const carve_scan_shape& s, bool packed, ScanPlan* p) {
  const int64_t tokens = packed ? s.T : (int64_t)s.B * s.T;
  if (tokens > kMaxTokens) return false;
  p->groups = (s.C + kCh - 1) / kCh;
  p->seg = packed;
  p->ranges = packed ? 1 : s.B;
  p->seqs = 1;
  int64_t len = s.T;
  if (!packed && s.T > 0 && s.T < kKeep && s.B > 1) {
    // short sequences share tiles: as many in a range as keeps two blocks
    // on every SM busy, and a full tile at least (a range for each sequence
    // leaves most of a tile empty: 64 x 33 x 2048 takes 10.3 us forward and
    // 16.0 backward this way, 15.0 and 16.5 that way; 64 x 63 x 2048 18.4 and
    // 24.9 against 25.6 and 29.9; from 64 tokens on the borders inside tiles
    // cost what they save, 64 x 100 x 2048 20 and 37 against 22 and 38)
    const int64_t want = (2 * sm_count() + p->groups - 1) / p->groups;
    int64_t n = (s.B + want - 1) / want;
    n = n > (kKeep + s.T - 1) / s.T ? n : (kKeep + s.T - 1) / s.T;
    n = n < s.B ? n : s.B;
    p->seg = true;
    p->seqs = (int)n;
    p->ranges = (int)((s.B + n - 1) / n);
    len = n * s.T;
  }
  p->tiles = (int)((len + kKeep - 1) / kKeep);
  return (int64_t)p->ranges * p->groups * kMaxCluster < (1LL << 31);
}

struct ScanWs {
  size_t keep, keep_h0, total;
};
ScanWs scan_ws(const carve_scan_shape& s, const ScanPlan& p, bool training) {
  ScanWs w{};
  w.keep = kHeaderBytes;
  w.keep_h0 = align256(w.keep + (size_t)p.ranges * p.tiles * s.C * 4);
  w.total = !training ? kHeaderBytes
                      : align256(w.keep_h0 + (p.seg ? (size_t)s.B * s.C * 4 : 0));
  return w;
}

// Clusters of n blocks that the device holds at once, two blocks an SM: fewer
// than the SMs would take, as a cluster stays within a group of SMs.  Each
// device is asked once.  The answer decides the size of the clusters, and that
// the rounding: alone, a block carries the state it has walked from tile to
// tile; in a cluster it is A h + H of whole tiles.
template <auto kernel>
int clusters_held(int n, size_t smem) {
  static std::atomic<int> held[kDevices][kMaxCluster + 1];
  const int dev = kept_device();
  int v = dev >= 0 ? held[dev][n].load() : 0;
  if (v > 0) return v;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  cluster_config(&cfg, at, dim3(n * 64), kThreads, smem, n);
  if (allow_smem<kernel>(smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&v, kernel, &cfg) != cudaSuccess || v < 1) {
    cudaGetLastError();
    return 2 * sm_count() / n;  // this call's guess, not kept
  }
  if (dev >= 0) held[dev][n].store(v);
  return v;
}

// Blocks of a cluster share a range's tokens: as many as the device still
// holds all clusters of at once, and no more than shorten the walk.  Forward
// and backward in us with 1, 2, 4, 8 blocks: 8 x 4096 x 2048 (takes 1) 68 and
// 117, 81 and 136, 87 and 142, 103 and 163; 2 x 4096 x 2048 (takes 4) 42 and
// 79, 28 and 50, 24 and 39, 29 and 44; 1 x 65536 x 2048 (takes 8) 618 and
// 1213, 398 and 735, 204 and 372, 169 and 283.  With 4, 5, 6, 7, 8:
// 1 x 8192 x 2560 (takes 6) 42 and 69, 37 and 58, 34 and 51, 47 and 74, 43
// and 70.
template <auto kernel>
int cluster_size(const ScanPlan& p, int tile, size_t smem) {
  const int64_t chains = (int64_t)p.ranges * p.groups;
  const int64_t tiles = ((int64_t)p.tiles * kKeep + tile - 1) / tile;
  int n = 1;
  for (int k = 2; k <= kMaxCluster && k <= tiles && chains * k <= 2 * sm_count(); ++k)
    if (chains <= clusters_held<kernel>(k, smem)) n = k;
  const int64_t steps = (tiles + n - 1) / n;
  return steps ? (int)((tiles + steps - 1) / steps) : 1;
}

template <typename IO, bool SEG, bool ACT>
cudaError_t run_fwd_act(const ScanArgs& a, int64_t blocks, int ncl, cudaStream_t st) {
  const size_t smem = sizeof(typename FwdTile<IO, SEG>::Smem);
  return a.comp ? launch<scan_fwd_kernel<IO, SEG, ACT, true>>(a, dim3((unsigned)blocks), kThreads, smem, st, ncl)
                : launch<scan_fwd_kernel<IO, SEG, ACT, false>>(a, dim3((unsigned)blocks), kThreads, smem, st, ncl);
}
template <typename IO, bool SEG>
cudaError_t run_fwd(const ScanArgs& a, const ScanPlan& p, cudaStream_t st) {
  const int ncl = cluster_size<scan_fwd_kernel<IO, SEG, false, false>>(
      p, FwdTile<IO, SEG>::TILE, sizeof(typename FwdTile<IO, SEG>::Smem));
  const int64_t blocks = (int64_t)p.ranges * p.groups * ncl;
  return a.dscale > 0.f ? run_fwd_act<IO, SEG, true>(a, blocks, ncl, st)
                        : run_fwd_act<IO, SEG, false>(a, blocks, ncl, st);
}
template <typename IO, bool SEG, bool ACT>
cudaError_t run_bwd_act(const ScanArgs& a, int64_t blocks, int ncl, cudaStream_t st) {
  const size_t smem = sizeof(typename BwdTile<IO, SEG>::Smem);
  return a.comp ? launch<scan_bwd_kernel<IO, SEG, ACT, true>>(a, dim3((unsigned)blocks), kThreads, smem, st, ncl)
                : launch<scan_bwd_kernel<IO, SEG, ACT, false>>(a, dim3((unsigned)blocks), kThreads, smem, st, ncl);
}
template <typename IO, bool SEG>
cudaError_t run_bwd(const ScanArgs& a, const ScanPlan& p, cudaStream_t st) {
  const int ncl = cluster_size<scan_bwd_kernel<IO, SEG, false, false>>(
      p, BwdTile<IO, SEG>::TILE, sizeof(typename BwdTile<IO, SEG>::Smem));
  const int64_t blocks = (int64_t)p.ranges * p.groups * ncl;
  return a.dscale > 0.f ? run_bwd_act<IO, SEG, true>(a, blocks, ncl, st)
                        : run_bwd_act<IO, SEG, false>(a, blocks, ncl, st);
}

ScanArgs scan_args(const carve_scan_shape& s, const ScanPlan& p) {
  ScanArgs a{};
  a.B = s.B; a.T = s.T; a.C = s.C; a.comp = s.complement; a.fill = s.fill_rest;
  a.dscale = s.decay_scale;
  a.xp = s.x_pitch ? s.x_pitch : s.C;
  a.gp = s.g_pitch ? s.g_pitch : s.C;
  a.ranges = p.ranges; a.seqs = p.seqs; a.groups = p.groups; a.tiles = p.tiles;
  test_knobs(&a.spin, &a.stall);
  return a;
}

}  // namespace
}  // namespace mix
}  // namespace carve

using namespace carve;
using namespace carve::mix;

extern "C" {

size_t carve_scan_workspace_bytes(const carve_scan_shape* shape, int packed,
                                  int training) {
  ScanPlan p;
  if (check_scan(shape) != CARVE_OK || !plan_scan(*shape, packed != 0, &p))
    return 0;
  return scan_ws(*shape, p, training != 0).total;
}

carve_status carve_scan_fwd(const carve_scan_shape* shape,
                            const int32_t* cu_seqlens, const void* x,
                            const void* g, const float* h0, void* h,
                            float* h_T, void* workspace,
                            size_t workspace_bytes, int training,
                            void* stream) {
  carve_status st = check_scan(shape);
  if (st != CARVE_OK) return st;
  const carve_scan_shape& s = *shape;
  ScanPlan p;
  if (!plan_scan(s, cu_seqlens != nullptr, &p)) return CARVE_ERR_UNSUPPORTED;
  if (s.T > 0 && (!ptr_ok(x) || !ptr_ok(g) || !ptr_ok(h)))
    return CARVE_ERR_INVALID_ARG;
  if (!opt_ptr_ok(cu_seqlens) || !opt_ptr_ok(h0) || !opt_ptr_ok(h_T))
    return CARVE_ERR_INVALID_ARG;
  const ScanWs w = scan_ws(s, p, training != 0);
  if (training || cu_seqlens) {
    if (!workspace || !aligned16(workspace) || workspace_bytes < w.total)
      return CARVE_ERR_WORKSPACE;
  }
  ScanArgs a = scan_args(s, p);
  a.x = x; a.g = g; a.h0 = h0; a.h = h; a.h_T = h_T; a.cu = cu_seqlens;
  a.status = status_word(workspace, workspace_bytes);
  if (training) {
    a.keep = (float*)((char*)workspace + w.keep);
    a.keep_h0 = p.seg ? (float*)((char*)workspace + w.keep_h0) : nullptr;
  }
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e;
  if (s.dtype == CARVE_BF16)
    e = p.seg ? run_fwd<__nv_bfloat16, true>(a, p, cs)
              : run_fwd<__nv_bfloat16, false>(a, p, cs);
  else
    e = p.seg ? run_fwd<float, true>(a, p, cs) : run_fwd<float, false>(a, p, cs);
  return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA;
}

carve_status carve_scan_bwd(const carve_scan_shape* shape,
                            const int32_t* cu_seqlens, const void* x,
                            const void* g, const void* d_h,
                            const float* dh_T, void* workspace,
                            size_t workspace_bytes, void* dx, void* dg,
                            float* dh0, void* stream) {
  carve_status st = check_scan(shape);
  if (st != CARVE_OK) return st;
  const carve_scan_shape& s = *shape;
  ScanPlan p;
  if (!plan_scan(s, cu_seqlens != nullptr, &p)) return CARVE_ERR_UNSUPPORTED;
  if (s.T > 0 && (!ptr_ok(x) || !ptr_ok(g) || !ptr_ok(d_h) || !ptr_ok(dx) ||
                  !ptr_ok(dg)))
    return CARVE_ERR_INVALID_ARG;
  if (!opt_ptr_ok(cu_seqlens) || !opt_ptr_ok(dh_T) || !opt_ptr_ok(dh0))
    return CARVE_ERR_INVALID_ARG;
  const ScanWs w = scan_ws(s, p, true);
  if (!workspace || !aligned16(workspace) || workspace_bytes < w.total)
    return CARVE_ERR_WORKSPACE;
  ScanArgs a = scan_args(s, p);
  a.x = x; a.g = g; a.d_h = d_h; a.dh_T = dh_T; a.dx = dx; a.dg = dg;
  a.dh0 = dh0; a.cu = cu_seqlens;
  a.status = static_cast<uint32_t*>(workspace);
  a.keep = (float*)((char*)workspace + w.keep);
  a.keep_h0 = p.seg ? (float*)((char*)workspace + w.keep_h0) : nullptr;
  cudaStream_t cs = (cudaStream_t)stream;
  cudaError_t e;
  if (s.dtype == CARVE_BF16)
    e = p.seg ? run_bwd<__nv_bfloat16, true>(a, p, cs)
              : run_bwd<__nv_bfloat16, false>(a, p, cs);
  else
    e = p.seg ? run_bwd<float, true>(a, p, cs) : run_bwd<float, false>(a, p, cs);
  return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA;
}

carve_status carve_scan_step(const carve_scan_shape* shape, const void* x,
                             const void* g, float* h, void* o, void* stream) {
  carve_status st = check_scan(shape);
  if (st != CARVE_OK) return st;
  const carve_scan_shape& s = *shape;
  if (!ptr_ok(x) || !ptr_ok(g) || !ptr_ok(h) || !ptr_ok(o))
    return CARVE_ERR_INVALID_ARG;
  ScanArgs a{};
  a.B = s.B; a.C = s.C; a.comp = s.complement; a.dscale = s.decay_scale;
  a.xp = s.x_pitch ? s.x_pitch : s.C;
  a.gp = s.g_pitch ? s.g_pitch : s.C;
  a.x = x; a.g = g; a.h_T = h; a.h = o;
  const int64_t blocks = ((int64_t)s.B * s.C / 2 + 127) / 128;
  if (blocks >= (1LL << 31)) return CARVE_ERR_UNSUPPORTED;
  const cudaStream_t cs = (cudaStream_t)stream;
  const dim3 grid((unsigned)blocks);
  const bool act = s.decay_scale > 0.f;
  cudaError_t e;
  if (s.dtype == CARVE_BF16)
    e = act ? launch<scan_step_kernel<__nv_bfloat16, true>>(a, grid, 128, 0, cs)
            : launch<scan_step_kernel<__nv_bfloat16, false>>(a, grid, 128, 0, cs);
  else
    e = act ? launch<scan_step_kernel<float, true>>(a, grid, 128, 0, cs)
            : launch<scan_step_kernel<float, false>>(a, grid, 128, 0, cs);
  return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA;
}

}  // extern "C"

// gated_scan.cuh -- the gated linear recurrence and its backward pass.
//
//   s = sigmoid(r), g = sigmoid(i), l = -decay * s, a = e^l, m = sqrt(1 - a^2)
//   h[t] = a h[t-1] + m g x[t]
//
// The gates.  Where a is next to 1 (a state that lives for thousands of
// tokens) both a and 1 - a^2 lose their digits if taken from a rounded
// exponential, and a's rounding is raised to the power of the lifetime.  So
// E = 1 - a is computed by the exponential's own series while |l| < 1/4, and
// a = 1 - E is then rounded once; 1 - a^2 = E (2 - E) keeps E's digits.
//
// The backward pass, with G[t] the whole gradient of h[t]:
//   G[t] = dy[t] + a[t+1] G[t+1]          (+ dh_last at the last token)
//   dx = G m g,  di = G m x g (1 - g)
//   dl = a G (h[t-1] - a g x / m)         (the second term 0 where m = 0)
//   dr = -decay dl s (1 - s),  ddecay = -sum s dl,  dh0 = a[0] G[0]
#pragma once

#include <cmath>

#include "ptx.cuh"
#include "seq_tile.cuh"

namespace convfwd {

// Constants of the gates, as pairs for packed instructions: kernel parameters,
// so that they are operands of an instruction (an immediate pair is not: it
// costs two moves each time).
struct GateConsts {
  float2 nlog2e, one, nhalf, p3, p4, p5, p6, two, none, unit;
};
inline GateConsts gate_consts() {
  const auto two = [](float v) { return make_float2(v, v); };
  return GateConsts{two(-kLog2e),        two(1.f),           two(-0.5f), two(1.f / 6.f), two(-1.f / 24.f),
                    two(1.f / 120.f), two(-1.f / 720.f), two(2.f),   two(-1.f),      two(0x1p-124f)};
}
template <int V>
__device__ __forceinline__ Vf<V> both(const float2& c) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = k & 1 ? c.y : c.x;
  return o;
}

// In the forward pass of 16-bit types the two sigmoids share a reciprocal: the
// special functions, 16 a clock and SM, are its first limit, and this leaves 5 of
// them an element (with 6, 65536 x 2048 bf16 takes 381 us in place of 359).  With
// E_r = 1 + e^-r and E_i = 2^-124 (1 + e^-i) the product E_r E_i is a normal number
// unless both gates are below 2^-124 (where both then are 0), so s = E_i / (E_r E_i)
// and g = 2^-124 E_r / (E_r E_i) are right down to fp32's least normal number, at r
// or i = -87.3.  Below, at -infinity too, they are 0: r and i stop at -87.5, and the
// last product takes what is subnormal as 0.  A NaN in either gate makes both NaN,
// as it makes u = m g x and every state behind it.
//
// Elsewhere each has a reciprocal of its own, whose flush of subnormal results
// closes the gates at the same place: in the backward pass, where a NaN in i leaves
// a, and through it the gradients of earlier tokens, as they are; for fp32, whose
// bytes take longer than six special functions (4 x 4096 x 2560: 133 us, with a
// shared one 136); and for single tokens, which wait for the memory.
constexpr float kGateLowest = -87.5f;  // exact in each type; e^87.5 is finite

// a b, with subnormal results as 0
__device__ __forceinline__ Vf<2> mul_ftz(const Vf<2>& a, const Vf<2>& b) {
  uint64_t d;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(a.v)), "l"(pack2(b.v)));
  Vf<2> o;
  unpack2(d, o.v);
  return o;
}

// Where 1 - a^2 is less (decay s under 6e-39), the approximate roots take it as 0: m
// is 0 in the forward pass, and in the backward pass, whose 1 / m would be infinite.
constexpr float kLeastNormal = 0x1p-126f;

template <int V>
struct GateValues {
  Vf<V> s, g, a, m;
};

// SHARED (V = 2): one reciprocal, r and i at least kGateLowest.  ROOT: m = sqrt(1 - a^2),
// else 1 - a^2.
template <int V, bool SHARED, bool ROOT>
__device__ __forceinline__ GateValues<V> gate_values(const GateConsts& c, const Vf<V>& r, const Vf<V>& i,
                                                     const Vf<V>& decay) {
  GateValues<V> o;
  const Vf<V> one = both<V>(c.one), none = both<V>(c.none);
  Vf<V> er = mul_v(r, both<V>(c.nlog2e)), ei = mul_v(i, both<V>(c.nlog2e));
#pragma unroll
  for (int k = 0; k < V; ++k) er[k] = ex2_approx(er[k]), ei[k] = ex2_approx(ei[k]);
  er = add_v(er, one);
  if constexpr (SHARED) {
    const Vf<V> unit = both<V>(c.unit);
    ei = fma_v(ei, unit, unit);
    Vf<V> inv = mul_v(er, ei);
#pragma unroll
    for (int k = 0; k < V; ++k) inv[k] = rcp_approx(inv[k]);
    o.s = mul_ftz(inv, ei);
    o.g = mul_ftz(mul_v(inv, er), unit);
  } else {
    ei = add_v(ei, one);
#pragma unroll
    for (int k = 0; k < V; ++k) o.s[k] = rcp_approx(er[k]), o.g[k] = rcp_approx(ei[k]);
  }
  const Vf<V> w = mul_v(decay, o.s);  // -l
  // 1 - e^-w = w (1 - w/2 + w^2/6 - w^3/24 + w^4/120 - w^5/720); the next term
  // is w^6/5040 < 5e-8 of it for w < 1/4
  Vf<V> p = fma_v(w, both<V>(c.p6), both<V>(c.p5));
  p = fma_v(w, p, both<V>(c.p4));
  p = fma_v(w, p, both<V>(c.p3));
  p = fma_v(w, p, both<V>(c.nhalf));
  p = fma_v(w, p, one);
  Vf<V> E = mul_v(w, p), far = mul_v(w, both<V>(c.nlog2e));
#pragma unroll
  for (int k = 0; k < V; ++k) far[k] = ex2_approx(far[k]);
  const Vf<V> near_a = fma_v(E, none, one), far_E = fma_v(far, none, one);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const bool near1 = w[k] < 0.25f;
    E[k] = near1 ? E[k] : far_E[k];
    o.a[k] = near1 ? near_a[k] : far[k];
  }
  o.m = mul_v(E, fma_v(E, none, both<V>(c.two)));
  if constexpr (ROOT) {
#pragma unroll
    for (int k = 0; k < V; ++k) o.m[k] = sqrt_approx(o.m[k]);
  }
  return o;
}
template <int V>
__device__ __forceinline__ Vf<V> gated_input(const GateValues<V>& v, const Vf<V>& m, const Vf<V>& x) {
  return mul_v(mul_v(m, v.g), x);
}

// Two gates of a 16-bit type as they are in memory, at least kGateLowest (NaN stays).
template <typename T>
__device__ __forceinline__ Vf<2> gate_input(uint32_t w) {
  const float2 lowest = make_float2(kGateLowest, kGateLowest);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 l = __float22half2_rn(lowest);
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(w) : "r"(*reinterpret_cast<const uint32_t*>(&l)));
  } else {
    const __nv_bfloat162 l = __float22bfloat162_rn(lowest);
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(*reinterpret_cast<const uint32_t*>(&l)));
  }
  Vf<2> o;
  unpack<T, 2>(w, o.v);
  return o;
}

struct ScanArgs {
  SeqIn x, r, i, dy;
  const float *decay, *h0, *dh_last;
  const int* cu;
  void *y, *dx, *dr, *di;
  float *h_last, *states, *dh0, *part;
  const float* states_in;
  int N, C, packed, fill;
  long long L;
  GateConsts consts;
};

// ---- one pass over time --------------------------------------------------
//
// A warp owns 64 neighbouring channels, two a lane, and a few tokens in a row; a
// CTA is kScanWarps warps, one behind the other in time; a cluster is up to eight
// CTAs one behind the other, and walks along a sequence in turns of as many tokens
// as it holds.  A segment of tokens is the map
// h -> P h + H (P the product of its a's, H its own end state), so per turn the
// warps leave (P, H) in shared memory, the CTAs' maps go to every CTA of the
// cluster through distributed shared memory, and once they are there every
// thread knows the state in front of its own tokens.  The inputs are read once
// and the outputs written once, and the order of the sums is fixed.  The
// backward pass is the same walk from the end.
//
// A map that begins a sequence takes nothing from in front of it: P = -1 marks
// it, and is tested rather than multiplied with, so that no NaN of one sequence
// reaches the next.
constexpr int kScanWarps = 8;
constexpr int kScanThreads = 32 * kScanWarps;
constexpr int kScanSteps = 8;
constexpr int kScanMaxCluster = 8;
static_assert(kScanWarps * kScanSteps == GATED_SCAN_STATE_EVERY, "a CTA's tokens begin at a kept state");

template <int V>
struct alignas(8 * V) ScanMap {
  Vf<V> P, H;
};
template <int V>
__device__ __forceinline__ ScanMap<V> no_map() {
  return ScanMap<V>{splat<V>(1.f), splat<V>(0.f)};
}

// h behind the map f.
template <bool PACKED, int V>
__device__ __forceinline__ Vf<V> follow(const ScanMap<V>& f, const Vf<V>& h) {
  Vf<V> o = fma_v(f.P, h, f.H);
  if (PACKED) {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = f.P[k] < 0.f ? f.H[k] : o[k];
  }
  return o;
}
// f, then g
template <bool PACKED, int V>
__device__ __forceinline__ ScanMap<V> then(const ScanMap<V>& f, const ScanMap<V>& g) {
  ScanMap<V> o;
  o.H = follow<PACKED>(g, f.H);
  o.P = mul_v(f.P, g.P);
  if (PACKED) {
#pragma unroll
    for (int k = 0; k < V; ++k) o.P[k] = f.P[k] < 0.f || g.P[k] < 0.f ? -1.f : o.P[k];
  }
  return o;
}
// f, then a token: h -> a h + u
template <bool PACKED, int V>
__device__ __forceinline__ void then_token(ScanMap<V>& f, const Vf<V>& a, const Vf<V>& u) {
  const Vf<V> P = mul_v(f.P, a);
  f.H = fma_v(a, f.H, u);
#pragma unroll
  for (int k = 0; k < V; ++k) f.P[k] = PACKED && f.P[k] < 0.f ? -1.f : P[k];
}

constexpr unsigned kScanAll = (1u << kScanSteps) - 1;

// What the tokens t0 .. t0 + STEPS - 1 are: bit j of `used` where token
// t0 + j is in a sequence, of `first` and `last` where it begins or ends one;
// lane j holds its sequence in `seq`.  Called by whole warps.
struct ScanTokens {
  unsigned used, first, last;
  int seq;
};

template <int STEPS, bool PACKED>
__device__ __forceinline__ ScanTokens scan_tokens(const ScanArgs& a, long long t0) {
  ScanTokens k = {0, 0, 0, 0};
  if constexpr (PACKED) {
    const int lane = threadIdx.x & 31;
    const long long t = t0 + lane;
    bool used = false, first = false, last = false;
    if (lane < STEPS && t >= 0 && t < a.L) {
      k.seq = seq_of_row(a.cu, a.N, t);
      if (k.seq < a.N) {
        used = true;
        first = t == 0 || __ldg(a.cu + k.seq) == t;
        last = __ldg(a.cu + k.seq + 1) == t + 1 || t + 1 == a.L;
      }
    }
    k.used = __ballot_sync(0xffffffffu, used);
    k.first = __ballot_sync(0xffffffffu, first);
    k.last = __ballot_sync(0xffffffffu, last);
  } else {
    const long long left = t0 < 0 ? 0 : a.L - t0;
    k.used = left >= STEPS ? (1u << STEPS) - 1 : left > 0 ? (1u << left) - 1 : 0;
  }
  return k;
}

// Channels c .. c + width - 1 (V at most) of row s of [rows, C] states; zeros
// without them.
template <int V>
__device__ __forceinline__ Vf<V> scan_initial(const float* h0, long long s, int C, int c, int width) {
  Vf<V> h;
#pragma unroll
  for (int k = 0; k < V; ++k) h[k] = h0 && k < width ? __ldg(h0 + s * C + c + k) : 0.f;
  return h;
}
// The decays of channels c .. c + width - 1.  An infinite one counts as the largest
// number: a is 0 all the same, and infinity times a closed gate, of which tokens
// that are not there are made, would be NaN.
template <int V>
__device__ __forceinline__ Vf<V> load_decay(const float* decay, int c, int width) {
  Vf<V> d = scan_initial<V>(decay, 0, 0, c, width);
#pragma unroll
  for (int k = 0; k < V; ++k) d[k] = min_nan(d[k], 0x1.fffffep127f);
  return d;
}
template <int V>
__device__ __forceinline__ void put_state(float* h, long long s, int C, int c, int width, const Vf<V>& v) {
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (k < width) h[s * C + c + k] = v[k];
}
// What sequences without a token pass on: `from` (or zeros) into `to`.
template <int V>
__device__ __forceinline__ void pass_empty(const ScanArgs& a, const float* from, float* to, int first, int step, int c,
                                           int width) {
  if (width <= 0 || !to) return;
  for (int s = first; s < a.N; s += step)
    if (__ldg(a.cu + s) >= __ldg(a.cu + s + 1))
      put_state<V>(to, s, a.C, c, width, scan_initial<V>(from, s, a.C, c, width));
}

// The maps of a turn: the CTA's warps', and one of each CTA of the cluster.
// Two of each, for a warp may be a turn ahead of another.
template <int V>
struct ScanShared {
  ScanMap<V> warp[2][kScanWarps][32];
  ScanMap<V> cta[2][kScanMaxCluster][32];
};

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The cluster's barrier in two halves.  The warp that wrote to other CTAs arrives
// with `wrote`, a release; that waits for all of the thread's accesses, its loads
// among them, so the other warps arrive without.
__device__ __forceinline__ void cluster_arrive(bool wrote) {
  if (wrote) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Stores a map to the same place in CTA `rank`'s shared memory.
template <int V>
__device__ __forceinline__ void store_remote(ScanMap<V>* p, int rank, const ScanMap<V>& m) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
  if constexpr (V == 2)
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(m.P[0]), "f"(m.P[1]), "f"(m.H[0]),
                 "f"(m.H[1])
                 : "memory");
  else
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(m.P[0]), "f"(m.H[0]) : "memory");
}

// Takes each warp's map of this turn (`mine`) and the state in front of the
// cluster's turn (`carry`); gives the state in front of the warp's own tokens
// and moves `carry` behind the turn.  b: the turn's parity.  `order` is the
// warp's place in time among the CTA's (0 first), `rank` the CTA's among the
// cluster's.  Every thread of the cluster calls it; inactive channels take part
// with whatever they hold.  `load` loads the next turn's rows: before the
// exchange, but in the warp that writes to the other CTAs only behind its
// release.
template <bool PACKED, int V, typename Load>
__device__ __forceinline__ Vf<V> scan_exchange(ScanShared<V>& sh, int b, int order, int rank, int ctas,
                                               const ScanMap<V>& mine, Vf<V>& carry, Load&& load) {
  const int lane = threadIdx.x & 31;
  const bool writer = ctas > 1 && order == kScanWarps - 1;
  Vf<V> before;
  sh.warp[b][order][lane] = mine;
  if (!writer) load();
  __syncthreads();
  ScanMap<V> front = no_map<V>();  // the CTA's warps in front of this one
#pragma unroll
  for (int w = 0; w < kScanWarps - 1; ++w)
    if (w < order) front = then<PACKED>(front, sh.warp[b][w][lane]);
  if (ctas > 1) {
    if (writer) {
      const ScanMap<V> all = then<PACKED>(front, mine);
      for (int r = 0; r < ctas; ++r) store_remote<V>(&sh.cta[b][rank][lane], r, all);
      cluster_arrive(true);
      load();
    } else {
      cluster_arrive(false);
    }
    cluster_wait();
    before = carry;
#pragma unroll
    for (int r = 0; r < kScanMaxCluster; ++r)
      if (r < ctas) {
        carry = follow<PACKED>(sh.cta[b][r][lane], carry);
        if (r < rank) before = carry;
      }
    before = follow<PACKED>(front, before);
  } else {
    before = follow<PACKED>(front, carry);
    ScanMap<V> all = no_map<V>();
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) all = then<PACKED>(all, sh.warp[b][w][lane]);
    carry = follow<PACKED>(all, carry);
  }
  return before;
}

// The forward pass.  Bounds: 8 bytes an element of a 16-bit type, and five
// special functions (40 of an SM quarter's cycles for 32 elements, where the
// bytes take 44).  Measured: 65536 x 2048 bf16 in 359 us, 2.99 TB/s (46 % of the
// copy rate), 4 x 4096 x 2560 bf16 in 108 us, fp32 in 133 (5.0 TB/s); without
// its loads or its stores it takes as long, so what bounds it is the issue of
// some 41 instructions an element at 16 warps an SM and the exchange of a turn.
// Tokens of a warp: the maps of a turn cost as much however many there are, but
// a and u of each stay in registers.  16 tokens and 2 CTAs an SM: 364 us; 8
// tokens and 3 or 4 CTAs: 420, 524; 4 or 16 warps a CTA: 416, 539; computing the
// next turn's gates during the exchange (two turns in registers, 8 tokens): 394,
// with a warp of its own for the exchange 484.
constexpr int kForwardSteps = 16;

template <typename T>
struct ForwardShared {
  ScanShared<2> maps;
  struct {
    RowTile<T, kForwardSteps> x, r, i;
  } warp[kScanWarps];
};

template <typename T, bool PACKED, bool ALIGNED>
__global__ void __launch_bounds__(kScanThreads, 2) gated_scan_kernel(const __grid_constant__ ScanArgs a) {
  constexpr int STEPS = kForwardSteps, V = 2;
  constexpr unsigned kAll = (1u << STEPS) - 1;
  extern __shared__ __align__(128) unsigned char smem[];
  ForwardShared<T>& sh = *reinterpret_cast<ForwardShared<T>*>(smem);
  ptx::pdl_wait_prev();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = cluster_rank(), ctas = cluster_size();
  const int c0 = static_cast<int>(blockIdx.x / ctas) * 64, c = c0 + lane * V, L = static_cast<int>(a.L);
  const int n = static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y);
  if (!PACKED && n >= a.N) return;  // all of the cluster
  // with rows that are not aligned C may be odd: the last channel stands alone
  const int width = min(V, a.C - c), there = a.C - c0;
  const bool in = width > 0;
  auto& tile = sh.warp[warp];
  const Vf<V> decay = load_decay<V>(a.decay, c, width);
  Vf<V> carry = PACKED ? splat<V>(0.f) : scan_initial<V>(a.h0, n, a.C, c, width);
  if (PACKED) pass_empty<V>(a, a.h0, a.h_last, rank * kScanWarps + warp, ctas * kScanWarps, c, width);
  if (ctas > 1) cluster_arrive(false), cluster_wait();  // every CTA runs before another writes to its shared memory
  const int span = ctas * kScanWarps * STEPS;
  const int turns = static_cast<int>((a.L + span - 1) / span);
  int left = L - (rank * kScanWarps + warp) * STEPS;  // rows from the warp's first of this turn to the end
  TileWalk<T, STEPS, ALIGNED> x, r, i;
  r.start(a.r, n, L - left, c0);
  i.start(a.i, n, L - left, c0);
  x.start(a.x, n, L - left, c0);
  r.load(tile.r, left, there);
  i.load(tile.i, left, there);
  x.load(tile.x, left, there);
  T* y = static_cast<T*>(a.y) + (n * a.L + L - left) * a.C + c;
  for (int turn = 0; turn < turns; ++turn, left -= span, y += static_cast<long long>(span) * a.C) {
    const ScanTokens tok = scan_tokens<STEPS, PACKED>(a, L - left);
    copies_done();
    if (tok.used != kAll) {
      void_rows(tile.r, tok.used, from_f32<T>(-INFINITY));
      void_rows(tile.i, tok.used, from_f32<T>(0.f));
      void_rows(tile.x, tok.used, from_f32<T>(0.f));
      __syncwarp();
    }
    Vf<V> av[STEPS], u[STEPS];
    ScanMap<V> mine = no_map<V>();
    const bool edge = tok.used != kAll || tok.first != 0 || tok.last != 0;
    const auto gates = [&](auto e) __attribute__((always_inline)) {
      constexpr bool EDGE = decltype(e)::value;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        constexpr bool SHARED = sizeof(T) == 2;
        Vf<V> rv, iv, xv;
        if constexpr (SHARED) {
          rv = gate_input<T>(row_pair(tile.r, j, lane)), iv = gate_input<T>(row_pair(tile.i, j, lane));
        } else {
          unpack<T, V>(row_pair(tile.r, j, lane), rv.v);
          unpack<T, V>(row_pair(tile.i, j, lane), iv.v);
        }
        unpack<T, V>(row_pair(tile.x, j, lane), xv.v);
        const GateValues<V> g = gate_values<V, SHARED, true>(a.consts, rv, iv, decay);
        u[j] = gated_input<V>(g, g.m, xv);
        av[j] = g.a;
        if (EDGE && (tok.first >> j & 1))
          mine = ScanMap<V>{splat<V>(-1.f), scan_initial<V>(a.h0, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width)};
        then_token<EDGE>(mine, av[j], u[j]);
      }
    };
    if (PACKED && edge) gates(std::true_type{});
    else gates(std::false_type{});
    __syncwarp();
    const auto load = [&] {
      r.next(span);
      i.next(span);
      x.next(span);
      r.load(tile.r, left - span, there);
      i.load(tile.i, left - span, there);
      x.load(tile.x, left - span, there);
    };
    Vf<V> h = scan_exchange<PACKED, V>(sh.maps, turn & 1, warp, rank, ctas, mine, carry, [&] {
      if constexpr (ALIGNED) load();
    });
    if (in && a.states && left > 0 && (L - left) % GATED_SCAN_STATE_EVERY == 0)
      put_state<V>(a.states,
                   n * ((a.L + GATED_SCAN_STATE_EVERY - 1) / GATED_SCAN_STATE_EVERY) + (L - left) / GATED_SCAN_STATE_EVERY,
                   a.C, c, width, h);
    const auto apply = [&](auto e) __attribute__((always_inline)) {
      constexpr bool EDGE = decltype(e)::value;
      T* out = y;
#pragma unroll
      for (int j = 0; j < STEPS; ++j, out += a.C) {
        if (EDGE && PACKED && (tok.first >> j & 1))
          h = scan_initial<V>(a.h0, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width);
        h = fma_v(av[j], h, u[j]);
        if (in && (!EDGE || (tok.used >> j & 1))) put_row<T, V, ALIGNED>(out, width, h);
        else if (EDGE && PACKED && in && a.fill && j < left) put_row<T, V, ALIGNED>(out, width, splat<V>(0.f));
        if (EDGE && PACKED && (tok.last >> j & 1)) {
          const int s = __shfl_sync(0xffffffffu, tok.seq, j);
          if (in && a.h_last) put_state<V>(a.h_last, s, a.C, c, width, h);
        }
      }
    };
    if (edge) apply(std::true_type{});
    else apply(std::false_type{});
    if constexpr (!ALIGNED) load();
  }
  copies_done();
  if (!PACKED && in && a.h_last && rank == 0 && warp == 0) put_state<V>(a.h_last, n, a.C, c, width, carry);
}

// ---- the backward pass -----------------------------------------------------
//
// Bounds: 14 bytes an element of a 16-bit type (11.1 from checkpoints).  Measured:
// 4 x 4096 x 2560 bf16 in 207 us, 2.8 TB/s (43 % of the copy rate), from
// checkpoints 229; fp32 340 (3.45 TB/s; its shared memory holds one CTA an SM);
// 16000 rows x 2048 f16 in 29 sequences from checkpoints 252.  It issues some 86
// instructions an element at 50 % of the rate, at 16 warps an SM; keeping s and m
// in shared memory instead of in spilled registers took 232 -> 217, a reciprocal
// for each sigmoid 214 -> 207, expanding checkpoints to tiles once instead of at
// each use 574 -> 237.

// x, r and i of the backward pass on their way to the tiles: elements with
// strides of their own, or with Q8 checkpoints' bytes, which each warp expands in
// place once they are there (they are exact in T): 16 a lane, of one row and one
// block of 32, whose step's byte the lane has loaded with them.
template <typename T, bool Q8, bool ALIGNED>
struct GradRows {
  TileWalk<T, kScanSteps, ALIGNED> x, r, i;
  __device__ __forceinline__ void start(const ScanArgs& a, int n, long long t0, int c0) {
    x.start(a.x, n, t0, c0);
    r.start(a.r, n, t0, c0);
    i.start(a.i, n, t0, c0);
  }
  template <typename Tiles>
  __device__ __forceinline__ void load(const ScanArgs&, Tiles& to, int rows, int width) {
    r.load(to.r, rows, width);
    i.load(to.i, rows, width);
    x.load(to.x, rows, width);
  }
  __device__ __forceinline__ void next(const ScanArgs&, long long span) {
    x.next(span);
    r.next(span);
    i.next(span);
  }
  template <typename Tiles>
  __device__ __forceinline__ void expand(Tiles&) const {}
};

template <typename T, bool ALIGNED>
struct GradRows<T, true, ALIGNED> {
  using Tile = RowTile<T, kScanSteps>;
  using Tile8 = RowTile<signed char, kScanSteps>;
  static_assert(kScanSteps == 8, "expand8 takes 8 rows");
  long long at, block;  // the walk's first element and the lane's step: the three are laid out alike
  int xs, rs, is;       // the lane's steps' bytes

  __device__ __forceinline__ void start(const ScanArgs& a, int n, long long t0, int c0) {
    const int lane = threadIdx.x & 31;
    at = (n * a.L + t0) * a.C + c0;
    block = (n * a.L + t0 + lane / 4) * ((a.C + ACT8_BLOCK - 1) / ACT8_BLOCK) + c0 / ACT8_BLOCK + lane % 4 / 2;
  }
  __device__ __forceinline__ int load_one(const ScanArgs& a, const SeqIn& in, Tile& tile, int rows, int width) const {
    const int lane = threadIdx.x & 31;
    TileWalk<signed char, kScanSteps, ALIGNED> walk;
    walk.start(SeqIn{static_cast<const signed char*>(in.p) + at, nullptr, 0, a.C}, 0, 0, 0);
    walk.load(reinterpret_cast<Tile8&>(tile), rows, width);
    return lane / 4 < rows && lane % 4 / 2 * ACT8_BLOCK < width ? __ldg(in.scale + block) : 0;
  }
  template <typename Tiles>
  __device__ __forceinline__ void load(const ScanArgs& a, Tiles& to, int rows, int width) {
    rs = load_one(a, a.r, to.r, rows, width);
    is = load_one(a, a.i, to.i, rows, width);
    xs = load_one(a, a.x, to.x, rows, width);
  }
  __device__ __forceinline__ void next(const ScanArgs& a, long long span) {
    at += span * a.C;
    block += span * ((a.C + ACT8_BLOCK - 1) / ACT8_BLOCK);
  }
  template <typename Tiles>
  __device__ __forceinline__ void expand(Tiles& t) const {
    expand8(t.r, 0, rs);
    expand8(t.i, 0, is);
    expand8(t.x, 0, xs);
  }
};

template <typename T>
struct GradShared {
  ScanShared<2> maps;
  ScanMap<2> ahead[2][kScanWarps][32];  // the forward maps, within the CTA
  struct {
    RowTile<T, kScanSteps> x, dy;
    union {
      struct {
        RowTile<T, kScanSteps> r, i;
      };
      float2 m[kScanSteps][32];  // m, once r and i are used
    };
  } tile[kScanWarps][2];  // the turn at hand and the next
  float2 s[kScanWarps][kScanSteps][32];
};

template <typename T, bool PACKED, bool ALIGNED, bool Q8>
__global__ void __launch_bounds__(kScanThreads, 2) gated_scan_grad_kernel(const __grid_constant__ ScanArgs a) {
  constexpr int STEPS = kScanSteps, V = 2;
  extern __shared__ __align__(128) unsigned char smem[];
  GradShared<T>& sh = *reinterpret_cast<GradShared<T>*>(smem);
  ptx::pdl_wait_prev();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = cluster_rank(), ctas = cluster_size();
  const int c0 = static_cast<int>(blockIdx.x / ctas) * 64, c = c0 + lane * V;
  const int n = static_cast<int>(blockIdx.z * gridDim.y + blockIdx.y);
  if (!PACKED && n >= a.N) return;  // all of the cluster
  const int width = min(V, a.C - c), there = a.C - c0;
  const bool in = width > 0;
  const long long blocks = (a.L + GATED_SCAN_STATE_EVERY - 1) / GATED_SCAN_STATE_EVERY;
  const Vf<V> decay = load_decay<V>(a.decay, c, width);
  Vf<V> carry = PACKED ? splat<V>(0.f) : scan_initial<V>(a.dh_last, n, a.C, c, width), dd = splat<V>(0.f);
  if (PACKED) pass_empty<V>(a, a.dh_last, a.dh0, rank * kScanWarps + warp, ctas * kScanWarps, c, width);
  if (ctas > 1) cluster_arrive(false), cluster_wait();  // every CTA runs before another writes to its shared memory
  const int span = ctas * GATED_SCAN_STATE_EVERY;
  const int turns = static_cast<int>((a.L + span - 1) / span);
  // from the last turn to the first; t0: the warp's first row
  long long t0 = (turns - 1) * static_cast<long long>(span) + rank * GATED_SCAN_STATE_EVERY + warp * STEPS;
  GradRows<T, Q8, ALIGNED> in3;
  TileWalk<T, STEPS, ALIGNED> dy;
  in3.start(a, n, t0, c0);
  dy.start(a.dy, n, t0, c0);
  const auto load = [&](auto& tile, long long t) {
    const int rows = t < 0 ? 0 : static_cast<int>(min(a.L - t, static_cast<long long>(STEPS)));
    in3.load(a, tile, rows, there);
    dy.load(tile.dy, rows, there);
  };
  if (turns > 0) load(sh.tile[warp][(turns - 1) & 1], t0);
  long long row = (n * a.L + t0) * a.C + c;
  for (int turn = turns - 1; turn >= 0; --turn, t0 -= span, row -= static_cast<long long>(span) * a.C) {
    const long long block = t0 / GATED_SCAN_STATE_EVERY;
    const int b = turn & 1;
    auto& tile = sh.tile[warp][b];
    const ScanTokens tok = scan_tokens<STEPS, PACKED>(a, t0);
    // the state in front of the CTA's tokens
    const bool start = !PACKED && block == 0;
    Vf<V> h = scan_initial<V>(start ? a.h0 : a.states_in, start ? n : n * blocks + block, a.C, c, block < blocks ? width : 0);
    copies_done();
    in3.expand(tile);
    if (tok.used != kScanAll) {
      void_rows(tile.r, tok.used, from_f32<T>(-INFINITY));
      void_rows(tile.i, tok.used, from_f32<T>(0.f));
      void_rows(tile.x, tok.used, from_f32<T>(0.f));
      void_rows(tile.dy, tok.used, from_f32<T>(0.f));
      __syncwarp();
    }
    const auto row_of = [&](const auto& t, int j) {
      Vf<V> v;
      unpack<T, V>(row_pair(t, j, lane), v.v);
      return v;
    };
    // over: 1 / m, next to 0 where a = 1; s and m go to shared memory
    Vf<V> av[STEPS], g[STEPS], over[STEPS];
    Vf<V> mv[STEPS];
    ScanMap<V> fwd = no_map<V>(), bwd = no_map<V>();
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      const GateValues<V> gv = gate_values<V, false, false>(a.consts, row_of(tile.r, j), row_of(tile.i, j), decay);
#pragma unroll
      for (int k = 0; k < V; ++k) over[j][k] = gv.m[k] >= kLeastNormal ? rsqrt_approx(gv.m[k]) : gv.m[k];
      mv[j] = mul_v(gv.m, over[j]);
      sh.s[warp][j][lane] = make_float2(gv.s[0], gv.s[1]);
      g[j] = gv.g;
      av[j] = gv.a;
      if (PACKED && (tok.first >> j & 1))
        fwd = ScanMap<V>{splat<V>(-1.f), scan_initial<V>(a.h0, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width)};
      then_token<PACKED>(fwd, av[j], gated_input<V>(gv, mv[j], row_of(tile.x, j)));
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < STEPS; ++j) tile.m[j][lane] = make_float2(mv[j][0], mv[j][1]);
#pragma unroll
    for (int j = STEPS - 1; j >= 0; --j) {
      if (PACKED && (tok.last >> j & 1))
        bwd = ScanMap<V>{splat<V>(-1.f), scan_initial<V>(a.dh_last, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width)};
      then_token<PACKED>(bwd, av[j], mul_v(av[j], row_of(tile.dy, j)));
    }
    // forward only within the CTA, whose first state is kept; backward through
    // the cluster, whose last warp comes first (the barriers inside cover both)
    sh.ahead[b][warp][lane] = fwd;
    Vf<V> G = scan_exchange<PACKED, V>(sh.maps, b, kScanWarps - 1 - warp, ctas - 1 - rank, ctas, bwd, carry, [&] {
      in3.next(a, -span);
      dy.next(-span);
      load(sh.tile[warp][b ^ 1], t0 - span);
    });
#pragma unroll
    for (int w = 0; w < kScanWarps - 1; ++w)
      if (w < warp) h = follow<PACKED>(sh.ahead[b][w][lane], h);
    const auto pair_of = [](const float2& v) { return Vf<V>{{v.x, v.y}}; };
    Vf<V> hp[STEPS];  // the state in front of each token
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
      if (PACKED && (tok.first >> j & 1))
        h = scan_initial<V>(a.h0, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width);
      hp[j] = h;
      h = fma_v(av[j], h, mul_v(mul_v(pair_of(tile.m[j][lane]), g[j]), row_of(tile.x, j)));
    }
    Vf<V> part = splat<V>(0.f);
#pragma unroll
    for (int j = STEPS - 1; j >= 0; --j) {
      if (PACKED && (tok.last >> j & 1))
        G = scan_initial<V>(a.dh_last, __shfl_sync(0xffffffffu, tok.seq, j), a.C, c, width);
      // a token's reads stay behind the one's in front: read ahead they spill 100 bytes
      // (16000 x 2048 f16 packed, from checkpoints: 282 us with them, 248 without)
      if (PACKED) __syncwarp();
      const Vf<V> one = both<V>(a.consts.one), none1 = both<V>(a.consts.none);
      const Vf<V> whole = add_v(row_of(tile.dy, j), G), vx = mul_v(g[j], row_of(tile.x, j));
      const Vf<V> Gm = mul_v(whole, pair_of(tile.m[j][lane]));
      G = mul_v(av[j], whole);
      const Vf<V> back = mul_v(mul_v(av[j], vx), over[j]);
      const Vf<V> sv = pair_of(sh.s[warp][j][lane]);
      const Vf<V> dl = mul_v(G, fma_v(back, none1, hp[j])), sdl = mul_v(sv, dl);
      const Vf<V> dx = mul_v(Gm, g[j]), di = mul_v(mul_v(Gm, vx), fma_v(g[j], none1, one));
      const Vf<V> dr = mul_v(mul_v(neg_v(decay), sdl), fma_v(sv, none1, one));
      const long long at = row + static_cast<long long>(j) * a.C;
      if (in && (tok.used >> j & 1)) {
        part = add_v(part, sdl);
        put_row<T, V, ALIGNED>(static_cast<T*>(a.dx) + at, width, dx);
        put_row<T, V, ALIGNED>(static_cast<T*>(a.dr) + at, width, dr);
        put_row<T, V, ALIGNED>(static_cast<T*>(a.di) + at, width, di);
      } else if (PACKED && in && a.fill && t0 + j < a.L) {
        put_row<T, V, ALIGNED>(static_cast<T*>(a.dx) + at, width, splat<V>(0.f));
        put_row<T, V, ALIGNED>(static_cast<T*>(a.dr) + at, width, splat<V>(0.f));
        put_row<T, V, ALIGNED>(static_cast<T*>(a.di) + at, width, splat<V>(0.f));
      }
      if (PACKED && (tok.first >> j & 1)) {
        const int q = __shfl_sync(0xffffffffu, tok.seq, j);
        if (in && a.dh0) put_state<V>(a.dh0, q, a.C, c, width, G);
      }
    }
    dd = add_v(dd, part);
    __syncwarp();
  }
  copies_done();
  if (!PACKED && in && a.dh0 && rank == 0 && warp == 0) put_state<V>(a.dh0, n, a.C, c, width, carry);
  // ddecay: the CTA's warps in order
  __syncthreads();
  sh.maps.warp[0][warp][lane].P = dd;
  __syncthreads();
  if (warp == 0 && in) {
    Vf<V> sum = splat<V>(0.f);
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) sum = add_v(sum, sh.maps.warp[0][w][lane].P);
    put_state<V>(a.part, static_cast<long long>(n) * ctas + rank, a.C, c, width, neg_v(sum));
  }
}

// ddecay: the partial sums [n][C], a thread every 8th of them in order, then the
// eight in order.
__global__ void __launch_bounds__(256) gated_scan_sum_kernel(const float* __restrict__ part, float* out, int n, int C) {
  __shared__ float sums[8][32];
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < C)
    for (int k = threadIdx.y; k < n; k += 8) sum += part[static_cast<long long>(k) * C + c];
  sums[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y != 0 || c >= C) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) sum += sums[r][threadIdx.x];
  out[c] = sum;
}

struct ScanStepArgs {
  const void *x, *r, *i;
  const float* decay;
  float* h;
  const int* index;
  void* y;
  int B, slots, C, fill;
  long long xs, rs, is;
  GateConsts consts;
};

constexpr int kStepThreads = 128;

// One token of B requests, V channels a thread.  A slot that several rows name
// belongs to the first of them, whose threads take all its rows in order.
template <typename T, int V>
__global__ void __launch_bounds__(kStepThreads) gated_scan_step_kernel(const ScanStepArgs a) {
  ptx::pdl_wait_prev();
  const int c = (blockIdx.y * kStepThreads + threadIdx.x) * V;
  int b = blockIdx.x;
  const int slot = a.index ? __ldg(a.index + b) : b;
  const int others = a.index && slot >= 0 && slot < a.slots ? same_slot(a.index, a.B, b, slot) : 0;
  if (c >= a.C || (others & 1)) return;
  T* y = static_cast<T*>(a.y) + c;
  if (slot < 0 || slot >= a.slots) {
    if (a.fill) store_zero<T, V>(y + static_cast<long long>(b) * a.C);
    return;
  }
  const Vf<V> decay = load_decay<V>(a.decay, c, V);
  Vf<V> h;
  float* hp = a.h + static_cast<long long>(slot) * a.C + c;
#pragma unroll
  for (int k = 0; k < V; ++k) h[k] = hp[k];
  do {
    Vf<V> x, r, i;
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.x) + b * a.xs + c), x.v);
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.r) + b * a.rs + c), r.v);
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.i) + b * a.is + c), i.v);
    const GateValues<V> v = gate_values<V, false, true>(a.consts, r, i, decay);
    h = fma_v(v.a, h, gated_input<V>(v, v.m, x));
    store_vec<T, V>(y + static_cast<long long>(b) * a.C, h.v);
    if (!(others & 2)) break;
    for (++b; b < a.B && __ldg(a.index + b) != slot;) ++b;
  } while (b < a.B);
#pragma unroll
  for (int k = 0; k < V; ++k) hp[k] = h[k];
}

}  // namespace convfwd

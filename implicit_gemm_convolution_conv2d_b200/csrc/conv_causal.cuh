// conv_causal.cuh -- the causal depthwise convolution of sequences, its
// gradients and its form for single tokens.
//
//   z[t] = bias + sum_{o < K} w[K-1-o] x[t-o],   y = z or z * sigmoid(z)
//
// A warp owns 64 channels and a run of tokens, two channels a lane, whose
// arithmetic is packed.  Its rows come through shared memory (seq_tile.cuh), and
// the K - 1 rows in front of the current ones stay in registers, so x is read
// once from memory (and K - 1 rows a run once more, out of L2).  Where a sequence
// begins the rows in the registers become that sequence's window, so no later
// token needs to know where it began.
//
// KT is the least of 2, 3, 4 and 8 that holds K; taps behind K are skipped, not
// multiplied by zero, as x may be infinite there.
//
// Bounds: 4 bytes an element of a 16-bit type, 6 for the gradients.  Measured,
// K = 4 with silu: 8 x 4096 x 2560 bf16 in 67 us, 5.0 TB/s (77 % of the copy
// rate), fp32 in 121 (5.5 TB/s); a thread of 8 channels that loaded straight
// into registers took 124.  Its gradients: 138 us, 3.65 TB/s (56 %), from
// checkpoints 160; they issue some 30 instructions an element at 54 % of the
// rate, each waiting 2.4 cycles for the one in front of it at 16 warps an SM.
#pragma once

#include "seq_tile.cuh"

namespace convfwd {

struct CausalArgs {
  SeqIn x, dy;
  const void *w, *bias, *state, *dstate_out;
  const int* cu;
  void *y, *state_out, *dx, *dstate;
  float* part;
  int N, C, K, silu, fill;
  int L;      // tokens of a sequence (packed: all rows)
  int run;    // tokens of a warp's run
  int runs;   // runs of a sequence (packed: of all rows)
  int blocks; // of kCausalWarps runs
};

// The sequence of a token, as the warps walk along it.
struct SeqAt {
  int s;           // its number, N where the row is in none
  int begin, end;  // its first token and the one behind its last
};

__device__ __forceinline__ void seq_find(SeqAt& q, const CausalArgs& a, int t) {
  q.s = seq_of_row(a.cu, a.N, t);
  if (q.s < a.N) {
    q.begin = max(0, __ldg(a.cu + q.s));
    q.end = min(a.L, __ldg(a.cu + q.s + 1));
  } else {  // unused rows: up to the next sequence's first token, or the end
    const int first = a.N > 0 ? __ldg(a.cu) : 0;
    q.begin = t;
    q.end = t < first ? min(a.L, first) : a.L;
  }
}

// `width` (V at most) channels from c on of row t of sequence q of x, or of its
// window where t is in front of it; zeros behind them.
template <typename T, int V, bool Q8>
__device__ __forceinline__ Vf<V> row_or_window(const CausalArgs& a, int n, const SeqAt& q, int t, int c, int width) {
  Vf<V> v = splat<V>(0.f);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (k >= width) continue;
    if (t >= q.begin) {
      const long long at = n * a.x.batch + t * a.x.token + c + k;
      if constexpr (Q8) {
        const long long row = static_cast<long long>(n) * a.L + t;
        v[k] = static_cast<float>(static_cast<const signed char*>(a.x.p)[at]) *
               act8_step(__ldg(a.x.scale + row * ((a.C + ACT8_BLOCK - 1) / ACT8_BLOCK) + (c + k) / ACT8_BLOCK));
      } else {
        v[k] = to_f32<T>(__ldg(static_cast<const T*>(a.x.p) + at));
      }
    } else if (a.state && q.s < a.N && t >= q.begin - (a.K - 1)) {
      const long long row = static_cast<long long>(q.s) * (a.K - 1) + (a.K - 1 + t - q.begin);
      v[k] = to_f32<T>(__ldg(static_cast<const T*>(a.state) + row * a.C + c + k));
    }
  }
  return v;
}

// w[c + k][K-1-o] in w[o][k], and the bias; zeros behind `width` channels.
template <typename T, int KT, int V>
__device__ __forceinline__ void load_filter(Vf<V> (&w)[KT], Vf<V>& bias, const void* wp, const void* bp, int K, int c, int width) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const bool in = k < width;
    bias[k] = bp && in ? to_f32<T>(static_cast<const T*>(bp)[c + k]) : 0.f;
#pragma unroll
    for (int o = 0; o < KT; ++o)
      w[o][k] = o < K && in ? to_f32<T>(static_cast<const T*>(wp)[static_cast<long long>(c + k) * K + K - 1 - o]) : 0.f;
  }
}

// Whether tap o exists: where KT is not K itself, known only now.
template <int KT>
__device__ __forceinline__ bool has_tap(int o, int K) {
  return KT == 3 || KT == 4 || o < K;
}

// sigmoid(z), and silu's slope s (1 + z (1 - s))
template <int V>
__device__ __forceinline__ Vf<V> sigmoid_v(const Vf<V>& z) {
  Vf<V> s;
#pragma unroll
  for (int k = 0; k < V; ++k) s[k] = rcp_approx(1.f + ex2_approx(z[k] * -kLog2e));
  return s;
}
template <int V>
__device__ __forceinline__ Vf<V> silu_slope(const Vf<V>& z) {
  const Vf<V> s = sigmoid_v(z);
  Vf<V> r;
#pragma unroll
  for (int k = 0; k < V; ++k) r[k] = 1.f - s[k];
  r = mul_v(z, r);
  return fma_v(s, r, s);
}

constexpr int kCausalWarps = 8;
constexpr int kCausalThreads = 32 * kCausalWarps;
// Rows of a tile (2 KB), and tokens that are computed together: their rows move
// through registers, which unrolled steps rename rather than copy.
template <typename T>
constexpr int kCausalRows = 32 / static_cast<int>(sizeof(T));
constexpr int kCausalTogether = 8;

template <typename T>
struct CausalShared {
  RowTile<T, kCausalRows<T>> x[kCausalWarps][2];  // the rows at hand and the next
};

template <int LEFT>
__device__ __forceinline__ void groups_done() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
  __syncwarp();
}
__device__ __forceinline__ void group_ends() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <typename T, int KT, bool ALIGNED>
__global__ void __launch_bounds__(kCausalThreads) conv_causal_kernel(const __grid_constant__ CausalArgs a) {
  constexpr int V = 2, ROWS = kCausalRows<T>, U = kCausalTogether, W = KT - 1;
  extern __shared__ __align__(128) unsigned char smem[];
  CausalShared<T>& sh = *reinterpret_cast<CausalShared<T>*>(smem);
  ptx::pdl_wait_prev();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * 64, c = c0 + lane * V, there = a.C - c0;
  const int width = min(V, a.C - c);
  const bool in = width > 0;
  const long long block = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y, job = block * kCausalWarps + warp;
  T* state_out = static_cast<T*>(a.state_out);
  if (state_out && in) {
    // sequences without a token leave their window as it was
    for (long long s = job; s < a.N; s += static_cast<long long>(gridDim.y) * gridDim.z * kCausalWarps) {
      if (a.cu ? __ldg(a.cu + s) < __ldg(a.cu + s + 1) : a.L > 0) continue;
      const SeqAt q{static_cast<int>(s), 0, 0};
      for (int j = 0; j < a.K - 1; ++j)
        put_row<T, V, ALIGNED>(state_out + (s * (a.K - 1) + j) * a.C + c, width,
                               row_or_window<T, V, false>(a, 0, q, j - (a.K - 1), c, width));
    }
  }
  if (job >= static_cast<long long>(a.runs) * (a.cu ? 1 : a.N)) return;
  const int n = a.cu ? 0 : static_cast<int>(job / a.runs);
  const int t0 = static_cast<int>(job - static_cast<long long>(n) * a.runs) * a.run, t1 = min(a.L, t0 + a.run);

  TileWalk<T, ROWS, ALIGNED> walk;
  walk.start(a.x, n, t0, c0);
  auto& tile = sh.x[warp];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    walk.load(tile[k], t1 - t0 - k * ROWS, there);
    walk.next(ROWS);
    group_ends();
  }
  Vf<V> w[KT], bias, X[W + U];  // X[W + u]: row t + u
  load_filter<T, KT, V>(w, bias, a.w, a.bias, a.K, c, width);
  SeqAt q{n, 0, a.L};
  if (a.cu) seq_find(q, a, t0);
#pragma unroll
  for (int o = 1; o <= W; ++o) X[W - o] = row_or_window<T, V, false>(a, n, q, t0 - o, c, width);

  T* out = static_cast<T*>(a.y) + (static_cast<long long>(n) * a.L + t0) * a.C + c;
  const auto put = [&](T* p, const Vf<V>& z) {
    if (in) put_row<T, V, ALIGNED>(p, width, z);
  };
  const auto compute = [&](int u) {
    Vf<V> z = fma_v(w[0], X[W + u], bias);
#pragma unroll
    for (int o = 1; o < KT; ++o)
      if (has_tap<KT>(o, a.K)) z = fma_v(w[o], X[W + u - o], z);
    return z;
  };
  int b = 0;
  for (int t = t0; t < t1; t += ROWS, b ^= 1) {
    groups_done<1>();
#pragma unroll 1
    for (int r = 0; r < ROWS; r += U, out += static_cast<long long>(U) * a.C) {
#pragma unroll
      for (int u = 0; u < U; ++u) unpack<T, V>(row_pair(tile[b], r + u, lane), X[W + u].v);
      const int at = t + r;
      if (q.s < a.N && at + U <= t1 && at + U < q.end + (state_out ? 0 : 1)) {
        T* p = out;
        if (a.silu) {
#pragma unroll
          for (int u = 0; u < U; ++u, p += a.C) {
            const Vf<V> z = compute(u);
            put(p, mul_v(z, sigmoid_v(z)));
          }
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u, p += a.C) put(p, compute(u));
        }
      } else {
        // a sequence or the run ends here
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (at + u >= t1) break;
          if (at + u >= q.end) {
            seq_find(q, a, at + u);
#pragma unroll
            for (int o = 1; o <= W; ++o) X[W + u - o] = row_or_window<T, V, false>(a, n, q, at + u - o, c, width);
          }
          T* p = out + static_cast<long long>(u) * a.C;
          if (q.s < a.N) {
            const Vf<V> z = compute(u);
            put(p, a.silu ? mul_v(z, sigmoid_v(z)) : z);
          } else if (a.fill) {
            put(p, splat<V>(0.f));
          }
          if (state_out && q.s < a.N && at + u == q.end - 1) {
#pragma unroll
            for (int o = 0; o < W; ++o)
              if (o < a.K - 1) put(state_out + (static_cast<long long>(q.s) * (a.K - 1) + a.K - 2 - o) * a.C + c, X[W + u - o]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) X[i] = X[i + U];
    }
    __syncwarp();
    walk.load(tile[b], t1 - t - 2 * ROWS, there);
    walk.next(ROWS);
    group_ends();
  }
  groups_done<0>();
}

// ---- gradients ----------------------------------------------------------
//
// A warp walks its run and the K - 1 tokens behind it: z is computed again from
// x, dz[t] = dy[t] * (slope of the activation), and each dz[t] goes to the K rows
// of dx that token t read.  A row is complete once the token K - 1 behind it is
// in, so the pending rows of dx move through registers like the rows of x.
//
// dw and dbias of the run's own tokens are summed per warp, the block's warps in
// shared memory in order, and blocks by conv_causal_sum_kernel in order.
constexpr int kGradTogether = 8;

template <typename T>
struct CausalGradShared {
  struct {
    RowTile<T, kCausalRows<T>> x, dy;
  } tile[kCausalWarps][2];
};

// A lane's registers.
template <typename T, int KT, bool Q8>
struct GradRegs {
  static constexpr int V = 2, U = kGradTogether, W = KT - 1;
  Vf<V> w[KT], bias, X[W + U], D[W + U], dw[KT], db;  // X[W + u], D[W + u]: rows t + u of x and dx
  unsigned used;                                       // bit i: row t - W + i is in a sequence, and the run's
  SeqAt q;

  // Token t + u of those together, its row of x and of dy.  EDGE: a sequence's or
  // the run's end, or the window's gradient, may touch it.  t1: behind the run;
  // t2: behind the last token that reads a row of it.
  template <bool EDGE>
  __device__ __forceinline__ void token(const CausalArgs& a, int n, int u, int t, int t1, int t2, int c, int width,
                                        const Raw<T, V>& x, const Raw<T, V>& dy) {
    X[W + u] = D[W + u] = splat<V>(0.f);
    int pos = KT;
    if (EDGE) {
      if (t + u >= t2) return;
      if (t + u >= q.end) {
        seq_find(q, a, t + u);
#pragma unroll
        for (int o = 1; o <= W; ++o) X[W + u - o] = row_or_window<T, V, Q8>(a, n, q, t + u - o, c, width);
      }
      if (q.s >= a.N) return;
      pos = min(t + u - q.begin, KT);
      const int slot = t + u - q.end + a.K - 1;  // of the window that the sequence leaves
      if (a.dstate_out && slot >= 0) {
        const T* g = static_cast<const T*>(a.dstate_out) + (static_cast<long long>(q.s) * (a.K - 1) + slot) * a.C + c;
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (k < width) D[W + u][k] = to_f32<T>(__ldg(g + k));
      }
    }
    const bool own = !EDGE || t + u < t1;
    if (own) used |= 1u << (W + u);
    Vf<V> dz;
    unpack<T, V>(x, X[W + u].v);
    unpack<T, V>(dy, dz.v);
    if (a.silu) {
      Vf<V> z = fma_v(w[0], X[W + u], bias);
#pragma unroll
      for (int o = 1; o < KT; ++o)
        if (has_tap<KT>(o, a.K)) z = fma_v(w[o], X[W + u - o], z);
      dz = mul_v(dz, silu_slope(z));
    }
    if (own) {
      db = add_v(db, dz);
#pragma unroll
      for (int o = 0; o < KT; ++o)
        if (has_tap<KT>(o, a.K)) dw[o] = fma_v(dz, X[W + u - o], dw[o]);
    }
#pragma unroll
    for (int o = 0; o < KT; ++o)
      if (has_tap<KT>(o, a.K) && (!EDGE || o <= pos)) D[W + u - o] = fma_v(w[o], dz, D[W + u - o]);
  }
};

template <typename T, int KT, bool ALIGNED, bool Q8>
__global__ void __launch_bounds__(kCausalThreads, 2) conv_causal_grad_kernel(const __grid_constant__ CausalArgs a) {
  constexpr int V = 2, ROWS = kCausalRows<T>, U = kGradTogether, W = KT - 1;
  extern __shared__ __align__(128) unsigned char smem[];
  CausalGradShared<T>& sh = *reinterpret_cast<CausalGradShared<T>*>(smem);
  ptx::pdl_wait_prev();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = blockIdx.x * 64, c = c0 + lane * V, there = a.C - c0;
  const int width = min(V, a.C - c);
  const bool in = width > 0;
  const long long block = static_cast<long long>(blockIdx.z) * gridDim.y + blockIdx.y, job = block * kCausalWarps + warp;
  GradRegs<T, KT, Q8> k;
  k.db = splat<V>(0.f);
#pragma unroll
  for (int o = 0; o < KT; ++o) k.dw[o] = splat<V>(0.f);
  if (job < static_cast<long long>(a.runs) * (a.cu ? 1 : a.N)) {
    const int n = a.cu ? 0 : static_cast<int>(job / a.runs);
    const int t0 = static_cast<int>(job - static_cast<long long>(n) * a.runs) * a.run, t1 = min(a.L, t0 + a.run);
    const int t2 = min(a.L, t1 + a.K - 1);  // behind the last token that reads a row of the run
    TileWalk<T, ROWS, ALIGNED> walk, walk_dy;
    TileWalk<signed char, ROWS, ALIGNED> walk8;
    const unsigned char* steps = nullptr;  // of the lane's row and block (see expand8)
    const int nblk = (a.C + ACT8_BLOCK - 1) / ACT8_BLOCK;
    if constexpr (Q8) {
      walk8.start(a.x, n, t0, c0);
      steps = a.x.scale + (static_cast<long long>(n) * a.L + t0 + lane / 4) * nblk + c0 / ACT8_BLOCK + lane % 4 / 2;
    } else {
      walk.start(a.x, n, t0, c0);
    }
    walk_dy.start(a.dy, n, t0, c0);
    int byte[2][ROWS / 8] = {};
    const auto load = [&](int b, int rows) {
      auto& tile = sh.tile[warp][b];
      if constexpr (Q8) {
        // bytes of eight rows at the beginning of each eight rows of the tile
        walk8.load(reinterpret_cast<RowTile<signed char, ROWS>&>(tile.x), rows, there);
        walk8.next(ROWS);
#pragma unroll
        for (int e = 0; e < ROWS / 8; ++e) {
          byte[b][e] = 0;
          if (lane / 4 + 8 * e < rows && lane % 4 / 2 * ACT8_BLOCK < there) byte[b][e] = __ldg(steps + 8 * e * nblk);
        }
        steps += ROWS * nblk;
      } else {
        walk.load(tile.x, rows, there);
        walk.next(ROWS);
      }
      walk_dy.load(tile.dy, rows, there);
      walk_dy.next(ROWS);
      group_ends();
    };
    load(0, t2 - t0);
    load(1, t2 - t0 - ROWS);
    load_filter<T, KT, V>(k.w, k.bias, a.w, a.bias, a.K, c, width);
    k.used = 0;
    k.q = SeqAt{n, 0, a.L};
    if (a.cu) seq_find(k.q, a, t0);
#pragma unroll
    for (int o = 1; o <= W; ++o) {
      k.X[W - o] = row_or_window<T, V, Q8>(a, n, k.q, t0 - o, c, width);
      k.D[W - o] = splat<V>(0.f);
    }
    T* out = static_cast<T*>(a.dx) + (static_cast<long long>(n) * a.L + t0 - W) * a.C + c;  // row t - W

    int b = 0;
    for (int t = t0; t < t1 + W; t += ROWS, b ^= 1) {
      groups_done<1>();
      auto& tile = sh.tile[warp][b];
      if constexpr (Q8) {
#pragma unroll
        for (int e = ROWS / 8 - 1; e >= 0; --e) {  // the bytes of later rows lie in front of their place
          move8(tile.x, e);
          expand8(tile.x, 8 * e, b ? byte[1][e] : byte[0][e]);
        }
      }
#pragma unroll 1
      for (int r = 0; r < ROWS; r += U, out += static_cast<long long>(U) * a.C) {
        const int at = t + r;
        const bool inside = k.q.s < a.N && at + U <= t1 && at - k.q.begin >= W &&
                            at + U <= k.q.end - (a.dstate_out ? a.K - 1 : 0);
        T* p = out;
        if (inside) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            k.template token<false>(a, n, u, at, t1, t2, c, width, row_pair(tile.x, r + u, lane), row_pair(tile.dy, r + u, lane));
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u)
            k.template token<true>(a, n, u, at, t1, t2, c, width, row_pair(tile.x, r + u, lane), row_pair(tile.dy, r + u, lane));
        }
#pragma unroll
        for (int i = 0; i < U; ++i, p += a.C) {
          if (in && (k.used >> i & 1)) put_row<T, V, ALIGNED>(p, width, k.D[i]);
          else if (in && a.fill && at - W + i >= t0 && at - W + i < t1) put_row<T, V, ALIGNED>(p, width, splat<V>(0.f));
        }
        k.used >>= U;
#pragma unroll
        for (int i = 0; i < W; ++i) k.X[i] = k.X[i + U], k.D[i] = k.D[i + U];
      }
      __syncwarp();
      load(b, t2 - t - 2 * ROWS);
    }
    groups_done<0>();
  }
  // the block's warps in order
  __syncthreads();
  Vf<V>(&sums)[kCausalWarps][32] = *reinterpret_cast<Vf<V>(*)[kCausalWarps][32]>(smem);
#pragma unroll
  for (int o = 0; o <= KT; ++o) {
    if (o < KT && o >= a.K) continue;
    sums[warp][lane] = o < KT ? k.dw[o < KT ? o : 0] : k.db;
    __syncthreads();
    const int row = o < KT ? a.K - 1 - o : a.K;
    if (warp == 0 && in && block < a.blocks) {
      Vf<V> sum = sums[0][lane];
#pragma unroll
      for (int r = 1; r < kCausalWarps; ++r) sum = add_v(sum, sums[r][lane]);
      float* part = a.part + (block * (a.K + 1) + row) * a.C + c;
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < width) part[e] = sum[e];
    }
    __syncthreads();
  }
}

// dw and dbias: the blocks' partial sums [blocks][K + 1][C], a thread every 8th
// of them in order, then the eight in order.
template <typename T>
__global__ void __launch_bounds__(256) conv_causal_sum_kernel(const float* __restrict__ part, T* dw, T* dbias, int blocks,
                                                              int C, int K) {
  __shared__ float sums[8][32];
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
  float sum = 0.f;
  if (c < C)
    for (int b = threadIdx.y; b < blocks; b += 8) sum += part[(static_cast<long long>(b) * (K + 1) + j) * C + c];
  sums[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y != 0 || c >= C) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) sum += sums[r][threadIdx.x];
  if (j < K) dw[static_cast<long long>(c) * K + j] = from_f32<T>(sum);
  else if (dbias) dbias[c] = from_f32<T>(sum);
}

// dstate: the window's rows are read by a sequence's first K - 1 tokens, and
// passed on by a sequence of fewer.  A thread a (sequence, channel).
template <typename T, bool Q8>
__global__ void __launch_bounds__(128) conv_causal_dstate_kernel(const __grid_constant__ CausalArgs a) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * 128 + threadIdx.x, K = a.K;
  if (c >= a.C) return;
  for (long long next = blockIdx.y; next < a.N; next += gridDim.y) {  // may pass 31 bits behind the last
    const int s = static_cast<int>(next), n = a.cu ? 0 : s;
    SeqAt q{s, 0, a.L};
    if (a.cu) {
      q.begin = max(0, min(a.L, __ldg(a.cu + s)));
      q.end = max(q.begin, min(a.L, __ldg(a.cu + s + 1)));
    }
    const int len = min(q.end - q.begin, K - 1);
    float w[CONV_CAUSAL_MAX_K], row[2 * CONV_CAUSAL_MAX_K], d[CONV_CAUSAL_MAX_K];
    for (int j = 0; j < K; ++j) w[j] = to_f32<T>(static_cast<const T*>(a.w)[static_cast<long long>(c) * K + j]);
    // row[j]: the window's rows, then the first tokens
    for (int j = 0; j < K - 1 + len; ++j) row[j] = row_or_window<T, 1, Q8>(a, n, q, q.begin + j - (K - 1), c, 1)[0];
    for (int m = 0; m < K - 1; ++m) d[m] = 0.f;
    for (int p = 0; p < len; ++p) {
      const long long t = q.begin + p;
      float dz = to_f32<T>(static_cast<const T*>(a.dy.p)[n * a.dy.batch + t * a.dy.token + c]);
      if (a.silu) {
        float z = a.bias ? to_f32<T>(static_cast<const T*>(a.bias)[c]) : 0.f;
        for (int j = 0; j < K; ++j) z = fmaf(w[j], row[p + j], z);
        dz *= silu_slope(Vf<1>{{z}})[0];
      }
      for (int j = 0; p + j < K - 1; ++j) d[p + j] = fmaf(w[j], dz, d[p + j]);
    }
    for (int m = 0; m < K - 1; ++m) {
      const long long at = (static_cast<long long>(s) * (K - 1) + m) * a.C + c;
      if (a.dstate_out && m - len >= 0 && q.end - q.begin < K - 1)
        d[m] += to_f32<T>(static_cast<const T*>(a.dstate_out)[at - static_cast<long long>(len) * a.C]);
      static_cast<T*>(a.dstate)[at] = from_f32<T>(d[m]);
    }
  }
}

// ---- single tokens ------------------------------------------------------

struct CausalStepArgs {
  const void *x, *w, *bias;
  void* state;
  const int* index;
  void* y;
  int B, slots, C, K, silu, fill;
  long long xs;
};

constexpr int kCausalStepThreads = 128;

// One token of B requests, V channels a thread.  A slot that several rows name
// belongs to the first of them, whose threads take all its rows in order.
template <typename T, int KT, int V>
__global__ void __launch_bounds__(kCausalStepThreads) conv_causal_step_kernel(const CausalStepArgs a) {
  ptx::pdl_wait_prev();
  const int c = (blockIdx.y * kCausalStepThreads + threadIdx.x) * V;
  int b = blockIdx.x;
  const int slot = a.index ? __ldg(a.index + b) : b;
  const bool held = slot >= 0 && slot < a.slots;
  const int others = a.index && held ? same_slot(a.index, a.B, b, slot) : 0;
  if (c >= a.C || (others & 1)) return;
  T* y = static_cast<T*>(a.y) + c;
  if (!held) {
    if (a.fill) store_zero<T, V>(y + static_cast<long long>(b) * a.C);
    return;
  }
  Vf<V> w[KT], bias, old[KT - 1];  // old[o]: the row o + 1 tokens ago
  load_filter<T, KT, V>(w, bias, a.w, a.bias, a.K, c, V);
  T* window = static_cast<T*>(a.state) + static_cast<long long>(slot) * (a.K - 1) * a.C + c;
#pragma unroll
  for (int o = 0; o < KT - 1; ++o)
    if (o < a.K - 1) {
      const Raw<T, V> raw = *reinterpret_cast<const Raw<T, V>*>(window + static_cast<long long>(a.K - 2 - o) * a.C);
      unpack<T, V>(raw, old[o].v);
    }
  do {
    Vf<V> x;
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.x) + b * a.xs + c), x.v);
    Vf<V> z = fma_v(w[0], x, bias);
#pragma unroll
    for (int o = 1; o < KT; ++o)
      if (has_tap<KT>(o, a.K)) z = fma_v(w[o], old[o - 1], z);
#pragma unroll
    for (int o = KT - 2; o > 0; --o) old[o] = old[o - 1];
    old[0] = x;
    if (a.silu) z = mul_v(z, sigmoid_v(z));
    store_vec<T, V>(y + static_cast<long long>(b) * a.C, z.v);
    if (!(others & 2)) break;
    for (++b; b < a.B && __ldg(a.index + b) != slot;) ++b;
  } while (b < a.B);
#pragma unroll
  for (int o = 0; o < KT - 1; ++o)
    if (o < a.K - 1) store_vec<T, V>(window + static_cast<long long>(a.K - 2 - o) * a.C, old[o].v);
}

}  // namespace convfwd

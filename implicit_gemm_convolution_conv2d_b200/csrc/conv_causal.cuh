// conv_causal.cuh -- the causal depthwise convolution of sequences, its
// gradients and its form for single tokens.
//
//   z[t] = bias + sum_{o < K} w[K-1-o] x[t-o],   y = z or z * sigmoid(z)
//
// A thread owns V neighbouring channels and a run of tokens, and keeps the
// K - 1 rows in front of the current one in registers, so x is read once from
// memory (and K - 1 rows a run once more, out of L2).  Where a sequence begins
// the rows in the registers become that sequence's window, so no later token
// needs to know where it began.
//
// KT is the least of 2, 3, 4 and 8 that holds K; taps behind K are skipped, not multiplied
// by zero, as x may be infinite there.
#pragma once

#include "seq_common.cuh"

namespace convfwd {

struct CausalArgs {
  const void *x, *w, *bias, *state, *dy, *dstate_out;
  const unsigned char* x_scale;
  const int* cu;
  void *y, *state_out, *dx, *dw, *dbias, *dstate;
  float* part;
  int N, C, K, silu, fill;
  long long L, x_batch, x_token, dy_batch, dy_token;
  int run;         // tokens of a thread's run
  long long runs;  // runs of a sequence (packed: of all rows)
};

__device__ __forceinline__ float causal_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// The sequence of a token, as the threads walk along it.
struct SeqAt {
  int s;                 // its number, N where the row is in none
  long long begin, end;  // its first token and the one behind its last
};

__device__ __forceinline__ void seq_find(SeqAt& q, const CausalArgs& a, long long t) {
  q.s = seq_of_row(a.cu, a.N, t);
  if (q.s < a.N) {
    q.begin = max(0, __ldg(a.cu + q.s));
    q.end = min(a.L, static_cast<long long>(__ldg(a.cu + q.s + 1)));
  } else {  // unused rows: up to the next sequence's first token, or the end
    const long long first = a.N > 0 ? __ldg(a.cu) : 0;
    q.begin = t;
    q.end = t < first ? min(a.L, first) : a.L;
  }
}

// V channels of row t of x.
template <typename T, int V, bool Q8>
struct XRow {
  using R = typename RawVec<Q8 ? V : static_cast<int>(sizeof(T)) * V>::type;
  R raw;
  unsigned char byte;
  __device__ __forceinline__ void load(const CausalArgs& a, int n, long long t, int c) {
    const long long at = n * a.x_batch + t * a.x_token + c;
    if constexpr (Q8) {
      raw = __ldg(reinterpret_cast<const R*>(static_cast<const signed char*>(a.x) + at));
      const long long row = n * a.L + t;
      byte = __ldg(a.x_scale + row * ((a.C + ACT8_BLOCK - 1) / ACT8_BLOCK) + c / ACT8_BLOCK);
    } else {
      raw = __ldg(reinterpret_cast<const R*>(static_cast<const T*>(a.x) + at));
    }
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (Q8) {
      union {
        R r;
        signed char e[V];
      } u;
      u.r = raw;
      const float step = act8_step(byte);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] = static_cast<float>(u.e[k]) * step;
    } else {
      unpack<T, V>(raw, v);
    }
  }
};

// Row `t` of sequence q of x, or of its window where t is in front of it.
template <typename T, int V, bool Q8>
__device__ __forceinline__ void row_or_window(float (&v)[V], const CausalArgs& a, int n, const SeqAt& q, long long t,
                                              int c) {
  if (t >= q.begin) {
    XRow<T, V, Q8> x;
    x.load(a, n, t, c);
    x.get(v);
  } else if (a.state && q.s < a.N && t >= q.begin - (a.K - 1)) {
    const long long row = static_cast<long long>(q.s) * (a.K - 1) + (a.K - 1 + t - q.begin);
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.state) + row * a.C + c), v);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 0.f;
  }
}

// w[c + k][K-1-o] in w[o][k], and the bias.
template <typename T, int KT, int V>
__device__ __forceinline__ void load_filter(float (&w)[KT][V], float (&bias)[V], const CausalArgs& a, int c) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    bias[k] = a.bias ? to_f32<T>(static_cast<const T*>(a.bias)[c + k]) : 0.f;
#pragma unroll
    for (int o = 0; o < KT; ++o)
      w[o][k] = o < a.K ? to_f32<T>(static_cast<const T*>(a.w)[static_cast<long long>(c + k) * a.K + a.K - 1 - o]) : 0.f;
  }
}

constexpr int kCausalThreads = 256;
constexpr int kCausalAhead = 4;  // rows loaded ahead of their use

template <typename T, int KT, int V>
__global__ void __launch_bounds__(kCausalThreads) conv_causal_kernel(const CausalArgs a) {
  ptx::pdl_wait_prev();
  const int nvec = a.C / V;
  const long long id = static_cast<long long>(blockIdx.x) * kCausalThreads + threadIdx.x;
  T* y = static_cast<T*>(a.y);
  T* state_out = static_cast<T*>(a.state_out);
  if (state_out) {
    // sequences without a token leave their window as it was
    const long long all = static_cast<long long>(gridDim.x) * kCausalThreads;
    for (long long k = id; k < static_cast<long long>(a.N) * nvec; k += all) {
      const int s = static_cast<int>(k / nvec), c = static_cast<int>(k - static_cast<long long>(s) * nvec) * V;
      if (a.cu ? __ldg(a.cu + s) < __ldg(a.cu + s + 1) : a.L > 0) continue;
      for (int j = 0; j < a.K - 1; ++j) {
        const long long at = (static_cast<long long>(s) * (a.K - 1) + j) * a.C + c;
        float v[V] = {};
        if (a.state) unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.state) + at), v);
        store_vec<T, V>(state_out + at, v);
      }
    }
  }
  const long long run = id / nvec;
  if (run >= a.runs * (a.cu ? 1 : a.N)) return;
  const int c = static_cast<int>(id - run * nvec) * V;
  const int n = a.cu ? 0 : static_cast<int>(run / a.runs);
  const long long t0 = (run - n * a.runs) * a.run, t1 = min(a.L, t0 + a.run);

  float w[KT][V], bias[V], old[KT - 1][V];  // old[o]: row t - 1 - o
  load_filter<T, KT, V>(w, bias, a, c);
  SeqAt q{n, 0, a.L};
  if (a.cu) seq_find(q, a, t0);
#pragma unroll
  for (int o = 0; o < KT - 1; ++o) row_or_window<T, V, false>(old[o], a, n, q, t0 - 1 - o, c);

  for (long long t = t0; t < t1; t += kCausalAhead) {
    XRow<T, V, false> ahead[kCausalAhead];
#pragma unroll
    for (int u = 0; u < kCausalAhead; ++u)
      if (t + u < t1) ahead[u].load(a, n, t + u, c);
#pragma unroll
    for (int u = 0; u < kCausalAhead; ++u) {
      if (t + u >= t1) break;
      if (t + u >= q.end) {
        seq_find(q, a, t + u);
#pragma unroll
        for (int o = 0; o < KT - 1; ++o) row_or_window<T, V, false>(old[o], a, n, q, t + u - 1 - o, c);
      }
      float x[V], z[V];
      ahead[u].get(x);
#pragma unroll
      for (int k = 0; k < V; ++k) z[k] = fmaf(w[0][k], x[k], bias[k]);
#pragma unroll
      for (int o = 1; o < KT; ++o)
        if (o < a.K)
#pragma unroll
          for (int k = 0; k < V; ++k) z[k] = fmaf(w[o][k], old[o - 1][k], z[k]);
#pragma unroll
      for (int o = KT - 2; o > 0; --o)
#pragma unroll
        for (int k = 0; k < V; ++k) old[o][k] = old[o - 1][k];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        old[0][k] = x[k];
        if (a.silu) z[k] = z[k] * causal_sigmoid(z[k]);
      }
      T* out = y + (n * a.L + t + u) * a.C + c;
      if (q.s < a.N) store_vec<T, V>(out, z);
      else if (a.fill) store_zero<T, V>(out);
      if (state_out && q.s < a.N && t + u == q.end - 1) {
#pragma unroll
        for (int o = 0; o < KT - 1; ++o)
          if (o < a.K - 1)
            store_vec<T, V>(state_out + (static_cast<long long>(q.s) * (a.K - 1) + a.K - 2 - o) * a.C + c, old[o]);
      }
    }
  }
}

// d silu(z) / dz
__device__ __forceinline__ float silu_slope(float z) {
  const float s = causal_sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

// ---- gradients ----------------------------------------------------------
//
// A thread walks its run and the K - 1 tokens behind it: z is computed again
// from x, dz[t] = dy[t] * (slope of the activation), and each dz[t] goes to the
// K rows of dx that token t read.  Those are complete once dz[t+K-1] is in, so
// the pending ones (`next`) live in registers like the rows of x.  dw and dbias
// of the run's own tokens are summed per run, runs into the thread's total,
// threads of a block in shared memory in order, and blocks by
// conv_causal_sum_kernel in order.
constexpr int kGradLanes = 32, kGradRows = 8;  // a block: 32 vectors of channels x 8 runs

template <typename T, int KT, int V, bool Q8>
__global__ void __launch_bounds__(kGradLanes * kGradRows) conv_causal_grad_kernel(const CausalArgs a) {
  ptx::pdl_wait_prev();
  const int c = (blockIdx.x * kGradLanes + threadIdx.x) * V;
  const long long all_runs = a.runs * (a.cu ? 1 : a.N);
  T* dx = static_cast<T*>(a.dx);
  float dw_sum[KT][V] = {}, db_sum[V] = {};
  if (c < a.C) {
    float w[KT][V], bias[V];
    load_filter<T, KT, V>(w, bias, a, c);
    for (long long run = static_cast<long long>(blockIdx.y) * kGradRows + threadIdx.y; run < all_runs;
         run += static_cast<long long>(gridDim.y) * kGradRows) {
      const int n = a.cu ? 0 : static_cast<int>(run / a.runs);
      const long long t0 = (run - n * a.runs) * a.run, t1 = min(a.L, t0 + a.run), t2 = min(a.L, t1 + a.K - 1);
      float old[KT - 1][V], next[KT][V] = {}, dw[KT][V] = {}, db[V] = {};  // next[o]: dx of row t - o
      SeqAt q{n, 0, a.L};
      if (a.cu) seq_find(q, a, t0);
#pragma unroll
      for (int o = 0; o < KT - 1; ++o) row_or_window<T, V, Q8>(old[o], a, n, q, t0 - 1 - o, c);
      bool used[KT] = {};  // of row t - o
      for (long long t = t0; t < t1 + a.K - 1; ++t) {
        // next[] moves on by a row: the one of t begins
#pragma unroll
        for (int o = KT - 1; o > 0; --o) {
          used[o] = used[o - 1];
#pragma unroll
          for (int k = 0; k < V; ++k) next[o][k] = next[o - 1][k];
        }
        used[0] = false;
#pragma unroll
        for (int k = 0; k < V; ++k) next[0][k] = 0.f;
        if (t < t2) {
          if (t >= q.end) {
            seq_find(q, a, t);
#pragma unroll
            for (int o = 0; o < KT - 1; ++o) row_or_window<T, V, Q8>(old[o], a, n, q, t - 1 - o, c);
          }
          used[0] = q.s < a.N;
          if (used[0]) {
            XRow<T, V, Q8> xr;
            xr.load(a, n, t, c);
            float x[V], dz[V];
            xr.get(x);
            unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.dy) + n * a.dy_batch + t * a.dy_token + c), dz);
            if (a.silu) {
              float z[V];
#pragma unroll
              for (int k = 0; k < V; ++k) z[k] = fmaf(w[0][k], x[k], bias[k]);
#pragma unroll
              for (int o = 1; o < KT; ++o)
                if (o < a.K)
#pragma unroll
                  for (int k = 0; k < V; ++k) z[k] = fmaf(w[o][k], old[o - 1][k], z[k]);
#pragma unroll
              for (int k = 0; k < V; ++k) dz[k] *= silu_slope(z[k]);
            }
            if (t < t1) {
#pragma unroll
              for (int k = 0; k < V; ++k) db[k] += dz[k], dw[0][k] = fmaf(dz[k], x[k], dw[0][k]);
#pragma unroll
              for (int o = 1; o < KT; ++o)
                if (o < a.K)
#pragma unroll
                  for (int k = 0; k < V; ++k) dw[o][k] = fmaf(dz[k], old[o - 1][k], dw[o][k]);
            }
            const long long slot = t - q.end + a.K - 1;  // of the window that the sequence leaves
            if (a.dstate_out && slot >= 0) {
              const long long row = static_cast<long long>(q.s) * (a.K - 1) + slot;
              unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.dstate_out) + row * a.C + c), next[0]);
            }
            const long long pos = t - q.begin;
#pragma unroll
            for (int o = 0; o < KT; ++o)
              if (o < a.K && o <= pos)
#pragma unroll
                for (int k = 0; k < V; ++k) next[o][k] = fmaf(w[o][k], dz[k], next[o][k]);
#pragma unroll
            for (int o = KT - 2; o > 0; --o)
#pragma unroll
              for (int k = 0; k < V; ++k) old[o][k] = old[o - 1][k];
#pragma unroll
            for (int k = 0; k < V; ++k) old[0][k] = x[k];
          }
        }
        const long long done = t - (a.K - 1);
        if (done >= t0 && done < t1) {
          T* out = dx + (n * a.L + done) * a.C + c;
#pragma unroll
          for (int o = 0; o < KT; ++o)
            if (o == a.K - 1) {
              if (used[o]) store_vec<T, V>(out, next[o]);
              else if (a.fill) store_zero<T, V>(out);
            }
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        db_sum[k] += db[k];
#pragma unroll
        for (int o = 0; o < KT; ++o) dw_sum[o][k] += dw[o][k];
      }
    }
  }
  // the block's eight threads of each channel, in order
  __shared__ float sums[kGradRows][kGradLanes * V];
#pragma unroll
  for (int o = 0; o <= KT; ++o) {
    if (o < KT && o >= a.K) continue;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) sums[threadIdx.y][threadIdx.x * V + k] = o < KT ? dw_sum[o < KT ? o : 0][k] : db_sum[k];
    __syncthreads();
    const int row = o < KT ? a.K - 1 - o : a.K;
    for (int k = threadIdx.y * kGradLanes + threadIdx.x; k < kGradLanes * V; k += kGradLanes * kGradRows) {
      const int ch = blockIdx.x * kGradLanes * V + k;
      if (ch >= a.C) continue;
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < kGradRows; ++r) sum += sums[r][k];
      a.part[(static_cast<long long>(blockIdx.y) * (a.K + 1) + row) * a.C + ch] = sum;
    }
  }
}

// dw and dbias: the blocks' partial sums [blocks][K + 1][C] added in order.
template <typename T>
__global__ void __launch_bounds__(256) conv_causal_sum_kernel(const float* __restrict__ part, T* dw, T* dbias, int blocks,
                                                              int C, int K) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * 256 + threadIdx.x, j = blockIdx.y;
  if (c >= C) return;
  float sum = 0.f;
  for (int b = 0; b < blocks; ++b) sum += part[(static_cast<long long>(b) * (K + 1) + j) * C + c];
  if (j < K) dw[static_cast<long long>(c) * K + j] = from_f32<T>(sum);
  else if (dbias) dbias[c] = from_f32<T>(sum);
}

// dstate: the window's rows are read by a sequence's first K - 1 tokens, and
// passed on by a sequence of fewer.  A thread a (sequence, channel).
template <typename T, bool Q8>
__global__ void __launch_bounds__(128) conv_causal_dstate_kernel(const CausalArgs a) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * 128 + threadIdx.x, K = a.K;
  if (c >= a.C) return;
  for (int s = blockIdx.y; s < a.N; s += gridDim.y) {
    const int n = a.cu ? 0 : s;
    SeqAt q{s, 0, a.L};
    if (a.cu) {
      q.begin = max(0LL, min(a.L, static_cast<long long>(__ldg(a.cu + s))));
      q.end = max(q.begin, min(a.L, static_cast<long long>(__ldg(a.cu + s + 1))));
    }
    const int len = static_cast<int>(min(q.end - q.begin, static_cast<long long>(K - 1)));
    float w[CONV_CAUSAL_MAX_K], row[2 * CONV_CAUSAL_MAX_K], d[CONV_CAUSAL_MAX_K];
    for (int j = 0; j < K; ++j) w[j] = to_f32<T>(static_cast<const T*>(a.w)[static_cast<long long>(c) * K + j]);
    // row[j]: the window's rows, then the first tokens
    for (int j = 0; j < K - 1 + len; ++j) {
      float v[1];
      row_or_window<T, 1, Q8>(v, a, n, q, q.begin + j - (K - 1), c);
      row[j] = v[0];
    }
    for (int m = 0; m < K - 1; ++m) d[m] = 0.f;
    for (int p = 0; p < len; ++p) {
      const long long t = q.begin + p;
      float dz = to_f32<T>(static_cast<const T*>(a.dy)[n * a.dy_batch + t * a.dy_token + c]);
      if (a.silu) {
        float z = a.bias ? to_f32<T>(static_cast<const T*>(a.bias)[c]) : 0.f;
        for (int j = 0; j < K; ++j) z = fmaf(w[j], row[p + j], z);
        dz *= silu_slope(z);
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
  CausalArgs f = {};
  f.w = a.w;
  f.bias = a.bias;
  f.K = a.K;
  float w[KT][V], bias[V], old[KT - 1][V];
  load_filter<T, KT, V>(w, bias, f, c);
  T* window = static_cast<T*>(a.state) + static_cast<long long>(slot) * (a.K - 1) * a.C + c;
#pragma unroll
  for (int o = 0; o < KT - 1; ++o)
    if (o < a.K - 1) {
      const Raw<T, V> raw = *reinterpret_cast<const Raw<T, V>*>(window + static_cast<long long>(a.K - 2 - o) * a.C);
      unpack<T, V>(raw, old[o]);
    }
  do {
    float x[V], z[V];
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.x) + b * a.xs + c), x);
#pragma unroll
    for (int k = 0; k < V; ++k) z[k] = fmaf(w[0][k], x[k], bias[k]);
#pragma unroll
    for (int o = 1; o < KT; ++o)
      if (o < a.K)
#pragma unroll
        for (int k = 0; k < V; ++k) z[k] = fmaf(w[o][k], old[o - 1][k], z[k]);
#pragma unroll
    for (int o = KT - 2; o > 0; --o)
#pragma unroll
      for (int k = 0; k < V; ++k) old[o][k] = old[o - 1][k];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      old[0][k] = x[k];
      if (a.silu) z[k] = z[k] * causal_sigmoid(z[k]);
    }
    store_vec<T, V>(y + static_cast<long long>(b) * a.C, z);
    if (!(others & 2)) break;
    for (++b; b < a.B && __ldg(a.index + b) != slot;) ++b;
  } while (b < a.B);
#pragma unroll
  for (int o = 0; o < KT - 1; ++o)
    if (o < a.K - 1) store_vec<T, V>(window + static_cast<long long>(a.K - 2 - o) * a.C, old[o]);
}

}  // namespace convfwd

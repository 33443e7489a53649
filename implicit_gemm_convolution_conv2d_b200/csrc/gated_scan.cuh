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

#include "seq_common.cuh"

namespace convfwd {

struct GateValues {
  float s, g, a, m;
};

__device__ __forceinline__ float fast_sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

__device__ __forceinline__ GateValues gate_values(float r, float i, float decay) {
  GateValues o;
  o.s = fast_sigmoid(r);
  o.g = fast_sigmoid(i);
  const float l = -decay * o.s;
  // 1 - e^l = -l (1 + l/2 + l^2/6 + l^3/24 + l^4/120 + l^5/720); the next term
  // is l^6/5040 < 5e-8 of it for |l| < 1/4
  float p = fmaf(l, 1.f / 720.f, 1.f / 120.f);
  p = fmaf(l, p, 1.f / 24.f);
  p = fmaf(l, p, 1.f / 6.f);
  p = fmaf(l, p, 0.5f);
  p = fmaf(l, p, 1.f);
  const float far = __expf(l);
  const bool near1 = l > -0.25f;
  const float E = near1 ? -l * p : 1.f - far;
  o.a = near1 ? 1.f - E : far;
  o.m = sqrtf(E * (2.f - E));
  return o;
}

struct ScanIn {  // a strided tensor, or a checkpoint
  const void* p;
  const unsigned char* scale;
  long long batch, token;
};

struct ScanArgs {
  ScanIn x, r, i, dy;
  const float *decay, *h0, *dh_last;
  const int* cu;
  void *y, *dx, *dr, *di;
  float *h_last, *states, *ddecay, *dh0, *part;
  const float* states_in;
  int N, C, packed, fill;
  long long L;
};

// element (n, t, c) of an input
template <typename T>
__device__ __forceinline__ float scan_value(const ScanIn& in, const ScanArgs& a, int n, long long t, int c) {
  const long long at = n * in.batch + t * in.token + c;
  if (!in.scale) return to_f32<T>(static_cast<const T*>(in.p)[at]);
  const int nblk = (a.C + ACT8_BLOCK - 1) / ACT8_BLOCK;
  const long long row = static_cast<long long>(n) * a.L + t;
  return static_cast<float>(static_cast<const signed char*>(in.p)[at]) *
         act8_step(in.scale[row * nblk + c / ACT8_BLOCK]);
}

constexpr int kScanThreads = 64;

// A thread a channel of a sequence, one token after the other.
template <typename T>
__global__ void __launch_bounds__(kScanThreads) gated_scan_kernel(const ScanArgs a) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * kScanThreads + threadIdx.x, s = blockIdx.y;
  if (c >= a.C) return;
  T* y = static_cast<T*>(a.y);
  const int n = a.packed ? 0 : s;
  const long long row0 = static_cast<long long>(n) * a.L, blocks = (a.L + 63) / 64;
  long long t0 = 0, t1 = a.L;
  if (a.packed) {
    t0 = max(0LL, min(a.L, static_cast<long long>(a.cu[s])));
    t1 = max(t0, min(a.L, static_cast<long long>(a.cu[s + 1])));
  }
  const float decay = a.decay[c];
  float h = a.h0 ? a.h0[static_cast<long long>(s) * a.C + c] : 0.f;
  for (long long t = t0; t < t1; ++t) {
    if (a.states && t % 64 == 0) a.states[(n * blocks + t / 64) * a.C + c] = t == t0 ? 0.f : h;
    const GateValues v =
        gate_values(scan_value<T>(a.r, a, n, t, c), scan_value<T>(a.i, a, n, t, c), decay);
    h = fmaf(v.a, h, v.m * v.g * scan_value<T>(a.x, a, n, t, c));
    y[(row0 + t) * a.C + c] = from_f32<T>(h);
  }
  if (a.h_last) a.h_last[static_cast<long long>(s) * a.C + c] = h;
  if (a.packed && s == a.N - 1) {
    for (long long t = t1; t < a.L; ++t) {
      if (a.fill) y[t * a.C + c] = from_f32<T>(0.f);
      if (a.states && t % 64 == 0) a.states[t / 64 * a.C + c] = 0.f;
    }
  }
  if (a.packed && s == 0)
    for (long long t = 0; t < t0; ++t) {
      if (a.fill) y[t * a.C + c] = from_f32<T>(0.f);
      if (a.states && t % 64 == 0) a.states[t / 64 * a.C + c] = 0.f;
    }
}

// A thread a channel of a sequence: blocks of 64 rows from the last to the
// first, the states of each recomputed from the one in front of it.
template <typename T>
__global__ void __launch_bounds__(kScanThreads) gated_scan_grad_kernel(const ScanArgs a) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * kScanThreads + threadIdx.x, s = blockIdx.y;
  if (c >= a.C) return;
  T *dx = static_cast<T*>(a.dx), *dr = static_cast<T*>(a.dr), *di = static_cast<T*>(a.di);
  const int n = a.packed ? 0 : s;
  const long long row0 = static_cast<long long>(n) * a.L, blocks = (a.L + 63) / 64;
  long long t0 = 0, t1 = a.L;
  if (a.packed) {
    t0 = max(0LL, min(a.L, static_cast<long long>(a.cu[s])));
    t1 = max(t0, min(a.L, static_cast<long long>(a.cu[s + 1])));
  }
  const long long sc = static_cast<long long>(s) * a.C + c;
  const float decay = a.decay[c];
  float carry = a.dh_last ? a.dh_last[sc] : 0.f, sum = 0.f;
  float h[65];
  for (long long end = t1; end > t0;) {
    const long long begin = max(t0, (end - 1) / 64 * 64);
    h[0] = begin == t0 ? (a.h0 ? a.h0[sc] : 0.f) : a.states_in[(n * blocks + begin / 64) * a.C + c];
    for (long long t = begin; t < end; ++t) {
      const GateValues v =
          gate_values(scan_value<T>(a.r, a, n, t, c), scan_value<T>(a.i, a, n, t, c), decay);
      h[t - begin + 1] = fmaf(v.a, h[t - begin], v.m * v.g * scan_value<T>(a.x, a, n, t, c));
    }
    float part = 0.f;
    for (long long t = end - 1; t >= begin; --t) {
      const GateValues v =
          gate_values(scan_value<T>(a.r, a, n, t, c), scan_value<T>(a.i, a, n, t, c), decay);
      const float x = scan_value<T>(a.x, a, n, t, c), G = scan_value<T>(a.dy, a, n, t, c) + carry;
      carry = v.a * G;
      const float back = v.m > 0.f ? v.a * v.g * x / v.m : 0.f;
      const float dl = carry * (h[t - begin] - back);
      const long long at = (row0 + t) * a.C + c;
      dx[at] = from_f32<T>(G * v.m * v.g);
      di[at] = from_f32<T>(G * v.m * x * v.g * (1.f - v.g));
      dr[at] = from_f32<T>(-decay * dl * v.s * (1.f - v.s));
      part = fmaf(-v.s, dl, part);
    }
    sum += part;
    end = begin;
  }
  if (a.dh0) a.dh0[sc] = carry;
  a.part[sc] = sum;
  if (a.packed && a.fill && s == a.N - 1)
    for (long long t = t1; t < a.L; ++t) dx[t * a.C + c] = dr[t * a.C + c] = di[t * a.C + c] = from_f32<T>(0.f);
  if (a.packed && a.fill && s == 0)
    for (long long t = 0; t < t0; ++t) dx[t * a.C + c] = dr[t * a.C + c] = di[t * a.C + c] = from_f32<T>(0.f);
}

// ddecay: the partial sums added in order.
__global__ void __launch_bounds__(kScanThreads) gated_scan_sum_kernel(const float* part, float* out, int n, int C) {
  ptx::pdl_wait_prev();
  const int c = blockIdx.x * kScanThreads + threadIdx.x;
  if (c >= C) return;
  float sum = 0.f;
  for (int k = 0; k < n; ++k) sum += part[static_cast<long long>(k) * C + c];
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
  float decay[V], h[V];
  float* hp = a.h + static_cast<long long>(slot) * a.C + c;
#pragma unroll
  for (int k = 0; k < V; ++k) decay[k] = __ldg(a.decay + c + k), h[k] = hp[k];
  do {
    float x[V], r[V], i[V];
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.x) + b * a.xs + c), x);
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.r) + b * a.rs + c), r);
    unpack<T, V>(load_raw<T, V>(static_cast<const T*>(a.i) + b * a.is + c), i);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const GateValues v = gate_values(r[k], i[k], decay[k]);
      h[k] = fmaf(v.a, h[k], v.m * v.g * x[k]);
    }
    store_vec<T, V>(y + static_cast<long long>(b) * a.C, h);
    if (!(others & 2)) break;
    for (++b; b < a.B && __ldg(a.index + b) != slot;) ++b;
  } while (b < a.B);
#pragma unroll
  for (int k = 0; k < V; ++k) hp[k] = h[k];
}

}  // namespace convfwd

// seq_common.cuh -- what the sequence operators share: vectors of a row's
// channels, checkpoint values, the sequence that a packed row belongs to, and
// host-side checks of strided and contiguous buffers.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/conv_seq.h"
#include "conv_simt.cuh"  // to_f32, from_f32; ptx.cuh
#include "launch.cuh"

namespace convfwd {

// `BYTES` bytes of a row as one load or store.
template <int BYTES>
struct RawVec;
template <>
struct RawVec<1> { using type = uint8_t; };
template <>
struct RawVec<2> { using type = uint16_t; };
template <>
struct RawVec<4> { using type = uint32_t; };
template <>
struct RawVec<8> { using type = uint2; };
template <>
struct RawVec<16> { using type = uint4; };

// V consecutive channels as fp32.  The raw value is loaded first and unpacked
// from registers (see load_raw): a vector that is unpacked through its address
// compiles to narrow loads.
template <typename T, int V>
using Raw = typename RawVec<static_cast<int>(sizeof(T)) * V>::type;

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  return __ldg(reinterpret_cast<const Raw<T, V>*>(p));
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& raw, float (&v)[V]) {
  union {
    Raw<T, V> r;
    T e[V];
  } u;
  u.r = raw;
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = to_f32<T>(u.e[k]);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  union {
    Raw<T, V> r;
    T e[V];
  } u;
#pragma unroll
  for (int k = 0; k < V; ++k) u.e[k] = from_f32<T>(v[k]);
  *reinterpret_cast<Raw<T, V>*>(p) = u.r;
}

template <typename T, int V>
__device__ __forceinline__ void store_zero(T* p) {
  float z[V] = {};
  store_vec<T, V>(p, z);
}

// ---- V fp32 values at once ----------------------------------------------
// Two are one packed instruction (fma.rn.f32x2 and its kin issue once for two
// channels); each rounds as its scalar form does.
template <int V>
struct Vf {
  float v[V];
  __device__ __forceinline__ float& operator[](int k) { return v[k]; }
  __device__ __forceinline__ const float& operator[](int k) const { return v[k]; }
};

template <int V>
__device__ __forceinline__ Vf<V> splat(float x) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = x;
  return o;
}

__device__ __forceinline__ uint64_t pack2(const float* v) {
  uint64_t o;
  asm("mov.b64 %0, {%1, %2};" : "=l"(o) : "f"(v[0]), "f"(v[1]));
  return o;
}
__device__ __forceinline__ void unpack2(uint64_t x, float* v) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(x));
}

template <int V>
__device__ __forceinline__ Vf<V> fma_v(const Vf<V>& a, const Vf<V>& b, const Vf<V>& c) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k + 1 < V; k += 2) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pack2(a.v + k)), "l"(pack2(b.v + k)), "l"(pack2(c.v + k)));
    unpack2(d, o.v + k);
  }
  if constexpr (V & 1) o[V - 1] = fmaf(a[V - 1], b[V - 1], c[V - 1]);
  return o;
}
template <int V>
__device__ __forceinline__ Vf<V> mul_v(const Vf<V>& a, const Vf<V>& b) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k + 1 < V; k += 2) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(a.v + k)), "l"(pack2(b.v + k)));
    unpack2(d, o.v + k);
  }
  if constexpr (V & 1) o[V - 1] = a[V - 1] * b[V - 1];
  return o;
}
template <int V>
__device__ __forceinline__ Vf<V> add_v(const Vf<V>& a, const Vf<V>& b) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k + 1 < V; k += 2) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(a.v + k)), "l"(pack2(b.v + k)));
    unpack2(d, o.v + k);
  }
  if constexpr (V & 1) o[V - 1] = a[V - 1] + b[V - 1];
  return o;
}
template <int V>
__device__ __forceinline__ Vf<V> neg_v(const Vf<V>& a) {
  Vf<V> o;
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = -a[k];
  return o;
}

// The hardware's approximations, subnormals taken as zero: 2^x (2 ulp), 1 / x
// (1 ulp), sqrt(x) (2^-23).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// NaN where either is (fminf would drop it)
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// The step of a checkpoint's block: 2^(byte - 127), NaN for 255 and 0 for 0
// (whose elements are all 0).
__device__ __forceinline__ float act8_step(unsigned char s) {
  return __uint_as_float(s == 255 ? 0x7fc00000u : static_cast<unsigned>(s) << 23);
}

// The sequence of packed row t: the last s with cu[s] <= t, if t < cu[s+1];
// n where t is in none.  Whatever cu holds, the result is in [0, n].
__device__ __forceinline__ int seq_of_row(const int* __restrict__ cu, int n, long long t) {
  int lo = 0, hi = n;  // the number of ends cu[1..n] that are <= t
  while (lo < hi) {
    const int mid = lo + ((hi - lo) >> 1);  // the sum may pass 31 bits
    if (__ldg(cu + mid + 1) <= t) lo = mid + 1; else hi = mid;
  }
  if (lo < n && t < __ldg(cu + lo)) lo = n;  // in front of the first sequence
  return lo;
}

// Whether requests before and after row b name the same slot: bit 0 an earlier
// one, bit 1 a later one.  Called by whole warps; the answer is warp-uniform.  Each
// warp reads the whole index: nothing beside a launch at some hundred requests, the
// larger part of a step at tens of thousands.
__device__ __forceinline__ int same_slot(const int* __restrict__ index, int B, int b, int slot) {
  bool earlier = false, later = false;
  for (int k = threadIdx.x & 31; k < B; k += 32) {
    const bool same = __ldg(index + k) == slot;
    earlier |= same && k < b;
    later |= same && k > b;
  }
  return (__any_sync(0xffffffffu, earlier) ? 1 : 0) | (__any_sync(0xffffffffu, later) ? 2 : 0);
}

// The first `width` of V channels into a row of an output (all of them where rows
// are ALIGNED).
template <typename T, int V, bool ALIGNED>
__device__ __forceinline__ void put_row(T* p, int width, const Vf<V>& v) {
  if constexpr (ALIGNED) {
    store_vec<T, V>(p, v.v);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < width) p[k] = from_f32<T>(v[k]);
  }
}
struct SeqIn {  // a strided input, or a checkpoint where it has scales
  const void* p;
  const unsigned char* scale;
  long long batch, token;
};

// ---- host side ----------------------------------------------------------

struct Span {  // the bytes from a buffer's first element to its last
  uintptr_t lo = 0, hi = 0;
};

inline Span span_of(const void* p, long long bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p && bytes > 0 ? Span{a, a + static_cast<uintptr_t>(bytes)} : Span{0, 0};
}

inline bool spans_meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// True if an output meets an input or another output.
inline bool any_alias(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int k = 0; k < n_out; ++k) {
    for (int m = 0; m < n_in; ++m)
      if (spans_meet(outs[k], ins[m])) return true;
    for (int m = 0; m < k; ++m)
      if (spans_meet(outs[k], outs[m])) return true;
  }
  return false;
}

constexpr long long kSeqMaxElems = 1LL << 46;  // of a tensor, and of a stride: offsets stay far inside 64 bits

inline int elem_size(int dtype) { return dtype == CONV_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == CONV_F32 || dtype == CONV_F16 || dtype == CONV_BF16; }

// Tokens of a sequence, sequences and channels: places behind the last (a warp's
// share, a block of 32 channels) fit 32 bits too.
constexpr long long kSeqMaxCount = 0x7fffffffLL - 4096;

// N sequences of L rows of C channels (packed: L rows in all): sizes that fit.
inline bool seq_sizes_ok(int N, long long L, long long C, bool packed) {
  if (N < 0 || L < 0 || C <= 0 || N > kSeqMaxCount || L > kSeqMaxCount || C > kSeqMaxCount) return false;
  const long long rows = packed ? L : L * N;  // both below 2^31
  return rows <= kSeqMaxElems / C && N <= kSeqMaxElems / C;
}

// Elements from the first to behind the last of a strided input.
inline bool strided_extent(int N, long long L, long long C, bool packed, long long batch, long long token,
                           long long& elems) {
  if (batch < 0 || token < 0 || batch > kSeqMaxElems || token > kSeqMaxElems) return false;
  elems = 0;
  if (N == 0 && !packed) return true;
  if (L == 0) return true;
  const long long nb = packed ? 0 : N - 1;
  if (nb > 0 && batch > kSeqMaxElems / nb) return false;
  if (L > 1 && token > kSeqMaxElems / (L - 1)) return false;
  elems = nb * batch + (L - 1) * token + C;
  return true;
}

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of a strided input that start on `a`-byte boundaries.
inline bool rows_aligned(const void* p, long long batch, long long token, int esize, size_t a) {
  return aligned_to(p, a) && (batch * esize) % static_cast<long long>(a) == 0 &&
         (token * esize) % static_cast<long long>(a) == 0;
}

// SMs of the current device.
inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

}  // namespace convfwd

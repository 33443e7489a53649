// act8.cuh -- 8-bit activation checkpoints: pack and unpack.
//
// Per block of 32 channels the step 2^e is the least power of two with
// amax <= 127 * 2^e, found from amax's bits alone: 127 = 1.984375 * 2^6, so e
// is amax's exponent - 6, and one more where its mantissa is above 1.984375.
// The elements are x * 2^-e rounded to nearest even.  Scaling by a power of two
// is exact, so that is the only rounding, and a packed block is the same bits
// wherever it is computed.  A power of two, rather than amax / 127, also makes
// q * 2^e (7 bits and a sign) exact in the 16-bit types.  In the type's top step size
// the rounding stops at 63 steps (act8_limit).
//
// Bounds: 3.03 bytes an element of a 16-bit type, each way.  Measured, 8 x 4096 x
// 2560: pack bf16 50 us, 5.1 TB/s (78 % of the copy rate; ALU-bound at 14
// instructions an element), fp32 63 (6.7 TB/s); unpack bf16 41 us (94 %), fp32 89
// (73 %: its two 16-byte stores a thread lie 32 bytes apart).
#pragma once

#include <cstring>

#include "seq_common.cuh"

namespace convfwd {

// The step's byte (e + 127) from the bits of a block's largest magnitude.
__device__ __forceinline__ int act8_scale_byte(unsigned amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255;
  if (amax_bits == 0) return 0;
  return max(1, static_cast<int>((amax_bits + 0x1ffffu) >> 23) - 6);
}

// The bound of |q|: 127, but 63 in the one step size where 64 * 2^e is past the
// type's largest value (e = 10 for f16, 122 for bf16 and f32), and 0 in a block
// that is NaN anyway.
template <typename T>
__device__ __forceinline__ float act8_limit(int byte) {
  constexpr int kTop = std::is_same<T, __half>::value ? 137 : 249;
  return byte == 255 ? 0.f : byte >= kTop ? 63.f : 127.f;
}

__device__ __forceinline__ float act8_inverse_step(int byte) {
  return byte == 255 ? 0.f : __uint_as_float(static_cast<unsigned>(254 - byte) << 23);
}

// x / 2^e rounded to nearest even, in the last byte: the sum with 1.5 * 2^23 is
// rounded once, to a whole number (a conversion and its rounding would take the
// special functions' pipe).  inv = 2^-e.  Where |q| could pass the limit, and in
// a block that is NaN, it is held at it.
__device__ __forceinline__ unsigned act8_quant(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.f));
}
__device__ __forceinline__ unsigned act8_quant_held(float x, float inv, float limit) {
  return __float_as_uint(fminf(fmaxf(fmaf(x, inv, 12582912.f), 12582912.f - limit), 12582912.f + limit));
}
constexpr int kAct8Threads = 256;
constexpr int kAct8Unroll = 4;  // vectors of a thread, loaded together
constexpr int kAct8Vec = 8;     // channels of a thread: one 16-byte load of a 16-bit type, two of fp32

// The bits of the largest magnitude of a 16-byte vector, as fp32: magnitudes
// order as their bits, NaN above infinity.
template <typename T>
__device__ __forceinline__ unsigned act8_amax(const uint4& raw) {
  if constexpr (sizeof(T) == 4) {
    const unsigned m = 0x7fffffffu;
    return max(max(raw.x & m, raw.y & m), max(raw.z & m, raw.w & m));
  } else {
    const unsigned m = 0x7fff7fffu;
    const unsigned two = __vmaxu2(__vmaxu2(raw.x & m, raw.y & m), __vmaxu2(raw.z & m, raw.w & m));
    const unsigned short one = static_cast<unsigned short>(max(two & 0xffffu, two >> 16));
    T v;
    memcpy(&v, &one, 2);
    return __float_as_uint(to_f32<T>(v));
  }
}

// C % 8 == 0 and 16-byte aligned rows: four threads a block of 32 channels.
// Items are (row, channel vector), the vectors of a row padded to whole blocks.
template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_pack_kernel(const T* __restrict__ x, signed char* __restrict__ q, unsigned char* __restrict__ scale,
                     long long rows, int C, long long x_row) {
  constexpr int V = kAct8Vec, kGroup = ACT8_BLOCK / V, kWords = sizeof(T) == 4 ? 2 : 1;
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, nvec = nblk * kGroup;
  const long long items = rows * nvec;
  const long long first = static_cast<long long>(blockIdx.x) * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const int more_rows = kAct8Threads / nvec, more_vecs = kAct8Threads - more_rows * nvec;
  uint4 raw[kAct8Unroll][kWords];
  long long row[kAct8Unroll];
  int cv[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    if (u == 0) {
      row[0] = items <= 0x7fffffffLL ? static_cast<int>(first) / nvec : first / nvec;
      cv[0] = static_cast<int>(first - row[0] * nvec);
    } else {  // kAct8Threads items on, without another division
      cv[u] = cv[u - 1] + more_vecs;
      row[u] = row[u - 1] + more_rows;
      if (cv[u] >= nvec) cv[u] -= nvec, ++row[u];
    }
    const bool in = first + u * kAct8Threads < items && cv[u] * V < C;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      raw[u][k] = make_uint4(0, 0, 0, 0);
      if (in) raw[u][k] = __ldg(reinterpret_cast<const uint4*>(x + row[u] * x_row + cv[u] * V) + k);
    }
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    unsigned amax = act8_amax<T>(raw[u][0]);
    if constexpr (kWords == 2) amax = max(amax, act8_amax<T>(raw[u][kWords - 1]));
#pragma unroll
    for (int o = 1; o < kGroup; o *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int byte = act8_scale_byte(amax);
    const float inv = act8_inverse_step(byte), limit = act8_limit<T>(byte);
    float v[V];
    if constexpr (kWords == 2) {
      float lo[4], hi[4];
      unpack<float, 4>(raw[u][0], lo);
      unpack<float, 4>(raw[u][kWords - 1], hi);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = lo[k], v[4 + k] = hi[k];
    } else {
      unpack<T, V>(raw[u][0], v);
    }
    unsigned n[V];
    if (limit == 127.f) {
#pragma unroll
      for (int k = 0; k < V; ++k) n[k] = act8_quant(v[k], inv);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) n[k] = act8_quant_held(v[k], inv, limit);
    }
    if (first + u * kAct8Threads < items) {
      if (cv[u] * V < C) {
        unsigned w[V / 4];
#pragma unroll
        for (int k = 0; k < V / 4; ++k)
          w[k] = __byte_perm(__byte_perm(n[4 * k], n[4 * k + 1], 0x0040), __byte_perm(n[4 * k + 2], n[4 * k + 3], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(q + row[u] * C + cv[u] * V) = make_uint2(w[0], w[1]);
      }
      if (cv[u] % kGroup == 0) scale[row[u] * nblk + cv[u] / kGroup] = static_cast<unsigned char>(byte);
    }
  }
}

// Any C, any alignment: a warp kAct8Unroll blocks of 32 channels of a row.
template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_pack_any_kernel(const T* __restrict__ x, signed char* __restrict__ q, unsigned char* __restrict__ scale,
                         long long rows, int C, long long x_row) {
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, lane = threadIdx.x & 31;
  const int groups = (nblk + kAct8Unroll - 1) / kAct8Unroll;
  const long long items = rows * groups, step = static_cast<long long>(gridDim.x) * (kAct8Threads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kAct8Threads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long row = items <= 0x7fffffffLL ? static_cast<int>(it) / groups : it / groups;
    const int blk = static_cast<int>(it - row * groups) * kAct8Unroll, c = blk * ACT8_BLOCK + lane;
    const T* from = x + row * x_row + c;
    signed char* to = q + row * C + c;
    float v[kAct8Unroll];
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) v[u] = c + u * ACT8_BLOCK < C ? to_f32<T>(from[u * ACT8_BLOCK]) : 0.f;
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u) {
      const int byte = act8_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[u]) & 0x7fffffffu));
      if (c + u * ACT8_BLOCK < C)
        to[u * ACT8_BLOCK] = static_cast<signed char>(act8_quant_held(v[u], act8_inverse_step(byte), act8_limit<T>(byte)));
      if (lane == 0 && blk + u < nblk) scale[row * nblk + blk + u] = static_cast<unsigned char>(byte);
    }
  }
}

// C % 8 == 0 (any block: 8 divides 32) and 16-byte aligned y.
template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_unpack_kernel(const signed char* __restrict__ q, const unsigned char* __restrict__ scale, T* __restrict__ y,
                       long long rows, int C) {
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, nvec = C / kAct8Vec;
  const long long items = rows * nvec;
  const long long first = static_cast<long long>(blockIdx.x) * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  const int more_rows = kAct8Threads / nvec, more_vecs = kAct8Threads - more_rows * nvec;
  long long row = 0;
  int cv = 0;
  uint2 raw[kAct8Unroll];
  unsigned char sb[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const long long it = first + u * kAct8Threads;
    if (u == 0) {
      row = items <= 0x7fffffffLL ? static_cast<int>(first) / nvec : first / nvec;
      cv = static_cast<int>(first - row * nvec);
    } else {
      cv += more_vecs;
      row += more_rows;
      if (cv >= nvec) cv -= nvec, ++row;
    }
    raw[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (it < items) {
      raw[u] = __ldg(reinterpret_cast<const uint2*>(q + it * kAct8Vec));
      sb[u] = __ldg(scale + row * nblk + cv / (ACT8_BLOCK / kAct8Vec));
    }
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const long long it = first + u * kAct8Threads;
    if (it >= items) continue;
    union {
      uint2 r;
      signed char e[8];
    } in;
    in.r = raw[u];
    const float step = act8_step(sb[u]);
    float v[kAct8Vec];
#pragma unroll
    for (int k = 0; k < kAct8Vec; ++k) v[k] = static_cast<float>(in.e[k]) * step;
    if constexpr (sizeof(T) == 4) {
      const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
      store_vec<float, 4>(y + it * kAct8Vec, lo);
      store_vec<float, 4>(y + it * kAct8Vec + 4, hi);
    } else {
      store_vec<T, kAct8Vec>(y + it * kAct8Vec, v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_unpack_any_kernel(const signed char* __restrict__ q, const unsigned char* __restrict__ scale,
                           T* __restrict__ y, long long rows, int C) {
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, lane = threadIdx.x & 31;
  const int groups = (nblk + kAct8Unroll - 1) / kAct8Unroll;
  const long long items = rows * groups, step = static_cast<long long>(gridDim.x) * (kAct8Threads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kAct8Threads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long row = items <= 0x7fffffffLL ? static_cast<int>(it) / groups : it / groups;
    const int blk = static_cast<int>(it - row * groups) * kAct8Unroll, c = blk * ACT8_BLOCK + lane;
    signed char v[kAct8Unroll];
    unsigned char sb[kAct8Unroll];
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u)
      if (c + u * ACT8_BLOCK < C) v[u] = q[row * C + c + u * ACT8_BLOCK], sb[u] = scale[row * nblk + blk + u];
#pragma unroll
    for (int u = 0; u < kAct8Unroll; ++u)
      if (c + u * ACT8_BLOCK < C) y[row * C + c + u * ACT8_BLOCK] = from_f32<T>(static_cast<float>(v[u]) * act8_step(sb[u]));
  }
}

}  // namespace convfwd

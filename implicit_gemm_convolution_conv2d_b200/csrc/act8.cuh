// act8.cuh -- 8-bit activation checkpoints: pack and unpack.
//
// Per block of 32 channels the step 2^e is the least power of two with
// amax <= 127 * 2^e, found from amax's bits alone: 127 = 1.984375 * 2^6, so e
// is amax's exponent - 6, and one more where its mantissa is above 1.984375.
// The elements are x * 2^-e rounded to nearest even.  Scaling by a power of two
// is exact, so that is the only rounding, and a packed block is the same bits
// wherever it is computed.  A power of two, rather than amax / 127, also makes
// q * 2^e (7 bits and a sign) exact in the 16-bit types.
#pragma once

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

// x / 2^e, rounded: inv = 2^-e.
__device__ __forceinline__ int act8_quant(float x, float inv, float limit) {
  return static_cast<int>(fminf(fmaxf(rintf(x * inv), -limit), limit));
}

__device__ __forceinline__ float act8_inverse_step(int byte) {
  return byte == 255 ? 0.f : __uint_as_float(static_cast<unsigned>(254 - byte) << 23);
}

constexpr int kAct8Threads = 256;
constexpr int kAct8Vec = 8;     // channels of a thread: 16 bytes of a 16-bit type
constexpr int kAct8Unroll = 4;  // vectors of a thread, loaded together

// C % 8 == 0 and 16-byte aligned rows: four threads a block of 32 channels.
// Items are (row, channel vector), the vectors of a row padded to whole blocks.
template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_pack_kernel(const T* __restrict__ x, signed char* __restrict__ q, unsigned char* __restrict__ scale,
                     long long rows, int C, long long x_row) {
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, nvec = nblk * (ACT8_BLOCK / kAct8Vec);
  const long long items = rows * nvec;
  const long long first = static_cast<long long>(blockIdx.x) * (kAct8Threads * kAct8Unroll) + threadIdx.x;
  constexpr int kWords = sizeof(T) == 4 ? 2 : 1;
  uint4 raw[kAct8Unroll][kWords];
  long long row[kAct8Unroll];
  int cv[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const long long it = first + u * kAct8Threads;
    row[u] = it / nvec;
    cv[u] = static_cast<int>(it - row[u] * nvec);
    const bool in = it < items && cv[u] * kAct8Vec < C;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      raw[u][k] = in ? __ldg(reinterpret_cast<const uint4*>(x + row[u] * x_row + cv[u] * kAct8Vec) + k)
                     : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    float v[kAct8Vec];
    if constexpr (sizeof(T) == 4) {
      float lo[4], hi[4];
      unpack<float, 4>(raw[u][0], lo);
      unpack<float, 4>(raw[u][1], hi);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = lo[k], v[4 + k] = hi[k];
    } else {
      unpack<T, kAct8Vec>(raw[u][0], v);
    }
    unsigned amax = 0;  // magnitudes order as their bits, NaN above infinity
#pragma unroll
    for (int k = 0; k < kAct8Vec; ++k) amax = max(amax, __float_as_uint(v[k]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int byte = act8_scale_byte(amax);
    const float inv = act8_inverse_step(byte), limit = act8_limit<T>(byte);
    union {
      uint2 r;
      signed char e[8];
    } out;
#pragma unroll
    for (int k = 0; k < kAct8Vec; ++k) out.e[k] = static_cast<signed char>(act8_quant(v[k], inv, limit));
    if (first + u * kAct8Threads < items) {
      if (cv[u] * kAct8Vec < C) *reinterpret_cast<uint2*>(q + row[u] * C + cv[u] * kAct8Vec) = out.r;
      if ((cv[u] & 3) == 0) scale[row[u] * nblk + (cv[u] >> 2)] = static_cast<unsigned char>(byte);
    }
  }
}

// Any C, any alignment: a warp a block of 32 channels.
template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_pack_any_kernel(const T* __restrict__ x, signed char* __restrict__ q, unsigned char* __restrict__ scale,
                         long long rows, int C, long long x_row) {
  ptx::pdl_wait_prev();
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK, lane = threadIdx.x & 31;
  const long long items = rows * nblk, step = static_cast<long long>(gridDim.x) * (kAct8Threads / 32);
  for (long long it = static_cast<long long>(blockIdx.x) * (kAct8Threads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long row = it / nblk;
    const int blk = static_cast<int>(it - row * nblk), c = blk * ACT8_BLOCK + lane;
    const float v = c < C ? to_f32<T>(x[row * x_row + c]) : 0.f;
    const unsigned amax = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
    const int byte = act8_scale_byte(amax);
    if (c < C) q[row * C + c] = static_cast<signed char>(act8_quant(v, act8_inverse_step(byte), act8_limit<T>(byte)));
    if (lane == 0) scale[row * nblk + blk] = static_cast<unsigned char>(byte);
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
  uint2 raw[kAct8Unroll];
  unsigned char sb[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const long long it = first + u * kAct8Threads;
    raw[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (it < items) {
      const long long row = it / nvec;
      raw[u] = __ldg(reinterpret_cast<const uint2*>(q + it * kAct8Vec));
      sb[u] = __ldg(scale + row * nblk + static_cast<int>(it - row * nvec) / (ACT8_BLOCK / kAct8Vec));
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
  const int nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK;
  const long long items = rows * C, step = static_cast<long long>(gridDim.x) * kAct8Threads;
  for (long long it = static_cast<long long>(blockIdx.x) * kAct8Threads + threadIdx.x; it < items; it += step) {
    const long long row = it / C;
    const int c = static_cast<int>(it - row * C);
    y[it] = from_f32<T>(static_cast<float>(q[it]) * act8_step(scale[row * nblk + c / ACT8_BLOCK]));
  }
}

}  // namespace convfwd

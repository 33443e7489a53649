// seq_tile.cuh -- rows of 64 channels on their way through shared memory.
//
// Each warp copies its own rows of the next turn there while it works on this
// one: 16 bytes an instruction and no registers, and only the warp itself waits
// for them.  Rows that are not 16-byte aligned (ALIGNED false) go element by
// element through registers.  A lane then reads two neighbouring channels of a
// row, a conflict-free 128 or 256 bytes a warp, at addresses known beforehand.
#pragma once

#include "ptx.cuh"
#include "seq_common.cuh"

namespace convfwd {

template <typename T, int STEPS>
struct alignas(16) RowTile {
  T v[STEPS][64];
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");  // zeros where it is not
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// Walks along an input, a warp's STEPS rows of 64 channels a turn, zeros outside
// of it.  The address of the lane's first element moves on by addition.
template <typename T, int STEPS, bool ALIGNED>
struct TileWalk {
  static constexpr int kPer = 16 / sizeof(T), kRow = 64 / kPer, kRows = 32 / kRow;  // elements a copy, copies a row, rows at once
  const T* p;       // of the lane's first row and channel
  long long token;  // elements from row to row

  // from row t0 on; `width` channels from c0 on are there
  __device__ __forceinline__ void start(const SeqIn& in, int n, long long t0, int c0) {
    const int lane = threadIdx.x & 31;
    token = in.token;
    p = static_cast<const T*>(in.p) + n * in.batch + c0 + t0 * token;
    if constexpr (ALIGNED) p += lane / kRow * token + lane % kRow * kPer;
  }
  // Copies the rows into `tile`: `rows` of them are there (any number: none
  // below 1, all from STEPS on).  Whole warps, behind their last use of the tile.
  __device__ __forceinline__ void load(RowTile<T, STEPS>& tile, int rows, int width) const {
    const int lane = threadIdx.x & 31;
    if constexpr (ALIGNED) {
      const int row = lane / kRow, col = lane % kRow * kPer;
      const int mine = col < width ? rows - row : 0;
      T* to = &tile.v[row][col];
      const T* from = p;
#pragma unroll
      for (int j = 0; j < STEPS; j += kRows) {
        copy16(to + j * 64, from, j < mine);
        if (j + kRows < mine) from += kRows * token;  // never behind the last row
      }
    } else {
      T v[STEPS][2];  // loaded together
      const T* from = p + lane;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        v[j][0] = j < rows && lane < width ? from[0] : T(0.f);
        v[j][1] = j < rows && lane + 32 < width ? from[32] : T(0.f);
        from += token;
      }
#pragma unroll
      for (int j = 0; j < STEPS; ++j) tile.v[j][lane] = v[j][0], tile.v[j][lane + 32] = v[j][1];
    }
  }
  __device__ __forceinline__ void next(long long span) { p += span * token; }
};

// Sets the rows whose bit in `used` is 0.  Whole warps.
template <typename T, int STEPS>
__device__ __forceinline__ void void_rows(RowTile<T, STEPS>& tile, unsigned used, T with) {
  const int lane = threadIdx.x & 31;
  for (int j = 0; j < STEPS; ++j)
    if (!(used >> j & 1)) tile.v[j][lane] = tile.v[j][lane + 32] = with;
}

template <typename T, int STEPS>
__device__ __forceinline__ Raw<T, 2> row_pair(const RowTile<T, STEPS>& tile, int j, int lane) {
  return *reinterpret_cast<const Raw<T, 2>*>(&tile.v[j][2 * lane]);
}

// Eight rows of a checkpoint, from row `first` of the tile on, in place: their
// bytes lie one after the other at the beginning of those rows, and are exact in
// T.  16 a lane, of one row and one block of 32; `byte` is that block's step's.
// Whole warps.
template <typename T, int STEPS>
__device__ __forceinline__ void expand8(RowTile<T, STEPS>& tile, int first, int byte) {
  const int lane = threadIdx.x & 31;
  const uint4 raw = reinterpret_cast<const uint4*>(&tile.v[first][0])[lane];
  const float step = act8_step(static_cast<unsigned char>(byte));
  __syncwarp();
  T* to = &tile.v[first + lane / 4][lane % 4 * 16];
  const unsigned words[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // q + 128 as the last byte of 2^23: a conversion would take the special functions' pipe
    const unsigned biased = words[q] ^ 0x80808080u;
    Vf<4> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7650 + k));
    v = mul_v(add_v(v, splat<4>(-8388736.f)), splat<4>(step));
    store_vec<T, 4>(to + 4 * q, v.v);
  }
  __syncwarp();
}

// Moves the bytes of rows 8 k .. 8 k + 7, which lie behind those of the rows in
// front of them, to the beginning of the tile's row 8 k.  Whole warps; the last
// eight first.
template <typename T, int STEPS>
__device__ __forceinline__ void move8(RowTile<T, STEPS>& tile, int k) {
  if (k == 0) return;
  const int lane = threadIdx.x & 31;
  const uint4 raw = reinterpret_cast<const uint4*>(&tile.v[0][0])[32 * k + lane];
  __syncwarp();
  reinterpret_cast<uint4*>(&tile.v[8 * k][0])[lane] = raw;
  __syncwarp();
}

}  // namespace convfwd

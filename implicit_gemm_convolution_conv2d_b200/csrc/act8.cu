// act8.cu -- C ABI of the 8-bit activation checkpoints (see act8.cuh).
#include "act8.cuh"

using namespace convfwd;

namespace {

template <typename T>
int pack(const void* x, signed char* q, unsigned char* scale, long long rows, int C, long long x_row,
         cudaStream_t st) {
  const T* xt = static_cast<const T*>(x);
  const long long nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK;
  cudaError_t e;
  if (C % kAct8Vec == 0 && rows_aligned(x, 0, x_row, sizeof(T), 16) && aligned_to(q, 8)) {
    const long long blocks = (rows * nblk * (ACT8_BLOCK / kAct8Vec) + kAct8Threads * kAct8Unroll - 1) /
                             (kAct8Threads * kAct8Unroll);
    if (blocks > 0x7fffffffLL) return CONV_EUNSUPPORTED;
    e = launch_pdl(act8_pack_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kAct8Threads), 0, st, 1, xt, q,
                   scale, rows, C, x_row);
  } else {
    const long long blocks = std::min<long long>((rows * ((nblk + kAct8Unroll - 1) / kAct8Unroll) + 7) / 8, 16LL * sm_count());
    e = launch_pdl(act8_pack_any_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kAct8Threads), 0, st, 1, xt, q,
                   scale, rows, C, x_row);
  }
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

template <typename T>
int unpack_rows(const signed char* q, const unsigned char* scale, void* y, long long rows, int C, cudaStream_t st) {
  T* yt = static_cast<T*>(y);
  cudaError_t e;
  if (C % kAct8Vec == 0 && aligned_to(y, 16) && aligned_to(q, 8)) {
    const long long blocks =
        (rows * (C / kAct8Vec) + kAct8Threads * kAct8Unroll - 1) / (kAct8Threads * kAct8Unroll);
    if (blocks > 0x7fffffffLL) return CONV_EUNSUPPORTED;
    e = launch_pdl(act8_unpack_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kAct8Threads), 0, st, 1, q, scale,
                   yt, rows, C);
  } else {
    const long long nblk = (C + ACT8_BLOCK - 1) / ACT8_BLOCK;
    const long long blocks =
        std::min<long long>((rows * ((nblk + kAct8Unroll - 1) / kAct8Unroll) + 7) / 8, 16LL * sm_count());
    e = launch_pdl(act8_unpack_any_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(kAct8Threads), 0, st, 1, q,
                   scale, yt, rows, C);
  }
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

}  // namespace

extern "C" {

int act8_pack(const void* x, signed char* q, unsigned char* scale, long long rows, int C, long long x_row, int dtype,
              conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  if (rows < 0 || C <= 0 || C > kSeqMaxCount || rows > kSeqMaxElems / C) return CONV_EINVAL;
  long long xe;
  if (x_row < 0 || x_row > kSeqMaxElems || (rows > 1 && x_row > kSeqMaxElems / (rows - 1))) return CONV_EINVAL;
  if (rows == 0) return CONV_OK;
  xe = (rows - 1) * x_row + C;
  if (!x || !q || !scale) return CONV_EINVAL;
  const int es = elem_size(dtype);
  if (!aligned_to(x, es)) return CONV_EALIGN;
  const Span in = span_of(x, xe * es);
  const Span outs[2] = {span_of(q, rows * C), span_of(scale, rows * ((C + ACT8_BLOCK - 1LL) / ACT8_BLOCK))};
  if (any_alias(outs, 2, &in, 1)) return CONV_EALIAS;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CONV_F32) return pack<float>(x, q, scale, rows, C, x_row, st);
  if (dtype == CONV_F16) return pack<__half>(x, q, scale, rows, C, x_row, st);
  return pack<__nv_bfloat16>(x, q, scale, rows, C, x_row, st);
}

int act8_unpack(const signed char* q, const unsigned char* scale, void* y, long long rows, int C, int dtype,
                conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  if (rows < 0 || C <= 0 || C > kSeqMaxCount || rows > kSeqMaxElems / C) return CONV_EINVAL;
  if (rows == 0) return CONV_OK;
  if (!q || !scale || !y) return CONV_EINVAL;
  const int es = elem_size(dtype);
  if (!aligned_to(y, es)) return CONV_EALIGN;
  const Span ins[2] = {span_of(q, rows * C), span_of(scale, rows * ((C + ACT8_BLOCK - 1LL) / ACT8_BLOCK))};
  const Span out = span_of(y, rows * C * es);
  if (any_alias(&out, 1, ins, 2)) return CONV_EALIAS;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CONV_F32) return unpack_rows<float>(q, scale, y, rows, C, st);
  if (dtype == CONV_F16) return unpack_rows<__half>(q, scale, y, rows, C, st);
  return unpack_rows<__nv_bfloat16>(q, scale, y, rows, C, st);
}

}  // extern "C"

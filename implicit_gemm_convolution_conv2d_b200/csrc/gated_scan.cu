// gated_scan.cu -- C ABI of the gated linear recurrence (see gated_scan.cuh):
// argument checks and launches.  Allocates nothing.
#include "gated_scan.cuh"

using namespace convfwd;

namespace {

long long state_rows(int N, long long L, bool packed) {
  return (packed ? 1 : N) * ((L + GATED_SCAN_STATE_EVERY - 1) / GATED_SCAN_STATE_EVERY);
}

// Sets `in` and the bytes it spans (values, then scales) in s[0], s[1].
int take_input(SeqIn& in, Span* s, const void* p, const unsigned char* scale, long long batch, long long token, int N,
               long long L, int C, bool packed, int esize) {
  long long elems;
  if (!strided_extent(N, L, C, packed, batch, token, elems)) return CONV_EINVAL;
  if (elems > 0 && !p) return CONV_EINVAL;
  if (!scale && !aligned_to(p, esize)) return CONV_EALIGN;
  in = SeqIn{p, scale, batch, token};
  s[0] = span_of(p, scale ? elems : elems * esize);
  s[1] = scale ? span_of(scale, (packed ? 1LL : N) * L * ((C + ACT8_BLOCK - 1LL) / ACT8_BLOCK)) : Span{0, 0};
  return CONV_OK;
}

// CTAs of a cluster, `tokens` each: the least power of two by which the grid has
// four CTAs for each SM of a 148-SM B200 (a fixed number: the order of ddecay's sum
// must not depend on the device), but no more than the tokens fill, nor eight.  Two
// fit an SM (one of the f32 gradient's), so such a grid takes two rounds, the last
// of them in part, and few channels of few sequences leave SMs without a CTA.
int cluster_of(int N, long long L, int C, bool packed, int tokens) {
  const long long chains = (packed ? 1LL : N) * ((C + 63) / 64);
  const long long turns = (L + tokens - 1) / tokens;
  int s = 1;
  while (s < kScanMaxCluster && s < turns && chains * s < 4 * 148) s *= 2;
  return s;
}

// Clusters along x; the batch along y, and along z where it passes y's limit.
dim3 scan_grid(const ScanArgs& a, int ctas, bool packed) {
  const unsigned n = packed ? 1 : a.N, y = std::min(n, 65535u);
  return dim3((a.C + 63) / 64 * ctas, y, (n + y - 1) / y);
}

bool rows_take16(const SeqIn& in, bool packed, int esize) {
  return rows_aligned(in.p, packed ? 0 : in.batch, in.token, in.scale ? 1 : esize, 16);
}

template <typename T, bool PACKED, bool ALIGNED>
cudaError_t forward_as(const ScanArgs& a, cudaStream_t st) {
  const int s = cluster_of(a.N, a.L, a.C, PACKED, kScanWarps * kForwardSteps);
  const dim3 grid = scan_grid(a, s, PACKED);
  auto* k = gated_scan_kernel<T, PACKED, ALIGNED>;
  const size_t smem = sizeof(ForwardShared<T>);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_pdl(k, grid, dim3(kScanThreads), smem, st, s, a);
}

template <typename T>
cudaError_t launch_forward(const ScanArgs& a, cudaStream_t st) {
  const bool p = a.packed, aligned = a.C % (16 / static_cast<int>(sizeof(T))) == 0 && rows_take16(a.x, p, sizeof(T)) &&
                                     rows_take16(a.r, p, sizeof(T)) && rows_take16(a.i, p, sizeof(T)) &&
                                     aligned_to(a.y, 2 * sizeof(T));
  if (aligned) return p ? forward_as<T, true, true>(a, st) : forward_as<T, false, true>(a, st);
  return p ? forward_as<T, true, false>(a, st) : forward_as<T, false, false>(a, st);
}

// `parts`: the partial sums of ddecay.
template <typename T, bool PACKED, bool ALIGNED, bool Q8>
cudaError_t grad_as(const ScanArgs& a, int& parts, cudaStream_t st) {
  const int s = cluster_of(a.N, a.L, a.C, PACKED, GATED_SCAN_STATE_EVERY);
  const dim3 grid = scan_grid(a, s, PACKED);
  parts = s * (PACKED ? 1 : a.N);
  auto* k = gated_scan_grad_kernel<T, PACKED, ALIGNED, Q8>;
  const size_t smem = sizeof(GradShared<T>);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_pdl(k, grid, dim3(kScanThreads), smem, st, s, a);
}

template <typename T, bool PACKED>
cudaError_t grad_by(const ScanArgs& a, int& parts, cudaStream_t st) {
  bool aligned = a.C % (16 / static_cast<int>(sizeof(T))) == 0;
  for (const SeqIn* in : {&a.x, &a.r, &a.i, &a.dy})
    aligned = aligned && (!in->scale || a.C % 16 == 0) && rows_take16(*in, PACKED, sizeof(T));
  for (const void* out : {a.dx, a.dr, a.di}) aligned = aligned && aligned_to(out, 2 * sizeof(T));
  if (a.x.scale)
    return aligned ? grad_as<T, PACKED, true, true>(a, parts, st) : grad_as<T, PACKED, false, true>(a, parts, st);
  return aligned ? grad_as<T, PACKED, true, false>(a, parts, st) : grad_as<T, PACKED, false, false>(a, parts, st);
}

template <typename T>
cudaError_t launch_grad(const ScanArgs& a, int& parts, cudaStream_t st) {
  return a.packed ? grad_by<T, true>(a, parts, st) : grad_by<T, false>(a, parts, st);
}

// A CONV_ code.
template <typename T>
int launch_step(const ScanStepArgs& a, cudaStream_t st) {
  constexpr int kV = 4;  // channels a thread: 8 bytes of a 16-bit type, 16 of fp32
  const int es = static_cast<int>(sizeof(T));
  const size_t v = static_cast<size_t>(es) * kV;
  const bool vec = a.C % kV == 0 && rows_aligned(a.x, 0, a.xs, es, v) && rows_aligned(a.r, 0, a.rs, es, v) &&
                   rows_aligned(a.i, 0, a.is, es, v) && aligned_to(a.y, v);
  const int per = kStepThreads * (vec ? kV : 1);
  const dim3 grid(a.B, (a.C + per - 1) / per);
  if (grid.y > 65535) return CONV_EUNSUPPORTED;
  const cudaError_t e = launch_pdl(vec ? gated_scan_step_kernel<T, kV> : gated_scan_step_kernel<T, 1>, grid,
                                   dim3(kStepThreads), 0, st, 1, a);
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

}  // namespace

extern "C" {

int gated_scan(const void* x, const void* r, const void* i, const float* decay, const float* h0, const int* cu, void* y,
               float* h_last, float* states, int N, long long L, int C, long long x_batch, long long x_token,
               long long r_batch, long long r_token, long long i_batch, long long i_token, int fill, int dtype,
               conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  const bool packed = cu != nullptr;
  if (!seq_sizes_ok(N, L, C, packed)) return CONV_EINVAL;
  const int es = elem_size(dtype);
  ScanArgs a = {};
  Span ins[9], outs[3];
  int rc = take_input(a.x, ins, x, nullptr, x_batch, x_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_input(a.r, ins + 2, r, nullptr, r_batch, r_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_input(a.i, ins + 4, i, nullptr, i_batch, i_token, N, L, C, packed, es);
  if (rc != CONV_OK) return rc;
  const long long rows = packed ? L : N * L, nc = static_cast<long long>(N) * C;
  if (!decay || (rows > 0 && !y)) return CONV_EINVAL;
  if (!aligned_to(y, es) || !aligned_to(decay, 4) || !aligned_to(h0, 4) || !aligned_to(cu, 4) ||
      !aligned_to(h_last, 4) || !aligned_to(states, 4))
    return CONV_EALIGN;
  ins[6] = span_of(decay, 4LL * C);
  ins[7] = span_of(h0, 4 * nc);
  ins[8] = span_of(cu, 4LL * (N + 1));
  outs[0] = span_of(y, rows * C * es);
  outs[1] = span_of(h_last, 4 * nc);
  outs[2] = span_of(states, 4 * state_rows(N, L, packed) * C);
  if (any_alias(outs, 3, ins, 9)) return CONV_EALIAS;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {
    if (fill && rows > 0 && cudaMemsetAsync(y, 0, static_cast<size_t>(rows) * C * es, st) != cudaSuccess)
      return CONV_ELAUNCH;
    return CONV_OK;
  }
  a.decay = decay;
  a.consts = gate_consts();
  a.h0 = h0;
  a.cu = cu;
  a.y = y;
  a.h_last = h_last;
  a.states = states;
  a.N = N;
  a.L = L;
  a.C = C;
  a.packed = packed;
  a.fill = fill != 0;
  const cudaError_t e = dtype == CONV_F32   ? launch_forward<float>(a, st)
                        : dtype == CONV_F16 ? launch_forward<__half>(a, st)
                                            : launch_forward<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

int gated_scan_grad_workspace_size(int N, long long L, int C, int packed, unsigned long long* bytes) {
  if (!seq_sizes_ok(N, L, C, packed != 0) || !bytes) return CONV_EINVAL;
  // a row for each CTA that has a channel
  *bytes = 4ull * (packed ? 1 : N) * cluster_of(N, L, C, packed != 0, GATED_SCAN_STATE_EVERY) * C;
  return CONV_OK;
}

int gated_scan_grad(const void* x, const unsigned char* x_scale, const void* r, const unsigned char* r_scale,
                    const void* i, const unsigned char* i_scale, const float* decay, const float* states,
                    const float* h0, const int* cu, const void* dy, const float* dh_last, void* dx, void* dr, void* di,
                    float* ddecay, float* dh0, int N, long long L, int C, long long x_batch, long long x_token,
                    long long r_batch, long long r_token, long long i_batch, long long i_token, long long dy_batch,
                    long long dy_token, int fill, int dtype, void* workspace, unsigned long long workspace_bytes,
                    conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  const bool packed = cu != nullptr;
  if (!seq_sizes_ok(N, L, C, packed)) return CONV_EINVAL;
  const int es = elem_size(dtype);
  ScanArgs a = {};
  Span ins[13], outs[6];
  int rc = take_input(a.x, ins, x, x_scale, x_batch, x_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_input(a.r, ins + 2, r, r_scale, r_batch, r_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_input(a.i, ins + 4, i, i_scale, i_batch, i_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_input(a.dy, ins + 6, dy, nullptr, dy_batch, dy_token, N, L, C, packed, es);
  if (rc != CONV_OK) return rc;
  if ((x_scale == nullptr) != (r_scale == nullptr) || (x_scale == nullptr) != (i_scale == nullptr))
    return CONV_EUNSUPPORTED;
  if (x_scale)  // checkpoints are contiguous
    for (const SeqIn* in : {&a.x, &a.r, &a.i})
      if ((L > 1 && in->token != C) || (!packed && N > 1 && in->batch != L * C)) return CONV_EUNSUPPORTED;
  const long long rows = packed ? L : N * L, nc = static_cast<long long>(N) * C;
  if (!decay || !ddecay || (rows > 0 && (!dx || !dr || !di || !states))) return CONV_EINVAL;
  unsigned long long need = 0;
  gated_scan_grad_workspace_size(N, L, C, packed, &need);
  if (need > 0 && (!workspace || workspace_bytes < need)) return CONV_EINVAL;
  if (!aligned_to(dx, es) || !aligned_to(dr, es) || !aligned_to(di, es) || !aligned_to(decay, 4) ||
      !aligned_to(states, 4) || !aligned_to(h0, 4) || !aligned_to(cu, 4) || !aligned_to(dh_last, 4) ||
      !aligned_to(ddecay, 4) || !aligned_to(dh0, 4) || !aligned_to(workspace, 16))
    return CONV_EALIGN;
  ins[8] = span_of(decay, 4LL * C);
  ins[9] = span_of(states, 4 * state_rows(N, L, packed) * C);
  ins[10] = span_of(h0, 4 * nc);
  ins[11] = span_of(cu, 4LL * (N + 1));
  ins[12] = span_of(dh_last, 4 * nc);
  outs[0] = span_of(dx, rows * C * es);
  outs[1] = span_of(dr, rows * C * es);
  outs[2] = span_of(di, rows * C * es);
  outs[3] = span_of(ddecay, 4LL * C);
  outs[4] = span_of(dh0, 4 * nc);
  outs[5] = span_of(workspace, static_cast<long long>(need));
  if (any_alias(outs, 6, ins, 13)) return CONV_EALIAS;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  a.decay = decay;
  a.consts = gate_consts();
  a.states_in = states;
  a.h0 = h0;
  a.cu = cu;
  a.dh_last = dh_last;
  a.dx = dx;
  a.dr = dr;
  a.di = di;
  a.dh0 = dh0;
  a.part = static_cast<float*>(workspace);
  a.N = N;
  a.L = L;
  a.C = C;
  a.packed = packed;
  a.fill = fill != 0;
  int parts = 0;
  if (N == 0) {
    const size_t bytes = static_cast<size_t>(rows) * C * es;
    if (fill && rows > 0)
      for (void* p : {dx, dr, di})
        if (cudaMemsetAsync(p, 0, bytes, st) != cudaSuccess) return CONV_ELAUNCH;
  } else {
    const cudaError_t e = dtype == CONV_F32   ? launch_grad<float>(a, parts, st)
                          : dtype == CONV_F16 ? launch_grad<__half>(a, parts, st)
                                              : launch_grad<__nv_bfloat16>(a, parts, st);
    if (e != cudaSuccess) return CONV_ELAUNCH;
  }
  const cudaError_t e = launch_pdl(gated_scan_sum_kernel, dim3((C + 31) / 32), dim3(32, 8), 0, st, 1,
                                   static_cast<const float*>(a.part), ddecay, parts, C);
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

int gated_scan_step(const void* x, const void* r, const void* i, const float* decay, float* h, const int* index, void* y,
                    int B, int slots, int C, long long x_token, long long r_token, long long i_token, int fill,
                    int dtype, conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  if (B < 0 || slots < 0 || !seq_sizes_ok(1, B, C, true) || slots > kSeqMaxElems / C) return CONV_EINVAL;
  if (!index && B > slots) return CONV_EINVAL;
  const int es = elem_size(dtype);
  SeqIn in;
  Span ins[8], outs[2];
  int rc = take_input(in, ins, x, nullptr, 0, x_token, 1, B, C, true, es);
  if (rc == CONV_OK) rc = take_input(in, ins + 2, r, nullptr, 0, r_token, 1, B, C, true, es);
  if (rc == CONV_OK) rc = take_input(in, ins + 4, i, nullptr, 0, i_token, 1, B, C, true, es);
  if (rc != CONV_OK) return rc;
  if (B == 0) return CONV_OK;
  if (!decay || !y || (slots > 0 && !h)) return CONV_EINVAL;
  if (!aligned_to(y, es) || !aligned_to(decay, 4) || !aligned_to(h, 4) || !aligned_to(index, 4)) return CONV_EALIGN;
  ins[6] = span_of(decay, 4LL * C);
  ins[7] = span_of(index, 4LL * B);
  outs[0] = span_of(y, static_cast<long long>(B) * C * es);
  outs[1] = span_of(h, 4LL * slots * C);
  if (any_alias(outs, 2, ins, 8)) return CONV_EALIAS;
  const ScanStepArgs a = {x, r, i, decay, h, index, y, B, slots, C, fill != 0, x_token, r_token, i_token, gate_consts()};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == CONV_F32) return launch_step<float>(a, st);
  if (dtype == CONV_F16) return launch_step<__half>(a, st);
  return launch_step<__nv_bfloat16>(a, st);
}

}  // extern "C"

// conv_causal.cu -- C ABI of the causal depthwise convolution (see
// conv_causal.cuh): argument checks and launches.  Allocates nothing.
#include "conv_causal.cuh"

using namespace convfwd;

namespace {

// Calls f with (T, KT) as types; KT is the least window of 2, 3, 4 and 8 taps
// that holds K.
template <typename T>
struct Type {
  using type = T;
};
template <int N>
struct Int {
  static constexpr int value = N;
};

template <typename F>
cudaError_t by_type_and_taps(int dtype, int K, F&& f) {
  const auto taps = [&](auto t) {
    if (K <= 2) return f(t, Int<2>{});
    if (K == 3) return f(t, Int<3>{});
    if (K == 4) return f(t, Int<4>{});
    return f(t, Int<8>{});
  };
  if (dtype == CONV_F32) return taps(Type<float>{});
  if (dtype == CONV_F16) return taps(Type<__half>{});
  return taps(Type<__nv_bfloat16>{});
}

bool shape_ok(int N, long long L, int C, int K, bool packed) {
  return K >= 1 && K <= CONV_CAUSAL_MAX_K && seq_sizes_ok(N, L, C, packed) &&
         static_cast<long long>(N) * (K - 1) <= kSeqMaxElems / C;
}

long long run_blocks(int N, long long L, int run, bool packed);

// Tokens a warp: as many as make the blocks fill a 148-SM B200's `per_sm` places
// an SM a whole number of times (a fixed number of SMs: the order of dw's sum must
// not depend on the device), between 16 and 512 and a multiple of 16; K - 1 rows a
// run are read again.  Against a length that left a part of a round: 8 x 4096 x
// 2560 bf16 forward 73 -> 67 us, its gradients 151 -> 138;
// 4 x 2048 x 2048 19.4 -> 17.8 and 46 -> 36.
int run_length(int N, long long L, int C, bool packed, int per_sm) {
  const long long rows = packed ? L : N * L, tiles = (C + 63) / 64, round = 148LL * per_sm;
  const long long warps = round * kCausalWarps, rounds = std::max<long long>(1, (rows * tiles + 512 * warps - 1) / (512 * warps));
  int run = static_cast<int>(std::min<long long>(512, (rows * tiles / (warps * rounds) / 16 + 1) * 16));
  while (run < 512 && run_blocks(N, L, run, packed) * tiles > round * rounds) run += 16;
  return run;
}

// Blocks an SM of the K = 4 kernels, by their registers (76 to 80; gradients up to
// 128).  Others are given the same count: with up to 3 taps (64 registers) four
// forward blocks fit, with 5 to 8 (90 to 114) two, so that their grids leave a part
// of a round.
constexpr int kForwardPlaces = 3, kGradPlaces = 2;

int grad_run(int N, long long L, int C, bool packed) { return run_length(N, L, C, packed, kGradPlaces); }

// Blocks along the runs, each with a partial sum of its own.
long long run_blocks(int N, long long L, int run, bool packed) {
  const long long runs = (L + run - 1) / run * (packed ? 1 : N);
  return std::max<long long>(1, (runs + kCausalWarps - 1) / kCausalWarps);
}

// Channels along x; the blocks along y, and along z where they pass y's limit.
dim3 run_grid(int C, long long blocks) {
  const long long y = std::min<long long>(blocks, 65535);
  return dim3((C + 63) / 64, static_cast<unsigned>(y), static_cast<unsigned>((blocks + y - 1) / y));
}

bool aligned_rows(const SeqIn& in, bool packed, int C, int esize) {
  const int e = in.scale ? 1 : esize;
  return C % (16 / e) == 0 && rows_aligned(in.p, packed ? 0 : in.batch, in.token, e, 16);
}

template <typename K>
cudaError_t launch_rows(K* k, dim3 grid, size_t smem, const CausalArgs& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e != cudaSuccess ? e : launch_pdl(k, grid, dim3(kCausalThreads), smem, st, 1, a);
}

// Checks shared by the forward and the backward pass.
int take_x(Span* s, const void* p, const unsigned char* scale, long long batch, long long token, int N, long long L,
           int C, bool packed, int esize) {
  long long elems;
  if (!strided_extent(N, L, C, packed, batch, token, elems)) return CONV_EINVAL;
  if (elems > 0 && !p) return CONV_EINVAL;
  if (!scale && !aligned_to(p, esize)) return CONV_EALIGN;
  s[0] = span_of(p, scale ? elems : elems * esize);
  s[1] = scale ? span_of(scale, (packed ? 1LL : N) * L * ((C + ACT8_BLOCK - 1LL) / ACT8_BLOCK)) : Span{0, 0};
  return CONV_OK;
}

}  // namespace

extern "C" {

int conv_causal(const void* x, const void* w, const void* bias, const void* state, const int* cu, void* y,
                void* state_out, int N, long long L, int C, int K, long long x_batch, long long x_token,
                int activation, int fill, int dtype, conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  const bool packed = cu != nullptr;
  if (!shape_ok(N, L, C, K, packed) || (activation != CONV_ACT_NONE && activation != CONV_ACT_SILU))
    return CONV_EINVAL;
  const int es = elem_size(dtype);
  Span ins[6], outs[2];
  const int rc = take_x(ins, x, nullptr, x_batch, x_token, N, L, C, packed, es);
  if (rc != CONV_OK) return rc;
  const long long rows = packed ? L : N * L, window = static_cast<long long>(N) * (K - 1) * C;
  if (!w || (rows > 0 && !y)) return CONV_EINVAL;
  for (const void* p : {w, bias, state, static_cast<const void*>(y), static_cast<const void*>(state_out)})
    if (!aligned_to(p, es)) return CONV_EALIGN;
  if (!aligned_to(cu, 4)) return CONV_EALIGN;
  ins[2] = span_of(w, static_cast<long long>(C) * K * es);
  ins[3] = span_of(bias, static_cast<long long>(C) * es);
  ins[4] = span_of(state, window * es);
  ins[5] = span_of(cu, 4LL * (N + 1));
  outs[0] = span_of(y, rows * C * es);
  outs[1] = span_of(state_out, window * es);
  if (any_alias(outs, 2, ins, 6)) return CONV_EALIAS;
  if (rows == 0 && window == 0) return CONV_OK;
  CausalArgs a = {};
  a.x = SeqIn{x, nullptr, x_batch, x_token};
  a.w = w, a.bias = bias, a.state = state, a.cu = cu, a.y = y, a.state_out = window > 0 ? state_out : nullptr;
  a.N = N, a.C = C, a.K = K, a.silu = activation == CONV_ACT_SILU, a.fill = fill != 0;
  a.L = static_cast<int>(L);
  a.run = run_length(N, L, C, packed, kForwardPlaces);
  a.runs = static_cast<int>((L + a.run - 1) / a.run);
  const long long by = run_blocks(N, L, a.run, packed);
  if (by > 0x7fffffffLL) return CONV_EUNSUPPORTED;
  a.blocks = static_cast<int>(by);
  const dim3 grid = run_grid(C, by);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = by_type_and_taps(dtype, K, [&](auto t, auto kt) {
    using T = typename decltype(t)::type;
    constexpr int KT = decltype(kt)::value;
    const bool aligned = aligned_rows(a.x, packed, C, es) && aligned_to(y, 2 * es) && aligned_to(state_out, 2 * es);
    return launch_rows(aligned ? conv_causal_kernel<T, KT, true> : conv_causal_kernel<T, KT, false>, grid,
                       sizeof(CausalShared<T>), a, st);
  });
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

int conv_causal_grad_workspace_size(int N, long long L, int C, int K, int packed, unsigned long long* bytes) {
  if (!shape_ok(N, L, C, K, packed != 0) || !bytes) return CONV_EINVAL;
  *bytes = 4ull * run_blocks(N, L, grad_run(N, L, C, packed != 0), packed != 0) * (K + 1) * C;
  return CONV_OK;
}

int conv_causal_grad(const void* x, const unsigned char* x_scale, const void* w, const void* bias, const void* state,
                     const int* cu, const void* dy, const void* dstate_out, void* dx, void* dw, void* dbias,
                     void* dstate, int N, long long L, int C, int K, long long x_batch, long long x_token,
                     long long dy_batch, long long dy_token, int activation, int fill, int dtype, void* workspace,
                     unsigned long long workspace_bytes, conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  const bool packed = cu != nullptr;
  if (!shape_ok(N, L, C, K, packed) || (activation != CONV_ACT_NONE && activation != CONV_ACT_SILU))
    return CONV_EINVAL;
  const int es = elem_size(dtype);
  Span ins[9], outs[5];
  int rc = take_x(ins, x, x_scale, x_batch, x_token, N, L, C, packed, es);
  if (rc == CONV_OK) rc = take_x(ins + 2, dy, nullptr, dy_batch, dy_token, N, L, C, packed, es);
  if (rc != CONV_OK) return rc;
  const long long rows = packed ? L : N * L, window = static_cast<long long>(N) * (K - 1) * C;
  if (!w || !dw || (bias && !dbias) || (rows > 0 && !dx) || (dstate && !state)) return CONV_EINVAL;
  unsigned long long need = 0;
  conv_causal_grad_workspace_size(N, L, C, K, packed, &need);
  if (!workspace || workspace_bytes < need) return CONV_EINVAL;
  for (const void* p : {w, bias, state, dstate_out, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(dbias), static_cast<const void*>(dstate)})
    if (!aligned_to(p, es)) return CONV_EALIGN;
  if (!aligned_to(cu, 4) || !aligned_to(workspace, 16)) return CONV_EALIGN;
  ins[4] = span_of(w, static_cast<long long>(C) * K * es);
  ins[5] = span_of(bias, static_cast<long long>(C) * es);
  ins[6] = span_of(state, window * es);
  ins[7] = span_of(cu, 4LL * (N + 1));
  ins[8] = span_of(dstate_out, window * es);
  outs[0] = span_of(dx, rows * C * es);
  outs[1] = span_of(dw, static_cast<long long>(C) * K * es);
  outs[2] = span_of(dbias, static_cast<long long>(C) * es);
  outs[3] = span_of(dstate, window * es);
  outs[4] = span_of(workspace, static_cast<long long>(need));
  if (any_alias(outs, 5, ins, 9)) return CONV_EALIAS;
  CausalArgs a = {};
  a.x = SeqIn{x, x_scale, x_batch, x_token}, a.dy = SeqIn{dy, nullptr, dy_batch, dy_token};
  a.w = w, a.bias = bias, a.state = state, a.cu = cu;
  a.dstate_out = window > 0 ? dstate_out : nullptr;
  a.dx = dx, a.dstate = dstate, a.part = static_cast<float*>(workspace);
  a.N = N, a.C = C, a.K = K, a.silu = activation == CONV_ACT_SILU, a.fill = fill != 0;
  a.L = static_cast<int>(L);
  a.run = grad_run(N, L, C, packed);
  a.runs = static_cast<int>((L + a.run - 1) / a.run);
  const long long by = run_blocks(N, L, a.run, packed);
  if (by > 0x7fffffffLL) return CONV_EUNSUPPORTED;
  a.blocks = static_cast<int>(by);
  const dim3 grid = run_grid(C, by);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = by_type_and_taps(dtype, K, [&](auto t, auto kt) {
    using T = typename decltype(t)::type;
    constexpr int KT = decltype(kt)::value;
    const bool aligned = aligned_rows(a.x, packed, C, es) && aligned_rows(a.dy, packed, C, es) && aligned_to(dx, 2 * es);
    auto* k = x_scale ? (aligned ? conv_causal_grad_kernel<T, KT, true, true> : conv_causal_grad_kernel<T, KT, false, true>)
                      : (aligned ? conv_causal_grad_kernel<T, KT, true, false> : conv_causal_grad_kernel<T, KT, false, false>);
    cudaError_t err = launch_rows(k, grid, sizeof(CausalGradShared<T>), a, st);
    if (err != cudaSuccess) return err;
    err = launch_pdl(conv_causal_sum_kernel<T>, dim3((C + 31) / 32, K + 1), dim3(32, 8), 0, st, 1,
                     static_cast<const float*>(a.part), static_cast<T*>(dw), static_cast<T*>(dbias), static_cast<int>(by), C,
                     K);
    if (err != cudaSuccess || !dstate || window == 0) return err;
    return launch_pdl(x_scale ? conv_causal_dstate_kernel<T, true> : conv_causal_dstate_kernel<T, false>,
                      dim3((C + 127) / 128, std::min(N, 65535)), dim3(128), 0, st, 1, a);
  });
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

int conv_causal_step(const void* x, const void* w, const void* bias, void* state, const int* index, void* y, int B,
                     int slots, int C, int K, long long x_token, int activation, int fill, int dtype,
                     conv_stream_t stream) {
  if (!dtype_ok(dtype)) return CONV_EDTYPE;
  if (B < 0 || slots < 0 || !shape_ok(slots, 0, C, K, false) || !seq_sizes_ok(1, B, C, true) ||
      (activation != CONV_ACT_NONE && activation != CONV_ACT_SILU) || (!index && B > slots))
    return CONV_EINVAL;
  const int es = elem_size(dtype);
  Span ins[5], outs[2];
  const int rc = take_x(ins, x, nullptr, 0, x_token, 1, B, C, true, es);
  if (rc != CONV_OK) return rc;
  if (B == 0) return CONV_OK;
  const long long window = static_cast<long long>(slots) * (K - 1) * C;
  if (!w || !y || (window > 0 && !state)) return CONV_EINVAL;
  for (const void* p : {w, bias, static_cast<const void*>(state), static_cast<const void*>(y)})
    if (!aligned_to(p, es)) return CONV_EALIGN;
  if (!aligned_to(index, 4)) return CONV_EALIGN;
  ins[2] = span_of(w, static_cast<long long>(C) * K * es);
  ins[3] = span_of(bias, static_cast<long long>(C) * es);
  ins[4] = span_of(index, 4LL * B);
  outs[0] = span_of(y, static_cast<long long>(B) * C * es);
  outs[1] = span_of(state, window * es);
  if (any_alias(outs, 2, ins, 5)) return CONV_EALIAS;
  const CausalStepArgs a = {x, w, bias, state, index, y, B, slots, C, K, activation == CONV_ACT_SILU, fill != 0, x_token};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  bool fits = true;
  const cudaError_t e = by_type_and_taps(dtype, K, [&](auto t, auto kt) {
    using T = typename decltype(t)::type;
    constexpr int KT = decltype(kt)::value, V = 4;
    const size_t bytes = V * sizeof(T);
    const bool vec = C % V == 0 && rows_aligned(x, 0, x_token, es, bytes) && aligned_to(y, bytes) &&
                     aligned_to(state, bytes);
    const int per = kCausalStepThreads * (vec ? V : 1);
    const dim3 grid(B, (C + per - 1) / per);
    fits = grid.y <= 65535;
    if (!fits) return cudaSuccess;
    return launch_pdl(vec ? conv_causal_step_kernel<T, KT, V> : conv_causal_step_kernel<T, KT, 1>, grid,
                      dim3(kCausalStepThreads), 0, st, 1, a);
  });
  if (!fits) return CONV_EUNSUPPORTED;
  return e == cudaSuccess ? CONV_OK : CONV_ELAUNCH;
}

}  // extern "C"

// kda_layer_api.cu -- C ABI of the operators around the recurrence (declared in
// include/kda.h): root-mean-square norm, short convolution, selective scan.
// Argument validation, workspace sizes, dispatch to the kernels.
#include <initializer_list>

#include "kda_conv.cuh"
#include "kda_norm.cuh"
#include "kda_scan.cuh"
#include "kda_scan_bwd.cuh"
#include "kda_status.h"

namespace kda {
cudaError_t take_layer_device_error(int* code) {
  *code = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_device_error, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
}
}  // namespace kda

namespace {

using kda::clear_status;
#define fail kda::set_status

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }
bool all_aligned(std::initializer_list<const void*> ps, unsigned a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return false;
  return true;
}
bool known(kda_dtype_t t) { return t == KDA_BF16 || t == KDA_F32; }
unsigned bytes_of(kda_dtype_t t) { return t == KDA_F32 ? 4u : 2u; }

kda_status_t finish(const char* fn, cudaError_t e) {
  return e == cudaSuccess ? KDA_OK : fail(KDA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

// Sizes shared by the sequence operators; *q describes the tokens.
kda_status_t check_seqs(const char* fn, const int32_t* cu, int num_seqs, int B, int T, kda::Seqs* q) {
  if (B < 0 || T < 0 || num_seqs < 0)
    return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes B=%d T=%d num_seqs=%d", fn, B, T, num_seqs);
  if (cu) {
    if (B != 1) return fail(KDA_ERR_INVALID_ARG, "%s: packed inputs need B == 1", fn);
    if (num_seqs < 1) return fail(KDA_ERR_INVALID_ARG, "%s: cu_seqlens needs num_seqs >= 1", fn);
    if (!aligned(cu, 4)) return fail(KDA_ERR_ALIGNMENT, "%s: cu_seqlens not 4-byte aligned", fn);
  } else if (num_seqs != 0) {
    return fail(KDA_ERR_INVALID_ARG, "%s: num_seqs=%d without cu_seqlens", fn, num_seqs);
  }
  *q = kda::Seqs{cu, cu ? num_seqs : B, T, (long long)B * T};
  return KDA_OK;
}
kda_status_t check_types(const char* fn, kda_dtype_t dtype, kda_dtype_t weight_dtype) {
  if (!known(dtype)) return fail(KDA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
  if (!known(weight_dtype)) return fail(KDA_ERR_UNSUPPORTED, "%s: unknown weight_dtype %d", fn, (int)weight_dtype);
  return KDA_OK;
}
kda_status_t misaligned(const char* fn, const char* what) {
  return fail(KDA_ERR_ALIGNMENT, "%s: %s", fn, what);
}
kda_status_t check_workspace(const char* fn, const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return fail(KDA_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws ? have : (size_t)0, need);
  if (need && !aligned(ws, 16)) return misaligned(fn, "workspace is not 16-byte aligned");
  return KDA_OK;
}
bool overlaps(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (const void* o : outs) {
    if (!o) continue;
    for (const void* i : ins)
      if (i == o) return true;
  }
  return false;
}
bool repeated(std::initializer_list<const void*> outs) {
  const void* const* p = outs.begin();
  for (size_t i = 0; i < outs.size(); ++i)
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (p[i] && p[i] == p[j]) return true;
  return false;
}

// -------------------------------------------------------------------- norm
kda_status_t norm_fwd_impl(const char* fn, int quant, const void* x, long long x_stride, const void* residual,
                           const void* weight, kda_dtype_t weight_dtype, void* y, float* scale, void* s,
                           long long rows, int D, int group, float eps, kda_dtype_t dtype, cudaStream_t stream) {
  clear_status();
  if (kda_status_t st = check_types(fn, dtype, weight_dtype)) return st;
  if (rows < 0 || D < 1 || x_stride < D)
    return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes rows=%lld D=%d x_stride=%lld", fn, rows, D, x_stride);
  if (D > kda::norm::kMaxDim || rows > 0x7fffffffLL)
    return fail(KDA_ERR_UNSUPPORTED, "%s: rows=%lld D=%d (need D <= %d, rows < 2^31)", fn, rows, D,
                kda::norm::kMaxDim);
  if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
  if (quant != kda::norm::kNone && group != 0) {
    if ((group != 32 && group != 64 && group != 128) || D % group)
      return fail(KDA_ERR_UNSUPPORTED, "%s: group=%d (need 0, or 32, 64, 128 dividing D=%d)", fn, group, D);
    quant = kda::norm::kGroup;
  }
  if (rows == 0) return KDA_OK;
  if (!x || !weight || !y || (quant != kda::norm::kNone && !scale))
    return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned es = bytes_of(dtype);
  if (!all_aligned({x, residual, s, quant == kda::norm::kNone ? y : nullptr}, es) ||
      !aligned(weight, bytes_of(weight_dtype)) || !all_aligned({scale}, 4))
    return misaligned(fn, "a pointer is not element-aligned");
  if (s && (s == y || s == x || s == (void*)scale))
    return fail(KDA_ERR_INVALID_ARG, "%s: s aliases x or another output", fn);
  if (y == residual || (void*)scale == y || overlaps({y, s, scale}, {weight}) ||
      overlaps({scale}, {x, residual}) || (y == x && (x_stride != D || quant != kda::norm::kNone)))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input", fn);
  const int vec = (int)(16 / es);
  const bool wide = D % vec == 0 && x_stride % vec == 0 &&
                    all_aligned({x, residual, s, quant == kda::norm::kNone ? y : nullptr}, 16) &&
                    (quant == kda::norm::kNone || aligned(y, vec)) &&
                    aligned(weight, weight_dtype == KDA_F32 ? 16u : 2u * vec);
  if (quant == kda::norm::kGroup && !wide)
    return misaligned(fn, "group scales need 16-byte aligned rows and pointers");
  kda::norm::FwdArgs a{x, x_stride, residual, weight, weight_dtype == KDA_BF16, y, scale, s, rows, D, group, eps, 1, 1};
  cudaError_t e = cudaErrorInvalidValue;
#define KDA_NORM_CASE(TYPE, V)                                                                        \
  e = quant == kda::norm::kNone  ? kda::norm::launch_fwd<TYPE, V, kda::norm::kNone>(a, stream)         \
      : quant == kda::norm::kRow ? kda::norm::launch_fwd<TYPE, V, kda::norm::kRow>(a, stream)          \
                                 : kda::norm::launch_fwd_groups<TYPE, V>(a, stream)
  if (dtype == KDA_BF16 && wide) KDA_NORM_CASE(__nv_bfloat16, 8);
  else if (dtype == KDA_F32 && wide) KDA_NORM_CASE(float, 4);
#undef KDA_NORM_CASE
#define KDA_NORM_CASE(TYPE)                                                                           \
  e = quant == kda::norm::kNone ? kda::norm::launch_fwd<TYPE, 1, kda::norm::kNone>(a, stream)          \
                                : kda::norm::launch_fwd<TYPE, 1, kda::norm::kRow>(a, stream)
  else if (dtype == KDA_BF16) KDA_NORM_CASE(__nv_bfloat16);
  else KDA_NORM_CASE(float);
#undef KDA_NORM_CASE
  return finish(fn, e);
}

size_t norm_lines(long long rows, int D) {
  size_t most = 0;
  for (int vec : {8, 4, 1}) {
    if (D % vec || D / vec > kda::norm::kMaxDim / vec) continue;
    const size_t lines = (size_t)kda::norm::bwd_grid(rows, D / vec, vec);
    if (lines > most) most = lines;
  }
  return most;
}

}  // namespace

extern "C" {

kda_status_t kda_rms_norm_fwd(const void* x, long long x_stride, const void* residual, const void* weight,
                              kda_dtype_t weight_dtype, void* y, void* s, long long rows, int D, float eps,
                              kda_dtype_t dtype, cudaStream_t stream) {
  return norm_fwd_impl("kda_rms_norm_fwd", kda::norm::kNone, x, x_stride, residual, weight, weight_dtype, y, nullptr,
                       s, rows, D, 0, eps, dtype, stream);
}

kda_status_t kda_rms_norm_quant_fwd(const void* x, long long x_stride, const void* residual, const void* weight,
                                    kda_dtype_t weight_dtype, void* q, float* scale, void* s, long long rows, int D,
                                    int group, float eps, kda_dtype_t dtype, cudaStream_t stream) {
  return norm_fwd_impl("kda_rms_norm_quant_fwd", kda::norm::kRow, x, x_stride, residual, weight, weight_dtype, q,
                       scale, s, rows, D, group, eps, dtype, stream);
}

size_t kda_rms_norm_bwd_workspace_size(long long rows, int D) {
  if (rows < 0 || D < 1 || D > kda::norm::kMaxDim) return 0;
  return norm_lines(rows, D) * (size_t)D * sizeof(float);
}

kda_status_t kda_rms_norm_bwd(const void* dy, const void* s, const void* weight, kda_dtype_t weight_dtype,
                              const void* ds, void* dx, float* dweight, long long rows, int D, float eps,
                              kda_dtype_t dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "kda_rms_norm_bwd";
  clear_status();
  if (kda_status_t st = check_types(fn, dtype, weight_dtype)) return st;
  if (rows < 0 || D < 1) return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes rows=%lld D=%d", fn, rows, D);
  if (D > kda::norm::kMaxDim)
    return fail(KDA_ERR_UNSUPPORTED, "%s: D=%d (need D <= %d)", fn, D, kda::norm::kMaxDim);
  if (!(eps >= 0.f)) return fail(KDA_ERR_INVALID_ARG, "%s: eps must not be negative", fn);
  if (!dweight || (rows > 0 && (!dy || !s || !weight || !dx)))
    return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned es = bytes_of(dtype);
  if (!all_aligned({dy, s, ds, dx}, es) || !all_aligned({weight}, bytes_of(weight_dtype)) || !aligned(dweight, 4))
    return misaligned(fn, "a pointer is not element-aligned");
  if (overlaps({dweight}, {dy, s, weight, ds, workspace, dx}) || overlaps({dx}, {s, weight, workspace}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input", fn);
  if (kda_status_t st =
          check_workspace(fn, workspace, workspace_bytes, kda_rms_norm_bwd_workspace_size(rows, D)))
    return st;
  const int vec = (int)(16 / es);
  const bool wide = D % vec == 0 && all_aligned({dy, s, ds, dx}, 16) &&
                    aligned(weight, weight_dtype == KDA_F32 ? 16u : 2u * vec);
  const kda::norm::BwdArgs a{dy, s, weight, weight_dtype == KDA_BF16, ds, dx, static_cast<float*>(workspace),
                             rows, D, eps};
  cudaError_t e;
  if (rows == 0) e = kda::launch_sum_lines(nullptr, dweight, nullptr, D, 0, D, stream);
  else if (dtype == KDA_BF16)
    e = wide ? kda::norm::launch_bwd<__nv_bfloat16, 8>(a, dweight, stream)
             : kda::norm::launch_bwd<__nv_bfloat16, 1>(a, dweight, stream);
  else
    e = wide ? kda::norm::launch_bwd<float, 4>(a, dweight, stream) : kda::norm::launch_bwd<float, 1>(a, dweight, stream);
  return finish(fn, e);
}

}  // extern "C"

// -------------------------------------------------------------- convolution
namespace {

kda_status_t conv_check(const char* fn, const void* x, long long x_stride, const void* weight, const void* bias,
                        kda_dtype_t weight_dtype, long long tokens, int D, int W, kda_dtype_t dtype) {
  if (kda_status_t st = check_types(fn, dtype, weight_dtype)) return st;
  if (D < 1 || x_stride < D) return fail(KDA_ERR_INVALID_ARG, "%s: bad sizes D=%d x_stride=%lld", fn, D, x_stride);
  if (W < 2 || W > 4) return fail(KDA_ERR_UNSUPPORTED, "%s: W=%d (need 2, 3 or 4)", fn, W);
  if (D > (1 << 26)) return fail(KDA_ERR_UNSUPPORTED, "%s: D=%d is too large", fn, D);
  if (!weight || (tokens > 0 && !x)) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all_aligned({x}, bytes_of(dtype)) || !all_aligned({weight, bias}, bytes_of(weight_dtype)))
    return misaligned(fn, "a pointer is not element-aligned");
  return KDA_OK;
}

// Weights and bias of `vec` channels start on a vector of theirs.
bool conv_params_wide(const void* weight, const void* bias, kda_dtype_t weight_dtype, int vec) {
  return all_aligned({weight, bias}, weight_dtype == KDA_F32 ? 16u : 2u * vec);
}

#define KDA_CONV_W(CALL) (W == 2 ? CALL(2) : W == 3 ? CALL(3) : CALL(4))

cudaError_t conv_fwd_dispatch(const kda::conv::FwdArgs& a, bool step, kda_dtype_t dtype, bool wide, int W,
                              cudaStream_t st) {
  using namespace kda::conv;
#define KDA_CALL(TYPE, V, WW) (step ? launch_step<TYPE, V, WW>(a, st) : launch_fwd<TYPE, V, WW>(a, st))
#define KDA_B8(WW) KDA_CALL(__nv_bfloat16, 8, WW)
#define KDA_B1(WW) KDA_CALL(__nv_bfloat16, 1, WW)
#define KDA_F4(WW) KDA_CALL(float, 4, WW)
#define KDA_F1(WW) KDA_CALL(float, 1, WW)
  if (dtype == KDA_BF16) return wide ? KDA_CONV_W(KDA_B8) : KDA_CONV_W(KDA_B1);
  return wide ? KDA_CONV_W(KDA_F4) : KDA_CONV_W(KDA_F1);
#undef KDA_CALL
#undef KDA_B8
#undef KDA_B1
#undef KDA_F4
#undef KDA_F1
}

template <typename T, typename TDY>
cudaError_t conv_bwd_dispatch(const kda::conv::BwdArgs& a, bool wide, int W, float* dw, float* db, cudaStream_t st) {
  using namespace kda::conv;
#define KDA_V4(WW) launch_bwd<T, TDY, 4, WW>(a, dw, db, st)
#define KDA_V1(WW) launch_bwd<T, TDY, 1, WW>(a, dw, db, st)
  return wide ? KDA_CONV_W(KDA_V4) : KDA_CONV_W(KDA_V1);
#undef KDA_V4
#undef KDA_V1
}

}  // namespace

extern "C" {

kda_status_t kda_short_conv_fwd(const void* x, long long x_stride, const void* weight, const void* bias,
                                kda_dtype_t weight_dtype, const void* state, void* y, void* state_out,
                                const int32_t* cu_seqlens, int num_seqs, int B, int T, int D, int W,
                                kda_dtype_t dtype, cudaStream_t stream) {
  const char* fn = "kda_short_conv_fwd";
  clear_status();
  kda::Seqs q;
  if (kda_status_t st = check_seqs(fn, cu_seqlens, num_seqs, B, T, &q)) return st;
  if (kda_status_t st = conv_check(fn, x, x_stride, weight, bias, weight_dtype, q.total, D, W, dtype)) return st;
  if (q.num == 0) return KDA_OK;
  if (q.total > 0 && !y) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned es = bytes_of(dtype);
  if (!all_aligned({state, y, state_out}, es)) return misaligned(fn, "a pointer is not element-aligned");
  if (overlaps({y, state_out}, {x, weight, bias, state, cu_seqlens}) || repeated({y, state_out}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  const int vec = (int)(16 / es);
  const bool wide = D % vec == 0 && x_stride % vec == 0 && all_aligned({x, state, y, state_out}, 16) &&
                    conv_params_wide(weight, bias, weight_dtype, vec);
  const kda::conv::FwdArgs a{x, x_stride, weight, bias, weight_dtype == KDA_BF16, state, y, state_out, q, D, 0, 0};
  return finish(fn, conv_fwd_dispatch(a, false, dtype, wide, W, stream));
}

kda_status_t kda_short_conv_step(const void* x, long long x_stride, const void* weight, const void* bias,
                                 kda_dtype_t weight_dtype, const void* state, void* y, void* state_out, int N, int D,
                                 int W, kda_dtype_t dtype, cudaStream_t stream) {
  const char* fn = "kda_short_conv_step";
  clear_status();
  if (N < 0) return fail(KDA_ERR_INVALID_ARG, "%s: bad size N=%d", fn, N);
  if (kda_status_t st = conv_check(fn, x, x_stride, weight, bias, weight_dtype, N, D, W, dtype)) return st;
  if (N == 0) return KDA_OK;
  if (!state || !y || !state_out) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned es = bytes_of(dtype);
  if (!all_aligned({state, y, state_out}, es)) return misaligned(fn, "a pointer is not element-aligned");
  if (overlaps({y}, {x, weight, bias, state}) || overlaps({state_out}, {x, weight, bias}) || repeated({y, state_out}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  const int vec = (int)(16 / es);
  const bool wide = D % vec == 0 && x_stride % vec == 0 && all_aligned({x, state, y, state_out}, 16) &&
                    conv_params_wide(weight, bias, weight_dtype, vec);
  const kda::conv::FwdArgs a{x,     x_stride,  weight, bias, weight_dtype == KDA_BF16,
                             state, y,         state_out, kda::Seqs{nullptr, N, 1, N}, D, 0, 0};
  return finish(fn, conv_fwd_dispatch(a, true, dtype, wide, W, stream));
}

size_t kda_short_conv_bwd_workspace_size(int B, int T, int D, int W) {
  if (B < 0 || T < 0 || D < 1 || W < 2 || W > 4) return 0;
  return (size_t)kda::conv::bwd_lines((long long)B * T, D) * D * (W + 1) * sizeof(float);
}

kda_status_t kda_short_conv_bwd(const void* x, long long x_stride, const void* weight, const void* bias,
                                kda_dtype_t weight_dtype, const void* state, const void* dy, kda_dtype_t dy_dtype,
                                const float* dstate, void* dx, float* dweight, float* dbias, float* dinit,
                                const int32_t* cu_seqlens, int num_seqs, int B, int T, int D, int W,
                                kda_dtype_t dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "kda_short_conv_bwd";
  clear_status();
  kda::Seqs q;
  if (kda_status_t st = check_seqs(fn, cu_seqlens, num_seqs, B, T, &q)) return st;
  if (kda_status_t st = conv_check(fn, x, x_stride, weight, bias, weight_dtype, q.total, D, W, dtype)) return st;
  if (!known(dy_dtype) || (dy_dtype != dtype && dy_dtype != KDA_F32))
    return fail(KDA_ERR_UNSUPPORTED, "%s: dy_dtype %d (need dtype or fp32)", fn, (int)dy_dtype);
  if (!dweight || (q.total > 0 && (!dy || !dx))) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const unsigned es = bytes_of(dtype);
  if (!all_aligned({state, dx}, es) || !all_aligned({dy}, bytes_of(dy_dtype)) ||
      !all_aligned({dstate, dweight, dbias, dinit}, 4))
    return misaligned(fn, "a pointer is not element-aligned");
  if (overlaps({dx, dweight, dbias, dinit}, {x, weight, bias, state, dy, dstate, cu_seqlens, workspace}) ||
      repeated({dx, dweight, dbias, dinit}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  if (kda_status_t st =
          check_workspace(fn, workspace, workspace_bytes, kda_short_conv_bwd_workspace_size(B, T, D, W)))
    return st;
  const bool wide = D % 4 == 0 && x_stride % 4 == 0 && all_aligned({x, state, dx}, 4 * es) &&
                    all_aligned({dy}, 4 * bytes_of(dy_dtype)) && all_aligned({dstate, dinit}, 16) &&
                    conv_params_wide(weight, bias, weight_dtype, 4);
  const kda::conv::BwdArgs a{x,  x_stride, weight, bias, weight_dtype == KDA_BF16, state, dy, dstate, dx, dinit,
                             static_cast<float*>(workspace), q, D, 0, 0};
  cudaError_t e;
  if (dtype == KDA_F32) e = conv_bwd_dispatch<float, float>(a, wide, W, dweight, dbias, stream);
  else if (dy_dtype == KDA_F32) e = conv_bwd_dispatch<__nv_bfloat16, float>(a, wide, W, dweight, dbias, stream);
  else e = conv_bwd_dispatch<__nv_bfloat16, __nv_bfloat16>(a, wide, W, dweight, dbias, stream);
  return finish(fn, e);
}

}  // extern "C"

// --------------------------------------------------------------------- scan
namespace {

kda_status_t scan_check_sizes(const char* fn, int d, int S, int groups, kda_dtype_t dtype) {
  if (!known(dtype)) return fail(KDA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
  if (d < 1 || groups < 1 || d % groups)
    return fail(KDA_ERR_INVALID_ARG, "%s: d=%d groups=%d (groups must divide d)", fn, d, groups);
  if (!kda::scan::supported_state(S)) return fail(KDA_ERR_UNSUPPORTED, "%s: S=%d (need 8, 16, 32 or 64)", fn, S);
  if (d > (1 << 24)) return fail(KDA_ERR_UNSUPPORTED, "%s: d=%d is too large", fn, d);
  return KDA_OK;
}

kda_status_t scan_check_inputs(const char* fn, const kda::scan::Args& a, long long tokens, int S, int groups,
                               kda_dtype_t dtype) {
  if (!a.A || (tokens > 0 && (!a.x || !a.dt || !a.B || !a.C))) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const long long bc = (long long)groups * S;
  if (a.xs < a.d || a.dts < a.d || (a.z && a.zs < a.d) || a.bs < bc || a.cs < bc)
    return fail(KDA_ERR_INVALID_ARG, "%s: a stride is smaller than its row", fn);
  if (!all_aligned({a.x, a.dt, a.z, a.B, a.C, a.y, a.dy}, bytes_of(dtype)) || !all_aligned({a.Dv, a.dt_bias}, 4))
    return misaligned(fn, "a pointer is not element-aligned");
  if (!all_aligned({a.A, a.S0, a.S_out, a.dS}, 16)) return misaligned(fn, "A or a state is not 16-byte aligned");
  return KDA_OK;
}

#define KDA_SCAN_DISPATCH(e, FN, ...)                                       \
  do {                                                                      \
    if (dtype == KDA_BF16) {                                                \
      if (S == 8) e = kda::scan::FN<__nv_bfloat16, 8>(__VA_ARGS__);         \
      else if (S == 16) e = kda::scan::FN<__nv_bfloat16, 16>(__VA_ARGS__);  \
      else if (S == 32) e = kda::scan::FN<__nv_bfloat16, 32>(__VA_ARGS__);  \
      else e = kda::scan::FN<__nv_bfloat16, 64>(__VA_ARGS__);               \
    } else {                                                                \
      if (S == 8) e = kda::scan::FN<float, 8>(__VA_ARGS__);                 \
      else if (S == 16) e = kda::scan::FN<float, 16>(__VA_ARGS__);          \
      else if (S == 32) e = kda::scan::FN<float, 32>(__VA_ARGS__);          \
      else e = kda::scan::FN<float, 64>(__VA_ARGS__);                       \
    }                                                                       \
  } while (0)

}  // namespace

extern "C" {

size_t kda_selective_scan_fwd_workspace_size(int B, int T, int d, int S, int groups, int num_seqs) {
  if (B < 0 || T < 0 || num_seqs < 0 || d < 1 || groups < 1 || d % groups || !kda::scan::supported_state(S)) return 0;
  const kda::scan::FwdPlan p = kda::scan::fwd_plan(B, T, d, groups, S);
  if (!p.split) return 0;
  return kda::scan::round256(kda::scan::carry_floats(p.chunks, d, S) * 4) + (size_t)p.chunks * d * 4;
}

kda_status_t kda_selective_scan_fwd(const void* x, long long x_stride, const void* dt, long long dt_stride,
                                    const float* A, const void* Bm, long long B_stride, const void* Cm,
                                    long long C_stride, const float* Dskip, const void* z, long long z_stride,
                                    const float* dt_bias, const float* S0, void* y, float* S_out,
                                    const int32_t* cu_seqlens, int num_seqs, int B, int T, int d, int S, int groups,
                                    kda_dtype_t dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "kda_selective_scan_fwd";
  clear_status();
  kda::scan::Args a = {};
  if (kda_status_t st = check_seqs(fn, cu_seqlens, num_seqs, B, T, &a.q)) return st;
  if (kda_status_t st = scan_check_sizes(fn, d, S, groups, dtype)) return st;
  if (a.q.num == 0) return KDA_OK;
  a.x = x, a.dt = dt, a.z = z, a.B = Bm, a.C = Cm;
  a.xs = x_stride, a.dts = dt_stride, a.zs = z_stride, a.bs = B_stride, a.cs = C_stride;
  a.A = A, a.Dv = Dskip, a.dt_bias = dt_bias, a.S0 = S0, a.y = y, a.S_out = S_out, a.d = d, a.cpg = d / groups;
  if (kda_status_t st = scan_check_inputs(fn, a, a.q.total, S, groups, dtype)) return st;
  if (a.q.total > 0 && !y) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (overlaps({y, S_out}, {x, dt, z, Bm, Cm, A, Dskip, dt_bias, S0, cu_seqlens, workspace}) || repeated({y, S_out}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  if (kda_status_t st = check_workspace(fn, workspace, workspace_bytes,
                                        kda_selective_scan_fwd_workspace_size(B, T, d, S, groups, num_seqs)))
    return st;
  const kda::scan::FwdPlan p = kda::scan::fwd_plan(B, T, d, groups, S);
  a.L = p.L, a.chunks = p.chunks;
  a.ncb = kda::scan::channel_blocks(d, groups, S);
  a.blocks_per_group = a.ncb / groups;
  if (p.split) {
    a.entry = static_cast<float*>(workspace);
    a.sumd = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                      kda::scan::round256(kda::scan::carry_floats(p.chunks, d, S) * 4));
  }
  cudaError_t e;
  KDA_SCAN_DISPATCH(e, launch_fwd, a, p.split, stream);
  return finish(fn, e);
}

kda_status_t kda_selective_scan_step(const void* x, long long x_stride, const void* dt, long long dt_stride,
                                     const float* A, const void* Bm, long long B_stride, const void* Cm,
                                     long long C_stride, const float* Dskip, const void* z, long long z_stride,
                                     const float* dt_bias, const float* St, void* y, float* S_out, int N, int d,
                                     int S, int groups, kda_dtype_t dtype, cudaStream_t stream) {
  const char* fn = "kda_selective_scan_step";
  clear_status();
  if (N < 0) return fail(KDA_ERR_INVALID_ARG, "%s: bad size N=%d", fn, N);
  if (kda_status_t st = scan_check_sizes(fn, d, S, groups, dtype)) return st;
  if (N == 0) return KDA_OK;
  kda::scan::Args a = {};
  a.q = kda::Seqs{nullptr, N, 1, N};
  a.x = x, a.dt = dt, a.z = z, a.B = Bm, a.C = Cm;
  a.xs = x_stride, a.dts = dt_stride, a.zs = z_stride, a.bs = B_stride, a.cs = C_stride;
  a.A = A, a.Dv = Dskip, a.dt_bias = dt_bias, a.S0 = St, a.y = y, a.S_out = S_out, a.d = d, a.cpg = d / groups;
  if (kda_status_t st = scan_check_inputs(fn, a, N, S, groups, dtype)) return st;
  if (!St || !y || !S_out) return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (overlaps({y}, {x, dt, z, Bm, Cm, A, Dskip, dt_bias, St}) ||
      overlaps({S_out}, {x, dt, z, Bm, Cm, A, Dskip, dt_bias}) || repeated({y, S_out}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  cudaError_t e;
  KDA_SCAN_DISPATCH(e, launch_step, a, stream);
  return finish(fn, e);
}

size_t kda_selective_scan_bwd_workspace_size(int B, int T, int d, int S, int groups) {
  if (B < 0 || T < 0 || d < 1 || groups < 1 || d % groups || !kda::scan::supported_state(S)) return 0;
  return kda::scan::bwd_layout((long long)B * T, d, groups, S).total;
}

kda_status_t kda_selective_scan_bwd(const void* x, long long x_stride, const void* dt, long long dt_stride,
                                    const float* A, const void* Bm, long long B_stride, const void* Cm,
                                    long long C_stride, const float* Dskip, const void* z, long long z_stride,
                                    const float* dt_bias, const float* S0, const void* dy, const float* dS, void* dx,
                                    void* ddt, float* dA, float* dB, float* dC, float* dDskip, void* dz,
                                    float* ddt_bias, float* dS0, const int32_t* cu_seqlens, int num_seqs, int B,
                                    int T, int d, int S, int groups, kda_dtype_t dtype, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "kda_selective_scan_bwd";
  clear_status();
  kda::scan::Args a = {};
  if (kda_status_t st = check_seqs(fn, cu_seqlens, num_seqs, B, T, &a.q)) return st;
  if (kda_status_t st = scan_check_sizes(fn, d, S, groups, dtype)) return st;
  a.x = x, a.dt = dt, a.z = z, a.B = Bm, a.C = Cm;
  a.xs = x_stride, a.dts = dt_stride, a.zs = z_stride, a.bs = B_stride, a.cs = C_stride;
  a.A = A, a.Dv = Dskip, a.dt_bias = dt_bias, a.S0 = S0, a.d = d, a.cpg = d / groups, a.dy = dy, a.dS = dS;
  if (kda_status_t st = scan_check_inputs(fn, a, a.q.total, S, groups, dtype)) return st;
  if (!dA || (a.q.total > 0 && (!dy || !dx || !ddt || !dB || !dC || (z && !dz))))
    return fail(KDA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!all_aligned({dx, ddt, dz}, bytes_of(dtype)) || !all_aligned({dA, dB, dC, dDskip, ddt_bias}, 4))
    return misaligned(fn, "a pointer is not element-aligned");
  if (!all_aligned({dS0}, 16)) return misaligned(fn, "dS0 is not 16-byte aligned");
  if (overlaps({dx, ddt, dz, dA, dB, dC, dDskip, ddt_bias, dS0},
               {x, dt, z, Bm, Cm, A, Dskip, dt_bias, S0, dy, dS, cu_seqlens, workspace}) ||
      repeated({dx, ddt, dz, dA, dB, dC, dDskip, ddt_bias, dS0}))
    return fail(KDA_ERR_INVALID_ARG, "%s: an output aliases an input or another output", fn);
  if (kda_status_t st = check_workspace(fn, workspace, workspace_bytes,
                                        kda_selective_scan_bwd_workspace_size(B, T, d, S, groups)))
    return st;
  kda::scan::BwdOut o = {};
  o.dx = dx, o.ddt = ddt, o.dz = dz, o.dS0 = dS0;
  cudaError_t e;
  KDA_SCAN_DISPATCH(e, launch_bwd, a, o, dA, dB, dC, dDskip, ddt_bias, groups, workspace, stream);
  return finish(fn, e);
}

}  // extern "C"

// kda_norm.cuh -- root-mean-square norm of rows, with the residual's addition
// and, on request, an e4m3 output with one scale a row or a group of columns;
// and its backward pass.
//
//   s = x + residual;  r = 1 / sqrt(mean(s^2) + eps);  y = s r w
//   quantised: scale = max(amax |y| over the group, 1e-10) / 448, q = e4m3(y / scale)
//   backward:  dx = r w dy - s r^3 mean(w dy s) + ds;  dw = sum over rows of dy s r
//
// A row is read once and stays in registers: TPR threads hold it as NV vectors
// each of VEC elements (16 bytes), strided so that neighbouring threads hold
// neighbouring vectors.  Rows of up to 32 vectors a lane group take part of a
// warp (several rows a warp), longer ones a whole CTA.  Sums are fp32.
// HBM-bound: the traffic is the inputs once and the outputs once.
#pragma once
#include <cuda_fp8.h>

#include "kda_layer_common.cuh"

namespace kda {
namespace norm {

constexpr float kFp8Max = 448.f;
constexpr float kScaleFloor = 1e-10f;
constexpr int kMaxDim = 16384;
enum QuantMode : int { kNone = 0, kRow = 1, kGroup = 2 };

struct FwdArgs {
  const void* x;
  long long x_stride;
  const void* residual;
  const void* weight;
  int w_bf16;
  void* y;      // T, or e4m3 bytes
  float* scale; // [rows, D / group]
  void* s;      // T, or nullptr
  long long rows;
  int D, group;
  float eps;
};

// Sum (or maximum) over the TPR threads of a row; every thread gets it.
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* smem) {
  constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, u) : v + u;
  }
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) smem[warp] = v;
    __syncthreads();
    v = smem[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v = kMax ? max_nan(v, smem[i]) : v + smem[i];
  }
  return v;
}

template <int VEC>
__device__ __forceinline__ void store_fp8(uint8_t* p, const float (&v)[VEC]) {
  // saturating round to nearest even; NaN stays NaN
  if constexpr (VEC == 1) {
    *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    if constexpr (VEC == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

template <typename T, int VEC, int TPR, int NV, int QUANT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) kda_rms_norm_fwd_kernel(const FwdArgs a) {
  constexpr int NT = TPR < 128 ? 128 : TPR;
  constexpr int RPC = NT / TPR;  // rows a CTA
  __shared__ float s_red[2][32];
  const int j = threadIdx.x % TPR;
  const long long row0 = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
  const bool live = row0 < a.rows;
  const long long row = live ? row0 : a.rows - 1;
  const int nvec = a.D / VEC;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.D : nullptr;

  float v[NV][VEC];
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = j + i * TPR;
    if (c < nvec) load_f32<T, VEC>(x + (long long)c * VEC, v[i]);
    else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
    }
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) {
        float u[VEC];
        load_f32<T, VEC>(res + (long long)c * VEC, u);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] += u[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc = fmaf(v[i][e], v[i][e], acc);
  // the sum is taken of the unrounded s (the stored s is rounded once, to T)
  const float r = rsqrtf(row_reduce<TPR, false>(acc, s_red[0]) / (float)a.D + a.eps);
  if (a.s && live) {
    T* s = static_cast<T*>(a.s) + row * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) store_pack<T, VEC>(s + (long long)c * VEC, v[i]);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = j + i * TPR;
    if (c < nvec) {
      float w[VEC];
      load_param<VEC>(a.weight, a.w_bf16, (long long)c * VEC, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] = v[i][e] * r * w[e];
        if (QUANT == kRow) amax = max_nan(amax, fabsf(v[i][e]));
      }
    }
  }
  if constexpr (QUANT == kNone) {
    if (!live) return;
    T* y = static_cast<T*>(a.y) + row * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) store_pack<T, VEC>(y + (long long)c * VEC, v[i]);
    }
  } else {
    uint8_t* q = static_cast<uint8_t*>(a.y) + row * a.D;
    if constexpr (QUANT == kRow) {
      amax = max_nan(row_reduce<TPR, true>(amax, s_red[1]), kScaleFloor);
      if (live && j == 0) a.scale[row] = amax / kFp8Max;
    }
    const int gl = QUANT == kGroup ? a.group / VEC : 1;  // lanes of one group
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if constexpr (QUANT == kGroup) {
        amax = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = max_nan(amax, fabsf(v[i][e]));
        for (int o = gl >> 1; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        amax = max_nan(amax, kScaleFloor);
        if (live && c < nvec && (c & (gl - 1)) == 0) a.scale[row * (a.D / a.group) + c / gl] = amax / kFp8Max;
      }
      const float inv = kFp8Max / amax;
      if (live && c < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] *= inv;
        store_fp8<VEC>(q + (long long)c * VEC, v[i]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  Each CTA takes rows in turn (blockIdx, + gridDim, ...) and keeps
// its threads' columns of dw in registers over all of them; one line of
// partial sums per row group goes to the workspace and a second kernel adds
// the lines in order, so the result does not depend on scheduling.
// ---------------------------------------------------------------------------
struct BwdArgs {
  const void *dy, *s, *weight;
  int w_bf16;
  const void* ds;
  void* dx;
  float* partial;  // [lines, D]
  long long rows;
  int D;
  float eps;
};

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) kda_rms_norm_bwd_kernel(const BwdArgs a) {
  constexpr int NT = TPR < 128 ? 128 : TPR;
  constexpr int RPC = NT / TPR;
  __shared__ float s_red[2][2][32];
  const int j = threadIdx.x % TPR;
  const int nvec = a.D / VEC;
  const long long line = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
  const long long step = (long long)gridDim.x * RPC;
  float dw[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
  int buf = 0;
  // every row group of the CTA runs the same number of turns (reductions are CTA-wide or warp-wide)
  for (long long base = (long long)blockIdx.x * RPC; base < a.rows; base += step, buf ^= 1) {
    const long long row0 = base + threadIdx.x / TPR;
    const bool live = row0 < a.rows;
    const long long row = live ? row0 : a.rows - 1;
    const T* dy = static_cast<const T*>(a.dy) + row * a.D;
    const T* s = static_cast<const T*>(a.s) + row * a.D;
    float g[NV][VEC], v[NV][VEC];
    float ss = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) {
        load_f32<T, VEC>(dy + (long long)c * VEC, g[i]);
        load_f32<T, VEC>(s + (long long)c * VEC, v[i]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[i][e] = v[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) {
        float w[VEC];
        load_param<VEC>(a.weight, a.w_bf16, (long long)c * VEC, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ss = fmaf(v[i][e], v[i][e], ss);
          gs = fmaf(g[i][e] * w[e], v[i][e], gs);
        }
      }
    }
    ss = row_reduce<TPR, false>(ss, s_red[buf][0]);
    gs = row_reduce<TPR, false>(gs, s_red[buf][1]);
    const float r = rsqrtf(ss / (float)a.D + a.eps);
    const float k = r * r * r * (gs / (float)a.D);
    T* dx = static_cast<T*>(a.dx) + row * a.D;
    const T* ds = a.ds ? static_cast<const T*>(a.ds) + row * a.D : nullptr;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = j + i * TPR;
        if (c < nvec) {
          float w[VEC], o[VEC], u[VEC];
          load_param<VEC>(a.weight, a.w_bf16, (long long)c * VEC, w);
          if (ds) load_f32<T, VEC>(ds + (long long)c * VEC, u);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            dw[i][e] = fmaf(g[i][e] * v[i][e], r, dw[i][e]);
            o[e] = r * w[e] * g[i][e] - k * v[i][e] + (ds ? u[e] : 0.f);
          }
          store_pack<T, VEC>(dx + (long long)c * VEC, o);
        }
      }
    }
  }
  float* p = a.partial + line * a.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = j + i * TPR;
    if (c < nvec) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) p[(long long)c * VEC + e] = dw[i][e];
    }
  }
}

// Host: the row shapes built, smallest first.  `vecs` vectors a row.
struct RowShape {
  int tpr, nv;
};
inline RowShape row_shape(int vecs) {
  if (vecs <= 8) return {8, 1};
  if (vecs <= 16) return {16, 1};
  if (vecs <= 32) return {32, 1};
  if (vecs <= 64) return {32, 2};
  if (vecs <= 128) return {32, 4};
  if (vecs <= 256) return {128, 2};
  if (vecs <= 512) return {128, 4};
  if (vecs <= 1024) return {256, 4};
  if (vecs <= 2048) return {512, 4};
  if (vecs <= 4096) return {512, 8};
  if (vecs <= 8192) return {512, 16};
  return {512, 32};
}

#define KDA_NORM_SHAPES(CASE) \
  CASE(8, 1) CASE(16, 1) CASE(32, 1) CASE(32, 2) CASE(32, 4) CASE(128, 2) CASE(128, 4) CASE(256, 4) CASE(512, 4)
#define KDA_NORM_SHAPES_LONG(CASE) CASE(512, 8)
#define KDA_NORM_SHAPES_SCALAR(CASE) CASE(512, 16) CASE(512, 32)

template <typename T, int VEC, int QUANT>
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t st) {
  const RowShape sh = row_shape(a.D / VEC);
#define KDA_CASE(TPR, NV)                                                                             \
  if (sh.tpr == TPR && sh.nv == NV) {                                                                  \
    constexpr int NT = TPR < 128 ? 128 : TPR;                                                           \
    const long long grid = (a.rows + NT / TPR - 1) / (NT / TPR);                                        \
    kda_rms_norm_fwd_kernel<T, VEC, TPR, NV, QUANT><<<(unsigned)grid, NT, 0, st>>>(a);                  \
    return cudaGetLastError();                                                                          \
  }
  KDA_NORM_SHAPES(KDA_CASE)
  if constexpr (VEC < 8) { KDA_NORM_SHAPES_LONG(KDA_CASE) }
  if constexpr (VEC == 1) { KDA_NORM_SHAPES_SCALAR(KDA_CASE) }
#undef KDA_CASE
  return cudaErrorInvalidValue;
}

// Lines of partial sums of the backward: one per row group of each CTA.
struct BwdPlan {
  int grid, rpc;
};
inline BwdPlan bwd_plan(long long rows, int vecs) {
  const RowShape sh = row_shape(vecs);
  const int nt = sh.tpr < 128 ? 128 : sh.tpr, rpc = nt / sh.tpr;
  const long long want = (rows + rpc - 1) / rpc, most = 148LL * (1024 / nt);
  return {(int)(want < most ? want : most), rpc};
}

template <typename T, int VEC>
cudaError_t launch_bwd(const BwdArgs& a, float* dweight, cudaStream_t st) {
  const RowShape sh = row_shape(a.D / VEC);
  const BwdPlan plan = bwd_plan(a.rows, a.D / VEC);
  cudaError_t e = cudaErrorInvalidValue;
#define KDA_CASE(TPR, NV)                                                                             \
  if (sh.tpr == TPR && sh.nv == NV) {                                                                  \
    kda_rms_norm_bwd_kernel<T, VEC, TPR, NV><<<plan.grid, TPR < 128 ? 128 : TPR, 0, st>>>(a);            \
    e = cudaGetLastError();                                                                             \
  }
  KDA_NORM_SHAPES(KDA_CASE)
  if constexpr (VEC < 8) { KDA_NORM_SHAPES_LONG(KDA_CASE) }
  if constexpr (VEC == 1) { KDA_NORM_SHAPES_SCALAR(KDA_CASE) }
#undef KDA_CASE
  if (e != cudaSuccess) return e;
  return launch_sum_lines(a.partial, dweight, nullptr, a.D, plan.grid * plan.rpc, a.D, st);
}

}  // namespace norm
}  // namespace kda

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
// neighbouring vectors.  Rows of up to 32 vectors take part of a warp, and a
// thread then takes RU = 2 rows at once, so that their loads and exchanges overlap;
// longer ones take a CTA.  Sums are fp32.  HBM-bound: the traffic is the inputs
// once and the outputs once.  16384 rows of 4096 bf16 with residual: 84 us, 6.4
// TB/s; backward with ds 89 us, 6.0 TB/s; 524288 rows of 128 to e4m3: 51 us, 4.0
// TB/s (two rows of a thread share too little: issue shows); 3001 rows of 1153 fp32
// to e4m3, element by element: 11 us, 4.1 TB/s.
#pragma once
#include <cuda_fp8.h>

#include "kda_layer_common.cuh"

namespace kda {
namespace norm {

constexpr float kFp8Max = 448.f;
constexpr float kScaleFloor = 1e-10f;
constexpr int kMaxDim = 16384;
// What is stored: T, e4m3 with a scale a row, or with a scale a group of columns
// (the mode is then the lanes of one group, 4 to 32).
enum QuantMode : int { kNone = 0, kRow = 1, kGroup = 4 };

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
  int groups;      // scales a row
  int turns;       // rows a thread takes one after the other (RU at a time)
};

// Sum (or maximum) of NVAL values each over the TPR threads of a row; every
// thread gets them.  Rows of several warps go through `smem` (a line of 32 a
// value); one barrier, so two lots of smem take turns.
template <int TPR, bool kMax, int NVAL>
__device__ __forceinline__ void row_reduce(float (&v)[NVAL], float (*smem)[32]) {
  constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NVAL; ++i) {
      const float u = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = kMax ? max_nan(v[i], u) : v[i] + u;
    }
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NVAL; ++i) smem[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NVAL; ++i) v[i] = smem[i][lane % NW];
#pragma unroll
    for (int o = NW / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < NVAL; ++i) {
        const float u = __shfl_xor_sync(0xffffffffu, v[i], o);
        v[i] = kMax ? max_nan(v[i], u) : v[i] + u;
      }
  }
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

// v /= scale, rounded as a division is, so that q is e4m3(y / scale) of the very
// scale that is stored and a quotient half way between two e4m3 values goes to
// the even one (one ten-thousandth of the quotients of bf16 rows are: the norm's
// factor cancels in them).  A quotient q by an approximate reciprocal i becomes
// q + (y - q scale) i, the remainder exact in a fused multiply-add (P. Markstein,
// IBM J. Res. Dev. 34, 1990).  An infinite scale gives 0, and NaN for what is
// infinite itself.
template <int VEC>
__device__ __forceinline__ void divide_by(float (&v)[VEC], float scale) {
  const bool inf = scale == INFINITY;
  float i = fast_rcp(scale);  // no flush: 1 / scale is between 1.3e-36 and 4.5e12
  i = inf ? 0.f : fmaf(i, fmaf(-scale, i, 1.f), i);
  const float d = inf ? 0.f : scale;
  // the remainder as q scale - y, times -i: so that -0 stays -0
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 q = mul2(make_float2(v[e], v[e + 1]), dup2(i));
      const float2 r = fma2(fma2(q, dup2(d), make_float2(-v[e], -v[e + 1])), dup2(-i), q);
      v[e] = r.x;
      v[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float q = v[e] * i;
      v[e] = fmaf(fmaf(q, d, -v[e]), -i, q);
    }
  }
}

constexpr int threads_of(int tpr) { return tpr <= 32 ? 128 : tpr; }  // a row of several warps has its CTA to itself
// Rows a thread takes at once: a row of one vector is too little work to cover
// its own loads and exchanges.
constexpr int rows_at_once(int tpr, int nv) { return tpr <= 32 && nv == 1 ? 2 : 1; }

// Rows in turn (rows of one vector a thread, at most a warp): inputs arrive by
// asynchronous copies kRing - 1 turns ahead, in a ring that each thread has to
// itself (a turn ahead in registers: 84 us for 524288 rows of 128, 36% of the
// copy rate).
constexpr int kRing = 4;

template <typename T, int VEC, int TPR, int NV, int QUANT>
__global__ void __launch_bounds__(threads_of(TPR)) kda_rms_norm_fwd_kernel(const FwdArgs a) {
  constexpr int NT = threads_of(TPR);
  constexpr int RPC = NT / TPR;  // row slots of a CTA
  constexpr int RU = rows_at_once(TPR, NV);
  constexpr bool kTurns = TPR <= 32 && NV == 1;
  constexpr bool kAsync = kTurns && VEC > 1;
  constexpr int GL = QUANT >= kGroup ? QUANT : 1;  // lanes of one group
  __shared__ float s_red[2][RU][32];
  __shared__ Pack<T, VEC> s_in[kAsync ? kRing : 1][kAsync ? RU : 1][2][kAsync ? NT : 1];
  const int j = threadIdx.x % TPR;
  const int nvec = a.D / VEC;
  const int turns = kTurns ? a.turns : 1;
  const long long row0 = ((long long)blockIdx.x * turns * RPC + threadIdx.x / TPR) * RU;  // the thread's first row
  constexpr int kStep = RPC * RU;
  // rows from row0 on; a turn's rows are counted from it
  const int left = (int)(a.rows - row0 < (1 << 20) ? a.rows - row0 : (1 << 20));
  const T* xp = static_cast<const T*>(a.x) + row0 * a.x_stride + j * VEC;
  const T* rp = a.residual ? static_cast<const T*>(a.residual) + row0 * a.D + j * VEC : nullptr;

  Pack<T, VEC> px[RU][NV], pr[RU][NV];
  // rows past the end are not read and not written
  auto fetch = [&](int first) {
    if constexpr (!kAsync) {
#pragma unroll
      for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (first + u < left && j + i * TPR < nvec) {
            px[u][i] = load_pack<T, VEC>(xp + u * a.x_stride + i * TPR * VEC);
            if (rp) pr[u][i] = load_pack<T, VEC>(rp + u * a.D + i * TPR * VEC);
          }
      xp += kStep * a.x_stride;
      if (rp) rp += (long long)kStep * a.D;
    }
  };
  int ahead = 0, slot = 0;  // first row to stage; the ring's slot to fill
  auto stage = [&] {
    if constexpr (kAsync) {
      if (ahead < turns * kStep && j < nvec) {
#pragma unroll
        for (int u = 0; u < RU; ++u)
          if (ahead + u < left) {
            copy_async<sizeof(T) * VEC>(&s_in[slot][u][0][threadIdx.x], xp + u * a.x_stride);
            if (rp) copy_async<sizeof(T) * VEC>(&s_in[slot][u][1][threadIdx.x], rp + u * a.D);
          }
      }
      copy_async_commit();
      xp += kStep * a.x_stride;
      if (rp) rp += (long long)kStep * a.D;
      ahead += kStep;
      slot = slot + 1 < kRing ? slot + 1 : 0;
    }
  };
  if constexpr (kAsync) {
#pragma unroll
    for (int g = 0; g < kRing - 1; ++g) stage();
  } else {
    fetch(0);
  }
  float w[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (j + i * TPR < nvec) load_param<VEC>(a.weight, a.w_bf16, (long long)(j + i * TPR) * VEC, w[i]);
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[i][e] = 0.f;
  }
  const float inv_d = 1.f / (float)a.D;
  char* yp = static_cast<char*>(a.y) + (row0 * a.D + j * VEC) * (QUANT == kNone ? sizeof(T) : 1);
  T* sp = a.s ? static_cast<T*>(a.s) + row0 * a.D + j * VEC : nullptr;
  float* scp = QUANT != kNone ? a.scale + row0 * a.groups + (QUANT >= kGroup ? j / GL : 0) : nullptr;
  int read = 0;
#pragma unroll 1
  for (int row = 0; row < turns * kStep; row += kStep) {
    if (RPC > 1 && row >= left + (int)(threadIdx.x / TPR) * RU) return;  // uniform: a CTA's slots are consecutive rows
    float v[RU][NV][VEC], acc[RU];
    if constexpr (kAsync) {
      stage();
      copy_async_wait<kRing - 1>();
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      acc[u] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (row + u < left && j + i * TPR < nvec) {
          unpack<T, VEC>(kAsync ? s_in[read][kAsync ? u : 0][0][kAsync ? threadIdx.x : 0] : px[u][i], v[u][i]);
          if (rp) {
            float q[VEC];
            unpack<T, VEC>(kAsync ? s_in[read][kAsync ? u : 0][1][kAsync ? threadIdx.x : 0] : pr[u][i], q);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[u][i][e] += q[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[u][i][e] = 0.f;
        }
        acc[u] += dot<VEC>(v[u][i], v[u][i]);
      }
    }
    if (kAsync) read = read + 1 < kRing ? read + 1 : 0;
    if (!kAsync && row + kStep < turns * kStep) fetch(row + kStep);
    if (sp) {
#pragma unroll
      for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (row + u < left && j + i * TPR < nvec) store_pack<T, VEC>(sp + u * a.D + i * TPR * VEC, v[u][i]);
      sp += (long long)kStep * a.D;
    }
    // the sum is taken of the unrounded s (the stored s is rounded once, to T)
    row_reduce<TPR, false>(acc, s_red[0]);
    float amax[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const float r = rsqrtf(acc[u] * inv_d + a.eps);
      amax[u] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        scale_by<VEC>(v[u][i], r);
        scale_by<VEC>(v[u][i], w[i]);
        if (QUANT == kRow) amax[u] = max_abs_nan<VEC>(amax[u], v[u][i]);
      }
    }
    if constexpr (QUANT == kNone) {
#pragma unroll
      for (int u = 0; u < RU; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (row + u < left && j + i * TPR < nvec)
            store_pack<T, VEC>(reinterpret_cast<T*>(yp) + u * a.D + i * TPR * VEC, v[u][i]);
      yp += (long long)kStep * a.D * sizeof(T);
    } else {
      if constexpr (QUANT == kRow) row_reduce<TPR, true>(amax, s_red[1]);
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        const bool live = row + u < left;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = j + i * TPR;
          float m = amax[u];
          if constexpr (QUANT >= kGroup) {
            m = max_abs_nan<VEC>(0.f, v[u][i]);
#pragma unroll
            for (int o = 1; o < GL; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
          }
          // m / 448, within a unit in the last place; the floor's quotient is exact
          const float scale = m <= kScaleFloor ? kScaleFloor / kFp8Max : m * (1.f / kFp8Max);
          if (live && c < nvec && (QUANT >= kGroup ? j % GL == 0 : c == 0))
            scp[u * a.groups + (QUANT >= kGroup ? i * (TPR / GL) : 0)] = scale;
          if (live && c < nvec) {
            divide_by<VEC>(v[u][i], scale);
            store_fp8<VEC>(reinterpret_cast<uint8_t*>(yp) + u * a.D + i * TPR * VEC, v[u][i]);
          }
        }
      }
      yp += (long long)kStep * a.D;
      scp += (long long)kStep * a.groups;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  Each CTA takes rows in turn (blockIdx, + gridDim, ...), loads the
// next while it works on one, and keeps its threads' columns of dw in registers
// over all of them; one line of partial sums per CTA goes to the workspace
// and a second kernel adds the lines in order, so the result does not depend on
// scheduling.
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

// Rows of up to two vectors a thread arrive by asynchronous copies, two turns
// ahead, in a ring that each thread has to itself.
constexpr int kBwdRing = 3;
constexpr bool bwd_async(int vec, int nv) { return vec > 1 && nv <= 2; }

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(threads_of(TPR), NV * VEC <= 16 ? 512 / threads_of(TPR) : 1)
    kda_rms_norm_bwd_kernel(const BwdArgs a) {
  constexpr int NT = threads_of(TPR);
  constexpr int RPC = NT / TPR;
  constexpr bool kKeepW = NV * VEC <= 16;  // weights in registers, or read again for each row
  constexpr bool kAsync = bwd_async(VEC, NV);
  constexpr bool kAhead = VEC == 1 && NV <= 4;  // the next row's loads in registers; longer rows hide their own
  extern __shared__ __align__(16) unsigned char smem_raw[];
  auto ring = reinterpret_cast<Pack<T, VEC>(*)[3][NV][NT]>(smem_raw);  // dy, s, ds
  __shared__ float s_red[2][2][32];
  const int j = threadIdx.x % TPR;
  const int nvec = a.D / VEC;
  const long long step = (long long)gridDim.x * RPC;
  float dw[NV][VEC], w[kKeepW ? NV : 1][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
    if (kKeepW && j + i * TPR < nvec) load_param<VEC>(a.weight, a.w_bf16, (long long)(j + i * TPR) * VEC, w[kKeepW ? i : 0]);
  }
  Pack<T, VEC> pg[NV], ps[NV], pd[NV];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (row < a.rows && c < nvec) {
        pg[i] = load_pack<T, VEC>(static_cast<const T*>(a.dy) + row * a.D + (long long)c * VEC);
        ps[i] = load_pack<T, VEC>(static_cast<const T*>(a.s) + row * a.D + (long long)c * VEC);
        if (kAhead && a.ds) pd[i] = load_pack<T, VEC>(static_cast<const T*>(a.ds) + row * a.D + (long long)c * VEC);
      }
    }
  };
  int slot = 0, read = 0;
  auto stage = [&](long long row) {
    if constexpr (kAsync) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = j + i * TPR;
        if (row < a.rows && c < nvec) {
          const long long at = row * a.D + (long long)c * VEC;
          copy_async<sizeof(T) * VEC>(&ring[slot][0][i][threadIdx.x], static_cast<const T*>(a.dy) + at);
          copy_async<sizeof(T) * VEC>(&ring[slot][1][i][threadIdx.x], static_cast<const T*>(a.s) + at);
          if (a.ds) copy_async<sizeof(T) * VEC>(&ring[slot][2][i][threadIdx.x], static_cast<const T*>(a.ds) + at);
        }
      }
      copy_async_commit();
      slot = slot + 1 < kBwdRing ? slot + 1 : 0;
    }
  };
  const long long own = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
  if constexpr (kAsync) {
#pragma unroll
    for (int g = 0; g < kBwdRing - 1; ++g) stage(own + g * step);
  }
  if (kAhead) fetch(own);
  int buf = 0;
  const float inv_d = 1.f / (float)a.D;
  // every row slot of the CTA runs the same number of turns (reductions are CTA-wide or warp-wide)
  for (long long base = (long long)blockIdx.x * RPC; base < a.rows; base += step, buf ^= 1) {
    const long long row = base + threadIdx.x / TPR;
    const bool live = row < a.rows;
    float g[NV][VEC], v[NV][VEC];
    Pack<T, VEC> d[kAhead ? NV : 1];
    if constexpr (kAsync) {
      stage(row + (kBwdRing - 1) * step);
      copy_async_wait<kBwdRing - 1>();
    } else if (!kAhead) {
      fetch(row);
    }
    float sums[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (live && c < nvec) {
        unpack<T, VEC>(kAsync ? ring[read][0][i][threadIdx.x] : pg[i], g[i]);
        unpack<T, VEC>(kAsync ? ring[read][1][i][threadIdx.x] : ps[i], v[i]);
        if (kAhead && a.ds) d[kAhead ? i : 0] = pd[i];
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[i][e] = v[i][e] = 0.f;
      }
    }
    if (kAhead) fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (j + i * TPR < nvec) {
        float gw[VEC];
        if (!kKeepW) load_param<VEC>(a.weight, a.w_bf16, (long long)(j + i * TPR) * VEC, gw);
#pragma unroll
        for (int e = 0; e < VEC; ++e) gw[e] = kKeepW ? w[kKeepW ? i : 0][e] : gw[e];
        scale_by<VEC>(gw, g[i]);
        sums[0] += dot<VEC>(v[i], v[i]);
        sums[1] += dot<VEC>(gw, v[i]);
      }
    }
    row_reduce<TPR, false>(sums, s_red[buf]);
    const float r = rsqrtf(sums[0] * inv_d + a.eps);
    // r^3 mean(w dy s), a factor r at a time: r^3 alone leaves fp32's range from rows of 1e13 on, and with eps = 0 below
    // 1e-13
    const float k = sums[1] * inv_d * r * r * r;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = j + i * TPR;
        if (c < nvec) {
          float o[VEC] = {}, wv[VEC], gv[VEC];
          if (a.ds) {
            if constexpr (kAsync) unpack<T, VEC>(ring[read][2][i][threadIdx.x], o);
            else if constexpr (kAhead) unpack<T, VEC>(d[kAhead ? i : 0], o);
            else load_f32<T, VEC>(static_cast<const T*>(a.ds) + row * a.D + (long long)c * VEC, o);
          }
          if (!kKeepW) load_param<VEC>(a.weight, a.w_bf16, (long long)c * VEC, wv);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            wv[e] = kKeepW ? w[kKeepW ? i : 0][e] : wv[e];
            gv[e] = g[i][e];
          }
          scale_by<VEC>(gv, v[i]);
          add_scaled<VEC>(dw[i], gv, r);
          add_scaled<VEC>(o, v[i], -k);
          scale_by<VEC>(wv, g[i]);
          add_scaled<VEC>(o, wv, r);
          store_pack<T, VEC>(static_cast<T*>(a.dx) + row * a.D + (long long)c * VEC, o);
        }
      }
    }
    if (kAsync) read = read + 1 < kBwdRing ? read + 1 : 0;
  }
  if constexpr (RPC > 1) {  // the row slots of the CTA, added in order
    __shared__ __align__(16) float s_dw[RPC][TPR * VEC * NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) store_floats<VEC>(&s_dw[threadIdx.x / TPR][(j + i * TPR) * VEC], dw[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += NT) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < RPC; ++i) sum += s_dw[i][c];
      a.partial[(long long)blockIdx.x * a.D + c] = sum;
    }
  } else {
    float* p = a.partial + (long long)blockIdx.x * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = j + i * TPR;
      if (c < nvec) store_floats<VEC>(p + (long long)c * VEC, dw[i]);
    }
  }
}

// Host: the row shapes built, smallest first.  `vecs` vectors a row of `vec`
// elements.  Up to a warp a thread takes one vector.  Longer rows give each
// thread two, which halves the exchanges between warps (rows of 2048 in bf16,
// one vector against two: 31.6 and 27.5 us for 8192 e4m3 rows; four: no better);
// rows read element by element take one warp group and up to 16 elements a
// thread (60000 rows of 500: 61 us, with 512 threads and one element 147 us).
// There, elements past the row's end cost as much as others (8 M bf16 elements in
// rows of 301: 3 a thread 20.6 us, 4 22.6, 5 24.7, 6 26.8; in rows of 1001: 8 15.5,
// 10 16.5, 12 20.6, 16 26.7), so no step from 3 on is more than a third.
struct RowShape {
  int tpr, nv;
};
inline RowShape row_shape(int vecs, int vec) {
  for (int tpr = 8; tpr <= 32; tpr *= 2)
    if (vecs <= tpr) return {tpr, 1};
  if (vec == 1) {
    for (int nv : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16})
      if (vecs <= 128 * nv) return {128, nv};
    for (int nv : {8, 16})
      if (vecs <= 512 * nv) return {512, nv};
    return {512, 32};
  }
  for (int tpr = 64; tpr <= 128; tpr *= 2)
    if (vecs <= tpr) return {tpr, 1};
  for (int tpr = 128; tpr <= 512; tpr *= 2)
    if (vecs <= 2 * tpr) return {tpr, 2};
  for (int nv : {3, 4})
    if (vecs <= 512 * nv) return {512, nv};
  return {512, 8};
}
// Backward: two vectors a thread where a row takes several warps, which keeps
// enough loads in flight; element by element up to four a thread, then 512
// threads (16000 rows of 1001: 85 us, with 128 threads of eight 145 us).
inline RowShape row_shape_bwd(int vecs, int vec) {
  for (int tpr = 8; tpr <= 32; tpr *= 2)
    if (vecs <= tpr) return {tpr, 1};
  if (vec == 1) {
    for (int nv : {1, 2, 4})
      if (vecs <= 128 * nv) return {128, nv};
    for (int nv : {2, 4, 8, 16})
      if (vecs <= 512 * nv) return {512, nv};
    return {512, 32};
  }
  for (int tpr = 32; tpr <= 512; tpr *= 2)
    if (vecs <= 2 * tpr) return {tpr, 2};
  for (int nv : {3, 4})
    if (vecs <= 512 * nv) return {512, nv};
  return {512, 8};
}

#define KDA_NORM_SMALL(CASE) CASE(8, 1) CASE(16, 1) CASE(32, 1)
#define KDA_NORM_LONG(CASE) CASE(512, 3) CASE(512, 4)
#define KDA_NORM_FWD_WIDE(CASE) \
  KDA_NORM_SMALL(CASE) CASE(64, 1) CASE(128, 1) CASE(128, 2) CASE(256, 2) CASE(512, 2) KDA_NORM_LONG(CASE)
#define KDA_NORM_FWD_SCALAR(CASE)                                                                                  \
  KDA_NORM_SMALL(CASE) CASE(128, 1) CASE(128, 2) CASE(128, 3) CASE(128, 4) CASE(128, 5) CASE(128, 6) CASE(128, 8)    \
  CASE(128, 10) CASE(128, 12) CASE(128, 16) CASE(512, 8) CASE(512, 16) CASE(512, 32)
#define KDA_NORM_BWD_WIDE(CASE) \
  KDA_NORM_SMALL(CASE) CASE(32, 2) CASE(64, 2) CASE(128, 2) CASE(256, 2) CASE(512, 2) KDA_NORM_LONG(CASE)
#define KDA_NORM_BWD_SCALAR(CASE)                                                                                   \
  KDA_NORM_SMALL(CASE) CASE(128, 1) CASE(128, 2) CASE(128, 4) CASE(512, 2) CASE(512, 4) CASE(512, 8) CASE(512, 16)    \
  CASE(512, 32)

// Turns of the forward's small rows: the set-up of a thread is worth several
// rows, as long as every SM has 8 CTAs (e4m3 output, at most 8, 16 and 32 turns:
// 524288 rows of 128 bf16 51.2, 51.7 and 55.8 us, 300000 rows of 100 fp32 47.8, 46.1
// and 51.9; 4 or 16 CTAs: no difference).
inline int fwd_turns(long long rows, int rows_a_turn) {
  const long long t = rows / ((long long)rows_a_turn * 148 * 8);
  return (int)(t < 1 ? 1 : t > 16 ? 16 : t);
}

template <typename T, int VEC, int QUANT>
cudaError_t launch_fwd(FwdArgs a, cudaStream_t st) {
  const RowShape sh = row_shape(a.D / VEC, VEC);
  a.groups = QUANT >= kGroup ? a.D / a.group : 1;
#define KDA_CASE(TPR, NV)                                                                               \
  if (sh.tpr == TPR && sh.nv == NV) {                                                                    \
    constexpr int NT = threads_of(TPR), RPC = NT / TPR * rows_at_once(TPR, NV);                           \
    a.turns = TPR <= 32 && NV == 1 ? fwd_turns(a.rows, RPC) : 1;                                          \
    const long long per = (long long)RPC * a.turns;                                                       \
    kda_rms_norm_fwd_kernel<T, VEC, TPR, NV, QUANT><<<(unsigned)((a.rows + per - 1) / per), NT, 0, st>>>(a); \
    return cudaGetLastError();                                                                            \
  }
  if constexpr (VEC == 1) {
    KDA_NORM_FWD_SCALAR(KDA_CASE)
  } else {
    KDA_NORM_FWD_WIDE(KDA_CASE)
    if constexpr (VEC < 8) { KDA_CASE(512, 8) }
  }
#undef KDA_CASE
  return cudaErrorInvalidValue;
}
// The group modes of a vector width.
template <typename T, int VEC>
cudaError_t launch_fwd_groups(const FwdArgs& a, cudaStream_t st) {
  switch (a.group / VEC) {
    case 4: return launch_fwd<T, VEC, 4>(a, st);
    case 8: return launch_fwd<T, VEC, 8>(a, st);
    case 16: return launch_fwd<T, VEC, 16>(a, st);
    case 32: return launch_fwd<T, VEC, 32>(a, st);
  }
  return cudaErrorInvalidValue;
}

// Lines of partial sums of the backward: one per CTA, as many CTAs as run at
// once (512 threads an SM).
inline int bwd_grid(long long rows, int vecs, int vec) {
  const RowShape sh = row_shape_bwd(vecs, vec);
  const int nt = threads_of(sh.tpr), rpc = nt / sh.tpr;
  const long long want = (rows + rpc - 1) / rpc, most = 148LL * (512 / nt);
  return (int)(want < most ? want : most);
}

template <typename T, int VEC>
cudaError_t launch_bwd(const BwdArgs& a, float* dweight, cudaStream_t st) {
  const RowShape sh = row_shape_bwd(a.D / VEC, VEC);
  const int grid = bwd_grid(a.rows, a.D / VEC, VEC);
  cudaError_t e = cudaErrorInvalidValue;
#define KDA_CASE(TPR, NV)                                                                          \
  if (sh.tpr == TPR && sh.nv == NV) {                                                               \
    constexpr size_t bytes =                                                                         \
        bwd_async(VEC, NV) ? (size_t)kBwdRing * 3 * NV * threads_of(TPR) * VEC * sizeof(T) : 0;         \
    if (bytes > 48 * 1024) {                                                                          \
      static PerDeviceOnce once;                                                                      \
      e = run_once_per_device(once, [] {                                                              \
        return cudaFuncSetAttribute(kda_rms_norm_bwd_kernel<T, VEC, TPR, NV>,                         \
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);         \
      });                                                                                             \
      if (e != cudaSuccess) return e;                                                                 \
    }                                                                                                 \
    kda_rms_norm_bwd_kernel<T, VEC, TPR, NV><<<grid, threads_of(TPR), bytes, st>>>(a);                \
    e = cudaGetLastError();                                                                           \
  }
  if constexpr (VEC == 1) {
    KDA_NORM_BWD_SCALAR(KDA_CASE)
  } else {
    KDA_NORM_BWD_WIDE(KDA_CASE)
    if constexpr (VEC < 8) { KDA_CASE(512, 8) }
  }
#undef KDA_CASE
  if (e != cudaSuccess) return e;
  return launch_sum_lines(a.partial, dweight, nullptr, a.D, grid, a.D, st);
}

}  // namespace norm
}  // namespace kda

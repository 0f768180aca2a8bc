// kda_layer_common.cuh -- device helpers shared by the kernels around the
// recurrence (norm, short convolution, selective scan): vector loads and
// stores with conversion, which packed sequence a token belongs to, and the
// sum of partial lines that makes every gradient of a shared weight
// independent of scheduling.
#pragma once
#include "kda_common.cuh"

namespace kda {

// VEC elements of T in one access (VEC * sizeof(T) bytes, that aligned).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const float (&x)[VEC]) {
  Pack<T, VEC> o;
#pragma unroll
  for (int i = 0; i < VEC; ++i) o.v[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Pack<T, VEC>*>(p) = o;
}
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Pack<T, VEC>& p, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) x[i] = to_f32<T>(p.v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void load_f32(const T* p, float (&x)[VEC]) {
  unpack<T, VEC>(load_pack<T, VEC>(p), x);
}
// VEC floats, 16 bytes an access where VEC allows it.
template <int VEC>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[VEC]) {
  constexpr int STEP = VEC >= 4 ? 4 : VEC;
#pragma unroll
  for (int i = 0; i < VEC; i += STEP) {
    const Pack<float, STEP> v = load_pack<float, STEP>(p + i);
#pragma unroll
    for (int e = 0; e < STEP; ++e) x[i + e] = v.v[e];
  }
}
template <int VEC>
__device__ __forceinline__ void store_floats(float* p, const float (&x)[VEC]) {
  constexpr int STEP = VEC >= 4 ? 4 : VEC;
#pragma unroll
  for (int i = 0; i < VEC; i += STEP) {
    Pack<float, STEP> v;
#pragma unroll
    for (int e = 0; e < STEP; ++e) v.v[e] = x[i + e];
    *reinterpret_cast<Pack<float, STEP>*>(p + i) = v;
  }
}
// VEC elements from element i of a parameter (weight, bias) whose type is a
// run-time choice; i * (2 or 4) bytes must suit the vector.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, int is_bf16, long long i, float (&out)[VEC]) {
  if (is_bf16) load_f32<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(p) + i, out);
  else load_floats<VEC>(static_cast<const float*>(p) + i, out);
}

// The sequences of a call: packed (cu != nullptr, num of them over `total`
// tokens) or num rows of T tokens each.
struct Seqs {
  const int32_t* cu;
  int num;
  long long T, total;
};

// The sequence token t (0 <= t < total) belongs to: the last one that starts
// at or before t.  Always in [0, num), whatever the table holds.
__device__ __forceinline__ int seq_of_token(const Seqs& q, long long t) {
  if (!q.cu) return (int)(t / q.T);
  int lo = 0, hi = q.num - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)q.cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ long long seq_start(const Seqs& q, int n) { return q.cu ? (long long)q.cu[n] : n * q.T; }
__device__ __forceinline__ long long seq_end(const Seqs& q, int n) {
  return q.cu ? (long long)q.cu[n + 1] : (n + 1) * q.T;
}
// The sequence of token t where sequence n has just ended there: the next one
// with tokens.  In [0, num) whatever the table holds.
__device__ __forceinline__ int next_seq(const Seqs& q, int n, long long t) {
  int m = n + 1 < q.num ? n + 1 : q.num - 1;
  if (q.cu)
    while (m + 1 < q.num && (long long)q.cu[m + 1] <= t) ++m;
  return m;
}
// Whether a call can have sequences without tokens.
__device__ __forceinline__ bool may_have_empty(const Seqs& q) { return q.cu || q.T == 0; }
__device__ __forceinline__ bool seq_empty(const Seqs& q, int n) { return seq_end(q, n) <= seq_start(q, n); }

// Raises the device error word if the packed table is not 0 .. total,
// non-decreasing.  The threads of one CTA call it.  The kernels stay inside
// the buffers with any table: token indices come from the grid, sequence
// indices from seq_of_token.
__device__ __forceinline__ void check_seq_table(const Seqs& q) {
  if (!q.cu) return;
  bool bad = threadIdx.x == 0 && (q.cu[0] != 0 || (long long)q.cu[q.num] != q.total);
  for (int n = threadIdx.x; n < q.num; n += blockDim.x) bad |= q.cu[n + 1] < q.cu[n];
  if (bad) raise_device_error(kDevErrBadSeqlens);
}

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-x); 0 and 1 at the ends (the reciprocal of infinity is 0).
__device__ __forceinline__ float fast_sigmoid(float x) { return fast_rcp(1.f + ex2(-x * kLog2eF)); }

// max that keeps NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Asynchronous copies to shared memory of BYTES (4, 8 or 16, both sides that
// aligned), the last of them only `bytes` long (the rest is zeroed).
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes = BYTES) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// max(m, |a|, |b|) that keeps NaN.
__device__ __forceinline__ float max_abs_nan(float m, float a, float b) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(m), "f"(a), "f"(b));
  return y;
}
// max(m, |x_e|) that keeps NaN; m >= 0.
template <int N>
__device__ __forceinline__ float max_abs_nan(float m, const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e + 1 < N; e += 2) m = max_abs_nan(m, x[e], x[e + 1]);
  if (N % 2) m = max_nan(m, fabsf(x[N - 1]));
  return m;
}

// Two fp32 lanes in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 dup2(float a) { return make_float2(a, a); }
// x *= y, pairwise where the length allows
template <int N>
__device__ __forceinline__ void scale_by(float (&x)[N], const float (&y)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 v = mul2(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]));
      x[e] = v.x;
      x[e + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] *= y[e];
  }
}
template <int N>
__device__ __forceinline__ void scale_by(float (&x)[N], float y) {
  float d[N];
#pragma unroll
  for (int e = 0; e < N; ++e) d[e] = y;
  scale_by<N>(x, d);
}
// acc += x y
template <int N>
__device__ __forceinline__ void add_scaled(float (&acc)[N], const float (&x)[N], float y) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 v = fma2(make_float2(x[e], x[e + 1]), dup2(y), make_float2(acc[e], acc[e + 1]));
      acc[e] = v.x;
      acc[e + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = fmaf(x[e], y, acc[e]);
  }
}
// sum of x y, in two partial sums where the length allows
template <int N>
__device__ __forceinline__ float dot(const float (&x)[N], const float (&y)[N]) {
  if constexpr (N % 2 == 0) {
    float2 s = mul2(make_float2(x[0], x[1]), make_float2(y[0], y[1]));
#pragma unroll
    for (int e = 2; e < N; e += 2) s = fma2(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]), s);
    return s.x + s.y;
  } else {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(x[e], y[e], s);
    return s;
  }
}

// Column sums of `lines` rows of src, `cols` wide, each in row order within 32
// slices: columns below `split` go to dst0, the rest to dst1 (either may be
// null: not written).
constexpr int kSumSlices = 32;
__global__ void __launch_bounds__(32 * kSumSlices) kda_sum_lines_kernel(const float* __restrict__ src,
                                                                        float* __restrict__ dst0,
                                                                        float* __restrict__ dst1, long long split,
                                                                        int lines, long long cols) {
  __shared__ float s[kSumSlices][33];
  const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c0 = (long long)blockIdx.x * 32;
  float acc = 0.f;
  if (c0 + l < cols) {
#pragma unroll 4
    for (int i = w; i < lines; i += kSumSlices) acc += src[(long long)i * cols + c0 + l];
  }
  s[w][l] = acc;
  __syncthreads();
  // warp w sums column w over the slices
  acc = s[l][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  const long long c = c0 + w;
  if (l == 0 && c < cols) {
    if (c < split) {
      if (dst0) dst0[c] = acc;
    } else if (dst1) {
      dst1[c - split] = acc;
    }
  }
}
inline cudaError_t launch_sum_lines(const float* src, float* dst0, float* dst1, long long split, int lines,
                                    long long cols, cudaStream_t st) {
  if (cols <= 0) return cudaSuccess;
  kda_sum_lines_kernel<<<(unsigned)((cols + 31) / 32), 32 * kSumSlices, 0, st>>>(src, dst0, dst1, split, lines, cols);
  return cudaGetLastError();
}

}  // namespace kda

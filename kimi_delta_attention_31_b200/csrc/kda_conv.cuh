// kda_conv.cuh -- short causal depthwise convolution with SiLU (width W = 2..4)
// over a batch or packed sequences, its single-token form and its backward
// pass.
//
//   p_t = bias + sum_j w[:, j] x_{t-W+1+j};  y_t = p_t sigmoid(p_t)
//   Rows before a sequence's first token are its state [W-1, D] (oldest first);
//   the state out is the last W-1 rows of (state, x).
//   backward: dp = dy (sg + p sg (1 - sg)), sg = sigmoid(p);
//     d row_r = sum_j w_j dp_{r-j} (+ d state_out for the last W-1 rows),
//     dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t.
//
// A thread owns VEC channels and walks a run of L tokens with the window in
// registers, so every input is read once but for the W-1 rows before each run
// (which the run before reads too: L2).  HBM-bound: tokens arrive by asynchronous
// copies in groups of kGroup, a few groups ahead, in a ring in shared memory that
// each thread has to itself (no barrier; loads ahead in registers left too few
// threads on an SM: 316 us for 65536 tokens of 4096 channels, 52% of the copy
// rate; through the ring 186 to 197 us, 5.5 TB/s and more).  The backward reads x and dy once
// and writes dx: 117 us for 16384 tokens (4.6 TB/s; its arithmetic and the sum of
// the weights' lines show); the step, 256 sequences of 12288 channels, 11 us
// (4.6 TB/s).  Products and sums are fp32, two at a time; the output is rounded once.
#pragma once
#include <type_traits>

#include "kda_layer_common.cuh"

namespace kda {
namespace conv {

constexpr int kThreads = 128;
constexpr int kGroup = 4;  // tokens of a group

// One thread's tokens [t0, t1) of one input, `stride` elements apart, GROUPS - 1
// groups ahead.  Threads with one element a token load them in order instead.
template <typename T, int VEC, int GROUPS>
struct Feed {
  Pack<T, VEC> (*ring)[kThreads];
  const T* p;
  long long stride, t1, next;
  int slot;
  __device__ __forceinline__ Feed(Pack<T, VEC> (*r)[kThreads], const T* src, long long st, long long t0, long long end)
      : ring(r), p(src + t0 * st), stride(st), t1(end), next(t0), slot(0) {}
  __device__ __forceinline__ void stage() {  // the next group; its slots were read a group ago
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (next + i < t1) copy_async<sizeof(T) * VEC>(&ring[slot * kGroup + i][threadIdx.x], p + i * stride);
    copy_async_commit();
    p += kGroup * stride;
    next += kGroup;
    slot = slot + 1 < GROUPS ? slot + 1 : 0;
  }
};
template <typename T, int VEC, int GROUPS>
__device__ __forceinline__ void read_group(const Feed<T, VEC, GROUPS>& f, int slot, int i, float (&out)[VEC]) {
  unpack<T, VEC>(f.ring[slot * kGroup + i][threadIdx.x], out);
}
// silu of the sums p, and (backward) its slope: silu' = sg + p sg (1 - sg).
template <int VEC>
__device__ __forceinline__ void sigmoids(const float (&p)[VEC], float (&sg)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) sg[e] = fast_sigmoid(p[e]);
}
// acc += x y
template <int VEC>
__device__ __forceinline__ void add_product(float (&acc)[VEC], const float (&x)[VEC], const float (&y)[VEC]) {
  if constexpr (VEC % 2 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 v = fma2(make_float2(x[e], x[e + 1]), make_float2(y[e], y[e + 1]), make_float2(acc[e], acc[e + 1]));
      acc[e] = v.x;
      acc[e + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = fmaf(x[e], y[e], acc[e]);
  }
}
// p = b + sum_j w_j rows[j]
template <int VEC, int W>
__device__ __forceinline__ void window_sum(const float (&wt)[W][VEC], const float (&b)[VEC], const float (*rows)[VEC],
                                           float (&p)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) p[e] = b[e];
#pragma unroll
  for (int j = 0; j < W; ++j) add_product<VEC>(p, wt[j], rows[j]);
}

struct FwdArgs {
  const void* x;
  long long x_stride;
  const void* w;
  const void* bias;
  int w_bf16;
  const void* state;  // [N, W-1, D] T, or nullptr (zeros)
  void* y;
  void* state_out;    // [N, W-1, D] T, or nullptr
  Seqs q;
  int D, ncol;
  long long L;
};

// Weights [D, W] and bias of the thread's VEC channels.
template <int VEC, int W>
__device__ __forceinline__ void load_weights(const void* w, const void* bias, int bf16, int c0, float (&wt)[W][VEC],
                                             float (&b)[VEC]) {
  float flat[W * VEC];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    float part[VEC];
    load_param<VEC>(w, bf16, (long long)c0 * W + i * VEC, part);
#pragma unroll
    for (int e = 0; e < VEC; ++e) flat[i * VEC + e] = part[e];
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) wt[j][e] = flat[e * W + j];
  if (bias) {
    load_param<VEC>(bias, bf16, c0, b);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = 0.f;
  }
}

// Row `r` of sequence n's state (zeros without one).
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_state_row(const void* state, int n, int r, int D, int c0, float (&out)[VEC]) {
  if (state) {
    load_f32<T, VEC>(static_cast<const T*>(state) + ((long long)n * (W - 1) + r) * D + c0, out);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e] = 0.f;
  }
}

// The W-1 rows before token t of sequence n (which starts at s0 <= t): x, and
// the state before the first token.
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_window(const void* x, long long x_stride, const void* state, int n,
                                            long long s0, long long t, int D, int c0, float (*rows)[VEC]) {
  const long long pos = t > s0 ? t - s0 : 0;  // s0 > t only with a malformed table
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int back = W - 1 - i;
    if (pos >= back && t >= back) load_f32<T, VEC>(static_cast<const T*>(x) + (t - back) * x_stride + c0, rows[i]);
    else load_state_row<T, VEC, W>(state, n, pos >= back ? 0 : (int)pos + i, D, c0, rows[i]);
  }
}

constexpr int kFwdGroups = 4;  // groups in the forward's ring

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads, 4) kda_short_conv_fwd_kernel(const FwdArgs a) {
  constexpr int U = kGroup;
  __shared__ Pack<T, VEC> s_ring[VEC > 1 ? kFwdGroups * U : 1][kThreads];
  const int col = (int)(blockIdx.x % a.ncol);
  const long long run = blockIdx.x / a.ncol;
  const int c0 = (col * kThreads + (int)threadIdx.x) * VEC;
  if (blockIdx.x == 0) check_seq_table(a.q);
  if (c0 >= a.D) return;
  T* state_out = static_cast<T*>(a.state_out);
  if (state_out && may_have_empty(a.q)) {  // sequences without tokens keep their state: every run looks at some
    for (long long n = run; n < a.q.num; n += gridDim.x / a.ncol)
      if (seq_empty(a.q, (int)n)) {
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
          float v[VEC];
          load_state_row<T, VEC, W>(a.state, (int)n, r, a.D, c0, v);
          store_pack<T, VEC>(state_out + (n * (W - 1) + r) * a.D + c0, v);
        }
      }
  }
  const long long t0 = run * a.L;
  const long long t1 = t0 + a.L < a.q.total ? t0 + a.L : a.q.total;
  if (t0 >= t1) return;

  const T* xp = static_cast<const T*>(a.x) + c0;
  Feed<T, VEC, kFwdGroups> feed(s_ring, xp, a.x_stride, t0, t1);
  if constexpr (VEC > 1) {
#pragma unroll
    for (int g = 0; g < kFwdGroups - 1; ++g) feed.stage();
  }
  float wt[W][VEC], b[VEC];
  load_weights<VEC, W>(a.w, a.bias, a.w_bf16, c0, wt, b);
  int n = seq_of_token(a.q, t0);
  long long end = seq_end(a.q, n);
  float xs[U + W - 1][VEC];
  load_window<T, VEC, W>(a.x, a.x_stride, a.state, n, seq_start(a.q, n), t0, a.D, c0, xs);
  T* yp = static_cast<T*>(a.y) + t0 * a.D + c0;
  Pack<T, VEC> next[VEC > 1 ? 1 : U];
  if constexpr (VEC == 1) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (t0 + i < t1) next[VEC > 1 ? 0 : i] = load_pack<T, VEC>(xp + (t0 + i) * a.x_stride);
  }
  int slot = 0;
  for (long long t = t0; t < t1; t += U) {
    if constexpr (VEC > 1) {
      feed.stage();
      copy_async_wait<kFwdGroups - 1>();
#pragma unroll
      for (int i = 0; i < U; ++i) read_group(feed, slot, i, xs[W - 1 + i]);
      slot = slot + 1 < kFwdGroups ? slot + 1 : 0;
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) unpack<T, VEC>(next[VEC > 1 ? 0 : i], xs[W - 1 + i]);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (t + U + i < t1) next[VEC > 1 ? 0 : i] = load_pack<T, VEC>(xp + (t + U + i) * a.x_stride);
    }
    auto tokens = [&](auto plain) {  // plain: U tokens inside one sequence, which ends later
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long ti = t + i;
        if (decltype(plain)::value || ti < t1) {
          if (!decltype(plain)::value && ti == end) {  // the first token of another sequence
            n = next_seq(a.q, n, ti);
            end = seq_end(a.q, n);
#pragma unroll
            for (int r = 0; r < W - 1; ++r) load_state_row<T, VEC, W>(a.state, n, r, a.D, c0, xs[i + r]);
          }
          float p[VEC], sg[VEC];
          window_sum<VEC, W>(wt, b, xs + i, p);
          sigmoids<VEC>(p, sg);
#pragma unroll
          for (int e = 0; e < VEC; ++e) p[e] *= sg[e];
          store_pack<T, VEC>(yp + (long long)i * a.D, p);
          if (!decltype(plain)::value && ti + 1 == end && state_out) {
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
              store_pack<T, VEC>(state_out + ((long long)n * (W - 1) + r) * a.D + c0, xs[i + 1 + r]);
          }
        }
      }
    };
    if (t + U <= t1 && (end > t + U || end < t)) tokens(std::true_type{});
    else tokens(std::false_type{});
    yp += (long long)U * a.D;
#pragma unroll
    for (int r = 0; r < W - 1; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) xs[r][e] = xs[U + r][e];
  }
}

// One token of each of N sequences; state_out may be state (each thread reads
// all its rows first).  (Two sequences a thread, to load the weights once: 14.3 us
// against 12.3 for 256 sequences of 12288 channels.)
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kThreads) kda_short_conv_step_kernel(const FwdArgs a) {
  const int col = (int)(blockIdx.x % a.ncol);
  const long long n = blockIdx.x / a.ncol;
  const int c0 = (col * kThreads + (int)threadIdx.x) * VEC;
  if (c0 >= a.D) return;
  const T* st = static_cast<const T*>(a.state) + n * (W - 1) * a.D + c0;
  T* so = static_cast<T*>(a.state_out) + n * (W - 1) * a.D + c0;
  Pack<T, VEC> rows[W];
#pragma unroll
  for (int r = 0; r < W - 1; ++r) rows[r] = load_pack<T, VEC>(st + (long long)r * a.D);
  rows[W - 1] = load_pack<T, VEC>(static_cast<const T*>(a.x) + n * a.x_stride + c0);
  float wt[W][VEC], b[VEC];
  load_weights<VEC, W>(a.w, a.bias, a.w_bf16, c0, wt, b);
#pragma unroll
  for (int r = 0; r < W - 1; ++r) *reinterpret_cast<Pack<T, VEC>*>(so + (long long)r * a.D) = rows[r + 1];
  float xs[W][VEC], p[VEC], sg[VEC];
#pragma unroll
  for (int j = 0; j < W; ++j) unpack<T, VEC>(rows[j], xs[j]);
  window_sum<VEC, W>(wt, b, xs, p);
  sigmoids<VEC>(p, sg);
  scale_by<VEC>(p, sg);
  store_pack<T, VEC>(static_cast<T*>(a.y) + n * a.D + c0, p);
}

// ---------------------------------------------------------------------------
// Backward.  A run owns tokens [t0, t1): it sums their dw, dbias into one line
// of partial sums and, as it passes token t, finishes the gradient of the row
// W-1 before it (and of the last W-1 rows when t ends its sequence).  The dp
// of the W-1 tokens before the run is computed again.
// ---------------------------------------------------------------------------
struct BwdArgs {
  const void* x;
  long long x_stride;
  const void* w;
  const void* bias;
  int w_bf16;
  const void* state;
  const void* dy;        // [tokens, D] TDY
  const float* dstate;   // [N, W-1, D], or nullptr
  void* dx;              // [tokens, D] T
  float* dinit;          // [N, W-1, D], or nullptr
  float* partial;        // [runs, D W + D]
  Seqs q;
  int D, ncol;
  long long L;
};

constexpr int kBwdGroups = 3;  // groups in the backward's rings

template <typename T, typename TDY, int VEC, int W>
__global__ void __launch_bounds__(kThreads, 4) kda_short_conv_bwd_kernel(const BwdArgs a) {
  constexpr int U = kGroup;
  __shared__ Pack<T, VEC> s_x[VEC > 1 ? kBwdGroups * U : 1][kThreads];
  __shared__ Pack<TDY, VEC> s_dy[VEC > 1 ? kBwdGroups * U : 1][kThreads];
  const int col = (int)(blockIdx.x % a.ncol);
  const long long run = blockIdx.x / a.ncol;
  const int c0 = (col * kThreads + (int)threadIdx.x) * VEC;
  if (blockIdx.x == 0) check_seq_table(a.q);
  if (c0 >= a.D) return;
  if (a.dinit && may_have_empty(a.q)) {  // sequences without tokens: the state out is the state
    for (long long n = run; n < a.q.num; n += gridDim.x / a.ncol)
      if (seq_empty(a.q, (int)n)) {
#pragma unroll
        for (int r = 0; r < W - 1; ++r) {
          const long long at = ((long long)n * (W - 1) + r) * a.D + c0;
          float v[VEC] = {};
          if (a.dstate) load_floats<VEC>(a.dstate + at, v);
          store_floats<VEC>(a.dinit + at, v);
        }
      }
  }
  const long long t0 = run * a.L;
  const long long t1 = t0 + a.L < a.q.total ? t0 + a.L : a.q.total;
  float dw[W][VEC] = {}, db[VEC] = {};
  if (t0 < t1) {
    float wt[W][VEC], b[VEC];
    load_weights<VEC, W>(a.w, a.bias, a.w_bf16, c0, wt, b);
    const T* xp = static_cast<const T*>(a.x) + c0;
    const TDY* dyp = static_cast<const TDY*>(a.dy) + c0;
    T* dxp = static_cast<T*>(a.dx) + c0;
    int n = seq_of_token(a.q, t0);
    long long start = seq_start(a.q, n), end = seq_end(a.q, n);
    long long tb = t0 - (W - 1) > start ? t0 - (W - 1) : start;  // where dp begins
    if (tb < 0 || tb > t0) tb = tb < 0 ? 0 : t0;                 // only with a malformed table
    float xs[U + W - 1][VEC];    // rows tb-W+1 ..
    float dps[U + W - 1][VEC];   // dp of the same tokens
    load_window<T, VEC, W>(a.x, a.x_stride, a.state, n, start, tb, a.D, c0, xs);
#pragma unroll
    for (int r = 0; r < W - 1; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dps[r][e] = 0.f;

    Feed<T, VEC, kBwdGroups> fx(s_x, xp, a.x_stride, tb, t1);
    Feed<TDY, VEC, kBwdGroups> fy(s_dy, dyp, a.D, tb, t1);
    if constexpr (VEC > 1) {
#pragma unroll
      for (int g = 0; g < kBwdGroups - 1; ++g) fx.stage(), fy.stage();
    }
    int slot = 0;
    Pack<T, VEC> nx[VEC > 1 ? 1 : U];
    Pack<TDY, VEC> ny[VEC > 1 ? 1 : U];
    if constexpr (VEC == 1) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (tb + i < t1) {
          nx[VEC > 1 ? 0 : i] = load_pack<T, VEC>(xp + (tb + i) * a.x_stride);
          ny[VEC > 1 ? 0 : i] = load_pack<TDY, VEC>(dyp + (tb + i) * a.D);
        }
    }
    for (long long t = tb; t < t1; t += U) {
      if constexpr (VEC > 1) {
        fx.stage();
        fy.stage();
        copy_async_wait<2 * (kBwdGroups - 1)>();  // x and dy are committed in turn
#pragma unroll
        for (int i = 0; i < U; ++i) {
          read_group(fx, slot, i, xs[W - 1 + i]);
          read_group(fy, slot, i, dps[W - 1 + i]);
        }
        slot = slot + 1 < kBwdGroups ? slot + 1 : 0;
      } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          unpack<T, VEC>(nx[VEC > 1 ? 0 : i], xs[W - 1 + i]);
          unpack<TDY, VEC>(ny[VEC > 1 ? 0 : i], dps[W - 1 + i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (t + U + i < t1) {
            nx[VEC > 1 ? 0 : i] = load_pack<T, VEC>(xp + (t + U + i) * a.x_stride);
            ny[VEC > 1 ? 0 : i] = load_pack<TDY, VEC>(dyp + (t + U + i) * a.D);
          }
      }
      auto tokens = [&](auto plain) {  // plain: U own tokens inside one sequence, past its first W-1, which ends later
        constexpr bool kPlain = decltype(plain)::value;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const long long ti = t + i;
          if (kPlain || ti < t1) {
            if (!kPlain && ti == end) {
              n = next_seq(a.q, n, ti);
              start = seq_start(a.q, n);
              end = seq_end(a.q, n);
#pragma unroll
              for (int r = 0; r < W - 1; ++r) {
                load_state_row<T, VEC, W>(a.state, n, r, a.D, c0, xs[i + r]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) dps[i + r][e] = 0.f;
              }
            }
            const bool own = kPlain || ti >= t0;
            float p[VEC], sg[VEC], drow[VEC] = {};
            window_sum<VEC, W>(wt, b, xs + i, p);
            sigmoids<VEC>(p, sg);
#pragma unroll
            for (int e = 0; e < VEC; ++e) dps[i + W - 1][e] *= fmaf(p[e] * sg[e], 1.f - sg[e], sg[e]);
            if (own) {
#pragma unroll
              for (int j = 0; j < W; ++j) add_product<VEC>(dw[j], dps[i + W - 1], xs[i + j]);
#pragma unroll
              for (int e = 0; e < VEC; ++e) db[e] += dps[i + W - 1][e];
#pragma unroll
              for (int j = 0; j < W; ++j) add_product<VEC>(drow, wt[j], dps[i + W - 1 - j]);
              const long long r = ti - start;  // the row finished here, counted from the state's first
              if (kPlain || r >= W - 1) {
                if (kPlain || ti >= W - 1) store_pack<T, VEC>(dxp + (ti - (W - 1)) * a.D, drow);
              } else if (a.dinit && r >= 0) {
                store_floats<VEC>(a.dinit + ((long long)n * (W - 1) + r) * a.D + c0, drow);
              }
              if (!kPlain && ti + 1 == end) {  // the rows that only the tokens up to here, and the state out, see
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                  float tail[VEC] = {};
                  if (a.dstate) load_floats<VEC>(a.dstate + ((long long)n * (W - 1) + k) * a.D + c0, tail);
#pragma unroll
                  for (int j = k + 1; j < W; ++j) add_product<VEC>(tail, wt[j], dps[i + W + k - j]);
                  const long long rk = r + 1 + k;
                  if (rk >= W - 1) {
                    if (ti + 1 + k >= W - 1) store_pack<T, VEC>(dxp + (ti + 1 + k - (W - 1)) * a.D, tail);
                  } else if (a.dinit && rk >= 0) {
                    store_floats<VEC>(a.dinit + ((long long)n * (W - 1) + rk) * a.D + c0, tail);
                  }
                }
              }
            }
          }
        }
      };
      if (t >= t0 && t + U <= t1 && t >= W - 1 && t - start >= W - 1 && end > t + U) tokens(std::true_type{});
      else tokens(std::false_type{});
#pragma unroll
      for (int r = 0; r < W - 1; ++r)
#pragma unroll
        for (int e = 0; e < VEC; ++e) xs[r][e] = xs[U + r][e], dps[r][e] = dps[U + r][e];
    }
  }
  const long long cols = (long long)a.D * (W + 1);
  float* line = a.partial + run * cols;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) line[(long long)(c0 + e) * W + j] = dw[j][e];
  }
  store_floats<VEC>(line + (long long)a.D * W + c0, db);
}

// Host: column blocks and the run length.
inline int columns(int D, int vec) { return (D + kThreads * vec - 1) / (kThreads * vec); }
// Forward runs: about eight CTAs an SM, between 16 tokens (3 of 19 rows are
// then read twice) and 64.
inline long long fwd_run(long long tokens, int ncol) {
  long long L = (tokens * ncol + 148 * 8 - 1) / (148 * 8);
  L = L < 16 ? 16 : L > 64 ? 64 : L;
  return (L + kGroup - 1) / kGroup * kGroup;
}
// Backward runs: every run writes a line of partial sums, so no more of them
// than run at once (four CTAs an SM; six: 123.6 us against 117.0 for 16384
// tokens of 4096 channels), none under 16 tokens.  The runs of a column block
// are counted first, rounded down: a few CTAs in a second wave would each walk
// a whole run on a card that is otherwise done (12288 channels, 24 runs of a
// column block against 25: 65536 tokens 1200 and 1404 us, 16384 tokens 315 and
// 318; 16384 channels, 18 against 19: 16384 tokens 431 and 420).
constexpr long long kBwdWave = 148 * 4;
inline long long bwd_run(long long tokens, int ncol) {
  const long long runs = ncol < kBwdWave ? kBwdWave / ncol : 1;
  long long L = (tokens + runs - 1) / runs;
  L = L < 16 ? 16 : L;
  return (L + kGroup - 1) / kGroup * kGroup;
}
inline long long runs_of(long long tokens, long long L) {
  const long long r = (tokens + L - 1) / L;
  return r > 0 ? r : 1;
}

template <typename T, int VEC, int W>
cudaError_t launch_fwd(FwdArgs a, cudaStream_t st) {
  a.ncol = columns(a.D, VEC);
  a.L = fwd_run(a.q.total, a.ncol);
  const long long grid = runs_of(a.q.total, a.L) * a.ncol;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kda_short_conv_fwd_kernel<T, VEC, W><<<(unsigned)grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}
template <typename T, int VEC, int W>
cudaError_t launch_step(FwdArgs a, cudaStream_t st) {
  a.ncol = columns(a.D, VEC);
  const long long grid = (long long)a.q.num * a.ncol;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kda_short_conv_step_kernel<T, VEC, W><<<(unsigned)grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}
// Lines of partial sums for these sizes (any alignment: the larger of both vector widths).
inline long long bwd_lines(long long tokens, int D) {
  const long long a = runs_of(tokens, bwd_run(tokens, columns(D, 4)));
  const long long b = runs_of(tokens, bwd_run(tokens, columns(D, 1)));
  return a > b ? a : b;
}
template <typename T, typename TDY, int VEC, int W>
cudaError_t launch_bwd(BwdArgs a, float* dweight, float* dbias, cudaStream_t st) {
  a.ncol = columns(a.D, VEC);
  a.L = bwd_run(a.q.total, a.ncol);
  const long long runs = runs_of(a.q.total, a.L), grid = runs * a.ncol;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kda_short_conv_bwd_kernel<T, TDY, VEC, W><<<(unsigned)grid, kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_sum_lines(a.partial, dweight, dbias, (long long)a.D * W, (int)runs, (long long)a.D * (W + 1), st);
}

}  // namespace conv
}  // namespace kda

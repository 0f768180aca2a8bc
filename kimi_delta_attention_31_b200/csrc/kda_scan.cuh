// kda_scan.cuh -- selective state space scan: the diagonal sibling of the
// recurrence, one state row of S numbers per channel.
//
//   delta_t = softplus(dt_t + dt_bias);  h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t
//   y_t = (C_t . h_t + D x_t) silu(z_t)
//
// Forward: a lane owns SPT states of one channel (S / SPT lanes a channel) and
// walks the tokens with them in registers; B and C of kTile tokens sit in shared
// memory in fp32, shared by the channels of the CTA.  What a (token, channel)
// needs once (time step, gate, skip, output) is done by one of the channel's
// lanes, each for its share of kStep tokens, a step ahead.  One exponential per
// (token, channel, state) is the arithmetic it cannot do without (16 a clock and
// SM), not HBM: 8 bytes per token and channel.  8 x 4096 tokens of 4096 channels,
// 16 states: 912 us, 2.4e12 exponentials a second (half the rate); the rest goes
// to shared-memory reads (18 words a lane and token: B, C, time step, input),
// to issue, and to 512 CTAs on 148 SMs.  Measured and not kept: four states a lane
// (1236 us), sixteen (1208), two channels a lane with four states of each (1011),
// a quarter of the exponentials by polynomial on the FMA pipe (1152, against 1008
// then).
//
// When a call has too few channels to fill the card (packed sequences, whose
// lengths are on the device only, count as one row), the token axis is cut into
// chunks wherever they fall: the kernel's kLocal form runs every chunk from a zero state,
// kda_scan_carry_kernel chains the chunks (h is linear in the state that enters:
// a whole chunk multiplies it by exp(A sum delta)), and the scan then runs each
// chunk from its entry state.  A chunk in which a sequence starts passes
// nothing on from before it.  65536 tokens of 1024 channels: 725 us (326 + 7 + 414
// under the profiler), against one thread column of 1024 chains on its own.
#pragma once
#include <initializer_list>

#include "kda_layer_common.cuh"

namespace kda {
namespace scan {

constexpr int kThreads = 128;
constexpr int kTile = 16;   // tokens staged at a time
constexpr int kStep = 8;    // tokens unrolled together
constexpr int kStages = 3;  // tiles of inputs in shared memory: one in use, two on their way

struct Args {
  const void *x, *dt, *z, *B, *C;
  long long xs, dts, zs, bs, cs;  // elements from one token to the next
  const float *A, *Dv, *dt_bias;  // [d, S], [d] or nullptr, [d] or nullptr
  const float* S0;                // [N, d, S] or nullptr (zeros)
  void* y;                        // [tokens, d]
  float* S_out;                   // [N, d, S] or nullptr
  Seqs q;
  int d, cpg, blocks_per_group, ncb;  // channels, channels a group, CTAs' channel blocks
  long long L;                        // tokens a chunk
  long long chunks;
  float* entry;  // [chunks, d, S]: local end states, then the states that enter
  float* sumd;   // [chunks, d]: sum of delta, or -1 where a sequence starts in the chunk
  // backward only
  const void* dy;    // [tokens, d]
  const float* dS;   // [N, d, S] or nullptr
  float* exitg;      // [chunks, d, S]: as entry, for the gradient that comes from the right
  int copy, copy_bc;  // bytes of one asynchronous copy of x, dt, z, dy and of B, C: 16, 8, 4, or 0 for 16-bit
                      // elements at odd places, which are loaded and stored one by one
};

template <int S>
struct Shape {
  static constexpr int SPT = S <= 16 ? 8 : 16;  // states a lane
  static constexpr int LPC = S / SPT;           // lanes a channel
  static constexpr int CH = kThreads / LPC;     // channels a CTA
  static constexpr int OWN = kStep / LPC;       // tokens of a step a lane prepares and finishes
};

// Sum over the NL lanes whose numbers differ in the bits STRIDE, 2 STRIDE, ..
// of NV values each.  The lane keeps max(1, NV / NL) of the sums in
// v[0 .. ); *index counts the first one.
template <int NV, int NL, int STRIDE>
__device__ __forceinline__ void reduce_scatter(float (&v)[NV], int lane, int* index) {
  int at = 0;
  int have = NV;
#pragma unroll
  for (int o = NL / 2; o > 0; o >>= 1) {
    const bool up = (lane & (o * STRIDE)) != 0;
    if (have > 1) {
      have >>= 1;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i)
        if (i < have) {
          const float send = up ? v[i] : v[i + have];
          const float keep = up ? v[i + have] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o * STRIDE);
        }
      at += up ? have : 0;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * STRIDE);
    }
  }
  *index = at;
}

// log(1 + e^v) of two values, to fp32 accuracy also where it is small:
// max(v, 0) + log1p(e), e = e^-|v| in (0, 1], with log1p(e) / e by its minimax
// polynomial of degree 9 on [0, 1] (fitted by Lawson's iteration).  With the
// coefficients as they stand in fp32 log1p(e) is within 2.7e-8, evaluated in fp32
// within 1.5e-7 (2.4 units of 2^-24).
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 e = make_float2(ex2(-fabsf(v.x) * kLog2eF), ex2(-fabsf(v.y) * kLog2eF));
  float2 q = dup2(-0.0032440247014164925f);
  q = fma2(q, e, dup2(0.019851461052894592f));
  q = fma2(q, e, dup2(-0.05695953220129013f));
  q = fma2(q, e, dup2(0.10603654384613037f));
  q = fma2(q, e, dup2(-0.15305592119693756f));
  q = fma2(q, e, dup2(0.1967593878507614f));
  q = fma2(q, e, dup2(-0.24954134225845337f));
  q = fma2(q, e, dup2(0.3332996368408203f));
  q = fma2(q, e, dup2(-0.4999990165233612f));
  q = fma2(q, e, dup2(1.f));
  // max that keeps NaN: a NaN time step makes its channel NaN
  return fma2(q, e, make_float2(max_nan(v.x, 0.f), max_nan(v.y, 0.f)));
}
__device__ __forceinline__ float softplus_f(float v) { return softplus2(dup2(v)).x; }

// exp(delta A) from A2 = A log2(e).  The hardware's ex2 lies low, by 0.3 to 0.8
// units of 2^-24 on average over exponents of -4 to -0.0005, and a state of
// hundreds of tokens' memory multiplies that many decays: an offset of 0.4 units
// in the exponent, which costs nothing (the product becomes a fused
// multiply-add), brings the average within 0.1 units between -0.5 and -0.003.
// An exponent of 0 still gives exactly 1.
constexpr float kEx2Bias = 0.4f / 16777216.f;
__device__ __forceinline__ float2 decay2(float2 delta, float2 A2) {
  const float2 e = fma2(delta, A2, make_float2(kEx2Bias, kEx2Bias));
  return make_float2(ex2(e.x), ex2(e.y));
}

// A lane's states: 2 N of them, four adjacent ones at a time, the next four
// STRIDE further (the lanes of a channel take turns, so that what they read
// together is adjacent).
template <int N, int STRIDE>
__device__ __forceinline__ void load_state(const float* p, float2 (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 v = *reinterpret_cast<const float4*>(p + i / 2 * STRIDE);
    h[i] = make_float2(v.x, v.y);
    h[i + 1] = make_float2(v.z, v.w);
  }
}
template <int N, int STRIDE>
__device__ __forceinline__ void store_state(float* p, const float2 (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<float4*>(p + i / 2 * STRIDE) = make_float4(h[i].x, h[i].y, h[i + 1].x, h[i + 1].y);
}
template <int N>
__device__ __forceinline__ void zero_state(float2 (&h)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) h[i] = make_float2(0.f, 0.f);
}

enum Mode : int { kForward = 0, kLocal = 1, kLocalBwd = 2 };

// The CTA's inputs of one tile, as they are in memory; B, C in fp32; what the
// lanes of a channel share.
template <typename T, int S, int MODE>
struct alignas(16) TileSmem {
  static constexpr int CH = Shape<S>::CH;
  static constexpr int NIN = MODE == 0 ? 3 : MODE == 1 ? 2 : 4;  // x, dt (, z (, dy))
  T in[kStages][NIN][kTile][CH];
  T raw[kStages][MODE == 1 ? 1 : 2][kTile][S];  // B, C as they are in memory
  static constexpr bool kConvert = sizeof(T) != 4;  // fp32 ones are read where they are
  float B[2][kConvert ? kTile : 1][kConvert ? S : 4];
  float C[2][kConvert && MODE != 1 ? kTile : 1][kConvert && MODE != 1 ? S : 4];
  float2 du[kStep][CH];                         // delta, delta x (each once: what lanes read bounds the kernel too)
  float gv[MODE == 2 ? kStep : 1][CH];          // dy silu(z)
};

// `rows` rows of `len` elements (len <= WIDTH), `stride` apart, to dst[.][WIDTH],
// ROWS of them at most, by THREADS threads: `bytes` a copy.  The narrow copies
// stay out of line: they would push the scan's own loop out of the instruction
// cache (4% on 16-byte inputs).
template <typename T, int WIDTH, int THREADS>
__device__ __noinline__ void stage_rows_narrow(T (*dst)[WIDTH], const T* src, long long stride, int rows, int len,
                                               int bytes) {
  if (bytes == 0) {  // element by element, eight loads at a time
    constexpr int U = 8;
    for (int e0 = threadIdx.x; e0 < rows * WIDTH; e0 += U * THREADS) {
      T v[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * THREADS, r = e / WIDTH, k = e % WIDTH;
        if (r < rows && k < len) v[i] = src[r * stride + k];
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = e0 + i * THREADS, r = e / WIDTH, k = e % WIDTH;
        if (r < rows && k < len) dst[r][k] = v[i];
      }
    }
    return;
  }
  const int shift = bytes == 8 ? (sizeof(T) == 2 ? 2 : 1) : sizeof(T) == 2 ? 1 : 0;  // elements: 1 << shift
  const int n = WIDTH >> shift;  // copies a row
#pragma unroll 4
  for (int e = threadIdx.x; e < rows * n; e += THREADS) {
    const int r = e / n, k = (e - r * n) << shift;
    if (k >= len) continue;
    const T* p = src + r * stride + k;
    const int have = (len - k) * (int)sizeof(T);
    if (bytes == 8) copy_async<8>(&dst[r][k], p, min(8, have));
    else copy_async<4>(&dst[r][k], p, min(4, have));
  }
}
template <typename T, int WIDTH, int ROWS, int THREADS>
__device__ __forceinline__ void stage_rows(T (*dst)[WIDTH], const T* src, long long stride, int rows, int len,
                                           int bytes) {
  if (bytes == 16) {
    constexpr int PER = 16 / sizeof(T), N = WIDTH / PER;  // copies a row
#pragma unroll
    for (int i = 0; i < (ROWS * N + THREADS - 1) / THREADS; ++i) {
      const int e = i * THREADS + (int)threadIdx.x, r = e / N, k = (e % N) * PER;
      if (r < rows && k < len) copy_async<16>(&dst[r][k], src + r * stride + k, min(16, (len - k) * (int)sizeof(T)));
    }
  } else {
    stage_rows_narrow<T, WIDTH, THREADS>(dst, src, stride, rows, len, bytes);
  }
}

// MODE kForward: the scan of each chunk from its entry state (S0 where a
//   sequence starts).  kLocal: the end state of each chunk from zero and the sum
//   of its deltas.  kLocalBwd: also the gradient that a chunk sends to the state
//   before it, with nothing coming from its right:
//     sum_t (prod_{s <= t} a_s) C_t dyy_t,  dyy = dy silu(z), up to the first
//   sequence start in the chunk.  The sum is written where that start is met: a
//   NaN or infinity behind it belongs to another sequence, and times a product
//   of decays set to zero it would still be one.
//
// Inputs arrive by asynchronous copies, two tiles ahead.  kStep tokens inside
// one sequence run without a branch, so that the exponentials of later tokens
// cover the chains of earlier ones; a step in which a sequence ends, or a last
// one that is not full, goes token by token.
template <typename T, int S, int MODE>
__global__ void __launch_bounds__(kThreads, 4) kda_selective_scan_kernel(const Args a) {
  using Sh = Shape<S>;
  constexpr int SPT = Sh::SPT, LPC = Sh::LPC, NP = SPT / 2, CH = Sh::CH, OWN = Sh::OWN;
  constexpr bool kC = MODE != kLocal, kZ = MODE != kLocal;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TileSmem<T, S, MODE>& sm = *reinterpret_cast<TileSmem<T, S, MODE>*>(smem_raw);

  const int cb = (int)(blockIdx.x % a.ncb);
  const long long chunk = blockIdx.x / a.ncb;
  const int grp = cb / a.blocks_per_group;
  const int cl0 = (cb % a.blocks_per_group) * CH;
  const int lane = threadIdx.x & 31;
  const int ch = (int)threadIdx.x / LPC;
  const int sl = (int)threadIdx.x % LPC;
  const int width = a.cpg - cl0 < CH ? a.cpg - cl0 : CH;  // channels of the CTA
  const bool active = ch < width;  // the others compute on whatever shared memory holds and write nothing
  const long long c0 = (long long)grp * a.cpg + cl0, c = c0 + (active ? ch : width - 1);
  const long long crow = c * S + sl * 4;

  if (blockIdx.x == 0) check_seq_table(a.q);
  if (MODE == kForward && a.S_out && may_have_empty(a.q)) {  // sequences without tokens keep their state
    for (long long n = chunk; n < a.q.num; n += a.chunks)
      if (seq_empty(a.q, (int)n) && active) {
        float2 v[NP];
        if (a.S0) load_state<NP, LPC * 4>(a.S0 + n * a.d * S + crow, v);
        else zero_state<NP>(v);
        store_state<NP, LPC * 4>(a.S_out + n * a.d * S + crow, v);
      }
  }
  const long long t0 = chunk * a.L;
  const long long t1 = t0 + a.L < a.q.total ? t0 + a.L : a.q.total;
  if (t0 >= t1) return;
  const bool gated = kZ && a.z;

  auto stage = [&](long long t, int st) {
    if (t < t1) {
      const int rows = t1 - t < kTile ? (int)(t1 - t) : kTile;
      stage_rows<T, CH, kTile, kThreads>(sm.in[st][0], static_cast<const T*>(a.x) + t * a.xs + c0, a.xs, rows, width, a.copy);
      stage_rows<T, CH, kTile, kThreads>(sm.in[st][1], static_cast<const T*>(a.dt) + t * a.dts + c0, a.dts, rows, width, a.copy);
      if constexpr (kZ)
        if (gated)
          stage_rows<T, CH, kTile, kThreads>(sm.in[st][kZ ? 2 : 0], static_cast<const T*>(a.z) + t * a.zs + c0, a.zs, rows, width,
                            a.copy);
      if constexpr (MODE == kLocalBwd)
        stage_rows<T, CH, kTile, kThreads>(sm.in[st][MODE == kLocalBwd ? 3 : 0], static_cast<const T*>(a.dy) + t * a.d + c0, a.d, rows,
                          width, a.copy);
      stage_rows<T, S, kTile, kThreads>(sm.raw[st][0], static_cast<const T*>(a.B) + t * a.bs + (long long)grp * S, a.bs, rows, S,
                       a.copy_bc);
      if constexpr (kC)
        stage_rows<T, S, kTile, kThreads>(sm.raw[st][kC ? 1 : 0], static_cast<const T*>(a.C) + t * a.cs + (long long)grp * S, a.cs, rows,
                         S, a.copy_bc);
    }
    copy_async_commit();
  };
  // B, C of a tile in fp32 (a barrier before and after); rows past the chunk are not used
  auto convert = [&](int st, int buf) {
    if constexpr (TileSmem<T, S, MODE>::kConvert) {
#pragma unroll
      for (int i = 0; i < (kTile * S + kThreads - 1) / kThreads; ++i) {
        const int e = i * kThreads + (int)threadIdx.x;
        if (e < kTile * S) {
          (&sm.B[buf][0][0])[e] = to_f32<T>((&sm.raw[st][0][0][0])[e]);
          if constexpr (kC) (&sm.C[buf][0][0])[e] = to_f32<T>((&sm.raw[st][kC ? 1 : 0][0][0])[e]);
        }
      }
    }
  };
  stage(t0, 0);
  stage(t0 + kTile, 1);

  float2 A2[NP], h[NP];
  load_state<NP, LPC * 4>(a.A + crow, A2);
#pragma unroll
  for (int i = 0; i < NP; ++i) A2[i] = mul2(A2[i], dup2(kLog2eF));
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
  const float Dc = kC && a.Dv ? a.Dv[c] : 0.f;

  int n = seq_of_token(a.q, t0);
  long long end = seq_end(a.q, n);
  bool cut = seq_start(a.q, n) == t0;
  if (cut && a.S0) load_state<NP, LPC * 4>(a.S0 + (long long)n * a.d * S + crow, h);
  else if (!cut && MODE == kForward && a.entry) load_state<NP, LPC * 4>(a.entry + chunk * a.d * S + crow, h);
  else zero_state<NP>(h);
  constexpr int NPB = MODE == kLocalBwd ? NP : 1;
  float2 P[NPB], R[NPB];  // kLocalBwd: product of the decays so far, gradient sent to the left
#pragma unroll
  for (int i = 0; i < NPB; ++i) P[i] = dup2(1.f), R[i] = dup2(0.f);
  auto send_left = [&] {
    if constexpr (MODE == kLocalBwd)
      if (active) store_state<NP, LPC * 4>(a.exitg + chunk * a.d * S + crow, R);
  };
  if (cut) send_left();
  float sumd = 0.f;  // of the tokens that this lane prepares

  // the first of the lane's own tokens of a step, as reduce_scatter deals them
  int own0 = 0;
  {
    int have = kStep;
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) {
      have >>= 1;
      own0 += (sl & o) ? have : 0;
    }
  }

  T* yp = MODE == kForward ? static_cast<T*>(a.y) + (t0 + own0) * a.d + c : nullptr;

  auto next_sequence = [&](long long t) {
    if (MODE == kForward && a.S_out && active) store_state<NP, LPC * 4>(a.S_out + (long long)n * a.d * S + crow, h);
    n = next_seq(a.q, n, t);
    end = seq_end(a.q, n);
    if (!cut) send_left();  // what P and R add up from here on is not used
    cut = true;
    if (a.S0) load_state<NP, LPC * 4>(a.S0 + (long long)n * a.d * S + crow, h);
    else zero_state<NP>(h);
  };
  // one token of the lane's states -> its part of C . h.  gv: dy silu(z) (kLocalBwd); last: with dS
  auto token = [&](float2 dd, float2 uu, float gv, const float* tb, const float* tc, bool last) -> float {
    float2 acc = dup2(0.f);
#pragma unroll
    for (int p = 0; p < NP; p += 2) {
      const float4 b4 = *reinterpret_cast<const float4*>(tb + (p / 2 * LPC + sl) * 4);
      const float2 w0 = decay2(dd, A2[p]), w1 = decay2(dd, A2[p + 1]);
      h[p] = fma2(w0, h[p], mul2(uu, make_float2(b4.x, b4.y)));
      h[p + 1] = fma2(w1, h[p + 1], mul2(uu, make_float2(b4.z, b4.w)));
      if constexpr (kC) {
        const float4 c4 = *reinterpret_cast<const float4*>(tc + (p / 2 * LPC + sl) * 4);
        if constexpr (MODE == kForward) {
          acc = p == 0 ? mul2(h[p], make_float2(c4.x, c4.y)) : fma2(h[p], make_float2(c4.x, c4.y), acc);
          acc = fma2(h[p + 1], make_float2(c4.z, c4.w), acc);
        } else {
          P[p] = mul2(P[p], w0);
          P[p + 1] = mul2(P[p + 1], w1);
          float2 g0 = mul2(dup2(gv), make_float2(c4.x, c4.y)), g1 = mul2(dup2(gv), make_float2(c4.z, c4.w));
          if (last) {
            const float4 s4 = *reinterpret_cast<const float4*>(a.dS + (long long)n * a.d * S + crow + p / 2 * LPC * 4);
            g0 = add2(g0, make_float2(s4.x, s4.y));
            g1 = add2(g1, make_float2(s4.z, s4.w));
          }
          R[p] = fma2(P[p], g0, R[p]);
          R[p + 1] = fma2(P[p + 1], g1, R[p + 1]);
        }
      }
    }
    return acc.x + acc.y;
  };

  // What the lane prepares of a step whose inputs lie at in[.][s0 ..]: time steps, inputs, and the gate (kForward) or
  // dy times it (kLocalBwd).  No branch: it runs between the tokens of the step before.
  float xn[OWN], dn[OWN], gn[OWN];
  auto prepare = [&](const T(*in)[kTile][CH], int s0) {
#pragma unroll
    for (int j = 0; j < OWN; ++j) dn[j] = to_f32<T>(in[1][s0 + own0 + j][ch]) + bias;
#pragma unroll
    for (int j = 0; j < OWN; j += 2) {
      const float2 d2 = softplus2(make_float2(dn[j], dn[OWN > 1 ? j + 1 : j]));
      dn[j] = d2.x;
      if (OWN > 1) dn[OWN > 1 ? j + 1 : j] = d2.y;
    }
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      xn[j] = to_f32<T>(in[0][s0 + own0 + j][ch]);
      gn[j] = 1.f;
      if constexpr (kZ) {
        const float zz = to_f32<T>(in[kZ ? 2 : 0][s0 + own0 + j][ch]);  // anything without a gate
        const float g = zz * fast_sigmoid(zz);
        gn[j] = gated ? g : 1.f;
      }
      if constexpr (MODE == kLocalBwd) gn[j] *= to_f32<T>(in[MODE == kLocalBwd ? 3 : 0][s0 + own0 + j][ch]);
    }
  };

  copy_async_wait<1>();
  __syncthreads();
  convert(0, 0);
  prepare(sm.in[0], 0);  // rows past the chunk's end are prepared from anything and not used
  int buf = 0, st = 0;
  for (long long t = t0; t < t1; t += kTile) {
    copy_async_wait<0>();  // the next tile's copies of this thread
    __syncthreads();       // ... of all threads; this tile's B, C; and the stage after next is free
    const int st1 = st + 1 < kStages ? st + 1 : 0, st2 = st1 + 1 < kStages ? st1 + 1 : 0;
    stage(t + 2 * kTile, st2);
    if (t + kTile < t1) convert(st1, buf ^ 1);
    const T(*in)[kTile][CH] = sm.in[st];
    const float *Bt, *Ct;  // this tile's B, C, S numbers a token
    if constexpr (TileSmem<T, S, MODE>::kConvert) {
      Bt = &sm.B[buf][0][0];
      Ct = &sm.C[buf][0][0];
    } else {
      Bt = &sm.raw[st][0][0][0];
      Ct = &sm.raw[st][kC ? 1 : 0][0][0];
    }
#pragma unroll 1
    for (int s0 = 0; s0 < kTile && t + s0 < t1; s0 += kStep) {
      const long long ts = t + s0;
      if (ts == end) next_sequence(ts);  // the first token of another sequence
      const T(*in_next)[kTile][CH] = s0 + kStep < kTile ? in : sm.in[st1];
      const int s_next = s0 + kStep < kTile ? s0 + kStep : 0;
      // a final state's gradient is added at its sequence's last token, so that step goes token by token too
      if (ts + kStep <= t1 && (ts >= end || ts + kStep + (MODE == kLocalBwd) <= end)) {
        __syncwarp();  // the step before has been read
        float xv[OWN], gv[OWN];
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
          const int i = own0 + j;
          xv[j] = xn[j];
          gv[j] = gn[j];
          sm.du[i][ch] = make_float2(dn[j], dn[j] * xn[j]);
          if constexpr (MODE == kLocalBwd) sm.gv[MODE == kLocalBwd ? i : 0][ch] = gn[j];
          sumd += dn[j];
        }
        __syncwarp();
        prepare(in_next, s_next);
        float yv[kStep];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          const float2 du = sm.du[i][ch];
          yv[i] = token(dup2(du.x), dup2(du.y), MODE == kLocalBwd ? sm.gv[MODE == kLocalBwd ? i : 0][ch] : 0.f, Bt + (s0 + i) * S,
                        Ct + (s0 + i) * S, false);
        }
        if constexpr (MODE == kForward) {
          int at;
          reduce_scatter<kStep, LPC, 1>(yv, lane, &at);
          if (active) {
#pragma unroll
            for (int j = 0; j < OWN; ++j)
              yp[(long long)j * a.d] = from_f32<T>(fmaf(Dc, xv[j], yv[j]) * gv[j]);
          }
        }
      } else {
        const int m = t1 - ts < kStep ? (int)(t1 - ts) : kStep;
#pragma unroll 1
        for (int i = 0; i < m; ++i) {
          if (i > 0 && ts + i == end) next_sequence(ts + i);
          const float xv = to_f32<T>(in[0][s0 + i][ch]);
          const float delta = softplus_f(to_f32<T>(in[1][s0 + i][ch]) + bias);
          float gv = 1.f;
          if (gated) {
            const float zz = to_f32<T>(in[kZ ? 2 : 0][s0 + i][ch]);
            gv = zz * fast_sigmoid(zz);
          }
          if (MODE == kLocalBwd) gv *= to_f32<T>(in[MODE == kLocalBwd ? 3 : 0][s0 + i][ch]);
          float y = token(dup2(delta), dup2(delta * xv), gv, Bt + (s0 + i) * S, Ct + (s0 + i) * S,
                          MODE == kLocalBwd && a.dS && ts + i + 1 == end);
          if (sl == 0) sumd += delta;
          if (MODE == kForward) {
#pragma unroll
            for (int o = LPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (active && sl == 0) yp[(long long)(i - own0) * a.d] = from_f32<T>(fmaf(Dc, xv, y) * gv);
          }
        }
        prepare(in_next, s_next);
      }
      if (MODE == kForward) yp += (long long)kStep * a.d;
    }
    buf ^= 1;
    st = st1;
  }
  if constexpr (MODE == kForward) {
    if (t1 == end && a.S_out && active) store_state<NP, LPC * 4>(a.S_out + (long long)n * a.d * S + crow, h);
  } else {
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) sumd += __shfl_xor_sync(0xffffffffu, sumd, o);
    if (!cut) send_left();
    if (active) {
      store_state<NP, LPC * 4>(a.entry + chunk * a.d * S + crow, h);
      if (sl == 0) a.sumd[chunk * a.d + c] = cut ? -1.f : sumd;
    }
  }
}

// Chains the chunks, one thread per (channel, state); HBM-bound, 16 chunks in
// flight (128 chunks of 65536 states both ways: 23 us, 5.9 TB/s): entry[k] becomes the
// state that enters chunk k, exitg[k] (blockIdx.y == 1) the gradient that
// enters it from the right.
__global__ void __launch_bounds__(128) kda_scan_carry_kernel(const float* __restrict__ A, float* entry, float* exitg,
                                                             const float* __restrict__ sumd, int d, int S,
                                                             long long chunks) {
  constexpr int U = 16;  // chunks loaded together
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long row = (long long)d * S;
  if (i >= row) return;
  const int c = (int)(i / S);
  const float A2 = A[i] * kLog2eF;
  const bool rev = blockIdx.y == 1;
  const long long step = rev ? -row : row, dstep = rev ? -d : d;
  float* v = (rev ? exitg + (chunks - 1) * row : entry) + i;
  const float* sp = sumd + (rev ? (chunks - 1) * d : 0) + c;
  float h = 0.f;
  for (long long k0 = 0; k0 < chunks; k0 += U) {
    const int m = chunks - k0 < U ? (int)(chunks - k0) : U;
    float loc[U], sd[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < m) {
        loc[u] = v[u * step];
        sd[u] = sp[u * dstep];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < m) {
        v[u * step] = h;
        h = sd[u] < 0.f ? loc[u] : fmaf(ex2(fmaf(sd[u], A2, kEx2Bias)), h, loc[u]);
      }
    v += U * step;
    sp += U * dstep;
  }
}

// ---------------------------------------------------------------------------
// One token of each of N sequences.  A warp takes 32 channels of one sequence:
// a lane holds four states of a channel at a time (16-byte accesses, a warp's
// are adjacent), S / 4 passes for all of them.  What a channel needs once (time
// step, input, gate) is computed by lane `channel` and handed to the channel's
// lanes by exchange.  HBM-bound: the state is read and written once.  S_out may
// be S0.  256 sequences of 4096 channels, 16 states: 24 us, 6.0 TB/s.
// ---------------------------------------------------------------------------
constexpr int kStepWarps = 4;
template <typename T, int S>
__global__ void __launch_bounds__(kStepWarps * 32) kda_selective_scan_step_kernel(const Args a) {
  constexpr int LPC = S / 4, CPP = 32 / LPC;  // lanes a channel, channels a pass
  constexpr int U = LPC < 4 ? LPC : 4;        // passes loaded together
  const int lane = threadIdx.x & 31, sl = lane % LPC;
  const int n = blockIdx.y;
  const int wide = a.blocks_per_group;  // warps a group of channels
  const int wi = blockIdx.x * kStepWarps + (threadIdx.x >> 5);
  const int grp = wi / wide, c0 = (wi - grp * wide) * 32;  // first channel in the group
  if (grp >= a.d / a.cpg) return;
  const int left = a.cpg - c0;
  const long long cbase = (long long)grp * a.cpg + c0;
  const float* st = a.S0 + ((long long)n * a.d + cbase) * S;
  float* so = a.S_out + ((long long)n * a.d + cbase) * S;
  const float* Ap = a.A + cbase * S;

  float4 h[LPC / U][U], A4[LPC / U][U];  // one group is live at a time: all are unrolled
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int ch = i * CPP + lane / LPC;
    if (ch < left) {
      h[0][i] = *reinterpret_cast<const float4*>(st + (long long)ch * S + sl * 4);
      A4[0][i] = *reinterpret_cast<const float4*>(Ap + (long long)ch * S + sl * 4);
    }
  }
  const T* Bp = static_cast<const T*>(a.B) + n * a.bs + (long long)grp * S + sl * 4;
  const T* Cp = static_cast<const T*>(a.C) + n * a.cs + (long long)grp * S + sl * 4;
  float b[4], cc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = to_f32<T>(Bp[e]), cc[e] = to_f32<T>(Cp[e]);
  const long long c = cbase + (lane < left ? lane : left - 1);
  const float xv = to_f32<T>(static_cast<const T*>(a.x)[n * a.xs + c]);
  const float raw = to_f32<T>(static_cast<const T*>(a.dt)[n * a.dts + c]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
  const float zz = a.z ? to_f32<T>(static_cast<const T*>(a.z)[n * a.zs + c]) : 0.f;
  const float skip = a.Dv ? a.Dv[c] * xv : 0.f;
  const float delta = softplus_f(raw), u = delta * xv;
  float y = 0.f;
#pragma unroll
  for (int g = 0; g < LPC / U; ++g) {
    if (g + 1 < LPC / U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int ch = ((g + 1) * U + i) * CPP + lane / LPC;
        if (ch < left) {
          h[g + 1 < LPC / U ? g + 1 : 0][i] = *reinterpret_cast<const float4*>(st + (long long)ch * S + sl * 4);
          A4[g + 1 < LPC / U ? g + 1 : 0][i] = *reinterpret_cast<const float4*>(Ap + (long long)ch * S + sl * 4);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int p = g * U + i, ch = p * CPP + lane / LPC;
      const float dc = __shfl_sync(0xffffffffu, delta, ch), uc = __shfl_sync(0xffffffffu, u, ch);
      const float2 dl = dup2(dc * kLog2eF);
      const float2 w0 = decay2(dl, make_float2(A4[g][i].x, A4[g][i].y));
      const float2 w1 = decay2(dl, make_float2(A4[g][i].z, A4[g][i].w));
      float4 v = h[g][i];
      v.x = fmaf(w0.x, v.x, uc * b[0]);
      v.y = fmaf(w0.y, v.y, uc * b[1]);
      v.z = fmaf(w1.x, v.z, uc * b[2]);
      v.w = fmaf(w1.y, v.w, uc * b[3]);
      if (ch < left) *reinterpret_cast<float4*>(so + (long long)ch * S + sl * 4) = v;
      float s = fmaf(v.x, cc[0], v.y * cc[1]) + fmaf(v.z, cc[2], v.w * cc[3]);
#pragma unroll
      for (int o = LPC / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      // hand channel p * CPP + k its sum: lane k of the channel order reads from its group's lanes
      s = __shfl_sync(0xffffffffu, s, (lane % CPP) * LPC);
      if (lane / CPP == p) y = s;
    }
  }
  if (lane < left) {
    y += skip;
    if (a.z) y *= zz * fast_sigmoid(zz);
    static_cast<T*>(a.y)[(long long)n * a.d + c] = from_f32<T>(y);
  }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
inline bool supported_state(int S) { return S == 8 || S == 16 || S == 32 || S == 64; }
inline int lanes_per_channel(int S) { return S <= 16 ? S / 8 : S / 16; }
inline int channel_blocks(int d, int groups, int S) {
  const int ch = kThreads / lanes_per_channel(S);
  return groups * ((d / groups + ch - 1) / ch);
}

// Chunks of the forward.  A split costs the exponentials a second time, a call
// without one leaves SMs idle: 4096 tokens of 1024 channels (64 warps a row), split
// and unsplit: 4 rows 228 and 461 us, 8 rows 409 and 455, 12 rows 588 and 586, 16
// rows 760 and 585.  Packed sequences, whose lengths are on the device only, are
// one row here: unsplit, a CTA walks all their tokens (4 packed prompts of 2048
// tokens, 16 states, cut and in one walk: 4096 channels, 256 warps: 1475 and 3307
// us for 8 of 4096; 8192 channels 841 and 840; 12288 1113 and 1081; 16384 1651 and
// 1081; uneven lengths the same).  So a call with a warp or more for every SM
// sub-partition runs unsplit; others have the token axis cut so that about 16
// warps an SM run at once, into chunks of 64 tokens at least.  A batch's rows of
// the same sizes run side by side in half to two thirds of the packed time.
struct FwdPlan {
  bool split;
  long long L, chunks;
};
// The widest copy that every row of these inputs allows (null ones do not
// count).  A CTA's channels start at a multiple of 16 of their group.
inline int copy_width(std::initializer_list<const void*> ps, std::initializer_list<long long> strides, int esize) {
  uintptr_t low = 0;
  for (const void* p : ps) low |= reinterpret_cast<uintptr_t>(p);
  for (const long long s : strides) low |= (uintptr_t)(s * esize);
  return low % 16 == 0 ? 16 : low % 8 == 0 ? 8 : low % 4 == 0 ? 4 : 0;
}
inline void set_copies(Args& a, int S, int esize) {
  a.copy = copy_width({a.x, a.dt, a.z, a.dy},
                      {a.xs, a.dts, a.z ? a.zs : 0, a.dy ? a.d : 0, a.cpg == a.d ? 0 : a.cpg}, esize);
  a.copy_bc = copy_width({a.B, a.C}, {a.bs, a.cs, S}, esize);
}
inline FwdPlan fwd_plan(long long B, long long T, int d, int groups, int S) {
  const long long tokens = B * T;
  const long long warps = (long long)channel_blocks(d, groups, S) * (kThreads / 32);
  // rows that run side by side, and their tokens: B of T, or all packed sequences as one (then B == 1)
  if (B * warps >= 148 * 4 || T < 128) return {false, T > 0 ? T : 1, B};
  long long chunks = 148 * 16 / warps;
  if (chunks < 1) chunks = 1;
  long long L = (tokens + chunks - 1) / chunks;
  L = L < 64 ? 64 : (L + kTile - 1) / kTile * kTile;
  chunks = (tokens + L - 1) / L;
  return {chunks > 1, L, chunks};
}
inline size_t carry_floats(long long chunks, int d, int S) { return (size_t)chunks * d * S; }

template <typename T, int S, int MODE>
cudaError_t launch_scan(Args a, cudaStream_t st) {
  const long long grid = a.chunks * a.ncb;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  set_copies(a, S, (int)sizeof(T));
  constexpr size_t bytes = sizeof(TileSmem<T, S, MODE>);
  if (bytes > 48 * 1024) {
    static PerDeviceOnce once;
    const cudaError_t e = run_once_per_device(once, [] {
      return cudaFuncSetAttribute(kda_selective_scan_kernel<T, S, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)bytes);
    });
    if (e != cudaSuccess) return e;
  }
  kda_selective_scan_kernel<T, S, MODE><<<(unsigned)grid, kThreads, bytes, st>>>(a);
  return cudaGetLastError();
}
inline cudaError_t launch_carry(const Args& a, int S, bool both, cudaStream_t st) {
  const long long row = (long long)a.d * S;
  kda_scan_carry_kernel<<<dim3((unsigned)((row + 127) / 128), both ? 2 : 1), 128, 0, st>>>(a.A, a.entry, a.exitg,
                                                                                          a.sumd, a.d, S, a.chunks);
  return cudaGetLastError();
}
template <typename T, int S>
cudaError_t launch_fwd(Args a, bool split, cudaStream_t st) {
  if (split) {
    cudaError_t e = launch_scan<T, S, kLocal>(a, st);
    if (e != cudaSuccess) return e;
    if ((e = launch_carry(a, S, false, st)) != cudaSuccess) return e;
  }
  return launch_scan<T, S, kForward>(a, st);
}
template <typename T, int S>
cudaError_t launch_step(Args a, cudaStream_t st) {
  a.blocks_per_group = (a.cpg + 31) / 32;
  const int warps = a.blocks_per_group * (a.d / a.cpg);
  const unsigned grid = (unsigned)((warps + kStepWarps - 1) / kStepWarps);
  for (long long n0 = 0; n0 < a.q.num; n0 += 65535) {  // the grid's second dimension ends at 65535
    Args part = a;
    const long long m = a.q.num - n0 < 65535 ? a.q.num - n0 : 65535;
    const size_t es = sizeof(T);
    part.x = static_cast<const char*>(a.x) + n0 * a.xs * es;
    part.dt = static_cast<const char*>(a.dt) + n0 * a.dts * es;
    if (a.z) part.z = static_cast<const char*>(a.z) + n0 * a.zs * es;
    part.B = static_cast<const char*>(a.B) + n0 * a.bs * es;
    part.C = static_cast<const char*>(a.C) + n0 * a.cs * es;
    part.S0 = a.S0 + n0 * a.d * S;
    part.S_out = a.S_out + n0 * a.d * S;
    part.y = static_cast<char*>(a.y) + n0 * a.d * es;
    kda_selective_scan_step_kernel<T, S><<<dim3(grid, (unsigned)m), kStepWarps * 32, 0, st>>>(part);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace scan
}  // namespace kda

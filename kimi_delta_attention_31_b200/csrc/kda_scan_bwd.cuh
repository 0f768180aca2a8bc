// kda_scan_bwd.cuh -- backward pass of the selective scan.
//
// With dyy = dy silu(z), a_t = exp(delta_t A), g_t = C_t dyy_t + r_t and
// r_{t-1} = a_t g_t (r past a sequence's last token: dS):
//   dB_t = sum_c g u,  u = delta x;      dC_t = sum_c dyy h
//   dx = delta sum_n g B + D dyy;        ddelta = sum_n A g a h_{t-1} + x sum_n g B
//   ddt = ddelta sigmoid(dt + bias);     dA = sum_t delta g a h_{t-1}
//   dz = dy (C.h + D x) sg (1 + z (1 - sg)), sg = sigmoid(z);  dD = sum_t dyy x
//   dS0 = r before the first token.
//
// The token axis is cut into tiles of kTokens wherever they fall.  The states
// that enter every tile from the left and the gradients that enter it from the
// right come from kda_scan_local / carry (kda_scan.cuh).  A CTA then owns one
// tile and a block of channels.  A lane owns four states of a channel, a warp
// kRun consecutive tokens of 32 / (S / 4) channels: the decays of its tokens and
// the states that enter them stay in registers between the forward and the
// reverse sweep, so an exponential is taken once; the warps of a CTA are
// chained through shared memory the way the tiles are.  dB and dC are sums over
// channels: every lane adds up its own over all the channels that it works on,
// and the lanes of a warp that hold the same state are summed once at the end
// (summing them for every token took a fifth of the instructions).  Sums over
// tokens or channel blocks leave as lines that a second kernel adds in order.
//
// 4 x 2048 tokens of 4096 channels, 16 states: 1515 us, of which this kernel 1.24
// ms, the local scan 232 us, carry and sums 48.  Bound by latency: at 255 registers
// (the decays, entering states and channel sums of 8 tokens by 4 states a lane) one
// CTA of 8 warps fits an SM, an eighth of its warps, which wait for their own
// results and at two barriers for every 32 / (S / 4) channels; no pipe is full
// (issue 39%, L1 and shared memory 46%, exponential unit 13%, DRAM 4%).  Smaller
// shares in one larger CTA were slower, its chain being longer: 6 tokens and 12
// warps 8%, 4 tokens and 16 warps 9%.  Not tried: taking the decays again in the
// reverse sweep, which would make room for a second, independent CTA.
#pragma once
#include <type_traits>

#include "kda_scan.cuh"

namespace kda {
namespace scan {

constexpr int kRun = 8;                    // tokens a warp
constexpr int kWarps = 8;
constexpr int kTokens = kRun * kWarps;     // tokens a tile
constexpr int kBwdThreads = kWarps * 32;
constexpr int kSlab = 32;                  // channels prepared at a time

struct BwdOut {
  void *dx, *ddt, *dz;  // [tokens, d] T
  float* dS0;           // [N, d, S] or nullptr
  float* dA_lines;      // [tiles, d, S] (the entry states' place: each is read before it is written)
  float* ch_lines;      // [tiles, 2, d]: dD, ddt_bias
  float* bc_lines;      // [channel blocks a group, tokens, 2, groups, S]: dB, dC
  int slabs;            // slabs a CTA
  int groups;
};

template <int S>
struct BwdShape {
  static constexpr int LPC = S / 4;        // lanes a channel
  static constexpr int CPW = 32 / LPC;     // channels a warp at a time
  static constexpr int ACC = 8 / CPW > 0 ? 8 / CPW : 1;  // dB, dC sums a lane keeps of a token at the end
  static constexpr int BT = LPC < 4 ? LPC : 4;           // tokens whose state sums are exchanged together
};

template <typename T, int S>
struct alignas(16) BwdSmem {
  T in[2][4][kTokens][kSlab];  // x, dt, dy, z as they are in memory: this slab's and the next one's
  float B[kTokens][S], C[kTokens][S];
  float2 du[kTokens][kSlab];   // delta, delta x (each once: what lanes read bounds the kernel too)
  float dyy[kTokens][kSlab];
  float sA[kTokens][kSlab], gB[kTokens][kSlab], yy[kTokens][kSlab];
  float P[kWarps][128], H[kWarps][128], R[kWarps][128], dA[2][kWarps][128];
  float ch[kWarps][2][kSlab];
  int first[kTokens], last[kTokens];  // the sequence that starts / ends at this token, or -1
  int cut;                            // bit w: a sequence starts in the tokens of warp w
};

__device__ __forceinline__ float2 lo2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(float4 v) { return make_float2(v.z, v.w); }

template <typename T, int S>
__global__ void __launch_bounds__(kBwdThreads, 1) kda_selective_scan_bwd_kernel(const Args a, const BwdOut o) {
  using Sh = BwdShape<S>;
  constexpr int LPC = Sh::LPC, CPW = Sh::CPW, ACC = Sh::ACC, BT = Sh::BT;
  constexpr int kSteps = kSlab / CPW;  // of a slab
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<T, S>& s = *reinterpret_cast<BwdSmem<T, S>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane % LPC, chl = lane / LPC;
  const int cb = (int)(blockIdx.x % a.ncb);
  const long long tile = blockIdx.x / a.ncb;
  const int grp = cb / a.blocks_per_group, cbl = cb % a.blocks_per_group;
  const long long t0 = tile * kTokens;
  const int live = (int)(a.q.total - t0 < kTokens ? a.q.total - t0 : kTokens);
  const int tw = warp * kRun;  // the warp's first token in the tile
  const long long gch = (long long)grp * a.cpg;  // the group's first channel

  if (tid == 0) s.cut = 0;
  if (tid < kTokens) {
    int f = -1, l = -1;
    if (tid < live) {
      const int n = seq_of_token(a.q, t0 + tid);
      if (seq_start(a.q, n) == t0 + tid) f = n;
      if (seq_end(a.q, n) == t0 + tid + 1) l = n;
    }
    s.first[tid] = f;
    s.last[tid] = l;
  }
  for (int e = tid; e < kTokens * S; e += kBwdThreads) {
    const int t = e / S, k = e % S;
    float b = 0.f, cc = 0.f;
    if (t < live) {
      b = to_f32<T>(static_cast<const T*>(a.B)[(t0 + t) * a.bs + (long long)grp * S + k]);
      cc = to_f32<T>(static_cast<const T*>(a.C)[(t0 + t) * a.cs + (long long)grp * S + k]);
    }
    s.B[t][k] = b;
    s.C[t][k] = cc;
  }
  __syncthreads();
  bool starts = false, edges = false;
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    starts |= s.first[tw + k] >= 0;
    edges |= s.last[tw + k] >= 0;
  }
  edges |= starts;
  if (lane == 0 && starts) atomicOr(&s.cut, 1 << warp);  // read after the next barrier

  // dB and dC of the lane's four states, for each of the warp's tokens, over the lane's channels
  float2 accB[kRun][2], accC[kRun][2];
#pragma unroll
  for (int k = 0; k < kRun; ++k) accB[k][0] = accB[k][1] = accC[k][0] = accC[k][1] = dup2(0.f);

  // The lane's four states in step `step` of the slab at channel slab0, as an offset within the group (the last channel
  // again past its end), and what enters the tile at the element that this thread chains.
  auto lane_row = [&](int slab0, int step) { return min(slab0 + step * CPW + chl, a.cpg - 1) * S + sl * 4; };
  auto chain_load = [&](const float* src, int slab0, int step) {  // (nothing enters past the group's end)
    const int cin = slab0 + step * CPW + (tid & 127) / S;
    return cin < a.cpg ? src[cin * S + (tid & 127) % S] : 0.f;
  };
  const float* Ag = a.A + gch * S;
  const float* S0g = a.S0 ? a.S0 + gch * S : nullptr;
  const float* dSg = a.dS ? a.dS + gch * S : nullptr;
  float* dS0g = o.dS0 ? o.dS0 + gch * S : nullptr;
  const float* chain_src = (tid < 128 ? a.entry : a.exitg) + (tile * a.d + gch) * S;
  float* dAg = o.dA_lines + (tile * a.d + gch) * S;

  // the inputs of a slab, by asynchronous copies where their places allow it
  auto stage_one = [&](T(*dst)[kSlab], const void* src, long long stride, int slab0, int width) {
    stage_rows<T, kSlab, kTokens, kBwdThreads>(dst, static_cast<const T*>(src) + t0 * stride + gch + slab0, stride, live,
                                               width, a.copy);
  };
  auto stage_slab = [&](int slab) {
    const int slab0 = (cbl * o.slabs + slab) * kSlab;
    if (slab < o.slabs && slab0 < a.cpg) {
      const int width = a.cpg - slab0 < kSlab ? a.cpg - slab0 : kSlab;
      stage_one(s.in[slab & 1][0], a.x, a.xs, slab0, width);
      stage_one(s.in[slab & 1][1], a.dt, a.dts, slab0, width);
      stage_one(s.in[slab & 1][2], a.dy, a.d, slab0, width);
      if (a.z) stage_one(s.in[slab & 1][3], a.z, a.zs, slab0, width);
    }
    copy_async_commit();
  };
  stage_slab(0);
  // of the step to come
  float4 A4 = *reinterpret_cast<const float4*>(Ag + lane_row(cbl * o.slabs * kSlab, 0));
  float chained = chain_load(chain_src, cbl * o.slabs * kSlab, 0);

  for (int slab = 0; slab < o.slabs; ++slab) {
    const int slab0 = (cbl * o.slabs + slab) * kSlab;  // first channel of the slab in the group
    if (slab0 >= a.cpg) break;
    const T(*in)[kTokens][kSlab] = s.in[slab & 1];
    copy_async_wait<0>();
    __syncthreads();  // everybody's copies of this slab; the other buffer is free
    stage_slab(slab + 1);
    // prepare: lane = channel, the warp's own tokens
    const bool ch_ok = slab0 + lane < a.cpg;
    const long long c = gch + (ch_ok ? slab0 + lane : a.cpg - 1);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, Dc = a.Dv ? a.Dv[c] : 0.f;
#pragma unroll
    for (int k = 0; k < kRun; k += 2) {
      const float2 d2 = softplus2(make_float2(to_f32<T>(in[1][tw + k][lane]) + bias, to_f32<T>(in[1][tw + k + 1][lane]) + bias));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = tw + k + e;
        const bool ok = ch_ok && t < live;  // elsewhere the memory holds anything
        const float delta = ok ? (e ? d2.y : d2.x) : 0.f;
        float g = ok ? to_f32<T>(in[2][t][lane]) : 0.f;
        if (a.z && ok) {
          const float zz = to_f32<T>(in[3][t][lane]);
          g *= zz * fast_sigmoid(zz);
        }
        const float u = ok ? delta * to_f32<T>(in[0][t][lane]) : 0.f;
        s.du[t][lane] = make_float2(delta, u);
        s.dyy[t][lane] = g;
      }
    }
    __syncwarp();

    for (int step = 0; step < kSteps; ++step) {
      const int ch = step * CPW + chl;  // channel in the slab
      const bool c_ok = slab0 + ch < a.cpg;
      const int crow = lane_row(slab0, step);
      const float2 A2[2] = {mul2(lo2(A4), dup2(kLog2eF)), mul2(hi2(A4), dup2(kLog2eF))};
      float2 da[kRun][2], hin[kRun][2];
      // local sweep: decays, end state from zero, gradient sent left with none from the right
      auto local_sweep = [&](auto with_edges) {
        constexpr bool kEdges = decltype(with_edges)::value;
        float2 h0 = dup2(0.f), h1 = dup2(0.f), P0 = dup2(1.f), P1 = dup2(1.f), r0 = dup2(0.f), r1 = dup2(0.f);
        bool open = true;  // no sequence has started among the warp's tokens yet: what comes after a start is sent to nobody
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t = tw + k;
          const float2 dux = s.du[t][ch];
          const float4 du = make_float4(dux.x, dux.x, dux.y, dux.y);
          const float2 gy = dup2(s.dyy[t][ch]);
          const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
          const float4 c4 = *reinterpret_cast<const float4*>(&s.C[t][sl * 4]);
          da[k][0] = decay2(lo2(du), A2[0]);
          da[k][1] = decay2(lo2(du), A2[1]);
          if (kEdges && s.first[t] >= 0) {
            h0 = h1 = dup2(0.f);
            if (S0g) {
              const float4 v = *reinterpret_cast<const float4*>(S0g + (long long)s.first[t] * a.d * S + crow);
              h0 = lo2(v), h1 = hi2(v);
            }
            open = false;
          }
          h0 = fma2(da[k][0], h0, mul2(hi2(du), lo2(b4)));
          h1 = fma2(da[k][1], h1, mul2(hi2(du), hi2(b4)));
          P0 = mul2(P0, da[k][0]);
          P1 = mul2(P1, da[k][1]);
          float2 g0 = mul2(gy, lo2(c4)), g1 = mul2(gy, hi2(c4));
          if (kEdges && s.last[t] >= 0 && dSg) {
            const float4 v = *reinterpret_cast<const float4*>(dSg + (long long)s.last[t] * a.d * S + crow);
            g0 = add2(g0, lo2(v));
            g1 = add2(g1, hi2(v));
          }
          if (!kEdges || open) {
            r0 = fma2(P0, g0, r0);
            r1 = fma2(P1, g1, r1);
          }
        }
        *reinterpret_cast<float4*>(&s.P[warp][lane * 4]) = make_float4(P0.x, P0.y, P1.x, P1.y);
        *reinterpret_cast<float4*>(&s.H[warp][lane * 4]) = make_float4(h0.x, h0.y, h1.x, h1.y);
        *reinterpret_cast<float4*>(&s.R[warp][lane * 4]) = make_float4(r0.x, r0.y, r1.x, r1.y);
      };
      if (edges) local_sweep(std::true_type{});
      else local_sweep(std::false_type{});
      __syncthreads();
      // chain the warps: 128 threads forward, 128 in reverse; then dA of the step before
      {
        const int i = tid & 127, cut = s.cut;
        float v = chained;
        float loc[kWarps], p[kWarps];  // in the order of the chain
        float(*own)[128] = tid < 128 ? s.H : s.R;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const int w = tid < 128 ? k : kWarps - 1 - k;
          loc[k] = own[w][i];
          p[k] = (cut >> w) & 1 ? 0.f : s.P[w][i];
        }
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const int w = tid < 128 ? k : kWarps - 1 - k;
          own[w][i] = v;
          v = p[k] == 0.f ? loc[k] : fmaf(p[k], v, loc[k]);  // nothing passes a start, an infinity neither
        }
        // (the next slab's first step follows the last one; past the block it is read and not used)
        A4 = *reinterpret_cast<const float4*>(Ag + lane_row(slab0, step + 1));
        chained = chain_load(chain_src, slab0, step + 1);
        if (step > 0 && tid >= kBwdThreads - 128) {
          const int cch = slab0 + (step - 1) * CPW + i / S;
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += s.dA[(step - 1) & 1][w][i];
          if (cch < a.cpg) dAg[cch * S + i % S] = sum;
        }
      }
      __syncthreads();
      auto final_sweeps = [&](auto with_edges) {
        constexpr bool kEdges = decltype(with_edges)::value;
        // the states that enter each token
        {
          const float4 v = *reinterpret_cast<const float4*>(&s.H[warp][lane * 4]);
          float2 h0 = lo2(v), h1 = hi2(v);
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            const int t = tw + k;
            if (kEdges && s.first[t] >= 0) {
              h0 = h1 = dup2(0.f);
              if (S0g) {
                const float4 q = *reinterpret_cast<const float4*>(S0g + (long long)s.first[t] * a.d * S + crow);
                h0 = lo2(q), h1 = hi2(q);
              }
            }
            hin[k][0] = h0;
            hin[k][1] = h1;
            if (k + 1 < kRun) {
              const float2 u = dup2(s.du[t][ch].y);
              const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
              h0 = fma2(da[k][0], h0, mul2(u, lo2(b4)));
              h1 = fma2(da[k][1], h1, mul2(u, hi2(b4)));
            }
          }
        }
        // reverse sweep
        const float4 v = *reinterpret_cast<const float4*>(&s.R[warp][lane * 4]);
        float2 r0 = lo2(v), r1 = hi2(v), dA0 = dup2(0.f), dA1 = dup2(0.f);
#pragma unroll
        for (int kb = kRun / BT - 1; kb >= 0; --kb) {
          float vA[BT], vG[BT], vY[BT];
#pragma unroll
          for (int kk = BT - 1; kk >= 0; --kk) {
            const int k = kb * BT + kk, t = tw + k;
            const float2 dux = s.du[t][ch];
            const float4 du = make_float4(dux.x, dux.x, dux.y, dux.y);
            const float2 gy = dup2(s.dyy[t][ch]), u = hi2(du);
            const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
            const float4 c4 = *reinterpret_cast<const float4*>(&s.C[t][sl * 4]);
            if (kEdges && s.last[t] >= 0) {  // what comes from the right is the final state's gradient
              r0 = r1 = dup2(0.f);
              if (dSg) {
                const float4 q = *reinterpret_cast<const float4*>(dSg + (long long)s.last[t] * a.d * S + crow);
                r0 = lo2(q), r1 = hi2(q);
              }
            }
            const float2 g0 = fma2(gy, lo2(c4), r0), g1 = fma2(gy, hi2(c4), r1);
            const float2 ah0 = mul2(da[k][0], hin[k][0]), ah1 = mul2(da[k][1], hin[k][1]);
            const float2 h0 = fma2(u, lo2(b4), ah0), h1 = fma2(u, hi2(b4), ah1);
            const float2 gb = fma2(g0, lo2(b4), mul2(g1, hi2(b4)));
            const float2 ga0 = mul2(g0, ah0), ga1 = mul2(g1, ah1);
            dA0 = fma2(lo2(du), ga0, dA0);
            dA1 = fma2(lo2(du), ga1, dA1);
            const float2 sa = fma2(A2[0], ga0, mul2(A2[1], ga1));
            const float2 yy = fma2(lo2(c4), h0, mul2(hi2(c4), h1));
            vA[kk] = sa.x + sa.y;
            vG[kk] = gb.x + gb.y;
            vY[kk] = yy.x + yy.y;
            accB[k][0] = fma2(g0, u, accB[k][0]);
            accB[k][1] = fma2(g1, u, accB[k][1]);
            accC[k][0] = fma2(gy, h0, accC[k][0]);
            accC[k][1] = fma2(gy, h1, accC[k][1]);
            r0 = mul2(da[k][0], g0);
            r1 = mul2(da[k][1], g1);
            if (kEdges && s.first[t] >= 0 && dS0g && c_ok)
              *reinterpret_cast<float4*>(dS0g + (long long)s.first[t] * a.d * S + crow) =
                  make_float4(r0.x, r0.y, r1.x, r1.y);
          }
          int at;
          reduce_scatter<BT, LPC, 1>(vA, lane, &at);
          reduce_scatter<BT, LPC, 1>(vG, lane, &at);
          reduce_scatter<BT, LPC, 1>(vY, lane, &at);
          if (sl % (LPC / BT) == 0) {
            const int t = tw + kb * BT + at;
            s.sA[t][ch] = vA[0];
            s.gB[t][ch] = vG[0];
            s.yy[t][ch] = vY[0];
          }
        }
        *reinterpret_cast<float4*>(&s.dA[step & 1][warp][lane * 4]) = make_float4(dA0.x, dA0.y, dA1.x, dA1.y);
      };
      if (edges) final_sweeps(std::true_type{});
      else final_sweeps(std::false_type{});
    }
    __syncwarp();
    // outputs per (token, channel): lane = channel, the warp's own tokens
    float dDs = 0.f, dbs = 0.f;
    if (ch_ok) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        if (tw + k < live) {
          const long long t = t0 + tw + k;
          const float xv = to_f32<T>(in[0][tw + k][lane]);
          const float raw = to_f32<T>(in[1][tw + k][lane]) + bias;
          const float delta = s.du[tw + k][lane].x, gy = s.dyy[tw + k][lane], gb = s.gB[tw + k][lane];
          const float ddelta = fmaf(gb, xv, s.sA[tw + k][lane] * kLn2F);
          const float ddt = ddelta * fast_sigmoid(raw);
          static_cast<T*>(o.dx)[t * a.d + c] = from_f32<T>(fmaf(gb, delta, Dc * gy));
          static_cast<T*>(o.ddt)[t * a.d + c] = from_f32<T>(ddt);
          dDs = fmaf(gy, xv, dDs);
          dbs += ddt;
          if (a.z) {
            const float zz = to_f32<T>(in[3][tw + k][lane]);
            const float dyo = to_f32<T>(in[2][tw + k][lane]);
            const float sg = fast_sigmoid(zz);
            const float y = fmaf(Dc, xv, s.yy[tw + k][lane]);
            static_cast<T*>(o.dz)[t * a.d + c] = from_f32<T>(dyo * y * sg * fmaf(zz, 1.f - sg, 1.f));
          }
        }
      }
    }
    s.ch[warp][0][lane] = dDs;
    s.ch[warp][1][lane] = dbs;
    __syncthreads();
    if (tid < 2 * kSlab && slab0 + lane < a.cpg) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s.ch[w][warp][lane];
      o.ch_lines[(tile * 2 + warp) * a.d + gch + slab0 + lane] = v;
    }
    if (tid >= 128 && tid < 256) {  // dA of the slab's last step
      const int i = tid & 127, cch = slab0 + (kSteps - 1) * CPW + i / S;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += s.dA[(kSteps - 1) & 1][w][i];
      if (cch < a.cpg) dAg[cch * S + i % S] = sum;
    }
  }

  // dB, dC of the block's channels: [block][token][2][group][S]
  const bool writer = CPW <= 8 || (chl & 1) == 0;  // CPW 16: two lanes hold each sum
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    float v[8] = {accB[k][0].x, accB[k][0].y, accB[k][1].x, accB[k][1].y,
                  accC[k][0].x, accC[k][0].y, accC[k][1].x, accC[k][1].y};
    int at;
    reduce_scatter<8, CPW, LPC>(v, lane, &at);
#pragma unroll
    for (int j = 0; j < ACC; ++j) {
      const int i = at + j;  // 0..3 dB, 4..7 dC of state sl * 4 + i % 4
      if (writer && tw + k < live)
        o.bc_lines[((((long long)cbl * a.q.total + t0 + tw + k) * 2 + i / 4) * o.groups + grp) * S + sl * 4 + i % 4] =
            v[j];
    }
  }
}

// dS0 of sequences without tokens: what comes from the right passes.
__global__ void __launch_bounds__(256) kda_scan_empty_bwd_kernel(const Seqs q, const float* dS, float* dS0,
                                                                 long long row) {
  if (blockIdx.x == 0) check_seq_table(q);
  for (int n = blockIdx.x; n < q.num; n += gridDim.x)
    if (seq_empty(q, n))
      for (long long i = threadIdx.x; i < row; i += blockDim.x) dS0[n * row + i] = dS ? dS[n * row + i] : 0.f;
}

// Sums of dB and dC over the channel blocks: lines [block][token][2][groups S].
__global__ void __launch_bounds__(256) kda_scan_sum_bc_kernel(const float* __restrict__ lines, float* __restrict__ dB,
                                                              float* __restrict__ dC, int blocks, long long tokens,
                                                              int row) {
  const long long total = tokens * 2 * row;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  float v = 0.f;
#pragma unroll 4
  for (int b = 0; b < blocks; ++b) v += lines[b * total + i];
  const long long t = i / (2 * row);
  const int r = (int)(i - t * 2 * row);
  if (r < row) dB[t * row + r] = v;
  else dC[t * row + r - row] = v;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct BwdPlan {
  long long tiles;
  int slabs, blocks_per_group;  // slabs a CTA, CTAs a group and tile
};
// Channel blocks: enough CTAs for about eight rounds of one an SM; fewer blocks
// mean fewer lines of dB and dC.
inline BwdPlan bwd_plan(long long tokens, int d, int groups) {
  BwdPlan p;
  p.tiles = (tokens + kTokens - 1) / kTokens;
  const int all = (d / groups + kSlab - 1) / kSlab;  // slabs a group
  const long long want = 148 * 8;
  long long per = (want + p.tiles * groups - 1) / (p.tiles > 0 ? p.tiles * groups : 1);
  per = per < 1 ? 1 : per > all ? all : per;
  p.slabs = (int)((all + per - 1) / per);
  p.blocks_per_group = (all + p.slabs - 1) / p.slabs;
  return p;
}
struct BwdLayout {
  size_t entry, exitg, sumd, ch, bc, total;  // bytes
};
inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }
inline BwdLayout bwd_layout(long long tokens, int d, int groups, int S) {
  const BwdPlan p = bwd_plan(tokens, d, groups);
  BwdLayout l;
  const size_t carry = round256((size_t)p.tiles * d * S * 4);
  l.entry = 0;
  l.exitg = carry;
  l.sumd = 2 * carry;
  l.ch = l.sumd + round256((size_t)p.tiles * d * 4);
  l.bc = l.ch + round256((size_t)p.tiles * 2 * d * 4);
  l.total = l.bc + round256((size_t)p.blocks_per_group * tokens * 2 * groups * S * 4);
  return l;
}

template <typename T, int S>
cudaError_t launch_bwd(Args a, BwdOut o, float* dA, float* dB, float* dC, float* dD, float* ddt_bias, int groups,
                       void* workspace, cudaStream_t st) {
  const long long tokens = a.q.total;
  const BwdPlan p = bwd_plan(tokens, a.d, groups);
  const BwdLayout l = bwd_layout(tokens, a.d, groups, S);
  char* ws = static_cast<char*>(workspace);
  a.entry = reinterpret_cast<float*>(ws + l.entry);
  a.exitg = reinterpret_cast<float*>(ws + l.exitg);
  a.sumd = reinterpret_cast<float*>(ws + l.sumd);
  o.dA_lines = a.entry;
  o.ch_lines = reinterpret_cast<float*>(ws + l.ch);
  o.bc_lines = reinterpret_cast<float*>(ws + l.bc);
  o.slabs = p.slabs;
  o.groups = groups;
  a.L = kTokens;
  a.chunks = p.tiles;
  cudaError_t e;
  const long long row = (long long)a.d * S;
  if (o.dS0 && a.q.num > 0 && (a.q.cu || tokens == 0)) {
    const int grid = a.q.num < 1024 ? a.q.num : 1024;
    kda_scan_empty_bwd_kernel<<<grid, 256, 0, st>>>(a.q, a.dS, o.dS0, row);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (tokens > 0) {
    a.ncb = channel_blocks(a.d, groups, S);
    a.blocks_per_group = a.ncb / groups;
    if ((e = launch_scan<T, S, kLocalBwd>(a, st)) != cudaSuccess) return e;
    if ((e = launch_carry(a, S, true, st)) != cudaSuccess) return e;
    set_copies(a, S, (int)sizeof(T));
    a.ncb = p.blocks_per_group * groups;
    a.blocks_per_group = p.blocks_per_group;
    static PerDeviceOnce once;
    e = run_once_per_device(once, [] {
      return cudaFuncSetAttribute(kda_selective_scan_bwd_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)sizeof(BwdSmem<T, S>));
    });
    if (e != cudaSuccess) return e;
    const long long grid = p.tiles * a.ncb;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kda_selective_scan_bwd_kernel<T, S><<<(unsigned)grid, kBwdThreads, sizeof(BwdSmem<T, S>), st>>>(a, o);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long bc = tokens * 2 * groups * S;
    kda_scan_sum_bc_kernel<<<(unsigned)((bc + 255) / 256), 256, 0, st>>>(o.bc_lines, dB, dC, p.blocks_per_group,
                                                                         tokens, groups * S);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if ((e = launch_sum_lines(o.dA_lines, dA, nullptr, row, (int)p.tiles, row, st)) != cudaSuccess) return e;
  return launch_sum_lines(o.ch_lines, dD, ddt_bias, a.d, (int)p.tiles, 2LL * a.d, st);
}

}  // namespace scan
}  // namespace kda

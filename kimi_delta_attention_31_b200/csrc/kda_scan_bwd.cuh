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
// channels: the lanes of a warp that hold the same state are summed by
// exchanges that halve the number of values at each step, and the result stays
// in registers over all the CTA's channels.  Sums over tokens or channel blocks
// leave as lines that a second kernel adds in order.
#pragma once
#include "kda_scan.cuh"

namespace kda {
namespace scan {

constexpr int kRun = 8;                    // tokens a warp
constexpr int kWarps = 8;
constexpr int kTokens = kRun * kWarps;     // tokens a tile
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
  static constexpr int ACC = 8 / CPW > 0 ? 8 / CPW : 1;  // dB, dC sums a lane keeps of a token
  static constexpr int BT = LPC < 4 ? LPC : 4;           // tokens whose state sums are exchanged together
};

template <int S>
struct alignas(16) BwdSmem {
  float B[kTokens][S], C[kTokens][S];
  float delta[kTokens][kSlab], u[kTokens][kSlab], dyy[kTokens][kSlab];
  float sA[kTokens][kSlab], gB[kTokens][kSlab], yy[kTokens][kSlab];
  float P[kWarps][128], H[kWarps][128], R[kWarps][128], dA[kWarps][128];
  float ch[kWarps][2][kSlab];
  int first[kTokens], last[kTokens];  // the sequence that starts / ends at this token, or -1
  int cut[kWarps];                    // a sequence starts in the warp's tokens
};

template <typename T, int S>
__global__ void __launch_bounds__(kWarps * 32, 2) kda_selective_scan_bwd_kernel(const Args a, const BwdOut o) {
  using Sh = BwdShape<S>;
  constexpr int LPC = Sh::LPC, CPW = Sh::CPW, ACC = Sh::ACC, BT = Sh::BT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<S>& s = *reinterpret_cast<BwdSmem<S>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane % LPC, chl = lane / LPC;
  const int cb = (int)(blockIdx.x % a.ncb);
  const long long tile = blockIdx.x / a.ncb;
  const int grp = cb / a.blocks_per_group, cbl = cb % a.blocks_per_group;
  const long long t0 = tile * kTokens;
  const int live = (int)(a.q.total - t0 < kTokens ? a.q.total - t0 : kTokens);
  const int tw = warp * kRun;  // the warp's first token in the tile

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
  for (int e = tid; e < kTokens * S; e += kWarps * 32) {
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
  if (lane == 0) {
    int any = 0;
#pragma unroll
    for (int k = 0; k < kRun; ++k) any |= s.first[tw + k] >= 0;
    s.cut[warp] = any;
  }

  float acc[kRun][ACC];
#pragma unroll
  for (int k = 0; k < kRun; ++k)
#pragma unroll
    for (int j = 0; j < ACC; ++j) acc[k][j] = 0.f;

  for (int slab = 0; slab < o.slabs; ++slab) {
    const int slab0 = (cbl * o.slabs + slab) * kSlab;  // first channel of the slab in the group
    if (slab0 >= a.cpg) break;
    // prepare: lane = channel, the warp's own tokens
    const bool ch_ok = slab0 + lane < a.cpg;
    const long long c = (long long)grp * a.cpg + (ch_ok ? slab0 + lane : a.cpg - 1);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, Dc = a.Dv ? a.Dv[c] : 0.f;
    {
      T rx[kRun], rdt[kRun], rz[kRun], rdy[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const long long t = t0 + (tw + k < live ? tw + k : live - 1);
        rx[k] = static_cast<const T*>(a.x)[t * a.xs + c];
        rdt[k] = static_cast<const T*>(a.dt)[t * a.dts + c];
        rdy[k] = static_cast<const T*>(a.dy)[t * a.d + c];
        if (a.z) rz[k] = static_cast<const T*>(a.z)[t * a.zs + c];
      }
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        const bool ok = ch_ok && tw + k < live;
        const float delta = softplus_f(to_f32<T>(rdt[k]) + bias);
        float g = to_f32<T>(rdy[k]);
        if (a.z) {
          const float zz = to_f32<T>(rz[k]);
          g *= zz * fast_sigmoid(zz);
        }
        s.delta[tw + k][lane] = ok ? delta : 0.f;
        s.u[tw + k][lane] = ok ? delta * to_f32<T>(rx[k]) : 0.f;
        s.dyy[tw + k][lane] = ok ? g : 0.f;
      }
    }
    __syncwarp();

    for (int step = 0; step < kSlab / CPW; ++step) {
      const int ch = step * CPW + chl;  // channel in the slab
      const int cin = slab0 + ch;
      const bool c_ok = cin < a.cpg;
      const long long crow = ((long long)grp * a.cpg + (c_ok ? cin : a.cpg - 1)) * S + sl * 4;
      const float4 A4 = *reinterpret_cast<const float4*>(a.A + crow);
      const float2 A2[2] = {make_float2(A4.x * kLog2eF, A4.y * kLog2eF), make_float2(A4.z * kLog2eF, A4.w * kLog2eF)};
      // local sweep: decays, end state from zero, gradient sent left with none from the right
      float2 da[kRun][2], hin[kRun][2];
      {
        float2 h0 = dup2(0.f), h1 = dup2(0.f), P0 = dup2(1.f), P1 = dup2(1.f), r0 = dup2(0.f), r1 = dup2(0.f);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t = tw + k;
          const float2 dl = dup2(s.delta[t][ch]), u = dup2(s.u[t][ch]), gy = dup2(s.dyy[t][ch]);
          const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
          const float4 c4 = *reinterpret_cast<const float4*>(&s.C[t][sl * 4]);
          da[k][0] = decay2(dl, A2[0]);
          da[k][1] = decay2(dl, A2[1]);
          if (s.first[t] >= 0) {
            h0 = h1 = dup2(0.f);
            if (a.S0) {
              const float4 v = *reinterpret_cast<const float4*>(a.S0 + (long long)s.first[t] * a.d * S + crow);
              h0 = make_float2(v.x, v.y), h1 = make_float2(v.z, v.w);
            }
            P0 = P1 = dup2(0.f);
          }
          h0 = fma2(da[k][0], h0, mul2(u, make_float2(b4.x, b4.y)));
          h1 = fma2(da[k][1], h1, mul2(u, make_float2(b4.z, b4.w)));
          P0 = mul2(P0, da[k][0]);
          P1 = mul2(P1, da[k][1]);
          float2 g0 = mul2(gy, make_float2(c4.x, c4.y)), g1 = mul2(gy, make_float2(c4.z, c4.w));
          if (s.last[t] >= 0 && a.dS) {
            const float4 v = *reinterpret_cast<const float4*>(a.dS + (long long)s.last[t] * a.d * S + crow);
            g0 = add2(g0, make_float2(v.x, v.y));
            g1 = add2(g1, make_float2(v.z, v.w));
          }
          r0 = fma2(P0, g0, r0);
          r1 = fma2(P1, g1, r1);
        }
        *reinterpret_cast<float4*>(&s.P[warp][lane * 4]) = make_float4(P0.x, P0.y, P1.x, P1.y);
        *reinterpret_cast<float4*>(&s.H[warp][lane * 4]) = make_float4(h0.x, h0.y, h1.x, h1.y);
        *reinterpret_cast<float4*>(&s.R[warp][lane * 4]) = make_float4(r0.x, r0.y, r1.x, r1.y);
      }
      __syncthreads();
      // chain the warps: 128 threads forward, 128 in reverse
      {
        const int i = tid & 127;
        const int cch = slab0 + step * CPW + i / S;
        const long long at = tile * a.d * S + ((long long)grp * a.cpg + (cch < a.cpg ? cch : a.cpg - 1)) * S + i % S;
        if (tid < 128) {
          float h = a.entry[at];
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float loc = s.H[w][i];
            s.H[w][i] = h;
            h = s.cut[w] ? loc : fmaf(s.P[w][i], h, loc);
          }
        } else {
          float r = a.exitg[at];
#pragma unroll
          for (int w = kWarps - 1; w >= 0; --w) {
            const float loc = s.R[w][i];
            s.R[w][i] = r;
            r = s.cut[w] ? loc : fmaf(s.P[w][i], r, loc);
          }
        }
      }
      __syncthreads();
      // the states that enter each token
      {
        const float4 v = *reinterpret_cast<const float4*>(&s.H[warp][lane * 4]);
        float2 h0 = make_float2(v.x, v.y), h1 = make_float2(v.z, v.w);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
          const int t = tw + k;
          if (s.first[t] >= 0) {
            h0 = h1 = dup2(0.f);
            if (a.S0) {
              const float4 q = *reinterpret_cast<const float4*>(a.S0 + (long long)s.first[t] * a.d * S + crow);
              h0 = make_float2(q.x, q.y), h1 = make_float2(q.z, q.w);
            }
          }
          hin[k][0] = h0;
          hin[k][1] = h1;
          if (k + 1 < kRun) {
            const float2 u = dup2(s.u[t][ch]);
            const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
            h0 = fma2(da[k][0], h0, mul2(u, make_float2(b4.x, b4.y)));
            h1 = fma2(da[k][1], h1, mul2(u, make_float2(b4.z, b4.w)));
          }
        }
      }
      // reverse sweep
      {
        const float4 v = *reinterpret_cast<const float4*>(&s.R[warp][lane * 4]);
        float2 r0 = make_float2(v.x, v.y), r1 = make_float2(v.z, v.w);
        float2 dA0 = dup2(0.f), dA1 = dup2(0.f);
#pragma unroll
        for (int kb = kRun / BT - 1; kb >= 0; --kb) {
          float vA[BT], vG[BT], vY[BT];
#pragma unroll
          for (int kk = BT - 1; kk >= 0; --kk) {
            const int k = kb * BT + kk, t = tw + k;
            const float delta = s.delta[t][ch];
            const float2 u = dup2(s.u[t][ch]), gy = dup2(s.dyy[t][ch]);
            const float4 b4 = *reinterpret_cast<const float4*>(&s.B[t][sl * 4]);
            const float4 c4 = *reinterpret_cast<const float4*>(&s.C[t][sl * 4]);
            const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
            const float2 c0 = make_float2(c4.x, c4.y), c1 = make_float2(c4.z, c4.w);
            if (s.last[t] >= 0) {  // what comes from the right is the final state's gradient
              r0 = r1 = dup2(0.f);
              if (a.dS) {
                const float4 q = *reinterpret_cast<const float4*>(a.dS + (long long)s.last[t] * a.d * S + crow);
                r0 = make_float2(q.x, q.y), r1 = make_float2(q.z, q.w);
              }
            }
            const float2 g0 = fma2(gy, c0, r0), g1 = fma2(gy, c1, r1);
            const float2 ah0 = mul2(da[k][0], hin[k][0]), ah1 = mul2(da[k][1], hin[k][1]);
            const float2 h0 = fma2(u, b0, ah0), h1 = fma2(u, b1, ah1);
            const float2 gb = fma2(g0, b0, mul2(g1, b1));
            const float2 ga0 = mul2(g0, ah0), ga1 = mul2(g1, ah1);
            dA0 = fma2(dup2(delta), ga0, dA0);
            dA1 = fma2(dup2(delta), ga1, dA1);
            const float2 sa = fma2(A2[0], ga0, mul2(A2[1], ga1));
            const float2 yy = fma2(c0, h0, mul2(c1, h1));
            vA[kk] = sa.x + sa.y;
            vG[kk] = gb.x + gb.y;
            vY[kk] = yy.x + yy.y;
            const float2 vb0 = mul2(g0, u), vb1 = mul2(g1, u), vc0 = mul2(gy, h0), vc1 = mul2(gy, h1);
            float bc[8] = {vb0.x, vb0.y, vb1.x, vb1.y, vc0.x, vc0.y, vc1.x, vc1.y};
            int at;
            reduce_scatter<8, CPW, LPC>(bc, lane, &at);
#pragma unroll
            for (int j = 0; j < ACC; ++j) acc[k][j] += bc[j];
            r0 = mul2(da[k][0], g0);
            r1 = mul2(da[k][1], g1);
            if (s.first[t] >= 0 && o.dS0 && c_ok)
              *reinterpret_cast<float4*>(o.dS0 + (long long)s.first[t] * a.d * S + crow) =
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
        *reinterpret_cast<float4*>(&s.dA[warp][lane * 4]) = make_float4(dA0.x, dA0.y, dA1.x, dA1.y);
      }
      __syncthreads();
      if (tid < 128) {
        const int cch = slab0 + step * CPW + tid / S;
        if (cch < a.cpg) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += s.dA[w][tid];
          o.dA_lines[tile * a.d * S + ((long long)grp * a.cpg + cch) * S + tid % S] = v;
        }
      }
    }
    // outputs per (token, channel): lane = channel, the warp's own tokens
    float dDs = 0.f, dbs = 0.f;
    if (ch_ok) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        if (tw + k < live) {
          const long long t = t0 + tw + k;
          const float xv = to_f32<T>(static_cast<const T*>(a.x)[t * a.xs + c]);
          const float raw = to_f32<T>(static_cast<const T*>(a.dt)[t * a.dts + c]) + bias;
          const float delta = s.delta[tw + k][lane], gy = s.dyy[tw + k][lane], gb = s.gB[tw + k][lane];
          const float ddelta = fmaf(gb, xv, s.sA[tw + k][lane] * kLn2F);
          const float ddt = ddelta * fast_sigmoid(raw);
          static_cast<T*>(o.dx)[t * a.d + c] = from_f32<T>(fmaf(gb, delta, Dc * gy));
          static_cast<T*>(o.ddt)[t * a.d + c] = from_f32<T>(ddt);
          dDs = fmaf(gy, xv, dDs);
          dbs += ddt;
          if (a.z) {
            const float zz = to_f32<T>(static_cast<const T*>(a.z)[t * a.zs + c]);
            const float dyo = to_f32<T>(static_cast<const T*>(a.dy)[t * a.d + c]);
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
      o.ch_lines[(tile * 2 + warp) * a.d + (long long)grp * a.cpg + slab0 + lane] = v;
    }
  }

  // dB, dC of the block's channels: [block][token][2][group][S]
  {
    int at = 0, have = 8;
#pragma unroll
    for (int b = CPW / 2; b > 0; b >>= 1) {
      if (have > 1) {
        have >>= 1;
        at += (lane & (b * LPC)) ? have : 0;
      }
    }
    const bool writer = CPW <= 8 || (chl & 1) == 0;  // CPW 16: two lanes hold each sum
#pragma unroll
    for (int k = 0; k < kRun; ++k)
#pragma unroll
      for (int j = 0; j < ACC; ++j) {
        const int v = at + j;  // 0..3 dB, 4..7 dC of state sl * 4 + v % 4
        if (writer && tw + k < live)
          o.bc_lines[((((long long)cbl * a.q.total + t0 + tw + k) * 2 + v / 4) * o.groups + grp) * S + sl * 4 + v % 4] =
              acc[k][j];
      }
  }
}

// dS0 of sequences without tokens: what comes from the right passes.
__global__ void __launch_bounds__(256) kda_scan_empty_bwd_kernel(const Seqs q, const float* dS, float* dS0,
                                                                 long long row) {
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
// Channel blocks: enough CTAs for about eight rounds of two an SM; fewer blocks
// mean fewer lines of dB and dC.
inline BwdPlan bwd_plan(long long tokens, int d, int groups) {
  BwdPlan p;
  p.tiles = (tokens + kTokens - 1) / kTokens;
  const int all = (d / groups + kSlab - 1) / kSlab;  // slabs a group
  const long long want = 148 * 16;
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
  if (o.dS0 && (a.q.cu || tokens == 0)) {
    const int grid = a.q.num < 1024 ? a.q.num : 1024;
    kda_scan_empty_bwd_kernel<<<grid, 256, 0, st>>>(a.q, a.dS, o.dS0, row);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (tokens > 0) {
    a.ncb = channel_blocks(a.d, groups, S);
    a.blocks_per_group = a.ncb / groups;
    if ((e = launch_scan<T, S, kLocalBwd>(a, st)) != cudaSuccess) return e;
    if ((e = launch_carry(a, S, true, st)) != cudaSuccess) return e;
    a.ncb = p.blocks_per_group * groups;
    a.blocks_per_group = p.blocks_per_group;
    static PerDeviceOnce once;
    e = run_once_per_device(once, [] {
      return cudaFuncSetAttribute(kda_selective_scan_bwd_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)sizeof(BwdSmem<S>));
    });
    if (e != cudaSuccess) return e;
    const long long grid = p.tiles * a.ncb;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kda_selective_scan_bwd_kernel<T, S><<<(unsigned)grid, kWarps * 32, sizeof(BwdSmem<S>), st>>>(a, o);
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

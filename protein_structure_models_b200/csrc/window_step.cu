// window_step.cu -- window attention with sinks for single tokens and short
// chunks of new tokens against a long cache (bfloat16, forward).
//
// Bound by reading the visible keys and values once.  There are few rows, so the
// columns are what is split: a tile of 16 rows belongs to a cluster of 1 to 8
// CTAs of 4 warps, and each warp walks every (4 x CTAs)-th tile of 16 columns
// with a ring of its own (four tiles in flight, no barrier in the loop), keeping
// the running maximum m, the sum l and O of window_mma.cu.  The partial results
// meet in shared memory, across the cluster by distributed shared memory, and
// are joined in a fixed order as sum_w exp(m_w - m) O_w: one launch, no workspace.
#include <cooperative_groups.h>
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

namespace cg = cooperative_groups;
constexpr int kWarps = 4;
constexpr int kStages = 4;
constexpr int kCols = 16;

template <int DP>
__global__ void __launch_bounds__(kWarps * 32) win_step_kernel(const WinArgs a, int nsplit) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int LD = Tile<DP>::ld, EL = kCols * LD;       // one tile of one tensor
  constexpr int OL = DP + 4;                              // row of partial sums
  __shared__ float wm[kWarps][16], wl[kWarps][16], wf[kWarps][16], cm[16], cl[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  bf16* Qs = reinterpret_cast<bf16*>(smem);
  bf16* ring = Qs + 16 * LD + warp * kStages * 2 * EL;
  const int F = a.Nq * a.G, tiles = (F + 15) / 16;
  const int split = blockIdx.x % nsplit, job = blockIdx.x / nsplit;
  const int tile = job % tiles, bh = job / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * 16, f1 = min(F, f0 + 16), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  const int W = kWarps * nsplit, first = split * kWarps + warp, all = (c.n + kCols - 1) / kCols;
  const int ntile = all > first ? (all - first + W - 1) / W : 0;
  load_tile<DP>(Qs, q, 16, threadIdx.x, kWarps * 32, [&](int r) -> const bf16* {
    const int f = f0 + r, i = f / a.G;
    return f < f1 && win_alive(a, b, q0 + i) ? q.p + i * q.sn + (f - i * a.G) * q.sh : nullptr;
  });
  auto load = [&](int t) -> uint32_t {                    // returns the tile's valid columns
    uint32_t bits = 0u;
    if (t < ntile) {
      const int u = (first + t * W) * kCols + (lane & 15);
      const bool on = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0);
      bits = __ballot_sync(0xffffffffu, on) & 0xffffu;
      bf16* st = ring + (t % kStages) * 2 * EL;
      const int u0 = (first + t * W) * kCols;
      auto at = [&](const Src& s) {
        return [&, bits, u0](int r) -> const bf16* { return (bits >> r) & 1u ? s.p + c.key(u0 + r) * s.sn : nullptr; };
      };
      load_tile<DP>(st, k, kCols, lane, 32, at(k));
      load_tile<DP>(st + EL, v, kCols, lane, 32, at(v));
    }
    cp_async_commit();
    return bits;
  };
  uint32_t bits[kStages];
#pragma unroll
  for (int t = 0; t < kStages - 1; ++t) bits[t] = load(t);
  WinRow row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + (lane >> 2) + 8 * i, p = q0 + f / a.G;
    row[i] = win_row(a, c, p, f < f1 && win_alive(a, b, p));
  }
  const Reach rc = reach(a, c, q0, f0, f1);
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  float acc[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  cp_wait<0>();                                           // Q (and the first tiles)
  __syncthreads();
  uint32_t qf[DP / 16][4];
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) ldsm4(qf[kk], a_addr<DP>(smem_u32(Qs), 0, 16 * kk, lane));
  for (int t0 = 0; t0 < ntile; t0 += kStages) {
#pragma unroll
    for (int j = 0; j < kStages; ++j) {
      const int t = t0 + j;
      if (t >= ntile) break;
      bits[(j + kStages - 1) % kStages] = load(t + kStages - 1);
      cp_wait<kStages - 1>();
      __syncwarp();
      const int u0 = (first + t * W) * kCols;
      const uint32_t wg = bits[j];
      if (wg != 0u && rc.any(u0)) {
        const uint32_t ks = smem_u32(ring + j * 2 * EL), vs = ks + 2 * EL;
        float s[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          if (kk >= kd) break;
          uint32_t bf[4];
          ldsm4(bf, b_addr<DP>(ks, 0, 16 * kk, lane));
          mma(s[0], qf[kk], bf[0], bf[1]);
          mma(s[1], qf[kk], bf[2], bf[3]);
        }
        if (wg != 0xffffu || !rc.all(u0)) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int u = 8 * h + col2 + (e & 1);
              if (!((wg >> u) & 1u) || !row[e >> 1].sees(u0 + u)) s[h][e] = -INFINITY;
            }
        }
        float mb[2], mx[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
          const float mn = fmaxf(m[i], mx[i]);
          mb[i] = mn == -INFINITY ? 0.f : mn * sc;
          const float f = ex2_approx(m[i] * sc - mb[i]);
          m[i] = mn;
          l[i] *= f;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            acc[n][2 * i] *= f;
            acc[n][2 * i + 1] *= f;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[h][e] = ex2_approx(fmaf(s[h][e], sc, -mb[e >> 1]));
            l[e >> 1] += s[h][e];
          }
        const uint32_t pf[4] = {pack(s[0][0], s[0][1]), pack(s[0][2], s[0][3]), pack(s[1][0], s[1][1]), pack(s[1][2], s[1][3])};
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          if (n >= kv) break;
          uint32_t bf[4];
          ldsm4t(bf, bt_addr<DP>(vs, 0, 16 * n, lane));
          mma(acc[2 * n], pf, bf[0], bf[1]);
          mma(acc[2 * n + 1], pf, bf[2], bf[3]);
        }
      }
      __syncwarp();
    }
  }
  cp_wait<0>();
  // the warps' maxima and sums, then O_w exp(m_w - m) of the CTA in the ring's memory
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if ((lane & 3) == 0) {
      wm[warp][(lane >> 2) + 8 * i] = m[i];
      wl[warp][(lane >> 2) + 8 * i] = l[i];
    }
  }
  __syncthreads();
  float* Po = reinterpret_cast<float*>(Qs + 16 * LD);     // [warp][16][OL], then [16][OL] of the CTA in place of warp 0's
  if (threadIdx.x < 16) {
    const int r = threadIdx.x;
    float x = -INFINITY, y = 0.f;
    for (int w = 0; w < kWarps; ++w) x = fmaxf(x, wm[w][r]);
    for (int w = 0; w < kWarps; ++w) {
      wf[w][r] = wm[w][r] == -INFINITY ? 0.f : ex2_approx((wm[w][r] - x) * sc);
      y = fmaf(wl[w][r], wf[w][r], y);
    }
    cm[r] = x;
    cl[r] = y;
  }
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(Po + (warp * 16 + (lane >> 2) + 8 * i) * OL + 8 * n + col2) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
  __syncthreads();
  const int rows = f1 - f0;
  for (int e = threadIdx.x; e < rows * DP; e += kWarps * 32) {
    const int r = e / DP, d = e % DP;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x = fmaf(Po[(w * 16 + r) * OL + d], wf[w][r], x);
    Po[r * OL + d] = x;
  }
  cg::cluster_group cl_ = cg::this_cluster();
  if (nsplit > 1) cl_.sync();
  else __syncthreads();
  // rows split, split + nsplit, ... of the cluster's results
  const bool pair = (a.Dv & 1) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 3) == 0;
  for (int r = split; r < rows; r += nsplit) {
    float x = -INFINITY;
    for (int s = 0; s < nsplit; ++s) x = fmaxf(x, *cl_.map_shared_rank(&cm[r], s));
    float den = 0.f;
    for (int s = 0; s < nsplit; ++s) {
      const float y = *cl_.map_shared_rank(&cm[r], s);
      den += y == -INFINITY ? 0.f : *cl_.map_shared_rank(&cl[r], s) * ex2_approx((y - x) * sc);
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    const int f = f0 + r, qi = f / a.G, h = hkv * a.G + (f - qi * a.G);
    bf16* o = static_cast<bf16*>(a.out) + (((long long)b * a.Nq + qi) * a.H + h) * a.Dv;
    for (int d = 2 * threadIdx.x; d < a.Dv; d += 2 * kWarps * 32) {
      float y0 = 0.f, y1 = 0.f;
      for (int s = 0; s < nsplit; ++s) {
        const float ms = *cl_.map_shared_rank(&cm[r], s);
        if (ms == -INFINITY) continue;
        const float2 p = *reinterpret_cast<const float2*>(cl_.map_shared_rank(&Po[r * OL + d], s));
        const float g = ex2_approx((ms - x) * sc);
        y0 = fmaf(p.x, g, y0);
        y1 = fmaf(p.y, g, y1);
      }
      y0 = den > 0.f ? y0 * inv : 0.f;
      y1 = den > 0.f ? y1 * inv : 0.f;
      if (pair) {
        *reinterpret_cast<uint32_t*>(o + d) = pack(y0, y1);
      } else {
        o[d] = __float2bfloat16_rn(y0);
        if (d + 1 < a.Dv) o[d + 1] = __float2bfloat16_rn(y1);
      }
    }
    if (a.lse != nullptr && threadIdx.x == 0)
      a.lse[((long long)b * a.H + h) * a.Nq + qi] = den > 0.f ? fmaf(x, a.scale, logf(den)) : -INFINITY;
  }
  if (nsplit > 1) cl_.sync();                             // no CTA leaves while another reads its shared memory
}

template <int DP>
cudaError_t step(const WinArgs& a, int nsplit, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(&win_step_kernel<DP>);
  const cudaError_t e = allow_max_smem(fn);
  if (e != cudaSuccess) return e;
  const size_t ring = (size_t)kWarps * kStages * 2 * kCols * Tile<DP>::ld * sizeof(bf16), sums = (size_t)kWarps * 16 * (DP + 4) * sizeof(float);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * ((a.Nq * a.G + 15) / 16) * nsplit));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = 16 * Tile<DP>::ld * sizeof(bf16) + (ring > sums ? ring : sums);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)nsplit, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, win_step_kernel<DP>, a, nsplit);
}

}  // namespace

cudaError_t launch_win_step(const WinArgs& a, cudaStream_t s) {
  // CTAs of a cluster: enough for two CTAs an SM, as long as each warp has two tiles of columns.
  const long long jobs = (long long)a.B * a.Hkv * ((a.Nq * a.G + 15) / 16);
  const long long cols = (long long)a.left + a.Nq + a.right + a.sinks, n = cols < a.Nk ? cols : a.Nk;
  int nsplit = 1;
  while (nsplit < 8 && jobs * nsplit < 148 * 2 && n > (long long)2 * nsplit * kWarps * kCols) nsplit *= 2;
  const int w = a.D > a.Dv ? a.D : a.Dv;
  return w <= 16 ? step<16>(a, nsplit, s) : (w <= 32 ? step<32>(a, nsplit, s) : (w <= 64 ? step<64>(a, nsplit, s) : step<128>(a, nsplit, s)));
}

}  // namespace fipa

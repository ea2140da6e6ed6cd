// window_step.cu -- window attention with sinks for single tokens and short
// chunks of new tokens against a long cache (bfloat16, forward).
//
// Bound by reading the visible keys and values once.  There are few rows, so the
// columns are what is split: a tile of 16 rows belongs to a cluster of 1 to 8
// CTAs of 4 warps, and each warp walks every (4 x CTAs)-th tile of 16 columns,
// keeping the running maximum m, the sum l and O of window_mma.cu.
//
// Keys and values go from memory to the operand registers of the matrix
// instructions without shared memory in between.  A sum over channels may take
// them in any order: with lane 4 g + c reading channels 8 c .. 8 c + 7 of key g
// in one 16-byte load, its words are the operand's pairs if Q is read with the
// same order.  Values pair up two keys: lane 4 g + c reads DP / 8 neighbouring
// channels of keys 2c, 2c + 1, 2c + 8, 2c + 9, a byte permutation pairs them,
// and column g of the product's j-th tile is channel DP / 8 g + j.  (A ring of
// tiles in shared memory took three times the instructions a tile and 25 us at
// 64 x 1028 keys of 4 x 64 channels, this way 21.6, 2.7 TB/s of what is seen.)
//
// The partial results meet in shared memory, across the cluster by distributed
// shared memory, and are joined in a fixed order as sum_w exp(m_w - m) O_w: one
// launch, no workspace.
#include <cooperative_groups.h>
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

namespace cg = cooperative_groups;
constexpr int kWarps = 4;
constexpr int kCols = 16;

// N words (2 N channels) of a row from channel d0 on; channels at or beyond the width are 0.
template <int N, bool VEC>
__device__ __forceinline__ void words(uint32_t (&w)[N], const bf16* p, int d0, int width, bool on) {
  if (VEC) {                                 // the width is a multiple of 8, and so is what a load covers or divides
    on = on && d0 < width;
    if (N >= 4) {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (on && d0 + 8 * k < width) x = __ldg(reinterpret_cast<const uint4*>(p + d0) + k);
        w[4 * k % N] = x.x; w[(4 * k + 1) % N] = x.y; w[(4 * k + 2) % N] = x.z; w[(4 * k + 3) % N] = x.w;
      }
    } else if (N == 2) {
      uint2 x = make_uint2(0u, 0u);
      if (on) x = __ldg(reinterpret_cast<const uint2*>(p + d0));
      w[0] = x.x; w[1 % N] = x.y;
    } else {
      w[0] = on ? __ldg(reinterpret_cast<const uint32_t*>(p + d0)) : 0u;
    }
  } else {
    const uint16_t* s = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int d = d0 + 2 * k;
      const uint32_t lo = on && d < width ? s[d] : 0u, hi = on && d + 1 < width ? s[d + 1] : 0u;
      w[k] = lo | hi << 16;
    }
  }
}

// VEC: every load of q, k and v is on a 16-byte boundary.  The slow loads are
// an instantiation of their own: beside the fast ones they would fill the instruction cache.
template <int DP, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, DP <= 16 ? 5 : (DP <= 64 ? 4 : 2)) win_step_kernel(const WinArgs a, int nsplit) {
  extern __shared__ __align__(16) float Po[];             // [warp][16][OL], then [16][OL] of the CTA in place of warp 0's
  constexpr int OL = DP + 4;                              // row of partial sums
  __shared__ float wm[kWarps][16], wl[kWarps][16], wf[kWarps][16], cm[16], cl[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c4 = lane & 3;
  const int F = a.Nq * a.G, tiles = (F + 15) / 16;
  const int split = blockIdx.x % nsplit, job = blockIdx.x / nsplit;
  const int tile = job % tiles, bh = job / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * 16, f1 = min(F, f0 + 16), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  const int W = kWarps * nsplit, first = split * kWarps + warp, all = (c.n + kCols - 1) / kCols;
  const int ntile = all > first ? (all - first + W - 1) / W : 0;
  constexpr int KW = DP / 8 < 4 ? DP / 8 : 4, KC = DP / (8 * KW);     // words of a key load, loads of a key
  constexpr int VW = DP / 16;                                          // words of a value load
  bool alive[2];
  WinRow row[2];
  uint32_t qf[KC][2][KW];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + g + 8 * i, qi = f / a.G, p = q0 + qi;
    alive[i] = f < f1 && win_alive(a, b, p);
    row[i] = win_row(a, c, p, alive[i]);
#pragma unroll
    for (int x = 0; x < KC; ++x)
      words<KW, VEC>(qf[x][i], alive[i] ? q.p + qi * q.sn + (f - qi * a.G) * q.sh : q.p, 8 * KW * x + 2 * KW * c4, a.D, alive[i]);
  }
  const Reach rc = reach(a, c, q0, f0, f1);
  float acc[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  constexpr int AHEAD = DP > 32 ? 1 : 2;                  // tiles in registers
  uint32_t kw[AHEAD][KC][2][KW], vw[AHEAD][4][VW];
  // This lane's offsets in a tile of neighbouring keys; tiles that end, are
  // masked or hold the seam between sinks and window are loaded key by key.
  const long long ko = g * k.sn + 2 * KW * c4, vo = 2 * c4 * v.sn + 2 * VW * g;
  const bool kin = 2 * KW * c4 < a.D, vin = 2 * VW * g < a.Dv;
  auto valid = [&](int t) -> uint32_t {                   // the tile's valid columns
    if (t >= ntile) return 0u;
    const int u0 = (first + t * W) * kCols;
    if (a.mask == nullptr) return u0 + kCols <= c.n ? 0xffffu : (1u << (c.n - u0)) - 1u;
    const int u = u0 + (lane & 15);
    return __ballot_sync(0xffffffffu, u < c.n && a.mask[(long long)b * a.Nk + c.key(u)] != 0) & 0xffffu;
  };
  auto plain = [&](int u0, uint32_t bits) { return VEC && bits == 0xffffu && (u0 >= c.s || u0 + kCols <= c.s); };
  auto load_k = [&](uint32_t (&kw)[KC][2][KW], int t, uint32_t bits) {
    const int u0 = (first + t * W) * kCols;
    if (plain(u0, bits)) {
      const bf16* p = k.p + c.key(u0) * k.sn + ko;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < KC; ++x) words<KW, true>(kw[x][h], p + 8 * h * k.sn + 8 * KW * x, 0, a.D - 8 * KW * x - 2 * KW * c4, kin);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool on = (bits >> (8 * h + g)) & 1u;
        const bf16* p = on ? k.p + c.key(u0 + 8 * h + g) * k.sn : k.p;
#pragma unroll
        for (int x = 0; x < KC; ++x) words<KW, VEC>(kw[x][h], p, 8 * KW * x + 2 * KW * c4, a.D, on);
      }
    }
  };
  auto load_v = [&](uint32_t (&vw)[4][VW], int t, uint32_t bits) {
    const int u0 = (first + t * W) * kCols;
    if (plain(u0, bits)) {
      const bf16* p = v.p + c.key(u0) * v.sn + vo;
#pragma unroll
      for (int h = 0; h < 4; ++h) words<VW, true>(vw[h], p + ((h & 1) + 8 * (h >> 1)) * v.sn, 0, a.Dv - 2 * VW * g, vin);
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int u = 2 * c4 + (h & 1) + 8 * (h >> 1);
        const bool on = (bits >> u) & 1u;
        words<VW, VEC>(vw[h], on ? v.p + c.key(u0 + u) * v.sn : v.p, 2 * VW * g, a.Dv, on);
      }
    }
  };
  auto tile_of = [&](uint32_t (&kw)[KC][2][KW], uint32_t (&vw)[4][VW], uint32_t& now, int t) {
    const int u0 = (first + t * W) * kCols;
    const uint32_t next = valid(t + AHEAD);
    const bool some = now != 0u && rc.any(u0);
    float s[2][4];
    if (some) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
#pragma unroll
        for (int x = 0; x < KC; ++x)
#pragma unroll
          for (int w = 0; w < KW; w += 2) {
            const uint32_t af[4] = {qf[x][0][w], qf[x][1][w], qf[x][0][w + 1], qf[x][1][w + 1]};
            mma(s[h], af, kw[x][h][w], kw[x][h][w + 1]);
          }
      }
    }
    load_k(kw, t + AHEAD, next);
    if (some) {
      if (now != 0xffffu || !rc.all(u0)) {
        const uint32_t on[2] = {now & row[0].sees(u0), now & row[1].sees(u0)};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][e] = (on[e >> 1] >> (8 * h + 2 * c4 + (e & 1))) & 1u ? s[h][e] : -INFINITY;
      }
      float mb[2], mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      // m follows the true maximum only when it would be left behind by 2^8: the
      // sums keep their relative precision, and most tiles rescale nothing
      if (__any_sync(0xffffffffu, (mx[0] - m[0]) * sc > kWinLag || (mx[1] - m[1]) * sc > kWinLag)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], mx[i]), f = ex2_approx(mn == -INFINITY ? -INFINITY : (m[i] - mn) * sc);
          m[i] = mn;
          l[i] *= f;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            acc[n][2 * i] *= f;
            acc[n][2 * i + 1] *= f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) mb[i] = m[i] == -INFINITY ? 0.f : m[i] * sc;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[h][e] = ex2_approx(fmaf(s[h][e], sc, -mb[e >> 1]));
          l[e >> 1] += s[h][e];
        }
      const uint32_t pf[4] = {pack(s[0][0], s[0][1]), pack(s[0][2], s[0][3]), pack(s[1][0], s[1][1]), pack(s[1][2], s[1][3])};
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        mma(acc[2 * w], pf, __byte_perm(vw[0][w], vw[1][w], 0x5410), __byte_perm(vw[2][w], vw[3][w], 0x5410));
        mma(acc[2 * w + 1], pf, __byte_perm(vw[0][w], vw[1][w], 0x7632), __byte_perm(vw[2][w], vw[3][w], 0x7632));
      }
      if (a.fine) {
        const uint32_t lo[4] = {rest(pf[0], s[0][0], s[0][1]), rest(pf[1], s[0][2], s[0][3]), rest(pf[2], s[1][0], s[1][1]), rest(pf[3], s[1][2], s[1][3])};
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          mma(acc[2 * w], lo, __byte_perm(vw[0][w], vw[1][w], 0x5410), __byte_perm(vw[2][w], vw[3][w], 0x5410));
          mma(acc[2 * w + 1], lo, __byte_perm(vw[0][w], vw[1][w], 0x7632), __byte_perm(vw[2][w], vw[3][w], 0x7632));
        }
      }
    }
    load_v(vw, t + AHEAD, next);
    now = next;
  };
  uint32_t bits[AHEAD];
#pragma unroll
  for (int x = 0; x < AHEAD; ++x) {
    bits[x] = valid(x);
    load_k(kw[x], x, bits[x]);
    load_v(vw[x], x, bits[x]);
  }
  for (int t = 0; t < ntile; t += AHEAD) {
#pragma unroll
    for (int x = 0; x < AHEAD; ++x)
      if (t + x < ntile) tile_of(kw[x], vw[x], bits[x], t + x);
  }
  // the warps' maxima and sums, then O of the CTA
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (c4 == 0) {
      wm[warp][g + 8 * i] = m[i];
      wl[warp][g + 8 * i] = alive[i] ? l[i] : 0.f;       // tiles of which every column is seen are not masked row by row
    }
  }
  __syncthreads();
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
    for (int e = 0; e < 4; ++e)
      Po[(warp * 16 + g + 8 * (e >> 1)) * OL + DP / 8 * (2 * c4 + (e & 1)) + n] = acc[n][e];
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
        const float w = ex2_approx((ms - x) * sc);
        y0 = fmaf(p.x, w, y0);
        y1 = fmaf(p.y, w, y1);
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

template <int DP, bool VEC>
cudaError_t step(const WinArgs& a, int nsplit, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(&win_step_kernel<DP, VEC>);
  const cudaError_t e = allow_max_smem(fn);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * ((a.Nq * a.G + 15) / 16) * nsplit));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = (size_t)kWarps * 16 * (DP + 4) * sizeof(float);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)nsplit, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, win_step_kernel<DP, VEC>, a, nsplit);
}

template <int DP>
cudaError_t step(const WinArgs& a, int nsplit, cudaStream_t s) {
  return win_vec(a) ? step<DP, true>(a, nsplit, s) : step<DP, false>(a, nsplit, s);
}

}  // namespace

cudaError_t launch_win_step(const WinArgs& a, cudaStream_t s) {
  const int w = a.D > a.Dv ? a.D : a.Dv;
  // CTAs of a cluster: as many as are resident at once (by the registers of each
  // width), as a CTA costs about 5 us of latency whatever it reads: 96 x 4 heads
  // of 64 x 68 keys take 11 us with one, 55 us with eight; 1 x 8 heads of
  // 32 x 260 keys 9.7 us with one, 6.7 us with eight.
  const long long jobs = (long long)a.B * a.Hkv * ((a.Nq * a.G + 15) / 16), slots = 148 * (w <= 16 ? 5 : (w <= 64 ? 4 : 2));
  const long long cols = (long long)a.left + a.Nq + a.right + a.sinks, n = cols < a.Nk ? cols : a.Nk;
  int nsplit = 1;
  while (nsplit < 8 && jobs * nsplit * 2 <= slots && n > (long long)nsplit * kWarps * kCols / 2) nsplit *= 2;
  return w <= 16 ? step<16>(a, nsplit, s) : (w <= 32 ? step<32>(a, nsplit, s) : (w <= 64 ? step<64>(a, nsplit, s) : step<128>(a, nsplit, s)));
}

}  // namespace fipa

// window_mma.cu -- window attention with sinks on bfloat16 tensors, forward and
// backward, with warp-level matrix instructions (m16n8k16, float32 sums).
//
// The mathematics, the row and column numbering and the visibility rule are
// those of window.h:
//   forward   m the running row maximum, l the running sum of exp(s - m), O that of
//             exp(s - m) v, both scaled by exp(m_old - m_new) when m grows;
//             out = O / l, lse = m + ln l
//   backward  p = exp(s - lse), ds = p (dO.v - delta) with delta = dO.out;
//             dq = scale sum ds k (row side), dv = sum p dO, dk = scale sum ds q (key
//             side).  Each side recomputes p, so that every sum has one owner and a
//             fixed order.
//  A warp owns 16 rows (forward, dq) or
// 16 keys (dk, dv) and keeps its scores, probabilities and sums in registers:
// the accumulator layout of one product is the operand layout of the next, so
// nothing of the softmax touches shared memory.  Because a warp covers only 16
// positions it walks just the columns that they see: columns are taken 16 at a
// time, skipped when no row of the warp sees them, and tested element by element
// only at the edges of the window, which is what makes short windows cheap.
// Tiles of 64 columns arrive by 16-byte asynchronous copies, the next one while
// the present one is in use; rows in shared memory are padded by 16 bytes, so
// that eight neighbouring rows start in different banks.
//
// Probabilities and ds go into the second product as bfloat16 (half a step is
// 2^-8 of each, the tensors' own rounding); l, m, delta and all sums are float32.
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

constexpr int T = kWinTile;            // rows and columns of a tile
constexpr int kThreads = 128;              // 4 warps x 16 rows
template <int DP>
constexpr int kElems = T * Tile<DP>::ld;

// Whether columns u0 .. u0+63 exist and are not masked: two words.
__device__ __forceinline__ void column_bits(uint32_t* bits, const WinArgs& a, int b, const WinCols& c, int u0) {
  if (threadIdx.x < T) {
    const int u = u0 + threadIdx.x;
    const bool on = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0);
    const uint32_t w = __ballot_sync(0xffffffffu, on);
    if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = w;
  }
}

// Rows f0 .. f0+63 (those below fh) of the queries and of dO, and columns u0 .. u0+63 of keys and values.
template <int DP>
__device__ __forceinline__ void load_queries(bf16* Qs, bf16* Os, const WinArgs& a, int b, int q0, const Src& q, const Src& g, int f0, int fh) {
  constexpr int step = kThreads / (DP / 8);
  const int first = threadIdx.x / (DP / 8);
  copy_padded<DP>(Qs, Os, a.D, a.Dv, walk_queries(a, q, g, min(f0 + first, fh - 1), step), first, step, T, fh - f0,
                  [&](int i) { return win_alive(a, b, q0 + i); });
}
template <int DP>
__device__ __forceinline__ void load_keys(bf16* Ks, bf16* Vs, const WinArgs& a, int b, const Src& k, const Src& v, const WinCols& c, int u0) {
  auto valid = [&](int j) { return a.mask == nullptr || a.mask[(long long)b * a.Nk + j] != 0; };
  constexpr int step = kThreads / (DP / 8);
  int first = threadIdx.x / (DP / 8);
  const int ns = min(max(c.s - u0, 0), T);                  // sinks first, then the window; a tile may hold the seam
  if (ns > 0) copy_padded<DP>(Ks, Vs, a.D, a.Dv, walk_keys(k, v, min(u0 + first, a.Nk - 1), step), first, step, ns, ns, valid);
  while (first < ns) first += step;
  if (first < T) copy_padded<DP>(Ks, Vs, a.D, a.Dv, walk_keys(k, v, min(c.key(u0 + first), a.Nk - 1), step), first, step, T, c.n - u0, valid);
}

template <int DP>
__global__ void __launch_bounds__(kThreads) win_fwd_mma_kernel(const WinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  bf16* Qs = reinterpret_cast<bf16*>(smem);
  bf16* Ks = Qs + kElems<DP>;                     // two stages each
  bf16* Vs = Ks + 2 * kElems<DP>;
  __shared__ uint32_t bits[2][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  const int F = a.Nq * a.G, tiles = (F + T - 1) / T;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * T, f1 = min(F, f0 + T), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  bool alive[2];
  WinRow row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, p = q0 + f / a.G;
    alive[i] = f < f1 && win_alive(a, b, p);
    row[i] = win_row(a, c, p, alive[i]);
  }
  const int ntile = __syncthreads_or(alive[0] || alive[1]) ? (c.n + T - 1) / T : 0;
  const Reach rc = reach(a, c, q0, f0 + 16 * warp, f1);
  auto load = [&](int t) {
    const int st = t & 1, u0 = t * T;
    load_keys<DP>(Ks + st * kElems<DP>, Vs + st * kElems<DP>, a, b, k, v, c, u0);
    column_bits(bits[st], a, b, c, u0);
    cp_async_commit();
  };
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  float acc[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  uint32_t qf[DP / 16][4];
  const float sc = a.scale * kLog2e;
  if (ntile > 0) {
    load_tile<DP>(Qs, q, T, threadIdx.x, kThreads, [&](int r) -> const bf16* {
      const int f = f0 + r, i = f / a.G;
      return f < f1 && win_alive(a, b, q0 + i) ? q.p + i * q.sn + (f - i * a.G) * q.sh : nullptr;
    });
    load(0);
  }
  for (int t = 0; t < ntile; ++t) {
    const int st = t & 1, u0 = t * T;
    if (t + 1 < ntile) {
      load(t + 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    if (t == 0) {
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) ldsm4(qf[kk], a_addr<DP>(smem_u32(Qs), 16 * warp, 16 * kk, lane));
    }
    const uint32_t ks = smem_u32(Ks + st * kElems<DP>), vs = smem_u32(Vs + st * kElems<DP>);
    const uint32_t w[2] = {bits[st][0], bits[st][1]};
    float s[8][4];
    bool on[4];
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t wg = (w[g >> 1] >> ((g & 1) * 16)) & 0xffffu;
      on[g] = wg != 0u && rc.any(u0 + 16 * g);
      if (!on[g]) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[2 * g + h][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        if (kk >= kd) break;
        uint32_t bf[4];
        ldsm4(bf, b_addr<DP>(ks, 16 * g, 16 * kk, lane));
        mma(s[2 * g], qf[kk], bf[0], bf[1]);
        mma(s[2 * g + 1], qf[kk], bf[2], bf[3]);
      }
      if (wg != 0xffffu || !rc.all(u0 + 16 * g)) {
        const uint32_t on[2] = {wg & row[0].sees(u0 + 16 * g), wg & row[1].sees(u0 + 16 * g)};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[2 * g + h][e] = (on[e >> 1] >> (8 * h + col2 + (e & 1))) & 1u ? s[2 * g + h][e] : -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], s[2 * g + h][e]);
    }
    if (on[0] || on[1] || on[2] || on[3]) {
      float mb[2], sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
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
      for (int g = 0; g < 4; ++g) {
        if (!on[g]) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[2 * g + h][e] = ex2_approx(fmaf(s[2 * g + h][e], sc, -mb[e >> 1]));
            sum[e >> 1] += s[2 * g + h][e];
          }
        const uint32_t pf[4] = {pack(s[2 * g][0], s[2 * g][1]), pack(s[2 * g][2], s[2 * g][3]),
                                pack(s[2 * g + 1][0], s[2 * g + 1][1]), pack(s[2 * g + 1][2], s[2 * g + 1][3])};
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          if (n >= kv) break;
          uint32_t bf[4];
          ldsm4t(bf, bt_addr<DP>(vs, 16 * g, 16 * n, lane));
          mma(acc[2 * n], pf, bf[0], bf[1]);
          mma(acc[2 * n + 1], pf, bf[2], bf[3]);
        }
        if (a.fine) add_rest<DP>(acc, pf, s[2 * g], s[2 * g + 1], vs, 16 * g, kv, lane);
      }
      l[0] += sum[0];
      l[1] += sum[1];
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i;
    if (f >= f1) continue;
    const int qi = f / a.G, h = hkv * a.G + (f - qi * a.G);
    const bool some = alive[i] && l[i] != 0.f;
    const float inv = some ? 1.f / l[i] : 0.f;
    bf16* o = static_cast<bf16*>(a.out) + (((long long)b * a.Nq + qi) * a.H + h) * a.Dv;
    const bool pair = (a.Dv & 1) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 3) == 0;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const int d = 8 * n + col2;
      const float x = some ? acc[n][2 * i] * inv : 0.f, y = some ? acc[n][2 * i + 1] * inv : 0.f;
      if (pair && d < a.Dv) {
        *reinterpret_cast<uint32_t*>(o + d) = pack(x, y);
      } else {
        if (d < a.Dv) o[d] = __float2bfloat16_rn(x);
        if (d + 1 < a.Dv) o[d + 1] = __float2bfloat16_rn(y);
      }
    }
    if (a.lse != nullptr && (lane & 3) == 0)
      a.lse[((long long)b * a.H + h) * a.Nq + qi] = some ? fmaf(m[i], a.scale, logf(l[i])) : -INFINITY;
  }
}

// delta = dO.out of a row tile, four neighbouring lanes a row (two passes of 32 rows); dead rows 0.
template <int DP>
__device__ __forceinline__ void row_delta(float* sdelta, const bf16* dOs, const WinArgs& a, const bf16* out, int b, int hkv, int q0,
                                          int f0, int f1) {
  for (int r = threadIdx.x >> 2; r < T; r += kThreads / 4) {
    const int f = f0 + r, i = f / a.G, h = hkv * a.G + (f - i * a.G);
    float x = 0.f;
    if (f < f1 && win_alive(a, b, q0 + i)) {
      const bf16* o = out + (((long long)b * a.Nq + i) * a.H + h) * a.Dv;
      if ((a.Dv & 7) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
        for (int d = (threadIdx.x & 3) * 8; d < a.Dv; d += 32) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(o + d));
          const uint4 g = *reinterpret_cast<const uint4*>(dOs + r * Tile<DP>::ld + d);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w}, gg[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x = fmaf(__uint_as_float(ww[e] << 16), __uint_as_float(gg[e] << 16), x);
            x = fmaf(__uint_as_float(ww[e] & 0xffff0000u), __uint_as_float(gg[e] & 0xffff0000u), x);
          }
        }
      } else {
        for (int d = threadIdx.x & 3; d < a.Dv; d += 4)
          x = fmaf(__bfloat162float(o[d]), __bfloat162float(dOs[r * Tile<DP>::ld + d]), x);
      }
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if ((threadIdx.x & 3) == 0) sdelta[r] = x;
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads) win_bwd_q_mma_kernel(const WinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  bf16* Qs = reinterpret_cast<bf16*>(smem);
  bf16* Os = Qs + kElems<DP>;
  bf16* Ks = Os + kElems<DP>;
  bf16* Vs = Ks + 2 * kElems<DP>;
  __shared__ uint32_t bits[2][2];
  __shared__ float sdelta[T];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  const int F = a.Nq * a.G, tiles = (F + T - 1) / T;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * T, f1 = min(F, f0 + T), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src g_ = source(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  bool alive[2];
  WinRow row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, p = q0 + f / a.G;
    alive[i] = f < f1 && win_alive(a, b, p);
    row[i] = win_row(a, c, p, alive[i]);
  }
  const int ntile = __syncthreads_or(alive[0] || alive[1]) ? (c.n + T - 1) / T : 0;
  const Reach rc = reach(a, c, q0, f0 + 16 * warp, f1);
  auto load = [&](int t) {
    const int st = t & 1, u0 = t * T;
    load_keys<DP>(Ks + st * kElems<DP>, Vs + st * kElems<DP>, a, b, k, v, c, u0);
    column_bits(bits[st], a, b, c, u0);
    cp_async_commit();
  };
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  float acc[DP / 8][4], avg[DP / 8][4], lse2[2] = {INFINITY, INFINITY}, del[2] = {0.f, 0.f}, eps[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = avg[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  if (ntile > 0) {
    load_queries<DP>(Qs, Os, a, b, q0, q, g_, f0, f1);
    load(0);
    cp_wait<0>();
    __syncthreads();
    row_delta<DP>(sdelta, Os, a, static_cast<const bf16*>(a.out), b, hkv, q0, f0, f1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * warp + (lane >> 2) + 8 * i, f = f0 + r, qi = f / a.G;
      del[i] = sdelta[r];
      if (alive[i]) {
        const float x = a.lse[((long long)b * a.H + hkv * a.G + (f - qi * a.G)) * a.Nq + qi];
        lse2[i] = x == -INFINITY ? INFINITY : x * kLog2e;     // a row that sees nothing: every p is 0
      }
    }
  }
  for (int t = 0; t < ntile; ++t) {
    const int st = t & 1, u0 = t * T;
    if (t + 1 < ntile) {
      load(t + 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    const uint32_t ks = smem_u32(Ks + st * kElems<DP>), vs = smem_u32(Vs + st * kElems<DP>);
    const uint32_t w[2] = {bits[st][0], bits[st][1]};
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t wg = (w[g >> 1] >> ((g & 1) * 16)) & 0xffffu;
      if (wg == 0u || !rc.any(u0 + 16 * g)) continue;
      float s[2][4], dp[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = dp[h][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t af[4], bf[4];
        if (kk < kd) {
          ldsm4(af, a_addr<DP>(smem_u32(Qs), 16 * warp, 16 * kk, lane));
          ldsm4(bf, b_addr<DP>(ks, 16 * g, 16 * kk, lane));
          mma(s[0], af, bf[0], bf[1]);
          mma(s[1], af, bf[2], bf[3]);
        }
        if (kk < kv) {
          ldsm4(af, a_addr<DP>(smem_u32(Os), 16 * warp, 16 * kk, lane));
          ldsm4(bf, b_addr<DP>(vs, 16 * g, 16 * kk, lane));
          mma(dp[0], af, bf[0], bf[1]);
          mma(dp[1], af, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = ex2_approx(fmaf(s[h][e], sc, -lse2[e >> 1]));
      if (wg != 0xffffu || !rc.all(u0 + 16 * g)) {
        const uint32_t on[2] = {wg & row[0].sees(u0 + 16 * g), wg & row[1].sees(u0 + 16 * g)};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[h][e] = (on[e >> 1] >> (8 * h + col2 + (e & 1))) & 1u ? s[h][e] : 0.f;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dp[h][e] = s[h][e] * (dp[h][e] - del[e >> 1]);
          eps[e >> 1] += dp[h][e];
        }
      const uint32_t pf[4] = {pack(s[0][0], s[0][1]), pack(s[0][2], s[0][3]), pack(s[1][0], s[1][1]), pack(s[1][2], s[1][3])};
      const uint32_t df[4] = {pack(dp[0][0], dp[0][1]), pack(dp[0][2], dp[0][3]), pack(dp[1][0], dp[1][1]), pack(dp[1][2], dp[1][3])};
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        if (n >= kd) break;
        uint32_t bf[4];
        ldsm4t(bf, bt_addr<DP>(ks, 16 * g, 16 * n, lane));
        mma(acc[2 * n], df, bf[0], bf[1]);
        mma(acc[2 * n + 1], df, bf[2], bf[3]);
        mma(avg[2 * n], pf, bf[0], bf[1]);
        mma(avg[2 * n + 1], pf, bf[2], bf[3]);
      }
      if (a.fine) add_rest<DP>(acc, df, dp[0], dp[1], ks, 16 * g, kd, lane);
    }
    __syncthreads();
  }
  take_back<DP>(acc, avg, eps);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, qi = f / a.G;
    if ((lane & 3) == 0 && f < f1) a.delta[((long long)b * a.H + hkv * a.G + (f - qi * a.G)) * a.Nq + qi] = del[i] + eps[i];
  }
  store_rows<DP>(acc, a.D, a.d_q, a.scale, lane, [&](int i, bool& keep) -> bf16* {
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, qi = f / a.G;
    keep = alive[i] && lse2[i] != INFINITY;
    return f < f1 ? static_cast<bf16*>(a.d_q) + (((long long)b * a.Nq + qi) * a.H + hkv * a.G + (f - qi * a.G)) * a.D : nullptr;
  });
}

// dk and dv.  SINK false: of one key tile over the rows of its window, a warp 16
// keys.  SINK true: of 16 keys that hold sinks, over one chunk of the rows beyond
// the window; the warps take every fourth 16 rows and are added in order.
template <int DP, bool SINK>
__global__ void __launch_bounds__(kThreads) win_bwd_k_mma_kernel(const WinArgs a) {
  constexpr int KR = SINK ? 16 : T;                     // keys of the CTA
  extern __shared__ __align__(16) uint8_t smem[];
  bf16* Ks = reinterpret_cast<bf16*>(smem);
  bf16* Vs = Ks + KR * Tile<DP>::ld;
  bf16* Qs = Vs + KR * Tile<DP>::ld;
  bf16* Os = Qs + 2 * kElems<DP>;
  __shared__ float slse[2][T], sdel[2][T];
  __shared__ int spos[2][T];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  const int per = SINK ? (a.sinks + 15) / 16 * a.nchunk : (a.Nk + T - 1) / T;
  const int job = blockIdx.x % per, bh = blockIdx.x / per, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int chunk = SINK ? job % a.nchunk : -1, q0 = win_q0(a, b);
  const int j0 = SINK ? job / a.nchunk * 16 : job * T, j1 = min(a.Nk, j0 + KR) - 1, wj = SINK ? 0 : 16 * warp;
  const bool split = !SINK && a.nchunk > 0 && j0 < a.sinks;
  const int pl = SINK ? a.sink_pos : max(0, j0 - a.right);
  const int ph = SINK || (j0 < a.sinks && !split) ? a.Nk - 1 : min(a.Nk - 1, split ? a.sink_pos - 1 : j1 + a.left);
  const int il = max(pl - q0, 0), ih = min(ph - q0, a.Nq - 1);
  int fl = il * a.G, fh = (ih + 1) * a.G;
  if (ih < il) fl = fh = 0;
  if (SINK) {
    fl = max(fl, chunk * a.chunk_tiles * T);
    fh = min(fh, (chunk + 1) * a.chunk_tiles * T);
  }
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src g_ = source(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  bool alive[2];
  int rlo[2], rhi[2];                                   // rows, counted from fl, that see this thread's keys
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = j0 + wj + (lane >> 2) + 8 * i;
    alive[i] = j <= j1 && win_alive(a, b, j);
    key_rows(a, q0, j, fl, fh, rlo[i], rhi[i]);
  }
  const int ka = j0 + wj, kb = min(ka + 15, j1);   // keys of the warp
  const int ntile = __syncthreads_or(alive[0] || alive[1]) && fh > fl ? (fh - fl + T - 1) / T : 0;
  float rl = 0.f, rd = 0.f;
  int rp = 0;
  auto load = [&](int t) {
    const int st = t & 1, f0 = fl + t * T;
    load_queries<DP>(Qs + st * kElems<DP>, Os + st * kElems<DP>, a, b, q0, q, g_, f0, fh);
    cp_async_commit();
    // a row's lse, delta and position wait in registers until the tile before is done
    if (threadIdx.x < T) {
      const int f = f0 + threadIdx.x, i = f / a.G;
      rl = -INFINITY;
      rd = 0.f;
      rp = q0 + i;
      if (f < fh && win_alive(a, b, rp)) {
        const long long o = ((long long)b * a.H + hkv * a.G + (f - i * a.G)) * a.Nq + i;
        rl = a.lse[o];
        rd = a.delta[o];
      }
    }
  };
  auto put = [&](int st) {
    if (threadIdx.x < T) {
      slse[st][threadIdx.x] = rl == -INFINITY ? INFINITY : rl * kLog2e;   // not there, or sees nothing: every p is 0
      sdel[st][threadIdx.x] = rd;
      spos[st][threadIdx.x] = rp;
    }
  };
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  if (ntile > 0) {
    auto keyed = [&](const Src& s) {
      return [&](int r) -> const bf16* { return j0 + r <= j1 && win_alive(a, b, j0 + r) ? s.p + (j0 + r) * s.sn : nullptr; };
    };
    load_tile<DP>(Ks, k, KR, threadIdx.x, kThreads, keyed(k));
    load_tile<DP>(Vs, v, KR, threadIdx.x, kThreads, keyed(v));
    load(0);
    put(0);
  }
  for (int t = 0; t < ntile; ++t) {
    const int st = t & 1;
    if (t + 1 < ntile) {
      load(t + 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    const uint32_t qs = smem_u32(Qs + st * kElems<DP>), os = smem_u32(Os + st * kElems<DP>);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (fl + t * T + 16 * g >= fh) break;
      if (SINK && g != warp) continue;
      const int pa = spos[st][16 * g], pb = spos[st][16 * g + 15];
      if (kb < ka || pb < ka - a.right || (pa > kb + a.left && ka >= a.sinks)) continue;
      uint32_t on[2] = {0xffffu, 0xffffu};
      if (pa < kb - a.right || pb > ka + a.left) {
#pragma unroll
        for (int i = 0; i < 2; ++i) on[i] = win_span(rlo[i] - t * T - 16 * g, rhi[i] - t * T - 16 * g);
      }
      float s[2][4], dp[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = dp[h][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t af[4], bf[4];
        if (kk < kd) {
          ldsm4(af, a_addr<DP>(smem_u32(Ks), wj, 16 * kk, lane));
          ldsm4(bf, b_addr<DP>(qs, 16 * g, 16 * kk, lane));
          mma(s[0], af, bf[0], bf[1]);
          mma(s[1], af, bf[2], bf[3]);
        }
        if (kk < kv) {
          ldsm4(af, a_addr<DP>(smem_u32(Vs), wj, 16 * kk, lane));
          ldsm4(bf, b_addr<DP>(os, 16 * g, 16 * kk, lane));
          mma(dp[0], af, bf[0], bf[1]);
          mma(dp[1], af, bf[2], bf[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * g + 8 * h + col2 + (e & 1), i = e >> 1;
          const float x = ex2_approx(fmaf(s[h][e], sc, -slse[st][r])), p = (on[i] >> (r - 16 * g)) & 1u ? x : 0.f;
          s[h][e] = p;
          dp[h][e] = p * (dp[h][e] - sdel[st][r]);
        }
      const uint32_t pf[4] = {pack(s[0][0], s[0][1]), pack(s[0][2], s[0][3]), pack(s[1][0], s[1][1]), pack(s[1][2], s[1][3])};
      const uint32_t df[4] = {pack(dp[0][0], dp[0][1]), pack(dp[0][2], dp[0][3]), pack(dp[1][0], dp[1][1]), pack(dp[1][2], dp[1][3])};
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t bf[4];
        if (n < kv) {
          ldsm4t(bf, bt_addr<DP>(os, 16 * g, 16 * n, lane));
          mma(dv[2 * n], pf, bf[0], bf[1]);
          mma(dv[2 * n + 1], pf, bf[2], bf[3]);
        }
        if (n < kd) {
          ldsm4t(bf, bt_addr<DP>(qs, 16 * g, 16 * n, lane));
          mma(dk[2 * n], df, bf[0], bf[1]);
          mma(dk[2 * n + 1], df, bf[2], bf[3]);
        }
      }
      if (a.fine) {
        add_rest<DP>(dv, pf, s[0], s[1], os, 16 * g, kv, lane);
        add_rest<DP>(dk, df, dp[0], dp[1], qs, 16 * g, kd, lane);
      }
    }
    if (t + 1 < ntile) put(st ^ 1);
    __syncthreads();
  }
  if (SINK) {
    // the warps' sums, in warp order, in the memory of the tiles
    constexpr int OL = 2 * DP + 4;
    float* red = reinterpret_cast<float*>(smem);
    for (int w = 0; w < 4; ++w) {
      if (warp == w) {
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* o = red + ((lane >> 2) + 8 * (e >> 1)) * OL + 8 * n + col2 + (e & 1);
            o[0] = dk[n][e] + (w == 0 ? 0.f : o[0]);
            o[DP] = dv[n][e] + (w == 0 ? 0.f : o[DP]);
          }
      }
      __syncthreads();
    }
    const int wd = a.D + a.Dv;
    for (int e = threadIdx.x; e < 16 * wd; e += kThreads) {
      const int r = e / wd, d = e - r * wd, j = j0 + r;
      if (j > j1 || j >= a.sinks) continue;
      const bool on = a.mask == nullptr || a.mask[(long long)b * a.Nk + j] != 0;
      a.part[(((long long)bh * (a.nchunk + 1) + chunk + 1) * a.sinks + j) * wd + d] = on ? red[r * OL + (d < a.D ? d : DP + d - a.D)] : 0.f;
    }
    return;
  }
  if (split) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + wj + (lane >> 2) + 8 * i;
      if (j > j1 || j >= a.sinks) continue;
      float* o = a.part + ((long long)bh * (a.nchunk + 1) * a.sinks + j) * (a.D + a.Dv);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 8 * n + col2 + e;
          if (d < a.D) o[d] = alive[i] ? dk[n][2 * i + e] : 0.f;
          if (d < a.Dv) o[a.D + d] = alive[i] ? dv[n][2 * i + e] : 0.f;
        }
    }
  }
  auto at = [&](void* base, int width, int i, bool& keep) -> bf16* {
    const int j = j0 + wj + (lane >> 2) + 8 * i;
    keep = alive[i];
    return j <= j1 && !(split && j < a.sinks) ? static_cast<bf16*>(base) + (((long long)b * a.Nk + j) * a.Hkv + hkv) * width : nullptr;
  };
  store_rows<DP>(dk, a.D, a.d_k, a.scale, lane, [&](int i, bool& keep) { return at(a.d_k, a.D, i, keep); });
  store_rows<DP>(dv, a.Dv, a.d_v, 1.f, lane, [&](int i, bool& keep) { return at(a.d_v, a.Dv, i, keep); });
}

__device__ __forceinline__ void stf(float* p, float x) { *p = x; }
__device__ __forceinline__ void stf(bf16* p, float x) { *p = __float2bfloat16_rn(x); }
// dk, dv of the sinks: the partial sums in chunk order, in 32 neighbouring stretches that are added in order.
template <typename E>
__global__ void __launch_bounds__(1024) win_sink_reduce_kernel(const WinArgs a) {
  __shared__ float red[32][32];
  const int w = a.D + a.Dv, bh = blockIdx.x / a.sinks, j = blockIdx.x - bh * a.sinks, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, d = blockIdx.y * 32 + lane, per = (a.nchunk + 32) / 32;
  float x = 0.f;
  if (d < w) {
    const float* p = a.part + ((long long)bh * (a.nchunk + 1) * a.sinks + j) * w + d;
    const int hi = min((part + 1) * per, a.nchunk + 1);
#pragma unroll 8
    for (int ch = part * per; ch < hi; ++ch) x += p[(long long)ch * a.sinks * w];
  }
  red[part][lane] = x;
  __syncthreads();
  if (part != 0 || d >= w) return;
  for (int k = 1; k < 32; ++k) x += red[k][lane];
  const long long r = ((long long)b * a.Nk + j) * a.Hkv + hkv;
  if (d < a.D) stf(static_cast<E*>(a.d_k) + r * a.D + d, x * a.scale);
  else stf(static_cast<E*>(a.d_v) + r * a.Dv + (d - a.D), x);
}

template <int DP>
cudaError_t fwd(const WinArgs& a, cudaStream_t s) {
  const long long grid = (long long)a.B * a.Hkv * (((long long)a.Nq * a.G + T - 1) / T);
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_fwd_mma_kernel<DP>));
  if (e != cudaSuccess) return e;
  win_fwd_mma_kernel<DP><<<(unsigned)grid, kThreads, 5 * kElems<DP> * sizeof(bf16), s>>>(a);
  return cudaGetLastError();
}

template <int DP>
cudaError_t bwd_q(const WinArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_bwd_q_mma_kernel<DP>));
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.B * a.Hkv * (((long long)a.Nq * a.G + T - 1) / T);
  win_bwd_q_mma_kernel<DP><<<(unsigned)grid, kThreads, 6 * kElems<DP> * sizeof(bf16), s>>>(a);
  return cudaGetLastError();
}
template <int DP, bool SINK>
cudaError_t bwd_k(const WinArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_bwd_k_mma_kernel<DP, SINK>));
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.B * a.Hkv * (SINK ? (long long)(a.sinks + 15) / 16 * a.nchunk : (a.Nk + T - 1) / T);
  const size_t smem = (size_t)(2 * (SINK ? 16 : T) + 4 * T) * Tile<DP>::ld * sizeof(bf16);
  win_bwd_k_mma_kernel<DP, SINK><<<(unsigned)grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
template <int DP>
cudaError_t bwd(const WinArgs& a, bool tc, cudaStream_t s) {
  cudaError_t e = tc ? launch_win_bwd_q_tc(a, s) : bwd_q<DP>(a, s);
  if (e == cudaSuccess) e = tc ? launch_win_bwd_k_tc(a, s) : bwd_k<DP, false>(a, s);
  if (e == cudaSuccess && a.nchunk > 0) e = bwd_k<DP, true>(a, s);
  if (e == cudaSuccess && a.nchunk > 0) e = launch_win_sink_reduce(a, 0, s);
  return e;
}
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether the outputs, which may be anywhere, are on 16-byte boundaries like the inputs.
bool vectors(const WinArgs& a, bool backward) {
  return on16(a.out) && (!backward || (on16(a.d_q) && on16(a.d_k) && on16(a.d_v)));
}
// Whether the tcgen05 kernels take a call: their tile of 128 rows and 64 columns
// pays when the window is wide and the rows long, and when there are rows to fill
// it.  Forward / backward in us, matrix instructions per warp against tcgen05:
//   16384 x 8 heads of 64, window 256: 91 / 334 against 56 / 165; 63: 44 / 170 against 41 / 118
//   2048 x 8 of 32, window 256: 16.5 / 56 against 14.8 / 55; 63: 10.0 / 40 against 12.3 / 46
//   2048 x 8 of 16, window 1001: 33 / 77 against 23 / 77; 256: 13.5 / 41 against 14.2 / 47
//   512 x 40 x 8 of 128: 113 / 341 against 120 / 503
bool use_tc(const WinArgs& a, bool backward) {
  const long long w = a.D > a.Dv ? a.D : a.Dv, all = (long long)a.left + a.right + 1, win = all < a.Nk ? all : a.Nk;
  if ((long long)a.B * a.Nq * a.H < 512) return false;     // four row tiles at most: the warp-level kernels, with win_is_fine's second products
  return win * w * w >= 200000 && (long long)a.Nq * a.G >= 64 && a.Nk >= 64 && vectors(a, backward);
}
}  // namespace

cudaError_t launch_win_sink_reduce(const WinArgs& a, int f32, cudaStream_t s) {
  const dim3 grid((unsigned)((long long)a.B * a.Hkv * a.sinks), (unsigned)((a.D + a.Dv + 31) / 32));
  if (f32) win_sink_reduce_kernel<float><<<grid, 1024, 0, s>>>(a);
  else win_sink_reduce_kernel<bf16><<<grid, 1024, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_win_fwd(const WinArgs& a, cudaStream_t s) {
  if (win_step_takes(a)) return launch_win_step(a, s);
  if (win_short_takes(a, false) && vectors(a, false)) return launch_win_short(a, false, s);
  if (use_tc(a, false)) return launch_win_fwd_tc(a, s);
  const int w = a.D > a.Dv ? a.D : a.Dv;
  return w <= 16 ? fwd<16>(a, s) : (w <= 32 ? fwd<32>(a, s) : (w <= 64 ? fwd<64>(a, s) : fwd<128>(a, s)));
}
cudaError_t launch_win_bwd(const WinArgs& in, cudaStream_t s) {
  WinArgs a = in;
  if (win_short_takes(a, true) && vectors(a, true)) return launch_win_short(a, true, s);
  const bool tc = use_tc(a, true);
  const WinSinkPlan sp = win_sink_plan(a, tc ? kWinTcRows : T);
  a.nchunk = sp.nchunk;
  a.chunk_tiles = sp.chunk_tiles;
  a.sink_pos = sp.sink_pos;
  const int w = a.D > a.Dv ? a.D : a.Dv;
  return w <= 16 ? bwd<16>(a, tc, s) : (w <= 32 ? bwd<32>(a, tc, s) : (w <= 64 ? bwd<64>(a, tc, s) : bwd<128>(a, tc, s)));
}

}  // namespace fipa

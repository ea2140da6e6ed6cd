// window_short.cu -- window attention with sinks on many short sequences
// (bfloat16): a CTA holds all rows and keys of one (sample, key head) in shared
// memory, so that everything is read once and, after one wait, no barrier is left
// in the loops; the backward is one kernel, without partial sums for the sinks.
//
// The mathematics and the operand layouts are those of window_mma.cu: a warp
// takes 16 rows (forward, dq), then 16 keys (dk, dv), and the columns that they
// see 16 at a time.  Bound by the copies in and out and, for windows of some 50
// keys and more, by the instructions of the softmax.
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

constexpr int kMaxWords = kWinShortRows / 32;
constexpr int kNowhere = -(1 << 30);       // position of a row that sees nothing

// Everything of one (b, hkv): padded tiles of queries (and dO) and of keys and values.
struct Seq {
  int b, hkv, q0, F, Fp, Kp;               // rows, rows rounded up to 16, keys to 32
  uint32_t q, g, k, v;                     // shared-memory addresses
};
template <int DP>
__device__ __forceinline__ Seq seq_of(const WinArgs& a, uint8_t* smem, bool backward) {
  Seq s;
  s.b = blockIdx.x / a.Hkv;
  s.hkv = blockIdx.x - s.b * a.Hkv;
  s.q0 = win_q0(a, s.b);
  s.F = a.Nq * a.G;
  s.Fp = (s.F + 15) & ~15;
  s.Kp = (a.Nk + 31) & ~31;
  constexpr int row = Tile<DP>::ld * 2;
  s.k = smem_u32(smem);
  s.v = s.k + s.Kp * row;
  s.q = s.v + s.Kp * row;
  s.g = s.q + (backward ? s.Fp * row : 0);
  return s;
}
template <int DP, typename At>
__device__ __forceinline__ void load_all(uint32_t dst, int rows, int width, const bf16* any, At at) {
  constexpr int CH = DP / 8;
  const int c = threadIdx.x % CH;
  const bool in = c * 8 < width;
#pragma unroll 4
  for (int r = threadIdx.x / CH; r < rows; r += blockDim.x / CH) {
    const bf16* p = at(r);
    const bool on = p != nullptr && in;
    cp16_zfill(dst + (r * Tile<DP>::ld + c * 8) * 2, on ? p + c * 8 : any, on);
  }
}
template <int DP>
__device__ __forceinline__ void load_seq(const WinArgs& a, const Seq& s, uint32_t* bits, bool backward) {
  const uint8_t* mask = a.mask == nullptr ? nullptr : a.mask + (long long)s.b * a.Nk;
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, s.b, s.hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, s.b, s.hkv);
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, s.b, s.hkv * a.G);
  auto key = [&](const Src& x) {
    return [&](int j) -> const bf16* { return j < a.Nk && (mask == nullptr || mask[j] != 0) ? x.p + j * x.sn : nullptr; };
  };
  auto row = [&](const Src& x) {
    return [&](int f) -> const bf16* {
      if (f >= s.F) return nullptr;
      const int i = a.G == 1 ? f : f / a.G, h = f - i * a.G, p = s.q0 + i;
      return p >= 0 && p < a.Nk && (mask == nullptr || mask[p] != 0) ? x.p + i * x.sn + h * x.sh : nullptr;
    };
  };
  load_all<DP>(s.k, s.Kp, a.D, k.p, key(k));
  load_all<DP>(s.v, s.Kp, a.Dv, v.p, key(v));
  load_all<DP>(s.q, s.Fp, a.D, q.p, row(q));
  if (backward) {
    const Src g = source(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, s.b, s.hkv * a.G);
    load_all<DP>(s.g, s.Fp, a.Dv, g.p, row(g));
  }
  cp_async_commit();
  for (int j0 = 0; j0 < 32 * kMaxWords; j0 += blockDim.x) {       // which keys exist, as bits
    const int j = j0 + threadIdx.x;
    const uint32_t w = __ballot_sync(0xffffffffu, j < a.Nk && (mask == nullptr || mask[j] != 0));
    if ((threadIdx.x & 31) == 0 && j < 32 * kMaxWords) bits[j >> 5] = w;
  }
}

// The columns of 16 rows in units of 32 neighbouring keys from a multiple of 32
// on: those of the sinks before the window's first unit, then the window's.
struct Units {
  int lo, hi, s;                           // first window unit, last key, sinks before the window (0: go there at once)
  __device__ __forceinline__ int first() const { return s > 0 ? 0 : lo; }
  __device__ __forceinline__ int next(int j0) const { return j0 < lo && j0 + 32 >= s ? lo : j0 + 32; }
};
__device__ __forceinline__ Units units_of(const WinArgs& a, const WinCols& c) {
  const int lo = c.lo & ~31;
  return Units{c.n == 0 ? 0 : lo, c.n == 0 ? -1 : c.hi, c.n == 0 ? 0 : min(a.sinks, lo)};
}
// What the row at position p sees of keys j0 .. j0+31, which exist as `there` says.
__device__ __forceinline__ uint32_t row_bits(const WinArgs& a, uint32_t there, int p, int j0) {
  uint32_t w = win_span(p - a.left - j0, p + a.right + 1 - j0);
  if (j0 < a.sinks) w |= win_span(0, min(a.sinks, p + a.right + 1) - j0);
  return w & there;
}

template <int DP>
__global__ void __launch_bounds__(128) win_short_fwd_kernel(const WinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t bits[kMaxWords];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  const Seq s = seq_of<DP>(a, smem, false);
  load_seq<DP>(a, s, bits, false);
  cp_wait<0>();
  __syncthreads();
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  const float sc = a.scale * kLog2e;
  for (int f0 = 16 * warp; f0 < s.F; f0 += 64) {
    const int f1 = min(s.F, f0 + 16);
    const Units un = units_of(a, win_cols(a, s.q0, f0, f1));
    bool alive[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = f0 + (lane >> 2) + 8 * i;
      pos[i] = s.q0 + (a.G == 1 ? f : f / a.G);
      alive[i] = f < f1 && pos[i] >= 0 && pos[i] < a.Nk && ((bits[pos[i] >> 5] >> (pos[i] & 31)) & 1u);
      if (!alive[i]) pos[i] = kNowhere;
    }
    const bool any = __any_sync(0xffffffffu, alive[0] || alive[1]);
    float acc[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2];
    float2 l2[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    uint32_t qf[DP / 16][4];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) ldsm4(qf[kk], a_addr<DP>(s.q, f0, 16 * kk, lane));
    for (int j0 = un.first(); any && j0 <= un.hi; j0 = un.next(j0)) {
      const uint32_t there = bits[j0 >> 5];
      const uint32_t on[2] = {row_bits(a, there, pos[0], j0), row_bits(a, there, pos[1], j0)};
      const uint32_t ob[2] = {on[0] >> col2, on[1] >> col2};
      float sc_[4][4], mx[2] = {-INFINITY, -INFINITY};
      bool go[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        go[g] = __any_sync(0xffffffffu, ((on[0] | on[1]) >> (16 * g) & 0xffffu) != 0u);
        if (!go[g]) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc_[2 * g + h][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          if (kk >= kd) break;
          uint32_t bf[4];
          ldsm4(bf, b_addr<DP>(s.k, j0 + 16 * g, 16 * kk, lane));
          mma(sc_[2 * g], qf[kk], bf[0], bf[1]);
          mma(sc_[2 * g + 1], qf[kk], bf[2], bf[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc_[2 * g + h][e] = ob[e >> 1] & (1u << (16 * g + 8 * h + (e & 1))) ? sc_[2 * g + h][e] : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], sc_[2 * g + h][e]);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      if (__any_sync(0xffffffffu, (mx[0] - m[0]) * sc > kWinLag || (mx[1] - m[1]) * sc > kWinLag)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float mn = fmaxf(m[i], mx[i]), f = ex2_approx(mn == -INFINITY ? -INFINITY : (m[i] - mn) * sc);
          m[i] = mn;
          l2[i] = mul2(l2[i], both(f));
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            acc[n][2 * i] *= f;
            acc[n][2 * i + 1] *= f;
          }
        }
      }
      const float mb[2] = {m[0] == -INFINITY ? 0.f : m[0] * sc, m[1] == -INFINITY ? 0.f : m[1] * sc};
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!go[g]) continue;
        uint32_t pf[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float2 p = fma2(make_float2(sc_[2 * g + h][2 * i], sc_[2 * g + h][2 * i + 1]), both(sc), both(-mb[i]));
            p = make_float2(ex2_approx(p.x), ex2_approx(p.y));
            l2[i] = add2(l2[i], p);
            pf[2 * h + i] = pack(p.x, p.y);
          }
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          if (n >= kv) break;
          uint32_t bf[4];
          ldsm4t(bf, bt_addr<DP>(s.v, j0 + 16 * g, 16 * n, lane));
          mma(acc[2 * n], pf, bf[0], bf[1]);
          mma(acc[2 * n + 1], pf, bf[2], bf[3]);
        }
      }
    }
    float inv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] = l2[i].x + l2[i].y;
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      inv[i] = alive[i] && l[i] != 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        acc[n][2 * i] *= inv[i];
        acc[n][2 * i + 1] *= inv[i];
      }
    }
    store_rows<DP>(acc, a.Dv, a.out, 1.f, lane, [&](int i, bool& keep) -> bf16* {
      const int f = f0 + (lane >> 2) + 8 * i, qi = a.G == 1 ? f : f / a.G;
      keep = inv[i] != 0.f;
      if (f >= f1) return nullptr;
      const int h = s.hkv * a.G + (f - qi * a.G);
      if (a.lse != nullptr && (lane & 3) == 0)
        a.lse[((long long)s.b * a.H + h) * a.Nq + qi] = keep ? fmaf(m[i], a.scale, logf(l[i])) : -INFINITY;
      return static_cast<bf16*>(a.out) + (((long long)s.b * a.Nq + qi) * a.H + h) * a.Dv;
    });
  }
}

template <int DP>
__global__ void __launch_bounds__(128) win_short_bwd_kernel(const WinArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t bits[kMaxWords];
  __shared__ float slse[kWinShortRows], sdel[kWinShortRows];
  __shared__ short spos[kWinShortRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col2 = (lane & 3) * 2;
  const Seq s = seq_of<DP>(a, smem, true);
  load_seq<DP>(a, s, bits, true);
  // delta = dO.out, four neighbouring lanes a row; lse in units of log 2, +inf where nothing is seen: every p is 0
  for (int r0 = 0; r0 < s.Fp; r0 += 32) {
    const int f = r0 + (threadIdx.x >> 2), i = a.G == 1 ? f : f / a.G, h = s.hkv * a.G + (f - i * a.G), p = s.q0 + i;
    const bool on = f < s.F && p >= 0 && p < a.Nk && (a.mask == nullptr || a.mask[(long long)s.b * a.Nk + p] != 0);
    float x = 0.f, y = -INFINITY;
    if (on) {
      const long long o = (((long long)s.b * a.Nq + i) * a.H + h) * a.Dv;
      const bf16 *u = static_cast<const bf16*>(a.out) + o, *w = static_cast<const bf16*>(a.d_out) + o;
      for (int d = (threadIdx.x & 3) * 8; d < a.Dv; d += 32) {
        const uint4 uu = __ldg(reinterpret_cast<const uint4*>(u + d)), ww = __ldg(reinterpret_cast<const uint4*>(w + d));
        const uint32_t ua[4] = {uu.x, uu.y, uu.z, uu.w}, wa[4] = {ww.x, ww.y, ww.z, ww.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x = fmaf(__uint_as_float(ua[e] << 16), __uint_as_float(wa[e] << 16), x);
          x = fmaf(__uint_as_float(ua[e] & 0xffff0000u), __uint_as_float(wa[e] & 0xffff0000u), x);
        }
      }
      y = a.lse[((long long)s.b * a.H + h) * a.Nq + i];
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if ((threadIdx.x & 3) == 0 && f < s.Fp) {
      sdel[f] = x;
      slse[f] = y == -INFINITY ? INFINITY : y * kLog2e;
      spos[f] = (short)max(-32768, min(32767, p));
    }
  }
  cp_wait<0>();
  __syncthreads();
  const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
  const float sc = a.scale * kLog2e;
  // ---- dq
  for (int f0 = 16 * warp; f0 < s.F; f0 += 64) {
    const int f1 = min(s.F, f0 + 16);
    const Units un = units_of(a, win_cols(a, s.q0, f0, f1));
    float lse2[2], del[2], eps[2], acc[DP / 8][4], avg[DP / 8][4];
    float2 e2[2] = {both(0.f), both(0.f)};
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = f0 + (lane >> 2) + 8 * i;
      lse2[i] = slse[f];
      del[i] = sdel[f];
      pos[i] = lse2[i] == INFINITY ? kNowhere : spos[f];
    }
    const bool any = __any_sync(0xffffffffu, lse2[0] != INFINITY || lse2[1] != INFINITY);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = avg[n][e] = 0.f;
    uint32_t qf[DP / 16][4], gf[DP / 16][4];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      ldsm4(qf[kk], a_addr<DP>(s.q, f0, 16 * kk, lane));
      ldsm4(gf[kk], a_addr<DP>(s.g, f0, 16 * kk, lane));
    }
    for (int j0 = un.first(); any && j0 <= un.hi; j0 = un.next(j0)) {
      const uint32_t there = bits[j0 >> 5];
      const uint32_t on[2] = {row_bits(a, there, pos[0], j0), row_bits(a, there, pos[1], j0)};
      const uint32_t ob[2] = {on[0] >> col2, on[1] >> col2};
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (!__any_sync(0xffffffffu, ((on[0] | on[1]) >> (16 * g) & 0xffffu) != 0u)) continue;
        float x[2][4], dp[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[h][e] = dp[h][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          uint32_t bf[4];
          if (kk < kd) {
            ldsm4(bf, b_addr<DP>(s.k, j0 + 16 * g, 16 * kk, lane));
            mma(x[0], qf[kk], bf[0], bf[1]);
            mma(x[1], qf[kk], bf[2], bf[3]);
          }
          if (kk < kv) {
            ldsm4(bf, b_addr<DP>(s.v, j0 + 16 * g, 16 * kk, lane));
            mma(dp[0], gf[kk], bf[0], bf[1]);
            mma(dp[1], gf[kk], bf[2], bf[3]);
          }
        }
        uint32_t pf[4], df[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 y = fma2(make_float2(x[h][2 * i], x[h][2 * i + 1]), both(sc), both(-lse2[i]));
            const float2 p = make_float2(ob[i] & (1u << (16 * g + 8 * h)) ? ex2_approx(y.x) : 0.f, ob[i] & (2u << (16 * g + 8 * h)) ? ex2_approx(y.y) : 0.f);
            const float2 d = mul2(p, add2(make_float2(dp[h][2 * i], dp[h][2 * i + 1]), both(-del[i])));
            e2[i] = add2(e2[i], d);
            pf[2 * h + i] = pack(p.x, p.y);
            df[2 * h + i] = pack(d.x, d.y);
          }
#pragma unroll
        for (int n = 0; n < DP / 16; ++n) {
          if (n >= kd) break;
          uint32_t bf[4];
          ldsm4t(bf, bt_addr<DP>(s.k, j0 + 16 * g, 16 * n, lane));
          mma(acc[2 * n], df, bf[0], bf[1]);
          mma(acc[2 * n + 1], df, bf[2], bf[3]);
          mma(avg[2 * n], pf, bf[0], bf[1]);
          mma(avg[2 * n + 1], pf, bf[2], bf[3]);
        }
      }
    }
    eps[0] = e2[0].x + e2[0].y;
    eps[1] = e2[1].x + e2[1].y;
    take_back<DP>(acc, avg, eps);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if ((lane & 3) == 0) sdel[f0 + (lane >> 2) + 8 * i] = del[i] + eps[i];
    store_rows<DP>(acc, a.D, a.d_q, a.scale, lane, [&](int i, bool& keep) -> bf16* {
      const int f = f0 + (lane >> 2) + 8 * i, qi = a.G == 1 ? f : f / a.G;
      keep = lse2[i] != INFINITY;
      return f < f1 ? static_cast<bf16*>(a.d_q) + (((long long)s.b * a.Nq + qi) * a.H + s.hkv * a.G + (f - qi * a.G)) * a.D : nullptr;
    });
  }
  __syncthreads();                           // delta
  // ---- dk, dv
  for (int k0 = 16 * warp; k0 < a.Nk; k0 += 64) {
    const int k1 = min(a.Nk, k0 + 16) - 1;
    const int pl = max(0, k0 - a.right), ph = k0 < a.sinks ? a.Nk - 1 : min(a.Nk - 1, k1 + a.left);
    const int il = max(pl - s.q0, 0), ih = min(ph - s.q0, a.Nq - 1);
    const int fl = ih < il ? 0 : il * a.G / 16 * 16, fh = ih < il ? 0 : (ih + 1) * a.G;
    bool alive[2];
    int rlo[2], rhi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = k0 + (lane >> 2) + 8 * i;
      alive[i] = j <= k1 && ((bits[j >> 5] >> (j & 31)) & 1u);
      key_rows(a, s.q0, j, 0, s.Fp, rlo[i], rhi[i]);
    }
    float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.f;
    uint32_t kf[DP / 16][4], vf[DP / 16][4];
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      ldsm4(kf[kk], a_addr<DP>(s.k, k0, 16 * kk, lane));
      ldsm4(vf[kk], a_addr<DP>(s.v, k0, 16 * kk, lane));
    }
    const bool any = __any_sync(0xffffffffu, alive[0] || alive[1]);
    for (int f0 = fl; any && f0 < fh; f0 += 16) {
      const uint32_t on[2] = {win_span(rlo[0] - f0, rhi[0] - f0), win_span(rlo[1] - f0, rhi[1] - f0)};
      if (!__any_sync(0xffffffffu, ((on[0] | on[1]) & 0xffffu) != 0u)) continue;
      const uint32_t ob[2] = {on[0] >> col2, on[1] >> col2};
      float x[2][4], dp[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[h][e] = dp[h][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        uint32_t bf[4];
        if (kk < kd) {
          ldsm4(bf, b_addr<DP>(s.q, f0, 16 * kk, lane));
          mma(x[0], kf[kk], bf[0], bf[1]);
          mma(x[1], kf[kk], bf[2], bf[3]);
        }
        if (kk < kv) {
          ldsm4(bf, b_addr<DP>(s.g, f0, 16 * kk, lane));
          mma(dp[0], vf[kk], bf[0], bf[1]);
          mma(dp[1], vf[kk], bf[2], bf[3]);
        }
      }
      uint32_t pf[4], df[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 ls = *reinterpret_cast<const float2*>(slse + f0 + 8 * h + col2), de = *reinterpret_cast<const float2*>(sdel + f0 + 8 * h + col2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 y = fma2(make_float2(x[h][2 * i], x[h][2 * i + 1]), both(sc), make_float2(-ls.x, -ls.y));
          const float2 p = make_float2(ob[i] & (1u << (8 * h)) ? ex2_approx(y.x) : 0.f, ob[i] & (2u << (8 * h)) ? ex2_approx(y.y) : 0.f);
          const float2 d = mul2(p, add2(make_float2(dp[h][2 * i], dp[h][2 * i + 1]), make_float2(-de.x, -de.y)));
          pf[2 * h + i] = pack(p.x, p.y);
          df[2 * h + i] = pack(d.x, d.y);
        }
      }
#pragma unroll
      for (int n = 0; n < DP / 16; ++n) {
        uint32_t bf[4];
        if (n < kv) {
          ldsm4t(bf, bt_addr<DP>(s.g, f0, 16 * n, lane));
          mma(dv[2 * n], pf, bf[0], bf[1]);
          mma(dv[2 * n + 1], pf, bf[2], bf[3]);
        }
        if (n < kd) {
          ldsm4t(bf, bt_addr<DP>(s.q, f0, 16 * n, lane));
          mma(dk[2 * n], df, bf[0], bf[1]);
          mma(dk[2 * n + 1], df, bf[2], bf[3]);
        }
      }
    }
    auto at = [&](void* base, int width, int i, bool& keep) -> bf16* {
      const int j = k0 + (lane >> 2) + 8 * i;
      keep = alive[i];
      return j <= k1 ? static_cast<bf16*>(base) + (((long long)s.b * a.Nk + j) * a.Hkv + s.hkv) * width : nullptr;
    };
    store_rows<DP>(dk, a.D, a.d_k, a.scale, lane, [&](int i, bool& keep) { return at(a.d_k, a.D, i, keep); });
    store_rows<DP>(dv, a.Dv, a.d_v, 1.f, lane, [&](int i, bool& keep) { return at(a.d_v, a.Dv, i, keep); });
  }
}

template <int DP>
cudaError_t run(const WinArgs& a, bool backward, cudaStream_t s) {
  const size_t smem = win_short_smem(a, DP, backward);
  const cudaError_t e = allow_max_smem(backward ? reinterpret_cast<const void*>(&win_short_bwd_kernel<DP>)
                                                : reinterpret_cast<const void*>(&win_short_fwd_kernel<DP>));
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)((long long)a.B * a.Hkv);
  if (backward) win_short_bwd_kernel<DP><<<grid, 128, smem, s>>>(a);
  else win_short_fwd_kernel<DP><<<grid, 128, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_win_short(const WinArgs& a, bool backward, cudaStream_t s) {
  const int w = a.D > a.Dv ? a.D : a.Dv;
  return w <= 16 ? run<16>(a, backward, s) : (w <= 32 ? run<32>(a, backward, s) : run<64>(a, backward, s));
}

}  // namespace fipa

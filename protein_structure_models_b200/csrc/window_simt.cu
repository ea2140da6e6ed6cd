// window_simt.cu -- window attention with sinks on float32 tensors, on the CUDA
// cores, whose products keep every bit of the operands (window.h has
// the visibility rule and the row / column numbering).
//
// Forward, one pass over a row tile's columns: m the running row maximum, l the
// running sum of exp(s - m), O the running sum of exp(s - m) v, both scaled by
// exp(m_old - m_new) when m grows; out = O / l, lse = m + ln l.
// Backward: p = exp(s - lse), ds = p (dO.v - delta) with delta = dO.out;
// dq = scale sum ds k (row side), dv = sum p dO, dk = scale sum ds q (key side).
// Each side recomputes p, so that every sum has one owner and a fixed order.
//
// 64 x 64 tiles, 256 threads, 4 x 4 scores a thread; every operand sits in
// shared memory width-major ([width][64 rows]), so that the score product reads
// four rows and four keys per 16-byte load and the second product four columns.
#include <math.h>

#include "kernels.h"
#include "window.h"

namespace fipa {
namespace {

constexpr int T = kWinSimtTile;
constexpr int LD = T + 4;          // padded row of a width-major tile
constexpr int kThreads = 256;

__device__ __forceinline__ float ldf(const float* p) { return *p; }
__device__ __forceinline__ float ldf(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void stf(float* p, float x) { *p = x; }
__device__ __forceinline__ void stf(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Row threadIdx.x % 64 of a tile into dst[width][64], zeros where p is null: a
// thread keeps its row and takes every fourth run of four channels, so that a
// warp's 32 stores of one channel lie side by side.
template <typename E>
__device__ __forceinline__ void load_row(float* dst, const E* p, int width) {
  const int r = threadIdx.x & (T - 1);
  const bool vec = sizeof(E) == 4 && (width & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
  for (int d = (threadIdx.x / T) * 4; d < width; d += kThreads / T * 4) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (p != nullptr) {
      if (vec) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(p + d));
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (d + k < width) x[k] = ldf(p + d + k);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (d + k < width) dst[(d + k) * LD + r] = x[k];
  }
}
// Rows [f0, f0 + 64) of (b, hkv); rows at or beyond f1 and rows that see nothing are zero.
template <typename E>
__device__ __forceinline__ void load_rows(float* dst, const E* base, long long sb, long long sn, long long sh, const WinArgs& a, int b,
                          int hkv, int q0, int f0, int f1, int width) {
  const int f = f0 + (threadIdx.x & (T - 1)), i = f / a.G;
  const bool on = f < f1 && win_alive(a, b, q0 + i);
  load_row(dst, on ? base + b * sb + i * sn + (hkv * a.G + (f - i * a.G)) * sh : nullptr, width);
}
// Keys of columns [u0, u0 + 64); masked keys and columns beyond the last are zero.
template <typename E>
__device__ __forceinline__ void load_cols(float* dst, const E* base, long long sb, long long sn, long long sh, const WinArgs& a, int b,
                          int hkv, const WinCols& c, int u0, int width) {
  const int u = u0 + (threadIdx.x & (T - 1)), j = c.key(u);
  const bool on = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + j] != 0);
  load_row(dst, on ? base + b * sb + j * sn + hkv * sh : nullptr, width);
}

// acc[i][j] = sum_d A[d][4 ty + i] B[d][4 tx + j]
__device__ __forceinline__ void product(const float* A, const float* B, int width, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < width; ++d) {
    const float4 x = *reinterpret_cast<const float4*>(A + d * LD + 4 * ty);
    const float4 y = *reinterpret_cast<const float4*>(B + d * LD + 4 * tx);
    const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xa[i], ya[j], acc[i][j]);
  }
}
// acc[i][c] += sum_k P[4 ty + i][k] V[tx + 16 c][k]   (V width-major, `width` rows)
template <int NC>
__device__ __forceinline__ void accumulate(const float* P, const float* V, int width, int ty, int tx, float (&acc)[4][NC]) {
#pragma unroll 2
  for (int k = 0; k < T; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (4 * ty + i) * LD + k);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (tx + 16 * c >= width) break;
      const float4 v = *reinterpret_cast<const float4*>(V + (tx + 16 * c) * LD + k);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][c] = fmaf(p[i].x, v.x, fmaf(p[i].y, v.y, fmaf(p[i].z, v.z, fmaf(p[i].w, v.w, acc[i][c]))));
    }
  }
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename E, int NC>
__global__ void __launch_bounds__(kThreads) win_fwd_simt_kernel(const WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + a.D * LD;
  float* Vs = Ks + a.D * LD;
  float* Ps = Vs + a.Dv * LD;
  __shared__ uint8_t live[T];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int F = a.Nq * a.G, tiles = (F + T - 1) / T;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * T, f1 = min(F, f0 + T), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  load_rows(Qs, static_cast<const E*>(a.q), a.qb, a.qn, a.qh, a, b, hkv, q0, f0, f1, a.D);
  WinRow row[4];
  float m[4], l[4], acc[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = f0 + 4 * ty + i, p = q0 + f / a.G;
    row[i] = win_row(a, c, p, f < f1 && win_alive(a, b, p));
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = 0.f;
  }
  for (int u0 = 0; u0 < c.n; u0 += T) {
    __syncthreads();
    load_cols(Ks, static_cast<const E*>(a.k), a.kb, a.kn, a.kh, a, b, hkv, c, u0, a.D);
    load_cols(Vs, static_cast<const E*>(a.v), a.vb, a.vn, a.vh, a, b, hkv, c, u0, a.Dv);
    if (threadIdx.x < T) {
      const int u = u0 + threadIdx.x;
      live[threadIdx.x] = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0);
    }
    __syncthreads();
    float s[4][4];
    product(Qs, Ks, a.D, ty, tx, s);
    uint32_t lv = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) lv |= live[4 * tx + j] ? 1u << j : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
      const uint32_t on = row[i].sees(u0 + 4 * tx) & lv;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (on >> j) & 1u ? s[i][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], max16(mx));
      const float mb = mn == -INFINITY ? 0.f : mn;
      const float f = expf(m[i] - mb);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - mb);
        sum += s[i][j];
      }
      l[i] = l[i] * f + sum16(sum);
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[i][j] *= f;
      *reinterpret_cast<float4*>(Ps + (4 * ty + i) * LD + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    __syncwarp();                       // a row's 64 scores come from the 16 lanes of one half warp
    accumulate<NC>(Ps, Vs, a.Dv, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = f0 + 4 * ty + i;
    if (f >= f1) continue;
    const int qi = f / a.G, h = hkv * a.G + (f - qi * a.G);
    const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
    E* o = static_cast<E*>(a.out) + (((long long)b * a.Nq + qi) * a.H + h) * a.Dv;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (tx + 16 * j < a.Dv) stf(o + tx + 16 * j, acc[i][j] * inv);
    if (a.lse != nullptr && tx == 0)
      a.lse[((long long)b * a.H + h) * a.Nq + qi] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
}

// Row side: delta, then dq.  Writes delta for the key side.
template <typename E, int NC>
__global__ void __launch_bounds__(kThreads) win_bwd_q_simt_kernel(const WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Os = Qs + a.D * LD;
  float* Ks = Os + a.Dv * LD;
  float* Vs = Ks + a.D * LD;
  float* Ps = Vs + a.Dv * LD;
  __shared__ uint8_t live[T];
  __shared__ float sdelta[T];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int F = a.Nq * a.G, tiles = (F + T - 1) / T;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * T, f1 = min(F, f0 + T), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const long long on = (long long)a.H * a.Dv, ob = on * a.Nq;
  load_rows(Qs, static_cast<const E*>(a.q), a.qb, a.qn, a.qh, a, b, hkv, q0, f0, f1, a.D);
  load_rows(Os, static_cast<const E*>(a.d_out), ob, on, (long long)a.Dv, a, b, hkv, q0, f0, f1, a.Dv);
  {
    // four threads a row
    const int r = threadIdx.x >> 2, f = f0 + r, i = f / a.G, h = hkv * a.G + (f - i * a.G);
    float x = 0.f;
    if (f < f1 && win_alive(a, b, q0 + i)) {
      const long long o = b * ob + i * on + (long long)h * a.Dv;
      for (int d = threadIdx.x & 3; d < a.Dv; d += 4)
        x = fmaf(ldf(static_cast<const E*>(a.d_out) + o + d), ldf(static_cast<const E*>(a.out) + o + d), x);
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if ((threadIdx.x & 3) == 0) {
      sdelta[r] = x;
      if (f < f1) a.delta[((long long)b * a.H + h) * a.Nq + i] = x;
    }
  }
  __syncthreads();
  WinRow row[4];
  float lse[4], del[4], acc[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = f0 + 4 * ty + i, qi = f / a.G, p = q0 + qi;
    lse[i] = f < f1 ? a.lse[((long long)b * a.H + hkv * a.G + (f - qi * a.G)) * a.Nq + qi] : -INFINITY;
    row[i] = win_row(a, c, p, f < f1 && lse[i] != -INFINITY && win_alive(a, b, p));
    del[i] = sdelta[4 * ty + i];
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[i][j] = 0.f;
  }
  for (int u0 = 0; u0 < c.n; u0 += T) {
    __syncthreads();
    load_cols(Ks, static_cast<const E*>(a.k), a.kb, a.kn, a.kh, a, b, hkv, c, u0, a.D);
    load_cols(Vs, static_cast<const E*>(a.v), a.vb, a.vn, a.vh, a, b, hkv, c, u0, a.Dv);
    if (threadIdx.x < T) {
      const int u = u0 + threadIdx.x;
      live[threadIdx.x] = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0);
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    product(Qs, Ks, a.D, ty, tx, s);
    uint32_t lv = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) lv |= live[4 * tx + j] ? 1u << j : 0u;
    product(Os, Vs, a.Dv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t on = row[i].sees(u0 + 4 * tx) & lv;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = (on >> j) & 1u ? expf(s[i][j] * a.scale - lse[i]) * (dp[i][j] - del[i]) : 0.f;
      }
      *reinterpret_cast<float4*>(Ps + (4 * ty + i) * LD + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    __syncwarp();
    accumulate<NC>(Ps, Ks, a.D, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = f0 + 4 * ty + i;
    if (f >= f1) continue;
    const int qi = f / a.G, h = hkv * a.G + (f - qi * a.G);
    E* o = static_cast<E*>(a.d_q) + (((long long)b * a.Nq + qi) * a.H + h) * a.D;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (tx + 16 * j < a.D) stf(o + tx + 16 * j, acc[i][j] * a.scale);
  }
}

// Key side: dk and dv of one key tile over the rows of its window, or (sink
// jobs) over one chunk of the rows beyond it.
template <typename E, int NC>
__global__ void __launch_bounds__(kThreads) win_bwd_k_simt_kernel(const WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + a.D * LD;
  float* Qs = Vs + a.Dv * LD;
  float* Os = Qs + a.D * LD;
  float* Ps = Os + a.Dv * LD;          // p^T, then ds^T
  __shared__ float slse[T], sdel[T];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int ktiles = (a.Nk + T - 1) / T;
  const int nsink = a.nchunk > 0 ? (a.sinks + T - 1) / T : 0;
  const int jobs = ktiles + nsink * a.nchunk;
  const int job = blockIdx.x % jobs, bh = blockIdx.x / jobs, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const bool sink_job = job >= ktiles;
  const int kt = sink_job ? (job - ktiles) / a.nchunk : job;
  const int chunk = sink_job ? (job - ktiles) % a.nchunk : -1;
  const int F = a.Nq * a.G, q0 = win_q0(a, b);
  const int j0 = kt * T, j1 = min(a.Nk, j0 + T) - 1;
  const bool split = kt < nsink;
  // positions whose rows this job sums over
  const int pl = sink_job ? a.sink_pos : max(0, j0 - a.right);
  const int ph = sink_job || (j0 < a.sinks && !split) ? a.Nk - 1 : min(a.Nk - 1, split ? a.sink_pos - 1 : j1 + a.left);
  const int il = max(pl - q0, 0), ih = min(ph - q0, a.Nq - 1);
  int fl = il * a.G, fh = (ih + 1) * a.G;
  if (ih < il) fl = fh = 0;
  if (sink_job) {
    fl = max(fl, chunk * a.chunk_tiles * T);
    fh = min(fh, (chunk + 1) * a.chunk_tiles * T);
  }
  const WinCols c{j0, j1, 0, j1 - j0 + 1};
  load_cols(Ks, static_cast<const E*>(a.k), a.kb, a.kn, a.kh, a, b, hkv, c, 0, a.D);
  load_cols(Vs, static_cast<const E*>(a.v), a.vb, a.vn, a.vh, a, b, hkv, c, 0, a.Dv);
  bool alive[4];
  float dk[4][NC], dv[4][NC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 4 * ty + i;
    alive[i] = j <= j1 && win_alive(a, b, j);
#pragma unroll
    for (int n = 0; n < NC; ++n) dk[i][n] = dv[i][n] = 0.f;
  }
  const long long on = (long long)a.H * a.Dv, ob = on * a.Nq;
  for (int f0 = fl; f0 < fh; f0 += T) {
    const int f1 = min(fh, f0 + T);
    __syncthreads();
    load_rows(Qs, static_cast<const E*>(a.q), a.qb, a.qn, a.qh, a, b, hkv, q0, f0, f1, a.D);
    load_rows(Os, static_cast<const E*>(a.d_out), ob, on, (long long)a.Dv, a, b, hkv, q0, f0, f1, a.Dv);
    if (threadIdx.x < T) {
      const int f = f0 + threadIdx.x, i = f / a.G;
      float x = -INFINITY, d = 0.f;
      if (f < f1 && win_alive(a, b, q0 + i)) {
        const long long o = ((long long)b * a.H + hkv * a.G + (f - i * a.G)) * a.Nq + i;
        x = a.lse[o];
        d = a.delta[o];
      }
      slse[threadIdx.x] = x;
      sdel[threadIdx.x] = d;
    }
    __syncthreads();
    float s[4][4], dp[4][4];
    product(Ks, Qs, a.D, ty, tx, s);
    product(Vs, Os, a.Dv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + 4 * ty + i;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int r = 4 * tx + n, p = q0 + (f0 + r) / a.G;
        const bool on_ = alive[i] && slse[r] != -INFINITY && j <= p + a.right && (j >= p - a.left || j < a.sinks);
        s[i][n] = on_ ? expf(s[i][n] * a.scale - slse[r]) : 0.f;
        dp[i][n] = on_ ? s[i][n] * (dp[i][n] - sdel[r]) : 0.f;
      }
      *reinterpret_cast<float4*>(Ps + (4 * ty + i) * LD + 4 * tx) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    __syncwarp();
    accumulate<NC>(Ps, Os, a.Dv, ty, tx, dv);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(Ps + (4 * ty + i) * LD + 4 * tx) = make_float4(dp[i][0], dp[i][1], dp[i][2], dp[i][3]);
    __syncwarp();
    accumulate<NC>(Ps, Qs, a.D, ty, tx, dk);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = j0 + 4 * ty + i;
    if (j > j1) continue;
    if (split && j < a.sinks) {
      float* o = a.part + (((long long)bh * (a.nchunk + 1) + chunk + 1) * a.sinks + j) * (a.D + a.Dv);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        if (tx + 16 * n < a.D) o[tx + 16 * n] = dk[i][n];
        if (tx + 16 * n < a.Dv) o[a.D + tx + 16 * n] = dv[i][n];
      }
    } else if (!sink_job) {
      E* ok = static_cast<E*>(a.d_k) + (((long long)b * a.Nk + j) * a.Hkv + hkv) * a.D;
      E* ov = static_cast<E*>(a.d_v) + (((long long)b * a.Nk + j) * a.Hkv + hkv) * a.Dv;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        if (tx + 16 * n < a.D) stf(ok + tx + 16 * n, dk[i][n] * a.scale);
        if (tx + 16 * n < a.Dv) stf(ov + tx + 16 * n, dv[i][n]);
      }
    }
  }
}

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

template <typename E, int NC>
cudaError_t fwd(const WinArgs& a, cudaStream_t s) {
  const long long grid = (long long)a.B * a.Hkv * (((long long)a.Nq * a.G + T - 1) / T);
  const size_t smem = ((size_t)(2 * a.D + a.Dv) * LD + T * LD) * sizeof(float);
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_fwd_simt_kernel<E, NC>));
  if (e != cudaSuccess) return e;
  win_fwd_simt_kernel<E, NC><<<(unsigned)grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename E, int NC>
cudaError_t bwd(const WinArgs& a, cudaStream_t s) {
  const size_t smem = ((size_t)(2 * a.D + 2 * a.Dv) * LD + T * LD) * sizeof(float);
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_bwd_q_simt_kernel<E, NC>));
  if (e != cudaSuccess) return e;
  e = allow_max_smem(reinterpret_cast<const void*>(&win_bwd_k_simt_kernel<E, NC>));
  if (e != cudaSuccess) return e;
  const long long gq = (long long)a.B * a.Hkv * (((long long)a.Nq * a.G + T - 1) / T);
  win_bwd_q_simt_kernel<E, NC><<<(unsigned)gq, kThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int nsink = a.nchunk > 0 ? (a.sinks + T - 1) / T : 0;
  const long long gk = (long long)a.B * a.Hkv * ((a.Nk + T - 1) / T + (long long)nsink * a.nchunk);
  win_bwd_k_simt_kernel<E, NC><<<(unsigned)gk, kThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return a.nchunk > 0 ? launch_win_sink_reduce(a, sizeof(E) == 4, s) : cudaSuccess;
}

}  // namespace

cudaError_t launch_win_sink_reduce(const WinArgs& a, int f32, cudaStream_t s) {
  const dim3 grid((unsigned)((long long)a.B * a.Hkv * a.sinks), (unsigned)((a.D + a.Dv + 31) / 32));
  if (f32) win_sink_reduce_kernel<float><<<grid, 1024, 0, s>>>(a);
  else win_sink_reduce_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_win_fwd_simt(const WinArgs& a, cudaStream_t s) {
  const int nc = (a.Dv + 15) / 16;
  return nc <= 2 ? fwd<float, 2>(a, s) : (nc <= 4 ? fwd<float, 4>(a, s) : fwd<float, 8>(a, s));
}
cudaError_t launch_win_bwd_simt(const WinArgs& in, cudaStream_t s) {
  WinArgs a = in;
  const WinSinkPlan sp = win_sink_plan(a, T);
  a.nchunk = sp.nchunk;
  a.chunk_tiles = sp.chunk_tiles;
  a.sink_pos = sp.sink_pos;
  const int nc = ((a.D > a.Dv ? a.D : a.Dv) + 15) / 16;
  return nc <= 2 ? bwd<float, 2>(a, s) : (nc <= 4 ? bwd<float, 4>(a, s) : bwd<float, 8>(a, s));
}

}  // namespace fipa

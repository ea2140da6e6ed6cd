// norm.cu -- the junction between two blocks of a residual network, and its
// gradient (fipa_norm_residual, fipa_norm_residual_backward):
//   y = Norm(u) post_w + post_b,  r = s + res_scale sigmoid(gate) y,
//   x = Norm(r) pre_w + pre_b,    Norm(z) = (z - mean z) rstd (layer) or z rstd (rms).
// With zhat = Norm(z) and h = w dy, dz = rstd (h - mean h - zhat mean(h zhat))
// (rms: without mean h).
//
// Bound by memory: one pass, every tensor read or written once, a row held in
// the registers of the 2^k threads (8 elements each) that own it.  The mean is
// subtracted before squares are summed, so a large mean costs no digits.  The
// backward recomputes r from s, u and gate (as many bytes as reading r, and not
// rounded to the stream's type).  Parameter gradients: every thread keeps the
// sums of its own columns over the rows its CTA walks; the CTAs' sums are added
// in CTA order by a second kernel.  All arithmetic is float32; a tensor's type
// is only how it is stored, rounded once.
#include <math.h>

#include "fipa.h"
#include "kernels.h"
#include "sm100.cuh"

#define FIPA_API extern "C" __attribute__((visibility("default")))

namespace fipa {
namespace {

constexpr int E = 8;                       // elements of a row per thread
constexpr int kNormMaxC = 8192;

struct NormArgs {
  const void *s, *u, *gate;
  const uint8_t* mask;
  const float *res_scale, *post_w, *post_b, *pre_w, *pre_b;
  void *r, *x;
  float* stats;                            // [rows][4]: mean u, rstd u, mean r, rstd r
  const void *d_r, *d_x;
  void *d_s, *d_u, *d_gate;
  float* part;                             // [grid][5][C]
  long long rows;
  int C, tpr, rms;                         // threads per row: a power of two
  float eps;
};

__device__ __forceinline__ float cvt(float x) { return x; }
__device__ __forceinline__ float cvt(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int H = E / 2;                   // pairs of a row per thread

// The thread's elements of a row: 8 neighbours by 16-byte accesses (VEC), or
// every tpr-th element, so that a warp's accesses are contiguous at any width.
template <bool VEC>
__device__ __forceinline__ int col(int t, int tpr, int e) { return VEC ? t * E + e : t + e * tpr; }

__device__ __forceinline__ void cp_zfill16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_zfill4(void* dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// A thread's part of one tensor's row on its way through shared memory: the
// thread that copies it is the one that reads it, so the copies of the next two
// rows need no barrier and no registers.  Elements off 16-byte lines arrive 4
// bytes at a time; 2-byte ones cannot and are loaded when they are used.
template <typename T, bool VEC, int BLOCK>
struct Slot {
  static constexpr bool kAsync = VEC || sizeof(T) == 4;
  static constexpr int kBytes = kAsync ? E * (int)sizeof(T) * BLOCK : 0;
  static __device__ __forceinline__ void fetch(uint8_t* slot, const T* p, int t, int tpr, int C, bool on) {
    if (VEC) {
      on = on && t * E < C;
#pragma unroll
      for (int h = 0; h < E * (int)sizeof(T) / 16; ++h)
        cp_zfill16(slot + (h * BLOCK + threadIdx.x) * 16, on ? p + t * E + h * (16 / (int)sizeof(T)) : p, on);
    } else if (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = t + e * tpr;
        cp_zfill4(slot + (e * BLOCK + threadIdx.x) * 4, on && c < C ? p + c : p, on && c < C);
      }
    }
  }
  static __device__ __forceinline__ void get(const uint8_t* slot, const T* p, int t, int tpr, int C, bool on, float2 (&x)[H]) {
    if (VEC && sizeof(T) == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(slot + threadIdx.x * 16);
      const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < H; ++e) x[e] = make_float2(__uint_as_float(ww[e] << 16), __uint_as_float(ww[e] & 0xffff0000u));
    } else if (VEC) {
      const float4 lo = *reinterpret_cast<const float4*>(slot + threadIdx.x * 16);
      const float4 hi = *reinterpret_cast<const float4*>(slot + (BLOCK + threadIdx.x) * 16);
      x[0] = make_float2(lo.x, lo.y); x[1] = make_float2(lo.z, lo.w);
      x[2] = make_float2(hi.x, hi.y); x[3] = make_float2(hi.z, hi.w);
    } else if (sizeof(T) == 4) {
      const float* f = reinterpret_cast<const float*>(slot) + threadIdx.x;
#pragma unroll
      for (int e = 0; e < H; ++e) x[e] = make_float2(f[2 * e * BLOCK], f[(2 * e + 1) * BLOCK]);
    } else {
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = t + e * tpr;
        f[e] = on && c < C ? cvt(p[c]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < H; ++e) x[e] = make_float2(f[2 * e], f[2 * e + 1]);
    }
  }
};
template <bool VEC, typename T>
__device__ __forceinline__ void put_row(T* p, int t, int tpr, int C, const float2 (&v)[H]) {
  if (VEC) {
    if (t * E >= C) return;
    if (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[e].x, v[e].y);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p + t * E) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4* q = reinterpret_cast<float4*>(p + t * E);
      q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const int c = t + 2 * e * tpr;
      if (c < C) put(p + c, v[e].x);
      if (c + tpr < C) put(p + c + tpr, v[e].y);
    }
  }
}
// The backward reads its parameters anew for every row: they stay in L1, and the
// registers go to the parameters' own sums.
template <bool VEC>
__device__ __forceinline__ void get_param(const float* p, float none, int t, int tpr, int C, float2 (&v)[H]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < H; ++e) v[e] = both(none);
  } else if (VEC) {
    float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
    if (t * E < C) {
      lo = __ldg(reinterpret_cast<const float4*>(p + t * E));
      hi = __ldg(reinterpret_cast<const float4*>(p + t * E) + 1);
    }
    v[0] = make_float2(lo.x, lo.y); v[1] = make_float2(lo.z, lo.w);
    v[2] = make_float2(hi.x, hi.y); v[3] = make_float2(hi.z, hi.w);
  } else {
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const int c = t + 2 * e * tpr;
      v[e] = make_float2(c < C ? __ldg(p + c) : 0.f, c + tpr < C ? __ldg(p + c + tpr) : 0.f);
    }
  }
}

// Sums over the tpr threads of a row, the same in all of them.  Every thread of
// the CTA calls it (rows of more than a warp meet in shared memory, in two places
// in turn, so that one barrier a sum is enough).
struct RowSum {
  float2 (*red)[32];
  int turn;
  __device__ __forceinline__ float operator()(float v, int tpr) {
    const int w = tpr < 32 ? tpr : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < w) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr > 32) v = across(make_float2(v, 0.f), tpr).x;
    return v;
  }
  __device__ __forceinline__ float2 operator()(float2 v, int tpr) {
    const int w = tpr < 32 ? tpr : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= w) continue;
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return tpr > 32 ? across(v, tpr) : v;
  }
  __device__ __forceinline__ float2 across(float2 v, int tpr) {
    const int nw = tpr >> 5, warp = threadIdx.x >> 5, first = warp / nw * nw;
    if ((threadIdx.x & 31) == 0) red[turn][warp] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
    for (int k = 0; k < nw; ++k) {
      v.x += red[turn][first + k].x;
      v.y += red[turn][first + k].y;
    }
    turn ^= 1;
    return v;
  }
};

// Elements of a row that this thread has: its first n (all or none with VEC).  The
// others hold 0, their parameters are 0 (see get_param) and they are never stored,
// so that only the sums of what is not 0 by itself have to leave them out.
template <bool VEC>
__device__ __forceinline__ int mine(int t, int tpr, int C) {
  if (VEC) return t * E < C ? E : 0;
  const int n = (C - t + tpr - 1) / tpr;
  return t < C ? (n < E ? n : E) : 0;
}

// Element pairs that exist, as factors 1 or 0 of what would not be 0 by itself (VEC: all or none).
template <bool VEC>
__device__ __forceinline__ float2 there(int e, int n) {
  return VEC ? both(1.f) : make_float2(2 * e < n ? 1.f : 0.f, 2 * e + 1 < n ? 1.f : 0.f);
}

// mean and rstd of the row; z becomes z - mean
template <bool VEC>
__device__ __forceinline__ float2 moments(float2 (&z)[H], int n, const NormArgs& a, int tpr, float inv, RowSum& sum) {
  float mean = 0.f;
  if (!a.rms) {
    const float2 v = add2(add2(z[0], z[1]), add2(z[2], z[3]));
    mean = sum(v.x + v.y, tpr) * inv;
  }
  float2 v = both(0.f);
#pragma unroll
  for (int e = 0; e < H; ++e) {
    z[e] = add2(z[e], both(-mean));
    if (!VEC) z[e] = mul2(z[e], there<VEC>(e, n));
    v = fma2(z[e], z[e], v);
  }
  const float q = VEC && n == 0 ? 0.f : v.x + v.y;
  return make_float2(mean, rsqrtf(sum(q, tpr) * inv + a.eps));
}

// 1 / (1 + 2^(-x log2 e)); the rounding of x log2 e, which 2^() would pass on
// multiplied by ln 2, is put back.  Beyond +-88, where that rounding would meet a
// power that is infinite, the result is 0 or 1 in float32 all the same; a NaN stays one.
__device__ __forceinline__ float within88(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-88.f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(88.f));
  return y;
}
__device__ __forceinline__ float2 sigmoid(float2 g) {
  constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
  const float2 x = make_float2(within88(g.x), within88(g.y));
  const float2 y = mul2(x, both(-kLog2e)), r = fma2(x, both(-kLog2e), make_float2(-y.x, -y.y));
  float2 p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(y.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(y.y));
  p = add2(fma2(p, mul2(r, both(kLn2)), p), both(1.f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(p.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(p.y));
  return p;
}

// The forward keeps its parameters in registers (reading them anew for each row
// took the shared-memory path a third of its time: 70 us against 57 at 76800 x 256),
// which leaves 512 threads an SM.
constexpr int fwd_ctas(int block) { return block > 512 ? 1 : 512 / block; }

template <typename TS, typename TB, bool VEC, int BLOCK, int TPR>
__global__ void __launch_bounds__(BLOCK, fwd_ctas(BLOCK)) norm_fwd_kernel(const NormArgs a) {
  typedef Slot<TS, VEC, BLOCK> SS;
  typedef Slot<TB, VEC, BLOCK> SB;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kStage = SS::kBytes + 2 * SB::kBytes;
  __shared__ float2 red[2][32];
  RowSum sum{red, 0};
  const int tpr = TPR > 0 ? TPR : a.tpr, t = threadIdx.x & (tpr - 1), rpb = BLOCK / tpr;
  const bool branch = a.u != nullptr, gated = a.gate != nullptr;
  const int n = mine<VEC>(t, tpr, a.C);
  const float inv = 1.f / (float)a.C;
  const long long step = (long long)gridDim.x * rpb;
  const long long first = (long long)blockIdx.x * rpb + threadIdx.x / tpr;     // this thread's rows: first, first + step, ...
  bool soon;                                                                     // whether the row to be fetched next is valid
  auto look = [&](long long row) { return row < a.rows && (a.mask == nullptr || a.mask[row] != 0); };
  auto fetch = [&](int k, long long row, bool live) {
    uint8_t* slot = ring + (k & 1) * kStage;
    const long long o = (row < a.rows ? row : 0) * a.C;
    SS::fetch(slot, static_cast<const TS*>(a.s) + o, t, tpr, a.C, row < a.rows);
    if (branch) SB::fetch(slot + SS::kBytes, static_cast<const TB*>(a.u) + o, t, tpr, a.C, live);
    if (gated) SB::fetch(slot + SS::kBytes + SB::kBytes, static_cast<const TB*>(a.gate) + o, t, tpr, a.C, live);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float2 pw[H], pb[H], ga[H], qw[H], qb[H];
  get_param<VEC>(a.post_w, 1.f, t, tpr, a.C, pw);
  get_param<VEC>(a.post_b, 0.f, t, tpr, a.C, pb);
  get_param<VEC>(a.res_scale, 1.f, t, tpr, a.C, ga);
  get_param<VEC>(a.pre_w, 1.f, t, tpr, a.C, qw);
  get_param<VEC>(a.pre_b, 0.f, t, tpr, a.C, qb);
  bool live0 = look(first), live1 = look(first + step);
  fetch(0, first, live0);
  fetch(1, first + step, live1);
  soon = look(first + 2 * step);
  long long row = first;
  for (int k = 0; (long long)blockIdx.x * rpb + k * step < a.rows; ++k, row += step) {
    const bool in = row < a.rows, live = live0;
    const long long o = (in ? row : 0) * a.C;
    const uint8_t* slot = ring + (k & 1) * kStage;
    float2 s[H], u[H], g[H];
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    SS::get(slot, static_cast<const TS*>(a.s) + o, t, tpr, a.C, in, s);
    if (branch) SB::get(slot + SS::kBytes, static_cast<const TB*>(a.u) + o, t, tpr, a.C, live, u);
    if (gated) SB::get(slot + SS::kBytes + SB::kBytes, static_cast<const TB*>(a.gate) + o, t, tpr, a.C, live, g);
    float2 mu = make_float2(0.f, 0.f), mr = mu;
    if (branch) {
      if (a.post_w != nullptr) {
        mu = moments<VEC>(u, n, a, tpr, inv, sum);
#pragma unroll
        for (int e = 0; e < H; ++e) u[e] = fma2(mul2(u[e], both(mu.y)), pw[e], pb[e]);
      }
#pragma unroll
      for (int e = 0; e < H; ++e) {
        if (gated) u[e] = mul2(u[e], sigmoid(g[e]));
        const float2 r = fma2(ga[e], u[e], s[e]);
        s[e] = live ? r : s[e];
      }
      if (in) put_row<VEC>(static_cast<TS*>(a.r) + o, t, tpr, a.C, s);
    }
    if (a.pre_w != nullptr) {
      mr = moments<VEC>(s, n, a, tpr, inv, sum);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 x = fma2(mul2(s[e], both(mr.y)), qw[e], qb[e]);
        s[e] = live ? x : both(0.f);
      }
      if (in) put_row<VEC>(static_cast<TB*>(a.x) + o, t, tpr, a.C, s);
    }
    if (a.stats != nullptr && in && t == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = live ? make_float4(mu.x, mu.y, mr.x, mr.y) : make_float4(0.f, 0.f, 0.f, 0.f);
    live0 = live1;                            // what was read of this slot has been used: the row after next may take it
    live1 = soon;
    fetch(k, row + 2 * step, live1);
    soon = look(row + 3 * step);
  }
}

// Rows ahead in the backward: two, or one where 1024 threads' five tensors fill the shared memory.
constexpr int bwd_slots(int block) { return block > 512 ? 1 : 2; }

template <typename TS, typename TB, bool VEC, int BLOCK, int TPR>
__global__ void __launch_bounds__(BLOCK, BLOCK > 512 ? 1 : 512 / BLOCK) norm_bwd_kernel(const NormArgs a) {
  typedef Slot<TS, VEC, BLOCK> SS;
  typedef Slot<TB, VEC, BLOCK> SB;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kStage = 2 * SS::kBytes + 3 * SB::kBytes, NS = bwd_slots(BLOCK);
  float* acc_s = reinterpret_cast<float*>(ring);          // [rows of the CTA][5][C] when several share it
  __shared__ float2 red[2][32];
  RowSum sums{red, 0};
  const int tpr = TPR > 0 ? TPR : a.tpr, t = threadIdx.x & (tpr - 1), rpb = BLOCK / tpr;
  const float inv = 1.f / (float)a.C;
  const bool branch = a.u != nullptr, gated = a.gate != nullptr, pre = a.d_x != nullptr, thru = a.d_r != nullptr;
  const int n = mine<VEC>(t, tpr, a.C);
  float2 dga[H], dpw[H], dpb[H], dqw[H], dqb[H];
#pragma unroll
  for (int e = 0; e < H; ++e) dga[e] = dpw[e] = dpb[e] = dqw[e] = dqb[e] = both(0.f);
  const long long step = (long long)gridDim.x * rpb;
  const long long first = (long long)blockIdx.x * rpb + threadIdx.x / tpr;     // this thread's rows: first, first + step, ...
  bool soon;                                                                     // whether the row to be fetched next is valid
  auto look = [&](long long row) { return row < a.rows && (a.mask == nullptr || a.mask[row] != 0); };
  auto fetch = [&](int k, long long row, bool live) {
    uint8_t* slot = ring + (k % NS) * kStage;
    const long long o = (row < a.rows ? row : 0) * a.C;
    SS::fetch(slot, static_cast<const TS*>(a.s) + o, t, tpr, a.C, live);
    if (thru) SS::fetch(slot + SS::kBytes, static_cast<const TS*>(a.d_r) + o, t, tpr, a.C, row < a.rows);
    slot += 2 * SS::kBytes;
    if (branch) SB::fetch(slot, static_cast<const TB*>(a.u) + o, t, tpr, a.C, live);
    if (gated) SB::fetch(slot + SB::kBytes, static_cast<const TB*>(a.gate) + o, t, tpr, a.C, live);
    if (pre) SB::fetch(slot + 2 * SB::kBytes, static_cast<const TB*>(a.d_x) + o, t, tpr, a.C, live);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  bool live0 = look(first), live1 = look(first + step);
  fetch(0, first, live0);
  if (NS == 2) fetch(1, first + step, live1);
  soon = look(first + 2 * step);
  float4 nst = live0 ? *reinterpret_cast<const float4*>(a.stats + 4 * first) : make_float4(0.f, 0.f, 0.f, 0.f);
  long long row = first;
  for (int k = 0; (long long)blockIdx.x * rpb + k * step < a.rows; ++k, row += step) {
    const bool in = row < a.rows, live = live0;
    const long long o = (in ? row : 0) * a.C;
    const uint8_t* slot = ring + (k % NS) * kStage;
    float2 s[H], u[H], g[H], dr[H], dx[H];
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
    SS::get(slot, static_cast<const TS*>(a.s) + o, t, tpr, a.C, live, s);
    if (thru) {
      SS::get(slot + SS::kBytes, static_cast<const TS*>(a.d_r) + o, t, tpr, a.C, in, dr);
    } else {
#pragma unroll
      for (int e = 0; e < H; ++e) dr[e] = both(0.f);
    }
    slot += 2 * SS::kBytes;
    if (branch) SB::get(slot, static_cast<const TB*>(a.u) + o, t, tpr, a.C, live, u);
    if (gated) SB::get(slot + SB::kBytes, static_cast<const TB*>(a.gate) + o, t, tpr, a.C, live, g);
    if (pre) SB::get(slot + 2 * SB::kBytes, static_cast<const TB*>(a.d_x) + o, t, tpr, a.C, live, dx);
    const float4 st = nst;
    if (live1) nst = *reinterpret_cast<const float4*>(a.stats + 4 * (row + step));
    else nst = make_float4(0.f, 0.f, 0.f, 0.f);
    float2 w[H];
    // u -> uhat; y in w; s -> r; gate -> sigmoid
    if (branch) {
      float2 pb[H], ga[H];
      get_param<VEC>(a.post_w, 1.f, t, tpr, a.C, w);
      get_param<VEC>(a.post_b, 0.f, t, tpr, a.C, pb);
      get_param<VEC>(a.res_scale, 1.f, t, tpr, a.C, ga);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        if (a.post_w != nullptr) {
          u[e] = mul2(add2(u[e], both(-st.x)), both(st.y));
          w[e] = fma2(u[e], w[e], pb[e]);
        } else {
          w[e] = u[e];
        }
        g[e] = gated ? sigmoid(g[e]) : both(1.f);
        s[e] = fma2(ga[e], mul2(g[e], w[e]), s[e]);
      }
    }
    if (pre) {
      float2 qw[H], mx = both(0.f), my = both(0.f);
      get_param<VEC>(a.pre_w, 1.f, t, tpr, a.C, qw);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        s[e] = mul2(add2(s[e], both(-st.z)), both(st.w));         // rhat
        dqw[e] = fma2(dx[e], s[e], dqw[e]);
        dqb[e] = add2(dqb[e], dx[e]);
        dx[e] = mul2(dx[e], qw[e]);
        mx = add2(mx, dx[e]);
        my = fma2(dx[e], s[e], my);
      }
      const float2 m = sums(make_float2(mx.x + mx.y, my.x + my.y), tpr);
      const float c1 = a.rms || (VEC && n == 0) ? 0.f : m.x * inv, c2 = VEC && n == 0 ? 0.f : m.y * inv;
#pragma unroll
      for (int e = 0; e < H; ++e) {                               // a masked row has st.w = 0
        float2 d = fma2(s[e], both(-c2), add2(dx[e], both(-c1)));
        if (!VEC) d = mul2(d, there<VEC>(e, n));
        dr[e] = fma2(both(st.w), d, dr[e]);
      }
    }
    if (a.d_s != nullptr && in) put_row<VEC>(static_cast<TS*>(a.d_s) + o, t, tpr, a.C, dr);
    if (branch) {
      float2 ga[H], pw[H], mx = both(0.f), my = both(0.f);
      get_param<VEC>(a.res_scale, 1.f, t, tpr, a.C, ga);
      get_param<VEC>(a.post_w, 1.f, t, tpr, a.C, pw);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 d = live ? dr[e] : both(0.f), gy = mul2(g[e], w[e]);
        dga[e] = fma2(d, gy, dga[e]);
        const float2 dgy = mul2(d, ga[e]), dy = mul2(dgy, g[e]);
        g[e] = mul2(mul2(dgy, gy), add2(both(1.f), make_float2(-g[e].x, -g[e].y)));
        dpw[e] = fma2(dy, u[e], dpw[e]);
        dpb[e] = add2(dpb[e], dy);
        w[e] = a.post_w != nullptr ? mul2(dy, pw[e]) : dy;
        mx = add2(mx, w[e]);
        my = fma2(w[e], u[e], my);
      }
      if (a.d_gate != nullptr && in) put_row<VEC>(static_cast<TB*>(a.d_gate) + o, t, tpr, a.C, g);
      if (a.post_w != nullptr) {
        const float2 m = sums(make_float2(mx.x + mx.y, my.x + my.y), tpr);
        const float e1 = a.rms ? 0.f : m.x * inv, e2 = m.y * inv;
#pragma unroll
        for (int e = 0; e < H; ++e) w[e] = mul2(both(st.y), fma2(u[e], both(-e2), add2(w[e], both(-e1))));
      }
      if (a.d_u != nullptr && in) put_row<VEC>(static_cast<TB*>(a.d_u) + o, t, tpr, a.C, w);
    }
    live0 = live1;
    live1 = soon;
    if (NS == 2) fetch(k, row + 2 * step, live1);
    else fetch(k, row + step, live0);
    soon = look(row + 3 * step);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();                           // the ring's memory now takes the sums
  // the CTA's rows in order, then one line of sums per CTA
  float* out = a.part + (size_t)blockIdx.x * 5 * a.C;
  float2* sum[5] = {dga, dpw, dpb, dqw, dqb};
  if (rpb == 1) {
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = col<VEC>(t, tpr, e);
        if (c < a.C) out[k * a.C + c] = e & 1 ? sum[k][e / 2].y : sum[k][e / 2].x;
      }
    return;
  }
  // every row's sums side by side, then one thread a column adds them in row order
  const int q = threadIdx.x / tpr, line = 5 * a.C;
#pragma unroll
  for (int k = 0; k < 5; ++k)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = col<VEC>(t, tpr, e);
      if (c < a.C) acc_s[q * line + k * a.C + c] = e & 1 ? sum[k][e / 2].y : sum[k][e / 2].x;
    }
  __syncthreads();
  for (int c = threadIdx.x; c < line; c += BLOCK) {
    float x = acc_s[c];
    for (int r = 1; r < rpb; ++r) x += acc_s[r * line + c];
    out[c] = x;
  }
}

// Sums over the CTAs' lines: 32 interleaved partial sums a column, added in order.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* part, int lines, int C, float* const o0, float* const o1,
                                                           float* const o2, float* const o3, float* const o4) {
  __shared__ float red[32][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5, n = 5 * C;
  float x = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int l = k; l < lines; l += 32) x += part[(size_t)l * n + c];
  }
  red[k][threadIdx.x & 31] = x;
  __syncthreads();
  if (k == 0 && c < n) {
    for (int q = 1; q < 32; ++q) x += red[q][threadIdx.x];
    const int which = c / C;
    float* p = which == 0 ? o0 : (which == 1 ? o1 : (which == 2 ? o2 : (which == 3 ? o3 : o4)));
    if (p != nullptr) p[c - which * C] = x;
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool params_aligned(const NormArgs& a) {
  return is_aligned(a.res_scale, 16) && is_aligned(a.post_w, 16) && is_aligned(a.post_b, 16) && is_aligned(a.pre_w, 16) &&
         is_aligned(a.pre_b, 16);
}

int norm_tpr(int C) {
  int t = 1;
  while (t * E < C) t *= 2;
  return t;
}
int norm_block(int tpr) { return tpr < 256 ? 256 : tpr; }
// CTAs of the backward: all that are resident at once (512 threads an SM, for
// 128 registers a thread: 40 sums, a row and the next row), as each leaves a
// line of parameter gradients.
int norm_bwd_grid(long long rows, int C) {
  const int block = norm_block(norm_tpr(C)), rpb = block / norm_tpr(C);
  const long long need = (rows + rpb - 1) / rpb, most = 148 * (block > 512 ? 1 : 512 / block);
  return (int)(need < most ? need : most);
}

template <typename TS, typename TB, bool VEC, int BLOCK, int TPR>
cudaError_t norm_launch(const NormArgs& a, bool bwd, int grid, cudaStream_t st) {
  const int ks = Slot<TS, VEC, BLOCK>::kBytes, kb = Slot<TB, VEC, BLOCK>::kBytes;
  size_t smem = bwd ? (size_t)bwd_slots(BLOCK) * (2 * ks + 3 * kb) : 2 * (size_t)(ks + 2 * kb);
  const size_t sums = bwd && BLOCK > a.tpr ? (size_t)(BLOCK / a.tpr) * 5 * a.C * sizeof(float) : 0;
  if (smem < sums) smem = sums;
  const cudaError_t e = allow_max_smem(bwd ? reinterpret_cast<const void*>(&norm_bwd_kernel<TS, TB, VEC, BLOCK, TPR>)
                                           : reinterpret_cast<const void*>(&norm_fwd_kernel<TS, TB, VEC, BLOCK, TPR>));
  if (e != cudaSuccess) return e;
  if (bwd) norm_bwd_kernel<TS, TB, VEC, BLOCK, TPR><<<grid, BLOCK, smem, st>>>(a);
  else norm_fwd_kernel<TS, TB, VEC, BLOCK, TPR><<<grid, BLOCK, smem, st>>>(a);
  return cudaGetLastError();
}
// Threads a row known at compile time where a row is a warp's (C of 129 to 256) or the
// CTA's (C beyond 1024): columns become constant offsets, sums unroll.  Forward / backward
// in us of a float32 stream with a bfloat16 branch, compiled in against passed, cold:
//   100000 x 200: 70 / 129 against 78 / 141
// The other widths are passed.  Up to 128 channels little is lost (156250 x 128: 66 / 109
// against 64 / 117), beyond 256 more (52083 x 384: 86 / 150 against 117 / 170,
// 19531 x 1024: 72 / 135 against 94 / 150); not built.
template <typename TS, typename TB, bool VEC>
cudaError_t norm_launch(const NormArgs& a, bool bwd, int grid, cudaStream_t st) {
  switch (a.tpr) {
    case 1024: return norm_launch<TS, TB, VEC, 1024, 1024>(a, bwd, grid, st);
    case 512: return norm_launch<TS, TB, VEC, 512, 512>(a, bwd, grid, st);
    case 256: return norm_launch<TS, TB, VEC, 256, 256>(a, bwd, grid, st);
    case 32: return norm_launch<TS, TB, VEC, 256, 32>(a, bwd, grid, st);
    default: return norm_launch<TS, TB, VEC, 256, 0>(a, bwd, grid, st);
  }
}
template <typename TS, typename TB>
cudaError_t norm_launch(const NormArgs& a, bool vec, bool bwd, int grid, cudaStream_t st) {
  return vec ? norm_launch<TS, TB, true>(a, bwd, grid, st) : norm_launch<TS, TB, false>(a, bwd, grid, st);
}

fipa_status norm_args(const fipa_norm_dims* d, const fipa_norm_inputs* in, NormArgs* a) {
  if (d == nullptr || in == nullptr) return FIPA_ERR_INVALID_ARG;
  if (d->rows < 0 || d->C <= 0) return FIPA_ERR_INVALID_ARG;
  if ((d->stream_dtype != FIPA_F32 && d->stream_dtype != FIPA_BF16) ||
      (d->branch_dtype != FIPA_F32 && d->branch_dtype != FIPA_BF16) ||
      (d->norm != FIPA_NORM_LAYER && d->norm != FIPA_NORM_RMS) || !((float)d->eps > 0.f) || !isfinite((float)d->eps))
    return FIPA_ERR_INVALID_ARG;
  if (d->C > kNormMaxC) return FIPA_ERR_UNSUPPORTED;
  const bool u = in->u != nullptr || d->rows == 0;           // an empty tensor may have no address
  if (d->rows > 0 && in->s == nullptr) return FIPA_ERR_INVALID_ARG;
  if (!u && (in->gate || in->res_scale || in->post_w)) return FIPA_ERR_INVALID_ARG;
  if ((in->post_b && !in->post_w) || (in->pre_b && !in->pre_w)) return FIPA_ERR_INVALID_ARG;
  if (!u && !in->pre_w) return FIPA_ERR_INVALID_ARG;
  const size_t es = d->stream_dtype == FIPA_F32 ? 4 : 2, eb = d->branch_dtype == FIPA_F32 ? 4 : 2;
  if (!is_aligned(in->s, es) || !is_aligned(in->u, eb) || !is_aligned(in->gate, eb) || !is_aligned(in->res_scale, 4) ||
      !is_aligned(in->post_w, 4) || !is_aligned(in->post_b, 4) || !is_aligned(in->pre_w, 4) || !is_aligned(in->pre_b, 4))
    return FIPA_ERR_INVALID_ARG;
  *a = NormArgs{};
  a->s = in->s; a->u = in->u; a->gate = in->gate; a->mask = in->mask;
  a->res_scale = in->res_scale; a->post_w = in->post_w; a->post_b = in->post_b; a->pre_w = in->pre_w; a->pre_b = in->pre_b;
  a->rows = d->rows;
  a->C = d->C;
  a->tpr = norm_tpr(d->C);
  a->rms = d->norm == FIPA_NORM_RMS;
  a->eps = (float)d->eps;
  return FIPA_OK;
}

cudaError_t norm_dispatch(const fipa_norm_dims* d, const NormArgs& a, bool vec, bool bwd, int grid, cudaStream_t st) {
  const bool s32 = d->stream_dtype == FIPA_F32, b32 = d->branch_dtype == FIPA_F32;
  if (s32 && b32) return norm_launch<float, float>(a, vec, bwd, grid, st);
  if (s32) return norm_launch<float, __nv_bfloat16>(a, vec, bwd, grid, st);
  if (b32) return norm_launch<__nv_bfloat16, float>(a, vec, bwd, grid, st);
  return norm_launch<__nv_bfloat16, __nv_bfloat16>(a, vec, bwd, grid, st);
}

}  // namespace
}  // namespace fipa

FIPA_API fipa_status fipa_norm_residual(const fipa_norm_dims* d, const fipa_norm_inputs* in, void* r, void* x, float* stats,
                                        void* stream) {
  using namespace fipa;
  NormArgs a;
  const fipa_status st = norm_args(d, in, &a);
  if (st != FIPA_OK) return st;
  if (d->rows == 0) return FIPA_OK;
  if ((r == nullptr) != (in->u == nullptr) || (x == nullptr) != (in->pre_w == nullptr)) return FIPA_ERR_INVALID_ARG;
  const size_t es = d->stream_dtype == FIPA_F32 ? 4 : 2, eb = d->branch_dtype == FIPA_F32 ? 4 : 2;
  if (!is_aligned(r, es) || !is_aligned(x, eb) || !is_aligned(stats, 16)) return FIPA_ERR_INVALID_ARG;
  a.r = r;
  a.x = x;
  a.stats = stats;
  const bool vec = a.C % E == 0 && params_aligned(a) && is_aligned(a.s, 16) && is_aligned(a.u, 16) && is_aligned(a.gate, 16) &&
                   is_aligned(r, 16) && is_aligned(x, 16);
  const int rpb = norm_block(a.tpr) / a.tpr;
  const long long need = (a.rows + rpb - 1) / rpb, most = 148 * fwd_ctas(norm_block(a.tpr));
  return norm_dispatch(d, a, vec, false, (int)(need < most ? need : most), static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FIPA_OK
             : FIPA_ERR_CUDA;
}

FIPA_API fipa_status fipa_norm_residual_backward_workspace_size(const fipa_norm_dims* d, size_t* bytes) {
  if (d == nullptr || bytes == nullptr || d->rows < 0 || d->C <= 0) return FIPA_ERR_INVALID_ARG;
  if (d->C > fipa::kNormMaxC) return FIPA_ERR_UNSUPPORTED;
  *bytes = (size_t)fipa::norm_bwd_grid(d->rows, d->C) * 5 * d->C * sizeof(float);
  return FIPA_OK;
}

FIPA_API fipa_status fipa_norm_residual_backward(const fipa_norm_dims* d, const fipa_norm_inputs* in, const float* stats,
                                                 const void* d_r, const void* d_x, const fipa_norm_grads* g,
                                                 void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fipa;
  NormArgs a;
  const fipa_status st = norm_args(d, in, &a);
  if (st != FIPA_OK) return st;
  if (g == nullptr) return FIPA_ERR_INVALID_ARG;
  if (d_x != nullptr && in->pre_w == nullptr) return FIPA_ERR_INVALID_ARG;
  if (d->rows > 0 && stats == nullptr) return FIPA_ERR_INVALID_ARG;
  if ((d->rows > 0 && ((g->u && !in->u) || (g->gate && !in->gate))) || (g->res_scale && !in->res_scale) || (g->post_w && !in->post_w) ||
      (g->post_b && !in->post_b) || (g->pre_w && !in->pre_w) || (g->pre_b && !in->pre_b))
    return FIPA_ERR_INVALID_ARG;
  const size_t es = d->stream_dtype == FIPA_F32 ? 4 : 2, eb = d->branch_dtype == FIPA_F32 ? 4 : 2;
  if (!is_aligned(stats, 16) || !is_aligned(d_r, es) || !is_aligned(d_x, eb) || !is_aligned(g->s, es) ||
      !is_aligned(g->u, eb) || !is_aligned(g->gate, eb) || !is_aligned(g->res_scale, 4) || !is_aligned(g->post_w, 4) ||
      !is_aligned(g->post_b, 4) || !is_aligned(g->pre_w, 4) || !is_aligned(g->pre_b, 4))
    return FIPA_ERR_INVALID_ARG;
  size_t need = 0;
  fipa_norm_residual_backward_workspace_size(d, &need);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FIPA_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return FIPA_ERR_INVALID_ARG;
  a.stats = const_cast<float*>(stats);
  a.d_r = d_r;
  a.d_x = d_x;
  a.d_s = g->s;
  a.d_u = g->u;
  a.d_gate = g->gate;
  a.part = static_cast<float*>(workspace);
  const bool vec = a.C % E == 0 && params_aligned(a) && is_aligned(a.s, 16) && is_aligned(a.u, 16) && is_aligned(a.gate, 16) &&
                   is_aligned(d_r, 16) && is_aligned(d_x, 16) && is_aligned(g->s, 16) && is_aligned(g->u, 16) &&
                   is_aligned(g->gate, 16);
  const int grid = norm_bwd_grid(d->rows, d->C);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (grid > 0 && norm_dispatch(d, a, vec, true, grid, s) != cudaSuccess) return FIPA_ERR_CUDA;
  norm_reduce_kernel<<<(5 * d->C + 31) / 32, 1024, 0, s>>>(a.part, grid, d->C, g->res_scale, g->post_w, g->post_b, g->pre_w,
                                                         g->pre_b);
  return cudaGetLastError() == cudaSuccess ? FIPA_OK : FIPA_ERR_CUDA;
}

// window_tf32.cu -- window attention with sinks on float32 tensors, forward and
// backward, with matrix instructions on split operands (m16n8k8, tf32).
//
// The mathematics, the row and column numbering and the visibility rule are
// those of window.h; the work is divided as in window_mma.cu (a warp owns 16 rows
// or 16 keys and walks the 16-column groups that they see).  A float32 operand x
// travels as two tf32 numbers, hi = x rounded to 11 bits and lo = x - hi, of which
// the product takes the upper 11 bits: x is kept to 2^-21, and a product is the sum
// lo hi + hi lo + hi hi (lo lo is below 2^-22 of it; with hi cut off instead of
// rounded it is 2^-20, always of one sign, and gradients were off by 1.6e-6).  The tensor cores add in float32 but
// cut off what does not fit, which over hundreds of keys would drift by 2^-24 a
// step: the second products are summed over 16 columns at a time and added to the
// running sums on the CUDA cores, rounded to nearest.
//
// Three products of 16 x 8 x 8 replace 32 multiply-adds and 10 shared-memory loads
// of a CUDA-core tile (training step of 8 x 256 residues, 8 heads of 16: 52 us
// against 129).  Bound by the latency of the products: 8 warps an SM at 128
// channels, where shared memory holds one CTA, wait for the one before in two of
// three cycles; two warps a row block, one on the even and one on the odd groups of
// columns, and products unrolled past the ends of a width keep more in flight.
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

constexpr int T = kWinTile;                // rows and columns of a tile
constexpr int kStep = 2;                    // products between two looks at the width: apart from them the compiler interleaves the loads
constexpr int kThreads = 256;              // 4 x 16 rows, by two warps each: one takes the even groups of columns, one the odd

template <int DP>
struct Ft {
  static constexpr int ld = DP + 4;        // floats of a padded row: 16-byte units of neighbouring rows differ by an odd number
  static constexpr int elems = T * ld;
};

__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;      // to nearest, in fewer cycles than the conversion takes
  lo = __float_as_uint(x - __uint_as_float(hi));
}
struct A4 {
  uint32_t hi[4], lo[4];
};
struct B2 {
  uint32_t hi[2], lo[2];
};
__device__ __forceinline__ void mma1(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// Three sums side by side: one after the other they would wait for each other.
struct C3 {
  float x[3][4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k][e] = 0.f;
  }
  __device__ __forceinline__ void add(const A4& a, const B2& b) {
    mma1(x[0], a.lo, b.hi);
    mma1(x[1], a.hi, b.lo);
    mma1(x[2], a.hi, b.hi);
  }
  __device__ __forceinline__ float sum(int e) const { return (x[0][e] + x[1][e]) + x[2][e]; }
};
// 16 rows from r0, depth k0 .. k0+7 of a tile; 16 columns from n0 (two operands of 8).
template <int DP>
__device__ __forceinline__ void load_a(A4& a, uint32_t base, int r0, int k0, int lane) {
  uint32_t r[4];
  ldsm4(r, base + 4 * ((r0 + (lane & 15)) * Ft<DP>::ld + k0 + ((lane >> 4) << 2)));
#pragma unroll
  for (int e = 0; e < 4; ++e) split(__uint_as_float(r[e]), a.hi[e], a.lo[e]);
}
template <int DP>
__device__ __forceinline__ void load_b(B2 (&b)[2], uint32_t base, int n0, int k0, int lane) {
  uint32_t r[4];
  ldsm4(r, base + 4 * ((n0 + (lane & 7) + ((lane >> 4) << 3)) * Ft<DP>::ld + k0 + (((lane >> 3) & 1) << 2)));
#pragma unroll
  for (int e = 0; e < 4; ++e) split(__uint_as_float(r[e]), b[e >> 1].hi[e & 1], b[e >> 1].lo[e & 1]);
}
// The operand whose depth is rows k0 .. k0+7 of a tile: an accumulator holds columns
// 2c and 2c + 1 where an operand wants depths c and c + 4, so the rows come in that order.
template <int DP>
__device__ __forceinline__ void load_bt(B2& b, const float* tile, int k0, int n0, int lane) {
  const float* p = tile + (k0 + 2 * (lane & 3)) * Ft<DP>::ld + n0 + (lane >> 2);
  split(p[0], b.hi[0], b.lo[0]);
  split(p[Ft<DP>::ld], b.hi[1], b.lo[1]);
}
// An accumulator of 16 x 8 as the A operand of depth 8 (in the same order).
__device__ __forceinline__ void as_a(A4& a, const float (&x)[4]) {
  split(x[0], a.hi[0], a.lo[0]);
  split(x[2], a.hi[1], a.lo[1]);
  split(x[1], a.hi[2], a.lo[2]);
  split(x[3], a.hi[3], a.lo[3]);
}
// sum += A (16 x 16, as two accumulators) times rows k0 .. k0+15 of a tile
template <int DP>
__device__ __forceinline__ void add_product(float (&sum)[DP / 8][4], const A4 (&a)[2], const float* tile, int k0, int width, int lane) {
#pragma unroll
  for (int n = 0; n < DP / 8; ++n) {
    if (n % kStep == 0 && 8 * n >= width) break;
    C3 c;
    c.zero();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      B2 b;
      load_bt<DP>(b, tile, k0 + 8 * k, 8 * n, lane);
      c.add(a[k], b);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[n][e] += c.sum(e);
  }
}
// s (16 x 16) = rows r0 .. of tile A times rows n0 .. of tile B
template <int DP>
__device__ __forceinline__ void scores(float (&s)[2][4], uint32_t A, int r0, uint32_t B, int n0, int width, int lane) {
  C3 c[2];
  c[0].zero();
  c[1].zero();
#pragma unroll
  for (int k = 0; k < DP / 8; ++k) {
    if (k % kStep == 0 && 8 * k >= width) break;
    A4 a;
    B2 b[2];
    load_a<DP>(a, A, r0, 8 * k, lane);
    load_b<DP>(b, B, n0, 8 * k, lane);
    c[0].add(a, b[0]);
    c[1].add(a, b[1]);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[h][e] = c[h].sum(e);
}

struct Fsrc {
  const float* p;
  long long sn, sh;
  int width;
};
__device__ __forceinline__ Fsrc fsource(const void* base, long long sb, long long sn, long long sh, int width, int b, int h0) {
  return Fsrc{static_cast<const float*>(base) + b * sb + h0 * sh, sn, sh, width};
}
// A tile of rows; at(r) gives row r's elements, or null for a row of zeros.
template <int DP, typename At>
__device__ __forceinline__ void load_f(float* dst, const Fsrc& s, int rows, At at) {
  constexpr int N = 4, CH = DP / N;
  const int c = threadIdx.x % CH * N;
  const uint32_t d = smem_u32(dst) + c * 4;
#pragma unroll 4
  for (int r = threadIdx.x / CH; r < rows; r += kThreads / CH) {
    const float* p = at(r);
    const bool on = p != nullptr && c < s.width;
    cp16_zfill(d + r * Ft<DP>::ld * 4, on ? p + c : s.p, on);
  }
}
__device__ __forceinline__ void column_words(uint32_t* bits, const WinArgs& a, int b, const WinCols& c, int u0) {
  if (threadIdx.x < T) {
    const int u = u0 + threadIdx.x;
    const bool on = u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0);
    const uint32_t w = __ballot_sync(0xffffffffu, on);
    if ((threadIdx.x & 31) == 0) bits[threadIdx.x >> 5] = w;
  }
}
template <int DP, typename At>
__device__ __forceinline__ void store_f(const float (&acc)[DP / 8][4], int width, float f, int lane, At at) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bool keep;
    float* o = at(i, keep);
    if (o == nullptr) continue;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const int d = 8 * n + (lane & 3) * 2;
      if (d < width) o[d] = keep ? acc[n][2 * i] * f : 0.f;
      if (d + 1 < width) o[d + 1] = keep ? acc[n][2 * i + 1] * f : 0.f;
    }
  }
}

// Forward (BWD false) and row side of the backward (BWD true: delta, dq).
template <int DP, bool BWD>
__global__ void __launch_bounds__(kThreads) win_rows_tf32_kernel(const WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr int EL = Ft<DP>::elems;
  float* Qs = sm;
  float* Os = Qs + EL;                                     // dO
  float* Ks = Qs + (BWD ? 2 : 1) * EL;                     // two stages each
  float* Vs = Ks + 2 * EL;
  __shared__ uint32_t bits[2][2];
  __shared__ float2 odd[T];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7, col2 = (lane & 3) * 2;
  const int F = a.Nq * a.G, tiles = (F + T - 1) / T;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int f0 = tile * T, f1 = min(F, f0 + T), q0 = win_q0(a, b);
  const WinCols c = win_cols(a, q0, f0, f1);
  const Fsrc q = fsource(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Fsrc g_ = fsource(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, b, hkv * a.G);
  const Fsrc k = fsource(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = fsource(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  bool alive[2];
  WinRow row[2];
  float lse2[2] = {INFINITY, INFINITY}, del[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, qi = f / a.G, h = hkv * a.G + (f - qi * a.G), p = q0 + qi;
    alive[i] = f < f1 && win_alive(a, b, p);
    row[i] = win_row(a, c, p, alive[i]);
    if (BWD) {
      if (alive[i]) {
        const float x = a.lse[((long long)b * a.H + h) * a.Nq + qi];
        lse2[i] = x == -INFINITY ? INFINITY : x * kLog2e;            // a row that sees nothing: every p is 0
        const long long o = (((long long)b * a.Nq + qi) * a.H + h) * a.Dv;
        const float *y = static_cast<const float*>(a.out) + o, *z = static_cast<const float*>(a.d_out) + o;
        for (int d = lane & 3; d < a.Dv; d += 4) del[i] = fmaf(y[d], z[d], del[i]);
      }
      del[i] += __shfl_xor_sync(0xffffffffu, del[i], 1);
      del[i] += __shfl_xor_sync(0xffffffffu, del[i], 2);
      if (f < f1 && (lane & 3) == 0 && half == 0) a.delta[((long long)b * a.H + h) * a.Nq + qi] = del[i];
    }
  }
  const int ntile = __syncthreads_or(alive[0] || alive[1]) ? (c.n + T - 1) / T : 0;
  const Reach rc = reach(a, c, q0, f0 + 16 * warp, f1);
  auto load = [&](int t) {
    const int st = t & 1, u0 = t * T;
    auto keyed = [&](const Fsrc& s) {
      return [&, u0](int r) -> const float* {
        const int u = u0 + r;
        return u < c.n && (a.mask == nullptr || a.mask[(long long)b * a.Nk + c.key(u)] != 0) ? s.p + c.key(u) * s.sn : nullptr;
      };
    };
    load_f<DP>(Ks + st * EL, k, T, keyed(k));
    load_f<DP>(Vs + st * EL, v, T, keyed(v));
    column_words(bits[st], a, b, c, u0);
    cp_async_commit();
  };
  float acc[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  if (ntile > 0) {
    auto rows = [&](const Fsrc& s) {
      return [&](int r) -> const float* {
        const int f = f0 + r, i = f / a.G;
        return f < f1 && win_alive(a, b, q0 + i) ? s.p + i * s.sn + (f - i * a.G) * s.sh : nullptr;
      };
    };
    load_f<DP>(Qs, q, T, rows(q));
    if (BWD) load_f<DP>(Os, g_, T, rows(g_));
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
    const float *Kt = Ks + st * EL, *Vt = Vs + st * EL;
    const uint32_t w[2] = {bits[st][0], bits[st][1]};
#pragma unroll(DP <= 32 ? 2 : 1)
    for (int g = half; g < 4; g += 2) {
      const uint32_t wg = (w[g >> 1] >> ((g & 1) * 16)) & 0xffffu;
      if (wg == 0u || !rc.any(u0 + 16 * g)) continue;
      float s[2][4];
      scores<DP>(s, smem_u32(Qs), 16 * warp, smem_u32(Kt), 16 * g, a.D, lane);
      uint32_t ob[2] = {0xffffffffu, 0xffffffffu};
      if (wg != 0xffffu || !rc.all(u0 + 16 * g)) {
        ob[0] = (wg & row[0].sees(u0 + 16 * g)) >> col2;
        ob[1] = (wg & row[1].sees(u0 + 16 * g)) >> col2;
      }
      A4 pa[2];
      if (BWD) {
        float dp[2][4];
        scores<DP>(dp, smem_u32(Os), 16 * warp, smem_u32(Vt), 16 * g, a.Dv, lane);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = exp2f(fmaf(s[h][e], sc, -lse2[e >> 1])) * (dp[h][e] - del[e >> 1]);
            s[h][e] = ob[e >> 1] & (1u << (8 * h + (e & 1))) ? y : 0.f;
          }
        as_a(pa[0], s[0]);
        as_a(pa[1], s[1]);
        add_product<DP>(acc, pa, Kt, 16 * g, a.D, lane);
      } else {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[h][e] = ob[e >> 1] & (1u << (8 * h + (e & 1))) ? s[h][e] : -INFINITY;
            mx[e >> 1] = fmaxf(mx[e >> 1], s[h][e]);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        }
        if (__any_sync(0xffffffffu, (mx[0] - m[0]) * sc > kWinLag || (mx[1] - m[1]) * sc > kWinLag)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[i], mx[i]), f = mn == -INFINITY ? 0.f : exp2f((m[i] - mn) * sc);
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
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[h][e] = m[e >> 1] == -INFINITY ? 0.f : exp2f((s[h][e] - m[e >> 1]) * sc);
            l[e >> 1] += s[h][e];
          }
        as_a(pa[0], s[0]);
        as_a(pa[1], s[1]);
        add_product<DP>(acc, pa, Vt, 16 * g, a.Dv, lane);
      }
    }
    __syncthreads();
  }
  // the odd groups' sums join the even ones'
  float* red = sm + (16 * warp + (lane >> 2)) * Ft<DP>::ld + col2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (half == 0) continue;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) *reinterpret_cast<float2*>(red + 8 * i * Ft<DP>::ld + 8 * n) = make_float2(acc[n][2 * i], acc[n][2 * i + 1]);
    if ((lane & 3) == 0) odd[16 * warp + (lane >> 2) + 8 * i] = make_float2(m[i], l[i]);
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 o = odd[16 * warp + (lane >> 2) + 8 * i];
    const float mn = fmaxf(m[i], o.x);
    const float x = BWD ? 1.f : (m[i] == -INFINITY ? 0.f : exp2f((m[i] - mn) * sc)), y = BWD ? 1.f : (o.x == -INFINITY ? 0.f : exp2f((o.x - mn) * sc));
    m[i] = mn;
    l[i] = l[i] * x + o.y * y;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const float2 z = *reinterpret_cast<const float2*>(red + 8 * i * Ft<DP>::ld + 8 * n);
      acc[n][2 * i] = acc[n][2 * i] * x + z.x * y;
      acc[n][2 * i + 1] = acc[n][2 * i + 1] * x + z.y * y;
    }
  }
  if (BWD) {
    store_f<DP>(acc, a.D, a.scale, lane, [&](int i, bool& keep) -> float* {
      const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, qi = f / a.G;
      keep = alive[i] && lse2[i] != INFINITY;
      return f < f1 ? static_cast<float*>(a.d_q) + (((long long)b * a.Nq + qi) * a.H + hkv * a.G + (f - qi * a.G)) * a.D : nullptr;
    });
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float inv = alive[i] && l[i] != 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        acc[n][2 * i] *= inv;
        acc[n][2 * i + 1] *= inv;
      }
    }
    store_f<DP>(acc, a.Dv, 1.f, lane, [&](int i, bool& keep) -> float* {
      const int f = f0 + 16 * warp + (lane >> 2) + 8 * i, qi = f / a.G, h = hkv * a.G + (f - qi * a.G);
      keep = alive[i] && l[i] != 0.f;
      if (f >= f1) return nullptr;
      if (a.lse != nullptr && (lane & 3) == 0) a.lse[((long long)b * a.H + h) * a.Nq + qi] = keep ? fmaf(m[i], a.scale, logf(l[i])) : -INFINITY;
      return static_cast<float*>(a.out) + (((long long)b * a.Nq + qi) * a.H + h) * a.Dv;
    });
  }
}

// dk and dv, as win_bwd_k_mma_kernel (SINK: 16 keys that hold sinks over one chunk of the rows beyond the window).
template <int DP, bool SINK>
__global__ void __launch_bounds__(kThreads) win_keys_tf32_kernel(const WinArgs a) {
  constexpr int KR = SINK ? 16 : T, EL = Ft<DP>::elems;
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + KR * Ft<DP>::ld;
  float* Qs = Vs + KR * Ft<DP>::ld;
  float* Os = Qs + 2 * EL;
  __shared__ float slse[2][T], sdel[2][T];
  __shared__ int spos[2][T];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, half = threadIdx.x >> 7, col2 = (lane & 3) * 2;
  const int per = SINK ? (a.sinks + 15) / 16 * a.nchunk : (a.Nk + T - 1) / T;
  const int job = blockIdx.x % per, bh = blockIdx.x / per, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int chunk = SINK ? job % a.nchunk : -1, q0 = win_q0(a, b);
  const int j0 = SINK ? job / a.nchunk * 16 : job * T, j1 = min(a.Nk, j0 + KR) - 1, wj = SINK ? 0 : 16 * warp;
  const bool part = !SINK && a.nchunk > 0 && j0 < a.sinks;
  const int pl = SINK ? a.sink_pos : max(0, j0 - a.right);
  const int ph = SINK || (j0 < a.sinks && !part) ? a.Nk - 1 : min(a.Nk - 1, part ? a.sink_pos - 1 : j1 + a.left);
  const int il = max(pl - q0, 0), ih = min(ph - q0, a.Nq - 1);
  int fl = il * a.G, fh = (ih + 1) * a.G;
  if (ih < il) fl = fh = 0;
  if (SINK) {
    fl = max(fl, chunk * a.chunk_tiles * T);
    fh = min(fh, (chunk + 1) * a.chunk_tiles * T);
  }
  const Fsrc q = fsource(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Fsrc g_ = fsource(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, b, hkv * a.G);
  const Fsrc k = fsource(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = fsource(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  bool alive[2];
  int rlo[2], rhi[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = j0 + wj + (lane >> 2) + 8 * i;
    alive[i] = j <= j1 && win_alive(a, b, j);
    key_rows(a, q0, j, fl, fh, rlo[i], rhi[i]);
  }
  const int ka = j0 + wj, kb = min(ka + 15, j1);
  const int ntile = __syncthreads_or(alive[0] || alive[1]) && fh > fl ? (fh - fl + T - 1) / T : 0;
  float rl = 0.f, rd = 0.f;
  int rp = 0;
  auto load = [&](int t) {
    const int st = t & 1, f0 = fl + t * T;
    auto rows = [&](const Fsrc& s) {
      return [&, f0](int r) -> const float* {
        const int f = f0 + r, i = f / a.G;
        return f < fh && win_alive(a, b, q0 + i) ? s.p + i * s.sn + (f - i * a.G) * s.sh : nullptr;
      };
    };
    load_f<DP>(Qs + st * EL, q, T, rows(q));
    load_f<DP>(Os + st * EL, g_, T, rows(g_));
    cp_async_commit();
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
      slse[st][threadIdx.x] = rl == -INFINITY ? INFINITY : rl * kLog2e;
      sdel[st][threadIdx.x] = rd;
      spos[st][threadIdx.x] = rp;
    }
  };
  float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.f;
  const float sc = a.scale * kLog2e;
  if (ntile > 0) {
    auto keyed = [&](const Fsrc& s) {
      return [&](int r) -> const float* { return j0 + r <= j1 && win_alive(a, b, j0 + r) ? s.p + (j0 + r) * s.sn : nullptr; };
    };
    load_f<DP>(Ks, k, KR, keyed(k));
    load_f<DP>(Vs, v, KR, keyed(v));
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
    const float *Qt = Qs + st * EL, *Ot = Os + st * EL;
#pragma unroll(DP <= 32 ? 2 : 1)
    for (int g = SINK ? warp : half; g < 4; g += SINK ? 4 : 2) {
      if (fl + t * T + 16 * g >= fh || (SINK && (t & 1) != half)) break;
      const int pa = spos[st][16 * g], pb = spos[st][16 * g + 15];
      if (kb < ka || pb < ka - a.right || (pa > kb + a.left && ka >= a.sinks)) continue;
      uint32_t ob[2] = {0xffffffffu, 0xffffffffu};
      if (pa < kb - a.right || pb > ka + a.left) {
#pragma unroll
        for (int i = 0; i < 2; ++i) ob[i] = win_span(rlo[i] - t * T - 16 * g, rhi[i] - t * T - 16 * g) >> col2;
      }
      float s[2][4], dp[2][4];
      scores<DP>(s, smem_u32(Ks), wj, smem_u32(Qt), 16 * g, a.D, lane);
      scores<DP>(dp, smem_u32(Vs), wj, smem_u32(Ot), 16 * g, a.Dv, lane);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * g + 8 * h + col2 + (e & 1), i = e >> 1;
          const float x = exp2f(fmaf(s[h][e], sc, -slse[st][r]));
          s[h][e] = ob[i] & (1u << (8 * h + (e & 1))) ? x : 0.f;
          dp[h][e] = s[h][e] * (dp[h][e] - sdel[st][r]);
        }
      A4 x[2];
      as_a(x[0], s[0]);
      as_a(x[1], s[1]);
      add_product<DP>(dv, x, Ot, 16 * g, a.Dv, lane);
      as_a(x[0], dp[0]);
      as_a(x[1], dp[1]);
      add_product<DP>(dk, x, Qt, 16 * g, a.D, lane);
    }
    if (t + 1 < ntile) put(st ^ 1);
    __syncthreads();
  }
  if (SINK) {
    constexpr int OL = 2 * DP + 4;
    for (int w = 0; w < 8; ++w) {
      if (warp + 4 * half == w) {
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* o = sm + ((lane >> 2) + 8 * (e >> 1)) * OL + 8 * n + col2 + (e & 1);
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
      a.part[(((long long)bh * (a.nchunk + 1) + chunk + 1) * a.sinks + j) * wd + d] = on ? sm[r * OL + (d < a.D ? d : DP + d - a.D)] : 0.f;
    }
    return;
  }
  float* red = sm + (16 * warp + (lane >> 2)) * (2 * Ft<DP>::ld) + col2;
  if (half == 1) {
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* o = red + 8 * i * (2 * Ft<DP>::ld) + 8 * n;
        *reinterpret_cast<float2*>(o) = make_float2(dk[n][2 * i], dk[n][2 * i + 1]);
        *reinterpret_cast<float2*>(o + Ft<DP>::ld) = make_float2(dv[n][2 * i], dv[n][2 * i + 1]);
      }
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* o = red + 8 * i * (2 * Ft<DP>::ld) + 8 * n;
      const float2 x = *reinterpret_cast<const float2*>(o), y = *reinterpret_cast<const float2*>(o + Ft<DP>::ld);
      dk[n][2 * i] += x.x;
      dk[n][2 * i + 1] += x.y;
      dv[n][2 * i] += y.x;
      dv[n][2 * i + 1] += y.y;
    }
  if (part) {
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
  auto at = [&](void* base, int width, int i, bool& keep) -> float* {
    const int j = j0 + wj + (lane >> 2) + 8 * i;
    keep = alive[i];
    return j <= j1 && !(part && j < a.sinks) ? static_cast<float*>(base) + (((long long)b * a.Nk + j) * a.Hkv + hkv) * width : nullptr;
  };
  store_f<DP>(dk, a.D, a.scale, lane, [&](int i, bool& keep) { return at(a.d_k, a.D, i, keep); });
  store_f<DP>(dv, a.Dv, 1.f, lane, [&](int i, bool& keep) { return at(a.d_v, a.Dv, i, keep); });
}

template <int DP, bool BWD>
cudaError_t rows(const WinArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_rows_tf32_kernel<DP, BWD>));
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.B * a.Hkv * (((long long)a.Nq * a.G + T - 1) / T);
  win_rows_tf32_kernel<DP, BWD><<<(unsigned)grid, kThreads, (BWD ? 6 : 5) * Ft<DP>::elems * sizeof(float), s>>>(a);
  return cudaGetLastError();
}
template <int DP, bool SINK>
cudaError_t keys(const WinArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_keys_tf32_kernel<DP, SINK>));
  if (e != cudaSuccess) return e;
  const long long grid = (long long)a.B * a.Hkv * (SINK ? (long long)(a.sinks + 15) / 16 * a.nchunk : (a.Nk + T - 1) / T);
  win_keys_tf32_kernel<DP, SINK><<<(unsigned)grid, kThreads, (size_t)(2 * (SINK ? 16 : T) + 4 * T) * Ft<DP>::ld * sizeof(float), s>>>(a);
  return cudaGetLastError();
}
template <int DP>
cudaError_t bwd(const WinArgs& a, cudaStream_t s) {
  cudaError_t e = rows<DP, true>(a, s);
  if (e == cudaSuccess) e = keys<DP, false>(a, s);
  if (e == cudaSuccess && a.nchunk > 0) e = keys<DP, true>(a, s);
  if (e == cudaSuccess && a.nchunk > 0) e = launch_win_sink_reduce(a, 1, s);
  return e;
}
template <int DP>
cudaError_t run(const WinArgs& a, bool backward, cudaStream_t s) {
  return backward ? bwd<DP>(a, s) : rows<DP, false>(a, s);
}

}  // namespace

cudaError_t launch_win_f32(const WinArgs& in, bool backward, cudaStream_t s) {
  WinArgs a = in;
  if (backward) {
    const WinSinkPlan sp = win_sink_plan(a, T);
    a.nchunk = sp.nchunk;
    a.chunk_tiles = sp.chunk_tiles;
    a.sink_pos = sp.sink_pos;
  }
  const int w = a.D > a.Dv ? a.D : a.Dv;
  return w <= 16 ? run<16>(a, backward, s) : (w <= 32 ? run<32>(a, backward, s) : (w <= 64 ? run<64>(a, backward, s) : run<128>(a, backward, s)));
}

}  // namespace fipa

// window_mma.cuh -- shared by the bfloat16 window attention kernels: tiles in
// padded shared memory, asynchronous copies into them, m16n8k16 products on them.
#pragma once

#include "sm100.cuh"
#include "window.h"

namespace fipa {
namespace {

typedef __nv_bfloat16 bf16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kWinLag = 8.f;

// Rows are padded by 16 bytes, so that eight neighbouring rows start in different banks.
template <int DP>
struct Tile {
  static constexpr int ld = DP + 8;        // elements of a padded row
};

__device__ __forceinline__ void cp16_zfill(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Src {                               // one of the inputs, for one (b, hkv)
  const bf16* p;
  long long sn, sh;
  int width;
};
// A tile of rows x width elements, by `threads` threads of which this is `me`; at(r) gives row r's elements, or null for a row of zeros.
template <int DP, typename At>
__device__ __forceinline__ void load_tile(bf16* dst, const Src& s, int rows, int me, int threads, At at) {
  constexpr int CH = DP / 8;
  for (int e = me; e < rows * CH; e += threads) {
    const int r = e / CH, c = e % CH;
    const bf16* p = at(r);
    bf16* d = dst + r * Tile<DP>::ld + c * 8;
    const bool on = p != nullptr && c * 8 < s.width;
    cp16_zfill(smem_u32(d), on ? p + c * 8 : s.p, on);
  }
}
__device__ __forceinline__ Src source(const void* base, long long sb, long long sn, long long sh, int width, int b, int h0) {
  Src s;
  s.p = static_cast<const bf16*>(base) + b * sb + h0 * sh;
  s.sn = sn;
  s.sh = sh;
  s.width = width;
  return s;
}
// A walk over rows of two tensors: the row that this thread copies next.  Keys
// step by a fixed distance; the row f = i G + h of the queries carries from h to
// i.  Additions only: a division a row kept the copies behind the products.
struct Walk {
  const bf16 *p0, *p1;
  long long d0, d1, c0, c1;               // a step, and what a carry adds
  int i, h, di, dh, G;
  __device__ __forceinline__ void next() {
    p0 += d0;
    p1 += d1;
    i += di;
    h += dh;
    if (h >= G) {
      h -= G;
      ++i;
      p0 += c0;
      p1 += c1;
    }
  }
};
__device__ __forceinline__ Walk walk_queries(const WinArgs& a, const Src& q, const Src& g, int f, int step) {
  Walk w;
  w.G = a.G;
  w.i = f / a.G;
  w.h = f - w.i * a.G;
  w.di = step / a.G;
  w.dh = step - w.di * a.G;
  w.p0 = q.p + w.i * q.sn + w.h * q.sh;
  w.p1 = g.p + w.i * g.sn + w.h * g.sh;
  w.d0 = w.di * q.sn + w.dh * q.sh;
  w.d1 = w.di * g.sn + w.dh * g.sh;
  w.c0 = q.sn - a.G * q.sh;
  w.c1 = g.sn - a.G * g.sh;
  return w;
}
__device__ __forceinline__ Walk walk_keys(const Src& k, const Src& v, int j, int step) {
  Walk w;
  w.G = 0x7fffffff;
  w.h = 0;
  w.dh = 0;
  w.i = j;
  w.di = step;
  w.p0 = k.p + j * k.sn;
  w.p1 = v.p + j * v.sn;
  w.d0 = step * k.sn;
  w.d1 = step * v.sn;
  w.c0 = w.c1 = 0;
  return w;
}

// Rows first, first + step, ... below `end` of a padded tile (step = threads / pieces
// a row), of which those below n exist; valid(i): row i is not masked.
template <int DP, typename Valid>
__device__ __forceinline__ void copy_padded(bf16* d0, bf16* d1, int w0, int w1, Walk w, int first, int step, int end, int n, Valid valid) {
  const int c = threadIdx.x % (DP / 8) * 8;
  const bool in0 = c < w0, in1 = c < w1;
  const bf16 *a0 = w.p0, *a1 = w.p1;       // somewhere readable
  uint32_t o0 = smem_u32(d0) + (first * Tile<DP>::ld + c) * 2, o1 = smem_u32(d1) + (first * Tile<DP>::ld + c) * 2;
#pragma unroll 4
  for (int r = first; r < end; r += step) {
    const bool on = r < n && valid(w.i);
    cp16_zfill(o0, on && in0 ? w.p0 + c : a0, on && in0);
    cp16_zfill(o1, on && in1 ? w.p1 + c : a1, on && in1);
    o0 += step * Tile<DP>::ld * 2;
    o1 += step * Tile<DP>::ld * 2;
    w.next();
  }
}

// The 16 x 16 A operand at row r0, depth k0 of a tile; the 16 x 16 B operand of
// columns n0 .. n0+15 at depth k0 (rows = columns of the product), and the one
// whose rows are the product's depth.
template <int DP>
__device__ __forceinline__ uint32_t a_addr(uint32_t base, int r0, int k0, int lane) {
  return base + 2 * ((r0 + (lane & 15)) * Tile<DP>::ld + k0 + ((lane >> 4) << 3));
}
template <int DP>
__device__ __forceinline__ uint32_t b_addr(uint32_t base, int n0, int k0, int lane) {
  return base + 2 * ((n0 + (lane & 7) + ((lane >> 4) << 3)) * Tile<DP>::ld + k0 + (((lane >> 3) & 1) << 3));
}
template <int DP>
__device__ __forceinline__ uint32_t bt_addr(uint32_t base, int k0, int n0, int lane) {
  return base + 2 * ((k0 + (lane & 7) + (((lane >> 3) & 1) << 3)) * Tile<DP>::ld + n0 + ((lane >> 4) << 3));
}

// What two packed bfloat16 leave of the numbers that they stand for.
__device__ __forceinline__ uint32_t rest(uint32_t hi, float x, float y) {
  return pack(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}
// acc += (what the operand `hi` of 16 x 16 leaves of x0 and x1) times rows r .. r+15 of a tile, for 16 n16 columns
template <int DP>
__device__ __forceinline__ void add_rest(float (&acc)[DP / 8][4], const uint32_t (&hi)[4], const float (&x0)[4], const float (&x1)[4],
                                         uint32_t tile, int r, int n16, int lane) {
  const uint32_t lo[4] = {rest(hi[0], x0[0], x0[1]), rest(hi[1], x0[2], x0[3]), rest(hi[2], x1[0], x1[1]), rest(hi[3], x1[2], x1[3])};
#pragma unroll
  for (int n = 0; n < DP / 16; ++n) {
    if (n >= n16) break;
    uint32_t bf[4];
    ldsm4t(bf, bt_addr<DP>(tile, r, 16 * n, lane));
    mma(acc[2 * n], lo, bf[0], bf[1]);
    mma(acc[2 * n + 1], lo, bf[2], bf[3]);
  }
}

// Columns that neighbouring rows see: any of them, and all of them (n columns from u on).
struct Reach {
  int s_any, s_all, a_any, a_all, e_any, e_all;       // sinks [0, s), window [a, e)
  __device__ __forceinline__ bool any(int u, int n = 16) const { return u < s_any || (u + n > a_any && u < e_any); }
  __device__ __forceinline__ bool all(int u, int n = 16) const { return u + n <= s_all || (u >= a_all && u + n <= e_all); }
};
__device__ __forceinline__ Reach reach(const WinArgs& a, const WinCols& c, int q0, int f, int f1, int rows = 16) {
  const int lo = min(max(q0 + f / a.G, 0), a.Nk - 1), hi = min(max(q0 + (min(f + rows, f1) - 1) / a.G, 0), a.Nk - 1);
  const WinRow x = win_row(a, c, lo, true), y = win_row(a, c, hi, true);
  if (f >= f1) return Reach{0, 0, 0, 0, 0, 0};
  return Reach{y.s1, x.s1, x.w0, y.w0, y.w1, x.w1};
}

// Rows f, counted from fl and at most to fh, of the positions that see key j.
__device__ __forceinline__ void key_rows(const WinArgs& a, int q0, int j, int fl, int fh, int& lo, int& hi) {
  const long long x = ((long long)j - a.right - q0) * a.G - fl, y = ((long long)j + a.left + 1 - q0) * a.G - fl, n = fh - fl;
  lo = (int)(x < 0 ? 0 : (x < n ? x : n));
  hi = (int)(j < a.sinks ? n : (y < 0 ? 0 : (y < n ? y : n)));
}

// delta = dO.out comes from the rounded out and is off by eps = sum_j ds_j, which
// is 0 for the right delta; sum_j ds_j k_j is then off by eps sum_j p_j k_j.  Under
// windows of a few keys that error would be as large as all other roundings
// together.  Adds up eps over the four lanes of a row and takes the error back.
template <int DP>
__device__ __forceinline__ void take_back(float (&acc)[DP / 8][4], const float (&avg)[DP / 8][4], float (&eps)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    eps[i] += __shfl_xor_sync(0xffffffffu, eps[i], 1);
    eps[i] += __shfl_xor_sync(0xffffffffu, eps[i], 2);
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      acc[n][2 * i] = fmaf(-eps[i], avg[n][2 * i], acc[n][2 * i]);
      acc[n][2 * i + 1] = fmaf(-eps[i], avg[n][2 * i + 1], acc[n][2 * i + 1]);
    }
  }
}

// Writes a warp's 16 x DP sums as bfloat16 rows; at(i) is the row of this thread's half i, null: not written.
template <int DP, typename At>
__device__ __forceinline__ void store_rows(const float (&acc)[DP / 8][4], int width, const void* base, float f, int lane, At at) {
  const bool pair = (width & 1) == 0 && (reinterpret_cast<uintptr_t>(base) & 3) == 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bool keep;
    bf16* o = at(i, keep);
    if (o == nullptr) continue;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n) {
      const int d = 8 * n + (lane & 3) * 2;
      const float x = keep ? acc[n][2 * i] * f : 0.f, y = keep ? acc[n][2 * i + 1] * f : 0.f;
      if (pair && d < width) {
        *reinterpret_cast<uint32_t*>(o + d) = pack(x, y);
      } else {
        if (d < width) o[d] = __float2bfloat16_rn(x);
        if (d + 1 < width) o[d + 1] = __float2bfloat16_rn(y);
      }
    }
  }
}

}  // namespace
}  // namespace fipa

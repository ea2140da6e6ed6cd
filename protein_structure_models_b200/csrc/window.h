// window.h -- argument block, geometry and launchers of the window attention
// with sinks (fipa_window_attention and its backward).
//
// Query i of sample b stands at position p = q_start[b] + i.  It sees key j iff
//   0 <= j < Nk,  j <= p + right,  j >= p - left or j < sinks,  mask[b, j],
// and nothing at all if p is outside [0, Nk) or mask[b, p] is 0.
//
// The G = H / Hkv query heads that share a key head are rows of one problem:
// row f = i G + g of (b, hkv) is query i of head hkv G + g, so that a row tile
// covers few positions, its window is short, and K and V are read once a group.
//
// Columns of a row tile are virtual: u < s are the sinks that lie before the
// tile's window, then come the window's keys lo .. hi.  Both ranges that a row
// sees are ranges of u (a sink inside the window has u = j as well).
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace fipa {

struct WinArgs {
  const void *q, *k, *v;             // [B,N,heads,width] with element strides, width contiguous
  long long qb, qn, qh, kb, kn, kh, vb, vn, vh;
  void* out;                         // [B,Nq,H,Dv]
  float* lse;                        // [B,H,Nq] or null (forward), given (backward)
  const uint8_t* mask;               // [B,Nk] or null
  const int* q_start;                // [B] or null: Nk - Nq
  int B, Nq, Nk, H, Hkv, G, D, Dv;
  int left, right, sinks;            // left, right <= Nk; sinks <= min(Nk, kWinMaxSinks)
  float scale;
  // backward
  const void* d_out;                 // [B,Nq,H,Dv]
  void *d_q, *d_k, *d_v;             // contiguous
  float* delta;                      // [B,H,Nq] workspace: sum_c d_out out
  float* part;                       // sink partials, see win_sink_plan
  int nchunk, chunk_tiles;           // sink jobs: chunks, row tiles of 64 each
  int sink_pos;                      // first position that belongs to them
  int* status;
  unsigned long long timeout_ns;
  void* pad;                         // workspace of window_pad.cu
  int fine;                          // bfloat16: probabilities and dS enter their products as two numbers, see win_is_fine
};

constexpr int kWinMaxD = 128;
constexpr int kWinMaxSinks = 128;

// The gradient of a sink key sums over every later query, which one CTA would
// walk alone: the queries beyond the window of the key tiles that hold sinks
// (from position `sink_pos` on) are cut into `nchunk` chunks of `chunk_tiles`
// tiles of 64 rows, whose float32 partial sums (and the window's own) are added
// in chunk order by win_sink_reduce.
struct WinSinkPlan {
  int nchunk, chunk_tiles, sink_pos;
  size_t part_floats;
};
inline WinSinkPlan win_sink_plan(const WinArgs& a, int key_tile) {
  WinSinkPlan s{0, 0, 0, 0};
  const long long end = (long long)(a.sinks + key_tile - 1) / key_tile * key_tile;
  s.sink_pos = (int)(end < a.Nk ? end : a.Nk) + a.left;
  if (a.sinks <= 0 || s.sink_pos >= a.Nk) return s;          // the window reaches every position
  const long long tiles = ((long long)a.Nq * a.G + 63) / 64;
  // chunks of at least two tiles, and no more of them than are resident at once (three CTAs an SM)
  const long long jobs = (long long)a.B * a.Hkv * ((a.sinks + 15) / 16), most = 444 / jobs < 1 ? 1 : 444 / jobs;
  s.chunk_tiles = (int)((tiles + most - 1) / most);
  if (s.chunk_tiles < 2) s.chunk_tiles = 2;
  s.nchunk = (int)((tiles + s.chunk_tiles - 1) / s.chunk_tiles);
  s.part_floats = (size_t)a.B * a.Hkv * (s.nchunk + 1) * a.sinks * (a.D + a.Dv);
  return s;
}

constexpr int kWinTcRows = 128, kWinTcCols = 64;      // tile of window_tc.cu

// Sequences that one CTA holds as a whole (window_short.cu): rows (with the heads of a group) and keys.
constexpr int kWinShortRows = 512;
inline size_t win_short_smem(const WinArgs& a, int dp, bool backward) {
  const size_t F = ((size_t)a.Nq * a.G + 15) / 16 * 16, K = ((size_t)a.Nk + 31) / 32 * 32;
  return (2 * K + (backward ? 2 : 1) * F) * (dp + 8) * 2;
}
// Whether a CTA takes a whole sequence: two of them fit an SM, and there are that many.
//   64 x 128 x 8 heads of 16, window 63: 11.7 / 21 us against 14.0 / 38; 8 x 256 x 8: 14.5 / 27 against 8.9 / 24
inline bool win_short_takes(const WinArgs& a, bool backward) {
  const int w = a.D > a.Dv ? a.D : a.Dv;
  if (w > 64 || a.Nk > kWinShortRows || (long long)a.Nq * a.G > kWinShortRows || (long long)a.B * a.Hkv < 296) return false;
  return win_short_smem(a, w <= 16 ? 16 : (w <= 32 ? 32 : 64), backward) <= 100 * 1024;
}
// Probabilities and dS are rounded to bfloat16 for their products, which adds about
// as much to a result's error as the rounding of the result itself.  Where there
// are few rows there is time for a second product with what the rounding left, in
// window_mma.cu and window_step.cu; the other kernels take their calls as they
// are.  Error of a result against 64 bits, relative to its norm, over that of
// rounding it once (sizes from 300 to 614400 rows, 8 inputs each, the worst):
//   window_tc.cu     out 1.42, d_q 1.31 (dS as two numbers at any size), d_k 1.47, d_v 1.46
//   window_short.cu  out 1.40, d_q 1.46, d_k 1.47, d_v 1.45
// An element's error does not depend on how many rows there are.
inline int win_is_fine(const WinArgs& a, bool backward) { return (long long)a.B * a.Nq * a.H < (backward ? 16384 : 1024); }

// Whether bfloat16 q, k and v can be read 16 bytes at a time.
inline bool win_vec(const WinArgs& a) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  return ((p & 15) | ((a.qb | a.qn | a.qh | a.kb | a.kn | a.kh | a.vb | a.vn | a.vh | a.D | a.Dv) & 7)) == 0;
}
// Whether the columns of a forward call are split over warps and CTAs instead of
// its rows (window_step.cu).  That pays for a unit of 16 rows with many columns,
// while there are few units, or few rows in each; us, split against row tiles:
//   units  rows each  columns   width 32     64          128
//       8          1      256   6.7 / 10.1   6.4 / 13.4  7.1 / 18.9
//       8         16      128   9.9 / 6.8    10.5 / 8.9  10.9 / 12.3
//      60         16      200   9.6 / 9.8    10.3 / 12.8 13.0 / 17.7
//     400          1      190   7.6 / 8.3    9.1 / 11.1  16.4 / 30.5
//     400         16      384   20 / 13      26 / 21     44 / 56
//     600         16     1015   54 / 66      84 / 92     116 / 197
//     800         16      256   36 / 10      43 / 15     59 / 40
// Tensors off 16-byte boundaries are read as they are where the copies that row
// tiles need would cost more (10 rows of 110 channels, 31 of 3582 keys: 18 against 42).
inline bool win_step_takes(const WinArgs& a) {
  const long long F = (long long)a.Nq * a.G, units = (long long)a.B * a.Hkv * ((F + 15) / 16);
  if (!win_vec(a) && (F <= 4 || (F <= 16 && (a.Nk > 256 || units <= 148)))) return true;
  const long long cols = (long long)a.left + a.Nq + a.right + a.sinks, n = cols < a.Nk ? cols : a.Nk;
  if (units <= 148 && F <= 128) return n >= (F <= 4 ? 128 : 160);
  return (F <= 4 && n >= 128) || (F <= 16 && n >= (a.D > 64 || a.Dv > 64 ? 256 : 768)) || (F <= 32 && n >= 1536);
}

#ifdef __CUDACC__
__device__ __forceinline__ int win_q0(const WinArgs& a, int b) {
  if (a.q_start == nullptr) return a.Nk - a.Nq;
  return min(max(a.q_start[b], -a.Nq), a.Nk);       // beyond these no row is inside [0, Nk), and p cannot overflow
}

// Virtual columns of the row tile [f0, f1) of a sample with first position q0.
struct WinCols {
  int lo, hi, s, n;       // window keys lo..hi, sinks before it, columns in all (0: the tile sees nothing)
  __device__ __forceinline__ int key(int u) const { return u < s ? u : lo + (u - s); }
};
__device__ __forceinline__ WinCols win_cols(const WinArgs& a, int q0, int f0, int f1) {
  const int pl = max(q0 + f0 / a.G, 0), ph = min(q0 + (f1 - 1) / a.G, a.Nk - 1);
  WinCols c{0, -1, 0, 0};
  if (pl > ph) return c;
  c.lo = max(0, pl - a.left);
  c.hi = min(a.Nk - 1, ph + a.right);
  c.s = min(a.sinks, c.lo);
  c.n = c.s + c.hi - c.lo + 1;
  return c;
}
// The columns lo .. hi-1 of 32, as bits (a shift by 32 or more leaves nothing in PTX).
__device__ __forceinline__ uint32_t win_from(int x) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(0xffffffffu), "r"(max(x, 0)));
  return r;
}
__device__ __forceinline__ uint32_t win_span(int lo, int hi) { return win_from(lo) & ~win_from(hi); }
// The two column ranges of the row at position p: [0, s1) and [w0, w1).  Masks of
// 32 columns from u0 on: element by element the compiler makes a branch of each
// comparison, which took ten times as long as the rest of a tile.
struct WinRow {
  int s1, w0, w1;
  __device__ __forceinline__ uint32_t sees(int u0) const { return win_span(0, s1 - u0) | win_span(w0 - u0, w1 - u0); }
};
__device__ __forceinline__ WinRow win_row(const WinArgs& a, const WinCols& c, int p, bool alive) {
  WinRow r{0, 0, 0};
  if (!alive) return r;
  r.s1 = min(a.sinks, p + a.right + 1);
  r.w0 = max(p - a.left, c.lo) - c.lo + c.s;
  r.w1 = min(p + a.right, c.hi) - c.lo + c.s + 1;
  return r;
}
__device__ __forceinline__ bool win_alive(const WinArgs& a, int b, int p) {
  return p >= 0 && p < a.Nk && (a.mask == nullptr || a.mask[(long long)b * a.Nk + p] != 0);
}
#endif

size_t win_pad_bytes(const WinArgs& a, int es, bool backward);           // workspace of launch_win at a.pad; es: bytes of an element
cudaError_t launch_win(const WinArgs& a, int es, bool backward, cudaStream_t s);  // any widths and strides, by the following:
cudaError_t launch_win_f32(const WinArgs& a, bool backward, cudaStream_t s);     // float32 tensors
cudaError_t launch_win_fwd(const WinArgs& a, cudaStream_t s);            // bfloat16 tensors: one of the following
cudaError_t launch_win_bwd(const WinArgs& a, cudaStream_t s);
cudaError_t launch_win_step(const WinArgs& a, cudaStream_t s);           // few rows
cudaError_t launch_win_short(const WinArgs& a, bool backward, cudaStream_t s);   // many short sequences
cudaError_t launch_win_fwd_tc(const WinArgs& a, cudaStream_t s);         // wide windows
cudaError_t launch_win_bwd_q_tc(const WinArgs& a, cudaStream_t s);
cudaError_t launch_win_bwd_k_tc(const WinArgs& a, cudaStream_t s);
cudaError_t launch_win_sink_reduce(const WinArgs& a, int f32, cudaStream_t s);

constexpr int kWinTile = 64;           // rows and keys of a tile of the warp-level kernels

}  // namespace fipa

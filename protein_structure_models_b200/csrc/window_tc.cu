// window_tc.cu -- window attention with sinks on bfloat16 tensors, forward and
// backward, on the fifth-generation tensor cores (tcgen05, tensor memory).
//
// The mathematics, the row and column numbering and the visibility rule are
// those of window.h and window_mma.cu.  Three kernels of one shape: a CTA keeps
// 128 rows of one side in shared memory and streams the other side past them,
// 64 columns a tile; every accumulator has the CTA's 128 rows as tensor-memory
// lanes, so that one thread finishes one row of the scores:
//   forward     rows = queries, stream = keys and values:  O  += P V
//   row side    rows = queries, stream = keys and values:  dQ += dS K
//   key side    rows = keys,    stream = queries and dO:   dV += P^T dO,  dK += dS^T Q
// S (and dP = dO V^T) comes from shared memory into tensor memory; its thread
// turns the row into P or dS as bfloat16 in place of S, which is the A operand
// of the second product (half a step is 2^-8 of each element, the tensors' own
// rounding); the streamed tile is its B operand read along the other axis.  The
// running maximum, l, delta and all sums are float32.
//
// Bound by the matrix instructions: one of 128 x 64 x 16 takes about 106 cycles of
// its pipe whatever it holds, which the 64-column tiles pay 8 to 20 times; then by
// the waits between products and softmax.  Two CTAs an SM (one in the backward
// beyond 64 channels) and four stages of tiles (two in the forward beyond 64) keep
// both sides busy; 16384 residues, 8 heads on 2 of 64, 511 keys before: training step
// 283 us.  Warps 0-3 finish rows, warp 4 issues the matrix instructions, warps 5-6
// copy tiles (16-byte asynchronous copies into the 128-byte swizzle, zeros for masked
// and missing rows, which a tensor map could not leave out).  Every wait is bounded.
#include <math.h>

#include "kernels.h"
#include "window_mma.cuh"

namespace fipa {
namespace {

constexpr int kFwd = 0, kRowSide = 1, kKeySide = 2;
constexpr int kRows = kWinTcRows, kCols = kWinTcCols;
constexpr int kFinish = 128, kLoaders = 64, kThreads = kFinish + 32 + kLoaders;

template <int MODE, int DP>
struct Lay {
  static constexpr int CH = DP / 64;                     // 128-byte chunks of a row
  static constexpr int A = kRows * 128 * CH, B = kCols * 128 * CH;
  static constexpr int NA = MODE == kFwd ? 1 : 2;
  static constexpr int NS = DP == 128 && MODE == kFwd ? 2 : 4;   // stages of the stream
  static constexpr int tail = NA * A + NS * 2 * B;
  static constexpr int bars = tail, info = tail + 128;   // info: per stage 64 x {lse, delta, position} or two words of column bits
  static_assert((2 * NS + 7) * 8 + 8 <= info - bars, "barriers, tensor-memory address, abort flag");
  static constexpr int smem = info + NS * (MODE == kKeySide ? 768 : 8) + 1024;
  // Tensor memory.  Forward: S of even and odd tiles, P in place of S.  Row side: S,
  // dP, dS and what its rounding left.  Key side: S and dP, P and dS in their places.
  static constexpr int S = 0, dP = 64, acc0 = MODE == kRowSide ? 192 : 128, acc1 = acc0 + DP;
  static constexpr int need = MODE == kKeySide ? acc1 + DP : acc0 + DP;
  static constexpr int cols = need <= 256 ? 256 : 512;
  static constexpr int per_sm = DP == 64 || MODE == kFwd ? 2 : 1;
  static __device__ __forceinline__ int s_of(int t) { return MODE == kFwd ? S + 64 * (t & 1) : S; }
  static __device__ __forceinline__ int p_of(int t) { return MODE == kRowSide ? 128 : s_of(t); }
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

// This thread's part of a tile of rows: neighbouring threads take neighbouring
// 16-byte pieces (2^lg a row), so that a thread's piece and its place in the
// swizzle stay the same from row to row.
struct Piece {
  int lg, c, first, step;                  // pieces a row, this one, first row, rows between two of this thread's
  bool in0, in1, z0, z1;                   // inside the tensors' widths; inside them rounded up to 16 channels
  __device__ __forceinline__ Piece(int w0, int w1, int me, int threads) {
    const int w = w0 > w1 ? w0 : w1;
    lg = w <= 16 ? 1 : (w <= 32 ? 2 : (w <= 64 ? 3 : 4));
    c = me & ((1 << lg) - 1);
    first = me >> lg;
    step = threads >> lg;
    in0 = c * 8 < w0;
    in1 = c * 8 < w1;
    z0 = c * 8 < ((w0 + 15) & ~15);
    z1 = c * 8 < ((w1 + 15) & ~15);
  }
};
// Rows first, first + step, ... below `end` of a tile of `rows`, of which those below n exist; valid(i): row i is not masked.
template <typename Valid>
__device__ __forceinline__ void copy_rows(uint32_t d0, uint32_t d1, const Piece& pc, Walk w, int rows, int end, int n, Valid valid) {
  const uint32_t chunk = (uint32_t)(pc.c >> 3) * rows * 128;
  const bf16 *a0 = w.p0, *a1 = w.p1;       // somewhere readable
#pragma unroll 4
  for (int r = pc.first; r < end; r += pc.step) {
    const bool on = r < n && valid(w.i);
    const uint32_t o = chunk + (uint32_t)r * 128 + (uint32_t)(((pc.c & 7) ^ (r & 7)) << 4);
    if (pc.z0) cp16_zfill(d0 + o, on && pc.in0 ? w.p0 + pc.c * 8 : a0, on && pc.in0);
    if (pc.z1) cp16_zfill(d1 + o, on && pc.in1 ? w.p1 + pc.c * 8 : a1, on && pc.in1);
    w.next();
  }
}

// Whether the phase is over, without waiting for it.
__device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > timeout_ns) break;
}

// Row r of a 128-lane accumulator, `width` columns from col on, times f, as bfloat16 (keep) or zeros.
__device__ __forceinline__ void write_row(uint32_t trow, int col, int width, float f, bool read, bool keep, bf16* o) {
  for (int c0 = 0; c0 < width; c0 += 32) {               // every lane of the warp takes part in the load
    uint32_t v[32];
    if (read) {
      tmem_ld32(trow + (uint32_t)(col + c0), v);
      tmem_ld_wait();
    }
    if (o == nullptr) continue;
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      if (c0 + e >= width) break;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = keep ? pack(__uint_as_float(v[e + 2 * k]) * f, __uint_as_float(v[e + 2 * k + 1]) * f) : 0u;
      *reinterpret_cast<uint4*>(o + c0 + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int MODE, int DP>
__global__ void __launch_bounds__(kThreads, (Lay<MODE, DP>::per_sm)) win_tc_kernel(const WinArgs a) {
  typedef Lay<MODE, DP> L;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* empty = full + NS;
  // Two of each: even and odd tiles.  The products run up to a tile ahead of the
  // rows, so in the forward a warp may finish tile t + 1 while another is still at
  // t: on one barrier its arrivals would stand for the other's, and P(t) V would read
  // scores that are not yet probabilities.
  uint64_t* s_full = empty + NS;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* drained = pv_done + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(drained + 1);
  int* abort_flag = reinterpret_cast<int*>(slot + 1);
  const uint32_t sA = smem_u32(smem), sB = sA + L::NA * L::A;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kRowsAreQueries = MODE != kKeySide;

  // what this CTA owns: 128 rows f (queries) or 128 keys j, and its stream [0, n)
  const int F = a.Nq * a.G, all = kRowsAreQueries ? F : a.Nk, tiles = (all + kRows - 1) / kRows;
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles, b = bh / a.Hkv, hkv = bh - b * a.Hkv;
  const int r0 = tile * kRows, r1 = min(all, r0 + kRows), q0 = win_q0(a, b);
  const bool split = !kRowsAreQueries && tile == 0 && a.nchunk > 0;       // key tile 0 holds the sinks
  WinCols c{0, -1, 0, 0};
  int fl = 0, n;
  if (kRowsAreQueries) {
    c = win_cols(a, q0, r0, r1);
    n = c.n;
  } else {
    const int pl = max(0, r0 - a.right);
    const int ph = min(a.Nk - 1, split ? a.sink_pos - 1 : (r0 < a.sinks ? a.Nk - 1 : r1 - 1 + a.left));
    const int il = max(pl - q0, 0), ih = min(ph - q0, a.Nq - 1);
    fl = il * a.G;
    n = ih < il ? 0 : (ih + 1) * a.G - fl;
  }
  const Src q = source(a.q, a.qb, a.qn, a.qh, a.D, b, hkv * a.G);
  const Src g = source(a.d_out, (long long)a.Nq * a.H * a.Dv, (long long)a.H * a.Dv, a.Dv, a.Dv, b, hkv * a.G);
  const Src k = source(a.k, a.kb, a.kn, a.kh, a.D, b, hkv), v = source(a.v, a.vb, a.vn, a.vh, a.Dv, b, hkv);
  const uint8_t* mask = a.mask == nullptr ? nullptr : a.mask + (long long)b * a.Nk;
  auto key_valid = [&](int j) { return mask == nullptr || mask[j] != 0; };
  auto query_valid = [&](int i) { return q0 + i >= 0 && q0 + i < a.Nk && key_valid(q0 + i); };
  // this thread's row
  bool alive = false;
  int mine = r0 + (int)threadIdx.x, pos = 0;
  if (threadIdx.x < kFinish && mine < r1) {
    pos = kRowsAreQueries ? q0 + mine / a.G : mine;
    alive = win_alive(a, b, pos);
  }
  const int ntile = __syncthreads_or(alive) ? (n + kCols - 1) / kCols : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], kLoaders);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kFinish);
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
    *abort_flag = 0;
  }
  if (warp == 4) {
    tmem_alloc(slot, L::cols);
    tmem_relinquish();
  }
  if (ntile > 0) {
    const int me = threadIdx.x < 128 ? (int)threadIdx.x : 1 << 20;        // the first 128 threads
    const Piece pc(a.D, MODE == kFwd ? 0 : a.Dv, me, 128);
    const int r = min(r0 + pc.first, r1 - 1);
    if (kRowsAreQueries) copy_rows(sA, sA + L::A, pc, walk_queries(a, q, MODE == kFwd ? q : g, r, pc.step), kRows, kRows, r1 - r0, query_valid);
    else copy_rows(sA, sA + L::A, pc, walk_keys(k, v, r, pc.step), kRows, kRows, r1 - r0, key_valid);
    cp_async_wait_all();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;
  const WaitCtx wc{abort_flag, a.status, a.timeout_ns};
  const float sc = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f, lse2 = INFINITY, del = 0.f;
  float2 eps = both(0.f);

  if (warp >= 5) {
    // ------------------------------------------------------------- copies
    const int me = threadIdx.x - 160;
    const Piece pc(a.D, a.Dv, me, kLoaders);
    auto landed = [&](int t) {                              // this thread's part of tile t is in place
      fence_proxy_async_smem();
      mbar_arrive(&full[t % NS]);
    };
    for (int t = 0; t <= ntile; ++t) {
      bool told = t == 0;
      if (t < ntile) {
        const int st = t % NS, u0 = t * kCols;
        const uint32_t ph = ((t / NS) & 1) ^ 1u;
        if (!__all_sync(0xffffffffu, test(&empty[st], ph))) {
          // the products may need the last tile before they give this place back
          if (!told) {
            cp_wait<0>();
            landed(t - 1);
            told = true;
          }
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ph, wc, 81))) break;
        }
        const uint32_t d0 = sB + st * 2 * L::B;
        uint8_t* inf = smem + L::info + st * (MODE == kKeySide ? 768 : 8);
        if (kRowsAreQueries) {
          // sinks first, then the window; a tile may hold the seam
          const int ns = min(max(c.s - u0, 0), kCols);
          if (ns > 0) copy_rows(d0, d0 + L::B, pc, walk_keys(k, v, min(u0 + pc.first, a.Nk - 1), pc.step), kCols, ns, ns, key_valid);
          if (ns < kCols) {
            Piece pw = pc;
            while (pw.first < ns) pw.first += pw.step;
            copy_rows(d0, d0 + L::B, pw, walk_keys(k, v, min(c.key(u0 + pw.first), a.Nk - 1), pw.step), kCols, kCols, n - u0, key_valid);
          }
          const int u = u0 + me;
          const bool on = u < n && key_valid(c.key(u));
          const uint32_t w = __ballot_sync(0xffffffffu, on);
          if (lane == 0) reinterpret_cast<uint32_t*>(inf)[me >> 5] = w;
        } else {
          copy_rows(d0, d0 + L::B, pc, walk_queries(a, q, g, min(fl + u0 + pc.first, fl + n - 1), pc.step), kCols, kCols, n - u0, query_valid);
          const int f = fl + u0 + me, i = f / a.G;
          float x = -INFINITY, d = 0.f;
          if (u0 + me < n && win_alive(a, b, q0 + i)) {
            const long long o = ((long long)b * a.H + hkv * a.G + (f - i * a.G)) * a.Nq + i;
            x = a.lse[o];
            d = a.delta[o];
          }
          reinterpret_cast<float*>(inf)[me] = x == -INFINITY ? INFINITY : x * kLog2e;     // not there, or sees nothing: every p is 0
          reinterpret_cast<float*>(inf)[64 + me] = d;
          reinterpret_cast<int*>(inf)[128 + me] = q0 + i;
        }
        cp_async_commit();
        if (told) continue;
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      if (!told) landed(t - 1);
    }
    cp_async_wait_all();
  } else if (warp == 4) {
    // ------------------------------------------------------------- products
    if (lane == 0 && ntile > 0) {
      const int kd = (a.D + 15) / 16, kv = (a.Dv + 15) / 16;
      const uint32_t idS = idesc_bf16(128, kCols, 0, 0), idD = idesc_bf16(128, 16 * kd, 0, 1), idV = idesc_bf16(128, 16 * kv, 0, 1);
      auto scores = [&](int t) -> bool {
        const int st = t % NS;
        const uint32_t b0 = sB + st * 2 * L::B, b1 = b0 + L::B;
        if (!mbar_wait(&full[st], (t / NS) & 1, wc, 82)) return false;
        tc_fence_after();
        for (int kk = 0; kk < kd; ++kk) {
          const uint32_t o = (kk & 3) * 32;
          mma_ss(tmem + L::s_of(t), desc_kmajor_sw128(sA + (kk >> 2) * (kRows * 128) + o), desc_kmajor_sw128(b0 + (kk >> 2) * (kCols * 128) + o),
                 idS, kk > 0);
        }
        if (MODE != kFwd) {
          for (int kk = 0; kk < kv; ++kk) {
            const uint32_t o = (kk & 3) * 32;
            mma_ss(tmem + L::dP, desc_kmajor_sw128(sA + L::A + (kk >> 2) * (kRows * 128) + o),
                   desc_kmajor_sw128(b1 + (kk >> 2) * (kCols * 128) + o), idS, kk > 0);
          }
        }
        tc_commit(&s_full[t & 1]);
        return true;
      };
      auto done = [&](int t) { return t < 0 || mbar_wait(&pv_done[t & 1], (t >> 1) & 1, wc, 83); };
      bool go = scores(0);
      for (int t = 0; t < ntile && go; ++t) {
        const int st = t % NS;
        const uint32_t b0 = sB + st * 2 * L::B, b1 = b0 + L::B;
        // the next scores as early as their place is free: at once (forward: P(t - 1)
        // has been used), when this tile's were read (row side), or when this tile's
        // P and dS have been used (key side)
        if (MODE == kFwd && t + 1 < ntile) go = done(t - 1) && scores(t + 1);
        if (!go || !mbar_wait(&p_full[t & 1], (t >> 1) & 1, wc, 84)) break;
        tc_fence_after();
        if (MODE == kRowSide && t + 1 < ntile) {
          go = scores(t + 1);
          if (!go) break;
        }
#pragma unroll
        for (int kk = 0; kk < kCols / 16; ++kk) {
          const uint32_t acc = t > 0 || kk > 0, p = tmem + L::p_of(t) + 8 * kk;
          if (MODE != kRowSide) mma_ts(tmem + L::acc0, p, desc_mnmajor_sw128(b1 + kk * 2048, kCols * 128), idV, acc);
          if (MODE == kRowSide) {
            mma_ts(tmem + L::acc0, p, desc_mnmajor_sw128(b0 + kk * 2048, kCols * 128), idD, acc);
            mma_ts(tmem + L::acc0, p + 32, desc_mnmajor_sw128(b0 + kk * 2048, kCols * 128), idD, 1u);
          }
          if (MODE == kKeySide) mma_ts(tmem + L::acc1, tmem + L::dP + 8 * kk, desc_mnmajor_sw128(b0 + kk * 2048, kCols * 128), idD, acc);
        }
        tc_commit(&empty[st]);
        tc_commit(&pv_done[t & 1]);
        if (MODE == kKeySide && t + 1 < ntile) go = done(t) && scores(t + 1);
      }
    }
  } else {
    // ------------------------------------------------------------- rows
    const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
    WinRow row{0, 0, 0};
    Reach rc{0, 0, 0, 0, 0, 0};
    int rlo = 0, rhi = 0;                                   // columns that see this thread's key
    const int first = r0 + 32 * warp, last = min(first + 31, r1 - 1);
    if (kRowsAreQueries) {
      row = win_row(a, c, pos, alive);
      if (first < r1) rc = reach(a, c, q0, first, last + 1, 32);
    } else {
      key_rows(a, q0, pos, fl, fl + n, rlo, rhi);
    }
    if (MODE == kRowSide && mine < r1) {
      const int i = mine / a.G, h = hkv * a.G + (mine - i * a.G);
      const long long o = ((long long)b * a.H + h) * a.Nq + i;
      if (alive) {
        const bf16* x = static_cast<const bf16*>(a.out) + (((long long)b * a.Nq + i) * a.H + h) * a.Dv;
        const bf16* y = static_cast<const bf16*>(a.d_out) + (((long long)b * a.Nq + i) * a.H + h) * a.Dv;
        for (int d = 0; d < a.Dv; d += 8) {
          const uint4 xx = __ldg(reinterpret_cast<const uint4*>(x + d)), yy = __ldg(reinterpret_cast<const uint4*>(y + d));
          const uint32_t xw[4] = {xx.x, xx.y, xx.z, xx.w}, yw[4] = {yy.x, yy.y, yy.z, yy.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            del = fmaf(__uint_as_float(xw[e] << 16), __uint_as_float(yw[e] << 16), del);
            del = fmaf(__uint_as_float(xw[e] & 0xffff0000u), __uint_as_float(yw[e] & 0xffff0000u), del);
          }
        }
        const float z = a.lse[o];
        lse2 = z == -INFINITY ? INFINITY : z * kLog2e;
      }
    }
    for (int t = 0; t < ntile; ++t) {
      const int st = t % NS, u0 = t * kCols;
      const uint8_t* inf = smem + L::info + st * (MODE == kKeySide ? 768 : 8);
      const bool there = mbar_wait(&full[st], (t / NS) & 1, wc, 85) && mbar_wait(&s_full[t & 1], (t >> 1) & 1, wc, 86);   // the tile's bits or row data; S
      if (!__all_sync(0xffffffffu, there)) break;
      tc_fence_after();
      if (MODE == kFwd) {
        const uint32_t w[2] = {reinterpret_cast<const uint32_t*>(inf)[0], reinterpret_cast<const uint32_t*>(inf)[1]};
        const bool edge = (w[0] & w[1]) != 0xffffffffu || !rc.all(u0, kCols);
        // 32 scores at a time, read twice: 64 at once do not fit the registers
        auto scores = [&](int h, uint32_t (&s)[32]) {
          tmem_ld32(trow + L::s_of(t) + 32 * h, s);
          tmem_ld_wait();
          if (edge) {
            const uint32_t on = w[h] & row.sees(u0 + 32 * h);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = (on >> e) & 1u ? s[e] : __float_as_uint(-INFINITY);
          }
        };
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32];
          scores(h, s);
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
        }
        mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // m follows the true maximum only when it would be left behind by 2^8
        if (__any_sync(0xffffffffu, (mx[0] - m) * sc > kWinLag)) {
          const float mn = fmaxf(m, mx[0]), f = ex2_approx(mn == -INFINITY ? -INFINITY : (m - mn) * sc);
          m = mn;
          l *= f;
          if (t > 0) {                                      // O with the last tile in it
            if (!__all_sync(0xffffffffu, mbar_wait(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, wc, 88))) break;
            tc_fence_after();
            for (int c0 = 0; c0 < a.Dv; c0 += 32) {
              uint32_t o[32];
              tmem_ld32(trow + (uint32_t)(L::acc0 + c0), o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(trow + (uint32_t)(L::acc0 + c0), o);
            }
          }
        }
        const float mb = m == -INFINITY ? 0.f : m * sc;
        float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32], p[16];
          scores(h, s);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 x = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), both(sc), both(-mb));
            x = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum[e & 1] = add2(sum[e & 1], x);
            p[e] = pack(x.x, x.y);
          }
          tmem_st16(trow + L::p_of(t) + 16 * h, p);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      } else if (MODE == kRowSide) {
        const uint32_t w[2] = {reinterpret_cast<const uint32_t*>(inf)[0], reinterpret_cast<const uint32_t*>(inf)[1]};
        const bool edge = (w[0] & w[1]) != 0xffffffffu || !rc.all(u0, kCols);
        bool free = t == 0;                                 // the last tile's dS has been used
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32], d[32], p[16], o[16];
          tmem_ld32(trow + L::S + 32 * h, s);
          tmem_ld32(trow + L::dP + 32 * h, d);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), both(sc), both(-lse2));
            const float2 y = mul2(make_float2(ex2_approx(x.x), ex2_approx(x.y)),
                                  add2(make_float2(__uint_as_float(d[e]), __uint_as_float(d[e + 1])), both(-del)));
            s[e] = __float_as_uint(y.x);
            s[e + 1] = __float_as_uint(y.y);
          }
          if (edge) {
            const uint32_t on = w[h] & row.sees(u0 + 32 * h);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[e] = (on >> e) & 1u ? s[e] : 0u;
          }
          // dS as two bfloat16 numbers: with one, its rounding would weigh as much as that of d_q itself
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
            eps = add2(eps, x);
            p[e] = pack(x.x, x.y);
            const float2 y = add2(x, make_float2(-__uint_as_float(p[e] << 16), -__uint_as_float(p[e] & 0xffff0000u)));
            o[e] = pack(y.x, y.y);
          }
          if (!free) {
            free = __all_sync(0xffffffffu, mbar_wait(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, wc, 89));
            if (!free) break;
            tc_fence_after();
          }
          tmem_st16(trow + L::p_of(t) + 16 * h, p);
          tmem_st16(trow + L::p_of(t) + 32 + 16 * h, o);
        }
        if (!free) break;
      } else {
        const float* sl = reinterpret_cast<const float*>(inf);
        const int* sp = reinterpret_cast<const int*>(inf) + 128;
        const int pa = sp[0], pb = sp[63];                  // positions grow along the tile
        const bool edge = pa < last - a.right || pb > first + a.left;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t s[32], d[32], p[16];
          tmem_ld32(trow + L::S + 32 * h, s);
          tmem_ld32(trow + L::dP + 32 * h, d);
          tmem_ld_wait();
          const uint32_t on = edge ? win_span(rlo - u0 - 32 * h, rhi - u0 - 32 * h) : 0xffffffffu;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sl + 32 * h + e), y = *reinterpret_cast<const float4*>(sl + 64 + 32 * h + e);
            const float2 xs[2] = {make_float2(-x.x, -x.y), make_float2(-x.z, -x.w)}, ys[2] = {make_float2(-y.x, -y.y), make_float2(-y.z, -y.w)};
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int i = e + 2 * z;
              const float2 u = fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), both(sc), xs[z]);
              const float2 pr = make_float2((on >> i) & 1u ? ex2_approx(u.x) : 0.f, (on >> (i + 1)) & 1u ? ex2_approx(u.y) : 0.f);
              const float2 ds = mul2(pr, add2(make_float2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), ys[z]));
              s[i] = __float_as_uint(pr.x);
              s[i + 1] = __float_as_uint(pr.y);
              d[i] = __float_as_uint(ds.x);
              d[i + 1] = __float_as_uint(ds.y);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
          tmem_st16(trow + L::S + 16 * h, p);
#pragma unroll
          for (int e = 0; e < 16; ++e) p[e] = pack(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]));
          tmem_st16(trow + L::dP + 16 * h, p);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[t & 1]);
    }
    bool done = ntile > 0 && mbar_wait(&pv_done[(ntile - 1) & 1], ((ntile - 1) >> 1) & 1, wc, 87);
    done = __all_sync(0xffffffffu, done);
    tc_fence_after();
    const bool ok = done || ntile == 0;                     // after a wait that ran out nothing is written
    if (MODE != kKeySide) {
      const int i = mine / a.G, h = hkv * a.G + (mine - i * a.G);
      const bool in = mine < r1 && ok;
      const long long o = ((long long)b * a.Nq + i) * a.H + h;
      if (MODE == kFwd) {
        const bool some = alive && l != 0.f;
        write_row(trow, L::acc0, a.Dv, some ? 1.f / l : 0.f, done, done && some, in ? static_cast<bf16*>(a.out) + o * a.Dv : nullptr);
        if (a.lse != nullptr && in) a.lse[((long long)b * a.H + h) * a.Nq + i] = some ? fmaf(m, a.scale, logf(l)) : -INFINITY;
      } else {
        // delta from the rounded out is off by the sum of dS, which is 0 for the right one: for the key side
        if (in) a.delta[((long long)b * a.H + h) * a.Nq + i] = del + (eps.x + eps.y);
        write_row(trow, L::acc0, a.D, a.scale, done, done && alive && lse2 != INFINITY, in ? static_cast<bf16*>(a.d_q) + o * a.D : nullptr);
      }
    } else if (split && first < a.sinks) {
      // the sinks' own window: one of the pieces that win_sink_reduce adds
      float* o = mine < r1 && mine < a.sinks && ok ? a.part + ((long long)bh * (a.nchunk + 1) * a.sinks + mine) * (a.D + a.Dv) : nullptr;
      const bool keep = done && alive;
      for (int part = 0; part < 2; ++part) {
        const int width = part == 0 ? a.D : a.Dv, col = part == 0 ? L::acc1 : L::acc0;
        for (int c0 = 0; c0 < width; c0 += 32) {
          uint32_t x[32];
          if (done) {
            tmem_ld32(trow + (uint32_t)(col + c0), x);
            tmem_ld_wait();
          }
          if (o != nullptr) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + e < width) o[(part == 0 ? 0 : a.D) + c0 + e] = keep ? __uint_as_float(x[e]) : 0.f;
          }
        }
      }
    }
    if (MODE == kKeySide) {
      const long long o = ((long long)b * a.Nk + mine) * a.Hkv + hkv;
      const bool in = mine < r1 && ok && !(split && mine < a.sinks), keep = done && alive;
      write_row(trow, L::acc1, a.D, a.scale, done, keep, in ? static_cast<bf16*>(a.d_k) + o * a.D : nullptr);
      write_row(trow, L::acc0, a.Dv, 1.f, done, keep, in ? static_cast<bf16*>(a.d_v) + o * a.Dv : nullptr);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    // whichever warp's wait ran out: what is in flight ends before the memory is given back
    if (lane == 0 && *abort_flag) {
      tc_commit(drained);
      drain(drained, 0, a.timeout_ns);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::cols);
  }
}

template <int MODE, int DP>
cudaError_t run(const WinArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(&win_tc_kernel<MODE, DP>));
  if (e != cudaSuccess) return e;
  const long long rows = MODE == kKeySide ? a.Nk : (long long)a.Nq * a.G;
  win_tc_kernel<MODE, DP><<<(unsigned)((long long)a.B * a.Hkv * ((rows + kRows - 1) / kRows)), kThreads, Lay<MODE, DP>::smem, s>>>(a);
  return cudaGetLastError();
}
template <int MODE>
cudaError_t run(const WinArgs& a, cudaStream_t s) {
  return a.D <= 64 && a.Dv <= 64 ? run<MODE, 64>(a, s) : run<MODE, 128>(a, s);
}

}  // namespace

cudaError_t launch_win_fwd_tc(const WinArgs& a, cudaStream_t s) { return run<kFwd>(a, s); }
cudaError_t launch_win_bwd_q_tc(const WinArgs& a, cudaStream_t s) { return run<kRowSide>(a, s); }
cudaError_t launch_win_bwd_k_tc(const WinArgs& a, cudaStream_t s) { return run<kKeySide>(a, s); }

}  // namespace fipa

// window_pad.cu -- window attention on widths, strides or addresses that 16-byte
// loads cannot take: the inputs are copied to widths rounded up to 16 bytes,
// filled with zeros (which add nothing to a product), the kernels run on the
// copies, and results of an odd width are copied back.
//
// The copies are O(N) beside kernels that read each key once a row tile, so they
// cost little; loads of single elements in the kernels' tiles took 2.5 to 3.5
// times as long as 16-byte ones (699 residues, 12 heads on 4 of 82: forward 73 us
// against 24 us at 88, backward 385 against 108).  Few rows against a long cache
// read the cache as it is (window_step.cu), and of the keys of a forward call
// only those that some row sees are copied.
#include "kernels.h"
#include "window.h"

namespace fipa {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = 5;                    // tensors of one launch
constexpr int kRows = 4;                    // rows that a thread has in flight

struct Part {
  const void* wide;                         // [B,N,heads,wp] contiguous, the width a multiple of 16 bytes
  const void* odd;                          // [B,N,heads,w] with strides
  long long sb, sn, sh;
  int N, heads, w, wp, lg;                  // 2^lg threads a row
  int keys;                                 // rows that no query sees are left out
  unsigned rows, end;                       // rows, and the first block behind this tensor's
};
struct Parts {
  Part t[kMost];
  int n;
  unsigned blocks() const { return n == 0 ? 0 : t[n - 1].end; }
  void add(const void* wide, const void* odd, long long sb, long long sn, long long sh, int B, int N, int heads, int w, int wp, int es, int keys) {
    Part p{wide, odd, sb, sn, sh, N, heads, w, wp, 0, keys, (unsigned)((long long)B * N * heads), 0};
    while ((16 / es << p.lg) < wp) ++p.lg;
    const unsigned per = (unsigned)(kThreads >> p.lg) * kRows;
    p.end = blocks() + (p.rows + per - 1) / per;
    t[n++] = p;
  }
};

// BACK: from the wide tensor to the odd one.
template <typename E, bool BACK>
__global__ void __launch_bounds__(kThreads) win_pad_kernel(const __grid_constant__ Parts parts, const WinArgs a) {
  constexpr int V = 16 / (int)sizeof(E);
  union Piece {
    uint4 v;
    E e[V];
  };
  int i = 0;
  while (blockIdx.x >= parts.t[i].end) ++i;
  const Part& p = parts.t[i];
  const unsigned block = blockIdx.x - (i > 0 ? parts.t[i - 1].end : 0), per = kThreads >> p.lg;
  const int c = (int)(threadIdx.x & ((1u << p.lg) - 1)) * V;
  const unsigned r0 = block * per * kRows + (threadIdx.x >> p.lg);
  if (c >= p.wp) return;
  Piece x[kRows];
  long long at[kRows];
  bool on[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const unsigned r = r0 + k * per, bn = r / p.heads, b = bn / p.N, h = r - bn * p.heads;
    const int n = (int)(bn - b * p.N);
    on[k] = r < p.rows;
    if (on[k] && p.keys) {
      const int q0 = win_q0(a, (int)b);
      on[k] = n < a.sinks || (n >= max(q0, 0) - a.left && n <= min(q0 + a.Nq - 1, a.Nk - 1) + a.right);
    }
    at[k] = b * p.sb + n * p.sn + h * p.sh + c;
    if (BACK) {
      if (on[k]) x[k].v = *(reinterpret_cast<const uint4*>(static_cast<const E*>(p.wide) + (size_t)r * p.wp + c));
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[k].e[e] = on[k] && c + e < p.w ? static_cast<const E*>(p.odd)[at[k] + e] : (E)0;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (!on[k]) continue;
    if (BACK) {
      E* o = const_cast<E*>(static_cast<const E*>(p.odd)) + at[k];
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (c + e < p.w) o[e] = x[k].e[e];
    } else {
      *reinterpret_cast<uint4*>(const_cast<E*>(static_cast<const E*>(p.wide)) + (size_t)(r0 + k * per) * p.wp + c) = x[k].v;
    }
  }
}

template <bool BACK>
cudaError_t copy(const Parts& parts, const WinArgs& a, int es, cudaStream_t s) {
  if (parts.n == 0) return cudaSuccess;
  if (es == 4) win_pad_kernel<uint32_t, BACK><<<parts.blocks(), kThreads, 0, s>>>(parts, a);
  else win_pad_kernel<uint16_t, BACK><<<parts.blocks(), kThreads, 0, s>>>(parts, a);
  return cudaGetLastError();
}

// The problem on padded widths, its copies laid out from a.pad on, and their bytes.
struct PadPlan {
  WinArgs a;
  Parts in, out;
  size_t bytes;
};
PadPlan plan(const WinArgs& a, int es, bool backward) {
  PadPlan p{a, {}, {}, 0};
  p.in.n = p.out.n = 0;
  p.a.fine = win_is_fine(a, backward);
  if (!backward && es == 2 && win_step_takes(a)) return p;          // reads what it is given
  const int V = 16 / es, D = (a.D + V - 1) / V * V, Dv = (a.Dv + V - 1) / V * V;
  p.a.D = D;
  p.a.Dv = Dv;
  auto take = [&](int N, int heads, int wp) {
    void* x = static_cast<uint8_t*>(a.pad) + p.bytes;
    p.bytes += ((size_t)a.B * N * heads * wp * es + 255) / 256 * 256;
    return x;
  };
  const int keys = !backward && (es == 4 || !win_short_takes(p.a, false));
  auto input = [&](const void*& x, long long& sb, long long& sn, long long& sh, int N, int heads, int w, int wp, int filter) {
    if (((reinterpret_cast<uintptr_t>(x) & 15) | ((sb | sn | sh | w) & (V - 1))) == 0) return;
    void* y = take(N, heads, wp);
    p.in.add(y, x, sb, sn, sh, a.B, N, heads, w, wp, es, filter);
    x = y;
    sb = (long long)N * heads * wp;
    sn = (long long)heads * wp;
    sh = wp;
  };
  input(p.a.q, p.a.qb, p.a.qn, p.a.qh, a.Nq, a.H, a.D, D, 0);
  input(p.a.k, p.a.kb, p.a.kn, p.a.kh, a.Nk, a.Hkv, a.D, D, keys);
  input(p.a.v, p.a.vb, p.a.vn, p.a.vh, a.Nk, a.Hkv, a.Dv, Dv, keys);
  auto dense = [&](Parts& to, const void* x, int N, int heads, int w, int wp) -> void* {      // a contiguous tensor
    if (w == wp) return const_cast<void*>(x);
    void* y = take(N, heads, wp);
    to.add(y, x, (long long)N * heads * w, (long long)heads * w, w, a.B, N, heads, w, wp, es, 0);
    return y;
  };
  p.a.out = dense(backward ? p.in : p.out, a.out, a.Nq, a.H, a.Dv, Dv);
  if (backward) {
    p.a.d_out = dense(p.in, a.d_out, a.Nq, a.H, a.Dv, Dv);
    p.a.d_q = dense(p.out, a.d_q, a.Nq, a.H, a.D, D);
    p.a.d_k = dense(p.out, a.d_k, a.Nk, a.Hkv, a.D, D);
    p.a.d_v = dense(p.out, a.d_v, a.Nk, a.Hkv, a.Dv, Dv);
  }
  return p;
}

}  // namespace

size_t win_pad_bytes(const WinArgs& a, int es, bool backward) { return plan(a, es, backward).bytes; }

cudaError_t launch_win(const WinArgs& a, int es, bool backward, cudaStream_t s) {
  const PadPlan p = plan(a, es, backward);
  cudaError_t e = copy<false>(p.in, a, es, s);
  if (e != cudaSuccess) return e;
  e = es == 4 ? launch_win_f32(p.a, backward, s) : (backward ? launch_win_bwd(p.a, s) : launch_win_fwd(p.a, s));
  return e == cudaSuccess ? copy<true>(p.out, a, es, s) : e;
}

}  // namespace fipa

// window_pad.cu -- window attention on widths, strides or addresses that 16-byte
// loads cannot take: the inputs are copied to widths rounded up to 16 bytes,
// filled with zeros (which add nothing to a product), the kernels run on the
// copies, and results of an odd width are copied back.
//
// The copies are O(N) beside kernels that read each key once a row tile, so they
// cost little; loads of single elements in the kernels' tiles took 2.5 to 3.5
// times as long as 16-byte ones (699 residues, 12 heads on 4 of 82: training step
// 458 us, this way 141, at 88 channels 128).  The copies go by words (15 x 1321
// residues, 4 heads of 106: training step 288 us, by elements 365).  Few rows against a long cache
// read the cache as it is (window_step.cu), and of the keys of a forward call
// only those that some row sees are copied.
#include "kernels.h"
#include "window.h"

namespace fipa {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = 5;                    // tensors of one launch

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
    const unsigned per = (unsigned)(kThreads >> p.lg);
    p.end = blocks() + (p.rows + per - 1) / per;
    t[n++] = p;
  }
};

// V elements of a row from p + c on (zeros from the width w on), by words: elements of
// 2 bytes may begin in the middle of one.  Words that reach outside the row are
// taken apart.
template <typename E, int V>
__device__ __forceinline__ uint4 gather(const E* __restrict__ p, int c, int w) {
  uint32_t r[4];
  if (sizeof(E) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = c + e < w ? reinterpret_cast<const uint32_t*>(p)[c + e] : 0u;
  } else {
    const int odd = (int)(reinterpret_cast<uintptr_t>(p + c) >> 1) & 1;
    uint32_t x[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int a = c + 2 * k - odd;                        // this word's first element
      x[k] = 0u;
      if (a >= 0 && a + 1 < w && (k < 4 || odd)) {
        x[k] = *reinterpret_cast<const uint32_t*>(p + a);
      } else if (k < 4 || odd) {
        if (a >= 0 && a < w) x[k] = reinterpret_cast<const uint16_t*>(p)[a];
        else if (a + 1 >= 0 && a + 1 < w) x[k] = (uint32_t)reinterpret_cast<const uint16_t*>(p)[a + 1] << 16;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = odd ? __funnelshift_r(x[e], x[e + 1], 16) : x[e];
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// And back.
template <typename E, int V>
__device__ __forceinline__ void scatter(E* p, int c, int w, const uint4& v) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  if (sizeof(E) == 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < w) reinterpret_cast<uint32_t*>(p)[c + e] = r[e];
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(p);
    const int odd = (int)(reinterpret_cast<uintptr_t>(p + c) >> 1) & 1;
    if (odd) {
      if (c < w) o[c] = (uint16_t)r[0];
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        const uint32_t x = __funnelshift_r(r[e], r[e + 1], 16);
        if (c + 2 * e + 2 < w) *reinterpret_cast<uint32_t*>(o + c + 2 * e + 1) = x;
        else if (c + 2 * e + 1 < w) o[c + 2 * e + 1] = (uint16_t)x;
      }
      if (c + 7 < w) o[c + 7] = (uint16_t)(r[3] >> 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (c + 2 * e + 1 < w) *reinterpret_cast<uint32_t*>(o + c + 2 * e) = r[e];
        else if (c + 2 * e < w) o[c + 2 * e] = (uint16_t)r[e];
      }
    }
  }
}

// BACK: from the wide tensor to the odd one.
template <typename E, bool BACK>
__global__ void __launch_bounds__(kThreads) win_pad_kernel(const __grid_constant__ Parts parts, const WinArgs a) {
  constexpr int V = 16 / (int)sizeof(E);
  int i = 0;
  while (blockIdx.x >= parts.t[i].end) ++i;
  const Part& p = parts.t[i];
  const unsigned block = blockIdx.x - (i > 0 ? parts.t[i - 1].end : 0), r = block * (kThreads >> p.lg) + (threadIdx.x >> p.lg);
  const int c = (int)(threadIdx.x & ((1u << p.lg) - 1)) * V;
  if (c >= p.wp || r >= p.rows) return;
  const unsigned bn = r / p.heads, b = bn / p.N, h = r - bn * p.heads;
  const int n = (int)(bn - b * p.N);
  if (p.keys) {
    const int q0 = win_q0(a, (int)b);
    if (n >= a.sinks && (n < max(q0, 0) - a.left || n > min(q0 + a.Nq - 1, a.Nk - 1) + a.right)) return;
  }
  const E* odd = static_cast<const E*>(p.odd) + (b * p.sb + n * p.sn + h * p.sh);
  uint4* wide = reinterpret_cast<uint4*>(const_cast<E*>(static_cast<const E*>(p.wide)) + (size_t)r * p.wp + c);
  if (BACK) scatter<E, V>(const_cast<E*>(odd), c, p.w, *wide);
  else *wide = gather<E, V>(odd, c, p.w);
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

// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens
// (fipa_embedding, fipa_embedding_backward):
//   out[t] = scale table[idx[t]]                     (idx outside [0, V): a zero row)
//   dtable[v] = scale sum over t with idx[t] = v of dout[t], in the order of t.
//
// Bound by memory: idx, dout and out once, the table's used rows, dtable once.
// The gradient sorts (index, token) by a stable radix sort on the bits that V
// needs, cuts the sorted list into chunks of equal length, one group of threads
// each, and adds rows of dout while the index stays the same (few tokens: see
// embed_few_kernel).  A run inside one
// chunk is final; the pieces of a run that crosses chunks are kept in float32
// and added in chunk order, so no sum depends on the order of atomics and a row
// with all the tokens costs what many rows cost.
#include "fipa.h"
#include "kernels.h"

#define FIPA_API extern "C" __attribute__((visibility("default")))

namespace fipa {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortItems = 2;                              // per thread (8: 83 us for 65536 tokens of 32000 x 512 with the forward, instead of 77)
constexpr int kSortBlock = kSortThreads * kSortItems;
constexpr int kSmallItems = 8;                             // likewise where one CTA sorts the whole list
constexpr int kSmallBlock = kSortThreads * kSmallItems;
constexpr int kDigits = 256;

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
};

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float* v);
template <>
__device__ __forceinline__ void unpack<float>(const uint4& w, float* v) {
  v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y); v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& w, float* v) {
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(ww[e] << 16);
    v[2 * e + 1] = __uint_as_float(ww[e] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* v);
template <>
__device__ __forceinline__ uint4 pack<float>(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <>
__device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float cvt(float x) { return x; }
__device__ __forceinline__ float cvt(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// 2^lg threads a token, each with every 2^lg-th piece (16 bytes, or one element)
// of its row, four tokens at a time: the tokens' indices, then their pieces, are in
// flight together.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const int* __restrict__ idx, const T* __restrict__ table, T* __restrict__ out,
                                                        long long rows, int V, int C, int pieces, int lg, float scale) {
  constexpr int N = VEC ? Vec<T>::n : 1, U = 4;
  const int me = threadIdx.x & ((1 << lg) - 1), groups = 256 >> lg;
  const long long step = (long long)gridDim.x * groups * U;
  for (long long t = ((long long)blockIdx.x * groups + (threadIdx.x >> lg)) * U; t < rows; t += step) {
    int v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = t + k < rows ? __ldg(idx + t + k) : -1;
    for (int p = me; p < pieces; p += 1 << lg) {
      uint4 w[U];
      T one[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool on = v[k] >= 0 && v[k] < V;
        const T* src = table + (long long)(on ? v[k] : 0) * C + p * N;
        if (VEC) w[k] = on ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
        else one[k] = on ? *src : T(0.f);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (t + k >= rows) break;
        T* dst = out + (t + k) * C + p * N;
        const bool on = v[k] >= 0 && v[k] < V;                // a skipped row is 0 whatever the scale
        if (VEC) {
          float x[N];
          unpack<T>(w[k], x);
#pragma unroll
          for (int e = 0; e < N; ++e) x[e] = on ? x[e] * scale : 0.f;
          *reinterpret_cast<uint4*>(dst) = pack<T>(x);
        } else {
          put(dst, on ? cvt(one[k]) * scale : 0.f);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- stable sort
// Digit counts of every block of 512 elements: hist[digit][block].
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int* __restrict__ key, int n, int V, int first, int shift,
                                                                  int mask, int* __restrict__ hist) {
  __shared__ int cnt[kDigits];
  cnt[threadIdx.x] = 0;
  __syncthreads();
  int v[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = blockIdx.x * kSortBlock + k * kSortThreads + threadIdx.x;
    v[k] = i < n ? key[i] : -1;
    if (first && i < n && (v[k] < 0 || v[k] >= V)) v[k] = V;
  }
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (v[k] < 0) continue;
    atomicAdd(&cnt[(v[k] >> shift) & mask], 1);
  }
  __syncthreads();
  if (threadIdx.x <= mask) hist[(size_t)threadIdx.x * gridDim.x + blockIdx.x] = cnt[threadIdx.x];
}
// Exclusive prefix sums of one digit's block counts, and its total (one CTA per digit).
__global__ void __launch_bounds__(256) sort_scan_kernel(int* __restrict__ hist, int* __restrict__ total, int nblk) {
  __shared__ int ws[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* h = hist + (size_t)blockIdx.x * nblk;
  int carry = 0;
  for (int b0 = 0; b0 < nblk; b0 += 256) {
    const int b = b0 + threadIdx.x, x = b < nblk ? h[b] : 0;
    int y = x;
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) ws[warp] = y;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += ws[w];
      all += ws[w];
    }
    if (b < nblk) h[b] = carry + before + y - x;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) total[blockIdx.x] = carry;
}
// Moves every element to its place.  A warp owns 64 neighbours and takes them
// 32 at a time: an element's rank among its warp's equal digits is the warp's
// running count plus the equal lanes below it.
__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const int* __restrict__ key, const int* __restrict__ tok, int n, int V,
                                                                 int first, int shift, int mask, const int* __restrict__ hist,
                                                                 const int* __restrict__ total, int nblk, int* __restrict__ okey,
                                                                 int* __restrict__ otok) {
  __shared__ int cnt[8][kDigits];
  __shared__ int base[kDigits];
  __shared__ int ws[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = 0; w < 8; ++w) cnt[w][threadIdx.x] = 0;
  // digits below this one, in all
  const int tot = threadIdx.x <= mask ? total[threadIdx.x] : 0;
  int y = tot;
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) ws[warp] = y;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += ws[w];
  if (threadIdx.x <= mask) base[threadIdx.x] = before + y - tot + hist[(size_t)threadIdx.x * nblk + blockIdx.x];
  int v[kSortItems], tk[kSortItems], rank[kSortItems];
  const int i0 = blockIdx.x * kSortBlock + warp * 32 * kSortItems + lane;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = i0 + k * 32;
    v[k] = -1;
    tk[k] = i;
    if (i < n) {
      v[k] = key[i];
      if (first) {
        if (v[k] < 0 || v[k] >= V) v[k] = V;
      } else {
        tk[k] = tok[i];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const bool on = v[k] >= 0;
    const int d = on ? (v[k] >> shift) & mask : kDigits;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const int below = __popc(same & ((1u << lane) - 1u));
    int c = 0;
    if (on) c = cnt[warp][d];
    rank[k] = c + below;
    __syncwarp();
    if (on && below == 0) cnt[warp][d] = c + __popc(same);
    __syncwarp();
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    if (v[k] < 0) continue;
    const int d = (v[k] >> shift) & mask;
    int p = base[d] + rank[k];
    for (int w = 0; w < warp; ++w) p += cnt[w][d];
    okey[p] = v[k];
    otok[p] = tk[k];
  }
}

// The whole sort of at most 2048 tokens in one CTA: the same passes, all of
// whose counts fit in shared memory (8 or more launches would cost more than
// the work).
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(const int* __restrict__ idx, int n, int V, int passes, int bits,
                                                                  int* __restrict__ okey, int* __restrict__ otok) {
  __shared__ int key[2][kSmallBlock], tok[2][kSmallBlock], cnt[8][kDigits], ws[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mask = (1 << bits) - 1;
  for (int i = threadIdx.x; i < n; i += kSortThreads) {
    const int v = idx[i];
    key[0][i] = v < 0 || v >= V ? V : v;
    tok[0][i] = i;
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int from = pass & 1, shift = pass * bits;
    for (int w = 0; w < 8; ++w) cnt[w][threadIdx.x] = 0;
    __syncthreads();
    int v[kSmallItems], tk[kSmallItems], rank[kSmallItems];
#pragma unroll
    for (int k = 0; k < kSmallItems; ++k) {
      const int i = (warp * kSmallItems + k) * 32 + lane;
      v[k] = i < n ? key[from][i] : -1;
      tk[k] = i < n ? tok[from][i] : 0;
      const int d = v[k] >= 0 ? (v[k] >> shift) & mask : kDigits;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const int below = __popc(same & ((1u << lane) - 1u));
      int c = 0;
      if (v[k] >= 0) c = cnt[warp][d];
      rank[k] = c + below;
      __syncwarp();
      if (v[k] >= 0 && below == 0) cnt[warp][d] = c + __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // digit d of warp w starts behind all smaller digits and the warps before
    int tot = 0;
    for (int w = 0; w < 8; ++w) tot += cnt[w][threadIdx.x];
    int y = tot;
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) ws[warp] = y;
    __syncthreads();
    int at = y - tot;
    for (int w = 0; w < warp; ++w) at += ws[w];
    for (int w = 0; w < 8; ++w) {
      const int c = cnt[w][threadIdx.x];
      cnt[w][threadIdx.x] = at;
      at += c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSmallItems; ++k) {
      if (v[k] < 0) continue;
      const int p = cnt[warp][(v[k] >> shift) & mask] + rank[k];
      key[from ^ 1][p] = v[k];
      tok[from ^ 1][p] = tk[k];
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kSortThreads) {
    okey[i] = key[passes & 1][i];
    otok[i] = tok[passes & 1][i];
  }
}

// ---------------------------------------------------------------- run sums
// A group of `tpc` threads adds one chunk of L (a multiple of 8) tokens of the
// sorted list for a slab of columns, eight rows of dout in flight a thread.
// part[chunk][0]: the run that came from the chunk before; [1]: the run that
// starts here and goes on.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4) embed_sum_kernel(const int* __restrict__ key, const int* __restrict__ tok, const T* __restrict__ dout,
                                                        int n, int V, int C, int L, int tpc, int slabs, float scale,
                                                        float* __restrict__ dtable, float* __restrict__ part, int nchunk) {
  constexpr int N = VEC ? Vec<T>::n : 1, U = 8;
  const int gpb = blockDim.x / tpc;
  const long long unit = (long long)blockIdx.x * gpb + threadIdx.x / tpc;
  const int chunk = (int)(unit / slabs), slab = (int)(unit - (long long)chunk * slabs);
  const int c = (slab * tpc + (int)threadIdx.x % tpc) * N;
  if (chunk >= nchunk || c >= C) return;
  const int b = chunk * L, e = min(n, b + L);
  float acc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  int cur = key[b];
  bool open = b > 0 && key[b - 1] == cur;                     // the run began in an earlier chunk
  auto flush = [&](float* dst, float f) {
    if (VEC) {
#pragma unroll
      for (int k = 0; k < N; k += 4)
        *reinterpret_cast<float4*>(dst + k) = make_float4(acc[k] * f, acc[k + 1] * f, acc[k + 2] * f, acc[k + 3] * f);
    } else {
      dst[0] = acc[0] * f;
    }
  };
  for (int i0 = b; i0 < e; i0 += U) {
    int kk[U], tt[U];
    if (i0 + U <= e) {                                        // the lists' parts are 32-byte aligned
#pragma unroll
      for (int j = 0; j < U; j += 4) {
        const int4 x = *reinterpret_cast<const int4*>(key + i0 + j), y = *reinterpret_cast<const int4*>(tok + i0 + j);
        kk[j] = x.x; kk[j + 1] = x.y; kk[j + 2] = x.z; kk[j + 3] = x.w;
        tt[j] = y.x; tt[j + 1] = y.y; tt[j + 2] = y.z; tt[j + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        kk[j] = i0 + j < e ? key[i0 + j] : V;
        tt[j] = i0 + j < e ? tok[i0 + j] : 0;
      }
    }
    uint4 raw[U];
    T one[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const T* p = dout + (long long)tt[j] * C + c;
      if (VEC) raw[j] = kk[j] < V ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
      else one[j] = kk[j] < V ? *p : T(0.f);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j >= e) break;
      if (kk[j] != cur) {
        if (cur < V) {
          if (open) flush(part + ((size_t)chunk * 2) * C + c, 1.f);
          else flush(dtable + (size_t)cur * C + c, scale);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.f;
        cur = kk[j];
        open = false;
      }
      float x[N];
      if (VEC) unpack<T>(raw[j], x);
      else x[0] = cvt(one[j]);
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] += x[k];
    }
  }
  if (cur >= V) return;
  const bool goes_on = e < n && key[e] == cur;
  if (open) flush(part + ((size_t)chunk * 2) * C + c, 1.f);
  else if (goes_on) flush(part + ((size_t)chunk * 2 + 1) * C + c, 1.f);
  else flush(dtable + (size_t)cur * C + c, scale);
}

__device__ __forceinline__ int lower_bound(const int* __restrict__ key, int n, int v) {
  int lo = 0, len = n;                     // the answer is in [lo, lo + len]; four parts a step, as each step waits for memory once
  while (len > 0) {
    const int s = len / 4, a = lo + s, b = lo + 2 * s, c = lo + 3 * s;
    const bool x = key[a] < v, y = key[b] < v, z = key[c] < v;
    if (z) {
      lo = c + 1;
      len -= 3 * s + 1;
    } else if (y) {
      lo = b + 1;
      len = s - 1;
    } else if (x) {
      lo = a + 1;
      len = s - 1;
    } else {
      len = s;
    }
  }
  return lo;
}
// Sum of the pieces [lo, hi) of a run that starts in chunk q, for N columns.
template <int N>
__device__ __forceinline__ void add_pieces(float (&x)[N], const float* part, int C, int c, int q, int lo, int hi) {
#pragma unroll 8
  for (int k = lo; k < hi; ++k) {
    const float* p = part + ((size_t)k * 2 + (k == q ? 1 : 0)) * C + c;
    if (N == 4) {
      const float4 y = *reinterpret_cast<const float4*>(p);
      x[0] += y.x; x[1 % N] += y.y; x[2 % N] += y.z; x[3 % N] += y.w;
    } else {
      x[0] += *p;
    }
  }
}
// CTAs [0, ncross): a warp looks at one chunk.  If a run starts in it and goes
// on, its pieces are added: up to 16 by the warp, more by all 16 warps of the
// CTA, in 16 neighbouring stretches whose sums are added in order.  CTAs beyond: a
// warp searches the list for 32 rows at once, one a lane, and writes zeros to those
// without a token.  blockIdx.y: slab of 32 N columns of the sums.
template <int N>
__global__ void __launch_bounds__(512) embed_join_kernel(const int* __restrict__ key, int n, int V, int C, int L, int nchunk,
                                                         int ncross, float scale, const float* __restrict__ part,
                                                         float* __restrict__ dtable) {
  __shared__ float red[16][32 * N];
  __shared__ int long_last[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.y * 32 * N, c = c0 + lane * N;
  if ((int)blockIdx.x >= ncross) {
    const long long step = (long long)(gridDim.x - ncross) * 16 * 32;
    for (long long v0 = ((long long)(blockIdx.x - ncross) * 16 + warp) * 32; v0 < V; v0 += step) {
      const long long v = v0 + lane;
      bool none = false;
      if (v < V) {
        const int b = lower_bound(key, n, (int)v);
        none = b >= n || key[b] != (int)v;
      }
      for (unsigned left = __ballot_sync(0xffffffffu, none); left != 0u; left &= left - 1u) {
        float* o = dtable + (v0 + __ffs(left) - 1) * C;
        if (c < C) {
          if (N == 4) *reinterpret_cast<float4*>(o + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          else o[c] = 0.f;
        }
      }
    }
    return;
  }
  const int q = blockIdx.x * 16 + warp, e = (q + 1) * L;
  if (lane == 0) long_last[warp] = -1;
  if (q + 1 < nchunk) {
    const int cur = key[e];
    if (cur < V && key[e - 1] == cur && !(q > 0 && key[q * L - 1] == cur)) {
      // last chunk that begins inside the run: 32 places of the rest at a time
      int lo = q + 1, hi = nchunk;                            // lo begins inside, hi does not (or the list ends)
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const unsigned in = __ballot_sync(0xffffffffu, at < hi && key[(size_t)at * L] == cur);
        const int k = in == 0xffffffffu ? 31 : __ffs(~in) - 2;   // the last place inside
        if (lo + (k + 1) * step < hi) hi = lo + (k + 1) * step;
        lo += k * step;
      }
      const int last = lo;
      if (last - q < 16) {
        if (c < C) {
          float x[N] = {0.f};
          add_pieces<N>(x, part, C, c, q, q, last + 1);
#pragma unroll
          for (int k = 0; k < N; ++k) dtable[(size_t)cur * C + c + k] = x[k] * scale;
        }
      } else if (lane == 0) {
        long_last[warp] = last;
      }
    }
  }
  __syncthreads();
  for (int w = 0; w < 16; ++w) {
    const int last = long_last[w], first = blockIdx.x * 16 + w;
    if (last < 0) continue;
    const int cur = key[(first + 1) * L], per = (last - first + 16) / 16;
    const int lo = first + warp * per, hi = min(lo + per, last + 1);
    float x[N] = {0.f};
    if (c < C) add_pieces<N>(x, part, C, c, first, lo, hi);
#pragma unroll
    for (int k = 0; k < N; ++k) red[warp][lane * N + k] = x[k];
    __syncthreads();
    if ((int)threadIdx.x < 32 * N && c0 + (int)threadIdx.x < C) {
      float y = 0.f;
      for (int v = 0; v < 16; ++v) y += red[v][threadIdx.x];
      dtable[(size_t)cur * C + c0 + threadIdx.x] = y * scale;
    }
    __syncthreads();
  }
}

// The whole gradient of at most kFew tokens in one launch, where the sort's three
// would cost more than the work (37 tokens, 44947 x 128, forward and backward: 8.3 us
// against 16.3; 128 of one row of 256: 10.8 against 12.6): a warp owns a row of the
// table and 32 pieces of columns, finds the row's tokens by comparing all of them,
// four a lane, and adds eight rows of dout at a time, in order.
constexpr int kFew = 128;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_few_kernel(const int* __restrict__ idx, const T* __restrict__ dout, int n, int V, int C,
                                                        int slabs, float scale, float* __restrict__ dtable) {
  constexpr int N = VEC ? Vec<T>::n : 1, W = kFew / 32, U = 8;
  const int lane = threadIdx.x & 31;
  int key[W];
#pragma unroll
  for (int j = 0; j < W; ++j) key[j] = 32 * j + lane < n ? idx[32 * j + lane] : -1;
  const long long units = (long long)V * slabs, step = (long long)gridDim.x * 8;
  for (long long x = blockIdx.x * 8ll + (threadIdx.x >> 5); x < units; x += step) {
    const int v = (int)(x / slabs), c = ((int)(x - (long long)v * slabs) * 32 + lane) * N;
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      unsigned mine = __ballot_sync(0xffffffffu, key[j] == v);
      while (mine != 0) {
        float w[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const T* p = dout + (size_t)(32 * j + __ffs(mine) - 1) * C + c;
          const bool on = mine != 0 && c < C;
          if (VEC) {
            unpack<T>(on ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0), w[u]);
          } else {
            w[u][0] = on ? cvt(p[0]) : 0.f;
          }
          mine &= mine - 1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < N; ++k) acc[k] += w[u][k];
      }
    }
    if (c >= C) continue;
    float* o = dtable + (size_t)v * C + c;
    if (VEC) {
#pragma unroll
      for (int k = 0; k < N; k += 4)
        *reinterpret_cast<float4*>(o + k) = make_float4(acc[k] * scale, acc[k + 1] * scale, acc[k + 2] * scale, acc[k + 3] * scale);
    } else {
      o[0] = acc[0] * scale;
    }
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Workspace of the gradient: two copies of (key, token), digit counts, pieces.
struct EmbedPlan {
  int nblk, passes, bits, L, nchunk;
  size_t off_key[2], off_tok[2], off_hist, off_total, off_part, total;
};
EmbedPlan embed_plan(long long T, int V, int C) {
  EmbedPlan p;
  int need = 1;
  while (need < 31 && (V >> need) != 0) ++need;              // bits of the values 0 .. V
  p.passes = (need + 7) / 8;
  p.bits = (need + p.passes - 1) / p.passes;
  p.nblk = (int)((T + kSortBlock - 1) / kSortBlock);
  // Chunks short enough for a full GPU of threads (16-byte pieces, 2048 an SM),
  // long enough that the pieces of runs stay a small part of the traffic.
  p.L = 16;
  while (p.L < 256 && (T / p.L) * ((C + 7) / 8) > 148 * 2048) p.L *= 2;
  p.nchunk = (int)((T + p.L - 1) / p.L);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  for (int k = 0; k < 2; ++k) {
    p.off_key[k] = take((size_t)T * 4);
    p.off_tok[k] = take((size_t)T * 4);
  }
  p.off_hist = take((size_t)p.nblk * kDigits * 4);
  p.off_total = take(kDigits * 4);
  p.off_part = take((size_t)p.nchunk * 2 * C * 4);
  p.total = o;
  return p;
}

template <typename T>
cudaError_t embed_fwd(const int* idx, const void* table, void* out, long long rows, int V, int C, float scale, cudaStream_t s) {
  const bool vec = C % Vec<T>::n == 0 && is_aligned(table, 16) && is_aligned(out, 16);
  const int pieces = vec ? C / Vec<T>::n : C;
  int lg = 0;
  while ((1 << lg) < pieces && lg < 8) ++lg;
  const long long need = (rows + 4 * (256 >> lg) - 1) / (4 * (256 >> lg)), most = 148 * 32;
  const unsigned grid = (unsigned)(need < most ? need : most);
  if (vec)
    embed_fwd_kernel<T, true><<<grid, 256, 0, s>>>(idx, static_cast<const T*>(table), static_cast<T*>(out), rows, V, C, pieces, lg, scale);
  else
    embed_fwd_kernel<T, false><<<grid, 256, 0, s>>>(idx, static_cast<const T*>(table), static_cast<T*>(out), rows, V, C, pieces, lg, scale);
  return cudaGetLastError();
}

template <typename T>
cudaError_t embed_few(const int* idx, const void* dout, int n, int V, int C, float scale, float* dtable, cudaStream_t s) {
  const bool vec = C % Vec<T>::n == 0 && is_aligned(dout, 16) && is_aligned(dtable, 16);
  const int slabs = (C + 32 * (vec ? Vec<T>::n : 1) - 1) / (32 * (vec ? Vec<T>::n : 1));
  const long long ctas = ((long long)V * slabs + 7) / 8;
  const unsigned grid = (unsigned)(ctas < 148 * 8 ? ctas : 148 * 8);
  if (vec) embed_few_kernel<T, true><<<grid, 256, 0, s>>>(idx, static_cast<const T*>(dout), n, V, C, slabs, scale, dtable);
  else embed_few_kernel<T, false><<<grid, 256, 0, s>>>(idx, static_cast<const T*>(dout), n, V, C, slabs, scale, dtable);
  return cudaGetLastError();
}

template <typename T>
cudaError_t embed_sum(const EmbedPlan& p, uint8_t* ws, int at, const void* dout, int n, int V, int C, float scale, float* dtable,
                      cudaStream_t s) {
  const bool vec = C % Vec<T>::n == 0 && is_aligned(dout, 16) && is_aligned(dtable, 16);
  const int pieces = vec ? C / Vec<T>::n : C;
  int tpc = 1;
  while (tpc < pieces && tpc < 256) tpc *= 2;
  const int slabs = (pieces + tpc - 1) / tpc, gpb = 256 / tpc;
  const unsigned grid = (unsigned)(((long long)p.nchunk * slabs + gpb - 1) / gpb);
  const int* key = reinterpret_cast<const int*>(ws + p.off_key[at]);
  const int* tok = reinterpret_cast<const int*>(ws + p.off_tok[at]);
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  if (vec)
    embed_sum_kernel<T, true><<<grid, 256, 0, s>>>(key, tok, static_cast<const T*>(dout), n, V, C, p.L, tpc, slabs, scale, dtable, part, p.nchunk);
  else
    embed_sum_kernel<T, false><<<grid, 256, 0, s>>>(key, tok, static_cast<const T*>(dout), n, V, C, p.L, tpc, slabs, scale, dtable, part, p.nchunk);
  return cudaGetLastError();
}

constexpr long long kEmbedMaxTokens = 1ll << 30;

fipa_status embed_check(fipa_dtype dtype, long long T, int V, int C, double scale) {
  if (dtype != FIPA_F32 && dtype != FIPA_BF16) return FIPA_ERR_INVALID_ARG;
  if (T < 0 || V <= 0 || C <= 0 || !isfinite((float)scale)) return FIPA_ERR_INVALID_ARG;
  if (T > kEmbedMaxTokens || C > 65536 || V > (1 << 30)) return FIPA_ERR_UNSUPPORTED;
  return FIPA_OK;
}

}  // namespace
}  // namespace fipa

FIPA_API fipa_status fipa_embedding(fipa_dtype dtype, const int32_t* idx, const void* table, int64_t T, int V, int C,
                                    double scale, void* out, void* stream) {
  const fipa_status st = fipa::embed_check(dtype, T, V, C, scale);
  if (st != FIPA_OK) return st;
  if (T == 0) return FIPA_OK;
  const size_t es = dtype == FIPA_F32 ? 4 : 2;
  if (idx == nullptr || table == nullptr || out == nullptr || !fipa::is_aligned(idx, 4) || !fipa::is_aligned(table, es) ||
      !fipa::is_aligned(out, es))
    return FIPA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == FIPA_F32 ? fipa::embed_fwd<float>(idx, table, out, T, V, C, (float)scale, s)
                                          : fipa::embed_fwd<__nv_bfloat16>(idx, table, out, T, V, C, (float)scale, s);
  return e == cudaSuccess ? FIPA_OK : FIPA_ERR_CUDA;
}

FIPA_API fipa_status fipa_embedding_backward_workspace_size(int64_t T, int V, int C, size_t* bytes) {
  if (bytes == nullptr) return FIPA_ERR_INVALID_ARG;
  const fipa_status st = fipa::embed_check(FIPA_F32, T, V, C, 1.0);
  if (st != FIPA_OK) return st;
  *bytes = fipa::embed_plan(T, V, C).total;
  return FIPA_OK;
}

FIPA_API fipa_status fipa_embedding_backward(fipa_dtype dtype, const int32_t* idx, const void* d_out, int64_t T, int V, int C,
                                             double scale, float* d_table, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fipa;
  const fipa_status st = embed_check(dtype, T, V, C, scale);
  if (st != FIPA_OK) return st;
  const size_t es = dtype == FIPA_F32 ? 4 : 2;
  if (d_table == nullptr || !is_aligned(d_table, 4)) return FIPA_ERR_INVALID_ARG;
  if (T > 0 && (idx == nullptr || d_out == nullptr || !is_aligned(idx, 4) || !is_aligned(d_out, es))) return FIPA_ERR_INVALID_ARG;
  const EmbedPlan p = embed_plan(T, V, C);
  if (workspace == nullptr || workspace_bytes < p.total) return FIPA_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return FIPA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n = (int)T;
  int* hist = reinterpret_cast<int*>(ws + p.off_hist);
  int* total = reinterpret_cast<int*>(ws + p.off_total);
  if (n <= kFew) {
    const cudaError_t e = dtype == FIPA_F32 ? embed_few<float>(idx, d_out, n, V, C, (float)scale, d_table, s)
                                            : embed_few<__nv_bfloat16>(idx, d_out, n, V, C, (float)scale, d_table, s);
    return e == cudaSuccess ? FIPA_OK : FIPA_ERR_CUDA;
  }
  const int* key = idx;
  const int* tok = nullptr;
  int at = 0;
  if (n <= kSmallBlock) {
    int* okey = reinterpret_cast<int*>(ws + p.off_key[0]);
    int* otok = reinterpret_cast<int*>(ws + p.off_tok[0]);
    sort_small_kernel<<<1, kSortThreads, 0, s>>>(idx, n, V, p.passes, p.bits, okey, otok);
    key = okey;
  } else {
    const int mask = (1 << p.bits) - 1;
    for (int k = 0; k < p.passes; ++k) {
      at = k & 1;
      int* okey = reinterpret_cast<int*>(ws + p.off_key[at]);
      int* otok = reinterpret_cast<int*>(ws + p.off_tok[at]);
      sort_count_kernel<<<p.nblk, kSortThreads, 0, s>>>(key, n, V, k == 0, k * p.bits, mask, hist);
      sort_scan_kernel<<<mask + 1, 256, 0, s>>>(hist, total, p.nblk);
      sort_move_kernel<<<p.nblk, kSortThreads, 0, s>>>(key, tok, n, V, k == 0, k * p.bits, mask, hist, total, p.nblk, okey, otok);
      key = okey;
      tok = otok;
    }
  }
  const cudaError_t e = dtype == FIPA_F32 ? embed_sum<float>(p, ws, at, d_out, n, V, C, (float)scale, d_table, s)
                                          : embed_sum<__nv_bfloat16>(p, ws, at, d_out, n, V, C, (float)scale, d_table, s);
  if (e != cudaSuccess) return FIPA_ERR_CUDA;
  const int ncross = p.nchunk > 1 ? (p.nchunk - 1 + 15) / 16 : 0;
  const long long fill = ((long long)V + 511) / 512;
  const unsigned gx = (unsigned)(ncross + (fill < 148 * 4 ? fill : 148 * 4));
  const float* part = reinterpret_cast<const float*>(ws + p.off_part);
  // Long runs want more CTAs, narrow ones; us of the gradient of T tokens of V x C in
  // bfloat16, cold, wide against narrow slabs:
  //   59574 of 2 x 256  59 / 45    160000 of 8 x 128   55 / 49    327680 of 64 x 128  53 / 61
  //   40000 of 1 x 512  74 / 55    100000 of 8 x 256   49 / 51    262144 of 32 x 64   45 / 43
  //   65536 of 4 x 256  45 / 41    200000 of 16 x 128  51 / 53    10000 of 1 x 512    35 / 29
  // From 5000 to 16384 tokens a row it is also a matter of how many rows and columns there are.
  if (C % 4 == 0 && is_aligned(d_table, 16) && n / V < 16384)
    embed_join_kernel<4><<<dim3(gx, (unsigned)((C + 127) / 128)), 512, 0, s>>>(key, n, V, C, p.L, p.nchunk, ncross, (float)scale, part, d_table);
  else
    embed_join_kernel<1><<<dim3(gx, (unsigned)((C + 31) / 32)), 512, 0, s>>>(key, n, V, C, p.L, p.nchunk, ncross, (float)scale, part, d_table);
  return cudaGetLastError() == cudaSuccess ? FIPA_OK : FIPA_ERR_CUDA;
}

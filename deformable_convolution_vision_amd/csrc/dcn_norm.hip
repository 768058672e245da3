// dcn_norm.hip -- gfx950 group normalisation of channels-last maps with the activation that
// follows it, and its gradients.
//
// x [B][P][C] (P positions), G groups of Cg = C / G adjacent channels, N = P * Cg values of a
// group of one batch element:
//
//   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps),
//   n = (x - mean) rstd,  z = n weight_c + bias_c,  out = act(z)
//
// and for an upstream gradient g, with gz = g act'(z):
//
//   grad_bias_c = sum_{b,p} gz,  grad_weight_c = sum_{b,p} gz n,
//   grad_x = rstd (weight_c gz - S1 / N - n S2 / N),
//     S1 = sum over the group of weight_c gz,  S2 = sum over the group of weight_c gz n.
//
// Two ways.  Where a group of one batch element fits the registers of a workgroup, that workgroup
// reads it once, sums, and writes (norm_slice_kernel, norm_grad_slice_kernel: one launch, and one
// more that adds the batch elements' parameter gradients).  Larger maps are read twice: a pass
// that sums over chunks of positions (one workgroup each, whole rows: contiguous memory), and a
// pass that first joins the chunks' parts and then writes.  Sums are joined in a fixed order;
// there are no atomics.
//
// In the second way the variance is formed from sums of d and d^2, d = x - r with r the middle one of three
// values of the channel in the chunk (a single one may lie far out), and chunks and channels are joined as
// (count, mean, sum of squares about the mean): nothing large cancels where the mean is far from 0.
//
// Arithmetic: fp32 throughout, every output rounded to its type once.
//
// What bounds it, measured: memory.  8 x 16800 positions of 256 bf16 channels (69 MB), silu: 15.3 us for
// the sums (4.5 TB/s) and 27.0 for the writing pass (5.1 TB/s, a copy's rate), 49 us a call on maps that
// are not in the cache; the second reading is the 14 us that a single one would save (the chip's
// registers could hold the map, in a cooperative launch whose workgroups wait for each other once:
// not tried).  Gradients at 2 x 16800: 13.1 us for 34.6 MB (2.6 TB/s: a CU has 32 KB of loads under
// way) and 13.8 for 52.  fp32 forward at 8 x 16800: 70 us, 55 by its bytes.  One map of 1050 positions:
// 6.4 us in one launch, which is that launch and one workgroup's chain (12.4 us as two passes, host
// included, against 9.1).  Groups of a size that is no multiple of a 16-byte vector are read element
// by element by a slice: 1050 positions of 8 groups of 12 bf16 channels 12.5 us, of 16 channels 8.9.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"

namespace dcn {
namespace norm {
namespace {

constexpr int kNT = 512;         // threads of the two passes
constexpr int kMaxC = 8192;

// How a pass is cut into workgroups.
struct Cut {
  int cb;                    // channels of a workgroup: whole groups
  int blocks;                // along the positions
  int64_t rows;              // positions of one
  int tc, tr;                // threads along its row, rows at a time
};

struct Args {
  const void *x, *w, *b, *g;
  void* out;                 // forward: out; backward: grad_x
  float *mean, *rstd;        // [B][G]
  void *gw, *gb;
  float* gpart;              // [B][G][chunks][2]
  float* cpart;              // backward: [B][chunks][C][2] (slices: one chunk, none for a single batch element)
  int64_t P;
  int B, C, G, Cg;
  Cut sum, write;
  float eps;
};

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));   // nearest even
}

// V adjacent elements: 16 bytes, or one element where rows do not start on 16 bytes
template <typename T, int V>
struct Vec {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load(const T* p) {
  Vec<T, V> v;
  if (V > 1) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    __builtin_memcpy(v.e, &u, 16);
  } else {
    v.e[0] = *p;
  }
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&f)[V]) {
  Vec<T, V> v;
#pragma unroll
  for (int j = 0; j < V; ++j) v.e[j] = narrow<T>(f[j]);
  if (V > 1) {
    uint4 u;
    __builtin_memcpy(&u, v.e, 16);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *p = v.e[0];
  }
}

// The normal distribution's lower tail c = Phi(-|z|) = erfc(|z| / sqrt(2)) / 2, and e = exp(-z^2 / 2),
// which it shares.  With t = 1 / (1 + a |z|) the quotient c / (e t) is smooth over 0 < t <= 1 and is
// taken as a polynomial (weighted least squares at Chebyshev points for |z| <= 13.3, beyond which e is
// 0 in fp32, weights raised where the relative error was largest).  The tail has no difference of near
// values, so gelu, which takes c or 1 - c, keeps its relative precision for z < 0.
//  - fp32: degree 8 (2.1e-8) in v = 1 - t = a |z| t, formed as a product, so that what is lost near
//    z = 0 is relative to v: c is off by (22 + 1.5 z^2) 2^-24 of itself at most, the z^2 from the
//    rounding of the exponential's argument.
//  - bf16, whose outputs keep 2^-9: degree 5 (4.6e-6) in t.  With fp32's polynomial 8 x 16800 positions
//    of 256 channels take 49.9 us forward, and 2 x 16800 31.0 backward; with this one 45.1 and 29.7.
// (erff takes a third of the gelu backward's instructions; a rational form of the error function of 5
// coefficients is off by 1.5e-7, which is 6e-5 of gelu's value at z in [-3, -2]; 44.6 and 28.6 us.)
template <typename T>
__device__ __forceinline__ float lower_tail(float z, float& e) {
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  if constexpr (sizeof(T) == 2) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.305000007f, 1.f));
    float p = fmaf(-0.0765512735f, t, 0.200597435f);
    p = fmaf(p, t, -0.0027701701f);
    p = fmaf(p, t, 0.139904127f);
    p = fmaf(p, t, 0.116830379f);
    p = fmaf(p, t, 0.121991396f);
    return p * t * e;
  } else {
    const float y = fminf(fabsf(z), 64.f) * 0.26f;   // (an infinity times its reciprocal would be none)
    const float t = __builtin_amdgcn_rcpf(1.f + y), v = y * t;
    float p = fmaf(0.0308960844f, v, -0.0924284607f);
    p = fmaf(p, v, 0.0373755172f);
    p = fmaf(p, v, 0.142099783f);
    p = fmaf(p, v, -0.0347089954f);
    p = fmaf(p, v, -0.574499309f);
    p = fmaf(p, v, 1.12941992f);
    p = fmaf(p, v, -1.03439236f);
    p = fmaf(p, v, 0.5f);
    return p * t * e;
  }
}
// Phi(z)
template <typename T>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float c = lower_tail<T>(z, e);
  return z < 0.f ? c : 1.f - c;
}
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
template <typename T, int ACT>
__device__ __forceinline__ float act(float z) {
  if (ACT == DCN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (ACT == DCN_ACT_SILU) return z * sigmoid(z);
  if (ACT == DCN_ACT_GELU) {
    float e;
    return z * normal_cdf<T>(z, e);
  }
  return z;
}
template <typename T, int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == DCN_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == DCN_ACT_SILU) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if (ACT == DCN_ACT_GELU) {
    float e;
    const float cdf = normal_cdf<T>(z, e);
    return fmaf(z * 0.39894228040143268f, e, cdf);
  }
  return 1.f;
}

__device__ __forceinline__ float not_below_0(float v) { return v < 0.f ? 0.f : v; }   // a NaN stays one

// sum over the `width` lanes (a power of two) that a lane belongs to
__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int w = width >> 1; w > 0; w >>= 1) v += __shfl_xor(v, w, 64);
  return v;
}
// lanes that join one group's parts: a power of two, all groups at once where they fit
__device__ __forceinline__ int lanes_of(int G) {
  int n = 64;
  while (n > 1 && n * G > kNT) n >>= 1;
  return n;
}

// A workgroup's share: channels c0 .. c0 + width - 1 (whole groups, g0 .. g0 + ng - 1) of batch
// element b.  Its threads form rows of tc vectors, tr rows at a time.
struct Share {
  int b, c0, width, g0, ng;
};
__device__ __forceinline__ Share share_of(const Args& a, const Cut& cut) {
  Share s;
  s.b = blockIdx.z;
  s.c0 = blockIdx.y * cut.cb;
  s.width = min(cut.cb, a.C - s.c0);
  s.g0 = s.c0 / a.Cg;
  s.ng = s.width / a.Cg;
  return s;
}

// Joins the threads' sums of V channels each over the rows of threads -> f(channel, sums).  Rows of
// threads that divide a wave are first added within it, lane by lane, which leaves one per wave.
template <int V, typename F>
__device__ __forceinline__ void join_rows(float (&s1)[V], float (&s2)[V], bool mine, const Args& a, int width, float2* red,
                                          F f) {
  const int tc = threadIdx.x % a.sum.tc;
  int rows = a.sum.tr, row = threadIdx.x / a.sum.tc;
  if (64 % a.sum.tc == 0 && a.sum.tc < 64) {
    for (int w = a.sum.tc; w < 64; w <<= 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s1[j] += __shfl_xor(s1[j], w, 64);
        s2[j] += __shfl_xor(s2[j], w, 64);
      }
    }
    rows = kNT / 64;
    row = threadIdx.x / 64;
    mine = mine && (threadIdx.x & 63) < a.sum.tc;
  }
  if (mine) {
#pragma unroll
    for (int j = 0; j < V; ++j) red[row * width + tc * V + j] = make_float2(s1[j], s2[j]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < width; c += kNT) {
    float2 s = red[c];
#pragma unroll 8
    for (int r = 1; r < rows; ++r) {
      const float2 v = red[r * width + c];
      s.x += v.x;
      s.y += v.y;
    }
    f(c, s);
  }
  __syncthreads();
}

// Rows that a thread has under way at a time (a load for a later row is issued as soon as a row
// has been used).  Of 2 to 8 these are the fastest; the backward has two tensors' rows under way.
constexpr int kAhead = 4, kGradAhead = 2;

__device__ __forceinline__ float middle(float a, float b, float c) { return __builtin_amdgcn_fmed3f(a, b, c); }

// One chunk's mean and sum of squares of each group.
template <typename T, int V>
__global__ __launch_bounds__(kNT) void norm_stats_kernel(Args a) {
  extern __shared__ float2 lds[];            // [cb] mean and squares of a channel, then the row threads' sums
  float2* chan = lds;
  float2* red = lds + a.sum.cb;
  const Share sh = share_of(a, a.sum);
  const int chunk = blockIdx.x;
  const int64_t r0 = chunk * a.sum.rows, r1 = min(a.P, r0 + a.sum.rows), rm = (r0 + r1) / 2;
  const float n = static_cast<float>(r1 - r0);
  const int tc = threadIdx.x % a.sum.tc, tr = threadIdx.x / a.sum.tc, VR = sh.width / V;
  const T* base = static_cast<const T*>(a.x) + static_cast<int64_t>(sh.b) * a.P * a.C + sh.c0;
  for (int v0 = 0; v0 < VR; v0 += a.sum.tc) {
    const int width = min(a.sum.tc, VR - v0) * V;
    const bool mine = tr < a.sum.tr && tc * V < width;
    float s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
    if (mine) {
      const T* p = base + (v0 + tc) * V;
      const Vec<T, V> x0 = load<T, V>(p + r0 * a.C), xm = load<T, V>(p + rm * a.C), x1 = load<T, V>(p + (r1 - 1) * a.C);
      Vec<T, V> v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (r0 + tr + k * a.sum.tr < r1) v[k] = load<T, V>(p + (r0 + tr + k * a.sum.tr) * a.C);
      float ref[V];
#pragma unroll
      for (int j = 0; j < V; ++j) ref[j] = middle(widen(x0.e[j]), widen(xm.e[j]), widen(x1.e[j]));
      for (int64_t r = r0 + tr; r < r1; r += kAhead * a.sum.tr) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int64_t row = r + k * a.sum.tr, next = row + kAhead * a.sum.tr;
          if (row >= r1) break;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float d = widen(v[k].e[j]) - ref[j];
            s1[j] += d;
            s2[j] = fmaf(d, d, s2[j]);
          }
          if (next < r1) v[k] = load<T, V>(p + next * a.C);
        }
      }
    }
    join_rows<V>(s1, s2, mine, a, width, red, [&](int c, float2 s) {
      const T* p = base + v0 * V + c;
      const float ref = middle(widen(p[r0 * a.C]), widen(p[rm * a.C]), widen(p[(r1 - 1) * a.C])), m = s.x / n;
      chan[v0 * V + c] = make_float2(ref + m, not_below_0(s.y - s.x * m));
    });
  }
  // channels -> groups, all of count n
  const int L = lanes_of(sh.ng), lane = threadIdx.x % L;
  for (int g = threadIdx.x / L; g < sh.ng; g += kNT / L) {
    const float2* c = chan + g * a.Cg;
    float m = 0.f, q = 0.f;
    for (int i = lane; i < a.Cg; i += L) m += c[i].x;
    m = lanes_sum(m, L) / a.Cg;
    for (int i = lane; i < a.Cg; i += L) {
      const float d = c[i].x - m;
      q += fmaf(n * d, d, c[i].y);
    }
    q = lanes_sum(q, L);
    if (lane == 0)
      reinterpret_cast<float2*>(a.gpart)[(static_cast<int64_t>(sh.b) * a.G + sh.g0 + g) * a.sum.blocks + chunk] =
          make_float2(m, q);
  }
}

// Joins the chunks' parts of the groups in its columns, then writes its rows; its first rows are
// loaded before the join, which would else be waited for with nothing under way.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_write_kernel(Args a) {
  extern __shared__ float2 lds[];            // [cb / Cg] mean, rstd
  const Share sh = share_of(a, a.write);
  const int64_t r0 = blockIdx.x * a.write.rows, r1 = min(a.P, r0 + a.write.rows);
  const int64_t base = static_cast<int64_t>(sh.b) * a.P * a.C + sh.c0;
  const int tc = threadIdx.x % a.write.tc, tr = threadIdx.x / a.write.tc, VR = sh.width / V;
  const bool writes = tr < a.write.tr;
  const T* x = static_cast<const T*>(a.x) + base;
  T* out = static_cast<T*>(a.out) + base;
  Vec<T, V> v[kAhead];
  const auto fetch = [&](int v0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (r0 + tr + k * a.write.tr < r1) v[k] = load<T, V>(x + (r0 + tr + k * a.write.tr) * a.C + v0 * V);
  };
  if (writes && tc < VR) fetch(tc);          // on their way while the parts are joined
  const int L = lanes_of(sh.ng), lane = threadIdx.x % L;
  const float2* part = reinterpret_cast<const float2*>(a.gpart) + (static_cast<int64_t>(sh.b) * a.G + sh.g0) * a.sum.blocks;
  const float nfull = static_cast<float>(a.sum.rows) * a.Cg;
  const float nlast = static_cast<float>(a.P - (a.sum.blocks - 1) * a.sum.rows) * a.Cg;
  const float total = static_cast<float>(a.P) * a.Cg;
  for (int g = threadIdx.x / L; g < sh.ng; g += kNT / L) {
    const float ref = part[g * a.sum.blocks].x;
    float s1 = 0.f, s2 = 0.f;
    for (int k = lane; k < a.sum.blocks; k += L) {
      const float2 p = part[g * a.sum.blocks + k];
      const float n = k == a.sum.blocks - 1 ? nlast : nfull, d = p.x - ref;
      s1 = fmaf(n, d, s1);
      s2 += fmaf(n * d, d, p.y);
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0) {
      const float m = s1 / total, var = not_below_0(s2 - s1 * m) / total;
      const float mean = ref + m, rstd = 1.f / sqrtf(var + a.eps);
      lds[g] = make_float2(mean, rstd);
      if (blockIdx.x == 0) {
        const int64_t at = static_cast<int64_t>(sh.b) * a.G + sh.g0 + g;
        if (a.mean != nullptr) a.mean[at] = mean;
        if (a.rstd != nullptr) a.rstd[at] = rstd;
      }
    }
  }
  __syncthreads();
  if (!writes) return;
  for (int v0 = tc; v0 < VR; v0 += a.write.tc) {
    float mean[V], scale[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = v0 * V + j;
      const float2 s = lds[c / a.Cg];
      mean[j] = s.x;
      scale[j] = a.w == nullptr ? s.y : s.y * widen(static_cast<const T*>(a.w)[sh.c0 + c]);
      bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[sh.c0 + c]);
    }
    if (v0 != tc) fetch(v0);
    for (int64_t r = r0 + tr; r < r1; r += kAhead * a.write.tr) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t row = r + k * a.write.tr, next = row + kAhead * a.write.tr;
        if (row >= r1) break;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = act<T, ACT>(fmaf(widen(v[k].e[j]) - mean[j], scale[j], bias[j]));
        if (next < r1) v[k] = load<T, V>(x + next * a.C + v0 * V);
        store<T, V>(out + row * a.C + v0 * V, y);
      }
    }
  }
}

// One chunk's sums of gz and gz n: of each channel (the parameters' gradients), and weighted, of each
// group.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_grad_sums_kernel(Args a) {
  extern __shared__ float2 lds[];            // [cb] sums of gz and gz n of a channel, then the row threads'
  float2* chan = lds;
  float2* red = lds + a.sum.cb;
  const Share sh = share_of(a, a.sum);
  const int chunk = blockIdx.x;
  const int64_t r0 = chunk * a.sum.rows, r1 = min(a.P, r0 + a.sum.rows);
  const int tc = threadIdx.x % a.sum.tc, tr = threadIdx.x / a.sum.tc, VR = sh.width / V;
  const int64_t base = static_cast<int64_t>(sh.b) * a.P * a.C + sh.c0;
  float2* cpart = reinterpret_cast<float2*>(a.cpart) + (static_cast<int64_t>(sh.b) * a.sum.blocks + chunk) * a.C + sh.c0;
  for (int v0 = 0; v0 < VR; v0 += a.sum.tc) {
    const int width = min(a.sum.tc, VR - v0) * V;
    const bool mine = tr < a.sum.tr && tc * V < width;
    float s1[V], s2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
    if (mine) {
      const T* p = static_cast<const T*>(a.x) + base + (v0 + tc) * V;
      const T* q = static_cast<const T*>(a.g) + base + (v0 + tc) * V;
      Vec<T, V> v[kGradAhead], gr[kGradAhead];
#pragma unroll
      for (int k = 0; k < kGradAhead; ++k)
        if (r0 + tr + k * a.sum.tr < r1) {
          v[k] = load<T, V>(p + (r0 + tr + k * a.sum.tr) * a.C);
          gr[k] = load<T, V>(q + (r0 + tr + k * a.sum.tr) * a.C);
        }
      float mean[V], rstd[V], w[V], bias[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = sh.c0 + (v0 + tc) * V + j, g = c / a.Cg;
        mean[j] = a.mean[static_cast<int64_t>(sh.b) * a.G + g];
        rstd[j] = a.rstd[static_cast<int64_t>(sh.b) * a.G + g];
        w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c]);
        bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
      }
      for (int64_t r = r0 + tr; r < r1; r += kGradAhead * a.sum.tr) {
#pragma unroll
        for (int k = 0; k < kGradAhead; ++k) {
          const int64_t row = r + k * a.sum.tr, next = row + kGradAhead * a.sum.tr;
          if (row >= r1) break;
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float n = (widen(v[k].e[j]) - mean[j]) * rstd[j];
            const float gz = widen(gr[k].e[j]) * slope<T, ACT>(fmaf(n, w[j], bias[j]));
            s1[j] += gz;
            s2[j] = fmaf(gz, n, s2[j]);
          }
          if (next < r1) {
            v[k] = load<T, V>(p + next * a.C);
            gr[k] = load<T, V>(q + next * a.C);
          }
        }
      }
    }
    join_rows<V>(s1, s2, mine, a, width, red, [&](int c, float2 s) {
      const float w = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[sh.c0 + v0 * V + c]);
      cpart[v0 * V + c] = s;
      chan[v0 * V + c] = make_float2(s.x * w, s.y * w);
    });
  }
  const int L = lanes_of(sh.ng), lane = threadIdx.x % L;
  for (int g = threadIdx.x / L; g < sh.ng; g += kNT / L) {
    const float2* c = chan + g * a.Cg;
    float s1 = 0.f, s2 = 0.f;
    for (int i = lane; i < a.Cg; i += L) {
      s1 += c[i].x;
      s2 += c[i].y;
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0)
      reinterpret_cast<float2*>(a.gpart)[(static_cast<int64_t>(sh.b) * a.G + sh.g0 + g) * a.sum.blocks + chunk] =
          make_float2(s1, s2);
  }
}

// Batch elements 0 .. B-1 write grad_x; the workgroups of "batch element" B of the grid add the
// chunks of 32 channels each for grad_weight and grad_bias.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_grad_write_kernel(Args a) {
  extern __shared__ float2 lds[];
  if (static_cast<int>(blockIdx.z) == a.B) {
    const int c = (blockIdx.y * gridDim.x + blockIdx.x) * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
    constexpr int PARTS = kNT / 32;
    const int64_t n = static_cast<int64_t>(a.B) * a.sum.blocks;
    float2 s = make_float2(0.f, 0.f);
    if (c < a.C)
#pragma unroll 4
      for (int64_t k = part; k < n; k += PARTS) {
        const float2 v = reinterpret_cast<const float2*>(a.cpart)[k * a.C + c];
        s.x += v.x;
        s.y += v.y;
      }
    lds[threadIdx.x] = s;
    __syncthreads();
    if (part != 0 || c >= a.C) return;
    for (int k = 1; k < PARTS; ++k) {
      s.x += lds[k * 32 + threadIdx.x].x;
      s.y += lds[k * 32 + threadIdx.x].y;
    }
    if (a.gw != nullptr) static_cast<T*>(a.gw)[c] = narrow<T>(s.y);
    if (a.gb != nullptr) static_cast<T*>(a.gb)[c] = narrow<T>(s.x);
    return;
  }
  if (static_cast<int>(blockIdx.x) >= a.write.blocks) return;
  const Share sh = share_of(a, a.write);
  const int64_t r0 = blockIdx.x * a.write.rows, r1 = min(a.P, r0 + a.write.rows);
  const int64_t base = static_cast<int64_t>(sh.b) * a.P * a.C + sh.c0;
  const int tc = threadIdx.x % a.write.tc, tr = threadIdx.x / a.write.tc, VR = sh.width / V;
  const bool writes = tr < a.write.tr;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* go = static_cast<const T*>(a.g) + base;
  T* out = static_cast<T*>(a.out) + base;
  Vec<T, V> v[kGradAhead], gr[kGradAhead];
  const auto fetch = [&](int v0) {
#pragma unroll
    for (int k = 0; k < kGradAhead; ++k)
      if (r0 + tr + k * a.write.tr < r1) {
        v[k] = load<T, V>(x + (r0 + tr + k * a.write.tr) * a.C + v0 * V);
        gr[k] = load<T, V>(go + (r0 + tr + k * a.write.tr) * a.C + v0 * V);
      }
  };
  if (writes && tc < VR) fetch(tc);
  const int L = lanes_of(sh.ng), lane = threadIdx.x % L;
  const int64_t group = static_cast<int64_t>(sh.b) * a.G + sh.g0;
  const float2* part = reinterpret_cast<const float2*>(a.gpart) + group * a.sum.blocks;
  const float inv = 1.f / (static_cast<float>(a.P) * a.Cg);
  for (int g = threadIdx.x / L; g < sh.ng; g += kNT / L) {
    float s1 = 0.f, s2 = 0.f;
    for (int k = lane; k < a.sum.blocks; k += L) {
      const float2 p = part[g * a.sum.blocks + k];
      s1 += p.x;
      s2 += p.y;
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0) lds[g] = make_float2(s1 * inv, s2 * inv);
  }
  __syncthreads();
  if (!writes) return;
  for (int v0 = tc; v0 < VR; v0 += a.write.tc) {
    float mean[V], rstd[V], w[V], bias[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = v0 * V + j, g = c / a.Cg;
      mean[j] = a.mean[group + g];
      rstd[j] = a.rstd[group + g];
      w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[sh.c0 + c]);
      bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[sh.c0 + c]);
      m1[j] = lds[g].x;
      m2[j] = lds[g].y;
    }
    if (v0 != tc) fetch(v0);
    for (int64_t r = r0 + tr; r < r1; r += kGradAhead * a.write.tr) {
#pragma unroll
      for (int k = 0; k < kGradAhead; ++k) {
        const int64_t row = r + k * a.write.tr, next = row + kGradAhead * a.write.tr;
        if (row >= r1) break;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float n = (widen(v[k].e[j]) - mean[j]) * rstd[j];
          const float gz = widen(gr[k].e[j]) * slope<T, ACT>(fmaf(n, w[j], bias[j]));
          y[j] = rstd[j] * (fmaf(gz, w[j], -m1[j]) - n * m2[j]);
        }
        if (next < r1) {
          v[k] = load<T, V>(x + next * a.C + v0 * V);
          gr[k] = load<T, V>(go + next * a.C + v0 * V);
        }
        store<T, V>(out + row * a.C + v0 * V, y);
      }
    }
  }
}

// ---- slices: a group of one batch element in the registers of a workgroup

constexpr int kST = 1024;        // threads
constexpr int kHeld = 8;         // vectors of a thread, in the forward
// and in the backward, which holds the map and the gradient
constexpr int grad_held(int es) { return es == 2 ? 4 : 6; }

// sums over the workgroup, the same in every thread
__device__ __forceinline__ float2 block_sum(float a, float b, float2* lds) {
  a = lanes_sum(a, 64);
  b = lanes_sum(b, 64);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
  if (lane == 0) lds[wave] = make_float2(a, b);
  __syncthreads();
  float2 s = lds[0];
#pragma unroll
  for (int i = 1; i < kST / 64; ++i) {
    s.x += lds[i].x;
    s.y += lds[i].y;
  }
  return s;
}

// Workgroups of a launch fall to the 8 XCDs in turn; groups that share lines of memory are given
// to one XCD: workgroup i of n takes unit (i % 8) * ceil(n / 8) + i / 8 (n or more: none).
__device__ __forceinline__ int unit_of(int n) { return static_cast<int>(blockIdx.x % 8) * ((n + 7) / 8) + blockIdx.x / 8; }

// A group in the registers of a workgroup, read once.  Threads form rows of vpr vectors (those of a
// group's row) and `rows` positions at a time, so that a thread keeps its channels.  Few workgroups
// (one for each group and batch element) against one launch and one reading: 1 x 1050 positions of
// 256 bf16 channels in 32 groups 9.1 us against 12.4 as two passes, 3 x 1551 of 96 fp32 channels in 8
// groups with their gradients 15.0 to 16.0 against 20.6.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kST) void norm_slice_kernel(Args a) {
  __shared__ float2 lds[kST / 64];
  const int unit = unit_of(a.B * a.G);
  if (unit >= a.B * a.G) return;
  const int b = unit / a.G, g = unit % a.G, vpr = a.Cg / V, rows = kST / vpr;
  const int sub = threadIdx.x % vpr, row = threadIdx.x / vpr, P = static_cast<int>(a.P);
  const int64_t at = static_cast<int64_t>(b) * a.P * a.C + g * a.Cg + sub * V;
  const T* x = static_cast<const T*>(a.x) + at;
  T* out = static_cast<T*>(a.out) + at;
  const bool mine = row < rows;
  Vec<T, V> v[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (mine && row + k * rows < P) v[k] = load<T, V>(x + static_cast<int64_t>(row + k * rows) * a.C);
  float w[V], bias[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = g * a.Cg + sub * V + j;
    w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c]);
    bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
  }
  const float inv = 1.f / (static_cast<float>(a.P) * a.Cg);
  // sums about a value that is taken to be near the mean (of the first position's first channels)
  const Vec<T, V> first = load<T, V>(static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.P * a.C + g * a.Cg);
  float ref = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) ref += widen(first.e[j]);
  ref *= 1.f / V;
  float s = 0.f, q = 0.f;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (mine && row + k * rows < P)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = widen(v[k].e[j]) - ref;
        s += d;
        q = fmaf(d, d, q);
      }
  float2 t = block_sum(s, q, lds);
  const float shift = t.x * inv, m = ref + shift;
  float var = not_below_0(t.y * inv - shift * shift);
  if (shift * shift > 16.f * var) {   // the value near the mean was not near it: its squares once more, about the mean
    q = 0.f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (mine && row + k * rows < P)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = widen(v[k].e[j]) - m;
          q = fmaf(d, d, q);
        }
    t = block_sum(q, 0.f, lds);
    var = t.x * inv;
  }
  const float rstd = 1.f / sqrtf(var + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[unit] = m;
    if (a.rstd != nullptr) a.rstd[unit] = rstd;
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (mine && row + k * rows < P) {
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = act<T, ACT>(fmaf(widen(v[k].e[j]) - m, rstd * w[j], bias[j]));
      store<T, V>(out + static_cast<int64_t>(row + k * rows) * a.C, y);
    }
}

template <typename T, int V, int ACT>
__global__ __launch_bounds__(kST) void norm_grad_slice_kernel(Args a) {
  constexpr int HELD = grad_held(sizeof(T));
  __shared__ float2 lds[kST / 64];
  extern __shared__ float2 sums[];           // [V][kST] sums of gz and gz n of each thread's channels
  const int unit = unit_of(a.B * a.G);
  if (unit >= a.B * a.G) return;
  const int b = unit / a.G, g = unit % a.G, vpr = a.Cg / V, rows = kST / vpr;
  const int sub = threadIdx.x % vpr, row = threadIdx.x / vpr, P = static_cast<int>(a.P);
  const int64_t at = static_cast<int64_t>(b) * a.P * a.C + g * a.Cg + sub * V;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* go = static_cast<const T*>(a.g) + at;
  const bool mine = row < rows, params = a.gw != nullptr || a.gb != nullptr;
  Vec<T, V> v[HELD], gr[HELD];
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (mine && row + k * rows < P) {
      v[k] = load<T, V>(x + static_cast<int64_t>(row + k * rows) * a.C);
      gr[k] = load<T, V>(go + static_cast<int64_t>(row + k * rows) * a.C);
    }
  const float mean = a.mean[unit], rstd = a.rstd[unit];
  float w[V], bias[V], s1[V], s2[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = g * a.Cg + sub * V + j;
    w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c]);
    bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
    s1[j] = s2[j] = 0.f;
  }
  const auto gz_of = [&](int k, int j, float& n) {
    n = (widen(v[k].e[j]) - mean) * rstd;
    return widen(gr[k].e[j]) * slope<T, ACT>(fmaf(n, w[j], bias[j]));
  };
#pragma unroll
  for (int k = 0; k < HELD; ++k)
    if (mine && row + k * rows < P)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float n;
        const float gz = gz_of(k, j, n);
        if constexpr (sizeof(T) == 4) gr[k].e[j] = gz;   // kept for the second use (bf16 has no room for it)
        s1[j] += gz;
        s2[j] = fmaf(gz, n, s2[j]);
      }
  float t1 = 0.f, t2 = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    t1 = fmaf(s1[j], w[j], t1);
    t2 = fmaf(s2[j], w[j], t2);
  }
  if (params) {
#pragma unroll
    for (int j = 0; j < V; ++j) sums[j * kST + threadIdx.x] = make_float2(s1[j], s2[j]);
  }
  const float2 t = block_sum(t1, t2, lds);   // (its barriers also complete `sums`)
  const float inv = 1.f / (static_cast<float>(a.P) * a.Cg), m1 = t.x * inv, m2 = t.y * inv;
  if (a.out != nullptr) {
    T* out = static_cast<T*>(a.out) + at;
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (mine && row + k * rows < P) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float n, gz;
          if constexpr (sizeof(T) == 4) {
            n = (widen(v[k].e[j]) - mean) * rstd;
            gz = widen(gr[k].e[j]);
          } else {
            gz = gz_of(k, j, n);
          }
          y[j] = rstd * (fmaf(gz, w[j], -m1) - n * m2);
        }
        store<T, V>(out + static_cast<int64_t>(row + k * rows) * a.C, y);
      }
  }
  if (!params) return;
  // the channels' sums over the rows of threads, 16 lanes for each channel
  const int used = min(rows, P);
  for (int c = threadIdx.x / 16; c < a.Cg; c += kST / 16) {
    float2 s = make_float2(0.f, 0.f);
    for (int r = threadIdx.x % 16; r < used; r += 16) {
      const float2 q = sums[(c % V) * kST + r * vpr + c / V];
      s.x += q.x;
      s.y += q.y;
    }
    s.x = lanes_sum(s.x, 16);
    s.y = lanes_sum(s.y, 16);
    if (threadIdx.x % 16 != 0) continue;
    const int ch = g * a.Cg + c;
    if (a.B > 1) {
      reinterpret_cast<float2*>(a.cpart)[static_cast<int64_t>(b) * a.C + ch] = s;
    } else {
      if (a.gw != nullptr) static_cast<T*>(a.gw)[ch] = narrow<T>(s.y);
      if (a.gb != nullptr) static_cast<T*>(a.gb)[ch] = narrow<T>(s.x);
    }
  }
}

// The slices' channel sums of the batch elements, added in order.
template <typename T>
__global__ __launch_bounds__(256) void norm_add_params_kernel(Args a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.C) return;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int b = 0; b < a.B; ++b) {
    const float2 q = reinterpret_cast<const float2*>(a.cpart)[static_cast<int64_t>(b) * a.C + c];
    s.x += q.x;
    s.y += q.y;
  }
  if (a.gw != nullptr) static_cast<T*>(a.gw)[c] = narrow<T>(s.y);
  if (a.gb != nullptr) static_cast<T*>(a.gb)[c] = narrow<T>(s.x);
}

int check(const dcn_norm_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  if (d->batch < 0 || d->positions < 1 || d->channels < 1 || d->groups < 1 || d->channels % d->groups != 0 ||
      !std::isfinite(d->eps) || d->eps < 0.f || d->activation < DCN_ACT_NONE || d->activation > DCN_ACT_GELU)
    return DCN_E_ARG;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  if (d->channels > kMaxC || d->batch > 65534 || d->positions > 2147483647) return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

constexpr int kMaxChunks = 256;

// Workgroups of whole groups of at least `bytes` of a row; `total` of them in all, of at least
// two sweeps of the threads, and at most `most` along the positions.
Cut cut_of(const Args& a, int V, int es, int bytes, int64_t total, int64_t most) {
  Cut c{};
  c.cb = a.Cg;
  while (c.cb % V != 0) c.cb += a.Cg;        // V is 1, 4 or 8 and divides C: ends at C at the latest
  const int unit = c.cb;
  while (c.cb < a.C && c.cb * es < bytes) c.cb += unit;
  c.cb = std::min(c.cb, a.C);
  c.tc = std::min(c.cb / V, kNT);
  c.tr = kNT / c.tc;
  const int64_t columns = static_cast<int64_t>(std::max(a.B, 1)) * ((a.C + c.cb - 1) / c.cb);
  const int64_t n = std::min(std::min(std::max<int64_t>(1, total / columns), most),
                             std::max<int64_t>(1, a.P / (2 * c.tr)));
  c.rows = (a.P + n - 1) / n;
  c.blocks = static_cast<int>((a.P + c.rows - 1) / c.rows);
  return c;
}

// The summing pass reads whole rows (4 KB at a time where they are longer): in columns of 128
// bytes it took 22 us where rows take 15.6 (8 x 16800 positions of 256 bf16 channels).  The
// writing pass takes columns of a line of memory (128 bytes), whose few groups are quick to
// join: whole rows took 27.8 us, these 26.  One workgroup for each CU in both: with two the
// backward at 2 x 16800 positions took 32 us, with one 26.4 (forward at batch 8: 43.5, 42.7; calls on one
// map, of which the 256 MB cache holds part).
void plan(const dcn_norm_desc* d, int V, int es, Args* a) {
  a->B = static_cast<int>(d->batch);
  a->P = d->positions;
  a->C = static_cast<int>(d->channels);
  a->G = static_cast<int>(d->groups);
  a->Cg = a->C / a->G;
  a->eps = d->eps;
  a->sum = cut_of(*a, V, es, 4096, 256, kMaxChunks);
  a->write = cut_of(*a, V, es, 128, 256, a->P);
}
int columns(const Args& a, const Cut& c) { return (a.C + c.cb - 1) / c.cb; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether a group's positions fit `held` vectors (of V elements, within the group) of each thread of
// a slice, and one launch takes a slice for each group and batch element: a dispatch counts its
// threads in 32 bits.
bool fits_slice(const dcn_norm_desc* d, int V, int held) {
  const int64_t Cg = d->channels / d->groups, most = (int64_t{1} << 32) / kST - 8;
  return Cg % V == 0 && Cg / V <= kST && d->positions <= held * (kST / (Cg / V)) && d->batch * d->groups <= most;
}

// What the parts of a call take, for either vector width (16-byte rows or single elements, known at
// the call): `group` bytes of the groups' parts, then `chan` of the channels'.  A pass of sums has
// max(B, 256) chunks at most over all batch elements (cut_of); a slice has no parts but the channels'
// sums of each batch element, and is certain where single elements fit it.
struct Parts {
  size_t group, chan;
};
Parts forward_parts(const dcn_norm_desc* d) {
  if (d->batch == 0 || fits_slice(d, 1, kHeld)) return {0, 0};
  return {up256(static_cast<size_t>(std::max<int64_t>(d->batch, kMaxChunks)) * d->groups * 8), 0};
}
Parts backward_parts(const dcn_norm_desc* d) {
  if (d->batch == 0) return {0, 0};
  if (fits_slice(d, 1, grad_held(d->dtype == DCN_BF16 ? 2 : 4)))
    return {0, d->batch > 1 ? up256(static_cast<size_t>(d->batch) * d->channels * 8) : 0};
  const size_t chunks = static_cast<size_t>(std::max<int64_t>(d->batch, kMaxChunks));
  return {up256(chunks * d->groups * 8), up256(chunks * d->channels * 8)};
}

size_t sums_lds(const Args& a, int V) {
  return (static_cast<size_t>(a.sum.cb) + static_cast<size_t>(a.sum.tr) * a.sum.tc * V) * sizeof(float2);
}

bool launch(const void* fn, dim3 grid, size_t lds, Args* a, hipStream_t stream, int threads = kNT) {
  void* args[] = {a};
  return hipLaunchKernel(fn, grid, dim3(threads), args, lds, stream) == hipSuccess;
}

template <typename T, int V>
const void* write_kernel(int act) {
  switch (act) {
    case DCN_ACT_RELU: return reinterpret_cast<const void*>(&norm_write_kernel<T, V, DCN_ACT_RELU>);
    case DCN_ACT_SILU: return reinterpret_cast<const void*>(&norm_write_kernel<T, V, DCN_ACT_SILU>);
    case DCN_ACT_GELU: return reinterpret_cast<const void*>(&norm_write_kernel<T, V, DCN_ACT_GELU>);
    default: return reinterpret_cast<const void*>(&norm_write_kernel<T, V, DCN_ACT_NONE>);
  }
}
template <typename T, int V>
const void* sums_kernel(int act) {
  switch (act) {
    case DCN_ACT_RELU: return reinterpret_cast<const void*>(&norm_grad_sums_kernel<T, V, DCN_ACT_RELU>);
    case DCN_ACT_SILU: return reinterpret_cast<const void*>(&norm_grad_sums_kernel<T, V, DCN_ACT_SILU>);
    case DCN_ACT_GELU: return reinterpret_cast<const void*>(&norm_grad_sums_kernel<T, V, DCN_ACT_GELU>);
    default: return reinterpret_cast<const void*>(&norm_grad_sums_kernel<T, V, DCN_ACT_NONE>);
  }
}
template <typename T, int V>
const void* grad_write_kernel(int act) {
  switch (act) {
    case DCN_ACT_RELU: return reinterpret_cast<const void*>(&norm_grad_write_kernel<T, V, DCN_ACT_RELU>);
    case DCN_ACT_SILU: return reinterpret_cast<const void*>(&norm_grad_write_kernel<T, V, DCN_ACT_SILU>);
    case DCN_ACT_GELU: return reinterpret_cast<const void*>(&norm_grad_write_kernel<T, V, DCN_ACT_GELU>);
    default: return reinterpret_cast<const void*>(&norm_grad_write_kernel<T, V, DCN_ACT_NONE>);
  }
}

template <typename T, int V>
const void* slice_kernel(int act) {
  switch (act) {
    case DCN_ACT_RELU: return reinterpret_cast<const void*>(&norm_slice_kernel<T, V, DCN_ACT_RELU>);
    case DCN_ACT_SILU: return reinterpret_cast<const void*>(&norm_slice_kernel<T, V, DCN_ACT_SILU>);
    case DCN_ACT_GELU: return reinterpret_cast<const void*>(&norm_slice_kernel<T, V, DCN_ACT_GELU>);
    default: return reinterpret_cast<const void*>(&norm_slice_kernel<T, V, DCN_ACT_NONE>);
  }
}
template <typename T, int V>
const void* grad_slice_kernel(int act) {
  switch (act) {
    case DCN_ACT_RELU: return reinterpret_cast<const void*>(&norm_grad_slice_kernel<T, V, DCN_ACT_RELU>);
    case DCN_ACT_SILU: return reinterpret_cast<const void*>(&norm_grad_slice_kernel<T, V, DCN_ACT_SILU>);
    case DCN_ACT_GELU: return reinterpret_cast<const void*>(&norm_grad_slice_kernel<T, V, DCN_ACT_GELU>);
    default: return reinterpret_cast<const void*>(&norm_grad_slice_kernel<T, V, DCN_ACT_NONE>);
  }
}

template <typename T, int V>
int forward(const dcn_norm_desc* d, Args* a, hipStream_t stream) {
  plan(d, V, sizeof(T), a);
  const bool whole = fits_slice(d, V, kHeld);
  if (whole || fits_slice(d, 1, kHeld))
    return launch(whole ? slice_kernel<T, V>(d->activation) : slice_kernel<T, 1>(d->activation),
                  dim3((a->B * a->G + 7) / 8 * 8), 0, a, stream, kST)
               ? DCN_OK
               : DCN_E_HIP;
  if (!launch(reinterpret_cast<const void*>(&norm_stats_kernel<T, V>), dim3(a->sum.blocks, columns(*a, a->sum), a->B), sums_lds(*a, V), a,
              stream))
    return DCN_E_HIP;
  return launch(write_kernel<T, V>(d->activation), dim3(a->write.blocks, columns(*a, a->write), a->B), a->write.cb / a->Cg * sizeof(float2), a, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

template <typename T, int V>
int backward(const dcn_norm_desc* d, Args* a, hipStream_t stream) {
  plan(d, V, sizeof(T), a);
  const bool params = a->gw != nullptr || a->gb != nullptr;
  if (a->B == 0 && !params) return DCN_OK;   // grad_x is empty: a grid of no batch element is no launch
  const bool whole = fits_slice(d, V, grad_held(sizeof(T)));
  if (a->B > 0 && (whole || fits_slice(d, 1, grad_held(sizeof(T))))) {
    if (!launch(whole ? grad_slice_kernel<T, V>(d->activation) : grad_slice_kernel<T, 1>(d->activation),
                dim3((a->B * a->G + 7) / 8 * 8), params ? static_cast<size_t>(V) * kST * sizeof(float2) : 0, a, stream,
                kST))
      return DCN_E_HIP;
    return !params || a->B == 1 ||
                   launch(reinterpret_cast<const void*>(&norm_add_params_kernel<T>), dim3((a->C + 255) / 256), 0, a,
                          stream, 256)
               ? DCN_OK
               : DCN_E_HIP;
  }
  if (a->B > 0 &&
      !launch(sums_kernel<T, V>(d->activation), dim3(a->sum.blocks, columns(*a, a->sum), a->B), sums_lds(*a, V), a, stream))
    return DCN_E_HIP;
  if (a->out == nullptr) a->write.blocks = 0;
  const int by = columns(*a, a->write), gx = std::max(a->write.blocks, params ? ((a->C + 31) / 32 + by - 1) / by : 0);
  if (gx == 0) return DCN_OK;
  return launch(grad_write_kernel<T, V>(d->activation), dim3(gx, by, a->B + (params ? 1 : 0)),
                static_cast<size_t>(std::max(a->write.cb / a->Cg, kNT)) * sizeof(float2), a, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int workspace_status(const void* ws, size_t have, size_t need) {
  return need > 0 && (ws == nullptr || have < need || reinterpret_cast<uintptr_t>(ws) % 256 != 0) ? DCN_E_WORKSPACE
                                                                                                  : DCN_OK;
}

}  // namespace
}  // namespace norm
}  // namespace dcn

extern "C" int dcn_group_norm_workspace_bytes(const dcn_norm_desc* d, size_t* bytes) {
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = dcn::norm::check(d);
  if (rc == DCN_OK) *bytes = dcn::norm::forward_parts(d).group;
  return rc;
}

extern "C" int dcn_group_norm(const dcn_norm_desc* d, const void* x, const void* weight, const void* bias, void* out,
                              float* mean, float* rstd, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  using namespace dcn::norm;
  int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0) return DCN_OK;
  if (x == nullptr || out == nullptr) return DCN_E_ARG;
  rc = workspace_status(workspace, workspace_bytes, forward_parts(d).group);
  if (rc != DCN_OK) return rc;
  Args a{};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.out = out;
  a.mean = mean;
  a.rstd = rstd;
  a.gpart = static_cast<float*>(workspace);
  const bool bf16 = d->dtype == DCN_BF16, vec = aligned(x) && aligned(out) && d->channels % (bf16 ? 8 : 4) == 0;
  if (bf16) return vec ? forward<uint16_t, 8>(d, &a, stream) : forward<uint16_t, 1>(d, &a, stream);
  return vec ? forward<float, 4>(d, &a, stream) : forward<float, 1>(d, &a, stream);
}

extern "C" int dcn_group_norm_backward_workspace_bytes(const dcn_norm_desc* d, size_t* bytes) {
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = dcn::norm::check(d);
  if (rc != DCN_OK) return rc;
  const dcn::norm::Parts need = dcn::norm::backward_parts(d);
  *bytes = need.group + need.chan;
  return DCN_OK;
}

extern "C" int dcn_group_norm_backward(const dcn_norm_desc* d, const void* x, const void* weight, const void* bias,
                                       const float* mean, const float* rstd, const void* grad_out, void* grad_x,
                                       void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  using namespace dcn::norm;
  int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch > 0 && (x == nullptr || mean == nullptr || rstd == nullptr || grad_out == nullptr)) return DCN_E_ARG;
  const Parts need = backward_parts(d);
  rc = workspace_status(workspace, workspace_bytes, need.group + need.chan);
  if (rc != DCN_OK) return rc;
  Args a{};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.g = grad_out;
  a.out = grad_x;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.gw = grad_weight;
  a.gb = grad_bias;
  a.gpart = static_cast<float*>(workspace);
  a.cpart = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + need.group);
  const bool bf16 = d->dtype == DCN_BF16;
  const bool vec = aligned(x) && aligned(grad_out) && aligned(grad_x) && d->channels % (bf16 ? 8 : 4) == 0;
  if (bf16) return vec ? backward<uint16_t, 8>(d, &a, stream) : backward<uint16_t, 1>(d, &a, stream);
  return vec ? backward<float, 4>(d, &a, stream) : backward<float, 1>(d, &a, stream);
}

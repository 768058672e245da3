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
// Both directions read their input twice: a pass that sums over chunks of positions (one
// workgroup each, whole rows: contiguous memory), and a pass that first joins the chunks'
// parts and then writes.  Sums are joined in a fixed order; there are no atomics.
//
// The variance is formed from sums of d and d^2, d = x - r with r the chunk's first value of
// the channel, and chunks and channels are joined as (count, mean, sum of squares about the
// mean): nothing large cancels where the mean is far from 0.
//
// Arithmetic: fp32 throughout, every output rounded to its type once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"

namespace dcn {
namespace norm {
namespace {

constexpr int kNT = 512;
constexpr int kMaxC = 8192;

struct Args {
  const void *x, *w, *b, *g;
  void* out;                 // forward: out; backward: grad_x
  float *mean, *rstd;        // [B][G]
  void *gw, *gb;
  float* gpart;              // [B][chunks][G][2]
  float* cpart;              // backward: [B][chunks][C][2]
  int64_t P;
  int B, C, G, Cg;
  int chunks;                // of the summing pass
  int64_t rpc;               // positions of one
  int ablocks;               // of the writing pass
  int64_t rpa;
  int tc, tr;                // threads along a row, rows at a time
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

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
template <int ACT>
__device__ __forceinline__ float act(float z) {
  if (ACT == DCN_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (ACT == DCN_ACT_SILU) return z * sigmoid(z);
  if (ACT == DCN_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}
template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == DCN_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == DCN_ACT_SILU) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if (ACT == DCN_ACT_GELU)
    return fmaf(z * 0.39894228040143268f, __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z),
                0.5f * (1.f + erff(z * 0.70710678118654752f)));
  return 1.f;
}

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

// joins sums over the row threads: [tr][width] pairs in `red` -> f(channel of the block, sum0, sum1)
template <typename F>
__device__ __forceinline__ void join_rows(const float2* red, int tr, int width, F f) {
  for (int c = threadIdx.x; c < width; c += kNT) {
    float2 s = red[c];
    for (int r = 1; r < tr; ++r) {
      const float2 v = red[r * width + c];
      s.x += v.x;
      s.y += v.y;
    }
    f(c, s);
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kNT) void norm_stats_kernel(Args a) {
  extern __shared__ float2 lds[];            // [C] mean and squares of a channel, then the row threads' sums
  float2* chan = lds;
  float2* red = lds + a.C;
  const int chunk = blockIdx.x, b = blockIdx.y;
  const int64_t r0 = chunk * a.rpc, r1 = min(a.P, r0 + a.rpc);
  const float n = static_cast<float>(r1 - r0);
  const int tc = threadIdx.x % a.tc, tr = threadIdx.x / a.tc, VR = a.C / V;
  const T* base = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.P * a.C;
  for (int c0 = 0; c0 < VR; c0 += a.tc) {
    const int width = min(a.tc, VR - c0) * V;
    if (tr < a.tr && tc * V < width) {
      const T* p = base + (c0 + tc) * V;
      const Vec<T, V> ref = load<T, V>(p + r0 * a.C);
      float s1[V], s2[V];
#pragma unroll
      for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.f;
#pragma unroll 4
      for (int64_t r = r0 + tr; r < r1; r += a.tr) {
        const Vec<T, V> v = load<T, V>(p + r * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = widen(v.e[j]) - widen(ref.e[j]);
          s1[j] += d;
          s2[j] = fmaf(d, d, s2[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) red[tr * width + tc * V + j] = make_float2(s1[j], s2[j]);
    }
    __syncthreads();
    join_rows(red, a.tr, width, [&](int c, float2 s) {
      const float ref = widen(base[r0 * a.C + c0 * V + c]), m = s.x / n;
      chan[c0 * V + c] = make_float2(ref + m, fmaxf(s.y - s.x * m, 0.f));
    });
    __syncthreads();
  }
  // channels -> groups, all of count n
  const int L = lanes_of(a.G), lane = threadIdx.x % L;
  for (int g = threadIdx.x / L; g < a.G; g += kNT / L) {
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
      reinterpret_cast<float2*>(a.gpart)[(static_cast<int64_t>(b) * a.chunks + chunk) * a.G + g] = make_float2(m, q);
  }
}

template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_write_kernel(Args a) {
  extern __shared__ float2 lds[];            // [G] mean, rstd
  const int b = blockIdx.y;
  const int L = lanes_of(a.G), lane = threadIdx.x % L;
  const float2* part = reinterpret_cast<const float2*>(a.gpart) + static_cast<int64_t>(b) * a.chunks * a.G;
  const float nfull = static_cast<float>(a.rpc) * a.Cg;
  const float nlast = static_cast<float>(a.P - (a.chunks - 1) * a.rpc) * a.Cg;
  const float total = static_cast<float>(a.P) * a.Cg;
  for (int g = threadIdx.x / L; g < a.G; g += kNT / L) {
    const float ref = part[g].x;
    float s1 = 0.f, s2 = 0.f;
    for (int k = lane; k < a.chunks; k += L) {
      const float2 v = part[static_cast<int64_t>(k) * a.G + g];
      const float n = k == a.chunks - 1 ? nlast : nfull, d = v.x - ref;
      s1 = fmaf(n, d, s1);
      s2 += fmaf(n * d, d, v.y);
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0) {
      const float m = s1 / total, var = fmaxf(s2 - s1 * m, 0.f) / total;
      const float mean = ref + m, rstd = 1.f / sqrtf(var + a.eps);
      lds[g] = make_float2(mean, rstd);
      if (blockIdx.x == 0) {
        if (a.mean != nullptr) a.mean[static_cast<int64_t>(b) * a.G + g] = mean;
        if (a.rstd != nullptr) a.rstd[static_cast<int64_t>(b) * a.G + g] = rstd;
      }
    }
  }
  __syncthreads();
  const int64_t r0 = blockIdx.x * a.rpa, r1 = min(a.P, r0 + a.rpa);
  const int tc = threadIdx.x % a.tc, tr = threadIdx.x / a.tc, VR = a.C / V;
  if (tr >= a.tr) return;
  const int64_t base = static_cast<int64_t>(b) * a.P * a.C;
  for (int c0 = tc; c0 < VR; c0 += a.tc) {
    float mean[V], scale[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = c0 * V + j;
      const float2 s = lds[c / a.Cg];
      mean[j] = s.x;
      scale[j] = a.w == nullptr ? s.y : s.y * widen(static_cast<const T*>(a.w)[c]);
      bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
    }
    const T* p = static_cast<const T*>(a.x) + base + c0 * V;
    T* o = static_cast<T*>(a.out) + base + c0 * V;
#pragma unroll 4
    for (int64_t r = r0 + tr; r < r1; r += a.tr) {
      const Vec<T, V> v = load<T, V>(p + r * a.C);
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = act<ACT>(fmaf(widen(v.e[j]) - mean[j], scale[j], bias[j]));
      store<T, V>(o + r * a.C, y);
    }
  }
}

template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_grad_sums_kernel(Args a) {
  extern __shared__ float2 lds[];            // [C] sums of gz and gz n of a channel, then the row threads'
  float2* chan = lds;
  float2* red = lds + a.C;
  const int chunk = blockIdx.x, b = blockIdx.y;
  const int64_t r0 = chunk * a.rpc, r1 = min(a.P, r0 + a.rpc);
  const int tc = threadIdx.x % a.tc, tr = threadIdx.x / a.tc, VR = a.C / V;
  const int64_t base = static_cast<int64_t>(b) * a.P * a.C;
  float2* cpart = reinterpret_cast<float2*>(a.cpart) + (static_cast<int64_t>(b) * a.chunks + chunk) * a.C;
  for (int c0 = 0; c0 < VR; c0 += a.tc) {
    const int width = min(a.tc, VR - c0) * V;
    if (tr < a.tr && tc * V < width) {
      float mean[V], rstd[V], w[V], bias[V], s1[V], s2[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (c0 + tc) * V + j, g = c / a.Cg;
        mean[j] = a.mean[static_cast<int64_t>(b) * a.G + g];
        rstd[j] = a.rstd[static_cast<int64_t>(b) * a.G + g];
        w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c]);
        bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
        s1[j] = s2[j] = 0.f;
      }
      const T* p = static_cast<const T*>(a.x) + base + (c0 + tc) * V;
      const T* q = static_cast<const T*>(a.g) + base + (c0 + tc) * V;
#pragma unroll 2
      for (int64_t r = r0 + tr; r < r1; r += a.tr) {
        const Vec<T, V> v = load<T, V>(p + r * a.C), gr = load<T, V>(q + r * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float n = (widen(v.e[j]) - mean[j]) * rstd[j];
          const float gz = widen(gr.e[j]) * slope<ACT>(fmaf(n, w[j], bias[j]));
          s1[j] += gz;
          s2[j] = fmaf(gz, n, s2[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) red[tr * width + tc * V + j] = make_float2(s1[j], s2[j]);
    }
    __syncthreads();
    join_rows(red, a.tr, width, [&](int c, float2 s) {
      const float w = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c0 * V + c]);
      cpart[c0 * V + c] = s;
      chan[c0 * V + c] = make_float2(s.x * w, s.y * w);
    });
    __syncthreads();
  }
  const int L = lanes_of(a.G), lane = threadIdx.x % L;
  for (int g = threadIdx.x / L; g < a.G; g += kNT / L) {
    const float2* c = chan + g * a.Cg;
    float s1 = 0.f, s2 = 0.f;
    for (int i = lane; i < a.Cg; i += L) {
      s1 += c[i].x;
      s2 += c[i].y;
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0)
      reinterpret_cast<float2*>(a.gpart)[(static_cast<int64_t>(b) * a.chunks + chunk) * a.G + g] = make_float2(s1, s2);
  }
}

// Batch elements 0 .. B-1 write grad_x; the workgroups of row B of the grid add the chunks of
// 32 channels each for grad_weight and grad_bias.
template <typename T, int V, int ACT>
__global__ __launch_bounds__(kNT) void norm_grad_write_kernel(Args a) {
  extern __shared__ float2 lds[];
  const int b = blockIdx.y;
  if (b == a.B) {
    const int c = blockIdx.x * 32 + threadIdx.x % 32, part = threadIdx.x / 32;
    constexpr int PARTS = kNT / 32;
    const int64_t n = static_cast<int64_t>(a.B) * a.chunks;
    float2 s = make_float2(0.f, 0.f);
    if (c < a.C)
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
  if (static_cast<int>(blockIdx.x) >= a.ablocks) return;
  const int L = lanes_of(a.G), lane = threadIdx.x % L;
  const float2* part = reinterpret_cast<const float2*>(a.gpart) + static_cast<int64_t>(b) * a.chunks * a.G;
  const float inv = 1.f / (static_cast<float>(a.P) * a.Cg);
  for (int g = threadIdx.x / L; g < a.G; g += kNT / L) {
    float s1 = 0.f, s2 = 0.f;
    for (int k = lane; k < a.chunks; k += L) {
      const float2 v = part[static_cast<int64_t>(k) * a.G + g];
      s1 += v.x;
      s2 += v.y;
    }
    s1 = lanes_sum(s1, L);
    s2 = lanes_sum(s2, L);
    if (lane == 0) lds[g] = make_float2(s1 * inv, s2 * inv);
  }
  __syncthreads();
  const int64_t r0 = blockIdx.x * a.rpa, r1 = min(a.P, r0 + a.rpa);
  const int tc = threadIdx.x % a.tc, tr = threadIdx.x / a.tc, VR = a.C / V;
  if (tr >= a.tr) return;
  const int64_t base = static_cast<int64_t>(b) * a.P * a.C;
  for (int c0 = tc; c0 < VR; c0 += a.tc) {
    float mean[V], rstd[V], w[V], bias[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = c0 * V + j, g = c / a.Cg;
      mean[j] = a.mean[static_cast<int64_t>(b) * a.G + g];
      rstd[j] = a.rstd[static_cast<int64_t>(b) * a.G + g];
      w[j] = a.w == nullptr ? 1.f : widen(static_cast<const T*>(a.w)[c]);
      bias[j] = a.b == nullptr ? 0.f : widen(static_cast<const T*>(a.b)[c]);
      m1[j] = lds[g].x;
      m2[j] = lds[g].y;
    }
    const T* p = static_cast<const T*>(a.x) + base + c0 * V;
    const T* q = static_cast<const T*>(a.g) + base + c0 * V;
    T* o = static_cast<T*>(a.out) + base + c0 * V;
#pragma unroll 2
    for (int64_t r = r0 + tr; r < r1; r += a.tr) {
      const Vec<T, V> v = load<T, V>(p + r * a.C), gr = load<T, V>(q + r * a.C);
      float y[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = (widen(v.e[j]) - mean[j]) * rstd[j];
        const float gz = widen(gr.e[j]) * slope<ACT>(fmaf(n, w[j], bias[j]));
        y[j] = rstd[j] * (fmaf(gz, w[j], -m1[j]) - n * m2[j]);
      }
      store<T, V>(o + r * a.C, y);
    }
  }
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

// Chunks of the summing pass: about two workgroups for each CU in all, of at least four sweeps
// of the threads; and at most 128 for one batch element, since every workgroup of the writing
// pass joins them.
void plan(const dcn_norm_desc* d, int V, Args* a) {
  a->B = static_cast<int>(d->batch);
  a->P = d->positions;
  a->C = static_cast<int>(d->channels);
  a->G = static_cast<int>(d->groups);
  a->Cg = a->C / a->G;
  a->eps = d->eps;
  const int VR = a->C / V;
  a->tc = std::min(VR, kNT);
  a->tr = kNT / a->tc;
  const int64_t per = std::max<int64_t>(1, 512 / std::max(a->B, 1));
  const int64_t most = std::max<int64_t>(1, d->positions / (4 * a->tr));
  int64_t n = std::min<int64_t>(std::min<int64_t>(per, 128), most);
  a->rpc = (d->positions + n - 1) / n;
  a->chunks = static_cast<int>((d->positions + a->rpc - 1) / a->rpc);
  n = std::min<int64_t>(std::max<int64_t>(1, 1024 / std::max(a->B, 1)), most);
  a->rpa = (d->positions + n - 1) / n;
  a->ablocks = static_cast<int>((d->positions + a->rpa - 1) / a->rpa);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// one upper bound for both vector widths (16-byte rows or single elements, known at the call)
size_t group_bytes(const dcn_norm_desc* d) {
  return up256(static_cast<size_t>(d->batch) * 128 * d->groups * 8);
}
size_t chan_bytes(const dcn_norm_desc* d) {
  return up256(static_cast<size_t>(d->batch) * 128 * d->channels * 8);
}

size_t sums_lds(const Args& a, int V) {
  return (static_cast<size_t>(a.C) + static_cast<size_t>(a.tr) * a.tc * V) * sizeof(float2);
}

bool launch(const void* fn, dim3 grid, size_t lds, Args* a, hipStream_t stream) {
  void* args[] = {a};
  return hipLaunchKernel(fn, grid, dim3(kNT), args, lds, stream) == hipSuccess;
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
int forward(const dcn_norm_desc* d, Args* a, hipStream_t stream) {
  plan(d, V, a);
  if (!launch(reinterpret_cast<const void*>(&norm_stats_kernel<T, V>), dim3(a->chunks, a->B), sums_lds(*a, V), a,
              stream))
    return DCN_E_HIP;
  return launch(write_kernel<T, V>(d->activation), dim3(a->ablocks, a->B), a->G * sizeof(float2), a, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

template <typename T, int V>
int backward(const dcn_norm_desc* d, Args* a, hipStream_t stream) {
  plan(d, V, a);
  if (a->B > 0 &&
      !launch(sums_kernel<T, V>(d->activation), dim3(a->chunks, a->B), sums_lds(*a, V), a, stream))
    return DCN_E_HIP;
  const bool params = a->gw != nullptr || a->gb != nullptr;
  if (a->out == nullptr) a->ablocks = 0;
  const int gx = std::max(a->ablocks, params ? (a->C + 31) / 32 : 0);
  if (gx == 0) return DCN_OK;
  return launch(grad_write_kernel<T, V>(d->activation), dim3(gx, a->B + (params ? 1 : 0)),
                static_cast<size_t>(std::max(a->G, kNT)) * sizeof(float2), a, stream)
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
  if (rc == DCN_OK) *bytes = dcn::norm::group_bytes(d);
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
  rc = workspace_status(workspace, workspace_bytes, group_bytes(d));
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
  if (rc == DCN_OK) *bytes = dcn::norm::group_bytes(d) + dcn::norm::chan_bytes(d);
  return rc;
}

extern "C" int dcn_group_norm_backward(const dcn_norm_desc* d, const void* x, const void* weight, const void* bias,
                                       const float* mean, const float* rstd, const void* grad_out, void* grad_x,
                                       void* grad_weight, void* grad_bias, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
  using namespace dcn::norm;
  int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch > 0 && (x == nullptr || mean == nullptr || rstd == nullptr || grad_out == nullptr)) return DCN_E_ARG;
  rc = workspace_status(workspace, workspace_bytes, group_bytes(d) + chan_bytes(d));
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
  a.cpart = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + group_bytes(d));
  const bool bf16 = d->dtype == DCN_BF16;
  const bool vec = aligned(x) && aligned(grad_out) && aligned(grad_x) && d->channels % (bf16 ? 8 : 4) == 0;
  if (bf16) return vec ? backward<uint16_t, 8>(d, &a, stream) : backward<uint16_t, 1>(d, &a, stream);
  return vec ? backward<float, 4>(d, &a, stream) : backward<float, 1>(d, &a, stream);
}

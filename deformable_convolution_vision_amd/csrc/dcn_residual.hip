// dcn_residual.hip -- gfx950 join of two blocks: the norm after a block, its gate and residual scale, the
// residual sum and the norm before the next block, and the gradients.
//
// For a row of C channels, with v = (y - m1) r1 the branch's row normed (v = y without a norm),
//
//   z = v w1 + b1,  o = x + gate scale z,  u = (o - m2) r2,  next = u w2 + b2,
//
// and for upstream gradients go and gn
//
//   gu = gn w2,  d = go + r2 (gu - mean(gu) - u mean(gu u))      (rms: without mean(gu)),
//   grad_x = d,  h = d gate scale,  gv = h w1,  grad_y = r1 (gv - mean(gv) - v mean(gv v)),
//   grad_w2 = sum gn u, grad_b2 = sum gn, grad_w1 = sum h v, grad_b1 = sum h,
//   grad_scale = sum d gate z, grad_gate = d scale z (summed over the positions where they share it).
//
// A row stays in the registers of the threads that take it (8 channels each), so everything is read
// once; a row of up to 512 channels is part of a wave, wider ones are a workgroup's.  In the gradients
// a workgroup takes a run of rows and adds its channels' sums in registers; the runs' parts are
// added by a second launch, in order.  Where a gate is shared by a batch element's positions a run
// ends with the batch element, and its sums are of d z, d v and d alone: the gate comes in when the
// parts are added.
//
// Arithmetic: fp32, every output rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"

namespace dcn {
namespace residual {
namespace {

constexpr int kE = 8;            // channels of a thread
constexpr int kMaxC = 8192;
constexpr int kSums = 5;         // of the gradients, for each channel: gn u, gn, d z, d v, d

struct Args {
  const void *x, *y, *gate, *scale, *w1, *b1, *w2, *b2;
  const void *go, *gn;
  void *out, *next;              // forward; backward: grad_x, grad_y
  void *ggate, *gscale, *gw1, *gb1, *gw2, *gb2;
  float* stats;                  // [rows][4]
  float* part;                   // [runs][kSums][C]
  int64_t rows;                  // B * P
  int64_t per_run;               // rows of a run
  int runs;                      // of a batch element where a gate is shared by its positions, else of all rows
  int P, C, B;
  int n1, n2, gkind;
  int sums, sum_of[kSums];       // sums over the rows that are wanted
  float eps, inv;                // 1 / C
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

// V adjacent elements in one access
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// A thread's 8 channels of a row, as read: kE / V vectors, TR vectors apart.
template <typename T, int V>
struct Raw {
  Vec<T, V> v[kE / V];
};
// Its place in rows of C channels: vector i starts at channel (i * tr + t) * V, where that is below C.
struct Lane {
  int t, tr, C;
  template <int V>
  __device__ __forceinline__ int at(int i) const { return (i * tr + t) * V; }
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const void* p, int64_t row, const Lane& l) {
  Raw<T, V> r;
  const T* base = static_cast<const T*>(p) + row * l.C;
#pragma unroll
  for (int i = 0; i < kE / V; ++i) {
    const int c = l.at<V>(i);
    if (c < l.C) {
      r.v[i] = *reinterpret_cast<const Vec<T, V>*>(base + c);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) r.v[i].e[j] = T(0);
    }
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void floats(const Raw<T, V>& r, float (&f)[kE]) {
#pragma unroll
  for (int i = 0; i < kE; ++i) f[i] = widen(r.v[i / V].e[i % V]);
}
template <typename T, int V>
__device__ __forceinline__ void store(void* p, int64_t row, const Lane& l, const float (&f)[kE]) {
  T* base = static_cast<T*>(p) + row * l.C;
#pragma unroll
  for (int i = 0; i < kE / V; ++i) {
    const int c = l.at<V>(i);
    Vec<T, V> v;
#pragma unroll
    for (int j = 0; j < V; ++j) v.e[j] = narrow<T>(f[i * V + j]);
    if (c < l.C) *reinterpret_cast<Vec<T, V>*>(base + c) = v;
  }
}
// A parameter's 8 channels, or `none` where there is none.
template <typename T, int V>
__device__ __forceinline__ void param(const void* p, int64_t row, const Lane& l, float none, float (&f)[kE]) {
  if (p != nullptr) {
    floats<T, V>(load<T, V>(p, row, l), f);
  } else {
#pragma unroll
    for (int i = 0; i < kE; ++i) f[i] = none;
  }
}

// Sums of N values over the threads of a row, in every one of them: TR lanes of a wave, or (TR 0) the waves of
// the workgroup, which leave their sums in the LDS.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dpp<0xb1>(v);                        // quads: lanes 1 0 3 2
  v += dpp<0x4e>(v);                        // 2 3 0 1
  v += dpp<0x141>(v);                       // 8 lanes mirrored
  if (LANES >= 16) v += dpp<0x140>(v);      // 16 lanes mirrored
  if (LANES >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (LANES >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}
// red: two places of 16 waves for N values, used in turn (a wave may be at the next sum while another
// still reads this one; the barrier of the next keeps it from the one after).
template <int TR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lanes_sum<TR == 0 ? 64 : TR>(v[n]);
  if constexpr (TR == 0) {
    float* r = red + (turn & 1) * 32;
    ++turn;
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) r[n * 16 + (threadIdx.x >> 6)] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0.f;
      for (int w = 0; w < waves; ++w) s += r[n * 16 + w];
      v[n] = s;
    }
  }
}

// The norm of a row's channels, in place: mean and 1 / deviation, from the squares about the mean.
template <int V, int TR>
__device__ __forceinline__ void normalise(float (&f)[kE], int kind, const Args& a, const Lane& l, float* red, int& turn,
                                          float& mean, float& rstd) {
  mean = 0.f;
  rstd = 1.f;
  if (kind == DCN_NORM_NONE) return;
  if (kind == DCN_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kE; ++i) s[0] += f[i];     // (channels beyond C are 0)
    row_sums<TR>(s, red, turn);
    mean = s[0] * a.inv;
#pragma unroll
    for (int i = 0; i < kE; ++i) f[i] = l.at<V>(i / V) < l.C ? f[i] - mean : 0.f;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kE; ++i) q[0] = fmaf(f[i], f[i], q[0]);
  row_sums<TR>(q, red, turn);
  rstd = 1.f / sqrtf(fmaf(q[0], a.inv, a.eps));
#pragma unroll
  for (int i = 0; i < kE; ++i) f[i] *= rstd;
}

// TR: threads of a row (8 to 64 lanes of a wave; 0: the whole workgroup).
template <typename T, int V, int TR>
__global__ __launch_bounds__(TR == 0 ? 1024 : 256) void residual_norm_kernel(Args a) {
  __shared__ float red[TR == 0 ? 64 : 1];
  const Lane l = {TR == 0 ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % (TR == 0 ? 1 : TR),
                  TR == 0 ? static_cast<int>(blockDim.x) : TR, a.C};
  const int step = TR == 0 ? 1 : 256 / (TR == 0 ? 1 : TR), mine = TR == 0 ? 0 : threadIdx.x / (TR == 0 ? 1 : TR);
  int turn = 0;
  const int64_t r1 = min(a.rows, (static_cast<int64_t>(blockIdx.x) + 1) * a.per_run);
  float w1[kE], b1[kE], w2[kE], b2[kE], sc[kE];
  param<T, V>(a.w1, 0, l, 1.f, w1);
  param<T, V>(a.b1, 0, l, 0.f, b1);
  param<T, V>(a.w2, 0, l, 1.f, w2);
  param<T, V>(a.b2, 0, l, 0.f, b2);
  param<T, V>(a.scale, 0, l, 1.f, sc);
  Raw<T, V> x, y, gt;
  const auto fetch = [&](int64_t row) {
    y = load<T, V>(a.y, row, l);
    x = load<T, V>(a.x, row, l);
    if (a.gkind != DCN_GATE_NONE) gt = load<T, V>(a.gate, a.gkind == DCN_GATE_FULL ? row : row / a.P, l);
  };
  const int64_t r0 = blockIdx.x * a.per_run + mine;
  if (r0 < r1) fetch(r0);
  for (int64_t row = r0; row < r1; row += step) {
    float f[kE], o[kE], g[kE];
    floats<T, V>(y, f);
    floats<T, V>(x, o);
    floats<T, V>(gt, g);
    if (row + step < r1) fetch(row + step);     // the next row's loads are under way over this one's sums
    float m1, r1s, m2, r2s;
    normalise<V, TR>(f, a.n1, a, l, red, turn, m1, r1s);
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float z = fmaf(f[i], w1[i], b1[i]);
      o[i] = fmaf(a.gkind != DCN_GATE_NONE ? g[i] * sc[i] : sc[i], z, o[i]);
      if (l.at<V>(i / V) >= l.C) o[i] = 0.f;
    }
    store<T, V>(a.out, row, l, o);
    normalise<V, TR>(o, a.n2, a, l, red, turn, m2, r2s);
    if (a.n2 != DCN_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < kE; ++i) o[i] = fmaf(o[i], w2[i], b2[i]);
      store<T, V>(a.next, row, l, o);
    }
    if (a.stats != nullptr && l.t == 0) *reinterpret_cast<float4*>(a.stats + row * 4) = make_float4(m1, r1s, m2, r2s);
  }
}

// (NT: the most threads of a workgroup.  Rows of up to 4096 channels are taken by 512, whose registers hold
// everything; with 1024 some of it goes to memory.)
template <typename T, int V, int TR, int NT>
__global__ __launch_bounds__(NT) void residual_grad_kernel(Args a) {
  constexpr int STEP = TR == 0 ? 1 : 256 / (TR == 0 ? 1 : TR);
  __shared__ float red[TR == 0 ? 64 : 256 * kE];
  const Lane l = {TR == 0 ? static_cast<int>(threadIdx.x) : static_cast<int>(threadIdx.x) % (TR == 0 ? 1 : TR),
                  TR == 0 ? static_cast<int>(blockDim.x) : TR, a.C};
  const int mine = TR == 0 ? 0 : threadIdx.x / (TR == 0 ? 1 : TR);
  const bool shared_gate = a.gkind == DCN_GATE_BATCH;
  int turn = 0;
  // the rows of this run: of a batch element where its positions share a gate
  const int b = shared_gate ? blockIdx.x / a.runs : 0;
  const int64_t first = shared_gate ? static_cast<int64_t>(b) * a.P : 0, end = shared_gate ? first + a.P : a.rows;
  const int64_t r0 = first + (blockIdx.x - static_cast<int64_t>(b) * a.runs) * a.per_run, r1 = min(end, r0 + a.per_run);
  float w1[kE], b1[kE], w2[kE], sc[kE], sum[kSums][kE], g[kE];
  param<T, V>(a.w1, 0, l, 1.f, w1);
  param<T, V>(a.b1, 0, l, 0.f, b1);
  param<T, V>(a.w2, 0, l, 1.f, w2);
  param<T, V>(a.scale, 0, l, 1.f, sc);
  param<T, V>(shared_gate ? a.gate : nullptr, b, l, 1.f, g);
#pragma unroll
  for (int n = 0; n < kSums; ++n)
#pragma unroll
    for (int i = 0; i < kE; ++i) sum[n][i] = 0.f;
  Raw<T, V> ry, rx, rgo, rgn, rg;
  float4 rst = make_float4(0.f, 1.f, 0.f, 1.f);
  const auto fetch = [&](int64_t row) {
    ry = load<T, V>(a.y, row, l);
    if (a.n2 != DCN_NORM_NONE) {
      rx = load<T, V>(a.x, row, l);
      rgn = a.gn != nullptr ? load<T, V>(a.gn, row, l) : Raw<T, V>{};
    }
    rgo = a.go != nullptr ? load<T, V>(a.go, row, l) : Raw<T, V>{};
    if (a.gkind == DCN_GATE_FULL) rg = load<T, V>(a.gate, row, l);
    rst = *reinterpret_cast<const float4*>(a.stats + row * 4);
  };
  if (r0 + mine < r1) fetch(r0 + mine);
  for (int64_t row = r0 + mine; row < r1; row += STEP) {
    const float4 st = rst;
    float v[kE], u[kE], d[kE], z[kE], gn[kE];
    floats<T, V>(ry, v);
    floats<T, V>(rx, u);
    floats<T, V>(rgn, gn);
    floats<T, V>(rgo, d);
    if (a.gkind == DCN_GATE_FULL) floats<T, V>(rg, g);
    if (row + STEP < r1) fetch(row + STEP);     // the next row's loads are under way over this one's sums
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      v[i] = l.at<V>(i / V) < l.C ? (v[i] - st.x) * st.y : 0.f;
      z[i] = fmaf(v[i], w1[i], b1[i]);
    }
    if (a.n2 != DCN_NORM_NONE) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        u[i] = l.at<V>(i / V) < l.C ? (fmaf(g[i] * sc[i], z[i], u[i]) - st.z) * st.w : 0.f;
        sum[0][i] = fmaf(gn[i], u[i], sum[0][i]);
        sum[1][i] += gn[i];
        gn[i] *= w2[i];
        s[0] += gn[i];
        s[1] = fmaf(gn[i], u[i], s[1]);
      }
      row_sums<TR>(s, red, turn);
      const float mg = a.n2 == DCN_NORM_LAYER ? s[0] * a.inv : 0.f, mu = s[1] * a.inv;
#pragma unroll
      for (int i = 0; i < kE; ++i) d[i] = fmaf(st.w, gn[i] - mg - u[i] * mu, d[i]);
    }
    if (a.out != nullptr) store<T, V>(a.out, row, l, d);
    if (a.gkind == DCN_GATE_FULL && a.ggate != nullptr) {
      float gg[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) gg[i] = d[i] * z[i] * sc[i];
      store<T, V>(a.ggate, row, l, gg);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if (l.at<V>(i / V) >= l.C) d[i] = 0.f;
      const float e = a.gkind == DCN_GATE_FULL ? d[i] * g[i] : d[i];
      sum[2][i] = fmaf(e, z[i], sum[2][i]);
      sum[3][i] = fmaf(e, v[i], sum[3][i]);
      sum[4][i] += e;
      d[i] *= g[i] * sc[i] * w1[i];       // gv
      s[0] += d[i];
      s[1] = fmaf(d[i], v[i], s[1]);
    }
    if (a.next != nullptr) {
      if (a.n1 != DCN_NORM_NONE) {
        row_sums<TR>(s, red, turn);
        const float mg = a.n1 == DCN_NORM_LAYER ? s[0] * a.inv : 0.f, mv = s[1] * a.inv;
#pragma unroll
        for (int i = 0; i < kE; ++i) d[i] = st.y * (d[i] - mg - v[i] * mv);
      }
      store<T, V>(a.next, row, l, d);
    }
  }
  if (a.part == nullptr) return;
  // this run's sums: the workgroup's rows of threads are added in order
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * kSums * a.C;
  if constexpr (TR == 0) {
#pragma unroll
    for (int n = 0; n < kSums; ++n)
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const int c = l.at<V>(i / V) + i % V;
        if (c < a.C) part[n * a.C + c] = sum[n][i];
      }
  } else {
    for (int n = 0; n < kSums; ++n) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kE; ++i) red[mine * TR * kE + l.at<V>(i / V) + i % V] = sum[n][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += 256) {
        float s = 0.f;
#pragma unroll 4
        for (int r = 0; r < STEP; ++r) s += red[r * TR * kE + c];
        part[n * a.C + c] = s;
      }
    }
  }
}

// Adds the runs' parts of one sum (blockIdx.y: of those that are wanted, then a shared gate's batch
// elements): 16 channels of a workgroup, 64 threads for each, so that a thread's loads are all under way at once.
template <typename T>
__global__ __launch_bounds__(1024) void residual_params_kernel(Args a) {
  __shared__ float red[64][17];
  const int lane = threadIdx.x % 16, k = threadIdx.x / 16, c = blockIdx.x * 16 + lane;
  const bool shared_gate = a.gkind == DCN_GATE_BATCH, in = c < a.C;
  const int b = static_cast<int>(blockIdx.y) - a.sums;                  // >= 0: the gate's gradient of a batch element
  const int n = b >= 0 ? 2 : a.sum_of[blockIdx.y];
  const int r0 = b >= 0 ? b * a.runs : 0, r1 = b >= 0 ? r0 + a.runs : a.runs * (shared_gate ? a.B : 1);
  const T* gate = b < 0 && n >= 2 && shared_gate ? static_cast<const T*>(a.gate) : nullptr;
  float s = 0.f;
  if (in) {
    const float* part = a.part + static_cast<int64_t>(n) * a.C + c;
#pragma unroll 8
    for (int r = r0 + k; r < r1; r += 64) {
      const float p = part[static_cast<int64_t>(r) * kSums * a.C];
      s = gate == nullptr ? s + p : fmaf(widen(gate[static_cast<int64_t>(r / a.runs) * a.C + c]), p, s);
    }
  }
  red[k][lane] = s;
  __syncthreads();
  if (k >= 4) return;
  s = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) s += red[4 * j + k][lane];
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if (k != 0 || !in) return;
  if ((b >= 0 || n >= 3) && a.scale != nullptr) s *= widen(static_cast<const T*>(a.scale)[c]);
  void* to = b >= 0 ? a.ggate : n == 0 ? a.gw2 : n == 1 ? a.gb2 : n == 2 ? a.gscale : n == 3 ? a.gw1 : a.gb1;
  static_cast<T*>(to)[b >= 0 ? static_cast<int64_t>(b) * a.C + c : c] = narrow<T>(s);
}

// ---- host side

int check(const dcn_residual_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  if (d->batch < 0 || d->positions < 0 || d->channels < 1 || !std::isfinite(d->eps) || d->eps < 0.f ||
      d->branch_norm < 0 || d->branch_norm > DCN_NORM_LAYER || d->next_norm < 0 || d->next_norm > DCN_NORM_LAYER ||
      d->gate < 0 || d->gate > DCN_GATE_FULL)
    return DCN_E_ARG;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  const double big = 2147483647.;
  if (d->channels > kMaxC || d->batch > big || d->positions > big ||
      static_cast<double>(d->batch) * d->positions > big || (d->gate == DCN_GATE_BATCH && d->batch > 65530))
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

// Threads of a row (0: whole workgroups of `threads`).
struct Shape {
  int tr, threads, step;   // step: rows at a time
};
Shape shape_of(int64_t C) {
  const int lanes = static_cast<int>((C + kE - 1) / kE);
  if (lanes > 64) return {0, (lanes + 63) / 64 * 64, 1};
  const int tr = lanes <= 8 ? 8 : lanes <= 16 ? 16 : lanes <= 32 ? 32 : 64;
  return {tr, 256, 256 / tr};
}

constexpr int64_t kRuns = 512, kForwardRuns = 1024;   // workgroups at most: 2 and 4 a CU
// Runs of the gradients: two workgroups for each CU at most, and whole steps of rows.
void runs_of(const dcn_residual_desc* d, const Shape& s, int* runs, int64_t* per_run) {
  const bool shared_gate = d->gate == DCN_GATE_BATCH;
  const int64_t rows = shared_gate ? d->positions : d->batch * d->positions;
  int64_t n = shared_gate ? std::max<int64_t>(1, kRuns / std::max<int64_t>(1, d->batch)) : kRuns;
  *per_run = std::max<int64_t>(1, (rows + n - 1) / n);
  *per_run = (*per_run + s.step - 1) / s.step * s.step;
  *runs = static_cast<int>((rows + *per_run - 1) / *per_run);
}

void fill(const dcn_residual_desc* d, Args* a) {
  a->rows = d->batch * d->positions;
  a->P = static_cast<int>(d->positions);
  a->C = static_cast<int>(d->channels);
  a->B = static_cast<int>(d->batch);
  a->n1 = d->branch_norm;
  a->n2 = d->next_norm;
  a->gkind = d->gate;
  a->eps = d->eps;
  a->inv = 1.f / static_cast<float>(d->channels);
}

template <typename T, int V>
const void* fwd_kernel(int tr) {
  switch (tr) {
    case 8: return reinterpret_cast<const void*>(&residual_norm_kernel<T, V, 8>);
    case 16: return reinterpret_cast<const void*>(&residual_norm_kernel<T, V, 16>);
    case 32: return reinterpret_cast<const void*>(&residual_norm_kernel<T, V, 32>);
    case 64: return reinterpret_cast<const void*>(&residual_norm_kernel<T, V, 64>);
    default: return reinterpret_cast<const void*>(&residual_norm_kernel<T, V, 0>);
  }
}
template <typename T, int V>
const void* bwd_kernel(const Shape& s) {
  switch (s.tr) {
    case 8: return reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 8, 256>);
    case 16: return reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 16, 256>);
    case 32: return reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 32, 256>);
    case 64: return reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 64, 256>);
    default:
      return s.threads <= 512 ? reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 0, 512>)
                              : reinterpret_cast<const void*>(&residual_grad_kernel<T, V, 0, 1024>);
  }
}
const void* kernel_of(bool bf16, int width, const Shape& s, bool backward) {
  if (bf16) {
    if (width == 8) return backward ? bwd_kernel<uint16_t, 8>(s) : fwd_kernel<uint16_t, 8>(s.tr);
    if (width == 2) return backward ? bwd_kernel<uint16_t, 2>(s) : fwd_kernel<uint16_t, 2>(s.tr);
    return backward ? bwd_kernel<uint16_t, 1>(s) : fwd_kernel<uint16_t, 1>(s.tr);
  }
  if (width == 4) return backward ? bwd_kernel<float, 4>(s) : fwd_kernel<float, 4>(s.tr);
  if (width == 2) return backward ? bwd_kernel<float, 2>(s) : fwd_kernel<float, 2>(s.tr);
  return backward ? bwd_kernel<float, 1>(s) : fwd_kernel<float, 1>(s.tr);
}

// The widest vectors that fit the channels and every address.
template <size_t N>
int width_of(const dcn_residual_desc* d, const void* const (&ptrs)[N]) {
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  for (int w : {16 / es, 2}) {
    bool ok = d->channels % w == 0;
    for (const void* p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % (static_cast<unsigned>(w) * es) == 0;
    if (ok) return w;
  }
  return 1;
}

bool launch(const void* fn, dim3 groups, int threads, Args* a, hipStream_t stream) {
  void* args[] = {a};
  return hipLaunchKernel(fn, groups, dim3(threads), args, 0, stream) == hipSuccess;
}

// Notes which sums over the rows are wanted; how many outputs [C] the second launch writes.
int64_t wanted_sums(Args* a) {
  const void* to[kSums] = {a->gw2, a->gb2, a->gscale, a->gw1, a->gb1};
  for (int n = 0; n < kSums; ++n)
    if (to[n] != nullptr) a->sum_of[a->sums++] = n;
  return a->sums + (a->gkind == DCN_GATE_BATCH && a->ggate != nullptr ? a->B : 0);
}

}  // namespace
}  // namespace residual
}  // namespace dcn

extern "C" int dcn_residual_norm(const dcn_residual_desc* d, const void* x, const void* branch, const void* gate,
                                 const void* scale, const void* branch_weight, const void* branch_bias,
                                 const void* next_weight, const void* next_bias, void* out, void* next, float* stats,
                                 hipStream_t stream) {
  using namespace dcn::residual;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->positions == 0) return DCN_OK;
  const bool then = d->next_norm != DCN_NORM_NONE;
  if (x == nullptr || branch == nullptr || out == nullptr || (then && (next == nullptr || next == out)) ||
      (d->gate != DCN_GATE_NONE && gate == nullptr))
    return DCN_E_ARG;
  if (reinterpret_cast<uintptr_t>(stats) % 16 != 0) return DCN_E_ARG;
  Args a{};
  fill(d, &a);
  a.x = x;
  a.y = branch;
  a.gate = d->gate != DCN_GATE_NONE ? gate : nullptr;
  a.scale = scale;
  if (d->branch_norm != DCN_NORM_NONE) {
    a.w1 = branch_weight;
    a.b1 = branch_bias;
  }
  if (then) {
    a.w2 = next_weight;
    a.b2 = next_bias;
    a.next = next;
  }
  a.out = out;
  a.stats = stats;
  const int w = width_of(d, {a.x, a.y, a.gate, a.scale, a.w1, a.b1, a.w2, a.b2, static_cast<const void*>(a.out),
                             static_cast<const void*>(a.next)});
  const Shape s = shape_of(d->channels);
  // runs of several steps share a thread's parameters
  const int64_t steps = (a.rows + s.step - 1) / s.step;
  a.per_run = std::max<int64_t>(1, (steps + kForwardRuns - 1) / kForwardRuns) * s.step;
  return launch(kernel_of(d->dtype == DCN_BF16, w, s, false), dim3((a.rows + a.per_run - 1) / a.per_run), s.threads, &a,
                stream)
             ? DCN_OK
             : DCN_E_HIP;
}

extern "C" int dcn_residual_norm_backward_workspace_bytes(const dcn_residual_desc* d, size_t* bytes) {
  using namespace dcn::residual;
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  *bytes = 0;
  if (d->batch == 0 || d->positions == 0) return DCN_OK;
  int runs;
  int64_t per_run;
  runs_of(d, shape_of(d->channels), &runs, &per_run);
  *bytes = static_cast<size_t>(runs) * (d->gate == DCN_GATE_BATCH ? d->batch : 1) * kSums * d->channels * sizeof(float);
  return DCN_OK;
}

extern "C" int dcn_residual_norm_backward(const dcn_residual_desc* d, const void* x, const void* branch,
                                          const void* gate, const void* scale, const void* branch_weight,
                                          const void* branch_bias, const void* next_weight, const float* stats,
                                          const void* grad_out, const void* grad_next, void* grad_x,
                                          void* grad_branch, void* grad_gate, void* grad_scale,
                                          void* grad_branch_weight, void* grad_branch_bias, void* grad_next_weight,
                                          void* grad_next_bias, void* workspace, size_t workspace_bytes,
                                          hipStream_t stream) {
  using namespace dcn::residual;
  int rc = check(d);
  if (rc != DCN_OK) return rc;
  const bool then = d->next_norm != DCN_NORM_NONE, first = d->branch_norm != DCN_NORM_NONE, any = d->batch > 0 && d->positions > 0;
  if ((any && (x == nullptr || branch == nullptr || stats == nullptr || reinterpret_cast<uintptr_t>(stats) % 16 != 0)) ||
      (d->gate != DCN_GATE_NONE && any && gate == nullptr) || (d->gate == DCN_GATE_NONE && grad_gate != nullptr) ||
      (!first && (grad_branch_weight != nullptr || grad_branch_bias != nullptr)) ||
      (!then && (grad_next_weight != nullptr || grad_next_bias != nullptr)))
    return DCN_E_ARG;
  Args a{};
  fill(d, &a);
  a.x = x;
  a.y = branch;
  a.gate = d->gate != DCN_GATE_NONE ? gate : nullptr;
  a.scale = scale;
  if (first) {
    a.w1 = branch_weight;
    a.b1 = branch_bias;
  }
  if (then) {
    a.w2 = next_weight;
    a.gn = grad_next;
  }
  a.stats = const_cast<float*>(stats);
  a.go = grad_out;
  a.out = grad_x;
  a.next = grad_branch;
  a.ggate = grad_gate;
  a.gscale = grad_scale;
  a.gw1 = grad_branch_weight;
  a.gb1 = grad_branch_bias;
  a.gw2 = grad_next_weight;
  a.gb2 = grad_next_bias;
  const bool bf16 = d->dtype == DCN_BF16;
  const int64_t outputs = wanted_sums(&a);
  const Shape s = shape_of(d->channels);
  if (any) {
    runs_of(d, s, &a.runs, &a.per_run);
    const int64_t groups = static_cast<int64_t>(a.runs) * (d->gate == DCN_GATE_BATCH ? a.B : 1);
    if (outputs > 0) {
      size_t need = 0;
      rc = dcn_residual_norm_backward_workspace_bytes(d, &need);
      if (rc != DCN_OK) return rc;
      if (workspace == nullptr || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return DCN_E_WORKSPACE;
      a.part = static_cast<float*>(workspace);
    }
    const int w = width_of(d, {a.x, a.y, a.gate, a.scale, a.w1, a.b1, a.w2, a.go, a.gn, static_cast<const void*>(a.out),
                               static_cast<const void*>(a.next),
                               d->gate == DCN_GATE_FULL ? static_cast<const void*>(a.ggate) : nullptr});
    if (!launch(kernel_of(bf16, w, s, true), dim3(groups), s.threads, &a, stream)) return DCN_E_HIP;
  }
  if (outputs > 0 &&
      !launch(bf16 ? reinterpret_cast<const void*>(&residual_params_kernel<uint16_t>)
                   : reinterpret_cast<const void*>(&residual_params_kernel<float>),
              dim3((d->channels + 15) / 16, outputs), 1024, &a, stream))
    return DCN_E_HIP;
  return DCN_OK;
}

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
// once; a row of up to 512 channels is part of a wave, wider ones are whole waves, and a workgroup takes several
// rows at a time.  In the gradients a workgroup takes a run of rows and adds its channels' sums in registers; the
// runs' parts are added by a second launch, in order.  Where a gate is shared by a batch element's positions a run
// ends with the batch element, and its sums are of d z, d v and d alone: the gate comes in when the
// parts are added.
//
// Rows of any width are read 16 bytes at a time, wherever they start (the memory takes 16-byte accesses at any
// element): the last vector of a row that is no whole number of them is moved back to end with the row, and the
// elements that it then shares with the one before are taken as zeros in its thread and not written.
//
// Arithmetic: fp32, every output rounded once.
//
// Memory bounds it.  8 x 16800 rows of 256 channels, bf16, two layer norms: 48.3 us for 275 MB, 5.7 TB/s (some of it
// stays in the caches from call to call; 61 us between other work, a copy of as many bytes 55).
// The gradients of 2 x 16800 rows, the gate shared by an image: 22.6 us for 104 MB, 4.6 TB/s, and 4.0 for the second
// launch.  Rows of 1030 channels in fp32, gated element by element, 3 x 517 of them: 20.9 us for 51 MB, four steps of
// two rows in each of 194 workgroups of six waves, which is what their registers (222) leave room for; rows of three
// waves, of which the third has one lane, and 3.03 rounds of the chip in four steps are what they lose.  Without the next
// row under way the first two took 65.3 and 47.2 us.

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
  int waves;                     // of a row, where it has whole ones
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

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes in memory, wherever an element may start
template <typename T>
struct Memory;
template <>
struct Memory<uint16_t> { typedef u32x4 vec __attribute__((aligned(2))); };
template <>
struct Memory<float> { typedef u32x4 vec __attribute__((aligned(4))); };

// A thread's 8 channels of a row, as read.
template <typename T>
struct Raw {
  static constexpr int V = 16 / static_cast<int>(sizeof(T)), K = kE / V;   // elements of a vector, vectors
  u32x4 v[K];
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = v[i / V][i % V * sizeof(T) / 4];
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    return __uint_as_float(i % 2 == 0 ? w << 16 : w & 0xffff0000u);
  }
};

// How rows lie on threads: 8 channels for every thread, some threads with fewer, or fewer than 8 in all.
enum Fit { kExact, kRagged, kTiny };

// A thread's place in rows of C channels, `tr` threads to a row: vector i starts at channel at[i], and elements that
// are another thread's, or none's, are told apart by own (the thread has all 8 where FIT is kExact).
template <typename T, Fit FIT>
struct Lane {
  static constexpr int V = Raw<T>::V, K = Raw<T>::K;
  int t, C;
  int at[K];
  uint32_t own;    // bit i: element i of the thread's 8 is its own
  __device__ __forceinline__ Lane(int thread, int tr, int channels) : t(thread), C(channels) {
    const int n = (C + V - 1) / V;
    own = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int v = i * tr + t;
      at[i] = v * V;
      int dead = 0;
      if (FIT == kRagged) {
        dead = v < n ? max(0, at[i] + V - C) : V;
        at[i] = v < n ? min(at[i], C - V) : 0;       // (a thread without a vector reads the first)
      }
#pragma unroll
      for (int j = 0; j < V; ++j) own |= j >= dead && at[i] + j < C ? 1u << (i * V + j) : 0u;
    }
  }
  __device__ __forceinline__ bool has(int i) const { return FIT == kExact || ((own >> i) & 1u); }
  __device__ __forceinline__ int channel(int i) const { return at[i / V] + i % V; }

  // of the row that starts `o` elements after p
  __device__ __forceinline__ Raw<T> load(const void* p, int64_t o) const {
    Raw<T> r;
    const T* base = static_cast<const T*>(p) + o;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (FIT == kTiny) {
        T e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = has(i * V + j) ? base[at[i] + j] : T(0);
        __builtin_memcpy(&r.v[i], e, 16);
      } else {
        r.v[i] = *reinterpret_cast<const typename Memory<T>::vec*>(base + at[i]);
      }
    }
    return r;
  }
  // what is not the thread's own becomes 0, whatever it was
  __device__ __forceinline__ void clear(float (&f)[kE]) const {
    if (FIT == kExact) return;
#pragma unroll
    for (int i = 0; i < kE; ++i)
      f[i] = __uint_as_float(__float_as_uint(f[i]) & static_cast<uint32_t>(static_cast<int32_t>(own << (31 - i)) >> 31));
  }
  __device__ __forceinline__ void floats(const Raw<T>& r, float (&f)[kE]) const {
#pragma unroll
    for (int i = 0; i < kE; ++i) f[i] = r.at(i);
  }
  // a parameter's 8 channels, or `none` where there is none
  __device__ __forceinline__ void param(const void* p, int64_t o, float none, float (&f)[kE]) const {
    if (p != nullptr) {
      floats(load(p, o), f);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) f[i] = none;
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t o, const float (&f)[kE]) const {
    T* base = static_cast<T*>(p) + o;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const uint32_t mine = (own >> (i * V)) & ((1u << V) - 1u);
      if (FIT == kExact || mine == (1u << V) - 1u) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4) {
            v[j] = __float_as_uint(f[4 * i + j]);
          } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 pair = {f[8 * i + 2 * j], f[8 * i + 2 * j + 1]};
            v[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(pair, bf16x2));   // nearest even
          }
        }
        *reinterpret_cast<typename Memory<T>::vec*>(base + at[i]) = v;
      } else if (mine != 0) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (has(i * V + j)) base[at[i] + j] = narrow<T>(f[i * V + j]);
      }
    }
  }
};

// Sums of N values over the threads of a row, in every one of them: TR lanes of a wave, or (TR 0) several waves,
// which leave their sums in the LDS.
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
// still reads this one; the barrier of the next keeps it from the one after).  With TR 0 every thread of the
// workgroup has to come here.
template <int TR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* red, int& turn, int waves) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = lanes_sum<TR == 0 ? 64 : TR>(v[n]);
  if constexpr (TR == 0) {
    float* r = red + (turn & 1) * 32;
    ++turn;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), first = wave / waves * waves;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) r[n * 16 + wave] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float s = 0.f;
      for (int w = 0; w < waves; ++w) s += r[n * 16 + first + w];
      v[n] = s;
    }
  }
}

// The norm of a row's channels, in place: mean and 1 / deviation, from the squares about the mean.
template <int TR, typename L>
__device__ __forceinline__ void normalise(float (&f)[kE], int kind, const Args& a, const L& l, float* red, int& turn,
                                          float& mean, float& rstd) {
  mean = 0.f;
  rstd = 1.f;
  if (kind == DCN_NORM_NONE) return;
  l.clear(f);
  if (kind == DCN_NORM_LAYER) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < kE; ++i) s[0] += f[i];
    row_sums<TR>(s, red, turn, a.waves);
    mean = s[0] * a.inv;
#pragma unroll
    for (int i = 0; i < kE; ++i) f[i] -= mean;
    l.clear(f);
  }
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kE; ++i) q[0] = fmaf(f[i], f[i], q[0]);
  row_sums<TR>(q, red, turn, a.waves);
  rstd = 1.f / sqrtf(fmaf(q[0], a.inv, a.eps));
#pragma unroll
  for (int i = 0; i < kE; ++i) f[i] *= rstd;
}

// Which of a workgroup's rows a thread is at: TR threads of a wave, or (TR 0) a.waves waves, to a row.
struct Seat {
  int thread, threads, group, groups;
};
template <int TR>
__device__ __forceinline__ Seat seat_of(const Args& a) {
  const int tid = threadIdx.x;
  if constexpr (TR > 0) return {tid % TR, TR, tid / TR, static_cast<int>(blockDim.x) / TR};
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = wave / a.waves;
  return {tid - g * a.waves * 64, a.waves * 64, g, static_cast<int>(blockDim.x >> 6) / a.waves};
}

// In the loops of both kernels a thread is at `row`, whose elements start at `o`.  Rows of part of a wave end where
// they end; where they are whole waves all threads of a workgroup make the same turns (they wait for each other in
// the sums), and `live` tells whether there is a row.
template <int TR>
__device__ __forceinline__ bool more(int64_t row, const Seat& seat, int64_t end) {
  return TR > 0 ? row < end : row - seat.group < end;
}

template <typename T, int TR, Fit FIT>
__global__ __launch_bounds__(TR == 0 ? 1024 : 256) void residual_norm_kernel(Args a) {
  __shared__ float red[TR == 0 ? 64 : 1];
  const Seat seat = seat_of<TR>(a);
  const Lane<T, FIT> l(seat.thread, seat.threads, a.C);
  int turn = 0;
  const int64_t r0 = blockIdx.x * a.per_run, r1 = min(a.rows, r0 + a.per_run);
  float w1[kE], b1[kE], w2[kE], b2[kE], sc[kE];
  l.param(a.w1, 0, 1.f, w1);
  l.param(a.b1, 0, 0.f, b1);
  l.param(a.w2, 0, 1.f, w2);
  l.param(a.b2, 0, 0.f, b2);
  l.param(a.scale, 0, 1.f, sc);
  int64_t row = r0 + seat.group, o = row * a.C;
  const int64_t step = static_cast<int64_t>(seat.groups) * a.C;
  Raw<T> x = {}, y = {}, gt = {};
  const auto fetch = [&](int64_t row, int64_t o) {
    if (row >= r1) return;
    y = l.load(a.y, o);
    x = l.load(a.x, o);
    if (a.gkind == DCN_GATE_FULL) gt = l.load(a.gate, o);
    else if (a.gkind == DCN_GATE_BATCH) gt = l.load(a.gate, row / a.P * a.C);
  };
  fetch(row, o);
  for (; more<TR>(row, seat, r1); row += seat.groups, o += step) {
    const bool live = TR > 0 || row < r1;
    float f[kE], s[kE];
    l.floats(y, f);
    l.floats(x, s);
    const Raw<T> g = gt;
    fetch(row + seat.groups, o + step);     // the next row's loads are under way over this one's sums
    float m1, r1s, m2, r2s;
    normalise<TR>(f, a.n1, a, l, red, turn, m1, r1s);
    if (a.gkind == DCN_GATE_NONE) {
#pragma unroll
      for (int i = 0; i < kE; ++i) s[i] = fmaf(sc[i], fmaf(f[i], w1[i], b1[i]), s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) s[i] = fmaf(g.at(i) * sc[i], fmaf(f[i], w1[i], b1[i]), s[i]);
    }
    if (live) l.store(a.out, o, s);
    normalise<TR>(s, a.n2, a, l, red, turn, m2, r2s);
    if (a.n2 != DCN_NORM_NONE) {
#pragma unroll
      for (int i = 0; i < kE; ++i) s[i] = fmaf(s[i], w2[i], b2[i]);
      if (live) l.store(a.next, o, s);
    }
    if (a.stats != nullptr && l.t == 0 && live)
      *reinterpret_cast<float4*>(a.stats + row * 4) = make_float4(m1, r1s, m2, r2s);
  }
}

// What there is on the branch's side: nothing (its gradient is the stream's, and only the next norm's sums are
// kept), a norm, scale or gate of the channels, or a gate of every element.
enum Side { kBare, kPlain, kGated };

// NT: the most threads of a workgroup.  AHEAD: the next row's loads are under way over this one's sums and the
// parameters stay in registers.  Else (a workgroup of 1024 threads has 128 registers a thread) a row is fetched when
// it is at hand, the parameters with it, and all of the channels' sums but one are kept in the LDS, each thread's where
// it alone reads them (2 x 525 rows of 8192, two layer norms, bf16: in registers, which spilled, 127 us, so 64).
template <typename T, int TR, int NT, Side SIDE, Fit FIT, bool AHEAD>
__global__ __launch_bounds__(NT) void residual_grad_kernel(Args a) {
  constexpr int SUMS = SIDE == kBare ? 2 : kSums;
  __shared__ float red[TR == 0 ? 64 : 1];
  __shared__ float add[NT > 512 ? 1 : NT * kE];
  __shared__ float4 kept[AHEAD ? 1 : (kSums - 1) * 2 * NT];
  const Seat seat = seat_of<TR>(a);
  const Lane<T, FIT> l(seat.thread, seat.threads, a.C);
  const bool shared_gate = SIDE == kPlain && a.gkind == DCN_GATE_BATCH;
  int turn = 0;
  // the rows of this run: of a batch element where its positions share a gate
  const int b = shared_gate ? blockIdx.x / a.runs : 0;
  const int64_t begin = shared_gate ? static_cast<int64_t>(b) * a.P : 0, end = shared_gate ? begin + a.P : a.rows;
  const int64_t r0 = begin + (blockIdx.x - static_cast<int64_t>(b) * a.runs) * a.per_run, r1 = min(end, r0 + a.per_run);
  // fs: gate and scale (kGated: scale); fw: that times the branch's weight.  Only a row's sums need what is not
  // the thread's own to be 0: the channels' sums and the gradients leave it out when they are written.
  float w1[kE], b1[kE], w2[kE], fs[kE], fw[kE], sum[AHEAD ? SUMS : 2][kE];   // (sum[0] of !AHEAD is not used)
  const auto params = [&] {
    if constexpr (SIDE != kBare) {
      l.param(a.w1, 0, 1.f, w1);
      l.param(a.b1, 0, 0.f, b1);
      l.param(a.scale, 0, 1.f, fs);
      if constexpr (SIDE == kPlain) {
        l.param(shared_gate ? a.gate : nullptr, static_cast<int64_t>(b) * a.C, 1.f, fw);
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          fs[i] *= fw[i];
          fw[i] = fs[i] * w1[i];
        }
      }
    }
  };
  const auto then_params = [&] { l.param(a.w2, 0, 1.f, w2); };
  if constexpr (AHEAD) {
    params();
    then_params();
  }
#pragma unroll
  for (int n = 0; n < (AHEAD ? SUMS : 2); ++n)
#pragma unroll
    for (int i = 0; i < kE; ++i) sum[n][i] = 0.f;
  // adds p q to sum n; what is kept of it
  const auto keep = [&](int n, int half) -> float4& { return kept[((n > 1 ? n - 1 : 0) * 2 + half) * NT + threadIdx.x]; };
  const auto accumulate = [&](int n, const float (&p)[kE], const float (&q)[kE]) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < kE; ++i) sum[n][i] = fmaf(p[i], q[i], sum[n][i]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 k = keep(n, h);
        k.x = fmaf(p[4 * h], q[4 * h], k.x);
        k.y = fmaf(p[4 * h + 1], q[4 * h + 1], k.y);
        k.z = fmaf(p[4 * h + 2], q[4 * h + 2], k.z);
        k.w = fmaf(p[4 * h + 3], q[4 * h + 3], k.w);
        keep(n, h) = k;
      }
    }
  };
  if constexpr (!AHEAD) {
#pragma unroll
    for (int n = 0; n < kSums; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (n != 1) keep(n, h) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  int64_t row = r0 + seat.group, o = row * a.C;
  const int64_t step = static_cast<int64_t>(seat.groups) * a.C;
  const bool then = a.n2 != DCN_NORM_NONE;
  // (what is not given stays 0)
  Raw<T> ry = {}, rx = {}, rgo = {}, rgn = {}, rg = {};
  float4 rst = make_float4(0.f, 1.f, 0.f, 1.f);
  const auto fetch = [&](int64_t row, int64_t o) {
    if (row >= r1) return;
    ry = l.load(a.y, o);
    if (then) rx = l.load(a.x, o);
    if (a.gn != nullptr) rgn = l.load(a.gn, o);
    if (a.go != nullptr) rgo = l.load(a.go, o);
    if constexpr (SIDE == kGated) rg = l.load(a.gate, o);
    rst = *reinterpret_cast<const float4*>(a.stats + row * 4);
  };
  if constexpr (AHEAD) fetch(row, o);
  for (; more<TR>(row, seat, r1); row += seat.groups, o += step) {
    const bool live = TR > 0 || row < r1;
    if constexpr (!AHEAD) {
      fetch(row, o);
      params();
    }
    const float4 st = rst;
    float v[kE], u[kE], d[kE], z[kE], gn[kE], g[kE];
    l.floats(ry, v);
    l.floats(rgo, d);
    if (then) {
      l.floats(rx, u);
      l.floats(rgn, gn);
    }
    if constexpr (SIDE == kGated) l.floats(rg, g);
    if constexpr (AHEAD) fetch(row + seat.groups, o + step);
    if constexpr (SIDE != kBare) {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        v[i] = (v[i] - st.x) * st.y;
        z[i] = fmaf(v[i], w1[i], b1[i]);
      }
    }
    if (then) {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        if constexpr (SIDE == kBare) u[i] += v[i];
        else u[i] = fmaf(SIDE == kGated ? g[i] * fs[i] : fs[i], z[i], u[i]);
        u[i] = (u[i] - st.z) * st.w;
      }
      if (live) {
        accumulate(0, gn, u);
#pragma unroll
        for (int i = 0; i < kE; ++i) sum[1][i] += gn[i];
      }
      float s[2] = {0.f, 0.f};
      l.clear(gn);
      if constexpr (!AHEAD) {
        __builtin_amdgcn_sched_barrier(0);   // (not sooner: registers)
        then_params();
      }
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        gn[i] *= w2[i];
        s[0] += gn[i];
        s[1] = fmaf(gn[i], u[i], s[1]);
      }
      row_sums<TR>(s, red, turn, a.waves);
      const float mg = a.n2 == DCN_NORM_LAYER ? s[0] * a.inv : 0.f, mu = s[1] * a.inv;
#pragma unroll
      for (int i = 0; i < kE; ++i) d[i] = fmaf(st.w, fmaf(-u[i], mu, gn[i] - mg), d[i]);
    }
    if (live && a.out != nullptr) l.store(a.out, o, d);
    if constexpr (!AHEAD) {
      __builtin_amdgcn_sched_barrier(0);
      params();
#pragma unroll
      for (int i = 0; i < kE; ++i) z[i] = fmaf(v[i], w1[i], b1[i]);
    }
    if constexpr (SIDE == kBare) {
      if (live && a.next != nullptr) l.store(a.next, o, d);
    } else {
      if (SIDE == kGated && live && a.ggate != nullptr) {
        float gg[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) gg[i] = d[i] * z[i] * fs[i];
        l.store(a.ggate, o, gg);
      }
      if constexpr (SIDE == kGated) {
#pragma unroll
        for (int i = 0; i < kE; ++i) d[i] *= g[i];
      }
      if (live) {
        const float ones[kE] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        accumulate(2, d, z);
        accumulate(3, d, v);
        accumulate(4, d, ones);
      }
      if (a.next != nullptr) {
        float s[2] = {0.f, 0.f};
        l.clear(d);
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          d[i] *= SIDE == kGated ? fs[i] * w1[i] : fw[i];       // gv
          s[0] += d[i];
          s[1] = fmaf(d[i], v[i], s[1]);
        }
        if (a.n1 != DCN_NORM_NONE) {
          row_sums<TR>(s, red, turn, a.waves);
          const float mg = a.n1 == DCN_NORM_LAYER ? s[0] * a.inv : 0.f, mv = s[1] * a.inv;
#pragma unroll
          for (int i = 0; i < kE; ++i) d[i] = st.y * fmaf(-v[i], mv, d[i] - mg);
        }
        if (live) l.store(a.next, o, d);
      }
    }
  }
  if (a.part == nullptr) return;
  // this run's sums: the workgroup's rows of threads are added in order
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * kSums * a.C;
  if (seat.groups == 1) {
#pragma unroll
    for (int n = 0; n < SUMS; ++n) {
      float f[kE];
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        if constexpr (AHEAD) f[i] = sum[n][i];
        else f[i] = n == 1 ? sum[1][i] : reinterpret_cast<const float*>(&keep(n, i / 4))[i % 4];
        if (l.has(i)) part[n * a.C + l.channel(i)] = f[i];
      }
    }
  } else if constexpr (NT <= 512) {
    const int pitch = seat.threads * kE;
#pragma unroll
    for (int n = 0; n < SUMS; ++n) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (l.has(i)) add[seat.group * pitch + l.channel(i)] = sum[n][i];
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
        float s = 0.f;
#pragma unroll 4
        for (int r = 0; r < seat.groups; ++r) s += add[r * pitch + c];
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

constexpr int64_t kForwardWaves = 4096;    // four on each SIMD

// Threads of a row (0: `waves` whole waves of them), of a workgroup, and rows of it at a time.
struct Shape {
  int tr, waves, threads, groups;
  Fit fit;
};
// most: threads of a workgroup of rows that are parts of a wave, or that several such rows fit.
Shape shape_of(int64_t C, int most) {
  const int lanes = static_cast<int>((C + kE - 1) / kE);
  if (lanes > 64) {
    const int waves = (lanes + 63) / 64, groups = std::max(1, most / (64 * waves));
    return {0, waves, waves * 64 * groups, groups, C == waves * 64 * kE ? kExact : kRagged};
  }
  const int tr = lanes <= 8 ? 8 : lanes <= 16 ? 16 : lanes <= 32 ? 32 : 64;
  return {tr, 1, most, most / tr, C == tr * kE ? kExact : C < kE ? kTiny : kRagged};
}
Shape forward_shape(int64_t C) { return shape_of(C, 256); }
Shape backward_shape(int64_t C) { return shape_of(C, 512); }

// Runs of the gradients, each of whole steps of rows: one round of the workgroups that the chip holds at two waves
// a SIMD (registers allow no more; four of those of 1024 threads).
void runs_of(const dcn_residual_desc* d, const Shape& s, int* runs, int64_t* per_run) {
  const bool shared_gate = d->gate == DCN_GATE_BATCH;
  const int64_t rows = shared_gate ? d->positions : d->batch * d->positions;
  const int64_t most = 256 * std::max(1, 8 / (s.threads / 64));
  const int64_t n = shared_gate ? std::max<int64_t>(1, most / std::max<int64_t>(1, d->batch)) : most;
  *per_run = std::max<int64_t>(1, (rows + n - 1) / n);
  *per_run = (*per_run + s.groups - 1) / s.groups * s.groups;
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

template <typename T, Fit FIT>
const void* fwd_kernel(int tr) {
  switch (tr) {
    case 8: return reinterpret_cast<const void*>(&residual_norm_kernel<T, 8, FIT>);
    case 16: return reinterpret_cast<const void*>(&residual_norm_kernel<T, 16, FIT>);
    case 32: return reinterpret_cast<const void*>(&residual_norm_kernel<T, 32, FIT>);
    case 64: return reinterpret_cast<const void*>(&residual_norm_kernel<T, 64, FIT>);
    default: return reinterpret_cast<const void*>(&residual_norm_kernel<T, 0, FIT>);
  }
}
template <typename T>
const void* fwd_kernel(const Shape& s) {
  return s.fit == kTiny    ? reinterpret_cast<const void*>(&residual_norm_kernel<T, 8, kTiny>)
         : s.fit == kExact ? fwd_kernel<T, kExact>(s.tr)
                           : fwd_kernel<T, kRagged>(s.tr);
}
template <typename T, Side SIDE, Fit FIT>
const void* bwd_kernel(const Shape& s) {
  switch (s.tr) {
    case 8: return reinterpret_cast<const void*>(&residual_grad_kernel<T, 8, 512, SIDE, FIT, true>);
    case 16: return reinterpret_cast<const void*>(&residual_grad_kernel<T, 16, 512, SIDE, FIT, true>);
    case 32: return reinterpret_cast<const void*>(&residual_grad_kernel<T, 32, 512, SIDE, FIT, true>);
    case 64: return reinterpret_cast<const void*>(&residual_grad_kernel<T, 64, 512, SIDE, FIT, true>);
    default:
      return s.threads <= 512 ? reinterpret_cast<const void*>(&residual_grad_kernel<T, 0, 512, SIDE, FIT, true>)
                              : reinterpret_cast<const void*>(&residual_grad_kernel<T, 0, 1024, SIDE, FIT, SIDE == kBare>);
  }
}
template <typename T, Side SIDE>
const void* bwd_kernel(const Shape& s) {
  return s.fit == kTiny    ? reinterpret_cast<const void*>(&residual_grad_kernel<T, 8, 512, SIDE, kTiny, true>)
         : s.fit == kExact ? bwd_kernel<T, SIDE, kExact>(s)
                           : bwd_kernel<T, SIDE, kRagged>(s);
}
template <typename T>
const void* bwd_kernel(const Shape& s, Side side) {
  return side == kBare ? bwd_kernel<T, kBare>(s) : side == kPlain ? bwd_kernel<T, kPlain>(s) : bwd_kernel<T, kGated>(s);
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
  const Shape s = forward_shape(d->channels);
  a.waves = s.waves;
  // runs of several steps share a thread's parameters
  const int64_t steps = (a.rows + s.groups - 1) / s.groups, most = std::max<int64_t>(1, kForwardWaves / (s.threads / 64));
  a.per_run = std::max<int64_t>(1, (steps + most - 1) / most) * s.groups;
  return launch(d->dtype == DCN_BF16 ? fwd_kernel<uint16_t>(s) : fwd_kernel<float>(s),
                dim3((a.rows + a.per_run - 1) / a.per_run), s.threads, &a, stream)
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
  runs_of(d, backward_shape(d->channels), &runs, &per_run);
  const size_t need = static_cast<size_t>(runs) * (d->gate == DCN_GATE_BATCH ? d->batch : 1) * kSums * d->channels * sizeof(float);
  *bytes = (need + 255) / 256 * 256;
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
  const Shape s = backward_shape(d->channels);
  a.waves = s.waves;
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
    const Side side = d->gate == DCN_GATE_FULL ? kGated
                      : d->branch_norm != DCN_NORM_NONE || d->gate != DCN_GATE_NONE || scale != nullptr || grad_scale != nullptr
                          ? kPlain
                          : kBare;
    const void* fn = bf16 ? bwd_kernel<uint16_t>(s, side) : bwd_kernel<float>(s, side);
    if (!launch(fn, dim3(groups), s.threads, &a, stream)) return DCN_E_HIP;
  }
  if (outputs > 0 &&
      !launch(bf16 ? reinterpret_cast<const void*>(&residual_params_kernel<uint16_t>)
                   : reinterpret_cast<const void*>(&residual_params_kernel<float>),
              dim3((d->channels + 15) / 16, outputs), 1024, &a, stream))
    return DCN_E_HIP;
  return DCN_OK;
}

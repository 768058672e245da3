// dcn_attention_grad.hip -- gfx950 gradients of cross attention.
//
// With P the softmax weights of the forward (P_rj = exp(s_rj - lse_r), zero where key j is
// padding), and delta_r = sum_d dout_rd out_rd:
//
//   dP = dout V^T,  dS = P o (dP - delta),
//   dV = P^T dout,  dK = scale dS^T Q,  dQ = scale dS K.
//
// delta uses sum_j P_rj dP_rj = dout_r . out_r, so no pass over the keys is needed for it.
// The weights are formed again from the scores and the forward's lse; nothing of size
// Lq x Lk is stored.
//
// Launches: the row pass (delta, and lse in powers of two), then dQ (32 or 128 rows of a
// workgroup, a loop over key tiles, as the forward), then dK and dV (32 or 128 keys of a
// workgroup, a loop over row tiles).  Each sum is formed by one wave, or by waves and
// workgroups whose parts are added in a fixed order: no atomics, the same bits each time.
// The heads that share a key head are rows of one problem, so their gradients add up inside
// the loop of dK and dV.
//
// Both kernels form the scores so that the first products' result registers are an operand
// of the second (see dcn_attention.h): dQ keeps a row per lane (S^T), dK/dV a key per lane
// (S).  Rows with no key have lse = -inf; it enters as +inf, which makes every weight 0.
//
// Arithmetic: fp32 sums; for bf16, P and dS are rounded to bf16 as operands of the second
// products, and the gradients once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"
#include "dcn_attention.h"

namespace dcn {
namespace attn {
namespace {

// One row of 16 lanes: delta and lse in powers of two.
template <typename T>
__global__ __launch_bounds__(256) void attn_rows_kernel(Args a) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.R;
  const int64_t prow = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (prow >= rows) return;
  const int sub = threadIdx.x & 15;
  const int bh = static_cast<int>(prow / a.R), r = static_cast<int>(prow % a.R);
  const int b = bh / a.Hkv, pos = r / a.g, head = (bh % a.Hkv) * a.g + r % a.g;
  const int64_t at = ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D;
  const T* o = static_cast<const T*>(a.out) + at;
  const T* go = static_cast<const T*>(a.dout) + at;
  float s = 0.f;
  for (int d = sub; d < a.D; d += 16) s = fmaf(widen(o[d]), widen(go[d]), s);
#pragma unroll
  for (int w = 8; w > 0; w >>= 1) s += __shfl_xor(s, w, 16);
  if (sub == 0) {
    const float lse = a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.Lq + pos];
    float* out = const_cast<float*>(a.delta) + prow * 2;
    out[0] = lse == kNegInf ? -kNegInf : lse * kLog2e;
    out[1] = s;
  }
}

// Adds the waves' parts of a transposed sum (DP x 32 per wave) through LDS and hands each
// row's 4 elements to store(row of the workgroup, element, values).
template <int DP, int WC, int WS, int DT, typename Store>
__device__ __forceinline__ void join_sum(const f32x16 (&o)[DT], float* os, Store store) {
  constexpr int OST = DP + 4, V4 = DP / 4, NT = 64 * WC * WS;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = tid >> 6;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<float4*>(os + (wave * 32 + (lane & 31)) * OST + 32 * i + acc_row(4 * r4, half)) =
          make_float4(o[i][4 * r4], o[i][4 * r4 + 1], o[i][4 * r4 + 2], o[i][4 * r4 + 3]);
  __syncthreads();
  for (int at = tid; at < WC * 32 * V4; at += NT) {
    const int rr = at / V4, d = (at % V4) * 4, grp = rr / 32, ri = rr % 32;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WS; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(os + ((grp * WS + w) * 32 + ri) * OST + d);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    store(rr, d, acc);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int d, int D, float4 v, float f) {
  const float vals[4] = {v.x * f, v.y * f, v.z * f, v.w * f};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (d + j < D) p[d + j] = narrow<T>(vals[j]);
}

template <typename T, int DP, int WQ, int WK, bool VEC>
__global__ __launch_bounds__(64 * WQ * WK) void attn_dq_kernel(Args a) {
  constexpr int NT = 64 * WQ * WK, KV = Elem<T>::kVec, ST = DP;
  constexpr int SUB = WK == 1 ? 2 : 1, KT = 32 * SUB * WK, VPR = DP / KV, NV = KT * VPR / NT, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* ks = reinterpret_cast<T*>(smem);
  T* vs = ks + KT * ST;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = tid >> 6;
  const int wq = wave / WK, wk = wave % WK;
  const int nbh = a.B * a.Hkv;
  int id = blockIdx.x;
  const int bh = id % nbh;
  id /= nbh;
  const int split = id % a.splits, rt = id / a.splits;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const T* kp = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const T* vp = static_cast<const T*>(a.v) + b * a.vs[0] + hk * a.vs[2];
  const uint8_t* mp = a.mask == nullptr ? nullptr : a.mask + b * a.ms;

  const int row = rt * 32 * WQ + wq * 32 + (lane & 31);
  Frag<T> qf[DP / 16], gf[DP / 16];
  float lse2 = -kNegInf, delta = 0.f;
  {
    const bool live = row < a.R;
    const int pos = live ? row / a.g : 0, head = hk * a.g + (live ? row % a.g : 0);
    const T* qp = static_cast<const T*>(a.q) + b * a.qs[0] + pos * a.qs[1] + head * a.qs[2];
    const T* gp = static_cast<const T*>(a.dout) + ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D;
    load_frags<T, DP, VEC>(qp, 0, a.D, live, qf);
    load_frags<T, DP, VEC>(gp, 0, a.D, live, gf);
    if (live) {
      const int64_t prow = static_cast<int64_t>(bh) * a.R + row;
      lse2 = a.delta[prow * 2];
      delta = a.delta[prow * 2 + 1];
    }
  }
  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc();

  const int tiles = (a.Lk + KT - 1) / KT;
  const int t0 = split * a.per_split, t1 = min(tiles, t0 + a.per_split);
  Vec16<T> kr[NV], vr[NV];
  const auto load_tile = [&](int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, key = t * KT + at / VPR, d = (at % VPR) * KV;
      // rows of padded keys are taken as zeros: their weight is 0, and 0 times a NaN is none
      bool live = key < a.Lk;
      if (mp != nullptr && live) live = mp[key] != 0;
      kr[i] = load_vec<T, VEC>(kp + key * a.ks[1], 0, d, a.D, live);
      vr[i] = load_vec<T, VEC>(vp + key * a.vs[1], 0, d, a.D, live);
    }
  };
  if (t0 < t1) load_tile(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, key = at / VPR, d = (at % VPR) * KV;
      *reinterpret_cast<uint4*>(ks + Tile<T, DP>::at(key, d)) = kr[i].u;
      *reinterpret_cast<uint4*>(vs + Tile<T, DP>::at(key, d)) = vr[i].u;
    }
    __syncthreads();
    if (t + 1 < t1) load_tile(t + 1);
    const int k0 = t * KT + wk * 32 * SUB;
    uint64_t word;
    {
      const int key = k0 + lane;
      bool live = lane < 32 * SUB && key < a.Lk;
      if (mp != nullptr && live) live = mp[key] != 0;
      word = __ballot(live);
    }
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const uint32_t w = static_cast<uint32_t>(word >> (32 * s));
      if (w == 0) continue;
      const int r0 = wk * 32 * SUB + s * 32;
      f32x16 sa = zero_acc(), pa = zero_acc();
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        sa = mma(row_frag<DP>(ks, r0, i), qf[i], sa);
        pa = mma(row_frag<DP>(vs, r0, i), gf[i], pa);
      }
      float ds[16];
      const uint32_t wh = w >> (4 * half);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = exp2_fast(fmaf(sa[r], a.c, -lse2));
        ds[r] = ((wh >> acc_row(r, 0)) & 1u) ? p * (pa[r] - delta) : 0.f;
      }
      typename POperand<T>::type pf;
      to_operand(ds, pf);
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] = mma_rows<DP>(ks, r0, 32 * i, pf, o[i]);
    }
  }
  join_sum<DP, WQ, WK>(o, reinterpret_cast<float*>(smem), [&](int rr, int d, float4 v) {
    const int orow = rt * 32 * WQ + rr;
    if (orow >= a.R) return;
    if (a.splits > 1) {
      const int64_t prow = (static_cast<int64_t>(split) * nbh + bh) * a.R + orow;
      *reinterpret_cast<float4*>(a.part + prow * DP + d) = v;
      return;
    }
    const int pos = orow / a.g, head = hk * a.g + orow % a.g;
    store4<T>(static_cast<T*>(a.dq) + ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D, d, a.D, v,
              a.scale);
  });
}

// WC waves of 32 keys each share the row tiles; with WS > 1 the waves take 32 rows each of a
// tile and the same keys.
template <typename T, int DP, int WC, int WS, bool VEC>
__global__ __launch_bounds__(64 * WC * WS) void attn_dkv_kernel(Args a) {
  constexpr int NT = 64 * WC * WS, KV = Elem<T>::kVec, ST = DP;
  constexpr int SUB = WS == 1 ? 2 : 1, RT = 32 * SUB * WS, VPR = DP / KV, NV = RT * VPR / NT, DT = DP / 32;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* qs = reinterpret_cast<T*>(smem);
  T* gs = qs + RT * ST;
  float* ls = reinterpret_cast<float*>(gs + RT * ST);   // [RT] lse, [RT] delta
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = tid >> 6;
  const int wc = wave / WS, wr = wave % WS;
  const int nbh = a.B * a.Hkv;
  int id = blockIdx.x;
  const int bh = id % nbh;
  id /= nbh;
  const int split = id % a.splits, kt = id / a.splits;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const T* qp = static_cast<const T*>(a.q) + b * a.qs[0];
  const T* gp = static_cast<const T*>(a.dout) + static_cast<int64_t>(b) * a.Lq * a.Hq * a.D;

  const int key = kt * 32 * WC + wc * 32 + (lane & 31);
  bool live = key < a.Lk;
  if (a.mask != nullptr && live) live = a.mask[b * a.ms + key] != 0;
  Frag<T> kf[DP / 16], vf[DP / 16];
  {
    const T* kp = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[2] + (live ? key : 0) * a.ks[1];
    const T* vp = static_cast<const T*>(a.v) + b * a.vs[0] + hk * a.vs[2] + (live ? key : 0) * a.vs[1];
    load_frags<T, DP, VEC>(kp, 0, a.D, live, kf);
    load_frags<T, DP, VEC>(vp, 0, a.D, live, vf);
  }
  f32x16 ok[DT], ov[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    ok[i] = zero_acc();
    ov[i] = zero_acc();
  }
  const bool any = __any(live);
  const int tiles = (a.R + RT - 1) / RT;
  const int t0 = split * a.per_split;
  // keys that are all padding have no gradient and read no rows
  const int t1 = __syncthreads_or(any) ? min(tiles, t0 + a.per_split) : t0;
  Vec16<T> qr[NV], gr[NV];
  float lr = 0.f;
  const auto load_tile = [&](int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, row = t * RT + at / VPR, d = (at % VPR) * KV;
      const bool in = row < a.R;
      const int pos = in ? row / a.g : 0, head = hk * a.g + (in ? row % a.g : 0);
      qr[i] = load_vec<T, VEC>(qp + pos * a.qs[1] + head * a.qs[2], 0, d, a.D, in);
      gr[i] = load_vec<T, VEC>(gp + (static_cast<int64_t>(pos) * a.Hq + head) * a.D, 0, d, a.D, in);
    }
    if (tid < 2 * RT) {
      const int row = t * RT + (tid >> 1);
      lr = row < a.R ? a.delta[(static_cast<int64_t>(bh) * a.R + row) * 2 + (tid & 1)]
                     : ((tid & 1) ? 0.f : -kNegInf);
    }
  };
  static_assert(2 * RT <= NT, "one thread per row value");
  if (t0 < t1) load_tile(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, row = at / VPR, d = (at % VPR) * KV;
      *reinterpret_cast<uint4*>(qs + Tile<T, DP>::at(row, d)) = qr[i].u;
      *reinterpret_cast<uint4*>(gs + Tile<T, DP>::at(row, d)) = gr[i].u;
    }
    if (tid < 2 * RT) ls[(tid & 1) * RT + (tid >> 1)] = lr;
    __syncthreads();
    if (t + 1 < t1) load_tile(t + 1);
    if (!any) continue;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const int r0 = wr * 32 * SUB + s * 32;
      f32x16 sa = zero_acc(), pa = zero_acc();
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        sa = mma(row_frag<DP>(qs, r0, i), kf[i], sa);
        pa = mma(row_frag<DP>(gs, r0, i), vf[i], pa);
      }
      float p[16], ds[16];
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const float4 lse = *reinterpret_cast<const float4*>(ls + r0 + acc_row(4 * r4, half));
        const float4 del = *reinterpret_cast<const float4*>(ls + RT + r0 + acc_row(4 * r4, half));
        const float le[4] = {lse.x, lse.y, lse.z, lse.w}, de[4] = {del.x, del.y, del.z, del.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * r4 + j;
          p[r] = live ? exp2_fast(fmaf(sa[r], a.c, -le[j])) : 0.f;
          ds[r] = p[r] * (pa[r] - de[j]);
        }
      }
      typename POperand<T>::type pf, df;
      to_operand(p, pf);
      to_operand(ds, df);
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        ov[i] = mma_rows<DP>(gs, r0, 32 * i, pf, ov[i]);
        ok[i] = mma_rows<DP>(qs, r0, 32 * i, df, ok[i]);
      }
    }
  }
  const int64_t keys = static_cast<int64_t>(nbh) * a.Lk;
  const auto store = [&](int rr, int d, float4 v, int which) {
    const int okey = kt * 32 * WC + rr;
    if (okey >= a.Lk) return;
    if (a.splits > 1) {
      const int64_t prow = (static_cast<int64_t>(split) * 2 + which) * keys + static_cast<int64_t>(bh) * a.Lk + okey;
      *reinterpret_cast<float4*>(a.part + prow * DP + d) = v;
      return;
    }
    T* out = static_cast<T*>(which ? a.dv : a.dk);
    if (out == nullptr) return;
    store4<T>(out + ((static_cast<int64_t>(b) * a.Lk + okey) * a.Hkv + hk) * a.D, d, a.D, v, which ? 1.f : a.scale);
  };
  join_sum<DP, WC, WS>(ok, reinterpret_cast<float*>(smem), [&](int rr, int d, float4 v) { store(rr, d, v, 0); });
  join_sum<DP, WC, WS>(ov, reinterpret_cast<float*>(smem), [&](int rr, int d, float4 v) { store(rr, d, v, 1); });
}

// Adds up split parts: one thread for 4 elements of a row; rows of dQ, or keys of dK, dV.
template <typename T, int DP, bool KEYS>
__global__ __launch_bounds__(256) void attn_add_kernel(Args a) {
  constexpr int V4 = DP / 4;
  const int nbh = a.B * a.Hkv, len = KEYS ? a.Lk : a.R;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t rows = static_cast<int64_t>(nbh) * len * (KEYS ? 2 : 1), prow = at / V4;
  const int d = static_cast<int>(at % V4) * 4;
  if (prow >= rows) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < a.splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(a.part + (s * rows + prow) * DP + d);
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const int which = KEYS && prow >= rows / 2;
  const int64_t one = prow - (which ? rows / 2 : 0);
  const int bh = static_cast<int>(one / len), r = static_cast<int>(one % len), b = bh / a.Hkv, hk = bh % a.Hkv;
  if (KEYS) {
    T* out = static_cast<T*>(which ? a.dv : a.dk);
    if (out == nullptr) return;
    store4<T>(out + ((static_cast<int64_t>(b) * a.Lk + r) * a.Hkv + hk) * a.D, d, a.D, acc, which ? 1.f : a.scale);
  } else {
    store4<T>(static_cast<T*>(a.dq) + ((static_cast<int64_t>(b) * a.Lq + r / a.g) * a.Hq + hk * a.g + r % a.g) * a.D,
              d, a.D, acc, a.scale);
  }
}

constexpr int kCUs = 256;

struct GradPlan {
  int dp, wide, splits, per_split, tile;
};
// `outer` rows (or keys) held by the waves, `inner` looped over.
GradPlan make_plan(int64_t nbh, int64_t outer, int64_t inner, int64_t D) {
  GradPlan p{};
  p.dp = D <= 32 ? 32 : D <= 64 ? 64 : 128;
  p.wide = outer > 96 && nbh * ((outer + 127) / 128) >= 2 * kCUs;
  p.tile = p.wide ? 64 : 128;
  const int64_t tiles = std::max<int64_t>(1, (inner + p.tile - 1) / p.tile);
  int64_t splits = 1;
  if (!p.wide) {
    const int64_t groups = std::max<int64_t>(1, nbh * ((outer + 31) / 32));
    splits = std::min<int64_t>(std::max<int64_t>(1, 2 * kCUs / groups), std::max<int64_t>(1, tiles / 2));
  }
  p.per_split = static_cast<int>((tiles + splits - 1) / splits);
  p.splits = static_cast<int>((tiles + p.per_split - 1) / p.per_split);
  return p;
}

size_t lds_bytes(const GradPlan& p, int es) {
  const size_t tile = static_cast<size_t>(2) * p.tile * p.dp * es + static_cast<size_t>(p.tile) * 8;
  return std::max(tile, static_cast<size_t>(4) * 32 * (p.dp + 4) * 4);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  GradPlan q, kv;
  size_t part_at, bytes;   // row values first, then the parts of whichever kernel runs
};

Layout make_layout(const dcn_attn_desc* d) {
  Layout y{};
  const int64_t nbh = d->batch * d->key_heads, R = d->query_len * (d->query_heads / d->key_heads);
  y.q = make_plan(nbh, R, d->key_len, d->head_dim);
  y.kv = make_plan(nbh, d->key_len, R, d->head_dim);
  y.part_at = up256(static_cast<size_t>(nbh) * R * 8);
  size_t part = 0;
  if (y.q.splits > 1) part = static_cast<size_t>(y.q.splits) * nbh * R * y.q.dp * 4;
  if (y.kv.splits > 1) part = std::max(part, static_cast<size_t>(y.kv.splits) * 2 * nbh * d->key_len * y.kv.dp * 4);
  y.bytes = y.part_at + up256(part);
  return y;
}

enum Which { DQ, DKV };
template <typename T, int DP, int A, int B, bool VEC>
const void* grad_kernel(Which w) {
  return w == DQ ? reinterpret_cast<const void*>(&attn_dq_kernel<T, DP, A, B, VEC>)
                 : reinterpret_cast<const void*>(&attn_dkv_kernel<T, DP, A, B, VEC>);
}
template <typename T, int DP>
const void* grad_kernel(Which w, bool wide, bool vec) {
  if (wide) return vec ? grad_kernel<T, DP, 4, 1, true>(w) : grad_kernel<T, DP, 4, 1, false>(w);
  return vec ? grad_kernel<T, DP, 1, 4, true>(w) : grad_kernel<T, DP, 1, 4, false>(w);
}
template <typename T>
const void* grad_kernel(Which w, int dp, bool wide, bool vec) {
  return dp == 32   ? grad_kernel<T, 32>(w, wide, vec)
         : dp == 64 ? grad_kernel<T, 64>(w, wide, vec)
                    : grad_kernel<T, 128>(w, wide, vec);
}
template <typename T, bool KEYS>
const void* add_kernel(int dp) {
  return dp == 32   ? reinterpret_cast<const void*>(&attn_add_kernel<T, 32, KEYS>)
         : dp == 64 ? reinterpret_cast<const void*>(&attn_add_kernel<T, 64, KEYS>)
                    : reinterpret_cast<const void*>(&attn_add_kernel<T, 128, KEYS>);
}

bool launch(const void* fn, int64_t grid, size_t lds, Args* a, hipStream_t stream) {
  void* args[] = {a};
  return grid == 0 ||
         hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(256), args, lds, stream) == hipSuccess;
}

}  // namespace
}  // namespace attn
}  // namespace dcn

extern "C" int dcn_cross_attention_backward_workspace_bytes(const dcn_attn_desc* d, size_t* bytes) {
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = dcn::attn::check(d);
  if (rc != DCN_OK) return rc;
  *bytes = d->batch == 0 ? 0 : dcn::attn::make_layout(d).bytes;
  return DCN_OK;
}

extern "C" int dcn_cross_attention_backward(const dcn_attn_desc* d, const void* q, const void* k, const void* v,
                                            const uint8_t* key_mask, const void* out, const float* lse,
                                            const void* grad_out, void* grad_q, void* grad_k, void* grad_v,
                                            void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace dcn::attn;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0) return DCN_OK;
  const bool rows = d->query_len > 0, keys = d->key_len > 0;
  if ((rows && (q == nullptr || out == nullptr || lse == nullptr || grad_out == nullptr)) ||
      (keys && (k == nullptr || v == nullptr)))
    return DCN_E_ARG;
  const Layout y = make_layout(d);
  if (y.bytes > 0 &&
      (workspace == nullptr || workspace_bytes < y.bytes || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return DCN_E_WORKSPACE;
  Args a{};
  fill_args(d, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.mask = key_mask;
  a.out = const_cast<void*>(out);
  a.lse = const_cast<float*>(lse);
  a.dout = grad_out;
  a.delta = static_cast<const float*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + y.part_at);
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const int64_t dense[3] = {0, 0, d->head_dim};
  const bool vec = vec_ok(q, d->q_stride, d->head_dim, es) && vec_ok(k, d->k_stride, d->head_dim, es) &&
                   vec_ok(v, d->v_stride, d->head_dim, es) && vec_ok(grad_out, dense, d->head_dim, es);
  const int64_t nbh = d->batch * d->key_heads, R = a.R;
  if (rows) {
    const void* fn = bf16 ? reinterpret_cast<const void*>(&attn_rows_kernel<uint16_t>)
                          : reinterpret_cast<const void*>(&attn_rows_kernel<float>);
    if (!launch(fn, (nbh * R + 15) / 16, 0, &a, stream)) return DCN_E_HIP;
  }
  if (grad_q != nullptr && rows) {
    a.splits = y.q.splits;
    a.per_split = y.q.per_split;
    const int64_t tiles = (R + (y.q.wide ? 127 : 31)) / (y.q.wide ? 128 : 32);
    const void* fn = bf16 ? grad_kernel<uint16_t>(DQ, y.q.dp, y.q.wide, vec) : grad_kernel<float>(DQ, y.q.dp, y.q.wide, vec);
    if (!launch(fn, nbh * tiles * a.splits, lds_bytes(y.q, es), &a, stream)) return DCN_E_HIP;
    if (a.splits > 1) {
      fn = bf16 ? add_kernel<uint16_t, false>(y.q.dp) : add_kernel<float, false>(y.q.dp);
      if (!launch(fn, (nbh * R * (y.q.dp / 4) + 255) / 256, 0, &a, stream)) return DCN_E_HIP;
    }
  }
  if ((grad_k != nullptr || grad_v != nullptr) && keys) {
    a.splits = y.kv.splits;
    a.per_split = y.kv.per_split;
    const int64_t tiles = (d->key_len + (y.kv.wide ? 127 : 31)) / (y.kv.wide ? 128 : 32);
    const void* fn =
        bf16 ? grad_kernel<uint16_t>(DKV, y.kv.dp, y.kv.wide, vec) : grad_kernel<float>(DKV, y.kv.dp, y.kv.wide, vec);
    if (!launch(fn, nbh * tiles * a.splits, lds_bytes(y.kv, es), &a, stream)) return DCN_E_HIP;
    if (a.splits > 1) {
      fn = bf16 ? add_kernel<uint16_t, true>(y.kv.dp) : add_kernel<float, true>(y.kv.dp);
      if (!launch(fn, (2 * nbh * d->key_len * (y.kv.dp / 4) + 255) / 256, 0, &a, stream)) return DCN_E_HIP;
    }
  }
  return DCN_OK;
}

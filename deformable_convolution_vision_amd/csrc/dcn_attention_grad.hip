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
// Launches: a pass over the rows (delta, and lse in powers of two); then dQ, and dK with dV, as
// workgroups of one launch, since neither fills the chip alone where one side is short: 128 rows
// and a loop over key tiles (as the forward), or 128 keys and a loop over row tiles, the tiles
// in a ring that buffer -> LDS loads fill ahead of use.  Where there are fewer tiles than the
// chip holds, their loops are split over workgroups, and a last launch adds the parts.  Each sum
// is formed in a fixed order: no atomics, the same bits each time.  The heads that share a key
// head are rows of one problem, so their gradients add up inside the loop of dK and dV.
//
// Both form the scores so that the first products' result registers are an operand
// of the second (see dcn_attention.h): dQ keeps a row per lane (S^T), dK/dV a key per lane
// (S).  Rows with no key have lse = -inf; it enters as +inf, which makes every weight 0.
//
// Arithmetic: fp32 sums; for bf16, P is rounded to bf16 as an operand of dV, dS enters dQ and dK as
// two bf16 operands (its rounded value and what that leaves: 16 bits of it), and the gradients
// are rounded once.  delta already carries the rounding of out; with a rounded dS on top of it dQ
// and dK were 1.4 to 1.6 times one rounding away from the exact gradients, with both parts 1.1.
// That costs a product more: 4200 queries over 1050 keys, 8 heads of 64, batch 2, 99 us without,
// 107 with both parts of dQ, 112 of dK too.
//
// What bounds it, measured: at that size the matrix units are busy 39 % of the time (the products are
// 14 Lq Lk D and 4 more for the second parts, of the formulas' 10), with the vector instructions for
// the weights beside them, which hardly overlap with the products of the same SIMD; the pass over
// the rows is 5 us, and adding the parts of split tiles (37 MB written, 28 read again) 8.  Two
// batches of 300 queries of 8 heads of 32 over 4200 keys, 32.3 us: 27 of the one round of loops,
// the rest the launches before and after it (4.8 and 4.7 alone).  fp32 (129 queries of 4 heads on 2 of 64 over 515 keys,
// batch 2, 25.5 us): 18 us are loops of one step each, the two other launches the rest.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"
#include "dcn_attention.h"

namespace dcn {
namespace attn {
namespace {

// delta, and lse in powers of two, of each row: float arrays of B * Hq * Lq rows (in the order of
// the pairs and their rows), one after the other.  16 bytes of a row (VEC) or one element a lane.
template <typename T, int DP, bool VEC>
__global__ __launch_bounds__(256) void attn_grad_rows_kernel(Args a) {
  constexpr int LPR = VEC ? Tile<T, DP>::kVecs : 16, RPB = 256 / LPR;   // lanes of a row, rows of a workgroup
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.R;
  const int64_t prow = (static_cast<int64_t>(a.first) + blockIdx.x) * RPB + threadIdx.x / LPR;
  if (prow >= rows) return;
  const int sub = threadIdx.x % LPR;
  const int bh = static_cast<int>(prow / a.R), r = static_cast<int>(prow % a.R);
  const int b = bh / a.Hkv, pos = r / a.g, head = (bh % a.Hkv) * a.g + r % a.g;
  const int64_t at = ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D;
  const T* o = static_cast<const T*>(a.out) + at;
  const T* go = static_cast<const T*>(a.dout) + at;
  float s = 0.f;
  if constexpr (VEC) {
    const Vec16<T> x = load_vec<T, true>(o, 0, sub * Elem<T>::kVec, a.D, true);
    const Vec16<T> y = load_vec<T, true>(go, 0, sub * Elem<T>::kVec, a.D, true);
#pragma unroll
    for (int j = 0; j < Elem<T>::kVec; ++j) s = fmaf(widen(x.e[j]), widen(y.e[j]), s);
  } else {
    for (int d = sub; d < a.D; d += LPR) s = fmaf(widen(o[d]), widen(go[d]), s);
  }
#pragma unroll
  for (int w = LPR / 2; w > 0; w >>= 1) s += __shfl_xor(s, w, LPR);
  if (sub == 0) {
    const float lse = a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.Lq + pos];
    float* out = const_cast<float*>(a.delta);
    out[prow] = lse == kNegInf ? -kNegInf : lse * kLog2e;   // a row with no key: every weight becomes 0
    out[rows + prow] = s;
  }
}

// Turns a wave's transposed sum (DP x 32) into rows through its own part of the LDS, 32 elements
// at a time, and hands 4 elements of row rr to store(rr, element, values).
template <int DT, typename Store>
__device__ __forceinline__ void rows_out(const f32x16 (&o)[DT], float* os, Store store) {
  constexpr int OST = 36;
  const int lane = threadIdx.x & 63, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < DT; ++i) {
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<float4*>(os + (lane & 31) * OST + acc_row(4 * r4, half)) =
          make_float4(o[i][4 * r4], o[i][4 * r4 + 1], o[i][4 * r4 + 2], o[i][4 * r4 + 3]);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int rr = n * 8 + lane / 8, d = (lane % 8) * 4;
      store(rr, 32 * i + d, *reinterpret_cast<const float4*>(os + rr * OST + d));
    }
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, int d, int D, float4 v, float f) {
  const float vals[4] = {v.x * f, v.y * f, v.z * f, v.w * f};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (d + j < D) p[d + j] = narrow<T>(vals[j]);
}

template <typename T>
__device__ __forceinline__ T* dq_row(const Args& a, const Work& w, int row) {
  return static_cast<T*>(a.dq) +
         ((static_cast<int64_t>(w.b) * a.Lq + row / a.g) * a.Hq + w.hk * a.g + row % a.g) * a.D;
}
template <typename T>
__device__ __forceinline__ T* dkv_row(const Args& a, const Work& w, int key, int which) {
  T* p = static_cast<T*>(which ? a.dv : a.dk);
  return p == nullptr ? p : p + ((static_cast<int64_t>(w.b) * a.Lk + key) * a.Hkv + w.hk) * a.D;
}

constexpr int kT = 64;           // rows of a tile in the LDS
constexpr int kRowVals = 2 * kT; // lse and delta of a row tile

// Waves of a SIMD (workgroups of a CU) that the registers allow.
// (fp32 rows of 64: 107 us with one, 74 with two and a few registers spilled, at B 4, Lq 55, Lk 1736, 8 heads on
// 2; bf16 rows of 128: 225 with one, 585 with two, at B 2, Lq = Lk = 2100, 8 heads.)
constexpr int waves_per_simd(int es, int dp) { return es * dp <= 64 ? 3 : es * dp <= 128 || (es == 4 && dp == 64) ? 2 : 1; }

// A wave's priority on its SIMD: first in its second products, so that they are not held up among
// the other wave's vector instructions.  (B 2, Lq 4200, Lk 1050, 8 heads of 64: 114.5 -> 112 us; Lq = Lk
// = 2100, 8 heads of 128: 241 -> 229; with three waves to a SIMD 32.6 -> 34 us, so not there.)
template <typename T, int DP>
__device__ __forceinline__ void go_first(bool first) {
  if constexpr (sizeof(T) == 2 && waves_per_simd(sizeof(T), DP) < 3) {
    if (first) __builtin_amdgcn_s_setprio(1);
    else __builtin_amdgcn_s_setprio(0);
  }
}

// What an operand of score gradients leaves of them by its rounding to bf16, as a second operand.
__device__ __forceinline__ POperand<uint16_t>::type rest_of(const float (&ds)[16], const POperand<uint16_t>::type& pf) {
  POperand<uint16_t>::type rest;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w2 = pf.f[h].w[j];
      rest.f[h].w[j] = pack_bf16(ds[8 * h + 2 * j] - __uint_as_float(w2 << 16),
                                 ds[8 * h + 2 * j + 1] - __uint_as_float(w2 & 0xffff0000u));
    }
  return rest;
}

template <typename T, int DP, int STAGES, bool VEC>
__device__ __forceinline__ void dq_part(const Args& a, int tile, T* lds) {
  constexpr int DT = DP / 32, BUF = 2 * kT * DP, AHEAD = STAGES - 1, LOADS = VEC ? 2 * tile_loads<T, DP, kT, 256> : 0;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = work_of(a, a.y, tile, 128, (a.Lk + kT - 1) / kT);
  const T* kp = static_cast<const T*>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2];
  const T* vp = static_cast<const T*>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2];
  const int row = w.row0 + wave * 32 + (lane & 31);
  const bool busy = w.row0 + wave * 32 < a.R;   // some of the wave's rows exist
  Frag<T> qf[DP / 16], gf[DP / 16];
  float lse2 = -kNegInf, delta = 0.f;
  {
    const bool live = row < a.R;
    const int pos = live ? row / a.g : 0, head = w.hk * a.g + (live ? row % a.g : 0);
    load_frags<T, DP, VEC>(static_cast<const T*>(a.q) + w.b * a.qs[0] + pos * a.qs[1] + head * a.qs[2], 0, a.D, live, qf);
    load_frags<T, DP, VEC>(static_cast<const T*>(a.dout) + ((static_cast<int64_t>(w.b) * a.Lq + pos) * a.Hq + head) * a.D,
                           0, a.D, live, gf);
    if (live) {
      const int64_t prow = static_cast<int64_t>(w.b * a.Hkv + w.hk) * a.R + row;
      lse2 = a.delta[prow];
      delta = a.delta[static_cast<int64_t>(a.B) * a.Hkv * a.R + prow];
    }
  }
  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc();
  const f32x16 zeros = zero_acc();

  KeyTiles tiles(a.mask == nullptr ? nullptr : a.mask + w.b * a.ms, a.Lk, w.s0, w.s1);
  // rows of padded keys are not read and taken as zeros: their weight is 0, and 0 times a NaN is none
  const auto send = [&](T* __restrict__ to) {
    int64_t k0;
    const uint64_t word = tiles.next(k0);
    if (word != 0) {
      fetch_tile<T, DP, kT, 256, VEC>(to, kp + k0 * a.ks[1], [&](int r) { return r * a.ks[1]; }, word, a.D, tid);
      fetch_tile<T, DP, kT, 256, VEC>(to + kT * DP, vp + k0 * a.vs[1], [&](int r) { return r * a.vs[1]; }, word,
                                      a.D, tid);
    }
    return word;
  };
  uint64_t word[AHEAD + 1];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) word[j] = send(lds + j * BUF);
  arrived(qf);
  arrived(gf);
  // one tile: `cur` is worked on while a later one is sent to `to`, another place (restrict: no
  // wait for what is on its way before `cur` is read)
  const auto turn = [&](const T* __restrict__ cur, T* __restrict__ to) {
    word[AHEAD] = send(to);
    const T* ks = cur;
    const T* vs = cur + kT * DP;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint32_t keep = static_cast<uint32_t>(word[0] >> (32 * n));
      if (keep == 0 || !busy) continue;
      f32x16 s = zeros, p = zeros;
      Frag<T> kf[DP / 16], vf[DP / 16];
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        kf[i] = row_frag<DP>(ks, 32 * n, i);
        vf[i] = row_frag<DP>(vs, 32 * n, i);
      }
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        s = mma(kf[i], qf[i], s);
        p = mma(vf[i], gf[i], p);
      }
      go_first<T, DP>(false);
      if (keep != 0xffffffffu) mask_scores(s, keep);
      float ds[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) ds[r] = exp2_fast(fmaf(s[r], a.c, -lse2)) * (p[r] - delta);
      typename POperand<T>::type pf;
      to_operand(ds, pf);
      if constexpr (sizeof(T) == 2) {
        const auto rest = rest_of(ds, pf);
        go_first<T, DP>(true);
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const Frag<T> c = col_frag<DP>(ks, 32 * n, 32 * i, h);
            o[i] = mma(c, pf.f[h], o[i]);
            o[i] = mma(c, rest.f[h], o[i]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] = mma_rows<DP>(ks, 32 * n, 32 * i, pf, o[i]);
      }
    }
  };
  int slot = 0;
  while (word[0] != 0) {
    if (AHEAD == 2 && word[1] != 0) wait_loads<LOADS>();
    else wait_loads<0>();
    lds_barrier();
    turn(lds + slot * BUF, lds + (slot == 0 ? STAGES - 1 : slot - 1) * BUF);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) word[j] = word[j + 1];
    slot = slot == STAGES - 1 ? 0 : slot + 1;
  }
  __syncthreads();
  rows_out(o, reinterpret_cast<float*>(lds) + wave * 32 * 36, [&](int rr, int d, float4 v) {
    const int at = wave * 32 + rr, orow = w.row0 + at;
    if (orow >= a.R) return;
    if (w.tail >= 0)
      *reinterpret_cast<float4*>(a.part + ((static_cast<int64_t>(w.tail) * a.y.splits + w.split) * 128 + at) * DP + d) = v;
    else
      store4<T>(dq_row<T>(a, w, orow), d, a.D, v, a.scale);
  });
}

template <typename T, int DP, int STAGES, bool VEC>
__device__ __forceinline__ void dkv_part(const Args& a, int tile, T* lds) {
  // a place in the ring: query rows, gradient rows, and lse and delta of each
  constexpr int DT = DP / 32, BUF = 2 * kT * DP + kRowVals * 4 / static_cast<int>(sizeof(T)), AHEAD = STAGES - 1;
  constexpr int LOADS = VEC ? 2 * tile_loads<T, DP, kT, 256> + 1 : 1;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = work_of(a, a.ykv, tile, 128, (a.R + kT - 1) / kT);
  const int key = w.row0 + wave * 32 + (lane & 31);
  bool live = key < a.Lk;
  if (a.mask != nullptr && live) live = a.mask[w.b * a.ms + key] != 0;
  Frag<T> kf[DP / 16], vf[DP / 16];
  load_frags<T, DP, VEC>(static_cast<const T*>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2] + (live ? key : 0) * a.ks[1], 0, a.D,
                         live, kf);
  load_frags<T, DP, VEC>(static_cast<const T*>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2] + (live ? key : 0) * a.vs[1], 0, a.D,
                         live, vf);
  f32x16 ok[DT], ov[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    ok[i] = zero_acc();
    ov[i] = zero_acc();
  }
  const f32x16 zeros = zero_acc();
  const bool any = __any(live);
  // keys that are all padding have no gradient, and no rows are read for them
  const int s1 = __syncthreads_or(any) ? w.s1 : w.s0;
  const T* qb = static_cast<const T*>(a.q) + w.b * a.qs[0] + w.hk * a.g * a.qs[2];
  const T* gb = static_cast<const T*>(a.dout) + (static_cast<int64_t>(w.b) * a.Lq * a.Hq + w.hk * a.g) * a.D;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.R, row_base = static_cast<int64_t>(w.b * a.Hkv + w.hk) * a.R;
  const auto send = [&](int t, T* __restrict__ to) {
    const int r0 = t * kT, n = min(kT, a.R - r0);
    const uint64_t in = n == 64 ? ~uint64_t{0} : (uint64_t{1} << n) - 1;
    // rows run over the heads that share the key head, then over positions
    const int pos0 = r0 / a.g, h0 = r0 - pos0 * a.g;
    const auto split = [&](int r, int& pos, int& h) {
      pos = r;
      h = 0;
      if (a.g > 1) {
        const unsigned x = static_cast<unsigned>(h0 + r);
        pos = static_cast<int>(x / static_cast<unsigned>(a.g));
        h = static_cast<int>(x) - pos * a.g;
      }
    };
    fetch_tile<T, DP, kT, 256, VEC>(to, qb + pos0 * a.qs[1], [&](int r) {
      int pos, h;
      split(r, pos, h);
      return pos * a.qs[1] + h * a.qs[2];
    }, in, a.D, tid);
    fetch_tile<T, DP, kT, 256, VEC>(to + kT * DP, gb + static_cast<int64_t>(pos0) * a.Hq * a.D, [&](int r) {
      int pos, h;
      split(r, pos, h);
      return (static_cast<int64_t>(pos) * a.Hq + h) * a.D;
    }, in, a.D, tid);
    // lse by waves 0 and 2, delta by 1 and 3 (a pair writes the same values, and every wave has as many loads
    // under way); rows beyond the last give zeros, and their zero query and gradient rows add nothing
    const int which = wave & 1;
    const __amdgpu_buffer_rsrc_t rs = rsrc_of(a.delta + which * rows + row_base + r0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(reinterpret_cast<float*>(to + 2 * kT * DP) + which * kT), 4,
                                             lane < n ? lane * 4 : kOutside, 0, 0, 0);
  };
#pragma unroll
  for (int j = 0; j < AHEAD; ++j)
    if (w.s0 + j < s1) send(w.s0 + j, lds + j * BUF);
  arrived(kf);
  arrived(vf);
  const auto turn = [&](int t, const T* __restrict__ cur, T* __restrict__ to) {
    if (t + AHEAD < s1) send(t + AHEAD, to);
    if (!any) return;
    const T* qs = cur;
    const T* gs = cur + kT * DP;
    const float* ls = reinterpret_cast<const float*>(cur + 2 * kT * DP);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int r0 = 32 * n;
      f32x16 s = zeros, dp = zeros;
      Frag<T> qf[DP / 16], gf[DP / 16];
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        qf[i] = row_frag<DP>(qs, r0, i);
        gf[i] = row_frag<DP>(gs, r0, i);
      }
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        s = mma(qf[i], kf[i], s);
        dp = mma(gf[i], vf[i], dp);
      }
      go_first<T, DP>(false);
      float p[16], ds[16];
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const float4 lse = *reinterpret_cast<const float4*>(ls + r0 + acc_row(4 * r4, half));
        const float4 del = *reinterpret_cast<const float4*>(ls + kT + r0 + acc_row(4 * r4, half));
        const float le[4] = {lse.x, lse.y, lse.z, lse.w}, de[4] = {del.x, del.y, del.z, del.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * r4 + j;
          p[r] = exp2_fast(fmaf(s[r], a.c, -le[j]));
          ds[r] = p[r] * (dp[r] - de[j]);
        }
      }
      typename POperand<T>::type pf, df;
      to_operand(p, pf);
      to_operand(ds, df);
      if constexpr (sizeof(T) == 2) {
        const auto rest = rest_of(ds, df);
        go_first<T, DP>(true);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          ov[i] = mma_rows<DP>(gs, r0, 32 * i, pf, ov[i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const Frag<T> c = col_frag<DP>(qs, r0, 32 * i, h);
            ok[i] = mma(c, df.f[h], ok[i]);
            ok[i] = mma(c, rest.f[h], ok[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          ov[i] = mma_rows<DP>(gs, r0, 32 * i, pf, ov[i]);
          ok[i] = mma_rows<DP>(qs, r0, 32 * i, df, ok[i]);
        }
      }
    }
  };
  int slot = 0;
  for (int t = w.s0; t < s1; ++t) {
    if (AHEAD == 2 && t + 1 < s1) wait_loads<LOADS>();
    else wait_loads<0>();
    lds_barrier();
    turn(t, lds + slot * BUF, lds + (slot == 0 ? STAGES - 1 : slot - 1) * BUF);
    slot = slot == STAGES - 1 ? 0 : slot + 1;
  }
  // a lane whose key is padding has summed the weights of a zero key row: its gradients are 0
  if (!live) {
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) ok[i][r] = ov[i][r] = 0.f;
  }
  __syncthreads();
  const auto store = [&](int rr, int d, float4 v, int which) {
    const int at = wave * 32 + rr, okey = w.row0 + at;
    if (okey >= a.Lk) return;
    if (w.tail >= 0) {
      const int64_t part = (static_cast<int64_t>(w.tail) * a.ykv.splits + w.split) * 2 + which;
      *reinterpret_cast<float4*>(a.part_kv + (part * 128 + at) * DP + d) = v;
      return;
    }
    T* out = dkv_row<T>(a, w, okey, which);
    if (out != nullptr) store4<T>(out, d, a.D, v, which ? 1.f : a.scale);
  };
  float* os = reinterpret_cast<float*>(lds) + wave * 32 * 36;
  rows_out(ok, os, [&](int rr, int d, float4 v) { store(rr, d, v, 0); });
  rows_out(ov, os, [&](int rr, int d, float4 v) { store(rr, d, v, 1); });
}

// Workgroups kv0 .. kv1 - 1: dK and dV; the others (from q0 on): dQ.  Those with the longer loops
// come first (dQ first: 38 -> 32 us at B 2, Lq 300, Lk 4200, 8 heads of 32).
template <typename T, int DP, int STAGES, bool VEC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(waves_per_simd(sizeof(T), DP), waves_per_simd(sizeof(T), DP))))
void attn_grad_kernel(Args a, int kv0, int kv1, int q0) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* lds = reinterpret_cast<T*>(smem);
  const int id = a.first + blockIdx.x;
  if (id < kv0 || id >= kv1) dq_part<T, DP, STAGES, VEC>(a, id - q0, lds);
  else dkv_part<T, DP, STAGES, VEC>(a, id - kv0, lds);
}

// Adds up the parts of split tiles: one thread for 4 elements of a row of dQ, or a key of dK or
// dV (vectors `q4` and beyond).
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_grad_add_kernel(Args a, int64_t q4, int64_t n4) {
  constexpr int V4 = DP / 4;
  int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= n4) return;
  const bool kv = at >= q4;
  if (kv) at -= q4;
  const Tiling& y = kv ? a.ykv : a.y;
  const int d = static_cast<int>(at % V4) * 4, rr = static_cast<int>(at / V4 % 128);
  const int64_t unit = at / V4 / 128;
  const int which = kv ? static_cast<int>(unit % 2) : 0, tail = static_cast<int>(kv ? unit / 2 : unit);
  const int nbh = a.B * a.Hkv, tile = y.full + tail, bh = tile % nbh;
  Work w;
  w.b = bh / a.Hkv;
  w.hk = bh % a.Hkv;
  w.row0 = tile / nbh * 128;
  if (w.row0 + rr >= (kv ? a.Lk : a.R)) return;
  const int64_t step = static_cast<int64_t>(kv ? 2 : 1) * 128 * DP;
  const float* p = (kv ? a.part_kv : a.part) + (static_cast<int64_t>(tail) * y.splits * (kv ? 2 : 1) + which) * 128 * DP +
                   static_cast<int64_t>(rr) * DP + d;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < y.splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(p + s * step);
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  T* out = kv ? dkv_row<T>(a, w, w.row0 + rr, which) : dq_row<T>(a, w, w.row0 + rr);
  if (out != nullptr) store4<T>(out, d, a.D, acc, which ? 1.f : a.scale);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  int dp;
  Tiling q, kv;
  size_t part_at, part_kv_at, bytes;   // the row values come first
};

Layout make_layout(const dcn_attn_desc* d) {
  Layout y{};
  y.dp = padded_head(d->head_dim);
  const int64_t nbh = d->batch * d->key_heads, R = d->query_len * (d->query_heads / d->key_heads);
  const int64_t rows = (R + kT - 1) / kT, keys = (d->key_len + kT - 1) / kT;
  // One launch holds both kinds of workgroups.  dK and dV are split to fill the chip by
  // themselves; dQ, where its tiles alone do not fill it, into what the last round has left.  A
  // step of fp32 is 16 times as many matrix cycles as one of bf16: there a single step is a part.
  const int es = d->dtype == DCN_BF16 ? 2 : 4, least = es == 2 ? 2 : 1;
  const int64_t slots = static_cast<int64_t>(kCUs) * waves_per_simd(es, y.dp), nq = nbh * ((R + 127) / 128);
  y.kv = tile_over(nbh * ((d->key_len + 127) / 128), rows, slots, least);
  int64_t left = slots;
  if (nq < slots) {
    left = slots - workgroups(y.kv) % slots;
    if (left < nq) left += slots;
    // ... or one round more, where these parts would outlast the others by far
    if ((keys * nq + left - 1) / left > 4 * y.kv.per_split) left += slots;
  }
  y.q = tile_over(nq, keys, left, least);
  y.part_at = up256(static_cast<size_t>(nbh) * R * 8);
  const size_t tile = static_cast<size_t>(128) * y.dp * 4;
  y.part_kv_at = y.part_at + static_cast<size_t>(y.q.tiles - y.q.full) * y.q.splits * tile;
  y.bytes = y.part_kv_at + static_cast<size_t>(y.kv.tiles - y.kv.full) * y.kv.splits * 2 * tile;
  return y;
}

size_t grad_lds(int row_bytes) {
  const size_t ring = static_cast<size_t>(stages_of(row_bytes)) * (2 * kT * row_bytes + kRowVals * 4);
  return std::max<size_t>(ring, 4 * 32 * 36 * 4);
}

template <typename T, int DP>
const void* grad_kernel(bool vec) {
  constexpr int S = stages_of(DP * sizeof(T));
  return vec ? reinterpret_cast<const void*>(&attn_grad_kernel<T, DP, S, true>)
             : reinterpret_cast<const void*>(&attn_grad_kernel<T, DP, S, false>);
}
template <typename T, int DP>
const void* rows_kernel(bool vec) {
  return vec ? reinterpret_cast<const void*>(&attn_grad_rows_kernel<T, DP, true>)
             : reinterpret_cast<const void*>(&attn_grad_rows_kernel<T, DP, false>);
}

template <typename T, int DP>
int run_grad(Args& a, const Layout& y, bool vec, hipStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * a.R;
  void* args[] = {&a};
  if (rows > 0) {
    const int per = vec ? 256 / Tile<T, DP>::kVecs : 16;
    if (!launch_groups(rows_kernel<T, DP>(vec), (rows + per - 1) / per, 256, args, &a, 0, stream)) return DCN_E_HIP;
  }
  const bool q = a.dq != nullptr && rows > 0, keys = (a.dk != nullptr || a.dv != nullptr) && a.Lk > 0;
  const int64_t kv = keys ? workgroups(y.kv) : 0, nq = q ? workgroups(y.q) : 0, grid = kv + nq;
  if (grid == 0) return DCN_OK;
  const bool q_first = y.q.per_split > y.kv.per_split;
  int kv0 = q_first ? static_cast<int>(nq) : 0, kv1 = kv0 + static_cast<int>(kv), q0 = q_first ? 0 : kv1;
  void* grad_args[] = {&a, &kv0, &kv1, &q0};
  if (!launch_groups(grad_kernel<T, DP>(vec), grid, 256, grad_args, &a, grad_lds(DP * sizeof(T)), stream)) return DCN_E_HIP;
  int64_t q4 = q ? static_cast<int64_t>(y.q.tiles - y.q.full) * 128 * (DP / 4) : 0;
  int64_t n4 = q4 + (keys ? static_cast<int64_t>(y.kv.tiles - y.kv.full) * 2 * 128 * (DP / 4) : 0);
  if (n4 == 0) return DCN_OK;
  void* add_args[] = {&a, &q4, &n4};
  return hipLaunchKernel(reinterpret_cast<const void*>(&attn_grad_add_kernel<T, DP>),
                         dim3(static_cast<unsigned>((n4 + 255) / 256)), dim3(256), add_args, 0, stream) == hipSuccess
             ? DCN_OK
             : DCN_E_HIP;
}
template <typename T>
int run_grad(Args& a, const Layout& y, bool vec, hipStream_t stream) {
  return y.dp == 32   ? run_grad<T, 32>(a, y, vec, stream)
         : y.dp == 64 ? run_grad<T, 64>(a, y, vec, stream)
                      : run_grad<T, 128>(a, y, vec, stream);
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
  a.part_kv = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + y.part_kv_at);
  a.dq = grad_q;
  a.dk = grad_k;
  a.dv = grad_v;
  a.y = y.q;
  a.ykv = y.kv;
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  // out and grad_out are dense; a row tile's positions have to lie within 32 bits of each other too
  const int64_t dense[3] = {0, d->query_heads * d->head_dim, d->head_dim};
  const bool vec = vec_ok(q, d->q_stride, d->head_dim, es) && vec_ok(k, d->k_stride, d->head_dim, es) &&
                   vec_ok(v, d->v_stride, d->head_dim, es) && vec_ok(grad_out, dense, d->head_dim, es) &&
                   vec_ok(out, dense, d->head_dim, es) && 64 * d->q_stride[1] + (a.g - 1) * d->q_stride[2] <= int64_t{1} << 28;
  return bf16 ? run_grad<uint16_t>(a, y, vec, stream) : run_grad<float>(a, y, vec, stream);
}

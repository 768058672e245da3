// dcn_attention.hip -- gfx950 cross attention to an encoder's states.
//
// For a query row q (one position of one head) and the keys j that its batch element's mask
// keeps, with s_j = scale * q . k_j:
//
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   lse = m + log sum_j exp(s_j - m)
//
// for any m; the kernel carries m as the running maximum over the key tiles seen so far, and
// rescales what it has summed when a tile raises it, so keys and values are read once and no
// score leaves the registers.  Scores are formed transposed, S^T = K Q^T (a lane holds one
// row q and 16 keys of it), because then the lane's own exponentials are the operand of the
// second product, out^T += V^T P^T, without an exchange between lanes, and the maximum, the
// sum and the rescaling factor are one value per lane.
//
// The heads that share a key head are rows of one problem (row r: position r / g, head r % g),
// so a single token of many heads reads each key once.
//
// Two forms of one kernel: `wide`, four waves of 32 rows share a 64-key tile; and narrow, 32
// rows, four waves take 32 keys each of a 128-key tile and join at the end.  Narrow launches
// may also split the keys over workgroups: each writes its maximum, sum and undivided output,
// and attn_join_kernel adds them up in split order.
//
// Arithmetic: products of bf16 (exact) or fp32 added in fp32; the softmax in fp32; for bf16
// the weights exp(s - m) are rounded to bf16 as the second product's operand (their sum is
// not), and the output is rounded once.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"
#include "dcn_attention.h"

namespace dcn {
namespace attn {
namespace {

template <typename T, int DP, int WQ, int WK, bool VEC>
__global__ __launch_bounds__(64 * WQ * WK) void attn_fwd_kernel(Args a) {
  constexpr int NT = 64 * WQ * WK, KV = Elem<T>::kVec, ST = DP + Elem<T>::kPad;
  constexpr int SUB = WK == 1 ? 2 : 1;         // 32-key blocks of a tile that one wave takes
  constexpr int KT = 32 * SUB * WK;            // keys of a tile
  constexpr int VPR = DP / KV;                 // 16-byte vectors of a row
  constexpr int NV = KT * VPR / NT;            // of a tile, per thread
  constexpr int DT = DP / 32;
  constexpr int OST = DP + 4;                  // LDS row of the joined output
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* ks = reinterpret_cast<T*>(smem);
  T* vs = ks + KT * ST;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = tid >> 6;
  const int wq = wave / WK, wk = wave % WK;
  // consecutive workgroups are consecutive (batch, head) pairs: the row tiles that read the
  // same keys then run on the same XCD when the pairs are a multiple of 8
  const int nbh = a.B * a.Hkv;
  int id = blockIdx.x;
  const int bh = id % nbh;
  id /= nbh;
  const int split = id % a.splits, rt = id / a.splits;
  const int b = bh / a.Hkv, hk = bh % a.Hkv;
  const T* kp = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[2];
  const T* vp = static_cast<const T*>(a.v) + b * a.vs[0] + hk * a.vs[2];
  const uint8_t* mp = a.mask == nullptr ? nullptr : a.mask + b * a.ms;

  // this lane's row
  const int row = rt * 32 * WQ + wq * 32 + (lane & 31);
  Frag<T> qf[DP / 16];
  {
    const bool live = row < a.R;
    const int pos = live ? row / a.g : 0, head = hk * a.g + (live ? row % a.g : 0);
    const T* qp = static_cast<const T*>(a.q) + b * a.qs[0] + pos * a.qs[1] + head * a.qs[2];
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) qf[i] = load_frag<T, VEC>(qp, 16 * i + 8 * half, a.D, live);
  }

  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc();
  float m = kNegInf, l = 0.f;

  const int tiles = (a.Lk + KT - 1) / KT;
  const int t0 = split * a.per_split, t1 = min(tiles, t0 + a.per_split);
  Vec16<T> kr[NV], vr[NV];
  const auto load_tile = [&](int t) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, key = t * KT + at / VPR, d = (at % VPR) * KV;
      bool live = key < a.Lk;
      kr[i] = load_vec<T, VEC>(kp + key * a.ks[1], d, a.D, live);
      // a padded key's weight is exactly 0, but 0 times an infinity or NaN in its value row
      // would not be: such rows are taken as zeros
      if (mp != nullptr && live) live = mp[key] != 0;
      vr[i] = load_vec<T, VEC>(vp + key * a.vs[1], d, a.D, live);
    }
  };
  if (t0 < t1) load_tile(t0);
  for (int t = t0; t < t1; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = tid + i * NT, key = at / VPR, d = (at % VPR) * KV;
      *reinterpret_cast<uint4*>(ks + key * ST + d) = kr[i].u;
      *reinterpret_cast<uint4*>(vs + key * ST + d) = vr[i].u;
    }
    __syncthreads();
    if (t + 1 < t1) load_tile(t + 1);
    // which of the wave's keys count: bit i of word is key k0 + i
    const int k0 = t * KT + wk * 32 * SUB;
    uint64_t word;
    {
      const int key = k0 + lane;
      bool live = lane < 32 * SUB && key < a.Lk;
      if (mp != nullptr && live) live = mp[key] != 0;
      word = __ballot(live);
    }
    if (word == 0) continue;
    float p[SUB][16];
    float mt = kNegInf;
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      f32x16 acc = zero_acc();
      const T* krow = ks + (wk * 32 * SUB + s * 32 + (lane & 31)) * ST + 8 * half;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) acc = mma(lds_frag(krow + 16 * i), qf[i], acc);
      const uint32_t w = static_cast<uint32_t>(word >> (32 * s));
#pragma unroll
      for (int r = 0; r < 16; ++r) p[s][r] = acc[r];
      if (w != 0xffffffffu) {
        const uint32_t wh = w >> (4 * half);
#pragma unroll
        for (int r = 0; r < 16; ++r) p[s][r] = (wh >> acc_row(r, 0)) & 1u ? p[s][r] : kNegInf;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) mt = fmaxf(mt, p[s][r]);
    }
    mt = max_halves(mt);
    const float mn = fmaxf(m, mt * a.c);
    const float ms = mn == kNegInf ? 0.f : mn;   // no key counted yet: exp2(-inf) = 0 below
    const float alpha = exp2_fast(m - ms);
    m = mn;
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < SUB; ++s)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        p[s][r] = exp2_fast(fmaf(p[s][r], a.c, -ms));
        sum += p[s][r];
      }
    l = fmaf(l, alpha, sum);
    if (__any(alpha != 1.f)) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
    }
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      typename POperand<T>::type pf;
      to_operand(p[s], pf);
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] = mma_rows(vs + (wk * 32 * SUB + s * 32) * ST, ST, 32 * i, pf, o[i]);
    }
  }

  // join the waves that took different keys of the same rows, through LDS (which also turns
  // the transposed registers into rows)
  l = sum_halves(l);
  float* os = reinterpret_cast<float*>(smem);             // [WQ*WK][32][OST]
  float* ml = os + WQ * WK * 32 * OST;                    // [WQ*WK][32][2]
  __syncthreads();
  if (half == 0) {
    ml[(wave * 32 + lane) * 2] = m;
    ml[(wave * 32 + lane) * 2 + 1] = l;
  }
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<float4*>(os + (wave * 32 + (lane & 31)) * OST + 32 * i + acc_row(4 * r4, half)) =
          make_float4(o[i][4 * r4], o[i][4 * r4 + 1], o[i][4 * r4 + 2], o[i][4 * r4 + 3]);
  __syncthreads();
  constexpr int V4 = DP / 4;
  for (int at = tid; at < WQ * 32 * V4; at += NT) {
    const int rr = at / V4, d = (at % V4) * 4, grp = rr / 32, ri = rr % 32;
    const int orow = rt * 32 * WQ + rr;
    if (orow >= a.R) continue;
    float mm = kNegInf, ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WK; ++w) mm = fmaxf(mm, ml[((grp * WK + w) * 32 + ri) * 2]);
    const float ms = mm == kNegInf ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const int slot = (grp * WK + w) * 32 + ri;
      const float f = exp2_fast(ml[slot * 2] - ms);
      const float4 v = *reinterpret_cast<const float4*>(os + slot * OST + d);
      ll = fmaf(f, ml[slot * 2 + 1], ll);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if (a.splits > 1) {
      const int64_t prow = (static_cast<int64_t>(split) * nbh + bh) * a.R + orow;
      *reinterpret_cast<float4*>(a.part + prow * DP + d) = acc;
      if (d == 0) {
        a.part_ml[prow * 2] = mm;
        a.part_ml[prow * 2 + 1] = ll;
      }
      continue;
    }
    const int pos = orow / a.g, head = hk * a.g + orow % a.g;
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);   // no key: zeros; a NaN sum stays NaN
    T* op = static_cast<T*>(a.out) + ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D;
    const float vals[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (d + j < a.D) op[d + j] = narrow<T>(vals[j]);
    if (d == 0 && a.lse != nullptr)
      a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.Lq + pos] =
          ll == 0.f ? kNegInf : fmaf(ms, kLn2, logf(ll));
  }
}

// Adds up the parts of split keys: one thread for 4 elements of a row.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(Args a) {
  constexpr int V4 = DP / 4;
  const int nbh = a.B * a.Hkv;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t rows = static_cast<int64_t>(nbh) * a.R, prow = at / V4;
  const int d = static_cast<int>(at % V4) * 4;
  if (prow >= rows) return;
  float mm = kNegInf, ll = 0.f;
  for (int s = 0; s < a.splits; ++s) mm = fmaxf(mm, a.part_ml[(s * rows + prow) * 2]);
  const float ms = mm == kNegInf ? 0.f : mm;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; ++s) {
    const float f = exp2_fast(a.part_ml[(s * rows + prow) * 2] - ms);
    const float4 v = *reinterpret_cast<const float4*>(a.part + (s * rows + prow) * DP + d);
    ll = fmaf(f, a.part_ml[(s * rows + prow) * 2 + 1], ll);
    acc[0] = fmaf(f, v.x, acc[0]);
    acc[1] = fmaf(f, v.y, acc[1]);
    acc[2] = fmaf(f, v.z, acc[2]);
    acc[3] = fmaf(f, v.w, acc[3]);
  }
  const int bh = static_cast<int>(prow / a.R), r = static_cast<int>(prow % a.R);
  const int b = bh / a.Hkv, pos = r / a.g, head = (bh % a.Hkv) * a.g + r % a.g;
  const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
  T* op = static_cast<T*>(a.out) + ((static_cast<int64_t>(b) * a.Lq + pos) * a.Hq + head) * a.D;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (d + j < a.D) op[d + j] = narrow<T>(acc[j] * inv);
  if (d == 0 && a.lse != nullptr)
    a.lse[(static_cast<int64_t>(b) * a.Hq + head) * a.Lq + pos] = ll == 0.f ? kNegInf : fmaf(ms, kLn2, logf(ll));
}

constexpr int kCUs = 256;

Plan make_plan(const dcn_attn_desc* d) {
  Plan p{};
  p.dp = d->head_dim <= 32 ? 32 : d->head_dim <= 64 ? 64 : 128;
  const int64_t nbh = d->batch * d->key_heads, R = d->query_len * (d->query_heads / d->key_heads);
  p.wide = R > 96 && nbh * ((R + 127) / 128) >= 2 * kCUs;
  p.tile = p.wide ? 64 : 128;
  const int64_t tiles = std::max<int64_t>(1, (d->key_len + p.tile - 1) / p.tile);
  int64_t splits = 1;
  if (!p.wide) {
    const int64_t groups = nbh * ((R + 31) / 32);
    splits = std::min<int64_t>(std::max<int64_t>(1, 2 * kCUs / groups), std::max<int64_t>(1, tiles / 2));
  }
  p.per_split = static_cast<int>((tiles + splits - 1) / splits);
  p.splits = static_cast<int>((tiles + p.per_split - 1) / p.per_split);
  return p;
}

size_t lds_bytes(const Plan& p, int es) {
  const int pad = es == 2 ? 16 : 4;
  const size_t tile = static_cast<size_t>(2) * p.tile * (p.dp + pad) * es;
  const size_t join = static_cast<size_t>(4) * 32 * (p.dp + 4 + 2) * 4;
  return std::max(tile, join);
}

size_t part_bytes(const dcn_attn_desc* d, const Plan& p, size_t* ml_at) {
  const size_t rows = static_cast<size_t>(p.splits) * d->batch * d->query_heads * d->query_len;
  *ml_at = (rows * p.dp * 4 + 255) / 256 * 256;
  return p.splits > 1 ? *ml_at + (rows * 8 + 255) / 256 * 256 : 0;
}

template <typename T, int DP>
const void* fwd_kernel(bool wide, bool vec) {
  if (wide)
    return vec ? reinterpret_cast<const void*>(&attn_fwd_kernel<T, DP, 4, 1, true>)
               : reinterpret_cast<const void*>(&attn_fwd_kernel<T, DP, 4, 1, false>);
  return vec ? reinterpret_cast<const void*>(&attn_fwd_kernel<T, DP, 1, 4, true>)
             : reinterpret_cast<const void*>(&attn_fwd_kernel<T, DP, 1, 4, false>);
}
template <typename T>
const void* fwd_kernel(int dp, bool wide, bool vec) {
  return dp == 32 ? fwd_kernel<T, 32>(wide, vec) : dp == 64 ? fwd_kernel<T, 64>(wide, vec) : fwd_kernel<T, 128>(wide, vec);
}
template <typename T>
const void* join_kernel(int dp) {
  return dp == 32   ? reinterpret_cast<const void*>(&attn_join_kernel<T, 32>)
         : dp == 64 ? reinterpret_cast<const void*>(&attn_join_kernel<T, 64>)
                    : reinterpret_cast<const void*>(&attn_join_kernel<T, 128>);
}

}  // namespace

int check(const dcn_attn_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  const int64_t big = 2147483647;
  if (d->batch < 0 || d->query_len < 0 || d->key_len < 0 || d->query_heads < 1 || d->key_heads < 1 ||
      d->head_dim < 1 || d->query_heads % d->key_heads != 0 || !std::isfinite(d->scale) || !(d->scale > 0.f) ||
      d->mask_stride < 0)
    return DCN_E_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0) return DCN_E_ARG;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  if (d->head_dim > 128) return DCN_E_UNSUPPORTED;
  // int32 row and workgroup counts; addresses are 64-bit
  if (d->batch > big || d->query_len > big || d->key_len > big - 256 || d->query_heads > big || d->key_heads > big)
    return DCN_E_UNSUPPORTED;
  const double rows = static_cast<double>(d->query_len) * (d->query_heads / d->key_heads);
  const double groups = static_cast<double>(d->batch) * d->key_heads;
  if (rows > big - 256 || groups * (rows + 128) > big || groups * (static_cast<double>(d->key_len) + 128) > big)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

void fill_args(const dcn_attn_desc* d, Args* a) {
  for (int i = 0; i < 3; ++i) {
    a->qs[i] = d->q_stride[i];
    a->ks[i] = d->k_stride[i];
    a->vs[i] = d->v_stride[i];
  }
  a->ms = d->mask_stride;
  a->B = static_cast<int>(d->batch);
  a->Lq = static_cast<int>(d->query_len);
  a->Lk = static_cast<int>(d->key_len);
  a->Hq = static_cast<int>(d->query_heads);
  a->Hkv = static_cast<int>(d->key_heads);
  a->g = a->Hq / a->Hkv;
  a->D = static_cast<int>(d->head_dim);
  a->R = a->Lq * a->g;
  a->scale = d->scale;
  a->c = d->scale * kLog2e;
}

}  // namespace attn
}  // namespace dcn

extern "C" int dcn_cross_attention_workspace_bytes(const dcn_attn_desc* d, size_t* bytes) {
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = dcn::attn::check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->query_len == 0) {
    *bytes = 0;
    return DCN_OK;
  }
  size_t at;
  *bytes = dcn::attn::part_bytes(d, dcn::attn::make_plan(d), &at);
  return DCN_OK;
}

extern "C" int dcn_cross_attention(const dcn_attn_desc* d, const void* q, const void* k, const void* v,
                                   const uint8_t* key_mask, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  using namespace dcn::attn;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->query_len == 0) return DCN_OK;
  if (q == nullptr || out == nullptr || (d->key_len > 0 && (k == nullptr || v == nullptr))) return DCN_E_ARG;
  const Plan p = make_plan(d);
  size_t ml_at;
  const size_t need = part_bytes(d, p, &ml_at);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return DCN_E_WORKSPACE;
  Args a{};
  fill_args(d, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.mask = key_mask;
  a.out = out;
  a.lse = lse;
  a.splits = p.splits;
  a.per_split = p.per_split;
  if (need > 0) {
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + ml_at);
  }
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const bool vec = vec_ok(q, d->q_stride, d->head_dim, es) && vec_ok(k, d->k_stride, d->head_dim, es) &&
                   vec_ok(v, d->v_stride, d->head_dim, es);
  const int rows = p.wide ? 128 : 32;
  const int64_t grid = static_cast<int64_t>(a.B) * a.Hkv * ((a.R + rows - 1) / rows) * p.splits;
  void* args[] = {&a};
  const void* fn = bf16 ? fwd_kernel<uint16_t>(p.dp, p.wide, vec) : fwd_kernel<float>(p.dp, p.wide, vec);
  if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(256), args, lds_bytes(p, es), stream) != hipSuccess)
    return DCN_E_HIP;
  if (p.splits > 1) {
    const int64_t n = static_cast<int64_t>(a.B) * a.Hkv * a.R * (p.dp / 4);
    fn = bf16 ? join_kernel<uint16_t>(p.dp) : join_kernel<float>(p.dp);
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), args, 0, stream) != hipSuccess)
      return DCN_E_HIP;
  }
  return DCN_OK;
}

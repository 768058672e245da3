// dcn_paged.hip -- gfx950 attention of one new token of each sequence to its pages of a cache.
//
// For sequence b, query head h and its key head n = h / g (g = Hq / Hkv), over positions j < lengths[b]:
//
//   s_j = scale q . k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + log sum_j exp(s_j - m)
//
// for any m, carried as the running maximum.  The g heads that share a key head are the rows of one
// problem, 16 at a time, so a key head's rows are read once for them.  Scores are formed transposed,
// S^T = K Q^T, on 16x16 matrix instructions: a lane holds one query head and 4 of 16 positions, which is what
// the second product, out^T += V^T P^T, takes as it stands.
//
// A wave takes blocks of 32 positions on its own: their keys come straight from memory as the first
// product's operand, their values through registers and the wave's own part of the LDS, from where they are
// read transposed.  A block's page entries are fetched two blocks ahead and its rows one block ahead, so
// that a page's look-up is never waited for in line.  Pages of any size: each position has its own address.
//
// Lengths are known on the device only, so every workgroup derives from them which part it has
// (parts_of): all sequences' steps are shared out evenly over as many workgroups as the chip
// holds.  A sequence of one part is written as it is; others leave their parts (maximum, sum, undivided output),
// which paged_join_kernel adds in order.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"
#include "dcn_attention.h"

namespace dcn {
namespace attn {
namespace {

struct PagedArgs {
  const void *q, *k, *v;
  const int32_t *table, *lengths;
  void* out;
  float* lse;
  float* part;             // [part][16][DP]
  float* part_ml;          // [part][16][2]
  int64_t qs[2], ks[3], vs[3], ts;
  int B, Hq, Hkv, g, D;
  int tiles;               // of 16 rows, of a key head
  int num_pages, page_size, capacity;
  int slots;               // parts of a key head's tile that the plan aims at
  int grid;                // workgroups of a key head's tile (the most parts that there can be)
  int64_t first;           // workgroups of launches before this one
  float c;                 // scale * log2(e)
};

constexpr int kKeys = 32;  // positions of a wave's block

__device__ __forceinline__ f32x4 mma16(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.b, b.b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.f[j], b.f[j], c, 0, 0, 0);
  return c;
}
// zeros that the compiler takes for unknown values (zero_acc, for four registers)
__device__ __forceinline__ f32x4 zero_acc4() {
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  asm volatile("" : "+v"(z));
  return z;
}

// 16 bytes of memory (said to be memory, for a generic address would be waited for as an LDS read too)
__device__ __forceinline__ uint4 load16(const void* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = *(const __attribute__((address_space(1))) u32x4*)(p);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// Orders a wave's LDS accesses of different lanes (no instruction: a wave's are carried out in order).
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// Over the four lanes that hold one query head (16 and 32 apart).
__device__ __forceinline__ float max_of_4(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_of_4(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

__device__ __forceinline__ int length_of(const PagedArgs& a, int b) { return min(max(a.lengths[b], 0), a.capacity); }

// Which part of which sequence workgroup `index` of a key head's tile has: a step is `keys` positions, and
// a sequence of n steps has ceil(n / quota) parts, one at least.  quota: so many steps that all parts
// fit `slots` (where there are sequences enough to fill the chip anyway, slots is more than it holds).
// All lanes of a wave take part; b < 0: no part is left for this workgroup.
struct Part {
  int b, split, splits, per, steps;
  int before;              // parts of the sequences before it
};
__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int w = 1; w < 64; w <<= 1) v += __shfl_xor(v, w, 64);
  return v;
}
__device__ __forceinline__ Part parts_of(const PagedArgs& a, int index, int keys) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int n = 0;
    if (b0 + lane < a.B) n = (length_of(a, b0 + lane) + keys - 1) / keys;
    total += wave_sum(n);
  }
  const int quota = max(1, static_cast<int>((total + a.slots - 1) / a.slots));
  Part p = {-1, 0, 1, quota, 0, 0};
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int n = 0, mine = 0;
    if (b0 + lane < a.B) {
      n = (length_of(a, b0 + lane) + keys - 1) / keys;
      mine = max(1, (n + quota - 1) / quota);
    }
    int upto = mine;       // parts of this chunk's sequences up to this one
#pragma unroll
    for (int w = 1; w < 64; w <<= 1) {
      const int v = __shfl_up(upto, w, 64);
      if (lane >= w) upto += v;
    }
    const int at = index - before;
    const uint64_t hit = __ballot(at < upto && at >= upto - mine && mine > 0);
    if (hit != 0) {
      const int who = __builtin_ctzll(hit);
      const int end = __builtin_amdgcn_readlane(upto, who), have = __builtin_amdgcn_readlane(mine, who);
      p.b = b0 + who;
      p.splits = have;
      p.split = at - (end - have);
      p.steps = __builtin_amdgcn_readlane(n, who);
      p.before = before + end - have;
      return p;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return p;
}

__device__ uint4 paged_zero_row[32];   // what positions without a row read: 512 bytes, a row of 128 fp32

template <typename T, int DP, int W, bool VEC>
__global__ __launch_bounds__(64 * W) void paged_kernel(PagedArgs a) {
  constexpr int DT = DP / 16, KS = DP / 32, VPR = DP * static_cast<int>(sizeof(T)) / 16, VL = kKeys * VPR / 64, KV = Elem<T>::kVec;
  constexpr int OST = 20;                                        // row of the join's tile of 16 rows x 16, padded
  constexpr int kLds = W * kKeys * DP * static_cast<int>(sizeof(T)), kJoin = (W * 16 * OST + 2 * W * 16) * 4;
  __shared__ __attribute__((aligned(16))) unsigned char smem[kLds > kJoin ? kLds : kJoin];
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, quad = lane >> 4,
            wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t at = a.first + blockIdx.x;
  const int heads = a.Hkv * a.tiles, ht = static_cast<int>(at % heads), hk = ht / a.tiles, tile = ht % a.tiles;
  const Part part = parts_of(a, static_cast<int>(at / heads), kKeys * W);
  if (part.b < 0) return;
  const int length = length_of(a, part.b);
  const int s0 = part.split * part.per, s1 = min(part.steps, s0 + part.per);
  T* const lds = reinterpret_cast<T*>(smem) + wave * kKeys * DP;
  const int32_t* table = a.table + part.b * a.ts;
  const T* const kp = static_cast<const T*>(a.k) + hk * a.ks[2];
  const T* const vp = static_cast<const T*>(a.v) + hk * a.vs[2];

  // the query head of this lane's column
  const int row = tile * 16 + col;
  const bool live = row < a.g;
  Frag<T> qf[KS];
  {
    const T* qp = static_cast<const T*>(a.q) + part.b * a.qs[0] + (hk * a.g + (live ? row : 0)) * a.qs[1];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int h = 0; h < 8 / KV; ++h) {
        const uint4 u = load_vec<T, VEC>(qp, 0, 32 * i + 8 * quad + KV * h, a.D, live).u;
        __builtin_memcpy(reinterpret_cast<char*>(&qf[i]) + 16 * h, &u, 16);
      }
  }

  // Block i of this wave: positions (s0 + i) * 32 W + 32 wave ...  Lane j < 32 (and j + 32) holds the page of position j.
  const auto entry = [&](int step) {
    const int key = (step * W + wave) * kKeys + (lane & 31);
    return step < s1 && key < length ? table[key / a.page_size] : -1;
  };
  Frag<T> kf[2][KS];
  Vec16<T> vf[VL];
  uint32_t kept = 0;   // of the block in kf, vf: positions that count
  const T* const zeros = reinterpret_cast<const T*>(paged_zero_row);
  const auto fetch = [&](int step, int page) {
    const int k0 = (step * W + wave) * kKeys, key = k0 + (lane & 31);
    const bool in = page >= 0 && page < a.num_pages;     // (an entry is only read for positions that exist)
    kept = static_cast<uint32_t>(__ballot(in));
    const int place = key - key / a.page_size * a.page_size;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = 16 * t + col, pg = __shfl(page, j, 64), pl = __shfl(place, j, 64);
      const bool ok = (kept >> j) & 1u;
      const T* r = kp + (ok ? pg * a.ks[0] + pl * a.ks[1] : 0);
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int h = 0; h < 8 / KV; ++h) {
          const int d = 32 * i + 8 * quad + KV * h;
          uint4 u;
          if (VEC) u = load16(ok && d < a.D ? r + d : zeros);
          else u = load_vec<T, false>(r, 0, d, a.D, ok).u;
          __builtin_memcpy(reinterpret_cast<char*>(&kf[t][i]) + 16 * h, &u, 16);
        }
    }
#pragma unroll
    for (int n = 0; n < VL; ++n) {
      const int j = (n * 64 + lane) / VPR, d = (n * 64 + lane) % VPR * KV, pg = __shfl(page, j, 64), pl = __shfl(place, j, 64);
      const bool ok = (kept >> j) & 1u;
      const T* r = vp + (ok ? pg * a.vs[0] + pl * a.vs[1] : 0);
      if (VEC) vf[n].u = load16(ok && d < a.D ? r + d : zeros);
      else vf[n] = load_vec<T, false>(r, 0, d, a.D, ok);
    }
  };

  f32x4 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc4();
  float m = kNegInf, l = 0.f;
  int next = entry(s0);
  fetch(s0, next);
  next = entry(s0 + 1);
  for (int step = s0; step < s1; ++step) {
    // this block's scores; its values move to the LDS
    f32x4 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t] = zero_acc4();
#pragma unroll
      for (int i = 0; i < KS; ++i) s[t] = mma16(kf[t][i], qf[i], s[t]);
    }
    wave_order();            // the last block's values have been read
#pragma unroll
    for (int n = 0; n < VL; ++n) {
      const int j = (n * 64 + lane) / VPR, d = (n * 64 + lane) % VPR * KV;
      *reinterpret_cast<uint4*>(lds + Tile<T, DP>::at(j, d)) = vf[n].u;
    }
    wave_order();
    const uint32_t word = kept;
    if (step + 1 < s1) fetch(step + 1, next);
    next = entry(step + 2);
    if (word != 0) {
      float mt = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (!((word >> (16 * t + 4 * quad + r)) & 1u)) s[t][r] = kNegInf;
          mt = fmaxf(mt, s[t][r]);
        }
      mt = max_of_4(mt) * a.c;
      if (__any(mt > m + 8.f)) {     // any m serves: raised only when scores exceed it by 2^8
        const float mn = fmaxf(m, mt), alpha = m == kNegInf ? 0.f : exp2_fast(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[i][r] *= alpha;
      }
      const float ms = m == kNegInf ? 0.f : m;
      float p[8];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p[4 * t + r] = exp2_fast(fmaf(s[t][r], a.c, -ms));
          l += p[4 * t + r];
        }
      if constexpr (sizeof(T) == 2) {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        Frag<T> pf;
#pragma unroll
        for (int j = 0; j < 4; ++j) pf.w[j] = pack_bf16(p[2 * j], p[2 * j + 1]);
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          Frag<T> vt;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            vt.s[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(lds + Tile<T, DP>::at(16 * t + 4 * quad + (col >> 2), 16 * i + 4 * (col & 3))));
          o[i] = mma16(vt, pf, o[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              o[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(lds[Tile<T, DP>::at(16 * t + 4 * quad + r, 16 * i + col)],
                                                          p[4 * t + r], o[i], 0, 0, 0);
      }
    }
  }
  l = sum_of_4(l);

  // the waves' parts of the 16 rows, 16 elements of the head at a time
  float* const os = reinterpret_cast<float*>(smem);              // [W][16][OST]
  float* const fs = os + W * 16 * OST;                           // [W][16] maxima
  float* const ls = fs + W * 16;                                 // [W][16] sums
  __syncthreads();
  if (quad == 0) {
    fs[wave * 16 + col] = m;
    ls[wave * 16 + col] = l;
  }
  const int rr = (tid & 63) / 4, d0 = (tid & 3) * 4, to = tile * 16 + rr, head = hk * a.g + to;
  const bool writes = tid < 64 && to < a.g;
  float f[W], mm = kNegInf, ll = 0.f, inv = 1.f;
  // parts are numbered by head tile, then along the tile's workgroups
  const int64_t prow = (static_cast<int64_t>(ht) * a.grid + part.before + part.split) * 16 + rr;
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    if (i > 0) __syncthreads();
    *reinterpret_cast<float4*>(os + (wave * 16 + col) * OST + 4 * quad) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
    __syncthreads();
    if (!writes) continue;
    if (i == 0) {
#pragma unroll
      for (int j = 0; j < W; ++j) mm = fmaxf(mm, fs[j * 16 + rr]);
      const float ms = mm == kNegInf ? 0.f : mm;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        f[j] = exp2_fast(fs[j * 16 + rr] - ms);
        ll = fmaf(f[j], ls[j * 16 + rr], ll);
      }
      if (part.splits > 1) {
        if (d0 == 0) *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(mm, ll);
      } else {
        inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);      // no position: zeros; a NaN sum stays NaN
        if (d0 == 0 && a.lse != nullptr)
          a.lse[static_cast<int64_t>(part.b) * a.Hq + head] = ll == 0.f ? kNegInf : fmaf(ms, kLn2, logf(ll));
      }
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(os + (j * 16 + rr) * OST + d0);
      acc.x = fmaf(f[j], v.x, acc.x);
      acc.y = fmaf(f[j], v.y, acc.y);
      acc.z = fmaf(f[j], v.z, acc.z);
      acc.w = fmaf(f[j], v.w, acc.w);
    }
    if (part.splits > 1) {
      *reinterpret_cast<float4*>(a.part + prow * DP + 16 * i + d0) = acc;
    } else {
      T* op = static_cast<T*>(a.out) + (static_cast<int64_t>(part.b) * a.Hq + head) * a.D;
      const float vals[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (16 * i + d0 + j < a.D) op[16 * i + d0 + j] = narrow<T>(vals[j]);
    }
  }
}

// Adds the parts of a sequence that was split: one workgroup for each sequence and query head; 8 threads of
// every 4 elements (16, 32 for smaller heads) take its parts in turn.
template <typename T, int DP>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedArgs a, int keys) {
  constexpr int V4 = DP / 4, S = 256 / V4;
  __shared__ float4 acc_of[S][V4 + 1];
  __shared__ float2 ml_of[S];
  const int64_t at = a.first + blockIdx.x;
  const int b = static_cast<int>(at / a.Hq), head = static_cast<int>(at % a.Hq), hk = head / a.g, row = head % a.g,
            tile = row / 16, rr = row % 16;
  // the same division into parts as the first launch's: this sequence's first part
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 64) {
    int n = 0;
    if (b0 + lane < a.B) n = (length_of(a, b0 + lane) + keys - 1) / keys;
    total += wave_sum(n);
  }
  const int quota = max(1, static_cast<int>((total + a.slots - 1) / a.slots));
  int before = 0;
  for (int b0 = 0; b0 < b; b0 += 64) {
    int mine = 0;
    if (b0 + lane < b) mine = max(1, ((length_of(a, b0 + lane) + keys - 1) / keys + quota - 1) / quota);
    before += wave_sum(mine);
  }
  const int steps = (length_of(a, b) + keys - 1) / keys, splits = max(1, (steps + quota - 1) / quota);
  if (splits == 1) return;
  const int64_t p0 = ((static_cast<int64_t>(hk) * a.tiles + tile) * a.grid + before) * 16 + rr;
  const int d = threadIdx.x % V4, k = threadIdx.x / V4;
  float m = kNegInf, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = k; s < splits; s += S) {
    const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (p0 + static_cast<int64_t>(s) * 16) * 2);
    const float4 v = *reinterpret_cast<const float4*>(a.part + (p0 + static_cast<int64_t>(s) * 16) * DP + d * 4);
    const float mn = fmaxf(m, x.x), ms = mn == kNegInf ? 0.f : mn, fa = exp2_fast(m - ms), fb = exp2_fast(x.x - ms);
    m = mn;
    l = fmaf(fb, x.y, fa * l);
    acc.x = fmaf(fb, v.x, fa * acc.x);
    acc.y = fmaf(fb, v.y, fa * acc.y);
    acc.z = fmaf(fb, v.z, fa * acc.z);
    acc.w = fmaf(fb, v.w, fa * acc.w);
  }
  acc_of[k][d] = acc;
  if (d == 0) ml_of[k] = make_float2(m, l);
  __syncthreads();
  if (k != 0) return;
  float mm = kNegInf, ll = 0.f;
  for (int s = 0; s < S; ++s) mm = fmaxf(mm, ml_of[s].x);
  const float ms = mm == kNegInf ? 0.f : mm;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < S; ++s) {
    const float f = exp2_fast(ml_of[s].x - ms);
    const float4 v = acc_of[s][d];
    ll = fmaf(f, ml_of[s].y, ll);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
  T* op = static_cast<T*>(a.out) + (static_cast<int64_t>(b) * a.Hq + head) * a.D;
  const float vals[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (4 * d + j < a.D) op[4 * d + j] = narrow<T>(vals[j]);
  if (d == 0 && a.lse != nullptr)
    a.lse[static_cast<int64_t>(b) * a.Hq + head] = ll == 0.f ? kNegInf : fmaf(ms, kLn2, logf(ll));
}

// ---- host side

int check(const dcn_paged_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  if (d->batch < 0 || d->query_heads < 1 || d->key_heads < 1 || d->head_dim < 1 || d->query_heads % d->key_heads != 0 ||
      d->num_pages < 0 || d->page_size < 1 || d->max_pages < 0 || d->table_stride < 0 || !std::isfinite(d->scale) ||
      !(d->scale > 0.f) || d->q_stride[0] < 0 || d->q_stride[1] < 0)
    return DCN_E_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->key_page_stride[i] < 0 || d->value_page_stride[i] < 0) return DCN_E_ARG;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  const double big = 2147483647.;
  if (d->head_dim > 128 || static_cast<double>(d->batch) * d->query_heads > big / 16 || d->num_pages > big ||
      d->page_size > big || static_cast<double>(d->max_pages) * d->page_size > big - 65536)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

// Waves of a workgroup, and positions of a step of it.
constexpr int waves_for(int es, int dp) { return es == 4 && dp == 128 ? 4 : 8; }

struct PagedPlan {
  int dp, waves, tiles, slots, grid;
};
PagedPlan plan_of(const dcn_paged_desc* d) {
  PagedPlan p{};
  p.dp = padded_head(d->head_dim);
  p.waves = waves_for(d->dtype == DCN_BF16 ? 2 : 4, p.dp);
  const int64_t g = d->query_heads / d->key_heads, capacity = d->max_pages * d->page_size;
  p.tiles = static_cast<int>((g + 15) / 16);
  // two workgroups a CU; all parts of a key head's tile fit where sequences are fewer than half of them
  const int64_t room = std::max<int64_t>(1, 2 * kCUs / (d->key_heads * p.tiles));
  p.slots = static_cast<int>(d->batch <= room / 2 ? room - d->batch : 4 * room);
  // ceil(n / quota) parts of each sequence: below slots + batch in all
  const int64_t steps = (capacity + kKeys * p.waves - 1) / (kKeys * p.waves);
  p.grid = static_cast<int>(std::min<int64_t>(p.slots + d->batch, d->batch * std::max<int64_t>(1, steps)));
  return p;
}
size_t workspace_of(const dcn_paged_desc* d, const PagedPlan& p, size_t* ml_at) {
  *ml_at = 0;
  if (p.grid <= d->batch) return 0;     // no sequence can have two parts
  const size_t rows = static_cast<size_t>(d->key_heads) * p.tiles * p.grid * 16;
  *ml_at = rows * p.dp * 4;
  return (*ml_at + rows * 8 + 255) / 256 * 256;
}

template <typename T, int DP>
const void* paged_fn(bool vec) {
  return vec ? reinterpret_cast<const void*>(&paged_kernel<T, DP, waves_for(sizeof(T), DP), true>)
             : reinterpret_cast<const void*>(&paged_kernel<T, DP, waves_for(sizeof(T), DP), false>);
}
template <typename T>
const void* paged_fn(int dp, bool vec) {
  return dp == 32 ? paged_fn<T, 32>(vec) : dp == 64 ? paged_fn<T, 64>(vec) : paged_fn<T, 128>(vec);
}
template <typename T>
const void* join_fn(int dp) {
  return dp == 32   ? reinterpret_cast<const void*>(&paged_join_kernel<T, 32>)
         : dp == 64 ? reinterpret_cast<const void*>(&paged_join_kernel<T, 64>)
                    : reinterpret_cast<const void*>(&paged_join_kernel<T, 128>);
}
bool launch_paged(const void* fn, int64_t n, int threads, void** args, PagedArgs* a, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 21;   // a dispatch counts its threads in 32 bits
  for (int64_t first = 0; first < n; first += kMost) {
    a->first = first;
    const int64_t now = n - first < kMost ? n - first : kMost;
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(now)), dim3(threads), args, 0, stream) != hipSuccess) return false;
  }
  return true;
}

bool vec_rows(const void* p, const int64_t* s, int n, int64_t D, int es) {
  const int64_t v = 16 / es;
  bool ok = reinterpret_cast<uintptr_t>(p) % 16 == 0 && D % v == 0;
  for (int i = 0; i < n; ++i) ok = ok && s[i] % v == 0;
  return ok;
}

}  // namespace
}  // namespace attn
}  // namespace dcn

extern "C" int dcn_paged_attention_workspace_bytes(const dcn_paged_desc* d, size_t* bytes) {
  using namespace dcn::attn;
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  size_t at;
  *bytes = d->batch == 0 ? 0 : workspace_of(d, plan_of(d), &at);
  return DCN_OK;
}

extern "C" int dcn_paged_attention(const dcn_paged_desc* d, const void* q, const void* key_pages,
                                   const void* value_pages, const int32_t* page_table, const int32_t* lengths,
                                   void* out, float* lse, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  using namespace dcn::attn;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0) return DCN_OK;
  const bool cache = d->num_pages > 0 && d->max_pages > 0;
  if (q == nullptr || out == nullptr || lengths == nullptr ||
      (cache && (key_pages == nullptr || value_pages == nullptr || page_table == nullptr)))
    return DCN_E_ARG;
  const PagedPlan p = plan_of(d);
  size_t ml_at;
  const size_t need = workspace_of(d, p, &ml_at);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return DCN_E_WORKSPACE;
  PagedArgs a{};
  a.q = q;
  a.k = key_pages;
  a.v = value_pages;
  a.table = page_table;
  a.lengths = lengths;
  a.out = out;
  a.lse = lse;
  if (need > 0) {
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + ml_at);
  }
  for (int i = 0; i < 2; ++i) a.qs[i] = d->q_stride[i];
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = d->key_page_stride[i];
    a.vs[i] = d->value_page_stride[i];
  }
  a.ts = d->table_stride;
  a.B = static_cast<int>(d->batch);
  a.Hq = static_cast<int>(d->query_heads);
  a.Hkv = static_cast<int>(d->key_heads);
  a.g = a.Hq / a.Hkv;
  a.D = static_cast<int>(d->head_dim);
  a.tiles = p.tiles;
  a.num_pages = static_cast<int>(d->num_pages);
  a.page_size = static_cast<int>(d->page_size);
  a.capacity = cache ? static_cast<int>(d->max_pages * d->page_size) : 0;
  a.slots = p.slots;
  a.grid = p.grid;
  a.c = d->scale * kLog2e;
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const bool vec = vec_rows(q, d->q_stride, 2, d->head_dim, es) && vec_rows(key_pages, d->key_page_stride, 3, d->head_dim, es) &&
                   vec_rows(value_pages, d->value_page_stride, 3, d->head_dim, es);
  void* args[] = {&a};
  if (!launch_paged(bf16 ? paged_fn<uint16_t>(p.dp, vec) : paged_fn<float>(p.dp, vec),
                    static_cast<int64_t>(p.grid) * a.Hkv * a.tiles, 64 * p.waves, args, &a, stream))
    return DCN_E_HIP;
  if (need > 0) {
    int keys = kKeys * p.waves;
    void* join_args[] = {&a, &keys};
    if (!launch_paged(bf16 ? join_fn<uint16_t>(p.dp) : join_fn<float>(p.dp), static_cast<int64_t>(a.B) * a.Hq, 256,
                      join_args, &a, stream))
      return DCN_E_HIP;
  }
  return DCN_OK;
}

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
// that a page's look-up is never waited for in line.  Pages of any size: each position has its own address,
// formed by one lane and handed to the lanes that load its row through the LDS.
//
// Lengths are known on the device only, so every workgroup derives from them which part it has (share_of; of many
// sequences a launch of its own does): the blocks of all sequences are dealt out evenly over as many workgroups as the
// chip holds.  A sequence of one part is written as it is; others leave their parts (maximum, sum, undivided output),
// which paged_join_kernel adds in order.
//
// Memory bounds long sequences: eight of 4200 to 16800 positions, 16 heads of 128 on 4, bf16, take 34.8 us for 166 MB,
// 4.8 TB/s (a large copy 4.99), and the join 4.8; 16 of up to 4200, 8 heads of 127 on 4 in vectors that are moved,
// 33.8 us in all for 93 MB.  A short one is a chain: 1050 positions, 8 heads of 64, 10.3 us in 8 workgroups, three
// blocks for each wave one after the other; in fp32 13 sequences to 2777, 6 heads of 40 on 3, 8.4 us (and the join 3.9)
// for 5.5 MB: the division, a look-up and one or two blocks for each wave.
//
// Arithmetic: as dcn_attention.hip, but for bf16 the weights enter the second product as three operands, which hold all
// of their 24 bits: the matrix units wait for memory here, and the output is then that of fp32 weights, rounded once.

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
  float* part;             // [key head's tile][slot][16][DP]: parts of sequences that have several,
  float* part_ml;          // [..][16][2]
  int4 *shares, *joins;    // of many sequences: paged_shares_kernel's lists (else null)
  int64_t qs[2], ks[3], vs[3], ts;
  int B, Hq, Hkv, g, D;
  int columns, tail, back; // of the output (see Rows): D, D and 0 where no vector is moved
  int tiles;               // of 16 rows, of a key head
  int num_pages, page_size, max_pages, capacity;
  int split;               // whether sequences may have several parts
  int aim;                 // parts of a key head's tile that the division aims at,
  int least;               // of so many blocks at least
  int grid, slots;         // workgroups of a key head's tile (the most parts that there can be); slots
  uint32_t first;          // workgroups of launches before this one
  uint32_t page_m;         // position / page_size is the upper half of position * page_m, shifted by page_s
  int page_s;              // (page_m 0: pages of one position)
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

// 16 bytes of memory, which takes them wherever an element may start (said to be memory, for a generic address would
// be waited for as an LDS read too)
__device__ __forceinline__ uint4 load16(const void* p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
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

// ---- which workgroup has what

__device__ __forceinline__ int length_of(const PagedArgs& a, int b) { return min(max(a.lengths[b], 0), a.capacity); }
__device__ __forceinline__ int blocks_of(const PagedArgs& a, int b) { return (length_of(a, b) + kKeys - 1) / kKeys; }
// of sequence `lane` (0 where there is none)
__device__ __forceinline__ int blocks_of_lane(const PagedArgs& a) {
  const int b = threadIdx.x & 63;
  return b < a.B ? blocks_of(a, b) : 0;
}
__device__ __forceinline__ int parts_of(int blocks, int quota) { return max(1, (blocks + quota - 1) / quota); }

// sums of the lanes up to each one
template <int CTRL, int ROWS>
__device__ __forceinline__ int from_lane(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, ROWS == 0xf);
}
__device__ __forceinline__ int running_sum(int v) {
  v += from_lane<0x111, 0xf>(v);     // 1, 2, 4, 8 lanes below, within 16
  v += from_lane<0x112, 0xf>(v);
  v += from_lane<0x114, 0xf>(v);
  v += from_lane<0x118, 0xf>(v);
  v += from_lane<0x142, 0xa>(v);     // the last lane of the 16 below
  v += from_lane<0x143, 0xc>(v);     // of the 32 below
  return v;
}
__device__ __forceinline__ int lanes_total(int v) { return __builtin_amdgcn_readlane(running_sum(v), 63); }

// Up to kLanes sequences: one for each lane, and every workgroup of both launches finds its part on its own.
constexpr int kLanes = 64;

// Blocks of a part: the fewest with which all sequences together have at most `aim` parts (aim is at least
// as many as there are sequences, so the search ends: it grows until one part holds the longest).  mine:
// blocks_of_lane.
__device__ __forceinline__ int quota_of(const PagedArgs& a, int mine) {
  // (as near as the search's first guess needs; in two sums, for 64 of 2^26 blocks pass 32 bits)
  const float total = static_cast<float>(lanes_total(mine >> 8)) * 256.f + static_cast<float>(lanes_total(mine & 255));
  int quota = max(a.least, static_cast<int>(total / static_cast<float>(a.aim)));
  while (lanes_total(static_cast<int>(threadIdx.x & 63) < a.B ? parts_of(mine, quota) : 0) > a.aim) quota += max(1, quota / 16);
  return quota;
}

// The part of workgroup `index` of a key head's tile: blocks first .. last - 1 of sequence b, in slot `slot` where the
// sequence has several parts (-1: it has one).  b < 0: no part is left for this workgroup.
struct Share {
  int b, first, last, slot;
};
__device__ __forceinline__ Share share_of(const PagedArgs& a, int index) {
  if (a.split == 0) return {index, 0, blocks_of(a, index), -1};
  if (a.shares != nullptr) {
    const int4 e = a.shares[index];
    return {e.x, e.y, e.z, e.w};
  }
  const int lane = threadIdx.x & 63, mine = blocks_of_lane(a), quota = quota_of(a, mine),
            parts = lane < a.B ? parts_of(mine, quota) : 0, upto = running_sum(parts);
  const uint64_t hit = __ballot(index < upto && index >= upto - parts);
  if (hit == 0) return {-1, 0, 0, -1};
  const int who = __builtin_ctzll(hit), blocks = __builtin_amdgcn_readlane(mine, who),
            have = __builtin_amdgcn_readlane(parts, who), part = index - (__builtin_amdgcn_readlane(upto, who) - have);
  const int first = part * quota;
  return {who, first, min(blocks, first + quota), have > 1 ? index : -1};
}

// More sequences: one workgroup makes lists first, for a search over all of them in every workgroup takes longer than its
// part (8 heads of 64, lengths to 4096: 512 sequences 762 us, from the lists 465, a copy of the bytes 434; 2048 sequences
// 7217, 1723 and 1767).  With a quota of total / (aim - B) blocks at least, the parts beyond one of each sequence
// are at most aim - B, sequences with several fewer than that, and their parts fewer than twice that.
__global__ __launch_bounds__(1024) void paged_shares_kernel(PagedArgs a) {
  __shared__ int64_t totals[16];
  __shared__ int sums[3][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, spare = a.aim - a.B;
  const int64_t per = (static_cast<int64_t>(a.B) + 1023) / 1024;      // a thread has as many sequences, side by side
  const int b0 = static_cast<int>(min<int64_t>(a.B, tid * per)), b1 = static_cast<int>(min<int64_t>(a.B, (tid + 1) * per));
  int64_t total = 0;
  for (int b = b0; b < b1; ++b) total += blocks_of(a, b);
#pragma unroll
  for (int n = 32; n > 0; n /= 2) total += __shfl_xor(total, n, 64);
  if (lane == 0) totals[wave] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < 16; ++w) total += totals[w];
  const int quota = static_cast<int>(min<int64_t>(max<int64_t>(a.least, (total + spare - 1) / spare), 0x7fffffff));
  int have[3] = {0, 0, 0};       // parts, sequences with several, slots
  for (int b = b0; b < b1; ++b) {
    const int n = blocks_of(a, b), parts = n > quota ? (n - 1) / quota + 1 : 1;
    have[0] += parts;
    if (parts > 1) {
      ++have[1];
      have[2] += parts;
    }
  }
  int before[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int upto = running_sum(have[i]);
    before[i] = upto - have[i];
    if (lane == 63) sums[i][wave] = upto;
  }
  __syncthreads();
  int all[2] = {0, 0};
  for (int w = 0; w < 16; ++w) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (w < wave) before[i] += sums[i][w];
      if (i < 2) all[i] += sums[i][w];
    }
  }
  for (int b = b0; b < b1; ++b) {
    const int n = blocks_of(a, b), parts = n > quota ? (n - 1) / quota + 1 : 1;
    if (parts > 1) a.joins[before[1]++] = make_int4(b, before[2], parts, 0);
    for (int k = 0; k < parts; ++k)
      a.shares[before[0]++] = make_int4(b, k * quota, min(n, (k + 1) * quota), parts > 1 ? before[2]++ : -1);
  }
  for (int i = all[0] + tid; i < a.grid; i += 1024) a.shares[i] = make_int4(-1, 0, 0, -1);
  for (int i = all[1] + tid; i < spare; i += 1024) a.joins[i] = make_int4(-1, 0, 0, 0);
}

__device__ uint4 paged_zero_row[32];   // what positions without a row read: 512 bytes, a row of 128 fp32

// The first `back` elements of the 16 bytes that start at element `tail` of a fragment (of 8; elsewhere none) become 0.
__device__ __forceinline__ void clear_first(Frag<uint16_t>& f, int tail, int back) {
#pragma unroll
  for (int w = 0; w < 4; ++w) f.w[w] &= tail != 0 || 2 * w >= back ? ~0u : 2 * w + 1 >= back ? 0xffff0000u : 0u;
}
__device__ __forceinline__ void clear_first(Frag<float>& f, int tail, int back) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (tail == e / 4 * 4 && e % 4 < back) f.f[e] = 0.f;
}

// How rows are read: 16 bytes at a time all the padded head's width; 16 bytes at a time where the head has them; heads
// of another size the same, with the last 16 bytes moved back to end with the row; or (heads below 16 bytes) element by
// element.  What the moved vector shares with the one before it is left out of the scores, and comes twice, alike, in
// the output, whose columns from `tail` on are those of the row `back` elements before.
enum Rows { kWhole, kVectors, kEnds, kElements };
__device__ __forceinline__ void put(const PagedArgs& a, uint16_t* row, int c, float v) {
  if (c < a.columns) row[c - (c >= a.tail ? a.back : 0)] = narrow<uint16_t>(v);
}
__device__ __forceinline__ void put(const PagedArgs& a, float* row, int c, float v) {
  if (c < a.columns) row[c - (c >= a.tail ? a.back : 0)] = v;
}

template <typename T, int DP, int W, Rows ROWS>
__global__ __launch_bounds__(64 * W) void paged_kernel(PagedArgs a) {
  constexpr int DT = DP / 16, KS = DP / 32, VPR = DP * static_cast<int>(sizeof(T)) / 16, VL = kKeys * VPR / 64, KV = Elem<T>::kVec;
  constexpr int CD = DT / 2;                                     // columns of 16 elements that are joined at a time
  constexpr int OST = 20;                                        // row of the join's tile of 16 rows x 16, padded
  constexpr int kLds = W * kKeys * DP * static_cast<int>(sizeof(T)), kJoin = (CD * W * 16 * OST + 2 * W * 16) * 4;
  __shared__ __attribute__((aligned(16))) unsigned char smem[kLds > kJoin ? kLds : kJoin];
  __shared__ ulonglong2 rows[W][kKeys];                          // addresses of a block's keys and values
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, quad = lane >> 4,
            wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t at = a.first + blockIdx.x, heads = a.Hkv * a.tiles, index = at / heads, ht = at - index * heads;
  const int hk = ht / a.tiles, tile = ht - hk * a.tiles;
  const Share part = share_of(a, index);
  if (part.b < 0) return;
  const int length = length_of(a, part.b);
  T* const lds = reinterpret_cast<T*>(smem) + wave * kKeys * DP;
  const int32_t* table = a.table + part.b * a.ts;
  const T* const kp = static_cast<const T*>(a.k) + hk * a.ks[2];
  const T* const vp = static_cast<const T*>(a.v) + hk * a.vs[2];

  // Where position `lane % 32` of a block lies: its page (-1: none) and its place there.
  struct Where {
    int page, place;
  };
  const auto entry = [&](int block) {
    const int key = block * kKeys + (lane & 31), n = a.page_m == 0 ? key : static_cast<int>(__umulhi(key, a.page_m) >> a.page_s);
    int page = -1;
    if (n < a.max_pages) page = table[n];      // (not held up by the length, which the first block's is fetched with)
    if (block >= part.last || key >= length) page = -1;
    return Where{page, key - n * a.page_size};
  };
  Where next = entry(part.first + wave);

  const T* const zeros = reinterpret_cast<const T*>(paged_zero_row);
  // 16 bytes of a row from element d on; zeros beyond D
  const auto take = [&](const T* r, int d) {
    if constexpr (ROWS == kWhole) return load16(r + d);
    if constexpr (ROWS == kVectors) return load16(d < a.D ? r + d : zeros);
    if constexpr (ROWS == kEnds) return load16(d < a.D ? r + min(d, a.D - KV) : zeros);
    return load_vec<T, false>(r, 0, d, a.D, true).u;
  };

  // of a fragment at element 32 i on: what a moved vector shares with the one before becomes 0 (infinities, too)
  const auto own = [&](Frag<T>& f, int i) {
    if constexpr (ROWS == kEnds) {
      if (i == a.tail / 32) clear_first(f, a.tail - 32 * i - 8 * quad, a.back);
    }
  };
  // the query head of this lane's column
  const int row = tile * 16 + col;
  const bool live = row < a.g;
  Frag<T> qf[KS];
  {
    const T* qp = live ? static_cast<const T*>(a.q) + part.b * a.qs[0] + (hk * a.g + row) * a.qs[1] : zeros;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int h = 0; h < 8 / KV; ++h) {
        const uint4 u = take(qp, 32 * i + 8 * quad + KV * h);
        __builtin_memcpy(reinterpret_cast<char*>(&qf[i]) + 16 * h, &u, 16);
      }
#pragma unroll
    for (int i = 0; i < KS; ++i) own(qf[i], i);
  }

  Frag<T> kf[2][KS];
  Vec16<T> vf[VL];
  uint32_t kept = 0;   // of the block in kf, vf: positions that count
  const auto fetch = [&](const Where& w) {
    const bool ok = w.page >= 0 && w.page < a.num_pages;
    kept = static_cast<uint32_t>(__ballot(ok));
    wave_order();
    if (lane < kKeys)
      rows[wave][lane] = make_ulonglong2(
          reinterpret_cast<uint64_t>(ok ? kp + w.page * a.ks[0] + w.place * a.ks[1] : zeros),
          reinterpret_cast<uint64_t>(ok ? vp + w.page * a.vs[0] + w.place * a.vs[1] : zeros));
    wave_order();
    const T *kr[2], *vr[VL];
#pragma unroll
    for (int t = 0; t < 2; ++t) kr[t] = reinterpret_cast<const T*>(rows[wave][16 * t + col].x);
#pragma unroll
    for (int n = 0; n < VL; ++n) vr[n] = reinterpret_cast<const T*>(rows[wave][(n * 64 + lane) / VPR].y);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int h = 0; h < 8 / KV; ++h) {
          const uint4 u = take(kr[t], 32 * i + 8 * quad + KV * h);
          __builtin_memcpy(reinterpret_cast<char*>(&kf[t][i]) + 16 * h, &u, 16);
        }
#pragma unroll
    for (int n = 0; n < VL; ++n) vf[n].u = take(vr[n], (n * 64 + lane) % VPR * KV);
  };

  f32x4 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc4();
  float m = kNegInf, l = 0.f;
  fetch(next);
  next = entry(part.first + wave + W);
  for (int block = part.first + wave; block < part.last; block += W) {
    // this block's scores; its values move to the LDS
    f32x4 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t] = zero_acc4();
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        own(kf[t][i], i);
        s[t] = mma16(kf[t][i], qf[i], s[t]);
      }
    }
    wave_order();            // the last block's values have been read
#pragma unroll
    for (int n = 0; n < VL; ++n) {
      const int j = (n * 64 + lane) / VPR, d = (n * 64 + lane) % VPR * KV;
      *reinterpret_cast<uint4*>(lds + Tile<T, DP>::at(j, d)) = vf[n].u;
    }
    wave_order();
    const uint32_t word = kept;
    if (block + W < part.last) fetch(next);
    next = entry(block + 2 * W);
    if (word != 0) {
      float mt = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (word != 0xffffffffu && !((word >> (16 * t + 4 * quad + r)) & 1u)) s[t][r] = kNegInf;
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
        // A weight as three operands, which together are the weight: each is the upper 16 bits of what the ones before
        // leave.  Where they leave nothing it is bf16's least number, 2^-133, for 0 would make an infinite value's
        // product NaN (of a weight of 0 all three are 0).
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        Frag<T> pf[3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float r0 = p[2 * j], r1 = p[2 * j + 1];
          u16x2 upper[3];
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            const uint32_t h0 = __float_as_uint(r0), h1 = __float_as_uint(r1);
            upper[n] = __builtin_bit_cast(u16x2, __builtin_amdgcn_perm(h1, h0, 0x07060302));
            r0 -= __uint_as_float(h0 & 0xffff0000u);
            r1 -= __uint_as_float(h1 & 0xffff0000u);
          }
          const u16x2 least = __builtin_elementwise_min(upper[0], u16x2{1, 1});
          pf[0].w[j] = __builtin_bit_cast(uint32_t, upper[0]);
#pragma unroll
          for (int n = 1; n < 3; ++n) pf[n].w[j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(upper[n], least));
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) {
          Frag<T> vt;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            vt.s[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(lds + Tile<T, DP>::at(16 * t + 4 * quad + (col >> 2), 16 * i + 4 * (col & 3))));
#pragma unroll
          for (int n = 0; n < 3; ++n) o[i] = mma16(vt, pf[n], o[i]);
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

  // the waves' parts of the 16 rows, CD columns of 16 elements of the head at a time: 64 threads for each column
  float* const os = reinterpret_cast<float*>(smem);              // [CD][W][16][OST]
  float* const fs = os + CD * W * 16 * OST;                      // [W][16] maxima
  float* const ls = fs + W * 16;                                 // [W][16] sums
  __syncthreads();
  if (quad == 0) {
    fs[wave * 16 + col] = m;
    ls[wave * 16 + col] = l;
  }
  const int rr = lane / 4, d0 = (lane & 3) * 4, to = tile * 16 + rr, head = hk * a.g + to;
  const bool writes = wave < CD && to < a.g;
  float f[W], mm = kNegInf, ll = 0.f, inv = 1.f;
  const int64_t prow = (static_cast<int64_t>(ht) * a.slots + part.slot) * 16 + rr;
#pragma unroll
  for (int i = 0; i < DT; i += CD) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int c = 0; c < CD; ++c)
      *reinterpret_cast<float4*>(os + ((c * W + wave) * 16 + col) * OST + 4 * quad) =
          make_float4(o[i + c][0], o[i + c][1], o[i + c][2], o[i + c][3]);
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
      const bool once = wave == 0 && d0 == 0;
      if (part.slot >= 0) {
        if (once) *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(mm, ll);
      } else {
        inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);      // no position: zeros; a NaN sum stays NaN
        if (once && a.lse != nullptr)
          a.lse[static_cast<int64_t>(part.b) * a.Hq + head] = ll == 0.f ? kNegInf : fmaf(ms, kLn2, logf(ll));
      }
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(os + ((wave * W + j) * 16 + rr) * OST + d0);
      acc.x = fmaf(f[j], v.x, acc.x);
      acc.y = fmaf(f[j], v.y, acc.y);
      acc.z = fmaf(f[j], v.z, acc.z);
      acc.w = fmaf(f[j], v.w, acc.w);
    }
    const int d = 16 * (i + wave) + d0;
    if (part.slot >= 0) {
      *reinterpret_cast<float4*>(a.part + prow * DP + d) = acc;
    } else {
      T* op = static_cast<T*>(a.out) + (static_cast<int64_t>(part.b) * a.Hq + head) * a.D;
      const float vals[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int j = 0; j < 4; ++j) put(a, op, d + j, vals[j]);
    }
  }
}

// Adds the parts of a sequence that was split: one workgroup for each such sequence (with up to kLanes of them, for
// each sequence) and query head; 8 threads of
// every 4 elements (16, 32 for smaller heads) take its parts in turn.
template <typename T, int DP>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedArgs a) {
  constexpr int V4 = DP / 4, S = 256 / V4;
  __shared__ float4 acc_of[S][V4 + 1];
  __shared__ float2 ml_of[S];
  const uint32_t at = a.first + blockIdx.x;
  const int number = at / a.Hq, head = at - number * a.Hq, hk = head / a.g, row = head % a.g, tile = row / 16, rr = row % 16;
  int b = number, splits, before;
  if (a.joins != nullptr) {
    const int4 e = a.joins[number];
    b = e.x;
    if (b < 0) return;
    before = e.y;
    splits = e.z;
  } else {       // the same division into parts as the first launch's: this sequence's first part
    const int lane = threadIdx.x & 63, mine = blocks_of_lane(a), quota = quota_of(a, mine),
              parts = lane < a.B ? parts_of(mine, quota) : 0;
    splits = __builtin_amdgcn_readlane(parts, b);
    if (splits == 1) return;
    before = __builtin_amdgcn_readlane(running_sum(parts), b) - splits;
  }
  const int64_t p0 = ((static_cast<int64_t>(hk) * a.tiles + tile) * a.slots + before) * 16 + rr;
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
  for (int j = 0; j < 4; ++j) put(a, op, 4 * d + j, vals[j]);
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

// Waves of a workgroup.  Wide: as many as the registers of a CU hold, for the shortest chain of blocks.  Narrow:
// half of that, so that one workgroup's start and end pass while another streams.
constexpr int waves_for(int es, int dp, bool wide) {
  return es == 2 ? (dp == 128 ? (wide ? 8 : 4) : wide ? 16 : 8) : dp == 128 ? 4 : wide ? 8 : 4;
}

struct PagedPlan {
  int dp, waves, tiles, aim, least, grid, slots;
  bool split, wide, rounds, listed;
};
// The division into parts.  A sequence has several only where its blocks may be more than kChain for each wave of a
// wide workgroup: below, the launch that joins them costs more than it saves (one sequence, 8 heads of 64:
// 1050 positions 10.3 us whole, 11.1 in parts; 2100 15.1 and 11.3).  Few sequences: one round of wide workgroups
// (16800 positions 15.3 us, of narrow ones 15.5; of 16 heads of 128 on 4, 16.2 and 16.5).  Many: kRounds rounds of
// narrow ones, in which their lengths even out, but of kLeast blocks for each wave at least (32 sequences to 4200, 8
// heads of 64, in one round 53 us, 47 in two or three; 64 to 2000, 4 of 128: 44.8 us with parts of one block, 41.4 of
// three, 54 of twelve).
constexpr int kChain = 3, kRounds = 3, kLeast = 3;
PagedPlan plan_of(const dcn_paged_desc* d) {
  PagedPlan p{};
  const int es = d->dtype == DCN_BF16 ? 2 : 4;
  p.dp = padded_head(d->head_dim);
  const int64_t g = d->query_heads / d->key_heads, blocks = (d->max_pages * d->page_size + kKeys - 1) / kKeys;
  p.tiles = static_cast<int>((g + 15) / 16);
  const int64_t heads = d->key_heads * p.tiles, groups = d->batch * heads;
  p.split = blocks > kChain * waves_for(es, p.dp, true);
  const int64_t room = std::max<int64_t>(1, kCUs / heads);     // parts of a key head's tile in one round of wide workgroups
  p.rounds = 4 * d->batch > room;
  p.wide = p.split ? !p.rounds : groups <= kCUs;
  p.waves = waves_for(es, p.dp, p.wide);
  p.aim = static_cast<int>(p.rounds ? d->batch + kRounds * 2 * room : room);
  p.least = (p.rounds ? kLeast : 1) * p.waves;
  p.grid = p.split ? p.aim : static_cast<int>(d->batch);
  p.listed = p.split && d->batch > kLanes;     // (these have rounds: aim is beyond the batch)
  p.slots = p.listed ? 2 * (p.aim - static_cast<int>(d->batch)) : p.aim;
  return p;
}
// The workspace: parts, their maxima and sums, the lists.
struct Layout {
  size_t ml, shares, joins, bytes;
};
Layout layout_of(const dcn_paged_desc* d, const PagedPlan& p) {
  Layout l{};
  if (!p.split) return l;
  const size_t rows = static_cast<size_t>(d->key_heads) * p.tiles * p.slots * 16;
  l.ml = rows * p.dp * 4;
  l.shares = l.joins = l.bytes = l.ml + rows * 8;
  if (p.listed) {
    l.joins = l.shares + static_cast<size_t>(p.grid) * sizeof(int4);
    l.bytes = l.joins + static_cast<size_t>(p.aim - d->batch) * sizeof(int4);
  }
  l.bytes = (l.bytes + 255) / 256 * 256;
  return l;
}

template <typename T, int DP, int W>
const void* paged_fn(Rows rows) {
  if constexpr (DP == 32)
    if (rows == kElements) return reinterpret_cast<const void*>(&paged_kernel<T, DP, W, kElements>);
  return rows == kWhole     ? reinterpret_cast<const void*>(&paged_kernel<T, DP, W, kWhole>)
         : rows == kVectors ? reinterpret_cast<const void*>(&paged_kernel<T, DP, W, kVectors>)
                            : reinterpret_cast<const void*>(&paged_kernel<T, DP, W, kEnds>);
}
template <typename T, int DP>
const void* paged_fn(bool wide, Rows rows) {
  return wide ? paged_fn<T, DP, waves_for(sizeof(T), DP, true)>(rows) : paged_fn<T, DP, waves_for(sizeof(T), DP, false)>(rows);
}
template <typename T>
const void* paged_fn(const PagedPlan& p, Rows rows) {
  return p.dp == 32 ? paged_fn<T, 32>(p.wide, rows) : p.dp == 64 ? paged_fn<T, 64>(p.wide, rows) : paged_fn<T, 128>(p.wide, rows);
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
    a->first = static_cast<uint32_t>(first);
    const int64_t now = n - first < kMost ? n - first : kMost;
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(now)), dim3(threads), args, 0, stream) != hipSuccess) return false;
  }
  return true;
}

}  // namespace
}  // namespace attn
}  // namespace dcn

extern "C" int dcn_paged_attention_workspace_bytes(const dcn_paged_desc* d, size_t* bytes) {
  using namespace dcn::attn;
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  *bytes = d->batch == 0 ? 0 : layout_of(d, plan_of(d)).bytes;
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
  const Layout l = layout_of(d, p);
  const size_t need = l.bytes;
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
    unsigned char* const w = static_cast<unsigned char*>(workspace);
    a.part = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float*>(w + l.ml);
    if (p.listed) {
      a.shares = reinterpret_cast<int4*>(w + l.shares);
      a.joins = reinterpret_cast<int4*>(w + l.joins);
    }
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
  a.max_pages = cache ? static_cast<int>(d->max_pages) : 0;
  a.capacity = cache ? static_cast<int>(d->max_pages * d->page_size) : 0;
  a.split = p.split;
  a.aim = p.aim;
  a.least = p.least;
  a.grid = p.grid;
  a.slots = p.slots;
  a.c = d->scale * kLog2e;
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const int kv = 16 / es;
  const Rows rows = a.D == p.dp ? kWhole : a.D % kv == 0 ? kVectors : a.D > kv ? kEnds : kElements;
  a.columns = a.tail = a.D;
  if (rows == kEnds) {
    a.tail = a.D / kv * kv;
    a.columns = a.tail + kv;
    a.back = a.columns - a.D;
  }
  if (d->page_size > 1) {
    // of positions below 2^31: with 2^s >= page_size, 2^(31 + s) / page_size rounded up is off by less than 2^-31 of it
    int s = 0;
    while ((int64_t{1} << s) < d->page_size) ++s;
    a.page_m = static_cast<uint32_t>(((uint64_t{1} << (31 + s)) + d->page_size - 1) / d->page_size);
    a.page_s = s - 1;
  }
  void* args[] = {&a};
  if (p.listed && !launch_paged(reinterpret_cast<const void*>(&paged_shares_kernel), 1, 1024, args, &a, stream)) return DCN_E_HIP;
  if (!launch_paged(bf16 ? paged_fn<uint16_t>(p, rows) : paged_fn<float>(p, rows),
                    static_cast<int64_t>(p.grid) * a.Hkv * a.tiles, 64 * p.waves, args, &a, stream))
    return DCN_E_HIP;
  if (p.split) {
    const int64_t several = p.listed ? p.aim - a.B : a.B;
    if (!launch_paged(bf16 ? join_fn<uint16_t>(p.dp) : join_fn<float>(p.dp), several * a.Hq, 256, args, &a, stream))
      return DCN_E_HIP;
  }
  return DCN_OK;
}

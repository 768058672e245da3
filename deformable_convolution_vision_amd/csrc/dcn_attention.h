// dcn_attention.h -- what the cross-attention kernels (dcn_attention.hip) and their
// gradients (dcn_attention_grad.hip) share: fragments, matrix products, tile loads, the
// argument block and the host-side checks.  Not part of the public ABI.
//
// Matrix products run on MFMA 32x32: 16 products deep for bf16, 2 deep for fp32.  With l
// a lane of the wave, half = l >> 5:
//   A operand   row l & 31 of a 32-row tile, elements k = 8*half .. 8*half+7 of a 16-wide step
//   B operand   column l & 31, the same elements
//   result      column l & 31, rows acc_row(r, half) for the 16 registers r
// fp32 keeps the same fragments of 8 elements and contracts them one at a time: the
// instruction's two elements are then k = j and 8 + j, an order both operands share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dcn.h"

namespace dcn {
namespace attn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

// How the tiles of all batch elements and key heads fall to workgroups.
struct Tiling {
  int tiles;
  int full;        // tiles below this one have a workgroup each; the inner loop of each of the others is
  int splits;      // split over this many workgroups,
  int per_split;   // of so many steps
};

struct Args {
  const void *q, *k, *v;
  const uint8_t* mask;         // [B][Lk] bytes, 0: the key is padding; or null
  void* out;                   // [B][Lq][Hq][D]
  float* lse;                  // [B][Hq][Lq] or null
  float* part;                 // split tiles' parts [tile][split][row][DP]: outputs not yet divided by their sums; dQ
  float* part_ml;              // forward: each row's maximum and sum, [tile][split][row][2]
  float* part_kv;              // parts of dK and dV [tile][split][2][key][DP]
  const void* dout;            // backward: [B][Lq][Hq][D]
  const float* delta;          // backward: [B][Hkv][R] lse in powers of two, then as many sum(dout * out)
  void *dq, *dk, *dv;
  int64_t qs[3], ks[3], vs[3]; // strides in elements: batch, position, head
  int64_t ms;                  // the mask's batch stride
  int B, Lq, Lk, Hq, Hkv, g, D;
  int R;                       // query rows of one key head: g * Lq, row r = position r / g, head r % g
  Tiling y, ykv;               // of the forward or dQ; of dK and dV
  int first;                   // workgroups of this kernel in launches before this one
  float c;                     // scale * log2(e): softmax runs in powers of two
  float scale;
};

__device__ __forceinline__ constexpr int acc_row(int r, int half) { return (r & 3) + 8 * (r >> 2) + 4 * half; }

// 16 bytes of a row: 8 bf16 or 4 fp32 elements
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
};

// 8 consecutive elements, one lane's share of an operand
template <typename T>
struct Frag;
template <>
struct Frag<uint16_t> {
  union {
    uint4 u;
    bf16x8 b;
    s16x4 s[2];
    uint32_t w[4];
  };
};
template <>
struct Frag<float> {
  union {
    float4 u[2];
    float f[8];
  };
};

__device__ __forceinline__ f32x16 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.b, b.b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(const Frag<float>& a, const Frag<float>& b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.f[j], b.f[j], c, 0, 0, 0);
  return c;
}

// Zeros that the compiler takes for unknown values.  A product whose accumulator it can prove
// zero takes the constant instead, and its result registers may then be placed over those of
// its operands, which has given wrong products; with these, kept in registers of their own
// for a kernel's whole time, a product of a new sum starts from them without writing zeros.
__device__ __forceinline__ f32x16 zero_acc() {
  f32x16 z;
#pragma unroll
  for (int r = 0; r < 16; ++r) z[r] = 0.f;
  asm volatile("" : "+v"(z));
  return z;
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Which of 64 blocks of 32 keys hold attended keys: lane i receives the mask bits of keys
// first + i * step .. + 31 as one word (0 beyond `end`); mp null: every key below Lk counts.
__device__ __forceinline__ uint32_t key_words(const uint8_t* mp, int64_t first, int64_t step, int64_t end, int Lk) {
  const int64_t k0 = first + (threadIdx.x & 63) * step;
  if (k0 >= end || k0 >= Lk) return 0;
  const int n = static_cast<int>(min(static_cast<int64_t>(32), Lk - k0));
  uint32_t word = n == 32 ? 0xffffffffu : (1u << n) - 1u;
  if (mp == nullptr) return word;
  uint32_t kept = 0;
  if (n == 32) {
    uint32_t w[8];
    __builtin_memcpy(w, mp + k0, 32);
#pragma unroll
    for (int i = 0; i < 32; ++i) kept |= ((w[i / 4] >> (8 * (i % 4))) & 0xffu) != 0 ? 1u << i : 0u;
  } else {
    for (int i = 0; i < n; ++i) kept |= mp[k0 + i] != 0 ? 1u << i : 0u;
  }
  return word & kept;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));   // nearest even
}

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  return static_cast<uint16_t>(pack_bf16(v, v) & 0xffffu);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max and sum over the two lanes l and l ^ 32 (which hold the same column)
__device__ __forceinline__ void swap_halves(float x, float& a, float& b) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_halves(float x) {
  float a, b;
  swap_halves(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float sum_halves(float x) {
  float a, b;
  swap_halves(x, a, b);
  return a + b;
}

// One 16-byte vector of a row in registers.
template <typename T>
struct Vec16 {
  union {
    uint4 u;
    T e[16 / sizeof(T)];
  };
};

// Elements d .. d+kVec-1 (of D) of a row that starts `offset` elements after base; zeros beyond
// D, and everywhere when !live.  VEC: rows are 16-byte aligned, D is a multiple of the vector
// and the offset in bytes fits 32 bits, so that the load takes a scalar base and one register.
template <typename T, bool VEC>
__device__ __forceinline__ Vec16<T> load_vec(const T* base, int64_t offset, int d, int D, bool live) {
  Vec16<T> v;
  v.u = make_uint4(0, 0, 0, 0);
  if (VEC) {
    const uint32_t at = static_cast<uint32_t>(offset + d) * static_cast<uint32_t>(sizeof(T));
    if (live && d < D) v.u = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + at);
  } else {
#pragma unroll
    for (int j = 0; j < Elem<T>::kVec; ++j)
      if (live && d + j < D) v.e[j] = base[offset + d + j];
  }
  return v;
}

// A lane's fragments of its row: elements 16 i + 8 half .. + 7 for every i.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_frags(const T* base, int64_t offset, int D, bool live, Frag<T> (&f)[DP / 16]) {
  const int d0 = 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < DP / 16; ++i)
#pragma unroll
    for (int h = 0; h < 8 / Elem<T>::kVec; ++h) {
      const uint4 u = load_vec<T, VEC>(base, offset, 16 * i + d0 + Elem<T>::kVec * h, D, live).u;
      __builtin_memcpy(reinterpret_cast<char*>(&f[i]) + 16 * h, &u, 16);
    }
}

// one lane's fragment of a row-major LDS tile: 8 consecutive elements of a row
__device__ __forceinline__ Frag<uint16_t> lds_frag(const uint16_t* p) {
  Frag<uint16_t> f;
  f.u = *reinterpret_cast<const uint4*>(p);
  return f;
}
__device__ __forceinline__ Frag<float> lds_frag(const float* p) {
  Frag<float> f;
  f.u[0] = *reinterpret_cast<const float4*>(p);
  f.u[1] = *reinterpret_cast<const float4*>(p + 4);
  return f;
}

// ---- tiles in LDS
//
// Tiles of rows are moved by buffer -> LDS loads, which hold no registers: lane i of a 1 KB
// load fills the 16 bytes i of its kilobyte, so rows stand one after the other without padding,
// and it is the choice of what a lane fetches that spreads them over the banks: vector j of row
// r is kept in place j ^ swz(r).  The swizzle serves both readers: 16 rows at one vector (the
// row fragments, 256 bytes a cycle) and 4 rows at 4 adjacent vectors (the transposing reads).
template <typename T, int DP>
struct Tile {
  static constexpr int kVecs = DP * static_cast<int>(sizeof(T)) / 16;   // 16-byte vectors of a row: 4 .. 32
  __device__ static __forceinline__ int swz(int r) {
    if (kVecs == 4) return (r >> 2) & 3;
    if (kVecs == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 1) << 1 | ((r >> 3) & 1);
    return (r & 3) << 2 | ((r >> 2) & 3);
  }
  // element d of row r
  __device__ static __forceinline__ int at(int r, int d) {
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    return r * DP + ((d / V) ^ swz(r)) * V + d % V;
  }
};

typedef __attribute__((address_space(3))) void lds_void;
constexpr uint32_t kOutside = 0xfffffff0u;   // a byte offset beyond every buffer: the load gives zeros

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, 0x7fffffff, 0x00020000);
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// The same where the places that the loads fill are restrict pointers of the function around it: the
// wait names them, for the compiler would else take it to concern other memory and might move the
// accesses that it stands between.
template <int N>
__device__ __forceinline__ void wait_loads(const void* cur, const void* to) {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N), "s"((const lds_void*)cur), "s"((const lds_void*)to) : "memory");
}
// waits for this wave's LDS reads and writes, but not for its loads, and for the other waves
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Rows 0 .. ROWS-1 of a tile into LDS by NT threads (thread `tid` of them): row r from element
// offset(r) after base, zeros where bit r of `live` is 0 and beyond D.  VEC: asynchronous, the
// same number of loads (tile_loads) of each wave; otherwise element by element and done on
// return, but for a barrier.
template <typename T, int DP, int ROWS, int NT>
constexpr int tile_loads = ROWS * Tile<T, DP>::kVecs / NT;
template <typename T, int DP, int ROWS, int NT, bool VEC, typename Offset>
__device__ __forceinline__ void fetch_tile(T* lds, const T* base, Offset offset, uint64_t live, int D, int tid) {
  using L = Tile<T, DP>;
  constexpr int N = tile_loads<T, DP, ROWS, NT>, KV = Elem<T>::kVec;
  static_assert(ROWS * L::kVecs % NT == 0 && ROWS <= 64, "whole loads");
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if constexpr (VEC) {
    const __amdgpu_buffer_rsrc_t rs = rsrc_of(base);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * NT + tid, r = at / L::kVecs, d = ((at % L::kVecs) ^ L::swz(r)) * KV;
      const uint32_t ofs = (static_cast<uint32_t>(offset(r)) + d) * static_cast<uint32_t>(sizeof(T));
      const bool in = ((live >> r) & 1u) && d < D;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(lds + (i * NT + wave * 64) * KV), 16,
                                               in ? ofs : kOutside, 0, 0, 0);
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const int at = i * NT + tid, r = at / L::kVecs, d = ((at % L::kVecs) ^ L::swz(r)) * KV;
      const Vec16<T> v = load_vec<T, false>(base, offset(r), d, D, (live >> r) & 1u);
      *reinterpret_cast<uint4*>(lds + at * KV) = v.u;
    }
  }
}

// Has what a fragment's loads bring awaited here, and not again in every turn of a loop that
// follows (where the wait would take in all that is on its way to the LDS).
template <typename T, int N>
__device__ __forceinline__ void arrived(Frag<T> (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < static_cast<int>(sizeof(T)) * 2; ++j) asm volatile("" : "+v"(reinterpret_cast<uint32_t*>(&f[i])[j]));
}

// The key tiles of a row tile that hold attended keys, 64 keys each, in order: mask bits and
// position.  32 tiles' bits are in the lanes at a time (the same in every wave).
struct KeyTiles {
  const uint8_t* mp;
  int Lk, end, win, t;
  uint32_t words;
  __device__ __forceinline__ KeyTiles(const uint8_t* mask, int keys, int t0, int t1)
      : mp(mask), Lk(keys), end(t1), win(t0), t(t0) {
    fill();
  }
  __device__ __forceinline__ void fill() {
    win = t;
    words = key_words(mp, static_cast<int64_t>(t) * 64, 32, static_cast<int64_t>(end) * 64, Lk);
  }
  // bits of the next tile with an attended key, whose first key is k0; 0 when there is none
  __device__ __forceinline__ uint64_t next(int64_t& k0) {
    uint64_t word = 0;
    for (; t < end && word == 0; ++t) {
      if (mp == nullptr && (t + 1) * 64 <= Lk) {
        word = ~uint64_t{0};
        continue;
      }
      if (t >= win + 32) fill();
      const int i = 2 * (t - win);
      word = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(words, i))) |
             static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(words, i + 1))) << 32;
    }
    k0 = static_cast<int64_t>(t - 1) * 64;
    return word;
  }
};

// Scores of keys that do not count become -inf.  The word is the same for all lanes, so which
// lanes keep register r are two runs of 32 lanes: bit acc_row(r, 0) and, for the upper half,
// acc_row(r, 1), spread by the scalar unit.
__device__ __forceinline__ void mask_scores(f32x16& s, uint32_t word) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const uint32_t lo = (word >> acc_row(r, 0)) & 1u ? 0xffffffffu : 0u, hi = (word >> acc_row(r, 1)) & 1u ? 0xffffffffu : 0u;
    const uint64_t keep = (static_cast<uint64_t>(hi) << 32) | lo;
    s[r] = __builtin_amdgcn_inverse_ballot_w64(keep) ? s[r] : kNegInf;
  }
}

// The second product of an attention step takes the first one's result registers as its B
// operand as they are (no exchange between lanes): register r of a lane is row
// acc_row(r, half) of the 32 rows, so the A operand has to hold the same rows in the same
// order.  acc += sum over the 32 rows of tile[row][d0 + (l & 31)] * p[r].  bf16 reads 4 rows x 16 columns at a time transposed (lane i of
// 16 hands in the address of row i / 4, columns 4*(i % 4), and receives column i of the 4
// rows); p is rounded to bf16, the operand type of the product.
struct PFrag16 {
  Frag<uint16_t> f[2];
};
struct PFrag32 {
  float p[16];
};
__device__ __forceinline__ void to_operand(const float* p, PFrag16& o) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) o.f[h].w[j] = pack_bf16(p[8 * h + 2 * j], p[8 * h + 2 * j + 1]);
}
__device__ __forceinline__ void to_operand(const float* p, PFrag32& o) {
#pragma unroll
  for (int r = 0; r < 16; ++r) o.p[r] = p[r];
}
template <typename T>
struct POperand;
template <>
struct POperand<uint16_t> { using type = PFrag16; };
template <>
struct POperand<float> { using type = PFrag32; };

// The transposed operand of 16 rows (h: the first or second 16 of the 32 that start at r0, a
// multiple of 32).
template <int DP>
__device__ __forceinline__ Frag<uint16_t> col_frag(const uint16_t* tile, int r0, int d0, int h) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int l = threadIdx.x & 63, i = l & 15, r = r0 + 4 * (l >> 5) + (i >> 2), d = d0 + 16 * ((l >> 4) & 1) + 4 * (i & 3);
  Frag<uint16_t> a;
  a.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + Tile<uint16_t, DP>::at(r + 16 * h, d)));
  a.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(tile + Tile<uint16_t, DP>::at(r + 16 * h + 8, d)));
  return a;
}
template <int DP>
__device__ __forceinline__ f32x16 mma_rows(const uint16_t* tile, int r0, int d0, const PFrag16& p, f32x16 acc) {
#pragma unroll
  for (int h = 0; h < 2; ++h) acc = mma(col_frag<DP>(tile, r0, d0, h), p.f[h], acc);
  return acc;
}
template <int DP>
__device__ __forceinline__ f32x16 mma_rows(const float* tile, int r0, int d0, const PFrag32& p, f32x16 acc) {
  const int l = threadIdx.x & 63, half = l >> 5;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(tile[Tile<float, DP>::at(r0 + acc_row(r, half), d0 + (l & 31))], p.p[r],
                                               acc, 0, 0, 0);
  return acc;
}
// A lane's fragment of row r0 + (lane & 31) at the 16-wide step i.
template <int DP>
__device__ __forceinline__ Frag<uint16_t> row_frag(const uint16_t* tile, int r0, int i) {
  const int l = threadIdx.x & 63;
  return lds_frag(tile + Tile<uint16_t, DP>::at(r0 + (l & 31), 16 * i + 8 * (l >> 5)));
}
template <int DP>
__device__ __forceinline__ Frag<float> row_frag(const float* tile, int r0, int i) {
  const int l = threadIdx.x & 63, r = r0 + (l & 31), d = 16 * i + 8 * (l >> 5);
  Frag<float> f;
  f.u[0] = *reinterpret_cast<const float4*>(tile + Tile<float, DP>::at(r, d));
  f.u[1] = *reinterpret_cast<const float4*>(tile + Tile<float, DP>::at(r, d + 4));
  return f;
}

// One workgroup's part of the problem: a tile of rows (or, for dK and dV, of keys) of one (batch
// element, key head), and steps s0 .. s1 - 1 of what it loops over.  Consecutive workgroups are consecutive pairs: the row tiles
// that read the same keys then run on the same XCD when the pairs are a multiple of 8.
struct Work {
  int b, hk, row0, split, tail;   // tail: index of a split tile, or -1
  int s0, s1;
};
__device__ __forceinline__ Work work_of(const Args& a, const Tiling& y, int at_tile, int rows, int steps) {
  Work w;
  int tile = at_tile;
  w.tail = -1;
  w.split = 0;
  w.s0 = 0;
  w.s1 = steps;
  if (tile >= y.full) {
    const int n = y.tiles - y.full, at = tile - y.full;
    w.tail = at % n;
    w.split = at / n;
    tile = y.full + w.tail;
    w.s0 = w.split * y.per_split;
    w.s1 = min(steps, w.s0 + y.per_split);
  }
  const int nbh = a.B * a.Hkv, bh = tile % nbh;
  w.b = bh / a.Hkv;
  w.hk = bh % a.Hkv;
  w.row0 = tile / nbh * rows;
  return w;
}

// ---- host side

// Tiling for `tiles` tiles of `steps` steps each on a chip that holds `slots` workgroups at a
// time: whole rounds of the chip go unsplit; the steps of each tile of the last, incomplete round
// are split so that the round fills the chip, but not below `least` steps.
inline Tiling tile_over(int64_t tiles, int64_t steps, int64_t slots, int64_t least) {
  Tiling y{};
  const int64_t tail = tiles % slots;
  int64_t splits = tail == 0 ? 1 : slots / tail;
  if (splits > steps / least) splits = steps / least > 1 ? steps / least : 1;
  y.tiles = static_cast<int>(tiles);
  y.per_split = static_cast<int>((steps + splits - 1) / splits);
  y.splits = y.per_split > 0 ? static_cast<int>((steps + y.per_split - 1) / y.per_split) : 1;
  if (y.splits < 1) y.splits = 1;
  y.full = static_cast<int>(y.splits > 1 ? tiles - tail : tiles);
  return y;
}
inline int64_t workgroups(const Tiling& y) { return y.full + static_cast<int64_t>(y.tiles - y.full) * y.splits; }
inline int padded_head(int64_t D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }
// Tiles of a ring in the LDS: three where two workgroups of a CU then have room (rows of 128 bytes:
// 48 KB a workgroup), else two (rows of 256 or 512 bytes: 64 or 128 KB).
constexpr int stages_of(int row_bytes) { return row_bytes <= 128 ? 3 : 2; }
constexpr int kCUs = 256;

// Launches n workgroups of `threads` threads.  A dispatch counts its threads in 32 bits: beyond that
// they go in several launches, each of which is told (Args::first) how many went before it.
inline bool launch_groups(const void* fn, int64_t n, int threads, void** args, Args* a, size_t lds, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 21;   // of up to 1024 threads
  for (int64_t first = 0; first < n; first += kMost) {
    a->first = static_cast<int>(first);
    const int64_t now = n - first < kMost ? n - first : kMost;
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(now)), dim3(threads), args, lds, stream) != hipSuccess) return false;
  }
  return true;
}

// Descriptor checks of every attention entry point: DCN_OK or a negative dcn_status.
int check(const dcn_attn_desc* d);
// 16-byte row accesses at 32-bit offsets are possible for a tensor of these strides at this address
inline bool vec_ok(const void* p, const int64_t* s, int64_t D, int es) {
  const int64_t n = 16 / es;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && D % n == 0 && s[0] % n == 0 && s[1] % n == 0 && s[2] % n == 0 &&
         s[1] <= int64_t{1} << 22;   // 128 rows within 32 bits of bytes of each other
}
void fill_args(const dcn_attn_desc* d, Args* a);

}  // namespace attn
}  // namespace dcn

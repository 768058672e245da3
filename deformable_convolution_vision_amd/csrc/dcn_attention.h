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

struct Args {
  const void *q, *k, *v;
  const uint8_t* mask;         // [B][Lk] bytes, 0: the key is padding; or null
  void* out;                   // [B][Lq][Hq][D]
  float* lse;                  // [B][Hq][Lq] or null
  float* part;                 // forward: partial outputs [S][B][Hkv][R][DP], not yet divided by their sums
  float* part_ml;              // ... with each row's maximum and sum, [S][B][Hkv][R][2]
  const void* dout;            // backward: [B][Lq][Hq][D]
  const float* delta;          // backward: [B][Hkv][R][2]: lse in powers of two, and sum(dout * out)
  void *dq, *dk, *dv;
  int64_t qs[3], ks[3], vs[3]; // strides in elements: batch, position, head
  int64_t ms;                  // the mask's batch stride
  int B, Lq, Lk, Hq, Hkv, g, D;
  int R;                       // query rows of one key head: g * Lq, row r = position r / g, head r % g
  int splits;                  // parts the keys (dK, dV: the rows) are split into
  int per_split;               // tiles of one part
  float c;                     // scale * log2(e): softmax runs in powers of two
  float scale;
};

__device__ __forceinline__ constexpr int acc_row(int r, int half) { return (r & 3) + 8 * (r >> 2) + 4 * half; }

// 16 bytes of a row: 8 bf16 or 4 fp32 elements
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;   // elements of 16 bytes
  static constexpr int kPad = 16;  // LDS rows DP + 16 long: 32-byte offsets that neither the 16-byte row reads nor
                                   // the transposing reads of 4 rows find on the same banks
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr int kPad = 4;
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

// A zero accumulator the compiler cannot see through: it may otherwise place an operand
// of the first product in the product's own result registers.
__device__ __forceinline__ f32x16 zero_acc() {
  f32x16 z;
#pragma unroll
  for (int r = 0; r < 16; ++r) z[r] = 0.f;
  asm volatile("" : "+v"(z));
  return z;
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

// elements d .. d+kVec-1 of a row of D elements; zeros beyond D, and everywhere when !live.
// VEC: rows are 16-byte aligned and D is a multiple of the vector.
template <typename T, bool VEC>
__device__ __forceinline__ Vec16<T> load_vec(const T* row, int d, int D, bool live) {
  Vec16<T> v;
  v.u = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (live && d < D) v.u = *reinterpret_cast<const uint4*>(row + d);
  } else {
#pragma unroll
    for (int j = 0; j < Elem<T>::kVec; ++j)
      if (live && d + j < D) v.e[j] = row[d + j];
  }
  return v;
}

template <typename T, bool VEC>
__device__ __forceinline__ Frag<T> load_frag(const T* row, int d, int D, bool live);
template <>
__device__ __forceinline__ Frag<uint16_t> load_frag<uint16_t, true>(const uint16_t* row, int d, int D, bool live) {
  Frag<uint16_t> f;
  f.u = load_vec<uint16_t, true>(row, d, D, live).u;
  return f;
}
template <>
__device__ __forceinline__ Frag<uint16_t> load_frag<uint16_t, false>(const uint16_t* row, int d, int D, bool live) {
  Frag<uint16_t> f;
  f.u = load_vec<uint16_t, false>(row, d, D, live).u;
  return f;
}
template <>
__device__ __forceinline__ Frag<float> load_frag<float, true>(const float* row, int d, int D, bool live) {
  Frag<float> f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 u = load_vec<float, true>(row, d + 4 * h, D, live).u;
    f.u[h] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
  }
  return f;
}
template <>
__device__ __forceinline__ Frag<float> load_frag<float, false>(const float* row, int d, int D, bool live) {
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f.f[j] = (live && d + j < D) ? row[d + j] : 0.f;
  return f;
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

// The second product of an attention step takes the first one's result registers as its B
// operand as they are (no exchange between lanes): register r of a lane is row
// acc_row(r, half) of the 32 rows, so the A operand has to hold the same rows in the same
// order.  acc += sum over the 32 rows of tile[row][d0 + (l & 31)] * p[r]; `tile` points at
// the first of the 32 rows.  bf16 reads 4 rows x 16 columns at a time transposed (lane i of
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

__device__ __forceinline__ f32x16 mma_rows(const uint16_t* tile, int stride, int d0, const PFrag16& p, f32x16 acc) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int l = threadIdx.x & 63, i = l & 15;
  const uint16_t* at = tile + (4 * (l >> 5) + (i >> 2)) * stride + d0 + 16 * ((l >> 4) & 1) + 4 * (i & 3);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    Frag<uint16_t> a;
    a.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + (16 * h) * stride));
    a.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + (16 * h + 8) * stride));
    acc = mma(a, p.f[h], acc);
  }
  return acc;
}
__device__ __forceinline__ f32x16 mma_rows(const float* tile, int stride, int d0, const PFrag32& p, f32x16 acc) {
  const int l = threadIdx.x & 63, half = l >> 5;
  const float* at = tile + d0 + (l & 31);
#pragma unroll
  for (int r = 0; r < 16; ++r)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(at[acc_row(r, half) * stride], p.p[r], acc, 0, 0, 0);
  return acc;
}

// ---- host side

struct Plan {
  int dp;        // head size the kernel is built for: 32, 64 or 128
  int wide;      // 1: four waves of 32 rows share each key tile; 0: four waves split the keys of 32 rows
  int splits;    // workgroups that share the keys of a row tile
  int per_split; // key tiles of each
  int tile;      // keys of a tile
};

// Descriptor checks of every attention entry point: DCN_OK or a negative dcn_status.
int check(const dcn_attn_desc* d);
// 16-byte row accesses are possible for a tensor of these strides at this address
inline bool vec_ok(const void* p, const int64_t* s, int64_t D, int es) {
  const int64_t n = 16 / es;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && D % n == 0 && s[0] % n == 0 && s[1] % n == 0 && s[2] % n == 0;
}
void fill_args(const dcn_attn_desc* d, Args* a);

}  // namespace attn
}  // namespace dcn

// dcn_rotary.h -- what rotary positions (dcn_rotary.hip) and the paged cache's append
// (dcn_append.hip) share: the angles, a pair's place in its head, vectors of a row, how rows fall to
// workgroups, and the host-side checks.  Not part of the public ABI.
//
// A workgroup takes a few rows.  It forms the cosines and sines of their angles once, in the LDS, where
// every head of the rows reads them; the elements' loads are under way meanwhile.  A thread's unit is a
// chunk of PV pairs of one head: two vectors of PV elements, wherever the layout has them.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dcn.h"

namespace dcn {
namespace rotary {

// The angles of a row and where its pairs stand.
struct Turns {
  const void* positions;
  const float* freq;
  int64_t ps[2];          // positions' strides: batch, row
  int end[3];             // pairs below end[0] turn with axis 0, below end[1] with axis 1, ...
  int start[4];           // each axis's first pair
  int axes, pairs, layout;
  bool whole;             // positions are int32
};

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));   // nearest even
}

// N adjacent elements in one access
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T e[N];
};

// cos and sin of pos * f.  The angle is formed in quarter turns in 64 bits and reduced there to the
// nearest quarter, |x| <= pi / 4; the remainder's sine and cosine are their Taylor polynomials of degree
// 9 and 10 (the first terms left out are 1.8e-9 and 1.2e-10 there, below 2^-24 of the value).
__device__ __forceinline__ void cos_sin(double pos, float f, float& c, float& s) {
  const double q = pos * (static_cast<double>(f) * 0.636619772367581343);
  const double n = __builtin_rint(q);
  const float x = static_cast<float>((q - n) * 1.57079632679489662), y = x * x;
  const int k = static_cast<int>(4.0 * __builtin_amdgcn_fract(0.25 * n));
  float ps = fmaf(y, 2.75573192e-6f, -1.98412698e-4f);
  ps = fmaf(ps, y, 8.33333333e-3f);
  ps = fmaf(ps, y, -0.166666667f);
  ps = fmaf(ps * y, x, x);
  float pc = fmaf(y, -2.75573192e-7f, 2.48015873e-5f);
  pc = fmaf(pc, y, -1.38888889e-3f);
  pc = fmaf(pc, y, 4.16666667e-2f);
  pc = fmaf(pc, y, -0.5f);
  pc = fmaf(pc, y, 1.f);
  const float a = (k & 1) != 0 ? ps : pc, b = (k & 1) != 0 ? pc : ps;
  c = ((k + 1) & 2) != 0 ? -a : a;
  s = (k & 2) != 0 ? -b : b;
}

// The axis that a pair turns with.
__device__ __forceinline__ int axis_of(const Turns& t, int pair) {
  return (pair >= t.end[0]) + (pair >= t.end[1]) + (pair >= t.end[2]);
}
__device__ __forceinline__ double position_of(const Turns& t, int b, int row, int axis) {
  const int64_t o = b * t.ps[0] + row * t.ps[1] + axis;
  return t.whole ? static_cast<double>(static_cast<const int32_t*>(t.positions)[o])
                 : static_cast<double>(static_cast<const float*>(t.positions)[o]);
}

// Division by a number that is known on the host, of n < 2^16 (both): the product with 2^32 / d, rounded
// up, is then off by less than 1 / d.
struct Div {
  uint32_t d, m;
  __device__ __forceinline__ int of(int n) const { return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m)); }
};

// The first elements of a chunk's two vectors.
struct Place {
  int e1, e2;
};
template <int PV>
__device__ __forceinline__ Place place_of(const Turns& t, int chunk, int rotated) {
  if (chunk >= rotated) {   // behind the pairs: copied
    const int e = 2 * t.pairs + (chunk - rotated) * 2 * PV;
    return {e, e + PV};
  }
  const int p = chunk * PV;
  if (t.layout == DCN_ROTARY_HALVES) return {p, p + t.pairs};
  if (t.layout == DCN_ROTARY_ADJACENT) return {2 * p, 2 * p + PV};
  const int a = axis_of(t, p);
  const int n = (a < t.axes - 1 ? t.end[a] : t.pairs) - t.start[a];
  return {p + t.start[a], p + t.start[a] + n};
}

// The pairs (x1, x2) of a chunk's two vectors, and back.  ADJ: a pair's elements are neighbours.
template <typename T, int PV, bool ADJ>
__device__ __forceinline__ void pairs_of(const Vec<T, PV>& u, const Vec<T, PV>& v, float (&x1)[PV], float (&x2)[PV]) {
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    if (ADJ && PV > 1) {
      x1[j] = widen<T>(2 * j < PV ? u.e[(2 * j) % PV] : v.e[(2 * j) % PV]);
      x2[j] = widen<T>(2 * j + 1 < PV ? u.e[(2 * j + 1) % PV] : v.e[(2 * j + 1) % PV]);
    } else {
      x1[j] = widen<T>(u.e[j]);
      x2[j] = widen<T>(v.e[j]);
    }
  }
}
template <typename T, int PV, bool ADJ>
__device__ __forceinline__ void vectors_of(const float (&y1)[PV], const float (&y2)[PV], Vec<T, PV>& u, Vec<T, PV>& v) {
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    if (ADJ && PV > 1) {
      (2 * j < PV ? u : v).e[(2 * j) % PV] = narrow<T>(y1[j]);
      (2 * j + 1 < PV ? u : v).e[(2 * j + 1) % PV] = narrow<T>(y2[j]);
    } else {
      u.e[j] = narrow<T>(y1[j]);
      v.e[j] = narrow<T>(y2[j]);
    }
  }
}
template <int PV>
__device__ __forceinline__ void turn(const float (&c)[PV], const float (&s)[PV], const float (&x1)[PV],
                                     const float (&x2)[PV], float (&y1)[PV], float (&y2)[PV]) {
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    y1[j] = fmaf(x1[j], c[j], -(x2[j] * s[j]));
    y2[j] = fmaf(x2[j], c[j], x1[j] * s[j]);
  }
}

// ---- host side

// Checks of the rotation's fields: DCN_OK or a negative status.
inline int check_turns(int32_t axes, const int32_t* sections, int32_t layout, int32_t position_type,
                       const int64_t* position_stride, int64_t head_dim) {
  if (axes < 0 || axes > 4 || layout < 0 || layout > DCN_ROTARY_BLOCKS || position_type < 0 ||
      position_type > DCN_POSITION_I32 || position_stride[0] < 0 || position_stride[1] < 0)
    return DCN_E_ARG;
  int64_t pairs = 0;
  for (int a = 0; a < axes; ++a) {
    if (sections[a] < 1) return DCN_E_ARG;
    pairs += sections[a];
  }
  return 2 * pairs > head_dim ? DCN_E_ARG : DCN_OK;
}
inline Turns turns_of(int32_t axes, const int32_t* sections, int32_t layout, int32_t position_type,
                      const int64_t* position_stride, const void* positions, const float* frequencies) {
  Turns t{};
  t.positions = positions;
  t.freq = frequencies;
  t.ps[0] = position_stride[0];
  t.ps[1] = position_stride[1];
  t.axes = axes;
  t.layout = layout;
  t.whole = position_type == DCN_POSITION_I32;
  for (int a = 0; a < axes; ++a) {
    t.start[a] = t.pairs;
    t.pairs += sections[a];
    if (a < 3) t.end[a] = t.pairs;
  }
  for (int a = axes; a < 3; ++a) t.end[a] = t.pairs;   // (no pair is at or behind it)
  return t;
}

// The widest vectors, in elements, that a rotation of these sections allows: the pairs of a chunk are
// then whole within each run of the layout.  `fit` halves it further for addresses and strides.
inline int width_of(const Turns& t, const int32_t* sections, int64_t head_dim, int es) {
  int w = 16 / es;
  while (w > 1 && (t.pairs % w != 0 || head_dim % w != 0)) w /= 2;
  if (t.layout == DCN_ROTARY_BLOCKS)
    for (int a = 0; a < t.axes; ++a)
      while (w > 1 && sections[a] % w != 0) w /= 2;
  return w;
}
inline int fit(int w, int es, const void* p) {
  while (w > 1 && reinterpret_cast<uintptr_t>(p) % (static_cast<unsigned>(w) * es) != 0) w /= 2;
  return w;
}
inline int fit(int w, const int64_t* strides, int n) {
  for (int i = 0; i < n; ++i)
    while (w > 1 && strides[i] % w != 0) w /= 2;
  return w;
}

// How rows and heads fall to workgroups of 256: `rows` rows and `heads` heads of each, of which a row has
// `groups`; a head has `chunks` chunks, `rotated` of them of pairs, the others copied.
constexpr int kTurns = 2048;      // cosines and sines of a workgroup: 16 KB
// Units of a thread under way at a time, by the bytes of a vector.  Two of 16 bytes fill the memory's queues and leave
// workgroups small enough for an even last round (rotary_c3_batch8 with 1, 2, 4 units: 32.9, 33.0, 36.6
// us); narrower ones take four (2 bytes, 16800 rows of 8 heads of 37: 21.7, 13.5, 12.1 us).
constexpr int units_of(int bytes) { return bytes == 16 ? 2 : 4; }
constexpr int kRows = 64;         // the most rows of a workgroup
struct Cut {
  int chunks, rotated, rows, heads, groups;
  Div by_chunks, by_row, by_pairs;   // by_row: heads * chunks
};
inline Div div_by(int64_t d) {
  return {static_cast<uint32_t>(d < 1 ? 1 : d), static_cast<uint32_t>(d < 2 ? 0 : (int64_t{1} << 32) / d + 1)};
}
// Rows share nothing, so a workgroup takes as many as fill its threads' units; where there are fewer than
// four workgroups a CU then, fewer rows each, and fewer heads of one row.
inline Cut cut_of(int width, int es, int pairs, int64_t head_dim, int64_t rows, int64_t heads) {
  Cut c{};
  c.rotated = pairs / width;
  c.chunks = c.rotated + static_cast<int>((head_dim - 2 * pairs + 2 * width - 1) / (2 * width));
  const int64_t most = units_of(width * es) * 256, wanted = 4 * 256;
  int64_t h = heads * c.chunks <= most ? heads : most / c.chunks > 1 ? most / c.chunks : 1;
  if (rows * ((heads + h - 1) / h) < wanted && h * c.chunks > 256) h = 256 / c.chunks > 1 ? 256 / c.chunks : 1;
  int64_t r = most / (h * c.chunks);
  if (pairs > 0 && r > kTurns / pairs) r = kTurns / pairs;
  const int64_t least = (256 + h * c.chunks - 1) / (h * c.chunks);   // a unit for each thread
  if (r > rows / wanted) r = rows / wanted > least ? rows / wanted : r < least ? r : least;
  if (r > kRows) r = kRows;
  c.rows = static_cast<int>(r < 1 ? 1 : r);
  c.heads = static_cast<int>(h);
  c.groups = static_cast<int>((heads + h - 1) / h);
  c.by_chunks = div_by(c.chunks);
  c.by_row = div_by(h * c.chunks);
  c.by_pairs = div_by(pairs);
  return c;
}

// Launches n workgroups of 256 threads; a dispatch counts its threads in 32 bits, so beyond 2^23 of them
// they go in several launches, each of which is told (*first) how many went before it.
inline bool launch(const void* fn, int64_t n, void** args, int64_t* first, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 23;
  for (int64_t at = 0; at < n; at += kMost) {
    *first = at;
    const int64_t now = n - at < kMost ? n - at : kMost;
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(now)), dim3(256), args, 0, stream) != hipSuccess) return false;
  }
  return true;
}

}  // namespace rotary
}  // namespace dcn

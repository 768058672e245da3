// dcn_rotary.h -- what rotary positions (dcn_rotary.hip) and the paged cache's append
// (dcn_append.hip) share: the angles, a pair's place in its head, vectors of a row, how rows fall to
// workgroups, and the host-side checks.  Not part of the public ABI.
//
// A workgroup takes a few rows.  It forms the cosines and sines of their angles once, in the LDS, where
// every head of the rows reads them.  Heads pass through the LDS (turn_heads): memory is read and written in
// whole vectors, one after the other, whatever pairs the layout makes of the elements.
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
// nearest quarter, |x| <= pi / 4; the remainder's sine and cosine are their Taylor polynomials of degree 11 and 12 (the
// first terms left out are below 2^-33), with the upper terms in 32 bits (their sum is below 2^-7 of a term that is
// there in 64) and the others in 64, so that both are off by their one rounding to fp32 and 2^-30.
__device__ __forceinline__ void cos_sin(double pos, float f, float& c, float& s) {
  const double q = pos * (static_cast<double>(f) * 0.636619772367581343);
  const double n = __builtin_rint(q);
  const double x = (q - n) * 1.57079632679489662, y = x * x;
  // n's last two bits stand at the end of this sum's (from 2^51 quarter turns on they are any, as the angle is)
  const int k = __double2loint(n + 6755399441055744.);
  const float z = static_cast<float>(y);
  float us = fmaf(z, -2.50521084e-8f, 2.75573192e-6f);
  us = fmaf(us, z, -1.98412698e-4f);
  us = fmaf(us, z, 8.33333333e-3f);
  float uc = fmaf(z, 2.08767570e-9f, -2.75573192e-7f);
  uc = fmaf(uc, z, 2.48015873e-5f);
  uc = fmaf(uc, z, -1.38888889e-3f);
  const float ps = static_cast<float>(fma(x, y * (static_cast<double>(us * z) - 1. / 6.), x));
  const float pc = static_cast<float>(fma(fma(static_cast<double>(uc * z) + 1. / 24., y, -0.5), y, 1.));
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

// The first elements of a chunk's two vectors: PV pairs from p on.
struct Place {
  int e1, e2;
};
template <int PV>
__device__ __forceinline__ Place place_of(const Turns& t, int p) {
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

// Row r of a workgroup whose first row is l0 of batch element b0 (L rows each).
struct Row {
  int b, l;
};
__device__ __forceinline__ Row row_of(int b0, int l0, int r, int L) {
  Row w = {b0, l0 + r};
  if (w.l >= L) {          // (seldom: the division is left out of the common case)
    const int n = static_cast<int>(static_cast<uint32_t>(w.l) / static_cast<uint32_t>(L));
    w.b += n;
    w.l -= n * L;
  }
  return w;
}

// Elements from a workgroup's first row and head to another of its own: in products of 24 bits, which cost a quarter of
// 32-bit ones (near_by says that they are enough; with 64-bit strides in every lane the addresses were most of the
// instructions: 83 us where 73 now for 8 x 4200 ragged rows of an append, 20 where 16 for 4 x 4200 rows of heads of 37).
__device__ __forceinline__ uint32_t apart(int r, int s1, int h, int s2) {
  return __umul24(static_cast<uint32_t>(r), static_cast<uint32_t>(s1)) + __umul24(static_cast<uint32_t>(h), static_cast<uint32_t>(s2));
}

// Cosines and sines of the rows' angles into the LDS, [row][pair], by all 256 threads: a thread keeps its pair and
// takes rows in turn, four positions on their way at a time.  position(row): of the pair's axis.
template <typename P>
__device__ __forceinline__ void form_turns(const Turns& t, int log_pairs, int rows, float sign, float2* cs, P position) {
  const int step = 256 >> log_pairs;
  for (int pair = threadIdx.x & ((1 << log_pairs) - 1); pair < t.pairs; pair += 256) {
    const float f = t.freq[pair];
    const int axis = axis_of(t, pair);
    for (int r0 = threadIdx.x >> log_pairs; r0 < rows; r0 += 4 * step) {
      double p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = r0 + k * step < rows ? position(r0 + k * step, axis) : 0.;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r0 + k * step >= rows) break;
        float c, s;
        cos_sin(p[k], f, c, s);
        cs[(r0 + k * step) * t.pairs + pair] = make_float2(c, sign * s);
      }
    }
  }
}

// How rows and heads fall to workgroups of 256.
constexpr int kTurns = 2048;      // cosines and sines of a workgroup at most: 16 KB
constexpr int kWave = 2048;       // bytes of heads of a wave in the LDS;
constexpr int held_by(int bytes) { return bytes == 2 ? kWave / 2 : kWave; }   // so many are used with vectors of so many
constexpr int kMostD = 512;       // elements of a head
struct Cut {
  int rows, heads, groups;        // of a workgroup: rows, and heads of each, of which a row has `groups` groups
  int at_once;                    // heads of a wave at a time
  int vectors, chunks;            // of a head
  Div by_heads, by_vectors, by_chunks;
  int log_pairs;                  // 2^log_pairs: threads that share a row's angles out, up to 256
};

// Orders a wave's LDS accesses of different lanes (no instruction: a wave's are carried out in order).
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// So many bytes in one access, and the same in memory, which takes them wherever an element may start.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int BYTES, int ELEMENT>
struct Bytes;
template <>
struct Bytes<16, 2> {
  typedef u32x4 type;
  typedef u32x4 memory __attribute__((aligned(2)));
};
template <>
struct Bytes<16, 4> {
  typedef u32x4 type;
  typedef u32x4 memory __attribute__((aligned(4)));
};
template <>
struct Bytes<4, 2> {
  typedef uint32_t type;
  typedef uint32_t memory __attribute__((aligned(2)));
};
template <>
struct Bytes<4, 4> {
  typedef uint32_t type;
  typedef uint32_t memory;
};
template <>
struct Bytes<2, 2> {
  typedef uint16_t type;
  typedef uint16_t memory;
};

// Moves heads 0 .. n-1 of a workgroup, at_once of them by each wave in turn, from from(i) to to(i) (null: not
// written), turned by the angles of row turned(i) (below 0: not turned).  WV: elements of a vector of memory; PV:
// pairs of a chunk, a vector of the LDS.  between(): called by every thread once the first heads' loads are under
// way; forms the angles.  The next heads' loads are under way while a wave's heads are turned.
template <typename T, int WV, int PV, bool ADJ, typename From, typename To, typename Turned, typename Between>
__device__ __forceinline__ void turn_heads(const Turns& t, const Cut& c, int n, T* lds, const float2* cs, From from, To to,
                                           Turned turned, Between between) {
  constexpr int NV = held_by(WV * static_cast<int>(sizeof(T))) / (64 * WV * static_cast<int>(sizeof(T)));
  using M = typename Bytes<WV * static_cast<int>(sizeof(T)), static_cast<int>(sizeof(T))>::type;
  using InMemory = typename Bytes<WV * static_cast<int>(sizeof(T)), static_cast<int>(sizeof(T))>::memory;
  using V = Vec<T, PV>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), step = 4 * c.at_once,
            vectors = c.at_once * c.vectors, chunks = c.at_once * c.chunks, D = c.vectors * WV;
  M held[NV];
  const auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * 64 + lane, g = c.by_vectors.of(v);
      if (v >= vectors || i0 + g >= n) continue;
      const T* x = from(i0 + g);
      if (x != nullptr) held[k] = *reinterpret_cast<const InMemory*>(x + (v - g * c.vectors) * WV);
    }
  };
  const int first = wave * c.at_once;
  fetch(first);
  between();
  for (int i0 = first; i0 < n; i0 += step) {
    wave_order();
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (k * 64 + lane < vectors) *reinterpret_cast<M*>(lds + (k * 64 + lane) * WV) = held[k];
    wave_order();
    if (i0 + step < n) fetch(i0 + step);
    for (int q = lane; q < chunks; q += 64) {
      const int g = c.by_chunks.of(q), p0 = (q - g * c.chunks) * PV, row = i0 + g < n ? turned(i0 + g) : -1;
      if (row < 0) continue;
      const Place p = place_of<PV>(t, p0);
      V u = *reinterpret_cast<const V*>(lds + g * D + p.e1), v = *reinterpret_cast<const V*>(lds + g * D + p.e2);
      const float2* turns = cs + row * t.pairs + p0;
      float co[PV], si[PV], x1[PV], x2[PV], y1[PV], y2[PV];
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        co[j] = turns[j].x;
        si[j] = turns[j].y;
      }
      pairs_of<T, PV, ADJ>(u, v, x1, x2);
      turn<PV>(co, si, x1, x2, y1, y2);
      vectors_of<T, PV, ADJ>(y1, y2, u, v);
      *reinterpret_cast<V*>(lds + g * D + p.e1) = u;
      *reinterpret_cast<V*>(lds + g * D + p.e2) = v;
    }
    wave_order();
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = k * 64 + lane, g = c.by_vectors.of(v);
      if (v >= vectors || i0 + g >= n) continue;
      T* y = to(i0 + g);
      if (y != nullptr) *reinterpret_cast<InMemory*>(y + (v - g * c.vectors) * WV) = *reinterpret_cast<const M*>(lds + v * WV);
    }
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

// Elements of a vector of memory: 16 bytes, 4 (bf16) or one element, the most that a head is a whole number of.
inline int narrower(int w, int es) { return es == 2 && w > 2 ? 2 : 1; }
inline int vector_of(int64_t head_dim, int es) {
  int w = 16 / es;
  while (w > 1 && head_dim % w != 0) w = narrower(w, es);
  return w;
}
// Pairs of a chunk: as many as a vector of memory has elements, if every run of the layout is whole chunks.
inline int pairs_at_once(const Turns& t, const int32_t* sections, int w, int es) {
  while (w > 1 && t.pairs % w != 0) w = narrower(w, es);
  if (t.layout == DCN_ROTARY_BLOCKS)
    for (int a = 0; a < t.axes; ++a)
      while (w > 1 && sections[a] % w != 0) w = narrower(w, es);
  return w;
}

inline Div div_by(int64_t d) {
  return {static_cast<uint32_t>(d < 1 ? 1 : d), static_cast<uint32_t>(d < 2 ? 0 : (int64_t{1} << 32) / d + 1)};
}
// A workgroup takes two or three times what its waves hold, in whole rows where they are short: of these the number
// that leaves the least of the last turn unused, fewer turns where that is equal (24 heads of 128, 33600 rows: 2
// rows, 3/4 of two turns, 108 us; 4 rows, three turns, 90).  Four turns were slower than three wherever tried.  Where that leaves fewer
// than four workgroups a CU, fewer rows each, and fewer heads of one row, down to what a wave holds.
inline Cut cut_of(int wv, int pv, int es, int pairs, int64_t head_dim, int64_t rows, int64_t heads) {
  Cut c{};
  c.at_once = static_cast<int>(held_by(wv * es) / (head_dim * es));
  c.vectors = static_cast<int>(head_dim / wv);
  c.chunks = pairs / pv;
  const int64_t turn = int64_t{4} * c.at_once, wanted = 4 * 256;
  int64_t h = heads < 2 * turn ? heads : 2 * turn;
  while (h > c.at_once && rows * ((heads + h - 1) / h) < wanted) h = (h + 1) / 2;
  int64_t most = 3 * turn / h;
  if (pairs > 0 && most > kTurns / pairs) most = kTurns / pairs;
  if (most > rows / wanted) most = rows / wanted;
  const auto turns = [&](int64_t r) { return (r * h + turn - 1) / turn; };
  int64_t best = most > 1 ? most : 1;
  for (int64_t r = best - 1; r >= 1 && turns(r) >= 2; --r)
    if (r * turns(best) >= best * turns(r)) best = r;      // rows a turn: as many, in fewer turns
  c.rows = static_cast<int>(best);
  c.heads = static_cast<int>(h);
  c.groups = static_cast<int>((heads + h - 1) / h);
  c.by_heads = div_by(h);
  c.by_vectors = div_by(c.vectors);
  c.by_chunks = div_by(c.chunks);
  while (c.log_pairs < 8 && (1 << c.log_pairs) < pairs) ++c.log_pairs;
  return c;
}

// Whether `apart` serves so many rows and heads with these strides.
inline bool near_by(int64_t rows, int64_t s1, int64_t heads, int64_t s2) {
  constexpr int64_t kMost = int64_t{1} << 24;
  return rows < kMost && s1 < kMost && heads < kMost && s2 < kMost && rows * s1 + heads * s2 < (int64_t{1} << 31);
}

// Launches n workgroups of 256 threads; a dispatch counts its threads in 32 bits, so beyond 2^23 of them
// they go in several launches, each of which is told (*first) how many went before it.
inline size_t turns_bytes(const Cut& c, const Turns& t) { return static_cast<size_t>(c.rows) * t.pairs * sizeof(float2); }
inline bool launch(const void* fn, int64_t n, void** args, size_t lds, uint32_t* first, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 23;
  for (int64_t at = 0; at < n; at += kMost) {
    *first = static_cast<uint32_t>(at);
    const int64_t now = n - at < kMost ? n - at : kMost;
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>(now)), dim3(256), args, lds, stream) != hipSuccess) return false;
  }
  return true;
}

}  // namespace rotary
}  // namespace dcn

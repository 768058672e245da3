// dcn_rotary.hip -- gfx950 rotary positions with several axes, and their gradients.
//
// Pair p of every head of row (b, l) turns by t = positions[b][l][axis(p)] * freq[p]:
//
//   y1 = x1 cos t - x2 sin t,  y2 = x2 cos t + x1 sin t
//
// and for an upstream gradient g the input's gradient is the rotation back,
//
//   gx1 = g1 cos t + g2 sin t,  gx2 = g2 cos t - g1 sin t,
//
// and the position's, from dy/dt = (-y2, y1) and lengths and angles that a rotation keeps,
//
//   grad_pos[b][l][a] = sum over heads and the axis's pairs of freq[p] (gx2 x1 - gx1 x2).
//
// The rotation, either way, is rotary_kernel (turn_heads does the work).  With the position's gradient it is
// rotary_grad_kernel: a workgroup has all heads of its rows, a thread takes chunks of pairs straight from memory and
// leaves each one's sum for each axis in the LDS, where one thread for each row and axis adds them in order.
//
// Memory bounds it: 8 x 16800 rows of 8 heads of 32, bf16, take 28.6 us for 137.8 MB, 4.8 TB/s of the 4.99 that a large
// copy reaches, and 2 x 8400 rows of 8 heads of 64 9.9 us for 34.5 MB, a round and a start of the chip.  Chunks of
// pairs straight from memory, each lane its two vectors, took 33.0 us for the first, and 64 where a head of 32 turns
// one pair (26 now): their vectors are as wide as the layout's runs allow, those of whole heads always 16 bytes.
// The positions' gradient of 2 x 900 rows takes 5.6 us, one round of 225 workgroups, each the chain of its loads,
// angles and sums; of 4 x 16800 rows 34 (104.3 MB, 3.1 TB/s: one thread adds a row's values for an axis while the
// workgroup waits), and 74 where uneven blocks make every chunk one pair, with 128 values to add (in one chain of
// additions in place of four side by side 93; 2 x 8400 rows of 16 heads of 128 74, now 55).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dcn.h"
#include "dcn_rotary.h"

namespace dcn {
namespace rotary {
namespace {

struct Args {
  const void* x;           // forward: x; backward: grad_out
  const void* x0;          // backward of positions: x
  void* out;               // out or grad_x (backward of positions: may be null)
  float* gp;               // [B][L][axes]
  Turns t;
  Cut cut;
  int64_t xs[3], x0s[3];   // strides of x and x0: batch, row, head
  uint32_t first;          // workgroups of launches before this one
  int rows;                // B * L
  int L, H, D;
  float sign;              // 1, or -1 to turn back
  bool near;               // near_by of x's strides
  // rotary_grad_kernel: chunks of a head, `turned` of them of pairs and the others copied
  int turned;
  Div by_row;              // chunks of a row
};

template <typename T, int WV, int PV, bool ADJ>
__global__ __launch_bounds__(256) void rotary_kernel(Args a) {
  extern __shared__ float2 cs[];
  __shared__ __attribute__((aligned(16))) unsigned char held[4 * kWave];
  const uint32_t at = a.first + blockIdx.x, block = at / a.cut.groups;
  const int row0 = static_cast<int>(block) * a.cut.rows, rows = min(a.cut.rows, a.rows - row0);
  const int h0 = static_cast<int>(at - block * a.cut.groups) * a.cut.heads, heads = min(a.cut.heads, a.H - h0);
  const int b0 = static_cast<int>(static_cast<uint32_t>(row0) / static_cast<uint32_t>(a.L)), l0 = row0 - b0 * a.L;
  const bool flat = a.near && l0 + rows <= a.L;        // (rows of one batch element)
  const T* const x = static_cast<const T*>(a.x) + b0 * a.xs[0] + l0 * a.xs[1] + h0 * a.xs[2];
  T* const out = static_cast<T*>(a.out) + (static_cast<int64_t>(row0) * a.H + h0) * a.D;
  // head i of the workgroup: its row and place there (the last group of heads may be smaller than the others)
  const auto row = [&](int i) { return a.cut.by_heads.of(i); };
  const auto head = [&](int i, int r) { return i - r * a.cut.heads; };
  turn_heads<T, WV, PV, ADJ>(
      a.t, a.cut, rows * a.cut.heads, reinterpret_cast<T*>(held + (threadIdx.x >> 6) * kWave), cs,
      [&](int i) {
        const int r = row(i), h = min(head(i, r), heads - 1);
        if (flat) return x + apart(r, static_cast<int>(a.xs[1]), h, static_cast<int>(a.xs[2]));
        const Row w = row_of(b0, l0, r, a.L);
        return static_cast<const T*>(a.x) + w.b * a.xs[0] + w.l * a.xs[1] + (h0 + h) * a.xs[2];
      },
      [&](int i) {
        const int r = row(i), h = head(i, r);
        // (a workgroup has a few thousand heads at most, one row where a row has several groups)
        return h < heads ? out + __umul24(__umul24(r, a.H) + h, a.D) : nullptr;
      },
      row,
      [&] {
        form_turns(a.t, a.cut.log_pairs, rows, a.sign, cs, [&](int r, int axis) {
          const Row w = row_of(b0, l0, r, a.L);
          return position_of(a.t, w.b, w.l, axis);
        });
        __syncthreads();
      });
}

template <typename T, int PV>
__device__ __forceinline__ Vec<T, PV> in_memory(const T* p) {
  using B = Bytes<PV * static_cast<int>(sizeof(T)), static_cast<int>(sizeof(T))>;
  return __builtin_bit_cast(Vec<T, PV>, static_cast<typename B::type>(*reinterpret_cast<const typename B::memory*>(p)));
}
template <typename T, int PV>
__device__ __forceinline__ void to_memory(T* p, const Vec<T, PV>& v) {
  using B = Bytes<PV * static_cast<int>(sizeof(T)), static_cast<int>(sizeof(T))>;
  *reinterpret_cast<typename B::memory*>(p) = __builtin_bit_cast(typename B::type, v);
}

// Chunks of a thread under way at a time, by the bytes of a vector.
constexpr int units_of(int bytes) { return bytes == 16 ? 2 : 4; }

template <typename T, int PV, bool ADJ>
__global__ __launch_bounds__(256) void rotary_grad_kernel(Args a) {
  using V = Vec<T, PV>;
  constexpr int kUnits = units_of(sizeof(V));
  extern __shared__ float2 cs[];
  __shared__ float red[4 * kUnits * 256];
  const int tid = threadIdx.x;
  const int row0 = static_cast<int>(a.first + blockIdx.x) * a.cut.rows, rows = min(a.cut.rows, a.rows - row0);
  const int b0 = static_cast<int>(static_cast<uint32_t>(row0) / static_cast<uint32_t>(a.L)), l0 = row0 - b0 * a.L;
  const int per = static_cast<int>(a.by_row.d), units = rows * per;
  float sum = 0.f;
  // the heads in groups, one after the other
  for (int h0 = 0; h0 < a.H; h0 += a.cut.heads) {
    V v1[kUnits], v2[kUnits], w1[kUnits], w2[kUnits];
    // Taken for unknown in every turn: places that were kept from one group of heads to the next cost 150 registers.
    int first = tid;
    asm volatile("" : "+v"(first));
    // unit k of this thread: its row of the workgroup, its head and chunk; false: none
    struct Unit {
      int r, h, chunk;
    };
    const auto unit = [&](int k, Unit& n) {
      const int u = k * 256 + first;
      n.r = a.by_row.of(u);
      const int in_row = u - n.r * per;
      n.h = a.cut.by_chunks.of(in_row);
      n.chunk = in_row - n.h * a.cut.chunks;
      n.h += h0;
      return u < units && n.h < a.H;
    };
    const auto place = [&](int chunk) {
      if (chunk < a.turned) return place_of<PV>(a.t, chunk * PV);
      const int e = 2 * a.t.pairs + (chunk - a.turned) * 2 * PV;
      return Place{e, e + PV};
    };
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      Unit n;
      if (!unit(k, n)) continue;
      const Place p = place(n.chunk);
      const Row w = row_of(b0, l0, n.r, a.L);
      const T* x = static_cast<const T*>(a.x) + w.b * a.xs[0] + w.l * a.xs[1] + n.h * a.xs[2];
      v1[k] = in_memory<T, PV>(x + p.e1);
      if (p.e2 < a.D) v2[k] = in_memory<T, PV>(x + p.e2);
      if (n.chunk < a.turned) {
        const T* x0 = static_cast<const T*>(a.x0) + w.b * a.x0s[0] + w.l * a.x0s[1] + n.h * a.x0s[2];
        w1[k] = in_memory<T, PV>(x0 + p.e1);
        w2[k] = in_memory<T, PV>(x0 + p.e2);
      }
    }
    if (h0 == 0) {
      form_turns(a.t, a.cut.log_pairs, rows, a.sign, cs, [&](int r, int axis) {
        const Row w = row_of(b0, l0, r, a.L);
        return position_of(a.t, w.b, w.l, axis);
      });
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      Unit n;
      const bool live = unit(k, n);
      float moved[4] = {0.f, 0.f, 0.f, 0.f};
      if (live) {
        const Place p = place(n.chunk);
        if (n.chunk < a.turned) {
          float c[PV], s[PV], x1[PV], x2[PV], y1[PV], y2[PV];
          const float2* turns = cs + n.r * a.t.pairs + n.chunk * PV;
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            c[j] = turns[j].x;
            s[j] = turns[j].y;
          }
          pairs_of<T, PV, ADJ>(v1[k], v2[k], x1, x2);
          turn<PV>(c, s, x1, x2, y1, y2);
          pairs_of<T, PV, ADJ>(w1[k], w2[k], x1, x2);
#pragma unroll
          for (int j = 0; j < PV; ++j) {
            const int pair = n.chunk * PV + j, axis = axis_of(a.t, pair);
            const float m = y2[j] * x1[j] - y1[j] * x2[j], f = a.t.freq[pair];
#pragma unroll
            for (int i = 0; i < 4; ++i) moved[i] = axis == i ? fmaf(f, m, moved[i]) : moved[i];   // (0 m could be NaN)
          }
          vectors_of<T, PV, ADJ>(y1, y2, v1[k], v2[k]);
        }
        if (a.out != nullptr) {
          T* y = static_cast<T*>(a.out) + (static_cast<int64_t>(row0 + n.r) * a.H + n.h) * a.D;
          to_memory<T, PV>(y + p.e1, v1[k]);
          if (p.e2 < a.D) to_memory<T, PV>(y + p.e2, v2[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < a.t.axes) red[i * kUnits * 256 + k * 256 + tid] = moved[i];
    }
    // thread i adds up row i / axes, axis i % axes
    __syncthreads();
    const int r = tid / a.t.axes, n = tid - r * a.t.axes;
    if (r < rows) {
      // (four sums side by side: a shorter chain, and fewer roundings on the way of each value)
      const float* p = red + n * kUnits * 256 + r * per;
      float part[4] = {0.f, 0.f, 0.f, 0.f};
      int u = 0;
      for (; u + 4 <= per; u += 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[i] += p[u + i];
      for (; u < per; ++u) part[0] += p[u];
      sum += (part[0] + part[1]) + (part[2] + part[3]);
    }
    __syncthreads();
  }
  if (tid < rows * a.t.axes) a.gp[static_cast<int64_t>(row0) * a.t.axes + tid] = sum;
}

// kernels for elements of a vector of memory and pairs of a chunk (one pair is two elements, whatever the layout)
template <typename T, int WV, int PV>
const void* turning_kernel(bool adjacent) {
  return adjacent && PV > 1 ? reinterpret_cast<const void*>(&rotary_kernel<T, WV, PV, (PV > 1)>)
                            : reinterpret_cast<const void*>(&rotary_kernel<T, WV, PV, false>);
}
const void* turning_kernel(bool bf16, int wv, int pv, bool adjacent) {
  if (bf16) {
    if (wv == 8) return pv == 8 ? turning_kernel<uint16_t, 8, 8>(adjacent) : pv == 2 ? turning_kernel<uint16_t, 8, 2>(adjacent)
                                                                                    : turning_kernel<uint16_t, 8, 1>(adjacent);
    if (wv == 2) return pv == 2 ? turning_kernel<uint16_t, 2, 2>(adjacent) : turning_kernel<uint16_t, 2, 1>(adjacent);
    return turning_kernel<uint16_t, 1, 1>(adjacent);
  }
  if (wv == 4) return pv == 4 ? turning_kernel<float, 4, 4>(adjacent) : turning_kernel<float, 4, 1>(adjacent);
  return turning_kernel<float, 1, 1>(adjacent);
}
template <typename T, int PV>
const void* grad_kernel(bool adjacent) {
  return adjacent && PV > 1 ? reinterpret_cast<const void*>(&rotary_grad_kernel<T, PV, (PV > 1)>)
                            : reinterpret_cast<const void*>(&rotary_grad_kernel<T, PV, false>);
}
const void* grad_kernel(bool bf16, int pv, bool adjacent) {
  if (bf16) return pv == 8 ? grad_kernel<uint16_t, 8>(adjacent) : pv == 2 ? grad_kernel<uint16_t, 2>(adjacent) : grad_kernel<uint16_t, 1>(adjacent);
  return pv == 4 ? grad_kernel<float, 4>(adjacent) : grad_kernel<float, 1>(adjacent);
}

// Rows of rotary_grad_kernel: as many as give each thread its chunks at a time (rows, heads of a group and chunks
// multiply to 256 units_of at most: a head has no more chunks than that), fewer where that leaves fewer than four
// workgroups a CU, down to a chunk for each thread.
void grad_cut(Args* a, int pv, int es) {
  Cut& c = a->cut;
  a->turned = a->t.pairs / pv;
  c.chunks = a->turned + (a->D - 2 * a->t.pairs + 2 * pv - 1) / (2 * pv);
  const int most = units_of(pv * es) * 256;
  c.heads = std::max(1, std::min(a->H, most / c.chunks));
  const int per = c.heads * c.chunks;
  int rows = std::min(most / per, kTurns / a->t.pairs);
  rows = std::min(rows, std::max(a->rows / 1024, (255 + per) / per));
  c.rows = std::max(1, std::min(rows, 64));
  a->by_row = div_by(per);
  c.by_chunks = div_by(c.chunks);
  c.log_pairs = 0;
  while (c.log_pairs < 8 && (1 << c.log_pairs) < a->t.pairs) ++c.log_pairs;
}

int check(const dcn_rotary_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  if (d->batch < 0 || d->length < 0 || d->heads < 1 || d->head_dim < 1 || d->axes < 1) return DCN_E_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->x_stride[i] < 0) return DCN_E_ARG;
  const int rc = check_turns(d->axes, d->sections, d->layout, d->position_type, d->position_stride, d->head_dim);
  if (rc != DCN_OK) return rc;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  const double big = 2147483648.;
  if (d->head_dim > kMostD || static_cast<double>(d->batch) * d->length * d->heads >= big || d->batch >= big ||
      d->length >= big || d->heads >= big)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

int run(const dcn_rotary_desc* d, Args* a, const void* positions, const float* frequencies, hipStream_t stream) {
  const bool bf16 = d->dtype == DCN_BF16, adjacent = d->layout == DCN_ROTARY_ADJACENT;
  const int es = bf16 ? 2 : 4;
  a->t = turns_of(d->axes, d->sections, d->layout, d->position_type, d->position_stride, positions, frequencies);
  a->L = static_cast<int>(d->length);
  a->H = static_cast<int>(d->heads);
  a->D = static_cast<int>(d->head_dim);
  a->rows = static_cast<int>(d->batch * d->length);
  const int w = vector_of(d->head_dim, es);
  const int pv = pairs_at_once(a->t, d->sections, w, es);
  const void* fn;
  if (a->gp != nullptr) {
    grad_cut(a, pv, es);
    a->cut.groups = 1;
    fn = grad_kernel(bf16, pv, adjacent);
  } else {
    a->cut = cut_of(w, pv, es, a->t.pairs, d->head_dim, a->rows, d->heads);
    a->near = near_by(a->cut.rows, a->xs[1], a->cut.heads, a->xs[2]);
    fn = turning_kernel(bf16, w, pv, adjacent);
  }
  void* args[] = {a};
  return launch(fn, (static_cast<int64_t>(a->rows) + a->cut.rows - 1) / a->cut.rows * a->cut.groups, args,
                turns_bytes(a->cut, a->t), &a->first, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

}  // namespace
}  // namespace rotary
}  // namespace dcn

extern "C" int dcn_rotary(const dcn_rotary_desc* d, const void* x, const void* positions, const float* frequencies,
                          void* out, hipStream_t stream) {
  using namespace dcn::rotary;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->length == 0) return DCN_OK;
  if (x == nullptr || positions == nullptr || frequencies == nullptr || out == nullptr) return DCN_E_ARG;
  Args a{};
  a.x = x;
  a.out = out;
  for (int i = 0; i < 3; ++i) a.xs[i] = d->x_stride[i];
  a.sign = 1.f;
  return run(d, &a, positions, frequencies, stream);
}

extern "C" int dcn_rotary_backward(const dcn_rotary_desc* d, const void* grad_out, const void* positions,
                                   const float* frequencies, const void* x, void* grad_x, float* grad_positions,
                                   hipStream_t stream) {
  using namespace dcn::rotary;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->length == 0) return DCN_OK;
  if (grad_out == nullptr || positions == nullptr || frequencies == nullptr ||
      (grad_positions != nullptr && x == nullptr))
    return DCN_E_ARG;
  if (grad_x == nullptr && grad_positions == nullptr) return DCN_OK;
  Args a{};
  a.x = grad_out;
  a.out = grad_x;
  a.gp = grad_positions;
  a.xs[2] = d->head_dim;
  a.xs[1] = d->heads * a.xs[2];
  a.xs[0] = d->length * a.xs[1];
  if (grad_positions != nullptr) {
    a.x0 = x;
    for (int i = 0; i < 3; ++i) a.x0s[i] = d->x_stride[i];
  }
  a.sign = -1.f;
  return run(d, &a, positions, frequencies, stream);
}

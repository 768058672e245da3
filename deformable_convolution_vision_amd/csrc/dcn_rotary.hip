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
// For the position's gradient a workgroup has all heads of its rows, and each unit leaves its sum for each
// axis in the LDS, where one thread for each row and axis adds them in order.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dcn.h"
#include "dcn_rotary.h"

namespace dcn {
namespace rotary {
namespace {

struct Args {
  const void* x;           // forward: x; backward: grad_out
  const void* x0;          // backward of positions: x
  void* out;               // out or grad_x (backward: may be null)
  float* gp;               // [B][L][axes]
  Turns t;
  Cut cut;
  int64_t xs[3], x0s[3];   // strides of x and x0: batch, row, head
  int64_t rows, first;     // B * L; workgroups of launches before this one
  int L, H, D;
  float sign;              // 1, or -1 to turn back
};

template <typename T, int PV, bool ADJ, bool POS>
__global__ __launch_bounds__(256) void rotary_kernel(Args a) {
  using V = Vec<T, PV>;
  constexpr int kUnits = units_of(sizeof(V));
  __shared__ float2 cs[kTurns];
  __shared__ float red[POS ? 4 * kUnits * 256 : 1];
  const int tid = threadIdx.x;
  const int64_t at = a.first + blockIdx.x, row0 = (POS ? at : at / a.cut.groups) * a.cut.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.cut.rows), a.rows - row0));
  // the heads of this workgroup; for the position's gradient one group of them after the other
  const int g0 = POS ? 0 : static_cast<int>(at % a.cut.groups), g1 = POS ? a.cut.groups : g0 + 1;
  float sum = 0.f;
  for (int g = g0; g < g1; ++g) {
    const int h0 = g * a.cut.heads, heads = min(a.cut.heads, a.H - h0);
    const int units = rows * static_cast<int>(a.cut.by_row.d);
    for (int u0 = 0; u0 < units; u0 += kUnits * 256) {
      V v1[kUnits], v2[kUnits], w1[POS ? kUnits : 1], w2[POS ? kUnits : 1];
      const auto unit = [&](int k, int& r, int& h, int& chunk) {   // false: no unit
        const int u = u0 + k * 256 + tid;
        r = a.cut.by_row.of(u);
        const int in_row = u - r * static_cast<int>(a.cut.by_row.d);
        h = a.cut.by_chunks.of(in_row);
        chunk = in_row - h * a.cut.chunks;
        return u < units && h < heads;
      };
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        int r, h, chunk;
        if (!unit(k, r, h, chunk)) continue;
        const uint32_t row = static_cast<uint32_t>(row0 + r), b = row / static_cast<uint32_t>(a.L), l = row - b * a.L;
        const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
        const T* x = static_cast<const T*>(a.x) + b * a.xs[0] + l * a.xs[1] + (h0 + h) * a.xs[2];
        v1[k] = *reinterpret_cast<const V*>(x + p.e1);
        if (p.e2 < a.D) v2[k] = *reinterpret_cast<const V*>(x + p.e2);
        if (POS && chunk < a.cut.rotated) {
          const T* x0 = static_cast<const T*>(a.x0) + b * a.x0s[0] + l * a.x0s[1] + (h0 + h) * a.x0s[2];
          w1[k] = *reinterpret_cast<const V*>(x0 + p.e1);
          w2[k] = *reinterpret_cast<const V*>(x0 + p.e2);
        }
      }
      if (g == g0 && u0 == 0) {
        for (int i = tid; i < rows * a.t.pairs; i += 256) {
          const int r = a.cut.by_pairs.of(i), pair = i - r * a.t.pairs;
          const uint32_t row = static_cast<uint32_t>(row0 + r), b = row / static_cast<uint32_t>(a.L), l = row - b * a.L;
          float c, s;
          cos_sin(position_of(a.t, b, l, axis_of(a.t, pair)), a.t.freq[pair], c, s);
          cs[i] = make_float2(c, a.sign * s);
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        int r, h, chunk;
        const bool live = unit(k, r, h, chunk);
        float moved[4] = {0.f, 0.f, 0.f, 0.f};
        if (live) {
          const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
          if (chunk < a.cut.rotated) {
            float c[PV], s[PV], x1[PV], x2[PV], y1[PV], y2[PV];
            const float2* turns = cs + r * a.t.pairs + chunk * PV;
#pragma unroll
            for (int j = 0; j < PV; ++j) {
              c[j] = turns[j].x;
              s[j] = turns[j].y;
            }
            pairs_of<T, PV, ADJ>(v1[k], v2[k], x1, x2);
            turn<PV>(c, s, x1, x2, y1, y2);
            if (POS) {
              pairs_of<T, PV, ADJ>(w1[k], w2[k], x1, x2);
#pragma unroll
              for (int j = 0; j < PV; ++j) {
                const int pair = chunk * PV + j, axis = axis_of(a.t, pair);
                const float m = a.t.freq[pair] * (y2[j] * x1[j] - y1[j] * x2[j]);
#pragma unroll
                for (int n = 0; n < 4; ++n) moved[n] += axis == n ? m : 0.f;
              }
            }
            vectors_of<T, PV, ADJ>(y1, y2, v1[k], v2[k]);
          }
          if (!POS || a.out != nullptr) {
            T* y = static_cast<T*>(a.out) + ((row0 + r) * a.H + h0 + h) * a.D;
            *reinterpret_cast<V*>(y + p.e1) = v1[k];
            if (p.e2 < a.D) *reinterpret_cast<V*>(y + p.e2) = v2[k];
          }
        }
        if constexpr (POS) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
            if (n < a.t.axes) red[n * kUnits * 256 + k * 256 + tid] = moved[n];
        }
      }
      if constexpr (POS) {
        // thread i adds up row i / axes, axis i % axes: the units of this turn that are the row's
        __syncthreads();
        const int r = tid / a.t.axes, n = tid - r * a.t.axes, per = static_cast<int>(a.cut.by_row.d);
        if (r < rows)
          for (int u = max(r * per, u0); u < min((r + 1) * per, u0 + kUnits * 256); ++u) sum += red[n * kUnits * 256 + u - u0];
        __syncthreads();
      }
    }
  }
  if constexpr (POS) {
    if (tid < rows * a.t.axes) a.gp[row0 * a.t.axes + tid] = sum;
  }
}

template <typename T, int PV>
const void* kernel_of(bool adjacent, bool positions) {
  if (positions)
    return adjacent ? reinterpret_cast<const void*>(&rotary_kernel<T, PV, true, true>)
                    : reinterpret_cast<const void*>(&rotary_kernel<T, PV, false, true>);
  return adjacent ? reinterpret_cast<const void*>(&rotary_kernel<T, PV, true, false>)
                  : reinterpret_cast<const void*>(&rotary_kernel<T, PV, false, false>);
}
const void* kernel_of(bool bf16, int width, bool adjacent, bool positions) {
  if (bf16)
    return width == 8   ? kernel_of<uint16_t, 8>(adjacent, positions)
           : width == 4 ? kernel_of<uint16_t, 4>(adjacent, positions)
           : width == 2 ? kernel_of<uint16_t, 2>(adjacent, positions)
                        : kernel_of<uint16_t, 1>(false, positions);   // (one pair: two elements, whatever the layout)
  return width == 4   ? kernel_of<float, 4>(adjacent, positions)
         : width == 2 ? kernel_of<float, 2>(adjacent, positions)
                      : kernel_of<float, 1>(false, positions);
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
  if (d->head_dim > 2 * kTurns || static_cast<double>(d->batch) * d->length * d->heads >= big || d->batch >= big ||
      d->length >= big || d->heads >= big)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

int run(const dcn_rotary_desc* d, Args* a, const void* positions, const float* frequencies, hipStream_t stream) {
  const bool bf16 = d->dtype == DCN_BF16, adjacent = d->layout == DCN_ROTARY_ADJACENT;
  const int es = bf16 ? 2 : 4;
  a->t = turns_of(d->axes, d->sections, d->layout, d->position_type, d->position_stride, positions, frequencies);
  a->rows = d->batch * d->length;
  a->L = static_cast<int>(d->length);
  a->H = static_cast<int>(d->heads);
  a->D = static_cast<int>(d->head_dim);
  int w = fit(fit(width_of(a->t, d->sections, d->head_dim, es), es, a->x), es, a->out);
  w = fit(w, a->xs, 3);
  if (a->x0 != nullptr) w = fit(fit(w, es, a->x0), a->x0s, 3);
  a->cut = cut_of(w, es, a->t.pairs, d->head_dim, a->rows, d->heads);
  void* args[] = {a};
  const int64_t groups = a->gp != nullptr ? 1 : a->cut.groups;
  return launch(kernel_of(bf16, w, adjacent, a->gp != nullptr), (a->rows + a->cut.rows - 1) / a->cut.rows * groups, args,
                &a->first, stream)
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

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
// A workgroup takes whole rows, so a row's sum over its heads stays in it: threads leave their sums
// in the LDS and one thread for each row and axis adds them in order.

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

constexpr int kHeads = 4;  // heads under way at a time

template <typename T, int PV, bool ADJ, bool POS>
__global__ __launch_bounds__(256) void rotary_kernel(Args a) {
  __shared__ float red[POS ? 4 * 256 : 1];
  const int tid = threadIdx.x, r = tid / a.cut.units, u0 = tid - r * a.cut.units;
  const int64_t row = (a.first + blockIdx.x) * a.cut.rows + r;
  const bool live = r < a.cut.rows && row < a.rows;
  float sums[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const int b = static_cast<int>(row / a.L), l = static_cast<int>(row - static_cast<int64_t>(b) * a.L);
    const At at = at_row(a.t, b, l);
    const T* const xr = static_cast<const T*>(a.x) + b * a.xs[0] + l * a.xs[1];
    const T* const x0r = POS ? static_cast<const T*>(a.x0) + b * a.x0s[0] + l * a.x0s[1] : nullptr;
    T* const yr = static_cast<T*>(a.out) + row * a.H * a.D;
    for (int u = u0; u < a.cut.units; u += 256) {   // once, unless a row has more units than a workgroup threads
      const int chunk = u % a.cut.chunks, group = u / a.cut.chunks;
      const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
      const bool turns = chunk < a.cut.rotated, second = p.e2 < a.D;
      float c[PV], s[PV], f[PV], moved[PV];
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        c[j] = 1.f;
        s[j] = f[j] = moved[j] = 0.f;
      }
      if (turns) {
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          f[j] = a.t.freq[chunk * PV + j];
          cos_sin(at.of(a.t, chunk * PV + j), f[j], c[j], s[j]);
          s[j] *= a.sign;
        }
      }
      using V = Vec<T, PV>;
      for (int h0 = group; h0 < a.H; h0 += kHeads * a.cut.groups) {
        V v1[kHeads], v2[kHeads], w1[kHeads], w2[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          const int h = h0 + i * a.cut.groups;
          if (h >= a.H) break;
          const T* x = xr + h * a.xs[2];
          v1[i] = *reinterpret_cast<const V*>(x + p.e1);
          if (second) v2[i] = *reinterpret_cast<const V*>(x + p.e2);
          if (POS && turns) {
            const T* x0 = x0r + h * a.x0s[2];
            w1[i] = *reinterpret_cast<const V*>(x0 + p.e1);
            w2[i] = *reinterpret_cast<const V*>(x0 + p.e2);
          }
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
          const int h = h0 + i * a.cut.groups;
          if (h >= a.H) break;
          T* y = yr + static_cast<int64_t>(h) * a.D;
          if (turns) {
            float x1[PV], x2[PV], y1[PV], y2[PV];
            pairs_of<T, PV, ADJ>(v1[i], v2[i], x1, x2);
            turn<PV>(c, s, x1, x2, y1, y2);
            if (POS) {
              float o1[PV], o2[PV];
              pairs_of<T, PV, ADJ>(w1[i], w2[i], o1, o2);
#pragma unroll
              for (int j = 0; j < PV; ++j) moved[j] += y2[j] * o1[j] - y1[j] * o2[j];
            }
            vectors_of<T, PV, ADJ>(y1, y2, v1[i], v2[i]);
          }
          if (!POS || a.out != nullptr) {
            *reinterpret_cast<V*>(y + p.e1) = v1[i];
            if (second) *reinterpret_cast<V*>(y + p.e2) = v2[i];
          }
        }
      }
      if (POS && turns) {
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          const int pair = chunk * PV + j, axis = (pair >= a.t.end[0]) + (pair >= a.t.end[1]) + (pair >= a.t.end[2]);
#pragma unroll
          for (int n = 0; n < 4; ++n) sums[n] += axis == n ? f[j] * moved[j] : 0.f;
        }
      }
    }
  }
  if constexpr (POS) {
#pragma unroll
    for (int n = 0; n < 4; ++n) red[n * 256 + tid] = sums[n];
    __syncthreads();
    const int units = min(a.cut.units, 256);
    for (int i = tid; i < a.cut.rows * a.t.axes; i += 256) {
      const int rr = i / a.t.axes, n = i - rr * a.t.axes;
      const int64_t to = (a.first + blockIdx.x) * a.cut.rows + rr;
      if (to >= a.rows) break;
      float sum = 0.f;
      for (int u = 0; u < units; ++u) sum += red[n * 256 + rr * units + u];
      a.gp[to * a.t.axes + n] = sum;
    }
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
  if (d->head_dim > 65536 || static_cast<double>(d->batch) * d->length * d->heads >= big || d->batch >= big ||
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
  a->cut = cut_of(w, a->t.pairs, d->head_dim, a->rows, d->heads);
  void* args[] = {a};
  return launch(kernel_of(bf16, w, adjacent, a->gp != nullptr), (a->rows + a->cut.rows - 1) / a->cut.rows, args,
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

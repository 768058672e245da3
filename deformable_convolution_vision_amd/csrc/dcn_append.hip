// dcn_append.hip -- gfx950 append of new keys and values to a cache in pages, rotated on the way,
// and the rotation of the same tokens' queries.
//
// Row (b, i) of the new tokens is position s = starts[b] + i of its sequence: row s % page_size of
// page page_table[b][s / page_size].  Queries, keys and values are one list of heads of that row: a
// thread forms the angles of its chunk of pairs once and turns that chunk of several heads (values
// are copied).  Nothing is read before the row's page is known but the row itself, whose loads
// are under way while the start and the table entry are fetched.
//
// A table entry that is no page of the cache, or a position outside the table, drops the row: the
// check stands before the address is formed.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dcn.h"
#include "dcn_rotary.h"

namespace dcn {
namespace rotary {
namespace {

struct AppendArgs {
  const void *q, *k, *v;
  void *qo, *kp, *vp;
  const int32_t *table, *starts, *counts;
  int32_t* lengths;
  Turns t;
  Cut cut;
  int64_t qs[3], ks[3], vs[3], kps[3], vps[3], ts;
  int64_t rows, first;     // B * max(L, 1); workgroups of launches before this one
  int L, per;              // rows of a sequence, and max(L, 1)
  int Hq, Hkv, D;
  int num_pages, page_size, max_pages;
};

constexpr int kHeads = 4;  // heads under way at a time

template <typename T, int PV, bool ADJ>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  using V = Vec<T, PV>;
  const int tid = threadIdx.x, r = tid / a.cut.units, u0 = tid - r * a.cut.units;
  const int64_t row = (a.first + blockIdx.x) * a.cut.rows + r;
  if (r >= a.cut.rows || row >= a.rows) return;
  const int b = static_cast<int>(row / a.per), i = static_cast<int>(row - static_cast<int64_t>(b) * a.per);
  const int start = a.starts[b];
  int count = a.L;
  if (a.counts != nullptr) count = min(max(a.counts[b], 0), a.L);
  if (i == 0 && u0 == 0 && a.lengths != nullptr) a.lengths[b] = start + count;
  if (i >= a.L) return;
  const int64_t s = static_cast<int64_t>(start) + i;
  int page = -1, place = 0;
  if (i < count && s >= 0 && s < static_cast<int64_t>(a.max_pages) * a.page_size) {
    const int at = static_cast<int>(s) / a.page_size;
    place = static_cast<int>(s) - at * a.page_size;
    page = a.table[b * a.ts + at];
  }
  const bool kept = page >= 0 && page < a.num_pages;
  const T* const qr = static_cast<const T*>(a.q) + b * a.qs[0] + i * a.qs[1];
  const T* const kr = static_cast<const T*>(a.k) + b * a.ks[0] + i * a.ks[1];
  const T* const vr = static_cast<const T*>(a.v) + b * a.vs[0] + i * a.vs[1];
  T* const qo = static_cast<T*>(a.qo) + row * a.Hq * a.D;   // (rows are B * L here: per == L)
  T* const ko = static_cast<T*>(a.kp) + (kept ? page * a.kps[0] + place * a.kps[1] : 0);
  T* const vo = static_cast<T*>(a.vp) + (kept ? page * a.vps[0] + place * a.vps[1] : 0);
  At at;
  if (a.t.axes > 0 && a.t.positions != nullptr) {
    at = at_row(a.t, b, i);
  } else {
    at.p0 = at.p1 = at.p2 = at.p3 = static_cast<double>(s);
  }
  const int heads = a.Hq + 2 * a.Hkv;
  for (int u = u0; u < a.cut.units; u += 256) {
    const int chunk = u % a.cut.chunks, group = u / a.cut.chunks;
    const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
    const bool turns = chunk < a.cut.rotated, second = p.e2 < a.D;
    float c[PV], sn[PV];
    if (turns) {
#pragma unroll
      for (int j = 0; j < PV; ++j) cos_sin(at.of(a.t, chunk * PV + j), a.t.freq[chunk * PV + j], c[j], sn[j]);
    }
    for (int h0 = group; h0 < heads; h0 += kHeads * a.cut.groups) {
      V v1[kHeads], v2[kHeads];
#pragma unroll
      for (int n = 0; n < kHeads; ++n) {
        const int h = h0 + n * a.cut.groups;
        if (h >= heads) break;
        const T* x = h < a.Hq             ? qr + h * a.qs[2]
                     : h < a.Hq + a.Hkv ? kr + (h - a.Hq) * a.ks[2]
                                        : vr + (h - a.Hq - a.Hkv) * a.vs[2];
        v1[n] = *reinterpret_cast<const V*>(x + p.e1);
        if (second) v2[n] = *reinterpret_cast<const V*>(x + p.e2);
      }
#pragma unroll
      for (int n = 0; n < kHeads; ++n) {
        const int h = h0 + n * a.cut.groups;
        if (h >= heads) break;
        T* y = h < a.Hq             ? qo + static_cast<int64_t>(h) * a.D
               : h < a.Hq + a.Hkv ? ko + (h - a.Hq) * a.kps[2]
                                  : vo + (h - a.Hq - a.Hkv) * a.vps[2];
        if (turns && h < a.Hq + a.Hkv) {
          float x1[PV], x2[PV], y1[PV], y2[PV];
          pairs_of<T, PV, ADJ>(v1[n], v2[n], x1, x2);
          turn<PV>(c, sn, x1, x2, y1, y2);
          vectors_of<T, PV, ADJ>(y1, y2, v1[n], v2[n]);
        }
        if (h < a.Hq || kept) {
          *reinterpret_cast<V*>(y + p.e1) = v1[n];
          if (second) *reinterpret_cast<V*>(y + p.e2) = v2[n];
        }
      }
    }
  }
}

template <typename T, int PV>
const void* kernel_of(bool adjacent) {
  return adjacent ? reinterpret_cast<const void*>(&append_kernel<T, PV, true>)
                  : reinterpret_cast<const void*>(&append_kernel<T, PV, false>);
}
const void* kernel_of(bool bf16, int width, bool adjacent) {
  if (bf16)
    return width == 8   ? kernel_of<uint16_t, 8>(adjacent)
           : width == 4 ? kernel_of<uint16_t, 4>(adjacent)
           : width == 2 ? kernel_of<uint16_t, 2>(adjacent)
                        : kernel_of<uint16_t, 1>(false);
  return width == 4 ? kernel_of<float, 4>(adjacent) : width == 2 ? kernel_of<float, 2>(adjacent) : kernel_of<float, 1>(false);
}

int check(const dcn_append_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  if (d->batch < 0 || d->length < 0 || d->query_heads < 0 || d->key_heads < 1 || d->head_dim < 1 || d->num_pages < 0 ||
      d->page_size < 1 || d->max_pages < 0 || d->table_stride < 0)
    return DCN_E_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0 || d->key_page_stride[i] < 0 ||
        d->value_page_stride[i] < 0)
      return DCN_E_ARG;
  const int rc = check_turns(d->axes, d->sections, d->layout, d->position_type, d->position_stride, d->head_dim);
  if (rc != DCN_OK) return rc;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  const double big = 2147483647.;
  const double heads = static_cast<double>(d->query_heads) + 2. * d->key_heads, length = d->length > 0 ? d->length : 1;
  if (d->head_dim > 65536 || heads > big || d->batch > big || length > big || d->batch * length * heads > big ||
      d->num_pages > big || d->page_size > big || static_cast<double>(d->max_pages) * d->page_size > big)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

}  // namespace
}  // namespace rotary
}  // namespace dcn

extern "C" int dcn_paged_append(const dcn_append_desc* d, const void* q, const void* k, const void* v,
                                const void* positions, const float* frequencies, const int32_t* page_table,
                                const int32_t* starts, const int32_t* counts, void* q_out, void* key_pages,
                                void* value_pages, int32_t* lengths, hipStream_t stream) {
  using namespace dcn::rotary;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0) return DCN_OK;
  const bool rows = d->length > 0, cache = rows && d->num_pages > 0 && d->max_pages > 0;
  if (starts == nullptr || (rows && (k == nullptr || v == nullptr)) ||
      (cache && (key_pages == nullptr || value_pages == nullptr || page_table == nullptr)) ||
      (rows && d->query_heads > 0 && (q == nullptr || q_out == nullptr)) ||
      (rows && d->axes > 0 && frequencies == nullptr) || (lengths != nullptr && (lengths == starts || lengths == counts)))
    return DCN_E_ARG;
  if (!rows && lengths == nullptr) return DCN_OK;
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.kp = key_pages;
  a.vp = value_pages;
  a.table = page_table;
  a.starts = starts;
  a.counts = counts;
  a.lengths = lengths;
  for (int i = 0; i < 3; ++i) {
    a.qs[i] = d->q_stride[i];
    a.ks[i] = d->k_stride[i];
    a.vs[i] = d->v_stride[i];
    a.kps[i] = d->key_page_stride[i];
    a.vps[i] = d->value_page_stride[i];
  }
  a.ts = d->table_stride;
  a.L = static_cast<int>(d->length);
  a.per = rows ? a.L : 1;
  a.rows = d->batch * a.per;
  a.Hq = static_cast<int>(d->query_heads);
  a.Hkv = static_cast<int>(d->key_heads);
  a.D = static_cast<int>(d->head_dim);
  a.num_pages = cache ? static_cast<int>(d->num_pages) : 0;
  a.page_size = static_cast<int>(d->page_size);
  a.max_pages = cache ? static_cast<int>(d->max_pages) : 0;
  a.t = turns_of(d->axes, d->sections, d->layout, d->position_type, d->position_stride, positions, frequencies);
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  int w = width_of(a.t, d->sections, d->head_dim, es);
  for (const void* p : {k, v, static_cast<const void*>(key_pages), static_cast<const void*>(value_pages)}) w = fit(w, es, p);
  for (const int64_t* s : {a.ks, a.vs, a.kps, a.vps}) w = fit(w, s, 3);
  if (a.Hq > 0) w = fit(fit(fit(w, es, q), es, q_out), a.qs, 3);
  a.cut = cut_of(w, a.t.pairs, d->head_dim, a.rows, a.Hq + 2 * a.Hkv);
  void* args[] = {&a};
  return launch(kernel_of(bf16, w, d->layout == DCN_ROTARY_ADJACENT), (a.rows + a.cut.rows - 1) / a.cut.rows, args,
                &a.first, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

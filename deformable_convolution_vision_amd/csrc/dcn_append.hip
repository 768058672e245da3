// dcn_append.hip -- gfx950 append of new keys and values to a cache in pages, rotated on the way,
// and the rotation of the same tokens' queries.
//
// Row (b, i) of the new tokens is position s = starts[b] + i of its sequence: row s % page_size of
// page page_table[b][s / page_size].  Queries, keys and values are one list of heads of that row, of which
// values are copied.  A workgroup's rows share their angles and places in the LDS; the elements' loads are
// under way while starts, table entries and angles are found.
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

template <typename T, int PV, bool ADJ>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  using V = Vec<T, PV>;
  constexpr int kUnits = units_of(sizeof(V));
  __shared__ float2 cs[kTurns];
  __shared__ int pages[kRows], places[kRows];      // of the rows; page -1: the row has none
  const int tid = threadIdx.x;
  const int64_t at = a.first + blockIdx.x, row0 = at / a.cut.groups * a.cut.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.cut.rows), a.rows - row0));
  const int h0 = static_cast<int>(at % a.cut.groups) * a.cut.heads, heads = min(a.cut.heads, a.Hq + 2 * a.Hkv - h0);
  const int units = a.L > 0 ? rows * static_cast<int>(a.cut.by_row.d) : 0;
  const auto unit = [&](int u, int& r, int& h, int& chunk) {   // false: no unit
    r = a.cut.by_row.of(u);
    const int in_row = u - r * static_cast<int>(a.cut.by_row.d);
    h = a.cut.by_chunks.of(in_row);
    chunk = in_row - h * a.cut.chunks;
    const bool live = u < units && h < heads;
    h += h0;
    return live;
  };
  V v1[kUnits], v2[kUnits];
  const auto load = [&](int u0) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int r, h, chunk;
      if (!unit(u0 + k * 256 + tid, r, h, chunk)) continue;
      const uint32_t row = static_cast<uint32_t>(row0 + r), b = row / static_cast<uint32_t>(a.per), i = row - b * a.per;
      const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
      const T* x = h < a.Hq           ? static_cast<const T*>(a.q) + b * a.qs[0] + i * a.qs[1] + h * a.qs[2]
                   : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + b * a.ks[0] + i * a.ks[1] + (h - a.Hq) * a.ks[2]
                                      : static_cast<const T*>(a.v) + b * a.vs[0] + i * a.vs[1] + (h - a.Hq - a.Hkv) * a.vs[2];
      v1[k] = *reinterpret_cast<const V*>(x + p.e1);
      if (p.e2 < a.D) v2[k] = *reinterpret_cast<const V*>(x + p.e2);
    }
  };
  load(0);
  for (int r = tid; r < rows; r += 256) {
    const uint32_t row = static_cast<uint32_t>(row0 + r), b = row / static_cast<uint32_t>(a.per), i = row - b * a.per;
    const int start = a.starts[b];
    int count = a.L, page = -1, place = 0;
    if (a.counts != nullptr) count = min(max(a.counts[b], 0), a.L);
    if (i == 0 && h0 == 0 && a.lengths != nullptr) a.lengths[b] = start + count;
    const int64_t s = static_cast<int64_t>(start) + i;
    if (static_cast<int>(i) < count && s >= 0 && s < static_cast<int64_t>(a.max_pages) * a.page_size) {
      const int n = static_cast<int>(s) / a.page_size;
      place = static_cast<int>(s) - n * a.page_size;
      page = a.table[b * a.ts + n];
    }
    pages[r] = page >= 0 && page < a.num_pages ? page : -1;
    places[r] = place;
  }
  if (units == 0) return;
  for (int i = tid; i < rows * a.t.pairs; i += 256) {
    const int r = a.cut.by_pairs.of(i), pair = i - r * a.t.pairs;
    const uint32_t row = static_cast<uint32_t>(row0 + r), b = row / static_cast<uint32_t>(a.per), l = row - b * a.per;
    const double pos = a.t.positions != nullptr ? position_of(a.t, b, l, axis_of(a.t, pair))
                                                : static_cast<double>(static_cast<int64_t>(a.starts[b]) + l);
    float c, s;
    cos_sin(pos, a.t.freq[pair], c, s);
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  for (int u0 = 0; u0 < units; u0 += kUnits * 256) {
    if (u0 > 0) load(u0);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int r, h, chunk;
      if (!unit(u0 + k * 256 + tid, r, h, chunk)) continue;
      const Place p = place_of<PV>(a.t, chunk, a.cut.rotated);
      const int page = pages[r], place = places[r];
      T* y = h < a.Hq           ? static_cast<T*>(a.qo) + ((row0 + r) * a.Hq + h) * a.D
             : h < a.Hq + a.Hkv ? static_cast<T*>(a.kp) + page * a.kps[0] + place * a.kps[1] + (h - a.Hq) * a.kps[2]
                                : static_cast<T*>(a.vp) + page * a.vps[0] + place * a.vps[1] + (h - a.Hq - a.Hkv) * a.vps[2];
      if (chunk < a.cut.rotated && h < a.Hq + a.Hkv) {
        float c[PV], s[PV], x1[PV], x2[PV], y1[PV], y2[PV];
        const float2* turns = cs + r * a.t.pairs + chunk * PV;
#pragma unroll
        for (int j = 0; j < PV; ++j) {
          c[j] = turns[j].x;
          s[j] = turns[j].y;
        }
        pairs_of<T, PV, ADJ>(v1[k], v2[k], x1, x2);
        turn<PV>(c, s, x1, x2, y1, y2);
        vectors_of<T, PV, ADJ>(y1, y2, v1[k], v2[k]);
      }
      if (h < a.Hq || page >= 0) {
        *reinterpret_cast<V*>(y + p.e1) = v1[k];
        if (p.e2 < a.D) *reinterpret_cast<V*>(y + p.e2) = v2[k];
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
  if (d->head_dim > 2 * kTurns || heads > big || d->batch > big || length > big || d->batch * length * heads > big ||
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
  a.cut = cut_of(w, es, a.t.pairs, d->head_dim, a.rows, a.Hq + 2 * a.Hkv);
  void* args[] = {&a};
  return launch(kernel_of(bf16, w, d->layout == DCN_ROTARY_ADJACENT),
                (a.rows + a.cut.rows - 1) / a.cut.rows * a.cut.groups, args, &a.first, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

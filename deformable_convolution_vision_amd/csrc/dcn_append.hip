// dcn_append.hip -- gfx950 append of new keys and values to a cache in pages, rotated on the way,
// and the rotation of the same tokens' queries.
//
// Row (b, i) of the new tokens is position s = starts[b] + i of its sequence: row s % page_size of
// page page_table[b][s / page_size].  Queries, keys and values are one list of heads of that row, of which
// values are not turned.  A workgroup's rows share their angles and places in the LDS; the first elements'
// loads are under way while starts, table entries and angles are found (turn_heads).
//
// A table entry that is no page of the cache, or a position outside the table, drops the row: the
// check stands before the address is formed.
//
// Memory bounds a prompt: 8 x 4200 rows, ragged, of 16 + 4 + 4 heads of 128, bf16, take 71 to 73 us for 340.7 MB, 4.7 to 4.8 TB/s (a
// large copy 4.99).  Whole turns of a workgroup's waves (cut_of) took as many rows without gaps from 108 us to 90, rows
// without tokens that are not read the ragged ones from 86 to 84, addresses in 24-bit products (apart) these to 73 and
// those to 82.  One token of eight sequences takes 5.3 us, a chain from its start and table
// entry to its address.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dcn.h"
#include "dcn_rotary.h"

namespace dcn {
namespace rotary {
namespace {

constexpr int kRows = 256;   // the most rows of a workgroup

struct AppendArgs {
  const void *q, *k, *v;
  void *qo, *kp, *vp;
  const int32_t *table, *starts, *counts;
  int32_t* lengths;
  Turns t;
  Cut cut;
  int64_t qs[3], ks[3], vs[3], kps[3], vps[3], ts;
  uint32_t first;          // workgroups of launches before this one
  int rows;                // B * max(L, 1)
  int L, per;              // rows of a sequence, and max(L, 1)
  int Hq, Hkv, D;
  int num_pages, page_size, max_pages;
  bool near;               // near_by of q's, k's and v's strides, and of the pages' heads
};

// One of two values, both at hand (choosing between places of them would put the kernel's arguments into memory).
template <typename V>
__device__ __forceinline__ V pick(bool first, V x, V y) {
  return first ? x : y;
}

template <typename T, int WV, int PV, bool ADJ>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  extern __shared__ float2 cs[];
  __shared__ __attribute__((aligned(16))) unsigned char held[4 * kWave];
  __shared__ int64_t places[2][kRows];      // of the rows in the key and value pages, in elements; -1: the row has none
  const uint32_t at = a.first + blockIdx.x, block = at / a.cut.groups;
  const int row0 = static_cast<int>(block) * a.cut.rows, rows = min(a.cut.rows, a.rows - row0);
  const int b0 = static_cast<int>(static_cast<uint32_t>(row0) / static_cast<uint32_t>(a.per)), l0 = row0 - b0 * a.per;
  const int h0 = static_cast<int>(at - block * a.cut.groups) * a.cut.heads, heads = min(a.cut.heads, a.Hq + 2 * a.Hkv - h0);
  // (a ragged batch: all rows behind the tokens of their sequence; only their queries are read)
  const bool dead = a.counts != nullptr && l0 + rows <= a.per && l0 >= a.counts[b0];
  const bool flat = a.near && l0 + rows <= a.per;      // (rows of one sequence)
  const T* const q = static_cast<const T*>(a.q) + b0 * a.qs[0] + l0 * a.qs[1];
  const T* const k = static_cast<const T*>(a.k) + b0 * a.ks[0] + l0 * a.ks[1];
  const T* const v = static_cast<const T*>(a.v) + b0 * a.vs[0] + l0 * a.vs[1];
  T* const out = static_cast<T*>(a.qo) + (static_cast<int64_t>(row0) * a.Hq + h0) * a.D;
  T *const kp = static_cast<T*>(a.kp), *const vp = static_cast<T*>(a.vp);
  const int64_t qs0 = a.qs[0], qs1 = a.qs[1], qs2 = a.qs[2], ks0 = a.ks[0], ks1 = a.ks[1], ks2 = a.ks[2], vs0 = a.vs[0],
                vs1 = a.vs[1], vs2 = a.vs[2], kps2 = a.kps[2], vps2 = a.vps[2];
  turn_heads<T, WV, PV, ADJ>(
      a.t, a.cut, a.L > 0 ? rows * a.cut.heads : 0, reinterpret_cast<T*>(held + (threadIdx.x >> 6) * kWave), cs,
      [&](int n) {
        const int r = a.cut.by_heads.of(n), h = h0 + min(n - r * a.cut.heads, heads - 1);
        if (dead && h >= a.Hq) return static_cast<const T*>(nullptr);
        const bool of_q = h < a.Hq, of_k = h < a.Hq + a.Hkv;
        const T* const p = pick(of_q, q, pick(of_k, k, v));
        const int hh = h - pick(of_q, 0, pick(of_k, a.Hq, a.Hq + a.Hkv));
        const int64_t s0 = pick(of_q, qs0, pick(of_k, ks0, vs0)), s1 = pick(of_q, qs1, pick(of_k, ks1, vs1)),
                      s2 = pick(of_q, qs2, pick(of_k, ks2, vs2));
        if (flat) return p + apart(r, static_cast<int>(s1), hh, static_cast<int>(s2));
        const Row w = row_of(b0, l0, r, a.per);
        return p + (w.b - b0) * s0 + (w.l - l0) * s1 + hh * s2;
      },
      [&](int n) -> T* {
        const int r = a.cut.by_heads.of(n), i = n - r * a.cut.heads, h = h0 + i;
        if (i >= heads) return nullptr;
        // (a workgroup has a few thousand heads at most, one row where a row has several groups)
        if (h < a.Hq) return out + __umul24(__umul24(r, a.Hq) + i, a.D);
        const bool of_k = h < a.Hq + a.Hkv;
        const int64_t place = places[of_k ? 0 : 1][r];
        if (place < 0) return nullptr;
        T* const to = pick(of_k, kp, vp);
        const int hh = h - pick(of_k, a.Hq, a.Hq + a.Hkv);
        const int64_t s2 = pick(of_k, kps2, vps2);
        return to + place + (a.near ? apart(0, 0, hh, static_cast<int>(s2)) : hh * s2);
      },
      [&](int n) {
        const int r = a.cut.by_heads.of(n);
        return h0 + n - r * a.cut.heads < a.Hq + a.Hkv ? r : -1;
      },
      [&] {
        for (int r = threadIdx.x; r < rows; r += 256) {
          const Row w = row_of(b0, l0, r, a.per);
          const int b = w.b, i = w.l, start = a.starts[b];
          int count = a.L, page = -1, place = 0;
          if (a.counts != nullptr) count = min(max(a.counts[b], 0), a.L);
          if (i == 0 && h0 == 0 && a.lengths != nullptr) a.lengths[b] = start + count;
          const int64_t s = static_cast<int64_t>(start) + i;
          if (i < count && s >= 0 && s < static_cast<int64_t>(a.max_pages) * a.page_size) {
            const int n = static_cast<int>(s) / a.page_size;
            place = static_cast<int>(s) - n * a.page_size;
            page = a.table[b * a.ts + n];
          }
          const bool ok = page >= 0 && page < a.num_pages;
          places[0][r] = ok ? page * a.kps[0] + place * a.kps[1] : -1;
          places[1][r] = ok ? page * a.vps[0] + place * a.vps[1] : -1;
        }
        if (a.L > 0)
          form_turns(a.t, a.cut.log_pairs, rows, 1.f, cs, [&](int r, int axis) {
            const Row w = row_of(b0, l0, r, a.per);
            return a.t.positions != nullptr ? position_of(a.t, w.b, w.l, axis)
                                            : static_cast<double>(static_cast<int64_t>(a.starts[w.b]) + w.l);
          });
        __syncthreads();
      });
}

template <typename T, int WV, int PV>
const void* kernel_of(bool adjacent) {
  return adjacent && PV > 1 ? reinterpret_cast<const void*>(&append_kernel<T, WV, PV, (PV > 1)>)
                            : reinterpret_cast<const void*>(&append_kernel<T, WV, PV, false>);
}
const void* kernel_of(bool bf16, int wv, int pv, bool adjacent) {
  if (bf16) {
    if (wv == 8) return pv == 8 ? kernel_of<uint16_t, 8, 8>(adjacent) : pv == 2 ? kernel_of<uint16_t, 8, 2>(adjacent)
                                                                                : kernel_of<uint16_t, 8, 1>(adjacent);
    if (wv == 2) return pv == 2 ? kernel_of<uint16_t, 2, 2>(adjacent) : kernel_of<uint16_t, 2, 1>(adjacent);
    return kernel_of<uint16_t, 1, 1>(adjacent);
  }
  if (wv == 4) return pv == 4 ? kernel_of<float, 4, 4>(adjacent) : kernel_of<float, 4, 1>(adjacent);
  return kernel_of<float, 1, 1>(adjacent);
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
  if (d->head_dim > kMostD || heads > big || d->batch > big || length > big || d->batch * length * heads > big ||
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
  a.rows = static_cast<int>(d->batch * a.per);
  a.Hq = static_cast<int>(d->query_heads);
  a.Hkv = static_cast<int>(d->key_heads);
  a.D = static_cast<int>(d->head_dim);
  a.num_pages = cache ? static_cast<int>(d->num_pages) : 0;
  a.page_size = static_cast<int>(d->page_size);
  a.max_pages = cache ? static_cast<int>(d->max_pages) : 0;
  a.t = turns_of(d->axes, d->sections, d->layout, d->position_type, d->position_stride, positions, frequencies);
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const int w = vector_of(d->head_dim, es);
  const int pv = pairs_at_once(a.t, d->sections, w, es);
  a.cut = cut_of(w, pv, es, a.t.pairs, d->head_dim, a.rows, a.Hq + 2 * a.Hkv);
  a.cut.rows = std::min(a.cut.rows, kRows);
  a.near = near_by(a.cut.rows, a.qs[1], a.Hq, a.qs[2]) && near_by(a.cut.rows, a.ks[1], a.Hkv, a.ks[2]) &&
           near_by(a.cut.rows, a.vs[1], a.Hkv, a.vs[2]) && near_by(1, 0, a.Hkv, a.kps[2]) && near_by(1, 0, a.Hkv, a.vps[2]);
  void* args[] = {&a};
  return launch(kernel_of(bf16, w, pv, d->layout == DCN_ROTARY_ADJACENT),
                (static_cast<int64_t>(a.rows) + a.cut.rows - 1) / a.cut.rows * a.cut.groups, args,
                turns_bytes(a.cut, a.t), &a.first, stream)
             ? DCN_OK
             : DCN_E_HIP;
}

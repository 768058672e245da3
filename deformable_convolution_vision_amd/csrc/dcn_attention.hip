// dcn_attention.hip -- gfx950 cross attention to an encoder's states.
//
// For a query row q (one position of one head) and the keys j that its batch element's mask
// keeps, with s_j = scale * q . k_j:
//
//   out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),   lse = m + log sum_j exp(s_j - m)
//
// for any m; the kernel carries m as the running maximum over the key tiles seen so far, and
// rescales what it has summed when a tile raises it, so keys and values are read once and no
// score leaves the registers.  Scores are formed transposed, S^T = K Q^T (a lane holds one
// row q and 16 keys of it), because then the lane's own exponentials are the operand of the
// second product, out^T += V^T P^T, without an exchange between lanes, and the maximum, the
// sum and the rescaling factor are one value per lane.
//
// The heads that share a key head are rows of one problem (row r: position r / g, head r % g),
// so a single token of many heads reads each key once.
//
// Two forms.  attn_rows_kernel: 128 rows in four waves, which share a ring of key tiles that
// buffer -> LDS loads fill ahead of use.  attn_few_rows_kernel: 32 rows, whose keys the waves of
// a workgroup take in turn, each at its own pace, and join at the end.  Where there are fewer
// row tiles than the chip holds (and for the last, incomplete round of them) the keys of a tile
// are also split over workgroups: each writes its maximum, sum and undivided output, and
// attn_join_kernel adds them up in split order.
//
// Arithmetic: products of bf16 (exact) or fp32 added in fp32; the softmax in fp32; for bf16
// the weights exp(s - m) are rounded to bf16 as the second product's operand (their sum is
// not), and the output is rounded once.  (That rounding is what the matrix units' bf16 rate costs:
// the output is 1.4 times one rounding away from the exact one.  The sum by a product with ones,
// 16 additions fewer a lane, would be the rounded weights' and put lse off by 1e-4: not done.)
//
// What bounds it, measured (copies reach 5.0 TB/s on this card, products 1253 TFLOP/s of bf16):
//  - Single tokens: the keys' and values' bytes.  8 batch elements of 16 heads of 128 on 4 key heads,
//    16800 keys, 203 MB attended: 58 us in all, of which the join of the parts is 4.5 and about 5 the
//    start of each workgroup's first loads, which nothing hides; 1.1 GB take 215 us, the rate of a
//    copy.  One row of 8 heads of 64 over 1050 keys: 10.3 us, a launch and one workgroup's chain of
//    five steps.
//  - 300 queries of 8 heads of 32 over 4200 keys, batch 2: 19.6 us, one round of 160 workgroups; each
//    wave's chain of load, product, softmax, product over its 9 blocks, and the join of 16 waves.
//  - 4200 queries over 16800 keys, 8 heads of 64, batch 2: 362 to 378 us, 765 to 798
//    TFLOP/s.  A tile of 64 keys and 32 rows is 512 cycles of products and 842 of vector instructions (at the rates a loop of each
//    alone reaches, four waves on a SIMD); about 1580 are measured: the two overlap little.  Eight waves on
//    two halves of the keys (390 against 371 us then) and the products of one tile among the
//    exponentials of another (398 against 396) did not change that.
//  - fp32: the matrix units, 16 times as many cycles as for bf16, at padded heads (32, 64 or 128): 4200
//    queries over 4200 keys, 8 heads of 40 or 64, 533 us (148 and 237 by the formulas' products at the
//    library's rate); of 72 to 128, 1310 us (266 to 473): there a CU holds one workgroup of the rows
//    form and the plan counts two, so 264 tiles take a second round of the chip.  One token of 8 heads
//    of 64 over 1050 keys: 27 us, the chain of five steps at that rate.
//  - Rows that are not read 16 bytes at a time: loads of single elements that are done before a tile's
//    products begin.  2 x 4200 queries over 4200 keys, 8 bf16 heads of 36: 308 us, of 40: 105.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "dcn.h"
#include "dcn_attention.h"

namespace dcn {
namespace attn {
namespace {

// A lane's row in registers.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_row(const Args& a, const Work& w, int row, Frag<T> (&f)[DP / 16]) {
  const bool live = row < a.R;
  const int pos = live ? row / a.g : 0, head = w.hk * a.g + (live ? row % a.g : 0);
  load_frags<T, DP, VEC>(static_cast<const T*>(a.q) + w.b * a.qs[0] + pos * a.qs[1] + head * a.qs[2], 0, a.D, live, f);
}

// A lane's running softmax: the maximum (in powers of two) of its row, and the sum of its own
// half of the weights.
struct Running {
  float m = kNegInf, l = 0.f;
};

// Takes the maximum of a lane's new scores into account.  Any m serves the formulas: it is only
// to keep the weights within range.  So it is raised, and what is summed is rescaled, only when
// scores exceed it by more than 2^8 (and at the first ones), which is seldom after a few tiles;
// the weights then reach up to 2^8.
template <int DT>
__device__ __forceinline__ void raise_max(float mt, Running& run, f32x16 (&o)[DT]) {
  if (__any(mt > run.m + 8.f)) {
    const float mn = fmaxf(run.m, mt), alpha = run.m == kNegInf ? 0.f : exp2_fast(run.m - mn);
    run.m = mn;
    run.l *= alpha;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] *= alpha;
  }
}

// Takes N blocks of 32 scores in (raw products; word: the attended keys of each), gives the
// weights as the second product's operands.  Maximum and sum run in four strands each: one would
// wait for itself.
template <typename T, int N, int DT>
__device__ __forceinline__ void softmax_step(f32x16 (&s)[N], const uint32_t (&word)[N], float c, Running& run,
                                             f32x16 (&o)[DT], typename POperand<T>::type (&pf)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (word[n] != 0xffffffffu) mask_scores(s[n], word[n]);
  float mt[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) mt[j] = fmaxf(s[0][4 * j], s[0][4 * j + 1]);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n > 0) mt[j] = max3(mt[j], s[n][4 * j], s[n][4 * j + 1]);
      mt[j] = max3(mt[j], s[n][4 * j + 2], s[n][4 * j + 3]);
    }
  raise_max(max_halves(fmaxf(max3(mt[0], mt[1], mt[2]), mt[3])) * c, run, o);
  const float ms = run.m == kNegInf ? 0.f : run.m;   // no key counted yet: exp2(-inf) = 0
  float sum[4] = {run.l, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float p[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      p[r] = exp2_fast(fmaf(s[n][r], c, -ms));
      sum[r & 3] += p[r];
    }
    to_operand(p, pf[n]);
  }
  run.l = (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Writes 4 elements of a finished row, or its part.
template <typename T, int DP>
__device__ __forceinline__ void put4(const Args& a, const Work& w, int rows, int rr, int d, float m, float l, float4 v) {
  const int row = w.row0 + rr;
  if (row >= a.R) return;
  if (w.tail >= 0) {
    const int64_t prow = (static_cast<int64_t>(w.tail) * a.y.splits + w.split) * rows + rr;
    *reinterpret_cast<float4*>(a.part + prow * DP + d) = v;
    if (d == 0) *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(m, l);
    return;
  }
  const int pos = row / a.g, head = w.hk * a.g + row % a.g;
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // no key: zeros; a NaN sum stays NaN
  T* op = static_cast<T*>(a.out) + ((static_cast<int64_t>(w.b) * a.Lq + pos) * a.Hq + head) * a.D;
  const float vals[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (d + j < a.D) op[d + j] = narrow<T>(vals[j]);
  if (d == 0 && a.lse != nullptr)
    a.lse[(static_cast<int64_t>(w.b) * a.Hq + head) * a.Lq + pos] =
        l == 0.f ? kNegInf : fmaf(m == kNegInf ? 0.f : m, kLn2, logf(l));
}

// Joins the W waves that took different keys of the same 32 rows, 32 elements of the head at a
// time, through LDS (which also turns the transposed registers into rows).  Called by all waves
// of the workgroup, G groups of W; `rr0`: the group's first row in the tile.
template <typename T, int DP, int W, int G, int DT>
__device__ __forceinline__ void join_waves(const Args& a, const Work& w, int rows, float m, float l,
                                           const f32x16 (&o)[DT], unsigned char* smem) {
  constexpr int OST = 36, NT = 64 * W * G;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  float* os = reinterpret_cast<float*>(smem);             // [G][W][32][OST]
  float* fs = os + G * W * 32 * OST;                      // [G][W][32] maxima, then each wave's factor
  float* ls = fs + G * W * 32;                            // [G][W][32] sums
  __syncthreads();
  if (half == 0) {
    fs[wave * 32 + lane] = m;
    ls[wave * 32 + lane] = l;
  }
  float mm = kNegInf, ll = 0.f;                            // of the row that this thread writes
  constexpr int RT = G * 32 * 8;                          // threads that write: 4 elements each
  float f[W];
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<float4*>(os + (wave * 32 + (lane & 31)) * OST + acc_row(4 * r4, half)) =
          make_float4(o[i][4 * r4], o[i][4 * r4 + 1], o[i][4 * r4 + 2], o[i][4 * r4 + 3]);
    __syncthreads();
#pragma unroll
    for (int at = tid; at < RT; at += NT) {
      const int rr = at / 8, d = (at % 8) * 4, g = rr / 32, ri = rr % 32;
      if (i == 0 || RT > NT) {
        mm = kNegInf;
        ll = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) mm = fmaxf(mm, fs[(g * W + j) * 32 + ri]);
        const float ms = mm == kNegInf ? 0.f : mm;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          f[j] = exp2_fast(fs[(g * W + j) * 32 + ri] - ms);
          ll = fmaf(f[j], ls[(g * W + j) * 32 + ri], ll);
        }
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(os + ((g * W + j) * 32 + ri) * OST + d);
        acc.x = fmaf(f[j], v.x, acc.x);
        acc.y = fmaf(f[j], v.y, acc.y);
        acc.z = fmaf(f[j], v.z, acc.z);
        acc.w = fmaf(f[j], v.w, acc.w);
      }
      put4<T, DP>(a, w, rows, rr, 32 * i + d, mm, ll, acc);
    }
  }
}
constexpr size_t join_lds(int waves) { return static_cast<size_t>(waves) * 32 * (36 + 2) * 4; }

// 32 rows; the W waves of a workgroup take every W-th block of 32 keys and join at the end, so
// no wave waits for another inside the loop (the single-token case above: 137 us with tiles shared by
// the waves and a mask byte waited for at each row, 65 with these and the mask in bits, 54 since no
// LDS read waits for loads under way).  Two blocks on their
// way instead of one need registers that a wave has not: 11.4 against 10.5 us for one token over
// 1050 keys, 25.5 against 24.9 for 333 queries in fp32.  A lane's key row comes straight from memory as
// the first product's operand; values go through two places in the LDS that are the wave's own.
// The next block's rows are on their way while one is worked on.
template <typename T, int DP, int W, bool VEC>
__global__ __launch_bounds__(64 * W) void attn_few_rows_kernel(Args a) {
  constexpr int AHEAD = 1;   // blocks on their way while one is worked on
  constexpr int DT = DP / 32, KL = DP * static_cast<int>(sizeof(T)) / 32, VL = tile_loads<T, DP, 32, 64>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  T* const lds = reinterpret_cast<T*>(smem) + wave * (AHEAD + 1) * 32 * DP;
  const Work w = work_of(a, a.y, a.first + blockIdx.x, 32, (a.Lk + 32 * W - 1) / (32 * W));
  const T* kp = static_cast<const T*>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2];
  const T* vp = static_cast<const T*>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2];
  const uint8_t* mp = a.mask == nullptr ? nullptr : a.mask + w.b * a.ms;
  Frag<T> qf[DP / 16];
  load_row<T, DP, VEC>(a, w, w.row0 + (lane & 31), qf);
  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc();
  Running run;

  Frag<T> kf[AHEAD + 1][DP / 16];
  // Rows of padded keys are taken as zeros and not read: a padded key's weight is exactly 0,
  // but 0 times an infinity or NaN in its value row would not be.
  const auto load_keys = [&](int64_t k0, uint32_t word, Frag<T> (&f)[DP / 16]) {
    const bool in = (word >> (lane & 31)) & 1u;
    if constexpr (VEC) {
      const __amdgpu_buffer_rsrc_t rs = rsrc_of(kp + k0 * a.ks[1]);
      const uint32_t ofs = (static_cast<uint32_t>(lane & 31) * static_cast<uint32_t>(a.ks[1]) + 8 * half) *
                           static_cast<uint32_t>(sizeof(T));
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h) {
          const bool at = in && 16 * i + 8 * half + h * Elem<T>::kVec < a.D;
          const auto u = __builtin_amdgcn_raw_buffer_load_b128(
              rs, at ? ofs + 16 * i * static_cast<uint32_t>(sizeof(T)) + 16 * h : kOutside, 0, 0);
          __builtin_memcpy(reinterpret_cast<char*>(&f[i]) + 16 * h, &u, 16);
        }
    } else {
      load_frags<T, DP, false>(kp + k0 * a.ks[1], (lane & 31) * a.ks[1], a.D, in, f);
    }
  };
  const auto load_values = [&](int64_t k0, uint32_t word, T* __restrict__ to) {
    fetch_tile<T, DP, 32, 64, VEC>(to, vp + k0 * a.vs[1], [&](int r) { return r * a.vs[1]; }, word, a.D,
                                   lane);
  };

  // the waves of all workgroups that share the tile take the blocks in turn: what a mask leaves
  // out is then missing from each alike
  const int64_t step = static_cast<int64_t>(32 * W) * (w.tail >= 0 ? a.y.splits : 1), first = 32 * (w.split * W + wave);
  for (int64_t win = first; win < a.Lk; win += 64 * step) {
    const uint32_t words = key_words(mp, win, step, a.Lk, a.Lk);
    uint64_t live = __ballot(words != 0);   // the blocks of the window not sent for yet
    // Sends for the next block that holds an attended key; its mask bits, or 0 when there is none
    // (the loads then all lie outside and fetch nothing: as many are under way either way, so
    // that a wait for the block before can leave them alone).
    const auto send = [&](Frag<T> (&f)[DP / 16], T* __restrict__ to) {
      const int at = live != 0 ? __builtin_ctzll(live) : 0;
      const uint32_t word = live != 0 ? __builtin_amdgcn_readlane(words, at) : 0u;
      live &= live - 1;
      load_keys(win + at * step, word, f);
      load_values(win + at * step, word, to);
      return word;
    };
    constexpr int N = AHEAD + 1;
    uint32_t word[N];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) word[j] = send(kf[j], lds + j * 32 * DP);
    if (win == first) arrived(qf);
    // One block: its values in `cur` while a later block's are sent to `to` (two places, and the
    // compiler is told so: see attn_rows_kernel).
    const auto turn = [&](Frag<T> (&k)[DP / 16], uint32_t mine, Frag<T> (&kn)[DP / 16], uint32_t& sent,
                          const T* __restrict__ cur, T* __restrict__ to) {
      sent = send(kn, to);
      f32x16 s[1] = {zero_acc()};   // (registers for standing zeros are not to spare here)
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) s[0] = mma(k[i], qf[i], s[0]);
      const uint32_t m1[1] = {mine};
      typename POperand<T>::type pf[1];
      softmax_step<T>(s, m1, a.c, run, o, pf);
      if constexpr (VEC) wait_loads<AHEAD * (KL + VL)>(cur, to);   // this block's values are there
#pragma unroll
      for (int i = 0; i < DT; ++i) o[i] = mma_rows<DP>(cur, 0, 32 * i, pf[0], o[i]);
    };
    bool more = true;
    while (more) {
      // one turn for each place, so that registers under way are named and never moved
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (word[j] == 0) {
          more = false;
          break;
        }
        turn(kf[j], word[j], kf[(j + AHEAD) % N], word[(j + AHEAD) % N], lds + j * 32 * DP, lds + (j + AHEAD) % N * 32 * DP);
      }
    }
    wait_loads<0>();   // what was sent for last must not land on what the LDS is used for next
  }
  join_waves<T, DP, W, 1>(a, w, 32, run.m, sum_halves(run.l), o, smem);
}

// Waves of a SIMD that the rows form leaves registers for (accumulators then stay in the ordinary
// registers: with more of them than needed the compiler moves them to the others and back).
// Rows of 64 bytes leave room for three: 4200 queries over 4200 keys, 8 heads of 32, batch 2, 82 us
// against 87 with two.  The plan still counts two to a CU: with tiles split to fill three it took 103.
constexpr int waves_per_simd(int row_bytes) { return row_bytes <= 64 ? 3 : row_bytes <= 256 ? 2 : 1; }

// Rows of 128 in four waves, which share a ring of STAGES key tiles of 64 in the LDS: while one
// is worked on, the next STAGES - 1 are on their way.  (4200 queries over 16800 keys, batch 2, 8 heads
// of 64: 453 us with loads through registers into one tile, 387 with the ring, 383 with the maximum
// raised lazily.)  A wave goes first on its SIMD from its second products to its next loads, so that
// its matrix instructions are not held up among the other wave's vector instructions: 381 -> 365 us
// there, 46 -> 41 for 900 queries over 16800 keys, 8 heads of 32.  (The few-rows form gains nothing.)
template <typename T, int DP, int STAGES, bool VEC>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(waves_per_simd(sizeof(T) * DP), waves_per_simd(sizeof(T) * DP)))) void attn_rows_kernel(Args a) {
  constexpr int KT = 64, DT = DP / 32, BUF = 2 * KT * DP, LOADS = 2 * tile_loads<T, DP, KT, 256>, AHEAD = STAGES - 1;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  T* const lds = reinterpret_cast<T*>(smem);              // [STAGES][keys, values][KT][DP]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Work w = work_of(a, a.y, a.first + blockIdx.x, 128, (a.Lk + KT - 1) / KT);
  const T* kp = static_cast<const T*>(a.k) + w.b * a.ks[0] + w.hk * a.ks[2];
  const T* vp = static_cast<const T*>(a.v) + w.b * a.vs[0] + w.hk * a.vs[2];
  const uint8_t* mp = a.mask == nullptr ? nullptr : a.mask + w.b * a.ms;
  Frag<T> qf[DP / 16];
  load_row<T, DP, VEC>(a, w, w.row0 + wave * 32 + (lane & 31), qf);
  f32x16 o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) o[i] = zero_acc();
  Running run;
  const f32x16 zeros = zero_acc();

  KeyTiles tiles(mp, a.Lk, w.s0, w.s1);
  // sends for the next tile that holds an attended key; its mask bits, or 0 when there is none
  const auto send = [&](T* __restrict__ to) {
    int64_t k0;
    const uint64_t word = tiles.next(k0);
    if (word != 0) {
      fetch_tile<T, DP, KT, 256, VEC>(to, kp + k0 * a.ks[1], [&](int r) { return r * a.ks[1]; }, word, a.D, tid);
      fetch_tile<T, DP, KT, 256, VEC>(to + KT * DP, vp + k0 * a.vs[1], [&](int r) { return r * a.vs[1]; }, word,
                                      a.D, tid);
    }
    return word;
  };
  uint64_t word[AHEAD + 1];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) word[j] = send(lds + j * BUF);
  arrived(qf);
  // One tile: `cur` is worked on while a later one is sent to `to`.  The two are different
  // places, and the compiler is told so (restrict): it would otherwise wait for everything that
  // is on its way to the LDS before it reads from it.
  const auto turn = [&](const T* __restrict__ cur, T* __restrict__ to) {
    word[AHEAD] = send(to);
    __builtin_amdgcn_s_setprio(0);
    const T* ks = cur;
    const T* vs = cur + KT * DP;
    f32x16 s[2];
    Frag<T> kf[2][DP / 16];
#pragma unroll
    for (int i = 0; i < DP / 16; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n) kf[n][i] = row_frag<DP>(ks, 32 * n, i);
#pragma unroll
    for (int i = 0; i < DP / 16; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n] = mma(kf[n][i], qf[i], i == 0 ? zeros : s[n]);
    const uint32_t both[2] = {static_cast<uint32_t>(word[0]), static_cast<uint32_t>(word[0] >> 32)};
    typename POperand<T>::type pf[2];
    softmax_step<T>(s, both, a.c, run, o, pf);
    __builtin_amdgcn_s_setprio(1);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        Frag<T> vf[DT][2];
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) vf[i][h] = col_frag<DP>(vs, 32 * n, 32 * i, h);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < DT; ++i) o[i] = mma(vf[i][h], pf[n].f[h], o[i]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] = mma_rows<DP>(vs, 32 * n, 32 * i, pf[n], o[i]);
    }
  };
  int slot = 0;
  while (word[0] != 0) {
    // this wave's share of the tile is there when only the later tiles' loads are under way
    if (AHEAD == 2 && word[1] != 0) wait_loads<LOADS>();
    else wait_loads<0>();
    lds_barrier();              // the other waves' shares too; and the tile before is no longer read
    turn(lds + slot * BUF, lds + (slot == 0 ? STAGES - 1 : slot - 1) * BUF);
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) word[j] = word[j + 1];
    slot = slot == STAGES - 1 ? 0 : slot + 1;
  }
  join_waves<T, DP, 1, 4>(a, w, 128, run.m, sum_halves(run.l), o, smem);
}

// Adds up the parts of split tiles: one thread for 4 elements of a row.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(Args a, int rows) {
  constexpr int V4 = DP / 4;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, prow = at / V4;
  Work w;
  const int tail = static_cast<int>(prow / rows), rr = static_cast<int>(prow % rows), tile = a.y.full + tail;
  if (tile >= a.y.tiles) return;
  const int nbh = a.B * a.Hkv, bh = tile % nbh, d = static_cast<int>(at % V4) * 4;
  w.b = bh / a.Hkv;
  w.hk = bh % a.Hkv;
  w.row0 = tile / nbh * rows;
  w.tail = -1;
  if (w.row0 + rr >= a.R) return;
  const int64_t p0 = static_cast<int64_t>(tail) * a.y.splits * rows + rr;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + p0;
  const float* part = a.part + p0 * DP + d;
  float mm = kNegInf, ll = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.y.splits; ++s) mm = fmaxf(mm, ml[static_cast<int64_t>(s) * rows].x);
  const float ms = mm == kNegInf ? 0.f : mm;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < a.y.splits; ++s) {
    const float2 x = ml[static_cast<int64_t>(s) * rows];
    const float f = exp2_fast(x.x - ms);
    const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(s) * rows * DP);
    ll = fmaf(f, x.y, ll);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  put4<T, DP>(a, w, rows, rr, d, mm, ll, acc);
}

// Waves of the few-rows form: as many as the registers of a CU hold at this head size (one workgroup
// a CU: with the splits sized for two or three, the parts of a second round only add to the join).
constexpr int waves_of(int es, int dp) { return es == 2 ? (dp == 32 ? 16 : 8) : (dp == 128 ? 4 : dp == 64 ? 8 : 16); }

struct Plan {
  int dp;
  bool wide;     // attn_rows_kernel (else attn_few_rows_kernel)
  int waves;     // of a workgroup
  int rows;      // of a tile
  Tiling y;
};

// The rows form where its tiles of 128 rows are filled and the few-rows form, of which a CU holds
// one workgroup, would need nearly more than one round of the chip.  Measured (bf16, few / rows):
// 160 tiles of 32 rows (2 x 300 rows of 8 heads of 32, 4200 keys) 20.1 / 23.3 us, 198 (fp32, 3 x
// 333 of 6 of 40, 1051 keys) 25.2 / 31.2, 232 (900 of 8 of 32, 16800 keys) 54.3 / 46.1, 320 (4 x
// 300 of 8 of 32, 4200 keys) 37.1 / 25.5.
// Splits: the few-rows form down to four steps (with fewer, the launch that joins them costs more
// than they save: one row, 8 heads of 64, 1050 keys 14.4 us in two parts, 10.6 unsplit).
Plan make_plan(const dcn_attn_desc* d) {
  Plan p{};
  const int es = d->dtype == DCN_BF16 ? 2 : 4;
  p.dp = padded_head(d->head_dim);
  const int64_t nbh = d->batch * d->key_heads, R = d->query_len * (d->query_heads / d->key_heads);
  p.wide = R > 96 && nbh * ((R + 31) / 32) * 8 > 7 * kCUs;
  p.waves = p.wide ? 4 : waves_of(es, p.dp);
  p.rows = p.wide ? 128 : 32;
  const int64_t step = p.wide ? 64 : 32 * p.waves;
  p.y = tile_over(nbh * ((R + p.rows - 1) / p.rows), (d->key_len + step - 1) / step, p.wide ? 2 * kCUs : kCUs,
                  p.wide ? 2 : 4);
  return p;
}

size_t lds_bytes(const Plan& p, int es) {
  const size_t row = static_cast<size_t>(p.dp) * es;
  return std::max((p.wide ? stages_of(row) * 2 * 64 : p.waves * 2 * 32) * row, join_lds(p.waves));
}

size_t part_bytes(const Plan& p, size_t* ml_at) {
  const size_t rows = static_cast<size_t>(p.y.tiles - p.y.full) * p.y.splits * p.rows;
  *ml_at = rows * p.dp * 4;
  return (*ml_at + rows * 8 + 255) / 256 * 256;
}

template <typename T, int DP>
const void* fwd_kernel(bool wide, bool vec) {
  if (wide)
    return vec ? reinterpret_cast<const void*>(&attn_rows_kernel<T, DP, stages_of(sizeof(T) * DP), true>)
               : reinterpret_cast<const void*>(&attn_rows_kernel<T, DP, stages_of(sizeof(T) * DP), false>);
  return vec ? reinterpret_cast<const void*>(&attn_few_rows_kernel<T, DP, waves_of(sizeof(T), DP), true>)
             : reinterpret_cast<const void*>(&attn_few_rows_kernel<T, DP, waves_of(sizeof(T), DP), false>);
}
template <typename T>
const void* fwd_kernel(int dp, bool wide, bool vec) {
  return dp == 32 ? fwd_kernel<T, 32>(wide, vec) : dp == 64 ? fwd_kernel<T, 64>(wide, vec) : fwd_kernel<T, 128>(wide, vec);
}
template <typename T>
const void* join_kernel(int dp) {
  return dp == 32   ? reinterpret_cast<const void*>(&attn_join_kernel<T, 32>)
         : dp == 64 ? reinterpret_cast<const void*>(&attn_join_kernel<T, 64>)
                    : reinterpret_cast<const void*>(&attn_join_kernel<T, 128>);
}

}  // namespace

int check(const dcn_attn_desc* d) {
  if (d == nullptr) return DCN_E_ARG;
  const int64_t big = 2147483647;
  if (d->batch < 0 || d->query_len < 0 || d->key_len < 0 || d->query_heads < 1 || d->key_heads < 1 ||
      d->head_dim < 1 || d->query_heads % d->key_heads != 0 || !std::isfinite(d->scale) || !(d->scale > 0.f) ||
      d->mask_stride < 0)
    return DCN_E_ARG;
  for (int i = 0; i < 3; ++i)
    if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0) return DCN_E_ARG;
  if (d->dtype != DCN_F32 && d->dtype != DCN_BF16) return DCN_E_UNSUPPORTED;
  if (d->head_dim > 128) return DCN_E_UNSUPPORTED;
  // int32 row and workgroup counts; addresses are 64-bit
  if (d->batch > big || d->query_len > big || d->key_len > big - 256 || d->query_heads > big || d->key_heads > big)
    return DCN_E_UNSUPPORTED;
  const double rows = static_cast<double>(d->query_len) * (d->query_heads / d->key_heads);
  const double groups = static_cast<double>(d->batch) * d->key_heads;
  if (rows > big - 256 || groups * (rows + 128) > big || groups * (static_cast<double>(d->key_len) + 128) > big)
    return DCN_E_UNSUPPORTED;
  return DCN_OK;
}

void fill_args(const dcn_attn_desc* d, Args* a) {
  for (int i = 0; i < 3; ++i) {
    a->qs[i] = d->q_stride[i];
    a->ks[i] = d->k_stride[i];
    a->vs[i] = d->v_stride[i];
  }
  a->ms = d->mask_stride;
  a->B = static_cast<int>(d->batch);
  a->Lq = static_cast<int>(d->query_len);
  a->Lk = static_cast<int>(d->key_len);
  a->Hq = static_cast<int>(d->query_heads);
  a->Hkv = static_cast<int>(d->key_heads);
  a->g = a->Hq / a->Hkv;
  a->D = static_cast<int>(d->head_dim);
  a->R = a->Lq * a->g;
  a->scale = d->scale;
  a->c = d->scale * kLog2e;
}

}  // namespace attn
}  // namespace dcn

extern "C" int dcn_cross_attention_workspace_bytes(const dcn_attn_desc* d, size_t* bytes) {
  if (bytes == nullptr) return DCN_E_ARG;
  const int rc = dcn::attn::check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->query_len == 0) {
    *bytes = 0;
    return DCN_OK;
  }
  size_t at;
  *bytes = dcn::attn::part_bytes(dcn::attn::make_plan(d), &at);
  return DCN_OK;
}

extern "C" int dcn_cross_attention(const dcn_attn_desc* d, const void* q, const void* k, const void* v,
                                   const uint8_t* key_mask, void* out, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  using namespace dcn::attn;
  const int rc = check(d);
  if (rc != DCN_OK) return rc;
  if (d->batch == 0 || d->query_len == 0) return DCN_OK;
  if (q == nullptr || out == nullptr || (d->key_len > 0 && (k == nullptr || v == nullptr))) return DCN_E_ARG;
  const Plan p = make_plan(d);
  size_t ml_at;
  const size_t need = part_bytes(p, &ml_at);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return DCN_E_WORKSPACE;
  Args a{};
  fill_args(d, &a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.mask = key_mask;
  a.out = out;
  a.lse = lse;
  a.y = p.y;
  if (need > 0) {
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + ml_at);
  }
  const bool bf16 = d->dtype == DCN_BF16;
  const int es = bf16 ? 2 : 4;
  const bool vec = vec_ok(q, d->q_stride, d->head_dim, es) && vec_ok(k, d->k_stride, d->head_dim, es) &&
                   vec_ok(v, d->v_stride, d->head_dim, es);
  const int tail = p.y.tiles - p.y.full;
  void* args[] = {&a};
  const void* fn = bf16 ? fwd_kernel<uint16_t>(p.dp, p.wide, vec) : fwd_kernel<float>(p.dp, p.wide, vec);
  if (!launch_groups(fn, workgroups(p.y), 64 * p.waves, args, &a, lds_bytes(p, es), stream)) return DCN_E_HIP;
  if (tail > 0) {
    const int64_t n = static_cast<int64_t>(tail) * p.rows * (p.dp / 4);
    int rows = p.rows;
    void* join_args[] = {&a, &rows};
    fn = bf16 ? join_kernel<uint16_t>(p.dp) : join_kernel<float>(p.dp);
    if (hipLaunchKernel(fn, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), join_args, 0, stream) != hipSuccess)
      return DCN_E_HIP;
  }
  return DCN_OK;
}

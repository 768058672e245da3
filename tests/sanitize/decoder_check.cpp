// decoder_check.cpp -- drives the host side of rotary positions, block joins and the paged cache with no GPU
// (hipLaunchKernel is this file's): descriptor checks, plans, workspace sizes, and every launch that they make
// for sizes that the checks admit, as it reaches the runtime.
// Test infrastructure: built with AddressSanitizer and UndefinedBehaviorSanitizer and run by
// tests/test_sanitizers_decoder.py on the CPU.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "dcn.h"

namespace {

int fails = 0, launches = 0;
int64_t groups = 0;   // workgroups of the calls since reset()
const char* now = "";

void reset(const char* what) {
  now = what;
  launches = 0;
  groups = 0;
}
void expect(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAIL %s: %s (%d launches, %lld workgroups)\n", now, what, launches, static_cast<long long>(groups));
    ++fails;
  }
}

}  // namespace

extern "C" hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
  expect(fn != nullptr && args != nullptr, "a kernel");
  const uint64_t g[3] = {grid.x, grid.y, grid.z}, b[3] = {block.x, block.y, block.z};
  for (int i = 0; i < 3; ++i) {
    expect(g[i] > 0 && b[i] > 0, "a grid of nothing");
    expect(g[i] * b[i] < uint64_t{1} << 32, "more threads than a dispatch counts");
  }
  expect(grid.y < 65536 && grid.z < 65536, "more workgroups along y or z than a launch takes");
  expect(block.x <= 1024 && block.x % 64 == 0 && block.y == 1 && block.z == 1, "whole waves, 1024 threads at most");
  expect(lds <= 16 * 1024, "more LDS than the angles of a workgroup take");
  ++launches;
  groups += grid.x;
  return hipSuccess;
}

namespace {

alignas(256) char mem[1024];
void* const p = mem;   // no call reads or writes it: nothing is launched
float* const f = reinterpret_cast<float*>(mem);
int32_t* const n = reinterpret_cast<int32_t*>(mem);

void sections_of(int32_t (&s)[4], int32_t* axes, int64_t pairs, int want) {
  *axes = 0;
  for (int a = 0; a < want && pairs > 0; ++a) {
    const int64_t part = a == want - 1 || pairs == 1 ? pairs : (pairs + 1) / 2;
    s[(*axes)++] = static_cast<int32_t>(part);
    pairs -= part;
  }
}

void rotary(int64_t B, int64_t L, int64_t H, int64_t D, int axes, int32_t layout, int32_t dt) {
  dcn_rotary_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.length = L;
  d.heads = H;
  d.head_dim = D;
  sections_of(d.sections, &d.axes, D / 2, axes);
  d.layout = layout;
  d.dtype = dt;
  reset("rotary");
  expect(dcn_rotary(&d, p, p, f, p, nullptr) == DCN_OK && (B == 0 || L == 0 || launches > 0), "forward");
  reset("rotary gradients");
  expect(dcn_rotary_backward(&d, p, p, f, nullptr, p, nullptr, nullptr) == DCN_OK, "backward");
  expect(dcn_rotary_backward(&d, p, p, f, p, p, f, nullptr) == DCN_OK, "backward of positions");
}

void join(int64_t B, int64_t P, int64_t C, int32_t n1, int32_t n2, int32_t gate, int32_t dt) {
  dcn_residual_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.positions = P;
  d.channels = C;
  d.eps = 1e-5f;
  d.branch_norm = n1;
  d.next_norm = n2;
  d.gate = gate;
  d.dtype = dt;
  void* const next = mem + 512;
  size_t nb = 0;
  reset("join");
  expect(dcn_residual_norm(&d, p, p, p, p, p, p, p, p, p, next, f, nullptr) == DCN_OK, "forward");
  if (B * P > 0) expect(launches == 1, "one launch");
  reset("join gradients");
  expect(dcn_residual_norm_backward_workspace_bytes(&d, &nb) == DCN_OK && nb % 256 == 0, "workspace");
  void* const w1 = n1 != DCN_NORM_NONE ? p : nullptr;
  void* const w2 = n2 != DCN_NORM_NONE ? p : nullptr;
  void* const gg = gate != DCN_GATE_NONE ? p : nullptr;
  expect(dcn_residual_norm_backward(&d, p, p, p, p, p, p, p, f, p, p, p, p, gg, p, w1, w1, w2, w2, p, nb, nullptr) == DCN_OK,
         "backward");
  if (B * P > 0) expect(launches == 2, "two launches");
  // each run's sums have room
  const int64_t runs = groups;
  if (B * P > 0) {
    reset("join gradients without parameters");
    expect(dcn_residual_norm_backward(&d, p, p, p, p, p, p, p, f, p, p, p, p, nullptr, nullptr, nullptr, nullptr, nullptr,
                                      nullptr, nullptr, 0, nullptr) == DCN_OK &&
               launches == 1,
           "one launch, no workspace");
    expect(groups <= runs && static_cast<size_t>(groups) * 5 * C * 4 <= nb, "runs beyond the workspace");
  }
}

void append(int64_t B, int64_t L, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t width, int32_t dt) {
  dcn_append_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.length = L;
  d.query_heads = Hq;
  d.key_heads = Hkv;
  d.head_dim = D;
  d.num_pages = 1000;
  d.page_size = page;
  d.max_pages = width;
  sections_of(d.sections, &d.axes, D / 2, 2);
  d.dtype = dt;
  static char what[128];
  std::snprintf(what, sizeof(what), "append %lld x %lld, heads %lld %lld of %lld, pages of %lld", (long long)B, (long long)L, (long long)Hq,
                (long long)Hkv, (long long)D, (long long)page);
  reset(what);
  expect(dcn_paged_append(&d, p, p, p, nullptr, f, n, n, nullptr, p, p, p, n + 8, nullptr) == DCN_OK && launches > 0, "status");
}

void paged(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t width, int32_t dt) {
  dcn_paged_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.query_heads = Hq;
  d.key_heads = Hkv;
  d.head_dim = D;
  d.num_pages = 1000;
  d.page_size = page;
  d.max_pages = width;
  d.scale = 0.125f;
  d.dtype = dt;
  size_t nb = 0;
  reset("paged attention");
  expect(dcn_paged_attention_workspace_bytes(&d, &nb) == DCN_OK && nb % 256 == 0, "workspace");
  expect(dcn_paged_attention(&d, p, p, p, n, n, p, f, p, nb, nullptr) == DCN_OK, "status");
  const int64_t tiles = (Hq / Hkv + 15) / 16;
  expect(groups >= B * Hkv * tiles, "a workgroup for each sequence and key head at least");
  if (nb == 0) return;
  if (B <= 64) {
    expect(nb >= static_cast<size_t>(groups - B * Hq) * 16 * (D + 2) * 4, "a part for each workgroup");
  } else {   // one workgroup makes lists of G workgroups of each tile and of G - B sequences that are joined, 16 bytes each
    const int64_t heads = Hkv * tiles, G = (groups - 1 + B * Hq) / (heads + Hq);
    expect(1 + G * heads + (G - B) * Hq == groups && G > B, "workgroups of the lists");
    expect(nb >= static_cast<size_t>(heads) * 2 * (G - B) * 16 * (D + 2) * 4 + static_cast<size_t>(2 * G - B) * 16,
           "two parts for each workgroup beyond the sequences, and the lists");
  }
}

}  // namespace

int main() {
  for (int32_t dt : {static_cast<int32_t>(DCN_F32), static_cast<int32_t>(DCN_BF16)}) {
    for (int32_t layout : {DCN_ROTARY_HALVES, DCN_ROTARY_ADJACENT, DCN_ROTARY_BLOCKS})
      for (int64_t D : {2, 3, 8, 37, 40, 64, 128, 250, 511, 512})
        for (int axes : {1, 2, 3, 4})
          for (int64_t H : {1, 3, 8, 300})
            for (int64_t L : {1, 7, 1050, 16800}) rotary(3, L, H, D, axes, layout, dt);
    rotary(0, 5, 2, 64, 1, 0, dt);
    rotary(1, 2147483647, 1, 64, 2, 2, dt);
    rotary(2147483647, 1, 1, 2, 1, 0, dt);
    rotary(1, 1, 2147483647, 512, 4, 1, dt);
    rotary(40000, 49, 1000, 32, 2, 2, dt);
    for (int32_t gate : {DCN_GATE_NONE, DCN_GATE_BATCH, DCN_GATE_FULL})
      for (int32_t n1 : {DCN_NORM_NONE, DCN_NORM_LAYER})
        for (int32_t n2 : {DCN_NORM_NONE, DCN_NORM_RMS})
          for (int64_t C : {1, 7, 8, 9, 64, 81, 96, 128, 256, 500, 512, 520, 1030, 1536, 2048, 2600, 3500, 4096, 5000, 8191, 8192})
            for (int64_t P : {0, 1, 2, 300, 1551, 16800}) {
              join(1, P, C, n1, n2, gate, dt);
              join(3, P, C, n1, n2, gate, dt);
              join(700, P, C, n1, n2, gate, dt);
            }
    join(65530, 32000, 64, 2, 2, DCN_GATE_BATCH, dt);
    join(1, 2147483647, 8192, 2, 2, DCN_GATE_FULL, dt);
    join(2147483647, 1, 1, 2, 1, DCN_GATE_NONE, dt);
    for (int64_t D : {2, 37, 40, 64, 128, 512})
      for (int64_t L : {0, 1, 5, 4200})
        for (int64_t B : {1, 8, 70, 2000}) {
          append(B, L, 16, 4, D, 64, 300, dt);
          append(B, L, 0, 1, D, 1, 4000, dt);
          append(B, L, 64, 64, D, 24, 7, dt);
        }
    append(1000000, 1, 512, 256, 128, 16, 100, dt);
    append(1, 1, 1, 1, 64, 2147483647, 1, dt);
    append(1, 1, 1, 1, 64, 1, 2147483647, dt);
    for (int64_t D : {1, 8, 37, 64, 72, 128})
      for (int64_t B : {1, 2, 8, 64, 300, 5000})
        for (int64_t g : {1, 4, 16, 17, 40})
          for (int64_t width : {0, 1, 16, 300, 100000}) {
            paged(B, 4 * g, 4, D, 16, width, dt);
            paged(B, g, 1, D, 24, width, dt);
            paged(B, 64 * g, 64, D, 1, width, dt);
          }
    paged(1, 8, 8, 64, 2147418111, 1, dt);
    paged((1 << 23) - 1, 16, 16, 64, 16, 200, dt);
    paged(1, (1 << 27) - 1, (1 << 27) - 1, 32, 16, 200, dt);
  }
  if (fails == 0) std::printf("DECODER SANITIZE OK\n");
  return fails == 0 ? 0 : 1;
}

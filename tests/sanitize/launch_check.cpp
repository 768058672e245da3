// launch_check.cpp -- records the launches of the attention and group norm entry points (no GPU:
// hipLaunchKernel is this file's) and checks that each can be made: a dispatch counts the
// threads of each dimension of its grid in 32 bits, and none may be 0.
// Test infrastructure: built and run by tests/test_launch_shapes.py on the CPU.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>

#include "dcn.h"

namespace {

int fails = 0, launches = 0;
int64_t groups = 0;   // workgroups along x of the calls since reset()
int64_t chunks = 0;   // chunks of all batch elements, of the first launch since then
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

extern "C" hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t lds, hipStream_t) {
  const uint64_t g[3] = {grid.x, grid.y, grid.z}, b[3] = {block.x, block.y, block.z};
  for (int i = 0; i < 3; ++i) {
    expect(g[i] > 0 && b[i] > 0, "a grid of nothing");
    expect(g[i] * b[i] < uint64_t{1} << 32, "more threads than a dispatch counts");
  }
  expect(grid.y < 65536 && grid.z < 65536, "more workgroups along y or z than a launch takes");
  expect(block.x * block.y * block.z <= 1024, "too many threads a workgroup");
  expect(lds <= 160 * 1024, "more LDS than a CU has");
  if (launches == 0) chunks = static_cast<int64_t>(grid.x) * grid.z;
  ++launches;
  groups += grid.x;
  return hipSuccess;
}

namespace {

alignas(256) char mem[512];
void* const p = mem;   // no call reads or writes it: nothing is launched

dcn_norm_desc norm(int64_t B, int64_t P, int64_t C, int64_t G, int32_t dt) {
  dcn_norm_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.positions = P;
  d.channels = C;
  d.groups = G;
  d.eps = 1e-5f;
  d.activation = DCN_ACT_GELU;
  d.dtype = dt;
  return d;
}

// at: an address in `mem` (of another alignment than 16 bytes: rows are read element by element)
void run_norm(const dcn_norm_desc& d, bool slice, const char* what, void* at = p) {
  float* const f = reinterpret_cast<float*>(mem);
  size_t nf = 0, nb = 0;
  expect(dcn_group_norm_workspace_bytes(&d, &nf) == DCN_OK && dcn_group_norm_backward_workspace_bytes(&d, &nb) == DCN_OK,
         "workspace status");
  const int64_t part = d.groups * 8, chan = d.channels * 8, ws = nf, wb = nb;
  reset(what);
  expect(dcn_group_norm(&d, at, p, p, p, f, f, p, nf, nullptr) == DCN_OK, "status");
  if (slice) expect(groups >= d.batch * d.groups, "a workgroup for each group");
  else expect(launches == 2 && chunks * part <= ws, "parts beyond the workspace");
  reset(what);
  expect(dcn_group_norm_backward(&d, at, p, p, f, f, p, p, p, p, p, nb, nullptr) == DCN_OK, "gradients' status");
  if (slice) expect(groups >= d.batch * d.groups, "a workgroup for each group of the gradients");
  if (slice) expect(d.batch == 1 || d.batch * chan <= wb, "sums of the batch elements beyond the workspace");
  else expect(launches == 2 && chunks * (part + chan) <= wb, "parts of the gradients beyond the workspace");
}

dcn_attn_desc attn(int64_t B, int64_t Lq, int64_t Lk, int64_t Hq, int64_t Hkv, int64_t D, int32_t dt) {
  dcn_attn_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.query_len = Lq;
  d.key_len = Lk;
  d.query_heads = Hq;
  d.key_heads = Hkv;
  d.head_dim = D;
  const int64_t row[3] = {0, 1 << 10, 128};
  std::memcpy(d.q_stride, row, sizeof(row));
  std::memcpy(d.k_stride, row, sizeof(row));
  std::memcpy(d.v_stride, row, sizeof(row));
  d.scale = 0.125f;
  d.dtype = dt;
  return d;
}

// rows: of a tile of the forward
void run_attn(const dcn_attn_desc& d, int rows, const char* what) {
  float* const f = reinterpret_cast<float*>(mem);
  const int64_t pairs = d.batch * d.key_heads, r = d.query_len * (d.query_heads / d.key_heads);
  reset(what);
  expect(dcn_cross_attention(&d, p, p, p, nullptr, p, f, p, SIZE_MAX, nullptr) == DCN_OK, "status");
  expect(groups >= pairs * ((r + rows - 1) / rows), "a workgroup for each tile");
  reset(what);
  expect(dcn_cross_attention_backward(&d, p, p, p, nullptr, p, f, p, p, p, p, p, SIZE_MAX, nullptr) == DCN_OK,
         "gradients' status");
  expect(groups >= pairs * ((r + 127) / 128 + (d.key_len + 127) / 128), "a workgroup for each tile of the gradients");
}

}  // namespace

int main() {
  for (int32_t dt : {static_cast<int32_t>(DCN_F32), static_cast<int32_t>(DCN_BF16)}) {
    run_norm(norm(2, 1050, 256, 32, dt), true, "norm of a small map");
    run_norm(norm(8, 16800, 256, 32, dt), false, "norm of large maps");
    run_norm(norm(65528, 49, 64, 64, dt), true, "norm of many small maps, nearly 2^22 groups");
    run_norm(norm(32768, 49, 128, 128, dt), false, "norm of many small maps, 2^22 groups");
    run_norm(norm(65534, 7, 8192, 8192, dt), false, "norm of the most groups");
    run_norm(norm(65534, 3000, 8192, 64, dt), false, "norm of the most batch elements");
    run_norm(norm(1, 2147483647, 1, 1, dt), false, "norm of the most positions");
    // two passes, whatever the vectors' width: parts stay within the workspace
    for (int64_t B : {1, 2, 3, 100, 255, 256, 257, 3000})
      for (int64_t P : {8200, 8201, 16800, 1000003})
        for (int64_t Cg : {1, 3, 8, 64, 1024})
          for (int64_t G : {1, 4, 8})
            for (void* at : {p, static_cast<void*>(mem + (dt == DCN_BF16 ? 2 : 4))})
              run_norm(norm(B, P, Cg * G, G, dt), false, "norm in two passes", at);
  }
  for (int32_t dt : {static_cast<int32_t>(DCN_F32), static_cast<int32_t>(DCN_BF16)})
    for (int64_t D : {8, 20, 64, 128}) {
      run_attn(attn(2, 300, 4200, 8, 8, D, dt), 32, "attention of queries");
      run_attn(attn(2, 4200, 16800, 8, 8, D, dt), 128, "attention of a map");
      run_attn(attn(1 << 20, 1, 9, 16, 8, D, dt), 32, "attention of 2^23 pairs of one token");
      run_attn(attn(1 << 20, 49, 49, 4, 4, D, dt), 32, "attention of 2^22 windows");
      run_attn(attn(2000000, 97, 97, 4, 4, D, dt), 128, "attention of 8000000 windows in the rows form");
      run_attn(attn(1, 2000000000, 5, 1, 1, D, dt), 128, "attention of 2000000000 rows");
    }
  if (fails == 0) std::printf("LAUNCHES OK\n");
  return fails == 0 ? 0 : 1;
}

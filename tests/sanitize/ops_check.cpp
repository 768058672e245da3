// ops_check.cpp -- drives the host side of cross attention and group norm (descriptor checks,
// plans, workspace sizes, argument errors) with no GPU, so a host build with AddressSanitizer and
// UndefinedBehaviorSanitizer sees those paths.  No call here reaches a kernel launch: each one
// returns from the host checks.
// Test infrastructure: built and run by tests/test_sanitizers_ops.py on the CPU.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "dcn.h"

namespace {

int fails = 0;
void expect(bool ok, const char* what) {
  if (!ok) {
    std::printf("FAIL %s\n", what);
    ++fails;
  }
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
  d.scale = 0.125f;
  d.dtype = dt;
  return d;
}

dcn_norm_desc norm(int64_t B, int64_t P, int64_t C, int64_t G, int32_t act, int32_t dt) {
  dcn_norm_desc d;
  std::memset(&d, 0, sizeof(d));
  d.batch = B;
  d.positions = P;
  d.channels = C;
  d.groups = G;
  d.eps = 1e-5f;
  d.activation = act;
  d.dtype = dt;
  return d;
}

int attn_plan(const dcn_attn_desc& d) {
  size_t nf = 0, nb = 0;
  const int rf = dcn_cross_attention_workspace_bytes(&d, &nf), rb = dcn_cross_attention_backward_workspace_bytes(&d, &nb);
  expect(rf == rb, "forward and backward judge a descriptor alike");
  if (rf != DCN_OK || d.batch == 0 || d.query_len == 0 || d.key_len == 0) return rf;
  alignas(256) static char dummy[512];
  expect(dcn_cross_attention(&d, nullptr, dummy, dummy, nullptr, dummy, nullptr, dummy, nf, nullptr) == DCN_E_ARG,
         "attention without q");
  expect(dcn_cross_attention(&d, dummy, dummy, dummy, nullptr, nullptr, nullptr, dummy, nf, nullptr) == DCN_E_ARG,
         "attention without out");
  float* f = reinterpret_cast<float*>(dummy);
  if (nf > 0) {
    expect(dcn_cross_attention(&d, dummy, dummy, dummy, nullptr, dummy, nullptr, dummy, nf - 1, nullptr) ==
               DCN_E_WORKSPACE, "attention with a small workspace");
    expect(dcn_cross_attention(&d, dummy, dummy, dummy, nullptr, dummy, nullptr, dummy + 8, nf, nullptr) ==
               DCN_E_WORKSPACE, "attention with a misaligned workspace");
  }
  expect(nb > 0, "the backward has a workspace");
  expect(dcn_cross_attention_backward(&d, dummy, dummy, dummy, nullptr, dummy, nullptr, dummy, dummy, dummy, dummy,
                                      dummy, nb, nullptr) == DCN_E_ARG, "attention gradients without lse");
  expect(dcn_cross_attention_backward(&d, dummy, dummy, dummy, nullptr, dummy, f, dummy, dummy, dummy, dummy, dummy,
                                      nb - 1, nullptr) == DCN_E_WORKSPACE, "attention gradients with a small workspace");
  return rf;
}

int norm_plan(const dcn_norm_desc& d) {
  size_t nf = 0, nb = 0;
  const int rf = dcn_group_norm_workspace_bytes(&d, &nf), rb = dcn_group_norm_backward_workspace_bytes(&d, &nb);
  expect(rf == rb, "forward and backward judge a norm's descriptor alike");
  if (rf != DCN_OK || d.batch == 0) return rf;
  alignas(256) static char dummy[512];
  float* f = reinterpret_cast<float*>(dummy);
  expect(dcn_group_norm(&d, nullptr, nullptr, nullptr, dummy, nullptr, nullptr, dummy, nf, nullptr) == DCN_E_ARG,
         "norm without x");
  if (nf > 0)
    expect(dcn_group_norm(&d, dummy, nullptr, nullptr, dummy, nullptr, nullptr, nullptr, 0, nullptr) == DCN_E_WORKSPACE,
           "norm without workspace");
  expect(dcn_group_norm_backward(&d, dummy, nullptr, nullptr, nullptr, f, dummy, dummy, nullptr, nullptr, dummy, nb,
                                 nullptr) == DCN_E_ARG, "norm gradients without mean");
  if (nb > 0)
    expect(dcn_group_norm_backward(&d, dummy, nullptr, nullptr, f, f, dummy, dummy, nullptr, nullptr, dummy, nb - 1,
                                   nullptr) == DCN_E_WORKSPACE, "norm gradients with a small workspace");
  return rf;
}

}  // namespace

int main() {
  const int64_t top = std::numeric_limits<int64_t>::max();
  for (int32_t dt : {static_cast<int32_t>(DCN_F32), static_cast<int32_t>(DCN_BF16)}) {
    for (int64_t B : {0, 1, 3, 64})
      for (int64_t Lq : {0, 1, 33, 129, 4200})
        for (int64_t Lk : {0, 1, 65, 1050, 300000})
          for (int64_t g : {1, 3, 16})
            for (int64_t D : {1, 32, 40, 128}) expect(attn_plan(attn(B, Lq, Lk, 2 * g, 2, D, dt)) == DCN_OK, "a plan");
    const dcn_attn_desc ok = attn(2, 3, 5, 4, 2, 8, dt);
    for (int64_t bad : {int64_t{-1}, -top - 1}) {
      dcn_attn_desc d[] = {ok, ok, ok, ok, ok, ok, ok, ok, ok, ok};
      d[0].batch = d[1].query_len = d[2].key_len = d[3].query_heads = d[4].key_heads = d[5].head_dim = bad;
      d[6].q_stride[0] = d[7].k_stride[1] = d[8].v_stride[2] = d[9].mask_stride = bad;
      for (const auto& x : d) expect(attn_plan(x) == DCN_E_ARG, "a negative size or stride");
    }
    dcn_attn_desc d[] = {ok, ok, ok, ok, ok};
    d[0].batch = d[1].query_len = d[2].key_len = d[3].head_dim = top;
    d[4].query_heads = d[4].key_heads = top;
    for (const auto& x : d) expect(attn_plan(x) == DCN_E_UNSUPPORTED, "a huge size");
    for (float scale : {0.f, -1.f, NAN, INFINITY}) {
      dcn_attn_desc x = ok;
      x.scale = scale;
      expect(attn_plan(x) == DCN_E_ARG, "a scale that is none");
    }
    dcn_attn_desc x = ok;
    x.query_heads = 5;
    expect(attn_plan(x) == DCN_E_ARG, "heads that do not divide");
    for (auto& s : x.q_stride) s = top;   // 64-bit strides are taken as they are
    x.query_heads = 4;
    expect(attn_plan(x) == DCN_OK, "large strides");

    for (int64_t B : {0, 1, 2, 9})
      for (int64_t P : {1, 7, 1050, 16800, 2000000})
        for (int64_t Cg : {1, 3, 8, 12, 256})
          for (int64_t G : {1, 5, 32})
            for (int32_t act = DCN_ACT_NONE; act <= DCN_ACT_GELU; ++act)
              expect(norm_plan(norm(B, P, Cg * G, G, act, dt)) == DCN_OK, "a norm's plan");
    const dcn_norm_desc n = norm(2, 9, 32, 4, DCN_ACT_SILU, dt);
    dcn_norm_desc m[] = {n, n, n, n, n, n, n};
    m[0].batch = -1;
    m[1].positions = 0;
    m[2].channels = 30;
    m[3].groups = 0;
    m[4].eps = -1.f;
    m[5].eps = NAN;
    m[6].activation = 4;
    for (const auto& y : m) expect(norm_plan(y) == DCN_E_ARG, "a norm's descriptor that is none");
    dcn_norm_desc h[] = {n, n, n};
    h[0].batch = h[1].positions = top;
    h[2].channels = h[2].groups = top;
    for (const auto& y : h) expect(norm_plan(y) == DCN_E_UNSUPPORTED, "a norm of a huge size");
  }
  expect(dcn_cross_attention_workspace_bytes(nullptr, nullptr) == DCN_E_ARG, "no descriptor");
  expect(dcn_group_norm_workspace_bytes(nullptr, nullptr) == DCN_E_ARG, "no norm descriptor");
  if (fails == 0) std::printf("OPS SANITIZE OK\n");
  return fails == 0 ? 0 : 1;
}

// Drives the host code of the layer operators (gdr_layer_api.cpp: argument checks
// and workspace sizes of every entry point) under AddressSanitizer and
// UndefinedBehaviorSanitizer, on a machine without a GPU.  The kernel launchers are
// stubs that count calls: no path here may reach one (invalid arguments are
// refused before, and a valid problem stops at the device check).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <random>

#include "gdr_kernels.h"
#include "gdr_layer.h"

static int g_launches = 0;
namespace gdr {
static hipError_t count() { ++g_launches; return hipErrorUnknown; }
int compute_units() { return 256; }
hipError_t launch_fwd_prep(bool, const Problem &, const Workspace &, bool, bool, hipStream_t) { return count(); }
hipError_t launch_fwd_walk(bool, const Problem &, const Workspace &, uint16_t *, float *, bool, bool, hipStream_t) { return count(); }
hipError_t launch_bwd_walk(bool, const Problem &, const Workspace &, const uint16_t *, const float *, float *, hipStream_t) { return count(); }
hipError_t launch_bwd_grad(bool, const Problem &, const Workspace &, const uint16_t *, uint16_t *, uint16_t *, uint16_t *, float *, void *, hipStream_t) { return count(); }
hipError_t launch_conv_fwd(const gdr_conv &, void *, int64_t, void *, hipStream_t) { return count(); }
hipError_t launch_conv_bwd(const gdr_conv &, const void *, int64_t, const void *, void *, int64_t, void *, float *, hipStream_t) { return count(); }
hipError_t launch_conv_step(const gdr_conv &, void *, int64_t, void *, const int32_t *, int32_t, hipStream_t) { return count(); }
hipError_t launch_gate_fwd(const gdr_gate &, float *, hipStream_t) { return count(); }
hipError_t launch_gate_bwd(const gdr_gate &, const float *, void *, int64_t, float *, hipStream_t) { return count(); }
hipError_t launch_step(bool, const gdr_step &, uint16_t *, hipStream_t) { return count(); }
hipError_t launch_norm_fwd(const gdr_norm &, void *, hipStream_t) { return count(); }
hipError_t launch_norm_bwd(const gdr_norm &, const void *, const void *, void *, int64_t, void *, int64_t, void *, float *, int, hipStream_t) { return count(); }
int norm_bwd_workers(const gdr_norm &) { return 1; }
hipError_t launch_conv_sum(const float *, int, int, int, float *, float *, hipStream_t) { return count(); }
hipError_t launch_gate_sum(const float *, int, int, int, float *, float *, hipStream_t) { return count(); }
hipError_t launch_norm_sum(const float *, int, int, float *, hipStream_t) { return count(); }
}  // namespace gdr

static int g_fail = 0;
#define CHECK(c)                                                          \
  do {                                                                    \
    if (!(c)) {                                                           \
      std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
      ++g_fail;                                                           \
    }                                                                     \
  } while (0)

static int32_t pick(std::mt19937 &r) {
  static const int32_t v[] = {INT32_MIN, -1, 0, 1, 2, 3, 4, 8, 48, 63, 64, 65, 128, 129, 4096, 16384, 16385, 65536, 1 << 24, 1 << 28, INT32_MAX};
  return v[r() % (sizeof v / sizeof *v)];
}

int main() {
  std::mt19937 r(5);
  alignas(256) static unsigned char buf[4096];  // never dereferenced by the calls: no launch happens
  auto ptr = [&]() -> void * { return r() % 5 ? buf + (r() % 4 ? 0 : r() % 9) : nullptr; };
  int refused = 0;
  for (int i = 0; i < 200000; ++i) {
    gdr_conv c{};
    c.T = pick(r); c.N = pick(r); c.C = pick(r); c.W = pick(r) % 10; c.dtype = r() % 3; c.w_dtype = r() % 3; c.activation = r() % 4;
    c.n_chunks = pick(r); c.x_stride = pick(r); c.x = ptr(); c.weight = ptr(); c.bias = ptr(); c.s0 = ptr();
    c.chunk_table = static_cast<const int32_t *>(ptr());
    refused += gdr_conv_fwd(&c, ptr(), pick(r), ptr(), nullptr) != GDR_OK;
    refused += gdr_conv_bwd(&c, ptr(), pick(r), ptr(), ptr(), pick(r), (float *)ptr(), (float *)ptr(), ptr(), ptr(), pick(r), nullptr) != GDR_OK;
    refused += gdr_conv_step(&c, ptr(), pick(r), ptr(), (const int32_t *)ptr(), pick(r), nullptr) != GDR_OK;
    const int64_t cb = gdr_conv_workspace_bytes(c.n_chunks, c.C, c.W, c.dtype);
    CHECK(cb < 0 ? cb >= -(int64_t)GDR_ERR_WORKSPACE : cb % 256 == 0);
    gdr_gate g{};
    g.T = pick(r); g.H = pick(r); g.D = pick(r); g.dtype = r() % 3; g.kind = r() % 3; g.floor = (int)(r() % 11) - 9; g.x_stride = pick(r);
    g.x = ptr(); g.a_log = (const float *)ptr(); g.bias = (const float *)ptr();
    refused += gdr_gate_fwd(&g, (float *)ptr(), nullptr) != GDR_OK;
    refused += gdr_gate_bwd(&g, (const float *)ptr(), ptr(), pick(r), (float *)ptr(), (float *)ptr(), ptr(), pick(r), nullptr) != GDR_OK;
    const int64_t gb = gdr_gate_workspace_bytes(g.T, g.H, g.D, g.dtype);
    CHECK(gb < 0 ? gb >= -(int64_t)GDR_ERR_WORKSPACE : gb % 256 == 0);
    gdr_step s{};
    s.T = pick(r); s.N = pick(r); s.H_qk = pick(r); s.H_v = pick(r); s.K = r() % 8 ? 128 : pick(r); s.V = 128; s.n_slots = pick(r);
    s.input_flags = r() % 5; s.scale = r() % 9 ? 1.f : 0.f / 0.f; s.q_stride = pick(r); s.k_stride = pick(r); s.v_stride = pick(r);
    s.q = s.k = s.v = (const uint16_t *)ptr(); s.g = (const float *)ptr(); s.beta = ptr(); s.cu_seqlens = (const int32_t *)ptr();
    s.slots = (const int32_t *)ptr(); s.state = (float *)ptr();
    refused += gdr_kda_step(&s, (uint16_t *)ptr(), nullptr) != GDR_OK;
    refused += gdr_gdn_step(&s, (uint16_t *)ptr(), nullptr) != GDR_OK;
    gdr_norm n{};
    n.T = pick(r); n.H = pick(r); n.D = pick(r); n.dtype = r() % 3; n.res_dtype = r() % 3; n.w_dtype = r() % 3; n.activation = r() % 4;
    n.placement = r() % 4; n.scale = 1.f; n.eps = (int)(r() % 3) - 1; n.x_stride = pick(r); n.gate_stride = pick(r);
    n.x = ptr(); n.weight = ptr(); n.gate = ptr(); n.residual = ptr(); n.s = ptr();
    refused += gdr_norm_fwd(&n, ptr(), nullptr) != GDR_OK;
    refused += gdr_norm_bwd(&n, ptr(), ptr(), ptr(), pick(r), ptr(), pick(r), ptr(), (float *)ptr(), ptr(), pick(r), nullptr) != GDR_OK;
    const int64_t nb = gdr_norm_workspace_bytes(n.T, n.H, n.D);
    CHECK(nb < 0 ? nb >= -(int64_t)GDR_ERR_WORKSPACE : nb % 256 == 0);
    CHECK(gdr_last_error() != nullptr);
  }
  CHECK(gdr_conv_fwd(nullptr, buf, 1, nullptr, nullptr) == GDR_ERR_INVALID_ARG);
  CHECK(gdr_gate_fwd(nullptr, nullptr, nullptr) == GDR_ERR_INVALID_ARG);
  CHECK(gdr_kda_step(nullptr, nullptr, nullptr) == GDR_ERR_INVALID_ARG);
  CHECK(gdr_norm_fwd(nullptr, nullptr, nullptr) == GDR_ERR_INVALID_ARG);
  // lane maps: every group of a row is some block's, and the workers' partials fit the size
  for (int groups = 1; groups < 5000; ++groups) {
    const gdr::Lanes l = gdr::lanes_for(groups);
    CHECK(l.lx >= 1 && l.ly >= 1 && l.threads <= 256 && l.threads % 64 == 0 && l.lx * l.ly <= l.threads);
    CHECK((int64_t)l.lx * l.nchb >= groups && (!l.uniform || l.lx % 64 == 0));
  }
  for (int i = 0; i < 100000; ++i) {
    const int nc = r() % 3 ? r() % 5000 : r() % (1 << 28), C = 1 + (r() % 2 ? r() % 4096 : r() % (1 << 24));
    const gdr::ConvBwdPlan p = gdr::conv_bwd_plan(nc, C);
    CHECK(p.workers % p.lanes.ly == 0 && p.workers >= 0 && (nc == 0) == (p.workers == 0));
    CHECK(64 % p.run == 0 && (int64_t)nc * (64 / p.run) < (int64_t(1) << 31));
    CHECK((int64_t)p.rows() * p.lanes.nchb < (int64_t(1) << 31));
  }
  std::printf("%d refused, %d failures, %d launches\n", refused, g_fail, g_launches);
  return g_fail || g_launches ? 1 : 0;
}

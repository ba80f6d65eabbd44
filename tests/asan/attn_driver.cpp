// Drives the host code of the softmax-attention layers' operators (gdr_attn_api.cpp:
// argument checks, tile planner, frequencies, workspace sizes) under AddressSanitizer and
// UndefinedBehaviorSanitizer, on a machine without a GPU.  The kernel launchers are
// stubs that count calls: no path here may reach one (invalid arguments are
// refused before, and a valid problem stops at the device check).
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "gdr_attn.h"
#include "gdr_kernels.h"

static int g_launches = 0;
namespace gdr {
static hipError_t count() { ++g_launches; return hipErrorUnknown; }
int compute_units() { return 256; }
hipError_t launch_fwd_prep(bool, const Problem &, const Workspace &, bool, bool, hipStream_t) { return count(); }
hipError_t launch_fwd_walk(bool, const Problem &, const Workspace &, uint16_t *, float *, bool, bool, hipStream_t) { return count(); }
hipError_t launch_bwd_walk(bool, const Problem &, const Workspace &, const uint16_t *, const float *, float *, hipStream_t) { return count(); }
hipError_t launch_bwd_grad(bool, const Problem &, const Workspace &, const uint16_t *, uint16_t *, uint16_t *, uint16_t *, float *, void *, hipStream_t) { return count(); }
hipError_t launch_rope(const gdr_rope &, bool, const void *, int64_t, const void *, int64_t, void *, int64_t, void *, int64_t, hipStream_t) { return count(); }
hipError_t launch_attn_fwd(const gdr_attn &, uint16_t *, float *, void *, hipStream_t) { return count(); }
hipError_t launch_attn_fwd_join(const gdr_attn &, uint16_t *, float *, void *, hipStream_t) { return count(); }
hipError_t launch_attn_dq(const gdr_attn &, const uint16_t *, const float *, const uint16_t *, uint16_t *, int64_t, void *, hipStream_t) { return count(); }
hipError_t launch_attn_dkv(const gdr_attn &, const uint16_t *, uint16_t *, int64_t, uint16_t *, int64_t, void *, hipStream_t) { return count(); }
hipError_t launch_attn_bwd_join(const gdr_attn &, uint16_t *, int64_t, uint16_t *, int64_t, uint16_t *, int64_t, void *, hipStream_t) { return count(); }
hipError_t launch_kv(const gdr_kv &, bool, int32_t, const int32_t *, const int32_t *, uint16_t *, int64_t, uint16_t *, int64_t, hipStream_t) { return count(); }
hipError_t launch_attn_step(const gdr_kv &, const gdr_attn_step &, uint16_t *, void *, const StepPlan &, hipStream_t) { return count(); }
hipError_t launch_attn_step_join(const gdr_kv &, const gdr_attn_step &, uint16_t *, void *, const StepPlan &, hipStream_t) { return count(); }
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
  static const int32_t v[] = {INT32_MIN, -1, 0, 1, 2, 3, 4, 8, 16, 48, 63, 64, 65, 128, 129, 256, 1024, 4096, 65536, 1 << 24, 1 << 28, 1 << 30, INT32_MAX};
  return v[r() % (sizeof v / sizeof *v)];
}
static void *address(std::mt19937 &r) {
  static const uintptr_t v[] = {0, 4096, 4098, 8192, 1 << 20, (1 << 20) + 16, 1 << 24};
  return reinterpret_cast<void *>(v[r() % (sizeof v / sizeof *v)]);
}
// Fields of a problem drawn at random, most of them from those of a valid one.
template <class T>
static T shake(const T &good, std::mt19937 &r) {
  T p = good;
  unsigned char *b = reinterpret_cast<unsigned char *>(&p);
  for (int i = 0; i < 2; ++i) {
    const size_t at = r() % (sizeof(T) / 4) * 4;
    const int32_t x = pick(r);
    std::memcpy(b + at, &x, 4);
  }
  return p;
}

int main() {
  std::mt19937 r(7);
  void *ws = reinterpret_cast<void *>(uintptr_t(1) << 26);
  for (int i = 0; i < 200000; ++i) {
    const int64_t s = pick(r), s2 = pick(r);
    gdr_rope rope{64, 1, 4, 2, 128, 64, GDR_BF16, GDR_ROPE_HALF, 1, 1.f, 512, 256, (void *)4096, (void *)8192, nullptr, (int32_t *)4096, (double *)4096};
    rope = shake(rope, r);
    CHECK(gdr_rope_fwd(&rope, address(r), s, address(r), s2, nullptr) != GDR_OK);
    CHECK(gdr_rope_bwd(&rope, address(r), s, address(r), s2, address(r), s, address(r), s2, nullptr) != GDR_OK);
    gdr_kv kv{10, 16, 2, 128, 3, 4, (uint8_t *)4096, (uint8_t *)8192, (uint8_t *)(1 << 20), (uint8_t *)(1 << 21), (int32_t *)(1 << 22)};
    gdr_attn_step step{3, 4, 0, 0.1f, 512, (uint16_t *)(1 << 23), (int32_t *)(1 << 24), nullptr};
    const gdr_kv c = shake(kv, r);
    CHECK(gdr_kv_store(&c, 3, nullptr, nullptr, (uint16_t *)address(r), s, (uint16_t *)address(r), s2, nullptr) != GDR_OK);
    CHECK(gdr_kv_load(&c, pick(r), (int32_t *)address(r), nullptr, (uint16_t *)address(r), s, (uint16_t *)address(r), s2, nullptr) != GDR_OK);
    const gdr_attn_step p = shake(step, r);
    CHECK(gdr_attn_step_fwd(&c, &p, (uint16_t *)address(r), ws, INT64_MAX, nullptr) != GDR_OK);
    gdr_attn_step_workspace_bytes(pick(r), pick(r), pick(r), pick(r), pick(r), pick(r));
    double f[512];
    const double v[] = {0., -1., 1., 1e4, 1e300, 1e-300, 1. / 0., 0. / 0.};
    gdr_rope_freqs(pick(r), v[r() % 8], pick(r) % 5, v[r() % 8], v[r() % 8], v[r() % 8], v[r() % 8], f);
  }
  for (int i = 0; i < 3000; ++i) {
    std::vector<int32_t> q{0}, k{0};
    for (int n = r() % 6; n > 0; --n) q.push_back(q.back() + (r() % 4 ? r() % 700 : 0)), k.push_back(k.back() + (r() % 4 ? r() % 9000 : 0));
    const int32_t N = (int32_t)q.size() - 1, causal = r() % 3 != 0, window = causal && r() % 2 ? 1 + r() % 800 : 0;
    gdr_attn_plan plan;
    CHECK(gdr_plan_attn(q.data(), k.data(), N, causal, window, nullptr, 0, &plan) == GDR_OK);
    std::vector<int32_t> table((size_t)plan.table_len);
    gdr_attn_plan again;
    CHECK(gdr_plan_attn(q.data(), k.data(), N, causal, window, table.data(), plan.table_len, &again) == GDR_OK || plan.table_len == 0);
    gdr_attn a{q.back(), k.back(), N, 4, 2, 128, causal, window, plan, 0.1f, 512, 256, 256, (uint16_t *)4096, (uint16_t *)8192, (uint16_t *)(1 << 20), (int32_t *)(1 << 21)};
    const int64_t fwd = gdr_attn_workspace_bytes(&a, 0), bwd = gdr_attn_workspace_bytes(&a, 1);
    CHECK(fwd >= 0 && bwd >= 0);
    // the share that a launch takes lies within the table
    for (const gdr::AttnShare &s : {gdr::attn_q_share(a), gdr::attn_k_share(a)})
      if (s.level >= 0) {
        CHECK(s.items + 2 * s.blocks <= plan.table_len);
        for (int64_t x = 0; x < s.blocks; ++x) CHECK(table[s.items + 2 * x] >= 0 && (table[s.items + 2 * x + 1] >> 16) <= s.parts);
      }
    for (int j = 0; j < 40; ++j) {
      const gdr_attn b = shake(a, r);
      CHECK(gdr_attn_fwd(&b, (uint16_t *)address(r), (float *)address(r), j % 2 ? ws : nullptr, INT64_MAX, nullptr) != GDR_OK);
      CHECK(gdr_attn_bwd(&b, (uint16_t *)4096, (float *)4096, (uint16_t *)8192, (uint16_t *)address(r), pick(r), (uint16_t *)address(r), 256, (uint16_t *)address(r), 256, ws,
                         INT64_MAX, nullptr) != GDR_OK);
      gdr_attn_workspace_bytes(&b, j % 2);
    }
  }
  std::printf("%d failures, %d launches\n", g_fail, g_launches);
  return g_fail != 0;
}

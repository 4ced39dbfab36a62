// Argument sweep of the attention entry points under host AddressSanitizer and
// UndefinedBehaviorSanitizer (built and run by tests/test_abi_kv_sanitize.py on
// a machine without a GPU).  Every call must return a status without touching
// memory it was not given; valid-looking calls stop at the device check, so no
// kernel is launched and the dummy addresses are never dereferenced.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "mq.h"

namespace {
int g_calls = 0, g_bad = 0;
void expect_status(int s, const char* what) {
  ++g_calls;
  if (s < MQ_OK || s > MQ_ERR_HIP) {
    std::printf("%s: status %d out of range\n", what, s);
    ++g_bad;
  }
}
}  // namespace

int main() {
  auto* P = reinterpret_cast<uint8_t*>(0x10000);
  auto* F = reinterpret_cast<float*>(0x10000);
  auto* I = reinterpret_cast<int32_t*>(0x10000);
  auto* D = reinterpret_cast<double*>(0x10000);
  auto* H = reinterpret_cast<uint16_t*>(0x10000);
  auto* H2 = reinterpret_cast<uint16_t*>(0x20000);
  const int64_t wide[] = {INT64_MIN, -1, 0, 1, 8, 64, 1024, (int64_t)1 << 20, (int64_t)1 << 31,
                          (int64_t)1 << 40, (int64_t)1 << 62, INT64_MAX};
  const int32_t ints[] = {INT_MIN, -1, 0, 1, 8, 16, 64, 128, 1 << 20, 1 << 24, INT_MAX};

  for (int64_t pages : wide)
    for (int32_t heads : ints)
      for (int32_t block : ints)
        for (int32_t dim : ints) {
          mq_kv_cache c{P, P, F, F, pages, heads, block, dim, MQ_KV_INT8};
          mq_kv_batch b{I, I, I, 4, 2, 8, 2};
          expect_status(mq_cache_read(&c, &b, P, P, MQ_F32, nullptr), "read");
          expect_status(mq_cache_append(&c, &b, nullptr, P, P, 1024, nullptr, 0, 0, MQ_BF16,
                                        nullptr, nullptr),
                        "append");
          (void)mq_cache_attend_workspace_bytes(&c, &b, 8, 0);
        }
  mq_kv_cache c{P, P, F, F, 100, 8, 64, 128, MQ_KV_E4M3};
  for (int64_t rows : wide)
    for (int32_t seqs : ints)
      for (int32_t table : ints)
        for (int32_t most : ints) {
          mq_kv_batch b{I, I, I, rows, seqs, table, most};
          expect_status(mq_cache_read(&c, &b, P, nullptr, MQ_BF16, nullptr), "read");
          for (int64_t qh : {(int64_t)8, (int64_t)32, (int64_t)8192, INT64_MAX}) {
            const size_t need = mq_cache_attend_workspace_bytes(&c, &b, qh, 0);
            expect_status(mq_cache_attend(&c, &b, H, 4096, qh, 0.1f, 0.f, 0, 1, H2, nullptr, P, need,
                                          nullptr),
                          "attend");
          }
        }
  mq_kv_batch b{I, I, I, 4, 2, 64, 2};
  for (int64_t w : wide)
    for (int64_t v : wide) {
      (void)mq_cache_attend_workspace_bytes(&c, &b, w, v);
      expect_status(mq_cache_attend(&c, &b, H, w, 32, 0.1f, 0.f, v, 1, H2, F, P, SIZE_MAX, nullptr),
                    "attend");
      expect_status(mq_cache_attend(&c, &b, H, 4096, w, NAN, -1.f, v, 2, H2, F, nullptr, 0, nullptr),
                    "attend");
      expect_status(mq_cache_append(&c, &b, nullptr, P, P, w, P, v, 32, MQ_F32, H2, nullptr),
                    "append");
      expect_status(mq_cache_append(&c, &b, nullptr, P, P, 1024, P, 4096, w, (int)v, H2, nullptr),
                    "append");
      for (int32_t rot : ints) {
        mq_rope_spec r{D, 1.0, rot, 0};
        expect_status(mq_rope(&r, I, P, MQ_BF16, w, 4, 8, v, H2, w, nullptr), "rope");
        expect_status(mq_rope(&r, I, P, MQ_F32, 1024, w, v, 128, H2, 1024, nullptr), "rope");
      }
    }
  mq_rope_spec r{D, 1.0, 64, 1};
  mq_linear l{P, F, F, 1024, 1024, 1024};
  mq_layer layer{8, l, l, l, l, l, l, l};
  for (int64_t m : wide)
    for (int32_t heads : ints) {
      mq_kv_cache lc{P, P, F, F, 100, heads, 64, 128, MQ_KV_INT8};
      mq_stack_attention at{&lc, &b, &r, nullptr, 8, 0.1f, 0.f};
      (void)mq_mixnmatch_attend_workspace_bytes(&layer, 1, &at, m);
      expect_status(mq_mixnmatch_attend(&layer, 1, &at, H, m, F, P, SIZE_MAX, nullptr), "stack");
      expect_status(mq_mixnmatch_attend(&layer, heads, nullptr, H, m, F, P, 0, nullptr), "stack");
    }
  std::printf("%d calls, %d unexpected\n", g_calls, g_bad);
  return g_bad != 0;
}

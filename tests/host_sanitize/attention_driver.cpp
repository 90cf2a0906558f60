// Host-only exercise of the attention-side host layer (attention_api.cpp, the rules in kv_attention.hip) under
// AddressSanitizer and UndefinedBehaviorSanitizer: argument checks with sizes and strides up to the largest their
// types hold.  The launchers below stand in for the GPU side and note what they are given.
// Prints "ok <checks>" and exits 0 when everything is as documented.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "../../calibration_free_w4a4_amd/csrc/attention.h"
#include "../../include/orbq.h"

namespace {
int g_checks = 0, g_fail = 0, g_launches = 0;

void expect(bool good, const char* what, int line) {
  ++g_checks;
  if (!good) {
    ++g_fail;
    std::printf("FAIL line %d: %s (%s)\n", line, what, orbq_last_error());
  }
}
#define EXPECT(x) expect((x), #x, __LINE__)
}  // namespace

namespace orbq {
int launch_rope(const RopeArgs&, int, hipStream_t) { return ++g_launches, 0; }
int launch_kv_append(const KvCache&, const KvTokens&, int, hipStream_t) { return ++g_launches, 0; }
int launch_kv_read(const KvCache&, const KvTokens&, int, hipStream_t) { return ++g_launches, 0; }
template <> int launch_attn<64>(const AttnArgs&, const AttnPlan&, hipStream_t) { return ++g_launches, 0; }
template <> int launch_attn<128>(const AttnArgs&, const AttnPlan&, hipStream_t) { return ++g_launches, 0; }
template <> int launch_attn<256>(const AttnArgs&, const AttnPlan&, hipStream_t) { return ++g_launches, 0; }
}  // namespace orbq

namespace {
void* const P = reinterpret_cast<void*>(uintptr_t{0x10000});
int32_t* const I = static_cast<int32_t*>(P);
float* const F = static_cast<float*>(P);
int8_t* const C = static_cast<int8_t*>(P);

int rope_with(int64_t xt, int64_t xh, int64_t yt, int64_t yh, int64_t n, int32_t heads, orbq_dtype type) {
  const orbq_rope r{1, {64, 0, 0, 0}, F, ORBQ_ROPE_PAIRS};
  const orbq_heads t{P, P, heads, xt, xh, yt, yh};
  return orbq_rope_apply(&r, F, n, n, 64, &t, 1, type, 0, nullptr);
}

orbq_kv_cache cache(int32_t heads = 2, int32_t page = 64, int32_t d = 128) { return {C, C, F, F, 8, heads, page, d}; }

int move(bool read, int64_t kt, int64_t kh, int64_t vt, int64_t vh) {
  const orbq_kv_cache c = cache();
  const orbq_page_table t{I, 4, 4, 2};
  return read ? orbq_kv_read(&c, &t, I, I, 6, 3, P, kt, kh, P, vt, vh, ORBQ_BF16, nullptr)
              : orbq_kv_append(&c, &t, I, I, 6, 3, P, kt, kh, P, vt, vh, ORBQ_BF16, nullptr);
}

int attend(int64_t qt, int64_t qh, int64_t ot, int64_t oh) {
  const orbq_kv_cache c = cache();
  const orbq_page_table t{I, 4, 4, 2};
  return orbq_kv_attention(&c, &t, I, I, 6, 3, 0, P, qt, qh, 4, P, ot, oh, nullptr, ORBQ_BF16, 0.1f, 1, 0, nullptr, 0, nullptr);
}

void strides() {
  const int64_t huge[] = {INT64_MAX, INT64_MAX - 1, INT64_MAX - 7, INT64_MAX / 2 + 1, INT64_MAX / 3, INT64_MAX / 16 * 16,
                          INT64_C(1) << 62, INT64_C(1) << 45};
  for (int64_t s : huge) {
    // a multiple of the alignment is not refused, whatever it is; others are, for that reason
    const bool by8 = s % 8 == 0, by4 = s % 4 == 0;
    EXPECT(rope_with(s, s, 64 * 5, 64, 6, 5, ORBQ_F32) == ORBQ_OK);
    EXPECT(rope_with(320, 64, s, 64, 6, 5, ORBQ_F32) == ORBQ_OK && rope_with(320, 64, 64, s, 6, 5, ORBQ_BF16) == ORBQ_OK);
    EXPECT(rope_with(320, 64, s, s, 6, 5, ORBQ_F32) == ORBQ_ERR_INVALID_ARG);
    EXPECT(rope_with(320, 64, s, s - 64, 2, 2, ORBQ_F32) == ORBQ_OK);
    EXPECT(rope_with(320, 64, s, s - 64, 16000, 16000, ORBQ_F32) == ORBQ_OK);
    EXPECT(rope_with(320, 64, s, s / 2, 3, 3, ORBQ_F32) == ORBQ_ERR_INVALID_ARG);
    for (const bool read : {false, true}) {
      EXPECT(move(read, s, 128, 256, 128) == (by8 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
      EXPECT(move(read, 256, 128, 128, s) == (by8 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
    }
    EXPECT(attend(s, 128, 512, 128) == (by8 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
    EXPECT(attend(512, s, 512, 128) == (by8 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
    EXPECT(attend(512, 128, s, 128) == (by4 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
    EXPECT(attend(512, 128, 128, s) == (by4 ? ORBQ_OK : ORBQ_ERR_ALIGNMENT));
  }
}
}  // namespace

int main() {
  strides();
  EXPECT(g_launches > 0);
  if (g_fail) {
    std::printf("%d of %d failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("ok %d\n", g_checks);
  return 0;
}

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

// ---- the plan: what the kernels take from it, recomputed here for sequences of every kind
struct Case {
  int32_t batch, max_new, heads, kv_heads, d, block, window;
  int64_t total, max_len;
  bool bound;
};

orbq::AttnPlan plan_of(const Case& c) {
  return orbq::plan_attention(c.batch, c.total, c.max_new, c.heads, c.kv_heads, c.d, c.max_len, c.block, c.window, c.bound, 256);
}

// visible keys of the query at `pos` of a sequence of `len`
void visible(const Case& c, int64_t pos, int64_t len, int64_t* lo, int64_t* hi) {
  *hi = len;
  if (c.block) {
    const int64_t end = pos < 0 ? 0 : (pos / c.block + 1) * c.block;
    if (end < *hi) *hi = end;
  }
  *lo = c.window && *hi > c.window ? *hi - c.window : 0;
}

// every row tile's 64-key tiles are covered by its parts, in order and without a gap, and the turned tiles hold them
void covers(const Case& c, const orbq::AttnPlan& p, int64_t len, int64_t rows) {
  const int64_t group = c.heads / c.kv_heads, tile_rows = p.many ? orbq::many_rows(c.d) : 16 * p.rt;
  const int64_t done = rows < c.max_new ? rows : c.max_new;
  int64_t lo, hi, stream_first;
  visible(c, len - rows, len, &lo, &hi);
  stream_first = lo / 64;
  EXPECT(done * group <= p.row_tiles * tile_rows);
  for (int64_t r0 = 0; r0 < done * group; r0 += tile_rows) {
    const int64_t r1 = r0 + tile_rows < done * group ? r0 + tile_rows : done * group;
    int64_t first, last, x;
    visible(c, len - rows + r0 / group, len, &first, &x);
    visible(c, len - rows + (r1 - 1) / group, len, &x, &last);
    const int64_t t_end = (last + 63) / 64;
    for (const int parts : {1, p.splits}) {
      int64_t at = first / 64;
      for (int split = 0; split < parts; ++split) {
        const int64_t t0 = first / 64 + static_cast<int64_t>(split) * p.chunk;
        const int64_t t1 = split + 1 < parts && t0 + p.chunk < t_end ? t0 + p.chunk : t_end;
        if (t0 >= t1) continue;
        if (t0 != at) return EXPECT(t0 == at);
        at = t1;
      }
      EXPECT(at == t_end || t_end <= first / 64);
    }
    if (p.turned) EXPECT(t_end - stream_first <= p.turned);
  }
}

void plans() {
  const int32_t dims[] = {64, 128, 256}, blocks[] = {0, 1, 37, 1560, 1 << 30}, windows[] = {0, 1, 500, 5000, INT32_MAX};
  const int64_t lens[] = {1, 64, 777, 5000, 40000};
  for (int32_t d : dims)
    for (int32_t block : blocks)
      for (int32_t window : windows)
        for (int64_t len : lens)
          for (int32_t max_new : {1, 3, 17, 70, 700, 4680})
            for (int32_t batch : {1, 5})
              for (int32_t heads : {2, 24})
                for (const bool even : {true, false}) {
                  const Case c{batch, max_new, heads, 2, d, block, window, even ? batch * int64_t{max_new} : batch * int64_t{max_new} / 2 + 1, len, even};
                  const orbq::AttnPlan p = plan_of(c);
                  EXPECT(p.splits >= 1 && p.chunk >= 1 && p.whole >= 0 && p.part_rows >= 0);
                  EXPECT(c.bound || !p.turned);
                  if (p.many) EXPECT(p.part_rows + int64_t{p.whole} * orbq::many_rows(d) == int64_t{batch} * 2 * p.row_tiles * orbq::many_rows(d));
                  for (const int64_t n : {len, len / 3, int64_t{0}})
                    for (const int64_t rows : {int64_t{1}, int64_t{max_new}, 2 * int64_t{max_new}}) covers(c, p, n, rows);
                }
}

// the largest sizes that the checks let through
void extremes() {
  for (int32_t d : {64, 128, 256})
    for (int32_t batch : {1, 65535})
      for (int32_t kv : {1, 16384})
        for (int32_t group : {1, 16384})
          for (int32_t max_new : {1, 64, 1 << 20, 1 << 30})
            for (int32_t block : {0, 1, INT32_MAX})
              for (int32_t window : {0, 1, INT32_MAX}) {
                if (kv * int64_t{group} > 16384 || max_new * int64_t{group} > (int64_t{1} << 36)) continue;
                for (const int64_t total : {int64_t{max_new}, int64_t{1} << 30}) {
                  const Case c{batch, max_new, kv * group, kv, d, block, window, total, int64_t{1} << 30, true};
                  const orbq::AttnPlan p = plan_of(c);
                  EXPECT(p.splits >= 1 && p.chunk >= 1 && p.whole >= 0 && p.part_rows >= 0 && p.row_tiles >= 1);
                }
              }
  // row tiles that no launch can count are refused, with no workspace asked for
  const orbq_kv_cache c = cache(64, 64, 128);
  const orbq_page_table t{I, 1 << 24, 1 << 24, 65535};
  const auto call = [&](int32_t most) {
    return orbq_kv_attention(&c, &t, I, I, 1 << 30, most, 0, P, 64 * 128, 128, 64, P, 64 * 128, 128, nullptr, ORBQ_BF16, 0.1f, 0, 0, nullptr,
                             0, nullptr);
  };
  EXPECT(call(1 << 30) == ORBQ_ERR_UNSUPPORTED);
  EXPECT(call(1 << 18) == ORBQ_ERR_UNSUPPORTED);
  EXPECT(call(1 << 16) == ORBQ_OK);
}
}  // namespace

int main() {
  strides();
  plans();
  extremes();
  EXPECT(g_launches > 0);
  if (g_fail) {
    std::printf("%d of %d failed\n", g_fail, g_checks);
    return 1;
  }
  std::printf("ok %d\n", g_checks);
  return 0;
}

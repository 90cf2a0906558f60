// kv_attention: which form a call takes and how its keys are split.  Kernels: kv_attention_kernel.h.
#include <algorithm>

#include "attention.h"

namespace orbq {

template <> int launch_attn<64>(const AttnArgs&, const AttnPlan&, hipStream_t);
template <> int launch_attn<128>(const AttnArgs&, const AttnPlan&, hipStream_t);
template <> int launch_attn<256>(const AttnArgs&, const AttnPlan&, hipStream_t);

AttnPlan plan_attention(int32_t batch, int64_t total, int32_t max_new, int32_t heads, int32_t kv_heads, int32_t d, int64_t max_len,
                        int32_t causal_block, int32_t window, bool bound, int cus) {
  AttnPlan p{};
  const int64_t rows = static_cast<int64_t>(max_new) * (heads / kv_heads);
  // The few-row form reads the cache once for each of its row tiles.  For 17 to 32 rows two single tiles beat
  // one double one while the second reading finds the cache on the card, and lose beyond (32 rows, 8 heads of 128: 61 MB
  // of cache 29 us against 35, 102 MB 40 and 45, 123 MB 47 and 48, 150 MB 55 and 52, 268 MB 85 and 73; heads of 64, whose
  // tiles cost less, are even at 61 MB, and 123 MB takes 43 and 37).  Above 32 rows double tiles win (64 rows over
  // 60000 tokens: 53 against 55, heads of 64 31 against 35) and beat the many-row form up to 64 rows (82); with heads of
  // 256 a double tile's registers spill, and the many-row form takes over at 33 rows.
  const double cached = 2.0 * max_len * batch * kv_heads * d;
  p.many = rows > (d == 256 ? 32 : 64);
  p.rt = d < 256 && (rows > 32 || (rows > 16 && cached > 0x1p27)) ? 2 : 1;
  const int tile_rows = p.many ? many_rows(d) : 16 * p.rt;
  p.row_tiles = static_cast<int32_t>((rows + tile_rows - 1) / tile_rows);
  // the keys that the rows of one stream can see together, in 64-key tiles: under a window more than one row tile sees,
  // so that the splits of a windowed call are longer than they need be and the last ones have nothing
  int64_t span = max_len;
  if (window) span = std::min<int64_t>(span, static_cast<int64_t>(window) + max_new + causal_block);
  const int64_t tiles = std::max<int64_t>(1, (span + 63) / 64 + (window ? 1 : 0));
  const int64_t groups = static_cast<int64_t>(batch) * kv_heads * p.row_tiles;
  int64_t splits = 1, whole = groups, part_tiles = tiles;
  p.waves = 4;
  if (p.many && groups <= kMostTiles) {  // more of them are refused
    // Workgroups resident at once: one a CU (LDS and registers), three with heads of 64.  Row tiles that fill whole
    // rounds are not split, those of the last round are, so that it is full too (2 x 4605 queries of 8 heads of 256,
    // 576 row tiles: all in three parts 528 us, the last 64 in four 435).  Sequences of unequal rows leave row
    // tiles empty, so rounds are not told apart there (ragged prompts: 82 us without, 93 with).  In tiles of one
    // workgroup: the rounds of splits, the joining launch (3) and the parts' way through memory, which takes a
    // full card about as long as 400 keys of the same rows.
    const int64_t want = static_cast<int64_t>(cus) * (d == 64 ? 3 : 1);
    const int64_t full = total == static_cast<int64_t>(batch) * max_new ? groups / want * want : 0, rest = groups - full;
    // the last round's row tiles are a sequence's first rows, which see less under a causal mask
    if (full && causal_block) span = std::min(span, std::max<int64_t>(0, max_len - max_new) + max_new * rest / groups + causal_block);
    part_tiles = std::min(tiles, (span + 63) / 64 + 1);
    const int64_t before = full / want * tiles;
    double least = static_cast<double>(before + (rest + want - 1) / want * part_tiles);
    const auto consider = [&](int64_t n) {
      if (n < 2 || 2 * n > part_tiles) return;
      const double cost = static_cast<double>(before + (rest * n + want - 1) / want * ((part_tiles + n - 1) / n)) + 3.0 +
                          400.0 / 64 * n * rest / want;
      if (cost < least) {
        least = cost;
        splits = n;
        whole = full;
      }
    };
    if (rest) {
      for (int n = 2; n <= 16; ++n) consider(n);
      for (int n = 1; n <= 3; ++n) consider(n * want / rest);
    }
    // Turning the codes once a call instead of once a row tile pays where some eight row tiles read each of
    // them (4680 queries over 32760 tokens, 12 heads of 128: 1165 us without, 1005 with; 327 queries with a
    // window of 19: 28 without, 36 with); with heads of 64 staging is too small a share (ragged prompts: 83 either
    // way, 4 x 4000 causal queries of 16 heads 202 without, 208 with, with a window of 500 72 and 78).
    const int64_t tile_tokens = std::max<int64_t>(1, many_rows(d) / (heads / kv_heads));
    int64_t readers = p.row_tiles;
    if (window) readers = std::min<int64_t>(readers, (static_cast<int64_t>(window) + causal_block + 63) / tile_tokens + 1);
    if (bound && d > 64 && readers >= 8 && static_cast<int64_t>(batch) * kv_heads * tiles * d <= (int64_t{1} << 22))
      p.turned = static_cast<int32_t>(tiles);  // at most 1 GiB of workspace
  } else if (!p.many && p.rt == 1 && d <= 128 && (tiles * d <= 17 * 128 || (4 * groups >= 3 * cus && groups <= cus))) {
    // Eight waves and no join, where the keys are few or where one such workgroup a CU fills the card without a second
    // round.  12 streams of heads of 128: 500 tokens 9.2 us against 10.2 with four waves and split keys, 1088 (17 tiles)
    // 12.2 and 12.3, 1400 14.4 and 13.1; of heads of 64: 2000 10.3 and 11.4, 2176 10.6 and 9.0.
    // 12000 tokens of heads of 128: 96 streams 90 and 66, 192 107 and 126, 256 141 and 153, 264 207 and 169.
    p.waves = 8;
  } else if (!p.many) {
    // as many workgroups as are resident at once (two a CU), if that leaves few idle; else enough small
    // ones that the dispatcher evens them out
    const int64_t want = static_cast<int64_t>(cus) * 2, fit = want / groups;
    if (groups < 2 * want) splits = fit >= 4 ? fit : (2 * want + groups - 1) / groups;
    splits = std::min(splits, (tiles + 3) / 4);
  }
  p.chunk = static_cast<int32_t>((part_tiles + splits - 1) / splits);
  p.splits = static_cast<int32_t>((part_tiles + p.chunk - 1) / p.chunk);
  p.whole = static_cast<int32_t>(std::min<int64_t>(whole, kMostTiles));
  p.part_rows = p.many ? (groups - whole) * tile_rows : total * heads;
  return p;
}

int launch_kv_attention(AttnArgs a, const AttnPlan& p, hipStream_t stream) {
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.whole = p.whole;
  switch (a.c.d) {
    case 64: return launch_attn<64>(a, p, stream);
    case 128: return launch_attn<128>(a, p, stream);
    default: return launch_attn<256>(a, p, stream);
  }
}

}  // namespace orbq

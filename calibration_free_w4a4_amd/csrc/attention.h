// Internal declarations of the attention-side operators: rotary positions, the 8-bit paged
// key/value cache, attention over it.  Host layer in attention_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace orbq {

enum : int { kF32 = 0, kBF16 = 1, kF16 = 2 };  // orbq_dtype
inline int dtype_size(int t) { return t == kF32 ? 4 : 2; }

// ---------------------------------------------------------------------------- rotary positions
struct RopeTensor {
  const void* x;
  void* y;
  int32_t heads;
  int64_t xt, xh, yt, yh;  // token and head strides in elements
};

struct RopeArgs {
  RopeTensor t[2];
  const float* pos;    // [n_pos][axes]
  const float* freqs;  // [pairs]
  int64_t n, n_pos;
  int32_t axes, pairs, d, halves, inverse;
  int32_t ends[4];     // one past the last pair of each axis
};

int launch_rope(const RopeArgs& a, int dtype, hipStream_t stream);

// ------------------------------------------------------------------------------------ the cache
constexpr float kScaleFloor = 0x1p-64f;  // the least scale of a block
constexpr float kScaleMost = 0x1p+126f;  // and the largest that attention takes (its reciprocal is a normal number)
constexpr float kScaleGrow = 1.25f;      // a scale that has to grow grows at least by this factor

struct KvCache {
  int8_t* k;    // [pages][heads][page][d]
  int8_t* v;    // [pages][heads][d][page]
  float* ks;    // [pages][heads]
  float* vs;
  int32_t pages, heads, page, d;
  const int32_t* table;  // [batch][ldt], the first max_pages entries of a row used
  int64_t ldt;
  int32_t max_pages, batch;
};

struct KvTokens {         // the tokens of a call, packed: sequence b has rows cu[b] .. cu[b + 1] - 1
  const int32_t* cu;      // NULL: total / batch rows each
  const int32_t* first;   // position of a sequence's first row
  int64_t total;
  int32_t max_rows;       // no sequence has more
  void* k;
  void* v;
  int64_t kt, kh, vt, vh;  // strides in elements
};

int launch_kv_append(const KvCache& c, const KvTokens& x, int dtype, hipStream_t stream);
int launch_kv_read(const KvCache& c, const KvTokens& x, int dtype, hipStream_t stream);

// what kv_append_rope does to q and k on the way
struct TurnArgs {
  const float* pos;    // [n_pos][axes]
  const float* freqs;  // [pairs]
  int64_t n_pos;
  int32_t axes, pairs, halves, inverse;  // inverse: 0
  int32_t ends[4];
  const float* q_weight;  // [d] or NULL: no norm
  const float* k_weight;
  float eps;
  RopeTensor q;  // heads 0: none
};

int launch_kv_append_rope_f32(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream);
int launch_kv_append_rope_bf16(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream);
int launch_kv_append_rope_f16(const KvCache& c, const KvTokens& x, const TurnArgs& r, hipStream_t stream);

// ------------------------------------------------------------------------------------ attention
struct AttnArgs {
  KvCache c;
  int32_t page_shift;
  const int32_t* lens;
  const int32_t* cu;  // NULL: total / batch queries each
  int64_t total;
  int32_t max_new, heads, group;
  const void* q;
  void* o;
  int64_t qt, qh, ot, oh;  // strides in elements
  float* lse;              // [total][heads] or NULL
  float scale_log2e;       // |scale| log2(e)
  int32_t negative;        // scale < 0: q enters with its sign turned
  int32_t f16;             // q and o are f16 (else bf16)
  int32_t causal_block, window;
  // the launch
  int32_t row_tiles, splits, chunk;  // chunk: 64-key tiles of a split
  int32_t whole;                     // many: the first row tiles in turn, which are not split
  int32_t first;                     // many: the launch's first workgroup
  float* part_o;                     // [rows][splits][d], splits > 1; rows as AttnPlan::part_rows counts them
  float* part_ml;                    // [rows][splits][2]
  void* turned;                      // AttnPlan::turned: f16 tiles [batch][cache heads][turned_tiles][16 d][8]
  void* factors;                     // and their factors [batch][cache heads][turned_tiles][4][4] fp32
  int32_t turned_tiles;
};

constexpr int64_t kMostTiles = 0x7fffffff;  // row tiles of a call in the form for many rows

// rows of a workgroup in the form for many rows, 32 a wave
constexpr int many_rows(int d) { return d == 128 ? 256 : 128; }

struct AttnPlan {
  int32_t many;    // the form for many rows (else few)
  int32_t rt;      // few: 16-row tiles a workgroup
  int32_t waves;   // few: waves a workgroup
  int32_t row_tiles, splits, chunk;
  int32_t whole;   // many: this many row tiles of all streams, in the order of the launch, are not split
  int64_t part_rows;  // rows with parts.  many: those of the split row tiles in turn; few: all, [total][heads]
  int32_t turned;  // many: the tiles a stream's keys are turned into f16 before (0: on the way into LDS)
};

// bound: no sequence can be longer than max_len
AttnPlan plan_attention(int32_t batch, int64_t total, int32_t max_new, int32_t heads, int32_t kv_heads, int32_t d, int64_t max_len,
                        int32_t causal_block, int32_t window, bool bound, int cus);
int launch_kv_attention(AttnArgs a, const AttnPlan& p, hipStream_t stream);

// one instantiation unit per head dimension
template <int D> int launch_attn(const AttnArgs& a, const AttnPlan& p, hipStream_t stream);

}  // namespace orbq

// Internal declarations of block_norm: the norms before and after a block of a transformer, fused with the block's
// gate and the residual stream.  Host layer in block_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attention.h"  // kF32, kBF16, kF16

namespace orbq {

enum : int { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };  // orbq_norm_kind

struct NormArgs {
  int64_t n;
  int32_t d, groups;
  const int32_t* cu;   // [groups + 1] or NULL: n / groups rows each
  int32_t norm, post;  // kNorm*
  float eps, post_eps;
  const void* w;       // [d] or NULL
  const void* pw;
  int32_t wtype, mtype;
  const void* gate;    // [groups][..] or NULL; row stride 0: one for all groups
  const void* scale;
  const void* shift;
  int64_t gld, scld, shld;
  // forward: x, y -> r, h.  backward: x is r, with dr and dh -> dx, dy
  const void* x;
  const void* y;
  int64_t xld, yld;
  void* r;
  void* h;
  int64_t rld, hld;
  const void* dr;
  const void* dh;
  int64_t drld, dhld;
  void* dx;
  void* dy;
  int64_t dxld, dyld;
  // backward, the vectors' gradients: sums of a chunk of rows within a group, [chunks + groups - 1][3][d] fp32
  float* part;  // NULL: none asked for
  int32_t chunk_rows;
};

// What becomes of the sums; NULL where it is not asked for.  Row stride 0: summed over the groups.
struct NormGrads {
  void* gate;
  void* scale;
  void* shift;
  int64_t gld, scld, shld;
  void* w;
  void* pw;
};

// rows of a chunk, and with it the number of chunks, of a call of n rows
int32_t norm_chunk_rows(int64_t n, int32_t d, int cus);

// wide: every address and stride allows 16-byte columns of 8 entries
int launch_block_norm(const NormArgs& a, int stream_type, int branch_type, bool wide, hipStream_t stream);
int launch_block_norm_backward(const NormArgs& a, const NormGrads& g, int stream_type, int branch_type, bool wide, hipStream_t stream);

}  // namespace orbq

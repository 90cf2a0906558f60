// rope: rotary positions with several axes.  Pair i of a head's first 2 * pairs entries belongs to
// one axis (time, height, width, ...) and is turned by angle pos[token][axis] * freqs[i]:
//   (a, b) -> (a cos - b sin, a sin + b cos);
// the turn is orthogonal, so the gradient is the same with the angle's sign turned (inverse).
//
// Each element is read once and written once, so the call is bound by HBM bytes.  A thread owns
// one 16-byte column of a head row (two columns in the split-half order, whose pairs lie
// half a rotary width apart) for one token, finds the columns' sines and cosines once and goes over
// `per` heads with them, q's heads first, then k's.  32760 tokens, 12 + 12 heads of 128 in bf16: 84 us, 4.8 TB/s
// (a large copy on the same card: 4.7); 4605 tokens, 24 + 8 heads in f32: 26 us; one token: 3.5 us.
#include <algorithm>

#include "rope_device.h"

namespace orbq {
int device_cus();
namespace {

// a workgroup takes as many whole tokens as fit; the scalar form's up to 512 columns fit one token
template <int E> constexpr int kThreads = E == 1 ? 512 : 256;

// E: elements of a thread's column (16 bytes, or the scalar form: one pair a thread, for strides,
// addresses and widths that 16-byte columns do not fit)
template <int DT, int E, bool HALVES>
__global__ __launch_bounds__(kThreads<E>) void k_rope(const RopeArgs a, int cols, int tokens, int per) {
  const int slot = threadIdx.x / cols, col = threadIdx.x - slot * cols, group = blockIdx.y;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * tokens + slot;
  if (slot >= tokens || token >= a.n) return;
  constexpr int P = HALVES ? E : (E == 1 ? 1 : E / 2);  // pairs of a thread
  const float* pos = a.pos + (a.n_pos == a.n ? token : token % a.n_pos) * a.axes;
  const int pair0 = col * P;
  // columns behind the pairs hold the entries that pass through
  int off0, off1 = 0;
  bool turned;
  if constexpr (HALVES) {
    turned = pair0 < a.pairs;
    off0 = turned ? pair0 : a.pairs + pair0;
    off1 = a.pairs + pair0;
  } else {
    turned = pair0 < a.pairs;
    off0 = E == 1 ? (turned ? 2 * pair0 : a.pairs + pair0) : col * E;
    off1 = off0 + 1;
  }
  float s[P], c[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    s[i] = 0.0f;
    c[i] = 1.0f;
    if (turned && pair0 + i < a.pairs) pair_sincos(a, pos, pair0 + i, &s[i], &c[i]);
  }
  const int h0 = group * per, all = a.t[0].heads + a.t[1].heads;
  const int h1 = h0 + per < all ? h0 + per : all;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const RopeTensor& t = a.t[h >= a.t[0].heads ? 1 : 0];
    const int hh = h >= a.t[0].heads ? h - a.t[0].heads : h;
    const int64_t xb = token * t.xt + hh * t.xh, yb = token * t.yt + hh * t.yh;
    float u[E], w[E];
    Vec<DT, E>::load(t.x, xb + off0, u);
    if constexpr (HALVES || E == 1) {
      if (turned) {
        Vec<DT, E>::load(t.x, xb + off1, w);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float p = u[i], q = w[i];
          turn(p, q, s[i], c[i], &u[i], &w[i]);
        }
        Vec<DT, E>::store(t.y, yb + off1, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        if (pair0 + i < a.pairs) {
          const float p = u[2 * i], q = u[2 * i + 1];
          turn(p, q, s[i], c[i], &u[2 * i], &u[2 * i + 1]);
        }
      }
    }
    Vec<DT, E>::store(t.y, yb + off0, u);
  }
}

template <int DT, int E, bool HALVES> int launch(const RopeArgs& a, hipStream_t stream) {
  const int rest = a.d - 2 * a.pairs;
  int cols;
  if (E == 1) cols = a.pairs + rest;
  else if (HALVES) cols = a.pairs / E + rest / E;
  else cols = a.d / E;
  const int all = a.t[0].heads + a.t[1].heads;
  // heads a thread goes over: more heads share the sines, fewer fill the card.
  const int64_t threads = a.n * cols, fill = static_cast<int64_t>(device_cus()) * 2048;
  const int per = static_cast<int>(std::min<int64_t>(8, std::max<int64_t>(1, threads * all / fill)));
  const int groups = (all + per - 1) / per;
  const int tokens = kThreads<E> / cols;
  const int64_t blocks = (a.n + tokens - 1) / tokens;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_rope<DT, E, HALVES>), dim3(static_cast<uint32_t>(blocks), groups), dim3(kThreads<E>), 0, stream, a,
                     cols, tokens, per);
  return static_cast<int>(hipGetLastError());
}

template <int DT> int launch_dt(const RopeArgs& a, hipStream_t stream) {
  constexpr int E = DT == kF32 ? 4 : 8;
  bool wide = a.d % E == 0 && (!a.halves || a.pairs % E == 0);
  for (const RopeTensor& t : a.t) {
    if (!t.heads) continue;
    wide = wide && !((t.xt | t.xh | t.yt | t.yh) % E) &&
           !((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) % 16);
  }
  if (wide) return a.halves ? launch<DT, E, true>(a, stream) : launch<DT, E, false>(a, stream);
  return a.halves ? launch<DT, 1, true>(a, stream) : launch<DT, 1, false>(a, stream);
}

}  // namespace

int launch_rope(const RopeArgs& a, int dtype, hipStream_t stream) {
  switch (dtype) {
    case kF32: return launch_dt<kF32>(a, stream);
    case kBF16: return launch_dt<kBF16>(a, stream);
    default: return launch_dt<kF16>(a, stream);
  }
}

}  // namespace orbq

// rope.cuh — rotation of a head's elements by the token's position, shared by the operators that
// rotate (paged_ops.cu).
//
// A pair turns by position x turns / 2^64 revolutions (gqa_rope).  The product is taken modulo 2^64, that is,
// modulo one revolution, exactly, so the angle that is left has the frequency's own error times the
// position and no error of its size.  A frequency is a power and a few products in 64 bits, at most 1 radian per position:
// off by 2^-51 of a radian at most (4e-10 of one at a million positions).  Sine and cosine then take the nearest fp32 to
// the angle in half revolutions (2^-25 of half a revolution at most).
#pragma once

#include <cuda_bf16.h>

#include "params.h"
#include "ptx.cuh"

namespace gqa {

__device__ __forceinline__ float2 rope_cos_sin(const gqa_rope& r, int j, int pos) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * r.turns[j];
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(t >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * r.gain, s * r.gain);
}

// A head's 16 chunks of 8 elements are shared by 8 threads, two chunks each: with h = rot_dim / 16,
// threads 0 .. h - 1 have those that they rotate with one another (pairs 8 i .. 8 i + 7 of thread i), the
// others two that keep their values.
struct RopeLane {
  bool turns;
  int a, b;  // chunks
  __device__ __forceinline__ RopeLane(const gqa_rope& r, bool rotate, int i) {
    const int h = r.rot_dim >> 4;
    turns = rotate && i < h;
    a = 2 * i;
    b = 2 * i + 1;
    if (turns && r.layout == GQA_ROPE_HALVES) {
      a = i;
      b = i + h;
    }
    // (the chunks behind 2 h are those of threads h .. 7 in both layouts)
  }
};

// cos and sin of the eight pairs of threads i: kSubs threads with the same i, one for each of as many heads, lie
// eight lanes apart and compute 8 / kSubs pairs each.  Called by whole warps.
template <int kSubs>
__device__ __forceinline__ void rope_coefficients(const gqa_rope& r, int pos, float2 (&cs)[8]) {
  constexpr int kOwn = 8 / kSubs;
  const int i = threadIdx.x & 7, sub = (threadIdx.x >> 3) & (kSubs - 1);
  float2 own[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) own[j] = rope_cos_sin(r, 8 * i + sub * kOwn + j, pos);
  if constexpr (kSubs == 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = own[j];
    return;
  }
  // (lanes of this token begin at the last multiple of 8 kSubs)
  const int from = (threadIdx.x & 31 & ~(8 * kSubs - 1)) + i;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j].x = __shfl_sync(0xffffffffu, own[j % kOwn].x, from + 8 * (j / kOwn));
    cs[j].y = __shfl_sync(0xffffffffu, own[j % kOwn].y, from + 8 * (j / kOwn));
  }
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Rotates a turning thread's two chunks.
__device__ __forceinline__ void rope_turn(int layout, const float2 (&cs)[8], float (&a)[8], float (&b)[8]) {
  if (layout == GQA_ROPE_HALVES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * cs[j].x - y * cs[j].y;
      b[j] = x * cs[j].y + y * cs[j].x;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1], z = b[2 * j], w = b[2 * j + 1];
      a[2 * j] = x * cs[j].x - y * cs[j].y;
      a[2 * j + 1] = x * cs[j].y + y * cs[j].x;
      b[2 * j] = z * cs[4 + j].x - w * cs[4 + j].y;
      b[2 * j + 1] = z * cs[4 + j].y + w * cs[4 + j].x;
    }
  }
}

}  // namespace gqa

// Query, key and value vectors of one token from the fused QKVG projection,
// shared by the decode attentions.
#pragma once
#include "common.cuh"

namespace dory {

// One warp forms up to NW vectors v of (q_0 .. q_{G-1}, k, v) of KV head kvh
// (vs[j] < 0: none) from the split-K partials of the fused QKVG output: q and
// k get rotate-half RoPE (rope: [hd/2] cos, sin of this position), the L2
// norm over the head and the per-dim scale (q also q_scale); k and v are
// rounded to BF16, the precision the cache holds.  Every load of every
// vector is issued before the first use (one L2 round trip).
template <int HD, int G, int NW>
__device__ __forceinline__ void form_vectors(const DecAttnArgs& a,
                                             const float* src, size_t pstride,
                                             int kvh, const int (&vs)[NW],
                                             float* vec_s) {
  constexpr int HALF = HD / 2;
  constexpr int NPR = (HALF + 31) / 32;       // rotation pairs per lane
  const Dims& dm = a.dm;
  const int lane = threadIdx.x & 31;
  float x1[NW][NPR], x2[NW][NPR], cs[NPR], sn[NPR], sc1[NW][NPR], sc2[NW][NPR];
#pragma unroll
  for (int j = 0; j < NPR; ++j) {
    const int i = lane + 32 * j;
    cs[j] = i < HALF ? a.rope[2 * i] : 0.f;
    sn[j] = i < HALF ? a.rope[2 * i + 1] : 0.f;
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int v = vs[w];
    const bool is_q = v < G, is_v = v == G + 1;
    const float* scale = is_q ? a.s_q + (kvh * G + v) * HD : a.s_k + kvh * HD;
#pragma unroll
    for (int j = 0; j < NPR; ++j) {
      const int i = lane + 32 * j;
      const bool in = v >= 0 && i < HALF && !is_v;
      x1[w][j] = x2[w][j] = 0.f;
      sc1[w][j] = in ? scale[i] : 0.f;
      sc2[w][j] = in ? scale[i + HALF] : 0.f;
    }
  }
  for (int s = 0; s < a.S; ++s) {
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int v = vs[w];
      if (v < 0) continue;
      const bool is_q = v < G, is_v = v == G + 1;
      const int col0 = is_q ? (kvh * G + v) * HD
                     : !is_v ? dm.qdim + kvh * HD : dm.qdim + dm.kvdim + kvh * HD;
      const float* sp = src + s * pstride + col0;
#pragma unroll
      for (int j = 0; j < NPR; ++j) {
        const int i = lane + 32 * j;
        if (i < HALF) {
          x1[w][j] += sp[i];
          x2[w][j] += sp[i + HALF];
        }
      }
    }
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int v = vs[w];
    if (v < 0) continue;
    const bool is_q = v < G, is_v = v == G + 1;
    float* dst = vec_s + v * HD;
    if (is_v) {
#pragma unroll
      for (int j = 0; j < NPR; ++j) {
        const int i = lane + 32 * j;
        if (i < HALF) {
          dst[i] = __bfloat162float(__float2bfloat16_rn(x1[w][j]));
          dst[i + HALF] = __bfloat162float(__float2bfloat16_rn(x2[w][j]));
        }
      }
      continue;
    }
    float r1[NPR], r2[NPR], ss = 0.f;
#pragma unroll
    for (int j = 0; j < NPR; ++j) {
      r1[j] = x1[w][j] * cs[j] - x2[w][j] * sn[j];
      r2[j] = x2[w][j] * cs[j] + x1[w][j] * sn[j];
      ss += r1[j] * r1[j] + r2[j] * r2[j];
    }
    const float inv = 1.f / fmaxf(sqrtf(warp_sum(ss)), 1e-12f);
    const float extra = is_q ? a.q_scale : 1.f;
#pragma unroll
    for (int j = 0; j < NPR; ++j) {
      const int i = lane + 32 * j;
      if (i < HALF) {
        float u = r1[j] * inv * sc1[w][j] * extra;
        float z = r2[j] * inv * sc2[w][j] * extra;
        if (!is_q) {
          u = __bfloat162float(__float2bfloat16_rn(u));
          z = __bfloat162float(__float2bfloat16_rn(z));
        }
        dst[i] = u;
        dst[i + HALF] = z;
      }
    }
  }
}

}  // namespace dory

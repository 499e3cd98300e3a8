// Drawing tokens from logits rows: temperature, top-k, min-p and top-p from
// given uniforms.
//
// With m = max z and w_i = exp((z_i - m) / T), order the vocabulary by
// (z descending, index ascending).  Kept is the prefix of that order that
//   holds at most top_k tokens, holds only tokens with w >= min_p, and, of
//   those, is the shortest with mass >= top_p times their mass (never empty);
// the token is the first kept one in index order whose running mass exceeds
// u times the kept mass.  Weights and masses are f64: a draw is decided by
// which side of one of up to V borders u falls, and in f32 those borders are
// off by more than neighbouring u differ.
//
// One block per row; every cutoff is found by bisection over the
// order-preserving integer image of the logits.
#include "common.cuh"

namespace dory {

namespace {

constexpr int kSampThreads = 1024;

// Order-preserving image of a logit; NaN counts as -inf (never drawn), and
// -0 as +0 (equal logits tie whatever their sign bit).
__device__ __forceinline__ uint32_t logit_key(float z) {
  if (!(z > -INFINITY)) z = -INFINITY;
  const uint32_t u = __float_as_uint(z + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

template <typename V>
__device__ V block_total(V v, V* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
  for (int i = 0; i < kSampThreads / 32; ++i) t += red[i];
  return t;
}

__global__ void __launch_bounds__(kSampThreads) sample_kernel(SampleArgs a) {
  __shared__ double red[32], pre[32];
  __shared__ int ired[32], s_pick;
  __shared__ uint32_t s_max;
  const int b = blockIdx.x, t = threadIdx.x, lane = t & 31, w = t >> 5;
  pdl_wait();
  pdl_trigger();
  const float* z = a.logits + (size_t)b * a.ld;
  const int V = a.V;
  if (t == 0) { s_max = 0; s_pick = 0x7fffffff; }
  __syncthreads();
  uint32_t mk = 0;
  for (int i = t; i < V; i += kSampThreads) mk = max(mk, logit_key(z[i]));
  atomicMax(&s_max, mk);
  __syncthreads();
  mk = s_max;
  const float m = key_logit(mk);
  if (m == -INFINITY) {              // nothing may be drawn
    if (t == 0) {
      a.tokens[b] = -1;
      if (a.logprobs) a.logprobs[b] = -INFINITY;
    }
    return;
  }
  const float T = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !(T > 0.f);
  const double inv_t = greedy ? 1.0 : 1.0 / (double)T;
  auto weight = [&](uint32_t k) -> double {
    if (k == mk) return 1.0;
    const float v = key_logit(k);
    return v > -INFINITY ? exp(((double)v - (double)m) * inv_t) : 0.0;
  };
  int n = a.top_k ? a.top_k[b] : 0;
  if (n <= 0 || n > V) n = V;
  if (greedy) n = 1;
  float minp = a.min_p ? a.min_p[b] : 0.f, topp = a.top_p ? a.top_p[b] : 1.f;
  minp = minp > 0.f ? fminf(minp, 1.f) : 0.f;

  // kept: key > cut, or key == cut and among the first `ties` of those
  uint32_t cut = 0;
  int ties = V;
  if (n < V) {
    uint32_t lo = 0, hi = mk;        // largest cut with count(key >= cut) >= n
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      int c = 0;
      for (int i = t; i < V; i += kSampThreads) c += logit_key(z[i]) >= mid;
      if (block_total(c, ired) >= n) lo = mid; else hi = mid - 1;
    }
    cut = lo;
    int c = 0;
    for (int i = t; i < V; i += kSampThreads) c += logit_key(z[i]) > cut;
    ties = n - block_total(c, ired);
  }
  if (minp > 0.f) {
    uint32_t lo = cut, hi = mk;      // smallest cut with weight >= min_p
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (weight(mid) >= (double)minp) hi = mid; else lo = mid + 1;
    }
    if (lo > cut) { cut = lo; ties = V; }
  }
  auto mass_above = [&](uint32_t c) {
    double s = 0;
    for (int i = t; i < V; i += kSampThreads) {
      const uint32_t k = logit_key(z[i]);
      if (k > c) s += weight(k);
    }
    return block_total(s, red);
  };
  auto count_at = [&](uint32_t c) {
    int s = 0;
    for (int i = t; i < V; i += kSampThreads) s += logit_key(z[i]) == c;
    return block_total(s, ired);
  };
  ties = min(ties, count_at(cut));
  const double total = mass_above(cut) + ties * weight(cut);
  if (topp < 1.f) {
    const double want = fmax((double)topp, 0.0) * total;
    uint32_t lo = cut, hi = mk;      // largest cut whose prefix still holds `want`
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (mass_above(mid - 1) >= want) lo = mid; else hi = mid - 1;
    }
    if (lo > cut) { cut = lo; ties = count_at(cut); }
    const double base = mass_above(cut), wc = weight(cut);
    int r = 0;
    while (r < ties && (base + r * wc < want || (cut == mk && r == 0))) ++r;
    ties = r;
  }
  const double kept = mass_above(cut) + ties * weight(cut);
  const float uf = a.uniform[b];
  const double target = (uf > 0.f ? fmin((double)uf, 1.0) : 0.0) * kept;

  // running mass in index order, kSampThreads tokens at a time
  double run = 0;
  int seen = 0, last = -1;
  for (int i0 = 0; i0 < V; i0 += kSampThreads) {
    const int i = i0 + t;
    const uint32_t k = i < V ? logit_key(z[i]) : 0;
    const bool tie = i < V && k == cut;
    const unsigned bal = __ballot_sync(0xffffffffu, tie);
    __syncthreads();
    if (lane == 0) ired[w] = __popc(bal);
    __syncthreads();
    int before = seen + __popc(bal & ((1u << lane) - 1));
    for (int j = 0; j < 32; ++j) {
      if (j < w) before += ired[j];
      seen += ired[j];
    }
    const bool keep = i < V && (k > cut || (tie && before < ties));
    const double wt = keep ? weight(k) : 0.0;
    double inc = wt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) pre[w] = inc;
    __syncthreads();
    double base = run;
    for (int j = 0; j < 32; ++j) {
      if (j < w) base += pre[j];
      run += pre[j];
    }
    if (wt > 0.0) {
      last = i;
      if (base + inc > target) atomicMin(&s_pick, i);
    }
    __syncthreads();
    if (s_pick != 0x7fffffff) break;
  }
  // u = 1 (or rounding at the very top): the last kept token
  if (s_pick == 0x7fffffff) {
    __syncthreads();
    if (t == 0) ired[0] = -1;
    __syncthreads();
    if (last >= 0) atomicMax(&ired[0], last);
    __syncthreads();
    if (t == 0) s_pick = ired[0];
    __syncthreads();
  }
  if (t == 0) {
    const int i = s_pick;
    a.tokens[b] = i;
    if (a.logprobs) {
      const uint32_t k = logit_key(z[i]);
      const double x = k == mk ? 0.0 : ((double)key_logit(k) - (double)m) * inv_t;
      a.logprobs[b] = (float)(x - log(kept));
    }
  }
}

}  // namespace

void launch_sample(const SampleArgs& a, cudaStream_t st) {
  launch_k(sample_kernel, dim3(a.B), dim3(kSampThreads), 0, st, a);
}

}  // namespace dory

// Drawing tokens from logits rows: temperature, top-k, min-p and top-p from
// given uniforms.
//
// With m = max z and w_i = exp((z_i - m) / T), order the vocabulary by
// (z descending, index ascending).  Kept is the prefix of that order that
//   holds at most top_k tokens, holds only tokens with w >= min_p, and, of
//   those, is the shortest with mass >= top_p times their mass (never empty);
// the token is the first kept one in index order whose running mass exceeds
// u times the kept mass.  Weights and sums are f64: a draw is decided by
// which side of one of up to V borders u falls, and in f32 those borders are
// off by more than neighbouring u differ.  (top-p's cutoff compares sums of
// weights rounded to 2^-46 or so in 64-bit integers, whose order of addition
// is free.)
//
// One thread-block cluster per row, up to 16 blocks: each keeps a slice of
// the row in shared memory, read from HBM once, and the blocks exchange
// maxima, histograms, candidates and sums by writing them into each other's
// shared memory, one cluster barrier per exchange; every block then takes the
// same decision from the same values.  A cutoff (top-k by count, top-p by
// mass) is found by histograms of kNB linear bins over the range of the
// logits still in question, narrowed until the bin that holds it has at most
// kGC logits per block (or equal ones), which are then ranked exactly: two
// exchanges per level, one or two levels unless the logits are adversarial.
// Rows without cutoffs need one exchange.
#include "async_copy.cuh"
#include "common.cuh"

namespace dory {

namespace {

typedef unsigned long long u64;

constexpr int kSampThreads = 512, kSW = kSampThreads / 32;
constexpr int kMaxC = 16;            // blocks per row
constexpr int kNB = 128;             // bins of a histogram
constexpr int kGC = 64;              // candidates per block

// NaN counts as -inf (never drawn).
__device__ __forceinline__ float clean(float z) { return z > -INFINITY ? z + 0.f : -INFINITY; }
// Order-preserving integer image of a float that is not NaN.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t u = __float_as_uint(z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 2^(j/16), correctly rounded.
__constant__ double kExpTab[16] = {
    1.0, 0x1.0b5586cf9890fp+0, 0x1.172b83c7d517bp+0, 0x1.2387a6e756238p+0,
    0x1.306fe0a31b715p+0, 0x1.3dea64c123422p+0, 0x1.4bfdad5362a27p+0, 0x1.5ab07dd485429p+0,
    0x1.6a09e667f3bcdp+0, 0x1.7a11473eb0187p+0, 0x1.8ace5422aa0dbp+0, 0x1.9c49182a3f090p+0,
    0x1.ae89f995ad3adp+0, 0x1.c199bdd85529cp+0, 0x1.d5818dcfba487p+0, 0x1.ea4afa2a490dap+0};

// e^x for x <= 0, relative error below (8 + |x|) 2^-53: x = (16 n + j) ln2 / 16 + r,
// |r| <= ln2 / 32, e^x = 2^n 2^(j/16) (Taylor series of e^r to r^6, whose
// next term is below 2^-50).  0 below -700.  tab: 2^(j/16) in shared memory
// (16 doubles, one per bank pair).
__device__ __forceinline__ double exp_neg(double x, const double* tab) {
  constexpr double kMagic = 0x1.8p52;
  const double t = fma(x, 16.0 / 0.693147180559945309417, kMagic);
  const int k = __double2loint(t);
  const double r = fma(t - kMagic, -0.693147180559945309417 / 16.0, x);
  double p = fma(r, 1.0 / 720, 1.0 / 120);
  p = fma(p, r, 1.0 / 24);
  p = fma(p, r, 1.0 / 6);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  p *= tab[k & 15];
  const double v = __hiloint2double(__double2hiint(p) + ((k >> 4) << 20), __double2loint(p));
  return x > -700.0 ? v : 0.0;
}

template <typename T>
__device__ __forceinline__ T wsum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- stores into the shared memory of another block of the cluster --------
__device__ __forceinline__ void put32(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put64(const void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(p, rank)), "l"(v) : "memory");
}

struct Cand {
  float z;
  int i;
  u64 w;
};

// What the blocks of a row write into each other (index: writer).  A buffer
// is written again only after a barrier that follows its last read.
struct Exchange {
  float max[kMaxC], min[kMaxC];
  int arg[kMaxC];
  uint32_t cnt[kMaxC][kNB];
  u64 mass[kMaxC][kNB];
  int g_n[kMaxC];
  float g_min[kMaxC], g_max[kMaxC];
  Cand g[kMaxC][kGC];
  int tie;
  double sum[kMaxC];
};

struct Local {
  Exchange ex;
  double tab[16];
  uint32_t cnt[kNB];
  u64 mass[kNB];
  Cand cand[kGC];
  int n;
  uint32_t kmin, kmax;
  // the chosen bin, and count and mass of what lies above it
  int bin, above;
  u64 mass_above, want;
  float cut_z;
  int cut_i;
  float fred[kSW], fred2[kSW];
  int ired[kSW];
  double dred[kSW];
  int pick;
};

__global__ void __launch_bounds__(kSampThreads, 2) sample_kernel(SampleArgs a, int C, int pw) {
  extern __shared__ __align__(16) uint8_t smraw[];
  Local& s = *reinterpret_cast<Local*>(smraw);
  float* zs = reinterpret_cast<float*>(smraw + sizeof(Local));
  const int row = blockIdx.x / C, rank = blockIdx.x - row * C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = kSW * pw, base = rank * per;      // this block's slice
  const int wbase = w * pw + lane;                  // this thread's first index in it
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (tid < 16) s.tab[tid] = kExpTab[tid];
  pdl_wait();
  pdl_trigger();
  const float* z = a.logits + (size_t)row * a.ld;
  const float T = a.temperature ? a.temperature[row] : 1.f;
  const bool greedy = !(T > 0.f);
  int k = a.top_k ? a.top_k[row] : 0;
  if (k <= 0 || k > a.V) k = a.V;
  float minp = a.min_p ? a.min_p[row] : 0.f, topp = a.top_p ? a.top_p[row] : 1.f;
  minp = minp > 0.f ? fminf(minp, 1.f) : 0.f;
  const float uf = a.uniform[row];

  // ---- the slice, its largest (and where) and smallest finite logit --------
  float zmax = -INFINITY, zmin = INFINITY;
  int amax = 0x7fffffff;
#pragma unroll 8
  for (int i = wbase; i < w * pw + pw; i += 32) {
    const int gi = base + i;
    const float v = gi < a.V ? clean(z[gi]) : -INFINITY;
    zs[i] = v;
    if (v > zmax) { zmax = v; amax = gi; }
    if (v > -INFINITY) zmin = fminf(zmin, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, zmax, o);
    const int i = __shfl_xor_sync(0xffffffffu, amax, o);
    if (v > zmax || (v == zmax && i < amax)) { zmax = v; amax = i; }
    zmin = fminf(zmin, __shfl_xor_sync(0xffffffffu, zmin, o));
  }
  if (lane == 0) { s.fred[w] = zmax; s.fred2[w] = zmin; s.ired[w] = amax; }
  __syncthreads();
  // every block has started: its shared memory may be written
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < C) {
#pragma unroll
    for (int j = 0; j < kSW; ++j) {
      const float v = s.fred[j];
      if (j == 0 || v > zmax || (v == zmax && s.ired[j] < amax)) { zmax = v; amax = s.ired[j]; }
      zmin = j ? fminf(zmin, s.fred2[j]) : s.fred2[0];
    }
    put32(&s.ex.max[rank], tid, __float_as_uint(zmax));
    put32(&s.ex.min[rank], tid, __float_as_uint(zmin));
    put32(&s.ex.arg[rank], tid, amax);
  }
  cluster_sync_all();
  float m = -INFINITY, lo = INFINITY;
  int arg = 0x7fffffff;
  for (int c = 0; c < C; ++c) {
    if (s.ex.max[c] > m) { m = s.ex.max[c]; arg = s.ex.arg[c]; }
    lo = fminf(lo, s.ex.min[c]);
  }
  if (m == INFINITY) lo = m;         // only these weigh anything
  if (m == -INFINITY || greedy) {    // nothing to draw, or nothing to draw for
    if (rank == 0 && tid == 0) {
      a.tokens[row] = m == -INFINITY ? -1 : arg;
      if (a.logprobs) a.logprobs[row] = m == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }
  const double inv_t = 1.0 / (double)T, md = (double)m;
  auto weight = [&](float v) -> double {
    const double x = ((double)v - md) * inv_t;
    return v == m ? 1.0 : exp_neg(x, s.tab);
  };
  // weights as integers: V of them add up to less than 2^63
  const double unit = (double)(1ull << (62 - (32 - __clz(a.V))));
  auto fixed = [&](float v) -> u64 { return __double2ull_rn(weight(v) * unit); };

  // kept: z > cz, or z == cz and index <= ci
  float cz = -INFINITY;
  int ci = -1;
  if (minp > 0.f) {
    // least logit with weight >= min_p: 32-way search of the integer images
    uint32_t l = key_of(lo), h = key_of(m);
    while (l < h) {
      const uint32_t step = (h - l) / 32 + 1;
      const uint32_t p = l + min(h - l, step * lane);
      const unsigned ok = __ballot_sync(0xffffffffu, weight(key_float(p)) >= (double)minp);
      const int f = ok ? __ffs(ok) - 1 : 32;          // lanes f.. hold
      if (f == 0) { h = l; break; }
      const uint32_t nl = l + min(h - l, step * (f - 1)) + 1;
      if (f < 32) h = l + min(h - l, step * f);
      l = nl;
    }
    cz = key_float(h);
    ci = 0x7fffffff;
    lo = fmaxf(lo, cz);
  }

  // ---- one cutoff: by count (top-k) or by mass (top-p) ----------------------
  auto select = [&](const bool by_mass) {
    float hi = m, low = lo;
    int above = 0;
    u64 mass_above = 0, want = 0;
    for (int level = 0;; ++level) {
      // histogram of the kept logits in [low, hi]; equal ones need none
      const bool flat = low == hi;
      const double sc = flat ? 0.0 : (double)kNB / ((double)hi - (double)low);
      auto bin_of = [&](float v) {
        return flat ? 0 : min((int)(((double)hi - (double)v) * sc), kNB - 1);
      };
      auto in_range = [&](float v, int i) {
        return v <= hi && v >= low && (v > cz || (v == cz && base + i <= ci));
      };
      __syncthreads();
      for (int i = tid; i < kNB; i += kSampThreads) { s.cnt[i] = 0; s.mass[i] = 0; }
      if (tid == 0) { s.n = 0; s.kmin = 0xffffffffu; s.kmax = 0; }
      __syncthreads();
      for (int i = wbase; i < w * pw + pw; i += 32) {
        const float v = zs[i];
        if (v > -INFINITY && in_range(v, i)) {
          const int bn = bin_of(v);
          atomicAdd(&s.cnt[bn], 1u);
          if (by_mass) {
            const u64 f = fixed(v);
            if (f) atomicAdd(&s.mass[bn], f);
          }
        }
      }
      __syncthreads();
      for (int i = tid; i < C * kNB; i += kSampThreads) {
        const int c = i / kNB, bn = i - c * kNB;
        put32(&s.ex.cnt[rank][bn], c, s.cnt[bn]);
        if (by_mass) put64(&s.ex.mass[rank][bn], c, s.mass[bn]);
      }
      cluster_sync_all();
      if (tid < kNB) {
        uint32_t n = 0;
        u64 f = 0;
        for (int c = 0; c < C; ++c) {
          n += s.ex.cnt[c][tid];
          if (by_mass) f += s.ex.mass[c][tid];
        }
        s.cnt[tid] = n;
        s.mass[tid] = f;
      }
      __syncthreads();
      if (w == 0) {
        // lane l holds bins 4l .. 4l + 3
        constexpr int Q = kNB / 32;
        int n = 0;
        u64 f = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) { n += s.cnt[Q * lane + q]; f += s.mass[Q * lane + q]; }
        int ni = n;
        u64 fi = f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, ni, o);
          const u64 x = __shfl_up_sync(0xffffffffu, fi, o);
          if (lane >= o) { ni += y; fi += x; }
        }
        if (by_mass && level == 0)
          want = max((u64)1, (u64)ceil(fmax((double)topp, 0.0) *
                                       (double)__shfl_sync(0xffffffffu, fi, 31)));
        int an = above + ni - n;
        u64 af = mass_above + fi - f;
        const bool hit = by_mass ? mass_above + fi >= want : above + ni >= k;
        const unsigned bal = __ballot_sync(0xffffffffu, hit);
        if (lane == (bal ? __ffs(bal) - 1 : 31)) {
          int bn = -1;
          if (bal) {
            for (bn = Q * lane; bn < Q * lane + Q - 1; ++bn) {
              if (by_mass ? af + s.mass[bn] >= want : an + (int)s.cnt[bn] >= k) break;
              an += s.cnt[bn];
              af += s.mass[bn];
            }
          }
          s.bin = bn;                   // -1: fewer than k are kept
          s.above = an;
          s.mass_above = af;
          s.want = want;
        }
      }
      __syncthreads();
      const int bin = s.bin;
      if (bin < 0) {
        cluster_sync_all();             // the histograms have been read
        return;
      }
      above = s.above;
      mass_above = s.mass_above;
      want = s.want;
      // the bin's logits
      uint32_t kmin = 0xffffffffu, kmax = 0;
      for (int i = wbase; i < w * pw + pw; i += 32) {
        const float v = zs[i];
        if (v > -INFINITY && in_range(v, i) && bin_of(v) == bin) {
          const int at = atomicAdd(&s.n, 1);
          if (at < kGC) s.cand[at] = Cand{v, base + i, by_mass ? fixed(v) : 0};
          kmin = min(kmin, key_of(v));
          kmax = max(kmax, key_of(v));
        }
      }
      kmin = __reduce_min_sync(0xffffffffu, kmin);
      kmax = __reduce_max_sync(0xffffffffu, kmax);
      if (lane == 0) { atomicMin(&s.kmin, kmin); atomicMax(&s.kmax, kmax); }
      __syncthreads();
      const int own = s.n;
      if (tid < C) {
        put32(&s.ex.g_n[rank], tid, own);
        put32(&s.ex.g_min[rank], tid, __float_as_uint(own ? key_float(s.kmin) : INFINITY));
        put32(&s.ex.g_max[rank], tid, __float_as_uint(own ? key_float(s.kmax) : -INFINITY));
      }
      const int send = min(own, kGC);
      for (int i = tid; i < C * send; i += kSampThreads) {
        const int c = i / send, j = i - c * send;
        put32(&s.ex.g[rank][j].z, c, __float_as_uint(s.cand[j].z));
        put32(&s.ex.g[rank][j].i, c, s.cand[j].i);
        put64(&s.ex.g[rank][j].w, c, s.cand[j].w);
      }
      cluster_sync_all();
      bool fits = true;
      int total = 0;
      low = INFINITY;
      hi = -INFINITY;
      for (int c = 0; c < C; ++c) {
        fits &= s.ex.g_n[c] <= kGC;
        total += s.ex.g_n[c];
        low = fminf(low, s.ex.g_min[c]);
        hi = fmaxf(hi, s.ex.g_max[c]);
      }
      if (fits) {
        // rank each candidate; the cutoff is the last one kept
        for (int e = tid; e < total; e += kSampThreads) {
          int c = 0, j = e;
          while (j >= s.ex.g_n[c]) j -= s.ex.g_n[c++];
          const Cand me = s.ex.g[c][j];
          int r = above;
          u64 f = mass_above;
          for (int c2 = 0; c2 < C; ++c2)
            for (int q = 0; q < s.ex.g_n[c2]; ++q) {
              const Cand& o = s.ex.g[c2][q];
              if (o.z > me.z || (o.z == me.z && o.i < me.i)) { ++r; f += o.w; }
            }
          if (by_mass ? f < want && f + me.w >= want : r == k - 1) {
            s.cut_z = me.z;
            s.cut_i = me.i;
          }
        }
        __syncthreads();
        cz = s.cut_z;
        ci = s.cut_i;
        return;
      }
      if (low == hi) {
        // equal logits: the r-th of them in index order
        u64 r = by_mass ? (want - mass_above - 1) / fixed(low) + 1 : (u64)(k - above);
        r = min(r, (u64)total);
        int c = 0;
        while ((u64)s.ex.g_n[c] < r) r -= s.ex.g_n[c++];
        if (rank == c) {
          int n = 0;
          for (int i = wbase; i < w * pw + pw; i += 32)
            n += __popc(__ballot_sync(0xffffffffu, zs[i] == low && in_range(zs[i], i)));
          if (lane == 0) s.ired[w] = n;
          __syncthreads();
          int before = 0;
          for (int j = 0; j < w; ++j) before += s.ired[j];
          if ((int)r > before && (int)r <= before + n) {
            for (int i = wbase; i < w * pw + pw; i += 32) {
              const bool t = zs[i] == low && in_range(zs[i], i);
              const unsigned bal = __ballot_sync(0xffffffffu, t);
              if (t && before + __popc(bal & ((2u << lane) - 1)) == (int)r)
                for (int q = 0; q < C; ++q) put32(&s.ex.tie, q, base + i);
              before += __popc(bal);
            }
          }
        }
        cluster_sync_all();
        cz = low;
        ci = s.ex.tie;
        return;
      }
    }
  };
  if (k < a.V) {
    select(false);
    lo = fmaxf(lo, cz);
  }
  if (topp < 1.f) select(true);

  // ---- the draw ---------------------------------------------------------------
  auto kept_weight = [&](int i) -> double {
    const float v = zs[i];
    return v > cz || (v == cz && base + i <= ci) ? weight(v) : 0.0;
  };
  double sum = 0.0;
#pragma unroll 4
  for (int i = wbase; i < w * pw + pw; i += 32) sum += kept_weight(i);
  sum = wsum(sum);
  if (lane == 0) s.dred[w] = sum;
  if (tid == 0) s.pick = -1;
  __syncthreads();
  if (tid < C) {
    double t = 0.0;
#pragma unroll
    for (int j = 0; j < kSW; ++j) t += s.dred[j];
    put64(&s.ex.sum[rank], tid, __double_as_longlong(t));
  }
  cluster_sync_all();
  double total = 0.0;
  for (int c = 0; c < C; ++c) total += s.ex.sum[c];
  const double target = (uf > 0.f ? fmin((double)uf, 1.0) : 0.0) * total;
  // the block and the warp whose share of the running mass holds the target;
  // past the end (u = 1): the last with any mass
  double run = 0.0, start = 0.0;
  int at = -1;
  for (int c = 0; c < C && (at < 0 || run <= target); ++c)
    if (s.ex.sum[c] > 0.0) {
      at = c;
      start = run;
      run += s.ex.sum[c];
    }
  if (rank != at) return;
  run = start;
  at = -1;
  for (int j = 0; j < kSW && (at < 0 || run <= target); ++j)
    if (s.dred[j] > 0.0) {
      at = j;
      start = run;
      run += s.dred[j];
    }
  if (w != at) return;
  run = start;
  int token = -1, last = -1;
  for (int i = wbase; i < w * pw + pw; i += 32) {
    const double x = kept_weight(i);
    double inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned any = __ballot_sync(0xffffffffu, x > 0.0);
    const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && run + inc > target);
    if (any) last = i - lane + 31 - __clz(any);
    if (hit) {
      token = i - lane + __ffs(hit) - 1;
      break;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (token < 0) token = last;
  if (lane == 0) {
    a.tokens[row] = base + token;
    if (a.logprobs) {
      const float v = zs[token];
      const double x = v == m ? 0.0 : ((double)v - md) * inv_t;
      a.logprobs[row] = (float)(x - log(total));
    }
  }
}

// ---- rows of any length ------------------------------------------------------
// One block per row, every cutoff by bisection over the integer images of the
// logits, which it reads again each time: rows that do not fit the shared
// memory of a cluster (more than 16 kFit).
constexpr int kAnyThreads = 1024;

__device__ __forceinline__ uint32_t any_key(float z) { return key_of(clean(z)); }

template <typename V>
__device__ V block_total(V v, V* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
  for (int i = 0; i < kAnyThreads / 32; ++i) t += red[i];
  return t;
}

__global__ void __launch_bounds__(kAnyThreads) sample_any_kernel(SampleArgs a) {
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
  for (int i = t; i < V; i += kAnyThreads) mk = max(mk, any_key(z[i]));
  atomicMax(&s_max, mk);
  __syncthreads();
  mk = s_max;
  const float m = key_float(mk);
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
    const float v = key_float(k);
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
      for (int i = t; i < V; i += kAnyThreads) c += any_key(z[i]) >= mid;
      if (block_total(c, ired) >= n) lo = mid; else hi = mid - 1;
    }
    cut = lo;
    int c = 0;
    for (int i = t; i < V; i += kAnyThreads) c += any_key(z[i]) > cut;
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
    for (int i = t; i < V; i += kAnyThreads) {
      const uint32_t k = any_key(z[i]);
      if (k > c) s += weight(k);
    }
    return block_total(s, red);
  };
  auto count_at = [&](uint32_t c) {
    int s = 0;
    for (int i = t; i < V; i += kAnyThreads) s += any_key(z[i]) == c;
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

  // running mass in index order, kAnyThreads tokens at a time
  double run = 0;
  int seen = 0, last = -1;
  for (int i0 = 0; i0 < V; i0 += kAnyThreads) {
    const int i = i0 + t;
    const uint32_t k = i < V ? any_key(z[i]) : 0;
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
      const uint32_t k = any_key(z[i]);
      const double x = k == mk ? 0.0 : ((double)key_float(k) - (double)m) * inv_t;
      a.logprobs[b] = (float)(x - log(kept));
    }
  }
}

// Slices of up to 16384 logits: shared memory that every GPC can give a
// 16-block cluster.
constexpr int kFit = 16384;
constexpr size_t kMaxSmem = sizeof(Local) + kFit * 4;

// Blocks per row: slices of up to 8192 logits, at most 16 blocks (8 where a
// 16-block cluster, a non-portable size, cannot be scheduled).
int max_cluster() {
  constexpr int kMax = 64;
  static int n[kMax];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMax) return 8;
  if (n[dev]) return n[dev];
  auto k = sample_kernel;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) !=
      cudaSuccess)
    return 8;
  int c = 8, fit = 0;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxC, 1, 1);
    cfg.blockDim = dim3(kSampThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxC;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&fit, k, &cfg) == cudaSuccess && fit >= 1) c = kMaxC;
  }
  cudaGetLastError();
  return n[dev] = c;
}

}  // namespace

void launch_sample(const SampleArgs& a, cudaStream_t st) {
  const int most = max_cluster();
  int C = 1;
  while (C < most && (int64_t)C * 8192 < a.V) C *= 2;
  if ((int64_t)C * kFit < a.V || (int64_t)C * a.B > 0x7fffffff) {
    launch_k(sample_any_kernel, dim3(a.B), dim3(kAnyThreads), 0, st, a);
    return;
  }
  const int pw = ((a.V + C * kSampThreads - 1) / (C * kSampThreads)) * 32;
  launch_k_cluster(sample_kernel, dim3(C * a.B), dim3(kSampThreads),
                   sizeof(Local) + (size_t)kSW * pw * 4, st, C, a, C, pw);
}

}  // namespace dory

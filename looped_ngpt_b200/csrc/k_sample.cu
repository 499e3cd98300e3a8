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
// off by more than neighbouring u differ.  (top-p's cutoff, and
// the mass that it keeps, are sums of weights rounded to 2^-43 in 64-bit
// integers, whose order of addition is free.)
//
// One thread-block cluster per row, up to 16 blocks: each keeps a slice of
// the row in shared memory, read from HBM once, and the blocks exchange
// maxima, histograms, candidates and sums by writing them into each other's
// shared memory, one cluster barrier per exchange; every block then takes the
// same decision from the same values.  A cutoff (top-k by count, top-p by
// mass) is found by histograms of kNB linear bins over the range of the
// logits still in question, narrowed until the bin that holds it has at most
// kRank logits (or equal ones), which are then ranked exactly: two exchanges
// per level, one or two levels unless the logits are adversarial.  The warps'
// shares of what a top-p keeps come from the same histograms.  A top-k that
// leaves up to kRank logits is finished from one list of them.  Rows without
// cutoffs need one exchange and no copy in shared memory.
//
// Reading 64 x 131072 logits takes 5.1 us at the copy rate.  The kernel takes
// 23 us without cutoffs, 45 us with top-p 0.9 and 34 us with top-k 50 and
// top-p 0.95 (12 us for one such row, 5.9 us for one without), where the largest
// logits lie apart.  Where over 32 of the top 50 lie in one block's slice (logits
// falling by index) the list does not hold them and top-p is looked for like any
// other: 58 us (21 for one row); rows masked with a large finite number need one
// level more (71 and 22 us; with -inf none).
//
// 64 rows are two waves of eight-block clusters (64 KB of logits and 45 KB of
// exchange per block, two blocks per SM).  Without cutoffs half of a wave's 10 us are the weights (44
// instructions per logit, of them 8 f64, which run at 60 lanes per clock and
// SM), the rest the launch, the first loads, one exchange and the draw.  With a
// top-p (95 instructions) a third is the first histogram, where shared memory
// is the limit (two atomics per logit at 13 lanes per clock, less what
// conflicts cost), and two thirds a chain of steps that each take 0.3 to 1.5
// us, six of them exchanges of 0.7 us.  Much of the code runs once, as fast as
// it can be fetched, so short loops are kept as loops where that is shorter
// (unrolled by the compiler's choice: 13.2 for 12.2 us with one row of top-k
// 50, 47 for 45 with 64 of top-p 0.9).
//
// Measured and not kept: 16-block clusters of 8192 logits for many rows (40 /
// 95 us where 8-block ones took 28.5 / 58), 256 threads with 128 registers (30
// / 60 against the same), one copy of the cutoff code for both kinds (29 / 55
// against 28 / 51), the bin and the blocks' shares found by every warp, and
// candidates sent by those that find them (three barriers and one exchange
// less: 48 against 47), one histogram of 16 columns for all warps (fewer bank
// conflicts, but warps meet in the same words: 49 against 47).
#include "async_copy.cuh"
#include "common.cuh"

#include <cfloat>

namespace dory {

namespace {

typedef unsigned long long u64;

constexpr int kSampThreads = 512, kSW = kSampThreads / 32;
constexpr int kMaxC = 16;            // blocks per row
constexpr int kNB = 128;             // bins of a histogram
constexpr int kRank = 128;           // candidates ranked by comparing each pair
constexpr int kU = 4;                // logits a thread handles at once

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

// 2^(y/16) for -1100 < y <= 0 (1 at 0) as p s, relative error below 2^-36.9: y
// = 16 n + j + f, |f| <= 1/2, with s = 2^n 2^(j/16) and p the polynomial of
// degree 4 through 1 at 0 whose largest relative error over |f| <= 1/2 is least
// (2^-38.5; fitted by reweighted least squares).  y is rounded to 2^-32 (2^-37.5
// of the weight) by adding 1.5 2^20 + 1/2, which leaves 16 n + j in the upper
// word and f + 1/2 in the lower.  tab: 2^(j/16), its upper word less j << 16,
// in shared memory (16 doubles, one per bank pair).  Errors of 2^-36.9 in the
// weights move the borders of a row's running sum so little that a uniform falls
// between with a chance below 1e-6 at V = 131072, while sampling is bound by
// the instructions of these lines.
constexpr double kExpBias = 0x1.8p20 + 0.5;
struct Pow2 {
  double p, s;
};
__device__ __forceinline__ Pow2 exp2_16th(double biased, const double* tab) {   // of y + kExpBias
  const int hi = __double2hiint(biased);
  const double f = __hiloint2double(0x43300000, __double2loint(biased)) - (0x1p52 + 0x1p31);
  double p = fma(f, 0x1.3b29bf8ba0f3ap-23 * 0x1p-128, 0x1.c6b3f5b3946b2p-17 * 0x1p-96);
  p = fma(p, f, 0x1.ebfbdfff31574p-11 * 0x1p-64);
  p = fma(p, f, 0x1.62e42fec3f16fp-5 * 0x1p-32);
  p = fma(p, f, 1.0);
  const double t = tab[hi & 15];
  return {p, __hiloint2double(__double2hiint(t) + (hi << 16), __double2loint(t))};
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

__device__ __forceinline__ double target_of(float u, double total) {
  return (u > 0.f ? fmin((double)u, 1.0) : 0.0) * total;
}

// Which part of a sequence of shares holds the target: lane i has share x (0:
// none); *start: what lies before it.  Past the end (u = 1): the last with any
// mass.
__device__ __forceinline__ int holder(double x, double from, double target, double* start) {
  const int lane = threadIdx.x & 31;
  double inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  const unsigned any = __ballot_sync(0xffffffffu, x > 0.0);
  const unsigned hit = __ballot_sync(0xffffffffu, x > 0.0 && from + inc > target);
  const int at = hit ? __ffs(hit) - 1 : 31 - __clz(any);
  const double before = __shfl_up_sync(0xffffffffu, inc, 1);
  *start = from + __shfl_sync(0xffffffffu, lane == 0 ? 0.0 : before, at);
  return at;
}

// Shared memory of a block.  `Fixed`, then, with C blocks per row and slices
// of `per` logits:
//   mass  u64 [C][kNB]     histograms, written by the row's blocks (index:
//                          writer), as everything in `Fixed::ex`
//   cands Cand [C][gc]     candidates, written likewise
//   hist  u32 [kSW][2][kNB] histograms of the warps' parts of the slice:
//                          counts, or (by mass) the low 22 and the upper bits
//                          of the weights, whose sums over up to 1024 logits
//                          stay below 2^32 (64-bit atomics on shared memory
//                          ran 17 times slower); then the own candidates
//   zs    f32 [per + 4]    the slice, shifted so that 16-byte chunks of the row
//                          stay 16-byte aligned
//   bins  u32 [][threads]  bins of each thread's logits in the first histogram,
//                          four to a word; later all kept logits, Cand [C][gc],
//                          written by the row's blocks, where there are few
// A buffer that other blocks write is written again only after a barrier that
// follows its last read.
struct Fixed {
  struct {
    uint32_t max[kMaxC], min[kMaxC];   // integer images
    int g_n[kMaxC];
    uint32_t g_min[kMaxC], g_max[kMaxC];
    int l_n[kMaxC];
    int tie;
    double sum[kMaxC];
  } ex;
  double tab[16];
  u64 bin_mass[kNB];
  // the chosen bin, and count and mass of what lies above it
  u64 mass_above, want;
  int bin, n;
  uint32_t kmin, kmax;
  float cut_z;
  int cut_i;
  uint32_t ured[2][kSW];
  int ired[kSW];
  double dred[kSW];
};
constexpr int kHistWords = kSW * 2 * kNB;
static_assert(sizeof(Fixed) % 16 == 0, "what follows is 16-byte aligned");

// Candidates per block: few blocks may send more each.
__host__ __device__ inline int cand_cap(int C) { return C >= 4 ? 32 : kRank / C; }
__host__ __device__ inline size_t bins_bytes(int C, int per) {
  const size_t bins = (size_t)(per / kSampThreads + 3) / 4 * kSampThreads * 4;
  const size_t list = (size_t)C * cand_cap(C) * sizeof(Cand);
  return bins > list ? bins : list;
}
__host__ __device__ inline size_t sample_smem(int C, int per) {
  return sizeof(Fixed) + (size_t)C * kNB * 8 + (size_t)C * cand_cap(C) * sizeof(Cand) +
         kHistWords * 4 + (size_t)(per + 4) * 4 + bins_bytes(C, per);
}
static_assert(kRank * (2 * sizeof(Cand) + 8) <= kHistWords * 4, "lists fit the histograms' place");

// The logit at which the running mass of a part of n <= N kSampThreads logits,
// of which one at least is kept, passes the target (`start`: the mass before the
// part): N neighbours per thread of the block; get(j), kept(v, j), weight(v);
// one thread calls found(j, v).  m is any logit with a weight.
template <int N, typename Get, typename Kept, typename Weight, typename Found>
__device__ __forceinline__ void draw_in_part(Fixed& s, int n, double start, double target, Get get,
                                             Kept kept, Weight weight, float m, Found found) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  double x[N], sum = 0.0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int j = min(N * tid + u, n - 1);
    const float v = get(j);
    const bool in = N * tid + u < n && kept(v, j);
    const double y = weight(in ? v : m);
    x[u] = in ? y : 0.0;
    sum += x[u];
  }
  const double mine = wsum(sum);
  __syncthreads();                                  // dred has been read
  if (lane == 0) s.dred[w] = mine;
  __syncthreads();
  if (holder(lane < kSW ? s.dred[lane] : 0.0, start, target, &start) != w) return;
  if (holder(sum, start, target, &start) != lane) return;
  int pick = -1;
#pragma unroll
  for (int u = 0; u < N; ++u)
    if (x[u] > 0.0 && (pick < 0 || !(start > target))) {
      pick = N * tid + u;
      start += x[u];
    }
  found(pick, get(pick));
}

// ---- rows without cutoffs ---------------------------------------------------
// One pass over the row in registers: each thread sums weights relative to the
// largest of its logits so far; threads, warps and blocks are brought to the
// row's largest when they are joined.  The part of one warp, which holds the
// draw, is read again.
__device__ __forceinline__ void draw_whole(const SampleArgs& a, Fixed& s, int row, int rank, int C,
                                           int pw, float T, float uf) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = kSW * pw, base = rank * per;
  const float* src = a.logits + (size_t)row * a.ld + base;
  const int cnt = max(0, min(per, a.V - base));
  // 16-byte chunks of the row: chunk j of the slice holds its logits 4 j - shift
  // .. + 3; pw / 4 chunks per warp, and the last warp has what is left
  const int shift = (int)((uintptr_t)src >> 2) & 3, j0 = w * (pw / 4);
  const double inv_t = 1.0 / (double)T, rate = inv_t * (16 / 0.693147180559945309417);
  auto floor_of = [&](float m) { return fmaxf(m - 44.f * T, -FLT_MAX); };
  auto part = [&](double x, float m, float top) -> double {    // x of weights to m, to top
    if (!(m >= floor_of(top))) return 0.0;
    const Pow2 p = exp2_16th(fma((double)m - (double)top, rate, kExpBias), s.tab);
    return x * (p.p * p.s);
  };
  auto load = [&](int j, float* v) {
    const int i = 4 * j - shift;
    if (i >= 0 && i + 4 <= cnt) {
      const float4 f = *reinterpret_cast<const float4*>(src + i);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = i + u >= 0 && i + u < cnt ? src[i + u] : -INFINITY;
    }
  };
  float top = -INFINITY;
  double sum = 0.0;
  constexpr int kQ = 4;                             // chunks at once
  const int rounds = pw / 128 + (w == kSW - 1 && shift);
#pragma unroll 1
  for (int t = 0; t < rounds; t += kQ) {
    float v[4 * kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      if (t + q < pw / 128)
        load(j0 + lane + 32 * (t + q), v + 4 * q);
      else if (t + q == pw / 128 && w == kSW - 1 && lane == 0)
        load(j0 + 32 * (t + q), v + 4 * q);
      else
        v[4 * q] = v[4 * q + 1] = v[4 * q + 2] = v[4 * q + 3] = -INFINITY;
    }
    float big = v[0];
#pragma unroll
    for (int u = 1; u < 4 * kQ; ++u) big = fmaxf(big, v[u]);     // (passes over NaN)
    if (big > top) {
      sum = part(sum, top, big);
      top = big;
    }
    const float from = floor_of(top);
    const double td = (double)top;
#pragma unroll
    for (int u = 0; u < 4 * kQ; ++u) {
      const Pow2 x = exp2_16th(fma((double)v[u] - td, rate, kExpBias), s.tab);
      if (v[u] >= from) sum = fma(x.p, x.s, sum);
    }
  }
  const uint32_t key = __reduce_max_sync(0xffffffffu, top > -INFINITY ? key_of(top + 0.f) : 0u);
  auto top_of = [](uint32_t k) { return k ? key_float(k) : -INFINITY; };
  sum = wsum(part(sum, top, top_of(key)));
  if (lane == 0) {
    s.ured[0][w] = key;
    s.dred[w] = sum;
  }
  __syncthreads();
  // every block has started: its shared memory may be written
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (w == 0) {
    const uint32_t k = s.ured[0][lane & (kSW - 1)], all = __reduce_max_sync(0xffffffffu, k);
    const double x = lane < kSW ? part(s.dred[lane], top_of(k), top_of(all)) : 0.0, t = wsum(x);
    if (lane < C) {
      put32(&s.ex.max[rank], lane, all);
      put64(&s.ex.sum[rank], lane, __double_as_longlong(t));
    }
  }
  cluster_sync_all();
  const uint32_t bk = lane < C ? s.ex.max[lane] : 0u, mk = __reduce_max_sync(0xffffffffu, bk);
  if (mk == 0) {                     // nothing to draw
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  const float m = key_float(mk), floor = floor_of(m);
  const uint32_t wk = s.ured[0][lane & (kSW - 1)];
  double share, of_warp;
  const int lo = 4 * j0 - shift;                    // the first logit of the warp's part
  if (m == INFINITY) {
    // beside +inf nothing weighs anything
    int n = 0;
    for (int i = lo + lane; i < lo + pw + (w == kSW - 1 ? 4 : 0); i += 32)
      n += i >= 0 && i < cnt && src[i] == m;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) s.dred[w] = n;
    __syncthreads();
    of_warp = lane < kSW ? s.dred[lane] : 0.0;
    share = wsum(of_warp);
    if (w == 0 && lane < C) put64(&s.ex.sum[rank], lane, __double_as_longlong(share));
    cluster_sync_all();
    share = lane < C ? s.ex.sum[lane] : 0.0;
  } else {
    share = lane < C ? part(s.ex.sum[lane], top_of(bk), m) : 0.0;
    of_warp = lane < kSW ? part(s.dred[lane], top_of(wk), m) : 0.0;
  }
  const double total = wsum(share), target = target_of(uf, total), md = (double)m;
  double start;
  if (holder(share, 0.0, target, &start) != rank) return;
  const int at = holder(of_warp, start, target, &start), first = at * pw - shift;
  draw_in_part<3>(
      s, pw + (at == kSW - 1 ? 4 : 0), start, target,
      [&](int j) {
        const int i = first + j;
        return i >= 0 && i < cnt ? src[i] : -INFINITY;
      },
      [&](float v, int) { return m == INFINITY ? v == m : v >= floor; },
      [&](float v) -> double {
        const Pow2 p = exp2_16th(fma(v == m ? 0.0 : (double)v - md, rate, kExpBias), s.tab);
        return p.p * p.s;
      },
      m,
      [&](int j, float v) {
        a.tokens[row] = base + first + j;
        if (a.logprobs)
          a.logprobs[row] = (float)((v == m ? 0.0 : ((double)v - md) * inv_t) - log(total));
      });
}

__global__ void __launch_bounds__(kSampThreads, 2) sample_kernel(SampleArgs a, int C, int pw) {
  extern __shared__ __align__(16) uint8_t smraw[];
  Fixed& s = *reinterpret_cast<Fixed*>(smraw);
  const int gc = cand_cap(C);
  u64* ex_mass = reinterpret_cast<u64*>(smraw + sizeof(Fixed));
  Cand* ex_cand = reinterpret_cast<Cand*>(ex_mass + C * kNB);
  uint32_t* hist_all = reinterpret_cast<uint32_t*>(ex_cand + C * gc);
  Cand* own_cand = reinterpret_cast<Cand*>(hist_all);
  float* zs0 = reinterpret_cast<float*>(hist_all + kHistWords);
  const int row = blockIdx.x / C, rank = blockIdx.x - row * C;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = kSW * pw, base = rank * per;      // this block's slice
  const int i0 = w * pw + lane, i1 = w * pw + pw;   // this thread's logits: i0, i0 + 32, ..
  uint32_t* bins = reinterpret_cast<uint32_t*>(zs0 + per + 4) + tid;
  const int run = pw / 32;                          // logits per thread: 4 .. 32, a multiple of kU
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (tid < 16)
    s.tab[tid] = __hiloint2double(__double2hiint(kExpTab[tid]) - (tid << 16), __double2loint(kExpTab[tid]));
  pdl_wait();
  pdl_trigger();
  const float* z = a.logits + (size_t)row * a.ld;
  const float T = a.temperature ? a.temperature[row] : 1.f;
  int k = a.top_k ? a.top_k[row] : 0;
  if (k <= 0 || k > a.V) k = a.V;
  const bool greedy = !(T > 0.f) || k == 1;
  float minp = a.min_p ? a.min_p[row] : 0.f, topp = a.top_p ? a.top_p[row] : 1.f;
  minp = minp > 0.f ? fminf(minp, 1.f) : 0.f;
  const float uf = a.uniform[row];
  const bool cuts = k < a.V || topp < 1.f;
  if (!greedy && !cuts && !(minp > 0.f)) {
    __syncthreads();                                // the table
    draw_whole(a, s, row, rank, C, pw, T, uf);
    return;
  }

  // ---- the slice, its largest and smallest finite logit ---------------------
  // In four parts, so that the first are looked at while the others arrive: a
  // thread looks at the chunks it copied.
  const float* src = z + base;
  const int cnt = max(0, min(per, a.V - base));
  const int shift = (int)((uintptr_t)src >> 2) & 3, head = min((4 - shift) & 3, cnt);
  float* zs = zs0 + shift;
  const int chunks = (cnt - head) / 4, tail = head + 4 * chunks;
  if (tid < head) zs[tid] = src[tid];
  if (tid < cnt - tail) zs[tail + tid] = src[tail + tid];
  for (int i = cnt + tid; i < per; i += kSampThreads) zs[i] = -INFINITY;
  const int rounds = (chunks + kSampThreads - 1) / kSampThreads, part = (rounds + 3) / 4;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll 1
    for (int t = g * part; t < (g + 1) * part; ++t) {
      const int i = tid + t * kSampThreads;
      if (i < chunks)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(su32(zs + head + 4 * i)),
                     "l"(src + head + 4 * i)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  const double inv_t = 1.0 / (double)T, rate = inv_t * (16 / 0.693147180559945309417);
  float vmax = -INFINITY, vmin = INFINITY;          // of what may be drawn
  auto look = [&](float v) {
    vmax = fmaxf(vmax, v);                          // (passes over NaN)
    if (cuts && v > -INFINITY) vmin = fminf(vmin, v);
  };
  if (tid < head) look(src[tid]);
  if (tid < cnt - tail) look(src[tail + tid]);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (g == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
    if (g == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
    if (g == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (g == 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
    for (int t = g * part; t < (g + 1) * part; ++t) {
      const int i = tid + t * kSampThreads;
      if (i < chunks) {
        const float4 v = *reinterpret_cast<const float4*>(zs + head + 4 * i);
        look(v.x);
        look(v.y);
        look(v.z);
        look(v.w);
      }
    }
  }
  // integer images (+ 0.f: -0 as +0)
  uint32_t kmax = vmax > -INFINITY ? key_of(vmax + 0.f) : 0u;
  uint32_t kmin = vmin < INFINITY ? key_of(vmin + 0.f) : 0xffffffffu;
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  if (lane == 0) {
    s.ured[0][w] = kmax;
    s.ured[1][w] = kmin;
  }
  __syncthreads();
  // every block has started: its shared memory may be written
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (w == 0) {
    kmax = __reduce_max_sync(0xffffffffu, s.ured[0][lane & (kSW - 1)]);
    kmin = __reduce_min_sync(0xffffffffu, s.ured[1][lane & (kSW - 1)]);
    if (lane < C) {
      put32(&s.ex.max[rank], lane, kmax);
      put32(&s.ex.min[rank], lane, kmin);
    }
  }
  cluster_sync_all();
  kmax = __reduce_max_sync(0xffffffffu, lane < C ? s.ex.max[lane] : 0u);
  kmin = __reduce_min_sync(0xffffffffu, lane < C ? s.ex.min[lane] : 0xffffffffu);
  if (kmax == 0) {                   // nothing to draw
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  // lo: the smallest logit where a cutoff is looked for, else -inf
  float m = key_float(kmax), lo = cuts ? fminf(m, key_float(kmin)) : -INFINITY;
  if (greedy) {
    // the lowest index of the largest logit, in the first block that has it
    const unsigned has = __ballot_sync(0xffffffffu, lane < C && s.ex.max[lane] == kmax);
    if (rank != __ffs(has) - 1) return;
    uint32_t at = 0xffffffffu;
    for (int i = i0; i < i1; i += 32)
      if (zs[i] == m) at = min(at, (uint32_t)i);
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.ured[0][w] = at;
    __syncthreads();
    at = __reduce_min_sync(0xffffffffu, s.ured[0][lane & (kSW - 1)]);
    if (tid == 0) {
      a.tokens[row] = base + at;
      if (a.logprobs) a.logprobs[row] = 0.f;
    }
    return;
  }
  if (m == INFINITY) {               // beside +inf nothing weighs anything
    for (int i = i0; i < i1; i += 32) zs[i] = zs[i] == m ? 0.f : -INFINITY;
    m = lo = 0.f;
    kmax = key_of(m);
  }
  const double md = (double)m;
  // Logits below `floor` weigh nothing: less than e^-44 of the largest, 2^-46
  // of the mass for all of a row.  (-inf never weighs, however large T.)
  const float floor = fmaxf(m - 44.f * T, -FLT_MAX);
  // N at a time, free of branches, so that they overlap; for v >= floor
  auto powers = [&](auto& x, const auto& v) {
    constexpr int N = sizeof(v) / sizeof(v[0]);
#pragma unroll
    for (int u = 0; u < N; ++u) x[u] = exp2_16th(fma((double)v[u] - md, rate, kExpBias), s.tab);
  };
  auto power = [&](float v) -> Pow2 {
    const float one[1] = {v};
    Pow2 x[1];
    powers(x, one);
    return x[0];
  };
  auto weight = [&](float v) -> double {
    const Pow2 x = power(v);
    return x.p * x.s;
  };
  // weights as integers of 43 bits, nearest (adding 2^52 leaves them in the
  // low bits of the double)
  auto as_fixed = [&](Pow2 x) -> u64 {
    const double s43 = __hiloint2double(__double2hiint(x.s) + (43 << 20), __double2loint(x.s));
    return (u64)__double_as_longlong(fma(x.p, s43, 0x1p52)) & 0xfffffffffffffull;
  };
  auto fixed = [&](float v) { return as_fixed(power(v)); };

  // kept: z > cz, or z == cz and index <= ci
  float cz = -INFINITY;
  int ci = -1;
  bool cut = false;
  if (minp > 0.f) {
    // least logit with weight >= min_p: 32-way search of the integer images
    uint32_t l = key_of(lo), h = kmax;
    while (l < h) {
      const uint32_t step = (h - l) / 32 + 1;
      const uint32_t p = l + min(h - l, step * lane);
      const float v = key_float(p);
      const unsigned ok = __ballot_sync(
          0xffffffffu, v >= floor ? weight(fmaxf(v, floor)) >= (double)minp : false);
      const int f = ok ? __ffs(ok) - 1 : 32;          // lanes f.. hold
      if (f == 0) {
        h = l;
        break;
      }
      const uint32_t nl = l + min(h - l, step * (f - 1)) + 1;
      if (f < 32) h = l + min(h - l, step * f);
      l = nl;
    }
    cz = key_float(h);
    ci = 0x7fffffff;
    cut = true;
    lo = fmaxf(lo, cz);
  }

  // ---- few logits: the row's blocks send each other those in their masks (at
  // `to`; s.n is 0), which hold the top k, and decide from the list; false if
  // a block has too many to send.  Block 0 then finishes the row.
  auto listed = [&](uint32_t mask, Cand* to) -> bool {
    const int mine = __popc(mask), warps = __reduce_add_sync(0xffffffffu, mine);
    if (warps) {
      int at = 0, inc = mine;
      if (lane == 0) at = atomicAdd(&s.n, warps);
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      at += inc - mine;
      for (uint32_t r = mask; r; r &= r - 1, ++at) {
        const int i = i0 + 32 * (__ffs(r) - 1);
        const float v = zs[i];
        const double x = v >= floor ? weight(fmaxf(v, floor)) : 0.0;
        if (at < gc) own_cand[at] = Cand{v, base + i, (u64)__double_as_longlong(x)};
      }
    }
    __syncthreads();
    const int own = s.n, send = own <= gc ? own : 0;
    if (tid < C) put32(&s.ex.l_n[rank], tid, own);
    for (int i = tid; i < C * send; i += kSampThreads) {
      const int c = i / send, j = i - c * send;
      const Cand x = own_cand[j];
      Cand* there = to + rank * gc + j;
      put32(&there->z, c, __float_as_uint(x.z));
      put32(&there->i, c, x.i);
      put64(&there->w, c, x.w);
    }
    cluster_sync_all();
    const int ln = lane < C ? s.ex.l_n[lane] : 0;
    const int n = __reduce_add_sync(0xffffffffu, ln);
    if (n > kRank || !__all_sync(0xffffffffu, ln <= gc)) return false;
    if (rank) return true;
    Cand* list = own_cand;                          // as they came
    Cand* by_index = list + kRank;
    double* kw = reinterpret_cast<double*>(by_index + kRank);
    for (int e = tid; e < C * gc; e += kSampThreads) {
      const int c = e / gc, j = e - c * gc;
      if (j < s.ex.l_n[c]) {
        int at = j;
        for (int q = 0; q < c; ++q) at += s.ex.l_n[q];
        list[at] = to[e];
      }
    }
    __syncthreads();
    if (tid < n) {
      // its place by index, and by (z, index): beyond k it weighs nothing
      Cand me = list[tid];
      int at = 0, before = 0;
#pragma unroll 4
      for (int q = 0; q < n; ++q) {
        const Cand o = list[q];
        at += o.i < me.i;
        before += o.z > me.z || (o.z == me.z && o.i < me.i);
      }
      if (before >= k) me.w = 0;                    // (+0.0)
      by_index[at] = me;
    }
    __syncthreads();
    if (tid < n) {
      // mass before it by (z, index), and of all
      const Cand me = by_index[tid];
      double before = 0.0, all = 0.0;
      bool first = true;
#pragma unroll 4
      for (int q = 0; q < n; ++q) {
        const Cand o = by_index[q];
        const double x = __longlong_as_double((long long)o.w);
        const bool b = o.z > me.z || (o.z == me.z && q < tid);
        all += x;
        before += b ? x : 0.0;
        first = first && !b;
      }
      const bool in = !(topp < 1.f) || first || before < (double)topp * all;
      kw[tid] = in ? __longlong_as_double((long long)me.w) : 0.0;
    }
    __syncthreads();
    if (w) return true;
    // running mass in index order, four neighbours per lane
    double x[kRank / 32], sum = 0.0;
#pragma unroll
    for (int u = 0; u < kRank / 32; ++u) {
      const int e = kRank / 32 * lane + u;
      x[u] = e < n ? kw[e] : 0.0;
      sum += x[u];
    }
    double inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const double total = __shfl_sync(0xffffffffu, inc, 31);
    const double target = (uf > 0.f ? fmin((double)uf, 1.0) : 0.0) * total;
    const unsigned any = __ballot_sync(0xffffffffu, sum > 0.0);
    const unsigned hit = __ballot_sync(0xffffffffu, sum > 0.0 && inc > target);
    if (lane == (hit ? __ffs(hit) - 1 : 31 - __clz(any))) {
      double c = inc - sum;
      int pick = -1;
#pragma unroll
      for (int u = 0; u < kRank / 32; ++u)
        if (x[u] > 0.0 && (pick < 0 || !(c > target))) {
          pick = kRank / 32 * lane + u;
          c += x[u];
        }
      const Cand me = by_index[pick];
      a.tokens[row] = me.i;
      if (a.logprobs)
        a.logprobs[row] = (float)((me.z == m ? 0.0 : ((double)me.z - md) * inv_t) - log(total));
    }
    return true;
  };

  u64 kept_mass = 0;                   // this thread's share of what top-p keeps

  // What a cutoff leaves out is taken out of the slice; each thread its logits.
  auto exclude = [&] {
    for (int q = 0; q < run; ++q) {
      const int i = i0 + 32 * q;
      const float v = zs[i];
      if (v < cz || (v == cz && base + i > ci)) zs[i] = -INFINITY;
    }
  };

  // ---- one cutoff: by count (top-k) or by mass (top-p); true if the row is
  // finished --------------------------------------------------------------------
  auto select = [&](const bool by_mass) -> bool {
    float hi = m, low = lo;
    // below m - 31 T integer weights are 0
    if (by_mass) low = fmaxf(fmaxf(low, m - 31.f * T), -FLT_MAX);
    low = fminf(low, hi);
    u64 mass_above = 0, want = 0;      // weights, or logits, before and up to the cutoff
    uint32_t mask = 0;                 // this thread's logits still in question
    auto masked_kept = [&] {           // the mass of those of them that are kept
      u64 f = 0;
      for (uint32_t r = mask; r; r &= r - 1) {
        const int i = i0 + 32 * (__ffs(r) - 1);
        const float v = zs[i];
        if (v > cz || (v == cz && base + i <= ci)) f += fixed(v);
      }
      return f;
    };
    for (int level = 0;; ++level) {
      // histogram of the kept logits in [low, hi]
      // bin of (hi - v) sc, rounded to nearest (monotone; the ends fall into the
      // first bin, half as wide as the others, and the last, half as wide again):
      // in f32, or in f64 where the range of the logits or its reciprocal leaves
      // f32's
      const float span = hi - low;
      const bool f32 = span > 1e-30f && span < 1e30f;
      const float sf = f32 ? (float)kNB / span : 0.f;
      const double hd = (double)hi, sc = f32 || low == hi ? 0.0 : (double)kNB / (hd - (double)low);
      auto bins_of = [&](auto& q, const auto& v) {      // for v <= hi
        constexpr int N = sizeof(v) / sizeof(v[0]);
        if (f32) {
#pragma unroll
          for (int u = 0; u < N; ++u)
            q[u] = __float_as_int(fmaf(hi - v[u], sf, 0x1.8p23f)) - 0x4b400000;
        } else {
#pragma unroll
          for (int u = 0; u < N; ++u)
            q[u] = __double2loint(fma(hd - (double)v[u], sc, 0x1.8p52));
        }
#pragma unroll
        for (int u = 0; u < N; ++u) q[u] = min(q[u], kNB - 1);
      };
      auto bin_of = [&](float v) {
        const float one[1] = {v};
        int q[1];
        bins_of(q, one);
        return q[0];
      };
      __syncthreads();
      for (int i = tid; i < kHistWords; i += kSampThreads) hist_all[i] = 0;
      if (tid == 0) {
        s.n = 0;
        s.kmin = 0xffffffffu;
        s.kmax = 0;
      }
      __syncthreads();
      uint32_t* hist = hist_all + w * 2 * kNB;
      auto count = [&](int bn, u64 f) {
        atomicAdd(hist + bn, (uint32_t)f & 0x3fffffu);
        if (by_mass) atomicAdd(hist + kNB + bn, (uint32_t)(f >> 22));
      };
      if (level == 0) {
#pragma unroll 1
        for (int q = 0; q < run; q += kU) {
          float v[kU];
          bool in[kU], any = false;
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const int i = i0 + 32 * (q + u);
            v[u] = zs[i];
            in[u] = v[u] >= low;
            any |= in[u];
          }
          uint32_t word = 0xffffffffu;
          if (__any_sync(0xffffffffu, any)) {
            int bn[kU];
            Pow2 x[kU];
            if (by_mass) powers(x, v);
            bins_of(bn, v);
#pragma unroll
            for (int u = 0; u < kU; ++u)
              if (in[u]) {
                word = __byte_perm(word, bn[u], 0x3210 + ((4 - u) << (4 * u)));
                count(bn[u], by_mass ? as_fixed(x[u]) : 1);
              }
          }
          bins[(q / kU) * kSampThreads] = word;
        }
      } else {
        for (uint32_t r = mask; r; r &= r - 1) {
          const float v = zs[i0 + 32 * (__ffs(r) - 1)];
          count(bin_of(v), by_mass ? fixed(v) : 1);
        }
      }
      __syncthreads();
      if (tid < kNB) {
        u64 f0 = 0, f1 = 0;
#pragma unroll
        for (int j = 0; j < kSW; ++j) {
          f0 += hist_all[j * 2 * kNB + tid];
          f1 += hist_all[j * 2 * kNB + kNB + tid];
        }
        const u64 f = f0 + (f1 << 22);
#pragma unroll 1
        for (int c = 0; c < C; ++c) put64(ex_mass + rank * kNB + tid, c, f);
      }
      cluster_sync_all();
      if (tid < kNB) {
        u64 f = 0;
        for (int c = 0; c < C; ++c) f += ex_mass[c * kNB + tid];
        s.bin_mass[tid] = f;
      }
      __syncthreads();
      if (w == 0) {
        // lane l holds bins 4l .. 4l + 3
        constexpr int Q = kNB / 32;
        u64 f = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) f += s.bin_mass[Q * lane + q];
        u64 fi = f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 x = __shfl_up_sync(0xffffffffu, fi, o);
          if (lane >= o) fi += x;
        }
        if (level == 0)
          want = by_mass ? max((u64)1, (u64)ceil(fmax((double)topp, 0.0) *
                                                 (double)__shfl_sync(0xffffffffu, fi, 31)))
                         : (u64)k;
        u64 af = mass_above + fi - f;
        const unsigned bal = __ballot_sync(0xffffffffu, mass_above + fi >= want);
        if (lane == (bal ? __ffs(bal) - 1 : 31)) {
          int bn = -1;
          if (bal)
            for (bn = Q * lane; bn < Q * lane + Q - 1; ++bn) {
              if (af + s.bin_mass[bn] >= want) break;
              af += s.bin_mass[bn];
            }
          s.bin = bn;                   // -1: fewer than k are kept
          s.mass_above = af;
          s.want = want;
        }
      }
      __syncthreads();
      const int bin = s.bin;
      if (bin < 0) {
        cluster_sync_all();             // the histograms have been read
        return false;
      }
      mass_above = s.mass_above;
      want = s.want;
      if (by_mass) {
        // the warp's share of what lies above the bin
#pragma unroll
        for (int q = 0; q < kNB / 32; ++q)
          if (kNB / 32 * lane + q < bin)
            kept_mass += hist[kNB / 32 * lane + q] + ((u64)hist[kNB + kNB / 32 * lane + q] << 22);
      }
      if (!by_mass && level == 0 && mass_above + s.bin_mass[bin] <= (u64)kRank) {
        // all logits down to the bin's end are few
        uint32_t upto = 0;
#pragma unroll 1
        for (int q = 0; q < run; q += kU) {
          const uint32_t e = __vcmpleu4(bins[(q / kU) * kSampThreads], bin * 0x01010101u) & 0x08040201u;
          upto |= ((e | e >> 8 | e >> 16 | e >> 24) & 15u) << q;
        }
        if (listed(upto, ex_cand)) return true;
        __syncthreads();
        if (tid == 0) s.n = 0;
        __syncthreads();
      }
      // the bin's logits
      if (level == 0) {
#pragma unroll 1
        for (int q = 0; q < run; q += kU) {
          const uint32_t e = __vcmpeq4(bins[(q / kU) * kSampThreads], bin * 0x01010101u) & 0x08040201u;
          mask |= ((e | e >> 8 | e >> 16 | e >> 24) & 15u) << q;
        }
      } else {
        for (uint32_t r = mask; r; r &= r - 1) {
          const int q = __ffs(r) - 1;
          if (bin_of(zs[i0 + 32 * q]) != bin) mask ^= 1u << q;
        }
      }
      float bmin = INFINITY, bmax = -INFINITY;
      for (uint32_t r = mask; r; r &= r - 1) {
        const float v = zs[i0 + 32 * (__ffs(r) - 1)];
        bmin = fminf(bmin, v);
        bmax = fmaxf(bmax, v);
      }
      const int mine = __popc(mask);
      const int warps = __reduce_add_sync(0xffffffffu, mine);
      int at = 0;
      if (warps) {
        const uint32_t k0 = __reduce_min_sync(0xffffffffu, mine ? key_of(bmin + 0.f) : 0xffffffffu);
        const uint32_t k1 = __reduce_max_sync(0xffffffffu, mine ? key_of(bmax + 0.f) : 0u);
        if (lane == 0) {
          at = atomicAdd(&s.n, warps);
          atomicMin(&s.kmin, k0);
          atomicMax(&s.kmax, k1);
        }
        at = __shfl_sync(0xffffffffu, at, 0);
      }
      __syncthreads();
      if (warps && s.n <= gc) {
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        at += inc - mine;
        for (uint32_t r = mask; r; r &= r - 1, ++at) {
          const int i = i0 + 32 * (__ffs(r) - 1);
          own_cand[at] = Cand{zs[i], base + i, by_mass ? fixed(zs[i]) : 1};
        }
      }
      __syncthreads();
      const int own = s.n;
      if (tid < C) {
        put32(&s.ex.g_n[rank], tid, own);
        put32(&s.ex.g_min[rank], tid, s.kmin);
        put32(&s.ex.g_max[rank], tid, s.kmax);
      }
      const int send = own <= gc ? own : 0;
      for (int i = tid; i < C * send; i += kSampThreads) {
        const int c = i / send, j = i - c * send;
        const Cand x = own_cand[j];
        Cand* to = ex_cand + rank * gc + j;
        put32(&to->z, c, __float_as_uint(x.z));
        put32(&to->i, c, x.i);
        put64(&to->w, c, x.w);
      }
      cluster_sync_all();
      const int gn = lane < C ? s.ex.g_n[lane] : 0;
      const int total = __reduce_add_sync(0xffffffffu, gn);
      low = key_float(__reduce_min_sync(0xffffffffu, lane < C ? s.ex.g_min[lane] : 0xffffffffu));
      hi = key_float(__reduce_max_sync(0xffffffffu, lane < C ? s.ex.g_max[lane] : 0u));
      if (total <= kRank && __all_sync(0xffffffffu, gn <= gc)) {
        // all candidates in one list; each is ranked by `span` neighbouring
        // lanes; the cutoff is the last one kept
        Cand* list = own_cand;
        for (int e = tid; e < C * gc; e += kSampThreads) {
          const int c = e / gc, j = e - c * gc;
          if (j < s.ex.g_n[c]) {
            int at = j;
            for (int q = 0; q < c; ++q) at += s.ex.g_n[q];
            list[at] = ex_cand[e];
          }
        }
        __syncthreads();
        int span = 32;
        while (span > 4 && span * total > kSampThreads) span /= 2;
        const int e = tid / span;
        const Cand me = list[min(e, total - 1)];
        u64 f = 0;
#pragma unroll 4
        for (int q = tid % span; q < total; q += span) {
          const Cand o = list[q];
          f += o.z > me.z || (o.z == me.z && o.i < me.i) ? o.w : 0;
        }
        for (int o = span / 2; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
        f += mass_above;
        if (e < total && f < want && f + me.w >= want) {
          s.cut_z = me.z;
          s.cut_i = me.i;
        }
        __syncthreads();
        cz = s.cut_z;
        ci = s.cut_i;
        if (by_mass) kept_mass += masked_kept();
        return false;
      }
      if (low == hi) {
        // equal logits: the r-th of them in index order
        u64 r = by_mass ? (want - mass_above - 1) / fixed(low) + 1 : want - mass_above;
        r = min(r, (u64)total);
        int c = 0;
        while ((u64)s.ex.g_n[c] < r) r -= s.ex.g_n[c++];
        if (rank == c) {
          const int n = __reduce_add_sync(0xffffffffu, mine);
          if (lane == 0) s.ired[w] = n;
          __syncthreads();
          int before = 0;
          for (int j = 0; j < w; ++j) before += s.ired[j];
          if ((int)r > before && (int)r <= before + n) {
            for (int q = 0; q < run; ++q) {
              const bool t = mask >> q & 1;
              const unsigned bal = __ballot_sync(0xffffffffu, t);
              if (t && before + __popc(bal & ((2u << lane) - 1)) == (int)r)
                for (int c2 = 0; c2 < C; ++c2) put32(&s.ex.tie, c2, base + i0 + 32 * q);
              before += __popc(bal);
            }
          }
        }
        cluster_sync_all();
        cz = low;
        ci = s.ex.tie;
        if (by_mass) kept_mass += masked_kept();
        return false;
      }
    }
  };
  if (k < a.V) {
    if (cut) exclude();
    if (select(false)) return;
    cut = true;
    lo = fmaxf(lo, cz);
  }
  // few kept, and not listed yet (the histogram's bin held too many)
  if (k <= kRank) {
    uint32_t mask = 0;
    for (int q = 0; q < run; ++q) {
      const int i = i0 + 32 * q;
      const float v = zs[i];
      mask |= (uint32_t)(v >= floor && (v > cz || (v == cz && base + i <= ci))) << q;
    }
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
    // (the bins have been read by now)
    if (listed(mask, reinterpret_cast<Cand*>(bins - tid))) return;
  }
  if (topp < 1.f) {
    if (cut) exclude();
    select(true);
    cut = true;
  }

  // ---- the draw ---------------------------------------------------------------
  // weight of logit i of the slice, 0 if it is not kept
  const float from = fmaxf(cz, floor);
  auto kept = [&](float v, int i) { return v >= from && (v > cz || (v == cz && base + i <= ci)); };
  double sum = 0.0;
  if (topp < 1.f) {
    sum = (double)kept_mass * 0x1p-43;
  } else {
    uint32_t mask = 0;                 // this thread's kept logits
#pragma unroll 1
    for (int q = 0; q < run; ++q) mask |= (uint32_t)kept(zs[i0 + 32 * q], i0 + 32 * q) << q;
    if (3 * (int)__reduce_max_sync(0xffffffffu, (unsigned)__popc(mask)) < run) {
      // few: each by itself
      for (uint32_t r = mask; r; r &= r - 1) sum += weight(zs[i0 + 32 * (__ffs(r) - 1)]);
    } else {
#pragma unroll 1
      for (int q = 0; q < run; q += kU) {
        float v[kU];
        Pow2 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = zs[i0 + 32 * (q + u)];
        powers(x, v);                  // (of anything that is not kept)
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (mask >> (q + u) & 1) sum = fma(x[u].p, x[u].s, sum);
      }
    }
  }
  sum = wsum(sum);
  if (lane == 0) s.dred[w] = sum;
  __syncthreads();
  if (w == 0) {
    const double t = wsum(lane < kSW ? s.dred[lane] : 0.0);
    if (lane < C) put64(&s.ex.sum[rank], lane, __double_as_longlong(t));
  }
  cluster_sync_all();
  const double share = lane < C ? s.ex.sum[lane] : 0.0, total = wsum(share);
  const double target = target_of(uf, total);
  double start;
  if (holder(share, 0.0, target, &start) != rank) return;
  // the warp whose part holds it
  const int part_of = holder(lane < kSW ? s.dred[lane] : 0.0, start, target, &start);
  draw_in_part<2>(
      s, pw, start, target, [&](int j) { return zs[part_of * pw + j]; },
      [&](float v, int j) { return kept(v, part_of * pw + j); }, weight, m,
      [&](int j, float v) {
        a.tokens[row] = base + part_of * pw + j;
        if (a.logprobs)
          a.logprobs[row] = (float)((v == m ? 0.0 : ((double)v - md) * inv_t) - log(total));
      });
}

// ---- rows of any length ------------------------------------------------------
// One block per row, every cutoff by bisection over the integer images of the
// logits, which it reads again each time: rows that do not fit the shared
// memory of a cluster (more than 16 kFit).  One of 262208 logits takes 0.6 ms
// without cutoffs, 2.1 with top-k 50 and top-p 0.95, 4.3 with top-p 0.9.
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
  // Logits below `floor` weigh nothing, as in a cluster's rows; nor does -inf,
  // or anything beside +inf
  const float floor = m < INFINITY ? fmaxf(m - 44.f * T, -FLT_MAX) : m;
  auto weight = [&](uint32_t k) -> double {
    if (k == mk) return 1.0;
    const float v = key_float(k);
    return v >= floor ? exp(((double)v - (double)m) * inv_t) : 0.0;
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
    // the least r with base + r wc >= want (at least one token): a quotient,
    // then to the side where the products say it is
    int r = base < want ? ties : 0;
    if (r && wc > 0.0) r = (int)fmin(ceil((want - base) / wc), (double)ties);
    while (r > 0 && base + (r - 1) * wc >= want) --r;
    while (r < ties && base + r * wc < want) ++r;
    ties = min(ties, max(r, cut == mk ? 1 : 0));
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

// Slices of up to 16384 logits (the warps' histograms allow 1024 each), in
// shared memory that every GPC can give a 16-block cluster.
constexpr int kFit = 16384;

// Most blocks per row: 16, or 8 where a 16-block cluster (a non-portable
// size) cannot be scheduled.
int max_cluster() {
  constexpr int kMax = 64;
  static int n[kMax];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMax) return 8;
  if (n[dev]) return n[dev];
  auto k = sample_kernel;
  const size_t smem = sample_smem(kMaxC, kFit);
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return 8;
  int c = 8, fit = 0;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxC, 1, 1);
    cfg.blockDim = dim3(kSampThreads);
    cfg.dynamicSmemBytes = smem;
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
  // few rows: small slices on as many SMs as there are; many: two blocks of
  // full slices per SM, in clusters that are easier to place
  const int slice = (int64_t)a.B * most <= 148 ? 8192 : kFit;
  int C = 1;
  while (C < most && (int64_t)C * slice < a.V) C *= 2;
  if ((int64_t)C * kFit < a.V || (int64_t)C * a.B > 0x7fffffff) {
    launch_k(sample_any_kernel, dim3(a.B), dim3(kAnyThreads), 0, st, a);
    return;
  }
  const int pw = ((a.V + C * kSW * 32 * kU - 1) / (C * kSW * 32 * kU)) * 32 * kU;
  launch_k_cluster(sample_kernel, dim3(C * a.B), dim3(kSampThreads),
                   sample_smem(C, kSW * pw), st, C, a, C, pw);
}

}  // namespace dory

// Attention of one query token per sequence over the 8-bit K/V cache.
//
// o = sum_j p_j v_j, p = softmax(scale q.k_j), over the visible positions
// [max(0, L - window), L) of each sequence; the G = Hq / Hkv query heads of a
// KV head share every byte read.  HBM-bound: 2 hd bytes per key and KV head,
// 4 G hd flops on them.
//
// Work is counted in blocks of 32 positions (one scale each).  The blocks of
// all (sequence, KV head) pairs are laid end to end and cut into equal runs,
// one per thread block, whatever the lengths are (they are known on the
// device only).  Inside a run each of the 8 warps takes every 8th block
// through its own ring of shared-memory stages, filled by 1-D bulk copies of
// 4 rows (16 per block), and keeps its own running max, sum and output; the
// warps meet only where a pair ends.  A pair cut between thread blocks leaves
// partials (m, l, O) in the workspace, and a second kernel joins them in
// order; a pair inside one run is finished in place.
//
// One block in a warp: S^T = K Q^T on m16n8k16 (keys as A rows, the heads as
// the 8 columns), online softmax per head (lane 4g + t owns heads 2t, 2t+1),
// P^T by an in-register transpose, O^T += V^T P^T.  Codes become f16 in
// registers (exact); q is f16 after an exact shift of its row by a power of
// two (bf16 has 8 significant bits, f16 11; elements 2^-22 below the row's
// largest lose bits that f32 sums would lose too).  Weights are f16 as
// p * 2^14: 11 bits, and none above 2^-38 of the largest is lost.  K's scale
// joins the score's factor, V's the f32 sum into O, so scales of any range
// are safe.
//
// Key 4 g + i of a block (g < 8, i < 4) sits in row group g: 4 rows of one
// bulk copy.  Fragment row g reads group g, so its 8 rows come from 8 copies,
// each placed 16 bytes further (mod 128): 16-byte loads of K and transposing
// ldmatrix of V then hit 8 different bank groups for every head_dim.
#include <algorithm>

#include "async_copy.cuh"
#include "common.cuh"
#include "kv8.cuh"
#include "warp_mma.cuh"

namespace dory {

namespace {

constexpr int NW = 8;                         // warps
constexpr int kThreads = 32 * NW;
constexpr float kShift = 14.f;                // weights are p * 2^14

// 2^x on the SFU (subnormal results flush to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int HD, int G>
struct Att {
  static constexpr int KS = HD / 16;
  static constexpr int COPY = 4 * HD;                  // bytes of one bulk copy
  static constexpr int MAT = 8 * (COPY + 16);          // K (or V) of one block
  static constexpr int STAGE = 2 * MAT;
  static constexpr int COMB = NW * G * (HD + 2) * 4;   // warp states of a pair
  static constexpr int NST = std::min(6, (210 * 1024 - COMB) / (NW * STAGE));
  static constexpr int PART = G * (HD + 2);            // floats of a partial
  static constexpr size_t smem(int B) {
    return 128 + (size_t)NW * NST * STAGE + COMB + (size_t)(2 * B + 1) * 4;
  }
  static_assert(NST >= 2, "two stages");
};

// Byte offset of row group g of a matrix (copies in the order 0 2 4 6 1 3 5 7).
template <int HD>
__device__ __forceinline__ int group_off(int g) {
  return ((g >> 1) + 4 * (g & 1)) * (4 * HD + 16);
}

// Workspace: prefix of blocks per sequence [B + 1], then two partial slots
// per thread block (its first pair, its last pair).
__host__ __device__ inline size_t prefix_bytes(int B) {
  return ((size_t)(B + 1) * 4 + 255) & ~(size_t)255;
}

// Blocks of the run of one thread block: at least one per warp.
__device__ __forceinline__ int run_blocks(int total, int grid) {
  return max((total + grid - 1) / grid, NW);
}

template <int HD, int G>
__global__ void __launch_bounds__(kThreads, 1) kv8_attend_kernel(const Kv8AttendArgs a) {
  using L = Att<HD, G>;
  constexpr int KS = L::KS, NST = L::NST;
  extern __shared__ uint8_t smraw[];
  uint8_t* stages = smraw + ((128 - (su32(smraw) & 127)) & 127);
  float* comb = reinterpret_cast<float*>(stages + NW * NST * L::STAGE);
  int* pre = reinterpret_cast<int*>(comb + NW * G * (HD + 2));   // [B + 1]
  int* lens = pre + a.B + 1;                                     // [B]
  __shared__ __align__(8) uint64_t full_[NW][NST];
  __shared__ int2 meta_[NW][NST];
  __shared__ int wsum[NW];

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int B = a.B, H = a.c.Hkv;
  uint64_t* full = full_[w];
  volatile int2* meta = meta_[w];
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  fence_proxy_async_global();          // rows that earlier kernels wrote

  // prefix of blocks per sequence
  for (int b0 = 0, run = 0; b0 < B; b0 += kThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < B) {
      int len = a.len[b];
      if (len < 0 || len > a.c.pages_per_seq * kPage) {
        if (blockIdx.x == 0) atomicOr(a.err, ERRBIT_BOUNDS);
        len = 0;
      }
      lens[b] = len;
      const int lo = a.window ? max(0, len - a.window) : 0;
      n = (len + kKv8Block - 1) / kKv8Block - lo / kKv8Block;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) wsum[w] = inc;
    __syncthreads();
    int base = run;
    for (int i = 0; i < NW; ++i) {
      if (i < w) base += wsum[i];
      run += wsum[i];
    }
    if (b < B) pre[b + 1] = base + inc;
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  const int total = pre[B] * H;
  const int per = run_blocks(total, gridDim.x);
  const int x0 = min(total, (int)blockIdx.x * per), x1 = min(total, x0 + per);
  if (blockIdx.x == 0) {
    int* out = reinterpret_cast<int*>(a.ws);
    for (int b = tid; b <= B; b += kThreads) out[b] = pre[b];
  }
  for (int b = blockIdx.x; b < B; b += gridDim.x)      // empty sequences
    if (pre[b + 1] == pre[b])
      for (int i = tid; i < H * G * HD; i += kThreads)
        a.out[(size_t)b * H * G * HD + i] = __float2bfloat16_rn(0.f);

  // sequence that holds linear block x
  auto seq_of = [&](int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (x < pre[mid + 1] * H) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  auto first_block = [&](int b) {
    return a.window ? max(0, lens[b] - a.window) / kKv8Block : 0;
  };

  // ---- this warp's items: blocks x0 + w + NW m ---------------------------
  const int items = x0 + w < x1 ? (x1 - x0 - w + NW - 1) / NW : 0;
  int plan_unit = -1, plan_j = 0;      // lane l: item 32 k + l of the batch
  const uint32_t st_base = su32(stages + (size_t)w * NST * L::STAGE);
  uint8_t* st_ptr = stages + (size_t)w * NST * L::STAGE;
  auto issue = [&](int m, int s) {
    if ((m & 31) == 0) {
      const int x = x0 + w + NW * (m + lane);
      plan_unit = -1;
      if (x < x1) {
        const int b = seq_of(x), nb = pre[b + 1] - pre[b], r = x - pre[b] * H;
        const int h = r / nb;
        plan_j = r - h * nb + first_block(b);
        const int page = a.c.block_table[(size_t)b * a.c.pages_per_seq + (plan_j >> 1)];
        if (page >= 0 && page < a.c.n_pages) plan_unit = (page * H + h) * 2 + (plan_j & 1);
        else atomicOr(a.err, ERRBIT_BOUNDS);
      }
    }
    const int u = __shfl_sync(0xffffffffu, plan_unit, m & 31);
    const int j = __shfl_sync(0xffffffffu, plan_j, m & 31);
    if (lane == 0) {
      meta[s].x = u;
      meta[s].y = j;
      mbar_expect_tx(full + s, u >= 0 ? 2 * kKv8Block * HD : 0);
    }
    __syncwarp();
    if (u >= 0 && lane < 16) {
      const int gg = lane & 7;
      const uint8_t* src = (lane < 8 ? a.c.k : a.c.v) + (size_t)u * (kKv8Block * HD) + gg * L::COPY;
      bulk_load(st_ptr + s * L::STAGE + (lane < 8 ? 0 : L::MAT) + group_off<HD>(gg), src, L::COPY,
                full + s);
    }
  };
  for (int m = 0; m < min(NST, items); ++m) issue(m, m);

  bool ok = true;
  int n = 0, s = 0;                    // items done; their stage
  uint32_t ph = 0;                     // and its parity
  float ks = 0.f, vs = 0.f;            // scales of item n
  auto load_scales = [&](int stage) {
    const int u = meta[stage].x;
    ks = u >= 0 ? a.c.k_scale[u] : 0.f;
    vs = u >= 0 ? a.c.v_scale[u] : 0.f;
  };
  if (items > 0) load_scales(0);

  // ---- the pairs of this run ----------------------------------------------
  for (int x = x0; x < x1;) {
    const int b = seq_of(x), nb = pre[b + 1] - pre[b];
    const int h = (x - pre[b] * H) / nb;
    const int xs = pre[b] * H + h * nb, xe = xs + nb;  // the pair's blocks
    const int xn = min(xe, x1);
    const int len = lens[b], lo = a.window ? max(0, len - a.window) : 0;

    // Q^T fragments: lane (g, t) holds head g; k-step 4c + i of 64-dim chunk
    // c pairs dims 64c + 16t + 4i + {0, 1} and {2, 3}, as the K loads do
    uint32_t qf[KS][2];
    float hs[2];                       // score factors of heads 2t, 2t + 1
    {
      uint2 raw[KS];
      uint32_t mx = 0;
      const bf16* qr = a.q + b * a.qs_b + (int64_t)(h * G + min(g, G - 1)) * a.qs_h;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int c = k >> 2, i = k & 3;
        const int d = c < HD / 64 ? 64 * c + 16 * t + 4 * i : 64 * c + 8 * t + 4 * i;
        raw[k] = *reinterpret_cast<const uint2*>(qr + d);
        mx = max(mx, max(kv8_amax2(raw[k].x), kv8_amax2(raw[k].y)));
      }
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the row's largest magnitude to [2^8, 2^9)
      const int e = mx ? min(max(127 + 8 - (int)(mx >> 23), -126), 126) : 0;
      const float f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const __half2 u0 = __floats2half2_rn(bf_lo(raw[k].x) * f, bf_hi(raw[k].x) * f);
        const __half2 u1 = __floats2half2_rn(bf_lo(raw[k].y) * f, bf_hi(raw[k].y) * f);
        qf[k][0] = g < G ? *reinterpret_cast<const uint32_t*>(&u0) : 0u;
        qf[k][1] = g < G ? *reinterpret_cast<const uint32_t*>(&u1) : 0u;
      }
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23) * a.scale * 1.4426950408889634f;
      hs[0] = __shfl_sync(0xffffffffu, inv, 8 * t);
      hs[1] = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
    }

    float m2[2] = {-INFINITY, -INFINITY}, l2[2] = {0.f, 0.f};
    float o[KS][4];
#pragma unroll
    for (int d = 0; d < KS; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

    for (; ok && n < items && x0 + w + NW * n < xn; ++n) {
      const float ksc = ks, vsc = vs;
      const int u = meta[s].x, j = meta[s].y;
      const int s1 = s + 1 == NST ? 0 : s + 1;
      if (n + 1 < items) load_scales(s1);
      ok = mbar_wait_warp(full + s, ph);
      if (ok && u >= 0) {
        const uint32_t ka = st_base + s * L::STAGE, va = ka + L::MAT;
        const int p0 = j * kKv8Block;
        const bool edge = p0 < lo || p0 + kKv8Block > len;
        if (edge) {
          // rows outside [lo, len) get weight 0; zero their V codes, so that
          // whatever they hold cannot turn 0 * v into NaN
          uint8_t* vt = st_ptr + s * L::STAGE + L::MAT;
          for (int e = lane; e < kKv8Block * (HD / 16); e += 32) {
            const int r = e / (HD / 16), c = e - r * (HD / 16);
            if (p0 + r < lo || p0 + r >= len)
              *reinterpret_cast<uint4*>(vt + group_off<HD>(r >> 2) + (r & 3) * HD + 16 * c) =
                  make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        // S^T: key 4g + i; sa rows i = 0 (c0, c1) and 1 (c2, c3), sb 2 and 3
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t kr = ka + group_off<HD>(g);
#pragma unroll
        for (int c = 0; c < (HD + 63) / 64; ++c) {
          uint32_t kw[4][4];
          const bool wide = c < HD / 64;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (wide)
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(kw[i][0]), "=r"(kw[i][1]), "=r"(kw[i][2]), "=r"(kw[i][3])
                           : "r"(kr + i * HD + 64 * c + 16 * t));
            else
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                           : "=r"(kw[i][0]), "=r"(kw[i][1])
                           : "r"(kr + i * HD + 64 * c + 8 * t));
          }
#pragma unroll
          for (int i = 0; i < (wide ? 4 : 2); ++i) {
            const int k = 4 * c + i;
            mma16816_f16(sa, kv8_f16x2(kw[0][i]), kv8_f16x2(kw[1][i]), kv8_f16x2(kw[0][i] >> 16),
                         kv8_f16x2(kw[1][i] >> 16), qf[k][0], qf[k][1]);
            mma16816_f16(sb, kv8_f16x2(kw[2][i]), kv8_f16x2(kw[3][i]), kv8_f16x2(kw[2][i] >> 16),
                         kv8_f16x2(kw[3][i] >> 16), qf[k][0], qf[k][1]);
          }
        }
        const float f0 = hs[0] * ksc, f1 = hs[1] * ksc;
        float sc[4][2] = {{sa[0] * f0, sa[1] * f1}, {sa[2] * f0, sa[3] * f1},
                          {sb[0] * f0, sb[1] * f1}, {sb[2] * f0, sb[3] * f1}};
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * g + i;
            if (p < lo || p >= len) sc[i][0] = sc[i][1] = -INFINITY;
          }
        }
        float corr[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float mx = fmaxf(fmaxf(sc[0][hh], sc[1][hh]), fmaxf(sc[2][hh], sc[3][hh]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
          const float mn = fmaxf(m2[hh], mx);
          corr[hh] = mn == -INFINITY ? 1.f : ex2(m2[hh] - mn);
          const float mm = mn == -INFINITY ? 0.f : mn - kShift;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[i][hh] = ex2(sc[i][hh] - mm);
            sum += sc[i][hh];
          }
          l2[hh] = l2[hh] * corr[hh] + sum;      // of this lane's keys
          m2[hh] = mn;
        }
        uint32_t pb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 v = __floats2half2_rn(sc[i][0], sc[i][1]);
          pb[i] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&v));
        }
        // O^T: rows g and g + 8 of 16-dim block d are dims 16d + 2g, 16d + 2g + 1
        const uint32_t vr = va + group_off<HD>(lane & 7) + (lane >> 3) * HD;
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          uint32_t r[4];
          ldsm_x4_t(vr + 16 * d, r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) r[i] = __byte_perm(r[i], 0, 0x3120);
          float tt[4] = {0.f, 0.f, 0.f, 0.f};
          mma16816_f16(tt, kv8_f16x2(r[0]), kv8_f16x2(r[0] >> 16), kv8_f16x2(r[1]),
                       kv8_f16x2(r[1] >> 16), pb[0], pb[1]);
          mma16816_f16(tt, kv8_f16x2(r[2]), kv8_f16x2(r[2] >> 16), kv8_f16x2(r[3]),
                       kv8_f16x2(r[3] >> 16), pb[2], pb[3]);
          o[d][0] = fmaf(tt[0], vsc, o[d][0] * corr[0]);
          o[d][1] = fmaf(tt[1], vsc, o[d][1] * corr[1]);
          o[d][2] = fmaf(tt[2], vsc, o[d][2] * corr[0]);
          o[d][3] = fmaf(tt[3], vsc, o[d][3] * corr[1]);
        }
        if (edge) fence_proxy_async_smem();
      }
      __syncwarp();                    // the stage has been read
      if (ok && n + NST < items) issue(n + NST, s);
      s = s1;
      if (s == 0) ph ^= 1;
    }

    // the pair's state in this thread block: the warps' states joined
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l2[hh] += __shfl_xor_sync(0xffffffffu, l2[hh], sh);
      const int head = 2 * t + hh;
      if (head < G) {
        float* ws = comb + (w * G + head) * (HD + 2);
        if (g == 0) {
          ws[0] = m2[hh];
          ws[1] = l2[hh];
        }
#pragma unroll
        for (int d = 0; d < KS; ++d)
          *reinterpret_cast<float2*>(ws + 2 + 16 * d + 2 * g) = make_float2(o[d][hh], o[d][hh + 2]);
      }
    }
    __syncthreads();
    const bool whole = x == xs && xn == xe;
    float* part = reinterpret_cast<float*>((char*)a.ws + prefix_bytes(B)) +
                  (size_t)(2 * blockIdx.x + (x != x0)) * L::PART;
    for (int i = tid; i < G * HD; i += kThreads) {
      const int head = i / HD, d = i - head * HD;
      const float* cs = comb + head * (HD + 2);
      float M = -INFINITY, Ls = 0.f, O = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) M = fmaxf(M, cs[k * G * (HD + 2)]);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float* ck = cs + k * G * (HD + 2);
        const float f = ck[0] == -INFINITY ? 0.f : ex2(ck[0] - M);
        Ls = fmaf(f, ck[1], Ls);
        O = fmaf(f, ck[2 + d], O);
      }
      if (whole) {
        a.out[((size_t)b * H + h) * G * HD + i] = __float2bfloat16_rn(Ls == 0.f ? 0.f : O / Ls);
      } else {
        part[2 * G + i] = O;
        if (d == 0) {
          part[head] = M;
          part[G + head] = Ls;
        }
      }
    }
    __syncthreads();
    x = xn;
  }
  // after a timeout, wait (bounded) for the copies still in flight
  if (!ok) {
    if (lane == 0) atomicOr(a.err, ERRBIT_TIMEOUT);
    for (int m = n; m < min(items, n + NST); ++m)
      if (!mbar_wait_warp(full + m % NST, (uint32_t)((m / NST) & 1))) break;
  }
}

// Joins the partials of pairs cut between thread blocks: one block per
// (query head, pair), warps over the partials.
template <int HD>
__global__ void __launch_bounds__(128) kv8_merge_kernel(const Kv8AttendArgs a, int grid) {
  constexpr int W = 4, D = HD / 32;
  __shared__ float sm[W], sl[W], so[W][HD];
  pdl_wait();
  pdl_trigger();
  const int G = a.G, H = a.c.Hkv, B = a.B;
  const int head = blockIdx.x % G, pair = blockIdx.x / G, b = pair / H, h = pair - b * H;
  const int* pre = reinterpret_cast<const int*>(a.ws);
  const int p0 = pre[b], nb = pre[b + 1] - p0;
  if (nb == 0) return;
  const int per = run_blocks(pre[B] * H, grid);
  const int xs = p0 * H + h * nb, c0 = xs / per, c1 = (xs + nb - 1) / per;
  if (c0 == c1) return;                // finished in place
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* parts = reinterpret_cast<const float*>((const char*)a.ws + prefix_bytes(B));
  float M = -INFINITY, Ls = 0.f, O[D];
#pragma unroll
  for (int d = 0; d < D; ++d) O[d] = 0.f;
#pragma unroll 2
  for (int c = c0 + w; c <= c1; c += W) {
    // a thread block's first slot holds the pair its run starts in
    const float* p = parts + (size_t)(2 * c + (c * per < xs)) * (G * (HD + 2));
    const float m = p[head], l = p[G + head];
    float v[D];
#pragma unroll
    for (int d = 0; d < D; ++d) v[d] = p[2 * G + head * HD + lane + 32 * d];
    const float mn = fmaxf(M, m);
    const float f0 = M == -INFINITY ? 0.f : ex2(M - mn), f1 = m == -INFINITY ? 0.f : ex2(m - mn);
    Ls = Ls * f0 + l * f1;
#pragma unroll
    for (int d = 0; d < D; ++d) O[d] = O[d] * f0 + v[d] * f1;
    M = mn;
  }
  if (lane == 0) {
    sm[w] = M;
    sl[w] = Ls;
  }
#pragma unroll
  for (int d = 0; d < D; ++d) so[w][lane + 32 * d] = O[d];
  __syncthreads();
  float MM = -INFINITY;
#pragma unroll
  for (int k = 0; k < W; ++k) MM = fmaxf(MM, sm[k]);
  for (int d = threadIdx.x; d < HD; d += 32 * W) {
    float L = 0.f, S = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float f = sm[k] == -INFINITY ? 0.f : ex2(sm[k] - MM);
      L = fmaf(f, sl[k], L);
      S = fmaf(f, so[k][d], S);
    }
    a.out[((size_t)pair * G + head) * HD + d] = __float2bfloat16_rn(L == 0.f ? 0.f : S / L);
  }
}

// Thread blocks: one per SM (its stages fill the shared memory).
int attend_grid() {
  constexpr int kMax = 64;
  static int n[kMax];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMax) return 148;
  if (!n[dev] &&
      cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n[dev];
}

template <int HD, int G>
void attend_t(const Kv8AttendArgs& a, cudaStream_t st) {
  using L = Att<HD, G>;
  const int grid = attend_grid();
  const size_t smem = L::smem(a.B);
  cudaFuncSetAttribute(kv8_attend_kernel<HD, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)smem);
  launch_k(kv8_attend_kernel<HD, G>, dim3(grid), dim3(kThreads), smem, st, a);
  launch_k(kv8_merge_kernel<HD>, dim3(a.B * a.c.Hkv * G), dim3(128), 0, st, a, grid);
}

template <int HD>
void attend_hd(const Kv8AttendArgs& a, cudaStream_t st) {
  switch (a.G) {
    case 1: attend_t<HD, 1>(a, st); break;
    case 2: attend_t<HD, 2>(a, st); break;
    case 4: attend_t<HD, 4>(a, st); break;
    default: attend_t<HD, 8>(a, st); break;
  }
}

}  // namespace

size_t kv8_attend_ws(int B, int G, int hd) {
  return prefix_bytes(B) + (size_t)2 * attend_grid() * G * (hd + 2) * 4;
}

void launch_kv8_attend(const Kv8AttendArgs& a, cudaStream_t st) {
  switch (a.c.hd) {
    case 64: attend_hd<64>(a, st); break;
    case 128: attend_hd<128>(a, st); break;
    default: attend_hd<160>(a, st); break;
  }
}

}  // namespace dory

// Attention of one query token per sequence over the 8-bit K/V cache.
//
// o = sum_j p_j v_j, p = softmax(scale q.k_j), over the visible positions
// [max(0, L - window), L) of each sequence; the G = Hq / Hkv query heads of a
// KV head share every byte read.  HBM-bound: 2 hd bytes per key and KV head,
// 4 G hd flops on them.
//
// Work is counted in blocks of 32 positions (one scale each).  The blocks of
// all (sequence, KV head) pairs are laid end to end and cut into equal runs,
// one per SM and again one per warp, whatever the lengths are (they are known
// on the device only).  A warp streams its run through its own ring of
// shared-memory stages, filled by TMA tile loads, with its own running max,
// sum and output; pairs inside its run it finishes alone.  Pieces of cut
// pairs (at most two per warp) are joined once the thread block is done, and
// pieces of pairs cut between thread blocks (at most two each) by a second
// kernel.  (Joining them in the last thread block to arrive instead, through
// a fence and a counter per pair, took 3 to 8 us longer than the dependent
// launch, at every size.)
//
// Where there are few pairs of short sequences each pair gets a cluster of up
// to 16 thread blocks instead, which share its blocks in the same way and join
// their pieces in each other's shared memory: one launch, no prefix sum over
// the lengths (head_dim 160, 4 KV heads, against runs: 1 sequence of 2048 7.2
// for 9.3 us, 16 of 1024 9.6 for 12.0 us).
//
// One block in a warp: S^T = K Q^T on m16n8k16 (keys as A rows, the heads as
// the 8 columns), online softmax per head (lane 4g + t owns heads 2t, 2t+1),
// P^T by an in-register transpose, O^T += V^T P^T.  Codes become f16 in
// registers (exact); q is f16 after an exact shift of its row by a power of
// two (bf16 has 8 significant bits, f16 11; elements 2^-22 below the row's
// largest lose bits that f32 sums would lose too).  Weights are f16, 11 bits:
// p * 2^9 against a reference max that moves only when a score passes it by
// 2^4 (any common reference gives the same o; so most blocks need no
// rescaling and no reduction across lanes, just one vote).  K's scale joins the
// score's factor.  V's scale, relative to the unit O is held in, joins the
// exponent of p when within 2^2: an f16 weight below 2^-23 of the largest is
// then off by up to 2^-34 of it, in O's unit.  The unit is the smallest scale
// so far (up to 2^2), so that such an error meets small values.  Blocks of
// larger scales have their weights scaled by their own largest first and their
// product added in f32: what is light may count as much as the rest by its
// values, down to weights of 2^-126 of the largest (f32).
//
// Row r = 8 i + perm(g) of a block (i < 4) is fragment row g.  Tiles carry the
// swizzle of their row width (128, 64 or 32 bytes), and perm lets two
// neighbouring g fall into different halves of the banks, so that 16-byte
// loads of K and the transposing ldmatrix of V are free of conflicts.  (One
// TMA instruction per tile: the same blocks as 16 bulk copies of 4 rows cost
// 160 issue slots per block, a third of the kernel's instructions.)
//
// Times in a graph of calls (head_dim 160, 4 query heads per KV head, 4 KV
// heads, of 6.55 TB/s): 64 sequences of 32768 tokens 416 us (98%), 4 of 131072
// 114 us (90%), one of 2048 7.2 us, a chain of length -> page -> tile -> product
// -> join (9.3 us where the block table is much longer than the sequence, as the
// form is chosen by the table).  48 sequences of up to 9001 tokens behind a
// 1024-token window (head_dim 128, 8 x 8 heads) take 32 us (46%): 10 blocks per
// warp do not amortise that chain.
#include <algorithm>
#include <mutex>

#include "async_copy.cuh"
#include "common.cuh"
#include "kv8.cuh"
#include "warp_mma.cuh"

namespace dory {

namespace {

// Polls of a bounded wait: about a second (a try_wait that fails suspends the
// thread for some microseconds).
constexpr long kPolls = 1L << 18;
constexpr float kShift = 9.f;                 // weights are p * 2^9 ...
constexpr float kSlack = 4.f;                 // ... and at most 2^4 more
constexpr int kNear = 2;                      // V scale within 2^this of O's unit: in p
constexpr int kFar = 36;                      // V scales 2^+-this: sums fit f32 in any unit
constexpr int kPlain = 256 + 127 + (int)kShift;
// Exponent field of O's unit for V's scale.
__device__ __forceinline__ int unit_for(int ev) { return abs(ev - 127) <= kFar ? ev : kPlain; }
constexpr int kMaxC = 16;                     // thread blocks per pair

// 2^x on the SFU (subnormal results flush to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^e for e <= 127 (subnormal ones too, then 0).
__device__ __forceinline__ float pow2i(int e) {
  return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : e >= -149 ? 1u << (e + 149) : 0u);
}

template <int HD>
struct Att {
  static constexpr int KS = HD / 16;
  static constexpr int W1 = HD == 64 ? 64 : 128;       // bytes of a row's first tile
  static constexpr int W2 = HD - W1;                   // and of its second (160: 32)
  static constexpr int MAT = 32 * HD;                  // K (or V) of one block
  static constexpr int STAGE = 2 * MAT;
  // Warps per thread block and stages per warp, 98 to 131 KB in flight per SM.
  // More does not help: at head_dim 160, 12 x 1, 8 x 2, 10 x 2 and 7 x 3 take
  // 420, 443, 448 and 451 us for 64 sequences of 32768 tokens (2.68 GB).
  static constexpr int NW = HD == 128 ? 8 : 12;
  static constexpr int NST = HD == 160 ? 1 : 2;
  static constexpr size_t smem(int B) {
    return 1024 + (size_t)NW * NST * STAGE + (size_t)(2 * B + 1) * 4;
  }
  static constexpr size_t smem_pair(int G) {
    return 1024 + (size_t)NW * NST * STAGE + (size_t)(G * HD + 2 * kMaxC * G) * 4;
  }
};

// Row of fragment row g within 8 rows.
template <int HD>
__device__ __forceinline__ int perm(int g) {
  return HD == 64 ? g : (g >> 1) + 4 * (g & 1);
}
// Byte offset of 16-byte chunk c of row r in a block's tiles.
template <int HD>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  if (HD == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  if (c < 8) return r * 128 + ((c ^ (r & 7)) << 4);
  return 32 * 128 + r * 32 + (((c - 8) ^ ((r >> 2) & 1)) << 4);
}

// Two neighbouring outputs, times their gate factors where there are any.
__device__ __forceinline__ void store_out2(const Kv8AttendArgs& a, size_t at, float x, float y) {
  if (a.gate) {
    const float2 g = *reinterpret_cast<const float2*>(a.gate + at);
    x *= g.x;
    y *= g.y;
  }
  *reinterpret_cast<uint32_t*>(a.out + at) = pack_bf16(x, y);
}

// A piece of a pair: O[G][hd] (unnormalised), m[G], l[G].
template <int HD, int G>
constexpr int kPart = (G * (HD + 2) + 3) & ~3;

// Workspace: two pieces per thread block (of its first pair, and of its
// last), then one per warp (of its first).

// Length of sequence b (0 if it is out of range), and the number of blocks
// its visible positions lie in.
__device__ __forceinline__ int length_of(const Kv8AttendArgs& a, int b) {
  const int len = a.len[b];
  return len < 0 || len > a.c.pages_per_seq * kPage ? 0 : len;
}
__device__ __forceinline__ int visible_blocks(const Kv8AttendArgs& a, int b) {
  const int len = length_of(a, b), lo = a.window ? max(0, len - a.window) : 0;
  return (len + kKv8Block - 1) / kKv8Block - lo / kKv8Block;
}

// PAIR: one pair per cluster of thread blocks, which share its blocks and join
// their pieces through each other's shared memory: no second kernel.
template <int HD, int G, bool PAIR>
__global__ void __launch_bounds__(32 * Att<HD>::NW, 1) kv8_attend_kernel(
    const __grid_constant__ Kv8Maps maps, const Kv8AttendArgs a, int C) {
  using L = Att<HD>;
  constexpr int KS = L::KS, NST = L::NST, NW = L::NW, kThreads = 32 * NW;
  constexpr int PART = kPart<HD, G>;
  extern __shared__ uint8_t smraw[];
  uint8_t* stages = smraw + ((1024 - (su32(smraw) & 1023)) & 1023);
  int* pre = reinterpret_cast<int*>(stages + NW * NST * L::STAGE);   // [B + 1]
  int* lens = pre + a.B + 1;                                         // [B]
  __shared__ __align__(8) uint64_t full_[NW][NST];
  __shared__ __align__(16) int4 meta_[NW][NST];     // block, pair, scales of K and V
  __shared__ int wsum[NW], s_piece[2 * NW];

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int B = a.B, H = a.c.Hkv;
  const int rank = PAIR ? (int)blockIdx.x % C : 0, own = PAIR ? (int)blockIdx.x / C : 0;   // pair
  if (PAIR) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  uint64_t* full = full_[w];
  int4* meta = meta_[w];
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  fence_proxy_async_global();          // rows that earlier kernels wrote

  int X0, X1;                          // this thread block's run
  int own_len = 0, own_nb = 0;         // PAIR: the pair's length and blocks
  if (PAIR) {
    const int b = own / H;
    own_len = length_of(a, b);
    own_nb = visible_blocks(a, b);
    if (tid == 0 && rank == 0 && own == b * H && own_len != a.len[b])
      atomicOr(a.err, ERRBIT_BOUNDS);
    const int per = (own_nb + C - 1) / C;
    X0 = min(own_nb, rank * per);
    X1 = min(own_nb, X0 + per);
  } else {
    // prefix of blocks per sequence
    for (int b0 = 0, run = 0; b0 < B; b0 += kThreads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < B) {
        lens[b] = length_of(a, b);
        if (blockIdx.x == 0 && lens[b] != a.len[b]) atomicOr(a.err, ERRBIT_BOUNDS);
        n = visible_blocks(a, b);
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
    const int per = (total + gridDim.x - 1) / gridDim.x;
    X0 = (int)min((int64_t)total, (int64_t)blockIdx.x * per);
    X1 = min(total, X0 + per);
  }
  const int perw = (X1 - X0 + NW - 1) / NW;
  const int x0 = min(X1, X0 + w * perw), x1 = min(X1, x0 + perw);
  float* ws_block = reinterpret_cast<float*>(a.ws);
  float* ws_warp = ws_block + (size_t)2 * gridDim.x * PART + (size_t)blockIdx.x * NW * PART;
  if (lane < 2) s_piece[2 * w + lane] = -1;
  for (int b = blockIdx.x; !PAIR && b < B; b += gridDim.x)      // empty sequences
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
  // first linear block of a pair, and its number of blocks
  auto start_of = [&](int pair, int* nb) {
    if (PAIR) {
      *nb = own_nb;
      return 0;
    }
    const int b = pair / H, h = pair - b * H;
    *nb = pre[b + 1] - pre[b];
    return pre[b] * H + h * *nb;
  };
  auto held = [&](int b) { return PAIR ? own_len : lens[b]; };
  auto first_block = [&](int b) {
    return a.window ? max(0, held(b) - a.window) / kKv8Block : 0;
  };

  // ---- this warp's items: blocks x0 + m ------------------------------------
  const int items = x1 - x0;
  int plan_u = -1;                     // lane l: item 32 k + l of the batch
  int4 plan = make_int4(-1, 0, 0, 0);
  const uint32_t st_base = su32(stages + (size_t)w * NST * L::STAGE);
  uint8_t* st_ptr = stages + (size_t)w * NST * L::STAGE;
  auto issue = [&](int m, int s) {
    if ((m & 31) == 0) {
      const int x = x0 + m + lane;
      plan_u = -1;
      plan.x = -1;                     // no block: a bad page
      if (x < x1) {
        int b, h, j;
        if (PAIR) {
          b = own / H;
          h = own - b * H;
          j = x;
        } else {
          b = seq_of(x);
          const int nb = pre[b + 1] - pre[b], r = x - pre[b] * H;
          h = r / nb;
          j = r - h * nb;
        }
        j += first_block(b);
        const int page = a.c.block_table[(size_t)b * a.c.pages_per_seq + (j >> 1)];
        plan.y = b * H + h;
        if (page < 0 || page >= a.c.n_pages) {
          atomicOr(a.err, ERRBIT_BOUNDS);
        } else {
          plan_u = (page * H + h) * 2 + (j & 1);
          plan.x = j;
          plan.z = __float_as_int(a.c.k_scale[plan_u]);
          plan.w = __float_as_int(a.c.v_scale[plan_u]);
        }
      }
    }
    const int u = __shfl_sync(0xffffffffu, plan_u, m & 31);
    if (lane == 0) {
      mbar_expect_tx(full + s, u >= 0 ? 2 * L::MAT : 0);
      if (u >= 0) {
        uint8_t* dst = st_ptr + s * L::STAGE;
        tma_load_2d(dst, &maps.k, 0, u * kKv8Block, full + s);
        tma_load_2d(dst + L::MAT, &maps.v, 0, u * kKv8Block, full + s);
        if (L::W2 > 0) {
          tma_load_2d(dst + 32 * L::W1, &maps.k2, L::W1, u * kKv8Block, full + s);
          tma_load_2d(dst + L::MAT + 32 * L::W1, &maps.v2, L::W1, u * kKv8Block, full + s);
        }
      }
    }
    if (lane == (m & 31)) meta[s] = plan;
    __syncwarp();
  };
  for (int m = 0; m < min(NST, items); ++m) issue(m, m);
  __syncwarp();

  bool ok = true;
  int n = 0, s = 0;                    // items done; their stage
  uint32_t ph = 0;                     // and its parity
  int pair = -1, len = 0, lo = 0;      // the current pair
  uint32_t qf[KS][2];
  float hs[2] = {0.f, 0.f};            // score factors of heads 2t, 2t + 1
  float m2[2], c2[2], l2[2], o[KS][4]; // reference max, kShift - it, sum, output
  int eu = 0;                          // O is held in units of 2^((eu & 255) - 127)
  for (;; ++n) {
    const int4 it = n < items ? meta[s] : make_int4(0, -1, 0, 0);
    if (it.y < 0 || it.y != pair) {
      if (pair >= 0) {
        // the pair's state in this warp: finished, or a piece: the run's last
        // in the warp's stages, which are idle by then, its first in the
        // workspace
        int nb;
        const int xs = start_of(pair, &nb);
        const bool whole = !PAIR && xs >= x0 && xs + nb <= x1, last = it.y < 0;
        float* part = last ? reinterpret_cast<float*>(st_ptr) : ws_warp + w * PART;
        if (!whole && lane == 0) s_piece[2 * w + (x0 < xs)] = 2 * pair + last;
        const float unit = pow2i((eu & 255) - 127 - (int)kShift);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) l2[hh] += __shfl_xor_sync(0xffffffffu, l2[hh], sh);
          l2[hh] *= 1.f / (1 << (int)kShift);
          const int head = 2 * t + hh;
          if (head < G) {
            const float f = whole ? (l2[hh] == 0.f ? 0.f : unit / l2[hh]) : unit;
            if (!whole && g == 0) {
              part[G * HD + head] = m2[hh];
              part[G * HD + G + head] = l2[hh];
            }
#pragma unroll
            for (int d = 0; d < KS; ++d) {
              const int at = head * HD + 16 * d + 2 * g;
              if (whole)
                store_out2(a, (size_t)pair * G * HD + at, o[d][hh] * f, o[d][hh + 2] * f);
              else
                *reinterpret_cast<float2*>(part + at) =
                    make_float2(o[d][hh] * f, o[d][hh + 2] * f);
            }
          }
        }
      }
      if (it.y < 0) break;
      pair = it.y;
      const int b = pair / H, h = pair - b * H;
      len = held(b);
      lo = a.window ? max(0, len - a.window) : 0;
      eu = unit_for((uint32_t)it.w >> 23);
      m2[0] = m2[1] = -INFINITY;
      c2[0] = c2[1] = INFINITY;
      l2[0] = l2[1] = 0.f;
#pragma unroll
      for (int d = 0; d < KS; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
      // Q^T fragments: lane (g, t) holds head g; k-step 4c + i of 64-dim chunk
      // c pairs dims 64c + 16t + 4i + {0, 1} and {2, 3}, as the K loads do
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

    const int j = it.x;
    ok = mbar_wait_warp(full + s, ph, kPolls);
    if (ok && j >= 0) {
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
            *reinterpret_cast<uint4*>(vt + tile_off<HD>(r, c)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      // S^T: key 8i + perm(g); sa rows i = 0 (c0, c1) and 1 (c2, c3), sb 2 and 3
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      const int pg = perm<HD>(g);
#pragma unroll
      for (int c = 0; c < (HD + 63) / 64; ++c) {
        uint32_t kw[4][4];
        const bool wide = c < HD / 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (wide)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(kw[i][0]), "=r"(kw[i][1]), "=r"(kw[i][2]), "=r"(kw[i][3])
                         : "r"(ka + tile_off<HD>(8 * i + pg, 4 * c + t)));
          else
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                         : "=r"(kw[i][0]), "=r"(kw[i][1])
                         : "r"(ka + tile_off<HD>(8 * i + pg, 8 + (t >> 1)) + 8 * (t & 1)));
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
      // V's scale against O's unit, which is the smallest scale so far (up to
      // 2^kNear), or 2^kShift (plain units) once one lies outside 2^+-kFar
      const int ev = (uint32_t)it.w >> 23;
      bool near = abs(ev - eu) <= kNear;
      if (!near && eu != kPlain && (ev < eu || abs(ev - 127) > kFar)) {
        const int to = unit_for(ev);
        const float f = pow2i(eu - (to & 255));
#pragma unroll
        for (int d = 0; d < KS; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[d][i] *= f;
        eu = to;
        near = ev == to;
      }
      const float lr = near ? (float)(ev - eu) : 0.f;

      const float ks = __int_as_float(it.z), f0 = hs[0] * ks, f1 = hs[1] * ks;
      const float x[4][2] = {{sa[0], sa[1]}, {sa[2], sa[3]}, {sb[0], sb[1]}, {sb[2], sb[3]}};
      float p[4][2], top = -INFINITY;
      auto scores = [&]() {
        const float a0 = c2[0] + lr, a1 = c2[1] + lr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i][0] = fmaf(x[i][0], f0, a0);
          p[i][1] = fmaf(x[i][1], f1, a1);
          if (edge) {
            const int pos = p0 + 8 * i + pg;
            if (pos < lo || pos >= len) p[i][0] = p[i][1] = -INFINITY;
          }
        }
      };
      scores();
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(p[i][0], p[i][1]));
      if (__any_sync(0xffffffffu, top > kShift + kSlack + lr)) {
        // a new reference max per head
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const float f = hh ? f1 : f0;
          float mx = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p[i][hh] != -INFINITY) mx = fmaxf(mx, x[i][hh] * f);
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
          const float mn = fmaxf(m2[hh], mx);
          const float corr = mn == -INFINITY ? 1.f : ex2(m2[hh] - mn);
          m2[hh] = mn;
          c2[hh] = kShift - mn;
          l2[hh] *= corr;
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            o[d][hh] *= corr;
            o[d][hh + 2] *= corr;
          }
        }
        scores();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i][0] = ex2(p[i][0]);
        p[i][1] = ex2(p[i][1]);
      }
      const float ir = near ? __uint_as_float((uint32_t)(127 + eu - ev) << 23) : 1.f;
      l2[0] = fmaf((p[0][0] + p[1][0]) + (p[2][0] + p[3][0]), ir, l2[0]);   // this lane's keys
      l2[1] = fmaf((p[0][1] + p[1][1]) + (p[2][1] + p[3][1]), ir, l2[1]);
      // Far blocks: each head's weights are brought to [2^8, 2^9) by its largest
      // one, so that the f16 ones keep their 11 bits however light the block is
      int eh[2] = {0, 0};
      if (!near) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float mx = fmaxf(fmaxf(p[0][hh], p[1][hh]), fmaxf(p[2][hh], p[3][hh]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
          const int e = (int)(__float_as_uint(mx) >> 23) - 127 - 8;      // p is 0, or normal
          eh[hh] = mx > 0.f && mx < INFINITY ? max(e, -126) : 0;
          const float f = __uint_as_float((uint32_t)(127 - eh[hh]) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i][hh] *= f;
        }
      }
      uint32_t pb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 v = __floats2half2_rn(p[i][0], p[i][1]);
        pb[i] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&v));
      }
      // O^T: rows g and g + 8 of 16-dim block d are dims 16d + 2g, 16d + 2g + 1
      const int vr = 8 * (lane >> 3) + perm<HD>(lane & 7);
      auto add_pv = [&](int d, float (&acc)[4]) {
        uint32_t r[4];
        ldsm_x4_t(va + tile_off<HD>(vr, d), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __byte_perm(r[i], 0, 0x3120);
        mma16816_f16(acc, kv8_f16x2(r[0]), kv8_f16x2(r[0] >> 16), kv8_f16x2(r[1]),
                     kv8_f16x2(r[1] >> 16), pb[0], pb[1]);
        mma16816_f16(acc, kv8_f16x2(r[2]), kv8_f16x2(r[2] >> 16), kv8_f16x2(r[3]),
                     kv8_f16x2(r[3] >> 16), pb[2], pb[3]);
      };
      if (near) {
#pragma unroll
        for (int d = 0; d < KS; ++d) add_pv(d, o[d]);
      } else {
        const float f0 = pow2i(ev - (eu & 255) + eh[0]), f1 = pow2i(ev - (eu & 255) + eh[1]);
#pragma unroll
        for (int d = 0; d < KS; ++d) {
          float tt[4] = {0.f, 0.f, 0.f, 0.f};
          add_pv(d, tt);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[d][i] = fmaf(tt[i], i & 1 ? f1 : f0, o[d][i]);
        }
      }
      if (edge) fence_proxy_async_smem();
    }
    __syncwarp();                      // the stage has been read
    if (!ok) break;
    if (n + NST < items) issue(n + NST, s);
    if (++s == NST) {
      s = 0;
      ph ^= 1;
    }
  }
  // after a timeout, wait (bounded) for the copies still in flight
  if (!ok) {
    if (lane == 0) atomicOr(a.err, ERRBIT_TIMEOUT);
    for (int m = n; m < min(items, n + NST); ++m)
      if (!mbar_wait_warp(full + m % NST, (uint32_t)((m / NST) & 1), kPolls)) break;
  }
  __syncthreads();

  // ---- pieces of this thread block: one (pair, head) per warp in turn -------
  constexpr int NV = (HD + 127) / 128;
  const int id = lane < 2 * NW ? s_piece[lane] : -1;   // lane 2w + slot
  const float* mine = nullptr;                         // and where that piece is
  if (id >= 0)
    mine = id & 1 ? reinterpret_cast<const float*>(stages + (size_t)(lane >> 1) * NST * L::STAGE)
                  : ws_warp + (lane >> 1) * PART;
  // one head of a pair from the pieces of lanes `of`: its max, sum and output
  float M, Ls;
  float4 O[NV];
  auto join = [&](bool in, unsigned of, int head) {
    const float m = in ? mine[G * HD + head] : -INFINITY;
    const float l = in ? mine[G * HD + G + head] : 0.f;
    M = warp_max(m);
    const float f = m == -INFINITY ? 0.f : ex2(m - M);
    Ls = warp_sum(l * f);
#pragma unroll
    for (int v = 0; v < NV; ++v) O[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (unsigned r = of; r; r &= r - 1) {
      const int k = __ffs(r) - 1;
      const float fk = __shfl_sync(0xffffffffu, f, k);
      const float* q = reinterpret_cast<const float*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), k)) + head * HD;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int d = 4 * (lane + 32 * v);
        if (d < HD) {
          const float4 y = *reinterpret_cast<const float4*>(q + d);
          O[v].x = fmaf(fk, y.x, O[v].x);
          O[v].y = fmaf(fk, y.y, O[v].y);
          O[v].z = fmaf(fk, y.z, O[v].z);
          O[v].w = fmaf(fk, y.w, O[v].w);
        }
      }
    }
  };
  if (PAIR) {
    // The cluster's pieces: block r gets outputs r n .. (r + 1) n - 1 of all of
    // them, and every block all maxima and sums.
    const int n = G * HD / C;
    float* got = reinterpret_cast<float*>(stages + NW * NST * L::STAGE);   // [C][n]
    float* got_m = got + G * HD;                                           // [C][2][G]
    auto put = [&](const float* p, int r, float v) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(p, r)), "f"(v) : "memory");
    };
    const unsigned of = __ballot_sync(0xffffffffu, id >= 0);
    // every block has started: its shared memory may be written
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int head = w; head < G; head += NW) {
      join(id >= 0, of, head);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int d = 4 * (lane + 32 * v);
        if (d >= HD) continue;
        const float x[4] = {O[v].x, O[v].y, O[v].z, O[v].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = head * HD + d + i, r = e / n;
          put(got + rank * n + e - r * n, r, x[i]);
        }
      }
      if (lane < C) {
        put(got_m + (2 * rank) * G + head, lane, M);
        put(got_m + (2 * rank + 1) * G + head, lane, Ls);
      }
    }
    cluster_sync_all();
    for (int i = tid; i < n; i += kThreads) {
      const int e = rank * n + i, head = e / HD;
      float top = -INFINITY, l = 0.f, x = 0.f;
      for (int c = 0; c < C; ++c) top = fmaxf(top, got_m[2 * c * G + head]);
      for (int c = 0; c < C; ++c) {
        const float m = got_m[2 * c * G + head], f = m == -INFINITY ? 0.f : ex2(m - top);
        l = fmaf(f, got_m[(2 * c + 1) * G + head], l);
        x = fmaf(f, got[c * n + i], x);
      }
      const size_t to = (size_t)own * G * HD + e;
      const float y = l == 0.f ? 0.f : x / l;
      a.out[to] = __float2bfloat16_rn(a.gate ? a.gate[to] * y : y);
    }
    return;
  }
  unsigned left = __ballot_sync(0xffffffffu, id >= 0);
  for (int task = 0; left;) {
    const int pr = __shfl_sync(0xffffffffu, id >> 1, __ffs(left) - 1);
    const bool in = id >= 0 && id >> 1 == pr;
    const unsigned of = __ballot_sync(0xffffffffu, in);
    left &= ~of;
    int nb;
    const int xs = start_of(pr, &nb);
    const bool whole = xs >= X0 && xs + nb <= X1;
    float* part = ws_block + (size_t)(2 * blockIdx.x + (X0 < xs)) * PART;
    for (int head = 0; head < G; ++head, ++task) {
      if (task % NW != w) continue;
      join(in, of, head);
      const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int d = 4 * (lane + 32 * v);
        if (d >= HD) continue;
        if (whole) {
          const size_t to = ((size_t)pr * G + head) * HD + d;
          store_out2(a, to, O[v].x * inv, O[v].y * inv);
          store_out2(a, to + 2, O[v].z * inv, O[v].w * inv);
        } else
          *reinterpret_cast<float4*>(part + head * HD + d) = O[v];
      }
      if (!whole && lane == 0) {
        part[G * HD + head] = M;
        part[G * HD + G + head] = Ls;
      }
    }
  }
}

// Joins the pieces of pairs cut between thread blocks, in order: one block per
// (pair, `heads` of its query heads), blockDim.y = heads x splits warps, each
// with an equal share of one head's pieces, four at a time (one L2 round
// trip), joined through shared memory.
template <int HD, int G>
__global__ void kv8_merge_kernel(const Kv8AttendArgs a, int grid, int heads) {
  constexpr int kMaxW = 16, NV = (HD + 127) / 128, U = 4, PART = kPart<HD, G>;
  __shared__ float sm[kMaxW], sl[kMaxW];
  __shared__ int si[kMaxW][3];
  __shared__ __align__(16) float so[kMaxW][HD];
  // The lengths were written before the attention kernel started, so they
  // may be read before it ends.
  const int H = a.c.Hkv, w = threadIdx.y, lane = threadIdx.x;
  const int pair = blockIdx.x, b = pair / H, h = pair - b * H;
  // blocks before sequence b, of it, and in all
  int v3[3] = {0, 0, 0};
  for (int i = 32 * w + lane; i < a.B; i += 32 * blockDim.y) {
    const int n = visible_blocks(a, i);
    v3[2] += n;
    if (i < b) v3[0] += n;
    if (i == b) v3[1] = n;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    v3[k] = __reduce_add_sync(0xffffffffu, v3[k]);
    if (lane == 0) si[w][k] = v3[k];
  }
  __syncthreads();
  int p0 = 0, nb = 0, total = 0;
  for (int i = 0; i < (int)blockDim.y; ++i) {
    p0 += si[i][0];
    nb += si[i][1];
    total += si[i][2];
  }
  total *= H;
  pdl_wait();
  pdl_trigger();
  if (nb == 0) return;
  const int per = (total + grid - 1) / grid;
  const int xs = p0 * H + h * nb, c0 = xs / per, c1 = (xs + nb - 1) / per;
  if (c0 == c1) return;                // finished in one thread block
  const int SP = blockDim.y / heads;
  const int head = blockIdx.y * heads + w / SP, sp = w % SP;
  const float* parts = reinterpret_cast<const float*>(a.ws);
  const int cnt = c1 - c0 + 1, share = (cnt + SP - 1) / SP;
  const int d0 = c0 + sp * share, d1 = min(c1 + 1, d0 + share);
  float M = -INFINITY, Ls = 0.f;
  float4 O[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) O[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e = d0; e < d1; e += U) {
    float m[U], l[U];
    float4 x[U][NV];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = e + i;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) x[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < d1) {
        // a thread block's first slot holds the pair it starts in
        const float* p = parts + (2 * (size_t)c + (c * per < xs)) * PART;
        m[i] = p[G * HD + head];
        l[i] = p[G * HD + G + head];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int q = 4 * (lane + 32 * v);
          if (q < HD) x[i][v] = *reinterpret_cast<const float4*>(p + head * HD + q);
        }
      }
    }
    float mn = M;
#pragma unroll
    for (int i = 0; i < U; ++i) mn = fmaxf(mn, m[i]);
    const float f0 = M == -INFINITY ? 0.f : ex2(M - mn);
    M = mn;
    Ls *= f0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      O[v] = make_float4(O[v].x * f0, O[v].y * f0, O[v].z * f0, O[v].w * f0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn);
      Ls = fmaf(f, l[i], Ls);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        O[v].x = fmaf(f, x[i][v].x, O[v].x);
        O[v].y = fmaf(f, x[i][v].y, O[v].y);
        O[v].z = fmaf(f, x[i][v].z, O[v].z);
        O[v].w = fmaf(f, x[i][v].w, O[v].w);
      }
    }
  }
  if (lane == 0) {
    sm[w] = M;
    sl[w] = Ls;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (4 * (lane + 32 * v) < HD) *reinterpret_cast<float4*>(&so[w][4 * (lane + 32 * v)]) = O[v];
  __syncthreads();
  const int nthr = 32 * blockDim.y;
  for (int i = w * 32 + lane; i < heads * HD; i += nthr) {
    const int hh = i / HD, d = i - hh * HD;
    float MM = -INFINITY, L = 0.f, S = 0.f;
    for (int k = 0; k < SP; ++k) MM = fmaxf(MM, sm[hh * SP + k]);
    for (int k = 0; k < SP; ++k) {
      const float f = sm[hh * SP + k] == -INFINITY ? 0.f : ex2(sm[hh * SP + k] - MM);
      L = fmaf(f, sl[hh * SP + k], L);
      S = fmaf(f, so[hh * SP + k][d], S);
    }
    const size_t to = ((size_t)pair * G + blockIdx.y * heads) * HD + i;
    const float y = L == 0.f ? 0.f : S / L;
    a.out[to] = __float2bfloat16_rn(a.gate ? a.gate[to] * y : y);
  }
}

// Thread blocks: one per SM (its stages fill the shared memory).
constexpr int kMaxDevices = 64;
int attend_grid() {
  static int n[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  if (!n[dev] &&
      cudaDeviceGetAttribute(&n[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n[dev];
}

// What a device takes of one instantiation, set up once.
struct Fit {
  bool set;
  int clusters[5];                     // at a time, of 1, 2, 4, 8 and 16 thread blocks
};

template <int HD, int G>
Fit fit_of() {
  using L = Att<HD>;
  static std::mutex mu;
  static Fit fit[kMaxDevices];
  int dev = 0;
  std::lock_guard<std::mutex> lock(mu);
  const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices;
  if (known && fit[dev].set) return fit[dev];
  Fit f = {};
  cudaFuncSetAttribute(kv8_attend_kernel<HD, G, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       (int)L::smem(kKv8MaxBatch));
  auto k = kv8_attend_kernel<HD, G, true>;
  const size_t smem = L::smem_pair(G);
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) ==
      cudaSuccess) {
    const bool wide =
        cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int i = 0; i < (wide ? 5 : 4); ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(1 << i, 1, 1);
      cfg.blockDim = dim3(32 * L::NW);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1 << i;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) == cudaSuccess) f.clusters[i] = n;
    }
  }
  cudaGetLastError();
  f.set = true;
  if (known) fit[dev] = f;
  return f;
}

template <int HD, int G>
void attend_t(const Kv8AttendArgs& a, const Kv8Maps& maps, cudaStream_t st) {
  using L = Att<HD>;
  const Fit fit = fit_of<HD, G>();
  const int64_t pairs = (int64_t)a.B * a.c.Hkv;
  const int grid = attend_grid();
  // Few pairs of short sequences: one cluster each, the largest that lets all
  // of them run at once.  It saves 2 to 3 us, but a thread block streams its
  // share of the longest sequence, whatever the others' lengths, and SMs are
  // left over: taken while that share is at most 128 KB more than an SM's share
  // of all pairs, at half the longest length.  (Equal lengths, head_dim 160, 64
  // SMs in clusters: 9.2 for 10.0 us at 96 KB more, 12.3 for 11.7 at 256 KB;
  // head_dim 64: 8.8 for 10.4 us at 100 KB, 12.0 for 12.5 at 200 KB.)
  int i = 4;
  while (i >= 0 && pairs > fit.clusters[i]) --i;
  int64_t blocks = 2ll * a.c.pages_per_seq;            // at most visible
  if (a.window) blocks = std::min<int64_t>(blocks, (a.window - 1) / kKv8Block + 2);
  if (i >= 0 &&
      ((double)blocks / (1 << i) - 0.5 * pairs * blocks / grid) * L::STAGE <= 128 * 1024) {
    launch_k_cluster(kv8_attend_kernel<HD, G, true>, dim3((unsigned)pairs << i),
                     dim3(32 * L::NW), L::smem_pair(G), st, 1 << i, maps, a, 1 << i);
    return;
  }
  launch_k(kv8_attend_kernel<HD, G, false>, dim3(grid), dim3(32 * L::NW), L::smem(a.B), st, maps,
           a, 1);
  // the fewer pairs, the more pieces each may have
  const bool few = pairs <= 64;
  const int heads = few ? 1 : G, warps = few ? (pairs <= 16 ? 16 : 8) : std::max(8, G);
  launch_k(kv8_merge_kernel<HD, G>, dim3((unsigned)pairs, G / heads), dim3(32, warps), 0, st, a,
           grid, heads);
}

template <int HD>
void attend_hd(const Kv8AttendArgs& a, const Kv8Maps& maps, cudaStream_t st) {
  switch (a.G) {
    case 1: attend_t<HD, 1>(a, maps, st); break;
    case 2: attend_t<HD, 2>(a, maps, st); break;
    case 4: attend_t<HD, 4>(a, maps, st); break;
    default: attend_t<HD, 8>(a, maps, st); break;
  }
}

}  // namespace

size_t kv8_attend_ws(int G, int hd) {
  const int nw = hd == 64 ? Att<64>::NW : hd == 128 ? Att<128>::NW : Att<160>::NW;
  return (size_t)(2 + nw) * attend_grid() * ((G * (hd + 2) + 3) & ~3) * sizeof(float);
}

bool make_kv8_maps(const Kv8& c, Kv8Maps* m) {
  const long rows = (long)c.n_pages * c.Hkv * kPage;
  const int w1 = c.hd == 64 ? 64 : 128;
  *m = Kv8Maps{};
  return make_map_bytes(&m->k, c.k, rows, c.hd, w1, kKv8Block) &&
         make_map_bytes(&m->v, c.v, rows, c.hd, w1, kKv8Block) &&
         (c.hd != 160 || (make_map_bytes(&m->k2, c.k, rows, c.hd, 32, kKv8Block) &&
                          make_map_bytes(&m->v2, c.v, rows, c.hd, 32, kKv8Block)));
}

void launch_kv8_attend(const Kv8AttendArgs& a, const Kv8Maps& maps, cudaStream_t st) {
  switch (a.c.hd) {
    case 64: attend_hd<64>(a, maps, st); break;
    case 128: attend_hd<128>(a, maps, st); break;
    default: attend_hd<160>(a, maps, st); break;
  }
}

}  // namespace dory

// The 8-bit K/V cache of one layer: appending rows and one-token attention.
//
// Codes are E4M3 in 64-token pages [n_pages][Hkv][64][hd]; every block of 32
// tokens of a page has one scale per KV head, a power of two s = 2^e, and
// stands for s * e4m3(code).  E4M3 keeps its 3 mantissa bits over 2^15 of
// range, so a power of two loses nothing against an arbitrary scale, and a
// block whose scale grows because a later token is larger is requantised by
// an exact shift (only codes that become subnormal round again).
#include "common.cuh"
#include "kv8.cuh"

namespace dory {

namespace {

// ---------------------------------------------------------------- append ----
// One block of threads per (32-token block, K or V, KV head, sequence): the
// new rows' largest finite magnitude sets the scale
//   s = max(s_old if older tokens are in the block, least 2^e with
//           max <= 448 * 2^e, e >= -126),
// new rows become RNE codes of x / s (NaN stays NaN, infinities saturate),
// older rows are brought to s if it grew; rows behind the new ones are left
// as they are.
constexpr int kAppThreads = 128;

template <int HD>
__global__ void __launch_bounds__(kAppThreads) kv8_append_kernel(Kv8AppendArgs a) {
  constexpr int CH = HD / 8;                   // 8-element chunks per row
  constexpr int N = (kKv8Block * CH + kAppThreads - 1) / kAppThreads;
  __shared__ uint32_t s_amax;
  const int b = blockIdx.z, h = blockIdx.y, kind = blockIdx.x & 1;
  pdl_wait();
  pdl_trigger();
  const int pos = a.pos[b], n = a.n ? a.n[b] : a.T;
  if (n == 0) return;
  if (pos < 0 || n < 0 || n > a.T || pos > a.c.pages_per_seq * kPage - n) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) atomicOr(a.err, ERRBIT_BOUNDS);
    return;
  }
  const int j = pos / kKv8Block + (blockIdx.x >> 1);      // block of the sequence
  const int p0 = j * kKv8Block;
  if (p0 >= pos + n) return;
  const int page = a.c.block_table[(size_t)b * a.c.pages_per_seq + p0 / kPage];
  if (page < 0 || page >= a.c.n_pages) {
    if (threadIdx.x == 0) atomicOr(a.err, ERRBIT_BOUNDS);
    return;
  }
  const size_t ph = (size_t)page * a.c.Hkv + h;
  const int half = (p0 / kKv8Block) & 1;
  uint8_t* codes = (kind ? a.c.v : a.c.k) + (ph * kPage + half * kKv8Block) * HD;
  float* scale = (kind ? a.c.v_scale : a.c.k_scale) + ph * 2 + half;
  const bf16* src = (kind ? a.v : a.k) + b * (kind ? a.vs_b : a.ks_b) +
                    h * (kind ? a.vs_h : a.ks_h);
  const int64_t st = kind ? a.vs_t : a.ks_t;
  const int r0 = max(0, pos - p0), r1 = min(kKv8Block, pos + n - p0);  // new rows

  if (threadIdx.x == 0) s_amax = 0;
  __syncthreads();
  uint4 x[N];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = threadIdx.x + i * kAppThreads, r = e / CH, c = e - r * CH;
    x[i] = make_uint4(0, 0, 0, 0);
    if (r >= r0 && r < r1) {
      x[i] = *reinterpret_cast<const uint4*>(src + (int64_t)(p0 + r - pos) * st + 8 * c);
      mx = max(max(mx, kv8_amax2(x[i].x)), max(kv8_amax2(x[i].y),
               max(kv8_amax2(x[i].z), kv8_amax2(x[i].w))));
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_amax, mx);
  __syncthreads();
  const float s_old = r0 > 0 ? *scale : 0.f;
  const float s = fmaxf(s_old, kv8_scale_for(s_amax));
  const float inv = kv8_inv(s);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = threadIdx.x + i * kAppThreads, r = e / CH, c = e - r * CH;
    if (r >= r0 && r < r1)
      *reinterpret_cast<uint2*>(codes + r * HD + 8 * c) = kv8_encode8(x[i], inv);
    else if (r < r0 && s != s_old)
      kv8_rescale8(codes + r * HD + 8 * c, s_old, inv);
  }
  __syncthreads();                             // every thread has read s_old
  if (threadIdx.x == 0) *scale = s;
}

// ---------------------------------------------------------------- attend ----
// One block per (KV head, sequence); warp w takes keys w, w + 8, ... with a
// running maximum and sum per query head, lanes split head_dim.
constexpr int kAttWarps = 8;

template <int HD, int G>
__global__ void __launch_bounds__(32 * kAttWarps) kv8_attend_kernel(Kv8AttendArgs a) {
  constexpr int D = HD / 32;
  __shared__ float sm[kAttWarps][G], sl[kAttWarps][G], so[kAttWarps][G][HD];
  const int b = blockIdx.y, h = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  int len = a.len[b];
  if (len < 0 || len > a.c.pages_per_seq * kPage) {
    if (h == 0 && threadIdx.x == 0) atomicOr(a.err, ERRBIT_BOUNDS);
    len = 0;
  }
  const int lo = a.window ? max(0, len - a.window) : 0;
  float q[G][D], m[G], l[G], o[G][D];
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    for (int d = 0; d < D; ++d) {
      q[g][d] = __bfloat162float(a.q[b * a.qs_b + (int64_t)(h * G + g) * a.qs_h + lane + 32 * d]);
      o[g][d] = 0.f;
    }
  }
  for (int p = lo + w; p < len; p += kAttWarps) {
    const int page = a.c.block_table[(size_t)b * a.c.pages_per_seq + p / kPage];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) atomicOr(a.err, ERRBIT_BOUNDS);
      continue;
    }
    const size_t ph = (size_t)page * a.c.Hkv + h;
    const int r = p % kPage;
    const float ks = a.c.k_scale[ph * 2 + r / kKv8Block], vs = a.c.v_scale[ph * 2 + r / kKv8Block];
    const uint8_t* k = a.c.k + (ph * kPage + r) * HD;
    const uint8_t* v = a.c.v + (ph * kPage + r) * HD;
    float kf[D], vf[D];
    for (int d = 0; d < D; ++d) {
      kf[d] = kv8_decode(k[lane + 32 * d]) * ks;
      vf[d] = kv8_decode(v[lane + 32 * d]) * vs;
    }
    for (int g = 0; g < G; ++g) {
      float s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(q[g][d], kf[d], s);
      s = warp_sum(s) * a.scale;
      const float mn = fmaxf(m[g], s);
      const float corr = __expf(m[g] - mn), e = __expf(s - mn);
      l[g] = l[g] * corr + e;
      for (int d = 0; d < D; ++d) o[g][d] = o[g][d] * corr + e * vf[d];
      m[g] = mn;
    }
  }
  for (int g = 0; g < G; ++g) {
    if (lane == 0) { sm[w][g] = m[g]; sl[w][g] = l[g]; }
    for (int d = 0; d < D; ++d) so[w][g][lane + 32 * d] = o[g][d];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * HD; i += 32 * kAttWarps) {
    const int g = i / HD;
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int k = 0; k < kAttWarps; ++k) M = fmaxf(M, sm[k][g]);
    for (int k = 0; k < kAttWarps; ++k) {
      const float f = sm[k][g] == -INFINITY ? 0.f : __expf(sm[k][g] - M);
      L = fmaf(f, sl[k][g], L);
      O = fmaf(f, so[k][g][i - g * HD], O);
    }
    a.out[((size_t)b * a.c.Hkv + h) * G * HD + i] = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
  }
}

template <int HD>
void attend_hd(const Kv8AttendArgs& a, cudaStream_t st) {
  const dim3 grid(a.c.Hkv, a.B), block(32 * kAttWarps);
  switch (a.G) {
    case 1: launch_k(kv8_attend_kernel<HD, 1>, grid, block, 0, st, a); break;
    case 2: launch_k(kv8_attend_kernel<HD, 2>, grid, block, 0, st, a); break;
    case 4: launch_k(kv8_attend_kernel<HD, 4>, grid, block, 0, st, a); break;
    default: launch_k(kv8_attend_kernel<HD, 8>, grid, block, 0, st, a); break;
  }
}

}  // namespace

void launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st) {
  // a run of T rows touches at most this many 32-token blocks
  const int nb = (int)(((int64_t)a.T + 2 * kKv8Block - 2) / kKv8Block);
  const dim3 grid(2 * nb, a.c.Hkv, a.B), block(kAppThreads);
  switch (a.c.hd) {
    case 64: launch_k(kv8_append_kernel<64>, grid, block, 0, st, a); break;
    case 128: launch_k(kv8_append_kernel<128>, grid, block, 0, st, a); break;
    default: launch_k(kv8_append_kernel<160>, grid, block, 0, st, a); break;
  }
}

size_t kv8_attend_ws(int, int, int, int) { return 0; }

void launch_kv8_attend(const Kv8AttendArgs& a, cudaStream_t st) {
  switch (a.c.hd) {
    case 64: attend_hd<64>(a, st); break;
    case 128: attend_hd<128>(a, st); break;
    default: attend_hd<160>(a, st); break;
  }
}

}  // namespace dory

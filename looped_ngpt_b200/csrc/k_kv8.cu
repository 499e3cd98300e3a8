// The 8-bit K/V cache of one layer: appending rows.
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

}  // namespace dory

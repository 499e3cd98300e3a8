// The 8-bit K/V cache of one layer: appending rows, and what the model's calls need around it.
//
// Codes are E4M3 in 64-token pages [n_pages][Hkv][64][hd]; every block of 32
// tokens of a page has one scale per KV head, a power of two s = 2^e, and
// stands for s * e4m3(code).  E4M3 keeps its 3 mantissa bits over 2^15 of
// range, so a power of two loses nothing against an arbitrary scale, and a
// block whose scale grows because a later token is larger is requantised by
// an exact shift (only codes that become subnormal round again).
#include "common.cuh"
#include "form_vectors.cuh"
#include "kv8.cuh"
#include "warp_mma.cuh"

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
//
// HBM-bound (2 bytes read, 1 written per element), if few instructions are
// spent on 8 elements: 8 row groups x one 16-byte chunk per thread, so that a
// thread's four chunks are 8 rows apart; magnitudes are compared as packed
// 16-bit integers, and again without infinities and NaN only where there are
// some.  The rows are asked for before the page number has arrived.  24 x up
// to 2048 rows of 8 heads x 128 (151 MB): 29 us, 80% of the copy rate (with 8
// elements per thread in order, f32 comparisons and the rows behind the page
// number: 37 us); 8192 rows of 4 x 160 6.7 us (floor 4.8); one row 1.9 us.
template <int HD, bool PAGED>
__global__ void __launch_bounds__(HD) kv8_append_kernel(Kv8AppendArgs a) {
  constexpr int CH = HD / 8, NT = HD;          // 16-byte chunks per row; threads
  constexpr int N = kKv8Block / 8;             // rows per thread
  __shared__ uint32_t s_amax[NT / 32];
  const int b = blockIdx.z, h = blockIdx.y, kind = blockIdx.x & 1, tid = threadIdx.x;
  const int rt = tid / CH, c = tid - rt * CH;  // rows rt, rt + 8, ..; chunk
  pdl_wait();
  pdl_trigger();
  int pos, n;
  if (PAGED) {
    pos = *a.n_ctx;
    n = row_writes_kv(a.row_loops, b, a.loop_t) ? a.T : 0;
  } else {
    pos = a.pos[b];
    n = a.n ? a.n[b] : a.T;
  }
  if (n == 0) return;
  if (pos < 0 || n < 0 || n > a.T || pos > a.c.pages_per_seq * kPage - n) {
    if (blockIdx.x == 0 && h == 0 && tid == 0) atomicOr(a.err, ERRBIT_BOUNDS);
    return;
  }
  const int j = pos / kKv8Block + (blockIdx.x >> 1);      // block of the sequence
  const int p0 = j * kKv8Block;
  if (p0 >= pos + n) return;
  const int r0 = max(0, pos - p0), r1 = min(kKv8Block, pos + n - p0);  // new rows
  const int half = j & 1;
  const int* entry = a.c.block_table + (size_t)b * a.c.pages_per_seq + p0 / kPage;
  auto unit_of = [&](int page) { return ((size_t)page * a.c.Hkv + h) * 2 + half; };

  uint4 x[N];
  int page;
  auto load = [&](const bf16* src, int64_t st) {          // row r at src + r st
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = rt + 8 * i;
      x[i] = make_uint4(0, 0, 0, 0);
      if (r >= r0 && r < r1) x[i] = *reinterpret_cast<const uint4*>(src + r * st + 8 * c);
    }
  };
  if (PAGED) {
    page = *entry;
    load((kind ? a.v : a.k) + unit_of(page) * kKv8Block * HD, HD);
  } else {
    const int64_t st = kind ? a.vs_t : a.ks_t;
    load((kind ? a.v : a.k) + b * (kind ? a.vs_b : a.ks_b) + h * (kind ? a.vs_h : a.ks_h) +
             (int64_t)(p0 - pos) * st, st);
    page = *entry;
  }
  if (page < 0 || page >= a.c.n_pages) {       // the same for the whole block
    if (tid == 0) atomicOr(a.err, ERRBIT_BOUNDS);
    return;
  }
  const size_t unit = unit_of(page);
  uint8_t* codes = (kind ? a.c.v : a.c.k) + unit * kKv8Block * HD + rt * HD + 8 * c;
  float* scale = (kind ? a.c.v_scale : a.c.k_scale) + unit;
  const float s_old = r0 > 0 ? *scale : 0.f;

  uint32_t mx = 0;                             // two bf16 magnitudes
#pragma unroll
  for (int i = 0; i < N; ++i)
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                               __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
  mx = max(mx & 0xffff0000u, mx << 16);        // the larger, as f32 bits
  if (mx >= 0x7f800000u) {                     // without what is not finite
    mx = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      mx = max(mx, max(max(kv8_amax2(x[i].x), kv8_amax2(x[i].y)),
                       max(kv8_amax2(x[i].z), kv8_amax2(x[i].w))));
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((tid & 31) == 0) s_amax[tid >> 5] = mx;
  __syncthreads();                             // (and s_old has been read)
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) mx = max(mx, s_amax[i]);
  const float s = fmaxf(s_old, kv8_scale_for(mx));
  const float inv = kv8_inv(s);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = rt + 8 * i;
    if (r >= r0 && r < r1) *reinterpret_cast<uint2*>(codes + 8 * i * HD) = kv8_encode8(x[i], inv);
    else if (r < r0 && s != s_old) kv8_rescale8(codes + 8 * i * HD, s_old, inv);
  }
  if (tid == 0) *scale = s;
}

// ------------------------------------------------------- one-token calls ----
// One block per (KV head, sequence), one warp per vector: q_0 .. q_{G-1}, k
// and v from the QKVG partials; then the gate, and the new row's codes.
template <int HD, int G>
__global__ void __launch_bounds__(32 * (G + 2)) kv8_form_kernel(const Kv8FormArgs a) {
  constexpr int NV = G + 2, NT = 32 * NV, CH = HD / 8;
  __shared__ float vec[NV * HD];
  const DecAttnArgs& d = a.d;
  const Dims& dm = d.dm;
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int p = *d.g.n_ctx;
  if (p >= d.g.max_ctx) {                      // uniform over the grid
    if (b == 0 && h == 0 && tid == 0) atomicOr(d.err, ERRBIT_BOUNDS);
    if (h == 0 && tid == 0) a.lens[b] = 0;
    return;
  }
  if (h == 0 && tid == 0) a.lens[b] = p + 1;
  const float* src = d.qkvg + (size_t)b * dm.rows_qkvg;
  const size_t pstride = (size_t)d.B * dm.rows_qkvg;
  const int vs[1] = {w};
  form_vectors<HD, G, 1>(d, src, pstride, h, vs, vec);
  const size_t q0 = (size_t)b * dm.qdim + h * G * HD;
  for (int i = tid; i < G * HD; i += NT) {
    float g = 0.f;
    for (int s = 0; s < d.S; ++s)
      g += src[s * pstride + dm.qdim + 2 * dm.kvdim + h * G * HD + i];
    a.gate[q0 + i] = sigmoidf_(g);
  }
  __syncthreads();
  for (int i = tid; i < G * HD; i += NT) a.q[q0 + i] = __float2bfloat16_rn(vec[i]);

  // the row's codes: warp 0 K, warp 1 V
  if (w > 1 || !row_writes_kv(d.row_loops, b, d.loop_t)) return;
  const int page = a.c.block_table[(size_t)b * a.c.pages_per_seq + p / kPage];
  const size_t ph = (size_t)page * a.c.Hkv + h;
  const int half = (p / kKv8Block) & 1, r0 = p % kKv8Block;
  uint8_t* codes = (w ? a.c.v : a.c.k) + (ph * kPage + half * kKv8Block) * HD;
  float* scale = (w ? a.c.v_scale : a.c.k_scale) + ph * 2 + half;
  const float* x = vec + (G + w) * HD;         // bf16 values
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) {
    const uint32_t u = __float_as_uint(x[lane + 32 * i]) & 0x7fffffffu;
    mx = max(mx, u < 0x7f800000u ? u : 0u);
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  const float s_old = r0 > 0 ? *scale : 0.f;
  const float s = fmaxf(s_old, kv8_scale_for(mx)), inv = kv8_inv(s);
  if (s != s_old)
    for (int e = lane; e < r0 * CH; e += 32) kv8_rescale8(codes + 8 * e, s_old, inv);
  if (lane < CH) {
    auto two = [&](int i) { return kv8_encode2(x[8 * lane + i] * inv, x[8 * lane + i + 1] * inv); };
    *reinterpret_cast<uint2*>(codes + r0 * HD + 8 * lane) =
        make_uint2(two(0) | two(2) << 16, two(4) | two(6) << 16);
  }
  __syncwarp();
  if (lane == 0) *scale = s;
}

// ------------------------------------------------------ multi-token calls ----
// Values of every 32-token block of the first n_ctx + T positions, as bf16.
// Bound by HBM and, nearly as much, by the divisions that find a block: 131072
// tokens of 4 x 160 take 97 us per layer (504 MB, 80% of the copy rate), 8 such
// sequences 806 us (76%), 2048 tokens 8.6 us.
template <int HD>
__global__ void __launch_bounds__(256) kv8_decode_kernel(Kv8 c, int B, const int* n_ctx, int T,
                                                         bf16* k, bf16* v) {
  constexpr int CH = HD / 16;                  // 16-byte chunks per row
  pdl_wait();
  pdl_trigger();
  const int n = min(*n_ctx + T, c.pages_per_seq * kPage);
  const int nb = (n + kKv8Block - 1) / kKv8Block;
  const int64_t total = (int64_t)B * c.Hkv * nb * 2 * (kKv8Block * CH);
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int e = (int)(i % (kKv8Block * CH));
    int64_t r = i / (kKv8Block * CH);
    const int kind = (int)(r & 1);
    r >>= 1;
    const int j = (int)(r % nb);
    r /= nb;
    const int h = (int)(r % c.Hkv), b = (int)(r / c.Hkv);
    const int page = c.block_table[(size_t)b * c.pages_per_seq + (j >> 1)];
    const size_t unit = ((size_t)page * c.Hkv + h) * 2 + (j & 1);
    const uint4 x = *reinterpret_cast<const uint4*>((kind ? c.v : c.k) + unit * (kKv8Block * HD) + 16 * e);
    const float s = (kind ? c.v_scale : c.k_scale)[unit];
    uint4* out = reinterpret_cast<uint4*>((kind ? v : k) + unit * (kKv8Block * HD) + 16 * e);
    auto two = [&](uint32_t u) {
      const uint32_t f = kv8_f16x2(u);
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f));
      return pack_bf16(y.x * s, y.y * s);
    };
    out[0] = make_uint4(two(x.x), two(x.x >> 16), two(x.y), two(x.y >> 16));
    out[1] = make_uint4(two(x.z), two(x.z >> 16), two(x.w), two(x.w >> 16));
  }
}

// Synthetic entries of one (32-token block, K or V, KV head, sequence) per
// block of threads.
__global__ void __launch_bounds__(128) kv8_fill_kernel(Kv8 c, int n, int block, int slot,
                                                       uint64_t seed, float ck, float cv) {
  __shared__ uint32_t s_amax;
  const int j = blockIdx.x >> 1, kind = blockIdx.x & 1, h = blockIdx.y, b = blockIdx.z;
  const int rows = min(kKv8Block, n - j * kKv8Block), CH = c.hd / 8;
  const int page = c.block_table[(size_t)b * c.pages_per_seq + (j >> 1)];
  const size_t unit = ((size_t)page * c.Hkv + h) * 2 + (j & 1);
  uint8_t* codes = (kind ? c.v : c.k) + unit * kKv8Block * c.hd;
  auto value = [&](int r, int d) {
    return __bfloat162float(__float2bfloat16_rn(
        synthetic_kv(kind, block, slot, b, h, j * kKv8Block + r, d, seed, kind ? cv : ck)));
  };
  if (threadIdx.x == 0) s_amax = 0;
  __syncthreads();
  uint32_t mx = 0;
  for (int e = threadIdx.x; e < rows * c.hd; e += 128)
    mx = max(mx, __float_as_uint(value(e / c.hd, e % c.hd)) & 0x7fffffffu);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) atomicMax(&s_amax, mx);
  __syncthreads();
  const float s = kv8_scale_for(s_amax), inv = kv8_inv(s);
  for (int e = threadIdx.x; e < rows * CH; e += 128) {
    const int r = e / CH, d = 8 * (e - r * CH);
    auto two = [&](int i) { return kv8_encode2(value(r, d + i) * inv, value(r, d + i + 1) * inv); };
    *reinterpret_cast<uint2*>(codes + r * c.hd + d) =
        make_uint2(two(0) | two(2) << 16, two(4) | two(6) << 16);
  }
  if (threadIdx.x == 0) (kind ? c.v_scale : c.k_scale)[unit] = s;
}

// Bound by the divisions per 16 bytes: one prefix of 131264 tokens of 4 x 160 to
// 8 sequences takes 0.58 ms per layer (1.34 GB written, 35% of the copy rate).
__global__ void __launch_bounds__(256) kv8_copy_prefix_kernel(Kv8 src, int src_b, Kv8 dst,
                                                              int B_dst, int n) {
  const int CH = src.hd / 16, H = src.Hkv;
  const int64_t total = (int64_t)B_dst * H * n * CH;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int v = (int)(i % CH);
    int64_t r = i / CH;
    const int p = (int)(r % n);
    r /= n;
    const int h = (int)(r % H), b = (int)(r / H);
    const size_t ps = (size_t)src.block_table[(size_t)src_b * src.pages_per_seq + p / kPage] * H + h;
    const size_t pd = (size_t)dst.block_table[(size_t)b * dst.pages_per_seq + p / kPage] * H + h;
    const size_t so = (ps * kPage + p % kPage) * src.hd + 16 * v;
    const size_t dt = (pd * kPage + p % kPage) * src.hd + 16 * v;
    *reinterpret_cast<uint4*>(dst.k + dt) = *reinterpret_cast<const uint4*>(src.k + so);
    *reinterpret_cast<uint4*>(dst.v + dt) = *reinterpret_cast<const uint4*>(src.v + so);
    if (v == 0 && p % kKv8Block == 0) {
      const int half = (p / kKv8Block) & 1;
      dst.k_scale[pd * 2 + half] = src.k_scale[ps * 2 + half];
      dst.v_scale[pd * 2 + half] = src.v_scale[ps * 2 + half];
    }
  }
}

template <int HD>
void append_hd(const Kv8AppendArgs& a, dim3 grid, cudaStream_t st) {
  if (a.pos) launch_k(kv8_append_kernel<HD, false>, grid, dim3(HD), 0, st, a);
  else launch_k(kv8_append_kernel<HD, true>, grid, dim3(HD), 0, st, a);
}

template <int HD>
void form_hd(const Kv8FormArgs& a, cudaStream_t st) {
  const int G = a.d.dm.Hq / a.d.dm.Hkv;
  const dim3 grid(a.d.dm.Hkv, a.d.B), block(32 * (G + 2));
  switch (G) {
    case 1: launch_k(kv8_form_kernel<HD, 1>, grid, block, 0, st, a); break;
    case 2: launch_k(kv8_form_kernel<HD, 2>, grid, block, 0, st, a); break;
    case 4: launch_k(kv8_form_kernel<HD, 4>, grid, block, 0, st, a); break;
    default: launch_k(kv8_form_kernel<HD, 8>, grid, block, 0, st, a); break;
  }
}

}  // namespace

void launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st) {
  // a run of T rows touches at most this many 32-token blocks
  const int nb = (int)(((int64_t)a.T + 2 * kKv8Block - 2) / kKv8Block);
  const dim3 grid(2 * nb, a.c.Hkv, a.B);
  switch (a.c.hd) {
    case 64: append_hd<64>(a, grid, st); break;
    case 128: append_hd<128>(a, grid, st); break;
    default: append_hd<160>(a, grid, st); break;
  }
}

void launch_kv8_form(const Kv8FormArgs& a, cudaStream_t st) {
  switch (a.c.hd) {
    case 64: form_hd<64>(a, st); break;
    case 128: form_hd<128>(a, st); break;
    default: form_hd<160>(a, st); break;
  }
}

void launch_kv8_decode(const Kv8& c, int B, const int* n_ctx, int T, bf16* k, bf16* v,
                       cudaStream_t st) {
  const dim3 grid(148 * 8), block(256);
  switch (c.hd) {
    case 64: launch_k(kv8_decode_kernel<64>, grid, block, 0, st, c, B, n_ctx, T, k, v); break;
    case 128: launch_k(kv8_decode_kernel<128>, grid, block, 0, st, c, B, n_ctx, T, k, v); break;
    default: launch_k(kv8_decode_kernel<160>, grid, block, 0, st, c, B, n_ctx, T, k, v); break;
  }
}

void launch_kv8_fill(const Kv8& c, int B, int n, int block, int slot, uint64_t seed, float ck,
                     float cv, cudaStream_t st) {
  if (n < 1) return;
  const int nb = (n + kKv8Block - 1) / kKv8Block;
  kv8_fill_kernel<<<dim3(2 * nb, c.Hkv, B), 128, 0, st>>>(c, n, block, slot, seed, ck, cv);
}

void launch_kv8_copy_prefix(const Kv8& src, int src_b, const Kv8& dst, int B_dst, int n,
                            cudaStream_t st) {
  if (n < 1) return;
  kv8_copy_prefix_kernel<<<148 * 4, 256, 0, st>>>(src, src_b, dst, B_dst, n);
}

}  // namespace dory

// Host side of the operators that act on caller buffers alone (no model):
// token sampling and the 8-bit K/V cache of one layer.
#include <climits>
#include <cmath>

#include "dory.h"
#include "dory_internal.h"

using namespace dory;

namespace {

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int launched() {
  return cudaGetLastError() == cudaSuccess ? DORY_OK : DORY_ERR_CUDA;
}

int check_kv8(const dory_kv8* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table ||
      c->n_pages < 1 || c->pages_per_seq < 1 || c->batch < 1 || c->n_kv_heads < 1)
    return DORY_ERR_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16) || !aligned(c->block_table, 4))
    return DORY_ERR_ARG;
  // positions are int32; grids take 65535 blocks in y and z
  if (c->pages_per_seq > INT_MAX / kPage || c->batch > 65535 || c->n_kv_heads > 1024)
    return DORY_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 160)
    return DORY_ERR_UNSUPPORTED;
  if (!aligned(c->plan, 64)) return DORY_ERR_ARG;
  return DORY_OK;
}

Kv8 to_kv8(const dory_kv8* c) {
  return Kv8{(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->block_table,
             c->n_pages, c->pages_per_seq, c->n_kv_heads, c->head_dim};
}

bool strides_ok(const int64_t* s, int n) {
  if (!s) return false;
  for (int i = 0; i < n; ++i)
    if (s[i] % 8) return false;
  return true;
}

}  // namespace

extern "C" {

int dory_sample(const float* d_logits, int64_t ld, int B, int V,
                const float* d_temperature, const int32_t* d_top_k,
                const float* d_top_p, const float* d_min_p,
                const float* d_uniform, int32_t* d_tokens, float* d_logprobs,
                void* stream) {
  if (B < 0 || V < 1 || ld < V) return DORY_ERR_ARG;
  if (V > 1 << 30) return DORY_ERR_UNSUPPORTED;     // 32-bit loops over a row
  if (B == 0) return DORY_OK;
  if (!d_logits || !d_uniform || !d_tokens || !aligned(d_logits, 4)) return DORY_ERR_ARG;
  cudaGetLastError();
  launch_sample(SampleArgs{d_logits, ld, B, V, d_temperature, d_top_k, d_top_p, d_min_p,
                           d_uniform, d_tokens, d_logprobs},
                (cudaStream_t)stream);
  return launched();
}

int dory_kv8_append(const dory_kv8* c, const void* d_k, const void* d_v,
                    const int64_t* k_strides, const int64_t* v_strides, int T,
                    const int32_t* d_pos, const int32_t* d_n, void* stream) {
  const int rc = check_kv8(c);
  if (rc) return rc;
  if (T < 0) return DORY_ERR_ARG;
  if (T == 0) return DORY_OK;
  if (!d_k || !d_v || !d_pos || !strides_ok(k_strides, 3) || !strides_ok(v_strides, 3) ||
      !aligned(d_k, 16) || !aligned(d_v, 16) || (int64_t)T > (int64_t)c->pages_per_seq * kPage)
    return DORY_ERR_ARG;
  cudaGetLastError();
  int* err = device_status_word();
  if (!err) return DORY_ERR_CUDA;
  launch_kv8_append(Kv8AppendArgs{to_kv8(c), c->batch, T, (const bf16*)d_k, (const bf16*)d_v,
                                  k_strides[0], k_strides[1], k_strides[2], v_strides[0],
                                  v_strides[1], v_strides[2], d_pos, d_n, err, nullptr,
                                  nullptr, 0},
                    (cudaStream_t)stream);
  return launched();
}

static_assert(sizeof(Kv8Maps) <= DORY_KV8_PLAN_BYTES, "the plan holds the maps");

int dory_kv8_plan(const dory_kv8* c, void* plan) {
  const int rc = check_kv8(c);
  if (rc) return rc;
  if (!plan || !aligned(plan, 64)) return DORY_ERR_ARG;
  if ((int64_t)c->n_pages * c->n_kv_heads * kPage > INT_MAX) return DORY_ERR_UNSUPPORTED;
  return make_kv8_maps(to_kv8(c), (Kv8Maps*)plan) ? DORY_OK : DORY_ERR_CUDA;
}

int dory_kv8_workspace_bytes(const dory_kv8* c, int n_q_heads, int64_t* bytes) {
  const int rc = check_kv8(c);
  if (rc) return rc;
  if (!bytes || n_q_heads < 1 || n_q_heads % c->n_kv_heads) return DORY_ERR_ARG;
  const int G = n_q_heads / c->n_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return DORY_ERR_UNSUPPORTED;
  // block counts and TMA rows are int32, and every sequence has an entry in shared memory
  if (c->batch > kKv8MaxBatch ||
      (int64_t)c->batch * c->pages_per_seq * 2 * c->n_kv_heads > INT_MAX / 2 ||
      (int64_t)c->n_pages * c->n_kv_heads * kPage > INT_MAX)
    return DORY_ERR_UNSUPPORTED;
  *bytes = (int64_t)kv8_attend_ws(G, c->head_dim);
  return DORY_OK;
}

int dory_kv8_attend(const dory_kv8* c, const void* d_q,
                    const int64_t* q_strides, int n_q_heads,
                    const int32_t* d_len, int window, float scale, void* d_out,
                    void* d_ws, int64_t ws_bytes, void* stream) {
  int64_t need = 0;
  const int rc = dory_kv8_workspace_bytes(c, n_q_heads, &need);
  if (rc) return rc;
  if (!d_q || !d_len || !d_out || window < 0 || !std::isfinite(scale) ||
      !strides_ok(q_strides, 2) || !aligned(d_q, 16) || !aligned(d_out, 16))
    return DORY_ERR_ARG;
  if (need > 0 && (!d_ws || !aligned(d_ws, 256))) return DORY_ERR_ARG;
  if (need > ws_bytes) return DORY_ERR_WORKSPACE;
  cudaGetLastError();
  int* err = device_status_word();
  Kv8Maps maps;
  if (!err || (!c->plan && !make_kv8_maps(to_kv8(c), &maps))) return DORY_ERR_CUDA;
  launch_kv8_attend(Kv8AttendArgs{to_kv8(c), c->batch, n_q_heads / c->n_kv_heads,
                                  (const bf16*)d_q, q_strides[0], q_strides[1], d_len, window,
                                  scale, (bf16*)d_out, d_ws, err, nullptr},
                    c->plan ? *(const Kv8Maps*)c->plan : maps, (cudaStream_t)stream);
  return launched();
}

}  // extern "C"

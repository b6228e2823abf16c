// Attention of drafted tokens over a paged cache and the tree of drafts.
// See include/lmoe.h for the contract.
#include <cmath>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

struct AttnArgs {
  lmoe_kv_cache c;
  const uint16_t *q, *k_new, *v_new;
  long long qs, ks, vs;
  const int32_t *offsets, *lens, *table, *pos;
  const uint64_t* mask;
  uint16_t* out;
  float* lse;
  Status* st;
  int B, T, max_n, hq, max_blocks, words, window;
  float scale;
};

// One warp per (row, query head): a pass over what the row sees with a running
// maximum and sum; a lane holds head_dim / 32 elements.
template <int D>
__global__ void __launch_bounds__(128) tree_attn_rows_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= a.hq) return;
  const int kvh = h / (a.hq / a.c.kv_heads);
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int t0 = a.offsets[b], t1 = a.offsets[b + 1], len = a.lens[b];
    if (t0 < 0 || t1 < t0 || t1 > a.T || t1 - t0 > a.max_n || len < 0 ||
        len > (long long)a.max_blocks * a.c.block_size) {
      if (lane == 0) set_error(a.st, LMOE_EDEVICE_CHECK, 211);
      continue;
    }
    for (int t = t0; t < t1; ++t) {
      const int p = a.pos ? max(a.pos[t], len) : len + t - t0;
      float q[E], o[E], m = -INFINITY, l = 0.f;
      for (int e = 0; e < E; ++e) {
        q[e] = bf16_bits_to_f32(a.q[(size_t)t * a.qs + (size_t)h * D + lane * E + e]) * a.scale;
        o[e] = 0.f;
      }
      auto key = [&](const uint16_t* k, const uint16_t* v) {
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += q[e] * bf16_bits_to_f32(k[lane * E + e]);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * f + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * bf16_bits_to_f32(v[lane * E + e]);
      };
      for (int x = a.window > 0 ? max(0, p - a.window + 1) : 0; x < len; ++x) {
        const int id = a.table[(size_t)b * a.max_blocks + x / a.c.block_size];
        if (id < 0 || id >= a.c.n_blocks) {
          if (lane == 0) set_error(a.st, LMOE_EDEVICE_CHECK, 212);
          continue;
        }
        const size_t at = (size_t)id * a.c.block_stride + (size_t)kvh * a.c.head_stride +
                          (size_t)(x % a.c.block_size) * a.c.slot_stride;
        key(a.c.k + at, a.c.v + at);
      }
      for (int j = t0; j < t1; ++j) {
        const int i = j - t0;
        const bool see = a.mask ? (i >> 6) < a.words && (a.mask[(size_t)t * a.words + (i >> 6)] >> (i & 63) & 1) : j <= t;
        if (!see) continue;
        if (a.window > 0 && p - (a.pos ? max(a.pos[j], len) : len + i) >= a.window) continue;
        key(a.k_new + (size_t)j * a.ks + (size_t)kvh * D, a.v_new + (size_t)j * a.vs + (size_t)kvh * D);
      }
      for (int e = 0; e < E; ++e)
        a.out[((size_t)t * a.hq + h) * D + lane * E + e] = f32_to_bf16_bits(l > 0.f ? o[e] / l : 0.f);
      if (a.lse && lane == 0) a.lse[(size_t)t * a.hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
    }
  }
}

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_attn(const lmoe_attn_dims* d, const lmoe_kv_cache* c, bool memory) {
  if (!d) return LMOE_EINVAL;
  const int rc = check_cache(c, memory);
  if (rc) return rc;
  if (d->n_requests < 1 || d->n_requests > 8192 || d->n_tokens < 1 || d->n_tokens > (1 << 20) ||
      d->max_request_tokens < 1 || d->max_request_tokens > 256 || d->q_heads < 1 || d->q_heads % c->kv_heads ||
      d->q_heads / c->kv_heads > 128 || d->max_blocks < 1 || d->max_blocks > (1 << 24) || d->mask_words < 1 ||
      d->mask_words > 4 || d->window < 0 || !(d->scale > 0.f) || !(d->scale < INFINITY))
    return LMOE_EINVAL;
  return LMOE_OK;
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_tree_attention_workspace_bytes(const lmoe_attn_dims* d, const lmoe_kv_cache* c) {
  if (check_attn(d, c, false) != LMOE_OK) return 0;
  return 256;
}

int lmoe_tree_attention(const lmoe_attn_dims* d, const lmoe_kv_cache* c, const uint16_t* q, int64_t q_stride,
                        const uint16_t* k_new, int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                        const int32_t* token_offsets, const int32_t* lens, const int32_t* block_table,
                        const uint64_t* mask, const int32_t* pos, uint16_t* out, float* lse, void* ws,
                        size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  int rc = check_attn(d, c, true);
  if (rc) return rc;
  const int64_t qrow = (int64_t)d->q_heads * c->head_dim, krow = (int64_t)c->kv_heads * c->head_dim;
  if (!al(q, 16) || !al(k_new, 16) || !al(v_new, 16) || !al(out, 16) || !al(token_offsets, 4) || !al(lens, 4) ||
      !al(block_table, 4) || (mask && !al(mask, 8)) || (pos && !al(pos, 4)) || (lse && !al(lse, 4)) ||
      q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
      (mask && 64 * d->mask_words < d->max_request_tokens) || !al(ws, 256))
    return LMOE_EINVAL;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  if (ws_bytes < lmoe_tree_attention_workspace_bytes(d, c)) return LMOE_EWORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Status* st;
  if ((rc = optional_status(ws, ws_bytes, s, &st))) return rc;
  const AttnArgs a = {*c,  q,   k_new, v_new, q_stride,      k_stride,    v_stride,   token_offsets,         lens,
                      block_table, pos, mask,  out,   lse, st, d->n_requests, d->n_tokens, d->max_request_tokens,
                      d->q_heads,  d->max_blocks, d->mask_words, d->window, d->scale};
  return launch_pdl("tree_attn_rows_kernel", dim3(d->n_requests, (d->q_heads + 3) / 4), dim3(128), 0, s,
                    c->head_dim == 64 ? tree_attn_rows_kernel<64> : tree_attn_rows_kernel<128>, a);
}

}  // extern "C"

// Attention of one new token a request over the 8-bit paged cache
// (include/lmoe.h has the contract).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct DecodeArgs {
  lmoe_kv_cache_fp8 c;
  const uint16_t* q;
  long long qs;
  const int32_t *lens, *table;
  uint16_t* out;
  float* lse;
  Status* st;
  int B, G, max_blocks, window, bs_shift;
  float scale_log2;
};

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// One warp a (request, query head), one key at a time.
template <int D>
__global__ void __launch_bounds__(256) decode_attn_kernel(const DecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, hq = a.c.kv_heads * a.G;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= a.B * hq) return;
  const int b = i / hq, qh = i - b * hq, h = qh / a.G, bs = 1 << a.bs_shift;
  const int len = a.lens[b];
  if (len < 0 || len > (long long)a.max_blocks * bs) {
    set_error(a.st, LMOE_EDEVICE_CHECK, 241);
    return;
  }
  constexpr int E = D / 32;
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e) q[e] = bf16_bits_to_f32(a.q[b * a.qs + qh * D + e * 32 + lane]) * a.scale_log2;
  float M = -INFINITY, L = 0.f;
  for (int p = a.window ? max(0, len - a.window) : 0; p < len; ++p) {
    const int block = a.table[(size_t)b * a.max_blocks + (p >> a.bs_shift)], in = p & (bs - 1);
    if (block < 0 || block >= a.c.n_blocks) {
      set_error(a.st, LMOE_EDEVICE_CHECK, 242);
      continue;
    }
    const size_t at = (size_t)block * a.c.block_stride + h * a.c.head_stride + (size_t)in * a.c.slot_stride + lane;
    const size_t sc = (((size_t)block * a.c.kv_heads + h) << a.bs_shift) + in;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], e4m3_to_f32(a.c.k[at + e * 32]), s);
    s = warp_sum(s) * e8m0_to_f32(a.c.k_scale[sc]);
    const float m = fmaxf(M, s), f = exp2f(M - m), w = exp2f(s - m), vs = e8m0_to_f32(a.c.v_scale[sc]);
    L = fmaf(L, f, w);
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], f, w * (vs * e4m3_to_f32(a.c.v[at + e * 32])));
    M = m;
  }
  for (int e = 0; e < E; ++e)
    a.out[((size_t)b * hq + qh) * D + e * 32 + lane] = f32_to_bf16_bits(L == 0.f ? 0.f : o[e] / L);
  if (a.lse && lane == 0) a.lse[(size_t)b * hq + qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_decode(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c, bool memory) {
  if (!d) return LMOE_EINVAL;
  const int rc = check_cache_fp8(c, memory);
  if (rc) return rc;
  if (d->n_requests < 1 || d->n_requests > 8192 || d->q_heads < 1 || d->q_heads % c->kv_heads ||
      d->q_heads / c->kv_heads > 128 || d->max_blocks < 1 || d->max_blocks > (1 << 24) || d->window < 0 ||
      !(d->scale > 0.f) || !(d->scale * kLog2e < INFINITY))
    return LMOE_EINVAL;
  return LMOE_OK;
}

size_t decode_ws(const lmoe_decode_dims*, const lmoe_kv_cache_fp8*, int) { return 256; }

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_decode_attention_fp8_workspace_bytes(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c) {
  if (check_decode(d, c, false) != LMOE_OK) return 0;
  DevInfo di;
  return decode_ws(d, c, dev_info(&di) == LMOE_OK ? di.sms : 152);
}

int lmoe_decode_attention_fp8(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c, const uint16_t* q,
                              int64_t q_stride, const int32_t* lens, const int32_t* block_table, uint16_t* out,
                              float* lse, void* ws, size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  int rc = check_decode(d, c, true);
  if (rc) return rc;
  if (!al(q, 16) || !al(out, 16) || !al(lens, 4) || !al(block_table, 4) || (lse && !al(lse, 4)) ||
      q_stride < (int64_t)d->q_heads * c->head_dim || q_stride % 8 || !al(ws, 256))
    return LMOE_EINVAL;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  if (ws_bytes < decode_ws(d, c, di.sms)) return LMOE_EWORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DecodeArgs a;
  if ((rc = optional_status(ws, ws_bytes, s, &a.st))) return rc;
  a.c = *c;
  a.q = q;
  a.qs = q_stride;
  a.lens = lens;
  a.table = block_table;
  a.out = out;
  a.lse = lse;
  a.B = d->n_requests;
  a.G = d->q_heads / c->kv_heads;
  a.max_blocks = d->max_blocks;
  a.window = d->window;
  a.bs_shift = 4;
  while ((1 << a.bs_shift) < c->block_size) ++a.bs_shift;
  a.scale_log2 = d->scale * kLog2e;
  const int n = a.B * d->q_heads;
  return launch_pdl("decode_attn_kernel", dim3((n + 7) / 8), dim3(256), 0, s,
                    c->head_dim == 64 ? decode_attn_kernel<64> : decode_attn_kernel<128>, a);
}

}  // extern "C"

// Writes to and reads from the 8-bit paged cache (include/lmoe.h has the
// contract).
//
// A row's scale is a power of two, so that x / scale is exact and a code is one
// rounding of x: the codes have one right answer whatever computes them, and
// code * scale is exact in bf16.  A scale with a mantissa would not make the
// codes finer, as their step is relative.
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Two E4M3 codes of a pair of fp32 values (a in the low byte), to nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(b), "f"(a));
  return c;
}

// A row's scale byte from its largest magnitude (15 bits of a bf16).  The magnitude is 1.m * 2^(E - 127) with 7 bits
// of m, and 448 = 1.75 * 2^8: e = E - 135, one more where 1.m > 1.75 (m > 96); the byte is e + 127.  255 for an
// infinity or a NaN.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  return top >= 0x7f80u ? 255u : (uint32_t)max((int)(top >> 7) - 8 + ((top & 127u) > 96u), 0);
}

// Eight bf16 values -> codes.
__device__ __forceinline__ uint2 codes_of(const uint4& x, uint32_t scale) {
  if (scale == 255) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  const float inv = __uint_as_float((254u - scale) << 23);  // 2^-e
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

__device__ __forceinline__ uint32_t top_of(const uint4& x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                              __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// ---------------------------------------------------------------------------
// write
// ---------------------------------------------------------------------------
// A thread takes 16 elements of a row's K and the same of its V; the LP lanes
// of a row find its largest magnitude together.  HBM bounds a prompt: 16384 tokens
// of 8 heads of 128 (101 MB) take 17.7 us, 5690 GB/s, 84% of the copy rate (with
// eight elements a thread 20.0 us); 64 tokens take 1.9 us, a launch.
template <int LP>
__global__ void __launch_bounds__(256)
    kv_write_fp8_kernel(const lmoe_kv_cache_fp8 c, const uint16_t* __restrict__ k_new, long long ks,
                        const uint16_t* __restrict__ v_new, long long vs, int n_rows, const int32_t* __restrict__ src,
                        const int32_t* __restrict__ slots, int n_tokens, int bs_shift, Status* st) {
  pdl_wait();
  pdl_trigger();
  const unsigned x = blockIdx.x * 256u + threadIdx.x, pieces = (unsigned)c.kv_heads * LP;
  const unsigned t = x / pieces, p = x - t * pieces, h = p / LP, d = (p % LP) * 16;
  bool live = t < (unsigned)n_tokens;
  int slot = -1, row = 0;
  if (live) {
    slot = slots[t];
    row = src ? src[t] : (int)t;
    live = slot >= 0;
    if (live && ((slot >> bs_shift) >= c.n_blocks || row < 0 || row >= n_rows)) {
      set_error(st, LMOE_EDEVICE_CHECK, 222);
      live = false;
    }
  }
  uint4 kx[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, vx[2] = {kx[0], kx[0]};
  if (live) {
    const uint4* const kp = reinterpret_cast<const uint4*>(k_new + (size_t)row * ks + (size_t)p * 16);
    const uint4* const vp = reinterpret_cast<const uint4*>(v_new + (size_t)row * vs + (size_t)p * 16);
    kx[0] = __ldcs(kp);
    kx[1] = __ldcs(kp + 1);
    vx[0] = __ldcs(vp);
    vx[1] = __ldcs(vp + 1);
  }
  uint32_t top = max(top_of(kx[0]), top_of(kx[1])) | max(top_of(vx[0]), top_of(vx[1])) << 16;  // both rows' at once
#pragma unroll
  for (int o = LP / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!live) return;
  const uint32_t k_scale = scale_of(top & 0xffffu), v_scale = scale_of(top >> 16);
  const uint2 k0 = codes_of(kx[0], k_scale), k1 = codes_of(kx[1], k_scale);
  const uint2 v0 = codes_of(vx[0], v_scale), v1 = codes_of(vx[1], v_scale);
  const size_t block = (size_t)(slot >> bs_shift), in = (size_t)(slot & ((1 << bs_shift) - 1));
  const size_t to = block * c.block_stride + h * c.head_stride + in * c.slot_stride + d;
  *reinterpret_cast<uint4*>(c.k + to) = make_uint4(k0.x, k0.y, k1.x, k1.y);
  *reinterpret_cast<uint4*>(c.v + to) = make_uint4(v0.x, v0.y, v1.x, v1.y);
  if (d == 0) {
    const size_t at = ((block * c.kv_heads + h) << bs_shift) + in;
    c.k_scale[at] = (uint8_t)k_scale;
    c.v_scale[at] = (uint8_t)v_scale;
  }
}

// ---------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------
constexpr int kReadTokens = 32;  // at most, of a CTA

// The last b in [lo, hi] with offsets[b] <= t, where offsets[lo] <= t.
__device__ __forceinline__ int request_of(const int32_t* offsets, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Eight codes times 2^(scale - 127) as bf16, rounded once.
__device__ __forceinline__ uint4 values_of(const uint2& codes, float scale) {
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w[i / 2] >> (i & 1) * 16)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// A CTA takes `per` tokens: a thread each finds their slots, then all threads move eight codes of K and of V at a
// time, so that a warp's stores follow one another (16 codes a thread, 32 bytes apart: 58.2 us instead of 56.7 for
// the 54000 rows of 16 requests, 331 MB, 5840 GB/s, 86% of the copy rate; two thirds of the bytes are written).  Four
// pieces a thread where that leaves eight CTAs an SM, else one: one request's 1021 rows take 2.8 us with one, 3.4 with
// four; the 16 requests 64.6 and 56.7.
__global__ void __launch_bounds__(256)
    kv_read_fp8_kernel(const lmoe_kv_cache_fp8 c, int B, int n_tokens, int max_blocks,
                       const int32_t* __restrict__ offsets, const int32_t* __restrict__ first,
                       const int32_t* __restrict__ table, uint16_t* __restrict__ k_out, long long ks,
                       uint16_t* __restrict__ v_out, long long vs, int per, int bs_shift, int p_shift, Status* st) {
  __shared__ int s_block[kReadTokens], s_in[kReadTokens];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < B; b += 256)
      if (offsets[b] < 0 || offsets[b + 1] < offsets[b] || offsets[b + 1] > n_tokens)
        set_error(st, LMOE_EDEVICE_CHECK, 231);
  const int t0 = blockIdx.x * per, nt = min(per, n_tokens - t0);
  if ((int)threadIdx.x < nt) {
    const int t = t0 + threadIdx.x;
    int block = -1, in = 0;
    if (offsets[0] <= t && t < offsets[B]) {
      const int b = request_of(offsets, 0, B - 1, t);
      const int begin = offsets[b], end = offsets[b + 1];
      if (begin >= 0 && begin <= t && end > t && end <= n_tokens) {
        const long long p = (long long)(first ? first[b] : 0) + (t - begin);
        const long long page = p >> bs_shift;
        if (p < 0 || page >= max_blocks) {
          set_error(st, LMOE_EDEVICE_CHECK, 232);
        } else {
          block = table[(size_t)b * max_blocks + page];
          in = (int)(p & ((1 << bs_shift) - 1));
          if (block < 0 || block >= c.n_blocks) {
            set_error(st, LMOE_EDEVICE_CHECK, 233);
            block = -1;
          }
        }
      }
    }
    s_block[threadIdx.x] = block;
    s_in[threadIdx.x] = in;
  }
  __syncthreads();
  const unsigned pieces = (unsigned)c.kv_heads << p_shift;  // of 8 elements, of a token
#pragma unroll 2
  for (unsigned x = threadIdx.x; x < (unsigned)nt * pieces; x += 256) {
    const unsigned t = x / pieces, p = x - t * pieces, h = p >> p_shift, d = (p & ((1u << p_shift) - 1)) * 8;
    const int block = s_block[t], in = s_in[t];
    if (block < 0) continue;
    const size_t from = (size_t)block * c.block_stride + h * c.head_stride + (size_t)in * c.slot_stride + d;
    const size_t at = (((size_t)block * c.kv_heads + h) << bs_shift) + in;
    const uint2 kc = *reinterpret_cast<const uint2*>(c.k + from), vc = *reinterpret_cast<const uint2*>(c.v + from);
    const float kf = e8m0_to_f32(c.k_scale[at]), vf = e8m0_to_f32(c.v_scale[at]);
    *reinterpret_cast<uint4*>(k_out + (size_t)(t0 + t) * ks + (size_t)p * 8) = values_of(kc, kf);
    *reinterpret_cast<uint4*>(v_out + (size_t)(t0 + t) * vs + (size_t)p * 8) = values_of(vc, vf);
  }
}

}  // namespace

int check_cache_fp8(const lmoe_kv_cache_fp8* c, bool memory) {
  if (!c || c->kv_heads < 1 || c->kv_heads > 256 || c->head_dim < 1) return LMOE_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return LMOE_EUNSUPPORTED;
  if (!memory) return LMOE_OK;
  if (!al(c->k, 16) || !al(c->v, 16) || !al(c->k_scale, 16) || !al(c->v_scale, 16) || c->n_blocks < 1 ||
      c->block_size < 1)
    return LMOE_EINVAL;
  const int bs = c->block_size;
  if (bs < 16 || bs > 256 || (bs & (bs - 1))) return LMOE_EUNSUPPORTED;
  if ((long long)c->n_blocks * bs > 0x7fffffffll) return LMOE_EUNSUPPORTED;  // slot numbers are 32-bit
  const int64_t st[3] = {c->block_stride, c->head_stride, c->slot_stride};
  for (int64_t x : st)
    if (x < 0 || x % 16) return LMOE_EINVAL;
  if (c->slot_stride < c->head_dim || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->n_blocks > 1 && c->block_stride < c->head_dim))
    return LMOE_EINVAL;
  return LMOE_OK;
}

}  // namespace lmoe

using namespace lmoe;

extern "C" {

int lmoe_kv_write_fp8(const lmoe_kv_cache_fp8* cache, const uint16_t* k_new, int64_t k_stride, const uint16_t* v_new,
                      int64_t v_stride, int32_t n_rows, const int32_t* src, const int32_t* slots, int32_t n_tokens,
                      void* ws, size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  int rc = check_cache_fp8(cache, true);
  if (rc) return rc;
  // distinct slots must not be written over one another, nor keys over values
  if (!rows_apart(cache->block_stride, cache->n_blocks, cache->head_stride, cache->kv_heads, cache->slot_stride,
                  cache->block_size, cache->head_dim) ||
      cache->k == cache->v || cache->k_scale == cache->v_scale)
    return LMOE_EINVAL;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (!al(k_new, 16) || !al(v_new, 16) || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 ||
      n_rows < 1 || n_tokens < 1 || n_tokens > (1 << 20) || (!src && n_tokens > n_rows) || (src && !al(src, 4)) ||
      !al(slots, 4))
    return LMOE_EINVAL;
  const long long total = (long long)n_tokens * (row / 16);
  if (total > 0x7fffffffll) return LMOE_EUNSUPPORTED;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Status* st;
  if ((rc = optional_status(ws, ws_bytes, s, &st))) return rc;
  return launch_pdl("kv_write_fp8_kernel", dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s,
                    cache->head_dim == 64 ? kv_write_fp8_kernel<4> : kv_write_fp8_kernel<8>, *cache, k_new,
                    (long long)k_stride, v_new, (long long)v_stride, n_rows, src, slots, n_tokens,
                    log2_of(cache->block_size), st);
}

int lmoe_kv_read_fp8(const lmoe_kv_cache_fp8* cache, int32_t n_requests, int32_t n_tokens, int32_t max_blocks,
                     const int32_t* token_offsets, const int32_t* first, const int32_t* block_table, uint16_t* k_out,
                     int64_t k_stride, uint16_t* v_out, int64_t v_stride, void* ws, size_t ws_bytes,
                     lmoe_stream_t stream) {
  calls_begin();
  int rc = check_cache_fp8(cache, true);
  if (rc) return rc;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (n_requests < 1 || n_requests > 8192 || n_tokens < 1 || n_tokens > (1 << 20) || max_blocks < 1 ||
      max_blocks > (1 << 24) || !al(token_offsets, 4) || (first && !al(first, 4)) || !al(block_table, 4) ||
      !al(k_out, 16) || !al(v_out, 16) || k_out == v_out || k_stride < row || v_stride < row || k_stride % 8 ||
      v_stride % 8)
    return LMOE_EINVAL;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Status* st;
  if ((rc = optional_status(ws, ws_bytes, s, &st))) return rc;
  const int pieces = (int)(row / 8);
  const int a_cta = (long long)n_tokens * pieces >= 1024ll * 8 * di.sms ? 1024 : 256;
  const int per = std::max(1, std::min(kReadTokens, a_cta / pieces));
  return launch_pdl("kv_read_fp8_kernel", dim3((n_tokens + per - 1) / per), dim3(256), 0, s, kv_read_fp8_kernel,
                    *cache, n_requests, n_tokens, max_blocks, token_offsets, first, block_table, k_out,
                    (long long)k_stride, v_out, (long long)v_stride, per, log2_of(cache->block_size),
                    log2_of(cache->head_dim / 8), st);
}

}  // extern "C"

// Norm of query and key heads and their rotation by position, in one pass over
// the rows (include/lmoe.h has the contract).
//
// Every element is read once and written once and takes some ten operations, so
// HBM bounds it.  A lane holds two runs of four elements of a head: with the
// halves of a head as pairs, four of the first half and the four that they are
// turned with; with neighbours as pairs, eight in a row.  So a pair never leaves
// its lane and the norm is the only thing that lanes exchange.
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a CTA
constexpr int kBatch = 4;       // heads that a lane has under way

struct RopeArgs {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  const uint16_t *q_gain, *k_gain;
  const int32_t *pos, *axis;
  const float* freq;
  long long qs, ks, qos, kos;
  int T, hq, heads, d, rot, axes;
  int tpc, hpc;  // tokens and heads of a CTA
  int norm;
  float eps;
};

// 2^64 turns of one position's step, f / (2 pi), modulo a turn: the product of f (24 bits) with 1 / (2 pi) in
// two doubles, of which the first part's whole turns are dropped.  Then pos * step wraps by itself.
__device__ __forceinline__ uint64_t turn_step(float f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double x = f, p = x * kHi, rest = fma(x, kLo, fma(x, kHi, -p));
  return (uint64_t)__double2ll_rn((p - rint(p)) * 0x1p64) + (uint64_t)__double2ll_rn(rest * 0x1p64);
}

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// LP lanes a head; PAIRS: neighbours are pairs (else the halves' elements).
template <int LP, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int S = kThreads / LP;  // heads that a CTA has in hand at a time
  __shared__ __align__(16) float s_cos[kMaxTokens * 128], s_sin[kMaxTokens * 128];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * a.tpc, h0 = blockIdx.y * a.hpc;
  const int nt = min(a.tpc, a.T - t0), nh = min(a.hpc, a.heads - h0), items = nt * nh;
  const int slot = threadIdx.x / LP, j = threadIdx.x % LP;
  const bool in = 8 * j < a.d, turned = 8 * j < a.rot;
  const int o1 = !PAIRS && turned ? 4 * j : 8 * j, o2 = !PAIRS && turned ? a.rot / 2 + 4 * j : 8 * j + 4;
  const int half = a.rot / 2;

  for (int base = slot; base - slot < items; base += S * kBatch) {
    uint2 x1[kBatch], x2[kBatch];
    int tok[kBatch], head[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * S;
      x1[u] = x2[u] = make_uint2(0, 0);
      tok[u] = a.tpc == 1 ? 0 : (int)((unsigned)i / (unsigned)nh);
      head[u] = h0 + i - tok[u] * nh;
      if (i < items && in) {
        const long long t = t0 + tok[u];
        const uint16_t* const row = head[u] < a.hq ? a.q + t * a.qs + (long long)head[u] * a.d
                                                   : a.k + t * a.ks + (long long)(head[u] - a.hq) * a.d;
        if constexpr (PAIRS) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + o1);
          x1[u] = make_uint2(w.x, w.y);
          x2[u] = make_uint2(w.z, w.w);
        } else {
          x1[u] = *reinterpret_cast<const uint2*>(row + o1);
          x2[u] = *reinterpret_cast<const uint2*>(row + o2);
        }
      }
    }
    if (base == slot) {  // while the first rows are on their way: cosine and sine of the CTA's tokens
      for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = (int)((unsigned)i / (unsigned)half), f = i - t * half;
        const int ax = a.axis ? a.axis[f] : 0;
        float s = 0.f, c = 1.f;
        if (ax >= 0 && ax < a.axes) {
          const long long p = a.pos[(size_t)ax * a.T + t0 + t];
          const uint64_t phase = (uint64_t)p * turn_step(a.freq[f]);
          sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
        }
        s_cos[i] = c;
        s_sin[i] = s;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = base + u * S;
      float v[8];
      const uint32_t w[4] = {x1[u].x, x1[u].y, x2[u].x, x2[u].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack(w[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
      }
      if (a.norm) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum / (float)a.d + a.eps);
        const uint16_t* const gain = head[u] < a.hq ? a.q_gain : a.k_gain;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r;
        if (gain && in) {
          const uint2 g1 = *reinterpret_cast<const uint2*>(gain + o1), g2 = *reinterpret_cast<const uint2*>(gain + o2);
          const uint32_t gw[4] = {g1.x, g1.y, g2.x, g2.y};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 g = unpack(gw[e]);
            v[2 * e] *= g.x;
            v[2 * e + 1] *= g.y;
          }
        }
      }
      if (i < items && in) {
        if (turned) {
          const float4 c4 = *reinterpret_cast<const float4*>(s_cos + tok[u] * half + 4 * j);
          const float4 s4 = *reinterpret_cast<const float4*>(s_sin + tok[u] * half + 4 * j);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float &p = v[PAIRS ? 2 * e : e], &r = v[PAIRS ? 2 * e + 1 : 4 + e];
            const float x = p, y = r;
            p = x * c[e] - y * s[e];
            r = y * c[e] + x * s[e];
          }
        }
        const long long t = t0 + tok[u];
        uint16_t* const row = head[u] < a.hq ? a.q_out + t * a.qos + (long long)head[u] * a.d
                                             : a.k_out + t * a.kos + (long long)(head[u] - a.hq) * a.d;
        const uint2 y1 = make_uint2(pack(v[0], v[1]), pack(v[2], v[3]));
        const uint2 y2 = make_uint2(pack(v[4], v[5]), pack(v[6], v[7]));
        if constexpr (PAIRS) {
          *reinterpret_cast<uint4*>(row + o1) = make_uint4(y1.x, y1.y, y2.x, y2.y);
        } else {
          *reinterpret_cast<uint2*>(row + o1) = y1;
          *reinterpret_cast<uint2*>(row + o2) = y2;
        }
      }
    }
  }
}

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int LP>
int run_rope(RopeArgs a, bool pairs, int sms, cudaStream_t s) {
  constexpr int S = kThreads / LP;
  // a CTA takes what its lanes can have under way at once: some tokens of few heads, or a token of many
  a.tpc = std::max(1, std::min(std::min(kMaxTokens, S * kBatch / a.heads), a.T / (4 * sms)));
  const int gx = (a.T + a.tpc - 1) / a.tpc;
  // few tokens: their heads on several CTAs, down to one for each of a CTA's places
  const int split = std::max(1, std::min((a.heads + S - 1) / S, 2 * sms / gx));
  a.hpc = (a.heads + split - 1) / split;
  const dim3 grid(gx, (a.heads + a.hpc - 1) / a.hpc);
  return launch_pdl("qk_norm_rope_kernel", grid, dim3(kThreads), 0, s,
                    pairs ? qk_norm_rope_kernel<LP, true> : qk_norm_rope_kernel<LP, false>, a);
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" int lmoe_qk_norm_rope(const lmoe_rope_dims* d, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                 int64_t k_stride, const uint16_t* q_gain, const uint16_t* k_gain, const int32_t* pos,
                                 const float* inv_freq, const int32_t* axis, uint16_t* q_out, int64_t q_out_stride,
                                 uint16_t* k_out, int64_t k_out_stride, lmoe_stream_t stream) {
  calls_begin();
  if (!d || d->n_tokens < 1 || d->n_tokens > (1 << 20) || d->q_heads < 0 || d->q_heads > 1024 || d->k_heads < 0 ||
      d->k_heads > 1024 || d->q_heads + d->k_heads < 1 || d->head_dim < 8 || d->rot_dim < 0 ||
      d->rot_dim > d->head_dim || d->n_axes < 1 || d->n_axes > 4 || (d->interleaved & ~1) || (d->norm & ~1) ||
      !(d->eps >= 0.f) || !(d->eps < INFINITY))
    return LMOE_EINVAL;
  if (d->head_dim > 256 || d->head_dim % 8 || d->rot_dim % 8) return LMOE_EUNSUPPORTED;
  const struct {
    int heads;
    const uint16_t *in, *out, *gain;
    int64_t is, os;
  } side[2] = {{d->q_heads, q, q_out, q_gain, q_stride, q_out_stride},
               {d->k_heads, k, k_out, k_gain, k_stride, k_out_stride}};
  for (const auto& x : side) {
    if (!x.heads) continue;
    const int64_t row = (int64_t)x.heads * d->head_dim;
    if (!al(x.in, 16) || !al(x.out, 16) || (x.gain && !al(x.gain, 8)) || x.is < row || x.os < row || x.is % 8 ||
        x.os % 8 || (x.in == x.out && x.is != x.os))
      return LMOE_EINVAL;
  }
  if (d->q_heads && d->k_heads && (q_out == k_out || q_out == k || k_out == q)) return LMOE_EINVAL;
  if (d->rot_dim && (!al(pos, 4) || !al(inv_freq, 4) || (axis && !al(axis, 4)))) return LMOE_EINVAL;
  DevInfo di;
  const int rc = dev_info(&di);
  if (rc) return rc;
  RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.pos = pos;
  a.axis = axis;
  a.freq = inv_freq;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  a.T = d->n_tokens;
  a.hq = d->q_heads;
  a.heads = d->q_heads + d->k_heads;
  a.d = d->head_dim;
  a.rot = d->rot_dim;
  a.axes = d->n_axes;
  a.norm = d->norm;
  a.eps = d->eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool pairs = d->interleaved != 0;
  if (a.d <= 64) return run_rope<8>(a, pairs, di.sms, s);
  return a.d <= 128 ? run_rope<16>(a, pairs, di.sms, s) : run_rope<32>(a, pairs, di.sms, s);
}

// Norm of query and key heads and their rotation by position, in one pass over
// the rows (include/lmoe.h has the contract).
//
// Every element is read once and written once and takes some ten operations, so
// HBM bounds it.  A lane holds two runs of four elements of a head: with the
// halves of a head as pairs, four of the first half and the four that they are
// turned with; with neighbours as pairs, eight in a row.  So a pair never leaves
// its lane, the norm is the only thing that lanes exchange, and the cosines and
// sines of a token are eight registers (as a table in shared memory, made by each
// token's CTA: 184 us instead of 113 for the prompt below).
//
// 16384 tokens of 72 heads of 128 (604 MB) take 98.7 us, 6120 GB/s, 90% of the copy
// rate; one token 2.7 us.  Heads of 80 use 10 of 16 lanes: 5003 tokens of 32 heads
// (51 MB) take 16.7 us, bound by instructions, 2.5 a clock (three heads on 30 lanes,
// with sums over ten lanes, took 4 us more).
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

constexpr int kThreads = 256;
// Units that a warp has under way, twice, and CTAs of an SM: the prompt takes 98.4 us, with three or five units a batch
// 110 and 98.2 (and the smaller video 1.3 and 0.5 us more), with three CTAs of three units 103.
constexpr int kBatch = 4, kCtas = 2;

struct RopeArgs {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  const uint16_t *q_gain, *k_gain;
  const int32_t *pos, *axis;
  const float* freq;
  long long qs, ks, qos, kos;
  int T, hq, hk, d, rot, axes;
  int uq, units;   // units of a token's queries, and all of its units
  int warps;       // among which the units of all tokens are cut
  int norm;
  float eps;
};

// One position's step f / (2 pi) in units of 2^-64 turns, modulo a turn, so that pos * step wraps by itself: f is
// m 2^-e with a whole m below 2^24, and m * 2^128 / (2 pi) shifted right by 64 + e.  (In double precision the steps
// of a launch took the SM's two lanes for it 9 us.)
__device__ __forceinline__ uint64_t turn_step(float f) {
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 2^128 / (2 pi)
  const uint32_t bits = __float_as_uint(f), x = bits >> 23 & 255;
  const uint32_t m = (bits & 0x7fffffu) | (x ? 0x800000u : 0u);
  const int e = 150 - (int)max(x, 1u);  // (below 0 from 2^24 on)
  const uint64_t w1 = m * kHi, more = __umul64hi(m, kLo), low = w1 + more;
  const uint64_t w2 = __umul64hi(m, kHi) + (low < w1);
  const uint64_t r = e <= 0 ? low : e < 64 ? low >> e | w2 << (64 - e) : e < 128 ? w2 >> (e - 64) : 0;
  return bits >> 31 ? 0 - r : r;
}

// 2^-64 turns modulo a turn as half turns, -1 to 1; the lower half goes along as a signed number, so that angles near 0
// of both signs keep their bits (without it the sine of 1e-7 is off by 1%; as one 64-bit conversion one token takes 2.9
// instead of 2.7 us, the video below 16.8 instead of 16.6).
__device__ __forceinline__ float half_turns(uint64_t x) {
  const int lo = (int)(uint32_t)x, hi = (int)((uint32_t)(x >> 32) + ((uint32_t)x >> 31));
  return fmaf((float)lo, 0x1p-63f, (float)hi * 0x1p-31f);
}

// Two fp32 values in one register pair.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 apart(Pair p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair unpack(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(Pair p) {
  const float2 f = apart(p);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ Pair swapped(Pair p) {
  const float2 f = apart(p);
  return pair(f.y, f.x);
}

// LP lanes a head, so that a unit is 32 / LP heads; PAIRS: neighbours are pairs (else the halves' elements); FULL: a head
// fills its lanes.  The units of all tokens, a token's queries first, are cut evenly over the warps.
template <int LP, bool PAIRS, bool FULL>
__global__ void __launch_bounds__(kThreads, kCtas) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int NP = 32 / LP;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, sub = lane / LP, j = lane % LP, half = a.rot / 2;
  const int id = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned all = (unsigned)a.T * (unsigned)a.units;
  const unsigned each = all / (unsigned)a.warps, more = all - each * (unsigned)a.warps;
  unsigned u = (unsigned)id * each + min((unsigned)id, more), left = id < a.warps ? each + ((unsigned)id < more) : 0;
  const int d = FULL ? 8 * LP : a.d;
  const bool in = FULL || 8 * j < d, turned = 8 * j < a.rot;
  const int o1 = !PAIRS && turned ? 4 * j : 8 * j, o2 = !PAIRS && turned ? half + 4 * j : 8 * j + 4;

  // this lane's frequencies and gains
  uint64_t step[4];
  int ax[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int f = 4 * j + e;
    ax[e] = turned && a.axis ? a.axis[f] : 0;
    if ((unsigned)ax[e] >= (unsigned)a.axes) ax[e] = -1;
    step[e] = turned && ax[e] >= 0 ? turn_step(a.freq[f]) : 0;
    ax[e] = max(ax[e], 0);
  }
  uint2 gain[2][2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const uint16_t* const g = side ? a.k_gain : a.q_gain;
    const bool there = g && in;
    gain[side][0] = there ? *reinterpret_cast<const uint2*>(g + o1) : make_uint2(0x3f803f80u, 0x3f803f80u);
    gain[side][1] = there ? *reinterpret_cast<const uint2*>(g + o2) : make_uint2(0x3f803f80u, 0x3f803f80u);
  }
  const float inv_d = 1.f / (float)d;

  // a batch is up to kBatch units of one token's queries (side 0) or keys; the next one's rows are on their way while
  // one is worked on, and with a token's first its positions
  struct Batch {
    unsigned t;
    int side, first, n;  // first unit of the side
    int pos[4];
    uint2 x[kBatch][2];
  };
  Batch next;
  next.t = u / (unsigned)a.units;
  int unit = (int)(u - next.t * (unsigned)a.units);  // of the token, the next to be fetched
  next.n = 0;
  auto fetch = [&] {
    if (unit == a.units) unit = 0, ++next.t;
    next.side = unit >= a.uq;
    next.first = next.side ? unit - a.uq : unit;
    next.n = (int)min((unsigned)min(kBatch, (next.side ? a.units : a.uq) - unit), left);
    if (next.n == 0) return;
    unit += next.n;
    left -= next.n;
#pragma unroll
    for (int e = 0; e < 4; ++e) next.pos[e] = turned ? a.pos[(size_t)ax[e] * a.T + next.t] : 0;
    const int heads = next.side ? a.hk : a.hq;
    const uint16_t* const src = (next.side ? a.k + (size_t)next.t * a.ks : a.q + (size_t)next.t * a.qs) +
                                (size_t)(next.first * NP + sub) * d;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = (next.first + i) * NP + sub;
      next.x[i][0] = next.x[i][1] = make_uint2(0, 0);
      if (i < next.n && h < heads && in) {
        const uint16_t* const row = src + i * NP * d;
        if constexpr (PAIRS) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + o1);
          next.x[i][0] = make_uint2(w.x, w.y);
          next.x[i][1] = make_uint2(w.z, w.w);
        } else {
          next.x[i][0] = *reinterpret_cast<const uint2*>(row + o1);
          next.x[i][1] = *reinterpret_cast<const uint2*>(row + o2);
        }
      }
    }
  };
  fetch();
  // cosines, sines and less the sines of the token, as pairs: of neighbours' angles, or of one angle for a pair
  // (cos, cos), (-sin, sin)
  Pair cc[PAIRS ? 4 : 2], ss[PAIRS ? 4 : 2], minus[PAIRS ? 1 : 2];
  unsigned at = ~0u;  // the token of the cosines
  while (next.n > 0) {
    const Batch now = next;
    fetch();
    if (now.t != at) {
      at = now.t;
      float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {};
      if (turned) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sincospif(half_turns((uint64_t)(long long)now.pos[e] * step[e]), &s[e], &c[e]);
      }
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) cc[e] = pair(c[e], c[e]), ss[e] = pair(-s[e], s[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          cc[e] = pair(c[2 * e], c[2 * e + 1]);
          ss[e] = pair(s[2 * e], s[2 * e + 1]);
          minus[e] = pair(-s[2 * e], -s[2 * e + 1]);
        }
      }
    }
    const uint2 g1 = now.side ? gain[1][0] : gain[0][0], g2 = now.side ? gain[1][1] : gain[0][1];
    const Pair g[4] = {unpack(g1.x), unpack(g1.y), unpack(g2.x), unpack(g2.y)};
    const int heads = now.side ? a.hk : a.hq;
    uint16_t* const dst = (now.side ? a.k_out + (size_t)now.t * a.kos : a.q_out + (size_t)now.t * a.qos) +
                          (size_t)(now.first * NP + sub) * d;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (i >= now.n) break;
      Pair v[4] = {unpack(now.x[i][0].x), unpack(now.x[i][0].y), unpack(now.x[i][1].x), unpack(now.x[i][1].y)};
      if (a.norm) {
        Pair q2 = mul2(v[0], v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) q2 = fma2(v[e], v[e], q2);
        const float2 q = apart(q2);
        float sum = q.x + q.y;
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(mul2(v[e], pair(r, r)), g[e]);
      }
      // (not by an angle of 0 what is not turned: an infinity would make its neighbour NaN; a branch around the pairs, as
      // around the halves, takes the video 17.0 instead of 16.6 us)
      if constexpr (PAIRS) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const Pair x = fma2(v[e], cc[e], mul2(swapped(v[e]), ss[e]));
          v[e] = turned ? x : v[e];
        }
      } else if (turned) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Pair x = v[e], y = v[2 + e];
          v[e] = fma2(x, cc[e], mul2(y, minus[e]));
          v[2 + e] = fma2(y, cc[e], mul2(x, ss[e]));
        }
      }
      const int h = (now.first + i) * NP + sub;
      if (h < heads && in) {
        uint16_t* const row = dst + i * NP * d;
        if constexpr (PAIRS) {
          *reinterpret_cast<uint4*>(row + o1) = make_uint4(pack(v[0]), pack(v[1]), pack(v[2]), pack(v[3]));
        } else {
          *reinterpret_cast<uint2*>(row + o1) = make_uint2(pack(v[0]), pack(v[1]));
          *reinterpret_cast<uint2*>(row + o2) = make_uint2(pack(v[2]), pack(v[3]));
        }
      }
    }
  }
}

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int LP>
int run_rope(RopeArgs a, bool pairs, int sms, cudaStream_t s) {
  constexpr int NP = 32 / LP, kWarps = kThreads / 32;
  a.uq = (a.hq + NP - 1) / NP;
  a.units = a.uq + (a.hk + NP - 1) / NP;
  a.warps = (int)std::min((long long)a.T * a.units, (long long)sms * kCtas * kWarps);
  void (*const kern[2][2])(const RopeArgs) = {{qk_norm_rope_kernel<LP, false, false>, qk_norm_rope_kernel<LP, false, true>},
                                              {qk_norm_rope_kernel<LP, true, false>, qk_norm_rope_kernel<LP, true, true>}};
  return launch_pdl("qk_norm_rope_kernel", dim3((a.warps + kWarps - 1) / kWarps), dim3(kThreads), 0, s,
                    kern[pairs][a.d == 8 * LP], a);
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
  // (only the gains that a norm reads: that of a side without heads may be any pointer)
  a.q_gain = d->norm && d->q_heads ? q_gain : nullptr;
  a.k_gain = d->norm && d->k_heads ? k_gain : nullptr;
  a.pos = pos;
  a.axis = axis;
  a.freq = inv_freq;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  a.T = d->n_tokens;
  a.hq = d->q_heads;
  a.hk = d->k_heads;
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

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

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTile = 32;        // keys of a tile
constexpr int kStages = 3;       // tiles of a warp's ring
constexpr float kShift = 14.f;   // P stands in f16 as p * 2^14, see below

struct DecodeArgs {
  lmoe_kv_cache_fp8 c;
  const uint16_t* q;
  long long qs;
  const int32_t *lens, *table;
  uint16_t* out;
  float* lse;
  Status* status;  // the workspace's status word
  int4* rec;       // [ctas] {request, head group, last CTA of the cut segment or -1, error}
  float2* ml;      // [2 ctas][NQ] maximum and sum of each piece's rows
  float* o;        // [2 ctas][NQ][D] their outputs
  float2* warp_ml; // [ctas kWarps][NQ], pieces that a warp has to put down on its way
  float* warp_o;
  int B, G, groups, max_blocks, window, bs_shift, ctas;
  float scale_log2;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {  // the low two
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return h;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {  // the rest is zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Pieces of a row joined: maximum, sum, and the outputs (of four columns) times it.
struct Sum {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

  __device__ __forceinline__ void add(float2 ml, float4 x) {
    const float top = fmaxf(m, ml.x), mu = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - mu), w = ex2(ml.x - mu) * ml.y;
    m = top;
    l = fmaf(l, f, w);
    o = make_float4(fmaf(w, x.x, o.x * f), fmaf(w, x.y, o.y * f), fmaf(w, x.z, o.z * f), fmaf(w, x.w, o.w * f));
  }
  __device__ __forceinline__ float lse() const { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }
};

// The tiles that a request's positions in sight take, and where the first one begins.
struct Span {
  int lo, len, n;
  __device__ __forceinline__ int p0(int tile) const { return (lo & ~(kTile - 1)) + tile * kTile; }
};

__device__ __forceinline__ Span span_of(const DecodeArgs& a, int len) {
  Span s;
  s.len = len;
  s.lo = a.window && len > a.window ? len - a.window : 0;
  const bool fine = len > 0 && ((unsigned)(len - 1) >> a.bs_shift) < (unsigned)a.max_blocks;
  s.n = fine ? (int)(((unsigned)(len - 1) >> 5) - ((unsigned)s.lo >> 5)) + 1 : 0;
  return s;
}

// A warp's walk over the line of tiles: request by request, in it segment (key head and query group) by segment.
struct Walk {
  int b, seg, tile;
  Span s;
  long long left;

  __device__ __forceinline__ void next(const DecodeArgs& a, int segs) {
    if (--left <= 0) return;
    if (++tile < s.n) return;
    tile = 0;
    if (++seg < segs) return;
    seg = 0;
    do {
      s = span_of(a, a.lens[++b]);
    } while (s.n == 0);  // (there are tiles left, so there is such a request)
  }
};

struct Tile {      // what is kept of a tile until it is computed
  int b, seg;
  int lo, hi;      // rows in sight
  int from;        // its segment starts with it (1), before it in this range (2) or before the range (0)
  int rest;        // tiles of its segment after it
};

// N8: groups of eight query rows that a key's codes are used for.
template <int D, int N8>
struct Cfg {
  static constexpr int kRows = 8 * N8;
  static constexpr int kChunks = D / 16;  // 16-byte pieces of a row
  static constexpr int kCodes = kTile * D;
  static constexpr int kStage = 2 * kCodes + 2 * kTile;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kPiece = kRows * D;  // floats of a piece's output
  static constexpr int kSmem = kRing;
  static_assert(kWarps * (kPiece * 4 + kRows * 8) <= kRing, "the last pieces take the ring's place");
};

// Where 16-byte piece c of row r stands in a tile: rows that are read together lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t place(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ ((r & 1) << 2 | (r >> 1 & 3))) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4);
}

template <int D, int N8>
__global__ void __launch_bounds__(kThreads, 1) decode_attn_kernel(const DecodeArgs a) {
  using C = Cfg<D, N8>;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ unsigned long long s_scan[kWarps];
  __shared__ int s_b[kWarps];
  __shared__ unsigned long long s_at[kWarps];
  __shared__ Tile s_tile[kWarps][4];
  __shared__ int2 s_seg[kWarps][2];  // segments of a warp's pieces: put down on the way, at its range's end
  __shared__ int2 s_flags[kWarps];
  __shared__ int s_rest;
  __shared__ int s_err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int segs = a.c.kv_heads * a.groups, hq = a.c.kv_heads * a.G;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_err = 0;

  // ---- the line of tiles, and this warp's part of it ----
  unsigned long long total, n_ctas, hi;
  long long todo;
  {
    const int run = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * run, b1 = min(a.B, b0 + run);
    unsigned long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const int len = a.lens[b];
      const Span s = span_of(a, len);
      bad |= len != 0 && s.n == 0;
      mine += s.n;
    }
    mine *= segs;
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    unsigned long long before = x - mine;
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    if (bad) atomicCAS(&s_err, 0, 241);
    // as many CTAs as have a tile for each warp
    n_ctas = min((unsigned long long)a.ctas, (total + kWarps - 1) / kWarps);
    const unsigned long long c = blockIdx.x, lo = c < n_ctas ? total * c / n_ctas : total;
    hi = c < n_ctas ? total * (c + 1) / n_ctas : total;
    for (int w = 0; w < kWarps; ++w) {
      const unsigned long long at = lo + (hi - lo) * w / kWarps;
      if (at >= before && at < before + mine) {
        unsigned long long skip = at - before;
        int b = b0;
        for (;; ++b) {
          const unsigned long long there = (unsigned long long)span_of(a, a.lens[b]).n * segs;
          if (skip < there) break;
          skip -= there;
        }
        s_b[w] = b;
        s_at[w] = skip;
      }
    }
    todo = (long long)((hi - lo) * (warp + 1) / kWarps - (hi - lo) * warp / kWarps);
  }
  // requests without positions
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (a.lens[b] != 0) continue;
    for (int i = threadIdx.x; i < hq * D / 8; i += kThreads)
      reinterpret_cast<uint4*>(a.out + (size_t)b * hq * D)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int i = threadIdx.x; i < hq; i += kThreads) a.lse[(size_t)b * hq + i] = -INFINITY;
  }
  __syncthreads();

  Walk walk;
  walk.left = todo;
  bool started = false;  // whether the current segment of the walk starts in this range
  if (walk.left > 0) {
    walk.b = s_b[warp];
    walk.s = span_of(a, a.lens[walk.b]);
    const unsigned long long at = s_at[warp];
    walk.seg = (int)(at / (unsigned)walk.s.n);
    walk.tile = (int)(at - (unsigned long long)walk.seg * walk.s.n);
  }
  uint8_t* const ring = s_ring + warp * kStages * C::kStage;
  const uint32_t ring32 = smem_u32(ring);

  // ---- a tile's way: its pages are looked up, its rows copied, its products formed ----
  int page = 0;  // block number of the page that holds this lane's half of the looked-up tile
  int look_h = 0, look_in = 0, look_lo = 0, look_hi = 0;
  int n_look = 0, n_copy = 0;
  auto look = [&] {  // (walk.left > 0)
    const int p0 = walk.s.p0(walk.tile);
    look_lo = max(walk.s.lo - p0, 0);
    look_hi = min(walk.s.len - p0, kTile);
    look_h = walk.seg / a.groups;
    look_in = p0;
    const int p = min(max(p0 + (lane & 16), p0 + look_lo), p0 + look_hi - 1);
    page = a.table[(size_t)walk.b * a.max_blocks + (p >> a.bs_shift)];
    if (walk.tile == 0) started = true;
    if (lane == 0) {
      Tile d;
      d.b = walk.b;
      d.seg = walk.seg;
      d.lo = look_lo;
      d.hi = look_hi;
      d.from = walk.tile == 0 ? 1 : started ? 2 : 0;
      d.rest = walk.s.n - 1 - walk.tile;
      s_tile[warp][n_look & 3] = d;
    }
    if (walk.tile + 1 == walk.s.n) started = false;
    ++n_look;
    walk.next(a, segs);
  };
  const size_t lane_off = (size_t)(lane / C::kChunks) * a.c.slot_stride + (lane % C::kChunks) * 16;
  constexpr int kStep = 32 / C::kChunks;  // rows that one copy instruction takes
  auto copy = [&] {  // the tile that was looked up
    const uint32_t dst = ring32 + (n_copy % kStages) * C::kStage;
    const int mask = (1 << a.bs_shift) - 1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      int block = __shfl_sync(0xffffffffu, page, half * 16);
      const bool any = look_lo < half * 16 + 16 && look_hi > half * 16;
      bool ok = true;
      if (block < 0 || block >= a.c.n_blocks) {
        if (any && lane == 0) atomicCAS(&s_err, 0, 242);
        block = 0;
        ok = false;
      }
      const int in = (look_in + half * 16) & mask;
      const size_t off = (size_t)block * a.c.block_stride + (size_t)look_h * a.c.head_stride +
                         (size_t)in * a.c.slot_stride + lane_off;
#pragma unroll
      for (int i = 0; i < 16 / kStep; ++i) {
        const int r = half * 16 + i * kStep + lane / C::kChunks;
        const uint32_t to = dst + place<D>(r, lane % C::kChunks);
        const uint32_t bytes = ok && r >= look_lo && r < look_hi ? 16 : 0;
        const size_t from = bytes ? off + (size_t)(i * kStep) * a.c.slot_stride : 0;
        copy16(to, a.c.k + from, bytes);
        copy16(to + C::kCodes, a.c.v + from, bytes);
      }
      // four scale bytes a lane: eight lanes for each half, the first four K
      if ((lane >> 3) == half) {
        const int r = half * 16 + (lane & 3) * 4;
        const uint32_t bytes = ok && r + 4 > look_lo && r < look_hi ? 4 : 0;
        const size_t from =
            bytes ? ((((size_t)block * a.c.kv_heads + look_h) << a.bs_shift) + in + (lane & 3) * 4) : 0;
        const bool v = lane & 4;
        copy4(dst + 2 * C::kCodes + (v ? kTile : 0) + r, (v ? a.c.v_scale : a.c.k_scale) + from, bytes);
      }
    }
    ++n_copy;
  };

  if (walk.left > 0) look();
  for (int i = 0; i < kStages - 1; ++i) {
    if (n_copy < n_look) {
      copy();
      if (walk.left > 0) look();
    }
    copies_end();
  }

  uint32_t qf[N8][D / 16][2];  // the queries' fragments, as f16 times a power of two of each row's
  float q_scale[N8][2];        // what makes a product with them a score to base 2, for this lane's two columns
  float o[C::kChunks][N8][4], M[N8][2], Mo[N8][2], L[N8][2];
  // this warp's pieces, put down on the way (x) and at its range's end (y): 1 there is one, 2 its segment started
  // before the range, 4 it ended
  int2 flags = make_int2(0, 0);
  int bank = 0;

  // the accumulators as outputs: put(row, column, the value and the next column's), and sums(row, M, L)
  auto results = [&](auto&& put, auto&& sums) {
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = L[n][j];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        // O 2^(Mo - M - kShift) / L; the power in two halves, each in range
        const float f = M[n][j] == -INFINITY ? 0.f : ex2(0.5f * (Mo[n][j] - M[n][j] - kShift));
        const float f2 = sum == 0.f ? 0.f : f / sum;
        const int r = n * 8 + 2 * t + j;
        if (g == 0) sums(r, M[n][j], sum);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) put(r, c * 16 + 2 * g, o[c][n][j] * f * f2, o[c][n][2 + j] * f * f2);
      }
  };

  for (; todo > 0; --todo) {
    copies_wait<kStages - 2>();
    __syncwarp();
    const Tile d = s_tile[warp][bank & 3];
    __syncwarp();
    // (the ring's oldest place is free: its tile was computed before the last __syncwarp)
    if (n_copy < n_look) {
      copy();
      if (walk.left > 0) look();
    }
    copies_end();
    const uint8_t* const st = ring + (bank % kStages) * C::kStage;
    const uint32_t st32 = ring32 + (bank % kStages) * C::kStage;
    ++bank;
    const int h = d.seg / a.groups, row0 = (d.seg - h * a.groups) * C::kRows;  // rows of the head's G
    const int rows = min(C::kRows, a.G - row0);
    if (d.from == 1 || bank == 1) {  // a segment's first tile here
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        const int r = n * 8 + g;
        const uint16_t* const src = a.q + (long long)d.b * a.qs + (size_t)(h * a.G + row0 + r) * D + t * 16;
        uint4 w[D / 64][2];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            w[i][j] = r < rows ? reinterpret_cast<const uint4*>(src + i * 64)[j] : make_uint4(0, 0, 0, 0);
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i][j].x & 0x7fff7fffu, w[i][j].y & 0x7fff7fffu),
                                         __vmaxu2(w[i][j].z & 0x7fff7fffu, w[i][j].w & 0x7fff7fffu)));
          }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = act_exponent(top << 16);
        const float up = ldexpf(1.f, e);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x[4] = {w[i][j].x, w[i][j].y, w[i][j].z, w[i][j].w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const __half2 hv = __floats2half2_rn(__uint_as_float(x[m] << 16) * up,
                                                   __uint_as_float(x[m] & 0xffff0000u) * up);
              qf[n][i * 4 + j * 2 + m / 2][m & 1] = *reinterpret_cast<const uint32_t*>(&hv);
            }
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ej = __shfl_sync(0xffffffffu, e, (2 * t + j) * 4);
          q_scale[n][j] = ldexpf(a.scale_log2, -ej);
          M[n][j] = Mo[n][j] = -INFINITY;
          L[n][j] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[c][n][j] = 0.f;
      }
    }

    // ---- scores: S[key][row] = codes . queries ----
    float s[2][N8][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[mt][n][j] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(st + place<D>(mt * 16 + g, i * 4 + t));
        const uint4 y = *reinterpret_cast<const uint4*>(st + place<D>(mt * 16 + g + 8, i * 4 + t));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a0 = e4m3x2_to_f16x2(xs[m]), a2 = e4m3x2_to_f16x2(xs[m] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(ys[m]), a3 = e4m3x2_to_f16x2(ys[m] >> 16);
#pragma unroll
          for (int n = 0; n < N8; ++n) mma_f16(s[mt][n], a0, a1, a2, a3, qf[n][i * 4 + m][0], qf[n][i * 4 + m][1]);
        }
      }
    }
    // ---- to base 2, with the keys' scales; the same with the values' scales for the products with them ----
    float so[2][N8][4];
    const bool edge = d.lo > 0 || d.hi < kTile;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = mt * 16 + k * 8 + g;
        const float ks = e8m0_to_f32(st[2 * C::kCodes + r]);
        const uint32_t vb = st[2 * C::kCodes + kTile + r];
        const float vs = vb == 255 ? NAN : (float)vb - 127.f;
        const bool see = !edge || (r >= d.lo && r < d.hi);
#pragma unroll
        for (int n = 0; n < N8; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& x = s[mt][n][k * 2 + j];
            x = see ? x * q_scale[n][j] * ks : -INFINITY;
            so[mt][n][k * 2 + j] = see ? x + vs : -INFINITY;
          }
      }
    // ---- running maxima ----
    bool more = false;
    float top[N8][2], top_o[N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[n][j] = fmaxf(fmaxf(s[0][n][j], s[0][n][2 + j]), fmaxf(s[1][n][j], s[1][n][2 + j]));
        top_o[n][j] = fmaxf(fmaxf(so[0][n][j], so[0][n][2 + j]), fmaxf(so[1][n][j], so[1][n][2 + j]));
        more |= top[n][j] > M[n][j] || top_o[n][j] > Mo[n][j];
      }
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            top[n][j] = fmaxf(top[n][j], __shfl_xor_sync(0xffffffffu, top[n][j], x));
            top_o[n][j] = fmaxf(top_o[n][j], __shfl_xor_sync(0xffffffffu, top_o[n][j], x));
          }
          const float m = fmaxf(M[n][j], top[n][j]), mo = fmaxf(Mo[n][j], top_o[n][j]);
          L[n][j] *= m == -INFINITY ? 0.f : ex2(M[n][j] - m);
          const float f = mo == -INFINITY ? 0.f : ex2(Mo[n][j] - mo);
          M[n][j] = m;
          Mo[n][j] = mo;
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            o[c][n][j] *= f;
            o[c][n][2 + j] *= f;
          }
        }
    }
    // ---- probabilities: their sums in fp32, and as f16 fragments ----
    uint32_t pf[2][N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n) {
      float mu[2], mo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mu[j] = M[n][j] == -INFINITY ? 0.f : M[n][j];
        mo[j] = (Mo[n][j] == -INFINITY ? 0.f : Mo[n][j]) - kShift;
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float p[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            L[n][j] += ex2(s[mt][n][k * 2 + j] - mu[j]);
            p[j] = ex2(so[mt][n][k * 2 + j] - mo[j]);
          }
          const __half2 hv = __floats2half2_rn(p[0], p[1]);
          pf[mt][n][k] = transposed(*reinterpret_cast<const uint32_t*>(&hv));
        }
    }
    // ---- products with the values: O[d][row] ----
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int c = 0; c < C::kChunks; c += 2) {
        uint32_t r[4];
        ldmatrix_x4_trans(r, st32 + C::kCodes + place<D>(mt * 16 + (lane & 15), c + (lane >> 4)));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // a word holds two keys by two columns: by columns, and each column's pair is a fragment's
          const uint32_t w0 = __byte_perm(r[2 * x], 0, 0x3120), w1 = __byte_perm(r[2 * x + 1], 0, 0x3120);
          const uint32_t a0 = e4m3x2_to_f16x2(w0), a1 = e4m3x2_to_f16x2(w0 >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(w1), a3 = e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
          for (int n = 0; n < N8; ++n) mma_f16(o[c + x][n], a0, a1, a2, a3, pf[mt][n][0], pf[mt][n][1]);
        }
      }

    // ---- the segment's end, or the range's ----
    if (d.rest == 0 && d.from != 0) {
      results(
          [&](int r, int col, float x, float y) {
            if (r < rows)
              *reinterpret_cast<uint32_t*>(a.out + ((size_t)d.b * hq + h * a.G + row0 + r) * D + col) = pack_bf16(x, y);
          },
          [&](int r, float m, float l) {
            if (r < rows && a.lse)
              a.lse[(size_t)d.b * hq + h * a.G + row0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          });
    } else if (d.rest == 0 && todo > 1) {  // started before this range: a piece
      const size_t at = (size_t)blockIdx.x * kWarps + warp;
      results([&](int r, int col, float x, float y) {
        *reinterpret_cast<float2*>(a.warp_o + at * C::kPiece + r * D + col) = make_float2(x, y);
      }, [&](int r, float m, float l) { a.warp_ml[at * C::kRows + r] = make_float2(m, l); });
      flags.x = 1 | 2 | 4;
      if (lane == 0) s_seg[warp][0] = make_int2(d.b, d.seg);
    } else if (todo == 1) {
      flags.y = 1 | (d.from == 0 ? 2 : 0) | (d.rest == 0 ? 4 : 0);
      if (lane == 0) {
        s_seg[warp][1] = make_int2(d.b, d.seg);
        if (warp == kWarps - 1) s_rest = d.rest;
      }
    }
  }

  // ---- the pieces of the warps joined, in the order of the line ----
  copies_wait<0>();
  __syncthreads();  // the ring's place is free
  float* const z_o = reinterpret_cast<float*>(s_ring);
  float2* const z_ml = reinterpret_cast<float2*>(z_o + kWarps * C::kPiece);
  if (flags.y)
    results([&](int r, int col, float x, float y) {
      *reinterpret_cast<float2*>(z_o + warp * C::kPiece + r * D + col) = make_float2(x, y);
    }, [&](int r, float m, float l) { z_ml[warp * C::kRows + r] = make_float2(m, l); });
  if (lane == 0) s_flags[warp] = flags;
  __syncthreads();
  int4 rec = make_int4(0, 0, -1, s_err);
  for (int e = threadIdx.x; e < C::kPiece / 4; e += kThreads) {
    const int r = e / (D / 4);
    Sum sum;
    bool open = false, outer = false;  // outer: the segment started before this CTA's range
    auto end = [&](int2 seg, bool ended) {
      const int h = seg.y / a.groups, row = (seg.y - h * a.groups) * C::kRows + r;
      const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
      if (!outer && ended) {
        if (row < a.G) {
          const size_t at = (size_t)seg.x * hq + h * a.G + row;
          *reinterpret_cast<uint2*>(a.out + at * D + (e % (D / 4)) * 4) =
              make_uint2(pack_bf16(sum.o.x * inv, sum.o.y * inv), pack_bf16(sum.o.z * inv, sum.o.w * inv));
          if (a.lse && e % (D / 4) == 0) a.lse[at] = sum.lse();
        }
      } else {
        const size_t at = (size_t)blockIdx.x * 2 + !outer;
        reinterpret_cast<float4*>(a.o + at * C::kPiece)[e] =
            make_float4(sum.o.x * inv, sum.o.y * inv, sum.o.z * inv, sum.o.w * inv);
        if (e % (D / 4) == 0) a.ml[at * C::kRows + r] = make_float2(sum.m, sum.l);
        if (!outer) rec = make_int4(seg.x, seg.y, (int)(((hi + s_rest) * n_ctas - 1) / total), rec.w);
      }
      open = false;
    };
    int2 seg = make_int2(0, 0);
    for (int w = 0; w < kWarps; ++w) {
      const int2 f = s_flags[w];
      if (f.x) {
        if (!open) sum = Sum(), outer = true;
        const size_t at = (size_t)blockIdx.x * kWarps + w;
        sum.add(a.warp_ml[at * C::kRows + r], reinterpret_cast<const float4*>(a.warp_o + at * C::kPiece)[e]);
        end(s_seg[w][0], true);
      }
      if (f.y) {
        if (!open) sum = Sum(), outer = (f.y & 2) != 0, open = true;
        seg = s_seg[w][1];
        sum.add(z_ml[w * C::kRows + r], reinterpret_cast<const float4*>(z_o + w * C::kPiece)[e]);
        if (f.y & 4) end(seg, true);
      }
    }
    if (open) end(seg, false);
  }
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

// A segment that several CTAs share: its pieces joined in the order of the line, a CTA for the one that its first
// piece is from.  The first CTA also reports what the others found wrong.
template <int D, int N8>
__global__ void __launch_bounds__(256) decode_merge_kernel(const DecodeArgs a) {
  using C = Cfg<D, N8>;
  constexpr int U = 8;  // pieces under way
  __shared__ int s_err;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) s_err = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.ctas; i += blockDim.x)
      if (const int e = a.rec[i].w) atomicMax(&s_err, e);
    __syncthreads();
    if (threadIdx.x == 0) *a.status = Status{s_err ? LMOE_EDEVICE_CHECK : LMOE_OK, s_err};
  }
  const int4 rec = a.rec[blockIdx.x];
  if (rec.z < 0) return;
  const int e = blockIdx.y * blockDim.x + threadIdx.x, r = e / (D / 4);
  const int h = rec.y / a.groups, row = (rec.y - h * a.groups) * C::kRows + r;
  if (row >= a.G) return;
  Sum sum;
  for (int p0 = blockIdx.x; p0 <= rec.z; p0 += U) {
    float2 ml[U];
    float4 o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = min(p0 + u, rec.z);
      const size_t at = (size_t)p * 2 + (p == (int)blockIdx.x);
      ml[u] = a.ml[at * C::kRows + r];
      o[u] = reinterpret_cast<const float4*>(a.o + at * C::kPiece)[e];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p0 + u <= rec.z) sum.add(ml[u], o[u]);
  }
  const float inv = sum.l == 0.f ? 0.f : 1.f / sum.l;
  const size_t at = (size_t)rec.x * a.c.kv_heads * a.G + h * a.G + row;
  *reinterpret_cast<uint2*>(a.out + at * D + (e % (D / 4)) * 4) =
      make_uint2(pack_bf16(sum.o.x * inv, sum.o.y * inv), pack_bf16(sum.o.z * inv, sum.o.w * inv));
  if (a.lse && e % (D / 4) == 0) a.lse[at] = sum.lse();
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

// Query heads of a kv head that one reading of its keys serves, in eights.
int eights(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c) { return d->q_heads / c->kv_heads <= 8 ? 1 : 2; }

struct DecodeWs {
  size_t rec, ml, o, warp_ml, warp_o, total;
};

DecodeWs decode_ws(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c, int ctas) {
  const size_t rows = 8 * (size_t)eights(d, c), row = c->head_dim * sizeof(float);
  DecodeWs w;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = (at + bytes + 255) & ~size_t(255);
    return x;
  };
  w.rec = take(sizeof(int4) * ctas);
  w.ml = take(2 * ctas * rows * sizeof(float2));
  w.o = take(2 * ctas * rows * row);
  w.warp_ml = take(kWarps * ctas * rows * sizeof(float2));
  w.warp_o = take(kWarps * ctas * rows * row);
  w.total = at;
  return w;
}

template <int D, int N8>
int run_decode(const DecodeArgs& a, cudaStream_t s) {
  using C = Cfg<D, N8>;
  static std::atomic<unsigned long long> done{0};
  int rc = allow_smem(done, decode_attn_kernel<D, N8>, C::kSmem);
  if (rc) return rc;
  rc = launch_pdl("decode_attn_kernel", dim3(a.ctas), dim3(kThreads), C::kSmem, s, decode_attn_kernel<D, N8>, a);
  if (rc) return rc;
  constexpr int kUnits = C::kPiece / 4, kBlock = kUnits < 256 ? kUnits : 256;
  return launch_pdl("decode_merge_kernel", dim3(a.ctas, kUnits / kBlock), dim3(kBlock), 0, s,
                    decode_merge_kernel<D, N8>, a);
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_decode_attention_fp8_workspace_bytes(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c) {
  if (check_decode(d, c, false) != LMOE_OK) return 0;
  DevInfo di;
  return decode_ws(d, c, dev_info(&di) == LMOE_OK ? di.sms : 152).total;
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
  const DecodeWs w = decode_ws(d, c, di.sms);
  if (ws_bytes < w.total) return LMOE_EWORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* const base = static_cast<char*>(ws);
  DecodeArgs a;
  a.c = *c;
  a.q = q;
  a.qs = q_stride;
  a.lens = lens;
  a.table = block_table;
  a.out = out;
  a.lse = lse;
  a.status = reinterpret_cast<Status*>(base);
  a.rec = reinterpret_cast<int4*>(base + w.rec);
  a.ml = reinterpret_cast<float2*>(base + w.ml);
  a.o = reinterpret_cast<float*>(base + w.o);
  a.warp_ml = reinterpret_cast<float2*>(base + w.warp_ml);
  a.warp_o = reinterpret_cast<float*>(base + w.warp_o);
  a.B = d->n_requests;
  a.G = d->q_heads / c->kv_heads;
  const int n8 = eights(d, c);
  a.groups = (a.G + 8 * n8 - 1) / (8 * n8);
  a.max_blocks = d->max_blocks;
  a.window = d->window;
  a.bs_shift = 4;
  while ((1 << a.bs_shift) < c->block_size) ++a.bs_shift;
  a.ctas = di.sms;
  a.scale_log2 = d->scale * kLog2e;
  if (c->head_dim == 64) return n8 == 1 ? run_decode<64, 1>(a, s) : run_decode<64, 2>(a, s);
  return n8 == 1 ? run_decode<128, 1>(a, s) : run_decode<128, 2>(a, s);
}

}  // extern "C"

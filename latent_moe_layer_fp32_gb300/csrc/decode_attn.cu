// Attention of one new token a request over the 8-bit paged cache
// (include/lmoe.h has the contract).
//
// A key head's codes are read once for up to 16 query heads: 2 D + 2 bytes a
// position for 4 D flops a query head, so HBM bounds it up to 8 of them, and the
// arithmetic from there on.  What follows from that:
//  - Keys (and the values' columns) are the 16 rows of a tensor-core product and
//    the query heads its 8 columns, so that 8 heads waste nothing.  Codes become
//    f16 exactly on their way from shared memory into the fragments; queries
//    are f16 after a power of two of their row, exactly down to 2^-31 of its
//    largest element.  A product takes 8 clocks of an SM
//    quarter and 23% of the tensor pipe's time: tcgen05 would have to read
//    queries and probabilities as further E4M3 parts from shared memory, for
//    a pipe that is not what bounds.  (Products of E4M3 codes with queries in
//    two E4M3 parts, which need no conversion of the keys, were slower: 70.2
//    instead of 67.8 us for 64 requests of 512 to 8191 positions.)
//  - The scales are powers of two for a whole row, so K's multiply a score, and
//    V's are an exponent that is added to the probability's: no element is
//    multiplied.  The sums O have a running maximum of their own for that, as a
//    key with small values may hold all of a row's weight.
//  - The tiles of all requests and heads stand in one line that is cut evenly
//    over all warps, with no host knowledge of lengths; a segment that is cut
//    leaves partial sums, joined in the order of the line (by the CTA in shared
//    memory, across CTAs by a second kernel), so results do not depend on timing.
//  - A warp has a ring of tiles of its own and meets the others only at the end.
//    Whole tiles come by bulk tensor copies, evict-first (16-byte copies by
//    lanes: 75 us instead of 68; without the hint 70 instead of 65); edges come by
//    lanes, which fill what is out of sight with zeros, so that NaN there has no
//    effect.  8 warps and 3 tiles with 128 columns, 12 and 2 with 64; a number
//    that is no multiple of 4 leaves the SM's quarters uneven (10 warps: 75 us).
//
// 64 requests of 512 to 8191 positions (365 MB) take 66.2 us, 5510 GB/s; 256 requests
// of 20 to 8191 (814 MB) 138 us, 5900 GB/s, 87% of the copy rate; one request at
// 131071 positions 50.8 us, at 1021 8.8 us.  About 8 us of each are start-up (launch,
// lengths, page numbers, first copy: 4.5), the join and the second kernel (3.5).  16
// heads a key head: 90 us for the 64 requests, bound by the arithmetic's latency (two
// warps an SM quarter, 1.7 instructions a clock, more than half of the stalls waits
// of fixed length).
#include <algorithm>
#include <atomic>
#include <cstring>
#include <utility>

#include "common.cuh"
#include "launch.cuh"
#include "tmap.cuh"

namespace lmoe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

// What a segment's end weighs in the cut, in tiles: 256 requests of 20 to 8191 positions take 168 us with 0, 146 with 1,
// 137 with 2, 139 with 4; 256 of 3 to 200 positions 21.5, 21.0, 21.4 and 22.6.
constexpr int kEnd = 2;
// The base of a row's powers is its largest score when it last moved.  It moves again where a power would pass
// 2^kSlackM, which fp32 sums do not mind, or one with its value's exponent 2^kSlackE, which keeps f16, where they stand
// times 2^kShift, below 2^16.  (Where it followed every new maximum, 64 requests of 16
// heads a key head took 88 us instead of 81.)
constexpr float kSlackM = 8.f, kSlackE = 1.9f, kShift = 14.f;

struct DecodeArgs {
  lmoe_kv_cache_fp8 c;
  const uint16_t* q;
  long long qs;
  const int32_t *lens, *table;
  uint16_t* out;
  float* lse;
  Status* status;  // the workspace's status word
  int4* rec;        // [ctas] {request, key head and query group, last CTA of a cut segment or -1, error}
  float2* ml;       // [2 ctas][rows] maximum and sum of each piece's rows
  float* o;         // [2 ctas][rows][D] their outputs
  float2* warp_ml;  // [ctas][warps][rows] and [D], pieces that a warp has to put down on its way
  float* warp_o;
  int B, G, groups, max_blocks, window, bs_shift, ctas;
  float scale_log2;
};

__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 to 127

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four codes as two pairs of f16.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n cvt.rn.f16x2.e4m3x2 %0, x;\n cvt.rn.f16x2.e4m3x2 %1, y;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

template <int DST>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {  // the rest is zero
  asm volatile("cp.async.cg.shared.global [%0 + %3], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(DST)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int OFF>
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF)
               : "memory");
}
template <int OFF>
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(OFF)
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
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Pieces of a row joined: maximum, sum, and the outputs (of four columns) times it.
struct Sum {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

  __device__ __forceinline__ void add(float w, float4 x) {
    l += w;
    o = make_float4(fmaf(w, x.x, o.x), fmaf(w, x.y, o.y), fmaf(w, x.z, o.z), fmaf(w, x.w, o.w));
  }
  __device__ __forceinline__ float lse() const { return l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2; }
};

// x / y; a 32-bit division where that is enough, as 64-bit ones take hundreds of clocks.
__device__ __forceinline__ unsigned long long quot(unsigned long long x, unsigned long long y) {
  return (x | y) >> 32 ? x / y : (unsigned long long)((unsigned)x / (unsigned)y);
}

// An even cut of n things into parts.
struct Cut {
  unsigned long long each, more;  // `more` parts have one more
  __device__ __forceinline__ Cut(unsigned long long n, unsigned parts) : each(quot(n, parts)), more(n - each * parts) {}
  __device__ __forceinline__ unsigned long long first(unsigned i) const {
    return i * each + min((unsigned long long)i, more);
  }
};

// The tiles of KT keys that a request's positions in sight take, and where the first one begins.
template <int KT>
struct Span {
  int lo, len, n;
  __device__ __forceinline__ int p0(int tile) const { return (lo & ~(KT - 1)) + tile * KT; }
};

template <int KT>
__device__ __forceinline__ Span<KT> span_of(const DecodeArgs& a, int len) {
  Span<KT> s;
  s.len = len;
  s.lo = a.window && len > a.window ? len - a.window : 0;
  const bool fine = len > 0 && ((unsigned)(len - 1) >> a.bs_shift) < (unsigned)a.max_blocks;
  s.n = fine ? (int)((unsigned)(len - 1) / KT - (unsigned)s.lo / KT) + 1 : 0;
  return s;
}

// A warp's walk over the line of tiles: request by request, in it key head by key head, in it group by group of
// query rows.  Behind each of these segments the line has room for what its end costs, as many tiles as `end`.
template <int KT>
struct Walk {
  int b, h, group, tile, end;
  Span<KT> s;
  long long left;  // of the range, from the tile on

  __device__ __forceinline__ bool last() const { return tile == s.n - 1; }  // of its segment
  __device__ __forceinline__ long long after() const { return left - (last() ? 1 + end : 1); }
  __device__ __forceinline__ void next(const DecodeArgs& a) {
    left = after();
    if (++tile >= s.n && left > 0) segment(a);
  }
  __device__ __forceinline__ void segment(const DecodeArgs& a) {
    tile = 0;
    if (++group < a.groups) return;
    group = 0;
    if (++h < a.c.kv_heads) return;
    h = 0;
    do {
      s = span_of<KT>(a, a.lens[++b]);
    } while (s.n == 0);  // (there is something left of the range, so there is such a request)
  }
};

// N8: groups of eight query rows that a key's codes are used for; W warps; S tiles of KT keys in a warp's ring.  Tiles
// of 8 KB: with 64 columns, 64 keys instead of 32 make more of a tile's steps independent (window layer 25.6 instead of
// 27.7 us, 8 heads a key head 39.9 instead of 46.7 us).
template <int D, int N8>
struct Cfg {
  static constexpr int W = D == 64 && N8 == 1 ? 12 : 8, KT = 4096 / D, S = D == 128 && N8 == 1 ? 3 : 2;
  static constexpr int kThreads = 32 * W;
  static constexpr int kRows = 8 * N8;
  static constexpr int kChunks = D / 16;  // 16-byte pieces of a row
  static constexpr int kCodes = KT * D;
  static constexpr int kStage = 2 * kCodes;
  static constexpr int kRing = W * S * kStage;
  static constexpr int kPiece = kRows * D;  // floats of a piece's output
  // with 16 query rows, their fragments stand in shared memory: registers are what bounds the number of warps
  static constexpr bool kQueriesInSmem = N8 == 2;
  static constexpr int kQueries = kQueriesInSmem ? W * N8 * kChunks * 32 * 8 : 0;
  static constexpr int kSmem = kRing + kQueries + 1024;  // (the ring starts on 1024 bytes, the swizzle's period)
  static_assert(8192 <= 32 * kThreads, "the most requests: no run has more than a warp's lanes");
  static_assert(kPiece * 4 <= S * kStage, "a warp's last piece takes its ring's place");
  static_assert(KT == 32 || KT == 64, "whole warps of keys");
};

// The 16-byte piece c of a tile's row r stands at r * D + ((c ^ swizzle(r)) << 4): the eight rows of one 8x8 matrix
// lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t swizzle(int r) {
  return D == 128 ? r & 7 : r >> 1 & 3;
}

// A loop over constants: the body gets them as types.
template <typename F, int... I>
__device__ __forceinline__ void unrolled_by(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  unrolled_by(f, std::make_integer_sequence<int, N>());
}

template <int D, int N8>
__global__ void __launch_bounds__(Cfg<D, N8>::kThreads, 1)
    decode_attn_kernel(const DecodeArgs a, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D, N8>;
  constexpr int W = C::W, KT = C::KT, MT = KT / 16;
  extern __shared__ uint8_t s_dynamic[];
  uint8_t* const s_ring = s_dynamic + (-smem_u32(s_dynamic) & 1023u);
  __shared__ uint64_t s_full[W][C::S];
  __shared__ float2 s_key[W][KT];  // of a tile's keys: the key's scale, the value's exponent
  __shared__ __align__(16) uint8_t s_scale[W][C::S][2 * KT];  // of the ring's tiles: K's, V's
  __shared__ unsigned long long s_scan[W], s_before[C::kThreads];
  __shared__ unsigned s_live[W];
  // a warp's pieces, put down on the way and at its range's end: {request, key head, first query row, flags}
  __shared__ int4 s_seg[W][2];
  __shared__ float2 s_ml[W][C::kRows];
  __shared__ int s_last, s_err;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int hq = a.c.kv_heads * a.G;
  auto piece_at = [&](int w) { return reinterpret_cast<float*>(s_ring + w * C::S * C::kStage); };
  // (what needs nothing of the launch before, while that one ends)
  if (threadIdx.x == 0) s_err = s_last = 0;
  if (lane < 2) s_seg[warp][lane] = make_int4(0, 0, 0, 0);
  if (lane < C::S) mbar_init(&s_full[warp][lane], 1);
  fence_barrier_init();
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  // ---- the line of tiles, and this warp's part of it ----
  unsigned long long total, hi;
  unsigned n_ctas;
  Walk<KT> walk;
  bool at_end;  // this warp's range ends with the CTA's
  {
    // runs of requests, a lane each; up to 256 requests every warp looks at all of them, else the CTA's warps share them
    const bool alone = a.B <= 256;
    const int run = alone ? (a.B + 31) / 32 : (a.B + C::kThreads - 1) / C::kThreads;
    const int b0 = (alone ? lane : (int)threadIdx.x) * run, b1 = min(a.B, b0 + run);
    const unsigned segs = (unsigned)(a.c.kv_heads * a.groups);
    unsigned long long tiles = 0;
    unsigned live = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const int len = a.lens[b];
      const Span<KT> s = span_of<KT>(a, len);
      bad |= len != 0 && s.n == 0;
      tiles += s.n;
      live += s.n != 0;
    }
    unsigned long long x = tiles;
    unsigned y = live;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x1 = __shfl_up_sync(0xffffffffu, x, o);
      const unsigned y1 = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += x1, y += y1;
    }
    unsigned long long tiles_before = x - tiles, all = __shfl_sync(0xffffffffu, x, 31);
    unsigned live_before = y - live, all_live = __shfl_sync(0xffffffffu, y, 31);
    if (!alone) {
      if (lane == 31) {
        s_scan[warp] = x;
        s_live[warp] = y;
      }
      __syncthreads();
      all = all_live = 0;
      for (int w = 0; w < W; ++w) {
        if (w < warp) tiles_before += s_scan[w], live_before += s_live[w];
        all += s_scan[w];
        all_live += s_live[w];
      }
    }
    if (bad) atomicCAS(&s_err, 0, 241);
    all *= segs;
    // what a segment's end weighs: no more than a warp has tiles
    walk.end = (int)min((unsigned long long)kEnd, quot(all, (unsigned)(a.ctas * W)));
    total = all + (unsigned long long)all_live * segs * walk.end;
    const unsigned long long before = (tiles_before + (unsigned long long)live_before * walk.end) * segs;
    // as many CTAs as have a tile for each warp
    n_ctas = (unsigned)min((unsigned long long)a.ctas, (all + W - 1) / W);
    const unsigned c = blockIdx.x;
    unsigned long long lo = total;
    hi = total;
    if (c < n_ctas) {
      const Cut ctas(total, n_ctas);
      lo = ctas.first(c);
      hi = ctas.first(c + 1);
    }
    const Cut warps(hi - lo, W);
    const unsigned long long at = lo + warps.first(warp);
    walk.left = (long long)(warps.each + ((unsigned)warp < warps.more));
    at_end = lo + warps.first(warp + 1) == hi;
    if (!alone) {
      s_before[threadIdx.x] = before;
      __syncthreads();
    }
    if (walk.left > 0) {
      // the last run of requests that begins at or before this warp's range, and in it the request: a lane each
      int owner = -1;
      unsigned long long skip;
      if (alone) {
        owner += __popc(__ballot_sync(0xffffffffu, before <= at));
        skip = at - __shfl_sync(0xffffffffu, before, owner);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) owner += __popc(__ballot_sync(0xffffffffu, s_before[i * 32 + lane] <= at));
        skip = at - s_before[owner];
      }
      walk.b = owner * run;
      if (run > 1) {
        const int b = walk.b + lane;
        const int n = lane < run && b < a.B ? span_of<KT>(a, a.lens[b]).n : 0;
        const unsigned long long mine = n ? (unsigned long long)(n + walk.end) * segs : 0;
        unsigned long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const int i = __ffs(__ballot_sync(0xffffffffu, x > skip)) - 1;
        skip -= __shfl_sync(0xffffffffu, x - mine, i);
        walk.b += i;
      }
      walk.s = span_of<KT>(a, a.lens[walk.b]);
      const int size = walk.s.n + walk.end, seg = (int)quot(skip, size);
      walk.tile = (int)(skip - (unsigned long long)seg * size);
      walk.h = seg / a.groups;
      walk.group = seg - walk.h * a.groups;
      if (walk.tile >= walk.s.n) {  // behind a segment's tiles
        walk.left -= size - walk.tile;
        if (walk.left > 0) walk.segment(a);
      }
    }
  }
  Walk<KT> ahead = walk;  // walks in front and looks pages up
  const uint32_t ring32 = smem_u32(s_ring + warp * C::S * C::kStage), scale32 = smem_u32(s_scale[warp]);

  // ---- a tile's way: its pages are looked up, its rows copied, its products formed ----
  constexpr int kLanes = 32 / MT;  // a group of lanes for each 16 keys
  // block numbers of 512 positions of a request, a lane for 16: those from the tile `pages_tile` on
  int pages = 0, pages_b = -1, pages_tile = 0;
  int look_h = 0, look_in = 0, look_lo = 0, look_hi = 0, look_part = 0;  // (its first 16 keys' lane of `pages`)
  bool looked = false;  // a tile has been looked up and not copied
  int to_stage = 0;
  auto look = [&] {
    looked = ahead.left > 0;
    if (!looked) return;
    const int p0 = ahead.s.p0(ahead.tile);
    look_lo = max(ahead.s.lo - p0, 0);
    look_hi = min(ahead.s.len - p0, KT);
    look_h = ahead.h;
    if (ahead.tile == 0) {  // its segment's queries will be wanted soon: 128 bytes a lane
      const int r = ahead.group * C::kRows + lane * 64 / D;
      if (r < a.G && lane * 64 < C::kPiece)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + (long long)ahead.b * a.qs +
                                                      (size_t)(ahead.h * a.G + r) * D + lane * 64 % D));
    }
    look_in = p0;
    if (ahead.b != pages_b || (unsigned)(ahead.tile - pages_tile) >= 512 / KT) {
      pages_b = ahead.b;
      pages_tile = ahead.tile;
      const long long at = (long long)p0 + lane * 16;
      const int p = (int)min(max(at, (long long)ahead.s.lo), (long long)ahead.s.len - 1);
      pages = a.table[(size_t)ahead.b * a.max_blocks + (p >> a.bs_shift)];
    }
    look_part = (ahead.tile - pages_tile) * MT;
    ahead.next(a);
  };
  constexpr int kStep = 32 / C::kChunks;  // rows that one copy instruction takes
  const int row = lane / C::kChunks, chunk = lane % C::kChunks;
  const size_t lane_off = (size_t)row * a.c.slot_stride + chunk * 16;
  const size_t step = (size_t)kStep * a.c.slot_stride;
  // (a step of four rows turns the swizzle's bit 2, a step of eight none)
  const uint32_t lane_to = row * D + ((chunk ^ swizzle<D>(row)) << 4);
  const uint64_t once = a.groups == 1 ? policy_evict_first() : policy_evict_normal();
  const int box = min(1 << a.bs_shift, KT);  // rows that a bulk copy takes
  // a bit for each place of the ring: its tile came in bulk, and has not been waited for; the parity of its next
  // bulk copy; it was last written by lanes
  uint32_t bulk = 0, parity = 0, by_lanes = 0;
  auto copy = [&] {  // the tile that was looked up
    const uint32_t to = ring32 + to_stage * C::kStage, bit = 1u << to_stage, mask = (1u << a.bs_shift) - 1;
    const int page = __shfl_sync(0xffffffffu, pages, look_part + lane / kLanes);
    const bool fine = __all_sync(0xffffffffu, (unsigned)page < (unsigned)a.c.n_blocks);
    if (look_lo == 0 && look_hi == KT && fine) {
      // all its rows are in sight: K and V in bulk, a lane a page
      if (by_lanes & bit) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      by_lanes &= ~bit;
      bulk |= bit;
      __syncwarp();
      uint64_t* const bar = &s_full[warp][to_stage];
      if (lane == 0) mbar_arrive_expect_tx(bar, C::kStage);
      __syncwarp();
      const int r = lane / kLanes * 16;
      if (lane % kLanes == 0 && r % box == 0) {
        const int in = (look_in + r) & mask;
        uint8_t* const dst = s_ring + (to - smem_u32(s_ring)) + r * D;
        tma_load_4d(dst, &k_map, 0, in, look_h, page, bar, once);
        tma_load_4d(dst + C::kCodes, &v_map, 0, in, look_h, page, bar, once);
      }
    } else {
      by_lanes |= bit;
      const uint32_t dst = to + lane_to, dst2 = kStep == 4 ? dst ^ 64 : dst;
      unrolled<MT>([&](auto part) {
        constexpr int kPart = part * 16 * D;
        int block = __shfl_sync(0xffffffffu, page, part * kLanes);
        int lo = look_lo - part * 16, n = look_hi - look_lo;  // rows in sight, from the part's first
        if (block < 0 || block >= a.c.n_blocks) {
          if (lane == 0 && lo < 16 && lo + n > 0) atomicCAS(&s_err, 0, 242);
          block = 0;
          n = 0;
        }
        const size_t off = (size_t)block * a.c.block_stride + (size_t)look_h * a.c.head_stride +
                           (size_t)((look_in + part * 16) & mask) * a.c.slot_stride + lane_off;
        const uint8_t *kp = a.c.k + off, *vp = a.c.v + off;
        unrolled<16 / kStep>([&](auto i) {
          const uint32_t bytes = (unsigned)(i * kStep + row - lo) < (unsigned)n ? 16 : 0;
          copy16<kPart + i * kStep * D>(i % 2 ? dst2 : dst, bytes ? kp : a.c.k, bytes);
          copy16<kPart + i * kStep * D + C::kCodes>(i % 2 ? dst2 : dst, bytes ? vp : a.c.v, bytes);
          kp += step;
          vp += step;
        });
      });
    }
    // four scale bytes a lane: eight lanes for each 16 keys, the first four K
    const int part = (lane >> 3) & (MT - 1), r = part * 16 + (lane & 3) * 4;
    const int block = __shfl_sync(0xffffffffu, page, part * kLanes);
    if (lane < KT / 2) {
      const uint32_t bytes = r + 4 > look_lo && r < look_hi && (unsigned)block < (unsigned)a.c.n_blocks ? 4 : 0;
      const size_t from =
          bytes ? ((((size_t)block * a.c.kv_heads + look_h) << a.bs_shift) + ((look_in + r) & mask)) : 0;
      const bool v = lane & 4;
      copy4(scale32 + to_stage * 2 * KT + (v ? KT : 0) + r, (v ? a.c.v_scale : a.c.k_scale) + from, bytes);
    }
    to_stage = to_stage == C::S - 1 ? 0 : to_stage + 1;
  };

  // the queries' fragments, as f16 times a power of two of each row's, in one place or the other
  uint2 qf[C::kQueriesInSmem ? 1 : N8][C::kChunks];
  uint2* const s_q = reinterpret_cast<uint2*>(s_ring + C::kRing) + warp * N8 * C::kChunks * 32 + lane;
  float q_scale[N8][2];  // what makes a product with them a score to base 2, for this lane's two columns
  // M, the running maximum of the scores s, and L, the sum of 2^(s - M); with the values' exponents e: E, the running
  // maximum of s - M + e, and O, the sum of 2^(s - M + e - E + kShift) times the values' codes
  float o[C::kChunks][N8][4], minus_M[N8][2], E[N8][2], L[N8][2];
  int stage = 0;
  bool fresh = true, whole = false;  // the segment has no tile here yet; its first tile is in this range
  unsigned based = 0;  // a bit for each of this lane's rows that has a base: a score above -infinity
  // this lane's row of a 16-key matrix pair, and its half of two pieces
  const uint32_t lane_at = (lane & 15) * D + (((lane >> 4) ^ swizzle<D>(lane & 15)) << 4);

  bool ok = true;
  // The first S rounds only look up and copy: one copy of the code for both, as small calls wait for code most of all.
  int ahead_only = C::S;
  while (walk.left > 0) {
    const bool compute = ahead_only == 0;
    const int h = walk.h, row0 = walk.group * C::kRows;  // rows of the head's G
    const int rows = min(C::kRows, a.G - row0);
    const bool last = walk.last(), final = walk.after() <= 0;  // of the segment, of the range
    const uint32_t st32 = ring32 + stage * C::kStage + lane_at;
    uint2 w[N8][C::kChunks];
    if (compute && fresh) {  // the segment's queries, on their way while its first tile is waited for
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        const int r = n * 8 + g;
        const uint16_t* const src = a.q + (long long)walk.b * a.qs + (size_t)(h * a.G + row0 + r) * D + t * 4;
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i)
          w[n][i] = r < rows ? *reinterpret_cast<const uint2*>(src + i * 16) : make_uint2(0, 0);
      }
    }
    if (compute) {
      copies_wait<C::S - 2>();
      if (bulk >> stage & 1) {
        // (one answer for the whole warp)
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[warp][stage], parity >> stage & 1, nullptr, 0));
        if (!ok) break;
        bulk ^= 1u << stage;
        parity ^= 1u << stage;
      }
      __syncwarp();
#pragma unroll
      for (int i = lane; i < KT; i += 32) {
        const uint32_t kb = s_scale[warp][stage][i], vb = s_scale[warp][stage][KT + i];
        s_key[warp][i] = make_float2(e8m0_to_f32(kb), vb == 255 ? NAN : (float)vb - 127.f);
      }
      __syncwarp();
    }
    // (the ring's oldest place is free: its tile was computed before the last __syncwarp)
    if (looked) copy();
    look();
    copies_end();
    if (!compute) {
      --ahead_only;
      continue;
    }
    stage = stage == C::S - 1 ? 0 : stage + 1;
    if (fresh) {
      fresh = false;
      based = 0;
      whole = walk.tile == 0;
#pragma unroll
      for (int n = 0; n < N8; ++n) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i)
          top = __vmaxu2(top, __vmaxu2(w[n][i].x & 0x7fff7fffu, w[n][i].y & 0x7fff7fffu));
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e brings the largest magnitude to 2^14 to 2^15 (a smaller one of 2^-113 or less stays smaller)
        const int e = min(126, 141 - (int)(top >> 7));
        const float up = two_to(e);
#pragma unroll
        for (int i = 0; i < C::kChunks; ++i) {
          const uint32_t x[2] = {w[n][i].x, w[n][i].y};
          uint32_t y[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const __half2 hv = __floats2half2_rn(__uint_as_float(x[m] << 16) * up,
                                                 __uint_as_float(x[m] & 0xffff0000u) * up);
            y[m] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          if constexpr (C::kQueriesInSmem) s_q[(n * C::kChunks + i) * 32] = make_uint2(y[0], y[1]);
          else qf[n][i] = make_uint2(y[0], y[1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int ej = __shfl_sync(0xffffffffu, e, (2 * t + j) * 4);
          q_scale[n][j] = a.scale_log2 * two_to(-ej);
          E[n][j] = -INFINITY;
          minus_M[n][j] = L[n][j] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[c][n][j] = 0.f;
      }
    }

    // ---- scores: S[key][row] = codes . queries ----
    float s[MT][N8][4];
    unrolled<C::kChunks / 2>([&](auto pair) {
      constexpr int c = 2 * pair;
      uint2 q[N8][2];
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (C::kQueriesInSmem) q[n][x] = s_q[(n * C::kChunks + c + x) * 32];
          else q[n][x] = qf[n][c + x];
        }
      unrolled<MT>([&](auto mt) {
        uint32_t r[4];  // keys g and g + 8, columns 4 t .. 4 t + 3 of piece c; the same of c + 1
        ldmatrix<mt * 16 * D>(r, st32 ^ (c << 4));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(r[2 * x], a0, a2);
          e4m3x4_to_f16x4(r[2 * x + 1], a1, a3);
#pragma unroll
          for (int n = 0; n < N8; ++n) {
            if (c + x == 0) mma_f16_zero(s[mt][n], a0, a1, a2, a3, q[n][x].x, q[n][x].y);
            else mma_f16(s[mt][n], a0, a1, a2, a3, q[n][x].x, q[n][x].y);
          }
        }
      });
    });
    // ---- s: to base 2, with the keys' scales, less the base M; so: with the values' exponents too ----
    float so[MT][N8][4];
    Pair vs[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 key = s_key[warp][mt * 16 + k * 8 + g];
        vs[mt][k] = pair(key.y, key.y);
#pragma unroll
        for (int n = 0; n < N8; ++n) {
          float* const x = &s[mt][n][k * 2];
          const float2 u = apart(fma2(mul2(pair(x[0], x[1]), pair(q_scale[n][0], q_scale[n][1])), pair(key.x, key.x),
                                      pair(minus_M[n][0], minus_M[n][1])));
          x[0] = u.x, x[1] = u.y;
        }
      }
    if (last || walk.tile == 0) {  // rows out of sight
      const int first = walk.s.p0(walk.tile);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int p = first + mt * 16 + k * 8 + g;
          const bool see = p >= walk.s.lo && (unsigned)p < (unsigned)walk.s.len;
          if (!see) vs[mt][k] = pair(0.f, 0.f);
#pragma unroll
          for (int n = 0; n < N8; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (!see) s[mt][n][k * 2 + j] = -INFINITY;
        }
    }
    auto add_vs = [&] {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < N8; ++n) {
            const float2 v = apart(add2(pair(s[mt][n][k * 2], s[mt][n][k * 2 + 1]), vs[mt][k]));
            so[mt][n][k * 2] = v.x, so[mt][n][k * 2 + 1] = v.y;
          }
    };
    add_vs();
    // ---- running maxima: M of the scores, E of what stands in so ----
    auto top_of = [&](const float (&x)[MT][N8][4], int n, int j) {
      float m = fmaxf(x[0][n][j], x[0][n][2 + j]);
#pragma unroll
      for (int mt = 1; mt < MT; ++mt) m = fmaxf(m, fmaxf(x[mt][n][j], x[mt][n][2 + j]));
      return m;
    };
    bool more = based != (1u << 2 * N8) - 1;
    float top[N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        top[n][j] = top_of(s, n, j);
        more |= top[n][j] > kSlackM || top_of(so, n, j) > E[n][j] + kSlackE;
      }
    if (__any_sync(0xffffffffu, more)) {
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = top[n][j];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          // how far the base moves: to the largest score, the first time also down (until then L is 0, or NaN)
          const bool had = based >> (2 * n + j) & 1;
          const float by = had ? fmaxf(m, 0.f) : m == -INFINITY ? 0.f : m;
          if (had) L[n][j] *= ex2(-by);
          if (m != -INFINITY) based |= 1u << (2 * n + j);
          E[n][j] -= by;
          minus_M[n][j] -= by;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            s[mt][n][j] -= by;
            s[mt][n][2 + j] -= by;
          }
        }
      add_vs();
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = top_of(so, n, j);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          m = fmaxf(m, E[n][j]);
          const float f = m == -INFINITY ? 0.f : ex2(E[n][j] - m);
          E[n][j] = m;
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            o[c][n][j] *= f;
            o[c][n][2 + j] *= f;
          }
        }
    }
    // ---- probabilities: their sums in fp32, and as fragments of two f16 parts (with one, of 11 bits, values that cancel
    // showed it: 2^-11 of sum p |v|; the second costs 64 requests 65.9 instead of 63.3 us, 256 requests 137 instead of
    // 136, the window layer 23.8 instead of 22.7, 16 heads a key head 89.4 instead of 78.8) ----
    uint32_t pf[MT][N8][2], rest[MT][N8][2];
#pragma unroll
    for (int n = 0; n < N8; ++n) {
      const Pair shift = pair(kShift - (E[n][0] == -INFINITY ? 0.f : E[n][0]),
                              kShift - (E[n][1] == -INFINITY ? 0.f : E[n][1]));
      Pair sum = pair(L[n][0], L[n][1]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float *const x = &s[mt][n][k * 2], *const y = &so[mt][n][k * 2];
          const float2 v = apart(add2(pair(y[0], y[1]), shift));
          sum = add2(sum, pair(ex2(x[0]), ex2(x[1])));
          const float2 p = make_float2(ex2(v.x), ex2(v.y));
          const __half2 hv = __floats2half2_rn(p.x, p.y);
          const float2 up = __half22float2(hv);
          const __half2 lv = __floats2half2_rn(p.x - up.x, p.y - up.y);
          pf[mt][n][k] = transposed(*reinterpret_cast<const uint32_t*>(&hv));
          rest[mt][n][k] = transposed(*reinterpret_cast<const uint32_t*>(&lv));
        }
      const float2 l = apart(sum);
      L[n][0] = l.x;
      L[n][1] = l.y;
    }
    // ---- products with the values: O[d][row] ----
    unrolled<MT>([&](auto mt) {
      unrolled<C::kChunks / 2>([&](auto pair) {
        constexpr int c = 2 * pair;
        uint32_t r[4];
        ldmatrix_trans<C::kCodes + mt * 16 * D>(r, st32 ^ (c << 4));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // a word holds two keys by two columns: by columns, and each column's pair is a fragment's
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(__byte_perm(r[2 * x], 0, 0x3120), a0, a1);
          e4m3x4_to_f16x4(__byte_perm(r[2 * x + 1], 0, 0x3120), a2, a3);
#pragma unroll
          for (int n = 0; n < N8; ++n) {
            mma_f16(o[c + x][n], a0, a1, a2, a3, pf[mt][n][0], pf[mt][n][1]);
            mma_f16(o[c + x][n], a0, a1, a2, a3, rest[mt][n][0], rest[mt][n][1]);
          }
        }
      });
    });

    // ---- the segment's end, or the range's ----
    if (last || final) {
      const bool done = last && whole, on_way = last && !final;
      // a piece: its columns in fp32 (in the ring, whose every tile has been used, unless the range goes on), and
      // each row's maximum and sum
      float* const po = on_way ? a.warp_o + ((size_t)blockIdx.x * W + warp) * C::kPiece : piece_at(warp);
      float2* const ml = on_way ? a.warp_ml + ((size_t)blockIdx.x * W + warp) * C::kRows : s_ml[warp];
      const size_t first_row = (size_t)walk.b * hq + h * a.G + row0;
#pragma unroll
      for (int n = 0; n < N8; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float sum = L[n][j];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          // O 2^(E - kShift) / L; the power in two halves, each in range
          const float M = sum == 0.f ? -INFINITY : -minus_M[n][j], f = ex2(0.5f * (E[n][j] - kShift));
          const float f2 = sum == 0.f ? 0.f : __fdividef(f, sum);
          const int r = n * 8 + 2 * t + j;
          if (!done) {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              *reinterpret_cast<float2*>(po + r * D + c * 16 + 2 * g) =
                  make_float2(o[c][n][j] * f * f2, o[c][n][2 + j] * f * f2);
            if (g == 0) ml[r] = make_float2(M, sum);
          } else if (r < rows) {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              *reinterpret_cast<uint32_t*>(a.out + (first_row + r) * D + c * 16 + 2 * g) =
                  pack_bf16(o[c][n][j] * f * f2, o[c][n][2 + j] * f * f2);
            if (a.lse && g == 0) a.lse[first_row + r] = sum == 0.f ? -INFINITY : (M + lg2(sum)) * kLn2;
          }
        }
      if (!done && lane == 0) {
        // 1 there is one, 2 its segment started before the range, 4 it ended in it
        s_seg[warp][on_way ? 0 : 1] = make_int4(walk.b, h, row0, 1 | (whole ? 0 : 2) | (last ? 4 : 0));
        if (at_end && !last) {  // the CTA that the segment ends in
          const unsigned long long end = hi - walk.left + (unsigned)(walk.s.n - 1 - walk.tile);
          const Cut ctas(total, n_ctas);
          const unsigned long long big = ctas.more * (ctas.each + 1);
          s_last = (int)(end < big ? quot(end, ctas.each + 1) : ctas.more + quot(end - big, ctas.each));
        }
      }
    }
    fresh = last;
    walk.next(a);
  }

  // ---- the pieces of the warps joined, in the order of the line ----
  copies_wait<0>();
  if (!ok) {  // a copy did not come: its CTA's results hold no meaning; the others in flight are waited for as long
    if (lane == 0) atomicExch(&s_err, 251);
    for (int i = 0; i < C::S; ++i)
      if (bulk >> i & 1) mbar_wait(&s_full[warp][i], parity >> i & 1, nullptr, 0);
  }
  __syncthreads();
  int4 rec = make_int4(0, 0, -1, s_err);
  // pieces by warps, two bits a warp: put down on the way, at the range's end.  One that was put down on the way ends
  // its segment; so a segment's pieces are those of a run of warps' ends, and perhaps one on the next one's way.
  const int what = lane < 2 * W ? s_seg[lane >> 1][lane & 1].w : 0;
  const unsigned there = __ballot_sync(0xffffffffu, what != 0), ends = __ballot_sync(0xffffffffu, (what & 4) != 0);
  for (int e = threadIdx.x; e < C::kPiece / 4; e += C::kThreads) {
    const int r = e / (D / 4);
    unsigned left = there;
#pragma unroll 1
    while (left) {
      const int i0 = __ffs(left) - 1, i1 = ends & left ? __ffs(ends & left) - 1 : 31 - __clz(left);
      left &= ~0u << i1 << 1;
      const int w0 = i0 >> 1, w1 = (i1 - 1) >> 1;  // whose ends' pieces they are (none, if w1 < w0)
      const bool way = (i1 & 1) == 0;
      const int4 seg = s_seg[i0 >> 1][i0 & 1];
      const bool outer = (seg.w & 2) != 0, ended = ends >> i1 & 1;  // outer: it started before this CTA's range
      float2 way_ml = make_float2(-INFINITY, 0.f);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (way) {
        const size_t at = (size_t)blockIdx.x * W + (i1 >> 1);
        way_ml = a.warp_ml[at * C::kRows + r];
        acc = reinterpret_cast<const float4*>(a.warp_o + at * C::kPiece)[e];
      }
      float m = way_ml.x;
      float2 ml[W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        ml[w] = w >= w0 && w <= w1 ? s_ml[w][r] : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, ml[w].x);
      }
      const float mu = m == -INFINITY ? 0.f : m;
      float l = ex2(way_ml.x - mu) * way_ml.y;
      acc = make_float4(acc.x * l, acc.y * l, acc.z * l, acc.w * l);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w >= w0 && w <= w1) x = reinterpret_cast<const float4*>(piece_at(w))[e];
        const float f = ex2(ml[w].x - mu) * ml[w].y;
        l += f;
        acc = make_float4(fmaf(f, x.x, acc.x), fmaf(f, x.y, acc.y), fmaf(f, x.z, acc.z), fmaf(f, x.w, acc.w));
      }
      const float inv = l == 0.f ? 0.f : __fdividef(1.f, l);
      const float4 x = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (!outer && ended) {
        if (seg.z + r < a.G) {
          const size_t at = (size_t)seg.x * hq + seg.y * a.G + seg.z + r;
          *reinterpret_cast<uint2*>(a.out + at * D + (e % (D / 4)) * 4) =
              make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
          if (a.lse && e % (D / 4) == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + lg2(l)) * kLn2;
        }
      } else {
        const size_t at = (size_t)blockIdx.x * 2 + !outer;
        reinterpret_cast<float4*>(a.o + at * C::kPiece)[e] = x;
        if (e % (D / 4) == 0) a.ml[at * C::kRows + r] = make_float2(m, l);
        if (!outer) rec = make_int4(seg.x, seg.y << 8 | seg.z / 8, s_last, rec.w);
      }
    }
  }
  if (rec.w > 250) rec.z = -1;
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

// A segment that several CTAs share: its pieces joined in the order of the line, a CTA for the one that its first
// piece is from.  Beside that the rows of requests without positions, and by the first CTA what the others found wrong.
template <int D, int N8>
__global__ void __launch_bounds__(256) decode_merge_kernel(const DecodeArgs a) {
  using C = Cfg<D, N8>;
  __shared__ int s_err;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    if (threadIdx.x == 0) s_err = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < a.ctas; i += blockDim.x)
      if (const int e = a.rec[i].w) atomicMax(&s_err, e);
    __syncthreads();
    if (threadIdx.x == 0)
      *a.status = Status{s_err > 250 ? LMOE_ETIMEOUT : s_err ? LMOE_EDEVICE_CHECK : LMOE_OK, s_err};
  }
  const int e = blockIdx.y * blockDim.x + threadIdx.x, r = e / (D / 4), hq = a.c.kv_heads * a.G;
  Sum sum;
  // n pieces from p0 on (those up to `end` are there) into the sum: fetched at once, then joined
  auto fetch = [&](auto n, auto& ml, auto& o, int p0, int end) {
#pragma unroll
    for (int u = 0; u < n; ++u) {
      const int p = min(p0 + u, end);
      const size_t at = (size_t)p * 2 + (p == (int)blockIdx.x);
      ml[u] = a.ml[at * C::kRows + r];
      o[u] = reinterpret_cast<const float4*>(a.o + at * C::kPiece)[e];
    }
  };
  auto join = [&](auto n, const auto& ml, const auto& o, int p0, int end) {
    float m = sum.m;
#pragma unroll
    for (int u = 0; u < n; ++u) m = p0 + u <= end ? fmaxf(m, ml[u].x) : m;
    const float mu = m == -INFINITY ? 0.f : m, f = ex2(sum.m - mu);
    sum.m = m;
    sum.l *= f;
    sum.o = make_float4(sum.o.x * f, sum.o.y * f, sum.o.z * f, sum.o.w * f);
#pragma unroll
    for (int u = 0; u < n; ++u)
      if (p0 + u <= end) sum.add(ex2(ml[u].x - mu) * ml[u].y, o[u]);
  };
  // the first pieces before it is known whether there are any
  constexpr std::integral_constant<int, 4> kFirst{};
  constexpr std::integral_constant<int, 8> kMore{};
  float2 ml[kFirst.value];
  float4 o[kFirst.value];
  fetch(kFirst, ml, o, blockIdx.x, a.ctas - 1);
  const int4 rec = a.rec[blockIdx.x];
  int len = (int)blockIdx.x < a.B && blockIdx.y == 0 ? a.lens[blockIdx.x] : 1;
  const int h = rec.y >> 8, row = (rec.y & 255) * 8 + r;
  if (rec.z >= 0 && row < a.G) {
    join(kFirst, ml, o, blockIdx.x, rec.z);
    for (int p0 = blockIdx.x + kFirst; p0 <= rec.z; p0 += kMore) {
      float2 ml8[kMore.value];
      float4 o8[kMore.value];
      fetch(kMore, ml8, o8, p0, rec.z);
      join(kMore, ml8, o8, p0, rec.z);
    }
    const float inv = sum.l == 0.f ? 0.f : __fdividef(1.f, sum.l);
    const size_t at = (size_t)rec.x * hq + h * a.G + row;
    *reinterpret_cast<uint2*>(a.out + at * D + (e % (D / 4)) * 4) =
        make_uint2(pack_bf16(sum.o.x * inv, sum.o.y * inv), pack_bf16(sum.o.z * inv, sum.o.w * inv));
    if (a.lse && e % (D / 4) == 0) a.lse[at] = sum.lse();
  }
  // requests without positions
  for (int b = blockIdx.x; b < a.B && blockIdx.y == 0;) {
    if (len == 0) {
      for (int i = threadIdx.x; i < hq * D / 8; i += blockDim.x)
        reinterpret_cast<uint4*>(a.out + (size_t)b * hq * D)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = threadIdx.x; i < hq; i += blockDim.x) a.lse[(size_t)b * hq + i] = -INFINITY;
    }
    if ((b += gridDim.x) < a.B) len = a.lens[b];
  }
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

// What a cache's copy descriptors depend on.
void maps_key(const lmoe_kv_cache_fp8* c, uint64_t (&key)[8]) {
  key[0] = reinterpret_cast<uintptr_t>(c->k);
  key[1] = reinterpret_cast<uintptr_t>(c->v);
  key[2] = (uint64_t)(uint32_t)c->n_blocks << 32 | (uint32_t)c->block_size;
  key[3] = (uint64_t)(uint32_t)c->kv_heads << 32 | (uint32_t)c->head_dim;
  key[4] = (uint64_t)c->block_stride;
  key[5] = (uint64_t)c->head_stride;
  key[6] = (uint64_t)c->slot_stride;
  key[7] = 1;
}

// K and V as [block][head][slot][d], copied by a page, or by a tile's rows of one.
int make_maps(const lmoe_kv_cache_fp8* c, lmoe_kv_maps_fp8* m) {
  static_assert(sizeof(m->map[0]) == sizeof(CUtensorMap), "a map's size");
  // a dimension of extent 1 never steps: any valid stride will do
  auto stride = [](int64_t bytes, int64_t extent) { return (uint64_t)(extent > 1 ? bytes : 64); };
  const uint64_t dims[4] = {(uint64_t)c->head_dim, (uint64_t)c->block_size, (uint64_t)c->kv_heads,
                            (uint64_t)c->n_blocks};
  const uint64_t strides[3] = {stride(c->slot_stride, c->block_size), stride(c->head_stride, c->kv_heads),
                               stride(c->block_stride, c->n_blocks)};
  const uint32_t box[4] = {(uint32_t)c->head_dim, (uint32_t)std::min(c->block_size, 4096 / c->head_dim), 1, 1};
  for (int i = 0; i < 2; ++i) {
    CUtensorMap t;
    if (encode_tmap(&t, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? c->v : c->k, dims, strides, box,
                    c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return LMOE_ECUDA;
    std::memcpy(m->map[i], &t, sizeof(t));
  }
  maps_key(c, m->made_for);
  return LMOE_OK;
}

// Query heads of a kv head that one reading of its keys serves, in eights.
int eights(const lmoe_decode_dims* d, const lmoe_kv_cache_fp8* c) { return d->q_heads / c->kv_heads <= 8 ? 1 : 2; }

struct DecodeWs {
  size_t rec, ml, o, warp_ml, warp_o, total;
};

constexpr int kMostWarps = 12;

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
  w.warp_ml = take(kMostWarps * ctas * rows * sizeof(float2));
  w.warp_o = take(kMostWarps * ctas * rows * row);
  w.total = at;
  return w;
}

template <int D, int N8>
int run_decode(const DecodeArgs& a, const CUtensorMap (&tm)[2], cudaStream_t s) {
  using C = Cfg<D, N8>;
  static std::atomic<unsigned long long> done{0};
  int rc = allow_smem(done, decode_attn_kernel<D, N8>, C::kSmem);
  if (rc) return rc;
  rc = launch_pdl("decode_attn_kernel", dim3(a.ctas), dim3(C::kThreads), C::kSmem, s, decode_attn_kernel<D, N8>, a,
                  tm[0], tm[1]);
  if (rc) return rc;
  constexpr int kUnits = C::kPiece / 4, kBlock = kUnits < 256 ? kUnits : 256;
  return launch_pdl("decode_merge_kernel", dim3(a.ctas, kUnits / kBlock), dim3(kBlock), 0, s,
                    decode_merge_kernel<D, N8>, a);
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

int lmoe_kv_maps_fp8_init(const lmoe_kv_cache_fp8* cache, lmoe_kv_maps_fp8* maps) {
  const int rc = check_cache_fp8(cache, true);
  if (rc) return rc;
  if (!maps) return LMOE_EINVAL;
  return make_maps(cache, maps);
}

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
  lmoe_kv_maps_fp8 own;
  const lmoe_kv_maps_fp8* maps = c->maps;
  maps_key(c, own.made_for);
  if (!maps || std::memcmp(maps->made_for, own.made_for, sizeof(own.made_for)) != 0) {
    if ((rc = make_maps(c, &own))) return rc;
    maps = &own;
  }
  CUtensorMap tm[2];
  std::memcpy(tm, maps->map, sizeof(tm));
  if (c->head_dim == 64) return n8 == 1 ? run_decode<64, 1>(a, tm, s) : run_decode<64, 2>(a, tm, s);
  return n8 == 1 ? run_decode<128, 1>(a, tm, s) : run_decode<128, 2>(a, tm, s);
}

}  // extern "C"

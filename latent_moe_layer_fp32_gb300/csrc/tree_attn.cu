// Attention of drafted tokens over a paged cache and the tree of drafts.
// See include/lmoe.h for the contract.
//
// Work.  The rows that share a key head's keys are one request's drafted
// tokens times the q_heads / kv_heads query heads of the group; 128 (or 256)
// of them form a row group, 128 keys a tile: the cached prefix in tiles of
// consecutive positions, then the drafts.  A segment is one (request, kv head,
// row group); its tiles are laid end to end with those of all other segments
// and the whole line is cut into equal ranges, one per CTA, so ragged lengths
// and single long requests both fill the GPU.  A segment inside one CTA's
// range is finished there; one that is cut leaves fp32 partial sums (running
// maximum, sum, unnormalised output), which tree_attn_merge_kernel joins in
// the order of the ranges, so results do not depend on timing.
//
// CTA.  Two producer warps copy K and V tiles page by page with TMA (128-byte
// swizzle) into a ring of 160 KB or more; one warp issues tcgen05.mma: S = Q K^T
// (both K-major from shared memory) into tensor memory, and O += P V with P read
// from tensor memory and V as an MN-major operand straight from its pages'
// layout.  Two softmax groups of four warps own a row per thread: they read S,
// keep the row's running maximum and sum in registers, write P (bf16, in place
// of S, with a second bf16 part where one key may dominate a row) and rescale O
// only when the maximum has grown by more than 2^8 (P is then at most 2^8, which
// bf16 and the fp32 sums hold without loss).
// Up to 128 rows per kv head: the groups take turns by segment, each with its
// own queries and its own O, so one loads queries, joins and stores while the
// other computes, and S of the next tile is computed during the softmax of
// this one.  More rows: the groups take a row tile each of the same segment.
// A further warp cleans the value tiles at an edge of what rows see, so that
// no bits of an unseen key reach a product.
//
// What bounds it, and what it takes (GB300; 64 query heads, 8 kv heads, 128
// columns; 6784 GB/s and 1940 TFLOP/s are the measured rates of a copy and of a
// bf16 GEMM).  Up to 128 rows, HBM: 16 requests of 12000 positions take 127 us
// with 8 drafts each (6240 GB/s, 92%) and 133 us with 16; 64 of one token and
// 512 to 8191 positions 110 us (6320 GB/s).  Past that the tensor cores: 64
// drafts each take 291 to 305 us by the box (1320 to 1380 TFLOP/s).  A tile of
// two row tiles then takes about 3050 clocks: its four products need 2048, and
// their operands and the copies of K and V alone keep shared memory busy for as
// many (128 bytes a clock); each group's softmax (1900) and its own two products
// follow one another, since 512 columns of tensor memory hold no second S.  A
// segment's end costs four such tiles or so, which is what ragged trees pay: 32
// requests with 33 to 64 drafts over 1024 to 8192 positions take 198 us (889
// TFLOP/s; rows that fill no row tile are 15% of that; 205 called from Python).
// Small calls are a chain of latencies: 8 drafts of one request over 1021
// positions take 13.1 us in a graph.  By the slowest CTA, from the end of the
// launch before: lengths summed at 1.2 us, ranges known at 2.1, first page numbers
// at 3.3, first scores at 5.3, softmax done at 6.8, product at 7.1, sums stored at
// 7.8, all CTAs over at 8.2; the merge kernel starts at 9.1, has read the pieces
// at 11.2, joined them at 12.3 and stored at 12.5.
// The warps' loops together are longer than the instruction cache, so code that
// is off the hot path costs time on it: several of the forms here were chosen
// for being short.
#include <atomic>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "launch.cuh"
#include "tc_attn.cuh"
#include "tmap.cuh"

namespace lmoe {

namespace {

constexpr int kTile = 128;  // keys per tile, rows per row tile
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* v_cache;  // also read directly where a value is not finite
  const uint16_t* v_new;
  long long qs, vs, block_stride, head_stride, slot_stride;
  const int32_t *offsets, *lens, *table, *pos;
  const uint64_t* mask;
  uint16_t* out;
  float* lse;
  Status* status;  // the workspace's status word
  Status* err;     // [CTAs], joined into *status by the merge kernel
  int4* cut;       // [CTAs][2], the segment that starts in a CTA's range and ends past it
  float2* part_ml; // [2 CTAs][rows] running maximum (base 2) and sum
  float* part_o;   // [2 CTAs][D / 4][rows][4]
  int B, T, max_n, hk, G, max_blocks, n_blocks, bs_shift, words, window, ctas;
  uint32_t wait_limit;  // of bar_wait
  float scale_log2;
};

// One request's share of the line of tiles: np tiles of 128 cached positions
// from base0 on (a page boundary at or below the first position in sight),
// then tiles of drafts, nt in all.  Up to 128 drafts move in behind the cached
// positions of the last, partial tile when they fit there (at column c0 > 0, a
// multiple of 8 rows for the copies), which saves a tile of its own.
struct Req {
  int t0, n, len, base0, np, nt, c0;
  int cut, full;  // tiles below cut hold positions that some row's window leaves out; from full on, not 128 positions
  __device__ __forceinline__ int base(int i) const { return base0 + (i << 7); }
  // cached positions in tile i; the drafts in it, from d0 on, at columns from col on
  __device__ __forceinline__ int cached(int i) const { return i < np ? min(kTile, len - base(i)) : 0; }
  __device__ __forceinline__ int d0(int i) const { return c0 ? 0 : (i - np) << 7; }
  __device__ __forceinline__ int drafts(int i) const {
    return i >= np ? min(kTile, n - ((i - np) << 7)) : (c0 && i == np - 1 ? n : 0);
  }
  __device__ __forceinline__ int col(int i) const { return i < np ? c0 : 0; }
  // whether some row sees only part of tile i: where a window cuts, the prefix's end, and drafts
  __device__ __forceinline__ bool edge(int i) const { return i < cut || i >= full; }
};

// 64-bit division is a long subroutine; nearly always 32 bits will do.
__device__ __forceinline__ unsigned long long quot(unsigned long long x, unsigned long long y) {
  return (x | y) >> 32 ? x / y : (unsigned)x / (unsigned)y;
}

// A wait bounded in SM clocks, counted in units of 2^32 (about two seconds): it runs out when the count has
// passed more than `limit` of them.  Some waits last as long as a CTA's part of a segment, so the limit grows
// with the longest request that the call admits (wait_limit).  The kernel's warps run different loops of it at
// once and wait for instructions where these do not fit the instruction cache together, so this is kept short:
// what ran out is noted in `failed` and reported once, at the kernel's end.  Each lane answers for itself, and
// at the limit two lanes' answers may differ.  So a warp leaves a loop only by a vote; half a warp that had
// left would have the other half wait for it at the next warp-wide step.  With votes at every wait of the
// issuing warp wide trees took 204 us instead of 199, so that one votes once a tile (a window layer: 40.5 us,
// 39.2 without any vote; the other cases the same).
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, int where, int& failed, uint32_t limit) {
  if (mbar_try_wait(bar, parity)) return true;
  uint32_t t0, t1;
  asm volatile("mov.u32 %0, %%clock_hi;" : "=r"(t0));
  do {
    if (mbar_try_wait(bar, parity)) return true;
    asm volatile("mov.u32 %0, %%clock_hi;" : "=r"(t1));
  } while (t1 - t0 <= limit);
  failed = where;
  return false;
}

// bar_wait with one answer for the whole warp (all 32 lanes wait).
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity, int where, int& failed, uint32_t limit) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, where, failed, limit));
}

// Whether phase `parity` of `bar` has completed, the same answer in every lane (all 32 ask).  The phase may
// complete between two lanes' probes; an answer that steers the whole warp has to be one for all of them.
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
}

// How the line of tiles is measured for the cut into equal ranges: a tile of two row tiles, of one, and the
// end of a segment (its sums joined and stored, the next one's queries, masks and first tiles).  Measured:
// the ends at two and a half tiles instead of half a one took 16 requests of 1000 to 32768 positions from
// 136 to 126 us; of two row tiles, 32 requests with 33 to 64 drafts take 201 us at 12, 202 at 18, 205 at 21
// (and took 253 at 3 instead of 221 at 18 when an end was slower).
// A range has to hold the start of a tile, so with few tiles the ends count less (end_cost).
template <int NT>
struct Cost {
  static constexpr int kTwo = NT == 2 ? 3 : 2, kOne = 2, kEnd = NT == 2 ? 12 : 5;
};

struct Load {
  int groups;        // row groups: a segment each per kv head
  int last;          // cost of a tile of the last group
  long long head;    // cost of a kv head's tiles
  bool bad;
  // of the request, with `end` for each segment's end
  __device__ __forceinline__ long long units(int hk, int end) const { return hk * (head + (long long)groups * end); }
};

template <int NT, int ROWS>
__device__ __forceinline__ Load load_req(const AttnArgs& a, int b, Req* r) {
  const int t0 = __ldg(a.offsets + b), t1 = __ldg(a.offsets + b + 1), len = __ldg(a.lens + b);
  Load w;
  w.bad = t0 < 0 || t1 < t0 || t1 > a.T || t1 - t0 > a.max_n || len < 0 ||
          len > ((long long)a.max_blocks << a.bs_shift);
  r->t0 = t0;
  r->n = w.bad ? 0 : t1 - t0;
  r->len = len;
  const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // the first position that any row sees
  r->base0 = lo & ~((1 << min(a.bs_shift, 7)) - 1);
  const int held = lo < len ? len - r->base0 : 0;
  r->np = (held >> 7) + ((held & 127) != 0);
  r->full = held >> 7;
  // the last row's window starts at len + n - window at most
  r->cut = a.window > 0 ? (max(0, len - r->base0 + min(0, r->n - a.window)) + 127) >> 7 : 0;
  const int tail = ((held & 127) + 7) & ~7;
  r->c0 = (held & 127) != 0 && tail + r->n <= kTile ? tail : 0;
  r->nt = r->np + (r->c0 ? 0 : (r->n + kTile - 1) >> 7);
  w.groups = (r->n * a.G + ROWS - 1) / ROWS;
  w.last = r->n * a.G - (w.groups - 1) * ROWS > kTile ? Cost<NT>::kTwo : Cost<NT>::kOne;
  w.head = w.groups == 0 ? 0 : (long long)r->nt * ((long long)(w.groups - 1) * Cost<NT>::kTwo + w.last);
  return w;
}

// Tiles that start below x, which lies within a segment (32 bits); a tile costs 2 or 3.
template <int NT>
__device__ __forceinline__ int tiles_below(long long x, int tile) {
  const unsigned y = (unsigned)x;
  return NT == 2 && tile == 3 ? (y + 2u) / 3u : (y + 1u) / 2u;
}

// A segment by its place in its request's part of the line.
struct Place {
  int h, m, tile;   // kv head, row group, cost of a tile
  long long start;  // where it starts
};

template <int NT>
__device__ __forceinline__ Place place(const Load& w, int nt, int end, long long off) {
  Place p;
  const long long head = w.units(1, end);
  // at most 256 heads: the quotient in floats is off by one at most
  p.h = (int)__fdividef((float)off, (float)head);
  p.h -= off < p.h * head;
  p.h += off >= (p.h + 1) * head;
  const long long r = off - p.h * head, group = (long long)nt * Cost<NT>::kTwo + end;
  p.m = NT == 1 || w.groups == 1 ? 0 : min((int)quot(r, group), w.groups - 1);
  p.tile = p.m == w.groups - 1 ? w.last : Cost<NT>::kTwo;
  p.start = p.h * head + p.m * group;
  return p;
}

// The part of one segment that falls into a CTA's range.
struct alignas(16) Seg {
  Req r;
  int b, h, m;   // request, kv head, row group
  int i0, i1;    // tiles [i0, i1) of r.nt; i1 = 0 marks the end of the CTA's segments
  int rows;      // valid rows of this row group
  int pad;
};
static_assert(sizeof(Seg) == 64, "four 16-byte pieces");

// Walks the segments of the CTA's range: a tile belongs to the range that it starts in.
template <int NT, int ROWS>
struct Walk {
  const AttnArgs& a;
  int b, cost;         // request; of a segment's end
  long long off, end;  // where the range goes on and where it ends, from request b's start
  long long at;        // where request b starts in the whole line
  long long last;      // where the last tile of the latest segment starts in it
  __device__ bool next(Seg* s) {
    while (off < end) {
      const Load w = load_req<NT, ROWS>(a, b, &s->r);
      const long long units = w.units(a.hk, cost);
      if (off >= units) {
        off -= units;
        end -= units;
        at += units;
        ++b;
        continue;
      }
      const int nt = s->r.nt;
      const Place p = place<NT>(w, nt, cost, off);
      const int i0 = tiles_below<NT>(off - p.start, p.tile);
      off = p.start + (long long)nt * p.tile + cost;
      if (i0 >= nt) continue;
      const int i1 = tiles_below<NT>(min(max(end - p.start, 0ll), (long long)nt * p.tile), p.tile);
      if (i1 <= i0) return false;
      last = at + p.start + (long long)(nt - 1) * p.tile;
      s->b = b;
      s->h = p.h;
      s->m = p.m;
      s->i0 = i0;
      s->i1 = i1;
      s->rows = min(ROWS, s->r.n * a.G - p.m * ROWS);
      return true;
    }
    return false;
  }
};

// A draft's position past the prefix's end (the position itself may pass 31 bits): at most the deepest place
// that n drafts can reach.
__device__ __forceinline__ int draft_depth(const AttnArgs& a, int t0, int n, int len, int j) {
  return a.pos ? min(max(__ldg(a.pos + t0 + j), len) - len, n - 1) : j;
}

__device__ __forceinline__ uint64_t range_bits(int lo, int hi) {  // bits [lo, hi) of a 64-bit word
  const int a = min(max(lo, 0), 64), b = min(max(hi, 0), 64);
  const uint64_t below_b = b == 64 ? ~0ull : (1ull << b) - 1ull, below_a = a == 64 ? ~0ull : (1ull << a) - 1ull;
  return below_b & ~below_a;
}

// What draft vi (vd positions past the prefix) of a segment's request sees of the 128 columns of tile i.
__device__ __forceinline__ ulonglong2 edge_bits(const AttnArgs& a, const Seg* s, int i, int vi, int vd) {
  uint64_t bits[2];
  const int cached = s->r.cached(i), first = a.window > 0 ? vd - a.window + 1 + (s->r.len - s->r.base(i)) : 0;
  bits[0] = range_bits(first, cached);
  bits[1] = range_bits(first - 64, cached - 64);
  const int nd = s->r.drafts(i);
  if (nd == 0) return make_ulonglong2(bits[0], bits[1]);
  const int d0 = s->r.d0(i), c = s->r.col(i), t0 = s->r.t0;
  // the drafts d0 .. d0 + 127 that the row sees, moved up to column c
  uint64_t m0, m1;
  if (a.mask) {
    const uint64_t* row = a.mask + (size_t)(t0 + vi) * a.words;
    const int w = d0 >> 6;
    m0 = w < a.words ? __ldg(row + w) : 0ull;
    m1 = w + 1 < a.words ? __ldg(row + w + 1) : 0ull;
  } else {
    m0 = range_bits(0, vi - d0 + 1);
    m1 = range_bits(0, vi - d0 - 63);
  }
  m0 &= range_bits(0, nd);
  m1 &= range_bits(0, nd - 64);
  const int n = s->r.n, len = s->r.len;
  if (a.window > 0 && n > a.window) {  // some pair of drafts may be a window apart
    for (uint64_t z = m0; z; z &= z - 1)
      if (vd - draft_depth(a, t0, n, len, d0 + __ffsll(z) - 1) >= a.window) m0 &= ~(z & -z);
    for (uint64_t z = m1; z; z &= z - 1)
      if (vd - draft_depth(a, t0, n, len, d0 + 63 + __ffsll(z)) >= a.window) m1 &= ~(z & -z);
  }
  if (c >= 64) {
    bits[1] |= m0 << (c - 64);
  } else if (c > 0) {
    bits[0] |= m0 << c;
    bits[1] |= m1 << c | m0 >> (64 - c);
  } else {
    bits[0] |= m0;
    bits[1] |= m1;
  }
  return make_ulonglong2(bits[0], bits[1]);
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 bytes global -> shared without registers; `bytes` 0 writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// pairs of floats: one instruction for two products or sums
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Turns U 16-byte units per lane into whole pieces of rows: afterwards unit j of lane l is unit l % U of
// lane l / U * U + j, so that U neighbouring lanes hold 16 U consecutive bytes of one row.
template <int U>
__device__ __forceinline__ void turn_units(uint32_t (&w)[U][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < U; s *= 2)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (!(u & s))
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t mine = lane & s ? w[u][j] : w[u | s][j];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, mine, s);
          if (lane & s)
            w[u][j] = got;
          else
            w[u | s][j] = got;
        }
}

// Stores 16 U bytes of each lane's row, at `row` (null: no row), U lanes to a row.
template <int U>
__device__ __forceinline__ void store_rows(uint32_t (&w)[U][4], void* row) {
  const int lane = threadIdx.x & 31;
  turn_units<U>(w);
#pragma unroll
  for (int j = 0; j < U; ++j) {
    char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), (lane & -U) + j));
    if (dst) *reinterpret_cast<uint4*>(dst + (lane % U) * 16) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
  }
}

// Adds the values that are not finite, of the keys that a row sees, to the thread's row of O: the cleaning
// warp took them out.  Runs only where there was one.
template <int D, int CW>
__device__ __forceinline__ void add_not_finite(const AttnArgs& a, const Seg* s, uint32_t o_addr, int part, bool valid,
                                            int vi, int vd, int i0, int n) {
#pragma unroll 1
  for (int col = 0; col < D; col += 16) {
    uint32_t o[16];
    tmem_ld16(o_addr + col, o);
    tmem_ld_wait();
    for (int i = i0; valid && i < i0 + n; ++i) {
      if (!s->r.edge(i)) continue;
      const ulonglong2 bits = edge_bits(a, s, i, vi, vd);
#pragma unroll 1
      for (int j = part * CW; j < part * CW + CW; ++j) {
        if (!((j >= 64 ? bits.y : bits.x) >> (j & 63) & 1ull)) continue;
        const uint16_t* val;
        if (j < s->r.cached(i)) {
          const int p = s->r.base(i) + j;
          const int id = __ldg(a.table + (size_t)s->b * a.max_blocks + (p >> a.bs_shift));
          if (id < 0 || id >= a.n_blocks) continue;
          val = a.v_cache + (size_t)id * a.block_stride + (size_t)s->h * a.head_stride +
                (size_t)(p & ((1 << a.bs_shift) - 1)) * a.slot_stride;
        } else {
          val = a.v_new + (size_t)(s->r.t0 + s->r.d0(i) + j - s->r.col(i)) * a.vs + s->h * D;
        }
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          const uint32_t x = val[col + d];
          if ((x & 0x7f80u) == 0x7f80u) o[d] = __float_as_uint(__uint_as_float(o[d]) + bf16_bits_to_f32(x));
        }
      }
    }
    __syncwarp();
    tmem_st16(o_addr + col, o);
  }
  tmem_st_wait();
}

// D: head width.  NT: row tiles of 128 rows per CTA.  KS: with few rows (128 / KS at most) each row
// stands KS times in the row tile, and the copies take 128 / KS of a tile's keys each, so that all four
// softmax warps work on 32 rows or less.
template <int D, int NT, int KS>
struct Cfg {
  static_assert(NT == 1 || KS == 1, "copies of rows only in a single row tile");
  static constexpr int kRows = NT * kTile / KS;
  static constexpr int kCols = kTile / KS;            // keys of a tile per softmax thread
  static constexpr int kStageBytes = kTile * D * 2;   // one K or V tile
  static constexpr int kQBytes = KS > 1 ? 32768 : kTile * D * 2;  // a group's queries; with copies also their sums
  static constexpr int kStages = D == 128 ? 5 : (KS > 1 ? 10 : 12);  // 160 KB of keys and values, or more, in flight
  static constexpr int kThreads = 384;                // two softmax groups, two producers, MMA, cleaning warp
  static constexpr int kMisc = 3 * 1024;
  static constexpr int kSmem = 2 * kQBytes + kStages * kStageBytes + kMisc;
  static constexpr uint32_t kO = 2 * kTile;           // first O column; S buffers at 0 and 128
  // the join of copies: each takes D / KS columns of the sum, in passes of kPass columns
  static constexpr int kOwn = D / KS;
  static constexpr int kPass = KS == 4 && D == 128 ? 16 : kOwn;
  static_assert(KS == 1 || kTile * (KS - 1) * kPass * 4 <= kQBytes, "room for the copies' sums");
  static_assert(kSmem <= 232448, "shared memory budget");
};

// Ring position of K and V of the CTA's tile g.  The groups in turns: K0 K1 V0 K2 V1 ... (S runs one tile
// ahead, also across segments; the place before the last V stays empty); two row tiles: K0 V0 K1 V1 ...
template <int NT>
__device__ __forceinline__ uint32_t k_pos(uint32_t g) {
  return NT == 2 ? 2 * g : (g == 0 ? 0 : 2 * g - 1);
}
template <int NT>
__device__ __forceinline__ uint32_t v_pos(uint32_t g) {
  return NT == 2 ? 2 * g + 1 : 2 * g + 2;
}

template <int D, int NT, int KS>
__global__ void __launch_bounds__(Cfg<D, NT, KS>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kn,
                     const __grid_constant__ CUtensorMap tm_vn, const __grid_constant__ CUtensorMap tm_k8,
                     const __grid_constant__ CUtensorMap tm_v8) {
  using C = Cfg<D, NT, KS>;
  constexpr int ST = C::kStages, ROWS = C::kRows, HALVES = D / 64;
  extern __shared__ __align__(1024) uint8_t smem[];  // no static shared memory: the base is 1024-byte aligned
  uint8_t* s_q = smem;
  uint8_t* s_ring = smem + 2 * C::kQBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ring + ST * C::kStageBytes);
  uint64_t* empty = full + ST;
  uint64_t* s_full = empty + ST;   // [S buffer] a tile's scores are in tensor memory
  uint64_t* p_full = s_full + 2;   // [S buffer][half] its probabilities for keys 0..63, 64..127 are
  uint64_t* pv_done = p_full + 4;  // [S buffer] its product with V has been added to O
  uint64_t* q_full = pv_done + 2;  // [group] the segment's queries are in shared memory
  uint64_t* s_first = q_full + 2;  // [group] scores of a segment's first tile
  uint64_t* v_edge = s_first + 2;  // an edge tile is next to be cleaned
  uint64_t* v_clean = v_edge + 1;  // it has been
  uint64_t* seg_full = v_clean + 1;   // [4] a segment's record is there
  uint64_t* seg_empty = seg_full + 4; // [4] every warp is through with it
  uint64_t* join = seg_empty + 4;     // [group] its four warps meet (a barrier whose wait is bounded)
  uint64_t* done = join + 2;
  long long* s_start = reinterpret_cast<long long*>(done + 1);  // request, units into it, units in the range
  unsigned long long* s_warp = reinterpret_cast<unsigned long long*>(s_start + 3);  // [threads / 32][2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_warp + 24);
  volatile uint32_t* s_lo = tmem_slot + 1;     // [S buffer] a byte per warp: P has a second part
  volatile uint32_t* s_dirty = tmem_slot + 3;  // [segment % 4] segment + 1 where a value was not finite
  Seg* s_seg = reinterpret_cast<Seg*>(reinterpret_cast<uint8_t*>(full) + 1024);  // [segment % 4]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kKeys = 8, kMma = 9, kValues = 10;  // warps 0 to 7: softmax; 11: cleaning
  Status* st = a.err + blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], KS == 1 ? 4 : 2);  // the warps that hold the half's keys
      mbar_init(&p_full[2 * i + 1], KS == 1 ? 4 : 2);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 4);
      mbar_init(&s_first[i], 1);
      mbar_init(&join[i], 4);
    }
    mbar_init(v_edge, 1);
    mbar_init(v_clean, 1);
    mbar_init(done, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 11);  // warps 9 to 11 and the eight softmax warps
      s_dirty[i] = 0;
    }
    fence_barrier_init();
    s_start[2] = 0;
  }
  if (warp == kMma) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's range of the line of tiles ----
  int end_cost;                          // of a segment's end
  long long line, ranges, first = 0;     // the line's length, its ranges, this range's start
  if (tid == 0) *st = Status{0, 0};
  {
    const int per = (a.B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    unsigned long long tiles = 0, segs = 0;  // of this thread's requests: the tiles' cost, the segments
    bool bad = false;
    Load w0{};
    for (int b = b0; b < b1; ++b) {
      Req r;
      const Load w = load_req<NT, ROWS>(a, b, &r);
      tiles += a.hk * w.head;
      segs += (unsigned)(a.hk * w.groups);
      bad |= w.bad;
      if (b == b0) w0 = w;
    }
    unsigned long long x = tiles, y = segs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x1 = __shfl_up_sync(0xffffffffu, x, o), y1 = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += x1, y += y1;
    }
    if (lane == 31) s_warp[2 * warp] = x, s_warp[2 * warp + 1] = y;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    unsigned long long tiles_before = x - tiles, segs_before = y - segs, all_tiles = 0, all_segs = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) tiles_before += s_warp[2 * w], segs_before += s_warp[2 * w + 1];
      all_tiles += s_warp[2 * w];
      all_segs += s_warp[2 * w + 1];
    }
    // the most that leaves every CTA a range with the start of a tile
    end_cost = (int)min((long long)Cost<NT>::kEnd,
                        max(0ll, (long long)quot(all_tiles, a.ctas) - Cost<NT>::kTwo));
    const unsigned long long before = tiles_before + segs_before * end_cost, mine = tiles + segs * end_cost;
    const unsigned long long total = all_tiles + all_segs * end_cost;
    if (bad) set_error(st, LMOE_EDEVICE_CHECK, 211);
    // ranges, each long enough to hold the start of a tile
    const unsigned long long n =
        total ? max(1ull, min((unsigned long long)a.ctas, quot(total, Cost<NT>::kTwo + end_cost))) : 0ull;
    const unsigned long long c = blockIdx.x;
    ranges = (long long)n;
    line = (long long)total;
    if (c < n) {
      const unsigned long long u0 = quot(total * c, n);
      first = (long long)u0;
      if (u0 >= before && u0 < before + mine) {
        int b = b0;
        unsigned long long at = before;
        for (Load w = w0;; ++b) {
          if (b > b0) {
            Req r;
            w = load_req<NT, ROWS>(a, b, &r);
          }
          const unsigned long long units = w.units(a.hk, end_cost);
          if (u0 < at + units) break;
          at += units;
        }
        s_start[0] = b;
        s_start[1] = (long long)(u0 - at);
        s_start[2] = (long long)(quot(total * (c + 1), n) - u0);
      }
    }
    __syncthreads();
  }
  const uint32_t tmem = *tmem_slot;
  // 384 threads start with 168 registers each; with a whole tile's scores per thread the service
  // warps hand some of theirs to the softmax warps (88 + 2 x 208 = 3 x 168)
  auto fewer = [] {
    if constexpr (KS == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  };
  int failed = 0;  // where a wait of this lane ran out
  auto gave_up = [&] { return __any_sync(0xffffffffu, failed != 0) != 0; };
  // the record of segment `i`, once it is there; warps take the segments in order
  auto seg_at = [&](uint32_t i) { return const_cast<const Seg*>(s_seg + (i & 3)); };
  auto seg_wait = [&](uint32_t i) { return bar_wait(&seg_full[i & 3], (i >> 2) & 1, 261, failed, a.wait_limit); };
  auto seg_done = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0 && failed == 0) mbar_arrive(&seg_empty[i & 3]);  // (never for a record that did not come)
  };

  if (warp == kKeys || warp == kValues) {
    // ---------------- TMA producers: a lane per page (or 8 rows) ----------------
    fewer();
    const bool keys = warp == kKeys;
    const uint64_t once = policy_evict_first(), again = NT == 2 ? policy_evict_normal() : once;
    const int box = min(1 << a.bs_shift, kTile);  // rows per copy of a whole cached tile
    const int ppt = kTile / box;                  // pages per such tile
    uint32_t g = 0, seg = 0, issued = 0;          // issued: past the last ring position that was issued
    bool ok = true;
    Walk<NT, ROWS> walk{a, (int)s_start[0], end_cost, s_start[1], s_start[1] + s_start[2], first - s_start[1], 0};
    int4 cut0 = make_int4(0, 0, 0, 0), cut1 = cut0;  // the latest segment, if it starts in this range and ends past it
    for (;; ++seg) {
      // the keys' producer walks the range and posts each segment's record, the others read it
      Seg s{};
      if (keys) {
        const bool more = walk.next(&s);
        if (!more)
          s.i0 = s.i1 = 0;
        else if (s.i0 == 0 && s.i1 < s.r.nt)
          cut0 = make_int4(1, s.r.t0, s.rows, s.h), cut1 = make_int4(s.m, 0, 0, 0);
        else
          cut0.x = 0;
        if (!(ok = bar_wait_warp(&seg_empty[seg & 3], ((seg >> 2) & 1) ^ 1, 262, failed, a.wait_limit))) break;
        if (lane == 0) {
          s_seg[seg & 3] = s;
          mbar_arrive(&seg_full[seg & 3]);
        }
        __syncwarp();
      } else {
        if (!(ok = __all_sync(0xffffffffu, seg_wait(seg)))) break;
        s = *seg_at(seg);
        seg_done(seg);
      }
      if (s.i1 == 0) break;
      // Keys and values stay in L2 for further row groups of the request, from three groups on (4 requests of
      // 8000 to 12000 positions with 256 drafts, eight groups: 241 us instead of 247; 8 with 128: 250 instead of
      // 254; with two groups the next one is close behind: 32 requests with 33 to 64 drafts 199.8 against 198.3).
      const int all_rows = s.r.n * a.G;
      const uint64_t pol = NT == 2 && all_rows > 2 * ROWS && (s.m + 1) * ROWS < all_rows ? again : once;
      const int32_t* const table = a.table + (size_t)s.b * a.max_blocks;
      auto page = [&](int i) {  // the block of this lane's cached rows of tile i
        const int cached = s.r.cached(i), rows = cached == kTile ? box : 8;
        return lane * rows < cached ? __ldg(table + ((s.r.base(i) + lane * rows) >> a.bs_shift)) : 0;
      };
      int id_next = page(s.i0);
      for (int i = s.i0; i < s.i1; ++i, ++g) {
        int id = id_next;
        if (i + 1 < s.i1) id_next = page(i + 1);
        if (id < 0 || id >= a.n_blocks) {  // out of the cache: the copy reads zeros
          set_error(st, LMOE_EDEVICE_CHECK, 212);
          id = a.n_blocks;
        }
        // a whole tile page by page, a partial one and the drafts 8 rows at a time
        const int cached = s.r.cached(i);
        const int rows = cached == kTile ? box : 8;
        const int nc = cached == kTile ? ppt : (cached + 7) >> 3, nd = (s.r.drafts(i) + 7) >> 3;
        auto copy = [&](uint32_t at) {
          const CUtensorMap* const tc = rows == 8 ? (keys ? &tm_k8 : &tm_v8) : (keys ? &tm_k : &tm_v);
          const uint32_t stage = at % ST;
          if (!bar_wait_warp(&empty[stage], ((at / ST) & 1) ^ 1, 221, failed, a.wait_limit)) return false;
          uint8_t* dst = s_ring + stage * C::kStageBytes;
          if (lane == 0) mbar_arrive_expect_tx(&full[stage], (nc * rows + nd * 8) * (128 * HALVES));
          __syncwarp();
          if (lane < nc) {
            const int slot = (s.r.base(i) + lane * rows) & ((1 << a.bs_shift) - 1);
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
              tma_load_4d(dst + hf * (kTile * 128) + lane * rows * 128, tc, hf * 64, slot, s.h, id, &full[stage], pol);
          } else if (lane < nc + nd) {
            const int j = (lane - nc) * 8;
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
              tma_load_3d(dst + hf * (kTile * 128) + (s.r.col(i) + j) * 128, keys ? &tm_kn : &tm_vn, hf * 64, s.h,
                          s.r.t0 + s.r.d0(i) + j, &full[stage], pol);
          }
          __syncwarp();
          issued = at + 1;
          return true;
        };
        if (!(ok = copy(keys ? k_pos<NT>(g) : v_pos<NT>(g)))) break;
      }
      if (!ok) break;
    }
    if (keys && lane == 0) {
      // for the merge: a cut segment's last CTA is the first one whose range ends after the start of its last tile
      if (cut0.x) cut0.x = (int)quot((walk.last + 1) * ranges + line - 1, line) - (int)blockIdx.x;
      a.cut[2 * blockIdx.x] = cut0;
      a.cut[2 * blockIdx.x + 1] = cut1;
    }
    // this warp's last copies land before the CTA can finish (also after a wait that ran out); a stage
    // that has been filled again since needs no wait
    const uint32_t end = ok ? v_pos<NT>(g - 1) + 1 : issued;
    for (uint32_t k = g < ST ? 0 : g - ST; k < g; ++k) {
      const uint32_t at = keys ? k_pos<NT>(k) : v_pos<NT>(k);
      if (at + ST >= end) bar_wait(&full[at % ST], (at / ST) & 1, 222, failed, a.wait_limit);
    }
  } else if (warp == kMma) {
    // ---------------- MMA issuer ----------------
    fewer();
    // the whole warp walks, so that addresses stay in uniform registers; one lane issues
    {
      const bool leader = elect_one();
      constexpr uint32_t kQk = idesc_bf16_f32(128, kTile);
      constexpr uint32_t kPv = idesc_bf16_f32(128, D) | kIdescBMnMajor;
      // a tile goes on after a wait that ran out, on whatever there is; the vote at the next one ends the loop
      auto ready = [&](uint64_t* bar, uint32_t parity, int where) { bar_wait(bar, parity, where, failed, a.wait_limit); };
      // descriptors step by their start address (bits 0 to 13, in units of 16 bytes)
      const uint64_t qd = smem_desc_sw128(smem_u32(s_q)), kd = smem_desc_sw128(smem_u32(s_ring));
      const uint64_t vd = smem_desc_sw128_mn(smem_u32(s_ring), kTile * 128);
      auto qk = [&](int grp, uint32_t buf, uint32_t stage) {
        const uint64_t q = qd + grp * (C::kQBytes >> 4), kk0 = kd + stage * (C::kStageBytes >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
            tc_mma_bf16(tmem + buf * kTile, q + o, kk0 + o, kQk, kk != 0);
          }
          tc_commit(&s_full[buf]);
        }
        __syncwarp();
      };
      // (after a wait that ran out no stage is given back: a copy may still be on its way into it)
      auto commit = [&](uint64_t* bar) {
        if (leader && failed == 0) tc_commit(bar);
        __syncwarp();
      };
      // O += P V for 64 keys at a time, each half as soon as its probabilities are there
      auto pv = [&](int grp, uint32_t buf, uint32_t stage, bool first, uint32_t parity) {
        const uint64_t v0 = vd + stage * (C::kStageBytes >> 4);
        const uint32_t p = tmem + buf * kTile, o = tmem + C::kO + grp * D;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          ready(&p_full[2 * buf + hf], parity, 233 + hf);
          tc_fence_after();
          const uint32_t lo = s_lo[buf], ph = p + hf * 64;
          const uint64_t vh = v0 + hf * (64 * 128 >> 4);
          // P of 16 keys each stands at 0, 8, 32 and 40 of a half's columns, the second parts 16 further on;
          // with copies of rows a 16-key step goes to the lanes whose copy holds those keys
          auto lanes = [&](int kk, bool second, uint32_t (&off)[4]) {
            const int part = KS == 1 ? 0 : KS == 2 ? hf : 2 * hf + (kk >> 1);
#pragma unroll
            for (int w = 0; w < 4; ++w) off[w] = w * KS / 4 == part && (!second || (lo >> (8 * w) & 1u)) ? 0u : 0xffffffffu;
          };
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t acc = !(first && (KS == 1 ? hf == 0 && kk == 0 : kk % (8 / KS) == 0));
              if constexpr (KS == 1) {
                tc_mma_bf16_ts(o, ph + (kk >> 1) * 32 + (kk & 1) * 8, vh + kk * (16 * 128 >> 4), kPv, acc);
              } else {
                uint32_t off[4];
                lanes(kk, false, off);
                tc_mma_bf16_ts_lanes(o, ph + (kk >> 1) * 32 + (kk & 1) * 8, vh + kk * (16 * 128 >> 4), kPv, acc, off);
              }
            }
            if (lo) {  // the second part, for the warps that wrote one
#pragma unroll 1
              for (int kk = 0; kk < 4; ++kk) {
                uint32_t off[4];
                lanes(kk, true, off);
                tc_mma_bf16_ts_lanes(o, ph + (kk >> 1) * 32 + (kk & 1) * 8 + 16, vh + kk * (16 * 128 >> 4), kPv, 1u, off);
              }
            }
            if (hf == 1) tc_commit(&pv_done[buf]);
          }
          __syncwarp();
        }
      };
      uint32_t ring = 0, ring_phase = 0;
      auto skip = [&] {
        if (++ring == ST) {
          ring = 0;
          ring_phase ^= 1;
        }
      };
      auto tile = [&](uint32_t* stage) {  // the next tile of the ring has landed (they are taken in its order)
        ready(&full[ring], ring_phase, 231);
        tc_fence_after();
        *stage = ring;
        skip();
      };
      // what this warp needs of a segment
      struct Part {
        int i0, i1, cut, full, rows;
        __device__ __forceinline__ bool edge(int i) const { return i < cut || i >= full; }
      };
      Part s{}, nx{};
      auto get = [&](uint32_t i, Part* p) {
        seg_wait(i);
        const Seg* x = seg_at(i);
        *p = Part{x->i0, x->i1, x->r.cut, x->r.full, x->rows};
        seg_done(i);
      };
      auto clean = [&](const Part& p, int i) {  // hands tile i to the cleaning warp if it is an edge
        if (p.edge(i) && lane == 0) mbar_arrive(v_edge);
        __syncwarp();
      };
      uint32_t edges = 0;  // edge tiles that came back from the cleaning warp
      uint32_t ks = 0, vs = 0;  // stages of the keys and values in use
      uint32_t nq = 0, np = 0;  // a bit per group (or S buffer): the phase of its queries, of its P
      // Tile by tile: the scores of the next one (of the same segment, or the next segment's first), and the
      // product of this one with its values.
      bool have = false;
      int i = 0;
      for (uint32_t seg = 0;;) {
        const bool same = have && i + 1 < s.i1;
        if (!same) get(seg, &nx);
        if (gave_up()) break;
        const Part t = same ? s : nx;  // of the next tile
        const int ti = same ? i + 1 : nx.i0;
        const bool more = same || nx.i1 > 0;
        if constexpr (NT == 1) {
          // group of this segment: seg is one past it
          const uint32_t tg = (same ? seg - 1 : seg) & 1, tb = have ? (np >> 2 & 1) ^ 1 : 0;
          if (more) {
            if (!same) {
              ready(&q_full[tg], nq >> tg & 1, 232);
              nq ^= 1u << tg;
            }
            tile(&ks);
            qk(tg, tb, ks);
            if (!same) commit(&s_first[tg]);
            commit(&empty[ks]);
          } else if (have) {
            skip();  // the place before the last values
          }
          if (have) {
            const uint32_t buf = np >> 2 & 1;
            tile(&vs);
            if (s.edge(i)) ready(v_clean, edges++ & 1, 236);
            if (more) clean(t, ti);
            pv((seg - 1) & 1, buf, vs, i == s.i0, np >> buf & 1);
            commit(&empty[vs]);
            np ^= 1u << buf | 4u;  // bit 2: the S buffer of the tile
          } else if (more) {
            clean(t, ti);
          }
        } else {
          if (have) {
            tile(&vs);
            if (s.edge(i)) ready(v_clean, edges++ & 1, 236);
          }
          if (more) clean(t, ti);  // (one at a time, so that no phase is missed)
#pragma unroll 1
          for (int grp = 0; grp < 2; ++grp) {
            if (have && (grp == 0 || s.rows > kTile)) {
              pv(grp, grp, vs, i == s.i0, np >> grp & 1);
              np ^= 1u << grp;
              if (grp == 1 || s.rows <= kTile) commit(&empty[vs]);
            }
            if (more && (grp == 0 || t.rows > kTile)) {
              if (!same) {
                ready(&q_full[grp], nq >> grp & 1, 232);
                nq ^= 1u << grp;
              }
              if (grp == 0) tile(&ks);
              tc_fence_after();
              qk(grp, grp, ks);
            }
          }
          if (more) commit(&empty[ks]);
        }
        if (!more) break;
        if (!same) ++seg;
        s = t;
        i = ti;
        have = true;
      }
      if (leader) tc_commit(done);  // every MMA issued has completed before TMEM is released
      __syncwarp();
      bar_wait(done, 0, 235, failed, a.wait_limit);
    }
  } else if (warp < kKeys) {
    // ---------------- softmax: one row per thread ----------------
    if constexpr (KS == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr int CW = C::kCols;
    const int grp = warp >> 2, row = tid & 127;  // group, row of its row tile
    const int part = KS == 1 ? 0 : row / (kTile / KS);  // which copy of the rows: keys part * CW .. + CW of each tile
    const int local = (NT == 2 ? grp * kTile : 0) + (KS == 1 ? row : row % (kTile / KS));  // row of the row group
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_base + C::kO + grp * D;
    uint8_t* const q_buf = s_q + grp * C::kQBytes;
    uint32_t seg = 0, g = 0, g_own = 0;           // segments and tiles of the CTA so far; tiles of this group
    // After a wait that ran out the warp goes on without waiting to the segment's end and leaves; what
    // it writes is void.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
      if (ok) ok = bar_wait(bar, parity, where, failed, a.wait_limit);
      tc_fence_after();
    };
    uint32_t meets = 0;
    auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&join[grp]);
      wait(&join[grp], meets++ & 1, 246);
    };
    // the thread's row of a segment's queries, in the swizzled K-major layout; rows past the last are zero
    auto load_q = [&](const Seg* sg) {
      const int r2 = sg->m * C::kRows + local;
      const bool valid = local < sg->rows;
      const int i = valid ? r2 / a.G : 0, h = valid ? sg->h * a.G + r2 - i * a.G : 0;
      const uint16_t* src = a.q + (size_t)(sg->r.t0 + i) * a.qs + (size_t)h * D;
      const uint32_t dst = smem_u32(q_buf) + row * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        cp_async16(dst + (c >> 3) * (kTile * 128) + (((c & 7) ^ (row & 7)) << 4), src + c * 8, valid ? 16 : 0);
    };
    auto q_loaded = [&] {
      cp_async_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[grp]);
    };
    bool early = false;  // the segment's queries were loaded during the one before
    for (;; ++seg) {
      if (ok) ok = seg_wait(seg);
      ok = __all_sync(0xffffffffu, ok);
      const Seg* const s = seg_at(seg);
      const int i0 = s->i0, n = s->i1 - i0;
      if (!ok || n == 0) break;
      if (NT == 1 ? (int)(seg & 1) != grp : (grp == 1 && s->rows <= kTile)) {  // not this group's
        seg_done(seg);
        g += n;
        continue;
      }
      const int cut = s->r.cut, full_from = s->r.full;
      const bool valid = local < s->rows;
      const bool warp_live = __any_sync(0xffffffffu, valid);
      if (!early) {
        load_q(s);
        q_loaded();
      }
      early = false;
      const int vi = valid ? (s->m * C::kRows + local) / a.G : 0;  // the row's draft
      auto depth = [&] { return a.window > 0 ? draft_depth(a, s->r.t0, s->r.n, s->r.len, vi) : 0; };
      // m_ref: the maximum that P refers to; l: the row's sum.  A tile whose maximum stays below
      // `limit` takes the plain path: no rescaling of O, one part of P.
      float m_ref = -INFINITY, l = 0.f, limit = valid ? -INFINITY : INFINITY;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int i = i0 + k;
        const uint32_t gt = g + k, go = g_own + k;
        const uint32_t buf = NT == 1 ? gt & 1 : grp;
        const bool edge = (i < cut || i >= full_from) && warp_live;
        ulonglong2 bits = make_ulonglong2(0, 0);
        if (edge) bits = edge_bits(a, s, i, vi, depth());  // (before the wait, which hides its loads)
        if (NT == 1 && k == 0)
          wait(&s_first[grp], (seg >> 1) & 1, 240);  // s_full may be phases behind until then
        else
          wait(&s_full[buf], NT == 1 ? (gt >> 1) & 1 : go & 1, 242);
        const uint32_t s_addr = tmem + lane_base + buf * kTile;
        auto p_ready = [&](int half) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * buf + half]);
        };
        if (warp_live) {
          // the tile's maximum
          float mx[2] = {-INFINITY, -INFINITY};
          auto most = [&](const uint32_t (&y)[32]) {
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              mx[(j >> 1) & 1] = max3(mx[(j >> 1) & 1], __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
          };
          if (edge) {
            // unseen keys' scores become -infinity, in place
#pragma unroll 1
            for (int c = 0; c < CW / 32; ++c) {
              const int w = part * (CW / 32) + c;
              const uint32_t x = valid ? (uint32_t)((w & 2 ? bits.y : bits.x) >> (32 * (w & 1))) : 0u;
              uint32_t y[32];
              tmem_ld32(s_addr + w * 32, y);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(x >> j & 1u)) y[j] = 0xff800000u;
              tmem_st32(s_addr + w * 32, y);
              most(y);
            }
            tmem_st_wait();
          } else {
            uint32_t y[2][32];
            tmem_ld32(s_addr + part * CW, y[0]);
#pragma unroll
            for (int c = 0; c < CW / 32; ++c) {
              tmem_ld_wait();
              if (c + 1 < CW / 32) tmem_ld32(s_addr + part * CW + (c + 1) * 32, y[(c + 1) & 1]);
              most(y[c & 1]);
            }
          }
          const float m_new = fmaxf(mx[0], mx[1]) * a.scale_log2;
          uint64_t sum[2] = {0, 0};
          // p = 2^(sc s - mu) of 32 keys, in place, and its bf16 part
          auto exps = [&](uint32_t (&y)[32], uint32_t (&p)[16], uint64_t sc2, uint64_t mu2) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float e0, e1;
              unpair(fma2(pair(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1])), sc2, mu2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[j & 1] = add2(sum[j & 1], pair(e0, e1));
              p[j] = pack_bf16(e0, e1);
              y[2 * j] = __float_as_uint(e0);
              y[2 * j + 1] = __float_as_uint(e1);
            }
          };
          const bool plain = !__any_sync(0xffffffffu, m_new > limit);
          if (plain) {
            if (lane == 0) reinterpret_cast<volatile uint8_t*>(s_lo + buf)[warp & 3] = 0;
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), mu2 = pair(-mu, -mu);
            // the scores once more: P takes the place of scores that have been read, 32 keys in 16 columns
            const uint32_t from = s_addr + part * CW;
            uint32_t y0[32], y1[32], p[16];
            tmem_ld32(from, y0);
            if constexpr (CW == 32) {
              tmem_ld_wait();
              exps(y0, p, sc2, mu2);
              tmem_st16(from, p);
            } else {
#pragma unroll 1
              for (int c = 0; c < CW / 32; c += 2) {
                tmem_ld_wait();
                tmem_ld32(from + c * 32 + 32, y1);
                exps(y0, p, sc2, mu2);
                tmem_st16(from + c * 32, p);
                tmem_ld_wait();
                if (c + 2 < CW / 32) tmem_ld32(from + c * 32 + 64, y0);
                exps(y1, p, sc2, mu2);
                tmem_st16(from + c * 32 + 32, p);
                if (KS == 1 && c == 0) {  // the first half's product can start
                  tmem_st_wait();
                  p_ready(0);
                }
              }
            }
          } else {
            const bool grow = m_new > m_ref + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
              const float f = grow ? ex2(m_ref - m_new) : 1.f;
              if (k > 0) {
                wait(&pv_done[NT == 1 ? (gt - 1) & 1 : grp], NT == 1 ? ((gt - 1) >> 1) & 1 : (go - 1) & 1, 243);
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                  uint32_t o[16];
                  tmem_ld16(o_addr + c * 16, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                  tmem_st16(o_addr + c * 16, o);
                }
                l *= f;
              }
              if (grow) m_ref = m_new;
            }
            const float mu = m_ref == -INFINITY ? 0.f : m_ref;
            // p = 2^(scale s - mu) in one fused step, whose error against the rounded mu is common to
            // the row.  Past 2^24 that error alone could overflow: there scale s is rounded first too.
            float sc = a.scale_log2;
            const bool huge = __any_sync(0xffffffffu, fabsf(mu) > 16777216.f);
            if (huge) sc = 1.f;
            const uint64_t sc2 = pair(sc, sc), mu2 = pair(-mu, -mu);
            // P as one bf16 part is off by up to 2^-8 of each key's share.  Where some key of a row
            // holds over 1/8 of the row's sum so far that would show in the output next to its own
            // rounding, so the remainder goes along as a second part; with more keys in play it
            // averages out.  After a prefix's first tiles this is rare.  On this path it goes along in any
            // case: to wait for the tile's sum takes longer than its products (32 requests with 33 to 64
            // drafts: 207 us instead of 203).
            if (lane == 0) reinterpret_cast<volatile uint8_t*>(s_lo + buf)[warp & 3] = 1;
#pragma unroll 1
            for (int c = 0; c < CW / 32; ++c) {
              const uint32_t at = s_addr + part * CW + c * 32;
              uint32_t y[32], p[16];
              tmem_ld32(at, y);
              tmem_ld_wait();
              if (huge) {
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * a.scale_log2);
              }
              exps(y, p, sc2, mu2);
              tmem_st16(at, p);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float e0 = __uint_as_float(y[2 * j]), e1 = __uint_as_float(y[2 * j + 1]);
                p[j] = pack_bf16(e0 - __uint_as_float(p[j] << 16), e1 - __uint_as_float(p[j] & 0xffff0000u));
              }
              tmem_st16(at + 16, p);
              if (KS == 1 && c == 1) {  // the first half's product can start
                tmem_st_wait();
                p_ready(0);
              }
            }
          }
          tmem_st_wait();
          p_ready(KS == 1 || part >= KS / 2 ? 1 : 0);
          float s0, s1;
          unpair(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          // below: no growth past 2^8, and no key over 1/8 of the sum so far
          if (valid) limit = fabsf(m_ref) <= 16777216.f ? m_ref + fminf(8.f, __log2f(l) - 3.f) : -INFINITY;
        } else {
          if (lane == 0) reinterpret_cast<volatile uint8_t*>(s_lo + buf)[warp & 3] = 0;
          if (KS == 1) p_ready(0);
          p_ready(KS == 1 || part >= KS / 2 ? 1 : 0);
        }
      }
      // ---- the segment's end: finished rows to out, cut ones to the partial sums ----
      const uint32_t ge = NT == 1 ? g + n - 1 : g_own + n - 1;  // the segment's last tile
      if (NT == 2 && bar_test(&seg_full[(seg + 1) & 3], ((seg + 1) >> 2) & 1)) {
        // every product with these queries is done: the next segment's may come in
        const Seg* nx = seg_at(seg + 1);
        early = nx->i1 > 0 && (grp == 0 || nx->rows > kTile);
        if (early) {
          load_q(nx);
          q_loaded();
        }
      }
      wait(&pv_done[NT == 1 ? ge & 1 : grp], NT == 1 ? (ge >> 1) & 1 : ge & 1, 245);
      const bool whole = i0 == 0 && n == s->r.nt;
      const int qh = s->h * a.G + (valid ? s->m * C::kRows + local - vi * a.G : 0), tok = s->r.t0 + vi;
      const bool dirty = s_dirty[seg & 3] == seg + 1;
      const int slot = 2 * blockIdx.x + (i0 == 0);
      if (dirty && warp_live) add_not_finite<D, CW>(a, s, o_addr, part, valid, vi, depth(), i0, n);
      // N columns of this thread's row of O
      auto sums = [&](int col, auto& y) {
        constexpr int N = sizeof(y) / 4;
        uint32_t* o = reinterpret_cast<uint32_t*>(&y[0]);
#pragma unroll
        for (int c = 0; c < N; c += 16) tmem_ld16(o_addr + col + c, *reinterpret_cast<uint32_t(*)[16]>(o + c));
        tmem_ld_wait();
      };
      // N columns of each row from col on (all lanes of the warp)
      auto put = [&](int col, const auto& y, float inv) {
        constexpr int N = sizeof(y) / 4;
        if (whole) {
          uint16_t* const dst = valid ? a.out + ((size_t)tok * (a.hk * a.G) + qh) * D + col : nullptr;
          uint32_t w[N / 8][4];
#pragma unroll
          for (int u = 0; u < N / 8; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) w[u][j] = pack_bf16(y[u * 8 + 2 * j] * inv, y[u * 8 + 2 * j + 1] * inv);
          if constexpr (KS == 1) {  // 128 rows' worth of 16-byte stores would queue up: 32 bytes of a row at a time
            store_rows<N / 8>(w, dst);
          } else if (dst) {
#pragma unroll
            for (int u = 0; u < N / 8; ++u)
              *reinterpret_cast<uint4*>(dst + u * 8) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
          }
        } else if (valid) {  // [slot][4 columns][row]: neighbouring lanes' pieces are neighbours
          float4* const dst = reinterpret_cast<float4*>(a.part_o) + ((size_t)slot * (D / 4) + col / 4) * C::kRows + local;
#pragma unroll
          for (int j = 0; j < N / 4; ++j)
            dst[j * C::kRows] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
      };
      if constexpr (KS == 1) {
        const float inv = l > 0.f ? __fdividef(1.f, l) : (l == 0.f ? 0.f : l);
        if (warp_live) {
#pragma unroll 1
          for (int col = 0; col < D; col += 16) {
            float y[16];
            sums(col, y);
            put(col, y, inv);
          }
        }
      } else {
        // join the copies of a row: M = max m_i, L = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M).  Each copy
        // finishes kOwn columns; the others hand theirs over through the queries' buffer (every product that
        // reads it is done), [owner][other copy][row][kPass] with 16-byte pieces swizzled against conflicts.
        constexpr int RP = kTile / KS, P = C::kPass, OWN = C::kOwn;
        float2* ml = reinterpret_cast<float2*>(q_buf);
        ml[row] = make_float2(m_ref, l);
        meet();
        float M = -INFINITY;
#pragma unroll
        for (int p = 0; p < KS; ++p) M = fmaxf(M, ml[p * RP + local].x);
        const float mu = M == -INFINITY ? 0.f : M;
        const float f = ex2(m_ref - mu);
        l = 0.f;
#pragma unroll
        for (int p = 0; p < KS; ++p) {
          const float2 y = ml[p * RP + local];
          l += y.y * ex2(y.x - mu);
        }
        m_ref = M;
        meet();
        const float inv = l > 0.f ? __fdividef(1.f, l) : (l == 0.f ? 0.f : l);
        auto piece = [&](int owner, int from, int j) {
          const int x = P == 16 ? (local >> 1) & 3 : local & 7;
          return reinterpret_cast<float4*>(
              q_buf + ((owner * (KS - 1) + (from > owner ? from - 1 : from)) * RP + local) * (P * 4) + ((j ^ x) << 4));
        };
#pragma unroll 1
        for (int q = 0; q < OWN; q += P) {
          if (q > 0) meet();
          if (warp_live) {
#pragma unroll
            for (int d = 1; d < KS; ++d) {
              const int owner = (part + d) % KS;
              float y[P];
              sums(owner * OWN + q, y);
#pragma unroll
              for (int j = 0; j < P / 4; ++j)
                *piece(owner, part, j) = make_float4(y[4 * j] * f, y[4 * j + 1] * f, y[4 * j + 2] * f, y[4 * j + 3] * f);
            }
          }
          float y[P];
          if (warp_live) sums(part * OWN + q, y);
          meet();
          if (warp_live) {
#pragma unroll
            for (int j = 0; j < P; ++j) y[j] *= f;
#pragma unroll
            for (int d = 1; d < KS; ++d) {
              const int from = (part + d) % KS;
#pragma unroll
              for (int j = 0; j < P / 4; ++j) {
                const float4 z = *piece(part, from, j);
                y[4 * j] += z.x;
                y[4 * j + 1] += z.y;
                y[4 * j + 2] += z.z;
                y[4 * j + 3] += z.w;
              }
            }
            put(part * OWN + q, y, inv);
          }
        }
        meet();  // the next queries overwrite the buffer
      }
      if (valid && part == 0) {
        if (!whole)
          a.part_ml[(size_t)slot * C::kRows + local] = make_float2(m_ref, l);
        else if (a.lse)
          a.lse[(size_t)tok * (a.hk * a.G) + qh] = l == 0.f ? -INFINITY : (m_ref + __log2f(l)) * 0.69314718055994531f;
      }
      seg_done(seg);
      g += n;
      g_own += n;
    }
  } else {
    // ---------------- cleaning: the value tiles at an edge ----------------
    // Values that no row sees become zero (0 * NaN would reach every row), and so do those that are not
    // finite among the keys that only some rows see: these are added back to the rows that see them at
    // the segment's end.  A warp's access covers 4 keys of 128 bytes.
    fewer();
    uint32_t g = 0, edges = 0;
    for (uint32_t seg = 0;; ++seg) {
      seg_wait(seg);
      if (gave_up()) break;
      const Seg s = *seg_at(seg);
      seg_done(seg);
      if (s.i1 == 0) break;
      for (int i = s.i0; i < s.i1; ++i, ++g) {
        if (!s.r.edge(i)) continue;
        bar_wait(v_edge, edges++ & 1, 251, failed, a.wait_limit);
        const uint32_t at = v_pos<NT>(g);
        bar_wait(&full[at % ST], (at / ST) & 1, 252, failed, a.wait_limit);
        uint8_t* const vt = s_ring + (at % ST) * C::kStageBytes + (lane & 7) * 16;
        const int base = s.r.base(i), hi = s.r.cached(i), nd = s.r.drafts(i), c0 = nd ? s.r.col(i) : hi, c1 = c0 + nd;
        // cached positions: seen by some row from `first` on, by every row from `all` on
        const int first = a.window > 0 ? min(max(s.r.len - base - a.window + 1, 0), hi) : 0;
        const int all = a.window > 0 ? min(max(s.r.len - base + (s.r.n - a.window), 0), hi) : 0;
        bool found = false;
        auto zero = [&](int from, int to) {
          for (int key = from + (lane >> 3); key < to; key += 4)
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf)
              *reinterpret_cast<uint4*>(vt + hf * (kTile * 128) + key * 128) = make_uint4(0u, 0u, 0u, 0u);
        };
        auto check = [&](int from, int to) {
          for (int key = from + (lane >> 3); key < to; key += 4)
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
              uint4* const w = reinterpret_cast<uint4*>(vt + hf * (kTile * 128) + key * 128);
              uint4 y = *w;
              uint32_t* const e = &y.x;
              uint32_t top = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
              for (int j = 0; j < 4; ++j) top |= (e[j] & 0x7f807f80u) + 0x00800080u;
              if (top & 0x80008000u) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if ((e[j] & 0x7f80u) == 0x7f80u) e[j] &= 0xffff0000u;
                  if ((e[j] & 0x7f800000u) == 0x7f800000u) e[j] &= 0xffffu;
                }
                *w = y;
                found = true;
              }
            }
        };
        zero(0, first);
        check(first, all);
        zero(hi, c0);
        check(c0, c1);
        zero(c1, kTile);
        if (found) s_dirty[seg & 3] = seg + 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_clean);
      }
    }
  }
  if (failed) set_error(st, LMOE_ETIMEOUT, failed);
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of each cut segment: block x is the CTA in whose range a segment starts, its pieces lie
// in that CTA's tail slot and the head slots of the CTAs after it.  A thread joins 4 columns of a row, a
// block 8 rows (4 or 16: 1% slower); 4 pieces are under way at a time (what there is so far is
// rescaled for them): 32 requests with 33 to 64 drafts 215 us with the attention, 2: 215, 8: 219, 16: 233; one
// request over 131071 positions 90.0 us, 2: 91.2, 8: 91.2, 16: 93.7.  Bound by the trip to L2; alone 4 to 6 us.
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum O_i 2^(m_i - M) / L
template <int D>
__global__ void __launch_bounds__(2 * D) tree_attn_merge_kernel(const AttnArgs a, int rows) {
  pdl_wait();
  pdl_trigger();
  const int4 c0 = a.cut[2 * blockIdx.x], c1 = a.cut[2 * blockIdx.x + 1];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {  // the call's status: the first CTA's error
    Status e{0, 0};
    for (int c = threadIdx.x; c < a.ctas; c += 32) {
      const Status x = a.err[c];
      if (e.code == 0) e = x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, e.code != 0);
    const int from = hit ? __ffs(hit) - 1 : 0;
    e.code = __shfl_sync(0xffffffffu, e.code, from);
    e.where = __shfl_sync(0xffffffffu, e.where, from);
    if (threadIdx.x == 0) *a.status = e;
  }
  const int pieces = c0.x, unit = threadIdx.x >> 3, local = blockIdx.y * 8 + (threadIdx.x & 7);
  if (pieces < 2 || local >= c0.z) return;
  auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + p)); };
  constexpr int U = 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), next_o[U];
  float2 next_ml[U];
  float M = -INFINITY, L = 0.f;
  auto fetch = [&](int p0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      next_ml[u] = make_float2(-INFINITY, 0.f);
      next_o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p0 + u < pieces) {
        next_ml[u] = a.part_ml[slot(p0 + u) * rows + local];
        next_o[u] = reinterpret_cast<const float4*>(a.part_o)[(slot(p0 + u) * (D / 4) + unit) * rows + local];
      }
    }
  };
  fetch(0);
#pragma unroll 1
  for (int p0 = 0; p0 < pieces; p0 += U) {
    float4 o[U];
    float2 ml[U];
#pragma unroll
    for (int u = 0; u < U; ++u) o[u] = next_o[u], ml[u] = next_ml[u];
    if (p0 + U < pieces) fetch(p0 + U);
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float mu = top == -INFINITY ? 0.f : top, f = ex2(M - mu);
    M = top;
    L *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p0 + u < pieces) {
        const float w = ex2(ml[u].x - mu);
        L = fmaf(w, ml[u].y, L);
        acc.x = fmaf(w, o[u].x, acc.x);
        acc.y = fmaf(w, o[u].y, acc.y);
        acc.z = fmaf(w, o[u].z, acc.z);
        acc.w = fmaf(w, o[u].w, acc.w);
      }
  }
  const int rr = c1.x * rows + local;
  const int i = rr / a.G, tok = c0.y + i, qh = c0.w * a.G + rr - i * a.G;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + ((size_t)tok * (a.hk * a.G) + qh) * D + unit * 4) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse && unit == 0)
    a.lse[(size_t)tok * (a.hk * a.G) + qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// What a cache's copy descriptors depend on.
void maps_key(const lmoe_kv_cache* c, uint64_t (&key)[8]) {
  key[0] = reinterpret_cast<uintptr_t>(c->k);
  key[1] = reinterpret_cast<uintptr_t>(c->v);
  key[2] = (uint64_t)(uint32_t)c->n_blocks << 32 | (uint32_t)c->block_size;
  key[3] = (uint64_t)(uint32_t)c->kv_heads << 32 | (uint32_t)c->head_dim;
  key[4] = (uint64_t)c->block_stride;
  key[5] = (uint64_t)c->head_stride;
  key[6] = (uint64_t)c->slot_stride;
  key[7] = 1;
}

// The cache as [block][head][slot][d], copied 64 columns by one page (at most a tile) at a time: K, V; and
// by 8 slots: K, V.
int make_maps(const lmoe_kv_cache* c, lmoe_kv_maps* m) {
  static_assert(sizeof(m->map[0]) == sizeof(CUtensorMap), "a map's size");
  // a dimension of extent 1 never steps: any valid stride will do
  auto stride = [](int64_t elements, int64_t extent) { return (uint64_t)(extent > 1 ? elements : 64) * 2; };
  const uint64_t dims[4] = {(uint64_t)c->head_dim, (uint64_t)c->block_size, (uint64_t)c->kv_heads,
                            (uint64_t)c->n_blocks};
  const uint64_t strides[3] = {stride(c->slot_stride, c->block_size), stride(c->head_stride, c->kv_heads),
                               stride(c->block_stride, c->n_blocks)};
  for (int i = 0; i < 4; ++i) {
    const uint32_t box[4] = {64, i < 2 ? (uint32_t)min(c->block_size, kTile) : 8u, 1, 1};
    CUtensorMap t;
    if (encode_tmap(&t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, i & 1 ? c->v : c->k, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return LMOE_ECUDA;
    std::memcpy(m->map[i], &t, sizeof(t));
  }
  maps_key(c, m->made_for);
  return LMOE_OK;
}

bool al(const void* p, unsigned n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_attn(const lmoe_attn_dims* d, const lmoe_kv_cache* c, bool memory) {
  if (!d) return LMOE_EINVAL;
  const int rc = check_cache(c, memory);
  if (rc) return rc;
  if (d->n_requests < 1 || d->n_requests > 8192 || d->n_tokens < 1 || d->n_tokens > (1 << 20) ||
      d->max_request_tokens < 1 || d->max_request_tokens > 256 || d->q_heads < 1 || d->q_heads % c->kv_heads ||
      d->q_heads / c->kv_heads > 128 || d->max_blocks < 1 || d->max_blocks > (1 << 24) || d->mask_words < 1 ||
      d->mask_words > 4 || d->window < 0 || !(d->scale > 0.f) ||
      !(d->scale * kLog2e < INFINITY))
    return LMOE_EINVAL;
  return LMOE_OK;
}

// Rows per CTA and segment, by the most rows that a request can have per kv head.  Below 128 copies of the
// rows share the softmax's work, which pays where that is what bounds a tile: always with 64 columns, whose
// tiles are half as long to copy (16 requests of 12000 positions, 64 rows: 70 us with two copies, 91 with
// one; 64 of one token, 8 rows: 62 with two, 91 with one, 64 with four); with 128 columns up to 32 rows (64
// requests of one token: 111 us with four copies, 114 with two, 115 with one), but not from 33 on (one user's
// 8 drafts, 64 rows: 13.5 us with one, 14.4 with two).  More than 128 rows take two row tiles, so that K and V
// are read once for both; at 128 rows one is better (16 requests of 1000 to 12000 positions: 62 us, 67 with
// two).
int group_rows(const lmoe_attn_dims* d, const lmoe_kv_cache* c) {
  const int rows = d->max_request_tokens * (d->q_heads / c->kv_heads);
  if (c->head_dim == 64 && rows <= 64) return 64;
  if (c->head_dim == 128 && rows <= 32) return 32;
  return rows <= 128 ? 128 : 256;
}

// Limit of the kernel's waits: 2 to 4 seconds, and further 8192 clocks (some three times what one takes) for
// each tile of the longest request that the block table has room for.
uint32_t wait_limit(const lmoe_attn_dims* d, const lmoe_kv_cache* c) {
  return 1 + (uint32_t)(((uint64_t)d->max_blocks * c->block_size / kTile * 8192) >> 32);
}

struct AttnWs {
  size_t err, cut, ml, o, total;
};

AttnWs attn_ws(const lmoe_attn_dims* d, const lmoe_kv_cache* c, int ctas) {
  const size_t rows = group_rows(d, c);
  AttnWs w;
  size_t at = 256;  // the status word
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = (at + bytes + 255) & ~size_t(255);
    return x;
  };
  w.err = take(sizeof(Status) * ctas);
  w.cut = take(2 * sizeof(int4) * ctas);
  w.ml = take(2 * (size_t)ctas * rows * sizeof(float2));
  w.o = take(2 * (size_t)ctas * rows * c->head_dim * sizeof(float));
  w.total = at;
  return w;
}

template <int D, int NT, int KS>
int run_attn(const AttnArgs& a, const CUtensorMap (&tm)[6], int max_rows, cudaStream_t s) {
  using C = Cfg<D, NT, KS>;
  static std::atomic<unsigned long long> done{0};
  int rc = allow_smem(done, tree_attn_kernel<D, NT, KS>, C::kSmem);
  if (rc) return rc;
  rc = launch_pdl("tree_attn_kernel", dim3(a.ctas), dim3(C::kThreads), C::kSmem, s, tree_attn_kernel<D, NT, KS>, a,
                  tm[0], tm[1], tm[2], tm[3], tm[4], tm[5]);
  if (rc) return rc;
  return launch_pdl("tree_attn_merge_kernel", dim3(a.ctas, (min(max_rows, C::kRows) + 7) / 8), dim3(2 * D), 0, s,
                    tree_attn_merge_kernel<D>, a, C::kRows);
}

template <int D>
int run_attn_rows(int rows, const AttnArgs& a, const CUtensorMap (&tm)[6], int max_rows, cudaStream_t s) {
  switch (rows) {
    case 128: return run_attn<D, 1, 1>(a, tm, max_rows, s);
    case 256: return run_attn<D, 2, 1>(a, tm, max_rows, s);
    default: return run_attn<D, 1, D / 32>(a, tm, max_rows, s);  // two copies of 64 columns, four of 128
  }
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

int lmoe_kv_maps_init(const lmoe_kv_cache* cache, lmoe_kv_maps* maps) {
  const int rc = check_cache(cache, true);
  if (rc) return rc;
  if (!maps) return LMOE_EINVAL;
  return make_maps(cache, maps);
}

size_t lmoe_tree_attention_workspace_bytes(const lmoe_attn_dims* d, const lmoe_kv_cache* c) {
  if (check_attn(d, c, false) != LMOE_OK) return 0;
  DevInfo di;
  return attn_ws(d, c, dev_info(&di) == LMOE_OK ? di.sms : 152).total;
}

int lmoe_tree_attention(const lmoe_attn_dims* d, const lmoe_kv_cache* c, const uint16_t* q, int64_t q_stride,
                        const uint16_t* k_new, int64_t k_stride, const uint16_t* v_new, int64_t v_stride,
                        const int32_t* token_offsets, const int32_t* lens, const int32_t* block_table,
                        const uint64_t* mask, const int32_t* pos, uint16_t* out, float* lse, void* ws,
                        size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  int rc = check_attn(d, c, true);
  if (rc) return rc;
  const int64_t D = c->head_dim, qrow = d->q_heads * D, krow = c->kv_heads * D;
  if (!al(q, 16) || !al(k_new, 16) || !al(v_new, 16) || !al(out, 16) || !al(token_offsets, 4) || !al(lens, 4) ||
      !al(block_table, 4) || (mask && !al(mask, 8)) || (pos && !al(pos, 4)) || (lse && !al(lse, 4)) ||
      q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 || k_stride % 8 || v_stride % 8 ||
      (mask && 64 * d->mask_words < d->max_request_tokens) || !al(ws, 256))
    return LMOE_EINVAL;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  const AttnWs w = attn_ws(d, c, di.sms);
  if (ws_bytes < w.total) return LMOE_EWORKSPACE;
  // tensor maps: those of the cache, and the drafts as [token][head][d], 64 columns by 8 tokens
  CUtensorMap tm[6];
  lmoe_kv_maps own;
  const lmoe_kv_maps* maps = c->maps;
  maps_key(c, own.made_for);
  if (!maps || std::memcmp(maps->made_for, own.made_for, sizeof(own.made_for)) != 0) {
    if ((rc = make_maps(c, &own))) return rc;
    maps = &own;
  }
  std::memcpy(&tm[0], maps->map[0], sizeof(CUtensorMap));
  std::memcpy(&tm[1], maps->map[1], sizeof(CUtensorMap));
  std::memcpy(&tm[4], maps->map[2], sizeof(CUtensorMap));
  std::memcpy(&tm[5], maps->map[3], sizeof(CUtensorMap));
  const uint16_t* const fresh[2] = {k_new, v_new};
  const uint64_t step[2] = {(uint64_t)k_stride * 2, (uint64_t)v_stride * 2};
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)c->kv_heads, (uint64_t)d->n_tokens};
    const uint64_t strides[2] = {(uint64_t)D * 2, step[i]};
    const uint32_t box[3] = {64, 1, 8};
    if (encode_tmap(&tm[2 + i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, fresh[i], dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return LMOE_ECUDA;
  }
  int bs_shift = 4;
  while ((1 << bs_shift) < c->block_size) ++bs_shift;
  char* base_ws = static_cast<char*>(ws);
  AttnArgs a;
  a.q = q;
  a.v_cache = c->v;
  a.v_new = v_new;
  a.qs = q_stride;
  a.vs = v_stride;
  a.block_stride = c->block_stride;
  a.head_stride = c->head_stride;
  a.slot_stride = c->slot_stride;
  a.offsets = token_offsets;
  a.lens = lens;
  a.table = block_table;
  a.pos = pos;
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  a.status = reinterpret_cast<Status*>(base_ws);
  a.err = reinterpret_cast<Status*>(base_ws + w.err);
  a.cut = reinterpret_cast<int4*>(base_ws + w.cut);
  a.part_ml = reinterpret_cast<float2*>(base_ws + w.ml);
  a.part_o = reinterpret_cast<float*>(base_ws + w.o);
  a.B = d->n_requests;
  a.T = d->n_tokens;
  a.max_n = d->max_request_tokens;
  a.hk = c->kv_heads;
  a.G = d->q_heads / c->kv_heads;
  a.max_blocks = d->max_blocks;
  a.n_blocks = c->n_blocks;
  a.bs_shift = bs_shift;
  a.words = d->mask_words;
  a.window = d->window;
  a.ctas = di.sms;
  a.wait_limit = wait_limit(d, c);
  a.scale_log2 = d->scale * kLog2e;
  const int max_rows = a.max_n * a.G;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = group_rows(d, c);
  return D == 64 ? run_attn_rows<64>(rows, a, tm, max_rows, s) : run_attn_rows<128>(rows, a, tm, max_rows, s);
}

}  // extern "C"

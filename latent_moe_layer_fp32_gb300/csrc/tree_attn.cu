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
// CTA.  One producer warp copies K and V tiles page by page with TMA (128-byte
// swizzle) into a ring; one thread issues tcgen05.mma: S = Q K^T (both K-major
// from shared memory) into tensor memory, and O += P V with P read from tensor
// memory and V as an MN-major operand straight from its pages' layout.  Two
// softmax groups of four warps own a row per thread: they read S, keep the
// row's running maximum and sum in registers, write P (bf16, with a second
// bf16 part where one key dominates a row, in place of S) and rescale O only
// when the maximum has grown by more than 2^8 (P is then at most 2^8, which
// bf16 and the fp32 sums hold without loss).
// Up to 128 rows per kv head: the groups take turns by segment, each with its
// own queries and its own O, so one loads queries, joins and stores while the
// other computes, and S of the next tile is computed during the softmax of
// this one.  More rows: the groups take a row tile each of the same segment.
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "launch.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace lmoe {

namespace {

constexpr int kTile = 128;  // keys per tile, rows per row tile

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
  float* part_o;   // [2 CTAs][rows][D]
  int B, T, max_n, hk, G, max_blocks, n_blocks, bs_shift, words, window, ctas;
  float scale_log2;
};

// One request's share of the line of tiles: np tiles of 128 cached positions
// from base0 on (a page boundary at or below the first position in sight),
// then nd tiles of drafts.  Up to 128 drafts move in behind the cached
// positions of the last, partial tile when they fit there (at column c0, a
// multiple of 8 rows for the copies), which saves a tile of its own.
struct Req {
  int t0, n, len, base0, np, nt, c0, groups;
  bool bad;
  long long units;
  __device__ __forceinline__ int base(int i) const { return base0 + (i << 7); }
  // cached positions in tile i, the drafts in it: n_draft of them from d0 on, at columns from col on
  __device__ __forceinline__ int cached(int i) const { return i < np ? min(kTile, len - base(i)) : 0; }
  __device__ __forceinline__ int d0(int i) const { return c0 ? 0 : (i - np) << 7; }
  __device__ __forceinline__ int drafts(int i) const {
    return i < nt - 1 && i < np ? 0 : (i < np ? (c0 ? n : 0) : min(kTile, n - ((i - np) << 7)));
  }
  __device__ __forceinline__ int col(int i) const { return i < np ? c0 : 0; }
};

template <int ROWS>
__device__ __forceinline__ Req load_req(const AttnArgs& a, int b) {
  Req r;
  const int t0 = __ldg(a.offsets + b), t1 = __ldg(a.offsets + b + 1), len = __ldg(a.lens + b);
  r.bad = t0 < 0 || t1 < t0 || t1 > a.T || t1 - t0 > a.max_n || len < 0 ||
          len > ((long long)a.max_blocks << a.bs_shift);
  r.t0 = t0;
  r.n = r.bad ? 0 : t1 - t0;
  r.len = len;
  const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // the first position that any row sees
  r.base0 = lo & ~((1 << min(a.bs_shift, 7)) - 1);
  const int held = lo < len ? len - r.base0 : 0;
  r.np = (held >> 7) + ((held & 127) != 0);
  const int tail = ((held & 127) + 7) & ~7;
  r.c0 = (held & 127) != 0 && tail + r.n <= kTile ? tail : 0;
  r.nt = r.np + (r.c0 ? 0 : (r.n + kTile - 1) >> 7);
  r.groups = (r.n * a.G + ROWS - 1) / ROWS;
  r.units = (long long)a.hk * r.groups * r.nt;
  return r;
}

// The part of one segment that falls into a CTA's range.
struct Seg {
  Req r;
  int b, h, m;   // request, kv head, row group
  int i0, i1;    // tiles [i0, i1) of r.nt
  int rows;      // valid rows of this row group
};

// Walks the segments of the unit range [u, end): every role of the CTA takes the same walk.
template <int ROWS>
struct Walk {
  const AttnArgs& a;
  int b;
  long long off, left;  // units into request b, units left in the range
  Req r;
  __device__ Walk(const AttnArgs& args, int b0, long long off0, long long n) : a(args), b(b0), off(off0), left(n) {
    if (left > 0) r = load_req<ROWS>(a, b);
  }
  __device__ bool next(Seg* s) {
    if (left <= 0) return false;
    while (off >= r.units) {
      off -= r.units;
      ++b;
      r = load_req<ROWS>(a, b);
    }
    const long long k = off / r.nt;
    s->r = r;
    s->b = b;
    s->h = (int)(k / r.groups);
    s->m = (int)(k - (long long)s->h * r.groups);
    s->i0 = (int)(off - k * r.nt);
    s->i1 = (int)min((long long)r.nt, s->i0 + left);
    s->rows = min(ROWS, r.n * a.G - s->m * ROWS);
    off += s->i1 - s->i0;
    left -= s->i1 - s->i0;
    return true;
  }
};

struct RowView {
  bool valid;
  int i, p;  // draft index, position
};

__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {  // bits [lo, hi) of a 32-bit word
  const int a = min(max(lo, 0), 32), b = min(max(hi, 0), 32);
  const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
  return below_b & ~below_a;
}

// 32 bits of a row's mask from draft j on (j may be negative; bits of drafts below 0 are 0).
__device__ __forceinline__ uint32_t mask_bits(const uint64_t* m, int words, int j) {
  const int w = j >> 6, o = j & 63;  // floor
  const uint64_t lo = w >= 0 && w < words ? __ldg(m + w) : 0ull;
  uint64_t x = lo >> o;
  if (o > 32 && w + 1 >= 0 && w + 1 < words) x |= __ldg(m + w + 1) << (64 - o);
  return (uint32_t)x;
}

// What a row sees of columns 32 w .. 32 w + 31 of tile i, as bits.
__device__ __noinline__ uint32_t tile_word(const AttnArgs& a, const Seg& s, int i, int w, const RowView& v,
                                           const int* s_dpos, bool dwindow) {
  if (!v.valid) return 0u;
  const int base = s.r.base(i) + 32 * w;
  uint32_t x = range_bits(a.window > 0 ? v.p - a.window + 1 - base : 0, s.r.cached(i) - 32 * w);
  const int nd = s.r.drafts(i);
  if (nd > 0) {
    const int d0 = s.r.d0(i), c = 32 * w - s.r.col(i);  // the first column's draft is d0 + c
    uint32_t y = range_bits(-c, nd - c);
    if (a.mask)
      y &= mask_bits(a.mask + (size_t)(s.r.t0 + v.i) * a.words, a.words, d0 + c);
    else
      y &= range_bits(0, v.i - d0 - c + 1);
    if (dwindow)
      for (int j = 0; j < 32; ++j)
        if ((y >> j & 1u) && v.p - s_dpos[d0 + c + j] >= a.window) y &= ~(1u << j);
    x |= y;
  }
  return x;
}

// Adds the values that are not finite, of the keys that a row sees, to 16
// elements of its output: sanitize() took them out of the tile so that they
// reach no other row.  Runs only where there was such a value.
__device__ __noinline__ void add_not_finite(const AttnArgs& a, const Seg& s, int i, int w, uint32_t bits, int d0,
                                            int width, float* o) {
  for (; bits; bits &= bits - 1) {
    const int j = 32 * w + __ffs(bits) - 1;
    const uint16_t* v;
    if (j < s.r.cached(i)) {
      const int p = s.r.base(i) + j;
      const int id = __ldg(a.table + (size_t)s.b * a.max_blocks + (p >> a.bs_shift));
      if (id < 0 || id >= a.n_blocks) continue;
      v = a.v_cache + (size_t)id * a.block_stride + (size_t)s.h * a.head_stride +
          (size_t)(p & ((1 << a.bs_shift) - 1)) * a.slot_stride;
    } else {
      v = a.v_new + (size_t)(s.r.t0 + s.r.d0(i) + j - s.r.col(i)) * a.vs + s.h * width;
    }
#pragma unroll
    for (int d = 0; d < 16; ++d) {
      const uint32_t x = v[d0 + d];
      if ((x & 0x7f80u) == 0x7f80u) o[d] += bf16_bits_to_f32(x);
    }
  }
}

__device__ __forceinline__ bool named_bar_or(int id, int nthreads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n barrier.cta.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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
  static constexpr int kThreads = 384;                // two softmax groups, producer, MMA, two idle warps
  static constexpr int kMisc = 3072;
  static constexpr int kSmem = 2 * kQBytes + kStages * kStageBytes + kMisc;
  static constexpr uint32_t kO = 2 * kTile;           // first O column; S buffers at 0 and 128
  // the join of copies: each takes D / KS columns of the sum, in passes of kPass columns
  static constexpr int kOwn = D / KS;
  static constexpr int kPass = KS == 4 && D == 128 ? 16 : kOwn;
  static_assert(KS == 1 || kTile * (KS - 1) * kPass * 4 <= kQBytes, "room for the copies' sums");
  static_assert(kSmem <= 232448, "shared memory budget");
};

// Ring position of K and V of the CTA's tile g of n.  The groups in turns: K0 K1 V0 K2 V1 ... (S runs one
// tile ahead, also across segments); two row tiles: K0 V0 K1 V1 ...
template <int NT>
__device__ __forceinline__ uint32_t k_pos(uint32_t g) {
  return NT == 2 ? 2 * g : (g == 0 ? 0 : 2 * g - 1);
}
template <int NT>
__device__ __forceinline__ uint32_t v_pos(uint32_t g, uint32_t n) {
  return NT == 2 || g == n - 1 ? 2 * g + 1 : 2 * g + 2;
}

template <int D, int NT, int KS>
__global__ void __launch_bounds__(Cfg<D, NT, KS>::kThreads, 1)
    tree_attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap tm_k,
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
  uint64_t* s_full = empty + ST;  // [S buffer] a tile's scores are in tensor memory
  uint64_t* p_full = s_full + 2;  // [S buffer] its probabilities are
  uint64_t* pv_done = p_full + 2; // [S buffer] its product with V has been added to O
  uint64_t* q_full = pv_done + 2; // [group] the segment's queries are in shared memory
  uint64_t* s_first = q_full + 2; // [group] scores of a segment's first tile
  uint64_t* done = s_first + 2;
  long long* s_start = reinterpret_cast<long long*>(done + 1);  // request, units into it, units in the range
  unsigned long long* s_warp = reinterpret_cast<unsigned long long*>(s_start + 3);  // [threads / 32]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_warp + 12);
  volatile uint32_t* s_lo = tmem_slot + 1;  // [S buffer] a byte per warp: P has a second part
  int* s_maxpos = reinterpret_cast<int*>(tmem_slot + 3);  // [group]
  int* s_dpos = s_maxpos + 2;  // [256] positions of the drafts, with a window ([group][128] where groups take turns)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kProducer = 8, kMma = 9;
  Status* st = a.err + blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], NT * 4);
      mbar_init(&s_first[i], 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    s_start[2] = 0;
  }
  if (warp == kMma) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's range of the line of tiles ----
  if (tid == 0) *st = Status{0, 0};
  {
    const int per = (a.B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    unsigned long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const Req r = load_req<ROWS>(a, b);
      mine += r.units;
      bad |= r.bad;
    }
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    unsigned long long before = x - mine, total = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    if (bad) set_error(st, LMOE_EDEVICE_CHECK, 211);
    const unsigned long long n = min((unsigned long long)a.ctas, total);  // ranges, none of them empty
    const unsigned long long c = blockIdx.x;
    if (c < n) {
      // the threads whose requests hold the range's first and last unit
      const unsigned long long u0 = total * c / n, u1 = total * (c + 1) / n;
      auto find = [&](unsigned long long u, unsigned long long* at, Req* r) {
        *at = before;
        int b = b0;
        for (;; ++b) {
          *r = load_req<ROWS>(a, b);
          if (u < *at + r->units) return b;
          *at += r->units;
        }
      };
      unsigned long long at;
      Req r;
      if (u0 >= before && u0 < before + mine) {
        s_start[0] = find(u0, &at, &r);
        s_start[1] = (long long)(u0 - at);
        s_start[2] = (long long)(u1 - u0);
      }
      if (u1 - 1 >= before && u1 - 1 < before + mine) {
        // does the range's last segment start in it and end past it?  Then its last CTA is the
        // first one whose range ends at or after the segment's end
        find(u1 - 1, &at, &r);
        const unsigned long long k = (u1 - 1 - at) / r.nt, start = at + k * r.nt, e = start + r.nt;
        int4 c0 = make_int4(0, 0, 0, 0), c1 = c0;
        if (start >= u0 && e > u1) {
          const int h = (int)(k / r.groups), m = (int)(k % r.groups);
          const int last = (int)((e * n + total - 1) / total) - 1;
          c0 = make_int4(last - (int)c + 1, r.t0, min(ROWS, r.n * a.G - m * ROWS), h);
          c1 = make_int4(m, 0, 0, 0);
        }
        a.cut[2 * c] = c0;
        a.cut[2 * c + 1] = c1;
      }
    } else if (tid == 0) {
      a.cut[2 * c] = make_int4(0, 0, 0, 0);
    }
    __syncthreads();
  }
  const uint32_t tmem = *tmem_slot;
  const uint32_t n_tiles = (uint32_t)s_start[2];
  // 384 threads start with 168 registers each; with a whole tile's scores per thread the service
  // warps hand some of theirs to the softmax warps (88 + 2 x 208 = 3 x 168)
  auto fewer = [] {
    if constexpr (KS == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  };
  Walk<ROWS> walk(a, (int)s_start[0], s_start[1], s_start[2]);
  Seg s{};

  if (warp == kProducer) {
    // ---------------- TMA producer: one lane per page (or 8 drafts) ----------------
    fewer();
    const uint64_t pol = policy_evict_first();
    const int box = min(1 << a.bs_shift, kTile);  // rows per copy of a whole cached tile
    const int ppt = kTile / box;                  // pages per such tile
    uint32_t issued = 0;                          // copies issued
    bool ok = true;
    // the lane's copies of tile i into ring position `at`: a whole tile page by page, a partial one and
    // the drafts 8 rows at a time; `id` is the block that holds the lane's cached rows
    auto copy = [&](const CUtensorMap* tp, const CUtensorMap* t8, const CUtensorMap* td, int i, int id, uint32_t at) {
      const uint32_t stage = at % ST;
      if (!mbar_wait(&empty[stage], ((at / ST) & 1) ^ 1, st, 221)) return false;
      uint8_t* dst = s_ring + stage * C::kStageBytes;
      const int cached = s.r.cached(i);
      const int rows = cached == kTile ? box : 8;
      const int nc = cached == kTile ? ppt : (cached + 7) >> 3, nd = (s.r.drafts(i) + 7) >> 3;
      if (lane == 0) mbar_arrive_expect_tx(&full[stage], (nc * rows + nd * 8) * (128 * HALVES));
      __syncwarp();
      if (lane < nc) {
        const int slot = (s.r.base(i) + lane * rows) & ((1 << a.bs_shift) - 1);
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          tma_load_4d(dst + hf * (kTile * 128) + lane * rows * 128, rows == 8 ? t8 : tp, hf * 64, slot, s.h, id,
                      &full[stage], pol);
      } else if (lane < nc + nd) {
        const int j = (lane - nc) * 8;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
          tma_load_3d(dst + hf * (kTile * 128) + (s.r.col(i) + j) * 128, td, hf * 64, s.h, s.r.t0 + s.r.d0(i) + j,
                      &full[stage], pol);
      }
      __syncwarp();
      issued = at + 1;
      return true;
    };
    auto checked = [&](int id) {
      if (id >= 0 && id < a.n_blocks) return id;
      set_error(st, LMOE_EDEVICE_CHECK, 212);
      return a.n_blocks;  // out of the cache: the copy reads zeros
    };
    auto page = [&](int i) {  // the block of this lane's cached rows of tile i
      const int cached = s.r.cached(i), rows = cached == kTile ? box : 8;
      if (lane * rows >= cached) return 0;
      return __ldg(a.table + (size_t)s.b * a.max_blocks + ((s.r.base(i) + lane * rows) >> a.bs_shift));
    };
    uint32_t g = 0;
    if constexpr (NT == 2) {
      while (ok && walk.next(&s)) {
        int id = page(s.i0);
        for (int i = s.i0; i < s.i1 && ok; ++i, ++g) {
          const int id_next = i + 1 < s.i1 ? page(i + 1) : 0;
          id = checked(id);
          ok = copy(&tm_k, &tm_k8, &tm_kn, i, id, k_pos<NT>(g)) && copy(&tm_v, &tm_v8, &tm_vn, i, id, v_pos<NT>(g, n_tiles));
          id = id_next;
        }
      }
    } else {
      // keys one tile ahead of values, also across segments
      Seg nx{};
      int i = 0, id = 0;  // the tile whose values are still to come
      while (ok && walk.next(&nx)) {
        Seg old = s;
        s = nx;
        int id_next = page(s.i0);
        for (int k = s.i0; k < s.i1 && ok; ++k, ++g) {
          const int id_k = checked(id_next);
          id_next = k + 1 < s.i1 ? page(k + 1) : 0;
          ok = copy(&tm_k, &tm_k8, &tm_kn, k, id_k, k_pos<NT>(g));
          if (g > 0) {
            if (k == s.i0) s = old;
            ok = ok && copy(&tm_v, &tm_v8, &tm_vn, i, id, v_pos<NT>(g - 1, n_tiles));
            if (k == s.i0 || k == nx.i0) s = nx;
          }
          i = k;
          id = id_k;
        }
      }
      if (ok && g > 0) copy(&tm_v, &tm_v8, &tm_vn, i, id, v_pos<NT>(g - 1, n_tiles));
    }
    // the last copies land before the CTA can finish (also after a wait that ran out)
    if (lane == 0)
      for (uint32_t k = issued < ST ? 0 : issued - ST; k < issued; ++k) mbar_wait(&full[k % ST], (k / ST) & 1, st, 222);
  } else if (warp == kMma) {
    // ---------------- MMA issuer ----------------
    fewer();
    // the whole warp walks, so that addresses stay in uniform registers; one lane issues
    {
      const bool leader = elect_one();
      constexpr uint32_t kQk = idesc_bf16_f32(128, kTile);
      constexpr uint32_t kPv = idesc_bf16_f32(128, D) | kIdescBMnMajor;
      bool ok = true;
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
      auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
      };
      auto pv = [&](int grp, uint32_t buf, uint32_t stage, bool first) {
        const uint64_t v0 = vd + stage * (C::kStageBytes >> 4);
        const uint32_t p = tmem + buf * kTile, o = tmem + C::kO + grp * D;
        const uint32_t lo = __shfl_sync(0xffffffffu, s_lo[buf], 0);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            const uint32_t acc = !(first && kk % (8 / KS) == 0);
            if constexpr (KS == 1) {
              tc_mma_bf16_ts(o, p + kk * 8, v0 + kk * (16 * 128 >> 4), kPv, acc);
            } else {  // a 16-key step goes to the lanes whose copy of the rows holds those keys
              uint32_t off[4];
#pragma unroll
              for (int w = 0; w < 4; ++w) off[w] = w * KS / 4 == kk * KS / 8 ? 0u : 0xffffffffu;
              tc_mma_bf16_ts_lanes(o, p + kk * 8, v0 + kk * (16 * 128 >> 4), kPv, acc, off);
            }
          }
          if (lo) {  // the second part, for the warps that wrote one
#pragma unroll
            for (int c = 0; c < KS; ++c) {
              uint32_t off[4], all = 0xffffffffu;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                off[w] = w * KS / 4 == c && (lo >> (8 * w) & 1u) ? 0u : 0xffffffffu;
                all &= off[w];
              }
              if (!all) {
#pragma unroll
                for (int kk = c * 8 / KS; kk < (c + 1) * 8 / KS; ++kk)
                  tc_mma_bf16_ts_lanes(o, p + kTile / 2 + kk * 8, v0 + kk * (16 * 128 >> 4), kPv, 1u, off);
              }
            }
          }
          tc_commit(&pv_done[buf]);
        }
        __syncwarp();
      };
      auto tile = [&](uint32_t at) {  // the tile at ring position `at` has landed
        if (!mbar_wait(&full[at % ST], (at / ST) & 1, st, 231)) return false;
        tc_fence_after();
        return true;
      };
      if constexpr (NT == 1) {
        uint32_t g = 0, seg = 0;
        auto first_qk = [&](uint32_t sg, uint32_t gt) {  // scores of segment sg's first tile gt
          const uint32_t at = k_pos<1>(gt);
          if (!mbar_wait(&q_full[sg & 1], (sg >> 1) & 1, st, 232) || !tile(at)) return false;
          tc_fence_after();
          qk(sg & 1, gt & 1, at % ST);
          commit(&s_first[sg & 1]);
          commit(&empty[at % ST]);
          return true;
        };
        bool more = walk.next(&s);
        if (more) ok = first_qk(0, 0);
        while (ok && more) {
          const int n = s.i1 - s.i0;
          more = walk.next(&s);
          for (int k = 0; k < n; ++k, ++g) {
            if (k + 1 < n) {
              const uint32_t at = k_pos<1>(g + 1);
              if (!(ok = tile(at))) break;
              qk(seg & 1, (g + 1) & 1, at % ST);
              commit(&empty[at % ST]);
            } else if (more && !(ok = first_qk(seg + 1, g + 1))) {
              break;
            }
            const uint32_t at = v_pos<1>(g, n_tiles);
            if (!(ok = tile(at)) || !(ok = mbar_wait(&p_full[g & 1], (g >> 1) & 1, st, 233))) break;
            tc_fence_after();
            pv(seg & 1, g & 1, at % ST, k == 0);
            commit(&empty[at % ST]);
          }
          ++seg;
        }
      } else {
        uint32_t g = 0, seg = 0, g1 = 0;  // g1: tiles of row tile 1 so far
        while (ok && walk.next(&s)) {
          const int n = s.i1 - s.i0;
          const bool two = s.rows > kTile;
          uint32_t ka = k_pos<2>(g);
          if (!(ok = mbar_wait(q_full, seg & 1, st, 232)) || !(ok = tile(ka))) break;
          tc_fence_after();
          qk(0, 0, ka % ST);
          if (two) qk(1, 1, ka % ST);
          commit(&empty[ka % ST]);
          for (int k = 0; k < n; ++k, ++g) {
            const uint32_t va = v_pos<2>(g, n_tiles);
            ka = k_pos<2>(g + 1);
            if (!(ok = tile(va)) || !(ok = mbar_wait(&p_full[0], g & 1, st, 233))) break;
            tc_fence_after();
            pv(0, 0, va % ST, k == 0);
            if (k + 1 < n) {
              if (!(ok = tile(ka))) break;
              qk(0, 0, ka % ST);
            }
            if (two) {
              if (!(ok = mbar_wait(&p_full[1], g1++ & 1, st, 234))) break;
              tc_fence_after();
              pv(1, 1, va % ST, k == 0);
            }
            commit(&empty[va % ST]);
            if (k + 1 < n) {
              if (two) qk(1, 1, ka % ST);
              commit(&empty[ka % ST]);
            }
          }
          ++seg;
        }
      }
      commit(done);  // every MMA issued has completed before TMEM is released
      mbar_wait(done, 0, st, 235);
    }
  } else if (warp < kProducer) {
    // ---------------- softmax: one row per thread ----------------
    if constexpr (KS == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    constexpr int CW = C::kCols;
    const int grp = warp >> 2, row = tid & 127;  // group, row of its row tile
    const int part = KS == 1 ? 0 : row / (kTile / KS);  // which copy of the rows: keys part * CW .. + CW of each tile
    const int local = (NT == 2 ? grp * kTile : 0) + (KS == 1 ? row : row % (kTile / KS));  // row of the row group
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_base + C::kO + grp * D;
    uint8_t* const q_buf = s_q + grp * C::kQBytes;
    int* const dpos = s_dpos + (NT == 2 ? 0 : grp * 128);
    int* const maxpos = s_maxpos + (NT == 2 ? 0 : grp);
    const int bar_seg = NT == 2 ? 3 : 4 + grp;    // barrier of the segment's threads
    uint32_t seg = 0, g = 0, g_own = 0;           // segments and tiles of the CTA so far; tiles of this group
    // After a wait that ran out the warp goes on without waiting: what it writes is void, but
    // the barriers between the warps stay complete and the CTA ends.
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
      if (ok) ok = mbar_wait(bar, parity, st, where);
      tc_fence_after();
    };
    auto edge_tile = [&](int i) {  // the prefix's end, drafts, and where a window cuts
      return i >= s.r.np || s.r.cached(i) < kTile || (a.window > 0 && s.r.base(i) < *maxpos - a.window + 1);
    };
    for (; walk.next(&s); ++seg) {
      const int n = s.i1 - s.i0;
      if (NT == 1 && (int)(seg & 1) != grp) {
        g += n;
        continue;
      }
      const bool two = NT == 2 && s.rows > kTile;
      const int group = two ? 256 : 128;  // threads that take part in this segment's edge tiles
      RowView v;
      v.valid = local < s.rows;
      const int rr = s.m * C::kRows + local;
      v.i = v.valid ? rr / a.G : 0;
      const int qh = s.h * a.G + (rr - v.i * a.G), tok = s.r.t0 + v.i;
      v.p = s.r.len + v.i;
      const bool warp_live = __any_sync(0xffffffffu, v.valid);
      bool dwindow = false;  // some pair of drafts may be a window apart
      if (a.window > 0) {
        if (v.valid && a.pos) v.p = max(__ldg(a.pos + tok), s.r.len);
        named_bar(bar_seg, NT * 128);
        for (int j = NT == 2 ? tid : row; j < s.r.n; j += NT * 128)
          dpos[j] = a.pos ? max(__ldg(a.pos + s.r.t0 + j), s.r.len) : s.r.len + j;
        if (row == 0) *maxpos = 0;
        named_bar(bar_seg, NT * 128);
        const int top = __reduce_max_sync(0xffffffffu, v.valid ? v.p : 0);
        if (lane == 0) atomicMax(maxpos, top);
        named_bar(bar_seg, NT * 128);
        dwindow = *maxpos - s.r.len >= a.window;
      }
      // queries: the thread's row, 16 bytes at a time, in the swizzled K-major layout
      if (warp_live) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (size_t)tok * a.qs + (size_t)qh * D);
        uint8_t* dst = q_buf + row * 128;
        uint4 w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = v.valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTile * 128) + (((c & 7) ^ (row & 7)) << 4)) = w[c];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[NT == 2 ? 0 : grp]);
      if (NT == 2 && grp == 1 && !two) {
        // no rows here: only keep in step with the segments
        wait(q_full, seg & 1, 241);
        g += n;
        continue;
      }
      float m_ref = -INFINITY, l = 0.f;
      bool dirty = false;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int i = s.i0 + k;
        const uint32_t gt = g + k, go = g_own + k;
        const uint32_t buf = NT == 1 ? gt & 1 : grp;
        if (NT == 1 && k == 0)
          wait(&s_first[grp], (seg >> 1) & 1, 240);  // s_full may be phases behind until then
        else
          wait(&s_full[buf], NT == 1 ? (gt >> 1) & 1 : go & 1, 242);
        const bool edge = edge_tile(i);
        const uint32_t s_addr = tmem + lane_base + buf * kTile;
        bool lo = false;
        if (warp_live) {
          if (edge) {
            // unseen keys' scores become -infinity, in place
#pragma unroll 1
            for (int c = 0; c < CW / 32; ++c) {
              const uint32_t addr = s_addr + part * CW + c * 32;
              const uint32_t bits = tile_word(a, s, i, part * (CW / 32) + c, v, dpos, dwindow);
              uint32_t y[32];
              tmem_ld32(addr, y);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(bits >> j & 1u)) y[j] = 0xff800000u;
              tmem_st32(addr, y);
            }
            tmem_st_wait();
          }
          uint32_t sv[CW];
          auto load = [&] {
#pragma unroll
            for (int c = 0; c < CW / 32; ++c)
              tmem_ld32(s_addr + part * CW + c * 32, *reinterpret_cast<uint32_t(*)[32]>(sv + c * 32));
            tmem_ld_wait();
          };
          load();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < CW; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(sv[j]));
          const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
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
          // P as one bf16 part is off by up to 2^-8 of each key's share.  Where some key of a row
          // holds over 1/16 of the row's sum so far that would show in the output next to its own
          // rounding, so the remainder goes along as a second part; with more keys in play it
          // averages out.  After a prefix's first tiles this is rare.
          lo = __any_sync(0xffffffffu, v.valid && ex2(m_new - mu) > l * 0.0625f);
          // p = 2^(scale s - mu) in one fused step, whose error against the rounded mu is common to
          // the row.  Past 2^24 that error alone could overflow: there scale s is rounded first too.
          float sc = a.scale_log2;
          if (__any_sync(0xffffffffu, fabsf(mu) > 16777216.f)) {
#pragma unroll 1
            for (int c = 0; c < CW / 16; ++c) {
              uint32_t y[16];
              tmem_ld16(s_addr + part * CW + c * 16, y);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * sc);
              tmem_st16(s_addr + part * CW + c * 16, y);
            }
            tmem_st_wait();
            load();
            sc = 1.f;
          }
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          auto exps = [&](bool two_parts) {
#pragma unroll
            for (int c = 0; c < CW / 32; ++c) {
              uint32_t p[16], p2[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float e0 = ex2(fmaf(__uint_as_float(sv[c * 32 + 2 * j]), sc, -mu));
                const float e1 = ex2(fmaf(__uint_as_float(sv[c * 32 + 2 * j + 1]), sc, -mu));
                sum[(2 * j) & 3] += e0;
                sum[(2 * j + 1) & 3] += e1;
                p[j] = pack_bf16(e0, e1);
                if (two_parts)
                  p2[j] = pack_bf16(e0 - __uint_as_float(p[j] << 16), e1 - __uint_as_float(p[j] & 0xffff0000u));
              }
              tmem_st16(s_addr + part * (CW / 2) + c * 16, p);
              if (two_parts) tmem_st16(s_addr + kTile / 2 + part * (CW / 2) + c * 16, p2);
            }
          };
          if (lo)
            exps(true);
          else
            exps(false);
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st_wait();
        }
        if (lane == 0) reinterpret_cast<volatile uint8_t*>(s_lo + buf)[warp & 3] = lo;
        if (edge) {
          // values that no row sees become zero, and those that are not finite too (0 * NaN would
          // reach every row): they are added back to the rows that see them at the end
          const uint32_t at = v_pos<NT>(gt, n_tiles);
          wait(&full[at % ST], (at / ST) & 1, 244);
          uint8_t* vt = s_ring + (at % ST) * C::kStageBytes;
          const int hi = s.r.cached(i), c0 = s.r.col(i), c1 = c0 + s.r.drafts(i);
          const int first = a.window > 0 ? s.r.len - a.window + 1 - s.r.base(i) : 0;
          bool found = false;
          for (int c = two ? tid : row; c < kTile * HALVES * 8; c += group) {
            const int key = (c >> 3) & (kTile - 1);
            uint4* w = reinterpret_cast<uint4*>(vt + (c << 4));
            if (!((key >= first && key < hi) || (key >= c0 && key < c1))) {
              *w = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            uint4 y = *w;
            uint32_t* e = &y.x;
            bool change = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if ((e[j] & 0x7f80u) == 0x7f80u) e[j] &= 0xffff0000u, change = true;
              if ((e[j] & 0x7f800000u) == 0x7f800000u) e[j] &= 0xffffu, change = true;
            }
            if (change) {
              *w = y;
              found = true;
            }
          }
          fence_proxy_async_smem();
          dirty |= named_bar_or(two ? 6 : 1 + grp, group, found);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // ---- the segment's end: finished rows to out, cut ones to the partial sums ----
      const uint32_t ge = NT == 1 ? g + n - 1 : g_own + n - 1;  // the segment's last tile
      wait(&pv_done[NT == 1 ? ge & 1 : grp], NT == 1 ? (ge >> 1) & 1 : ge & 1, 245);
      const bool whole = s.i0 == 0 && s.i1 == s.r.nt;
      const size_t prow = (size_t)(2 * blockIdx.x + (s.i0 == 0)) * C::kRows + local;
      // 16 columns of this thread's row of O
      auto sums = [&](int col, float (&y)[16]) {
        uint32_t o[16];
        tmem_ld16(o_addr + col, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(o[j]);
        if (dirty && v.valid) {
          float z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = y[j];
          for (int i = s.i0; i < s.i1; ++i)
            if (edge_tile(i))
              for (int w = 0; w < CW / 32; ++w)
                add_not_finite(a, s, i, part * (CW / 32) + w,
                               tile_word(a, s, i, part * (CW / 32) + w, v, dpos, dwindow), col, D, z);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = z[j];
        }
      };
      auto put = [&](int col, const float (&y)[16], float inv) {
        if (!v.valid) return;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)tok * (a.hk * a.G) + qh) * D + col);
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = pack_bf16(y[2 * j] * inv, y[2 * j + 1] * inv);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_o + prow * D + col);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
      };
      if constexpr (KS == 1) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
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
        named_bar(1 + grp, 128);
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
        named_bar(1 + grp, 128);
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        auto piece = [&](int owner, int from, int j) {
          const int x = P == 16 ? (local >> 1) & 3 : local & 7;
          return reinterpret_cast<float4*>(
              q_buf + ((owner * (KS - 1) + (from > owner ? from - 1 : from)) * RP + local) * (P * 4) + ((j ^ x) << 4));
        };
#pragma unroll 1
        for (int q = 0; q < OWN; q += P) {
          if (q > 0) named_bar(1 + grp, 128);
          if (warp_live) {
#pragma unroll 1
            for (int d = 1; d < KS; ++d) {
              const int owner = (part + d) % KS;
#pragma unroll 1
              for (int c = 0; c < P; c += 16) {
                float y[16];
                sums(owner * OWN + q + c, y);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  *piece(owner, part, c / 4 + j) =
                      make_float4(y[4 * j] * f, y[4 * j + 1] * f, y[4 * j + 2] * f, y[4 * j + 3] * f);
              }
            }
          }
          named_bar(1 + grp, 128);
          if (warp_live) {
#pragma unroll 1
            for (int c = 0; c < P; c += 16) {
              float y[16];
              sums(part * OWN + q + c, y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] *= f;
#pragma unroll
              for (int d = 1; d < KS; ++d) {
                const int from = (part + d) % KS;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float4 z = *piece(part, from, c / 4 + j);
                  y[4 * j] += z.x;
                  y[4 * j + 1] += z.y;
                  y[4 * j + 2] += z.z;
                  y[4 * j + 3] += z.w;
                }
              }
              put(part * OWN + q + c, y, inv);
            }
          }
        }
        named_bar(1 + grp, 128);  // the next queries overwrite the buffer
      }
      if (v.valid && part == 0) {
        if (!whole)
          a.part_ml[prow] = make_float2(m_ref, l);
        else if (a.lse)
          a.lse[(size_t)tok * (a.hk * a.G) + qh] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
      }
      g += n;
      g_own += n;
    }
  } else {
    fewer();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of each cut segment, one warp per row: block x is the CTA in
// whose range a segment starts, its pieces lie in that CTA's tail slot and the
// head slots of the CTAs after it.
//   M = max m_i,  L = sum l_i 2^(m_i - M),  out = sum O_i 2^(m_i - M) / L
template <int D>
__global__ void __launch_bounds__(256) tree_attn_merge_kernel(const AttnArgs a, int rows) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {  // the call's status: the first CTA's error
    Status e{0, 0};
    for (int c = lane; c < a.ctas; c += 32) {
      const Status x = a.err[c];
      if (e.code == 0) e = x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, e.code != 0);
    const int from = hit ? __ffs(hit) - 1 : 0;
    e.code = __shfl_sync(0xffffffffu, e.code, from);
    e.where = __shfl_sync(0xffffffffu, e.where, from);
    if (lane == 0) *a.status = e;
  }
  const int4 c0 = a.cut[2 * blockIdx.x];
  const int pieces = c0.x, local = blockIdx.y * 8 + warp;
  if (pieces < 2 || local >= c0.z) return;
  const int rr = a.cut[2 * blockIdx.x + 1].x * rows + local;
  const int i = rr / a.G, tok = c0.y + i, qh = c0.w * a.G + rr - i * a.G;
  auto slot = [&](int p) { return (size_t)(p == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + p)) * rows + local; };
  float M = -INFINITY;
  for (int p = lane; p < pieces; p += 32) M = fmaxf(M, a.part_ml[slot(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  constexpr int E = D / 32;
  float acc[E] = {}, L = 0.f;
  for (int p0 = 0; p0 < pieces; p0 += 32) {
    float w = 0.f, lw = 0.f;
    if (p0 + lane < pieces) {
      const float2 ml = a.part_ml[slot(p0 + lane)];
      w = ex2(ml.x - mu);
      lw = w * ml.y;
    }
    L += warp_sum(lw);
    const int np = min(32, pieces - p0);
#pragma unroll 4
    for (int p = 0; p < np; ++p) {
      const float wp = __shfl_sync(0xffffffffu, w, p);
      const float* o = a.part_o + slot(p0 + p) * D + lane * E;
      if constexpr (E == 4) {
        const float4 y = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(wp, y.x, acc[0]);
        acc[1] = fmaf(wp, y.y, acc[1]);
        acc[2] = fmaf(wp, y.z, acc[2]);
        acc[3] = fmaf(wp, y.w, acc[3]);
      } else {
        const float2 y = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(wp, y.x, acc[0]);
        acc[1] = fmaf(wp, y.y, acc[1]);
      }
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((size_t)tok * (a.hk * a.G) + qh) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[(size_t)tok * (a.hk * a.G) + qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
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

// Rows per CTA and segment, by the most rows that a request can have per kv head.
int group_rows(const lmoe_attn_dims* d, const lmoe_kv_cache* c) {
  const int rows = d->max_request_tokens * (d->q_heads / c->kv_heads);
  return rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
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
  return launch_pdl("tree_attn_merge_kernel", dim3(a.ctas, (min(max_rows, C::kRows) + 7) / 8), dim3(256), 0, s,
                    tree_attn_merge_kernel<D>, a, C::kRows);
}

template <int D>
int run_attn_rows(int rows, const AttnArgs& a, const CUtensorMap (&tm)[6], int max_rows, cudaStream_t s) {
  switch (rows) {
    case 32: return run_attn<D, 1, 4>(a, tm, max_rows, s);
    case 64: return run_attn<D, 1, 2>(a, tm, max_rows, s);
    case 128: return run_attn<D, 1, 1>(a, tm, max_rows, s);
    default: return run_attn<D, 2, 1>(a, tm, max_rows, s);
  }
}

}  // namespace

}  // namespace lmoe

using namespace lmoe;

extern "C" {

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
  // tensor maps: the cache as [block][head][slot][d], copied 64 columns by one page (at most a
  // tile) or by 8 slots at a time; the drafts as [token][head][d], 64 columns by 8 tokens
  CUtensorMap tm[6];
  const uint16_t* const base[4] = {c->k, c->v, k_new, v_new};
  const uint64_t step[2] = {(uint64_t)k_stride * 2, (uint64_t)v_stride * 2};
  // a dimension of extent 1 never steps: any valid stride will do
  auto stride = [](int64_t elements, int64_t extent) { return (uint64_t)(extent > 1 ? elements : 64) * 2; };
  for (int i = 0; i < 2; ++i) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)c->block_size, (uint64_t)c->kv_heads, (uint64_t)c->n_blocks};
    const uint64_t strides[3] = {stride(c->slot_stride, c->block_size), stride(c->head_stride, c->kv_heads),
                                 stride(c->block_stride, c->n_blocks)};
    const uint32_t box[4] = {64, (uint32_t)min(c->block_size, kTile), 1, 1};
    if (encode_tmap(&tm[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base[i], dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return LMOE_ECUDA;
    const uint32_t box8[4] = {64, 8, 1, 1};
    if (encode_tmap(&tm[4 + i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base[i], dims, strides, box8,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return LMOE_ECUDA;
    const uint64_t ndims[3] = {(uint64_t)D, (uint64_t)c->kv_heads, (uint64_t)d->n_tokens};
    const uint64_t nstrides[2] = {(uint64_t)D * 2, step[i]};
    const uint32_t nbox[3] = {64, 1, 8};
    if (encode_tmap(&tm[2 + i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base[2 + i], ndims, nstrides, nbox,
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
  a.scale_log2 = d->scale * 1.4426950408889634f;
  const int max_rows = a.max_n * a.G;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rows = group_rows(d, c);
  return D == 64 ? run_attn_rows<64>(rows, a, tm, max_rows, s) : run_attn_rows<128>(rows, a, tm, max_rows, s);
}

}  // extern "C"

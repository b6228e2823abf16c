// The paged key/value cache's bookkeeping: tree masks of drafted tokens, block
// tables and slots from request lengths, and the write of rows into slots.
// See include/lmoe.h for the contract of every call.
//
// All three move few bytes, so what bounds them is the launch and the chain of
// dependent loads, except the write of a prompt, which is a copy.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.cuh"

namespace lmoe {

namespace {

// ---------------------------------------------------------------------------
// tree masks
// ---------------------------------------------------------------------------
// One CTA per request, one thread per drafted row.  Ancestor sets by pointer
// doubling: after round r a row's mask holds its nearest 2^r ancestors-or-self
// and up points past them, so ceil(log2 n) rounds close any tree and the loop
// ends as soon as every pointer has left the tree.  A chain of dependent loads
// and rounds bounds it: 8 drafts take 1.8 us, 1024 trees of up to 200 drafts
// (4.1 MB) 5.5 us.  Those are one wave (eight CTAs fit an SM); their warps wait at
// the rounds' barriers first, next for the parents' loads, and shared memory is
// busy for half of the time that an SM works.  Masks are stored 16 bytes at a time
// where they are aligned (5.5 instead of 6.1 us).
template <int W>
__global__ void __launch_bounds__(64 * W)
    tree_masks_kernel(int n_tokens, const int32_t* __restrict__ offsets, const int32_t* __restrict__ parents,
                      const int32_t* __restrict__ lens, uint64_t* __restrict__ mask, int32_t* __restrict__ pos,
                      Status* st) {
  constexpr int N = 64 * W;
  __shared__ uint64_t s_mask[2][W][N];
  __shared__ int s_up[2][N];
  __shared__ int s_depth[2][N];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, i = threadIdx.x;
  const int t0 = offsets[b], t1 = offsets[b + 1];
  const int len = lens ? lens[b] : 0;
  if (t0 < 0 || t1 < t0 || t1 > n_tokens) {
    if (i == 0) set_error(st, LMOE_EDEVICE_CHECK, 201);
    return;
  }
  const int n = t1 - t0;
  if (n > N) {
    if (i == 0) set_error(st, LMOE_EDEVICE_CHECK, 202);
    for (int r = i; r < n; r += N) {
      for (int w = 0; w < W; ++w) mask[(size_t)(t0 + r) * W + w] = 0;
      pos[t0 + r] = len;
    }
    return;
  }
  int up = -1;
  if (i < n) {
    up = parents[t0 + i];
    if (up >= i || up < -1) {
      set_error(st, LMOE_EDEVICE_CHECK, 203);
      up = -1;
    }
  }
  uint64_t m[W];
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = (i >> 6) == w ? 1ull << (i & 63) : 0ull;
  int depth = 0;  // ancestors counted so far
  int span = up >= 0 ? 1 : 0;
  int cur = 0;
  while (__syncthreads_or(up >= 0)) {
#pragma unroll
    for (int w = 0; w < W; ++w) s_mask[cur][w][i] = m[w];
    s_up[cur][i] = up;
    s_depth[cur][i] = span;
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) m[w] |= s_mask[cur][w][up];
      span += s_depth[cur][up];
      up = s_up[cur][up];
    }
    cur ^= 1;
  }
  depth = span;
  if (i < n) {
    uint64_t* const row = mask + (size_t)(t0 + i) * W;
    if (W % 2 == 0 && (reinterpret_cast<uintptr_t>(mask) & 15u) == 0) {
#pragma unroll
      for (int w = 0; w + 1 < W; w += 2) *reinterpret_cast<ulonglong2*>(row + w) = make_ulonglong2(m[w], m[w + 1]);
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) row[w] = m[w];
    }
    pos[t0 + i] = len + depth;
  }
}

// ---------------------------------------------------------------------------
// block plan
// ---------------------------------------------------------------------------
constexpr int kPlanMaxRequests = 8192;

struct PlanArgs {
  int B, bs, max_blocks, n_slots, ring_size;
  const int32_t *lens, *add, *owned, *ring_state;
  int32_t *table, *ring, *lens_out, *owned_out, *ring_state_out, *offsets, *slots;
  bool wide;  // lens, add and owned are 16-byte aligned
};

// ceil of (len + add) / bs, at most one past the table; a sum past 31 bits fits no table (lengths and positions
// are int32)
__device__ __forceinline__ int blocks_for(int len, int add, int bs, int max_blocks) {
  const unsigned held = (unsigned)len + (unsigned)add, q = held / (unsigned)bs;
  return held > 0x7fffffffu ? max_blocks + 1 : (int)min(q + (held != q * (unsigned)bs), (unsigned)max_blocks + 1u);
}

// Sum of v over the threads before this one, and over all in *total.
template <int NT>
__device__ __forceinline__ unsigned long long scan_excl(unsigned long long v, unsigned long long* s_warp,
                                                        unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  unsigned long long w = lane < NT / 32 ? s_warp[lane] : 0ull;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, NT / 32 - 1);
  const unsigned long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return x - v + (warp ? before : 0ull);
}

// Four ints at 16-byte aligned places (or in registers).
__device__ __forceinline__ void copy4(int* to, const int* from) {
  *reinterpret_cast<int4*>(to) = *reinterpret_cast<const int4*>(from);
}
// Ints of each per-request array in shared memory: B + 1 at least, in whole fours.
__host__ __device__ constexpr int plan_ints(int b) { return (b + 4) & ~3; }

// (head + i) % size for a head and an i below size
__device__ __forceinline__ int ring_at(int head, long long i, int size) {
  const long long x = head + i;
  return (int)(x >= size ? x - size : x);
}

// Every CTA scans all requests itself (L2-resident lengths, a run of up to 8 requests per thread, two block
// scans) and keeps what a token needs of its request in shared memory; then it takes its share of the
// requests (a warp each) and of the tokens (a thread each, its request found by bisection).  Nothing is
// passed between CTAs, so one launch does it.  What bounds it is the chain of dependent loads and the shared
// memory accesses of the scan: 4096 requests with 76000 tokens take 8.6 us, 8 requests 2.8 us (with a scan per
// 1024 requests and lengths fetched again per token: 14.9 and 4.0 us; with a run's values moved one by one
// instead of four at a time: 9.6 us).
template <int NT, int PER>
__global__ void __launch_bounds__(NT) kv_plan_kernel(const PlanArgs a) {
  extern __shared__ __align__(16) int s_plan[];
  const int held_n = plan_ints(a.B);  // of each array, a multiple of 4
  int* s_tok = s_plan;                // [B + 1] first token of each request, at most n_slots
  int* s_pop = s_tok + held_n;        // [B] blocks popped by the requests before it; -1: not served
  int* s_push = s_pop + held_n;       // [B] blocks pushed by the requests before it; -1: it does not end
  int* s_len = s_push + held_n;       // [B] tokens held
  int* s_own = s_len + held_n;        // [B] blocks held
  __shared__ unsigned long long s_warp[32];
  __shared__ int s_taken;
  pdl_wait();
  pdl_trigger();
  const int b0 = threadIdx.x * PER;
  alignas(16) int add[PER], len[PER], own[PER];  // all at once: one trip to memory
  if (PER % 4 == 0 && a.wide && b0 + PER <= a.B) {
#pragma unroll
    for (int j = 0; j < PER; j += 4) {
      copy4(add + j, a.add + b0 + j);
      copy4(len + j, a.lens + b0 + j);
      copy4(own + j, a.owned + b0 + j);
    }
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const bool in = b0 + j < a.B;
      add[j] = in ? a.add[b0 + j] : 0;
      len[j] = in ? a.lens[b0 + j] : 0;
      own[j] = in ? a.owned[b0 + j] : 0;
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    len[j] = max(len[j], 0);
    own[j] = min(max(own[j], 0), a.max_blocks);
  }
  const int head = a.ring_state[0], count = min(max(a.ring_state[1], 0), a.ring_size);
  const int hd = head < 0 || head >= a.ring_size ? 0 : head;
  if (threadIdx.x == 0) s_taken = 0;
  unsigned long long sum = 0, n_tok, n_both;
#pragma unroll
  for (int j = 0; j < PER; ++j) sum += (unsigned)max(add[j], 0);
  unsigned long long t0 = scan_excl<NT>(sum, s_warp, &n_tok);
  // blocks asked for (high half) and given back (low half) by the requests that fit
  unsigned long long at = t0, both = 0;
  int need[PER];
  unsigned fit = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int more = max(add[j], 0), after = blocks_for(len[j], more, a.bs, a.max_blocks);
    const bool fits = add[j] >= 0 && after <= a.max_blocks && at + more <= (unsigned long long)a.n_slots;
    need[j] = fits ? max(after - own[j], 0) : 0;
    fit |= (unsigned)fits << j;
    at += more;
    both += (unsigned long long)need[j] << 32 | (unsigned)(add[j] < 0 ? own[j] : 0);
  }
  both = scan_excl<NT>(both, s_warp, &n_both);
  int taken = 0;
  alignas(16) int tok[PER], popped[PER], pushed[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int b = b0 + j;
    const unsigned long long pop = both >> 32;
    const bool served = (fit >> j & 1u) && (need[j] == 0 || pop + need[j] <= (unsigned long long)count);
    if (served && need[j] > 0) taken = (int)(pop + need[j]);
    tok[j] = (int)min(t0, (unsigned long long)a.n_slots);
    popped[j] = served ? (int)min(pop, 0x7fffffffull) : -1;
    pushed[j] = add[j] < 0 ? (int)(both & 0xffffffffu) : -1;
    if (blockIdx.x == 0 && b < a.B) a.offsets[b] = (int)min(t0, 0x7fffffffull);
    t0 += max(add[j], 0);
    both += (unsigned long long)need[j] << 32 | (unsigned)(add[j] < 0 ? own[j] : 0);
  }
  // (past the last request: nothing asked for, the total's token; the arrays have room for whole fours)
  if constexpr (PER % 4 == 0) {
#pragma unroll
    for (int j = 0; j < PER; j += 4)
      if (b0 + j < a.B) {
        copy4(s_tok + b0 + j, tok + j);
        copy4(s_pop + b0 + j, popped + j);
        copy4(s_push + b0 + j, pushed + j);
        copy4(s_len + b0 + j, len + j);
        copy4(s_own + b0 + j, own + j);
      }
  } else if (b0 < a.B) {
    s_tok[b0] = tok[0];
    s_pop[b0] = popped[0];
    s_push[b0] = pushed[0];
    s_len[b0] = len[0];
    s_own[b0] = own[0];
  }
  if (taken > 0) atomicMax(&s_taken, taken);
  if (threadIdx.x == 0) {
    s_tok[a.B] = (int)min(n_tok, (unsigned long long)a.n_slots);
    if (blockIdx.x == 0) a.offsets[a.B] = (int)min(n_tok, 0x7fffffffull);
  }
  __syncthreads();
  const int room = a.ring_size - count;  // ring entries that hold no free block
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const int back = (int)min(n_both & 0xffffffffull, (unsigned long long)room);
    a.ring_state_out[0] = ring_at(hd, s_taken, a.ring_size);
    a.ring_state_out[1] = count - s_taken + back;
  }
  const int lane = threadIdx.x & 31;
  for (int b = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); b < a.B; b += gridDim.x * (NT / 32)) {
    int32_t* row = a.table + (size_t)b * a.max_blocks;
    const int owned = s_own[b], push = s_push[b], pop = s_pop[b], held = s_len[b];
    if (push >= 0) {  // it ends
      for (int j = lane; j < owned && push + j < room; j += 32)
        a.ring[ring_at(hd, (long long)count + push + j, a.ring_size)] = row[j];
      if (lane == 0) a.lens_out[b] = a.owned_out[b] = 0;
    } else if (pop >= 0) {
      const int more = s_tok[b + 1] - s_tok[b], after = max(blocks_for(held, more, a.bs, a.max_blocks), owned);
      for (int j = lane; j < after - owned; j += 32) row[owned + j] = a.ring[ring_at(hd, pop + j, a.ring_size)];
      if (lane == 0) {
        a.lens_out[b] = held + more;
        a.owned_out[b] = after;
      }
    } else if (lane == 0) {
      a.lens_out[b] = a.lens[b];
      a.owned_out[b] = a.owned[b];
    }
  }
  // a token's slot: from the table for a block held before the call, else straight from the ring
  const int last = s_tok[a.B];
  // (unsigned: a step past the last slot may pass 31 bits)
  for (unsigned x = blockIdx.x * NT + threadIdx.x; x < (unsigned)a.n_slots; x += gridDim.x * NT) {
    const int t = (int)x;
    int slot = -1;
    if (t < last) {
      int lo = 0, hi = a.B - 1;  // the last request whose first token is at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tok[mid] <= t) lo = mid; else hi = mid - 1;
      }
      if (s_pop[lo] >= 0) {
        const int p = s_len[lo] + t - s_tok[lo], blk = p / a.bs, owned = s_own[lo];
        const int id = blk < owned ? a.table[(size_t)lo * a.max_blocks + blk]
                                   : a.ring[ring_at(hd, (long long)s_pop[lo] + blk - owned, a.ring_size)];
        const long long at = (long long)id * a.bs + (p - blk * a.bs);
        slot = id >= 0 && at <= 0x7fffffff ? (int)at : -1;
      }
    }
    a.slots[t] = slot;
  }
}

// Threads per CTA and requests per thread for B requests: few threads meet sooner (8 requests: 2.8 us with
// 256, 3.7 with 1024), more than 256 requests need more of them.  A CTA per NT / 32 requests (its warps' one
// round) or NT tokens, whichever asks for more.
template <int NT, int PER>
int run_plan(const PlanArgs& a, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  const int rc = allow_smem(done, kv_plan_kernel<NT, PER>, 5 * plan_ints(NT * PER) * 4);
  if (rc) return rc;
  const int want = max((a.B + NT / 32 - 1) / (NT / 32), (int)((a.n_slots + NT - 1ll) / NT));
  return launch_pdl("kv_plan_kernel", dim3(min(want, sms)), dim3(NT), 5 * (size_t)plan_ints(a.B) * 4, s,
                    kv_plan_kernel<NT, PER>, a);
}

// ---------------------------------------------------------------------------
// slot writes
// ---------------------------------------------------------------------------
// A thread moves one 16-byte piece of a row's K and the same of its V.  A prompt's write is a copy, bound by
// HBM: 16384 tokens of 8 heads of 128 columns (134 MB moved) take 22.6 us, 5950 GB/s (22.8 with a grid of 16
// CTAs an SM that loops; two or four pieces a thread: 22.3, but 211 accepted rows 2.4 and 3.2 us instead of 1.9).
__global__ void __launch_bounds__(256)
    kv_write_kernel(const lmoe_kv_cache c, const uint16_t* __restrict__ k_new, long long ks,
                    const uint16_t* __restrict__ v_new, long long vs, int n_rows, const int32_t* __restrict__ src,
                    const int32_t* __restrict__ slots, int n_tokens, int pieces, int bs_shift, int d_shift,
                    Status* st) {
  pdl_wait();
  pdl_trigger();
  const unsigned x = blockIdx.x * 256u + threadIdx.x;
  if (x >= (unsigned)n_tokens * (unsigned)pieces) return;
  const unsigned t = x / (unsigned)pieces, p = x - t * (unsigned)pieces;
  const int slot = slots[t];
  if (slot < 0) return;
  const int row = src ? src[t] : (int)t;
  const int block = slot >> bs_shift;
  if (block >= c.n_blocks || row < 0 || row >= n_rows) {
    set_error(st, LMOE_EDEVICE_CHECK, 221);
    return;
  }
  const unsigned h = p >> d_shift, d = (p & ((1u << d_shift) - 1)) * 8;
  const size_t to = (size_t)block * c.block_stride + (size_t)h * c.head_stride +
                    (size_t)(slot & ((1 << bs_shift) - 1)) * c.slot_stride + d;
  const uint4 kv = __ldcs(reinterpret_cast<const uint4*>(k_new + (size_t)row * ks + (size_t)p * 8));
  const uint4 vv = __ldcs(reinterpret_cast<const uint4*>(v_new + (size_t)row * vs + (size_t)p * 8));
  *reinterpret_cast<uint4*>(c.k + to) = kv;
  *reinterpret_cast<uint4*>(c.v + to) = vv;
}

bool al16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al8(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool al4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace

bool rows_apart(int64_t block_stride, int64_t n_blocks, int64_t head_stride, int64_t kv_heads, int64_t slot_stride,
                int64_t block_size, int64_t head_dim) {
  struct {
    int64_t stride, extent;
  } dim[3] = {{block_stride, n_blocks}, {head_stride, kv_heads}, {slot_stride, block_size}};
  std::sort(dim, dim + 3, [](const auto& x, const auto& y) { return x.stride < y.stride; });
  int64_t span = head_dim;
  for (const auto& x : dim) {
    if (x.extent == 1) continue;  // it never steps
    if (x.stride < span || x.stride > (INT64_MAX - span) / (x.extent - 1)) return false;
    span += x.stride * (x.extent - 1);
  }
  return true;
}

int optional_status(void* ws, size_t ws_bytes, cudaStream_t s, Status** st) {
  *st = nullptr;
  if (!ws) return LMOE_OK;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return LMOE_EINVAL;
  if (ws_bytes < sizeof(Status)) return LMOE_EWORKSPACE;
  *st = static_cast<Status*>(ws);
  return launch_pdl("status_zero_kernel", dim3(1), dim3(32), 0, s, status_zero_kernel, *st);
}

int check_cache(const lmoe_kv_cache* c, bool memory) {
  if (!c || c->kv_heads < 1 || c->kv_heads > 256 || c->head_dim < 1) return LMOE_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128) return LMOE_EUNSUPPORTED;
  if (!memory) return LMOE_OK;
  if (!al16(c->k) || !al16(c->v) || c->n_blocks < 1 || c->block_size < 1) return LMOE_EINVAL;
  const int bs = c->block_size;
  if (bs < 16 || bs > 256 || (bs & (bs - 1))) return LMOE_EUNSUPPORTED;
  // slot numbers are 32-bit
  if ((long long)c->n_blocks * bs > 0x7fffffffll) return LMOE_EUNSUPPORTED;
  const int64_t st[3] = {c->block_stride, c->head_stride, c->slot_stride};
  for (int64_t x : st)
    if (x < 0 || x % 8) return LMOE_EINVAL;
  // heads, slots and blocks next to one another do not overlap (rows_apart tells for all of them)
  if (c->slot_stride < c->head_dim || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
      (c->n_blocks > 1 && c->block_stride < c->head_dim))
    return LMOE_EINVAL;
  return LMOE_OK;
}

}  // namespace lmoe

using namespace lmoe;

extern "C" {

int lmoe_tree_masks(int32_t n_requests, int32_t n_tokens, int32_t mask_words, const int32_t* token_offsets,
                    const int32_t* parents, const int32_t* lens, uint64_t* mask, int32_t* pos, void* ws,
                    size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  if (n_requests < 1 || n_requests > kPlanMaxRequests || n_tokens < 1 || n_tokens > (1 << 20) || mask_words < 1 ||
      mask_words > 4 || !al4(token_offsets) || !al4(parents) || (lens && !al4(lens)) || !al8(mask) || !al4(pos))
    return LMOE_EINVAL;
  DevInfo di;
  int rc = dev_info(&di);
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Status* st;
  if ((rc = optional_status(ws, ws_bytes, s, &st))) return rc;
  void (*const kern[4])(int, const int32_t*, const int32_t*, const int32_t*, uint64_t*, int32_t*, Status*) = {
      tree_masks_kernel<1>, tree_masks_kernel<2>, tree_masks_kernel<3>, tree_masks_kernel<4>};
  return launch_pdl("tree_masks_kernel", dim3(n_requests), dim3(64 * mask_words), 0, s, kern[mask_words - 1], n_tokens,
                    token_offsets, parents, lens, mask, pos, st);
}

int lmoe_kv_plan(int32_t n_requests, int32_t block_size, int32_t max_blocks, int32_t n_slots, const int32_t* lens,
                 const int32_t* new_tokens, const int32_t* owned, int32_t* block_table, int32_t* ring,
                 int32_t ring_size, const int32_t* ring_state, int32_t* lens_out, int32_t* owned_out,
                 int32_t* ring_state_out, int32_t* token_offsets, int32_t* slots, lmoe_stream_t stream) {
  calls_begin();
  if (n_requests < 1 || n_requests > kPlanMaxRequests || block_size < 1 || max_blocks < 1 || max_blocks > (1 << 24) || n_slots < 1 ||
      ring_size < 1)
    return LMOE_EINVAL;
  const void* in[] = {lens, new_tokens, owned, block_table, ring, ring_state};
  const void* out[] = {lens_out, owned_out, ring_state_out, token_offsets, slots};
  for (const void* p : in)
    if (!al4(p)) return LMOE_EINVAL;
  for (int i = 0; i < 5; ++i) {
    if (!al4(out[i])) return LMOE_EINVAL;
    for (const void* p : in)
      if (out[i] == p) return LMOE_EINVAL;
    for (int j = 0; j < i; ++j)
      if (out[i] == out[j]) return LMOE_EINVAL;
  }
  if (block_table == ring) return LMOE_EINVAL;
  DevInfo di;
  int rc = dev_info(&di);
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const PlanArgs a = {n_requests, block_size,  max_blocks, n_slots,  ring_size, lens,           new_tokens, owned,
                      ring_state, block_table, ring,       lens_out, owned_out, ring_state_out, token_offsets, slots,
                      ((reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(new_tokens) |
                        reinterpret_cast<uintptr_t>(owned)) & 15u) == 0};
  if (n_requests <= 256) return run_plan<256, 1>(a, di.sms, s);
  if (n_requests <= 1024) return run_plan<1024, 1>(a, di.sms, s);
  if (n_requests <= 4096) return run_plan<1024, 4>(a, di.sms, s);
  return run_plan<1024, 8>(a, di.sms, s);
}

int lmoe_kv_write(const lmoe_kv_cache* cache, const uint16_t* k_new, int64_t k_stride, const uint16_t* v_new,
                  int64_t v_stride, int32_t n_rows, const int32_t* src, const int32_t* slots, int32_t n_tokens,
                  void* ws, size_t ws_bytes, lmoe_stream_t stream) {
  calls_begin();
  int rc = check_cache(cache, true);
  if (rc) return rc;
  if (!rows_apart(cache->block_stride, cache->n_blocks, cache->head_stride, cache->kv_heads, cache->slot_stride,
                  cache->block_size, cache->head_dim))
    return LMOE_EINVAL;  // (distinct slots would be written over one another)
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (!al16(k_new) || !al16(v_new) || k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8 || n_rows < 1 ||
      n_tokens < 1 || n_tokens > (1 << 20) || (!src && n_tokens > n_rows) || (src && !al4(src)) || !al4(slots))
    return LMOE_EINVAL;
  DevInfo di;
  if ((rc = dev_info(&di))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Status* st;
  if ((rc = optional_status(ws, ws_bytes, s, &st))) return rc;
  const int pieces = (int)(row / 8);
  const long long total = (long long)n_tokens * pieces;
  if (total > 0x7fffffffll) return LMOE_EUNSUPPORTED;
  const int grid = (int)((total + 255) / 256);
  return launch_pdl("kv_write_kernel", dim3(grid), dim3(256), 0, s, kv_write_kernel, *cache, k_new,
                    (long long)k_stride, v_new, (long long)v_stride, n_rows, src, slots, n_tokens, pieces,
                    log2_of(cache->block_size), log2_of(cache->head_dim / 8), st);
}

}  // extern "C"

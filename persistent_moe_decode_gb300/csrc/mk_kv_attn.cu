// Attention of packed query rows over the BF16 paged cache (mk_kv_attention).
//
// Mathematics.  A row's running reference r (of its scores' maximum) and sum
// l = sum exp(s - r), with O = sum exp(s - r) v beside it, a key tile of 128 at a
// time; parts of a row over different keys add up as (r, l, O) again.  Scores and
// O are fp32 sums of BF16 products.  Weights are rounded to BF16 for theirs with the
// values (not in l): the tensor cores take both operands of one type, and a second
// product for the weights' low halves would double that half of the work.  It costs
// 0.4 to 0.7e-3 of the results' norm beside 1.4 to 1.7e-3 of their own rounding.
//
// Rows.  A block of work is 2 tiles of 128 rows of one KV head: the query heads
// of its group, token after token (row = token * grp + head), so that few tokens
// of many heads fill a tile as many tokens of few heads do.  A tile holds
// floor(128 / grp) whole tokens.  Rows that fit one tile are `narrow`: the two
// softmax warpgroups then take key tiles in turn, and add up at the end.
//
// Shares.  Lengths are on the device only, so the blocks cut the work
// themselves: all (task, KV head, row block) items laid end to end, an item as
// long as its keys and a little for its start and end, and each block of the grid
// takes an equal stretch (mk_kv_sched.cuh).  A task is a sequence's own keys
// (causal), or a group's common ones (all of them seen).  A block meets at most
// one item that it does not begin and one that it does not end; these leave their
// sums in the workspace, and the merge kernel adds them up in order.  No atomics.
//
// A block, one an SM, 12 warps: two softmax warpgroups, a thread a row; a warp
// that plans and copies K and V pages (TMA, a ring of 128-key tiles), one of MMAs
// for each softmax warpgroup, one that copies Q and clears values that some row
// does not see.  S = Q K^T goes to tensor memory (128 columns a stream); the
// softmax threads turn it into weights and write them over it as BF16; O += P V
// takes them from there (128 columns a stream, all 512 in use).  While one
// stream's softmax runs, the tensor cores work for the other's.
//
// Measured, one GB300 (kernels in a graph; 32 query and 4 KV heads of 128 dims):
// a prompt of 32,768 tokens 5.3 ms, 1660 TFLOP/s (86 % of the measured matrix
// product rate; 5.7 ms a call among others, at a lower clock), of 8192 0.374-0.396 ms
// (1390-1470), of 2048 49-51 us; one token of 262,144 94 us (5.7 TB/s), of 8192 15-17
// us, of 128 8-9 us; 8192 tokens of 16 heads of 64 dims 186 us.  What bounds it:
// - wide items: the chain of one stream, scores - weights - products: 1,250
//   cycles of softmax (690 instructions a warp and tile; issue 45 %, exponentials
//   33 % of their rate) and 1,050 of products after it; the other stream fills
//   the tensor cores for two thirds of that (66 % of active cycles at 8192 tokens);
// - narrow items: a tile's 64 KB pass the SM's copy engine at 41 bytes a cycle,
//   1,600 cycles, and one warp's issue makes 2,000 of it; all SMs together then
//   ask for more than the HBM gives;
// - short calls: a block takes 9,000 to 12,000 cycles until its first scores
//   (plan, page table, copies, each cold), an item's end 4,000 to 6,000, the
//   merge 3 to 4 us.
// Tried and slower: one warp for all products (32K: 6.2 ms: an issued product
// holds its warp for its 64 cycles, so the waits between them idle the tensor
// cores), two without turns (6.7), scores taken by 32 columns (5.4-5.8), rows
// handed to lanes by shuffles for the output (5.6); the first kernel launched
// before the end of what precedes it gains 0.3 us.
#include <cfloat>
#include <cmath>
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "mk.h"
#include "mk_kv_sched.cuh"
#include "mk_tc.cuh"

namespace mk {
namespace {

constexpr int kThreads = 384;
constexpr int kItems = 4;                // ring of work items
constexpr int kReaders = 11;             // warps that read an item: 8 softmax, 2 MMA, Q and clearing
#ifndef MK_KV_WAIT_NS                    // a test builds these kernels with waits that run out
#define MK_KV_WAIT_NS kKvWaitNs
#endif
constexpr unsigned long long kWaitNs = MK_KV_WAIT_NS, kSettleNs = kKvWaitNs;
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * 168, "register split");

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kSmem = 2 * kTileBytes + kStages * kTileBytes + 1024;
};

constexpr int kEnd = 8;                   // Item::flags: there are no more

struct alignas(16) Item : Part {
  int bad, dirty;          // a page outside the cache; cleared values were not finite
};

// what the merge kernel reads of a slot
struct alignas(16) Slot {
  int state;               // 0: not used, 1: the next block's first slot goes on, 2: the last part
  int tok0, ntok, head, kbeg, lim, flags, nan;
};

struct Ws {
  Slot* slots;             // [2 blocks]: 2 c the part that block c did not begin, 2 c + 1 that it did
  float* data;             // [2 blocks][slot_floats]
  // groups: a row's sums over common keys and over own ones; line l of total_q *
  // hq is (KV head, token, head of its group)
  float* part_o;           // [2][D / 4][lines][4]
  float* part_m;           // [2][lines] log2 of the sum of exponentials
  int32_t* rows;           // [4] those that sequences own (owned_rows)
};

__host__ __device__ __forceinline__ size_t slot_floats(int d) { return (size_t)256 * d + 512; }

__host__ __device__ __forceinline__ Ws ws_of(uint8_t* p, int d, int hq, int total_q, int blocks) {
  Ws w;
  w.slots = (Slot*)p;
  w.data = (float*)(p + (size_t)2 * blocks * sizeof(Slot));
  w.part_o = w.data + 2 * blocks * slot_floats(d);
  w.part_m = w.part_o + (size_t)2 * total_q * hq * d;
  w.rows = (int32_t*)(w.part_m + (size_t)2 * total_q * hq);
  return w;
}

// ------------------------------------------------------------------------ waits

// a block's stretch and the item it begins in
struct Plan {
  Begin begin;
  long long pos, end, share;
};

struct Sync {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t raw_full[10];                 // a tile that is cleared before it counts as full
  uint64_t q_full[2], q_empty[2], s_full[2], o_full[2];
  uint64_t p_full[2][2];                 // a stream's weights of the first, the last 64 columns
  uint64_t turn[2];                      // wide items: the other warp has issued its products
  uint64_t pair_full, pair_empty;        // narrow items: the second warpgroup's sums are there, are read
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t drain[2];
  uint32_t tmem;
  volatile int stop;
  uint32_t kv_loads, kv_raw, kv_raw_use, q_loads[2];     // copies that were issued, for a block that gives up
  long long scan[kThreads / 32];
  Plan plan;                             // of many tasks
  int planned;
  Sound sound;
  int ordered;                           // all starts of few tasks are
  int first[2], last[2];                 // starts out of order, of groups and of sequences: the outermost
  float pair[2][kTile];
};

// Waits for the phase of this parity; false once the block gives up, or after
// kWaitNs (ITEM: of a wait that lasts over a whole item, kKvItemWaits times that),
// which makes it give up.
template <bool ITEM = false>
__device__ __forceinline__ bool wait(Sync& s, uint64_t* bar, uint32_t parity, int32_t* status) {
  // a look may last as long as the hardware likes: a limit of microseconds takes short ones
  constexpr bool kShort = kWaitNs < 1000000;
  auto done = [&] { return kShort ? mbar_try_wait(bar, parity) : mbar_wait_some(bar, parity); };
  if (done()) return true;
  unsigned long long t0 = 0;
  for (int i = 1;; i++) {
    if (done()) return true;
    if (kShort || (i & 15) == 0) {
      if (s.stop) return false;
      const unsigned long long t = gtime_ns();
      if (!t0) t0 = t;
      if (t - t0 > (ITEM ? kKvItemWaits : 1) * kWaitNs) {
        s.stop = 1;
        flag(status, MK_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
template <bool ITEM = false>
__device__ __forceinline__ bool wait_warp(Sync& s, uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, wait<ITEM>(s, bar, parity, status));
}
// what is in flight must have landed before the block ends
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = gtime_ns();
  while (!mbar_try_wait(bar, parity) && gtime_ns() - t0 < kSettleNs) {}
}

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// one BF16 pair's elements that are not finite: bit 15, bit 31
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// One warp: this block's stretch, if it begins in a task of this warp.  Each lane
// has a task k (number t) or none, of `mine` keys after `before` others, `per` a
// KV head.
__device__ __forceinline__ bool find_plan(const KvAttnArgs& a, Plan& plan, const Task& k, int t, long long before,
                                          long long mine, long long per, long long total, int tb, int lane) {
  const long long share = share_of(total, a.per_block);
  const long long pos = share * blockIdx.x;
  const unsigned owner = __ballot_sync(0xffffffffu, pos < total && before <= pos && pos < before + mine);
  if (!owner) return false;
  const int from = __ffs(owner) - 1;
  Task o;
#pragma unroll
  for (int w = 0; w < (int)(sizeof(Task) / 4); w++)
    reinterpret_cast<int*>(&o)[w] = __shfl_sync(0xffffffffu, reinterpret_cast<const int*>(&k)[w], from);
  plan.begin = begin_of(o, __shfl_sync(0xffffffffu, t, from), tb, __shfl_sync(0xffffffffu, before, from),
                        __shfl_sync(0xffffffffu, per, from), pos, lane);
  plan.pos = pos, plan.end = min(total, pos + share), plan.share = share;
  return true;
}

__device__ __forceinline__ long long scan(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// ----------------------------------------------------------------------- kernel

// Softmax (a warpgroup), item after item: of one of its two tiles of rows, over
// all its keys; or, where its rows fit one tile, of every second key tile, the
// two sums being added at the end.
template <int D>
__device__ void softmax_role(const KvAttnArgs& a, Sync& s, Item* items, const Ws& ws, int group, int tt) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row = 32 * warp + lane;
  const uint32_t tm = s.tmem + ((uint32_t)(32 * warp) << 16);
  const uint32_t tm_s = tm + 128 * group, tm_o = tm + 256 + D * group;
  const float scale = a.scale_log2;
  const int my_tok = row / a.grp, my_head = row - my_tok * a.grp;
  uint32_t steps = 0, parts = 0, pairs = 0;
  for (int it = 0;; it++) {
    Item* slot = &items[it % kItems];
    if (!wait_warp(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status)) return;
    const Part m = *slot;
    if (m.flags & kEnd) return;
    const bool narrow = m.ntok <= tt;
    const int tok = narrow ? my_tok : group * tt + my_tok, every = narrow ? 2 : 1;
    const bool mine = my_tok < tt && tok < m.ntok;
    const int lim = m.flags & kCausal ? m.lim + tok : m.kend;
    const int least = __reduce_min_sync(0xffffffffu, mine ? lim : 0x7fffffff);
    const int j0 = narrow ? m.k0 + group : m.k0;
    float top = -INFINITY, sum = 0.f;
    for (int j = j0; j < m.k1; j += every, steps++) {
      if (!wait_warp(s, &s.s_full[group], steps & 1, a.status)) return;
      tc_fence_after();
      const int t0 = m.kbeg + kTile * j;
      const bool masked = t0 + kTile > least, paged = narrow && D == 128;
      const int seen = min(max(lim - t0, 0), kTile);
      // 64 columns at a time, read once for the maximum and once for the weights:
      // the loop is half as long as one over 128 registers, and what the second
      // read costs the instruction cache gives back (packed prompts 74 us against
      // 71, questions to a shared text 108 against 99, 32K prompt 5.30 ms against
      // 5.26).
      auto scores = [&](int h, float* x) {
        tc_ld32(tm_s + 64 * h, (uint32_t*)x), tc_ld32(tm_s + 64 * h + 32, (uint32_t*)x + 32);
        tc_wait_ld();
        if (!masked) return;
        // columns that are seen: the first of each 64 (a narrow item's pages have
        // their first 8 keys in the first 64 columns, the others in the last)
        const int n = paged ? 8 * (seen >> 4) + min(max((seen & 15) - 8 * h, 0), 8) : seen - 64 * h;
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          const uint32_t bits = n - c >= 32 ? 0xffffffffu : n - c <= 0 ? 0u : (1u << (n - c)) - 1;
#pragma unroll
          for (int u = 0; u < 32; u++) x[c + u] = bits >> u & 1 ? x[c + u] : -INFINITY;
        }
      };
      float high = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        float x[64];
        scores(h, x);
        float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[2], x[3]), m2 = fmaxf(x[4], x[5]), m3 = fmaxf(x[6], x[7]);
#pragma unroll
        for (int u = 8; u < 64; u += 8)
          m0 = fmaxf(fmaxf(m0, x[u]), x[u + 1]), m1 = fmaxf(fmaxf(m1, x[u + 2]), x[u + 3]),
          m2 = fmaxf(fmaxf(m2, x[u + 4]), x[u + 5]), m3 = fmaxf(fmaxf(m3, x[u + 6]), x[u + 7]);
        high = fmaxf(fmaxf(high, fmaxf(m0, m1)), fmaxf(m2, m3));
      }
      // The reference moves only when a weight would pass 2^8: sums and
      // products stay within 2^8 of their size, and O is rarely rescaled.
      const bool move = high > top && (high - top) * scale > 8.f;
      if (j == j0) {
        if (high > top) top = high;
      } else if (__any_sync(0xffffffffu, move)) {
        // S of this step is complete, so P V of the step before is too
        const float keep = move ? tc_ex2((top - high) * scale) : 1.f;
        if (move) top = high;
        sum *= keep;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tc_ld32(tm_o + c, o);
          tc_wait_ld();
#pragma unroll
          for (int u = 0; u < 32; u++) o[u] = __float_as_uint(__uint_as_float(o[u]) * keep);
          tc_st32(tm_o + c, o);
        }
      }
      const float off = top == -INFINITY ? 0.f : -top * scale;
      const float2 sc2 = make_float2(scale, scale), off2 = make_float2(off, off);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
      for (int h = 0; h < 2; h++) {
        float x[64];
        uint32_t p[32];
        scores(h, x);
#pragma unroll
        for (int u = 0; u < 32; u++) {
          float2 e = __ffma2_rn(make_float2(x[2 * u], x[2 * u + 1]), sc2, off2);
          e.x = tc_ex2(e.x), e.y = tc_ex2(e.y);
          acc[u & 1] = __fadd2_rn(acc[u & 1], e);
          p[u] = cvt_bf2(e.x, e.y);
        }
        tc_st32(tm_s + 32 * h, p);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[group][h]);     // its product starts while the other half is made
      }
      sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
    }
    // -------------------------------------------------------------- the result
    if (m.k1 > j0) {
      if (!wait_warp(s, &s.o_full[group], parts & 1, a.status)) return;
      parts++;
      tc_fence_after();
    }
    // A weight that rounds to zero still multiplies: a NaN that the row sees must
    // not depend on where its keys were cut.
    float keep0 = 1.f, keep1 = 1.f;
    if (narrow) {
      if (group == 1) {
        s.pair[0][row] = top, s.pair[1][row] = sum;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.pair_full);
        if (!wait_warp(s, &s.pair_empty, pairs++ & 1, a.status)) return;
        if (lane == 0) mbar_arrive(&s.item_empty[it % kItems]);
        continue;
      }
      if (!wait_warp(s, &s.pair_full, pairs++ & 1, a.status)) return;
      tc_fence_after();
      const float top1 = s.pair[0][row], sum1 = s.pair[1][row], high = fmaxf(top, top1);
      if (high > -INFINITY) {
        keep0 = top == high ? 1.f : tc_ex2((top - high) * scale);
        keep1 = top1 == high ? 1.f : tc_ex2((top1 - high) * scale);
      }
      sum = fmaf(keep0, sum, keep1 * sum1);
      top = high;
    }
    const int first = m.kbeg + kTile * m.k0, last = min(m.kend, m.kbeg + kTile * m.k1);
    const bool some = m.k1 > m.k0, second = narrow && m.k1 > m.k0 + 1;
    const bool nan = (m.flags & kNan) || ((volatile Item*)slot)->bad;
    const bool dirty = ((volatile Item*)slot)->dirty;
    const bool sees = some && lim > first;                   // something in this part
    const float ref = top == -INFINITY ? (sees ? -FLT_MAX : -INFINITY) : top * scale;
    const bool whole = m.slot < 0, parted = a.groups > 0;
    const bool zero = sees && sum == 0.f;                    // every score is -infinity
    const float mul = !whole ? 1.f : !sees ? 0.f : zero ? (parted ? 1.f : NAN) : 1.f / sum;
    const int64_t token = m.tok0 + tok;
    const int head = m.head * a.grp + my_head;
    const size_t lines = (size_t)a.total_q * a.hq, at = ((size_t)m.head * a.total_q + token) * a.grp + my_head;
    const int own = m.flags & kPrefix ? 0 : 1, line = narrow ? row : 128 * group + row;
    // four dims of all rows lie side by side: a warp writes 512 bytes
    float* data = ws.data + (whole ? 0 : m.slot) * slot_floats(D);
    float4* quads = whole ? (float4*)ws.part_o + own * (D / 4) * lines + at : (float4*)data + line;
    const size_t quad_step = whole ? lines : 256;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      uint32_t r[32];
      float* o = (float*)r;
      tc_ld32(tm_o + c, r);
      if (second) {
        uint32_t r1[32];
        tc_ld32(tm_o + D + c, r1);
        tc_wait_ld();
#pragma unroll
        for (int u = 0; u < 32; u++) o[u] = fmaf(keep0, o[u], keep1 * __uint_as_float(r1[u]));
      } else {
        tc_wait_ld();
        if (!some) {
#pragma unroll
          for (int u = 0; u < 32; u++) o[u] = 0.f;
        }
      }
      if (dirty && mine) {
        // values that were not finite and that this row sees: whatever their weight, they are in its sum
        for (int t = max(first, m.flags & kCausal ? m.lim : m.kend); t < min(lim, last); t++) {
          const int page = a.page_tables[(int64_t)m.table * a.max_pages + t / kKvPage];
          if (page < 0 || page >= a.num_pages) continue;
          const uint16_t* v = a.v_pool + (((int64_t)page * a.hkv + m.head) * kKvPage + t % kKvPage) * D + c;
#pragma unroll
          for (int u = 0; u < 32; u++) {
            const float f = bf16f(v[u]);
            if (!(fabsf(f) <= FLT_MAX)) o[u] += f;
          }
        }
      }
      if (mine && whole) {
#pragma unroll
        for (int u = 0; u < 32; u++) o[u] = nan ? NAN : o[u] * mul;
      }
      if (mine && whole && !parted) {
        uint32_t b[16];
#pragma unroll
        for (int u = 0; u < 16; u++) b[u] = cvt_bf2(o[2 * u], o[2 * u + 1]);
        uint16_t* out = a.out + token * a.out_stride + (int64_t)head * D + c;
        st_32(out, b, a.aligned32), st_32(out + 16, b + 8, a.aligned32);
      } else if (mine) {
#pragma unroll
        for (int u = 0; u < 8; u++)
          quads[(c / 4 + u) * quad_step] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
      }
      __syncwarp();        // the next tensor memory load is the whole warp's
    }
    if (mine && whole && parted) ws.part_m[own * lines + at] = nan ? NAN : ref == -INFINITY || ref == -FLT_MAX ? ref : ref + log2f(sum);
    if (mine && !whole) data[256 * D + line] = ref, data[256 * D + 256 + line] = sum;
    tc_fence_before();       // O has been read before the next item's first P is announced
    __syncwarp();
    if (lane == 0) {
      if (narrow) mbar_arrive(&s.pair_empty);
      mbar_arrive(&s.item_empty[it % kItems]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_kernel(const KvAttnArgs a, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap page_k,
                        const __grid_constant__ CUtensorMap page_v) {
  using S = Shape<D>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Sync s;
  __shared__ Item items[kItems];
  const uint32_t q_smem = (smem_u32(raw_smem) + 1023u) & ~1023u, kv_smem = q_smem + 2 * S::kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tt = kTile / a.grp, tb = 2 * tt, tasks = a.groups + a.batch;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, gridDim.x);

  // Up to 32 tasks: the warp that copies pages makes its plan at once, while the
  // others get ready.
  const bool few = tasks <= 32;
  Plan plan;
  bool work = false;
  if (few && warp == 8) {
    Task k{};
    long long per = 0;
    if (lane < tasks) {
      k = load_task(a, lane, tb, blockIdx.x == 0);
      per = cost_before(k, k.nb, tb);
    }
    const bool ordered = !__any_sync(0xffffffffu, k.flags & kOrder);
    if (lane == 0) s.ordered = ordered, s.sound = all_hold();
    const long long mine = per * a.hkv, incl = scan(mine, lane), total = __shfl_sync(0xffffffffu, incl, 31);
    work = find_plan(a, plan, k, lane, incl - mine, mine, per, total, tb, lane);
  }
  if (tid == kThreads - 32) {
    for (int i = 0; i < S::kStages; i++) mbar_init(&s.kv_full[i], 1), mbar_init(&s.kv_empty[i], 2), mbar_init(&s.raw_full[i], 1);
    for (int t = 0; t < 2; t++) {
      mbar_init(&s.q_full[t], 1), mbar_init(&s.q_empty[t], t ? 1 : 2), mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_full[t][0], 4), mbar_init(&s.p_full[t][1], 4), mbar_init(&s.turn[t], 1), mbar_init(&s.o_full[t], 1);
    }
    for (int i = 0; i < kItems; i++) mbar_init(&s.item_full[i], 1), mbar_init(&s.item_empty[i], kReaders);
    mbar_init(&s.pair_full, 4), mbar_init(&s.pair_empty, 4), mbar_init(&s.drain[0], 1), mbar_init(&s.drain[1], 1);
    s.stop = 0, s.planned = 0;
    s.first[0] = s.first[1] = 0x7fffffff, s.last[0] = s.last[1] = -1;
    mbar_fence_init();
  }
  if (warp == 9) tc_alloc(&s.tmem, 512);

  if (warp == 10 && lane < 4) tma_prefetch_map(lane == 0 ? &map_k : lane == 1 ? &page_v : lane == 2 ? &map_q : &page_k);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;

  // many tasks: all threads add up their cost, and one warp finds the item that
  // this block's stretch begins in.  So too for few whose starts are out of order,
  // which keeps what that takes out of the way of all other calls.
  if (!few || !s.ordered) {
    const int chunk = (tasks + kThreads - 1) / kThreads;
    int t = min(tasks, tid * chunk);
    const int end = min(tasks, t + chunk);
    long long mine, before, total = 0, per = 0;
    Task k{};
    Sound so = all_hold();
    for (bool again = false;; again = true) {
      bool wrong = false;
      mine = 0;
      for (int i = t; i < end; i++) {
        k = load_task(a, i, tb, blockIdx.x == 0, so);
        per = cost_before(k, k.nb, tb);
        mine += per * a.hkv;
        wrong |= !again && k.flags & kOrder;
      }
      const long long incl = scan(mine, lane);
      before = incl - mine;
      if (lane == 31) s.scan[warp] = incl;
      if (!__syncthreads_or(wrong)) break;
      // starts out of order: once more, with what holds
      for (int i = t; i < end; i++)
        if (!in_order(a, i)) {
          const int q = i >= a.groups, x = q ? i - a.groups : i;
          atomicMin(&s.first[q], x), atomicMax(&s.last[q], x);
        }
      __syncthreads();
      if (s.last[0] >= 0) holding(a.group_starts, a.groups, s.first[0], s.last[0], &so.g0, &so.g1);
      if (s.last[1] >= 0) holding(a.q_starts, a.batch, s.first[1], s.last[1], &so.b0, &so.b1);
    }
    if (tid == 0) s.sound = so;
    for (int w = 0; w < kThreads / 32; w++) {
      const long long x = s.scan[w];
      if (w < warp) before += x;
      total += x;
    }
    if (chunk > 1) {                       // the thread that holds the position finds its task
      const long long pos = share_of(total, a.per_block) * blockIdx.x;
      if (before <= pos && pos < before + mine)
        for (;; t++) {
          k = load_task(a, t, tb, false, so);
          per = cost_before(k, k.nb, tb);
          mine = per * a.hkv;
          if (pos < before + mine) break;
          before += mine;
        }
    }
    if (find_plan(a, plan, k, t, before, mine, per, total, tb, lane) && lane == 0) s.plan = plan, s.planned = 1;
    __syncthreads();
    plan = s.plan, work = s.planned;
  }

  if (warp < 8) {
    regs_up<kRegsSoftmax>();
    softmax_role<D>(a, s, items, ws, warp >> 2, tt);
  } else {
    regs_down<kRegsOther>();
    if (warp == 8) {
      // ------------------------------------------- items, K and V (whole warp)
      Slot desc[2] = {};
      uint32_t loads = 0, raw = 0, raw_use = 0;    // stages whose last tile goes through raw_full; its uses, modulo 2
      int it = 0;
      bool ok = true;
      if (work) {
        auto pages_of = [&](const Part& p, int j) { return min(8, (p.kend - p.kbeg - kTile * j + kKvPage - 1) / kKvPage); };
        auto page_of = [&](const Part& p, int j) {
          return j < p.k1 && lane < pages_of(p, j)
                     ? a.page_tables[(int64_t)p.table * a.max_pages + p.kbeg / kKvPage + 8 * j + lane] : 0;
        };
        Stretch w(a, tt, plan.begin, plan.pos, plan.end, plan.share, &s.sound);
        Part m, nx;
        bool have = w.next(&m, 2 * (int)blockIdx.x);
        int page[3], npage[3] = {0, 0, 0};
        if (have)
          for (int x = 0; x < 3; x++) page[x] = page_of(m, m.k0 + x);
        while (have) {
          Item* dst = &items[it % kItems];
          ok = wait_warp(s, &s.item_empty[it % kItems], ((it / kItems) & 1) ^ 1, a.status);
          if (!ok) break;
          if (lane == 0) {
            *static_cast<Part*>(dst) = m;
            dst->bad = dst->dirty = 0;
            mbar_arrive(&s.item_full[it % kItems]);
          }
          it++;
          bool bad = false;
          const bool narrow = m.ntok <= tt;
          const int clear = (m.flags & kCausal ? m.lim : m.kend) - m.kbeg;
          auto load = [&](bool value, int j, int pg) {
            const uint32_t st = loads % S::kStages;
            if (!wait_warp(s, &s.kv_empty[st], ((loads / S::kStages) & 1) ^ 1, a.status)) return false;
            const int np = pages_of(m, j);
            const bool out = lane < np && (pg < 0 || pg >= a.num_pages);
            if (__any_sync(0xffffffffu, out)) {
              bad = true;
              if (lane == 0) ((volatile Item*)dst)->bad = 1, flag(a.status, MK_ERR_BAD_PAGE);
            }
            const bool through = value && kTile * (j + 1) > clear;
            raw = (raw & ~(1u << st)) | (uint32_t)through << st;
            raw_use ^= (uint32_t)through << st;
            uint64_t* bar = through ? &s.raw_full[st] : &s.kv_full[st];
            // a page outside the cache: past the last one, which the copy fills with zeros
            const int from = out ? a.num_pages : pg;
            int ids[8];
#pragma unroll
            for (int i = 0; i < 8; i++) ids[i] = __shfl_sync(0xffffffffu, from, i);
            // One lane issues (sixteen lanes at once took 150 cycles a copy, 2500 a
            // tile; one lane about 1000), whole pages where their layout serves:
            // all but the keys of wide items, whose product wants 16 atoms at one
            // stride.
            if (tc_elect()) {
              const uint32_t to = kv_smem + st * S::kTileBytes;
              mbar_arrive_expect_tx(bar, np * S::kHalves * 2048);
              if (value || narrow || S::kHalves == 1) {
                const CUtensorMap* map = value ? &page_v : &page_k;
#pragma unroll
                for (int i = 0; i < 8; i++)
                  if (i < np) tma_load_4d(to + i * S::kHalves * 2048, map, 0, kKvPage * m.head, 0, ids[i], bar);
              } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                  if (i < np)
#pragma unroll
                    for (int h = 0; h < S::kHalves; h++)
                      tma_load_3d(to + h * 16384 + i * 2048, &map_k, 64 * h, kKvPage * m.head, ids[i], bar);
              }
            }
            __syncwarp();
            loads++;
            return true;
          };
          // in the order of their use: K of the first step (narrow: two), then V of one and K of a later one
          ok = m.k1 == m.k0 || load(false, m.k0, page[0]);
          if (ok && narrow && m.k1 > m.k0 + 1) ok = load(false, m.k0 + 1, page[1]);
          bool more = false;
          for (int j = m.k0; ok && (j < m.k1 || j == m.k0); j++) {
            const int later = page_of(m, j + 3);
            if (j < m.k1) ok = load(true, j, page[0]);
            if (ok && !narrow && j + 1 < m.k1) ok = load(false, j + 1, page[1]);
            if (ok && narrow && j + 2 < m.k1) ok = load(false, j + 2, page[2]);
            page[0] = page[1], page[1] = page[2], page[2] = later;
            if (j == m.k0) {
              // the next part and its first pages, while this one's copies are under way
              more = w.next(&nx, 2 * (int)blockIdx.x);
              if (more)
                for (int x = 0; x < 3; x++) npage[x] = page_of(nx, nx.k0 + x);
            }
          }
          if (m.slot >= 0)
            desc[m.k0 == 0] = Slot{m.k1 < m.n ? 1 : 2, m.tok0, m.ntok, m.head, m.kbeg, m.lim, m.flags, bad};
          if (!ok) break;
          have = more, m = nx;
          for (int x = 0; x < 3; x++) page[x] = npage[x];
        }
      }
      if (ok && wait_warp(s, &s.item_empty[it % kItems], ((it / kItems) & 1) ^ 1, a.status) && lane == 0) {
        items[it % kItems].flags = kEnd;
        mbar_arrive(&s.item_full[it % kItems]);
      }
      if (lane < 2) ws.slots[2 * blockIdx.x + lane] = lane ? desc[1] : desc[0];
      if (a.groups && blockIdx.x == 0 && lane == 0) owned_rows(a, s.sound, ws.rows);
      if (lane == 0) s.kv_loads = loads, s.kv_raw = raw, s.kv_raw_use = raw_use;
    } else if (warp < 11) {
      // ---------- MMAs, a warp each for the two softmax warpgroups: together,
      // one lane issues.  Wide items: stream t is a tile of rows, and each step's
      // K and V serve both.  Narrow ones: the streams take key tiles in turn.
      // Either way a warp sees every load of the ring, in order.
      constexpr uint32_t idesc_s = tc_idesc(kTile, false), idesc_half = tc_idesc(64, false), idesc_o = tc_idesc(D, true);
      const int t = __shfl_sync(0xffffffffu, warp - 9, 0);
      uint32_t loads = 0, used_q[2] = {0, 0}, steps = 0, turns = 0;
      bool ok = true;
      auto commit = [&](uint64_t* bar) {
        if (tc_elect()) tc_commit(bar);
        __syncwarp();
      };
      auto full = [&](uint32_t load) {
        ok = ok && wait_warp(s, &s.kv_full[load % S::kStages], (load / S::kStages) & 1, a.status);
        tc_fence_after();
        return ok;
      };
      auto used = [&](bool by_me) {                          // this load's stage; on to the next
        uint64_t* bar = &s.kv_empty[loads++ % S::kStages];
        if (tc_elect()) {
          if (by_me) tc_commit(bar);
          else mbar_arrive(bar);
        }
        __syncwarp();
      };
      for (int it = 0; ok; it++) {
        ok = wait_warp(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status);
        if (!ok) break;
        const Item& m = items[it % kItems];
        const int flags = m.flags, n = m.k1 - m.k0;
        const bool narrow = m.ntok <= tt;
        if (flags & kEnd) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.item_empty[it % kItems]);
        if (n == 0) continue;
        const int tile = narrow ? 0 : t, every = narrow ? 2 : 1;
        const uint64_t q_desc = tc_desc(q_smem + tile * S::kTileBytes);
        // Keys of a narrow item lie page by page, both halves of the dims in each:
        // their atoms (8 keys) are 4096 apart, so S takes the first 8 keys of all
        // pages, then the last 8 (two products of 64 keys), and the values follow
        // that order.  Values of a wide item are taken page by page.
        const bool paged = narrow && S::kHalves == 2;
        const uint64_t k_desc = tc_desc(kv_smem, paged ? 4096 : 1024);
        const uint64_t v_desc = tc_desc(kv_smem, paged ? 4096 : 1024, 2048);
        auto mine = [&](int j) { return !narrow || (j & 1) == t; };
        auto last = [&](int j) { return j + every >= n; };   // of this stream
        auto qk = [&](int j, uint32_t load) {                // one lane: S of key tile j
          const uint64_t kd = k_desc + load % S::kStages * (S::kTileBytes / 16);
          if (paged) {
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
              for (int c = 0; c < D / 16; c++)
                tc_mma_ss(tmem + 128 * t + 64 * h, q_desc + (c / 4 * 16384 + c % 4 * 32) / 16,
                          kd + (1024 * h + c / 4 * 2048 + c % 4 * 32) / 16, idesc_half, c > 0);
          } else {
#pragma unroll
            for (int c = 0; c < D / 16; c++) {
              const int off = (c / 4 * 16384 + c % 4 * 32) / 16;
              tc_mma_ss(tmem + 128 * t, q_desc + off, kd + off, idesc_s, c > 0);
            }
          }
          tc_commit(&s.s_full[t]);
          if (last(j)) tc_commit(&s.q_empty[tile]);
        };
        auto pv = [&](int j, uint32_t load) {                // O of key tile j, half by half
          const uint64_t vd = v_desc + load % S::kStages * (S::kTileBytes / 16);
          const uint32_t par = steps++ & 1;
#pragma unroll
          for (int h = 0; h < 2; h++) {
            ok = ok && wait_warp(s, &s.p_full[t][h], par, a.status);
            if (!ok) return;
            tc_fence_after();
            if (tc_elect()) {
#pragma unroll
              for (int c = 4 * h; c < 4 * h + 4; c++) {
                const int at = paged ? c % 4 * 8192 + c / 4 * 1024 : c * S::kHalves * 2048;
                tc_mma_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * c, vd + at / 16, idesc_o, j >= every || c > 0);
              }
              if (h == 1 && last(j)) tc_commit(&s.o_full[t]);
            }
            __syncwarp();
          }
        };
        ok = wait_warp(s, &s.q_full[0], used_q[0]++ & 1, a.status);
        if (ok && !narrow && t == 1) ok = wait_warp(s, &s.q_full[1], used_q[1]++ & 1, a.status);
        // tile 0 of Q is free when both have done with it
        if (t == 1 && (!narrow || n == 1) && lane == 0) mbar_arrive(&s.q_empty[0]);
        __syncwarp();
        for (int j = 0; ok && j < min(n, every); j++) {
          if (!full(loads)) break;
          if (mine(j) && tc_elect()) qk(j, loads);
          __syncwarp();
          used(mine(j));
        }
        if (!narrow) {
          // The warps take turns, products of one stream after those of the
          // other: in step with each other both softmaxes would run at once, and
          // then both products (32K prompt: 6.7 ms without turns, 5.4 with).
          for (int j = 0; ok && j < n; j++) {
            // all else first: the weights come last
            const bool more = j + 1 < n;
            if (!full(loads) || (more && !full(loads + 1))) break;
            ok = wait_warp(s, &s.turn[t], (turns++ & 1) ^ (t == 0), a.status);
            pv(j, loads);
            if (!ok) break;
            if (tc_elect()) {
              tc_commit(&s.kv_empty[loads % S::kStages]);
              if (more) {
                qk(j + 1, loads + 1);
                tc_commit(&s.kv_empty[(loads + 1) % S::kStages]);
              }
              mbar_arrive(&s.turn[t ^ 1]);
            }
            __syncwarp();
            loads += more ? 2 : 1;
          }
        } else {
          for (int j = 0; ok && j < n; j++) {
            if (!full(loads)) break;
            if (mine(j)) pv(j, loads);
            if (!ok) break;
            used(mine(j));
            if (j + 2 < n) {
              if (!full(loads)) break;
              if (mine(j) && tc_elect()) qk(j + 2, loads);
              __syncwarp();
              used(mine(j));
            }
          }
        }
      }
      // nothing may arrive on a barrier after the block's end
      commit(&s.drain[t]);
      settle(&s.drain[t], 0);
    } else {
      // ---------------- Q, and values that some row does not see (whole warp): a
      // weight of zero times NaN or an infinity is no zero, so those are taken
      // out, and what a page holds past the sequence with them
      // All of its waits may last over an item; what they wait for the other warps
      // wait for too, tile by tile.
      uint8_t* kv = raw_smem + (kv_smem - smem_u32(raw_smem));
      uint32_t loads = 0, uses = 0, q_loads[2] = {0, 0};
      const uint32_t q_bytes = (uint32_t)(tt * a.grp) * 128 * S::kHalves;
      bool ok = true;
      for (int it = 0; ok; it++) {
        ok = wait_warp<true>(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status);
        if (!ok) break;
        Item* slot = &items[it % kItems];
        const Part m = *slot;
        if (m.flags & kEnd) break;
        for (int t = 0; ok && m.k1 > m.k0 && t < 2 && m.ntok > t * tt; t++) {
          ok = wait_warp<true>(s, &s.q_empty[t], (q_loads[t] & 1) ^ 1, a.status);
          if (!ok) break;
          q_loads[t]++;
          if (tc_elect()) {
            mbar_arrive_expect_tx(&s.q_full[t], q_bytes);
#pragma unroll
            for (int h = 0; h < S::kHalves; h++)
              tma_load_3d(q_smem + t * S::kTileBytes + h * 16384, &map_q, 64 * h, m.head * a.grp, m.tok0 + t * tt,
                          &s.q_full[t]);
          }
          __syncwarp();
        }
        const int clear = (m.flags & kCausal ? m.lim : m.kend) - m.kbeg;
        for (int j = m.k0; ok && j < m.k1; j++) {
          if (kTile * (j + 1) <= clear) continue;
          const uint32_t i = loads + (j - m.k0) + min(j - m.k0 + (m.ntok <= tt ? 2 : 1), m.k1 - m.k0), st = i % S::kStages;
          ok = wait_warp<true>(s, &s.raw_full[st], uses >> st & 1, a.status);
          if (!ok) break;
          uses ^= 1u << st;
          const int lo = max(0, clear - kTile * j), held = min(kTile, m.kend - m.kbeg - kTile * j);
          bool found = false;
          // 16 bytes a lane, eight loads at a time: rows [lo, held) are looked over, those after them zeroed
          auto chunk = [&](int c, int h) {           // 16 bytes c % 8 of half h of row c / 8
            return (uint4*)(kv + st * S::kTileBytes + (c >> 7) * (S::kHalves * 2048) + h * 2048 + (c & 127) * 16);
          };
          for (int c = 8 * lo + lane; c < 8 * held; c += 4 * 32) {
            uint4 w[4][S::kHalves];
#pragma unroll
            for (int u = 0; u < 4; u++)
#pragma unroll
              for (int h = 0; h < S::kHalves; h++) {
                w[u][h] = make_uint4(0, 0, 0, 0);
                if (c + 32 * u < 8 * held) w[u][h] = *chunk(c + 32 * u, h);
              }
#pragma unroll
            for (int u = 0; u < 4; u++)
#pragma unroll
              for (int h = 0; h < S::kHalves; h++) {
                uint32_t* x = reinterpret_cast<uint32_t*>(&w[u][h]);
                if (not_finite(x[0]) | not_finite(x[1]) | not_finite(x[2]) | not_finite(x[3])) {
                  found = true;
#pragma unroll
                  for (int e = 0; e < 4; e++) {
                    const uint32_t b = not_finite(x[e]);
                    x[e] &= ~((b & 0x8000u ? 0xffffu : 0u) | (b & 0x80000000u ? 0xffff0000u : 0u));
                  }
                  *chunk(c + 32 * u, h) = w[u][h];
                }
              }
          }
          for (int c = 8 * max(held, 0) + lane; c < 8 * kTile; c += 32)
#pragma unroll
            for (int h = 0; h < S::kHalves; h++) *chunk(c, h) = make_uint4(0, 0, 0, 0);
          if (found) ((volatile Item*)slot)->dirty = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.kv_full[st]);
        }
        loads += 2 * (m.k1 - m.k0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.item_empty[it % kItems]);
      }
      if (lane == 0) s.q_loads[0] = q_loads[0], s.q_loads[1] = q_loads[1];
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // A block that gave up: the warps that copy may have ended well before the wait
  // that ran out, so their copies are waited for here, where no warp goes on.
  if (s.stop) {
    if (warp == 8) {
      const uint32_t loads = s.kv_loads;
      for (uint32_t i = loads > S::kStages ? loads - S::kStages : 0; i < loads; i++) {
        const uint32_t st = i % S::kStages;
        if (s.kv_raw >> st & 1) settle(&s.raw_full[st], (s.kv_raw_use >> st & 1) ^ 1);
        else settle(&s.kv_full[st], (i / S::kStages) & 1);
      }
    } else if (warp == 11) {
      for (int t = 0; t < 2; t++)
        if (s.q_loads[t]) settle(&s.q_full[t], (s.q_loads[t] - 1) & 1);
    }
    __syncthreads();
  }
  if (warp == 9) tc_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------ merge

// Adds up an item's parts in key order: block c's item, if it goes on, and the
// first slots of the blocks after it.  A warp takes 8 rows and 64 of their dims,
// kBatch parts at a time.  Two need 64 registers, four blocks an SM, and win where
// there are many rows, whose chains are short and fill the SMs (questions to a
// shared text 96.6 us with two, 97.8 with four); four win where there are few,
// whose chains are long (16 tokens behind one prefix, 23 parts: 42.8 and 36.6 us);
// even at 8192 rows.  32 dims a warp make more blocks than run at once, each of
// which first fetches its slot (98.4 and 38.6).
template <int D, int kBatch>
__global__ void __launch_bounds__(256, 8 / kBatch) kv_merge_kernel(const KvAttnArgs a) {
  constexpr int kVecs = 4;               // of 4 dims, a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, blocks = gridDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, blocks);
  const Slot m = ws.slots[2 * c + 1];
  if (m.state != 1) return;
  const int job = blockIdx.y * 8 + warp, r = job / (D / 64) * 8 + (lane & 7), c4 = job % (D / 64) * 16 + (lane >> 3);
  if (r - (lane & 7) >= m.ntok * a.grp) return;
  int parts = 1;
  bool nan = m.nan;
  for (int i0 = c + 1; i0 < blocks; i0 += 32) {
    const int i = i0 + lane;
    const int state = i < blocks ? ws.slots[2 * i].state : 2, bad = i < blocks ? ws.slots[2 * i].nan : 0;
    const unsigned last = __ballot_sync(0xffffffffu, state != 1);
    const int n = last ? __ffs(last) : 32;
    nan |= (__ballot_sync(0xffffffffu, bad) & (n == 32 ? 0xffffffffu : (1u << n) - 1)) != 0;
    parts += n;
    if (last) break;
  }
  if (r >= m.ntok * a.grp) return;
  const int tt = kTile / a.grp, tok = r / a.grp, h = r - tok * a.grp, tile = tok / tt;
  const int row = 128 * tile + (tok - tile * tt) * a.grp + h;
  float top = -INFINITY, den = 0.f;
  float4 num[kVecs] = {};
  for (int i0 = 0; i0 < parts; i0 += kBatch) {
    float ref[kBatch], l[kBatch];
    float4 o[kBatch][kVecs];
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      ref[u] = -INFINITY, l[u] = 0.f;
#pragma unroll
      for (int v = 0; v < kVecs; v++) o[u][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < parts) {
        const float* d = ws.data + (i0 + u ? 2 * (c + i0 + u) : 2 * c + 1) * slot_floats(D);
        ref[u] = d[256 * D + row], l[u] = d[256 * D + 256 + row];
#pragma unroll
        for (int v = 0; v < kVecs; v++) o[u][v] = ((const float4*)d)[(c4 + 4 * v) * 256 + row];
      }
    }
    float high = top;
#pragma unroll
    for (int u = 0; u < kBatch; u++) high = fmaxf(high, ref[u]);
    if (high == -INFINITY) continue;
    const float keep = top == high ? 1.f : tc_ex2(top - high);
    den *= keep;
#pragma unroll
    for (int v = 0; v < kVecs; v++) num[v].x *= keep, num[v].y *= keep, num[v].z *= keep, num[v].w *= keep;
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      const float w = ref[u] == high ? 1.f : tc_ex2(ref[u] - high);
      den = fmaf(l[u], w, den);
#pragma unroll
      for (int v = 0; v < kVecs; v++) {
        num[v].x = fmaf(o[u][v].x, w, num[v].x), num[v].y = fmaf(o[u][v].y, w, num[v].y);
        num[v].z = fmaf(o[u][v].z, w, num[v].z), num[v].w = fmaf(o[u][v].w, w, num[v].w);
      }
    }
    top = high;
  }
  const int64_t token = m.tok0 + tok;
  const int head = m.head * a.grp + h;
  const bool sees = (m.flags & kCausal ? m.lim + tok : m.lim) > m.kbeg;
  const bool zero = sees && den == 0.f;        // every score is -infinity
  const float inv = zero && a.groups ? 1.f : 1.f / den;
  const size_t lines = (size_t)a.total_q * a.hq, at = ((size_t)m.head * a.total_q + token) * a.grp + h;
  const int own = m.flags & kPrefix ? 0 : 1;
#pragma unroll
  for (int v = 0; v < kVecs; v++) {
    float4 o = make_float4(num[v].x * inv, num[v].y * inv, num[v].z * inv, num[v].w * inv);
    if (!sees) o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nan || (zero && !a.groups)) o = make_float4(NAN, NAN, NAN, NAN);
    const int d = 4 * (c4 + 4 * v);
    if (a.groups) ((float4*)ws.part_o)[(own * (D / 4) + d / 4) * lines + at] = o;
    else *(uint2*)(a.out + token * a.out_stride + (int64_t)head * D + d) = make_uint2(cvt_bf2(o.x, o.y), cvt_bf2(o.z, o.w));
  }
  if (a.groups && c4 == 0) ws.part_m[own * lines + at] = nan ? NAN : !sees ? -INFINITY : top == -FLT_MAX ? top : top + log2f(den);
}

// Groups: a row's common and own keys together.  A warp takes 8 lines and 32 of
// their dims.  Bound by memory where there are many rows (23,424 of 128 dims: 10
// us, 30 MB), by latency else (4 us).
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttnArgs a, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, blocks);
  const int r0 = ws.rows[0], r1 = ws.rows[1], r2 = ws.rows[2], r3 = ws.rows[3];
  const int64_t lines = (int64_t)a.total_q * a.hq;
  const float4* o = (const float4*)ws.part_o;
  for (int64_t job = blockIdx.x * 8 + (threadIdx.x >> 5); job < (lines + 7) / 8 * (D / 32); job += gridDim.x * 8) {
    const int64_t r = job / (D / 32) * 8 + (lane & 7);
    const int c4 = (int)(job % (D / 32)) * 8 + (lane >> 3);
    if (r >= lines) continue;
    const int64_t per = (int64_t)a.total_q * a.grp;
    const int kv = (int)(r / per), token = (int)((r - kv * per) / a.grp), head = kv * a.grp + (int)(r % a.grp);
    // of no sequence: nothing was written here for it
    if ((token < r0 || token >= r1) && (token < r2 || token >= r3)) continue;
    const float m0 = ws.part_m[r], m1 = ws.part_m[lines + r], high = fmaxf(m0, m1);
    const bool nan = m0 != m0 || m1 != m1 || high == -FLT_MAX, none = high == -INFINITY;   // -FLT_MAX: -infinities alone
    const float w0 = m0 == high ? 1.f : tc_ex2(m0 - high), w1 = m1 == high ? 1.f : tc_ex2(m1 - high), inv = 1.f / (w0 + w1);
#pragma unroll
    for (int v = 0; v < 2; v++) {
      const float4 x = o[(int64_t)(c4 + 4 * v) * lines + r], y = o[(int64_t)(D / 4 + c4 + 4 * v) * lines + r];
      auto both = [&](float p, float q) {
        return nan ? NAN : none ? 0.f : fmaf(w0, p, w1 * q) * inv;
      };
      *(uint2*)(a.out + token * a.out_stride + (int64_t)head * D + 4 * (c4 + 4 * v)) =
          make_uint2(cvt_bf2(both(x.x, y.x), both(x.y, y.y)), cvt_bf2(both(x.z, y.z), both(x.w, y.w)));
    }
  }
}

// ------------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_relaxed);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn.store(f, std::memory_order_relaxed);
  }
  return (PFN_cuTensorMapEncodeTiled_v12000)f;
}

// BF16 tensor of `rank` dims (innermost first; strides of the others in
// elements), 128-byte swizzle
bool make_map(CUtensorMap* map, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t bytes[3];
  for (int i = 0; i < rank - 1; i++) bytes[i] = 2 * strides[i];
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, bytes, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

template <int D>
int launch(const KvAttnArgs& a, int sms, cudaStream_t st) {
  static std::atomic<unsigned long long> raised[2];      // shared memory, once on each device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return MK_ERR_CUDA;
  if (!(raised[dev / 64].load(std::memory_order_relaxed) >> (dev % 64) & 1)) {
    if (cudaFuncSetAttribute(kv_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem) !=
        cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    raised[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_relaxed);
  }
  CUtensorMap map_q, map_k, page_k, page_v;
  const cuuint64_t page = (cuuint64_t)a.hkv * kKvPage * D;
  const cuuint64_t q_stride = a.total_q > 1 ? (cuuint64_t)a.q_stride : (cuuint64_t)a.hq * D;
  // q: 64 dims of a group's heads of a tile's tokens; pools: 64 dims of a page
  // of a head, and all its dims as halves of 64
  const cuuint64_t q_dims[3] = {D, (cuuint64_t)a.hq, (cuuint64_t)a.total_q}, q_strides[2] = {D, q_stride};
  const cuuint64_t k_dims[3] = {D, (cuuint64_t)a.hkv * kKvPage, (cuuint64_t)a.num_pages}, k_strides[2] = {D, page};
  const cuuint64_t p_dims[4] = {64, (cuuint64_t)a.hkv * kKvPage, D / 64, (cuuint64_t)a.num_pages};
  const cuuint64_t p_strides[3] = {D, 64, page};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)a.grp, (cuuint32_t)(kTile / a.grp)}, k_box[3] = {64, kKvPage, 1};
  const cuuint32_t p_box[4] = {64, kKvPage, D / 64, 1};
  if (!make_map(&map_q, a.q, 3, q_dims, q_strides, q_box) || !make_map(&map_k, a.k_pool, 3, k_dims, k_strides, k_box) ||
      !make_map(&page_k, a.k_pool, 4, p_dims, p_strides, p_box) ||
      !make_map(&page_v, a.v_pool, 4, p_dims, p_strides, p_box))
    return MK_ERR_CUDA;
  KvAttnArgs b = a;
  b.per_block = per_block(sms);
  b.aligned32 = (((uintptr_t)a.out | 2 * (uintptr_t)a.out_stride) & 31) == 0;
  kv_attention_kernel<D><<<sms, kThreads, Shape<D>::kSmem, st>>>(b, map_q, map_k, page_k, page_v);
  int rc = launched(cudaGetLastError());
  if (rc) return rc;
  // no item of up to three key tiles is cut (two parts have two each): nothing to merge
  static_assert(kMinPart == 2 && kMinWidePart >= kMinPart, "least parts");
  const bool merge = a.max_pages * kKvPage > 3 * kTile;
  if (!merge && !a.groups) return MK_OK;
  // the next kernels are launched while the one before runs, and wait for its end
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = st, cfg.attrs = &at, cfg.numAttrs = 1;
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3(sms, D / 16);      // 256 rows: 32 groups of 8 rows, D / 64 of dims, 8 warps a block
  const bool many = (long long)a.total_q * a.hq > 64 * sms;
  if (merge) rc = launched(cudaLaunchKernelEx(&cfg, many ? kv_merge_kernel<D, 2> : kv_merge_kernel<D, 4>, a));
  if (rc || !a.groups) return rc;
  cfg.gridDim = dim3((unsigned)std::min<long long>(8 * sms, ((long long)a.total_q * a.hq + 7) / 8 * (D / 32) / 8 + 1));
  return launched(cudaLaunchKernelEx(&cfg, kv_join_kernel<D>, a, sms));
}

}  // namespace

size_t kv_attention_ws(int head_dim, int hq, int total_q, int groups, int sms) {
  size_t n = (size_t)2 * sms * (sizeof(Slot) + 4 * slot_floats(head_dim));
  if (groups) n += (size_t)2 * total_q * hq * (head_dim + 1) * 4 + 16;
  return n;
}

int kv_attention_launch(const KvAttnArgs& a, int sms, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return a.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace mk

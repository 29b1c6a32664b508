// Attention of packed query rows over the BF16 paged cache (mk_kv_attention).
//
// Rows.  A block of work is 2 tiles of 128 rows of one KV head: the query heads
// of its group, token after token (row = token * grp + head), so that few tokens
// of many heads fill a tile as many tokens of few heads do.  A tile holds
// floor(128 / grp) whole tokens.  Its keys are taken 128 at a time.
//
// Shares.  Lengths are on the device only, so the blocks cut the work
// themselves: all (task, KV head, row block) items laid end to end, an item as
// long as its key tiles and kStart for its start and end, and each block of the
// grid takes an equal stretch.  A task is a sequence's own keys (causal), or a
// group's common ones (all of them seen).  A block meets at most one item that
// it does not begin and one that it does not end; these leave their sums in the
// workspace, and the merge kernel adds them up in order.  No atomics.
//
// A block, one an SM, 12 warps: two softmax warpgroups, a tile each, a thread a
// row; one warp each that copies K and V pages (TMA, a ring of 128-key tiles),
// issues the MMAs, copies Q, and clears values that some row does not see.
// S = Q K^T goes to tensor memory; the softmax threads turn it into weights and
// write them over it as BF16; O += P V takes them from there.  While one tile's
// softmax runs, the tensor cores work for the other's.
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
constexpr int kReaders = 11;             // warps that read an item: 8 softmax, MMA, Q, clear
constexpr unsigned long long kWaitNs = 4000000000ull;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
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
  float* data;             // [2 blocks][kSlotFloats]
  float* part_o;           // groups: [2][total_q][hq][D], common keys, own keys
  float* part_m;           // [2][total_q][hq] log2 of the sum of exponentials
};

__host__ __device__ __forceinline__ size_t slot_floats(int d) { return (size_t)256 * d + 512; }

__host__ __device__ __forceinline__ Ws ws_of(uint8_t* p, int d, int hq, int total_q, int blocks) {
  Ws w;
  w.slots = (Slot*)p;
  w.data = (float*)(p + (size_t)2 * blocks * sizeof(Slot));
  w.part_o = w.data + 2 * blocks * slot_floats(d);
  w.part_m = w.part_o + (size_t)2 * total_q * hq * d;
  return w;
}

// ------------------------------------------------------------------------ waits

struct Sync {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t raw_full[10];                 // a tile that is cleared before it counts as full
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t drain;
  uint32_t tmem;
  volatile int stop;
  long long scan[kThreads / 32];
  long long total, start;
  int task;
};

// Waits for the phase of this parity; false once the block gives up, or after
// kWaitNs, which makes it give up.
__device__ __forceinline__ bool wait(Sync& s, uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (int i = 1;; i++) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255) == 0) {
      if (s.stop) return false;
      const unsigned long long t = gtime_ns();
      if (!t0) t0 = t;
      if (t - t0 > kWaitNs) {
        s.stop = 1;
        flag(status, MK_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_warp(Sync& s, uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, wait(s, bar, parity, status));
}
// after giving up: what is in flight must have landed before the block ends
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = gtime_ns();
  while (!mbar_try_wait(bar, parity) && gtime_ns() - t0 < kWaitNs) {}
}

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// one BF16 pair's elements that are not finite: bit 15, bit 31
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// ----------------------------------------------------------------------- kernel

// Softmax of one tile of rows (a warpgroup), item after item
template <int D>
__device__ void softmax_role(const KvAttnArgs& a, Sync& s, Item* items, const Ws& ws, int tile, int tt) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row = 32 * warp + lane;
  const uint32_t tm = s.tmem + ((uint32_t)(32 * warp) << 16);
  const uint32_t tm_s = tm + 128 * tile, tm_o = tm + 256 + D * tile;
  const float scale = a.scale_log2;
  const int my_tok = row / a.grp, my_head = row - my_tok * a.grp;
  uint32_t steps = 0, parts = 0;
  for (int it = 0;; it++) {
    Item* slot = &items[it % kItems];
    if (!wait_warp(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status)) return;
    const Part m = *slot;
    if (m.flags & kEnd) return;
    const int tok = tile * tt + my_tok;
    const bool mine = my_tok < tt && tok < m.ntok;
    if (m.ntok > tile * tt) {
      const int lim = m.flags & kCausal ? m.lim + tok : m.kend;
      const int least = __reduce_min_sync(0xffffffffu, mine ? lim : 0x7fffffff);
      float top = -INFINITY, sum = 0.f;
      for (int j = m.k0; j < m.k1; j++, steps++) {
        if (!wait_warp(s, &s.s_full[tile], steps & 1, a.status)) return;
        tc_fence_after();
        float x[kTile];
#pragma unroll
        for (int c = 0; c < 4; c++) tc_ld32(tm_s + 32 * c, (uint32_t*)x + 32 * c);
        tc_wait_ld();
        const int t0 = m.kbeg + kTile * j;
        if (t0 + kTile > least) {
          const int seen = lim - t0;
#pragma unroll
          for (int c = 0; c < kTile; c++) x[c] = c < seen ? x[c] : -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < kTile; c += 8) {
#pragma unroll
          for (int u = 0; u < 4; u++)
            mx[u] = c + 4 + u < kTile ? fmaxf(fmaxf(mx[u], x[c + u]), x[c + 4 + u]) : fmaxf(mx[u], x[c + u]);
        }
        const float high = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // The reference moves only when a weight would pass 2^8: sums and
        // products stay within 2^8 of their size, and O is rarely rescaled.
        const bool move = high > top && (high - top) * scale > 8.f;
        if (j == m.k0) {
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
#pragma unroll
        for (int h = 0; h < 2; h++) {
          uint32_t p[32];
#pragma unroll
          for (int u = 0; u < 32; u++) {
            float2 e = __ffma2_rn(make_float2(x[64 * h + 2 * u], x[64 * h + 2 * u + 1]), sc2, off2);
            e.x = tc_ex2(e.x), e.y = tc_ex2(e.y);
            acc[u & 1] = __fadd2_rn(acc[u & 1], e);
            p[u] = cvt_bf2(e.x, e.y);
          }
          tc_st32(tm_s + 32 * h, p);
        }
        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[tile]);
      }
      // ------------------------------------------------------------ the result
      const int first = m.kbeg + kTile * m.k0, last = min(m.kend, m.kbeg + kTile * m.k1);
      const bool some = m.k1 > m.k0;
      if (some) {
        if (!wait_warp(s, &s.o_full[tile], parts & 1, a.status)) return;
        parts++;
        tc_fence_after();
      }
      const bool nan = (m.flags & kNan) || ((volatile Item*)slot)->bad;
      const bool dirty = ((volatile Item*)slot)->dirty;
      const bool sees = lim > first;                         // something in this part
      float ref = top == -INFINITY ? (sees && some ? -FLT_MAX : -INFINITY) : top * scale;
      const bool whole = m.slot < 0, parted = a.groups > 0;
      float mul = 1.f;
      if (whole) mul = sees && some ? 1.f / sum : 0.f;       // all weights zero: 1 / 0, NaN below
      const int64_t token = m.tok0 + tok;
      const int head = m.head * a.grp + my_head;
      const size_t at = ((m.flags & kPrefix ? 0 : (size_t)a.total_q) + token) * a.hq + head;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        float* o = (float*)r;
        if (some) {
          tc_ld32(tm_o + c, r);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int u = 0; u < 32; u++) o[u] = 0.f;
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
          for (int u = 0; u < 32; u++) o[u] = nan || (sees && some && sum == 0.f) ? NAN : o[u] * mul;
        }
        if (mine && whole && !parted) {
          uint4* out = (uint4*)(a.out + token * a.out_stride + (int64_t)head * D + c);
#pragma unroll
          for (int u = 0; u < 4; u++)
            out[u] = make_uint4(cvt_bf2(o[8 * u], o[8 * u + 1]), cvt_bf2(o[8 * u + 2], o[8 * u + 3]),
                                cvt_bf2(o[8 * u + 4], o[8 * u + 5]), cvt_bf2(o[8 * u + 6], o[8 * u + 7]));
        } else if (mine) {
          float4* out = (float4*)(whole ? ws.part_o + at * D + c
                                        : ws.data + m.slot * slot_floats(D) + (size_t)(128 * tile + row) * D + c);
#pragma unroll
          for (int u = 0; u < 8; u++) out[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
        __syncwarp();          // the next tensor memory load is the whole warp's
      }
      if (mine && whole && parted) ws.part_m[at] = nan ? NAN : ref == -INFINITY || ref == -FLT_MAX ? ref : ref + log2f(sum);
      if (mine && !whole) {
        float* d = ws.data + m.slot * slot_floats(D) + 256 * D + 128 * tile + row;
        d[0] = ref, d[256] = sum;
      }
      tc_fence_before();       // O has been read before the next item's first P is announced
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_empty[it % kItems]);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_kernel(const KvAttnArgs a, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using S = Shape<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Sync s;
  __shared__ Item items[kItems];
  const uint32_t q_smem = (smem_u32(raw) + 1023u) & ~1023u, kv_smem = q_smem + 2 * S::kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tt = kTile / a.grp, tb = 2 * tt, tasks = a.groups + a.batch;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, gridDim.x);

  if (tid == 0) {
    for (int i = 0; i < S::kStages; i++) mbar_init(&s.kv_full[i], 1), mbar_init(&s.kv_empty[i], 1), mbar_init(&s.raw_full[i], 1);
    for (int t = 0; t < 2; t++) {
      mbar_init(&s.q_full[t], 1), mbar_init(&s.q_empty[t], 1), mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_full[t], 4), mbar_init(&s.o_full[t], 1);
    }
    for (int i = 0; i < kItems; i++) mbar_init(&s.item_full[i], 1), mbar_init(&s.item_empty[i], kReaders);
    mbar_init(&s.drain, 1);
    s.stop = 0, s.task = -1;
    mbar_fence_init();
  }
  if (warp == 8) tc_alloc(&s.tmem, 512);

  // all tasks' cost, and the task that this block's stretch begins in
  const int chunk = (tasks + kThreads - 1) / kThreads, first = min(tasks, tid * chunk), end = min(tasks, first + chunk);
  long long mine = 0;
  for (int t = first; t < end; t++) {
    const Task k = load_task(a, t, tb, blockIdx.x == 0);
    mine += cost_before(k, k.nb, tb) * a.hkv;
  }
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) s.scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long before = incl - mine, total = 0;
  for (int w = 0; w < kThreads / 32; w++) {
    if (w < warp) before += s.scan[w];
    total += s.scan[w];
  }
  const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinShare);
  const long long pos = share * blockIdx.x, stop = min(total, pos + share);
  if (pos < total && before <= pos && pos < before + mine) {
    long long at = before;
    for (int t = first; t < end; t++) {
      const Task k = load_task(a, t, tb, false);
      const long long c = cost_before(k, k.nb, tb) * a.hkv;
      if (pos < at + c) {
        s.task = t, s.start = at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  const uint32_t tmem = s.tmem;

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
      if (s.task >= 0) {
        Stretch w(a, tt, s.task, s.start, pos, stop, lane);
        Part m;
        while (ok && w.next(&m, 2 * (int)blockIdx.x)) {
          {
            const int k0 = m.k0, k1 = m.k1, head = m.head;
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
            const int i = S::kHalves == 2 ? lane >> 1 : lane, half = S::kHalves == 2 ? lane & 1 : 0;
            const int32_t* table = a.page_tables + (int64_t)m.table * a.max_pages + m.kbeg / kKvPage + i;
            // pages of tile j for this lane; none past the keys
            auto pages_of = [&](int j) { return min(8, (m.kend - m.kbeg - kTile * j + kKvPage - 1) / kKvPage); };
            auto page_of = [&](int j) { return j < k1 && i < pages_of(j) ? table[8 * j] : 0; };
            const int clear = (m.flags & kCausal ? m.lim : m.kend) - m.kbeg;
            auto load = [&](const CUtensorMap& map, int j, int page, bool value) {
              const uint32_t st = loads % S::kStages;
              if (!wait_warp(s, &s.kv_empty[st], ((loads / S::kStages) & 1) ^ 1, a.status)) return false;
              const int np = pages_of(j);
              const bool out = i < np && (page < 0 || page >= a.num_pages);
              if (__any_sync(0xffffffffu, out)) {
                bad = true;
                if (lane == 0) ((volatile Item*)dst)->bad = 1, flag(a.status, MK_ERR_BAD_PAGE);
              }
              const bool through = value && kTile * (j + 1) > clear;
              raw = (raw & ~(1u << st)) | (uint32_t)through << st;
              raw_use ^= (uint32_t)through << st;
              uint64_t* bar = through ? &s.raw_full[st] : &s.kv_full[st];
              if (lane == 0) mbar_arrive_expect_tx(bar, np * S::kHalves * 2048);
              __syncwarp();
              // a page outside the cache: past the last one, which the copy fills with zeros
              if (i < np)
                tma_load_3d(kv_smem + st * S::kTileBytes + half * 16384 + i * 2048, &map, 64 * half, kKvPage * head,
                            out ? a.num_pages : page, bar);
              loads++;
              return true;
            };
            int cur = page_of(k0), next = page_of(k0 + 1);
            ok = k1 == k0 || load(map_k, k0, cur, false);
            for (int j = k0; ok && j < k1; j++) {
              const int later = page_of(j + 2);
              ok = load(map_v, j, cur, true);
              if (ok && j + 1 < k1) ok = load(map_k, j + 1, next, false);
              cur = next, next = later;
            }
            if (m.slot >= 0)
              desc[k0 == 0] = Slot{k1 < m.n ? 1 : 2, m.tok0, m.ntok, head, m.kbeg, m.lim, m.flags, bad};
          }
        }
      }
      if (ok && wait_warp(s, &s.item_empty[it % kItems], ((it / kItems) & 1) ^ 1, a.status) && lane == 0) {
        items[it % kItems].flags = kEnd;
        mbar_arrive(&s.item_full[it % kItems]);
      }
      if (lane < 2) ws.slots[2 * blockIdx.x + lane] = lane ? desc[1] : desc[0];
      if (s.stop) {
        for (uint32_t i = loads > S::kStages ? loads - S::kStages : 0; i < loads; i++) {
          const uint32_t st = i % S::kStages;
          if (raw >> st & 1) settle(&s.raw_full[st], (raw_use >> st & 1) ^ 1);
          else settle(&s.kv_full[st], (i / S::kStages) & 1);
        }
      }
    } else if (warp == 9) {
      // -------------------------------------------------- MMAs (one thread)
      if (lane == 0) {
        constexpr uint32_t idesc_s = tc_idesc(kTile, false), idesc_o = tc_idesc(D, true);
        uint32_t loads = 0, items_q[2] = {0, 0}, steps[2] = {0, 0};
        bool ok = true;
        auto qk = [&](int t, uint32_t st) {
          const uint32_t qa = q_smem + t * S::kTileBytes, kb = kv_smem + st * S::kTileBytes;
#pragma unroll
          for (int c = 0; c < D / 16; c++) {
            const uint32_t off = c / 4 * 16384 + c % 4 * 32;
            tc_mma_ss(tmem + 128 * t, tc_desc(qa + off), tc_desc(kb + off), idesc_s, c > 0);
          }
        };
        auto pv = [&](int t, uint32_t st, bool acc) {
          const uint32_t vb = kv_smem + st * S::kTileBytes;
#pragma unroll
          for (int c = 0; c < kTile / 16; c++)
            tc_mma_ts(tmem + 256 + D * t, tmem + 128 * t + 8 * c, tc_desc(vb + 2048 * c, 16384), idesc_o, acc || c > 0);
        };
        auto full = [&](uint32_t i) {
          ok = ok && wait(s, &s.kv_full[i % S::kStages], (i / S::kStages) & 1, a.status);
          tc_fence_after();
        };
        for (int it = 0; ok; it++) {
          ok = wait(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status);
          if (!ok) break;
          const Item& m = items[it % kItems];
          const int flags = m.flags, k0 = m.k0, k1 = m.k1, tiles = m.ntok > tt ? 2 : 1;
          if (flags & kEnd) break;
          mbar_arrive(&s.item_empty[it % kItems]);
          if (k1 == k0) continue;
          full(loads);
          for (int t = 0; ok && t < tiles; t++) {
            ok = wait(s, &s.q_full[t], items_q[t]++ & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            qk(t, loads % S::kStages);
            tc_commit(&s.s_full[t]);
            if (k1 == k0 + 1) tc_commit(&s.q_empty[t]);
          }
          tc_commit(&s.kv_empty[loads % S::kStages]);
          loads++;
          for (int j = k0; ok && j < k1; j++) {
            const uint32_t sv = loads % S::kStages, sk = (loads + 1) % S::kStages;
            const bool more = j + 1 < k1;
            full(loads);
            for (int t = 0; ok && t < tiles; t++) {
              ok = wait(s, &s.p_full[t], steps[t]++ & 1, a.status);
              if (!ok) break;
              tc_fence_after();
              pv(t, sv, j > k0);
              if (more) {
                if (t == 0) full(loads + 1);
                if (!ok) break;
                qk(t, sk);
                tc_commit(&s.s_full[t]);
                if (j + 2 == k1) tc_commit(&s.q_empty[t]);
              } else {
                tc_commit(&s.o_full[t]);
              }
            }
            tc_commit(&s.kv_empty[sv]);
            if (more) tc_commit(&s.kv_empty[sk]);
            loads += more ? 2 : 1;
          }
        }
        // nothing may arrive on a barrier after the block's end
        tc_commit(&s.drain);
        settle(&s.drain, 0);
      }
    } else if (warp == 10) {
      // --------------------------------------------------- Q (one thread)
      if (lane == 0) {
        uint32_t loads[2] = {0, 0};
        bool ok = true;
        const uint32_t bytes = (uint32_t)(tt * a.grp) * 128 * S::kHalves;
        for (int it = 0; ok; it++) {
          ok = wait(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status);
          if (!ok) break;
          const Part m = items[it % kItems];
          if (m.flags & kEnd) break;
          mbar_arrive(&s.item_empty[it % kItems]);
          for (int t = 0; ok && m.k1 > m.k0 && t < 2 && m.ntok > t * tt; t++) {
            ok = wait(s, &s.q_empty[t], (loads[t] & 1) ^ 1, a.status);
            if (!ok) break;
            loads[t]++;
            mbar_arrive_expect_tx(&s.q_full[t], bytes);
            for (int h = 0; h < S::kHalves; h++)
              tma_load_3d(q_smem + t * S::kTileBytes + h * 16384, &map_q, 64 * h, m.head * a.grp, m.tok0 + t * tt,
                          &s.q_full[t]);
          }
        }
        if (s.stop)
          for (int t = 0; t < 2; t++)
            if (loads[t]) settle(&s.q_full[t], (loads[t] - 1) & 1);
      }
    } else {
      // ---------------- values that some row does not see (whole warp): a
      // weight of zero times NaN or an infinity is no zero, so those are taken
      // out, and what a page holds past the sequence with them
      uint32_t loads = 0, uses = 0;
      bool ok = true;
      for (int it = 0; ok; it++) {
        ok = wait_warp(s, &s.item_full[it % kItems], (it / kItems) & 1, a.status);
        if (!ok) break;
        Item* slot = &items[it % kItems];
        const Part m = *slot;
        if (m.flags & kEnd) break;
        const int clear = (m.flags & kCausal ? m.lim : m.kend) - m.kbeg;
        for (int j = m.k0; ok && j < m.k1; j++) {
          if (kTile * (j + 1) <= clear) continue;
          const uint32_t i = loads + 2 * (j - m.k0) + 1, st = i % S::kStages;
          ok = wait_warp(s, &s.raw_full[st], uses >> st & 1, a.status);
          if (!ok) break;
          uses ^= 1u << st;
          const int lo = max(0, clear - kTile * j), held = m.kend - m.kbeg - kTile * j;
          const uint32_t base = kv_smem + st * S::kTileBytes;
          bool found = false;
#pragma unroll 4
          for (int c = 8 * lo + lane; c < 8 * kTile; c += 32) {
#pragma unroll
            for (int h = 0; h < S::kHalves; h++) {
              const uint32_t at = base + 16384 * h + 16 * c;
              uint32_t w[4];
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
              const bool past = c / 8 >= held;
              const uint32_t nf = not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
              if (past || nf) {
                found |= !past;
#pragma unroll
                for (int u = 0; u < 4; u++) {
                  const uint32_t b = not_finite(w[u]);
                  w[u] = past ? 0u : w[u] & ~((b & 0x8000u ? 0xffffu : 0u) | (b & 0x80000000u ? 0xffff0000u : 0u));
                }
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
              }
            }
          }
          if (found) ((volatile Item*)slot)->dirty = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.kv_full[st]);
        }
        loads += 2 * (m.k1 - m.k0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.item_empty[it % kItems]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tc_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------ merge

// Adds up an item's parts in key order, a warp a row: part c's first item (if
// it goes on) and the first slots of the blocks after it.
constexpr int kMergeRows = 16;             // blocks of rows (gridDim.y)

template <int D>
__global__ void __launch_bounds__(256) kv_merge_kernel(const KvAttnArgs a) {
  constexpr int V = D / 32, kBatch = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, blocks = gridDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, blocks);
  const Slot m = ws.slots[2 * c + 1];
  if (m.state != 1) return;
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
  const int tt = kTile / a.grp;
  for (int r = blockIdx.y + gridDim.y * warp; r < m.ntok * a.grp; r += gridDim.y * 8) {
    const int tok = r / a.grp, h = r - tok * a.grp, tile = tok / tt;
    const int row = 128 * tile + (tok - tile * tt) * a.grp + h;
    float top = -INFINITY, den = 0.f, num[V];
#pragma unroll
    for (int v = 0; v < V; v++) num[v] = 0.f;
    for (int i0 = 0; i0 < parts; i0 += kBatch) {
      float ref[kBatch], l[kBatch], o[kBatch][V];
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        ref[u] = -INFINITY, l[u] = 0.f;
#pragma unroll
        for (int v = 0; v < V; v++) o[u][v] = 0.f;
        if (i0 + u < parts) {
          const float* d = ws.data + (i0 + u ? 2 * (c + i0 + u) : 2 * c + 1) * slot_floats(D);
          ref[u] = d[256 * D + row], l[u] = d[256 * D + 256 + row];
#pragma unroll
          for (int v = 0; v < V; v++) o[u][v] = d[(size_t)row * D + 32 * v + lane];
        }
      }
      float high = top;
#pragma unroll
      for (int u = 0; u < kBatch; u++) high = fmaxf(high, ref[u]);
      if (high == -INFINITY) continue;
      const float keep = top == high ? 1.f : tc_ex2(top - high);
      den = keep == 0.f ? 0.f : den * keep;
#pragma unroll
      for (int v = 0; v < V; v++) num[v] = keep == 0.f ? 0.f : num[v] * keep;
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const float w = ref[u] == high ? 1.f : tc_ex2(ref[u] - high);
        if (w == 0.f) continue;            // nothing of it is left, whatever it holds
        den = fmaf(l[u], w, den);
#pragma unroll
        for (int v = 0; v < V; v++) num[v] = fmaf(o[u][v], w, num[v]);
      }
      top = high;
    }
    const int64_t token = m.tok0 + tok;
    const int head = m.head * a.grp + h;
    const bool sees = (m.flags & kCausal ? m.lim + tok : m.lim) > m.kbeg;
#pragma unroll
    for (int v = 0; v < V; v++) num[v] = nan ? NAN : sees ? num[v] / den : 0.f;
    if (a.groups) {
      const size_t at = ((m.flags & kPrefix ? 0 : (size_t)a.total_q) + token) * a.hq + head;
#pragma unroll
      for (int v = 0; v < V; v++) ws.part_o[at * D + 32 * v + lane] = num[v];
      if (lane == 0) ws.part_m[at] = nan ? NAN : !sees ? -INFINITY : top == -FLT_MAX ? top : top + log2f(den);
    } else {
      uint16_t* out = a.out + token * a.out_stride + (int64_t)head * D;
#pragma unroll
      for (int v = 0; v < V; v++) out[32 * v + lane] = f2bf(num[v]);
    }
  }
}

// Groups: a row's common and own keys together
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttnArgs a, int blocks) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const Ws ws = ws_of(a.ws, D, a.hq, a.total_q, blocks);
  const int t0 = max(0, a.q_starts[0]), t1 = min(a.total_q, a.q_starts[a.batch]);
  const int64_t rows = (int64_t)a.total_q * a.hq;
  for (int64_t r = (int64_t)t0 * a.hq + blockIdx.x * 8 + (threadIdx.x >> 5); r < (int64_t)t1 * a.hq; r += gridDim.x * 8) {
    const float m0 = ws.part_m[r], m1 = ws.part_m[rows + r];
    const float high = fmaxf(m0, m1);
    float o[V];
    if (m0 != m0 || m1 != m1) {
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = NAN;
    } else if (high == -INFINITY) {
#pragma unroll
      for (int v = 0; v < V; v++) o[v] = 0.f;
    } else {
      const float w0 = m0 == high ? 1.f : tc_ex2(m0 - high), w1 = m1 == high ? 1.f : tc_ex2(m1 - high);
      const float inv = 1.f / (w0 + w1);
#pragma unroll
      for (int v = 0; v < V; v++) {
        const float x = w0 == 0.f ? 0.f : w0 * ws.part_o[r * D + 32 * v + lane];
        const float y = w1 == 0.f ? 0.f : w1 * ws.part_o[(rows + r) * D + 32 * v + lane];
        o[v] = (x + y) * inv;
      }
    }
    uint16_t* out = a.out + r / a.hq * a.out_stride + r % a.hq * D;
#pragma unroll
    for (int v = 0; v < V; v++) out[32 * v + lane] = f2bf(o[v]);
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

// [n2][n1][D] BF16, rows of D elements at stride1 elements, planes at stride2;
// boxes of 64 dims x box1 x box2
bool make_map(CUtensorMap* map, const void* p, int d, uint64_t n1, uint64_t n2, uint64_t stride1, uint64_t stride2,
              uint32_t box1, uint32_t box2) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, n1, n2}, strides[2] = {stride1 * 2, stride2 * 2};
  const cuuint32_t box[3] = {64, box1, box2}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
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
  CUtensorMap mq, mk_, mv;
  const uint64_t page = (uint64_t)a.hkv * kKvPage * D;
  const uint64_t q_stride = a.total_q > 1 ? (uint64_t)a.q_stride : (uint64_t)a.hq * D;
  if (!make_map(&mq, a.q, D, a.hq, a.total_q, D, q_stride, a.grp, kTile / a.grp) ||
      !make_map(&mk_, a.k_pool, D, (uint64_t)a.hkv * kKvPage, a.num_pages, D, page, kKvPage, 1) ||
      !make_map(&mv, a.v_pool, D, (uint64_t)a.hkv * kKvPage, a.num_pages, D, page, kKvPage, 1))
    return MK_ERR_CUDA;
  kv_attention_kernel<D><<<sms, kThreads, Shape<D>::kSmem, st>>>(a, mq, mk_, mv);
  int rc = launched(cudaGetLastError());
  if (rc) return rc;
  // the next kernels are launched while the one before runs, and wait for its end
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = st, cfg.attrs = &at, cfg.numAttrs = 1;
  cfg.blockDim = dim3(256);
  cfg.gridDim = dim3(sms, kMergeRows);
  rc = launched(cudaLaunchKernelEx(&cfg, kv_merge_kernel<D>, a));
  if (rc || !a.groups) return rc;
  cfg.gridDim = dim3((unsigned)std::min<long long>(8 * sms, ((long long)a.total_q * a.hq + 7) / 8));
  return launched(cudaLaunchKernelEx(&cfg, kv_join_kernel<D>, a, sms));
}

}  // namespace

size_t kv_attention_ws(int head_dim, int hq, int total_q, int groups, int sms) {
  size_t n = (size_t)2 * sms * (sizeof(Slot) + 4 * slot_floats(head_dim));
  if (groups) n += (size_t)2 * total_q * hq * (head_dim + 1) * 4;
  return n;
}

int kv_attention_launch(const KvAttnArgs& a, int sms, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  return a.head_dim == 128 ? launch<128>(a, sms, st) : launch<64>(a, sms, st);
}

}  // namespace mk

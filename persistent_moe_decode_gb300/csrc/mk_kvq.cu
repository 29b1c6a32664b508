// Operators of the 4-bit key/value cache (declared in include/mk.h): rows or
// pages quantised into it, read back from it, and one-token attention over it.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "../../include/mk.h"
#include "mk_kvq.cuh"

using namespace mk;

namespace {

// rows of keys and values outside the cache, as the kernels see them
struct Rows {
  void *k, *v;
  long long page, row, head;               // strides in elements
  int count;                               // rows (or pages) there are
};

struct Cache {
  uint8_t* pool;
  int32_t* status;
  int pages, hkv;
};

__device__ __forceinline__ void flag_bad(const Cache& c, int code) {
  if (c.status) *c.status = code;          // every writer stores a code of an error
}

// eight consecutive elements
__device__ __forceinline__ void load8(float* x, const uint16_t* p) {
  const uint4 t = __ldg((const uint4*)p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ void load8(float* x, const float* p) {
  const float4 a = __ldg((const float4*)p), b = __ldg((const float4*)p + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float* x) {
  *(uint4*)p = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
  *((float4*)p + 1) = make_float4(x[4], x[5], x[6], x[7]);
}

// Token `i` of a call whose indexes count units of 1 token or of a page:
// the row of the outside view and the slot of the cache it goes with, or < 0.
__device__ __forceinline__ long long unit_token(const int32_t* index, int i, int unit) {
  const int u = i / unit;
  const int at = index ? index[u] : u;
  return at < 0 ? -1 : (long long)at * unit + i % unit;
}

// Eight dims a thread, the eight threads of a scale group side by side: group
// octet e = ((token hkv + head) 2 + key / value) NG + group.
struct Octet {
  int i, head, val, group;
};
template <int D>
__device__ __forceinline__ Octet octet(long long e, int hkv) {
  constexpr int NG = D / kKvqGroup;
  Octet o;
  o.group = (int)(e % NG);
  e /= NG;
  o.val = (int)(e & 1);
  e >>= 1;
  o.head = (int)(e % hkv);
  o.i = (int)(e / hkv);
  return o;
}

template <int D, class T>
__global__ void __launch_bounds__(256) kvq_write_kernel(Cache c, Rows src, const int32_t* src_index,
                                                        const int32_t* dst_index, int tokens, int unit) {
  using R = KvqRec<D>;
  const long long octets = (long long)tokens * c.hkv * 2 * R::NG;
  const int wi = threadIdx.x & 7;
  const unsigned mask = 0xffu << (threadIdx.x & 24);
  for (long long e = (blockIdx.x * 256ll + threadIdx.x) >> 3; e < octets; e += gridDim.x * 32ll) {
    const Octet o = octet<D>(e, c.hkv);
    const long long from = unit_token(src_index, o.i, unit), to = unit_token(dst_index, o.i, unit);
    if (from < 0 || to < 0) continue;
    if (from >= (long long)src.count * unit || to >= (long long)c.pages * kKvqPage) {
      flag_bad(c, MK_ERR_BAD_PAGE);
      continue;
    }
    const T* row = (const T*)(o.val ? src.v : src.k) + from / kKvqPage * src.page + from % kKvqPage * src.row +
                   o.head * src.head + o.group * kKvqGroup + wi * 8;
    float x[8];
    load8(x, row);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) {
      lo = fmin_nan(lo, x[i]);
      hi = fmax_nan(hi, x[i]);
    }
#pragma unroll
    for (int sh = 1; sh < 8; sh <<= 1) {
      lo = fmin_nan(lo, __shfl_xor_sync(mask, lo, sh));
      hi = fmax_nan(hi, __shfl_xor_sync(mask, hi, sh));
    }
    const KvqScale s = kvq_scale(lo, hi);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) word |= kvq_code(x[i], s) << (4 * i);
    const int t = (int)(to % kKvqPage);
    uint8_t* rec = c.pool + ((to / kKvqPage) * c.hkv + o.head) * R::kBytes;
    if (o.val) {
      *(uint16_t*)(rec + R::val_half(t, wi, o.group, 0)) = (uint16_t)word;
      *(uint16_t*)(rec + R::val_half(t, wi, o.group, 1)) = (uint16_t)(word >> 16);
    } else {
      *(uint32_t*)(rec + R::key_word(t, wi, o.group)) = word;
    }
    if (wi == 0)
      *(uint32_t*)(rec + (o.val ? R::kValScale : R::kKeyScale) + 4 * (t * R::NG + o.group)) = s.word();
  }
}

template <int D, class T>
__global__ void __launch_bounds__(256) kvq_read_kernel(Cache c, const int32_t* src_index, Rows dst,
                                                       const int32_t* dst_index, int tokens, int unit) {
  using R = KvqRec<D>;
  const long long octets = (long long)tokens * c.hkv * 2 * R::NG;
  const int wi = threadIdx.x & 7;
  for (long long e = (blockIdx.x * 256ll + threadIdx.x) >> 3; e < octets; e += gridDim.x * 32ll) {
    const Octet o = octet<D>(e, c.hkv);
    const long long from = unit_token(src_index, o.i, unit), to = unit_token(dst_index, o.i, unit);
    if (to < 0) continue;
    if (from >= (long long)c.pages * kKvqPage || to >= (long long)dst.count * unit) {
      flag_bad(c, MK_ERR_BAD_PAGE);
      continue;
    }
    float x[8];
    if (from < 0) {
#pragma unroll
      for (int i = 0; i < 8; i++) x[i] = 0.f;
    } else {
      const int t = (int)(from % kKvqPage);
      const uint8_t* rec = c.pool + ((from / kKvqPage) * c.hkv + o.head) * R::kBytes;
      uint32_t word;
      if (o.val)
        word = *(const uint16_t*)(rec + R::val_half(t, wi, o.group, 0)) |
               ((uint32_t)*(const uint16_t*)(rec + R::val_half(t, wi, o.group, 1)) << 16);
      else
        word = *(const uint32_t*)(rec + R::key_word(t, wi, o.group));
      const uint32_t s =
          *(const uint32_t*)(rec + (o.val ? R::kValScale : R::kKeyScale) + 4 * (t * R::NG + o.group));
#pragma unroll
      for (int i = 0; i < 8; i++) x[i] = fmaf((float)((word >> (4 * i)) & 15u), bf16lo(s), bf16hi(s));
    }
    T* row = (T*)(o.val ? dst.v : dst.k) + to / kKvqPage * dst.page + to % kKvqPage * dst.row + o.head * dst.head +
             o.group * kKvqGroup + wi * 8;
    store8(row, x);
  }
}

// ---------------------------------------------------------------- attention
//
// The pages of all tasks (sequence, KV head, 8 of its query heads) are cut
// into segments by the blocks themselves from the lengths on the device, so
// the host neither reads lengths nor launches for the longest one:
//   few pages (less than kMinPages a block): segments of kMinPages pages, one
//     page a warp, dealt to the blocks in turn;
//   many: block i takes units T i / G .. T (i + 1) / G of the T pages of all
//     tasks in order, so every block moves the same bytes whatever the mix of
//     lengths.
// A task that is one segment is written at once.  The segments of the others
// leave (reference, sum, weighted sum) in workspace slots, at most two a block,
// and a second kernel merges them in page order: no atomics, one result.

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = kAttnWarps * 32;
// resident blocks: the fp32 kernel with 128 dims needs more than the 128
// registers a thread that two blocks leave
template <int D, class T>
constexpr int kBlocksPerSm = D == 128 && sizeof(T) == 4 ? 1 : 2;
constexpr int kMinPages = kAttnWarps;
constexpr int kRing = 4;                   // pages of a warp in flight and in use

struct AttnArgs {
  Cache c;
  const void* q;
  void* out;
  const int32_t* page_tables;
  const int32_t* seq_lens;
  uint8_t* ws;                             // AttnWs
  long long q_stride, out_stride;          // elements between two sequences
  int grp, tiles, batch, max_pages;        // tiles = ceil(grp / 8)
  int split;                               // 0: every task is one segment
  float scale_log2;
};

// workspace: the slot count, a header per slot, then the slots
struct AttnSlot {
  int b, j;                                // sequence; KV head and head tile
  int parts;                               // of the task, in its first slot; 0 in the others
  int step;                                // 1: parts in consecutive slots; 2: in the even slots after the first
};

struct AttnWs {
  int32_t* count;
  AttnSlot* slots;
  float* data;
};

__host__ __device__ inline size_t attn_slot_floats(int d) { return 8 * (size_t)d + 16; }

__host__ __device__ inline size_t attn_ws_bytes(int blocks, int d) {
  const size_t slots = 2 * (size_t)blocks;
  return 16 + slots * sizeof(AttnSlot) + slots * attn_slot_floats(d) * 4;
}

__device__ __forceinline__ AttnWs attn_ws(uint8_t* p, int blocks) {
  return {(int32_t*)p, (AttnSlot*)(p + 16), (float*)(p + 16 + 2 * (size_t)blocks * sizeof(AttnSlot))};
}

__device__ __forceinline__ void stf(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// pages of sequence b; -1 for a length out of range
__device__ __forceinline__ int seq_pages(const AttnArgs& a, int b) {
  const int len = a.seq_lens[b];
  return len < 0 || len > a.max_pages * kKvqPage ? -1 : (len + kKvqPage - 1) / kKvqPage;
}

// Position in the list of sequences: the sums before sequence b of its pages
// (or segments) and of its split segments
struct Cursor {
  int b;
  long long units;
  int split;
};

struct PlanSmem {
  long long units[kAttnWarps];
  int split[kAttnWarps];
  Cursor found;
};

// The sequence, from `c` on, whose pages (seg: segments) hold number `target`;
// batch if there is none.  All threads call it and get the same answer.
__device__ Cursor find_sequence(const AttnArgs& a, PlanSmem& S, Cursor c, long long target, bool seg) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  while (c.b < a.batch) {
    const int b = c.b + tid;
    const int np = b < a.batch ? max(seq_pages(a, b), 0) : 0;
    const int n = seg ? (np + kMinPages - 1) / kMinPages : np;
    const int m = seg && n > 1 ? n : 0;
    long long u = n;
    int sp = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, u, o);
      const int y = __shfl_up_sync(0xffffffffu, sp, o);
      if (lane >= o) u += x, sp += y;
    }
    if (lane == 31) S.units[warp] = u, S.split[warp] = sp;
    __syncthreads();
    long long ub = c.units, ut = c.units;
    int sb = c.split, st = c.split;
    for (int w = 0; w < kAttnWarps; w++) {
      if (w == warp) ub = ut, sb = st;
      ut += S.units[w];
      st += S.split[w];
    }
    const long long before = ub + u - n;
    if (n > 0 && before <= target && target < before + n) S.found = {b, before, sb + sp - m};
    __syncthreads();
    if (target < ut) {
      c = S.found;
      __syncthreads();                     // the next call writes S again
      return c;
    }
    c = {c.b + kAttnThreads, ut, st};
  }
  c.b = a.batch;
  return c;
}

// output row of head h of task (b, j)
template <int D, class T>
__device__ __forceinline__ T* out_row(const AttnArgs& a, int b, int j, int h) {
  const int g = j / a.tiles, h0 = j % a.tiles * 8;
  return (T*)a.out + b * a.out_stride + (long long)(g * a.grp + h0 + h) * D;
}

template <int D, class T>
struct AttnBlock {
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  using R = KvqRec<D>;
  using A = KvqAttn<D, TERMS, TERMS>;
  static constexpr int NG = R::NG;
  static constexpr int kPad = D + 8;       // row of the merge buffer: rows of one store fall in distinct banks
  static constexpr size_t kRingBytes = (size_t)kAttnWarps * kRing * R::kBytes;
  static constexpr size_t kMergeBytes = (size_t)kAttnWarps * 8 * (kPad + 2) * 4;
  static constexpr size_t kSmem = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;

  // pages [p0, p1) of task (b, j): its output row, or slot `slot` of the workspace
  static __device__ void segment(const AttnArgs& a, uint8_t* smem, int b, int j, int p0, int p1, float* slot) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane >> 2, cq = lane & 3;
    const int g = j / a.tiles, h0 = j % a.tiles * 8, heads = min(8, a.grp - h0);
    const int len = a.seq_lens[b];
    uint8_t* ring = smem + (size_t)warp * kRing * R::kBytes;
    const int32_t* table = a.page_tables + (long long)b * a.max_pages + p0 + warp;
    const int n = (p1 - p0 - warp + kAttnWarps - 1) / kAttnWarps;   // this warp's pages (may be <= 0)
    bool bad = false;
    // page numbers: 32 of the warp's pages at a time, a lane each
    int ids = lane < n ? table[lane * kAttnWarps] : 0;
    auto fetch = [&](int i) {              // page i of the warp into its ring slot
      if (i < n) {
        if (i && (i & 31) == 0) ids = i + lane < n ? table[(long long)(i + lane) * kAttnWarps] : 0;
        int id = __shfl_sync(0xffffffffu, ids, i & 31);
        if (id < 0 || id >= a.c.pages) {
          bad = true;
          id = 0;
        }
        const uint8_t* src = a.c.pool + ((long long)id * a.c.hkv + g) * R::kBytes;
        uint8_t* dst = ring + (i % kRing) * R::kBytes;
#pragma unroll
        for (int k = 0; k < (R::kBytes + 511) / 512; k++)
          if (k * 512 + lane * 16 < R::kBytes) cp_async16(dst + k * 512 + lane * 16, src + k * 512 + lane * 16);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; i++) fetch(i);

    A at;
    {
      float x[NG][16];
      const T* q = (const T*)a.q + b * a.q_stride + (long long)(g * a.grp + h0 + min(gl, heads - 1)) * D + cq * 16;
#pragma unroll
      for (int k = 0; k < NG; k++) {
        load8(x[k], q + k * kKvqGroup);
        load8(x[k] + 8, q + k * kKvqGroup + 8);
        if (gl >= heads)
#pragma unroll
          for (int i = 0; i < 16; i++) x[k][i] = 0.f;
      }
      at.init(x, a.scale_log2, lane);
    }
    for (int i = 0; i < n; i++) {
      cp_async_wait<kRing - 2>();
      __syncwarp();
      typename A::Page pg;
      A::load(pg, ring + (i % kRing) * R::kBytes, lane);
      // the slot fetched into now was read in the iteration before
      fetch(i + kRing - 1);
      at.page(pg, min(kKvqPage, len - (p0 + warp + i * kAttnWarps) * kKvqPage), lane);
    }
    cp_async_wait<0>();
    if (bad && lane == 0) flag_bad(a.c, MK_ERR_BAD_PAGE);

    float v[NG][2][8];
    at.finish(v);
    __syncthreads();                       // every warp is through its ring
    float* mo = (float*)smem;              // [warp][8][kPad], then references and sums [warp][8] each
    float* mr = mo + (size_t)kAttnWarps * 8 * kPad;
    float* ml = mr + kAttnWarps * 8;
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int k = 0; k < NG; k++) {
        float* dst = mo + (warp * 8 + 2 * cq + h) * kPad + k * kKvqGroup + 8 * gl;
        *(float4*)dst = make_float4(v[k][h][0], v[k][h][1], v[k][h][2], v[k][h][3]);
        *(float4*)(dst + 4) = make_float4(v[k][h][4], v[k][h][5], v[k][h][6], v[k][h][7]);
      }
      if (gl == 0) {
        mr[warp * 8 + 2 * cq + h] = at.r[h];
        ml[warp * 8 + 2 * cq + h] = bad ? NAN : at.l[h];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * (D / 4); i += kAttnThreads) {
      const int h = i / (D / 4), dim = i % (D / 4) * 4;
      float m = -FLT_MAX, den = 0.f, num[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kAttnWarps; w++) m = fmaxf(m, mr[w * 8 + h]);
#pragma unroll
      for (int w = 0; w < kAttnWarps; w++) {
        const float k = ex2(mr[w * 8 + h] - m);
        const float4 o = *(const float4*)(mo + (w * 8 + h) * kPad + dim);
        num[0] = fmaf(k, o.x, num[0]);
        num[1] = fmaf(k, o.y, num[1]);
        num[2] = fmaf(k, o.z, num[2]);
        num[3] = fmaf(k, o.w, num[3]);
        den = fmaf(k, ml[w * 8 + h], den);
      }
      if (slot) {
        *(float4*)(slot + h * D + dim) = make_float4(num[0], num[1], num[2], num[3]);
        if (dim == 0) {
          slot[8 * D + h] = m;
          slot[8 * D + 8 + h] = den;
        }
      } else {
        T* dst = out_row<D, T>(a, b, j, h) + dim;
#pragma unroll
        for (int k = 0; k < 4; k++) stf(dst + k, num[k] / den);
      }
    }
    __syncthreads();                       // the ring may be filled again
  }
};

template <int D, class T>
__global__ void __launch_bounds__(kAttnThreads, kBlocksPerSm<D, T>) kvq_attention_kernel(AttnArgs a) {
  using B = AttnBlock<D, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ PlanSmem S;
  const int tid = threadIdx.x, G = gridDim.x, me = blockIdx.x, HT = a.c.hkv * a.tiles;

  // all pages; rows of sequences without one
  long long total = 0;
  for (int b = tid; b < a.batch; b += kAttnThreads) total += max(seq_pages(a, b), 0);
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if ((tid & 31) == 0) S.units[tid >> 5] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kAttnWarps; w++) total += S.units[w];
  __syncthreads();
  for (int b = me; b < a.batch; b += G) {
    const int np = seq_pages(a, b);
    if (np > 0) continue;
    if (np < 0 && tid == 0) flag_bad(a.c, MK_ERR_BAD_ARG);
    for (int i = tid; i < a.c.hkv * a.grp * D; i += kAttnThreads)
      stf((T*)a.out + b * a.out_stride + i, np < 0 ? NAN : 0.f);
  }

  const unsigned long long T0 = (unsigned long long)total * HT;
  const AttnWs ws = attn_ws(a.ws, G);
  if (!a.split || T0 < (unsigned long long)G * kMinPages) {
    Cursor cur{0, 0, 0};
    for (long long s = me;; s += G) {
      cur = find_sequence(a, S, cur, s / HT, true);
      if (cur.b >= a.batch) break;
      const int np = seq_pages(a, cur.b), nc = (np + kMinPages - 1) / kMinPages;
      const long long rem = s - cur.units * HT;
      const int j = (int)(rem / nc), k = (int)(rem % nc);
      const int slot = cur.split * HT + (int)rem;
      if (nc > 1 && tid == 0) ws.slots[slot] = {cur.b, j, k == 0 ? nc : 0, 1};
      B::segment(a, smem, cur.b, j, k * kMinPages, min(np, (k + 1) * kMinPages),
                 nc > 1 ? ws.data + slot * attn_slot_floats(D) : nullptr);
    }
    if (a.split && me == 0 && tid == 0) *ws.count = cur.split * HT;
  } else {
    if (me == 0 && tid == 0) *ws.count = 2 * G;
    unsigned long long u = T0 * me / G;
    const unsigned long long end = T0 * (me + 1) / G;
    Cursor cur{0, 0, 0};
    bool first = true;
    if (tid < 2) ws.slots[2 * me + tid].parts = 0;
    __syncthreads();
    while (u < end) {
      cur = find_sequence(a, S, cur, (long long)(u / HT), false);
      const int np = seq_pages(a, cur.b);
      const unsigned long long rem = u - (unsigned long long)cur.units * HT;
      const int j = (int)(rem / np), p0 = (int)(rem % np);
      const unsigned long long task = u - p0;              // first unit of the task
      const int p1 = (int)min((unsigned long long)np, p0 + (end - u));
      const bool part = p0 > 0 || p1 < np;
      const int slot = 2 * me + (first ? 0 : 1);
      if (p0 == 0 && part && tid == 0) {
        // the block that holds the task's last unit x: the largest i with T0 i / G <= x
        const int last = (int)(((task + np) * G - 1) / T0);
        ws.slots[slot] = {cur.b, j, last - me + 1, 2};
      }
      B::segment(a, smem, cur.b, j, p0, p1, part ? ws.data + slot * attn_slot_floats(D) : nullptr);
      first = false;
      u += p1 - p0;
    }
  }
}

constexpr int kMergeThreads = 256;
constexpr int kMaxSlots = 1024;

// Merges the parts of split tasks.  Every block lists the first slots, then
// takes (task, head) pairs in turn: 8 parts at a time, a warp each.
template <int D, class T>
__global__ void __launch_bounds__(kMergeThreads) kvq_merge_kernel(AttnArgs a, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32;                // dims of a lane
  __shared__ int list[kMaxSlots], counts[8];
  __shared__ float so[8][D], sr[8], sl[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnWs ws = attn_ws(a.ws, blocks);
  const int count = *ws.count;
  int n = 0;
  for (int s0 = 0; s0 < count; s0 += kMergeThreads) {
    const int s = s0 + tid;
    const bool is = s < count && ws.slots[s].parts > 0;
    const unsigned m = __ballot_sync(0xffffffffu, is);
    if (lane == 0) counts[warp] = __popc(m);
    __syncthreads();
    int at = n;
    for (int w = 0; w < 8; w++) {
      if (w < warp) at += counts[w];
      n += counts[w];
    }
    if (is) list[at + __popc(m & ((1u << lane) - 1))] = s;
    __syncthreads();
  }
  for (int w = blockIdx.x; w < n * 8; w += gridDim.x) {
    const int s = list[w / 8], h = w % 8;
    const AttnSlot t = ws.slots[s];
    if (h >= min(8, a.grp - t.j % a.tiles * 8)) continue;
    float m = -FLT_MAX, den = 0.f, num[V];
#pragma unroll
    for (int k = 0; k < V; k++) num[k] = 0.f;
    for (int i = warp; i < t.parts; i += 8) {
      const int slot = i == 0 ? s : t.step == 1 ? s + i : (s & ~1) + 2 * i;
      const float* p = ws.data + slot * attn_slot_floats(D);
      const float r = p[8 * D + h], l = p[8 * D + 8 + h];
      float o[V];
#pragma unroll
      for (int k = 0; k < V; k++) o[k] = p[h * D + lane + 32 * k];
      const float mn = fmaxf(m, r), ka = ex2(m - mn), kb = ex2(r - mn);
      den = den * ka + l * kb;
#pragma unroll
      for (int k = 0; k < V; k++) num[k] = num[k] * ka + o[k] * kb;
      m = mn;
    }
#pragma unroll
    for (int k = 0; k < V; k++) so[warp][lane + 32 * k] = num[k];
    if (lane == 0) sr[warp] = m, sl[warp] = den;
    __syncthreads();
    if (tid < D) {
      float M = -FLT_MAX, sn = 0.f, sd = 0.f;
      for (int i = 0; i < 8; i++) M = fmaxf(M, sr[i]);
      for (int i = 0; i < 8; i++) {
        const float k = ex2(sr[i] - M);
        sn = fmaf(k, so[i][tid], sn);
        sd = fmaf(k, sl[i], sd);
      }
      stf(out_row<D, T>(a, t.b, t.j, h) + tid, sn / sd);
    }
    __syncthreads();
  }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_cache(const mk_kvq_cache* c) {
  if (!c) return MK_ERR_BAD_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->num_pages < 1 ||
      c->num_pages > 0x7fffffff / kKvqPage)
    return MK_ERR_BAD_CONFIG;
  if (!c->pool || !aligned(c->pool, 16) || !aligned(c->status, 4)) return MK_ERR_BAD_ARG;
  return MK_OK;
}

int check_rows(const mk_kv_rows* r, const mk_kvq_cache* c, int n, int unit, const int32_t* view_index,
               const int32_t* cache_index) {
  if (!r || (unit != 1 && unit != kKvqPage) || n < 0 || n > 0x7fffffff / unit) return MK_ERR_BAD_ARG;
  if (r->type != MK_TYPE_BF16 && r->type != MK_TYPE_F32) return MK_ERR_BAD_ARG;
  if (n == 0) return MK_OK;
  if (!r->k || !r->v || !aligned(r->k, 16) || !aligned(r->v, 16) || r->count < 0 ||
      (long long)r->count * unit > 0x7fffffffll)
    return MK_ERR_BAD_ARG;
  const long long q = r->type == MK_TYPE_BF16 ? 8 : 4;   // 16-byte loads
  if (r->page_stride % q || r->row_stride % q || r->head_stride % q) return MK_ERR_BAD_ARG;
  if (!view_index && n > r->count) return MK_ERR_BAD_ARG;
  if (!cache_index && (long long)n * unit > (long long)c->num_pages * kKvqPage) return MK_ERR_BAD_PAGE;
  return MK_OK;
}

Cache cache_of(const mk_kvq_cache* c) { return Cache{(uint8_t*)c->pool, c->status, c->num_pages, c->n_kv_heads}; }

Rows rows_of(const mk_kv_rows* r, int unit) {
  // a row index counts tokens with unit 1: page and row strides then agree
  return Rows{r->k, r->v, unit == 1 ? r->row_stride * kKvqPage : r->page_stride, r->row_stride, r->head_stride,
              r->count};
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

int check_heads(const mk_kvq_cache* c, int n_q_heads, int batch) {
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads > 65536) return MK_ERR_BAD_CONFIG;
  return batch < 0 || batch > 65535 ? MK_ERR_BATCH_TOO_LARGE : MK_OK;
}

// blocks that fill the GPU, two slots each
int attn_blocks(int sms, int per_sm) { return std::min(sms * per_sm, kMaxSlots / 2); }

template <int D, class T>
int attention(const AttnArgs& a, int sms, cudaStream_t st) {
  // the kernel's shared memory is raised once on each device
  static std::atomic<unsigned long long> raised[2];
  constexpr size_t smem = AttnBlock<D, T>::kSmem;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return MK_ERR_CUDA;
  if (!(raised[dev / 64].load(std::memory_order_relaxed) >> (dev % 64) & 1)) {
    if (cudaFuncSetAttribute(kvq_attention_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    raised[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_relaxed);
  }
  // no more blocks than there can be segments, unless some rows are empty
  const long long tasks = (long long)a.batch * a.c.hkv * a.tiles;
  const long long most = tasks * std::max(1, (a.max_pages + kMinPages - 1) / kMinPages);
  const int blocks = (int)std::min<long long>(attn_blocks(sms, kBlocksPerSm<D, T>), most);
  kvq_attention_kernel<D, T><<<blocks, kAttnThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return MK_ERR_CUDA;
  if (!a.split) return MK_OK;
  // the merge is launched while the first kernel runs and waits for its end
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)std::min<long long>(sms, tasks * 8));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kvq_merge_kernel<D, T>, a, blocks) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA; }

}  // namespace

extern "C" {

size_t mk_kvq_page_bytes(int n_kv_heads, int head_dim) {
  if (n_kv_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)n_kv_heads * 18 * head_dim;
}

int mk_kvq_write(const mk_kvq_cache* c, const mk_kv_rows* src, const int32_t* src_index, const int32_t* dst_index,
                 int n, int unit, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_rows(src, c, n, unit, src_index, dst_index);
  if (rc || n == 0) return rc;
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  const int tokens = n * unit;
  const long long threads = (long long)tokens * c->n_kv_heads * (c->head_dim / 4);
  const int blocks = (int)std::min<long long>((threads + 255) / 256, sms * 8ll);
  const Cache cc = cache_of(c);
  const Rows rr = rows_of(src, unit);
  cudaStream_t st = (cudaStream_t)stream;
  if (c->head_dim == 128)
    src->type == MK_TYPE_BF16
        ? kvq_write_kernel<128, uint16_t><<<blocks, 256, 0, st>>>(cc, rr, src_index, dst_index, tokens, unit)
        : kvq_write_kernel<128, float><<<blocks, 256, 0, st>>>(cc, rr, src_index, dst_index, tokens, unit);
  else
    src->type == MK_TYPE_BF16
        ? kvq_write_kernel<64, uint16_t><<<blocks, 256, 0, st>>>(cc, rr, src_index, dst_index, tokens, unit)
        : kvq_write_kernel<64, float><<<blocks, 256, 0, st>>>(cc, rr, src_index, dst_index, tokens, unit);
  return launched();
}

int mk_kvq_read(const mk_kvq_cache* c, const int32_t* src_index, const mk_kv_rows* dst, const int32_t* dst_index,
                int n, int unit, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_rows(dst, c, n, unit, dst_index, src_index);
  if (rc || n == 0) return rc;
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  const int tokens = n * unit;
  const long long threads = (long long)tokens * c->n_kv_heads * (c->head_dim / 4);
  const int blocks = (int)std::min<long long>((threads + 255) / 256, sms * 8ll);
  const Cache cc = cache_of(c);
  const Rows rr = rows_of(dst, unit);
  cudaStream_t st = (cudaStream_t)stream;
  if (c->head_dim == 128)
    dst->type == MK_TYPE_BF16
        ? kvq_read_kernel<128, uint16_t><<<blocks, 256, 0, st>>>(cc, src_index, rr, dst_index, tokens, unit)
        : kvq_read_kernel<128, float><<<blocks, 256, 0, st>>>(cc, src_index, rr, dst_index, tokens, unit);
  else
    dst->type == MK_TYPE_BF16
        ? kvq_read_kernel<64, uint16_t><<<blocks, 256, 0, st>>>(cc, src_index, rr, dst_index, tokens, unit)
        : kvq_read_kernel<64, float><<<blocks, 256, 0, st>>>(cc, src_index, rr, dst_index, tokens, unit);
  return launched();
}

size_t mk_kvq_workspace(const mk_kvq_cache* c, int n_q_heads, int batch) {
  if (check_cache(c) || check_heads(c, n_q_heads, batch)) return 0;
  const int sms = sm_count();
  return sms ? attn_ws_bytes(attn_blocks(sms, 2), c->head_dim) : 0;
}

int mk_kvq_attention(const mk_kvq_cache* c, const void* q, int64_t q_stride, void* out, int64_t out_stride, int type,
                     int n_q_heads, int batch, const int32_t* page_tables, int max_pages, const int32_t* seq_lens,
                     float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_heads(c, n_q_heads, batch);
  if (rc) return rc;
  if (type != MK_TYPE_BF16 && type != MK_TYPE_F32) return MK_ERR_BAD_ARG;
  if (max_pages < 0 || max_pages > 0x7fffffff / kKvqPage || !isfinite(scale)) return MK_ERR_BAD_ARG;
  if (batch == 0) return MK_OK;
  const int64_t v = type == MK_TYPE_BF16 ? 8 : 4;
  if (!q || !out || !seq_lens || (max_pages && !page_tables) || !aligned(q, 16) || !aligned(out, 16) ||
      q_stride % v || out_stride % v || (batch > 1 && out_stride < (int64_t)n_q_heads * c->head_dim))
    return MK_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  AttnArgs a{};
  a.c = cache_of(c);
  a.q = q;
  a.out = out;
  a.page_tables = page_tables;
  a.seq_lens = seq_lens;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.grp = n_q_heads / c->n_kv_heads;
  a.tiles = (a.grp + 7) / 8;
  a.batch = batch;
  a.max_pages = max_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.split = max_pages > kMinPages;
  if (a.split) {
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < attn_ws_bytes(attn_blocks(sms, 2), c->head_dim))
      return MK_ERR_BAD_ARG;
    a.ws = (uint8_t*)workspace;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (c->head_dim == 128)
    return type == MK_TYPE_BF16 ? attention<128, uint16_t>(a, sms, st) : attention<128, float>(a, sms, st);
  return type == MK_TYPE_BF16 ? attention<64, uint16_t>(a, sms, st) : attention<64, float>(a, sms, st);
}

}  // extern "C"

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

// ------------------------------------------------------------ write and read
//
// Each moves 2 (or 4) bytes and 9/16 of a byte a value.  Tokens come in any
// order, so a token's row is eight values a thread and the eight threads of a
// scale group side by side.  Whole pages (unit 16) are read a page and head a
// warp and written a page's keys or values a warp, head after head: codes of
// both tokens of a pair meet in one lane, every record is moved in 16-byte
// pieces, and a writer loads the next head's half page while it computes the
// other half.  262,144 tokens of 4 heads of 128 dims in BF16, 688 MB: read 104 us
// (98 % of the measured copy rate), written 125 us (81 %; issue slots 69 %, DRAM
// 66 % of its peak: 24 warps an SM do not hide every wait).
// Measured of the writer: both halves of keys and values held by one warp
// without the overlap 151 (16 warps an SM) and 136 us (32, registers spill),
// keys or values a warp without it 133, half a page a warp 149; 64 registers
// with the overlap 126, 48 148.  8191 tokens by row: 7 us written, 6 read (12.3 and
// 8.2 with a cold cache, for 3.2 us of bytes each), bound by latency: a thread's
// index, address and row are one chain of loads with nothing of another token in
// flight (issue slots 32 %, ALU 41-49 %, DRAM 7-17 %).

// eight consecutive elements as they lie in memory, moved 16 bytes at a time;
// load() is for memory that nothing writes while the kernel runs
template <class T>
struct Raw8 {
  static constexpr int W = 2 * (int)sizeof(T);
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 t = __ldg((const uint4*)p + i / 4);
      w[i] = t.x, w[i + 1] = t.y, w[i + 2] = t.z, w[i + 3] = t.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < W; i += 4) *((uint4*)p + i / 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
  __device__ __forceinline__ void get(float* x) const {
#pragma unroll
    for (int i = 0; i < W; i++)
      if constexpr (sizeof(T) == 2) {
        x[2 * i] = bf16lo(w[i]);
        x[2 * i + 1] = bf16hi(w[i]);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
  }
  __device__ __forceinline__ void set(const float* x) {
#pragma unroll
    for (int i = 0; i < W; i++)
      if constexpr (sizeof(T) == 2)
        w[i] = pack_bf2(x[2 * i], x[2 * i + 1]);
      else
        w[i] = __float_as_uint(x[i]);
  }
};

// scale of the group of which a thread holds `raw`, as fp32 x
__device__ __forceinline__ KvqScale row_scale(const Raw8<uint16_t>& raw, const float*, unsigned mask) {
  return kvq_group_scale(raw.w, mask);
}
__device__ __forceinline__ KvqScale row_scale(const Raw8<float>&, const float* x, unsigned mask) {
  return kvq_group_scale(x, mask);
}

// eight elements of the query, by ordinary loads: out may be q, so the memory
// is not read-only while the kernel runs
template <class T>
__device__ __forceinline__ void load8(float* x, const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < Raw8<T>::W; i += 4) {
    const uint4 t = *((const uint4*)p + i / 4);
    r.w[i] = t.x, r.w[i + 1] = t.y, r.w[i + 2] = t.z, r.w[i + 3] = t.w;
  }
  r.get(x);
}

// values of the eight codes of a word: step * code + low in fp32.  A nibble
// under the exponent of 2^23 is 2^23 + code; both operations that follow are
// exact up to the last.
__device__ __forceinline__ void kvq_values(float* x, uint32_t word, uint32_t scale) {
  const float step = bf16lo(scale), low = bf16hi(scale);
#pragma unroll
  for (int i = 0; i < 8; i++)
    x[i] = fmaf(__uint_as_float((word >> (4 * i) & 15u) | 0x4b000000u) - 8388608.f, step, low);
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 t = __ldcs((const uint4*)p);
    w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
  } else if constexpr (N == 2) {
    const uint2 t = __ldcs((const uint2*)p);
    w[0] = t.x, w[1] = t.y;
  } else {
    w[0] = __ldcs((const uint32_t*)p);
  }
}
template <int N>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t* w) {
  if constexpr (N == 4)
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 2)
    *(uint2*)p = make_uint2(w[0], w[1]);
  else
    *(uint32_t*)p = w[0];
}

// a unit of the call: its indexes on the two sides, false if it is skipped
__device__ __forceinline__ bool unit_pair(const Cache& c, const int32_t* src_index, int src_count,
                                          const int32_t* dst_index, int dst_count, int i, int& from, int& to) {
  from = src_index ? src_index[i] : i;
  to = dst_index ? dst_index[i] : i;
  if (to < 0) return false;
  if (from >= src_count || to >= dst_count) {
    flag_bad(c, MK_ERR_BAD_PAGE);
    return false;
  }
  return true;
}

constexpr int kCopyThreads = 256;

// The thread's eight dims of a token call: block (x, y) takes kTokens tokens
// and `heads` KV heads from y heads on, eight threads a (token, key or value,
// group); one head a block where there are few tokens, several where the
// indexes and addresses would cost more than the row.  The call's tokens 2 k
// and 2 k + 1 are kPartner lanes apart in a warp: where they lie side by side
// in the cache (a prompt's do), their value codes, 16 bits of a word each, are
// exchanged and moved as whole words.
template <int D>
struct TokenLane {
  static constexpr int NG = D / kKvqGroup, kPartner = 8 * NG;
  static constexpr int kTokens = kCopyThreads / 8 / (2 * NG);
  int wi, group, val, odd, i;
  __device__ __forceinline__ TokenLane() {
    const int o = threadIdx.x >> 3;
    wi = threadIdx.x & 7;
    group = o % NG;
    odd = o / NG & 1;
    val = o / (2 * NG) & 1;
    i = blockIdx.x * kTokens + o / (4 * NG) * 2 + odd;
  }
  // this thread's slot and its partner's are the two halves of a pair
  __device__ __forceinline__ bool paired(int slot) const {
    const int other = __shfl_xor_sync(0xffffffffu, slot, kPartner);
    return val && slot >= 0 && other == (slot ^ 1) && (slot & 1) == odd;
  }
};

template <int D, class T>
__global__ void __launch_bounds__(kCopyThreads) kvq_write_kernel(Cache c, Rows src, const int32_t* src_index,
                                                                 const int32_t* dst_index, int n, int heads) {
  using R = KvqRec<D>;
  const TokenLane<D> o;
  const int h0 = blockIdx.y * heads, h1 = min(c.hkv, h0 + heads);
  int from = -1, to = -1;
  const bool live = o.i < n &&
                    unit_pair(c, src_index, src.count, dst_index, c.pages * kKvqPage, o.i, from, to) && from >= 0;
  if (!live) from = 0, to = -1;
  const bool pair = o.paired(to);
  const int t = max(to, 0) % kKvqPage;
  const T* row = (const T*)(o.val ? src.v : src.k) + from * src.row + h0 * src.head + o.group * kKvqGroup + o.wi * 8;
  uint8_t* rec = c.pool + ((long long)(max(to, 0) / kKvqPage) * c.hkv + h0) * R::kBytes;
#pragma unroll 2
  for (int h = h0; h < h1; h++, row += src.head, rec += R::kBytes) {
    Raw8<T> raw = {};
    if (live) raw.load(row);
    float x[8];
    raw.get(x);
    const KvqScale s = row_scale(raw, x, 0xffffffffu);
    const uint32_t word = kvq_codes(x, s);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, TokenLane<D>::kPartner);
    if (pair) {
      *(uint32_t*)(rec + R::val_half(t & ~1, o.wi, o.group, o.odd)) =
          o.odd ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
      if (o.wi == 0) *(uint32_t*)(rec + R::kValScale + 4 * (t * R::NG + o.group)) = s.word();
    } else if (live) {
      kvq_store_row<D>(rec, t, o.wi, o.group, o.val, word, s);
    }
  }
}

template <int D, class T>
__global__ void __launch_bounds__(kCopyThreads) kvq_read_kernel(Cache c, const int32_t* src_index, Rows dst,
                                                                const int32_t* dst_index, int n, int heads) {
  using R = KvqRec<D>;
  const TokenLane<D> o;
  const int h0 = blockIdx.y * heads, h1 = min(c.hkv, h0 + heads);
  int from = -1, to = -1;
  const bool live =
      o.i < n && unit_pair(c, src_index, c.pages * kKvqPage, dst_index, dst.count, o.i, from, to);
  if (!live) from = -1, to = 0;
  const bool pair = o.paired(from);
  const int t = max(from, 0) % kKvqPage;
  const uint8_t* rec = c.pool + ((long long)(max(from, 0) / kKvqPage) * c.hkv + h0) * R::kBytes;
  T* row = (T*)(o.val ? dst.v : dst.k) + to * dst.row + h0 * dst.head + o.group * kKvqGroup + o.wi * 8;
#pragma unroll 2
  for (int h = h0; h < h1; h++, row += dst.head, rec += R::kBytes) {
    uint32_t word = 0, scale = 0;          // no source: zeros
    if (from >= 0) {
      if (pair)
        word = *(const uint32_t*)(rec + R::val_half(t & ~1, o.wi, o.group, o.odd));
      else if (o.val)
        word = *(const uint16_t*)(rec + R::val_half(t, o.wi, o.group, 0)) |
               ((uint32_t)*(const uint16_t*)(rec + R::val_half(t, o.wi, o.group, 1)) << 16);
      else
        word = *(const uint32_t*)(rec + R::key_word(t, o.wi, o.group));
      scale = *(const uint32_t*)(rec + (o.val ? R::kValScale : R::kKeyScale) + 4 * (t * R::NG + o.group));
    }
    const uint32_t other = __shfl_xor_sync(0xffffffffu, word, TokenLane<D>::kPartner);
    if (pair) word = o.odd ? __byte_perm(other, word, 0x7632) : __byte_perm(word, other, 0x5410);
    float x[8];
    kvq_values(x, word, scale);
    Raw8<T> raw;
    raw.set(x);
    if (live) raw.store(row);
  }
}

template <int D, class T>
__global__ void __launch_bounds__(kCopyThreads, sizeof(T) == 2 ? 3 : 2)
    kvq_write_pages_kernel(Cache c, Rows src, const int32_t* src_index, const int32_t* dst_index, int n, int heads) {
  using R = KvqRec<D>;
  constexpr int NG = R::NG;
  const int lane = threadIdx.x & 31, val = threadIdx.x >> 5 & 1;
  const int i = blockIdx.x * (kCopyThreads / 64) + (threadIdx.x >> 6);
  const int h0 = blockIdx.y * heads, h1 = min(c.hkv, h0 + heads);
  int from, to;
  if (i >= n || !unit_pair(c, src_index, src.count, dst_index, c.pages, i, from, to) || from < 0) return;
  const int pr = lane >> 3, wi = lane & 7;
  // raw[e]: keys of tokens 8 e + pr and 8 e + pr + 4, or values of tokens 8 e + 2 pr and the next; dims 64 g + 8 wi ..
  const int t0 = val ? 2 * pr : pr, dt = val ? 1 : 4;
  const T* p = (const T*)(val ? src.v : src.k) + from * src.page + h0 * src.head + t0 * src.row + wi * 8;
  uint8_t* rec = c.pool + ((long long)to * c.hkv + h0) * R::kBytes;
  Raw8<T> raw[2][2][NG];
  auto load = [&](int e) {
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int g = 0; g < NG; g++) raw[e][t][g].load(p + (8 * e + t * dt) * src.row + g * kKvqGroup);
  };
  load(0);
  load(1);
#pragma unroll 1
  for (int h = h0; h < h1; h++, rec += R::kBytes) {
    p += src.head;
#pragma unroll
    for (int e = 0; e < 2; e++) {
      uint32_t w[2][NG], sw[2][NG];
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int g = 0; g < NG; g++) {
          float x[8];
          raw[e][t][g].get(x);
          const KvqScale s = row_scale(raw[e][t][g], x, 0xffffffffu);
          w[t][g] = kvq_codes(x, s);
          sw[t][g] = s.word();
        }
      if (h + 1 < h1) load(e);               // the next head's, while this one's other half is computed
      if (val) {
        const int pair = pr + 4 * e;
        uint32_t vw[2 * NG];
#pragma unroll
        for (int g = 0; g < NG; g++) {
          vw[2 * g] = __byte_perm(w[0][g], w[1][g], 0x5410);
          vw[2 * g + 1] = __byte_perm(w[0][g], w[1][g], 0x7632);
        }
        store_words<2 * NG>(rec + R::kVal + pair * D + wi * 8 * NG, vw);
        if (wi == 0) store_words<2 * NG>(rec + R::kValScale + pair * 8 * NG, sw[0]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const int t = pr + 8 * e + 4 * k;
          if constexpr (NG == 2) {
            // a column's 16 bytes are both words of group 0, then of group 1: two threads hold one of each
            const uint32_t got = __shfl_xor_sync(0xffffffffu, wi & 1 ? w[k][0] : w[k][1], 1);
            if (wi & 1)
              w[k][0] = got;
            else
              w[k][1] = got;
          }
          store_words<NG>(rec + t * (D / 2) + wi * 4 * NG, w[k]);
          if (wi == 0) store_words<NG>(rec + R::kKeyScale + t * 4 * NG, sw[k]);
        }
      }
    }
  }
}

template <int D, class T>
__global__ void __launch_bounds__(kCopyThreads) kvq_read_pages_kernel(Cache c, const int32_t* src_index, Rows dst,
                                                                      const int32_t* dst_index, int n) {
  using R = KvqRec<D>;
  constexpr int NG = R::NG;
  const int lane = threadIdx.x & 31, head = blockIdx.y;
  const int i = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  int from, to;
  if (i >= n || !unit_pair(c, src_index, c.pages, dst_index, dst.count, i, from, to)) return;
  T* kb = (T*)dst.k + to * dst.page + head * dst.head;
  T* vb = (T*)dst.v + to * dst.page + head * dst.head;
  const int pr = lane >> 3, wi = lane & 7;
  uint32_t kw[4][NG] = {}, ks[4][NG] = {}, vw[2][2 * NG] = {}, vs[2][2 * NG] = {};   // no source: zeros
  if (from >= 0) {
    const uint8_t* rec = c.pool + ((long long)from * c.hkv + head) * R::kBytes;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      load_words<NG>(kw[e], rec + (pr + 4 * e) * (D / 2) + wi * 4 * NG);
      load_words<NG>(ks[e], rec + R::kKeyScale + (pr + 4 * e) * 4 * NG);
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
      load_words<2 * NG>(vw[e], rec + R::kVal + (pr + 4 * e) * D + wi * 8 * NG);
      load_words<2 * NG>(vs[e], rec + R::kValScale + (pr + 4 * e) * 8 * NG);
    }
  }
  float x[8];
  Raw8<T> raw;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if constexpr (NG == 2) {               // as in the write, the other way round
      const uint32_t got = __shfl_xor_sync(0xffffffffu, wi & 1 ? kw[e][0] : kw[e][1], 1);
      if (wi & 1)
        kw[e][0] = got;
      else
        kw[e][1] = got;
    }
#pragma unroll
    for (int g = 0; g < NG; g++) {
      kvq_values(x, kw[e][g], ks[e][g]);
      raw.set(x);
      raw.store(kb + (pr + 4 * e) * dst.row + g * kKvqGroup + wi * 8);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; e++)
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
      for (int g = 0; g < NG; g++) {
        kvq_values(x, __byte_perm(vw[e][2 * g], vw[e][2 * g + 1], t ? 0x7632 : 0x5410), vs[e][t * NG + g]);
        raw.set(x);
        raw.store(vb + (2 * (pr + 4 * e) + t) * dst.row + g * kKvqGroup + wi * 8);
      }
}

// ---------------------------------------------------------------- attention
//
// The pages of all tasks (sequence, KV head, 8 of its query heads) are cut
// into segments by the blocks themselves from the lengths on the device, so
// the host neither reads lengths nor launches for the longest one:
//   few pages (no more than a segment a block): segments of kMinPages pages,
//     one page a warp;
//   many: block i takes units T i / G .. T (i + 1) / G of the T units of all
//     tasks in order, so that every block has the same work whatever the mix of
//     lengths.  A unit is a page; a task's last segment counts as a whole one,
//     and a task kTaskCost units more, for what a block spends on a segment
//     beside its pages.  48 against 0, 24 and 96, 16 sequences of 1K-32K: 45.0 us
//     against 50.3, 46.4, 46.1 (4 KV heads of 128 dims); 76.2 against 86.1, 77.5,
//     77.1 (8 heads); 20.0 against 21.7, 20.2, 20.3 (1 head); 28.5 against 31.5,
//     29.3, 29.6 (64 dims); fp32 54.1 against 69.3, 61.8, 55.9 (64 dims 34.9
//     against 37.9, 35.4, 36.3); 64 of up to 9000: 46.5 against 63.0, 48.0, 51.0;
//     one of 256K: 42.0 against 40.7, 40.9, 41.9.
// A task that is one segment is written at once.  The segments of the others
// leave (reference, sum, weighted sum) in workspace slots, at most two a block,
// and a second kernel merges them in page order: no atomics, one result.
// A warp takes every eighth page of a segment through a ring of four in shared
// memory (three on their way: 110 KB an SM, twice what the latency needs).
// 32 query and 4 KV heads of 128 dims, BF16: 262,144 tokens in 42 us, 39 of them
// in the first kernel, against 22 us for its 151 MB at the measured copy rate
// (fp32: 50 us, one block an SM; 64 dims: 25 us BF16, 32 fp32, for 75 MB);
// 16 sequences of 1K-32K in 45 us (152 MB), fp32 54.  About 350 instructions a page
// and head (4096 codes).  Counted in the source: 40 to mask key codes, 72 to mask
// and centre value codes, 50 for scales, 40 for weights and references, 25 to
// fetch; the rest are 16 matrix products, 4 transposes, 8 shared loads,
// exponentials, packing, the vote and the loop.  Issue slots
// 50-58 %, ALU pipe 52 %, DRAM 49 %, tensor pipe 20 %: what bounds it is a page's
// chain (loads, products, vote, products) with 16 warps an SM.  Slower or no
// faster: two pages a warp at a time (49 us, registers spill), the next page's
// scores ahead of this one's values (42 us, spills too), 18 warps an SM at 96
// registers (60 us), shifts as multiplications (43 us), a ring of five (45 us).

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = kAttnWarps * 32;
// resident blocks: the fp32 kernel with 128 dims needs more than the 128
// registers a thread that two blocks leave
constexpr int attn_per_sm(int d, int type) { return d == 128 && type == MK_TYPE_F32 ? 1 : 2; }
template <int D, class T>
constexpr int kBlocksPerSm = attn_per_sm(D, sizeof(T) == 4 ? MK_TYPE_F32 : MK_TYPE_BF16);
constexpr int kMinPages = kAttnWarps;
constexpr int kTaskCost = 48;
constexpr int kRing = 4;                   // pages of a warp, in flight and in use

struct AttnArgs {
  Cache c;
  const void* q;
  void* out;
  const int32_t* page_tables;
  const int32_t* seq_lens;
  uint8_t* ws;                             // AttnWs
  long long q_stride, out_stride;          // elements between two sequences
  int grp, tiles, batch, max_pages;        // tiles = ceil(grp / 8)
  float scale_log2;
};

// workspace: the slot count, a header per slot, then the slots
struct __align__(16) AttnSlot {
  int b, j;                                // sequence; KV head and head tile
  int parts;                               // of the task, in its first slot; 0 in the others
  int step;                                // 1: parts in consecutive slots; 2: in the even slots after the first
};

struct AttnWs {
  int32_t* count;
  AttnSlot* slots;
  float* data;
};

__host__ __device__ constexpr size_t attn_slot_floats(int d) { return 8 * (size_t)d + 16; }

__host__ __device__ constexpr size_t attn_ws_bytes(int blocks, int d) {
  const size_t slots = 2 * (size_t)blocks;
  return 16 + slots * sizeof(AttnSlot) + slots * attn_slot_floats(d) * 4;
}

__device__ __forceinline__ AttnWs attn_ws(uint8_t* p, int blocks) {
  return {(int32_t*)p, (AttnSlot*)(p + 16), (float*)(p + 16 + 2 * (size_t)blocks * sizeof(AttnSlot))};
}

__device__ __forceinline__ void stf(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }

// 16 bytes, of which `bytes` (16 or 0) are read and the rest are zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// A place in the list of sequences: the pages of sequence b and what comes
// before it, in units of one task each and in chunks of split tasks
struct Place {
  int b, np;
  long long units, split;
};

// What comes before a sequence: units (kMinPages for each started kMinPages
// pages), chunks of split tasks, sequences with a page
struct Before {
  long long units, split;
  int tasks;
};

struct PlanSmem {
  long long units[kAttnWarps], marks[kAttnWarps];
  Place found;
  // the window: a sequence a thread
  int np[kAttnThreads];
  Before before[kAttnThreads];
  int b0;
  Before end;                              // before the next window
};

__device__ __forceinline__ int seq_units(int np) { return (np + kMinPages - 1) / kMinPages * kMinPages; }

// Sums over the sequences, a window of one sequence a thread at a time (in
// shared memory: between segments nothing stays in registers).  All threads
// of the block make every call together.
__device__ void plan_window(const AttnArgs& a, PlanSmem& S, int first, Before end) {
  constexpr int kTaskBits = 20;            // chunks and sequences are added up in one word
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int np = first + tid < a.batch ? max(seq_pages(a, first + tid), 0) : 0;
  const long long n = seq_units(np);
  const long long m = ((long long)(np > kMinPages ? n / kMinPages : 0) << kTaskBits) + (np > 0);
  long long u = n, k = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, k, o);
    if (lane >= o) u += x, k += y;
  }
  if (lane == 31) S.units[warp] = u, S.marks[warp] = k;
  __syncthreads();
  long long units = u - n, marks = k - m, all_units = 0, all_marks = 0;
  for (int w = 0; w < kAttnWarps; w++) {
    if (w < warp) units += S.units[w], marks += S.marks[w];
    all_units += S.units[w];
    all_marks += S.marks[w];
  }
  constexpr long long kMask = (1 << kTaskBits) - 1;
  S.np[tid] = np;
  S.before[tid] = {end.units + units, end.split + (marks >> kTaskBits), end.tasks + (int)(marks & kMask)};
  if (tid == 0) {
    S.b0 = first;
    S.end = {end.units + all_units, end.split + (all_marks >> kTaskBits), end.tasks + (int)(all_marks & kMask)};
  }
  __syncthreads();
}

// the next window, false after the last
__device__ bool plan_next(const AttnArgs& a, PlanSmem& S) {
  const int first = S.b0 + kAttnThreads;
  const Before end = S.end;
  __syncthreads();
  if (first >= a.batch) return false;
  plan_window(a, S, first, end);
  return true;
}

// the sequence that holds unit `target`, not before the window, where each
// sequence has `cost` units more; false past the last
__device__ bool plan_find(const AttnArgs& a, PlanSmem& S, int cost, long long target, Place& at) {
  while (target >= S.end.units + (long long)cost * S.end.tasks)
    if (!plan_next(a, S)) return false;
  const int tid = threadIdx.x, np = S.np[tid];
  const Before b = S.before[tid];
  const long long units = b.units + (long long)cost * b.tasks;
  if (np > 0 && units <= target && target < units + seq_units(np) + cost) S.found = {S.b0 + tid, np, units, b.split};
  __syncthreads();
  at = S.found;
  __syncthreads();                         // the next call writes it again
  return true;
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
  static constexpr int kChunks = (R::kBytes / 16 + 31) / 32;
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
    int fetched = 0, id = n > 0 ? table[0] : 0;   // the next page to fetch, read an iteration ahead
    const int last = max(n - 1, 0) * kAttnWarps;
    const uint8_t* base = a.c.pool + (long long)g * R::kBytes + lane * 16;
    const long long page_bytes = (long long)a.c.hkv * R::kBytes;
    // the lane's 16-byte chunks lie 512 bytes apart, in the ring slot too: value chunks from one place (32 of
    // them are whole fours of token pairs), the others from another
    constexpr int kVal0 = R::kVal / 512, kVal1 = R::kKeyScale / 512;
    const uint32_t line = smem_u32(ring) + lane * 16;
    const uint32_t line_v = smem_u32(ring) + A::staged(R::kVal / 16 + lane) * 16 - R::kVal;
    // the warp's next page into the ring, `slot` bytes in; without branches: past the warp's last page nothing is read
    auto fetch = [&](uint32_t slot) {
      const bool live = fetched < n, ok = (unsigned)id < (unsigned)a.c.pages;
      bad |= live && !ok;
      const uint8_t* src = base + (ok ? id : 0) * page_bytes;
      const int bytes = live ? 16 : 0;
#pragma unroll
      for (int k = 0; k < kChunks; k++)
        if (k * 32 + 32 <= R::kBytes / 16 || k * 32 + lane < R::kBytes / 16)
          cp_async16((k >= kVal0 && k < kVal1 ? line_v : line) + slot + k * 512, src + k * 512, bytes);
      fetched++;
      if (n > 0) id = table[min(fetched * kAttnWarps, last)];
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; i++) fetch(i * R::kBytes);

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
    uint32_t rd = 0, wr = (kRing - 1) * R::kBytes;
    auto next = [&]() {                    // the next page has arrived; another goes into the slot read before it
      cp_async_wait<kRing - 2>();
      __syncwarp();
      fetch(wr);
      wr = wr == (kRing - 1) * R::kBytes ? 0 : wr + R::kBytes;
      const uint8_t* rec = ring + rd;
      rd = rd == (kRing - 1) * R::kBytes ? 0 : rd + R::kBytes;
      return rec;
    };
    // only the sequence's last page can have rows past its end
    const int tail = len - (p0 + warp + (n - 1) * kAttnWarps) * kKvqPage;
    const int full = tail >= kKvqPage ? n : n - 1;
    for (int i = 0; i < full; i++) {
      const uint8_t* const rec[1] = {next()};
      at.template pages<1, true, false>(rec, {kKvqPage}, lane);
    }
    if (n > 0 && full < n) {
      const uint8_t* const rec[1] = {next()};
      at.template pages<1, true, true>(rec, {tail}, lane);
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
  // the merge may be set up as soon as there is room for it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int b = me; b < a.batch; b += G) {
    const int np = seq_pages(a, b);
    if (np > 0) continue;                  // rows of sequences without a page
    if (np < 0 && tid == 0) flag_bad(a.c, MK_ERR_BAD_ARG);
    for (int i = tid; i < a.c.hkv * a.grp * D; i += kAttnThreads)
      stf((T*)a.out + b * a.out_stride + i, np < 0 ? NAN : 0.f);
  }
  const AttnWs ws = attn_ws(a.ws, G);
  Place at;
  plan_window(a, S, 0, Before{0, 0, 0});
  while (plan_next(a, S)) {}
  const Before all = S.end;
  if (a.batch > kAttnThreads) {            // the plan is at its end
    __syncthreads();
    plan_window(a, S, 0, Before{0, 0, 0});
  }
  if ((unsigned long long)all.units * HT <= (unsigned long long)G * kMinPages) {
    if (me == 0 && tid == 0) *ws.count = (int)(all.split * HT);
    // segment s is the s-th chunk of kMinPages pages
    for (long long s = me; plan_find(a, S, 0, s / HT * kMinPages, at); s += G) {
      const int nc = seq_units(at.np) / kMinPages;
      const long long rem = s - at.units / kMinPages * HT;
      const int j = (int)(rem / nc), k = (int)(rem % nc);
      const int slot = (int)(at.split * HT + rem);
      if (nc > 1 && tid == 0) ws.slots[slot] = {at.b, j, k == 0 ? nc : 0, 1};
      B::segment(a, smem, at.b, j, k * kMinPages, min(at.np, (k + 1) * kMinPages),
                 nc > 1 ? ws.data + slot * attn_slot_floats(D) : nullptr);
    }
  } else {
    if (me == 0 && tid == 0) *ws.count = 2 * G;
    if (tid == 0) ws.slots[2 * me].parts = ws.slots[2 * me + 1].parts = 0;
    const unsigned long long total = (unsigned long long)(all.units + (long long)kTaskCost * all.tasks) * HT;
    unsigned long long u = total * me / G;
    const unsigned long long end = total * (me + 1) / G;
    bool first = true;
    while (u < end) {
      plan_find(a, S, kTaskCost, (long long)(u / HT), at);
      const int nu = seq_units(at.np) + kTaskCost;
      const unsigned long long rem = u - (unsigned long long)at.units * HT;
      const int j = (int)(rem / nu), p0 = (int)(rem % nu);
      const unsigned long long task = u - p0;              // first unit of the task
      const int step = (int)min((unsigned long long)(nu - p0), end - u);
      const int p1 = min(at.np, p0 + step);
      if (p0 < at.np) {                    // else the run begins behind the task's last page
        const bool part = p0 > 0 || p1 < at.np;
        const int slot = 2 * me + (first ? 0 : 1);
        if (p0 == 0 && part && tid == 0) {
          // the block that holds the task's last page, unit x: the largest i with total i / G <= x
          const int last = (int)(((task + at.np) * G - 1) / total);
          ws.slots[slot] = {at.b, j, last - me + 1, 2};
        }
        B::segment(a, smem, at.b, j, p0, p1, part ? ws.data + slot * attn_slot_floats(D) : nullptr);
      }
      first = false;
      u += step;
    }
  }
}

// Short page tables: a cluster of up to kMaxCluster blocks takes a task, page
// ranges of equal length, and merges over distributed shared memory: one
// launch, no workspace, no plan (attn_cluster below has the rule).
constexpr int kMaxCluster = 16;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

template <int D, class T>
__global__ void __launch_bounds__(kAttnThreads, kBlocksPerSm<D, T>) kvq_attention_cluster_kernel(AttnArgs a, int blocks) {
  using B = AttnBlock<D, T>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float part[attn_slot_floats(D)];
  const int tid = threadIdx.x, HT = a.c.hkv * a.tiles, rank = blockIdx.x % blocks;
  const long long task = blockIdx.x / blocks;
  const int b = (int)(task / HT), j = (int)(task % HT);
  const int np = seq_pages(a, b), n = max(np, 0);
  if (np < 0 && rank == 0 && tid == 0) flag_bad(a.c, MK_ERR_BAD_ARG);
  if (n > 0) B::segment(a, smem, b, j, (int)((long long)n * rank / blocks), (int)((long long)n * (rank + 1) / blocks), part);
  cluster_sync();
  const int heads = min(8, a.grp - j % a.tiles * 8);
  for (int i = rank + blocks * tid; i < heads * (D / 4); i += blocks * kAttnThreads) {
    const int h = i / (D / 4), dim = i % (D / 4) * 4;
    float m = -FLT_MAX, den = 0.f, num[4] = {0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
      constexpr int W = 8;                 // peers' loads in flight
      for (int k0 = 0; k0 < blocks; k0 += W) {
        float r[W], l[W];
        float4 o[W];
#pragma unroll
        for (int k = 0; k < W; k++) {
          r[k] = -FLT_MAX, l[k] = 0.f, o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < blocks) {
            uint32_t peer;
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_u32(part)), "r"(k0 + k));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r[k]) : "r"(peer + (8 * D + h) * 4));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(l[k]) : "r"(peer + (8 * D + 8 + h) * 4));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[k].x), "=f"(o[k].y), "=f"(o[k].z), "=f"(o[k].w)
                         : "r"(peer + (h * D + dim) * 4));
          }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < W; k++) mn = fmaxf(mn, r[k]);
        const float keep = ex2(m - mn);
        m = mn;
        den *= keep;
#pragma unroll
        for (int e = 0; e < 4; e++) num[e] *= keep;
#pragma unroll
        for (int k = 0; k < W; k++) {
          const float c = ex2(r[k] - m);
          num[0] = fmaf(c, o[k].x, num[0]);
          num[1] = fmaf(c, o[k].y, num[1]);
          num[2] = fmaf(c, o[k].z, num[2]);
          num[3] = fmaf(c, o[k].w, num[3]);
          den = fmaf(c, l[k], den);
        }
      }
    }
    T* dst = out_row<D, T>(a, b, j, h) + dim;
#pragma unroll
    for (int k = 0; k < 4; k++) stf(dst + k, n > 0 ? num[k] / den : np < 0 ? NAN : 0.f);
  }
  cluster_sync();                          // a block's shared memory stays until its peers have read it
}

constexpr int kMergeThreads = 256;
constexpr int kMaxSlots = 1024;

// Merges the parts of split tasks.  Every block lists the first slots, then
// takes (task, head) pairs in turn: a warp each eighth part, kBatch of them in
// flight (one load after the other, 76 parts of a 256K context took 11 us).
template <int D, class T>
__global__ void __launch_bounds__(kMergeThreads) kvq_merge_kernel(AttnArgs a, int blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int V = D / 32, kBatch = 5;    // dims of a lane
  __shared__ int list[kMaxSlots], n_list;  // first slots
  __shared__ AttnSlot head[kMaxSlots];     // and what they say
  __shared__ float so[8][D], sr[8], sl[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttnWs ws = attn_ws(a.ws, blocks);
  if (warp == 0) {
    // the first slots in order; nothing past the count is used, but it is read with it
    const int count = *ws.count;
    int n = 0;
    for (int s0 = 0; s0 < 2 * blocks; s0 += 32 * 10) {
      AttnSlot t[10];
#pragma unroll
      for (int i = 0; i < 10; i++) {
        const int s = s0 + 32 * i + lane;
        t[i].parts = 0;
        if (s < 2 * blocks) *(int4*)&t[i] = *(const int4*)&ws.slots[s];
      }
#pragma unroll
      for (int i = 0; i < 10; i++) {
        const int s = s0 + 32 * i + lane;
        const bool is = s < count && t[i].parts > 0;
        const unsigned m = __ballot_sync(0xffffffffu, is);
        const int at = n + __popc(m & ((1u << lane) - 1));
        if (is) list[at] = s, head[at] = t[i];
        n += __popc(m);
      }
    }
    if (lane == 0) n_list = n;
  }
  __syncthreads();
  for (int w = blockIdx.x; w < n_list * 8; w += gridDim.x) {
    const int s = list[w / 8], h = w % 8;
    const AttnSlot t = head[w / 8];
    if (h >= min(8, a.grp - t.j % a.tiles * 8)) continue;
    float m = -FLT_MAX, den = 0.f, num[V];
#pragma unroll
    for (int k = 0; k < V; k++) num[k] = 0.f;
    for (int i0 = warp; i0 < t.parts; i0 += 8 * kBatch) {
      float r[kBatch], l[kBatch], o[kBatch][V];
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const int i = i0 + 8 * u;
        const int slot = i == 0 ? s : t.step == 1 ? s + i : (s & ~1) + 2 * i;
        const float* p = ws.data + slot * attn_slot_floats(D);
        r[u] = -FLT_MAX, l[u] = 0.f;
#pragma unroll
        for (int k = 0; k < V; k++) o[u][k] = 0.f;
        if (i < t.parts) {
          r[u] = p[8 * D + h];
          l[u] = p[8 * D + 8 + h];
#pragma unroll
          for (int k = 0; k < V; k++) o[u][k] = p[h * D + lane + 32 * k];
        }
      }
      float mn = m;
#pragma unroll
      for (int u = 0; u < kBatch; u++) mn = fmaxf(mn, r[u]);
      const float keep = ex2(m - mn);
      den *= keep;
#pragma unroll
      for (int k = 0; k < V; k++) num[k] *= keep;
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const float c = ex2(r[u] - mn);
        den = fmaf(l[u], c, den);
#pragma unroll
        for (int k = 0; k < V; k++) num[k] = fmaf(o[u][k], c, num[k]);
      }
      m = mn;
    }
#pragma unroll
    for (int k = 0; k < V; k++) so[warp][lane + 32 * k] = num[k];
    if (lane == 0) sr[warp] = m, sl[warp] = den;
    __syncthreads();
    if (tid < D) {
      float M = -FLT_MAX, sn = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) M = fmaxf(M, sr[i]);
#pragma unroll
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

bool cache_shape(int n_kv_heads, int head_dim) {
  return (head_dim == 64 || head_dim == 128) && n_kv_heads >= 1 && n_kv_heads <= 1024;
}

int check_cache(const mk_kvq_cache* c) {
  if (!c) return MK_ERR_BAD_ARG;
  if (!cache_shape(c->n_kv_heads, c->head_dim) || c->num_pages < 1 || c->num_pages > 0x7fffffff / kKvqPage)
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

// A read's rows lie apart: no two of them share an element (nested strides, in
// whatever order), and keys and values have a place each
bool disjoint(const mk_kv_rows* r, const mk_kvq_cache* c, int unit) {
  struct Dim {
    unsigned long long stride;
    long long size;
  };
  auto size_of = [](int64_t s) { return s < 0 ? 0ull - (unsigned long long)s : (unsigned long long)s; };
  Dim d[3] = {{size_of(r->head_stride), c->n_kv_heads},
              {size_of(r->row_stride), unit == 1 ? r->count : kKvqPage},
              {size_of(r->page_stride), unit == 1 ? 1 : r->count}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  unsigned long long extent = (unsigned long long)c->head_dim;
  for (const Dim& x : d) {
    if (x.size <= 1) continue;
    if (x.stride < extent) return false;
    if (x.stride > (1ull << 62) / (unsigned long long)x.size) return false;   // no memory is that long
    extent += x.stride * (unsigned long long)(x.size - 1);
  }
  return r->k != r->v;
}

Cache cache_of(const mk_kvq_cache* c) { return Cache{(uint8_t*)c->pool, c->status, c->num_pages, c->n_kv_heads}; }

dim3 copy_grid(int n, int per_block, const mk_kvq_cache* c, int heads = 1) {
  return dim3((unsigned)(((long long)n + per_block - 1) / per_block), (unsigned)((c->n_kv_heads + heads - 1) / heads));
}

// KV heads of a block of a token call: as many as leave every SM the six
// blocks it can hold, in equal parts (8191 tokens of 4 heads stored and read
// back: 14 us with several heads a block, 16 with one)
int token_heads(int n, int per_block, const mk_kvq_cache* c, int sms) {
  const long long blocks = ((long long)n + per_block - 1) / per_block * c->n_kv_heads;
  const int most = (int)std::max(1ll, std::min<long long>(c->n_kv_heads, blocks / (6ll * sms)));
  const int parts = (c->n_kv_heads + most - 1) / most;
  return (c->n_kv_heads + parts - 1) / parts;
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

int check_tables(int type, int max_pages) {
  if (type != MK_TYPE_BF16 && type != MK_TYPE_F32) return MK_ERR_BAD_ARG;
  return max_pages < 0 || max_pages > 0x7fffffff / kKvqPage ? MK_ERR_BAD_ARG : MK_OK;
}

// blocks that fill the GPU, two slots each
int attn_blocks(int sms, int per_sm) { return std::min(sms * per_sm, kMaxSlots / 2); }

// Blocks of the cluster that takes a whole task, or 0: the two kernels with a
// workspace.  The cluster is the largest power of two with which all tasks run
// at once (half of the slots where it spans 8 SMs or more: a GPC holds two of
// those at best).  Its warps then have `mine` pages each of the longest
// sequence the page tables can hold, with all blocks sharing every page evenly
// it would be `even`; a page costs a warp about half a microsecond, the second
// kernel and the plan 1.5 to 8, and a batch with one long sequence among
// short ones must not wait for one cluster.  Measured, cluster against two
// kernels in a graph, 32 query and 4 KV heads of 128 dims: one sequence of 512
// 6.4 : 8.0 us, 8K 9.1 : 11.8, 16K 11.2 : 14.9; four of 8K 15.8 : 16.3, one of 8K
// and three of 100 11.6 : 12.1; sixteen up to 2K 11.7 : 18.4, of 4000 15.9 : 24.1;
// fp32, one of 12,000 11.5 : 12.0.  24,500 tokens are past the rule: 16.1.
int attn_cluster(long long tasks, int max_pages, int sms, int per_sm) {
  const long long slots = (long long)sms * per_sm;
  int n = 1;
  while (n < kMaxCluster && n * kAttnWarps < max_pages && 2 * n * tasks <= (2 * n >= 8 * per_sm ? slots / 2 : slots))
    n *= 2;
  const long long mine = (max_pages + n * kAttnWarps - 1) / (n * kAttnWarps);
  const long long even = tasks * max_pages / (slots * kAttnWarps);
  return mine <= 12 && mine - even <= 8 && tasks * n <= 0x7fffffff ? n : 0;
}

template <int D, class T>
int attention(AttnArgs& a, void* workspace, size_t workspace_bytes, int sms, cudaStream_t st) {
  // the kernels' shared memory is raised once on each device
  static std::atomic<unsigned long long> raised[2];
  constexpr size_t smem = AttnBlock<D, T>::kSmem;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return MK_ERR_CUDA;
  if (!(raised[dev / 64].load(std::memory_order_relaxed) >> (dev % 64) & 1)) {
    if (cudaFuncSetAttribute(kvq_attention_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kvq_attention_cluster_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem) != cudaSuccess ||
        cudaFuncSetAttribute(kvq_attention_cluster_kernel<D, T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    raised[dev / 64].fetch_or(1ull << (dev % 64), std::memory_order_relaxed);
  }
  const long long tasks = (long long)a.batch * a.c.hkv * a.tiles;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const int cluster = attn_cluster(tasks, a.max_pages, sms, kBlocksPerSm<D, T>);
  if (cluster) {
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(tasks * cluster));
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = smem;
    if (cudaLaunchKernelEx(&cfg, kvq_attention_cluster_kernel<D, T>, a, cluster) != cudaSuccess) {
      cudaGetLastError();
      return MK_ERR_CUDA;
    }
    return MK_OK;
  }
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < attn_ws_bytes(attn_blocks(sms, 2), D))
    return MK_ERR_BAD_ARG;
  a.ws = (uint8_t*)workspace;
  // no more blocks than there can be segments
  const long long most = tasks * std::max(1, (a.max_pages + kMinPages - 1) / kMinPages);
  const int blocks = (int)std::min<long long>(attn_blocks(sms, kBlocksPerSm<D, T>), most);
  kvq_attention_kernel<D, T><<<blocks, kAttnThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return MK_ERR_CUDA;
  // the merge is launched while the first kernel runs and waits for its end
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)std::min<long long>(sms, tasks * 8));
  cfg.blockDim = dim3(kMergeThreads);
  if (cudaLaunchKernelEx(&cfg, kvq_merge_kernel<D, T>, a, blocks) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return MK_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA; }

Rows rows_of(const mk_kv_rows* r) { return Rows{r->k, r->v, r->page_stride, r->row_stride, r->head_stride, r->count}; }

template <int D, class T>
int write_rows(const mk_kvq_cache* c, const mk_kv_rows* src, const int32_t* src_index, const int32_t* dst_index, int n,
               int unit, void* stream) {
  constexpr int kTokens = TokenLane<D>::kTokens;
  cudaStream_t st = (cudaStream_t)stream;
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  if (unit == 1) {
    const int heads = token_heads(n, kTokens, c, sms);
    kvq_write_kernel<D, T><<<copy_grid(n, kTokens, c, heads), kCopyThreads, 0, st>>>(cache_of(c), rows_of(src), src_index,
                                                                                    dst_index, n, heads);
  } else {
    const int heads = token_heads(n, kCopyThreads / 64, c, sms);
    kvq_write_pages_kernel<D, T><<<copy_grid(n, kCopyThreads / 64, c, heads), kCopyThreads, 0, st>>>(
        cache_of(c), rows_of(src), src_index, dst_index, n, heads);
  }
  return launched();
}

template <int D, class T>
int read_rows(const mk_kvq_cache* c, const int32_t* src_index, const mk_kv_rows* dst, const int32_t* dst_index, int n,
              int unit, void* stream) {
  constexpr int kTokens = TokenLane<D>::kTokens;
  cudaStream_t st = (cudaStream_t)stream;
  if (unit == 1) {
    const int sms = sm_count();
    if (!sms) return MK_ERR_CUDA;
    const int heads = token_heads(n, kTokens, c, sms);
    kvq_read_kernel<D, T><<<copy_grid(n, kTokens, c, heads), kCopyThreads, 0, st>>>(cache_of(c), src_index, rows_of(dst),
                                                                                   dst_index, n, heads);
  } else {
    kvq_read_pages_kernel<D, T><<<copy_grid(n, kCopyThreads / 32, c), kCopyThreads, 0, st>>>(
        cache_of(c), src_index, rows_of(dst), dst_index, n);
  }
  return launched();
}

}  // namespace

extern "C" {

size_t mk_kvq_page_bytes(int n_kv_heads, int head_dim) {
  if (!cache_shape(n_kv_heads, head_dim)) return 0;
  return (size_t)n_kv_heads * 18 * head_dim;
}

int mk_kvq_write(const mk_kvq_cache* c, const mk_kv_rows* src, const int32_t* src_index, const int32_t* dst_index,
                 int n, int unit, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_rows(src, c, n, unit, src_index, dst_index);
  if (rc || n == 0) return rc;
  if (c->head_dim == 128)
    return src->type == MK_TYPE_BF16 ? write_rows<128, uint16_t>(c, src, src_index, dst_index, n, unit, stream)
                                     : write_rows<128, float>(c, src, src_index, dst_index, n, unit, stream);
  return src->type == MK_TYPE_BF16 ? write_rows<64, uint16_t>(c, src, src_index, dst_index, n, unit, stream)
                                   : write_rows<64, float>(c, src, src_index, dst_index, n, unit, stream);
}

int mk_kvq_read(const mk_kvq_cache* c, const int32_t* src_index, const mk_kv_rows* dst, const int32_t* dst_index,
                int n, int unit, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_rows(dst, c, n, unit, dst_index, src_index);
  if (rc || n == 0) return rc;
  if (!disjoint(dst, c, unit)) return MK_ERR_BAD_ARG;
  if (c->head_dim == 128)
    return dst->type == MK_TYPE_BF16 ? read_rows<128, uint16_t>(c, src_index, dst, dst_index, n, unit, stream)
                                     : read_rows<128, float>(c, src_index, dst, dst_index, n, unit, stream);
  return dst->type == MK_TYPE_BF16 ? read_rows<64, uint16_t>(c, src_index, dst, dst_index, n, unit, stream)
                                   : read_rows<64, float>(c, src_index, dst, dst_index, n, unit, stream);
}

size_t mk_kvq_workspace(const mk_kvq_cache* c, int type, int n_q_heads, int batch, int max_pages) {
  if (check_cache(c) || check_heads(c, n_q_heads, batch) || check_tables(type, max_pages) || batch == 0) return 0;
  const int sms = sm_count();
  if (!sms) return 0;
  const int grp = n_q_heads / c->n_kv_heads;
  const long long tasks = (long long)batch * c->n_kv_heads * ((grp + 7) / 8);
  return attn_cluster(tasks, max_pages, sms, attn_per_sm(c->head_dim, type)) ? 0
                                                                             : attn_ws_bytes(attn_blocks(sms, 2), c->head_dim);
}

int mk_kvq_attention(const mk_kvq_cache* c, const void* q, int64_t q_stride, void* out, int64_t out_stride, int type,
                     int n_q_heads, int batch, const int32_t* page_tables, int max_pages, const int32_t* seq_lens,
                     float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_heads(c, n_q_heads, batch);
  if (!rc) rc = check_tables(type, max_pages);
  if (rc) return rc;
  if (!isfinite(scale)) return MK_ERR_BAD_ARG;
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
  cudaStream_t st = (cudaStream_t)stream;
  if (c->head_dim == 128)
    return type == MK_TYPE_BF16 ? attention<128, uint16_t>(a, workspace, workspace_bytes, sms, st)
                                : attention<128, float>(a, workspace, workspace_bytes, sms, st);
  return type == MK_TYPE_BF16 ? attention<64, uint16_t>(a, workspace, workspace_bytes, sms, st)
                              : attention<64, float>(a, workspace, workspace_bytes, sms, st);
}

}  // extern "C"

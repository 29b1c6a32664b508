// How the blocks of the paged cache's attention share its work: tasks, row
// blocks, key tiles, and the stretch that each block takes.  Compiled for the
// host too, where a test walks every block's stretch.
#pragma once
#include <stdint.h>

#include "mk.h"
#include "mk_kv.cuh"

namespace mk {

constexpr int kTile = 128;               // keys a step, rows a tile

// Cost of a row block, in keys: its own, and its start and end.  Fitted to the
// blocks' clocks over batches of prompts and single tokens: a key tile takes 2,300
// to 2,900 cycles where the rows fill two tiles (wide), 2,000 to 2,400 where they
// fit one (narrow); a start and an end 11,000 and 4,000 to 8,000.  (With 3 and 1
// tiles for these: packed prompts 89 us, 74 with 5 and 4.)
constexpr int kWideStart = 5 * kTile, kNarrowStart = 4 * kTile;
constexpr int kMinShare = 4 * kTile;              // no block takes less
// No part of an item has fewer key tiles: a part costs an end and its share of
// the merge, so that a wide one of less is better left where it is.
constexpr int kMinWidePart = 4, kMinPart = 2;

enum : int { kCausal = 1, kNan = 2, kPrefix = 4, kOrder = 16 };   // kOrder: its starts are out of order

template <class T>
MK_HD inline T hd_min(T a, T b) { return a < b ? a : b; }
template <class T>
MK_HD inline T hd_max(T a, T b) { return a > b ? a : b; }

// a stretch of key tiles [k0, k1) of n of one row block of one KV head
struct Part {
  int tok0, ntok;          // packed rows of q
  int head, table;         // KV head; page table row
  int kbeg, kend;          // keys of the block
  int lim;                 // keys that its first token sees end here; a causal one's next token sees one more
  int k0, k1, n;
  int flags;
  int slot;                // workspace slot of a part, -1: the whole item
};

// Sequences (b) and groups (g) that hold: those below b0, g0 and from b1, g1 on.
// Starts in order and in range hold all of them.  Else those before the first
// place that is not so hold and those after the last, but for what both sides
// name; all others have no rows, so that no row is two sequences' or two groups'.
struct Sound {
  int b0, b1, g0, g1;
};
MK_HD inline Sound all_hold() { return {0x7fffffff, 0x7fffffff, 0x7fffffff, 0x7fffffff}; }

MK_HD inline bool in_order(const int32_t* starts, int i, int end) {
  const int x = starts[i], y = starts[i + 1];
  return 0 <= x && x <= y && y <= end;
}

// of task t: a group's start and end, or a sequence's
MK_HD inline bool in_order(const KvAttnArgs& a, int t) {
  const bool g = t < a.groups;
  return in_order(g ? a.group_starts : a.q_starts, g ? t : t - a.groups, g ? a.batch : a.total_q);
}

// x0 and x1 of n starts and their end; first and last: the outermost that are out of order
MK_HD inline void holding(const int32_t* starts, int n, int first, int last, int* x0, int* x1) {
  int lo = first, hi = last + 1;
  if (first > 0 && last + 1 < n) {           // both sides are in order, each by itself
    const int to = starts[first], from = starts[last + 1];
    int a = -1, b = first;                   // the last start of the one side that is not past the other's first
    while (b > a) {
      const int mid = a + (b - a + 1) / 2;
      if (starts[mid] <= from) a = mid; else b = mid - 1;
    }
    lo = a < 0 ? 0 : a;
    a = last + 1, b = n;                     // the first of the other that is not before the one's last
    while (a < b) {
      const int mid = a + (b - a) / 2;
      if (starts[mid] >= to) b = mid; else a = mid + 1;
    }
    hi = a;
  }
  *x0 = lo, *x1 = hi;
}

// The packed rows that sequences own, as ends of two ranges.
MK_HD inline void owned_rows(const KvAttnArgs& a, const Sound& so, int32_t* rows) {
  rows[0] = a.q_starts[0], rows[1] = a.q_starts[so.b0 < a.batch ? so.b0 : a.batch];
  rows[2] = a.q_starts[so.b1 < a.batch ? so.b1 : a.batch], rows[3] = a.q_starts[a.batch];
}

struct Task {
  int tok0, ntok, nb;      // rows, row blocks
  int table, kbeg, kend;
  int c0;                  // causal: token i sees keys below c0 + i + 1
  int flags;
};

MK_HD inline Task load_task(const KvAttnArgs& a, int t, int tb, bool report, const Sound& so = all_hold()) {
  Task k{};
  if (t < a.groups) {
    const int s0 = a.group_starts[t], s1 = a.group_starts[t + 1], prefix = a.prefix_lens[t];
    const bool order = 0 <= s0 && s0 <= s1 && s1 <= a.batch;
    k.flags = order ? kPrefix : kPrefix | kOrder;
    bool ok = order && (t < so.g0 || t >= so.g1) &&
              (s0 == s1 || (prefix >= 0 && prefix % kKvPage == 0 && prefix <= a.max_pages * kKvPage));
    int q0 = 0, q1 = 0;
    if (ok) {                              // rows of those sequences that hold, and between them
      const int b0 = s0 < so.b0 ? s0 : hd_max(s0, so.b1), b1 = s1 > so.b1 ? s1 : hd_min(s1, so.b0);
      if (b0 < b1) q0 = a.q_starts[b0], q1 = a.q_starts[b1];
      ok = 0 <= q0 && q0 <= q1 && q1 <= a.total_q;
    }
    if (!ok) {
      if (report) flag(a.status, MK_ERR_BAD_ARG);
      q0 = q1 = 0;
    }
    k.tok0 = q0, k.ntok = q1 - q0;
    k.table = s0, k.kbeg = 0, k.kend = prefix;
  } else {
    const int b = t - a.groups;
    const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1], len = a.seq_lens[b];
    const bool order = 0 <= q0 && q0 <= q1 && q1 <= a.total_q, ok = order && (b < so.b0 || b >= so.b1);
    k.flags = order ? kCausal : kCausal | kOrder;
    k.tok0 = ok ? q0 : 0, k.ntok = ok ? q1 - q0 : 0;
    int prefix = 0;
    bool fit = len >= 0 && len <= a.max_pages * kKvPage;
    if (a.groups) {
      int lo = 0, hi = a.groups;          // the last group that starts at or before b, of those that hold on its side
      if (so.g0 < a.groups) {
        if (so.g0 > 0 && b < a.group_starts[so.g0]) hi = so.g0;
        else lo = hd_min(so.g1, hi - 1);
      }
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.group_starts[mid] <= b) lo = mid; else hi = mid;
      }
      // groups without sequences start there too
      prefix = a.prefix_lens[lo];
      const int s0 = a.group_starts[lo], s1 = a.group_starts[lo + 1];
      if (!(0 <= s0 && s0 <= b && b < s1 && s1 <= a.batch && (lo < so.g0 || lo >= so.g1))) fit = false;
      if (prefix < 0 || prefix % kKvPage || (fit && prefix > 0 && k.ntok > 0 && prefix > len - k.ntok)) fit = false;
    }
    if (!(ok && fit) && report) flag(a.status, MK_ERR_BAD_ARG);
    k.table = b;
    if (fit) k.kbeg = prefix, k.kend = len, k.c0 = len - k.ntok;
    else k.flags |= kNan;
  }
  k.nb = (k.ntok + tb - 1) / tb;
  return k;
}

MK_HD inline int block_end(const Task& k, int b, int tb) {      // end of a row block's keys
  if (k.flags & kNan) return k.kbeg;
  return k.flags & kCausal ? hd_max(k.kbeg, k.c0 + hd_min(k.ntok, (b + 1) * tb)) : k.kend;
}

MK_HD inline int block_tiles(const Task& k, int b, int tb) {
  return (block_end(k, b, tb) - k.kbeg + kTile - 1) / kTile;
}

// all row blocks but a task's last are wide
MK_HD inline bool wide(const Task& k, int b, int tb) { return b < k.nb - 1 || 2 * (k.ntok - b * tb) > tb; }

MK_HD inline int block_cost(const Task& k, int b, int tb) {
  return block_end(k, b, tb) - k.kbeg + (wide(k, b, tb) ? kWideStart : kNarrowStart);
}

// cost of the row blocks before b, b <= nb
MK_HD inline long long cost_before(const Task& k, int b, int tb) {
  if (b == 0) return 0;
  const int full = hd_min(b, k.nb - 1);
  long long keys = 0;
  if (full > 0) {
    if (k.flags & kCausal && !(k.flags & kNan)) {      // the sum of base + tb (i + 1) where that is positive
      const int base = k.c0 - k.kbeg, skip = base >= 0 ? 0 : hd_min(full, -base / tb);
      keys = (long long)(full - skip) * base +
             ((long long)full * (full + 1) - (long long)skip * (skip + 1)) / 2 * tb;
    } else if (!(k.flags & kNan)) {
      keys = (long long)full * (k.kend - k.kbeg);
    }
  }
  return keys + (long long)full * kWideStart + (b > full ? block_cost(k, b - 1, tb) : 0);
}

// An equal share of `total` for each block, from above, and no less than the least:
// total / blocks by a product with the blocks' reciprocal, which the host makes.
inline unsigned long long per_block(int blocks) { return ~0ull / (unsigned)blocks; }

MK_HD inline long long share_of(long long total, unsigned long long per) {
#ifdef __CUDA_ARCH__
  const unsigned long long high = __umul64hi((unsigned long long)total, per);
#else
  const unsigned long long high = (unsigned long long)((unsigned __int128)total * per >> 64);
#endif
  return hd_max((long long)high + 1, (long long)kMinShare);
}

// Where a border x keys into an item of n key tiles cuts it: the same for the
// block before and the block after.  Small shares are cut as they fall.
MK_HD inline int cut(long long x, bool wide, int n, long long share) {
  const int least = wide ? (int)hd_max(hd_min(share >> 10, (long long)kMinWidePart), (long long)kMinPart) : kMinPart;
  const int k = (int)((x + kTile / 2) / kTile);
  return k < least ? 0 : n - k < least ? n : k;
}

// floor(x / y) of 0 <= x, 0 < y whose quotient is small: a float's guess, put right
MK_HD inline int quotient(long long x, long long y) {
  int q = (int)((float)x / (float)y);
  while (q > 0 && q * y > x) q--;
  while ((q + 1) * y <= x) q++;
  return q;
}

// Where a block begins: in row block b of KV head `head` of task t, whose items
// begin at `at`.
struct Begin {
  Task k;
  int t, head, b;
  long long at;
};

// The item that holds position pos of task k, which begins at `start` and has
// `per` keys a KV head.  On the GPU a warp finds it together.
MK_HD inline Begin begin_of(const Task& k, int t, int tb, long long start, long long per, long long pos, int lane) {
  Begin g{k, t, 0, 0, start};
  g.head = quotient(pos - start, per);
  g.at += g.head * per;
  if (k.nb == 1) return g;
  const long long r = pos - g.at;
  int lo = 0, hi = k.nb;                 // the last row block that begins at or before pos
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
#ifdef __CUDA_ARCH__
    const int c = lo + step * lane;
    const int n = __popc(__ballot_sync(0xffffffffu, c < hi && cost_before(k, c, tb) <= r));
#else
    int n = 0;
    for (int i = 0; i < 32; i++) n += lo + step * i < hi && cost_before(k, lo + step * i, tb) <= r;
#endif
    lo += step * (n - 1);
    hi = hd_min(hi, lo + step);
  }
  g.b = lo;
  g.at += cost_before(k, lo, tb);
  return g;
}

// The parts of one block: its stretch [pos, stop) of all items laid end to end.
// On the GPU a warp walks it together.
struct Stretch {
  const KvAttnArgs& a;
  const Sound* so;         // NULL: all hold
  const int tb;
  int t, head, b;
  long long at;
  const long long pos, stop, share;
  Task k;

  MK_HD Stretch(const KvAttnArgs& args, int tt, const Begin& g, long long pos, long long stop, long long share,
                const Sound* sound = nullptr)
      : a(args), so(sound), tb(2 * tt), t(g.t), head(g.head), b(g.b), at(g.at), pos(pos), stop(stop), share(share), k(g.k) {}

  // The next task with rows.  Slots without any (a batch is padded with them) are
  // looked over 32 at a time: one by one, 4096 of them took 770 us, 3,960 with
  // groups.
  MK_HD void advance() {
    const int tasks = a.groups + a.batch;
    for (t++; t < tasks; t++) {
      k = load_task(a, t, tb, false, so ? *so : all_hold());
      if (k.nb) return;
#ifdef __CUDA_ARCH__
      unsigned some;
      do {
        const int x = t + 1 + (threadIdx.x & 31);
        some = __ballot_sync(0xffffffffu, x < tasks && may_have_rows(x));
        t += some ? __ffs(some) - 1 : 32;
      } while (!some && t + 1 < tasks);
#endif
    }
  }

  MK_HD bool may_have_rows(int x) const {
    if (x >= a.groups) return a.q_starts[x - a.groups] != a.q_starts[x - a.groups + 1];
    const int s0 = a.group_starts[x], s1 = a.group_starts[x + 1];
    if (so && so->b0 < a.batch) return true;             // its ends may not be those of what holds
    return 0 <= s0 && s0 < s1 && s1 <= a.batch && a.q_starts[s0] != a.q_starts[s1];
  }

  // the next part with anything to do; slots 2 c and 2 c + 1 are the block's
  MK_HD bool next(Part* m, int slot) {
    while (t < a.groups + a.batch && at < stop) {
      const int end = block_end(k, b, tb), n = block_tiles(k, b, tb), len = block_cost(k, b, tb);
      const bool w = wide(k, b, tb);
      const int k0 = at < pos ? cut(pos - at, w, n, share) : 0, k1 = at + len <= stop ? n : cut(stop - at, w, n, share);
      const bool some = k1 > k0 || (n == 0 && at >= pos);
      if (some) {
        m->tok0 = k.tok0 + b * tb, m->ntok = hd_min(tb, k.ntok - b * tb);
        m->head = head, m->table = k.table;
        m->kbeg = k.kbeg, m->kend = end;
        m->lim = k.flags & kCausal ? k.c0 + b * tb + 1 : k.kend;
        m->k0 = k0, m->k1 = k1, m->n = n, m->flags = k.flags;
        m->slot = k0 == 0 && k1 == n ? -1 : slot + (k0 == 0);
      }
      at += len;
      if (++b == k.nb) {
        b = 0;
        if (++head == a.hkv) {
          head = 0;
          if (at < stop) advance();
        }
      }
      if (some) return true;
    }
    return false;
  }
};

}  // namespace mk

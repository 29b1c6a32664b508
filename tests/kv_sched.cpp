// Walks every block's stretch of the paged cache's attention on the host: each
// (row block, KV head, key tile) is taken once, parts of an item follow each
// other from block to block in the slots where the merge looks for them, shares
// are even, and no part names a row, page table entry or head outside the call,
// whatever the starts, lengths and groups hold.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "mk_kv_sched.cuh"

using namespace mk;

static std::mt19937 rng;
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }
static int wide(int hi) { return pick(0, 3) ? pick(0, hi) : pick(0, 3); }

#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      std::printf("line %d: %s\n", __LINE__, #x);                    \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

static void walk(const KvAttnArgs& a, int blocks, bool sound) {
  const int tt = kTile / a.grp, tb = 2 * tt, tasks = a.groups + a.batch;
  std::vector<long long> at(tasks + 1, 0);
  for (int t = 0; t < tasks; t++) {
    const Task k = load_task(a, t, tb, true);
    CHECK(k.ntok >= 0 && k.tok0 >= 0 && (k.ntok == 0 || k.tok0 + k.ntok <= a.total_q));
    long long n = 0;
    for (int b = 0; b < k.nb; b++) {
      CHECK(cost_before(k, b, tb) == n);
      n += block_cost(k, b, tb);
      CHECK(block_cost(k, b, tb) == block_end(k, b, tb) - k.kbeg + (std::min(tb, k.ntok - b * tb) > tt ? kWideStart : kNarrowStart));
    }
    CHECK(cost_before(k, k.nb, tb) == n);
    at[t + 1] = at[t] + n * a.hkv;
  }
  const long long total = at[tasks], share = std::max((total + blocks - 1) / blocks, (long long)kMinShare);
  // (tok0, head, prefix) of an item -> its tiles taken so far
  std::map<std::tuple<int, int, int>, int> done;
  int open = 0;                                  // parts of the item that the block before left open
  std::tuple<int, int, int> open_key;
  for (int c = 0; c < blocks; c++) {
    const long long pos = share * c, stop = std::min(total, pos + share);
    if (pos >= total) {
      CHECK(!open);
      continue;
    }
    int t = 0;
    while (!(at[t] <= pos && pos < at[t + 1])) t++;
    const Task k = load_task(a, t, tb, false);
    Stretch w(a, tt, begin_of(k, t, tb, at[t], (at[t + 1] - at[t]) / a.hkv, pos, 0), pos, stop, share);
    Part m;
    long long units = 0;
    int used[2] = {0, 0};
    bool first = true, leaves = false;
    while (w.next(&m, 2 * c)) {
      CHECK(!leaves);                            // what is left open is the last
      const auto key = std::make_tuple(m.tok0, m.head, m.flags & kPrefix);
      CHECK(m.ntok >= 1 && m.ntok <= tb && m.tok0 >= 0 && m.tok0 + m.ntok <= a.total_q);
      CHECK(m.head >= 0 && m.head < a.hkv && m.table >= 0 && m.table < a.batch);
      CHECK(m.n == 0 || (m.kbeg >= 0 && m.kbeg % kKvPage == 0 && m.kend <= a.max_pages * kKvPage));
      CHECK(m.n == (m.kend - m.kbeg + kTile - 1) / kTile && 0 <= m.k0 && m.k0 <= m.k1 && m.k1 <= m.n);
      if (sound) CHECK((done.count(key) ? done[key] : 0) == m.k0 && (m.k0 > 0 || !done.count(key)));
      done[key] = m.k1;
      CHECK((m.slot < 0) == (m.k0 == 0 && m.k1 == m.n));
      if (m.slot >= 0) {
        CHECK(m.slot == 2 * c + (m.k0 == 0) && !used[m.k0 == 0]++);
        CHECK(m.k1 - m.k0 >= kMinPart && m.n > 3);        // three key tiles are never cut
      }
      if (m.k0 > 0) CHECK(first && open && key == open_key);
      leaves = m.k1 < m.n;
      if (first && open) CHECK(m.k0 > 0);
      if (leaves) open_key = key;
      first = false;
      units += std::min(kTile * m.k1, m.kend - m.kbeg) - kTile * m.k0 + (m.ntok > tt ? kWideStart : kNarrowStart);
    }
    open = leaves;
    CHECK(units <= share + 2 * kWideStart + 2 * (kMinWidePart + 1) * kTile);
  }
  CHECK(!open);
  if (!sound) return;
  for (int t = 0; t < tasks; t++) {
    const Task k = load_task(a, t, tb, false);
    for (int b = 0; b < k.nb; b++)
      for (int h = 0; h < a.hkv; h++) {
        const auto it = done.find(std::make_tuple(k.tok0 + b * tb, h, k.flags & kPrefix));
        CHECK(it != done.end() && it->second == block_tiles(k, b, tb));
      }
  }
}

int main(int argc, char** argv) {
  const int runs = argc > 1 ? std::atoi(argv[1]) : 300;
  rng.seed(argc > 2 ? std::atoi(argv[2]) : 0);
  for (int r = 0; r < runs; r++) {
    KvAttnArgs a{};
    const bool sound = pick(0, 3) > 0, big = pick(0, 40) == 0;
    a.head_dim = 128, a.hkv = pick(1, 6), a.grp = pick(0, 3) ? 1 << pick(0, 7) : pick(1, 128), a.hq = a.hkv * a.grp;
    a.batch = big ? pick(1, 3) : pick(1, 40);
    a.groups = pick(0, 1) ? pick(1, 5) : 0;
    std::vector<int32_t> starts(1, pick(0, 3)), lens, gs(1, 0), pl;
    std::vector<int> own(a.batch);
    int longest = 0;
    for (int g = 0; g < a.groups; g++) {
      gs.push_back(g + 1 == a.groups ? a.batch : pick(gs.back(), a.batch));
      pl.push_back(kKvPage * wide(big ? 4000 : 40));
      for (int b = gs[g]; b < gs[g + 1]; b++) own[b] = pl[g];
    }
    for (int b = 0; b < a.batch; b++) {
      const int n = wide(big ? 60000 : 700);
      lens.push_back(std::max(own[b] ? own[b] + n : 0, n + wide(big ? 90000 : 3000) - (own[b] ? 0 : pick(0, 30))));
      starts.push_back(starts.back() + n);
      longest = std::max(longest, lens.back());
    }
    a.max_pages = (longest + 15) / 16 + pick(0, 3);
    a.total_q = starts.back() + pick(0, 5);
    if (!sound)
      for (int x = 0; x < 4; x++) {
        const int32_t v = pick(0, 2) ? pick(-5, 2 * a.total_q + 20) : (pick(0, 1) ? INT32_MAX : INT32_MIN);
        switch (pick(0, 3)) {
          case 0: starts[pick(0, a.batch)] = v; break;
          case 1: lens[pick(0, a.batch - 1)] = v; break;
          case 2: if (a.groups) gs[pick(0, a.groups)] = v; break;
          default: if (a.groups) pl[pick(0, a.groups - 1)] = v;
        }
      }
    int32_t status = 0;
    a.q_starts = starts.data(), a.seq_lens = lens.data(), a.group_starts = gs.data(), a.prefix_lens = pl.data();
    a.status = &status;
    walk(a, pick(0, 1) ? 152 : pick(1, 200), sound);
    if (sound && status) {
      std::printf("a sound call was flagged\n");
      return 1;
    }
  }
  std::printf("ok\n");
}

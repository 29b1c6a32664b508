// The share that each block of the paged cache's attention takes, as the kernel
// computes it, on the host: the blocks together take everything, none more than
// one key above an equal part, and the stretches cut so cover every key tile once.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <tuple>
#include <vector>

#include "mk_kv_sched.cuh"

using namespace mk;

static std::mt19937_64 rng;
static long long pick(long long lo, long long hi) { return std::uniform_int_distribution<long long>(lo, hi)(rng); }

#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      std::printf("line %d: %s\n", __LINE__, #x);                    \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

static void shares() {
  for (int run = 0; run < 200000; run++) {
    const int blocks = run % 4 ? 152 : (int)pick(1, 1024);
    // up to 65535 sequences of 2^28 tokens and 1024 KV heads, and around multiples of the blocks
    long long total = pick(0, 1ll << pick(1, 54));
    if (run % 3 == 0) total = total / blocks * blocks + pick(-1, 1);
    if (total < 0) total = 0;
    const long long share = share_of(total, per_block(blocks));
    CHECK(share >= kMinShare && (__int128)share * blocks >= total);
    CHECK(share == kMinShare || share <= total / blocks + 1);
  }
}

// the kernel's own way to a block's first item: the task from the sums, then begin_of
static void walk(const KvAttnArgs& a, int blocks) {
  const int tt = kTile / a.grp, tb = 2 * tt, tasks = a.groups + a.batch;
  std::vector<long long> at(tasks + 1, 0), per(tasks, 0);
  for (int t = 0; t < tasks; t++) {
    const Task k = load_task(a, t, tb, false);
    per[t] = cost_before(k, k.nb, tb);
    at[t + 1] = at[t] + per[t] * a.hkv;
  }
  const long long total = at[tasks], share = share_of(total, per_block(blocks));
  std::map<std::tuple<int, int, int>, std::vector<int>> taken;
  for (int c = 0; c < blocks; c++) {
    const long long pos = share * c, stop = std::min(total, pos + share);
    for (int t = 0; t < tasks && pos < total; t++) {
      if (!(at[t] <= pos && pos < at[t + 1])) continue;
      Stretch w(a, tt, begin_of(load_task(a, t, tb, false), t, tb, at[t], per[t], pos, 0), pos, stop, share);
      Part m;
      while (w.next(&m, 2 * c)) {
        auto& v = taken[std::make_tuple(m.tok0, m.head, m.flags & kPrefix)];
        v.resize(m.n, 0);
        for (int j = m.k0; j < m.k1; j++) v[j]++;
      }
    }
  }
  for (int t = 0; t < tasks; t++) {
    const Task k = load_task(a, t, tb, false);
    for (int b = 0; b < k.nb; b++)
      for (int h = 0; h < a.hkv; h++) {
        const auto it = taken.find(std::make_tuple(k.tok0 + b * tb, h, k.flags & kPrefix));
        CHECK(it != taken.end() && (int)it->second.size() == block_tiles(k, b, tb));
        for (int n : it->second) CHECK(n == 1);
      }
  }
}

int main(int argc, char** argv) {
  rng.seed(argc > 1 ? std::atoi(argv[1]) : 0);
  shares();
  for (int run = 0; run < 150; run++) {
    KvAttnArgs a{};
    a.head_dim = 128, a.hkv = (int)pick(1, 8), a.grp = 1 << pick(0, 7), a.hq = a.hkv * a.grp;
    a.batch = (int)pick(1, 30), a.groups = pick(0, 1) ? 1 : 0;
    std::vector<int32_t> starts{0}, lens, groups{0, a.batch}, prefix{kKvPage * (int)pick(0, 2000)};
    for (int b = 0; b < a.batch; b++) {
      const int n = (int)(pick(0, 2) ? pick(0, 3) : pick(0, 3000));
      starts.push_back(starts.back() + n);
      lens.push_back((a.groups ? prefix[0] : 0) + n + (int)pick(0, pick(0, 5) ? 4000 : 200000));
    }
    a.total_q = starts.back(), a.max_pages = 1 << 20;
    a.q_starts = starts.data(), a.seq_lens = lens.data(), a.group_starts = groups.data(), a.prefix_lens = prefix.data();
    walk(a, pick(0, 2) ? 152 : (int)pick(1, 300));
  }
  std::printf("ok\n");
}

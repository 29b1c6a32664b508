// Sequences without rows behind the last that has some, on the host: the block
// whose stretch ends there does not look at them (their lengths lie outside the
// arrays that it is given: the address sanitizer sees a read).
#include <cstdio>
#include <vector>

#include "mk_kv_sched.cuh"

using namespace mk;

int main() {
  for (int groups = 0; groups < 2; groups++) {
    const int live = 3, idle = 1000, tt = 16, tb = 2 * tt;
    KvAttnArgs a{};
    a.head_dim = 128, a.hkv = 2, a.grp = 8, a.hq = 16, a.batch = live + idle, a.total_q = live, a.max_pages = 100;
    std::vector<int32_t> starts(a.batch + 1, live), group_starts{0, a.batch}, prefix{0};
    for (int b = 0; b < live; b++) starts[b] = b;
    if (groups) a.groups = 1, a.group_starts = group_starts.data(), a.prefix_lens = prefix.data();
    int32_t* lens = new int32_t[live]{700, 20, 1500};
    a.q_starts = starts.data(), a.seq_lens = lens;
    long long total = 0;
    Task first{};
    for (int t = 0; t < groups + live; t++) {
      const Task k = load_task(a, t, tb, false);
      if (t == 0) first = k;
      total += cost_before(k, k.nb, tb) * a.hkv;
    }
    // one block takes everything
    Stretch w(a, tt, begin_of(first, 0, tb, 0, cost_before(first, first.nb, tb), 0, 0), 0, total, total);
    Part m;
    int parts = 0;
    while (w.next(&m, 0)) parts++;
    delete[] lens;
    if (parts != 2 * (live + groups)) {
      std::printf("%d parts\n", parts);
      return 1;
    }
  }
  std::printf("ok\n");
}

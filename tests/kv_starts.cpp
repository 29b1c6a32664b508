// Starts out of order or out of range, on the host: which sequences and groups
// hold, and that every packed row which the join of own and common keys takes
// has one sequence and, unless that one is NaN, one group.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "mk_kv_sched.cuh"

using namespace mk;

static std::mt19937 rng;
static int pick(int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); }

#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      std::printf("line %d: %s\n", __LINE__, #x);                    \
      std::exit(1);                                                  \
    }                                                                \
  } while (0)

// pairs of x that are out of order, the outermost; none: n and -1
static void outermost(const std::vector<int32_t>& x, int end, int* first, int* last) {
  const int n = (int)x.size() - 1;
  *first = n, *last = -1;
  for (int i = 0; i < n; i++)
    if (!in_order(x.data(), i, end)) *first = std::min(*first, i), *last = i;
}

// what holds, from the definition: before the first and after the last pair out of order, and on one side only
static std::vector<bool> hold(const std::vector<int32_t>& x, int end) {
  const int n = (int)x.size() - 1;
  int first, last;
  outermost(x, end, &first, &last);
  std::vector<bool> h(n, last < 0);
  if (last < 0) return h;
  for (int i = 0; i < first; i++) h[i] = last + 1 >= n || x[i + 1] <= x[last + 1];
  for (int i = last + 1; i < n; i++) h[i] = first == 0 || x[i] >= x[first];
  return h;
}

static std::vector<int32_t> starts(int n, int end, bool spoil) {
  std::vector<int32_t> x(n + 1);
  for (auto& v : x) v = pick(0, end);
  std::sort(x.begin(), x.end());
  for (int k = spoil ? pick(1, 4) : 0; k > 0; k--)
    x[pick(0, n)] = pick(0, 3) ? pick(-3, end + 3) : pick(0, 1) ? INT32_MAX : INT32_MIN;
  return x;
}

int main(int argc, char** argv) {
  rng.seed(argc > 1 ? std::atoi(argv[1]) : 0);
  for (int run = 0; run < 4000; run++) {
    KvAttnArgs a{};
    a.hkv = 1, a.grp = 1 << pick(0, 5), a.hq = a.grp, a.head_dim = 64;
    a.batch = pick(1, 12), a.groups = pick(0, 3) ? pick(1, 6) : 0, a.total_q = pick(1, 40), a.max_pages = 40;
    const bool spoil_q = pick(0, 2) > 0, spoil_g = pick(0, 2) == 0;
    const auto qs = starts(a.batch, a.total_q, spoil_q);
    auto gs = starts(std::max(a.groups, 1), a.batch, false);
    if (pick(0, 2)) gs[0] = 0, gs.back() = a.batch;
    if (spoil_g) gs[pick(0, (int)gs.size() - 1)] = pick(-2, a.batch + 2);
    std::vector<int32_t> lens(a.batch), prefix(std::max(a.groups, 1));
    for (auto& v : lens) v = pick(0, 9) ? pick(100, 640) : pick(-20, 700);
    for (auto& v : prefix) v = pick(0, 4) ? kKvPage * pick(0, 3) : pick(0, 1) ? 7 : 100000 * kKvPage;
    int32_t status = 0;
    a.q_starts = qs.data(), a.seq_lens = lens.data(), a.group_starts = gs.data(), a.prefix_lens = prefix.data();
    a.status = &status;

    Sound so = all_hold();
    int first, last;
    bool bad = false;
    outermost(qs, a.total_q, &first, &last);
    if (last >= 0) holding(qs.data(), a.batch, first, last, &so.b0, &so.b1), bad = true;
    const auto seq_holds = hold(qs, a.total_q);
    for (int b = 0; b < a.batch; b++) CHECK(seq_holds[b] == (b < so.b0 || b >= so.b1));
    std::vector<bool> group_holds;
    if (a.groups) {
      outermost(gs, a.batch, &first, &last);
      if (last >= 0) holding(gs.data(), a.groups, first, last, &so.g0, &so.g1), bad = true;
      group_holds = hold(gs, a.batch);
      for (int g = 0; g < a.groups; g++) CHECK(group_holds[g] == (g < so.g0 || g >= so.g1));
    }

    const int tb = 2 * (kTile / a.grp);
    std::vector<int> own(a.total_q, 0), common(a.total_q, 0), nan(a.total_q, 0);
    for (int t = 0; t < a.groups + a.batch; t++) {
      CHECK(in_order(a, t) == (t < a.groups ? in_order(gs.data(), t, a.batch) : in_order(qs.data(), t - a.groups, a.total_q)));
      const Task k = load_task(a, t, tb, true, so);
      CHECK(k.ntok >= 0 && k.tok0 >= 0 && k.tok0 + k.ntok <= a.total_q);
      if (t >= a.groups) {
        const int b = t - a.groups;
        CHECK(k.ntok == (seq_holds[b] ? qs[b + 1] - qs[b] : 0));
        bool fits = lens[b] >= 0 && lens[b] <= a.max_pages * kKvPage;
        if (a.groups) {                               // its group, by looking at all of them
          int mine = 0, common = 0;
          for (int g = 0; g < a.groups; g++)
            if (group_holds[g] && gs[g] <= b && b < gs[g + 1]) mine++, common = prefix[g];
          CHECK(mine <= 1);
          fits = fits && mine && common % kKvPage == 0 && (k.ntok == 0 || common <= std::max(0, lens[b] - k.ntok));
          if (!(k.flags & kNan)) CHECK(k.kbeg == common);
        }
        if (k.ntok) CHECK(!(k.flags & kNan) == fits);
      }
      for (int r = k.tok0; r < k.tok0 + k.ntok; r++) (t < a.groups ? common : own)[r]++, nan[r] |= k.flags & kNan;
    }
    int32_t rows[4];
    owned_rows(a, so, rows);
    for (int r = 0; r < a.total_q; r++) {
      const bool owned = (rows[0] <= r && r < rows[1]) || (rows[2] <= r && r < rows[3]);
      CHECK(own[r] == (int)owned && common[r] <= 1);
      if (a.groups && owned && !nan[r]) CHECK(common[r] == 1);
    }
    if (bad) CHECK(status || a.total_q == 0);
  }
  std::printf("ok\n");
}

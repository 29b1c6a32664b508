// What the BF16 paged cache's attention (mk_kv_attn.cu) and its entry points
// (mk_kv.cu) share.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MK_HD __host__ __device__
#else
#define MK_HD
#endif

namespace mk {

MK_HD inline void flag(int32_t* status, int code) {
  if (status) *(volatile int32_t*)status = code;
}

constexpr int kKvPage = 16;
// A sequence's pages, at most.  An item is all of its keys for one block of rows:
// 2^21 key tiles of up to 2,900 cycles, 4.2 s at the 1455 MHz of long matrix products.
constexpr int kKvMaxPages = 1 << 24;
// A wait of the attention kernel for a key tile gives up after so long; one that may
// last over an item after so many times that.
constexpr unsigned long long kKvWaitNs = 4000000000ull;
constexpr int kKvItemWaits = 16;

struct KvAttnArgs {
  const uint16_t *q, *k_pool, *v_pool;
  uint16_t* out;
  const int32_t *q_starts, *page_tables, *seq_lens, *group_starts, *prefix_lens;
  int32_t* status;
  uint8_t* ws;
  int64_t q_stride, out_stride;
  int head_dim, hq, hkv, grp, total_q, batch, groups, max_pages, num_pages;
  float scale_log2;
  unsigned long long per_block;   // 2^64 / blocks of the grid, set by the launch
  int aligned32;                  // out and its rows lie at 32 bytes, likewise
};

// workspace bytes on a device of `sms` multiprocessors
size_t kv_attention_ws(int head_dim, int hq, int total_q, int groups, int sms);

// checked arguments; returns an mk_status
int kv_attention_launch(const KvAttnArgs& a, int sms, void* stream);

}  // namespace mk

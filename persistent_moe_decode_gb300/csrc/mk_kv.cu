// Operators on one layer's BF16 KV pools (include/mk.h, mk_rope_* and mk_kv_*):
// rotary positions, rows into the cache, attention over packed prompts and over
// a prefix that sequences share.
#include <cfloat>
#include <cmath>
#include <algorithm>

#include <cuda_runtime.h>

#include "mk.h"
#include "mk_kv.cuh"
#include "mk_ptx.cuh"

using namespace mk;

namespace {

constexpr int kPage = kKvPage;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------ rotary positions
//
// A block takes a few rows.  Its threads first put cos and sin of every (row,
// pair) in shared memory, once for all heads: the angle in turns is the high
// word of position * turns modulo 2^64, so no large angle is ever formed and the
// reduction costs one integer product.  Then each thread takes units of 16 dims
// of a head: two groups of 8 that are each other's partners, or 16 neighbours.
// Bound by memory: 32,768 rows of 36 heads of 128 dims in 100 us, 6.0 TB/s (89 %
// of the measured copy rate); 8191 rows with the append in 32 us, 5.3 TB/s (the
// last blocks leave SMs idle); 16 rows in 2.2 us.  Two units a thread at a time
// (64 registers instead of 44) took 110 and 40 us.
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxRows = 8;

struct RopeArgs {
  const uint64_t* turns;
  const int32_t* positions;
  const int32_t* slots;       // append: NULL otherwise
  int32_t* status;
  mk_head_rows q, k, v, q_out, k_out;
  uint16_t *k_pool, *v_pool;  // append: [pages][hkv][16][d]
  int n, rows_per_block, half, interleaved, num_pages;
  float magnitude;
};

template <class T>
__device__ __forceinline__ void load8(const T* p, float* f);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float* f) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; i++) f[2 * i] = bf16lo(u[i]), f[2 * i + 1] = bf16hi(u[i]);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float* f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float* f) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// T: type of the inputs, and of the outputs without the cache
template <int D, class T, bool APPEND>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr int U = D / 16;                     // units of a head
  __shared__ float2 cs[kRopeMaxRows * (D / 2)];
  const int row0 = blockIdx.x * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.n - row0);
  for (int i = threadIdx.x; i < rows * a.half; i += kRopeThreads) {
    const int t = i / a.half, p = i - t * a.half;
    const uint64_t phase = (uint64_t)(int64_t)a.positions[row0 + t] * a.turns[p];
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);     // half turns in [-1, 1]
    cs[i] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  __syncthreads();
  const int u = threadIdx.x % U, heads = a.q.n_heads + a.k.n_heads + (APPEND ? a.v.n_heads : 0);
  const int live = a.half / 8;                  // units that turn
  // the heads are shared out over the blocks of a row as well (gridDim.y)
  int at = threadIdx.x / U + blockIdx.y * (kRopeThreads / U), t = 0;
  const int step = kRopeThreads / U * gridDim.y;
  for (;; at += step) {
    while (at >= heads) at -= heads, t++;
    if (t >= rows) break;
    const int64_t row = row0 + t;
    int h = at;
    const mk_head_rows* src = &a.q;
    const mk_head_rows* dst = &a.q_out;
    int kind = 0;
    if (h >= a.q.n_heads) {
      h -= a.q.n_heads, src = &a.k, dst = &a.k_out, kind = 1;
      if (APPEND && h >= a.k.n_heads) h -= a.k.n_heads, src = &a.v, kind = 2;
    }
    const int lo = u < live && !a.interleaved ? 8 * u : 16 * u;
    const int hi = u < live && !a.interleaved ? a.half + 8 * u : 16 * u + 8;
    int64_t slot = 0;
    if (APPEND && kind) {
      slot = a.slots[row];
      if (slot >= (int64_t)a.num_pages * kPage) {
        flag(a.status, MK_ERR_BAD_PAGE);
        slot = -1;
      }
      if (slot < 0) continue;
    }
    const T* in = (const T*)src->data + row * src->row_stride + h * src->head_stride;
    float x[8], y[8];
    load8(in + lo, x);
    load8(in + hi, y);
    if (u < live && kind < 2) {
      if (a.interleaved) {
        const float2* w = cs + t * a.half + 8 * u;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float2 e = w[i], f = w[4 + i];
          const float p = x[2 * i], q = x[2 * i + 1], r = y[2 * i], s = y[2 * i + 1];
          x[2 * i] = p * e.x - q * e.y, x[2 * i + 1] = p * e.y + q * e.x;
          y[2 * i] = r * f.x - s * f.y, y[2 * i + 1] = r * f.y + s * f.x;
        }
      } else {
        const float2* w = cs + t * a.half + 8 * u;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float2 e = w[i];
          const float p = x[i], q = y[i];
          x[i] = p * e.x - q * e.y, y[i] = p * e.y + q * e.x;
        }
      }
    }
    if (APPEND && kind) {
      uint16_t* out = (kind == 1 ? a.k_pool : a.v_pool) +
                      (((slot / kPage) * a.k.n_heads + h) * kPage + slot % kPage) * D;
      store8(out + lo, x);
      store8(out + hi, y);
    } else {
      using O = typename std::conditional<APPEND, uint16_t, T>::type;
      O* out = (O*)dst->data + row * dst->row_stride + h * dst->head_stride;
      store8(out + lo, x);
      store8(out + hi, y);
    }
  }
}

// ------------------------------------------------------------------------ host

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int check_cache(const mk_kv_cache* c) {
  if (!c) return MK_ERR_BAD_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->num_pages < 1 ||
      c->num_pages >= 1 << 26)
    return MK_ERR_BAD_CONFIG;
  if (!c->k_pool || !c->v_pool || !aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->status, 4))
    return MK_ERR_BAD_ARG;
  return MK_OK;
}

int check_rope(const mk_rope* r) {
  if (!r) return MK_ERR_BAD_ARG;
  if ((r->head_dim != 64 && r->head_dim != 128) || r->rotary_dim < 16 || r->rotary_dim > r->head_dim ||
      r->rotary_dim % 16 || (r->interleaved != 0 && r->interleaved != 1))
    return MK_ERR_BAD_CONFIG;
  return !r->turns || !aligned(r->turns, 8) || !std::isfinite(r->magnitude) ? MK_ERR_BAD_ARG : MK_OK;
}

// rows of heads that a kernel may load 16 bytes at a time
int check_rows(const mk_head_rows* r, int n, int elem) {
  if (!r) return MK_ERR_BAD_ARG;
  if (r->n_heads < 0 || r->n_heads > 65536) return MK_ERR_BAD_CONFIG;
  if (n == 0 || r->n_heads == 0) return MK_OK;
  const int v = 16 / elem;
  return !r->data || !aligned(r->data, 16) || r->row_stride % v || r->head_stride % v ? MK_ERR_BAD_ARG : MK_OK;
}

// an output's rows and heads lie apart (one inside the other, in either order)
bool apart(const mk_head_rows* r, int n, int d) {
  const int64_t rs = r->row_stride, hs = r->head_stride;
  if (r->n_heads == 0 || n == 0) return true;
  if ((n > 1 && rs < d) || (r->n_heads > 1 && hs < d)) return false;
  if (n == 1 || r->n_heads == 1) return true;
  return rs <= hs ? hs >= rs * (n - 1) + d : rs >= hs * (r->n_heads - 1) + d;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <int D, class T, bool APPEND>
int launch_rope(RopeArgs& a, cudaStream_t st) {
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  const int heads = a.q.n_heads + a.k.n_heads + (APPEND ? a.v.n_heads : 0);
  // Rows a block: as many as still leave every SM eight blocks, so that a long
  // call's cos and sin are computed by full warps; below one row an SM the
  // row's heads are split over blocks, so that a step's few rows do not wait
  // for one block each.
  a.rows_per_block = std::max(1, std::min(kRopeMaxRows, a.n / (8 * sms)));
  const int per_row = (heads * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  const int split = a.n < sms ? std::max(1, std::min(per_row, 65535)) : 1;
  const dim3 grid((unsigned)((a.n + a.rows_per_block - 1) / a.rows_per_block), (unsigned)split);
  rope_kernel<D, T, APPEND><<<grid, kRopeThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

RopeArgs rope_args(const mk_rope* r, int n, const int32_t* positions) {
  RopeArgs a{};
  a.turns = r->turns;
  a.positions = positions;
  a.n = n;
  a.half = r->rotary_dim / 2;
  a.interleaved = r->interleaved;
  a.magnitude = r->magnitude;
  return a;
}

int check_attention(const mk_kv_cache* c, int n_q_heads, int total_q, int batch, int groups) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > 128) return MK_ERR_BAD_CONFIG;
  if (total_q < 0 || total_q > 1 << 24 || batch < 0 || batch > 65535 || groups < 0 || groups > 65535)
    return MK_ERR_BATCH_TOO_LARGE;
  return MK_OK;
}

}  // namespace

extern "C" {

int mk_rope_apply(const mk_rope* r, int n, const int32_t* positions, int type, const mk_head_rows* q,
                  const mk_head_rows* k, const mk_head_rows* q_out, const mk_head_rows* k_out, void* stream) {
  int rc = check_rope(r);
  if (rc) return rc;
  if (n < 0 || (type != MK_TYPE_BF16 && type != MK_TYPE_F32)) return MK_ERR_BAD_ARG;
  const int elem = type == MK_TYPE_BF16 ? 2 : 4;
  const mk_head_rows* in[2] = {q, k};
  const mk_head_rows* out[2] = {q_out, k_out};
  for (int i = 0; i < 2; i++) {
    if ((rc = check_rows(in[i], n, elem)) || (rc = check_rows(out[i], n, elem))) return rc;
    if (in[i]->n_heads != out[i]->n_heads || !apart(out[i], n, r->head_dim)) return MK_ERR_BAD_ARG;
  }
  if (n == 0 || q->n_heads + k->n_heads == 0) return MK_OK;
  if (!positions || !aligned(positions, 4)) return MK_ERR_BAD_ARG;
  RopeArgs a = rope_args(r, n, positions);
  a.q = *q, a.k = *k, a.q_out = *q_out, a.k_out = *k_out;
  cudaStream_t st = (cudaStream_t)stream;
  if (r->head_dim == 128)
    return elem == 2 ? launch_rope<128, uint16_t, false>(a, st) : launch_rope<128, float, false>(a, st);
  return elem == 2 ? launch_rope<64, uint16_t, false>(a, st) : launch_rope<64, float, false>(a, st);
}

int mk_kv_append(const mk_kv_cache* c, const mk_rope* r, int n, const int32_t* positions, int type,
                 const mk_head_rows* q, const mk_head_rows* k, const mk_head_rows* v, const int32_t* slots,
                 const mk_head_rows* q_out, void* stream) {
  int rc = check_cache(c);
  if (!rc) rc = check_rope(r);
  if (rc) return rc;
  if (r->head_dim != c->head_dim) return MK_ERR_BAD_CONFIG;
  if (n < 0 || (type != MK_TYPE_BF16 && type != MK_TYPE_F32)) return MK_ERR_BAD_ARG;
  const int elem = type == MK_TYPE_BF16 ? 2 : 4;
  if ((rc = check_rows(q, n, elem)) || (rc = check_rows(k, n, elem)) || (rc = check_rows(v, n, elem)) ||
      (rc = check_rows(q_out, n, 2)))
    return rc;
  if (k->n_heads != c->n_kv_heads || v->n_heads != c->n_kv_heads || q_out->n_heads != q->n_heads ||
      !apart(q_out, n, c->head_dim))
    return MK_ERR_BAD_ARG;
  if (n == 0) return MK_OK;
  if (!positions || !aligned(positions, 4) || !slots || !aligned(slots, 4)) return MK_ERR_BAD_ARG;
  RopeArgs a = rope_args(r, n, positions);
  a.q = *q, a.k = *k, a.v = *v, a.q_out = *q_out;
  a.slots = slots;
  a.status = c->status;
  a.k_pool = (uint16_t*)c->k_pool;
  a.v_pool = (uint16_t*)c->v_pool;
  a.num_pages = c->num_pages;
  cudaStream_t st = (cudaStream_t)stream;
  if (r->head_dim == 128)
    return elem == 2 ? launch_rope<128, uint16_t, true>(a, st) : launch_rope<128, float, true>(a, st);
  return elem == 2 ? launch_rope<64, uint16_t, true>(a, st) : launch_rope<64, float, true>(a, st);
}

size_t mk_kv_workspace(const mk_kv_cache* c, int n_q_heads, int total_q, int batch, int groups) {
  if (check_attention(c, n_q_heads, total_q, batch, groups) || total_q == 0 || batch == 0) return 0;
  const int sms = sm_count();
  return sms ? kv_attention_ws(c->head_dim, n_q_heads, total_q, groups, sms) : 0;
}

int mk_kv_attention(const mk_kv_cache* c, const void* q, int64_t q_stride, void* out, int64_t out_stride,
                    int n_q_heads, int total_q, int batch, const int32_t* q_starts, const int32_t* page_tables,
                    int max_pages, const int32_t* seq_lens, int groups, const int32_t* group_starts,
                    const int32_t* prefix_lens, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_attention(c, n_q_heads, total_q, batch, groups);
  if (rc) return rc;
  if (max_pages < 0 || max_pages > kKvMaxPages || !(scale > 0.f) || scale >= 0x1p20f) return MK_ERR_BAD_ARG;
  if (total_q == 0 || batch == 0) return MK_OK;
  const int64_t row = (int64_t)n_q_heads * c->head_dim;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8 ||
      (total_q > 1 && (q_stride < row || out_stride < row)) || !q_starts || !aligned(q_starts, 4) || !seq_lens ||
      !aligned(seq_lens, 4) || (max_pages && (!page_tables || !aligned(page_tables, 4))) ||
      (groups && (!group_starts || !aligned(group_starts, 4) || !prefix_lens || !aligned(prefix_lens, 4))))
    return MK_ERR_BAD_ARG;
  const int sms = sm_count();
  if (!sms) return MK_ERR_CUDA;
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < kv_attention_ws(c->head_dim, n_q_heads, total_q, groups, sms))
    return MK_ERR_BAD_ARG;
  KvAttnArgs a{};
  a.ws = (uint8_t*)workspace;
  a.head_dim = c->head_dim;
  a.q = (const uint16_t*)q;
  a.k_pool = (const uint16_t*)c->k_pool;
  a.v_pool = (const uint16_t*)c->v_pool;
  a.out = (uint16_t*)out;
  a.q_starts = q_starts, a.page_tables = page_tables, a.seq_lens = seq_lens;
  a.group_starts = group_starts, a.prefix_lens = prefix_lens;
  a.status = c->status;
  a.q_stride = q_stride, a.out_stride = out_stride;
  a.hq = n_q_heads, a.hkv = c->n_kv_heads, a.grp = n_q_heads / c->n_kv_heads;
  a.total_q = total_q, a.batch = batch, a.groups = groups, a.max_pages = max_pages, a.num_pages = c->num_pages;
  a.scale_log2 = scale * kLog2e;
  return kv_attention_launch(a, sms, stream);
}

}  // extern "C"

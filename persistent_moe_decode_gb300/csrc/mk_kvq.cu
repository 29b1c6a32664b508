// Operators of the 4-bit key/value cache (declared in include/mk.h): rows or
// pages quantised into it, read back from it, and one-token attention over it.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

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

struct AttnArgs {
  Cache c;
  const void* q;
  void* out;
  const int32_t* page_tables;
  const int32_t* seq_lens;
  long long q_stride, out_stride;          // elements between two sequences
  int hq, grp, batch, max_pages;
  float scale_log2;
};

constexpr int kAttnWarps = 8;

__device__ __forceinline__ void stf(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void stf(float* p, float v) { *p = v; }

// one block per (sequence, KV head, 8 of its query heads); its warps take the
// sequence's pages in turn and merge at the end
template <int D, class T>
__global__ void __launch_bounds__(kAttnWarps * 32, 2) kvq_attention_kernel(AttnArgs a) {
  constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  using R = KvqRec<D>;
  using A = KvqAttn<D, TERMS, TERMS>;
  constexpr int NG = R::NG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gl = lane >> 2, cq = lane & 3;
  const int tiles = (a.grp + 7) / 8, b = blockIdx.y, g = blockIdx.x / tiles, h0 = blockIdx.x % tiles * 8;
  const int heads = min(8, a.grp - h0);
  __shared__ float sm_o[kAttnWarps][8][D];
  __shared__ float sm_r[kAttnWarps][8], sm_l[kAttnWarps][8];

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
  int len = a.seq_lens[b];
  bool bad = false;
  if (len < 0 || len > a.max_pages * kKvqPage) {
    if (threadIdx.x == 0) flag_bad(a.c, MK_ERR_BAD_ARG);
    bad = true;
    len = 0;
  }
  const int np = (len + kKvqPage - 1) / kKvqPage;
  for (int p = warp; p < np; p += kAttnWarps) {
    int id = a.page_tables[(long long)b * a.max_pages + p];
    if (id < 0 || id >= a.c.pages) {
      if (lane == 0) flag_bad(a.c, MK_ERR_BAD_PAGE);
      bad = true;
      id = 0;
    }
    typename A::Page pg;
    A::load(pg, a.c.pool + ((long long)id * a.c.hkv + g) * R::kBytes, lane);
    at.page(pg, min(kKvqPage, len - p * kKvqPage), lane);
  }
  float v[NG][2][8];
  at.finish(v);
#pragma unroll
  for (int h = 0; h < 2; h++) {
#pragma unroll
    for (int k = 0; k < NG; k++) {
      float* dst = &sm_o[warp][2 * cq + h][k * kKvqGroup + 8 * gl];
      *(float4*)dst = make_float4(v[k][h][0], v[k][h][1], v[k][h][2], v[k][h][3]);
      *(float4*)(dst + 4) = make_float4(v[k][h][4], v[k][h][5], v[k][h][6], v[k][h][7]);
    }
    if (gl == 0) {
      sm_r[warp][2 * cq + h] = at.r[h];
      sm_l[warp][2 * cq + h] = bad ? NAN : at.l[h];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * D; i += kAttnWarps * 32) {
    const int h = i / D, dim = i % D;
    float m = -FLT_MAX, num = 0.f, den = 0.f;
    for (int w = 0; w < kAttnWarps; w++) m = fmaxf(m, sm_r[w][h]);
    for (int w = 0; w < kAttnWarps; w++) {
      const float k = ex2(sm_r[w][h] - m);
      num = fmaf(k, sm_o[w][h][dim], num);
      den = fmaf(k, sm_l[w][h], den);
    }
    // no key at all: zeros
    stf((T*)a.out + b * a.out_stride + (long long)(g * a.grp + h0 + h) * D + dim, den == 0.f ? 0.f : num / den);
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
  (void)c, (void)n_q_heads, (void)batch;
  return 0;
}

int mk_kvq_attention(const mk_kvq_cache* c, const void* q, int64_t q_stride, void* out, int64_t out_stride, int type,
                     int n_q_heads, int batch, const int32_t* page_tables, int max_pages, const int32_t* seq_lens,
                     float scale, void* workspace, size_t workspace_bytes, void* stream) {
  (void)workspace, (void)workspace_bytes;
  int rc = check_cache(c);
  if (rc) return rc;
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads > 65536) return MK_ERR_BAD_CONFIG;
  if (type != MK_TYPE_BF16 && type != MK_TYPE_F32) return MK_ERR_BAD_ARG;
  if (batch < 0 || batch > 65535) return MK_ERR_BATCH_TOO_LARGE;
  if (max_pages < 0 || max_pages > 0x7fffffff / kKvqPage || !isfinite(scale)) return MK_ERR_BAD_ARG;
  if (batch == 0) return MK_OK;
  const int64_t v = type == MK_TYPE_BF16 ? 8 : 4;
  if (!q || !out || !seq_lens || (max_pages && !page_tables) || !aligned(q, 16) || !aligned(out, 16) ||
      q_stride % v || out_stride % v || (batch > 1 && out_stride < (int64_t)n_q_heads * c->head_dim))
    return MK_ERR_BAD_ARG;
  AttnArgs a{};
  a.c = cache_of(c);
  a.q = q;
  a.out = out;
  a.page_tables = page_tables;
  a.seq_lens = seq_lens;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.hq = n_q_heads;
  a.grp = n_q_heads / c->n_kv_heads;
  a.batch = batch;
  a.max_pages = max_pages;
  a.scale_log2 = scale * 1.4426950408889634f;
  const dim3 grid(c->n_kv_heads * ((a.grp + 7) / 8), batch);
  cudaStream_t st = (cudaStream_t)stream;
  if (c->head_dim == 128)
    type == MK_TYPE_BF16 ? kvq_attention_kernel<128, uint16_t><<<grid, kAttnWarps * 32, 0, st>>>(a)
                         : kvq_attention_kernel<128, float><<<grid, kAttnWarps * 32, 0, st>>>(a);
  else
    type == MK_TYPE_BF16 ? kvq_attention_kernel<64, uint16_t><<<grid, kAttnWarps * 32, 0, st>>>(a)
                         : kvq_attention_kernel<64, float><<<grid, kAttnWarps * 32, 0, st>>>(a);
  return launched();
}

}  // extern "C"

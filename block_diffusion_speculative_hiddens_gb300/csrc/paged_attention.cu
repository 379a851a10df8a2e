// Attention of a ragged batch of new tokens over a caller's paged cache.
//
// One warp per (row, query head): each lane holds head_dim/32 dims of the
// query and of the running output; a key's score is a warp sum, the softmax
// runs in one pass with a running maximum and sum (log2 domain).
#include "common.cuh"
#include "internal.h"

namespace {

struct PagedParams {
  const uint16_t* q;
  uint16_t* out;
  long long q_row, q_head, o_row, o_head;
  float* lse;
  long long lse_row, lse_head;
  const uint16_t* k;
  const uint16_t* v;
  long long kp, ks, kh, vp, vs, vh;
  const int* table;
  long long table_stride;
  int max_pages, n_pages, shift;
  const int* cu;
  const int* ctx;
  const int* kv_len;
  int rows, batch, hq, group, causal, window;
  float scale_log2;
  uint32_t* status;
};

template <bool BF16>
DFL_DEV float to_float(uint16_t v) {
  if constexpr (BF16) return __bfloat162float(*reinterpret_cast<bf16*>(&v));
  else return __half2float(*reinterpret_cast<f16*>(&v));
}

template <bool BF16, int D>
__global__ void __launch_bounds__(128) k_paged_attn(const PagedParams p) {
  constexpr int E = D / 32;
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int sb;
  if (threadIdx.x == 0) sb = -1;
  __syncthreads();
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
    if (t >= p.cu[b] && t < p.cu[b + 1]) sb = b;
  __syncthreads();
  const int b = sb;
  if (b < 0) return;
  const int n = p.cu[b + 1] - p.cu[b];
  const long long pos = (long long)p.ctx[b] + t - p.cu[b];
  long long kv = p.kv_len ? p.kv_len[b] : (long long)p.ctx[b] + n;
  const long long cap = (long long)p.max_pages << p.shift;
  if (kv > cap) {
    dev_error(p.status, DFLASH_DEV_PAGE);
    kv = cap;
  }
  const long long hi = p.causal && pos + 1 < kv ? pos + 1 : kv;
  const long long lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
  for (int h = warp; h < p.hq; h += 4) {
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
      q[e] = to_float<BF16>(p.q[t * p.q_row + h * p.q_head + lane * E + e]);
      o[e] = 0.f;
    }
    const int kvh = h / p.group;
    for (long long j = lo; j < hi; ++j) {
      const int pg = p.table[b * p.table_stride + (j >> p.shift)];
      const bool ok = pg >= 0 && pg < p.n_pages;
      if (!ok) dev_error(p.status, DFLASH_DEV_PAGE);
      const long long in = j & ((1 << p.shift) - 1);
      const uint16_t* kr = p.k + (ok ? pg * p.kp + in * p.ks + kvh * p.kh : 0);
      const uint16_t* vr = p.v + (ok ? pg * p.vp + in * p.vs + kvh * p.vh : 0);
      float s = 0.f;
      for (int e = 0; e < E; ++e) s += q[e] * (ok ? to_float<BF16>(kr[lane * E + e]) : 0.f);
      s = warp_sum(s) * p.scale_log2;
      const float mn = fmaxf(m, s);
      const float a = mn == -INFINITY ? 1.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
      l = l * a + w;
      m = mn;
      for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * (ok ? to_float<BF16>(vr[lane * E + e]) : 0.f);
    }
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    for (int e = 0; e < E; ++e) {
      const float y = o[e] * inv;
      uint16_t r;
      if constexpr (BF16) {
        bf16 z = __float2bfloat16_rn(y);
        r = *reinterpret_cast<uint16_t*>(&z);
      } else {
        f16 z = __float2half_rn(y);
        r = *reinterpret_cast<uint16_t*>(&z);
      }
      p.out[t * p.o_row + h * p.o_head + lane * E + e] = r;
    }
    if (p.lse && lane == 0)
      p.lse[t * p.lse_row + h * p.lse_head] = l > 0.f ? (m + log2f(l)) * 0.69314718056f : l == 0.f ? -INFINITY : l;
  }
}

bool rows_ok(const dflash_rows& r) {
  return (reinterpret_cast<uintptr_t>(r.data) & 15) == 0 && r.row_stride % 8 == 0 && r.head_stride % 8 == 0;
}

}  // namespace

extern "C" {

size_t dflash_paged_attention_workspace(const dflash_paged_cache* c, int32_t rows, int32_t batch, int32_t q_heads) {
  (void)rows;
  (void)batch;
  (void)q_heads;
  return paged_cache_check(c) ? 0 : 256;
}

int dflash_paged_attention(const dflash_paged_cache* c, const dflash_attention_args* a, void* stream) {
  if (!a || a->rows < 0 || a->batch < 0 || a->window < 0 || !(a->scale == a->scale)) return DFLASH_ERR_INVALID_ARG;
  if (int e = paged_cache_check(c)) return e;
  const int D = c->head_dim;
  if ((D != 64 && D != 128) || a->q_heads < 1 || a->q_heads % c->kv_heads || a->q_heads / c->kv_heads > 32)
    return DFLASH_ERR_SHAPE;
  if (a->rows == 0 || a->batch == 0) return DFLASH_OK;
  if (!a->q.data || !a->out.data || !a->cu_rows || !a->ctx_len || !rows_ok(a->q) || !rows_ok(a->out) ||
      !rows_ok({c->k, c->k_pos_stride, c->k_head_stride}) || !rows_ok({c->v, c->v_pos_stride, c->v_head_stride}) ||
      c->k_page_stride % 8 || c->v_page_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 255) || a->workspace_bytes < 0 ||
      (size_t)a->workspace_bytes < dflash_paged_attention_workspace(c, a->rows, a->batch, a->q_heads))
    return DFLASH_ERR_WORKSPACE;
  PagedParams p = {};
  p.q = static_cast<const uint16_t*>(a->q.data);
  p.out = static_cast<uint16_t*>(a->out.data);
  p.q_row = a->q.row_stride;
  p.q_head = a->q.head_stride;
  p.o_row = a->out.row_stride;
  p.o_head = a->out.head_stride;
  p.lse = a->lse;
  p.lse_row = a->lse_row_stride;
  p.lse_head = a->lse_head_stride;
  p.k = static_cast<const uint16_t*>(c->k);
  p.v = static_cast<const uint16_t*>(c->v);
  p.kp = c->k_page_stride, p.ks = c->k_pos_stride, p.kh = c->k_head_stride;
  p.vp = c->v_page_stride, p.vs = c->v_pos_stride, p.vh = c->v_head_stride;
  p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.shift = page_shift(c->page_size);
  p.cu = a->cu_rows;
  p.ctx = a->ctx_len;
  p.kv_len = a->kv_len;
  p.rows = a->rows;
  p.batch = a->batch;
  p.hq = a->q_heads;
  p.group = a->q_heads / c->kv_heads;
  p.causal = a->causal != 0;
  p.window = a->window;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.status = c->status;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (c->dtype == DFLASH_BF16) {
    if (D == 64) k_paged_attn<true, 64><<<p.rows, 128, 0, s>>>(p);
    else k_paged_attn<true, 128><<<p.rows, 128, 0, s>>>(p);
  } else {
    if (D == 64) k_paged_attn<false, 64><<<p.rows, 128, 0, s>>>(p);
    else k_paged_attn<false, 128><<<p.rows, 128, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"

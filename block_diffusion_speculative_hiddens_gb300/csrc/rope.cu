// Rotary positions and the append to a caller's paged cache.
//
// A rotated pair (a, b) of dims at position p becomes
//   (a cos(p w) - b sin(p w), a sin(p w) + b cos(p w)) * amplitude.
// The angle is kept as turns modulo 1 in 64-bit fixed point: turn[i] =
// w_i / 2 pi in units of 2^-64, so p * turn[i] in wrapping 64-bit arithmetic
// drops the whole turns exactly and far positions lose nothing (a float angle
// is off by 2^-24 of itself: 0.06 rad at position 10^6).  The top 32 bits, as
// a signed fraction of a half turn, go through sincospif.
//
// Each row's cos and sin are computed once per CTA into shared memory and
// serve all of its heads.  A thread moves two 16-byte vectors of one head at a
// time: the two halves of 8 pairs, or 16 adjacent dims, so a pair never
// crosses threads and an output may be its own input.
//
// Bound by memory: each value is read and written once.  Replayed in a graph,
// 8,191 rows of 40 heads of 128 (168 MB) take 27.7 us, 6.1 TB/s, 0.89 of the copy
// rate; 7,500 rows appended with their queries (184 MB) 32.8 us, 5.6 TB/s.  A row a
// CTA with two units of a thread in flight: four rows a CTA took 29.4 and 37.5 us,
// one or three units in flight 31.3 and 29.6; the page looked up by a warp that
// also computes angles 35.1 for 33.4 us of appending.  A call of 16 rows is 2.6 us
// of launch, load, angles and store.
// A row's sequence is searched 32 at a time by a warp: an append of one row each
// takes 3.3 us for up to 64 sequences, 4.5 for 256 and 11.5 for 1,024.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace {

struct RowsIn {
  const uint16_t* src;
  long long row, head;  // strides, elements
};
struct RowsOut {
  uint16_t* dst;
  long long row, head;
};

struct RopeParams {
  RowsIn in[3];   // q, k, v (heads 0 where absent)
  RowsOut out[2]; // q, k of dflash_rope; [0] of the append
  int heads[3];
  int rows, D, rd, interleaved, backward;
  float amplitude;
  const int* positions;  // dflash_rope
  // append
  const int* cu;
  const int* ctx;
  int batch;
  RowsOut pool[2];               // k, v: row = position stride
  long long page_stride[2];
  const int* table;
  long long table_stride;
  int max_pages, n_pages, page_shift;
  uint32_t* status;
  int rows_per_cta, lanes;  // lanes: heads that a pass of the block takes
  uint64_t turn[DFLASH_ROPE_MAX_PAIRS];
};

template <bool BF16>
DFL_DEV float2 unpack2(uint32_t v) {
  if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&v));
  else return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <bool BF16>
DFL_DEV uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}
template <bool BF16>
DFL_DEV float unpack1(uint16_t v) {
  if constexpr (BF16) return __bfloat162float(*reinterpret_cast<bf16*>(&v));
  else return __half2float(*reinterpret_cast<f16*>(&v));
}
template <bool BF16>
DFL_DEV uint16_t pack1(float a) {
  if constexpr (BF16) {
    bf16 v = __float2bfloat16_rn(a);
    return *reinterpret_cast<uint16_t*>(&v);
  } else {
    f16 v = __float2half_rn(a);
    return *reinterpret_cast<uint16_t*>(&v);
  }
}

constexpr int ROPE_MAX_ROWS = 8;   // rows of a CTA
constexpr int ROPE_THREADS = 256;  // at most
constexpr int ROPE_AHEAD = 2;      // units of a thread whose loads are in flight at once

struct RowPlace {
  int valid;            // 0: padding row
  int write;            // its page exists
  int seq;
  long long pos;
  long long off[2];     // element offset of its place in the k and v pools
};

// VEC: a unit is two 16-byte vectors (16 dims); else one pair of dims.
template <bool BF16, bool VEC, bool APPEND>
__global__ void __launch_bounds__(ROPE_THREADS) k_rope(const __grid_constant__ RopeParams p) {
  __shared__ RowPlace place[ROPE_MAX_ROWS];
  __shared__ __align__(16) float2 cs[ROPE_MAX_ROWS][DFLASH_ROPE_MAX_PAIRS];
  const int row0 = blockIdx.x * p.rows_per_cta;
  const int nr = min(p.rows_per_cta, p.rows - row0);
  const int U = VEC ? p.D >> 4 : p.D >> 1;      // units of a head
  const int c = threadIdx.x % U;
  const int H = p.heads[0] + p.heads[1] + (APPEND ? p.heads[2] : 0);
  const int step = p.lanes;
  const int rot = VEC ? p.rd >> 4 : p.rd >> 1;  // rotated units of a head
  const bool turned = c < rot;
  // first element of the unit's two parts
  int e0, e1;
  if (VEC) {
    if (p.interleaved) e0 = 16 * c, e1 = e0 + 8;
    else if (turned) e0 = 8 * c, e1 = e0 + (p.rd >> 1);
    else e0 = p.rd + 16 * (c - rot), e1 = e0 + 8;
  } else {
    if (p.interleaved) e0 = 2 * c, e1 = e0 + 1;
    else if (turned) e0 = c, e1 = e0 + (p.rd >> 1);
    else e0 = p.rd + 2 * (c - rot), e1 = e0 + 1;
  }
  using Part = typename std::conditional<VEC, uint4, uint16_t>::type;
  struct Unit {
    Part a, b;
    int r, which, h;  // row of the CTA (-1: none), tensor, head
  };
  auto load = [&](Unit& u, int it) {
    u.r = it >= nr * H ? -1 : nr == 1 ? 0 : it / H;  // a row a CTA needs no division
    if (u.r < 0) return;
    u.h = it - u.r * H;
    u.which = u.h < p.heads[0] ? 0 : u.h < p.heads[0] + p.heads[1] ? 1 : 2;
    u.h -= u.which == 0 ? 0 : u.which == 1 ? p.heads[0] : p.heads[0] + p.heads[1];
    const RowsIn& in = p.in[u.which];
    const uint16_t* src = in.src + (long long)(row0 + u.r) * in.row + u.h * in.head;
    u.a = *reinterpret_cast<const Part*>(src + e0);
    u.b = *reinterpret_cast<const Part*>(src + e1);
  };
  pdl_launch_dependents();
  pdl_wait();
  // the first units' loads need no position: they are on their way while the
  // row's place and angles are found
  Unit unit[ROPE_AHEAD];
  int it = threadIdx.x / U;
  if (it >= step) it = nr * H;  // a thread that only fills the last warp
#pragma unroll
  for (int i = 0; i < ROPE_AHEAD; ++i) load(unit[i], it + i * step);
  if (APPEND) {
    // a warp finds a row's sequence and position; its page is looked up while
    // the angles are computed
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    for (int r = threadIdx.x >> 5; r < nr; r += warps) {
      const int t = row0 + r;
      RowPlace w = {};
      __syncwarp();  // the loads above, and the last row's search, may have parted the lanes
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        const bool in = b < p.batch;
        const int lo = in ? p.cu[b] : 0, hi = in ? p.cu[b + 1] : 0, ctx = in ? p.ctx[b] : 0;
        const uint32_t found = __ballot_sync(0xffffffffu, in && t >= lo && t < hi);
        if (!found) continue;
        if (lane == __ffs(found) - 1) {
          w.valid = 1;
          w.seq = b;
          w.pos = (long long)ctx + (t - lo);
          place[r] = w;
        }
        w.valid = 1;
        break;
      }
      if (!w.valid && lane == 0) place[r] = w;
    }
    __syncthreads();
    const int mine = blockDim.x - 1 - threadIdx.x;  // by the last threads: the first ones have the angles
    if (mine < nr && place[mine].valid) {
      RowPlace& w = place[mine];
      const long long pi = w.pos >> p.page_shift;
      const int pg = w.pos >= 0 && pi < p.max_pages ? p.table[w.seq * p.table_stride + pi] : -1;
      if (pg >= 0 && pg < p.n_pages) {
        const long long in_page = w.pos & ((1 << p.page_shift) - 1);
        w.write = 1;
        w.off[0] = pg * p.page_stride[0] + in_page * p.pool[0].row;
        w.off[1] = pg * p.page_stride[1] + in_page * p.pool[1].row;
      } else {
        dev_error(p.status, DFLASH_DEV_PAGE);
      }
    }
  }
  const int pairs = p.rd >> 1;
  for (int i = threadIdx.x; i < nr * pairs; i += blockDim.x) {
    const int r = i / pairs, j = i - r * pairs;
    const long long pos = APPEND ? (place[r].valid ? place[r].pos : 0) : (long long)p.positions[row0 + r];
    const uint64_t turns = (uint64_t)pos * p.turn[j];
    float s, co;
    sincospif((float)(int32_t)(uint32_t)(turns >> 32) * 0x1p-31f, &s, &co);
    cs[r][j] = make_float2(co * p.amplitude, (p.backward ? -s : s) * p.amplitude);
  }
  __syncthreads();

  auto finish = [&](Unit& u) {
    if (u.r < 0 || (APPEND && !place[u.r].valid)) return;
    uint16_t* dst;
    if (APPEND && u.which > 0) {
      if (!place[u.r].write) return;
      dst = p.pool[u.which - 1].dst + place[u.r].off[u.which - 1] + u.h * p.pool[u.which - 1].head;
    } else {
      dst = p.out[u.which].dst + (long long)(row0 + u.r) * p.out[u.which].row + u.h * p.out[u.which].head;
    }
    if (turned && u.which < 2) {
      if constexpr (VEC) {
        uint32_t x[4] = {u.a.x, u.a.y, u.a.z, u.a.w}, y[4] = {u.b.x, u.b.y, u.b.z, u.b.w};
        const float4* w4 = reinterpret_cast<const float4*>(&cs[u.r][8 * c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = w4[i];  // two pairs' (cos, sin)
          if (p.interleaved) {     // words of the unit's 8 pairs in order
            uint32_t& u0 = i < 2 ? x[2 * i] : y[2 * i - 4];
            uint32_t& u1 = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
            const float2 f0 = unpack2<BF16>(u0), f1 = unpack2<BF16>(u1);
            u0 = pack2<BF16>(f0.x * w.x - f0.y * w.y, f0.x * w.y + f0.y * w.x);
            u1 = pack2<BF16>(f1.x * w.z - f1.y * w.w, f1.x * w.w + f1.y * w.z);
          } else {
            const float2 fa = unpack2<BF16>(x[i]), fb = unpack2<BF16>(y[i]);
            x[i] = pack2<BF16>(fa.x * w.x - fb.x * w.y, fa.y * w.z - fb.y * w.w);
            y[i] = pack2<BF16>(fa.x * w.y + fb.x * w.x, fa.y * w.w + fb.y * w.z);
          }
        }
        u.a = make_uint4(x[0], x[1], x[2], x[3]);
        u.b = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        const float2 w = cs[u.r][c];
        const float fa = unpack1<BF16>(u.a), fb = unpack1<BF16>(u.b);
        u.a = pack1<BF16>(fa * w.x - fb * w.y);
        u.b = pack1<BF16>(fa * w.y + fb * w.x);
      }
    }
    *reinterpret_cast<Part*>(dst + e0) = u.a;
    *reinterpret_cast<Part*>(dst + e1) = u.b;
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) finish(unit[i]);
    it += ROPE_AHEAD * step;
    if (it >= nr * H) break;
#pragma unroll
    for (int i = 0; i < ROPE_AHEAD; ++i) load(unit[i], it + i * step);
  }
}

// Clears bits that the host has read, and none that were set since.
__global__ void k_clear_status(uint32_t* status, uint32_t bits) { atomicAnd(status, ~bits); }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <bool APPEND>
int launch_rope(RopeParams& p, bool bf16_, bool vec, cudaStream_t s) {
  // One row a CTA, its heads ROPE_AHEAD units a thread if that fits; rows with
  // few heads share a CTA.
  const int U = vec ? p.D / 16 : p.D / 2;
  const int H = p.heads[0] + p.heads[1] + p.heads[2], per = ROPE_THREADS / U;  // heads a pass, at most
  p.rows_per_cta = std::max(1, std::min(ROPE_MAX_ROWS, ROPE_AHEAD * per / std::max(H, 1)));
  const int items = p.rows_per_cta * H;
  p.lanes = std::min(per, std::max((items + ROPE_AHEAD - 1) / ROPE_AHEAD, (64 + U - 1) / U));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows + p.rows_per_cta - 1) / p.rows_per_cta));
  cfg.blockDim = dim3((unsigned)((U * p.lanes + 31) / 32 * 32));  // whole warps: the append's search takes one a row
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (bf16_) e = vec ? cudaLaunchKernelEx(&cfg, k_rope<true, true, APPEND>, p)
                     : cudaLaunchKernelEx(&cfg, k_rope<true, false, APPEND>, p);
  else e = vec ? cudaLaunchKernelEx(&cfg, k_rope<false, true, APPEND>, p)
               : cudaLaunchKernelEx(&cfg, k_rope<false, false, APPEND>, p);
  return cuda_status(e);
}

void set_plan(RopeParams& p, const dflash_rope_plan* plan) {
  p.rd = plan->rotary_dim;
  p.interleaved = plan->interleaved;
  p.amplitude = plan->amplitude;
  for (int i = 0; i < p.rd / 2; ++i) p.turn[i] = plan->turn[i];
}

bool plan_ok(const dflash_rope_plan* plan, int D) {
  return plan->rotary_dim >= 2 && plan->rotary_dim <= D && plan->rotary_dim % 2 == 0 &&
         (plan->interleaved == 0 || plan->interleaved == 1);
}

bool vec_ok(const dflash_rows& r) { return aligned16(r.data) && r.row_stride % 8 == 0 && r.head_stride % 8 == 0; }

}  // namespace

// Waits for the device, returns a status word and clears the bits that it returns.
int read_status_word(uint32_t* status, int device, uint32_t* out) {
  DeviceGuard guard(device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  uint32_t bits = 0;
  if (int e = cuda_status(cudaDeviceSynchronize())) return e;
  if (int e = cuda_status(cudaMemcpy(&bits, status, sizeof(bits), cudaMemcpyDeviceToHost))) return e;
  if (bits) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = cfg.blockDim = dim3(1);
    if (int e = cuda_status(cudaLaunchKernelEx(&cfg, k_clear_status, status, bits))) return e;
    if (int e = cuda_status(cudaDeviceSynchronize())) return e;
  }
  *out = bits;
  return DFLASH_OK;
}

extern "C" {

int dflash_rope_init(const dflash_rope_config* c, dflash_rope_plan* plan) {
  if (!c || !plan) return DFLASH_ERR_INVALID_ARG;
  const int rd = c->rotary_dim;
  if (rd < 2 || rd > 2 * DFLASH_ROPE_MAX_PAIRS || rd % 2 || (c->interleaved != 0 && c->interleaved != 1) ||
      !(c->theta > 1.0) || !std::isfinite(c->theta) || c->scaling < DFLASH_ROPE_PLAIN || c->scaling > DFLASH_ROPE_FACTORS)
    return DFLASH_ERR_INVALID_ARG;
  const int kind = c->scaling;
  const double pi2 = 6.283185307179586476925286766559;
  const double f = kind == DFLASH_ROPE_PLAIN || kind == DFLASH_ROPE_FACTORS ? 1.0 : c->factor;
  if (!(f > 0.0) || !std::isfinite(f)) return DFLASH_ERR_INVALID_ARG;
  double amplitude = 1.0, theta = c->theta, lo = 0.0, hi = 0.0;
  if (kind == DFLASH_ROPE_NTK) {
    if (rd == 2) return DFLASH_ERR_INVALID_ARG;
    theta *= std::pow(f, rd / (rd - 2.0));
    if (!(theta > 1.0) || !std::isfinite(theta)) return DFLASH_ERR_INVALID_ARG;
  }
  if (kind == DFLASH_ROPE_YARN || kind == DFLASH_ROPE_LLAMA3) {
    if (c->original_len < 1) return DFLASH_ERR_INVALID_ARG;
  }
  if (kind == DFLASH_ROPE_YARN) {
    if (!(c->beta_slow > 0.0) || !(c->beta_fast >= c->beta_slow) || !std::isfinite(c->beta_fast))
      return DFLASH_ERR_INVALID_ARG;
    // the pair index that makes beta turns over original_len positions
    auto at = [&](double beta) { return rd * std::log(c->original_len / (beta * pi2)) / (2.0 * std::log(theta)); };
    lo = std::fmax(std::floor(at(c->beta_fast)), 0.0);
    hi = std::fmin(std::ceil(at(c->beta_slow)), rd - 1.0);
    amplitude = 0.1 * std::log(f) + 1.0;
  }
  if (kind == DFLASH_ROPE_LLAMA3 &&
      (!(c->low_freq >= 0.0) || !(c->high_freq > c->low_freq) || !std::isfinite(c->high_freq)))
    return DFLASH_ERR_INVALID_ARG;
  if (kind == DFLASH_ROPE_FACTORS) {
    if (!c->factors) return DFLASH_ERR_INVALID_ARG;
    for (int i = 0; i < rd / 2; ++i)
      if (!(c->factors[i] > 0.0) || !std::isfinite(c->factors[i])) return DFLASH_ERR_INVALID_ARG;
  }
  if (kind == DFLASH_ROPE_YARN || kind == DFLASH_ROPE_FACTORS) {
    if (!(c->attention_factor >= 0.0) || !std::isfinite(c->attention_factor)) return DFLASH_ERR_INVALID_ARG;
    if (c->attention_factor > 0.0) amplitude = c->attention_factor;
  }
  dflash_rope_plan out = {};
  out.rotary_dim = rd;
  out.interleaved = c->interleaved;
  out.amplitude = (float)amplitude;
  for (int i = 0; i < rd / 2; ++i) {
    double w = std::pow(theta, -2.0 * i / rd);
    if (kind == DFLASH_ROPE_LINEAR) w /= f;
    if (kind == DFLASH_ROPE_FACTORS) w /= c->factors[i];
    if (kind == DFLASH_ROPE_YARN) {
      const double m = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      w = w * (1.0 - m) + w / f * m;
    }
    if (kind == DFLASH_ROPE_LLAMA3) {
      const double turns = c->original_len * w / pi2;
      const double m = std::fmin(std::fmax((turns - c->low_freq) / (c->high_freq - c->low_freq), 0.0), 1.0);
      w = w * m + w / f * (1.0 - m);
    }
    double whole;
    const double turn = std::modf(w / pi2, &whole);  // in [0, 1): 2^64 of it fits 64 bits
    out.turn[i] = (uint64_t)std::ldexp(turn, 64);
  }
  *plan = out;
  return DFLASH_OK;
}

int dflash_rope(const dflash_rope_plan* plan, const dflash_rope_args* a, void* stream) {
  if (!plan || !a || a->rows < 0 || a->q_heads < 0 || a->k_heads < 0 || (a->dtype != DFLASH_F16 && a->dtype != DFLASH_BF16))
    return DFLASH_ERR_INVALID_ARG;
  const int D = a->head_dim;
  if (D < 2 || D > 2 * DFLASH_ROPE_MAX_PAIRS || D % 2 || !plan_ok(plan, D)) return DFLASH_ERR_SHAPE;
  RopeParams p = {};
  p.heads[0] = a->q.data ? a->q_heads : 0;
  p.heads[1] = a->k.data ? a->k_heads : 0;
  if (a->rows == 0 || p.heads[0] + p.heads[1] == 0) return DFLASH_OK;
  if (!a->positions || (p.heads[0] && !a->q_out.data) || (p.heads[1] && !a->k_out.data)) return DFLASH_ERR_INVALID_ARG;
  const dflash_rows* in[2] = {&a->q, &a->k};
  const dflash_rows* out[2] = {&a->q_out, &a->k_out};
  bool vec = D % 16 == 0 && plan->rotary_dim % 16 == 0;
  for (int i = 0; i < 2; ++i) {
    if (!p.heads[i]) continue;
    p.in[i] = {static_cast<const uint16_t*>(in[i]->data), in[i]->row_stride, in[i]->head_stride};
    p.out[i] = {static_cast<uint16_t*>(out[i]->data), out[i]->row_stride, out[i]->head_stride};
    vec = vec && vec_ok(*in[i]) && vec_ok(*out[i]);
  }
  const Strided qo = strided_rows(a->q_out, a->rows, p.heads[0], D), ko = strided_rows(a->k_out, a->rows, p.heads[1], D);
  const Strided q = input_of(a->q_out, a->q, a->rows, p.heads[0], D), k = input_of(a->k_out, a->k, a->rows, p.heads[1], D);
  if (!apart({qo, ko}, {q, k, strided_ints(a->positions, a->rows)})) return DFLASH_ERR_INVALID_ARG;
  p.rows = a->rows;
  p.D = D;
  p.backward = a->backward != 0;
  p.positions = a->positions;
  set_plan(p, plan);
  DeviceGuard guard(a->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  return launch_rope<false>(p, a->dtype == DFLASH_BF16, vec, static_cast<cudaStream_t>(stream));
}

int dflash_paged_read_status(const dflash_paged_cache* c, uint32_t* out) {
  if (!out) return DFLASH_ERR_INVALID_ARG;
  if (int e = paged_cache_check(c)) return e;
  return read_status_word(c->status, c->device, out);
}

int dflash_paged_append(const dflash_paged_cache* c, const dflash_rope_plan* plan, const dflash_append_args* a,
                        void* stream) {
  if (!a || a->rows < 0 || a->batch < 0 || a->q_heads < 0) return DFLASH_ERR_INVALID_ARG;
  if (int e = paged_cache_check(c)) return e;
  const int D = c->head_dim;
  if (D < 2 || D > 2 * DFLASH_ROPE_MAX_PAIRS || D % 2 || (plan && !plan_ok(plan, D))) return DFLASH_ERR_SHAPE;
  if (a->rows == 0 || a->batch == 0) return DFLASH_OK;
  if (!a->k.data || !a->v.data || !a->cu_rows || !a->ctx_len || (a->q.data && !a->q_out.data)) return DFLASH_ERR_INVALID_ARG;
  RopeParams p = {};
  p.heads[0] = a->q.data ? a->q_heads : 0;
  p.heads[1] = p.heads[2] = c->kv_heads;
  bool vec = D % 16 == 0 && (!plan || plan->rotary_dim % 16 == 0);
  const dflash_rows pk = {c->k, c->k_pos_stride, c->k_head_stride}, pv = {c->v, c->v_pos_stride, c->v_head_stride};
  vec = vec && vec_ok(a->k) && vec_ok(a->v) && vec_ok(pk) && vec_ok(pv) && c->k_page_stride % 8 == 0 && c->v_page_stride % 8 == 0;
  p.in[1] = {static_cast<const uint16_t*>(a->k.data), a->k.row_stride, a->k.head_stride};
  p.in[2] = {static_cast<const uint16_t*>(a->v.data), a->v.row_stride, a->v.head_stride};
  if (p.heads[0]) {
    vec = vec && vec_ok(a->q) && vec_ok(a->q_out);
    p.in[0] = {static_cast<const uint16_t*>(a->q.data), a->q.row_stride, a->q.head_stride};
    p.out[0] = {static_cast<uint16_t*>(a->q_out.data), a->q_out.row_stride, a->q_out.head_stride};
  }
  const Strided kp = strided_pool(c, false), vp = strided_pool(c, true), table = strided_table(c, a->batch),
                cu = strided_ints(a->cu_rows, a->batch + 1ll), ctx = strided_ints(a->ctx_len, a->batch),
                status = strided_ints(reinterpret_cast<const int32_t*>(c->status), 1);
  if (!apart({kp, vp}, {table, cu, ctx, status}) ||
      !apart({strided_rows(a->q_out, a->rows, p.heads[0], D)},
             {input_of(a->q_out, a->q, a->rows, p.heads[0], D), strided_rows(a->k, a->rows, c->kv_heads, D),
              strided_rows(a->v, a->rows, c->kv_heads, D), kp, vp, table, cu, ctx, status}))
    return DFLASH_ERR_INVALID_ARG;
  p.pool[0] = {static_cast<uint16_t*>(c->k), c->k_pos_stride, c->k_head_stride};
  p.pool[1] = {static_cast<uint16_t*>(c->v), c->v_pos_stride, c->v_head_stride};
  p.page_stride[0] = c->k_page_stride;
  p.page_stride[1] = c->v_page_stride;
  p.rows = a->rows;
  p.batch = a->batch;
  p.cu = a->cu_rows;
  p.ctx = a->ctx_len;
  p.D = D;
  p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.page_shift = page_shift(c->page_size);
  p.status = c->status;
  if (plan) set_plan(p, plan);
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  return launch_rope<true>(p, c->dtype == DFLASH_BF16, vec, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

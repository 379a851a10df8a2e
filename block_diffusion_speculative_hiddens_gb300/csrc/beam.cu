// The next beams of a search: the n best of beams * vocab continuations a
// request, scored by the running score and the logarithm of the softmax.
//
// One pass over the logits, a part of a row a CTA: each thread sums
// exp(logit - reference) and keeps its maximum.  The n-th largest of the CTA's
// thread maxima bounds its n-th largest logit from below, and only the n threads
// whose maximum reaches it can hold one of the n: their logits are read again
// (from L2) and the n best kept, sorted.  A second kernel, a CTA a request, joins
// the parts' sums and chooses among their lists in the same way, by score.
//
// The order within a row is the logits' own, so equal logits tie exactly.  Between
// rows the scores are compared in 64 bits; the sums behind them are kept so that
// rows with equal logits get equal sums, whatever their alignment: which thread
// takes a logit goes by its index alone.
//
// Sums: exponents are taken to base 2 against an integer reference, so that the
// parts' sums join by exact shifts; a thread's sum is a float (600 terms at most
// between two parts' ends), its join a 64-bit fixed-point sum.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace {

#ifndef BEAM_SLOTS
#define BEAM_SLOTS (152 * 4)
#endif
#ifndef BEAM_AHEAD
#define BEAM_AHEAD 4
#endif
constexpr int SCAN_THREADS = 256;
constexpr int AHEAD = BEAM_AHEAD;          // vectors of a thread in flight
constexpr int SEGMENTS = 4;       // of a part, with a maximum each
constexpr int MAX_SPLITS = 64;    // parts of a row
constexpr int MAX_LISTS = 1024;   // parts of a request's rows
constexpr int JOIN_THREADS = 512;
constexpr int LIST_LANES = 8;     // of the join that look through a list together
constexpr int KEEP = 640;         // keys that a selection holds: a push of one a thread, and what was kept before it

// log2(e) in two floats: their sum is off by 2^-50.
constexpr float LOG2E_HI = 1.44269502162933349609f;
constexpr float LOG2E_LO = 1.92596299112661746887e-8f;
constexpr double LN2 = 0.693147180559945309417232121458;

// What a part of a row leaves: the sum of exp(x - reference).  The reference is
// q * ln 2 if `base2`, else the part's largest logit (which is too large or too
// small for the shared exponent).
struct PartSum {
  unsigned long long sum;  // units of 2^-FIX
  float q;
  float top;               // largest logit; -inf: no tokens are offered
  int base2;
  int reserved;
};
constexpr int FIX = 34;

struct BeamParams {
  const char* logits;
  long long row_bytes;
  const float* scores;
  const uint8_t* done;
  float* scores_out;
  int* parents;
  int* tokens;
  uint32_t* status;
  PartSum* sums;             // [rows][splits]
  unsigned long long* best;  // [rows][splits][n] keys
  int batch, beams, vocab, n, splits, part;  // part: vectors of a split
  int done_token;
};

DFL_DEV void flag_nan(uint32_t* status) {
  if (status) dev_error(status, DFLASH_DEV_NAN);
}

// A float's bits in the order of its value (-0 as 0).
DFL_DEV uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
DFL_DEV float unordered(uint32_t o) { return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu)); }
DFL_DEV unsigned long long ordered(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
DFL_DEV double unordered(unsigned long long o) {
  return __longlong_as_double((long long)(o ^ ((o >> 63) ? 1ull << 63 : ~0ull)));
}

DFL_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats in a register pair, for the packed operations.
struct Pair {
  unsigned long long v;
};
DFL_DEV Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
DFL_DEV void unpair(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
DFL_DEV Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
DFL_DEV Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// Sixteen bytes of logits.  top: the largest (NaN are passed over).
template <int T> struct Vec;
template <> struct Vec<DFLASH_F32> {
  static constexpr int N = 4, SIZE = 4;
  static constexpr uint32_t NONE = 0xff800000u;  // -inf
  DFL_DEV static void floats(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
  template <int M>
  DFL_DEV static float top(const uint4 (&v)[M]) {
    float m = __uint_as_float(NONE);
#pragma unroll
    for (int i = 0; i < M; ++i)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                         fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
    return m;
  }
};
template <> struct Vec<DFLASH_BF16> {
  static constexpr int N = 8, SIZE = 2;
  static constexpr uint32_t NONE = 0xff80ff80u;
  DFL_DEV static void floats(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  DFL_DEV static __nv_bfloat162 two(const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  template <int M>
  DFL_DEV static float top(const uint4 (&v)[M]) {
    __nv_bfloat162 m = __hmax2(__hmax2(two(v[0].x), two(v[0].y)), __hmax2(two(v[0].z), two(v[0].w)));
#pragma unroll
    for (int i = 1; i < M; ++i)
      m = __hmax2(m, __hmax2(__hmax2(two(v[i].x), two(v[i].y)), __hmax2(two(v[i].z), two(v[i].w))));
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
};
template <> struct Vec<DFLASH_F16> {
  static constexpr int N = 8, SIZE = 2;
  static constexpr uint32_t NONE = 0xfc00fc00u;
  DFL_DEV static void floats(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  DFL_DEV static __half2 two(const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); }
  template <int M>
  DFL_DEV static float top(const uint4 (&v)[M]) {
    __half2 m = __hmax2(__hmax2(two(v[0].x), two(v[0].y)), __hmax2(two(v[0].z), two(v[0].w)));
#pragma unroll
    for (int i = 1; i < M; ++i)
      m = __hmax2(m, __hmax2(__hmax2(two(v[i].x), two(v[i].y)), __hmax2(two(v[i].z), two(v[i].w))));
    return fmaxf(__half2float(m.x), __half2float(m.y));
  }
};

// Sixteen of 32 bytes, from word W and `bits` on.
template <int W>
DFL_DEV uint4 cut(const uint32_t* w, unsigned bits) {
  return make_uint4(__funnelshift_r(w[W], w[W + 1], bits), __funnelshift_r(w[W + 1], w[W + 2], bits),
                    __funnelshift_r(w[W + 2], w[W + 3], bits), __funnelshift_r(w[W + 3], w[W + 4], bits));
}

// A row's vectors, by index, wherever the row begins.  Off a 16-byte boundary a
// vector is cut out of the two aligned ones that it lies in; at the row's ends,
// where one of those is not all the row's own, it goes value by value.
template <int T, bool ALIGNED>
struct Row {
  const char* data;
  int vocab;
  // vectors [1, inner()) lie inside
  DFL_DEV int inner() const { return vocab / Vec<T>::N - 1; }
  DFL_DEV uint4 load_inner(int i) const {
    const char* at = data + (long long)i * 16;
    if (ALIGNED) return __ldg(reinterpret_cast<const uint4*>(at));
    const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(data) & 15);
    const uint4* a = reinterpret_cast<const uint4*>(at - shift);
    const uint4 x = __ldg(a);
    if (shift == 0) return x;
    const uint4 y = __ldg(a + 1);
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    switch (shift >> 2) {  // the same for the whole row
      case 0: return cut<0>(w, (shift & 3) * 8);
      case 1: return cut<1>(w, (shift & 3) * 8);
      case 2: return cut<2>(w, (shift & 3) * 8);
      default: return cut<3>(w, (shift & 3) * 8);
    }
  }
  DFL_DEV uint4 load_end(int i) const {
    constexpr int N = Vec<T>::N, SIZE = Vec<T>::SIZE;
    const char* at = data + (long long)i * 16;
    const int left = vocab - i * N;  // values from here on
    uint32_t w[4] = {Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (j >= left) break;
      if (SIZE == 4) {
        w[j] = *reinterpret_cast<const uint32_t*>(at + 4 * j);
      } else {
        const uint32_t h = *reinterpret_cast<const uint16_t*>(at + 2 * j);
        w[j >> 1] = j & 1 ? (w[j >> 1] & 0xffffu) | h << 16 : (w[j >> 1] & 0xffff0000u) | h;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  DFL_DEV uint4 load(int i) const { return i > 0 && i < inner() ? load_inner(i) : load_end(i); }
};

// Groups whose maxima bound the n-th largest: enough for about n to 1.4 n values
// to reach the bound (G ln(G / (G - n)) of independent ones), no more, since each
// group is compared with all.
DFL_DEV int groups_for(int n) { return n <= 24 ? 64 : n <= 64 ? 128 : 256; }

DFL_DEV float pow2_or_0(float e) {  // 2^e for whole e <= 0, 0 where it is too small to matter
  return e < -120.0f ? 0.0f : __uint_as_float((uint32_t)(127 + (int)e) << 23);
}

template <int T, bool ALIGNED>
#ifndef BEAM_MINB
#define BEAM_MINB 4
#endif
__global__ void __launch_bounds__(SCAN_THREADS, BEAM_MINB) k_beam_scan(const BeamParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int WARPS = SCAN_THREADS / 32;
  const float INF = __uint_as_float(0x7f800000u);
  __shared__ float top_of[SEGMENTS * SCAN_THREADS];  // threads' largest logits of a part's quarters
  __shared__ float group_top[SCAN_THREADS];
  __shared__ float warp_top[WARPS], warp_q[WARPS];
  __shared__ unsigned long long total;
  __shared__ float bound_s;
  __shared__ uint16_t chosen[SEGMENTS * SCAN_THREADS];  // those that hold candidates
  __shared__ unsigned long long keys[KEEP], sorted[DFLASH_BEAM_MAX_N];
  __shared__ int ranks[KEEP];
  __shared__ int count_s, chosen_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  pdl_launch_dependents();
  pdl_wait();
  const float score = p.scores[row];
  if (!(score > -INF) || score == INF || (p.done && p.done[row])) return;  // no logits are asked for
  const Row<T, ALIGNED> in = {p.logits + row * p.row_bytes, p.vocab};
  const int vecs = (p.vocab + N - 1) / N;
  const int v0 = split * p.part, v1 = min(vecs, v0 + p.part);

  // ---- the sum and the largest logit
  float top = -INF, q = -1e30f;
  Pair sum2 = pair(0.0f, 0.0f);
  const Pair hi2 = pair(LOG2E_HI, LOG2E_HI), lo2 = pair(LOG2E_LO, LOG2E_LO);
  auto take = [&](auto& v) {  // some vectors
    const float m = Vec<T>::top(v);
    top = fmaxf(top, m);
    const float t = m * LOG2E_HI;
    if (t > q + 2.0f) {  // terms stay below 2^2.5
      const float to = rintf(t), f = pow2_or_0(q - to);
      sum2 = fma2(sum2, pair(f, f), pair(0.0f, 0.0f));
      q = to;
    }
    const Pair ref = pair(-q, -q);
#pragma unroll
    for (int j = 0; j < (int)(sizeof(v) / sizeof(uint4)); ++j) {
      float x[N];
      Vec<T>::floats(v[j], x);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const Pair x2 = pair(x[e], x[e + 1]);
        float a, b;
        unpair(fma2(x2, lo2, fma2(x2, hi2, ref)), a, b);
        sum2 = add2(sum2, pair(ex2(a), ex2(b)));
      }
    }
  };
  // Batches of AHEAD rounds; a round is a vector a thread.  What does not lie wholly
  // inside the row goes vector by vector: which batches do goes by their index alone.
  constexpr int BATCH = AHEAD * SCAN_THREADS;
  const int batches = (v1 - v0 + BATCH - 1) / BATCH, seg_len = (batches + SEGMENTS - 1) / SEGMENTS;
  int seg = 0, left = seg_len;  // batches to the segment's end
  auto batch_done = [&]() {
    if (--left) return;
    top_of[seg++ * SCAN_THREADS + tid] = top;
    top = -INF;
    left = seg_len;
  };
  auto ends = [&](int b) {
    for (int j = 0; j < AHEAD; ++j) {
      const int k = v0 + (b * AHEAD + j) * SCAN_THREADS + tid;
      if (k >= v1) break;
      const uint4 v[1] = {in.load(k)};
      take(v);
    }
    batch_done();
  };
  const int b1 = max(0, (min(v1, in.inner()) - v0) / BATCH);  // batches inside end here
  int b = 0;
  if (v0 == 0) ends(b++);
  if (b < b1) {
    uint4 v[AHEAD];
    auto fetch = [&]() {
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) v[j] = in.load_inner(v0 + (b * AHEAD + j) * SCAN_THREADS + tid);
    };
    fetch();
    for (;;) {
      uint4 now[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) now[j] = v[j];
      const bool more = ++b < b1;
      if (more) fetch();
      take(now);
      batch_done();
      if (!more) break;
    }
  }
  while (b < batches) ends(b++);
  for (; seg < SEGMENTS; ++seg, top = -INF) top_of[seg * SCAN_THREADS + tid] = top;
  auto whole_top = [&]() {
    float m = top_of[tid];
#pragma unroll
    for (int i = 1; i < SEGMENTS; ++i) m = fmaxf(m, top_of[i * SCAN_THREADS + tid]);
    return m;
  };
  top = whole_top();  // its own values
  float s0, s1;
  unpair(sum2, s0, s1);
  float s = s0 + s1;
  auto block_tops = [&](float a, float b) {
    for (int d = 16; d; d >>= 1) {
      a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
      b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
    }
    if (lane == 0) warp_top[warp] = a, warp_q[warp] = b;
  };
  block_tops(top, s > 0.0f ? q : -1e30f);
  if (tid == 0) total = 0, count_s = chosen_s = 0;
  const bool odd = __syncthreads_or(!(s < 1e37f));
  float part_top = warp_top[0], part_q = warp_q[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) part_top = fmaxf(part_top, warp_top[w]), part_q = fmaxf(part_q, warp_q[w]);
  // NaN, infinity, or logits whose exponent does not fit: once more, against the largest finite one
  const bool plain = !odd && (part_top == -INF || part_q > -1e30f);
  if (!plain) {
    auto clean = [&](float x) { return x <= FLT_MAX ? x : -INF; };
    bool bad = false;
    for (int i = 0; i < SEGMENTS; ++i) {
      float m = -INF;
      for (int r = i * seg_len * AHEAD; r < (i + 1) * seg_len * AHEAD; ++r) {
        const int k = v0 + r * SCAN_THREADS + tid;
        if (k >= v1) break;
        float x[N];
        Vec<T>::floats(in.load(k), x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          bad |= !(x[e] <= FLT_MAX);
          m = fmaxf(m, clean(x[e]));
        }
      }
      top_of[i * SCAN_THREADS + tid] = m;
    }
    top = whole_top();
    if (bad) flag_nan(p.status);
    __syncthreads();
    block_tops(top, 0.0f);
    __syncthreads();
    part_top = warp_top[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) part_top = fmaxf(part_top, warp_top[w]);
    s = 0.0f;
    if (part_top > -INF) {
      for (int i = v0 + tid; i < v1; i += SCAN_THREADS) {
        float x[N];
        Vec<T>::floats(in.load(i), x);
#pragma unroll
        for (int e = 0; e < N; ++e) s += expf(clean(x[e]) - part_top);
      }
    }
  }
  const float scale = plain ? pow2_or_0(q - part_q) : 1.0f;
  unsigned long long fixed = __float2ull_rn(s * scale * (float)(1ull << FIX));
  for (int d = 16; d; d >>= 1) fixed += __shfl_xor_sync(0xffffffffu, fixed, d);
  if (lane == 0 && fixed) atomicAdd(&total, fixed);

  // ---- a bound below n of the part's logits
  const int G = groups_for(p.n), per = SCAN_THREADS / G;  // threads of a group: 4, 2, 1
  float g_top = top;
  if (per >= 2) g_top = fmaxf(g_top, __shfl_xor_sync(0xffffffffu, g_top, 1));
  if (per >= 4) g_top = fmaxf(g_top, __shfl_xor_sync(0xffffffffu, g_top, 2));
  const int g = tid / per;
  if (tid % per == 0) group_top[g] = g_top;
  __syncthreads();
  int above = 0;
  for (int u = tid % per; u < G; u += per) above += group_top[u] > g_top || (group_top[u] == g_top && u < g);
  if (per >= 2) above += __shfl_xor_sync(0xffffffffu, above, 1);
  if (per >= 4) above += __shfl_xor_sync(0xffffffffu, above, 2);
  if (above == p.n - 1) bound_s = g_top;  // of one group
  __syncthreads();
  const float bound = fmaxf(bound_s, -FLT_MAX);  // -inf: no token
  if (tid == 0) {
    PartSum r = {total, part_q, part_top, plain, 0};
    p.sums[row * p.splits + split] = r;
  }

  // ---- the threads' quarters that can hold one of the n, and their logits again
  if (top >= bound)
    for (int i = 0; i < SEGMENTS; ++i)
      if (top_of[i * SCAN_THREADS + tid] >= bound) chosen[atomicAdd(&chosen_s, 1)] = (uint16_t)(i * SCAN_THREADS + tid);
  __syncthreads();
  const int n_chosen = chosen_s;
  unsigned long long least = (unsigned long long)ordered(bound) << 32;  // keys at or below are not wanted
  auto prune = [&]() {  // the n largest keys, sorted
    __syncthreads();
    const int count = count_s;
    const int width = min(SCAN_THREADS, max(32, (count + 31) & ~31)), parts = SCAN_THREADS / width;  // threads of a key
    for (int i = tid; i < count; i += SCAN_THREADS) ranks[i] = 0;
    __syncthreads();
    const int part = tid / width;
    for (int i = tid - part * width; i < count && part < parts; i += width) {
      const unsigned long long k = keys[i];
      int rank = 0;
#pragma unroll 4
      for (int j = part; j < count; j += parts) rank += keys[j] > k;
      if (rank) atomicAdd(&ranks[i], rank);
    }
    __syncthreads();
    for (int i = tid; i < count; i += SCAN_THREADS)
      if (ranks[i] < p.n) sorted[ranks[i]] = keys[i];
    __syncthreads();
    const int kept = min(count, p.n);
    for (int i = tid; i < kept; i += SCAN_THREADS) keys[i] = sorted[i];
    if (kept == p.n) least = max(least, sorted[p.n - 1]);
    if (tid == 0) count_s = kept;
    __syncthreads();
  };
  const int rounds = seg_len * AHEAD;  // of a quarter
  const int items = rounds * n_chosen;
  for (int i0 = 0; i0 < items; i0 += SCAN_THREADS) {
    const int it = i0 + tid;
    unsigned long long key[N];
    bool any = false;
#pragma unroll
    for (int e = 0; e < N; ++e) key[e] = 0;
    if (it < items) {
      const int r = it / n_chosen, c = chosen[it - r * n_chosen];
      const int i = v0 + (c / SCAN_THREADS * rounds + r) * SCAN_THREADS + c % SCAN_THREADS;
      if (i < v1) {
        float x[N];
        Vec<T>::floats(in.load(i), x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (!(x[e] >= bound && x[e] <= FLT_MAX)) continue;
          key[e] = (unsigned long long)ordered(x[e]) << 32 | (0xffffffffu - (uint32_t)(i * N + e));
          any |= key[e] > least;
        }
      }
    }
    const int pushers = __syncthreads_count(any);
    if (pushers == 0) continue;
    if (count_s + pushers * N <= KEEP) {
      __syncthreads();  // count_s is read by all
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (key[e] > least) keys[atomicAdd(&count_s, 1)] = key[e];
    } else {  // many at once: one a thread at a time, as many as fit
#pragma unroll
      for (int e = 0; e < N; ++e) {
        __syncthreads();
        if (count_s + SCAN_THREADS > KEEP) prune();  // leaves at most DFLASH_BEAM_MAX_N
        __syncthreads();
        if (key[e] > least) keys[atomicAdd(&count_s, 1)] = key[e];
      }
    }
    __syncthreads();
  }
  prune();
  unsigned long long* best = p.best + (long long)(row * p.splits + split) * p.n;
  const int kept = count_s;
  for (int i = tid; i < p.n; i += SCAN_THREADS) best[i] = i < kept ? keys[i] : 0;
}

// ------------------------------------------------------------------ the join

// The natural logarithm to about 2^-42, by the series of 2 atanh((m - 1) / (m + 1)) for m in [0.7, 1.42): a third of
// the 64-bit operations of log(), which run at a 64th of the 32-bit rate.
DFL_DEV double ln(unsigned long long v) {
  int e = 63 - __clzll((long long)v);
  double m = (double)v;  // v < 2^63: in [2^e, 2^(e + 1)], its exponent replaced below
  m = __longlong_as_double(__double_as_longlong(m) - ((long long)e << 52));
  if (m > 1.414) m *= 0.5, ++e;
  const double d = m + 1.0;
  double r = (double)(1.0f / (float)d);
  r = r * (2.0 - d * r);
  r = r * (2.0 - d * r);
  const double z = (m - 1.0) * r, w = z * z;
  double s = 1.0 / 15;
  s = s * w + 1.0 / 13;
  s = s * w + 1.0 / 11;
  s = s * w + 1.0 / 9;
  s = s * w + 1.0 / 7;
  s = s * w + 1.0 / 5;
  s = s * w + 1.0 / 3;
  s = s * w + 1.0;
  return 2.0 * z * s + e * LN2;
}

struct Cand {
  unsigned long long score;  // ordered; 0: none
  unsigned long long key;    // of the logit and token in its row
  int beam;
};
// The larger score; of equal ones the lower beam, of one beam the larger logit
// (64 bits lose what is below 2^-53 of a score), then the lower token.
DFL_DEV bool better(const Cand& a, const Cand& b) {
  return a.score > b.score || (a.score == b.score && (a.beam < b.beam || (a.beam == b.beam && a.key > b.key)));
}

__global__ void __launch_bounds__(JOIN_THREADS) k_beam_join(const BeamParams p) {
  constexpr int WARPS = JOIN_THREADS / 32;
  const float INF = __uint_as_float(0x7f800000u);
  enum { DEAD, RUNS, ENDED };
  __shared__ double base[DFLASH_BEAM_MAX], ref[DFLASH_BEAM_MAX];  // score = base + (logit - ref)
  __shared__ unsigned long long sum_of[DFLASH_BEAM_MAX];
  __shared__ float floor_of[DFLASH_BEAM_MAX];                    // logits below it do not reach the bound
  __shared__ uint8_t state[DFLASH_BEAM_MAX];
  __shared__ unsigned long long head_score[MAX_LISTS];
  __shared__ Cand group_head[JOIN_THREADS];
  __shared__ int above[JOIN_THREADS];
  __shared__ Cand bound_s;
  __shared__ uint16_t chosen[MAX_LISTS];
  __shared__ unsigned long long score_of[KEEP], key_of[KEEP];
  __shared__ uint8_t beam_of[KEEP];
  __shared__ int ranks[KEEP];
  __shared__ Cand sorted[DFLASH_BEAM_MAX_N];
  __shared__ int count_s, chosen_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
  const int S = p.splits, lists = p.beams * S;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) {
    count_s = chosen_s = 0;
    bound_s = {0, 0, DFLASH_BEAM_MAX};
  }
  above[tid] = 0;
  const unsigned long long* best = p.best + (long long)b * lists * p.n;
  // The depth at which the lists are compared: with fewer than four lists a
  // candidate asked for, deeper, so that few of the lists are above the bound.
  int depth = 1;
  while (depth < p.n && lists < 4 * ((p.n + depth - 1) / depth)) depth *= 2;
  depth = min(depth, p.n);
  const int nth = (p.n + depth - 1) / depth;
  const bool few = lists * p.n <= JOIN_THREADS / 2;  // candidates: all of them are ranked
  const unsigned long long mine_key = few && tid < lists * p.n ? best[tid] : 0;
  // the lists' best keys and those at the depth, on their way while the sums are joined
  unsigned long long head[MAX_LISTS / JOIN_THREADS], deep[MAX_LISTS / JOIN_THREADS];
#pragma unroll
  for (int i = 0; i < MAX_LISTS / JOIN_THREADS; ++i) {
    const int l = tid + i * JOIN_THREADS;
    head[i] = l < lists && !few ? best[(long long)l * p.n] : 0;  // of a beam that does not run: not looked at
    deep[i] = l < lists && !few ? best[(long long)l * p.n + depth - 1] : 0;
  }
  // ---- each beam's sum
  for (int k = warp; k < p.beams; k += WARPS) {
    const int row = b * p.beams + k;
    const float score = p.scores[row];
    PartSum a[MAX_SPLITS / 32];
#pragma unroll
    for (int i = 0; i < MAX_SPLITS / 32; ++i) {
      const int s = lane + 32 * i;
      a[i].top = -INF;
      if (s < S) a[i] = p.sums[row * S + s];
    }
    int st = DEAD;
    if (!(score <= FLT_MAX)) {
      if (lane == 0) flag_nan(p.status);
    } else if (score > -INF) {
      st = p.done && p.done[row] ? ENDED : RUNS;
    }
    double r = 0.0;
    unsigned long long sum = 0;
    if (st == RUNS) {
      float top = -INF, q = -INF;
      bool all2 = true;
#pragma unroll
      for (int i = 0; i < MAX_SPLITS / 32; ++i) {
        if (a[i].top == -INF) continue;
        top = fmaxf(top, a[i].top);
        if (a[i].base2) q = fmaxf(q, a[i].q);
        else all2 = false;
      }
      for (int d = 16; d; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, d));
      }
      all2 = __all_sync(0xffffffffu, all2);
      if (top == -INF) {
        st = DEAD;
      } else if (all2) {  // shifts to the largest reference
        r = q * LN2;
#pragma unroll
        for (int i = 0; i < MAX_SPLITS / 32; ++i)
          if (a[i].top > -INF && q - a[i].q < 63.0f) sum += a[i].sum >> (int)(q - a[i].q);
      } else {
        r = -DBL_MAX;
#pragma unroll
        for (int i = 0; i < MAX_SPLITS / 32; ++i)
          if (a[i].top > -INF) r = fmax(r, a[i].base2 ? a[i].q * LN2 : (double)a[i].top);
        for (int d = 16; d; d >>= 1) r = fmax(r, __shfl_xor_sync(0xffffffffu, r, d));
#pragma unroll
        for (int i = 0; i < MAX_SPLITS / 32; ++i)
          if (a[i].top > -INF)
            sum += (unsigned long long)((double)a[i].sum * exp((a[i].base2 ? a[i].q * LN2 : (double)a[i].top) - r));
      }
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (lane == 0) base[k] = score, ref[k] = r, sum_of[k] = sum, state[k] = (uint8_t)st, floor_of[k] = -INF;
  }
  __syncthreads();
  if (tid < p.beams && state[tid] == RUNS) base[tid] -= ln(sum_of[tid]) - FIX * LN2;
  __syncthreads();

  auto put = [&](const Cand& c) {
    const int i = atomicAdd(&count_s, 1);
    score_of[i] = c.score, key_of[i] = c.key, beam_of[i] = (uint8_t)c.beam;
  };
  auto value = [&](int k, unsigned long long key) {
    const Cand c = {ordered(base[k] + ((double)unordered((uint32_t)(key >> 32)) - ref[k])), key, k};
    return c;
  };
  if (tid < p.beams && state[tid] == ENDED) {  // one candidate, itself
    const Cand c = {ordered(base[tid]), 0xffffffffu - (uint32_t)p.done_token, tid};
    put(c);
  }
  Cand least = {0, 0, DFLASH_BEAM_MAX};  // what is not below it is wanted
  auto prune = [&]() {  // the n best, sorted
    __syncthreads();
    const int count = count_s;
    const int width = min(JOIN_THREADS, max(32, (count + 31) & ~31)), parts = JOIN_THREADS / width;  // threads of a candidate
    for (int i = tid; i < count; i += JOIN_THREADS) ranks[i] = 0;
    __syncthreads();
    const int part = tid / width;
    for (int i = tid - part * width; i < count && part < parts; i += width) {
      const unsigned long long score = score_of[i], key = key_of[i];
      const int beam = beam_of[i];
      int rank = 0;
#pragma unroll 4
      for (int j = part; j < count; j += parts) {
        const unsigned long long o = score_of[j];
        rank += o > score;
        if (o == score && j != i) rank += beam_of[j] < beam || (beam_of[j] == beam && key_of[j] > key);
      }
      if (rank) atomicAdd(&ranks[i], rank);
    }
    __syncthreads();
    for (int i = tid; i < count; i += JOIN_THREADS)
      if (ranks[i] < p.n) sorted[ranks[i]] = {score_of[i], key_of[i], beam_of[i]};
    __syncthreads();
    const int kept = min(count, p.n);
    for (int i = tid; i < kept; i += JOIN_THREADS)
      score_of[i] = sorted[i].score, key_of[i] = sorted[i].key, beam_of[i] = (uint8_t)sorted[i].beam;
    if (kept == p.n && better(sorted[p.n - 1], least)) least = sorted[p.n - 1];
    if (tid == 0) count_s = kept;
    __syncthreads();
  };

  if (few) {
    const int k = tid / (S * p.n);
    if (mine_key && state[k] == RUNS) put(value(k, mine_key));
  } else {
    // ---- a bound below n candidates: the nth largest of the lists' `depth`-th ones, in groups
    Cand mine = {0, 0, DFLASH_BEAM_MAX};
#pragma unroll
    for (int i = 0; i < MAX_LISTS / JOIN_THREADS; ++i) {
      const int l = tid + i * JOIN_THREADS, k = l / S;
      if (l >= lists) break;
      Cand c = {0, 0, DFLASH_BEAM_MAX}, d = c;
      if (state[k] == RUNS && head[i]) c = value(k, head[i]);
      if (state[k] == RUNS && deep[i]) d = value(k, deep[i]);
      head_score[l] = c.score;
      if (better(d, mine)) mine = d;
    }
    group_head[tid] = mine;
    __syncthreads();
    const int G = groups_for(nth), live = min(G, lists), parts = JOIN_THREADS / G;
    const int g = tid % G, part = tid / G;
    if (tid < G) {
      for (int u = tid + G; u < JOIN_THREADS; u += G)
        if (better(group_head[u], mine)) mine = group_head[u];
      group_head[tid] = mine;
    }
    __syncthreads();
    if (g < live) {
      const Cand c = group_head[g];
      int n = 0;
      for (int u = part; u < live; u += parts) n += better(group_head[u], c);
      if (c.score && n) atomicAdd(&above[g], n);
    }
    __syncthreads();
    if (tid < live && group_head[tid].score && above[tid] == nth - 1) bound_s = group_head[tid];
    __syncthreads();
    least = bound_s;
    if (least.score && tid < p.beams && state[tid] == RUNS) {
      const double score = unordered(least.score), lost = (fabs(score) + fabs(base[tid]) + fabs(ref[tid])) * 0x1p-50;
      const float f = (float)(score - base[tid] + ref[tid] - lost);  // below what rounds to the bound in 64 bits
      floor_of[tid] = f - fabsf(f) * 1e-6f - 1e-30f;                 // and a few last places
    }
    for (int l = tid; l < lists; l += JOIN_THREADS) {
      const unsigned long long h = head_score[l];  // equal ones are looked into
      if (h && h >= least.score) chosen[atomicAdd(&chosen_s, 1)] = (uint16_t)l;
    }
    __syncthreads();

    // ---- the candidates of the lists that reach it
    // LIST_LANES threads a list: its next entries at once, until one is below
    const int n_chosen = chosen_s;
    constexpr int ABREAST = JOIN_THREADS / LIST_LANES;
    for (int c0 = 0; c0 < n_chosen; c0 += ABREAST) {
      const int at = c0 + tid / LIST_LANES;
      const int l = at < n_chosen ? chosen[at] : 0, k = l / S;
      bool open = at < n_chosen;
      for (int e0 = 0; e0 < p.n; e0 += LIST_LANES) {
        const int e = e0 + tid % LIST_LANES;
        Cand c = {0, 0, DFLASH_BEAM_MAX};
        bool push = false;
        if (open && e < p.n) {
          const unsigned long long key = best[(long long)l * p.n + e];
          if (key && unordered((uint32_t)(key >> 32)) >= floor_of[k]) {
            c = value(k, key);
            push = !better(least, c);
          }
        }
        const unsigned some = __ballot_sync(0xffffffffu, push);
        open = open && (some >> (lane / LIST_LANES * LIST_LANES) & ((1u << LIST_LANES) - 1)) == (1u << LIST_LANES) - 1;
        const int pushers = __syncthreads_count(push);
        if (count_s + pushers > KEEP) prune();
        __syncthreads();
        if (push && !better(least, c)) put(c);
        if (!__syncthreads_or(open)) break;
      }
    }
  }
  prune();
  const int kept = count_s;
  for (int i = tid; i < p.n; i += JOIN_THREADS) {
    const bool some = i < kept;
    const long long o = (long long)b * p.n + i;
    p.scores_out[o] = some ? (float)unordered(score_of[i]) : -INF;
    p.parents[o] = some ? b * p.beams + beam_of[i] : -1;
    p.tokens[o] = some ? (int)(0xffffffffu - (uint32_t)key_of[i]) : -1;
  }
}

// ------------------------------------------------------------------ host

struct Plan {
  int splits, part;
  size_t sums, best, bytes;  // offsets
};
constexpr int MAX_VOCAB = 1 << 24;  // of a row: the fixed-point sums' range

int beam_check(int batch, int beams, int vocab, int n, int dtype) {
  if (batch < 0 || beams < 0 || vocab < 0 || n < 0 || (dtype != DFLASH_F16 && dtype != DFLASH_BF16 && dtype != DFLASH_F32))
    return DFLASH_ERR_INVALID_ARG;
  if (beams < 1 || beams > DFLASH_BEAM_MAX || n < 1 || n > DFLASH_BEAM_MAX_N || vocab < 1 || vocab > MAX_VOCAB ||
      (long long)beams * vocab > 0x7fffffffll)
    return DFLASH_ERR_SHAPE;
  return (long long)batch * beams * MAX_SPLITS > 0x7fffffffll ? DFLASH_ERR_CAPACITY : DFLASH_OK;
}

// Parts of a row: as many CTAs as run at once, none with less than half a step
// of loads.
Plan plan_of(int batch, int beams, int vocab, int n, int dtype) {
  const int per = dtype == DFLASH_F32 ? 4 : 8, vecs = (vocab + per - 1) / per;
  const long long rows = std::max(1ll, (long long)batch * beams);
  const int least = SCAN_THREADS * AHEAD / 2;
  long long splits = std::min<long long>(BEAM_SLOTS / rows, (vecs + least - 1) / least);
  splits = std::max(1ll, std::min<long long>(splits, std::min(MAX_SPLITS, MAX_LISTS / beams)));
  Plan r;
  r.part = (int)((vecs + splits - 1) / splits + SCAN_THREADS - 1) / SCAN_THREADS * SCAN_THREADS;
  r.splits = (vecs + r.part - 1) / r.part;
  r.sums = 0;
  r.best = (rows * r.splits * sizeof(PartSum) + 255) / 256 * 256;
  r.bytes = r.best + rows * r.splits * n * sizeof(unsigned long long);
  return r;
}

template <int T>
int launch_beam(const BeamParams& p, bool aligned, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * p.beams * p.splits));
  cfg.blockDim = dim3(SCAN_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (int e = cuda_status(aligned ? cudaLaunchKernelEx(&cfg, k_beam_scan<T, true>, p)
                                  : cudaLaunchKernelEx(&cfg, k_beam_scan<T, false>, p)))
    return e;
  cfg.gridDim = dim3((unsigned)p.batch);
  cfg.blockDim = dim3(JOIN_THREADS);
  return cuda_status(cudaLaunchKernelEx(&cfg, k_beam_join, p));
}

}  // namespace

extern "C" {

size_t dflash_beam_select_workspace(int32_t batch, int32_t beams, int32_t vocab, int32_t n, int32_t dtype) {
  if (beam_check(batch, beams, vocab, n, dtype) || batch == 0) return 0;
  return plan_of(batch, beams, vocab, n, dtype).bytes;
}

int dflash_beam_select(const dflash_beam_args* a, void* stream) {
  if (!a) return DFLASH_ERR_INVALID_ARG;
  if (int e = beam_check(a->batch, a->beams, a->vocab, a->n, a->dtype)) return e;
  if (a->batch == 0) return DFLASH_OK;
  if (!a->logits || !a->scores || !a->scores_out || !a->parents || !a->tokens || a->device < 0 ||
      (a->done && (a->done_token < 0 || a->done_token >= a->vocab)))
    return DFLASH_ERR_INVALID_ARG;
  const Plan plan = plan_of(a->batch, a->beams, a->vocab, a->n, a->dtype);
  if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 255) || a->workspace_bytes < (int64_t)plan.bytes)
    return DFLASH_ERR_WORKSPACE;
  const long long size = a->dtype == DFLASH_F32 ? 4 : 2, rows = (long long)a->batch * a->beams, outs = (long long)a->batch * a->n;
  uintptr_t low = reinterpret_cast<uintptr_t>(a->logits) % size;
  for (const void* w : {static_cast<const void*>(a->scores), static_cast<const void*>(a->scores_out),
                        static_cast<const void*>(a->parents), static_cast<const void*>(a->tokens),
                        static_cast<const void*>(a->status)})
    low |= reinterpret_cast<uintptr_t>(w) & 3;
  if (low) return DFLASH_ERR_INVALID_ARG;
  auto f32 = [](const float* p, long long n) { return strided_ints(reinterpret_cast<const int32_t*>(p), n); };
  const bool same = a->scores_out == a->scores && a->n == a->beams;
  if (!apart({f32(a->scores_out, outs), strided_ints(a->parents, outs), strided_ints(a->tokens, outs),
              strided_ints(reinterpret_cast<const int32_t*>(a->status), 1), strided(a->workspace, (long long)plan.bytes, {})},
             {strided(a->logits, size * a->vocab, {{size * a->row_stride, rows}}), same ? Strided() : f32(a->scores, rows),
              strided(a->done, rows, {})}))
    return DFLASH_ERR_INVALID_ARG;
  BeamParams p = {};
  p.logits = static_cast<const char*>(a->logits);
  p.row_bytes = size * a->row_stride;
  p.scores = a->scores;
  p.done = a->done;
  p.scores_out = a->scores_out;
  p.parents = a->parents;
  p.tokens = a->tokens;
  p.status = a->status;
  p.sums = reinterpret_cast<PartSum*>(static_cast<char*>(a->workspace) + plan.sums);
  p.best = reinterpret_cast<unsigned long long*>(static_cast<char*>(a->workspace) + plan.best);
  p.batch = a->batch;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.n = a->n;
  p.splits = plan.splits;
  p.part = plan.part;
  p.done_token = a->done_token;
  const bool aligned = (reinterpret_cast<uintptr_t>(a->logits) & 15) == 0 && (rows == 1 || p.row_bytes % 16 == 0);
  DeviceGuard guard(a->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->dtype == DFLASH_F32) return launch_beam<DFLASH_F32>(p, aligned, s);
  if (a->dtype == DFLASH_BF16) return launch_beam<DFLASH_BF16>(p, aligned, s);
  return launch_beam<DFLASH_F16>(p, aligned, s);
}

}  // extern "C"

// The next beams of a search: the n best of beams * vocab continuations a
// request, scored by the running score and the logarithm of the softmax.
//
// One pass over the logits, a part of a row a CTA: the sum of exp(logit -
// reference), and the largest logit of each cell, some tens of vectors that a
// thread or four neighbours take.  A second kernel, a CTA a request, joins the
// parts' sums to each beam's logarithm.  The n-th largest of some groups' cells, by
// score, bounds the n-th best continuation from below; only cells that reach the
// bound can hold one, hardly more than n, and their logits alone are read again.
//
// The order within a row is the logits' own, so equal logits tie exactly.  Between
// rows the scores are compared in 64 bits; the sums behind them are kept so that
// rows with equal logits get equal sums, whatever their alignment: which thread
// takes a logit goes by its index alone.
//
// Sums: exponents are taken to base 2 against an integer reference, so that sums
// join by shifts.  A thread's sum is two floats of 256 terms each at most, then a
// 64-bit fixed-point number, as a warp's and a row's is (floats that took all of a
// long row's 32,768 terms were off by up to 5e-4; 0.2 us of the batch below).  Logits
// that do not fit such a reference, and what is not finite, take a second pass: 3 x 32
// beams, f32, half of each row masked by the type's lowest value, 28.8 us against 21.7
// with -1e9 or -inf.
//
// Measured in graphs of six calls (bf16, 151,936 tokens).  64 requests of 8 beams,
// 156 MB: 36.5 us, 23 of them the logits' at the copy rate; the scan alone 28 to 30,
// 512 CTAs of a row each on 608 places (two or three parts a row: 39 to 42 us in all,
// an odd number of CTAs an SM costs less than the parts' ends), then 4 to 5 of join
// behind it.  One request of 4 beams 8.3 us: 3.5 of scan, 5 of join, a chain of some
// twenty dependent steps of 100 to 1,000 cycles each.  Rows at odd addresses (f16,
// 100,003 tokens, 11 x 5) 11.7 us; where memory binds, 512 x 8 rows of 50,257 tokens 147
// us, 88 with 50,256.  f32, 3 x 32 beams, n 64, 98 % masked 22.3 us, 9 of scan: three CTAs look into 80 cells of 96 vectors each (28.9 with a vector a thread
// in turns and scores at once, 24.3 with four vectors on their way, 23.8 with eight,
// which spill).
// Tried and left: the n best of every part chosen in the scan, from which the join
// chose again (the scan's ends took 7,000 cycles a part: 37 and 9.5 us, but 26.5 for
// the masked rows); one batch of loads on its way (38.3 us); 128 bits compared as one
// integer (no faster); log() (1.1 us of a join); more registers a join (80: 35.8 us for
// the batch, but 35.4 instead of 29.8 for 220 requests of 2, one CTA an SM); twice the
// cells in a join's registers (41 for the batch, 10.7 for one request) or two thirds of
// them (7 us more for the masked rows); the cells in shared memory, by asynchronous
// copies (38.0, 9.0, and 13.5 for the odd rows).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace {

constexpr int SCAN_THREADS = 256;
constexpr int SCAN_CTAS = 4;      // of an SM
constexpr int SLOTS = 152 * SCAN_CTAS;  // CTAs that run at once
constexpr int AHEAD = 4;          // vectors of a thread's batch
constexpr int FOLD = 16;          // batches of a thread whose terms a float takes: 256 of 16-bit logits, 128 of others
constexpr int MAX_SEGMENTS = 8;   // of a part, with cells of their own
constexpr int MAX_SPLITS = 32;    // parts of a row: a lane each when they are joined
constexpr int JOIN_LOG = 9, JOIN_THREADS = 1 << JOIN_LOG;
constexpr int CELL_LOADS = 6;     // of a thread of the join: four cells each, held in registers
constexpr int CELLS = 4 * CELL_LOADS * JOIN_THREADS;  // of a request
constexpr int CHOSEN = 4 * JOIN_THREADS;  // cells that are looked into at a time: a load of every thread, at least
constexpr int KEEP = 1024;        // candidates that are kept at a time

// log2(e) in two floats: their sum is off by 2^-50.
constexpr float LOG2E_HI = 1.44269502162933349609f;
constexpr float LOG2E_LO = 1.92596299112661746887e-8f;
constexpr double LN2 = 0.693147180559945309417232121458;
// Logits below it have references that fit: the rounded x * LOG2E_HI is whole and
// below 2^31, and within 92 of the logit's exponent (half of its unit, 128 there, and
// x * LOG2E_LO, 27), which a float's range holds.
constexpr float EXACT = 1.4e9f;

// A sum of exponentials: units of 2^(q - FIX).
struct Sum {
  unsigned long long v;
  int q;
};
constexpr int FIX = 34;

// What a part of a row leaves: the sum of exp(x - reference).  The reference is
// q * ln 2 if `base2`, else the part's largest logit (which is too large or too
// small for the shared exponent).
struct PartSum {
  unsigned long long sum;  // units of 2^-FIX
  int q;
  float top;               // largest logit; -inf: no tokens are offered
  int base2;
  int reserved;
};

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
  float* cells;              // [rows][splits][segments][SCAN_THREADS / quad] largest logits
  int batch, beams, vocab, n, done_token;
  int splits, part;          // parts of a row, vectors of one
  int segments, seg_len;     // of a part; batches of one
  int quad, quad_log;        // threads of a cell: a power of two up to 32
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
  DFL_DEV static float one(const char* p) { return *reinterpret_cast<const float*>(p); }
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
  DFL_DEV static float one(const char* p) { return __bfloat162float(*reinterpret_cast<const bf16*>(p)); }
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
  DFL_DEV static float one(const char* p) { return __half2float(*reinterpret_cast<const f16*>(p)); }
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
  DFL_DEV uint4 load(int i) const {  // one of those
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
  DFL_DEV float at(int token) const { return Vec<T>::one(data + (long long)token * Vec<T>::SIZE); }
};

DFL_DEV float pow2_or_0(float e) {  // 2^e for whole e <= 0, 0 where it is too small to matter
  return e < -120.0f ? 0.0f : __uint_as_float((uint32_t)(127 + (int)e) << 23);
}

DFL_DEV unsigned long long shifted(unsigned long long v, unsigned by) { return by < 64 ? v >> by : 0; }
// s * 2^q, s at or above 0: by its exponent, whatever it is.  Also 0 for an s or a q
// that a part's largest logit does not leave.
DFL_DEV Sum scaled(float s, float q) {
  const uint32_t u = __float_as_uint(s);
  if (!(s >= FLT_MIN) || fabsf(q) > 2.1e9f) return {0, INT_MIN};
  return {(unsigned long long)((u & 0x7fffffu) | 0x800000u) << (FIX - 23), (int)q + (int)(u >> 23) - 127};
}
DFL_DEV Sum joined(const Sum& a, const Sum& b) {
  const int q = max(a.q, b.q);
  return {shifted(a.v, (unsigned)q - (unsigned)a.q) + shifted(b.v, (unsigned)q - (unsigned)b.q), q};
}

template <int T, bool ALIGNED>
__global__ void __launch_bounds__(SCAN_THREADS, SCAN_CTAS) k_beam_scan(const BeamParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int WARPS = SCAN_THREADS / 32;
  constexpr int BATCH = AHEAD * SCAN_THREADS;  // vectors of AHEAD rounds; a round is a vector a thread
  const float INF = __uint_as_float(0x7f800000u);
  __shared__ uint32_t cell[MAX_SEGMENTS * SCAN_THREADS];  // the part's, in order
  __shared__ float warp_top[WARPS];
  __shared__ int warp_q[WARPS];
  __shared__ unsigned long long warp_sum[WARPS];
  __shared__ Sum held[SCAN_THREADS];  // a thread's sum but for its last terms

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / p.splits, part = blockIdx.x - row * p.splits;
  const Row<T, ALIGNED> in = {p.logits + row * p.row_bytes, p.vocab};
  const int vecs = (p.vocab + N - 1) / N, inner = in.inner();
  const int v0 = part * p.part, v1 = min(vecs, v0 + p.part), end = min(v1, inner);
  const int batches = (v1 - v0 + BATCH - 1) / BATCH;
  const int wide = SCAN_THREADS >> p.quad_log;  // cells of a segment
  const uint4 none = make_uint4(Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE, Vec<T>::NONE);
  pdl_launch_dependents();
  pdl_wait();

  // ---- the sum and the largest logits
  // Two batches are on their way at a time.  What does not lie wholly inside the
  // row is left to its ends.
  uint4 even[AHEAD], odds[AHEAD];
  int k = v0 + tid;  // of the next batch
  auto fetch = [&](uint4 (&v)[AHEAD]) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j, k += SCAN_THREADS) v[j] = k > 0 && k < end ? in.load(k) : none;
  };
  fetch(even);
  if (batches > 1) fetch(odds);
  const float score = p.scores[row];
  const bool done = p.done && p.done[row];
  if (!(score > -INF) || score == INF || done) return;  // no logits are asked for
  float top = -INF, whole = -INF, q = -1e30f;  // of the segment, of all
  Pair sum2 = pair(0.0f, 0.0f);
  const Pair hi2 = pair(LOG2E_HI, LOG2E_HI), lo2 = pair(LOG2E_LO, LOG2E_LO);
  auto see = [&](float m) {  // a maximum, before its terms
    top = fmaxf(top, m);
    const float t = m * LOG2E_HI;
    if (t > q + 2.0f) {  // terms stay below 2^2.5 (below 2^92 near EXACT)
      const float to = rintf(t), f = pow2_or_0(q - to);
      sum2 = fma2(sum2, pair(f, f), pair(0.0f, 0.0f));
      q = to;
    }
  };
  auto add = [&](float x0, float x1) {
    const Pair x2 = pair(x0, x1), ref = pair(-q, -q);
    float a, b;
    unpair(fma2(x2, lo2, fma2(x2, hi2, ref)), a, b);
    sum2 = add2(sum2, pair(ex2(a), ex2(b)));
  };
  const bool folds = batches >= FOLD;
  if (folds) held[tid] = {0, INT_MIN};
  auto fold = [&]() {
    float a, b;
    unpair(sum2, a, b);
    if (!(a + b < 1e37f)) return;  // stays what it is, and is seen below
    held[tid] = joined(held[tid], scaled(a + b, q));
    sum2 = pair(0.0f, 0.0f);
  };
  auto close = [&](int seg) {  // the segment's cells
    whole = fmaxf(whole, top);
    float m = top;
    for (int d = 1; d < p.quad; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & (p.quad - 1)) == 0) cell[seg * wide + (tid >> p.quad_log)] = ordered(m);
    top = -INF;
  };
  int seg = 0, left = p.seg_len;  // batches to the segment's end
  auto batch = [&](uint4 (&v)[AHEAD], int b) {
    see(Vec<T>::top(v));
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      float x[N];
      Vec<T>::floats(v[j], x);
#pragma unroll
      for (int e = 0; e < N; e += 2) add(x[e], x[e + 1]);
    }
    if (b + 2 < batches) fetch(v);
  };
#pragma unroll 1
  for (int b = 0; b < batches; b += 2) {
    batch(even, b);
    if (--left == 0) close(seg++), left = p.seg_len;
    if (b + 1 >= batches) break;
    batch(odds, b + 1);
    if (--left == 0) close(seg++), left = p.seg_len;
    if ((b + 2) % FOLD == 0) fold();
  }
#pragma unroll 1
  for (; seg < p.segments; ++seg) close(seg);
  __syncwarp();  // a cell is a warp's
  // the row's ends, after the rest whatever its alignment
#pragma unroll 1
  for (int i = v0 == 0 ? 0 : max(inner, v0); i < v1; i = max(inner, i + 1)) {  // three vectors at most
    if ((i - v0) % SCAN_THREADS != tid) continue;
    float x[N], m = -INF;
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = i * N + e < p.vocab ? in.at(i * N + e) : -INF;
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, x[e]);
    see(m);
#pragma unroll
    for (int e = 0; e < N; e += 2) add(x[e], x[e + 1]);
    whole = fmaxf(whole, m);
    atomicMax(&cell[(i - v0) / (p.seg_len * BATCH) * wide + (tid >> p.quad_log)], ordered(m));
  }

  // ---- joined over the block
  auto warp_max = [&](float m) {
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
  };
  auto total = [&](unsigned long long f) {
#pragma unroll
    for (int d = 16; d; d >>= 1) f += __shfl_xor_sync(0xffffffffu, f, d);
    return f;
  };
  float s, s1;
  unpair(sum2, s, s1);
  s += s1;
  const bool odd = !(s < 1e37f);
  {
    Sum mine = scaled(odd ? 0.0f : s, q);
    if (folds) mine = joined(mine, held[tid]);
    const int most = __reduce_max_sync(0xffffffffu, mine.q);
    const float m = warp_max(whole);
    const unsigned long long f = total(shifted(mine.v, (unsigned)most - (unsigned)mine.q));
    if (lane == 0) warp_top[warp] = m, warp_q[warp] = most, warp_sum[warp] = f;
  }
  const bool any_odd = __syncthreads_or(odd);
  float part_top = warp_top[0];
  int part_q = warp_q[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) part_top = fmaxf(part_top, warp_top[w]), part_q = max(part_q, warp_q[w]);
  // Threads without a logit near the part's largest may have references that do not
  // fit (masks of the type's lowest value): their sums are far below it.
  const bool plain = !any_odd && (part_top == -INF || fabsf(part_top) < EXACT);
  if (!plain) {
    // NaN, infinity, or logits whose exponent does not fit: once more, against the largest finite one
    auto clean = [&](float x) { return x <= FLT_MAX ? x : -INF; };
    __syncthreads();  // the maxima are read
    if (any_odd) {  // the cells' maxima without what is not finite
      auto each = [&](int from, int to, auto&& f) {  // this thread's logits of some rounds
#pragma unroll 1
        for (int r = from; r < to; ++r) {
          const int i = v0 + r * SCAN_THREADS + tid;
          if (i >= v1) break;
          if (i > 0 && i < inner) {
            float x[N];
            Vec<T>::floats(in.load(i), x);
#pragma unroll
            for (int e = 0; e < N; ++e) f(x[e]);
          } else {
#pragma unroll 1
            for (int token = i * N; token < min(p.vocab, (i + 1) * N); ++token) f(in.at(token));
          }
        }
      };
      bool bad = false;
      whole = -INF;
#pragma unroll 1
      for (int i = 0; i < p.segments; ++i) {
        top = -INF;
        each(i * p.seg_len * AHEAD, (i + 1) * p.seg_len * AHEAD, [&](float x) {
          bad |= !(x <= FLT_MAX);
          top = fmaxf(top, clean(x));
        });
        __syncwarp();
        close(i);
      }
      if (bad) flag_nan(p.status);
      whole = warp_max(whole);
      if (lane == 0) warp_top[warp] = whole;
      __syncthreads();
      part_top = warp_top[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) part_top = fmaxf(part_top, warp_top[w]);
    }
    part_q = 0;
    auto fixed = [](float v) { return __float2ull_rn(v * (float)(1ull << FIX)); };
    unsigned long long f = 0;
    s = 0.0f;
    k = v0 + tid;
    auto term = [&](float x) {
      const float d = clean(x) - part_top;
      s += ex2(fmaf(d, LOG2E_HI, d * LOG2E_LO));
    };
#pragma unroll 1
    for (int b = 0; b < batches && part_top > -INF; ++b) {
      fetch(even);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        float x[N];
        Vec<T>::floats(even[j], x);
#pragma unroll
        for (int e = 0; e < N; ++e) term(x[e]);
      }
      if ((b + 1) % FOLD == 0) f += fixed(s), s = 0.0f;
    }
#pragma unroll 1
    for (int i = v0 == 0 ? 0 : max(inner, v0); i < v1 && part_top > -INF; i = max(inner, i + 1)) {  // the row's ends
      if ((i - v0) % SCAN_THREADS != tid) continue;
#pragma unroll 1
      for (int token = i * N; token < min(p.vocab, (i + 1) * N); ++token) term(in.at(token));
    }
    f += fixed(s);
    __syncwarp();
    f = total(f);
    if (lane == 0) warp_sum[warp] = f, warp_q[warp] = 0;
    __syncthreads();
  }
  const long long at = row * p.splits + part;
  if (tid == 0) {
    unsigned long long sum = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      sum += shifted(warp_sum[w], (unsigned)part_q - (unsigned)warp_q[w]);
    const PartSum r = {sum, part_q, part_top, plain, 0};
    p.sums[at] = r;
  }
  float* cells = p.cells + at * (p.segments * wide);
#pragma unroll 1
  for (int i = tid; i < p.segments * wide; i += SCAN_THREADS) cells[i] = unordered(cell[i]);
}

// ------------------------------------------------------------------ the join

// The natural logarithm to 2^-27, as a sum of two floats and `e` ln 2: the series of 2 atanh(z), z = (m - 1) /
// (m + 1), m in [0.7, 1.42), with the quotient to 46 bits by error-free sums and products (Dekker, Knuth).  64-bit
// operations run at a 64th of the 32-bit rate: log() took 1.1 us of a 5 us join.
struct Log {
  float hi, lo;
  int e;
};
DFL_DEV Log ln(unsigned long long v) {  // v > 0
  int e = 63 - __clzll((long long)v);
  const unsigned long long top = v << (63 - e);                 // its 64 leading bits
  float mh = (float)(uint32_t)(top >> 40), ml = (float)(uint32_t)(top >> 16 & 0xffffffu);  // 24 and 24 more
  mh *= 0x1p-23f, ml *= 0x1p-47f;                               // [1, 2)
  if (mh > 1.414f) mh *= 0.5f, ml *= 0.5f, ++e;
  const float n = mh - 1.0f, d = mh + 1.0f, dl = (mh - (d - 1.0f)) + ml;  // n exact; d + dl = m + 1
  const float r = 1.0f / d, q = n * r;
  const float ql = ((fmaf(-q, d, n) + ml) - q * dl) * r;
  const float w = q * q;
  float s = 1.0f / 13;
  s = fmaf(s, w, 1.0f / 11);
  s = fmaf(s, w, 1.0f / 9);
  s = fmaf(s, w, 1.0f / 7);
  s = fmaf(s, w, 1.0f / 5);
  s = fmaf(s, w, 1.0f / 3);
  return {2.0f * q, 2.0f * (ql + q * (s * w)), e};
}

// A candidate: its score's order, and what goes before among equal scores: the
// lower beam, of one beam the larger logit (64 bits lose what is below 2^-53 of a
// score), then the lower token.  No two are equal.
struct __align__(16) Cand {
  unsigned long long score;  // 0: none
  unsigned long long tie;    // 63 - beam, the logit's order, 2^24 - 1 - token
};
DFL_DEV bool better(const Cand& a, const Cand& b) {  // without branches
  return (a.score > b.score) | ((a.score == b.score) & (a.tie > b.tie));
}
DFL_DEV Cand cand(double score, int beam, uint32_t logit, uint32_t token) {
  return {ordered(score), (unsigned long long)(DFLASH_BEAM_MAX - 1 - beam) << 56 | (unsigned long long)logit << 24 | (0xffffffu - token)};
}
DFL_DEV int beam_of(const Cand& c) { return DFLASH_BEAM_MAX - 1 - (int)(c.tie >> 56); }
DFL_DEV int token_of(const Cand& c) { return 0xffffff - (int)(c.tie & 0xffffffu); }

// A part's sum against the row's largest reference r, where the references are not
// all powers of two; a row's parts are in W lanes.
__device__ __noinline__ unsigned long long sum_of_any(const PartSum& part, bool some, int W, double& r) {
  const double mine = !some ? -DBL_MAX : part.base2 ? part.q * LN2 : (double)part.top;
  r = mine;
  for (int d = W >> 1; d; d >>= 1) r = fmax(r, __shfl_xor_sync(0xffffffffu, r, d));
  return some ? (unsigned long long)((double)part.sum * exp(mine - r)) : 0;
}

// Groups whose best bound the n-th best: enough for about n to 1.4 n values to
// reach the bound (G ln(G / (G - n)) of independent ones), no more, since each
// group is compared with all.
DFL_DEV int groups_for(int n) { return n <= 24 ? 64 : n <= 64 ? 128 : 256; }

// Lanes that rank one of `count` values together: a power of two, up to a warp.
DFL_DEV int rank_lanes(int count) {
  const int per = JOIN_THREADS / max(count, 1);
  return per < 2 ? 1 : min(32, 1 << (31 - __clz(per)));
}

template <int T, bool ALIGNED>
__global__ void __launch_bounds__(JOIN_THREADS, 2) k_beam_join(const BeamParams p) {
  constexpr int N = Vec<T>::N;
  const float INF = __uint_as_float(0x7f800000u);
  enum { DEAD, RUNS, ENDED };
  __shared__ double base[DFLASH_BEAM_MAX], ref[DFLASH_BEAM_MAX];  // score = base + (logit - ref)
  __shared__ float2 near_of[DFLASH_BEAM_MAX];                    // base and ref, rounded
  __shared__ float off_of[DFLASH_BEAM_MAX];                      // what the rounding of ref may be
  __shared__ float floor_of[DFLASH_BEAM_MAX];                    // logits less ref below it do not reach the bound
  __shared__ float cut_of[DFLASH_BEAM_MAX];                      // logits below it are worse than the n kept ones,
  __shared__ int limit_of[DFLASH_BEAM_MAX];                      // those at it from this token on
  __shared__ uint8_t state[DFLASH_BEAM_MAX];
  __shared__ float bound_s;
  __shared__ int2 chosen[CHOSEN];                                // first vector; beam, above the part's end
  __shared__ Cand kept[KEEP], sorted[DFLASH_BEAM_MAX_N];
  __shared__ int count_s, chosen_s;

  const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.x;
  const int S = p.splits, wide = SCAN_THREADS >> p.quad_log;
  const float per_row_cell = 1.0f / (float)(S * p.segments * wide);
  auto row_of = [&](int c) { return (int)(((float)c + 0.5f) * per_row_cell); };  // of a cell: below 2^14, half a cell from the next
  const int row_cells = S * p.segments * wide, all_cells = p.beams * row_cells;  // multiples of 8, at most CELLS
  const float4* cells = reinterpret_cast<const float4*>(p.cells + (long long)b * all_cells);
  if (tid == 0) count_s = chosen_s = 0;
  pdl_launch_dependents();
  pdl_wait();
  // the cells are on their way while the sums are joined; those of a beam that does not run are not looked at
  float4 cell[CELL_LOADS];
#pragma unroll
  for (int i = 0; i < CELL_LOADS; ++i) {
    const int c = tid + i * JOIN_THREADS;
    cell[i] = make_float4(-INF, -INF, -INF, -INF);
    if (4 * c < all_cells) cell[i] = __ldcg(cells + c);
  }

  // ---- each beam's sum, a lane a part
  const int W = S > 1 ? 1 << (32 - __clz(S - 1)) : 1;  // lanes of a beam
#pragma unroll 1
  for (int k0 = 0; k0 < p.beams; k0 += JOIN_THREADS / W) {
    const int k = k0 + tid / W, at = tid & (W - 1), row = b * p.beams + k;
    PartSum part = {};
    part.top = -INF;
    float score = -INF;
    bool done = false;
    if (k < p.beams) {
      if (at < S) part = p.sums[row * S + at];
      score = p.scores[row];
      done = p.done && p.done[row];
    }
    if (!(score <= FLT_MAX) && at == 0) flag_nan(p.status);
    const bool runs = score > -INF && score <= FLT_MAX && !done;
    const bool some = runs && part.top > -INF;  // a beam's parts hold anything only where it runs
    const unsigned group = (W == 32 ? 0xffffffffu : (1u << W) - 1) << (lane & ~(W - 1));
    const bool any = __ballot_sync(0xffffffffu, some) & group;
    const bool bare = __ballot_sync(0xffffffffu, some && !part.base2) & group;
    int q = some && part.base2 ? part.q : INT_MIN;
    for (int d = W >> 1; d; d >>= 1) q = max(q, __shfl_xor_sync(0xffffffffu, q, d));
    double r = q * LN2;
    unsigned long long sum = some ? shifted(part.sum, (unsigned)q - (unsigned)part.q) : 0;  // shifted to the largest reference
    if (__any_sync(0xffffffffu, bare)) {  // ref is then a logit, or one of the powers of two
      double r2 = 0.0;
      const unsigned long long sum2 = sum_of_any(part, some, W, r2);
      if (bare) r = r2, sum = sum2;
    }
    for (int d = W >> 1; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (k < p.beams && at == 0) {
      double c = score;
      if (any) {
        const Log l = ln(sum);
        c += (FIX - l.e) * LN2 - (double)l.hi - (double)l.lo;
      } else {
        r = 0.0;
      }
      base[k] = c;
      ref[k] = r;
      near_of[k] = make_float2((float)c, (float)r);
      off_of[k] = (float)fabs(r - (double)(float)r);
      cut_of[k] = -INF;
      limit_of[k] = INT_MAX;
      state[k] = (uint8_t)(any ? RUNS : score > -INF && score <= FLT_MAX && done ? ENDED : DEAD);
      floor_of[k] = -INF;
    }
  }
  __syncthreads();

  auto put = [&](const Cand& c) { kept[atomicAdd(&count_s, 1)] = c; };
  auto value = [&](int k, float x, int token) {
    return cand(base[k] + ((double)x - ref[k]), k, ordered(x), (uint32_t)token);
  };
  if (tid < p.beams && state[tid] == ENDED) put(cand(base[tid], tid, 0, (uint32_t)p.done_token));  // one candidate, itself

  // ---- a bound below n candidates: the n-th best of some groups' best cells, in 32
  // bits with what those may be off by taken away
  {
    auto lower = [&](int k, float x) {
      const float2 near = near_of[k];
      const float d = x - near.y, score = near.x + d;
      const float off = (fabsf(score) + fabsf(near.x) + fabsf(d)) * 0x1p-21f + 2.0f * off_of[k];  // eight roundings, and ref's
      return x > -INF ? score - off : -INF;
    };
    float* group_best = reinterpret_cast<float*>(chosen);  // not used yet
    if (all_cells <= JOIN_THREADS) {  // few: a cell each, not the best of a thread's
      if (4 * tid < all_cells) {
        const int k = row_of(4 * tid);
        const bool runs = state[k] == RUNS;
        const float x[4] = {cell[0].x, cell[0].y, cell[0].z, cell[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) group_best[4 * tid + j] = runs ? lower(k, x[j]) : -INF;
      }
      if (tid >= all_cells) group_best[tid] = -INF;
    } else {
      float best = -INF;
#pragma unroll
      for (int i = 0; i < CELL_LOADS; ++i) {
        const int c = 4 * (tid + i * JOIN_THREADS), k = row_of(c);
        if (c >= all_cells || state[k] != RUNS) continue;
        best = fmaxf(best, lower(k, fmaxf(fmaxf(cell[i].x, cell[i].y), fmaxf(cell[i].z, cell[i].w))));
      }
      group_best[tid] = best;
    }
    __syncthreads();
    // a group's members: threads G apart, a little more from one to the next, so
    // that short rows, which begin alike, fall into different groups
    const int G = groups_for(p.n), lanes = JOIN_THREADS / G, g = tid / lanes, nth = tid % lanes;
    float m = group_best[nth * G + ((g + 11 * nth) & (G - 1))];
    for (int d = lanes >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    __syncthreads();
    if (tid % lanes == 0) group_best[g] = m;
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int u = tid % lanes; u < G; u += lanes) {
      const float o = group_best[u];
      above += (o > m) | ((o == m) & (u < g));
    }
    for (int d = lanes >> 1; d; d >>= 1) above += __shfl_xor_sync(0xffffffffu, above, d);
    if (above == p.n - 1 && tid % lanes == 0) bound_s = m;  // of one group; -inf: there are not as many
    __syncthreads();
  }
  if (tid < p.beams && state[tid] == RUNS) {
    const float2 near = near_of[tid];
    const float d = bound_s - near.x;
    floor_of[tid] = bound_s > -INF && fabsf(near.x) <= FLT_MAX
                        ? d - (fabsf(bound_s) + fabsf(near.x) + fabsf(d)) * 0x1p-21f - 2.0f * off_of[tid] : -INF;
  }
  Cand least = {0, 0};  // what is not below it is wanted
  __syncthreads();

  auto ranked = [&](int count, auto&& f) {  // every candidate with its rank
    const int lanes = rank_lanes(count), at = tid & (lanes - 1);
#pragma unroll 1
    for (int i0 = 0; i0 < count; i0 += JOIN_THREADS / lanes) {
      const int i = i0 + tid / lanes;
      if (i0 + (tid & ~31) / lanes >= count) break;  // a warp without any
      const Cand c = kept[min(i, count - 1)];
      int rank = 0;
#pragma unroll 4
      for (int j = at; j < count; j += lanes) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&kept[j]);
        rank += better({o.x, o.y}, c);
      }
      for (int d = lanes >> 1; d; d >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, d);
      if (at == 0 && i < count && rank < p.n) f(c, rank);
    }
  };
  auto prune = [&]() {  // to the n best
    const int count = count_s;
    ranked(count, [&](const Cand& c, int rank) { sorted[rank] = c; });
    __syncthreads();
    const int left = min(count, p.n);
#pragma unroll 1
    for (int i = tid; i < left; i += JOIN_THREADS) kept[i] = sorted[i];
    if (left == p.n && better(sorted[p.n - 1], least)) least = sorted[p.n - 1];
    if (tid == 0) count_s = left;
    __syncthreads();
  };

  // Whether a logit, or a cell's largest, may be one of the n.
  auto may_be = [&](int k, float x) { return x - near_of[k].y >= floor_of[k] && x >= -FLT_MAX && x <= FLT_MAX; };
  // Behind a prune: each beam's lowest logit that goes before the last of the kept
  // ones (in the last one's own beam the logit itself, up to its token), so that
  // thousands of equal ones are passed over by a comparison.
  auto cut = [&]() {
    if (least.score && tid < p.beams && state[tid] == RUNS) {
      const int of = beam_of(least);
      auto before = [&](float x) {
        const unsigned long long s = ordered(base[tid] + ((double)x - ref[tid]));
        return s > least.score || (s == least.score && tid < of);
      };
      float x = (float)(unordered(least.score) - base[tid] + ref[tid]);
      int left = 64;  // steps; it is a place or two away
      limit_of[tid] = INT_MAX;
      if (tid == of) {
        cut_of[tid] = unordered((uint32_t)(least.tie >> 24));
        limit_of[tid] = token_of(least);
      } else if (before(x)) {
        float below = nextafterf(x, -INF);
        while (left-- && before(below)) x = below, below = nextafterf(x, -INF);
        cut_of[tid] = left < 0 ? -INF : x;
      } else {
        while (left-- && !before(x)) x = nextafterf(x, INF);
        cut_of[tid] = x;  // what is below is known to be worse
      }
    }
    __syncthreads();
  };

  // ---- the cells that reach it, and their logits
  const int rounds = p.seg_len * AHEAD, cell_vecs = rounds << p.quad_log;
  const int vecs = (p.vocab + N - 1) / N;
  unsigned hits = 0;  // of this thread's cells
#pragma unroll
  for (int i = 0; i < CELL_LOADS; ++i) {
    const int c = 4 * (tid + i * JOIN_THREADS), k = row_of(c);
    if (c >= all_cells || state[k] != RUNS) continue;
    hits |= (may_be(k, cell[i].x) | may_be(k, cell[i].y) << 1 | may_be(k, cell[i].z) << 2 | may_be(k, cell[i].w) << 3) << 4 * i;
  }
  auto choose = [&](unsigned h) {  // false: there was no room
    if (h == 0) return true;
    int o = atomicAdd(&chosen_s, __popc(h));
    if (o + __popc(h) > CHOSEN) return false;
#pragma unroll 1
    for (; h; h &= h - 1) {
      const int bit = __ffs(h) - 1, c = 4 * (tid + (bit >> 2) * JOIN_THREADS) + (bit & 3);
      const int k = row_of(c), at = c - k * row_cells;  // beam, cell of its row
      const int seg = at / wide, part = seg / p.segments;   // segment of the row, part
      const int first = part * p.part + (seg - part * p.segments) * rounds * SCAN_THREADS + ((at - seg * wide) << p.quad_log);
      chosen[o++] = make_int2(first, k << 25 | min(vecs, (part + 1) * p.part));
    }
    return true;
  };
  auto vector_of = [&](int first, int nth) {  // of a cell: its nth
    return first + (nth >> p.quad_log) * SCAN_THREADS + (nth & (p.quad - 1));
  };
  const int before = count_s;
  // A vector's tokens that are not below the floor; at an end of the row all of them.
  auto wanted_of = [&](const Row<T, ALIGNED>& in, int i, bool inside, const uint4& v, float ref_x, float least_d) {
    unsigned w = 0;
    if (inside) {
      float x[N];
      Vec<T>::floats(v, x);
#pragma unroll
      for (int e = 0; e < N; ++e) w |= (x[e] - ref_x >= least_d) << e;
    } else {
      w = (1u << min(N, p.vocab - i * N)) - 1;
    }
    return w;
  };
  // Into the chosen cells.  False: more was wanted than is kept.
  auto look = [&]() {
    const int cells_n = chosen_s, items = cells_n * cell_vecs;
    bool full = false;
    if (items <= JOIN_THREADS) {  // a vector each: 0.3 us less than teams would take
      const int o = tid / cell_vecs;
      if (o < cells_n) {
        const int2 c = chosen[o];
        const int k = c.y >> 25, v1 = c.y & 0x1ffffff, i = vector_of(c.x, tid - o * cell_vecs);
        const Row<T, ALIGNED> in = {p.logits + (b * p.beams + k) * p.row_bytes, p.vocab};
        const bool inside = i > 0 && i < min(v1, in.inner());
        uint4 v = {};
        if (inside) v = in.load(i);
        unsigned wanted = i < v1 ? wanted_of(in, i, inside, v, near_of[k].y, floor_of[k]) : 0;
#pragma unroll 1
        for (; wanted; wanted &= wanted - 1) {
          const int token = i * N + __ffs(wanted) - 1;
          const float x = in.at(token);
          if (!may_be(k, x)) continue;
          const Cand r = value(k, x, token);
          const int to = atomicAdd(&count_s, 1);
          if (to < KEEP) kept[to] = r;
          else full = true;
        }
      }
      return !__syncthreads_or(full);
    }
    // A team of threads a cell, LOOKS vectors of a thread on their way at once.  The
    // scores wait for the end, a thread each: a 64-bit sum takes some 400 cycles.
    constexpr int LOOKS = ALIGNED ? 6 : 4;
    const int least_log = min(4, 32 - __clz(cell_vecs - 1));
    const int team_log = max(least_log, JOIN_LOG - (32 - __clz(cells_n - 1)));
    const int team = 1 << team_log, at = tid & (team - 1);
#pragma unroll 1
    for (int o = tid >> team_log; o < cells_n && !full; o += JOIN_THREADS >> team_log) {
      const int2 c = chosen[o];
      const int k = c.y >> 25, v1 = c.y & 0x1ffffff;
      const Row<T, ALIGNED> in = {p.logits + (b * p.beams + k) * p.row_bytes, p.vocab};
      const int inner = min(v1, in.inner());
      const float ref_x = near_of[k].y, least_d = floor_of[k];
#pragma unroll 1
      for (int nth = at; nth < cell_vecs && !full; nth += team * LOOKS) {
        uint4 v[LOOKS][1];
#pragma unroll
        for (int u = 0; u < LOOKS; ++u) {
          const int i = vector_of(c.x, nth + u * team);
          if (nth + u * team < cell_vecs && i > 0 && i < inner) v[u][0] = in.load(i);
        }
        unsigned hits = 0;  // vectors that may hold one; those at the row's ends are gone through
#pragma unroll
        for (int u = 0; u < LOOKS; ++u) {
          const int i = vector_of(c.x, nth + u * team);
          const bool inside = i > 0 && i < inner;
          if (nth + u * team < cell_vecs && i < v1) hits |= (!inside || Vec<T>::top(v[u]) - ref_x >= least_d) << u;
        }
#pragma unroll 1
        for (; hits; hits &= hits - 1) {
          const int i = vector_of(c.x, nth + (__ffs(hits) - 1) * team);
          const bool inside = i > 0 && i < inner;
          uint4 again = {};
          if (inside) again = in.load(i);
#pragma unroll 1
          for (unsigned wanted = wanted_of(in, i, inside, again, ref_x, least_d); wanted; wanted &= wanted - 1) {
            const int token = i * N + __ffs(wanted) - 1;
            const float x = in.at(token);
            if (!may_be(k, x)) continue;
            const int to = atomicAdd(&count_s, 1);
            if (to < KEEP) kept[to] = {__float_as_uint(x), (unsigned long long)k << 32 | (unsigned)token};
            else full = true;
          }
        }
      }
    }
    if (__syncthreads_or(full)) return false;
#pragma unroll 1
    for (int i = before + tid; i < count_s; i += JOIN_THREADS) {
      const Cand raw = kept[i];
      kept[i] = value((int)(raw.tie >> 32), __uint_as_float((uint32_t)raw.score), (int)(uint32_t)raw.tie);
    }
    __syncthreads();
    return true;
  };
  // The same, however many are wanted: a token of each thread in turns, pruned
  // between them.
  auto look_in_turns = [&]() {
    const int items = chosen_s * cell_vecs;
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += JOIN_THREADS) {
      int k = 0, first = 0, count = 0;  // of a vector: beam, token, tokens
      if (i0 + tid < items) {
        const int o = (i0 + tid) / cell_vecs;
        const int2 c = chosen[o];
        const int i = vector_of(c.x, i0 + tid - o * cell_vecs);
        k = c.y >> 25;
        first = i * N;
        if (i < (c.y & 0x1ffffff)) count = min(N, p.vocab - first);
      }
      const Row<T, ALIGNED> in = {p.logits + (b * p.beams + k) * p.row_bytes, p.vocab};
#pragma unroll 1
      for (int e = 0; e < N; ++e) {
        const int token = first + e;
        const float x = e < count ? in.at(token) : -INF;
        const bool wanted = may_be(k, x) && (x > cut_of[k] || (x == cut_of[k] && token < limit_of[k]));
        const int pushers = __syncthreads_count(wanted);
        if (pushers == 0) continue;
        if (count_s + pushers > KEEP / 2) {  // leaves at most DFLASH_BEAM_MAX_N; looked at by all before it is changed
          prune();
          cut();
        }
        __syncthreads();
        if (wanted) {
          const Cand c = value(k, x, token);
          if (!better(least, c)) put(c);
        }
        __syncthreads();
      }
    }
  };
  // All of them at once; or, where there is no room for the cells or for what they
  // hold, a load of every thread at a time, in turns.
  const bool room = choose(hits);
  if (__syncthreads_or(!room) || !look()) {
#pragma unroll 1
    for (int i = 0; i < CELL_LOADS; ++i) {
      __syncthreads();
      if (tid == 0) {
        chosen_s = 0;
        if (i == 0) count_s = before;
      }
      __syncthreads();
      choose(hits & 15u << 4 * i);
      __syncthreads();
      look_in_turns();
    }
  }

  // ---- the n best, sorted
  const int count = count_s;
  const long long o = (long long)b * p.n;
  ranked(count, [&](const Cand& c, int rank) {
    p.scores_out[o + rank] = (float)unordered(c.score);
    p.parents[o + rank] = b * p.beams + beam_of(c);
    p.tokens[o + rank] = token_of(c);
  });
  for (int i = count + tid; i < p.n; i += JOIN_THREADS) p.scores_out[o + i] = -INF, p.parents[o + i] = p.tokens[o + i] = -1;
}

// ------------------------------------------------------------------ host

struct Plan {
  int splits, part, segments, seg_len, quad, quad_log;
  size_t cells, bytes;  // offset of the cells; of the sums: 0
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

// Parts of a row: together no more CTAs than run at once, none with less than half a
// batch.  From 305 rows on a row is one part, and from 609 on the last ones run behind
// the others (80 x 8 beams of 151,936 tokens 48 us, 64 x 8 of them 36.5).
// Cells: a thread's in up to MAX_SEGMENTS segments, but no more of a request than
// the join holds: fewer segments, then more threads a cell.  That fits: 608 parts of
// 256 / 32 cells, or 64 of one part each.
Plan plan_of(int batch, int beams, int vocab, int dtype) {
  const int per = dtype == DFLASH_F32 ? 4 : 8, vecs = (vocab + per - 1) / per;
  const long long rows = std::max(1ll, (long long)batch * beams);
  const int least = SCAN_THREADS * AHEAD / 2;
  long long splits = std::min<long long>(SLOTS / rows, (vecs + least - 1) / least);
  splits = std::max(1ll, std::min<long long>(splits, MAX_SPLITS));
  Plan r;
  r.part = (int)((vecs + splits - 1) / splits + SCAN_THREADS - 1) / SCAN_THREADS * SCAN_THREADS;
  r.splits = (vecs + r.part - 1) / r.part;
  const int batches = (r.part + SCAN_THREADS * AHEAD - 1) / (SCAN_THREADS * AHEAD);
  r.segments = std::min(MAX_SEGMENTS, batches);
  r.quad = 1, r.quad_log = 0;
  auto cells = [&]() { return (long long)beams * r.splits * r.segments * (SCAN_THREADS / r.quad); };
  while (r.segments > 1 && cells() > CELLS) r.segments = (r.segments + 1) / 2;
  while (r.quad < 32 && cells() > CELLS) r.quad *= 2, ++r.quad_log;
  r.seg_len = (batches + r.segments - 1) / r.segments;
  r.segments = (batches + r.seg_len - 1) / r.seg_len;
  r.cells = (rows * r.splits * sizeof(PartSum) + 255) / 256 * 256;
  r.bytes = r.cells + rows * r.splits * r.segments * (SCAN_THREADS / r.quad) * sizeof(float);
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
  return cuda_status(aligned ? cudaLaunchKernelEx(&cfg, k_beam_join<T, true>, p)
                             : cudaLaunchKernelEx(&cfg, k_beam_join<T, false>, p));
}

}  // namespace

extern "C" {

size_t dflash_beam_select_workspace(int32_t batch, int32_t beams, int32_t vocab, int32_t n, int32_t dtype) {
  if (beam_check(batch, beams, vocab, n, dtype) || batch == 0) return 0;
  return plan_of(batch, beams, vocab, dtype).bytes;
}

int dflash_beam_select(const dflash_beam_args* a, void* stream) {
  if (!a) return DFLASH_ERR_INVALID_ARG;
  if (int e = beam_check(a->batch, a->beams, a->vocab, a->n, a->dtype)) return e;
  if (a->batch == 0) return DFLASH_OK;
  if (!a->logits || !a->scores || !a->scores_out || !a->parents || !a->tokens || a->device < 0 ||
      (a->done && (a->done_token < 0 || a->done_token >= a->vocab)))
    return DFLASH_ERR_INVALID_ARG;
  const Plan plan = plan_of(a->batch, a->beams, a->vocab, a->dtype);
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
  p.sums = static_cast<PartSum*>(a->workspace);
  p.cells = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + plan.cells);
  p.batch = a->batch;
  p.beams = a->beams;
  p.vocab = a->vocab;
  p.n = a->n;
  p.splits = plan.splits;
  p.part = plan.part;
  p.segments = plan.segments;
  p.seg_len = plan.seg_len;
  p.quad = plan.quad;
  p.quad_log = plan.quad_log;
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

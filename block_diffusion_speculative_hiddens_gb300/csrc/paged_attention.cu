// Attention of a ragged batch of new tokens over a caller's paged cache, on
// the 5th-generation tensor cores.
//
// The rows of one KV head -- its G query heads of consecutive tokens -- share
// its keys, so they are packed into M tiles of 128 rows (tok = 128 / G tokens
// each).  An item is one or two (NM) M tiles of one sequence and KV head; its
// work is the 128-key tiles its rows see.  All items' tiles, in order
// (sequence, token tile, KV head), are cut into equal runs, one for each CTA
// of a persistent grid: a batch of ragged single tokens, one verify block over
// a long context and a prompt all load the SMs evenly.  A run that covers
// only part of an item leaves its share (O unnormalised, running maximum and
// sum, float32) in the workspace, and k_paged_merge joins the shares in order.
// Few items over little cache take a cluster of CTAs each instead, which join
// their shares over distributed shared memory (see plan_call).
//
// Per key tile and M tile:
//   S = Q K^T   tcgen05.mma M=128 x N=128 keys x K=D, operands in shared memory,
//   softmax     one row a thread, S read from TMEM twice (maximum, then
//               weights; log2 domain) against a running reference that moves
//               only when a tile's maximum exceeds it by more than 2^8 (then
//               the row's O is rescaled in TMEM): P is the same softmax up to a
//               power of two that the sum shares, and stays inside f16.  P is
//               rounded to the operands' 16 bits, as the tensor core takes it;
//               maxima, sums and O are float32.  Outputs are then 0.0022 of
//               their size from the 64-bit result in bf16 and 0.00028 in f16,
//               where the output's own rounding alone gives 0.0017 and 0.0002.
//   O += P V    tcgen05.mma with P as the TMEM A operand (over the S it came
//               from) and V as it lies in the cache (N-major).
// The tensor core runs one thread's MMAs in issue order, so S of the next tile
// may overwrite the P that the O MMA before it read.
// Warps: 4 NM softmax, one issuing MMAs, one loading.
//
// Bounds and measurements (GB300; 32 query and 8 KV heads of 128, bf16; replayed
// in a graph from idle, near the highest clock: among other calls the clock falls
// and the chunk takes 724 to 743 us, the whole prompt 385):
// - One token each for 64 requests of 512 to 4,096 positions reads 605 MB in
//   100 us (6.0 TB/s, 0.89 of the copy rate); the runs themselves keep 0.95,
//   finding them, the first load and the merge take 9 us.
// - A chunk of 2,048 over 30,001 positions is 1.04 PFLOP in 641 us (1.62
//   PFLOP/s, 0.84 of the cuBLAS burst rate); a whole prompt of 8,192 360 us.  A
//   tile's two S and O MMAs are 2,048 cycles, and a tile takes 2,800: what a
//   row's softmax takes from S to P, and the hand-overs between it, the
//   issuing warp and the tensor core, which leave that idle in between (tensor
//   pipe 0.74, issue slots 0.40).
// - The same chunk at 64 wide 480 us, a tile 2,300 cycles: S runs a tile ahead
//   there (537 without), and what is left is the softmax's own instructions in
//   sequence (issue slots 0.51, exponentials 0.45, tensor pipe 0.45).
// - Without any exponential the chunks take 648 (for 662 in that run) and 466 us;
//   one in four by a polynomial of degree 3 instead 712 and 587.
// - What moved it (chunk, us): softmax in short loops over TMEM 904 -> 733, one
//   elect.sync a tile, counted ring places 730 -> 708, 64 columns of S in
//   flight 708 -> 688 (first pass) and 666 -> 641 (second), warp-uniform values
//   told to the compiler 689 -> 662.
// - Measured and not kept: two threads a row (16 softmax warps, 96 registers:
//   859 for 729), an issuing warp for each M tile (their MMAs interleave and both
//   end late: 868), the row in registers over both passes (645 for 641, but
//   whole prompts 382 for 360: what spills costs at every item's end), MMAs
//   issued by one lane (793 for 728), Q double-buffered with a ring of three
//   tiles (826 for 716).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace {

constexpr int KT = 128;  // keys of a tile
constexpr int MAX_BATCH = 8192;  // sequences of a call
constexpr float LOG2E = 1.4426950408889634f;
// What an item costs beside its tiles, in tiles: the load of Q, the first and
// last tile that overlap nothing, the output.  Measured with 1, 2 and 3 (us):
// a prompt of 8,192 428 / 357 / 358, a window of 1,024 146 / 142 / 142, ragged
// prompts of 64-wide heads 61.4 / 57.9 / 59.7; NM = 1 with 0, 1 and 2: blocks
// of 24 requests 16.2 / 14.8 / 14.6, a token each for 64 103.5 / 102.7 / 103.4.
template <int NM>
constexpr int SETUP = NM == 2 ? 2 : 1;

struct PagedParams {
  uint16_t* out;
  long long o_row, o_head;
  int wide_out;       // rows of out are 32-byte aligned
  float* lse;
  long long lse_row, lse_head;
  const int* table;
  long long table_stride;
  int max_pages, n_pages, shift;
  int cap;            // positions a table row can hold
  const int* cu;
  const int* ctx;
  const int* kv_len;
  int rows, batch, hkv, group, causal, window;
  int tok;            // tokens of an M tile
  float scale_log2;   // > 0
  int negate;         // the caller's scale is negative
  uint32_t* status;
  char* ws;
  int cs;             // > 0: a cluster of cs CTAs an item, its shares joined over distributed shared memory
};

// Workspace: a header, one record a CTA, two partial slots a CTA.
// The cost of all items in runs of `each`, the first `more` of them one longer.
struct Runs {
  long long each;
  int more, ctas;
};
DFL_DEV long long run_start(const Runs& r, int c) { return r.each * c + min(c, r.more); }
struct WsCta {
  int at, cost;        // of the item its run begins in: cost before the run, cost of the item
  int row0, rows, head;  // the item's first row of q, its rows x heads, its first head
  int pad[3];
};
constexpr size_t ws_records(int grid) { return 256 + ((size_t)grid * sizeof(WsCta) + 255) / 256 * 256; }
// One slot: O [D/4][rows] float4, running maxima [rows], sums [rows].
constexpr size_t ws_slot_floats(int rows, int D) { return (size_t)rows * (D + 2); }  // a multiple of 4

// The MMAs of a whole tile under one elect.sync: with one for each MMA the
// issuing warp is what the tensor core waits for.
// S = Q K^T, K = D: both operands in 64-dim panels 16 KB apart, 16 dims = 32 bytes a step.
template <int D>
DFL_DEV void tc_mma_s(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  if constexpr (D == 128)
    asm volatile(
          "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
          "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
          "add.s64 a, %1, 0;\n\tadd.s64 b, %2, 0;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
          "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 1024;\n\tadd.s64 b, %2, 1024;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 1026;\n\tadd.s64 b, %2, 1026;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 1028;\n\tadd.s64 b, %2, 1028;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 1030;\n\tadd.s64 b, %2, 1030;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(0u)
        : "memory");
  else
    asm volatile(
          "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
          "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
          "add.s64 a, %1, 0;\n\tadd.s64 b, %2, 0;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
          "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
          "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t}" ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(0u)
        : "memory");
}
// O (+)= P V, K = 128 keys: P in TMEM, 8 columns a step, V 16 keys = 2 KB a step.
DFL_DEV void tc_mma_o(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
          "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 c;\n\t"
          "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
          "add.u32 c, %1, 0;\n\tadd.s64 b, %2, 0;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, p;\n\t"
          "add.u32 c, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 32;\n\tadd.s64 b, %2, 512;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 40;\n\tadd.s64 b, %2, 640;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 48;\n\tadd.s64 b, %2, 768;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t"
          "add.u32 c, %1, 56;\n\tadd.s64 b, %2, 896;\n\t"
          "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [c], b, %3, t;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}

template <int D, int NM>
struct PCfg {
  static constexpr int ROWS = 128 * NM;
  static constexpr int PANEL = 128 * 128;            // 128 rows x 64 dims
  static constexpr int TILE = (D / 64) * PANEL;      // Q of an M tile, K or V of a key tile
  // Q of the next item lands beside this one's where there is room for both
  static constexpr int QBUFS = D == 128 && NM == 2 ? 1 : 2;
  static constexpr int SLOTS = D == 64 ? 10 : NM == 2 ? 4 : 5;  // NM = 2: a fifth made nothing faster
  static constexpr int OFF_RING = QBUFS * NM * TILE;
  static constexpr int OFF_BAR = OFF_RING + SLOTS * TILE;
  static constexpr int OFF_ITEM = OFF_BAR + 576;     // the loading warp's notes of the next items
  static constexpr int SMEM = 1024 + OFF_ITEM + 128;  // + 1024 for aligning the base
  static constexpr int THREADS = 128 * NM + 64;
  // S buffers of 128 columns.  AHEAD: one more than M tiles, taken in turn in
  // issue order, so that S of an M tile's next key tile is there when the
  // softmax of this one ends.  Two 128-wide O leave no room for it: there each M
  // tile has its buffer, and S follows the O MMA whose P it overwrites.
  static constexpr int S_BUFS = D == 64 && NM == 2 ? 3 : 2;
  static constexpr bool AHEAD = S_BUFS > NM;
  static constexpr int S_COL = 0;
  static constexpr int O_COL = 128 * S_BUFS;
  static constexpr uint32_t TMEM_COLS = 512;
};

template <bool BF16>
DFL_DEV uint32_t pack16(float a, float b) {
  if constexpr (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    return pack_f16x2(a, b);
  }
}

// The rest of a bounded wait that has not succeeded at once; out of line, since
// the kernel's code is fetched by warps in several places of it at once.
static __device__ __noinline__ bool wait_rest(uint64_t* bar, uint32_t par, uint32_t* status) {
  bool aborted = false;
  return mbar_wait(bar, par, status, &aborted);
}

// A value that is the same in every lane, told to the compiler: addresses and
// loop bounds made of it need no code for lanes that differ.
DFL_DEV int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

DFL_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

DFL_DEV float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two float32 in one register pair.
DFL_DEV uint64_t pack_u32x2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
DFL_DEV uint64_t pack_f32x2(float lo, float hi) { return pack_u32x2(__float_as_uint(lo), __float_as_uint(hi)); }
DFL_DEV void unpack_f32x2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
DFL_DEV uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
DFL_DEV uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The n lowest bits (n outside 0..32: none, all).
DFL_DEV uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// 32 bytes to a 32-byte aligned address.
DFL_DEV void st_global_32(void* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

DFL_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
DFL_DEV void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 32 columns of this thread's TMEM lane; the registers are valid after tmem_wait_ld().
DFL_DEV void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
DFL_DEV void tmem_st16_nowait(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
DFL_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor of an N-major operand (V: rows of keys, 64 dims =
// 128 bytes each, 128-byte swizzle): 64-dim panels PANEL bytes apart (leading
// offset), groups of 8 keys 1024 bytes apart (stride offset).
DFL_DEV uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// A place in the ring of tiles: slot and phase.
template <int SLOTS>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  DFL_DEV void next() {
    if (++s == SLOTS) s = 0, phase ^= 1u;
  }
};

// A sequence as the kernel sees it; lengths outside the batch's rows or the
// table are cut to them.
struct Seq {
  int row0, n;        // rows of q
  long long ctx;
  int kv;             // keys
};
DFL_DEV Seq load_seq(const PagedParams& p, int b) {
  Seq s;
  const int lo = min(max(p.cu[b], 0), p.rows), hi = min(max(p.cu[b + 1], lo), p.rows);
  s.row0 = lo;
  s.n = hi - lo;
  s.ctx = p.ctx[b];
  const long long kv = p.kv_len ? (long long)p.kv_len[b] : s.ctx + s.n;
  s.kv = (int)min(max(kv, 0ll), (long long)p.cap);
  return s;
}
// The keys [lo, hi) that any of the tokens [t0, t1) sees, and the key tiles over them.
struct Span {
  int lo, hi, tile0, tiles;
};
DFL_DEV Span load_span(const PagedParams& p, const Seq& s, int t0, int t1) {
  Span r;
  r.lo = p.window > 0 ? (int)min(max(s.ctx + t0 - p.window + 1, 0ll), (long long)s.kv) : 0;
  r.hi = p.causal ? (int)min(max(s.ctx + t1, 0ll), (long long)s.kv) : s.kv;
  r.tile0 = r.lo / KT;
  r.tiles = r.hi > r.lo ? (r.hi + KT - 1) / KT - r.tile0 : 0;
  return r;
}

// A CTA's run through the items.  An item's cost is SETUP, then one a tile.
struct Walk {
  int b, mt, kvh, at;  // the item and the part of its cost that lies before this CTA's run
  long long left;      // cost still to come
  Seq s;
  Span span;
  int t0, t1;          // the item's tokens
  int off, n;          // this CTA's tiles of the item
  bool out;            // it has something to write: tiles, or the zeros of an item without any
};
template <int NM>
DFL_DEV void walk_item(const PagedParams& p, Walk& w) {
  w.t0 = w.mt * p.tok * NM;
  w.t1 = min(w.t0 + p.tok * NM, w.s.n);
  w.span = load_span(p, w.s, w.t0, w.t1);
  const int end = (int)min((long long)(SETUP<NM> + w.span.tiles), w.at + w.left);
  w.off = max(w.at - SETUP<NM>, 0);
  w.n = max(end - SETUP<NM>, 0) - w.off;
  w.out = w.n > 0 || (w.span.tiles == 0 && w.at == 0);
}
template <int NM>
DFL_DEV bool walk_next(const PagedParams& p, Walk& w) {
  w.left -= SETUP<NM> + w.span.tiles - w.at;
  if (w.left <= 0) return false;
  w.at = 0;
  if (++w.kvh == p.hkv) {
    w.kvh = 0;
    ++w.mt;
    if (w.mt * p.tok * NM >= w.s.n) {
      w.mt = 0;
      do {
        if (++w.b >= p.batch) return false;
        w.s = load_seq(p, w.b);
      } while (w.s.n == 0);
    }
  }
  walk_item<NM>(p, w);
  return true;
}

// Inclusive sum over the CTA in thread order; *total receives the whole.
// `part`: one value a warp.
DFL_DEV long long cta_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // the last use of part is over
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) before += part[i];
    all += part[i];
  }
  *total = all;
  return v + before;
}

// A segment as the issuing and the softmax warps need it: written by the
// loading warp, which is ahead of them, since each working it out from its own
// place in the run costs a microsecond between two items.
struct Item {
  int tiles;   // this CTA's key tiles (0: its rows get zeros; -1: no more items)
  int key0;    // first key of the first of them
  int row0;    // first row of q
  int tokens;
  int pos0;    // position of the first token
  int kv;      // keys of the sequence
  int kvh;
  int share;   // 0: all of the item's tiles; 1: its first ones, 2: later ones
};
constexpr int ITEMS = 4;  // noted ahead, at most

struct Sched {
  long long part[16];
  int b, mt, cost;
  long long before;  // cost before the pair (b, mt)
};

// Where this CTA's run begins.  Pairs (sequence, token tile) are counted and
// weighed by the whole CTA, blockDim.x at a time; the tile area, free until
// the loads begin, holds the sequences (`seqs`, as long as each thread has one
// at most) and their first pairs (`first` [batch + 1]).  False: no work at
// all, or none for this CTA.
template <int NM>
DFL_DEV bool locate(const PagedParams& p, Sched* sc, Seq* seqs, int* first, Walk& w, Runs* runs) {
  const int per = p.tok * NM;
  const bool kept = p.batch <= (int)blockDim.x;
  long long pairs = 0, total = 0, all;
  int b = 0, mt = 0, u = 0;  // this thread's pair and its cost
  long long incl = 0;
  bool once = kept;  // one round over the pairs
  auto weigh = [&](int pair, int* b_out, int* mt_out) {
    int lo = 0, hi = p.batch - 1;  // the last sequence whose first pair is not behind
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= pair) lo = mid;
      else hi = mid - 1;
    }
    const Seq s = kept ? seqs[lo] : load_seq(p, lo);
    const int mt = pair - first[lo], t0 = mt * per;
    *b_out = lo;
    *mt_out = mt;
    return SETUP<NM> + load_span(p, s, t0, min(t0 + per, s.n)).tiles;
  };
  bool alone = false;  // each sequence has one pair at most, and a thread
  if (kept) {
    const bool in = (int)threadIdx.x < p.batch;
    Seq s = {0, 0, 0, 0};
    if (in) {
      s = load_seq(p, threadIdx.x);
      seqs[threadIdx.x] = s;
    }
    alone = !__syncthreads_or(s.n > per);
    if (alone) {
      b = threadIdx.x;
      u = s.n > 0 ? SETUP<NM> + load_span(p, s, 0, s.n).tiles : 0;
      pairs = p.batch;
      incl = cta_scan((long long)u * p.hkv, sc->part, &total);
    }
  }
  if (!alone) {
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
      const int bb = b0 + threadIdx.x;
      const int m = bb < p.batch ? ((kept ? seqs[bb].n : load_seq(p, bb).n) + per - 1) / per : 0;
      const long long at = cta_scan(m, sc->part, &all);
      if (bb < p.batch) first[bb] = (int)(pairs + at - m);
      pairs += all;
    }
    __syncthreads();
    once = pairs <= blockDim.x;
    for (long long p0 = 0; p0 < pairs; p0 += blockDim.x) {
      const long long pair = p0 + threadIdx.x;
      u = pair < pairs ? weigh((int)pair, &b, &mt) : 0;
      incl = cta_scan((long long)u * p.hkv, sc->part, &all);
      total += all;
    }
  }
  if (total == 0) return false;
  runs->ctas = (int)min((long long)gridDim.x, total);
  if (total < (1ll << 31)) {  // a 64-bit division takes a hundred cycles more
    runs->each = (uint32_t)total / (uint32_t)runs->ctas;
    runs->more = (int)((uint32_t)total % (uint32_t)runs->ctas);
  } else {
    runs->each = total / runs->ctas;
    runs->more = (int)(total % runs->ctas);
  }
  if ((int)blockIdx.x >= runs->ctas) return false;
  const long long u0 = run_start(*runs, blockIdx.x), u1 = run_start(*runs, blockIdx.x + 1);
  long long base = 0;
  for (long long p0 = 0; p0 < pairs; p0 += blockDim.x) {
    if (!once) {
      const long long pair = p0 + threadIdx.x;
      u = pair < pairs ? weigh((int)pair, &b, &mt) : 0;
      incl = base + cta_scan((long long)u * p.hkv, sc->part, &all);
      base += all;
    }
    if (u > 0 && incl > u0 && incl - (long long)u * p.hkv <= u0) {
      sc->b = b;
      sc->mt = mt;
      sc->cost = u;
      sc->before = incl - (long long)u * p.hkv;
    }
    if (!once && base > u0) break;  // uniform: base is the CTA's
  }
  __syncthreads();
  const long long in = u0 - sc->before;
  w.b = sc->b;
  w.mt = sc->mt;
  w.kvh = in < (1ll << 31) ? (int)((uint32_t)in / (uint32_t)sc->cost) : (int)(in / sc->cost);
  w.at = (int)(in - (long long)w.kvh * sc->cost);
  w.left = u1 - u0;
  w.s = kept ? seqs[w.b] : load_seq(p, w.b);
  walk_item<NM>(p, w);
  return true;
}

// The item of this CTA's cluster and its share of the item's tiles.
DFL_DEV bool locate_cluster(const PagedParams& p, Sched* sc, Walk& w) {
  const int item = blockIdx.x / p.cs, rank = blockIdx.x - item * p.cs;
  int pair = item / p.hkv;
  w.kvh = item - pair * p.hkv;
  w.b = 0;
  if (p.batch > 1) {
    int before = 0;
    if (threadIdx.x == 0) sc->b = -1;
    for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
      const int b = b0 + threadIdx.x;
      const int m = b < p.batch ? (load_seq(p, b).n + p.tok - 1) / p.tok : 0;
      long long all;
      const int at = before + (int)cta_scan(m, sc->part, &all);  // its barriers order the write above
      if (pair < at && pair >= at - m) {
        sc->b = b;
        sc->mt = pair - (at - m);
      }
      before += (int)all;
    }
    __syncthreads();
    if (sc->b < 0) return false;
    w.b = sc->b;
    pair = sc->mt;
  }
  w.mt = pair;
  w.s = load_seq(p, w.b);
  w.t0 = w.mt * p.tok;
  w.t1 = min(w.t0 + p.tok, w.s.n);
  if (w.t0 >= w.t1) return false;
  w.span = load_span(p, w.s, w.t0, w.t1);
  w.off = (int)((long long)w.span.tiles * rank / p.cs);
  w.n = (int)((long long)w.span.tiles * (rank + 1) / p.cs) - w.off;
  w.out = w.n > 0;
  w.at = 0;
  w.left = 0;  // and nothing after it
  return true;
}

// Joins the shares that the CTAs of a cluster left in their shared memory:
// O [128][D + 4] unnormalised, maxima [128], sums [128].  Each takes every
// cs-th row; a thread has the loads of CS shares of PIECES of 4 columns in flight.
constexpr int MAX_CLUSTER = 16;
constexpr long long CLUSTER_TILES = 640;  // key tiles that a call's tables can hold
template <bool BF16, int D, int CS, int PIECES>
DFL_DEV void join_cluster(const PagedParams& p, const uint8_t* sm, int row0, int rows, int head0) {
  constexpr int PS = D + 4;
  const uint32_t at = smem_u32(sm);
  const int rank = (int)cluster_ctarank();
  const int all = (rows - rank + p.cs - 1) / p.cs * (D / 4);
  for (int e0 = threadIdx.x; e0 < all; e0 += PIECES * blockDim.x) {
    float m[PIECES][CS], l[PIECES][CS];
    float4 o[PIECES][CS];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int e = min(e0 + i * (int)blockDim.x, all - 1);
      const int r = rank + e / (D / 4) * p.cs, d = e % (D / 4) * 4;
#pragma unroll
      for (int x = 0; x < CS; ++x) {
        m[i][x] = -INFINITY;
        l[i][x] = 0.f;
        o[i][x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < p.cs) {
          const uint32_t a = dsmem_addr(at, (uint32_t)x);
          m[i][x] = ld_dsmem(a + 4u * (uint32_t)(128 * PS + r));
          l[i][x] = ld_dsmem(a + 4u * (uint32_t)(128 * PS + 128 + r));
          o[i][x] = ld_dsmem4(a + 4u * (uint32_t)(r * PS + d));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int e = e0 + i * (int)blockDim.x;
      if (e >= all) break;
      const int r = rank + e / (D / 4) * p.cs, d = e % (D / 4) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int x = 0; x < CS; ++x)
        if (l[i][x] != 0.f) M = fmaxf(M, m[i][x]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < CS; ++x) {
        if (l[i][x] == 0.f) continue;  // a share without a key of the row
        const float wgt = ex2(m[i][x] - M);
        L += wgt * l[i][x];
        acc.x += wgt * o[i][x].x;
        acc.y += wgt * o[i][x].y;
        acc.z += wgt * o[i][x].z;
        acc.w += wgt * o[i][x].w;
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const long long t = row0 + r / p.group, h = head0 + r % p.group;
      *reinterpret_cast<uint2*>(p.out + t * p.o_row + h * p.o_head + d) =
          make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
      if (p.lse && d == 0)
        p.lse[t * p.lse_row + h * p.lse_head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
  }
}

template <bool BF16, int D, int NM>
__global__ void __launch_bounds__(PCfg<D, NM>::THREADS, 1)
    k_paged_attn(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const PagedParams p) {
  using C = PCfg<D, NM>;
  extern __shared__ __align__(128) uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint64_t* full = bars;                // [SLOTS] tile landed
  uint64_t* empty = full + C::SLOTS;    // [SLOTS] tile's MMAs done
  uint64_t* s_full = empty + C::SLOTS;  // [2 m + i & 1] S i of M tile m (and every MMA before it) done
  uint64_t* p_full = s_full + 4;        // [2] P written: of M tile m, or (NM = 1) of tiles of one parity
  uint64_t* o_done = p_full + 2;        // [2] an O MMA done, likewise
  uint64_t* o_empty = o_done + 2;       // [2] O read out
  uint64_t* q_full = o_empty + 2;       // [QBUFS]
  uint64_t* q_empty = q_full + 2;
  uint64_t* mdone = q_empty + 2;
  uint64_t* item_full = mdone + 1;      // [ITEMS]
  uint64_t* item_empty = item_full + ITEMS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_empty + ITEMS);
  Sched* sched = reinterpret_cast<Sched*>(sm + C::OFF_BAR + 384);
  Item* items = reinterpret_cast<Item*>(sm + C::OFF_ITEM);
  static_assert((2 * C::SLOTS + 15 + 2 * ITEMS) * 8 + 8 <= 384 && sizeof(Sched) <= 192 && sizeof(Item) * ITEMS == 128,
                "barrier area");
  static_assert(C::THREADS * sizeof(Seq) + (MAX_BATCH + 1) * sizeof(int) <= C::OFF_BAR, "tile area");

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  constexpr int MMA_WARP = 4 * NM, LOAD_WARP = 4 * NM + 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 2 * i, 1);
      mbar_init(s_full + 2 * i + 1, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
      mbar_init(o_empty + i, 4);
    }
    for (int i = 0; i < C::QBUFS; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    mbar_init(mdone, 1);
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, 4 * NM + 1);
    }
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == LOAD_WARP && lane == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  pdl_launch_dependents();
  pdl_wait();

  Walk w;
  Runs runs = {0, 0, 0};
  Seq* seqs = reinterpret_cast<Seq*>(sm);
  const bool in_cluster = NM == 1 && p.cs > 0;
  const bool work = in_cluster ? locate_cluster(p, sched, w)
                               : locate<NM>(p, sched, seqs, reinterpret_cast<int*>(seqs + C::THREADS), w, &runs);
  if (threadIdx.x == 0 && !in_cluster) {
    if (blockIdx.x == 0) *reinterpret_cast<Runs*>(p.ws) = runs;
    if (work) {
      WsCta* rec = reinterpret_cast<WsCta*>(p.ws + 256) + blockIdx.x;
      rec->at = w.at;
      rec->cost = SETUP<NM> + w.span.tiles;
      rec->row0 = w.s.row0 + w.t0;
      rec->rows = (w.t1 - w.t0) * p.group;
      rec->head = w.kvh * p.group;
    }
  }
  fence_proxy_async_smem();  // the sequences were written and read before the loads land over them
  __syncthreads();
  bool aborted = false;
  auto wait_all = [&](uint64_t* bar, uint32_t par) {  // warp-uniform
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
    if (aborted || !__all_sync(0xffffffffu, wait_rest(bar, par, p.status))) aborted = true;
    return !aborted;
  };
  // The next item, for a warp that takes them in turn; false after the last.
  auto next_item = [&](int& taken, Item& x) {
    const int i = taken % ITEMS;
    if (!wait_all(item_full + i, (uint32_t)((taken / ITEMS) & 1))) return false;
    ++taken;
    x = items[i];
    x.tiles = uniform(x.tiles);
    x.key0 = uniform(x.key0);
    x.tokens = uniform(x.tokens);
    x.kv = uniform(x.kv);
    if (lane == 0) mbar_arrive(item_empty + i);
    return x.tiles >= 0;
  };
  if (!work) {
    // nothing for this CTA
  } else if (warp == LOAD_WARP) {
    // ------------------------------------------------ loads
    // A thread has only a few copies in flight at a time, so every box of a
    // tile has a lane of its own: `boxes` pages (or one part of a page) of
    // each 64-dim panel.
    const int page = 1 << p.shift, box = min(page, KT), boxes = KT / box;
    const int bi = lane % boxes, bh = lane / boxes;  // this lane's box, if bh is a panel
    int seg = 0;
    int noted = 0;     // items
    Ring<C::SLOTS> at;
    bool lap = false;  // the ring has been filled once
    bool ok = true;
    auto note = [&](const Item& x) {
      const int i = noted % ITEMS;
      if (noted >= ITEMS && !wait_all(item_empty + i, (uint32_t)((noted / ITEMS - 1) & 1))) return false;
      if (lane == 0) {
        items[i] = x;
        mbar_arrive(item_full + i);
      }
      ++noted;
      return true;
    };
    do {
      const int tiles = uniform(w.n);
      if (!w.out && !in_cluster) continue;
      const int far = 0x7ff00000;  // farther than any key, and a tile's tokens more still fit
      if (!(ok = note({tiles, (w.span.tile0 + w.off) * KT, w.s.row0 + w.t0, w.t1 - w.t0,
                       (int)min(max(w.s.ctx + w.t0, -(long long)far), (long long)far), w.s.kv, w.kvh,
                       tiles == w.span.tiles ? 0 : w.off == 0 ? 1 : 2})))
        break;
      // also of an item without a tile: its window may lie past what the table holds
      if (lane == 0 && (p.kv_len ? (long long)p.kv_len[w.b] : w.s.ctx + w.s.n) > p.cap)
        dev_error(p.status, DFLASH_DEV_PAGE);
      if (tiles == 0) continue;
      auto load_q = [&] {
        const int qb = seg % C::QBUFS;
        if (seg >= C::QBUFS && !wait_all(q_empty + qb, (uint32_t)((seg / C::QBUFS - 1) & 1))) return false;
        const int nm = NM == 2 && w.t0 + p.tok < w.t1 ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(q_full + qb, (uint32_t)(nm * (D / 64) * p.tok * p.group * 128));
        __syncwarp();
        const int m = lane / (D / 64), h = lane % (D / 64);
        if (m < nm)
          tma_load_3d(sm + (qb * NM + m) * C::TILE + h * C::PANEL, &qmap, q_full + qb, 64 * h, w.kvh * p.group,
                      w.s.row0 + w.t0 + m * p.tok);
        ++seg;
        return true;
      };
      if (C::QBUFS == 2 && !load_q()) break;
      const int* row = p.table + w.b * p.table_stride;
      const int first_page = w.span.lo >> p.shift, end_page = (w.span.hi + page - 1) >> p.shift;
      int base = -64, ids = 0;  // lanes hold 32 entries of the table row from `base` on
      for (int j = 0; j < tiles && ok; ++j) {
        const int key0 = (w.span.tile0 + w.off + j) * KT;
        const int e0 = key0 >> p.shift;
        if (e0 < base || e0 + boxes > base + 32) {
          base = e0;
          const int e = base + lane;
          ids = p.n_pages;  // not read: a box behind the pool lands as zeros
          if (e >= first_page && e < end_page) {
            const int id = row[e];
            if (id >= 0 && id < p.n_pages) ids = id;
            else dev_error(p.status, DFLASH_DEV_PAGE);
          }
        }
        const int id = __shfl_sync(0xffffffffu, ids, e0 + bi - base);
        for (int kv = 0; kv < 2; ++kv) {  // K, then V
          const int s = at.s;
          if (lap && !wait_all(empty + s, at.phase ^ 1u)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full + s, C::TILE);
          __syncwarp();
          if (bh < D / 64)
            tma_load_4d(sm + C::OFF_RING + s * C::TILE + bh * C::PANEL + bi * box * 128, kv ? &vmap : &kmap, full + s,
                        64 * bh, page > KT ? key0 & (page - 1) : 0, w.kvh, id);
          at.next();
          lap = lap || at.s == 0;
        }
        // one Q buffer: its load waits for the last item's S, the first tiles do not
        if (C::QBUFS == 1 && j == 0 && ok) ok = load_q();
      }
    } while (ok && walk_next<NM>(p, w));
    if (ok) note({-1, 0, 0, 0, 0, 0, 0, 0});
    // every copy lands before the CTA may exit
    for (int i = lap ? 0 : C::SLOTS - at.s; i < C::SLOTS; ++i) {  // from the oldest slot on
      const int s = lap ? (at.s + i) % C::SLOTS : i - (C::SLOTS - at.s);
      wait_rest(full + s, s < at.s ? at.phase : at.phase ^ 1u, p.status);
    }
    for (int i = seg > C::QBUFS ? seg - C::QBUFS : 0; i < seg; ++i) {
      wait_rest(q_full + i % C::QBUFS, (uint32_t)((i / C::QBUFS) & 1), p.status);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------ MMA issue (converged warp, one elected lane)
    // This warp's scalar work between two MMAs is what the tensor core waits
    // for: slots and phases are counted, not divided out, and descriptors added up.
    const uint32_t idesc_s = idesc_f16_f32(128, KT, BF16 ? 1 : 0);
    const uint32_t idesc_o = idesc_f16_f32(128, D, BF16 ? 1 : 0) | (1u << 16);  // V is N-major
    const uint64_t q_desc = sdesc_sw128(smem_u32(sm)), k_desc = sdesc_sw128(smem_u32(sm + C::OFF_RING));
    const uint64_t v_desc = sdesc_sw128_mn(smem_u32(sm + C::OFF_RING), C::PANEL);
    int seg = 0;
    Ring<C::SLOTS> kr, vr;  // the next tile of K and of V
    vr.next();
    int sb = 0, pb = 0;          // S buffer of the next S and of the next P
    uint32_t s_odd = 0;          // bit m: parity of M tile m's next S
    uint32_t p_phase = 0;        // bit b: phase of the next P on barrier b
    int sg[2] = {0, 0};          // segments of each M tile
    bool ok = true;
    int taken = 0;
    Item x;
    while (ok && next_item(taken, x)) {
      const int tiles = x.tiles;
      if (tiles == 0) continue;
      const int nm = NM == 2 && x.tokens > p.tok ? 2 : 1;
      const int qb = seg % C::QBUFS;
      if (!wait_all(q_full + qb, (uint32_t)((seg / C::QBUFS) & 1)) || !wait_all(full + kr.s, kr.phase)) break;
      ++seg;
      tc_fence_after();
      // S of M tile m's key tile j.  The first of each M tile, and with AHEAD one
      // more, go before the first O MMA; every other follows one.
      auto issue_s = [&](int m, int j) {
        if (m == 0 && j > 0) {
          if (!wait_all(full + kr.s, kr.phase)) return false;
          tc_fence_after();
        }
        const int buf = C::AHEAD ? sb : m;
        tc_mma_s<D>(tmem + (uint32_t)(C::S_COL + 128 * buf), q_desc + (uint64_t)((qb * NM + m) * (C::TILE >> 4)),
                    k_desc + (uint64_t)(kr.s * (C::TILE >> 4)), idesc_s);
        tc_commit_elect(s_full + 2 * m + (C::AHEAD ? s_odd >> m & 1u : 0u));
        if (C::AHEAD) {
          s_odd ^= 1u << m;
          sb = sb + 1 == C::S_BUFS ? 0 : sb + 1;
        }
        if (m == nm - 1) {
          tc_commit_elect(empty + kr.s);
          kr.next();
          kr.next();
          if (j + 1 == tiles) tc_commit_elect(q_empty + qb);
        }
        return true;
      };
      for (int m = 0; m < nm; ++m) issue_s(m, 0);
      if (C::AHEAD && tiles > 1 && !(ok = issue_s(0, 1))) break;
      // keys of the sequence behind the start of its last tile, if that tile ends inside a page
      const int last_v = x.kv - x.key0 - (tiles - 1) * KT;
      for (int j = 0; j < tiles && ok; ++j) {
        if (!(ok = wait_all(full + vr.s, vr.phase))) break;
        if (j + 1 == tiles && last_v < KT && (last_v & ((1 << p.shift) - 1))) {
          // the sequence ends inside a page: what lies behind it (stale,
          // perhaps not finite) must not meet P's zeros in the MMA
          const int v1 = min(KT, ((last_v >> p.shift) + 1) << p.shift);
          uint8_t* vt = sm + C::OFF_RING + vr.s * C::TILE;
          for (int i = lane; i < (v1 - last_v) * 8; i += 32)
            for (int h = 0; h < D / 64; ++h)
              *reinterpret_cast<uint4*>(vt + h * C::PANEL + (last_v + (i >> 3)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t vd = v_desc + (uint64_t)(vr.s * (C::TILE >> 4));
        for (int m = 0; m < nm; ++m) {
          if (j == 0 && sg[m]++ > 0 && !(ok = wait_all(o_empty + m, (uint32_t)((sg[m] - 2) & 1)))) break;
          const int buf = C::AHEAD ? pb : m, bar = NM == 2 ? m : pb;
          if (!(ok = wait_all(p_full + bar, p_phase >> bar & 1u))) break;
          tc_fence_after();
          tc_mma_o(tmem + (uint32_t)(C::O_COL + D * m), tmem + (uint32_t)(C::S_COL + 128 * buf), vd, idesc_o, j > 0 ? 1u : 0u);
          p_phase ^= 1u << bar;
          if (C::AHEAD) pb = pb + 1 == C::S_BUFS ? 0 : pb + 1;
          tc_commit_elect(o_done + bar);
          if (m == nm - 1) tc_commit_elect(empty + vr.s);
          const int n = !C::AHEAD ? m : m + 1 == nm ? 0 : m + 1, nj = C::AHEAD && n == 0 ? j + 2 : j + 1;
          if (nj < tiles && !(ok = issue_s(n, nj))) break;
        }
        vr.next();
        vr.next();
      }
    }
    // every issued MMA completes before the columns are freed
    tc_commit_elect(mdone);
    wait_rest(mdone, 0, p.status);
  } else {
    // ------------------------------------------------ softmax: one row a thread
    const int m = warp >> 2;
    const int r = threadIdx.x & 127;
    const int rt = r / p.group, rh = r - rt * p.group;  // the row's token in the M tile and head in the group
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_base = lane_base + (uint32_t)(C::O_COL + D * m);
    int it = 0;  // S tiles of this M tile
    bool ok = true;
    // The O MMA of S tile i, and with it every one before.  A barrier tells
    // only whether one phase is over, so it may be neither two ahead of who
    // waits nor two behind.  NM = 2: every warp knows O i done before it gives
    // P i + 1: from S i + 1, which follows it, or, where S runs ahead, by waiting
    // each time.  NM = 1 has a barrier for each parity of P and O instead and
    // waits for O only where it moves (each time: 8,192 positions 14.8 -> 15.3 us).
    constexpr bool EACH = NM == 2 && C::AHEAD;
    auto wait_o = [&](int i) {
      return NM == 2 ? wait_all(o_done + m, (uint32_t)(i & 1)) : wait_all(o_done + (i & 1), (uint32_t)((i >> 1) & 1));
    };
    int sb0 = 0;  // S buffer of the item's first S tile
    int taken = 0;
    Item x;
    while (next_item(taken, x)) {
      const int tiles = x.tiles;
      const int tm = m * p.tok + rt;  // the row's token in the item
      const int nm = NM == 2 && x.tokens > p.tok ? 2 : 1;
      int buf = C::AHEAD ? (sb0 + m) % C::S_BUFS : m;
      sb0 = (sb0 + tiles * nm) % C::S_BUFS;
      if (m >= nm) continue;  // no row in this M tile
      const bool valid = rt < p.tok && tm < x.tokens;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // the keys this row sees; rows that do not exist mask nothing (they are not written)
      int lo = 0, hi = 1 << 30;
      if (valid) {
        const int pos = x.pos0 + tm;
        hi = p.causal ? min(max(pos + 1, 0), x.kv) : x.kv;
        lo = p.window > 0 ? (int)min(max((long long)pos - p.window + 1, 0ll), (long long)x.kv) : 0;
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < tiles; ++j, ++it) {
        if (!(ok = C::AHEAD ? wait_all(s_full + 2 * m + (it & 1), (uint32_t)(it >> 1 & 1))
                            : wait_all(s_full + 2 * m, (uint32_t)(it & 1))))
          break;
        tc_fence_after();
        const uint32_t s_base = lane_base + (uint32_t)(C::S_COL + 128 * buf);
        if (C::AHEAD) buf = buf + nm < C::S_BUFS ? buf + nm : buf + nm - C::S_BUFS;
        if (warp_valid) {
          const int key0 = x.key0 + j * KT;
          const int h = hi - key0, l = lo - key0;
          uint32_t sx[32], sy[32];
          if (p.negate || __any_sync(0xffffffffu, h < KT || l > 0)) {
            // S as the two passes below want it: its sign turned, -inf where the row does not see
            auto edit = [&](uint32_t* v, int c) {
              const uint32_t seen = low_bits(h - c) & ~low_bits(l - c);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (p.negate) v[k] ^= 0x80000000u;
                if (!(seen & (1u << k))) v[k] = 0xff800000u;
              }
              tmem_st16_nowait(s_base + c, v);
              tmem_st16_nowait(s_base + c + 16, v + 16);
            };
#pragma unroll 1
            for (int c = 0; c < KT; c += 64) {
              tmem_ld32_nowait(s_base + c, sx);
              tmem_ld32_nowait(s_base + c + 32, sy);
              tmem_wait_ld();
              edit(sx, c);
              edit(sy, c + 32);
            }
            tmem_wait_st();
          }
          // Both passes read S from TMEM, 64 columns at a time and ahead of the arithmetic.
          float mx = -INFINITY;
          {
            float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
            auto take = [&](const uint32_t* v) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                m0 = max3(m0, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                m1 = max3(m1, __uint_as_float(v[k + 2]), __uint_as_float(v[k + 3]));
                m2 = max3(m2, __uint_as_float(v[k + 4]), __uint_as_float(v[k + 5]));
                m3 = max3(m3, __uint_as_float(v[k + 6]), __uint_as_float(v[k + 7]));
              }
            };
            tmem_ld32_nowait(s_base, sx);
            tmem_ld32_nowait(s_base + 32, sy);
            tmem_wait_ld();
            take(sx);
            tmem_ld32_nowait(s_base + 64, sx);
            take(sy);
            tmem_ld32_nowait(s_base + 96, sy);
            tmem_wait_ld();
            take(sx);
            tmem_ld32_nowait(s_base, sx);
            take(sy);
            mx = max3(fmaxf(m0, m1), m2, m3) * p.scale_log2;
          }
          if (EACH && !(ok = wait_o(it - 1))) break;
          const bool move = mx > m_run + 8.f;
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mx : m_run;
            if (j > 0) {  // O of the tiles before is against m_run
              if (NM == 1 && !(ok = wait_o(it - 1))) break;
              tc_fence_after();
              const float alpha = move ? ex2(m_run - m_new) : 1.f;
              tmem_wait_ld();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                float o[16];
                tmem_ld16(o_base + c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= alpha;
                tmem_st16(o_base + c, o);
              }
              l_run *= alpha;
            }
            m_run = m_new;
          }
          const float ref = m_run == -INFINITY ? 0.f : -m_run;  // a row that has seen no key yet adds 0
          const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2), ref2 = pack_f32x2(ref, ref);
          uint64_t sum0 = 0, sum1 = 0;  // pairs of partial sums
          auto weigh = [&](const uint32_t* v, int c) {  // 32 columns of S into 16 of P
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const uint64_t f = fma_f32x2(pack_u32x2(v[k], v[k + 1]), scale2, ref2);
              const uint64_t g = fma_f32x2(pack_u32x2(v[k + 2], v[k + 3]), scale2, ref2);
              float a, b, d, e;
              unpack_f32x2(f, a, b);
              unpack_f32x2(g, d, e);
              a = ex2(a);
              b = ex2(b);
              d = ex2(d);
              e = ex2(e);
              sum0 = add_f32x2(sum0, pack_f32x2(a, b));
              sum1 = add_f32x2(sum1, pack_f32x2(d, e));
              pk[k / 2] = pack16<BF16>(a, b);
              pk[k / 2 + 1] = pack16<BF16>(d, e);
            }
            tmem_st16_nowait(s_base + c / 2, pk);
          };
          tmem_ld32_nowait(s_base + 32, sy);
          tmem_wait_ld();
          weigh(sx, 0);
          tmem_ld32_nowait(s_base + 64, sx);
          weigh(sy, 32);
          tmem_ld32_nowait(s_base + 96, sy);
          tmem_wait_ld();
          weigh(sx, 64);
          weigh(sy, 96);
          float a, b;
          unpack_f32x2(add_f32x2(sum0, sum1), a, b);
          l_run += a + b;
          tmem_wait_st();
        } else if (EACH && !(ok = wait_o(it - 1))) {
          break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + (NM == 2 ? m : it & 1));
      }
      if (!ok) break;
      // the segment's O
      if (tiles > 0) {
        if (!(ok = wait_o(it - 1))) break;
        tc_fence_after();
      }
      const bool to_cluster = NM == 1 && p.cs > 1, whole = x.share == 0 && !to_cluster;
      if (warp_valid || to_cluster) {
        // where the row's O goes: out, this CTA's share in the workspace, or
        // (the tile area being free: every load has been used) in shared memory
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        const int head = x.kvh * p.group + rh;
        const long long qrow = x.row0 + tm;
        uint16_t* dst = p.out + qrow * p.o_row + head * p.o_head;
        const int row = m * 128 + r, stride = to_cluster ? 1 : C::ROWS;  // of the share's float4 columns
        float* share = reinterpret_cast<float*>(p.ws + ws_records(gridDim.x)) +
                       (2 * (size_t)blockIdx.x + (x.share == 1)) * ws_slot_floats(C::ROWS, D);
        float4* part = reinterpret_cast<float4*>(to_cluster ? reinterpret_cast<float*>(sm) + r * (D + 4) : share + 4 * row);
#pragma unroll 1  // once an item: a longer loop waits on instruction fetch
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (tiles > 0) {
            tmem_ld32_nowait(o_base + c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!whole && (valid || to_cluster)) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              part[(c / 4 + e) * stride] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                       __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
          if (whole && valid) {
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              y[e] = pack16<BF16>(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            if (p.wide_out) {  // a row a thread: whole 32-byte sectors, half the store instructions
              st_global_32(dst + c, y);
              st_global_32(dst + c + 16, y + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(dst + c + 8 * e) = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
            }
          }
        }
        if (to_cluster) {  // without a tile: a share without keys
          float* ml = reinterpret_cast<float*>(sm) + 128 * (D + 4);
          ml[r] = m_run;
          ml[128 + r] = l_run;
        } else if (valid && !whole) {
          share[(size_t)C::ROWS * D + row] = m_run;
          share[(size_t)C::ROWS * (D + 1) + row] = l_run;
        } else if (valid && p.lse) {
          p.lse[qrow * p.lse_row + head * p.lse_head] =
              l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
        }
      }
      if (tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty + m);
      }
    }
  }
  tc_fence_before();
  __syncthreads();  // every MMA and TMEM read done, every tile landed
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (NM == 1 && p.cs > 1 && work) {  // the whole cluster's answer
    cluster_sync_all();
    const int row0 = w.s.row0 + w.t0, rows = (w.t1 - w.t0) * p.group, head0 = w.kvh * p.group;
    if (p.cs <= 4) join_cluster<BF16, D, 4, 4>(p, sm, row0, rows, head0);
    else join_cluster<BF16, D, MAX_CLUSTER, 1>(p, sm, row0, rows, head0);
    cluster_sync_all();  // this CTA's share is there until every other has read it
  }
}

// Joins the shares of the items that more than one CTA worked on.  CTA x is
// the boundary between runs x and x + 1; the first boundary inside an item
// joins it, in the order of the runs.  One thread takes 4 columns of a row.
constexpr int MERGE_ROWS = 8, MERGE_AHEAD = 16;

template <bool BF16, int D, int NM>
__global__ void __launch_bounds__(MERGE_ROWS * D / 4) k_paged_merge(const PagedParams p, int grid) {
  constexpr int ROWS = 128 * NM;
  extern __shared__ float merge_sm[];
  float(*wm)[MERGE_ROWS] = reinterpret_cast<float(*)[MERGE_ROWS]>(merge_sm);  // [grid]
  float(*wl)[MERGE_ROWS] = wm + grid;
  __shared__ float red[D / 4][MERGE_ROWS];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x + 1;
  const Runs runs = *reinterpret_cast<const Runs*>(p.ws);
  const WsCta rec = reinterpret_cast<const WsCta*>(p.ws + 256)[c];  // its bytes exist for every c < grid
  if (c >= runs.ctas || rec.at <= SETUP<NM>) return;                // the run begins with the item's first tile
  const long long item0 = run_start(runs, c) - rec.at, item1 = item0 + rec.cost;
  if (run_start(runs, c - 1) > item0 + SETUP<NM>) return;  // an earlier boundary joins this item
  int n = 2;                                               // runs c - 1 .. c - 2 + n hold a share
  while (c - 1 + n < runs.ctas && run_start(runs, c - 1 + n) < item1) ++n;
  const int per = p.tok * p.group;  // rows of an M tile
  constexpr size_t SF = ws_slot_floats(ROWS, D);
  const float* parts = reinterpret_cast<const float*>(p.ws + ws_records(grid)) + 2 * (size_t)(c - 1) * SF;
  auto share = [&](int x) { return (2 * (size_t)x + (x == 0 ? 1 : 0)) * SF; };
  const int i = threadIdx.x % MERGE_ROWS, d4 = threadIdx.x / MERGE_ROWS;
  // this CTA's rows, MERGE_ROWS at a time
  for (int r0 = blockIdx.y * MERGE_ROWS; r0 < rec.rows; r0 += gridDim.y * MERGE_ROWS) {
    const int ri = min(r0 + i, rec.rows - 1), mi = ri / per, row = mi * 128 + (ri - mi * per);
    // the first shares' outputs are on their way while the weights are made
    const float* q = parts + ((size_t)d4 * ROWS + row) * 4;
    float4 o[MERGE_AHEAD];
#pragma unroll
    for (int k = 0; k < MERGE_AHEAD; ++k)
      if (k < n) o[k] = *reinterpret_cast<const float4*>(q + share(k));
    // the shares' maxima and sums, and with them their weights: thread (i, d4) takes shares d4, d4 + D / 4, ...
    float M = -INFINITY;
    for (int x = d4; x < n; x += D / 4) {
      const float* ml = parts + share(x) + (size_t)ROWS * D + row;
      const float m = ml[0], l = ml[ROWS];
      wm[x][i] = m;
      wl[x][i] = l;
      if (l != 0.f) M = fmaxf(M, m);
    }
    red[d4][i] = M;
    __syncthreads();
#pragma unroll 8
    for (int x = 0; x < min(n, D / 4); ++x) M = fmaxf(M, red[x][i]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int x0 = 0; x0 < n; x0 += MERGE_AHEAD) {
      if (x0 > 0) {
#pragma unroll
        for (int k = 0; k < MERGE_AHEAD; ++k)
          if (x0 + k < n) o[k] = *reinterpret_cast<const float4*>(q + share(x0 + k));
      }
#pragma unroll
      for (int k = 0; k < MERGE_AHEAD; ++k) {
        if (x0 + k >= n) break;
        const float l = wl[x0 + k][i];
        if (l == 0.f) continue;  // this share saw no key of the row
        const float wgt = ex2(wm[x0 + k][i] - M);
        L += wgt * l;
        acc.x += wgt * o[k].x;
        acc.y += wgt * o[k].y;
        acc.z += wgt * o[k].z;
        acc.w += wgt * o[k].w;
      }
    }
    if (r0 + i < rec.rows) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const long long t = rec.row0 + ri / p.group, h = rec.head + ri % p.group;
      *reinterpret_cast<uint2*>(p.out + t * p.o_row + h * p.o_head + 4 * d4) =
          make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
      if (p.lse && d4 == 0)
        p.lse[t * p.lse_row + h * p.lse_head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
    __syncthreads();  // the weights are read
  }
}

bool shape_ok(const dflash_paged_cache* c, int q_heads) {
  return (c->head_dim == 64 || c->head_dim == 128) && q_heads >= 1 && q_heads % c->kv_heads == 0 &&
         q_heads / c->kv_heads <= 32;
}

bool rows_ok(const dflash_rows& r) {
  return (reinterpret_cast<uintptr_t>(r.data) & 15) == 0 && r.row_stride % 8 == 0 && r.head_stride % 8 == 0;
}

// Two M tiles an item when a sequence has more than one on average: they share
// the key tiles.
int m_tiles(int rows, int batch, int group) { return (long long)rows * group > 128ll * batch ? 2 : 1; }

size_t workspace_bytes(int grid, int nm, int D) {
  return ws_records(grid) + 2 * (size_t)grid * ws_slot_floats(128 * nm, D) * sizeof(float);
}

// What a device offers, asked once; the kernels' launch limits are set then.
constexpr int MAX_DEVICES = 64;
struct Device {
  int sms = 0;                    // one CTA an SM
  int clusters[2 * MAX_CLUSTER] = {};  // clusters of n CTAs it holds at once (n = 2, 4, 8, 16)
};
Device g_devices[MAX_DEVICES];
std::atomic<bool> g_known[MAX_DEVICES];
std::mutex g_devices_lock;

template <bool BF16, int D, int NM>
cudaError_t allow() {
  auto kern = k_paged_attn<BF16, D, NM>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PCfg<D, NM>::SMEM);
  if (!e && NM == 1) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

const Device* device_of(int device) {
  if (device < 0 || device >= MAX_DEVICES) return nullptr;
  Device& d = g_devices[device];
  if (g_known[device].load(std::memory_order_acquire)) return &d;
  std::lock_guard<std::mutex> lock(g_devices_lock);
  if (g_known[device].load(std::memory_order_acquire)) return &d;
  DeviceGuard guard(device);
  if (!guard.ok || cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, device) || d.sms < 1 ||
      allow<true, 64, 1>() || allow<true, 64, 2>() || allow<true, 128, 1>() || allow<true, 128, 2>() ||
      allow<false, 64, 1>() || allow<false, 64, 2>() || allow<false, 128, 1>() || allow<false, 128, 2>()) {
    cudaGetLastError();
    return nullptr;
  }
  for (int n = 2; n <= MAX_CLUSTER; n *= 2) {  // the 128-wide kernel's shared memory is the larger one
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n);
    cfg.blockDim = dim3(PCfg<128, 1>::THREADS);
    cfg.dynamicSmemBytes = PCfg<128, 1>::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&d.clusters[n], k_paged_attn<true, 128, 1>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      d.clusters[n] = 0;
    }
  }
  g_known[device].store(true, std::memory_order_release);
  return &d;
}

// How a call is launched.
struct Plan {
  int nm;       // M tiles an item
  int cs;       // > 0: a cluster of cs CTAs an item
  int grid;
  size_t ws;
};
// Items to launch a cluster for: a sequence of n rows has ceil(n / tok) token tiles; the most that any lengths make.
long long max_items(int rows, int batch, int tok, int hkv) {
  return std::min<long long>(rows, ((long long)rows + (long long)batch * (tok - 1)) / tok) * hkv;
}
Plan plan_call(const Device& dev, const dflash_paged_cache* c, int rows, int batch, int q_heads) {
  const int group = q_heads / c->kv_heads, D = c->head_dim;
  Plan pl = {m_tiles(rows, batch, group), 0, dev.sms, 0};
  const int tok = 128 / group, each = (rows + batch - 1) / batch;
  const long long items = (long long)batch * ((each + tok - 1) / tok) * c->kv_heads;  // of sequences of equal length
  const long long tiles = (((long long)c->max_pages << page_shift(c->page_size)) + KT - 1) / KT;  // of a sequence, at most
  // Few items over little cache: a cluster each, the largest that lets all run
  // at once (those of unequal sequences may take a second round).  That saves
  // the merge's launch, but leaves SMs idle.  Clusters against runs of equal
  // length (us): a token over 100 positions 8.0 / 10.5, 16 over 2,048 11.8 /
  // 14.9, 16 blocks over 3,000 with one KV head 17.0 / 20.1, 8 over 1,000 with 4
  // 12.5 / 14.7, a token over 8,192 15.9 / 16.6 (8 to 520 tiles); two of 16,000
  // with 4 KV heads 22.8 / 19.5, 16 over 32,000 39.9 / 35.6 (1,000 and 2,000
  // tiles).  Pairs only over short caches: 16 tokens over 500 with 4 KV heads
  // 10.9 / 13.0, but 24 blocks over up to 2,000 with 2 17.4 / 15.0.
  if (pl.nm == 1 && items * tiles <= CLUSTER_TILES) {
    int cs = 1;
    while (cs < MAX_CLUSTER && cs < tiles && items <= dev.clusters[2 * cs]) cs *= 2;
    if (items <= dev.sms && (cs >= 4 || tiles <= 2 * cs)) {
      pl.cs = cs;
      pl.grid = (int)max_items(rows, batch, tok, c->kv_heads) * cs;
    }
  }
  if (!pl.cs) pl.ws = workspace_bytes(dev.sms, pl.nm, D);
  return pl;
}

template <bool BF16, int D, int NM>
int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const Plan& pl,
           cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)pl.grid);
  cfg.blockDim = dim3(PCfg<D, NM>::THREADS);
  cfg.dynamicSmemBytes = PCfg<D, NM>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)std::max(pl.cs, 1);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.cs ? 2 : 1;
  if (int e = cuda_status(cudaLaunchKernelEx(&cfg, k_paged_attn<BF16, D, NM>, q, k, v, p))) return e;
  if (pl.cs || pl.grid == 1) return DFLASH_OK;
  cudaLaunchConfig_t mc = cfg;
  mc.gridDim = dim3((unsigned)(pl.grid - 1), 8);
  mc.blockDim = dim3(MERGE_ROWS * D / 4);
  mc.dynamicSmemBytes = (size_t)pl.grid * 2 * MERGE_ROWS * sizeof(float);
  return cuda_status(cudaLaunchKernelEx(&mc, k_paged_merge<BF16, D, NM>, p, pl.grid));
}

}  // namespace

extern "C" {

size_t dflash_paged_attention_workspace(const dflash_paged_cache* c, int32_t rows, int32_t batch, int32_t q_heads) {
  if (paged_cache_check(c) || !shape_ok(c, q_heads) || rows < 1 || batch < 1) return 0;
  const Device* dev = device_of(c->device);
  return dev ? plan_call(*dev, c, rows, batch, q_heads).ws : 0;
}

int dflash_paged_attention(const dflash_paged_cache* c, const dflash_attention_args* a, void* stream) {
  if (!a || a->rows < 0 || a->batch < 0 || a->window < 0 || !std::isfinite(a->scale * LOG2E)) return DFLASH_ERR_INVALID_ARG;
  if (int e = paged_cache_check(c)) return e;
  const int D = c->head_dim;
  if (!shape_ok(c, a->q_heads)) return DFLASH_ERR_SHAPE;
  if (a->rows == 0 || a->batch == 0) return DFLASH_OK;
  if (!a->q.data || !a->out.data || !a->cu_rows || !a->ctx_len || !rows_ok(a->q) || !rows_ok(a->out) ||
      !rows_ok({c->k, c->k_pos_stride, c->k_head_stride}) || !rows_ok({c->v, c->v_pos_stride, c->v_head_stride}) ||
      c->k_page_stride % 8 || c->v_page_stride % 8)
    return DFLASH_ERR_INVALID_ARG;
  // the sequences' first pairs, up to 33 KB, lie behind `seqs` in the tile area, which holds nothing else then
  if (a->batch > MAX_BATCH) return DFLASH_ERR_CAPACITY;
  if ((reinterpret_cast<uintptr_t>(a->workspace) & 255) || a->workspace_bytes < 0) return DFLASH_ERR_WORKSPACE;
  const int hq = a->q_heads;
  const Strided q = strided_rows(a->q, a->rows, hq, D), out = strided_rows(a->out, a->rows, hq, D),
                lse = strided(a->lse, 4, {{4 * a->lse_row_stride, a->rows}, {4 * a->lse_head_stride, hq}}),
                kp = strided_pool(c, false), vp = strided_pool(c, true), table = strided_table(c, a->batch),
                cu = strided_ints(a->cu_rows, a->batch + 1ll), ctx = strided_ints(a->ctx_len, a->batch),
                kv = strided_ints(a->kv_len, a->batch),
                status = strided_ints(reinterpret_cast<const int32_t*>(c->status), 1);
  if (!apart({out, lse}, {input_of(a->out, a->q, a->rows, hq, D), kp, vp, table, cu, ctx, kv, status}) || meet(lse, q))
    return DFLASH_ERR_INVALID_ARG;
  const Device* dev = device_of(c->device);
  if (!dev) return DFLASH_ERR_CUDA;
  const int group = a->q_heads / c->kv_heads;
  const Plan pl = plan_call(*dev, c, a->rows, a->batch, a->q_heads);
  if (pl.ws && (!a->workspace || (size_t)a->workspace_bytes < pl.ws)) return DFLASH_ERR_WORKSPACE;
  if (!apart({strided(a->workspace, (long long)pl.ws, {})}, {out, lse, q, kp, vp, table, cu, ctx, kv, status}))
    return DFLASH_ERR_INVALID_ARG;
  PagedParams p = {};
  p.out = static_cast<uint16_t*>(a->out.data);
  p.o_row = a->out.row_stride;
  p.o_head = a->out.head_stride;
  p.wide_out = (reinterpret_cast<uintptr_t>(a->out.data) & 31) == 0 && p.o_row % 16 == 0 && p.o_head % 16 == 0;
  p.lse = a->lse;
  p.lse_row = a->lse_row_stride;
  p.lse_head = a->lse_head_stride;
  p.table = c->page_table;
  p.table_stride = c->table_stride;
  p.max_pages = c->max_pages;
  p.n_pages = c->n_pages;
  p.shift = page_shift(c->page_size);
  const long long cap = (long long)c->max_pages << p.shift;
  p.cap = (int)(cap < (1ll << 30) ? cap : (1ll << 30));
  p.cu = a->cu_rows;
  p.ctx = a->ctx_len;
  p.kv_len = a->kv_len;
  p.rows = a->rows;
  p.batch = a->batch;
  p.hkv = c->kv_heads;
  p.group = group;
  p.causal = a->causal != 0;
  p.window = a->window;
  p.tok = 128 / group;
  // a scale of zero weighs every key alike; the tiny one does, and keeps a mask's -inf
  const float scale = a->scale * LOG2E;
  p.negate = scale < 0.f;
  p.scale_log2 = scale == 0.f ? 1e-30f : p.negate ? -scale : scale;
  p.status = c->status;
  p.ws = static_cast<char*>(a->workspace);
  p.cs = pl.cs;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  const bool bf = c->dtype == DFLASH_BF16;
  CUtensorMap qm, km, vm;
  const uint64_t qd[3] = {(uint64_t)D, (uint64_t)a->q_heads, (uint64_t)a->rows};
  const uint64_t qs[2] = {(uint64_t)a->q.head_stride * 2, (uint64_t)a->q.row_stride * 2};
  const uint32_t qb[3] = {64, (uint32_t)group, (uint32_t)p.tok};
  const uint64_t kd[4] = {(uint64_t)D, (uint64_t)c->page_size, (uint64_t)c->kv_heads, (uint64_t)c->n_pages};
  const uint64_t ks[3] = {(uint64_t)c->k_pos_stride * 2, (uint64_t)c->k_head_stride * 2, (uint64_t)c->k_page_stride * 2};
  const uint64_t vs[3] = {(uint64_t)c->v_pos_stride * 2, (uint64_t)c->v_head_stride * 2, (uint64_t)c->v_page_stride * 2};
  const uint32_t kb[4] = {64, (uint32_t)(c->page_size < KT ? c->page_size : KT), 1, 1};
  if (!tmap_tiled(&qm, a->q.data, 3, qd, qs, qb, bf) || !tmap_tiled(&km, c->k, 4, kd, ks, kb, bf) ||
      !tmap_tiled(&vm, c->v, 4, kd, vs, kb, bf))
    return DFLASH_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 128) {
    if (pl.nm == 2) return bf ? launch<true, 128, 2>(qm, km, vm, p, pl, s) : launch<false, 128, 2>(qm, km, vm, p, pl, s);
    return bf ? launch<true, 128, 1>(qm, km, vm, p, pl, s) : launch<false, 128, 1>(qm, km, vm, p, pl, s);
  }
  if (pl.nm == 2) return bf ? launch<true, 64, 2>(qm, km, vm, p, pl, s) : launch<false, 64, 2>(qm, km, vm, p, pl, s);
  return bf ? launch<true, 64, 1>(qm, km, vm, p, pl, s) : launch<false, 64, 1>(qm, km, vm, p, pl, s);
}

}  // extern "C"

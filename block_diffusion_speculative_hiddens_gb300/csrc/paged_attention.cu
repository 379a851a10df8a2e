// Attention of a ragged batch of new tokens over a caller's paged cache, on
// the 5th-generation tensor cores.
//
// The rows of one KV head -- its G query heads of consecutive tokens -- share
// its keys, so they are packed into M tiles of 128 rows (TOK = 128 / G tokens
// each).  An item is one or two (NM) M tiles of one sequence and KV head; its
// work is the 128-key tiles its rows see.  All items' tiles, in order
// (sequence, token tile, KV head), are cut into equal runs, one for each CTA
// of a persistent grid: a batch of ragged single tokens, one verify block over
// a long context and a prompt all load the SMs evenly.  A run that covers
// only part of an item leaves its share (O unnormalised, running maximum and
// sum, float32) in the workspace, and k_paged_merge joins the shares in order.
//
// Per key tile and M tile:
//   S = Q K^T   tcgen05.mma M=128 x N=128 keys x K=D, operands in shared memory,
//   softmax     one row a thread, S read from TMEM, one pass with a running
//               maximum (log2 domain) that moves only when a tile's maximum
//               exceeds it by more than 2^8 (then the row's O is rescaled in
//               TMEM): P is the same softmax up to a power of two that the sum
//               shares, and stays inside f16,
//   O += P V    tcgen05.mma with P as the TMEM A operand (16 bits, over the S
//               it came from) and V as it lies in the cache (N-major).
// The tensor core runs the MMAs in issue order, so S of the next tile may
// overwrite the P that the O MMA before it read.
// Warps: 4 NM softmax, one issuing MMAs, one loading.
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int KT = 128;  // keys of a tile

struct PagedParams {
  uint16_t* out;
  long long o_row, o_head;
  float* lse;
  long long lse_row, lse_head;
  const int* table;
  long long table_stride;
  int max_pages, n_pages, shift;
  int cap;            // positions a table row can hold
  const int* cu;
  const int* ctx;
  const int* kv_len;
  int rows, batch, hq, hkv, group, causal, window;
  int tok;            // tokens of an M tile
  float scale_log2;   // > 0
  int negate;         // the caller's scale is negative
  uint32_t* status;
  char* ws;
};

// Workspace: a header, one record a CTA, two partial slots a CTA.
struct WsHead {
  long long units;
  int ctas;
};
struct WsCta {
  int off, units;  // of the item its run begins in: tiles before it, tiles of the item
  int b, mt, kvh, pad[3];
};
constexpr size_t ws_records(int grid) { return 256 + ((size_t)grid * sizeof(WsCta) + 255) / 256 * 256; }
// One slot: O [D/4][rows] float4, running maxima [rows], sums [rows].
constexpr size_t ws_slot_floats(int rows, int D) { return (size_t)rows * (D + 2); }

template <int D, int NM>
struct PCfg {
  static constexpr int ROWS = 128 * NM;
  static constexpr int PANEL = 128 * 128;            // 128 rows x 64 dims
  static constexpr int TILE = (D / 64) * PANEL;      // Q of an M tile, K or V of a key tile
  static constexpr int SLOTS = (D == 128 ? 7 : 12) - NM;
  static constexpr int OFF_RING = NM * TILE;
  static constexpr int OFF_BAR = OFF_RING + SLOTS * TILE;
  static constexpr int SMEM = 1024 + OFF_BAR + 512;  // + 1024 for aligning the base
  // NM = 2: a third warpgroup issues and loads, and hands registers to the softmax ones
  static constexpr int THREADS = NM == 2 ? 384 : 192;
  static constexpr int S_COL = 0;                    // two S buffers of 128 columns
  static constexpr int O_COL = 256;
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

DFL_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
DFL_DEV void tmem_st32_nowait(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
      "%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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

// A CTA's run through the items.
struct Walk {
  int b, mt, kvh, off;  // the item and the first of its tiles that is this CTA's
  long long left;       // units still to do
  Seq s;
  Span span;
  int t0, t1;           // the item's tokens
  int n;                // units of this segment
  int units;            // units of the item (1 if it has no tile: its rows get zeros)
};
template <int NM>
DFL_DEV void walk_item(const PagedParams& p, Walk& w) {
  w.t0 = w.mt * p.tok * NM;
  w.t1 = min(w.t0 + p.tok * NM, w.s.n);
  w.span = load_span(p, w.s, w.t0, w.t1);
  w.units = max(w.span.tiles, 1);
  w.n = (int)min((long long)(w.units - w.off), w.left);
}
template <int NM>
DFL_DEV bool walk_next(const PagedParams& p, Walk& w) {
  w.left -= w.n;
  if (w.left <= 0) return false;
  w.off = 0;
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

struct Sched {
  long long part[16];
  int b, mt, units, pairs;
  long long before;  // units before the pair (b, mt)
};

// Where this CTA's run begins.  Pairs (sequence, token tile) are counted and
// weighed by the whole CTA, blockDim.x at a time; `first` [batch + 1] receives
// the sequences' first pairs.  False: no work at all, or none for this CTA.
template <int NM>
DFL_DEV bool locate(const PagedParams& p, Sched* sc, int* first, Walk& w, long long* units_out, int* ctas_out) {
  const int per = p.tok * NM;
  long long pairs = 0;
  for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int m = 0;
    if (b < p.batch) m = (load_seq(p, b).n + per - 1) / per;
    long long all;
    const long long at = cta_scan(m, sc->part, &all);
    if (b < p.batch) first[b] = (int)(pairs + at - m);
    pairs += all;
  }
  if (threadIdx.x == 0) first[p.batch] = (int)pairs;
  __syncthreads();
  auto weigh = [&](int pair, int* b_out, int* mt_out) {
    int lo = 0, hi = p.batch - 1;  // the last sequence whose first pair is not behind
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= pair) lo = mid;
      else hi = mid - 1;
    }
    const Seq s = load_seq(p, lo);
    const int mt = pair - first[lo], t0 = mt * per;
    *b_out = lo;
    *mt_out = mt;
    return max(load_span(p, s, t0, min(t0 + per, s.n)).tiles, 1);
  };
  long long total = 0, all;
  int b = 0, mt = 0, u = 0;
  long long incl = 0;
  const bool once = pairs <= blockDim.x;
  for (long long p0 = 0; p0 < pairs; p0 += blockDim.x) {
    const long long pair = p0 + threadIdx.x;
    u = pair < pairs ? weigh((int)pair, &b, &mt) : 0;
    incl = cta_scan((long long)u * p.hkv, sc->part, &all);
    total += all;
  }
  if (total == 0) return false;
  const int ctas = (int)min((long long)gridDim.x, total);
  *units_out = total;
  *ctas_out = ctas;
  if ((int)blockIdx.x >= ctas) return false;
  const long long u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
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
      sc->units = u;
      sc->before = incl - (long long)u * p.hkv;
    }
    if (!once && base > u0) break;  // uniform: base is the CTA's
  }
  __syncthreads();
  const long long in = u0 - sc->before;
  w.b = sc->b;
  w.mt = sc->mt;
  w.kvh = (int)(in / sc->units);
  w.off = (int)(in % sc->units);
  w.left = u1 - u0;
  w.s = load_seq(p, w.b);
  walk_item<NM>(p, w);
  return true;
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
  uint64_t* s_full = empty + C::SLOTS;  // [2] S (and every MMA before it) done
  uint64_t* p_full = s_full + 2;        // [2] P written
  uint64_t* o_done = p_full + 2;        // [2] an O MMA done
  uint64_t* o_empty = o_done + 2;       // [2] O read out
  uint64_t* q_full = o_empty + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mdone = q_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  Sched* sched = reinterpret_cast<Sched*>(sm + C::OFF_BAR + 320);
  static_assert((2 * C::SLOTS + 11) * 8 + 8 <= 320 && sizeof(Sched) <= 192, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int MMA_WARP = 4 * NM, LOAD_WARP = 4 * NM + 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(o_done + i, 1);
      mbar_init(o_empty + i, 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(mdone, 1);
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
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  Walk w;
  long long units = 0;
  int ctas = 0;
  // the tile area is free until the loads begin: it holds the sequences' first pairs
  const bool work = locate<NM>(p, sched, reinterpret_cast<int*>(sm), w, &units, &ctas);
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *reinterpret_cast<WsHead*>(p.ws) = WsHead{units, ctas};
    if (work) {
      WsCta* rec = reinterpret_cast<WsCta*>(p.ws + 256) + blockIdx.x;
      rec->off = w.off;
      rec->units = w.units;
      rec->b = w.b;
      rec->mt = w.mt;
      rec->kvh = w.kvh;
    }
  }
  fence_proxy_async_smem();  // the first pairs were written and read before the loads land over them
  __syncthreads();
  bool aborted = false;
  auto wait_all = [&](uint64_t* bar, uint32_t par) {  // warp-uniform
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par, p.status, &aborted));
    if (!ok) aborted = true;
    return ok;
  };

  // registers of the NM = 2 roles: 168 a thread at launch, 384 threads; 2 x 200 + 104 is as much
  if (!work) {
    // nothing for this CTA
  } else if (warp > LOAD_WARP) {
    if (NM == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  } else if (warp == LOAD_WARP) {
    if (NM == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    // ------------------------------------------------ loads
    const int page = 1 << p.shift, box = min(page, KT), boxes = KT / box;
    int seg = 0;
    long long nt = 0;  // ring slots filled
    bool ok = true;
    do {
      const int tiles = w.span.tiles ? w.n : 0;
      if (tiles == 0) continue;
      if (lane == 0 && (p.kv_len ? (long long)p.kv_len[w.b] : w.s.ctx + w.s.n) > p.cap)
        dev_error(p.status, DFLASH_DEV_PAGE);
      if (seg > 0 && !wait_all(q_empty, (uint32_t)((seg - 1) & 1))) break;
      const int nm = NM == 2 && w.t0 + p.tok < w.t1 ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(nm * (D / 64) * p.tok * p.group * 128));
        for (int m = 0; m < nm; ++m)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sm + m * C::TILE + h * C::PANEL, &qmap, q_full, 64 * h, w.kvh * p.group,
                        w.s.row0 + w.t0 + m * p.tok);
      }
      ++seg;
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
        for (int kv = 0; kv < 2; ++kv, ++nt) {  // K, then V
          const int s = (int)(nt % C::SLOTS);
          if (nt >= C::SLOTS && !wait_all(empty + s, (uint32_t)((nt / C::SLOTS - 1) & 1))) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full + s, C::TILE);
          uint8_t* dst = sm + C::OFF_RING + s * C::TILE;
          for (int i = 0; i < boxes; ++i) {
            const int id = __shfl_sync(0xffffffffu, ids, e0 + i - base);
            if (lane == 0)
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(dst + h * C::PANEL + i * box * 128, kv ? &vmap : &kmap, full + s, 64 * h,
                            page > KT ? key0 & (page - 1) : 0, w.kvh, id);
          }
        }
      }
    } while (ok && walk_next<NM>(p, w));
    // every copy lands before the CTA may exit
    for (long long i = nt > C::SLOTS ? nt - C::SLOTS : 0; i < nt; ++i) {
      bool drain = false;
      mbar_wait(full + i % C::SLOTS, (uint32_t)((i / C::SLOTS) & 1), p.status, &drain);
    }
    if (seg > 0) {
      bool drain = false;
      mbar_wait(q_full, (uint32_t)((seg - 1) & 1), p.status, &drain);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------ MMA issue (converged warp, one elected lane)
    if (NM == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const uint32_t idesc_s = idesc_f16_f32(128, KT, BF16 ? 1 : 0);
    const uint32_t idesc_o = idesc_f16_f32(128, D, BF16 ? 1 : 0) | (1u << 16);  // V is N-major
    int seg = 0;
    long long nt = 0;          // ring slots used
    int it[2] = {0, 0};        // S tiles issued for each M tile
    int sg[2] = {0, 0};        // segments of each M tile
    auto issue_s = [&](int m, long long slot) {
      const uint32_t qa = smem_u32(sm + m * C::TILE), ka = smem_u32(sm + C::OFF_RING + (int)(slot % C::SLOTS) * C::TILE);
      const int buf = NM == 2 ? m : it[0] & 1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = (uint32_t)((kk >> 2) * C::PANEL);
        tc_mma_f16_elect(tmem + (uint32_t)(C::S_COL + 128 * buf), sdesc_sw128(qa + o) + (uint64_t)(2 * (kk & 3)),
                         sdesc_sw128(ka + o) + (uint64_t)(2 * (kk & 3)), idesc_s, kk > 0 ? 1u : 0u);
      }
      tc_commit_elect(s_full + buf);
      ++it[m];
    };
    bool ok = true;
    do {
      const int tiles = w.span.tiles ? w.n : 0;
      if (tiles == 0) continue;
      const int nm = NM == 2 && w.t0 + p.tok < w.t1 ? 2 : 1;
      auto wait_full = [&](long long slot) { return wait_all(full + slot % C::SLOTS, (uint32_t)((slot / C::SLOTS) & 1)); };
      // S of tile j for every M tile (NM = 2: after its O MMA of tile j - 1)
      if (!wait_all(q_full, (uint32_t)(seg & 1)) || !wait_full(nt)) break;
      ++seg;
      tc_fence_after();
      for (int m = 0; m < nm; ++m) issue_s(m, nt);
      tc_commit_elect(empty + nt % C::SLOTS);
      if (tiles == 1) tc_commit_elect(q_empty);
      for (int j = 0; j < tiles && ok; ++j, nt += 2) {
        const long long vs = nt + 1, ks = nt + 2;
        if (NM == 1 && j + 1 < tiles) {  // two S buffers: the next S runs beside this tile's softmax
          if (!(ok = wait_full(ks))) break;
          tc_fence_after();
          issue_s(0, ks);
          tc_commit_elect(empty + ks % C::SLOTS);
          if (j + 2 == tiles) tc_commit_elect(q_empty);
        }
        for (int m = 0; m < nm; ++m) {
          const int done = NM == 2 ? it[m] - 1 : it[0] - 1 - (j + 1 < tiles);  // the S tile whose P is next
          const int buf = NM == 2 ? m : done & 1;
          if (m == 0) {
            if (!(ok = wait_full(vs))) break;
            const int key0 = (w.span.tile0 + w.off + j) * KT;
            const int v0 = w.s.kv - key0;
            if (v0 < KT && (v0 & ((1 << p.shift) - 1))) {
              // the sequence ends inside a page: what lies behind it (stale,
              // perhaps not finite) must not meet P's zeros in the MMA
              const int v1 = min(KT, ((v0 >> p.shift) + 1) << p.shift);
              uint8_t* vt = sm + C::OFF_RING + (int)(vs % C::SLOTS) * C::TILE;
              for (int i = lane; i < (v1 - v0) * 8; i += 32)
                for (int h = 0; h < D / 64; ++h)
                  *reinterpret_cast<uint4*>(vt + h * C::PANEL + (v0 + (i >> 3)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc_fence_after();
          }
          if (j == 0 && sg[m]++ > 0 && !(ok = wait_all(o_empty + m, (uint32_t)((sg[m] - 2) & 1)))) break;
          if (!(ok = wait_all(p_full + buf, (uint32_t)((NM == 2 ? done : done >> 1) & 1)))) break;
          tc_fence_after();
          const uint32_t va = smem_u32(sm + C::OFF_RING + (int)(vs % C::SLOTS) * C::TILE);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            tc_mma_f16_ts_elect(tmem + (uint32_t)(C::O_COL + D * m), tmem + (uint32_t)(C::S_COL + 128 * buf + 8 * kk),
                                sdesc_sw128_mn(va + 2048u * kk, C::PANEL), idesc_o, (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit_elect(o_done + m);
          if (m == nm - 1) tc_commit_elect(empty + vs % C::SLOTS);
          if (NM == 2 && j + 1 < tiles) {
            if (m == 0) {
              if (!(ok = wait_full(ks))) break;
              tc_fence_after();
            }
            issue_s(m, ks);
            if (m == nm - 1) {
              tc_commit_elect(empty + ks % C::SLOTS);
              if (j + 2 == tiles) tc_commit_elect(q_empty);
            }
          }
        }
      }
    } while (ok && walk_next<NM>(p, w));
    // every issued MMA completes before the columns are freed
    tc_commit_elect(mdone);
    bool drain = false;
    mbar_wait(mdone, 0, p.status, &drain);
  } else {
    // ------------------------------------------------ softmax: one row a thread
    if (NM == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int m = warp >> 2;
    const int r = threadIdx.x & 127;
    const int rt = r / p.group, rh = r - rt * p.group;  // the row's token in the M tile and head in the group
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_base = lane_base + (uint32_t)(C::O_COL + D * m);
    int it = 0;  // S tiles of this M tile
    bool ok = true;
    do {
      const int tiles = w.span.tiles ? w.n : 0;
      const int t = w.t0 + m * p.tok + rt;
      const bool valid = rt < p.tok && t < w.t1;
      if (NM == 2 && m == 1 && w.t0 + p.tok >= w.t1) continue;  // no row in this M tile
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // the keys this row sees; rows that do not exist mask nothing (they are not written)
      int lo = 0, hi = 1 << 30;
      if (valid) {
        hi = p.causal ? (int)min(max(w.s.ctx + t + 1, 0ll), (long long)w.s.kv) : w.s.kv;
        lo = p.window > 0 ? (int)min(max(w.s.ctx + t - p.window + 1, 0ll), (long long)w.s.kv) : 0;
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < tiles; ++j, ++it) {
        const int buf = NM == 2 ? m : it & 1;
        const uint32_t par = (uint32_t)((NM == 2 ? it : it >> 1) & 1);
        if (!(ok = wait_all(s_full + buf, par))) break;
        tc_fence_after();
        const uint32_t s_base = lane_base + (uint32_t)(C::S_COL + 128 * buf);
        if (warp_valid) {
          uint32_t u[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_nowait(s_base + 32 * c, u + 32 * c);
          tmem_wait_ld();
          float* s = reinterpret_cast<float*>(u);
          const int key0 = (w.span.tile0 + w.off + j) * KT;
          if (p.negate) {
#pragma unroll
            for (int k = 0; k < 128; ++k) s[k] = -s[k];
          }
          const int h = hi - key0, l = lo - key0;
          if (__any_sync(0xffffffffu, h < KT || l > 0)) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (k >= h || k < l) s[k] = -INFINITY;
          }
          float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
          for (int k = 4; k < 128; k += 4) {
            mx0 = fmaxf(mx0, s[k]);
            mx1 = fmaxf(mx1, s[k + 1]);
            mx2 = fmaxf(mx2, s[k + 2]);
            mx3 = fmaxf(mx3, s[k + 3]);
          }
          const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * p.scale_log2;
          const bool move = mx > m_run + 8.f;
          if (__any_sync(0xffffffffu, move)) {
            const float m_new = move ? mx : m_run;
            if (j > 0) {  // O of the tiles before is against m_run
              if (NM == 1 && !(ok = wait_all(o_done + m, (uint32_t)((it - 1) & 1)))) break;
              tc_fence_after();
              const float alpha = move ? ex2(m_run - m_new) : 1.f;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_nowait(o_base + 32 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32_nowait(o_base + 32 * c, o);
              }
              tmem_wait_st();
              l_run *= alpha;
            }
            m_run = m_new;
          }
          const float ref = m_run == -INFINITY ? 0.f : m_run;  // a row that has seen no key yet adds 0
          float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f, sum3 = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float a = ex2(fmaf(s[64 * c + 2 * k], p.scale_log2, -ref));
              const float b = ex2(fmaf(s[64 * c + 2 * k + 1], p.scale_log2, -ref));
              const float d = ex2(fmaf(s[64 * c + 2 * k + 2], p.scale_log2, -ref));
              const float e = ex2(fmaf(s[64 * c + 2 * k + 3], p.scale_log2, -ref));
              sum0 += a;
              sum1 += b;
              sum2 += d;
              sum3 += e;
              pk[k] = pack16<BF16>(a, b);
              pk[k + 1] = pack16<BF16>(d, e);
            }
            tmem_st32_nowait(s_base + 32 * c, pk);
          }
          l_run += (sum0 + sum1) + (sum2 + sum3);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + buf);
      }
      if (!ok) break;
      // the segment's O
      if (tiles > 0) {
        if (NM == 1 && tiles > 1 && !(ok = wait_all(o_done + m, (uint32_t)((it - 2) & 1)))) break;
        if (!(ok = wait_all(o_done + m, (uint32_t)((it - 1) & 1)))) break;
        tc_fence_after();
      }
      const bool whole = w.n == w.units;
      if (warp_valid) {
        if (whole) {
          const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
          const long long head = w.kvh * p.group + rh, row = w.s.row0 + t;
          uint16_t* dst = p.out + row * p.o_row + head * p.o_head;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            if (tiles > 0) {
              tmem_ld32_nowait(o_base + 32 * c, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
            if (valid) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  y[i] = pack16<BF16>(__uint_as_float(o[8 * e + 2 * i]) * inv, __uint_as_float(o[8 * e + 2 * i + 1]) * inv);
                *reinterpret_cast<uint4*>(dst + 32 * c + 8 * e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
          if (p.lse && valid)
            p.lse[row * p.lse_row + head * p.lse_head] =
                l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.6931471805599453f;
        } else {
          const int slot = 2 * blockIdx.x + (w.off == 0 ? 1 : 0);
          float* part = reinterpret_cast<float*>(p.ws + ws_records(gridDim.x)) + slot * ws_slot_floats(C::ROWS, D);
          const int row = m * 128 + r;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_nowait(o_base + 32 * c, o);
            tmem_wait_ld();
            if (valid) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(part + ((size_t)(8 * c + e) * C::ROWS + row) * 4) =
                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
          if (valid) {
            part[(size_t)C::ROWS * D + row] = m_run;
            part[(size_t)C::ROWS * (D + 1) + row] = l_run;
          }
        }
      }
      if (tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty + m);
      }
    } while (walk_next<NM>(p, w));
  }
  tc_fence_before();
  __syncthreads();  // every MMA and TMEM read done, every tile landed
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the shares of the items that more than one CTA worked on.  CTA x is
// the boundary between runs x and x + 1; the first boundary inside an item
// joins it, in the order of the runs.  One thread takes 4 columns of a row.
template <bool BF16, int D, int NM>
__global__ void __launch_bounds__(256) k_paged_merge(const PagedParams p, int grid) {
  constexpr int ROWS = 128 * NM;
  pdl_launch_dependents();
  pdl_wait();
  const WsHead head = *reinterpret_cast<const WsHead*>(p.ws);
  const int c = blockIdx.x + 1;
  if (c >= head.ctas) return;
  const WsCta rec = reinterpret_cast<const WsCta*>(p.ws + 256)[c];
  if (rec.off == 0) return;  // the run begins with its item
  auto start = [&](int x) { return head.units * x / head.ctas; };
  const long long item0 = start(c) - rec.off, item1 = item0 + rec.units;
  if (start(c - 1) > item0) return;  // an earlier boundary joins this item
  int end = c + 1;                   // runs c - 1 .. end - 1 hold a share
  while (end < head.ctas && start(end) < item1) ++end;
  const Seq s = load_seq(p, rec.b);
  const int t0 = rec.mt * p.tok * NM, tokens = min(p.tok * NM, s.n - t0);
  const int per = p.tok * p.group;  // rows of an M tile
  const int rows = tokens * p.group;
  const float* parts = reinterpret_cast<const float*>(p.ws + ws_records(grid));
  constexpr size_t SF = ws_slot_floats(ROWS, D);
  auto share = [&](int x) { return parts + (2 * (size_t)x + (x == c - 1 ? 1 : 0)) * SF; };
  for (int e = blockIdx.y * blockDim.x + threadIdx.x; e < rows * (D / 4); e += gridDim.y * blockDim.x) {
    const int d4 = e / rows, i = e - d4 * rows;         // i: token-major row of the item
    const int mi = i / per, row = mi * 128 + (i - mi * per);
    float M = -INFINITY;
    for (int x = c - 1; x < end; ++x) {
      const float* q = share(x);
      if (q[(size_t)ROWS * (D + 1) + row] != 0.f) M = fmaxf(M, q[(size_t)ROWS * D + row]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    for (int x = c - 1; x < end; ++x) {
      const float* q = share(x);
      const float l = q[(size_t)ROWS * (D + 1) + row];
      if (l == 0.f) continue;  // this share saw no key of the row
      const float wgt = exp2f(q[(size_t)ROWS * D + row] - M);
      const float4 o = *reinterpret_cast<const float4*>(q + ((size_t)d4 * ROWS + row) * 4);
      acc.x += wgt * o.x;
      acc.y += wgt * o.y;
      acc.z += wgt * o.z;
      acc.w += wgt * o.w;
      L += wgt * l;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const long long t = s.row0 + t0 + i / p.group, h = rec.kvh * p.group + i % p.group;
    *reinterpret_cast<uint2*>(p.out + t * p.o_row + h * p.o_head + 4 * d4) =
        make_uint2(pack16<BF16>(acc.x * inv, acc.y * inv), pack16<BF16>(acc.z * inv, acc.w * inv));
    if (p.lse && d4 == 0)
      p.lse[t * p.lse_row + h * p.lse_head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
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

// One CTA an SM: the SMs of a device, 0 if it has none to give.  The kernels'
// shared-memory limits are set when a device is first asked for.
constexpr int MAX_DEVICES = 64;
std::atomic<int> g_sms[MAX_DEVICES];

template <bool BF16, int D, int NM>
bool allow_smem() {
  return cudaFuncSetAttribute(k_paged_attn<BF16, D, NM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              PCfg<D, NM>::SMEM) == cudaSuccess;
}
template <bool BF16>
bool allow_all() {
  return allow_smem<BF16, 64, 1>() && allow_smem<BF16, 64, 2>() && allow_smem<BF16, 128, 1>() && allow_smem<BF16, 128, 2>();
}

int device_grid(int device) {
  if (device < 0 || device >= MAX_DEVICES) return 0;
  int n = g_sms[device].load(std::memory_order_acquire);
  if (n) return n;
  DeviceGuard guard(device);
  if (!guard.ok || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1 ||
      !allow_all<true>() || !allow_all<false>()) {
    cudaGetLastError();
    return 0;
  }
  g_sms[device].store(n, std::memory_order_release);
  return n;
}

template <bool BF16, int D, int NM>
int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, int grid,
           cudaStream_t s) {
  auto kern = k_paged_attn<BF16, D, NM>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(PCfg<D, NM>::THREADS);
  cfg.dynamicSmemBytes = PCfg<D, NM>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, q, k, v, p) != cudaSuccess) return DFLASH_ERR_CUDA;
  if (grid == 1) return DFLASH_OK;
  cudaLaunchConfig_t mc = cfg;
  mc.gridDim = dim3((unsigned)(grid - 1), 4);
  mc.blockDim = dim3(256);
  mc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&mc, k_paged_merge<BF16, D, NM>, p, grid) == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t dflash_paged_attention_workspace(const dflash_paged_cache* c, int32_t rows, int32_t batch, int32_t q_heads) {
  if (paged_cache_check(c) || rows < 0 || batch < 0 || q_heads < 1 || q_heads % c->kv_heads) return 0;
  const int grid = device_grid(c->device);
  return grid ? workspace_bytes(grid, m_tiles(rows, batch, q_heads / c->kv_heads), c->head_dim) : 0;
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
  if (a->batch > 8192) return DFLASH_ERR_CAPACITY;  // the sequences' first pairs lie in one M tile's shared memory
  if (!a->workspace || (reinterpret_cast<uintptr_t>(a->workspace) & 255)) return DFLASH_ERR_WORKSPACE;
  const int group = a->q_heads / c->kv_heads, nm = m_tiles(a->rows, a->batch, group);
  if (a->workspace_bytes <= 0) return DFLASH_ERR_WORKSPACE;
  const int grid = device_grid(c->device);
  if (!grid) return DFLASH_ERR_CUDA;
  if ((size_t)a->workspace_bytes < workspace_bytes(grid, nm, D)) return DFLASH_ERR_WORKSPACE;
  PagedParams p = {};
  p.out = static_cast<uint16_t*>(a->out.data);
  p.o_row = a->out.row_stride;
  p.o_head = a->out.head_stride;
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
  p.hq = a->q_heads;
  p.hkv = c->kv_heads;
  p.group = group;
  p.causal = a->causal != 0;
  p.window = a->window;
  p.tok = 128 / group;
  // a scale of zero weighs every key alike; the tiny one does, and keeps a mask's -inf
  const float scale = a->scale * 1.4426950408889634f;
  p.negate = scale < 0.f;
  p.scale_log2 = scale == 0.f ? 1e-30f : p.negate ? -scale : scale;
  p.status = c->status;
  p.ws = static_cast<char*>(a->workspace);
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
    if (nm == 2) return bf ? launch<true, 128, 2>(qm, km, vm, p, grid, s) : launch<false, 128, 2>(qm, km, vm, p, grid, s);
    return bf ? launch<true, 128, 1>(qm, km, vm, p, grid, s) : launch<false, 128, 1>(qm, km, vm, p, grid, s);
  }
  if (nm == 2) return bf ? launch<true, 64, 2>(qm, km, vm, p, grid, s) : launch<false, 64, 2>(qm, km, vm, p, grid, s);
  return bf ? launch<true, 64, 1>(qm, km, vm, p, grid, s) : launch<false, 64, 1>(qm, km, vm, p, grid, s);
}

}  // extern "C"

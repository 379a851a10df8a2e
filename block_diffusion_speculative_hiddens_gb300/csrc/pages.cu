// The pages of a caller's paged cache: who holds them, the copies that sharing
// takes, and the copies' bytes.
//
// A pool's state is refs (holders of each page), a table and lens.  There is no
// free list: a free page is one with refs 0, found by a scan, so nothing can fall
// out of step with the counts, the pages handed out do not depend on the order of
// atomics (the lowest free ones, by rank), and compact needs no other view.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "overlap.h"

namespace {

struct Pool {
  int* refs;
  int* table;
  long long stride;
  int* lens;
  uint32_t* status;  // [0] bits, [1] ticket
  int n_pages, shift, max_pages, batch;
};

DFL_DEV int pages_of(int len, int shift) { return (int)(((unsigned)len + (1u << shift) - 1) >> shift); }
DFL_DEV bool len_fits(const Pool& p, int len) { return len >= 0 && pages_of(len, p.shift) <= p.max_pages; }

// One holder more and less of each of four entries' pages, those with their bit
// set.  Whether a page is pinned does not change during a call, so it is looked up
// once; without `pins` none of the pool's pages is.  A page given up has a holder
// until then, or its count was too low: the value that the subtraction found says so
// (two entries may both take away the last holder), and the one goes back.
DFL_DEV void count_entries(const Pool& p, const int (&more)[4], unsigned m, const int (&less)[4], unsigned l, bool pins) {
  int rm[4], was[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)  // all of them on their way at once
    rm[j] = m >> j & 1 && (unsigned)more[j] < (unsigned)p.n_pages ? __ldcg(p.refs + more[j]) : INT_MIN;
  if (pins) {
    int rl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) rl[j] = l >> j & 1 && (unsigned)less[j] < (unsigned)p.n_pages ? __ldcg(p.refs + less[j]) : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) l &= ~((unsigned)(rl[j] < 0) << j);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)  // outside the pool: as if nobody held it
    was[j] = l >> j & 1 ? (unsigned)less[j] < (unsigned)p.n_pages ? atomicSub(p.refs + less[j], 1) : 0 : 1;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (rm[j] >= 0) atomicAdd(p.refs + more[j], 1);
    bad |= m >> j & 1 && (unsigned)more[j] >= (unsigned)p.n_pages;
    if (was[j] > 0) continue;
    if ((unsigned)less[j] < (unsigned)p.n_pages) atomicAdd(p.refs + less[j], 1);
    bad |= was[j] == 0;  // who finds it below 0 came behind one who found it 0
  }
  if (bad) dev_error(p.status, DFLASH_DEV_PAGE);
}

// ------------------------------------------------------------------ fork
//
// A column of the table depends on the same column alone, so a CTA takes a few
// columns of every row: it loads what the rows will hold, and writes after a
// barrier; the table is its own output without a second copy.  Rows and entries
// that stay as they are (a long shared prefix) cost their reads only.  The
// lengths, which every CTA reads, are written by the last one.
// Bound by latency: parents, lengths, entries and counts are four loads deep, each
// 0.4 us, and the value that a subtraction found.  Four rows of 33 pages 2.4 us; 512
// rows of 16 to 512 pages 4.4 us (4 without looking at that value; counting an entry's
// two pages one after the other: 5.7; every row's units unrolled, 69 KB of code that
// each call fetches anew: 7.7).  Rows of more units than threads, several a thread:
// 1,025 of up to 32 pages 10 us, 2,048 of up to 64 19, 8,192 of up to 128 72.
constexpr int FORK_THREADS = 1024;

DFL_DEV int4 load_entries(const Pool& p, int row, int col, bool vec) {
  const int* at = p.table + row * p.stride + col;
  if (vec && col + 4 <= p.max_pages) return *reinterpret_cast<const int4*>(at);
  int4 v = make_int4(-1, -1, -1, -1);
  if (col < p.max_pages) v.x = at[0];
  if (col + 1 < p.max_pages) v.y = at[1];
  if (col + 2 < p.max_pages) v.z = at[2];
  if (col + 3 < p.max_pages) v.w = at[3];
  return v;
}

DFL_DEV unsigned entries_below(int n) { return n <= 0 ? 0 : n >= 4 ? 15u : (1u << n) - 1; }  // of four

// What becomes of row b: it keeps its entries (src = b), or goes on as row src.
struct Step {
  int src, len;   // -1: empty; its new length
  int had, has;   // pages before and after
  bool bad;
};
DFL_DEV Step step_of(const Pool& p, const int* parents, int b) {
  Step s;
  s.src = parents[b];
  const int mine = p.lens[b];
  const bool any = s.src >= 0 && s.src < p.batch;
  s.len = any ? p.lens[s.src] : 0;
  s.bad = s.src != b && ((!any && s.src != -1) || !len_fits(p, s.len) || !len_fits(p, mine));
  if (s.bad) s.src = b;
  if (s.src == b) s.len = mine;
  s.had = pages_of(mine, p.shift);
  s.has = pages_of(s.len, p.shift);
  return s;
}

// Four entries of a row: the new ones in place of the old ones, and the counts.
DFL_DEV void change_entries(const Pool& p, int b, int col, const Step& s, const int4& now, const int4& was, bool vec) {
  const int w[4] = {was.x, was.y, was.z, was.w}, n[4] = {now.x, now.y, now.z, now.w};
  int out[4];
  unsigned differ = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool held = col + j < s.had, holds = col + j < s.has;
    out[j] = holds ? n[j] : held ? -1 : w[j];
    differ |= (held != holds || (held && w[j] != n[j])) << j;
  }
  if (!differ) return;
  int* at = p.table + b * p.stride + col;
  count_entries(p, n, differ & entries_below(s.has - col), w, differ & entries_below(s.had - col), true);
  if (vec && col + 4 <= p.max_pages) {
    *reinterpret_cast<int4*>(at) = make_int4(out[0], out[1], out[2], out[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < max(s.has, s.had)) at[j] = out[j];
  }
}

// Whether this is the grid's last CTA here, which finds what the others have done
// and read done; the count is back at 0 behind it.
DFL_DEV bool last_of(uint32_t* ticket) {
  unsigned old;
  asm volatile("atom.inc.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(ticket), "r"(gridDim.x - 1) : "memory");
  return old == gridDim.x - 1;
}

// ONE: a unit of four entries a thread, in registers; else in shared memory [units].
template <bool ONE>
__global__ void __launch_bounds__(FORK_THREADS, 1) k_fork(const Pool p, const int* parents, int cols, bool vec) {
  extern __shared__ __align__(16) int4 rows[];
  pdl_launch_dependents();
  pdl_wait();
  const int col0 = blockIdx.x * cols, quads = cols >> 2, units = p.batch * quads;
  const int tid = threadIdx.x;
  // the lengths: the first column's threads of each row have them
  if (ONE) {
    const int b = tid / quads, col = col0 + 4 * (tid - b * quads);
    Step s = {};
    int4 now = make_int4(-1, -1, -1, -1), was = now;
    if (tid < units) {
      s = step_of(p, parents, b);
      if (s.src != b) {
        if (col < s.has) now = load_entries(p, s.src, col, vec);
        if (col < max(s.has, s.had)) was = load_entries(p, b, col, vec);
      }
    }
    __syncthreads();
    if (tid < units && s.src != b && col < max(s.has, s.had)) change_entries(p, b, col, s, now, was, vec);
    if (tid < units && s.bad && col == 0) dev_error(p.status, DFLASH_DEV_ARG);
    __shared__ bool last;
    if (gridDim.x > 1) {
      if (tid == 0) last = last_of(p.status + 1);
      __syncthreads();
      if (!last) return;
    }
    if (tid < units && tid == b * quads && s.src != b) p.lens[b] = s.len;
  } else {
#pragma unroll 1
    for (int u = tid; u < units; u += FORK_THREADS) {
      const int b = u / quads, col = col0 + 4 * (u - b * quads);
      const Step s = step_of(p, parents, b);
      if (s.src != b && col < s.has) rows[u] = load_entries(p, s.src, col, vec);
      if (s.bad && col == 0) dev_error(p.status, DFLASH_DEV_ARG);
    }
    __syncthreads();
#pragma unroll 1
    for (int u = tid; u < units; u += FORK_THREADS) {
      const int b = u / quads, col = col0 + 4 * (u - b * quads);
      const Step s = step_of(p, parents, b);
      if (s.src != b && col < max(s.has, s.had)) change_entries(p, b, col, s, rows[u], load_entries(p, b, col, vec), vec);
    }
    __shared__ bool last;
    __syncthreads();
    if (tid == 0) last = last_of(p.status + 1);
    __syncthreads();
    if (!last) return;
    int* lens = reinterpret_cast<int*>(rows);
#pragma unroll 1
    for (int b = tid; b < p.batch; b += FORK_THREADS) lens[b] = step_of(p, parents, b).len;
    __syncthreads();
#pragma unroll 1
    for (int b = tid; b < p.batch; b += FORK_THREADS) p.lens[b] = lens[b];
  }
}

// ------------------------------------------------------------------ scans of refs
//
// resize and compact run as one cluster, each warp with a part of refs, 128
// pages a step; ranks go from warp to warp and from CTA to CTA.
constexpr int SCAN_THREADS = 1024;
constexpr int SCAN_WARPS = SCAN_THREADS / 32;
constexpr int SCAN_CTAS = 8;  // of a cluster, at most (the portable limit)

DFL_DEV uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// behind: what is read behind the end.
DFL_DEV int4 load_refs(const int* refs, int i, int end, bool vec, int behind) {
  if (vec && i + 4 <= end) return __ldcg(reinterpret_cast<const int4*>(refs + i));
  int4 v = make_int4(behind, behind, behind, behind);
  if (i < end) v.x = __ldcg(refs + i);
  if (i + 1 < end) v.y = __ldcg(refs + i + 1);
  if (i + 2 < end) v.z = __ldcg(refs + i + 2);
  if (i + 3 < end) v.w = __ldcg(refs + i + 3);
  return v;
}

DFL_DEV int warp_total(int v) { return __reduce_add_sync(0xffffffffu, v); }
// Sum of the lower lanes' values.
DFL_DEV int warp_before(int v) {
  const int lane = threadIdx.x & 31;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  return s - v;
}

// Every warp's count (one value a warp, the same in its lanes) summed over the
// warps before it in the cluster, and over all.  buf: [SCAN_WARPS + 1], the
// caller's own for each use.  Contains a cluster barrier: what was read before it
// anywhere may be written behind it.
struct Before {
  int before, total;
};
DFL_DEV Before cluster_before(int count, int* buf, int ctas, int rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[warp] = count;
  __syncthreads();
  if (warp == 0) {
    const int t = warp_total(buf[lane]);
    if (lane == 0) buf[SCAN_WARPS] = t;
  }
  Before r;
  r.before = warp_total(lane < warp ? buf[lane] : 0);
  __syncwarp();
  cluster_sync_all();
  const int mine = lane < ctas ? (int)ld_dsmem_u32(dsmem_addr(smem_u32(buf + SCAN_WARPS), lane)) : 0;
  r.total = warp_total(mine);
  r.before += warp_total(lane < rank ? mine : 0);
  return r;
}

// The pages of a warp: [first, end), whole steps of 128.
struct Part {
  int first, end;
};
DFL_DEV Part scan_part(int n_pages, int ctas, int rank) {
  const int warps = ctas * SCAN_WARPS, me = rank * SCAN_WARPS + (threadIdx.x >> 5);
  const int steps = (n_pages + 127) >> 7, each = (steps + warps - 1) / warps;
  Part r;
  r.first = min(n_pages, me * each * 128);
  r.end = min(n_pages, r.first + each * 128);
  return r;
}

// ------------------------------------------------------------------ resize
//
// One cluster.  Every CTA goes through the whole batch by itself (who shares a last
// page with whom, pages taken before each sequence), then through its part of refs;
// one exchange of counts gives every free page its rank, and a search in the batch
// the place that it goes to.  Nothing is written before that exchange, so a call
// that does not fit changes nothing.
// Bound by latency: 64 requests for 16 positions more in a pool of 3,700 pages 4.7
// us.  512 beams for one more over 24,000 pages, some 140 with a copy of a shared last
// page, while 104 leave with 27,000 entries: 13.4 us, about 5 of them the leavers' counts,
// which eight SMs take at about two entries a cycle (16 us in a pool with pins, where each
// count is read before it is changed); a second launch with all SMs would cost every
// other call 3 us of launching and waiting.  refs are what a large pool costs: 2^20
// pages 13 us, 2^24 204.

// Exclusive sum over the block of a value a thread (need in the low 48 bits,
// copies above).  buf: [SCAN_WARPS + 1].
DFL_DEV unsigned long long block_before(unsigned long long v, unsigned long long* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned long long s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) buf[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const unsigned long long w = buf[lane];
    unsigned long long t = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += o;
    }
    buf[lane] = t - w;
    if (lane == 31) buf[SCAN_WARPS] = t;
  }
  __syncthreads();
  return buf[warp] + s - v;
}

// Shared last pages of growing sequences: page -> their number and the lowest.
struct Sharers {
  int* page;        // [slots], -1 empty
  uint32_t* who;    // number << 16 | lowest sequence (both below 2^14)
  int mask;
};
DFL_DEV int first_slot(const Sharers& h, int page) { return (int)(((unsigned)page * 2654435769u) >> 7) & h.mask; }
DFL_DEV int slot_of(const Sharers& h, int page) {
  int s = first_slot(h, page);
  while (h.page[s] != page) s = (s + 1) & h.mask;  // it was put there
  return s;
}
DFL_DEV void add_sharer(const Sharers& h, int page, int b) {
  int s = first_slot(h, page);
  for (;;) {  // there are as many slots as sequences, at least
    const int was = atomicCAS(h.page + s, -1, page);
    if (was == -1 || was == page) break;
    s = (s + 1) & h.mask;
  }
  uint32_t old = h.who[s], seen;
  do {
    seen = old;
    const uint32_t next = ((seen >> 16) + 1) << 16 | min(seen & 0xffffu, (uint32_t)b);
    old = atomicCAS(h.who + s, seen, next);
  } while (old != seen);
}

// What is known of a sequence in the call, in shared memory.
struct Change {
  int had, has;    // pages; -1: the sequence stays as it is
  int page;        // its last one, where the sequence grows inside one that is shared or pinned (else -1)
  unsigned off;    // pages taken before it; until that is known, the count of `page`
};
// In a word beside it: copies before it, whether `page` is copied and whether it
// is counted (not pinned), positions held of it.
constexpr uint32_t COPIED = 1u << 15, COUNTED = 1u << 14, INSIDE = 0x1ff;

__global__ void __launch_bounds__(SCAN_THREADS, 1) k_resize(const Pool p, const int* new_lens, int* moves, int capacity,
                                                         int ctas, int slots, bool vec, bool tvec) {
  extern __shared__ __align__(16) char smem[];
  __shared__ unsigned long long sums[SCAN_WARPS + 1];
  __shared__ int counts[SCAN_WARPS + 1];
  __shared__ int shrinks, pinned;
  Change* seq = reinterpret_cast<Change*>(smem);                      // [batch]
  uint32_t* copies = reinterpret_cast<uint32_t*>(seq + p.batch);     // [batch]
  Sharers shared;
  shared.page = reinterpret_cast<int*>(copies + p.batch);             // [slots]
  shared.who = reinterpret_cast<uint32_t*>(shared.page + slots);      // [slots]
  shared.mask = slots - 1;
  const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < slots; i += SCAN_THREADS) {
    shared.page[i] = -1;
    shared.who[i] = 0xffffu;
  }
  if (threadIdx.x == 0) shrinks = pinned = 0;
  pdl_wait();
  const Part part = scan_part(p.n_pages, ctas, rank);
  const int4 head = load_refs(p.refs, part.first + 4 * lane, part.end, vec, 1);  // on its way meanwhile; behind the end: held
  __syncthreads();

  // every CTA goes through the whole batch, a thread a few sequences in a row
  const int per = (p.batch + SCAN_THREADS - 1) / SCAN_THREADS;
  const int b0 = min(p.batch, (int)threadIdx.x * per), b1 = min(p.batch, b0 + per);
  const bool speaks = rank == 0;
  bool less = false;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int len = p.lens[b], now = new_lens[b];
    Change c = {-1, -1, -1, 0};
    int inside = 0;
    if (!len_fits(p, len) || !len_fits(p, now)) {
      if (speaks) dev_error(p.status, now < 0 || !len_fits(p, len) ? DFLASH_DEV_ARG : DFLASH_DEV_CAPACITY);
    } else {
      c.had = pages_of(len, p.shift);
      c.has = pages_of(now, p.shift);
      less |= c.has < c.had;
      if (now > len) inside = len & ((1 << p.shift) - 1);
    }
    if (inside) {
      const int page = p.table[b * p.stride + c.had - 1];
      const int r = (unsigned)page < (unsigned)p.n_pages ? p.refs[page] : 0;
      if (r > 1) add_sharer(shared, page, b);
      if (r > 1 || r < 0) c.page = page, c.off = (unsigned)r;
      if (r == 0 && speaks) dev_error(p.status, DFLASH_DEV_PAGE);  // none, or one that nobody holds
    }
    seq[b] = c;
    copies[b] = (uint32_t)inside;
  }
  if (less) shrinks = 1;
  __syncthreads();
  unsigned long long sum = 0;  // pages taken, copies above 2^48
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Change c = seq[b];
    bool copy = false;
    if (c.page >= 0) {
      const int r = (int)c.off;
      copy = r < 0;
      if (!copy) {
        const uint32_t w = shared.who[slot_of(shared, c.page)];
        copy = (int)(w >> 16) < r || (int)(w & 0xffffu) != b;
      }
      if (copy) copies[b] |= COPIED | (r > 0 ? COUNTED : 0);
    }
    sum += (unsigned long long)max(c.has - c.had, 0) + copy + ((unsigned long long)copy << 48);
  }
  unsigned long long before = block_before(sum, sums);
  const unsigned long long all = sums[SCAN_WARPS];
  const unsigned long long want = all & ((1ull << 48) - 1);
  const int n_copies = (int)(all >> 48);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Change c = seq[b];
    const uint32_t w = copies[b];
    const bool copy = w & COPIED;
    seq[b].off = (unsigned)before;  // all of them fit if the call does
    copies[b] = (uint32_t)(before >> 48) << 16 | (w & 0xffffu);
    before += (unsigned long long)max(c.has - c.had, 0) + copy + ((unsigned long long)copy << 48);
  }

  // the free pages
  auto refs_at = [&](int i) { return i == part.first ? head : load_refs(p.refs, i + 4 * lane, part.end, vec, 1); };
  int mine = 0;
#pragma unroll 1
  for (int i = part.first; i < part.end; i += 128) {
    const int4 r = refs_at(i);
    mine += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    if (min(min(r.x, r.y), min(r.z, r.w)) < 0) pinned = 1;
  }
  const Before found = cluster_before(warp_total(mine), counts, ctas, rank);
  // whether any page of the pool is pinned: if not, what is given up need not be looked up first
  const bool pins = __any_sync(0xffffffffu, lane < ctas && ld_dsmem_u32(dsmem_addr(smem_u32(&pinned), lane)));
  const bool fits = want <= (unsigned long long)found.total;

  // moves: their number, and nothing behind the last
  const int used = fits ? n_copies : 0;
  const int tid = rank * SCAN_THREADS + threadIdx.x;
  if (tid < 3) moves[tid] = tid == 0 ? used : 0;
#pragma unroll 1
  for (int i = used + 1 + tid; i <= capacity; i += ctas * SCAN_THREADS) {
    moves[3ll * i] = moves[3ll * i + 1] = -1;
    moves[3ll * i + 2] = 0;
  }
  if (!fits) {
    if (tid == 0) dev_error(p.status, DFLASH_DEV_CAPACITY);
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its sums are read
    return;
  }
  int next = found.before;
#pragma unroll 1
  for (int i = part.first; i < part.end && next < (int)want; i += 128) {
    const int4 r = refs_at(i);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    const int n = f[0] + f[1] + f[2] + f[3];
    // the step's free pages in order, then a lane each
    int* list = shared.page + (threadIdx.x >> 5) * 128;  // the sharers are done with
    int at = warp_before(n);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (f[j]) list[at++] = i + 4 * lane + j;
    __syncwarp();
    const int total = min(warp_total(n), (int)want - next);
#pragma unroll 1
    for (int k = lane; k < total; k += 32) {
      const int page = list[k], place = next + k;
      int lo = 0, hi = p.batch;  // the last sequence with off <= place: one that takes pages
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int)seq[mid].off <= place) lo = mid;
        else hi = mid;
      }
      const Change c = seq[lo];
      const uint32_t w = copies[lo];
      const int nth = place - (int)c.off, copy = (w & COPIED) != 0;
      int* row = p.table + lo * p.stride;
      p.refs[page] = 1;
      if (copy && nth == 0) {
        int* m = moves + 3ll * (1 + (w >> 16));
        m[0] = c.page;
        m[1] = page;
        m[2] = w & INSIDE;
        row[c.had - 1] = page;
      } else {
        row[c.had + nth - copy] = page;
      }
    }
    next += total;
  }
  __syncwarp();
  cluster_sync_all();  // the free pages are found, and no length is read any more
  // what is given up, 128 entries a warp at a time, the pages that were copied, and the new lengths
  if (shrinks) {
    const int pieces = (p.max_pages + 127) >> 7, items = p.batch * pieces;
    const int warps = ctas * SCAN_WARPS;
    constexpr int ABREAST = 2;  // pieces of a warp with their loads on their way
#pragma unroll 1
    for (int it = rank * SCAN_WARPS + (threadIdx.x >> 5); it < items; it += ABREAST * warps) {
      int4 v[ABREAST];
      unsigned lost[ABREAST];
      int* row[ABREAST];
#pragma unroll
      for (int u = 0; u < ABREAST; ++u) {
        const int t = it + u * warps, b = t / pieces, i = ((t - b * pieces) << 7) + 4 * lane;
        lost[u] = 0;
        if (t >= items) continue;
        lost[u] = entries_below(seq[b].had - i) & ~entries_below(seq[b].has - i);
        row[u] = p.table + b * p.stride + i;
        if (lost[u]) v[u] = load_entries(p, b, i, tvec);
      }
#pragma unroll
      for (int u = 0; u < ABREAST; ++u) {
        if (!lost[u]) continue;
        const int id[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        count_entries(p, id, 0, id, lost[u], pins);
        if (tvec && lost[u] == 15) {
          *reinterpret_cast<int4*>(row[u]) = make_int4(-1, -1, -1, -1);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (lost[u] >> j & 1) row[u][j] = -1;
        }
      }
    }
  }
#pragma unroll 1
  for (int b = tid; b < p.batch; b += ctas * SCAN_THREADS) {
    const int page[4] = {seq[b].page};
    count_entries(p, page, 0, page, (copies[b] & COPIED) && (copies[b] & COUNTED), false);
    if (seq[b].had >= 0) p.lens[b] = new_lens[b];
  }
}

// ------------------------------------------------------------------ compact
//
// The same scan, with free pages ranked below the border and held ones above it.
// Ranks pair them; moves is the list of pairs, remap their table form.  225 pages with
// 16 rows of 48 entries 4.5 us, 3,501 pages with 32 rows of 68 7.6 us: three exchanges
// of counts and two passes over memory behind one another.  Large pools are gone
// through three times by eight SMs: 2^20 pages 81 us, 2^24 1,364, with nothing to move.

// REMAP_EACH entries of a row, `width` apart, to their pages' new places.
constexpr int REMAP_THREADS = 256;
constexpr int REMAP_EACH = 4;
constexpr int REMAP_PIECES = 2;  // of a warp of the scanning cluster, at most

DFL_DEV void remap_entries(const Pool& p, const int* remap, int b, int i0, int width) {
  const int len = p.lens[b];
  if (!len_fits(p, len)) {
    if (i0 == 0) dev_error(p.status, DFLASH_DEV_ARG);
    return;
  }
  const int held = pages_of(len, p.shift);
  int* row = p.table + b * p.stride;
  int id[REMAP_EACH], to[REMAP_EACH];
#pragma unroll
  for (int j = 0; j < REMAP_EACH; ++j) id[j] = i0 + j * width < held ? row[i0 + j * width] : 0;
#pragma unroll
  for (int j = 0; j < REMAP_EACH; ++j) {
    to[j] = id[j];  // what lies past the held ones stays
    if (i0 + j * width < held) to[j] = (unsigned)id[j] < (unsigned)p.n_pages ? __ldcg(remap + id[j]) : -1;
  }
#pragma unroll
  for (int j = 0; j < REMAP_EACH; ++j) {
    if (to[j] < 0) dev_error(p.status, DFLASH_DEV_PAGE);  // outside the pool, or held and yet free: left as it is
    else if (to[j] != id[j]) row[i0 + j * width] = to[j];
  }
}

__global__ void __launch_bounds__(REMAP_THREADS) k_remap(const Pool p, const int* remap, int blocks_per_row) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x / blocks_per_row, part = blockIdx.x - b * blocks_per_row;
  remap_entries(p, remap, b, part * REMAP_THREADS * REMAP_EACH + threadIdx.x, REMAP_THREADS);
}

// with_table: the table is small enough for the cluster to go through it too.
__global__ void __launch_bounds__(SCAN_THREADS, 1) k_compact(const Pool p, int* moves, int capacity, int* remap, int ctas,
                                                          bool vec, bool with_table) {
  __shared__ int free_counts[SCAN_WARPS + 1], held_counts[SCAN_WARPS + 1], low[SCAN_WARPS + 1];
  const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const Part part = scan_part(p.n_pages, ctas, rank);
  const int4 head = load_refs(p.refs, part.first + 4 * lane, part.end, vec, -1);
  auto refs_at = [&](int i) { return i == part.first ? head : load_refs(p.refs, i + 4 * lane, part.end, vec, -1); };
  int f = 0, h = 0;
#pragma unroll 1
  for (int i = part.first; i < part.end; i += 128) {
    const int4 r = refs_at(i);
    f += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    h += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  const Before holes = cluster_before(warp_total(f), free_counts, ctas, rank);
  const int used = p.n_pages - holes.total;  // pages in use: they shall lie below this
  const Before held = cluster_before(warp_total(h), held_counts, ctas, rank);
  // held pages below `used` stay
  int stay = 0;
#pragma unroll 1
  for (int i = part.first; i < min(part.end, used); i += 128) {
    const int q = i + 4 * lane;
    const int4 r = refs_at(i);
    stay += (r.x > 0 && q < used) + (r.y > 0 && q + 1 < used) + (r.z > 0 && q + 2 < used) + (r.w > 0 && q + 3 < used);
  }
  const int staying = cluster_before(warp_total(stay), low, ctas, rank).total;
  const int n = held.total - staying;  // that move; at least as many free pages lie below `used`
  int hole = holes.before, mover = held.before - staying;
#pragma unroll 1
  for (int i = part.first; i < part.end; i += 128) {
    const int q = i + 4 * lane;
    const int4 v = refs_at(i);
    const int r[4] = {v.x, v.y, v.z, v.w};
    int nf = 0, nh = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) nf += r[j] == 0, nh += r[j] > 0;
    int kf = hole + warp_before(nf), kh = mover + warp_before(nh);
    hole += warp_total(nf);
    mover += warp_total(nh);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int page = q + j;
      if (page >= part.end) break;
      if (r[j] == 0) {
        if (page < used && kf < n) moves[3ll * (1 + kf) + 1] = page;
        ++kf;
        remap[page] = -1;
      } else {
        if (r[j] > 0) {
          if (page >= used) moves[3ll * (1 + kh)] = page;
          ++kh;
        }
        if (r[j] < 0 || page < used) remap[page] = page;
      }
    }
  }
  const int tid = rank * SCAN_THREADS + threadIdx.x, threads = ctas * SCAN_THREADS;
  if (tid < 3) moves[tid] = tid == 0 ? n : 0;
  __syncwarp();
  cluster_sync_all();  // the pairs are whole, and refs are read
  for (int i = 1 + tid; i <= capacity; i += threads) {
    int* m = moves + 3ll * i;
    if (i <= n) {
      const int src = __ldcg(m), dst = __ldcg(m + 1);
      m[2] = 1 << p.shift;
      remap[src] = dst;
      p.refs[dst] = __ldcg(p.refs + src);
      p.refs[src] = 0;
    } else {
      m[0] = m[1] = -1;
      m[2] = 0;
    }
  }
  if (!with_table) return;
  __syncwarp();
  cluster_sync_all();  // remap is whole
  const int per_row = (p.max_pages + 32 * REMAP_EACH - 1) / (32 * REMAP_EACH);  // pieces, a warp each
#pragma unroll 1
  for (int it = tid >> 5; it < per_row * p.batch; it += threads >> 5) {
    const int b = it / per_row;
    remap_entries(p, remap, b, (it - b * per_row) * 32 * REMAP_EACH + lane, 32);
  }
}

// ------------------------------------------------------------------ copy
//
// Bound by memory: every byte is read and written once.  A work item is some
// 8 KB of one page in one pool, four 16-byte vectors a thread in flight; items
// go round the CTAs.  The number of copies is known on the device only.
// 448 last pages, half full on average, in 8 layers (925 MB) 148 us, 6.25 TB/s, 0.92
// of the copy rate; 769 whole pages in 5 layers (2.0 GB) 318 us with the compaction
// before them.  Two vectors a thread in flight 170 us, five blocks of 256 an SM 157,
// a page's chunks next to one another in the round (then whole CTAs have the empty
// ones) 167, bulk copies through a ring in shared memory 152 to 164 (3 to 8 slots of 8
// to 32 KB, 64 to 192 KB an SM on their way); four pages in one layer 2.5 us.
// 400 whole pages of 64 x 8 x 128 in 4 layers (839 MB) 132 us; with heads 136 apart 178;
// heads 129 apart, which take 2 bytes an access, 606; heads of 127 next to one another,
// also 2 bytes, 319.
constexpr int COPY_THREADS = 128;
constexpr int COPY_AHEAD = 4;
constexpr int COPY_CTAS = 16;    // of an SM
constexpr int COPY_CACHES = 64;  // of a launch

struct PoolAt {
  char* data;
  long long page, pos, head;  // strides, bytes
};
struct CopyParams {
  const int* moves;
  int capacity, n_pools, n_pages, page_size;
  int per_head, per_pos;      // vectors
  int chunk, chunks;          // positions of an item, items of a page
  bool flat;                  // positions follow one another
  uint32_t* status;
  PoolAt pool[2 * COPY_CACHES];
};

template <typename V>
__global__ void __launch_bounds__(COPY_THREADS) k_copy_pages(const __grid_constant__ CopyParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int n = min(max(p.moves[0], 0), min(p.capacity, p.n_pages));  // no page is copied to twice
  // the first chunk of every page, then the second: pages of which little is
  // copied then cost every CTA alike
  const unsigned pages = (unsigned)n * (unsigned)p.n_pools;  // of all pools: below 2^31
  if (pages == 0) return;
  const unsigned step = gridDim.x % pages;
  const int step_c = (int)(gridDim.x / pages);
  int c = (int)(blockIdx.x / pages);
  for (unsigned at = blockIdx.x % pages; c < p.chunks; at += step, c += step_c) {
    if (at >= pages) at -= pages, ++c;
    if (c >= p.chunks) break;
    const int m = (int)(at / (unsigned)p.n_pools), which = (int)(at - (unsigned)m * p.n_pools);
    const int* mv = p.moves + 3ll * (m + 1);
    const int src = mv[0], dst = mv[1], count = min(mv[2], p.page_size);
    const int p0 = c * p.chunk;
    if (p0 >= count) continue;
    if ((unsigned)src >= (unsigned)p.n_pages || (unsigned)dst >= (unsigned)p.n_pages) {
      if (threadIdx.x == 0) dev_error(p.status, DFLASH_DEV_PAGE);
      continue;
    }
    const PoolAt& pool = p.pool[which];
    const char* from = pool.data + src * pool.page + p0 * pool.pos;
    char* to = pool.data + dst * pool.page + p0 * pool.pos;
    const int vecs = min(p.chunk, count - p0) * p.per_pos;
    for (int i0 = threadIdx.x; i0 < vecs; i0 += COPY_AHEAD * COPY_THREADS) {
      V v[COPY_AHEAD];
      long long at[COPY_AHEAD];
#pragma unroll
      for (int j = 0; j < COPY_AHEAD; ++j) {
        const int i = i0 + j * COPY_THREADS;
        if (i >= vecs) break;
        if (p.flat) {
          at[j] = (long long)i * sizeof(V);
        } else {
          const int pos = i / p.per_pos, r = i - pos * p.per_pos, head = r / p.per_head;
          at[j] = pos * pool.pos + head * pool.head + (long long)(r - head * p.per_head) * sizeof(V);
        }
        v[j] = *reinterpret_cast<const V*>(from + at[j]);
      }
#pragma unroll
      for (int j = 0; j < COPY_AHEAD; ++j) {
        if (i0 + j * COPY_THREADS >= vecs) break;
        *reinterpret_cast<V*>(to + at[j]) = v[j];
      }
    }
  }
}

// ------------------------------------------------------------------ host

bool words(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

int pool_check(const dflash_page_pool* c) {
  if (!c || !c->refs || !c->page_table || !c->lens || !c->status || c->n_pages < 1 || c->max_pages < 1 || c->batch < 1 ||
      c->table_stride < c->max_pages || c->device < 0 || !words(c->refs) || !words(c->page_table) || !words(c->lens) ||
      !words(c->status))
    return DFLASH_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return DFLASH_ERR_SHAPE;
  if (c->batch > DFLASH_POOL_MAX_BATCH || c->n_pages > DFLASH_POOL_MAX_PAGES) return DFLASH_ERR_CAPACITY;
  return DFLASH_OK;
}

Pool pool_of(const dflash_page_pool* c) {
  // entries that no length reaches are never looked at: at most 2^27, far from where indexes end
  const int reached = 0x7fffffff / c->page_size + 1;
  return {c->refs, c->page_table, c->table_stride, c->lens, c->status, c->n_pages, page_shift(c->page_size),
          std::min(c->max_pages, reached), c->batch};
}

struct PoolParts {
  Strided refs, table, lens, status;
};
PoolParts pool_parts(const dflash_page_pool* c) {
  return {strided_ints(c->refs, c->n_pages),
          strided(c->page_table, 4ll * c->max_pages, {{4 * c->table_stride, c->batch}}), strided_ints(c->lens, c->batch),
          strided_ints(reinterpret_cast<const int32_t*>(c->status), 2)};
}

bool table_vec(const dflash_page_pool* c) {
  return (reinterpret_cast<uintptr_t>(c->page_table) & 15) == 0 && c->table_stride % 4 == 0;
}

template <typename... P, typename... A>
int launch(void (*k)(P...), dim3 grid, int threads, size_t smem, int cluster, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cuda_status(cudaLaunchKernelEx(&cfg, k, static_cast<P>(args)...));
}

constexpr int MAX_MOVES = 1 << 30;  // of a list that a call fills

// CTAs that scan refs: a step of 128 pages a warp each, at most eight.
int scan_ctas(int n_pages) {
  int c = 1;
  while (c < SCAN_CTAS && c * SCAN_WARPS * 128 < n_pages) c *= 2;
  return c;
}

// Slots of the shared pages: twice the sequences, or as many as there are at least where that does not fit.
int resize_slots(int batch) {
  int slots = SCAN_WARPS * 128 / 2;  // their memory serves the lists of free pages afterwards
  while (slots < (batch > 4096 ? batch : 2 * batch)) slots *= 2;
  return slots;
}
size_t resize_smem(int batch) { return (sizeof(Change) + 4ull) * batch + 8ull * resize_slots(batch); }

}  // namespace

extern "C" {

int dflash_pool_read_status(const dflash_page_pool* c, uint32_t* out) {
  if (!out) return DFLASH_ERR_INVALID_ARG;
  if (int e = pool_check(c)) return e;
  return read_status_word(c->status, c->device, out);
}

int dflash_pages_fork(const dflash_page_pool* c, const int32_t* parents, void* stream) {
  if (int e = pool_check(c)) return e;
  if (!parents || !words(parents)) return DFLASH_ERR_INVALID_ARG;
  const PoolParts w = pool_parts(c);
  if (!apart({w.refs, w.table, w.lens, w.status}, {strided_ints(parents, c->batch)})) return DFLASH_ERR_INVALID_ARG;
  // Columns of a CTA: as many as give every thread one unit of four entries, but
  // no fewer than four: larger batches take several units a thread.
  const Pool p = pool_of(c);
  int cols = 4;
  while (cols * 2 * p.batch <= 4 * FORK_THREADS && cols < p.max_pages) cols *= 2;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  const dim3 grid((unsigned)((p.max_pages + cols - 1) / cols));
  const int units = p.batch * (cols / 4);
  if (units <= FORK_THREADS)
    return launch(k_fork<true>, grid, (units + 31) / 32 * 32, 0, 1, stream, p, parents, cols, table_vec(c));
  if (int e = cuda_status(cudaFuncSetAttribute(k_fork<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               DFLASH_POOL_MAX_BATCH * (int)sizeof(int4))))
    return e;
  return launch(k_fork<false>, grid, FORK_THREADS, units * sizeof(int4), 1, stream, p, parents, cols, table_vec(c));
}

int dflash_pages_resize(const dflash_page_pool* c, const int32_t* new_lens, int32_t* moves, int32_t capacity,
                        void* stream) {
  if (int e = pool_check(c)) return e;
  if (!new_lens || !moves || capacity < 0 || !words(new_lens) || !words(moves)) return DFLASH_ERR_INVALID_ARG;
  if (capacity < c->batch || capacity > MAX_MOVES) return DFLASH_ERR_CAPACITY;
  const PoolParts w = pool_parts(c);
  if (!apart({w.refs, w.table, w.lens, w.status, strided_ints(moves, 3 + 3ll * capacity)},
             {strided_ints(new_lens, c->batch)}))
    return DFLASH_ERR_INVALID_ARG;
  const Pool p = pool_of(c);
  if ((long long)p.batch * ((p.max_pages + 127) / 128) > 0x7fffffffll) return DFLASH_ERR_CAPACITY;
  const size_t smem = resize_smem(c->batch);
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  if (smem > 48 * 1024)
    if (int e = cuda_status(cudaFuncSetAttribute(k_resize, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)resize_smem(DFLASH_POOL_MAX_BATCH))))
      return e;
  const int ctas = scan_ctas(c->n_pages);
  return launch(k_resize, dim3((unsigned)ctas), SCAN_THREADS, smem, ctas, stream, p, new_lens, moves, capacity,
                ctas, resize_slots(c->batch), (reinterpret_cast<uintptr_t>(c->refs) & 15) == 0, table_vec(c));
}

int dflash_pages_compact(const dflash_page_pool* c, int32_t* moves, int32_t capacity, int32_t* remap, void* stream) {
  if (int e = pool_check(c)) return e;
  if (!moves || !remap || capacity < 0 || !words(moves) || !words(remap)) return DFLASH_ERR_INVALID_ARG;
  if (capacity < c->n_pages / 2 || capacity > MAX_MOVES) return DFLASH_ERR_CAPACITY;
  const PoolParts w = pool_parts(c);
  if (!apart({w.refs, w.table, w.status, strided_ints(moves, 3 + 3ll * capacity), strided_ints(remap, c->n_pages)}, {w.lens}))
    return DFLASH_ERR_INVALID_ARG;
  const Pool p = pool_of(c);
  const int per_row = (p.max_pages + REMAP_THREADS * REMAP_EACH - 1) / (REMAP_THREADS * REMAP_EACH);
  const long long blocks = (long long)per_row * p.batch;
  if (blocks > 0x7fffffffll) return DFLASH_ERR_CAPACITY;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  // A table of some pieces a warp is gone through by the same cluster; a larger one
  // by a grid of its own, which takes a launch more and has all SMs.
  const long long pieces = (long long)((p.max_pages + 32 * REMAP_EACH - 1) / (32 * REMAP_EACH)) * p.batch;
  const int ctas = scan_ctas((int)std::min<long long>(DFLASH_POOL_MAX_PAGES, std::max<long long>(c->n_pages, pieces * 128)));
  const bool with_table = pieces <= REMAP_PIECES * SCAN_WARPS * ctas;
  if (int e = launch(k_compact, dim3((unsigned)ctas), SCAN_THREADS, 0, ctas, stream, p, moves, capacity, remap, ctas,
                     (reinterpret_cast<uintptr_t>(c->refs) & 15) == 0, with_table))
    return e;
  if (with_table) return DFLASH_OK;
  return launch(k_remap, dim3((unsigned)blocks), REMAP_THREADS, 0, 1, stream, p, remap, per_row);
}

int dflash_pages_copy(const dflash_paged_cache* caches, int32_t n_caches, const int32_t* moves, int32_t capacity,
                      void* stream) {
  if (n_caches < 0 || capacity < 0 || !moves || !words(moves) || (n_caches > 0 && !caches)) return DFLASH_ERR_INVALID_ARG;
  if (n_caches == 0 || capacity == 0) return DFLASH_OK;
  const dflash_paged_cache& c0 = caches[0];
  bool vec = true, flat = true;
  for (int i = 0; i < n_caches; ++i) {
    const dflash_paged_cache& c = caches[i];
    if (int e = paged_cache_check(&c)) return e;
    if (c.n_pages != c0.n_pages || c.page_size != c0.page_size || c.kv_heads != c0.kv_heads || c.head_dim != c0.head_dim ||
        c.device != c0.device || c.head_dim < 1 || ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 1) ||
        !words(c.status))
      return DFLASH_ERR_INVALID_ARG;
    const Strided k = strided_pool(&c, false), v = strided_pool(&c, true);
    if (!apart({k, v}, {strided_ints(moves, 3 + 3ll * capacity),
                        strided_ints(reinterpret_cast<const int32_t*>(c0.status), 1)}))
      return DFLASH_ERR_INVALID_ARG;
    const dflash_rows pk = {c.k, c.k_pos_stride, c.k_head_stride}, pv = {c.v, c.v_pos_stride, c.v_head_stride};
    for (const dflash_rows* r : {&pk, &pv}) {
      vec = vec && (reinterpret_cast<uintptr_t>(r->data) & 15) == 0 && r->row_stride % 8 == 0 && r->head_stride % 8 == 0;
      flat = flat && (r->head_stride == c.head_dim || c.kv_heads == 1) && r->row_stride == (int64_t)c.kv_heads * c.head_dim;
    }
    vec = vec && c.k_page_stride % 8 == 0 && c.v_page_stride % 8 == 0;
  }
  vec = vec && c0.head_dim % 8 == 0;
  const int vb = vec ? 16 : 2;
  if ((long long)c0.kv_heads * c0.head_dim * c0.page_size > (1 << 30)) return DFLASH_ERR_SHAPE;
  CopyParams p;
  p.moves = moves;
  p.capacity = capacity;
  p.n_pages = c0.n_pages;
  p.page_size = c0.page_size;
  p.per_head = c0.head_dim * 2 / vb;
  p.per_pos = p.per_head * c0.kv_heads;
  p.chunk = std::max(1, std::min(c0.page_size, COPY_THREADS * COPY_AHEAD / p.per_pos));
  p.chunks = (c0.page_size + p.chunk - 1) / p.chunk;
  p.flat = flat;
  p.status = c0.status;
  const long long most = std::min(capacity, c0.n_pages);
  const int per = (int)std::min<long long>(COPY_CACHES, 0x3fffffffll / most);  // page copies of a launch fit 31 bits
  if (per < 1) return DFLASH_ERR_CAPACITY;
  DeviceGuard guard(c0.device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  for (int at = 0; at < n_caches; at += per) {
    const int n = std::min(per, n_caches - at);
    p.n_pools = 2 * n;
    for (int i = 0; i < n; ++i) {
      const dflash_paged_cache& c = caches[at + i];
      p.pool[2 * i] = {static_cast<char*>(c.k), 2 * c.k_page_stride, 2 * c.k_pos_stride, 2 * c.k_head_stride};
      p.pool[2 * i + 1] = {static_cast<char*>(c.v), 2 * c.v_page_stride, 2 * c.v_pos_stride, 2 * c.v_head_stride};
    }
    const unsigned grid = (unsigned)std::min<long long>(152 * COPY_CTAS, most * p.n_pools * p.chunks);
    const int e = vec ? launch(k_copy_pages<uint4>, dim3(grid), COPY_THREADS, 0, 1, stream, p)
                      : launch(k_copy_pages<uint16_t>, dim3(grid), COPY_THREADS, 0, 1, stream, p);
    if (e) return e;
  }
  return DFLASH_OK;
}

}  // extern "C"

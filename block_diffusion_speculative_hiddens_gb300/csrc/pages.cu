// The pages of a caller's paged cache: who holds them, the copies that sharing
// takes, and the copies' bytes.
//
// A pool's state is refs (holders of each page), a table and lens.  There is no
// free list: a free page is one with refs 0, found by a scan, so nothing can fall
// out of step with the counts, the pages handed out do not depend on the order of
// atomics (the lowest free ones, by rank), and compact needs no other view.
#include <algorithm>
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

// One holder more or less of a page.  Whether a page is pinned does not change
// during a call, and a page given up has a holder until then.
DFL_DEV void hold(const Pool& p, int id) {
  if ((unsigned)id >= (unsigned)p.n_pages) dev_error(p.status, DFLASH_DEV_PAGE);
  else if (__ldcg(p.refs + id) >= 0) atomicAdd(p.refs + id, 1);
}
DFL_DEV void give_up(const Pool& p, int id) {
  if ((unsigned)id >= (unsigned)p.n_pages) {
    dev_error(p.status, DFLASH_DEV_PAGE);
    return;
  }
  const int r = __ldcg(p.refs + id);
  if (r > 0) atomicSub(p.refs + id, 1);
  else if (r == 0) dev_error(p.status, DFLASH_DEV_PAGE);
}

// ------------------------------------------------------------------ fork
//
// A column of the table depends on the same column alone, so a CTA takes a few
// columns of every row: it loads what the rows will hold, and writes after a
// barrier; the table is its own output without a second copy.  Rows and entries
// that stay as they are (a long shared prefix) cost their reads only.  The
// lengths, which every CTA reads, are written by the last one.
constexpr int FORK_THREADS = 1024;
constexpr int FORK_UNITS = DFLASH_POOL_MAX_BATCH / FORK_THREADS;  // of four entries, a thread

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

// What row b becomes: its parent's row, or -1 (empty), or b itself (as it is).
DFL_DEV int parent_of(const Pool& p, const int* parents, int b, int& len, bool& bad) {
  const int src = parents[b];
  bad = false;
  if (src == b) return b;
  len = 0;
  const int mine = p.lens[b];
  if (src >= 0 && src < p.batch) len = p.lens[src];
  if (src < -1 || src >= p.batch || !len_fits(p, len) || !len_fits(p, mine)) {
    bad = true;
    return b;
  }
  return src;
}

__global__ void __launch_bounds__(FORK_THREADS) k_fork(const Pool p, const int* parents, int cols, bool vec) {
  pdl_launch_dependents();
  pdl_wait();
  const int col0 = blockIdx.x * cols, quads = cols >> 2, units = p.batch * quads;
  int4 now[FORK_UNITS];
#pragma unroll
  for (int i = 0; i < FORK_UNITS; ++i) {
    const int u = threadIdx.x + i * FORK_THREADS;
    if (u >= units) break;
    const int b = u / quads, col = col0 + 4 * (u - b * quads);
    int len;
    bool bad;
    const int src = parent_of(p, parents, b, len, bad);
    if (bad && blockIdx.x == 0 && col == 0) dev_error(p.status, DFLASH_DEV_ARG);
    if (src != b && src >= 0 && col < pages_of(len, p.shift)) now[i] = load_entries(p, src, col, vec);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FORK_UNITS; ++i) {
    const int u = threadIdx.x + i * FORK_THREADS;
    if (u >= units) break;
    const int b = u / quads, col = col0 + 4 * (u - b * quads);
    int len;
    bool bad;
    const int src = parent_of(p, parents, b, len, bad);
    if (src == b) continue;
    const int has = src < 0 ? 0 : pages_of(len, p.shift), had = pages_of(p.lens[b], p.shift);
    if (col >= max(has, had)) continue;
    const int4 was = load_entries(p, b, col, vec);
    const int w[4] = {was.x, was.y, was.z, was.w}, n[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
    int out[4];
    bool changed = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool held = col + j < had, holds = col + j < has;
      out[j] = holds ? n[j] : held ? -1 : w[j];
      if (held && holds && w[j] == n[j]) continue;
      changed |= held || holds;
      if (holds) hold(p, n[j]);
      if (held) give_up(p, w[j]);
    }
    if (!changed) continue;
    int* at = p.table + b * p.stride + col;
    if (vec && col + 4 <= p.max_pages) {
      *reinterpret_cast<int4*>(at) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < max(has, had)) at[j] = out[j];
    }
  }
  // the lengths, once every CTA has read them
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicInc(p.status + 1, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  int lens[FORK_UNITS];
#pragma unroll
  for (int i = 0; i < FORK_UNITS; ++i) {
    const int b = threadIdx.x + i * FORK_THREADS;
    if (b >= p.batch) break;
    bool bad;
    if (parent_of(p, parents, b, lens[i], bad) == b) lens[i] = p.lens[b];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < FORK_UNITS; ++i) {
    const int b = threadIdx.x + i * FORK_THREADS;
    if (b >= p.batch) break;
    p.lens[b] = lens[i];
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

DFL_DEV int4 load_refs(const int* refs, int i, int end, bool vec) {
  if (vec && i + 4 <= end) return __ldcg(reinterpret_cast<const int4*>(refs + i));
  // behind the end: pages that are neither free nor held
  int4 v = make_int4(-1, -1, -1, -1);
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

// What a sequence asks for.
struct Change {
  bool valid;
  int had, has;  // pages
  int inside;    // positions of the last page held, where the sequence grows inside it (else 0)
};
DFL_DEV Change change_of(const Pool& p, int len, int now) {
  Change c = {};
  c.valid = len_fits(p, len) && len_fits(p, now);
  if (!c.valid) return c;
  c.had = pages_of(len, p.shift);
  c.has = pages_of(now, p.shift);
  if (now > len) c.inside = len & ((1 << p.shift) - 1);
  return c;
}

// Shared last pages of growing sequences: page -> their number and the lowest.
struct Sharers {
  int* page;        // [slots], -1 empty
  uint32_t* who;    // number << 16 | lowest sequence (both below 2^14)
  int mask;
};
DFL_DEV int slot_of(const Sharers& h, int page) {
  int s = (int)(((unsigned)page * 2654435769u) >> 7) & h.mask;
  while (h.page[s] != page) s = (s + 1) & h.mask;  // it was put there
  return s;
}
DFL_DEV void add_sharer(const Sharers& h, int page, int b) {
  int s = (int)(((unsigned)page * 2654435769u) >> 7) & h.mask;
  for (;;) {  // at most half of the slots are taken
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

__global__ void __launch_bounds__(SCAN_THREADS) k_resize(const Pool p, const int* new_lens, int* moves, int capacity,
                                                         int ctas, int slots, bool vec) {
  extern __shared__ __align__(16) char smem[];
  __shared__ unsigned long long sums[SCAN_WARPS + 1];
  __shared__ int counts[SCAN_WARPS + 1];
  unsigned* off = reinterpret_cast<unsigned*>(smem);                // [batch + 1] pages taken before a sequence
  Sharers shared;
  shared.page = reinterpret_cast<int*>(off + p.batch + 1);          // [slots]
  shared.who = reinterpret_cast<uint32_t*>(shared.page + slots);    // [slots]
  shared.mask = slots - 1;
  uint16_t* copies = reinterpret_cast<uint16_t*>(shared.who + slots);  // [batch] copies up to and with a sequence's
  const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < slots; i += SCAN_THREADS) {
    shared.page[i] = -1;
    shared.who[i] = 0xffffu;
  }
  pdl_wait();
  __syncthreads();

  // every CTA goes through the whole batch, a thread a few sequences in a row
  const int per = (p.batch + SCAN_THREADS - 1) / SCAN_THREADS;
  const int b0 = min(p.batch, (int)threadIdx.x * per), b1 = min(p.batch, b0 + per);
  const bool speaks = rank == 0;
  for (int b = b0; b < b1; ++b) {
    const int len = p.lens[b], now = new_lens[b];
    const Change c = change_of(p, len, now);
    if (!c.valid && speaks)
      dev_error(p.status, len < 0 || now < 0 || !len_fits(p, len) ? DFLASH_DEV_ARG : DFLASH_DEV_CAPACITY);
    if (c.inside) {
      const int page = p.table[b * p.stride + c.had - 1];
      if ((unsigned)page >= (unsigned)p.n_pages) {
        if (speaks) dev_error(p.status, DFLASH_DEV_PAGE);
      } else {
        const int r = p.refs[page];
        if (r > 1) add_sharer(shared, page, b);
        else if (r == 0 && speaks) dev_error(p.status, DFLASH_DEV_PAGE);
      }
    }
  }
  __syncthreads();
  unsigned long long sum = 0;
  auto takes = [&](int b, unsigned long long& need, bool& copy) {
    const Change c = change_of(p, p.lens[b], new_lens[b]);
    copy = false;
    if (c.inside) {
      const int page = p.table[b * p.stride + c.had - 1];
      if ((unsigned)page < (unsigned)p.n_pages) {
        const int r = p.refs[page];
        if (r > 1) {
          const uint32_t w = shared.who[slot_of(shared, page)];
          copy = (int)(w >> 16) < r || (int)(w & 0xffffu) != b;
        } else {
          copy = r < 0;
        }
      }
    }
    need = (unsigned long long)max(c.has - c.had, 0) + copy;
  };
  for (int b = b0; b < b1; ++b) {
    unsigned long long need;
    bool copy;
    takes(b, need, copy);
    sum += need | (unsigned long long)copy << 48;
  }
  unsigned long long before = block_before(sum, sums);
  const unsigned long long all = sums[SCAN_WARPS];
  const unsigned long long want = all & ((1ull << 48) - 1);
  const int n_copies = (int)(all >> 48);
  if (want <= (unsigned long long)p.n_pages) {  // else it does not fit anyway, nor 32 bits
    for (int b = b0; b < b1; ++b) {
      unsigned long long need;
      bool copy;
      takes(b, need, copy);
      off[b] = (unsigned)before;
      before += need | (unsigned long long)copy << 48;
      copies[b] = (uint16_t)(before >> 48);
    }
    if (threadIdx.x == 0) off[p.batch] = (unsigned)want;
  }

  // the free pages
  const int lane = threadIdx.x & 31;
  const Part part = scan_part(p.n_pages, ctas, rank);
  int mine = 0;
  for (int i = part.first; i < part.end; i += 128) {
    const int4 r = load_refs(p.refs, i + 4 * lane, part.end, vec);
    mine += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  const Before found = cluster_before(warp_total(mine), counts, ctas, rank);
  const bool fits = want <= (unsigned long long)found.total;

  // moves: their number, and nothing behind the last
  const int used = fits ? n_copies : 0;
  const int tid = rank * SCAN_THREADS + threadIdx.x;
  if (tid < 3) moves[tid] = tid == 0 ? used : 0;
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
  for (int i = part.first; i < part.end && next < (int)want; i += 128) {
    const int4 r = load_refs(p.refs, i + 4 * lane, part.end, vec);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    const int n = f[0] + f[1] + f[2] + f[3];
    int place = next + warp_before(n);
    next += warp_total(n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!f[j]) continue;
      const int k = place++;
      if (k >= (int)want) continue;
      const int page = i + 4 * lane + j;
      int lo = 0, hi = p.batch;  // the last b with off[b] <= k: one that takes pages
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int)off[mid] <= k) lo = mid;
        else hi = mid;
      }
      const int b = lo, len = p.lens[b];
      const int had = pages_of(len, p.shift);
      const bool copy = copies[b] != (b > 0 ? copies[b - 1] : 0);
      int* row = p.table + b * p.stride;
      const int at = k - (int)off[b];
      p.refs[page] = 1;
      if (copy && at == 0) {
        const int from = row[had - 1];
        int* m = moves + 3ll * copies[b];
        m[0] = from;
        m[1] = page;
        m[2] = len & ((1 << p.shift) - 1);
        row[had - 1] = page;
        give_up(p, from);
      } else {
        row[had + at - copy] = page;
      }
    }
  }
  __syncwarp();
  cluster_sync_all();  // the free pages are found, and no length is read any more
  // what is given up, a warp a sequence, and the new lengths
  for (int b = rank * SCAN_WARPS + (threadIdx.x >> 5); b < p.batch; b += ctas * SCAN_WARPS) {
    const int len = p.lens[b], now = new_lens[b];
    const Change c = change_of(p, len, now);
    __syncwarp();
    if (!c.valid) continue;
    for (int i = c.has + lane; i < c.had; i += 32) {
      int* at = p.table + b * p.stride + i;
      give_up(p, *at);
      *at = -1;
    }
    if (lane == 0) p.lens[b] = now;
  }
}

// ------------------------------------------------------------------ compact

__global__ void __launch_bounds__(SCAN_THREADS) k_compact(const Pool p, int* moves, int capacity, int* remap, int ctas,
                                                          bool vec) {
  __shared__ int free_counts[SCAN_WARPS + 1], held_counts[SCAN_WARPS + 1], low[SCAN_WARPS + 1];
  const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const Part part = scan_part(p.n_pages, ctas, rank);
  int f = 0, h = 0;
  for (int i = part.first; i < part.end; i += 128) {
    const int4 r = load_refs(p.refs, i + 4 * lane, part.end, vec);
    f += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    h += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  const Before holes = cluster_before(warp_total(f), free_counts, ctas, rank);
  const int used = p.n_pages - holes.total;  // pages in use: they shall lie below this
  const Before held = cluster_before(warp_total(h), held_counts, ctas, rank);
  // held pages below `used` stay
  int stay = 0;
  for (int i = part.first; i < min(part.end, used); i += 128) {
    const int q = i + 4 * lane;
    const int4 r = load_refs(p.refs, q, part.end, vec);
    stay += (r.x > 0 && q < used) + (r.y > 0 && q + 1 < used) + (r.z > 0 && q + 2 < used) + (r.w > 0 && q + 3 < used);
  }
  const int staying = cluster_before(warp_total(stay), low, ctas, rank).total;
  const int n = held.total - staying;  // that move; at least as many free pages lie below `used`
  int hole = holes.before, mover = held.before - staying;
  for (int i = part.first; i < part.end; i += 128) {
    const int q = i + 4 * lane;
    const int4 v = load_refs(p.refs, q, part.end, vec);
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
}

constexpr int REMAP_THREADS = 256;
constexpr int REMAP_EACH = 4;  // entries of a thread, a block's width apart

__global__ void __launch_bounds__(REMAP_THREADS) k_remap(const Pool p, const int* remap, int blocks_per_row) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x / blocks_per_row, part = blockIdx.x - b * blocks_per_row;
  const int len = p.lens[b];
  if (!len_fits(p, len)) {
    if (part == 0 && threadIdx.x == 0) dev_error(p.status, DFLASH_DEV_ARG);
    return;
  }
  const int held = pages_of(len, p.shift);
  int* row = p.table + b * p.stride;
  const int i0 = part * REMAP_THREADS * REMAP_EACH + threadIdx.x;
  int id[REMAP_EACH];
#pragma unroll
  for (int j = 0; j < REMAP_EACH; ++j) {
    const int i = i0 + j * REMAP_THREADS;
    id[j] = i < held ? row[i] : -2;
  }
#pragma unroll
  for (int j = 0; j < REMAP_EACH; ++j) {
    if (id[j] == -2 && i0 + j * REMAP_THREADS >= held) continue;
    if ((unsigned)id[j] >= (unsigned)p.n_pages) {
      dev_error(p.status, DFLASH_DEV_PAGE);
      continue;
    }
    const int to = remap[id[j]];
    if (to < 0) dev_error(p.status, DFLASH_DEV_PAGE);  // held, and yet free: left as it is
    else if (to != id[j]) row[i0 + j * REMAP_THREADS] = to;
  }
}

// ------------------------------------------------------------------ copy
//
// Bound by memory: every byte is read and written once.  A work item is some
// 16 KB of one page in one pool, four 16-byte vectors a thread in flight; items
// go round the CTAs.  The number of copies is known on the device only.
constexpr int COPY_THREADS = 256;
constexpr int COPY_AHEAD = 4;
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
  const int n = min(max(p.moves[0], 0), p.capacity);
  const long long items = (long long)n * p.n_pools * p.chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const long long mp = it / p.chunks;
    const int c = (int)(it - mp * p.chunks);
    const int m = (int)(mp / p.n_pools), which = (int)(mp - (long long)m * p.n_pools);
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
  return {c->refs, c->page_table, c->table_stride, c->lens, c->status, c->n_pages, page_shift(c->page_size),
          c->max_pages, c->batch};
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

// CTAs that scan refs: a step of 128 pages a warp each, at most eight.
int scan_ctas(int n_pages) {
  int c = 1;
  while (c < SCAN_CTAS && c * SCAN_WARPS * 128 < n_pages) c *= 2;
  return c;
}

size_t resize_smem(int batch, int slots) { return 4ull * (batch + 1) + 8ull * slots + 2ull * batch; }

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
  // no fewer than four: then up to eight units a thread.
  int cols = 4;
  while (cols * 2 * c->batch <= 4 * FORK_THREADS && cols < c->max_pages) cols *= 2;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  return launch(k_fork, dim3((unsigned)((c->max_pages + cols - 1) / cols)), FORK_THREADS, 0, 1, stream, pool_of(c), parents,
                cols, table_vec(c));
}

int dflash_pages_resize(const dflash_page_pool* c, const int32_t* new_lens, int32_t* moves, int32_t capacity,
                        void* stream) {
  if (int e = pool_check(c)) return e;
  if (!new_lens || !moves || capacity < 0 || !words(new_lens) || !words(moves)) return DFLASH_ERR_INVALID_ARG;
  if (capacity < c->batch) return DFLASH_ERR_CAPACITY;
  const PoolParts w = pool_parts(c);
  if (!apart({w.refs, w.table, w.lens, w.status, strided_ints(moves, 3 + 3ll * capacity)},
             {strided_ints(new_lens, c->batch)}))
    return DFLASH_ERR_INVALID_ARG;
  int slots = 64;
  while (slots < 2 * c->batch) slots *= 2;
  const size_t smem = resize_smem(c->batch, slots);
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  if (smem > 48 * 1024)
    if (int e = cuda_status(cudaFuncSetAttribute(k_resize, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)resize_smem(DFLASH_POOL_MAX_BATCH, 2 * DFLASH_POOL_MAX_BATCH))))
      return e;
  const int ctas = scan_ctas(c->n_pages);
  return launch(k_resize, dim3((unsigned)ctas), SCAN_THREADS, smem, ctas, stream, pool_of(c), new_lens, moves, capacity,
                ctas, slots, (reinterpret_cast<uintptr_t>(c->refs) & 15) == 0);
}

int dflash_pages_compact(const dflash_page_pool* c, int32_t* moves, int32_t capacity, int32_t* remap, void* stream) {
  if (int e = pool_check(c)) return e;
  if (!moves || !remap || capacity < 0 || !words(moves) || !words(remap)) return DFLASH_ERR_INVALID_ARG;
  if (capacity < c->n_pages / 2) return DFLASH_ERR_CAPACITY;
  const PoolParts w = pool_parts(c);
  if (!apart({w.refs, w.table, w.status, strided_ints(moves, 3 + 3ll * capacity), strided_ints(remap, c->n_pages)}, {w.lens}))
    return DFLASH_ERR_INVALID_ARG;
  DeviceGuard guard(c->device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  const int ctas = scan_ctas(c->n_pages);
  if (int e = launch(k_compact, dim3((unsigned)ctas), SCAN_THREADS, 0, ctas, stream, pool_of(c), moves, capacity, remap, ctas,
                     (reinterpret_cast<uintptr_t>(c->refs) & 15) == 0))
    return e;
  const int per_row = (c->max_pages + REMAP_THREADS * REMAP_EACH - 1) / (REMAP_THREADS * REMAP_EACH);
  const long long blocks = (long long)per_row * c->batch;
  if (blocks > 0x7fffffffll) return DFLASH_ERR_CAPACITY;
  return launch(k_remap, dim3((unsigned)blocks), REMAP_THREADS, 0, 1, stream, pool_of(c), remap, per_row);
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
  DeviceGuard guard(c0.device);
  if (!guard.ok) return DFLASH_ERR_CUDA;
  for (int at = 0; at < n_caches; at += COPY_CACHES) {
    const int n = std::min(COPY_CACHES, n_caches - at);
    p.n_pools = 2 * n;
    for (int i = 0; i < n; ++i) {
      const dflash_paged_cache& c = caches[at + i];
      p.pool[2 * i] = {static_cast<char*>(c.k), 2 * c.k_page_stride, 2 * c.k_pos_stride, 2 * c.k_head_stride};
      p.pool[2 * i + 1] = {static_cast<char*>(c.v), 2 * c.v_page_stride, 2 * c.v_pos_stride, 2 * c.v_head_stride};
    }
    const unsigned grid = (unsigned)std::min<long long>(152 * 8, (long long)capacity * p.n_pools * p.chunks);
    const int e = vec ? launch(k_copy_pages<uint4>, dim3(grid), COPY_THREADS, 0, 1, stream, p)
                      : launch(k_copy_pages<uint16_t>, dim3(grid), COPY_THREADS, 0, 1, stream, p);
    if (e) return e;
  }
  return DFLASH_OK;
}

}  // extern "C"

// Whether tensors of a call share memory.  Host only.
//
// A tensor is runs of bytes at every sum of multiples of its strides.  Views of
// one buffer interleave without meeting (heads of a fused projection, pools
// that alternate by page), so comparing first and last addresses is not enough:
// the widest stride is taken apart first, and of its multiples only those whose
// bytes can meet the other tensor's are looked at, usually one or two.
#pragma once
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "../../include/dflash.h"

struct Strided {
  long long at = 0, run = 0;  // address, bytes of a run (0: empty)
  int n = 0;                  // dimensions, the widest stride first
  long long stride[3] = {}, count[3] = {};  // bytes; strides > 0, counts > 1
  bool folded = false;        // a dimension of several elements has stride 0
};

// `run` bytes at `data`, repeated by up to three (stride in bytes, count).
inline Strided strided(const void* data, long long run, std::initializer_list<std::pair<long long, long long>> dims) {
  Strided s;
  if (!data || run <= 0) return s;
  s.at = (long long)reinterpret_cast<intptr_t>(data);
  s.run = run;
  for (auto d : dims) {
    if (d.second <= 0) return Strided();
    if (d.second == 1) continue;
    if (d.first == 0) {
      s.folded = true;
      continue;
    }
    if (d.first < 0) {
      s.at += d.first * (d.second - 1);
      d.first = -d.first;
    }
    int i = s.n++;
    for (; i > 0 && s.stride[i - 1] < d.first; --i) s.stride[i] = s.stride[i - 1], s.count[i] = s.count[i - 1];
    s.stride[i] = d.first;
    s.count[i] = d.second;
  }
  // dimensions that continue one another, and the run, are one
  while (s.n > 0 && s.stride[s.n - 1] == s.run) s.run *= s.count[--s.n];
  for (int i = s.n - 1; i > 0; --i) {
    if (s.stride[i - 1] != s.stride[i] * s.count[i]) continue;
    s.stride[i - 1] = s.stride[i];
    s.count[i - 1] *= s.count[i];
    for (int j = i; j + 1 < s.n; ++j) s.stride[j] = s.stride[j + 1], s.count[j] = s.count[j + 1];
    --s.n;
  }
  return s;
}

// Bytes from the first to behind the last, of the dimensions from d on.
inline long long extent(const Strided& s, int d = 0) {
  long long e = s.run;
  for (; d < s.n; ++d) e += s.stride[d] * (s.count[d] - 1);
  return e;
}

// Whether every element has bytes of its own, as far as nested strides tell.
inline bool distinct(const Strided& s) {
  if (s.folded) return false;
  for (int d = 0; d < s.n; ++d)
    if (s.stride[d] < extent(s, d + 1)) return false;
  return true;
}

// a's dimensions from da on against b's from db on, b's first byte `off` behind
// a's.  After `left` comparisons the answer is yes, to be safe.
inline bool meet_from(const Strided& a, int da, const Strided& b, int db, long long off, int& left) {
  const long long ea = extent(a, da), eb = extent(b, db);
  if (off >= ea || off + eb <= 0) return false;
  if (da == a.n && db == b.n) return true;
  if (--left < 0) return true;
  auto below = [](long long x, long long y) { return x / y - (x % y != 0 && (x < 0) != (y < 0)); };  // floor of x / y
  if (da < a.n && db < b.n && a.stride[da] == b.stride[db]) {  // only the difference of the two multiples counts
    const long long s = a.stride[da], ra = extent(a, da + 1), rb = extent(b, db + 1);
    long long lo = below(-rb - off, s) + 1, hi = -below(off - ra, s) - 1;
    if (lo < 1 - a.count[da]) lo = 1 - a.count[da];
    if (hi > b.count[db] - 1) hi = b.count[db] - 1;
    for (long long d = lo; d <= hi; ++d)
      if (meet_from(a, da + 1, b, db + 1, off + d * s, left)) return true;
    return false;
  }
  if (da == a.n || (db < b.n && b.stride[db] > a.stride[da])) return meet_from(b, db, a, da, -off, left);
  const long long s = a.stride[da], ra = extent(a, da + 1);
  long long lo = below(off - ra, s) + 1, hi = -below(-(off + eb), s) - 1;
  if (lo < 0) lo = 0;
  if (hi > a.count[da] - 1) hi = a.count[da] - 1;
  for (long long i = lo; i <= hi; ++i)
    if (meet_from(a, da + 1, b, db, off - i * s, left)) return true;
  return false;
}
inline bool meet(const Strided& a, const Strided& b) {
  if (!a.run || !b.run) return false;
  int left = 1 << 14;
  return meet_from(a, 0, b, 0, b.at - a.at, left);
}

// Whether what a call writes lies apart from itself and from everything else of the call.
inline bool apart(std::initializer_list<Strided> written, std::initializer_list<Strided> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    if (!distinct(*w)) return false;
    for (auto x = w + 1; x != written.end(); ++x)
      if (meet(*w, *x)) return false;
    for (const Strided& r : read)
      if (meet(*w, r)) return false;
  }
  return true;
}

// Rows of 16-bit values, int32 values, a cache's pools.
inline Strided strided_rows(const dflash_rows& r, int rows, int heads, int D) {
  return strided(r.data, 2ll * D, {{2 * r.row_stride, rows}, {2 * r.head_stride, heads}});
}
inline Strided strided_ints(const int32_t* p, long long n) { return strided(p, 4 * n, {}); }
inline Strided strided_pool(const dflash_paged_cache* c, bool v) {
  return strided(v ? c->v : c->k, 2ll * c->head_dim,
                 {{2 * (v ? c->v_page_stride : c->k_page_stride), c->n_pages},
                  {2 * (v ? c->v_pos_stride : c->k_pos_stride), c->page_size},
                  {2 * (v ? c->v_head_stride : c->k_head_stride), c->kv_heads}});
}
inline Strided strided_table(const dflash_paged_cache* c, int batch) {
  return strided(c->page_table, 4ll * c->max_pages, {{4 * c->table_stride, batch}});
}
// An output's input, or nothing where the output is that input itself (in place).
inline Strided input_of(const dflash_rows& out, const dflash_rows& in, int rows, int heads, int D) {
  if (out.data == in.data && (rows == 1 || out.row_stride == in.row_stride) &&
      (heads == 1 || out.head_stride == in.head_stride))
    return Strided();
  return strided_rows(in, rows, heads, D);
}

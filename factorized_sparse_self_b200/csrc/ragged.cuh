// Index arithmetic of attention over ragged sequences (packed one behind the
// other, or kept in a paged cache) restricted to the factorized patterns.
//
// The sets are those of the dense-batch calls: strided A1 (window), A2
// (stride), fixed A1 (block), A2 (summary), and the unions. As there, every set
// is split into segments in a row order that makes it dense, but the sequences
// here have any length, so nothing is padded: each order lists a sequence's
// positions one after the other,
//   natural  0, 1, 2, ...
//   summary  the last c positions of every l-block, packed (keys only)
//   class    residue class by residue class (p, p + l, p + 2l, ...), beginning
//            with the class of the first query: a chunk's queries then stand in
//            the classes that follow one another, not at both ends of the order
// and in its order every query row's live keys are ONE interval [lo, hi) whose
// ends never decrease from row to row. A tile of rows therefore meets the keys from its
// first row's lo to its last row's hi; the rows that a key meets are an interval
// of the query order in the same way.
//
// Grouped heads: the query heads that share a key/value head and have the same
// index set form the rows of one unit, row x = e * Gc + g being query e of the
// order, head g of the group, so that a K / V tile serves the whole group.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_common.cuh"

namespace st {
namespace rag {

#define ST_HD __host__ __device__ __forceinline__

ST_HD int qdiv(int n, FastDiv f, int d) {
#ifdef __CUDA_ARCH__
  (void)d;
  return fdiv(n, f);
#else
  (void)f;
  return n / d;
#endif
}

struct Seg {
  int32_t kview;  // View of the keys
  int32_t rule;   // Rule
};

// One head class in one query order: its segments are attended by one softmax
// (or, for the strided union, joined with the other order's result).
struct Job {
  int32_t hc;     // heads: 0 / 1 = even / odd heads only, -1 = all
  int32_t qview;  // View of the queries
  int32_t nseg;
  Seg seg[2];
};

// Rows of one tensor as a matrix of d-element rows: the row of head h of a
// token (packed: token index; paged: through the page table).
struct Rows {
  int32_t tok;   // rows from one token (slot) to the next
  int32_t head;  // rows from one head to the next
  int32_t page;  // rows from one page to the next (paged only)
};

struct Geo {
  int32_t S, total;       // sequences, token rows
  int32_t H, Hkv, G, d;
  int32_t l, c, split;    // split: even / odd heads have different sets
  FastDiv fl, fc;
  FastDiv fheads[3];      // division by G, (G + 1) / 2, G / 2
  const int32_t* cu;      // [S + 1] first token row of every sequence
  // paged cache (null kv_lens: packed, keys are the sequence's own rows)
  const int32_t* kv_lens; // [S]
  const int32_t* table;   // [S, max_pages]
  int32_t page_size, max_pages, num_pages;
  FastDiv fpage;
  Rows q, k, v;
  int* status;
};

// One sequence.
struct Seq {
  int32_t s, qb;     // index, first token row
  int32_t nq, nk;    // query rows, keys
  int32_t off;       // position of query row 0 (nk - nq; negative rows attend nothing)
  int32_t nqv;       // query rows at positions >= 0
  int32_t P, rem;    // nk / l, nk mod l
  int32_t Po, remo;  // the same of max(off, 0)
  int32_t nsum;      // summary positions among the keys
  int32_t rotk, rotq;  // keys / queries of the classes below the first query's
};

ST_HD int imin(int a, int b) { return a < b ? a : b; }
ST_HD int imax(int a, int b) { return a > b ? a : b; }

ST_HD Seq make_seq(const Geo& g, int s, int qb, int nq, int nk) {
  Seq q;
  q.s = s;
  q.qb = qb;
  q.nq = nq;
  q.nk = nk;
  q.off = nk - nq;
  const int o = imax(q.off, 0);
  q.nqv = nk - o;
  q.P = qdiv(nk, g.fl, g.l);
  q.rem = nk - q.P * g.l;
  q.Po = qdiv(o, g.fl, g.l);
  q.remo = o - q.Po * g.l;
  q.rotk = q.remo * q.P + imin(q.remo, q.rem);
  q.rotq = q.rotk - q.remo * q.Po - q.remo;
  q.nsum = q.P * g.c + imax(0, q.rem - (g.l - g.c));
  return q;
}

// First index of class r in the class order of the keys 0 .. nk-1.
ST_HD int cls_key_start(const Seq& q, int r) {
  const int s = r * q.P + imin(r, q.rem) - q.rotk;
  return r >= q.remo ? s : s + q.nk;
}

// Position of key index e of an order (0 <= e < number of keys in it).
ST_HD int key_pos(const Geo& g, const Seq& q, int view, int e) {
  if (view == VIEW_NAT) return e;
  if (view == VIEW_SUM) {
    const int b = qdiv(e, g.fc, g.c);
    return b * g.l + (g.l - g.c) + (e - b * g.c);
  }
  e += e >= q.nk - q.rotk ? q.rotk - q.nk : q.rotk;
  const int big = q.rem * (q.P + 1);  // <= nk
  if (e < big) {
    const int r = e / (q.P + 1);
    return (e - r * (q.P + 1)) * g.l + r;
  }
  const int r = (e - big) / q.P;  // P >= 1 here: e - big < (l - rem) * P
  return (e - big - r * q.P) * g.l + q.rem + r;
}

ST_HD int n_keys(const Seq& q, int view) { return view == VIEW_SUM ? q.nsum : q.nk; }

// Token row of query index e of an order (0 <= e < nq), relative to the
// sequence; its position is row + off. In the class order the rows at negative
// positions come last.
ST_HD int query_row(const Geo& g, const Seq& q, int view, int e) {
  if (view == VIEW_NAT) return e;
  if (e >= q.nqv) return e - q.nqv;
  e += e >= q.nqv - q.rotq ? q.rotq - q.nqv : q.rotq;
  // Classes start at slope D = P - Po, one more between remo and rem (or one
  // less between rem and remo): three pieces of equal classes.
  const int D = q.P - q.Po;
  const int a = imin(q.rem, q.remo), b = imax(q.rem, q.remo);
  const int Dm = q.rem >= q.remo ? D + 1 : D - 1;
  const int s1 = a * D, s2 = s1 + (b - a) * Dm;
  int r, p;
  if (e < s1) {
    r = e / D;
    p = e - r * D;
  } else if (e < s2) {
    r = (e - s1) / Dm;
    p = e - s1 - r * Dm;
    r += a;
  } else {
    r = (e - s2) / D;
    p = e - s2 - r * D;
    r += b;
  }
  // the class's first query position is the first one >= max(off, 0)
  const int first = q.Po + (r < q.remo ? 1 : 0);
  return (first + p) * g.l + r - q.off;
}

// Live keys [lo, hi) of the query at position i (>= 0), in the segment's key
// order.
ST_HD void live_keys(const Geo& g, const Seq& q, int rule, int i, int& lo, int& hi) {
  lo = 0;
  hi = i + 1;
  if (rule == RULE_CAUSAL) return;
  if (rule == RULE_BAND) {
    lo = imax(0, i - g.l);
    return;
  }
  const int b = qdiv(i, g.fl, g.l);
  const int r = i - b * g.l;
  switch (rule) {
    case RULE_BLOCK:
      lo = b * g.l;
      break;
    case RULE_STRIDE:
      lo = cls_key_start(q, r);
      hi = lo + b + 1;
      break;
    case RULE_STRIDE_FAR:
      lo = cls_key_start(q, r);
      hi = imax(lo, lo + b - 1);
      break;
    case RULE_SUMMARY:
      hi = b * g.c + imax(0, r + 1 - (g.l - g.c));
      break;
    default:  // RULE_SUMMARY_EARLIER
      hi = b * g.c;
      break;
  }
}

// Query indexes of an order that attend anything: [qv0, qv1).
ST_HD void valid_rows(const Seq& q, int view, int& v0, int& v1) {
  v0 = view == VIEW_NAT ? q.nq - q.nqv : 0;
  v1 = view == VIEW_NAT ? q.nq : q.nqv;
}

// Query indexes [a, b) whose live interval holds key index k, for a packed
// sequence (as many queries as keys).
ST_HD void live_queries(const Geo& g, const Seq& q, int rule, int k, int& a, int& b) {
  a = k;
  b = q.nq;
  switch (rule) {
    case RULE_CAUSAL:
      return;
    case RULE_BAND:
      if (b - k > g.l) b = k + g.l + 1;
      return;
    case RULE_BLOCK:
      b = k + imin(b - k, g.l - (k - qdiv(k, g.fl, g.l) * g.l));
      return;
    case RULE_STRIDE:
    case RULE_STRIDE_FAR: {
      // the rest of the key's class, from the key itself or two rows later
      const int big = q.rem * (q.P + 1);
      b = k < big ? (k / (q.P + 1) + 1) * (q.P + 1) : big + ((k - big) / imax(q.P, 1) + 1) * q.P;
      if (rule == RULE_STRIDE_FAR) a = imin(k + 2, b);
      return;
    }
    default: {
      const int blk = qdiv(k, g.fc, g.c);  // k counts summary positions
      if (rule == RULE_SUMMARY) a = blk * g.l + (g.l - g.c) + (k - blk * g.c);
      else a = imin(blk, q.P) * g.l + imin(g.l, q.nq - imin(blk, q.P) * g.l);
      return;
    }
  }
}

// Query heads of a group that belong to a job: head = first + step * g.
struct Heads3 {
  int32_t first, step, n;
  FastDiv f;  // division by n
};
ST_HD Heads3 heads_of_group(const Geo& g, int hc, int kvh) {
  Heads3 h;
  h.first = kvh * g.G;
  h.step = 1;
  h.n = g.G;
  h.f = g.fheads[0];
  if (hc >= 0) {
    h.first += (hc ^ h.first) & 1;
    h.step = 2;
    const int end = kvh * g.G + g.G;
    h.n = h.first < end ? (end - h.first + 1) / 2 : 0;
    h.f = 2 * h.n > g.G ? g.fheads[1] : g.fheads[2];
  }
  return h;
}
// The most heads of one job in a group: unit slots are numbered with it.
ST_HD int most_heads(const Geo& g, int hc) { return hc >= 0 ? (g.G + 1) / 2 : g.G; }

// Unit slots: sequence s owns the slots from floor(cu[s] * mult / BM) + s up to
// the next sequence's first, at least ceil(n_s * mult / BM) of them, so a slot's
// sequence is found by bisection of cu and no table of units is built. Slots below
// the first sequence's (its rows need not start at 0) belong to no sequence: their
// tile lies past every sequence's rows.
ST_HD long long slot_count(const Geo& g, int mult, int BM) {
  return (long long)g.total * mult / BM + g.S;
}
ST_HD int slot_first(int cu_s, int s, int mult, int BM) {
  return (int)((long long)cu_s * mult / BM) + s;
}
ST_HD int slot_tile(int slot, int first, int BM) {
  return slot >= first ? slot - first : 0x7fffffff / BM;
}

#ifdef __CUDACC__
__device__ __forceinline__ int cu_at(const Geo& g, int s) {
  return imin(imax(__ldg(g.cu + s), 0), g.total);
}

__device__ __forceinline__ Seq load_seq(const Geo& g, int s) {
  const int a = cu_at(g, s);
  const int b = imax(a, cu_at(g, s + 1));
  int nk = b - a;
  if (g.kv_lens) {
    const int want = __ldg(g.kv_lens + s);
    nk = imin(imax(want, 0), g.max_pages * g.page_size);
    if (nk != want) set_status(g.status, ST_ERR_INVALID);
  }
  return make_seq(g, s, a, b - a, nk);
}

// The last of 0 .. n-1 for which pred holds (true up to some index, which
// includes 0, then false), by a whole warp: 32 probes a round instead of one, for
// each round waits for memory.
template <class P>
__device__ __forceinline__ int last_true(int n, P pred) {
  const int lane = threadIdx.x & 31;
  int a = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5, x = a + lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, lane * step < n && pred(x));
    const int c = imax(__popc(yes), 1) - 1;
    a += c * step;
    n = imin(step, n - c * step);
  }
  return a;
}

// Sequence and tile of a slot (the tile may be past the sequence's rows), by a
// whole warp.
__device__ __forceinline__ int find_slot(const Geo& g, int mult, int BM, int slot, int& tile) {
  auto first = [&](int s) { return slot_first(cu_at(g, s), s, mult, BM); };
  const int s = last_true(g.S, [&](int x) { return first(x) <= slot; });
  tile = slot_tile(slot, first(s), BM);
  return s;
}

// Page number pg of a sequence; one outside the cache is reported and read as
// page 0.
__device__ __forceinline__ int page_of(const Geo& g, const Seq& q, int pg) {
  int page = __ldg(g.table + (size_t)q.s * g.max_pages + pg);
  if ((unsigned)page >= (unsigned)g.num_pages) {
    set_status(g.status, ST_ERR_INVALID);
    page = 0;
  }
  return page;
}

// Rows (in units of d elements) of key position j, key/value head kvh, of k and v.
__device__ __forceinline__ void kv_rows(const Geo& g, const Seq& q, int j, int kvh, int& rk, int& rv) {
  if (!g.kv_lens) {
    rk = (q.qb + j) * g.k.tok + kvh * g.k.head;
    rv = (q.qb + j) * g.v.tok + kvh * g.v.head;
    return;
  }
  const int pg = fdiv(j, g.fpage);
  rk = rv = page_of(g, q, pg) * g.k.page + (j - pg * g.page_size) * g.k.tok + kvh * g.k.head;
}
__device__ __forceinline__ int k_row(const Geo& g, const Seq& q, int j, int kvh) {
  int rk, rv;
  kv_rows(g, q, j, kvh, rk, rv);
  return rk;
}
__device__ __forceinline__ int v_row(const Geo& g, const Seq& q, int j, int kvh) {
  int rk, rv;
  kv_rows(g, q, j, kvh, rk, rv);
  return rv;
}

// Row of token t (absolute), query head h.
__device__ __forceinline__ int q_row(const Geo& g, int t, int h) {
  return t * g.q.tok + h * g.q.head;
}
// Query row x of a unit's order: token row (absolute), head, position; false
// past the unit's rows.
struct QRow {
  int t, h, pos;
};
__device__ __forceinline__ bool query_at(const Geo& g, const Seq& q, int view, const Heads3& hs,
                                         int x, QRow& r) {
  if (x >= q.nq * hs.n) return false;
  const int e = fdiv(x, hs.f);
  const int row = query_row(g, q, view, e);
  r.t = q.qb + row;
  r.pos = row + q.off;
  r.h = hs.first + hs.step * (x - e * hs.n);
  return true;
}

// Key tiles [j0, j1) of bn keys that the unit's rows x0 .. x0+rows-1 meet in a
// segment.
__device__ __forceinline__ void tile_range(const Geo& g, const Seq& q, const Job& job, int seg,
                                           const Heads3& hs, int x0, int rows, int bn, int& j0,
                                           int& j1) {
  j0 = j1 = 0;
  int v0, v1;
  valid_rows(q, job.qview, v0, v1);
  const int e0 = imax(fdiv(x0, hs.f), v0), e1 = imin(fdiv(imin(x0 + rows, q.nq * hs.n) - 1, hs.f), v1 - 1);
  if (e0 > e1) return;
  int lo, hi, a, b;
  live_keys(g, q, job.seg[seg].rule, query_row(g, q, job.qview, e0) + q.off, lo, hi);
  live_keys(g, q, job.seg[seg].rule, query_row(g, q, job.qview, e1) + q.off, a, b);
  if (b > lo) {
    j0 = lo / bn;
    j1 = (b + bn - 1) / bn;
  }
}
#endif

}  // namespace rag
}  // namespace st

// C ABI of attention over ragged sequences and paged caches: argument checks,
// workspace plans and launch sequences. See include/sparse_transformer_attn.h
// for the contract of every entry point.
#include <cmath>

#include "ragged.h"

using namespace st;
using namespace st::rag;

namespace {

constexpr int kPartsLimit = 32;  // most key ranges of one row
// Most query rows per key/value head for the few-row kernel. Dense, Hkv = 8, d = 128,
// 64 sequences of 4096 keys, 16, 32, 64 rows: 213, 311, 584 us against the tile
// kernel's 389, 391, 412.
constexpr int kFewRows = 32;
constexpr long long kPartsBytes = 256LL << 20;  // most workspace that key ranges may take
constexpr int64_t kMaxRows = 0x7fff0000;  // most query rows or keys: 32-bit numbers, rounded up to tiles

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool known(st_dtype t) { return t == ST_F32 || t == ST_BF16 || t == ST_F16; }

// The jobs (head class x query order) of a pattern.
int make_jobs(const st_pattern_desc& p, Job jobs[2]) {
  const bool split = p.head_mode == ST_HEADS_SPLIT;
  auto one = [](int hc, int qv, int kv, int rule) {
    return Job{hc, qv, 1, {{kv, rule}, {VIEW_NAT, RULE_CAUSAL}}};
  };
  if (p.kind == ST_DENSE_CAUSAL) {
    jobs[0] = one(-1, VIEW_NAT, VIEW_NAT, RULE_CAUSAL);
    return 1;
  }
  if (p.kind == ST_STRIDED) {
    jobs[0] = one(split ? 0 : -1, VIEW_NAT, VIEW_NAT, RULE_BAND);
    jobs[1] = one(split ? 1 : -1, VIEW_CLS, VIEW_CLS, split ? RULE_STRIDE : RULE_STRIDE_FAR);
    return 2;
  }
  if (split) {
    jobs[0] = one(0, VIEW_NAT, VIEW_NAT, RULE_BLOCK);
    jobs[1] = one(1, VIEW_NAT, VIEW_SUM, RULE_SUMMARY);
    return 2;
  }
  jobs[0] = Job{-1, VIEW_NAT, 2, {{VIEW_NAT, RULE_BLOCK}, {VIEW_SUM, RULE_SUMMARY_EARLIER}}};
  return 1;
}

// Whether a row's result is joined from two query orders.
bool two_orders(const st_pattern_desc& p) {
  return p.kind == ST_STRIDED && p.head_mode == ST_HEADS_MERGED;
}

st_status check_pattern(const st_pattern_desc* p) {
  if (!p || p->T < 1) return ST_ERR_INVALID;
  if (p->kind != ST_STRIDED && p->kind != ST_FIXED && p->kind != ST_DENSE_CAUSAL)
    return ST_ERR_INVALID;
  if (p->kind != ST_DENSE_CAUSAL) {
    if (p->head_mode != ST_HEADS_SPLIT && p->head_mode != ST_HEADS_MERGED) return ST_ERR_INVALID;
    if (p->l < 1) return ST_ERR_INVALID;
    if (p->kind == ST_FIXED && (p->c < 1 || p->c > p->l)) return ST_ERR_INVALID;
  }
  return ST_OK;
}

// Rows of d elements from token to token; false for a stride that is no
// multiple of d or too small for the heads.
bool stride_rows(int64_t stride, int heads, int d, int32_t* out) {
  if (stride == 0) stride = (int64_t)heads * d;
  if (stride < (int64_t)heads * d || stride % d) return false;
  if (stride / d > 0x7fffffff) return false;
  *out = (int32_t)(stride / d);
  return true;
}

st_status fill_geo(const st_pattern_desc* p, st_dtype dtype, const st_packed_desc* x, bool sizes_16,
                   Geo& g) {
  st_status s = check_pattern(p);
  if (s != ST_OK) return s;
  if (!x || !known(dtype)) return ST_ERR_INVALID;
  if (x->n_seqs < 1 || x->total < 0 || x->H < 1 || x->Hkv < 1 || x->d < 1 || x->H % x->Hkv)
    return ST_ERR_INVALID;
  if (sizes_16) {
    const bool ok = dtype == ST_F32 ? (x->d == 32 || x->d == 64 || x->d == 128)
                                    : (x->d == 64 || x->d == 128);
    if (!ok) return ST_ERR_UNSUPPORTED;
  }
  g = Geo{};
  g.S = x->n_seqs;
  g.total = x->total;
  g.H = x->H;
  g.Hkv = x->Hkv;
  g.G = x->H / x->Hkv;
  g.d = x->d;
  const bool dense = p->kind == ST_DENSE_CAUSAL;
  g.l = dense ? 1 : p->l;
  g.c = p->kind == ST_FIXED ? p->c : 1;
  g.split = !dense && p->head_mode == ST_HEADS_SPLIT;
  g.fl = make_fastdiv(g.l);
  g.fc = make_fastdiv(g.c);
  g.fheads[0] = make_fastdiv(g.G);
  g.fheads[1] = make_fastdiv((g.G + 1) / 2);
  g.fheads[2] = make_fastdiv(g.G / 2);
  if (!stride_rows(x->q_stride, x->H, x->d, &g.q.tok) ||
      !stride_rows(x->k_stride, x->Hkv, x->d, &g.k.tok) ||
      !stride_rows(x->v_stride, x->Hkv, x->d, &g.v.tok))
    return ST_ERR_INVALID;
  g.q.head = g.k.head = g.v.head = 1;
  // grids and row numbers are 31-bit
  if ((int64_t)g.total * g.q.tok > 0x7fffffff || (int64_t)g.total * g.k.tok > 0x7fffffff ||
      (int64_t)g.total * g.v.tok > 0x7fffffff || (int64_t)g.total * g.H > kMaxRows ||
      (int64_t)g.total * g.G + g.S > kMaxRows || g.Hkv > 65535)
    return ST_ERR_UNSUPPORTED;
  return ST_OK;
}

st_status fill_cache(const st_cache_desc* c, Geo& g) {
  if (!c || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1) return ST_ERR_INVALID;
  const int64_t d = g.d;
  if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0 || c->page_stride % d ||
      c->slot_stride % d || c->head_stride % d)
    return ST_ERR_INVALID;
  const int64_t page = c->page_stride / d, slot = c->slot_stride / d, head = c->head_stride / d;
  if (std::max({page, slot, head}) > 0x7fffffff) return ST_ERR_UNSUPPORTED;
  const int64_t pages = (c->num_pages - 1) * page, slots = (c->page_size - 1) * slot,
                heads = (g.Hkv - 1) * head;  // below 2^62 each
  if (std::max({pages, slots, heads}) >= 0x7fffffff || pages + slots + heads >= 0x7fffffff ||
      (int64_t)c->max_pages * c->page_size > kMaxRows || (int64_t)g.S * c->max_pages > 0x7fffffff)
    return ST_ERR_UNSUPPORTED;
  g.num_pages = c->num_pages;
  g.page_size = c->page_size;
  g.max_pages = c->max_pages;
  g.fpage = make_fastdiv(c->page_size);
  g.k.tok = (int32_t)slot;
  g.k.head = (int32_t)head;
  g.k.page = (int32_t)page;
  g.v = g.k;
  return ST_OK;
}

// The status word of the current device; the first call creates it.
st_status get_status(Geo& g) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return ST_ERR_CUDA;
  g.status = device_status(dev, true);
  return g.status ? ST_OK : ST_ERR_CUDA;
}

// How a forward call is cut up.
struct FwdPlan {
  bool few;     // the few-row kernel
  int nsplit;   // most key ranges per unit and job
  int least;    // fewest key tiles (of the kernel) of a range
  int nparts;   // parts of a row (0: rows are written directly)
  bool taper;   // ranges get shorter, and short ones go last
  bool merge;   // the second order joins the first's part itself
  bool fits;    // the units of a launch can be numbered
  size_t parts_o, bytes;
};

// The tile kernels number the units of a launch in 31 bits.
bool units_fit(const Geo& g, int mult, int rows, long long per_slot) {
  return slot_count(g, mult, rows) * g.Hkv * per_slot <= 0x7fffffff;
}

// Rows that one query row's pattern lets it attend, at most, in a sequence of T.
long long most_keys(const st_pattern_desc& p) {
  if (p.kind == ST_DENSE_CAUSAL) return p.T;
  const long long a = p.kind == ST_STRIDED ? (long long)p.l + 1 : p.l;
  const long long b = p.kind == ST_STRIDED ? (p.T + p.l - 1LL) / p.l
                                           : ((long long)p.T / p.l + 1) * p.c;
  return std::min<long long>(p.T, p.head_mode == ST_HEADS_MERGED ? a + b : std::max(a, b));
}

int clamp_int(long long x, long long lo, long long hi) {
  return (int)std::max(lo, std::min(x, hi));
}

// Whether the few-row kernel takes a strided chunk of more rows than kFewRows. The rows
// lie in many classes, so 256 of them may meet most of the context, one tile after the
// other; units of 16 rows meet little, but those of one class, or of one window, each
// read its keys again. So: where 256-row units would not fill a quarter of the GPU,
// unless the 16-row units of all heads read more keys an SM than 1.5 times what the
// tile kernel has to go through one after the other (its longest key range, or its
// share of all units; and 256 keys for its start). us by the few-row kernel and by the tile
// kernel, one chunk of n behind 16 K keys, merged, d = 128 (last column: split, behind 4 K):
//   n, l           64, 64   256, 128  512, 128  256, 16   256, 4    512, 512
//   H = 32, Hkv 8  39, 379  88, 131   86, 90    104, 74*  216, 76*  74, 43*
//   H = 8, Hkv 2   23, 376  34, 129   41, 86    53, 69    88, 43*   33, 41
// (*: goes to the tile kernel). Over 720 such calls (d 64, 128; l 4 to 512; 1 to 16 chunks
// of 32 to 512) the choice takes 2 % longer than the better kernel of each, 2.0 times
// at worst; the quarter of the GPU alone 7 %, 3.0 times at worst.
template <class Units, class Ranges>
bool strided_by_few(const Geo& g, const st_pattern_desc& p, int G, long long max_q, Units units,
                    Ranges ranges) {
  const long long sms = sm_count(), T = p.T, l = std::min<long long>(p.l, T);
  const long long longest = units(256, max_q), all = std::max(longest, units(256, g.total));
  if (p.kind != ST_STRIDED || 4 * all >= sms) return false;
  const long long cls_rows = G * std::max(1LL, max_q / l), cls_keys = (T + l - 1) / l;
  // keys that one unit meets in either order, and the units of all sequences
  auto meets = [&](long long rows, long long& band, long long& cls) {
    rows = std::min(rows, max_q * G);
    band = std::min(T, l + 1 + (rows + G - 1) / G);
    cls = std::min(T, std::max(1LL, rows / cls_rows) * cls_keys);
  };
  const long long seqs = std::max(1, std::min(g.S, g.total)), mean = (g.total + seqs - 1) / seqs;
  long long b16, c16, b256, c256;
  meets(16, b16, c16);
  meets(256, b256, c256);
  const long long few = seqs * units(16, mean) * (b16 + c16);
  const long long tiles = seqs * units(256, mean) * (b256 + c256);
  const long long range = std::max(b256, c256) / ranges(longest, all);
  return 2 * few <= 3 * std::max(sms * (range + 256), tiles + sms * 256);
}

// Key ranges (the kernels cut short units into fewer). Units go to free SMs one
// by one, so only few units leave SMs idle: those of one longest sequence (the
// others may be short) have to be worth the GPU. A prompt's units see 1 .. T
// keys, the longest ones first; a chunk's see all of the context, so they come in
// twos per SM, fewer where other sequences bring units too, and taper: the first
// range of every unit, the longest, goes first, the short ones fill the end. Dense, H =
// 32, Hkv = 8, d = 128, us:
//                                              tapered  ranges of one length
//   2, 3, 4 per SM: chunks of 512 behind 32 K, 8 K, 4 K keys   395, 400, 426   444, 451, 476
//   128 tokens behind 64 K keys                158, 176, 180   211, 211, 206
//   256 behind 16 K, four times                389, 419, 436   406, 440, 451
//   (that one by this rule, 6 ranges: 350)
FwdPlan plan_fwd(const Geo& g, const st_pattern_desc& p, st_dtype dtype, long long max_q, bool paged) {
  FwdPlan f{};
  const long long sms = sm_count(), keys = most_keys(p);
  const int G = g.split ? (g.G + 1) / 2 : g.G;
  auto units = [&](int rows, long long tokens) { return (tokens * G + rows - 1) / rows * g.Hkv; };
  // the tile kernels' key ranges
  auto ranges = [&](long long longest, long long all) {
    long long n = 1;
    if (all < 4 * sms) {
      n = ((paged ? 2 : 1) * sms + longest - 1) / longest;
      if (paged) n = std::min(n, std::max(4LL, 6 * sms / all));
    }
    return std::max(1LL, std::min(n, keys / 512));
  };
  f.few = paged && dtype != ST_F32 && (max_q * G <= kFewRows || strided_by_few(g, p, G, max_q, units, ranges));
  const int rows = f.few ? 16 : dtype == ST_F32 ? 64 : 256;
  const int key_tile = f.few ? 16 : dtype == ST_F32 ? 64 : 128;
  const long long longest = std::max(1LL, units(rows, max_q));
  const long long all = std::max(longest, units(rows, g.total));
  const size_t qrows = (size_t)g.total * g.H;
  const long long fit = std::max(1LL, kPartsBytes / (long long)std::max<size_t>(1, qrows * g.d * sizeof(float)));
  if (f.few) {
    // ranges of 128 to 1024 keys, about four for each of the CTAs that run at once
    const long long want = keys * all / (8 * sms);
    f.least = clamp_int(want, 128, 1024) / key_tile;
    f.nsplit = clamp_int((keys + f.least * key_tile - 1) / (f.least * key_tile), 1, std::min<long long>(fit, kPartsLimit));
  } else {
    f.least = 512 / key_tile;
    f.nsplit = clamp_int(ranges(longest, all), 1, std::min<long long>(fit, kPartsLimit));
    // ranges of one length: shorter sequences are cut into fewer
    f.least = (int)std::max<long long>(f.least, (keys + key_tile - 1) / key_tile / f.nsplit);
  }
  f.taper = paged && !f.few && longest * f.nsplit > sms;
  const bool two = two_orders(p);
  f.merge = two && f.nsplit == 1 && !f.few;
  f.nparts = f.merge ? 1 : two ? 2 * f.nsplit : f.nsplit > 1 ? f.nsplit : 0;
  Job jobs[2];
  const int launched = f.merge ? 1 : make_jobs(p, jobs);
  f.fits = f.few || dtype == ST_F32 || units_fit(g, G, rows, (long long)launched * f.nsplit);
  f.parts_o = round256(qrows * g.d * sizeof(float) * f.nparts);
  f.bytes = f.nparts ? f.parts_o + round256(qrows * sizeof(float) * f.nparts) : 0;
  return f;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0);
}

st_status run_fwd(const st_pattern_desc& p, st_dtype dtype, Geo& g, float scale, const FwdPlan& f,
                  const void* q, const void* k, const void* v, void* o, float* lse, void* ws,
                  cudaStream_t stream) {
  FwdLaunch a{};
  a.g = g;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.parts.o = static_cast<float*>(ws);
  a.parts.lse = reinterpret_cast<float*>(static_cast<char*>(ws) + f.parts_o);
  a.nsplit = f.nsplit;
  a.least = f.least;
  a.taper = f.taper;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)g.d)) * 1.4426950408889634f;
  a.wait_ns = wait_limit_ns();
  a.force_timeout = !f.few && dtype != ST_F32 && take_force_timeout();
  a.stream = stream;
  Job jobs[2];
  const int n = make_jobs(p, jobs);
  auto go = [&]() {
    return f.few ? few_rows_fwd(a, dtype) : dtype == ST_F32 ? simt_ragged_fwd(a) : tc_ragged_fwd(a, dtype);
  };
  cudaError_t e = cudaSuccess;
  if (f.merge) {
    // the second order reads what the first left
    a.njobs = 1;
    for (int j = 0; j < n && e == cudaSuccess; ++j) {
      a.job = jobs[j];
      a.mode = j == 0 ? OUT_PARTIAL : OUT_MERGE;
      e = go();
    }
  } else {
    a.job = jobs[0];
    a.job1 = jobs[n - 1];
    a.njobs = n;
    a.part1 = two_orders(p) ? f.nsplit : 0;
    a.mode = f.nparts ? OUT_PARTIAL : OUT_FINAL;
    e = go();
  }
  if (e == cudaSuccess && f.nparts && !f.merge)
    e = join_parts(g, dtype, a.parts, f.nparts, o, lse, stream);
  return e == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

// How a backward call is cut up: key jobs (one segment each), query-row ranges
// per key tile.
struct BwdPlan {
  Job kjob[2];
  int njobs, nsplit;
  bool parts;  // dK, dV are joined from parts
  bool merge;  // the second launch adds the first one's part itself
  bool fits;   // as of the forward
  int mend_tiles, mend_below;
  size_t delta, dq_part, parts_bytes, bytes;
};

BwdPlan plan_bwd(const Geo& g, const st_pattern_desc& p, st_dtype dtype) {
  BwdPlan b{};
  // Units of at most two key tiles are where rows have few keys. With two orders
  // the sums of both are needed: all units, if the band is short; else rows have few
  // keys only where the second order has none for them, below position 2 l.
  if (dtype != ST_F32) {
    b.mend_tiles = two_orders(p) && p.l < 128 ? 0x7fffffff : 2;
    b.mend_below = two_orders(p) && p.l >= 128 && p.l < 0x40000000 ? 2 * p.l : 0x7fffffff;
  }
  Job jobs[2];
  const int n = make_jobs(p, jobs);
  for (int j = 0; j < n; ++j)
    for (int s = 0; s < jobs[j].nseg; ++s)
      b.kjob[b.njobs++] = Job{jobs[j].hc, jobs[j].qview, 1, {jobs[j].seg[s], jobs[j].seg[s]}};
  // key tiles of one longest sequence against the query rows that reach them
  const size_t qrows = (size_t)g.total * g.H, krows = (size_t)g.total * g.Hkv;
  const long long sms = sm_count(), units = ((long long)p.T + 127) / 128 * g.Hkv;
  const long long all = std::max(units, ((long long)g.total + 127) / 128 * g.Hkv);
  const long long fit = std::max(1LL, kPartsBytes / (long long)std::max<size_t>(1, krows * 2 * g.d * sizeof(float) * b.njobs));
  b.nsplit = 1;
  if (units < sms && all < 2 * sms)
    b.nsplit = clamp_int(std::min((sms + units - 1) / units, (long long)p.T * g.G / 512), 1,
                         std::min<long long>(fit, kPartsLimit));
  // Two jobs of every key head and units enough for each job to fill the GPU: the
  // second order goes first and leaves a part, the first order lists every key and
  // adds it. Backward, d = 64, H = 16, Hkv = 8, l = 32, strided, both patterns per head,
  // 64, 256, 512, 1024 key tiles: 68, 154, 215, 373 us against one launch and a join's
  // 57, 155, 236, 428.
  const bool both = b.njobs == 2 && (!g.split || g.G > 1);
  b.merge = both && b.nsplit == 1 && all >= 2 * sms;
  // one part is enough only where every key head has one job over all its keys
  b.parts = !b.merge && (b.nsplit > 1 || (b.njobs == 2 && (both || b.kjob[1].seg[0].kview == VIEW_SUM)));
  b.fits = dtype == ST_F32 ||
           (units_fit(g, g.split ? (g.G + 1) / 2 : g.G, 128, two_orders(p) ? 1 : n) &&
            units_fit(g, 1, 128, (long long)(b.merge ? 1 : b.njobs) * b.nsplit));
  b.delta = round256(qrows * sizeof(float));
  b.dq_part = two_orders(p) ? round256(qrows * g.d * sizeof(float)) : 0;
  const int nparts = b.merge ? 1 : b.parts ? b.njobs * b.nsplit : 0;
  b.parts_bytes = round256(krows * 2 * g.d * sizeof(float) * nparts);
  b.bytes = b.delta + b.dq_part + b.parts_bytes;
  if (b.dq_part && b.mend_tiles > 2) b.bytes += b.delta + b.dq_part;
  return b;
}

}  // namespace

extern "C" {

st_status st_packed_attn_fwd_workspace(const st_pattern_desc* p, st_dtype dtype,
                                       const st_packed_desc* x, size_t* bytes) {
  Geo g;
  if (!bytes) return ST_ERR_INVALID;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s != ST_OK) return s;
  const FwdPlan f = plan_fwd(g, *p, dtype, p->T, false);
  *bytes = f.bytes;
  return f.fits ? ST_OK : ST_ERR_UNSUPPORTED;
}

st_status st_packed_attn_fwd(const st_pattern_desc* p, st_dtype dtype, const st_packed_desc* x,
                             float scale, const void* q, const void* k, const void* v,
                             const int32_t* cu, void* o, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
  Geo g;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s != ST_OK) return s;
  if (g.total == 0) return ST_OK;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned4(cu))
    return ST_ERR_INVALID;
  const FwdPlan f = plan_fwd(g, *p, dtype, p->T, false);
  if (!f.fits) return ST_ERR_UNSUPPORTED;
  if (!workspace_ok(ws, ws_bytes, f.bytes)) return ST_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = get_status(g);
  if (s != ST_OK) return s;
  g.cu = cu;
  return run_fwd(*p, dtype, g, scale, f, q, k, v, o, lse, ws, cs);
}

st_status st_packed_attn_bwd_workspace(const st_pattern_desc* p, st_dtype dtype,
                                       const st_packed_desc* x, size_t* bytes) {
  Geo g;
  if (!bytes) return ST_ERR_INVALID;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s != ST_OK) return s;
  const BwdPlan b = plan_bwd(g, *p, dtype);
  *bytes = b.bytes;
  return b.fits ? ST_OK : ST_ERR_UNSUPPORTED;
}

st_status st_packed_attn_bwd(const st_pattern_desc* p, st_dtype dtype, const st_packed_desc* x,
                             float scale, const void* q, const void* k, const void* v,
                             const void* o, const float* lse, const void* dout, const int32_t* cu,
                             void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                             void* stream) {
  Geo g;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s != ST_OK) return s;
  BwdLaunch a{};
  if (!stride_rows(x->dq_stride, g.H, g.d, &a.dq_rows.tok) ||
      !stride_rows(x->dk_stride, g.Hkv, g.d, &a.dk_rows.tok) ||
      !stride_rows(x->dv_stride, g.Hkv, g.d, &a.dv_rows.tok))
    return ST_ERR_INVALID;
  a.dq_rows.head = a.dk_rows.head = a.dv_rows.head = 1;
  if (g.total == 0) return ST_OK;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned4(cu))
    return ST_ERR_INVALID;
  const BwdPlan b = plan_bwd(g, *p, dtype);
  if (!b.fits) return ST_ERR_UNSUPPORTED;
  if (!workspace_ok(ws, ws_bytes, b.bytes)) return ST_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = get_status(g);
  if (s != ST_OK) return s;
  g.cu = cu;
  a.g = g;
  for (int j = 0; j < 2; ++j) a.job[j] = b.kjob[j];
  a.njobs = b.njobs;
  a.nsplit = b.nsplit;
  a.q = q;
  a.k = k;
  a.v = v;
  a.dout = dout;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  char* w = static_cast<char*>(ws);
  float* delta = reinterpret_cast<float*>(w);
  a.delta = delta;
  w += b.delta;
  a.dq_part = reinterpret_cast<float*>(w);
  w += b.dq_part;
  a.parts = reinterpret_cast<float*>(w);
  w += b.parts_bytes;
  a.mend_tiles = b.mend_tiles;
  a.mend_below = b.mend_below;
  a.r_part = reinterpret_cast<float*>(w);
  a.kb_part = reinterpret_cast<float*>(w + b.delta);
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)g.d);
  a.wait_ns = wait_limit_ns();
  a.stream = cs;
  cudaError_t e = row_delta(g, dtype, o, dout, delta, cs);
  Job jobs[2];
  const int n = make_jobs(*p, jobs);
  auto go_dq = [&]() { return dtype == ST_F32 ? simt_ragged_dq(a) : tc_ragged_dq(a, dtype); };
  if (two_orders(*p)) {
    a.nqjobs = 1;
    for (int j = 0; j < n && e == cudaSuccess; ++j) {
      a.qjob[0] = jobs[j];
      a.mode = j == 0 ? OUT_PARTIAL : OUT_MERGE;
      if (j == 1 && a.mend_tiles == 2) a.mend_tiles = 0;  // the first order has mended
      e = go_dq();
    }
  } else if (e == cudaSuccess) {
    a.qjob[0] = jobs[0];
    a.qjob[1] = jobs[n - 1];
    a.nqjobs = n;
    a.mode = OUT_FINAL;
    e = go_dq();
  }
  auto go_dkv = [&]() { return dtype == ST_F32 ? simt_ragged_dkv(a) : tc_ragged_dkv(a, dtype); };
  if (b.merge) {
    a.njobs = 1;
    a.part_view = b.kjob[1].seg[0].kview;
    for (int j = 1; j >= 0 && e == cudaSuccess; --j) {
      a.job[0] = b.kjob[j];
      a.mode = j == 1 ? OUT_PARTIAL : OUT_MERGE;
      e = go_dkv();
    }
  } else if (e == cudaSuccess) {
    a.mode = OUT_FINAL;
    e = go_dkv();
  }
  if (e == cudaSuccess && b.parts) e = join_dkv(a, dtype);
  return e == cudaSuccess ? ST_OK : ST_ERR_CUDA;
}

st_status st_paged_attn_workspace(const st_pattern_desc* p, st_dtype dtype,
                                  const st_packed_desc* x, const st_cache_desc* c, int32_t max_q,
                                  size_t* bytes) {
  Geo g;
  if (!bytes || max_q < 1) return ST_ERR_INVALID;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s == ST_OK) s = fill_cache(c, g);
  if (s != ST_OK) return s;
  const FwdPlan f = plan_fwd(g, *p, dtype, max_q, true);
  *bytes = f.bytes;
  return f.fits ? ST_OK : ST_ERR_UNSUPPORTED;
}

st_status st_paged_attn(const st_pattern_desc* p, st_dtype dtype, const st_packed_desc* x,
                        const st_cache_desc* c, int32_t max_q, float scale, const void* q,
                        const void* kc, const void* vc, const int32_t* table, const int32_t* cu,
                        const int32_t* kv_lens, void* o, float* lse, void* ws, size_t ws_bytes,
                        void* stream) {
  Geo g;
  if (max_q < 1) return ST_ERR_INVALID;
  st_status s = fill_geo(p, dtype, x, true, g);
  if (s == ST_OK) s = fill_cache(c, g);
  if (s != ST_OK) return s;
  if (g.total == 0) return ST_OK;
  if (!aligned16(q) || !aligned16(kc) || !aligned16(vc) || !aligned16(o) || !aligned16(lse) ||
      !aligned4(cu) || !aligned4(kv_lens) || !aligned4(table))
    return ST_ERR_INVALID;
  const FwdPlan f = plan_fwd(g, *p, dtype, max_q, true);
  if (!f.fits) return ST_ERR_UNSUPPORTED;
  if (!workspace_ok(ws, ws_bytes, f.bytes)) return ST_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = get_status(g);
  if (s != ST_OK) return s;
  g.cu = cu;
  g.kv_lens = kv_lens;
  g.table = table;
  return run_fwd(*p, dtype, g, scale, f, q, kc, vc, o, lse, ws, cs);
}

st_status st_cache_append(st_dtype dtype, const st_packed_desc* x, const st_cache_desc* c,
                          const void* k, const void* v, void* kc, void* vc, const int32_t* table,
                          const int32_t* cu, const int32_t* kv_lens, void* stream) {
  Geo g;
  const st_pattern_desc dense = {ST_DENSE_CAUSAL, ST_HEADS_MERGED, 1, 1, 1};
  if (!x) return ST_ERR_INVALID;
  st_packed_desc y = *x;
  y.H = y.Hkv;
  y.q_stride = 0;
  st_status s = fill_geo(&dense, dtype, &y, false, g);
  if (s != ST_OK) return s;
  if (g.d % (dtype == ST_F32 ? 4 : 8)) return ST_ERR_UNSUPPORTED;
  Geo gc = g;
  s = fill_cache(c, gc);
  if (s != ST_OK) return s;
  if (g.total == 0) return ST_OK;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kc) || !aligned16(vc) || !aligned4(table) ||
      !aligned4(cu) || !aligned4(kv_lens))
    return ST_ERR_INVALID;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  s = get_status(gc);
  if (s != ST_OK) return s;
  gc.cu = cu;
  gc.kv_lens = kv_lens;
  gc.table = table;
  return cache_append(gc, g.k, g.v, dtype == ST_F32 ? 4 : 2, k, v, kc, vc, cs) == cudaSuccess
             ? ST_OK
             : ST_ERR_CUDA;
}

}  // extern "C"

// CUDA-core kernels for attention over ragged sequences: the float32 forward
// and backward (fp32 products and sums throughout), and the streaming kernels
// around every path (delta, joins of parts).
//
// One block of 256 threads (16 x 16) owns 64 rows; 64 x 64 tiles of products
// come from shared memory with a 4 x 4 micro-tile per thread. At 64 rows the
// products do 16 FMAs for 2 float4 loads, so the kernels are bound by shared
// memory and the FMA pipe together. Small calls are bound by latency: the rows of a
// step are loaded together, and the next tile's while one is worked on (256 tokens, H
// = 2, d = 32, strided, forward and backward: 49 us; 61 with one load after the
// other). Dense, 4096 tokens, H = 8: d = 64 0.93 ms forward (18.5 TFLOP/s) and 2.9
// backward, d = 128 1.75 and 5.1.
#include "ragged.h"
#include "tc_common.cuh"

namespace st {
namespace rag {
namespace {

constexpr int BM = 64;   // rows of a unit
constexpr int BN = 64;   // rows of the tiles it meets
constexpr int NT = 256;
constexpr int SP = BN + 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value(__half x) { return __half2float(x); }

// 64 rows of D elements on their way to shared memory, [64][D + 4] there: all loads
// of a step are under way together, and the next tile's while this one is worked on.
template <int D>
struct Staged {
  static constexpr int C4 = D / 4, N = BM * C4 / NT;
  float4 v[N];
  // row(i) gives the row index of tile row i, or -1 for a row of zeros.
  template <class F>
  __device__ __forceinline__ void load(const float* base, F row) {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int y = threadIdx.x + x * NT, i = y / C4, r = row(i);
      v[x] = r >= 0 ? load4(base + (size_t)r * D + (y - i * C4) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* dst) const {
#pragma unroll
    for (int x = 0; x < N; ++x) {
      const int y = threadIdx.x + x * NT, i = y / C4;
      *reinterpret_cast<float4*>(dst + i * (D + 4) + (y - i * C4) * 4) = v[x];
    }
  }
};

// acc[i][j] += A[4 ty + i] . B[tx + 16 j] over D
template <int D>
__device__ __forceinline__ void dot_tile(const float* A, const float* B, int ty, int tx,
                                         float acc[4][4]) {
#pragma unroll 4
  for (int k = 0; k < D; k += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * (D + 4) + k);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (D + 4) + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z,
                         fmaf(a[i].w, b[j].w, acc[i][j]))));
  }
}

// acc[i][j] += sum_k W[4 ty + i][k] * B[k][tx + 16 j]
template <int D>
__device__ __forceinline__ void weigh_tile(const float* W, const float* B, int ty, int tx,
                                           float acc[4][D / 16]) {
#pragma unroll 2
  for (int k = 0; k < BN; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(W + (4 * ty + i) * SP + k);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const float* b = B + k * (D + 4) + tx + 16 * j;
      const float b0 = b[0], b1 = b[D + 4], b2 = b[2 * (D + 4)], b3 = b[3 * (D + 4)];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][j] = fmaf(w[i].w, b3, fmaf(w[i].z, b2, fmaf(w[i].y, b1, fmaf(w[i].x, b0, acc[i][j]))));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(NT, 2) ragged_fwd_simt(const __grid_constant__ FwdLaunch a) {
  extern __shared__ float sm[];
  float* A = sm;
  float* B = A + BM * (D + 4);
  float* W = B + BN * (D + 4);
  float* scl = W + BM * SP;  // per row: factor of the old accumulator
  float* den = scl + BM;     // per row: 1 / sum, at the end
  const Geo& g = a.g;
  const int kvh = blockIdx.y, jb = blockIdx.z / a.nsplit, part = blockIdx.z - jb * a.nsplit;
  const Job& job = jb ? a.job1 : a.job;
  const int part0 = jb ? a.part1 : a.part0;
  int tile;
  const int s = find_slot(g, most_heads(g, job.hc), BM, gridDim.x - 1 - blockIdx.x, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int x0 = tile * BM;
  if (hs.n == 0 || x0 >= q.nq * hs.n) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float* qp = static_cast<const float*>(a.q);
  const float* kp = static_cast<const float*>(a.k);
  const float* vp = static_cast<const float*>(a.v);
  Staged<D> sq, sk, sv;
  sq.load(qp, [&](int i) {
    QRow r;
    return query_at(g, q, job.qview, hs, x0 + i, r) ? q_row(g, r.t, r.h) : -1;
  });
  float acc[4][D / 16] = {};
  // softmax state of row tid / 4, kept by four threads
  const int row = tid >> 2;
  QRow qr;
  const bool have = query_at(g, q, job.qview, hs, x0 + row, qr);
  float m = -INFINITY, sum = 0.f;
  int cnt[2] = {0, 0}, j0[2] = {0, 0}, total = 0;
  for (int sg = 0; sg < job.nseg; ++sg) {
    int j1;
    tile_range(g, q, job, sg, hs, x0, BM, BN, j0[sg], j1);
    cnt[sg] = j1 - j0[sg];
    total += cnt[sg];
  }
  const int parts = parts_of(total, a.nsplit, a.least);
  if (part >= parts) return;
  const int it0 = (int)((long long)total * part / parts), it1 = (int)((long long)total * (part + 1) / parts);
  // key tile it: its segment, its first key
  auto seg_of = [&](int it) { return it >= cnt[0] ? 1 : 0; };
  auto first_key = [&](int it) { return (j0[seg_of(it)] + it - (seg_of(it) ? cnt[0] : 0)) * BN; };
  auto key = [&](int it, int i) {
    const int e = first_key(it) + i, view = job.seg[seg_of(it)].kview;
    return e < n_keys(q, view) ? key_pos(g, q, view, e) : -1;
  };
  auto load_k = [&](int it) {
    sk.load(kp, [&](int i) {
      const int p = key(it, i);
      return p >= 0 ? k_row(g, q, p, kvh) : -1;
    });
  };
  if (it0 < it1) load_k(it0);
  sq.store(A);
  for (int it = it0; it < it1; ++it) {
    const int sg = seg_of(it), kb = first_key(it);
    __syncthreads();
    sk.store(B);
    sv.load(vp, [&](int i) {
      const int p = key(it, i);
      return p >= 0 ? v_row(g, q, p, kvh) : -1;
    });
    __syncthreads();
    float sc[4][4] = {};
    dot_tile<D>(A, B, ty, tx, sc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) W[(4 * ty + i) * SP + tx + 16 * j] = sc[i][j] * a.scale_log2;
    __syncthreads();
    sv.store(B);
    if (it + 1 < it1) load_k(it + 1);
    int lo = 0, hi = 0;
    if (have && qr.pos >= 0) live_keys(g, q, job.seg[sg].rule, qr.pos, lo, hi);
    float mt = -INFINITY;
    for (int x = tid & 3; x < BN; x += 4) {
      const int k = kb + x;
      float v = W[row * SP + x];
      v = (k >= lo && k < hi) ? v : -INFINITY;
      W[row * SP + x] = v;
      mt = fmaxf(mt, v);
    }
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
    mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
    const float mn = fmaxf(m, mt);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float al = exp2f(m - mu);
    float ps = 0.f;
    for (int x = tid & 3; x < BN; x += 4) {
      const float p = exp2f(W[row * SP + x] - mu);
      W[row * SP + x] = p;
      ps += p;
    }
    ps += __shfl_xor_sync(0xffffffffu, ps, 1);
    ps += __shfl_xor_sync(0xffffffffu, ps, 2);
    sum = sum * al + ps;
    m = mn;
    if ((tid & 3) == 0) scl[row] = al;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = scl[4 * ty + i];
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[i][j] *= f;
    }
    weigh_tile<D>(W, B, ty, tx, acc);
  }
  // log-sum-exp of the row; joined with the other order's where asked
  const float lse = sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
  float wc = sum != 0.f ? 1.f / sum : 0.f, wp = 0.f, out = lse;
  const size_t rr = have ? (size_t)qr.t * g.H + qr.h : 0;
  if (a.mode == OUT_MERGE && have) {
    const float lp = a.parts.lse[rr];
    const float mx = fmaxf(lp, lse);
    if (lp != -INFINITY || lse != -INFINITY) {  // NaN stays NaN
      out = mx + logf(expf(lp - mx) + expf(lse - mx));
      wp = expf(lp - out);
      wc *= expf(lse - out);
    }
  }
  __syncthreads();
  if ((tid & 3) == 0) {
    scl[row] = wp;
    den[row] = wc;
    if (have) {
      if (a.mode == OUT_PARTIAL) {
        a.parts.lse[(size_t)(part0 + part) * g.total * g.H + rr] = out;
        if (part == 0)
          for (int p = parts; p < a.nsplit; ++p)
            a.parts.lse[(size_t)(part0 + p) * g.total * g.H + rr] = -INFINITY;
      } else {
        a.lse[rr] = out;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    QRow r;
    if (!query_at(g, q, job.qview, hs, x0 + 4 * ty + i, r)) continue;
    const size_t o = ((size_t)r.t * g.H + r.h) * D;
    const float f = den[4 * ty + i], fp = scl[4 * ty + i];
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const int c = tx + 16 * j;
      float v = acc[i][j] * f;
      if (a.mode == OUT_PARTIAL) {
        a.parts.o[(size_t)(part0 + part) * g.total * g.H * D + o + c] = v;
      } else {
        if (a.mode == OUT_MERGE && fp != 0.f) v = fmaf(fp, a.parts.o[o + c], v);
        static_cast<float*>(a.o)[o + c] = v;
      }
    }
  }
}

// dQ of 64 query rows: S and dP = dO V^T again, dS = P (dP - delta), dQ += dS K.
template <int D>
__global__ void __launch_bounds__(NT, D == 128 ? 1 : 2) ragged_dq_simt(const __grid_constant__ BwdLaunch a) {
  extern __shared__ float sm[];
  float* A = sm;
  float* A2 = A + BM * (D + 4);
  float* B = A2 + BM * (D + 4);
  float* B2 = B + BN * (D + 4);
  float* W = B2 + BN * (D + 4);
  __shared__ float sl[BM], sd[BM];
  __shared__ int slo[BM], shi[BM];
  const Geo& g = a.g;
  const int kvh = blockIdx.y;
  const Job& job = a.qjob[blockIdx.z];
  int tile;
  const int s = find_slot(g, most_heads(g, job.hc), BM, gridDim.x - 1 - blockIdx.x, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int x0 = tile * BM;
  if (hs.n == 0 || x0 >= q.nq * hs.n) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float *kp = static_cast<const float*>(a.k), *vp = static_cast<const float*>(a.v);
  Staged<D> s1, s2;  // Q and dO, then K and V tiles
  s1.load(static_cast<const float*>(a.q), [&](int i) {
    QRow r;
    return query_at(g, q, job.qview, hs, x0 + i, r) ? q_row(g, r.t, r.h) : -1;
  });
  s2.load(static_cast<const float*>(a.dout), [&](int i) {
    QRow r;
    return query_at(g, q, job.qview, hs, x0 + i, r) ? r.t * g.H + r.h : -1;
  });
  QRow mine = {0, 0, -1};
  if (tid < BM) {
    const bool have = query_at(g, q, job.qview, hs, x0 + tid, mine);
    sl[tid] = have ? a.lse[(size_t)mine.t * g.H + mine.h] * kLog2e : 0.f;
    sd[tid] = have ? a.delta[(size_t)mine.t * g.H + mine.h] : 0.f;
    if (!have) mine.pos = -1;
  }
  s1.store(A);
  s2.store(A2);
  const float sc2 = a.scale * kLog2e;
  float acc[4][D / 16] = {};
  for (int sg = 0; sg < job.nseg; ++sg) {
    int j0, j1;
    tile_range(g, q, job, sg, hs, x0, BM, BN, j0, j1);
    const int view = job.seg[sg].kview, nk = n_keys(q, view);
    auto load = [&](int j) {
      s1.load(kp, [&](int i) { return j * BN + i < nk ? k_row(g, q, key_pos(g, q, view, j * BN + i), kvh) : -1; });
      s2.load(vp, [&](int i) { return j * BN + i < nk ? v_row(g, q, key_pos(g, q, view, j * BN + i), kvh) : -1; });
    };
    if (j0 < j1) load(j0);
    __syncthreads();
    if (tid < BM) {
      int lo = 0, hi = 0;
      if (mine.pos >= 0) live_keys(g, q, job.seg[sg].rule, mine.pos, lo, hi);
      slo[tid] = lo;
      shi[tid] = hi;
    }
    for (int j = j0; j < j1; ++j) {
      const int kb = j * BN;
      __syncthreads();
      s1.store(B);
      s2.store(B2);
      if (j + 1 < j1) load(j + 1);
      __syncthreads();
      float sc[4][4] = {}, dp[4][4] = {};
      dot_tile<D>(A, B, ty, tx, sc);
      dot_tile<D>(A2, B2, ty, tx, dp);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int r = 4 * ty + i, k = kb + tx + 16 * jj;
          const bool live = k >= slo[r] && k < shi[r];
          W[r * SP + tx + 16 * jj] =
              live ? exp2f(sc[i][jj] * sc2 - sl[r]) * (dp[i][jj] - sd[r]) : 0.f;
        }
      __syncthreads();
      weigh_tile<D>(W, B, ty, tx, acc);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    QRow r;
    if (!query_at(g, q, job.qview, hs, x0 + 4 * ty + i, r)) continue;
    const size_t po = ((size_t)r.t * g.H + r.h) * D;
    const size_t o = ((size_t)r.t * a.dq_rows.tok + r.h * a.dq_rows.head) * D;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const int c = tx + 16 * j;
      float v = acc[i][j] * a.scale;
      if (a.mode == OUT_PARTIAL) {
        a.dq_part[po + c] = v;
      } else {
        if (a.mode == OUT_MERGE) v += a.dq_part[po + c];
        static_cast<float*>(a.dq)[o + c] = v;
      }
    }
  }
}

// dK, dV of 64 keys: S^T, dP^T = V dO^T, P^T and dS^T, dV += P^T dO, dK += dS^T Q.
template <int D>
__global__ void __launch_bounds__(NT, D == 128 ? 1 : 2) ragged_dkv_simt(const __grid_constant__ BwdLaunch a) {
  extern __shared__ float sm[];
  float* A = sm;
  float* A2 = A + BM * (D + 4);
  float* B = A2 + BM * (D + 4);
  float* B2 = B + BN * (D + 4);
  float* W = B2 + BN * (D + 4);
  float* W2 = W + BM * SP;
  __shared__ float sl[BN], sd[BN];
  __shared__ int sa[BM], sb[BM], lim[2];
  const Geo& g = a.g;
  const int kvh = blockIdx.y;
  const int jb = blockIdx.z / a.nsplit, split = blockIdx.z - jb * a.nsplit;
  const Job& job = a.job[jb];
  int tile;
  const int s = find_slot(g, 1, BM, blockIdx.x, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int view = job.seg[0].kview, rule = job.seg[0].rule;
  const int k0 = tile * BM, nk = n_keys(q, view);
  if (hs.n == 0 || k0 >= nk) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float *kp = static_cast<const float*>(a.k), *vp = static_cast<const float*>(a.v);
  Staged<D> s1, s2;  // K and V, then Q and dO tiles
  s1.load(kp, [&](int i) { return k0 + i < nk ? k_row(g, q, key_pos(g, q, view, k0 + i), kvh) : -1; });
  s2.load(vp, [&](int i) { return k0 + i < nk ? v_row(g, q, key_pos(g, q, view, k0 + i), kvh) : -1; });
  s1.store(A);
  s2.store(A2);
  if (tid < BM) {
    int x = 0, y = 0;
    if (k0 + tid < nk) live_queries(g, q, rule, k0 + tid, x, y);
    sa[tid] = x * hs.n;
    sb[tid] = y * hs.n;
    if (tid == 0) lim[0] = x * hs.n;
    if (k0 + tid == imin(k0 + BM, nk) - 1) lim[1] = y * hs.n;
  }
  __syncthreads();
  const int t0 = lim[0] / BN, t1 = lim[1] > lim[0] ? (lim[1] + BN - 1) / BN : t0;
  const int tb = t0 + (int)((long long)(t1 - t0) * split / a.nsplit);
  const int te = t0 + (int)((long long)(t1 - t0) * (split + 1) / a.nsplit);
  const float sc2 = a.scale * kLog2e;
  float dk[4][D / 16] = {}, dv[4][D / 16] = {};
  float nl = 0.f, nd = 0.f;  // LSE log2(e) and D of row tid
  auto load = [&](int t) {
    s1.load(static_cast<const float*>(a.q), [&](int i) {
      QRow r;
      return query_at(g, q, job.qview, hs, t * BN + i, r) ? q_row(g, r.t, r.h) : -1;
    });
    s2.load(static_cast<const float*>(a.dout), [&](int i) {
      QRow r;
      return query_at(g, q, job.qview, hs, t * BN + i, r) ? r.t * g.H + r.h : -1;
    });
    if (tid < BN) {
      QRow r;
      const bool have = query_at(g, q, job.qview, hs, t * BN + tid, r);
      nl = have ? a.lse[(size_t)r.t * g.H + r.h] * kLog2e : 0.f;
      nd = have ? a.delta[(size_t)r.t * g.H + r.h] : 0.f;
    }
  };
  if (tb < te) load(tb);
  for (int t = tb; t < te; ++t) {
    const int xb = t * BN;
    __syncthreads();
    s1.store(B);
    s2.store(B2);
    if (tid < BN) {
      sl[tid] = nl;
      sd[tid] = nd;
    }
    if (t + 1 < te) load(t + 1);
    __syncthreads();
    float sc[4][4] = {}, dp[4][4] = {};
    dot_tile<D>(A, B, ty, tx, sc);
    dot_tile<D>(A2, B2, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * ty + i, cq = tx + 16 * j, x = xb + cq;
        const bool live = x >= sa[r] && x < sb[r];
        const float p = live ? exp2f(sc[i][j] * sc2 - sl[cq]) : 0.f;
        W[r * SP + cq] = p;
        W2[r * SP + cq] = live ? p * (dp[i][j] - sd[cq]) : 0.f;
      }
    __syncthreads();
    weigh_tile<D>(W, B2, ty, tx, dv);
    weigh_tile<D>(W2, B, ty, tx, dk);
  }
  const bool direct = dkv_direct(a, kvh);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = k0 + 4 * ty + i;
    if (k >= nk) continue;
    const int pos = key_pos(g, q, view, k), t = q.qb + pos;
    float* p = a.parts + (((size_t)blockIdx.z * g.total + t) * g.Hkv + kvh) * 2 * D;
    const bool add = a.mode == OUT_MERGE && view_lists(g, a.part_view, pos);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      const int c = tx + 16 * j;
      dk[i][j] *= a.scale;
      if (add) {
        dk[i][j] += p[c];
        dv[i][j] += p[D + c];
      }
      if (direct) {
        static_cast<float*>(a.dk)[((size_t)t * a.dk_rows.tok + kvh * a.dk_rows.head) * D + c] =
            dk[i][j];
        static_cast<float*>(a.dv)[((size_t)t * a.dv_rows.tok + kvh * a.dv_rows.head) * D + c] = dv[i][j];
      } else {
        p[c] = dk[i][j];
        p[D + c] = dv[i][j];
      }
    }
  }
}

// Sequence of token row t (the warp's), or false for a row of no sequence.
__device__ __forceinline__ bool seq_of_token(const Geo& g, int t, int& s) {
  // the last sequence that starts at or before t
  s = last_true(g.S, [&](int x) { return cu_at(g, x) <= t; });
  return t >= cu_at(g, s) && t < cu_at(g, s + 1);
}

constexpr int kJoinRows = 8;  // rows (warps) of a block of the streaming kernels

// Whether token row t belongs to a sequence (they follow one another).
__device__ __forceinline__ bool in_sequence(const Geo& g, int t) {
  return t >= cu_at(g, 0) && t < cu_at(g, g.S);
}

// Position of a token row in its sequence, by one thread.
__device__ __forceinline__ int token_pos(const Geo& g, int t) {
  int a = 0, b = g.S - 1;
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (cu_at(g, m) <= t) a = m;
    else b = m - 1;
  }
  return t - cu_at(g, a);
}

template <class T>
__device__ __forceinline__ void store4(T* p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack2<false>(v.x, v.y), tc::pack2<false>(v.z, v.w));
}
template <>
__device__ __forceinline__ void store4<__half>(__half* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack2<true>(v.x, v.y), tc::pack2<true>(v.z, v.w));
}

constexpr int kJoinThreads = 256;

// o = sum_p exp(lse_p - lse) o_p: one thread per four elements of a query row. A part
// whose LSE is NaN makes the row NaN.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
    join_parts_kernel(const __grid_constant__ Geo g, const Parts parts, int nparts, int shift, T* o,
                      float* lse) {
  const long long x = (long long)blockIdx.x * kJoinThreads + threadIdx.x;
  const long long row = x >> shift;
  const int c = (int)(x - (row << shift)) * 4;
  const long long rows = (long long)g.total * g.H;
  if (row >= rows || !in_sequence(g, (int)(row / g.H))) return;
  float m = -INFINITY;
  bool any = false;  // whether a part is not empty (fmaxf passes over NaN)
#pragma unroll 4
  for (int p = 0; p < nparts; ++p) {
    const float f = __ldg(parts.lse + p * rows + row);
    m = fmaxf(m, f);
    any |= f != -INFINITY;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (any) {
#pragma unroll 4
    for (int p = 0; p < nparts; ++p) {
      const float w = expf(__ldg(parts.lse + p * rows + row) - m);
      if (w != 0.f) {  // a part without weight may not have been written
        const float4 v = __ldg(reinterpret_cast<const float4*>(parts.o + (p * rows + row) * g.d + c));
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
        sum += w;
      }
    }
    const float inv = 1.f / sum;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
  store4(o + row * g.d + c, acc);
  if (c == 0) lse[row] = any ? m + logf(sum) : -INFINITY;
}

// delta = dout . o of every row: 16 bytes a lane of o and of dout, 2^shift lanes a
// row, four rows of a lane in flight.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
    row_delta_kernel(long long rows, int shift, const T* o, const T* dout, float* delta) {
  constexpr int E = 16 / sizeof(T), U = 4;
  const int lane = threadIdx.x & 31, per = 32 >> shift;  // rows of a warp at a time
  const long long first = ((long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5)) * U * per;
  const int sub = lane >> shift, c = (lane & ((1 << shift) - 1)) * E;
  const int d = E << shift;
  uint4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = first + u * per + sub;
    if (row < rows) {
      a[u] = __ldg(reinterpret_cast<const uint4*>(o + row * d + c));
      b[u] = __ldg(reinterpret_cast<const uint4*>(dout + row * d + c));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long row = first + u * per + sub;
    float acc = 0.f;
    if (row < rows) {
      const T* x = reinterpret_cast<const T*>(&a[u]);
      const T* y = reinterpret_cast<const T*>(&b[u]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc = fmaf(value(x[e]), value(y[e]), acc);
    }
    for (int y = 1 << (shift - 1); y; y >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, y);
    if (c == 0 && row < rows) delta[row] = acc;
  }
}

// dK, dV: the parts that hold a key row, added in order; one thread per four
// elements of the pair.
template <class T>
__global__ void __launch_bounds__(kJoinThreads)
    join_dkv_kernel(const __grid_constant__ BwdLaunch a, int shift) {
  const Geo& g = a.g;
  const long long x = (long long)blockIdx.x * kJoinThreads + threadIdx.x;
  const long long row = x >> shift, rows = (long long)g.total * g.Hkv;
  const int c = (int)(x - (row << shift)) * 4;
  if (row >= rows) return;
  const int t = (int)(row / g.Hkv), kvh = (int)(row - (long long)t * g.Hkv);
  if (dkv_direct(a, kvh) || !in_sequence(g, t)) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < a.njobs; ++j) {
    if (!job_reaches(g, a.job[j], kvh)) continue;
    const int view = a.job[j].seg[0].kview;
    if (view == VIEW_SUM && !view_lists(g, view, token_pos(g, t))) continue;
#pragma unroll 4
    for (int p = j * a.nsplit; p < (j + 1) * a.nsplit; ++p) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.parts + (p * rows + row) * 2 * g.d + c));
      acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
    }
  }
  T* dst = c < g.d ? static_cast<T*>(a.dk) + ((size_t)t * a.dk_rows.tok + kvh * a.dk_rows.head) * g.d + c
                   : static_cast<T*>(a.dv) + ((size_t)t * a.dv_rows.tok + kvh * a.dv_rows.head) * g.d + c - g.d;
  store4(dst, acc);
}

// One warp per new token: the 16-byte chunks of its key and value rows, head by
// head, go to the slot of its position, eight in flight a lane. Tokens at negative
// positions are dropped; so are positions past the page table and pages outside
// the cache, which are reported, as is a length outside the page table. Bound by
// the copy itself: 36.8 k tokens of 4 KB (302 MB moved) take 53 us, 5.7 TB/s (a warp
// per token and head: 111 us, each looking its sequence and page up for 512 bytes).
__global__ void __launch_bounds__(32 * kJoinRows)
    cache_append_kernel(const __grid_constant__ Geo g, const Rows kin, const Rows vin, int row_chunks,
                        FastDiv frow, const uint4* k, const uint4* v, uint4* kc, uint4* vc) {
  const int t = blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (t >= g.total) return;
  int s;
  if (!seq_of_token(g, t, s)) return;
  const int len = __ldg(g.kv_lens + s);
  if (len < 0 || len > g.max_pages * g.page_size) set_status(g.status, ST_ERR_INVALID);
  if (len < 0) return;
  const int pos = len - (cu_at(g, s + 1) - t);
  if (pos < 0) return;
  const int pg = fdiv(pos, g.fpage);
  const int page = pg < g.max_pages ? __ldg(g.table + (size_t)s * g.max_pages + pg) : -1;
  if ((unsigned)page >= (unsigned)g.num_pages) {
    set_status(g.status, ST_ERR_INVALID);
    return;
  }
  const size_t slot = (size_t)page * g.k.page + (size_t)(pos - pg * g.page_size) * g.k.tok;
  const int n = g.Hkv * row_chunks;  // of K, and of V
  const uint4* ks = k + (size_t)t * kin.tok * row_chunks;
  const uint4* vs = v + (size_t)t * vin.tok * row_chunks;
  for (int c0 = lane; c0 < n; c0 += 128) {
    uint4 a[4], b[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (c0 + 32 * x < n) {
        a[x] = __ldg(ks + c0 + 32 * x);
        b[x] = __ldg(vs + c0 + 32 * x);
      }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int c = c0 + 32 * x;
      if (c < n) {
        const int h = fdiv(c, frow);
        const size_t dst = (slot + (size_t)h * g.k.head) * row_chunks + (c - h * row_chunks);
        kc[dst] = a[x];
        vc[dst] = b[x];
      }
    }
  }
}

template <class K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int D>
cudaError_t fwd_t(const FwdLaunch& a) {
  const size_t smem = sizeof(float) * (2 * BM * (D + 4) + BM * SP + 2 * BM);
  cudaError_t e = allow_smem(ragged_fwd_simt<D>, smem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(a.g, most_heads(a.g, a.job.hc), BM);
  ragged_fwd_simt<D><<<dim3((unsigned)slots, a.g.Hkv, a.njobs * a.nsplit), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t dq_t(const BwdLaunch& a) {
  const size_t smem = sizeof(float) * (4 * BM * (D + 4) + BM * SP);
  cudaError_t e = allow_smem(ragged_dq_simt<D>, smem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(a.g, most_heads(a.g, a.qjob[0].hc), BM);
  ragged_dq_simt<D><<<dim3((unsigned)slots, a.g.Hkv, a.nqjobs), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t dkv_t(const BwdLaunch& a) {
  const size_t smem = sizeof(float) * (4 * BM * (D + 4) + 2 * BM * SP);
  cudaError_t e = allow_smem(ragged_dkv_simt<D>, smem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(a.g, 1, BM);
  ragged_dkv_simt<D>
      <<<dim3((unsigned)slots, a.g.Hkv, a.njobs * a.nsplit), NT, smem, a.stream>>>(a);
  return cudaGetLastError();
}

template <class F>
cudaError_t pick(int d, F f) {
  switch (d) {
    case 32: return f.template run<32>();
    case 64: return f.template run<64>();
    case 128: return f.template run<128>();
  }
  return cudaErrorInvalidValue;
}

struct RunFwd {
  const FwdLaunch& a;
  template <int D>
  cudaError_t run() { return fwd_t<D>(a); }
};
struct RunDq {
  const BwdLaunch& a;
  template <int D>
  cudaError_t run() { return dq_t<D>(a); }
};
struct RunDkv {
  const BwdLaunch& a;
  template <int D>
  cudaError_t run() { return dkv_t<D>(a); }
};

unsigned join_blocks(long long rows) { return (unsigned)((rows + kJoinRows - 1) / kJoinRows); }

}  // namespace

cudaError_t simt_ragged_fwd(const FwdLaunch& a) { return pick(a.g.d, RunFwd{a}); }
cudaError_t simt_ragged_dq(const BwdLaunch& a) {
  return pick(a.g.d, RunDq{a});
}
cudaError_t simt_ragged_dkv(const BwdLaunch& a) {
  return pick(a.g.d, RunDkv{a});
}

namespace {
int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
unsigned join_grid(long long threads) { return (unsigned)((threads + kJoinThreads - 1) / kJoinThreads); }

template <class T>
cudaError_t join_parts_t(const Geo& g, const Parts& parts, int nparts, void* o, float* lse, cudaStream_t s) {
  const int shift = log2_of(g.d / 4);
  join_parts_kernel<T><<<join_grid(((long long)g.total * g.H) << shift), kJoinThreads, 0, s>>>(
      g, parts, nparts, shift, static_cast<T*>(o), lse);
  return cudaGetLastError();
}
template <class T>
cudaError_t row_delta_t(const Geo& g, const void* o, const void* dout, float* delta, cudaStream_t s) {
  const long long rows = (long long)g.total * g.H;
  const int shift = log2_of(g.d * (int)sizeof(T) / 16);
  const long long per = (32 >> shift) * 4;
  row_delta_kernel<T><<<join_grid((rows + per - 1) / per * 32), kJoinThreads, 0, s>>>(
      rows, shift, static_cast<const T*>(o), static_cast<const T*>(dout), delta);
  return cudaGetLastError();
}
template <class T>
cudaError_t join_dkv_t(const BwdLaunch& a) {
  const int shift = log2_of(a.g.d / 2);
  join_dkv_kernel<T><<<join_grid(((long long)a.g.total * a.g.Hkv) << shift), kJoinThreads, 0, a.stream>>>(a, shift);
  return cudaGetLastError();
}
}  // namespace

cudaError_t join_parts(const Geo& g, int dtype, const Parts& parts, int nparts, void* o, float* lse,
                       cudaStream_t s) {
  return dtype == ST_F32    ? join_parts_t<float>(g, parts, nparts, o, lse, s)
         : dtype == ST_BF16 ? join_parts_t<__nv_bfloat16>(g, parts, nparts, o, lse, s)
                            : join_parts_t<__half>(g, parts, nparts, o, lse, s);
}

cudaError_t row_delta(const Geo& g, int dtype, const void* o, const void* dout, float* delta,
                      cudaStream_t s) {
  return dtype == ST_F32    ? row_delta_t<float>(g, o, dout, delta, s)
         : dtype == ST_BF16 ? row_delta_t<__nv_bfloat16>(g, o, dout, delta, s)
                            : row_delta_t<__half>(g, o, dout, delta, s);
}

cudaError_t join_dkv(const BwdLaunch& a, int dtype) {
  return dtype == ST_F32    ? join_dkv_t<float>(a)
         : dtype == ST_BF16 ? join_dkv_t<__nv_bfloat16>(a)
                            : join_dkv_t<__half>(a);
}

cudaError_t cache_append(const Geo& g, const Rows& kin, const Rows& vin, int elem_bytes,
                         const void* k, const void* v, void* kc, void* vc, cudaStream_t s) {
  const int row_chunks = g.d * elem_bytes / 16;
  cache_append_kernel<<<join_blocks(g.total), 32 * kJoinRows, 0, s>>>(
      g, kin, vin, row_chunks, make_fastdiv(row_chunks), static_cast<const uint4*>(k),
      static_cast<const uint4*>(v), static_cast<uint4*>(kc), static_cast<uint4*>(vc));
  return cudaGetLastError();
}

}  // namespace rag
}  // namespace st

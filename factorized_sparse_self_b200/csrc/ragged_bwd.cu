// Backward of attention over packed ragged sequences on the tensor cores (bf16,
// fp16; d = 64, 128): two kernels of one build.
//
// dS = P (dP - D) with P = exp(s - LSE) formed again, dP = dO V^T, D = dO . O.
//   query-major (dQ):    resident Q, dO of 128 query rows; K, V tiles pass by:
//                        S = Q K^T, dP = dO V^T, dQ += dS K
//   key-major (dK, dV):  resident K, V of 128 keys; Q, dO tiles pass by:
//                        S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
// That is seven products where a single kernel needs five, but every gradient
// row is summed in TMEM by one CTA: no fp32 accumulators in memory, no atomics,
// and the results are the same in every run. Rows of a unit are (query, head of
// the group) pairs, so dK and dV of grouped heads are sums over more rows.
//
// D = dO . O comes from the rounded O. Where a row has many keys O is small beside
// dP and so is that error; where it has few, it is as large as the rounding of dS.
// Rows of dS sum to zero, so r = sum_j P (dP - D) is what D lost. In units of few
// key tiles the query-major kernel also sums P K, takes r times it from dQ, and
// hands D + r to the key-major kernel, which therefore runs after it. (Errors of dQ
// and dK over that of rounding the result: strided, l = 100, split, fp16 1.72 -> 1.42;
// fixed, l = 20, bf16 1.68 -> 1.42; dense, 2000 tokens 1.51 -> 1.41.) At d = 128 the sum
// takes the second S's place in TMEM for those units (dQ of a dense step 264 -> 272 us).
//
// One CTA per SM (384 threads), units claimed from the grid. Warps 0..7 are two
// warpgroups that share the 128 rows and take 64 columns each of a 128 x 128
// tile (thread = row = TMEM lane); P and dS go back to TMEM as 16-bit pairs over
// columns that have been read and are the A operand from there, so they never pass
// through shared memory. Both are rounded to the tensors' type: one type for both
// operands of a product (a weight of dV errs by 2^-8 in bf16, 2^-11 in fp16, relative
// to itself). Warp 9 issues the products, warps 8 and 11 load rows, warp 10 decodes
// units.
// TMEM: S, dP (key-major: transposed), 128 columns each, then the accumulators, d
// columns each: dQ and P K, or dV and dK. P and dS both go over dP, so S is free as
// soon as it is in registers and the next tile's is formed under this one's
// exponentials. Query-major there is room for two S (not at d = 128 where units of any
// length mend): P and dS go over S, and the next dP is formed before the tile's
// products, not behind them (backward of 12288 rasters, l = 192, split: 223 against 241
// us).
#include "ragged_tc.cuh"

namespace st {
namespace rag {
namespace {

constexpr int kThreads = 384;
constexpr int kSched = 2;  // ring of decoded units
constexpr int kAhead = 3;  // tiles before a unit's end at which the next is claimed
constexpr uint32_t kRegsCompute = 200, kRegsIssue = 104;  // 168 at launch: 2 * 200 + 104 = 3 * 168
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = 128 * D * 2;
  // ring slots of the first streamed operand (K or Q, held until the tile's last
  // product) and of the second (V or dO, let go earlier)
  static constexpr int kA = D == 64 ? 4 : 3, kB = D == 64 ? 4 : 2;
  // resident buffers: with two the next unit's rows load under this one (d = 128
  // has no room)
  static constexpr int kRes = D == 64 ? 2 : 1;
};

// 128 rows of one (sequence, key/value head): query rows or keys.
struct BUnit {
  int32_t live;
  Seq q;
  Heads3 hs;
  int32_t kvh, job, split;
  int32_t r0;      // first row (query-major: of the unit's rows; key-major: key index)
  int32_t t0, t1;  // tiles of the other side
  int32_t cnt0;    // query-major: tiles of segment 0
  int32_t u0[2];   // query-major: first tile of each segment
  int32_t mend;    // query-major: whether its rows' D is mended
};

template <int D>
struct alignas(1024) Smem {
  uint8_t res[Cfg<D>::kRes][2][Cfg<D>::kTileBytes];  // Q, dO or K, V
  uint8_t ring[Cfg<D>::kA + Cfg<D>::kB][Cfg<D>::kTileBytes];
  float nlse[2][128], ndel[2][128];    // key-major: -LSE log2(e) and -D of a tile's query rows
                                       // (mend: ndel holds the two halves of r)
  uint64_t r_full[Cfg<D>::kRes], r_empty[Cfg<D>::kRes];
  uint64_t full[Cfg<D>::kA + Cfg<D>::kB], empty[Cfg<D>::kA + Cfg<D>::kB];
  uint64_t s_full[2], s_free, dp_full, ds_ready, acc_full, r_sum, kb_read;
  uint64_t row_full[2], row_empty[2];
  uint64_t sched_full[kSched], sched_empty[kSched];
  uint64_t fin;
  alignas(16) uint4 claim;
  uint64_t claim_bar, want;
  BUnit unit[kSched];
  uint32_t tmem;
  int abort;
};

// Query-major unit n of the query jobs (all segments), or key-major unit n.
template <bool DKV>
__device__ __forceinline__ bool decode(const BwdLaunch& a, int slots, int n, BUnit* out) {
  const Geo& g = a.g;
  const int lane = threadIdx.x & 31;
  int split = 0, jb = 0, m = n;
  if constexpr (DKV) {
    split = m % a.nsplit;
    m /= a.nsplit;
  }
  const int nj = DKV ? a.njobs : a.nqjobs;
  jb = m % nj;
  m /= nj;
  const Job& job = DKV ? a.job[jb] : a.qjob[jb];
  const int kvh = m % g.Hkv;
  // query-major: a sequence's last rows see the most keys; key-major: its first
  // keys are seen by the most rows
  const int slot = DKV ? m / g.Hkv : slots - 1 - m / g.Hkv;
  int tile;
  const int s = find_slot(g, DKV ? 1 : most_heads(g, job.hc), 128, slot, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int r0 = tile * 128;
  if (hs.n == 0) return false;
  int t0, t1, cnt0 = 0, u0[2] = {0, 0};
  if constexpr (DKV) {
    const int nk = n_keys(q, job.seg[0].kview);
    if (r0 >= nk) return false;
    int x0, x1, y;
    live_queries(g, q, job.seg[0].rule, r0, x0, y);
    live_queries(g, q, job.seg[0].rule, imin(r0 + 128, nk) - 1, y, x1);
    t0 = x0 * hs.n / 128;
    t1 = x1 > x0 ? (x1 * hs.n + 127) / 128 : t0;
    const int c = t1 - t0;
    t1 = t0 + (int)((long long)c * (split + 1) / a.nsplit);
    t0 = t0 + (int)((long long)c * split / a.nsplit);
  } else {
    if (r0 >= q.nq * hs.n) return false;
    int e0, e1, c1 = 0;
    tile_range(g, q, job, 0, hs, r0, 128, 128, e0, e1);
    u0[0] = e0;
    cnt0 = e1 - e0;
    if (job.nseg > 1) {
      tile_range(g, q, job, 1, hs, r0, 128, 128, e0, e1);
      u0[1] = e0;
      c1 = e1 - e0;
    }
    t0 = 0;
    t1 = cnt0 + c1;
  }
  if (lane == 0) {
    out->live = 1;
    out->q = q;
    out->hs = hs;
    out->kvh = kvh;
    out->job = jb;
    out->split = split;
    out->r0 = r0;
    out->t0 = t0;
    out->t1 = t1;
    out->cnt0 = cnt0;
    out->u0[0] = u0[0];
    out->u0[1] = u0[1];
    // (positions by the natural order; a limit is set for no other)
    out->mend = !DKV && a.mend_tiles > 0 && t1 - t0 <= a.mend_tiles &&
                fdiv(imin(r0 + 128, q.nq * hs.n) - 1, hs.f) < a.mend_below;
  }
  __syncwarp();
  return true;
}

// MEND (query-major): some units (those of few key tiles) mend D; ALL: any unit may
// (d = 128: tensor memory then has no room for a second S).
template <int D, bool F16, bool DKV, bool MEND, bool ALL>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_bwd_tc(const __grid_constant__ BwdLaunch a, const __grid_constant__ TileMaps maps, int slots) {
  extern __shared__ __align__(1024) uint8_t raw[];
  Smem<D>& S = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int NA = Cfg<D>::kA, NB = Cfg<D>::kB, NS = NA + NB, TB = Cfg<D>::kTileBytes,
                NR = Cfg<D>::kRes;
  constexpr bool TWO_S = !DKV && (D == 64 || !ALL);
  // d = 128: a unit that mends has one S, its sums P K take the place of the other
  constexpr bool SHARE = MEND && TWO_S && D == 128;
  constexpr uint32_t kDP = TWO_S ? 256 : 128, kAcc = kDP + 128;
  constexpr uint32_t kDQ = kAcc, kKB = SHARE ? 128 : kAcc + D, kDV = kAcc, kDK = kAcc + D;
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = a.wait_ns;
  volatile int* abort = &S.abort;
  if (smem_u32(raw) & 1023) {  // operand tiles need it; without static shared memory it holds
    if (threadIdx.x == 0) set_status(g.status, ST_ERR_UNSUPPORTED);
    return;
  }
  if (threadIdx.x == 0) {
    S.abort = 0;
    for (int i = 0; i < NR; ++i) {
      mbar_init(&S.r_full[i], 2);  // both producers
      mbar_init(&S.r_empty[i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.full[i], 2);
      mbar_init(&S.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.row_full[i], 2);
      mbar_init(&S.row_empty[i], 8);
    }
    mbar_init(&S.s_full[0], 1);
    mbar_init(&S.s_full[1], 1);
    mbar_init(&S.dp_full, 1);
    mbar_init(&S.s_free, 256);
    mbar_init(&S.ds_ready, 256);
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.r_sum, 256);
    mbar_init(&S.kb_read, 256);
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&S.sched_full[i], 1);
      mbar_init(&S.sched_empty[i], 11);  // two producers, MMA, eight compute warps
    }
    mbar_init(&S.fin, 1);
    mbar_init(&S.claim_bar, 1);
    mbar_init(&S.want, 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&S.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  auto fail = [&]() {
    S.abort = 1;
    set_status(g.status, ST_ERR_DEVICE_TIMEOUT);
  };

  if (warp >= 8) {
    regs_decrease<kRegsIssue>();
    if (warp == 10) {
      // ---------------- scheduler ----------------
      int k = 0;
      bool ok = true;
      auto slot_free = [&]() {
        return k < kSched || __all_sync(0xffffffffu, bar_wait(&S.sched_empty[k % kSched],
                                                              (k / kSched + 1) & 1, limit, abort));
      };
      Claims claims = {&S.claim, &S.claim_bar, &S.want, 0, 0, 0, true};
      for (int n = blockIdx.x; n >= 0;) {
        ok = slot_free();
        if (!ok) break;
        const bool some = decode<DKV>(a, slots, n, &S.unit[k % kSched]);
        if (some) {
          __threadfence_block();
          if (lane == 0) mbar_arrive(&S.sched_full[k % kSched]);
          ++k;
        }
        n = claims_take(claims, some, limit, abort);
        ok = n != -2;
      }
      if (ok) ok = slot_free();
      if (ok && lane == 0) {
        S.unit[k % kSched].live = 0;
        __threadfence_block();
        mbar_arrive(&S.sched_full[k % kSched]);
      }
      if (!ok) {
        if (lane == 0) fail();
        claims_drop(claims, limit);
      }
    } else if (warp != 9) {
      // ---------------- producers ----------------
      const int pw = warp == 8 ? 0 : 1;  // rows 64 pw .. of every tile
      int used = 0, tt = 0;              // units with tiles, tiles
      bool ok = true;
      Gathers gath;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, bar_test(bar, parity))) {
          gath.flush();  // what others wait for before they free this
          ok = __all_sync(0xffffffffu, bar_wait(bar, parity, limit, abort));
        }
        return ok;
      };
      for (int n = 0;; ++n) {
        if (!wait(&S.sched_full[n % kSched], (n / kSched) & 1) || !S.unit[n % kSched].live) break;
        const BUnit& u = S.unit[n % kSched];
        if (u.t1 > u.t0) {
          const Job& job = DKV ? a.job[u.job] : a.qjob[u.job];
          const int xrows = u.q.nq * u.hs.n;
          // row numbers of Q (in q) and dO (contiguous) of query row x
          auto query_rows = [&](int x, int& rq, int& ro) {
            QRow qr;
            query_at(g, u.q, job.qview, u.hs, imin(x, xrows - 1), qr);
            rq = q_row(g, qr.t, qr.h);
            ro = qr.t * g.H + qr.h;
          };
          auto key_rows = [&](int view, int e, int& rk, int& rv) {
            const int pos = key_pos(g, u.q, view, imin(e, n_keys(u.q, view) - 1));
            kv_rows(g, u.q, pos, u.kvh, rk, rv);
          };
          const int rs = used % NR;
          if (used >= NR && !wait(&S.r_empty[rs], (used / NR + 1) & 1)) break;
          ++used;
          const int rview = job.seg[0].kview;
          const int rbox = DKV ? box_rows(maps, g, u.q, rview, u.r0 / 128)
                               : (job.qview == VIEW_NAT && u.r0 + 128 <= xrows ? maps.q_tokens : 0);
          if (rbox) {
            // each producer loads one of the two tiles
            if (DKV) load_boxes<D>(smem_u32(S.res[rs][pw]), maps, pw, &S.r_full[rs], g, u.q, rview, u.r0 / 128, u.kvh, rbox);
            else load_query_boxes<D>(smem_u32(S.res[rs][pw]), pw ? &maps.dout : &maps.q, &S.r_full[rs], maps, u.q, u.hs, u.r0);
          } else {
            int ra[2], rb[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int e = u.r0 + pw * 64 + y * 32 + lane;
              if (DKV) key_rows(job.seg[0].kview, e, ra[y], rb[y]);
              else query_rows(e, ra[y], rb[y]);
            }
            gather64<D>(smem_u32(S.res[rs][0]), pw * 64, DKV ? a.k : a.q, ra[0], ra[1]);
            gather64<D>(smem_u32(S.res[rs][1]), pw * 64, DKV ? a.v : a.dout, rb[0], rb[1]);
            gath.add(&S.r_full[rs]);
          }
          for (int t = u.t0; t < u.t1; ++t, ++tt) {
            if (pw == 0 && lane == 0 && t == imax(u.t0, u.t1 - kAhead)) mbar_arrive(&S.want);
            int view = 0, j = t, R;
            if constexpr (DKV) {
              R = job.qview == VIEW_NAT && j * 128 + 128 <= xrows ? maps.q_tokens : 0;
            } else {
              const int seg = t >= u.cnt0 ? 1 : 0;
              j = u.u0[seg] + t - (seg ? u.cnt0 : 0);
              view = job.seg[seg].kview;
              R = box_rows(maps, g, u.q, view, j);
            }
            int ra[2], rb[2];
            float vl[2], vd[2];
            if (DKV || !R) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int e = j * 128 + pw * 64 + y * 32 + lane;
                if (DKV) query_rows(e, ra[y], rb[y]);
                else key_rows(view, e, ra[y], rb[y]);
              }
            }
            if (DKV) {
              // -LSE log2(e) and -D of the tile's rows 64 pw ..; rows with an
              // empty set have no live entry and get 0
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float f = __ldg(a.lse + rb[y]);
                vl[y] = f == -INFINITY ? 0.f : -f * kLog2e;
                vd[y] = -__ldg(a.delta + rb[y]);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int n = i ? NB : NA, s = (i ? NA : 0) + tt % n;
              if (tt >= n && !wait(&S.empty[s], (tt / n + 1) & 1)) break;
              if (!R) {
                gather64<D>(smem_u32(S.ring[s]), pw * 64, DKV ? (i ? a.dout : a.q) : (i ? a.v : a.k),
                            i ? rb[0] : ra[0], i ? rb[1] : ra[1]);
                gath.add(&S.full[s]);
              } else {
                gath.flush();
                if (pw == 1) {
                  if (lane == 0) mbar_arrive(&S.full[s]);
                } else if (DKV) {
                  load_query_boxes<D>(smem_u32(S.ring[s]), i ? &maps.dout : &maps.q, &S.full[s], maps, u.q, u.hs,
                                      j * 128);
                } else {
                  load_boxes<D>(smem_u32(S.ring[s]), maps, i, &S.full[s], g, u.q, view, j, u.kvh, R);
                }
              }
              if (DKV && i == 0) {
                const int b = tt & 1;
                if (tt >= 2 && !wait(&S.row_empty[b], (tt / 2 + 1) & 1)) break;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  S.nlse[b][pw * 64 + y * 32 + lane] = vl[y];
                  S.ndel[b][pw * 64 + y * 32 + lane] = vd[y];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.row_full[b]);
              }
            }
            if (!ok) break;
          }
          if (!ok) break;
        } else if (pw == 0 && lane == 0) {
          mbar_arrive(&S.want);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.sched_empty[n % kSched]);
      }
      gath.flush();
      if (!ok && lane == 0) fail();
      // copies in flight land before the CTA may exit (another role may have given up
      // without waiting for them); a tile that was begun may have filled its slots
      const int end = ok ? tt : tt + 1;
      for (int i = imax(0, used - NR); i < used; ++i) mbar_wait_drain(&S.r_full[i % NR], (i / NR) & 1, limit);
      for (int i = imax(0, end - NA); i < end; ++i) mbar_wait_drain(&S.full[i % NA], (i / NA) & 1, limit);
      for (int i = imax(0, end - NB); i < end; ++i) mbar_wait_drain(&S.full[NA + i % NB], (i / NB) & 1, limit);
    } else {
      // ---------------- MMA issuer ----------------
      const uint32_t idS = idesc_16(128, 128, false, false, F16);
      const uint32_t idA = idesc_16(128, D, false, true, F16);
      // A lane's failed wait is remembered and agreed on at the end of the unit:
      // until then the warp goes on (later waits of that lane return at once).
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = bar_wait(bar, parity, limit, abort);
        __syncwarp();
      };
      const uint64_t res0 = sdesc(smem_u32(S.res[0][0]), 16, 1024);
      const uint64_t bk = sdesc(smem_u32(S.ring[0]), 16, 1024), bm = sdesc(smem_u32(S.ring[0]), 16384, 1024);
      int used = 0;     // units with tiles
      uint32_t ts = 0;  // tiles so far
      uint32_t shared = 0;  // SHARE: units that mended so far
      bool kept = false;    // and whether the last unit is one
      // ring slots of tile t (counted from the first): its first operand, its second
      auto slot_a = [&](uint32_t t) { return (int)(t % NA); };
      auto slot_b = [&](uint32_t t) { return NA + (int)(t % NB); };
      auto wait_a = [&](uint32_t t) { wait(&S.full[slot_a(t)], (t / NA) & 1); };
      auto wait_b = [&](uint32_t t) { wait(&S.full[slot_b(t)], (t / NB) & 1); };
      // scores: resident tile (ad) times ring slot i, both K-major
      auto scores = [&](uint64_t ad, int i, uint32_t col, uint64_t* bar) {
        const uint64_t bd = sdesc_at(bk, i * TB);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_ss(tmem + col, sdesc_at(ad, (x & 3) * 32 + (x >> 2) * 16384),
                   sdesc_at(bd, (x & 3) * 32 + (x >> 2) * 16384), idS, x > 0);
          mma_commit(bar);
        }
        __syncwarp();
      };
      // accumulator (col) += weights (16-bit, 64 keys or rows at columns w and w + 64) times
      // ring slot i, which is let go when done
      auto weigh = [&](uint32_t w, int i, uint32_t col, bool fresh, bool done, uint64_t* more) {
        const uint64_t bd = sdesc_at(bm, i * TB);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mma_ts(tmem + col, tmem + w + (x & 3) * 8 + (x >> 2) * 64, sdesc_at(bd, x * 2048), idA,
                   !fresh || x > 0);
          if (done) mma_commit(&S.empty[i]);
          if (more) mma_commit(more);
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      for (int n = 0;; ++n) {
        wait(&S.sched_full[n % kSched], (n / kSched) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const BUnit& u = S.unit[n % kSched];
        if (!u.live) break;
        const int T = u.t1 - u.t0;
        if (T > 0) {
          const int rb = used % NR;
          const uint64_t a1 = sdesc_at(res0, rb * 2 * TB), a2 = sdesc_at(a1, TB);
          wait(&S.r_full[rb], (used / NR) & 1);
          ++used;
          const bool mend = MEND && u.mend;
          // S of tile ts + i of the unit's T; its buffer, P and dS columns
          const uint32_t tb = ts;
          auto buf = [&](uint32_t t) { return TWO_S ? (t - tb) & 1 : 0u; };
          auto next_s = [&](uint32_t t, uint32_t b) {
            wait_a(t);
            if (!TWO_S && t != ts) wait(&S.s_free, (t - 1) & 1);
            scores(a1, slot_a(t), b * 128, &S.s_full[b]);
          };
          auto next_dp = [&](uint32_t t) {
            scores(a2, slot_b(t), kDP, &S.dp_full);
            if (!DKV) commit(&S.empty[slot_b(t)]);
          };
          next_s(ts, 0);
          wait_b(ts);
          next_dp(ts);
          if (T == 1) commit(&S.r_empty[rb]);
          if (SHARE && kept) wait(&S.kb_read, (shared - 1) & 1);  // the second S's place is free again
          if (SHARE && mend) {
            ++shared;
            kept = true;
            for (int t = 0; t < T; ++t, ++ts) {
              const bool more = t + 1 < T;
              if (more) wait_b(ts + 1);
              wait(&S.ds_ready, ts & 1);
              if (more) next_dp(ts + 1);
              weigh(0, slot_a(ts), kKB, t == 0, false, nullptr);
              weigh(32, slot_a(ts), kDQ, t == 0, true, more ? nullptr : &S.acc_full);
              if (more) next_s(ts + 1, 0);
              if (t + 2 == T) commit(&S.r_empty[rb]);
            }
          } else {
            kept = false;
            if (TWO_S && T > 1) next_s(ts + 1, 1);
            for (int t = 0; t < T; ++t, ++ts) {
              const bool more = t + 1 < T;
              if (!TWO_S && more) next_s(ts + 1, 0);  // under this tile's exponentials
              if (more) wait_b(ts + 1);
              wait(&S.ds_ready, ts & 1);
              uint64_t* full = more ? nullptr : &S.acc_full;
              const uint32_t cp = TWO_S ? buf(ts) * 128 : kDP;
              if (TWO_S && more) next_dp(ts + 1);
              if constexpr (DKV) {
                weigh(cp, slot_b(ts), kDV, t == 0, true, nullptr);
                weigh(cp + 32, slot_a(ts), kDK, t == 0, true, full);
              } else {
                if (!SHARE && mend) weigh(cp, slot_a(ts), kKB, t == 0, false, nullptr);
                weigh(cp + 32, slot_a(ts), kDQ, t == 0, true, full);
              }
              if (!TWO_S && more) next_dp(ts + 1);
              if (t + 2 == T) commit(&S.r_empty[rb]);
              if (TWO_S && t + 2 < T) next_s(ts + 2, buf(ts));
            }
          }
        }
        if (lane == 0) mbar_arrive(&S.sched_empty[n % kSched]);
        __syncwarp();
      }
      if (!ok && lane == 0) fail();
      commit(&S.fin);
      if (!mbar_wait_drain(&S.fin, 0, limit) && lane == 0) fail();
      __syncwarp();
    }
  } else {
    regs_increase<kRegsCompute>();
    // ---------------- compute ----------------
    const int w = warp >> 2;  // columns 64 w .. 64 w + 63 of every tile
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;
    const float sc2 = a.scale * kLog2e;
    bool ok = true;
    uint32_t ts = 0, us = 0, rs = 0;  // tiles, units with tiles, mended units so far
    uint32_t sp = 0;                  // bit b: parity of S buffer b
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, bar_wait(bar, parity, limit, abort));
      return ok;
    };
    for (int n = 0;; ++n) {
      if (!wait(&S.sched_full[n % kSched], (n / kSched) & 1)) break;
      const BUnit& u = S.unit[n % kSched];
      if (!u.live) break;
      const Job& job = DKV ? a.job[u.job] : a.qjob[u.job];
      const int t0 = u.t0, t1 = u.t1;
      const bool mend = MEND && u.mend;
      // live columns of this thread's row, in the unit's tile numbering
      int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
      float nl = 0.f, nd = 0.f;  // query-major: -LSE log2(e), -D
      float r0 = 0.f, r1 = 0.f;  // mend: sums of dS
      if constexpr (DKV) {
        if (u.r0 + row < n_keys(u.q, job.seg[0].kview)) {
          live_queries(g, u.q, job.seg[0].rule, u.r0 + row, lo0, hi0);
          lo0 *= u.hs.n;
          hi0 *= u.hs.n;
        }
      } else {
        QRow qr;
        if (query_at(g, u.q, job.qview, u.hs, u.r0 + row, qr)) {
          live_keys(g, u.q, job.seg[0].rule, qr.pos, lo0, hi0);
          if (job.nseg > 1) live_keys(g, u.q, job.seg[1].rule, qr.pos, lo1, hi1);
          const size_t rr = (size_t)qr.t * g.H + qr.h;
          const float f = a.lse[rr];
          nl = f == -INFINITY ? 0.f : -f * kLog2e;
          nd = -a.delta[rr];
        }
        lo0 -= u.u0[0] * 128;
        hi0 -= u.u0[0] * 128;
        lo1 -= (u.u0[1] - u.cnt0) * 128;
        hi1 -= (u.u0[1] - u.cnt0) * 128;
      }
      const int tsplit = DKV ? t1 : u.cnt0;
      for (int t = t0; t < t1; ++t, ++ts) {
        const int buf = TWO_S && !(SHARE && mend) ? (t - t0) & 1 : 0;
        const uint32_t tS = tmem + tl + buf * 128 + w * 64, tDP = tmem + tl + kDP + w * 64;
        const uint32_t tP = TWO_S ? tS : tDP;  // where P and dS go
        if (!wait(&S.s_full[buf], (sp >> buf) & 1)) break;
        sp ^= 1u << buf;
        tc_fence_after();
        float p[64];
        tmem_ld32(tS, reinterpret_cast<uint32_t*>(p));
        tmem_ld32(tS + 32, reinterpret_cast<uint32_t*>(p) + 32);
        tmem_wait_ld();
        if (!TWO_S) {
          tc_fence_before();
          mbar_arrive(&S.s_free);
        }
        const int kl = (t >= tsplit ? lo1 : lo0) - t * 128 - w * 64;
        const int kh = (t >= tsplit ? hi1 : hi0) - t * 128 - w * 64;
        if (!__all_sync(0xffffffffu, kl <= 0 && kh >= 64)) mask_bits<2>(p, kl, kh);
        if constexpr (DKV) {
          if (!wait(&S.row_full[ts & 1], (ts >> 1) & 1)) break;
          const float4* L = reinterpret_cast<const float4*>(S.nlse[ts & 1] + w * 64);
#pragma unroll
          for (int x = 0; x < 64; x += 4) {
            const float4 f = L[x / 4];
            ffma2(p[x], p[x + 1], p[x], p[x + 1], sc2, sc2, f.x, f.y);
            ffma2(p[x + 2], p[x + 3], p[x + 2], p[x + 3], sc2, sc2, f.z, f.w);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 64; x += 2) ffma2(p[x], p[x + 1], p[x], p[x + 1], sc2, sc2, nl, nl);
        }
#pragma unroll
        for (int x = 0; x < 64; ++x) p[x] = fast_exp2(p[x]);
        uint32_t pk[32], pp[32];
        if (DKV || mend) {
#pragma unroll
          for (int x = 0; x < 32; ++x) pp[x] = pack2<F16>(p[2 * x], p[2 * x + 1]);
        }
        if (!wait(&S.dp_full, ts & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float dp[32];
          tmem_ld32(tDP + c * 32, reinterpret_cast<uint32_t*>(dp));
          tmem_wait_ld();
          if constexpr (DKV) {
            const float4* Dl = reinterpret_cast<const float4*>(S.ndel[ts & 1] + w * 64 + c * 32);
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 f = Dl[x / 4];
              float* y = p + c * 32 + x;
              fadd2(dp[x], dp[x + 1], dp[x], dp[x + 1], f.x, f.y);
              fadd2(dp[x + 2], dp[x + 3], dp[x + 2], dp[x + 3], f.z, f.w);
              fmul2(y[0], y[1], y[0], y[1], dp[x], dp[x + 1]);
              fmul2(y[2], y[3], y[2], y[3], dp[x + 2], dp[x + 3]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float* y = p + c * 32 + x;
              fadd2(dp[x], dp[x + 1], dp[x], dp[x + 1], nd, nd);
              fmul2(y[0], y[1], y[0], y[1], dp[x], dp[x + 1]);
            }
            if (mend) {
#pragma unroll
              for (int x = 0; x < 32; x += 2) fadd2(r0, r1, r0, r1, p[c * 32 + x], p[c * 32 + x + 1]);
            }
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[c * 16 + x] = pack2<F16>(p[c * 32 + 2 * x], p[c * 32 + 2 * x + 1]);
        }
        if constexpr (DKV) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.row_empty[ts & 1]);
        }
        if (DKV || mend) tmem_st32(tP, pp);
        tmem_st32(tP + 32, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&S.ds_ready);
      }
      if (!ok) break;
      // ---- the unit's rows ----
      if constexpr (!DKV) {
        QRow qr;
        const bool have = query_at(g, u.q, job.qview, u.hs, u.r0 + row, qr);
        if (!have) qr = QRow{0, 0, 0};
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.sched_empty[n % kSched]);
        if (t1 > t0) {
          if (!wait(&S.acc_full, us & 1)) break;
          ++us;
          tc_fence_after();
        }
        const size_t rr = have ? (size_t)qr.t * g.H + qr.h : 0;
        uint16_t* out = static_cast<uint16_t*>(a.dq) + ((size_t)qr.t * a.dq_rows.tok + qr.h * a.dq_rows.head) * D;
        const bool wide = (reinterpret_cast<uintptr_t>(a.dq) & 31) == 0;
        auto load = [&](float* o, uint32_t col) {
          __syncwarp();  // rows past the unit's end left the last turn early
          if (t1 > t0) {
            tmem_ld32(tmem + tl + col, reinterpret_cast<uint32_t*>(o));
            tmem_wait_ld();
          }
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = t1 > t0 ? o[x] * a.scale : 0.f;
        };
        if (mend) {
          float r = 0.f;  // what D lost: both warpgroups' columns, both orders
          if (t1 > t0) {
            S.ndel[w][row] = r0 + r1;
            mbar_arrive(&S.r_sum);
            if (!wait(&S.r_sum, rs & 1)) break;
            ++rs;
            r = S.ndel[0][row] + S.ndel[1][row];
          }
          if (have && a.mode == OUT_MERGE) r += a.r_part[rr];
          // the first of two orders: either every unit leaves its sums to the second, or
          // units of rows that only this order reaches mend by themselves
          const bool leave = a.mode == OUT_PARTIAL && a.mend_tiles > 2;
          if (have && w == 0) {
            if (leave) a.r_part[rr] = r;
            else a.delta[rr] = r - nd;  // for the key-major kernel; this unit has read its rows
          }
#pragma unroll 1
          for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += 32) {
            float o[32], kb[32];
            load(o, kDQ + c);
            load(kb, kKB + c);
            if (!have) continue;
            const size_t at = rr * D + c;
            if (leave) {
              store_row32(a.dq_part + at, o);
              store_row32(a.kb_part + at, kb);
              continue;
            }
            if (a.mode == OUT_MERGE) {
              add_row32(o, a.dq_part + at);
              add_row32(kb, a.kb_part + at);
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = fmaf(-r, kb[x], o[x]);
            if (a.mode == OUT_PARTIAL) store_row32(a.dq_part + at, o);
            else store_row16<F16>(out + c, o, wide);
          }
          if (SHARE && t1 > t0) {
            tc_fence_before();
            mbar_arrive(&S.kb_read);
          }
        } else {
#pragma unroll 1
          for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += 32) {
            float o[32];
            load(o, kDQ + c);
            if (!have) continue;
            if (a.mode == OUT_PARTIAL) {
              store_row32(a.dq_part + rr * D + c, o);
              continue;
            }
            if (a.mode == OUT_MERGE) add_row32(o, a.dq_part + rr * D + c);
            store_row16<F16>(out + c, o, wide);
          }
        }
        tc_fence_before();
      } else {
        const int view = job.seg[0].kview, kvh = u.kvh;
        const bool have = u.r0 + row < n_keys(u.q, view);
        const int pos = have ? key_pos(g, u.q, view, u.r0 + row) : 0, tok = u.q.qb + pos;
        const bool direct = dkv_direct(a, kvh);
        const bool add = a.mode == OUT_MERGE && view_lists(g, a.part_view, pos);
        float* part = a.parts + (((size_t)(u.job * a.nsplit + u.split) * g.total + tok) * g.Hkv + kvh) * 2 * D + w * D;
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.sched_empty[n % kSched]);
        if (t1 > t0) {
          if (!wait(&S.acc_full, us & 1)) break;
          ++us;
          tc_fence_after();
        }
        // warpgroup 0 writes dK, warpgroup 1 dV
        uint16_t* out = w ? static_cast<uint16_t*>(a.dv) + ((size_t)tok * a.dv_rows.tok + kvh * a.dv_rows.head) * D
                          : static_cast<uint16_t*>(a.dk) + ((size_t)tok * a.dk_rows.tok + kvh * a.dk_rows.head) * D;
        const float f = w ? 1.f : a.scale;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          __syncwarp();  // keys past the unit's end left the last turn early
          if (t1 > t0) {
            tmem_ld32(tmem + tl + (w ? kDV : kDK) + c, reinterpret_cast<uint32_t*>(o));
            tmem_wait_ld();
          }
          if (!have) continue;
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = t1 > t0 ? o[x] * f : 0.f;
          if (add) add_row32(o, part + c);
          if (direct) store_row16<F16>(out + c, o, (reinterpret_cast<uintptr_t>(w ? a.dv : a.dk) & 31) == 0);
          else store_row32(part + c, o);
        }
        tc_fence_before();
      }
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, bool F16, bool DKV, bool MEND, bool ALL>
cudaError_t launch(const BwdLaunch& a) {
  const Geo& g = a.g;
  TileMaps m = {};
  const Rows whole = {g.H, 1, 0};
  if (!make_query_map(&m.q, m, g, g.q, a.q, F16) || !make_query_map(&m.dout, m, g, whole, a.dout, F16) ||
      !make_key_maps(m, g, a.k, a.v, F16))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<D>);
  static_assert(sizeof(Smem<D>) <= 232448, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(ragged_bwd_tc<D, F16, DKV, MEND, ALL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(g, DKV ? 1 : most_heads(g, a.qjob[0].hc), 128);
  const long long units = slots * g.Hkv * (DKV ? a.njobs * a.nsplit : a.nqjobs);
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  ragged_bwd_tc<D, F16, DKV, MEND, ALL><<<(unsigned)units, kThreads, smem, a.stream>>>(a, m, (int)slots);
  return cudaGetLastError();
}

}  // namespace

cudaError_t tc_ragged_dq(const BwdLaunch& a, int dtype) {
  const bool h = dtype == ST_F16;
  if (a.g.d == 64) return h ? launch<64, true, false, true, false>(a) : launch<64, false, false, true, false>(a);
  if (a.mend_tiles > 2) return h ? launch<128, true, false, true, true>(a) : launch<128, false, false, true, true>(a);
  return h ? launch<128, true, false, true, false>(a) : launch<128, false, false, true, false>(a);
}
cudaError_t tc_ragged_dkv(const BwdLaunch& a, int dtype) {
  const bool h = dtype == ST_F16;
  if (a.g.d == 64) return h ? launch<64, true, true, false, false>(a) : launch<64, false, true, false, false>(a);
  return h ? launch<128, true, true, false, false>(a) : launch<128, false, true, false, false>(a);
}

}  // namespace rag
}  // namespace st

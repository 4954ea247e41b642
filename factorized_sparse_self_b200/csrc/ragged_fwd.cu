// Forward of attention over ragged and paged sequences on the tensor cores
// (bf16, fp16; d = 64, 128).
//
// One CTA per SM (384 threads) that goes on with the units of CTAs that have not
// started (cluster launch control). A unit is 256 query rows of one
// (sequence, key/value head): two halves of 128 rows that share every K and V
// tile, so a tile brought from L2 serves 256 rows and the two halves' softmax and
// products alternate. Warp roles:
//   warp 10      scheduler: decodes the CTA's units into a small ring;
//   warps 8, 11  producers: Q rows, then K and V tiles of 128 rows in turn into
//                one ring. Rows are gathered through the order's index map and the
//                page table, or come as TMA boxes where they lie evenly. Rows behind the last key repeat it: masked entries have
//                weight 0 and must not meet another sequence's infinities;
//   warp 9       MMA issuer: S_h = Q_h K^T (128 x 128 fp32 in TMEM), O_h += P_h V
//                with P_h read from TMEM; the order S0 S1 | P0V S0' | P1V S1' | ..
//                keeps one half's products under the other half's softmax;
//   warps 0..7   softmax of half 0 and 1: thread = query row = TMEM lane, running
//                maximum (O is rescaled in TMEM only when it grows by more than 2^8)
//                and sum in fp32, P as 16-bit pairs over S.
// The softmax holds a row's 128 scores in 208 registers; 256 bytes of its other state
// are spilled at d = 128, 208 at d = 64.
// TMEM: S0 S1 (P0 P1 in their first 64 columns) O0 O1, 128 columns each.
#include "ragged_tc.cuh"

namespace st {
namespace rag {
namespace {

constexpr int kThreads = 384;
constexpr int kRows = 256;  // query rows of a unit
constexpr int kSched = 2;   // ring of decoded units
constexpr int kAhead = 3;   // tiles before a unit's end at which the next is claimed
constexpr uint32_t kRegsSoftmax = 208, kRegsIssue = 88;  // 168 at launch: 2 * 208 + 88 = 3 * 168
constexpr float kRescale = 8.f;  // log2
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = D == 64 ? 8 : 5;
  static constexpr int kQ = D == 64 ? 2 : 1;  // Q buffers (d = 128 has no room for a second)
};

template <int D>
struct alignas(1024) Smem {
  uint8_t q[Cfg<D>::kQ][2][Cfg<D>::kTileBytes];
  uint8_t kv[Cfg<D>::kStages][Cfg<D>::kTileBytes];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[Cfg<D>::kStages], kv_empty[Cfg<D>::kStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t sched_full[kSched], sched_empty[kSched];
  uint64_t fin;
  alignas(16) uint4 claim;
  uint64_t claim_bar, want;
  Unit unit[kSched];
  uint32_t tmem;
  int abort;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_fwd_tc(const __grid_constant__ FwdLaunch a, const __grid_constant__ TileMaps maps, int slots) {
  extern __shared__ uint8_t raw[];
  Smem<D>& S = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  constexpr int NS = Cfg<D>::kStages, TB = Cfg<D>::kTileBytes, QB = Cfg<D>::kQ;
  constexpr uint32_t kColO = 256;
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = a.wait_ns;
  volatile int* abort = &S.abort;
  if (threadIdx.x == 0) {
    S.abort = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.kv_full[i], 2);
      mbar_init(&S.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.q_full[i], 2);  // both producers
      mbar_init(&S.q_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 128);
      mbar_init(&S.o_full[i], 1);
    }
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&S.sched_full[i], 1);
      mbar_init(&S.sched_empty[i], 11);  // two producers, MMA, eight softmax warps
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
        const bool some = decode_unit(a, slots, n, kRows, &S.unit[k % kSched]);
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
      const int pw = warp == 8 ? 0 : 1;  // loads half pw of the Q rows, rows 64 pw .. of K and V tiles
      if (pw == 0 && lane == 0 && maps.nat_rows) {
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.v);
      }
      int used = 0, kt = 0;  // units with tiles, ring slots filled
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
        const Unit& u = S.unit[n % kSched];
        if (u.t1 > u.t0) {
          const Job& job = u.job ? a.job1 : a.job;
          const int qb = used % QB;
          if (used >= QB && !wait(&S.q_empty[qb], (used / QB + 1) & 1)) break;
          ++used;
          const int rows = u.q.nq * u.hs.n, x0 = u.x0 + pw * 128;
          if (maps.q_tokens && job.qview == VIEW_NAT && x0 + 128 <= rows) {
            load_query_boxes<D>(smem_u32(S.q[qb][pw]), &maps.q, &S.q_full[qb], maps, u.q, u.hs, x0);
          } else {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              int r[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                QRow qr;
                query_at(g, u.q, job.qview, u.hs, imin(x0 + i * 64 + y * 32 + lane, rows - 1), qr);
                r[y] = q_row(g, qr.t, qr.h);
              }
              gather64<D>(smem_u32(S.q[qb][pw]), i * 64, a.q, r[0], r[1]);
            }
            gath.add(&S.q_full[qb]);
          }
          for (int t = u.t0; t < u.t1 && ok; ++t) {
            if (pw == 0 && lane == 0 && t == imax(u.t0, u.t1 - kAhead)) mbar_arrive(&S.want);
            int seg, j;
            unit_tile(u, t, seg, j);
            const int view = job.seg[seg].kview, R = box_rows(maps, g, u.q, view, j);
            int rk[2], rv[2];
            if (!R) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int e = imin(j * 128 + pw * 64 + y * 32 + lane, n_keys(u.q, view) - 1);
                kv_rows(g, u.q, key_pos(g, u.q, view, e), u.kvh, rk[y], rv[y]);
              }
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++kt) {
              const int s = kt % NS;
              if (a.force_timeout && kt == 0) continue;  // test hook: this stage never fills
              if (kt >= NS && !wait(&S.kv_empty[s], (kt / NS + 1) & 1)) break;
              if (!R) {
                gather64<D>(smem_u32(S.kv[s]), pw * 64, kv ? a.v : a.k, kv ? rv[0] : rk[0], kv ? rv[1] : rk[1]);
                gath.add(&S.kv_full[s]);
              } else {
                gath.flush();
                if (pw == 0) load_boxes<D>(smem_u32(S.kv[s]), maps, kv, &S.kv_full[s], g, u.q, view, j, u.kvh, R);
                else if (lane == 0) mbar_arrive(&S.kv_full[s]);
              }
            }
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
      // without waiting for them)
      for (int i = imax(0, used - QB); i < used; ++i) mbar_wait_drain(&S.q_full[i % QB], (i / QB) & 1, limit);
      for (int i = imax(0, kt - NS); i < kt; ++i) mbar_wait_drain(&S.kv_full[i % NS], (i / NS) & 1, limit);
    } else if (warp == 9) {
      // ---------------- MMA issuer ----------------
      const uint32_t idS = idesc_16(128, 128, false, false, F16);
      const uint32_t idPV = idesc_16(128, D, false, true, F16);
      int kt = 0, used = 0;  // ring slots consumed, units with tiles
      int np[2] = {0, 0};    // tiles of each half so far
      // A lane's failed wait is remembered and agreed on at the end of the unit:
      // until then the warp goes on (later waits of that lane return at once).
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = bar_wait(bar, parity, limit, abort);
        __syncwarp();
      };
      const uint64_t qd0 = sdesc(smem_u32(S.q[0][0]), 16, 1024);
      const uint64_t kd0 = sdesc(smem_u32(S.kv[0]), 16, 1024);
      const uint64_t vd0 = sdesc(smem_u32(S.kv[0]), 16384, 1024);
      auto issue_s = [&](int h, int stage, int qb) {
        const uint64_t qd = sdesc_at(qd0, (2 * qb + h) * TB), kd = sdesc_at(kd0, stage * TB);
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_ss(tmem + h * 128, sdesc_at(qd, (x & 3) * 32 + (x >> 2) * 16384),
                   sdesc_at(kd, (x & 3) * 32 + (x >> 2) * 16384), idS, x > 0);
          mma_commit(&S.s_full[h]);
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
        const Unit& u = S.unit[n % kSched];
        if (!u.live) break;
        const int t0 = u.t0, t1 = u.t1, cnt0 = u.cnt0, first0 = u.u0[0], first1 = u.u0[1] - cnt0;
        if (t1 > t0) {
          // the tiles of a half, as numbers t, segment by segment, and its last
          int a0[2], b0[2], a1[2], b1[2], last[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a0[h] = u.ja[h][0] - first0;
            b0[h] = u.jb[h][0] - first0;
            a1[h] = imax(u.ja[h][1] - first1, cnt0);
            b1[h] = u.jb[h][1] - first1;
            last[h] = imin(b1[h], t1) > imax(a1[h], t0) ? imin(b1[h], t1) - 1 : imin(imin(b0[h], cnt0), t1) - 1;
          }
          auto meets = [&](int h, int t) {
            return t < t1 && (t < cnt0 ? t >= a0[h] && t < b0[h] : t >= a1[h] && t < b1[h]);
          };
          const int qb = used % QB;
          wait(&S.q_full[qb], (used / QB) & 1);
          ++used;
          bool fresh[2] = {true, true};
          bool act[2] = {meets(0, t0), meets(1, t0)};
          wait(&S.kv_full[kt % NS], (kt / NS) & 1);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (act[h]) issue_s(h, kt % NS, qb);
          commit(&S.kv_empty[kt % NS]);
          if (t0 + 1 == t1) commit(&S.q_empty[qb]);
          int sv = (kt + 1) % NS, pv = ((kt + 1) / NS) & 1;
          for (int t = t0; t < t1; ++t, kt += 2) {
            int sk = sv + 1, pk = pv;
            if (sk == NS) {
              sk = 0;
              pk ^= 1;
            }
            const bool more = t + 1 < t1;
            const bool nact[2] = {meets(0, t + 1), meets(1, t + 1)};
            const uint64_t vd = sdesc_at(vd0, sv * TB);
            wait(&S.kv_full[sv], pv);
            if (more) wait(&S.kv_full[sk], pk);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (act[h]) {
                wait(&S.p_full[h], np[h] & 1);
                ++np[h];
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                  for (int x = 0; x < 8; ++x)
                    mma_ts(tmem + kColO + h * D, tmem + h * 128 + x * 8, sdesc_at(vd, x * 2048), idPV,
                           !fresh[h] || x > 0);
                  // the next S of this half is issued behind this product, so
                  // only the unit's last one needs a signal of its own
                  if (t == last[h]) mma_commit(&S.o_full[h]);
                }
                __syncwarp();
                fresh[h] = false;
              }
              if (nact[h]) issue_s(h, sk, qb);
            }
            commit(&S.kv_empty[sv]);
            if (more) {
              commit(&S.kv_empty[sk]);
              if (t + 2 == t1) commit(&S.q_empty[qb]);
            }
            act[0] = nact[0];
            act[1] = nact[1];
            sv = sk + 1;
            pv = pk;
            if (sv == NS) {
              sv = 0;
              pv ^= 1;
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
    regs_increase<kRegsSoftmax>();
    // ---------------- softmax ----------------
    const int h = warp >> 2;
    const uint32_t tl = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + tl + h * 128, tO = tmem + tl + kColO + h * D;
    const int row = (warp & 3) * 32 + lane;
    const bool wide = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;
    bool ok = true;
    int ns = 0, no = 0;  // tiles of this half so far, units with tiles
    for (int n = 0;; ++n) {
      ok = __all_sync(0xffffffffu, bar_wait(&S.sched_full[n % kSched], (n / kSched) & 1, limit, abort));
      if (!ok) break;
      const Unit& su = S.unit[n % kSched];
      if (!su.live) break;
      const Job& job = su.job ? a.job1 : a.job;
      int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;
      {
        QRow qr;
        if (query_at(g, su.q, job.qview, su.hs, su.x0 + h * 128 + row, qr) && qr.pos >= 0) {
          live_keys(g, su.q, job.seg[0].rule, qr.pos, lo0, hi0);
          if (job.nseg > 1) live_keys(g, su.q, job.seg[1].rule, qr.pos, lo1, hi1);
        }
      }
      const int t1 = su.t1;
      float m = -INFINITY, l = 0.f;
      bool any = false;
      for (int t = su.t0; t < t1; ++t) {
        int seg, j;
        unit_tile(su, t, seg, j);
        if (!half_meets(su, h, seg, j)) continue;
        ok = __all_sync(0xffffffffu, bar_wait(&S.s_full[h], ns & 1, limit, abort));
        if (!ok) break;
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, reinterpret_cast<uint32_t*>(s) + c * 32);
        tmem_wait_ld();
        const int kl = (seg ? lo1 : lo0) - j * 128, kh = (seg ? hi1 : hi0) - j * 128;
        if (!__all_sync(0xffffffffu, kl <= 0 && kh >= 128)) mask_bits<4>(s, kl, kh);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 128; x += 8) {
          m4[0] = fmax3(m4[0], s[x + 0], s[x + 1]);
          m4[1] = fmax3(m4[1], s[x + 2], s[x + 3]);
          m4[2] = fmax3(m4[2], s[x + 4], s[x + 5]);
          m4[3] = fmax3(m4[3], s[x + 6], s[x + 7]);
        }
        const float mt = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * a.scale_log2;
        float alpha = 1.f;
        bool rescale = false;
        if (mt > m + kRescale) {
          rescale = m != -INFINITY;
          alpha = fast_exp2(m - mt);
          m = mt;
        }
        const float nmu = m == -INFINITY ? 0.f : -m;
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            float a0, a1;
            ffma2(a0, a1, s[c * 64 + x], s[c * 64 + x + 1], a.scale_log2, a.scale_log2, nmu, nmu);
            const float p0 = fast_exp2(a0), p1 = fast_exp2(a1);
            const int y = (x >> 1) & 3;
            fadd2(sa[y], sb[y], sa[y], sb[y], p0, p1);
            pk[x >> 1] = pack2<F16>(p0, p1);
          }
          tmem_st32(tS + c * 32, pk);
        }
        l = l * alpha + (((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3])));
        if (__any_sync(0xffffffffu, rescale)) {
          // the previous tile's P V was issued before this tile's S, so it has ended
          const float f = rescale ? alpha : 1.f;
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {
            uint32_t o[8];
            tmem_ld8(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            tmem_st8(tO + c, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&S.p_full[h]);
        any = true;
        ++ns;
      }
      if (!ok) break;
      // ---- the unit's rows ----
      // (the row is worked out again: kept over the tiles it would cost them registers)
      QRow qr;
      const bool have = query_at(g, su.q, job.qview, su.hs, su.x0 + h * 128 + row, qr);
      const int part = su.part, parts = su.parts, part0 = su.job ? a.part1 : a.part0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.sched_empty[n % kSched]);
      if (any) {
        ok = __all_sync(0xffffffffu, bar_wait(&S.o_full[h], no & 1, limit, abort));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      // (a sum that is not a number is kept, here and where parts are joined: the row
      // must not pass for an empty one)
      float L = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
      float wc = l != 0.f ? 1.f / l : 0.f, wp = 0.f;
      const size_t rr = have ? (size_t)qr.t * g.H + qr.h : 0;
      if (a.mode == OUT_MERGE && have) {
        const float lp = a.parts.lse[rr], mx = fmaxf(lp, L);
        if (lp != -INFINITY || L != -INFINITY) {
          const float out = mx + __logf(__expf(lp - mx) + __expf(L - mx));
          wp = __expf(lp - out);
          wc *= __expf(L - out);
          L = out;
        }
      }
      if (have) {
        if (a.mode == OUT_PARTIAL) {
          a.parts.lse[(size_t)(part0 + part) * g.total * g.H + rr] = L;
          if (part == 0)
            for (int p = parts; p < a.nsplit; ++p)
              a.parts.lse[(size_t)(part0 + p) * g.total * g.H + rr] = -INFINITY;
        } else {
          a.lse[rr] = L;
        }
      }
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        __syncwarp();  // rows past the unit's end left the last turn early
        if (any) {
          tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
        }
        if (!have) continue;
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = any ? o[x] * wc : 0.f;
        if (a.mode == OUT_PARTIAL) {
          if (wc != 0.f) {  // a part without weight is not read
            store_row32(a.parts.o + ((size_t)(part0 + part) * g.total * g.H + rr) * D + c, o);
          }
          continue;
        }
        if (a.mode == OUT_MERGE && wp != 0.f) {
          const float4* src = reinterpret_cast<const float4*>(a.parts.o + rr * D + c);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float4 f = src[x];
            o[4 * x] = fmaf(wp, f.x, o[4 * x]);
            o[4 * x + 1] = fmaf(wp, f.y, o[4 * x + 1]);
            o[4 * x + 2] = fmaf(wp, f.z, o[4 * x + 2]);
            o[4 * x + 3] = fmaf(wp, f.w, o[4 * x + 3]);
          }
        }
        store_row16<F16>(static_cast<uint16_t*>(a.o) + rr * D + c, o, wide);
      }
      tc_fence_before();
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, bool F16>
cudaError_t launch(const FwdLaunch& a) {
  const Geo& g = a.g;
  TileMaps m = {};
  if (!make_key_maps(m, g, a.k, a.v, F16) || !make_query_map(&m.q, m, g, g.q, a.q, F16))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(sizeof(Smem<D>) + 1024 <= 232448, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(ragged_fwd_tc<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(g, most_heads(g, a.job.hc), kRows);
  const long long units = slots * g.Hkv * a.njobs * a.nsplit;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  ragged_fwd_tc<D, F16><<<(unsigned)units, kThreads, smem, a.stream>>>(a, m, (int)slots);
  return cudaGetLastError();
}

}  // namespace

cudaError_t tc_ragged_fwd(const FwdLaunch& a, int dtype) {
  if (a.g.d == 64) return dtype == ST_F16 ? launch<64, true>(a) : launch<64, false>(a);
  return dtype == ST_F16 ? launch<128, true>(a) : launch<128, false>(a);
}

}  // namespace rag
}  // namespace st

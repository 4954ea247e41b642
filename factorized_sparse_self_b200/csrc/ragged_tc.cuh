// What the tensor-core kernels for ragged sequences share: the loads of operand
// tiles, and the units that a scheduler warp decodes for the other warps of its
// CTA.
#pragma once

#include "ragged.h"
#include "tc_common.cuh"

namespace st {
namespace rag {

using namespace st::tc;

constexpr int kNeed = 128;  // rows of an operand tile

// One lane of the (converged) warp, the same one every time. The MMA warps run
// their control flow with all lanes and pick the issuing lane around the
// tcgen05 instructions only: descriptors then stay in uniform registers. With
// the whole role inside `if (lane == 0)` each MMA took 80 to 130 cycles to
// issue (d = 64's P V needs 32 on the pipe).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Whether a phase is complete, at once (try_wait may hold the thread for
// microseconds first).
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for a phase; gives up after limit_ns or when another role raised
// `abort`. The clock and the flag are looked at after every 64 attempts only:
// read in every attempt, they delay the waking thread.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                         volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 63) == 0) {
      if (*abort) return false;
      const uint64_t now = globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit_ns) return false;
    }
  }
}

// Sets v[x] = -inf for the columns x (< 32 * N) outside [lo, hi). The live columns
// of 32 form a word whose bits become predicates several at a time; chunks that
// every row of the warp keeps are left alone.
template <int N>
__device__ __forceinline__ void mask_bits(float* v, int lo, int hi) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const int a = imin(imax(lo - c * 32, 0), 32), b = imin(imax(hi - c * 32, 0), 32);
    const uint32_t bits = (uint32_t)((1ull << b) - 1) & ~(uint32_t)((1ull << a) - 1);
    if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
      for (int x = 0; x < 32; ++x) v[c * 32 + x] = (bits & (1u << x)) ? v[c * 32 + x] : -INFINITY;
    }
  }
}

// Stores 32 values of a row in 16 bits, 32 bytes at a time where the row allows it.
template <bool F16>
__device__ __forceinline__ void store_row16(void* dst, const float* o, bool wide) {
  uint32_t w[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) w[x] = pack2<F16>(o[2 * x], o[2 * x + 1]);
  uint4* p = static_cast<uint4*>(dst);
  if (wide) {
    st_global_v8(p, w);
    st_global_v8(p + 2, w + 8);
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
  }
}
// 32 fp32 values (parts of a workspace, whose rows lie on 32-byte boundaries).
__device__ __forceinline__ void store_row32(float* dst, const float* o) {
#pragma unroll
  for (int x = 0; x < 4; ++x) st_global_v8(dst + 8 * x, reinterpret_cast<const uint32_t*>(o) + 8 * x);
}
// o += 32 fp32 values of such a part.
__device__ __forceinline__ void add_row32(float* o, const float* part) {
#pragma unroll
  for (int x = 0; x < 32; x += 4) {
    const float4 f = *reinterpret_cast<const float4*>(part + x);
    o[x] += f.x;
    o[x + 1] += f.y;
    o[x + 2] += f.z;
    o[x + 3] += f.w;
  }
}

// ---- rows gathered into an operand tile -----------------------------------------
// A tile is 128 rows of D 16-bit elements as D / 64 blocks of [128][64] with the
// 128-byte swizzle, 16 KB each. A warp copies 64 of its rows, 16 bytes a lane
// (asynchronously, past L1): lane i knows the row numbers of rows i and 32 + i.
// (The TMA's row gather moves 4 rows of 128 bytes in about 100 cycles, whatever
// issues it: with it chunks of 512 tokens behind up to 32 K keys took 1195 us, with these copies 666.)
template <int D>
__device__ __forceinline__ void gather64(uint32_t dst, int row0, const void* base, int ra, int rb) {
  constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows per instruction
  const int lane = threadIdx.x & 31;
  const int chunk = lane % CH, sub = lane / CH;
  const uint32_t col = dst + (chunk >> 3) * 16384;
#pragma unroll 1
  for (int i0 = 0; i0 < 64 / RPI; i0 += 8) {
    int r[8];  // eight lookups, then eight copies: one by one each waits for its shuffle
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r[i] = __shfl_sync(0xffffffffu, (i0 + i) * RPI < 32 ? ra : rb, ((i0 + i) * RPI + sub) & 31);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int y = row0 + (i0 + i) * RPI + sub;
      const char* src = static_cast<const char*>(base) + (size_t)r[i] * (D * 2) + chunk * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(col + y * 128 +
                                                                    (((chunk & 7) ^ (y & 7)) << 4)),
                   "l"(src)
                   : "memory");
    }
  }
}
__device__ __forceinline__ void gather_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void gather_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A warp's gathers that are under way, oldest first: the barrier of each gets one
// arrival once its copies have landed and are visible to the tensor cores.
struct Gathers {
  uint64_t* bar[3];
  int n = 0;
  __device__ __forceinline__ void arrive_oldest() {
    fence_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar[0]);
    bar[0] = bar[1];
    bar[1] = bar[2];
    --n;
  }
  __device__ __forceinline__ void add(uint64_t* b) {
    gather_commit();
    if (n == 0) bar[0] = b;
    else if (n == 1) bar[1] = b;
    else bar[2] = b;
    if (++n == 3) {
      gather_wait<2>();
      arrive_oldest();
    }
  }
  __device__ __forceinline__ void flush() {
    if (n == 0) return;
    gather_wait<0>();
    while (n) arrive_oldest();
  }
};

// ---- boxes ---------------------------------------------------------------------
// Rows that lie evenly in memory come as TMA boxes of 64 columns: 128 / R boxes of
// R rows (a multiple of 8, so each starts on a swizzle boundary).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c,
                                        int head, int row, int outer) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(head), "r"(row),
      "r"(outer)
      : "memory");
}

// Maps of one launch. Keys and values: boxes of nat_rows consecutive positions
// (packed: 128 tokens; paged: within a page) and of the sum_rows = c summary
// positions of a block (packed only); 0: none. Query-side tensors: boxes of the G
// heads of q_tokens = 128 / G tokens.
struct TileMaps {
  CUtensorMap k, v, ksum, vsum, q, dout;
  int32_t nat_rows, sum_rows, q_tokens;
};

// Whether key tile j of an order is made of whole boxes, and their rows.
__device__ __forceinline__ int box_rows(const TileMaps& m, const Geo& g, const Seq& q, int view, int j) {
  if (view == VIEW_NAT) return (j + 1) * 128 <= q.nk ? m.nat_rows : 0;
  if (view == VIEW_SUM) return (j + 1) * 128 <= q.P * g.c ? m.sum_rows : 0;
  return 0;
}
// Loads the tile (one warp; R = box_rows(...) > 0); the barrier gets one arrival.
template <int D>
__device__ __forceinline__ void load_boxes(uint32_t dst, const TileMaps& m, bool value, uint64_t* bar,
                                           const Geo& g, const Seq& q, int view, int j, int kvh, int R) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_arrive_expect_tx(bar, 128 * D * 2);
  __syncwarp();
  if (lane * R < 128) {
    int row, outer = 0;
    const CUtensorMap* map = value ? &m.v : &m.k;
    if (view == VIEW_SUM) {
      map = value ? &m.vsum : &m.ksum;
      row = q.qb + (fdiv(j * 128, g.fc) + lane + 1) * g.l - g.c;
    } else if (!g.kv_lens) {
      row = q.qb + j * 128;
    } else {
      const int pos = j * 128 + lane * R, pg = fdiv(pos, g.fpage);
      row = pos - pg * g.page_size;
      outer = page_of(g, q, pg);
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_box(dst + c * 16384 + lane * R * 128, map, bar, c * 64, kvh, row, outer);
  }
  __syncwarp();
}
// 128 rows (query, head of the group) from row x0 of a query-side tensor.
template <int D>
__device__ __forceinline__ void load_query_boxes(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                                 const TileMaps& m, const Seq& q, const Heads3& hs, int x0) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    mbar_arrive_expect_tx(bar, 128 * D * 2);
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_box(dst + c * 16384, map, bar, c * 64, hs.first, q.qb + x0 / 128 * m.q_tokens, 0);
  }
  __syncwarp();
}

// ---- work claimed from the grid ------------------------------------------------
// A kernel is launched with one CTA per unit; a running CTA takes over units
// whose CTAs have not started yet (cluster launch control), so units go to
// whichever SM is free, in order, without a counter in memory.

// Asks for the next CTA of the grid; the 16-byte answer lands in `dst`.
__device__ __forceinline__ void claim_next(void* dst, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(dst)),
      "r"(smem_u32(bar))
      : "memory");
}
// The claimed CTA's index, or -1 if none was left.
__device__ __forceinline__ int claimed(const void* src) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(src))
      : "memory");
  return ok ? (int)x : -1;
}

// One scheduler warp's claims. The next unit is claimed when the producers come to
// the last tiles of the current one (`want`, one arrival a unit), not before: a CTA
// that claims while its long unit runs keeps short ones from idle SMs (dense, 4096
// tokens, 256 key-major units on 148 SMs: SMs busy 69 % of the time with two units
// claimed ahead).
struct Claims {
  uint4* slot;    // shared memory
  uint64_t* bar;
  uint64_t* want;
  int n, units;   // claims made, units handed on
  int read;       // answers read
  bool left;      // false once the grid was used up (it may not be asked again)
};
__device__ __forceinline__ void claims_ask(Claims& c) {
  if ((threadIdx.x & 31) == 0) {
    fence_async_smem();  // the answer before this one was read
    mbar_arrive_expect_tx(c.bar, 16);
    claim_next(c.slot, c.bar);
  }
  ++c.n;
}
__device__ __forceinline__ int claims_answer(Claims& c) {
  const int got = claimed(c.slot);
  __syncwarp();
  ++c.read;
  c.left = got >= 0;
  return got;
}
// Next unit index (by a whole warp): -1 when the grid is used up, -2 when a wait
// ran out.
__device__ __forceinline__ int claims_take(Claims& c, bool handed_on, uint64_t limit, volatile int* abort) {
  if (handed_on) {
    const int u = c.units++;
    if (!__all_sync(0xffffffffu, bar_wait(c.want, u & 1, limit, abort))) return -2;
  }
  claims_ask(c);
  if (!__all_sync(0xffffffffu, bar_wait(c.bar, (c.n - 1) & 1, limit, abort))) return -2;
  return claims_answer(c);
}
// After a wait that ran out: a claim in flight lands before the CTA may exit, and
// the units that have not started are claimed and dropped, for in a launch that has
// failed each of their CTAs would wait as long again.
__device__ __forceinline__ void claims_drop(Claims& c, uint64_t limit) {
  while (c.left) {
    if (c.read == c.n) claims_ask(c);
    if (!__all_sync(0xffffffffu, mbar_wait_drain(c.bar, (c.n - 1) & 1, limit))) return;
    claims_answer(c);
  }
}

// Host: the boxes of a launch. False when the driver refuses one.
bool make_key_maps(TileMaps& m, const Geo& g, const void* k, const void* v, bool f16);
bool make_query_map(CUtensorMap* out, TileMaps& m, const Geo& g, const Rows& rows, const void* base, bool f16);

// One query-major unit: 2 x 128 rows of one (sequence, key/value head, job),
// against the key tiles it meets. Key tiles are numbered through the job's
// segments: t < cnt0 is tile u0[0] + t of segment 0, later ones of segment 1.
struct Unit {
  int32_t live;  // 0: no more units
  Seq q;
  Heads3 hs;
  int32_t kvh, job, x0, part, parts;  // parts: how many its keys are cut into
  int32_t t0, t1;          // key tiles of this unit
  int32_t cnt0;            // of segment 0
  int32_t u0[2];           // first tile of each segment
  int32_t ja[2][2], jb[2][2];  // [128-row half][segment]: tiles it meets
};

__device__ __forceinline__ void unit_tile(const Unit& u, int t, int& seg, int& j) {
  seg = t >= u.cnt0 ? 1 : 0;
  j = u.u0[seg] + t - (seg ? u.cnt0 : 0);
}
__device__ __forceinline__ bool half_meets(const Unit& u, int w, int seg, int j) {
  return j >= u.ja[w][seg] && j < u.jb[w][seg];
}

// Decodes unit number n into *out (by a whole warp); false if it has no rows.
// Slots are taken from the last to the first: a sequence's last tiles have the
// most keys.
__device__ __forceinline__ bool decode_unit(const FwdLaunch& a, int slots, int n, int rows, Unit* out) {
  const Geo& g = a.g;
  const int nsplit = a.nsplit, least = a.least;
  const int lane = threadIdx.x & 31;
  const int per = slots * g.Hkv * a.njobs;
  const int part = a.taper ? n / per : n % nsplit;
  int m = a.taper ? n - part * per : n / nsplit;
  const int jb = m % a.njobs;
  m /= a.njobs;
  const Job& job = jb ? a.job1 : a.job;
  const int kvh = m % g.Hkv, slot = slots - 1 - m / g.Hkv;
  int tile;
  const int s = find_slot(g, most_heads(g, job.hc), rows, slot, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int x0 = tile * rows;
  if (hs.n == 0 || x0 >= q.nq * hs.n) return false;
  // lane 2 * half + segment: the tiles that half meets in that segment
  const int w = (lane >> 1) & 1, sg = lane & 1;
  int j0 = 0, j1 = 0;
  if (lane < 4 && sg < job.nseg && w * kNeed < rows && x0 + w * kNeed < q.nq * hs.n)
    tile_range(g, q, job, sg, hs, x0 + w * kNeed, kNeed, kNeed, j0, j1);
  // both halves together: rows follow one another, and so do their intervals
  const int o0 = __shfl_xor_sync(0xffffffffu, j0, 2), o1 = __shfl_xor_sync(0xffffffffu, j1, 2);
  int u0 = j0, u1 = j1;
  if (o1 > o0) {
    u0 = j1 > j0 ? imin(j0, o0) : o0;
    u1 = j1 > j0 ? imax(j1, o1) : o1;
  }
  const int cnt = u1 - u0;
  const int total = __shfl_sync(0xffffffffu, cnt, 0) + __shfl_sync(0xffffffffu, cnt, 1);
  const int parts = parts_of(total, nsplit, least);
  if (part >= parts) return false;
  // tapered: the rest shrinks with the square of the parts that are left
  auto cut = [&](int p) {
    const long long P = parts, left = parts - p;
    return a.taper ? (int)(total - total * (left * left) / (P * P)) : (int)(total * (long long)p / P);
  };
  if (lane < 4) {
    out->ja[w][sg] = j0;
    out->jb[w][sg] = j1;
    if (lane < 2) out->u0[sg] = u0;
    if (lane == 0) {
      out->live = 1;
      out->q = q;
      out->hs = hs;
      out->kvh = kvh;
      out->job = jb;
      out->x0 = x0;
      out->part = part;
      out->cnt0 = cnt;
      out->parts = parts;
      out->t0 = cut(part);
      out->t1 = cut(part + 1);
    }
  }
  __syncwarp();
  return true;
}

}  // namespace rag
}  // namespace st

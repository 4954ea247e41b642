// Attention of a few query rows per key/value head over a paged cache: decoding
// steps (one new token, the heads of a group as rows), very short chunks and the
// chunks of few strided sequences, in bf16 or fp16.
//
// Such a call reads every live key and value once and does 4 d flops a row with
// each, far below the tensor cores' rate at 16 rows, so memory bounds it; what
// counts is bytes in flight. A unit is 16 query rows of one (sequence, key/value
// head, job, key range), one CTA of four warps. Each warp takes every fourth tile
// of 16 keys on its own: its ring of K / V tiles in shared memory is filled by
// 16-byte asynchronous copies through the page table, no barrier stands between
// warps until the end, and the two CTAs of an SM (rings of 96 KB each at d = 128, of
// 80 at d = 64; a third would not fit) keep about 128 KB in flight. Scores and
// products are 16 x 8 x 16 matrix instructions (the rows fill their 16-row operand;
// tcgen05 would want 128), the softmax is online with fp32 statistics: the
// accumulator is rescaled only when a row's maximum grows by more than 2^8. The four
// warps' results are joined in shared memory; key ranges are joined by the parts
// kernel.
#include "ragged.h"
#include "tc_common.cuh"

namespace st {
namespace rag {
namespace {

using namespace st::tc;

constexpr int kWarps = 4;
constexpr int kKeys = 16;  // keys of a tile
constexpr int kRowsU = 16;
constexpr float kLn2 = 0.69314718055994531f;

template <int D>
struct Cfg {
  static constexpr int kStages = D == 64 ? 5 : 3;
  static constexpr int kTile = kKeys * D * 2;  // bytes of one K or V tile
  static constexpr int kSmem = kWarps * kStages * 2 * kTile;
};

template <int D>
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
  return (uint32_t)(row * (D * 2) + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32, 2)
    few_rows_kernel(const __grid_constant__ FwdLaunch a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NS = Cfg<D>::kStages, TB = Cfg<D>::kTile;
  constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows per copy instruction
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  const int jb = blockIdx.z / a.nsplit, part = blockIdx.z - jb * a.nsplit;
  const Job& job = jb ? a.job1 : a.job;
  int tile;
  const int s = find_slot(g, most_heads(g, job.hc), kRowsU, blockIdx.x, tile);
  const Seq q = load_seq(g, s);
  const Heads3 hs = heads_of_group(g, job.hc, kvh);
  const int x0 = tile * kRowsU;
  if (hs.n == 0 || x0 >= q.nq * hs.n) return;
  const int rows = imin(kRowsU, q.nq * hs.n - x0);

  int j0[2] = {0, 0}, cnt[2] = {0, 0};
#pragma unroll
  for (int sg = 0; sg < 2; ++sg)
    if (sg < job.nseg) {
      int j1;
      tile_range(g, q, job, sg, hs, x0, kRowsU, kKeys, j0[sg], j1);
      cnt[sg] = j1 - j0[sg];
    }
  const int total = cnt[0] + cnt[1];
  const int parts = parts_of(total, a.nsplit, a.least);
  if (part >= parts) return;
  const int t0 = (int)((long long)total * part / parts), t1 = (int)((long long)total * (part + 1) / parts);

  // rows of this thread: lane / 4 and lane / 4 + 8
  const int r0 = lane >> 2, cq = (lane & 3) * 2;
  int lo[2][2], hi[2][2];  // [row][segment]
  uint32_t qf[D / 16][4];
  {
    const uint16_t* qp = static_cast<const uint16_t*>(a.q);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      lo[y][0] = hi[y][0] = lo[y][1] = hi[y][1] = 0;
      QRow qr;
      const bool have = query_at(g, q, job.qview, hs, x0 + r0 + 8 * y, qr);
      if (have && qr.pos >= 0) {
        live_keys(g, q, job.seg[0].rule, qr.pos, lo[y][0], hi[y][0]);
        if (job.nseg > 1) live_keys(g, q, job.seg[1].rule, qr.pos, lo[y][1], hi[y][1]);
      }
      const uint16_t* src = qp + (size_t)(have ? q_row(g, qr.t, qr.h) : 0) * D + cq;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        qf[x][y] = have ? __ldg(reinterpret_cast<const uint32_t*>(src + x * 16)) : 0u;
        qf[x][2 + y] = have ? __ldg(reinterpret_cast<const uint32_t*>(src + x * 16 + 8)) : 0u;
      }
    }
  }

  const uint32_t ring = smem_u32(smem) + warp * (NS * 2 * TB);
  const int nt = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;  // tiles of this warp
  auto seg_tile = [&](int i, int& sg, int& j) {
    const int t = t0 + warp + i * kWarps;
    sg = t >= cnt[0] ? 1 : 0;
    j = (sg ? j0[1] - cnt[0] : j0[0]) + t;
  };
  const char *kb = static_cast<const char*>(a.k), *vb = static_cast<const char*>(a.v);
  auto load = [&](int i) {
    if (i < nt) {
      int sg, j;
      seg_tile(i, sg, j);
      const int view = sg ? job.seg[1].kview : job.seg[0].kview;
      // rows behind the last key repeat it (their weights are 0, and 0 times an
      // infinity in an unused slot would not be)
      const int e = imin(j * kKeys + (lane & 15), n_keys(q, view) - 1);
      const int r = k_row(g, q, key_pos(g, q, view, e), kvh);
      const uint32_t dst = ring + (i % NS) * (2 * TB);
      const int chunk = lane % CH, sub = lane / CH;
#pragma unroll
      for (int x = 0; x < kKeys / RPI; ++x) {
        const int y = x * RPI + sub;
        const size_t off = (size_t)__shfl_sync(0xffffffffu, r, y) * (D * 2) + chunk * 16;
        const uint32_t at = dst + swz<D>(y, chunk);
        cp16(at, kb + off);
        cp16(at + TB, vb + off);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) load(i);

  float o[D / 8][4];
#pragma unroll
  for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int i = 0; i < nt; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    __syncwarp();
    load(i + NS - 1);
    const uint32_t kt = ring + (i % NS) * (2 * TB), vt = kt + TB;
    int sg, j;
    seg_tile(i, sg, j);
    float c[2][4] = {};
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      // matrices: keys 0..7 and 8..15, two 16-byte chunks each
      uint32_t b[4];
      ldsm4(kt + swz<D>((lane & 7) + ((lane >> 4) << 3), x * 2 + ((lane >> 3) & 1)), b);
      mma16<F16>(c[0], qf[x], b[0], b[1]);
      mma16<F16>(c[1], qf[x], b[2], b[3]);
    }
    uint32_t p[4];
    float up[2];
    bool any = false;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int kl = (sg ? lo[y][1] : lo[y][0]) - j * kKeys, kh = (sg ? hi[y][1] : hi[y][0]) - j * kKeys;
      float mt = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int k = n * 8 + cq + z;
          float& v = c[n][2 * y + z];
          v = (k >= kl && k < kh) ? v * a.scale_log2 : -INFINITY;
          mt = fmaxf(mt, v);
        }
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
      up[y] = 1.f;
      if (mt > m[y] + 8.f) {
        up[y] = fast_exp2(m[y] - mt);
        m[y] = mt;
        any = true;
      }
      const float mu = m[y] == -INFINITY ? 0.f : m[y];
      float ps = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = fast_exp2(c[n][2 * y] - mu), p1 = fast_exp2(c[n][2 * y + 1] - mu);
        ps += p0 + p1;
        p[n * 2 + y] = pack2<F16>(p0, p1);
      }
      l[y] = l[y] * up[y] + ps;
    }
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        o[x][0] *= up[0];
        o[x][1] *= up[0];
        o[x][2] *= up[1];
        o[x][3] *= up[1];
      }
    }
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      uint32_t b[4];
      ldsm4t(vt + swz<D>(lane & 15, x * 2 + (lane >> 4)), b);
      mma16<F16>(o[2 * x], p, b[0], b[1]);
      mma16<F16>(o[2 * x + 1], p, b[2], b[3]);
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
  }

  // ---- join the four warps ----
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  constexpr int OP = D + 4;
  float* so = reinterpret_cast<float*>(smem);  // [warp][16][D + 4]
  float* sm = so + kWarps * kRowsU * OP;       // [warp][16] maximum, then sum
  static_assert(sizeof(float) * (kWarps * kRowsU * OP + 2 * kWarps * kRowsU) <= Cfg<D>::kSmem, "join buffer");
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    float* dst = so + (warp * kRowsU + r0 + 8 * y) * OP + cq;
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      *reinterpret_cast<float2*>(dst + x * 8) = make_float2(o[x][2 * y], o[x][2 * y + 1]);
    if ((lane & 3) == 0) {
      sm[warp * kRowsU + r0 + 8 * y] = m[y];
      sm[(kWarps + warp) * kRowsU + r0 + 8 * y] = l[y];
    }
  }
  __syncthreads();
  const int part0 = jb ? a.part1 : a.part0;
  for (int row = warp; row < rows; row += kWarps) {
    QRow qr;
    query_at(g, q, job.qview, hs, x0 + row, qr);
    const size_t rr = (size_t)qr.t * g.H + qr.h;
    float mx = -INFINITY, sum = 0.f, w[kWarps];
#pragma unroll
    for (int x = 0; x < kWarps; ++x) mx = fmaxf(mx, sm[x * kRowsU + row]);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      w[x] = mx > -INFINITY ? fast_exp2(sm[x * kRowsU + row] - mx) : 0.f;
      sum += w[x] * sm[(kWarps + x) * kRowsU + row];
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;  // NaN stays NaN
    const float L = sum != 0.f ? (mx + __log2f(sum)) * kLn2 : -INFINITY;
    const size_t stride = (size_t)g.total * g.H;
    for (int c = lane * 2; c < D; c += 64) {
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float2 f = *reinterpret_cast<const float2*>(so + (x * kRowsU + row) * OP + c);
        v0 = fmaf(w[x], f.x, v0);
        v1 = fmaf(w[x], f.y, v1);
      }
      if (a.mode == OUT_PARTIAL)
        *reinterpret_cast<float2*>(a.parts.o + ((part0 + part) * stride + rr) * D + c) =
            make_float2(v0 * inv, v1 * inv);
      else
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + rr * D + c) = pack2<F16>(v0 * inv, v1 * inv);
    }
    if (lane == 0) {
      if (a.mode == OUT_PARTIAL)
        a.parts.lse[(part0 + part) * stride + rr] = L;
      else
        a.lse[rr] = L;
    }
    if (a.mode == OUT_PARTIAL && part == 0)
      for (int p = parts + lane; p < a.nsplit; p += 32) a.parts.lse[(part0 + p) * stride + rr] = -INFINITY;
  }
}

template <int D, bool F16>
cudaError_t launch(const FwdLaunch& a) {
  const Geo& g = a.g;
  cudaError_t e = cudaFuncSetAttribute(few_rows_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  const long long slots = slot_count(g, most_heads(g, a.job.hc), kRowsU);
  few_rows_kernel<D, F16>
      <<<dim3((unsigned)slots, g.Hkv, a.njobs * a.nsplit), kWarps * 32, Cfg<D>::kSmem, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t few_rows_fwd(const FwdLaunch& a, int dtype) {
  if (a.g.d == 64) return dtype == ST_F16 ? launch<64, true>(a) : launch<64, false>(a);
  return dtype == ST_F16 ? launch<128, true>(a) : launch<128, false>(a);
}

}  // namespace rag
}  // namespace st

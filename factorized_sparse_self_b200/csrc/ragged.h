// Host-side launch entry points of the kernels for ragged and paged sequences
// (internal; CUDA files only).
#pragma once

#include "launch.h"
#include "ragged.cuh"

namespace st {
namespace rag {

// What becomes of a unit's output rows.
enum OutMode : int32_t {
  OUT_FINAL = 0,    // O and LSE are written
  OUT_PARTIAL = 1,  // fp32 O and LSE go to a part, joined later
  OUT_MERGE = 2     // joined with part 0 (another order's result), then written
};

// Several results of one query row over disjoint key sets ("parts"): fp32 O
// [parts][total][H][d] and natural-log LSE [parts][total][H], joined by their
// log-sum-exp.
struct Parts {
  float* o;
  float* lse;
};

// A unit's keys are cut into at most nsplit parts of at least `least` key tiles;
// its first part marks the parts it does not use as empty (LSE = -inf).
ST_HD int parts_of(int tiles, int nsplit, int least) {
  return imax(1, imin(nsplit, (tiles + least - 1) / least));
}

// One launch of a forward kernel: one or two jobs, each unit's keys cut into up
// to nsplit parts.
struct FwdLaunch {
  Geo g;
  Job job, job1;
  int32_t njobs;
  const void *q, *k, *v;
  void* o;
  float* lse;
  Parts parts;
  int32_t part0, part1;  // first part of each job
  int32_t nsplit;  // OUT_PARTIAL: most key ranges of a unit
  int32_t least;   // fewest key tiles of a range
  int32_t taper;   // ranges get shorter, and short ones go last
  int32_t mode;    // OutMode
  float scale_log2;
  int32_t force_timeout;  // test hook: each CTA's first key tile is never loaded
  uint64_t wait_ns;
  cudaStream_t stream;
};

// Backward, one key order's share of dK and dV: fp32 parts [parts][total][Hkv][2][d]
// when several jobs or key ranges add up, else written directly.
struct BwdLaunch {
  Geo g;
  Job job[2];        // key jobs: one segment each
  int32_t njobs;
  Job qjob[2];       // query jobs of this launch
  int32_t nqjobs, mode;
  int32_t part_view;  // dK, dV by OUT_MERGE: keys that the first order's part holds
  const void *q, *k, *v, *dout;
  const float* lse;
  float* delta;  // mended in place
  void *dq, *dk, *dv;
  Rows dq_rows, dk_rows, dv_rows;  // of the gradients
  float* parts;      // dK, dV parts
  float* dq_part;    // fp32 dQ [total][H][d] of the first query order
  int32_t mend_tiles;  // 16-bit: key tiles up to which a unit's rows have their delta mended,
  int32_t mend_below;  // if all are at positions below this
  float *kb_part, *r_part;  // of the first query order: sums P K, lost part of delta
  int32_t nsplit;
  float scale;
  uint64_t wait_ns;
  cudaStream_t stream;
};

#ifdef __CUDACC__
// Key heads that a job reaches: whether any query head of the group is in its
// class.
__device__ __forceinline__ bool job_reaches(const Geo& g, const Job& job, int kvh) {
  return heads_of_group(g, job.hc, kvh).n > 0;
}
// Whether kvh's dK, dV come from one unit alone and are written by it: one key
// range, one job, and an order that lists every key.
__device__ __forceinline__ bool dkv_direct(const BwdLaunch& a, int kvh) {
  if (a.mode == OUT_MERGE) return true;
  if (a.mode == OUT_PARTIAL || a.nsplit > 1) return false;
  int n = 0, view = VIEW_NAT;
  for (int j = 0; j < a.njobs; ++j)
    if (job_reaches(a.g, a.job[j], kvh)) {
      ++n;
      view = a.job[j].seg[0].kview;
    }
  return n == 1 && view != VIEW_SUM;
}
// Whether a view lists the key at a position of its sequence.
__device__ __forceinline__ bool view_lists(const Geo& g, int view, int pos) {
  return view != VIEW_SUM || pos - fdiv(pos, g.fl) * g.l >= g.l - g.c;
}
#endif

// Tensor-core forward: bf16 / fp16, d = 64 or 128.
cudaError_t tc_ragged_fwd(const FwdLaunch& a, int dtype);

// Tensor-core backward of packed sequences: dQ of one query order, and dK, dV.
cudaError_t tc_ragged_dq(const BwdLaunch& a, int dtype);
cudaError_t tc_ragged_dkv(const BwdLaunch& a, int dtype);

// Few query rows per key/value head over a paged cache (decoding steps): bf16 /
// fp16, d = 64 or 128.
cudaError_t few_rows_fwd(const FwdLaunch& a, int dtype);

// CUDA-core kernels for float32 tensors.
cudaError_t simt_ragged_fwd(const FwdLaunch& a);
cudaError_t simt_ragged_dq(const BwdLaunch& a);
cudaError_t simt_ragged_dkv(const BwdLaunch& a);

// Joins nparts parts of every query row (rows of no sequence are skipped).
cudaError_t join_parts(const Geo& g, int dtype, const Parts& parts, int nparts,
                       void* o, float* lse, cudaStream_t stream);
// delta[t][h] = dout . o
cudaError_t row_delta(const Geo& g, int dtype, const void* o, const void* dout, float* delta,
                      cudaStream_t stream);
// Sums the parts of dK, dV and rounds them.
cudaError_t join_dkv(const BwdLaunch& a, int dtype);

// Writes the token rows of k, v (rows kin, vin) into their slots of the cache.
cudaError_t cache_append(const Geo& g, const Rows& kin, const Rows& vin, int elem_bytes,
                         const void* k, const void* v, void* kc, void* vc, cudaStream_t s);

}  // namespace rag
}  // namespace st

// Verification of drafted tokens against the target's probabilities, and the
// token drawn after the last one that stands. Contract in include/bws.h.
//
// A request is one cluster of CTAs. Its first warp's lanes test the drafts (a
// product of two FP32 numbers is exact in FP64, so the test has no rounding);
// the number that stand picks the row to draw from, whose w = max(p - q, 0) the
// cluster sums once: every warp owns a contiguous range of the vocabulary and
// sends its sum to every CTA over distributed shared memory. CTA 0 finds the
// range in which the running sum passes u * total and reads only that one again
// (now in L2), first by sixteenths, a warp each, then word by word.
// A warp adds FP32 numbers in two words (the rounded sum and what the rounding
// left), which carries 48 bits: FP64 adds run at about 2 a clock and SM here and
// would set the time. FP64 takes over at the warps' sums, in one warp.
// Bound: the chain of dependent loads, the cluster's two barriers and the
// launch for few requests (one with eight rows of 248320: 10.0 us); the bytes of
// one or two rows a request for many (64 requests at 157184: 19.7 us for 69 MB,
// 3.5 TB/s: clusters that refused a draft read twice what the others do, and one
// wave holds them all, so the mean SM is busy two thirds of the time; 17.0 for 40
// MB where the drafts were certain).
#include <cooperative_groups.h>

#include <atomic>

#include "bws_abi_util.h"
#include "bws_common.cuh"
#include "bws_internal.h"

namespace cg = cooperative_groups;

namespace bws {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxRows = 32;
constexpr int kVerifyMaxCluster = 16;

struct VerifyParams {
  const float* target;
  long long target_stride;
  const float* draft;
  long long draft_stride;
  const int32_t* tokens;
  int n_rows, vocab;
  const int32_t* row_start;
  const float *accept_u, *sample_u;
  int max_rows;
  int32_t *out, *n_out;
  int vec;   // rows start on 16-byte boundaries
};

// hi + lo += w, w >= 0 (Knuth's two-sum: the rounded sum and its exact error)
BWS_DEV void two_word_add(float& hi, float& lo, float w) {
  const float s = __fadd_rn(hi, w);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(w, b)));
  hi = s;
}

// The row to draw from: w(v) = max(p - q, 0); q is a row, or certain at token
// `certain`, or nothing.
struct Row {
  const float* p;
  const float* q;
  int certain;
};

BWS_DEV float weight_of(float p, float q) { return fmaxf(__fsub_rn(p, q), 0.0f); }   // NaN gives 0

BWS_DEV float weight_at(const Row& row, int v) {
  if (v == row.certain) return 0.0f;
  return weight_of(__ldg(row.p + v), row.q != nullptr ? __ldg(row.q + v) : 0.0f);
}

BWS_DEV float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// hi + lo += b's two words
BWS_DEV void two_word_join(float& hi, float& lo, float bh, float bl) {
  const float s = __fadd_rn(hi, bh);
  const float b = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(bh, b));
  lo = __fadd_rn(__fadd_rn(lo, bl), e);
  hi = s;
}

// Sum of w over [a, b) by one warp (the same in every lane). a % 4 == 0.
template <bool VEC, bool HAS_Q>
BWS_DEV double range_sum(const Row& row, int a, int b, int lane) {
  float hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
  if constexpr (VEC) {
    constexpr int U = 4;   // loads in flight: U rows of 512 bytes from p, and from q
    for (int v = a + lane * 4; v < b; v += U * 128) {
      float4 x[U], y[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = v + u * 128;
        x[u] = y[u] = make_float4(0, 0, 0, 0);
        if (at + 3 < b) {
          x[u] = load4(row.p + at);
          if constexpr (HAS_Q) y[u] = load4(row.q + at);
        } else if (at < b) {   // the vocabulary's last words; a row may end with them
          x[u].x = __ldg(row.p + at);
          if (at + 1 < b) x[u].y = __ldg(row.p + at + 1);
          if (at + 2 < b) x[u].z = __ldg(row.p + at + 2);
          if constexpr (HAS_Q) {
            y[u].x = __ldg(row.q + at);
            if (at + 1 < b) y[u].y = __ldg(row.q + at + 1);
            if (at + 2 < b) y[u].z = __ldg(row.q + at + 2);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int d = row.certain - (v + u * 128);
        two_word_add(hi[0], lo[0], d == 0 ? 0.0f : weight_of(x[u].x, y[u].x));
        two_word_add(hi[1], lo[1], d == 1 ? 0.0f : weight_of(x[u].y, y[u].y));
        two_word_add(hi[2], lo[2], d == 2 ? 0.0f : weight_of(x[u].z, y[u].z));
        two_word_add(hi[3], lo[3], d == 3 ? 0.0f : weight_of(x[u].w, y[u].w));
      }
    }
  } else {
    for (int v = a + lane; v < b; v += 256) {
      float x[8], y[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        x[u] = y[u] = 0.0f;
        if (v + u * 32 < b) {
          x[u] = __ldg(row.p + v + u * 32);
          if constexpr (HAS_Q) y[u] = __ldg(row.q + v + u * 32);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        two_word_add(hi[u & 3], lo[u & 3], v + u * 32 == row.certain ? 0.0f : weight_of(x[u], y[u]));
    }
  }
#pragma unroll
  for (int k = 1; k < 4; ++k) two_word_join(hi[0], lo[0], hi[k], lo[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, hi[0], o), l = __shfl_xor_sync(0xffffffffu, lo[0], o);
    two_word_join(hi[0], lo[0], h, l);
  }
  return (double)hi[0] + (double)lo[0];
}

BWS_DEV double warp_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

BWS_DEV double sum_of(const VerifyParams& p, const Row& row, int a, int b, int lane) {
  if (p.vec)
    return row.q != nullptr ? range_sum<true, true>(row, a, b, lane) : range_sum<true, false>(row, a, b, lane);
  return row.q != nullptr ? range_sum<false, true>(row, a, b, lane) : range_sum<false, false>(row, a, b, lane);
}

// One warp: the first of n (a multiple of 16, at most 256) ranges whose running
// sum passes target(total); else, where rounding leaves none, the last that has
// any weight; -1 if no range has. *before: the sum of the ranges ahead of it.
template <class F>
BWS_DEV int pick_range(const double* sums, int n, F target, double* before, int lane) {
  constexpr int kMost = kVerifyMaxCluster * kVerifyWarps / 32;
  const int each = (n + 31) / 32;
  double x[kMost], mine = 0.0;   // a lane's ranges, in order
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int k = lane * each + i;
    x[i] = i < each && k < n ? sums[k] : 0.0;
    mine += x[i];
  }
  const double upto = warp_scan(mine, lane);
  const double t = target(__shfl_sync(0xffffffffu, upto, 31));
  double run = upto - mine, found_at = 0.0, last_at = 0.0;
  int found = -1, last = -1;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (x[i] > 0.0) {
      last = lane * each + i;
      last_at = run;
      if (found < 0 && run + x[i] > t) {
        found = last;
        found_at = run;
      }
    }
    run += x[i];
  }
  const unsigned fb = __ballot_sync(0xffffffffu, found >= 0), lb = __ballot_sync(0xffffffffu, last >= 0);
  const int from = fb != 0u ? __ffs(fb) - 1 : lb != 0u ? 31 - __clz(lb) : 0;
  *before = __shfl_sync(0xffffffffu, fb != 0u ? found_at : last_at, from);
  return __shfl_sync(0xffffffffu, fb != 0u ? found : last, from);
}

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double s_sum[kVerifyMaxCluster * kVerifyWarps], s_part[kVerifyWarps], s_left;
  __shared__ int s_pick;
  __shared__ int s_stand;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_cta = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int r = (int)blockIdx.x / n_cta;
  cluster.barrier_arrive();   // every CTA has started before any writes to another
  pdl_launch_dependents();
  pdl_wait();
  const int start = min(max(p.row_start[r], 0), p.n_rows);
  const int rows = max(min(p.row_start[r + 1], p.n_rows) - start, 0);
  if (rows == 0 || rows > p.max_rows) {   // nothing to verify, or no room for it: the whole cluster leaves
    if (rank == 0) {
      for (int i = threadIdx.x; i < p.max_rows; i += kVerifyThreads) p.out[(size_t)r * p.max_rows + i] = -1;
      if (threadIdx.x == 0) p.n_out[r] = rows == 0 ? 0 : -1;
    }
    cluster.barrier_wait();
    return;
  }
  int token = -1;   // lane i of warp 0: draft i
  if (warp == 0) {
    bool ok = false;
    if (lane < rows - 1) {
      token = p.tokens[start + lane];
      if (token >= 0 && token < p.vocab) {
        const float u = p.accept_u[start + lane];
        const float t = p.target[(start + lane) * p.target_stride + token];
        const float d = p.draft != nullptr ? p.draft[(start + lane) * p.draft_stride + token] : 1.0f;
        ok = (double)u * (double)d < (double)t;
      }
    }
    const unsigned b = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_stand = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
  }
  __syncthreads();
  const int stand = s_stand;
  const int here = start + stand;
  Row row;
  row.p = p.target + here * p.target_stride;
  const bool refused = stand < rows - 1;
  row.q = refused && p.draft != nullptr ? p.draft + here * p.draft_stride : nullptr;
  row.certain = refused && p.draft == nullptr ? max(p.tokens[here], -1) : -1;

  // a warp's range: a multiple of four words, as even as that allows
  const int n_warps = n_cta * kVerifyWarps;
  const int quads = (p.vocab + 3) / 4, per = (quads + n_warps - 1) / n_warps;
  const int w = rank * kVerifyWarps + warp;
  auto range_begin = [&](int i) { return (int)min((long long)i * per * 4, (long long)p.vocab); };
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const double s = sum_of(p, row, range_begin(w), range_begin(w + 1), lane);
    if (pass == 0) cluster.barrier_wait();
    // every CTA gets every warp's sum: none reads another's memory afterwards
    if (lane < n_cta) cluster.map_shared_rank(s_sum, lane)[w] = s;
    cluster.sync();
    if (row.q == nullptr && row.certain < 0) break;
    bool any = false;   // is anything left of the target?
    for (int i = lane; i < n_warps; i += 32) any |= __double_as_longlong(s_sum[i]) > 0;
    if (__any_sync(0xffffffffu, any)) break;
    row.q = nullptr;
    row.certain = -1;
    cluster.sync();   // every read of the sums, before they are formed again
  }
  if (rank != 0) return;

  // ---- CTA 0: the range in which the running sum passes u * total ...
  // (one warp: FP64 runs at about 2 a clock and SM)
  if (warp == 0) {
    double t, before;
    const int k = pick_range(s_sum, n_warps, [&](double total) { return t = (double)p.sample_u[r] * total; }, &before, lane);
    if (lane == 0) {
      s_pick = k;
      s_left = t - before;
    }
  }
  __syncthreads();
  const int k = s_pick;
  const double left = s_left;
  int drawn = -1;
  if (k >= 0) {
    // ... its sixteenths, a warp each, and the one in which it passes
    const int a = range_begin(k), b = range_begin(k + 1);
    const int part = ((b - a + 4 * kVerifyWarps - 1) / (4 * kVerifyWarps)) * 4;
    const int a1 = min(a + warp * part, b), b1 = min(a1 + part, b);
    const double s = sum_of(p, row, a1, b1, lane);
    if (lane == 0) s_part[warp] = s;
    __syncthreads();
    if (warp != 0) return;
    double before1;
    const int k1 = pick_range(s_part, kVerifyWarps, [&](double) { return left; }, &before1, lane);
    // ... and the word
    if (k1 >= 0) {
      const int a2 = min(a + k1 * part, b), b2 = min(a2 + part, b);
      double base = before1;
      int fallback = -1;
      for (int v0 = a2; v0 < b2 && drawn < 0; v0 += 128) {
        const int v = v0 + lane * 4;
        float x[4];
        double own = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v + i < b2 ? weight_at(row, v + i) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) own += x[i];
        const double scan = warp_scan(own, lane);
        double at = base + (scan - own);
        int mine_v = -1, mine_last = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          at += x[i];
          if (x[i] > 0.0f) {
            mine_last = v + i;
            if (mine_v < 0 && at > left) mine_v = v + i;
          }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, mine_v >= 0), any = __ballot_sync(0xffffffffu, mine_last >= 0);
        if (hit != 0u) drawn = __shfl_sync(0xffffffffu, mine_v, __ffs(hit) - 1);
        if (any != 0u) fallback = __shfl_sync(0xffffffffu, mine_last, 31 - __clz(any));
        base += __shfl_sync(0xffffffffu, scan, 31);
      }
      if (drawn < 0) drawn = fallback;
    }
  } else if (warp != 0) {
    return;
  }
  if (lane < p.max_rows) {
    int32_t v = -1;
    if (lane < stand) v = token;
    else if (lane == stand) v = drawn;
    p.out[(size_t)r * p.max_rows + lane] = v;
  }
  if (lane == 0) p.n_out[r] = stand + 1;
}

}  // namespace
}  // namespace bws

extern "C" int bws_draft_verify(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                                const int32_t* tokens, int n_rows, int vocab, const int32_t* row_start, int n_requests,
                                const float* accept_u, const float* sample_u, int max_rows, int32_t* out,
                                int32_t* n_out, void* stream) {
  using namespace bws;
  const char* name = "bws_draft_verify";
  if (n_requests < 0 || n_requests > (1 << 20) || n_rows < 0)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_requests = %d, n_rows = %d", name, n_requests, n_rows);
  if (max_rows < 1 || max_rows > kVerifyMaxRows)
    return fail(BWS_ERR_INVALID_ARG, "%s: max_rows = %d must be in [1, %d]", name, max_rows, kVerifyMaxRows);
  if (vocab < 1 || vocab > (1 << 28)) return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: vocab = %d", name, vocab);
  if (n_requests == 0) {
    clear_error();
    return BWS_OK;
  }
  if (!row_start || !sample_u || !out || !n_out || (n_rows > 0 && (!target || !tokens || !accept_u)))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (target_stride < vocab || (draft && draft_stride < vocab))
    return fail(BWS_ERR_INVALID_ARG, "%s: row strides must be at least the vocabulary", name);
  const void* ptrs[] = {target, draft, tokens, row_start, accept_u, sample_u, out, n_out};
  for (const void* q : ptrs)
    if (!aligned(q, 4)) return fail(BWS_ERR_MISALIGNED, "%s: 4-byte alignment needed", name);
  VerifyParams p = {target, target_stride, draft, draft_stride, tokens, n_rows, vocab, row_start,
                    accept_u, sample_u, max_rows, out, n_out, 0};
  p.vec = aligned(target, 16) && target_stride % 4 == 0 &&
          (draft == nullptr || (aligned(draft, 16) && draft_stride % 4 == 0));
  // One request is bound by what an SM can load: as many CTAs as a cluster
  // takes. Many requests fill the GPU with smaller clusters.
  int cluster = kVerifyMaxCluster;
  while (cluster > 1 && (long long)n_requests * cluster > 2LL * num_sms()) cluster >>= 1;
  // a warp with less than 128 words only adds to the joining
  while (cluster > 1 && (long long)cluster * kVerifyWarps * 128 > 2LL * vocab) cluster >>= 1;
  static std::atomic<unsigned long long> attr{0};
  const unsigned long long bit = 1ull << (current_device() & 63);
  if (!(attr.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return cuda_status(e, name);
    attr.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_requests * cluster));
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = as_stream(stream);
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = (unsigned)cluster;
  a[1].val.clusterDim.y = 1;
  a[1].val.clusterDim.z = 1;
  cfg.attrs = a;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, verify_kernel, p), name);
}

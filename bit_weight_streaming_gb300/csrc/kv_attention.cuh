// Shared by the attention kernels over the 8-bit cache (kv_attention.cu for few
// query rows, kv_attention_wide.cu for many) and over the 4-bit one
// (kv4_attention.cu, kv4_attention_wide.cu): their parameters, the line of shares, the
// rows without a result, the shared-memory tiles. Each cache joins its partial results by
// a kernel of its own.
#pragma once
#include <cuda.h>

#include "bws_abi_util.h"
#include "bws_common.cuh"
#include "bws_internal.h"

namespace bws {

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kBox = 16;                   // cached tokens of a TMA box: never across a block
constexpr int kAttnMaxRows = kMaxTokens;   // rows of a request
constexpr int kAttnMaxGroup = 16;          // query heads of a kv head
constexpr uint32_t kAttnPolls = 1u << 20;
constexpr float kNone = -3.0e38f;           // a running maximum of nothing
// Weights are 2^(x - m), at most 2^kTop in f16: m is set kTop - margin below the
// largest exponent and follows only where one passes it by kTop. So a weight is
// rounded by 2^-11 down to 2^-(kTop - margin + 14) of a row's largest; below that
// f16's step is fixed. That tail counts: a token that takes most of the weight and
// carries no value leaves the result to all the others. A smaller margin reaches
// further down and moves the maxima more often. With a margin of 4 / 6 / 8, us: 8
// rows of 24 heads of 256 at 100001 70.0 / 67.5 / 66.6, of 64 heads of 64 92.3 /
// 88.9 / 87.8, 24 short requests of up to 8 rows of 24 heads of 256 35.5 / 35.0 /
// 34.2; one row a request alike.
constexpr float kTop = 15.0f, kMargin = 6.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the attention kernels of every cache share: the call, the line of shares,
// the partial results.
struct AttnLine {
  const uint16_t* q;
  long long q_row_stride, q_head_stride;
  int n_rows, H, K, G;
  int B, n_blocks;
  uint32_t b_inverse; // ceil(2^32 / (B / 16)), 0 for B = 16
  const int32_t* table;
  int max_blocks, R;
  int max_tokens;     // of a table row
  const int32_t *row_start, *kv_lens;
  int max_rows;
  float scale;
  uint16_t* out;
  float* lse;
  float* part_o;      // [2 * CTAs][group_rows][D]
  float2* part_ml;    // [2 * CTAs][group_rows]
  int4* cut;          // [max(CTAs, segments)][2]: segments that other CTAs go on with
  int by_segment;     // cut's index: the segment, else the CTA that starts it
  int max_groups;     // row groups of a full request
  uint32_t* failed;   // [CTAs]: bws_status_bits
  uint32_t* hdr;
  int n_ctas, least;  // CTAs; smallest share in units
  int lead;           // what a segment costs beside its units, in units
  int unit;           // cached tokens of a unit
  int group_rows;     // rows of a row group
};

struct AttnParams : AttnLine {
  CUtensorMap k, v;
  const float *k_scale, *v_scale;
};

// ---- the line of units -----------------------------------------------------------

// token / B, exactly: in units of 16 the quotient's error, below 16 * 2^27 / 2^32, never reaches the next whole.
BWS_DEV int block_index(const AttnLine& p, int token) {
  const uint32_t t = (uint32_t)token >> 4;
  return (int)(p.b_inverse != 0u ? __umulhi(t, p.b_inverse) : t);
}

struct Request {
  int start, all, len;    // its first row; its rows, of which max_rows are computed; its tokens, by the caller's word
  int units, groups;      // units of one segment; row groups
  // What follows from these is formed where it is used: kept beside them it cost registers that the loops need.
  BWS_DEV int rows(const AttnLine& p) const { return min(all, p.max_rows); }
  BWS_DEV int kv(const AttnLine& p) const { return min(len, p.max_tokens); }   // tokens that the table row can hold
  BWS_DEV int seen0() const { return len - all; }   // the last token that row 0 sees; row j sees j more
};

BWS_DEV Request request_from(const AttnLine& p, int begin, int end, int kv, int group_rows) {
  Request q;
  q.start = min(max(begin, 0), p.n_rows);
  q.all = max(min(end, p.n_rows) - q.start, 0);
  q.len = max(kv, 0);
  // a request without tokens still writes its rows; unsigned, since kv may be all but 2^31
  q.units = max(1, (int)((uint32_t)(q.kv(p) + p.unit - 1u) / (uint32_t)p.unit));
  q.groups = (q.rows(p) * p.G + group_rows - 1) / group_rows;
  return q;
}

BWS_DEV Request request_of(const AttnLine& p, int r, int group_rows) {
  return request_from(p, p.row_start[r], p.row_start[r + 1], p.kv_lens[r], group_rows);
}

BWS_DEV long long length_of(const AttnLine& p, const Request& q) {
  return (long long)p.K * q.groups * (p.lead + q.units);
}

struct Line {
  long long total, share;
  int r;            // request that holds the asked position
  long long base;   // its first position
};

// The whole CTA: the line's length, the share, and the request at position
// cta * share, if the line has it. s_status (set before) gains a bit where a
// request has too many rows.
BWS_DEV Line find_on_line(const AttnLine& p, int group_rows, int cta, long long* s_warp, long long* s_found,
                          uint32_t* s_status) {
  const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + n - 1) / n;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  long long mine = 0;
  bool excess = false;
  for (int r = r0; r < r1; ++r) {
    const Request q = request_of(p, r, group_rows);
    mine += length_of(p, q);
    excess |= q.all > p.max_rows;
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (excess) atomicOr(s_status, (uint32_t)BWS_STATUS_KV_ROWS);
  long long before = inc - mine, total = 0;
  for (int w = 0; w < n / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  Line line;
  line.total = total;
  const long long share = (total + p.n_ctas - 1) / p.n_ctas;
  line.share = share < p.least ? p.least : share;
  const long long u = cta * line.share;
  if (u >= before && u < before + mine) {
    long long b = before;
    int r = r0;
    for (; r < r1 - 1; ++r) {
      const long long k = length_of(p, request_of(p, r, group_rows));
      if (u < b + k) break;
      b += k;
    }
    s_found[0] = r;
    s_found[1] = b;
  }
  __syncthreads();
  line.r = (int)s_found[0];
  line.base = s_found[1];
  return line;
}

// One CTA's part of a segment: units [first, last).
struct Segment {
  Request rq;
  int r, head, row0, first, last;
  bool whole;      // the CTA has every unit
  bool starts;     // the CTA has the first unit
  int pieces;      // CTAs that have units, from the one that starts it on
};

// A CTA's way along its share, segment by segment. The next request's numbers
// are asked for when this one is entered, and a segment follows the one before
// without a division: looked up and divided for, a step took 1100 cycles.
struct Walk {
  long long u, u0, u1, share;
  long long at;          // where segment seg of request r starts on the line
  int r, seg, cta;
  Request rq;            // request r
  int end, next_end, next_kv;   // row_start[r + 1], row_start[r + 2], kv_lens[r + 1]

  BWS_DEV void look_ahead(const AttnLine& p) {
    const bool there = r + 1 < p.R;
    next_end = there ? p.row_start[r + 2] : end;
    next_kv = there ? p.kv_lens[r + 1] : 0;
  }
  // (the whole CTA)
  BWS_DEV void start(const AttnLine& p, int group_rows, long long* s_warp, long long* s_found, uint32_t* s_status) {
    cta = blockIdx.x;
    const Line line = find_on_line(p, group_rows, cta, s_warp, s_found, s_status);
    share = line.share;
    u = u0 = cta * share;
    u1 = min(line.total, u0 + share);
    if (u < u1) {
      r = line.r;
      const int begin = p.row_start[r], kv = p.kv_lens[r];
      end = p.row_start[r + 1];
      look_ahead(p);
      rq = request_from(p, begin, end, kv, group_rows);
      const int len = p.lead + rq.units;
      const long long in = u - line.base;   // the short division where it holds it
      seg = in >> 32 == 0 ? (int)((uint32_t)in / (uint32_t)len) : (int)(in / len);
      at = line.base + (long long)seg * len;
    }
    if (threadIdx.x == 0 && !p.by_segment) p.cut[2 * cta + 1] = make_int4(0, 0, 0, 0);
  }
  // The next segment that the share has units of; false: the share is done.
  BWS_DEV bool next(const AttnLine& p, int group_rows, Segment& sg) {
    while (u < u1) {
      if (seg >= p.K * rq.groups) {
        ++r;
        seg = 0;
        rq = request_from(p, end, next_end, next_kv, group_rows);
        end = next_end;
        look_ahead(p);
        continue;
      }
      const long long b = at + p.lead + rq.units, first_unit = at + p.lead;
      const long long from = max(u, first_unit), to = min(u1, b);
      const int s = seg;
      u = to;
      if (to == b) {
        ++seg;
        at = b;
      }
      if (from >= to) continue;   // the share ends before the first unit
      sg.rq = rq;
      sg.r = r;
      sg.head = rq.groups == 1 ? s : s / rq.groups;
      sg.row0 = (s - sg.head * rq.groups) * group_rows;
      sg.first = (int)(from - first_unit);
      sg.last = (int)(to - first_unit);
      sg.starts = first_unit >= u0;
      sg.whole = sg.starts && to == b;
      sg.pieces = sg.starts && !sg.whole ? (int)((b - 1) / share) - cta + 1 : 1;
      if (sg.starts && threadIdx.x == 0 && (sg.pieces > 1 || p.by_segment)) {   // for the join
        const int c = p.by_segment ? (r * p.K + sg.head) * p.max_groups + s - sg.head * rq.groups : cta;
        p.cut[2 * c] = make_int4(rq.start, min(rq.rows(p) * p.G - sg.row0, group_rows), sg.head, sg.row0);
        p.cut[2 * c + 1] = make_int4(sg.pieces, cta, 0, 0);
      }
      return true;
    }
    return false;
  }
};

// ---- rows without a result, and the status ---------------------------------------

// Output rows without a result of their own become what a row without tokens is:
// rows of no request (before `begin`, from `end` on), as a captured step's padding,
// and a request's rows past max_rows. n_ctas CTAs take them in turn. Out of
// line: the join lasts a few loads, and a call without such rows fetches none of it.
template <int D>
static __device__ __noinline__ void clear_rows(const AttnLine& p, int begin, int end, bool excess, int cta, int n_ctas) {
  auto clear = [&](int from, int to) {
    for (int row = from + cta; row < to; row += n_ctas) {
      uint4* const out = reinterpret_cast<uint4*>(p.out + (size_t)row * p.H * D);
      for (int i = threadIdx.x; i < p.H * (D / 8); i += blockDim.x) out[i] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (int i = threadIdx.x; i < p.H; i += blockDim.x) p.lse[(size_t)row * p.H + i] = -INFINITY;
    }
  };
  clear(0, min(begin, p.n_rows));
  clear(max(end, 0), p.n_rows);
  for (int r = 0; excess && r < p.R; ++r) {
    const Request q = request_of(p, r, p.group_rows);
    clear(q.start + q.rows(p), q.start + q.all);
  }
}

// ---- tiles ---------------------------------------------------------------------

// A box of 16 tokens (from `token` of a block's head): all panels of 128 bytes of their rows, panel by panel.
BWS_DEV void tma_load_box(uint32_t dst, const void* tmap, int token, int head, int block, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %2, %4, %5}], [%6], %7;"
      :: "r"(dst), "l"(tmap), "r"(0), "r"(token), "r"(head), "r"(block), "r"(bar), "l"(pol) : "memory");
}
BWS_DEV void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
BWS_DEV void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// mma_f16_16816 as a value of its operands alone: free to be scheduled.
BWS_DEV void mma_free(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
BWS_DEV uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
BWS_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
BWS_DEV void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Byte offset of 16-byte chunk `c` of token row `row` in a side.
template <int D>
BWS_DEV uint32_t chunk_at(int row, int c) {
  if constexpr (D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  else return (c >> 3) * (kBox * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

// kv_attention_wide.cu: nt tiles of 8 rows, 6 or 8, of 256 also 4.
constexpr int kWideTile = 128;   // cached tokens of its unit
cudaError_t launch_attn_wide(int D, int nt, const AttnParams& p, cudaStream_t st);

// kv_attention.cu: the host's part that every cache shares.
// Where a workspace holds what a call of n_ctas CTAs and row groups of
// group_rows rows of D leaves for the join.
struct AttnLayout {
  size_t off_cut, off_failed, off_ml, off_o, total;
};
AttnLayout attn_layout(int n_ctas, int group_rows, int D);
bool attn_dims_ok(int H, int K, int D, int max_rows);
// The call as its arguments give it.
struct AttnCall {
  const uint16_t* q;
  int64_t q_row_stride, q_head_stride;
  int n_rows, n_q_heads;
  const int32_t* block_table;
  int max_blocks, n_requests;
  const int32_t *row_start, *kv_lens;
  int max_rows;
  float scale;
  uint16_t* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
};
// Argument checks over a cache of K heads of D in blocks of B tokens: BWS_OK or
// a status; *nothing: there is nothing to do.
int check_attn_call(const AttnCall& c, int K, int D, int B, const char* name, bool* nothing);
// The line's parameters from a checked call, but for least, lead and unit.
void fill_attn_line(AttnLine& p, const AttnCall& c, int K, int B, int n_blocks, int n_ctas, int group_rows,
                    const AttnLayout& L);

}  // namespace bws

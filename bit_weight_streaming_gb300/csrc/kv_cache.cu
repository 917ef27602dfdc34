// The 8-bit key/value cache: block tables and slots from request lengths, and
// the norm, rotation and E4M3 write of a step's queries, keys and values.
// Contracts in include/bws.h.
#include <atomic>

#include "bws_abi_util.h"
#include "bws_common.cuh"
#include "bws_internal.h"
#include "kv_cache.cuh"

namespace bws {
namespace {

// ---- block tables and slots -----------------------------------------------------
//
// Everything follows from two running sums over the requests: rows before a
// request and blocks taken before it. Every CTA forms both sums for all
// requests itself (two loads a request, shared by L2) and then fills its share
// of the rows and of the taken blocks, so one launch suffices and no CTA waits
// for another. A row inside a block that this call takes reads it from the
// free list, not from the table entry another CTA is writing.
// Bound: launch and the chain of two dependent loads for few requests (one of
// eight rows: 3.5 us); 384 requests with 374000 rows, 3.0 MB: 6.4 us, of which the
// launch, the CTAs' own sums and the search of a row's request are all but half a
// microsecond.

constexpr int kPlanThreads = 256;
constexpr int kPlanMaxRequests = 4096;

struct PlanParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int R, B;
  int32_t* table;
  int max_blocks;
  const int32_t* free_blocks;
  int n_list;   // entries of free_blocks: *n_free, read here, may not be trusted with them
  const int32_t* n_free;
  int n_rows;
  int32_t *slots, *positions, *row_start, *kv_lens, *n_free_out, *status;
  int vec;   // slots and positions on 16-byte boundaries
};

// Largest r in [0, n) with a[r] <= i, a non-decreasing and a[0] = 0.
BWS_DEV int last_not_above(const int* a, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Blocks that hold n tokens; n may be the sum of two lengths, below 2^32 - B.
BWS_DEV uint32_t blocks_of(uint32_t n, int B) { return n / (uint32_t)B + (n % (uint32_t)B != 0 ? 1u : 0u); }

BWS_DEV int clamp_i32(long long v) { return v > 0x7fffffffLL ? 0x7fffffff : (int)v; }

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanParams p) {
  extern __shared__ int s_plan[];   // rows before [R + 1], blocks before [R + 1], lengths [R]
  int* s_row = s_plan;
  int* s_blk = s_plan + p.R + 1;
  int* s_seq = s_plan + 2 * (p.R + 1);
  __shared__ long long s_wr[kPlanThreads / 32], s_wb[kPlanThreads / 32];
  __shared__ int s_over;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) s_over = 0;
  const int n_given = *p.n_free, n_free = min(max(n_given, 0), p.n_list);
  const int per = (p.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  long long rows = 0, blks = 0;
  bool over = false;
  for (int r = r0; r < r1; ++r) {
    const uint32_t seq = max(p.seq_lens[r], 0), nw = max(p.new_lens[r], 0);
    const uint32_t have = blocks_of(seq, p.B), need = blocks_of(seq + nw, p.B);
    s_row[r] = (int)nw;
    s_seq[r] = (int)seq;
    const uint32_t most = (uint32_t)p.max_blocks;   // what the table row cannot hold is not taken
    const uint32_t take = min(need, most) - min(have, most);
    s_blk[r] = (int)take;
    rows += nw;
    blks += take;
    over |= need > most;
  }
  long long ir = rows, ib = blks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, ir, o), b = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) { ir += a; ib += b; }
  }
  if (lane == 31) { s_wr[warp] = ir; s_wb[warp] = ib; }
  __syncthreads();
  if (over) s_over = 1;
  long long br = ir - rows, bb = ib - blks, tr = 0, tb = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) { br += s_wr[w]; bb += s_wb[w]; }
    tr += s_wr[w];
    tb += s_wb[w];
  }
  for (int r = r0; r < r1; ++r) {   // sums past 2^31 - 1 saturate: rows and free blocks end far below
    const int nr = s_row[r], nb = s_blk[r];
    s_row[r] = clamp_i32(br);
    s_blk[r] = clamp_i32(bb);
    br += nr;
    bb += nb;
  }
  if (tid == 0) { s_row[p.R] = clamp_i32(tr); s_blk[p.R] = clamp_i32(tb); }
  __syncthreads();
  const int total = s_row[p.R], taken = s_blk[p.R];
  if (blockIdx.x == 0) {
    for (int r = tid; r <= p.R; r += kPlanThreads) {
      p.row_start[r] = s_row[r];
      if (r < p.R) p.kv_lens[r] = clamp_i32((long long)s_seq[r] + max(p.new_lens[r], 0));
    }
    if (tid == 0) {
      *p.n_free_out = max(n_free - taken, 0);
      *p.status = (taken > n_free ? BWS_KV_NO_BLOCKS : 0) | (s_over ? BWS_KV_TABLE_FULL : 0) |
                  (total > p.n_rows ? BWS_KV_NO_ROWS : 0) | (n_given > p.n_list ? BWS_KV_LIST_SHORT : 0);
    }
  }
  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  for (long long i = first; i < taken; i += step) {
    const int r = last_not_above(s_blk, p.R, (int)i);
    const long long c = blocks_of(s_seq[r], p.B) + (i - s_blk[r]);
    p.table[(size_t)r * p.max_blocks + c] = i < n_free ? p.free_blocks[n_free - 1 - i] : -1;
  }
  // Four rows a thread: B is a multiple of 16, so a thread whose rows belong to
  // one request meets at most two blocks.
  for (long long t0 = 4LL * first; t0 < p.n_rows; t0 += 4LL * step) {
    int slot[4], pos[4];
    int r = t0 < total ? last_not_above(s_row, p.R, (int)t0) : 0;
    int c_known = -1;
    int blk = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = t0 + i;
      slot[i] = pos[i] = -1;
      if (t < total) {
        if (t >= s_row[r + 1]) {   // the next request with rows
          do ++r; while (t >= s_row[r + 1]);
          c_known = -1;
        }
        const int seq = s_seq[r];
        const uint32_t at = (uint32_t)seq + (uint32_t)(t - s_row[r]);
        const uint32_t c = at / (uint32_t)p.B;
        if ((int)c != c_known) {
          c_known = (int)c;
          blk = -1;
          const uint32_t have = blocks_of(seq, p.B);
          if (c < (uint32_t)p.max_blocks) {
            if (c < have) {
              blk = p.table[(size_t)r * p.max_blocks + c];
            } else {
              const long long k = s_blk[r] + (long long)(c - have);
              if (k < n_free) blk = p.free_blocks[n_free - 1 - k];
            }
          }
        }
        pos[i] = clamp_i32(at);
        if (blk >= 0) slot[i] = clamp_i32((long long)blk * p.B + (at - c * p.B));
      }
    }
    if (p.vec && t0 + 3 < p.n_rows) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < p.n_rows) {
          p.slots[t0 + i] = slot[i];
          p.positions[t0 + i] = pos[i];
        }
    }
  }
}

// ---- norm, rotation, cache write ------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;

struct AppendParams {
  bws_qkv in;
  bws_kv_cache c;
  uint16_t* q_out;
  int span;          // rows whose runs one key/value CTA writes, or one warp of it:
  int own_spans;
  int n_kv_ctas;     // spans * kv heads * 2, before the query CTAs
  int heads_per;     // query heads a warp takes of one row
  int solo_rows;     // the longest run that one warp takes
  int stage_rows;    // rows of a longer run kept in shared memory between the passes
};

// A head is held eight values a lane by D / 8 neighbouring lanes ("group"), so
// a warp works on 32 / (D / 8) rows at once and every load is 16 bytes.
template <int D>
struct Head {
  static constexpr int kLanes = D / 8;
  static constexpr int kRows = 32 / kLanes;
};

BWS_DEV void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int D>
BWS_DEV void norm_head(float (&x)[8], const float (&w)[8], float eps) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
  for (int o = Head<D>::kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = rsqrtf(s * (1.0f / D) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

// cos and sin of position * inv_freq[i] for a row's rot / 2 pairs, in turns:
// f = inv_freq / 2 pi as two FP32 parts (48 bits, formed once per warp), and
// only the turn's fraction is kept. Below 2^24 the position is exact in FP32:
// the high product is exact as a rounded product and its FMA remainder, so
// whole turns leave it before the parts are added. FP64 runs at about 2 a clock
// and SM here (formed that way, f alone held the FP64 pipe 73 % busy in a
// verify batch); only positions from 2^24 on take their product in it. Either
// way the fraction is off by a few 2^-24.
// sin and cos of 2 pi t, |t| <= 1/2: quarter turns off, then the Taylor series
// within an eighth of a turn (terms to x^9 and x^8: 2^-25 and below is left out),
// so that a key's rounding to E4M3 is its own and not the angle's. Half the
// instructions of sincospif; the fast pair (2^-21) moved ten times the codes
// across a midpoint.
BWS_DEV void sincos_turn(float t, float& s, float& c) {
  const float q = rintf(4.0f * t);
  const float x = (t - 0.25f * q) * 6.2831853071795865f, z = x * x;   // t - q / 4 is exact
  const float sx = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -1.6666667e-1f), x);
  const float cx = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 2.4801587e-5f, -1.3888889e-3f), 4.1666667e-2f), -0.5f), 1.0f);
  const int n = (int)q;
  s = (n & 1) ? cx : sx;
  c = (n & 1) ? sx : cx;
  if (n & 2) s = -s;
  if ((n + 1) & 2) c = -c;
}

// The turn of a far position: FP64, out of line so that nothing of it runs for near ones.
__device__ __noinline__ float far_turn(float f, int pos) {
  const double d = (double)f * 0.15915494309189533577 * (double)pos;
  return (float)(d - rint(d));
}

// How a head's pairs lie: (2 i, 2 i + 1); (i, i + half) with half a whole number
// of lanes' eights; any other half.
enum Pairs { kInterleaved, kSplitLanes, kSplitAny };

// A lane forms four of a row's angles: of the pairs it holds (interleaved), or
// half of the eight that it shares with the lane of the pairs' other halves, which
// a shuffle brings. Only kSplitAny takes them through shared memory: as a table
// there, read eight words apart by neighbouring lanes, they cost a round of keys
// 2500 cycles (a 628-row chunk at 256: 50 us, now 31). Where at most half of the
// head turns, the group's upper lanes form two of the lower lanes' four.
template <int D>
struct Angles {
  float fh[4], fl[4];

  static BWS_DEV bool helped(Pairs pairs, int half) { return pairs != kSplitAny && 4 * half <= D; }
  static BWS_DEV int pair_of(Pairs pairs, int k, int half, int sl) {
    if (helped(pairs, half) && sl >= Head<D>::kLanes / 2) {
      sl -= Head<D>::kLanes / 2;
      k += 2;
    }
    const int base = sl * 8;
    if (pairs == kInterleaved) return sl * 4 + k;
    if (pairs == kSplitLanes) return base < half ? base + k : base - half + 4 + k;
    return sl + k * Head<D>::kLanes;
  }
  BWS_DEV void init(const float* inv_freq, Pairs pairs, int half, int sl) {
    constexpr double kTurn = 0.15915494309189533577;      // 1 / 2 pi
    constexpr float kHi = (float)kTurn, kLo = (float)(kTurn - (double)kHi);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = pair_of(pairs, k, half, sl);
      const float f = i < half ? inv_freq[i] : 0.0f;
      fh[k] = f * kHi;
      fl[k] = fmaf(f, kLo, fmaf(f, kHi, -fh[k]));
    }
  }
  // c, s: of this lane's eight values, s with the sign that its partner's value
  // takes (interleaved: of its four pairs). cs: the group's table for kSplitAny.
  BWS_DEV void form(int pos, const float* inv_freq, Pairs pairs, int half, int sl, float2* cs, float (&c)[8],
                    float (&s)[8]) const {
    const int base = sl * 8;
    const bool help = helped(pairs, half);   // k = 2, 3 come from other lanes
    float t[4], u[4], v[4];
    if (pos < (1 << 24) && pos > -(1 << 24)) {
      const float fp = (float)pos;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k >= 2 && help) break;
        const float a = fh[k] * fp, e = fmaf(fh[k], fp, -a);
        t[k] = (a - rintf(a)) + fmaf(fl[k], fp, e);
        t[k] -= rintf(t[k]);
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int i = pair_of(pairs, k, half, sl);
        const float x = i < half ? far_turn(inv_freq[i], pos) : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = j == k ? x : t[j];
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= 2 && help) break;
      sincos_turn(t[k], v[k], u[k]);
    }
    if (help) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u[k + 2] = __shfl_down_sync(0xffffffffu, u[k], Head<D>::kLanes / 2);
        v[k + 2] = __shfl_down_sync(0xffffffffu, v[k], Head<D>::kLanes / 2);
      }
    }
    if (pairs == kInterleaved) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = u[k];
        s[k] = v[k];
      }
    } else if (pairs == kSplitLanes) {
      const bool low = base < half;
      const int partner = (threadIdx.x & 31) + (low ? half >> 3 : base < 2 * half ? -(half >> 3) : 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float pu = __shfl_sync(0xffffffffu, u[k], partner), pv = __shfl_sync(0xffffffffu, v[k], partner);
        c[k] = low ? u[k] : pu;
        s[k] = low ? -v[k] : pv;
        c[k + 4] = low ? pu : u[k];
        s[k + 4] = low ? -pv : v[k];
      }
    } else {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = sl + k * Head<D>::kLanes;
        if (i < half) cs[i] = make_float2(u[k], v[k]);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int d = base + k;
        const float2 a = d < 2 * half ? cs[d < half ? d : d - half] : make_float2(1.0f, 0.0f);
        c[k] = a.x;
        s[k] = d < half ? -a.y : a.y;
      }
    }
  }
};

// Rotates a head by its row's angles; buf: the group's own D floats for kSplitAny.
template <int D>
BWS_DEV void rotate_head(float (&x)[8], const float (&c)[8], const float (&s)[8], Pairs pairs, int half, float* buf,
                         int sl) {
  const int base = sl * 8, rot = 2 * half;
  if (pairs == kInterleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (base + 2 * k < rot) {
        const float u = x[2 * k], v = x[2 * k + 1];
        x[2 * k] = u * c[k] - v * s[k];
        x[2 * k + 1] = v * c[k] + u * s[k];
      }
    }
    return;
  }
  float y[8];
  if (pairs == kSplitLanes) {
    const int partner = (threadIdx.x & 31) + (base < half ? half >> 3 : base < rot ? -(half >> 3) : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], partner);
    if (base < rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + y[i] * s[i];
    }
    return;
  }
  __syncwarp();   // the last head's reads of buf are done
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[base + i] = x[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = base + i;
    if (d < rot) x[i] = x[i] * c[i] + buf[d < half ? d + half : d - half] * s[i];
  }
}


// e of the smallest 2^e with amax <= 448 * 2^e, in [-60, 60]; 448 = 1.75 * 2^8.
BWS_DEV int scale_exponent(float amax) {
  if (amax == 0.0f) return -60;
  const int x = floor_log2_abs(amax);
  const int e = amax > ldexp_exact(1.75f, x) ? x - 7 : x - 8;
  return min(max(e, -60), 60);
}

BWS_DEV void store_codes(uint8_t* p, const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = f32x2_to_e4m3x2(x[2 * i + 1] * inv, x[2 * i] * inv);
  *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Query warps take Head::kRows rows and heads_per heads of them, whose angles
// they form once. Key/value CTAs: one span of rows, one kv head, one side; each
// run of rows that starts in the span is normed and rotated, its largest
// magnitude found, and written under the scale that follows. Between the two
// passes the values wait in shared memory (of a run that is longer than it, the
// rest is formed again: the rows are in L1 by then). One rolled loop serves
// short and long runs: with the short ones unrolled in registers a quarter of
// the issue slots waited for instructions (a 12382-row chunk: 128 us, and 162
// with a CTA per run).
// Bound: launch and three dependent loads for a decoded token (one: 3.8 us; 48
// requests of five rows: 8.9 us, a serial run per warp). A 12382-row chunk at 64:
// 55 us for 127 MB, 2.3 TB/s: 20 % of DRAM and 52 % of the issue slots, so it is the
// latency of loads and dependent instructions at 21 warps an SM, which 80 registers
// and 64 KB of shared memory a CTA allow.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 3) append_kernel(const __grid_constant__ AppendParams p) {
  using Hd = Head<D>;
  constexpr int kStep = kAppendWarps * Hd::kRows;   // rows of a key/value CTA's round
  extern __shared__ __align__(16) float s_stage[];  // [stage_rows][D]
  __shared__ float s_amax[kAppendWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / Hd::kLanes, sl = lane % Hd::kLanes;
  const bws_qkv& in = p.in;
  const int half = in.rot >> 1;
  // a group's heads and angles, there where kSplitAny needs them
  float* const buf = s_stage + (p.stage_rows + warp * Hd::kRows + sub) * D;
  float2* const cs = reinterpret_cast<float2*>(s_stage + (p.stage_rows + (kAppendWarps + warp) * Hd::kRows + sub) * D);
  const Pairs pairs = in.interleaved ? kInterleaved : half % 8 == 0 ? kSplitLanes : kSplitAny;
  float cos_of[8], sin_of[8];
  pdl_launch_dependents();
  pdl_wait();
  Angles<D> angles;

  if ((int)blockIdx.x >= p.n_kv_ctas) {
    const int groups = (in.n_q_heads + p.heads_per - 1) / p.heads_per;
    const long long unit = (long long)(blockIdx.x - p.n_kv_ctas) * kAppendWarps + warp;
    const int row0 = (int)(unit / groups) * Hd::kRows, row = row0 + sub;
    if (row0 >= in.n_rows) return;
    const bool live = row < in.n_rows;
    const int h0 = (int)(unit % groups) * p.heads_per, h1 = min(h0 + p.heads_per, in.n_q_heads);
    const uint16_t* src = in.q + (live ? row : row0) * in.q_row_stride + sl * 8;
    uint4 raw = *reinterpret_cast<const uint4*>(src + h0 * in.q_head_stride);
    float w[8];
    if (in.q_weight != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = in.q_weight[sl * 8 + i];
    }
    if (half > 0) {
      const int pos = in.positions[live ? row : row0];
      angles.init(in.inv_freq, pairs, half, sl);
      angles.form(pos, in.inv_freq, pairs, half, sl, cs, cos_of, sin_of);
    }
    for (int h = h0; h < h1; ++h) {
      const uint4 now = raw;
      if (h + 1 < h1) raw = *reinterpret_cast<const uint4*>(src + (h + 1) * in.q_head_stride);
      float x[8];
      unpack8(now, x);
      if (in.q_weight != nullptr) norm_head<D>(x, w, in.eps);
      if (half > 0) rotate_head<D>(x, cos_of, sin_of, pairs, half, buf, sl);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (live)
        *reinterpret_cast<uint4*>(p.q_out + ((size_t)row * in.n_q_heads + h) * D + sl * 8) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
    return;
  }

  const bws_kv_cache& c = p.c;
  const int B = c.block_tokens, K = c.n_kv_heads;
  const int side = blockIdx.x & 1, head = (int)(blockIdx.x >> 1) % K;
  const int group = (int)((blockIdx.x >> 1) / K);
  const int t0 = (p.own_spans ? group * kAppendWarps + warp : group) * p.span, t1 = min(t0 + p.span, in.n_rows);
  const long long n_slots = (long long)c.n_blocks * B;
  const long long row_stride = side ? in.v_row_stride : in.k_row_stride;
  const uint16_t* src = (side ? in.v + head * in.v_head_stride : in.k + head * in.k_head_stride) + sl * 8;
  const bool normed = !side && in.k_weight != nullptr, turned = !side && half > 0;
  auto row_at = [&](int row) { return *reinterpret_cast<const uint4*>(src + min(row, in.n_rows - 1) * row_stride); };
  auto pos_at = [&](int row) { return turned ? in.positions[min(row, in.n_rows - 1)] : 0; };
  float w[8];
  if (normed) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = in.k_weight[sl * 8 + i];
  }
  if (turned) angles.init(in.inv_freq, pairs, half, sl);
  auto form = [&](const uint4& raw, int pos, float (&x)[8]) {
    unpack8(raw, x);
    if (normed) norm_head<D>(x, w, in.eps);
    if (turned) {
      angles.form(pos, in.inv_freq, pairs, half, sl, cs, cos_of, sin_of);
      rotate_head<D>(x, cos_of, sin_of, pairs, half, buf, sl);
    }
  };

  // The runs that start in the span, in order. Where the CTA shares it, every
  // warp finds them all; a short one is a warp's alone, with no barrier; a long
  // one is the whole CTA's.
  int turn = 0;   // short runs so far
  for (int t = t0; t < t1; t += 31) {
    // rows t - 1 .. t + 30's slots, a lane each
    const int at = t - 1 + lane;
    const int window = at >= 0 && at < in.n_rows ? in.slots[at] : -2;
    const int before = __shfl_up_sync(0xffffffffu, window, 1);
    const bool live = window >= 0 && window < n_slots;
    const bool fresh = !live || window % B == 0 || before != window - 1;   // not the next row of a run
    const unsigned breaks = __ballot_sync(0xffffffffu, fresh);
    unsigned starts = __ballot_sync(0xffffffffu, fresh && live && lane > 0 && at < t1);
    while (starts != 0u) {
      const int j = __ffs(starts) - 1;
      starts &= starts - 1;
      const int row = t - 1 + j;   // the run's first
      const int slot = __shfl_sync(0xffffffffu, window, j);
      const int off = slot % B, room = B - off, block = slot / B;
      const unsigned next = j < 31 ? breaks >> (j + 1) : 0u;
      int m = next != 0u ? __ffs(next) : 32 - j;
      if (next == 0u) {   // past the window
        while (m < room) {
          const int i = m + lane;
          const bool on = i < room && row + i < in.n_rows && in.slots[row + i] == slot + i;
          const unsigned b = __ballot_sync(0xffffffffu, on);
          const int n = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
          m += n;
          if (n < 32) break;
        }
      }
      float* scale_at = (side ? c.v_scale : c.k_scale) + (size_t)block * K + head;
      const bool solo = p.own_spans || m <= p.solo_rows;
      if (solo && !p.own_spans && turn++ % kAppendWarps != warp) continue;
      const int step = solo ? Hd::kRows : kStep, mine = (solo ? 0 : warp * Hd::kRows) + sub;
      float* const stage = s_stage + (solo ? warp * p.solo_rows * D : 0) + sl * 8;
      const int staged = solo ? p.solo_rows : p.stage_rows;
      if (!solo) __syncthreads();   // a warp may still read a short run's values where this one's will lie
      const float old = *scale_at;
      float amax = 0.0f;
      uint4 raw = row_at(row + mine);
      int pos = pos_at(row + mine);
#pragma unroll 1
      for (int i0 = 0; i0 < m; i0 += step) {
        const int i = i0 + mine;
        const uint4 now = raw;
        const int here = pos;
        if (i0 + step < m) {
          raw = row_at(row + i + step);
          pos = pos_at(row + i + step);
        }
        float x[8];
        form(now, here, x);
        if (i < m) {
          float top = 0.0f;   // NaN and infinity set no scale
#pragma unroll
          for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
          if (top == INFINITY) {
            top = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fabsf(x[k]) < INFINITY ? fmaxf(top, fabsf(x[k])) : top;
          }
          amax = fmaxf(amax, top);
          if (i < staged) {
            float4* st = reinterpret_cast<float4*>(stage + i * D);
            st[0] = make_float4(x[0], x[1], x[2], x[3]);
            st[1] = make_float4(x[4], x[5], x[6], x[7]);
          }
        }
      }
      amax = warp_max(amax);
      if (!solo) {
        if (lane == 0) s_amax[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAppendWarps; ++i) amax = fmaxf(amax, s_amax[i]);
      }
      const float need = exp2i(scale_exponent(amax));
      const float scale = off == 0 ? need : fmaxf(old, need), inv = 1.0f / scale;
      uint8_t* codes = (side ? c.v : c.k) + (size_t)block * c.block_stride + (size_t)head * c.head_stride;
      if (off != 0 && scale != old) {   // the scale grew: the block's earlier codes again, under it
        const float f = old / scale;
        uint32_t* w32 = reinterpret_cast<uint32_t*>(codes);
        for (int i = solo ? lane : threadIdx.x; i < off * (D / 4); i += solo ? 32 : kAppendThreads) {
          uint32_t lo, hi;
          e4m3x4_to_f16x2x2(w32[i], lo, hi);
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          w32[i] = f32x2_to_e4m3x2(a.y * f, a.x * f) | (f32x2_to_e4m3x2(b.y * f, b.x * f) << 16);
        }
      }
      uint8_t* dst = codes + (size_t)off * D + sl * 8;
      const int kept = min(m, staged);
      for (int i = mine; i < kept; i += step) {
        const float4* st = reinterpret_cast<const float4*>(stage + i * D);
        const float4 a = st[0], b = st[1];
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        store_codes(dst + (size_t)i * D, x, inv);
      }
#pragma unroll 1
      for (int i0 = staged; i0 < m; i0 += step) {   // staged is a multiple of step
        const int i = i0 + mine;
        float x[8];
        form(row_at(row + i), pos_at(row + i), x);
        if (i < m) store_codes(dst + (size_t)i * D, x, inv);
      }
      if (solo) __syncwarp();   // every thread has read the old scale, and s_amax
      else __syncthreads();
      if (solo ? lane == 0 : threadIdx.x == 0) *scale_at = scale;
    }
  }
}

template <int D>
cudaError_t launch_append(unsigned grid, size_t smem, cudaStream_t st, const AppendParams& p) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, append_kernel<D>, kAppendWarps * 10 * 256 * 4);
  return e != cudaSuccess ? e : launch_pdl(append_kernel<D>, dim3(grid), kAppendThreads, smem, st, p);
}

}  // namespace

int check_kv_cache(const bws_kv_cache* c, const char* name) {
  if (c == nullptr) return fail(BWS_ERR_INVALID_ARG, "%s: null cache", name);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: head_dim = %d must be 64, 128 or 256", name, c->head_dim);
  if (c->block_tokens < 16 || c->block_tokens > 256 || c->block_tokens % 16 != 0)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: block_tokens = %d must be a multiple of 16 in [16, 256]", name,
                c->block_tokens);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 128)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: n_kv_heads = %d must be in [1, 128]", name, c->n_kv_heads);
  if (c->n_blocks < 1 || (long long)c->n_blocks * c->block_tokens >= (1LL << 31))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: n_blocks = %d (1 or more, below 2^31 tokens)", name, c->n_blocks);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return fail(BWS_ERR_INVALID_ARG, "%s: null cache pointer", name);
  const size_t rows = (size_t)c->block_tokens * c->head_dim;
  if (c->block_stride % 16 || c->head_stride % 16 || !aligned(c->k, 16) || !aligned(c->v, 16) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: cache codes and strides 16-byte, scales 4-byte alignment needed", name);
  // blocks and heads must not overlap: [blocks][heads] or [heads][blocks] order
  const bool by_block = c->head_stride >= rows && c->block_stride >= c->head_stride * (c->n_kv_heads - 1) + rows;
  const bool by_head = c->block_stride >= rows && c->head_stride >= c->block_stride * ((size_t)c->n_blocks - 1) + rows;
  if (!(by_block || by_head) || c->block_stride >= (1ull << 40) || c->head_stride >= (1ull << 40))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: cache strides (%zu, %zu) overlap or are out of range", name,
                c->block_stride, c->head_stride);
  return BWS_OK;
}

}  // namespace bws

extern "C" {

int bws_kv_plan(const int32_t* seq_lens, const int32_t* new_lens, int n_requests, int block_tokens,
                int32_t* block_table, int max_blocks, const int32_t* free_blocks, const int32_t* n_free, int n_rows,
                int32_t* slots, int32_t* positions, int32_t* row_start, int32_t* kv_lens, int32_t* n_free_out,
                int32_t* status, void* stream) {
  return bws_kv_plan_bounded(seq_lens, new_lens, n_requests, block_tokens, block_table, max_blocks, free_blocks,
                             INT32_MAX, n_free, n_rows, slots, positions, row_start, kv_lens, n_free_out, status, stream);
}

int bws_kv_plan_bounded(const int32_t* seq_lens, const int32_t* new_lens, int n_requests, int block_tokens,
                        int32_t* block_table, int max_blocks, const int32_t* free_blocks, int n_list,
                        const int32_t* n_free, int n_rows, int32_t* slots, int32_t* positions, int32_t* row_start,
                        int32_t* kv_lens, int32_t* n_free_out, int32_t* status, void* stream) {
  using namespace bws;
  const char* name = "bws_kv_plan";
  if (n_requests < 0 || n_requests > kPlanMaxRequests)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_requests = %d must be in [0, %d]", name, n_requests, kPlanMaxRequests);
  if (n_rows < 0 || max_blocks < 0 || n_list < 0)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d, max_blocks = %d, n_list = %d", name, n_rows, max_blocks, n_list);
  if (block_tokens < 16 || block_tokens > 256 || block_tokens % 16 != 0)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: block_tokens = %d must be a multiple of 16 in [16, 256]", name,
                block_tokens);
  if (!n_free || !row_start || !n_free_out || !status || (n_requests > 0 && (!seq_lens || !new_lens || !kv_lens)) ||
      (n_requests > 0 && max_blocks > 0 && !block_table) || (n_rows > 0 && (!slots || !positions)))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (n_free == n_free_out) return fail(BWS_ERR_INVALID_ARG, "%s: n_free_out must not be n_free", name);
  const void* ptrs[] = {seq_lens, new_lens, block_table, free_blocks, n_free, slots, positions, row_start, kv_lens,
                        n_free_out, status};
  for (const void* q : ptrs)
    if (!aligned(q, 4)) return fail(BWS_ERR_MISALIGNED, "%s: 4-byte alignment needed", name);
  // CTAs read every length while another writes kv_lens
  if (n_requests > 0 && (kv_lens == seq_lens || kv_lens == new_lens))
    return fail(BWS_ERR_INVALID_ARG, "%s: kv_lens must not be seq_lens or new_lens", name);
  if (free_blocks == nullptr) n_list = 0;   // an empty list has no address
  PlanParams p = {seq_lens, new_lens, n_requests, block_tokens, block_table, max_blocks, free_blocks, n_list, n_free,
                  n_rows, slots, positions, row_start, kv_lens, n_free_out, status,
                  aligned(slots, 16) && aligned(positions, 16)};
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, plan_kernel, (int)sizeof(int) * (3 * kPlanMaxRequests + 2));
  if (e != cudaSuccess) return cuda_status(e, name);
  // four rows a thread, up to two CTAs an SM
  const long long want = ((long long)n_rows + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  const long long most = 2LL * num_sms();
  const unsigned grid = (unsigned)(want < 1 ? 1 : want > most ? most : want);
  return cuda_status(launch_pdl(plan_kernel, dim3(grid), kPlanThreads, sizeof(int) * (3 * (size_t)n_requests + 2),
                                as_stream(stream), p), name);
}

int bws_qk_norm_rope_append(const bws_qkv* in, const bws_kv_cache* cache, uint16_t* q_out, void* stream) {
  using namespace bws;
  const char* name = "bws_qk_norm_rope_append";
  if (in == nullptr) return fail(BWS_ERR_INVALID_ARG, "%s: null input", name);
  const int rc = check_kv_cache(cache, name);
  if (rc) return rc;
  const int D = cache->head_dim, K = cache->n_kv_heads, H = in->n_q_heads;
  if (in->n_rows < 0 || H < 1 || H > 1024)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d, n_q_heads = %d (1..1024)", name, in->n_rows, H);
  if (in->rot < 0 || in->rot > D || in->rot % 2)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: rot = %d must be even and at most head_dim", name, in->rot);
  if (in->n_rows == 0) {
    clear_error();
    return BWS_OK;
  }
  if (!in->q || !in->k || !in->v || !in->positions || !in->slots || !q_out || (in->rot > 0 && !in->inv_freq))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!(in->eps >= 0.0f)) return fail(BWS_ERR_INVALID_ARG, "%s: eps must not be negative", name);
  if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(q_out, 16) ||
      !aligned(in->positions, 4) || !aligned(in->slots, 4) || !aligned(in->inv_freq, 4) ||
      !aligned(in->q_weight, 4) || !aligned(in->k_weight, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: rows 16-byte, other pointers 4-byte alignment needed", name);
  const int64_t strides[] = {in->q_row_stride, in->q_head_stride, in->k_row_stride,
                             in->k_head_stride, in->v_row_stride, in->v_head_stride};
  for (int64_t s : strides)
    if (s % 8 != 0) return fail(BWS_ERR_MISALIGNED, "%s: strides must be multiples of 8 elements", name);
  AppendParams p;
  p.in = *in;
  p.c = *cache;
  p.q_out = q_out;
  const long long sms = num_sms();
  // Where the blocks alone are work for eight warps an SM, every warp takes a
  // span of its own, a block long. Else a CTA's warps share one: eight rows at
  // least, which in a decode batch are a run for each.
  const long long rows = in->n_rows, B = cache->block_tokens;
  p.own_spans = rows * K * 2 >= sms * 8 * B;
  long long span = p.own_spans ? B : rows * K * 2 / (sms * 4);
  span = span < kAppendWarps ? kAppendWarps : span > kAppendWarps * B ? kAppendWarps * B : span;
  p.span = (int)span;
  const long long per_cta = p.own_spans ? span * kAppendWarps : span;
  const long long spans = (rows + per_cta - 1) / per_cta;
  const long long kv_ctas = spans * K * 2;
  // heads of a row that share a warp's angles, as long as every SM keeps 8 warps
  const long long row_groups = (rows + 256 / D - 1) / (256 / D);
  long long per = row_groups * H / (sms * 8);
  per = per < 1 ? 1 : per > 8 ? 8 : per;
  p.heads_per = (int)per;
  const long long groups = (H + per - 1) / per;
  const long long q_ctas = (row_groups * groups + kAppendWarps - 1) / kAppendWarps;
  if (kv_ctas + q_ctas >= (1LL << 31)) return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: too many rows", name);
  p.n_kv_ctas = (int)kv_ctas;
  // A warp takes runs of up to eight rounds where the rows are many, two where
  // a run's other warps would have nothing to do.
  const int round = 256 / D;
  p.solo_rows = round * (rows * K * 2 >= sms * 16 ? 8 : 2);
  p.stage_rows = kAppendWarps * p.solo_rows;
  const bool pair_buffer = !in->interleaved && (in->rot / 2) % 8 != 0;
  const size_t smem = (size_t)p.stage_rows * D * 4 + (pair_buffer ? 2 * kAppendWarps * 256 * 4 : 0);
  const unsigned grid = (unsigned)(kv_ctas + q_ctas);
  cudaStream_t st = as_stream(stream);
  cudaError_t e;
  if (D == 64) e = launch_append<64>(grid, smem, st, p);
  else if (D == 128) e = launch_append<128>(grid, smem, st, p);
  else e = launch_append<256>(grid, smem, st, p);
  return cuda_status(e, name);
}

}  // extern "C"

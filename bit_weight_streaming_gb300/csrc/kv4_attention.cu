// Attention of a step's 1..8 rows per request over the 4-bit cache. Contract in
// include/bws.h.
//
// Mathematics. As over the 8-bit cache (kv_attention.cu): S^T = K Q^T, O^T = V^T P^T on
// m16n8k16 with f16 operands and FP32 sums, cached tokens and dimensions on the M
// side. An E2M1 code times its E4M3 scale has at most six significant bits and lies
// within f16's reach, so keys and values are exact operands; the heads' FP32 numbers
// are taken into the scale of the scores and out of the sum. A query row is scaled by
// a power of two. With x the score times log2(e), w = 2^(x - m), m about the running
// maximum, out = g_v sum w v / sum w: a weight is rounded to f16, the sum of weights
// takes them unrounded.
//
// Work. The line of units and its shares are kv_attention.cuh's. A unit is U boxes of
// 16 cached tokens, so that every unit is 2 KB of codes and 256 bytes of scales a
// side where registers allow. A warp copies its units into a ring of its own with
// cp.async, 16 bytes a lane, rows swizzled so that ldmatrix meets every bank once.
//
// Bound. A token's head is 9/16 of the 8-bit cache's bytes and costs a conversion of
// every code and a product with its scale besides: over long contexts the issue slots
// (55 to 62 %) and HBM (4.4 to 4.9 TB/s over the call) are both near what a chain of
// dependent steps a warp allows. 131071 tokens, 4 heads of 256: 34.5 us, 25 of them the
// stream, the rest the line's start, the first copies and the join; 80 requests of up
// to 9001 tokens, 8 heads of 128: 86.6 us, 0.72 of the copy rate; 24 requests of up to 5
// rows, 16 heads of 64: 29 us, 0.40, a third of it segments' starts and ends. Kept step by
// step: addresses formed once a box, scales converted once a unit, codes of two tokens
// paired before their conversion, the next segment's first units and queries asked for
// before the join: 119 -> 85 us for the 80 requests.
#include <string.h>

#include <algorithm>
#include <atomic>

#include "device_counts.h"
#include "kv4_attention.cuh"
#include "kv4_cache.cuh"
#include "kv_cache.cuh"
#include "stream_tile.cuh"

namespace bws {
namespace {

template <int D, int NT, bool kMany>
struct Shape4 {
  static constexpr bool kNarrow = NT == 1;
  // Up to eight rows: registers for two CTAs of eight warps an SM, or one of twelve at 256
  // dimensions (131071 tokens: 34.9 us; one of eight 37.0, two of eight 37.9).
  // Of many segments smaller CTAs, and more of them, so that the others' units pass while
  // one ends and another starts (300 requests of 120 tokens, 8 heads of 128: 34.5 -> 21.6
  // us; of 60 tokens, 4 of 256: 35 -> 18.3; 200 of up to 900, 16 of 64: 58 -> 43; 224
  // segments of 16 rows of 256: 9.3 -> 11.3).
  static constexpr int kWarps = kMany ? 4 : kNarrow && D == 256 ? 12 : 8;
  static constexpr int kOnce = kNarrow ? (D == 256 ? 1 : 2) : NT * D <= 128 ? 2 : 1;
  static constexpr int kCtas = !kMany ? kOnce : kNarrow && D == 256 ? 3 : 2 * kOnce;
  static constexpr int kBoxes = (D == 64 && NT <= 2) || (D == 128 && NT == 1) ? 2 : 1;   // boxes of a unit
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = kBoxes * kBox;
  static constexpr int kBoxCodes = kBox * D / 2, kBoxScales = kBox * D / 16;   // bytes a side
  static constexpr int kCodes = kBoxes * kBoxCodes, kScales = kBoxes * kBoxScales;
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kRows = 8 * NT;
  // A warp's O in FP32, at the segment's end, lies in the ring's first stages; the
  // next segment's units begin behind them.
  static constexpr int kJoinRow = D + 4;     // floats: eight rows of a store on all banks
  static constexpr int kJoin = kRows * kJoinRow * 4;
  static constexpr int kRoom = (kCtas == 4 ? 51 : kCtas == 3 ? 68 : kCtas == 2 ? 104 : 206) * 1024 / kWarps;
  static constexpr int kFit = kRoom / kStage, kLeast = kJoin / kStage + 1;
  static constexpr int kStages = kFit > 8 ? (kLeast > 8 ? kLeast : 8) : kFit;
  static constexpr int kJoinStages = (kJoin + kStage - 1) / kStage;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kAhead = kStages - 1;                                  // units asked for beyond the one in work
  static constexpr int kEarly = kStages - kJoinStages < kAhead ? kStages - kJoinStages : kAhead;   // of them before the join
  // Query fragments stay in registers where these allow it (kept at 128 dimensions and up
  // to eight rows, 80 requests took 88 us, not 85).
  static constexpr bool kQInRegs = kNarrow ? D == 64 : NT * D <= 256;
  static constexpr int kQStride = 2 * D + 64;                 // bytes of a query row: fragments of two rows on all banks
  static_assert(kStages >= 2 && kRing >= kJoin && kStages <= 32, "ring");
};

template <int D, int NT, bool kMany>
struct __align__(16) Tail4 {
  static constexpr int kWarps = Shape4<D, NT, kMany>::kWarps;
  uint8_t q[8 * NT * Shape4<D, NT, kMany>::kQStride];
  float q_scale[8 * NT];
  float m[kWarps][8 * NT];
  float l[kWarps][8 * NT];
  float2 spread_ml[8 * NT];       // this CTA's, where a segment is a cluster's
  uint32_t nan_mask[2][D / 16];   // bit j: token j of the rows' own has a NaN there
  // A warp's unit's scales in f16: the keys' by token, half of a chunk and chunk; the
  // values' by half, pair of tokens and chunk, the pair's two side by side.
  alignas(16) uint32_t scales[kWarps][Shape4<D, NT, kMany>::kBoxes * D];
  uint32_t there[kWarps][Shape4<D, NT, kMany>::kStages];      // by stage: which boxes of the unit are in the cache
  long long line_warp[kWarps];
  long long line_found[2];
  // The CTA's way along its share, kept here by thread 0, and its segments: this
  // one, the next, and the one that is looked for at this one's end.
  Walk walk;
  Segment seg[3];
  int more[3];
  uint32_t status;
};

// 16 bytes global -> shared, zeros where `there` is false; an L2 policy.
BWS_DEV void copy16(uint32_t dst, const void* src, bool there, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;"
               :: "r"(dst), "l"(src), "r"(there ? 16u : 0u), "l"(pol) : "memory");
}

BWS_DEV void sts_pair(uint32_t at, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" :: "r"(at), "r"(a), "r"(b) : "memory");
}

// A unit's scales to f16, once for the warp (every fragment's own lanes would form
// each of them two to four times, and a conversion takes as long as two others): of
// UD bytes a side, eight of the keys' and a word of two tokens of the values' a lane.
template <int D, int U>
BWS_DEV void convert_scales(uint32_t k_at, uint32_t v_at, uint32_t to, int lane) {
  constexpr int kWords = D / 64;   // of a token
  if (U * D >= 256 || lane < U * D / 8) {
    uint32_t w[2], h[2][2];   // [word][half]
    lds_words<2>(k_at + 8 * lane, w);
#pragma unroll
    for (int i = 0; i < 2; ++i) e4m3x4_to_f16x2x2(__byte_perm(w[i], 0, 0x3120), h[i][0], h[i][1]);
    if constexpr (D == 64) {   // two tokens
      sts_pair(to + 16 * lane, h[0][0], h[0][1]);
      sts_pair(to + 16 * lane + 8, h[1][0], h[1][1]);
    } else {
      constexpr int kPairs = kWords / 2;   // of a token's words
      const uint32_t at = to + (lane / kPairs) * (D / 8) + (lane % kPairs) * 8;
      sts_pair(at, h[0][0], h[1][0]);
      sts_pair(at + D / 16, h[0][1], h[1][1]);
    }
  }
  if (U * D >= 256 || lane < U * D / 8) {
    const int pair = lane / kWords, word = lane % kWords;
    uint32_t a, b, h[4];
    lds_words<1>(v_at + 2 * pair * (D / 16) + word * 4, &a);
    lds_words<1>(v_at + (2 * pair + 1) * (D / 16) + word * 4, &b);
    e4m3x4_to_f16x2x2(__byte_perm(a, b, 0x6240), h[0], h[1]);
    e4m3x4_to_f16x2x2(__byte_perm(a, b, 0x7351), h[2], h[3]);
    const uint32_t at = to + U * 2 * D + pair * (D / 8) + word * 8;
    sts_pair(at, h[0], h[1]);
    sts_pair(at + U * D, h[2], h[3]);
  }
}

constexpr int kMaxSpread = 8;   // CTAs of a cluster
BWS_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release; barrier.cluster.wait.acquire;" ::: "memory");
}
BWS_DEV uint32_t peer_addr(uint32_t at, int cta) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(cta));
  return r;
}
BWS_DEV float2 peer_float2(uint32_t at, int cta) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_addr(at, cta)) : "memory");
  return v;
}
BWS_DEV float4 peer_float4(uint32_t at, int cta) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_addr(at, cta)) : "memory");
  return v;
}

// Four dimensions of a row's result, from the sums of a whole segment.
template <int D>
BWS_DEV void store_result(const AttnLine& p, size_t at, int d, const float4& a, float top, float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  *reinterpret_cast<uint2*>(p.out + at * D + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse != nullptr && d == 0) p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The CTAs of a y row of the join: what the first row's do in kv_attention.cu.
template <int D>
BWS_DEV void clear_and_report(const AttnLine& p) {
  __shared__ uint32_t s_bad;
  const int begin = p.row_start[0], end = p.row_start[p.R];
  const bool excess = (p.failed[0] & BWS_STATUS_KV_ROWS) != 0u;   // every CTA says it
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_ctas; i += blockDim.x)
      if (p.failed[i] != 0) atomicOr(&s_bad, p.failed[i]);
    __syncthreads();
    if (threadIdx.x == 0) {
      p.hdr[0] = 0;
      p.hdr[1] = s_bad;
    }
  }
  if (begin > 0 || end < p.n_rows || excess) clear_rows<D>(p, begin, end, excess, blockIdx.x, gridDim.x);
}

// The same where there is no join.
template <int D>
BWS_DEV void clear_direct(const AttnLine& p, int cta, int n_ctas) {
  bool many = false;
  for (int r = threadIdx.x; r < p.R; r += blockDim.x) many |= request_of(p, r, p.group_rows).all > p.max_rows;
  const bool excess = __syncthreads_or(many) != 0;
  const int begin = p.row_start[0], end = p.row_start[p.R];
  if (cta == 0 && threadIdx.x == 0) {
    p.hdr[0] = 0;
    p.hdr[1] = excess ? (uint32_t)BWS_STATUS_KV_ROWS : 0u;
  }
  if (begin > 0 || end < p.n_rows || excess) clear_rows<D>(p, begin, end, excess, cta, n_ctas);
}

template <int D, int NT, bool kMany>
__global__ void __launch_bounds__(Shape4<D, NT, kMany>::kThreads, Shape4<D, NT, kMany>::kCtas) attn4_kernel(const __grid_constant__ Attn4Params p) {
  using S = Shape4<D, NT, kMany>;
  constexpr int U = S::kBoxes, W = S::kWarps;
  constexpr int kMT = D / 16;      // m tiles of O^T
  constexpr int kChunks = D / 32;  // 16-byte chunks of a token's codes
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (base - smem_u32(smem_raw));   // rings, then the warps' O, then the tail
  Tail4<D, NT, kMany>& T = *reinterpret_cast<Tail4<D, NT, kMany>*>(smem + S::kRing * W);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = base + warp * S::kRing;
  float* const join = reinterpret_cast<float*>(smem);
  constexpr int kJoinStep = S::kRing / 4;    // floats from warp to warp
  constexpr int kFirstStage = S::kJoinStages % S::kStages;   // of a segment's first unit
  if (tid == 0) T.status = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int cta = blockIdx.x;
  if (p.direct) {
    if (cta >= p.direct) {
      clear_direct<D>(p, cta - p.direct, gridDim.x - p.direct);
      return;
    }
    if (tid == 0) {
      Segment& sg = T.seg[0];
      const int segment = cta / p.spread, rank = cta - segment * p.spread;
      const int per = p.K * p.max_groups, in = segment % per;
      sg.r = segment / per;
      sg.rq = request_of(p, sg.r, S::kRows);
      sg.head = in / p.max_groups;
      sg.row0 = (in - sg.head * p.max_groups) * S::kRows;
      const int share = (sg.rq.units + p.spread - 1) / p.spread;
      sg.first = min(rank * share, sg.rq.units);
      sg.last = min(sg.first + share, sg.rq.units);
      sg.whole = sg.starts = true;
      sg.pieces = 1;
      T.more[0] = sg.row0 < sg.rq.rows(p) * p.G;
      T.more[1] = 0;
    }
  } else if (p.R <= 32) {
    if (warp == 0) {
      Walk walk;
      const bool excess = start_small(p, S::kRows, walk);
      if (lane == 0) {
        if (excess) T.status = BWS_STATUS_KV_ROWS;
        T.more[0] = walk.next(p, S::kRows, T.seg[0]);
        T.walk = walk;
      }
    }
  } else {
    Walk walk;
    walk.start(p, S::kRows, T.line_warp, T.line_found, &T.status);
    if (tid == 0) {
      T.more[0] = walk.next(p, S::kRows, T.seg[0]);
      T.walk = walk;
    }
  }
  __syncthreads();
  const uint64_t pol = l2_evict_first();
  // this lane's ldmatrix row: tokens 0-7 and 8-15 of one chunk, then of the next
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lchunk = lane >> 4;

  const uint32_t sc16 = smem_u32(T.scales[warp]);

  int turn = 0;   // of T.seg
  // ---- copies: 32 boxes of the warp's units (first + warp, + W, ...) at a time, a box
  // a lane: where its codes and scales lie, -1: not there. The next 32 boxes'
  // blocks are asked for half a batch ahead.
  constexpr int kBatch = 32 / U;   // units
  int mine, tok_first;             // this warp's units; the first one's first token
  long long code_at, scale_at;
  int next_block, next_tok;
  const uint8_t *k_src, *v_src, *s_src;   // this lane's place in a box
  constexpr int kScaleChunks = S::kScales / 16, kBoxScaleChunks = S::kBoxScales / 16;
  static_assert(kScaleChunks <= 16, "scales of a side in half a warp");
  const int s_chunk = lane & 15, s_box = min(s_chunk / kBoxScaleChunks, U - 1);
  const uint32_t c_dst = codes_at<D>(lane / kChunks, lane % kChunks);
  auto look_up = [&](int i0) {   // asks for the blocks of units i0 .. i0 + kBatch - 1
    const Segment& sg = T.seg[turn];
    const int i = i0 + lane / U;
    const uint32_t t = (uint32_t)tok_first + (uint32_t)i * (S::kUnit * W) + lane % U * kBox;
    next_block = -1;
    next_tok = 0;
    if (i < mine && t < (uint32_t)sg.rq.kv(p)) {
      const int q = block_index(p, (int)t);
      next_block = p.table[(size_t)sg.r * p.max_blocks + q];
      next_tok = (int)t - q * p.B;
    }
  };
  auto take_batch = [&]() {
    const bool there = next_block >= 0 && next_block < p.n_blocks;
    code_at = there ? next_block * p.block_stride + next_tok * (D / 2) : -1;
    scale_at = there ? next_block * p.scale_block_stride + next_tok * (D / 16) : -1;
  };
  auto issue = [&](int i, int s) {   // the whole warp; unit i of this warp into stage s
    const int in = i % kBatch, from = in * U;
    if (in == 0 && i > 0) take_batch();
    if (in == kBatch / 2) look_up(i - in + kBatch);
    const uint32_t dst = ring + s * S::kStage;
    uint32_t there = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = __shfl_sync(0xffffffffu, code_at, from + u);
      const bool is = at >= 0;
      there |= (is ? 1u : 0u) << u;
      const uint8_t *k = k_src + (is ? at : 0), *v = v_src + (is ? at : 0);
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {   // (16 chunk columns on, the swizzle of 256 dimensions turns once)
        const uint32_t to = dst + u * S::kBoxCodes + ((D == 256 && (j & 1) ? c_dst ^ 64u : c_dst) + j * 512);
        copy16(to, k + j * 512, is, pol);
        copy16(to + S::kCodes, v + j * 512, is, pol);
      }
    }
    const long long at = __shfl_sync(0xffffffffu, scale_at, from + s_box);
    if (s_chunk < kScaleChunks)   // the lower lanes the keys', the upper ones the values'
      copy16(dst + 2 * S::kCodes + (lane >> 4) * S::kScales + s_chunk * 16, s_src + (at >= 0 ? at : 0), at >= 0, pol);
    if (lane == 0) T.there[warp][s] = there;
  };
  // A segment's start, in two steps, so that block ids and query rows are on
  // their way while the segment before is joined.
  constexpr int kOwnRows = (S::kRows + W - 1) / W;   // of a warp
  uint32_t qx[kOwnRows][D / 64];   // dimensions 2 lane + 64 i and the next, BF16
  float g_k, g_v;
  auto ask_queries = [&](const Segment& sg) {
    const int n_rows = min(sg.rq.rows(p) * p.G - sg.row0, S::kRows);
#pragma unroll
    for (int k = 0; k < kOwnRows; ++k) {
      const int n = warp + k * W;
      if (n < n_rows) {
        const int j = (sg.row0 + n) / p.G, h = sg.head * p.G + (sg.row0 + n) % p.G;
        const uint16_t* src = p.q + (sg.rq.start + j) * p.q_row_stride + h * p.q_head_stride + 2 * lane;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) qx[k][i] = *reinterpret_cast<const uint32_t*>(src + 64 * i);
      } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) qx[k][i] = 0;
      }
    }
  };
  auto ask_segment = [&]() {
    const Segment& sg = T.seg[turn];
    const int head = sg.head;
    mine = (sg.last - sg.first - warp + W - 1) / W;
    tok_first = (int)((uint32_t)(sg.first + warp) * S::kUnit);
    look_up(0);
    g_k = p.k_global != nullptr ? p.k_global[head] : 1.0f;
    g_v = p.v_global != nullptr ? p.v_global[head] : 1.0f;
    k_src = p.k + head * p.head_stride + lane * 16;
    v_src = p.v + head * p.head_stride + lane * 16;
    s_src = (lane < 16 ? p.k_scale : p.v_scale) + head * p.scale_head_stride + s_chunk % kBoxScaleChunks * 16;
  };
  // The first units' copies, a group each, empty ones too: units from .. to - 1.
  auto open_units = [&](int from, int to) {
#pragma unroll 1
    for (int i = from; i < to; ++i) {
      if (i < mine) issue(i, kFirstStage + i < S::kStages ? kFirstStage + i : kFirstStage + i - S::kStages);
      cp_async_commit();
    }
  };
  // The query rows to f16, each scaled by a power of two; clears a NaN mask. A row that
  // holds an infinity is all NaN: its scores are none, but of keys of one sign there they
  // would all be -infinity, which is what tokens that a row does not see get.
  auto store_queries = [&](int slot) {
#pragma unroll
    for (int k = 0; k < kOwnRows; ++k) {
      const int n = warp + k * W;
      if (n >= S::kRows) break;
      __half2* dst = reinterpret_cast<__half2*>(T.q + n * S::kQStride);
      float x[D / 32];
      float top = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = __uint_as_float(i % 2 ? qx[k][i / 2] & 0xFFFF0000u : qx[k][i / 2] << 16);
        if (fabsf(x[i]) < INFINITY) top = fmaxf(top, fabsf(x[i]));
        else bad = true;
      }
      bad = __any_sync(0xffffffffu, bad);
      top = warp_max(top);
      const int e = top > 0.0f ? min(max(floor_log2_abs(top), -100), 126) : 0;
      const float f = exp2i(-e);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) dst[lane + 32 * i] = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
      if (lane == 0) T.q_scale[n] = bad ? NAN : p.scale * kLog2e * exp2i(e);
    }
    if (tid < D / 16) T.nan_mask[slot][tid] = 0;
  };

  bool more = T.more[0] != 0;
  const bool spread = more && p.spread > 1;
  int nan_slot = 0;
  if (more) {
    ask_segment();
    ask_queries(T.seg[0]);
    take_batch();
    open_units(0, S::kEarly);
    store_queries(0);
    if (tid == 0 && !p.direct) T.more[1] = T.walk.next(p, S::kRows, T.seg[1]);
  }
  while (more) {
    __syncthreads();
    open_units(S::kEarly, S::kAhead);   // where the last segment's O lay
    const Segment& cur = T.seg[turn];
    const int after = turn == 2 ? 0 : turn + 1;
    constexpr bool kAskEarly = NT * D <= 256;   // where the registers allow: their latency passes beside the units
    if (kAskEarly && T.more[after] != 0) ask_queries(T.seg[after]);
    const int row0 = cur.row0;
    const int seen0 = cur.rq.seen0();   // row j sees tokens <= seen0 + j
    uint32_t* const nan_mask = T.nan_mask[nan_slot];
    const float g_out = g_v;

    uint4 qf[S::kQInRegs ? kChunks : 1][S::kQInRegs ? NT : 1];
    const uint8_t* const q_frag = T.q + g * S::kQStride + t4 * 16;   // this lane's fragments of chunk 0, row g
    if constexpr (S::kQInRegs) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) qf[c][n] = *reinterpret_cast<const uint4*>(q_frag + n * 8 * S::kQStride + c * 64);
    }
    float qs[NT][2], m[NT][2], l[NT][2];
    float o[kMT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qs[n][k] = T.q_scale[n * 8 + t4 * 2 + k] * g_k;
        m[n][k] = kNone;
        l[n][k] = 0.0f;
      }
#pragma unroll
    for (int c = 0; c < kMT; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[c][n][k] = 0.0f;

    int s = kFirstStage;
    for (int i = 0; i < mine; ++i) {
      {   // into the stage that the unit before has left
        const int ahead = i + S::kAhead;
        if (ahead < mine) issue(ahead, s == 0 ? S::kStages - 1 : s - 1);
        cp_async_commit();
      }
      cp_async_wait<S::kAhead>();
      __syncwarp();
      const uint32_t ks_at = ring + s * S::kStage, vs_at = ks_at + S::kCodes, sc_at = vs_at + S::kCodes;
      const uint32_t there = T.there[warp][s];
      s = s == S::kStages - 1 ? 0 : s + 1;
      const int tok0 = (int)((uint32_t)tok_first + (uint32_t)i * (S::kUnit * W));
      if (there == 0u) continue;
      const bool ragged = tok0 + S::kUnit - 1 > seen0 || there != (1u << U) - 1u;   // the end, or a box that is not there
      if (ragged) {
        // Values that no row or not every row may see: tokens past the end get a zero
        // scale (their memory may hold anything), and a NaN scale among the rows' own
        // tokens is taken out here and put back at the end for the rows that do see it.
        for (int b = lane; b < S::kScales; b += 32) {
          const int tk = b / (D / 16), own = tok0 + tk - seen0;
          if (own <= 0) continue;
          const uint32_t at = sc_at + S::kScales + b;
          const bool bad = (lds_u8(at) & 0x7Fu) == 0x7Fu, past = tok0 + tk >= cur.rq.len;
          if (!past && bad) atomicOr(&nan_mask[b % (D / 16)], 1u << min(own, 31));
          if (past || bad) asm volatile("st.shared.u8 [%0], %1;" :: "r"(at), "r"(0) : "memory");
        }
        __syncwarp();
      }
      convert_scales<D, U>(sc_at, sc_at + S::kScales, sc16, lane);
      __syncwarp();
      // ---- S^T: 16 tokens a box x rows
      float x[U][NT][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        constexpr int kChains = U * NT == 1 ? 2 : 1;
        float acc[kChains][NT][4];
#pragma unroll
        for (int j = 0; j < kChains; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][n][k] = 0.0f;
        // two tokens' scales of this lane's half of every chunk
        uint32_t sa[kChunks / 2], sb[kChunks / 2];
        const uint32_t row_at = sc16 + (u * kBox + g) * (D / 8) + (t4 >> 1) * (D / 16);
        lds_words<kChunks / 2>(row_at, sa);
        lds_words<kChunks / 2>(row_at + 8 * (D / 8), sb);
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
          uint32_t w[4];
          ldsm_x4(ks_at + codes_at<D>(u * kBox + lrow, c + lchunk), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16x2x4(w[2 * h], a[0], a[1], a[2], a[3]);
            e2m1x8_to_f16x2x4(w[2 * h + 1], b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a[k] = h ? scaled_hi(a[k], sa[c / 2]) : scaled_lo(a[k], sa[c / 2]);
              b[k] = h ? scaled_hi(b[k], sb[c / 2]) : scaled_lo(b[k], sb[c / 2]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint4 q;
              if constexpr (S::kQInRegs) q = qf[c + h][n];
              else q = *reinterpret_cast<const uint4*>(q_frag + n * 8 * S::kQStride + (c + h) * 64);
              mma_free(acc[0][n], a[0], b[0], a[1], b[1], q.x, q.y);
              mma_free(acc[kChains - 1][n], a[2], b[2], a[3], b[3], q.z, q.w);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kChains == 2) acc[0][n][k] += acc[1][n][k];
            x[u][n][k] = acc[0][n][k] * qs[n][k & 1];
          }
      }
      // ---- masks
      if (ragged) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int t = tok0 + u * kBox;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              int lim = min(seen0 + (row0 + n * 8 + t4 * 2 + k) / p.G, cur.rq.len - 1);
              if (!((there >> u) & 1u)) lim = -1;
              if (t + g > lim) x[u][n][k] = -INFINITY;
              if (t + g + 8 > lim) x[u][n][k + 2] = -INFINITY;
            }
        }
      }
      // ---- running maximum: m follows only past a margin, so that most units
      // compare and vote and no more
      bool grew = false;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) grew |= x[u][n][k] > m[n][k & 1] + kTop;
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) v = fmaxf(v, fmaxf(x[u][n][k], x[u][n][k + 2]));
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, y));
            const float to = fmaxf(m[n][k], v - (kTop - kMargin)), f = exp2_fast(m[n][k] - to);
            m[n][k] = to;
            l[n][k] *= f;
#pragma unroll
            for (int c = 0; c < kMT; ++c) {
              o[c][n][k] *= f;
              o[c][n][k + 2] *= f;
            }
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // ---- weights, their sums, P^T as the second product's B operand
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float wv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) wv[k] = exp2_fast(x[u][n][k] - m[n][k & 1]);
          l[n][0] += wv[0] + wv[2];
          l[n][1] += wv[1] + wv[3];
          const __half2 h0 = __floats2half2_rn(wv[0], wv[1]), h1 = __floats2half2_rn(wv[2], wv[3]);
          pb[n][0] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h0));
          pb[n][1] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h1));
        }
        // ---- O^T += V^T P^T; of a chunk's two m tiles, row g is dimension 4 g (+ 2), g + 8 the next
        // (scales of tokens 2 t4 and the next, 2 t4 + 8 and the next)
        uint32_t fa[kChunks], fb[kChunks];
        const uint32_t row_at = sc16 + U * 2 * D + (g >> 2) * (U * D) + (u * 8 + t4) * (D / 8);
        lds_words<kChunks>(row_at, fa);
        lds_words<kChunks>(row_at + 4 * (D / 8), fb);
#pragma unroll
        for (int c = 0; c < kChunks; c += 2) {
          uint32_t w[4];
          ldsm_x4_t(vs_at + codes_at<D>(u * kBox + lrow, c + lchunk), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // Four dimensions of two tokens a word, their codes paired up in bytes,
            // so that a conversion gives the two tokens' values side by side.
            const uint32_t even = __byte_perm(w[2 * h], w[2 * h + 1], 0x5410), odd = __byte_perm(w[2 * h], w[2 * h + 1], 0x7632);
            uint32_t x[4], z[4];   // dimensions 4 g, + 2 and + 1, + 3; of the first tokens, then of the second
            e2m1x8_to_f16x2x4((even & 0x0F0F0F0Fu) | ((odd << 4) & 0xF0F0F0F0u), x[0], x[1], x[2], x[3]);
            e2m1x8_to_f16x2x4(((even >> 4) & 0x0F0F0F0Fu) | (odd & 0xF0F0F0F0u), z[0], z[1], z[2], z[3]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t a0 = hmul2_u32(x[y], fa[c + h]), a1 = hmul2_u32(z[y], fa[c + h]);
              const uint32_t a2 = hmul2_u32(x[y + 2], fb[c + h]), a3 = hmul2_u32(z[y + 2], fb[c + h]);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_free(o[2 * (c + h) + y][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            }
          }
        }
      }
      __syncwarp();   // every lane has read the stage before it is copied to again
    }
    cp_async_wait<0>();
    const int had = mine;
    const int n_live = min(cur.last - cur.first, W);   // warps that had a unit

    // ---- the segment's end: join the warps' m, l, O
    more = T.more[after] != 0;
    turn = after;
    if (more) {
      ask_segment();
      if (!kAskEarly) ask_queries(T.seg[turn]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], x);
        if (g == 0) {
          T.m[warp][n * 8 + t4 * 2 + k] = m[n][k];
          T.l[warp][n * 8 + t4 * 2 + k] = l[n][k];
        }
      }
    if (had > 0) {
      float* const own = join + warp * kJoinStep;
#pragma unroll
      for (int c = 0; c < kMT; c += 2)   // a chunk's two m tiles hold four neighbouring dimensions a lane
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float4*>(own + (n * 8 + t4 * 2 + k) * S::kJoinRow + c * 16 + 4 * g) =
                make_float4(o[c][n][k], o[c][n][k + 2], o[c + 1][n][k], o[c + 1][n][k + 2]);
    }
    if (more) {
      take_batch();
      open_units(0, S::kEarly);
    }
    __syncthreads();
    if (more) store_queries(nan_slot ^ 1);
    const int n_group_rows = min(cur.rq.rows(p) * p.G - row0, S::kRows);
    const bool whole = cur.whole;
    const int slot = cta * 2 + (cur.starts ? 1 : 0);
    for (int e = tid; e < n_group_rows * (D / 4); e += S::kThreads) {
      const int n = e / (D / 4), d = (e % (D / 4)) * 4;
      float mw[W], top = kNone, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) mw[w] = w < n_live ? T.m[w][n] : kNone;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, mw[w]);
      float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w >= n_live) break;
        const float f = exp2_fast(mw[w] - top);
        const float4 b = *reinterpret_cast<const float4*>(join + w * kJoinStep + n * S::kJoinRow + d);
        sum = fmaf(T.l[w][n], f, sum);
        a.x = fmaf(b.x, f, a.x);
        a.y = fmaf(b.y, f, a.y);
        a.z = fmaf(b.z, f, a.z);
        a.w = fmaf(b.w, f, a.w);
      }
      const int j = (row0 + n) / p.G, h = cur.head * p.G + (row0 + n) % p.G;
      if (nan_mask[d / 16] & ((2u << j) - 1u)) a = make_float4(NAN, NAN, NAN, NAN);
      a.x *= g_out;
      a.y *= g_out;
      a.z *= g_out;
      a.w *= g_out;
      if (p.spread > 1) {   // for the cluster, where warp 0's lay
        *reinterpret_cast<float4*>(join + n * S::kJoinRow + d) = a;
        if (d == 0) T.spread_ml[n] = make_float2(top, sum);
      } else if (whole) {
        store_result<D>(p, (size_t)(cur.rq.start + j) * p.H + h, d, a, top, sum);
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * S::kRows + n) * D + d) = a;
        if (d == 0) p.part_ml[(size_t)slot * S::kRows + n] = make_float2(top, sum);
      }
    }
    if (tid == 0) {   // the segment after the next
      const int later = turn == 2 ? 0 : turn + 1;
      T.more[later] = more && T.walk.next(p, S::kRows, T.seg[later]);
    }
    nan_slot ^= 1;
  }
  if (spread) {   // a cluster's CTAs join a segment's parts, a slice of the rows' dimensions each
    cluster_sync();
    const Segment& sg = T.seg[0];
    const int rank = cta % p.spread, n_group_rows = min(sg.rq.rows(p) * p.G - sg.row0, S::kRows);
    for (int e = rank * S::kThreads + tid; e < n_group_rows * (D / 4); e += p.spread * S::kThreads) {
      const int n = e / (D / 4), d = (e % (D / 4)) * 4;
      const uint32_t ml_at = smem_u32(&T.spread_ml[n]), a_at = smem_u32(join + n * S::kJoinRow + d);
      float2 ml[kMaxSpread];
      float4 b[kMaxSpread];
      float top = kNone, sum = 0.0f;
#pragma unroll
      for (int c = 0; c < kMaxSpread; ++c)
        if (c < p.spread) {
          ml[c] = peer_float2(ml_at, c);
          b[c] = peer_float4(a_at, c);
          top = fmaxf(top, ml[c].x);
        }
      float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < kMaxSpread; ++c)
        if (c < p.spread) {
          const float f = exp2_fast(ml[c].x - top);
          sum = fmaf(ml[c].y, f, sum);
          a.x = fmaf(b[c].x, f, a.x);
          a.y = fmaf(b[c].y, f, a.y);
          a.z = fmaf(b[c].z, f, a.z);
          a.w = fmaf(b[c].w, f, a.w);
        }
      const int j = (sg.row0 + n) / p.G, h = sg.head * p.G + (sg.row0 + n) % p.G;
      store_result<D>(p, (size_t)(sg.rq.start + j) * p.H + h, d, a, top, sum);
    }
    cluster_sync();   // the others have read this CTA's
  }
  if (p.direct) return;
  __syncthreads();
  if (tid == 0) p.failed[cta] = T.status;
}

// Joins the partial results of a cut segment, x: its number where the segments are
// fewer than the CTAs, else the CTA that starts it. A row a CTA of the y axis, four
// floats a thread and kPer pieces side by side, four of a thread's asked for
// together. The last y clears the rows without a result and gathers the status.
template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads) join4_kernel(const __grid_constant__ AttnLine p) {
  const int kRows = p.group_rows;
  constexpr int kLanes = D / 4, kPer = kThreads / kLanes;
  __shared__ float4 s_a[kPer][kLanes];
  __shared__ float2 s_ml[kPer];
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, n = blockIdx.y;
  if (n == (int)gridDim.y - 1) {
    clear_and_report<D>(p);
    return;
  }
  const int4 cut = p.cut[2 * c], more = p.cut[2 * c + 1];
  if (p.by_segment) {   // a request's missing row groups have no entry
    const int r = c / (p.K * p.max_groups);
    if (c % p.max_groups >= request_of(p, r, kRows).groups) return;
  }
  const int pieces = more.x, first = more.y;
  if (pieces < 2 || n >= cut.y) return;
  const int d4 = threadIdx.x % kLanes, at = threadIdx.x / kLanes;
  float m = kNone, l = 0.0f;
  float4 a = make_float4(0, 0, 0, 0);
  for (int i0 = at; i0 < pieces; i0 += 4 * kPer) {
    float2 ml[4];
    float4 b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kPer;
      ml[k] = make_float2(kNone, 0.0f);
      b[k] = make_float4(0, 0, 0, 0);
      if (i < pieces) {
        const size_t row = (size_t)((first + i) * 2 + (i == 0 ? 1 : 0)) * kRows + n;
        ml[k] = p.part_ml[row];
        b[k] = reinterpret_cast<const float4*>(p.part_o + row * D)[d4];
      }
    }
    const float to = fmaxf(m, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x))), f = exp2_fast(m - to);
    m = to;
    l *= f;
    a.x *= f;
    a.y *= f;
    a.z *= f;
    a.w *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = exp2_fast(ml[k].x - to);
      l = fmaf(ml[k].y, e, l);
      a.x = fmaf(b[k].x, e, a.x);
      a.y = fmaf(b[k].y, e, a.y);
      a.z = fmaf(b[k].z, e, a.z);
      a.w = fmaf(b[k].w, e, a.w);
    }
  }
  s_a[at][d4] = a;
  if (d4 == 0) s_ml[at] = make_float2(m, l);
  __syncthreads();
  if (at != 0) return;
  const int live = min(pieces, kPer);
  float top = kNone;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = i < live ? fmaxf(top, s_ml[i].x) : top;
  l = 0.0f;
  a = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i >= live) break;
    const float2 ml = s_ml[i];
    const float4 b = s_a[i][d4];
    const float e = exp2_fast(ml.x - top);
    l = fmaf(ml.y, e, l);
    a.x = fmaf(b.x, e, a.x);
    a.y = fmaf(b.y, e, a.y);
    a.z = fmaf(b.z, e, a.z);
    a.w = fmaf(b.w, e, a.w);
  }
  const int head = cut.z, row0 = cut.w;
  const int j = (row0 + n) / p.G, h = head * p.G + (row0 + n) % p.G;
  const size_t o = (size_t)(cut.x + j) * p.H + h;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  reinterpret_cast<uint2*>(p.out + o * D)[d4] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse != nullptr && d4 == 0) p.lse[o] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// ---- host ------------------------------------------------------------------------

template <int D>
cudaError_t launch_join4_d(const AttnLine& p, cudaStream_t st) {
  const unsigned rows = (unsigned)(p.max_rows * p.G < p.group_rows ? p.max_rows * p.G : p.group_rows);
  // Few segments are cut into many pieces each, many into few.
  constexpr int kMost = D == 256 ? 1024 : 512;
  if (p.by_segment)
    return launch_pdl(join4_kernel<D, kMost>, dim3((unsigned)(p.R * p.K * p.max_groups), rows + 1), kMost, 0, st, p);
  return launch_pdl(join4_kernel<D, 256>, dim3((unsigned)p.n_ctas, rows + 1), 256, 0, st, p);
}

cudaError_t launch_join4(int D, const AttnLine& p, cudaStream_t st) {
  return D == 64 ? launch_join4_d<64>(p, st) : D == 128 ? launch_join4_d<128>(p, st) : launch_join4_d<256>(p, st);
}

// n8 tiles of a kernel for a request's rows: a warp holds O for every dimension, so
// NT * D <= 512; more rows go in groups, each of which reads the cache again.
int tiles_for(int D, int rows) {
  const int want = (rows + 7) / 8;
  int nt = 1;
  while (nt < want && nt < 512 / D) nt *= 2;
  return nt;
}

template <int D, int NT, bool kMany>
constexpr int attn4_smem() { return Shape4<D, NT, kMany>::kRing * Shape4<D, NT, kMany>::kWarps + (int)sizeof(Tail4<D, NT, kMany>) + 1024; }

// Tokens times dimensions of a table up to which a CTA takes a whole segment: no line, no
// parts, no join's launch (2.2 us of the host's time too). Device us, whole and cut: one
// request, 256 dimensions 33 tokens 5.2 and 7.6, 500 8.6 and 8.9, 1000 12.7 and 9.2; 128
// dimensions 500 6.2 and 7.9, 1000 8.9 and 8.2; 64 dimensions 1000 6.9 and 8.1, 2000 10.1
// and 8.6. Of more segments than CTAs run at once the next follows as one ends: 26 requests
// of 32 rows of 128, 113 tokens, 8 heads 14.1 and 22.9; 300 requests of 120 tokens, 8
// heads of 128 34.5 and 37.9. From two rounds on, twice as long ones too: 400 requests of
// 700 tokens, 4 heads of 256 53.5 and 73.8, 96 of 1700, 8 of 128 32.4 and 34.0 (four times:
// 200 of 3000, 8 of 128 81 and 85.5, but one long request among short ones would wait
// for its one CTA).
constexpr long long kDirect = 512 * 256;

// Few segments over longer tables: each by a cluster of up to eight CTAs, which join
// their parts through distributed shared memory, where as many clusters run at once. From
// this length (tokens times dimensions) on, and to a CTA's kDirect, or half more where
// they fill half of the GPU; as whole segments, or on the line, and so, device us: one request, 4 heads of 256 200 tokens 6.9 and 7.2,
// 400 7.9 and 6.9, 800 9.2 and 7.5, 3000 9.9 and 9.7, 6000 (past it) 10.3 and 12.7; 8 rows
// of 6 heads of 256 over 400 tokens 12.0 and 8.9, 1600 14.4 and 11.0; 4 requests of 3000
// tokens, 8 heads of 128 11.0 and 8.9, of 800 8.2 and 6.6; 2 rows, 16 heads of 64 over
// 3000 11.7 and 8.9, of 9000 18.1 and 16.1. 16 clusters of eight CTAs that do not run at once: 14.8 for 11.0. Not
// kept, 777 tokens: clusters of sixteen 8.5, CTAs of four warps 8.2, for 7.5.
constexpr long long kSpread = 1 << 16, kSpreadLeast = 1 << 13;   // and a CTA's least

struct Plan4 {
  int ctas, unit, warps;
  cudaError_t (*launch)(const Attn4Params&, cudaStream_t);
  int (*clusters)(int);   // of so many CTAs that run at once
};

template <int D, int NT, bool kMany>
cudaError_t launch_attn4(const Attn4Params& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, attn4_kernel<D, NT, kMany>, attn4_smem<D, NT, kMany>());
  if (e != cudaSuccess) return e;
  const unsigned clear = 1 + std::min(p.n_rows, 4096) / 8;   // of the rows of no request
  const unsigned ctas = p.direct ? p.direct + (clear + p.spread - 1) / p.spread * p.spread : p.n_ctas;
  return launch_pdl(attn4_kernel<D, NT, kMany>, dim3(ctas), Shape4<D, NT, kMany>::kThreads, attn4_smem<D, NT, kMany>(), st, p,
                    p.spread);
}

template <int D, int NT, bool kMany>
int clusters_of(int ctas) {
  static DeviceCounts<kMaxDevices, kMaxSpread + 1> counts;
  return counts.get(current_device(), ctas, [&]() {
    static std::atomic<unsigned long long> attr{0};
    if (set_smem_once(attr, attn4_kernel<D, NT, kMany>, attn4_smem<D, NT, kMany>()) != cudaSuccess) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(Shape4<D, NT, kMany>::kThreads);
    cfg.dynamicSmemBytes = attn4_smem<D, NT, kMany>();
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = (unsigned)ctas;
    a[0].val.clusterDim.y = 1;
    a[0].val.clusterDim.z = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, attn4_kernel<D, NT, kMany>, &cfg) == cudaSuccess) return n;
    cudaGetLastError();
    return -1;
  });
}

template <int D, int NT, bool kMany>
Plan4 plan_of() { return {num_sms() * Shape4<D, NT, kMany>::kCtas, Shape4<D, NT, kMany>::kUnit, Shape4<D, NT, kMany>::kWarps, launch_attn4<D, NT, kMany>,
          clusters_of<D, NT, kMany>}; }

template <bool kMany>
Plan4 plan4_of(int D, int nt) {
  if (D == 64)
    return nt == 1 ? plan_of<64, 1, kMany>() : nt == 2 ? plan_of<64, 2, kMany>() : nt == 4 ? plan_of<64, 4, kMany>() : plan_of<64, 8, kMany>();
  if (D == 128) return nt == 1 ? plan_of<128, 1, kMany>() : nt == 2 ? plan_of<128, 2, kMany>() : plan_of<128, 4, kMany>();
  return nt == 1 ? plan_of<256, 1, kMany>() : plan_of<256, 2, kMany>();
}
Plan4 plan4_for(int D, int nt, bool many) { return many ? plan4_of<true>(D, nt) : plan4_of<false>(D, nt); }

// n8 tiles of the wide kernel, 0: not for it. More than 64 rows go in groups. The other
// kernel holds 16 rows at 256 dimensions and 32 at 128 (more read the cache again), where
// both take the same: 16 rows of 256 over 200001 tokens 39 us here and 43 there.
int wide_tiles_for(int D, int rows) {
  if (D == 64 || rows <= (D == 256 ? 16 : 32)) return 0;
  const int want = (rows + 7) / 8, groups = (want + 7) / 8, each = (want + groups - 1) / groups;
  return (each + 1) / 2 * 2;
}

// A segment's start costs the wide kernel 6 us (queries to planes), so it has work of
// some length only, by the tables' width: a table's tokens times dimensions, and these
// times tables and heads. us, wide and not: 8 rows of 6 heads of 256 over 100001 tokens 55
// and 97, over 20000 28 and 30, over 6000 22 and 19; 40 such requests of 6000 81 and 101,
// of 2000 50 and 50, of 777 41 and 37; 40 rows of 128 over 100001 68 and 118, 30000 33 and
// 45, 6000 20 and 20, 40 such requests of 2000 58 and 61.
constexpr long long kWideTable = 1 << 18, kWideWork = 1 << 24;

size_t workspace_of(int D, int rows) {
  const int nt = tiles_for(D, rows), wide = wide_tiles_for(D, rows);
  const size_t a = attn_layout(plan4_for(D, nt, D == 64 && nt == 1).ctas, 8 * nt, D).total, b = wide ? attn_layout(num_sms(), 8 * wide, D).total : 0;
  return a > b ? a : b;
}

}  // namespace
}  // namespace bws

extern "C" {

size_t bws_kv4_attention_workspace_size(int n_q_heads, int n_kv_heads, int head_dim, int max_rows) {
  using namespace bws;
  if (!attn_dims_ok(n_q_heads, n_kv_heads, head_dim, max_rows)) return 0;
  return workspace_of(head_dim, max_rows * (n_q_heads / n_kv_heads));
}

int bws_kv4_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int n_rows, int n_q_heads,
                      const bws_kv4_cache* cache, const int32_t* block_table, int max_blocks, int n_requests,
                      const int32_t* row_start, const int32_t* kv_lens, int max_rows, float scale, uint16_t* out,
                      float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bws;
  const char* name = "bws_kv4_attention";
  int rc = check_kv4_cache(cache, name);
  if (rc) return rc;
  const int D = cache->head_dim, K = cache->n_kv_heads, B = cache->block_tokens;
  const AttnCall call = {q, q_row_stride, q_head_stride, n_rows, n_q_heads, block_table, max_blocks, n_requests,
                         row_start, kv_lens, max_rows, scale, out, lse, workspace, workspace_bytes};
  bool nothing;
  rc = check_attn_call(call, K, D, B, name, &nothing);
  if (rc || nothing) return rc;
  const int rows = max_rows * (n_q_heads / K);
  const size_t need = workspace_of(D, rows);
  if (!workspace || workspace_bytes < need)
    return fail(BWS_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", name, need, workspace_bytes);
  if (!aligned(workspace, 256)) return fail(BWS_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", name);
  Attn4Params p;
  memset(&p, 0, sizeof(p));
  p.k = cache->k;
  p.v = cache->v;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.k_global = cache->k_global;
  p.v_global = cache->v_global;
  p.block_stride = (long long)cache->block_stride;
  p.head_stride = (long long)cache->head_stride;
  p.scale_block_stride = (long long)cache->scale_block_stride;
  p.scale_head_stride = (long long)cache->scale_head_stride;
  cudaStream_t st = as_stream(stream);
  const int nt = tiles_for(D, rows), wide = wide_tiles_for(D, rows);
  const long long segments = (long long)n_requests * K * ((rows + 8 * nt - 1) / (8 * nt));
  const long long once = plan4_for(D, nt, false).ctas, length = (long long)max_blocks * B * D;
  const bool by_tile = wide && length >= kWideTable && std::min(length, kWideWork) * n_requests * K >= kWideWork;
  int spread = 1;
  if (length >= kSpread && !by_tile && 2 * segments <= once) {
    spread = kMaxSpread;
    while (spread > 1 && (length < kSpreadLeast * spread || segments > plan4_for(D, nt, false).clusters(spread))) spread /= 2;
    if (length > (2 * segments * spread > once ? kDirect + kDirect / 2 : kDirect) * spread) spread = 1;
  }
  const bool whole = spread > 1 || (!by_tile && length <= (segments >= 2 * once ? 2 * kDirect : kDirect) && segments < (1LL << 30));
  const bool many = whole ? segments > (D == 256 ? 2 : 1) * once : D == 64 && nt == 1 && segments >= 4 * once;
  const Plan4 plan = plan4_for(D, nt, many);
  const int ctas = by_tile ? num_sms() : whole ? (int)once : plan.ctas, group_rows = 8 * (by_tile ? wide : nt);
  fill_attn_line(p, call, K, B, cache->n_blocks, ctas, group_rows, attn_layout(ctas, group_rows, D));
  p.spread = spread;
  if (whole) p.direct = (int)segments * p.spread;
  cudaError_t e;
  if (by_tile) {
    if (!tensor_maps_available()) return fail(BWS_ERR_CUDA, "%s: the driver's tensor-map encoder is unavailable", name);
    const uint64_t bytes = D / 2;
    const uint64_t dims[5] = {bytes, (uint64_t)B, 1, (uint64_t)K, (uint64_t)cache->n_blocks};
    const uint64_t strides[4] = {bytes, bytes, cache->head_stride, cache->block_stride};
    for (p.box_log = 4; p.box_log < 7 && B % (2 << p.box_log) == 0;) ++p.box_log;
    const uint32_t box[5] = {(uint32_t)bytes, 1u << p.box_log, 1, 1, 1};
    if (!encode_5d(&p.k_map, cache->k, dims, strides, box) || !encode_5d(&p.v_map, cache->v, dims, strides, box))
      return fail(BWS_ERR_CUDA, "%s: tensor map encoding failed", name);
    p.unit = kWide4Tile;
    p.least = 1;
    p.lead = 1024 / p.unit;
    e = launch_attn4_wide(D, wide, p, st);
  } else {
    p.unit = plan.unit;
    p.least = plan.warps;
    p.lead = (D == 64 ? 768 : 512) / p.unit;
    e = plan.launch(p, st);
  }
  if (e == cudaSuccess && !p.direct) e = launch_join4(D, p, st);
  return cuda_status(e, name);
}

}  // extern "C"

// Attention of a step's 1..8 rows per request over the 8-bit cache. Contract in
// include/bws.h.
//
// Mathematics. A kv head's query rows (tokens of the request times the query
// heads of the group) are the N side of both products, cached tokens and head
// dimensions the M side: S^T = K Q^T, then O^T = V^T P^T, on m16n8k16 with f16
// operands and FP32 sums. E4M3 codes are exact in f16. A query row is scaled
// by a power of two to fit f16 (exact but for values 2^-24 below the row's
// largest). With a block's scales ks and vs,
//   x = scale * log2(e) * ks * (q . code) + log2(vs),   w = 2^(x - m),
//   out = sum w code_v / sum (w / vs),
// m about the running maximum of x: taking the value scale into the exponent
// keeps every weight within f16's reach (at most 2^15), whatever the blocks'
// scales, and its rounding to f16 (2^-11 down to 2^-23 of the row's largest; finer
// than the BF16 result) relative to the terms of the sum that it stands in. The
// sum of weights takes them unrounded; a term leaves it only 2^135 below the
// largest w.
//
// Work. A segment is one (request, kv head, group of 8 NT rows); its unit is 16
// cached tokens (one TMA box a side; never across a block). All units of all
// segments lie on one line that is cut into equal shares, one per CTA, so the
// CTAs finish together whatever the lengths are; before its units each segment
// has a lead, the length that its start and end cost. A segment cut by a share's
// border leaves one partial result (m, l, O) per share in the workspace, which
// the second kernel joins in share order (no atomics: same bits every run).
// Lengths are read on the device: every CTA forms the line's prefix itself.
//
// Inside a CTA the eight warps are independent: each takes every eighth unit
// through a ring of its own (TMA boxes, 128-byte swizzle, so that ldmatrix
// reads without bank conflicts) and keeps its own m, l and O in registers; no
// barrier joins them before the segment's end.
// Bound: for few rows HBM and what a CTA spends at its start, a segment's end and
// the join. One request of 131071 tokens, four kv heads of 256, one row: 50 us
// for 268 MB (5.4 TB/s; 8 us of it start, end and join). 80 requests, 751 MB at
// 128: 122 us (6.2 TB/s). 24 requests of five rows at 64, 141 MB: 37 us (3.8
// TB/s), where neither memory nor issue is full: a unit there is 2 KB against as
// many instructions of softmax a token as at 256, in one dependent chain a warp. Two CTAs an SM up to NT D = 128.
// Copies of several boxes at once, and keys' and values' rings apart, lost 2 to
// 18 us to fewer units in flight a warp. An unmarked L2 policy instead of
// evict_first cost 21 us in the batch of 80.
#include <string.h>

#include <atomic>

#include "kv_attention.cuh"
#include "kv_cache.cuh"
#include "stream_tile.cuh"

namespace bws {
namespace {

template <int D, int NT>
struct Shape {
  static constexpr int kSide = kBox * D;                     // bytes of a unit's keys, or values
  static constexpr int kStage = 2 * kSide;
  static constexpr int kRows = 8 * NT;
  // a warp's O in FP32, for the segment's end; four words between rows put the
  // eight rows of a store on all banks
  static constexpr int kJoinRow = D + 4;
  static constexpr int kJoin = kRows * kJoinRow * 4;
  // Up to NT * D = 256 the warps' O has memory of its own, so that the next
  // segment's copies run during the join; wider ones use the drained ring.
  static constexpr bool kOverlap = NT * D <= 256;
  static constexpr int kCtas = NT * D <= 128 ? 2 : 1;         // CTAs an SM, by registers
  static constexpr int kStages = !kOverlap ? NT + 1 : ((kCtas == 2 ? 100 : 200) * 1024 / kAttnWarps - kJoin) / kStage;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kWarpBytes = kRing + (kOverlap ? kJoin : 0);
  static constexpr bool kQInRegs = NT * D <= 256;
  static constexpr int kQStride = 2 * D + 32;                 // bytes of a query row: four rows of fragments on all banks
  static_assert(kStages >= 2 && (kOverlap || kRing >= kJoin), "ring");
};

template <int D, int NT>
struct __align__(16) Tail {
  uint8_t q[8 * NT * Shape<D, NT>::kQStride];
  float q_scale[8 * NT];
  float m[kAttnWarps][8 * NT];
  float l[kAttnWarps][8 * NT];
  uint32_t nan_mask[2][D];                                    // bit j: token j of the rows' own has a NaN there
  unsigned long long full[kAttnWarps][Shape<D, NT>::kStages];
  long long line_warp[kAttnWarps];
  long long line_found[2];
  uint32_t status;
};

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, Shape<D, NT>::kCtas) attn_kernel(const __grid_constant__ AttnParams p) {
  using S = Shape<D, NT>;
  constexpr int kMT = D / 16;   // m tiles of O^T
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (base - smem_u32(smem_raw));   // rings, then the warps' O, then the tail
  Tail<D, NT>& T = *reinterpret_cast<Tail<D, NT>*>(smem + S::kWarpBytes * kAttnWarps);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = base + warp * S::kRing;
  float* const join = reinterpret_cast<float*>(smem + (S::kOverlap ? S::kRing * kAttnWarps : 0));
  constexpr int kJoinStep = (S::kOverlap ? S::kJoin : S::kRing) / 4;    // floats from warp to warp
  const uint32_t bar0 = smem_u32(&T.full[warp][0]);
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(bar0 + 8 * s, 1);
    mbar_fence_init();
  }
  if (tid == 0) T.status = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int cta = blockIdx.x;
  Walk walk;
  walk.start(p, S::kRows, T.line_warp, T.line_found, &T.status);
  const uint64_t pol = l2_evict_first();
  uint32_t phase_base = 0;   // units this warp has put through its ring
  bool dead = false;
  // this lane's ldmatrix row: tokens 0-7 and 8-15 of one chunk, then of the next
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lchunk = lane >> 4;

  Segment sg = {};
  // ---- copies: 32 of the warp's units (first + warp, + 8, ...) at a time, a unit
  // a lane: the block (-1: not there) and the token in it.
  int mine, ids, toks;
  auto token_of = [&](int i) { return (int)((uint32_t)(sg.first + warp + i * kAttnWarps) * kBox); };   // asked past the end too
  auto look_up = [&](int i, int& block, int& tok) {
    block = -1;
    tok = 0;
    const int t = token_of(i);
    if (i < mine && t < sg.rq.kv(p)) {
      const int q = block_index(p, t);
      const int b = p.table[(size_t)sg.r * p.max_blocks + q];
      tok = t - q * p.B;
      block = b >= 0 && b < p.n_blocks ? b : -1;
    }
  };
  auto issue = [&](int i, int s) {   // the whole warp; unit i of this warp into stage s
    if ((i & 31) == 0 && i > 0) look_up(i + lane, ids, toks);
    const int b = __shfl_sync(0xffffffffu, ids, i & 31), tok = __shfl_sync(0xffffffffu, toks, i & 31);
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * s, dst = ring + s * S::kStage;
      if (b >= 0) {
        mbar_arrive_expect_tx(bar, S::kStage);
        tma_load_box(dst, &p.k, tok, sg.head, b, bar, pol);
        tma_load_box(dst + S::kSide, &p.v, tok, sg.head, b, bar, pol);
      } else {
        mbar_arrive(bar);
      }
    }
  };
  // Scales of 32 units, one a lane: ks (-1: the block is not there) and vs as
  // they are read, and when they are used log2(vs) and 1 / vs.
  struct Scales {
    float ks, vs;
  };
  Scales sc_n;
  float ks_l, lvs_l, rvs_l;
  auto scales_of = [&](int b) {
    Scales s = {-1.0f, 1.0f};
    if (b >= 0) {
      const size_t at = (size_t)b * p.K + sg.head;
      s.ks = p.k_scale[at];
      s.vs = p.v_scale[at];
    }
    return s;
  };
  auto use_scales = [&](const Scales& s) {
    const float vs = fminf(fmaxf(s.vs, 0x1p-60f), 0x1p60f);
    ks_l = s.ks;
    lvs_l = log2f(vs);
    rvs_l = 1.0f / vs;
  };
  // A segment's start, in two steps, so that block ids and query rows are on
  // their way while the segment before is joined: what is asked for first, and
  // the copies and scales that need the ids.
  uint32_t qx[NT][D / 64];   // dimensions 2 lane + 64 i and the next, BF16
  auto ask_segment = [&]() {
    mine = (sg.last - sg.first - warp + kAttnWarps - 1) / kAttnWarps;
    look_up(lane, ids, toks);
    const int n_rows = min(sg.rq.rows(p) * p.G - sg.row0, S::kRows);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int n = warp + k * kAttnWarps;
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
  auto open_segment = [&]() {
    if (!dead) {
      const int ahead = min(mine, S::kStages);
      for (int i = 0; i < ahead; ++i) issue(i, (int)((phase_base + i) % S::kStages));
    }
    sc_n = scales_of(ids);
  };
  // The query rows to f16, each scaled by a power of two. `slot`: the NaN mask to clear.
  auto store_queries = [&](int slot) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int n = warp + k * kAttnWarps;
      __half2* dst = reinterpret_cast<__half2*>(T.q + n * S::kQStride);
      float x[D / 32];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = __uint_as_float(i % 2 ? qx[k][i / 2] & 0xFFFF0000u : qx[k][i / 2] << 16);
        if (fabsf(x[i]) < INFINITY) top = fmaxf(top, fabsf(x[i]));
      }
      top = warp_max(top);
      const int e = top > 0.0f ? min(max(floor_log2_abs(top), -100), 126) : 0;
      const float f = exp2i(-e);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) dst[lane + 32 * i] = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
      if (lane == 0) T.q_scale[n] = p.scale * kLog2e * exp2i(e);
    }
    for (int i = tid; i < D; i += kAttnThreads) T.nan_mask[slot][i] = 0;
  };

  bool more = walk.next(p, S::kRows, sg);
  int turn = 0;
  if (more) {
    ask_segment();
    open_segment();
    store_queries(0);
  }
  while (more) {
    __syncthreads();
    const Segment cur = sg;
    const Request& rq = cur.rq;
    const int row0 = cur.row0, head = cur.head;
    const int n_group_rows = min(rq.rows(p) * p.G - row0, S::kRows);
    const int seen0 = rq.seen0();   // row j sees tokens <= seen0 + j
    uint32_t* const nan_mask = T.nan_mask[turn];

    uint32_t qf[S::kQInRegs ? kMT : 1][S::kQInRegs ? NT : 1][2];
    const uint8_t* const q_frag = T.q + g * S::kQStride + t4 * 8;   // this lane's fragment of chunk 0, row g
    if constexpr (S::kQInRegs) {
#pragma unroll
      for (int c = 0; c < kMT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint2 b = *reinterpret_cast<const uint2*>(q_frag + n * 8 * S::kQStride + c * 32);
          qf[c][n][0] = b.x;
          qf[c][n][1] = b.y;
        }
    }
    float qs[NT][2], m[NT][2], l[NT][2];
    float o[kMT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qs[n][k] = T.q_scale[n * 8 + t4 * 2 + k];
        m[n][k] = kNone;
        l[n][k] = 0.0f;
      }
#pragma unroll
    for (int c = 0; c < kMT; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[c][n][k] = 0.0f;

    use_scales(sc_n);
    for (int i = 0; i < mine; ++i) {
      const uint32_t it = phase_base + i;
      const int s = (int)(it % S::kStages);
      const uint32_t ks_at = ring + s * S::kStage, vs_at = ks_at + S::kSide;
      if (!dead && !mbar_wait_bounded(bar0 + 8 * s, (it / S::kStages) & 1, kAttnPolls)) dead = true;
      if (__any_sync(0xffffffffu, dead)) {
        dead = true;
        if (lane == 0) atomicOr(&T.status, (uint32_t)BWS_STATUS_WAIT_TIMEOUT);
        for (int k = i + 1; k < min(i + S::kStages, mine); ++k) {   // the copies still on their way
          const uint32_t at = phase_base + k;
          mbar_wait_bounded(bar0 + 8 * (at % S::kStages), (at / S::kStages) & 1, kAttnPolls);
        }
        break;
      }
      if ((i & 31) == 16) {   // half a batch ahead
        int b, tok;
        look_up((i & ~31) + 32 + lane, b, tok);
        sc_n = scales_of(b);
      }
      if ((i & 31) == 0 && i > 0) use_scales(sc_n);
      const float ks = __shfl_sync(0xffffffffu, ks_l, i & 31);
      const int tok0 = token_of(i);
      if (ks != -1.0f) {
        const float lvs = __shfl_sync(0xffffffffu, lvs_l, i & 31), rvs = __shfl_sync(0xffffffffu, rvs_l, i & 31);
        // ---- S^T: 16 tokens x rows
        // (two chains of sums, of even and of odd chunks, where the rows are few)
        constexpr int kChains = NT == 1 ? 2 : 1;
        float acc[kChains][NT][4];
#pragma unroll
        for (int j = 0; j < kChains; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][n][k] = 0.0f;
#pragma unroll
        for (int c = 0; c < kMT; c += 2) {
          uint32_t w[4];
          ldsm_x4(ks_at + chunk_at<D>(lrow, c + lchunk), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2x2(w[2 * h], a0, a2);
            e4m3x4_to_f16x2x2(w[2 * h + 1], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t b0, b1;
              if constexpr (S::kQInRegs) {
                b0 = qf[c + h][n][0];
                b1 = qf[c + h][n][1];
              } else {
                const uint2 b = *reinterpret_cast<const uint2*>(q_frag + n * 8 * S::kQStride + (c + h) * 32);
                b0 = b.x;
                b1 = b.y;
              }
              mma_free(acc[h % kChains][n], a0, a1, a2, a3, b0, b1);
            }
          }
        }
        // ---- exponents, masks
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (kChains == 2) acc[0][n][k] += acc[1][n][k];
            x[n][k] = fmaf(acc[0][n][k], ks * qs[n][k & 1], lvs);
          }
        if (tok0 + kBox - 1 > seen0) {   // the end: some rows do not see all 16
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int lim = min(seen0 + (row0 + n * 8 + t4 * 2 + k) / p.G, rq.len - 1);
              if (tok0 + g > lim) x[n][k] = -INFINITY;
              if (tok0 + g + 8 > lim) x[n][k + 2] = -INFINITY;
            }
          // Values no row or not every row may see: rows past the end are
          // zeroed (their memory may hold anything), and a NaN among the rows'
          // own tokens is taken out here and put back at the end for the rows
          // that do see it; 0 * NaN would reach the others.
          __syncwarp();
          for (int b = lane; b < kBox * (D / 4); b += 32) {
            const int tk = b / (D / 4), byte = (b % (D / 4)) * 4, own = tok0 + tk - seen0;
            if (own <= 0) continue;
            const uint32_t at = vs_at + chunk_at<D>(tk, byte >> 4) + (byte & 15);
            uint32_t word;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(word) : "r"(at) : "memory");
            if (tok0 + tk >= rq.len) {   // (a table row ends with a box)
              word = 0;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (((word >> (8 * k)) & 0x7Fu) == 0x7Fu) {
                  word &= ~(0xFFu << (8 * k));
                  atomicOr(&nan_mask[byte + k], 1u << min(own, 31));
                }
            }
            asm volatile("st.shared.u32 [%0], %1;" :: "r"(at), "r"(word) : "memory");
          }
          proxy_fence();   // before TMA writes the stage again
          __syncwarp();
        }
        // ---- running maximum: m follows only past a margin, so that most units
        // compare and vote and no more
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) grew |= x[n][k] > m[n][k & 1] + kTop;
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float v = fmaxf(x[n][k], x[n][k + 2]);
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
        // ---- weights, their sums, P^T as the second product's B operand
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float wv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) wv[k] = exp2_fast(x[n][k] - m[n][k & 1]);
          l[n][0] = fmaf(wv[0] + wv[2], rvs, l[n][0]);
          l[n][1] = fmaf(wv[1] + wv[3], rvs, l[n][1]);
          const __half2 h0 = __floats2half2_rn(wv[0], wv[1]), h1 = __floats2half2_rn(wv[2], wv[3]);
          pb[n][0] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h0));
          pb[n][1] = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h1));
        }
        // ---- O^T += V^T P^T; m row g is dimension 2 g of the chunk, g + 8 is 2 g + 1
#pragma unroll
        for (int c = 0; c < kMT; c += 2) {
          uint32_t w[4];
          ldsm_x4_t(vs_at + chunk_at<D>(lrow, c + lchunk), w);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2x2(__byte_perm(w[2 * h], 0, 0x3120), a0, a1);
            e4m3x4_to_f16x2x2(__byte_perm(w[2 * h + 1], 0, 0x3120), a2, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_free(o[c + h][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
          }
        }
      }
      __syncwarp();
      if (i + S::kStages < mine) issue(i + S::kStages, s);
    }
    phase_base += mine;
    const int had = mine;
    const int n_live = min(cur.last - cur.first, kAttnWarps);   // warps that had a unit

    // ---- the segment's end: join the warps' m, l, O
    more = walk.next(p, S::kRows, sg);
    if (more) ask_segment();
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
      for (int c = 0; c < kMT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float2*>(own + (n * 8 + t4 * 2 + k) * S::kJoinRow + c * 16 + 2 * g) =
                make_float2(o[c][n][k], o[c][n][k + 2]);
    }
    if (S::kOverlap && more) open_segment();
    __syncthreads();
    const bool whole = cur.whole;
    const int slot = cta * 2 + (cur.starts ? 1 : 0);
    if (S::kOverlap && more) store_queries(turn ^ 1);
    for (int e = tid; e < n_group_rows * (D / 4); e += kAttnThreads) {
      const int n = e / (D / 4), d = (e % (D / 4)) * 4;
      float top = kNone;
      for (int w = 0; w < n_live; ++w) top = fmaxf(top, T.m[w][n]);
      float sum = 0.0f;
      float4 a = make_float4(0, 0, 0, 0);
      for (int w = 0; w < n_live; ++w) {
        const float mw = T.m[w][n];
        const float f = exp2_fast(mw - top);
        const float4 b = *reinterpret_cast<const float4*>(join + w * kJoinStep + n * S::kJoinRow + d);
        sum = fmaf(T.l[w][n], f, sum);
        a.x = fmaf(b.x, f, a.x);
        a.y = fmaf(b.y, f, a.y);
        a.z = fmaf(b.z, f, a.z);
        a.w = fmaf(b.w, f, a.w);
      }
      const int j = (row0 + n) / p.G, h = head * p.G + (row0 + n) % p.G;
      const uint32_t see = (2u << j) - 1u;
      if (nan_mask[d] & see) a.x = NAN;
      if (nan_mask[d + 1] & see) a.y = NAN;
      if (nan_mask[d + 2] & see) a.z = NAN;
      if (nan_mask[d + 3] & see) a.w = NAN;
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
        const size_t at = (size_t)(rq.start + j) * p.H + h;
        *reinterpret_cast<uint2*>(p.out + at * D + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        if (p.lse != nullptr && d == 0) p.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((size_t)slot * S::kRows + n) * D + d) = a;
        if (d == 0) p.part_ml[(size_t)slot * S::kRows + n] = make_float2(top, sum);
      }
    }
    if (!S::kOverlap && more) {
      proxy_fence();   // O lay where TMA writes next
      __syncthreads();
      open_segment();
      store_queries(turn ^ 1);
    }
    turn ^= 1;
  }
  __syncthreads();
  if (tid == 0) p.failed[cta] = T.status;
}

// Output rows without a result of their own become what a row without tokens is:
// rows of no request (before `begin`, from `end` on), as a captured step's padding,
// and a request's rows past max_rows. The first row's CTAs take them in turn. Out of
// line: the join lasts a few loads, and a call without such rows fetches none of it.
template <int D>
__device__ __noinline__ void clear_rows(const AttnParams& p, int begin, int end, bool excess) {
  auto clear = [&](int from, int to) {
    for (int row = from + blockIdx.x; row < to; row += gridDim.x) {
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

// Joins the partial results of a cut segment, x: its number where the segments
// are fewer than the CTAs, else the CTA that starts it. One row a CTA of the y
// axis, four floats a thread.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnParams p) {
  const int kRows = p.group_rows;
  constexpr int kLanes = D / 4;            // threads of a row
  constexpr int kPer = 256 / kLanes;       // pieces read side by side
  __shared__ float4 s_a[kPer][kLanes];
  __shared__ float s_l[kPer];
  __shared__ uint32_t s_bad;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x;
  const int4 cut = p.cut[2 * c], more = p.cut[2 * c + 1];
  if (blockIdx.y == 0) {
    const int begin = p.row_start[0], end = p.row_start[p.R];
    const bool excess = (p.failed[0] & BWS_STATUS_KV_ROWS) != 0u;   // every CTA says it
    if (c == 0) {
      if (threadIdx.x == 0) s_bad = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < p.n_ctas; i += 256)
        if (p.failed[i] != 0) atomicOr(&s_bad, p.failed[i]);
      __syncthreads();
      if (threadIdx.x == 0) {
        p.hdr[0] = 0;
        p.hdr[1] = s_bad;
      }
    }
    if (begin > 0 || end < p.n_rows || excess) clear_rows<D>(p, begin, end, excess);
  }
  if (p.by_segment) {   // a request's missing row groups have no entry
    const int r = c / (p.K * p.max_groups);
    if (c % p.max_groups >= request_of(p, r, kRows).groups) return;
  }
  const int n = blockIdx.y;
  const int pieces = more.x, first = more.y;
  if (pieces < 2 || n >= cut.y) return;
  const int head = cut.z, row0 = cut.w;
  auto slot_of = [&](int i) { return (first + i) * 2 + (i == 0 ? 1 : 0); };
  const int d4 = threadIdx.x % kLanes, at = threadIdx.x / kLanes;
  float top = kNone;
  // a piece a lane: one after the other in every thread they cost 131071 tokens in 152 shares 3 us
  for (int i = threadIdx.x & 31; i < pieces; i += 32) top = fmaxf(top, p.part_ml[(size_t)slot_of(i) * kRows + n].x);
  top = warp_max(top);
  float4 a = make_float4(0, 0, 0, 0);
  float l = 0.0f;
#pragma unroll 4
  for (int i = at; i < pieces; i += kPer) {
    const size_t row = (size_t)slot_of(i) * kRows + n;
    const float2 ml = p.part_ml[row];
    const float4 b = reinterpret_cast<const float4*>(p.part_o + row * D)[d4];
    const float f = exp2_fast(ml.x - top);
    l = fmaf(ml.y, f, l);
    a.x = fmaf(b.x, f, a.x);
    a.y = fmaf(b.y, f, a.y);
    a.z = fmaf(b.z, f, a.z);
    a.w = fmaf(b.w, f, a.w);
  }
  s_a[at][d4] = a;
  if (d4 == 0) s_l[at] = l;
  __syncthreads();
  if (at != 0) return;
#pragma unroll
  for (int i = 1; i < kPer; ++i) {
    const float4 b = s_a[i][d4];
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
    l += s_l[i];
  }
  const int j = (row0 + n) / p.G, h = head * p.G + (row0 + n) % p.G;
  const size_t o = (size_t)(cut.x + j) * p.H + h;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  reinterpret_cast<uint2*>(p.out + o * D)[d4] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (p.lse != nullptr && d4 == 0) p.lse[o] = l == 0.0f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// ---- host ------------------------------------------------------------------------

// The kernel and its n8 tiles for a request's rows. A warp of attn_kernel holds
// O for every dimension, NT * D <= 512; more rows of a wide head go to the other
// kernel, up to 64 at a time (at 48 rows of 256 attn_kernel's three passes over
// the cache took 112 us for 100001 tokens, the wide kernel 67); what is still
// more goes in groups, each of which reads the cache again.
struct Form {
  bool wide;
  int nt;
};

Form form_for(int D, int rows) {
  const int want = (rows + 7) / 8;
  if (D > 64 && want * D > 512) {
    const int groups = (want + 7) / 8, each = (want + groups - 1) / groups;
    return {true, each <= 4 && D == 256 ? 4 : each <= 6 ? 6 : 8};
  }
  int nt = 1;
  while (nt < want && nt < 512 / D) nt *= 2;
  return {false, nt};
}

template <int D, int NT>
constexpr int attn_smem() { return Shape<D, NT>::kWarpBytes * kAttnWarps + (int)sizeof(Tail<D, NT>) + 1024; }

struct AttnLayout {
  size_t off_cut, off_failed, off_ml, off_o, total;
  int n_ctas;
  Form form;
};

AttnLayout attn_layout(int H, int K, int D, int max_rows) {
  AttnLayout L;
  L.form = form_for(D, max_rows * (H / K));
  L.n_ctas = num_sms() * (!L.form.wide && L.form.nt * D <= 128 ? 2 : 1);   // as their launch bounds ask
  const size_t rows = (size_t)2 * L.n_ctas * 8 * L.form.nt;
  // bws_status_word reads 8 bytes here and eight words from 512 on
  size_t o = 1024;
  L.off_cut = o; o += align256(2 * sizeof(int4) * (size_t)L.n_ctas);
  L.off_failed = o; o += align256(sizeof(uint32_t) * (size_t)L.n_ctas);
  L.off_ml = o; o += align256(sizeof(float2) * rows);
  L.off_o = o; o += align256(sizeof(float) * rows * D);
  L.total = o;
  return L;
}

bool attn_dims_ok(int H, int K, int D, int max_rows) {
  return (D == 64 || D == 128 || D == 256) && K >= 1 && K <= 128 && H >= K && H % K == 0 && H / K <= kAttnMaxGroup &&
         max_rows >= 1 && max_rows <= kAttnMaxRows;
}

template <int D, int NT>
cudaError_t launch_attn(const AttnParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, attn_kernel<D, NT>, attn_smem<D, NT>());
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_kernel<D, NT>, dim3((unsigned)p.n_ctas), kAttnThreads, attn_smem<D, NT>(), st, p);
}

template <int D>
cudaError_t launch_attn_d(Form form, const AttnParams& p, cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;
  if (form.wide) e = launch_attn_wide(D, form.nt, p, st);
  else if (form.nt == 1) e = launch_attn<D, 1>(p, st);
  else if (form.nt == 2) e = launch_attn<D, 2>(p, st);
  if constexpr (D <= 128) {
    if (!form.wide && form.nt == 4) e = launch_attn<D, 4>(p, st);
  }
  if constexpr (D <= 64) {
    if (!form.wide && form.nt == 8) e = launch_attn<D, 8>(p, st);
  }
  if (e != cudaSuccess) return e;
  const int rows = p.max_rows * p.G;
  const dim3 grid((unsigned)(p.by_segment ? p.R * p.K * p.max_groups : p.n_ctas),
                  (unsigned)(rows < p.group_rows ? rows : p.group_rows));
  return launch_pdl(join_kernel<D>, grid, 256, 0, st, p);
}

}  // namespace
}  // namespace bws

extern "C" {

size_t bws_kv_attention_workspace_size(int n_q_heads, int n_kv_heads, int head_dim, int max_rows) {
  using namespace bws;
  if (!attn_dims_ok(n_q_heads, n_kv_heads, head_dim, max_rows)) return 0;
  return attn_layout(n_q_heads, n_kv_heads, head_dim, max_rows).total;
}

int bws_kv_attention(const uint16_t* q, int64_t q_row_stride, int64_t q_head_stride, int n_rows, int n_q_heads,
                     const bws_kv_cache* cache, const int32_t* block_table, int max_blocks, int n_requests,
                     const int32_t* row_start, const int32_t* kv_lens, int max_rows, float scale, uint16_t* out,
                     float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace bws;
  const char* name = "bws_kv_attention";
  const int rc = check_kv_cache(cache, name);
  if (rc) return rc;
  const int D = cache->head_dim, K = cache->n_kv_heads;
  if (max_rows < 1 || max_rows > kAttnMaxRows)
    return fail(BWS_ERR_INVALID_ARG, "%s: max_rows = %d must be in [1, %d]", name, max_rows, kAttnMaxRows);
  if (!attn_dims_ok(n_q_heads, K, D, max_rows))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: n_q_heads = %d must be 1 to %d times n_kv_heads = %d", name, n_q_heads,
                kAttnMaxGroup, K);
  if (n_rows < 0 || n_requests < 0 || n_requests > (1 << 20) || max_blocks < 0)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d, n_requests = %d, max_blocks = %d", name, n_rows, n_requests,
                max_blocks);
  if ((long long)max_blocks * cache->block_tokens >= (1LL << 31))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: a table row of %d blocks passes 2^31 tokens", name, max_blocks);
  if (n_rows == 0 || n_requests == 0) {
    clear_error();
    return BWS_OK;
  }
  if (!q || !out || !row_start || !kv_lens || (max_blocks > 0 && !block_table))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!(scale > -INFINITY && scale < INFINITY)) return fail(BWS_ERR_INVALID_ARG, "%s: scale must be finite", name);
  if (!aligned(q, 16) || !aligned(out, 16) || q_row_stride % 8 || q_head_stride % 8 || !aligned(block_table, 4) ||
      !aligned(row_start, 4) || !aligned(kv_lens, 4) || !aligned(lse, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: q and out 16-byte, strides of 8 elements, other pointers 4-byte needed", name);
  const AttnLayout L = attn_layout(n_q_heads, K, D, max_rows);
  if (!workspace || workspace_bytes < L.total)
    return fail(BWS_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", name, L.total, workspace_bytes);
  if (!aligned(workspace, 256)) return fail(BWS_ERR_MISALIGNED, "%s: workspace must be 256-byte aligned", name);
  if (!tensor_maps_available()) return fail(BWS_ERR_CUDA, "%s: the driver's tensor-map encoder is unavailable", name);
  char* w = static_cast<char*>(workspace);
  AttnParams p;
  memset(&p, 0, sizeof(p));
  const uint32_t panel = D < 128 ? D : 128;
  const uint64_t dims[5] = {panel, (uint64_t)cache->block_tokens, D / panel, (uint64_t)K, (uint64_t)cache->n_blocks};
  const uint64_t strides[4] = {(uint64_t)D, panel, cache->head_stride, cache->block_stride};
  const uint32_t box[5] = {panel, kBox, L.form.wide ? 1 : D / panel, 1, 1};   // the wide kernel lays panels further apart
  if (!encode_5d(&p.k, cache->k, dims, strides, box) || !encode_5d(&p.v, cache->v, dims, strides, box))
    return fail(BWS_ERR_CUDA, "%s: tensor map encoding failed", name);
  p.q = q;
  p.q_row_stride = q_row_stride;
  p.q_head_stride = q_head_stride;
  p.n_rows = n_rows;
  p.H = n_q_heads;
  p.K = K;
  p.G = n_q_heads / K;
  p.B = cache->block_tokens;
  const uint32_t boxes = (uint32_t)p.B / kBox;
  p.b_inverse = boxes == 1 ? 0u : (uint32_t)(((1ull << 32) + boxes - 1) / boxes);
  p.n_blocks = cache->n_blocks;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.max_tokens = max_blocks * cache->block_tokens;
  p.R = n_requests;
  p.row_start = row_start;
  p.kv_lens = kv_lens;
  p.max_rows = max_rows;
  p.scale = scale;
  p.out = out;
  p.lse = lse;
  p.hdr = reinterpret_cast<uint32_t*>(w);
  p.cut = reinterpret_cast<int4*>(w + L.off_cut);
  p.failed = reinterpret_cast<uint32_t*>(w + L.off_failed);
  p.part_ml = reinterpret_cast<float2*>(w + L.off_ml);
  p.part_o = reinterpret_cast<float*>(w + L.off_o);
  p.n_ctas = L.n_ctas;
  p.group_rows = 8 * L.form.nt;
  p.max_groups = (max_rows * p.G + p.group_rows - 1) / p.group_rows;
  p.by_segment = (long long)n_requests * K * p.max_groups <= L.n_ctas;
  p.unit = L.form.wide ? kWideTile : kBox;
  // A box for every warp: 777 tokens took 12.1 us so, 12.8 with half, 15.1 with twice.
  p.least = L.form.wide ? 1 : kAttnWarps;
  // What a segment's start and end cost beside its tokens: about 512 tokens'
  // time, 1024 in the wide kernel, whose pipeline is longer. (Without it a share
  // of many short segments took 105 us of a batch whose CTAs averaged 39; between
  // a quarter and twice this the batches measured change by less than a tenth.)
  p.lead = (L.form.wide ? 1024 : 512) / p.unit;
  cudaStream_t st = as_stream(stream);
  cudaError_t e;
  if (D == 64) e = launch_attn_d<64>(L.form, p, st);
  else if (D == 128) e = launch_attn_d<128>(L.form, p, st);
  else e = launch_attn_d<256>(L.form, p, st);
  return cuda_status(e, name);
}

}  // extern "C"

// Attention over the 8-bit cache for many query rows a kv head (a verify pass
// of several tokens, wide groups): the mathematics and the line of shares are
// those of kv_attention.cu, the CTA's work is cut the other way.
//
// With more than 16 rows of 256 (32 of 128) a warp cannot hold O for every
// dimension, so here the eight warps share a tile of 128 cached tokens: for
// S^T = K Q^T a warp takes 16 tokens and all rows, for O^T += V^T P^T an eighth
// of the dimensions and all tokens. P crosses through shared memory in the
// fragment order of the second product. One running maximum per row serves the
// CTA: it follows only where an exponent passes it by more than 8, which the
// barrier before P is written also votes on, so most tiles meet two barriers
// and no exchange. Keys are a warp's own (its ring needs no barrier); values are
// read by all, so their next copy waits for the tile's first barrier.
// Bound: mma.sync (m16n8k16 takes 8 cycles of a quarter SM: 48 rows of 256 need
// 3072 cycles a tile, of which HBM gives one in 2750), then shared memory.
#include <atomic>

#include "kv_attention.cuh"

namespace bws {
namespace {

template <int D, int NT>
struct Wide {
  static constexpr int kRows = 8 * NT;
  static constexpr int kBoxBytes = kBox * D;                  // a warp's keys, or values, of a tile
  static constexpr int kSide = kAttnWarps * kBoxBytes;
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kQStride = 2 * D + 32;                 // bytes of a query row: four rows of fragments on all banks
  static constexpr int kMT = D / 16 / kAttnWarps;             // m tiles of O^T a warp holds
  static constexpr int kPBytes = kAttnWarps * NT * 256;       // P of a tile, in fragments
};

template <int D, int NT>
struct __align__(16) WideTail {
  uint8_t p[Wide<D, NT>::kPBytes];
  uint8_t q[8 * NT * Wide<D, NT>::kQStride];
  float q_scale[8 * NT];
  float top[kAttnWarps][8 * NT];
  float l[kAttnWarps][8 * NT];
  uint32_t nan_mask[2][D];
  unsigned long long k_full[kAttnWarps][Wide<D, NT>::kStages];
  unsigned long long v_full[Wide<D, NT>::kStages];
  long long line_warp[kAttnWarps];
  long long line_found[2];
  uint32_t failed;
};

template <int D, int NT>
constexpr int wide_smem() { return 2 * Wide<D, NT>::kStages * Wide<D, NT>::kSide + (int)sizeof(WideTail<D, NT>) + 1024; }

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_wide_kernel(const __grid_constant__ AttnParams p) {
  using S = Wide<D, NT>;
  constexpr int kChunks = D / 16;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (base - smem_u32(smem_raw));   // keys' stages, values' stages, tail
  WideTail<D, NT>& T = *reinterpret_cast<WideTail<D, NT>*>(smem + 2 * S::kStages * S::kSide);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t k_ring = base + warp * S::kBoxBytes, v_ring = base + S::kStages * S::kSide;
  const uint32_t k_bar = smem_u32(&T.k_full[warp][0]), v_bar = smem_u32(&T.v_full[0]);
  if (lane == 0)
    for (int s = 0; s < S::kStages; ++s) mbar_init(k_bar + 8 * s, 1);
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(v_bar + 8 * s, kAttnWarps);
    T.failed = 0;
  }
  mbar_fence_init();
  pdl_launch_dependents();
  pdl_wait();
  Walk walk(p, S::kRows, T.line_warp, T.line_found);   // its barriers publish the mbarriers too
  const uint64_t pol = l2_evict_first();
  uint32_t phase_base = 0;   // tiles put through the rings
  bool dead = false;
  // this lane's ldmatrix rows: tokens 0-7 and 8-15 of one chunk, then of the next
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lchunk = lane >> 4;

  Segment sg = {};
  // ---- copies: this warp's 16 tokens of 32 tiles at a time, a tile a lane
  int n_tiles = 0, ids = -1, toks = 0;
  auto token_of = [&](int i) { return (sg.first + i) * kWideTile + warp * kBox; };
  auto look_up = [&](int i, int& block, int& tok) {
    block = -1;
    tok = 0;
    const int t = token_of(i);
    if (i < n_tiles && t < sg.rq.kv) {
      const int q = t / p.B;
      const int b = p.table[(size_t)sg.r * p.max_blocks + q];
      tok = t - q * p.B;
      block = b >= 0 && b < p.n_blocks ? b : -1;
    }
  };
  // Tile i's keys or values of this warp's tokens, by the whole warp. A batch is
  // looked up with its first keys; the values of the batch before are all on
  // their way by then.
  auto issue = [&](int i, bool values) {
    if (!values && (i & 31) == 0 && i > 0) look_up(i + lane, ids, toks);
    const int b = __shfl_sync(0xffffffffu, ids, i & 31), tok = __shfl_sync(0xffffffffu, toks, i & 31);
    if (lane == 0) {
      const int s = (int)((phase_base + i) % S::kStages);
      const uint32_t bar = (values ? v_bar : k_bar) + 8 * s;
      const uint32_t dst = values ? v_ring + s * S::kSide + warp * S::kBoxBytes : k_ring + s * S::kSide;
      if (b >= 0) {
        mbar_arrive_expect_tx(bar, S::kBoxBytes);
        tma_load_box(dst, values ? &p.v : &p.k, tok, sg.head, b, bar, pol);
      } else {
        mbar_arrive(bar);
      }
    }
  };
  struct Scales {
    float ks, lvs, rvs;   // ks -1: the block is not there
  };
  Scales sc_l = {-1.0f, 0.0f, 0.0f}, sc_n = sc_l;
  auto scales_of = [&](int b) {
    Scales s = {-1.0f, 0.0f, 0.0f};
    if (b >= 0) {
      const size_t at = (size_t)b * p.K + sg.head;
      s.ks = p.k_scale[at];
      const float vs = fminf(fmaxf(p.v_scale[at], 0x1p-60f), 0x1p60f);
      s.lvs = log2f(vs);
      s.rvs = 1.0f / vs;
    }
    return s;
  };
  uint16_t qx[NT][D / 32];
  auto open_segment = [&]() {
    n_tiles = sg.last - sg.first;
    look_up(lane, ids, toks);
    const int n_rows = min(sg.rq.rows * p.G - sg.row0, S::kRows);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int n = warp + k * kAttnWarps;
      if (n < n_rows) {
        const int j = (sg.row0 + n) / p.G, h = sg.head * p.G + (sg.row0 + n) % p.G;
        const uint16_t* src = p.q + (sg.rq.start + j) * p.q_row_stride + h * p.q_head_stride + lane;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qx[k][i] = src[32 * i];
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) qx[k][i] = 0;
      }
    }
    if (!dead) {
      for (int i = 0; i < min(n_tiles, S::kStages); ++i) {
        issue(i, false);
        if (i < S::kStages - 1) issue(i, true);
      }
    }
    sc_l = scales_of(ids);
  };
  // The query rows to f16, each scaled by a power of two; clears a NaN mask.
  auto store_queries = [&](int slot) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int n = warp + k * kAttnWarps;
      uint16_t* dst = reinterpret_cast<uint16_t*>(T.q + n * S::kQStride);
      float x[D / 32];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = __uint_as_float((uint32_t)qx[k][i] << 16);
        if (fabsf(x[i]) < INFINITY) top = fmaxf(top, fabsf(x[i]));
      }
      top = warp_max(top);
      const int e = top > 0.0f ? min(max(floor_log2_abs(top), -100), 126) : 0;
      const float f = exp2i(-e);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) dst[lane + 32 * i] = __half_as_ushort(__float2half_rn(x[i] * f));
      if (lane == 0) T.q_scale[n] = p.scale * kLog2e * exp2i(e);
    }
    for (int i = tid; i < D; i += kAttnThreads) T.nan_mask[slot][i] = 0;
  };

  bool more = walk.next(p, S::kRows, sg);
  int turn = 0;
  if (more) {
    open_segment();
    store_queries(0);
  }
  while (more) {
    __syncthreads();
    const Segment cur = sg;
    const Request& rq = cur.rq;
    const int row0 = cur.row0;
    const int n_group_rows = min(rq.rows * p.G - row0, S::kRows);
    const int seen0 = rq.kv - rq.rows;   // row j sees tokens <= seen0 + j
    uint32_t* const nan_mask = T.nan_mask[turn];
    const uint8_t* const q_frag = T.q + g * S::kQStride + t4 * 8;   // this lane's fragment of chunk 0, row g
    const uint8_t* const p_frag = T.p + lane * 8;
    float qs[NT][2], m[NT][2], l[NT][2];
    float o[S::kMT][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        qs[n][k] = T.q_scale[n * 8 + t4 * 2 + k];
        m[n][k] = kNone;
        l[n][k] = 0.0f;
      }
#pragma unroll
    for (int c = 0; c < S::kMT; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[c][n][k] = 0.0f;

    const int tiles = n_tiles;
    for (int i = 0; i < tiles; ++i) {
      const uint32_t it = phase_base + i;
      const int s = (int)(it % S::kStages), parity = (int)((it / S::kStages) & 1);
      const uint32_t ks_at = k_ring + s * S::kSide, vs_at = v_ring + s * S::kSide;
      const uint32_t v_own = vs_at + warp * S::kBoxBytes;
      // A wait that runs out: the warp goes on without waiting or copying, in
      // step with the barriers, and the result is reported as not valid.
      if (!dead && !mbar_wait_bounded(k_bar + 8 * s, parity, kAttnPolls)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if ((i & 31) == 16) {   // half a batch ahead
        int b, tok;
        look_up((i & ~31) + 32 + lane, b, tok);
        sc_n = scales_of(b);
      }
      if ((i & 31) == 0 && i > 0) sc_l = sc_n;
      const float ks = __shfl_sync(0xffffffffu, sc_l.ks, i & 31), lvs = __shfl_sync(0xffffffffu, sc_l.lvs, i & 31),
                  rvs = __shfl_sync(0xffffffffu, sc_l.rvs, i & 31);
      const int tok0 = token_of(i);
      const bool there = ks != -1.0f && !dead;
      // ---- S^T: this warp's 16 tokens x rows, as exponents
      float x[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[n][k] = there ? 0.0f : -INFINITY;
      if (there) {
        // a chunk's query fragments and the next two chunks' keys are asked for
        // before the chunk before is multiplied
        uint2 qb[2][NT];
        uint32_t w[2][4];
        ldsm_x4(ks_at + chunk_at<D>(lrow, lchunk), w[0]);
#pragma unroll
        for (int n = 0; n < NT; ++n) qb[0][n] = *reinterpret_cast<const uint2*>(q_frag + n * 8 * S::kQStride);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c + 1 < kChunks) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              qb[(c + 1) & 1][n] = *reinterpret_cast<const uint2*>(q_frag + n * 8 * S::kQStride + (c + 1) * 32);
          }
          if (c % 2 == 0 && c + 2 < kChunks) ldsm_x4(ks_at + chunk_at<D>(lrow, c + 2 + lchunk), w[(c / 2 + 1) & 1]);
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2x2(w[(c / 2) & 1][2 * (c & 1)], a0, a2);
          e4m3x4_to_f16x2x2(w[(c / 2) & 1][2 * (c & 1) + 1], a1, a3);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_free(x[n], a0, a1, a2, a3, qb[c & 1][n].x, qb[c & 1][n].y);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[n][k] = fmaf(x[n][k], ks * qs[n][k & 1], lvs);
      }
      const bool ragged = !there || tok0 + kBox - 1 > seen0;   // some rows do not see all 16
      if (ragged) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int lim = min(seen0 + (row0 + n * 8 + t4 * 2 + k) / p.G, rq.kv - 1);
            if (tok0 + g > lim) x[n][k] = -INFINITY;
            if (tok0 + g + 8 > lim) x[n][k + 2] = -INFINITY;
          }
      }
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) grew |= x[n][k] > m[n][k & 1] + 8.0f;
      // ---- barrier 1: the last tile's values and P are read, the keys are read
      const bool move = __syncthreads_or(grew);
      if (!dead) {
        if (i + S::kStages - 1 < tiles) issue(i + S::kStages - 1, true);
        if (i + S::kStages < tiles) issue(i + S::kStages, false);
      }
      if (move) {   // the same in every thread: new maxima, the same in every warp
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = fmaxf(x[n][k], x[n][k + 2]);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, y));
            if (g == 0) T.top[warp][n * 8 + t4 * 2 + k] = v;
          }
        __syncthreads();   // T.top is next written after another barrier 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float to = m[n][k];
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) to = fmaxf(to, T.top[w][n * 8 + t4 * 2 + k]);
            const float f = exp2_fast(m[n][k] - to);
            m[n][k] = to;
            l[n][k] *= f;
#pragma unroll
            for (int c = 0; c < S::kMT; ++c) {
              o[c][n][k] *= f;
              o[c][n][k + 2] *= f;
            }
          }
      }
      // ---- weights and their sums; P in the fragments of the second product
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float wv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) wv[k] = exp2_fast(x[n][k] - m[n][k & 1]);
        l[n][0] = fmaf(wv[0] + wv[2], rvs, l[n][0]);
        l[n][1] = fmaf(wv[1] + wv[3], rvs, l[n][1]);
        const __half2 h0 = __floats2half2_rn(wv[0], wv[1]), h1 = __floats2half2_rn(wv[2], wv[3]);
        const uint32_t b0 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h0));
        const uint32_t b1 = transpose_8x8(*reinterpret_cast<const uint32_t*>(&h1));
        *reinterpret_cast<uint2*>(T.p + (warp * NT + n) * 256 + lane * 8) = make_uint2(b0, b1);
      }
      if (!dead && !mbar_wait_bounded(v_bar + 8 * s, parity, kAttnPolls)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (ragged) {
        // Values no row or not every row may see: rows past the end, or without
        // a block, are zeroed (the memory may hold anything), and a NaN among the
        // rows' own tokens is taken out here and put back at the end for the rows
        // that do see it; 0 * NaN would reach the others.
        __syncwarp();
        for (int b = lane; b < kBox * (D / 4); b += 32) {
          const int tk = b / (D / 4), byte = (b % (D / 4)) * 4, own = tok0 + tk - seen0;
          if (there && own <= 0) continue;
          const uint32_t at = v_own + chunk_at<D>(tk, byte >> 4) + (byte & 15);
          uint32_t word;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(word) : "r"(at) : "memory");
          if (!there || tok0 + tk >= rq.kv) {
            word = 0;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (((word >> (8 * k)) & 0x7Fu) == 0x7Fu) {
                word &= ~(0xFFu << (8 * k));
                atomicOr(&nan_mask[byte + k], 1u << own);
              }
          }
          asm volatile("st.shared.u32 [%0], %1;" :: "r"(at), "r"(word) : "memory");
        }
        proxy_fence();   // before TMA writes the stage again
      }
      __syncthreads();   // ---- barrier 2: P is written
      // ---- O^T += V^T P^T over the tile's 128 tokens; m row g is dimension 2 g of a chunk, g + 8 is 2 g + 1
      // (fragments of the next box asked for before a box is multiplied)
      constexpr int kPer = 2 / S::kMT, kSteps = kAttnWarps / kPer;   // boxes a step: two chunks of one, or one of two
      auto v_at = [&](int w) {
        return S::kMT == 2 ? vs_at + w * S::kBoxBytes + chunk_at<D>(lrow, 2 * warp + lchunk)
                           : vs_at + (w * kPer + lchunk) * S::kBoxBytes + chunk_at<D>(lrow, warp);
      };
      uint32_t v[2][4];
      uint2 pb[2][NT];
      ldsm_x4_t(v_at(0), v[0]);
#pragma unroll
      for (int n = 0; n < NT; ++n) pb[0][n] = *reinterpret_cast<const uint2*>(p_frag + n * 256);
#pragma unroll
      for (int w = 0; w < kSteps; ++w) {
        if (w + 1 < kSteps) ldsm_x4_t(v_at(w + 1), v[(w + 1) & 1]);
        uint32_t a[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e4m3x4_to_f16x2x2(__byte_perm(v[w & 1][2 * h], 0, 0x3120), a[h][0], a[h][1]);
          e4m3x4_to_f16x2x2(__byte_perm(v[w & 1][2 * h + 1], 0, 0x3120), a[h][2], a[h][3]);
        }
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
          const int box = w * kPer + h;
          if (box + 1 < kAttnWarps) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              pb[(box + 1) & 1][n] = *reinterpret_cast<const uint2*>(p_frag + ((box + 1) * NT + n) * 256);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 b = pb[box & 1][n];
            if constexpr (S::kMT == 2) {
              mma_free(o[0][n], a[0][0], a[0][1], a[0][2], a[0][3], b.x, b.y);
              mma_free(o[1][n], a[1][0], a[1][1], a[1][2], a[1][3], b.x, b.y);
            } else {
              mma_free(o[0][n], a[h][0], a[h][1], a[h][2], a[h][3], b.x, b.y);
            }
          }
        }
      }
    }
    if (dead && lane == 0) {
      T.failed = 1;
      for (int s = 0; s < S::kStages; ++s) {   // the copies still on their way
        mbar_wait_bounded(k_bar + 8 * s, (int)((phase_base / S::kStages) & 1), kAttnPolls);
        mbar_wait_bounded(v_bar + 8 * s, (int)((phase_base / S::kStages) & 1), kAttnPolls);
      }
    }
    phase_base += tiles;

    // ---- the segment's end: the warps' sums, then each its dimensions
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[n][k] += __shfl_xor_sync(0xffffffffu, l[n][k], y);
        if (g == 0) T.l[warp][n * 8 + t4 * 2 + k] = l[n][k];
      }
    __syncthreads();
    more = walk.next(p, S::kRows, sg);
    if (more) {
      open_segment();
      store_queries(turn ^ 1);
    }
    const int slot = walk.cta * 2 + (cur.starts ? 1 : 0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = n * 8 + t4 * 2 + k;
        if (row >= n_group_rows) continue;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) sum += T.l[w][row];
        const int j = (row0 + row) / p.G, h = cur.head * p.G + (row0 + row) % p.G;
        const size_t at = (size_t)(rq.start + j) * p.H + h;
        const uint32_t see = (2u << j) - 1u;
        const float inv = cur.whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
#pragma unroll
        for (int c = 0; c < S::kMT; ++c) {
          const int d = (warp * S::kMT + c) * 16 + 2 * g;
          const float a = (nan_mask[d] & see) ? NAN : o[c][n][k] * inv, b = (nan_mask[d + 1] & see) ? NAN : o[c][n][k + 2] * inv;
          if (cur.whole) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            *reinterpret_cast<uint32_t*>(p.out + at * D + d) = *reinterpret_cast<const uint32_t*>(&v);
          } else {
            *reinterpret_cast<float2*>(p.part_o + ((size_t)slot * S::kRows + row) * D + d) = make_float2(a, b);
          }
        }
        if (warp == 0 && g == 0) {
          if (!cur.whole) p.part_ml[(size_t)slot * S::kRows + row] = make_float2(m[n][k], sum);
          else if (p.lse != nullptr) p.lse[at] = sum == 0.0f ? -INFINITY : (m[n][k] + log2f(sum)) * kLn2;
        }
      }
    turn ^= 1;
  }
  __syncthreads();
  if (tid == 0) p.failed[walk.cta] = T.failed;
}

template <int D, int NT>
cudaError_t launch_wide(const AttnParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, attn_wide_kernel<D, NT>, wide_smem<D, NT>());
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_ctas);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = wide_smem<D, NT>();
  cfg.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = a;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_wide_kernel<D, NT>, p);
}

}  // namespace

cudaError_t launch_attn_wide(int D, int nt, const AttnParams& p, cudaStream_t st) {
  if (D == 256 && nt == 4) return launch_wide<256, 4>(p, st);
  if (D == 256 && nt == 6) return launch_wide<256, 6>(p, st);
  if (D == 256 && nt == 8) return launch_wide<256, 8>(p, st);
  if (D == 128 && nt == 6) return launch_wide<128, 6>(p, st);
  if (D == 128 && nt == 8) return launch_wide<128, 8>(p, st);
  return cudaErrorInvalidValue;
}

}  // namespace bws

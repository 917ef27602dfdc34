// Attention over the 8-bit cache for many query rows a kv head (a verify pass
// of several tokens, wide groups): the mathematics and the line of shares are
// those of kv_attention.cu, the CTA's work is cut the other way.
//
// mma.sync would set the time here: m16n8k16 keeps its pipe for 16 cycles of a
// quarter SM, 67 us for both products of 48 rows of 256 over 100001 tokens, and
// three arrangements of eight or sixteen warps all took 82 to 89 us. So the scores
// go to the fifth-generation tensor cores, which take the keys as they are:
// S^T = K Q^T as tcgen05.mma kind::f8f6f4 of M = 128 cached tokens, K's 128-byte
// swizzled panels straight from TMA. A query row, scaled by a power of two to
// 128..256 at its largest, is two E4M3 numbers, hi and 2^5 (q - hi): exact for
// BF16 down to 2^-14 of the row's largest, off by 2^-22 of it below. Both stand
// side by side in the N side (hi rows, then lo rows) and in TMEM, and are added
// in FP32. The values' product stays on mma.sync in f16: weights in E4M3, of
// however many parts on one scale, would drop what lies 2^-18 below a row's
// largest, which over a long context can be a tenth of its sum.
//
// Roles, one CTA of sixteen warps an SM, along the tiles of 128 cached tokens:
// warps 0-7 take a token and half the rows a thread (a TMEM lane's columns), form
// the exponents and the weights P; warps 8-15 take an eighth of
// the dimensions each and add V^T P^T to their registers, one of them also
// issues the scores' products two tiles ahead, and each copies a box of keys and
// values.
// mbarriers with bounded waits join them; a wait that runs out marks the result
// and goes on. One running maximum per row serves the CTA: it follows only past a
// margin, on which warps 0-7 vote, so most tiles exchange no maxima.
// Bound: the chain of a tile, 4900 cycles at 48 rows of 256, of which the values'
// mma.sync needs 3100 at 16 a quarter SM and HBM 2750: 100001 tokens of four kv
// heads, 205 MB, take 67 us with the join (3.0 TB/s, 292 TFLOP/s). A segment costs
// 8 to 10 us beside its tokens: its first tile passes every stage alone, through
// code that is fetched anew.
#include <atomic>

#include "copy_ring.h"
#include "kv_attention.cuh"
#include "kv_cache.cuh"

namespace bws {
namespace {

constexpr int kSoftWarps = 8, kValueWarps = 8, kQuads = 4;   // a quad: 32 tokens, two of warps 0-7
constexpr int kMmaWarp = 7;                                  // of the value warps
constexpr int kWideThreads = 32 * (kSoftWarps + kValueWarps);
constexpr int kBoxes = kWideTile / kBox;
constexpr int kTmemCols = 256;               // two buffers of 128 columns
constexpr int kBarSoft = 1;                  // named barrier of warps 0-7
constexpr float kLoScale = 1.0f / 32.0f;     // a query's low part is held times 2^5

template <int D, int NT>
struct Wide {
  static constexpr int kRows = 8 * NT;
  static constexpr int kPanels = D / 128;
  static constexpr int kPanel = kWideTile * 128;              // bytes: 128 tokens' 128 dimensions
  static constexpr int kSide = kPanels * kPanel;              // a tile's keys, or values
  static constexpr int kBoxBytes = kBox * D;
  // Keys are scored two tiles ahead of their weights' use, so a stage more of
  // them keeps HBM's latency off that chain (eight tiles of rows leave no room).
  static constexpr int kVStages = D == 256 ? 2 : 4;
  static constexpr int kKStages = D == 256 ? (NT <= 6 ? 3 : 2) : 4;
  static constexpr int kQPanel = 2 * kRows * 128;             // hi rows, then lo rows
  static constexpr int kPStride = 16 * NT + 16;               // bytes of a token's weights: eight tokens on all banks
  static constexpr int kMT = D / 16 / kValueWarps;            // m tiles of O^T a value warp holds
  // D FP32, A and B E4M3, both K-major, N = 2 kRows, M = 128
  static constexpr uint32_t kIdesc = (1u << 4) | ((2u * kRows >> 3) << 17) | ((128u >> 4) << 24);
};

template <int D, int NT>
struct __align__(1024) WideTail {
  uint8_t q[Wide<D, NT>::kPanels][Wide<D, NT>::kQPanel];      // swizzled as the keys are
  uint8_t p[2][kWideTile * Wide<D, NT>::kPStride];
  alignas(16) float2 row[8 * NT];   // scale (with log2 e and the row's power of two), what exponents are taken less, or 0
  uint32_t fresh[2];           // bit r: row r has seen no token yet, and its maximum stands for nothing
  float up[8 * NT];            // how far the maxima went in a tile that moved them
  float top[kQuads][8 * NT];
  float l[kQuads][8 * NT];
  float m[8 * NT];             // the segment's final maxima
  float factor[2][8 * NT];     // what O shrinks by before the tile, where moved is set
  uint32_t moved[2];
  uint32_t nan_mask[2][D];
  unsigned long long k_full[Wide<D, NT>::kKStages];
  unsigned long long v_full[Wide<D, NT>::kVStages], v_free[Wide<D, NT>::kVStages];
  unsigned long long s_full[2], p_full[2], p_free[2], drain;
  long long line_warp[kSoftWarps + kValueWarps];
  long long line_found[2];
  // the CTA's way along its share and its segments, kept here by thread 0
  Walk walk;
  Segment seg[2];
  int more;
  uint32_t started[kSoftWarps + kValueWarps];   // tiles whose box a warp has started to copy
  uint32_t tmem;
  uint32_t status;
};

template <int D, int NT>
constexpr int wide_smem() { return (Wide<D, NT>::kKStages + Wide<D, NT>::kVStages) * Wide<D, NT>::kSide + (int)sizeof(WideTail<D, NT>) + 1024; }

// Shared-memory descriptor of a K-major operand of 128-byte swizzled rows.
BWS_DEV uint64_t operand(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
BWS_DEV void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
BWS_DEV void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
BWS_DEV void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
BWS_DEV void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// This thread's lane of eight columns, twice (hi and lo of eight rows).
BWS_DEV void load_scores(uint32_t hi_at, uint32_t lo_at, uint32_t* a, uint32_t* b) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7])
               : "r"(hi_at) : "memory");
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7])
               : "r"(lo_at) : "memory");
}
BWS_DEV void wait_scores(uint32_t* a, uint32_t* b) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :: "memory");
}
// A box of 16 tokens' panel of 128 dimensions.
BWS_DEV void tma_load_panel(uint32_t dst, const void* tmap, int token, int panel, int head, int block, uint32_t bar,
                            uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;"
      :: "r"(dst), "l"(tmap), "r"(0), "r"(token), "r"(panel), "r"(head), "r"(block), "r"(bar), "l"(pol) : "memory");
}
// Byte offset of 16-byte chunk `c` of a token's row in a tile's side.
BWS_DEV uint32_t tile_chunk_at(int token, int c) {
  return (c >> 3) * (kWideTile * 128) + token * 128 + (((c & 7) ^ (token & 7)) << 4);
}

template <int D, int NT>
__global__ void __launch_bounds__(kWideThreads, 1) attn_wide_kernel(const __grid_constant__ AttnParams p) {
  using S = Wide<D, NT>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (base - smem_u32(smem_raw));   // keys' stages, values' stages, tail
  WideTail<D, NT>& T = *reinterpret_cast<WideTail<D, NT>*>(smem + (S::kKStages + S::kVStages) * S::kSide);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t k_ring = base, v_ring = base + S::kKStages * S::kSide;
  const uint32_t k_full = smem_u32(T.k_full), v_full = smem_u32(T.v_full), v_free = smem_u32(T.v_free),
                 s_full = smem_u32(T.s_full), p_full = smem_u32(T.p_full), p_free = smem_u32(T.p_free);
  const uint64_t pol = l2_evict_first();
  if (warp == kSoftWarps + kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&T.tmem)),
                 "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (lane == 0) T.started[warp] = 0;
  if (tid == 0) {
    for (int s = 0; s < S::kKStages; ++s) mbar_init(k_full + 8 * s, kBoxes);
    for (int s = 0; s < S::kVStages; ++s) {
      mbar_init(v_full + 8 * s, kBoxes);
      mbar_init(v_free + 8 * s, kValueWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full + 8 * b, 1);
      mbar_init(p_full + 8 * b, kSoftWarps);
      mbar_init(p_free + 8 * b, kValueWarps);
    }
    mbar_init(smem_u32(&T.drain), 1);
    T.status = 0;
    mbar_fence_init();
  }
  fence_before();
  pdl_launch_dependents();
  pdl_wait();
  {
    Walk walk;
    walk.start(p, S::kRows, T.line_warp, T.line_found, &T.status);   // its barriers publish the mbarriers and the TMEM address too
    if (tid == 0) {
      T.walk = walk;
      T.more = T.walk.next(p, S::kRows, T.seg[0]);
    }
  }
  __syncthreads();
  fence_after();
  const uint32_t tmem = T.tmem;
  uint32_t phase_base = 0;   // tiles gone by
  bool dead = false;         // of this warp's lanes alike
  int turn = 0;
  // The (it / n)-th use of barrier it % n.
  auto wait_for = [&](uint32_t bars, uint32_t it, int n, bool freed) {
    const uint32_t use = it / n;
    if (freed && use == 0) return;   // nothing was there before
    const uint32_t bar = bars + 8 * (it % n), parity = (freed ? use - 1 : use) & 1;
    if (dead || __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    dead = __any_sync(0xffffffffu, !mbar_wait_bounded(bar, parity, kAttnPolls));
  };
  // Block and first token of box b of tile i of the segment; block -1: not there.
  auto look_up = [&](int i, int b, int& block, int& tok) {
    const Segment& sg = T.seg[turn];
    block = -1;
    tok = 0;
    // (unsigned: asked past the end too, and the last tile may end at 2^31)
    const uint32_t t = (uint32_t)(sg.first + i) * kWideTile + b * kBox;
    if (i < sg.last - sg.first && t < (uint32_t)sg.rq.kv(p)) {
      const int q = block_index(p, t);
      const int id = p.table[(size_t)sg.r * p.max_blocks + q];
      tok = t - q * p.B;
      block = id >= 0 && id < p.n_blocks ? id : -1;
    }
  };
  // The segment's query rows as E4M3 pairs, a warp of 0-7 a row; clears a NaN mask.
  auto store_queries = [&]() {
    constexpr int E = D / 32;   // neighbouring values a lane
    const Segment& sg = T.seg[turn];
    const int n_rows = min(sg.rq.rows(p) * p.G - sg.row0, S::kRows);
    // Every row is asked for before the first is used; lane r knows where the r-th
    // lies. The rows are then converted by one rolled loop, whose instructions
    // are fetched once.
    uint2 raw[NT][E / 4];
    const int of_lane = min(warp + lane * kSoftWarps, max(n_rows - 1, 0));
    const int of_j = (sg.row0 + of_lane) / p.G, of_h = sg.head * p.G + (sg.row0 + of_lane) - of_j * p.G;
    const long long at_lane = (sg.rq.start + of_j) * p.q_row_stride + of_h * p.q_head_stride;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const uint16_t* src = p.q + __shfl_sync(0xffffffffu, at_lane, r) + lane * E;
      const bool live = warp + r * kSoftWarps < n_rows;
#pragma unroll
      for (int i = 0; i < E / 4; ++i) raw[r][i] = live ? *reinterpret_cast<const uint2*>(src + 4 * i) : make_uint2(0u, 0u);
    }
#pragma unroll 1
    for (int n = warp; n < S::kRows; n += kSoftWarps) {
      float x[E];
      float top = 0.0f;
      bool bad = false;   // an infinity would saturate: a row that holds one is all NaN, as its scores are
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        x[4 * i] = __uint_as_float(raw[0][i].x << 16);
        x[4 * i + 1] = __uint_as_float(raw[0][i].x & 0xFFFF0000u);
        x[4 * i + 2] = __uint_as_float(raw[0][i].y << 16);
        x[4 * i + 3] = __uint_as_float(raw[0][i].y & 0xFFFF0000u);
#pragma unroll
        for (int r = 0; r + 1 < NT; ++r) raw[r][i] = raw[r + 1][i];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        bad |= !(fabsf(x[i]) < INFINITY);
        top = fmaxf(top, fabsf(x[i]));
      }
      top = warp_max(top);
      bad = __any_sync(0xffffffffu, bad);
      const int e = top > 0.0f && !bad ? min(max(floor_log2_abs(top), -100), 126) - 7 : 0;
      const float f = exp2i(-e);
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        uint32_t hi = 0, lo = 0;
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float a = x[i + k] * f, b = x[i + k + 1] * f;
          const uint32_t h2 = f32x2_to_e4m3x2(b, a);
          const uint32_t back = e4m3x2_to_f16x2(h2);
          const float2 r2 = __half22float2(*reinterpret_cast<const __half2*>(&back));
          hi |= h2 << (8 * k);
          lo |= f32x2_to_e4m3x2((b - r2.y) * 32.0f, (a - r2.x) * 32.0f) << (8 * k);
        }
        if (bad) hi = lo = 0x7F7F7F7Fu;
        const int d = lane * E + i, c = (d & 127) >> 4;
        uint8_t* at = T.q[d >> 7] + n * 128 + ((c ^ (n & 7)) << 4) + (d & 15);
        *reinterpret_cast<uint32_t*>(at) = hi;
        *reinterpret_cast<uint32_t*>(at + S::kRows * 128) = lo;   // kRows is a multiple of 8: the same swizzle
      }
      if (lane == 0) T.row[n] = make_float2(p.scale * kLog2e * exp2i(e), 0.0f);
    }
    for (int i = tid; i < D; i += 32 * kSoftWarps) T.nan_mask[turn][i] = 0;
    if (tid < 2) T.fresh[tid] = S::kRows >= 32 * (tid + 1) ? 0xffffffffu : (1u << (S::kRows & 31)) - 1u;
    proxy_fence();   // the tensor cores read the queries
  };
  // One lane's box (its block and first token) of a tile into stage s.
  auto copy_box = [&](uint32_t bars, uint32_t ring, const CUtensorMap* map, int s, int b, int block, int tok) {
    const uint32_t bar = bars + 8 * s, dst = ring + s * S::kSide + b * (kBox * 128);
    if (block >= 0) {
      mbar_arrive_expect_tx(bar, S::kBoxBytes);
#pragma unroll
      for (int x = 0; x < S::kPanels; ++x)
        tma_load_panel(dst + x * S::kPanel, map, tok, x, T.seg[turn].head, block, bar, pol);
    } else {
      mbar_arrive(bar);
    }
  };
  // Each warp copies a box, its first lane: warps 0-7 the keys', the value warps
  // the values'. (A copy takes about 90 cycles to issue: all sixteen boxes' 32
  // panels from one warp took 2900 of a tile's 5800 cycles.)
  const bool keys = warp < kSoftWarps, copies = lane == 0;
  const int my_box = warp & (kBoxes - 1);
  const uint32_t my_bars = keys ? k_full : v_full, my_ring = keys ? k_ring : v_ring, my_stages = keys ? S::kKStages : S::kVStages;
  auto open_copies = [&]() {
    constexpr int kMost = S::kKStages > S::kVStages ? S::kKStages : S::kVStages;
    const int ahead = min(T.seg[turn].last - T.seg[turn].first, (int)my_stages);
    if (!dead && copies) {
      int block[kMost], tok[kMost];
#pragma unroll
      for (int i = 0; i < kMost; ++i) look_up(i, my_box, block[i], tok[i]);
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (i < ahead)
          copy_box(my_bars, my_ring, keys ? &p.k : &p.v, (int)((phase_base + i) % my_stages), my_box, block[i], tok[i]);
      T.started[warp] = phase_base + ahead;
    }
    __syncwarp();
  };

  bool more = T.more != 0;
  if (more) {
    open_copies();
    if (warp < kSoftWarps) store_queries();
  }
  while (more) {
    __syncthreads();
    const Segment& cur = T.seg[turn];
    const Request& rq = cur.rq;
    const int tiles = cur.last - cur.first;
    uint32_t* const nan_mask = T.nan_mask[turn];
    float o[S::kMT][NT][4];              // the value warps'
    const int g = lane >> 2, t4 = lane & 3;

    if (warp < kSoftWarps) {
      // ---- a token and half the rows a thread: exponents and weights
      constexpr int kHalf = 4 * NT;
      const int quad = warp & 3, row_a = (warp >> 2) * kHalf, token = quad * 32 + lane;
      float l[kHalf];    // this thread's tokens' sums
#pragma unroll
      for (int n = 0; n < kHalf; ++n) l[n] = 0.0f;
      // This thread's box: its block is asked for two tiles ahead, its scales one.
      auto block_of = [&](int i) {
        int b, tok;
        look_up(i, token / kBox, b, tok);
        return b;
      };
      auto scales_of = [&](int b, float& ks, float& vs) {
        ks = -1.0f;   // the block is not there
        vs = 1.0f;
        if (b >= 0) {
          const size_t at = (size_t)b * p.K + cur.head;
          ks = p.k_scale[at];
          vs = p.v_scale[at];
        }
      };
      int next_block = -1, next_tok = 0;   // of the next keys to copy
      if (copies) look_up(S::kKStages, my_box, next_block, next_tok);
      float ks_n, vs_n;
      int block_n = block_of(1);
      scales_of(block_of(0), ks_n, vs_n);
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        const int buf = (int)(it & 1);
        const float ks = ks_n, vs = fminf(fmaxf(vs_n, 0x1p-60f), 0x1p60f);
        scales_of(block_n, ks_n, vs_n);
        block_n = block_of(i + 2);
        const float lvs = log2f(vs), rvs = 1.0f / vs;
        const int tok = (cur.first + i) * kWideTile + token, own = min(tok - rq.seen0(), 31);   // row j sees tokens <= seen0 + j
        const bool there = ks != -1.0f && tok < rq.kv(p);
        // rows below `hidden` do not see the token: the j-th token of the rows'
        // own is seen from row j on
        const int hidden = !there ? S::kRows : own > 0 ? min(max(own * p.G - cur.row0, 0), S::kRows) : 0;
        const bool ragged = __any_sync(0xffffffffu, !there || own > 0);
        wait_for(s_full, it, 2, false);
        fence_after();
        const uint32_t s_at = tmem + buf * 128 + ((uint32_t)(32 * quad) << 16) + row_a;
        const float2* const rows = T.row + row_a;
        // exponents of every row, less what stands for its maximum
        float x[kHalf];
        float top = -INFINITY;
        uint32_t hi[kHalf], lo[kHalf];
#pragma unroll
        for (int n = 0; n < kHalf; n += 8) load_scores(s_at + n, s_at + S::kRows + n, hi + n, lo + n);
#pragma unroll
        for (int n = 0; n < kHalf; n += 8) wait_scores(hi + n, lo + n);
#pragma unroll
        for (int n = 0; n < kHalf; n += 2) {
          const float4 row = *reinterpret_cast<const float4*>(rows + n);
          x[n] = fmaf(fmaf(__uint_as_float(lo[n]), kLoScale, __uint_as_float(hi[n])), ks * row.x, lvs - row.y);
          x[n + 1] = fmaf(fmaf(__uint_as_float(lo[n + 1]), kLoScale, __uint_as_float(hi[n + 1])), ks * row.z, lvs - row.w);
        }
        fence_before();
        if (ragged) {
#pragma unroll
          for (int n = 0; n < kHalf; ++n)
            if (row_a + n < hidden) x[n] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < kHalf; ++n) top = fmaxf(top, x[n]);
        const bool grew = top > kTop || ((T.fresh[0] | T.fresh[1]) != 0u && top != -INFINITY);
        uint32_t any;
        asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
                     : "=r"(any) : "r"((uint32_t)grew), "n"(kBarSoft), "n"(32 * kSoftWarps) : "memory");
        wait_for(p_free, it, 2, true);   // the value warps are done with P and the factors of the tile before last
        if (any != 0u) {                 // new maxima
#pragma unroll
          for (int n = 0; n < kHalf; ++n) {
            const float v = warp_max(x[n]);
            if (lane == n) T.top[quad][row_a + n] = v;
          }
          named_bar_sync(kBarSoft, 32 * kSoftWarps);
          if (tid < 64) {
            const bool row = tid < S::kRows, fresh = row && ((T.fresh[warp] >> lane) & 1u) != 0u;
            float up = -INFINITY;
            if (row)
              for (int w = 0; w < kQuads; ++w) up = fmaxf(up, T.top[w][tid] - (kTop - kMargin));
            const bool still = fresh && up == -INFINITY;
            if (!fresh || still) up = fmaxf(up, 0.0f);
            if (row) {
              T.row[tid].y += up;
              T.up[tid] = up;
              T.factor[buf][tid] = fresh ? 1.0f : exp2_fast(-up);   // a fresh row's O and sum are 0
            }
            const unsigned left = __ballot_sync(0xffffffffu, still);
            if (lane == 0) T.fresh[warp] = left;
          }
          named_bar_sync(kBarSoft, 32 * kSoftWarps);
#pragma unroll
          for (int n = 0; n < kHalf; ++n) {
            x[n] -= T.up[row_a + n];
            l[n] *= T.factor[buf][row_a + n];
          }
        }
        if (tid == 0) T.moved[buf] = any;
        uint8_t* const p_row = T.p[buf] + token * S::kPStride + 2 * row_a;
#pragma unroll
        for (int n = 0; n < kHalf; n += 8) {
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float a = exp2_fast(x[n + k]), b = exp2_fast(x[n + k + 1]);
            l[n + k] = fmaf(a, rvs, l[n + k]);
            l[n + k + 1] = fmaf(b, rvs, l[n + k + 1]);
            const __half2 h2 = __floats2half2_rn(a, b);
            h[k / 2] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          *reinterpret_cast<uint4*>(p_row + 2 * n) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (ragged) {
          // Values no row or not every row may see: rows past the end, or without
          // a block, are zeroed (the memory may hold anything), and a NaN among
          // the rows' own tokens is taken out here and put back at the end for
          // the rows that do see it; 0 * NaN would reach the others.
          wait_for(v_full, it, S::kVStages, false);
          const uint32_t side = v_ring + (uint32_t)(it % S::kVStages) * S::kSide;
          // the quad's two warps take its tokens in turn, a word a lane
          unsigned todo = __ballot_sync(0xffffffffu, !there || own > 0);
          const unsigned live = __ballot_sync(0xffffffffu, there);
          todo &= warp < kQuads ? 0x55555555u : 0xAAAAAAAAu;
          while (todo != 0u) {
            const int tk = __ffs(todo) - 1;
            todo &= todo - 1;
            const int its = (cur.first + i) * kWideTile + quad * 32 + tk - rq.seen0();
#pragma unroll
            for (int byte = 4 * lane; byte < D; byte += 128) {
              const uint32_t at = side + tile_chunk_at(quad * 32 + tk, byte >> 4) + (byte & 15);
              uint32_t word = 0;
              if ((live >> tk) & 1u) {
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(word) : "r"(at) : "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (((word >> (8 * k)) & 0x7Fu) == 0x7Fu) {
                    word &= ~(0xFFu << (8 * k));
                    atomicOr(&nan_mask[byte + k], 1u << min(its, 31));
                  }
              }
              asm volatile("st.shared.u32 [%0], %1;" :: "r"(at), "r"(word) : "memory");
            }
          }
          proxy_fence();   // before TMA writes the stage again
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full + 8 * buf);
          // the tile's products have read its keys: the next into their place
          if (!dead && i + S::kKStages < tiles) {
            copy_box(k_full, k_ring, &p.k, (int)(it % S::kKStages), my_box, next_block, next_tok);
            T.started[warp] = it + S::kKStages + 1;
          }
          look_up(i + S::kKStages + 1, my_box, next_block, next_tok);
        }
        __syncwarp();
      }
#pragma unroll
      for (int n = 0; n < kHalf; ++n) {
        const float v = warp_sum(l[n]);
        if (lane == n) T.l[quad][row_a + n] = v;
      }
      if (tid < S::kRows) T.m[tid] = ((T.fresh[warp] >> lane) & 1u) != 0u ? kNone : T.row[tid].y;
    } else {
      // ---- O^T += V^T P^T, an eighth of the dimensions; m row g is dimension 2 g
      // of a chunk, g + 8 is 2 g + 1
      const int vw = warp - kSoftWarps;
      const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lhalf = lane >> 4;   // this lane's ldmatrix row
#pragma unroll
      for (int c = 0; c < S::kMT; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[c][n][k] = 0.0f;
      auto score = [&](int i) {   // the whole warp: tile i's scores into their buffer, which is free
        const uint32_t it = phase_base + i;
        wait_for(k_full, it, S::kKStages, false);
        if (!dead && lane == 0) {
          fence_after();
          const uint32_t d = tmem + (it & 1) * 128, keys_at = k_ring + (it % S::kKStages) * S::kSide;
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_scores(d, operand(keys_at + (k >> 2) * S::kPanel + (k & 3) * 32),
                       operand(smem_u32(T.q[k >> 2]) + (k & 3) * 32), S::kIdesc, k > 0);
          commit(s_full + 8 * (it & 1));
        }
        __syncwarp();
      };
      if (vw == kMmaWarp)
        for (int i = 0; i < min(tiles, 2); ++i) score(i);
      // Values are copied while the tile's weights are awaited, a stage less than
      // the ring: the value warps have left that place by then.
      int next_block = -1, next_tok = 0;   // of the next box to copy
      if (copies) look_up(S::kVStages, my_box, next_block, next_tok);
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        const int s = (int)(it % S::kVStages), buf = (int)(it & 1);
        if (i > 0) {
          wait_for(v_free, it + S::kVStages - 1, S::kVStages, true);
          if (copies) {
            if (!dead && i + S::kVStages - 1 < tiles) {
              copy_box(v_full, v_ring, &p.v, (int)((it + S::kVStages - 1) % S::kVStages), my_box, next_block, next_tok);
              T.started[warp] = it + S::kVStages;
            }
            look_up(i + S::kVStages, my_box, next_block, next_tok);
          }
          __syncwarp();
        }
        wait_for(p_full, it, 2, false);
        if (vw == kMmaWarp && i + 2 < tiles) score(i + 2);   // P is there: its scores are read
        wait_for(v_full, it, S::kVStages, false);
        if (T.moved[buf] != 0u) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float f = T.factor[buf][n * 8 + t4 * 2 + k];
#pragma unroll
              for (int c = 0; c < S::kMT; ++c) {
                o[c][n][k] *= f;
                o[c][n][k + 2] *= f;
              }
            }
        }
        const uint32_t vs_at = v_ring + s * S::kSide;
        const uint32_t p_at = smem_u32(T.p[buf]) + lrow * S::kPStride + lhalf * 16;
        constexpr int kPer = 2 / S::kMT;   // boxes a step: two chunks of one, or one of two
#pragma unroll
        for (int w = 0; w < kBoxes; w += kPer) {
          uint32_t v[4];
          ldsm_x4_t(vs_at + (S::kMT == 2 ? tile_chunk_at(w * kBox + lrow, 2 * vw + lhalf)
                                         : tile_chunk_at((w + lhalf) * kBox + lrow, vw)), v);
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            e4m3x4_to_f16x2x2(__byte_perm(v[2 * h], 0, 0x3120), a[h][0], a[h][1]);
            e4m3x4_to_f16x2x2(__byte_perm(v[2 * h + 1], 0, 0x3120), a[h][2], a[h][3]);
          }
#pragma unroll
          for (int h = 0; h < kPer; ++h)
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
              uint32_t b[4];   // fragments of two tiles of rows
              ldsm_x4_t(p_at + (w + h) * kBox * S::kPStride + n * 16, b);
              if constexpr (S::kMT == 2) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  mma_free(o[c][n], a[c][0], a[c][1], a[c][2], a[c][3], b[0], b[1]);
                  mma_free(o[c][n + 1], a[c][0], a[c][1], a[c][2], a[c][3], b[2], b[3]);
                }
              } else {
                mma_free(o[0][n], a[h][0], a[h][1], a[h][2], a[h][3], b[0], b[1]);
                mma_free(o[0][n + 1], a[h][0], a[h][1], a[h][2], a[h][3], b[2], b[3]);
              }
            }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_free + 8 * s);
          mbar_arrive(p_free + 8 * buf);
        }
      }
    }
    if (dead && lane == 0) {
      atomicOr(&T.status, (uint32_t)BWS_STATUS_WAIT_TIMEOUT);
      // this warp's copies still on their way; it starts no more
      const uint32_t started = T.started[warp];
      for (uint32_t it = ring_oldest(started, my_stages); it < started; ++it)
        mbar_wait_bounded(my_bars + 8 * ring_stage(it, my_stages), ring_parity(it, my_stages), kAttnPolls);
      T.started[warp] = 0;
    }
    phase_base += tiles;
    if (tid == 0) T.more = T.walk.next(p, S::kRows, T.seg[turn ^ 1]);
    __syncthreads();   // the rows' sums and maxima, and the next segment, are there

    // ---- the segment's end, and the next one's start
    more = T.more != 0;
    turn ^= 1;
    if (more) open_copies();
    if (warp < kSoftWarps) {
      if (more) store_queries();
    } else {
      const int vw = warp - kSoftWarps, row0 = cur.row0, n_group_rows = min(rq.rows(p) * p.G - row0, S::kRows);
      const int slot = blockIdx.x * 2 + (cur.starts ? 1 : 0);
      const bool whole = cur.whole;
      // A row's place, factor and sight are formed by a lane of their own and
      // shuffled to those that hold the row: this code runs once a segment, and
      // formed by each for its rows (divisions, sums, twelve times over) it was
      // the fetching of its instructions that took 12000 cycles.
      constexpr int kSets = (S::kRows + 31) / 32;
      long long place[kSets];
      float factor[kSets];
      uint32_t see[kSets];
#pragma unroll
      for (int q = 0; q < kSets; ++q) {
        const int row = q * 32 + lane, live = min(row, n_group_rows - 1);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kQuads; ++w) sum += T.l[w][live];
        const int j = (row0 + live) / p.G, h = cur.head * p.G + (row0 + live) - j * p.G;
        const long long at = (long long)(rq.start + j) * p.H + h, part = (long long)slot * S::kRows + live;
        place[q] = (whole ? at : part) * D;
        factor[q] = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
        see[q] = (2u << j) - 1u;
        if (vw == 0 && row < n_group_rows) {
          if (!whole) p.part_ml[part] = make_float2(T.m[row], sum);
          else if (p.lse != nullptr) p.lse[at] = sum == 0.0f ? -INFINITY : (T.m[row] + log2f(sum)) * kLn2;
        }
      }
      constexpr int kOwn = S::kMT * 16;   // this warp's dimensions
      if (__any_sync(0xffffffffu, lane < kOwn && nan_mask[vw * kOwn + (lane & (kOwn - 1))] != 0u)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t sight = __shfl_sync(0xffffffffu, see[n / 4], (n & 3) * 8 + t4 * 2 + k);
#pragma unroll
            for (int c = 0; c < S::kMT; ++c) {
              const int d = vw * kOwn + c * 16 + 2 * g;
              if (nan_mask[d] & sight) o[c][n][k] = NAN;
              if (nan_mask[d + 1] & sight) o[c][n][k + 2] = NAN;
            }
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int from = (n & 3) * 8 + t4 * 2 + k;
          const long long at = __shfl_sync(0xffffffffu, place[n / 4], from) + vw * kOwn + 2 * g;
          const float f = __shfl_sync(0xffffffffu, factor[n / 4], from);
          if (n * 8 + t4 * 2 + k >= n_group_rows) continue;
#pragma unroll
          for (int c = 0; c < S::kMT; ++c) {
            const float a = o[c][n][k] * f, b = o[c][n][k + 2] * f;
            if (whole) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
              *reinterpret_cast<uint32_t*>(p.out + at + c * 16) = *reinterpret_cast<const uint32_t*>(&v);
            } else {
              *reinterpret_cast<float2*>(p.part_o + at + c * 16) = make_float2(a, b);
            }
          }
        }
    }
  }
  __syncthreads();
  if (tid == 0) p.failed[blockIdx.x] = T.status;
  if (warp == kSoftWarps + kMmaWarp) {   // every product has finished before the columns are released
    if (lane == 0) {
      commit(smem_u32(&T.drain));
      mbar_wait_bounded(smem_u32(&T.drain), 0, kAttnPolls);
    }
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

template <int D, int NT>
cudaError_t launch_wide(const AttnParams& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  const cudaError_t e = set_smem_once(attr, attn_wide_kernel<D, NT>, wide_smem<D, NT>());
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_wide_kernel<D, NT>, dim3((unsigned)p.n_ctas), kWideThreads, wide_smem<D, NT>(), st, p);
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

// Attention over the 4-bit cache for many query rows a kv head (a verify pass of
// several tokens, wide groups): the mathematics and the line of shares are those of
// kv4_attention.cu, both products run on the fifth-generation tensor cores.
//
// Scores. The keys are an operand as they lie: S^T = K Q^T as tcgen05.mma
// kind::mxf4nvf4 of M = 128 cached tokens, E2M1 codes straight from TMA, a scale for
// every 16 dimensions in TMEM. The queries have to come in the same format: a row,
// scaled by a power of two, is a sum of kPlanes rows of it, each the format's
// rounding of what the ones before leave, so that a value is off by 2^-15 of its 16's
// largest (a plane leaves 1/6 and a little) or 2^-21 of its row's, whichever is more.
// Planes stand side by side in N by twos, the pairs are added by the tensor cores, the
// two in FP32 by the reader.
// Values. A code times its scale is exact in f16 (six bits): four warps write parts
// of a tile to shared memory as the transposed operand, and O^T += V^T P^T is
// kind::f16 of M = 128 dimensions with O in TMEM; weights are f16 as in the other
// kernel. Where maxima move past their margin the values' warps rescale O in place.
//
// Roles, one CTA of sixteen warps an SM, along the tiles of 128 cached tokens: warps
// 0-7 take a token and half the rows a thread (a TMEM lane's columns) and form exponents
// and weights; warps 8-11 convert the values; two issue a product each, a tile's scores
// ahead of the weights of the tile before; two copy, keys with their scales and values.
// mbarriers with bounded waits join them; a wait that runs out marks the result and goes on.
//
// Bound: a tile's chain. 8 rows of 6 heads over 100001 tokens take 55.0 us, 20.7 tiles a
// CTA of some 3300 cycles each: scores to weights all of them (of it 490 for new maxima
// and 680 of waits for the sum, which waits while O is rescaled), the values' conversion
// 2200 beside and 840 more where O is rescaled, both products 2300 if shared memory gave
// 128 bytes a cycle (it feeds every operand); the start (queries to planes) 10,000, the end
// 5,000. Two planes instead of six would save 3 us, a quarter of the conversion 4. Steps:
// a thread's keys' scales to TMEM and fourteen warps 98 -> 69, copies and scales by two
// warps of their own 64, six planes and O rescaled beside the weights' warps 63, a tile's
// values in two parts 55. Of 128 dimensions (8 rows of 5 heads, 8 kv heads, as long) 67.7
// us: keys' scales copied, not read a tile ahead, and larger boxes save one.
// Room above a row's maximum is the other kernels' (kMargin). Ten binades instead of six
// take 51.3 us for 55.0, but f16's least step is then 2^-29 of a row's largest weight:
// tokens 28.5 octaves behind one that carries no value gave a result 29 % off.
#include <atomic>

#include "copy_ring.h"
#include "kv4_attention.cuh"
#include "kv_cache.cuh"

namespace bws {
namespace {

constexpr int kSoftWarps = 8, kValueWarps = 4, kQuads = 4;   // a quad: 32 tokens, two of warps 0-7
constexpr int kScoreWarp = kSoftWarps + kValueWarps, kSumWarp = kScoreWarp + 1;   // issue the products
constexpr int kKeyWarp = kSumWarp + 1, kValueCopyWarp = kKeyWarp + 1;             // copy
constexpr int kWarps = kValueCopyWarp + 1;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = kWide4Tile;
constexpr int kPlanes = 6, kPairs = kPlanes / 2;
constexpr int kBarSoft = 1, kBarWork = 3;   // named barriers of warps 0-3, 4-7 (kBarSoft + 1) and 0-11
constexpr float kLeastScale = 1.0f / 512.0f;   // of E4M3
// Polls of a wait, each of which sleeps 10 us at most: without that time given the
// waiting warps took a quarter of the issue slots.
constexpr uint32_t kWidePolls = 1u << 16, kSleepNs = 10000;
// TMEM columns: scores of two tiles, O, the keys' scales of two tiles, the queries'
constexpr int kTmemCols = 512, kColO = 256, kColKeys = 384, kColQueries = 416;

template <int D, int NT>
struct Wide4 {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = D / 2;                       // of codes; the operands' swizzle too
  static constexpr int kSteps = D / 64;                         // products of 64 dimensions
  static constexpr int kCodes = kTile * kRowBytes;
  static constexpr int kScales = kTile * D / 16;
  // A tile's values in f16, given in parts (of 64 tokens 55 us, of 32 61; two buffers of
  // 32, not a tile's four, 63).
  static constexpr int kPart = 64, kParts = kTile / kPart;
  static constexpr int kPanel = kPart * 128;                    // 64 dimensions of a part
  static constexpr int kPartBytes = D / 64 * kPanel;
  static constexpr int kPlane = kRows * kRowBytes;
  static constexpr int kWeights = kRows / 8 * kTile * 16;       // P: [rows / 8][token][8]
  static constexpr int kKStages = D == 128 ? 4 : NT <= 6 ? 3 : 2;
  static constexpr int kVStages = D == 128 ? 4 : NT <= 4 ? 3 : 2;
  static constexpr int kOffV = kKStages * kCodes, kOffParts = kOffV + kVStages * kCodes, kOffQ = kOffParts + kParts * kPartBytes;
  static constexpr int kOffP = kOffQ + (kPlanes * kPlane + 1023) / 1024 * 1024, kOffScales = kOffP + 2 * kWeights;
  static constexpr int kOffKScales = kOffScales + kVStages * kScales;       // as they lie in the cache
  static constexpr int kOffKeyScales = kOffKScales + kKStages * kScales;    // of two tiles: [64 dimensions][token % 32][token / 32] words
  static constexpr int kOffTail = kOffKeyScales + 2 * kScales;
  static constexpr int kOHalves = D / 128;                      // M = 128 of O^T
  // D FP32; A and B E2M1, both K-major, E4M3 scales; N = 2 planes, M = 128
  static constexpr uint32_t kIdescS = (1u << 7) | (1u << 10) | ((2u * kRows >> 3) << 17) | ((128u >> 4) << 24);
  // D FP32; A and B f16, both with their own dimension innermost
  static constexpr uint32_t kIdescO = (1u << 4) | (1u << 15) | (1u << 16) | (((uint32_t)kRows >> 3) << 17) | ((128u >> 4) << 24);
  static_assert(kRows % 16 == 0 && 2 * kRows <= 128 && kOHalves * kRows <= kColKeys - kColO, "tiles of rows");
  static_assert(kPairs * kSteps * 128 * 4 <= 2 * kWeights, "the queries' scales wait where weights lie");
};

template <int D, int NT>
struct __align__(16) WideTail4 {
  alignas(16) float2 row[8 * NT];   // scale (with log2 e, the row's power of two and the head's number), what exponents are taken less, or 0
  uint32_t fresh[2];           // of half the rows a word: the row has seen no token yet, and its maximum stands for nothing
  uint32_t moved[4][2];        // likewise, of a tile: its maximum moves
  float up[8 * NT];            // how far the maxima went in a tile that moved them
  float top[kQuads][8 * NT];
  float l[kQuads][8 * NT];
  float m[8 * NT];             // the segment's final maxima
  long long place[8 * NT];     // of the rows' results, and what they are multiplied by, and their sight
  float2 last[8 * NT];
  float factor[2][8 * NT];     // what O shrinks by then, of two tiles
  uint32_t nan_mask[2][D / 16];
  unsigned long long k_full[Wide4<D, NT>::kKStages];
  unsigned long long v_full[Wide4<D, NT>::kVStages], v_free[Wide4<D, NT>::kVStages];
  // boxes of a tile that are in the cache, by tile, and by stage of the copies
  uint32_t there[4], k_there[Wide4<D, NT>::kKStages], v_there[Wide4<D, NT>::kVStages];
  unsigned long long h_full[Wide4<D, NT>::kParts], h_free[Wide4<D, NT>::kParts];
  unsigned long long f_full[2], s_full[2], p_full[2], pv_done[2], o_ready, drain;
  long long line_warp[kWarps];
  long long line_found[2];
  // the CTA's way along its share and its segments, kept here by thread 0
  Walk walk;
  Segment seg[2];
  int more;
  uint32_t tmem;
  uint32_t status;
  uint32_t rescales;      // of O, gone by
  uint32_t started[2];    // tiles that a copying warp has started to copy
};

template <int D, int NT>
constexpr int wide4_smem() { return Wide4<D, NT>::kOffTail + (int)sizeof(WideTail4<D, NT>) + 1024; }

// Shared-memory descriptors: the low word holds the address and the leading
// dimension's stride, the high word, a constant, the other stride and the swizzle.
// (Formed as 64-bit numbers for every product, a product took 110 cycles to issue.)
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) { return (sbo >> 4) | (1u << 14) | (layout << 29); }
BWS_DEV uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }
template <uint32_t kHi, uint32_t kIdesc>
BWS_DEV void mma_codes(uint32_t d, uint32_t a, uint32_t b, uint32_t sfa, uint32_t sfb, uint32_t add) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.u32 p, %5, 0; mov.b64 x, {%1, %6}; mov.b64 y, {%2, %6};"
      " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], x, y, %7, [%3], [%4], p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(sfa), "r"(sfb), "r"(add), "n"(kHi), "r"(kIdesc)
      : "memory");
}
template <uint32_t kHiA, uint32_t kHiB, uint32_t kIdesc>
BWS_DEV void mma_half(uint32_t d, uint32_t a, uint32_t b, uint32_t add) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.u32 p, %3, 0; mov.b64 x, {%1, %4}; mov.b64 y, {%2, %5};"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %6, p; }" ::"r"(d),
      "r"(a), "r"(b), "r"(add), "n"(kHiA), "n"(kHiB), "r"(kIdesc)
      : "memory");
}
// 128 words of scales, [32][4], to four columns, the same in every quad's lanes; the
// products that this thread issues after it see them.
BWS_DEV void copy_scales(uint32_t d, uint32_t src) {
  asm volatile("{ .reg .b64 x; mov.b64 x, {%1, %2}; tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], x; }" ::"r"(d),
               "r"(desc_lo(src, 128)), "n"(desc_hi(128, 0)) : "memory");
}
BWS_DEV void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
BWS_DEV void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
BWS_DEV void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// This thread's lane of eight columns.
BWS_DEV void tmem_load8(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at) : "memory");
}
BWS_DEV void tmem_loaded8(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]) :: "memory");
}
BWS_DEV void tmem_store8(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
BWS_DEV void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The warp's largest, by one instruction.
BWS_DEV float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
BWS_DEV float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The largest magnitude of three.
BWS_DEV float max_abs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// x[0], x[1] plus the halves of v times d, exact products rounded once.
BWS_DEV void add_halves(float* x, uint32_t v, uint16_t d) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; fma.rn.f32.f16 %0, l, %3, %0; fma.rn.f32.f16 %1, h, %3, %1; }"
      : "+f"(x[0]), "+f"(x[1]) : "r"(v), "h"(d));
}
// E2M1 codes of two numbers times f.
BWS_DEV uint32_t codes_of_two(const float* x, unsigned long long ff) {
  uint32_t r;
  asm("{ .reg .b64 y; .reg .f32 l, h; .reg .b8 c; mov.b64 y, {%1, %2}; mul.rn.f32x2 y, y, %3; mov.b64 {l, h}, y;"
      " cvt.rn.satfinite.e2m1x2.f32 c, h, l; cvt.u32.u8 %0, c; }" : "=r"(r) : "f"(x[0]), "f"(x[1]), "l"(ff));
  return r;
}
BWS_DEV bool wait_bounded(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWidePolls; ++i) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(bar), "r"(parity), "r"(kSleepNs) : "memory");
    if (ok) return true;
  }
  return false;
}
// A box of 16 tokens' codes.
BWS_DEV void copy_codes(uint32_t dst, const void* map, int token, int head, int block, uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %2, %4, %5}], [%6], %7;"
      :: "r"(dst), "l"(map), "r"(0), "r"(token), "r"(head), "r"(block), "r"(bar), "l"(pol) : "memory");
}
BWS_DEV void copy_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(pol) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn4_wide_kernel(const __grid_constant__ Attn4Params p) {
  using S = Wide4<D, NT>;
  constexpr int R = S::kRows, kRowBytes = S::kRowBytes;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* const smem = smem_raw + (base - smem_u32(smem_raw));
  WideTail4<D, NT>& T = *reinterpret_cast<WideTail4<D, NT>*>(smem + S::kOffTail);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool works = warp < kScoreWarp;
  const uint32_t k_ring = base, v_ring = base + S::kOffV, parts = base + S::kOffParts, q_at = base + S::kOffQ,
                 p_at = base + S::kOffP, vs_ring = base + S::kOffScales, ks_ring = base + S::kOffKScales;
  const uint32_t k_full = smem_u32(T.k_full), v_full = smem_u32(T.v_full), v_free = smem_u32(T.v_free),
                 f_full = smem_u32(T.f_full), s_full = smem_u32(T.s_full), p_full = smem_u32(T.p_full), pv_done = smem_u32(T.pv_done),
                 h_full = smem_u32(T.h_full), h_free = smem_u32(T.h_free), o_ready = smem_u32(&T.o_ready);
  if (warp == kScoreWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&T.tmem)),
                 "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int s = 0; s < S::kKStages; ++s) mbar_init(k_full + 8 * s, kTile >> p.box_log);
    for (int s = 0; s < S::kVStages; ++s) {
      mbar_init(v_full + 8 * s, kTile >> p.box_log);
      mbar_init(v_free + 8 * s, kValueWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(f_full + 8 * b, 1);
      mbar_init(s_full + 8 * b, 1);
      mbar_init(p_full + 8 * b, kSoftWarps);
      mbar_init(pv_done + 8 * b, 1);
    }
    for (int h = 0; h < S::kParts; ++h) {
      mbar_init(h_full + 8 * h, kValueWarps);
      mbar_init(h_free + 8 * h, 1);
    }
    mbar_init(smem_u32(&T.o_ready), kValueWarps);
    mbar_init(smem_u32(&T.drain), 1);
    T.status = T.rescales = T.started[0] = T.started[1] = 0;
    mbar_fence_init();
  }
  fence_before();
  pdl_launch_dependents();
  pdl_wait();
  if (p.R <= 32) {
    __syncthreads();   // the status word is clear
    if (warp == 0) {
      Walk walk;
      const bool excess = start_small(p, R, walk);
      if (lane == 0) {
        if (excess) T.status = BWS_STATUS_KV_ROWS;
        T.more = walk.next(p, R, T.seg[0]);
        T.walk = walk;
      }
    }
  } else {
    Walk walk;
    walk.start(p, R, T.line_warp, T.line_found, &T.status);
    if (tid == 0) {
      T.more = walk.next(p, R, T.seg[0]);
      T.walk = walk;
    }
  }
  __syncthreads();   // the mbarriers and the TMEM address too
  fence_after();
  const uint32_t tmem = T.tmem;
  const uint32_t quad_at = tmem + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's lanes
  // what the copies of a segment go by
  const int32_t* table_row;
  int seg_head, seg_first, seg_tiles, seg_kv;
  auto enter = [&](const Segment& sg) {
    table_row = p.table + (size_t)sg.r * p.max_blocks;
    seg_head = sg.head;
    seg_first = sg.first;
    seg_tiles = sg.last - sg.first;
    seg_kv = sg.rq.kv(p);
  };
  uint32_t phase_base = 0;   // tiles gone by
  bool dead = false;         // of this warp's lanes alike
  int turn = 0;
  // The (it / n)-th use of barrier it % n.
  auto wait_for = [&](uint32_t bars, uint32_t it, int n, bool freed) {
    const uint32_t use = it / n;
    if (freed && use == 0) return;   // nothing was there before
    const uint32_t bar = bars + 8 * (it % n), parity = (freed ? use - 1 : use) & 1;
    if (!dead) dead = __any_sync(0xffffffffu, !wait_bounded(bar, parity));
  };
  // Block (as the table has it) and first token of box b of tile i of the segment; token
  // -1: past the end. Whether the block is one of the cache's is asked where it is used, a
  // tile later, and a lane past the end reads something else: asked or branched over
  // here, the warp waits a thousand cycles for the table.
  auto look_up = [&](int i, int b, int& block, int& tok) {
    // (unsigned: asked past the end too, and the last tile may end at 2^31)
    const uint32_t t = (uint32_t)(seg_first + i) * kTile + (b << p.box_log);
    const bool in = i < seg_tiles && t < (uint32_t)seg_kv;
    const int q = block_index(p, in ? (int)t : 0);
    block = *(in ? table_row + q : p.row_start);
    tok = in ? (int)t - q * p.B : -1;
  };
  auto is_there = [&](int block, int tok) { return (uint32_t)block < (uint32_t)p.n_blocks && tok >= 0; };

  // ---- copies: a box (as many tokens as a power of two allows in a block) and its scales
  // a lane, by the keys' warp and the values' warp (from one warp they took longer than a
  // tile).
  auto my_box = [&]() { return lane & ((kTile >> p.box_log) - 1); };
  int next_block, next_tok;            // this lane's box of the next tile to copy
  auto copy_box = [&](uint32_t codes_to, uint32_t scales_to, const void* map, const uint8_t* scales, uint32_t bar, uint32_t* there_at) {
    const int box = 1 << p.box_log, n_boxes = kTile >> p.box_log;
    const bool is = is_there(next_block, next_tok);
    const unsigned there = __ballot_sync(0xffffffffu, is && lane < n_boxes);
    if (lane == 0) *there_at = there;
    __syncwarp();
    if (lane < n_boxes) {
      if (is) {
        mbar_arrive_expect_tx(bar, box * (kRowBytes + D / 16));
        copy_codes(codes_to + lane * box * kRowBytes, map, next_tok, seg_head, next_block, bar, l2_evict_first());
        copy_bytes(scales_to + lane * box * (D / 16),
                   scales + next_block * p.scale_block_stride + seg_head * p.scale_head_stride + next_tok * (D / 16),
                   box * (D / 16), bar, l2_evict_first());
      } else {
        mbar_arrive(bar);
      }
    }
  };
  auto copy_keys = [&](uint32_t it) {
    const uint32_t s = it % S::kKStages;
    copy_box(k_ring + s * S::kCodes, ks_ring + s * S::kScales, &p.k_map, p.k_scale, k_full + 8 * s, &T.k_there[s]);
    if (lane == 0) T.started[0] = it + 1;
  };
  auto copy_values = [&](uint32_t it) {
    const uint32_t s = it % S::kVStages;
    copy_box(v_ring + s * S::kCodes, vs_ring + s * S::kScales, &p.v_map, p.v_scale, v_full + 8 * s, &T.v_there[s]);
    if (lane == 0) T.started[1] = it + 1;
  };
  // The keys' scales go on to TMEM, where each column holds a word of 32 tokens: lane l
  // takes tokens l, l + 32, l + 64, l + 96 of a tile. (Read from the cache a tile ahead
  // by this warp, not copied, they took it 2450 cycles a tile, all that one of 128
  // dimensions has.)
  auto give_scales = [&](uint32_t it) {
    const uint32_t s = it % S::kKStages, from = ks_ring + s * S::kScales + lane * (D / 16);
    uint32_t sf[4][S::kSteps];
#pragma unroll
    for (int j = 0; j < 4; ++j) lds_words<S::kSteps>(from + j * 32 * (D / 16), sf[j]);
    unsigned char* const at = smem + S::kOffKeyScales + (it & 1) * S::kScales + lane * 16;
#pragma unroll
    for (int k = 0; k < S::kSteps; ++k)
      *reinterpret_cast<uint4*>(at + k * 512) = make_uint4(sf[0][k], sf[1][k], sf[2][k], sf[3][k]);
    if (lane == 0) T.there[it & 3] = T.k_there[s];
    proxy_fence();   // the tensor cores' copy reads them
    __syncwarp();
    if (lane == 0) mbar_arrive(f_full + 8 * (it & 1));
  };
  // A segment's first copies.
  auto open_copies = [&]() {
    // (set by every warp: what only the copying warps keep would else take registers from
    // the others in their loops)
    next_block = 0;
    next_tok = -1;
    if (warp == kKeyWarp) {
      int block[S::kKStages], tok[S::kKStages];
#pragma unroll
      for (int i = 0; i < S::kKStages; ++i) look_up(i, my_box(), block[i], tok[i]);
#pragma unroll
      for (int i = 0; i < S::kKStages; ++i) {
        next_block = block[i];
        next_tok = tok[i];
        if (!dead && i < seg_tiles) copy_keys(phase_base + i);
      }
      look_up(S::kKStages, my_box(), next_block, next_tok);
    } else if (warp == kValueCopyWarp) {
      int block[S::kVStages], tok[S::kVStages];
#pragma unroll
      for (int i = 0; i < S::kVStages; ++i) look_up(i, my_box(), block[i], tok[i]);
#pragma unroll
      for (int i = 0; i < S::kVStages; ++i) {
        next_block = block[i];
        next_tok = tok[i];
        if (!dead && i < seg_tiles) copy_values(phase_base + i);
      }
      look_up(S::kVStages, my_box(), next_block, next_tok);
    }
    __syncwarp();
  };

  // ---- the segment's query rows as planes, by warps 0-11, a row or two at a time (eight
  // values a lane) and a warp's turns side by side: a plane is a chain of some 300 cycles.
  // Clears a NaN mask.
  constexpr int kQueryWarps = kSoftWarps + kValueWarps;
  auto store_queries = [&]() {
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kTurns = (R + kQueryWarps * kAtOnce - 1) / (kQueryWarps * kAtOnce);
    const Segment& sg = T.seg[turn];
    const int n_rows = min(sg.rq.rows(p) * p.G - sg.row0, R);
    const float g_k = p.k_global != nullptr ? p.k_global[sg.head] : 1.0f;
    uint8_t* const staged = smem + S::kOffP;   // the planes' scales, [pair][step][row of the pair % 32][its / 32] words
    const int first = warp * kAtOnce + lane / kLanes, in = lane % kLanes;   // this lane's rows: first, and every kStep-th
    constexpr int kStep = kQueryWarps * kAtOnce;
    // lane l knows where the warp's l-th row lies
    const int of_lane = min(warp * kAtOnce + lane % kAtOnce + lane / kAtOnce * kStep, max(n_rows - 1, 0));
    const int of_j = (sg.row0 + of_lane) / p.G, of_h = sg.head * p.G + (sg.row0 + of_lane) - of_j * p.G;
    const long long at_lane = (sg.rq.start + of_j) * p.q_row_stride + of_h * p.q_head_stride;
    uint4 raw[kTurns];
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const uint16_t* src = p.q + __shfl_sync(0xffffffffu, at_lane, r * kAtOnce + lane / kLanes) + in * 8;
      raw[r] = first + r * kStep < n_rows ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
    }
    float x[kTurns][8], most[kTurns];
    bool bad[kTurns];   // a row that holds an infinity is all NaN, as its scores are
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const uint32_t w[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
      float top = 0.0f;
      bool is_bad = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[r][i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        is_bad |= !(fabsf(x[r][i]) < INFINITY);
        top = fmaxf(top, fabsf(x[r][i]));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const unsigned lanes = kLanes == 32 ? 0xffffffffu : 0xFFFFu << (lane & 16);
      bad[r] = (__ballot_sync(0xffffffffu, is_bad) & lanes) != 0u;
      // the largest to 2^10 .. 2^11, the first plane's scale below 448; codes of the least
      // scale, 2^-9, are off by 2^-11
      const int e = top > 0.0f && !bad[r] ? min(max(floor_log2_abs(top), -100), 126) - 10 : 0;
      const float f = exp2i(-e);
      most[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[r][i] *= f;
        most[r] = fmaxf(most[r], fabsf(x[r][i]));
      }
      if (in == 0 && first + r * kStep < R) T.row[first + r * kStep] = make_float2(p.scale * kLog2e * exp2i(e) * g_k, 0.0f);
    }
    const int group = in / 2;   // of 16 dimensions
    unsigned char* to[kTurns];
#pragma unroll
    for (int r = 0; r < kTurns; ++r) to[r] = smem + S::kOffQ + codes_at<D>(first + r * kStep, in >> 2) + (in & 3) * 4;
#pragma unroll 1
    for (int plane = 0; plane < kPlanes; ++plane) {
#pragma unroll
      for (int r = 0; r < kTurns; ++r) {
        const int n = first + r * kStep;
        most[r] = fmaxf(most[r], __shfl_xor_sync(0xffffffffu, most[r], 1));
        const uint32_t code = bad[r] ? 0x7Fu : f32x2_to_e4m3x2(0.0f, fmaxf(most[r] * (1.0f / 6.0f), kLeastScale)) & 0xFFu;
        const uint32_t d = bad[r] ? 0x3C00u : e4m3x2_to_f16x2(code) & 0xFFFFu;   // in f16, exact
        const float inv = rcp_fast(__half2float(__ushort_as_half((unsigned short)d)));
        unsigned long long inv2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
        most[r] = 0.0f;
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t two = codes_of_two(&x[r][i], inv2);
          word |= two << (4 * i);
          add_halves(&x[r][i], e2m1x2_to_f16x2(two), (uint16_t)(d | 0x8000u));
          most[r] = max_abs3(x[r][i], x[r][i + 1], most[r]);
        }
        if (n >= R) continue;
        *reinterpret_cast<uint32_t*>(to[r] + plane * S::kPlane) = word;
        const int of = (plane & 1) * R + n;   // row of the pair
        if ((in & 1) == 0)
          staged[((plane >> 1) * S::kSteps + (group >> 2)) * 512 + (of & 31) * 16 + (of >> 5) * 4 + (group & 3)] = (uint8_t)code;
      }
    }
    if (tid < D / 16) T.nan_mask[turn][tid] = 0;
    if (tid < 2) T.fresh[tid] = R == 64 ? 0xffffffffu : (1u << (R / 2 & 31)) - 1u;
    if (tid < 8) T.moved[tid >> 1][tid & 1] = 0;
    proxy_fence();   // the tensor cores read the queries
  };

  bool more = T.more != 0;
  if (more) {
    enter(T.seg[0]);
    open_copies();
    if (works) store_queries();
  }
  while (more) {
    __syncthreads();
    fence_after();
    const Segment& cur = T.seg[turn];
    const Request& rq = cur.rq;
    const int tiles = cur.last - cur.first;
    uint32_t* const nan_mask = T.nan_mask[turn];

    if (warp < kSoftWarps) {
      // ---- a token and half the rows a thread: exponents and weights
      constexpr int kHalf = 4 * NT;
      const int quad = warp & 3, half = warp >> 2, row_a = half * kHalf, token = quad * 32 + lane;
      float l[kHalf];    // this thread's tokens' sums
#pragma unroll
      for (int n = 0; n < kHalf; ++n) l[n] = 0.0f;
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        const int buf = (int)(it & 1);
        const int tok = (cur.first + i) * kTile + token, own = min(tok - rq.seen0(), 31);   // row j sees tokens <= seen0 + j
        wait_for(s_full, it, 2, false);
        fence_after();
        const bool there = ((T.there[it & 3] >> (token >> p.box_log)) & 1u) != 0u && tok < seg_kv;
        // rows below `hidden` do not see the token: the j-th token of the rows'
        // own is seen from row j on
        const int hidden = !there ? R : own > 0 ? min(max(own * p.G - cur.row0, 0), R) : 0;
        const bool ragged = __any_sync(0xffffffffu, !there || own > 0);
        const uint32_t s_at = quad_at + buf * 128 + row_a;
        const float2* const rows = T.row + row_a;
        // exponents of every row, less what stands for its maximum
        float x[kHalf];
        uint32_t a[kHalf], b[kHalf];
        // (all asked for at once where the registers allow it: at 256 dimensions that spills
        // and takes 1.3 us more of the 55, at 128 it saves two of 70)
        auto ask = [&](int n) {
          tmem_load8(s_at + n, a + n);
          tmem_load8(s_at + R + n, b + n);
        };
        if constexpr (D == 128) {
#pragma unroll
          for (int n = 0; n < kHalf; n += 8) ask(n);
        }
#pragma unroll
        for (int n = 0; n < kHalf; n += 8) {
          if constexpr (D != 128) ask(n);
          tmem_loaded8(a + n);
          tmem_loaded8(b + n);
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float4 row = *reinterpret_cast<const float4*>(rows + n + k);
            x[n + k] = fmaf(__uint_as_float(a[n + k]) + __uint_as_float(b[n + k]), row.x, -row.y);
            x[n + k + 1] = fmaf(__uint_as_float(a[n + k + 1]) + __uint_as_float(b[n + k + 1]), row.z, -row.w);
          }
        }
        float top = -INFINITY;
        if (ragged) {
#pragma unroll
          for (int n = 0; n < kHalf; ++n)
            if (row_a + n < hidden) x[n] = -INFINITY;
        }
#pragma unroll
        for (int n = 0; n < kHalf; ++n) top = fmaxf(top, x[n]);
        const uint32_t fresh = T.fresh[half];
        uint32_t any;   // of the half's four warps
        asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
                     : "=r"(any) : "r"((uint32_t)(top > kTop || (fresh != 0u && top != -INFINITY))), "r"(kBarSoft + half),
                       "n"(32 * kQuads) : "memory");
        if (any != 0u) {                 // new maxima, of every row that has grown since its last
#pragma unroll
          for (int n = 0; n < kHalf; ++n) {
            const float v = redux_max(x[n]);
            if (lane == n) T.top[quad][row_a + n] = v;
          }
          named_bar_sync(kBarSoft + half, 32 * kQuads);
          if (quad == 0) {
            wait_for(pv_done, it, 2, true);   // the factors of the tile before last are used
            const int row = row_a + lane;
            bool still = false, moves = false;
            if (lane < kHalf) {
              const bool first = ((fresh >> lane) & 1u) != 0u;
              float up = -INFINITY;
              for (int w = 0; w < kQuads; ++w) up = fmaxf(up, T.top[w][row] - (kTop - kMargin));
              still = first && up == -INFINITY;
              if (!first || still) up = fmaxf(up, 0.0f);
              moves = up != 0.0f;
              T.row[row].y += up;
              T.up[row] = up;
              T.factor[buf][row] = first ? 1.0f : exp2_fast(-up);   // a fresh row's O and sum are 0
            }
            const unsigned left = __ballot_sync(0xffffffffu, still), moved = __ballot_sync(0xffffffffu, moves);
            if (lane == 0) {
              T.fresh[half] = left;
              T.moved[it & 3][half] = moved;
            }
          }
          named_bar_sync(kBarSoft + half, 32 * kQuads);
#pragma unroll
          for (int n = 0; n < kHalf; ++n) {
            x[n] -= T.up[row_a + n];
            l[n] *= T.factor[buf][row_a + n];
          }
        }
        wait_for(pv_done, it, 2, true);   // the products of the tile before last have read their weights
        if (quad == 0 && lane == 0) T.moved[(it + 2) & 3][half] = 0;
        unsigned char* const p_row = smem + S::kOffP + buf * S::kWeights + (row_a / 8) * (kTile * 16) + token * 16;
#pragma unroll
        for (int n = 0; n < kHalf; n += 8) {
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            const float a = exp2_fast(x[n + k]), b = exp2_fast(x[n + k + 1]);
            l[n + k] += a;
            l[n + k + 1] += b;
            const __half2 h2 = __floats2half2_rn(a, b);
            h[k / 2] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          *reinterpret_cast<uint4*>(p_row + (n / 8) * (kTile * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        proxy_fence();   // the tensor cores read the weights
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * buf);
      }
#pragma unroll
      for (int n = 0; n < kHalf; ++n) {
        const float v = warp_sum(l[n]);
        if (lane == n) T.l[quad][row_a + n] = v;
      }
      if (quad == 0 && lane < kHalf) T.m[row_a + lane] = ((T.fresh[half] >> lane) & 1u) != 0u ? kNone : T.row[row_a + lane].y;
      wait_for(pv_done, phase_base + tiles - 1, 2, false);   // the queries' next scales wait where the weights lie
    } else if (warp == kScoreWarp) {
      // ---- S^T = K Q^T
      if (!dead && lane == 0)
        for (int k = 0; k < kPairs * S::kSteps; ++k) copy_scales(tmem + kColQueries + 4 * k, p_at + 512 * k);
      __syncwarp();
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        wait_for(k_full, it, S::kKStages, false);
        wait_for(f_full, it, 2, false);
        wait_for(p_full, it, 2, true);   // the scores of the tile before last are read
        if (!dead && lane == 0) {
          fence_after();
#pragma unroll
          for (int k = 0; k < S::kSteps; ++k)
            copy_scales(tmem + kColKeys + 16 * (it & 1) + 4 * k, base + S::kOffKeyScales + (it & 1) * S::kScales + 512 * k);
          const uint32_t d = tmem + (it & 1) * 128, sfa = tmem + kColKeys + 16 * (it & 1);
          const uint32_t keys = desc_lo(k_ring + (it % S::kKStages) * S::kCodes, 16), queries = desc_lo(q_at, 16);
          constexpr uint32_t kHi = desc_hi(8 * kRowBytes, kRowBytes == 128 ? 2 : 4);
#pragma unroll
          for (int j = 0; j < kPairs; ++j)
#pragma unroll
            for (int k = 0; k < S::kSteps; ++k)
              mma_codes<kHi, S::kIdescS>(d, keys + 2 * k, queries + (2 * j * S::kPlane + 32 * k) / 16, sfa + 4 * k,
                                         tmem + kColQueries + 4 * (j * S::kSteps + k), j + k > 0 ? 1u : 0u);
          commit(s_full + 8 * (it & 1));
        }
        __syncwarp();
      }
    } else if (warp == kSumWarp) {
      // ---- O^T += V^T P^T
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        const int buf = (int)(it & 1);
        wait_for(p_full, it, 2, false);
        for (int h = 0; h < S::kParts; ++h) {
          wait_for(h_full + 8 * h, it, 1, false);
          if (h == 0 && i > 0 && (T.moved[it & 3][0] | T.moved[it & 3][1]) != 0u) {
            wait_for(o_ready, T.rescales, 1, false);
            __syncwarp();
            if (lane == 0) T.rescales += 1;
          }
          if (!dead && lane == 0) {
            fence_after();
            const uint32_t values = desc_lo(parts + h * S::kPartBytes, S::kPanel);
            const uint32_t weights = desc_lo(p_at + buf * S::kWeights + h * (S::kPart * 16), 128);
#pragma unroll
            for (int k = 0; k < S::kPart / 16; ++k)
#pragma unroll
              for (int o = 0; o < S::kOHalves; ++o)
                mma_half<desc_hi(1024, 2), desc_hi(kTile * 16, 0), S::kIdescO>(
                    tmem + kColO + o * R, values + (o * 2 * S::kPanel + k * 2048) / 16, weights + k * 16,
                    k > 0 ? 1u : (uint32_t)(i + h > 0));
            commit(h_free + 8 * h);
            if (h == S::kParts - 1) commit(pv_done + 8 * buf);
          }
          __syncwarp();
        }
      }
    } else if (warp == kKeyWarp) {
      // ---- keys' copies and scales
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        wait_for(s_full, it, 2, true);   // the products of the tile before last have read its keys and scales
        if (!dead && i >= 2 && i - 2 + S::kKStages < tiles) copy_keys(it - 2 + S::kKStages);
        if (i >= 2) look_up(i - 1 + S::kKStages, my_box(), next_block, next_tok);
        wait_for(k_full, it, S::kKStages, false);
        give_scales(it);
      }
    } else if (warp == kValueCopyWarp) {
      // ---- values' copies
      for (int i = 0; i + S::kVStages < tiles; ++i) {
        const uint32_t it = phase_base + i;
        wait_for(v_free, it, S::kVStages, false);
        if (!dead) copy_values(it + S::kVStages);
        look_up(i + S::kVStages + 1, my_box(), next_block, next_tok);
      }
    } else {
      // ---- values: 32 dimensions of a token (a chunk) a lane, codes to f16 under their scales
      const int vw = warp - kSoftWarps;
      constexpr int kChunks = D / 32 / kValueWarps, kRounds = S::kPart / 32;   // chunks of a warp: vw, vw + 4; rounds of tokens
      for (int i = 0; i < tiles; ++i) {
        const uint32_t it = phase_base + i;
        const int s = (int)(it % S::kVStages);
        wait_for(v_full, it, S::kVStages, false);
        const uint32_t there = T.v_there[s];
        const int end = seg_kv - (cur.first + i) * kTile;   // the tile's first token past the end
        const uint32_t codes = v_ring + s * S::kCodes, scales = vs_ring + s * S::kScales;
        const int first_own = rq.seen0() + 1 - (cur.first + i) * kTile;   // the tile's first token that not every row sees
#pragma unroll 1
        for (int h = 0; h < S::kParts; ++h) {
          wait_for(h_free + 8 * h, it, 1, true);
          const uint32_t part_at = parts + h * S::kPartBytes;
          uint32_t two[kRounds * kChunks];
          uint4 w[kRounds * kChunks];
#pragma unroll
          for (int r = 0; r < kRounds; ++r)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int token = h * S::kPart + r * 32 + lane, chunk = vw + c * kValueWarps;
              two[r * kChunks + c] = lds_u16(scales + token * (D / 16) + 2 * chunk);
              w[r * kChunks + c] = lds_v4(codes + codes_at<D>(token, chunk));
            }
          // tokens past the end or without a block get a zero scale (the memory may hold
          // anything); a NaN scale among the rows' own tokens is taken out here and put
          // back at the end for the rows that do see it: 0 * NaN would reach the others
          if ((h + 1) * S::kPart > first_own || there != (1u << (kTile >> p.box_log)) - 1u) {
#pragma unroll
            for (int r = 0; r < kRounds; ++r)
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                const int token = h * S::kPart + r * 32 + lane, chunk = vw + c * kValueWarps;
                uint32_t& s2 = two[r * kChunks + c];
                if (((there >> (token >> p.box_log)) & 1u) == 0u || token >= end) s2 = 0;
                else if (token >= first_own) {
#pragma unroll
                  for (int y = 0; y < 2; ++y)
                    if (((s2 >> (8 * y)) & 0x7Fu) == 0x7Fu) {
                      s2 &= ~(0xFFu << (8 * y));
                      atomicOr(&nan_mask[2 * chunk + y], 1u << min(token - first_own + 1, 31));
                    }
                }
              }
          }
#pragma unroll
          for (int r = 0; r < kRounds; ++r)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const int t = r * 32 + lane, chunk = vw + c * kValueWarps;
              const uint32_t f = e4m3x2_to_f16x2(two[r * kChunks + c]);
              const uint4& x = w[r * kChunks + c];
              const uint32_t words[4] = {x.x, x.y, x.z, x.w};
              const uint32_t row_at = part_at + (chunk >> 1) * S::kPanel + t * 128;
#pragma unroll
              for (int k = 0; k < 4; ++k) {   // eight dimensions
                uint32_t v[4];
                e2m1x8_to_f16x2x4(words[k], v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int y = 0; y < 4; ++y) v[y] = k < 2 ? scaled_lo(v[y], f) : scaled_hi(v[y], f);
                const uint32_t at = row_at + ((((chunk & 1) * 4 + k) ^ (t & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
              }
            }
          // Where maxima moved, O by the factors, once the tile before is in it. (Before
          // the last part is given: this tile's products cannot end while p_full is asked.)
          if (h == S::kParts - 1) {
            wait_for(p_full, it, 2, false);
            const uint32_t moved0 = T.moved[it & 3][0], moved1 = T.moved[it & 3][1];
            if (i > 0 && (moved0 | moved1) != 0u) {
              wait_for(pv_done, it - 1, 2, false);
              fence_after();
#pragma unroll 1
              for (int n = 0; n < R; n += 8) {
                if (((n < R / 2 ? moved0 >> n : moved1 >> (n - R / 2)) & 0xFFu) == 0u) continue;
#pragma unroll 1
                for (int o = 0; o < S::kOHalves; ++o) {
                  uint32_t a[8];
                  tmem_load8(quad_at + kColO + o * R + n, a);
                  tmem_loaded8(a);
#pragma unroll
                  for (int k = 0; k < 8; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * T.factor[it & 1][n + k]);
                  tmem_store8(quad_at + kColO + o * R + n, a);
                }
              }
              tmem_stored();
              fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(o_ready);
            }
          }
          proxy_fence();   // the tensor cores read them
          __syncwarp();
          if (lane == 0) mbar_arrive(h_full + 8 * h);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(v_free + 8 * s);
      }
      wait_for(pv_done, phase_base + tiles - 1, 2, false);
    }
    if (dead && lane == 0) {
      atomicOr(&T.status, (uint32_t)BWS_STATUS_WAIT_TIMEOUT);
      if (warp >= kKeyWarp) {   // this warp's copies still on their way; it starts no more
        const uint32_t bars = warp == kKeyWarp ? k_full : v_full, stages = warp == kKeyWarp ? S::kKStages : S::kVStages;
        const uint32_t started = T.started[warp - kKeyWarp];
        for (uint32_t it = ring_oldest(started, stages); it < started; ++it)
          wait_bounded(bars + 8 * ring_stage(it, stages), ring_parity(it, stages));
        T.started[warp - kKeyWarp] = 0;
      }
    }
    phase_base += tiles;
    if (tid == 0) T.more = T.walk.next(p, R, T.seg[turn ^ 1]);
    __syncthreads();   // the rows' sums and maxima, and the next segment, are there

    // ---- the segment's end, and the next one's start
    more = T.more != 0;
    turn ^= 1;
    if (more) {
      enter(T.seg[turn]);
      open_copies();
      if (works) store_queries();
    }
    if (works) {
      // O^T: a lane a dimension, a row a column; a row's place, factor and sight are
      // formed once
      const int row0 = cur.row0, n_group_rows = min(rq.rows(p) * p.G - row0, R);
      const int slot = blockIdx.x * 2 + (cur.starts ? 1 : 0);
      const bool whole = cur.whole;
      const int row = tid;
      fence_after();
      if (row < n_group_rows) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kQuads; ++w) sum += T.l[w][row];
        const int j = (row0 + row) / p.G, h = cur.head * p.G + (row0 + row) - j * p.G;
        const long long at = (long long)(rq.start + j) * p.H + h, part = (long long)slot * R + row;
        const float g_v = p.v_global != nullptr ? p.v_global[cur.head] : 1.0f;
        T.place[row] = (whole ? at : part) * D;
        T.last[row] = make_float2(g_v * (!whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum), __uint_as_float((2u << j) - 1u));
        if (!whole) p.part_ml[part] = make_float2(T.m[row], sum);
        else if (p.lse != nullptr) p.lse[at] = sum == 0.0f ? -INFINITY : (T.m[row] + log2f(sum)) * kLn2;
      }
      named_bar_sync(kBarWork, 32 * kQueryWarps);
#pragma unroll 1
      for (int o = 0; o < S::kOHalves; ++o) {
        const int d = o * 128 + (warp & 3) * 32 + lane;
        const uint32_t nans = nan_mask[d / 16], o_at = quad_at + kColO + o * R;
#pragma unroll 1
        for (int n = 8 * (warp >> 2); n < n_group_rows; n += 2 * kQueryWarps) {
          uint32_t a[8];
          tmem_load8(o_at + n, a);
          tmem_loaded8(a);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (n + k >= n_group_rows) break;
            const long long at = T.place[n + k] + d;
            const float2 f = T.last[n + k];
            float v = __uint_as_float(a[k]) * f.x;
            if (nans & __float_as_uint(f.y)) v = NAN;
            if (whole) {
              const __nv_bfloat16 b = __float2bfloat16_rn(v);
              p.out[at] = *reinterpret_cast<const uint16_t*>(&b);
            } else {
              p.part_o[at] = v;
            }
          }
        }
      }
      fence_before();   // before the next segment's products write O
    }
  }
  __syncthreads();
  if (tid == 0) p.failed[blockIdx.x] = T.status;
  if (warp == kScoreWarp) {   // every product has finished before the columns are released
    if (lane == 0) {
      commit(smem_u32(&T.drain));
      wait_bounded(smem_u32(&T.drain), 0);
    }
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

template <int D, int NT>
cudaError_t launch_wide4(const Attn4Params& p, cudaStream_t st) {
  static std::atomic<unsigned long long> attr{0};
  static_assert(wide4_smem<D, NT>() <= 227 * 1024, "shared memory");
  const cudaError_t e = set_smem_once(attr, attn4_wide_kernel<D, NT>, wide4_smem<D, NT>());
  if (e != cudaSuccess) return e;
  return launch_pdl(attn4_wide_kernel<D, NT>, dim3((unsigned)p.n_ctas), kThreads, wide4_smem<D, NT>(), st, p);
}

}  // namespace

cudaError_t launch_attn4_wide(int D, int nt, const Attn4Params& p, cudaStream_t st) {
  if (D == 256 && nt == 4) return launch_wide4<256, 4>(p, st);
  if (D == 256 && nt == 6) return launch_wide4<256, 6>(p, st);
  if (D == 256 && nt == 8) return launch_wide4<256, 8>(p, st);
  if (D == 128 && nt == 6) return launch_wide4<128, 6>(p, st);
  if (D == 128 && nt == 8) return launch_wide4<128, 8>(p, st);
  return cudaErrorInvalidValue;
}

}  // namespace bws

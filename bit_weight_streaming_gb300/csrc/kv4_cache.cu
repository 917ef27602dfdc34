// The 4-bit key/value cache: the write of a step's keys and values, and the
// reading back of requests' tokens. Contracts in include/bws.h.
#include <limits.h>

#include "bws_abi_util.h"
#include "bws_common.cuh"
#include "bws_internal.h"
#include "kv4_cache.cuh"
#include "kv_cache.cuh"

namespace bws {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Kv4Side {
  uint8_t* codes;
  uint8_t* scales;
  const float* global;
};

BWS_DEV Kv4Side side_of(const bws_kv4_cache& c, int side) {
  return side ? Kv4Side{c.v, c.v_scale, c.v_global} : Kv4Side{c.k, c.k_scale, c.k_global};
}

// ---- write -------------------------------------------------------------------------
//
// A thread takes 16 values, which share a scale: their largest magnitude is an
// integer maximum of BF16 patterns (a NaN is above infinity's, and becomes the
// scale's NaN), then a sixth of it, a division by the head's number where it has one, a
// reciprocal and sixteen products, each rounded as IEEE's operation is, so that the codes
// can be formed again bit for bit. A warp takes one head of the rows whose codes are 256
// bytes and whose scales are one sector.
//
// Bound: the latency of a round's loads at 41 warps an SM (65 % of issue slots). Long
// writes take two rounds a warp, both asked for at once (12382 rows of 16 heads of 64:
// 13.6 us, 0.70 of the copy rate; one round 14.3, four 14.8, eight 19.2); 134 rows of 8
// heads of 128, 1.8 us, are a launch and two dependent loads.

struct Append4Params {
  const uint16_t* x[2];
  long long row_stride[2], head_stride[2];
  const int32_t* slots;
  int n_rows;
  uint32_t b_inverse;   // ceil(2^32 / (block_tokens / 16)), 0 for blocks of 16
  bws_kv4_cache c;
};

// E2M1 codes of eight BF16 values times `inv`, each rounded to FP32 before.
BWS_DEV uint32_t codes_of(const uint32_t* w, float inv) {
  float y[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    y[2 * k] = __fmul_rn(__uint_as_float(w[k] << 16), inv);
    y[2 * k + 1] = __fmul_rn(__uint_as_float(w[k] & 0xFFFF0000u), inv);
  }
  uint32_t r;
  asm("{ .reg .b8 b0, b1, b2, b3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "  mov.b32 %0, {b0, b1, b2, b3}; }"
      : "=r"(r) : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

template <int D, int kPer>
__global__ void __launch_bounds__(kThreads) append4_kernel(const __grid_constant__ Append4Params p) {
  constexpr int kLanes = D / 16;           // lanes of a row
  constexpr int kRows = 32 / kLanes;       // rows of a warp's round
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bws_kv4_cache& c = p.c;
  const int side = blockIdx.y;
  const long long unit = (long long)blockIdx.x * kWarps + warp;
  const int head = (int)(unit % c.n_kv_heads);
  const long long row0 = unit / c.n_kv_heads * (kRows * kPer) + lane / kLanes;
  const int group = lane % kLanes;
  pdl_launch_dependents();
  pdl_wait();
  if (row0 - lane / kLanes >= p.n_rows) return;
  const Kv4Side s = side_of(c, side);
  const uint16_t* src = p.x[side] + head * p.head_stride[side] + group * 16;
  uint4 a[kPer], b[kPer];
  int slot[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long row = row0 + i * kRows;
    const bool live = row < p.n_rows;
    const uint4* at = reinterpret_cast<const uint4*>(src + (live ? row : 0) * p.row_stride[side]);
    slot[i] = live ? p.slots[row] : -1;
    a[i] = at[0];
    b[i] = at[1];
  }
  const float g = s.global != nullptr ? s.global[head] : 1.0f;
  uint8_t* const codes = s.codes + head * c.head_stride + group * 8;
  uint8_t* const scales = s.scales + head * c.scale_head_stride + group;
  const uint32_t n_slots = (uint32_t)c.n_blocks * (uint32_t)c.block_tokens;   // below 2^31
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if ((uint32_t)slot[i] >= n_slots) continue;   // negative ones too
    const uint32_t w[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    const float a0 = __uint_as_float(top << 16), sixth = top < 0x7F80u ? sixth_of(a0) : a0;
    const float need = g == 1.0f ? sixth : __fdiv_rn(sixth, g);
    const uint32_t code = f32x2_to_e4m3x2(0.0f, need) & 0xFFu;
    const float d = __fmul_rn(e4m3_to_f32(code), g);
    uint32_t out[2] = {0u, 0u};
    if (d > 0.0f) {
      const float inv = __frcp_rn(d);
      out[0] = codes_of(w, inv);
      out[1] = codes_of(w + 4, inv);
    }
    const uint32_t box = (uint32_t)slot[i] >> 4, block = p.b_inverse != 0u ? __umulhi(box, p.b_inverse) : box;
    const uint32_t at = (uint32_t)slot[i] - block * c.block_tokens;
    *reinterpret_cast<uint2*>(codes + block * c.block_stride + at * (D / 2)) = make_uint2(out[0], out[1]);
    scales[block * c.scale_block_stride + at * (D / 16)] = (uint8_t)code;
  }
}

// ---- reading back ------------------------------------------------------------------
//
// A CTA takes kTile rows of the output: one warp finds their slots, then each
// warp takes heads of keys or values, four bytes of codes and 16 bytes of result
// a lane.
//
// Bound: HBM, most of it writes (24 requests of up to 8001 tokens, 8 heads of 128: 150 us,
// 0.87 of the copy rate); of short ones four or five dependent loads. Tiles of eight rows
// where those of 32 would leave SMs without one, and the requests of a tile's rows
// looked through by shuffles, not a load after the other: 777 tokens, 4 heads of 256
// 6.2 -> 3.5 us, 48 requests of 1 to 3 tokens, 8 of 128 7.9 -> 3.8.

struct Read4Params {
  bws_kv4_cache c;
  const int32_t* table;
  int max_blocks, R;
  const int32_t *first, *row_start;
  int n_rows;
  uint16_t* out[2];
};

// The last request that starts at or before `row`, by one warp; R >= 1.
BWS_DEV int request_at(const int32_t* row_start, int R, int row, int lane) {
  int lo = 0, n = R;   // among requests lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const bool below = i < n && row_start[lo + i] <= row;
    const unsigned b = __ballot_sync(0xffffffffu, below);
    const int at = b == 0u ? 0 : 31 - __clz(b);
    lo += at * step;
    n = min(step, n - at * step);
  }
  return lo;
}

// Of a warp's rows, one a lane and in order, the last request that starts at or before
// each; `r` is one that does for every row, the starts behind it are looked through 32
// at a time.
BWS_DEV int request_of_row(const int32_t* row_start, int R, int r, int row, int lane) {
  const int last = __shfl_sync(0xffffffffu, row, 31);
  for (int base = r + 1; base < R; base += 32) {
    const int start = base + lane < R ? row_start[base + lane] : INT_MAX;
    int n = 0;   // starts at or before the row
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
      if (__shfl_sync(0xffffffffu, start, n + step - 1) <= row) n += step;
    n += __shfl_sync(0xffffffffu, start, n) <= row ? 1 : 0;
    r += n;
    if (__shfl_sync(0xffffffffu, start, 31) > last) break;
  }
  return r;
}

template <int D, int kTile>
__global__ void __launch_bounds__(kThreads) read4_kernel(const __grid_constant__ Read4Params p) {
  constexpr int kLanes = D / 8, kUnits = kTile * kLanes / 32, kStep = kUnits < 4 ? kUnits : 4;
  __shared__ int2 s_at[kTile];   // a row's block, -1: none, and its token there
  const bws_kv4_cache& c = p.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int row0 = blockIdx.x * kTile;
  pdl_launch_dependents();
  pdl_wait();
  if (warp == 0) {
    const int row = row0 + min(lane, kTile - 1);
    int2 at = make_int2(-1, 0);
    const int r = request_of_row(p.row_start, p.R, p.R <= 33 ? 0 : request_at(p.row_start, p.R, row0, lane), row, lane);
    if (row < p.n_rows) {
      const int begin = p.row_start[r];
      if (row >= begin && row < p.row_start[r + 1]) {
        const long long token = (long long)p.first[r] + (row - begin);
        if (token >= 0 && token < (long long)p.max_blocks * c.block_tokens) {
          const int q = (int)token / c.block_tokens, block = p.table[(size_t)r * p.max_blocks + q];
          if (block >= 0 && block < c.n_blocks) at = make_int2(block, (int)token - q * c.block_tokens);
        }
      }
    }
    if (lane < kTile) s_at[lane] = at;
  }
  __syncthreads();
  const int chunk = lane % kLanes;
  for (int hs = warp; hs < 2 * c.n_kv_heads; hs += warps) {
    const int head = hs >> 1, side = hs & 1;
    const Kv4Side s = side_of(c, side);
    const float g = s.global != nullptr ? s.global[head] : 1.0f;
    const uint8_t* codes = s.codes + head * c.head_stride + chunk * 4;
    const uint8_t* scales = s.scales + head * c.scale_head_stride + chunk / 2;
    uint16_t* out = p.out[side] + ((size_t)row0 * c.n_kv_heads + head) * D + chunk * 8;
#pragma unroll 1
    for (int u0 = 0; u0 < kUnits; u0 += kStep) {
      uint32_t w[kStep], sc[kStep];
      int t[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        t[i] = ((u0 + i) * 32 + lane) / kLanes;
        const int2 at = s_at[t[i]];
        w[i] = sc[i] = 0;
        if (at.x >= 0) {
          w[i] = *reinterpret_cast<const uint32_t*>(codes + at.x * c.block_stride + at.y * (D / 2));
          sc[i] = scales[at.x * c.scale_block_stride + at.y * (D / 16)];
        }
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        if (row0 + t[i] >= p.n_rows) continue;
        uint32_t h[4];
        e2m1x8_to_f16x2x4(w[i], h[0], h[1], h[2], h[3]);
        const uint32_t two = bcast_lo(e4m3x2_to_f16x2(sc[i]));
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = hmul2_u32(h[k], two);   // exact: six significant bits
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
          const __nv_bfloat162 x = __floats2bfloat162_rn(f.x * g, f.y * g);
          o[k] = *reinterpret_cast<const uint32_t*>(&x);
        }
        *reinterpret_cast<uint4*>(out + (size_t)t[i] * c.n_kv_heads * D) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// The wanted strides of one array of (block, head)s of `bytes` each do not overlap.
bool apart(size_t block_stride, size_t head_stride, size_t bytes, int n_blocks, int n_heads) {
  if (block_stride >= (1ull << 40) || head_stride >= (1ull << 40)) return false;
  const bool by_block = head_stride >= bytes && block_stride >= head_stride * (n_heads - 1) + bytes;
  const bool by_head = block_stride >= bytes && head_stride >= block_stride * ((size_t)n_blocks - 1) + bytes;
  return by_block || by_head;
}

}  // namespace

int check_kv4_cache(const bws_kv4_cache* c, const char* name) {
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
  if (c->block_stride % 16 || c->head_stride % 16 || c->scale_block_stride % 16 || c->scale_head_stride % 16 ||
      !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->k_global, 4) || !aligned(c->v_global, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: codes, scales and their strides 16-byte, the heads' numbers 4-byte alignment needed",
                name);
  const size_t rows = (size_t)c->block_tokens * c->head_dim;
  if (!apart(c->block_stride, c->head_stride, rows / 2, c->n_blocks, c->n_kv_heads) ||
      !apart(c->scale_block_stride, c->scale_head_stride, rows / 16, c->n_blocks, c->n_kv_heads))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: cache strides (%zu, %zu; scales %zu, %zu) overlap or are out of range", name,
                c->block_stride, c->head_stride, c->scale_block_stride, c->scale_head_stride);
  return BWS_OK;
}

}  // namespace bws

extern "C" {

int bws_kv4_append(const uint16_t* k, int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                   int64_t v_row_stride, int64_t v_head_stride, const int32_t* slots, int n_rows,
                   const bws_kv4_cache* cache, void* stream) {
  using namespace bws;
  const char* name = "bws_kv4_append";
  const int rc = check_kv4_cache(cache, name);
  if (rc) return rc;
  if (n_rows < 0) return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d", name, n_rows);
  if (n_rows == 0) {
    clear_error();
    return BWS_OK;
  }
  if (!k || !v || !slots) return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: rows 16-byte, slots 4-byte alignment needed", name);
  if (k_row_stride % 8 || k_head_stride % 8 || v_row_stride % 8 || v_head_stride % 8)
    return fail(BWS_ERR_MISALIGNED, "%s: strides must be multiples of 8 elements", name);
  Append4Params p = {};
  p.x[0] = k;
  p.x[1] = v;
  p.row_stride[0] = k_row_stride;
  p.row_stride[1] = v_row_stride;
  p.head_stride[0] = k_head_stride;
  p.head_stride[1] = v_head_stride;
  p.slots = slots;
  p.n_rows = n_rows;
  const uint32_t boxes = (uint32_t)cache->block_tokens / 16;
  p.b_inverse = boxes == 1 ? 0u : (uint32_t)(((1ull << 32) + boxes - 1) / boxes);
  p.c = *cache;
  const int D = cache->head_dim;
  // Two rounds a warp, so that its loads are on their way together, where that
  // still leaves 32 warps an SM (12382 rows of 16 heads of 64: one round 14.3 us, two
  // 13.6, four 14.8, eight 19.2).
  const long long rounds = ((long long)n_rows + 512 / D - 1) / (512 / D) * cache->n_kv_heads;
  const int per = rounds * 2 >= 64LL * num_sms() ? 2 : 1;
  const long long rows = 512 / D * per;
  const long long units = (n_rows + rows - 1) / rows * cache->n_kv_heads;
  const long long ctas = (units + kWarps - 1) / kWarps;
  if (ctas >= (1LL << 31)) return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: too many rows", name);
  const dim3 grid((unsigned)ctas, 2);
  cudaStream_t st = as_stream(stream);
  cudaError_t e;
  if (D == 64) e = per == 2 ? launch_pdl(append4_kernel<64, 2>, grid, kThreads, 0, st, p) : launch_pdl(append4_kernel<64, 1>, grid, kThreads, 0, st, p);
  else if (D == 128) e = per == 2 ? launch_pdl(append4_kernel<128, 2>, grid, kThreads, 0, st, p) : launch_pdl(append4_kernel<128, 1>, grid, kThreads, 0, st, p);
  else e = per == 2 ? launch_pdl(append4_kernel<256, 2>, grid, kThreads, 0, st, p) : launch_pdl(append4_kernel<256, 1>, grid, kThreads, 0, st, p);
  return cuda_status(e, name);
}

int bws_kv4_read(const bws_kv4_cache* cache, const int32_t* block_table, int max_blocks, int n_requests,
                 const int32_t* first, const int32_t* row_start, int n_rows, uint16_t* k_out, uint16_t* v_out,
                 void* stream) {
  using namespace bws;
  const char* name = "bws_kv4_read";
  const int rc = check_kv4_cache(cache, name);
  if (rc) return rc;
  if (n_rows < 0 || n_requests < 0 || n_requests > (1 << 20) || max_blocks < 0)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d, n_requests = %d, max_blocks = %d", name, n_rows, n_requests,
                max_blocks);
  if ((long long)max_blocks * cache->block_tokens >= (1LL << 31))
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: a table row of %d blocks passes 2^31 tokens", name, max_blocks);
  if (n_rows == 0 || n_requests == 0) {
    clear_error();
    return BWS_OK;
  }
  if (!first || !row_start || !k_out || !v_out || (max_blocks > 0 && !block_table))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(block_table, 4) || !aligned(first, 4) || !aligned(row_start, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: outputs 16-byte, other pointers 4-byte alignment needed", name);
  Read4Params p = {};
  p.c = *cache;
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.R = n_requests;
  p.first = first;
  p.row_start = row_start;
  p.n_rows = n_rows;
  p.out[0] = k_out;
  p.out[1] = v_out;
  const int sides = 2 * cache->n_kv_heads;
  const unsigned block = 32u * (sides < kWarps ? sides : kWarps);
  cudaStream_t st = as_stream(stream);
  const bool few = n_rows < 64LL * num_sms();
  const dim3 grid((unsigned)(((long long)n_rows + (few ? 7 : 31)) / (few ? 8 : 32)));
  cudaError_t e;
  if (cache->head_dim == 64) e = few ? launch_pdl(read4_kernel<64, 8>, grid, block, 0, st, p) : launch_pdl(read4_kernel<64, 32>, grid, block, 0, st, p);
  else if (cache->head_dim == 128) e = few ? launch_pdl(read4_kernel<128, 8>, grid, block, 0, st, p) : launch_pdl(read4_kernel<128, 32>, grid, block, 0, st, p);
  else e = few ? launch_pdl(read4_kernel<256, 8>, grid, block, 0, st, p) : launch_pdl(read4_kernel<256, 32>, grid, block, 0, st, p);
  return cuda_status(e, name);
}

}  // extern "C"

// Per-head RMS norm of queries and keys and their rotation by positions of up to
// four axes, BF16 to BF16. Contract in include/bws.h.
//
// A warp takes 32 / (D / 8) rows and some of their heads, queries' then keys', and
// forms the rows' angles once (qk_rotate.cuh); kAhead heads are asked for together.
// rope_kernel holds both values of a pair in one lane, as two 8-byte loads, so that
// nothing but the norm's sum passes between lanes, and takes the weights into the
// angles: a pair costs six operations. kAll: every dimension turns; otherwise a lane's
// further dimensions pass through the same products, each without the other's (3001 rows
// of 28 heads of 256, a quarter turning, 20.6 -> 21.9 us for the eight selects). Pairs
// (i, i + half) whose half is no multiple of four go to rope_any_kernel, which brings them
// together in shared memory.
//
// Bound: HBM, and the loads' latency at 24 warps an SM: 8191 rows of 32 + 8 heads of 128
// in 30.7 us, 0.81 of the copy rate, 54 % of issue slots. (Pairs brought together by
// shuffles, the norm's weight a product of its own: 56 us.) One row, 2.8 us, is a launch
// and three dependent loads.
#include <type_traits>

#include "bws_abi_util.h"
#include "bws_common.cuh"
#include "bws_internal.h"
#include "kv_cache.cuh"
#include "qk_rotate.cuh"

namespace bws {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kAhead = 4;   // 8191 rows of 40 heads of 128: 30.7 us, three 31.9, two 34.6

struct RopeParams {
  bws_qk in;
  uint16_t *q_out, *k_out;
  int heads_per;   // heads a warp takes of a row
};

// Two FP32 numbers in a register pair, which one instruction works on.
using Two = unsigned long long;
BWS_DEV Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BWS_DEV void halves(Two x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
BWS_DEV Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BWS_DEV Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Two chunks of four values a lane.
struct Eight {
  uint2 a, b;
};

template <int D, bool kAdjacent, bool kAll>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  using Hd = Head<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / Hd::kLanes, sl = lane % Hd::kLanes;
  const bws_qk& in = p.in;
  const int half = in.rot >> 1, heads = in.n_q_heads + in.n_k_heads;
  const int groups = (heads + p.heads_per - 1) / p.heads_per;
  const long long unit = (long long)blockIdx.x * kRopeWarps + warp;
  const int row0 = (int)(unit / groups) * Hd::kRows;
  pdl_launch_dependents();
  pdl_wait();
  if (row0 >= in.n_rows) return;
  const bool live = row0 + sub < in.n_rows;
  const int row = live ? row0 + sub : row0;
  const int h0 = (int)(unit % groups) * p.heads_per, h1 = min(h0 + p.heads_per, heads);
  // this lane's chunks, and its pairs: the first 4 of them, or none (it passes 8 values)
  const int turned = half / 4;   // lanes that turn
  const int first = kAdjacent ? sl * 8 : sl < turned ? sl * 4 : in.rot + (sl - turned) * 8;
  const int gap = kAdjacent || sl >= turned ? 4 : half, second = first + gap;
  const int turning = kAll ? 4 : half - sl * 4;   // of this lane's pairs
  float c[4], s[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    c[k] = 1.0f;
    s[k] = 0.0f;
  }
  if (turning > 0) {
    constexpr double kTurn = 0.15915494309189533577;      // 1 / 2 pi
    constexpr float kHi = (float)kTurn, kLo = (float)(kTurn - (double)kHi);
    int pos[4];
    float f[4];
    bool near = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = min(sl * 4 + k, half - 1);   // adjacent pairs may end inside a lane
      f[k] = in.inv_freq[i];
      int a = in.axis != nullptr ? in.axis[i] : 0;
      if ((unsigned)a >= (unsigned)in.n_axes) a = 0;
      pos[k] = in.positions[(size_t)a * in.n_rows + row];
      near = near && pos[k] < (1 << 24) && pos[k] > -(1 << 24);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float t;
      if (near) {   // as Angles<D>::form
        const float fp = (float)pos[k], fh = f[k] * kHi, fl = fmaf(f[k], kLo, fmaf(f[k], kHi, -fh));
        const float a = fh * fp, e = fmaf(fh, fp, -a);
        t = (a - rintf(a)) + fmaf(fl, fp, e);
        t -= rintf(t);
      } else {
        t = far_turn(f[k], pos[k]);
      }
      if (sl * 4 + k < half) sincos_turn(t, s[k], c[k]);
    }
  }
  auto turn = [&](const uint16_t* src, long long head_stride, uint16_t* dst, const float* weight, int from, int to) {
    if (from >= to) return;
    // of pairs k and k + 1, (x, y) becomes (x m[0] + y m[1], x m[2] + y m[3]): weights
    // and angles in one
    Two m[2][4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float wx[2], wy[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int x = kAdjacent ? first + 2 * (k + j) : first + k + j, y = kAdjacent ? x + 1 : second + k + j;
        wx[j] = weight != nullptr ? weight[x] : 1.0f;
        wy[j] = weight != nullptr ? weight[y] : 1.0f;
      }
      m[k / 2][0] = two(wx[0] * c[k], wx[1] * c[k + 1]);
      m[k / 2][1] = two(-wy[0] * s[k], -wy[1] * s[k + 1]);
      m[k / 2][2] = two(wx[0] * s[k], wx[1] * s[k + 1]);
      m[k / 2][3] = two(wy[0] * c[k], wy[1] * c[k + 1]);
      if constexpr (!kAll) {
        if (k >= turning) m[k / 2][1] = m[k / 2][2] = two(-0.0f, -0.0f);
        else if (k + 1 >= turning) {
          m[k / 2][1] = two(-wy[0] * s[k], -0.0f);
          m[k / 2][2] = two(wx[0] * s[k], -0.0f);
        }
      }
    }
    // What pairs k and k + 1 take of each other's value: of pairs that do not turn
    // nothing, a zero, since 0 times an infinity or a NaN is NaN (and the factor is -0, so
    // that a value of -0 stays one).
    auto others = [&](Two v, int k) {
      float lo, hi;
      halves(v, lo, hi);
      return two(k < turning ? lo : 0.0f, k + 1 < turning ? hi : 0.0f);
    };
    const uint16_t* const here = src + first;
    uint16_t* const there = dst + first;
#pragma unroll 1
    for (int h = from; h < to; h += kAhead) {
      Eight raw[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u < to) {
          const uint16_t* at = here + (h + u) * head_stride;
          raw[u].a = *reinterpret_cast<const uint2*>(at);
          raw[u].b = *reinterpret_cast<const uint2*>(at + gap);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u >= to) break;
        const uint32_t w[4] = {raw[u].a.x, raw[u].a.y, raw[u].b.x, raw[u].b.y};
        // x and y of pairs 0, 1 and 2, 3: neighbours in a word are a pair, or x's of two
        Two x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t u0 = kAdjacent ? w[2 * i] : w[i], u1 = kAdjacent ? w[2 * i + 1] : w[2 + i];
          const float a0 = __uint_as_float(u0 << 16), b0 = __uint_as_float(u0 & 0xFFFF0000u);
          const float a1 = __uint_as_float(u1 << 16), b1 = __uint_as_float(u1 & 0xFFFF0000u);
          x[i] = kAdjacent ? two(a0, a1) : two(a0, b0);
          y[i] = kAdjacent ? two(b0, b1) : two(a1, b1);
        }
        Two r = two(1.0f, 1.0f);
        if (weight != nullptr) {
          const Two q = fma2(x[0], x[0], fma2(x[1], x[1], fma2(y[0], y[0], mul2(y[1], y[1]))));
          float lo, hi;
          halves(q, lo, hi);
          float sum = lo + hi;
#pragma unroll
          for (int o = Hd::kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          sum = rsqrtf(sum * (1.0f / D) + in.eps);
          r = two(sum, sum);
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a0, a1, b0, b1;
          Two xc = x[i], yc = y[i];
          if constexpr (!kAll) {
            xc = others(x[i], 2 * i);
            yc = others(y[i], 2 * i);
          }
          halves(mul2(fma2(x[i], m[i][0], mul2(yc, m[i][1])), r), a0, a1);
          halves(mul2(fma2(y[i], m[i][3], mul2(xc, m[i][2])), r), b0, b1);
          const __nv_bfloat162 p = kAdjacent ? __floats2bfloat162_rn(a0, b0) : __floats2bfloat162_rn(a0, a1);
          const __nv_bfloat162 q = kAdjacent ? __floats2bfloat162_rn(a1, b1) : __floats2bfloat162_rn(b0, b1);
          o[kAdjacent ? 2 * i : i] = *reinterpret_cast<const uint32_t*>(&p);
          o[kAdjacent ? 2 * i + 1 : 2 + i] = *reinterpret_cast<const uint32_t*>(&q);
        }
        if (live) {
          uint16_t* at = there + (h + u) * D;   // at most 1024 heads of 256
          *reinterpret_cast<uint2*>(at) = make_uint2(o[0], o[1]);
          *reinterpret_cast<uint2*>(at + gap) = make_uint2(o[2], o[3]);
        }
      }
    }
  };
  const int H = in.n_q_heads, K = in.n_k_heads;
  turn(in.q + row * in.q_row_stride, in.q_head_stride, p.q_out + (size_t)row * H * D, in.q_weight, h0, min(h1, H));
  turn(in.k + row * in.k_row_stride, in.k_head_stride, p.k_out + (size_t)row * K * D, in.k_weight, max(h0 - H, 0), h1 - H);
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RopeParams p) {
  using Hd = Head<D>;
  extern __shared__ __align__(16) float s_pairs[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / Hd::kLanes, sl = lane % Hd::kLanes;
  const bws_qk& in = p.in;
  const int half = in.rot >> 1, heads = in.n_q_heads + in.n_k_heads;
  float* const buf = s_pairs + (warp * Hd::kRows + sub) * D;
  float2* const cs = reinterpret_cast<float2*>(s_pairs + ((kRopeWarps + warp) * Hd::kRows + sub) * D);
  constexpr Pairs pairs = kSplitAny;
  const int groups = (heads + p.heads_per - 1) / p.heads_per;
  const long long unit = (long long)blockIdx.x * kRopeWarps + warp;
  const int row0 = (int)(unit / groups) * Hd::kRows;
  pdl_launch_dependents();
  pdl_wait();
  if (row0 >= in.n_rows) return;
  const bool live = row0 + sub < in.n_rows;
  const int row = live ? row0 + sub : row0;
  const int h0 = (int)(unit % groups) * p.heads_per, h1 = min(h0 + p.heads_per, heads);
  float cos_of[8], sin_of[8];
  if (half > 0) {
    Angles<D> angles;
    angles.init(in.inv_freq, pairs, half, sl);
    int pos[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = Angles<D>::pair_of(pairs, k, half, sl);
      int a = in.axis != nullptr && i < half ? in.axis[i] : 0;
      if ((unsigned)a >= (unsigned)in.n_axes) a = 0;
      pos[k] = in.positions[(size_t)a * in.n_rows + row];
    }
    angles.form([&](int k) { return pos[k]; }, in.inv_freq, pairs, half, sl, cs, cos_of, sin_of);
  }
  auto turn = [&](const uint16_t* src, long long head_stride, uint16_t* dst, const float* weight, int from, int to) {
    if (from >= to) return;
    float w[8];
    if (weight != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = weight[sl * 8 + i];
    }
#pragma unroll 1
    for (int h = from; h < to; h += kAhead) {
      uint4 raw[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) raw[u] = *reinterpret_cast<const uint4*>(src + min(h + u, to - 1) * head_stride);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (h + u >= to) break;
        float x[8];
        unpack8(raw[u], x);
        if (weight != nullptr) norm_head<D>(x, w, in.eps);
        if (half > 0) rotate_head<D>(x, cos_of, sin_of, pairs, half, buf, sl);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          o[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (live) *reinterpret_cast<uint4*>(dst + (size_t)(h + u) * D) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  };
  const int H = in.n_q_heads, K = in.n_k_heads;
  turn(in.q + row * in.q_row_stride + sl * 8, in.q_head_stride, p.q_out + (size_t)row * H * D + sl * 8, in.q_weight, h0,
       min(h1, H));
  turn(in.k + row * in.k_row_stride + sl * 8, in.k_head_stride, p.k_out + (size_t)row * K * D + sl * 8, in.k_weight,
       max(h0 - H, 0), h1 - H);
}

}  // namespace
}  // namespace bws

extern "C" int bws_qk_norm_rope(const bws_qk* in, uint16_t* q_out, uint16_t* k_out, void* stream) {
  using namespace bws;
  const char* name = "bws_qk_norm_rope";
  if (in == nullptr) return fail(BWS_ERR_INVALID_ARG, "%s: null input", name);
  const int D = in->head_dim, H = in->n_q_heads, K = in->n_k_heads;
  if (D != 64 && D != 128 && D != 256)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: head_dim = %d must be 64, 128 or 256", name, D);
  if (in->n_rows < 0 || H < 0 || H > 1024 || K < 0 || K > 1024)
    return fail(BWS_ERR_INVALID_ARG, "%s: n_rows = %d, n_q_heads = %d, n_k_heads = %d (0..1024)", name, in->n_rows, H, K);
  if (in->rot < 0 || in->rot > D || in->rot % 2)
    return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: rot = %d must be even and at most head_dim", name, in->rot);
  if (in->n_axes < 1 || in->n_axes > 4 || (in->n_axes > 1 && in->rot > 0 && !in->axis))
    return fail(BWS_ERR_INVALID_ARG, "%s: n_axes = %d must be in [1, 4], with an axis for every pair above 1", name,
                in->n_axes);
  if (in->n_rows == 0 || H + K == 0) {
    clear_error();
    return BWS_OK;
  }
  if ((H > 0 && (!in->q || !q_out)) || (K > 0 && (!in->k || !k_out)) || (in->rot > 0 && (!in->positions || !in->inv_freq)))
    return fail(BWS_ERR_INVALID_ARG, "%s: null pointer", name);
  if (!(in->eps >= 0.0f)) return fail(BWS_ERR_INVALID_ARG, "%s: eps must not be negative", name);
  if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(in->positions, 4) || !aligned(in->axis, 4) || !aligned(in->inv_freq, 4) || !aligned(in->q_weight, 4) ||
      !aligned(in->k_weight, 4))
    return fail(BWS_ERR_MISALIGNED, "%s: rows 16-byte, other pointers 4-byte alignment needed", name);
  if (in->q_row_stride % 8 || in->q_head_stride % 8 || in->k_row_stride % 8 || in->k_head_stride % 8)
    return fail(BWS_ERR_MISALIGNED, "%s: strides must be multiples of 8 elements", name);
  RopeParams p;
  p.in = *in;
  p.q_out = q_out;
  p.k_out = k_out;
  // Warps of a row, by what the fullest SM has to do: rounds of its 32 warps, each of
  // so many heads and the angles before them (about three heads' time).
  const long long row_groups = ((long long)in->n_rows + 256 / D - 1) / (256 / D), at_once = 32LL * num_sms();
  long long per = 1, least = -1;
  for (int g = 1; g <= H + K; ++g) {
    const long long heads = (H + K + g - 1) / g, cost = (row_groups * g + at_once - 1) / at_once * (heads + 3);
    if (least < 0 || cost < least) {
      least = cost;
      per = heads;
    }
    if (heads == 1) break;
  }
  p.heads_per = (int)per;
  const long long ctas = (row_groups * ((H + K + per - 1) / per) + kRopeWarps - 1) / kRopeWarps;
  if (ctas >= (1LL << 31)) return fail(BWS_ERR_UNSUPPORTED_SHAPE, "%s: too many rows", name);
  const dim3 grid((unsigned)ctas);
  cudaStream_t st = as_stream(stream);
  auto launch = [&](auto d) {
    constexpr int kD = decltype(d)::value;
    if (in->interleaved && in->rot == kD) return launch_pdl(rope_kernel<kD, true, true>, grid, kRopeThreads, 0, st, p);
    if (in->interleaved) return launch_pdl(rope_kernel<kD, true, false>, grid, kRopeThreads, 0, st, p);
    if (in->rot == kD) return launch_pdl(rope_kernel<kD, false, true>, grid, kRopeThreads, 0, st, p);
    if (in->rot / 2 % 4 == 0) return launch_pdl(rope_kernel<kD, false, false>, grid, kRopeThreads, 0, st, p);
    return launch_pdl(rope_any_kernel<kD>, grid, kRopeThreads, 2 * kRopeWarps * 256 * 4, st, p);
  };
  const cudaError_t e = D == 64 ? launch(std::integral_constant<int, 64>()) : D == 128 ? launch(std::integral_constant<int, 128>())
                                                                          : launch(std::integral_constant<int, 256>());
  return cuda_status(e, name);
}

// Appending new tokens whose keys and queries are normed head by head, or
// that stand at a drafted tree's positions.
#include "kvc_paged.h"

namespace kvc {
namespace {

// For a head's row x of D elements: y = x (mean(x^2) + eps)^-1/2 w, turned by
// the position's angles.  A row is read once, its sum of squares, norm and
// rotation are binary32, and the result is rounded once to the stored type;
// so the floor is q, k and v in and out, as for k_append.
//
// A head is D / 16 lanes (of 4, 8 or 16) with 16 elements each: the same two
// vectors as in k_append, so that a pair that turns together is in one lane;
// the squares are summed over the lanes by exchanges in a fixed order.
//
// What bounds it is HBM: 7,078 tokens of 40 + 40 + 40 heads x 128 (437 MB) take
// 85 us, 5.1 TB/s, 3 us more than k_append takes for the same bytes; eight single
// tokens take 3.4 us, a launch.  Weights kept in registers over several tokens
// (a loop over rows) cost 20% for the waves that it left out of flight, and
// whole waves of keys, values or queries (scalar pointers, sums by DPP) 2%.
struct NormArgs {
  Seqs s;
  uint8_t *k_cache, *v_cache;
  const uint8_t *k, *v, *q;
  uint8_t *q_out;
  uint64_t k_stride, v_stride, q_stride, q_out_stride;  // bytes
  uint64_t row;                                         // bytes of a cached token's K (or V) row
  uint32_t kv_heads, heads;                             // heads: 0 without queries
  uint32_t rotary, interleaved;
  const float *cos_sin;
  uint32_t n_positions;
  const float *q_weight, *k_weight;  // NULL: no norm
  float eps;
  const int32_t *depth;  // or NULL
  int32_t *status;
};

__device__ inline void load_f8(const float *p, float *x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(p + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
  }
}

template <class TI, class TC, int D, bool kStream>
__global__ __launch_bounds__(256) void k_append_norm(NormArgs a) {
  constexpr uint32_t T = D / 16, G = T <= 4 ? 4 : T <= 8 ? 8 : 16;  // lanes: at work, to a head
  const uint32_t row = blockIdx.x;
  const uint32_t b = a.s.q_start ? seq_of_row(a.s, row) : row;
  uint32_t r0, n;
  a.s.rows(b, r0, n);
  const bool first = threadIdx.x == 0 && blockIdx.y == 0;
  if (blockIdx.x == 0 && blockIdx.y == 0) a.s.check(a.status);
  if (a.s.rows_bad(b) || a.s.len_bad(b)) return;
  if (row < r0 || row - r0 >= n) return;  // before the first or behind the last sequence
  const int32_t base = a.s.lens[b] - (int32_t)n;
  const int32_t pos = base + (int32_t)(row - r0);
  if (pos < 0) return;  // padding
  const int64_t at = a.depth ? (int64_t)base + a.depth[row] : pos;  // the rotation's position
  uint32_t slot;
  if (!a.s.slot_of(a.s.table + (uint64_t)b * a.s.table_stride, (uint32_t)pos, slot) ||
      at < 0 || (a.rotary && at >= a.n_positions)) {
    if (first) set_status(a.status, KVC_ERR_SHAPE);
    return;
  }
  const float *cs = a.cos_sin + (uint64_t)at * a.rotary;
  // heads in the order keys, values, queries
  const uint32_t item = blockIdx.y * (256u / G) + threadIdx.x / G, t = threadIdx.x % G;
  if (item >= 2 * a.kv_heads + a.heads) return;
  const bool is_k = item < a.kv_heads, is_q = item >= 2 * a.kv_heads;
  const uint32_t head = is_k ? item : is_q ? item - 2 * a.kv_heads : item - a.kv_heads;
  const uint8_t *src = is_k ? a.k + row * a.k_stride
                            : is_q ? a.q + row * a.q_stride : a.v + row * a.v_stride;
  uint8_t *dst = is_k ? a.k_cache + (uint64_t)slot * a.row
                      : is_q ? a.q_out + row * a.q_out_stride : a.v_cache + (uint64_t)slot * a.row;
  src += (uint64_t)head * D * 2;
  dst += (uint64_t)head * D * 2;
  const bool plain = !is_k && !is_q;
  const uint32_t half = a.rotary / 2;
  const bool split = a.rotary && !a.interleaved && !plain;
  const bool pair = split && t < half / 8;  // the lane's vectors turn with each other
  uint32_t d0 = t * 8, d1 = d0 + D / 2;
  if (pair) {
    d1 = d0 + half;
  } else if (split) {
    d0 = a.rotary + (t - half / 8) * 8;
    d1 = d0 + (D - a.rotary) / 2;
  }
  const bool live = T == G || t < T;
  u32x4 w0 = {0, 0, 0, 0}, w1 = {0, 0, 0, 0};
  if (live) {
    w0 = move_load<kStream>(src + d0 * 2);
    w1 = move_load<kStream>(src + d1 * 2);
  }
  const float *weight = is_k ? a.k_weight : a.q_weight;
  const bool normed = weight != nullptr && !plain;
  if (plain || (!normed && !a.rotary)) {  // the bits, where the types agree
    if (!live) return;
    if (is_q) {
      move_store<kStream>(dst + d0 * 2, w0);
      move_store<kStream>(dst + d1 * 2, w1);
    } else {
      move_store<kStream>(dst + d0 * 2, convert8<TI, TC>(w0));
      move_store<kStream>(dst + d1 * 2, convert8<TI, TC>(w1));
    }
    return;
  }
  float x[8], y[8];
  widen8<TI>(w0, x);
  widen8<TI>(w1, y);
  if (normed) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum = __builtin_fmaf(x[i], x[i], sum);
      sum = __builtin_fmaf(y[i], y[i], sum);
    }
#pragma unroll
    for (uint32_t d = 1; d < G; d <<= 1) sum += __shfl_xor(sum, d);
    const float rs = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, 1.0f / D, a.eps));
    float wx[8] = {}, wy[8] = {};
    if (live) {
      load_f8(weight + d0, wx);
      load_f8(weight + d1, wy);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = x[i] * rs * wx[i];
      y[i] = y[i] * rs * wy[i];
    }
  }
  if (!live) return;
  if (pair) {
    float c[8], s[8];
    load_f8(cs + d0, c);
    load_f8(cs + half + d0, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = __builtin_fmaf(x[i], c[i], -(y[i] * s[i]));
      y[i] = __builtin_fmaf(y[i], c[i], x[i] * s[i]);
      x[i] = u;
    }
  } else if (a.rotary && a.interleaved) {
    const auto turn = [&](float *z, uint32_t d) {
      if (d >= a.rotary) return;
      const f32x4 c = *reinterpret_cast<const f32x4 *>(cs + d / 2);
      const f32x4 s = *reinterpret_cast<const f32x4 *>(cs + half + d / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = __builtin_fmaf(z[2 * i], c[i], -(z[2 * i + 1] * s[i]));
        z[2 * i + 1] = __builtin_fmaf(z[2 * i + 1], c[i], z[2 * i] * s[i]);
        z[2 * i] = u;
      }
    };
    turn(x, d0);
    turn(y, d1);
  }
  if (is_q) {
    move_store<kStream>(dst + d0 * 2, narrow8<TI>(x));
    move_store<kStream>(dst + d1 * 2, narrow8<TI>(y));
  } else {
    move_store<kStream>(dst + d0 * 2, narrow8<TC>(x));
    move_store<kStream>(dst + d1 * 2, narrow8<TC>(y));
  }
}

template <class TI, class TC, int D>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
  constexpr uint32_t per = 256 / (D <= 64 ? 4 : D <= 128 ? 8 : 16);  // heads to a block
  const uint32_t items = 2 * a.kv_heads + a.heads;
  const dim3 grid(a.s.n_tokens, (items + per - 1) / per);
  if (2ull * a.s.n_tokens * items * D * 2 > kStreamBytes)
    hipLaunchKernelGGL((k_append_norm<TI, TC, D, true>), grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((k_append_norm<TI, TC, D, false>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <class TI, class TC>
hipError_t launch_norm_t(const kvc_paged_desc &p, const NormArgs &a, hipStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_norm<TI, TC, 64>(a, stream);
    case 96: return launch_norm<TI, TC, 96>(a, stream);
    case 128: return launch_norm<TI, TC, 128>(a, stream);
    default: return launch_norm<TI, TC, 256>(a, stream);
  }
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_append_norm(const kvc_paged_desc *p, const kvc_paged_batch *b,
                                      uint32_t layer, void *pool, const void *k, uint64_t k_stride,
                                      const void *v, uint64_t v_stride, const void *q,
                                      uint64_t q_stride, void *q_out, uint64_t q_out_stride,
                                      const kvc_rope *rope, const kvc_head_norm *norm,
                                      const int32_t *depth, int32_t *dev_status,
                                      hipStream_t stream) {
  kvc_status st = append_check(p, b, layer, pool, k, k_stride, v, v_stride, q, q_stride, q_out,
                               q_out_stride, rope, dev_status);
  if (st != KVC_OK) return st;
  if (norm) {
    if (norm->reserved != 0) return KVC_ERR_INVALID_ARG;
    if (!(norm->eps >= 1.17549435e-38f && norm->eps <= 3.4028234664e38f))
      return KVC_ERR_INVALID_ARG;
    if (!norm->k_weight || !aligned(norm->k_weight, 16)) return KVC_ERR_INVALID_ARG;
    if (q && !norm->q_weight) return KVC_ERR_INVALID_ARG;
    if (!aligned(norm->q_weight, 16)) return KVC_ERR_INVALID_ARG;
  }
  if (!aligned(depth, 4)) return KVC_ERR_INVALID_ARG;
  if (b->n_seqs == 0 || b->n_tokens == 0) return KVC_OK;
  NormArgs a{};
  a.s = to_seqs(p, b);
  a.k_cache = static_cast<uint8_t *>(pool) + 2ull * layer * plane_bytes(p);
  a.v_cache = a.k_cache + plane_bytes(p);
  a.k = static_cast<const uint8_t *>(k);
  a.v = static_cast<const uint8_t *>(v);
  a.q = static_cast<const uint8_t *>(q);
  a.q_out = static_cast<uint8_t *>(q_out);
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.q_stride = q_stride * 2;
  a.q_out_stride = q_out_stride * 2;
  a.row = (uint64_t)p->n_kv_heads * p->head_dim * 2;
  a.kv_heads = p->n_kv_heads;
  a.heads = q ? p->n_heads : 0;
  if (rope) {
    a.rotary = rope->rotary_dim;
    a.interleaved = rope->interleaved;
    a.cos_sin = rope->cos_sin;
    a.n_positions = rope->n_positions;
  }
  if (norm) {
    a.q_weight = norm->q_weight;
    a.k_weight = norm->k_weight;
    a.eps = norm->eps;
  }
  a.depth = depth;
  a.status = dev_status;
  hipError_t e;
  if (p->io_dtype == KVC_F16)
    e = launch_norm_t<f16, f16>(*p, a, stream);
  else if (p->cache_dtype == KVC_BF16)
    e = launch_norm_t<bf16, bf16>(*p, a, stream);
  else
    e = launch_norm_t<bf16, f16>(*p, a, stream);
  return e == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

// The paged KV cache's entry points (argument checks), appending new tokens
// with their rotation, and moving a context between pages and a tensor.
#include "kvc_paged.h"

namespace kvc {
namespace {

// ------------------------------------------------------------------ append
// Each new token's rows are moved once: q to q_out and k to its slot, turned
// by the position's angles, v to its slot.  Nothing is reused but the
// rotation row (shared by the heads, from cache), so the floor is the bytes
// of q, k and v read and written.
//
// A thread owns two 8-element vectors of one head half a head (or half the
// rotated part) apart, so that the pairs of the split form meet in one
// thread and neighbouring lanes touch neighbouring 16-byte vectors in both
// forms.  The angles' products and sums are binary32 (fused), rounded once
// to the stored type.
//
// A call's q, k and v were just written by a projection and its outputs are
// read by the attention that follows, so they are left in the caches unless
// there is more than these hold (kStream; 62 MB moved: 12.3 us against 14.1
// streamed; 443 MB: 87 against 78).
struct AppendArgs {
  Seqs s;
  uint8_t *k_cache, *v_cache;
  const uint8_t *k, *v, *q;
  uint8_t *q_out;
  uint64_t k_stride, v_stride, q_stride, q_out_stride;  // bytes
  uint64_t row;                                         // bytes of a cached token's K (or V) row
  uint32_t q_items, k_items;  // items of a token's queries (0: none) and of its keys
  FastDiv head_items;         // head_dim / 16
  uint32_t head_dim, rotary, interleaved;
  const float *cos_sin;
  uint32_t n_positions;
  int32_t *status;
};

// 8 elements as binary32 and back.
template <class T>
__device__ inline void widen8(u32x4 w, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = elem_lo<T>(w[i]);
    x[2 * i + 1] = elem_hi<T>(w[i]);
  }
}
template <class T>
__device__ inline u32x4 narrow8(const float *x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
  return w;
}

// A vector without rotation: its bits if the types agree (NaN payloads kept).
template <class TI, class TO>
__device__ inline u32x4 convert8(u32x4 w) {
  if constexpr (std::is_same<TI, TO>::value) {
    return w;
  } else {
    float x[8];
    widen8<TI>(w, x);
    return narrow8<TO>(x);
  }
}

// 4 pairs (2j, 2j + 1) in a vector, with their 4 cosines and sines.
template <class TI, class TO>
__device__ inline u32x4 turn_inter(u32x4 w, const float *c, const float *s) {
  float x[8], y[8];
  widen8<TI>(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __builtin_fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i]));
    y[2 * i + 1] = __builtin_fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]);
  }
  return narrow8<TO>(y);
}

template <class TI, class TO, bool kStream>
__device__ inline void append_item(const AppendArgs &a, const uint8_t *src, uint8_t *dst,
                                   uint32_t item, bool turn, const float *cs) {
  const uint32_t head = a.head_items.div(item), t = item - head * a.head_items.d;
  const uint32_t base = head * a.head_dim;
  const uint32_t half = a.rotary / 2;
  if (turn && !a.interleaved) {
    if (t < half / 8) {
      const uint32_t d0 = t * 8, d1 = d0 + half;
      const u32x4 w0 = move_load<kStream>(src + (uint64_t)(base + d0) * 2);
      const u32x4 w1 = move_load<kStream>(src + (uint64_t)(base + d1) * 2);
      float x[8], y[8], u[8], v[8], c[8], s[8];
      widen8<TI>(w0, x);
      widen8<TI>(w1, y);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 cv = *reinterpret_cast<const f32x4 *>(cs + d0 + 4 * i);
        const f32x4 sv = *reinterpret_cast<const f32x4 *>(cs + half + d0 + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[4 * i + e] = cv[e];
          s[4 * i + e] = sv[e];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = __builtin_fmaf(x[i], c[i], -(y[i] * s[i]));
        v[i] = __builtin_fmaf(y[i], c[i], x[i] * s[i]);
      }
      move_store<kStream>(dst + (uint64_t)(base + d0) * 2, narrow8<TO>(u));
      move_store<kStream>(dst + (uint64_t)(base + d1) * 2, narrow8<TO>(v));
      return;
    }
    const uint32_t d0 = a.rotary + (t - half / 8) * 8, d1 = d0 + (a.head_dim - a.rotary) / 2;
    const u32x4 w0 = move_load<kStream>(src + (uint64_t)(base + d0) * 2);
    const u32x4 w1 = move_load<kStream>(src + (uint64_t)(base + d1) * 2);
    move_store<kStream>(dst + (uint64_t)(base + d0) * 2, convert8<TI, TO>(w0));
    move_store<kStream>(dst + (uint64_t)(base + d1) * 2, convert8<TI, TO>(w1));
    return;
  }
  const uint32_t d[2] = {t * 8, t * 8 + a.head_dim / 2};
  u32x4 w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) w[i] = move_load<kStream>(src + (uint64_t)(base + d[i]) * 2);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (turn && d[i] < a.rotary) {
      float c[4], s[4];
      const f32x4 cv = *reinterpret_cast<const f32x4 *>(cs + d[i] / 2);
      const f32x4 sv = *reinterpret_cast<const f32x4 *>(cs + half + d[i] / 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c[e] = cv[e];
        s[e] = sv[e];
      }
      w[i] = turn_inter<TI, TO>(w[i], c, s);
    } else {
      w[i] = convert8<TI, TO>(w[i]);
    }
    move_store<kStream>(dst + (uint64_t)(base + d[i]) * 2, w[i]);
  }
}

// The last sequence whose first row is at most `row` (q_start[0] <= row).
__device__ inline uint32_t seq_of_row(const Seqs &s, uint32_t row) {
  uint32_t lo = 0, hi = s.n_seqs;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (s.q_start[mid] <= (int32_t)row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <class TI, class TC, bool kStream>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
  const uint32_t row = blockIdx.x;
  const uint32_t b = a.s.q_start ? seq_of_row(a.s, row) : row;
  uint32_t r0, n;
  a.s.rows(b, r0, n);
  const bool first = threadIdx.x == 0 && blockIdx.y == 0;
  if (blockIdx.x == 0 && blockIdx.y == 0) a.s.check(a.status);
  if (a.s.rows_bad(b) || a.s.len_bad(b)) return;
  if (row < r0 || row - r0 >= n) return;  // before the first or behind the last sequence
  const int32_t pos = a.s.lens[b] - (int32_t)n + (int32_t)(row - r0);
  if (pos < 0) return;  // padding
  uint32_t slot;
  if (!a.s.slot_of(a.s.table + (uint64_t)b * a.s.table_stride, (uint32_t)pos, slot) ||
      (a.rotary && (uint32_t)pos >= a.n_positions)) {
    if (first) set_status(a.status, KVC_ERR_SHAPE);
    return;
  }
  const float *cs = a.cos_sin + (uint64_t)(uint32_t)pos * a.rotary;
  const bool turn = a.rotary != 0;
  const uint32_t item = blockIdx.y * 256u + threadIdx.x;
  if (item < a.k_items) {
    append_item<TI, TC, kStream>(a, a.k + row * a.k_stride, a.k_cache + (uint64_t)slot * a.row,
                                 item, turn, cs);
  } else if (item < 2 * a.k_items) {
    append_item<TI, TC, kStream>(a, a.v + row * a.v_stride, a.v_cache + (uint64_t)slot * a.row,
                                 item - a.k_items, false, cs);
  } else if (item < 2 * a.k_items + a.q_items) {
    append_item<TI, TI, kStream>(a, a.q + row * a.q_stride, a.q_out + row * a.q_out_stride,
                                 item - 2 * a.k_items, turn, cs);
  }
}

// -------------------------------------------------------------- page moves
// A block moves kPageRows token rows of one (layer, K/V); the rows' slots are
// looked up once into LDS.  16 bytes a lane, lanes along the channels, four
// loads in flight; past the caches (kStream) if they could not hold the data
// (2.9 GB moved: 558 us with plain loads and stores).
constexpr uint32_t kPageRows = 16;

struct PageArgs {
  uint8_t *pool, *flat;
  Seqs s;                          // its pages and page table
  uint64_t row;                    // bytes of a token's row
  uint64_t pool_tokens, T_total;   // token rows of a (layer, K/V) plane
  uint32_t first, n, flat_first;
  FastDiv vecs;                    // 16-byte vectors of a row
  int32_t *status;
};

template <bool OUT, bool kStream>
__global__ __launch_bounds__(256) void k_page_copy(PageArgs a) {
  __shared__ int64_t slots[kPageRows];
  const uint32_t t0 = blockIdx.x * kPageRows;
  const uint32_t rows = min(kPageRows, a.n - t0);
  if (threadIdx.x < rows) {
    uint32_t at;
    int64_t slot = -1;
    if (a.s.slot_of(a.s.table, a.first + t0 + threadIdx.x, at))
      slot = at;
    else if (blockIdx.y == 0)
      set_status(a.status, KVC_ERR_SHAPE);
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
  uint8_t *pool = a.pool + (uint64_t)blockIdx.y * a.pool_tokens * a.row;
  uint8_t *flat = a.flat + ((uint64_t)blockIdx.y * a.T_total + a.flat_first + t0) * a.row;
  const uint32_t total = rows * a.vecs.d;
  for (uint32_t i0 = threadIdx.x; i0 < total; i0 += 4 * 256) {
    uint8_t *from[4], *to[4];
    u32x4 v[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t i = i0 + j * 256;
      to[j] = nullptr;
      if (i >= total) continue;
      const uint32_t r = a.vecs.div(i), c = i - r * a.vecs.d;
      const int64_t slot = slots[r];
      if (slot < 0) continue;
      uint8_t *pp = pool + (uint64_t)slot * a.row + c * 16u;
      uint8_t *fp = flat + (uint64_t)r * a.row + c * 16u;
      from[j] = OUT ? pp : fp;
      to[j] = OUT ? fp : pp;
      v[j] = move_load<kStream>(from[j]);
    }
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
      if (to[j]) move_store<kStream>(to[j], v[j]);
  }
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool paged_ok(const kvc_paged_desc *p) {
  if (!p) return false;
  if (p->n_layers < 1 || p->n_kv_heads < 1 || p->n_heads < 1) return false;
  if (p->n_heads % p->n_kv_heads != 0 || p->n_heads / p->n_kv_heads > 128) return false;
  if (p->n_heads > 4096 || p->n_layers > 32767) return false;  // launch grids
  if (p->head_dim != 64 && p->head_dim != 96 && p->head_dim != 128 && p->head_dim != 256)
    return false;
  if (p->page_tokens < 1 || p->n_pages < 1) return false;
  if ((uint64_t)p->page_tokens * p->n_pages >= (1ull << 31)) return false;
  if (p->cache_dtype > KVC_BF16 || p->io_dtype > KVC_BF16) return false;
  return !(p->cache_dtype == KVC_BF16 && p->io_dtype == KVC_F16);
}

// The batch's sizes (not its pointers).
kvc_status batch_sizes(const kvc_paged_desc *p, const kvc_paged_batch *b) {
  if (!paged_ok(p) || !b) return KVC_ERR_INVALID_ARG;
  // one block per row or row tile: launch grids below 2^32 threads
  if (b->n_seqs > (1u << 20) || b->n_tokens > (1u << 20)) return KVC_ERR_SHAPE;
  if (!b->q_start && b->n_tokens != b->n_seqs) return KVC_ERR_SHAPE;
  if (b->max_len > (1u << 30)) return KVC_ERR_SHAPE;  // a tile's end stays in 31 bits
  if (b->n_seqs && b->max_len > (uint64_t)b->table_stride * p->page_tokens) return KVC_ERR_SHAPE;
  return KVC_OK;
}

kvc_status batch_check(const kvc_paged_desc *p, const kvc_paged_batch *b, uint32_t layer,
                       const void *pool, const int32_t *dev_status) {
  const kvc_status st = batch_sizes(p, b);
  if (st != KVC_OK) return st;
  if (layer >= p->n_layers) return KVC_ERR_SHAPE;
  if (!pool || !aligned(pool, 16) || !dev_status || !aligned(dev_status, 4))
    return KVC_ERR_INVALID_ARG;
  if (b->n_seqs && (!b->lens || !aligned(b->lens, 4))) return KVC_ERR_INVALID_ARG;
  if (b->n_seqs && b->max_len && (!b->table || !aligned(b->table, 4))) return KVC_ERR_INVALID_ARG;
  if (b->q_start && !aligned(b->q_start, 4)) return KVC_ERR_INVALID_ARG;
  return KVC_OK;
}

// Rows [n][heads][head_dim] `stride` elements apart.
kvc_status rows_check(const void *p, uint64_t stride, uint32_t n, uint64_t width) {
  if (!p || !aligned(p, 16) || stride % 8 != 0) return KVC_ERR_INVALID_ARG;
  if (n > 1 && stride < width) return KVC_ERR_SHAPE;
  if (stride > (1ull << 40)) return KVC_ERR_SHAPE;
  return KVC_OK;
}

Seqs to_seqs(const kvc_paged_desc *p, const kvc_paged_batch *b) {
  Seqs s;
  s.table = b->table;
  s.lens = b->lens;
  s.q_start = b->q_start;
  s.n_seqs = b->n_seqs;
  s.table_stride = b->table_stride;
  s.n_tokens = b->n_tokens;
  s.max_len = b->max_len;
  s.n_pages = p->n_pages;
  s.page = FastDiv::make(p->page_tokens);
  return s;
}

uint64_t plane_bytes(const kvc_paged_desc *p) {
  return (uint64_t)p->n_pages * p->page_tokens * p->n_kv_heads * p->head_dim * 2;
}

kvc_status page_copy(const kvc_paged_desc *p, void *pool, const int32_t *table,
                     uint32_t table_entries, uint32_t first_token, uint32_t n_tokens, void *flat,
                     uint32_t T_total, uint32_t flat_first, bool out, int32_t *dev_status,
                     hipStream_t stream) {
  if (!paged_ok(p)) return KVC_ERR_INVALID_ARG;
  if (!pool || !aligned(pool, 16) || !dev_status || !aligned(dev_status, 4))
    return KVC_ERR_INVALID_ARG;
  if ((uint64_t)first_token + n_tokens > (uint64_t)table_entries * p->page_tokens ||
      (uint64_t)first_token + n_tokens >= (1ull << 31))
    return KVC_ERR_SHAPE;
  if (n_tokens > (1u << 27)) return KVC_ERR_SHAPE;  // launch grids below 2^32 threads
  if ((uint64_t)flat_first + n_tokens > T_total) return KVC_ERR_SHAPE;
  if (n_tokens == 0) return KVC_OK;
  if (!table || !aligned(table, 4) || !flat || !aligned(flat, 16)) return KVC_ERR_INVALID_ARG;
  const uint64_t row = (uint64_t)p->n_kv_heads * p->head_dim * 2;
  const uintptr_t pa = (uintptr_t)pool, pe = pa + 2ull * p->n_layers * plane_bytes(p);
  const uintptr_t fa = (uintptr_t)flat, fe = fa + 2ull * p->n_layers * T_total * row;
  if (pa < fe && fa < pe) return KVC_ERR_SHAPE;
  return launch_page_copy(*p, pool, table, first_token, n_tokens, flat, T_total, flat_first, out,
                          dev_status, stream) == hipSuccess
             ? KVC_OK
             : KVC_ERR_HIP;
}

kvc_status attend(const kvc_paged_desc *p, const kvc_paged_batch *b, uint32_t layer,
                  const void *pool, const void *q, uint64_t q_stride, float scale, uint32_t window,
                  void *out, uint64_t out_stride, float *lse, void *ws, uint64_t ws_bytes,
                  int32_t *dev_status, hipStream_t stream, bool prompt) {
  kvc_status st = batch_check(p, b, layer, pool, dev_status);
  if (st != KVC_OK) return st;
  if (prompt != (b->q_start != nullptr)) return KVC_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.44269504088896340736f;
  if (!(__builtin_fabsf(scale_log2) <= 3.4028234664e38f)) return KVC_ERR_INVALID_ARG;
  if ((uint64_t)b->n_tokens * p->n_heads > (1u << 23)) return KVC_ERR_SHAPE;  // launch grids
  if (b->n_seqs == 0 || b->n_tokens == 0) return KVC_OK;
  const uint64_t width = (uint64_t)p->n_heads * p->head_dim;
  if ((st = rows_check(q, q_stride, b->n_tokens, width)) != KVC_OK) return st;
  if ((st = rows_check(out, out_stride, b->n_tokens, width)) != KVC_OK) return st;
  if (q == out && q_stride != out_stride && b->n_tokens > 1) return KVC_ERR_SHAPE;
  if (!aligned(lse, 4)) return KVC_ERR_INVALID_ARG;
  const uint64_t need = attend_ws_bytes(*p, *b);
  if (need && (!ws || !aligned(ws, 256))) return KVC_ERR_INVALID_ARG;
  if (ws_bytes < need) return KVC_ERR_CAPACITY;
  AttendArgs a{};
  a.s = to_seqs(p, b);
  const uint8_t *base = static_cast<const uint8_t *>(pool);
  a.k = base + 2ull * layer * plane_bytes(p);
  a.v = base + (2ull * layer + 1) * plane_bytes(p);
  a.row = (uint64_t)p->n_kv_heads * p->head_dim;
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.n_heads = p->n_heads;
  a.n_kv_heads = p->n_kv_heads;
  a.group = p->n_heads / p->n_kv_heads;
  a.group_div = FastDiv::make(a.group);
  a.scale = scale_log2;
  a.window = window;
  a.status = dev_status;
  return launch_attend(*p, *b, a, ws, stream) == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

}  // namespace

hipError_t launch_append(const kvc_paged_desc &p, const Seqs &s, uint32_t layer, void *pool,
                         const void *k, uint64_t k_stride, const void *v, uint64_t v_stride,
                         const void *q, uint64_t q_stride, void *q_out, uint64_t q_out_stride,
                         const kvc_rope *rope, int32_t *status, hipStream_t stream) {
  AppendArgs a{};
  a.s = s;
  a.k_cache = static_cast<uint8_t *>(pool) + 2ull * layer * plane_bytes(&p);
  a.v_cache = a.k_cache + plane_bytes(&p);
  a.k = static_cast<const uint8_t *>(k);
  a.v = static_cast<const uint8_t *>(v);
  a.q = static_cast<const uint8_t *>(q);
  a.q_out = static_cast<uint8_t *>(q_out);
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.q_stride = q_stride * 2;
  a.q_out_stride = q_out_stride * 2;
  a.row = (uint64_t)p.n_kv_heads * p.head_dim * 2;
  a.head_items = FastDiv::make(p.head_dim / 16);
  a.k_items = p.n_kv_heads * (p.head_dim / 16);
  a.q_items = q ? p.n_heads * (p.head_dim / 16) : 0;
  a.head_dim = p.head_dim;
  a.status = status;
  if (rope) {
    a.rotary = rope->rotary_dim;
    a.interleaved = rope->interleaved;
    a.cos_sin = rope->cos_sin;
    a.n_positions = rope->n_positions;
  }
  const dim3 grid(s.n_tokens, (2 * a.k_items + a.q_items + 255) / 256);
  const uint64_t bytes = 2ull * s.n_tokens * (2 * a.k_items + a.q_items) * 32;
  const auto launch = [&](auto ti, auto tc) {
    using TI = decltype(ti);
    using TC = decltype(tc);
    if (bytes > kStreamBytes)
      hipLaunchKernelGGL((k_append<TI, TC, true>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_append<TI, TC, false>), grid, dim3(256), 0, stream, a);
  };
  if (p.io_dtype == KVC_F16)
    launch(f16{}, f16{});
  else if (p.cache_dtype == KVC_BF16)
    launch(bf16{}, bf16{});
  else
    launch(bf16{}, f16{});
  return hipGetLastError();
}

hipError_t launch_page_copy(const kvc_paged_desc &p, void *pool, const int32_t *table,
                            uint32_t first_token, uint32_t n_tokens, void *flat, uint32_t T_total,
                            uint32_t flat_first, bool out, int32_t *status, hipStream_t stream) {
  PageArgs a{};
  a.pool = static_cast<uint8_t *>(pool);
  a.flat = static_cast<uint8_t *>(flat);
  a.s.table = table;
  a.row = (uint64_t)p.n_kv_heads * p.head_dim * 2;
  a.pool_tokens = (uint64_t)p.n_pages * p.page_tokens;
  a.T_total = T_total;
  a.first = first_token;
  a.n = n_tokens;
  a.flat_first = flat_first;
  a.s.n_pages = p.n_pages;
  a.s.page = FastDiv::make(p.page_tokens);
  a.vecs = FastDiv::make(p.n_kv_heads * p.head_dim / 8);
  a.status = status;
  const dim3 grid((n_tokens + kPageRows - 1) / kPageRows, 2 * p.n_layers);
  const bool stream_past = 4ull * p.n_layers * n_tokens * a.row > kStreamBytes;
  const auto kernel = out ? (stream_past ? k_page_copy<true, true> : k_page_copy<true, false>)
                          : (stream_past ? k_page_copy<false, true> : k_page_copy<false, false>);
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace kvc

using namespace kvc;

extern "C" {

kvc_status kvc_validate_paged_desc(const kvc_paged_desc *p) {
  return paged_ok(p) ? KVC_OK : KVC_ERR_INVALID_ARG;
}

kvc_status kvc_append(const kvc_paged_desc *p, const kvc_paged_batch *b, uint32_t layer,
                      void *pool, const void *k, uint64_t k_stride, const void *v,
                      uint64_t v_stride, const void *q, uint64_t q_stride, void *q_out,
                      uint64_t q_out_stride, const kvc_rope *rope, int32_t *dev_status,
                      hipStream_t stream) {
  kvc_status st = batch_check(p, b, layer, pool, dev_status);
  if (st != KVC_OK) return st;
  if (rope) {
    if (rope->reserved != 0 || rope->interleaved > 1) return KVC_ERR_INVALID_ARG;
    if (rope->rotary_dim < 16 || rope->rotary_dim % 16 != 0 || rope->rotary_dim > p->head_dim)
      return KVC_ERR_INVALID_ARG;
    if (!rope->cos_sin || !aligned(rope->cos_sin, 16)) return KVC_ERR_INVALID_ARG;
  }
  if ((q == nullptr) != (q_out == nullptr)) return KVC_ERR_INVALID_ARG;
  if (b->n_seqs == 0 || b->n_tokens == 0) return KVC_OK;
  const uint64_t kw = (uint64_t)p->n_kv_heads * p->head_dim;
  const uint64_t qw = (uint64_t)p->n_heads * p->head_dim;
  if ((st = rows_check(k, k_stride, b->n_tokens, kw)) != KVC_OK) return st;
  if ((st = rows_check(v, v_stride, b->n_tokens, kw)) != KVC_OK) return st;
  if (q) {
    if ((st = rows_check(q, q_stride, b->n_tokens, qw)) != KVC_OK) return st;
    if ((st = rows_check(q_out, q_out_stride, b->n_tokens, qw)) != KVC_OK) return st;
    if (q == q_out && q_stride != q_out_stride) return KVC_ERR_SHAPE;
  }
  return launch_append(*p, to_seqs(p, b), layer, pool, k, k_stride, v, v_stride, q, q_stride,
                       q_out, q_out_stride, rope, dev_status, stream) == hipSuccess
             ? KVC_OK
             : KVC_ERR_HIP;
}

uint64_t kvc_attend_ws_bytes(const kvc_paged_desc *p, const kvc_paged_batch *b) {
  return batch_sizes(p, b) == KVC_OK ? attend_ws_bytes(*p, *b) : 0;
}

kvc_status kvc_attend(const kvc_paged_desc *p, const kvc_paged_batch *b, uint32_t layer,
                      const void *pool, const void *q, uint64_t q_stride, float scale,
                      uint32_t window, void *out, uint64_t out_stride, float *lse, void *ws,
                      uint64_t ws_bytes, int32_t *dev_status, hipStream_t stream) {
  return attend(p, b, layer, pool, q, q_stride, scale, window, out, out_stride, lse, ws, ws_bytes,
                dev_status, stream, false);
}

kvc_status kvc_attend_prompt(const kvc_paged_desc *p, const kvc_paged_batch *b, uint32_t layer,
                             const void *pool, const void *q, uint64_t q_stride, float scale,
                             uint32_t window, void *out, uint64_t out_stride, float *lse,
                             void *ws, uint64_t ws_bytes, int32_t *dev_status,
                             hipStream_t stream) {
  return attend(p, b, layer, pool, q, q_stride, scale, window, out, out_stride, lse, ws, ws_bytes,
                dev_status, stream, true);
}

kvc_status kvc_page_out(const kvc_paged_desc *p, const void *pool, const int32_t *table,
                        uint32_t table_entries, uint32_t first_token, uint32_t n_tokens,
                        void *kv_out, uint32_t T_total, uint32_t out_first, int32_t *dev_status,
                        hipStream_t stream) {
  return page_copy(p, const_cast<void *>(pool), table, table_entries, first_token, n_tokens,
                   kv_out, T_total, out_first, true, dev_status, stream);
}

kvc_status kvc_page_in(const kvc_paged_desc *p, const void *kv_in, uint32_t T_total,
                       uint32_t in_first, void *pool, const int32_t *table,
                       uint32_t table_entries, uint32_t first_token, uint32_t n_tokens,
                       int32_t *dev_status, hipStream_t stream) {
  return page_copy(p, pool, table, table_entries, first_token, n_tokens, const_cast<void *>(kv_in),
                   T_total, in_first, false, dev_status, stream);
}

}  // extern "C"

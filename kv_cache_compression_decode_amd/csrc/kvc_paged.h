// Definitions shared by the paged-cache kernels and their host code.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// Element types inside the kernels.
typedef _Float16 f16;
typedef __bf16 bf16;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 16 bytes of a 16-byte aligned address.
__device__ inline u32x4 load16(const void *p) { return *reinterpret_cast<const u32x4 *>(p); }
__device__ inline void store16(void *p, u32x4 v) { *reinterpret_cast<u32x4 *>(p) = v; }

// The same, past the caches if kStream (non-temporal).  Calls that move more
// than kStreamBytes, which the caches (256 MB) would not hold until the next
// reader anyway, use it.
constexpr uint64_t kStreamBytes = 256ull << 20;
template <bool kStream>
__device__ inline u32x4 move_load(const void *p) {
  return kStream ? __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)) : load16(p);
}
template <bool kStream>
__device__ inline void move_store(void *p, u32x4 v) {
  if (kStream)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
  else
    store16(p, v);
}

// The two elements of a dword, widened (both types widen exactly).
template <class T>
__device__ inline float elem_lo(uint32_t w);
template <class T>
__device__ inline float elem_hi(uint32_t w);
template <>
__device__ inline float elem_lo<f16>(uint32_t w) { return h2f((uint16_t)w); }
template <>
__device__ inline float elem_hi<f16>(uint32_t w) { return h2f((uint16_t)(w >> 16)); }
template <>
__device__ inline float elem_lo<bf16>(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
template <>
__device__ inline float elem_hi<bf16>(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// Two binary32 values rounded to nearest even in a dword of T.  (The hardware
// conversion to bfloat16 takes two values; NaN stays NaN.)
template <class T>
__device__ inline uint32_t pack2(float a, float b) {
  typedef T pair __attribute__((ext_vector_type(2)));
  pair r;
  r[0] = (T)a;
  r[1] = (T)b;
  return __builtin_bit_cast(uint32_t, r);
}

// Quotient by a divisor fixed for the launch, for numerators below 2^31:
// with s = ceil(log2 d) and M = ceil(2^(31+s) / d), M - 2^(31+s)/d < 1 and so
// n M / 2^(31+s) exceeds n/d by less than n / 2^(31+s) <= 1/d: the floor is
// the same.
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv make(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return {d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
  }
  __host__ __device__ inline uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * mul) >> shift);
  }
};

// A batch as the kernels read it.
struct Seqs {
  const int32_t *table;
  const int32_t *lens;
  const int32_t *q_start;  // or nullptr: sequence b has row b only
  uint32_t n_seqs, table_stride, n_tokens, max_len, n_pages;
  FastDiv page;

  // rows [row, row + n) are the sequence's new tokens, clamped to the batch
  __host__ __device__ inline void rows(uint32_t b, uint32_t &row, uint32_t &n) const {
    if (q_start == nullptr) {
      row = b;
      n = 1;
      return;
    }
    const int32_t a = q_start[b], e = q_start[b + 1];
    const int32_t lim = (int32_t)n_tokens;
    row = (uint32_t)(a < 0 ? 0 : a > lim ? lim : a);
    const uint32_t end = (uint32_t)(e < 0 ? 0 : e > lim ? lim : e);
    n = end > row ? end - row : 0;
  }
  __host__ __device__ inline bool rows_bad(uint32_t b) const {
    return q_start != nullptr &&
           (q_start[b] < 0 || q_start[b + 1] < q_start[b] || q_start[b + 1] > (int32_t)n_tokens);
  }
  // the length, within [0, max_len]
  __host__ __device__ inline int32_t clamp_len(int32_t m) const {
    return m < 0 ? 0 : m > (int32_t)max_len ? (int32_t)max_len : m;
  }
  __host__ __device__ inline bool len_out(int32_t m) const {
    return m < 0 || m > (int32_t)max_len;
  }
  __host__ __device__ inline int32_t len(uint32_t b) const { return clamp_len(lens[b]); }
  __host__ __device__ inline bool len_bad(uint32_t b) const { return len_out(lens[b]); }
  // A workgroup reports what is wrong with any sequence's rows or length.
  __device__ inline void check(int32_t *status) const {
    bool bad = false;
    for (uint32_t b = threadIdx.x; b < n_seqs; b += blockDim.x)
      bad = bad || rows_bad(b) || len_bad(b);
    if (bad) set_status(status, KVC_ERR_SHAPE);
  }
  // Slot (token row of the pool) of token `in` of page `id`.  False for an id
  // outside the pool; the slot is then one inside it, so that a caller that
  // goes on reads nothing out of bounds.
  __host__ __device__ inline bool slot_in(uint32_t id, uint32_t in, uint32_t &slot) const {
    const bool ok = id < n_pages;
    slot = (ok ? id : 0) * page.d + in;
    return ok;
  }
  // ... of token j, 0 <= j < max_len, of the sequence with page ids `ids`
  __host__ __device__ inline bool slot_of(const int32_t *ids, uint32_t j, uint32_t &slot) const {
    const uint32_t e = page.div(j);
    return slot_in((uint32_t)ids[e], j - e * page.d, slot);
  }
};

hipError_t launch_append(const kvc_paged_desc &p, const Seqs &s, uint32_t layer, void *pool,
                         const void *k, uint64_t k_stride, const void *v, uint64_t v_stride,
                         const void *q, uint64_t q_stride, void *q_out, uint64_t q_out_stride,
                         const kvc_rope *rope, int32_t *status, hipStream_t stream);
hipError_t launch_page_copy(const kvc_paged_desc &p, void *pool, const int32_t *table,
                            uint32_t first_token, uint32_t n_tokens, void *flat, uint32_t T_total,
                            uint32_t flat_first, bool out, int32_t *status, hipStream_t stream);

// One attention call.
struct AttendArgs {
  Seqs s;
  const void *k, *v;  // the layer's keys and values: [n_pages * page_tokens][C]
  uint64_t row;       // elements from one cached token to the next (C)
  const void *q;
  uint64_t q_stride;
  void *out;
  uint64_t out_stride;
  float *lse;
  // workspace: parts of row tiles, [part][rows][head_dim] unnormalised sums,
  // [part][2][rows] maxima and sums of probabilities, and what joins them
  float *part, *part_ml;
  void *info;
  uint32_t n_heads, n_kv_heads, group;
  FastDiv group_div;
  uint32_t splits;     // of the kernel for prompts
  uint32_t seq_tiles;  // row tiles of a sequence and KV head (16-row kernel)
  uint32_t step_shift;  // log2 of the tokens of a step of the 16-row kernel, at least 5
  uint32_t min_steps;  // of the 16-row kernel: steps a workgroup takes at least
  uint32_t pieces;     // its workgroups
  uint32_t wg_heads;   // KV heads to one of them (1, 2 or 4)
  uint32_t head_groups;
  bool by_unit;        // the layout of its join records
  bool whole;          // the 16-row kernel takes sequences as a whole
  float scale;      // scale * log2(e)
  uint32_t window;
  int32_t *status;
};
uint64_t attend_ws_bytes(const kvc_paged_desc &p, const kvc_paged_batch &b);
hipError_t launch_attend(const kvc_paged_desc &p, const kvc_paged_batch &b, AttendArgs a, void *ws,
                         hipStream_t stream);

}  // namespace kvc

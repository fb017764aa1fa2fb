// Attention of new tokens over the paged KV cache.
//
// A row is one (new token, query head); the rows of one sequence that share a
// KV head are (token, head in group) pairs r = i * group + g.  For a row at
// position p, with s_j = scale q.k_j over its visible tokens j,
//   m = max s_j,  l = sum exp(s_j - m),  out = sum exp(s_j - m) v_j / l,
// computed in one pass over the keys and values with a running m: the sums so
// far are multiplied by exp(m_old - m_new) when the maximum grows.
#include <algorithm>

#include "kvc_paged.h"

namespace kvc {
namespace {

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// D = A B + C on 16 x 16 tiles over 32 products.  Lane l holds of A row l%16
// and of B column l%16, products (l/16)*8 .. +7 of both; of C and D column
// l%16, rows (l/16)*4 .. +3.
template <class T>
__device__ inline f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (std::is_same<T, f16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The same on 32 x 32 tiles over 16 products: lane l holds of A row l%32 and
// of B column l%32, products (l/32)*8 .. +7; of C and D column l%32 and, as
// element i, row (i/4)*8 + (l/32)*4 + i%4.
template <class T>
__device__ inline f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (std::is_same<T, f16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Combines lanes l and l ^ 32.
__device__ inline float other_half(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

constexpr float kLn2 = 0.69314718055994530942f;
__device__ inline float ninf() { return -__builtin_inff(); }

// The probabilities are rounded to the cache's type for the second product,
// half a step of that type each (2^-11 or 2^-8 relative), while their sum l
// is taken in binary32 before the rounding.  A binary16 probability is
// scaled by 2^14 (added to the exponent, so l carries it too and it cancels
// in the quotient): its smallest step becomes 2^-38 of the largest
// probability instead of 2^-24, so a long tail of small ones is not lost.
template <class T>
constexpr float kShift = std::is_same<T, f16>::value ? 14.0f : 0.0f;
// In the kernel for prompts a probability may pass 1 by 2^kGrow before the
// sums are rescaled, and binary16 holds less than 2^16.
constexpr float kGrow = 4.0f;
template <class T>
constexpr float kShiftBig = std::is_same<T, f16>::value ? 11.0f : 0.0f;

// The scale's sign goes into the queries, and a scale of 0 makes them 0 (with
// a scale of 1), so that the kernels multiply by a positive number: the
// largest product then has the largest score, and a hidden token's -infinity
// stays one.
struct Scale {
  uint32_t q_and, q_xor;
  float s;
};
__device__ inline Scale scale_of(float s) {
  return {s == 0.0f ? 0u : 0xFFFFFFFFu, s < 0.0f ? 0x80008000u : 0u,
          s == 0.0f ? 1.0f : __builtin_fabsf(s)};
}

// 8 consecutive elements of a query row in the cache's type.
template <class TI, class TC>
__device__ inline u32x4 load_q8(const TI *p, const Scale &sc) {
  u32x4 w = load16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (w[i] & sc.q_and) ^ sc.q_xor;
  if constexpr (!std::is_same<TI, TC>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<TC>(elem_lo<TI>(w[i]), elem_hi<TI>(w[i]));
  }
  return w;
}

template <int N>
struct Words {
  uint32_t w[N];
};
// N dwords from a 4-byte aligned address, used once: marked so that they do
// not stay in the caches (an eighth faster than plain loads where HBM is the
// bound; the keys' loads, which take half a cache line at a time, are better
// kept).
template <int N>
__device__ inline Words<N> stream_words(const void *p) {
  Words<N> r;
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4 *>(p) + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[4 * i + e] = v[e];
    }
  } else if constexpr (N == 3) {
    typedef uint32_t u32x3 __attribute__((ext_vector_type(3), aligned(4)));
    const u32x3 v = __builtin_nontemporal_load(static_cast<const u32x3 *>(p));
    r.w[0] = v[0];
    r.w[1] = v[1];
    r.w[2] = v[2];
  } else {
    static_assert(N == 2, "head dimension");
    const u32x2 v = __builtin_nontemporal_load(static_cast<const u32x2 *>(p));
    r.w[0] = v[0];
    r.w[1] = v[1];
  }
  return r;
}

// The transposing LDS read: in each group of 16 lanes, lane 4r + c names 8
// bytes (elements 4c .. 4c+3 of row r), and lane i receives element i of rows
// 0 .. 3.
__device__ inline u32x2 read_tr(const uint8_t *p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4 *)p));
}

// A dword holds two elements: is either an infinity or NaN?
template <class T>
__device__ inline bool nonfinite2(uint32_t w) {
  constexpr uint32_t e = std::is_same<T, f16>::value ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}

// A row's visible tokens are counted in one run, sinks included (a batch of 45
// with windows of 4,096 and 16 sinks, 693 MB, runs at 6.1 TB/s in k_attend_rows,
// as without sinks): the s sinks
// that its window, from token lo on, does not reach stand for the tokens
// [lo - s, lo), so that only a token's lookup knows of the gap between them.
__device__ inline int32_t token_of(int32_t j, int32_t lo, int32_t first) {
  return j < lo ? j - first : j;
}

// ---------------------------------------------------- sharing out the tokens
// One new token a sequence, up to 16 query heads to a KV head: the work of a
// call is a line of steps (a tile of 32 tokens of one KV head; more tiles where
// a call's steps would pass 31 bits): head by head, in each the sequences, in
// each its tokens.  The line is cut into equal pieces, one to a workgroup,
// wherever the cuts fall, so workgroups finish together however uneven the
// lengths are (20 sequences of 1,000 to 8,900 tokens: 6.2 TB/s).  A workgroup
// that holds all of a sequence's steps writes its rows' outputs; one that holds
// a part writes its sums, maxima and unnormalised output to the workspace (at
// most two parts, at its piece's two ends) and k_attend_rows_join adds them up.
//
// A workgroup's four waves take four neighbouring KV heads of the same tokens
// where there are so many (two and two, or one, otherwise: then the waves of
// a head take its tiles in turn and are joined through LDS): a head's rows
// are short, and four side by side are fetched from HBM a tenth faster than
// four rows of one head.  "Head" below is such a group of a.wg_heads heads.
//
// Where no cache is longer than a few steps (`whole`), every workgroup takes a
// sequence and head as a whole, and nothing needs a join; there may then be
// more than 16 query heads, in row tiles of 16.

// Workgroups that the 256 CUs hold at once (by registers): the pieces at most.
constexpr uint32_t kCus = 256;
constexpr uint32_t resident(uint32_t head_dim) { return (head_dim == 256 ? 1 : 2) * kCus; }
constexpr uint32_t kRowTile = 16;
constexpr uint32_t kTok = 32;

struct Work {
  uint32_t b;  // the sequence
  int32_t len;

  // steps of a sequence: at least one, so that every row is written
  __device__ static uint32_t steps_of(const AttendArgs &a, int32_t len) {
    if (a.whole) return 1;
    const int32_t n = len - first_of(a, len);
    return (n > 0 ? ((uint32_t)n - 1) >> a.step_shift : 0) + 1;
  }
  // the window's first token
  __device__ static int32_t window_of(const AttendArgs &a, int32_t len) {
    return a.window != 0 && (uint32_t)len > a.window ? len - (int32_t)a.window : 0;
  }
  // The visible tokens are [first_of, len), the sinks counted as the tokens
  // next before the window (token_of).
  __device__ static int32_t first_of(const AttendArgs &a, int32_t len) {
    const int32_t lo = window_of(a, len);
    return lo - (int32_t)min((uint32_t)lo, a.sinks);
  }
  __device__ void load(const AttendArgs &a, uint32_t seq) {
    b = seq;
    len = a.s.len(b);
  }
  // the next sequence; after the last one, the first one's next head
  __device__ void next(const AttendArgs &a, uint32_t &head) {
    uint32_t s = b + 1;
    if (s == a.s.n_seqs) {
      s = 0;
      ++head;
    }
    load(a, s);
  }
};

// Inclusive sum over the wave's lanes (DPP: within rows of 16 lanes, then each
// row's last lane into the rows above).
__device__ inline uint32_t wave_sums(uint32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
  return x;
}

// 256 sequences' steps at a time, four to a lane (their loads in flight
// together).
struct Steps {
  uint32_t w[4], upto;  // the lane's sequences; inclusive sum over the lanes
  __device__ void load(const AttendArgs &a, uint32_t b0, bool check) {
    const uint32_t lane = threadIdx.x & 63;
    int32_t len[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) len[i] = a.s.lens[min(b0 + lane * 4 + i, a.s.n_seqs - 1)];
    uint32_t sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad = bad || a.s.len_out(len[i]);
      w[i] = b0 + lane * 4 + i < a.s.n_seqs ? Work::steps_of(a, a.s.clamp_len(len[i])) : 0;
      sum += w[i];
    }
    if (check && bad) set_status(a.status, KVC_ERR_SHAPE);
    upto = wave_sums(sum);
  }
};

// Piece w of `parts` equal pieces of the line: the first `rem` pieces are one
// step longer.
struct Pieces {
  uint32_t parts, per, rem;
  __device__ uint32_t start(uint32_t w) const { return w * per + min(w, rem); }
  __device__ uint32_t owner(uint32_t x) const {
    const uint32_t edge = rem * (per + 1);
    return x < edge ? x / (per + 1) : rem + (x - edge) / per;
  }
};

// What the workgroup that holds a sequence's first part (of a head) leaves for
// the join: whether there are others, and which workgroups hold them.  One for
// each workgroup (whose last part alone can be cut and the first of its
// sequence), or, where sequences and heads are fewer, one for each of those
// (`by_unit`), so that the join launches no idle workgroups.
struct JoinInfo {
  uint32_t cut, b, head, first, last, slot, pad[2];
};

// ------------------------------------------------- one new token a sequence
// A row tile is up to 16 of the query heads that share a KV head; all see the
// same tokens.  The waves of a head take tiles of 32 tokens in turn.
//
// What bounds it is HBM: 4 head_dim bytes a token and head, against which a
// wave has some 150 vector instructions and 16 products for 32 tokens (a
// tenth of the time).  20 sequences of 32 heads x 128 (1.33 GB): 215 us, 6.2
// TB/s (a bare read of the same pages in the same order: 6.4).
//
// Scores are computed transposed, S^T = K Q^T: lane l holds row l%16's scores
// of tokens (l/16)*4 .. +3 of both halves of the tile.  That is the layout in
// which the second product O^T = V^T P^T wants P^T, if product k = (l/16)*8+j
// stands for token (l/16)*4 + j of the first half (j < 4) or (l/16)*4 + j - 4
// of the second: P never leaves its lane.  V^T wants, for the same eight
// tokens, one dimension a lane: a lane loads E = head_dim/16 consecutive
// dimensions of its eight tokens (16 lanes cover whole rows, so the loads are
// contiguous) and the i-th product takes dimension l%16 * E + i, a byte
// permutation in registers.  Neither K nor V passes through LDS.
template <class TI, class TC, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attend_rows(AttendArgs a) {
  constexpr int E = D / 16;
  constexpr int KK = D / 32;
  constexpr int EC = E < 8 ? E : 8;  // dimensions a lane joins at a time
  __shared__ float s_o[4][16][16 * EC + 4];
  __shared__ float s_m[4][16], s_l[4][16];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t n16 = lane & 15, g4 = lane >> 4;

  // this workgroup's piece of the line, and where it begins
  Work u;
  uint32_t hg;
  uint32_t row_tile = 0;
  uint32_t at, stop, off;  // off: steps of the first sequence before the piece
  Pieces pc{gridDim.x, 1, 0};
  JoinInfo *info = static_cast<JoinInfo *>(a.info);
  if (a.whole) {  // a row tile to a workgroup: no search
    const uint32_t unit = blockIdx.x / a.head_groups;
    hg = blockIdx.x - unit * a.head_groups;
    u.load(a, unit / a.seq_tiles);
    row_tile = unit - u.b * a.seq_tiles;
    at = off = 0;
    stop = 1;
    if (threadIdx.x == 0 && a.s.len_bad(u.b)) set_status(a.status, KVC_ERR_SHAPE);
  } else {
    if (!a.by_unit && threadIdx.x == 0) info[blockIdx.x].cut = 0;
    const bool check = blockIdx.x == 0 && wave == 0;
    Steps st;
    uint32_t total = 0;
    for (uint32_t b0 = 0; b0 < a.s.n_seqs; b0 += 256) {
      st.load(a, b0, check);
      total += __builtin_amdgcn_readlane(st.upto, 63);
    }
    const uint32_t line = total * a.head_groups;
    // at least min_steps to a workgroup
    pc.parts = min(gridDim.x, (line + a.min_steps - 1) / a.min_steps);
    if (blockIdx.x >= pc.parts) return;
    pc.per = line / pc.parts;
    pc.rem = line - pc.per * pc.parts;
    at = pc.start(blockIdx.x);
    stop = pc.start(blockIdx.x + 1);
    hg = at / total;
    uint32_t x = at - hg * total;
    uint32_t base = 0;
    for (uint32_t b0 = 0;; b0 += 256) {  // some sequence holds step x < total
      if (b0 >= a.s.n_seqs) return;
      if (a.s.n_seqs > 256) st.load(a, b0, false);
      const uint64_t above = __ballot(base + st.upto > x);
      if (above == 0) {
        base += __builtin_amdgcn_readlane(st.upto, 63);
        continue;
      }
      const int src = __builtin_ctzll(above);
      uint32_t w[4], before = __builtin_amdgcn_readlane(st.upto, src);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __builtin_amdgcn_readlane(st.w[i], src);
        before -= w[i];
      }
      x -= base + before;
      uint32_t b = b0 + (uint32_t)src * 4;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (b == b0 + (uint32_t)src * 4 + i && x >= w[i]) {
          x -= w[i];
          ++b;
        }
      u.load(a, b);
      break;
    }
    off = x;
  }
  const uint32_t piece = at;
  const Scale sc_q = scale_of(a.scale);
  const TC *kcache = static_cast<const TC *>(a.k), *vcache = static_cast<const TC *>(a.v);
  bool bad = false;

  const uint32_t turns = 4 / a.wg_heads;  // waves to a head
  const uint32_t my_head = wave / turns, turn = wave - my_head * turns;
  while (at < stop && hg < a.head_groups) {
    const uint32_t hk = hg * a.wg_heads + my_head;
    // the part of sequence u.b that this workgroup holds: steps [off, off + left)
    const uint32_t steps = Work::steps_of(a, u.len);
    const uint32_t left = min(steps - off, stop - at);
    const uint32_t first = row_tile * kRowTile, rows = min(kRowTile, a.group - first);
    const bool live = n16 < rows;
    const int32_t begin = Work::first_of(a, u.len), end = u.len;
    const int32_t lo = Work::window_of(a, u.len);
    const int32_t tiles = end > begin ? (int32_t)(((uint32_t)(end - begin) + kTok - 1) / kTok) : 0;
    // a step is 2^(step_shift - 5) tiles
    const uint32_t per_step = a.step_shift - 5;
    const int32_t t_lo = a.whole ? 0 : (int32_t)(off << per_step);
    const int32_t t_hi = a.whole ? tiles : min(tiles, (int32_t)((off + left) << per_step));
    const uint32_t qh = hk * a.group + first + (live ? n16 : 0);

    float m = ninf(), l = 0.0f;
    f32x4 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = f32x4{0, 0, 0, 0};
    const int32_t *table = a.s.table + (uint64_t)u.b * a.s.table_stride;
    const TC *kbase = kcache + (uint64_t)hk * D, *vbase = vcache + (uint64_t)hk * D;
    const int32_t last = end - 1;
    // Each lane looks up one token of a tile (the others' slots come by
    // shuffle), a tile ahead of its use.
    uint32_t next_id = 0, next_in = 0;  // page id; token within the page
    auto look_up = [&](int32_t ti) {
      int32_t j = begin + ti * (int32_t)kTok + (int32_t)(lane & 31);
      j = token_of(j < last ? j : last, lo, begin);
      const uint32_t page = a.s.page.div((uint32_t)j);
      next_id = (uint32_t)table[page];
      next_in = (uint32_t)j - page * a.s.page.d;
    };
    if (t_lo + (int32_t)turn < t_hi) look_up(t_lo + (int32_t)turn);
    u32x4 qf[KK];
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) qf[kk] = u32x4{0, 0, 0, 0};
    if (live) {
      const TI *q = static_cast<const TI *>(a.q) + (uint64_t)u.b * a.q_stride +
                    (uint64_t)qh * D + g4 * 8;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) qf[kk] = load_q8<TI, TC>(q + kk * 32, sc_q);
    }

    for (int32_t ti = t_lo + (int32_t)turn; ti < t_hi; ti += (int32_t)turns) {
      const int32_t j0 = begin + ti * (int32_t)kTok;
      // slots of this lane's two key rows and eight value rows
      uint32_t slot, kslot[2], vslot[8];
      bad = !a.s.slot_in(next_id, next_in, slot) || bad;
      kslot[0] = __shfl(slot, n16);
      kslot[1] = __shfl(slot, 16 + n16);
#pragma unroll
      for (int i = 0; i < 8; ++i) vslot[i] = __shfl(slot, (i >> 2) * 16 + g4 * 4 + (i & 3));
      u32x4 kf[2][KK];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const TC *kp = kbase + (uint64_t)kslot[h] * a.row + g4 * 8;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) kf[h][kk] = load16(kp + kk * 32);
      }
      Words<E / 2> vf[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        vf[i] = stream_words<E / 2>(vbase + (uint64_t)vslot[i] * a.row + n16 * E);

      if (ti + (int32_t)turns < t_hi) look_up(ti + (int32_t)turns);

      f32x4 sc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sc[h] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) sc[h] = mfma16<TC>(kf[h][kk], qf[kk], sc[h]);
      }
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = sc[i >> 2][i & 3] * sc_q.s;
      const bool edge = j0 + (int32_t)kTok > end;  // some tokens are hidden
      if (edge) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = j0 + (i >> 2) * 16 + (int32_t)g4 * 4 + (i & 3) < end ? x[i] : ninf();
      }
      float mt = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mt = __builtin_fmaxf(mt, x[i]);
      mt = __builtin_fmaxf(mt, __shfl_xor(mt, 16));
      mt = __builtin_fmaxf(mt, __shfl_xor(mt, 32));
      const float mn = __builtin_fmaxf(m, mt);
      const float ref = mn == ninf() ? 0.0f : mn;  // nothing visible yet: exp2(-inf - 0) = 0
      const float alpha = __builtin_amdgcn_exp2f(m - ref);
      m = mn;
      float p[8];
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(x[i] - ref + kShift<TC>);
        sum += p[i];
      }
      l = __builtin_fmaf(l, alpha, sum);
      u32x4 pf;
#pragma unroll
      for (int i = 0; i < 4; ++i) pf[i] = pack2<TC>(p[2 * i], p[2 * i + 1]);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= alpha;

      if (edge) {
        // A hidden token's probability is 0, but 0 times an infinity or NaN of
        // its value row would not be.
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int w = 0; w < E / 2; ++w)
            if (j0 + (i >> 2) * 16 + (int32_t)g4 * 4 + (i & 3) >= end) vf[i].w[w] = 0;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        u32x4 vt;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vt[i] = __builtin_amdgcn_perm(vf[2 * i + 1].w[e / 2], vf[2 * i].w[e / 2],
                                        (e & 1) ? 0x07060302u : 0x05040100u);
        o[e] = mfma16<TC>(vt, pf, o[e]);
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);

    const bool some = end > begin;
    const bool single = off == 0 && left == steps;
    const uint32_t slot = at == piece ? 0 : 1;
    const uint64_t part = ((uint64_t)blockIdx.x * 2 + slot) * a.wg_heads + my_head;
    float mm = m, ll = l;
    if (turns > 1) {  // the common maximum of the head's waves and their sum
      if (lane < 16) {
        s_m[wave][lane] = m;
        s_l[wave][lane] = l;
      }
      __syncthreads();
      for (uint32_t w = 0; w < turns; ++w)
        mm = __builtin_fmaxf(mm, s_m[my_head * turns + w][n16]);
      ll = 0.0f;
      for (uint32_t w = 0; w < turns; ++w)
        ll = __builtin_fmaf(s_l[my_head * turns + w][n16],
                            __builtin_amdgcn_exp2f(s_m[my_head * turns + w][n16] -
                                                   (mm == ninf() ? 0.0f : mm)), ll);
    }
    const float f = __builtin_amdgcn_exp2f(m - (mm == ninf() ? 0.0f : mm)) *
                    (single ? (some ? 1.0f / ll : 0.0f) : 1.0f);
    if (turn == 0 && lane < rows) {
      if (!single) {
        a.part_ml[part * 32 + lane] = mm;
        a.part_ml[part * 32 + 16 + lane] = ll;
      } else if (a.lse) {
        a.lse[(uint64_t)u.b * a.n_heads + qh] =
            some ? (mm - kShift<TC> + __builtin_amdgcn_logf(ll)) * kLn2 : ninf();
      }
    }
    TI *out = static_cast<TI *>(a.out) + (uint64_t)u.b * a.out_stride + (uint64_t)qh * D;
    float *part_o = a.part + (part * 16 + n16) * D;
    if (turns == 1) {
      // a lane's 4E values are dimensions g4 * 4E on of its row
      if (live) {
        float v[4 * E];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < E; ++e) v[c * E + e] = o[e][c] * f;
        if (single) {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = some ? pack2<TI>(v[8 * i + 2 * e], v[8 * i + 2 * e + 1]) : 0u;
            store16(out + g4 * 4 * E + 8 * i, w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            *reinterpret_cast<f32x4 *>(part_o + g4 * 4 * E + 4 * i) =
                f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        }
      }
    } else {
#pragma unroll
      for (int e0 = 0; e0 < E; e0 += EC) {
        if (e0) __syncthreads();
#pragma unroll
        for (int e = 0; e < EC; ++e)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s_o[wave][n16][(g4 * 4 + c) * EC + e] = o[e0 + e][c] * f;
        __syncthreads();
        // the head's waves add up 16 rows of 16 * EC dimensions, two dimensions
        // at a time; x of them stands for dimension x / EC * E + e0 + x % EC
        for (uint32_t i = turn * 64 + lane; i < rows * 8u * EC; i += turns * 64) {
          const uint32_t r = i / (8u * EC), x = (i - r * (8u * EC)) * 2;
          float v0 = 0.0f, v1 = 0.0f;
          for (uint32_t w = 0; w < turns; ++w) {
            v0 += s_o[my_head * turns + w][r][x];
            v1 += s_o[my_head * turns + w][r][x + 1];
          }
          const uint32_t dim = E == EC ? x : (x / EC) * E + e0 + x % EC;
          if (single) {
            uint32_t *op = reinterpret_cast<uint32_t *>(
                static_cast<TI *>(a.out) + (uint64_t)u.b * a.out_stride +
                (uint64_t)(hk * a.group + first + r) * D + dim);
            *op = some ? pack2<TI>(v0, v1) : 0u;
          } else {
            float *op = a.part + (part * 16 + r) * D + dim;
            op[0] = v0;
            op[1] = v1;
          }
        }
      }
    }
    if (threadIdx.x == 0 && off == 0 && info) {
      const bool cut = left < steps;
      const uint32_t id = a.by_unit ? u.b * a.head_groups + hg : blockIdx.x;
      if (cut)
        info[id] = JoinInfo{1, u.b, hg, blockIdx.x, pc.owner(at + steps - 1), slot, {0, 0}};
      else if (a.by_unit)
        info[id].cut = 0;
    }
    at += left;
    off = 0;
    if (at < stop) {
      u.next(a, hg);
      if (turns > 1) __syncthreads();  // s_m, s_l and s_o are free again
    }
  }
  if (__ballot(bad) && lane == 0) set_status(a.status, KVC_ERR_SHAPE);
}

// Joins the parts of a sequence that k_attend_rows cut: a workgroup for each
// JoinInfo, row and head of the group.  Its W waves share the parts and are
// added up through LDS in a fixed order: 16 waves where there are few rows to
// join and so many parts to each, 4 otherwise.
template <class TI, class TC, int D, uint32_t W>
__global__ __launch_bounds__(W * 64) void k_attend_rows_join(AttendArgs a) {
  constexpr int N = D > 128 ? 4 : D > 64 ? 2 : 1;  // dimensions a lane
  constexpr uint32_t kParts = 2 * kCus;  // parts at most
  constexpr uint32_t M = (kParts + W * 64 - 1) / (W * 64);
  __shared__ float s_acc[W][D], s_f[kParts], s_m[W], s_l[W];
  const JoinInfo info = static_cast<const JoinInfo *>(a.info)[blockIdx.x];
  if (info.cut != 1 || info.b >= a.s.n_seqs || info.first > info.last || info.last >= a.pieces)
    return;
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = blockIdx.y;
  if (info.head >= a.head_groups) return;
  const uint32_t parts = info.last - info.first + 1;
  auto part_of = [&](uint32_t i) {
    return ((uint64_t)(info.first + i) * 2 + (i == 0 ? info.slot : 0)) * a.wg_heads + blockIdx.z;
  };
  // Everything is asked for before anything is waited for: the parts' maxima
  // and sums, a thread each, and each wave's first eight parts.
  float m[M], ls[M];
#pragma unroll
  for (uint32_t j = 0; j < M; ++j) {
    const uint32_t i = threadIdx.x + j * W * 64, ic = min(i, parts - 1);
    m[j] = a.part_ml[part_of(ic) * 32 + r];
    ls[j] = a.part_ml[part_of(ic) * 32 + 16 + r];
    if (i >= parts) m[j] = ninf();
  }
  const bool mine = lane * N < D;
  float x[8][N], acc[N] = {};
  auto load8 = [&](uint32_t i) {  // past the last one: the last one, unused
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float *op = a.part + (part_of(min(i + j * W, parts - 1)) * 16 + r) * D + lane * N;
#pragma unroll
      for (int e = 0; e < N; ++e) x[j][e] = mine ? op[e] : 0.0f;
    }
  };
  if (wave < parts) load8(wave);
  const int32_t len = a.s.len(info.b);
  float mm = m[0];
#pragma unroll
  for (uint32_t j = 1; j < M; ++j) mm = __builtin_fmaxf(mm, m[j]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mm = __builtin_fmaxf(mm, __shfl_xor(mm, d));
  s_m[wave] = mm;
  __syncthreads();
#pragma unroll
  for (uint32_t w = 0; w < W; ++w) mm = __builtin_fmaxf(mm, s_m[w]);
  const float ref = mm == ninf() ? 0.0f : mm;
  float l = 0.0f;
#pragma unroll
  for (uint32_t j = 0; j < M; ++j) {
    const uint32_t i = threadIdx.x + j * W * 64;
    const float f = __builtin_amdgcn_exp2f(m[j] - ref);
    if (i < parts) {
      s_f[i] = f;
      l = __builtin_fmaf(ls[j], f, l);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
  s_l[wave] = l;
  __syncthreads();
  for (uint32_t i = wave; i < parts; i += 8 * W) {
    if (i != wave) load8(i);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = i + j * W < parts ? s_f[i + j * W] : 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] = f == 0.0f ? acc[e] : __builtin_fmaf(x[j][e], f, acc[e]);
    }
  }
  if (mine)
#pragma unroll
    for (int e = 0; e < N; ++e) s_acc[wave][lane * N + e] = acc[e];
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (uint32_t w = 0; w < W; ++w) l += s_l[w];
  const bool some = len > 0;
  const float inv = some ? 1.0f / l : 0.0f;
  const uint32_t h = (info.head * a.wg_heads + blockIdx.z) * a.group + r;
  TI *out = static_cast<TI *>(a.out) + (uint64_t)info.b * a.out_stride + (uint64_t)h * D;
  if (threadIdx.x < D / 2) {
    const uint32_t x = threadIdx.x * 2;
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < W; ++w) {
      v0 += s_acc[w][x];
      v1 += s_acc[w][x + 1];
    }
    *reinterpret_cast<uint32_t *>(out + x) = some ? pack2<TI>(v0 * inv, v1 * inv) : 0u;
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(uint64_t)info.b * a.n_heads + h] =
        some ? (mm - kShift<TC> + __builtin_amdgcn_logf(l)) * kLn2 : ninf();
}

// ----------------------------------------------- 128 or 256 rows a workgroup
// For prompts: NW waves of 32 rows each share tiles of 64 tokens in LDS (32
// where head_dim is 256), so a key or value is fetched once for all of them.
// Scores are transposed here too (S^T = K Q^T on 32 x 32 tiles): a lane holds
// half a row's scores, the other half of the row in lane ^ 32, so a row's
// maximum is a chain in one lane and one exchange, and P^T is again the second
// operand of O^T = V^T P^T without leaving its lane.  V^T comes from LDS
// through the transposing read, four tokens of a dimension at a time.
//
// The next tile is loaded to registers among the products of this one's
// scores (in a burst the eight waves' loads would stall each other) and
// stored to the other buffer at the step's end: one barrier a tile.  Rows of
// K are padded by 16 bytes, so that 16-byte reads of 16 rows fall into
// different banks, rows of V to 64 or 192 bytes mod 256, so that the four rows
// of a transposing read do (no conflict left; with V padded by 32 bytes they
// were a quarter of the LDS's busy cycles).
//
// The matrix and the vector unit can work at the same time, for different
// waves.  The two waves of a SIMD leave a barrier together, so the waves from
// the fourth on (late) put off a tile's second product to the next step's
// beginning, while the others are in their first: values have three buffers
// for that (2% faster).  Software pipelining inside a wave (the next tile's
// scores among this one's exponentials) was slower, 13%: the registers that
// it holds are missing for LDS reads ahead of the matrix unit.
//
// The sums are rescaled only when some row of the wave grew by more than
// kGrow binary orders since its reference was set.
//
// 256 rows against 128: five prompts over long contexts (1.55 TFLOP) 1.63
// against 1.79 ms.
template <int D>
constexpr uint32_t kBigTok = D == 256 ? 32 : 64;  // 32: a tile's registers would not fit
template <int D>
constexpr uint32_t kKeyStride = D * 2 + 16;
template <int D>
constexpr uint32_t kValStride = D * 2 + (D == 96 ? 0 : 64);
template <int D>
constexpr uint32_t kKeyBuf = kBigTok<D> * kKeyStride<D>;
template <int D>
constexpr uint32_t kValBuf = kBigTok<D> * kValStride<D>;
constexpr int val_bufs(int waves) { return waves == 8 ? 3 : 2; }
template <int D, int NW>
constexpr uint32_t kBigLds = 2 * kKeyBuf<D> + val_bufs(NW) * kValBuf<D> + 32;
__device__ inline uint32_t next_odd_of(uint32_t i) { return i == 2 ? 0 : i + 1; }

// Rows [first, first + rows) of sequence b.
struct Tile {
  uint32_t b, row0, n;  // the sequence, its first token row and token count
  uint32_t first, rows;
};

// Where a row writes, and its visible tokens: [lo, hi) and the sinks; in a
// tree of new tokens those before `base` and those of them that its mask holds.
struct Row {
  uint32_t token, head;  // row of q and out; head within the group
  int32_t lo, hi;
  int32_t base, i;  // the sequence's first new token; this row's among them
};
__device__ inline Row row_of(const AttendArgs &a, const Tile &t, int32_t len, uint32_t r) {
  Row w;
  const uint32_t i = a.group_div.div(r);
  w.head = r - i * a.group;
  w.token = t.row0 + i;
  w.base = len - (int32_t)t.n;
  w.i = (int32_t)i;
  const int32_t pos = w.base + w.i;
  w.hi = pos < 0 ? 0 : pos + 1;
  w.lo = a.window != 0 && (uint32_t)w.hi > a.window ? w.hi - (int32_t)a.window : 0;
  return w;
}

// The lowest n bits; none or all where n is outside [0, 64].
__device__ inline uint64_t ones(int32_t n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Which of the 64 tokens from j0 on a row of a tree sees; needs j0 + 64 >
// base (all before are seen).  A row sees itself whatever its mask says, and
// nothing behind itself.
__device__ inline uint64_t tree_sees(const AttendArgs &a, const Row &row, int32_t j0) {
  const uint64_t *mask = a.mask + (uint64_t)row.token * a.mask_words;
  const auto word = [&](uint32_t k) { return k < a.mask_words ? mask[k] : 0ull; };
  const int32_t t0 = j0 - row.base;
  uint64_t see;
  if (t0 < 0) {
    see = word(0) << -t0 | ((1ull << -t0) - 1);
  } else {
    const uint32_t k = (uint32_t)t0 >> 6, sh = (uint32_t)t0 & 63;
    see = word(k) >> sh;
    if (sh) see |= word(k + 1) << (64 - sh);
  }
  const int32_t self = row.i - t0;
  see |= (uint64_t)(self >= 0 && self < 64) << (self & 63);
  return see & ones(row.hi - j0);
}

// Row tile `t` of the call: the sequences in order, of each its last tile (the
// one with the most visible tokens) first, so that a launch ends with short
// ones (6,001 tokens from the first on: a fifth less time).  Each wave
// finds it by itself: 64 sequences at a time, a scan of their tile counts.
// False if the batch has fewer tiles.
template <uint32_t kRows>
__device__ inline bool find_tile(const AttendArgs &a, uint32_t t, Tile &out) {
  const uint32_t lane = threadIdx.x & 63;
  uint32_t base = 0;
  for (uint32_t b0 = 0; b0 < a.s.n_seqs; b0 += 64) {
    uint32_t row0 = 0, n = 0;
    const uint32_t b = b0 + lane;
    if (b < a.s.n_seqs) {
      a.s.rows(b, row0, n);
    }
    const uint32_t mine = (n * a.group + kRows - 1) / kRows;
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(sum, d);
      if (lane >= (uint32_t)d) sum += o;
    }
    const uint64_t above = __ballot(base + sum > t);
    if (above) {
      const int src = __builtin_ctzll(above);
      out.b = b0 + (uint32_t)src;
      out.row0 = __shfl(row0, src);
      out.n = __shfl(n, src);
      const uint32_t k = t - base - __shfl(sum - mine, src);
      const uint32_t tiles = (out.n * a.group + kRows - 1) / kRows;
      if (k >= tiles) return false;  // only if q_start overlaps itself
      out.first = (tiles - 1 - k) * kRows;
      out.rows = min(kRows, out.n * a.group - out.first);
      return true;
    }
    base += __shfl(sum, 63);
  }
  return false;
}

// A part of a row tile's tokens: which of equal splits, or in trees which
// steps of 2^step_shift tokens; and where its sums go (the output if it is all).
struct Part {
  uint32_t lo, hi, of;  // split lo of `of`; steps [lo, hi)
  uint64_t at;
  bool all;
};

// What a row sees: up to its position (and of that a window), also sinks, or a
// tree's mask.
enum Mask { kCausal, kSinks, kTreeMask };

template <class TI, class TC, int D, int NW, Mask kMask>
__device__ __forceinline__ void attend_part(const AttendArgs &a, uint8_t *lds, const Tile &t,
                                            uint32_t hk, const Part &part) {
  constexpr bool kTree = kMask == kTreeMask;
  constexpr int TOK = kBigTok<D>, HT = TOK / 32;
  constexpr uint32_t kThreads = NW * 64, kRows = NW * 32;
  constexpr int VB = val_bufs(NW);
  constexpr int KK = D / 16;        // steps of the first product
  constexpr int DT = D / 32;        // dimension tiles of the second
  constexpr int CH = D / 8;         // 16-byte vectors of a row
  constexpr int TT = kThreads / TOK;  // threads to a token
  constexpr int NC = (CH + TT - 1) / TT;  // vectors each moves at most
  uint8_t *const s_val = lds + 2 * kKeyBuf<D>;
  uint32_t *const s_odd = reinterpret_cast<uint32_t *>(s_val + VB * kValBuf<D>);  // [3][2]
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t n32 = lane & 31, hi = lane >> 5;
  const int32_t len = a.s.len(t.b);
  const uint32_t w0 = wave * 32;
  const bool busy = w0 < t.rows;  // the wave has rows
  const bool live = w0 + n32 < t.rows;
  const Row row = row_of(a, t, len, t.first + (live ? w0 + n32 : 0));
  const Row r_first = row_of(a, t, len, t.first), r_last = row_of(a, t, len, t.first + t.rows - 1);
  const Row w_first = row_of(a, t, len, t.first + (busy ? w0 : 0));
  const Row w_last = row_of(a, t, len, t.first + (busy ? min(w0 + 31, t.rows - 1) : 0));
  // r_first's window is the first to begin; the sinks before it (token_of)
  const int32_t lo = r_first.lo;
  const int32_t begin = kMask == kSinks ? lo - (int32_t)min((uint32_t)lo, a.sinks) : lo;
  // tokens below are sinks
  const int32_t sink_end = kMask == kSinks ? max(lo, (int32_t)a.sinks) : begin;
  const int32_t end = r_last.hi, last = end - 1;
  // tokens below are seen by every row of the workgroup, of the wave
  const int32_t r_full = kTree ? r_first.base : r_first.hi;
  const int32_t w_full = kTree ? r_first.base : w_first.hi;
  const int32_t n_tiles = end > begin ? (end - begin + TOK - 1) / TOK : 0;
  constexpr uint32_t kTileShift = TOK == 64 ? 6 : 5;
  const uint32_t up = a.step_shift - kTileShift;  // of trees: log2 of a step's tiles
  const int32_t t_lo = kTree ? (int32_t)min((uint32_t)n_tiles, part.lo << up)
                             : (int32_t)((int64_t)n_tiles * part.lo / part.of);
  const int32_t t_hi = kTree ? (int32_t)min((uint32_t)n_tiles, part.hi << up)
                             : (int32_t)((int64_t)n_tiles * (part.lo + 1) / part.of);
  const uint32_t qh = hk * a.group + row.head;
  const Scale sc_q = scale_of(a.scale);

  u32x4 qf[KK];
#pragma unroll
  for (int kk = 0; kk < KK; ++kk) qf[kk] = u32x4{0, 0, 0, 0};
  if (live) {
    const TI *q = static_cast<const TI *>(a.q) + (uint64_t)row.token * a.q_stride +
                  (uint64_t)qh * D + hi * 8;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) qf[kk] = load_q8<TI, TC>(q + kk * 16, sc_q);
  }
  float ref = ninf(), l = 0.0f;
  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

  const int32_t *table = a.s.table + (uint64_t)t.b * a.s.table_stride;
  const TC *kbase = static_cast<const TC *>(a.k) + (uint64_t)hk * D;
  const TC *vbase = static_cast<const TC *>(a.v) + (uint64_t)hk * D;
  bool bad = false;

  // This thread moves vectors my_c + TT i of token my_t of each tile: one
  // lookup a tile, made a tile before the loads.
  const uint32_t my_t = threadIdx.x / TT, my_c = threadIdx.x % TT;
  const TC *kmine = kbase + my_c * 8;
  const int64_t k_to_v = static_cast<const TC *>(a.v) - static_cast<const TC *>(a.k);
  u32x4 kr[NC], vr[NC];
  uint32_t next_id = 0, next_in = 0;  // page id; token within the page
  auto look_up = [&](int32_t ti) {
    int32_t j = begin + ti * TOK + (int32_t)my_t;
    j = j < last ? j : last;
    if (kMask == kSinks) j = token_of(j, lo, begin);
    const uint32_t page = a.s.page.div((uint32_t)j);
    next_id = (uint32_t)table[page];
    next_in = (uint32_t)j - page * a.s.page.d;
  };
  auto mine = [&](int i) { return CH % TT == 0 || my_c + TT * i < (uint32_t)CH; };
  auto load_tile = [&]() {
    uint32_t slot;
    bad = !a.s.slot_in(next_id, next_in, slot) || bad;
    const TC *kp = kmine + (uint64_t)slot * a.row;
    const TC *vp = kp + k_to_v;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (mine(i)) kr[i] = load16(kp + i * TT * 8);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (mine(i)) vr[i] = load16(vp + i * TT * 8);
  };
  // Hidden tokens of a value tile must not meet the second product with an
  // infinity or NaN (0 times it is NaN): tokens past the end are zeroed, and
  // a token that some rows see and others do not is noted in s_odd.
  auto store_tile = [&](int32_t ti, uint32_t odd_at) {
    const int32_t j0 = begin + ti * TOK;
    uint8_t *kb = lds + (ti & 1) * kKeyBuf<D>;
    uint8_t *vb = s_val + (VB == 3 ? odd_at : ti & 1) * kValBuf<D>;
    if (j0 < r_last.lo || j0 + TOK > r_full) {
      bool nf = false;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (j0 + (int32_t)my_t >= end) vr[i] = u32x4{0, 0, 0, 0};
        if (mine(i))
#pragma unroll
          for (int w = 0; w < 4; ++w) nf = nf || nonfinite2<TC>(vr[i][w]);
      }
      if (nf) atomicOr(&s_odd[odd_at * 2 + (my_t >> 5)], 1u << (my_t & 31));
    }
    kb += my_t * kKeyStride<D> + my_c * 16;
    vb += my_t * kValStride<D> + my_c * 16;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (mine(i)) store16(kb + i * TT * 16, kr[i]);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (mine(i)) store16(vb + i * TT * 16, vr[i]);
  };

  // O^T += V^T P^T with the values at vb.  Lane l reads token (l%16)/4 (+ 4 for
  // the upper half), dimensions (l/16%2)*16 + (l%4)*4 .. +3 and receives four
  // tokens of dimension l%32.
  u32x4 pf[2 * HT];
  auto values = [&](const uint8_t *vb) {
    const uint8_t *vp = vb + (hi * 4 + ((lane & 15) >> 2)) * kValStride<D> +
                        ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int st = 0; st < 2 * HT; ++st)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const uint8_t *p0 = vp + st * 16 * kValStride<D> + d * 64;
        const u32x2 v0 = read_tr(p0), v1 = read_tr(p0 + 8 * kValStride<D>);
        o[d] = mfma32<TC>(u32x4{v0[0], v0[1], v1[0], v1[1]}, pf[st], o[d]);
      }
    // two products' operands ahead
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < 2 * HT * DT - 2; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
    __builtin_amdgcn_s_setprio(0);
  };
  const bool late = VB == 3 && wave >= 4;
  bool pending = false;  // pf waits for its values

  if (threadIdx.x < 6) s_odd[threadIdx.x] = 0;
  uint32_t odd_at = 0;  // of the tile being multiplied: its number mod 3
  if (t_lo < t_hi) {
    look_up(t_lo);
    load_tile();
    if (t_lo + 1 < t_hi) look_up(t_lo + 1);
    __syncthreads();  // s_odd is zero
    store_tile(t_lo, 0);
    __syncthreads();
  }
  for (int32_t ti = t_lo; ti < t_hi; ++ti) {
    const int32_t j0 = begin + ti * TOK;
    uint8_t *kb = lds + (ti & 1) * kKeyBuf<D>;
    uint8_t *vb = s_val + (VB == 3 ? odd_at : ti & 1) * kValBuf<D>;
    const bool more = ti + 1 < t_hi;
    const uint32_t next_odd = next_odd_of(odd_at);
    uint64_t odd = 0;
    // the slot that tile ti + 2 will use: last read a barrier ago
    if (threadIdx.x < 2) s_odd[next_odd_of(next_odd) * 2 + threadIdx.x] = 0;
    if (j0 < r_last.lo || j0 + TOK > r_full) {
      odd = s_odd[odd_at * 2] | (uint64_t)s_odd[odd_at * 2 + 1] << 32;
      if (odd) {
        __syncthreads();  // every wave has read the mask
        for (uint32_t i = threadIdx.x; i < (uint32_t)(TOK * CH); i += kThreads)
          if ((odd >> (i / CH)) & 1)
            store16(vb + (i / CH) * kValStride<D> + (i % CH) * 16, u32x4{0, 0, 0, 0});
        __syncthreads();
      }
    }
    if (late && pending) {  // of the tile before, two words of s_odd on
      values(s_val + next_odd_of(next_odd) * kValBuf<D>);
      pending = false;
    }
    // a wave has nothing to do where none of its rows sees a token
    if (busy && j0 < w_last.hi && (j0 + TOK > w_first.lo || (kMask == kSinks && j0 < sink_end))) {
      // the matrix unit's feeder goes first where another wave has vector work
      __builtin_amdgcn_s_setprio(1);
      f32x16 s[HT];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[h][i] = 0.0f;
        const uint8_t *kp = kb + (h * 32 + n32) * kKeyStride<D> + hi * 16;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) s[h] = mfma32<TC>(load16(kp + kk * 32), qf[kk], s[h]);
      }
      // past the last tile these load the last token again
      load_tile();
      look_up(ti + 2);
      {  // four keys ahead of the matrix unit, the loads spread out
        constexpr int total = HT * KK, depth = 4, gap = std::max(1, (total - depth) / (2 * NC + 1));
        __builtin_amdgcn_sched_group_barrier(0x100, depth, 0);
#pragma unroll
        for (int i = 0; i < total - depth; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          if (i % gap == gap - 1) __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, depth, 0);
      }
      uint64_t see = ~0ull;
      if (j0 < w_last.lo || j0 + TOK > w_full) {
        if constexpr (kMask != kCausal) {
          see = kTree ? tree_sees(a, row, j0)
                      : ones(row.hi - j0) & (~ones(row.lo - j0) | ones(sink_end - j0));
          const uint64_t mine = see >> (hi * 4);
#pragma unroll
          for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[h][i] = (mine >> (h * 32 + (i >> 2) * 8 + (i & 3))) & 1 ? s[h][i] : ninf();
        } else {
#pragma unroll
          for (int h = 0; h < HT; ++h)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int32_t j = j0 + h * 32 + (i >> 2) * 8 + (int32_t)hi * 4 + (i & 3);
              s[h][i] = j >= row.lo && j < row.hi ? s[h][i] : ninf();
            }
        }
      }
      __builtin_amdgcn_s_setprio(0);
      float mt = s[0][0];
#pragma unroll
      for (int i = 1; i < HT * 16; ++i) mt = __builtin_fmaxf(mt, s[i >> 4][i & 15]);
      mt = __builtin_fmaxf(mt, other_half(mt)) * sc_q.s;
      if (__any(mt > ref + kGrow)) {
        const float nr = __builtin_fmaxf(ref, mt);
        const float alpha = nr == ninf() ? 1.0f : __builtin_amdgcn_exp2f(ref - nr);
        ref = nr;
        l *= alpha;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= alpha;
      }
      const float off = kShiftBig<TC> - (ref == ninf() ? 0.0f : ref);
      float sum = 0.0f;
#pragma unroll
      for (int h = 0; h < HT; ++h)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          s[h][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[h][i], sc_q.s, off));
          sum += s[h][i];
        }
      l += sum;
      // tokens noted in s_odd: added lane by lane where the row sees them
      for (uint64_t left = odd; left; left &= left - 1) {
        const uint32_t jt = (uint32_t)__builtin_ctzll(left), e = jt & 31;
        const uint32_t at = (jt >> 5) * 16 + (e >> 3) * 4 + (e & 3);
        float pj = 0.0f;
#pragma unroll
        for (int i = 0; i < HT * 16; ++i) pj = at == (uint32_t)i ? s[i >> 4][i & 15] : pj;
        pj = __shfl(pj, (int)(n32 + 32 * ((e >> 2) & 1)));
        const int32_t j = j0 + (int32_t)jt;
        uint32_t sj;
        const int32_t jc = j < last ? j : last;
        a.s.slot_of(table, (uint32_t)(kMask == kSinks ? token_of(jc, lo, begin) : jc), sj);
        if (kMask != kCausal ? (see >> jt) & 1 : j >= row.lo && j < row.hi) {
          const TC *vp = vbase + (uint64_t)sj * a.row + hi * 4;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[d][i] = __builtin_fmaf(pj, (float)vp[d * 32 + (i >> 2) * 8 + (i & 3)], o[d][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8 * HT; ++i)
        pf[i >> 2][i & 3] = pack2<TC>(s[i >> 3][2 * i & 15], s[i >> 3][(2 * i & 15) + 1]);
      pending = true;
    } else {
      load_tile();
      look_up(ti + 2);
    }
    if (!late && pending) {
      values(vb);
      pending = false;
    }
    if (more) store_tile(ti + 1, next_odd);
    odd_at = next_odd;
    __syncthreads();
  }
  if (late && pending) values(s_val + next_odd_of(next_odd_of(odd_at)) * kValBuf<D>);
  if (__ballot(bad) && lane == 0) set_status(a.status, KVC_ERR_SHAPE);
  l += other_half(l);
  // A tree's workgroup may go on to another part: there, lanes without a row
  // compute as the others do and leave out the stores alone.  With nothing but
  // stores in the branches that only some lanes take, no value that goes on has
  // to change its register inside one.
  if (!kTree && !live) return;
  if (part.all) {
    const bool some = row.hi > row.lo;
    const float inv = some ? 1.0f / l : 0.0f;
    TI *op = static_cast<TI *>(a.out) + (uint64_t)row.token * a.out_stride + (uint64_t)qh * D +
             hi * 4;
    u32x2 w[DT][4];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[d][i][0] = some ? pack2<TI>(o[d][4 * i] * inv, o[d][4 * i + 1] * inv) : 0u;
        w[d][i][1] = some ? pack2<TI>(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv) : 0u;
      }
    if (live) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x2 *>(op + d * 32 + i * 8) = w[d][i];
    }
    if (live && hi == 0 && a.lse)
      a.lse[(uint64_t)row.token * a.n_heads + qh] =
          some ? (ref - kShiftBig<TC> + __builtin_amdgcn_logf(l)) * kLn2 : ninf();
  } else {
    float *op = a.part + (part.at * kRows + w0 + n32) * D + hi * 4;
    if (live) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4 *>(op + d * 32 + i * 8) =
              f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
    }
    if (live && hi == 0) {
      a.part_ml[part.at * (2 * kRows) + w0 + n32] = ref;
      a.part_ml[part.at * (2 * kRows) + kRows + w0 + n32] = l;
    }
  }
}

template <class TI, class TC, int D, int NW, Mask kMask>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : 8 / NW) void k_attend_tile(AttendArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const uint32_t hk = blockIdx.x % a.n_kv_heads;
  const uint32_t rest = blockIdx.x / a.n_kv_heads;
  const uint32_t split = rest % a.splits, tile = rest / a.splits;
  Tile t;
  if (blockIdx.x == 0) a.s.check(a.status);
  if (!find_tile<NW * 32>(a, tile, t)) return;
  attend_part<TI, TC, D, NW, kMask>(
      a, lds, t, hk,
      Part{split, 0, a.splits, ((uint64_t)tile * a.n_kv_heads + hk) * a.splits + split,
           a.splits == 1});
}

// Joins the splits of k_attend_tile: a wave per (row tile, KV head, row).
template <class TI, class TC, int D, uint32_t kRows>
__global__ __launch_bounds__(256) void k_attend_tile_join(AttendArgs a) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x / (kRows / 4);
  const uint32_t r = (blockIdx.x % (kRows / 4)) * 4 + (threadIdx.x >> 6);
  const uint32_t hk = unit % a.n_kv_heads, tile = unit / a.n_kv_heads;
  Tile t;
  if (!find_tile<kRows>(a, tile, t)) return;
  if (r >= t.rows) return;
  const Row row = row_of(a, t, a.s.len(t.b), t.first + r);
  const uint64_t part = ((uint64_t)tile * a.n_kv_heads + hk) * a.splits;
  float mm = ninf();
  for (uint32_t s = lane; s < a.splits; s += 64)
    mm = __builtin_fmaxf(mm, a.part_ml[(part + s) * (2 * kRows) + r]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mm = __builtin_fmaxf(mm, __shfl_xor(mm, d));
  const float ref = mm == ninf() ? 0.0f : mm;
  float acc[(D + 127) / 128 * 2] = {};
  float l = 0.0f;
#pragma unroll 4
  for (uint32_t s = 0; s < a.splits; ++s) {
    const float f = __builtin_amdgcn_exp2f(a.part_ml[(part + s) * (2 * kRows) + r] - ref);
    l = __builtin_fmaf(a.part_ml[(part + s) * (2 * kRows) + kRows + r], f, l);
    const float *op = a.part + ((part + s) * kRows + r) * D;
#pragma unroll
    for (int k = 0; k < (D + 127) / 128; ++k) {
      const uint32_t dim = (lane + 64 * k) * 2;
      if (dim < D) {
        acc[2 * k] = __builtin_fmaf(op[dim], f, acc[2 * k]);
        acc[2 * k + 1] = __builtin_fmaf(op[dim + 1], f, acc[2 * k + 1]);
      }
    }
  }
  const bool some = row.hi > row.lo;
  const float inv = some ? 1.0f / l : 0.0f;
  const uint32_t h = hk * a.group + row.head;
  uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<TI *>(a.out) +
                                               (uint64_t)row.token * a.out_stride +
                                               (uint64_t)h * D);
#pragma unroll
  for (int k = 0; k < (D + 127) / 128; ++k) {
    const uint32_t dim = (lane + 64 * k) * 2;
    if (dim < D) out[dim / 2] = some ? pack2<TI>(acc[2 * k] * inv, acc[2 * k + 1] * inv) : 0u;
  }
  if (lane == 0 && a.lse)
    a.lse[(uint64_t)row.token * a.n_heads + h] =
        some ? (mm - kShiftBig<TC> + __builtin_amdgcn_logf(l)) * kLn2 : ninf();
}

// ---------------------------------------------------------- trees of new tokens
// The same tiles, shared out as k_attend_rows does: the work of a KV head is a
// line of steps, the sequences in order, in each its row tiles, in each its
// tokens; as many workgroups as the chip holds take equal pieces of the heads'
// lines, wherever the cuts fall.  A drafted tree is a few dozen rows over a long
// cache, and caches of a batch differ by a factor of ten: cut into equal splits
// of whole sequences, the longest one's workgroups ran on alone.
//
// Neighbouring workgroups take the same piece of neighbouring heads, whose rows
// lie side by side in HBM.  A sequence's rows are shared evenly among its tiles
// (in waves of 32), and every tile reads the keys and values again: with 256
// rows a workgroup needs a tile of 64 tokens (32 KB at head_dim 128) every 2.7
// us, half of what HBM gives 256 of them, so no locality among a sequence's tiles
// is asked for.
//
// 15 trees of 17 to 60 tokens over 1,500 to 16,000, 8 heads to each of 8 KV heads
// (156 GFLOP): 258 to 264 us (331 in equal splits of whole sequences; 300 with
// 128-row tiles).  The matrix units are busy 27% of it and the vector units as much;
// 27% of the tiles' rows are empty.  Steps weighted by their tile's waves moved
// the cuts but gained nothing.

// Piece w of `parts` pieces of a line: equal lines one after another, in as many
// pieces each, are cut at their ends.
struct TreePieces {
  uint32_t parts, line;
  __device__ uint32_t start(uint32_t w) const { return (uint32_t)((uint64_t)w * line / parts); }
  __device__ uint32_t owner(uint32_t x) const {
    return (uint32_t)((((uint64_t)x + 1) * parts - 1) / line);
  }
};

// A row tile whose tokens several workgroups hold, for the join: which they are
// and what its rows are.  One for each workgroup (whose last part alone can be
// cut and its tile's first), or, where they are fewer, one for each tile and
// head (`by_unit`), so that the join launches no idle workgroups.
struct TreeInfo {
  uint32_t cut, head, first, last, slot;  // first, last: pieces of the head
  int32_t len;
  Tile t;
  uint32_t pad[5];
};
// The workspace's records begin with the tiles that the call has.
struct TreeHead {
  uint32_t tiles, pad[15];
};

template <uint32_t kRows>
struct TreeWork {
  uint32_t b, row0, n, tiles, steps;
  uint32_t before, tile0;  // rows (raw) and tiles of the sequences before it

  // Rows that overlap others (q_start falls somewhere) are left out, so that
  // the tiles are no more than the host counted.
  __device__ static uint32_t rows_of(const AttendArgs &a, uint32_t raw, uint32_t before) {
    return before + raw <= a.s.n_tokens ? raw : 0;
  }
  __device__ static uint32_t tiles_of(const AttendArgs &a, uint32_t n) {
    return (n * a.group + kRows - 1) / kRows;
  }
  __device__ static uint32_t steps_of(const AttendArgs &a, int32_t len) {
    return (len > 0 ? ((uint32_t)len - 1) >> a.step_shift : 0) + 1;
  }
  __device__ static uint32_t saturate(uint32_t rows) { return min(rows, 1u << 21); }
  __device__ void load(const AttendArgs &a) {
    a.s.rows(b, row0, n);
    const uint32_t raw = n;
    n = rows_of(a, raw, before);
    tiles = tiles_of(a, n);
    steps = steps_of(a, a.s.len(b));
    upto = saturate(before + raw);
  }
  // the next sequence with rows; false behind the last one
  __device__ bool next(const AttendArgs &a) {
    do {
      before = upto;
      tile0 += tiles;
      if (++b >= a.s.n_seqs) return false;
      load(a);
    } while (tiles == 0);
    return true;
  }
  // rows [first, first + rows) of the sequence's tile k
  __device__ static Tile tile(const AttendArgs &a, uint32_t b, uint32_t row0, uint32_t n,
                              uint32_t tiles, uint32_t k) {
    const uint32_t all = n * a.group;
    // (more tiles than waves: a last one could stay without rows)
    const uint32_t per = tiles > kRows / 32 ? kRows : ((all + tiles - 1) / tiles + 31) & ~31u;
    Tile t;
    t.b = b;
    t.row0 = row0;
    t.n = n;
    t.first = k * per;
    t.rows = min(per, all - t.first);
    return t;
  }
  // The sequence that holds step x of the line, with x left relative to it; or,
  // with find false, the line's steps, and tile0 as the call's tiles.
  __device__ bool search(const AttendArgs &a, bool find, uint32_t &x, uint32_t &total) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t rows0 = 0, tiles0 = 0, sum0 = 0;
    for (uint32_t b0 = 0; b0 < a.s.n_seqs; b0 += 64) {
      uint32_t first = 0, raw = 0;
      int32_t length = 0;
      if (b0 + lane < a.s.n_seqs) {
        a.s.rows(b0 + lane, first, raw);
        length = a.s.len(b0 + lane);
      }
      const uint32_t rows1 = wave_sums(raw);
      const uint32_t mine = tiles_of(a, rows_of(a, raw, rows0 + rows1 - raw));
      const uint32_t w = mine * steps_of(a, length);
      const uint32_t tiles1 = wave_sums(mine), sum1 = wave_sums(w);
      if (find) {
        const uint64_t above = __ballot(sum0 + sum1 > x);
        if (above) {
          const int src = __builtin_ctzll(above);
          b = b0 + (uint32_t)src;
          before = saturate(rows0 + __builtin_amdgcn_readlane(rows1 - raw, src));
          tile0 = tiles0 + __builtin_amdgcn_readlane(tiles1 - mine, src);
          x -= sum0 + __builtin_amdgcn_readlane(sum1 - w, src);
          load(a);
          return true;
        }
      }
      rows0 = saturate(rows0 + __builtin_amdgcn_readlane(rows1, 63));
      tiles0 += __builtin_amdgcn_readlane(tiles1, 63);
      sum0 += __builtin_amdgcn_readlane(sum1, 63);
    }
    total = sum0;
    tile0 = tiles0;
    return false;
  }

 private:
  uint32_t upto;
};

template <class TI, class TC, int D, int NW>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : 8 / NW) void k_attend_tree(AttendArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  using W = TreeWork<NW * 32>;
  TreeHead *const head = static_cast<TreeHead *>(a.info);
  TreeInfo *const info = reinterpret_cast<TreeInfo *>(head + 1);
  if (head && !a.by_unit && threadIdx.x == 0) info[blockIdx.x].cut = 0;
  if (blockIdx.x == 0) {
    a.s.check(a.status);
    a.s.check_new(a.max_new, a.status);
  }
  const uint32_t w = blockIdx.x / a.n_kv_heads, hk = blockIdx.x - w * a.n_kv_heads;
  W u;
  uint32_t x = 0, total = 0;
  u.search(a, false, x, total);
  if (head && blockIdx.x == 0 && threadIdx.x == 0) head->tiles = u.tile0;
  // at least min_steps to a workgroup
  const TreePieces pc{min(a.pieces, (total + a.min_steps - 1) / a.min_steps), total};
  if (w >= pc.parts) return;
  uint32_t at = pc.start(w);
  const uint32_t piece = at, stop = pc.start(w + 1);
  x = at;
  if (!u.search(a, true, x, total)) return;
  uint32_t k = x / u.steps, off = x - k * u.steps;
  while (at < stop) {
    const uint32_t left = min(u.steps - off, stop - at);
    const bool all = left == u.steps;
    const uint32_t slot = at == piece ? 0 : 1;
    const Tile t = W::tile(a, u.b, u.row0, u.n, u.tiles, k);
    attend_part<TI, TC, D, NW, kTreeMask>(
        a, lds, t, hk, Part{off, off + left, 0, (uint64_t)blockIdx.x * 2 + slot, all});
    const uint32_t id = a.by_unit ? (u.tile0 + k) * a.n_kv_heads + hk : blockIdx.x;
    if (threadIdx.x == 0 && off == 0 && head && id < a.infos) {
      if (!all)
        info[id] = TreeInfo{1, hk, w, pc.owner(at + u.steps - 1), slot, a.s.len(u.b), t, {}};
      else if (a.by_unit)
        info[id].cut = 0;
    }
    at += left;
    off = 0;
    if (at < stop && ++k == u.tiles) {
      k = 0;
      if (!u.next(a)) return;
    }
  }
}

// A tree of up to 16 R rows to a KV head: as k_attend_rows, without LDS, the
// keys and values of 32 tokens going from HBM to registers once for all rows.
// Each wave takes a piece of a head's line by itself; neighbouring waves the
// same piece of neighbouring heads.  HBM bounds it: 12 trees of 1 to 8 tokens over
// 900 to 9,000, 32 heads x 128 (562 MB), 92 us, 6.1 TB/s (k_attend_tree with
// 128-row tiles: 114).
template <class TI, class TC, int D, int R>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_attend_few(AttendArgs a) {
  constexpr int E = D / 16, KK = D / 32;
  constexpr uint32_t kRows = 16 * R;
  using W = TreeWork<kRows>;
  const uint32_t lane = threadIdx.x & 63, n16 = lane & 15, g4 = lane >> 4;
  const uint32_t v = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t w = v / a.n_kv_heads, hk = v - w * a.n_kv_heads;
  TreeHead *const head = static_cast<TreeHead *>(a.info);
  TreeInfo *const info = reinterpret_cast<TreeInfo *>(head + 1);
  if (head && !a.by_unit && lane == 0 && v < a.infos) info[v].cut = 0;
  if (blockIdx.x == 0) {
    a.s.check(a.status);
    a.s.check_new(a.max_new, a.status);
  }
  if (w >= a.pieces) return;
  W u;
  uint32_t x0 = 0, total = 0;
  u.search(a, false, x0, total);
  if (head && v == 0 && lane == 0) head->tiles = u.tile0;
  const TreePieces pc{min(a.pieces, (total + a.min_steps - 1) / a.min_steps), total};
  if (w >= pc.parts) return;
  uint32_t at = pc.start(w);
  const uint32_t piece = at, stop = pc.start(w + 1);
  x0 = at;
  if (!u.search(a, true, x0, total)) return;
  uint32_t k = x0 / u.steps, off = x0 - k * u.steps;
  const Scale sc_q = scale_of(a.scale);
  const TC *const kbase = static_cast<const TC *>(a.k) + (uint64_t)hk * D;
  const TC *const vbase = static_cast<const TC *>(a.v) + (uint64_t)hk * D;
  bool bad = false;
  while (at < stop) {
    const uint32_t left = min(u.steps - off, stop - at);
    const bool all = left == u.steps;
    const Tile t = W::tile(a, u.b, u.row0, u.n, u.tiles, k);
    const int32_t len = a.s.len(u.b), base = len - (int32_t)u.n, last = len - 1;
    const int32_t tiles = len > 0 ? (int32_t)(((uint32_t)len + kTok - 1) / kTok) : 0;
    const int32_t t_lo = min(tiles, (int32_t)(off << (a.step_shift - 5)));
    const int32_t t_hi = min(tiles, (int32_t)((off + left) << (a.step_shift - 5)));
    const int32_t *table = a.s.table + (uint64_t)u.b * a.s.table_stride;
    // Each lane looks up one token of a tile, a tile ahead of its use.
    uint32_t next_id = 0, next_in = 0;
    auto look_up = [&](int32_t ti) {
      int32_t j = ti * (int32_t)kTok + (int32_t)(lane & 31);
      j = j < last ? j : last;
      const uint32_t page = a.s.page.div((uint32_t)j);
      next_id = (uint32_t)table[page];
      next_in = (uint32_t)j - page * a.s.page.d;
    };
    if (t_lo < t_hi) look_up(t_lo);
    float m[R], l[R];
    f32x4 o[R][E];
    u32x4 qf[R][KK];
    Row row[R];
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      live[r] = r * 16 + n16 < t.rows;
      row[r] = row_of(a, t, len, t.first + (live[r] ? r * 16 + n16 : 0));
      m[r] = ninf();
      l[r] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = f32x4{0, 0, 0, 0};
      const TI *q = static_cast<const TI *>(a.q) + (uint64_t)row[r].token * a.q_stride +
                    (uint64_t)(hk * a.group + row[r].head) * D + g4 * 8;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
        qf[r][kk] = live[r] ? load_q8<TI, TC>(q + kk * 32, sc_q) : u32x4{0, 0, 0, 0};
    }

    for (int32_t ti = t_lo; ti < t_hi; ++ti) {
      const int32_t j0 = ti * (int32_t)kTok;
      // slots of this lane's two key rows and eight value rows
      uint32_t slot, kslot[2], vslot[8];
      bad = !a.s.slot_in(next_id, next_in, slot) || bad;
      kslot[0] = __shfl(slot, n16);
      kslot[1] = __shfl(slot, 16 + n16);
#pragma unroll
      for (int i = 0; i < 8; ++i) vslot[i] = __shfl(slot, (i >> 2) * 16 + g4 * 4 + (i & 3));
      u32x4 kf[2][KK];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const TC *kp = kbase + (uint64_t)kslot[h] * a.row + g4 * 8;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) kf[h][kk] = load16(kp + kk * 32);
      }
      Words<E / 2> vf[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        vf[i] = stream_words<E / 2>(vbase + (uint64_t)vslot[i] * a.row + n16 * E);
      if (ti + 1 < t_hi) look_up(ti + 1);

      float x[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 sc = {0, 0, 0, 0};
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) sc = mfma16<TC>(kf[h][kk], qf[r][kk], sc);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[r][h * 4 + i] = sc[i] * sc_q.s;
        }
      // token of element i: (i >> 2) * 16 + g4 * 4 + (i & 3)
      const bool edge = j0 + (int32_t)kTok > base;  // some tokens are hidden from some rows
      uint32_t see[R], odd = 0;
      if (edge) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          see[r] = (uint32_t)tree_sees(a, row[r], j0);
          const uint32_t mine = see[r] >> (g4 * 4);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[r][i] = (mine >> ((i >> 2) * 16 + (i & 3))) & 1 ? x[r][i] : ninf();
        }
        // A hidden token's probability is 0, but 0 times an infinity or NaN of
        // its value row would not be: such rows are left out of the product
        // and added below where they are seen.
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t e0 = (i >> 2) * 16 + (i & 3);
          bool nf = false;
#pragma unroll
          for (int e = 0; e < E / 2; ++e) nf = nf || nonfinite2<TC>(vf[i].w[e]);
          const uint64_t any = __ballot(nf);
          if (any) {
#pragma unroll
            for (uint32_t g = 0; g < 4; ++g)
              if ((any >> (16 * g)) & 0xFFFF) odd |= 1u << (e0 + g * 4);
          }
          if ((odd >> (e0 + g4 * 4)) & 1)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) vf[i].w[e] = 0;
        }
      }
      u32x4 pf[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float mt = x[r][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mt = __builtin_fmaxf(mt, x[r][i]);
        mt = __builtin_fmaxf(mt, __shfl_xor(mt, 16));
        mt = __builtin_fmaxf(mt, __shfl_xor(mt, 32));
        const float mn = __builtin_fmaxf(m[r], mt);
        const float ref = mn == ninf() ? 0.0f : mn;  // nothing visible yet: exp2(-inf - 0) = 0
        const float alpha = __builtin_amdgcn_exp2f(m[r] - ref);
        m[r] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[r][i] = __builtin_amdgcn_exp2f(x[r][i] - ref + kShiftBig<TC>);
          sum += x[r][i];
        }
        l[r] = __builtin_fmaf(l[r], alpha, sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) pf[r][i] = pack2<TC>(x[r][2 * i], x[r][2 * i + 1]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] *= alpha;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        u32x4 vt;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vt[i] = __builtin_amdgcn_perm(vf[2 * i + 1].w[e / 2], vf[2 * i].w[e / 2],
                                        (e & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int r = 0; r < R; ++r) o[r][e] = mfma16<TC>(vt, pf[r], o[r][e]);
      }
      for (; odd; odd &= odd - 1) {
        const uint32_t jt = (uint32_t)__builtin_ctz(odd);
        const int32_t j = j0 + (int32_t)jt;
        uint32_t sj;
        a.s.slot_of(table, (uint32_t)(j < last ? j : last), sj);
        const TC *vp = vbase + (uint64_t)sj * a.row + g4 * 4 * E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float pj = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) pj = (jt >> 4) * 4 + (jt & 3) == (uint32_t)i ? x[r][i] : pj;
          pj = __shfl(pj, (int)(((jt >> 2) & 3) * 16 + n16));
          if ((see[r] >> jt) & 1)
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                o[r][e][c] = __builtin_fmaf(pj, (float)vp[c * E + e], o[r][e][c]);
        }
      }
    }
    const uint32_t slot = at == piece ? 0 : 1;
    const uint64_t part = (uint64_t)v * 2 + slot;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor(l[r], 16);
      l[r] += __shfl_xor(l[r], 32);
      // (every lane computes; those without a row leave out the stores alone)
      // a lane's 4 E values are dimensions g4 * 4 E on of its row
      const bool some = row[r].hi > row[r].lo;
      const float f = all ? (some ? 1.0f / l[r] : 0.0f) : 1.0f;
      float val[4 * E];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) val[c * E + e] = o[r][e][c] * f;
      const uint32_t h = hk * a.group + row[r].head;
      if (all) {
        TI *out = static_cast<TI *>(a.out) + (uint64_t)row[r].token * a.out_stride +
                  (uint64_t)h * D + g4 * 4 * E;
        u32x4 wv[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            wv[i][e] = some ? pack2<TI>(val[8 * i + 2 * e], val[8 * i + 2 * e + 1]) : 0u;
        if (live[r]) {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) store16(out + 8 * i, wv[i]);
        }
        if (live[r] && g4 == 0 && a.lse)
          a.lse[(uint64_t)row[r].token * a.n_heads + h] =
              some ? (m[r] - kShiftBig<TC> + __builtin_amdgcn_logf(l[r])) * kLn2 : ninf();
      } else {
        float *op = a.part + (part * kRows + r * 16 + n16) * D + g4 * 4 * E;
        if (live[r]) {
#pragma unroll
          for (int i = 0; i < E; ++i)
            *reinterpret_cast<f32x4 *>(op + 4 * i) =
                f32x4{val[4 * i], val[4 * i + 1], val[4 * i + 2], val[4 * i + 3]};
        }
        if (live[r] && g4 == 0) {
          a.part_ml[part * (2 * kRows) + r * 16 + n16] = m[r];
          a.part_ml[part * (2 * kRows) + kRows + r * 16 + n16] = l[r];
        }
      }
    }
    const uint32_t id = a.by_unit ? (u.tile0 + k) * a.n_kv_heads + hk : v;
    if (lane == 0 && off == 0 && head && id < a.infos) {
      if (!all)
        info[id] = TreeInfo{1, hk, w, pc.owner(at + u.steps - 1), slot, len, t, {}};
      else if (a.by_unit)
        info[id].cut = 0;
    }
    at += left;
    off = 0;
    if (at < stop && ++k == u.tiles) {
      k = 0;
      if (!u.next(a)) break;
    }
  }
  if (__ballot(bad) && lane == 0) set_status(a.status, KVC_ERR_SHAPE);
}

// Joins the parts of a row tile that k_attend_tree or k_attend_few cut.  A workgroup takes 8 / S
// rows of a TreeInfo; a row has S groups of D / 4 lanes, which take its parts
// in turn and are added up through LDS in a fixed order.  What it reads are the
// parts, once: 4 D + 8 bytes for each row and part.
template <class TI, class TC, int D, uint32_t kRows, uint32_t S>
__global__ __launch_bounds__(D * 2) void k_attend_tree_join(AttendArgs a) {
  constexpr uint32_t L = D / 4, R = 8 / S;
  constexpr int U = S == 1 ? 4 : 8;  // parts in flight to a lane
  __shared__ float s_acc[8][D], s_l[8];
  const TreeHead *const head = static_cast<const TreeHead *>(a.info);
  const TreeInfo info = reinterpret_cast<const TreeInfo *>(head + 1)[blockIdx.x];
  // records behind the call's tiles were not written
  if (a.by_unit && blockIdx.x >= head->tiles * a.n_kv_heads) return;
  const uint32_t r0 = blockIdx.y * R;
  if (info.cut != 1 || r0 >= info.t.rows || info.first > info.last || info.last >= a.pieces ||
      info.head >= a.n_kv_heads || info.t.rows > kRows)
    return;
  const uint32_t g = threadIdx.x / L, lane = threadIdx.x - g * L, stream = g % S;
  const uint32_t r = r0 + g / S, rc = min(r, info.t.rows - 1);
  const uint32_t parts = info.last - info.first + 1;
  const auto part_of = [&](uint32_t i) {
    return ((uint64_t)(info.first + i) * a.n_kv_heads + info.head) * 2 + (i == 0 ? info.slot : 0);
  };
  float m = ninf(), l = 0.0f;
  f32x4 acc = {0, 0, 0, 0};
  for (uint32_t i0 = stream; i0 < parts; i0 += U * S) {
    float pm[U], pl[U];
    f32x4 x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {  // past the last one: the last one, unused
      const uint64_t part = part_of(min(i0 + j * S, parts - 1));
      pm[j] = a.part_ml[part * (2 * kRows) + rc];
      pl[j] = a.part_ml[part * (2 * kRows) + kRows + rc];
      x[j] = *reinterpret_cast<const f32x4 *>(a.part + (part * kRows + rc) * D + lane * 4);
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j * S >= parts) pm[j] = ninf();
      top = __builtin_fmaxf(top, pm[j]);
    }
    const float ref = top == ninf() ? 0.0f : top;
    const float alpha = __builtin_amdgcn_exp2f(m - ref);
    m = top;
    l *= alpha;
    acc *= alpha;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j * S >= parts) continue;
      // A part in which the row sees nothing adds zeros; so does one whose scores
      // are all minus infinity.  Its maximum is that of one whose scores are all
      // NaN, too, which must come through: no part is left out by its maximum.
      const float f = __builtin_amdgcn_exp2f(pm[j] - ref);
      l = __builtin_fmaf(pl[j], f, l);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(x[j][e], f, acc[e]);
    }
  }
  if constexpr (S > 1) {
    static_assert(S == 8, "one row to a workgroup");
    __shared__ float s_m[8];
    if (lane == 0) s_m[stream] = m;
    __syncthreads();
    float mm = s_m[0];
#pragma unroll
    for (uint32_t i = 1; i < S; ++i) mm = __builtin_fmaxf(mm, s_m[i]);
    const float f = __builtin_amdgcn_exp2f(m - (mm == ninf() ? 0.0f : mm));
    if (lane == 0) s_l[stream] = l * f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s_acc[stream][lane * 4 + e] = acc[e] * f;
    __syncthreads();
    if (g != 0) return;
    m = mm;
    l = 0.0f;
    acc = f32x4{0, 0, 0, 0};
#pragma unroll
    for (uint32_t i = 0; i < S; ++i) {
      l += s_l[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] += s_acc[i][lane * 4 + e];
    }
  }
  if (r >= info.t.rows) return;
  const Row row = row_of(a, info.t, info.len, info.t.first + r);
  const bool some = row.hi > row.lo;
  const float inv = some ? 1.0f / l : 0.0f;
  const uint32_t h = info.head * a.group + row.head;
  u32x2 v;
  v[0] = some ? pack2<TI>(acc[0] * inv, acc[1] * inv) : 0u;
  v[1] = some ? pack2<TI>(acc[2] * inv, acc[3] * inv) : 0u;
  *reinterpret_cast<u32x2 *>(static_cast<TI *>(a.out) + (uint64_t)row.token * a.out_stride +
                             (uint64_t)h * D + lane * 4) = v;
  if (lane == 0 && a.lse)
    a.lse[(uint64_t)row.token * a.n_heads + h] =
        some ? (m - kShiftBig<TC> + __builtin_amdgcn_logf(l)) * kLn2 : ninf();
}

// ------------------------------------------------------------------- host
struct Plan {
  uint32_t rows;      // 16, 128 or 256 to a workgroup
  uint32_t grid;      // workgroups of the 16-row kernel
  uint32_t wg_heads;  // KV heads to one of them
  bool whole, join;   // it cuts nothing; a second launch is needed
  bool by_unit;       // JoinInfo records: one for each sequence and head
  uint64_t infos;
  uint32_t shift;     // log2 of the tokens of a step
  uint32_t pieces;     // of the line: workgroups, for trees those of a head
  uint32_t min_steps;  // steps to a workgroup at least
  uint32_t tiles, splits;             // of k_attend_tile
  uint64_t part, part_ml, info, total;  // workspace offsets
};

// Caches of at most this many steps are not cut.
constexpr uint32_t kWholeSteps = 16;

// A 16-row workgroup takes at least a step for each wave of a head.
uint32_t min_steps(const Plan &w) { return 4 / w.wg_heads; }

// Caches of at most this many tokens are not cut for a tree's rows: the tiles of
// a cut would cost less than its join.
constexpr uint32_t kWholeTree = 256;

Plan make_tree_plan(const kvc_paged_desc &p, const kvc_paged_batch &b, uint32_t max_new) {
  Plan w{};
  w.wg_heads = 1;
  const uint32_t group = p.n_heads / p.n_kv_heads;
  const uint64_t most = (uint64_t)max_new * group, avg = (uint64_t)b.n_tokens * group / b.n_seqs;
  // 32 rows of 256 dimensions do not fit the registers.  The lower tiles are for
  // sequences that fill one of them on average: 8 heads to each of 8 KV heads, 16
  // sequences of 8,000, 128 rows each take 132 us in tiles of 128 and 147 in tiles
  // of 256, 136 rows 168 and 158, 384 rows 355 and 284; 48 sequences of 3,000: 128
  // rows 169 and 176, 136 rows 257 and 189.
  w.rows = most <= 16                         ? 16
           : most <= 32 && p.head_dim != 256  ? 32
           : avg <= 128 || p.head_dim == 256  ? 128
                                              : 256;
  w.tiles = (uint32_t)((uint64_t)b.n_tokens * group / w.rows) + std::min(b.n_seqs, b.n_tokens);
  const uint64_t units = (uint64_t)w.tiles * p.n_kv_heads;
  // a tile of k_attend_few, and one of attend_part
  const uint32_t tok = w.rows <= 32 || p.head_dim == 256 ? 5 : 6;
  const bool whole = b.max_len <= kWholeTree;
  w.shift = tok;
  const auto steps = [&]() {
    return std::max<uint64_t>(1, ((uint64_t)b.max_len + (1ull << w.shift) - 1) >> w.shift);
  };
  while (whole ? steps() > 1 : units * steps() >= (1ull << 31)) ++w.shift;
  w.min_steps = whole ? 1 : std::max(1u, (w.rows <= 32 ? 128u : 256u) >> w.shift);
  // pieces of a head's line: waves of k_attend_few, workgroups of k_attend_tree
  const uint32_t slots =
      w.rows <= 32 ? resident(p.head_dim) * 4 : resident(p.head_dim) * 128 / w.rows;
  w.pieces = (uint32_t)std::min<uint64_t>(std::min(512u, std::max(1u, slots / p.n_kv_heads)),
                                          (w.tiles * steps() + w.min_steps - 1) / w.min_steps);
  const uint32_t grid = w.pieces * p.n_kv_heads;
  w.grid = w.rows <= 32 ? (grid + 3) / 4 : grid;
  w.join = !whole && w.pieces > 1;
  if (w.join) {
    w.by_unit = units < grid;
    w.infos = w.by_unit ? units : grid;
    w.part_ml = 2ull * grid * w.rows * p.head_dim * 4;
    w.info = w.part_ml + 2ull * grid * w.rows * 2 * 4;
    w.total = w.info + sizeof(TreeHead) + w.infos * sizeof(TreeInfo);
    w.total = (w.total + 255) & ~uint64_t(255);
  }
  return w;
}

Plan make_plan(const kvc_paged_desc &p, const kvc_paged_batch &b, uint32_t max_new) {
  Plan w{};
  if (b.n_seqs == 0 || b.n_tokens == 0) return w;
  if (max_new) return make_tree_plan(p, b, max_new);
  const uint32_t group = p.n_heads / p.n_kv_heads;
  const uint32_t slots = resident(p.head_dim);
  // The 16-row kernel reads a cache once for every 16 rows.  Several tokens go
  // to the tile kernel however few they are (8 sequences of 4 tokens and 8
  // heads to a KV head, 8,000 in the cache: 67 us against 99 for 16-row tiles),
  // and so do single ones with more than 16 heads to a KV head unless caches
  // are short (64 sequences of 8,000, 64 heads to one KV head: 66 us against
  // 159; 20 heads, 300 tokens: 20 against 15).  256-row tiles (keys and values
  // fetched half as often, on average half a tile of a sequence empty) are
  // taken from 1,024 rows a sequence on.
  const uint64_t steps32 = std::max<uint64_t>(1, ((uint64_t)b.max_len + kTok - 1) / kTok);
  w.whole = !b.q_start && steps32 <= kWholeSteps;
  const uint64_t avg = b.q_start ? (uint64_t)b.n_tokens * group / b.n_seqs : 0;
  w.rows = !b.q_start ? (group <= 16 || w.whole ? 16 : 128)
           : avg < 1024 || p.head_dim == 256 ? 128 : 256;
  // every sequence's last tile may be partly filled
  w.tiles = w.rows == 16 ? b.n_seqs * ((group + 15) / 16)
                         : (uint32_t)((uint64_t)b.n_tokens * group / w.rows) +
                               std::min(b.n_seqs, b.n_tokens);
  w.wg_heads = p.n_kv_heads % 4 == 0 ? 4 : p.n_kv_heads % 2 == 0 ? 2 : 1;
  if (w.rows != 16) w.wg_heads = 1;
  const uint64_t units = (uint64_t)w.tiles * (p.n_kv_heads / w.wg_heads);
  uint64_t parts = 0;
  if (w.rows == 16) {
    uint64_t steps = steps32;
    w.shift = 5;
    while (!w.whole && units * steps >= (1ull << 31)) {
      ++w.shift;
      steps = (steps + 1) / 2;
    }
    if (w.whole) {
      w.grid = (uint32_t)units;
    } else {
      w.grid = (uint32_t)std::min<uint64_t>(
          slots, (units * steps + min_steps(w) - 1) / min_steps(w));
      w.join = true;
      w.by_unit = units < w.grid;
      w.infos = w.by_unit ? units : w.grid;
      parts = 2ull * w.grid * w.wg_heads;
    }
  } else {
    // Equal splits of every row tile, of 256 tokens at least, if the tiles do
    // not fill the chip.  (More, for the sake of uneven lengths, cost more in
    // parts and their join than they gain: with three times as many, 48
    // sequences of 400 to 12,150 tokens and two new ones each took 294 us
    // instead of 331, but 64 equal ones 246 instead of 187.)
    const uint64_t most = std::max<uint64_t>(1, ((uint64_t)b.max_len + 255) / 256);
    w.splits = (uint32_t)std::max<uint64_t>(
        1, std::min<uint64_t>(slots * 128 / w.rows / units, most));
    w.join = w.splits > 1;
    parts = w.join ? units * w.splits : 0;
  }
  w.min_steps = min_steps(w);
  w.pieces = w.grid;
  if (w.join) {
    w.part_ml = parts * w.rows * p.head_dim * 4;
    w.info = w.part_ml + parts * w.rows * 2 * 4;
    w.total = w.info + w.infos * sizeof(JoinInfo);
    w.total = (w.total + 255) & ~uint64_t(255);
  }
  return w;
}

template <class TI, class TC, int D, uint32_t kRows>
void launch_tree_join(const AttendArgs &a, const Plan &w, hipStream_t stream) {
  if (!w.join) return;
  const uint32_t rows = (uint32_t)std::min<uint64_t>((uint64_t)a.max_new * a.group, kRows);
  const uint64_t units = (uint64_t)w.tiles * a.n_kv_heads;
  // a tile's parts are shared among a row's lanes where they are many
  if ((uint64_t)w.pieces * a.n_kv_heads > 4 * units)
    hipLaunchKernelGGL((k_attend_tree_join<TI, TC, D, kRows, 8>), dim3((uint32_t)w.infos, rows),
                       dim3(D * 2), 0, stream, a);
  else
    hipLaunchKernelGGL((k_attend_tree_join<TI, TC, D, kRows, 1>),
                       dim3((uint32_t)w.infos, (rows + 7) / 8), dim3(D * 2), 0, stream, a);
}

template <class TI, class TC, int D>
hipError_t launch_d(const AttendArgs &a, const Plan &w, hipStream_t stream) {
  const uint32_t units = w.tiles * a.n_kv_heads;
  if (a.mask && w.rows <= 32) {
    const auto few = [&](auto r) {
      constexpr int R = decltype(r)::value;
      hipLaunchKernelGGL((k_attend_few<TI, TC, D, R>), dim3(w.grid), dim3(256), 0, stream, a);
      launch_tree_join<TI, TC, D, 16 * R>(a, w, stream);
    };
    if constexpr (D != 256)
      if (w.rows == 32) {
        few(std::integral_constant<int, 2>{});
        return hipGetLastError();
      }
    few(std::integral_constant<int, 1>{});
    return hipGetLastError();
  }
  if (w.rows == 16) {
    hipLaunchKernelGGL((k_attend_rows<TI, TC, D>), dim3(w.grid), dim3(256), 0, stream, a);
    if (w.join) {
      const dim3 grid((uint32_t)w.infos, std::min(kRowTile, a.group), w.wg_heads);
      if ((uint64_t)grid.x * grid.y * grid.z <= 2 * kCus)
        hipLaunchKernelGGL((k_attend_rows_join<TI, TC, D, 16>), grid, dim3(1024), 0, stream, a);
      else
        hipLaunchKernelGGL((k_attend_rows_join<TI, TC, D, 4>), grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
  }
  const auto tile = [&](auto nw) {
    constexpr int NW = decltype(nw)::value;
    if (a.mask) {
      hipLaunchKernelGGL((k_attend_tree<TI, TC, D, NW>), dim3(w.grid), dim3(NW * 64),
                         (kBigLds<D, NW>), stream, a);
      launch_tree_join<TI, TC, D, NW * 32>(a, w, stream);
      return;
    }
    const auto kernel = a.sinks ? k_attend_tile<TI, TC, D, NW, kSinks>
                                : k_attend_tile<TI, TC, D, NW, kCausal>;
    hipLaunchKernelGGL(kernel, dim3(units * w.splits), dim3(NW * 64), (kBigLds<D, NW>), stream, a);
    if (w.join)
      hipLaunchKernelGGL((k_attend_tile_join<TI, TC, D, NW * 32>), dim3(units * (NW * 8)),
                         dim3(256), 0, stream, a);
  };
  if constexpr (D != 256)
    if (w.rows == 256) {
      tile(std::integral_constant<int, 8>{});
      return hipGetLastError();
    }
  tile(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

template <class TI, class TC>
hipError_t launch_t(const kvc_paged_desc &p, const AttendArgs &a, const Plan &w,
                    hipStream_t stream) {
  switch (p.head_dim) {
    case 64: return launch_d<TI, TC, 64>(a, w, stream);
    case 96: return launch_d<TI, TC, 96>(a, w, stream);
    case 128: return launch_d<TI, TC, 128>(a, w, stream);
    default: return launch_d<TI, TC, 256>(a, w, stream);
  }
}

}  // namespace

uint64_t attend_ws_bytes(const kvc_paged_desc &p, const kvc_paged_batch &b, uint32_t max_new) {
  return make_plan(p, b, max_new).total;
}

hipError_t launch_attend(const kvc_paged_desc &p, const kvc_paged_batch &b, AttendArgs a, void *ws,
                         hipStream_t stream) {
  const Plan w = make_plan(p, b, a.max_new);
  a.splits = w.splits;
  a.whole = w.whole;
  a.seq_tiles = (a.group + kRowTile - 1) / kRowTile;
  a.step_shift = w.shift;
  a.by_unit = w.by_unit;
  a.pieces = w.pieces;
  a.min_steps = w.min_steps;
  a.infos = (uint32_t)w.infos;
  a.wg_heads = w.wg_heads;
  a.head_groups = a.n_kv_heads / w.wg_heads;
  uint8_t *base = static_cast<uint8_t *>(ws);
  a.part = reinterpret_cast<float *>(base + w.part);
  a.part_ml = reinterpret_cast<float *>(base + w.part_ml);
  a.info = w.infos ? base + w.info : nullptr;
  if (p.io_dtype == KVC_F16) return launch_t<f16, f16>(p, a, w, stream);
  if (p.cache_dtype == KVC_BF16) return launch_t<bf16, bf16>(p, a, w, stream);
  return launch_t<bf16, f16>(p, a, w, stream);
}

}  // namespace kvc

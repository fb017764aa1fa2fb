// The pages of a cache after a step: a drafted tree's accepted path moved into
// place, sequences forked, and their pages resized with copy on write.
#include <algorithm>

#include "kvc_paged.h"

namespace kvc {
namespace {

uint64_t row_bytes(const kvc_paged_desc *p) { return (uint64_t)p->n_kv_heads * p->head_dim * 2; }

// Do n entries at p and m at q share one?
bool overlap(const int32_t *p, uint64_t n, const int32_t *q, uint64_t m) {
  return p < q + m && q < p + n;
}

// -------------------------------------------------------------------- keep
// Token rows base + path[i] go to base + i, in every layer's keys and values.
// The path rises, so path[i] >= i: a thread that owns 16 bytes of the rows of
// one (layer, K/V) moves them in order, kKeepRows loads before as many stores,
// and never stores over a row that it has still to load.  Each byte moved is
// read and written once; lanes lie along the row.
//
// 47 sequences, 95 tokens moved in 80 layers of 8 x 128 (62 MB): 16.7 us, 3.7
// TB/s; with a workgroup for every 256 vectors (3,840) 21.5: each begins with a
// chain of dependent lookups (lengths, path, page ids), so it has to move more.
constexpr uint32_t kKeepRows = 8;
constexpr uint32_t kKeepBlocks = 2048;  // what the chip holds at once

struct KeepArgs {
  Seqs s;
  uint8_t *pool;
  uint64_t row, plane;  // bytes of a token's row; of a (layer, K/V)
  const int32_t *path, *kept;
  uint32_t path_stride;
  int32_t *new_lens;
  FastDiv vecs;    // 16-byte vectors of a row
  uint32_t items;  // of a token, over all layers, K and V
  int32_t *status;
};

__global__ __launch_bounds__(256) void k_keep(KeepArgs a) {
  extern __shared__ uint32_t s_from[];  // [path_stride]
  uint32_t *const s_to = s_from + a.path_stride;
  const uint32_t b = blockIdx.x;
  uint32_t row0, n;
  a.s.rows(b, row0, n);
  const int32_t len = a.s.lens[b], kept = a.kept[b], base = len - (int32_t)n;
  const bool first = blockIdx.y == 0 && threadIdx.x == 0;
  bool bad = a.s.rows_bad(b) || a.s.len_bad(b);
  const bool unused = !bad && len == 0;
  bad = bad || (!unused && (kept < 0 || kept > (int32_t)n || kept > (int32_t)a.path_stride ||
                            base < 0));
  const uint32_t m = bad || unused ? 0 : (uint32_t)kept;
  const int32_t *path = a.path + (uint64_t)b * a.path_stride;
  const int32_t *table = a.s.table + (uint64_t)b * a.s.table_stride;
  for (uint32_t i = threadIdx.x; i < m; i += 256) {
    const int32_t at = path[i];
    const bool ok = at < (int32_t)n && at > (i ? path[i - 1] : -1);
    uint32_t from = 0, to = 0;
    if (ok && (uint32_t)at != i)
      bad = !a.s.slot_of(table, (uint32_t)(base + at), from) ||
            !a.s.slot_of(table, (uint32_t)base + i, to) || bad;
    bad = bad || !ok;
    s_from[i] = from;  // both 0: stays
    s_to[i] = to;
  }
  bad = __syncthreads_or(bad);
  if (first) {
    if (bad) set_status(a.status, KVC_ERR_SHAPE);
    a.new_lens[b] = bad || unused ? len : base + (int32_t)m;
  }
  if (bad) return;
  for (uint32_t item = blockIdx.y * 256u + threadIdx.x; item < a.items; item += gridDim.y * 256u) {
    const uint32_t plane = a.vecs.div(item), c = item - plane * a.vecs.d;
    uint8_t *base_p = a.pool + (uint64_t)plane * a.plane + c * 16u;
    for (uint32_t i0 = 0; i0 < m; i0 += kKeepRows) {
      u32x4 v[kKeepRows];
#pragma unroll
      for (uint32_t j = 0; j < kKeepRows; ++j)
        if (i0 + j < m && s_from[i0 + j] != s_to[i0 + j])
          v[j] = load16(base_p + (uint64_t)s_from[i0 + j] * a.row);
#pragma unroll
      for (uint32_t j = 0; j < kKeepRows; ++j)
        if (i0 + j < m && s_from[i0 + j] != s_to[i0 + j])
          store16(base_p + (uint64_t)s_to[i0 + j] * a.row, v[j]);
    }
  }
}

// ------------------------------------------------------------ page ledgers
// A page is free where its count is 0; a row of the table counts once for
// each page that its length reaches.
struct LedgerArgs {
  int32_t *table, *lens, *refs;
  uint32_t n_rows, table_stride, n_pages, max_len;
  FastDiv page;
  int32_t *status;

  __device__ bool len_ok(int32_t len) const { return len >= 0 && len <= (int32_t)max_len; }
  __device__ uint32_t pages_of(int32_t len) const {
    return len ? page.div((uint32_t)len - 1) + 1 : 0;
  }
  __device__ int32_t *row(uint32_t r) const { return table + (uint64_t)r * table_stride; }
  // A row gives up a page.  False: an id outside the pool, or a free page.
  __device__ bool release(int32_t id) const {
    if ((uint32_t)id >= n_pages) return false;
    if (atomicSub(&refs[id], 1) > 0) return true;
    atomicAdd(&refs[id], 1);
    return false;
  }
};

// -------------------------------------------------------------------- fork
// A workgroup to a fork: what the destination holds is released, and the
// source's page ids are copied and counted.  Counts are sums, so their order
// does not show.  Forks that get in each other's way (a destination twice, or
// a source too) would depend on it: every workgroup looks through the list for
// such and leaves them out.  It is a chain of five dependent accesses: 3.1 us for
// 4 forks, 4.8 for 64.
__global__ __launch_bounds__(256) void k_fork(LedgerArgs a, const int32_t *src, const int32_t *dst,
                                              uint32_t n) {
  const uint32_t i = blockIdx.x;
  const int32_t s = src[i], d = dst[i];
  if (s < 0) return;  // left out by the caller
  bool bad = s >= (int32_t)a.n_rows || d < 0 || d >= (int32_t)a.n_rows;
  bool clash = false;
  for (uint32_t j = threadIdx.x; j < n; j += 256) {
    const int32_t sj = src[j], dj = dst[j];
    clash = clash || (sj >= 0 && (sj == d || dj == s || (j != i && dj == d)));
  }
  // Both lengths are read, and looked at, before the barrier: thread 0 stores
  // the new one when its own wave is done, while others may still be at work.
  int32_t from = 0, held = 0;
  if (!bad) {
    from = a.lens[s];
    held = a.lens[d];
    bad = !a.len_ok(from) || !a.len_ok(held);
  }
  bad = __syncthreads_or(bad || clash);
  if (bad) {
    if (threadIdx.x == 0) set_status(a.status, KVC_ERR_SHAPE);
    return;
  }
  int32_t *to = a.row((uint32_t)d);
  const int32_t *ids = a.row((uint32_t)s);
  const uint32_t gone = a.pages_of(held), taken = a.pages_of(from);
  for (uint32_t e = threadIdx.x; e < max(gone, taken); e += 256) {
    if (e < gone) bad = !a.release(to[e]) || bad;
    if (e < taken) {
      const int32_t id = ids[e];
      if ((uint32_t)id < a.n_pages)
        atomicAdd(&a.refs[id], 1);
      else
        bad = true;
      to[e] = id;
    }
  }
  if (threadIdx.x == 0) a.lens[d] = from;
  if (bad) set_status(a.status, KVC_ERR_SHAPE);
}

// ------------------------------------------------------------------ resize
// One workgroup plans: rows that shrink release pages, rows that grow out of
// a shared, partly filled page are noted, and the pages needed are found among
// the counts, lowest first, and handed out row by row.  The counts' scan reads
// 4 n_pages bytes at most (16,384 counts at a time) and ends when enough are
// found.  It is latency: 8.4 to 9.4 us for 5 rows, 11.7 to 14 for 80 (18.4 and 21.8
// with fences for other workgroups, which there are none of, and the found pages
// passed through memory).  Where the free pages lie behind 100,000 held ones the
// scan takes 28 us, behind 1,000,000 it takes 318.  A second launch copies the shared pages' tokens:
// each byte once in and once out, 64 pages of 64 tokens in 32 layers of 8 x 128
// (384 MB) in 47 us, which is more than HBM gives a copy (4.8 TB/s): the last-level
// cache holds part of it.
constexpr uint32_t kRows = 2048;  // rows of a ledger at most: two to a thread
constexpr uint32_t kScan = 16;    // counts to a thread and turn

struct Copy {
  int32_t from, to, tokens, pad;
};
struct ResizePlan {
  uint32_t copies;
  uint32_t pad[63];
  Copy copy[kRows];
};

// Inclusive sum over a workgroup of 1,024, and the total.
__device__ inline uint64_t block_sums(uint64_t x, uint64_t *s_wave, uint64_t &total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = __shfl_up(x, d);
    if (lane >= (uint32_t)d) x += o;
  }
  __syncthreads();  // s_wave is free
  if (lane == 63) s_wave[wave] = x;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (uint32_t w = 0; w < 16; ++w) {
    if (w < wave) before += s_wave[w];
    total += s_wave[w];
  }
  return before + x;
}

__global__ __launch_bounds__(1024) void k_resize(LedgerArgs a, const int32_t *new_lens,
                                                 ResizePlan *plan, int32_t *found) {
  __shared__ int32_t s_old[kRows], s_new[kRows], s_page[kRows];
  __shared__ uint32_t s_off[kRows];
  __shared__ uint64_t s_wave[16];
  __shared__ uint32_t s_free[kScan * 16];
  __shared__ int32_t s_found[kRows];  // the first pages found; more go to `found`
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  bool bad = false;
  for (uint32_t r = threadIdx.x; r < a.n_rows; r += 1024) {
    int32_t old = a.lens[r], now = new_lens[r];
    const bool ok = a.len_ok(old) && a.len_ok(now);
    bad = bad || !ok;
    if (!ok) old = now = 0;  // left as it is
    s_old[r] = ok ? old : -1;
    s_new[r] = ok ? now : -1;
    s_page[r] = -1;
  }
  __syncthreads();
  for (uint32_t r = wave; r < a.n_rows; r += 16) {
    const int32_t old = s_old[r], now = s_new[r];
    if (now >= old) continue;
    const int32_t *ids = a.row(r);
    for (uint32_t e = a.pages_of(now) + lane; e < a.pages_of(old); e += 64)
      bad = !a.release(ids[e]) || bad;
    if (lane == 0) a.lens[r] = now;
  }
  __syncthreads();  // each release has its answer by now
  // Shared pages that a row would grow into.  Row by row, each takes a copy
  // while more than one holds the page; so the last of them may keep it.
  int32_t shared[2] = {0, 0};
  uint64_t need[2] = {0, 0}, upto[2], total = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t r = threadIdx.x + k * 1024;
    if (r >= a.n_rows || s_new[r] <= s_old[r]) continue;
    const uint32_t e = a.page.div((uint32_t)s_old[r]);
    if ((uint32_t)s_old[r] == e * a.page.d) continue;  // its last page is full
    const int32_t id = a.row(r)[e];
    if ((uint32_t)id >= a.n_pages) {
      bad = true;
      continue;
    }
    shared[k] = __hip_atomic_load(&a.refs[id], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    bad = bad || shared[k] <= 0;
    if (shared[k] > 1) s_page[r] = id;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t r = threadIdx.x + k * 1024;
    bool copy = false;
    if (r < a.n_rows && s_new[r] > s_old[r]) {
      if (s_page[r] >= 0) {
        int32_t left = shared[k];
#pragma unroll 8
        for (uint32_t j = 0; j < r; ++j) left -= s_page[j] == s_page[r];
        copy = left > 1;
      }
      need[k] = a.pages_of(s_new[r]) - a.pages_of(s_old[r]) + (copy ? 1u : 0u);
      if (copy) need[k] |= 1ull << 48;
    }
    upto[k] = total;
    if (k * 1024u < a.n_rows) {
      uint64_t t;
      upto[k] += block_sums(need[k], s_wave, t);
      total += t;
    }
  }
  const uint64_t want = total & ((1ull << 48) - 1);
  uint64_t have = 0;
  for (uint64_t at = 0; at < a.n_pages && have < want && want <= a.n_pages; at += kScan * 1024) {
    uint64_t free[kScan];
#pragma unroll
    for (uint32_t k = 0; k < kScan; ++k) {
      const uint64_t id = at + k * 1024 + threadIdx.x;
      const int32_t c = id < a.n_pages ? __hip_atomic_load(&a.refs[id], __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT)
                                       : 1;
      free[k] = __ballot(c == 0);
    }
    __syncthreads();  // s_free is free
#pragma unroll
    for (uint32_t k = 0; k < kScan; ++k)
      if (lane == 0) s_free[k * 16 + wave] = (uint32_t)__popcll(free[k]);
    __syncthreads();
    uint64_t t;
    const uint64_t mine = threadIdx.x < kScan * 16 ? s_free[threadIdx.x] : 0;
    const uint64_t sum = block_sums(mine, s_wave, t);
    __syncthreads();
    if (threadIdx.x < kScan * 16) s_free[threadIdx.x] = (uint32_t)(sum - mine);
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k < kScan; ++k) {
      const uint64_t pos = have + s_free[k * 16 + wave] +
                           __popcll(free[k] & ((1ull << lane) - 1));
      if ((free[k] >> lane) & 1 && pos < want) {
        const int32_t id = (int32_t)(at + k * 1024 + threadIdx.x);
        if (pos < kRows)
          s_found[pos] = id;
        else
          found[pos] = id;
      }
    }
    have += t;
  }
  const bool enough = have >= want;
  if (bad) set_status(a.status, KVC_ERR_SHAPE);
  if (threadIdx.x == 0) {
    if (!enough) set_status(a.status, KVC_ERR_CAPACITY);
    plan->copies = enough ? (uint32_t)(total >> 48) : 0;
  }
  if (!enough) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t r = threadIdx.x + k * 1024;
    if (r >= a.n_rows) continue;
    const uint64_t before = upto[k] - need[k];
    uint32_t off = (uint32_t)before;  // below 2^31: at most n_pages
    if (need[k] >> 48) {
      const uint32_t e = a.page.div((uint32_t)s_old[r]);
      const int32_t tokens = s_old[r] - (int32_t)(e * a.page.d);
      plan->copy[before >> 48] = Copy{s_page[r], (int32_t)off, tokens, 0};
      s_page[r] = (int32_t)(before >> 48);
    } else {
      s_page[r] = -1;
    }
    s_off[r] = off;
  }
  __syncthreads();
  const auto page_at = [&](uint32_t i) { return i < kRows ? s_found[i] : found[i]; };
  for (uint32_t r = wave; r < a.n_rows; r += 16) {
    const int32_t old = s_old[r], now = s_new[r];
    if (now <= old) continue;
    int32_t *ids = a.row(r);
    uint32_t off = s_off[r];
    if (s_page[r] >= 0) {
      if (lane == 0) {
        Copy &c = plan->copy[s_page[r]];
        const int32_t id = page_at(off);
        c.to = id;
        ids[a.page.div((uint32_t)old)] = id;
        a.refs[id] = 1;
        atomicSub(&a.refs[c.from], 1);
      }
      ++off;
    }
    const uint32_t e0 = a.pages_of(old), e1 = a.pages_of(now);
    for (uint32_t e = e0 + lane; e < e1; e += 64) {
      const int32_t id = page_at(off + (e - e0));
      ids[e] = id;
      a.refs[id] = 1;
    }
    if (lane == 0) a.lens[r] = now;
  }
}

struct CopyArgs {
  uint8_t *pool;
  uint64_t row, plane, page;  // bytes: of a token's row, a (layer, K/V), a page's rows
  FastDiv planes;
  const ResizePlan *plan;
};

__global__ __launch_bounds__(256) void k_copy_pages(CopyArgs a) {
  const uint32_t units = a.plan->copies * a.planes.d;
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const uint32_t at = a.planes.div(u), plane = u - at * a.planes.d;
    const Copy c = a.plan->copy[at];
    uint8_t *base = a.pool + (uint64_t)plane * a.plane;
    const uint8_t *from = base + (uint64_t)c.from * a.page;
    uint8_t *to = base + (uint64_t)c.to * a.page;
    const uint64_t bytes = (uint64_t)c.tokens * a.row;
    const uint64_t step = (uint64_t)gridDim.y * 256 * 16 * 4;
    for (uint64_t x0 = (uint64_t)blockIdx.y * 256 * 16 * 4 + threadIdx.x * 16u; x0 < bytes;
         x0 += step) {
      u32x4 v[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (x0 + j * 4096 < bytes) v[j] = load16(from + x0 + j * 4096);
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j)
        if (x0 + j * 4096 < bytes) store16(to + x0 + j * 4096, v[j]);
    }
  }
}

kvc_status ledger_check(const kvc_paged_desc *p, const kvc_ledger *g) {
  if (!paged_ok(p) || !g || g->n_rows > kRows) return !paged_ok(p) || !g ? KVC_ERR_INVALID_ARG
                                                                          : KVC_ERR_SHAPE;
  if (g->n_rows == 0) return KVC_OK;
  if (!g->lens || !aligned(g->lens, 4) || !g->refs || !aligned(g->refs, 4))
    return KVC_ERR_INVALID_ARG;
  if (g->table_stride && (!g->table || !aligned(g->table, 4))) return KVC_ERR_INVALID_ARG;
  return KVC_OK;
}

// n entries at p, which a call reads, over what it writes
bool over_ledger(const kvc_paged_desc *p, const kvc_ledger *g, const int32_t *in, uint64_t n) {
  return overlap(in, n, g->table, (uint64_t)g->n_rows * g->table_stride) ||
         overlap(in, n, g->lens, g->n_rows) || overlap(in, n, g->refs, p->n_pages);
}

LedgerArgs to_ledger(const kvc_paged_desc *p, const kvc_ledger *g, int32_t *status) {
  LedgerArgs a;
  a.table = g->table;
  a.lens = g->lens;
  a.refs = g->refs;
  a.n_rows = g->n_rows;
  a.table_stride = g->table_stride;
  a.n_pages = p->n_pages;
  a.max_len = (uint32_t)std::min<uint64_t>((uint64_t)g->table_stride * p->page_tokens, 1u << 30);
  a.page = FastDiv::make(p->page_tokens);
  a.status = status;
  return a;
}

uint64_t found_at() { return sizeof(ResizePlan); }

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" {

kvc_status kvc_keep(const kvc_paged_desc *p, const kvc_paged_batch *b, void *pool,
                    const int32_t *path, uint32_t path_stride, const int32_t *kept,
                    int32_t *new_lens, int32_t *dev_status, hipStream_t stream) {
  kvc_status st = batch_check(p, b, 0, pool, dev_status);
  if (st != KVC_OK) return st;
  if (!b->q_start) return KVC_ERR_INVALID_ARG;
  if (path_stride > kTreeTokens) return KVC_ERR_SHAPE;
  const uint64_t items = 2ull * p->n_layers * (row_bytes(p) / 16);
  if (items >= (1ull << 31)) return KVC_ERR_SHAPE;
  if (b->n_seqs == 0) return KVC_OK;
  if (!kept || !aligned(kept, 4) || !new_lens || !aligned(new_lens, 4)) return KVC_ERR_INVALID_ARG;
  if (path_stride && (!path || !aligned(path, 4))) return KVC_ERR_INVALID_ARG;
  // workgroups read these while others write new_lens
  const auto over = [&](const int32_t *p, uint64_t n) {
    return overlap(new_lens, b->n_seqs, p, n);
  };
  if (over(b->lens, b->n_seqs) || over(kept, b->n_seqs) ||
      over(path, (uint64_t)b->n_seqs * path_stride) || over(b->q_start, b->n_seqs + 1ull) ||
      over(b->table, (uint64_t)b->n_seqs * b->table_stride))
    return KVC_ERR_SHAPE;
  KeepArgs a;
  a.s = to_seqs(p, b);
  a.pool = static_cast<uint8_t *>(pool);
  a.row = row_bytes(p);
  a.plane = plane_bytes(p);
  a.path = path;
  a.kept = kept;
  a.path_stride = path_stride;
  a.new_lens = new_lens;
  a.vecs = FastDiv::make((uint32_t)(a.row / 16));
  a.items = (uint32_t)items;
  a.status = dev_status;
  // workgroups over a sequence's items: all of them, unless sequences are many
  const uint32_t y = (uint32_t)std::min<uint64_t>((items + 255) / 256,
                                                  std::max(1u, kKeepBlocks / b->n_seqs));
  hipLaunchKernelGGL(k_keep, dim3(b->n_seqs, y), dim3(256), path_stride * 8, stream, a);
  return hipGetLastError() == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

kvc_status kvc_fork(const kvc_paged_desc *p, const kvc_ledger *g, const int32_t *src,
                    const int32_t *dst, uint32_t n, int32_t *dev_status, hipStream_t stream) {
  const kvc_status st = ledger_check(p, g);
  if (st != KVC_OK) return st;
  if (!dev_status || !aligned(dev_status, 4)) return KVC_ERR_INVALID_ARG;
  if (n > kRows) return KVC_ERR_SHAPE;
  if (n == 0) return KVC_OK;
  if (!src || !aligned(src, 4) || !dst || !aligned(dst, 4)) return KVC_ERR_INVALID_ARG;
  // workgroups read the lists while others write the ledger
  if (g->n_rows && (over_ledger(p, g, src, n) || over_ledger(p, g, dst, n))) return KVC_ERR_SHAPE;
  hipLaunchKernelGGL(k_fork, dim3(n), dim3(256), 0, stream, to_ledger(p, g, dev_status), src, dst,
                     n);
  return hipGetLastError() == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

uint64_t kvc_resize_ws_bytes(const kvc_paged_desc *p) {
  return paged_ok(p) ? (found_at() + 4ull * p->n_pages + 255) & ~255ull : 0;
}

kvc_status kvc_resize(const kvc_paged_desc *p, const kvc_ledger *g, const int32_t *new_lens,
                      void *pool, void *ws, uint64_t ws_bytes, int32_t *dev_status,
                      hipStream_t stream) {
  const kvc_status st = ledger_check(p, g);
  if (st != KVC_OK) return st;
  if (!dev_status || !aligned(dev_status, 4) || !pool || !aligned(pool, 16))
    return KVC_ERR_INVALID_ARG;
  if (g->n_rows == 0) return KVC_OK;
  if (!new_lens || !aligned(new_lens, 4) || !ws || !aligned(ws, 256)) return KVC_ERR_INVALID_ARG;
  if (ws_bytes < kvc_resize_ws_bytes(p)) return KVC_ERR_CAPACITY;
  // (lengths put into the ledger itself would not be seen to change)
  if (over_ledger(p, g, new_lens, g->n_rows)) return KVC_ERR_SHAPE;
  ResizePlan *plan = static_cast<ResizePlan *>(ws);
  int32_t *found = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + found_at());
  hipLaunchKernelGGL(k_resize, dim3(1), dim3(1024), 0, stream, to_ledger(p, g, dev_status),
                     new_lens, plan, found);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p->page_tokens > 1) {  // a page of one token is never partly filled
    CopyArgs a;
    a.pool = static_cast<uint8_t *>(pool);
    a.row = row_bytes(p);
    a.plane = plane_bytes(p);
    a.page = a.row * p->page_tokens;
    a.planes = FastDiv::make(2 * p->n_layers);
    a.plan = plan;
    const uint64_t units = (uint64_t)g->n_rows * 2 * p->n_layers;
    const uint32_t y = (uint32_t)std::min<uint64_t>((a.page + (1 << 16) - 1) >> 16, 64);
    const uint32_t x = (uint32_t)std::min<uint64_t>(units, std::max(256u, 8192 / y));
    hipLaunchKernelGGL(k_copy_pages, dim3(x, y), dim3(256), 0, stream, a);
    e = hipGetLastError();
  }
  return e == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

}  // extern "C"

// A tree of drafted tokens: which of them each one sees, and its depth.
#include "kvc_paged.h"

namespace kvc {

bool tree_ok(const kvc_tree *t) {
  return t && t->reserved == 0 && t->max_tokens >= 1 && t->max_tokens <= kTreeTokens;
}

namespace {

// A workgroup to a sequence: the parents go to LDS, and a thread walks from
// its token to the root, setting a bit for each token it meets.  Parents come
// before their children, so the walk meets falling numbers: it ends, and each
// word of the mask is complete when the walk leaves it.  A step of the walk is
// an LDS read (some 64 cycles), so the launch is what it costs: 4.6 us for 15
// trees of 17 to 60 tokens, once for all layers.
__global__ __launch_bounds__(256) void k_tree(Seqs s, const int32_t *parent, uint64_t *mask,
                                              int32_t *depth, uint32_t max_new, int32_t *status) {
  __shared__ int32_t up[kTreeTokens];
  const uint32_t b = blockIdx.x, words = (max_new + 63) / 64;
  uint32_t row, n;
  s.rows(b, row, n);
  bool bad = s.rows_bad(b) || n > max_new;
  if (!bad) {
    for (uint32_t i = threadIdx.x; i < n; i += 256) {
      const int32_t p = parent[row + i];
      const bool ok = p >= -1 && p < (int32_t)i;
      bad = bad || !ok;
      up[i] = ok ? p : -1;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n; i += 256) {
      uint64_t *m = mask + (uint64_t)(row + i) * words, bits = 0;
      uint32_t w = words - 1;  // the word that `bits` holds
      int32_t steps = 0;
      for (int32_t at = (int32_t)i; at >= 0; at = up[at], ++steps) {
        for (; w > (uint32_t)at >> 6; --w) {
          m[w] = bits;
          bits = 0;
        }
        bits |= 1ull << (at & 63);
      }
      for (;; --w) {
        m[w] = bits;
        bits = 0;
        if (w == 0) break;
      }
      depth[row + i] = steps - 1;
    }
  }
  if (bad) set_status(status, KVC_ERR_SHAPE);
}

}  // namespace
}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_tree_build(const kvc_paged_desc *p, const kvc_paged_batch *b,
                                     const kvc_tree *tree, int32_t *dev_status,
                                     hipStream_t stream) {
  const kvc_status st = batch_sizes(p, b);
  if (st != KVC_OK) return st;
  if (!tree_ok(tree) || !dev_status || !aligned(dev_status, 4)) return KVC_ERR_INVALID_ARG;
  if (!b->q_start || !aligned(b->q_start, 4)) return KVC_ERR_INVALID_ARG;
  if (b->n_seqs == 0 || b->n_tokens == 0) return KVC_OK;
  if (!tree->parent || !aligned(tree->parent, 4) || !tree->mask || !aligned(tree->mask, 8) ||
      !tree->depth || !aligned(tree->depth, 4))
    return KVC_ERR_INVALID_ARG;
  hipLaunchKernelGGL(k_tree, dim3(b->n_seqs), dim3(256), 0, stream, to_seqs(p, b), tree->parent,
                     tree->mask, tree->depth, tree->max_tokens, dev_status);
  return hipGetLastError() == hipSuccess ? KVC_OK : KVC_ERR_HIP;
}

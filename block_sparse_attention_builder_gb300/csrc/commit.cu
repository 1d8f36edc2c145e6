// The accepted path of each drafted tree moved to the positions that it takes
// in its sequence (mxsa_tree_commit): the rows of tokens path[0] < path[1] <
// ... of the tree go to places 0, 1, ... behind the committed keys, K, V and
// index keys, any cache type, bytes as they are.
//
// One CTA for each sequence and head.  A row may be the source of one move and
// the destination of another, so a CTA first loads what it moves into
// registers, up to kMovePieces pieces of 8 bytes a thread, and stores after a
// barrier.  A longer path goes in passes: path[j] >= j, and a pass writes
// places before its own end only, so no later pass reads a row that an earlier
// one has written.  Bound: latency (lengths, path, tables, rows: four rounds to
// memory and a launch); the rows of 128 paths of eight heads are 2 MB.
#include "internal.h"

namespace mxsa {

namespace {

constexpr int kMoveThreads = 256, kMovePieces = 4;

struct CommitArgs {
  const int64_t* cu;
  const int32_t *lens, *block_tables, *path, *path_lens;
  uint8_t* cache[3];      // K, V, index keys (may be null)
  int32_t* lens_out;      // may be null
  int32_t* flags;         // may be null
  int32_t total_q, Hkv, idx_heads, page_shift, max_pages, num_pages, max_path;
  int32_t row[2];         // bytes of a row: K / V, index keys
  int32_t fp4;            // K and V rows are 64 bytes of codes, and 8 of scales behind the page's codes
};

__global__ void __launch_bounds__(kMoveThreads) k_commit(CommitArgs a) {
  const int tid = threadIdx.x, heads = a.Hkv + a.idx_heads;
  const int s = blockIdx.x / heads, hx = blockIdx.x - s * heads;
  const bool idx = hx >= a.Hkv;
  pdl_launch_dependents();
  pdl_wait();
  const long long c0 = a.cu[s], c1 = a.cu[s + 1];
  const int len = a.lens[s], n = a.path_lens[s], max_len = a.max_pages << a.page_shift;
  const int32_t* path = a.path + (size_t)s * a.max_path;
  int bad = c0 < 0 || c1 < c0 || c1 > a.total_q ? MXSA_FLAG_CU : 0;
  const int tq = bad ? 0 : (int)(c1 - c0);
  if (len < 0 || len > max_len) bad |= MXSA_FLAG_LEN;
  const int L = min(max(len, 0), max_len), base = L - tq;
  if (base < 0) bad |= MXSA_FLAG_CAUSAL_LEN;
  if (!(bad & MXSA_FLAG_CU) && (n < 0 || n > a.max_path || n > tq)) bad |= MXSA_FLAG_TREE;
  if (!bad) {
    int wrong = 0;
    for (int k = tid; k < n; k += kMoveThreads) wrong |= path[k] <= (k ? path[k - 1] : -1) || path[k] >= tq;
    if (__syncthreads_or(wrong)) bad = MXSA_FLAG_TREE;
  }
  if (hx == 0 && tid == 0) {
    if (a.lens_out) a.lens_out[s] = max(base, 0) + (bad ? 0 : n);
    if (bad && a.flags) atomicOr(a.flags, bad);
  }
  if (bad) return;  // (the same in every thread)

  const int row_bytes = idx ? a.row[1] : a.row[0];
  const int per_row = row_bytes / 8, caches = idx ? 1 : 2;          // pieces of a row, rows of a token
  const int rows = max(kMoveThreads * kMovePieces / (per_row * caches), 1);  // tokens of a pass
  const int hn = idx ? a.idx_heads : a.Hkv, h = idx ? hx - a.Hkv : hx;
  // byte offset of piece x of the row at position p; -1: no page there
  auto at = [&](int p, int x) -> long long {
    const int page = a.block_tables[(size_t)s * a.max_pages + (p >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) return -1;
    const long long slab = ((long long)page * hn + h) << a.page_shift;
    const int off = p & ((1 << a.page_shift) - 1);
    if (a.fp4 && !idx) return x < 8 ? slab * 72 + off * 64 + 8 * x : slab * 72 + (64LL << a.page_shift) + off * 8;
    return (slab + off) * row_bytes + 8 * x;
  };
  for (int k0 = 0; k0 < n; k0 += rows) {
    const int pieces = min(rows, n - k0) * caches * per_row;
    for (int x0 = 0; x0 < pieces; x0 += kMoveThreads * kMovePieces) {  // (more than one round: rows == 1 only)
      uint2 v[kMovePieces];
      long long to[kMovePieces];
#pragma unroll
      for (int i = 0; i < kMovePieces; ++i) {
        const int x = x0 + i * kMoveThreads + tid;
        to[i] = -1;
        if (x >= pieces) continue;
        const int r = x / per_row, k = k0 + r / caches, c = idx ? 2 : r % caches;
        const int from = path[k];
        if (from == k) continue;
        const long long src = at(base + from, x - r * per_row);
        to[i] = at(base + k, x - r * per_row);
        if (src < 0 || to[i] < 0) {
          if (a.flags) atomicOr(a.flags, MXSA_FLAG_PAGE);
          to[i] = -1;
          continue;
        }
        v[i] = *reinterpret_cast<const uint2*>(a.cache[c] + src);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMovePieces; ++i)
        if (to[i] >= 0) {
          const int r = (x0 + i * kMoveThreads + tid) / per_row;
          *reinterpret_cast<uint2*>(a.cache[idx ? 2 : r % caches] + to[i]) = v[i];
        }
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(const mxsa_problem& p, const int64_t* cu, const int32_t* lens,
                               const int32_t* block_tables, const int32_t* path, int max_path,
                               const int32_t* path_lens, void* k_cache, void* v_cache, void* idx_cache,
                               int idx_heads, int idx_dim, int32_t* lens_out, int32_t* flags, cudaStream_t st) {
  CommitArgs a{};
  a.cu = cu;
  a.lens = lens;
  a.block_tables = block_tables;
  a.path = path;
  a.path_lens = path_lens;
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.cache[2] = static_cast<uint8_t*>(idx_cache);
  a.lens_out = lens_out;
  a.flags = flags;
  a.total_q = p.total_q;
  a.Hkv = p.num_kv_heads;
  a.idx_heads = idx_cache ? idx_heads : 0;
  a.page_shift = p.page_size == 128 ? 7 : 6;
  a.max_pages = p.max_pages_per_seq;
  a.num_pages = p.num_pages;
  a.max_path = max_path;
  const int kind = cache_kind(p), elem = kind == kKind16 ? 2 : 1;
  a.fp4 = kind == kKindFp4;
  a.row[0] = a.fp4 ? 72 : 128 * elem;
  a.row[1] = idx_cache ? idx_dim * elem : 8;
  return launch_pdl(k_commit, dim3((unsigned)(p.num_seqs * (a.Hkv + a.idx_heads))), dim3(kMoveThreads), 0, st, a);
}

}  // namespace mxsa

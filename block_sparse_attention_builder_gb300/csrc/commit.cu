// The accepted path of each drafted tree moved to the positions that it takes
// in its sequence (mxsa_tree_commit): the rows of tokens path[0] < path[1] <
// ... of the tree go to places 0, 1, ... behind the committed keys, K, V and
// index keys, any cache type, bytes as they are.
//
// One CTA for each sequence and head.  A row may be the source of one move and
// the destination of another, so a CTA first loads what it moves into
// registers, kMoveDepth pieces a thread, and stores after a barrier.  A longer
// path goes in passes: path[j] >= j, and a pass writes places before its own end
// only, so no later pass reads a row that an earlier one has written.
//
// Bound: latency (lengths, path, tables, rows: four rounds to memory and a
// launch): 1.3 us for one path of two heads, 4.1 us for 128 of eight (FP8, 2 MB).
#include "internal.h"

namespace mxsa {

namespace {

constexpr int kMoveThreads = 256, kMoveDepth = 4;

struct CommitArgs {
  const int64_t* cu;
  const int32_t *lens, *block_tables, *path, *path_lens;
  uint8_t *k_cache, *v_cache, *idx_cache;  // (index keys may be null)
  int32_t* lens_out;                       // may be null
  int32_t* flags;                          // may be null
  int32_t total_q, Hkv, idx_heads, idx_row, page_shift, max_pages, num_pages, max_path;  // idx_row: bytes
};

// Moves the rows of one sequence and head.  A pass takes kMoveDepth rounds of
// kMoveThreads pieces; piece x belongs to path entry x / (1 << kShift) where the
// pieces of an entry are a power of two (kShift >= 0), else x / per.  at(slot,
// part): a piece's address; null where it is padding.
template <typename Piece, int kShift, typename At>
__device__ __forceinline__ void move_rows(const CommitArgs& a, const int32_t* path, const int32_t* table, int n,
                                          int base, int per, At at) {
  const int tid = threadIdx.x;
  auto slot = [&](int p) -> long long {  // -1: no page there
    const int page = table[p >> a.page_shift];
    return page < 0 || page >= a.num_pages ? -1
                                           : ((long long)page << a.page_shift) | (p & ((1 << a.page_shift) - 1));
  };
  for (long long x0 = 0; x0 < (long long)n * per; x0 += kMoveThreads * kMoveDepth) {
    Piece v[kMoveDepth];
    Piece* to[kMoveDepth];
#pragma unroll
    for (int i = 0; i < kMoveDepth; ++i) {
      const long long x = x0 + i * kMoveThreads + tid;
      const int k = kShift >= 0 ? (int)(x >> (kShift >= 0 ? kShift : 0)) : (int)(x / per), part = (int)(x - (long long)k * per);
      to[i] = nullptr;
      if (k >= n) continue;
      const int from = path[k];
      if (from == k) continue;
      const long long src = slot(base + from), dst = slot(base + k);
      if (src < 0 || dst < 0) {
        if (a.flags) atomicOr(a.flags, MXSA_FLAG_PAGE);
        continue;
      }
      const Piece* p = at(src, part);
      if (!p) continue;
      v[i] = *p;
      to[i] = at(dst, part);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoveDepth; ++i)
      if (to[i]) *to[i] = v[i];
  }
}

template <int kKind>
__global__ void __launch_bounds__(kMoveThreads) k_commit(CommitArgs a) {
  const int tid = threadIdx.x, heads = a.Hkv + a.idx_heads;
  const int s = blockIdx.x / heads, hx = blockIdx.x - s * heads;
  pdl_launch_dependents();
  pdl_wait();
  const long long c0 = a.cu[s], c1 = a.cu[s + 1];
  const int len = a.lens[s], n = a.path_lens[s], max_len = a.max_pages << a.page_shift;
  const int32_t* path = a.path + (size_t)s * a.max_path;
  const int32_t* table = a.block_tables + (size_t)s * a.max_pages;
  // (the path's first entries are on their way before its length is known)
  const int mine = tid < a.max_path ? path[tid] : 0, before = tid > 0 && tid < a.max_path ? path[tid - 1] : -1;
  int bad = c0 < 0 || c1 < c0 || c1 > a.total_q ? MXSA_FLAG_CU : 0;
  const int tq = bad ? 0 : (int)(c1 - c0);
  if (len < 0 || len > max_len) bad |= MXSA_FLAG_LEN;
  const int L = min(max(len, 0), max_len), base = L - tq;
  if (base < 0) bad |= MXSA_FLAG_CAUSAL_LEN;
  if (!(bad & MXSA_FLAG_CU) && (n < 0 || n > a.max_path || n > tq)) bad |= MXSA_FLAG_TREE;
  if (!bad) {
    int wrong = tid < n && (mine <= before || mine >= tq);
    for (int k = tid + kMoveThreads; k < n; k += kMoveThreads) wrong |= path[k] <= path[k - 1] || path[k] >= tq;
    if (__syncthreads_or(wrong)) bad = MXSA_FLAG_TREE;
  }
  if (hx == 0 && tid == 0) {
    if (a.lens_out) a.lens_out[s] = max(base, 0) + (bad ? 0 : n);
    if (bad && a.flags) atomicOr(a.flags, bad);
  }
  if (bad) return;  // (the same in every thread)
  const long long ps = 1LL << a.page_shift, in_page = ps - 1;
  if (hx >= a.Hkv) {  // index keys, pieces of 8 bytes
    const int h = hx - a.Hkv;
    move_rows<uint2, -1>(a, path, table, n, base, a.idx_row / 8, [&](long long slot, int part) {
      const long long row = (((slot >> a.page_shift) * a.idx_heads + h) << a.page_shift) | (slot & in_page);
      return reinterpret_cast<uint2*>(a.idx_cache + row * a.idx_row) + part;
    });
    return;
  }
  // K and V, pieces of 16 bytes: 16 (or 8) of a K row, then as many of the V row.
  constexpr int kShift = kKind == kKind16 ? 5 : 4, kPieces = 1 << (kShift - 1);
  if (kKind != kKindFp4) {
    move_rows<uint4, kShift>(a, path, table, n, base, 2 * kPieces, [&](long long slot, int part) {
      const long long row = (((slot >> a.page_shift) * a.Hkv + hx) << a.page_shift) | (slot & in_page);
      uint8_t* cache = part < kPieces ? a.k_cache : a.v_cache;
      return reinterpret_cast<uint4*>(cache + row * (16 * kPieces)) + (part & (kPieces - 1));
    });
  } else {
    // (pieces of 8: eight of the codes and one of the scales, K and V, 32 with padding)
    move_rows<uint2, 5>(a, path, table, n, base, 32, [&](long long slot, int part) -> uint2* {
      uint8_t* slab = (part < 16 ? a.k_cache : a.v_cache) + (((slot >> a.page_shift) * a.Hkv + hx) << a.page_shift) * 72;
      const int x = part & 15;
      if (x > 8) return nullptr;
      return reinterpret_cast<uint2*>(x < 8 ? slab + (slot & in_page) * 64 + 8 * x
                                            : slab + 64 * ps + (slot & in_page) * 8);
    });
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
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.idx_cache = static_cast<uint8_t*>(idx_cache);
  a.lens_out = lens_out;
  a.flags = flags;
  a.total_q = p.total_q;
  a.Hkv = p.num_kv_heads;
  a.idx_heads = idx_cache ? idx_heads : 0;
  a.page_shift = p.page_size == 128 ? 7 : 6;
  a.max_pages = p.max_pages_per_seq;
  a.num_pages = p.num_pages;
  a.max_path = max_path;
  const int kind = cache_kind(p);
  a.idx_row = idx_cache ? idx_dim * (kind == kKind16 ? 2 : 1) : 8;
  auto* kern = kind == kKind16 ? k_commit<kKind16> : (kind == kKindFp8 ? k_commit<kKindFp8> : k_commit<kKindFp4>);
  return launch_pdl(kern, dim3((unsigned)(p.num_seqs * (a.Hkv + a.idx_heads))), dim3(kMoveThreads), 0, st, a);
}

}  // namespace mxsa

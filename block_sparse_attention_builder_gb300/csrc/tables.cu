// A serving step's bookkeeping on the GPU (mxsa_build_tables): from the
// requests' cached and new tokens the block tables (pages popped from a free
// list, those of finished requests pushed back), cu_seqlens_q, lengths,
// positions and cache slots; and the ancestor masks of drafted trees
// (mxsa_tree_mask).
//
// Tables.  One CTA with a thread for each request makes the plan: three sums
// over the requests (new tokens, pages wanted, pages given back) give every
// request its place in the token axis and in the free list, and the moves of
// pages are then spread over the threads by number, not by request, so that a
// long prompt beside decoding ones costs no more than its share.  The tokens'
// positions and slots (16 bytes a token) follow in the same CTA when there are
// few and in a second launch of many CTAs when there are more: see
// kTablesOneCta.  Bound: latency (three rounds to memory and a launch): 3.6 us
// for 64 decoding requests, 9.4 us for 250000 tokens of 250 (4 MB).
// Mask.  A thread for each token walks from it to its root.  Parents come
// before their children, so that the words of a row are finished one by one
// from the last to the first and written once.  Bound: latency (a round to L1
// for each ancestor, 0.18 us): 2.0 us for 8 trees of 16 tokens and depth five,
// 4.6 us for 256 of 125 and ten; chains of 125 tokens 24 us, of 2048 375 us.  A
// walk ends after as many ancestors as a row can have bits: a sequence that is
// too long for its masks, and flagged, costs no more (a chain of 100000 tokens
// 452 us; 9478 us to its root).
#include <algorithm>
#include <climits>

#include "internal.h"

namespace mxsa {

namespace {

constexpr int kTMaxSeqs = 1024;
constexpr int kPlanThreads = 1024, kFillThreads = 256;
// Returned pages that a thread of the plan keeps between check and move: the
// check costs a step with finished requests 0.4 us so (64 requests, 8 finished:
// 4.7 to 5.1), 3.3 where 12800 pages go back (14.1 to 17.5; 23.9 with every page
// looked up twice).
constexpr int kBackKept = 8;
// Up to so many tokens the plan's CTA writes them itself: 512 tokens 4.1 us
// against 5.0 in two launches, 2048 4.3 and 4.8, 4096 5.2 and 4.8, 16384 12.5
// and 5.3.
constexpr int kTablesOneCta = 2048;

struct TablesArgs {
  const int32_t *kv_lens, *new_lens, *pages_held;
  int32_t *block_tables, *free_pages;
  const int32_t* free_count;
  int64_t* cu;
  int32_t* used;
  int64_t *positions, *loc;
  int32_t *held_out, *free_count_out;
  int32_t* flags;  // may be null
  int32_t num_seqs, total_q, page_shift, num_pages, max_pages;
  int32_t fill;    // the plan's CTA writes the tokens too
};

// the last index i of a[0 .. n) (non-decreasing, a[0] <= x) with a[i] <= x
__device__ __forceinline__ int find_le(const int32_t* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Position and slot of tokens t and t + 1 (t even); start: cu_seqlens_q, in
// shared memory.  The arrays' last token may be the first of a pair alone.
__device__ __forceinline__ void fill_tokens(const TablesArgs& a, const int32_t* start, const int32_t* base, int t) {
  longlong2 pos = make_longlong2(-1, -1), loc = make_longlong2(-1, -1);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int x = t + k;
    if (x >= start[a.num_seqs]) continue;
    const int s = find_le(start, a.num_seqs, x);
    const int p = base[s] + x - start[s];
    const int page = a.block_tables[(size_t)s * a.max_pages + (p >> a.page_shift)];
    long long slot = -1;
    if (page >= 0 && page < a.num_pages)
      slot = ((long long)page << a.page_shift) | (p & ((1 << a.page_shift) - 1));
    else if (a.flags)
      atomicOr(a.flags, MXSA_FLAG_PAGE);
    (k ? pos.y : pos.x) = p;
    (k ? loc.y : loc.x) = slot;
  }
  if (t + 1 < a.total_q) {
    *reinterpret_cast<longlong2*>(a.positions + t) = pos;
    *reinterpret_cast<longlong2*>(a.loc + t) = loc;
  } else {
    a.positions[t] = pos.x;
    a.loc[t] = loc.x;
  }
}

__global__ void __launch_bounds__(kPlanThreads) k_tables_plan(TablesArgs a) {
  __shared__ int32_t start[kTMaxSeqs + 1], want0[kTMaxSeqs + 1], back0[kTMaxSeqs + 1], held[kTMaxSeqs],
      base[kTMaxSeqs];
  __shared__ long long part[3][kPlanThreads / 32];
  const int s = threadIdx.x, lane = s & 31, w = s >> 5, B = a.num_seqs;
  pdl_launch_dependents();
  pdl_wait();
  const int count = *a.free_count;
  int o = 0, n = 0, h = 0, bad = 0;
  if (s < B) {
    o = a.kv_lens[s];
    n = a.new_lens[s];
    h = a.pages_held[s];
  }
  const int o_in = o, h_in = h;
  const bool done = n < 0;
  long long v[3] = {0, 0, 0};  // new tokens, pages wanted, pages given back
  if (s < B) {
    const long long cap = (long long)a.max_pages << a.page_shift;
    if (h < 0 || h > a.max_pages || (!done && (o < 0 || (long long)o > ((long long)h << a.page_shift) ||
                                               (long long)o + n > cap))) {
      bad = MXSA_FLAG_LEN;
    } else if (done) {
      v[2] = h;
    } else {
      const int pages = (int)(((long long)o + n + (1 << a.page_shift) - 1) >> a.page_shift);
      v[0] = n;
      v[1] = max(pages - h, 0);
    }
  }
  long long x[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) x[i] = v[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long y = __shfl_up_sync(0xffffffffu, x[i], d);
      if (lane >= d) x[i] += y;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) part[i][w] = x[i];
  const bool len_bad = __syncthreads_or(bad);  // (also: the warps' sums are there)
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long y = part[i][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y += z;
    }
    const long long before = __shfl_sync(0xffffffffu, y, max(w - 1, 0));
    total[i] = __shfl_sync(0xffffffffu, y, 31);
    x[i] += w ? before : 0;  // inclusive
  }
  if (len_bad) bad = MXSA_FLAG_LEN;
  if (total[0] > a.total_q) bad |= MXSA_FLAG_CU;
  const bool list_ok = count >= 0 && count + total[2] <= a.num_pages;
  if (!len_bad && (!list_ok || total[1] > count + total[2])) bad |= MXSA_FLAG_PAGES;
  const int gives = bad ? 0 : (int)total[2];
  // page k of those that finished requests give back; the first ones of a thread stay in registers
  auto returned = [&](int k) {
    const int r = find_le(back0, B, k);
    return a.block_tables[(size_t)r * a.max_pages + k - back0[r]];
  };
  int kept[kBackKept];
  if (gives > 0) {  // (uniform) what goes back has to be pages: looked at before anything is written
    if (s < B) back0[s] = (int)(x[2] - v[2]);
    __syncthreads();
    int wrong = 0;
    auto look = [&](int page) { wrong |= page < 0 || page >= a.num_pages; };
#pragma unroll
    for (int i = 0; i < kBackKept; ++i) kept[i] = s + i * kPlanThreads < gives ? returned(s + i * kPlanThreads) : 0;
#pragma unroll
    for (int i = 0; i < kBackKept; ++i) look(kept[i]);
#pragma unroll 4
    for (int k = s + kBackKept * kPlanThreads; k < gives; k += kPlanThreads) look(returned(k));
    if (__syncthreads_or(wrong)) bad = MXSA_FLAG_PAGES;
  }
  if (bad) {  // (the same in every thread) nothing is given out or taken back
    if (s < B) {
      a.used[s] = o_in;
      a.held_out[s] = h_in;
      a.cu[s] = 0;
      start[s] = 0;
    }
    if (s == 0) {
      a.cu[B] = 0;
      start[B] = 0;
      *a.free_count_out = count;
      if (a.flags) atomicOr(a.flags, bad);
    }
  } else {
    const int top = count + gives, wants = (int)total[1];
    if (s < B) {
      start[s] = (int)(x[0] - v[0]);
      want0[s] = (int)(x[1] - v[1]);
      held[s] = h;
      base[s] = o;
      a.cu[s] = x[0] - v[0];
      a.used[s] = done ? 0 : o + n;
      a.held_out[s] = done ? 0 : h + (int)v[1];
    }
    if (s == 0) {
      start[B] = (int)total[0];
      a.cu[B] = total[0];
      *a.free_count_out = top - wants;
    }
    __syncthreads();
    if (gives > 0) {  // finished requests' pages, behind the free ones
#pragma unroll
      for (int i = 0; i < kBackKept; ++i)
        if (s + i * kPlanThreads < gives) a.free_pages[count + s + i * kPlanThreads] = kept[i];
#pragma unroll 4
      for (int k = s + kBackKept * kPlanThreads; k < gives; k += kPlanThreads) a.free_pages[count + k] = returned(k);
      __syncthreads();
    }
    for (int k = s; k < wants; k += kPlanThreads) {
      const int r = find_le(want0, B, k);
      a.block_tables[(size_t)r * a.max_pages + held[r] + k - want0[r]] = a.free_pages[top - 1 - k];
    }
  }
  if (a.fill) {
    __syncthreads();
    for (int t = 2 * s; t < a.total_q; t += 2 * kPlanThreads) fill_tokens(a, start, base, t);
  }
}

// The tokens of a step with many: 16 bytes written for each, the page looked
// up in L1 but for the first token of a page.
__global__ void __launch_bounds__(kFillThreads) k_tables_fill(TablesArgs a, int per_cta) {
  __shared__ int32_t start[kTMaxSeqs + 1], base[kTMaxSeqs];
  pdl_launch_dependents();
  pdl_wait();
  for (int i = threadIdx.x; i <= a.num_seqs; i += kFillThreads) {
    const int c = (int)a.cu[i];
    start[i] = c;
    if (i < a.num_seqs) base[i] = a.used[i] - ((int)a.cu[i + 1] - c);
  }
  __syncthreads();
  // (64 bits: the last round may pass 2^31)
  const long long t0 = (long long)blockIdx.x * per_cta, t1 = min((long long)a.total_q, t0 + per_cta);
  for (long long t = t0 + 2 * threadIdx.x; t < t1; t += 2 * kFillThreads) fill_tokens(a, start, base, (int)t);
}

struct MaskArgs {
  const int32_t* parents;
  const int64_t* cu;
  const int32_t* lens;
  uint32_t* mask;
  int64_t* positions;  // may be null
  int32_t* flags;      // may be null
  int32_t num_seqs, total_q, words, max_len;
};

__global__ void __launch_bounds__(kFillThreads) k_tree_mask(MaskArgs a) {
  __shared__ int32_t start[kTMaxSeqs + 1];
  pdl_launch_dependents();
  pdl_wait();
  int bad = 0;
  for (int i = threadIdx.x; i <= a.num_seqs; i += kFillThreads) {
    const long long c = a.cu[i], next = i < a.num_seqs ? a.cu[i + 1] : a.total_q;
    if (c < 0 || c > next) bad = 1;
    start[i] = (int)c;
  }
  if (__syncthreads_or(bad)) {  // nothing is written
    if (threadIdx.x == 0 && blockIdx.x == 0 && a.flags) atomicOr(a.flags, MXSA_FLAG_CU);
    return;
  }
  const int t = blockIdx.x * kFillThreads + threadIdx.x;
  if (t >= a.total_q || t < start[0] || t >= start[a.num_seqs]) return;
  const int s = find_le(start, a.num_seqs, t), b0 = start[s], tq = start[s + 1] - b0;
  int i = t - b0, depth = 0, flag = tq > 32 * a.words ? MXSA_FLAG_TREE : 0;
  uint32_t* row = a.mask + (size_t)t * a.words;
  int w = a.words - 1;  // the word that is being put together
  uint32_t bits = 0;
  while (true) {
    if ((i >> 5) <= w) {  // (tokens that the words do not reach are left out)
      for (; w > (i >> 5); --w) {
        row[w] = bits;
        bits = 0;
      }
      bits |= 1u << (i & 31);
    }
    const int up = a.parents[b0 + i];
    if (up < -1 || up >= i) flag |= MXSA_FLAG_TREE;
    if (up < 0 || up >= i || depth == 32 * kMaxMaskWords) break;
    i = up;
    ++depth;
  }
  for (; w >= 0; --w) {
    row[w] = bits;
    bits = 0;
  }
  const int len = a.lens[s], L = min(max(len, 0), a.max_len);
  if (L != len) flag |= MXSA_FLAG_LEN;
  if (L < tq) flag |= MXSA_FLAG_CAUSAL_LEN;
  if (a.positions) a.positions[t] = (long long)L - tq + depth;
  if (flag && a.flags) atomicOr(a.flags, flag);
}

}  // namespace

cudaError_t launch_tables(const mxsa_problem& p, const int32_t* kv_lens, const int32_t* new_lens,
                          const int32_t* pages_held, int32_t* block_tables, int32_t* free_pages,
                          const int32_t* free_count, int64_t* cu, int32_t* used, int64_t* positions, int64_t* loc,
                          int32_t* held_out, int32_t* free_count_out, int32_t* flags, cudaStream_t st) {
  TablesArgs a{};
  a.kv_lens = kv_lens;
  a.new_lens = new_lens;
  a.pages_held = pages_held;
  a.block_tables = block_tables;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.cu = cu;
  a.used = used;
  a.positions = positions;
  a.loc = loc;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  a.flags = flags;
  a.num_seqs = p.num_seqs;
  a.total_q = p.total_q;
  a.page_shift = p.page_size == 128 ? 7 : 6;
  a.num_pages = p.num_pages;
  a.max_pages = p.max_pages_per_seq;
  a.fill = p.total_q <= kTablesOneCta;
  cudaError_t e = launch_pdl(k_tables_plan, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e != cudaSuccess || a.fill) return e;
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // two CTAs per SM, each at least one round of its threads, an even number of tokens
  const long long round = 2 * kFillThreads;
  const long long per = std::max(round, ((long long)p.total_q + 2LL * sms - 1) / (2LL * sms) + round - 1) / round * round;
  const unsigned blocks = (unsigned)((p.total_q + per - 1) / per);
  return launch_pdl(k_tables_fill, dim3(blocks), dim3(kFillThreads), 0, st, a, (int)per);
}

cudaError_t launch_tree_mask(const mxsa_problem& p, const int32_t* parents, const int64_t* cu, const int32_t* lens,
                             int words, uint32_t* mask, int64_t* positions, int32_t* flags, cudaStream_t st) {
  if (p.total_q == 0) return cudaSuccess;
  MaskArgs a{};
  a.parents = parents;
  a.cu = cu;
  a.lens = lens;
  a.mask = mask;
  a.positions = positions;
  a.flags = flags;
  a.num_seqs = p.num_seqs;
  a.total_q = p.total_q;
  a.words = words;
  a.max_len = p.max_pages_per_seq * p.page_size;
  const unsigned blocks = (unsigned)(((long long)p.total_q + kFillThreads - 1) / kFillThreads);
  return launch_pdl(k_tree_mask, dim3(blocks), dim3(kFillThreads), 0, st, a);
}

}  // namespace mxsa

// Dense paged attention for a batch whose sequences share prefixes in groups
// (mxsa_dense_shared_fwd): a group's common keys are loaded and multiplied
// once for the rows of all its sequences, each sequence's own keys once for
// its rows, both split over the CTAs along the key axis, and the pieces of a
// row are joined by their log-sum-exps.
//
// Work.  A *job* is a token range and a key range of one block table row:
// the prefix keys [0, P) of a group for the tokens of all its sequences, and
// the keys [P, L) of a sequence for its own tokens.  Per kv head a job's
// tokens fall into *row tiles* of up to 2T tokens (T = 128 / G; two halves
// of up to 128 (token, head) rows) and its 128-key blocks into chunks; a
// *tile* is one chunk of one row tile.  Tiles are numbered row tile fastest,
// then chunk, so the CTAs that run at the same time read the same keys and
// meet in L2.  The tiles' blocks form one line of steps with a cost each,
// and the line is cut into one equal range per CTA: a tile cut by a range's
// end becomes two *segments*.  A chunk is about one range long, so the
// number of pieces a row falls into stays near the number of CTAs that its
// keys are worth, and the partial buffer is bounded by the shapes alone.
//
// Three launches: k_shared_plan (one CTA: jobs, tiles, ranges), k_shared
// (persistent, one CTA per SM) and k_shared_join.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"

namespace mxsa {

namespace {

constexpr int kHMaxSeqs = 1024;
constexpr int kHMaxCtas = 160;     // ranges; workspaces are sized for this many
constexpr int kHCostRows = 4;      // cost of one block for a tile of two halves
constexpr int kHCostKeys = 2;      // ... of one half (the halves then split the blocks)
constexpr int kHCostTile = 2;      // a tile's own: its q, the first block's latency, the epilogue

// One tile: keys [128 blk0, 128 (blk0 + nblk)) of [lo, hi) for ntok tokens.
struct alignas(16) HTile {
  int32_t tok0, ntok, g, row;      // first token, tokens, kv head, block table row
  int32_t lo, hi, blk0, nblk;
  long long cost0;                 // cost before its first step
  long long part0;                 // first partial row
  int32_t cta0;                    // first range that holds a step of it
  int32_t nseg;                    // ranges that do
  int32_t keys;                    // 1: one half of rows, the halves take alternate blocks
  int32_t pad;
};

struct HJob {
  int32_t tok0, ntok, row, lo, hi;
  int32_t tile0;                   // first tile
  int32_t nch, chunk, nrt;         // chunks, blocks of one, row tiles
};

struct HHeader {
  long long share;                 // cost of one range
  int32_t tiles, pad;
  int2 range[kHMaxCtas];           // first and last tile of each CTA's range (first > last: none)
};

struct HPtrs {
  HHeader* hdr;
  HJob* jobs;                      // [2 * num_seqs]: sequences' own keys, then the groups' prefixes
  int32_t* seq_job;                // [num_seqs]: the sequence's prefix job or -1
  int2* tok;                       // [total_q]: sequence (-1: none) and visible keys
  HTile* tiles;
  float* part_o;
  float* part_lse;                 // log2 units
};

struct HLayout {
  size_t hdr, jobs, seq_job, tok, tiles, part_o, part_lse, total;
  long long tile_cap, row_cap;
};

HLayout shared_layout(const mxsa_problem& p) {
  const long long G = p.num_q_heads / p.num_kv_heads, T = 128 / G;
  // (job, kv head, row tile) triples: each token lies in at most two jobs, a
  // job's last row tile may be short, and there are at most B + B / 2 jobs
  const long long triples = p.num_kv_heads * (2 * (p.total_q / (2 * T)) + 2LL * p.num_seqs);
  // chunks beyond the first: at most the CTAs' ranges, twice where a tile of
  // one half (half the cost) takes its job's longer chunk
  const long long extra = (kHCostRows / kHCostKeys) * kHMaxCtas;
  HLayout L;
  L.tile_cap = triples + extra;
  // a row and its twin (halves that split the blocks) in two jobs, and the
  // cuts, each of at most 256 rows
  L.row_cap = 4LL * p.total_q * p.num_q_heads + 256LL * (extra + kHMaxCtas);
  size_t o = 0;
  auto take = [&o](size_t n) {
    const size_t at = o;
    o = (o + n + 255) / 256 * 256;
    return at;
  };
  L.hdr = take(sizeof(HHeader));
  L.jobs = take(sizeof(HJob) * 2 * p.num_seqs);
  L.seq_job = take(4ull * p.num_seqs);
  L.tok = take(8ull * p.total_q);
  L.tiles = take(sizeof(HTile) * L.tile_cap);
  L.part_o = take(512ull * L.row_cap);
  L.part_lse = take(4ull * L.row_cap);
  L.total = o;
  return L;
}

HPtrs shared_ptrs(const HLayout& L, void* ws) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  HPtrs x;
  x.hdr = reinterpret_cast<HHeader*>(b + L.hdr);
  x.jobs = reinterpret_cast<HJob*>(b + L.jobs);
  x.seq_job = reinterpret_cast<int32_t*>(b + L.seq_job);
  x.tok = reinterpret_cast<int2*>(b + L.tok);
  x.tiles = reinterpret_cast<HTile*>(b + L.tiles);
  x.part_o = reinterpret_cast<float*>(b + L.part_o);
  x.part_lse = reinterpret_cast<float*>(b + L.part_lse);
  return x;
}

// ------------------------------------------------------------------- plan
struct HPlanArgs {
  const int64_t* cu;
  const int32_t* lens;
  const int32_t* group_ptr;
  const int32_t* prefix_lens;
  int32_t* flags;  // may be null
  HPtrs ws;
  long long tile_cap, row_cap;
  int32_t num_seqs, num_groups, total_q, Hkv, G, T, max_len, causal, ctas;
};

constexpr int kHPlanThreads = 1024;

struct HPlanSmem {
  int32_t cu[kHMaxSeqs + 1], len[kHMaxSeqs], seq_group[kHMaxSeqs];
  int32_t gp[kHMaxSeqs + 1], prefix[kHMaxSeqs];  // prefix: the group's shortest length, then its prefix length
  int32_t tile0[2 * kHMaxSeqs + 1];
  HJob job[2 * kHMaxSeqs];
  long long scan[32];
  int32_t first[kHMaxCtas], last[kHMaxCtas];
};

// exclusive sum over the block; *total gets the whole (1024 threads)
__device__ __forceinline__ long long block_scan(long long v, long long* s, long long* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous scan's readers are done
  if (lane == 31) s[w] = x;
  __syncthreads();
  long long y = s[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  const long long before = __shfl_sync(0xffffffffu, y, (w + 31) & 31);
  *total = __shfl_sync(0xffffffffu, y, 31);
  return x - v + (w ? before : 0);
}

// the last index i of a[0 .. n) (non-decreasing, a[0] <= x) with a[i] <= x
__device__ __forceinline__ int last_le(const int32_t* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kHPlanThreads) k_shared_plan(HPlanArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  HPlanSmem& s = *reinterpret_cast<HPlanSmem*>(smem_raw);
  const int tid = threadIdx.x, B = a.num_seqs, NG = a.num_groups;
  pdl_launch_dependents();
  pdl_wait();

  bool cu_ok = true, gp_ok = true;
  for (int i = tid; i <= B; i += kHPlanThreads) {
    const long long v = a.cu[i], nx = i < B ? a.cu[i + 1] : a.total_q;
    if (v < 0 || v > nx) cu_ok = false;
    s.cu[i] = (int)v;
  }
  for (int i = tid; i < B; i += kHPlanThreads) {
    const int L = a.lens[i];
    if ((L < 0 || L > a.max_len) && a.flags) atomicOr(a.flags, MXSA_FLAG_LEN);
    s.len[i] = min(max(L, 0), a.max_len);
    s.seq_group[i] = -1;
  }
  for (int i = tid; i <= NG && NG > 0; i += kHPlanThreads) {  // (no groups: the pointer may be null)
    const int v = a.group_ptr[i], nx = i < NG ? a.group_ptr[i + 1] : B;
    if (v < 0 || v > nx) gp_ok = false;
    s.gp[i] = v;
    if (i < NG) s.prefix[i] = a.max_len;
  }
  for (int i = tid; i < a.ctas; i += kHPlanThreads) {
    s.first[i] = INT_MAX;
    s.last[i] = -1;
  }
  cu_ok = __syncthreads_and(cu_ok);
  gp_ok = __syncthreads_and(gp_ok);
  if (tid == 0 && a.flags) {
    if (!cu_ok) atomicOr(a.flags, MXSA_FLAG_CU);
    if (!gp_ok) atomicOr(a.flags, MXSA_FLAG_GROUP);
  }
  if (!cu_ok) {  // no sequence has tokens: no tile, no row
    for (int t = tid; t < a.total_q; t += kHPlanThreads) a.ws.tok[t] = make_int2(-1, 0);
    for (int c = tid; c < a.ctas; c += kHPlanThreads) a.ws.hdr->range[c] = make_int2(0, -1);
    if (tid == 0) a.ws.hdr->share = 1, a.ws.hdr->tiles = 0;
    return;
  }
  // a group's prefix is at most its shortest sequence with tokens
  if (gp_ok && NG > 0)
    for (int i = tid; i < B; i += kHPlanThreads) {
      if (i < s.gp[0] || i >= s.gp[NG]) continue;
      const int j = last_le(s.gp, NG + 1, i);
      if (s.gp[j + 1] - s.gp[j] < 2) continue;  // one sequence alone shares nothing
      s.seq_group[i] = j;
      if (s.cu[i + 1] > s.cu[i]) atomicMin(&s.prefix[j], s.len[i]);
    }
  __syncthreads();
  for (int j = tid; j < NG; j += kHPlanThreads) {
    const int want = min(max(a.prefix_lens[j], 0), s.prefix[j]);
    const bool alone = !gp_ok || s.gp[j + 1] - s.gp[j] < 2;
    s.prefix[j] = alone ? 0 : want;
  }
  __syncthreads();
  for (int i = tid; i < B; i += kHPlanThreads)
    if (s.seq_group[i] >= 0 && s.prefix[s.seq_group[i]] == 0) s.seq_group[i] = -1;
  __syncthreads();

  // jobs, and the whole cost as far as it is known without causal trimming
  const int njobs = B + NG, T2 = 2 * a.T;
  long long cost = 0, total = 0;
  for (int q = tid; q < njobs; q += kHPlanThreads) {
    HJob j;
    if (q < B) {
      j.tok0 = s.cu[q];
      j.ntok = s.cu[q + 1] - s.cu[q];
      j.row = q;
      j.lo = s.seq_group[q] >= 0 ? s.prefix[s.seq_group[q]] : 0;
      j.hi = s.len[q];
      a.ws.seq_job[q] = s.seq_group[q] >= 0 ? B + s.seq_group[q] : -1;
    } else {
      const int r = q - B;
      const bool on = s.prefix[r] > 0;
      j.row = on ? s.gp[r] : 0;
      j.tok0 = on ? s.cu[s.gp[r]] : 0;
      j.ntok = on ? s.cu[s.gp[r + 1]] - j.tok0 : 0;
      j.lo = 0;
      j.hi = s.prefix[r];
    }
    const int nb = j.ntok > 0 && j.hi > j.lo ? ((j.hi + 127) >> 7) - (j.lo >> 7) : 0;
    const int rem = j.ntok % T2;
    const int keys = rem > 0 && rem <= a.T;
    j.nrt = nb > 0 ? (j.ntok + T2 - 1) / T2 : 0;
    j.chunk = j.nrt > keys ? kHCostRows : kHCostKeys;  // the cost of a block that sets the chunk, for now
    j.nch = nb;
    if (nb > 0)
      cost += (long long)a.Hkv * ((j.nrt - keys) * (nb * kHCostRows + kHCostTile) + keys * (nb * kHCostKeys + kHCostTile));
    s.job[q] = j;
  }
  block_scan(cost, s.scan, &total);
  const long long goal = max((total + a.ctas - 1) / a.ctas, 1LL);
  // a thread's jobs and tiles are consecutive from here on
  const int jper = (njobs + kHPlanThreads - 1) / kHPlanThreads;
  long long mine = 0, all = 0;
  __syncthreads();
  for (int q = tid * jper; q < min(njobs, (tid + 1) * jper); ++q) {
    HJob& j = s.job[q];
    const int nb = j.nch;
    j.chunk = (int)min((goal + j.chunk - 1) / j.chunk, (long long)max(nb, 1));
    j.nch = (nb + j.chunk - 1) / j.chunk;
    mine += (long long)a.Hkv * j.nch * j.nrt;
  }
  long long at = block_scan(mine, s.scan, &all);
  for (int q = tid * jper; q < min(njobs, (tid + 1) * jper); ++q) {
    HJob& j = s.job[q];
    j.tile0 = (int)at;
    s.tile0[q] = (int)at;
    at += (long long)a.Hkv * j.nch * j.nrt;
    a.ws.jobs[q] = j;
  }
  const int ntiles = (int)min(all, a.tile_cap);  // (all is within the cap: see shared_layout)
  __syncthreads();

  auto tile_of = [&](int i, HTile* t) {
    const int q = last_le(s.tile0, njobs, i);
    const HJob& j = s.job[q];
    int rel = i - j.tile0;
    const int rt = rel % j.nrt;
    rel /= j.nrt;
    const int ch = rel % j.nch;
    t->g = rel / j.nch;
    t->tok0 = j.tok0 + rt * T2;
    t->ntok = min(T2, j.ntok - rt * T2);
    t->row = j.row;
    t->lo = j.lo;
    t->hi = j.hi;
    int end = (j.hi + 127) >> 7;
    if (a.causal && q < B)  // keys past the last token's position are nobody's
      end = min(end, (max(j.hi - j.ntok + rt * T2 + t->ntok, 0) + 127) >> 7);
    t->blk0 = (j.lo >> 7) + ch * j.chunk;
    t->nblk = max(min(t->blk0 + j.chunk, end) - t->blk0, 0);
    t->keys = t->ntok <= a.T;
    t->pad = 0;
    return t->nblk ? (long long)t->nblk * (t->keys ? kHCostKeys : kHCostRows) + kHCostTile : 0LL;
  };
  const int tper = (ntiles + kHPlanThreads - 1) / kHPlanThreads;
  const int i0 = min(ntiles, tid * tper), i1 = min(ntiles, (tid + 1) * tper);
  HTile t;
  cost = 0;
  for (int i = i0; i < i1; ++i) cost += tile_of(i, &t);
  const long long before = block_scan(cost, s.scan, &total);
  const long long share = max((total + a.ctas - 1) / a.ctas, (long long)kHCostRows);
  // a tile's ranges: those that hold the start of one of its steps
  auto ranges = [&](HTile* x, long long c0) {
    const int w = x->keys ? kHCostKeys : kHCostRows;
    c0 += kHCostTile;
    x->cost0 = c0;
    x->cta0 = (int)(c0 / share);
    x->nseg = x->nblk > 0 ? (int)((c0 + (long long)(x->nblk - 1) * w) / share) - x->cta0 + 1 : 0;
    // a range may begin after the tile's first step and before its second:
    // share >= the cost of a step, so each range in between holds one
    return (long long)x->nseg * x->ntok * a.G * (x->keys ? 2 : 1);
  };
  long long run = before, rows = 0;
  for (int i = i0; i < i1; ++i) {
    const long long c = tile_of(i, &t);
    rows += ranges(&t, run);
    run += c;
  }
  long long part = block_scan(rows, s.scan, &all);
  run = before;
  for (int i = i0; i < i1; ++i) {
    const long long c = tile_of(i, &t);
    const long long n = ranges(&t, run);
    run += c;
    t.part0 = part;
    part += n;
    a.ws.tiles[i] = t;
    for (int k = 0; k < t.nseg; ++k) {
      atomicMin(&s.first[t.cta0 + k], i);
      atomicMax(&s.last[t.cta0 + k], i);
    }
  }
  for (int i = tid; i < a.total_q; i += kHPlanThreads) {
    int2 v = make_int2(-1, 0);
    if (i >= s.cu[0] && i < s.cu[B]) {
      const int q = last_le(s.cu, B, i);
      const int L = s.len[q];
      v.x = q;
      v.y = a.causal ? min(max(L - (s.cu[q + 1] - i) + 1, 0), L) : L;
    }
    a.ws.tok[i] = v;
  }
  __syncthreads();
  for (int c = tid; c < a.ctas; c += kHPlanThreads) a.ws.hdr->range[c] = make_int2(s.first[c], s.last[c]);
  if (tid == 0) {
    a.ws.hdr->share = share;
    a.ws.hdr->tiles = ntiles;
  }
}

// ---------------------------------------------------------------- forward
// 384 threads: two softmax groups (warps 0-3 and 4-7; thread = TMEM lane =
// row), a producer warp, two MMA issuers, and a warp that only makes the last
// warpgroup whole: it gives registers to the softmax groups, whose
// threads hold a row's 128 scores.  A tile of two halves gives each
// group its own 128 rows over the same blocks; a tile of one half gives both
// groups the same rows and alternate blocks (each then makes a partial of
// its own).  Per block: S = q k^T (TMEM), a lazily raised running maximum
// (raised when a score passes it by 2^8, O in TMEM is then rescaled),
// P = exp2(S - m) rounded to the 16-bit type over S, l += sum P, O += P V.
// Each group has an issuer: P V of a block, then q k^T of the group's next
// one, so that while one group runs its softmax the tensor pipe has the
// other's two products.  S is overwritten by the MMA after the one that reads
// P from it; both are issued by one thread, which the pipe keeps in
// order.  K and V blocks have a stage of 32 KB each in a ring of five, in the
// order in which the issuer takes them (K0 K1 V0 K2 V1 ... ), so 160 KB of
// loads are in flight when the CTA waits for memory.
constexpr int kHThreads = 384;
constexpr int kHProducer = 8, kHMma = 9;
constexpr uint32_t kHTileBytes = 32768;  // 128 rows x 128 x 16-bit
constexpr int kHStages = 5;
constexpr float kHRescale = 8.f;         // log2 units
constexpr uint32_t kHOffKV = 2 * kHTileBytes;
constexpr uint32_t kHOffCtrl = kHOffKV + kHStages * kHTileBytes;
// registers of a softmax thread and of the others: 256 x 216 + 128 x 72 is
// the launch's 384 x 168
constexpr int kHSoftmaxRegs = 216, kHOtherRegs = 72;
constexpr int kHSmallQ = 4;              // halves of at most this many tokens load their q token by token

// A role may pass over places and q slots of the other group without looking
// at their barriers.  A parity only tells a phase from the one before, so a
// stage's (and a q buffer's) uses alternate between two "full" barriers: to
// mistake a phase a role would have to be two uses ahead of the copies, and
// each wait comes after one for a copy that was issued later than that.
struct HCtrl {
  uint64_t q_full[4], q_empty[2], kv_full[2 * kHStages], kv_empty[kHStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], turn[2], done;
  uint32_t tmem_base;
  int32_t abort_flag, local_flags;
};

struct HArgs {
  const int32_t* block_tables;
  int32_t* flags;  // may be null
  HPtrs ws;
  int32_t G, T, Hkv, page_shift, max_pages, num_pages, causal;
  float scale_log2;
};

// The part of a tile that range c holds: blocks [b0, b0 + n) of the keys.
struct HSeg {
  HTile t;
  int b0, n;
};

__device__ __forceinline__ HTile load_tile(const HTile* p) {
  HTile t;
  const int4* s = reinterpret_cast<const int4*>(p);
  int4* d = reinterpret_cast<int4*>(&t);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(HTile) / 16); ++i) d[i] = s[i];
  return t;
}

// first step of the tile that costs at least `cost` from the line's start
__device__ __forceinline__ int step_at(const HTile& t, long long cost) {
  const long long d = cost - t.cost0;
  if (d <= 0) return 0;
  const int w = t.keys ? kHCostKeys : kHCostRows;
  return (int)min((d + w - 1) / w, (long long)t.nblk);
}

__device__ __forceinline__ void cut(HSeg* s, long long share, int c) {
  const int i0 = step_at(s->t, c * share), i1 = step_at(s->t, (c + 1) * share);
  s->b0 = s->t.blk0 + i0;
  s->n = i1 - i0;
}

// ring places of a segment's blocks, relative to the segment's first: K0, K1,
// V0, K2, V1, ..., K(n-1), V(n-2), V(n-1)
__device__ __forceinline__ int place_k(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int place_v(int i, int n) { return i < n - 1 ? 2 * i + 2 : 2 * n - 1; }

__device__ __forceinline__ float hmax3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// the larger of two; NaN when one is
__device__ __forceinline__ float hmax_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t hpack2(float a, float b) {
  if (kBf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ bool hwarp_all(bool v) { return __all_sync(0xffffffffu, v); }

// eight consecutive floats to global memory (32-byte aligned)
__device__ __forceinline__ void st_global_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// One lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Low words of the operands' shared-memory descriptors (the high word is the
// same for all: 1024 bytes between groups of 8 rows, version 1, 128-byte
// swizzle); the address field counts 16 bytes and does not overflow below.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k_major(uint32_t saddr) { return saddr >> 4; }
__device__ __forceinline__ uint32_t desc_mn_major(uint32_t saddr) { return (saddr >> 4) | ((16384u >> 4) << 16); }
// a value that all lanes hold, in a form the compiler knows to be uniform
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The eight products over 16 columns each of one block.  S = q k^T: both
// operands K-major, 64 columns to a 16 KB half, 32 bytes a step.  O (+)= P V:
// P in TMEM, 8 columns a step, V MN-major, 16 rows (2 KB) a step.
template <int kStep>
__device__ __forceinline__ void mma_qk_step(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  constexpr int off = ((kStep >> 2) * 16384 + (kStep & 3) * 32) >> 4;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 u, v;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tadd.u32 u, %1, %5;\n\tadd.u32 v, %2, %5;\n\t"
      "mov.b64 x, {u, %6};\n\tmov.b64 y, {v, %6};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(q), "r"(k), "r"(idesc), "n"(kStep > 0), "n"(off), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  mma_qk_step<0>(d, q, k, idesc);
  mma_qk_step<1>(d, q, k, idesc);
  mma_qk_step<2>(d, q, k, idesc);
  mma_qk_step<3>(d, q, k, idesc);
  mma_qk_step<4>(d, q, k, idesc);
  mma_qk_step<5>(d, q, k, idesc);
  mma_qk_step<6>(d, q, k, idesc);
  mma_qk_step<7>(d, q, k, idesc);
}
template <int kStep>
__device__ __forceinline__ void mma_pv_step(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t.reg .b32 x, v;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tadd.u32 x, %1, %5;\n\tadd.u32 v, %2, %6;\n\tmov.b64 y, {v, %7};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
      "r"(tp), "r"(v), "r"(idesc), "r"(acc), "n"(kStep * 8), "n"(kStep * (2048 >> 4)), "r"(kDescHi)
      : "memory");
}
// the first and the second 64 keys
__device__ __forceinline__ void mma_pv_lo(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc, uint32_t acc) {
  mma_pv_step<0>(d, tp, v, idesc, acc);
  mma_pv_step<1>(d, tp, v, idesc, 1u);
  mma_pv_step<2>(d, tp, v, idesc, 1u);
  mma_pv_step<3>(d, tp, v, idesc, 1u);
}
__device__ __forceinline__ void mma_pv_hi(uint32_t d, uint32_t tp, uint32_t v, uint32_t idesc) {
  mma_pv_step<4>(d, tp, v, idesc, 1u);
  mma_pv_step<5>(d, tp, v, idesc, 1u);
  mma_pv_step<6>(d, tp, v, idesc, 1u);
  mma_pv_step<7>(d, tp, v, idesc, 1u);
}

// two floats in a 64-bit register, and their packed arithmetic
__device__ __forceinline__ uint64_t pack_f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack_f2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// a warpgroup's registers per thread, from or to the launch's pool
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <bool kBf16>
__global__ void __launch_bounds__(kHThreads, 1)
    k_shared(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmq1,
             const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, HArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  HCtrl& c = *reinterpret_cast<HCtrl*>(sm + kHOffCtrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_full[i + 2], 1);
      mbar_init(&c.q_empty[i], 2);  // (see the issuers)
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 4);
      mbar_init(&c.p_full[i], 4);   // one arrival per warp of the group
      mbar_init(&c.o_full[i], 1);
      mbar_init(&c.turn[i], 1);
      mbar_init(&c.o_empty[i], 4);
    }
    for (int i = 0; i < kHStages; ++i) {
      mbar_init(&c.kv_full[i], 1);
      mbar_init(&c.kv_full[i + kHStages], 1);
      mbar_init(&c.kv_empty[i], 2);
    }
    mbar_init(&c.done, 2);
    c.abort_flag = 0;
    c.local_flags = 0;
    fence_mbar_init();
  }
  if (warp == kHMma) {
    tmem_alloc(&c.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  volatile int* abort_flag = &c.abort_flag;
  int32_t* const fl = a.flags ? a.flags : &c.local_flags;
  const uint32_t sbase = smem_u32(sm);
  const int G = a.G, cta = blockIdx.x;
  pdl_wait();  // the plan
  const int2 range = a.ws.hdr->range[cta];
  const long long share = a.ws.hdr->share;

  if (warp >= 8) {
    regs_dec<kHOtherRegs>();
    if (warp == kHProducer) {
      // -------------------------------------------------------------- producer
      if (lane == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmq1);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
      }
      const int ps = 1 << a.page_shift, npg = ps == 128 ? 1 : 2;
      int at = 0, qn = 0;  // ring places taken so far
      bool ok = true;
      HSeg s;
      for (int ti = range.x; ti <= range.y && ok; ++ti) {
        s.t = load_tile(a.ws.tiles + ti);  // (the ring holds loads for longer than this takes)
        cut(&s, share, cta);
        if (s.n <= 0) continue;
        const int nh = s.t.keys ? 1 : 2;
        for (int h = 0; h < nh && ok; ++h, ++qn) {
          const int b = qn & 1;
          ok = hwarp_all(
              mbar_wait(&c.q_empty[b], ((qn >> 1) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
          if (!ok) break;
          if (lane == 0) {
            uint8_t* qd = sm + b * kHTileBytes;
            uint64_t* full = &c.q_full[qn & 3];
            const int t0 = s.t.tok0 + h * a.T, nt = min(a.T, s.t.ntok - h * a.T);
            if (nt > kHSmallQ) {  // one box; rows past the tile's tokens are never used
              mbar_arrive_expect_tx(full, (uint32_t)(G * a.T) * 256u);
              tma_load_3d(qd, &tmq, full, 0, s.t.g * G, t0);
              tma_load_3d(qd + 16384, &tmq, full, 64, s.t.g * G, t0);
            } else {
              mbar_arrive_expect_tx(full, (uint32_t)(G * nt) * 256u);
              for (int x = 0; x < nt; ++x) {
                tma_load_3d(qd + x * G * 128, &tmq1, full, 0, s.t.g * G, t0 + x);
                tma_load_3d(qd + 16384 + x * G * 128, &tmq1, full, 64, s.t.g * G, t0 + x);
              }
            }
          }
        }
        // block i's pages come from a window of 32 blocks that the lanes hold;
      // the next window is loaded while this one is used
      const int32_t* row = a.block_tables + (size_t)s.t.row * a.max_pages;
      auto pages_at = [&](int i, int pg) -> int {  // lane's page pg of block i + lane, -1: none or not needed
        const int b = s.b0 + i + lane;
        const int p0 = b * 128 + pg * 64;  // its first key
        if (pg >= npg || i + lane >= s.n || p0 >= s.t.hi || p0 + ps <= s.t.lo) return -1;
        const int phys = row[p0 >> a.page_shift];
        if (phys >= 0 && phys < a.num_pages) return phys;
        atomicOr(fl, MXSA_FLAG_PAGE);
        return -1;
      };
      int win[2] = {pages_at(0, 0), pages_at(0, 1)}, ahead[2] = {pages_at(32, 0), pages_at(32, 1)};
      int prev[2] = {-1, -1};
      for (int i = 0; i <= s.n && ok; ++i) {
        int cur[2] = {-1, -1};
        if (i < s.n) {
          if ((i & 31) == 0 && i > 0) {
#pragma unroll
            for (int pg = 0; pg < 2; ++pg) {
              win[pg] = ahead[pg];
              ahead[pg] = pages_at(i + 32, pg);
            }
          }
          cur[0] = __shfl_sync(0xffffffffu, win[0], i & 31);
          cur[1] = __shfl_sync(0xffffffffu, win[1], i & 31);
        }
        // K of block i, then V of block i - 1: the ring's order
#pragma unroll
          for (int kv = 0; kv < 2 && ok; ++kv) {
            if (kv == 0 ? i >= s.n : i == 0) continue;
            const int* pg = kv == 0 ? cur : prev;
            const int st = at % kHStages, use = at / kHStages;
            ok = hwarp_all(mbar_wait(&c.kv_empty[st], (use & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
            if (!ok) break;
            ++at;
            if (lane == 0) {
              uint64_t* full = &c.kv_full[(at - 1) % (2 * kHStages)];
              uint8_t* dst = sm + kHOffKV + st * kHTileBytes;
              const int present = (pg[0] >= 0) + (pg[1] >= 0);
              const CUtensorMap* tm = kv == 0 ? &tmk : &tmv;
              mbar_arrive_expect_tx(full, (uint32_t)present * (uint32_t)ps * 256u);
              for (int x = 0; x < npg; ++x) {
                if (pg[x] < 0) continue;
                const int z = pg[x] * a.Hkv + s.t.g;
                tma_load_3d(dst + x * 8192, tm, full, 0, 0, z);
                tma_load_3d(dst + 16384 + x * 8192, tm, full, 64, 0, z);
              }
            }
          }
          prev[0] = cur[0];
          prev[1] = cur[1];
        }
      }
      // drain: the copies in flight land before the CTA may exit
      if (lane == 0) {
        for (int k = max(0, at - kHStages); k < at; ++k)
          mbar_drain(&c.kv_full[k % (2 * kHStages)], (k / (2 * kHStages)) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
        for (int k = max(0, qn - 2); k < qn; ++k)
          mbar_drain(&c.q_full[k & 3], (k >> 2) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == kHMma || warp == kHMma + 1) {
      // --------------------------------------------------------- MMA issuers
      // One warp per group.  The whole warp walks the loop and one elected
      // lane issues: what the instructions take from uniform registers is
      // then uniform.  After a run of products the warp stands still until
      // the pipe has taken them, so P V and the next q k^T go out together
      // when K is there, and the other warp's products fill the time between.
      const int h = warp - kHMma;
      const uint32_t id_qk = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 0);
      const uint32_t id_pv = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 1);
      int at = 0, qn = 0;
      int np = 0, no = 0;           // products P V issued, tiles finished
      int nt = 0;                   // turns taken
      int owed = -1, bits = 0;      // ring place of the V that the next P V takes; bit 0: first of its tile, 1: last,
                                    // 2: no other group reads V
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        ok = ok && hwarp_all(mbar_wait(bar, parity, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      };
      auto wait_v = [&] {  // V and, at a tile's start, O of the group's previous tile read out
        wait(&c.kv_full[owed % (2 * kHStages)], (owed / (2 * kHStages)) & 1);
        if ((bits & 1) && no > 0) wait(&c.o_empty[h], (no - 1) & 1);
      };
      // P V: its first half once P's first 64 keys are there, the second by
      // `rest` (the elected lane, after P's second half)
      auto start_pv = [&](uint32_t tS, uint32_t dv) {
        wait(&c.p_half[h], np & 1);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) mma_pv_lo(tS + 128, tS, dv, id_pv, (bits & 1) ? 0u : 1u);
        __syncwarp();
        wait(&c.p_full[h], np & 1);
      };
      auto rest_pv = [&](uint32_t tS, uint32_t dv, uint64_t* empty) {
        mma_pv_hi(tS + 128, tS, dv, id_pv);
        mma_commit(empty);
        if (bits & 4) mma_commit(empty);
        if (bits & 2) mma_commit(&c.o_full[h]);
      };
      auto done_pv = [&] {
        ++np;
        no += (bits >> 1) & 1;
        owed = -1;
      };
      const uint32_t tS = uniform(tmem + h * 256);
      for (int ti = range.x; ti <= range.y && ok; ++ti) {
        HSeg s;
        s.t = load_tile(a.ws.tiles + ti);  // (the last blocks' softmax takes longer than this)
        cut(&s, share, cta);
        if (s.n <= 0) continue;
        const int n = s.n, keys = s.t.keys, stride = keys ? 2 : 1;
        const int half = keys ? h ^ (qn & 1) : 0;  // (see the softmax)
        const int qp = keys ? qn : qn + h;
        for (int i = half; i < n && ok; i += stride) {
          const int kp = at + place_k(i), st = kp % kHStages;
          const int sv = max(owed, 0) % kHStages;
          const uint32_t dv = uniform(desc_mn_major(sbase + kHOffKV + sv * kHTileBytes));
          const uint32_t dq = uniform(desc_k_major(sbase + (qp & 1) * kHTileBytes));
          const uint32_t dk = uniform(desc_k_major(sbase + kHOffKV + st * kHTileBytes));
          // In a tile of two halves the groups take turns at the pipe: left
          // alone they can fall into step, both in their softmax at once and
          // then both waiting for each other's products.
          if (!keys) {
            if (h == 1 || nt > 0) wait(&c.turn[h], (nt + h + 1) & 1);
            ++nt;
            if (!ok) break;
          }
          if (owed >= 0) {
            wait_v();
            // P V alone when K (or a new tile's q) may not be there yet
            const bool alone =
                i == half || !hwarp_all(mbar_test(&c.kv_full[kp % (2 * kHStages)], (kp / (2 * kHStages)) & 1));
            start_pv(tS, dv);
            if (!ok) break;
            if (alone) {
              tc_fence_after();
              if (elect_one()) rest_pv(tS, dv, &c.kv_empty[sv]);
              __syncwarp();
              done_pv();
            }
          }
          if (owed < 0) {
            if (i == half) wait(&c.q_full[qp & 3], (qp >> 2) & 1);
            wait(&c.kv_full[kp % (2 * kHStages)], (kp / (2 * kHStages)) & 1);
            if (!ok) break;
          }
          const bool last = i + stride >= n;
          tc_fence_after();
          if (elect_one()) {
            if (owed >= 0) rest_pv(tS, dv, &c.kv_empty[sv]);
            mma_qk(tS, dq, dk, id_qk);
            mma_commit(&c.s_full[h]);
            // (two arrivals free a stage or a q buffer: one of each group, or both of the only one)
            mma_commit(&c.kv_empty[st]);
            if (keys) mma_commit(&c.kv_empty[st]);
            if (last) mma_commit(&c.q_empty[qp & 1]);
            if (last && !keys) mma_commit(&c.q_empty[qp & 1]);
            if (!keys) mbar_arrive(&c.turn[h ^ 1]);
          }
          __syncwarp();
          if (owed >= 0) done_pv();
          owed = at + place_v(i, n);
          bits = (i == half ? 1 : 0) | (last ? 2 : 0) | (keys ? 4 : 0);
        }
        if (half >= n && ok) {  // no block of this tile is the group's: nothing else would free what it owes
          if (owed >= 0) {
            const int sv = owed % kHStages;
            const uint32_t dv = uniform(desc_mn_major(sbase + kHOffKV + sv * kHTileBytes));
            wait_v();
            start_pv(tS, dv);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) rest_pv(tS, dv, &c.kv_empty[sv]);
            __syncwarp();
            done_pv();
          }
          wait(&c.q_full[qp & 3], (qp >> 2) & 1);
          if (!ok) break;
          if (elect_one()) mma_commit(&c.q_empty[qp & 1]);
          __syncwarp();
        }
        at += 2 * n;
        qn += keys ? 1 : 2;
      }
      if (ok && owed >= 0) {
        const int sv = owed % kHStages;
        const uint32_t dv = uniform(desc_mn_major(sbase + kHOffKV + sv * kHTileBytes));
        wait_v();
        start_pv(tS, dv);
        tc_fence_after();
        if (ok && elect_one()) rest_pv(tS, dv, &c.kv_empty[sv]);
        __syncwarp();
      }
      if (elect_one()) {
        mma_commit(&c.done);
        mbar_drain(&c.done, 0, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else {
    regs_inc<kHSoftmaxRegs>();
    // --------------------------------------------------------------- softmax
    const int h = warp >> 2;
    const int r = tid & 127;  // row of the half == TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + h * 256 + lane_addr, tO = tS + 128;
    const int rt = r / G;
    int at = 0, qn = 0, n_s = 0, n_o = 0;
    bool ok = true;
    HTile next = range.x <= range.y ? load_tile(a.ws.tiles + range.x) : HTile{};
    for (int ti = range.x; ti <= range.y && ok; ++ti) {
      // what the block loop and the epilogue need of the tile, and no more:
      // a row's 128 scores leave few registers
      HSeg s;
      s.t = next;
      cut(&s, share, cta);
      const int n = s.n, b0 = s.b0, lo = s.t.lo, key_end = s.t.hi, keys = s.t.keys, stride = keys ? 2 : 1;
      // the group that takes a one-half tile's first block changes with the q
      // buffer, so that short tiles keep both groups busy
      const int half = keys ? h ^ (qn & 1) : 0;
      if (n > 0) qn += keys ? 1 : 2;
      const int tt = rt + (keys ? 0 : h * a.T);  // the row's token within the tile
      const bool live = rt < a.T && tt < s.t.ntok;
      const long long rows = (long long)s.t.ntok * G;
      const long long pr =
          s.t.part0 + (cta - s.t.cta0) * rows * stride + half * rows + tt * G + (r - rt * G);
      const bool warp_live = __any_sync(0xffffffffu, live);
      int hi = key_end;  // the row sees the keys [lo, hi), all of the warp's rows [lo, warp_hi)
      if (n > 0 && a.causal && live) hi = min(hi, a.ws.tok[s.t.tok0 + tt].y);
      const int warp_hi = __reduce_min_sync(0xffffffffu, hi);
      float m = -INFINITY, l = 0.f;
      bool mine = false;  // this group has blocks of the segment
      for (int i = half; i < n && ok; i += stride, ++n_s) {
        const int k0 = (b0 + i) << 7;  // the block's first key
        ok = hwarp_all(mbar_wait(&c.s_full[h], n_s & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
        if (!ok) break;
        if (k0 < lo || k0 + 128 > key_end) {
          // V rows of keys outside [lo, hi): zeros, since a stale row may hold
          // NaN bits and 0 * NaN would reach O.  (Their stage has landed
          // once its barrier says so; the writers' proxy fence orders them
          // before the product.)
          const int pl = at + place_v(i, n), st = pl % kHStages;
          ok = hwarp_all(mbar_wait(&c.kv_full[pl % (2 * kHStages)], (pl / (2 * kHStages)) & 1, abort_flag, fl,
                                   MXSA_FLAG_TIMEOUT, kWaitLimitNs));
          if (!ok) break;
          if (k0 + r < lo || k0 + r >= key_end) {
            const uint32_t vs = sbase + kHOffKV + st * kHTileBytes + r * 128;
            for (int ch = 0; ch < 16; ++ch)
              st_shared_v4(vs + (ch >> 3) * 16384u + (((ch & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (warp_live) {
          tc_fence_after();
          float sv[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sv + q * 32);
          tmem_ld_wait();
          if (k0 < lo || k0 + 128 > warp_hi) {
            const int rlo = lo - k0, rhi = hi - k0;
#pragma unroll
            for (int k = 0; k < 128; ++k) sv[k] = k >= rlo && k < rhi ? sv[k] : -INFINITY;
          }
          float b0 = -INFINITY, b1 = -INFINITY, b2 = -INFINITY, b3 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 128; k += 8) {
            b0 = hmax3(b0, sv[k], sv[k + 1]);
            b1 = hmax3(b1, sv[k + 2], sv[k + 3]);
            b2 = hmax3(b2, sv[k + 4], sv[k + 5]);
            b3 = hmax3(b3, sv[k + 6], sv[k + 7]);
          }
          const float bm = fmaxf(fmaxf(b0, b1), fmaxf(b2, b3)) * a.scale_log2;
          const bool raise = live && (bm > m + kHRescale || (m == -INFINITY && bm > -INFINITY));
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? (m == -INFINITY ? 0.f : ex2_approx(m - bm)) : 1.f;
            if (mine) {
              // O holds the segment's blocks so far and is complete: S's
              // barrier follows every product issued before
#pragma unroll
              for (int cb = 0; cb < 8; ++cb) {  // 16 columns at a time: the scores keep their registers
                uint32_t w[16];
                tmem_ld16(tO + cb * 16, w);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
                tmem_st16(tO + cb * 16, w);
              }
            }
            if (raise) {
              l *= f;
              m = bm;
            }
          }
          const float mm = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = pack_f2(a.scale_log2, a.scale_log2), off2 = pack_f2(-mm, -mm);
          uint64_t l0 = pack_f2(0.f, 0.f), l1 = l0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 x = unpack_f2(fma_f2(pack_f2(sv[32 * q + 2 * k], sv[32 * q + 2 * k + 1]), scale2, off2));
              const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
              if (k & 1) l1 = add_f2(l1, pack_f2(p0, p1));
              else l0 = add_f2(l0, pack_f2(p0, p1));
              pk[k] = hpack2<kBf16>(p0, p1);
            }
            tmem_st16(tS + 16 * q, pk);
            if (q == 1) {  // the first 64 keys: their half of P V may start
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&c.p_half[h]);
            }
          }
          const float2 ls = unpack_f2(add_f2(l0, l1));
          l += ls.x + ls.y;
          tmem_st_wait();
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.p_half[h]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full[h]);
        mine = true;
      }
      at += 2 * max(n, 0);
      if (ti < range.y) next = load_tile(a.ws.tiles + ti + 1);
      if (!ok || !mine) continue;
      // ---- the segment's partial rows
      ok = hwarp_all(mbar_wait(&c.o_full[h], n_o & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      if (!ok) break;
      ++n_o;
      if (warp_live) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN stays one)
        float* po = a.ws.part_o + pr * 128;
#pragma unroll
        for (int cb = 0; cb < 4; ++cb) {
          float ov[32];
          tmem_ld32(tO + cb * 32, ov);  // every lane: the load is warp-collective
          tmem_ld_wait();
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; ++k) ov[k] *= inv;
#pragma unroll
            for (int k = 0; k < 32; k += 8) st_global_v8(po + cb * 32 + k, ov + k);
          }
        }
        if (live) a.ws.part_lse[pr] = l == 0.f ? -INFINITY : m + lg2_approx(l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.o_empty[h]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kHMma) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- join
// out = sum w_k o_k / sum w_k, w_k = 2^(lse_k - max lse), over the partials of
// a (token, query head) row: those of its sequence's own tile and of its
// group's, a chunk and a range each.  One CTA per (token, kv head): its G
// rows have the same list of partials, made once; a warp then takes a row.
constexpr int kHJoinThreads = 128;
// Partials of one row: its two jobs have a chunk each, plus at most `ctas`
// further chunks (2 x where the job's chunk is counted at twice the tile's
// cost) and `ctas` cuts, all of them possibly in two halves.
constexpr int kHJoinMax = 2 * (2 + 3 * kHMaxCtas);

struct HJoinArgs {
  HPtrs ws;
  uint8_t* out;
  float* lse;  // may be null
  int32_t Hkv, G, T, total_q, ctas;
};

template <bool kBf16>
__global__ void __launch_bounds__(kHJoinThreads) k_shared_join(HJoinArgs a) {
  __shared__ int32_t count;
  __shared__ long long list[kHJoinMax];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x / a.Hkv, g = blockIdx.x - t * a.Hkv;
  pdl_launch_dependents();
  if (tid == 0) count = 0;
  pdl_wait();
  __syncthreads();
  const int2 tk = a.ws.tok[t];
  if (tk.x < 0) return;  // outside every sequence: not written
  if (warp == 0) {
    int n = 0;
    const int pj = a.ws.seq_job[tk.x];
    const long long share = a.ws.hdr->share;
    for (int w = 0; w < 2; ++w) {
      const int ji = w == 0 ? pj : tk.x;
      if (ji < 0) continue;
      const HJob j = a.ws.jobs[ji];
      if (j.nrt == 0) continue;
      const int base = j.tile0 + g * j.nch * j.nrt + (t - j.tok0) / (2 * a.T);
      for (int c0 = 0; c0 < j.nch; c0 += 32) {
        HSeg s;
        s.t.nseg = 0;
        int mine = 0;
        if (c0 + lane < j.nch) {
          s.t = load_tile(a.ws.tiles + base + (c0 + lane) * j.nrt);
          for (int k = 0; k < s.t.nseg; ++k) {
            cut(&s, share, s.t.cta0 + k);
            mine += s.t.keys && s.n > 1 ? 2 : 1;
          }
        }
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        int at = n + x - mine;
        n += __shfl_sync(0xffffffffu, x, 31);
        const long long rows = (long long)s.t.ntok * a.G;
        for (int k = 0; k < s.t.nseg; ++k) {
          cut(&s, share, s.t.cta0 + k);
          const int nh = s.t.keys && s.n > 1 ? 2 : 1;
          for (int hh = 0; hh < nh; ++hh, ++at)
            if (at < kHJoinMax)
              list[at] = s.t.part0 + (k * (s.t.keys ? 2 : 1) + hh) * rows + (long long)(t - s.t.tok0) * a.G;
        }
      }
    }
    if (lane == 0) count = min(n, kHJoinMax);
  }
  __syncthreads();
  const int n = count;
  for (int hh = warp; hh < a.G; hh += kHJoinThreads / 32) {
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = hmax_nan(M, a.ws.part_lse[list[i] + hh]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = hmax_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float W = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const long long pr = list[i] + hh;
        const float w = ex2_approx(a.ws.part_lse[pr] - M);
        const float4 o = __ldcs(reinterpret_cast<const float4*>(a.ws.part_o + pr * 128) + lane);
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
        W += w;
      }
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;
    const int h = g * a.G + hh;
    reinterpret_cast<uint2*>(a.out + ((size_t)t * a.Hkv * a.G + h) * 256)[lane] =
        make_uint2(hpack2<kBf16>(acc.x * inv, acc.y * inv), hpack2<kBf16>(acc.z * inv, acc.w * inv));
    if (a.lse && lane == 0)
      a.lse[(size_t)h * a.total_q + t] = W == 0.f ? -INFINITY : (M + lg2_approx(W)) * 0.69314718055994530942f;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 shared_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

}  // namespace

size_t shared_workspace_bytes(const mxsa_problem& p) { return shared_layout(p).total; }

cudaError_t launch_dense_shared(const mxsa_problem& p, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, const int64_t* cu, const int32_t* lens, int num_groups,
                                const int32_t* group_ptr, const int32_t* prefix_lens, void* ws, void* out, float* lse,
                                int32_t* flags, cudaStream_t st) {
  if (p.total_q == 0) return cudaSuccess;
  auto fn = shared_encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const int G = p.num_q_heads / p.num_kv_heads, T = 128 / G;
  const bool bf16 = p.q_dtype == MXSA_BF16;
  const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto map3 = [&](CUtensorMap* m, const void* base, cuuint64_t d1, cuuint64_t d2, cuuint32_t b1, cuuint32_t b2) {
    cuuint64_t dims[3] = {128, d1, d2}, strides[2] = {256, 256 * d1};
    cuuint32_t box[3] = {64, b1, b2}, es[3] = {1, 1, 1};
    return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  CUtensorMap tmq, tmq1, tmk, tmv;
  const cuuint64_t slabs = (cuuint64_t)p.num_pages * p.num_kv_heads;
  if (!map3(&tmq, q, p.num_q_heads, p.total_q, G, T) || !map3(&tmq1, q, p.num_q_heads, p.total_q, G, 1) ||
      !map3(&tmk, k_cache, p.page_size, slabs, p.page_size, 1) ||
      !map3(&tmv, v_cache, p.page_size, slabs, p.page_size, 1))
    return cudaErrorInvalidValue;
  const HLayout L = shared_layout(p);
  const HPtrs ptrs = shared_ptrs(L, ws);
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int ctas = std::min(sms, kHMaxCtas);
  const size_t smem = kHOffCtrl + sizeof(HCtrl) + 1024;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [smem] {
    const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    attr_err = cudaFuncSetAttribute(k_shared<true>, a, (int)smem);
    if (attr_err == cudaSuccess) attr_err = cudaFuncSetAttribute(k_shared<false>, a, (int)smem);
    if (attr_err == cudaSuccess) attr_err = cudaFuncSetAttribute(k_shared_plan, a, (int)sizeof(HPlanSmem));
  });
  if (attr_err != cudaSuccess) return attr_err;

  HPlanArgs pa{};
  pa.cu = cu;
  pa.lens = lens;
  pa.group_ptr = group_ptr;
  pa.prefix_lens = prefix_lens;
  pa.flags = flags;
  pa.ws = ptrs;
  pa.tile_cap = L.tile_cap;
  pa.row_cap = L.row_cap;
  pa.num_seqs = p.num_seqs;
  pa.num_groups = num_groups;
  pa.total_q = p.total_q;
  pa.Hkv = p.num_kv_heads;
  pa.G = G;
  pa.T = T;
  pa.max_len = p.max_pages_per_seq * p.page_size;
  pa.causal = p.causal;
  pa.ctas = ctas;
  cudaError_t e = launch_pdl(k_shared_plan, dim3(1), dim3(kHPlanThreads), sizeof(HPlanSmem), st, pa);
  if (e != cudaSuccess) return e;

  HArgs fa{};
  fa.block_tables = block_tables;
  fa.flags = flags;
  fa.ws = ptrs;
  fa.G = G;
  fa.T = T;
  fa.Hkv = p.num_kv_heads;
  fa.page_shift = p.page_size == 128 ? 7 : 6;
  fa.max_pages = p.max_pages_per_seq;
  fa.num_pages = p.num_pages;
  fa.causal = p.causal;
  const float scale = p.softmax_scale > 0.f ? p.softmax_scale : 0.08838834764831845f;  // 1/sqrt(128)
  fa.scale_log2 = scale * 1.4426950408889634f;
  e = launch_pdl(bf16 ? k_shared<true> : k_shared<false>, dim3(ctas), dim3(kHThreads), smem, st, tmq, tmq1, tmk, tmv,
                 fa);
  if (e != cudaSuccess) return e;

  HJoinArgs ja{};
  ja.ws = ptrs;
  ja.out = static_cast<uint8_t*>(out);
  ja.lse = lse;
  ja.Hkv = p.num_kv_heads;
  ja.G = G;
  ja.T = T;
  ja.total_q = p.total_q;
  ja.ctas = ctas;
  return launch_pdl(bf16 ? k_shared_join<true> : k_shared_join<false>, dim3((unsigned)p.total_q * p.num_kv_heads),
                    dim3(kHJoinThreads), 0, st, ja);
}

}  // namespace mxsa

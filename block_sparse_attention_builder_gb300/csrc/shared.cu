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
// *tile* is one chunk of one row tile.  Every tile writes partial rows of its
// own, so it does not matter which CTA takes it, nor when.
//
// Tiles of two halves are bound by the tensor pipe and the softmax, tiles of
// one half (decoding sequences' own keys) by memory.  They stand in two
// queues; each CTA takes from the one until it is empty, then from the
// other, and as many CTAs begin with each as it has of the work, so that
// both kinds run at the same time and the CTAs end together.  (Equal shares
// of the work fixed beforehand, tiles cut where a share ended: the slowest
// CTAs took 540 us where the median took 490 us.)  A queue's tiles are in row
// tile order within a chunk, so the CTAs that run at the same time read the
// same keys and meet in L2.  A chunk is half of a CTA's share of all work,
// which bounds the partial buffer by the shapes alone.
//
// Three launches: k_shared_plan (one CTA: jobs, tiles, queues), k_shared
// (persistent, one CTA per SM) and k_shared_join.  64 decoding sequences of
// 64 + 8 heads on a prefix of 32768 keys and 128 to 2048 of their own: 7, 84
// and 8 us, 109 to 110 us in all.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace mxsa {

namespace {

constexpr int kHMaxSeqs = 1024;
constexpr int kHMaxCtas = 160;     // workspaces are sized for this many
// Costs, in units of about 0.2 us: one block of a tile of two halves, of one
// half (whose halves then split the blocks), and a tile's own (its q, the
// first block's latency, the epilogue).  They set the chunks and how many
// CTAs begin with which queue.
constexpr int kHCostRows = 8, kHCostKeys = 4, kHCostTile = 10;
constexpr int kHCostRatio = (kHCostRows + kHCostKeys - 1) / kHCostKeys;
// A CTA's share of all work is kHPerCta chunks (3, or a column's end cut finer
// so that the CTAs end together: more partial rows, and slower); a share of at
// most kHOneChunk blocks is one.
constexpr int kHPerCta = 2, kHOneChunk = 24;

// One tile: keys [128 blk0, 128 (blk0 + nblk)) of [lo, hi) for ntok tokens.
struct alignas(16) HTile {
  int32_t tok0, ntok, g, row;      // first token, tokens, kv head, block table row
  int32_t lo, hi, blk0, nblk;
  long long part0;                 // first partial row
  int32_t keys;                    // 0: two halves; else one half, the groups take alternate blocks, and its rows
                                   // stand this often in the MMA's (see copies_of)
  int32_t pad;
};

// What the join needs of a tile: its rows' partials and how many of each (two
// where the groups took alternate blocks, the second `ntok` tokens on).
struct alignas(16) HPieces {
  int32_t part0, tok0, ntok, pieces;
};

struct HJob {
  int32_t tok0, ntok, row, lo, hi;
  int32_t tile0;                   // first tile
  int32_t nch, chunk, nrt;         // chunks, blocks of one, row tiles
};

// A token: its sequence (-1: none), the keys it sees, and the tiles of its
// sequence's own keys and of its group's prefix: for kv head g and chunk c <
// nch, number base + (g * nch + c) * nrt.
struct alignas(16) HTok {
  int32_t seq, keys, own_base, own_nch;
  int32_t own_nrt, pre_base, pre_nch, pre_nrt;
};

// The queues: 0 tiles of two halves, 1 of one half.
struct HHeader {
  int32_t count[2];                // tiles
  int32_t next[2];                 // places taken; the first `ctas` of a queue go to the CTAs that begin with it
  int32_t ctas[2];
};

struct HPtrs {
  HHeader* hdr;
  HTok* tok;                       // [total_q]
  HPieces* pieces;                 // by tile number
  HTile* queue[2];
  float* part_o;
  float* part_lse;                 // log2 units
};

struct HLayout {
  size_t hdr, tok, pieces, queue, part_o, part_lse, total;
  long long tile_cap, row_cap;
  int join_cap;  // partials of one row
};

HLayout shared_layout(const mxsa_problem& p) {
  const long long G = p.num_q_heads / p.num_kv_heads, T = 128 / G;
  // (job, kv head, row tile) triples: each token lies in at most two jobs, a
  // job's last row tile may be short, and there are at most B + B / 2 jobs
  const long long triples = p.num_kv_heads * (2 * (p.total_q / (2 * T)) + 2LL * p.num_seqs);
  // Chunks beyond the first.  A job's chunk is at least 1 / kHPerCta of a
  // CTA's share of the whole cost, in blocks of two halves' cost where the
  // job has such tiles; a tile of one half then costs kHCostRatio less.  A
  // column of x chunks is cut into at most x + 1/2 and no more than there are
  // blocks.  A kv head has its share.
  const long long blocks = max_blocks_per_seq(p);
  const long long by_cost = (long long)kHPerCta * kHCostRatio * kHMaxCtas;
  const long long extra = std::min(by_cost, triples * (blocks - 1));
  HLayout L;
  L.tile_cap = triples + extra;
  // A row in each of its token's jobs (a prefix needs a second sequence), its
  // twin in a job's last row tile where that is of one half (halves that split
  // the blocks, at most T tokens); a further chunk's tile has at most 256
  // rows, twins counted.
  const long long rows = (long long)p.total_q * G, in_jobs = (p.num_seqs > 1 ? 2 : 1) * rows;
  const long long jobs = p.num_seqs + p.num_seqs / 2;
  L.row_cap = p.num_kv_heads * (in_jobs + std::min(in_jobs, jobs * T * G)) + std::min(256LL, 2 * rows) * extra;
  L.join_cap = (int)(2 * std::min(2 + by_cost / p.num_kv_heads, 2 * blocks + 2));
  size_t o = 0;
  auto take = [&o](size_t n) {
    const size_t at = o;
    o = (o + n + 255) / 256 * 256;
    return at;
  };
  L.hdr = take(sizeof(HHeader));
  L.tok = take(sizeof(HTok) * (size_t)p.total_q);
  L.pieces = take(sizeof(HPieces) * L.tile_cap);
  L.queue = take(2 * sizeof(HTile) * L.tile_cap);
  L.part_o = take(512ull * L.row_cap);
  L.part_lse = take(4ull * L.row_cap);
  L.total = o;
  return L;
}

HPtrs shared_ptrs(const HLayout& L, void* ws) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  HPtrs x;
  x.hdr = reinterpret_cast<HHeader*>(b + L.hdr);
  x.tok = reinterpret_cast<HTok*>(b + L.tok);
  x.pieces = reinterpret_cast<HPieces*>(b + L.pieces);
  x.queue[0] = reinterpret_cast<HTile*>(b + L.queue);
  x.queue[1] = x.queue[0] + L.tile_cap;
  x.part_o = reinterpret_cast<float*>(b + L.part_o);
  x.part_lse = reinterpret_cast<float*>(b + L.part_lse);
  return x;
}

// How often a one-half tile's q rows stand in its 128 MMA rows: few rows (of
// few tokens, whose q is loaded token by token) stand there four times or
// twice, 32 or 64 rows apart, and each copy's warps take a quarter or half of
// every block's keys.
constexpr int kHSmallQ = 8;
__device__ __forceinline__ int copies_of(int ntok, int G) {
  return ntok > kHSmallQ || ntok * G > 64 ? 1 : (ntok * G > 32 ? 2 : 4);
}

__device__ __forceinline__ long long ceil_div(long long x, int y) {
  return x < INT_MAX - 4096 ? (uint32_t)(x + y - 1) / (uint32_t)y : (x + y - 1) / y;
}

// ------------------------------------------------------------------- plan
struct HPlanArgs {
  const int64_t* cu;
  const int32_t* lens;
  const int32_t* group_ptr;
  const int32_t* prefix_lens;
  int32_t* flags;  // may be null
  HPtrs ws;
  long long tile_cap;
  int32_t num_seqs, num_groups, total_q, Hkv, G, T, max_len, causal, ctas;
};

// One CTA that the forward waits for: few barriers, and what a thread does
// per tile kept short.  256 threads: 512 and 1024 take up to 2 us longer with
// few sequences and are not faster with 256.
constexpr int kHPlanThreads = 256;

struct HPlanSmem {
  int32_t cu[kHMaxSeqs + 1], len[kHMaxSeqs], seq_group[kHMaxSeqs];
  int32_t gp[kHMaxSeqs + 1], want[kHMaxSeqs], shortest[kHMaxSeqs];
  int32_t tile0[2 * kHMaxSeqs];
  HJob job[2 * kHMaxSeqs];
  long long scan[5][kHPlanThreads / 32];
};

// Exclusive sums over the block of kN values at once; total gets the wholes.
// `s`: kN words per warp, not used by another call of the launch.
template <int kN>
__device__ __forceinline__ void block_scan(long long (&v)[kN], long long* s, long long (&total)[kN]) {
  constexpr int kWarps = kHPlanThreads / 32;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long x[kN], y[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const long long z = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += z;
    }
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i * kWarps + w] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) y[i] = s[i * kWarps + (lane & (kWarps - 1))];
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const long long z = __shfl_up_sync(0xffffffffu, y[i], o);
      if ((lane & (kWarps - 1)) >= o) y[i] += z;
    }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const long long before = __shfl_sync(0xffffffffu, y[i], max(w - 1, 0));
    total[i] = __shfl_sync(0xffffffffu, y[i], kWarps - 1);
    v[i] = x[i] - v[i] + (w ? before : 0);
  }
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

// A place in the line of tiles: row tile fastest, then chunk, kv head, job.
struct HCursor {
  int q, g, ch, rt;
};

__global__ void __launch_bounds__(kHPlanThreads) k_shared_plan(HPlanArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  HPlanSmem& s = *reinterpret_cast<HPlanSmem*>(smem_raw);
  const int tid = threadIdx.x, B = a.num_seqs, NG = a.num_groups;
  pdl_launch_dependents();
  pdl_wait();

  int bad = 0;  // status bits
  for (int i = tid; i <= B; i += kHPlanThreads) {  // (NG <= B; no groups: the pointers may be null)
    // everything is on its way before anything is looked at
    const long long v = a.cu[i], nx = i < B ? a.cu[i + 1] : a.total_q;
    const int L = i < B ? a.lens[i] : 0;
    const int gv = NG > 0 && i <= NG ? a.group_ptr[i] : 0, gn = i < NG ? a.group_ptr[i + 1] : B;
    const int want = i < NG ? a.prefix_lens[i] : 0;
    if (v < 0 || v > nx) bad |= MXSA_FLAG_CU;
    s.cu[i] = (int)v;
    if (i < B) {
      if (L < 0 || L > a.max_len) bad |= MXSA_FLAG_LEN;
      s.len[i] = min(max(L, 0), a.max_len);
      s.seq_group[i] = -1;
    }
    if (NG > 0 && i <= NG) {
      if (gv < 0 || gv > gn) bad |= MXSA_FLAG_GROUP;
      s.gp[i] = gv;
      if (i < NG) {
        s.want[i] = want;
        s.shortest[i] = a.max_len;
      }
    }
  }
  const bool cu_ok = !__syncthreads_or(bad & MXSA_FLAG_CU), gp_ok = !__syncthreads_or(bad & MXSA_FLAG_GROUP);
  if (bad && a.flags) atomicOr(a.flags, bad);
  if (!cu_ok) {  // no sequence has tokens: no tile, no row
    for (int t = tid; t < a.total_q; t += kHPlanThreads) a.ws.tok[t] = HTok{-1, 0, 0, 0, 0, 0, 0, 0};
    if (tid == 0) *a.ws.hdr = HHeader{{0, 0}, {0, 0}, {a.ctas, 0}};
    return;
  }
  // a group's prefix is at most its shortest sequence with tokens
  if (gp_ok && NG > 0)
    for (int i = tid; i < B; i += kHPlanThreads) {
      if (i < s.gp[0] || i >= s.gp[NG]) continue;
      const int j = last_le(s.gp, NG + 1, i);
      if (s.gp[j + 1] - s.gp[j] < 2) continue;  // one sequence alone shares nothing
      s.seq_group[i] = j;
      if (s.cu[i + 1] > s.cu[i]) atomicMin(&s.shortest[j], s.len[i]);
    }
  __syncthreads();
  auto prefix_of = [&](int j) {  // 0: no prefix (also for the group number -1)
    return j >= 0 && gp_ok && s.gp[j + 1] - s.gp[j] >= 2 ? min(max(s.want[j], 0), s.shortest[j]) : 0;
  };

  // Jobs: the groups' prefixes, whose tiles are the longest and go first, then
  // the sequences' own keys.  A thread's jobs are consecutive, and its tiles
  // below.
  const int njobs = B + NG, T2 = 2 * a.T;
  const int jper = (njobs + kHPlanThreads - 1) / kHPlanThreads;
  const int q0 = min(njobs, tid * jper), q1 = min(njobs, q0 + jper);
  long long cost[2] = {0, 0}, total[2];  // of the two kinds of tiles
  for (int q = q0; q < q1; ++q) {
    HJob j;
    if (q < NG) {
      const int P = prefix_of(q);
      j.row = P > 0 ? s.gp[q] : 0;
      j.tok0 = P > 0 ? s.cu[s.gp[q]] : 0;
      j.ntok = P > 0 ? s.cu[s.gp[q + 1]] - j.tok0 : 0;
      j.lo = 0;
      j.hi = P;
    } else {
      const int r = q - NG;
      j.tok0 = s.cu[r];
      j.ntok = s.cu[r + 1] - s.cu[r];
      j.row = r;
      j.lo = prefix_of(s.seq_group[r]);
      j.hi = s.len[r];
    }
    const int nb = j.ntok > 0 && j.hi > j.lo ? ((j.hi + 127) >> 7) - (j.lo >> 7) : 0;
    const int rem = j.ntok % T2;
    const int keys = rem > 0 && rem <= a.T;
    j.nrt = nb > 0 ? (j.ntok + T2 - 1) / T2 : 0;
    j.chunk = j.nrt > keys;  // for now: whether tiles of two halves set the chunk
    j.nch = nb;
    // (as far as it is known without causal trimming)
    if (nb > 0) {
      cost[0] += (long long)a.Hkv * (j.nrt - keys) * (nb * kHCostRows + kHCostTile);
      cost[1] += (long long)a.Hkv * keys * (nb * kHCostKeys + kHCostTile);
    }
    s.job[q] = j;
  }
  block_scan<2>(cost, s.scan[0], total);
  const long long share = max(ceil_div(total[0] + total[1], a.ctas), 1LL);
  long long tiles[1] = {0}, all[1];
  for (int q = q0; q < q1; ++q) {
    HJob& j = s.job[q];
    const int nb = j.nch;
    const long long whole =
        j.chunk ? (share + kHCostRows - 1) / kHCostRows : (share + kHCostKeys - 1) / kHCostKeys;
    const int want = (int)min(whole <= kHOneChunk ? whole : (whole + kHPerCta - 1) / kHPerCta, (long long)max(nb, 1));
    j.nch = nb > 0 ? max((nb + want / 2) / want, 1) : 0;  // of one size, the nearest number of them
    j.chunk = nb > 0 ? (nb + j.nch - 1) / j.nch : 1;
    tiles[0] += (long long)a.Hkv * j.nch * j.nrt;
  }
  block_scan<1>(tiles, s.scan[2], all);
  long long at = tiles[0];
  for (int q = q0; q < q1; ++q) {
    HJob& j = s.job[q];
    j.tile0 = (int)at;
    s.tile0[q] = (int)at;
    at += (long long)a.Hkv * j.nch * j.nrt;
  }
  const int ntiles = (int)min(all[0], a.tile_cap);  // (all is within the cap: see shared_layout)
  __syncthreads();

  const int tper = (ntiles + kHPlanThreads - 1) / kHPlanThreads;
  const int i0 = min(ntiles, tid * tper), i1 = min(ntiles, i0 + tper);
  HCursor c0{0, 0, 0, 0};
  if (i0 < i1) {
    c0.q = last_le(s.tile0, njobs, i0);
    const HJob& j = s.job[c0.q];
    const int rel = i0 - j.tile0, x = rel / j.nrt;
    c0.rt = rel - x * j.nrt;
    c0.g = x / j.nch;
    c0.ch = x - c0.g * j.nch;
  }
  auto advance = [&](HCursor* c) {
    const HJob* j = &s.job[c->q];
    if (++c->rt < j->nrt) return;
    c->rt = 0;
    if (++c->ch < j->nch) return;
    c->ch = 0;
    if (++c->g < a.Hkv) return;
    c->g = 0;
    do ++c->q;
    while (c->q < njobs && s.job[c->q].nrt == 0);
  };
  // blocks and tokens of the tile at c
  auto size_of = [&](const HCursor& c, int* blk0, int* nblk, int* ntok) {
    const HJob& j = s.job[c.q];
    *ntok = min(T2, j.ntok - c.rt * T2);
    int end = (j.hi + 127) >> 7;
    if (a.causal && c.q >= NG)  // keys past the last token's position are nobody's
      end = min(end, (max(j.hi - j.ntok + c.rt * T2 + *ntok, 0) + 127) >> 7);
    *blk0 = (j.lo >> 7) + c.ch * j.chunk;
    *nblk = max(min(*blk0 + j.chunk, end) - *blk0, 0);
  };
  // tiles of each queue (in one word) and partial rows before the thread's own
  long long sums[2] = {0, 0}, wholes[2];
  int blk0, nblk, ntok;
  HCursor c = c0;
  for (int i = i0; i < i1; ++i, advance(&c)) {
    size_of(c, &blk0, &nblk, &ntok);
    const bool keys = ntok <= a.T;
    if (nblk) {
      sums[0] += keys ? 1LL << 32 : 1LL;
      sums[1] += ntok * a.G * (keys ? 2 : 1);
    }
  }
  block_scan<2>(sums, s.scan[3], wholes);
  long long place = sums[0], part = sums[1];
  c = c0;
  for (int i = i0; i < i1; ++i, advance(&c)) {
    size_of(c, &blk0, &nblk, &ntok);
    const HJob& j = s.job[c.q];
    const bool keys = ntok <= a.T;
    HTile t;
    t.tok0 = j.tok0 + c.rt * T2;
    t.ntok = ntok;
    t.g = c.g;
    t.row = j.row;
    t.lo = j.lo;
    t.hi = j.hi;
    t.blk0 = blk0;
    t.nblk = nblk;
    t.part0 = part;
    t.keys = keys ? copies_of(ntok, a.G) : 0;
    t.pad = 0;
    a.ws.pieces[i] = HPieces{(int)part, t.tok0, ntok, keys ? min(nblk, 2) : min(nblk, 1)};  // (rows fit 32 bits)
    if (nblk) {
      part += ntok * a.G * (keys ? 2 : 1);
      a.ws.queue[keys][keys ? place >> 32 : (int)place] = t;
      place += keys ? 1LL << 32 : 1LL;
    }
  }
  for (int i = tid; i < a.total_q; i += kHPlanThreads) {
    HTok v{-1, 0, 0, 0, 0, 0, 0, 0};
    if (i >= s.cu[0] && i < s.cu[B]) {
      const int q = last_le(s.cu, B, i), L = s.len[q];
      v.seq = q;
      v.keys = a.causal ? min(max(L - (s.cu[q + 1] - i) + 1, 0), L) : L;
      const HJob& own = s.job[NG + q];
      if (own.nrt > 0) {
        v.own_base = own.tile0 + (i - own.tok0) / T2;
        v.own_nch = own.nch;
        v.own_nrt = own.nrt;
      }
      if (prefix_of(s.seq_group[q]) > 0) {
        const HJob& pre = s.job[s.seq_group[q]];
        v.pre_base = pre.tile0 + (i - pre.tok0) / T2;
        v.pre_nch = pre.nch;
        v.pre_nrt = pre.nrt;
      }
    }
    a.ws.tok[i] = v;
  }
  if (tid == 0) {
    const int n0 = (int)wholes[0], n1 = (int)(wholes[0] >> 32);
    // (5/8 of the share: the second kind's smaller tiles fill up the end)
    int with1 = (int)(total[1] * a.ctas * 5 / 8 / max(total[0] + total[1], 1LL));
    with1 = n1 == 0 ? 0 : (n0 == 0 ? a.ctas : min(max(with1, 1), a.ctas - 1));
    *a.ws.hdr = HHeader{{n0, n1}, {a.ctas - with1, with1}, {a.ctas - with1, with1}};
  }
}

// ---------------------------------------------------------------- forward
// 384 threads: two softmax groups (warps 0-3 and 4-7; thread = TMEM lane =
// row), a producer, two MMA issuers and a scheduler (a warp each).  A tile of
// two halves gives each group its own 128 rows over the same blocks; a tile of
// one half gives both groups the same rows and alternate blocks (each then
// makes a partial of its own).  Per block: S = q k^T (TMEM), a lazily raised
// running maximum (raised when a score passes it by 2^8, O in TMEM is then
// rescaled), P = exp2(S - m) rounded to the 16-bit type over S, l += sum P,
// O += P V.  Each group has an issuer: P V of a block, then q k^T of the
// group's next one, so that while one group runs its softmax the tensor pipe
// has the other's two products.  S is overwritten by the MMA after the one
// that reads P from it; both are issued by one thread, which the pipe keeps in
// order.  K and V blocks have a stage of 32 KB each in a ring of five, in the
// order in which the issuer takes them (K0 K1 V0 K2 V1 ... ), so 160 KB of
// loads are in flight when the CTA waits for memory.  What waits for global
// memory otherwise (claims, records, pages) is the scheduler's: in the
// producer's way it cost 1900 cycles a block of a decode tile.
//
// Bound.  Tiles of two halves: a group's chain of softmax (1650 cycles a
// block: 500 for the maximum, 16 a pair of exponentials), two hand-overs
// (250 and 300) and its products; the tensor pipe's own 2176 cycles of both
// groups' four products are 0.7 of it.  256 decoding sequences of 64 + 8
// heads on a shared prefix of 65536 keys and 64 to 2048 of their own (558
// GFLOP, 1.36 GB): 525 to 543 us in all on different GPUs, 1.03 to 1.06
// PFLOP/s.  Tiles of one half: memory; 256 sequences with 2048 keys of their
// own and no prefix (2.16 GB): 332 us, 6.5 TB/s.  Code that is run once or
// rarely is kept in loops: unrolled, its first use in a launch costs 3 to 4 us
// of instruction fetches.
constexpr int kHThreads = 384;
constexpr int kHProducer = 8, kHMma = 9, kHSched = 11;
constexpr uint32_t kHTileBytes = 32768;  // 128 rows x 128 x 16-bit
constexpr int kHStages = 5;
constexpr int kHWork = 4, kHWindows = 2, kHWindow = 3;
constexpr float kHRescale = 8.f;         // log2 units
constexpr uint32_t kHOffKV = 2 * kHTileBytes;
constexpr uint32_t kHOffCtrl = kHOffKV + kHStages * kHTileBytes;

// Some blocks of a tile, from the scheduler to the producer: the pages' third
// coordinates (two a block; -1: none).  No blocks: the end.
struct alignas(16) HWindow {
  int2 z[kHWindow];
  int32_t n, first, last;  // blocks; whether they are their tile's first and last ones
};

// A role may pass over places and q slots of the other group without looking
// at their barriers.  A parity only tells a phase from the one before, so a
// stage's (and a q buffer's) uses alternate between two "full" barriers: to
// mistake a phase a role would have to be two uses ahead of the copies, and
// each wait comes after one for a copy that was issued later than that.
struct HCtrl {
  uint64_t q_full[4], q_empty[2], kv_full[2 * kHStages], kv_empty[kHStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], turn[2], done;
  uint64_t work_full[kHWork], work_empty[kHWork];
  uint64_t win_full[kHWindows], win_empty[kHWindows];
  HTile work[kHWork];  // the CTA's tiles, from the scheduler to the issuers and the softmax; no blocks: the end
  HWindow win[kHWindows];
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

__device__ __forceinline__ HTile load_tile(const HTile* p) {
  HTile t;
  const int4* s = reinterpret_cast<const int4*>(p);
  int4* d = reinterpret_cast<int4*>(&t);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(HTile) / 16); ++i) d[i] = s[i];
  return t;
}

// ring places of a tile's blocks, relative to the tile's first: K0, K1,
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

// O of the thread's row times f, 16 columns at a time
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
#pragma unroll 1
  for (int cb = 0; cb < 8; ++cb) {
    uint32_t w[16];
    tmem_ld16(tO + cb * 16, w);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
    tmem_st16(tO + cb * 16, w);
  }
}

// S of the thread's row outside columns [lo, hi) to -infinity.  A pass of its
// own over S, in a loop: edges are few, and unrolled beside the block's other
// code they cost a launch 3 us of instruction fetches at its first edge.
__device__ __forceinline__ void mask_s(uint32_t tS, int lo, int hi) {
#pragma unroll 1
  for (int cb = 0; cb < 128; cb += 16) {
    uint32_t w[16];
    tmem_ld16(tS + cb, w);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) w[k] = cb + k >= lo && cb + k < hi ? w[k] : 0xFF800000u;
    tmem_st16(tS + cb, w);
  }
  tmem_st_wait();
}

// One block of a tile whose rows stand 128 / kKeys times in the MMA's: copy
// `copy` takes the keys kKeys x copy .. of the block, with a maximum and a sum
// of its own, and writes zeros as the other keys' weights.  A decode tile's
// 8 rows then cost a quarter of the time of one warp with 128 keys to a
// thread.
template <int kKeys, bool kBf16>
__device__ __forceinline__ void few_rows(uint32_t tS, int copy, int k0, int lo, int hi, int warp_hi, bool live,
                                         bool mine, float scale_log2, float* m, float* l) {
  float sv[kKeys];
#pragma unroll
  for (int q = 0; q < kKeys / 32; ++q) tmem_ld32(tS + copy * kKeys + q * 32, sv + q * 32);
  tmem_ld_wait();
  const int first = k0 + copy * kKeys;
  if (first < lo || first + kKeys > warp_hi) {
#pragma unroll
    for (int k = 0; k < kKeys; ++k) sv[k] = first + k >= lo && first + k < hi ? sv[k] : -INFINITY;
  }
  float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < kKeys; k += 4) {
    b0 = hmax3(b0, sv[k], sv[k + 1]);
    b1 = hmax3(b1, sv[k + 2], sv[k + 3]);
  }
  const float bm = fmaxf(b0, b1) * scale_log2;
  const bool raise = live && (bm > *m + kHRescale || (*m == -INFINITY && bm > -INFINITY));
  if (__any_sync(0xffffffffu, raise)) {
    const float f = raise ? (*m == -INFINITY ? 0.f : ex2_approx(*m - bm)) : 1.f;
    if (mine) scale_o(tS + 128, f);
    if (raise) {
      *l *= f;
      *m = bm;
    }
  }
  const float mm = *m == -INFINITY ? 0.f : *m;
  const uint64_t scale2 = pack_f2(scale_log2, scale_log2), off2 = pack_f2(-mm, -mm);
  uint64_t l0 = pack_f2(0.f, 0.f);
#pragma unroll
  for (int q = 0; q < kKeys / 32; ++q) {
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = unpack_f2(fma_f2(pack_f2(sv[32 * q + 2 * k], sv[32 * q + 2 * k + 1]), scale2, off2));
      const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
      l0 = add_f2(l0, pack_f2(p0, p1));
      pk[k] = hpack2<kBf16>(p0, p1);
    }
    tmem_st16(tS + (copy * kKeys + q * 32) / 2, pk);
  }
  const uint32_t none[16] = {};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (q / (kKeys / 32) != copy) tmem_st16(tS + 16 * q, none);
  const float2 ls = unpack_f2(l0);
  *l += ls.x + ls.y;
}

// Barrier of softmax group h's four warps.  A named one knows no limit, so a
// warp that gave up, or leaves after another role did, arrives once as it goes:
// the others are let through, see the abort flag and leave too (false).  An
// mbarrier, whose waits have a limit of their own, cost the 64 decoding
// sequences' call 1 to 3 us of 110.
__device__ __forceinline__ bool group_sync(int h, volatile int* abort_flag) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory");
  return hwarp_all(*abort_flag == 0);
}
__device__ __forceinline__ void group_leave(int h, volatile int* abort_flag) {
  if (!hwarp_all(*abort_flag == 0)) asm volatile("bar.arrive %0, 128;" ::"r"(1 + h) : "memory");
}

// The partial rows of a tile with copies: the copies' sums join over shared
// memory (32 KB at `mem`, the stage of the group's last V), 64 columns at a
// time, 16-byte pieces of a row at places that change with the row.  False
// when a wait gave up.
__device__ __forceinline__ bool join_copies(uint32_t mem, uint32_t tO, int h, volatile int* abort_flag, int r, int row,
                                            int copy, int copies, int rows, bool live, float m, float l,
                                            float* part_o, float* part_lse) {
  const int apart = 128 / copies;
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(mem + r * 8), "f"(m), "f"(l) : "memory");
  if (!group_sync(h, abort_flag)) return false;
  float mq[4], lq[4], M = -INFINITY, L = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    mq[q] = -INFINITY;
    lq[q] = 0.f;
    if (q < copies) {
      const uint2 v = ld_shared_v2(mem + (q * apart + row) * 8);
      mq[q] = __uint_as_float(v.x);
      lq[q] = __uint_as_float(v.y);
    }
    M = fmaxf(M, mq[q]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) L += lq[q] * (M == -INFINITY ? 1.f : ex2_approx(mq[q] - M));  // (a NaN stays one)
  const float f = L == 0.f ? 0.f : (M == -INFINITY ? 1.f : ex2_approx(m - M)) / L;
  if (live && copy == 0) part_lse[row] = L == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) + lg2_approx(L);
  if (!group_sync(h, abort_flag)) return false;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float ov[32];
      tmem_ld32(tO + pass * 64 + cb * 32, ov);  // every lane: the load is warp-collective
      tmem_ld_wait();
      if (live)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_shared_v4(mem + r * 256 + (((cb * 8 + k) ^ (r & 15)) << 4), __float_as_uint(ov[4 * k] * f),
                       __float_as_uint(ov[4 * k + 1] * f), __float_as_uint(ov[4 * k + 2] * f),
                       __float_as_uint(ov[4 * k + 3] * f));
    }
    if (!group_sync(h, abort_flag)) return false;
    for (int x = r; x < rows * 16; x += 128) {
      const int rr = x >> 4, c4 = x & 15;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int q = 0; q < copies; ++q) {
        const int at = q * apart + rr;
        const uint4 v = ld_shared_v4(mem + at * 256 + ((c4 ^ (at & 15)) << 4));
        sum.x += __uint_as_float(v.x);
        sum.y += __uint_as_float(v.y);
        sum.z += __uint_as_float(v.z);
        sum.w += __uint_as_float(v.w);
      }
      *reinterpret_cast<float4*>(part_o + rr * 128 + pass * 64 + c4 * 4) = sum;
    }
    fence_proxy_async_smem();  // the stage's next copy comes after what was done here
    if (!group_sync(h, abort_flag)) return false;
  }
  return true;
}

#ifdef MXSA_TEST_HOOKS
// Test builds only: CTA g_skip_window keeps its first window of pages to
// itself, so that every role's next wait runs out.
__device__ int g_skip_window = -1;
#endif

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
    for (int i = 0; i < kHWork; ++i) {
      mbar_init(&c.work_full[i], 1);
      mbar_init(&c.work_empty[i], 10);  // the issuers' and the softmax groups' warps
    }
    for (int i = 0; i < kHWindows; ++i) {
      mbar_init(&c.win_full[i], 1);
      mbar_init(&c.win_empty[i], 1);
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
  // The next tile of a role that is not the producer; false at the end (or
  // when a wait gave up).
  int taken = 0;
  auto next_tile = [&](HTile* t) {
    const int w = taken % kHWork;
    if (!hwarp_all(mbar_wait(&c.work_full[w], (taken / kHWork) & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs)))
      return false;
    *t = c.work[w];
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.work_empty[w]);
    ++taken;
    return t->nblk > 0;
  };

  if (warp >= 8) {
    if (warp == kHProducer) {
      // -------------------------------------------------------------- producer
      // One lane that only waits for stages and issues copies: a block takes
      // it less than the copies take to land, so the ring stays full.
      if (lane == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        const uint32_t page_bytes = 256u << a.page_shift;
        int at = 0, st = 0, full = 0;  // ring places taken; the next one's stage and full barrier
        uint32_t parity = 1;
        auto load = [&](const CUtensorMap* tm, int2 z) {
          if (!mbar_wait(&c.kv_empty[st], parity, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs)) return false;
          uint64_t* bar = &c.kv_full[full];
          uint8_t* dst = sm + kHOffKV + st * kHTileBytes;
          mbar_arrive_expect_tx(bar, (uint32_t)((z.x >= 0) + (z.y >= 0)) * page_bytes);
          if (z.x >= 0) {
            tma_load_3d(dst, tm, bar, 0, 0, z.x);
            tma_load_3d(dst + 16384, tm, bar, 64, 0, z.x);
          }
          if (z.y >= 0) {
            tma_load_3d(dst + 8192, tm, bar, 0, 0, z.y);
            tma_load_3d(dst + 16384 + 8192, tm, bar, 64, 0, z.y);
          }
          ++at;
          if (++st == kHStages) st = 0, parity ^= 1;
          if (++full == 2 * kHStages) full = 0;
          return true;
        };
        int2 prev = make_int2(-1, -1);
        bool ok = true;
        for (int w = 0; ok; ++w) {
          const int x = w % kHWindows;
          if (!mbar_wait(&c.win_full[x], (w / kHWindows) & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs)) break;
          const int n = c.win[x].n, first = c.win[x].first, last = c.win[x].last;
          if (n == 0) break;
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i) {  // K of a block, then V of the one before: the ring's order
            const int2 z = c.win[x].z[i];
            if (i == n - 1) mbar_arrive(&c.win_empty[x]);
            ok = load(&tmk, z);
            if (ok && (i > 0 || !first)) ok = load(&tmv, prev);
            prev = z;
          }
          if (ok && last) ok = load(&tmv, prev);
        }
        // drain: the copies in flight land before the CTA may exit
        for (int k = max(0, at - kHStages); k < at; ++k)
          mbar_drain(&c.kv_full[k % (2 * kHStages)], (k / (2 * kHStages)) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      }
      __syncwarp();
    } else if (warp == kHSched) {
      // ------------------------------------------------------------- scheduler
      // Claims tiles, hands them to the other roles, looks up their pages and
      // loads q: what waits for global memory, and would keep the producer
      // from its copies.
      if (lane == 0) {
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmq1);
      }
      const int ps = 1 << a.page_shift, npg = ps == 128 ? 1 : 2;
      int qn = 0;  // q buffers filled
      bool ok = true;
      // The CTA's queue: the second kind's CTAs are spread over the grid.
      const int with1 = a.ws.hdr->ctas[1], count[2] = {a.ws.hdr->count[0], a.ws.hdr->count[1]};
      const int before1 = (int)((long long)cta * with1 / gridDim.x);
      int q = (int)((long long)(cta + 1) * with1 / gridDim.x) - before1;
      bool other = false;          // the queue it began with is empty
      auto claim = [&]() -> int {  // lane 0: a place of queue q (none is left behind the CTAs' own: no atomic)
        return (q ? count[1] <= with1 : count[0] <= (int)gridDim.x - with1) ? INT_MAX
                                                                            : atomicAdd(&a.ws.hdr->next[q], 1);
      };
      auto resolve = [&](int place) {  // the tile at a place of queue q, or of the other queue; no blocks: none left
        place = __shfl_sync(0xffffffffu, place, 0);
        if (place >= (q ? count[1] : count[0]) && !other) {
          other = true;
          q ^= 1;
          if (lane == 0) place = claim();
          place = __shfl_sync(0xffffffffu, place, 0);
        }
        return place >= (q ? count[1] : count[0]) ? HTile{} : load_tile((q ? a.ws.queue[1] : a.ws.queue[0]) + place);
      };
      // A window's pages, one to a lane: page lane % 2 of block i + lane / 2,
      // where the window holds it and it has keys of the tile.
      auto needed = [&](const HTile& t, int i, int n) {
        const int k = i + (lane >> 1), p0 = (t.blk0 + k) * 128 + (lane & 1) * 64;
        return (lane >> 1) < n && k < t.nblk && (lane & 1) < npg && p0 < t.hi && p0 + ps > t.lo;
      };
      auto page_of = [&](const HTile& t, int i, int n) {
        const int p0 = (t.blk0 + i + (lane >> 1)) * 128 + (lane & 1) * 64;
        return needed(t, i, n) ? a.block_tables[(size_t)t.row * a.max_pages + (p0 >> a.page_shift)] : -1;
      };
      auto load_q = [&](const HTile& t) {
        const int nh = t.keys ? 1 : 2;
        for (int h = 0; h < nh && ok; ++h, ++qn) {
          const int b = qn & 1;
          ok = hwarp_all(
              mbar_wait(&c.q_empty[b], ((qn >> 1) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
          if (!ok) break;
          uint8_t* qd = sm + b * kHTileBytes;
          uint64_t* full = &c.q_full[qn & 3];
          const int t0 = t.tok0 + h * a.T, nt = min(a.T, t.ntok - h * a.T);
          if (nt > kHSmallQ) {  // one box; rows past the tile's tokens are never used
            if (lane == 0) {
              mbar_arrive_expect_tx(full, (uint32_t)(G * a.T) * 256u);
              tma_load_3d(qd, &tmq, full, 0, t.g * G, t0);
              tma_load_3d(qd + 16384, &tmq, full, 64, t.g * G, t0);
            }
          } else {  // token by token, each copy of the rows
            const int copies = max(t.keys, 1), apart = 128 / copies;
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(G * nt * copies) * 256u);
            __syncwarp();
            for (int x = lane; x < nt * copies * 2; x += 32) {
              const int col = x & 1, cp = (x >> 1) % copies, tk = (x >> 1) / copies;
              tma_load_3d(qd + col * 16384 + (cp * apart + tk * G) * 128, &tmq1, full, col * 64, t.g * G, t0 + tk);
            }
          }
        }
      };
      int wn = 0;  // windows handed over
      auto window_free = [&] {
        ok = ok && hwarp_all(mbar_wait(&c.win_empty[wn % kHWindows], ((wn / kHWindows) & 1) ^ 1, abort_flag, fl,
                                       MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      };
      HTile t = resolve(q ? before1 : cta - before1);  // the first place is the CTA's own
      for (int n = 0; ok; ++n) {
        // windows: a short one first, so that the last one gives the next
        // tile's claim and look-ups time
        int k = 0, size = t.nblk ? (t.nblk - 1) % kHWindow + 1 : 0;
        int page = page_of(t, 0, size), ahead = page_of(t, size, kHWindow);  // of this window, of the next
        const int w = n % kHWork;
        ok = hwarp_all(
            mbar_wait(&c.work_empty[w], ((n / kHWork) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
        if (!ok) break;
        if (lane == 0) {
          c.work[w] = t;
          mbar_arrive(&c.work_full[w]);
        }
        do {
          window_free();
          if (!ok) break;
          HWindow& x = c.win[wn % kHWindows];
          if (lane < 2 * kHWindow) {
            const bool want = needed(t, k, size), there = page >= 0 && page < a.num_pages;
            if (want && !there) atomicOr(fl, MXSA_FLAG_PAGE);
            reinterpret_cast<int32_t*>(x.z)[lane] = want && there ? page * a.Hkv + t.g : -1;
          }
          if (lane == 0) {
            x.n = size;
            x.first = k == 0;
            x.last = k + size >= t.nblk;
          }
          __syncwarp();
#ifdef MXSA_TEST_HOOKS
          const bool skip = cta == g_skip_window && wn == 0;
#else
          constexpr bool skip = false;
#endif
          if (lane == 0 && !skip) mbar_arrive(&c.win_full[wn % kHWindows]);
          ++wn;
          k += size;
          page = ahead;
          if (k + kHWindow < t.nblk) ahead = page_of(t, k + kHWindow, kHWindow);
          // (the first keys are on their way before the q buffers are waited for)
          if (k == size && size) load_q(t);
          size = kHWindow;
        } while (k < t.nblk && ok);
        if (t.nblk == 0 || !ok) break;
        // The next tile is claimed when the producer comes to this one's last
        // window, not sooner: a claimed tile waits for this CTA.
        window_free();
        if (!ok) break;
        int place = 0;
        if (lane == 0) place = claim();
        t = resolve(place);
      }
      if (lane == 0)  // drain
        for (int k = max(0, qn - 2); k < qn; ++k)
          mbar_drain(&c.q_full[k & 3], (k >> 2) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
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
                                    // 2: no other group reads V, 3: the softmax frees V
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
        if (!(bits & 8)) {
          mma_commit(empty);
          if (bits & 4) mma_commit(empty);
        }
        if (bits & 2) mma_commit(&c.o_full[h]);
      };
      auto done_pv = [&] {
        ++np;
        no += (bits >> 1) & 1;
        owed = -1;
      };
      const uint32_t tS = uniform(tmem + h * 256);
      HTile t;
      while (ok && next_tile(&t)) {
        const int n = t.nblk, keys = t.keys, stride = keys ? 2 : 1;
        const int half = keys ? h ^ (qn & 1) : 0;  // (see the softmax)
        const int qp = keys ? qn : qn + h;
        for (int i = half; i < n && ok; i += stride) {
          const int kp = at + place_k(i), st = kp % kHStages;
          const int sv = max(owed, 0) % kHStages;
          const uint32_t dv = uniform(desc_mn_major(sbase + kHOffKV + sv * kHTileBytes));
          const uint32_t dq = uniform(desc_k_major(sbase + (qp & 1) * kHTileBytes));
          const uint32_t dk = uniform(desc_k_major(sbase + kHOffKV + st * kHTileBytes));
          if (owed >= 0) wait_v();
          // P V alone when K (or a new tile's q) may not be there yet
          const bool alone =
              i == half || !hwarp_all(mbar_test(&c.kv_full[kp % (2 * kHStages)], (kp / (2 * kHStages)) & 1));
          // In a tile of two halves the groups take turns at the pipe: left
          // alone they can fall into step, both in their softmax at once and
          // then both waiting for each other's products.
          if (!keys) {
            if (h == 1 || nt > 0) wait(&c.turn[h], (nt + h + 1) & 1);
            ++nt;
          }
          if (!ok) break;
          if (owed >= 0) {
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
            if (!keys) mbar_arrive(&c.turn[h ^ 1]);
            // (two arrivals free a stage or a q buffer: one of each group, or both of the only one)
            mma_commit(&c.kv_empty[st]);
            if (keys) mma_commit(&c.kv_empty[st]);
            if (last) mma_commit(&c.q_empty[qp & 1]);
            if (last && !keys) mma_commit(&c.q_empty[qp & 1]);
          }
          __syncwarp();
          if (owed >= 0) done_pv();
          owed = at + place_v(i, n);
          bits = (i == half ? 1 : 0) | (last ? 2 : 0) | (keys ? 4 : 0) | (last && keys > 1 ? 8 : 0);
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
    // --------------------------------------------------------------- softmax
    const int h = warp >> 2;
    const int r = tid & 127;  // row of the half == TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + h * 256 + lane_addr, tO = tS + 128;
    int at = 0, qn = 0, n_s = 0, n_o = 0;
    bool ok = true;
    HTile t;
    while (ok && next_tile(&t)) {
      // (what the block loop and the epilogue need of the tile, and no more)
      const int n = t.nblk, b0 = t.blk0, lo = t.lo, key_end = t.hi, keys = t.keys, stride = keys ? 2 : 1;
      // the group that takes a one-half tile's first block changes with the q
      // buffer, so that short tiles keep both groups busy
      const int half = keys ? h ^ (qn & 1) : 0;
      qn += keys ? 1 : 2;
      // the thread's row of the tile's (copies of a one-half tile's rows stand
      // `apart` rows apart) and its token within the tile
      const int apart = keys > 1 ? 128 / keys : 128;
      const int row = r & (apart - 1), copy = r / apart;
      const int rt = row / G, tt = rt + (keys ? 0 : h * a.T);
      const bool live = rt < a.T && tt < t.ntok;
      const long long rows = (long long)t.ntok * G;
      const long long base = t.part0 + half * rows, pr = base + tt * G + (row - rt * G);
      const bool warp_live = __any_sync(0xffffffffu, live);
      int hi = key_end;  // the row sees the keys [lo, hi), all of the warp's rows [lo, warp_hi)
      if (a.causal && live) hi = min(hi, a.ws.tok[t.tok0 + tt].keys);
      const int warp_hi = __reduce_min_sync(0xffffffffu, hi);
      float m = -INFINITY, l = 0.f;
      bool mine = false;  // this group has blocks of the tile
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
        if (keys > 1) {
          tc_fence_after();
          if (keys == 4)
            few_rows<32, kBf16>(tS, copy, k0, lo, hi, warp_hi, live, mine, a.scale_log2, &m, &l);
          else
            few_rows<64, kBf16>(tS, copy, k0, lo, hi, warp_hi, live, mine, a.scale_log2, &m, &l);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.p_half[h]);
        } else if (warp_live) {
          tc_fence_after();
          if (k0 < lo || k0 + 128 > warp_hi) mask_s(tS, lo - k0, hi - k0);
          // S 64 keys at a time, twice: the second ones and the first ones for
          // the maximum, then again the second ones for their exponentials.
          // A row's 128 scores at once would need registers that the other
          // warps then lack.
          float sv[64];
          float b0 = -INFINITY, b1 = -INFINITY, b2 = -INFINITY, b3 = -INFINITY;
#pragma unroll
          for (int hf = 1; hf >= 0; --hf) {
            tmem_ld32(tS + 64 * hf, sv);
            tmem_ld32(tS + 64 * hf + 32, sv + 32);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 64; k += 8) {
              b0 = hmax3(b0, sv[k], sv[k + 1]);
              b1 = hmax3(b1, sv[k + 2], sv[k + 3]);
              b2 = hmax3(b2, sv[k + 4], sv[k + 5]);
              b3 = hmax3(b3, sv[k + 6], sv[k + 7]);
            }
          }
          const float bm = fmaxf(fmaxf(b0, b1), fmaxf(b2, b3)) * a.scale_log2;
          const bool raise = live && (bm > m + kHRescale || (m == -INFINITY && bm > -INFINITY));
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? (m == -INFINITY ? 0.f : ex2_approx(m - bm)) : 1.f;
            if (mine) {
              // O holds the tile's blocks so far and is complete: S's
              // barrier follows every product issued before
              scale_o(tO, f);
            }
            if (raise) {
              l *= f;
              m = bm;
            }
          }
          const float mm = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = pack_f2(a.scale_log2, a.scale_log2), off2 = pack_f2(-mm, -mm);
          uint64_t l0 = pack_f2(0.f, 0.f), l1 = l0;
          // (a loop: its code is fetched once for both halves; unrolled over
          // 128 keys the warps stood without instructions, 275 us against 253
          // with 2048 rows per kv head on 32768 keys)
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float2 x = unpack_f2(fma_f2(pack_f2(sv[32 * q + 2 * k], sv[32 * q + 2 * k + 1]), scale2, off2));
                const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                if (k & 1) l1 = add_f2(l1, pack_f2(p0, p1));
                else l0 = add_f2(l0, pack_f2(p0, p1));
                pk[k] = hpack2<kBf16>(p0, p1);
              }
              tmem_st16(tS + 32 * hf + 16 * q, pk);
            }
            if (hf == 0) {  // the first 64 keys: their half of P V may start
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&c.p_half[h]);
              tmem_ld32(tS + 64, sv);
              tmem_ld32(tS + 96, sv + 32);
              tmem_ld_wait();
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
      at += 2 * n;
      if (!ok || !mine) continue;
      // ---- the tile's partial rows
      ok = hwarp_all(mbar_wait(&c.o_full[h], n_o & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      if (!ok) break;
      ++n_o;
      if (keys > 1) {
        tc_fence_after();
        const int pl = at - 2 * n + place_v(((n - 1 - half) & ~1) + half, n), st = pl % kHStages;  // its last block's V
        ok = join_copies(sbase + kHOffKV + st * kHTileBytes, tO, h, abort_flag, r, row, copy, keys, (int)rows, live, m,
                         l, a.ws.part_o + base * 128, a.ws.part_lse + base);
        if (!ok) break;
        if (r == 0) {
          mbar_arrive(&c.kv_empty[st]);
          mbar_arrive(&c.kv_empty[st]);
        }
      } else if (warp_live) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN stays one)
        float* po = a.ws.part_o + pr * 128;
#pragma unroll 1
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
    group_leave(h, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kHMma) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- join
// out = sum w_k o_k / sum w_k, w_k = 2^(lse_k - max lse), over the partials of
// a (token, query head) row: those of its sequence's own tiles and of its
// group's, one or two for each chunk.  One CTA per kv head and `tokens` tokens
// (several when there are many: a row's chain of dependent loads, token,
// tiles, log-sum-exps, partials, is what it waits for).  A warp lists a
// token's partials, which its G rows share; then a warp takes a row at a
// time, kHJoinDepth partials in flight.  With fewer rows than warps several
// warps take a row's partials in turn and add up in shared memory.
constexpr int kHJoinWarps = 8;
constexpr int kHJoinDepth = 8;
constexpr int kHJoinTokens = 8;
struct HJoinArgs {
  HPtrs ws;
  uint8_t* out;
  float* lse;  // may be null
  int32_t Hkv, G, total_q;
  int32_t tokens;  // of one CTA
  int32_t slots;   // rows at once: a power of two, at most the warps
  int32_t cap;     // partials of one row, at most
};

template <bool kBf16>
__global__ void __launch_bounds__(kHJoinWarps * 32) k_shared_join(HJoinArgs a) {
  extern __shared__ int32_t lists[];  // [tokens][cap]
  __shared__ int32_t count[kHJoinTokens];
  __shared__ float4 sum[kHJoinWarps][32];
  __shared__ float weight[kHJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tg = blockIdx.x / a.Hkv, g = blockIdx.x - tg * a.Hkv;
  const int t0 = tg * a.tokens, nt = min(a.tokens, a.total_q - t0);
  pdl_launch_dependents();
  pdl_wait();
  if (warp < nt) {
    const int t = t0 + warp;
    int32_t* list = lists + warp * a.cap;
    const HTok tk = a.ws.tok[t];
    int n = 0;
    for (int x0 = 0; x0 < tk.own_nch + tk.pre_nch; x0 += 32) {
      const int x = x0 + lane;
      HPieces p{0, 0, 0, 0};
      if (x < tk.own_nch + tk.pre_nch)
        p = a.ws.pieces[x < tk.pre_nch ? tk.pre_base + (g * tk.pre_nch + x) * tk.pre_nrt
                                       : tk.own_base + (g * tk.own_nch + x - tk.pre_nch) * tk.own_nrt];
      int y = p.pieces;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      int at = n + y - p.pieces;
      n += __shfl_sync(0xffffffffu, y, 31);
      for (int k = 0; k < p.pieces; ++k, ++at)
        if (at < a.cap) list[at] = p.part0 + (k * p.ntok + t - p.tok0) * a.G;  // (within the cap: see shared_layout)
    }
    if (lane == 0) count[warp] = tk.seq < 0 ? -1 : min(n, a.cap);  // -1: outside every sequence
  }
  __syncthreads();
  const int splits = kHJoinWarps / a.slots, slot = warp & (a.slots - 1), part = warp / a.slots;
  for (int i0 = 0; i0 < nt * a.G; i0 += a.slots) {
    const int row = i0 + slot, x = row / a.G, hh = row - x * a.G;
    const int n = row < nt * a.G ? count[x] : -1;
    const int32_t* list = lists + x * a.cap;
    float M = -INFINITY, W = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* po = reinterpret_cast<const float4*>(a.ws.part_o) + lane;
    float4 o[kHJoinDepth];
    float w[kHJoinDepth];
    auto fetch = [&](int j0) {
#pragma unroll
      for (int u = 0; u < kHJoinDepth; ++u) {
        const int j = j0 + u * splits;
        w[u] = -INFINITY;
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < n) {  // warp-uniform
          const long long pr = list[j] + hh;
          w[u] = a.ws.part_lse[pr];
          o[u] = __ldcs(po + pr * 32);
        }
      }
    };
    fetch(part);  // on their way before the log-sum-exps are known
    for (int i = lane; i < n; i += 32) M = hmax_nan(M, a.ws.part_lse[list[i] + hh]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = hmax_nan(M, __shfl_xor_sync(0xffffffffu, M, x));
    if (n > 0 && M != -INFINITY) {
      for (int j0 = part; j0 < n; j0 += kHJoinDepth * splits) {
        if (j0 > part) fetch(j0);
#pragma unroll
        for (int u = 0; u < kHJoinDepth; ++u) {
          w[u] = ex2_approx(w[u] - M);
          acc.x = fmaf(w[u], o[u].x, acc.x);
          acc.y = fmaf(w[u], o[u].y, acc.y);
          acc.z = fmaf(w[u], o[u].z, acc.z);
          acc.w = fmaf(w[u], o[u].w, acc.w);
          W += w[u];
        }
      }
    }
    if (splits > 1) {
      __syncthreads();  // the previous rows' sums have been read
      sum[warp][lane] = acc;
      if (lane == 0) weight[warp] = W;
      __syncthreads();
      if (part == 0)
        for (int k = 1; k < splits; ++k) {
          const float4 y = sum[warp + k * a.slots][lane];
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
          W += weight[warp + k * a.slots];
        }
    }
    if (n >= 0 && part == 0) {
      const float inv = W == 0.f ? 0.f : 1.f / W;
      const int h = g * a.G + hh, t = t0 + x;
      reinterpret_cast<uint2*>(a.out + ((size_t)t * a.Hkv * a.G + h) * 256)[lane] =
          make_uint2(hpack2<kBf16>(acc.x * inv, acc.y * inv), hpack2<kBf16>(acc.z * inv, acc.w * inv));
      if (a.lse && lane == 0)
        a.lse[(size_t)h * a.total_q + t] = W == 0.f ? -INFINITY : (M + lg2_approx(W)) * 0.69314718055994530942f;
    }
  }
}

}  // namespace

size_t shared_workspace_bytes(const mxsa_problem& p) { return shared_layout(p).total; }

// The join lists partial rows in 32 bits (2^31 rows would take 1.1 TB).
bool shared_rows_fit(const mxsa_problem& p) { return shared_layout(p).row_cap < INT_MAX; }

cudaError_t launch_dense_shared(const mxsa_problem& p, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, const int64_t* cu, const int32_t* lens, int num_groups,
                                const int32_t* group_ptr, const int32_t* prefix_lens, void* ws, void* out, float* lse,
                                int32_t* flags, cudaStream_t st) {
  if (p.total_q == 0) return cudaSuccess;
  auto fn = tensor_map_encoder();
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
  static PerDevice limits;
  cudaError_t e = limits([smem] {
    const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t x = cudaFuncSetAttribute(k_shared<true>, a, (int)smem);
    if (x == cudaSuccess) x = cudaFuncSetAttribute(k_shared<false>, a, (int)smem);
    if (x == cudaSuccess) x = cudaFuncSetAttribute(k_shared_plan, a, (int)sizeof(HPlanSmem));
    return x;
  });
  if (e != cudaSuccess) return e;

  HPlanArgs pa{};
  pa.cu = cu;
  pa.lens = lens;
  pa.group_ptr = group_ptr;
  pa.prefix_lens = prefix_lens;
  pa.flags = flags;
  pa.ws = ptrs;
  pa.tile_cap = L.tile_cap;
  pa.num_seqs = p.num_seqs;
  pa.num_groups = num_groups;
  pa.total_q = p.total_q;
  pa.Hkv = p.num_kv_heads;
  pa.G = G;
  pa.T = T;
  pa.max_len = p.max_pages_per_seq * p.page_size;
  pa.causal = p.causal;
  pa.ctas = ctas;
  e = launch_pdl(k_shared_plan, dim3(1), dim3(kHPlanThreads), sizeof(HPlanSmem), st, pa);
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
  ja.total_q = p.total_q;
  // several tokens to a CTA once there are four CTAs per SM
  const long long pairs = (long long)p.total_q * p.num_kv_heads;
  ja.cap = L.join_cap;
  ja.tokens = (int)std::max(1LL, std::min<long long>({kHJoinTokens, pairs / (4LL * sms), 40960 / (4LL * ja.cap)}));
  ja.slots = 1;
  while (ja.slots < G * ja.tokens && ja.slots < kHJoinWarps) ja.slots *= 2;
  const long long blocks = (long long)((p.total_q + ja.tokens - 1) / ja.tokens) * p.num_kv_heads;
  return launch_pdl(bf16 ? k_shared_join<true> : k_shared_join<false>, dim3((unsigned)blocks), dim3(kHJoinWarps * 32),
                    (size_t)ja.tokens * ja.cap * 4, st, ja);
}

}  // namespace mxsa

#ifdef MXSA_TEST_HOOKS
// Test builds only: the CTA of the next dense_shared_fwd launches that keeps
// its first window to itself; -1 turns the switch off.  Synchronous.
extern "C" mxsa_status mxsa_test_skip_window(int32_t cta) {
  return cudaMemcpyToSymbol(mxsa::g_skip_window, &cta, sizeof(cta)) == cudaSuccess ? MXSA_OK : MXSA_ERR_CUDA;
}
#endif

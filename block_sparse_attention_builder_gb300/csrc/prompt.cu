// Attention of whole prompts, packed one behind the other and read straight
// from the projection (mxsa_prompt_fwd): softmax(q k^T * scale) v over the
// sequence's own tokens, up to the row's own one when causal.
//
// A tile is 2T tokens (T = 128 / G) x the G query heads of one kv head of one
// sequence: two halves of up to 128 (token, head) rows that share every
// 128-key block of K and V.  Persistent, one CTA per SM, 384 threads:
//   warp 0     producer: claims tiles, K and V blocks into a ring of five
//              32 KB stages in the order K0 V0 K1 V1 ...
//   warp 1     q halves.
//   warps 2, 3 MMA issuers, one per group: P V of a block (its first 64 keys
//              once their P is there) and q k^T of the next one, in turns, so
//              that each group's softmax runs under the other's products.  S
//              is overwritten by the product after the one that reads P from
//              it; one thread issues both, and the pipe keeps their order.
//   warps 4-7, 8-11  softmax groups, one per half: thread = TMEM lane = row.
// TMEM: S (P over it) and O of each group, 512 columns.
//
// Softmax of a block, 64 keys at a time.  P = 2^(S - m) is made with the
// reference m of the blocks before; the sum of the 64, which is there anyway, says
// whether a row has passed m by much (rare past the first blocks).  Only then the
// maximum is looked for, m raised, O in TMEM rescaled and P made again.  So neither
// a maximum nor a second reading of S is in the way of the exponentials.  First and
// masked keys have their maximum found first.
//
// Bound: a group's chain of softmax (1300 cycles a block; 64 exponentials, sums and
// conversions of 32 rows take 356 at least while the other group is at its own),
// its hand-overs (230 and 300) and its products (1024); with both groups in turn
// 2690 cycles a block pair, of which the tensor pipe works 2048.  8192 tokens of
// 64 + 8 heads, causal, the GPU at rest before: 634 us, 1.73 PFLOP/s; 16384: 2.44
// ms, 1.80.  Under lasting load power lowers the SM clock from 2.07 GHz, to 1.83,
// 1.79 and, at 32768 tokens, 1.73: 688 us, 2.69 and 10.75 ms, 1.60 to 1.64.  On the
// way there, 8192 tokens: one issuer for both groups 841 us (its own bookkeeping of 600 cycles a
// block stood between the products), without turns 731, P handed over whole 747,
// rows written one to a thread 705, a maximum found beside the exponentials 681.
// Two warps to a row, each with 64 of a block's keys and 104 registers a thread,
// were slower (716: they meet at barriers, and the unit that makes exponentials and
// conversions is the same), and so were a row's 128 scores held at once, loads of
// the second 64 ahead of the first ones' exponentials, a split of the registers
// between the warps, masks as bits, and a hand-over of the turn before q k^T's last
// products.  A run over the rows' code ahead of the first tile, so that it is
// fetched by then, changed nothing.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "internal.h"
#include "mma_tiles.cuh"
#include "ptx.cuh"

namespace mxsa {

namespace {

constexpr int kRMaxSeqs = 1024;
constexpr int kRThreads = 384;
constexpr int kRProducer = 0, kRQuery = 1, kRMma = 2;  // warps 2, 3: the issuers of groups 0, 1
constexpr uint32_t kRTile = 32768;  // 128 rows x 128 x 16-bit
constexpr int kRStages = 5, kRWork = 2;
constexpr uint32_t kROffKV = 2 * kRTile;
constexpr uint32_t kROffCtrl = kROffKV + kRStages * kRTile;

// Tokens t0 .. t0 + ntok of a sequence of len tokens from token key0 on; n0,
// n1: key blocks that the two halves see (n1 is 0 or at least n0, or n0 is 0: see
// the producer).
struct alignas(16) RTile {
  int32_t key0, len, t0, ntok;
  int32_t n0, n1, g, pad;
};

struct RHeader {
  int32_t count, next;  // tiles (times kv heads), the next one to claim
};

// The full barriers alternate between two for a stage: a role that passes over
// places of the other half could otherwise take a phase for the one before.
struct RCtrl {
  uint64_t q_full[2], q_empty[2], kv_full[2 * kRStages], kv_empty[kRStages];
  uint64_t s_full[2], p_half[2], lo_done[2], p_full[2], o_full[2], o_empty[2], turn[2], done;
  uint64_t work_full[kRWork], work_empty[kRWork];
  RTile work[kRWork];
  uint32_t tmem_base;
  int32_t abort_flag, local_flags;
};

struct RArgs {
  const int64_t* cu;
  uint8_t* out;
  float* lse;      // may be null
  int32_t* flags;  // may be null
  RHeader* hdr;    // null: CTA i has tile i and no other
  const RTile* tiles;
  int32_t num_seqs, total_q, Hq, Hkv, G, T, causal;
  uint32_t inv_G;  // x / G == x * inv_G >> 16 for x < 128
  float scale_log2;
};

// The tile of tokens t0 .. of a sequence (its head is not set).
__device__ __forceinline__ RTile prompt_tile(int key0, int len, int t0, int T, int causal) {
  RTile t;
  t.key0 = key0;
  t.len = len;
  t.t0 = t0;
  t.ntok = min(2 * T, len - t0);
  const int all = (len + 127) >> 7;
  t.n0 = causal ? (min(t0 + T, len) + 127) >> 7 : all;
  t.n1 = t.ntok <= T ? 0 : (causal ? (t0 + t.ntok + 127) >> 7 : all);
  t.g = 0;
  t.pad = 0;
  return t;
}

// ------------------------------------------------------------------- plan
// Where there are more tiles than CTAs: the tiles in an order of falling
// length (their key blocks, in kRBuckets steps), which the CTAs claim one by
// one.  Equal ones stand in any order: each is computed by itself.
constexpr int kRPlanThreads = 1024, kRBuckets = 2048;

__global__ void __launch_bounds__(kRPlanThreads) k_prompt_plan(RArgs a, RHeader* hdr, RTile* tiles, int grid) {
  __shared__ int32_t start[kRMaxSeqs + 1], first[kRMaxSeqs + 1], bucket[kRBuckets], part[32];
  __shared__ int32_t longest;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, B = a.num_seqs;
  pdl_launch_dependents();
  pdl_wait();
  long long c0 = 0, c1 = 0;
  int bad = 0;
  if (tid < B) {
    c0 = a.cu[tid];
    c1 = a.cu[tid + 1];
    bad = c0 < 0 || c1 < c0 || c1 > a.total_q;
    start[tid] = (int)c0;
    if (tid == B - 1) start[B] = (int)c1;
  }
  if (tid == 0) longest = 0;
  bucket[tid] = bucket[tid + kRPlanThreads] = 0;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      *hdr = RHeader{0, grid};
      if (a.flags) atomicOr(a.flags, MXSA_FLAG_CU);
    }
    return;
  }
  const int len = (int)(c1 - c0), per = 2 * a.T, mine = (len + per - 1) / per;
  int x = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) part[w] = x;
  if (len > 0) atomicMax(&longest, (len + 127) >> 7);
  __syncthreads();
  int y = part[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  const int total = __shfl_sync(0xffffffffu, y, 31), before = __shfl_sync(0xffffffffu, y, max(w - 1, 0));
  if (tid < B) first[tid] = x - mine + (w ? before : 0);
  int shift = 0;
  while ((longest >> shift) >= kRBuckets) ++shift;
  __syncthreads();
  auto tile = [&](int i) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    return prompt_tile(start[lo], start[lo + 1] - start[lo], (i - first[lo]) * per, a.T, a.causal);
  };
  auto place = [&](const RTile& t) { return kRBuckets - 1 - (max(t.n0, t.n1) >> shift); };
  for (int i = tid; i < total; i += kRPlanThreads) atomicAdd(&bucket[place(tile(i))], 1);
  __syncthreads();
  const int b0 = bucket[2 * tid], b1 = bucket[2 * tid + 1];
  x = b0 + b1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += z;
  }
  if (lane == 31) part[w] = x;
  __syncthreads();
  y = part[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += z;
  }
  const int base = __shfl_sync(0xffffffffu, y, max(w - 1, 0));
  x += (w ? base : 0) - b0 - b1;
  bucket[2 * tid] = x;
  bucket[2 * tid + 1] = x + b0;
  __syncthreads();
  for (int i = tid; i < total; i += kRPlanThreads) {
    const RTile t = tile(i);
    tiles[atomicAdd(&bucket[place(t)], 1)] = t;
  }
  if (tid == 0) *hdr = RHeader{total * a.Hkv, grid};
}

// ---------------------------------------------------------------- forward
// The 4 x 4 words that four neighbouring lanes hold, transposed.
__device__ __forceinline__ void quad_transpose(uint32_t* w, int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!(k & d)) {
        const uint32_t x = __shfl_xor_sync(0xffffffffu, up ? w[k] : w[k + d], d);
        if (up) w[k] = x;
        else w[k + d] = x;
      }
  }
}

#ifdef MXSA_TEST_HOOKS
// Test builds only: CTA g_skip_record keeps its first tile's record to itself,
// so that every other role's first wait runs out.
__device__ int g_skip_record = -1;
#endif

template <bool kBf16>
__global__ void __launch_bounds__(kRThreads, 1)
    k_prompt(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
             const __grid_constant__ CUtensorMap tmv, RArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RCtrl& c = *reinterpret_cast<RCtrl*>(sm + kROffCtrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.q_full[i], 1);
      mbar_init(&c.q_empty[i], 1);
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 4);  // one arrival per warp of the group
      mbar_init(&c.p_full[i], 4);
      mbar_init(&c.lo_done[i], 1);
      mbar_init(&c.o_full[i], 1);
      mbar_init(&c.o_empty[i], 4);
      mbar_init(&c.turn[i], 1);
    }
    for (int i = 0; i < kRStages; ++i) {
      mbar_init(&c.kv_full[i], 1);
      mbar_init(&c.kv_full[i + kRStages], 1);
      mbar_init(&c.kv_empty[i], 2);  // (see the issuers)
    }
    for (int i = 0; i < kRWork; ++i) {
      mbar_init(&c.work_full[i], 1);
      mbar_init(&c.work_empty[i], 11);  // the q warp, the issuers and the softmax groups' warps
    }
    mbar_init(&c.done, 2);
    c.abort_flag = 0;
    c.local_flags = 0;
    fence_mbar_init();
  }
  if (warp == kRMma) {
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
  pdl_wait();
  // The next tile of a role that is not the producer; false at the end (or
  // when a wait gave up).
  int taken = 0;
  auto next_tile = [&](RTile* t) {
    const int w = taken % kRWork;
    if (!hwarp_all(mbar_wait(&c.work_full[w], (taken / kRWork) & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs)))
      return false;
    *t = c.work[w];
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.work_empty[w]);
    ++taken;
    return max(t->n0, t->n1) > 0;
  };

  if (warp < 4) {
    if (warp == kRProducer) {
      // -------------------------------------------------------------- producer
      if (lane == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
      }
      const int count = a.hdr ? a.hdr->count : 0;
      // tile number x (kv heads next to each other); no blocks: the end
      auto fetch = [&](int x) {
        RTile t{};
        if (x < count) {
          const int rec = x / a.Hkv;
          t = a.tiles[rec];
          t.g = x - rec * a.Hkv;
        }
        return t;
      };
      // without a plan: the CTA's one tile, from the sequences' starts
      auto own = [&]() {
        RTile t{};
        const int rec = blockIdx.x / a.Hkv, per = 2 * a.T;
        int before = 0, bad = 0;
        for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
          const int s = s0 + lane;
          long long c0 = 0, c1 = 0;
          if (s < a.num_seqs) {
            c0 = a.cu[s];
            c1 = a.cu[s + 1];
            bad |= c0 < 0 || c1 < c0 || c1 > a.total_q;
          }
          const int n = bad ? 0 : (int)((c1 - c0 + per - 1) / per);
          int x = n;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
          }
          const int at = before + x - n;
          const unsigned hit = __ballot_sync(0xffffffffu, rec >= at && rec < at + n);
          if (hit) {
            const int src = __ffs(hit) - 1;
            const int key0 = __shfl_sync(0xffffffffu, (int)c0, src), len = __shfl_sync(0xffffffffu, (int)(c1 - c0), src);
            t = prompt_tile(key0, len, (rec - __shfl_sync(0xffffffffu, at, src)) * per, a.T, a.causal);
            t.g = blockIdx.x - rec * a.Hkv;
          }
          before += __shfl_sync(0xffffffffu, x, 31);
        }
        if (__any_sync(0xffffffffu, bad)) {
          if (lane == 0) atomicOr(fl, MXSA_FLAG_CU);
          t = RTile{};
        }
        return t;
      };
      int at = 0;
      bool ok = true, second = false;
      RTile t = a.hdr ? fetch(blockIdx.x) : own();
      for (int n = 0;; ++n) {
        const int w = n % kRWork;
        ok = hwarp_all(
            mbar_wait(&c.work_empty[w], ((n / kRWork) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
        if (!ok) break;
#ifdef MXSA_TEST_HOOKS
        const bool skip = (int)blockIdx.x == g_skip_record && n == 0;
#else
        constexpr bool skip = false;
#endif
        // A tile of one half goes to the groups in turn, so that two of them overlap:
        // to the second one as the second half of a tile that begins T tokens earlier
        // and has no first half (256 prompts of 100 tokens, 16 + 16 heads: 93 us with
        // all in the first group, 72 so; 300 of 14, 64 + 8: 60 and 45).
        if (t.n0 > 0 && t.n1 == 0) {
          if (second) {
            t.n1 = t.n0;
            t.n0 = 0;
            t.t0 -= a.T;
            t.ntok += a.T;
          }
          second = !second;
        }
        if (lane == 0) {
          c.work[w] = t;
          if (!skip) mbar_arrive(&c.work_full[w]);
        }
        const int blocks = max(t.n0, t.n1);
        if (blocks == 0) break;
        int claimed = INT_MAX;
        if (lane == 0) {
          for (int p = 0; p < 2 * blocks && ok; ++p, ++at) {
            const int st = at % kRStages;
            ok = mbar_wait(&c.kv_empty[st], ((at / kRStages) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
            if (!ok) break;
            // the next tile, while this one's last copies are on their way
            if (p == 2 * blocks - 2 && a.hdr) claimed = atomicAdd(&a.hdr->next, 1);
            uint8_t* dst = sm + kROffKV + st * kRTile;
            const int row = t.key0 + (p >> 1) * 128;
            const CUtensorMap* tm = p & 1 ? &tmv : &tmk;
            uint64_t* full = &c.kv_full[at % (2 * kRStages)];
            mbar_arrive_expect_tx(full, kRTile);
            tma_load_3d(dst, tm, full, 0, t.g, row);
            tma_load_3d(dst + 16384, tm, full, 64, t.g, row);
          }
        }
        ok = hwarp_all(ok);
        if (!ok) break;
        t = fetch(__shfl_sync(0xffffffffu, claimed, 0));
      }
      at = __shfl_sync(0xffffffffu, at, 0);
      if (lane == 0)  // drain: the copies in flight land before the CTA may exit
        for (int k = max(0, at - kRStages); k < at; ++k)
          mbar_drain(&c.kv_full[k % (2 * kRStages)], (k / (2 * kRStages)) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      __syncwarp();
    } else if (warp == kRQuery) {
      // --------------------------------------------------------------- queries
      if (lane == 0) tma_prefetch_desc(&tmq);
      int nq0 = 0, nq1 = 0;
      bool ok = true;
      RTile t;
      while (ok && next_tile(&t)) {
        for (int h = 0; h < 2; ++h) {
          if ((h ? t.n1 : t.n0) == 0) continue;
          ok = hwarp_all(
              mbar_wait(&c.q_empty[h], ((h ? nq1 : nq0) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
          if (!ok) break;
          if (lane == 0) {  // one box; rows past the half's tokens are never used
            uint8_t* qd = sm + h * kRTile;
            mbar_arrive_expect_tx(&c.q_full[h], (uint32_t)(a.G * a.T) * 256u);
            tma_load_3d(qd, &tmq, &c.q_full[h], 0, t.g * a.G, t.key0 + t.t0 + h * a.T);
            tma_load_3d(qd + 16384, &tmq, &c.q_full[h], 64, t.g * a.G, t.key0 + t.t0 + h * a.T);
          }
          (h ? nq1 : nq0) += 1;
        }
      }
      if (lane == 0) {
        if (nq0) mbar_drain(&c.q_full[0], (nq0 - 1) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
        if (nq1) mbar_drain(&c.q_full[1], (nq1 - 1) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      }
      __syncwarp();
    } else {
      // --------------------------------------------------------- MMA issuers
      // One warp per group: while it stands at its group's softmax the pipe has
      // the other group's products, and what it does between its own (some
      // hundred cycles) is under them.  The whole warp walks the loop and one
      // elected lane issues, so that what the instructions take from uniform
      // registers is known to be uniform.
      const int h = warp - kRMma;
      const uint32_t id_qk = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 0);
      const uint32_t id_pv = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 1);
      const uint32_t tS = uniform(tmem + h * 256);
      const uint32_t dq = uniform(desc_k_major(sbase + h * kRTile));
      const uint32_t dk0 = desc_k_major(sbase + kROffKV), dv0 = desc_mn_major(sbase + kROffKV);
      int st = 0, full = 0, par = 0;  // the next ring place: stage, full barrier and its parity
      int np = 0, nt = 0, turns = 0;  // P V products, tiles and turns of the group
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        ok = ok && hwarp_all(mbar_wait(bar, parity, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      };
      auto pass = [&] {
        if (++st == kRStages) st = 0;
        if (++full == 2 * kRStages) full = 0, par ^= 1;
      };
      RTile t;
      while (ok && next_tile(&t)) {
        const int n = h ? t.n1 : t.n0, blocks = max(t.n0, t.n1);
        // In a tile of two halves the groups take turns at the pipe.  Left alone
        // they fall into step: both sets of products in the pipe at once, then
        // both groups in their softmax.
        const bool both = t.n0 > 0 && t.n1 > 0;
        for (int i = 0; i <= (both ? blocks : n) && ok; ++i) {
          if (i > n || n == 0) {  // nothing left of this group's: its turns pass
            if (!both) break;
            if (h == 1 || turns > 0) wait(&c.turn[h], (turns + h + 1) & 1);
            ++turns;
            if (ok && lane == 0) mbar_arrive(&c.turn[h ^ 1]);
            __syncwarp();
            continue;
          }
          // Two arrivals free a stage: one of each group, or both of the only
          // one that reads it.
          const bool alone_v = h ? i - 1 >= t.n0 : t.n1 == 0, alone_k = h ? i >= t.n0 : t.n1 == 0;
          int vs = 0, ks = 0;
          if (i > 0) {  // V of the block before
            vs = st;
            wait(&c.kv_full[full], par);
            pass();
          }
          if (i < n) {
            ks = st;
            wait(&c.kv_full[full], par);
            pass();
          }
          const uint32_t dv = uniform(dv0 + vs * (kRTile >> 4)), dk = uniform(dk0 + ks * (kRTile >> 4));
          if (i == 0) wait(&c.q_full[h], nt & 1);
          if (i == 1 && nt > 0) wait(&c.o_empty[h], (nt - 1) & 1);
          if (i > 0) wait(&c.p_half[h], np & 1);
          if (both) {
            if (h == 1 || turns > 0) wait(&c.turn[h], (turns + h + 1) & 1);
            ++turns;
          }
          if (i > 0) {
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              mma_pv_lo(tS + 128, tS, dv, id_pv, i > 1);
              mma_commit(&c.lo_done[h]);
            }
            __syncwarp();
            wait(&c.p_full[h], np++ & 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (i > 0) {
              mma_pv_hi(tS + 128, tS, dv, id_pv);
              if (i == n) mma_commit(&c.o_full[h]);
            }
            if (i < n) {
              mma_qk(tS, dq, dk, id_qk);
              if (both) mbar_arrive(&c.turn[h ^ 1]);
              mma_commit(&c.s_full[h]);
              mma_commit(&c.kv_empty[ks]);
              if (alone_k) mma_commit(&c.kv_empty[ks]);
              if (i == n - 1) mma_commit(&c.q_empty[h]);
            } else if (both) {
              mbar_arrive(&c.turn[h ^ 1]);
            }
            if (i > 0) {
              mma_commit(&c.kv_empty[vs]);
              if (alone_v) mma_commit(&c.kv_empty[vs]);
            }
          }
          __syncwarp();
        }
        for (int p = 2 * n; p < 2 * blocks; ++p) pass();
        if (n > 0) ++nt;
      }
      if (elect_one()) {
        mma_commit(&c.done);
        mbar_drain(&c.done, 0, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int h = (warp >> 2) - 1, r = tid & 127;  // row of the half == TMEM lane
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + h * 256 + lane_addr, tO = tS + 128;
    const int rt = r * a.inv_G >> 16, tt = h * a.T + rt;
    int at = 0, n_s = 0, n_o = 0;
    bool ok = true;
    RTile t;
    while (ok && next_tile(&t)) {
      const int n = h ? t.n1 : t.n0;
      const int at0 = at;
      at += 2 * max(t.n0, t.n1);
      if (n == 0) continue;
      const bool live = rt < a.T && tt < t.ntok;
      const bool warp_live = __any_sync(0xffffffffu, live);
      // keys that the row sees (padding rows see all: nobody reads them)
      const int see = live ? (a.causal ? t.t0 + tt + 1 : t.len) : INT_MAX;
      const int warp_see = __reduce_min_sync(0xffffffffu, see);
      // A row that is not live, whose q may be anything, has P of zero: it must have
      // no say in what its warp does, or the others' bits would not be the same
      // every time.
      float m = live ? -INFINITY : INFINITY, l = 0.f;
      bool fresh = true;  // there are rows without a finite maximum
      for (int i = 0; i < n && ok; ++i, ++n_s) {
        const int k0 = i << 7;
        ok = hwarp_all(mbar_wait(&c.s_full[h], n_s & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
        if (!ok) break;
        if (k0 + 128 > t.len) {
          // V rows behind the sequence: zeros, since another sequence's may be
          // NaN and 0 * NaN would reach O (the writers' proxy fence orders them
          // before the product)
          const int pl = at0 + 2 * i + 1, st = pl % kRStages;
          ok = hwarp_all(mbar_wait(&c.kv_full[pl % (2 * kRStages)], (pl / (2 * kRStages)) & 1, abort_flag, fl,
                                   MXSA_FLAG_TIMEOUT, kWaitLimitNs));
          if (!ok) break;
          if (k0 + r >= t.len) {
            const uint32_t vs = sbase + kROffKV + st * kRTile + r * 128;
            for (int ch = 0; ch < 16; ++ch)
              st_shared_v4(vs + (ch >> 3) * 16384u + (((ch & 7) ^ (r & 7)) << 4), 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (warp_live) {
          tc_fence_after();
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            float sv[64];
            tmem_ld32(tS + 64 * hf, sv);
            tmem_ld32(tS + 64 * hf + 32, sv + 32);
            tmem_ld_wait();
            const int kh = k0 + 64 * hf;
            const bool masked = kh + 64 > warp_see;
            float sum;
            // m is looked at first where keys are masked or there is none yet, else
            // once the P say that they are too large (all these conditions are the same
            // in every lane)
            float gap = kGapKnown;
            for (bool known = masked || fresh;; known = true, gap = kGapSum) {
              if (__builtin_expect(known, 0)) {
                if (masked) {
#pragma unroll
                  for (int k = 0; k < 64; ++k) sv[k] = kh + k < see ? sv[k] : -INFINITY;
                }
                const float bm = max64(sv) * a.scale_log2;
                const bool raise = bm > m + gap;
                if (__any_sync(0xffffffffu, raise)) {
                  // O is complete up to the block before (S's barrier follows
                  // every product issued before it); in the second half the
                  // first one's product has to be done too
                  if (hf) {
                    ok = hwarp_all(mbar_wait(&c.lo_done[h], n_s & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
                    if (!ok) break;
                    tc_fence_after();
                  }
                  const float f = raise ? (m == -INFINITY ? 0.f : ex2_approx(m - bm)) : 1.f;
                  tmem_st_wait();
                  if (kh > 0) scale_o(tO, f);
                  if (raise) {
                    l *= f;
                    m = bm;
                  }
                  fresh = __any_sync(0xffffffffu, m == -INFINITY);
                }
              }
              sum = exp_half<kBf16>(sv, a.scale_log2, m == -INFINITY ? 0.f : m, tS + 32 * hf);
              if (__builtin_expect(known || !__any_sync(0xffffffffu, sum > (hf ? kSumHigh : kSumLow)), 1)) break;
            }
            if (!ok) break;
            l += sum;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(hf ? &c.p_full[h] : &c.p_half[h]);
          }
        } else if (lane == 0) {
          mbar_arrive(&c.p_half[h]);
          mbar_arrive(&c.p_full[h]);
        }
      }
      if (!ok) break;
      // ---- the half's output rows
      ok = hwarp_all(mbar_wait(&c.o_full[h], n_o & 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
      if (!ok) break;
      ++n_o;
      if (warp_live) {
        tc_fence_after();
        const float inv = l == 0.f ? 0.f : rcp_approx(l);  // (a NaN stays one; off by 2^-23 at most)
        // 16 rows and 64 columns at a time, a row's columns spread over four
        // lanes, which then exchange words until each has 16 consecutive bytes:
        // a store then covers 64 bytes of 8 rows.  (With a row to a thread it
        // touches 32 rows, and the eight warps' stores take 4000 cycles.)
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
          const int r0 = (part >> 1) * 16, c0 = (part & 1) * 64;
          float v[32];
          tmem_ld16x256b_x8(tO + ((uint32_t)r0 << 16) + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 2; ++x) {  // rows lane / 4 and lane / 4 + 8 of the 16
            const int src = r0 + (lane >> 2) + 8 * x, row = (warp & 3) * 32 + src;
            const float f = __shfl_sync(0xffffffffu, inv, src);
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = hpack2<kBf16>(v[4 * k + 2 * x] * f, v[4 * k + 2 * x + 1] * f);
            quad_transpose(w, lane);
            quad_transpose(w + 4, lane);
            const int to = row * a.inv_G >> 16, ho = row - to * a.G;
            if (to < a.T && h * a.T + to < t.ntok) {
              uint8_t* orow = a.out + (((size_t)t.key0 + t.t0 + h * a.T + to) * a.Hq + (size_t)t.g * a.G + ho) * 256 +
                              c0 * 2 + (lane & 3) * 16;
              *reinterpret_cast<uint4*>(orow) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(orow + 64) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
        if (live && a.lse)
          a.lse[(size_t)(t.g * a.G + r - rt * a.G) * a.total_q + t.key0 + t.t0 + tt] =
              l == 0.f ? -INFINITY : (m + lg2_approx(l)) * 0.69314718055994530942f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.o_empty[h]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kRMma) tmem_dealloc(tmem, 512);
}

// tiles of one kv head, at most
long long prompt_tile_cap(const mxsa_problem& p) {
  const int T = 128 / (p.num_q_heads / p.num_kv_heads);
  return p.total_q / (2 * T) + (long long)p.num_seqs;
}

}  // namespace

size_t prompt_workspace_bytes(const mxsa_problem& p) { return 256 + sizeof(RTile) * (size_t)prompt_tile_cap(p); }

cudaError_t launch_prompt(const mxsa_problem& p, const void* q, long long q_stride, const void* k, long long k_stride,
                          const void* v, long long v_stride, const int64_t* cu, void* ws, void* out, float* lse,
                          int32_t* flags, cudaStream_t st) {
  if (p.total_q == 0) return cudaSuccess;
  auto fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  const int G = p.num_q_heads / p.num_kv_heads, T = 128 / G;
  const bool bf16 = p.q_dtype == MXSA_BF16;
  const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto map3 = [&](CUtensorMap* m, const void* base, int heads, long long stride, cuuint32_t b1, cuuint32_t b2) {
    cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)p.total_q}, strides[2] = {256, 2 * (cuuint64_t)stride};
    cuuint32_t box[3] = {64, b1, b2}, es[3] = {1, 1, 1};
    return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  CUtensorMap tmq, tmk, tmv;
  if (!map3(&tmq, q, p.num_q_heads, q_stride, G, T) || !map3(&tmk, k, p.num_kv_heads, k_stride, 1, 128) ||
      !map3(&tmv, v, p.num_kv_heads, v_stride, 1, 128))
    return cudaErrorInvalidValue;
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const size_t smem = kROffCtrl + sizeof(RCtrl) + 1024;
  static PerDevice limits;
  cudaError_t e = limits([smem] {
    const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t x = cudaFuncSetAttribute(k_prompt<true>, a, (int)smem);
    return x == cudaSuccess ? cudaFuncSetAttribute(k_prompt<false>, a, (int)smem) : x;
  });
  if (e != cudaSuccess) return e;
  RArgs a{};
  a.cu = cu;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.flags = flags;
  a.num_seqs = p.num_seqs;
  a.total_q = p.total_q;
  a.Hq = p.num_q_heads;
  a.Hkv = p.num_kv_heads;
  a.G = G;
  a.T = T;
  a.inv_G = 65535 / G + 1;
  a.causal = p.causal;
  const float scale = p.softmax_scale > 0.f ? p.softmax_scale : 0.08838834764831845f;  // 1/sqrt(128)
  a.scale_log2 = scale * 1.4426950408889634f;
  // Few tiles: CTA i takes tile i, found by itself; else the plan's order.
  const long long cap = prompt_tile_cap(p) * p.num_kv_heads;
  const int grid = (int)std::min<long long>(cap, sms);
  if (cap > sms) {
    a.hdr = static_cast<RHeader*>(ws);
    RTile* tiles = reinterpret_cast<RTile*>(static_cast<uint8_t*>(ws) + 256);
    a.tiles = tiles;
    e = launch_pdl(k_prompt_plan, dim3(1), dim3(kRPlanThreads), 0, st, a, a.hdr, tiles, grid);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(bf16 ? k_prompt<true> : k_prompt<false>, dim3(grid), dim3(kRThreads), smem, st, tmq, tmk, tmv, a);
}

}  // namespace mxsa

#ifdef MXSA_TEST_HOOKS
// Test builds only: the CTA of the next prompt_fwd launches that keeps its
// first tile's record to itself; -1 turns the switch off.  Synchronous.
extern "C" mxsa_status mxsa_test_skip_record(int32_t cta) {
  return cudaMemcpyToSymbol(mxsa::g_skip_record, &cta, sizeof(cta)) == cudaSuccess ? MXSA_OK : MXSA_ERR_CUDA;
}
#endif

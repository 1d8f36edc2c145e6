// Attention of drafted trees in one launch (mxsa_tree_fwd on few sequences of
// moderate length, without groups; see launch_tree_small): a cluster of C CTAs
// takes the rows of T = 128 / G tokens of one kv head of one sequence, its CTAs
// every C-th 128-key block each, and the pieces are joined over distributed
// shared memory.  The general path (shared.cu) makes a plan, fills partial
// buffers and joins them in three launches that wait for one another, 18 us for
// the smallest call; here there is nothing to wait for but the keys.
//
// 384 threads: warp 0 finds the tile, loads q and then K and V blocks (TMA
// through the block table) into a ring of five 32 KB stages; warps 2 and 3 issue
// the MMAs of the two softmax groups, warps 4-7 and 8-11, which have the same
// rows and alternate blocks (thread = TMEM lane = row, softmax as in
// prompt.cu).  After their last block the groups write O (FP32), maximum and sum
// to shared memory, where the ring was; after a barrier of the cluster each CTA
// joins every C-th row from the cluster's 2 C pieces and writes it.
//
// Bound: latency, a chain of lengths, table, keys, q k^T, softmax, P V, join: one
// sequence of 8 tokens on 1000 keys, 16 + 2 heads, 8.7 us (17.6 in three
// launches); 4 of 5 on 2000, 64 + 8 heads, 13.1 (21.4).
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

constexpr int kTThreads = 384;
constexpr int kTProducer = 0, kTMma = 2;
constexpr uint32_t kTTile = 32768;  // 128 rows x 128 x 16-bit
constexpr int kTStages = 5;
constexpr uint32_t kTOffKV = kTTile;
constexpr uint32_t kTOffCtrl = kTOffKV + kTStages * kTTile;
constexpr uint32_t kTPiece = 128 * 512;         // O of one group, over the ring
static_assert(2 * kTPiece <= kTStages * kTTile, "the groups' rows fit where the ring was");

struct TTile {
  int32_t tok0, ntok, row, len;  // first token, tokens (0: nothing to do), block table row, keys
  int32_t base, g, nblk, pad;    // committed keys (may be negative), kv head, blocks of the sequence
};

struct TCtrl {
  uint64_t found, q_full, kv_full[2 * kTStages], kv_empty[kTStages];
  uint64_t s_full[2], p_half[2], lo_done[2], p_full[2], o_full[2], done;
  TTile tile;
  uint32_t tmem_base;
  int32_t abort_flag, local_flags;
  float m[2][128], l[2][128];  // of each group's rows, log2 units
};

struct TArgs {
  const int64_t* cu;
  const int32_t *lens, *block_tables;
  const uint32_t* mask;
  uint8_t* out;
  float* lse;      // may be null
  int32_t* flags;  // may be null
  int32_t num_seqs, total_q, Hq, Hkv, G, T, page_shift, max_pages, num_pages, words, cluster;
  float scale_log2;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of `saddr` in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Byte offset of columns 4 c .. of a row in a piece: chunks at places that
// change with the row, so that neither the writers' rows nor the readers'
// chunks meet in a bank.
__device__ __forceinline__ uint32_t piece_at(int row, int c) { return row * 512 + ((c ^ (row & 31)) << 4); }

#ifdef MXSA_TEST_HOOKS
// Test builds only: CTA g_skip_found keeps its tile to itself, so that its
// issuers' and softmax warps' first wait runs out.
__device__ int g_skip_found = -1;
#endif

template <bool kBf16>
__global__ void __launch_bounds__(kTThreads, 1)
    k_tree_small(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, TArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TCtrl& c = *reinterpret_cast<TCtrl*>(sm + kTOffCtrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(&c.found, 1);
    mbar_init(&c.q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_half[i], 4);  // one arrival per warp of the group
      mbar_init(&c.p_full[i], 4);
      mbar_init(&c.lo_done[i], 1);
      mbar_init(&c.o_full[i], 1);
    }
    for (int i = 0; i < kTStages; ++i) {
      mbar_init(&c.kv_full[i], 1);
      mbar_init(&c.kv_full[i + kTStages], 1);
      mbar_init(&c.kv_empty[i], 1);
    }
    mbar_init(&c.done, 2);
    c.abort_flag = 0;
    c.local_flags = 0;
    fence_mbar_init();
  }
  if (warp == kTMma) {
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
  const int C = a.cluster, rank = blockIdx.x % C, cid = blockIdx.x / C;
  auto wait = [&](uint64_t* bar, int parity) {
    return hwarp_all(mbar_wait(bar, parity, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs));
  };
  pdl_wait();

  if (warp == kTProducer) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&tmq);
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
    }
    // The cluster's tile: row tile cid / Hkv of the batch, kv head cid % Hkv.
    // CTA 0 looks at every length on the way, for the flags.
    const int rec = cid / a.Hkv, max_len = a.max_pages << a.page_shift;
    TTile t{};
    int before = 0, bad = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
      const int s = s0 + lane;
      long long c0 = 0, c1 = 0;
      int len = 0;
      if (s < a.num_seqs) {
        c0 = a.cu[s];
        c1 = a.cu[s + 1];
        len = a.lens[s];
        if (c0 < 0 || c1 < c0 || c1 > a.total_q) bad |= MXSA_FLAG_CU;
      }
      const int L = min(max(len, 0), max_len);
      const int tq = bad & MXSA_FLAG_CU ? 0 : (int)(c1 - c0), n = (tq + a.T - 1) / a.T;
      if (L != len) bad |= MXSA_FLAG_LEN;
      if (tq > L) bad |= MXSA_FLAG_CAUSAL_LEN;
      if (tq > 32 * a.words) bad |= MXSA_FLAG_TREE;
      int x = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      const int at = before + x - n;
      const unsigned hit = __ballot_sync(0xffffffffu, rec >= at && rec < at + n);
      if (hit) {
        const int src = __ffs(hit) - 1, first = (rec - __shfl_sync(0xffffffffu, at, src)) * a.T;
        t.row = s0 + src;
        t.tok0 = (int)__shfl_sync(0xffffffffu, c0, src) + first;
        t.ntok = min(a.T, __shfl_sync(0xffffffffu, tq, src) - first);
        t.len = __shfl_sync(0xffffffffu, L, src);
        t.base = t.len - __shfl_sync(0xffffffffu, tq, src);
        t.g = cid % a.Hkv;
        t.nblk = (t.len + 127) >> 7;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (bad & MXSA_FLAG_CU) {  // nothing is written
      bad = MXSA_FLAG_CU;
      t = TTile{};
    }
#ifdef MXSA_TEST_HOOKS
    const bool skip = (int)blockIdx.x == g_skip_found;
#else
    constexpr bool skip = false;
#endif
    if (lane == 0) {
      c.tile = t;
      if (!skip) mbar_arrive(&c.found);
      if (t.ntok) {  // rows past the tile's tokens are never used
        mbar_arrive_expect_tx(&c.q_full, (uint32_t)(a.G * a.T) * 256u);
        tma_load_3d(sm, &tmq, &c.q_full, 0, t.g * a.G, t.tok0);
        tma_load_3d(sm + 16384, &tmq, &c.q_full, 64, t.g * a.G, t.tok0);
      }
      if (bad && blockIdx.x == 0) atomicOr(fl, bad);
    }
    const int ps = 1 << a.page_shift, npg = ps == 128 ? 1 : 2;
    const int n = t.ntok && t.nblk > rank ? (t.nblk - rank + C - 1) / C : 0;  // blocks of this CTA
    int at = 0;
    bool ok = true;
    for (int i = 0; i < n && ok; i += 16) {
      // the pages of 16 blocks at once, two to a block
      const int blk = rank + (i + (lane >> 1)) * C, p0 = blk * 128 + (lane & 1) * 64;
      const bool need = i + (lane >> 1) < n && (lane & 1) < npg && p0 < t.len;
      int page = need ? a.block_tables[(size_t)t.row * a.max_pages + (p0 >> a.page_shift)] : -1;
      if (need && (page < 0 || page >= a.num_pages)) {
        atomicOr(fl, MXSA_FLAG_PAGE);
        page = -1;
      }
      const int z = page < 0 ? -1 : page * a.Hkv + t.g;
      for (int k = 0; k < min(16, n - i) && ok; ++k) {
        const int z0 = __shfl_sync(0xffffffffu, z, 2 * k), z1 = __shfl_sync(0xffffffffu, z, 2 * k + 1);
        if (lane == 0)
          for (int kv = 0; kv < 2 && ok; ++kv, ++at) {
            const int st = at % kTStages;
            ok = mbar_wait(&c.kv_empty[st], ((at / kTStages) & 1) ^ 1, abort_flag, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
            if (!ok) break;
            uint64_t* full = &c.kv_full[at % (2 * kTStages)];
            uint8_t* dst = sm + kTOffKV + st * kTTile;
            const CUtensorMap* tm = kv ? &tmv : &tmk;
            mbar_arrive_expect_tx(full, (uint32_t)((z0 >= 0) + (z1 >= 0)) * (256u << a.page_shift));
            if (z0 >= 0) {
              tma_load_3d(dst, tm, full, 0, 0, z0);
              tma_load_3d(dst + 16384, tm, full, 64, 0, z0);
            }
            if (z1 >= 0) {
              tma_load_3d(dst + 8192, tm, full, 0, 0, z1);
              tma_load_3d(dst + 16384 + 8192, tm, full, 64, 0, z1);
            }
          }
        ok = hwarp_all(ok);
      }
    }
    at = __shfl_sync(0xffffffffu, at, 0);
    if (lane == 0) {  // drain: the copies in flight land before the memory is used again, or the CTA exits
      for (int k = max(0, at - kTStages); k < at; ++k)
        mbar_drain(&c.kv_full[k % (2 * kTStages)], (k / (2 * kTStages)) & 1, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
      if (t.ntok) mbar_drain(&c.q_full, 0, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kTMma || warp == kTMma + 1) {
    // ------------------------------------------------------------ MMA issuers
    // Group h has the CTA's blocks h, h + 2, ...: P V of one, then q k^T of the
    // next.  A stage has one reader.
    const int h = warp - kTMma;
    const uint32_t id_qk = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 0);
    const uint32_t id_pv = idesc_f16(128, 128, kBf16 ? 1u : 0u, 0, 1);
    // (in a cluster a shared address holds the CTA's rank above its offset, where
    // a descriptor has another field)
    const uint32_t own = sbase & 0xFFFFFFu;
    const uint32_t tS = uniform(tmem + h * 256), dq = uniform(desc_k_major(own));
    const uint32_t dk0 = desc_k_major(own + kTOffKV), dv0 = desc_mn_major(own + kTOffKV);
    bool ok = wait(&c.found, 0);
    const TTile t = c.tile;
    const int all = t.ntok && t.nblk > rank ? (t.nblk - rank + C - 1) / C : 0;
    const int n = ok && all > h ? (all - h + 1) / 2 : 0;
    if (n) ok = wait(&c.q_full, 0);
    for (int i = 0; i <= n && n && ok; ++i) {
      const int vp = 2 * (2 * (i - 1) + h) + 1, kp = 2 * (2 * i + h);  // ring places of V (block i - 1) and K (block i)
      if (i > 0) {
        const uint32_t dv = uniform(dv0 + (vp % kTStages) * (kTTile >> 4));
        ok = wait(&c.kv_full[vp % (2 * kTStages)], (vp / (2 * kTStages)) & 1) && wait(&c.p_half[h], (i - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_pv_lo(tS + 128, tS, dv, id_pv, i > 1);
          mma_commit(&c.lo_done[h]);
        }
        __syncwarp();
        ok = wait(&c.p_full[h], (i - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_pv_hi(tS + 128, tS, dv, id_pv);
          mma_commit(&c.kv_empty[vp % kTStages]);
          if (i == n) mma_commit(&c.o_full[h]);
        }
        __syncwarp();
      }
      if (i < n) {
        const uint32_t dk = uniform(dk0 + (kp % kTStages) * (kTTile >> 4));
        ok = wait(&c.kv_full[kp % (2 * kTStages)], (kp / (2 * kTStages)) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          mma_qk(tS, dq, dk, id_qk);
          mma_commit(&c.s_full[h]);
          mma_commit(&c.kv_empty[kp % kTStages]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      mma_commit(&c.done);
      mbar_drain(&c.done, 0, fl, MXSA_FLAG_TIMEOUT, kWaitLimitNs);
    }
    __syncwarp();
  }

  // ------------------------------------------------------------------ softmax
  const int h = (warp >> 2) - 1, r = tid & 127;  // row of the tile == TMEM lane
  const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t tS = tmem + (h & 1) * 256 + lane_addr, tO = tS + 128;
  bool ok = true;
  if (warp >= 4) {
    ok = wait(&c.found, 0);
    const TTile t = c.tile;
    const int all = t.ntok && t.nblk > rank ? (t.nblk - rank + C - 1) / C : 0;
    const int n = ok && all > h ? (all - h + 1) / 2 : 0;
    const int rt = r / a.G;
    const bool live = rt < t.ntok;
    const bool warp_live = __any_sync(0xffffffffu, live);
    // keys below base are seen by all rows (a row that is not live: everything)
    const int base = live ? t.base : INT_MAX / 2;
    const uint32_t* const mask = live ? a.mask + (size_t)(t.tok0 + rt) * a.words : a.mask;
    const int warp_see = __reduce_min_sync(0xffffffffu, min(base, t.len));
    float m = live ? -INFINITY : INFINITY, l = 0.f;  // (P of zero where it is not: as in prompt.cu)
    bool fresh = true;  // there are rows without a finite maximum
    for (int i = 0; i < n && ok; ++i) {
      const int j = 2 * i + h, k0 = (rank + j * C) << 7;
      ok = wait(&c.s_full[h], i & 1);
      if (!ok) break;
      if (k0 + 128 > t.len) {  // V rows behind the sequence: zeros (as in prompt.cu)
        const int pl = 2 * j + 1, st = pl % kTStages;
        ok = wait(&c.kv_full[pl % (2 * kTStages)], (pl / (2 * kTStages)) & 1);
        if (!ok) break;
        if (k0 + r >= t.len) {
          const uint32_t vs = sbase + kTOffKV + st * kTTile + r * 128;
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
          float gap = kGapKnown;
          for (bool known = masked || fresh;; known = true, gap = kGapSum) {  // (as in prompt.cu)
            if (__builtin_expect(known, 0)) {
              if (masked) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                  const int kq = kh + 32 * q;
                  uint32_t seen = tree_bits(mask, a.words, kq - base);
                  if (kq + 32 > t.len) seen &= kq >= t.len ? 0u : 0xFFFFFFFFu >> (kq + 32 - t.len);
#pragma unroll
                  for (int k = 0; k < 32; ++k) sv[32 * q + k] = seen >> k & 1 ? sv[32 * q + k] : -INFINITY;
                }
              }
              const float bm = max64(sv) * a.scale_log2;
              const bool raise = bm > m + gap;
              if (__any_sync(0xffffffffu, raise)) {
                if (hf) {  // (the first half's product has to be done)
                  ok = wait(&c.lo_done[h], i & 1);
                  if (!ok) break;
                  tc_fence_after();
                }
                const float f = raise ? (m == -INFINITY ? 0.f : ex2_approx(m - bm)) : 1.f;
                tmem_st_wait();
                if (i > 0 || hf) scale_o(tO, f);
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
    if (n && ok) ok = wait(&c.o_full[h], 0);
    if (!ok) l = 0.f;  // (what is joined then is undefined, and flagged)
    c.m[h][r] = m;
    c.l[h][r] = l;
  }
  // Every product is done and every copy has landed: the ring's memory is free.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp >= 4) {
    const bool some = __any_sync(0xffffffffu, c.l[h][r] != 0.f);
    if (some) {
      const uint32_t piece = sbase + kTOffKV + h * kTPiece;
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        float ov[32];
        tmem_ld32(tO + cb * 32, ov);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_shared_v4(piece + piece_at(r, cb * 8 + k), __float_as_uint(ov[4 * k]), __float_as_uint(ov[4 * k + 1]),
                       __float_as_uint(ov[4 * k + 2]), __float_as_uint(ov[4 * k + 3]));
      }
    }
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp >= 4 && c.tile.ntok) {
    // --------------------------------------------------------------- the join
    // A warp takes a row at a time, a lane four columns; lane q < 2 C has
    // piece q's maximum and sum (CTA q / 2, group q % 2).  A piece without keys
    // holds no O.
    const TTile t = c.tile;
    const int rows = t.ntok * a.G;
    const uint32_t ms = smem_u32(&c.m[0][0]), ls = smem_u32(&c.l[0][0]), ring = sbase + kTOffKV;
    for (int row = rank + (warp - 4) * C; row < rows; row += 8 * C) {
      float mq = -INFINITY, lq = 0.f;
      if (lane < 2 * C) {
        mq = ld_cluster(in_cta(ms + ((lane & 1) * 128 + row) * 4, lane >> 1));
        lq = ld_cluster(in_cta(ls + ((lane & 1) * 128 + row) * 4, lane >> 1));
      }
      float M = lq == 0.f ? -INFINITY : mq;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float wq = lq == 0.f ? 0.f : (M == -INFINITY ? 1.f : ex2_approx(mq - M));
      float L = lq * wq;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (unsigned left = __ballot_sync(0xffffffffu, lq != 0.f); left; left &= left - 1) {
        const int q = __ffs(left) - 1;
        const float w = __shfl_sync(0xffffffffu, wq, q);
        const float4 v = ld_cluster_v4(in_cta(ring + (q & 1) * kTPiece + piece_at(row, lane), q >> 1));
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;  // (a NaN stays one)
      const int rt = row / a.G, head = t.g * a.G + row - rt * a.G;
      const size_t tok = (size_t)t.tok0 + rt;
      reinterpret_cast<uint2*>(a.out + (tok * a.Hq + head) * 256)[lane] =
          make_uint2(hpack2<kBf16>(o.x * inv, o.y * inv), hpack2<kBf16>(o.z * inv, o.w * inv));
      if (a.lse && lane == 0)
        a.lse[(size_t)head * a.total_q + tok] =
            L == 0.f ? -INFINITY : ((M == -INFINITY ? 0.f : M) + lg2_approx(L)) * 0.69314718055994530942f;
    }
  }
  cluster_sync();  // no CTA leaves while another reads its memory
  if (warp == kTMma) tmem_dealloc(tmem, 512);
}

}  // namespace

// The cluster's size where the one-launch path is taken, 0 where it is not.  As
// large as leaves all clusters of the row tiles on the SMs at once (of 8 CTAs 14
// do, 16 took twice as long).  Tiles are counted as if the sequences had equally
// many tokens (more of them only wait for their turn).  A cluster's own keys cost
// 0.8 us a block and CTA, the general path's plan and join 8 to 15 us; the fewer
// SMs the clusters leave idle, the later the general path, which uses all of
// them, is ahead.  The host knows the tables' width and not the lengths: the
// limits are widths at which the longest tables' worth of keys took no longer
// here (5% for the spread), and shorter sequences in such tables gain up to
// twofold.  Microseconds of this and of the general path, page 64, lengths from a
// third of L to L, inputs from memory:
//   C = 8, 2 tiles (one sequence of 5 tokens, 16 + 2 heads): L 1000 8 and 16, 8000
//   17 and 30, 16000 23 and 42, 24000 30 and 45, 64000 63 and 52; 1 tile (8 + 1):
//   16000 22 and 24, 24000 29 and 28; 4 tiles (8 tokens, 12 + 4): 16000 23 and 25,
//   24000 30 and 28; 8 tiles (60 tokens, 16 + 2): 16000 28 and 30, 24000 35 and 31;
//   10 to 14 tiles: 24000 31 and 36, 35 and 38, 36 and 36, 38 and 43;
//   C = 4, 16 and 20 tiles: 8000 28 and 28, 27 and 29, 16000 42 and 39, 41 and 39; 24
//   to 32 tiles: 16000 38 and 40, 45 and 48, 42 and 47, 24000 51 and 48, 57 and 55;
//   C = 2, 40 to 72 tiles: 8000 42 and 41, 44 and 46, 47 and 50, 44 and 55, 16000 66
//   and 64, 73 and 72, 77 and 82, 24000 109 and 107;
//   C = 1, 80 to 104 tiles: 4000 43 and 46, 46 and 47, 46 and 53, 8000 69 and 58, 75
//   and 75; 109 to 152 tiles: 8000 74 and 78, 72 and 75, 82 and 91, 84 and 98, 16000
//   134 and 120; 110 sequences of 20 tokens, 8 + 1 heads, which are 138 tiles in
//   number but 220 as they lie: 4000 73 and 69, 8000 114 and 97.
// Where several row tiles read the same keys the general path, which takes two of
// a sequence at a time, is ahead earlier: 5 sequences of 8 tokens, 128 + 1 heads
// (C = 2), 4000 28 and 27, 8000 42 and 33; 6 of 14, 64 + 4, 8000 42 and 36.
int tree_small_cluster(const mxsa_problem& p, int num_groups) {
  if (num_groups > 0) return 0;
  const long long T = 128 / (p.num_q_heads / p.num_kv_heads), B = p.num_seqs;
  const long long tiles = std::max(B, (p.total_q + T - 1) / T) * p.num_kv_heads;
  // (as they lie, where the sequences have equally many tokens: none has two sequences' rows)
  const long long whole = B * (((p.total_q + B - 1) / B + T - 1) / T) * p.num_kv_heads;
  const long long blocks = max_blocks_per_seq(p);
  // Up to so many tiles; for tables of up to so many blocks, and of more with at
  // least so many tiles that do all have their SMs.
  struct Rule {
    int cluster, tiles, blocks, many, many_blocks;
  };
  for (const Rule r : {Rule{8, 14, 128, 9, 192}, Rule{4, 32, 64, 23, 128}, Rule{2, 72, 64, 0, 64},
                       Rule{1, 152, 32, 109, 64}})
    if (tiles <= r.tiles)
      return blocks <= (tiles >= r.many && whole <= r.tiles ? r.many_blocks : r.blocks) ? r.cluster : 0;
  return 0;
}

cudaError_t launch_tree_small(const mxsa_problem& p, int cluster, const void* q, const void* k_cache,
                              const void* v_cache, const int32_t* block_tables, const int64_t* cu, const int32_t* lens,
                              const uint32_t* mask, int words, void* out, float* lse, int32_t* flags,
                              cudaStream_t st) {
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
  CUtensorMap tmq, tmk, tmv;
  const cuuint64_t slabs = (cuuint64_t)p.num_pages * p.num_kv_heads;
  if (!map3(&tmq, q, p.num_q_heads, p.total_q, G, T) || !map3(&tmk, k_cache, p.page_size, slabs, p.page_size, 1) ||
      !map3(&tmv, v_cache, p.page_size, slabs, p.page_size, 1))
    return cudaErrorInvalidValue;
  const size_t smem = kTOffCtrl + sizeof(TCtrl) + 1024;
  static PerDevice limits;
  const cudaError_t e = limits([smem] {
    const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const cudaError_t x = cudaFuncSetAttribute(k_tree_small<true>, a, (int)smem);
    return x == cudaSuccess ? cudaFuncSetAttribute(k_tree_small<false>, a, (int)smem) : x;
  });
  if (e != cudaSuccess) return e;
  TArgs a{};
  a.cu = cu;
  a.lens = lens;
  a.block_tables = block_tables;
  a.mask = mask;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.flags = flags;
  a.num_seqs = p.num_seqs;
  a.total_q = p.total_q;
  a.Hq = p.num_q_heads;
  a.Hkv = p.num_kv_heads;
  a.G = G;
  a.T = T;
  a.page_shift = p.page_size == 128 ? 7 : 6;
  a.max_pages = p.max_pages_per_seq;
  a.num_pages = p.num_pages;
  a.words = words;
  a.cluster = cluster;
  const float scale = p.softmax_scale > 0.f ? p.softmax_scale : 0.08838834764831845f;  // 1/sqrt(128)
  a.scale_log2 = scale * 1.4426950408889634f;
  const long long tiles = ((long long)p.total_q / T + p.num_seqs) * p.num_kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(kTThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, bf16 ? k_tree_small<true> : k_tree_small<false>, tmq, tmk, tmv, a);
}

}  // namespace mxsa

#ifdef MXSA_TEST_HOOKS
// Test builds only: the CTA of the next tree_fwd launches (one-launch path) that
// keeps its tile to itself; -1 turns the switch off.  Synchronous.
extern "C" mxsa_status mxsa_test_skip_found(int32_t cta) {
  return cudaMemcpyToSymbol(mxsa::g_skip_found, &cta, sizeof(cta)) == cudaSuccess ? MXSA_OK : MXSA_ERR_CUDA;
}
#endif

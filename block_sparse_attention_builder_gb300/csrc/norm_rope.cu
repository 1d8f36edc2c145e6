// The prologue of an attention layer over the paged caches: every query and
// key head is normed and rotated by its token's position, and K, V and the
// index keys go into the caches in the same pass.
//
// Per head row x of D = 128 (index rows: 64 or 128) values, with weight w and
// the token's cosines c_i and sines s_i, i < R / 2 (R = rot_dim):
//     y = x / sqrt(mean(x^2) + eps) * w
//     (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i),
//         a, b = i, i + R / 2   (interleaved: 2 i, 2 i + 1)
// in FP32, rounded once: into q's type for q_out and a 16-bit cache, else by
// the cache's cast (the store's, applied to the FP32 value).  V rows are cast
// as they are.
//
// Bound: HBM.  Each row is read once and written once; a token's cosines and
// sines (up to 512 bytes) and the weight rows come from L1/L2.  Sixteen lanes
// hold a row (eight an index row of 64), two pieces of 4 values each.  With
// pairs (i, i + R / 2) a lane's pieces are the two halves of its pairs, so the
// rotation needs no other lane; otherwise they are neighbours.  A half-warp
// takes kRopeRows rows of one token: that many loads are in flight per lane,
// and position, slot, cosines, sines and shared weights are read once.
//
// What held it back was instructions, 221 per 32 lanes of 8 values (68% of the
// issue slots, DRAM at 42%), until the arithmetic was packed in pairs, the
// row addresses became steps and each half-warp its own shuffle group.
// 32768 tokens of 64 + 8 + 8 heads, bf16 (1.36 GB, 203 us at the copy rate):
// 386 us with sixteen consecutive bytes to a lane and the partner's bytes by
// shuffle, each value normed twice; 324 us with a lane's pieces as above (runs
// of a token's rows with the next rows prefetched: 340 us); 240 us, 5.7 TB/s,
// now.  2 or 8 rows at a time: 294 and 332 us.  FP8 cache 257 us (193 us at
// the copy rate), NVFP4 341 us (189 us; its casts are 100 us of it: 452 us
// with a division and the comparisons for each value).  All forms but NVFP4
// with pairs side by side spill registers, 36 to 84 bytes stored and 52 to 248
// loaded a thread (the most: FP8 with pairs (i, i + R/2)), which takes issue
// slots too; launch bounds with more registers, and fewer warps, were slower.
#include <algorithm>
#include <climits>

#include "cast.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mxsa {

namespace {

constexpr int kRopeRows = 4;      // rows of a task
constexpr int kRopeThreads = 256;

// what a part's rows become
enum : int { kDstDense16 = 0, kDstDenseCast = 1, kDstCache = 2 };

struct RopePart {
  const uint16_t* src;
  const uint16_t* w;   // null: no norm
  uint8_t* dst;
  long long stride;    // elements between tokens
  int32_t heads, dim, tasks;  // tasks: kRopeRows x 16 lanes of one token's rows
  int32_t dst_kind, rotate, w_stride;
};

struct RopeArgs {
  RopePart part[5];    // q, k, v, index q, index k (tasks 0: absent)
  const int64_t* positions;
  const int64_t* loc;
  const float* cos_sin;
  int32_t* flags;      // may be null
  long long num_positions, slots;
  uint32_t total;      // tasks of this launch
  int32_t per_token, rot, page_shift;
  float eps;
};

// four packed 16-bit values as two pairs
template <bool kBf16>
__device__ __forceinline__ void unpack4(const uint2& s, uint64_t* x) {
  const uint32_t w[2] = {s.x, s.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (kBf16) {
      x[i] = pack_f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[i] = pack_f2(f.x, f.y);
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint2 pack4(const uint64_t* y) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = unpack_f2(y[i]);
    if (kBf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(f.x, f.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t pack4_e4m3(const uint64_t* y) {
  const float2 f = unpack_f2(y[0]), g = unpack_f2(y[1]);
  return e4m3_code2(f.x, f.y) | (e4m3_code2(g.x, g.y) << 16);
}

// kKind: the caches' kind.  kInter: rotated pairs side by side.
template <int kKind, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kKind == kKindFp4 ? 4 : 5) k_norm_rope(const __grid_constant__ RopeArgs a) {
  // a lane's pieces are the halves of its pairs; not for NVFP4, whose groups
  // of 16 values are then two neighbouring lanes
  constexpr bool kPair = !kInter && kKind != kKindFp4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, hl = lane & 15;
  const uint32_t hmask = 0xFFFFu << (lane & 16);  // the half-warp: all of it takes the same way below
  const uint32_t task = blockIdx.x * (kRopeThreads / 16) + (threadIdx.x >> 4);
  if (task >= a.total) return;
  const uint32_t t = task / (uint32_t)a.per_token;
  int r = (int)(task - t * (uint32_t)a.per_token), pi = 0;
  while (r >= a.part[pi].tasks) r -= a.part[pi++].tasks;
  const RopePart& p = a.part[pi];
  const int lpr = p.dim >> 3;         // lanes of a row: 16 or 8
  const int rpp = lpr == 16 ? 1 : 2;  // rows side by side in 16 lanes
  const int l = hl & (lpr - 1);
  const int h0 = r * (kRopeRows * rpp) + (lpr == 16 ? 0 : hl >> 3);
  const int left = (p.heads - h0 + rpp - 1) / rpp;  // rows of the lane's column, at most kRopeRows of them here
  // first columns of the lane's two pieces
  const int half = a.rot >> 1;
  int ea = 8 * l, eb = 8 * l + 4;
  bool turn = p.rotate && ea < a.rot;
  if (kPair && p.rotate) {
    const int turning = half >> 2;  // lanes that hold pairs
    turn = l < turning;
    ea = turn ? 4 * l : a.rot + 8 * (l - turning);
    eb = turn ? ea + half : ea + 4;
  }

  // the rows first: nothing they need waits for the position
  uint2 ra[kRopeRows], rb[kRopeRows];
  const uint16_t* src = p.src + (long long)t * p.stride + h0 * p.dim;
  const int step = rpp * p.dim;
#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    ra[u] = rb[u] = make_uint2(0, 0);
    if (u < left) {
      ra[u] = *reinterpret_cast<const uint2*>(src + u * step + ea);
      rb[u] = *reinterpret_cast<const uint2*>(src + u * step + eb);
    }
  }
  const long long pos = a.positions[t];
  if (pos < 0) return;  // padding: the token is left out
  if (pos >= a.num_positions) {
    if (a.flags && pi == 0 && r == 0 && hl == 0) atomicOr(a.flags, MXSA_FLAG_POS);
    return;
  }
  // where the first row goes, and the bytes from one row to the next
  const int es = kKind == kKindFp8 && p.dst_kind != kDstDense16 ? 1 : 2;
  uint8_t* dst = p.dst + ((long long)t * p.heads + h0) * (p.dim * es);
  long long dstep = step * es, off = 0;
  if (p.dst_kind == kDstCache) {
    const long long slot = a.loc[t];
    if (slot >= a.slots && a.flags && pi == 1 && r == 0 && hl == 0) atomicOr(a.flags, MXSA_FLAG_PAGE);
    if (slot < 0 || slot >= a.slots) return;
    off = slot & ((1LL << a.page_shift) - 1);
    const long long slab = (slot >> a.page_shift) * p.heads + h0;
    if (kKind == kKindFp4) {
      dst = p.dst + slab * (72LL << a.page_shift);
      dstep = (72LL * rpp) << a.page_shift;
    } else {
      dst = p.dst + (slab << a.page_shift | off) * (p.dim * es);
      dstep <<= a.page_shift;
    }
  }

  if (!p.rotate && kKind != kKindFp4) {  // V: the store's own cast
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u)
      if (u < left)
        put_chunk(make_uint4(ra[u].x, ra[u].y, rb[u].x, rb[u].y), dst + u * dstep, ea, kKind == kKindFp8, kBf16);
    return;
  }

  // Cosines and sines of the lane's four pairs.  kPair: as pairs of
  // neighbours.  Side by side: each twice, the sines' first copy negated.
  // NVFP4 with pairs (i, i + R/2): of its eight columns, the sines signed for
  // the partner's value.
  constexpr int kAngles = kPair ? 2 : 4;
  uint64_t c[kAngles], s[kAngles], w[4];
  if (turn) {
    const float* cs = a.cos_sin + pos * a.rot;
    const int j = kPair ? ea : (kInter ? ea >> 1 : (ea < half ? ea : ea - half));
    const float sign = !kPair && !kInter && ea < half ? -1.f : 1.f;
#pragma unroll
    for (int i = 0; i < (kPair || kInter ? 1 : 2); ++i) {
      const float4 cv = reinterpret_cast<const float4*>(cs + j)[i];
      const float4 sv = reinterpret_cast<const float4*>(cs + half + j)[i];
      if (kInter) {
        c[0] = pack_f2(cv.x, cv.x), c[1] = pack_f2(cv.y, cv.y), c[2] = pack_f2(cv.z, cv.z), c[3] = pack_f2(cv.w, cv.w);
        s[0] = pack_f2(-sv.x, sv.x), s[1] = pack_f2(-sv.y, sv.y);
        s[2] = pack_f2(-sv.z, sv.z), s[3] = pack_f2(-sv.w, sv.w);
      } else {
        c[2 * i] = pack_f2(cv.x, cv.y), c[2 * i + 1] = pack_f2(cv.z, cv.w);
        s[2 * i] = pack_f2(sign * sv.x, sign * sv.y), s[2 * i + 1] = pack_f2(sign * sv.z, sign * sv.w);
      }
    }
  }
  const uint16_t* wr = p.w + h0 * p.w_stride;
  auto load_weights = [&](int u) {
    unpack4<kBf16>(*reinterpret_cast<const uint2*>(wr + u * rpp * p.w_stride + ea), w);
    unpack4<kBf16>(*reinterpret_cast<const uint2*>(wr + u * rpp * p.w_stride + eb), w + 2);
  };
  if (p.w && p.w_stride == 0) load_weights(0);

#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    // (rows past the last head hold zeros and are not written; the lanes keep
    // to the half-warp's shuffles)
    uint64_t y[4];
    unpack4<kBf16>(ra[u], y);
    unpack4<kBf16>(rb[u], y + 2);
    if (p.w) {
      const float2 s2 = unpack_f2(fma_f2(y[3], y[3], fma_f2(y[2], y[2], fma_f2(y[1], y[1], mul_f2(y[0], y[0])))));
      float ss = s2.x + s2.y;
      ss += __shfl_xor_sync(hmask, ss, 1);
      ss += __shfl_xor_sync(hmask, ss, 2);
      ss += __shfl_xor_sync(hmask, ss, 4);
      if (lpr == 16) ss += __shfl_xor_sync(hmask, ss, 8);
      const float rms = rsqrtf(fmaf(ss, lpr == 16 ? 1.f / 128 : 1.f / 64, a.eps));
      if (p.w_stride && u < left) load_weights(u);
      const uint64_t rms2 = pack_f2(rms, rms);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul_f2(mul_f2(y[i], rms2), w[i]);
    }
    if (kPair) {
      if (turn) {  // (columns past R keep infinities and NaN to themselves)
        const uint64_t minus = pack_f2(-1.f, -1.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t ya = y[i], yb = y[i + 2];
          y[i] = fma_f2(mul_f2(yb, s[i]), minus, mul_f2(ya, c[i]));
          y[i + 2] = fma_f2(ya, s[i], mul_f2(yb, c[i]));
        }
      }
    } else if (kInter) {
      if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack_f2(y[i]);
          y[i] = fma_f2(pack_f2(f.y, f.x), s[i & (kAngles - 1)], mul_f2(y[i], c[i & (kAngles - 1)]));
        }
      }
    } else {
      const int partner = turn ? (ea < half ? lane + (half >> 3) : lane - (half >> 3)) : lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t o = __shfl_sync(hmask, y[i], partner);
        if (turn) y[i] = fma_f2(o, s[i & (kAngles - 1)], mul_f2(y[i], c[i & (kAngles - 1)]));
      }
    }
    uint8_t* to = dst + u * dstep;
    if (kKind == kKindFp4 && p.dst_kind == kDstCache) {
      float x[8], amax = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_f2(y[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));  // fmaxf drops a NaN operand
      }
      amax = fmaxf(amax, __shfl_xor_sync(hmask, amax, 1));
      float sd;
      const uint32_t sc = nvfp4_scale(amax, &sd);
      const uint32_t codes = nvfp4_codes8(x, sd);
      if (u < left) {
        *reinterpret_cast<uint32_t*>(to + off * 64 + (ea >> 1)) = codes;
        if (!(lane & 1)) to[(64LL << a.page_shift) + off * 8 + (ea >> 4)] = (uint8_t)sc;
      }
    } else if (u < left) {
      if (es == 1) {
        *reinterpret_cast<uint32_t*>(to + ea) = pack4_e4m3(y);
        *reinterpret_cast<uint32_t*>(to + eb) = pack4_e4m3(y + 2);
      } else {
        *reinterpret_cast<uint2*>(to + 2 * ea) = pack4<kBf16>(y);
        *reinterpret_cast<uint2*>(to + 2 * eb) = pack4<kBf16>(y + 2);
      }
    }
  }
}

template <int kKind, bool kBf16>
cudaError_t launch_kind(const RopeArgs& a, bool inter, unsigned blocks, cudaStream_t st) {
  auto* kern = inter ? k_norm_rope<kKind, kBf16, true> : k_norm_rope<kKind, kBf16, false>;
  return launch_pdl(kern, dim3(blocks), dim3(kRopeThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_norm_rope(const mxsa_problem& p, const mxsa_norm_rope& cfg, const NormRopePtrs& b, long long n,
                             cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  RopeArgs a{};
  auto set = [&](int i, const void* src, const void* w, void* dst, long long stride, int heads, int dim, int dst_kind,
                 int rotate) {
    RopePart& q = a.part[i];
    q.src = static_cast<const uint16_t*>(src);
    q.w = static_cast<const uint16_t*>(w);
    q.dst = static_cast<uint8_t*>(dst);
    q.stride = stride;
    q.heads = heads;
    q.dim = dim;
    const int rows = kRopeRows * (dim == 64 ? 2 : 1);
    q.tasks = (heads + rows - 1) / rows;
    q.dst_kind = dst_kind;
    q.rotate = rotate;
    q.w_stride = cfg.weight_per_head ? dim : 0;
    a.per_token += q.tasks;
  };
  set(0, b.q, b.q_weight, b.q_out, cfg.q_stride, p.num_q_heads, 128, kDstDense16, 1);
  set(1, b.k, b.k_weight, b.k_cache, cfg.k_stride, p.num_kv_heads, 128, kDstCache, 1);
  set(2, b.v, nullptr, b.v_cache, cfg.v_stride, p.num_kv_heads, 128, kDstCache, 0);
  if (cfg.idx_dim) {
    set(3, b.idx_q, b.idx_q_weight, b.idx_q_out, cfg.idx_q_stride, p.num_kv_heads, cfg.idx_dim, kDstDenseCast, 1);
    set(4, b.idx_k, b.idx_k_weight, b.idx_cache, cfg.idx_k_stride, p.num_kv_heads, cfg.idx_dim, kDstCache, 1);
  }
  a.cos_sin = b.cos_sin;
  a.flags = b.flags;
  a.num_positions = cfg.num_positions;
  a.slots = (long long)p.num_pages * p.page_size;
  a.rot = cfg.rot_dim;
  a.page_shift = p.page_size == 128 ? 7 : 6;
  a.eps = cfg.eps;
  const int out_bytes[2] = {p.num_q_heads * 256, cfg.idx_dim * p.num_kv_heads * (p.kv_dtype == MXSA_FP8_E4M3 ? 1 : 2)};
  // 32-bit task numbers: a launch takes the tokens that fit them
  const long long max_tokens = std::max(1LL, (long long)INT32_MAX / a.per_token);
  RopePart base[5];
  std::copy(a.part, a.part + 5, base);
  for (long long t0 = 0; t0 < n; t0 += max_tokens) {
    const long long m = std::min(max_tokens, n - t0);
    for (int i = 0; i < 5; ++i)
      if (base[i].tasks) a.part[i].src = base[i].src + t0 * base[i].stride;
    a.part[0].dst = base[0].dst + t0 * out_bytes[0];
    if (cfg.idx_dim) a.part[3].dst = base[3].dst + t0 * out_bytes[1];
    a.positions = b.positions + t0;
    a.loc = b.loc + t0;
    a.total = (uint32_t)(m * a.per_token);
    const unsigned blocks = (a.total + kRopeThreads / 16 - 1) / (kRopeThreads / 16);
    const bool bf16 = p.q_dtype == MXSA_BF16, inter = cfg.interleaved != 0;
    cudaError_t e;
    switch (cache_kind(p)) {
      case kKindFp8: e = bf16 ? launch_kind<kKindFp8, true>(a, inter, blocks, st)
                              : launch_kind<kKindFp8, false>(a, inter, blocks, st); break;
      case kKindFp4: e = bf16 ? launch_kind<kKindFp4, true>(a, inter, blocks, st)
                              : launch_kind<kKindFp4, false>(a, inter, blocks, st); break;
      default: e = bf16 ? launch_kind<kKind16, true>(a, inter, blocks, st)
                        : launch_kind<kKind16, false>(a, inter, blocks, st);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mxsa

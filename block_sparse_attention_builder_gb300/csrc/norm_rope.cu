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
// hold a row, 8 values (16 bytes) each, so a row's loads and stores are whole
// lines, its sum of squares is four shuffles, and a partner half is one
// shuffle of the raw 16 bytes away (4 registers, not 8 normed floats).  A
// half-warp takes kRopeRows rows of one token: that many 16-byte loads are in
// flight per lane, and the cosines, sines and weights are read once for them.
#include <algorithm>
#include <climits>

#include "cast.cuh"
#include "internal.h"

namespace mxsa {

namespace {

constexpr int kRopeRows = 4;      // rows of a 16-lane group
constexpr int kRopeThreads = 256;

// what a part's rows become
enum : int { kDstDense16 = 0, kDstDenseCast = 1, kDstCache = 2 };

struct RopePart {
  const uint16_t* src;
  const uint16_t* w;   // null: no norm
  uint8_t* dst;
  long long stride;    // elements between tokens
  int32_t heads, dim, tasks;  // tasks: 16-lane groups of one token
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

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& s, float* x) {
  const uint32_t w[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint4 pack8(const float* y) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 pack8_e4m3(const float* y) {
  return make_uint2(e4m3_code2(y[0], y[1]) | (e4m3_code2(y[2], y[3]) << 16),
                    e4m3_code2(y[4], y[5]) | (e4m3_code2(y[6], y[7]) << 16));
}

// kKind: the caches' kind.  kInter: rotated pairs side by side.
template <int kKind, bool kBf16, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) k_norm_rope(const __grid_constant__ RopeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, hl = lane & 15;
  uint32_t task = blockIdx.x * (kRopeThreads / 16) + (threadIdx.x >> 4);
  bool live = task < a.total;
  if (!live) task = 0;  // keeps its lanes for the warp's shuffles
  const uint32_t t = task / (uint32_t)a.per_token;
  int r = (int)(task - t * (uint32_t)a.per_token), pi = 0;
  while (r >= a.part[pi].tasks) r -= a.part[pi++].tasks;
  const RopePart& p = a.part[pi];
  const int lpr = p.dim >> 3;        // lanes of a row: 16 or 8
  const int rpp = lpr == 16 ? 1 : 2; // rows side by side in 16 lanes
  const int e = (hl & (lpr - 1)) * 8;
  const int h0 = r * (kRopeRows * rpp) + (lpr == 16 ? 0 : hl >> 3);

  // the rows first: nothing they need waits for the position
  uint4 raw[kRopeRows];
  const uint16_t* src = p.src + (long long)t * p.stride + e;
#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    const int h = h0 + u * rpp;
    raw[u] = live && h < p.heads ? *reinterpret_cast<const uint4*>(src + (long long)h * p.dim)
                                 : make_uint4(0, 0, 0, 0);
  }
  const long long pos = a.positions[t];
  if (pos < 0) live = false;  // padding: the token is left out
  if (pos >= a.num_positions) {
    if (live && a.flags && pi == 0 && r == 0 && hl == 0) atomicOr(a.flags, MXSA_FLAG_POS);
    live = false;
  }
  long long page = 0, off = 0;
  if (p.dst_kind == kDstCache) {
    const long long l = a.loc[t];
    if (l >= a.slots && live && a.flags && pi == 1 && r == 0 && hl == 0) atomicOr(a.flags, MXSA_FLAG_PAGE);
    if (l < 0 || l >= a.slots) live = false;
    page = l >> a.page_shift;
    off = l & ((1LL << a.page_shift) - 1);
  }

  const int half = a.rot >> 1;
  const bool turn = p.rotate && e < a.rot;
  float c[8], s[8];  // interleaved: the first four of each
  if (turn && live) {
    const float* cs = a.cos_sin + pos * a.rot;
    const int j = kInter ? e >> 1 : (e < half ? e : e - half);
#pragma unroll
    for (int i = 0; i < (kInter ? 1 : 2); ++i) {
      const float4 cv = reinterpret_cast<const float4*>(cs + j)[i];
      const float4 sv = reinterpret_cast<const float4*>(cs + half + j)[i];
      c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
      s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  }
  // half layout: the lane that holds the other value of this lane's pairs
  const int step = half >> 3;
  const int partner = turn ? (e < half ? lane + step : lane - step) : lane;
  const int pe = turn ? (e < half ? e + half : e - half) : e;  // its first column
  const float sign = e < half ? -1.f : 1.f;

#pragma unroll
  for (int u = 0; u < kRopeRows; ++u) {
    const int h = h0 + u * rpp;
    const bool row = live && h < p.heads;
    float x[8], y[8];
    unpack8<kBf16>(raw[u], x);
    // every lane of the warp takes part in the shuffles: its two halves may
    // hold rows of different parts
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    ss += __shfl_xor_sync(0xffffffffu, ss, 4);
    const float side = __shfl_xor_sync(0xffffffffu, ss, 8);
    if (lpr == 16) ss += side;
    const float rms = __frsqrt_rn(ss / (float)p.dim + a.eps);
    uint4 other = raw[u];
    if (!kInter) {
      other.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
      other.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
      other.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
      other.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
    }
    if (p.w && row) {
      const uint16_t* wr = p.w + (long long)h * p.w_stride;
      float w[8];
      unpack8<kBf16>(*reinterpret_cast<const uint4*>(wr + e), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i] * rms * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = x[i];
    }
    if (turn) {
      if (kInter) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float ya = y[2 * i], yb = y[2 * i + 1];
          y[2 * i] = ya * c[i] - yb * s[i];
          y[2 * i + 1] = yb * c[i] + ya * s[i];
        }
      } else {
        float yo[8];
        unpack8<kBf16>(other, yo);
        if (p.w && row) {
          float w[8];
          unpack8<kBf16>(*reinterpret_cast<const uint4*>(p.w + (long long)h * p.w_stride + pe), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) yo[i] = yo[i] * rms * w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * c[i] + sign * yo[i] * s[i];
      }
    }
    float amax = 0.f;
    if (kKind == kKindFp4) {  // a group of 16 values is two lanes
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(y[i]));  // fmaxf drops a NaN operand
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    }
    if (p.dst_kind == kDstCache) {
      const long long at = page * p.heads + h;  // (page, head) slab
      if (kKind == kKindFp4) {
        if (row) {
          float sd;
          const uint32_t sc = nvfp4_scale(amax, &sd);
          uint32_t codes = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) codes |= nvfp4_code(y[i], sd) << (4 * i);
          uint8_t* slab = p.dst + at * (72LL << a.page_shift);
          *reinterpret_cast<uint32_t*>(slab + off * 64 + (e >> 1)) = codes;
          if (!(lane & 1)) slab[(64LL << a.page_shift) + off * 8 + (e >> 4)] = (uint8_t)sc;
        }
      } else if (row) {
        const long long elem = (at << a.page_shift | off) * p.dim + e;
        if (!p.rotate) put_chunk(raw[u], p.dst, elem, kKind == kKindFp8, kBf16);  // V: the store's own cast
        else if (kKind == kKindFp8) *reinterpret_cast<uint2*>(p.dst + elem) = pack8_e4m3(y);
        else *reinterpret_cast<uint4*>(p.dst + 2 * elem) = pack8<kBf16>(y);
      }
    } else if (row) {
      const long long elem = ((long long)t * p.heads + h) * p.dim + e;
      if (kKind == kKindFp8 && p.dst_kind == kDstDenseCast)
        *reinterpret_cast<uint2*>(p.dst + elem) = pack8_e4m3(y);
      else
        *reinterpret_cast<uint4*>(p.dst + 2 * elem) = pack8<kBf16>(y);
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

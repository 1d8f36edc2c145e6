// Paged-cache load: the read side of the store.  Row (t, h) of the output
// [n][heads][dim] is the cache row of slot loc[t], page = loc[t] / page_size,
// offset = loc[t] % page_size, widened to the 16-bit type exactly: every
// e4m3 value, and every product of an E2M1 value and an E4M3 scale (at most
// 6 significant bits, 2^-10 .. 2688), is a bf16 and an fp16 value.
//
// Bound: HBM, the cached rows once and the 16-bit rows once.  One thread
// makes 16 output bytes (8 values) of K and the same 8 of V, and the index
// keys' chunks follow, as in the store: consecutive threads read and write
// consecutive bytes, and the slot is looked up once for both.  36864 tokens
// of 8 heads, e4m3 (227 MB): 37.4 us, 6.1 TB/s; 30011 of 4 heads, NVFP4 (79
// MB): 16.1 us, 4.9 TB/s with the launch.
#include <algorithm>
#include <climits>

#include "cast.cuh"
#include "internal.h"

namespace mxsa {

namespace {

struct LoadArgs {
  const int64_t* loc;
  const uint8_t* src[3];   // K, V, index-key caches
  uint8_t* dst[3];         // 16-bit rows of this launch's first token
  int32_t heads[2];        // K / V, index keys
  int32_t row_chunks[2];   // dim / 8
  int32_t rc_shift[2], heads_shift[2];
  uint32_t chunks[2];
  long long slots;
  int32_t page_shift;
  int32_t* flags;          // may be null
};

// packed halves to packed values of the 16-bit type
template <bool kBf16>
__device__ __forceinline__ uint32_t from_f16x2(uint32_t h2) {
  if (!kBf16) return h2;
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// the 8 values of chunk `part` of the row at (slab, off)
template <int kKind, bool kBf16>
__device__ __forceinline__ uint4 get_chunk(const uint8_t* cache, long long slab, long long off, int page_shift,
                                           uint32_t rc, uint32_t part) {
  if (kKind == kKindFp4) {
    const uint8_t* s = cache + slab * (72LL << page_shift);
    const uint32_t codes = __ldcs(reinterpret_cast<const uint32_t*>(s + off * 64 + 4 * part));
    const uint32_t sc = __ldcs(s + (64LL << page_shift) + off * 8 + (part >> 1));
    const uint32_t sd = e4m3x2_to_f16x2((uint16_t)(sc | (sc << 8)));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t v;
      asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(v) : "r"(codes >> (8 * i)));
      const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&sd));
      o[i] = from_f16x2<kBf16>(*reinterpret_cast<const uint32_t*>(&p));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
  const long long elem = (slab << page_shift | off) * (8LL * rc) + 8LL * part;
  if (kKind == kKindFp8) {
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(cache + elem));
    return make_uint4(from_f16x2<kBf16>(e4m3x2_to_f16x2((uint16_t)c.x)),
                      from_f16x2<kBf16>(e4m3x2_to_f16x2((uint16_t)(c.x >> 16))),
                      from_f16x2<kBf16>(e4m3x2_to_f16x2((uint16_t)c.y)),
                      from_f16x2<kBf16>(e4m3x2_to_f16x2((uint16_t)(c.y >> 16))));
  }
  return __ldcs(reinterpret_cast<const uint4*>(cache + 2 * elem));
}

template <int kKind, bool kBf16>
__global__ void __launch_bounds__(256) k_load(LoadArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t total = a.chunks[0] + a.chunks[1];
  const uint32_t stride = gridDim.x * blockDim.x;
  for (uint32_t c = blockIdx.x * blockDim.x + threadIdx.x; c < total; c += stride) {
    const bool kv = c < a.chunks[0];
    const uint32_t cc = kv ? c : c - a.chunks[0];
    const uint32_t rc = (uint32_t)(kv ? a.row_chunks[0] : a.row_chunks[1]);
    const uint32_t heads = (uint32_t)(kv ? a.heads[0] : a.heads[1]);
    const int rcs = kv ? a.rc_shift[0] : a.rc_shift[1];
    const int hs = kv ? a.heads_shift[0] : a.heads_shift[1];
    const uint32_t row = rcs >= 0 ? cc >> rcs : cc / rc, part = cc - row * rc;
    const uint32_t t = hs >= 0 ? row >> hs : row / heads, h = row - t * heads;
    const long long l = a.loc[t];
    if (l < 0) continue;  // the token's rows are left as they are
    if (l >= a.slots) {
      if (a.flags && kv && h == 0 && part == 0) atomicOr(a.flags, MXSA_FLAG_PAGE);
      continue;
    }
    const long long off = l & ((1LL << a.page_shift) - 1);
    const long long slab = (l >> a.page_shift) * heads + h;
    if (kv) {
      const uint4 k = get_chunk<kKind, kBf16>(a.src[0], slab, off, a.page_shift, rc, part);
      const uint4 v = get_chunk<kKind, kBf16>(a.src[1], slab, off, a.page_shift, rc, part);
      reinterpret_cast<uint4*>(a.dst[0])[cc] = k;
      reinterpret_cast<uint4*>(a.dst[1])[cc] = v;
    } else if (kKind != kKindFp4) {  // (no NVFP4 index keys)
      reinterpret_cast<uint4*>(a.dst[2])[cc] =
          get_chunk<kKind, kBf16>(a.src[2], slab, off, a.page_shift, rc, part);
    }
  }
}

}  // namespace

cudaError_t launch_load(const mxsa_problem& p, long long n, const int64_t* loc, const void* k_cache,
                        const void* v_cache, void* k, void* v, const void* idx_cache, void* idx_k, int idx_heads,
                        int idx_dim, int32_t* flags, cudaStream_t st) {
  const int idx_rc = idx_cache ? idx_dim / 8 : 0;
  const long long per_token = 16LL * p.num_kv_heads + (long long)(idx_cache ? idx_heads : 0) * idx_rc;
  if (n == 0) return cudaSuccess;
  int sms = 148, dev = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const bool bf16 = p.q_dtype == MXSA_BF16;
  void (*kern)(LoadArgs);
  switch (cache_kind(p)) {
    case kKindFp8: kern = bf16 ? k_load<kKindFp8, true> : k_load<kKindFp8, false>; break;
    case kKindFp4: kern = bf16 ? k_load<kKindFp4, true> : k_load<kKindFp4, false>; break;
    default: kern = k_load<kKind16, true>;  // bits copied: one form for both types
  }
  const long long max_tokens = std::max(1LL, (long long)INT32_MAX / per_token);  // 32-bit chunk numbers
  for (long long t0 = 0; t0 < n; t0 += max_tokens) {
    const long long m = std::min(max_tokens, n - t0);
    LoadArgs a{};
    a.loc = loc + t0;
    a.src[0] = static_cast<const uint8_t*>(k_cache);
    a.src[1] = static_cast<const uint8_t*>(v_cache);
    a.src[2] = static_cast<const uint8_t*>(idx_cache);
    a.dst[0] = static_cast<uint8_t*>(k) + t0 * p.num_kv_heads * 256;
    a.dst[1] = static_cast<uint8_t*>(v) + t0 * p.num_kv_heads * 256;
    a.dst[2] = idx_cache ? static_cast<uint8_t*>(idx_k) + t0 * idx_heads * idx_dim * 2 : nullptr;
    a.heads[0] = p.num_kv_heads;
    a.heads[1] = idx_cache ? idx_heads : 1;
    a.row_chunks[0] = 16;
    a.row_chunks[1] = idx_cache ? idx_rc : 1;
    for (int i = 0; i < 2; ++i) {
      a.rc_shift[i] = log2_exact(a.row_chunks[i]);
      a.heads_shift[i] = log2_exact(a.heads[i]);
    }
    a.chunks[0] = (uint32_t)(m * p.num_kv_heads * 16);
    a.chunks[1] = idx_cache ? (uint32_t)(m * idx_heads * idx_rc) : 0u;
    a.slots = (long long)p.num_pages * p.page_size;
    a.page_shift = p.page_size == 128 ? 7 : 6;
    a.flags = flags;
    const long long total = (long long)a.chunks[0] + a.chunks[1];
    const unsigned blocks = (unsigned)std::min((total + 255) / 256, (long long)sms * 8);
    const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(256), 0, st, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mxsa

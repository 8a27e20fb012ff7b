// Digests of the 4-bit cache's pages: for each of a page's 576 channels the
// largest and the smallest value over its tokens, as 8-bit integers rounded
// outwards on a power-of-two grid of the page (one for the latents, one for
// the rope part).
//
// Values are E2M1 codes times a power of two, or BF16: exact in BF16, and a
// maximum is exact too, so a digest does not depend on the order in which
// tokens are looked at.  A CTA takes a page.  Latents: a thread takes a block
// of 32 (16 bytes of codes, one scale byte) of every 16th token; rope rows: a
// 16-byte chunk of every 32nd token.  Maxima and minima are kept in packed
// BF16, joined across a warp by shuffles and across warps in shared memory.
// Bound by memory (400 bytes a token) where there are many pages, by the
// latency table -> codes -> barriers where there are few.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kDigestThreads = 256;
constexpr int kDigestWarps = kDigestThreads / 32;
constexpr int kDigestCtasPerSm = 2;
constexpr int kDigestExpMin = -60, kDigestExpMax = 60;

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest and smallest of N pairs of values.
template <int N>
struct Extremes {
  uint32_t hi[N], lo[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) hi[i] = 0xFF80FF80u, lo[i] = 0x7F807F80u;  // -infinity, +infinity
  }
  __device__ __forceinline__ void take(int i, uint32_t v) {
    hi[i] = max_bf16x2(hi[i], v);
    lo[i] = min_bf16x2(lo[i], v);
  }
  __device__ __forceinline__ void join(int lanes) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], lanes));
      lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], lanes));
    }
  }
};

struct DigestShared {
  uint32_t hi[kDigestWarps][kOutDim / 2], lo[kDigestWarps][kOutDim / 2];  // pairs of channels, latents first
  uint32_t amax[kDigestWarps];
  uint32_t rope_amax;
  unsigned bad[kDigestWarps];  // bit 0: of the latents, bit 1: of the rope part
};

// Bits of the larger magnitude of a pair's extremes as FP32.
__device__ __forceinline__ uint32_t pair_amax(uint32_t hi, uint32_t lo) {
  const uint32_t m = __vmaxu2(hi & 0x7FFF7FFFu, lo & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16) << 16;
}

// Smallest e >= -60 with amax <= 127 * 2^e: 127/64 = 1 + 0x7E0000 * 2^-23.
__device__ __forceinline__ int digest_exponent(uint32_t amax) {
  return max(static_cast<int>((amax + 0x01FFFFu) >> 23) - 127 - 6, kDigestExpMin);
}

// A pair's two bytes: largest rounded up, smallest rounded down.
__device__ __forceinline__ void put_pair(uint8_t* hi_at, uint8_t* lo_at, uint32_t hi, uint32_t lo, int e, bool bad) {
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const int h0 = __float2int_ru(bf16_lo(hi) * f), h1 = __float2int_ru(bf16_hi(hi) * f);
  const int l0 = __float2int_rd(bf16_lo(lo) * f), l1 = __float2int_rd(bf16_hi(lo) * f);
  *reinterpret_cast<uint16_t*>(hi_at) = bad ? 0 : static_cast<uint16_t>((h0 & 0xFF) | (h1 & 0xFF) << 8);
  *reinterpret_cast<uint16_t*>(lo_at) = bad ? 0 : static_cast<uint16_t>((l0 & 0xFF) | (l1 & 0xFF) << 8);
}

// The digest of the page at `base`, into `out`.  All threads call.
__device__ __forceinline__ void digest_page(DigestShared& s, const uint8_t* base, int shift, uint8_t* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tokens = 1 << shift;
  unsigned bad = 0;

  // rope rows, asked for first: chunk c of tokens r, r + 32, ..
  const int c = tid & 7, r = tid >> 3;
  Extremes<4> rope;
  rope.clear();
  constexpr int kRopeEach = 128 * 8 / kDigestThreads;
  uint4 row[kRopeEach];
#pragma unroll
  for (int i = 0; i < kRopeEach; ++i)
    if (r + 32 * i < tokens) row[i] = ld_u128(base + kv4_rope_off(r + 32 * i, shift) + 16 * (c ^ (r & 7)));

  // blocks of latents: block b of tokens w, w + 16, ..; four tokens in flight
  const int b = tid & 15, w = tid >> 4;
  Extremes<16> lat;
  lat.clear();
#pragma unroll 1
  for (int t0 = 0; t0 < tokens; t0 += 64) {
    uint4 codes[4];
    uint32_t scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + w + 16 * i;
      if (t >= tokens) break;
      codes[i] = ld_u128(base + kv4_code_off(t) + 16 * b);
      scale[i] = base[kv4_scale_off(t, shift) + b];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + w + 16 * i >= tokens) break;
      bad |= scale[i] == kKv4ScaleNan;
      const uint32_t f = kv4_scale_bf16x2(scale[i]);
      const uint32_t word[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o[4];
        kv4_word_bf16(word[q], o);
#pragma unroll
        for (int u = 0; u < 4; ++u) lat.take(4 * q + u, mul_bf16x2(o[u], f));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRopeEach; ++i) {
    if (r + 32 * i >= tokens) break;
    const uint32_t v[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if ((v[u] & 0x7F80u) == 0x7F80u || (v[u] & 0x7F800000u) == 0x7F800000u) bad |= 2u;
      rope.take(u, v[u]);
    }
  }

  lat.join(16);
  rope.join(8);
  rope.join(16);
  bad = __reduce_or_sync(0xffffffffu, bad);
  __syncthreads();  // what the page before left here has been read
  if (lane == 0) s.bad[warp] = bad;
  if (lane < 16) {
    // blocks with bit 2 set hold their halves in swapped order
    const int half = (b & 4) ? 8 : 0;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      *reinterpret_cast<uint4*>(&s.hi[warp][16 * b + (i ^ half)]) = make_uint4(lat.hi[i], lat.hi[i + 1], lat.hi[i + 2], lat.hi[i + 3]);
      *reinterpret_cast<uint4*>(&s.lo[warp][16 * b + (i ^ half)]) = make_uint4(lat.lo[i], lat.lo[i + 1], lat.lo[i + 2], lat.lo[i + 3]);
    }
  }
  if (lane < 8) {
    *reinterpret_cast<uint4*>(&s.hi[warp][kLatent / 2 + 4 * c]) = make_uint4(rope.hi[0], rope.hi[1], rope.hi[2], rope.hi[3]);
    *reinterpret_cast<uint4*>(&s.lo[warp][kLatent / 2 + 4 * c]) = make_uint4(rope.lo[0], rope.lo[1], rope.lo[2], rope.lo[3]);
  }
  __syncthreads();
  // a pair of latents a thread; warp 0 a pair of the rope part besides
  auto joined = [&](int pair, uint32_t& hi, uint32_t& lo) {
    hi = s.hi[0][pair], lo = s.lo[0][pair];
#pragma unroll
    for (int i = 1; i < kDigestWarps; ++i) hi = max_bf16x2(hi, s.hi[i][pair]), lo = min_bf16x2(lo, s.lo[i][pair]);
  };
  uint32_t hi, lo, rhi = 0, rlo = 0;
  joined(tid, hi, lo);
  const uint32_t top = __reduce_max_sync(0xffffffffu, pair_amax(hi, lo));
  if (lane == 0) s.amax[warp] = top;
  if (warp == 0) {
    joined(kLatent / 2 + lane, rhi, rlo);
    const uint32_t rtop = __reduce_max_sync(0xffffffffu, pair_amax(rhi, rlo));
    if (lane == 0) s.rope_amax = rtop;
  }
  __syncthreads();
  uint32_t amax = 0;
  bad = 0;
#pragma unroll
  for (int i = 0; i < kDigestWarps; ++i) amax = max(amax, s.amax[i]), bad |= s.bad[i];
  const int e = digest_exponent(amax), re = digest_exponent(s.rope_amax);
  const bool lat_bad = (bad & 1u) || e > kDigestExpMax, rope_bad = (bad & 2u) || re > kDigestExpMax;
  put_pair(out + 2 * tid, out + kLatent + 2 * tid, hi, lo, e, lat_bad);
  if (warp == 0) {
    uint8_t* at = out + 2 * kLatent + 2 * lane;
    put_pair(at, at + kRope, rhi, rlo, re, rope_bad);
    if (lane < 4) {
      const uint32_t exps = lane ? 0u : (lat_bad ? 255u : static_cast<uint32_t>(e + 127)) | (rope_bad ? 255u : static_cast<uint32_t>(re + 127)) << 8;
      *reinterpret_cast<uint32_t*>(out + 2 * kOutDim + 4 * lane) = exps;
    }
  }
}

__global__ void __launch_bounds__(kDigestThreads, kDigestCtasPerSm)
    mlaqp_kv4_digest_kernel(const __grid_constant__ Kv4DigestParams p) {
  __shared__ DigestShared s;
  pdl_launch_dependents();
  pdl_wait();
  const int shift = p.cache.shift;
  const int per = ((p.max_new - 1) >> shift) + 1;  // pages that max_new tokens can fill
  const int64_t jobs = static_cast<int64_t>(p.n) * per;
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int i = static_cast<int>(job / per), j = static_cast<int>(job % per);
    const int seq = p.seqs[i], fresh = p.new_tokens[i];
    bool bad = seq < 0 || seq >= p.num_seqs || fresh < 0 || fresh > p.max_new;
    int len = 0;
    if (!bad) {
      len = p.seq_lens[seq];
      bad = len < 0 || len > p.table_stride << shift || len > p.cache.num_pages << shift;
    }
    if (bad) {
      if (j == 0 && threadIdx.x == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
      continue;
    }
    const int page_at = ((len - min(fresh, len)) >> shift) + j;  // of the sequence
    if (page_at >= len >> shift) continue;
    const int page = p.block_table[seq * p.table_stride + page_at];
    if (page < 0 || page >= p.cache.num_pages) {
      if (threadIdx.x == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
      continue;
    }
    digest_page(s, p.cache.base + page * p.cache.page_stride, shift, p.digests + page * p.digest_stride);
  }
}

}  // namespace

cudaError_t kv4_digest(const Kv4DigestParams& p, int sm_count, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4DigestParams*>(&p)};
  const int64_t jobs = static_cast<int64_t>(p.n) * (((p.max_new - 1) >> p.cache.shift) + 1);
  const int64_t most = static_cast<int64_t>(kDigestCtasPerSm) * sm_count;
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_digest_kernel),
                    static_cast<unsigned>(jobs < most ? jobs : most), kDigestThreads, 0, stream, args);
}

cudaError_t kv4_digest_setup() {
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_digest_kernel));
}

cudaError_t device_status_kv4_digest(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

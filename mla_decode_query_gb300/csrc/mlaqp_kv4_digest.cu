// Digests of the 4-bit cache's pages: for each of a page's 576 channels the
// largest and the smallest value over its tokens, as 8-bit integers rounded
// outwards on a power-of-two grid of the page (one for the latents, one for
// the rope part).
//
// A maximum is exact, so a digest does not depend on the order in which tokens
// are looked at.  A page is a CTA's of two or four warps, each of which takes as many
// tokens, and a lane has 16 latents and two rope elements of all of them: what
// crosses lanes are the page's magnitude, the scales by way of shared memory and,
// at the end, the rope part's chunks and the warps' extremes.
//
// Latents in FP16, relative to the page's largest scale S: code * 2^max(s-S,-13).
// Their FP16 have lower bytes of zero, so one byte permute looks four up in the
// eight magnitudes of the block's scale, which two products put together, and the
// pairs stay as they lie, with another code's byte below each: it decides between
// equals only and is dropped at the end.  A value more than 13
// octaves down is not exact, but so far below the page's largest, which S is taken
// from, that its bound is 0, 1 or -1 by its sign alone: with the largest at least 2
// in these units the grid's step is 2^-5 or more, and 6 * 2^-13 less than it.  Where
// the largest is below 2 (scale bytes larger than their codes need, which the
// cache's own calls do not write but for magnitudes below 2^-39), the page is done
// in BF16.
//
// What bounds it.  1024 pages of 64 tokens: 9.4 us with other pages in every call, 27
// MB at 2.9 TB/s (6000 of them 40 us, 4.0 TB/s): the ALU, some 40 instructions a token
// and warp, 16 of them maxima and minima, which an SM issues two of a cycle.  64
// candidates of which some fill a page of 16: 2.9 us, the chain lists -> lengths ->
// table -> scales, codes -> join.  With a warp 64 latents of all tokens instead of all
// of some, and the maxima joined within warps: 12.5 and 3.2 us.

#include <algorithm>

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kDigestWarpsPerSm = 16;  // 128 registers a thread
constexpr int kDigestAhead = 8;        // tokens of a warp under way
constexpr int kDigestMaxPage = 128;
constexpr int kDigestExpMin = -60, kDigestExpMax = 60;

template <int Warps>
struct DigestShared {
  alignas(16) uint8_t scales[Warps][kDigestMaxPage][kKv4Blocks];  // of a page, a warp's own
  int32_t page[32];
  uint32_t part[Warps - 1][18][32];  // of all warps but the first
};

// Of two pairs of values, FP16 (neither is a NaN) or BF16 (a NaN stays one).
template <bool F16>
__device__ __forceinline__ uint32_t max_x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool F16>
__device__ __forceinline__ uint32_t min_x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest and smallest of a pair of values.
template <bool F16>
struct Extremes {
  uint32_t hi, lo;
  __device__ __forceinline__ void clear() {
    hi = F16 ? 0xFC00FC00u : 0xFF80FF80u;  // -infinity
    lo = hi ^ 0x80008000u;
  }
  __device__ __forceinline__ void take(uint32_t v) { take(v, v); }
  __device__ __forceinline__ void take(uint32_t h, uint32_t l) {
    hi = max_x2<F16>(hi, h);
    lo = min_x2<F16>(lo, l);
  }
  __device__ __forceinline__ void take_lane(Extremes of, int mask) {
    take(__shfl_xor_sync(0xffffffffu, of.hi, mask), __shfl_xor_sync(0xffffffffu, of.lo, mask));
  }
  // bits of the larger magnitudes
  __device__ __forceinline__ uint32_t magnitudes() const { return __vmaxu2(hi & 0x7FFF7FFFu, lo & 0x7FFF7FFFu); }
};

// The larger half, over the warp.
__device__ __forceinline__ uint32_t warp_max_half(uint32_t two) {
  return __reduce_max_sync(0xffffffffu, max(two & 0xFFFFu, two >> 16));
}

// Smallest e >= -60 with amax <= 127 * 2^e: 127/64 = 1 + 0x7E0000 * 2^-23.
__device__ __forceinline__ int digest_exponent(uint32_t amax) {
  return max(static_cast<int>((amax + 0x01FFFFu) >> 23) - 127 - 6, kDigestExpMin);
}

__device__ __forceinline__ float f16_lo(uint32_t bits) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(bits));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t bits) { return f16_lo(bits >> 16); }

// v * f, |v * f| <= 127 and exact, rounded up or down to a whole number: it is the
// low byte of 1.5 * 2^23 plus that.
__device__ __forceinline__ uint32_t whole_up(float v, float f) { return __float_as_uint(__fmaf_ru(v, f, 12582912.f)); }
__device__ __forceinline__ uint32_t whole_down(float v, float f) { return __float_as_uint(__fmaf_rd(v, f, 12582912.f)); }
// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// First of the 16 latents of this lane: the cache's blocks with bit 2 set hold
// their halves in swapped order.
__device__ __forceinline__ int lane_latents() {
  const int lane = threadIdx.x & 31;
  return 16 * (lane ^ ((lane >> 3) & 1));
}

// Bounds of a page's latents where FP16 does not hold them: in BF16.  The warp
// calls; returns the exponent byte.
__device__ __noinline__ uint32_t digest_any(const uint8_t* base, int shift, uint8_t* out) {
  const int lane = threadIdx.x & 31;
  Extremes<false> lat[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lat[i].clear();
#pragma unroll 1
  for (int t = 0; t < 1 << shift; ++t) {
    const uint8_t* at = base + kv4_code_off(t) + 8 * lane;
    const uint32_t f = kv4_scale_bf16x2(base[kv4_scale_off(t, shift) + (lane >> 1)]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t o[4];
      kv4_word_bf16(ld_u32(at + 4 * k), o);
#pragma unroll
      for (int u = 0; u < 4; ++u) lat[4 * k + u].take(mul_bf16x2(o[u], f));
    }
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) most = __vmaxu2(most, lat[i].magnitudes());
  const int e = digest_exponent(warp_max_half(most) << 16);
  const bool bad = e > kDigestExpMax;
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Extremes<false> a = lat[2 * i], b = lat[2 * i + 1];
    hi[i] = bad ? 0u : low_bytes(whole_up(bf16_lo(a.hi), f), whole_up(bf16_hi(a.hi), f), whole_up(bf16_lo(b.hi), f), whole_up(bf16_hi(b.hi), f));
    lo[i] = bad ? 0u : low_bytes(whole_down(bf16_lo(a.lo), f), whole_down(bf16_hi(a.lo), f), whole_down(bf16_lo(b.lo), f), whole_down(bf16_hi(b.lo), f));
  }
  st_u128(out + lane_latents(), make_uint4(hi[0], hi[1], hi[2], hi[3]));
  st_u128(out + kLatent + lane_latents(), make_uint4(lo[0], lo[1], lo[2], lo[3]));
  return bad ? 255u : static_cast<uint32_t>(e + 127);
}

// The digest of the page at `base`, into `out`.  All threads call.
template <int Warps>
__device__ __forceinline__ void digest_page(DigestShared<Warps>& s, const uint8_t* base, int shift, uint8_t* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tokens = 1 << shift;
  const int count = tokens / Warps, begin = warp * count;  // this warp's

  const uint8_t* const code_at = base + kv4_code_off(begin) + 8 * lane;
  const uint8_t* const rope_at = base + kv4_rope_off(begin, shift) + 4 * lane;
  uint2 codes[kDigestAhead];
  uint32_t rope[kDigestAhead];
  auto load = [&](int i, int t) {
    asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(codes[i].x), "=r"(codes[i].y) : "l"(code_at + t * kKv4CodeBytes));
    rope[i] = ld_u32(rope_at + t * kKv4RopeBytes);
  };
  uint4 by[kDigestMaxPage / 32];
#pragma unroll
  for (int i = 0; i < kDigestMaxPage / 32; ++i) {
    by[i] = make_uint4(0, 0, 0, 0);
    if (32 * i + lane < tokens) by[i] = ld_u128(base + kv4_scale_off(32 * i + lane, shift));
  }
#pragma unroll
  for (int i = 0; i < kDigestAhead; ++i)
    if (i < count) load(i, i);

  __syncwarp();  // (the scales of the page before have been read)
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kDigestMaxPage / 32; ++i) {
    if (32 * i + lane < tokens) *reinterpret_cast<uint4*>(s.scales[warp][32 * i + lane]) = by[i];
    const uint32_t w[4] = {by[i].x, by[i].y, by[i].z, by[i].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) most = __vmaxu2(most, __vmaxu2(w[u] & 0x00FF00FFu, w[u] >> 8 & 0x00FF00FFu));
  }
  most = warp_max_half(most);
  __syncwarp();
  const bool has_nan = most == kKv4ScaleNan;
  const int top_scale = static_cast<int>(min(max(most, static_cast<uint32_t>(kKv4ScaleMin)), static_cast<uint32_t>(kKv4ScaleMax)));
  const int low_scale = max(top_scale - 13, kKv4ScaleMin);

  // of the latents: elements (1, 3), (0, 2), (5, 7), (4, 6) of two words; of the rope
  // part: the pair that lies here, by the token's position modulo 8, which its
  // 16-byte chunks are swizzled by
  Extremes<true> lat[8];
  Extremes<false> turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lat[i].clear(), turn[i].clear();
  const uint8_t* const scale_at = &s.scales[warp][begin][lane >> 1];
#pragma unroll 1
  for (int t0 = 0; t0 < count; t0 += kDigestAhead) {
#pragma unroll
    for (int i = 0; i < kDigestAhead; ++i) {
      if (i % 4 == 0 && t0 + i >= count) break;  // (16 tokens to four warps)
      const uint32_t d = min(max(static_cast<int>(scale_at[(t0 + i) * kKv4Blocks]), low_scale), top_scale) - top_scale;
      // the upper bytes of the eight magnitudes, an octave 4 of them
      const uint32_t small = d * 0x04040400u + 0x3E3C3800u, large = d * 0x04040404u + 0x46444240u;
      const uint32_t word[2] = {codes[i].x, codes[i].y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t m = word[k] & 0x77777777u;
        const uint32_t a = __byte_perm(small, large, m) | (word[k] & 0x80808080u);
        const uint32_t b = __byte_perm(small, large, m >> 16) | ((word[k] * 16u) & 0x80808080u);
        lat[4 * k].take(a);
        lat[4 * k + 1].take(a * 256u);
        lat[4 * k + 2].take(b);
        lat[4 * k + 3].take(b * 256u);
      }
      turn[i % 8].take(rope[i]);
      if (t0 + kDigestAhead < count) load(i, t0 + kDigestAhead + i);
    }
  }
  // chunk lane / 4 of the rope part, wherever it lay (turn i is of the position
  // i ^ (begin & 7): begin is a multiple of count, and that a power of two)
#pragma unroll
  for (int n = 4; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) turn[i].take_lane(turn[i + n], 4 * n);
  Extremes<false> pair = turn[0];
  pair.hi = __shfl_xor_sync(0xffffffffu, pair.hi, 4 * (begin & 7));
  pair.lo = __shfl_xor_sync(0xffffffffu, pair.lo, 4 * (begin & 7));

  if (warp > 0) {
    uint32_t(*mine)[32] = s.part[warp - 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[2 * i][lane] = lat[i].hi, mine[2 * i + 1][lane] = lat[i].lo;
    mine[16][lane] = pair.hi, mine[17][lane] = pair.lo;
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 0; w < Warps - 1; ++w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lat[i].take(s.part[w][2 * i][lane], s.part[w][2 * i + 1][lane]);
      pair.take(s.part[w][16][lane], s.part[w][17][lane]);
    }
  }
  __syncthreads();  // (the next page's may be written)
  if (warp > 0) return;

  uint32_t size = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lat[i].hi &= 0xFF00FF00u;
    lat[i].lo &= 0xFF00FF00u;
    size = __vmaxu2(size, lat[i].magnitudes());
  }
  const uint32_t amax = warp_max_half(size);
  uint32_t byte;
  if (!has_nan && amax > 0 && amax < 0x4000u) {  // the largest is below 2
    byte = digest_any(base, shift, out);
  } else {
    const float unit = __uint_as_float(static_cast<uint32_t>(top_scale) << 23);  // 2^(S-127)
    const int e = digest_exponent(__float_as_uint(f16_lo(amax) * unit));
    const bool bad = has_nan || e > kDigestExpMax;
    const float f = unit * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Extremes<true> a = lat[2 * i + 1], b = lat[2 * i];  // elements 0, 2 and 1, 3 of four
      hi[i] = bad ? 0u : low_bytes(whole_up(f16_lo(a.hi), f), whole_up(f16_lo(b.hi), f), whole_up(f16_hi(a.hi), f), whole_up(f16_hi(b.hi), f));
      lo[i] = bad ? 0u : low_bytes(whole_down(f16_lo(a.lo), f), whole_down(f16_lo(b.lo), f), whole_down(f16_hi(a.lo), f), whole_down(f16_hi(b.lo), f));
    }
    st_u128(out + lane_latents(), make_uint4(hi[0], hi[1], hi[2], hi[3]));
    st_u128(out + kLatent + lane_latents(), make_uint4(lo[0], lo[1], lo[2], lo[3]));
    byte = bad ? 255u : static_cast<uint32_t>(e + 127);
  }

  const uint32_t rope_amax = warp_max_half(pair.magnitudes());
  const int e = digest_exponent(rope_amax << 16);
  const bool bad = rope_amax >= 0x7F80u || e > kDigestExpMax;
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint8_t* at = out + 2 * kLatent + 2 * lane;
  const uint32_t up = __byte_perm(whole_up(bf16_lo(pair.hi), f), whole_up(bf16_hi(pair.hi), f), 0x0040);
  const uint32_t down = __byte_perm(whole_down(bf16_lo(pair.lo), f), whole_down(bf16_hi(pair.lo), f), 0x0040);
  *reinterpret_cast<uint16_t*>(at) = bad ? 0 : static_cast<uint16_t>(up);
  *reinterpret_cast<uint16_t*>(at + kRope) = bad ? 0 : static_cast<uint16_t>(down);
  if (lane == 0)
    st_u128(out + 2 * kOutDim, make_uint4(byte | (bad ? 255u : static_cast<uint32_t>(e + 127)) << 8, 0u, 0u, 0u));
}

// The page of a job (an item of the list, and one of the `per` pages that it may
// have filled), -1: none.
__device__ __forceinline__ int digest_job(const Kv4DigestParams& p, int64_t job, int per) {
  const int shift = p.cache.shift;
  const int i = static_cast<int>(job / per), j = static_cast<int>(job % per);
  const int seq = p.seqs[i], fresh = p.new_tokens[i];
  bool bad = seq < 0 || seq >= p.num_seqs || fresh < 0 || fresh > p.max_new;
  int len = 0;
  if (!bad) {
    len = p.seq_lens[seq];
    bad = len < 0 || len > p.table_stride << shift || len > p.cache.num_pages << shift;
  }
  if (bad) {
    if (j == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    return -1;
  }
  const int at = ((len - min(fresh, len)) >> shift) + j;  // of the sequence
  if (at >= len >> shift) return -1;
  const int page = p.block_table[seq * p.table_stride + at];
  if (page < 0 || page >= p.cache.num_pages) {
    atomicOr(&g_device_status, kDevStatusBadIndex);
    return -1;
  }
  return page;
}

template <int Warps>
__global__ void __launch_bounds__(32 * Warps, kDigestWarpsPerSm / Warps)
    mlaqp_kv4_digest_kernel(const __grid_constant__ Kv4DigestParams p) {
  __shared__ DigestShared<Warps> s;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int per = p.per;
  const int64_t jobs = static_cast<int64_t>(p.n) * per, ctas = gridDim.x;
  // The lookups are three loads one after the other: a lane a job, for 32 at once.
  for (int64_t j0 = blockIdx.x; j0 < jobs; j0 += 32 * ctas) {
    if (threadIdx.x < 32) s.page[lane] = j0 + ctas * lane < jobs ? digest_job(p, j0 + ctas * lane, per) : -1;
    __syncthreads();
    const int mine = s.page[lane];
    for (unsigned left = __ballot_sync(0xffffffffu, mine >= 0); left; left &= left - 1) {
      const int page = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
      digest_page<Warps>(s, p.cache.base + page * p.cache.page_stride, p.cache.shift, p.digests + page * p.digest_stride);
    }
    __syncthreads();
  }
}

const void* digest_kernel(int warps) {
  return warps == 4 ? reinterpret_cast<const void*>(&mlaqp_kv4_digest_kernel<4>)
                    : reinterpret_cast<const void*>(&mlaqp_kv4_digest_kernel<2>);
}

}  // namespace

// Four warps a page while all CTAs find room at once, two beyond.  Pages of 64 tokens,
// others in every call, with four, two and one: 100 of them 3.6, 4.1, 5.7 us; 600: 5.8,
// 6.6, 7.8; 1024: 10.9, 9.7, 13.7; 2048: 18.3, 17.9, 16.5; 6000: 45.6, 39.9, 41.4.
// Rounds of CTAs make the steps: for 2048 a warp a page is one round less.  A candidate
// that fills no page costs a lane its lookup: 64 sequences of a page each 1.5 us, with
// room for 131072 new tokens in pages of 16 (524288 candidates) 5.7.
cudaError_t kv4_digest(const Kv4DigestParams& params, int sm_count, cudaStream_t stream) {
  Kv4DigestParams p = params;
  void* args[1] = {&p};
  // as many as max_new tokens can fill, as a row holds and as there are
  const int64_t most_full = std::min<int64_t>(p.table_stride, p.cache.num_pages);
  p.per = static_cast<int>(std::min<int64_t>(((p.max_new - 1) >> p.cache.shift) + 1, most_full));
  const int64_t jobs = static_cast<int64_t>(p.n) * p.per;
  const int warps = jobs * 4 <= static_cast<int64_t>(kDigestWarpsPerSm) * sm_count ? 4 : 2;
  const int64_t most = static_cast<int64_t>(kDigestWarpsPerSm / warps) * sm_count;
  return kv4_launch(digest_kernel(warps), static_cast<unsigned>(jobs < most ? jobs : most), 32 * warps, 0, stream, args);
}

cudaError_t kv4_digest_setup() {
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, digest_kernel(2));
  return e == cudaSuccess ? cudaFuncGetAttributes(&a, digest_kernel(4)) : e;
}

cudaError_t device_status_kv4_digest(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

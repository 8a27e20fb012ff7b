// Digests of the 4-bit cache's pages: for each of a page's 576 channels the
// largest and the smallest value over its tokens, as 8-bit integers rounded
// outwards on a power-of-two grid of the page (one for the latents, one for
// the rope part).
//
// A maximum is exact, so a digest does not depend on the order in which tokens
// are looked at.  A CTA takes a page, a warp 64 channels of all its tokens, and
// maxima and minima are kept as packed 16-bit floats and joined across a warp;
// only the page's magnitude crosses warps.
//
// What bounds it.  1024 pages of 64 tokens: 12.8 us, 27 MB at 2.1 TB/s; the
// ALU (decoding, scaling, maxima and minima of 576 elements a token: 0.52
// instructions issued a cycle over the whole call) and, as a CTA does two or
// three pages, the latencies at both ends.  64 candidates of which some fill a
// page of 16: 3.2 us, the chain lists -> lengths -> table -> scales, codes ->
// barriers.  With two or four CTAs an SM instead of three 14.4 and 14.6 us.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kDigestThreads = 256;
constexpr int kDigestWarps = kDigestThreads / 32;
constexpr int kDigestCtasPerSm = 3;
constexpr int kDigestAhead = 4;  // tokens of a lane under way: 32 of the page
constexpr int kDigestExpMin = -60, kDigestExpMax = 60;

template <bool F16>
__device__ __forceinline__ uint32_t max_x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool F16>
__device__ __forceinline__ uint32_t min_x2(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (F16)
    asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest and smallest of N pairs of values, FP16 or BF16.
template <int N, bool F16 = false>
struct Extremes {
  uint32_t hi[N], lo[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) hi[i] = F16 ? 0xFC00FC00u : 0xFF80FF80u, lo[i] = hi[i] ^ 0x80008000u;  // -infinity, +infinity
  }
  __device__ __forceinline__ void take(int i, uint32_t v) {
    hi[i] = max_x2<F16>(hi[i], v);
    lo[i] = min_x2<F16>(lo[i], v);
  }
  // Joined with the lane that differs in bit `mask`: the first half of the
  // pairs stays with the one that has it clear, the second with the other.
  __device__ __forceinline__ Extremes<N / 2, F16> halve(int mask) const {
    Extremes<N / 2, F16> r;
    const bool up = (threadIdx.x & mask) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t h = __shfl_xor_sync(0xffffffffu, up ? hi[i] : hi[i + N / 2], mask);
      const uint32_t l = __shfl_xor_sync(0xffffffffu, up ? lo[i] : lo[i + N / 2], mask);
      r.hi[i] = max_x2<F16>(up ? hi[i + N / 2] : hi[i], h);
      r.lo[i] = min_x2<F16>(up ? lo[i + N / 2] : lo[i], l);
    }
    return r;
  }
  __device__ __forceinline__ void join(int mask) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      hi[i] = max_x2<F16>(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], mask));
      lo[i] = min_x2<F16>(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], mask));
    }
  }
};

constexpr int kDigestJobs = kDigestThreads;  // looked up at once
struct DigestShared {
  int32_t page[kDigestJobs];
  alignas(16) uint8_t scales[2][128][kKv4Blocks];  // a page's
  uint32_t scale[2][kDigestWarps];
  // by warp, of two pages by turns
  uint32_t amax[2][kDigestWarps], rope_amax[2][kDigestWarps];
  unsigned bad[2][kDigestWarps];  // bit 0: of the latents, bit 1: of the rope part
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

// Value of FP16 bits.
__device__ __forceinline__ float f16_value(uint32_t bits) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(bits));
  return f;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A pair's two bytes: largest rounded up, smallest rounded down.
__device__ __forceinline__ void put_pair(uint8_t* hi_at, uint8_t* lo_at, uint32_t hi, uint32_t lo, int e, bool bad) {
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const int h0 = __float2int_ru(bf16_lo(hi) * f), h1 = __float2int_ru(bf16_hi(hi) * f);
  const int l0 = __float2int_rd(bf16_lo(lo) * f), l1 = __float2int_rd(bf16_hi(lo) * f);
  *reinterpret_cast<uint16_t*>(hi_at) = bad ? 0 : static_cast<uint16_t>((h0 & 0xFF) | (h1 & 0xFF) << 8);
  *reinterpret_cast<uint16_t*>(lo_at) = bad ? 0 : static_cast<uint16_t>((l0 & 0xFF) | (l1 & 0xFF) << 8);
}

// Rope rows: the first four warps take two 16-byte chunks each, lanes of even
// and odd number one of the two, of tokens lane / 2, + 16, ..
struct RopePart {
  Extremes<4> all;
  Extremes<1> mine;  // pair lane / 8 of the chunk, when joined
  uint32_t top;
  __device__ __forceinline__ static bool has() { return threadIdx.x < 32 * (kRope / 16); }
  __device__ __forceinline__ static int chunk() { return 2 * (threadIdx.x >> 5) + (threadIdx.x & 1); }
  // (of 32 tokens)
  __device__ __forceinline__ static void load(uint4 (&row)[2], const uint8_t* base, int shift, int t0) {
    const int first = (threadIdx.x & 31) >> 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + first + 16 * i;
      if (t < 1 << shift) row[i] = ld_u128(base + kv4_rope_off(t, shift) + 16 * (chunk() ^ (t & 7)));
    }
  }
  // whether something is not finite
  __device__ __forceinline__ bool take(const uint4 (&row)[2], int shift, int t0) {
    const int first = (threadIdx.x & 31) >> 1;
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (t0 + first + 16 * i >= 1 << shift) break;
      const uint32_t v[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // a half's exponent of all ones carries into its sign
        odd |= (v[u] & 0x7F807F80u) + 0x00800080u;
        all.take(u, v[u]);
      }
    }
    return (odd & 0x80008000u) != 0;
  }
  __device__ __forceinline__ void join() {
    mine = all.halve(16).halve(8);
    mine.join(4);
    mine.join(2);
    top = __reduce_max_sync(0xffffffffu, pair_amax(mine.hi[0], mine.lo[0]));
  }
};

// The page's exponent of the rope part and its bytes, and the exponent bytes.
__device__ __forceinline__ void put_rope(uint8_t* out, const RopePart& rope, uint32_t amax, bool bad, bool lat_bad, int e) {
  const int lane = threadIdx.x & 31;
  const int re = digest_exponent(amax);
  bad |= re > kDigestExpMax;
  if (RopePart::has() && (lane & 6) == 0) {
    uint8_t* at = out + 2 * kLatent + 2 * (4 * RopePart::chunk() + (lane >> 3));
    put_pair(at, at + kRope, rope.mine.hi[0], rope.mine.lo[0], re, bad);
  }
  const int i = static_cast<int>(threadIdx.x) - (kDigestThreads - 4);
  if (i >= 0) {
    const uint32_t exps = (lat_bad ? 255u : static_cast<uint32_t>(e + 127)) | (bad ? 255u : static_cast<uint32_t>(re + 127)) << 8;
    *reinterpret_cast<uint32_t*>(out + 2 * kOutDim + 4 * i) = i ? 0u : exps;
  }
}

// Bounds of a page's latents where FP16 does not hold them (below): in BF16.
// Warp w takes the blocks 2w and 2w + 1, lanes of even and odd number one of the
// two, of tokens lane / 2, + 16, ..  All threads call.
__device__ __noinline__ void digest_any(DigestShared& s, const uint8_t* base, int shift, uint8_t* out, int turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = lane >> 1, block = 2 * warp + (lane & 1);
  Extremes<16> lat;
  lat.clear();
#pragma unroll 1
  for (int t = first; t < 1 << shift; t += 16) {
    const uint4 codes = ld_u128(base + kv4_code_off(t) + 16 * block);
    const uint32_t f = kv4_scale_bf16x2(base[kv4_scale_off(t, shift) + block]);
    const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t o[4];
      kv4_word_bf16(word[q], o);
#pragma unroll
      for (int u = 0; u < 4; ++u) lat.take(4 * q + u, mul_bf16x2(o[u], f));
    }
  }
  // lane 2r + (block & 1) is left with pair r of its block
  const Extremes<1> mine = lat.halve(16).halve(8).halve(4).halve(2);
  const uint32_t top = __reduce_max_sync(0xffffffffu, pair_amax(mine.hi[0], mine.lo[0]));
  __syncthreads();  // (s.amax has been read)
  if (lane == 0) s.amax[turn][warp] = top;
  __syncthreads();
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < kDigestWarps; ++i) amax = max(amax, s.amax[turn][i]);
  const int e = digest_exponent(amax);
  // blocks with bit 2 set hold their halves in swapped order
  const int pair = 16 * block + (first ^ ((block & 4) ? 8 : 0));
  put_pair(out + 2 * pair, out + kLatent + 2 * pair, mine.hi[0], mine.lo[0], e, e > kDigestExpMax);
  if (threadIdx.x == 0) out[2 * kOutDim] = static_cast<uint8_t>(e > kDigestExpMax ? 255 : e + 127);
}

// The digest of the page at `base`, into `out`.  All threads call; turn: 0 and 1
// by turns.
//
// Latents in FP16, relative to the page's largest scale S: code * 2^max(s-S,-13).
// The codes' FP16 have their lower bytes zero, so one byte permute looks four up,
// and the pairs stay as they lie, with another code's byte below each: it decides
// between equals only and is dropped at the end.  (That is 8 cycles a word of eight
// and a CTA's warp on an SM, BF16 with its two bytes 15.)  A value more than 13
// octaves down is not exact, but so far below the page's largest, which S is taken
// from, that its bound is 0, 1 or -1 by its sign alone: with the largest at least 2
// in these units the grid's step is 2^-5 or more, and 6 * 2^-13 less than it.  Where
// the largest is below 2 (scale bytes larger than their codes need, which the
// cache's own calls do not write but for magnitudes below 2^-39), the page is done
// once more in BF16.
//
// Warp w takes the blocks 2w and 2w + 1, a lane two words (8 bytes) of every
// eighth token.
__device__ __forceinline__ void digest_page(DigestShared& s, const uint8_t* base, int shift, uint8_t* out, int turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tokens = 1 << shift;
  const int sub = lane & 3, first = lane >> 2;
  const int block = 2 * warp + (sub >> 1);

  const int tid = threadIdx.x;
  uint4 by = make_uint4(0, 0, 0, 0);
  if (tid < tokens) by = ld_u128(base + kv4_scale_off(tid, shift));
  uint2 codes[kDigestAhead];
  auto load = [&](int t0) {
#pragma unroll
    for (int i = 0; i < kDigestAhead; ++i)
      if (t0 + 8 * i < tokens)
        asm volatile("ld.global.v2.b32 {%0,%1}, [%2];"
                     : "=r"(codes[i].x), "=r"(codes[i].y)
                     : "l"(base + kv4_code_off(t0 + 8 * i + first) + 32 * warp + 8 * sub));
  };
  load(0);
  uint4 row[2];
  RopePart rope;
  rope.all.clear();
  if (RopePart::has()) RopePart::load(row, base, shift, 0);

  uint32_t most = 0;
  if (tid < tokens) {
    *reinterpret_cast<uint4*>(s.scales[turn][tid]) = by;
    const uint32_t w[4] = {by.x, by.y, by.z, by.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) most = __vmaxu2(most, __vmaxu2(w[i] & 0x00FF00FFu, w[i] >> 8 & 0x00FF00FFu));
    most = max(most & 0xFFFFu, most >> 16);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) s.scale[turn][warp] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDigestWarps; ++i) most = max(most, s.scale[turn][i]);
  unsigned bad = most == kKv4ScaleNan;  // bit 0: of the latents
  const int top_scale = static_cast<int>(min(max(most, static_cast<uint32_t>(kKv4ScaleMin)), static_cast<uint32_t>(kKv4ScaleMax)));

  Extremes<8, true> lat;
  lat.clear();
#pragma unroll 1
  for (int t0 = 0; t0 < tokens; t0 += 8 * kDigestAhead) {
#pragma unroll
    for (int i = 0; i < kDigestAhead; ++i) {
      if (t0 + 8 * i >= tokens) break;
      const int sc = min(max(static_cast<int>(s.scales[turn][t0 + 8 * i + first][block]), kKv4ScaleMin), kKv4ScaleMax);
      const uint32_t f = static_cast<uint32_t>(max(sc - top_scale, -13) + 15) * 0x04000400u;
      const uint32_t word[2] = {codes[i].x, codes[i].y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t m = word[k] & 0x77777777u;
        const uint32_t a = __byte_perm(0x3E3C3800u, 0x46444240u, m) | (word[k] & 0x80808080u);
        const uint32_t b = __byte_perm(0x3E3C3800u, 0x46444240u, m >> 16) | ((word[k] * 16u) & 0x80808080u);
        lat.take(4 * k, mul_f16x2(a, f));             // elements 1, 3
        lat.take(4 * k + 1, mul_f16x2(a * 256u, f));  // 0, 2
        lat.take(4 * k + 2, mul_f16x2(b, f));         // 5, 7
        lat.take(4 * k + 3, mul_f16x2(b * 256u, f));  // 4, 6
      }
    }
    if (t0 + 8 * kDigestAhead < tokens) load(t0 + 8 * kDigestAhead);
    if (RopePart::has()) {
      bad |= rope.take(row, shift, t0) ? 2u : 0u;
      if (t0 + 8 * kDigestAhead < tokens) RopePart::load(row, base, shift, t0 + 8 * kDigestAhead);
    }
  }
  // lane (first, sub) is left with pair `first` of its eight
  Extremes<1, true> mine = lat.halve(16).halve(8).halve(4);
  mine.hi[0] &= 0xFF00FF00u;
  mine.lo[0] &= 0xFF00FF00u;
  const uint32_t m2 = __vmaxu2(mine.hi[0] & 0x7FFF7FFFu, mine.lo[0] & 0x7FFF7FFFu);
  const uint32_t top = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  if (RopePart::has()) rope.join();
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) {
    s.amax[turn][warp] = top;
    s.rope_amax[turn][warp] = RopePart::has() ? rope.top : 0u;
    s.bad[turn][warp] = bad;
  }
  __syncthreads();
  uint32_t amax = 0, rope_amax = 0;
  bad = 0;
#pragma unroll
  for (int i = 0; i < kDigestWarps; ++i) {
    amax = max(amax, s.amax[turn][i]);
    rope_amax = max(rope_amax, s.rope_amax[turn][i]);
    bad |= s.bad[turn][i];
  }
  const bool again = !(bad & 1u) && amax > 0 && amax < 0x4000u;  // the largest is below 2
  const float unit = __uint_as_float(static_cast<uint32_t>(top_scale) << 23);  // 2^(S-127)
  const int e = digest_exponent(__float_as_uint(f16_value(amax) * unit));
  const bool lat_bad = (bad & 1u) || e > kDigestExpMax;
  const float f = unit * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t two = 0;  // bytes: the largest of the pair, the smallest of it
  if (!lat_bad) {
    const int h0 = __float2int_ru(f16_value(mine.hi[0] & 0xFFFFu) * f), h1 = __float2int_ru(f16_value(mine.hi[0] >> 16) * f);
    const int l0 = __float2int_rd(f16_value(mine.lo[0] & 0xFFFFu) * f), l1 = __float2int_rd(f16_value(mine.lo[0] >> 16) * f);
    two = (h0 & 0xFF) | (h1 & 0xFF) << 8 | (l0 & 0xFF) << 16 | static_cast<uint32_t>(l1 & 0xFF) << 24;
  }
  // elements (1, 3) or (5, 7) here and (0, 2) or (4, 6) with the neighbour make
  // four in a row: this lane writes their largest, that one their smallest
  const uint32_t other = __shfl_xor_sync(0xffffffffu, two, 4);
  const bool low = first & 1;
  const uint32_t four = low ? __byte_perm(two, other, 0x7362) : __byte_perm(other, two, 0x5140);
  const int word = (2 * (sub & 1) + (first >> 2)) ^ ((block & 4) ? 2 : 0);
  *reinterpret_cast<uint32_t*>(out + (low ? kLatent : 0) + 32 * block + 8 * word + 4 * (first >> 1 & 1)) = four;
  put_rope(out, rope, rope_amax, (bad & 2u) != 0, lat_bad, e);
  if (again) {
    __syncthreads();  // (what is written above is written over)
    digest_any(s, base, shift, out, turn);
  }
}

// The page of a job (an item of the list, and one of the pages that so many new
// tokens can fill), -1: none.
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

__global__ void __launch_bounds__(kDigestThreads, kDigestCtasPerSm)
    mlaqp_kv4_digest_kernel(const __grid_constant__ Kv4DigestParams p) {
  __shared__ DigestShared s;
  pdl_launch_dependents();
  pdl_wait();
  const int per = ((p.max_new - 1) >> p.cache.shift) + 1;  // pages that max_new tokens can fill
  const int64_t jobs = static_cast<int64_t>(p.n) * per;
  // The lookups are three loads one after the other: a thread a job, for all
  // jobs of the CTA at once.
  int turn = 0;
  for (int64_t j0 = blockIdx.x; j0 < jobs; j0 += static_cast<int64_t>(gridDim.x) * kDigestJobs) {
    const int64_t job = j0 + static_cast<int64_t>(gridDim.x) * threadIdx.x;
    const int mine = job < jobs ? digest_job(p, job, per) : -1;
    __syncthreads();  // the list before is done with
    s.page[threadIdx.x] = mine;
    __syncthreads();
    const int count = static_cast<int>(min(static_cast<int64_t>(kDigestJobs), (jobs - j0 + gridDim.x - 1) / gridDim.x));
    for (int i = 0; i < count; ++i) {
      const int page = s.page[i];
      if (page < 0) continue;
      digest_page(s, p.cache.base + page * p.cache.page_stride, p.cache.shift, p.digests + page * p.digest_stride, turn);
      turn ^= 1;
    }
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

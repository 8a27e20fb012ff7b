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
constexpr int kDigestCtasPerSm = 4;
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
  // Joined with the lane that differs in bit `mask`: the first half of the
  // pairs stays with the one that has it clear, the second with the other.
  __device__ __forceinline__ Extremes<N / 2> halve(int mask) const {
    Extremes<N / 2> r;
    const bool up = (threadIdx.x & mask) != 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t h = __shfl_xor_sync(0xffffffffu, up ? hi[i] : hi[i + N / 2], mask);
      const uint32_t l = __shfl_xor_sync(0xffffffffu, up ? lo[i] : lo[i + N / 2], mask);
      r.hi[i] = max_bf16x2(up ? hi[i + N / 2] : hi[i], h);
      r.lo[i] = min_bf16x2(up ? lo[i + N / 2] : lo[i], l);
    }
    return r;
  }
  __device__ __forceinline__ void join(int mask) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], mask));
      lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], mask));
    }
  }
};

constexpr int kDigestJobs = kDigestThreads;  // looked up at once
struct DigestShared {
  int32_t page[kDigestJobs];
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

// A pair's two bytes: largest rounded up, smallest rounded down.
__device__ __forceinline__ void put_pair(uint8_t* hi_at, uint8_t* lo_at, uint32_t hi, uint32_t lo, int e, bool bad) {
  const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const int h0 = __float2int_ru(bf16_lo(hi) * f), h1 = __float2int_ru(bf16_hi(hi) * f);
  const int l0 = __float2int_rd(bf16_lo(lo) * f), l1 = __float2int_rd(bf16_hi(lo) * f);
  *reinterpret_cast<uint16_t*>(hi_at) = bad ? 0 : static_cast<uint16_t>((h0 & 0xFF) | (h1 & 0xFF) << 8);
  *reinterpret_cast<uint16_t*>(lo_at) = bad ? 0 : static_cast<uint16_t>((l0 & 0xFF) | (l1 & 0xFF) << 8);
}

// The digest of the page at `base`, into `out`.  Warp w takes the blocks 2w and
// 2w + 1 of the latents, and of the first four two chunks of the rope rows, each
// of all tokens: 32 bytes of a row, so that maxima are joined within the warp,
// lanes of even and odd number one of the two, and only the page's magnitude
// across warps.  All threads call; turn: 0 and 1 by turns.
__device__ __forceinline__ void digest_page(DigestShared& s, const uint8_t* base, int shift, uint8_t* out, int turn) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tokens = 1 << shift;
  unsigned bad = 0;
  const int first = lane >> 1;  // tokens first, first + 16, ..

  // rope rows, asked for first
  const bool has_rope = warp < kRope / 16;
  const int chunk = 2 * warp + (lane & 1);
  Extremes<4> rope;
  rope.clear();
  uint4 row[4];
  auto rope_rows = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + first + 16 * i;
      if (t < tokens) row[i] = ld_u128(base + kv4_rope_off(t, shift) + 16 * (chunk ^ (t & 7)));
    }
  };
  auto rope_take = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + first + 16 * i >= tokens) break;
      const uint32_t v[4] = {row[i].x, row[i].y, row[i].z, row[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if ((v[u] & 0x7F80u) == 0x7F80u || (v[u] & 0x7F800000u) == 0x7F800000u) bad |= 2u;
        rope.take(u, v[u]);
      }
    }
  };
  if (has_rope) rope_rows(0);

  const int block = 2 * warp + (lane & 1);
  Extremes<16> lat;
  lat.clear();
#pragma unroll 1
  for (int t0 = 0; t0 < tokens; t0 += 64) {
    uint4 codes[4];
    uint32_t scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + first + 16 * i;
      if (t >= tokens) break;
      codes[i] = ld_u128(base + kv4_code_off(t) + 16 * block);
      scale[i] = base[kv4_scale_off(t, shift) + block];
    }
    if (t0 > 0 && has_rope) rope_rows(t0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + first + 16 * i >= tokens) break;
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
    if (has_rope) rope_take(t0);
  }

  // lane 2r + (block & 1) is left with pair r of its block
  const Extremes<1> mine = lat.halve(16).halve(8).halve(4).halve(2);
  const uint32_t top = __reduce_max_sync(0xffffffffu, pair_amax(mine.hi[0], mine.lo[0]));
  uint32_t rtop = 0;
  Extremes<1> rmine;
  if (has_rope) {  // pair lane >> 3 of the chunk
    rmine = rope.halve(16).halve(8);
    rmine.join(4);
    rmine.join(2);
    rtop = __reduce_max_sync(0xffffffffu, pair_amax(rmine.hi[0], rmine.lo[0]));
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) s.amax[turn][warp] = top, s.rope_amax[turn][warp] = rtop, s.bad[turn][warp] = bad;
  __syncthreads();
  uint32_t amax = 0, rope_amax = 0;
  bad = 0;
#pragma unroll
  for (int i = 0; i < kDigestWarps; ++i) {
    amax = max(amax, s.amax[turn][i]);
    rope_amax = max(rope_amax, s.rope_amax[turn][i]);
    bad |= s.bad[turn][i];
  }
  const int e = digest_exponent(amax), re = digest_exponent(rope_amax);
  const bool lat_bad = (bad & 1u) || e > kDigestExpMax, rope_bad = (bad & 2u) || re > kDigestExpMax;
  // blocks with bit 2 set hold their halves in swapped order
  const int pair = 16 * block + (first ^ ((block & 4) ? 8 : 0));
  put_pair(out + 2 * pair, out + kLatent + 2 * pair, mine.hi[0], mine.lo[0], e, lat_bad);
  if (has_rope && (lane & 6) == 0) {
    uint8_t* at = out + 2 * kLatent + 2 * (4 * chunk + (lane >> 3));
    put_pair(at, at + kRope, rmine.hi[0], rmine.lo[0], re, rope_bad);
  }
  if (tid >= kDigestThreads - 4) {
    const int i = tid - (kDigestThreads - 4);
    const uint32_t exps =
        (lat_bad ? 255u : static_cast<uint32_t>(e + 127)) | (rope_bad ? 255u : static_cast<uint32_t>(re + 127)) << 8;
    *reinterpret_cast<uint32_t*>(out + 2 * kOutDim + 4 * i) = i ? 0u : exps;
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

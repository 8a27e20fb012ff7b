// Choosing the pages that a query token attends to: scores from the pages'
// digests, and the best of them.
//
// Score of page p for query token m, H heads: the bound
//   sum_h sum_c max over the page's tokens of q[h,c] * v[t,c]
//     <= sum_c up[c] * largest[c] + down[c] * smallest[c]
//   up[c] = sum_h max(q[h,c], 0)   down[c] = sum_h min(q[h,c], 0)
// which is linear in the digest: the heads are summed once per query token,
// and a page costs 1152 products whatever H is.  q is held in 12 bits (one
// power of two a token), so up and down fit 16 bits, the digest's numbers are 8:
// a dp2a is two products, and the sums stay below 2^31 (512 * 16 * 2047 * 127),
// exact, so the choice does not depend on the order of anything.
//
// A sequence is a cluster's.  Its CTAs make up and down of the query tokens (of
// several, each CTA some for all), then a warp takes four pages at a time, a lane
// 16 + 16 + 4 bytes of each digest straight into registers, a batch ahead; up
// and down lie in shared memory in the lanes' order, read once for four pages.
// The keys go to the CTA that chooses for their query token, by distributed
// shared memory (by the workspace where there are more than it holds).  There a
// histogram of 512 places over the range of up to 1024 keys, which every warp
// scans for itself, leaves a few keys to rank, and a prefix sum puts the pages in
// order; more keys, or more of them in one place, take rounds of 2048 places.
// One launch: a score kernel that cut all pages into equal stretches, with a
// choice kernel behind it, took 21.7 us instead of 10.1.
//
// What bounds it.  64 sequences of 16000 to 32768 tokens, pages of 64, H = 16:
// 10.1 us, 28 MB of digests; 0.65 us pass until the lengths are there, 2.2 with
// the queries, 2.5 to 3.5 in the scores, 1 waiting for the longest of the cluster
// and 1.9 in the choice.  On an SM four pages cost a query token some 70 cycles
// (72 dp2a at two a cycle, 8 sums over the warp at half of one).  16 of up to 569
// pages with 4 query tokens: 11.3, of which the longest sequence scores for 4.6.
//
// The cluster's size follows from the table's width and the batch, so the longest
// sequence decides: 40 of 2000 tokens in pages of 64 take 5.8 us, with one of 131071
// beside them, on four CTAs, 18.9.  One sequence of 1024 pages takes 6.7 us with 8
// heads and digests of normalised latents; with 16 heads and random digests 8.9,
// and so one of 2048 pages 11.3 (64 of them taken).  Longer ones leave shared memory:
// their keys go through the workspace and one CTA reads them several times, 4096
// pages 26 us, 8192 47, 40009 233 (128, 256, 256 taken).

#include <atomic>

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kSelectThreads = 256;                  // eight warps: with two CTAs an SM 128 registers a thread
constexpr int kSelectChunks = kLatent / 8;           // latents: a thread's are eight channels of four heads
constexpr int kSelectHeadGroups = kSelectThreads / kSelectChunks;
constexpr int kRopeChunks = kRope / 8;               // rope part: eight channels of one head, half of the threads
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectCtasPerSm = 2;
constexpr int kScorePages = 4;                       // in flight per warp
constexpr int kScoreLane = 20;                       // a lane's 18 pairs of up / down apart: 16-byte loads without bank conflicts
constexpr int kQueryWords = 32 * kScoreLane;         // of a query token
constexpr int kTokenAt = 20;                         // bits of a page's place in its sequence
constexpr uint32_t kNoPage = 0xFFFFFFFFu;
constexpr int kBins = 2048, kBinsLog = 11;
constexpr int kBinsEach = kBins / kSelectThreads;
constexpr int kCandidates = 32;                      // keys that a warp ranks
constexpr int kFewEach = 4, kFewKeys = kFewEach * kSelectThreads;  // keys that the threads hold
constexpr int kFewBins = 512, kFewBinsLog = 9;
constexpr int kHeldKeys = 2048;                      // keys and pages that stay in shared memory
constexpr int kChooseEach = 4;                       // pages of a thread in one sweep in order
static_assert(kRopeChunks * MLAQP_KV4_MAX_HEADS <= kSelectThreads && kBinsEach == 8 && kFewEach == 4, "threads");
static_assert(MLAQP_KV4_MAX_PAGES <= 1 << kTokenAt && MLAQP_KV4_MAX_Q_LEN <= 1 << (31 - kTokenAt), "pages and tokens in a word");

// Dynamic shared memory: this, then the queries' words.
struct SelectShared {
  uint32_t amax[kSelectWarps];
  uint32_t lo[kSelectWarps], hi[kSelectWarps];
  int scan[kSelectWarps][2];
  uint32_t from;   // first key of the place that holds the last one taken
  int above, in;   // keys above that place, in it
  int found;       // candidates
  uint32_t candidate[kCandidates];
  alignas(16) unsigned bins[kBins];
  alignas(16) uint32_t keys[kHeldKeys];  // of this CTA's query tokens, one after the other
  union {
    struct {  // up << 16 | -down
      alignas(16) uint32_t part[kSelectHeadGroups][kLatent];        // sums over a thread's heads
      alignas(16) uint32_t rope_part[MLAQP_KV4_MAX_HEADS][kRope];   // of a head
    };
    alignas(16) int32_t pages[kHeldKeys];                   // (later) of the sequence, up to the last ones
  };
};
constexpr int kWordsAt = (sizeof(SelectShared) + 15) / 16 * 16;

__device__ __forceinline__ int pages_of(int tokens, int shift) { return tokens > 0 ? ((tokens - 1) >> shift) + 1 : 0; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// The .aligned forms want a warp's threads together, and loops and branches by
// thread come before them.  (Relaxed: nothing but that this CTA runs.)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;");
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of shared memory of the cluster's CTA `rank`, at this CTA's address.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(addr), "r"(rank), "r"(v)
      : "memory");
}
// Asynchronous copy of a word into shared memory, and the wait for this thread's.
__device__ __forceinline__ void copy_4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint32_t ld_l2(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ int dp2a(uint32_t two16, uint32_t four8, int c, bool upper) {
  return upper ? __dp2a_hi(static_cast<int>(two16), static_cast<int>(four8), c)
               : __dp2a_lo(static_cast<int>(two16), static_cast<int>(four8), c);
}

// Larger-is-better order of scores as unsigned numbers; 0 is left for a page
// out of range.
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

// --------------------------------------------------------------------------
// Queries: up and down of a query token, in the order in which lanes use them
// --------------------------------------------------------------------------
constexpr int kQueryHeads = MLAQP_KV4_MAX_HEADS / kSelectHeadGroups;
struct QueryPart {
  // this thread's eight latent channels of its heads, then its rope channels:
  // pairs of BF16, or E4M3 codes in the first two
  uint32_t v[kQueryHeads + 1][4];
};

// Four E4M3 codes as FP16 pairs (exact; NaN stays one).
__device__ __forceinline__ uint2 e4m3x4_f16(uint32_t c) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(c));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) { return f16_lo(v >> 16); }

template <bool E4>
__device__ __forceinline__ void load_query(const Kv4SelectParams& p, int64_t m, QueryPart& q) {
  const int tid = threadIdx.x, chunk = tid % kSelectChunks, g = tid / kSelectChunks;
#pragma unroll
  for (int i = 0; i <= kQueryHeads; ++i) {
    const bool rope = i == kQueryHeads;
    const int h = rope ? tid / kRopeChunks : g + kSelectHeadGroups * i;
    const int c = rope ? kLatent + 8 * (tid % kRopeChunks) : 8 * chunk;
    uint32_t(&v)[4] = q.v[i];
    v[0] = v[1] = v[2] = v[3] = 0;
    if (h >= p.H) continue;
    const int64_t at = m * p.q_ts + h * kOutDim + c;
    if constexpr (E4) {
      asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p.q + at));
    } else {
      const uint4 w = ld_u128(reinterpret_cast<const uint16_t*>(p.q) + at);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
  }
}

// Its largest magnitude, for all: into s.amax, behind a barrier of the caller.
template <bool E4>
__device__ __forceinline__ void query_top(SelectShared& s, QueryPart& q) {
  uint32_t amax = 0;  // bits of the largest magnitude, BF16 or FP16
#pragma unroll
  for (int i = 0; i <= kQueryHeads; ++i) {
    if constexpr (E4) {
      const uint2 x = e4m3x4_f16(q.v[i][0]), y = e4m3x4_f16(q.v[i][1]);
      q.v[i][0] = x.x, q.v[i][1] = x.y, q.v[i][2] = y.x, q.v[i][3] = y.y;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) amax = __vmaxu2(amax, q.v[i][u] & 0x7FFF7FFFu);
  }
  amax = __reduce_max_sync(0xffffffffu, max(amax & 0xFFFFu, amax >> 16));
  if ((threadIdx.x & 31) == 0) s.amax[threadIdx.x >> 5] = amax;
}

// Into `words` ([32 lanes][kScoreLane], this CTA's address) of `ctas` CTAs of
// the cluster, or of this one alone (0).  All threads call.
template <bool E4>
__device__ __forceinline__ void query_words(SelectShared& s, const QueryPart& q, uint32_t* words, int ctas) {
  const int tid = threadIdx.x;
  uint32_t amax = 0;
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) amax = max(amax, s.amax[w]);
  const bool none = amax >= (E4 ? 0x7C00u : 0x7F80u);  // a NaN or an infinity
  // 2047/1024 = 1 + 0x7FE000 * 2^-23
  const uint32_t top = __float_as_uint(E4 ? f16_lo(amax) : __uint_as_float(amax << 16));
  const int f = max(static_cast<int>((top + 0x1FFFu) >> 23) - 127 - 10, -100);
  const float scale = none ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - f) << 23);
  // v + 1.5 * 2^23 rounds v to a whole number n, ties to even, and its bits are
  // those of 1.5 * 2^23 plus n: sums are of integers from there on.
  constexpr float kWhole = 12582912.f;
  constexpr int kWholeBits = 0x4B400000;
  int up[8] = {}, all[8] = {};
  auto add = [&](const uint32_t (&v)[4]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t two = v[u >> 1];
      const float x = E4 ? (u & 1 ? f16_hi(two) : f16_lo(two)) : (u & 1 ? bf16_hi(two) : bf16_lo(two));
      const int n = __float_as_int(__fmaf_rn(x, scale, kWhole));
      all[u] += n - kWholeBits;
      up[u] += max(n, kWholeBits) - kWholeBits;
    }
  };
  auto put = [&](uint32_t* to) {
    uint32_t two[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) two[u] = none ? 0u : static_cast<uint32_t>(up[u] << 16 | (up[u] - all[u]));
    *reinterpret_cast<uint4*>(to) = make_uint4(two[0], two[1], two[2], two[3]);
    *reinterpret_cast<uint4*>(to + 4) = make_uint4(two[4], two[5], two[6], two[7]);
  };
#pragma unroll
  for (int i = 0; i < kQueryHeads; ++i) add(q.v[i]);
  put(&s.part[tid / kSelectChunks][8 * (tid % kSelectChunks)]);
  if (tid < kRopeChunks * MLAQP_KV4_MAX_HEADS) {
#pragma unroll
    for (int u = 0; u < 8; ++u) up[u] = all[u] = 0;
    add(q.v[kQueryHeads]);
    put(&s.rope_part[tid / kRopeChunks][8 * (tid % kRopeChunks)]);
  }
  __syncthreads();
  // Words w < 16 of lane l: pairs of up for the latents 16l.., of down for the
  // same; 16 and 17: of up (l < 16) or down for four rope elements.  Neither half
  // of a sum overflows: 16 heads * 2047.  Two warps see to the rope elements, the
  // others to the latents.
  constexpr int kLatentThreads = kSelectThreads - 64;
  auto word = [&](int l, int w, uint2 sum, bool high) {
    const uint32_t two = high ? __byte_perm(sum.x, sum.y, 0x7632) : __vneg2(__byte_perm(sum.x, sum.y, 0x5410));
    if (ctas == 0) {
      words[l * kScoreLane + w] = two;
    } else {
      const uint32_t at = smem_u32(&words[l * kScoreLane + w]);
      for (int r = 0; r < ctas; ++r) st_cluster(at, r, two);
    }
  };
#pragma unroll
  for (int i = tid; i < 32 * 16 && tid < kLatentThreads; i += kLatentThreads) {
    const int l = i / 16, w = i % 16;
    uint2 sum = make_uint2(0, 0);
#pragma unroll
    for (int a = 0; a < kSelectHeadGroups; ++a) {
      const uint2 x = *reinterpret_cast<const uint2*>(&s.part[a][16 * l + 2 * (w & 7)]);
      sum.x += x.x, sum.y += x.y;
    }
    word(l, w, sum, w < 8);
  }
  if (tid >= kLatentThreads) {
    const int l = (tid - kLatentThreads) / 2, w = tid % 2;
    uint2 sum = make_uint2(0, 0);
#pragma unroll
    for (int a = 0; a < MLAQP_KV4_MAX_HEADS; ++a) {
      const uint2 x = *reinterpret_cast<const uint2*>(&s.rope_part[a][4 * (l & 15) + 2 * w]);
      sum.x += x.x, sum.y += x.y;
    }
    word(l, 16 + w, sum, l < 16);
  }
}

// --------------------------------------------------------------------------
// Scores of four pages at a time
// --------------------------------------------------------------------------

// A lane's share of four digests: 16 bytes of either bound of the latents, 4 of
// the rope part's.
struct PageBatch {
  uint4 hi[kScorePages], lo[kScorePages];
  uint32_t rope[kScorePages];
  // of the digests whose addresses lanes first .. first + 3 hold
  __device__ __forceinline__ void load(const uint8_t* at, int first) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kScorePages; ++u) {
      const uint8_t* d = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(at), first + u));
      hi[u] = ld_u128(d + 16 * lane);
      lo[u] = ld_u128(d + kLatent + 16 * lane);
      rope[u] = ld_u32(d + 2 * kLatent + 4 * lane);
    }
  }
};

// Sums of four pages for the query token of `words`; lane l gets page l % 4's.
__device__ __forceinline__ int2 score_batch(const PageBatch& batch, const uint32_t* words) {
  const int lane = threadIdx.x & 31;
  const uint32_t* w = words + lane * kScoreLane;
  int a[kScorePages], r[kScorePages];
#pragma unroll
  for (int u = 0; u < kScorePages; ++u) a[u] = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint4 x = *reinterpret_cast<const uint4*>(w + 8 * half), y = *reinterpret_cast<const uint4*>(w + 8 * half + 4);
#pragma unroll
    for (int u = 0; u < kScorePages; ++u) {
      const uint4 d = half ? batch.lo[u] : batch.hi[u];
      a[u] = dp2a(x.x, d.x, a[u], false), a[u] = dp2a(x.y, d.x, a[u], true);
      a[u] = dp2a(x.z, d.y, a[u], false), a[u] = dp2a(x.w, d.y, a[u], true);
      a[u] = dp2a(y.x, d.z, a[u], false), a[u] = dp2a(y.y, d.z, a[u], true);
      a[u] = dp2a(y.z, d.w, a[u], false), a[u] = dp2a(y.w, d.w, a[u], true);
    }
  }
  const uint2 z = *reinterpret_cast<const uint2*>(w + 16);
#pragma unroll
  for (int u = 0; u < kScorePages; ++u) {
    r[u] = __reduce_add_sync(0xffffffffu, dp2a(z.y, batch.rope[u], dp2a(z.x, batch.rope[u], 0, false), true));
    a[u] = __reduce_add_sync(0xffffffffu, a[u]);
  }
  const int u = lane & (kScorePages - 1);
  return make_int2(u & 2 ? (u & 1 ? a[3] : a[2]) : (u & 1 ? a[1] : a[0]),
                   u & 2 ? (u & 1 ? r[3] : r[2]) : (u & 1 ? r[1] : r[0]));
}

// Key of a page: its sums, its exponents, negative for a page out of the pool.
__device__ __forceinline__ uint32_t key_of_sums(int2 sums, int exps) {
  const uint32_t ea = exps & 255u, er = exps >> 8 & 255u;
  float f = __fadd_rn(__fmul_rn(static_cast<float>(sums.x), __uint_as_float(ea << 23)),
                      __fmul_rn(static_cast<float>(sums.y), __uint_as_float(er << 23)));
  // (what is not a digest may give a NaN, which no key stands for)
  if (ea == 255u || er == 255u || isnan(f)) f = INFINITY;
  return exps < 0 ? 0u : score_key(f);
}

// --------------------------------------------------------------------------
// Choice of a query token's pages
// --------------------------------------------------------------------------

// Exclusive sums of two numbers over the CTA, in thread order (x, y), and their
// totals (z, w).  Not inlined: code that is run for the first time waits for
// its fetch.
__device__ __noinline__ int4 choose_scan(SelectShared& s, int a, int b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) x += u, y += v;
  }
  __syncthreads();  // of an earlier call
  if (lane == 31) s.scan[warp][0] = x, s.scan[warp][1] = y;
  __syncthreads();
  int4 sum = make_int4(x - a, y - b, 0, 0);
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    if (w < warp) sum.x += s.scan[w][0], sum.y += s.scan[w][1];
    sum.z += s.scan[w][0], sum.w += s.scan[w][1];
  }
  return sum;
}

// What query token m, which sees n tokens, takes anyway, and what lies behind.
// row: its sequence's pages.  All threads call.
__device__ __forceinline__ void put_fixed(const Kv4SelectParams& p, int m, int n, const int32_t* row) {
  const int tid = threadIdx.x;
  const int pages = pages_of(n, p.shift), taken = min(pages, p.k);
  int32_t* out = p.table + m * p.sel_stride;
  if (tid == 0) p.lens[m] = pages > 0 ? ((taken - 1) << p.shift) + (n - ((pages - 1) << p.shift)) : 0;
  for (int r = taken + tid; r < p.k; r += kSelectThreads) out[r] = -1;
  const bool all = pages <= p.k;
  const int head = all ? pages : p.first, fixed = all ? pages : p.first + p.last;
  for (int r = tid; r < fixed; r += kSelectThreads) {
    const int gap = r < head ? 0 : r - head;
    out[r < head ? r : p.k - p.last + gap] = row[r < head ? r : pages - p.last + gap];
  }
}

// The best `keep` of `count` <= kFewKeys keys from `keys` on, in order, into
// `out`: keys in registers, one histogram of 512 places over their range, which
// every warp scans for itself, and the few keys of the place that holds the last
// one taken ranked.  Four barriers.  False, with nothing written, where too many
// fall there.  All threads call.
__device__ __forceinline__ bool choose_few(SelectShared& s, const uint32_t* keys, const int32_t* pages,
                                           int count, int keep, int32_t* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t key[kFewEach];
  const int j0 = kFewEach * tid;
#pragma unroll
  for (int u = 0; u < kFewEach; ++u) key[u] = 0u;
  if (j0 < count) {  // (what lies behind the last one is not used)
    const uint4 x = *reinterpret_cast<const uint4*>(keys + j0);
    key[0] = x.x, key[1] = x.y, key[2] = x.z, key[3] = x.w;
  }
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
  for (int u = 0; u < kFewEach; ++u) {
    if (j0 + u < count) lo = min(lo, key[u]), hi = max(hi, key[u]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  if (tid < kFewBins / 4) reinterpret_cast<uint4*>(s.bins)[tid] = make_uint4(0, 0, 0, 0);
  if (tid == 0) s.found = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) lo = min(lo, s.lo[w]), hi = max(hi, s.hi[w]);
  const int drop = max(32 - __clz(hi - lo) - kFewBinsLog, 0);
#pragma unroll
  for (int u = 0; u < kFewEach; ++u)
    if (j0 + u < count) atomicAdd(&s.bins[(key[u] - lo) >> drop], 1u);
  __syncthreads();
  // the 16 places that hold it: lane l sums places 16 (31 - l) to 16 (31 - l) + 15
  int sum = 0;
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(s.bins + 16 * (31 - lane) + e);
    sum += static_cast<int>(x.x + x.y + (x.z + x.w));
  }
  int above = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, above, d);
    if (lane >= d) above += x;
  }
  int who = __ffs(__ballot_sync(0xffffffffu, keep <= above)) - 1;
  const int top = 16 * (31 - who) + 15;
  const int before16 = __shfl_sync(0xffffffffu, above - sum, who);
  // then the place: lane l < 16 has the l-th from the top
  const int n = static_cast<int>(s.bins[top - (lane & 15)]);
  above = n;
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, above, d);
    if ((lane & 15) >= d) above += x;
  }
  above += before16 - n;
  who = __ffs(__ballot_sync(0xffffffffu, keep <= above + n)) - 1;
  const int place = top - who;
  above = __shfl_sync(0xffffffffu, above, who);
  const int in = __shfl_sync(0xffffffffu, n, who);
  const bool rank = above + in != keep && drop > 0;  // some of them, and they differ
  if (rank && in > kCandidates) return false;
  lo += static_cast<uint32_t>(place) << drop;
  hi = min(hi, lo + ((1u << drop) - 1u));
  if (rank) {
    // every warp ranks those that are left
#pragma unroll
    for (int u = 0; u < kFewEach; ++u)
      if (j0 + u < count && key[u] >= lo && key[u] <= hi) s.candidate[atomicAdd(&s.found, 1)] = key[u];
    __syncthreads();
    const uint32_t mine = lane < in ? s.candidate[lane] : 0u;
    int more = 0, same = 0;
#pragma unroll 1
    for (int c = 0; c < in; ++c) {
      const uint32_t other = __shfl_sync(0xffffffffu, mine, c);
      more += other > mine;
      same += other == mine;
    }
    const bool last = lane < in && above + more < keep && keep <= above + more + same;
    const int who2 = __ffs(__ballot_sync(0xffffffffu, last)) - 1;
    lo = hi = __shfl_sync(0xffffffffu, mine, who2);
    above += __shfl_sync(0xffffffffu, more, who2);
  }
  // taken: keys above hi, and of those from lo to hi the first keep - above
  int mine = 0;  // of this thread: above, equal << 16
#pragma unroll
  for (int u = 0; u < kFewEach; ++u)
    if (j0 + u < count) mine += key[u] > hi ? 1 : key[u] >= lo ? 1 << 16 : 0;
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) s.scan[warp][0] = before;
  __syncthreads();
  before -= mine;
  for (int w = 0; w < warp; ++w) before += s.scan[w][0];
  int nth = before >> 16;
  int at = (before & 0xFFFF) + min(nth, keep - above);
#pragma unroll
  for (int u = 0; u < kFewEach; ++u) {
    if (j0 + u >= count) break;
    const bool mid = key[u] >= lo && key[u] <= hi;
    if (key[u] > hi || (mid && nth < keep - above)) out[at++] = pages[j0 + u];
    nth += mid;
  }
  return true;
}

// The same for any number of keys, by histograms of 2048 places over the range
// that is still open: mostly one or two, then every warp ranks what is left.
// held: the place of the keys in s.keys, -1 where they are in the workspace.
// All threads call.
__device__ __forceinline__ void choose_by_bins(const Kv4SelectParams& p, SelectShared& s, int m, const int32_t* row,
                                               int held_at, int count, int keep) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* out = p.table + m * p.sel_stride;
  const bool held = held_at >= 0;
  const uint32_t* far_keys = p.keys + m * p.width + p.first;
  auto key_of = [&](int j) { return held ? s.keys[held_at + j] : ld_l2(far_keys + j); };

  // the range of the keys
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  __syncthreads();  // the bins of the token before, or the stages, are done with
  for (int j = tid; j < count; j += kSelectThreads) {
    const uint32_t key = key_of(j);
    lo = min(lo, key);
    hi = max(hi, key);
  }
  if (tid == 0) s.found = 0;
  for (int e = tid; e < kBins / 4; e += kSelectThreads) reinterpret_cast<uint4*>(s.bins)[e] = make_uint4(0, 0, 0, 0);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) lo = min(lo, s.lo[w]), hi = max(hi, s.hi[w]);
  // Keys from `lo` to `hi`, `open` bits of them undecided: the place that holds
  // the last one taken, until all in it are taken or all in it are equal.
  int open = 32 - __clz(hi - lo), above = 0, in = count;
  while (open > 0 && above + in != keep) {
    const int drop = max(open - kBinsLog, 0);
    for (int j = tid; j < count; j += kSelectThreads) {
      const uint32_t key = key_of(j);
      if (key >= lo && key - lo <= hi - lo) atomicAdd(&s.bins[(key - lo) >> drop], 1u);
    }
    __syncthreads();
    // thread t: eight bins from the top, cleared for the next round
    unsigned here[kBinsEach] = {};
    int sum = 0;
    {
      uint4* at = reinterpret_cast<uint4*>(s.bins + kBins - kBinsEach * (tid + 1));
      const uint4 x = at[0], y = at[1];
      at[0] = at[1] = make_uint4(0, 0, 0, 0);
      here[0] = y.w, here[1] = y.z, here[2] = y.y, here[3] = y.x;
      here[4] = x.w, here[5] = x.z, here[6] = x.y, here[7] = x.x;
#pragma unroll
      for (int e = 0; e < kBinsEach; ++e) sum += here[e];
    }
    int before = above + choose_scan(s, sum, 0).x;
    if (before < keep && keep <= before + sum) {
#pragma unroll
      for (int e = 0; e < kBinsEach; ++e) {
        const int with = before + static_cast<int>(here[e]);
        if (before < keep && keep <= with) {
          s.from = lo + (static_cast<uint32_t>(kBins - 1 - (tid * kBinsEach + e)) << drop);
          s.above = before;
          s.in = here[e];
        }
        before = with;
      }
    }
    __syncthreads();
    lo = s.from;
    hi = min(hi, lo + ((1u << drop) - 1u));
    above = s.above;
    in = s.in;
    open = drop;
    if (open > 0 && above + in != keep && in <= kCandidates) {
      // few are left: every warp ranks them
      for (int j = tid; j < count; j += kSelectThreads) {
        const uint32_t key = key_of(j);
        if (key >= lo && key <= hi) s.candidate[atomicAdd(&s.found, 1)] = key;
      }
      __syncthreads();
      const uint32_t mine = lane < in ? s.candidate[lane] : 0u;
      int more = 0, same = 0;
#pragma unroll 1
      for (int c = 0; c < in; ++c) {
        const uint32_t key = __shfl_sync(0xffffffffu, mine, c);
        more += key > mine;
        same += key == mine;
      }
      const bool last = lane < in && above + more < keep && keep <= above + more + same;
      const int who = __ffs(__ballot_sync(0xffffffffu, last)) - 1;
      lo = hi = __shfl_sync(0xffffffffu, mine, who);
      above += __shfl_sync(0xffffffffu, more, who);
      open = 0;
    }
  }
  // taken: keys above hi, and of those from lo to hi the first keep - above
  int done = 0, equal = 0;
  for (int j0 = 0; j0 < count; j0 += kSelectThreads * kChooseEach) {
    uint32_t key[kChooseEach];
    int a = 0, e = 0;
    const int j = j0 + tid * kChooseEach;
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      key[u] = j + u < count ? key_of(j + u) : 0;
      if (j + u < count) a += key[u] > hi, e += key[u] >= lo && key[u] <= hi;
    }
    const int4 before = choose_scan(s, a, e);
    int nth = equal + before.y;
    int at = p.first + done + before.x + min(nth, keep - above);
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      if (j + u >= count) break;
      const bool mid = key[u] >= lo && key[u] <= hi;
      if (key[u] > hi || (mid && nth < keep - above)) out[at++] = held ? s.pages[p.first + j + u] : row[p.first + j + u];
      nth += mid;
    }
    done += before.z;
    equal += before.w;
  }
}

// --------------------------------------------------------------------------
// One cluster a sequence: queries, scores, choice
// --------------------------------------------------------------------------
template <bool E4>
__global__ void __launch_bounds__(kSelectThreads, kSelectCtasPerSm)
    mlaqp_kv4_select_kernel(const __grid_constant__ Kv4SelectParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + kWordsAt);  // [q_len][kQueryWords]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = p.cluster, rank = static_cast<int>(cluster_rank());
  const int b = blockIdx.x / ctas;
  pdl_launch_dependents();
  if (ctas > 1) cluster_arrive_relaxed();
  pdl_wait();
  // Several query tokens are shared out: each CTA sees to some of them, for all.
  const bool share = ctas > 1 && p.q_len > 1;
  const int64_t m0 = static_cast<int64_t>(b) * p.q_len;
  const int step = share ? ctas : 1;
  int i = share ? rank : 0;
  QueryPart q;
  if (i < p.q_len) load_query<E4>(p, m0 + i, q);  // (where nothing is to be scored, for nothing)
  const int seq = p.seqs ? p.seqs[b] : b;
  bool bad = seq < 0 || seq >= p.num_seqs;
  int len = 0;
  if (!bad) {
    len = p.seq_lens[seq];
    bad = len < 0 || len > p.table_stride << p.shift || len > p.num_pages << p.shift;
  }
  if (bad) {
    if (tid == 0 && rank == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    len = 0;
  }
  const int32_t* row = p.block_table + (bad ? 0 : seq * p.table_stride);
  // pages to be scored: those between the first and the last ones of the last
  // query token, which sees the most
  const int pages = pages_of(len, p.shift);
  const int count = pages > p.k ? pages - p.first - p.last : 0;
  const int tokens = (p.q_len + ctas - 1) / ctas;  // a CTA chooses for tokens rank, rank + ctas, ..
  const int room = (count + 3) / 4 * 4;            // for a token's keys
  const bool held = count > 0 && pages <= kHeldKeys && static_cast<int64_t>(tokens) * room <= kHeldKeys;
  if (count > 0) {
    const int32_t* between = row + p.first;
    // Batch k of this warp is four entries, its lane u + 4 (k % 8) seeing to entry
    // u: addresses and exponents of eight batches at a time.  In the place of a
    // page out of the pool, and behind the last one, page 0's digest is read and
    // not used.  A page out of the pool is reported here: also where there is nothing
    // to choose.
    const int warps = kSelectWarps * ctas, mine = ctas * warp + rank;  // a last, incomplete round is shared by all CTAs
    const int batches = ((count + kScorePages - 1) / kScorePages - mine + warps - 1) / warps;
    auto in_pool = [&](int page) { return page >= 0 && page < p.num_pages; };
    bool lost = false;  // any of this lane's entries
    auto entry = [&](int k0) {
      const int n = kScorePages * (warps * (k0 + lane / kScorePages) + mine) + lane % kScorePages;
      if (n >= count) return -1;
      const int page = between[n];
      lost |= !in_pool(page);
      return page;
    };
    auto digest_of = [&](int page) { return p.digests + (in_pool(page) ? page : 0) * p.digest_stride; };
    auto exps_of = [&](int page, const uint8_t* digest) {
      const int e = static_cast<int>(ld_u32(digest + 2 * kOutDim) & 0xFFFFu);
      return in_pool(page) ? e : -1;
    };
    // the queries' largest magnitude while the first entries are under way, the rest
    // of the queries while the first digests are
    int next = entry(0);
    if (i < p.q_len) query_top<E4>(s, q);
    __syncthreads();
    const uint8_t *digest = digest_of(next), *next_digest = digest;
    PageBatch even, odd;
    even.load(digest, 0);
    int exps = exps_of(next, digest), next_exps = exps;
    if (ctas > 1) cluster_wait();  // the others are there: their shared memory may be written
    while (i < p.q_len) {
      query_words<E4>(s, q, words + i * kQueryWords, share ? ctas : 0);
      i += step;
      if (i >= p.q_len) break;
      load_query<E4>(p, m0 + i, q);
      __syncthreads();  // (s.amax and s.part have been read)
      query_top<E4>(s, q);
      __syncthreads();
    }
    if (share) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    if (held && rank < p.q_len)  // for the choice
      for (int j = tid; j < pages; j += kSelectThreads) copy_4(smem_u32(&s.pages[j]), row + j);
    // Sums wait in the lanes, four for a batch and query token, until all lanes
    // have some: a warp makes 32 keys at once.
    int2 sums = make_int2(0, 0);
    int sums_exps = 0, filled = 0;
    uint32_t sums_of = kNoPage;  // page between the fixed ones, token << kTokenAt
    const int ctas_log = 31 - __clz(ctas);
    auto put_keys = [&]() {
      if (sums_of != kNoPage) {
        const uint32_t key = key_of_sums(sums, sums_exps);
        const int n = sums_of & ((1u << kTokenAt) - 1u), t = sums_of >> kTokenAt;
        if (!held)
          p.keys[(m0 + t) * p.width + p.first + n] = key;
        else
          st_cluster(smem_u32(&s.keys[(t >> ctas_log) * room + n]), t & (ctas - 1), key);
      }
      sums_of = kNoPage;
      filled = 0;
    };
    // While a batch is scored the one behind it is under way, and its entries
    // and exponents long before.
    auto round = [&](const PageBatch& now, PageBatch& then, int k) {
      if (k % 8 == 0) next = entry(k + 8);
      if (k % 8 == 4) {
        next_digest = digest_of(next);
        next_exps = exps_of(next, next_digest);
      }
      if (k + 1 < batches) then.load(k % 8 < 7 ? digest : next_digest, (k + 1) % 8 * kScorePages);
      const int n = kScorePages * (warps * k + mine) + lane % kScorePages;
      const int e = __shfl_sync(0xffffffffu, exps, k % 8 * kScorePages + lane % kScorePages);
#pragma unroll 1
      for (int t = 0; t < p.q_len; ++t) {
        const int2 sum = score_batch(now, words + t * kQueryWords);
        if (lane / kScorePages == filled) {
          sums = sum;
          sums_exps = e;
          sums_of = n < count ? static_cast<uint32_t>(n) | static_cast<uint32_t>(t) << kTokenAt : kNoPage;
        }
        if (++filled == 32 / kScorePages) put_keys();
      }
      if (k % 8 == 7) digest = next_digest, exps = next_exps;
    };
#pragma unroll 1
    for (int k = 0; k < batches; k += 2) {
      round(even, odd, k);
      if (k + 1 < batches) round(odd, even, k + 1);
    }
    put_keys();
    if (lost) atomicOr(&g_device_status, kDevStatusBadIndex);
    copy_wait();
    if (ctas > 1) cluster_arrive();
  }
  for (int t = rank; t < p.q_len; t += ctas) put_fixed(p, static_cast<int>(m0) + t, max(0, len - (p.q_len - 1 - t)), row);
  if (ctas > 1)
    cluster_wait();  // all keys are there
  else
    __syncthreads();
  if (count == 0) return;
  for (int t = rank; t < p.q_len; t += ctas) {
    const int m = static_cast<int>(m0) + t, at = held ? t / ctas * room : -1;
    const int sees = pages_of(max(0, len - (p.q_len - 1 - t)), p.shift);
    const int keep = p.k - p.first - p.last, from = sees - p.first - p.last;
    if (sees <= p.k || keep == 0) continue;
    if (held && from <= kFewKeys &&
        choose_few(s, s.keys + at, s.pages + p.first, from, keep, p.table + m * p.sel_stride + p.first))
      continue;
    choose_by_bins(p, s, m, row, at, from, keep);
  }
}

const void* select_kernel(bool e4m3) {
  return e4m3 ? reinterpret_cast<const void*>(&mlaqp_kv4_select_kernel<true>)
              : reinterpret_cast<const void*>(&mlaqp_kv4_select_kernel<false>);
}

// CTAs of a sequence.  As many as find room at two an SM, up to 8 (64 sequences
// of up to 512 pages: 10.7 us with 4, 14.0 with 2, 16.3 with 8; 16 sequences of
// up to 569 pages, 4 query tokens: 11.8 with 8, 13.5 with 4, 16.5 with 16), 16
// where those are no more than the SMs (one sequence of 1024 pages: 6.6 us, 8.0
// with 8); no more than have a batch for each warp.
constexpr int kSelectCluster = 8, kSelectWideCluster = 16;
int select_cluster(int B, int64_t width, int sm_count, bool wide) {
  int n = wide && B * kSelectWideCluster <= sm_count ? kSelectWideCluster : kSelectCluster;
  while (n > 1 && B * n > kSelectCtasPerSm * sm_count) n /= 2;
  const int64_t some = kSelectWarps * kScorePages;
  while (n > 1 && n / 2 * some >= width) n /= 2;
  return n;
}

// Whether a device has room for clusters of 16 of either kernel (BF16, E4M3 queries).
std::atomic<bool> g_wide[kMaxDevices][2];

constexpr size_t select_bytes(int q_len) { return kWordsAt + sizeof(uint32_t) * kQueryWords * static_cast<size_t>(q_len); }

}  // namespace

cudaError_t kv4_select(const Kv4SelectParams& params, bool q_e4m3, int sm_count, cudaStream_t stream) {
  Kv4SelectParams p = params;
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  p.cluster = select_cluster(p.B, p.width, sm_count, g_wide[device][q_e4m3].load(std::memory_order_relaxed));
  void* args[1] = {&p};
  return kv4_launch(select_kernel(q_e4m3), static_cast<unsigned>(p.B * p.cluster), kSelectThreads, select_bytes(p.q_len),
                    stream, args, static_cast<unsigned>(p.cluster));
}

cudaError_t kv4_select_setup() {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  cudaFuncAttributes a;
  for (bool e4m3 : {false, true}) {
    const void* k = select_kernel(e4m3);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(select_bytes(MLAQP_KV4_MAX_Q_LEN)));
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSelectWideCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSelectWideCluster, 1, 1);
  cfg.blockDim = dim3(kSelectThreads, 1, 1);
  cfg.dynamicSmemBytes = select_bytes(MLAQP_KV4_MAX_Q_LEN);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (bool e4m3 : {false, true}) {
    int room = 0;
    const cudaError_t asked = cudaOccupancyMaxActiveClusters(&room, select_kernel(e4m3), &cfg);
    if (asked != cudaSuccess) cudaGetLastError();  // then not
    g_wide[device][e4m3].store(asked == cudaSuccess && room > 0, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

cudaError_t device_status_kv4_select(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

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
// Score kernel: the pages that have to be scored form one line over the
// sequences, and every CTA takes an equal stretch.  A warp takes four pages at a
// time, a lane 16 + 16 + 4 bytes of each digest; up and down lie in shared
// memory in the lanes' order, read once for four pages.  Bound by memory (1168
// bytes a page); the chain lengths -> queries -> up, down -> digests is what
// short calls wait for.
//
// Choice kernel: a CTA a query token.  The k-th highest score by histograms of
// 2048 places over the range that is still open (mostly two), then the pages
// from there on in order of position.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kMaxSeqs = MLAQP_MAX_M;

// --------------------------------------------------------------------------
// Scores
// --------------------------------------------------------------------------
constexpr int kScoreChunks = kOutDim / 8;            // of eight channels
constexpr int kScoreHeadGroups = 4;                  // heads h, h + 4, .. of a thread
constexpr int kScoreThreads = kScoreChunks * kScoreHeadGroups;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreCtasPerSm = 2;
constexpr int kScorePages = 4;                       // in flight per warp
constexpr int kScoreWords = 18;                      // pairs of up / down of a lane: 8 + 8 + 2
constexpr int kScoreLane = 20;                       // a lane's words apart: 16-byte loads without bank conflicts
static_assert(kScoreThreads % 32 == 0 && kScoreThreads >= kMaxSeqs, "whole warps, a thread a sequence");

struct ScoreShared {
  int prefix[kMaxSeqs + 1];    // pages to score before each sequence
  int scan[kScoreWarps];
  uint32_t amax[kScoreWarps];
  int part[kScoreHeadGroups][kOutDim];  // up << 16 | down & 0xFFFF, sums over a thread's heads
};

// Number of tokens of call row b (its table row in *seq), 0 where something is
// out of range.
__device__ __forceinline__ int select_len(const Kv4SelectParams& p, int b, int* seq, bool tell) {
  const int s = p.seqs ? p.seqs[b] : b;
  bool bad = s < 0 || s >= p.num_seqs;
  int len = 0;
  if (!bad) {
    len = p.seq_lens[s];
    bad = len < 0 || len > p.table_stride << p.shift || len > p.num_pages << p.shift;
  }
  if (bad && tell) atomicOr(&g_device_status, kDevStatusBadIndex);
  *seq = s;
  return bad ? 0 : len;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return tokens > 0 ? ((tokens - 1) >> shift) + 1 : 0; }

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

// up and down of query token m into `words`, [32 lanes][kScoreLane].
template <bool E4>
__device__ __forceinline__ void score_query(const Kv4SelectParams& p, ScoreShared& s, int64_t m, uint32_t* words) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = tid % kScoreChunks, g = tid / kScoreChunks;
  constexpr int N = MLAQP_KV4_MAX_HEADS / kScoreHeadGroups;
  uint32_t v[N][4];  // BF16 pairs
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = g + kScoreHeadGroups * i;
    v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
    if (h >= p.H) continue;
    const int64_t at = m * p.q_ts + h * kOutDim + 8 * chunk;
    if constexpr (E4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p.q + at);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t two = (u < 2 ? w.x : w.y) >> (16 * (u & 1));
        v[i][u] = mul_bf16x2(e4m3x2_to_bf16x2_scaled(two), 0x7B807B80u);  // 2^120
        if ((two & 0x7Fu) == 0x7Fu || (two & 0x7F00u) == 0x7F00u) v[i][u] = 0x7FC07FC0u;
      }
    } else {
      const uint4 w = ld_u128(reinterpret_cast<const uint16_t*>(p.q) + at);
      v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int u = 0; u < 4; ++u) amax = __vmaxu2(amax, v[i][u] & 0x7FFF7FFFu);
  amax = __reduce_max_sync(0xffffffffu, max(amax & 0xFFFFu, amax >> 16));
  __syncthreads();  // the query before has been read, from here and from `words`
  if (lane == 0) s.amax[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreWarps; ++w) amax = max(amax, s.amax[w]);
  // 2047/1024 = 1 + 0x7FE000 * 2^-23; BF16's exponent and significand are FP32's upper half
  const int f = max(static_cast<int>(((amax << 16) + 0x1FFFu) >> 23) - 127 - 10, -100);
  const float scale = amax >= 0x7F80u ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - f) << 23);
  int up[8] = {}, down[8] = {};
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float x = u & 1 ? bf16_hi(v[i][u >> 1]) : bf16_lo(v[i][u >> 1]);
      const int q = amax >= 0x7F80u ? 0 : __float2int_rn(x * scale);
      up[u] += max(q, 0);
      down[u] += min(q, 0);
    }
#pragma unroll
  for (int u = 0; u < 8; ++u) s.part[g][8 * chunk + u] = up[u] << 16 | (down[u] & 0xFFFF);
  __syncthreads();
  // word w of lane l: pairs of up for the latents 16l.., of down for the same,
  // and of up (l < 16) or down for four rope elements
  for (int i = tid; i < 32 * kScoreWords; i += kScoreThreads) {
    const int l = i / kScoreWords, w = i % kScoreWords;
    const bool rope = w >= 16, high = rope ? l < 16 : w < 8;
    const int c = rope ? kLatent + 4 * (l & 15) + 2 * (w - 16) : 16 * l + 2 * (w & 7);
    uint32_t two = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int sum = 0;
#pragma unroll
      for (int a = 0; a < kScoreHeadGroups; ++a) {
        const int x = s.part[a][c + e];
        sum += high ? x >> 16 : static_cast<int>(static_cast<int16_t>(x & 0xFFFF));
      }
      two |= (static_cast<uint32_t>(sum) & 0xFFFFu) << (16 * e);
    }
    words[l * kScoreLane + w] = two;
  }
  // (the caller's barrier comes before `words` are read)
}

template <bool E4>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtasPerSm)
    mlaqp_kv4_score_kernel(const __grid_constant__ Kv4SelectParams p) {
  __shared__ ScoreShared s;
  extern __shared__ __align__(16) uint32_t words[];  // [q_len][32][kScoreLane]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  // pages to be scored: those between the first and the last ones of the
  // sequence's last query token, which sees the most
  int mine = 0;
  if (tid < p.B) {
    int seq;
    const int pages = pages_of(select_len(p, tid, &seq, false), p.shift);
    mine = pages > p.k ? pages - p.first - p.last : 0;
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) s.scan[warp] = inc;
  __syncthreads();
  for (int w = 0; w < warp; ++w) inc += s.scan[w];
  if (tid < kMaxSeqs) s.prefix[tid + 1] = inc;
  if (tid == 0) s.prefix[0] = 0;
  __syncthreads();
  const int64_t total = s.prefix[kMaxSeqs];
  const int t1 = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  int t = static_cast<int>(total * blockIdx.x / gridDim.x);
  if (t >= t1) return;
  int b = 0;  // the sequence that holds place t
  for (int step = kMaxSeqs / 2; step; step >>= 1)
    if (s.prefix[b + step] <= t) b += step;
#pragma unroll 1
  for (; t < t1; ++b) {
    const int count = min(s.prefix[b + 1], t1) - t;
    if (count <= 0) continue;
    const int j0 = t - s.prefix[b] + p.first;
    t += count;
    const int seq = p.seqs ? p.seqs[b] : b;
    const int32_t* row = p.block_table + seq * p.table_stride + j0;
#pragma unroll 1
    for (int i = 0; i < p.q_len; ++i)
      score_query<E4>(p, s, static_cast<int64_t>(b) * p.q_len + i, words + i * 32 * kScoreLane);
    __syncthreads();
#pragma unroll 1
    for (int n0 = kScorePages * warp; n0 < count; n0 += kScorePages * kScoreWarps) {
      uint4 hi[kScorePages], lo[kScorePages];
      uint32_t pe[kScorePages], exps[kScorePages];
      bool good[kScorePages];
#pragma unroll
      for (int u = 0; u < kScorePages; ++u) {
        hi[u] = lo[u] = make_uint4(0, 0, 0, 0);
        pe[u] = exps[u] = 0;
        const int page = n0 + u < count ? row[n0 + u] : -1;
        good[u] = page >= 0 && page < p.num_pages;
        if (!good[u]) continue;
        const uint8_t* d = p.digests + page * p.digest_stride;
        hi[u] = ld_u128(d + 16 * lane);
        lo[u] = ld_u128(d + kLatent + 16 * lane);
        pe[u] = ld_u32(d + 2 * kLatent + 4 * lane);
        exps[u] = ld_u32(d + 2 * kOutDim);
      }
#pragma unroll 1
      for (int i = 0; i < p.q_len; ++i) {
        const uint32_t* w = words + (i * 32 + lane) * kScoreLane;
        int a[kScorePages], r[kScorePages];
#pragma unroll
        for (int u = 0; u < kScorePages; ++u) a[u] = 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4 x = *reinterpret_cast<const uint4*>(w + 8 * half), y = *reinterpret_cast<const uint4*>(w + 8 * half + 4);
#pragma unroll
          for (int u = 0; u < kScorePages; ++u) {
            const uint4 d = half ? lo[u] : hi[u];
            a[u] = dp2a(x.x, d.x, a[u], false), a[u] = dp2a(x.y, d.x, a[u], true);
            a[u] = dp2a(x.z, d.y, a[u], false), a[u] = dp2a(x.w, d.y, a[u], true);
            a[u] = dp2a(y.x, d.z, a[u], false), a[u] = dp2a(y.y, d.z, a[u], true);
            a[u] = dp2a(y.z, d.w, a[u], false), a[u] = dp2a(y.w, d.w, a[u], true);
          }
        }
        const uint2 z = *reinterpret_cast<const uint2*>(w + 16);
        uint32_t key = 0;
#pragma unroll
        for (int u = 0; u < kScorePages; ++u) {
          r[u] = dp2a(z.y, pe[u], dp2a(z.x, pe[u], 0, false), true);
          a[u] = __reduce_add_sync(0xffffffffu, a[u]);
          r[u] = __reduce_add_sync(0xffffffffu, r[u]);
          const uint32_t ea = exps[u] & 255u, er = exps[u] >> 8 & 255u;
          float f = __fadd_rn(__fmul_rn(static_cast<float>(a[u]), __uint_as_float(ea << 23)),
                              __fmul_rn(static_cast<float>(r[u]), __uint_as_float(er << 23)));
          if (ea == 255u || er == 255u) f = INFINITY;
          if (lane == u) key = good[u] ? score_key(f) : 0u;
        }
        if (lane < kScorePages && n0 + lane < count)
          p.keys[(static_cast<int64_t>(b) * p.q_len + i) * p.width + j0 + n0 + lane] = key;
      }
    }
  }
}

// --------------------------------------------------------------------------
// Choice
// --------------------------------------------------------------------------
constexpr int kChooseThreads = 256;
constexpr int kChooseWarps = kChooseThreads / 32;
constexpr int kChooseEach = 4;             // pages of a thread in one sweep in order
constexpr int kBins = 2048, kBinsLog = 11;
constexpr int kBinsEach = kBins / kChooseThreads;

struct ChooseShared {
  unsigned bins[kBins];
  uint32_t lo[kChooseWarps], hi[kChooseWarps];
  int scan[kChooseWarps][2];
  uint32_t from;   // first key of the place that holds the k-th
  int above, in;   // keys above that place, in it
};

// Exclusive sums of two numbers over the CTA, in thread order; totals in *ta, *tb.
__device__ __forceinline__ int2 choose_scan(ChooseShared& s, int a, int b, int* ta, int* tb) {
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
  int2 before = make_int2(x - a, y - b);
  *ta = *tb = 0;
#pragma unroll
  for (int w = 0; w < kChooseWarps; ++w) {
    if (w < warp) before.x += s.scan[w][0], before.y += s.scan[w][1];
    *ta += s.scan[w][0], *tb += s.scan[w][1];
  }
  return before;
}

__global__ void __launch_bounds__(kChooseThreads) mlaqp_kv4_choose_kernel(const __grid_constant__ Kv4SelectParams p) {
  __shared__ ChooseShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int m = blockIdx.x, b = m / p.q_len, i = m % p.q_len;
  int seq;
  const int len = select_len(p, b, &seq, tid == 0 && i == 0);
  const int n = max(0, len - (p.q_len - 1 - i));
  const int pages = pages_of(n, p.shift);
  const int taken = min(pages, p.k);
  int32_t* out = p.table + m * p.sel_stride;
  if (tid == 0) p.lens[m] = pages > 0 ? ((taken - 1) << p.shift) + (n - ((pages - 1) << p.shift)) : 0;
  for (int r = taken + tid; r < p.k; r += kChooseThreads) out[r] = -1;
  const int32_t* row = p.block_table + seq * p.table_stride;
  if (pages <= p.k) {
    for (int r = tid; r < pages; r += kChooseThreads) out[r] = row[r];
    return;
  }
  for (int r = tid; r < p.first; r += kChooseThreads) out[r] = row[r];
  for (int r = tid; r < p.last; r += kChooseThreads) out[p.k - p.last + r] = row[pages - p.last + r];
  const int keep = p.k - p.first - p.last, count = pages - p.first - p.last;  // of the pages between
  if (keep == 0) return;
  const uint32_t* keys = p.keys + m * p.width + p.first;

  // the range of the keys
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  bool left_out = false;
  for (int j = tid; j < count; j += kChooseThreads) {
    const uint32_t key = keys[j];
    left_out |= key == 0;
    lo = min(lo, key);
    hi = max(hi, key);
  }
  if (left_out) atomicOr(&g_device_status, kDevStatusBadIndex);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kChooseWarps; ++w) lo = min(lo, s.lo[w]), hi = max(hi, s.hi[w]);
  // Keys from `lo` on, `open` bits of them undecided: the place that holds the
  // keep-th highest one, until all in it are taken or all in it are equal.
  int open = 32 - __clz(hi - lo), above = 0, in = count;
  while (open > 0 && above + in != keep) {
    const int drop = max(open - kBinsLog, 0);
    __syncthreads();
    for (int e = tid; e < kBins; e += kChooseThreads) s.bins[e] = 0;
    __syncthreads();
    for (int j = tid; j < count; j += kChooseThreads) {
      const uint32_t key = keys[j];
      if (key >= lo && key - lo <= hi - lo) atomicAdd(&s.bins[(key - lo) >> drop], 1u);
    }
    __syncthreads();
    // thread t: bins from the top
    int sum = 0;
#pragma unroll
    for (int e = 0; e < kBinsEach; ++e) sum += s.bins[kBins - 1 - (tid * kBinsEach + e)];
    int total, none;
    int before = above + choose_scan(s, sum, 0, &total, &none).x;
    if (before < keep && keep <= before + sum) {
#pragma unroll 1
      for (int e = 0;; ++e) {
        const int bin = kBins - 1 - (tid * kBinsEach + e);
        const int here = s.bins[bin];
        if (keep <= before + here) {
          s.from = lo + (static_cast<uint32_t>(bin) << drop);
          s.above = before;
          s.in = here;
          break;
        }
        before += here;
      }
    }
    __syncthreads();
    lo = s.from;
    hi = lo + ((1u << drop) - 1u);
    above = s.above;
    in = s.in;
    open = drop;
  }
  // taken: keys above hi, and of those from lo to hi the first keep - above
  int done = 0, equal = 0;
  for (int j0 = 0; j0 < count; j0 += kChooseThreads * kChooseEach) {
    uint32_t key[kChooseEach];
    int a = 0, e = 0;
    const int j = j0 + tid * kChooseEach;
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      key[u] = j + u < count ? keys[j + u] : 0;
      if (j + u < count) a += key[u] > hi, e += key[u] >= lo && key[u] <= hi;
    }
    int all_a, all_e;
    const int2 before = choose_scan(s, a, e, &all_a, &all_e);
    int nth = equal + before.y;
    int at = done + before.x + min(nth, keep - above);
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      if (j + u >= count) break;
      const bool mid = key[u] >= lo && key[u] <= hi;
      if (key[u] > hi || (mid && nth < keep - above)) out[p.first + at++] = row[p.first + j + u];
      nth += mid;
    }
    done += all_a;
    equal += all_e;
  }
}

const void* score_kernel(bool e4m3) {
  return e4m3 ? reinterpret_cast<const void*>(&mlaqp_kv4_score_kernel<true>)
              : reinterpret_cast<const void*>(&mlaqp_kv4_score_kernel<false>);
}

}  // namespace

cudaError_t kv4_select(const Kv4SelectParams& p, bool q_e4m3, int sm_count, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4SelectParams*>(&p)};
  const size_t words = sizeof(uint32_t) * 32 * kScoreLane * p.q_len;
  const cudaError_t e = kv4_launch(score_kernel(q_e4m3), static_cast<unsigned>(kScoreCtasPerSm * sm_count), kScoreThreads,
                                   words, stream, args);
  if (e != cudaSuccess) return e;
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_choose_kernel), static_cast<unsigned>(p.B * p.q_len),
                    kChooseThreads, 0, stream, args);
}

cudaError_t kv4_select_setup() {
  cudaFuncAttributes a;
  cudaError_t e = cudaSuccess;
  for (const void* k : {score_kernel(false), score_kernel(true)}) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sizeof(uint32_t) * 32 * kScoreLane * MLAQP_KV4_MAX_Q_LEN);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
  }
  return e == cudaSuccess ? cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_choose_kernel)) : e;
}

cudaError_t device_status_kv4_select(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

// Page operations of the 4-bit latent cache: extend, fork, release, compact
// and plain page copies.
//
// The state is a count per page (0: free), a table row and a length per
// sequence, all in device memory.  Operations that hand out pages run as one
// CTA: it turns the counts into a bitmap in shared memory (32 pages a word),
// scans the words' populations once, and then finds the k-th free page by a
// search of that scan, so that "lowest index first, in list order" costs no
// serial walk.  Page contents are moved by a second kernel of many CTAs that
// reads the jobs the first one left in the workspace; it is bound by memory:
// a compaction that moves 214 MB reads and writes them in 63 us, 6.8 TB/s.
// The one-CTA kernels are chains of loads and barriers, 7 to 12 us cold up to
// 16384 pages (release: a CTA a sequence, 5 to 6 us); beyond, the counts are
// what one SM takes in: extending by a page takes 17 us in a pool of 2^17, 83
// in one of 2^20 (some 7 less with 16-byte loads of the counts, not worth a
// second path).

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;  // 16-byte vectors a copying thread has in flight

// Job lists in the workspace: [0] the number of jobs, from word 4 the lists.
constexpr int kJobsAt = 4;

__device__ __forceinline__ void report(unsigned bits) { atomicOr(&g_device_status, bits); }

template <class T>
__device__ __forceinline__ T warp_inclusive(T v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, d);
    if (static_cast<int>(threadIdx.x & 31) >= d) v += u;
  }
  return v;
}

// Exclusive sum over the CTA's kPlanThreads values; *total gets the sum.
template <class T>
__device__ __forceinline__ T block_exclusive(T v, T* scratch, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T inc = warp_inclusive(v);
  __syncthreads();  // scratch may still be read from an earlier call
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  if (warp == 0) scratch[lane] = warp_inclusive(scratch[lane]);
  __syncthreads();
  *total = scratch[kPlanWarps - 1];
  return inc - v + (warp ? scratch[warp - 1] : T(0));
}

struct PlanShared {
  unsigned long long scan64[kPlanWarps];
  int scan[kPlanWarps];
  int prefix[kPlanThreads];  // free pages before the thread's words
  // one batch of list items
  int seq[kPlanThreads];
  int other[kPlanThreads];   // extend: tokens; fork: parent
  int len[kPlanThreads];
  int first[kPlanThreads];   // rank of the item's first new page, or -1: left out
};

// Bitmap of the pages whose count is zero (free = true) or not; bits at and
// above num_pages are 0.
__device__ __forceinline__ void build_bitmap(const int32_t* ref, int num_pages, int words, uint32_t* map, bool free) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w0 = warp * 4; w0 < words; w0 += kPlanWarps * 4) {
    int c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = 32 * (w0 + u) + lane;
      c[u] = i < num_pages ? ref[i] : (free ? 1 : 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t bits = __ballot_sync(0xffffffffu, (c[u] == 0) == free);
      if (lane == 0 && w0 + u < words) map[w0 + u] = bits;
    }
  }
  __syncthreads();
}

// Index of the k-th set bit (k < total): the thread whose words hold it by
// bisection of the prefix sums, then the word, then the bit.
__device__ __forceinline__ int kth_page(const uint32_t* map, const int* prefix, int wpt, int k) {
  int lo = 0, hi = kPlanThreads;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= k) lo = mid; else hi = mid;
  }
  int r = k - prefix[lo];
  int w = lo * wpt;
  while (r >= __popc(map[w])) r -= __popc(map[w++]);
  uint32_t bits = map[w];
  for (; r > 0; --r) bits &= bits - 1;
  return 32 * w + __ffs(bits) - 1;
}

// The common start of extend and fork; returns the number of free pages.
__device__ __forceinline__ int plan_free(const Kv4Tables& t, uint32_t* map, PlanShared& s, int* wpt_out) {
  const int words = (t.num_pages + 31) / 32;
  const int wpt = (words + kPlanThreads - 1) / kPlanThreads;
  build_bitmap(t.ref_count, t.num_pages, words, map, true);
  int mine = 0;
  for (int k = 0; k < wpt; ++k) {  // each lane begins at another of its words: they are wpt words, so many banks, apart
    const int w = threadIdx.x * wpt + (k + threadIdx.x) % wpt;
    if (w < words) mine += __popc(map[w]);
  }
  int total = 0;
  s.prefix[threadIdx.x] = block_exclusive(mine, s.scan, &total);
  __syncthreads();
  *wpt_out = wpt;
  return total;
}

__global__ void __launch_bounds__(kPlanThreads) mlaqp_kv4_extend_kernel(const __grid_constant__ Kv4PagesParams p) {
  extern __shared__ uint32_t map[];
  __shared__ PlanShared s;
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Tables& t = p.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int wpt = 0;
  const int n_free = plan_free(t, map, s, &wpt);
  const int mask = (1 << t.shift) - 1;
  int taken = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0, seq = -1, add = 0, len = 0;
    if (i < p.n) {
      seq = p.list_a[i];
      add = p.list_b[i];
      bool ok = seq >= 0 && seq < t.num_seqs && add >= 0 && add <= p.max_new;
      if (ok) {
        len = t.seq_lens[seq];
        const int64_t end = static_cast<int64_t>(len) + add;
        ok = len >= 0 && end <= t.stride << t.shift && end <= 0x7fffffff;
      }
      if (ok && add > 0 && (len & mask) != 0) {  // the page that the new tokens begin in
        const int pg = t.block_table[seq * t.stride + (len >> t.shift)];
        ok = pg >= 0 && pg < t.num_pages;
      }
      if (ok) {
        // in 64 bits: a length near the int's end plus the page's mask
        need = static_cast<int>((static_cast<int64_t>(len) + add + mask) >> t.shift) -
               static_cast<int>((static_cast<int64_t>(len) + mask) >> t.shift);
      } else {
        report(kDevStatusBadIndex);
        seq = -1;
      }
    }
    unsigned long long sum = 0;
    const unsigned long long before = block_exclusive(static_cast<unsigned long long>(need), s.scan64, &sum);
    const long long first = taken + static_cast<long long>(before);
    if (seq >= 0 && need > 0 && first + need > n_free) {
      report(kDevStatusOutOfPages);
      seq = -1;
    }
    s.seq[tid] = seq;
    s.other[tid] = add;
    s.len[tid] = len;
    s.first[tid] = static_cast<int>(first);
    // later items' ranks lie behind this batch's, whether or not it fitted
    taken = static_cast<int>(min(static_cast<unsigned long long>(taken) + sum, 1ull << 30));
    __syncthreads();
    for (int k = warp; k < min(kPlanThreads, p.n - base); k += kPlanWarps) {
      const int sq = s.seq[k];
      int32_t* out = p.slots + static_cast<int64_t>(base + k) * p.max_new;
      if (sq < 0) {
        for (int j = lane; j < p.max_new; j += 32) out[j] = -1;
        continue;
      }
      const int ln = s.len[k], ad = s.other[k];
      int32_t* row = t.block_table + sq * t.stride;
      const int have = static_cast<int>((static_cast<int64_t>(ln) + mask) >> t.shift);
      const int end = static_cast<int>((static_cast<int64_t>(ln) + ad + mask) >> t.shift);
      for (int j = have + lane; j < end; j += 32) {
        const int pg = kth_page(map, s.prefix, wpt, s.first[k] + j - have);
        row[j] = pg;
        t.ref_count[pg] = 1;
      }
      __syncwarp();
      for (int j = lane; j < p.max_new; j += 32) {
        const int at = ln + j;
        out[j] = j < ad ? (row[at >> t.shift] << t.shift) | (at & mask) : -1;
      }
      if (lane == 0) t.seq_lens[sq] = ln + ad;
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kPlanThreads) mlaqp_kv4_fork_kernel(const __grid_constant__ Kv4PagesParams p) {
  extern __shared__ uint32_t map[];
  __shared__ PlanShared s;
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Tables& t = p.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int wpt = 0;
  const int n_free = plan_free(t, map, s, &wpt);
  const int mask = (1 << t.shift) - 1;
  int32_t* src = p.ws + kJobsAt;
  int32_t* dst = src + p.n;
  int32_t* tok = dst + p.n;
  // All lengths are taken as they were before the call: a child of one item
  // that is the parent of another still counts as empty there.
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int parent = p.list_a[i], child = p.list_b[i];
    bool ok = parent >= 0 && parent < t.num_seqs && child >= 0 && child < t.num_seqs && child != parent;
    int len = 0;
    if (ok) {
      len = t.seq_lens[parent];
      ok = len >= 0 && len <= t.stride << t.shift && t.seq_lens[child] == 0;
    }
    if (!ok) report(kDevStatusBadIndex);
    tok[i] = ok ? len : -1;
  }
  __syncthreads();
  // A parent with a page that is none is left out before free pages are
  // counted: neither its child nor a count may learn of it halfway.
  for (int i = warp; i < p.n; i += kPlanWarps) {
    const int len = tok[i];
    if (len <= 0) continue;
    const int32_t* from = t.block_table + p.list_a[i] * t.stride;
    const int pages = static_cast<int>((static_cast<int64_t>(len) + mask) >> t.shift);
    bool bad = false;
    for (int j = lane; j < pages; j += 32) {
      const int pg = from[j];
      bad |= pg < 0 || pg >= t.num_pages;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) {
      report(kDevStatusBadIndex);
      tok[i] = -1;
    }
  }
  __syncthreads();
  int taken = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    const int len = i < p.n ? tok[i] : -1;
    const int need = len > 0 && (len & mask) != 0;
    int child = len >= 0 ? p.list_b[i] : -1;
    const int parent = len >= 0 ? p.list_a[i] : 0;
    int sum = 0;
    const int first = taken + block_exclusive(need, s.scan, &sum);
    if (child >= 0 && need && first >= n_free) {
      report(kDevStatusOutOfPages);
      child = -1;
    }
    taken += sum;
    s.seq[tid] = child;
    s.other[tid] = parent;
    s.len[tid] = len;
    s.first[tid] = first;
    __syncthreads();
    for (int k = warp; k < min(kPlanThreads, p.n - base); k += kPlanWarps) {
      const int ch = s.seq[k];
      const int ln = s.len[k], full = ln >> t.shift, tail = ln & mask;
      const int32_t* from = t.block_table + s.other[k] * t.stride;
      int job_src = -1, job_dst = -1;
      if (ch >= 0) {
        int32_t* row = t.block_table + ch * t.stride;
        for (int j = lane; j < full; j += 32) {
          const int pg = from[j];
          row[j] = pg;
          atomicAdd(&t.ref_count[pg], 1);
        }
        if (tail) {
          job_src = from[full];
          job_dst = kth_page(map, s.prefix, wpt, s.first[k]);
        }
        if (lane == 0) {
          if (tail) {
            row[full] = job_dst;
            t.ref_count[job_dst] = 1;
          }
          t.seq_lens[ch] = ln;
        }
      }
      if (lane == 0) {
        src[base + k] = job_src;
        dst[base + k] = job_dst;
        tok[base + k] = tail;
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(128) mlaqp_kv4_release_kernel(const __grid_constant__ Kv4PagesParams p) {
  __shared__ int s_len;
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Tables& t = p.t;
  const int seq = p.list_a[blockIdx.x];
  if (seq < 0 || seq >= t.num_seqs) {
    if (threadIdx.x == 0) report(kDevStatusBadIndex);
    return;
  }
  // The exchange lets a sequence that is listed twice go once only; a bad
  // length stays as it is.
  if (threadIdx.x == 0) {
    const int len = t.seq_lens[seq];
    const bool ok = len >= 0 && len <= t.stride << t.shift;
    if (!ok) report(kDevStatusBadIndex);
    s_len = ok && atomicCAS(&t.seq_lens[seq], len, 0) == len ? len : 0;
  }
  __syncthreads();
  const int len = s_len;
  const int pages = static_cast<int>((static_cast<int64_t>(len) + (1 << t.shift) - 1) >> t.shift);
  int32_t* row = t.block_table + seq * t.stride;
  for (int j = threadIdx.x; j < pages; j += blockDim.x) {
    const int pg = row[j];
    row[j] = -1;
    if (pg >= 0 && pg < t.num_pages) atomicSub(&t.ref_count[pg], 1); else report(kDevStatusBadIndex);
  }
}

// Workspace of a compaction: src[half], dst[half], then job[num_pages], which
// move a page is part of (written for moved pages only).
__host__ __device__ inline int compact_half(int num_pages) { return num_pages / 2 + 1; }

__global__ void __launch_bounds__(kPlanThreads) mlaqp_kv4_compact_kernel(const __grid_constant__ Kv4PagesParams p) {
  extern __shared__ uint32_t map[];
  __shared__ PlanShared s;
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Tables& t = p.t;
  const int tid = threadIdx.x;
  const int words = (t.num_pages + 31) / 32;
  const int wpt = (words + kPlanThreads - 1) / kPlanThreads;
  build_bitmap(t.ref_count, t.num_pages, words, map, false);
  const int w0 = min(words, tid * wpt), w1 = min(words, (tid + 1) * wpt);
  int live = 0, n = 0;
  for (int w = w0; w < w1; ++w) live += __popc(map[w]);
  block_exclusive(live, s.scan, &n);
  // free pages below n and live pages at or above it: as many of each
  auto below = [n](int w) { return 32 * w + 32 <= n ? 0xffffffffu : (32 * w >= n ? 0u : (1u << (n & 31)) - 1u); };
  unsigned long long mine = 0, total = 0;
  for (int w = w0; w < w1; ++w)
    mine += (static_cast<unsigned long long>(__popc(~map[w] & below(w))) << 32) | __popc(map[w] & ~below(w));
  const unsigned long long at = block_exclusive(mine, s.scan64, &total);
  int32_t* src = p.ws + kJobsAt;
  int32_t* dst = src + compact_half(t.num_pages);
  int32_t* job = dst + compact_half(t.num_pages);
  int h = static_cast<int>(at >> 32), m = static_cast<int>(at & 0xffffffffu);
  for (int w = w0; w < w1; ++w) {
    for (uint32_t b = ~map[w] & below(w); b; b &= b - 1) dst[h++] = 32 * w + __ffs(b) - 1;
    for (uint32_t b = map[w] & ~below(w); b; b &= b - 1) src[m++] = 32 * w + __ffs(b) - 1;
  }
  __syncthreads();
  const int moves = static_cast<int>(total & 0xffffffffu);
  for (int k = tid; k < moves; k += kPlanThreads) {
    const int a = src[k], b = dst[k];
    job[a] = k;
    t.ref_count[b] = t.ref_count[a];
    t.ref_count[a] = 0;
  }
  if (tid == 0) {
    p.ws[0] = moves;
    *p.n_live = n;
  }
}

// Move page contents: job k copies the first tok[k] tokens (tok null: the
// whole page) of page src[k] to page dst[k] in every layer; a negative index
// is no job.  job, when given, also rewrites the table entries that point at
// or above *n_live: those whose page is a job's source, so that what an earlier
// call left in the workspace counts for nothing.
struct CopyJobs {
  const int32_t* count;  // null: n
  int n;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* tok;
  const int32_t* job;
  const int32_t* n_live;
};

__global__ void __launch_bounds__(kCopyThreads)
    mlaqp_kv4_copy_kernel(const __grid_constant__ Kv4Cache c, const __grid_constant__ Kv4Tables t,
                          const __grid_constant__ CopyJobs jobs) {
  pdl_launch_dependents();
  pdl_wait();
  const int n = jobs.count ? *jobs.count : jobs.n;
  const int page = 1 << c.shift;
  const int64_t tasks = static_cast<int64_t>(n) * c.layers;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int k = static_cast<int>(task / c.layers), layer = static_cast<int>(task % c.layers);
    const int a = jobs.src[k], b = jobs.dst[k];
    if (a < 0 || b < 0) continue;
    if (a >= c.num_pages || b >= c.num_pages) {
      if (threadIdx.x == 0) report(kDevStatusBadIndex);
      continue;
    }
    const int tok = jobs.tok ? jobs.tok[k] : page;
    const uint8_t* from = c.base + layer * c.layer_stride + a * c.page_stride;
    uint8_t* to = c.base + layer * c.layer_stride + b * c.page_stride;
    // 25 vectors a token: 16 of codes, 8 of rope, 1 of scales
    const int vecs = 25 * tok;
    for (int v0 = threadIdx.x; v0 < vecs; v0 += kCopyThreads * kCopyVecs) {
      uint4 v[kCopyVecs];
      uint32_t off[kCopyVecs];
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u) {
        const int i = v0 + u * kCopyThreads;
        off[u] = i < 16 * tok ? 16 * i
                              : (i < 24 * tok ? kKv4CodeBytes * page + 16 * (i - 16 * tok)
                                              : (kKv4CodeBytes + kKv4RopeBytes) * page + 16 * (i - 24 * tok));
        if (i < vecs) v[u] = ld_u128(from + off[u]);
      }
#pragma unroll
      for (int u = 0; u < kCopyVecs; ++u)
        if (v0 + u * kCopyThreads < vecs) st_u128(to + off[u], v[u]);
    }
  }
  if (jobs.job == nullptr) return;
  const int live = *jobs.n_live;
  const int64_t entries = t.num_seqs * t.stride;
  for (int64_t i = blockIdx.x * kCopyThreads + threadIdx.x; i < entries; i += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    const int len = t.seq_lens[i / t.stride];
    if ((i % t.stride) << t.shift >= len) continue;
    const int pg = t.block_table[i];
    if (pg < live) continue;  // in place, or none
    const int k = pg < t.num_pages ? jobs.job[pg] : -1;
    if (k >= 0 && k < n && jobs.src[k] == pg) t.block_table[i] = jobs.dst[k]; else report(kDevStatusBadIndex);
  }
}

size_t bitmap_bytes(int num_pages) { return static_cast<size_t>((num_pages + 31) / 32) * 4; }

cudaError_t launch_copy(const Kv4PagesParams& p, const CopyJobs& jobs, int sm_count, cudaStream_t stream) {
  Kv4Cache c = p.cache;
  Kv4Tables t = p.t;
  CopyJobs j = jobs;
  void* args[3] = {&c, &t, &j};
  const int64_t tasks = static_cast<int64_t>(jobs.n) * p.cache.layers;
  const int64_t most = 8ll * sm_count;
  const int64_t work = jobs.job ? most : (tasks < most ? tasks : most);
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_copy_kernel), static_cast<unsigned>(work), kCopyThreads, 0,
                    stream, args);
}

}  // namespace

cudaError_t kv4_extend(const Kv4PagesParams& p, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4PagesParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_extend_kernel), 1, kPlanThreads, bitmap_bytes(p.t.num_pages),
                    stream, args);
}

cudaError_t kv4_fork(const Kv4PagesParams& p, int sm_count, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4PagesParams*>(&p)};
  const cudaError_t e = kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_fork_kernel), 1, kPlanThreads,
                                   bitmap_bytes(p.t.num_pages), stream, args);
  if (e != cudaSuccess) return e;
  const int32_t* src = p.ws + kJobsAt;
  return launch_copy(p, CopyJobs{nullptr, p.n, src, src + p.n, src + 2 * static_cast<int64_t>(p.n), nullptr, nullptr},
                     sm_count, stream);
}

cudaError_t kv4_release(const Kv4PagesParams& p, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4PagesParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_release_kernel), static_cast<unsigned>(p.n), 128, 0, stream,
                    args);
}

cudaError_t kv4_compact(const Kv4PagesParams& p, int sm_count, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4PagesParams*>(&p)};
  const cudaError_t e = kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_compact_kernel), 1, kPlanThreads,
                                   bitmap_bytes(p.t.num_pages), stream, args);
  if (e != cudaSuccess) return e;
  const int half = compact_half(p.t.num_pages);
  const int32_t* src = p.ws + kJobsAt;
  return launch_copy(p, CopyJobs{p.ws, p.t.num_pages / 2, src, src + half, nullptr, src + 2 * half, p.n_live}, sm_count,
                     stream);
}

cudaError_t kv4_copy_pages(const Kv4PagesParams& p, int sm_count, cudaStream_t stream) {
  return launch_copy(p, CopyJobs{nullptr, p.n, p.list_a, p.list_b, nullptr, nullptr, nullptr}, sm_count, stream);
}

cudaError_t kv4_pages_setup() {
  const void* plans[3] = {reinterpret_cast<const void*>(&mlaqp_kv4_extend_kernel),
                          reinterpret_cast<const void*>(&mlaqp_kv4_fork_kernel),
                          reinterpret_cast<const void*>(&mlaqp_kv4_compact_kernel)};
  for (const void* fn : plans) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(bitmap_bytes(1 << 20)));
    if (e != cudaSuccess) return e;
  }
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_release_kernel));
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_copy_kernel));
  return e;
}

int64_t kv4_pages_workspace(int num_pages, int n) {
  const int64_t fork = 3ll * n, compact = 2ll * compact_half(num_pages) + num_pages;
  return 4 * (kJobsAt + (fork > compact ? fork : compact));
}

cudaError_t device_status_kv4_pages(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

// What the entry points of the 4-bit cache share: argument checks (everything
// the host can see is checked before the device is touched) and kernels made
// ready at the first call.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <string>

#include "mlaqp_host.h"
#include "mlaqp_kv4.h"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int page_shift(int page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

inline int bad_arg(const std::string& msg) { return host_fail(MLAQP_ERR_INVALID_ARG, msg); }

struct Range {
  uintptr_t lo, hi;
};
inline Range span(const void* p, uint64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + bytes};
}
inline bool overlaps(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

inline int check_pool(int num_pages, int page_size) {
  if (page_shift(page_size) < 0) return host_fail(MLAQP_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (num_pages < 1) return bad_arg("num_pages must be >= 1");
  if (num_pages > MLAQP_KV4_MAX_PAGES) return host_fail(MLAQP_ERR_UNSUPPORTED, "num_pages must be <= 2^20");
  return MLAQP_OK;
}

// The cache of `layers` layers (layer_stride 0 and layers 1: one layer).
inline int check_cache(const void* cache, int64_t page_stride, int64_t layer_stride, int layers, int num_pages,
                       int page_size, Kv4Cache* out) {
  const int st = check_pool(num_pages, page_size);
  if (st != MLAQP_OK) return st;
  if (!cache) return bad_arg("cache is required");
  if (!aligned(cache, 16)) return bad_arg("cache must be 16-byte aligned");
  const int64_t page = mlaqp_kv4_page_bytes(page_size);
  if (page_stride < page || page_stride % 16 != 0)
    return bad_arg("page_stride must be >= 400*page_size bytes and a multiple of 16");
  if (layers < 1) return bad_arg("layers must be >= 1");
  if (layers > 1) {
    if (layer_stride < 0 || layer_stride % 16 != 0) return bad_arg("layer_stride must be >= 0 and a multiple of 16");
    // whole layers one behind the other, or layers interleaved within a page's stride
    const bool outer = layer_stride >= page_stride * (num_pages - 1) + page;
    const bool inner = layer_stride >= page && page_stride >= layer_stride * (layers - 1) + page;
    if (!outer && !inner) return bad_arg("the layers' pages overlap (page_stride, layer_stride)");
  }
  *out = Kv4Cache{static_cast<uint8_t*>(const_cast<void*>(cache)), page_stride, layers > 1 ? layer_stride : 0,
                  layers, num_pages, page_shift(page_size)};
  return MLAQP_OK;
}

inline Range cache_span(const Kv4Cache& c) {
  return span(c.base, static_cast<uint64_t>(c.page_stride) * (c.num_pages - 1) +
                          static_cast<uint64_t>(c.layer_stride) * (c.layers - 1) +
                          (static_cast<uint64_t>(MLAQP_KV4_TOKEN_BYTES) << c.shift));
}

// What is read of a block table: no more of a row than a sequence can have pages.
inline Range table_span(const int32_t* block_table, int64_t stride, int num_seqs, int num_pages) {
  const uint64_t row = static_cast<uint64_t>(stride < num_pages ? stride : num_pages);
  return span(block_table, 4 * (static_cast<uint64_t>(num_seqs - 1) * static_cast<uint64_t>(stride) + row));
}

inline int check_list(const int32_t* list, int n, const char* what) {
  if (n < 0) return bad_arg("n must be >= 0");
  if (n > 0 && (!list || !aligned(list, 4))) return bad_arg(std::string(what) + " must be a 4-byte aligned list");
  return MLAQP_OK;
}

// Which groups of kernels are ready, by device.
template <int Groups>
struct ReadyGroups {
  std::atomic<bool> ready[kMaxDevices][Groups];
  std::mutex mutex;
};

// The current (or given) device checked and the group's kernels made ready on
// it, once per device, by set_up(group).  The first call sees to all groups, so
// that others may have their first call inside a graph capture.
template <int Groups, class SetUp>
int ready_device(ReadyGroups<Groups>& groups, int device, int group, SetUp set_up, int* sm_count) {
  int dev = 0;
  const int st = host_device(device, &dev, sm_count);
  if (st != MLAQP_OK) return st;
  std::atomic<bool>& ready = groups.ready[dev][group];
  if (!ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(groups.mutex);
    if (!ready.load(std::memory_order_acquire)) {
      int prev = -1;
      cudaError_t e = cudaGetDevice(&prev);
      if (e == cudaSuccess && prev != dev) e = cudaSetDevice(dev);
      for (int g = 0; g < Groups && e == cudaSuccess; ++g) {
        if (groups.ready[dev][g].load(std::memory_order_relaxed)) continue;
        const cudaError_t up = set_up(g);
        if (up == cudaSuccess) groups.ready[dev][g].store(true, std::memory_order_release);
        else if (g == group) e = up;
        else cudaGetLastError();  // its own calls will say so
      }
      if (prev >= 0 && prev != dev) cudaSetDevice(prev);
      if (e != cudaSuccess) return host_fail_cuda("preparing the 4-bit cache kernels", e);
    }
  }
  return MLAQP_OK;
}

inline int launched(cudaError_t e) { return e == cudaSuccess ? MLAQP_OK : host_fail_cuda("cudaLaunchKernelExC", e); }

}  // namespace mlaqp

// Launch interfaces of the 4-bit cache kernels, between the argument checks
// of mlaqp_kv4_api.cu and the kernels' translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace mlaqp {

constexpr int kMaxDevices = 64;  // that a process can use

// Launch with programmatic dependent launch: every kernel of the 4-bit cache
// waits for the previous one before it touches memory.
inline cudaError_t kv4_launch(const void* fn, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                              void** args, unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

struct Kv4Cache {
  uint8_t* base;
  int64_t page_stride;   // bytes
  int64_t layer_stride;  // bytes (page operations)
  int layers;
  int num_pages;
  int shift;             // log2(page_size)
};

struct Kv4RowsParams {
  Kv4Cache cache;
  const uint16_t* latent;  // append
  const uint16_t* k_pe;
  int64_t latent_ts, k_pe_ts;
  uint16_t* out;           // gather
  int64_t out_ts;
  const int32_t* slots;
  int T;
};
cudaError_t kv4_append(const Kv4RowsParams& p, cudaStream_t stream);
cudaError_t kv4_gather(const Kv4RowsParams& p, cudaStream_t stream);
cudaError_t kv4_rows_setup();

struct Kv4RopeParams {
  Kv4Cache cache;
  const uint16_t* latent;
  const uint16_t* k_pe;
  int64_t latent_ts, k_pe_ts;
  const uint16_t* norm_weight;  // nullptr: no norm
  float eps;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* q_out;
  int64_t q_out_ts, q_out_hs;
  int H;
  const int32_t* positions;
  const float* cos_sin;
  int num_positions;
  const int32_t* slots;
  int T;
};
cudaError_t kv4_append_rope(const Kv4RopeParams& p, bool halves, cudaStream_t stream);
cudaError_t kv4_rope_setup();

struct Kv4DigestParams {
  Kv4Cache cache;
  uint8_t* digests;
  int64_t digest_stride;   // bytes
  const int32_t* block_table;
  int64_t table_stride;
  int num_seqs;
  const int32_t* seq_lens;
  const int32_t* seqs;
  const int32_t* new_tokens;
  int n, max_new;
  int per;                 // pages of an item that are looked at (set by kv4_digest)
};
cudaError_t kv4_digest(const Kv4DigestParams& p, int sm_count, cudaStream_t stream);
cudaError_t kv4_digest_setup();

struct Kv4SelectParams {
  const uint8_t* q;
  int64_t q_ts;            // elements
  const uint8_t* digests;
  int64_t digest_stride;   // bytes
  int num_pages, shift;
  const int32_t* block_table;
  int64_t table_stride;
  int num_seqs;
  const int32_t* seq_lens;
  const int32_t* seqs;
  int B, q_len, H;
  int k, first, last;
  int32_t* table;
  int64_t sel_stride;
  int32_t* lens;
  uint32_t* keys;          // [B*q_len][width]
  int64_t width;
  int cluster;             // CTAs of a sequence (set by kv4_select)
};
cudaError_t kv4_select(const Kv4SelectParams& p, bool q_e4m3, int sm_count, cudaStream_t stream);
cudaError_t kv4_select_setup();

// The sequence tables that the page operations change.
struct Kv4Tables {
  int32_t* block_table;
  int64_t stride;      // entries per row
  int num_seqs;
  int32_t* seq_lens;
  int32_t* ref_count;
  int num_pages;
  int shift;
};
struct Kv4PagesParams {
  Kv4Tables t;
  Kv4Cache cache;
  const int32_t* list_a;  // extend: seqs; fork: parents; release: seqs; copy: src
  const int32_t* list_b;  // extend: new_tokens; fork: children; copy: dst
  int n;
  int32_t* slots;         // extend
  int max_new;
  int32_t* n_live;        // compact
  int32_t* ws;            // fork, compact: copy jobs
};
cudaError_t kv4_extend(const Kv4PagesParams& p, cudaStream_t stream);
cudaError_t kv4_fork(const Kv4PagesParams& p, int sm_count, cudaStream_t stream);
cudaError_t kv4_release(const Kv4PagesParams& p, cudaStream_t stream);
cudaError_t kv4_compact(const Kv4PagesParams& p, int sm_count, cudaStream_t stream);
cudaError_t kv4_copy_pages(const Kv4PagesParams& p, int sm_count, cudaStream_t stream);
cudaError_t kv4_pages_setup();
int64_t kv4_pages_workspace(int num_pages, int n);

struct Kv4AttendParams {
  Kv4Cache cache;
  const uint8_t* q;
  int64_t q_ts;            // elements
  const float* q_scale;    // E4M3 queries
  const int32_t* block_table;
  int64_t table_stride;
  int num_seqs;
  const int32_t* seq_lens;
  const int32_t* seqs;
  int B, q_len, H;
  float softmax_scale;
  uint16_t* x;
  int64_t x_ts;
  float* lse;
  uint8_t* ws;
  uint32_t wait_ns;        // limit of a wait in the attention kernel
  int held;                // test of the waits: the hand-over that never happens, 0: none
  unsigned held_first, held_count;  // its barriers, which expect an arrival too many (set by kv4_attend)
};
// The hand-overs between the attention kernel's warps, in the order of its
// barriers: copies landed, copy units free, scales, rope rows landed, rope rows
// free, codes converted, their tiles free, scores, scores read, probabilities,
// output products, queries, output read.
constexpr int kAttStages = 13;
cudaError_t kv4_attend(const Kv4AttendParams& p, bool q_e4m3, int sm_count, cudaStream_t stream);
cudaError_t kv4_attend_setup(int rows);  // 16 or 32: the kernels for that many rows
int kv4_attend_rows(int q_len, int H);   // of a row group
int64_t kv4_attend_workspace(int B, int q_len, int H, int sm_count);

}  // namespace mlaqp

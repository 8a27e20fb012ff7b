// Host side of the C ABI declared in include/mlaqp_kv4.h: argument checks
// and launches.  Everything the host can see is checked before the device is
// touched; what only the device can see (indexes, lengths) is checked by the
// kernels.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "mlaqp_kv4_checks.h"

namespace {

using mlaqp::aligned;
using mlaqp::bad_arg;
using mlaqp::cache_span;
using mlaqp::check_cache;
using mlaqp::check_list;
using mlaqp::check_pool;
using mlaqp::host_fail;
using mlaqp::launched;
using mlaqp::overlaps;
using mlaqp::page_shift;
using mlaqp::Range;
using mlaqp::span;

// Kernels whose attributes are set together.  A build in which one group
// cannot run leaves the others usable.
enum Group { kRowsGroup, kPagesGroup, kAttend16Group, kAttend32Group, kGroups };

mlaqp::ReadyGroups<kGroups> g_ready;

cudaError_t set_up(Group group) {
  switch (group) {
    case kRowsGroup: return mlaqp::kv4_rows_setup();
    case kPagesGroup: return mlaqp::kv4_pages_setup();
    case kAttend16Group: return mlaqp::kv4_attend_setup(16);
    default: return mlaqp::kv4_attend_setup(32);
  }
}

Group attend_group(int q_len, int H) {
  return mlaqp::kv4_attend_rows(q_len, H) == 16 ? kAttend16Group : kAttend32Group;
}

// The current (or given) device checked and the group's kernels made ready on it.
int kv4_device(int device, Group group, int* sm_count) {
  return mlaqp::ready_device(g_ready, device, group, [](int g) { return set_up(static_cast<Group>(g)); }, sm_count);
}

int check_tables(int32_t* block_table, int64_t stride, int num_seqs, int32_t* seq_lens, int32_t* ref_count,
                 int num_pages, int page_size, mlaqp::Kv4Tables* out) {
  const int st = check_pool(num_pages, page_size);
  if (st != MLAQP_OK) return st;
  if (!block_table || !seq_lens || !ref_count) return bad_arg("block_table, seq_lens and ref_count are required");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(ref_count, 4))
    return bad_arg("block_table, seq_lens and ref_count must be 4-byte aligned");
  if (num_seqs < 1) return bad_arg("num_seqs must be >= 1");
  if (stride < 1 || stride > (1ll << 31)) return bad_arg("block_table_stride must be in 1..2^31");
  *out = mlaqp::Kv4Tables{block_table, stride, num_seqs, seq_lens, ref_count, num_pages, page_shift(page_size)};
  return MLAQP_OK;
}

}  // namespace

extern "C" {

int64_t mlaqp_kv4_page_bytes(int page_size) {
  return page_shift(page_size) < 0 ? 0 : static_cast<int64_t>(MLAQP_KV4_TOKEN_BYTES) * page_size;
}

int mlaqp_kv4_append(const void* latent, int64_t latent_token_stride, const void* k_pe, int64_t k_pe_token_stride,
                     void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* slots, int T,
                     mlaqp_stream_t stream) {
  mlaqp::Kv4RowsParams p = {};
  int st = check_cache(cache, page_stride, 0, 1, num_pages, page_size, &p.cache);
  if (st != MLAQP_OK) return st;
  if (T < 0) return bad_arg("T must be >= 0");
  if (T == 0) return MLAQP_OK;
  if (!latent || !k_pe || !slots) return bad_arg("latent, k_pe and slots are required");
  if (!aligned(latent, 16) || !aligned(k_pe, 16)) return bad_arg("latent and k_pe must be 16-byte aligned");
  if (!aligned(slots, 4)) return bad_arg("slots must be 4-byte aligned");
  if (latent_token_stride < 0 || latent_token_stride % 8 != 0 || k_pe_token_stride < 0 || k_pe_token_stride % 8 != 0)
    return bad_arg("latent and k_pe strides must be >= 0 and multiples of 8 elements");
  const Range c = cache_span(p.cache);
  if (overlaps(c, span(latent, 2ull * ((T - 1) * static_cast<uint64_t>(latent_token_stride) + 512))) ||
      overlaps(c, span(k_pe, 2ull * ((T - 1) * static_cast<uint64_t>(k_pe_token_stride) + 64))) ||
      overlaps(c, span(slots, 4ull * T)))
    return bad_arg("the cache overlaps an input");
  int sms = 0;
  st = kv4_device(-1, kRowsGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.latent = static_cast<const uint16_t*>(latent);
  p.k_pe = static_cast<const uint16_t*>(k_pe);
  p.latent_ts = latent_token_stride;
  p.k_pe_ts = k_pe_token_stride;
  p.slots = slots;
  p.T = T;
  return launched(mlaqp::kv4_append(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_gather(const void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* slots, int T,
                     void* out, int64_t out_token_stride, mlaqp_stream_t stream) {
  mlaqp::Kv4RowsParams p = {};
  int st = check_cache(cache, page_stride, 0, 1, num_pages, page_size, &p.cache);
  if (st != MLAQP_OK) return st;
  if (T < 0) return bad_arg("T must be >= 0");
  if (T == 0) return MLAQP_OK;
  if (!slots || !out) return bad_arg("slots and out are required");
  if (!aligned(slots, 4)) return bad_arg("slots must be 4-byte aligned");
  if (!aligned(out, 16)) return bad_arg("out must be 16-byte aligned");
  if (out_token_stride < 576 || out_token_stride % 8 != 0)
    return bad_arg("out_token_stride must be >= 576 elements and a multiple of 8");
  const Range o = span(out, 2ull * ((T - 1) * static_cast<uint64_t>(out_token_stride) + 576));
  if (overlaps(o, cache_span(p.cache)) || overlaps(o, span(slots, 4ull * T))) return bad_arg("out overlaps an input");
  int sms = 0;
  st = kv4_device(-1, kRowsGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.out = static_cast<uint16_t*>(out);
  p.out_ts = out_token_stride;
  p.slots = slots;
  p.T = T;
  return launched(mlaqp::kv4_gather(p, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

int check_attend_sizes(int B, int q_len, int H) {
  if (H < 1 || H > MLAQP_KV4_MAX_HEADS) return host_fail(MLAQP_ERR_UNSUPPORTED, "num_heads must be in 1..16");
  if (q_len < 1 || q_len > MLAQP_KV4_MAX_Q_LEN) return host_fail(MLAQP_ERR_UNSUPPORTED, "q_len must be in 1..16");
  if (B < 0) return bad_arg("B must be >= 0");
  if (static_cast<int64_t>(B) * q_len > MLAQP_MAX_M) return host_fail(MLAQP_ERR_UNSUPPORTED, "B*q_len must be <= 256");
  return MLAQP_OK;
}

}  // namespace

}  // extern "C"

namespace {

constexpr uint32_t kWaitNs = 1000000000u;
static_assert(MLAQP_KV4_ATTEND_STAGES == mlaqp::kAttStages, "the public number of hand-overs");

int attend_impl(const void* q, int64_t q_token_stride, int q_dtype, const float* q_scale, const void* cache,
                int64_t page_stride, int num_pages, int page_size, const int32_t* block_table,
                int64_t block_table_stride, int num_seqs, const int32_t* seq_lens, const int32_t* seqs, int B, int q_len,
                int H, float softmax_scale, void* x, int64_t x_token_stride, float* lse, void* workspace,
                int64_t workspace_bytes, uint32_t wait_ns, int held, mlaqp_stream_t stream) {
  mlaqp::Kv4AttendParams p = {};
  if (q_dtype != MLAQP_OUT_BF16 && q_dtype != MLAQP_OUT_E4M3) return bad_arg("unknown q_dtype");
  const bool e4m3 = q_dtype == MLAQP_OUT_E4M3;
  int st = check_attend_sizes(B, q_len, H);
  if (st != MLAQP_OK) return st;
  st = check_cache(cache, page_stride, 0, 1, num_pages, page_size, &p.cache);
  if (st != MLAQP_OK) return st;
  if (B == 0) return MLAQP_OK;
  if (!q || !block_table || !seq_lens || !x) return bad_arg("q, block_table, seq_lens and x are required");
  if (e4m3 && !q_scale) return bad_arg("E4M3 queries require q_scale");
  if (!e4m3 && q_scale) return bad_arg("BF16 queries take no q_scale (pass NULL)");
  if (!aligned(q, 16) || !aligned(x, 16)) return bad_arg("q and x must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(seqs, 4) || !aligned(lse, 4) ||
      !aligned(q_scale, 4))
    return bad_arg("block_table, seq_lens, seqs, lse and q_scale must be 4-byte aligned");
  const int eb = e4m3 ? 1 : 2;
  if (q_token_stride < 576ll * H || (q_token_stride * eb) % 16 != 0)
    return bad_arg("q_token_stride must be >= 576*H elements and a multiple of 16 bytes");
  if (x_token_stride < 512ll * H || x_token_stride % 8 != 0)
    return bad_arg("x_token_stride must be >= 512*H elements and a multiple of 8");
  if (num_seqs < 1) return bad_arg("num_seqs must be >= 1");
  if (!seqs && num_seqs < B) return bad_arg("num_seqs must be >= B where seqs is NULL");
  if (block_table_stride < 1 || block_table_stride > (1ll << 31)) return bad_arg("block_table_stride must be in 1..2^31");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return bad_arg("softmax_scale must be finite and > 0");
  const int M = B * q_len;
  const Range outs[3] = {span(x, 2ull * ((M - 1) * static_cast<uint64_t>(x_token_stride) + 512ull * H)),
                         span(lse, lse ? 4ull * M * H : 0),
                         span(workspace, workspace && workspace_bytes > 0 ? static_cast<uint64_t>(workspace_bytes) : 0)};
  const Range ins[6] = {span(q, static_cast<uint64_t>(eb) * ((M - 1) * static_cast<uint64_t>(q_token_stride) + 576ull * H)),
                        cache_span(p.cache),
                        mlaqp::table_span(block_table, block_table_stride, num_seqs, num_pages),
                        span(seq_lens, 4ull * num_seqs),
                        span(seqs, seqs ? 4ull * B : 0),
                        span(q_scale, q_scale ? 4 : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : ins)
      if (overlaps(outs[i], r)) return bad_arg("x, lse or workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return bad_arg("x, lse and workspace overlap");
  }
  int sms = 0;
  st = kv4_device(-1, attend_group(q_len, H), &sms);
  if (st != MLAQP_OK) return st;
  if (!workspace || !aligned(workspace, 16)) return bad_arg("workspace must be a 16-byte aligned buffer");
  if (workspace_bytes < mlaqp::kv4_attend_workspace(B, q_len, H, sms))
    return bad_arg("workspace is smaller than mlaqp_kv4_attend_workspace()");
  p.q = static_cast<const uint8_t*>(q);
  p.q_ts = q_token_stride;
  p.q_scale = q_scale;
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.num_seqs = num_seqs;
  p.seq_lens = seq_lens;
  p.seqs = seqs;
  p.B = B;
  p.q_len = q_len;
  p.H = H;
  p.softmax_scale = softmax_scale;
  p.x = static_cast<uint16_t*>(x);
  p.x_ts = x_token_stride;
  p.lse = lse;
  p.ws = static_cast<uint8_t*>(workspace);
  p.wait_ns = wait_ns;
  p.held = held;
  return launched(mlaqp::kv4_attend(p, e4m3, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int mlaqp_kv4_attend(const void* q, int64_t q_token_stride, int q_dtype, const float* q_scale, const void* cache,
                     int64_t page_stride, int num_pages, int page_size, const int32_t* block_table,
                     int64_t block_table_stride, int num_seqs, const int32_t* seq_lens, const int32_t* seqs, int B,
                     int q_len, int H, float softmax_scale, void* x, int64_t x_token_stride, float* lse,
                     void* workspace, int64_t workspace_bytes, mlaqp_stream_t stream) {
  return attend_impl(q, q_token_stride, q_dtype, q_scale, cache, page_stride, num_pages, page_size, block_table,
                     block_table_stride, num_seqs, seq_lens, seqs, B, q_len, H, softmax_scale, x, x_token_stride, lse,
                     workspace, workspace_bytes, kWaitNs, 0, stream);
}

int mlaqp_debug_kv4_attend_bounded_wait(const void* q, int64_t q_token_stride, int q_dtype, const float* q_scale,
                                        const void* cache, int64_t page_stride, int num_pages, int page_size,
                                        const int32_t* block_table, int64_t block_table_stride, int num_seqs,
                                        const int32_t* seq_lens, const int32_t* seqs, int B, int q_len, int H,
                                        float softmax_scale, void* x, int64_t x_token_stride, float* lse,
                                        void* workspace, int64_t workspace_bytes, unsigned int wait_limit_ns, int held,
                                        mlaqp_stream_t stream) {
  if (wait_limit_ns == 0 || wait_limit_ns > kWaitNs) return bad_arg("wait_limit_ns must be in 1..10^9");
  if (held < 0 || held > MLAQP_KV4_ATTEND_STAGES) return bad_arg("held must be in 0..MLAQP_KV4_ATTEND_STAGES");
  return attend_impl(q, q_token_stride, q_dtype, q_scale, cache, page_stride, num_pages, page_size, block_table,
                     block_table_stride, num_seqs, seq_lens, seqs, B, q_len, H, softmax_scale, x, x_token_stride, lse,
                     workspace, workspace_bytes, wait_limit_ns, held, stream);
}

int64_t mlaqp_kv4_attend_workspace(int B, int q_len, int H, int device) {
  if (check_attend_sizes(B, q_len, H) != MLAQP_OK) return -1;
  int sms = 0;
  if (kv4_device(device, attend_group(q_len, H), &sms) != MLAQP_OK) return -1;
  return mlaqp::kv4_attend_workspace(B, q_len, H, sms);
}

int mlaqp_kv4_extend(int32_t* block_table, int64_t block_table_stride, int num_seqs, int32_t* seq_lens,
                     int32_t* ref_count, int num_pages, int page_size, const int32_t* seqs, const int32_t* new_tokens,
                     int n, int32_t* slots, int max_new, mlaqp_stream_t stream) {
  mlaqp::Kv4PagesParams p = {};
  int st = check_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, &p.t);
  if (st == MLAQP_OK) st = check_list(seqs, n, "seqs");
  if (st == MLAQP_OK) st = check_list(new_tokens, n, "new_tokens");
  if (st != MLAQP_OK) return st;
  if (max_new < 1) return bad_arg("max_new must be >= 1");
  if (n == 0) return MLAQP_OK;
  if (!slots || !aligned(slots, 4)) return bad_arg("slots must be a 4-byte aligned buffer");
  int sms = 0;
  st = kv4_device(-1, kPagesGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.list_a = seqs;
  p.list_b = new_tokens;
  p.n = n;
  p.slots = slots;
  p.max_new = max_new;
  return launched(mlaqp::kv4_extend(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_fork(int32_t* block_table, int64_t block_table_stride, int num_seqs, int32_t* seq_lens,
                   int32_t* ref_count, int num_pages, int page_size, const int32_t* parents, const int32_t* children,
                   int n, void* cache, int64_t page_stride, int64_t layer_stride, int layers, void* workspace,
                   int64_t workspace_bytes, mlaqp_stream_t stream) {
  mlaqp::Kv4PagesParams p = {};
  int st = check_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, &p.t);
  if (st == MLAQP_OK) st = check_cache(cache, page_stride, layer_stride, layers, num_pages, page_size, &p.cache);
  if (st == MLAQP_OK) st = check_list(parents, n, "parents");
  if (st == MLAQP_OK) st = check_list(children, n, "children");
  if (st != MLAQP_OK) return st;
  if (n == 0) return MLAQP_OK;
  if (!workspace || !aligned(workspace, 16)) return bad_arg("workspace must be a 16-byte aligned buffer");
  if (workspace_bytes < mlaqp::kv4_pages_workspace(num_pages, n))
    return bad_arg("workspace is smaller than mlaqp_kv4_pages_workspace()");
  int sms = 0;
  st = kv4_device(-1, kPagesGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.list_a = parents;
  p.list_b = children;
  p.n = n;
  p.ws = static_cast<int32_t*>(workspace);
  return launched(mlaqp::kv4_fork(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_release(int32_t* block_table, int64_t block_table_stride, int num_seqs, int32_t* seq_lens,
                      int32_t* ref_count, int num_pages, int page_size, const int32_t* seqs, int n,
                      mlaqp_stream_t stream) {
  mlaqp::Kv4PagesParams p = {};
  int st = check_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, &p.t);
  if (st == MLAQP_OK) st = check_list(seqs, n, "seqs");
  if (st != MLAQP_OK) return st;
  if (n == 0) return MLAQP_OK;
  int sms = 0;
  st = kv4_device(-1, kPagesGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.list_a = seqs;
  p.n = n;
  return launched(mlaqp::kv4_release(p, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_compact(int32_t* block_table, int64_t block_table_stride, int num_seqs, int32_t* seq_lens,
                      int32_t* ref_count, int num_pages, int page_size, void* cache, int64_t page_stride,
                      int64_t layer_stride, int layers, int32_t* n_live, void* workspace, int64_t workspace_bytes,
                      mlaqp_stream_t stream) {
  mlaqp::Kv4PagesParams p = {};
  int st = check_tables(block_table, block_table_stride, num_seqs, seq_lens, ref_count, num_pages, page_size, &p.t);
  if (st == MLAQP_OK) st = check_cache(cache, page_stride, layer_stride, layers, num_pages, page_size, &p.cache);
  if (st != MLAQP_OK) return st;
  if (!n_live || !aligned(n_live, 4)) return bad_arg("n_live must be a 4-byte aligned int");
  if (!workspace || !aligned(workspace, 16)) return bad_arg("workspace must be a 16-byte aligned buffer");
  if (workspace_bytes < mlaqp::kv4_pages_workspace(num_pages, 0))
    return bad_arg("workspace is smaller than mlaqp_kv4_pages_workspace()");
  int sms = 0;
  st = kv4_device(-1, kPagesGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.n_live = n_live;
  p.ws = static_cast<int32_t*>(workspace);
  return launched(mlaqp::kv4_compact(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_copy_pages(void* cache, int64_t page_stride, int64_t layer_stride, int layers, int num_pages,
                         int page_size, const int32_t* src, const int32_t* dst, int n, mlaqp_stream_t stream) {
  mlaqp::Kv4PagesParams p = {};
  int st = check_cache(cache, page_stride, layer_stride, layers, num_pages, page_size, &p.cache);
  if (st == MLAQP_OK) st = check_list(src, n, "src");
  if (st == MLAQP_OK) st = check_list(dst, n, "dst");
  if (st != MLAQP_OK) return st;
  if (n == 0) return MLAQP_OK;
  int sms = 0;
  st = kv4_device(-1, kPagesGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.list_a = src;
  p.list_b = dst;
  p.n = n;
  return launched(mlaqp::kv4_copy_pages(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t mlaqp_kv4_pages_workspace(int num_pages, int n) {
  if (num_pages < 1 || num_pages > MLAQP_KV4_MAX_PAGES || n < 0) {
    host_fail(MLAQP_ERR_INVALID_ARG, "num_pages must be in 1..2^20 and n >= 0");
    return -1;
  }
  return mlaqp::kv4_pages_workspace(num_pages, n);
}

int mlaqp_kv4_prewarm(int device) {
  int sms = 0, st = MLAQP_OK;
  for (int g = 0; g < kGroups && st == MLAQP_OK; ++g) st = kv4_device(device, static_cast<Group>(g), &sms);
  return st;
}

}  // extern "C"

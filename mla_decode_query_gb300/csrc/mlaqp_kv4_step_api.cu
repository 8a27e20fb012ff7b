// Host side of the C ABI declared in include/mlaqp_kv4_step.h: argument checks
// and launches.  What only the device can see (indexes, lengths) is checked by
// the kernels.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "mlaqp_kv4_checks.h"
#include "mlaqp_kv4_step.h"

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
using mlaqp::table_span;

enum Group { kRopeGroup, kDigestGroup, kSelectGroup, kGroups };
mlaqp::ReadyGroups<kGroups> g_ready;

int step_device(int device, Group group, int* sm_count) {
  return mlaqp::ready_device(
      g_ready, device, group,
      [](int g) {
        return g == kRopeGroup ? mlaqp::kv4_rope_setup() : g == kDigestGroup ? mlaqp::kv4_digest_setup() : mlaqp::kv4_select_setup();
      },
      sm_count);
}

// T rows of `bytes` bytes, `stride` bytes apart.
struct Rows {
  const void* at;
  uint64_t bytes, stride;
};

// Whether rows that are written and rows that are read share a byte.  Rows of
// the same stride (views into one buffer) may lie side by side.
bool rows_overlap(Rows a, Rows b, int T) {
  if (!a.at || !b.at || !a.bytes || !b.bytes) return false;
  const uint64_t n = static_cast<uint64_t>(T - 1);
  if (!overlaps(span(a.at, n * a.stride + a.bytes), span(b.at, n * b.stride + b.bytes))) return false;
  if (T == 1 || a.stride != b.stride || a.stride < a.bytes || b.stride < b.bytes) return true;
  // place of b's rows behind a's, whichever two
  const int64_t stride = static_cast<int64_t>(a.stride);
  int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at)) % stride;
  if (off < 0) off += stride;
  return off < static_cast<int64_t>(a.bytes) || off + static_cast<int64_t>(b.bytes) > stride;
}

int check_sequences(const int32_t* block_table, int64_t stride, int num_seqs, const int32_t* seq_lens) {
  if (!block_table || !seq_lens) return bad_arg("block_table and seq_lens are required");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4)) return bad_arg("block_table and seq_lens must be 4-byte aligned");
  if (num_seqs < 1) return bad_arg("num_seqs must be >= 1");
  if (stride < 1 || stride > (1ll << 31)) return bad_arg("block_table_stride must be in 1..2^31");
  return MLAQP_OK;
}

int check_digests(const void* digests, int64_t stride) {
  if (!digests || !aligned(digests, 16)) return bad_arg("digests must be a 16-byte aligned buffer");
  if (stride < MLAQP_KV4_DIGEST_BYTES || stride % 16 != 0)
    return bad_arg("digest_stride must be >= 1168 bytes and a multiple of 16");
  return MLAQP_OK;
}

Range digest_span(const void* digests, int64_t stride, int num_pages) {
  return span(digests, static_cast<uint64_t>(stride) * (num_pages - 1) + MLAQP_KV4_DIGEST_BYTES);
}

int check_select_sizes(int B, int q_len) {
  if (q_len < 1 || q_len > MLAQP_KV4_MAX_Q_LEN) return host_fail(MLAQP_ERR_UNSUPPORTED, "q_len must be in 1..16");
  if (B < 0) return bad_arg("B must be >= 0");
  if (static_cast<int64_t>(B) * q_len > MLAQP_MAX_M) return host_fail(MLAQP_ERR_UNSUPPORTED, "B*q_len must be <= 256");
  return MLAQP_OK;
}

// Pages of a sequence that there can be a score for.
int64_t key_width(int64_t block_table_stride, int num_pages) {
  return std::min<int64_t>(block_table_stride, num_pages);
}

}  // namespace

extern "C" {

int mlaqp_kv4_append_rope(const void* latent, int64_t latent_token_stride, const void* norm_weight, float norm_eps,
                          const void* k_pe, int64_t k_pe_token_stride, const void* q_pe, int64_t q_token_stride,
                          int64_t q_head_stride, void* q_pe_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                          int H, const int32_t* positions, const float* cos_sin, int num_positions, int rope_style,
                          void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* slots, int T,
                          mlaqp_stream_t stream) {
  mlaqp::Kv4RopeParams p = {};
  int st = check_cache(cache, page_stride, 0, 1, num_pages, page_size, &p.cache);
  if (st != MLAQP_OK) return st;
  if (rope_style != MLAQP_ROPE_INTERLEAVED && rope_style != MLAQP_ROPE_HALVES) return bad_arg("unknown rope_style");
  if (H < 0) return bad_arg("H must be >= 0");
  if (H > 128) return host_fail(MLAQP_ERR_UNSUPPORTED, "H must be <= 128");
  if (T < 0) return bad_arg("T must be >= 0");
  if (num_positions < 1) return bad_arg("num_positions must be >= 1");
  if (T == 0) return MLAQP_OK;
  if (!latent || !k_pe || !positions || !cos_sin || !slots)
    return bad_arg("latent, k_pe, positions, cos_sin and slots are required");
  if (!aligned(latent, 16) || !aligned(k_pe, 16) || !aligned(norm_weight, 16) || !aligned(cos_sin, 16))
    return bad_arg("latent, k_pe, norm_weight and cos_sin must be 16-byte aligned");
  if (!aligned(positions, 4) || !aligned(slots, 4)) return bad_arg("positions and slots must be 4-byte aligned");
  if (latent_token_stride < 0 || latent_token_stride % 8 != 0 || k_pe_token_stride < 0 || k_pe_token_stride % 8 != 0)
    return bad_arg("latent and k_pe strides must be >= 0 and multiples of 8 elements");
  if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps))) return bad_arg("norm_eps must be finite and >= 0");
  Rows in = {nullptr, 0, 0}, out = {nullptr, 0, 0};
  if (H > 0) {
    if (!q_pe || !q_pe_out) return bad_arg("q_pe and q_pe_out are required where H > 0");
    if (!aligned(q_pe, 16) || !aligned(q_pe_out, 16)) return bad_arg("q_pe and q_pe_out must be 16-byte aligned");
    if (q_token_stride < 0 || q_token_stride % 8 != 0 || q_head_stride < 0 || q_head_stride % 8 != 0)
      return bad_arg("q_pe strides must be >= 0 and multiples of 8 elements");
    if (q_out_token_stride < 0 || q_out_token_stride % 8 != 0 || q_out_head_stride < 0 || q_out_head_stride % 8 != 0)
      return bad_arg("q_pe_out strides must be >= 0 and multiples of 8 elements");
    if (H > 1 && q_out_head_stride < 64) return bad_arg("q_out_head_stride must be >= 64 elements");
    const int64_t out_row = (H - 1) * q_out_head_stride + 64;
    if (T > 1 && q_out_token_stride < out_row) return bad_arg("the tokens' rows of q_pe_out overlap");
    in = Rows{q_pe, 2 * (static_cast<uint64_t>(H - 1) * q_head_stride + 64), 2 * static_cast<uint64_t>(q_token_stride)};
    out = Rows{q_pe_out, 2 * static_cast<uint64_t>(out_row), 2 * static_cast<uint64_t>(q_out_token_stride)};
    const bool in_place = q_pe == q_pe_out && (T == 1 || q_token_stride == q_out_token_stride) &&
                          (H == 1 || q_head_stride == q_out_head_stride);
    if (!in_place && rows_overlap(out, in, T)) return bad_arg("q_pe_out overlaps q_pe and is not the same view");
  } else if (q_pe || q_pe_out) {
    return bad_arg("q_pe and q_pe_out must be NULL where H is 0");
  }
  const Rows lat = {latent, 1024, 2 * static_cast<uint64_t>(latent_token_stride)};
  const Rows key = {k_pe, 128, 2 * static_cast<uint64_t>(k_pe_token_stride)};
  if (rows_overlap(out, lat, T) || rows_overlap(out, key, T)) return bad_arg("q_pe_out overlaps latent or k_pe");
  const Range c = cache_span(p.cache);
  const uint64_t n = static_cast<uint64_t>(T - 1);
  const Range out_span = span(out.at, out.at ? n * out.stride + out.bytes : 0);
  const Range rest[4] = {span(norm_weight, norm_weight ? 1024 : 0), span(positions, 4ull * T), span(slots, 4ull * T),
                         span(cos_sin, 256ull * num_positions)};
  for (const Range& r : rest)
    if (overlaps(c, r) || overlaps(out_span, r)) return bad_arg("the cache or q_pe_out overlaps an input");
  for (const Rows& r : {lat, key, in, out})
    if (r.at && overlaps(c, span(r.at, n * r.stride + r.bytes))) return bad_arg("the cache overlaps an input or q_pe_out");
  int sms = 0;
  st = step_device(-1, kRopeGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.latent = static_cast<const uint16_t*>(latent);
  p.k_pe = static_cast<const uint16_t*>(k_pe);
  p.latent_ts = latent_token_stride;
  p.k_pe_ts = k_pe_token_stride;
  p.norm_weight = static_cast<const uint16_t*>(norm_weight);
  p.eps = norm_eps;
  p.q = static_cast<const uint16_t*>(q_pe);
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.q_out = static_cast<uint16_t*>(q_pe_out);
  p.q_out_ts = q_out_token_stride;
  p.q_out_hs = q_out_head_stride;
  p.H = H;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.num_positions = num_positions;
  p.slots = slots;
  p.T = T;
  return launched(mlaqp::kv4_append_rope(p, rope_style == MLAQP_ROPE_HALVES, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_digest(const void* cache, int64_t page_stride, int num_pages, int page_size, const int32_t* block_table,
                     int64_t block_table_stride, int num_seqs, const int32_t* seq_lens, const int32_t* seqs,
                     const int32_t* new_tokens, int n, int max_new, void* digests, int64_t digest_stride,
                     mlaqp_stream_t stream) {
  mlaqp::Kv4DigestParams p = {};
  int st = check_cache(cache, page_stride, 0, 1, num_pages, page_size, &p.cache);
  if (st == MLAQP_OK) st = check_sequences(block_table, block_table_stride, num_seqs, seq_lens);
  if (st == MLAQP_OK) st = check_digests(digests, digest_stride);
  if (st == MLAQP_OK) st = check_list(seqs, n, "seqs");
  if (st == MLAQP_OK) st = check_list(new_tokens, n, "new_tokens");
  if (st != MLAQP_OK) return st;
  if (max_new < 1) return bad_arg("max_new must be >= 1");
  if (n == 0) return MLAQP_OK;
  const Range d = digest_span(digests, digest_stride, num_pages);
  const Range ins[5] = {cache_span(p.cache), table_span(block_table, block_table_stride, num_seqs, num_pages),
                        span(seq_lens, 4ull * num_seqs), span(seqs, 4ull * n), span(new_tokens, 4ull * n)};
  for (const Range& r : ins)
    if (overlaps(d, r)) return bad_arg("digests overlap an input");
  int sms = 0;
  st = step_device(-1, kDigestGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.digests = static_cast<uint8_t*>(digests);
  p.digest_stride = digest_stride;
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.num_seqs = num_seqs;
  p.seq_lens = seq_lens;
  p.seqs = seqs;
  p.new_tokens = new_tokens;
  p.n = n;
  p.max_new = max_new;
  return launched(mlaqp::kv4_digest(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t mlaqp_kv4_select_workspace(int B, int q_len, int64_t block_table_stride, int num_pages) {
  if (check_select_sizes(B, q_len) != MLAQP_OK) return -1;
  if (block_table_stride < 1 || block_table_stride > (1ll << 31) || num_pages < 1 || num_pages > MLAQP_KV4_MAX_PAGES) {
    bad_arg("block_table_stride must be in 1..2^31 and num_pages in 1..2^20");
    return -1;
  }
  return (4 * static_cast<int64_t>(B) * q_len * key_width(block_table_stride, num_pages) + 15) / 16 * 16;
}

int mlaqp_kv4_select(const void* q, int64_t q_token_stride, int q_dtype, const void* digests, int64_t digest_stride,
                     int num_pages, int page_size, const int32_t* block_table, int64_t block_table_stride, int num_seqs,
                     const int32_t* seq_lens, const int32_t* seqs, int B, int q_len, int H, int k, int first, int last,
                     int32_t* sel_table, int64_t sel_stride, int32_t* sel_lens, void* workspace,
                     int64_t workspace_bytes, mlaqp_stream_t stream) {
  mlaqp::Kv4SelectParams p = {};
  if (q_dtype != MLAQP_OUT_BF16 && q_dtype != MLAQP_OUT_E4M3) return bad_arg("unknown q_dtype");
  const bool e4m3 = q_dtype == MLAQP_OUT_E4M3;
  if (H < 1 || H > MLAQP_KV4_MAX_HEADS) return host_fail(MLAQP_ERR_UNSUPPORTED, "num_heads must be in 1..16");
  int st = check_select_sizes(B, q_len);
  if (st == MLAQP_OK) st = check_pool(num_pages, page_size);
  if (st == MLAQP_OK) st = check_digests(digests, digest_stride);
  if (st != MLAQP_OK) return st;
  if (k < 1 || first < 0 || last < 1 || static_cast<int64_t>(first) + last > k)
    return bad_arg("k >= 1, first >= 0, last >= 1 and first + last <= k are required");
  if (k > MLAQP_KV4_MAX_PAGES) return host_fail(MLAQP_ERR_UNSUPPORTED, "k must be <= 2^20");
  if (sel_stride < k || sel_stride > (1ll << 31)) return bad_arg("sel_stride must be in k..2^31");
  if (B == 0) return MLAQP_OK;
  st = check_sequences(block_table, block_table_stride, num_seqs, seq_lens);
  if (st != MLAQP_OK) return st;
  if (!q || !sel_table || !sel_lens) return bad_arg("q, sel_table and sel_lens are required");
  if (!aligned(q, 16)) return bad_arg("q must be 16-byte aligned");
  if (!aligned(seqs, 4) || !aligned(sel_table, 4) || !aligned(sel_lens, 4))
    return bad_arg("seqs, sel_table and sel_lens must be 4-byte aligned");
  const int eb = e4m3 ? 1 : 2;
  if (q_token_stride < 576ll * H || (q_token_stride * eb) % 16 != 0)
    return bad_arg("q_token_stride must be >= 576*H elements and a multiple of 16 bytes");
  if (!seqs && num_seqs < B) return bad_arg("num_seqs must be >= B where seqs is NULL");
  if (!workspace || !aligned(workspace, 16)) return bad_arg("workspace must be a 16-byte aligned buffer");
  if (workspace_bytes < mlaqp_kv4_select_workspace(B, q_len, block_table_stride, num_pages))
    return bad_arg("workspace is smaller than mlaqp_kv4_select_workspace()");
  const uint64_t M = static_cast<uint64_t>(B) * q_len;
  const Range outs[3] = {span(sel_table, 4 * ((M - 1) * static_cast<uint64_t>(sel_stride) + k)), span(sel_lens, 4 * M),
                         span(workspace, static_cast<uint64_t>(workspace_bytes))};
  const Range ins[5] = {span(q, eb * ((M - 1) * static_cast<uint64_t>(q_token_stride) + 576ull * H)),
                        digest_span(digests, digest_stride, num_pages),
                        table_span(block_table, block_table_stride, num_seqs, num_pages), span(seq_lens, 4ull * num_seqs),
                        span(seqs, seqs ? 4ull * B : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : ins)
      if (overlaps(outs[i], r)) return bad_arg("sel_table, sel_lens or workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return bad_arg("sel_table, sel_lens and workspace overlap");
  }
  int sms = 0;
  st = step_device(-1, kSelectGroup, &sms);
  if (st != MLAQP_OK) return st;
  p.q = static_cast<const uint8_t*>(q);
  p.q_ts = q_token_stride;
  p.digests = static_cast<const uint8_t*>(digests);
  p.digest_stride = digest_stride;
  p.num_pages = num_pages;
  p.shift = page_shift(page_size);
  p.block_table = block_table;
  p.table_stride = block_table_stride;
  p.num_seqs = num_seqs;
  p.seq_lens = seq_lens;
  p.seqs = seqs;
  p.B = B;
  p.q_len = q_len;
  p.H = H;
  p.k = k;
  p.first = first;
  p.last = last;
  p.table = sel_table;
  p.sel_stride = sel_stride;
  p.lens = sel_lens;
  p.keys = static_cast<uint32_t*>(workspace);
  p.width = key_width(block_table_stride, num_pages);
  return launched(mlaqp::kv4_select(p, e4m3, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int mlaqp_kv4_step_prewarm(int device) {
  int sms = 0, st = MLAQP_OK;
  for (int g = 0; g < kGroups && st == MLAQP_OK; ++g) st = step_device(device, static_cast<Group>(g), &sms);
  return st;
}

}  // extern "C"

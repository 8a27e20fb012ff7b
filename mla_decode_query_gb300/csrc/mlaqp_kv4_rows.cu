// Writing tokens into the 4-bit latent cache and reading them back.
//
// Append, per block of 32 latents: s = the smallest scale byte with
// amax <= 7 * 2^(s-127), codes = rne_e2m1(value * 2^(127-s)).  7 is the
// midpoint between the top code 6 and the 8 that E2M1 lacks, so saturating
// there still rounds to nearest.  Gather: value = code * 2^(s-127), exact in
// BF16.  Both move 1152 + 400 bytes a token and are bound by memory, or by
// the latency of slot -> row where there are few tokens.  A lane takes words
// lane and lane + 32 of a token (eight latents, 16 BF16 bytes, each), so that
// every access of a warp is one contiguous piece of 128 or 512 bytes; with
// two neighbouring words a lane, its 16-byte accesses 32 bytes apart, the
// gather of 65536 tokens took 20.0 us instead of 17.8 (5.7 TB/s of 6.8).
// That gather has two tokens a warp in flight: one or four take 2 us more.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

namespace {

constexpr int kRowsThreads = 256;
constexpr int kGatherTokens = 2;

// Byte of this lane's k-th word (eight latents) among a token's codes: word
// lane + 32k, blocks with bit 2 set having their halves swapped.
__device__ __forceinline__ uint32_t rows_word(int k) {
  const uint32_t lane = threadIdx.x & 31;
  return 128 * k + 4 * (lane ^ ((lane >> 3) & 2));
}

__global__ void __launch_bounds__(kRowsThreads) mlaqp_kv4_append_kernel(const __grid_constant__ Kv4RowsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int slot = p.slots[t];
  if (slot < 0) return;
  const int page = slot >> p.cache.shift;
  if (page >= p.cache.num_pages) {
    if (lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    return;
  }
  const uint32_t pos = slot & ((1 << p.cache.shift) - 1);
  uint8_t* base = p.cache.base + page * p.cache.page_stride;
  const uint16_t* src = p.latent + t * p.latent_ts + 8 * lane;
  const uint4 v[2] = {ld_u128(src), ld_u128(src + 256)};
  uint4 pe = make_uint4(0, 0, 0, 0);
  if (lane < 8) pe = ld_u128(p.k_pe + t * p.k_pe_ts + 8 * lane);

#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    uint32_t amax = 0;  // BF16 bits of the largest magnitude; NaN bits lie above those of infinity
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // a block is four lanes
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool bad = amax >= 0x7F80u;
    // exponent - 2, one more when the significand exceeds 1.75 = 7/4
    const int e = static_cast<int>((amax + 0x1Fu) >> 7) - 2;
    const int s = min(max(e, kKv4ScaleMin), kKv4ScaleMax);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - s) << 23);
    float a[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = bf16_lo(w[i]) * inv;
      a[2 * i + 1] = bf16_hi(w[i]) * inv;
    }
    *reinterpret_cast<uint32_t*>(base + kv4_code_off(pos) + rows_word(k)) = bad ? 0u : kv4_word(a);
    if ((lane & 3) == 0)
      base[kv4_scale_off(pos, p.cache.shift) + 8 * k + (lane >> 2)] = static_cast<uint8_t>(bad ? kKv4ScaleNan : s);
  }
  if (lane < 8) st_u128(base + kv4_rope_off(pos, p.cache.shift) + 16 * (lane ^ (pos & 7)), pe);
}

__global__ void __launch_bounds__(kRowsThreads) mlaqp_kv4_gather_kernel(const __grid_constant__ Kv4RowsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t0 = (blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5)) * kGatherTokens;
  uint32_t codes[kGatherTokens][2], scale[kGatherTokens][2];
  uint4 pe[kGatherTokens];
#pragma unroll
  for (int n = 0; n < kGatherTokens; ++n) {
    const int slot = t0 + n < p.T ? p.slots[t0 + n] : -1;
    const int page = slot >> p.cache.shift;
    const bool ok = slot >= 0 && page < p.cache.num_pages;
    if (slot >= 0 && !ok && lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    pe[n] = make_uint4(0, 0, 0, 0);
    codes[n][0] = codes[n][1] = scale[n][0] = scale[n][1] = 0;
    if (ok) {
      const uint32_t pos = slot & ((1 << p.cache.shift) - 1);
      const uint8_t* base = p.cache.base + page * p.cache.page_stride;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        codes[n][k] = *reinterpret_cast<const uint32_t*>(base + kv4_code_off(pos) + rows_word(k));
        scale[n][k] = base[kv4_scale_off(pos, p.cache.shift) + 8 * k + (lane >> 2)];
      }
      if (lane < 8) pe[n] = ld_u128(base + kv4_rope_off(pos, p.cache.shift) + 16 * (lane ^ (pos & 7)));
    }
  }
#pragma unroll
  for (int n = 0; n < kGatherTokens; ++n) {
    if (t0 + n >= p.T) return;
    uint16_t* dst = p.out + (t0 + n) * p.out_ts;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t o[4];
      kv4_word_bf16(codes[n][k], o);
      const uint32_t s = kv4_scale_bf16x2(scale[n][k]);
      st_u128(dst + 256 * k + 8 * lane,
              make_uint4(mul_bf16x2(o[0], s), mul_bf16x2(o[1], s), mul_bf16x2(o[2], s), mul_bf16x2(o[3], s)));
    }
    if (lane < 8) st_u128(dst + kLatent + 8 * lane, pe[n]);
  }
}

// CTAs for T tokens, `each` of them to a warp.
unsigned rows_grid(int T, int each) {
  const unsigned n = kRowsThreads / 32 * each;
  return (static_cast<unsigned>(T) + n - 1) / n;
}

}  // namespace

cudaError_t kv4_append(const Kv4RowsParams& p, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4RowsParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_append_kernel), rows_grid(p.T, 1), kRowsThreads, 0, stream,
                    args);
}

cudaError_t kv4_gather(const Kv4RowsParams& p, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4RowsParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_gather_kernel), rows_grid(p.T, kGatherTokens), kRowsThreads,
                    0, stream, args);
}

cudaError_t kv4_rows_setup() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_append_kernel));
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_gather_kernel));
  return e;
}

cudaError_t device_status_kv4_rows(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

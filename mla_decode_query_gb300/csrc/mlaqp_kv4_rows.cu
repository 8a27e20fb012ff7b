// Writing tokens into the 4-bit latent cache and reading them back.
//
// Append, per block of 32 latents: s = the smallest scale byte with
// amax <= 7 * 2^(s-127), codes = rne_e2m1(value * 2^(127-s)).  7 is the
// midpoint between the top code 6 and the 8 that E2M1 lacks, so saturating
// there still rounds to nearest.  Gather: value = code * 2^(s-127), exact in
// BF16.  Both move 1152 + 400 bytes a token and are bound by memory; a warp
// takes one token, a lane 16 latents (32 BF16 bytes, 8 code bytes), so that
// each of the three rows is one contiguous access of the warp.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

namespace {

constexpr int kRowsThreads = 256;

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
  const uint16_t* src = p.latent + t * p.latent_ts + 16 * lane;
  const uint4 v0 = ld_u128(src);
  const uint4 v1 = ld_u128(src + 8);
  uint4 pe = make_uint4(0, 0, 0, 0);
  if (lane < 8) pe = ld_u128(p.k_pe + t * p.k_pe_ts + 8 * lane);

  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t amax = 0;  // BF16 bits of the largest magnitude; NaN bits lie above those of infinity
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // a block is two lanes
  const bool bad = amax >= 0x7F80u;
  // exponent - 2, one more when the significand exceeds 1.75 = 7/4
  const int e = static_cast<int>((amax + 0x1Fu) >> 7) - 2;
  const int s = min(max(e, kKv4ScaleMin), kKv4ScaleMax);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - s) << 23);
  float a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] = bf16_lo(w[i]) * inv;
    a[2 * i + 1] = bf16_hi(w[i]) * inv;
    b[2 * i] = bf16_lo(w[4 + i]) * inv;
    b[2 * i + 1] = bf16_hi(w[4 + i]) * inv;
  }
  uint2 codes = make_uint2(kv4_word(a), kv4_word(b));
  if (bad) codes = make_uint2(0u, 0u);
  const int j = lane >> 1, half = lane & 1;
  *reinterpret_cast<uint2*>(base + kv4_code_off(pos) + 16 * j + 8 * (half ^ ((j >> 2) & 1))) = codes;
  if (half == 0) base[kv4_scale_off(pos, p.cache.shift) + j] = static_cast<uint8_t>(bad ? kKv4ScaleNan : s);
  if (lane < 8) st_u128(base + kv4_rope_off(pos, p.cache.shift) + 16 * (lane ^ (pos & 7)), pe);
}

__global__ void __launch_bounds__(kRowsThreads) mlaqp_kv4_gather_kernel(const __grid_constant__ Kv4RowsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int slot = p.slots[t];
  const int page = slot >> p.cache.shift;
  const bool ok = slot >= 0 && page < p.cache.num_pages;
  if (slot >= 0 && !ok && lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  uint4 pe = make_uint4(0, 0, 0, 0);
  if (ok) {
    const uint32_t pos = slot & ((1 << p.cache.shift) - 1);
    const uint8_t* base = p.cache.base + page * p.cache.page_stride;
    const int j = lane >> 1, half = lane & 1;
    const uint2 codes =
        *reinterpret_cast<const uint2*>(base + kv4_code_off(pos) + 16 * j + 8 * (half ^ ((j >> 2) & 1)));
    const uint32_t s = kv4_scale_bf16x2(base[kv4_scale_off(pos, p.cache.shift) + j]);
    if (lane < 8) pe = ld_u128(base + kv4_rope_off(pos, p.cache.shift) + 16 * (lane ^ (pos & 7)));
    uint32_t a[4], b[4];
    kv4_word_bf16(codes.x, a);
    kv4_word_bf16(codes.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = mul_bf16x2(a[i], s);
      o[4 + i] = mul_bf16x2(b[i], s);
    }
  }
  uint16_t* dst = p.out + t * p.out_ts;
  st_u128(dst + 16 * lane, make_uint4(o[0], o[1], o[2], o[3]));
  st_u128(dst + 16 * lane + 8, make_uint4(o[4], o[5], o[6], o[7]));
  if (lane < 8) st_u128(dst + kLatent + 8 * lane, pe);
}

unsigned rows_grid(int T) { return (static_cast<unsigned>(T) + kRowsThreads / 32 - 1) / (kRowsThreads / 32); }

}  // namespace

cudaError_t kv4_append(const Kv4RowsParams& p, int, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4RowsParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_append_kernel), rows_grid(p.T), kRowsThreads, 0, stream,
                    args);
}

cudaError_t kv4_gather(const Kv4RowsParams& p, int, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4RowsParams*>(&p)};
  return kv4_launch(reinterpret_cast<const void*>(&mlaqp_kv4_gather_kernel), rows_grid(p.T), kRowsThreads, 0, stream,
                    args);
}

cudaError_t kv4_rows_setup() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_append_kernel));
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&mlaqp_kv4_gather_kernel));
  return e;
}

cudaError_t device_status_kv4_rows(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

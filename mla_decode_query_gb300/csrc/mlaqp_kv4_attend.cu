// MLA decode attention over the paged 4-bit latent cache: the plain kernel.
// One CTA takes one query token with all its heads and walks the sequence in
// tiles of 32 tokens, decoded to FP32 in shared memory, with the running
// maximum and sum of the softmax.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

namespace {

constexpr int kAttendThreads = 256;
constexpr int kAttendTile = 32;
constexpr int kKeyStride = kOutDim + 1;

struct AttendSmem {
  float q[16][kOutDim];
  float k[kAttendTile][kKeyStride];
  float p[16][kAttendTile];
  float alpha[16], top[16], sum[16];
  uint8_t valid[kAttendTile];
};

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  const uint32_t two = e4m3x2_to_bf16x2_scaled(c);
  if ((c & 0x7F) == 0x7F) return __uint_as_float(0x7FC00000u);
  return bf16_lo(two) * 0x1p120f;
}

template <bool E4M3>
__global__ void __launch_bounds__(kAttendThreads) mlaqp_kv4_attend_kernel(const __grid_constant__ Kv4AttendParams p) {
  extern __shared__ uint8_t raw[];
  AttendSmem& s = *reinterpret_cast<AttendSmem*>(raw);
  pdl_launch_dependents();
  pdl_wait();
  const int m = blockIdx.x, b = m / p.q_len, i = m % p.q_len;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = p.seqs ? p.seqs[b] : b;
  int64_t n = 0;
  if (seq >= 0 && seq < p.num_seqs) {
    n = p.seq_lens[seq];
    if (n < 0 || n > p.table_stride << p.cache.shift) {
      if (tid == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
      n = 0;
    }
  } else if (tid == 0) {
    atomicOr(&g_device_status, kDevStatusBadIndex);
  }
  n -= p.q_len - 1 - i;
  const float qs = E4M3 ? *p.q_scale : 1.f;
  for (int e = tid; e < p.H * kOutDim; e += kAttendThreads) {
    const int64_t at = m * p.q_ts + e;
    float v;
    if constexpr (E4M3) v = e4m3_value(p.q[at]) * qs;
    else v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.q)[at]) << 16);
    s.q[e / kOutDim][e % kOutDim] = v;
  }
  if (tid < 16) {
    s.top[tid] = -INFINITY;
    s.sum[tid] = 0.f;
  }
  float acc[2][16];
  for (int h = 0; h < 16; ++h) acc[0][h] = acc[1][h] = 0.f;
  const int32_t* table = p.block_table + seq * p.table_stride;
  for (int64_t t0 = 0; t0 < n; t0 += kAttendTile) {
    __syncthreads();
    for (int k = warp; k < kAttendTile; k += kAttendThreads / 32) {
      const int64_t t = t0 + k;
      const int page = t < n ? table[t >> p.cache.shift] : -1;
      const bool ok = t < n && page >= 0 && page < p.cache.num_pages;
      if (t < n && !ok && lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
      if (lane == 0) s.valid[k] = ok;
      float* key = s.k[k];
      if (ok) {
        const uint32_t pos = t & ((1 << p.cache.shift) - 1);
        const uint8_t* base = p.cache.base + page * p.cache.page_stride;
        const int j = lane >> 1, half = lane & 1;
        const uint2 codes =
            *reinterpret_cast<const uint2*>(base + kv4_code_off(pos) + 16 * j + 8 * (half ^ ((j >> 2) & 1)));
        const uint32_t sc = kv4_scale_bf16x2(base[kv4_scale_off(pos, p.cache.shift) + j]);
        uint32_t a[4], c[4];
        kv4_word_bf16(codes.x, a);
        kv4_word_bf16(codes.y, c);
        for (int e = 0; e < 4; ++e) {
          a[e] = mul_bf16x2(a[e], sc);
          c[e] = mul_bf16x2(c[e], sc);
          key[16 * lane + 2 * e] = bf16_lo(a[e]);
          key[16 * lane + 2 * e + 1] = bf16_hi(a[e]);
          key[16 * lane + 8 + 2 * e] = bf16_lo(c[e]);
          key[16 * lane + 8 + 2 * e + 1] = bf16_hi(c[e]);
        }
        const uint32_t r = ld_u32(base + kv4_rope_off(pos, p.cache.shift) + 16 * ((lane >> 2) ^ (pos & 7)) + 4 * (lane & 3));
        key[kLatent + 2 * lane] = bf16_lo(r);
        key[kLatent + 2 * lane + 1] = bf16_hi(r);
      } else {
        for (int e = lane; e < kOutDim; e += 32) key[e] = 0.f;
      }
    }
    __syncthreads();
    for (int e = tid; e < p.H * kAttendTile; e += kAttendThreads) {
      const int h = e / kAttendTile, k = e % kAttendTile;
      float d = 0.f;
      for (int c = 0; c < kOutDim; ++c) d += s.q[h][c] * s.k[k][c];
      s.p[h][k] = s.valid[k] ? d * p.softmax_scale : -INFINITY;
    }
    __syncthreads();
    for (int h = warp; h < p.H; h += kAttendThreads / 32) {
      const float v = s.p[h][lane];
      float top = v;
      bool nan = v != v;
      float sum;
      for (int d = 16; d; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      }
      nan = __any_sync(0xffffffffu, nan);
      const float old = s.top[h];
      top = nan ? __uint_as_float(0x7FC00000u) : fmaxf(old, top);
      if (old != old) top = old;
      const float ref = top == -INFINITY ? 0.f : top;
      const float e = expf(v - ref);
      sum = e;
      for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      s.p[h][lane] = e;
      __syncwarp();
      if (lane == 0) {
        const float alpha = expf(old - ref);
        s.alpha[h] = alpha;
        s.sum[h] = s.sum[h] * alpha + sum;
        s.top[h] = top;
      }
    }
    __syncthreads();
    for (int h = 0; h < p.H; ++h) {
      float a0 = acc[0][h] * s.alpha[h], a1 = acc[1][h] * s.alpha[h];
      for (int k = 0; k < kAttendTile; ++k) {
        a0 += s.p[h][k] * s.k[k][tid];
        a1 += s.p[h][k] * s.k[k][tid + 256];
      }
      acc[0][h] = a0;
      acc[1][h] = a1;
    }
  }
  __syncthreads();
  for (int h = 0; h < p.H; ++h) {
    const float sum = s.sum[h];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* x = p.x + m * p.x_ts + h * kLatent;
    x[tid] = static_cast<uint16_t>(pack_bf16x2(0.f, acc[0][h] * inv));
    x[tid + 256] = static_cast<uint16_t>(pack_bf16x2(0.f, acc[1][h] * inv));
    if (tid == 0 && p.lse) p.lse[m * p.H + h] = sum == 0.f ? -INFINITY : s.top[h] + logf(sum);
  }
}

}  // namespace

cudaError_t kv4_attend(const Kv4AttendParams& p, bool q_e4m3, int, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4AttendParams*>(&p)};
  const void* fn = q_e4m3 ? reinterpret_cast<const void*>(&mlaqp_kv4_attend_kernel<true>)
                          : reinterpret_cast<const void*>(&mlaqp_kv4_attend_kernel<false>);
  return kv4_launch(fn, static_cast<unsigned>(p.B * p.q_len), kAttendThreads, sizeof(AttendSmem), stream, args);
}

cudaError_t kv4_attend_setup() {
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&mlaqp_kv4_attend_kernel<true>),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AttendSmem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&mlaqp_kv4_attend_kernel<false>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AttendSmem));
  return e;
}

int64_t kv4_attend_workspace(int, int, int, int) { return 16; }

cudaError_t device_status_kv4_attend(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

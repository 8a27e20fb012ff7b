// Writing tokens into the 4-bit latent cache with what comes before it: the
// latents' root-mean-square norm, and the rotation of the key parts and of the
// queries' parts by the tokens' positions.
//
// A token is a warp's.  Its latents are lane's words of eight (lane and
// lane + 32, as in the plain append), normalised in registers and quantised
// from FP32: y = (x * r) * w, r = 1/sqrt(ms + eps).  The squares are
// summed in two floats (a square of a BF16 is exact in FP32, and two-sum keeps
// what an addition rounds off), so r is the number that an exact sum would
// give but for ties to 2^-45: codes at a border do not depend on the order of
// a reduction.  That costs 7 operations a latent (4 operations, with a sum that
// begins at a power of two: 18.2 us instead of 18.5 below, but rows end at 2^63
// instead of the end of FP32; no norm at all: 16.1).
//
// Rotation: pair (a, b) -> (a cos - b sin, b cos + a sin).  A lane keeps the
// angles of its pairs for all heads: of four pairs in one 16-byte chunk
// (interleaved), or of eight pairs in chunks c and c + 4 (halves).
//
// What bounds it.  16385 tokens with 16 heads: 18.5 us (halves 19.0), 97 MB at 5.2
// TB/s, 77% of a copy's rate: memory, and a start and an end of some 4 us beside it
// (3.4 rounds of CTAs; 65536 tokens take 59.2 us, 6.5 TB/s; 0.67 instructions issued
// a cycle).  With 32 heads 32.0 us (halves 29.3) of 24.1 at a copy's rate, with 128
// 116 (93.5) of 83.2: from head 17 on a lane has one head in flight, of which halves
// are two chunks.  1027 tokens with 11 heads 2.5 us, 64 tokens 2.4: the chain launch
// -> position, slot -> angles -> stores.  Four tokens a CTA: eight or sixteen took
// 19.3 and 21.3 us, and 64 tokens 2.7.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

namespace {

constexpr int kRopeThreads = 128;

// Sum of `hi` and what `lo` holds beyond its last bit.
struct TwoFloat {
  float hi, lo;
};
__device__ __forceinline__ TwoFloat two_add(TwoFloat s, float v) {
  const float t = __fadd_rn(s.hi, v);
  const float b = __fadd_rn(t, -s.hi);
  const float err = __fadd_rn(__fadd_rn(s.hi, -__fadd_rn(t, -b)), __fadd_rn(v, -b));
  return TwoFloat{t, __fadd_rn(s.lo, err)};
}

// r of a token, x its latents of this lane.
__device__ __forceinline__ float rope_norm(const uint4 (&v)[2], float eps) {
  TwoFloat s = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = two_add(s, __fmul_rn(bf16_lo(w[i]), bf16_lo(w[i])));
      s = two_add(s, __fmul_rn(bf16_hi(w[i]), bf16_hi(w[i])));
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, s.hi, d), lo = __shfl_xor_sync(0xffffffffu, s.lo, d);
    // the same on both sides: two_add's error is exact, so the order of its operands does not matter
    s = two_add(TwoFloat{s.hi, __fadd_rn(s.lo, lo)}, hi);
  }
  // (an overflow leaves infinities of both signs or NaN in lo)
  const float sum = isfinite(s.hi) ? __fadd_rn(s.hi, s.lo) : s.hi;
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.f / kLatent), eps)));
}

// Angles of a lane's pairs: Pairs cosines and sines.
template <int Pairs>
struct Angles {
  float cos[Pairs], sin[Pairs];
};
template <int Pairs>
__device__ __forceinline__ void load_angles(Angles<Pairs>& a, const float* row, int c) {
#pragma unroll
  for (int i = 0; i < Pairs; i += 4) {
    const uint4 x = ld_u128(row + Pairs * c + i), y = ld_u128(row + 32 + Pairs * c + i);
    a.cos[i] = __uint_as_float(x.x), a.cos[i + 1] = __uint_as_float(x.y);
    a.cos[i + 2] = __uint_as_float(x.z), a.cos[i + 3] = __uint_as_float(x.w);
    a.sin[i] = __uint_as_float(y.x), a.sin[i + 1] = __uint_as_float(y.y);
    a.sin[i + 2] = __uint_as_float(y.z), a.sin[i + 3] = __uint_as_float(y.w);
  }
}

// One head's chunk c (interleaved) or chunks c and c + 4 (halves).
template <bool Halves>
struct RopeChunk {
  uint4 v[Halves ? 2 : 1];

  __device__ __forceinline__ void load(const uint16_t* row, int c) {
    v[0] = ld_u128(row + 8 * c);
    if constexpr (Halves) v[1] = ld_u128(row + 8 * (c + 4));
  }
  __device__ __forceinline__ void rotate(const Angles<Halves ? 8 : 4>& t) {
    if constexpr (Halves) {
      uint32_t* a = reinterpret_cast<uint32_t*>(&v[0]);
      uint32_t* b = reinterpret_cast<uint32_t*>(&v[1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = bf16_lo(a[i]), a1 = bf16_hi(a[i]), b0 = bf16_lo(b[i]), b1 = bf16_hi(b[i]);
        const float c0 = t.cos[2 * i], c1 = t.cos[2 * i + 1], s0 = t.sin[2 * i], s1 = t.sin[2 * i + 1];
        a[i] = pack_bf16x2(a1 * c1 - b1 * s1, a0 * c0 - b0 * s0);
        b[i] = pack_bf16x2(b1 * c1 + a1 * s1, b0 * c0 + a0 * s0);
      }
    } else {
      uint32_t* w = reinterpret_cast<uint32_t*>(&v[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = bf16_lo(w[i]), b = bf16_hi(w[i]);
        w[i] = pack_bf16x2(b * t.cos[i] + a * t.sin[i], a * t.cos[i] - b * t.sin[i]);
      }
    }
  }
};

template <bool Halves>
__global__ void __launch_bounds__(kRopeThreads) mlaqp_kv4_append_rope_kernel(const __grid_constant__ Kv4RopeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int Chunks = Halves ? 4 : 8;  // lanes of a head
  constexpr int Heads = 32 / Chunks;      // heads of a pass
  constexpr int Pairs = 32 / Chunks;
  constexpr int Passes = 16 / Heads;      // in flight
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const int pos = p.positions[t], slot = p.slots[t];
  const int c = lane % Chunks, h0 = lane / Chunks;

  // what does not wait for the position
  const uint16_t* src = p.latent + t * p.latent_ts + 8 * lane;
  const uint4 v[2] = {ld_u128(src), ld_u128(src + 256)};
  RopeChunk<Halves> key = {};
  if (h0 == 0) key.load(p.k_pe + t * p.k_pe_ts, c);
  const uint16_t* q = p.q + t * p.q_ts;
  RopeChunk<Halves> part[Passes] = {};
#pragma unroll
  for (int i = 0; i < Passes; ++i)
    if (h0 + Heads * i < p.H) part[i].load(q + (h0 + Heads * i) * p.q_hs, c);

  if (pos < 0 || pos >= p.num_positions) {
    if (pos >= 0 && lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    return;
  }
  Angles<Pairs> turn;
  load_angles(turn, p.cos_sin + static_cast<int64_t>(pos) * kRope, c);

  const int page = slot >> p.cache.shift;
  if (slot >= 0 && page >= p.cache.num_pages && lane == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
  if (slot >= 0 && page < p.cache.num_pages) {
    const uint32_t at = slot & ((1 << p.cache.shift) - 1);
    uint8_t* base = p.cache.base + page * p.cache.page_stride;
    const bool normed = p.norm_weight != nullptr;
    const float r = normed ? rope_norm(v, p.eps) : 1.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16_lo(w[i]);
        y[2 * i + 1] = bf16_hi(w[i]);
      }
      if (normed) {
        const uint4 g = ld_u128(p.norm_weight + 256 * k + 8 * lane);
        const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = __fmul_rn(__fmul_rn(y[2 * i], r), bf16_lo(gw[i]));
          y[2 * i + 1] = __fmul_rn(__fmul_rn(y[2 * i + 1], r), bf16_hi(gw[i]));
        }
      }
      kv4_put_word(base, at, p.cache.shift, k, y);
    }
    if (h0 == 0) {
      key.rotate(turn);
      uint8_t* row = base + kv4_rope_off(at, p.cache.shift);
      st_u128(row + 16 * (c ^ (at & 7)), key.v[0]);
      if constexpr (Halves) st_u128(row + 16 * ((c + 4) ^ (at & 7)), key.v[1]);
    }
  }

  uint16_t* out = p.q_out + t * p.q_out_ts;
  auto put = [&](RopeChunk<Halves>& x, int h) {
    x.rotate(turn);
    st_u128(out + h * p.q_out_hs + 8 * c, x.v[0]);
    if constexpr (Halves) st_u128(out + h * p.q_out_hs + 8 * (c + 4), x.v[1]);
  };
#pragma unroll
  for (int i = 0; i < Passes; ++i)
    if (h0 + Heads * i < p.H) put(part[i], h0 + Heads * i);
#pragma unroll 1
  for (int h = h0 + 16; h < p.H; h += Heads) {
    part[0].load(q + h * p.q_hs, c);
    put(part[0], h);
  }
}

const void* rope_kernel(bool halves) {
  return halves ? reinterpret_cast<const void*>(&mlaqp_kv4_append_rope_kernel<true>)
                : reinterpret_cast<const void*>(&mlaqp_kv4_append_rope_kernel<false>);
}

}  // namespace

cudaError_t kv4_append_rope(const Kv4RopeParams& p, bool halves, cudaStream_t stream) {
  void* args[1] = {const_cast<Kv4RopeParams*>(&p)};
  const unsigned tokens = kRopeThreads / 32;
  return kv4_launch(rope_kernel(halves), (static_cast<unsigned>(p.T) + tokens - 1) / tokens, kRopeThreads, 0, stream,
                    args);
}

cudaError_t kv4_rope_setup() {
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, rope_kernel(false));
  return e == cudaSuccess ? cudaFuncGetAttributes(&a, rope_kernel(true)) : e;
}

cudaError_t device_status_kv4_rope(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

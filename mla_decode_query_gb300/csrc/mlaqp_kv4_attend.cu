// The attention kernel of the 4-bit latent cache, its join kernel and their
// launch.  The mathematics and the layout are in mlaqp_kv4_attend.cuh.

#include <cuda_fp16.h>

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4_attend.cuh"

namespace mlaqp {

namespace {

__device__ __forceinline__ uint32_t att_clock() {
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}

// What a wait may take; 0 once one has run out, and all others give up too.
__device__ __forceinline__ volatile uint32_t& att_limit(AttSchedule& s) {
  return *reinterpret_cast<volatile uint32_t*>(&s.wait_ns);
}

// Bounded wait of one thread.  (Kept short: it is inlined some thirty times,
// and a larger kernel than the instruction caches hold runs at half the speed.
// So the host's word is set once, at the kernel's end.)
__device__ __forceinline__ bool att_wait_one(uint32_t bar, uint32_t parity, AttSchedule& s) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = att_clock();
#pragma unroll 1
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (att_clock() - t0 < att_limit(s));
  att_limit(s) = 0;
  return false;
}

// The wait for what is in flight once a wait has run out: does not end with the
// others, only with its own limit.
__device__ __forceinline__ void att_settle(uint32_t bar, uint32_t parity, uint32_t t0, uint32_t limit) {
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (att_clock() - t0 >= limit) return;
  }
}

// The same for a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool att_wait(uint32_t bar, uint32_t parity, AttSchedule& s) {
  return __all_sync(0xffffffffu, att_wait_one(bar, parity, s));
}

// The row groups of the CTA's stretch in order.
struct AttItem {
  int v;      // row group
  int first;  // its first tile here
  int count;  // tiles here
  int next;   // place on the line behind it: of a row group's first tile, or the stretch's end
};

// The one that holds the tile at place t, v or one behind it.
__device__ __forceinline__ AttItem att_item(const int* prefix, int v, int t, int end) {
  while (prefix[v + 1] <= t) ++v;
  AttItem it;
  it.v = v;
  it.first = t - prefix[v];
  const int last = prefix[v + 1] - kAttEndTiles;
  it.count = min(last, end) - t;
  it.next = end < last ? end : prefix[v + 1];
  return it;
}

// Tiles of the stretch.
__device__ __forceinline__ int att_tiles(const AttSchedule& s, int t, int end) {
  int n = 0;
#pragma unroll 1
  for (int v = s.group; t < end;) {
    const AttItem it = att_item(s.prefix, v, t, end);
    n += it.count;
    v = it.v;
    t = it.next;
  }
  return n;
}

// Position in a ring of N buffers and the parity of its barriers' phase.
template <int N>
struct AttRing {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      parity ^= 1;
    }
  }
};

// --------------------------------------------------------------------------
// Warp 16: pages into shared memory.
// --------------------------------------------------------------------------
template <int R, bool E4>
__device__ __forceinline__ void att_load(const Kv4AttendParams& p, typename AttPlan<R, E4>::Shared& s, uint32_t smem, uint32_t bars,
                                         int t0, int t1) {
  using L = AttPlan<R, E4>;
  const int lane = threadIdx.x & 31;
  const int shift = p.cache.shift;
  const int entries = kAttTile >> shift;  // pages of a tile
  const int groups = (p.q_len * p.H + R - 1) / R;
  const uint8_t* const cache = p.cache.base;
  const int64_t page_stride = p.cache.page_stride;
  const int num_pages = p.cache.num_pages;

  // A unit lies in one page or in several whole ones (parts).  Lane 2e copies
  // the codes of its part e, lane 2e+1 the scales, all with one instruction;
  // what a lane copies differs from unit to unit by constants only.
  constexpr int kLog = L::Unit == 64 ? 6 : 5;
  const int log_parts = max(kLog - shift, 0);
  const int parts = 1 << log_parts;
  const bool scales = lane & 1;
  const int part = min(lane >> 1, parts - 1);
  const bool copies = lane >> 1 < parts;
  const uint32_t row_bytes = scales ? kKv4Blocks : kKv4CodeBytes;
  const uint32_t bytes = row_bytes * (L::Unit >> log_parts);
  const uint32_t plane = scales ? kv4_scale_off(0, shift) : 0u;
  const uint32_t to = smem + L::Raw + part * bytes + (scales ? L::UnitCodes : 0);
  const uint32_t unit_tx = (kKv4CodeBytes + kKv4Blocks) * L::Unit >> log_parts;
  const uint32_t page_mask = (1u << shift) - 1u;
  const uint32_t rope_plane = kv4_rope_off(0, shift), rope_bytes = kKv4RopeBytes << shift;
  const unsigned tile_pages = (1u << entries) - 1u;

  // Rope rows of tile kr, a page per lane.  Their buffer comes free when the
  // tile's scores begin, the codes' when those have been fetched, so neither
  // waits behind the other: the warp polls for both.
  int k = 0, u = 0, kr = 0;
  AttRing<L::Units> ring;
  auto load_rope = [&]() {
    const int page = lane < entries ? s.pages[kr % kAttPageTiles][lane] : -1;
    const int rb = kr % L::RopeBufs;
    const uint32_t bar = bars + 8 * (L::RopeFull + rb);
    const unsigned have = __ballot_sync(0xffffffffu, page >= 0);
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * rope_bytes);
    __syncwarp();
    if (page >= 0)
      bulk_load_1d(smem + L::Rope + rb * kRopeTile + lane * rope_bytes, cache + page * page_stride + rope_plane, rope_bytes, bar);
    ++kr;
  };
  auto rope_empty = [&]() { return bars + 8 * (L::RopeEmpty + kr % L::RopeBufs); };
  auto rope_free = [&]() { return kr < L::RopeBufs || mbar_test(rope_empty(), (kr / L::RopeBufs - 1) & 1); };
  // Rope rows of all tiles up to `tile`.
  auto finish_rope = [&](int tile) -> bool {
#pragma unroll 1
    while (kr <= tile) {
      if (kr >= L::RopeBufs && !att_wait(rope_empty(), (kr / L::RopeBufs - 1) & 1, s)) return false;
      load_rope();
    }
    return true;
  };
  // The copy stage at hand is empty (or a wait ran out: false); tiles up to
  // `tile` may have their rope rows copied meanwhile.
  auto stage_free = [&]() {
    return u < L::Units || __all_sync(0xffffffffu, mbar_test(bars + 8 * (L::RawEmpty + ring.at), ring.parity ^ 1));
  };
  auto wait_stage = [&](int tile) -> bool {
    if (stage_free()) return true;
    const uint32_t t_in = att_clock();
#pragma unroll 1
    for (int i = 1;; ++i) {
      if (kr <= tile && __all_sync(0xffffffffu, rope_free())) load_rope();
      if (stage_free()) return true;
      if ((i & 63) == 0 && __any_sync(0xffffffffu, att_clock() - t_in >= att_limit(s))) {
        att_limit(s) = 0;
        return false;
      }
    }
  };
  bool ok = true;
  for (int t = t0, v = s.group; ok && t < t1;) {
    const AttItem it = att_item(s.prefix, v, t, t1);
    t = it.next;
    v = it.v;
    // Each lane holds one entry of the table row and the page's address (0:
    // no page); the entries after these are loaded long before their turn,
    // so that a tile costs this warp, alone with its latencies, little.
    const int32_t* row = p.block_table + (p.seqs ? p.seqs[it.v / groups] : it.v / groups) * p.table_stride;
    const int64_t len = s.len[it.v];
    int64_t at = (static_cast<int64_t>(it.first) << 7 >> shift) + lane;  // of the entries loaded last
    int entry = 0, raw = -1, id = -1;
    unsigned have = 0;
    uint64_t addr = 0;
    bool in = at << shift < len;
    if (in) raw = row[at];
#pragma unroll 1
    for (int n = 0; n < it.count; ++n, ++k) {
      if ((entry & 31) == 0) {
        const bool good = in && raw >= 0 && raw < num_pages;
        if (in && !good) atomicOr(&g_device_status, kDevStatusBadIndex);
        addr = good ? reinterpret_cast<uint64_t>(cache) + static_cast<uint64_t>(raw) * page_stride : 0;
        have = __ballot_sync(0xffffffffu, good);
        id = good ? raw : -1;
        at += 32;
        in = at << shift < len;
        if (in) raw = row[at];
        entry = 0;
      }
      const unsigned pages = have >> entry & tile_pages;
      ok = finish_rope(k - kAttPageTiles);
      if (!ok) break;
      if (lane >= entry && lane < entry + entries) s.pages[k % kAttPageTiles][lane - entry] = id;
      if (lane == 0) {
        // copied 16-token parts of the tile, a bit each
        uint32_t mask = 0xFFu;
        if (pages != tile_pages) {
          mask = 0;
          const int rep = 1 << (shift - 4);
#pragma unroll 1
          for (int e = 0; e < entries; ++e) mask |= (pages >> e & 1) ? ((1u << rep) - 1u) << (e * rep) : 0u;
        }
        s.tmask[k % kAttMaskTiles] = mask;
      }
      __syncwarp();
      if (__all_sync(0xffffffffu, rope_free())) load_rope();
#pragma unroll 1
      for (int q = 0; q < L::PerTile; ++q) {
        const int e = q << kLog >> shift;  // the (first) page of the unit in the tile
        const uint64_t page = __shfl_sync(0xffffffffu, addr, entry + e + part);
        const uint32_t off = plane + (static_cast<uint32_t>(q << kLog) & page_mask) * row_bytes;
        const uint32_t bar = bars + 8 * (L::RawFull + ring.at);
        ok = wait_stage(k);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(pages >> e & ((1u << parts) - 1u)) * unit_tx);
        __syncwarp();
        if (copies && page)
          bulk_load_1d(to + ring.at * L::UnitBytes, reinterpret_cast<const uint8_t*>(page + off), bytes, bar);
        ring.next();
        ++u;
      }
      if (!ok) break;
      entry += entries;
    }
  }
  if (ok) finish_rope(k - 1);
  if (lane == 0) {
    s.units = u;
    s.ropes = kr;
  }
}

// --------------------------------------------------------------------------
// Warp 19: scale bytes, one token per lane.  s_t = the largest of the 16;
// s_t - s_j, at most 31, picks the row of the E4M3 table.  Bytes are taken as
// pairs of 16-bit numbers; none of the differences borrows.
// --------------------------------------------------------------------------
template <int R, bool E4>
__device__ __forceinline__ void att_scales(typename AttPlan<R, E4>::Shared& s, uint8_t* smem, uint32_t bars, int tiles) {
  using L = AttPlan<R, E4>;
  const int lane = threadIdx.x & 31;
  AttRing<L::Units> ring;
  for (int k = 0; k < tiles; ++k) {
    const int kb = k % kAttScaleTiles;
#pragma unroll 1
    for (int q = 0; q < L::PerTile; ++q, ring.next()) {
      const int st = ring.at;
      if (!att_wait(bars + 8 * (L::RawFull + st), ring.parity, s)) return;
#pragma unroll
      for (int g = 0; g < L::Unit / 32; ++g) {
        const int tok = 32 * g + lane;
        const uint4 x =
            *reinterpret_cast<const uint4*>(smem + L::Raw + st * L::UnitBytes + L::UnitCodes + tok * kKv4Blocks);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t e[4], o[4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = w[i] & 0x00FF00FFu;
          o[i] = (w[i] >> 8) & 0x00FF00FFu;
          m = __vmaxu2(m, __vmaxu2(e[i], o[i]));
        }
        m = max(m & 0xFFFFu, m >> 16);
        const bool nan = m == kKv4ScaleNan;
        m = min(max(m, kKv4ScaleMin), kKv4ScaleMax);
        const uint32_t mm = m * 0x00010001u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the differences cannot borrow: no byte above mm
          e[i] = __vminu2(__vmaxu2(e[i], kKv4ScaleMin * 0x00010001u), mm);
          o[i] = __vminu2(__vmaxu2(o[i], kKv4ScaleMin * 0x00010001u), mm);
        }
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r[i] = __vminu2(mm - e[i], 0x001F001Fu) | (__vminu2(mm - o[i], 0x001F001Fu) << 8);
        *reinterpret_cast<uint4*>(&s.rel[(st * L::Unit + tok) * kKv4Blocks]) = make_uint4(r[0], r[1], r[2], r[3]);
        s.smax[kb][L::Unit * q + tok] = static_cast<uint8_t>(nan ? kKv4ScaleNan : m);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (L::ScaleFull + (k & 1) * L::PerTile + q));
    }
  }
}

// --------------------------------------------------------------------------
// Code warps: codes -> E4M3 tile.  A quarter of them takes a block of 128
// latents of the tile, a warp WarpTokens of its tokens, a thread a block of 32
// latents of every eighth token.  So the output product gives the tile back,
// and the score product takes it, block by block, and a warp still has one
// wait, one fence and one arrival a tile.  (All warps on one block after the
// other spent 900 cycles a block, mostly there.)
// --------------------------------------------------------------------------
template <int R, bool E4>
__device__ __forceinline__ void att_dequant(typename AttPlan<R, E4>::Shared& s, uint8_t* smem, uint32_t bars, int tiles) {
  using L = AttPlan<R, E4>;
  constexpr int N = L::WarpTokens / 8;                                      // tokens of a thread
  constexpr int Parts = L::WarpTokens > L::Unit ? L::WarpTokens / L::Unit : 1;  // copy units of a warp
  constexpr int Each = N / Parts;
  const int lane = threadIdx.x & 31, dw = (threadIdx.x >> 5) - kAttSoftWarps;
  const int blk = dw / (kAttDequantWarps / 4), jj = lane & 3;  // 128 latents, 32 of them
  const int row = L::WarpTokens * (dw % (kAttDequantWarps / 4)) + (lane >> 2);
  const int unit = row / L::Unit, tok = row % L::Unit;         // its (first) copy unit in the tile, token there
  // The two 16-byte chunks' places: the order of a block's halves alternates
  // with the 128 latents.  Eight rows on, the swizzle is the same.
  const uint32_t half = blk & 1;
  const uint32_t at0 = blk * kK8Block + row * 128 + (((2 * jj + half) ^ (row & 7)) << 4);
  const uint32_t at1 = blk * kK8Block + row * 128 + (((2 * jj + (half ^ 1)) ^ (row & 7)) << 4);
  const uint32_t raw0 = L::Raw + tok * kKv4CodeBytes + 64 * blk + 16 * jj, rel0 = tok * kKv4Blocks + 4 * blk + jj;
  int st = unit % L::Units;  // every PerTile-th copy unit is the warp's
#pragma unroll 1
  for (int k = 0; k < tiles; ++k) {
    const int b = k & 1;
    uint8_t* tile = smem + L::K8 + b * kK8Tile;
    uint4 w[N];
    uint32_t rel[N];
#pragma unroll
    for (int c = 0; c < Parts; ++c) {
      // The scale warp has seen the copies land.  (Its barriers go by the
      // unit's place in two tiles: a stage's own barrier would pass phases
      // that this warp does not wait for.)
      if (!att_wait(bars + 8 * (L::ScaleFull + b * L::PerTile + unit + c), (k >> 1) & 1, s)) return;
      const uint8_t* raw = smem + raw0 + st * L::UnitBytes;
#pragma unroll
      for (int i = 0; i < Each; ++i) {
        rel[c * Each + i] = s.rel[st * L::Unit * kKv4Blocks + rel0 + 8 * i * kKv4Blocks];
        w[c * Each + i] = *reinterpret_cast<const uint4*>(raw + 8 * i * kKv4CodeBytes);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + 8 * (L::RawEmpty + st));
      st = (st + (c + 1 < Parts ? 1 : L::PerTile - Parts + 1)) % L::Units;
    }
    // the block of the tile two before has been multiplied
    if (k >= 2 && !att_wait(bars + 8 * (L::K8Empty + 4 * b + blk), (k / 2 - 1) & 1, s)) return;
#pragma unroll
    for (int i0 = 0; i0 < N; i0 += 4) {
      uint2 lut[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) lut[i] = *reinterpret_cast<const uint2*>(s.lut[rel[i0 + i]]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        auto word = [&](uint32_t c, uint32_t& lo, uint32_t& hi) {
          const uint32_t m = c & 0x77777777u;
          lo = prmt(lut[i].x, lut[i].y, m) | (c & 0x80808080u);
          hi = prmt(lut[i].x, lut[i].y, m >> 16) | ((c * 16u) & 0x80808080u);
        };
        uint4 a, c;
        word(w[i0 + i].x, a.x, a.y);
        word(w[i0 + i].y, a.z, a.w);
        word(w[i0 + i].z, c.x, c.y);
        word(w[i0 + i].w, c.z, c.w);
        *reinterpret_cast<uint4*>(tile + at0 + (i0 + i) * 1024) = a;
        *reinterpret_cast<uint4*>(tile + at1 + (i0 + i) * 1024) = c;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8 * (L::K8Full + 4 * b + blk));
  }
}

// --------------------------------------------------------------------------
// Warps 17 and 18 issue the MMAs of the scores and of the output.  Two warps,
// because each product has to go as soon as its operands are there: from one
// thread in program order, the output product that frees a K8 tile waited
// behind the scores of the next one.  The whole warp goes through the loop and
// one lane issues, so that descriptors are computed once a warp: a lone
// thread's MMAs came 175 cycles apart.
// --------------------------------------------------------------------------

template <int R, bool E4>
__device__ __forceinline__ void att_mma_scores(typename AttPlan<R, E4>::Shared& s, uint32_t smem, uint32_t bars,
                                               uint32_t tmem, int t0, int t1) {
  using L = AttPlan<R, E4>;
  constexpr uint32_t id_s = att_idesc(kAttTile, L::NQ, kFmtE4M3, kFmtE4M3, false, false);
  constexpr uint32_t id_r = att_idesc(kAttTile, R, kFmtBf16, kFmtBf16, false, false);
  const bool leader = elect_one();
  // operands 32 bytes apart along the contraction, blocks of 128 latents behind each other
  const uint64_t a_k8 = smem_desc_sw128(smem + L::K8, 16, 1024), b_q = smem_desc_sw128(smem + L::Q, 16, 1024);
  const uint64_t a_rope = smem_desc_sw128(smem + L::Rope, 16, 1024), b_pe = smem_desc_sw128(smem + L::QPe, 16, 1024);
  bool ok = true;
  int k = 0, item = 0;
  for (int t = t0, v = s.group; ok && t < t1; ++item) {
    const AttItem it = att_item(s.prefix, v, t, t1);
    t = it.next;
    v = it.v;
    ok = att_wait(bars + 8 * L::QFull, item & 1, s);
#pragma unroll 1
    for (int n = 0; ok && n < it.count; ++n, ++k) {
      const int b = k & 1, sb = k % L::SBufs, rb = k % L::RopeBufs;
      if (k >= L::SBufs) ok = att_wait(bars + 8 * (L::SEmpty + sb), (k / L::SBufs - 1) & 1, s);
      if (!ok) break;
      const uint32_t d = tmem + sb * L::SCols;
      ok = att_wait(bars + 8 * (L::RopeFull + rb), (k / L::RopeBufs) & 1, s);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          umma_bf16(d + L::NQ, a_rope + rb * (kRopeTile >> 4) + 2 * c, b_pe + 2 * c, id_r, c > 0);
        umma_commit(bars + 8 * (L::RopeEmpty + rb));
      }
      const uint64_t a_tile = a_k8 + static_cast<uint64_t>(b * (kK8Tile >> 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ok) ok = att_wait(bars + 8 * (L::K8Full + 4 * b + i), (k / 2) & 1, s);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            umma_f8(d, a_tile + i * (kK8Block >> 4) + 2 * c, b_q + i * (L::QBlock >> 4) + 2 * c, id_s, i + c > 0);
        }
      }
      if (!ok) break;
      if (leader) umma_commit(bars + 8 * (L::SFull + sb));
      __syncwarp();
    }
  }
}

template <int R, bool E4>
__device__ __forceinline__ void att_mma_output(typename AttPlan<R, E4>::Shared& s, uint32_t smem, uint32_t bars,
                                               uint32_t tmem, int t0, int t1) {
  using L = AttPlan<R, E4>;
  constexpr uint32_t id_o = att_idesc(kAttTile, L::NP, kFmtE4M3, kFmtE5M2, true, true);
  const bool leader = elect_one();
  // A: 128 latents, 32 tokens (8-token groups 1024 bytes apart) 4096 on;
  // B: 16-row chunks PChunk apart (SBO), 8-token groups 128 apart (LBO)
  const uint64_t a_k8 = smem_desc_sw128(smem + L::K8, 16, 1024);
  const uint64_t b_p = smem_desc_plain(smem + L::P, 128, L::PChunk);
  bool ok = true;
  int k = 0, item = 0;
  for (int t = t0, v = s.group; ok && t < t1; ++item) {
    const AttItem it = att_item(s.prefix, v, t, t1);
    t = it.next;
    v = it.v;
    if (item > 0) ok = att_wait(bars + 8 * L::OEmpty, (item - 1) & 1, s);
#pragma unroll 1
    for (int n = 0; ok && n < it.count; ++n, ++k) {
      ok = att_wait(bars + 8 * L::PFull, k & 1, s);
      if (!ok) break;
      tc_fence_after();
      const uint64_t a_tile = a_k8 + static_cast<uint64_t>((k & 1) * (kK8Tile >> 4));
      if (leader) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int ks = 0; ks < kAttTile / 32; ++ks)
            umma_f8(tmem + L::OCol + mt * L::NP, a_tile + mt * (kK8Block >> 4) + ks * (4096 >> 4),
                    b_p + ks * (512 >> 4), id_o, (n == 0 && ks == 0) ? 0u : 1u);
          umma_commit(bars + 8 * (L::K8Empty + 4 * (k & 1) + mt));
        }
        umma_commit(bars + 8 * L::PvDone);
      }
      __syncwarp();
    }
  }
}

// What copies and products a CTA in which a wait has run out has in flight
// lands before it gives its shared and tensor memory back, whichever warp gave
// up: the ones that copy and issue may have had nothing to wait for.  (Where
// none ran out the waits have seen all of it land: O is read behind the last
// product.  Done by the warps at the end of their roles in any case, this cost
// 32 sequences of up to 8191 tokens 0.5 us.)
template <int R, bool E4>
__device__ __forceinline__ void att_land(typename AttPlan<R, E4>::Shared& s, uint32_t bars, uint32_t limit) {
  using L = AttPlan<R, E4>;
  const int warp = threadIdx.x >> 5;
  const uint32_t at = att_clock();
  if (warp == kAttLoadWarp) {
    const int u = s.units, kr = s.ropes;
#pragma unroll 1
    for (int i = max(0, u - L::Units); i < u; ++i)
      att_settle(bars + 8 * (L::RawFull + i % L::Units), (i / L::Units) & 1, at, limit);
#pragma unroll 1
    for (int i = max(0, kr - L::RopeBufs); i < kr; ++i)
      att_settle(bars + 8 * (L::RopeFull + i % L::RopeBufs), (i / L::RopeBufs) & 1, at, limit);
  } else if (warp == kAttScoreWarp || warp == kAttOutputWarp) {
    const uint32_t bar = bars + 8 * (L::Drain + (warp == kAttOutputWarp ? 1 : 0));
    if (elect_one()) umma_commit(bar);  // the lane that issued: the same at every call
    att_settle(bar, 0, at, limit);
  }
}

// --------------------------------------------------------------------------
// Warps 0-7
// --------------------------------------------------------------------------

// Queries of row group v into shared memory, and what its rows need (turn:
// which of the two copies).
template <int R, bool E4>
__device__ __forceinline__ void att_query(const Kv4AttendParams& p, typename AttPlan<R, E4>::Shared& s, uint8_t* smem, uint32_t bars, int v,
                                          int turn) {
  using L = AttPlan<R, E4>;
  constexpr int TPR = 128 / L::HalfRows;  // threads per row; each group of four warps sees to its own rows
  const int tid = threadIdx.x;
  const int r = tid / TPR, sub = tid % TPR;
  const int rows = p.q_len * p.H;
  const int groups = (rows + R - 1) / R;
  const int b = v / groups, rr = (v % groups) * R + r;
  const bool real = rr < rows;
  const int i = real ? rr / p.H : 0, h = real ? rr % p.H : 0;
  const int64_t m = static_cast<int64_t>(b) * p.q_len + i;
  const int64_t at = m * p.q_ts + h * kOutDim;
  uint8_t* q8 = smem + L::Q;
  float cr = p.softmax_scale * 1.4426950408889634f;
  if constexpr (E4) {
    const uint8_t* src = p.q + at;
#pragma unroll 1
    for (int c = sub; c < 36; c += TPR) {  // 16-byte chunks: 32 of latents, 4 of rope
      uint4 x = make_uint4(0, 0, 0, 0);
      if (real) x = ld_u128(src + 16 * c);
      if (c < 32) {
        *reinterpret_cast<uint4*>(q8 + (c >> 3) * L::QBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = x;
      } else {  // rope codes -> BF16, exact
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t o[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const uint32_t two = w[2 * e + (f >> 1)] >> (16 * (f & 1));
            o[f] = mul_bf16x2(e4m3x2_to_bf16x2_scaled(two), 0x7B807B80u);  // 2^120
            if ((two & 0x7Fu) == 0x7Fu) o[f] |= 0x7FC0u;
            if ((two & 0x7F00u) == 0x7F00u) o[f] |= 0x7FC00000u;
          }
          const int ch = 2 * (c - 32) + e;
          *reinterpret_cast<uint4*>(smem + L::QPe + r * 128 + ((ch ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    cr *= *p.q_scale;
  } else {
    constexpr int N = 64 / TPR;  // chunks of eight latents of a thread
    const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + at;
    uint4 x[N], pe = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = real ? ld_u128(src + 8 * (n * TPR + sub)) : make_uint4(0, 0, 0, 0);
    if (real && sub < 8) pe = ld_u128(src + kLatent + 8 * sub);  // TPR >= 8: one chunk of rope at most
    auto top = [](uint4 a) {
      const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu), __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu));
      return max(m & 0xFFFFu, m >> 16);
    };
    uint32_t ml = 0, mp = top(pe);
#pragma unroll
    for (int n = 0; n < N; ++n) ml = max(ml, top(x[n]));
#pragma unroll
    for (int d = 1; d < TPR; d <<= 1) {
      ml = max(ml, __shfl_xor_sync(0xffffffffu, ml, d));
      mp = max(mp, __shfl_xor_sync(0xffffffffu, mp, d));
    }
    // exponent of the row: its latents' largest, but not so far below the
    // rope part's that scaling that part would overflow
    const int e = max(max(static_cast<int>(ml >> 7), static_cast<int>(mp >> 7) - 40), 8);
    const bool bad = ml >= 0x7F80u || mp >= 0x7F80u;  // NaN or infinity: the whole row
    const float f = bad ? __uint_as_float(0x7FC00000u) : exp2f(static_cast<float>(134 - e));
    cr *= exp2f(static_cast<float>(e - 134));
#pragma unroll
    for (int n = 0; n < N; ++n) {  // elements 8c..8c+7: half of 16-byte E4M3 chunk c/2
      const int c = n * TPR + sub;
      const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a = bf16_lo(w[q]) * f, c1 = bf16_hi(w[q]) * f;
        const uint32_t t8 = pack_e4m3x2(c1, a);
        // the code back as a float: bits * 2^-120 in BF16, exact
        const uint32_t back = mul_bf16x2(e4m3x2_to_bf16x2_scaled(t8), 0x7B807B80u);
        const uint32_t l8 = pack_e4m3x2((c1 - bf16_hi(back)) * 16.f, (a - bf16_lo(back)) * 16.f);
        hi[q >> 1] |= t8 << (16 * (q & 1));
        lo[q >> 1] |= l8 << (16 * (q & 1));
      }
      uint8_t* to = q8 + (c >> 4) * L::QBlock + ((((c >> 1) & 7) ^ (r & 7)) << 4) + 8 * (c & 1);
      *reinterpret_cast<uint2*>(to + r * 128) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(to + (R + r) * 128) = make_uint2(lo[0], lo[1]);
    }
    if (sub < 8) {
      const uint32_t w[4] = {pe.x, pe.y, pe.z, pe.w};
      uint32_t o[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) o[g] = pack_bf16x2(bf16_hi(w[g]) * f, bf16_lo(w[g]) * f);
      *reinterpret_cast<uint4*>(smem + L::QPe + r * 128 + ((sub ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (sub == 0) {
    s.cr[turn][r] = real ? cr : 0.f;
    s.limit[turn][r] = real ? s.len[v] - (p.q_len - 1 - i) : 0x7fffffff;
    s.xoff[turn][r] = real ? m * p.x_ts + h * kLatent : -1;
    s.lseoff[turn][r] = static_cast<int>(m) * p.H + h;
  }
  fence_proxy_async_smem();
  mbar_arrive(bars + 8 * L::QFull);
}

template <int R, bool E4>
__device__ __forceinline__ void att_softmax(const Kv4AttendParams& p, typename AttPlan<R, E4>::Shared& s, uint8_t* smem, uint32_t bars,
                                            uint32_t tmem, int t0, int t1) {
  using L = AttPlan<R, E4>;
  constexpr int HR = L::HalfRows;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = warp >> 2, tok = tid & 127;  // half of the rows, token of the tile
  const int row0 = group * HR;
  const uint32_t here = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + row0;  // first row's columns
  float* mref = s.mref[warp];
  float* alpha = s.alpha[warp];
  // A wait that runs out ends the warp's work, but not its part in the
  // barriers of its group (`gave_up`).  Nothing may go on behind such a wait:
  // tensor memory may still be a product's.
  // Row group -1 has no tiles: it only prepares the first one's queries.
  AttItem it = {s.group, 0, 0, t0};
  int k = 0, n = 0;
  int due = 0;  // barriers ahead of a warp that gave up: 0 tile n's and on, 1 the next tile's and on, 2 the next row group's
  for (int t = t0, item = -1; t < t1; ++item) {
    const int turn = item & 1;
    // every warp has left the row group before (what follows reuses its
    // places), and this one's rows are known
    soft_barrier(group);
    const int next_t = it.next;
    AttItem next = it;
    if (next_t < t1) next = att_item(s.prefix, it.v, next_t, t1);
    float top = -INFINITY;  // M of row `lane`
    float l[HR], cr[HR];
#pragma unroll
    for (int r = 0; r < HR; ++r) {
      l[r] = 0.f;
      cr[r] = s.cr[turn][row0 + r];
    }
    if (lane < HR) mref[lane] = kAttUnseen;
    __syncwarp();
    for (n = item < 0 ? -1 : 0; n < it.count; ++n) {
      const int sb = k % L::SBufs;
      if (n >= 0 && !att_wait(bars + 8 * (L::SFull + sb), (k / L::SBufs) & 1, s)) goto gave_up;
      // the scores of the row group's last tile are in: its queries are done with
      if (n == it.count - 1 && next_t < t1) att_query<R, E4>(p, s, smem, bars, next.v, turn ^ 1);
      if (n < 0) continue;
      tc_fence_after();
      // the scores, in flight while the scales are looked at
      uint32_t v[(L::QTerms + 1) * HR];
#pragma unroll
      for (int part = 0; part <= L::QTerms; ++part)
        tmem_ld_begin<HR>(here + sb * L::SCols + part * R, &v[HR * part]);
      if (!att_wait(bars + 8 * (L::K8Full + 4 * (k & 1)), (k / 2) & 1, s)) goto gave_up;  // the tile's scales are in, too
      const uint32_t sm = s.smax[k % kAttScaleTiles][tok];
      const float ts = sm == kKv4ScaleNan ? __uint_as_float(0x7FC00000u) : __uint_as_float((sm - 6u) << 23);
      const float its = __uint_as_float((260u - sm) << 23);
      const float et = static_cast<float>(static_cast<int>(sm) - 133);
      const int64_t tile_tok = static_cast<int64_t>(it.first + n) * kAttTile;
      const uint32_t mask = s.tmask[k % kAttMaskTiles];
      const bool whole = mask == 0xFFu && tile_tok + kAttTile <= s.limit[turn][row0];
      float y[HR];
      tmem_ld_end(v);
#pragma unroll
      for (int r = 0; r < HR; ++r) {
        float d = __uint_as_float(v[r]);
        if constexpr (!E4) d = fmaf(__uint_as_float(v[HR + r]), 0.0625f, d);  // the second query term
        y[r] = fmaf(fmaf(d, ts, __uint_as_float(v[HR * L::QTerms + r])), cr[r], et);
      }
      tc_fence_before();
      mbar_arrive(bars + 8 * (L::SEmpty + sb));
      if (!whole) {
        const bool copied = mask >> (tok >> 4) & 1;
#pragma unroll
        for (int r = 0; r < HR; ++r)
          if (!copied || tile_tok + tok >= s.limit[turn][row0 + r]) y[r] = -INFINITY;
      }
      // Has any row outgrown its reference?  Mostly not: then one barrier
      // tells, and no maximum is taken.
      float x[HR], high = -INFINITY;
#pragma unroll
      for (int r = 0; r < HR; r += 4) {
        const float4 m = *reinterpret_cast<const float4*>(&mref[r]);
        x[r] = y[r] - m.x;
        x[r + 1] = y[r + 1] - m.y;
        x[r + 2] = y[r + 2] - m.z;
        x[r + 3] = y[r + 3] - m.w;
        high = fmaxf(fmaxf(high, fmaxf(x[r], x[r + 1])), fmaxf(x[r + 2], x[r + 3]));
      }
      if (soft_barrier_any(group, high > kAttShift + kAttSlack || n == 0)) {
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          const float4 m = make_float4(warp_max(y[r]), warp_max(y[r + 1]), warp_max(y[r + 2]), warp_max(y[r + 3]));
          if (lane == 0) *reinterpret_cast<float4*>(&s.wmax[warp][r]) = m;
        }
        soft_barrier(group);
        if (lane < HR) {
          const float(*wm)[HR] = &s.wmax[4 * group];
          const float tm = fmaxf(fmaxf(wm[0][lane], wm[1][lane]), fmaxf(wm[2][lane], wm[3][lane]));
          const bool up = tm > top;
          alpha[lane] = up ? (top == -INFINITY ? 0.f : ex2(top - tm)) : 1.f;
          if (up) {
            top = tm;
            mref[lane] = tm - kAttShift;
          }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          const float4 a = *reinterpret_cast<const float4*>(&alpha[r]);
          const float4 m = *reinterpret_cast<const float4*>(&mref[r]);
          l[r] *= a.x;
          l[r + 1] *= a.y;
          l[r + 2] *= a.z;
          l[r + 3] *= a.w;
          x[r] = y[r] - m.x;
          x[r + 1] = y[r + 1] - m.y;
          x[r + 2] = y[r + 2] - m.z;
          x[r + 3] = y[r + 3] - m.w;
        }
        if (n > 0) {
          due = 1;
          if (!att_wait(bars + 8 * L::PvDone, (k - 1) & 1, s)) goto gave_up;
          due = 0;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 12; ++c) {  // four blocks of latents, three terms
            const uint32_t at = here + L::OCol + c * R;
            uint32_t o[HR];
            tmem_ld_begin<HR>(at, o);
            tmem_ld_end(o);
#pragma unroll
            for (int r = 0; r < HR; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * alpha[r]);
            tmem_st<HR>(at, o);
          }
          tmem_wait_st();
        }
      }
      due = 1;
      if (k > 0 && !att_wait(bars + 8 * L::PvDone, (k - 1) & 1, s)) goto gave_up;  // P is free
      due = 0;
      uint32_t terms[3][HR / 4];
#pragma unroll
      for (int r = 0; r < HR; r += 4) {
        const float e0 = ex2(x[r]), e1 = ex2(x[r + 1]), e2 = ex2(x[r + 2]), e3 = ex2(x[r + 3]);
        l[r] = fmaf(e0, its, l[r]);
        l[r + 1] = fmaf(e1, its, l[r + 1]);
        l[r + 2] = fmaf(e2, its, l[r + 2]);
        l[r + 3] = fmaf(e3, its, l[r + 3]);
        // three E5M2 terms: the top bytes of FP16, rounded, are E5M2 and the
        // differences exact.  Rounding to nearest leaves at most half a step,
        // so three terms of 3 bits hold FP16's 11 (truncated, they held 9:
        // up to 2^-9.2 off).  A NaN may round to zero here: it is in l.
        __half2 a = __floats2half2_rn(e0, e1), c = __floats2half2_rn(e2, e3);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const uint32_t au = *reinterpret_cast<uint32_t*>(&a) + 0x00800080u;
          const uint32_t cu = *reinterpret_cast<uint32_t*>(&c) + 0x00800080u;
          terms[q][r / 4] = prmt(au, cu, 0x7531u);
          if (q < 2) {
            uint32_t ah = au & 0xFF00FF00u, ch = cu & 0xFF00FF00u;
            a = __hsub2(a, *reinterpret_cast<__half2*>(&ah));
            c = __hsub2(c, *reinterpret_cast<__half2*>(&ch));
          }
        }
      }
      // 16 rows of a token lie side by side: half of that, or one of two
      uint8_t* ps = smem + L::P + tok * 16 + (HR == 8 ? group * 8 : group * L::PChunk);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint8_t* to = ps + q * (R / 16) * L::PChunk;
        if constexpr (HR == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(terms[q][0], terms[q][1]);
        else
          *reinterpret_cast<uint4*>(to) = make_uint4(terms[q][0], terms[q][1], terms[q][HR / 4 - 2], terms[q][HR / 4 - 1]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bars + 8 * L::PFull);
      ++k;
    }
    if (item < 0) {
      it = next;
      continue;
    }

    // The row group's end here: sums over the tokens, O from tensor memory.
    const int tiles = s.prefix[it.v + 1] - s.prefix[it.v] - kAttEndTiles;
    const bool complete = it.count == tiles;
    float mine = 0.f;
#pragma unroll
    for (int r = 0; r < HR; ++r) {
      float v = l[r];
#pragma unroll
      for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
      if (lane == r) mine = v;
    }
    soft_barrier(group);  // the maxima of the last tile have been read
    if (lane < HR) s.wmax[warp][lane] = mine;
    soft_barrier(group);
    // (one answer for all lanes: another warp may give up at this moment)
    due = 2;
    if (!att_wait(bars + 8 * L::PvDone, (k - 1) & 1, s) || __any_sync(0xffffffffu, att_limit(s) == 0)) goto gave_up;
    due = 0;
    tc_fence_after();
    float* part = nullptr;
    if (!complete) {
      const int slot = 2 * blockIdx.x + (s.prefix[it.v] > s.cut ? 1 : 0);  // begun here or before
      part = reinterpret_cast<float*>(p.ws + kAttGroupBytes) + slot * att_slot_floats<R>();
    }
    __syncwarp();
    if (lane < HR) {
      const float(*ws)[HR] = &s.wmax[4 * group];
      const float sum = (ws[0][lane] + ws[1][lane]) + (ws[2][lane] + ws[3][lane]);
      const float m = mref[lane];
      const int row = row0 + lane;
      const int64_t xo = s.xoff[turn][row];
      const bool first = (warp & 3) == 0;
      if (complete) {
        const bool none = sum == 0.f;  // no token, or none whose page is there (a NaN is not 0)
        alpha[lane] = none ? 0.f : 1.f / sum;
        if (first && xo >= 0 && p.lse)
          p.lse[s.lseoff[turn][row]] = none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      } else if (first) {
        part[R * kLatent + row] = top == -INFINITY ? top : m;
        part[R * kLatent + R + row] = sum;
      }
    }
    __syncwarp();
#pragma unroll 1
    for (int mt = 0; mt < 4; ++mt) {
      const int col = mt * 128 + 32 * (warp & 3) + lane;
      uint32_t v[3 * HR];
      const uint32_t d = here + L::OCol + mt * L::NP;
#pragma unroll
      for (int q = 0; q < 3; ++q) tmem_ld_begin<HR>(d + q * R, &v[q * HR]);
      tmem_ld_end(v);
      float o[HR];
#pragma unroll
      for (int r = 0; r < HR; ++r)
        o[r] = __uint_as_float(v[r]) + (__uint_as_float(v[HR + r]) + __uint_as_float(v[2 * HR + r]));
      if (!complete) {
#pragma unroll
        for (int r = 0; r < HR; ++r) part[(row0 + r) * kLatent + col] = o[r];
      } else {
        // two rows at a time: even lanes take the first row's two latents, odd lanes the second's
#pragma unroll
        for (int r = 0; r < HR; r += 2) {
          const float a = o[r] * alpha[r], c = o[r + 1] * alpha[r + 1];
          const bool odd = lane & 1;
          const float got = __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
          const int64_t xo = s.xoff[turn][row0 + r + (odd ? 1 : 0)];
          const uint32_t two = odd ? pack_bf16x2(c, got) : pack_bf16x2(got, a);
          if (xo >= 0) *reinterpret_cast<uint32_t*>(p.x + xo + (col & ~1)) = two;
        }
      }
    }
    tc_fence_before();
    mbar_arrive(bars + 8 * L::OEmpty);
    t = next_t;
    it = next;
  }
  return;

gave_up:
  tmem_wait_ld();  // the scores' loads
  if (due == 0 && soft_barrier_any(group, false)) soft_barrier(group);
  for (;;) {
    if (due < 2) {
#pragma unroll 1
      for (++n; n < it.count; ++n)
        if (soft_barrier_any(group, false)) soft_barrier(group);
      soft_barrier(group);
      soft_barrier(group);
    }
    if (it.next >= t1) return;
    it = att_item(s.prefix, it.v, it.next, t1);
    n = -1;
    due = 1;
    soft_barrier(group);
  }
}

// Rows of the groups that see no token.
template <int R>
__device__ __forceinline__ void att_empty_rows(const Kv4AttendParams& p, const AttSchedule& s, int V) {
  const int rows = p.q_len * p.H;
  const int groups = (rows + R - 1) / R;
  for (int v = blockIdx.x; v < V; v += gridDim.x) {
    if (s.prefix[v + 1] != s.prefix[v]) continue;
    const int r0 = (v % groups) * R, n = min(R, rows - r0);
    for (int e = threadIdx.x; e < n * 64; e += 32 * kAttSoftWarps) {
      const int rr = r0 + e / 64;
      const int64_t m = static_cast<int64_t>(v / groups) * p.q_len + rr / p.H;
      st_u128(p.x + m * p.x_ts + (rr % p.H) * kLatent + 8 * (e % 64), make_uint4(0, 0, 0, 0));
      if (e % 64 == 0 && p.lse) p.lse[m * p.H + rr % p.H] = -INFINITY;
    }
  }
}

// What the join kernel needs of the row groups, 32 groups a CTA: here, where a
// warp has nothing to do yet, it costs nothing; in the join kernel, in every
// CTA, the lengths' latency and these quotients were 2 us.
__device__ __forceinline__ void att_groups(const Kv4AttendParams& p, const AttSchedule& s, int V) {
  for (int v = 32 * blockIdx.x + (threadIdx.x & 31); v < V; v += 32 * gridDim.x) {
    AttGroup g = {0, 0};
    if (s.prefix[v] < s.prefix[v + 1]) {
      const AttCut cut(s.prefix[V], gridDim.x);
      const int c = cut.owner(s.prefix[V], s.prefix[v]);
      g.slot = 2 * c + (s.prefix[v] > cut.begin(c) ? 1 : 0);
      g.pieces = cut.owner(s.prefix[V], s.prefix[v + 1] - kAttEndTiles - 1) - c + 1;
    }
    reinterpret_cast<AttGroup*>(p.ws)[v] = g;
  }
}

template <int R, bool E4>
__global__ void __launch_bounds__(kAttThreads, 1) mlaqp_kv4_attend_kernel(const __grid_constant__ Kv4AttendParams p) {
  using L = AttPlan<R, E4>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // The MMA tiles need a 1024-byte boundary.  Dynamic shared memory begins on
  // one where a kernel has no other (it does, behind the first KB of the
  // window, on sm_103), and there is no room to round up.
  uint8_t* smem = smem_raw;
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(&g_device_status, kDevStatusWaitTimeout);
    return;
  }
  typename L::Shared& s = *reinterpret_cast<typename L::Shared*>(smem + L::Misc);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t bars = smem_u32(s.bars);
  if (tid < L::BarCount) {
    uint32_t count = 1;
    if (tid >= L::RawEmpty && tid < L::ScaleFull) count = L::UnitWarps;
    if (tid >= L::K8Full && tid < L::K8Empty) count = kAttDequantWarps / 4;
    if ((tid >= L::SEmpty && tid <= L::PFull) || tid == L::QFull || tid == L::OEmpty) count = 32 * kAttSoftWarps;
    if (tid - p.held_first < p.held_count) ++count;  // (none outside the test of the waits)
    mbar_init(bars + 8 * tid, count);
    fence_barrier_init();
  }
  if (tid < 32) {
    // row k: the magnitudes times 2^(6-k) as E4M3, exact up to k = 14
    const float f = __uint_as_float(static_cast<uint32_t>(133 - tid) << 23);
    s.lut[tid][0] = pack_e4m3x2(0.5f * f, 0.f) | (pack_e4m3x2(1.5f * f, f) << 16);
    s.lut[tid][1] = pack_e4m3x2(3.f * f, 2.f * f) | (pack_e4m3x2(6.f * f, 4.f * f) << 16);
    if (tid == 0) {
      s.wait_ns = p.wait_ns;
      s.units = s.ropes = 0;
    }
  }
  pdl_wait();
  if (warp == kAttScoreWarp) tmem_alloc(smem_u32(&s.tmem), 512);
  const int V = att_schedule(p, R, s, blockIdx.x == 0);
  if (warp < kAttMaxSeqs / 32) {
    // once for all warps: five of them share a scheduler
    const AttCut cut(s.prefix[V], gridDim.x);
    const bool mine = s.prefix[V] > 0 && static_cast<int>(blockIdx.x) < cut.n;
    const int t0 = mine ? cut.begin(blockIdx.x) : 0;
    if (tid < V && s.prefix[tid] <= t0 && t0 < s.prefix[tid + 1]) {
      s.group = tid;
      s.begin = t0 < s.prefix[tid + 1] - kAttEndTiles ? t0 : s.prefix[tid + 1];
    }
    if (tid == 0) {
      s.cut = t0;
      s.end = mine ? cut.begin(blockIdx.x + 1) : 0;
      if (!mine) s.begin = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s.tmem);
  const int t0 = s.begin, t1 = s.end;
  const uint32_t base = smem_u32(smem);
  // every warpgroup does this, and the shares fit what the launch has
  if (warp < kAttSoftWarps) {
    att_set_regs<L::SoftRegs>();
  } else if (warp < kAttLoadWarp) {
    att_set_regs<L::CodeRegs>();
  } else {
    att_set_regs<L::OtherRegs>();
  }
  if (warp < kAttSoftWarps) {
    att_empty_rows<R>(p, s, V);
    if (t0 < t1) att_softmax<R, E4>(p, s, smem, bars, tmem, t0, t1);
  } else if (warp == kAttScaleWarp) {
    att_groups(p, s, V);
    if (t0 < t1) att_scales<R, E4>(s, smem, bars, att_tiles(s, t0, t1));
  } else if (t0 < t1) {
    if (warp < kAttLoadWarp) {
      att_dequant<R, E4>(s, smem, bars, att_tiles(s, t0, t1));
    } else if (warp == kAttLoadWarp) {
      att_load<R, E4>(p, s, base, bars, t0, t1);
    } else if (warp == kAttScoreWarp) {
      att_mma_scores<R, E4>(s, base, bars, tmem, t0, t1);
    } else if (warp == kAttOutputWarp) {
      att_mma_output<R, E4>(s, base, bars, tmem, t0, t1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (att_limit(s) == 0) {  // the same for all: nothing sets it behind the barrier
    att_land<R, E4>(s, bars, p.wait_ns);
    tc_fence_before();
    __syncthreads();
  }
  tc_fence_after();
  __syncwarp();
  if (tid == 0 && s.wait_ns == 0) atomicOr(&g_device_status, kDevStatusWaitTimeout);
  if (warp == kAttScoreWarp) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------------------
// Join: the pieces of a row group that several CTAs worked on, in their
// order, so that the result does not depend on which CTA was first.  A job is
// a row, or 128 of its 512 latents where there are few rows; the CTA's eight
// warps take the pieces in turn.  Bound by latency: what the attention kernel
// noted of the row groups, then M, l and the first pieces' sums at once.
// Where there are more rows than a quarter of the CTAs and none has more than
// eight pieces, 128 latents of a row are a warp's job, without a barrier: 64
// sequences of up to 32768 tokens 152 -> 149 us (both kernels), 16 of up to 4100
// tokens with 4 query tokens 27.8 -> 25.1, 64 of 2048 30.5 -> 27.4, 256 of up to
// 4000 76.7 -> 70.5.  For fewer rows it took 0.4 us more, and for both kinds in a
// call as much again.  Two CTAs per SM, without that: 32 sequences of up to 8191
// tokens take 27.3 us, with one 29.0, with three 29.8, with four 32.7; 16 of up to
// 4100 tokens, 4 query tokens, 27.1, 29.9, 30.7 and 33.8; 64 of up to 32768 152,
// 156, 155 and 159.
// --------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
constexpr int kJoinCtasPerSm = 2;
constexpr int kJoinFew = 8;  // pieces that a warp joins

struct JoinShared {
  AttGroup group[kAttMaxSeqs];
  int split[kAttMaxSeqs];
  int split_warp[8];
  float m[8];
  float weight[kAttMaxCtas], l[kAttMaxCtas];  // of a piece
  float wsum[8];
  alignas(16) float part[8][kLatent];
};

// One row's pieces: their weights into j.weight, their l into j.l, and the sums
// of BL x 128 latents from `col`, by warp, into j.part and j.wsum.  The first
// pieces' sums are asked for before M and l.  Returns the largest M.
template <int R, int BL, class Slot>
__device__ __forceinline__ float join_sums(JoinShared& j, int np, int r, int col, const Slot& slot) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int U = 8 / BL;  // pieces in flight
  float4 o[U][BL];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < BL; ++b)
        if (c0 + 8 * u < np)
          o[u][b] = *reinterpret_cast<const float4*>(slot(c0 + 8 * u) + r * kLatent + col + 128 * b + 4 * lane);
  };
  float m = -INFINITY, l = 0.f;
  if (tid < np) {
    m = slot(tid)[R * kLatent + r];
    l = slot(tid)[R * kLatent + R + r];
  }
  load(warp);
  const float wm = warp_max(m);
  if (lane == 0) j.m[warp] = wm;
  __syncthreads();
  float top = j.m[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) top = fmaxf(top, j.m[w]);
  if (tid < np) {
    j.weight[tid] = m == -INFINITY ? 0.f : ex2(m - top);  // nothing summed: also where that is all pieces'
    j.l[tid] = l;
  }
  __syncthreads();
  float4 acc[BL];
#pragma unroll
  for (int b = 0; b < BL; ++b) acc[b] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int c0 = warp; c0 < np;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + 8 * u >= np) break;
      const float f = j.weight[c0 + 8 * u];
      sum = fmaf(j.l[c0 + 8 * u], f, sum);
#pragma unroll
      for (int b = 0; b < BL; ++b) {
        acc[b].x = fmaf(o[u][b].x, f, acc[b].x);
        acc[b].y = fmaf(o[u][b].y, f, acc[b].y);
        acc[b].z = fmaf(o[u][b].z, f, acc[b].z);
        acc[b].w = fmaf(o[u][b].w, f, acc[b].w);
      }
    }
    c0 += 8 * U;
    load(c0);
  }
#pragma unroll
  for (int b = 0; b < BL; ++b) *reinterpret_cast<float4*>(&j.part[warp][128 * b + 4 * lane]) = acc[b];
  if (lane == 0) j.wsum[warp] = sum;
  return top;
}

// 128 latents of a row of at most kJoinFew pieces by a warp, without a barrier: the
// same sums in the same order as above.
template <class Slot>
__device__ __forceinline__ void join_few(const Kv4AttendParams& p, int R, int np, int r, int col, int64_t q, int h,
                                         const Slot& slot) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
  if (lane < np) {
    m = slot(lane)[R * kLatent + r];
    l = slot(lane)[R * kLatent + R + r];
  }
  float4 o[kJoinFew];
#pragma unroll
  for (int c = 0; c < kJoinFew; ++c)
    if (c < np) o[c] = *reinterpret_cast<const float4*>(slot(c) + r * kLatent + col + 4 * lane);
  const float top = warp_max(m);
  const float weight = m == -INFINITY ? 0.f : ex2(m - top);
  const float part = __fmul_rn(l, weight);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kJoinFew; ++c) {
    if (c >= np) break;
    const float f = __shfl_sync(0xffffffffu, weight, c);
    sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, part, c));
    x.x = __fadd_rn(x.x, __fmul_rn(o[c].x, f)), x.y = __fadd_rn(x.y, __fmul_rn(o[c].y, f));
    x.z = __fadd_rn(x.z, __fmul_rn(o[c].z, f)), x.w = __fadd_rn(x.w, __fmul_rn(o[c].w, f));
  }
  const bool none = sum == 0.f;
  const float inv = 1.f / sum;
  *reinterpret_cast<uint2*>(p.x + q * p.x_ts + h * kLatent + col + 4 * lane) =
      none ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(x.y * inv, x.x * inv), pack_bf16x2(x.w * inv, x.z * inv));
  if (lane == 0 && col == 0 && p.lse)
    p.lse[q * p.H + h] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int R>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm)
    mlaqp_kv4_join_kernel(const __grid_constant__ Kv4AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  JoinShared& j = *reinterpret_cast<JoinShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = p.q_len * p.H, groups = (rows + R - 1) / R, V = p.B * groups;
  const int per_group = min(R, rows);
  // Neither kernel lets the one behind it start early: its CTAs would find no
  // room beside the attention's, and calls one behind the other took longer
  // (64 sequences of up to 32768 tokens 164 us instead of 159, one of 131071
  // 26.5 instead of 25.0).
  pdl_wait();
  static_assert(kJoinThreads == kAttMaxSeqs, "a thread a row group");
  AttGroup mine = {0, 0};
  if (tid < V) mine = reinterpret_cast<const AttGroup*>(p.ws)[tid];
  // (an attention kernel that gave up before it noted anything)
  if (mine.slot < 0 || mine.pieces > min(static_cast<int>(gridDim.x) / kJoinCtasPerSm, kAttMaxCtas) - (mine.slot >> 1))
    mine.pieces = 0;
  j.group[tid] = mine;
  // the row groups that more than one CTA worked on, in order, and whether any of
  // them has more pieces than a warp joins (a bit beside a warp's count: with
  // __syncthreads_or 32 sequences of up to 8191 tokens took 27.6 us instead of 27.4,
  // one of 131071 26.4 instead of 26.25)
  const bool split = mine.pieces > 1;
  const unsigned who = __ballot_sync(0xffffffffu, split);
  const bool warp_many = __any_sync(0xffffffffu, mine.pieces > kJoinFew);
  if (lane == 0) j.split_warp[warp] = __popc(who) | (warp_many ? 64 : 0);
  __syncthreads();
  int rank = __popc(who & ((1u << lane) - 1u)), n_split = 0;
  bool many = false;
  for (int w = 0; w < 8; ++w) {
    const int n = j.split_warp[w] & 63;
    if (w < warp) rank += n;
    n_split += n;
    many |= j.split_warp[w] >= 64;
  }
  if (split) j.split[rank] = tid;
  __syncthreads();
  const int cuts = n_split * per_group * 4 <= static_cast<int>(gridDim.x) ? 4 : 1;
  const float* const base = reinterpret_cast<const float*>(p.ws + kAttGroupBytes);
  if (cuts == 1 && !many) {
    const int rows4 = per_group * 4, step = static_cast<int>(gridDim.x) * (kJoinThreads / 32);
    for (int job = blockIdx.x + static_cast<int>(gridDim.x) * warp; job < n_split * rows4; job += step) {
      const int v = j.split[job / rows4], r = job / 4 % per_group, rr = (v % groups) * R + r;
      if (rr >= rows) continue;
      const int at = j.group[v].slot;
      join_few(p, R, j.group[v].pieces, r, job % 4 * 128, static_cast<int64_t>(v / groups) * p.q_len + rr / p.H, rr % p.H,
               [&](int c) { return base + (c == 0 ? at : (at & ~1) + 2 * c) * att_slot_floats<R>(); });
    }
    return;
  }
  const int jobs = n_split * per_group * cuts;
  for (int job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int v = j.split[job / (per_group * cuts)], r = job / cuts % per_group, col = job % cuts * 128;
    const int rr = (v % groups) * R + r;
    if (rr >= rows) continue;
    const int np = j.group[v].pieces, at = j.group[v].slot;
    auto slot = [&](int c) { return base + (c == 0 ? at : (at & ~1) + 2 * c) * att_slot_floats<R>(); };
    const float top = cuts == 1 ? join_sums<R, 4>(j, np, r, 0, slot) : join_sums<R, 1>(j, np, r, col, slot);
    __syncthreads();
    const int n = kLatent / cuts;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += j.wsum[w];
    const int i = rr / p.H, h = rr % p.H;
    const int64_t q = static_cast<int64_t>(v / groups) * p.q_len + i;
    const bool none = sum == 0.f;
    const float inv = 1.f / sum;
    if (2 * tid < n) {
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 a = *reinterpret_cast<const float2*>(&j.part[w][2 * tid]);
        o.x += a.x;
        o.y += a.y;
      }
      *reinterpret_cast<uint32_t*>(p.x + q * p.x_ts + h * kLatent + col + 2 * tid) =
          none ? 0u : pack_bf16x2(o.y * inv, o.x * inv);
    }
    if (tid == 0 && col == 0 && p.lse)
      p.lse[q * p.H + h] = none ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    __syncthreads();
  }
}

struct AttKernels {
  const void* main;
  const void* join;
  int smem;
  bool splits_regs;           // its warps share the launch's registers out anew
  int stage[kAttStages + 1];  // first barrier of each hand-over, and of what follows the last
};

template <int R, bool E4>
AttKernels att_kernels() {
  using L = AttPlan<R, E4>;
  return AttKernels{reinterpret_cast<const void*>(&mlaqp_kv4_attend_kernel<R, E4>),
                    reinterpret_cast<const void*>(&mlaqp_kv4_join_kernel<R>), L::Bytes, L::SoftRegs != kAttRegs,
                    {L::RawFull, L::RawEmpty, L::ScaleFull, L::RopeFull, L::RopeEmpty, L::K8Full, L::K8Empty, L::SFull,
                     L::SEmpty, L::PFull, L::PvDone, L::QFull, L::OEmpty, L::Drain}};
}

// 16 rows where all (query token, head) pairs of a sequence fit, else groups
// of 32, each reading the cache once: tensor memory holds no more (three
// terms of P, four blocks of latents, 32 rows: 384 columns, and the scores).
AttKernels att_pick(int q_len, int H, bool e4m3) {
  if (kv4_attend_rows(q_len, H) == 16) return e4m3 ? att_kernels<16, true>() : att_kernels<16, false>();
  return e4m3 ? att_kernels<32, true>() : att_kernels<32, false>();
}

}  // namespace

cudaError_t kv4_attend(const Kv4AttendParams& params, bool q_e4m3, int sm_count, cudaStream_t stream) {
  Kv4AttendParams p = params;
  const AttKernels k = att_pick(p.q_len, p.H, q_e4m3);
  const int ctas = sm_count < kAttMaxCtas ? sm_count : kAttMaxCtas;
  if (p.held > 0) {
    p.held_first = static_cast<unsigned>(k.stage[p.held - 1]);
    p.held_count = static_cast<unsigned>(k.stage[p.held] - k.stage[p.held - 1]);
  }
  void* args[1] = {&p};
  const cudaError_t e = kv4_launch(k.main, static_cast<unsigned>(ctas), kAttThreads, k.smem, stream, args);
  if (e != cudaSuccess) return e;
  return kv4_launch(k.join, static_cast<unsigned>(kJoinCtasPerSm * sm_count), kJoinThreads, sizeof(JoinShared), stream,
                    args);
}

int kv4_attend_rows(int q_len, int H) { return q_len * H <= 16 ? 16 : 32; }

cudaError_t kv4_attend_setup(int rows) {
  const AttKernels both[2] = {rows == 16 ? att_kernels<16, false>() : att_kernels<32, false>(),
                              rows == 16 ? att_kernels<16, true>() : att_kernels<32, true>()};
  for (const AttKernels& k : both) {
    cudaError_t e = cudaFuncSetAttribute(k.main, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k.main);
    // a split shares out what this many registers a thread make; with fewer it would wait for them for ever
    if (e == cudaSuccess && k.splits_regs && a.numRegs < kAttRegs) e = cudaErrorInvalidKernelImage;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k.join);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int64_t kv4_attend_workspace(int, int q_len, int H, int sm_count) {
  const int64_t slot = kv4_attend_rows(q_len, H) == 16 ? att_slot_floats<16>() : att_slot_floats<32>();
  return kAttGroupBytes + 2 * sm_count * slot * 4;
}

cudaError_t device_status_kv4_attend(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp

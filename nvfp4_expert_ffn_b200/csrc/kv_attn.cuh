// Shared parts of the attention kernels over the paged NVFP4 key/value cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Weights are 2^(score - m), held in float16, with a reference m that follows the running maximum:
// it is set kLead below a maximum, and again only when a weight passes 2^(kLead + kRaise), so that
// most tiles rescale nothing. Weights so reach up to 2^15, half of float16's largest, and a key whose
// weight is 2^-21 of the largest or more keeps all 11 bits; below that it is off by 2^-32 of the largest
// at most. (With the largest at 2^0, long contexts beside one dominant key lost their tail: it
// counted in the float32 sum, but in the products weights below 2^-25 were zero.)
constexpr float kLead = 7.0f;
constexpr float kRaise = 8.0f;
constexpr float kNoMax = -3.402823466e38f;  // no key seen yet
MOE_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The factor of scores of a head. A tensor scale of the keys (or a scale) that is infinite has infinities
// of both signs among its products, so its rows are to become NaN like those of a NaN one: see where
// it is used.
MOE_DEV float score_scale(const KvAttnArgs& a, int h) {
  return a.scale * kLog2e * (a.cache.k_ts ? a.cache.k_ts[h] : 1.0f);
}

MOE_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// two E4M3 bytes (low, high) -> f16x2, exact
MOE_DEV uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

MOE_DEV uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// mbar_wait with the limit read once per block: short in code (the roles of a block share the
// instruction caches) and without a load from global memory in every wait.
struct Patience {
  volatile int abort;
  unsigned long long limit;
};
MOE_DEV bool wait_soon(uint64_t* bar, uint32_t parity, Patience* w, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (w->abort) return false;
    if (globaltimer_ns() - t0 > w->limit) {
      w->abort = 1;
      atomicExch(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// A sequence of the batch, clamped so that no index made from it leaves its array.
struct SeqSpan {
  int q0, n_q, ctx;
};

MOE_DEV SeqSpan load_seq(const KvAttnArgs& a, int b) {
  SeqSpan s;
  const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
  s.q0 = min(max(lo, 0), a.T);
  s.n_q = max(min(hi, a.T) - s.q0, 0);
  s.ctx = (int)min((int64_t)max(a.ctx_lens[b], 0), (int64_t)a.max_pages * a.cache.page_size);
  return s;
}

// The tensor-core kernel's tiles: rows of one key head, keys, and a row tile's start and end (its
// queries in, its rows out) in key tiles: 14500 cycles of 3300 for D <= 128, 19000 of 1800 for 256.
template <int D>
struct TileShape {
  static constexpr int rows = D == 256 ? 128 : 256;
  static constexpr int kt = D == 256 ? 64 : 128;
  static constexpr int start_cost = D == 256 ? 10 : 4;
};

// Row tiles of one key head, in order; a tile's share of the work starts at `start`.
struct RowTile {
  int b, tile, n_units, pad;
  long long start;
  long long pad2;
};

// keys that the tile's last row sees
MOE_DEV int tile_keys(const KvAttnArgs& a, const SeqSpan& s, int tile, int tile_rows) {
  if (!a.causal) return s.ctx;
  const int last = min(s.n_q * a.G, (tile + 1) * tile_rows) - 1;
  return min(s.ctx, max(s.ctx - s.n_q + last / a.G + 1, 0));
}

MOE_DEV int seq_tiles(const KvAttnArgs& a, const SeqSpan& s, int tile_rows) {
  const int rows = s.n_q * a.G;
  return rows > a.dec_max_rows ? (rows + tile_rows - 1) / tile_rows : 0;
}

// Exclusive block scan of one value per thread (at most 32 warps); *total the sum.
template <int THREADS>
MOE_DEV long long plan_scan(long long v, long long* tmp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < THREADS / 32 ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < THREADS / 32) tmp[lane] = w;
  }
  __syncthreads();
  *total = tmp[THREADS / 32 - 1];
  return (warp ? tmp[warp - 1] : 0) + x - v;
}

// One block: the list of row tiles and the prefix sums of their work. A block of the kernel of few
// rows does it, beside the others' keys: a kernel of its own added 3 us to every call.
template <int THREADS, int D>
MOE_DEV void plan_tiles(const KvAttnArgs& a, long long* tmp) {
  constexpr int tile_rows = TileShape<D>::rows, kt = TileShape<D>::kt, start_cost = TileShape<D>::start_cost;
  RowTile* tiles = reinterpret_cast<RowTile*>(a.tiles);
  // 1. the tiles of every sequence, in order
  long long at = 0;
  for (int b0 = 0; b0 < a.n_seqs; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const int n = b < a.n_seqs ? seq_tiles(a, load_seq(a, b), tile_rows) : 0;
    long long sum;
    const long long first = at + plan_scan<THREADS>(n, tmp, &sum);
    for (int i = 0; i < n && first + i < a.max_tiles; ++i) {
      tiles[first + i].b = b;
      tiles[first + i].tile = i;
    }
    at += sum;
  }
  __syncthreads();  // (and with it the writes above, for this block)
  // more tiles than T rows can have: cu_q is not ascending
  if (at > a.max_tiles && threadIdx.x == 0) atomicMax(a.status, kStatusInvalid);
  const int n_tiles = (int)min(at, (long long)a.max_tiles);
  // 2. their work
  at = 0;
  for (int i0 = 0; i0 < n_tiles; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    int units = 0;
    if (i < n_tiles) {
      const SeqSpan s = load_seq(a, tiles[i].b);
      units = max(1, (tile_keys(a, s, tiles[i].tile, tile_rows) + kt - 1) / kt);
    }
    long long sum;
    const long long start = at + plan_scan<THREADS>(i < n_tiles ? units + start_cost : 0, tmp, &sum);
    if (i < n_tiles) {
      tiles[i].n_units = units;
      tiles[i].start = start;
    }
    at += sum;
  }
  if (threadIdx.x == 0) {
    a.plan[0] = at;  // work of one key head
    a.plan[1] = n_tiles;
  }
}

}  // namespace moe

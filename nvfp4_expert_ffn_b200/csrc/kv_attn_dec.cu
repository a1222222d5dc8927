// Attention of few query rows per key head over the paged NVFP4 cache (decode steps, a few
// speculative tokens): out = softmax(scale q K^T) V with K and V read as 4-bit codes.
//
// Bound by the cache's bytes: 9/16 byte per element of K and V, read once per group of 8 NR
// query rows. A byte of codes is two elements, so the work per byte is what has to be small:
// the codes go from global memory straight into the operand registers of mma.sync (m16n8k16,
// float16 in, float32 out) without passing shared memory. The tensor pipe is idle most of the
// time here (8 query columns), tcgen05 would need the expanded tiles in shared memory.
//   S^T = K Q^T: keys are the 16 rows of the A operand. The order of the head's elements
//     along k is free as long as K and Q agree, so a thread's share of a key row is one
//     contiguous quarter: 16-byte loads, and a byte of codes expands (one conversion) to one
//     f16x2 register of the fragment, times the block's scale (one multiply, exact: 2 + 4
//     significant bits).
//   O^T = V^T P^T: the A operand pairs two keys of one element, so the codes of two keys are
//     interleaved nibble by nibble first (half an instruction per element); the scores'
//     fragments turn into P^T operands with movmatrix.
// q is scaled by a power of two per row into float16's range (exact; the factor returns in
// the softmax scale), the weights P are rounded to float16 (11 bits; the result is bf16, 8),
// sums, maxima and the output stay in float32.
//
// The keys of all sequences and heads are cut into chunks of kChunk and dealt to the blocks in
// equal contiguous runs, so a batch of any shape fills the machine; a run that starts or ends
// inside a sequence leaves its partial result (row maxima, sums, unnormalised output) in the
// workspace, and a second small kernel joins them in a fixed order.
#include <cuda_bf16.h>

#include "kv_attn.cuh"

namespace moe {

namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kChunk = 64;  // keys

MOE_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

MOE_DEV uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int BYTES>
MOE_DEV void load_codes(uint32_t* dst, const uint8_t* src) {
  if constexpr (BYTES == 4) {
    dst[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (BYTES == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
    dst[0] = v.x;
    dst[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
      dst[4 * i] = v.x;
      dst[4 * i + 1] = v.y;
      dst[4 * i + 2] = v.z;
      dst[4 * i + 3] = v.w;
    }
  }
}

template <int BYTES>
MOE_DEV uint32_t load_scales(const uint8_t* src) {
  if constexpr (BYTES == 1) return __ldg(src);
  if constexpr (BYTES == 2) return __ldg(reinterpret_cast<const uint16_t*>(src));
  return __ldg(reinterpret_cast<const uint32_t*>(src));
}

// One thread's share of 16 keys: of K, rows g and g + 8, a quarter c of the head each; of V,
// keys 2c, 2c+1, 2c+8, 2c+9, an eighth g of the head each.
template <int D>
struct Tile {
  static constexpr int KW = D / 32, VW = D / 64;  // words of codes per row
  static constexpr int KS = D / 64;               // scale bytes per K row
  static constexpr int VS = D >= 128 ? D / 128 : 1;
  uint32_t k[2][KW], v[4][VW];
  uint32_t ks[2], vs[4];

  MOE_DEV void zero() {  // rows of a page number outside the cache
#pragma unroll
    for (int i = 0; i < KW; ++i) k[0][i] = k[1][i] = 0u;
#pragma unroll
    for (int i = 0; i < VW; ++i) v[0][i] = v[1][i] = v[2][i] = v[3][i] = 0u;
    ks[0] = ks[1] = vs[0] = vs[1] = vs[2] = vs[3] = 0u;
  }

  MOE_DEV void load(const KvCacheArgs& c, int64_t row0, int g, int q) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = row0 + g + 8 * i;
      load_codes<KW * 4>(k[i], c.k_codes + row * (D / 2) + q * (D / 8));
      ks[i] = load_scales<KS>(c.k_scales + row * (D / 16) + q * KS);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + 2 * q + (i & 1) + 8 * (i >> 1);
      load_codes<VW * 4>(v[i], c.v_codes + row * (D / 2) + g * (D / 16));
      vs[i] = load_scales<VS>(c.v_scales + row * (D / 16) + (D >= 128 ? g * VS : g / 2));
    }
  }
};

struct Segment {
  int b, h, rg;      // sequence, key head, group of rows
  int k0, k1, n_ch;  // chunks [k0, k1) of the item's n_ch
};

MOE_DEV int seq_chunks(const SeqSpan& s) { return max(1, (s.ctx + kChunk - 1) / kChunk); }

// Chunks of all items of a sequence; 0 for one that this kernel leaves to the other.
MOE_DEV int64_t seq_cost(const KvAttnArgs& a, const SeqSpan& s, int rows_per_group) {
  const int rows = s.n_q * a.G;
  if (rows == 0 || rows > a.dec_max_rows) return 0;
  return (int64_t)seq_chunks(s) * a.cache.Hkv * ((rows + rows_per_group - 1) / rows_per_group);
}

template <int D, int NR>
__global__ void __launch_bounds__(kDecThreads, D == 256 || NR > 1 ? 1 : 2) kv_attn_dec_kernel(const KvAttnArgs a) {
  constexpr int RB = 8 * NR;
  constexpr int KSTEPS = D / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  float* s_o = reinterpret_cast<float*>(smem_raw);  // [warps][RB][D]
  __shared__ float s_m[kDecWarps][RB], s_l[kDecWarps][RB], s_f[kDecWarps][RB];
  __shared__ float s_mm[RB], s_ll[RB];
  __shared__ long long s_scan[kDecWarps];
  __shared__ int s_b;
  __shared__ long long s_local;
  MOE_PDL_PROLOGUE();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;

  // ---- this block's run of chunks
  const int per = (a.n_seqs + kDecThreads - 1) / kDecThreads;
  const int b_lo = min(tid * per, a.n_seqs), b_hi = min(b_lo + per, a.n_seqs);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += seq_cost(a, load_seq(a, b), RB);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before += incl - mine;
  const int grid = (int)min((long long)gridDim.x, total);  // blocks that get any; each of them at least one chunk
  if (tid == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if ((int)blockIdx.x >= grid) return;
  const long long c_begin = total * blockIdx.x / grid, c_end = total * (blockIdx.x + 1) / grid;
  if (mine > 0 && before <= c_begin && c_begin < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long cost = seq_cost(a, load_seq(a, b), RB);
      if (c_begin < at + cost) {
        s_b = b;
        s_local = c_begin - at;
        break;
      }
      at += cost;
    }
  }
  __syncthreads();

  long long left = c_end - c_begin;
  int b = s_b;
  long long local = s_local;
  long long at = c_begin;  // global index of the next chunk
  while (left > 0 && b < a.n_seqs) {
    const SeqSpan sq = load_seq(a, b);
    const long long cost = seq_cost(a, sq, RB);
    if (local >= cost) {
      local = 0;
      ++b;
      continue;
    }
    const int n_ch = seq_chunks(sq);
    const int rows = sq.n_q * a.G, n_rg = (rows + RB - 1) / RB;
    const int item = (int)(local / n_ch), k0 = (int)(local - (long long)item * n_ch);
    const int k1 = (int)min((long long)n_ch, k0 + left);
    const int h = item / n_rg, rg = item - h * n_rg;
    const int row_first = rg * RB;
    local += k1 - k0;
    left -= k1 - k0;
    at += k1 - k0;

    // ---- queries: thread (g, c) holds row g's quarter c as the B operand of every k step
    uint32_t bq[NR][KSTEPS][2];
    float fac[NR][2];
    int lim[NR][2], lim_min = 0x7fffffff;
    const float kts = a.cache.k_ts ? a.cache.k_ts[h] : 1.0f;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = row_first + 8 * r + g;
      const bool ok = row < rows;
      const int tok = ok ? row / a.G : 0, head = h * a.G + (ok ? row - tok * a.G : 0);
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(sq.q0 + tok) * a.q_stride + (int64_t)head * D +
                                                        c * (D / 4));
      uint4 raw[D / 32];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        raw[i] = ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        mx = __vmaxu2(mx, raw[i].x & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].y & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].z & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].w & 0x7FFF7FFFu);
      }
      int e = (int)(max(mx & 0xFFFFu, mx >> 16) >> 7) - 127;
      e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
      e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
      e = max(e, -100);
      const float up = __int_as_float((127 + 13 - e) << 23);  // the row's largest element becomes 2^13..2^14
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          bq[r][2 * i + (j >> 1)][j & 1] =
              pack_f16(bf16_to_f32(w[j] & 0xFFFFu) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ej = __shfl_sync(0xffffffffu, e, 4 * (2 * c + j));
        fac[r][j] = a.scale * kLog2e * kts * __int_as_float((127 - 13 + ej) << 23);
        const int rj = row_first + 8 * r + 2 * c + j;
        // keys that row may see: all of the context, or up to its own position
        lim[r][j] = rj >= rows ? 0 : a.causal ? max(sq.ctx - sq.n_q + rj / a.G + 1, 0) : sq.ctx;
        if (rj < rows) lim_min = min(lim_min, lim[r][j]);
      }
    }
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 1));
    lim_min = min(lim_min, __shfl_xor_sync(0xffffffffu, lim_min, 2));

    float o[NR][KSTEPS][4];
    float m[NR][2], l[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[r][i][j] = 0.0f;
      m[r][0] = m[r][1] = kNoMax;
      l[r][0] = l[r][1] = 0.0f;
    }

    // ---- keys: tiles of 16, dealt to the warps in turn
    const int tok_end = min(k1 * kChunk, sq.ctx);
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    const int ps = a.cache.page_size, psl = a.page_shift;
    auto page_of = [&](int t0) -> int {
      if (t0 >= tok_end) return -1;
      const int page = __ldg(table + (t0 >> psl));
      if (page < 0 || page >= a.cache.n_pages) {
        if (lane == 0) atomicExch(a.status, kStatusInvalid);
        return -1;
      }
      return page;
    };
    auto row_of = [&](int page, int t0) -> int64_t {
      return ((int64_t)page * a.cache.Hkv + h) * ps + (t0 & (ps - 1));
    };
    int t0 = k0 * kChunk + warp * 16;
    const int page = page_of(t0);
    Tile<D> cur, nxt;
    if (page >= 0)
      cur.load(a.cache, row_of(page, t0), g, c);
    else
      cur.zero();
    int page_n = page_of(t0 + kDecWarps * 16);
    for (; t0 < tok_end; t0 += kDecWarps * 16) {
      const int t1 = t0 + kDecWarps * 16;
      if (page_n >= 0)
        nxt.load(a.cache, row_of(page_n, t1), g, c);
      else
        nxt.zero();
      const int page_nn = page_of(t1 + kDecWarps * 16);
      // S^T = K Q^T
      float s[NR][4];
#pragma unroll
      for (int r = 0; r < NR; ++r) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.0f;
#pragma unroll
      for (int w = 0; w < Tile<D>::KW; ++w) {  // 8 elements of both rows: two k steps
        uint32_t f0[4], f1[4];
        e2m1x8_to_f16x2x4(cur.k[0][w], f0);
        e2m1x8_to_f16x2x4(cur.k[1][w], f1);
        // the scale of block w / 2 of this quarter in both halves
        const uint32_t sel = (w / 2) * 0x0011u;
        const uint32_t s0 = e4m3x2_to_f16x2(__byte_perm(cur.ks[0], 0, sel)),
                       s1 = e4m3x2_to_f16x2(__byte_perm(cur.ks[1], 0, sel));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f0[i] = hmul2(f0[i], s0);
          f1[i] = hmul2(f1[i], s1);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t fa[4] = {f0[2 * u], f1[2 * u], f0[2 * u + 1], f1[2 * u + 1]};
#pragma unroll
          for (int r = 0; r < NR; ++r) mma_f16(s[r], fa, bq[r][2 * w + u][0], bq[r][2 * w + u][1]);
        }
      }
      // softmax: columns (query rows) 2c and 2c + 1, keys g and g + 8
      const bool edge = t0 + 16 > lim_min;
      uint32_t pb[NR][2];
      bool raise = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[r][j] *= fac[r][j & 1];
          if (edge && t0 + g + 8 * (j >> 1) >= lim[r][j & 1]) s[r][j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) raise |= fmaxf(s[r][j], s[r][j + 2]) > m[r][j] + kRaise;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float fix[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[r][j], s[r][j + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            x = fmaxf(x, m[r][j]);
            fix[j] = ex2(m[r][j] - x);
            m[r][j] = x;
            l[r][j] *= fix[j];
          }
#pragma unroll
          for (int i = 0; i < KSTEPS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[r][i][j] *= fix[j & 1];
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = ex2(s[r][j] - m[r][j & 1]);
        l[r][0] += p[0] + p[2];
        l[r][1] += p[1] + p[3];
        pb[r][0] = transpose8x8(pack_f16(p[0], p[1]));
        pb[r][1] = transpose8x8(pack_f16(p[2], p[3]));
      }
      // O^T += V^T P^T
      uint32_t vs[4] = {cur.vs[0], cur.vs[1], cur.vs[2], cur.vs[3]};
      if (t0 + 16 > sq.ctx) {  // keys past the end: whatever the page holds there counts as 0
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t0 + 2 * c + (i & 1) + 8 * (i >> 1) >= sq.ctx) vs[i] = 0;
      }
      const uint32_t va = __byte_perm(vs[0], vs[1], 0x5140), vb = __byte_perm(vs[2], vs[3], 0x5140);
#pragma unroll
      for (int w = 0; w < Tile<D>::VW; ++w) {
        const uint32_t sa = e4m3x2_to_f16x2(w < 2 ? va & 0xFFFFu : va >> 16),
                       sb = e4m3x2_to_f16x2(w < 2 ? vb & 0xFFFFu : vb >> 16);
        const uint32_t x0 = cur.v[0][w], x1 = cur.v[1][w], x2 = cur.v[2][w], x3 = cur.v[3][w];
        constexpr uint32_t lo = 0x0F0F0F0Fu;
        uint32_t fe[4], fo[4], he[4], ho[4];
        e2m1x8_to_f16x2x4((x0 & lo) | ((x1 << 4) & ~lo), fe);
        e2m1x8_to_f16x2x4(((x0 >> 4) & lo) | (x1 & ~lo), fo);
        e2m1x8_to_f16x2x4((x2 & lo) | ((x3 << 4) & ~lo), he);
        e2m1x8_to_f16x2x4(((x2 >> 4) & lo) | (x3 & ~lo), ho);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t fa[4] = {hmul2(fe[i], sa), hmul2(fo[i], sa), hmul2(he[i], sb), hmul2(ho[i], sb)};
#pragma unroll
          for (int r = 0; r < NR; ++r) mma_f16(o[r][4 * w + i], fa, pb[r][0], pb[r][1]);
        }
      }
      cur = nxt;
      page_n = page_nn;
    }

    // ---- join the warps
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[r][j] += __shfl_xor_sync(0xffffffffu, l[r][j], d);
        if (g == 0) {
          s_m[warp][8 * r + 2 * c + j] = m[r][j];
          s_l[warp][8 * r + 2 * c + j] = l[r][j];
        }
      }
    __syncthreads();
    if (tid < RB) {
      float mm = kNoMax, ll = 0.0f;
      for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, s_m[w][tid]);
      for (int w = 0; w < kDecWarps; ++w) {
        const float f = ex2(s_m[w][tid] - mm);
        s_f[w][tid] = f;
        ll += s_l[w][tid] * f;
      }
      s_mm[tid] = mm;
      s_ll[tid] = ll;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * r + 2 * c + j;
        const float f = s_f[warp][row];
        float* dst = s_o + ((size_t)warp * RB + row) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < KSTEPS; ++i)
          *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[r][i][j] * f, o[r][i][j + 2] * f);
      }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == n_ch;
    const int side = k0 > 0 ? 0 : 1;
    float* part = a.partial + ((size_t)blockIdx.x * 2 + side) * a.part_stride;
    const float vts = a.cache.v_ts ? a.cache.v_ts[h] : 1.0f;
    for (int i = tid; i < RB * (D / 4); i += kDecThreads) {
      const int row = i / (D / 4), d4 = i - row * (D / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 v = reinterpret_cast<const float4*>(s_o + ((size_t)w * RB + row) * D)[d4];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (whole) {
        const int rr = row_first + row;
        if (rr < rows) {
          const int tok = rr / a.G, head = h * a.G + rr - tok * a.G;
          const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + head;
          const float ll = s_ll[row], f = ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
          const __nv_bfloat162 p0 = __floats2bfloat162_rn(acc.x * f, acc.y * f),
                               p1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
          *reinterpret_cast<uint2*>(a.out + out_row * D + d4 * 4) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
          if (a.lse && d4 == 0) a.lse[out_row] = ll == 0.0f ? -INFINITY : (s_mm[row] + log2f(ll)) * kLn2;
        }
      } else {
        reinterpret_cast<float4*>(part + 2 * RB)[i] = acc;
        if (d4 == 0) {
          part[row] = s_mm[row];
          part[RB + row] = s_ll[row];
        }
      }
    }
    if (!whole && side == 1 && tid == 0) {
      // the blocks after this one that hold the rest of the item
      const long long item_end = at + (n_ch - k1);
      int last = blockIdx.x + 1;
      while (total * (last + 1) / grid < item_end) ++last;
      a.meta[blockIdx.x] = make_int4(b, h, row_first, last);
    }
    __syncthreads();
  }
}

// One block per (run that ends inside an item, row): joins the item's partial results.
template <int D, int RB>
__global__ void __launch_bounds__(D / 4) kv_attn_join_kernel(const KvAttnArgs a) {
  MOE_PDL_PROLOGUE();
  const int4 meta = a.meta[blockIdx.x];
  if (meta.x < 0) return;
  const SeqSpan sq = load_seq(a, meta.x);
  const int row = blockIdx.y, rr = meta.z + row;
  if (rr >= sq.n_q * a.G) return;
  const int first = blockIdx.x, last = meta.w;
  auto part = [&](int i) { return a.partial + ((size_t)i * 2 + (i == first ? 1 : 0)) * a.part_stride; };
  float mm = kNoMax;
  for (int i = first; i <= last; ++i) mm = fmaxf(mm, part(i)[row]);
  float ll = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = first; i <= last; ++i) {
    const float* p = part(i);
    const float f = ex2(p[row] - mm);
    ll += p[RB + row] * f;
    const float4 v = reinterpret_cast<const float4*>(p + 2 * RB)[row * (D / 4) + threadIdx.x];
    acc.x += v.x * f;
    acc.y += v.y * f;
    acc.z += v.z * f;
    acc.w += v.w * f;
  }
  const int tok = rr / a.G, head = meta.y * a.G + rr - tok * a.G;
  const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + head;
  const float vts = a.cache.v_ts ? a.cache.v_ts[meta.y] : 1.0f;
  const float f = ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
  const __nv_bfloat162 p0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), p1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  *reinterpret_cast<uint2*>(a.out + out_row * D + threadIdx.x * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
  if (a.lse && threadIdx.x == 0) a.lse[out_row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

constexpr int dec_smem(int D, int NR) { return kDecWarps * 8 * NR * D * 4; }
constexpr int dec_blocks(int D, int NR) { return D == 256 || NR > 1 ? 1 : 2; }  // blocks of an SM

template <int D, int NR>
cudaError_t launch_dec(KvAttnArgs a, int num_sms, cudaStream_t st) {
  const int grid = num_sms * dec_blocks(D, NR);
  cudaError_t e = launch_pdl(kv_attn_dec_kernel<D, NR>, dim3(grid), dim3(kDecThreads), dec_smem(D, NR), st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_attn_join_kernel<D, 8 * NR>, dim3(grid, 8 * NR), dim3(D / 4), 0, st, a);
}

template <int D>
cudaError_t attributes_dec() {
  cudaError_t e = cudaFuncSetAttribute(kv_attn_dec_kernel<D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       dec_smem(D, 1));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kv_attn_dec_kernel<D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, dec_smem(D, 2));
}

}  // namespace

size_t kv_attn_dec_part_floats(int D) { return 16 * (size_t)(D + 2); }

cudaError_t init_kv_attn_dec_attributes() {
  cudaError_t e = attributes_dec<64>();
  if (e == cudaSuccess) e = attributes_dec<128>();
  if (e == cudaSuccess) e = attributes_dec<256>();
  return e;
}

cudaError_t launch_kv_attn_dec(const KvAttnArgs& a, int D, int num_sms, cudaStream_t st) {
  // one group of 8 rows where every sequence fits it, else groups of 16
  const bool one = (int64_t)a.max_q * a.G <= 8;
  if (D == 64) return one ? launch_dec<64, 1>(a, num_sms, st) : launch_dec<64, 2>(a, num_sms, st);
  if (D == 128) return one ? launch_dec<128, 1>(a, num_sms, st) : launch_dec<128, 2>(a, num_sms, st);
  return one ? launch_dec<256, 1>(a, num_sms, st) : launch_dec<256, 2>(a, num_sms, st);
}

}  // namespace moe

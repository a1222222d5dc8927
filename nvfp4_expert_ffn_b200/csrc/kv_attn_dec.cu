// Attention of few query rows per key head over the paged NVFP4 cache (decode steps, a few
// speculative tokens): out = softmax(scale q K^T) V with K and V read as 4-bit codes.
//
// Bound by the cache's bytes: 9/16 byte per element of K and V, read once per group of 8 NR
// query rows. A byte of codes is two elements, so the instructions per byte are what has to be
// few: the codes come by bulk copies into a ring that each warp keeps for itself (32 keys a
// stage, no registers and no address arithmetic while they are under way) and go from there
// straight into the operand registers of mma.sync (m16n8k16, float16 in, float32 out). The
// tensor pipe is idle most of the time here (8 query columns); tcgen05 would need the expanded
// tiles in shared memory.
//   S^T = K Q^T: keys are the 16 rows of the A operand. The order of the head's elements
//     along k is free as long as K and Q agree, so a thread's share of a key row is one
//     contiguous quarter: 16-byte loads, and a byte of codes expands (one conversion) to one
//     f16x2 register of the fragment, times the block's scale (one multiply, exact: 2 + 4
//     significant bits).
//   O^T = V^T P^T: the A operand pairs two keys of one element, so the codes of two keys are
//     interleaved nibble by nibble first (a quarter of an instruction per element); the scores'
//     fragments turn into P^T operands with movmatrix. Row r of a tile is key key_of(r), which
//     makes a thread's four keys of V four rows apart: a warp reads four whole rows at a time.
// What bounds it now is those instructions and the chain they make: 384 a warp for 16 keys of 128
// elements, from the codes to the products of P and V each waiting for the one before; 61% of the issue
// slots are used, the integer pipe (which converts the codes) is 55% busy, and 4 warps a scheduler do
// not cover the rest. One B200: 64 sequences over up to 8192 keys, 32 + 8 heads of 128, 100 us (3.6
// TB/s), 14 + 2 heads of 64 26.6 us (1.7 TB/s); 8 sequences near 16384 keys, 16 + 2 heads of 256, 31 us;
// one over 1000 keys 12.8 us. (With heads of 256 some registers are spilled: 92 bytes a thread by 8
// rows, 244 by 16.)
// q is scaled by a power of two per row into float16's range (exact; the factor returns in
// the softmax scale), the weights P are rounded to float16 (11 bits; the result is bf16, 8; see kLead),
// sums, maxima and the output stay in float32.
//
// The keys of all sequences and heads are cut into chunks of kChunk and dealt to the blocks in
// equal contiguous runs, so a batch of any shape fills the machine. A run that starts or ends
// inside a sequence leaves its partial result (row maxima, sums, unnormalised output) in the
// workspace, and a second small kernel joins them, a block a row, in the order of the keys. (The
// last block to finish a sequence joining its parts itself took longer: 14 us for nine parts of a
// D = 256 head, one load latency after another in a single block, against 3 us.)
#include <cuda_bf16.h>

#include "kv_attn.cuh"
#include "sm100.cuh"

namespace moe {

namespace {

constexpr int kChunk = 64;       // keys of a unit of work
constexpr int kStageKeys = 32;   // keys of a warp's stage
constexpr int kStages = 2;

// Warps of a block: what the registers of an SM allow (O and Q alone are 12 D / 32 NR of them).
__host__ __device__ constexpr int dec_warps(int D, int NR) { return D == 256 && NR == 1 ? 12 : 8; }
__host__ __device__ constexpr int dec_blocks(int D, int NR) { return D == 256 || NR > 1 ? 1 : 2; }  // of an SM
__host__ __device__ constexpr int stage_bytes(int D) { return kStageKeys * 2 * (D / 2 + D / 16); }
// The warps' outputs side by side: rows of D + 8 floats, so that the two rows' stores of lanes
// 8 apart fall into different banks. They lie over the ring where there is no room beside it.
__host__ __device__ constexpr int join_bytes(int D, int NR) { return dec_warps(D, NR) * 8 * NR * (D + 8) * 4; }
__host__ __device__ constexpr int ring_bytes(int D, int NR) { return dec_warps(D, NR) * kStages * stage_bytes(D); }
__host__ __device__ constexpr bool join_apart(int D, int NR) {
  return (ring_bytes(D, NR) + join_bytes(D, NR) + 2048) * dec_blocks(D, NR) <= 226 * 1024;
}
__host__ __device__ constexpr int dec_smem(int D, int NR) {
  const int ring = ring_bytes(D, NR), join = join_bytes(D, NR);
  return join_apart(D, NR) ? ring + join : ring > join ? ring : join;
}

// the key of a tile's row r: the rows that one thread holds as the k index of V (2c, 2c + 1,
// 2c + 8, 2c + 9) are keys c, c + 4, c + 8, c + 12
MOE_DEV int key_of(int r) { return (r & 8) | ((r & 1) << 2) | ((r & 7) >> 1); }

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

template <int WORDS>
MOE_DEV void load_words(uint32_t* dst, const uint8_t* src) {
  if constexpr (WORDS == 1) {
    dst[0] = *reinterpret_cast<const uint32_t*>(src);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    dst[0] = v.x;
    dst[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(src)[i];
      dst[4 * i] = v.x;
      dst[4 * i + 1] = v.y;
      dst[4 * i + 2] = v.z;
      dst[4 * i + 3] = v.w;
    }
  }
}

template <int BYTES>
MOE_DEV uint32_t load_scales(const uint8_t* src) {
  if constexpr (BYTES == 1) return *src;
  if constexpr (BYTES == 2) return *reinterpret_cast<const uint16_t*>(src);
  return *reinterpret_cast<const uint32_t*>(src);
}

// What the start and end of an item cost a block (queries, first keys, joining the warps), in
// chunks: 8 us of 0.5 us at D = 256, 4 us of 0.55 us below. Every block starts one item; the cost
// counts the further ones.
__host__ __device__ constexpr int start_chunks(int D) { return D == 256 ? 16 : 7; }

MOE_DEV int seq_chunks(const SeqSpan& s) { return max(1, (s.ctx + kChunk - 1) / kChunk); }

// Work of all items of a sequence (chunks and starts); 0 for one that this kernel leaves to the other.
MOE_DEV int64_t seq_cost(const KvAttnArgs& a, const SeqSpan& s, int rows_per_group, int start) {
  const int rows = s.n_q * a.G;
  if (rows == 0 || rows > a.dec_max_rows) return 0;
  return (int64_t)(seq_chunks(s) + start) * a.cache.Hkv * ((rows + rows_per_group - 1) / rows_per_group);
}

// Rows of outputs are kept in the order of the fragments: place 16 i + 2 g + e holds element
// g D / 8 + 2 i + e (m tile i, thread row g). Writes the four places from 4 q on.
template <int D>
MOE_DEV void write_row(const KvAttnArgs& a, const SeqSpan& sq, int h, int rr, int q, float4 v, float mm, float ll, float vts) {
  const int tok = rr / a.G;
  const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + h * a.G + rr - tok * a.G;
  const float f = ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
  uint16_t* dst = a.out + out_row * D + (q & 3) * 2 * (D / 8) + (q >> 2) * 2;
  *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(v.x * f, v.y * f);
  *reinterpret_cast<__nv_bfloat162*>(dst + D / 8) = __floats2bfloat162_rn(v.z * f, v.w * f);
  if (a.lse && q == 0) a.lse[out_row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// A run of key chunks [k0, k1) of one sequence, key head and group of rows.
struct Item {
  SeqSpan sq;
  int b, h, row_first, k0, k1, n_ch;
  long long end;  // where the item's work ends, counted over all items
};

template <int D, int NR>
__global__ void __launch_bounds__(32 * dec_warps(D, NR), dec_blocks(D, NR)) kv_attn_dec_kernel(const KvAttnArgs a) {
  constexpr int RB = 8 * NR, W = dec_warps(D, NR), THREADS = 32 * W;
  constexpr int KSTEPS = D / 16, start = start_chunks(D);
  constexpr int KW = D / 32, VW = D / 64;  // words of codes that a thread holds of a K row, of a V row
  constexpr int KS = D / 64, VS = D >= 128 ? D / 128 : 1;  // bytes of scales
  // a stage: codes of K, codes of V, scales of K, scales of V
  constexpr int kV = kStageKeys * D / 2, kKs = 2 * kV, kVs = kKs + kStageKeys * D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr bool kApart = join_apart(D, NR);
  float* s_o = reinterpret_cast<float*>(smem + (kApart ? ring_bytes(D, NR) : 0));  // [warps][RB][D + 8]
  __shared__ uint64_t s_full[W][kStages];
  __shared__ uint32_t s_bad[W][kStages];  // 16-key halves whose page number is outside the cache
  __shared__ float s_m[W][RB], s_l[W][RB];
  __shared__ __align__(16) uint4 s_q[RB * D / 8];
  __shared__ int s_e[RB];
  __shared__ float s_mm[RB], s_ll[RB];
  __shared__ long long s_scan[32];
  __shared__ long long s_local;
  __shared__ SeqSpan s_seq;
  __shared__ int s_b;
  __shared__ Patience s_wait;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  if (tid < W * kStages) {
    mbar_init(&s_full[tid / kStages][tid % kStages], 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    s_wait.abort = 0;
    s_wait.limit = wait_limit_ns();
  }
  MOE_PDL_PROLOGUE();

  if (a.dec_max_rows < 0x7fffffff && blockIdx.x == gridDim.x - 1) {
    plan_tiles<THREADS, D>(a, s_scan);
    __syncthreads();
  }

  // ---- this block's run of chunks
  const int per = (a.n_seqs + THREADS - 1) / THREADS;
  const int b_lo = min(tid * per, a.n_seqs), b_hi = min(b_lo + per, a.n_seqs);
  long long mine = 0;
  SeqSpan one = {};  // of a thread with one sequence, read once
  for (int b = b_lo; b < b_hi; ++b) {
    one = load_seq(a, b);
    mine += seq_cost(a, one, RB, start);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before += incl - mine;
  const int grid = (int)min((long long)gridDim.x, total);  // blocks that get any
  if (tid == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if ((int)blockIdx.x >= grid) return;
  const long long c_begin = total * blockIdx.x / grid, c_end = total * (blockIdx.x + 1) / grid;
  if (mine > 0 && before <= c_begin && c_begin < before + mine) {
    long long at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const SeqSpan sq = per == 1 ? one : load_seq(a, b);
      const long long cost = seq_cost(a, sq, RB, start);
      if (c_begin < at + cost) {
        s_seq = sq;
        s_b = b;
        s_local = c_begin - at;
        break;
      }
      at += cost;
    }
  }
  __syncthreads();

  uint8_t* ring = smem + warp * kStages * stage_bytes(D);
  uint32_t n_issued = 0, n_used = 0;  // this warp's stages
  const int ps = a.cache.page_size, rows_copy = min(ps, kStageKeys), copies = kStageKeys / rows_copy;
  // lanes 0..7 copy: array lane / 2 (codes of K, of V, scales of K, of V), part lane % 2
  const int arr = lane >> 1, part = lane & 1;
  const uint8_t* arr_src = arr == 0 ? a.cache.k_codes : arr == 1 ? a.cache.v_codes : arr == 2 ? a.cache.k_scales : a.cache.v_scales;
  const int arr_row = arr < 2 ? D / 2 : D / 16;
  const int arr_at = (arr == 0 ? 0 : arr == 1 ? kV : arr == 2 ? kKs : kVs) + part * rows_copy * arr_row;

  // ---- the runs of this block, one after the other
  long long at = c_begin, local = s_local;
  int b = s_b;
  SeqSpan sq = s_seq;
  auto next_item = [&](Item* it) {
    while (at < c_end && b < a.n_seqs) {
      const long long cost = seq_cost(a, sq, RB, start);
      if (local < cost) {
        const int n_ch = seq_chunks(sq), n_rg = (sq.n_q * a.G + RB - 1) / RB, cost1 = n_ch + start;
        const int item = (int)(local / cost1), lo = (int)(local - (long long)item * cost1);
        const int hi = (int)min((long long)cost1, lo + c_end - at);
        const int k0 = max(0, lo - start), k1 = max(0, hi - start);
        local += hi - lo;
        at += hi - lo;
        *it = Item{sq, b, item / n_rg, item % n_rg * RB, k0, k1, n_ch, at + cost1 - hi};
        if (k1 > k0) return true;
        continue;
      }
      local = 0;
      if (++b < a.n_seqs) sq = load_seq(a, b);
    }
    return false;
  };

  // ---- keys: stages of 32, dealt to the warps in turn
  constexpr int kStep = W * kStageKeys;
  int t_issue = 0, page = 0;
  auto tok_end_of = [](const Item& it) { return min(it.k1 * kChunk, it.sq.ctx); };
  // Does this lane copy of the stage that starts at key t, and from which page: the number is read a
  // stage early, and may be any.
  const bool copier = lane < 8 && part < copies;
  auto wanted_at = [&](const Item& it, int t) { return copier && t + part * rows_copy < tok_end_of(it); };
  auto page_of = [&](const Item& it, int t) {
    return wanted_at(it, t) ? a.block_table[(int64_t)it.b * a.max_pages + ((t + part * rows_copy) >> a.page_shift)] : 0;
  };
  auto issue = [&](const Item& it) {
    const int next = page_of(it, t_issue + kStep);
    if (t_issue < tok_end_of(it)) {
      const uint32_t slot = n_issued++ % kStages;
      const bool wanted = wanted_at(it, t_issue), good = wanted && page >= 0 && page < a.cache.n_pages;
      const uint32_t bads = __ballot_sync(0xffffffffu, wanted && !good), goods = __ballot_sync(0xffffffffu, good);
      if (lane == 0) {
        if (bads) atomicMax(a.status, kStatusInvalid);
        s_bad[warp][slot] = copies == 1 ? (bads ? 3u : 0u) : bads & 3u;
        mbar_arrive_expect_tx(&s_full[warp][slot], (__popc(goods & 0x0Fu) * (D / 2) + __popc(goods & 0xF0u) * (D / 16)) * rows_copy);
      }
      __syncwarp();
      if (good) {
        const int64_t row = ((int64_t)page * a.cache.Hkv + it.h) * ps + ((t_issue + part * rows_copy) & (ps - 1));
        bulk_g2s(ring + slot * stage_bytes(D) + arr_at, arr_src + row * arr_row, rows_copy * arr_row, &s_full[warp][slot]);
      }
    }
    page = next;
    t_issue += kStep;
  };
  auto prime = [&](const Item& it) {
    t_issue = it.k0 * kChunk + warp * kStageKeys;
    page = page_of(it, t_issue);
  };
  auto fill = [&](const Item& it) {
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue(it);
  };

  Item it, coming;
  bool more = next_item(&it), filled = false;
  while (more) {
    if (!filled) prime(it);  // (the page number comes beside the queries)
    const int tok_end = tok_end_of(it), rows = it.sq.n_q * a.G, row_first = it.row_first, h = it.h;
    // ---- queries: converted once by the block, 8 elements a thread, into shared memory; then thread
    // (g, c) holds row g's quarter c as the B operand of every k step. (Every warp converting for
    // itself was 300 instructions of code that runs once: its fetches took 4 us at D = 256.)
    constexpr int QL = D / 8;  // threads of a row; a quarter's 16-byte pieces are turned about by
                               // row and quarter, so that 8 lanes read 8 different places
    auto turned = [](int row, int qtr, int piece) {
      const int x = D == 256 ? ((row & 1) << 2) | qtr : D == 128 ? ((row & 1) << 1) | (qtr >> 1) : row & 1;
      return row * (D / 8) + qtr * (D / 32) + (piece ^ x);
    };
#pragma unroll 1
    for (int i = tid; i < (RB * QL + 31) / 32 * 32; i += THREADS) {
      const int r = i / QL, piece = i % QL, row = row_first + r;
      const bool live = row < rows && r < RB;
      const int tok = live ? row / a.G : 0, head = h * a.G + (live ? row - tok * a.G : 0);
      const uint4 raw = live ? reinterpret_cast<const uint4*>(a.q + (int64_t)(it.sq.q0 + tok) * a.q_stride + (int64_t)head * D)[piece]
                             : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t m2 = __vmaxu2(__vmaxu2(raw.x & 0x7FFF7FFFu, raw.y & 0x7FFF7FFFu), __vmaxu2(raw.z & 0x7FFF7FFFu, raw.w & 0x7FFF7FFFu));
      int e = (int)(max(m2 & 0xFFFFu, m2 >> 16) >> 7) - 127;
#pragma unroll
      for (int d = QL / 2; d > 0; d >>= 1) e = max(e, __shfl_xor_sync(0xffffffffu, e, d));
      e = max(e, -100);
      const float up = __int_as_float((127 + 13 - e) << 23);  // the row's largest element becomes 2^13..2^14
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = pack_f16(bf16_to_f32(w[j] & 0xFFFFu) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
      s_q[turned(r, piece / (D / 32), piece % (D / 32))] = make_uint4(f[0], f[1], f[2], f[3]);
      if (piece == 0) s_e[r] = e;
    }
    if (!filled) fill(it);
    __syncthreads();
    uint32_t bq[NR][KSTEPS][2];
    float fac[NR][2];
    int lim[NR][2], lim_min = 0x7fffffff;
    float ks = score_scale(a, h);
    ks += ks - ks;  // an infinity becomes NaN (a comparison and a choice took 0.3 us of 30.5)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 f = s_q[turned(8 * r + g, c, i)];
        bq[r][2 * i][0] = f.x;
        bq[r][2 * i][1] = f.y;
        bq[r][2 * i + 1][0] = f.z;
        bq[r][2 * i + 1][1] = f.w;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int ej = s_e[8 * r + 2 * c + j];
        fac[r][j] = ks * __int_as_float((127 - 13 + ej) << 23);
        const int rj = row_first + 8 * r + 2 * c + j;
        // keys that row may see: all of the context, or up to its own position
        lim[r][j] = rj >= rows ? 0 : a.causal ? max(it.sq.ctx - it.sq.n_q + rj / a.G + 1, 0) : it.sq.ctx;
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

#pragma unroll 1
    for (int t_stage = it.k0 * kChunk + warp * kStageKeys; t_stage < tok_end; t_stage += kStep) {
      const uint32_t slot = n_used % kStages;
      if (!__all_sync(0xffffffffu, wait_soon(&s_full[warp][slot], (n_used / kStages) & 1, &s_wait, a.status))) break;
      ++n_used;
      uint8_t* st = ring + slot * stage_bytes(D);
      const uint32_t bad = s_bad[warp][slot];
      if (bad || t_stage + kStageKeys > it.sq.ctx) {
        // keys past the end, whatever the page holds there, and rows of no page count as zeros
        for (int i = lane; i < kStageKeys * (D / 16); i += 32) {
          const int r = i / (D / 16);
          if (((bad >> (r / 16)) & 1u) || t_stage + r >= it.sq.ctx) st[kKs + i] = st[kVs + i] = 0;
        }
        fence_proxy_async_smem();  // (before the next copy over them)
        __syncwarp();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t0 = t_stage + 16 * half;
        if (t0 >= tok_end) break;
        const uint8_t* kc = st + (16 * half + key_of(g)) * (D / 2) + c * (D / 8);
        const uint8_t* vc = st + kV + (16 * half + c) * (D / 2) + g * (D / 16);
        uint32_t kk[2][KW], vv[4][VW], ks[2], vs[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_words<KW>(kk[i], kc + i * 8 * (D / 2));
          ks[i] = load_scales<KS>(st + kKs + (16 * half + key_of(g) + 8 * i) * (D / 16) + c * KS);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          load_words<VW>(vv[i], vc + i * 4 * (D / 2));
          vs[i] = load_scales<VS>(st + kVs + (16 * half + c + 4 * i) * (D / 16) + (D >= 128 ? g * VS : g / 2));
        }
        // S^T = K Q^T
        float s[NR][4];
#pragma unroll
        for (int r = 0; r < NR; ++r) s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.0f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {  // 8 elements of both rows: two k steps
          uint32_t f0[4], f1[4];
          e2m1x8_to_f16x2x4(kk[0][w], f0);
          e2m1x8_to_f16x2x4(kk[1][w], f1);
          // the scale of block w / 2 of this quarter in both halves
          const uint32_t sel = (w / 2) * 0x0011u;
          const uint32_t s0 = e4m3x2_to_f16x2(__byte_perm(ks[0], 0, sel)), s1 = e4m3x2_to_f16x2(__byte_perm(ks[1], 0, sel));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t fa[4] = {hmul2(f0[2 * u], s0), hmul2(f1[2 * u], s1), hmul2(f0[2 * u + 1], s0), hmul2(f1[2 * u + 1], s1)};
#pragma unroll
            for (int r = 0; r < NR; ++r) mma_f16(s[r], fa, bq[r][2 * w + u][0], bq[r][2 * w + u][1]);
          }
        }
        // softmax: columns (query rows) 2c and 2c + 1, tile rows g and g + 8
        const bool edge = t0 + 16 > lim_min;
        uint32_t pb[NR][2];
        bool raise = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[r][j] *= fac[r][j & 1];
            if (edge && t0 + key_of(g) + 8 * (j >> 1) >= lim[r][j & 1]) s[r][j] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) raise |= fmaxf(s[r][j], s[r][j + 2]) - m[r][j] > kLead + kRaise;
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
              x = fmaxf(x - kLead, m[r][j]);
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
        const uint32_t va = __byte_perm(vs[0], vs[1], 0x5140), vb = __byte_perm(vs[2], vs[3], 0x5140);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t sa = e4m3x2_to_f16x2(w < 2 ? va & 0xFFFFu : va >> 16),
                         sb = e4m3x2_to_f16x2(w < 2 ? vb & 0xFFFFu : vb >> 16);
          const uint32_t x0 = vv[0][w], x1 = vv[1][w], x2 = vv[2][w], x3 = vv[3][w];
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
      }
      __syncwarp();  // the stage has been read by all lanes
      issue(it);
    }
    // (a wait that ran out: no copy may land in what follows)
    for (; n_used < n_issued; ++n_used) {
      volatile int no_abort = 0;
      mbar_wait(&s_full[warp][n_used % kStages], (n_used / kStages) & 1, &no_abort, a.status);
    }

    // the next run's first keys come while this one is joined
    more = next_item(&coming);
    filled = kApart && more;
    if (filled) {
      prime(coming);
      fill(coming);
    }

    // ---- join the warps' results
    const bool whole = it.k0 == 0 && it.k1 == it.n_ch;
    const float vts = a.cache.v_ts ? a.cache.v_ts[h] : 1.0f;
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
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * r + 2 * c + j;
        float mm = kNoMax;
#pragma unroll 4
        for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][row]);
        const float f = ex2(m[r][j] - mm);
        float* dst = s_o + (warp * RB + row) * (D + 8) + 2 * g;
#pragma unroll
        for (int i = 0; i < KSTEPS; ++i)
          *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[r][i][j] * f, o[r][i][j + 2] * f);
      }
    if (tid < RB) {
      float mm = kNoMax, ll = 0.0f;
#pragma unroll 4
      for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][tid]);
#pragma unroll 4
      for (int w = 0; w < W; ++w) ll += s_l[w][tid] * ex2(s_m[w][tid] - mm);
      s_mm[tid] = mm;
      s_ll[tid] = ll;
    }
    __syncthreads();
    float* part_out = a.partial + ((size_t)blockIdx.x * 2 + (it.k0 > 0 ? 0 : 1)) * a.part_stride;
#pragma unroll 1
    for (int i = tid; i < RB * (D / 4); i += THREADS) {
      const int row = i / (D / 4), q = i - row * (D / 4);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < W; ++w) {
        const float4 v = reinterpret_cast<const float4*>(s_o + (w * RB + row) * (D + 8))[q];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (whole) {
        if (row_first + row < rows) write_row<D>(a, it.sq, h, row_first + row, q, acc, s_mm[row], s_ll[row], vts);
      } else {
        reinterpret_cast<float4*>(part_out + 2 * RB)[i] = acc;
        if (q == 0) {
          part_out[row] = s_mm[row];
          part_out[RB + row] = s_ll[row];
        }
      }
    }
    if (!whole && it.k0 == 0 && tid == 0) {
      // the blocks after this one that hold the rest of the item
      int last = blockIdx.x + 1;
      while (total * (last + 1) / grid < it.end) ++last;
      a.meta[blockIdx.x] = make_int4(it.b, h, row_first, last);
    }
    __syncthreads();
    if (more) {
      it = coming;
      if (!kApart) {
        fence_proxy_async_smem();  // the ring's next copies come after these reads and writes of it
        __syncthreads();
      }
    }
  }
}

// One block per (run that ends inside an item, row): joins the item's parts, eight loads at a time.
template <int D, int RB>
__global__ void __launch_bounds__(D / 4) kv_attn_join_kernel(const KvAttnArgs a) {
  MOE_PDL_PROLOGUE();
  const int first = blockIdx.x, row = blockIdx.y, q = threadIdx.x;
  const int4 meta = a.meta[first];
  if (meta.x < 0) return;
  const SeqSpan sq = load_seq(a, meta.x);
  const int rr = meta.z + row, last = meta.w;
  const float vts = a.cache.v_ts ? a.cache.v_ts[meta.y] : 1.0f;
  float mm = kNoMax, ll = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = first; j0 <= last; j0 += 8) {
    float pm[8], pl[8];
    float4 pv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = min(j0 + j, last);
      const float* p = a.partial + ((size_t)k * 2 + (k == first ? 1 : 0)) * a.part_stride;
      pm[j] = p[row];
      pl[j] = p[RB + row];
      pv[j] = reinterpret_cast<const float4*>(p + 2 * RB + row * D)[q];
    }
    float top = mm;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, pm[j]);
    const float f0 = ex2(mm - top);
    mm = top;
    ll *= f0;
    acc = make_float4(acc.x * f0, acc.y * f0, acc.z * f0, acc.w * f0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = j0 + j <= last ? ex2(pm[j] - top) : 0.0f;  // (past the last: the last again, not counted)
      ll += pl[j] * f;
      acc.x += pv[j].x * f;
      acc.y += pv[j].y * f;
      acc.z += pv[j].z * f;
      acc.w += pv[j].w * f;
    }
  }
  if (rr < sq.n_q * a.G) write_row<D>(a, sq, meta.y, rr, q, acc, mm, ll, vts);
}

template <int D, int NR>
cudaError_t launch_dec(const KvAttnArgs& a, int num_sms, cudaStream_t st) {
  const int grid = num_sms * dec_blocks(D, NR);
  cudaError_t e = launch_pdl(kv_attn_dec_kernel<D, NR>, dim3(grid), dim3(32 * dec_warps(D, NR)), dec_smem(D, NR), st, a);
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

int64_t kv_attn_dec_units(int64_t T, int n_seqs, int G, int Hkv, int D, int64_t keys) {
  return (T * G / 16 + n_seqs) * Hkv * ((keys + kChunk - 1) / kChunk + start_chunks(D));
}

cudaError_t set_wait_limit_kv_attn_dec(unsigned long long ns) { return set_wait_limit_here(ns); }

cudaError_t init_kv_attn_dec_attributes() {
  cudaError_t e = attributes_dec<64>();
  if (e == cudaSuccess) e = attributes_dec<128>();
  if (e == cudaSuccess) e = attributes_dec<256>();
  return e;
}

cudaError_t launch_kv_attn_dec(const KvAttnArgs& a, int D, int num_sms, cudaStream_t st) {
  // Rows 8 at a time where every sequence fits that, and where the longer ones are the other kernel's
  // and a single token fits it (beside a prompt, most of the rest are single tokens); else 16 at a
  // time, at half the warps. 64 single tokens over 4096 keys beside a prompt of 512, 32 + 8 heads of
  // 128: 125 us by 8, 162 by 16; 16 sequences of 4 tokens (16 rows) beside one: 88 and 80.
  const bool one = a.G <= 8 && ((int64_t)a.max_q * a.G <= 8 || a.dec_max_rows < 0x7fffffff);
  if (D == 64) return one ? launch_dec<64, 1>(a, num_sms, st) : launch_dec<64, 2>(a, num_sms, st);
  if (D == 128) return one ? launch_dec<128, 1>(a, num_sms, st) : launch_dec<128, 2>(a, num_sms, st);
  return one ? launch_dec<256, 1>(a, num_sms, st) : launch_dec<256, 2>(a, num_sms, st);
}

}  // namespace moe

// Attention of many query rows per key head over the paged NVFP4 cache (prompts and chunks of
// prompts): out = softmax(scale q K^T) V, both products on the tcgen05 tensor cores.
//
// A block takes tiles of query rows of one key head (row = token * G + head of the group, so the
// G heads that share keys share the expanded keys too), 256 rows for D <= 128 and 128 for D = 256,
// and walks over the keys KT at a time:
//   loader warp: a tile's codes and scales by bulk copies (a page's rows of one head are
//     contiguous) into a ring of raw slots, some ahead.
//   expander warps: raw slots to float16 (exact: 2 + 4 significant bits) in the 128-byte
//     swizzle. K rows are the K-major B operand of S = Q K^T; V rows, stored the same way, are
//     the MN-major B operand of O += P V, so neither is transposed.
//   two MMA warps: S = Q K^T, and O += P V. Q is float16, scaled by a power of two per row; P, an
//     A operand in TMEM, float16 too.
//   softmax warps: they copy S to registers first, so the next Q K^T can overwrite it while they
//     work. O is rescaled only when a row's maximum rises by more than 2^8 over the one in use;
//     the weights are below 2^15 in float16 (kLead), the sums in float32.
// D <= 128: two groups of 128 rows, a softmax thread to a row, KT = 128. The groups share the
//   expanded keys, which are a third of a softmax's instructions again, and S; O of both, S and
//   both P fill TMEM, so Q is in shared memory. Bound by the softmax warps' instructions and the
//   exponentials (256 x 128 scores in 3400 cycles, the products alone 2450). One group of 128 rows
//   a block with two threads a row took 2430 cycles for half as many: 27140 tokens in chunks over
//   caches up to 16K (32 + 8 heads, D = 128) 3350 us, now 2280 us (1220 TFLOP/s; 2650 us in a row
//   with itself, under the power limit). A prompt of 16384, 14 + 2 heads of 64, 734 us (655 TFLOP/s:
//   half the products for the same exponentials).
// D = 256: O, Q and S of 128 rows leave no columns for a second group or more than KT = 64 keys,
//   at which a Q K^T costs as much as at 128; bound by the products (1536 cycles of 1750 a tile).
//   A prompt of 16384 (16 + 2 heads) 2045 us (1075 TFLOP/s), 2280 us in a row with itself.
// The loops are kept short where that costs nothing: the roles' code together passes the
// instruction cache (an expander unrolled 16 times instead of 4 made the softmax 12% slower).
//
// Tiles have different numbers of keys (causal, ragged), so the work (key tiles, plus a few for
// each row tile's start and end) is dealt to the blocks in equal contiguous runs by prefix sums
// (plan_tiles), and row tiles that lie in more than one block are joined afterwards.
#include <cuda_bf16.h>

#include <type_traits>

#include "kv_attn.cuh"
#include "sm100.cuh"

namespace moe {

namespace {

constexpr int kHalf = 128;  // rows of one M = 128 product
constexpr int kSoftWarps = 8;

// The two forms. `pair`: two threads share a row of scores and a tile has 128 rows; otherwise a
// thread has a row, and a tile 256 rows, half of them to each group of four softmax warps.
template <int D>
struct Tc {
  static constexpr bool pair = D == 256;
  static constexpr int rows = TileShape<D>::rows, kt = TileShape<D>::kt;
  static_assert(rows == (pair ? kHalf : 2 * kHalf), "rows of a tile");
  static constexpr int exp_warps = pair ? 8 : 4;         // expanders, half of them for K
  static constexpr int mma_warp = kSoftWarps + exp_warps, load_warp = mma_warp + 2;
  static constexpr int threads = 32 * (kSoftWarps + exp_warps + 4);  // whole warpgroups
  // Registers of a thread: at the launch (what so many threads may have), then by role. A role's
  // setmaxnreg waits for registers that others gave back, so the shares must not exceed the
  // launch's.
  static constexpr int launch_regs = pair ? 96 : 128, soft_regs = pair ? 144 : 184;
  static constexpr int exp_regs = pair ? 64 : 72, last_regs = pair ? 64 : 72;
  static_assert(32 * (kSoftWarps * soft_regs + exp_warps * exp_regs + 4 * last_regs) <= threads * launch_regs, "registers");
  // TMEM columns: O, Q, S, two P; or the groups' O, S, and the groups' P
  static constexpr uint32_t q_col = D, s_col = pair ? q_col + D / 2 : 2 * D, p_col = s_col + kt;
  static_assert(p_col + kt <= 512, "TMEM columns");
  static constexpr int stages = 2;                       // expanded tiles of K, and of V
  // Raw tiles, K and V in turn. Copies may land in any order, and a wait for a parity is over while
  // the barrier is still in the phase before, so the expanders of K and of V must each have barriers
  // of their own: with an odd number of slots, whose fills take turns, twice as many as slots.
  static constexpr int raw_slots = D == 128 ? 3 : 8;
  static constexpr int raw_bars = raw_slots % 2 ? 2 * raw_slots : raw_slots;
  static_assert(raw_bars % 2 == 0 && raw_bars <= 8, "barriers of the raw tiles");
  static constexpr int tile_bytes = kt * D * 2;
  static constexpr int raw_bytes = kt * (D / 2 + D / 16);
  static constexpr int q_bytes = pair ? 0 : rows * D * 2;
  static constexpr int smem = q_bytes + 2 * stages * tile_bytes + raw_slots * raw_bytes + 1024;
};

struct TcShared {
  uint64_t raw_full[8], raw_empty[8], k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t q_full[2], s_full[2], s_empty, p_full[2], pv_done[2], drained[2];
  uint32_t bad[8];  // of a raw slot: groups of 16 keys whose page number is outside the cache
  uint32_t tmem;
  int idx;
  Patience wait;
  float x[2][kHalf];
  int e[2][kHalf];
};

// ---------------------------------------------------------------- TMEM helpers
MOE_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}

MOE_DEV void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

MOE_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] x B[smem], float16 -> float32, K = 16
MOE_DEV void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= A[smem] x B[smem]^T, float16 -> float32, K = 16
MOE_DEV void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, float16 A and B, float32 accumulator; B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// MN-major operand in the 128-byte swizzle: rows of 64 elements along N, one per k; 8 rows are
// 1024 bytes, the next 64 elements along N are `lbo` bytes on.
MOE_DEV uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <int N>
MOE_DEV void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
MOE_DEV void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// true in one lane of the (whole) warp, the same one every time
MOE_DEV bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// bar.sync over `n` threads with an OR of their predicates
MOE_DEV bool bar_or(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

// the largest of three
MOE_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Waits for two barriers at once, every other lane for the second (a wait that is over at once
// still costs the round trip). For a whole warp; the same answer in all lanes.
MOE_DEV bool wait_both(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1, Patience* w, int32_t* status) {
  const bool odd = threadIdx.x & 1;
  const bool ok = __all_sync(0xffffffffu, wait_soon(odd ? bar1 : bar0, odd ? parity1 : parity0, w, status));
  __syncwarp();  // what a barrier has made visible to the lanes that waited for it holds for the others (a vote orders no memory)
  return ok;
}

// The factor of a row's scores, 2^(e - 13) of the head's. Never zero, so that a masked score stays
// -infinity; NaN only for a row that sees a key, for the same reason. (In arithmetic, as the kernel of
// few rows has it, it cost 0.6% here, by the registers.)
MOE_DEV float row_factor(float ks, int e, int keys) {
  const float f = fmaxf(fabsf(ks) * __int_as_float((127 - 13 + e) << 23), 1.2e-38f);
  return !(fabsf(ks) < INFINITY) && keys > 0 ? __int_as_float(0x7fffffff) : f;
}

// Can a row of the warp have scores (s * fac, with |s| up to D times 2^14 times 6 * 448) past 2^22? There
// one fused step s * fac - m can leave a weight outside float16's range, because m is a rounded product:
// the products are then rounded first.
template <int D>
MOE_DEV bool scores_far(float fac) { return __any_sync(0xffffffffu, fac * (D * 16384.0f * 2688.0f) > 0x1p22f); }

// A run of key tiles of one row tile.
struct Run {
  int b, h, tile, u0, u1, n_units;
  long long end;  // where the row tile's work ends, counted over all heads
};

// Walks over the block's runs; every role of the block makes the same walk.
struct Walk {
  const RowTile* tiles;
  long long per_head, at, end;
  int n_tiles, idx, h, start;  // start: start_cost

  MOE_DEV bool next(Run* r) {
    while (at < end) {
      const RowTile t = tiles[idx];
      const long long first = (long long)h * per_head + t.start;
      const long long lo = at - first;
      const long long total = t.n_units + start;
      const long long hi = min(total, end - first);
      r->b = t.b;
      r->h = h;
      r->tile = t.tile;
      r->n_units = t.n_units;
      r->u0 = (int)max(0ll, lo - start);
      r->u1 = (int)max(0ll, hi - start);
      r->end = first + total;
      at = first + hi;
      if (hi == total && ++idx == n_tiles) {
        idx = 0;
        ++h;
      }
      if (r->u1 > r->u0) return true;
    }
    return false;
  }
};


// The run after this one and the start of its queries' way here, before the wait for the last
// product: four dependent loads (tile, sequence, query rows) otherwise stand between two runs.
template <int D>
struct NextRun {
  Run run;
  SeqSpan sq;
  bool more;

  MOE_DEV void get(const KvAttnArgs& a, Walk& walk, int row, int half) {
    more = walk.next(&run);
    if (!more) return;
    sq = load_seq(a, run.b);
    const int rr = run.tile * Tc<D>::rows + row;
    if (rr >= sq.n_q * a.G) return;
    const int tok = rr / a.G;
    const uint16_t* src = a.q + (int64_t)(sq.q0 + tok) * a.q_stride + (int64_t)(run.h * a.G + rr - tok * a.G) * D;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(src + half * 128));
    if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
  }
};

// ---------------------------------------------------------------- softmax, two threads a row
template <int D>
MOE_DEV void softmax_pair(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint32_t tmem, long long total, int grid) {
  using C = Tc<D>;
  constexpr int KT = C::kt, HK = KT / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quarter = warp & 3;  // half of the keys, of Q and of O
  const int row = quarter * 32 + lane;
  const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
  uint32_t tc = 0;  // key tiles so far
  bool ok = true;
  NextRun<D> next;
  next.get(a, walk, row, half);
  while (ok && next.more) {
    const Run run = next.run;
    const SeqSpan sq = next.sq;
    const int rows = sq.n_q * a.G, rr = run.tile * kHalf + row;
    const bool live = rr < rows;
    const int tok = live ? rr / a.G : 0, head = run.h * a.G + (live ? rr - tok * a.G : 0);
    const float ks = score_scale(a, run.h);
    const int lim = !live ? 0x7fffffff : a.causal ? max(sq.ctx - sq.n_q + tok + 1, 0) : sq.ctx;
    // ---- Q: this thread's half of the row
    float fac;
    {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(sq.q0 + tok) * a.q_stride +
                                                        (int64_t)head * D + half * (D / 2));
      uint4 raw[D / 16];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        raw[i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        mx = __vmaxu2(mx, raw[i].x & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].y & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].z & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].w & 0x7FFF7FFFu);
      }
      sh.e[half][row] = (int)(max(mx & 0xFFFFu, mx >> 16) >> 7) - 127;
      named_bar_sync(5, kSoftWarps * 32);
      const int e = max(max(sh.e[0][row], sh.e[1][row]), -100);
      // the row's largest element becomes 2^13..2^14; a negative scale turns its sign here
      const float up = copysignf(__int_as_float((127 + 13 - e) << 23), ks);
      fac = row_factor(ks, e, lim);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t f[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w[4] = {raw[4 * i + j].x, raw[4 * i + j].y, raw[4 * i + j].z, raw[4 * i + j].w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            f[4 * j + u] = pack_f16(bf16_to_f32(w[u] & 0xFFFFu) * up, __uint_as_float(w[u] & 0xFFFF0000u) * up);
        }
        tmem_st16(tl + C::q_col + half * (D / 4) + 16 * i, f);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[0]);
    }
    // keys that every row of the tile sees
    const int first_tok = run.tile * kHalf / a.G;
    const int lim_min = a.causal ? max(sq.ctx - sq.n_q + first_tok + 1, 0) : sq.ctx;
    float m = kNoMax;
    uint64_t l2 = pack2(0.0f, 0.0f);
    const uint64_t fac2 = pack2(fac, fac);
    auto keys = [&](auto rounded) {  // (two loops: a choice in one cost 1%)
      for (int u = run.u0; u < run.u1; ++u, ++tc) {
        // the scores, and the product that last read this tile's columns of P
        if (tc >= 2)
          ok = wait_both(&sh.s_full[0], tc & 1, &sh.pv_done[tc & 1], ((tc >> 1) - 1) & 1, &sh.wait, a.status) && ok;
        else
          ok = __all_sync(0xffffffffu, wait_soon(&sh.s_full[0], tc & 1, &sh.wait, a.status)) && ok;
        tc_fence_after();
        uint32_t s[HK];
#pragma unroll
        for (int i = 0; i < HK; i += 32) tmem_ld32(tl + C::s_col + half * HK + i, *reinterpret_cast<uint32_t(*)[32]>(&s[i]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty);
        if (u * KT + KT > lim_min) {
          const int left = lim - u * KT - half * HK;
#pragma unroll
          for (int i = 0; i < HK; ++i)
            if (i >= left) s[i] = 0xff800000u;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < HK; i += 2)
          mx4[(i / 2) & 3] = max3(mx4[(i / 2) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fac;
        // the two warps of these 32 rows decide together
        if (bar_or(1 + quarter, 64, mx - m > kLead + kRaise || !ok)) {
          sh.x[half][row] = mx;
          if (bar_or(1 + quarter, 64, !ok)) {
            ok = false;
            break;
          }
          const float top = fmaxf(fmaxf(sh.x[0][row], sh.x[1][row]) - kLead, m);
          if (u > run.u0) {
            const float fix = ex2(m - top);
            float a0, a1;
            unpack2(l2, a0, a1);
            l2 = pack2(a0 * fix, a1 * fix);
            ok = __all_sync(0xffffffffu, wait_soon(&sh.pv_done[(tc - 1) & 1], ((tc - 1) >> 1) & 1, &sh.wait, a.status));
            tc_fence_after();
            if (ok) {
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 32) {
                uint32_t o[32];
                tmem_ld32(tl + half * (D / 2) + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
                tmem_st32(tl + half * (D / 2) + c, o);
              }
              tmem_st_wait();
            }
          }
          m = top;
          bar_or(1 + quarter, 64, false);  // s_x is free again
        }
        const uint64_t nm2 = pack2(-m, -m);
        const uint32_t tp = tl + C::p_col + (tc & 1) * (KT / 2) + half * (HK / 2);
#pragma unroll
        for (int q = 0; q < HK / 32; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float s0 = __uint_as_float(s[32 * q + 2 * i]), s1 = __uint_as_float(s[32 * q + 2 * i + 1]);
            if constexpr (decltype(rounded)::value) {  // (in scalars: a product and a sum of pairs are fused)
              s0 = __fadd_rn(__fmul_rn(s0, fac), -m);
              s1 = __fadd_rn(__fmul_rn(s1, fac), -m);
            }
            const uint64_t x = decltype(rounded)::value ? pack2(s0, s1) : fma2(pack2(s0, s1), fac2, nm2);
            float x0, x1;
            unpack2(x, x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            l2 = add2(l2, pack2(x0, x1));
            p[i] = pack_f16(x0, x1);
          }
          tmem_st16(tp + 16 * q, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[tc & 1]);
      }
    };
    if (scores_far<D>(fac))
      keys(std::true_type{});
    else
      keys(std::false_type{});
    // ---- the run's result
    next.get(a, walk, row, half);
    float l0, l1;
    unpack2(l2, l0, l1);
    sh.x[half][row] = l0 + l1;
    if (ok) ok = __all_sync(0xffffffffu, wait_soon(&sh.pv_done[(tc - 1) & 1], ((tc - 1) >> 1) & 1, &sh.wait, a.status));
    tc_fence_after();
    if (bar_or(5, kSoftWarps * 32, !ok)) break;
    const float ll = sh.x[0][row] + sh.x[1][row];
    const bool whole = run.u0 == 0 && run.u1 == run.n_units;
    const float vts = a.cache.v_ts ? a.cache.v_ts[run.h] : 1.0f;
    const float f = !whole ? 1.0f : ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
    const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + head;
    const int side = run.u0 > 0 ? 0 : 1;
    float* part = a.partial + ((size_t)blockIdx.x * 2 + side) * a.part_stride;
#pragma unroll
    for (int c = 0; c < D / 2; c += 32) {
      uint32_t o[32];
      tmem_ld32(tl + half * (D / 2) + c, o);
      tmem_ld_wait();
      if (whole) {
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + half * (D / 2) + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * j]) * f,
                                                             __uint_as_float(o[8 * i + 2 * j + 1]) * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
        float4* dst = reinterpret_cast<float4*>(part + 2 * kHalf + row * D + half * (D / 2) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                               __uint_as_float(o[4 * i + 3]));
      }
    }
    if (half == 0) {
      if (!whole) {
        part[row] = m;
        part[kHalf + row] = ll;
      } else if (live && a.lse) {
        a.lse[out_row] = ll == 0.0f ? -INFINITY : (m + log2f(ll)) * kLn2;
      }
    }
    if (!whole && side == 1 && threadIdx.x == 0) {
      int last = blockIdx.x + 1;
      while (total * (last + 1) / grid < run.end) ++last;
      a.meta[blockIdx.x] = make_int4(run.b, run.h, run.tile * kHalf, last);
    }
    tc_fence_before();
    named_bar_sync(5, kSoftWarps * 32);  // s_x and s_e are free again, O has been read
  }
}

// ---------------------------------------------------------------- softmax, a thread a row
// Group g of four warps has the rows g * 128.. of the tile, and its own O and P in TMEM; group 1
// passes over a tile of no more than 128 rows. Both use one S: a group copies its scores to
// registers first, and the other group's Q K^T follows into the same columns, so the groups work
// half a period apart and neither waits for its own products.
template <int D>
MOE_DEV void softmax_rows(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint32_t tmem, uint8_t* s_q, long long total,
                          int grid) {
  using C = Tc<D>;
  constexpr int KT = C::kt;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp >> 2, quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16), to = tl + g * D, tp = tl + C::p_col + g * (KT / 2);
  uint32_t tc = 0;  // key tiles of this group so far
  bool ok = true;
  NextRun<D> next;
  next.get(a, walk, g * kHalf + row, 0);
  while (ok && next.more) {
    const Run run = next.run;
    const SeqSpan sq = next.sq;
    const int rows = sq.n_q * a.G, n = run.u1 - run.u0, first_row = run.tile * C::rows + g * kHalf;
    if (g == 1 && rows - run.tile * C::rows <= kHalf) {
      next.get(a, walk, g * kHalf + row, 0);
      continue;
    }
    const int rr = first_row + row;
    const bool live = rr < rows;
    const int tok = live ? rr / a.G : 0, head = run.h * a.G + (live ? rr - tok * a.G : 0);
    float m = kNoMax;
    uint64_t l2 = pack2(0.0f, 0.0f);
    float fac;
    const float ks = score_scale(a, run.h);
    const int lim = !live ? 0x7fffffff : a.causal ? max(sq.ctx - sq.n_q + tok + 1, 0) : sq.ctx;
    // ---- Q, float16 scaled by a power of two, K-major in the 128-byte swizzle
    {
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(sq.q0 + tok) * a.q_stride + (int64_t)head * D);
      uint4 raw[D / 8];
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        raw[i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        mx = __vmaxu2(mx, raw[i].x & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].y & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].z & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, raw[i].w & 0x7FFF7FFFu);
      }
      const int e = max((int)(max(mx & 0xFFFFu, mx >> 16) >> 7) - 127, -100);
      // the row's largest element becomes 2^13..2^14; a negative scale turns its sign here
      const float up = copysignf(__int_as_float((127 + 13 - e) << 23), ks);
      fac = row_factor(ks, e, lim);
      uint8_t* dst = s_q + g * (kHalf * D * 2) + row * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t f[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          f[u] = pack_f16(bf16_to_f32(w[u] & 0xFFFFu) * up, __uint_as_float(w[u] & 0xFFFF0000u) * up);
        *reinterpret_cast<uint4*>(dst + (i / 8) * (kHalf * 128) + (((i % 8) ^ (row & 7)) << 4)) =
            make_uint4(f[0], f[1], f[2], f[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();  // O of the run before has been read
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[g]);
    }
    // keys that every row of this half sees
    const int lim_min = a.causal ? max(sq.ctx - sq.n_q + first_row / a.G + 1, 0) : sq.ctx;
    const uint64_t fac2 = pack2(fac, fac);
    auto keys = [&](auto rounded) {  // (two loops: a choice in one cost 1%)
      for (int j = 0; j < n; ++j, ++tc) {
        ok = __all_sync(0xffffffffu, wait_soon(&sh.s_full[g], tc & 1, &sh.wait, a.status));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[KT];
#pragma unroll
        for (int i = 0; i < KT; i += 32) tmem_ld32(tl + C::s_col + i, *reinterpret_cast<uint32_t(*)[32]>(&s[i]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty);
        const int k0 = (run.u0 + j) * KT;
        if (k0 + KT > lim_min) {
          const int left = lim - k0;
#pragma unroll
          for (int i = 0; i < KT; ++i)
            if (i >= left) s[i] = 0xff800000u;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < KT; i += 2)
          mx4[(i / 2) & 3] = max3(mx4[(i / 2) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fac;
        if (__any_sync(0xffffffffu, mx - m > kLead + kRaise)) {
          const float top = fmaxf(mx - kLead, m);
          if (j > 0) {
            const float fix = ex2(m - top);
            float a0, a1;
            unpack2(l2, a0, a1);
            l2 = pack2(a0 * fix, a1 * fix);
            ok = __all_sync(0xffffffffu, wait_soon(&sh.pv_done[g], (tc - 1) & 1, &sh.wait, a.status));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fix);
              tmem_st16(to + c, o);
            }
            tmem_st_wait();
          }
          m = top;
        }
        const uint64_t nm2 = pack2(-m, -m);
#pragma unroll
        for (int q = 0; q < KT / 32; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float s0 = __uint_as_float(s[32 * q + 2 * i]), s1 = __uint_as_float(s[32 * q + 2 * i + 1]);
            if constexpr (decltype(rounded)::value) {  // (in scalars: a product and a sum of pairs are fused)
              s0 = __fadd_rn(__fmul_rn(s0, fac), -m);
              s1 = __fadd_rn(__fmul_rn(s1, fac), -m);
            }
            const uint64_t x = decltype(rounded)::value ? pack2(s0, s1) : fma2(pack2(s0, s1), fac2, nm2);
            float x0, x1;
            unpack2(x, x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            l2 = add2(l2, pack2(x0, x1));
            p[i] = pack_f16(x0, x1);
          }
          if (q == 0 && tc > 0) {  // the product that last read these columns
            ok = __all_sync(0xffffffffu, wait_soon(&sh.pv_done[g], (tc - 1) & 1, &sh.wait, a.status));
            tc_fence_after();
          }
          tmem_st16(tp + 16 * q, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sh.p_full[g]);
      }
    };
    if (scores_far<D>(fac))
      keys(std::true_type{});
    else
      keys(std::false_type{});
    if (!ok) break;
    next.get(a, walk, g * kHalf + row, 0);
    ok = __all_sync(0xffffffffu, wait_soon(&sh.pv_done[g], (tc - 1) & 1, &sh.wait, a.status));
    if (!ok) break;
    tc_fence_after();
    // ---- the run's result
    float l0, l1;
    unpack2(l2, l0, l1);
    const float ll = l0 + l1;
    const bool whole = run.u0 == 0 && run.u1 == run.n_units;
    const float vts = a.cache.v_ts ? a.cache.v_ts[run.h] : 1.0f;
    const float f = !whole ? 1.0f : ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
    const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + head;
    const int side = run.u0 > 0 ? 0 : 1;
    float* part = a.partial + ((size_t)blockIdx.x * 2 + side) * a.part_stride;
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      uint32_t o[32];
      tmem_ld32(to + c, o);
      tmem_ld_wait();
      if (whole) {
        if (live) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * j]) * f,
                                                             __uint_as_float(o[8 * i + 2 * j + 1]) * f);
              w[j] = *reinterpret_cast<const uint32_t*>(&v);
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
        float4* dst = reinterpret_cast<float4*>(part + 2 * C::rows + (g * kHalf + row) * D + c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                               __uint_as_float(o[4 * i + 3]));
      }
    }
    if (!whole) {
      part[g * kHalf + row] = m;
      part[C::rows + g * kHalf + row] = ll;
    } else if (live && a.lse) {
      a.lse[out_row] = ll == 0.0f ? -INFINITY : (m + log2f(ll)) * kLn2;
    }
    if (!whole && side == 1 && threadIdx.x == 0) {
      int last = blockIdx.x + 1;
      while (total * (last + 1) / grid < run.end) ++last;
      a.meta[blockIdx.x] = make_int4(run.b, run.h, run.tile * C::rows, last);
    }
  }
}

// ---------------------------------------------------------------- expanders
// 16 elements (8 bytes of codes, one scale) a lane and step, lanes side by side in the raw
// slot. A step is a whole number of 8 rows on, so a lane keeps its place in the swizzle; of its
// two 16-byte stores, lanes that would meet in a bank take the second one first.
template <int D>
MOE_DEV void expand(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint8_t* s_k, uint8_t* s_v, uint8_t* s_raw) {
  constexpr int KT = Tc<D>::kt, NS = Tc<D>::stages, RAW = Tc<D>::raw_slots, BARS = Tc<D>::raw_bars;
  constexpr int EW = Tc<D>::exp_warps / 2;  // expander warps of K, and of V
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int P = D / 16;                 // lanes of a row
  constexpr int STEPS = KT * P / (32 * EW), ROWS = 32 / P * EW;  // rows of a step
  constexpr int BATCH = STEPS < 4 ? STEPS : 4;  // loads before the first use
  static_assert(ROWS % 8 == 0 && STEPS % BATCH == 0, "a lane keeps its row modulo 8");
  const int pw = (warp - kSoftWarps) % EW;
  const bool is_v = warp >= kSoftWarps + EW;
  uint64_t* full = is_v ? sh.v_full : sh.k_full;
  uint64_t* empty = is_v ? sh.v_empty : sh.k_empty;
  const int row0 = (pw * 32 + lane) / P, part = lane % P;
  const bool swap = D >= 128 && (part & 4);
  const uint32_t off0 = (part >> 2) * (KT * 128) + row0 * 128 + (((((part & 3) << 1) | (swap ? 1 : 0)) ^ (row0 & 7)) << 4);
  const uint32_t off1 = off0 ^ 16;
  uint32_t tc = 0;
  bool ok = true;
  Run run;
  while (ok && walk.next(&run)) {
    const int ctx = load_seq(a, run.b).ctx;
#pragma unroll 1
    for (int u = run.u0; u < run.u1; ++u, ++tc) {
      const uint32_t n_raw = 2 * tc + (is_v ? 1 : 0), slot = n_raw % RAW, s = tc % NS;
      ok = wait_both(&sh.raw_full[n_raw % BARS], (n_raw / BARS) & 1, &empty[s], ((tc / NS) & 1) ^ 1, &sh.wait, a.status);
      if (!ok) break;
      const uint8_t* raw = s_raw + slot * Tc<D>::raw_bytes;
      const uint32_t bad = sh.bad[slot];
      const int left = ctx - u * KT;
      uint8_t* dst = (is_v ? s_v : s_k) + s * Tc<D>::tile_bytes;
#pragma unroll 1
      for (int first = 0; first < STEPS; first += BATCH) {
        uint2 codes[BATCH];
        uint32_t scales[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          codes[i] = reinterpret_cast<const uint2*>(raw)[((first + i) * EW + pw) * 32 + lane];
          scales[i] = (raw + KT * (D / 2))[((first + i) * EW + pw) * 32 + lane];
        }
        if (bad || left < KT) {  // keys past the end, and pages outside the cache, count as zeros
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int row = row0 + (first + i) * ROWS;
            if (row >= left || ((bad >> (row / 16)) & 1u)) scales[i] = 0u;
          }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const uint32_t w0 = swap ? codes[i].y : codes[i].x, w1 = swap ? codes[i].x : codes[i].y;
          const uint32_t sc = e4m3x2_to_f16x2(scales[i] * 0x0101u);
          uint32_t f[4];
          e2m1x8_to_f16x2x4(w0, f);
          *reinterpret_cast<uint4*>(dst + off0 + (first + i) * (ROWS * 128)) =
              make_uint4(hmul2(f[0], sc), hmul2(f[1], sc), hmul2(f[2], sc), hmul2(f[3], sc));
          e2m1x8_to_f16x2x4(w1, f);
          *reinterpret_cast<uint4*>(dst + off1 + (first + i) * (ROWS * 128)) =
              make_uint4(hmul2(f[0], sc), hmul2(f[1], sc), hmul2(f[2], sc), hmul2(f[3], sc));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.raw_empty[slot]);
        mbar_arrive(&full[s]);
      }
    }
  }
}

// ---------------------------------------------------------------- loader
template <int D>
MOE_DEV void load_raw(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint8_t* s_raw) {
  constexpr int KT = Tc<D>::kt, RAW = Tc<D>::raw_slots, BARS = Tc<D>::raw_bars;
  const int lane = threadIdx.x & 31;
  // a lane copies one page's part of the tile: at most KT / 16 pages
  uint32_t n_raw = 0;
  bool ok = true;
  Run run;
  const int ps = a.cache.page_size;
  const int rows = min(ps, KT);               // of a copy
  const int copies = KT / rows;               // of a slot
  while (ok && walk.next(&run)) {
    const int ctx = load_seq(a, run.b).ctx;
    const int32_t* table = a.block_table + (int64_t)run.b * a.max_pages;
    auto page_of = [&](int u) {
      const int t = u * KT + lane * rows;
      return lane < copies && t < ctx ? table[t >> a.page_shift] : 0;
    };
    int page = page_of(run.u0);
    for (int u = run.u0; u < run.u1 && ok; ++u) {
      const int next = page_of(u + 1);
      const int t = u * KT + lane * rows;
      const bool wanted = lane < copies && t < ctx;
      const bool good = wanted && page >= 0 && page < a.cache.n_pages;
      if (wanted && !good) atomicMax(a.status, kStatusInvalid);
      const uint32_t bads = __ballot_sync(0xffffffffu, wanted && !good), goods = __ballot_sync(0xffffffffu, good);
      const int64_t row = ((int64_t)page * a.cache.Hkv + run.h) * ps + (t & (ps - 1));
      uint32_t bad = 0;  // a copy of `rows` keys is rows / 16 groups of 16
      for (int j = 0; bads && j < copies; ++j)
        if ((bads >> j) & 1u) bad |= ((1u << (rows / 16)) - 1u) << (j * (rows / 16));
#pragma unroll 1
      for (int i = 0; i < 2; ++i, ++n_raw) {  // K, then V
        const uint32_t slot = n_raw % RAW;
        ok = __all_sync(0xffffffffu, wait_soon(&sh.raw_empty[slot], ((n_raw / RAW) & 1) ^ 1, &sh.wait, a.status));
        if (!ok) break;
        uint64_t* landed = &sh.raw_full[n_raw % BARS];
        uint8_t* raw = s_raw + slot * Tc<D>::raw_bytes;
        if (lane == 0) {
          sh.bad[slot] = bad;
          mbar_arrive_expect_tx(landed, __popc(goods) * rows * (D / 2 + D / 16));
        }
        __syncwarp();
        if (good) {
          bulk_g2s(raw + lane * rows * (D / 2), (i ? a.cache.v_codes : a.cache.k_codes) + row * (D / 2), rows * (D / 2),
                   landed);
          bulk_g2s(raw + KT * (D / 2) + lane * rows * (D / 16), (i ? a.cache.v_scales : a.cache.k_scales) + row * (D / 16),
                   rows * (D / 16), landed);
        }
      }
      page = next;
    }
  }
  // no copy may still be landing when the block ends
  __syncwarp();
  for (uint32_t j = n_raw > RAW ? n_raw - RAW : 0; j < n_raw; ++j) {
    volatile int no_abort = 0;
    mbar_wait(&sh.raw_full[j % BARS], (j / BARS) & 1, &no_abort, a.status);
  }
}

// ---------------------------------------------------------------- products
// One warp issues S = Q K^T and another O += P V, each with its own waits: an issue holds its warp
// until the tensor core has taken the instruction, and one warp for both left the core idle for
// the length of every wait. The whole warp takes the walk and the waits, so that descriptors are
// the same in every lane (uniform registers); one elected lane issues.

// row groups of a run (a form of one group has one)
template <int D>
MOE_DEV int run_groups(const KvAttnArgs& a, const Run& run) {
  return !Tc<D>::pair && load_seq(a, run.b).n_q * a.G - run.tile * Tc<D>::rows > kHalf ? 2 : 1;
}

// TMEM and shared memory are given back only after every product is done with them
MOE_DEV void drain(uint64_t* bar, int32_t* status) {
  if (elect_one()) {
    mma_commit(bar);
    volatile int no_abort = 0;
    mbar_wait(bar, 0, &no_abort, status);
  }
  __syncwarp();
}

template <int D>
MOE_DEV void products_qk(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint32_t tmem, const uint8_t* s_q, const uint8_t* s_k) {
  using C = Tc<D>;
  constexpr int KT = C::kt, NS = C::stages;
  constexpr uint32_t idesc = idesc_f16(kHalf, KT, false);
  uint32_t tc = 0, n_s = 0, items[2] = {0, 0};  // key tiles, S, and runs of each group so far
  bool ok = true;
  Run run;
  const uint64_t desc_q = sdesc_sw128(smem_u32(s_q)), desc_k = sdesc_sw128(smem_u32(s_k));
  while (ok && walk.next(&run)) {
    const int groups = run_groups<D>(a, run), n = run.u1 - run.u0;
    for (int i = 0; i < n * groups; ++i, ++n_s) {
      const int g = groups == 2 ? i & 1 : 0, j = groups == 2 ? i >> 1 : i;
      const uint32_t t = tc + j, s = t % NS;
      if (j == 0) ok = __all_sync(0xffffffffu, wait_soon(&sh.q_full[g], (g ? items[1] : items[0]) & 1, &sh.wait, a.status));
      // once the scores before have been copied
      ok = ok && wait_both(&sh.k_full[s], (t / NS) & 1, &sh.s_empty, (n_s & 1) ^ 1, &sh.wait, a.status);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dq = desc_q + ((g * (kHalf * D * 2)) >> 4), dk = desc_k + s * (C::tile_bytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t in = (kk % 4) * 32, bk = ((kk / 4) * (KT * 128) + in) >> 4;
          if constexpr (C::pair)
            mma_f16_ts(tmem + C::s_col, tmem + C::q_col + 8 * kk, dk + bk, idesc, kk ? 1u : 0u);
          else
            mma_f16_ss(tmem + C::s_col, dq + (((kk / 4) * (kHalf * 128) + in) >> 4), dk + bk, idesc, kk ? 1u : 0u);
        }
        mma_commit(&sh.s_full[g]);
        if (g + 1 == groups) mma_commit(&sh.k_empty[s]);
      }
      __syncwarp();
    }
    tc += n;
    items[0] += 1;
    items[1] += groups - 1;
  }
  drain(&sh.drained[0], a.status);
}

template <int D>
MOE_DEV void products_pv(const KvAttnArgs& a, TcShared& sh, Walk& walk, uint32_t tmem, const uint8_t* s_v) {
  using C = Tc<D>;
  constexpr int KT = C::kt, NS = C::stages;
  constexpr uint32_t idesc = idesc_f16(kHalf, D, true);
  uint32_t tc = 0, used[2] = {0, 0};  // key tiles, and of each group, so far
  bool ok = true;
  Run run;
  const uint64_t desc_v = sdesc_mn_sw128(smem_u32(s_v), KT * 128);
  while (ok && walk.next(&run)) {
    const int groups = run_groups<D>(a, run), n = run.u1 - run.u0;
    for (int i = 0; i < n * groups; ++i) {
      const int g = groups == 2 ? i & 1 : 0, j = groups == 2 ? i >> 1 : i;
      const uint32_t t = tc + j, s = t % NS;
      // the buffer of P and its turn
      const uint32_t b = C::pair ? t & 1 : g, at = C::pair ? t >> 1 : (g ? used[1] : used[0]) + j;
      ok = wait_both(&sh.p_full[b], at & 1, &sh.v_full[s], (t / NS) & 1, &sh.wait, a.status);
      if (!ok) break;
      tc_fence_after();
      const uint64_t dv = desc_v + s * (C::tile_bytes >> 4);
      const uint32_t p = tmem + C::p_col + b * (KT / 2), add = j ? 1u : 0u;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_f16_ts(tmem + g * D, p + 8 * kk, dv + ((kk * 2048) >> 4), idesc, kk ? 1u : add);
        mma_commit(&sh.pv_done[b]);
        if (g + 1 == groups) mma_commit(&sh.v_empty[s]);
      }
      __syncwarp();
    }
    tc += n;
    used[0] += n;
    used[1] += (groups - 1) * n;
  }
  drain(&sh.drained[1], a.status);
}

template <int D>
__global__ void __launch_bounds__(Tc<D>::threads, 1) kv_attn_tc_kernel(const KvAttnArgs a) {
  using C = Tc<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* s_q = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* s_k = s_q + C::q_bytes;
  uint8_t* s_v = s_k + C::stages * C::tile_bytes;
  uint8_t* s_raw = s_v + C::stages * C::tile_bytes;
  __shared__ TcShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    constexpr int EW = C::exp_warps / 2, soft = C::pair ? kSoftWarps : kSoftWarps / 2;
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(&sh.k_full[s], EW);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_full[s], EW);
      mbar_init(&sh.v_empty[s], 1);
    }
    for (int i = 0; i < C::raw_bars; ++i) mbar_init(&sh.raw_full[i], 1);
    for (int i = 0; i < C::raw_slots; ++i) mbar_init(&sh.raw_empty[i], EW);
    mbar_init(&sh.s_empty, soft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], soft);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], soft);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.drained[i], 1);
    }
    fence_barrier_init();
    sh.wait.abort = 0;
    sh.wait.limit = wait_limit_ns();
  }
  MOE_PDL_PROLOGUE();
  // (not before the wait: a block of an earlier kernel that has yet to allocate would wait for this one)
  if (warp == C::mma_warp) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // ---- this block's run of the work
  Walk walk;
  walk.tiles = reinterpret_cast<const RowTile*>(a.tiles);
  walk.per_head = a.plan[0];
  walk.n_tiles = (int)a.plan[1];
  const long long total = walk.per_head * a.cache.Hkv;
  const int grid = (int)min((long long)gridDim.x, total);
  walk.at = walk.end = 0;
  walk.start = TileShape<D>::start_cost;
  if ((int)blockIdx.x < grid) {
    walk.at = total * blockIdx.x / grid;
    walk.end = total * (blockIdx.x + 1) / grid;
    walk.h = (int)(walk.at / walk.per_head);
    const long long x = walk.at - walk.h * walk.per_head;
    if (warp == 0) {  // the last tile that starts at or before x: 32 probes a round
      int lo = 0, hi = walk.n_tiles;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int probe = lo + lane * step;
        const bool le = probe < hi && walk.tiles[probe].start <= x;
        const int n = __popc(__ballot_sync(0xffffffffu, le));
        lo += (n - 1) * step;
        hi = min(hi, lo + step);
      }
      if (lane == 0) sh.idx = lo;
    }
  }
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  walk.idx = sh.idx;

  if (warp < kSoftWarps) {
    more_registers<C::soft_regs>();
    if constexpr (C::pair)
      softmax_pair<D>(a, sh, walk, tmem, total, grid);
    else
      softmax_rows<D>(a, sh, walk, tmem, s_q, total, grid);
  } else if (warp < C::mma_warp) {
    fewer_registers<C::exp_regs>();
    expand<D>(a, sh, walk, s_k, s_v, s_raw);
  } else {
    fewer_registers<C::last_regs>();
    if (warp == C::load_warp) {
      load_raw<D>(a, sh, walk, s_raw);
    } else if (warp == C::mma_warp) {
      products_qk<D>(a, sh, walk, tmem, s_q, s_k);
    } else if (warp == C::mma_warp + 1) {
      products_pv<D>(a, sh, walk, tmem, s_v);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::mma_warp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the row tiles that lie in several blocks: one block per (run that ends inside a row
// tile, 8 rows), a warp a row.
template <int D>
__global__ void __launch_bounds__(256) kv_attn_tc_join_kernel(const KvAttnArgs a) {
  MOE_PDL_PROLOGUE();
  const int4 meta = a.meta[blockIdx.x];
  if (meta.x < 0) return;
  const SeqSpan sq = load_seq(a, meta.x);
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31, rr = meta.z + row;
  if (rr >= sq.n_q * a.G) return;
  const int first = blockIdx.x, last = meta.w;
  auto part = [&](int i) { return a.partial + ((size_t)i * 2 + (i == first ? 1 : 0)) * a.part_stride; };
  constexpr int V = D / 64, N = 4;  // float2 of a lane
  float mm = kNoMax, ll = 0.0f;
  float2 acc[V] = {};
  // N parts' loads under way together: a few rows over a long context have many (74 for 16 tokens over
  // 16000 keys, 69 us one by one, 63 so; eight at a time cost the usual two or three 3 us)
  for (int i0 = first; i0 <= last; i0 += N) {
    float pm[N], pl[N];
    float2 v[N][V];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool some = i0 + k <= last;
      const float* p = part(some ? i0 + k : last);
      pm[k] = some ? p[row] : kNoMax;
      pl[k] = some ? p[Tc<D>::rows + row] : 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j)
        v[k][j] = some ? reinterpret_cast<const float2*>(p + 2 * Tc<D>::rows + row * D)[j * 32 + lane] : make_float2(0.0f, 0.0f);
    }
    float top = mm;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, pm[k]);
    const float f0 = ex2(mm - top);
    mm = top;
    ll *= f0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      acc[j].x *= f0;
      acc[j].y *= f0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float f = ex2(pm[k] - top);
      ll += pl[k] * f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        acc[j].x += v[k][j].x * f;
        acc[j].y += v[k][j].y * f;
      }
    }
  }
  const int tok = rr / a.G, head = meta.y * a.G + rr - tok * a.G;
  const int64_t out_row = (int64_t)(sq.q0 + tok) * a.Hq + head;
  const float vts = a.cache.v_ts ? a.cache.v_ts[meta.y] : 1.0f;
  const float f = ll > 0.0f ? vts / ll : (ll == 0.0f ? 0.0f : ll);
#pragma unroll
  for (int j = 0; j < V; ++j)
    reinterpret_cast<__nv_bfloat162*>(a.out + out_row * D)[j * 32 + lane] = __floats2bfloat162_rn(acc[j].x * f, acc[j].y * f);
  if (a.lse && lane == 0) a.lse[out_row] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

template <int D>
cudaError_t launch_tc(const KvAttnArgs& a, int num_sms, cudaStream_t st) {
  using C = Tc<D>;
  cudaError_t e = launch_pdl(kv_attn_tc_kernel<D>, dim3(num_sms), dim3(C::threads), C::smem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_attn_tc_join_kernel<D>, dim3(num_sms, C::rows / 8), dim3(256), 0, st, a);
}

}  // namespace

size_t kv_attn_tc_part_floats(int D) { return (size_t)(D == 256 ? Tc<256>::rows : Tc<128>::rows) * (D + 2); }
int kv_attn_tc_max_tiles(int64_t T, int n_seqs, int G) { return (int)(T * G / kHalf + n_seqs + 1); }
size_t kv_attn_tc_tiles_bytes(int64_t T, int n_seqs, int G) {
  return (size_t)kv_attn_tc_max_tiles(T, n_seqs, G) * sizeof(RowTile);
}

cudaError_t set_wait_limit_kv_attn_tc(unsigned long long ns) { return set_wait_limit_here(ns); }

template <int D>
static cudaError_t attributes_tc() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, kv_attn_tc_kernel<D>);
  if (e != cudaSuccess) return e;
  if (at.numRegs != Tc<D>::launch_regs) return cudaErrorInvalidKernelImage;  // the roles' shares would not add up
  return cudaFuncSetAttribute(kv_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::smem);
}

cudaError_t init_kv_attn_tc_attributes() {
  cudaError_t e = attributes_tc<64>();
  if (e == cudaSuccess) e = attributes_tc<128>();
  if (e == cudaSuccess) e = attributes_tc<256>();
  return e;
}

cudaError_t launch_kv_attn_tc(const KvAttnArgs& a, int D, int num_sms, cudaStream_t st) {
  if (D == 64) return launch_tc<64>(a, num_sms, st);
  if (D == 128) return launch_tc<128>(a, num_sms, st);
  return launch_tc<256>(a, num_sms, st);
}

}  // namespace moe

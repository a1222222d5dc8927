// Writing and reading the paged NVFP4 key/value cache, and the norm and rotation of queries
// and keys that goes before the write.
//
// Per head row x of D elements:  y = x / sqrt(mean(x^2) + eps) * w, then the first R elements
// rotated in pairs by pos * f_p (cos and sin times a factor m), rounded to float32 and then to
// bf16. A cached key is the NVFP4 quantisation of that bf16 row, so the fused write stores
// exactly what the norm/rotation call followed by nvfp4_quantize_act would.
//
// Angles are float64 everywhere (positions times frequencies reach 10^6 radians). Keys are
// float64 up to their rounding: a row that differs by one float32 rounding can land on the other
// side of a bf16 step, that on the other side of an E2M1 step, and the stored value is then off
// by up to half of itself. Queries end in bf16 and are float32.
//
// Per token Hq + 2 Hkv rows of 2D bytes are read, Hq rows written, 9/16 byte a cached element: for
// many tokens HBM's bytes would bound it. Nothing is full: issue slots 73 to 74%, 7 of 16 warps a scheduler
// (64 registers a thread, and the tables' shared memory), which wait for dependent instructions, shared
// memory and loads in about equal parts. One B200: norm and rotation of 16384 tokens (32 + 8 heads of
// 128) 78 to 80 us, 4.3 TB/s; with the write of keys and values, and those read back, 27140 tokens 199 us,
// 3.7 TB/s. For a few tokens the launch and the float64 sine and cosine: 4.1 us for 8 tokens (16 + 2 heads
// of 256), 7.4 us with the write and the read back.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_attn.cuh"

namespace moe {

namespace {

// Many tokens: blocks of four warps, each with a token of its own, whose rows it walks over with
// constant strides. Few: a block of eight warps for every token.
constexpr int kManyWarps = 4, kFewWarps = 8;

MOE_DEV void unpack8x2(const uint4& p, uint64_t (&v)[4]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// Quotients by Markstein's theorem (P. Markstein, IBM J. Res. Dev. 34, 1990): with y the
// correctly rounded 1 / d, q = x y, r = x - q d (exact in a fused step), q + r y is the correctly
// rounded x / d, unless d's significand is all ones, or a step over- or underflows.
MOE_DEV bool good_divisor(float d) {
  return d > 0x1p-60f && d < 0x1p60f && (__float_as_uint(d) & 0x7FFFFFu) != 0x7FFFFFu;
}
MOE_DEV float quotient(float x, float d, float y) {
  const float q = __fmul_rn(x, y);
  return __fmaf_rn(__fmaf_rn(-q, d, x), y, q);
}

// Two lanes hold a block of 16 (8 elements each); amax is the block's, y the correctly rounded
// 1 / ts. The scale and codes of quantize_block16 (common.cuh): E2M1 of the correctly rounded
// x / denom. Blocks that the theorem does not cover are divided (an underflow on the way is none:
// the result is 0 either way). The sign is x's own where the theorem is used: that of a zero is
// lost on the way.
MOE_DEV uint32_t quantize_half16(const uint4& p, float amax, float ts, float y, uint32_t* codes) {
  const bool good = good_divisor(ts) && amax < 0x1p60f;
  const float sb = good ? quotient(quotient(amax, kE2M1Max, 1.0f / kE2M1Max), ts, y) : __fdiv_rn(__fdiv_rn(amax, kE2M1Max), ts);
  const uint32_t s = f32_to_e4m3_sat(sb);
  *codes = 0;
  if ((s & 0x7Fu) == 0) return s;
  const float d = __fmul_rn(__half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(s))), ts);
  uint64_t v[4];
  unpack8x2(p, v);
  if (!good || !good_divisor(d)) {
    const float denom = __fmul_rn(e4m3_to_f32(s), ts);  // (which takes the scale of a NaN for a number)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(v[i], lo, hi);
      *codes |= f32x2_to_e2m1x2(__fdiv_rn(lo, denom), __fdiv_rn(hi, denom)) << (8 * i);
    }
    return s;
  }
  float q[8];
  const float yd = __frcp_rn(d);
  const uint64_t y2 = pack2(yd, yd), d2 = pack2(-d, -d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t q0 = mul2(v[i], y2);
    unpack2(fma2(fma2(q0, d2, v[i]), y2, q0), q[2 * i], q[2 * i + 1]);
  }
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[2 * i] = __uint_as_float((__float_as_uint(q[2 * i]) & 0x7FFFFFFFu) | ((w[i] << 16) & 0x80000000u));
    q[2 * i + 1] = __uint_as_float((__float_as_uint(q[2 * i + 1]) & 0x7FFFFFFFu) | (w[i] & 0x80000000u));
  }
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(*codes)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return s;
}

MOE_DEV void unpack8(const uint4& p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

MOE_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// An angle less its whole turns, 2 pi in two parts (Cody and Waite): exact to 2^-50 up to 2^40
// radians. The library's own reduction of arguments beyond 10^5 takes a slow path.
MOE_DEV double whole_turns_off(double t) {
  constexpr double kTurn = 6.283185307179586, kTurnLow = 2.4492935982947064e-16;
  if (!(fabs(t) < 0x1p40)) return t;
  const double k = rint(t * (1.0 / kTurn));
  return fma(-k, kTurnLow, fma(-k, kTurn, t));
}

// A row's norm factor from its sum of squares: one Newton step in float64 from the float32
// reciprocal square root (2^-22 off) leaves 2^-43.
MOE_DEV double norm_factor(double ss, int D, double eps) {
  const double x = ss / D + eps;
  if (!(x > 1e-30 && x < 1e30)) return 1.0 / sqrt(x);
  const double y = (double)rsqrtf((float)x);
  return y * (1.5 - 0.5 * x * y * y);
}

// A bf16 of a packed pair as float64, 2^-896 of it: the exponent's bits are only moved, zeros
// and subnormals included, in a quarter of a conversion's time. (Infinities and NaN become
// numbers.)
constexpr double kUp = 0x1p896;
MOE_DEV double widen(uint32_t w, int high) {
  const uint32_t hi = high ? ((w & 0x7FFF0000u) >> 3) | (w & 0x80000000u) : ((w & 0x7FFFu) << 13) | ((w & 0x8000u) << 16);
  return __hiloint2double((int)hi, 0);
}
MOE_DEV double bf16_to_f64(uint32_t w, int high) { return (double)__uint_as_float(high ? w & 0xFFFF0000u : w << 16); }

// Calls body(row's 16 bytes, head, live) for the heads first + sub, first + step + sub, ... of a
// token, PF rows' loads under way: one row at a time leaves most of the memory's latency
// uncovered.
template <int PF, typename Body>
MOE_DEV void each_row(const uint16_t* x, int heads, int first, int sub, int step, int D, int e0, Body body) {
  const uint16_t* src = x + (first + sub) * D + e0;
  int ahead = first + sub;
  uint4 p[PF];
  auto load = [&]() {
    const uint4 v = ahead < heads ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
    ahead += step;
    src += step * D;
    return v;
  };
#pragma unroll
  for (int i = 0; i < PF; ++i) p[i] = load();
#pragma unroll 1
  for (int h = first; h < heads;) {
#pragma unroll
    for (int i = 0; i < PF; ++i) {
      if (h >= heads) break;
      const uint4 v = p[i];
      p[i] = load();
      body(v, h + sub, h + sub < heads);
      h += step;
    }
  }
}

// D/8 lanes a head row, 16 bytes a lane; a warp takes 32 * 8 / D rows of one kind (key, value or
// query) at a time. Weight, sine and cosine of a token's elements are the same for all its heads:
// element e of a row becomes (x_e A_e + x_partner B_e) * norm factor, with A = w cos and B = -/+ w
// of the partner * sin, in tables that a block builds for its `tokens` tokens. The tables are
// turned (element 8 lane + i at row i, column lane), so that lanes read words side by side.
template <int D>
__global__ void __launch_bounds__(32 * kFewWarps, 4) qkv_prep_kernel(const QkvPrepArgs a, int tokens) {
  MOE_PDL_PROLOGUE();
  constexpr int L = D / 8;      // lanes of a row
  constexpr int RPW = 32 / L;   // rows of a warp
  constexpr int NT = kManyWarps;
  const int threads = blockDim.x;
  __shared__ __align__(16) double s_ka[NT][D], s_kb[NT][D];
  __shared__ __align__(16) float s_qa[NT][D], s_qb[NT][D];
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, a.T - t0);
  const int half = a.rot / 2;
  const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31, lane = wl % L, sub = wl / L, e0 = lane * 8;
  auto at_k = [](int e) { return (e & 7) * L + (e >> 3); };
  auto at_q = [](int e) { return (((e & 7) >> 1) * L + (e >> 3)) * 2 + (e & 1); };
  for (int i = threadIdx.x; i < nt * half; i += threads) {
    const int t = i / half, p = i - t * half;
    const int lo = a.interleaved ? 2 * p : p, hi = a.interleaved ? 2 * p + 1 : p + half;
    double sn, cs;
    sincos(whole_turns_off((double)a.positions[t0 + t] * (double)a.inv_freq[p]), &sn, &cs);
    sn *= a.rot_scale;
    cs *= a.rot_scale;
    if (a.Hq) {
      const double wl = a.q_weight ? (double)a.q_weight[lo] : 1.0, wh = a.q_weight ? (double)a.q_weight[hi] : 1.0;
      s_qa[t][at_q(lo)] = (float)(wl * cs);
      s_qa[t][at_q(hi)] = (float)(wh * cs);
      s_qb[t][at_q(lo)] = (float)(-wh * sn);
      s_qb[t][at_q(hi)] = (float)(wl * sn);
    }
    if (a.Hk) {
      const double wl = a.k_weight ? (double)a.k_weight[lo] : 1.0, wh = a.k_weight ? (double)a.k_weight[hi] : 1.0;
      s_ka[t][at_k(lo)] = wl * cs;
      s_ka[t][at_k(hi)] = wh * cs;
      s_kb[t][at_k(lo)] = -wh * sn * kUp;
      s_kb[t][at_k(hi)] = wl * sn * kUp;
    }
  }
  const int rest = D - a.rot;  // elements that are not turned
  for (int i = threadIdx.x; i < nt * rest; i += threads) {
    const int t = i / rest, e = a.rot + i - t * rest;
    if (a.Hq) s_qa[t][at_q(e)] = a.q_weight ? a.q_weight[e] : 1.0f;
    if (a.Hk) s_ka[t][at_k(e)] = a.k_weight ? (double)a.k_weight[e] : 1.0;
  }
  __syncthreads();
  // the partner of a half-split pair sits half a rotation away; of an interleaved one, beside it
  const bool turned = e0 < a.rot, hop = !a.interleaved && half;
  const int from_lane = (wl - lane) + (!turned ? lane : e0 < half ? lane + half / 8 : lane - half / 8);
  auto partner = [&](const uint4& p) {
    return make_uint4(__shfl_sync(0xffffffffu, p.x, from_lane), __shfl_sync(0xffffffffu, p.y, from_lane),
                      __shfl_sync(0xffffffffu, p.z, from_lane), __shfl_sync(0xffffffffu, p.w, from_lane));
  };
  auto beside = [](const uint4& p) {
    return make_uint4(__funnelshift_l(p.x, p.x, 16), __funnelshift_l(p.y, p.y, 16), __funnelshift_l(p.z, p.z, 16),
                      __funnelshift_l(p.w, p.w, 16));
  };
  // this warp's token, and its share of the token's rows
  const bool many = tokens > 1;
  const int t = many ? warp : 0, tok = t0 + t;
  if (t >= nt) return;
  const int step = RPW * (many ? 1 : threads / 32);
  // (with a block to a token the kinds start at different warps, to keep all of them busy)
  const int nk = (a.Hk + RPW - 1) / RPW, nv = (a.Hv + RPW - 1) / RPW;
  auto first = [&](int before) { return many ? 0 : ((warp - before) & (kFewWarps - 1)) * RPW; };
  int64_t cache_row = -1;  // the token's cache row of head 0
  if (a.slots) {
    const int slot = a.slots[tok], n_slots = a.cache.n_pages * a.cache.page_size;
    if (slot >= n_slots) atomicMax(a.status, kStatusInvalid);
    if (slot >= 0 && slot < n_slots)
      cache_row = (int64_t)(slot >> a.page_shift) * a.cache.Hkv * a.cache.page_size + (slot & (a.cache.page_size - 1));
  }
  // the quantised write of a lane's 8 elements of a key or value (p: packed bf16)
  auto store = [&](const uint4& p, int h, bool live, const float* tsp, uint8_t* codes, uint8_t* scales) {
    uint32_t m = (p.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, p.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, p.z & 0x7FFF7FFFu);
    m = __vmaxu2(m, p.w & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (m > 0x7F80u) {  // NaN: the largest of the numbers beside it
      float top = 0.0f, v[8];
      unpack8(p, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
      m = __float_as_uint(fmaxf(top, __shfl_xor_sync(3u << (wl & ~1), top, 1))) >> 16;
    }
    if (!live || cache_row < 0) return;
    const float ts = tsp ? tsp[h] : 1.0f;
    uint32_t c;
    const uint32_t s = quantize_half16(p, bf16_to_f32(m), ts, __frcp_rn(ts), &c);
    const int64_t row = cache_row + (int64_t)h * a.cache.page_size;
    *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + e0 / 2) = c;
    if ((lane & 1) == 0) scales[row * (D / 16) + e0 / 16] = (uint8_t)s;
  };

  // ---- keys, in float64
  if (a.Hk) each_row<2>(a.k + tok * a.k_stride, a.Hk, first(0), sub, step, D, e0, [&](uint4 p, int h, bool live) {
    const uint4 pp = hop ? partner(p) : beside(p);
    uint32_t m = __vmaxu2(__vmaxu2(p.x & 0x7FFF7FFFu, p.y & 0x7FFF7FFFu), __vmaxu2(p.z & 0x7FFF7FFFu, p.w & 0x7FFF7FFFu));
    if (__any_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16) >= 0x7F80u)) {
      // infinities or NaN in one of the warp's rows (which hold the partners too): the same, converted as
      // what they are, in short code
      auto element = [](const uint4& w, int i) { return bf16_to_f64(i & 4 ? (i & 2 ? w.w : w.z) : (i & 2 ? w.y : w.x), i & 1); };
      double rs = 1.0;
      if (a.k_weight) {
        double ss = 0.0;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) ss = fma(element(p, i), element(p, i), ss);
#pragma unroll 1
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = norm_factor(ss, D, a.eps);
      }
      if (a.k_weight || turned) {
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          double z = element(p, i) * s_ka[t][i * L + lane];
          if (turned) z = fma(element(pp, i) * (1.0 / kUp), s_kb[t][i * L + lane], z);
          // in at the top of y, the others 16 bits down
          y = make_uint4(__funnelshift_r(y.x, y.y, 16), __funnelshift_r(y.y, y.z, 16), __funnelshift_r(y.z, y.w, 16),
                         __funnelshift_r(y.w, pack_bf16((float)(z * rs), 0.0f), 16));
        }
        p = y;
      }
    } else if (a.k_weight || turned) {
      uint32_t x[4] = {p.x, p.y, p.z, p.w};
      const uint32_t xp[4] = {pp.x, pp.y, pp.z, pp.w};
      double v[8], rs = 1.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = widen(x[i >> 1], i & 1) * kUp;
      if (a.k_weight) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma(v[i], v[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = norm_factor(ss, D, a.eps);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double z = v[i] * s_ka[t][i * L + lane];
        if (turned) z = fma(widen(xp[i >> 1], i & 1), s_kb[t][i * L + lane], z);
        v[i] = z * rs;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = pack_bf16((float)v[2 * i], (float)v[2 * i + 1]);
      p = make_uint4(x[0], x[1], x[2], x[3]);
    }
    if (live && a.k_out) *reinterpret_cast<uint4*>(a.k_out + ((int64_t)tok * a.Hk + h) * D + e0) = p;
    if (a.slots) store(p, h, live, a.cache.k_ts, a.cache.k_codes, a.cache.k_scales);
  });

  // ---- values
  if (a.Hv) each_row<2>(a.v + tok * a.v_stride, a.Hv, first(nk), sub, step, D, e0, [&](const uint4& p, int h, bool live) {
    store(p, h, live, a.cache.v_ts, a.cache.v_codes, a.cache.v_scales);
  });

  // ---- queries, in float32, two elements an instruction
  if (a.Hq) each_row<2>(a.q + tok * a.q_stride, a.Hq, first(nk + nv), sub, step, D, e0, [&](const uint4& p, int h, bool live) {
    uint64_t y[4];
    unpack8x2(p, y);
    float rs = 1.0f;
    float up = 1.0f;
    if (a.q_weight) {
      uint64_t s2 = mul2(y[0], y[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s2 = fma2(y[i], y[i], s2);
      float sa, sb;
      unpack2(s2, sa, sb);
      float ss = sa + sb;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      rs = rsqrtf(ss * (1.0f / D) + (float)a.eps);
      const bool far = !(ss < 1e36f && (ss > 1e-30f || a.eps > 1e-25)) && live;  // squares near the ends of float32's range
      if (__any_sync(0xffffffffu, far)) {  // once more, 2^100 larger or smaller
        if (far) up = ss > 1.0f ? 0x1p-100f : 0x1p100f;
        const uint64_t u2 = pack2(up, up);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], u2);
        s2 = mul2(y[0], y[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = fma2(y[i], y[i], s2);
        unpack2(s2, sa, sb);
        ss = sa + sb;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss * (1.0f / D) + (float)a.eps * up * up);
      }
    }
    const uint4 pp = hop ? partner(p) : beside(p);
    uint64_t q[4];
    unpack8x2(pp, q);
    if (up != 1.0f) {
      const uint64_t u2 = pack2(up, up);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = mul2(q[i], u2);
    }
    const uint64_t* ta = reinterpret_cast<const uint64_t*>(s_qa[t]) + lane;
    const uint64_t* tb = reinterpret_cast<const uint64_t*>(s_qb[t]) + lane;
    const uint64_t r2 = pack2(rs, rs);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = mul2(y[i], ta[i * L]);
      if (turned) y[i] = fma2(q[i], tb[i * L], y[i]);
      float lo, hi;
      unpack2(mul2(y[i], r2), lo, hi);
      o[i] = pack_bf16(lo, hi);
    }
    if (live)
      *reinterpret_cast<uint4*>(a.q_out + ((int64_t)tok * a.Hq + h) * D + e0) = make_uint4(o[0], o[1], o[2], o[3]);
  });
}

// 8 elements a thread and output: 4 bytes of codes and the block's scale -> one 16-byte store
// (bf16) or two (float32), of the key and the value at once. A thread keeps its head and place
// and walks over the rows, four at a time, so that their loads are under way together, and reads the
// slots of the next four before (6 us less). Bound by the bytes written: 65536 rows of 2 heads of 256
// as bf16, 33.5 us (5.1 TB/s, launch included), as float32 81 us (3.8 TB/s).
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvCacheArgs c, int page_shift, const int32_t* slots,
                                                      int64_t n, void* k_out, void* v_out,
                                                      int32_t* status) {
  MOE_PDL_PROLOGUE();
  constexpr int L = D / 8, U = 4;
  const int X = c.Hkv * L;                      // threads of a row
  const int per = X < 256 ? 256 / X : 1;        // rows of a block at a time
  const int in = threadIdx.x / X;               // which of them
  if (in >= per) return;
  const int n_slots = c.n_pages * c.page_size;
  const int64_t step = (int64_t)gridDim.x * per;
  for (int x = threadIdx.x - in * X; x < X; x += 256) {
    const int h = x / L, lane = x % L;
    const float kts = c.k_ts ? c.k_ts[h] : 1.0f, vts = c.v_ts ? c.v_ts[h] : 1.0f;
    int next[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t r = (int64_t)blockIdx.x * per + in + i * step;
      next[i] = r < n ? slots[r] : -1;
    }
    for (int64_t r0 = (int64_t)blockIdx.x * per + in; r0 < n; r0 += step * U) {
      int64_t row[U];
      uint32_t w[2][U], s[2][U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int slot = next[i];
        const int64_t r = r0 + (i + U) * step;
        next[i] = r < n ? slots[r] : -1;
        if (slot >= n_slots) atomicMax(status, kStatusInvalid);
        row[i] = slot < 0 || slot >= n_slots
                     ? -1
                     : ((int64_t)(slot >> page_shift) * c.Hkv + h) * c.page_size + (slot & (c.page_size - 1));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t at = row[i] < 0 ? 0 : row[i];
        w[0][i] = k_out ? *reinterpret_cast<const uint32_t*>(c.k_codes + at * (D / 2) + lane * 4) : 0u;
        s[0][i] = k_out ? c.k_scales[at * (D / 16) + lane / 2] : 0u;
        w[1][i] = v_out ? *reinterpret_cast<const uint32_t*>(c.v_codes + at * (D / 2) + lane * 4) : 0u;
        s[1][i] = v_out ? c.v_scales[at * (D / 16) + lane / 2] : 0u;
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        void* out = side ? v_out : k_out;
        if (!out) continue;
        const float ts = side ? vts : kts;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int64_t r = r0 + i * step;
          if (r >= n) break;
          const float sc = row[i] < 0 ? 0.0f : __half2float(__ushort_as_half((unsigned short)e4m3x2_to_f16x2(s[side][i])));  // (0x7F and 0xFF are NaN)
          uint32_t f[4];
          e2m1x8_to_f16x2x4(row[i] < 0 ? 0u : w[side][i], f);
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&f[j]));
            v[2 * j] = __fmul_rn(g.x * sc, ts);  // e2m1 * e4m3 is exact
            v[2 * j + 1] = __fmul_rn(g.y * sc, ts);
          }
          const int64_t j = r * X + x;
          if (F32) {
            float4* dst = reinterpret_cast<float4*>(out) + j * 2;
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            reinterpret_cast<uint4*>(out)[j] =
                make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_qkv_prep(const QkvPrepArgs& a, int D, int num_sms, cudaStream_t st) {
  const int tokens = a.T > 4 * num_sms ? kManyWarps : 1;
  const dim3 grid((a.T + tokens - 1) / tokens), block(32 * (tokens > 1 ? kManyWarps : kFewWarps));
  if (D == 64) return launch_pdl(qkv_prep_kernel<64>, grid, block, 0, st, a, tokens);
  if (D == 128) return launch_pdl(qkv_prep_kernel<128>, grid, block, 0, st, a, tokens);
  return launch_pdl(qkv_prep_kernel<256>, grid, block, 0, st, a, tokens);
}

template <int D>
static cudaError_t launch_kv_read_d(const KvCacheArgs& c, const int32_t* slots, int64_t n, void* k, void* v, bool f32,
                                    int32_t* status, int num_sms, cudaStream_t st) {
  const int X = c.Hkv * (D / 8), per = X < 256 ? 256 / X : 1;
  // a block for every `per` rows while that is few; then as many as are resident, each of which walks,
  // four rows at a time (8 a multiprocessor, in two waves, took 2 us more)
  const int64_t want = (n + per - 1) / per, most = (int64_t)num_sms * 4;
  const dim3 grid((unsigned)(want < most ? want : most)), block(256);
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  if (f32) return launch_pdl(kv_read_kernel<D, true>, grid, block, 0, st, c, shift, slots, n, k, v, status);
  return launch_pdl(kv_read_kernel<D, false>, grid, block, 0, st, c, shift, slots, n, k, v, status);
}

cudaError_t launch_kv_read(const KvCacheArgs& c, int D, const int32_t* slots, int64_t n, void* k, void* v, bool f32,
                           int32_t* status, int num_sms, cudaStream_t st) {
  if (D == 64) return launch_kv_read_d<64>(c, slots, n, k, v, f32, status, num_sms, st);
  if (D == 128) return launch_kv_read_d<128>(c, slots, n, k, v, f32, status, num_sms, st);
  return launch_kv_read_d<256>(c, slots, n, k, v, f32, status, num_sms, st);
}

}  // namespace moe

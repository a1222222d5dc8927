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
// Bound by HBM bytes for many tokens (per token: Hq + 2 Hkv rows of 2D bytes read, Hq rows
// written, 9/16 byte per cached element), with the keys' float64 conversions (a quarter of the
// rate of other float64 steps) next; for a decode step by launch latency and the float64 sine
// and cosine.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepTokens = 4;  // tokens of a block when there are many: 64 pairs each fill its threads

// Two lanes hold a block of 16 (8 elements each); amax is the block's, signs the sign bits of the
// elements where their codes have them. The codes of quantize_block16 (common.cuh): E2M1 of the
// correctly rounded quotients x / denom. Those come from one reciprocal per block by Markstein's
// theorem (P. Markstein, IBM J. Res. Dev. 34, 1990): with y the correctly rounded 1 / d,
// q = x y, r = x - q d (exact in a fused step), q + r y is the correctly rounded x / d, unless
// d's significand is all ones, or a step over- or underflows. Blocks where that could be are
// divided (an underflow of x y is none: the code is 0 either way).
MOE_DEV uint32_t quantize_half16(const float (&v)[8], uint32_t signs, float amax, float ts, uint32_t* codes) {
  const uint32_t s = f32_to_e4m3_sat(__fdiv_rn(__fdiv_rn(amax, kE2M1Max), ts));
  const float sval = e4m3_to_f32(s);
  *codes = 0;
  if (sval == 0.0f) return s;
  const float d = __fmul_rn(sval, ts);
  float q[8];
  if (d > 0x1p-60f && d < 0x1p60f && amax < 0x1p60f && (__float_as_uint(d) & 0x7FFFFFu) != 0x7FFFFFu) {
    const float y = __frcp_rn(d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = fabsf(v[i]), q0 = __fmul_rn(x, y);
      q[i] = __fmaf_rn(__fmaf_rn(-q0, d, x), y, q0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fabsf(__fdiv_rn(v[i], d));
  }
  uint32_t c = signs;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t r;
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tcvt.u32.u8 %0, q;\n\t}" : "=r"(r) : "f"(q[2 * i]), "f"(q[2 * i + 1]));
    c |= r << (8 * i);
  }
  *codes = c;
  return s;
}

// sign bits of 8 packed bf16 values, at bit 4 i + 3 for element i
MOE_DEV uint32_t sign_bits(const uint4& p) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
  uint32_t s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) s |= (((w[i] >> 12) & 0x8u) | ((w[i] >> 24) & 0x80u)) << (8 * i);
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

// (weights need 4-byte alignment only)
MOE_DEV float4 ldg4(const float* p) { return make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3)); }

MOE_DEV uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A row's norm factor from its sum of squares: one Newton step in float64 from the float32
// reciprocal square root (2^-22 off) leaves 2^-43.
MOE_DEV double norm_factor(double ss, int D, double eps) {
  const double x = ss / D + eps;
  if (!(x > 1e-30 && x < 1e30)) return 1.0 / sqrt(x);
  const double y = (double)rsqrtf((float)x);
  return y * (1.5 - 0.5 * x * y * y);
}

// D/8 lanes a head row, 16 bytes a lane; a warp takes 32 * 8 / D rows of one kind (key, value or
// query) at a time. A block takes `tokens` tokens and all their rows, so that the sines and
// cosines of a token are computed once for all its heads.
template <int D>
__global__ void __launch_bounds__(kPrepThreads) qkv_prep_kernel(const QkvPrepArgs a, int tokens) {
  MOE_PDL_PROLOGUE();
  constexpr int L = D / 8;      // lanes of a row
  constexpr int RPW = 32 / L;   // rows of a warp
  __shared__ double s_cos[kPrepTokens][D / 2], s_sin[kPrepTokens][D / 2];
  __shared__ float s_cosf[kPrepTokens][D / 2], s_sinf[kPrepTokens][D / 2];
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, a.T - t0);
  const int half = a.rot / 2;
  const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31, lane = wl % L, e0 = lane * 8;
  // a block's rows: units of RPW rows, keys first (they take longest), then values, then queries
  const int nk = (nt * a.Hk + RPW - 1) / RPW, nv = (nt * a.Hv + RPW - 1) / RPW, nq = (nt * a.Hq + RPW - 1) / RPW;
  const int units = nk + nv + nq;
  auto source = [&](int u, int* kind, int* t, int* h, bool* live) -> uint4 {
    *kind = u < nk ? 1 : u < nk + nv ? 2 : 0;
    const int heads = *kind == 1 ? a.Hk : *kind == 2 ? a.Hv : a.Hq;
    const int row = (u - (*kind == 1 ? 0 : *kind == 2 ? nk : nk + nv)) * RPW + wl / L;
    *live = u < units && row < nt * heads;
    *t = *live ? row / heads : 0;
    *h = *live ? row - *t * heads : 0;
    const uint16_t* x = *kind == 1 ? a.k : *kind == 2 ? a.v : a.q;
    const int64_t stride = *kind == 1 ? a.k_stride : *kind == 2 ? a.v_stride : a.q_stride;
    return *live ? *reinterpret_cast<const uint4*>(x + (int64_t)(t0 + *t) * stride + (int64_t)*h * D + e0)
                 : make_uint4(0u, 0u, 0u, 0u);
  };
  int kind, t, h, kind_n, t_n, h_n;
  bool live, live_n;
  uint4 p_n = source(warp, &kind_n, &t_n, &h_n, &live_n);  // a unit ahead
  for (int i = threadIdx.x; i < nt * half; i += kPrepThreads) {
    const int ti = i / half, p = i - ti * half;
    double sn, cs;
    sincos((double)a.positions[t0 + ti] * (double)a.inv_freq[p], &sn, &cs);
    s_cos[ti][p] = cs * a.rot_scale;
    s_sin[ti][p] = sn * a.rot_scale;
    s_cosf[ti][p] = (float)(cs * a.rot_scale);
    s_sinf[ti][p] = (float)(sn * a.rot_scale);
  }
  __syncthreads();
  const int n_slots = a.cache.n_pages * a.cache.page_size;
  // the partner of a half-split pair sits R/16 lanes away
  const int hop = half / 8;
  const bool lower = e0 < half, turned = e0 < a.rot;
  const int from = (lower ? lane + hop : lane - hop) & (L - 1), from_lane = (wl - lane) + from;
  const int pe = from * 8, p0 = a.interleaved ? e0 / 2 : lower ? e0 : e0 - half;
#pragma unroll 1
  for (int u = warp; u < units; u += kPrepThreads / 32) {
    uint4 p = p_n;
    kind = kind_n; t = t_n; h = h_n; live = live_n;
    p_n = source(u + kPrepThreads / 32, &kind_n, &t_n, &h_n, &live_n);
    float y[8];
    unpack8(p, y);
    float q[8];
    if (kind != 2 && !a.interleaved && half) {
      uint4 pp;
      pp.x = __shfl_sync(0xffffffffu, p.x, from_lane);
      pp.y = __shfl_sync(0xffffffffu, p.y, from_lane);
      pp.z = __shfl_sync(0xffffffffu, p.z, from_lane);
      pp.w = __shfl_sync(0xffffffffu, p.w, from_lane);
      unpack8(pp, q);
    }
    if (kind == 0) {
      // ---- a query, in float32
      if (a.q_weight) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        float rs = 1.0f / sqrtf(ss / D + (float)a.eps);
        const bool far = !(ss < 1e36f && ss > 1e-30f);  // squares near the ends of float32's range
        if (__any_sync(0xffffffffu, far)) {
          double sd = 0.0;
#pragma unroll
          for (int i = 0; i < 8; ++i) sd = fma((double)y[i], (double)y[i], sd);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, o);
          if (far) {
            const double r = norm_factor(sd, D, a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y[i] = (float)(y[i] * r);
              if (turned && !a.interleaved) q[i] = (float)(q[i] * r);
            }
            rs = 1.0f;
          }
        }
        const float4 w0 = ldg4(a.q_weight + e0), w1 = ldg4(a.q_weight + e0 + 4);
        const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= rs * w[i];
        if (turned && !a.interleaved) {
          const float4 x0 = ldg4(a.q_weight + pe), x1 = ldg4(a.q_weight + pe + 4);
          const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] *= rs * x[i];
        }
      }
      if (turned) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float c = s_cosf[t][p0 + i], s = s_sinf[t][p0 + i], lo = y[2 * i], hi = y[2 * i + 1];
            y[2 * i] = lo * c - hi * s;
            y[2 * i + 1] = hi * c + lo * s;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float c = s_cosf[t][p0 + i], s = s_sinf[t][p0 + i];
            y[i] = lower ? y[i] * c - q[i] * s : y[i] * c + q[i] * s;
          }
        }
      }
      if (live)
        *reinterpret_cast<uint4*>(a.q_out + ((int64_t)(t0 + t) * a.Hq + h) * D + e0) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      continue;
    }
    if (kind == 1) {
      // ---- a key, in float64
      double rs = 1.0;
      if (a.k_weight) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fma((double)y[i], (double)y[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = norm_factor(ss, D, a.eps);
      }
      double z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = a.k_weight ? (double)y[i] * rs * (double)__ldg(a.k_weight + e0 + i) : (double)y[i];
      if (turned) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const double c = s_cos[t][p0 + i], s = s_sin[t][p0 + i], lo = z[2 * i], hi = z[2 * i + 1];
            z[2 * i] = lo * c - hi * s;
            z[2 * i + 1] = hi * c + lo * s;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const double o = a.k_weight ? (double)q[i] * rs * (double)__ldg(a.k_weight + pe + i) : (double)q[i];
            const double c = s_cos[t][p0 + i], s = s_sin[t][p0 + i];
            z[i] = lower ? z[i] * c - o * s : z[i] * c + o * s;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (float)z[i];
      p = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      if (live && a.k_out) *reinterpret_cast<uint4*>(a.k_out + ((int64_t)(t0 + t) * a.Hk + h) * D + e0) = p;
      if (!a.slots) continue;
      unpack8(p, y);
    }
    // ---- the quantised write of a key or value
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(y[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (!live) continue;
    const int slot = a.slots[t0 + t];
    if (slot < 0 || slot >= n_slots) {
      if (slot >= 0) atomicExch(a.status, kStatusInvalid);
      continue;
    }
    const float* tsp = kind == 1 ? a.cache.k_ts : a.cache.v_ts;
    uint32_t c;
    const uint32_t s = quantize_half16(y, sign_bits(p), amax, tsp ? tsp[h] : 1.0f, &c);
    const int page = slot >> a.page_shift, off = slot & (a.cache.page_size - 1);
    const int64_t row = ((int64_t)page * a.cache.Hkv + h) * a.cache.page_size + off;
    uint8_t* codes = kind == 1 ? a.cache.k_codes : a.cache.v_codes;
    uint8_t* scales = kind == 1 ? a.cache.k_scales : a.cache.v_scales;
    *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + e0 / 2) = c;
    if ((lane & 1) == 0) scales[row * (D / 16) + e0 / 16] = (uint8_t)s;
  }
}

// 8 elements a thread and output: 4 bytes of codes and the block's scale -> one 16-byte store
// (bf16) or two (float32), of the key and the value at once. A thread keeps its head and place
// and walks over the rows, four at a time, so that their loads are under way together. Bound by
// the bytes written.
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvCacheArgs c, int page_shift, const int32_t* __restrict__ slots,
                                                      int64_t n, void* __restrict__ k_out, void* __restrict__ v_out,
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
    for (int64_t r0 = (int64_t)blockIdx.x * per + in; r0 < n; r0 += step * U) {
      int64_t row[U];
      uint32_t w[2][U], s[2][U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t r = r0 + i * step;
        const int slot = r < n ? slots[r] : -1;
        if (slot >= n_slots) atomicExch(status, kStatusInvalid);
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
          const float sc = row[i] < 0 ? 0.0f : e4m3_to_f32(s[side][i]);
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
  // few tokens: a block each, so that all of them run at once
  const int tokens = a.T > 8 * num_sms ? kPrepTokens : 1;
  const dim3 grid((a.T + tokens - 1) / tokens), block(kPrepThreads);
  if (D == 64) return launch_pdl(qkv_prep_kernel<64>, grid, block, 0, st, a, tokens);
  if (D == 128) return launch_pdl(qkv_prep_kernel<128>, grid, block, 0, st, a, tokens);
  return launch_pdl(qkv_prep_kernel<256>, grid, block, 0, st, a, tokens);
}

template <int D>
static cudaError_t launch_kv_read_d(const KvCacheArgs& c, const int32_t* slots, int64_t n, void* k, void* v, bool f32,
                                    int32_t* status, int num_sms, cudaStream_t st) {
  const int X = c.Hkv * (D / 8), per = X < 256 ? 256 / X : 1;
  // a block for every `per` rows while that is few; then each walks, four rows at a time
  const int64_t want = (n + per - 1) / per, most = (int64_t)num_sms * 8;
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

// Writing and reading the paged NVFP4 key/value cache, and the norm and rotation of queries
// and keys that goes before the write.
//
// Per head row x of D elements:  y = x / sqrt(mean(x^2) + eps) * w, then the first R elements
// rotated in pairs by pos * f_p (cos and sin times a factor m), rounded to float32 and then to
// bf16. A cached key is the NVFP4 quantisation of that bf16 row, so the fused write stores
// exactly what the norm/rotation call followed by nvfp4_quantize_act would.
//
// Everything before the rounding to bf16 is in float64: a row that differs by one float32
// rounding can land on the other side of a bf16 step, that on the other side of an E2M1 step,
// and the stored value is then off by up to half of itself.
//
// Bound by HBM bytes for many tokens (per token: Hq + 2 Hkv rows of 2D bytes read, Hq rows
// written, 9/16 byte per cached element); for a decode step by launch latency and the float64
// sine and cosine.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kPrepTokens = 4;  // tokens of a block when there are many: 64 pairs each fill its threads

// Two lanes hold a block of 16 (8 elements each); amax is the block's. The steps of
// quantize_block16 (common.cuh), which the cache's codes have to equal.
MOE_DEV uint32_t quantize_half16(const float (&v)[8], float amax, float ts, uint32_t* codes) {
  const uint32_t s = f32_to_e4m3_sat(__fdiv_rn(__fdiv_rn(amax, kE2M1Max), ts));
  const float sval = e4m3_to_f32(s);
  uint32_t c = 0;
  if (sval != 0.0f) {
    const float denom = __fmul_rn(sval, ts);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c |= f32x2_to_e2m1x2(__fdiv_rn(v[2 * i], denom), __fdiv_rn(v[2 * i + 1], denom)) << (8 * i);
  }
  *codes = c;
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

// One group of D/8 lanes per head row, 16 bytes a lane; a block takes `tokens` tokens and all
// their rows, so that the sines and cosines of a token are computed once for all its heads.
template <int D>
__global__ void __launch_bounds__(kPrepThreads) qkv_prep_kernel(const QkvPrepArgs a, int tokens) {
  MOE_PDL_PROLOGUE();
  constexpr int L = D / 8;               // lanes of a row
  constexpr int G = kPrepThreads / L;    // rows in flight in a block
  __shared__ double s_cos[kPrepTokens][D / 2], s_sin[kPrepTokens][D / 2];
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, a.T - t0);
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < nt * half; i += kPrepThreads) {
    const int t = i / half, p = i - t * half;
    double sn, cs;
    sincos((double)a.positions[t0 + t] * (double)a.inv_freq[p], &sn, &cs);
    s_cos[t][p] = cs * a.rot_scale;
    s_sin[t][p] = sn * a.rot_scale;
  }
  __syncthreads();
  const int lane = threadIdx.x % L, e0 = lane * 8;
  const int rows = a.Hq + a.Hk + a.Hv;
  const int n_slots = a.cache.n_pages * a.cache.page_size;
  // every lane of a warp takes the same number of turns (the shuffles below name all lanes)
  const int total = nt * rows;
  for (int base = 0; base < total; base += G) {
    const int item = base + threadIdx.x / L;
    const bool live = item < total;
    const int t = live ? item / rows : 0, r = live ? item - t * rows : 0;
    const int kind = r < a.Hq ? 0 : r < a.Hq + a.Hk ? 1 : 2;  // query, key, value
    const int h = kind == 0 ? r : kind == 1 ? r - a.Hq : r - a.Hq - a.Hk;
    const uint16_t* src = kind == 0   ? a.q + (int64_t)(t0 + t) * a.q_stride
                          : kind == 1 ? a.k + (int64_t)(t0 + t) * a.k_stride
                                      : a.v + (int64_t)(t0 + t) * a.v_stride;
    uint4 p = make_uint4(0u, 0u, 0u, 0u);
    if (live) p = *reinterpret_cast<const uint4*>(src + (int64_t)h * D + e0);
    float y[8];
    unpack8(p, y);
    const float* w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fma((double)y[i], (double)y[i], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // the partner of a half-split pair sits R/16 lanes away
    const int hop = half / 8;
    const bool lower = e0 < half;
    const int base_lane = (threadIdx.x & 31) - lane;
    const int from = (lower ? lane + hop : lane - hop) & (L - 1);
    uint4 pp;
    pp.x = __shfl_sync(0xffffffffu, p.x, base_lane + from);
    pp.y = __shfl_sync(0xffffffffu, p.y, base_lane + from);
    pp.z = __shfl_sync(0xffffffffu, p.z, base_lane + from);
    pp.w = __shfl_sync(0xffffffffu, p.w, base_lane + from);
    if (kind < 2) {
      const double rs = w ? 1.0 / sqrt(ss / D + a.eps) : 1.0;
      double z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = w ? (double)y[i] * rs * (double)__ldg(w + e0 + i) : (double)y[i];
      if (e0 < a.rot) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const double c = s_cos[t][e0 / 2 + i], s = s_sin[t][e0 / 2 + i];
            const double lo = z[2 * i], hi = z[2 * i + 1];
            z[2 * i] = lo * c - hi * s;
            z[2 * i + 1] = hi * c + lo * s;
          }
        } else {
          float q[8];
          unpack8(pp, q);
          const int pe = from * 8, p0 = lower ? e0 : e0 - half;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const double o = w ? (double)q[i] * rs * (double)__ldg(w + pe + i) : (double)q[i];
            const double c = s_cos[t][p0 + i], s = s_sin[t][p0 + i];
            z[i] = lower ? z[i] * c - o * s : z[i] * c + o * s;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (float)z[i];
      p = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
      uint16_t* dst = kind == 0 ? a.q_out : a.k_out;
      if (live && dst)
        *reinterpret_cast<uint4*>(dst + ((int64_t)(t0 + t) * (kind == 0 ? a.Hq : a.Hk) + h) * D + e0) = p;
      unpack8(p, y);
    }
    if (a.slots) {
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(y[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      if (live && kind > 0) {
        const int slot = a.slots[t0 + t];
        if (slot >= n_slots) atomicExch(a.status, kStatusInvalid);
        if (slot >= 0 && slot < n_slots) {
          const float* tsp = kind == 1 ? a.cache.k_ts : a.cache.v_ts;
          uint32_t c;
          const uint32_t s = quantize_half16(y, amax, tsp ? tsp[h] : 1.0f, &c);
          const int page = slot / a.cache.page_size, off = slot - page * a.cache.page_size;
          const int64_t row = ((int64_t)page * a.cache.Hkv + h) * a.cache.page_size + off;
          uint8_t* codes = kind == 1 ? a.cache.k_codes : a.cache.v_codes;
          uint8_t* scales = kind == 1 ? a.cache.k_scales : a.cache.v_scales;
          *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + e0 / 2) = c;
          if ((lane & 1) == 0) scales[row * (D / 16) + e0 / 16] = (uint8_t)s;
        }
      }
    }
  }
}

// 8 elements a thread: 4 bytes of codes and the block's scale -> one 16-byte store (bf16) or
// two (float32). Bound by the bytes written.
template <int D, bool F32>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvCacheArgs c, const int32_t* __restrict__ slots, int64_t n,
                                                      void* __restrict__ k_out, void* __restrict__ v_out,
                                                      int32_t* status) {
  MOE_PDL_PROLOGUE();
  constexpr int L = D / 8;
  const int n_slots = c.n_pages * c.page_size;
  const int64_t per = n * c.Hkv * L;  // threads of one of the two outputs
  const int sides = (k_out ? 1 : 0) + (v_out ? 1 : 0);
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < per * sides;
       i += (int64_t)gridDim.x * blockDim.x) {
    const bool is_v = !k_out || i >= per;
    const int64_t j = i >= per ? i - per : i;
    const int lane = (int)(j % L);
    const int64_t rh = j / L;  // row * Hkv + head
    const int64_t r = rh / c.Hkv;
    const int h = (int)(rh - r * c.Hkv);
    const int slot = slots[r];
    uint32_t w = 0;
    float s = 0.0f;
    if (slot >= n_slots) atomicExch(status, kStatusInvalid);
    if (slot >= 0 && slot < n_slots) {
      const int page = slot / c.page_size, off = slot - page * c.page_size;
      const int64_t row = ((int64_t)page * c.Hkv + h) * c.page_size + off;
      w = *reinterpret_cast<const uint32_t*>((is_v ? c.v_codes : c.k_codes) + row * (D / 2) + lane * 4);
      s = e4m3_to_f32((is_v ? c.v_scales : c.k_scales)[row * (D / 16) + lane / 2]);
    }
    const float* tsp = is_v ? c.v_ts : c.k_ts;
    const float ts = tsp ? tsp[h] : 1.0f;
    uint32_t f[4];
    e2m1x8_to_f16x2x4(w, f);
    float x[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[q]));
      x[2 * q] = __fmul_rn(v.x * s, ts);  // e2m1 * e4m3 is exact
      x[2 * q + 1] = __fmul_rn(v.y * s, ts);
    }
    void* out = is_v ? v_out : k_out;
    if (F32) {
      float4* dst = reinterpret_cast<float4*>(out) + j * 2;
      dst[0] = make_float4(x[0], x[1], x[2], x[3]);
      dst[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      reinterpret_cast<uint4*>(out)[j] =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
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
  const int64_t threads = n * c.Hkv * (D / 8) * ((k ? 1 : 0) + (v ? 1 : 0));
  const int64_t want = (threads + 255) / 256, most = (int64_t)num_sms * 32;
  const dim3 grid((unsigned)(want < most ? want : most)), block(256);
  if (f32) return launch_pdl(kv_read_kernel<D, true>, grid, block, 0, st, c, slots, n, k, v, status);
  return launch_pdl(kv_read_kernel<D, false>, grid, block, 0, st, c, slots, n, k, v, status);
}

cudaError_t launch_kv_read(const KvCacheArgs& c, int D, const int32_t* slots, int64_t n, void* k, void* v, bool f32,
                           int32_t* status, int num_sms, cudaStream_t st) {
  if (D == 64) return launch_kv_read_d<64>(c, slots, n, k, v, f32, status, num_sms, st);
  if (D == 128) return launch_kv_read_d<128>(c, slots, n, k, v, f32, status, num_sms, st);
  return launch_kv_read_d<256>(c, slots, n, k, v, f32, status, num_sms, st);
}

}  // namespace moe

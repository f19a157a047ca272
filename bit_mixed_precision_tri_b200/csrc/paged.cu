// Writes into a paged key/value cache: rotary tables with stretched angles,
// QK-Norm + RoPE + append of a batch of rows, and copies of pages.
//
//  * rope_table_scaled_kernel: (cos, sin) of p f_i, f_i = theta^(-2i/rot)
//    under one of four scalings, all in float64, stored as float32 pairs.
//  * paged_append_kernel: per row and head, y = x / sqrt(mean x^2 + eps) * g,
//    the pairs of the first `rot` features turned by the row's angles, fp32,
//    rounded once: fp16, or e4m3 of y / scale clamped to +-448.
//  * copy_pages_kernel: page src[i] of every pool to page dst[i].
#include <cuda_fp8.h>

#include "tri_internal.cuh"

namespace tri {
namespace {

// ---------------------------------------------------------------- rotary table
struct RopeFreq {
  double theta, factor, context, low, high;   // theta already stretched for NTK
  double ramp_a, ramp_b, gain;
  int kind, rot;
};

__device__ double rope_freq(const RopeFreq& r, int i) {
  const double f = pow(r.theta, -2.0 * (double)i / (double)r.rot);
  if (r.kind == TRI_ROPE_LINEAR) return f / r.factor;
  if (r.kind == TRI_ROPE_BANDS) {
    const double turns = r.context * f / 6.283185307179586476925;     // context / wavelength
    if (turns > r.high) return f;
    if (turns < r.low) return f / r.factor;
    const double s = (turns - r.low) / (r.high - r.low);
    return f * ((1.0 - s) / r.factor + s);
  }
  if (r.kind == TRI_ROPE_RAMP) {
    const double t = fmin(fmax(((double)i - r.ramp_a) / (r.ramp_b - r.ramp_a), 0.0), 1.0);
    return f * ((1.0 - t) + t / r.factor);
  }
  return f;
}

__global__ void rope_table_scaled_kernel(float2* __restrict__ cs, int64_t n, RopeFreq r) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= n) return;
  const int half = r.rot / 2;
  const int64_t p = idx / half;
  double s, c;
  sincos((double)p * rope_freq(r, (int)(idx % half)), &s, &c);
  cs[idx] = make_float2((float)(c * r.gain), (float)(s * r.gain));
}

// ---------------------------------------------------------------- append
struct AppendParams {
  const __half* qkv;
  const int *pos, *seq, *table;
  const __half *gq, *gk;
  const float* cs;
  const float *k_scale, *v_scale;
  __half* q_out;
  void *k, *v;
  int64_t qkv_stride, q_stride, table_stride, page_stride, T, cs_rows;
  int H, Hkv, rot, pages, seqs, page_shift, max_pos;
  int tokens_per_cta, head_step;
  float eps;
  bool interleaved;
};

__device__ __forceinline__ uint32_t h2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// eight fp32 values as fp16 (16 bytes) or as e4m3 of value / scale (8 bytes; the
// IEEE quotient, so that the bytes are those of the plain definition)
template <bool FP8>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float (&y)[8], float scale) {
  if constexpr (FP8) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(y[4 * h], scale), __fdiv_rn(y[4 * h + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(y[4 * h + 2], scale), __fdiv_rn(y[4 * h + 3], scale)), __NV_SATFINITE, __NV_E4M3);
      w[h] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + elem) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__half*>(base) + elem) =
        make_uint4(h2_bits(y[0], y[1]), h2_bits(y[2], y[3]), h2_bits(y[4], y[5]), h2_bits(y[6], y[7]));
  }
}

// A group of DH / 8 lanes owns one head: lane l holds features 8l .. 8l + 7
// (one 16-byte load), the sum of squares is a shuffle reduction over the group,
// and the partner of a rotate-half pair sits rot / 16 lanes away (rot is a
// multiple of 16, so lanes rotate whole).  A group keeps its row's angles in
// registers over all heads it takes, and has the loads of four heads in flight.
template <int DH, bool FP8>
__global__ void __launch_bounds__(256)
paged_append_kernel(const AppendParams p) {
  constexpr int LPH = DH / 8, GROUPS = 256 / LPH, U = 4;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPH, grp = threadIdx.x / LPH;
  const int gpt = GROUPS / p.tokens_per_cta;                    // groups per row
  const int64_t t = (int64_t)blockIdx.x * p.tokens_per_cta + grp / gpt;
  const int first = (int)blockIdx.y * gpt + grp % gpt;
  const int nh = p.H + 2 * p.Hkv;
  // the row's place; shuffles below need whole warps, so rows that do not
  // exist stay and do nothing
  int pp = -1, sq = -1, page = -1;
  if (t < p.T) {
    pp = p.pos[t];
    sq = p.seq ? p.seq[t] : (t < p.seqs ? (int)t : -1);
    if (pp < 0 || pp >= p.max_pos || pp >= p.cs_rows || sq < 0 || sq >= p.seqs) pp = -1;
  }
  const bool valid = pp >= 0;
  if (valid) {
    page = p.table[(int64_t)sq * p.table_stride + (pp >> p.page_shift)];
    if (page >= p.pages) page = -1;
  }
  // angles: c and the signed s of own features (the partner's share of each)
  const int hl = p.rot / 16;                                    // lanes of half the rotated features
  const bool rotates = 8 * l < p.rot;
  float c[8], s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  int partner = lane;
  if (rotates && valid) {
    const float4* row = reinterpret_cast<const float4*>(p.cs + (int64_t)pp * p.rot);
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float4 w = row[2 * l + e];                        // pairs 4l + 2e, 4l + 2e + 1
        c[4 * e] = c[4 * e + 1] = w.x, s[4 * e] = -w.y, s[4 * e + 1] = w.y;
        c[4 * e + 2] = c[4 * e + 3] = w.z, s[4 * e + 2] = -w.w, s[4 * e + 3] = w.w;
      }
    } else {
      const int lo = l < hl ? l : l - hl;
      const float sg = l < hl ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 w = row[4 * lo + e];
        c[2 * e] = w.x, s[2 * e] = sg * w.y, c[2 * e + 1] = w.z, s[2 * e + 1] = sg * w.w;
      }
    }
  }
  if (rotates && !p.interleaved) partner = l < hl ? lane + hl : lane - hl;
  uint4 gq = make_uint4(0, 0, 0, 0), gk = gq;
  if (p.gq) {
    gq = reinterpret_cast<const uint4*>(p.gq)[l];
    gk = reinterpret_cast<const uint4*>(p.gk)[l];
  }
  const __half* src = p.qkv + t * p.qkv_stride;
  const int off = pp & ((1 << p.page_shift) - 1);
  for (int b = 0; b < nh; b += U * p.head_step) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = b + u * p.head_step + first;
      raw[u] = valid && j < nh ? __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)j * DH) + l)
                               : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * p.head_step >= nh) break;                     // the same for every lane
      const int j = b + u * p.head_step + first;
      float y[8];
      const __half2* h = reinterpret_cast<const __half2*>(&raw[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(h[e]);
        y[2 * e] = f.x, y[2 * e + 1] = f.y;
      }
      const bool is_v = j >= p.H + p.Hkv;
      if (p.gq) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (!is_v) {
          const float rstd = 1.f / sqrtf(ss / (float)DH + p.eps);
          const __half2* g = reinterpret_cast<const __half2*>(j < p.H ? &gq : &gk);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __half22float2(g[e]);
            y[2 * e] *= rstd * f.x, y[2 * e + 1] *= rstd * f.y;
          }
        }
      }
      float o[8];
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = y[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xFFFFFFFFu, y[e], partner);
      }
      if (!is_v && rotates) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], c[e], o[e] * s[e]);
      }
      if (!valid || j >= nh) continue;
      if (j < p.H) {
        store8<false>(p.q_out, t * p.q_stride + (int64_t)j * DH + 8 * l, y, 1.f);
      } else if (page >= 0) {
        const int kv = is_v ? j - p.H - p.Hkv : j - p.H;
        const int64_t at =
            (int64_t)page * p.page_stride + ((((int64_t)kv << p.page_shift) + off) * DH) + 8 * l;
        const float scale = FP8 ? (is_v ? p.v_scale : p.k_scale)[kv] : 1.f;
        store8<FP8>(is_v ? p.v : p.k, at, y, scale);
      }
    }
  }
}

// ---------------------------------------------------------------- page copies
constexpr int kCopyUnit = 2048;                                 // bytes a warp moves at once: 4 x 16 per lane

__global__ void __launch_bounds__(256)
copy_pages_kernel(uint8_t* __restrict__ pools, int64_t n_pools, int64_t pool_stride, int pages,
                  int64_t page_stride, int64_t page_bytes, const int* __restrict__ src,
                  const int* __restrict__ dst, int64_t n, int64_t units_per_page) {
  const int lane = threadIdx.x & 31;
  const int64_t units = n * n_pools * units_per_page;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t c = u % units_per_page, pl = (u / units_per_page) % n_pools, i = u / units_per_page / n_pools;
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= pages || b < 0 || b >= pages || a == b) continue;
    const int64_t at = c * kCopyUnit + lane * 16;
    const uint8_t* from = pools + pl * pool_stride + a * page_stride + at;
    uint8_t* to = pools + pl * pool_stride + b * page_stride + at;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + 512 * k < page_bytes) v[k] = __ldcs(reinterpret_cast<const uint4*>(from + 512 * k));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + 512 * k < page_bytes) __stcs(reinterpret_cast<uint4*>(to + 512 * k), v[k]);
  }
}

}  // namespace

cudaError_t launch_rope_table_scaled(float2* cs, int64_t Lmax, int64_t rot, double theta,
                                     const tri_rope_scaling* sc, cudaStream_t s) {
  RopeFreq r = {};
  r.theta = theta;
  r.rot = (int)rot;
  r.gain = 1.0;
  r.factor = 1.0;
  if (sc) {
    r.kind = sc->kind;
    r.factor = sc->factor, r.context = sc->context, r.low = sc->low, r.high = sc->high;
    if (sc->kind == TRI_ROPE_NTK) r.theta = theta * pow(sc->factor, (double)rot / (double)(rot - 2));
    if (sc->kind == TRI_ROPE_RAMP) {
      const double two_pi = 6.283185307179586476925;
      auto c = [&](double turns) {
        return (double)rot * log(sc->context / (two_pi * turns)) / (2.0 * log(theta));
      };
      r.ramp_a = fmax(floor(c(sc->high)), 0.0);
      r.ramp_b = fmin(ceil(c(sc->low)), (double)rot - 1.0);
      if (r.ramp_b == r.ramp_a) r.ramp_b = r.ramp_a + 0.001;
      r.gain = 0.1 * log(sc->factor) + 1.0;
    }
  }
  const int64_t n = Lmax * (rot / 2);
  rope_table_scaled_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(cs, n, r);
  return cudaGetLastError();
}

cudaError_t launch_paged_qknorm_rope(const __half* qkv, int64_t qkv_stride, const int* pos, const int* seq,
                                     const __half* gq, const __half* gk, const float* cs, int64_t cs_rows,
                                     int64_t rot, bool interleaved, __half* q_out, int64_t q_stride,
                                     const tri_paged_cache& c, int64_t T, int64_t H, float eps, int sms,
                                     cudaStream_t s) {
  AppendParams p = {};
  p.qkv = qkv, p.pos = pos, p.seq = seq, p.table = c.table, p.gq = gq, p.gk = gk, p.cs = cs;
  p.k_scale = c.k_scale, p.v_scale = c.v_scale, p.q_out = q_out, p.k = c.k, p.v = c.v;
  p.qkv_stride = qkv_stride, p.q_stride = q_stride, p.table_stride = c.table_stride;
  p.page_stride = c.page_stride, p.T = T, p.cs_rows = cs_rows;
  p.H = (int)H, p.Hkv = (int)c.heads, p.rot = (int)rot, p.pages = (int)c.pages;
  p.seqs = (int)c.seqs, p.max_pos = (int)(c.seq_pages * c.page_size), p.eps = eps, p.interleaved = interleaved;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  // Few rows: one head per group and the heads spread over CTAs (latency);
  // many: a row per as many groups as give each about four heads, so that the
  // row's lookups and angles are paid once and four loads are in flight.
  const int groups = (int)(256 * 8 / c.head_dim);
  const int64_t nh = H + 2 * c.heads;
  int gpt = 1;
  while (gpt < groups && gpt * 4 < nh) gpt *= 2;
  int64_t splits = 1;
  if (T * ceil_div(nh, groups) <= 2 * (int64_t)sms) {
    gpt = groups;
    splits = ceil_div(nh, groups);
  }
  p.tokens_per_cta = groups / gpt;
  p.head_step = (int)(gpt * splits);
  const dim3 grid((unsigned)ceil_div(T, p.tokens_per_cta), (unsigned)splits);
  if (c.dtype == TRI_CACHE_E4M3) {
    if (c.head_dim == 128) paged_append_kernel<128, true><<<grid, 256, 0, s>>>(p);
    else paged_append_kernel<64, true><<<grid, 256, 0, s>>>(p);
  } else {
    if (c.head_dim == 128) paged_append_kernel<128, false><<<grid, 256, 0, s>>>(p);
    else paged_append_kernel<64, false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(uint8_t* pools, int64_t n_pools, int64_t pool_stride, int64_t pages,
                              int64_t page_stride, int64_t page_bytes, const int* src, const int* dst,
                              int64_t n, int sms, cudaStream_t s) {
  const int64_t upp = ceil_div(page_bytes, kCopyUnit);
  const int64_t ctas = ceil_div(n * n_pools, 8) < (int64_t(1) << 40) / upp ? ceil_div(n * n_pools * upp, 8)
                                                                             : (int64_t(1) << 40);
  const int64_t most = (int64_t)sms * 8;
  copy_pages_kernel<<<(unsigned)(ctas < most ? ctas : most), 256, 0, s>>>(
      pools, n_pools, pool_stride, (int)pages, page_stride, page_bytes, src, dst, n, upp);
  return cudaGetLastError();
}

}  // namespace tri

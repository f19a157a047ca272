// Writes into a paged key/value cache: rotary tables with stretched angles,
// QK-Norm + RoPE + append of a batch of rows, and copies of pages.
//
//  * rope_table_scaled_kernel: (cos, sin) of p f_i, f_i = theta^(-2i/rot)
//    under one of four scalings, all in float64, stored as float32 pairs.
//  * paged_append_kernel (few rows) and paged_append_stream_kernel (many): per row
//    and head, y = x / sqrt(mean x^2 + eps) * g, the pairs of the first `rot`
//    features turned by the row's angles, fp32, rounded once: fp16, or e4m3 of
//    y / scale clamped to +-448.
//  * copy_pages_kernel: page src[i] of every pool to page dst[i].
#include <cuda_fp8.h>

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "sm100_ptx.cuh"
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
  float eps;
  unsigned polls;                               // of a wait for a stage
  // of the many-row kernel: rows and heads of an item, chunks of heads per row,
  // blocks of rows, steps of gridDim.x items, log2 of the groups of lanes per row
  int rows, heads, chunks, next_chunk, gpt_shift, stage_bytes;
  int64_t blocks, next_block;
  unsigned* error;
};

__device__ __forceinline__ uint32_t h2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four consecutive features of a head.  e4m3: value / scale (the IEEE quotient, so that the bytes are those of the
// plain definition), clamped to +-448.
template <bool FP8>
__device__ __forceinline__ void store4(void* base, int64_t elem, const float* y, float scale) {
  if constexpr (FP8) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[0], scale), __fdiv_rn(y[1], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(y[2], scale), __fdiv_rn(y[3], scale)),
                                                 __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(base) + elem) = lo | (hi << 16);
  } else {
    *reinterpret_cast<uint2*>(static_cast<__half*>(base) + elem) = make_uint2(h2_bits(y[0], y[1]), h2_bits(y[2], y[3]));
  }
}

__device__ __forceinline__ void unpack4(uint2 raw, float* x) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// A group of DH / 8 lanes owns one head; a lane holds two runs of four features
// such that both members of a rotated pair are its own: lane l with 4l < rot / 2
// has pairs 4l .. 4l + 3, i.e. features 4l.. and rot/2 + 4l.. (rotate-half) or 8l..
// and 8l + 4.. (interleaved); the lanes after those share the features from rot
// on.  The sum of squares is a shuffle reduction over the group.  With the norm's
// factor r the result is r (x_i (g_i c_i) + x_j (g_j s_i)), j the partner of i and
// s_i its signed sine: the products of gain and angle are formed once per row and
// kind of head.
struct Eight {
  uint2 lo, hi;
};

// two fp32 operations in one instruction
__device__ __forceinline__ float2 mul2(float a0, float a1, float b0, float b1) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}" : "=f"(d.x), "=f"(d.y) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
  return d;
}
__device__ __forceinline__ float2 fma2(float a0, float a1, float b0, float b1, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c.x), "f"(c.y));
  return d;
}

template <int DH, bool INTER>
struct Turner {
  static constexpr int LPH = DH / 8;
  static constexpr int P = INTER ? 1 : 4;       // feature e's partner is e ^ P
  float a[8], b[8];
  int f0, f1;                                   // first features of the two runs
  bool rotates, all;                            // this lane; every lane

  __device__ explicit Turner(int rot) {
    const int l = threadIdx.x % LPH;
    all = rot == DH;
    rotates = 4 * l < rot / 2;
    f0 = INTER || !rotates ? 8 * l : 4 * l;     // past the rotated ones: rot + 2 (4l - rot / 2) = 8l
    f1 = INTER || !rotates ? 8 * l + 4 : rot / 2 + 4 * l;
  }
  __device__ __forceinline__ Eight load(const __half* head) const {
    return {*reinterpret_cast<const uint2*>(head + f0), *reinterpret_cast<const uint2*>(head + f1)};
  }
  // angles: the row's (cos, sin) pairs; gains: or null
  __device__ __forceinline__ void coefficients(const __half* gains, const float4* angles) {
    float g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = 1.f;
    if (gains) {
      const Eight r = load(gains);
      unpack4(r.lo, g);
      unpack4(r.hi, g + 4);
    }
    if (!rotates) {
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = g[e], b[e] = 0.f;
      return;
    }
    const int l = threadIdx.x % LPH;
    const float4 w0 = angles[2 * l], w1 = angles[2 * l + 1];    // pairs 4l .. 4l + 3
    const float c[4] = {w0.x, w0.z, w1.x, w1.z}, s[4] = {w0.y, w0.w, w1.y, w1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = INTER ? 2 * i : i, y = x ^ P;
      a[x] = g[x] * c[i], b[x] = -g[y] * s[i];
      a[y] = g[y] * c[i], b[y] = g[x] * s[i];
    }
  }
  // a head's eight features, normed and turned; every lane of the warp calls it
  __device__ __forceinline__ void turn(const Eight& r, bool norm, float eps, float (&y)[8]) const {
    float x[8];
    unpack4(r.lo, x);
    unpack4(r.hi, x + 4);
    float rstd = 1.f;
    if (norm) {
      float2 s2 = mul2(x[0], x[1], x[0], x[1]);
#pragma unroll
      for (int e = 2; e < 8; e += 2) s2 = fma2(x[e], x[e + 1], x[e], x[e + 1], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int d = LPH / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      // off by a few units of 2^-24; its argument is 0 or at least 2^-55 (the smallest fp16 squared, / 128)
      asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(rstd) : "f"(fmaf(ss, 1.f / (float)DH, eps)));
    }
    if (all) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 own = mul2(x[e], x[e + 1], a[e], a[e + 1]);
        const float2 v = fma2(x[e ^ P], x[(e + 1) ^ P], b[e], b[e + 1], own);
        const float2 w = mul2(v.x, v.y, rstd, rstd);
        y[e] = w.x, y[e + 1] = w.y;
      }
    } else {
      // lanes that do not rotate leave the partner out: its b is 0, and 0 x Inf would not be
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (rotates ? fmaf(x[e ^ P], b[e], x[e] * a[e]) : x[e] * a[e]) * rstd;
    }
  }
  template <bool FP8>
  __device__ __forceinline__ void store(void* base, int64_t head, const float (&y)[8], float scale) const {
    store4<FP8>(base, head + f0, y, scale);
    store4<FP8>(base, head + f1, y + 4, scale);
  }
};

// row t's position (-1: it writes nothing) and sequence
__device__ __forceinline__ int row_position(const AppendParams& p, int64_t t, int& sq) {
  const int pp = p.pos[t];
  sq = p.seq ? p.seq[t] : (t < p.seqs ? (int)t : -1);
  return pp < p.max_pos && pp < p.cs_rows && sq >= 0 && sq < p.seqs && pp >= 0 ? pp : -1;
}
__device__ __forceinline__ int row_page(const AppendParams& p, int pp, int sq) {
  const int page = p.table[(int64_t)sq * p.table_stride + (pp >> p.page_shift)];
  return page < p.pages ? page : -1;
}

// where element 0 of head 0 of a row's page slot lies
__device__ __forceinline__ int64_t row_place(const AppendParams& p, int page, int pp, int dh) {
  return (int64_t)page * p.page_stride + (int64_t)(pp & ((1 << p.page_shift) - 1)) * dh;
}
// value head kv of a row: as given (bit for bit), or in e4m3
template <int DH, bool FP8, bool INTER>
__device__ __forceinline__ void store_value(const AppendParams& p, const Turner<DH, INTER>& tn, int64_t place, int kv,
                                            const Eight& raw) {
  const int64_t at = place + ((int64_t)kv << p.page_shift) * DH;
  if constexpr (FP8) {
    float y[8];
    unpack4(raw.lo, y);
    unpack4(raw.hi, y + 4);
    tn.template store<true>(p.v, at, y, p.v_scale[kv]);
  } else {
    __half* dst = static_cast<__half*>(p.v) + at;
    *reinterpret_cast<uint2*>(dst + tn.f0) = raw.lo;
    *reinterpret_cast<uint2*>(dst + tn.f1) = raw.hi;
  }
}

// Few rows: one head per group, spread over the CTAs, every load issued at once.
// Latency: 2.0 us a call for one row of 80 heads (the kernel below: 3.9), in a graph.
template <int DH, bool FP8, bool INTER>
__global__ void __launch_bounds__(256)
paged_append_kernel(const AppendParams p) {
  constexpr int LPH = DH / 8, GROUPS = 256 / LPH;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();                                          // what follows may be the last kernel's
  const int64_t t = blockIdx.x;
  const int j = (int)blockIdx.y * GROUPS + threadIdx.x / LPH;
  const bool exists = j < p.H + 2 * p.Hkv;
  Turner<DH, INTER> tn(p.rot);
  Eight raw = {};
  if (exists) raw = tn.load(p.qkv + t * p.qkv_stride + (int64_t)j * DH);
  int sq;
  const int pp = row_position(p, t, sq);
  if (pp < 0) return;                                           // the whole CTA: it has one row
  const int page = row_page(p, pp, sq);
  tn.coefficients(j < p.H ? p.gq : p.gk, reinterpret_cast<const float4*>(p.cs + (int64_t)pp * p.rot));
  float y[8];
  tn.turn(raw, p.gq, p.eps, y);
  if (!exists) return;
  if (j < p.H) {
    tn.template store<false>(p.q_out, t * p.q_stride + (int64_t)j * DH, y, 1.f);
  } else if (page >= 0) {
    const int kv = j - p.H;
    const int64_t place = row_place(p, page, pp, DH);
    if (kv < p.Hkv)
      tn.template store<FP8>(p.k, place + ((int64_t)kv << p.page_shift) * DH, y, FP8 ? p.k_scale[kv] : 1.f);
    else
      store_value<DH, FP8>(p, tn, place, kv - p.Hkv, raw);
  }
}

// Many rows: persistent CTAs.  An item is `rows` consecutive rows (all heads), or
// a run of one row's heads where a row is long; up to 25 KB.  The producer warp
// looks the rows up an item ahead (a lane per row) and bulk-copies them and
// their angles into a ring of stages, so that every load's latency is behind
// the items before it; eight warps turn and store.  Bound by memory: 16384 rows of 80
// heads of 128 in fp16 123-125 us (5.5 TB/s, 84 % of a copy's rate, in graphs of calls
// under the power cap; 117 before it sets in, 122 then without the arithmetic), 5001 rows
// of 96 heads of 64 25.6 us (4.85 TB/s: 2501 items of two rows, 5.6 a CTA).
// CTAs per SM of the few-row kernel up to which it is taken.  Few / many rows' kernel: 4 per SM (118 rows
// of 80 heads) 3.0 / 5.1 us, 8 (592 of 20) 4.1 / 5.0, 16 (1184 of 20) 6.4 / 6.2, 20 (590 of 80) 7.4 / 8.2,
// 32 (2400 of 20) 11.0 / 9.4, 40 (1180 of 80) 12.9 / 12.6
constexpr int kFewCtasPerSm = 14;
constexpr int kItemBytes = 25 * 1024 + 512;
constexpr int kAppendStages = 2;
constexpr int kAppendThreads = 288;
constexpr unsigned kAppendProducerCode = 61, kAppendConsumerCode = 62, kAppendDrainCode = 63;

// the items of a CTA: block (of rows) and chunk (of heads), gridDim.x apart
struct Item {
  int64_t block;
  int chunk;
  __device__ explicit Item(const AppendParams& p)
      : block(blockIdx.x / p.chunks), chunk((int)(blockIdx.x % p.chunks)) {}
  __device__ void next(const AppendParams& p) {
    block += p.next_block;
    chunk += p.next_chunk;
    if (chunk >= p.chunks) chunk -= p.chunks, ++block;
  }
};

template <int DH, bool FP8, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, 3)
paged_append_stream_kernel(const AppendParams p) {
  using namespace ptx;
  constexpr int LPH = DH / 8, GROUPS = 256 / LPH;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t full[kAppendStages], empty[kAppendStages];
  __shared__ int2 place[kAppendStages][32];                     // (position or -1, page or -1) of the item's rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kAppendStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 8);
    }
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();
  const int nh = p.H + 2 * p.Hkv;
  int st = 0;
  if (warp == 8) {
    uint32_t phase = 1;
    int64_t n = 0;
    auto look = [&](const Item& it, int& sq) -> int {
      const int64_t t = it.block * p.rows + lane;
      return lane < p.rows && t < p.T ? row_position(p, t, sq) : -1;
    };
    int sq = 0, sq_next = 0;
    Item item(p), item2(p);
    int pp = look(item, sq);
    int page = pp >= 0 ? row_page(p, pp, sq) : -1;
    item2.next(p);
    int pp_next = look(item2, sq_next);
    item2.next(p);
    for (; item.block < p.blocks && p.polls != 0; item.next(p), item2.next(p), ++n, ++st) {   // 0: a test's, nothing is loaded
      if (st == kAppendStages) st = 0, phase ^= 1;
      const int page_next = pp_next >= 0 ? row_page(p, pp_next, sq_next) : -1;
      int sq2 = 0;
      const int pp2 = look(item2, sq2);
      // a wait that runs out ends the loads: a stage that is not free is not armed again
      if (n >= kAppendStages && !__all_sync(0xFFFFFFFFu, mbar_wait_after_poll(&empty[st], phase, p.polls))) {
        if (lane == 0) record_wait_failure(p.error, kAppendProducerCode);
        break;
      }
      const int h0 = item.chunk * p.heads, nhc = nh - h0 < p.heads ? nh - h0 : p.heads;
      place[st][lane] = make_int2(pp, page);
      const int live = __popc(__ballot_sync(0xFFFFFFFFu, pp >= 0));
      __syncwarp();                                             // a vote orders no memory: the places, then the arrival
      if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)(live * (nhc * DH * 2 + p.rot * 4)));
      __syncwarp();
      if (pp >= 0) {
        uint8_t* dst = sm + st * p.stage_bytes;
        bulk_load(dst + lane * p.heads * DH * 2, p.qkv + (item.block * p.rows + lane) * p.qkv_stride + (int64_t)h0 * DH,
                  (uint32_t)(nhc * DH * 2), &full[st]);
        bulk_load(dst + p.rows * p.heads * DH * 2 + lane * p.rot * 4, p.cs + (int64_t)pp * p.rot,
                  (uint32_t)(p.rot * 4), &full[st]);
      }
      pp = pp_next, page = page_next, pp_next = pp2, sq_next = sq2;
    }
    // every copy has landed before the CTA may leave
    for (int64_t i = n > kAppendStages ? n - kAppendStages : 0; i < n; ++i)
      if (!mbar_wait(&full[i % kAppendStages], (uint32_t)(i / kAppendStages) & 1, kWaitPolls) && lane == 0)
        record_wait_failure(p.error, kAppendDrainCode);
    return;
  }
  const int grp = threadIdx.x / LPH, gi = grp & ((1 << p.gpt_shift) - 1), gr = grp >> p.gpt_shift;
  const int gpt = 1 << p.gpt_shift, per_pass = GROUPS >> p.gpt_shift;
  Turner<DH, INTER> tn(p.rot);
  uint32_t phase = 0;
  for (Item item(p); item.block < p.blocks; item.next(p), ++st) {
    if (st == kAppendStages) st = 0, phase ^= 1;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_after_poll(&full[st], phase, p.polls))) {
      if (lane == 0) record_wait_failure(p.error, kAppendConsumerCode);
      return;                                                   // this warp stores nothing more, and frees no stage
    }
    const int64_t t0 = item.block * p.rows;
    const int h0 = item.chunk * p.heads, nhc = nh - h0 < p.heads ? nh - h0 : p.heads;
    // of the item's heads, h0 .. h0 + nhc - 1: queries, keys, values
    auto below = [&](int end) { return end - h0 < 0 ? 0 : (end - h0 < nhc ? end - h0 : nhc); };
    const int nq = below(p.H), nqk = below(p.H + p.Hkv);
    // keys follow on from the groups that had the last queries, values from theirs
    const int gk = nq + ((gi - nq) & (gpt - 1)), gv = nqk + ((gi - nqk) & (gpt - 1));
    const uint8_t* stage = sm + st * p.stage_bytes;
    for (int r0 = 0; r0 < p.rows; r0 += per_pass) {             // shuffles below: trip counts are the CTA's
      const bool real = r0 + gr < p.rows;
      const int r = r0 + gr < p.rows ? r0 + gr : p.rows - 1;
      const int2 at = place[st][r];
      const bool valid = real && at.x >= 0;
      const __half* src = reinterpret_cast<const __half*>(stage) + r * p.heads * DH;
      const float4* angles = reinterpret_cast<const float4*>(stage + p.rows * p.heads * DH * 2 + r * p.rot * 4);
      if (nq > 0) {
        tn.coefficients(p.gq, angles);
        __half* dst = p.q_out + (t0 + r) * p.q_stride + (int64_t)h0 * DH;
#pragma unroll 1
        for (int j0 = 0; j0 < nq; j0 += gpt) {
          const int j = j0 + gi;
          float y[8];
          tn.turn(tn.load(src + (j < nq ? j : 0) * DH), p.gq, p.eps, y);
          if (valid && j < nq) tn.template store<false>(dst, j * DH, y, 1.f);
        }
      }
      const int64_t place_kv = row_place(p, at.y, at.x, DH);
      if (__any_sync(0xFFFFFFFFu, gk < nqk)) {
        tn.coefficients(p.gk, angles);
        for (int j0 = 0; j0 < nqk - nq; j0 += gpt) {
          const int j = j0 + gk;
          if (!__any_sync(0xFFFFFFFFu, j < nqk)) break;
          float y[8];
          tn.turn(tn.load(src + (j < nqk ? j : 0) * DH), p.gq, p.eps, y);
          const int kv = h0 + j - p.H;
          if (valid && j < nqk && at.y >= 0)
            tn.template store<FP8>(p.k, place_kv + ((int64_t)kv << p.page_shift) * DH, y, FP8 ? p.k_scale[kv] : 1.f);
        }
      }
      if (valid && at.y >= 0)
        for (int j = gv; j < nhc; j += gpt)
          store_value<DH, FP8>(p, tn, place_kv, h0 + j - p.H - p.Hkv, tn.load(src + j * DH));
      __syncwarp();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
}

// ---------------------------------------------------------------- page copies
// bytes a warp moves at once: 4 x 16 per lane.  1500 pages of 128 KB in 4 pools: 240 us,
// 6.6 TB/s read and written, the rate of a copy (1 KB a warp: 268 us, 4 KB: 257, when 8
// CTAs per SM walked the pages; they do so 64 at a time now)
constexpr int kCopyUnit = 2048;

__global__ void __launch_bounds__(256)
copy_pages_kernel(uint8_t* __restrict__ pools, int64_t n_pools, int64_t pool_stride, int pages,
                  int64_t page_stride, int64_t page_bytes, const int* __restrict__ src,
                  const int* __restrict__ dst, int64_t n, int64_t units_per_page) {
  const int lane = threadIdx.x & 31;
  const int64_t units = n * n_pools * units_per_page;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
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

// programmatic launch: the kernel may start while the one before it ends, and
// waits for its end before it touches memory
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
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
  p.seqs = (int)c.seqs, p.max_pos = (int)(c.seq_pages * c.page_size), p.polls = wait_polls();
  // below the normal numbers the root would flush it, and a head of zeros be 0 x Inf; to a mean
  // that is not 0, 2^-55 at least, neither adds anything
  p.eps = eps > 0.f && eps < FLT_MIN ? FLT_MIN : eps;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  const int groups = (int)(256 * 8 / c.head_dim);
  const int64_t nh = H + 2 * c.heads, head_bytes = c.head_dim * 2;
  const bool fp8 = c.dtype == TRI_CACHE_E4M3;
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  auto pick = [&](auto run) -> cudaError_t {
    if (c.head_dim == 128) {
      if (fp8) return interleaved ? run(D128{}, std::true_type{}, std::true_type{}) : run(D128{}, std::true_type{}, std::false_type{});
      return interleaved ? run(D128{}, std::false_type{}, std::true_type{}) : run(D128{}, std::false_type{}, std::false_type{});
    }
    if (fp8) return interleaved ? run(D64{}, std::true_type{}, std::true_type{}) : run(D64{}, std::true_type{}, std::false_type{});
    return interleaved ? run(D64{}, std::false_type{}, std::true_type{}) : run(D64{}, std::false_type{}, std::false_type{});
  };
  if (T * ceil_div(nh, groups) <= kFewCtasPerSm * (int64_t)sms) {
    const dim3 grid((unsigned)T, (unsigned)ceil_div(nh, groups));
    return pick([&](auto dh, auto e, auto il) -> cudaError_t {
      return launch_chained(paged_append_kernel<decltype(dh)::value, decltype(e)::value, decltype(il)::value>, grid,
                            256, 0, s, p);
    });
  }
  const int64_t row_bytes = nh * head_bytes + rot * 4;
  p.rows = row_bytes >= kItemBytes ? 1 : (int)(kItemBytes / row_bytes < 32 ? kItemBytes / row_bytes : 32);
  p.heads = (int)(nh <= kItemBytes / head_bytes ? nh : kItemBytes / head_bytes);
  p.chunks = (int)ceil_div(nh, p.heads);
  p.blocks = ceil_div(T, p.rows);
  p.stage_bytes = (int)((p.rows * (p.heads * head_bytes + rot * 4) + 127) & ~int64_t(127));
  // as few groups of lanes per row (its coefficients are formed by each) as leave none without a row
  while ((groups >> p.gpt_shift) > p.rows) ++p.gpt_shift;
  const int64_t items = p.blocks * p.chunks, most = 3 * (int64_t)sms;
  const int ctas = (int)(items < most ? items : most);
  p.next_block = ctas / p.chunks, p.next_chunk = ctas % p.chunks;
  cudaError_t err = wait_status_word(&p.error);
  if (err != cudaSuccess) return err;
  const int smem = kAppendStages * p.stage_bytes;
  return pick([&](auto dh, auto e, auto il) -> cudaError_t {
    auto kernel = paged_append_stream_kernel<decltype(dh)::value, decltype(e)::value, decltype(il)::value>;
    static std::atomic<bool> ready[64] = {};                    // host threads may call at once
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    if (dev >= 64 || !ready[dev]) {
      r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAppendStages * (kItemBytes + 1024));
      if (r != cudaSuccess) return r;
      if (dev < 64) ready[dev] = true;
    }
    return launch_chained(kernel, dim3((unsigned)ctas), kAppendThreads, (size_t)smem, s, p);
  });
}

cudaError_t launch_copy_pages(uint8_t* pools, int64_t n_pools, int64_t pool_stride, int64_t pages,
                              int64_t page_stride, int64_t page_bytes, const int* src, const int* dst,
                              int64_t n, int sms, cudaStream_t s) {
  const int64_t upp = ceil_div(page_bytes, kCopyUnit);
  const int64_t ctas = ceil_div(n * n_pools, 8) < (int64_t(1) << 40) / upp ? ceil_div(n * n_pools * upp, 8)
                                                                             : (int64_t(1) << 40);
  const int64_t most = (int64_t)sms * 64;
  return launch_chained(copy_pages_kernel, dim3((unsigned)(ctas < most ? ctas : most)), 256, 0, s, pools, n_pools,
                        pool_stride, (int)pages, page_stride, page_bytes, src, dst, n, upp);
}

}  // namespace tri

// Attention of new tokens over a paged key/value cache:
//   out = sum_p w_p V_p / sum_p w_p,  w_p = exp(scale q . K_p - max),
// over the positions 0..pos of the row whose page is present.  One CTA per
// (row, query head): 128 positions at a time, one per thread, the running
// maximum and sum in fp32; then thread d sums feature d.
#include <cuda_fp8.h>

#include "tri_internal.cuh"

namespace tri {
namespace {

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_fp8_e4m3 x) { return static_cast<float>(x); }

template <typename E, int DH>
__global__ void __launch_bounds__(128)
paged_attn_simple_kernel(const __half* __restrict__ q, int64_t q_stride, const int* __restrict__ pos,
                         const int* __restrict__ seq, const tri_paged_cache c, __half* __restrict__ out,
                         int64_t out_stride, int H, float scale) {
  __shared__ float qs[DH], w[128], red[4];
  __shared__ int pg[128];
  const int64_t m = blockIdx.x / H;
  const int h = (int)(blockIdx.x % H), kv = h / (H / (int)c.heads), t = threadIdx.x;
  const int ps = (int)c.page_size;
  const int s = seq ? seq[m] : (m < c.seqs ? (int)m : -1);
  int64_t L = (int64_t)pos[m] + 1;
  if (s < 0 || s >= c.seqs || L < 0) L = 0;
  if (L > c.seq_pages * ps) L = c.seq_pages * ps;
  if (t < DH) qs[t] = __half2float(q[m * q_stride + (int64_t)h * DH + t]);
  const float ks = c.dtype == TRI_CACHE_E4M3 ? c.k_scale[kv] : 1.f;
  const float vs = c.dtype == TRI_CACHE_E4M3 ? c.v_scale[kv] : 1.f;
  const E* kp = static_cast<const E*>(c.k);
  const E* vp = static_cast<const E*>(c.v);
  float mx = -INFINITY, l = 0.f, acc = 0.f;
  __syncthreads();
  for (int64_t p0 = 0; p0 < L; p0 += 128) {
    const int64_t p = p0 + t;
    int page = p < L ? c.table[(int64_t)s * c.table_stride + p / ps] : -1;
    if (page >= c.pages) page = -1;
    float sc = -INFINITY;
    if (page >= 0) {
      const E* row = kp + page * c.page_stride + ((int64_t)kv * ps + p % ps) * DH;
      float d = 0.f;
      for (int i = 0; i < DH; ++i) d = fmaf(qs[i], to_float(row[i]), d);
      sc = d * scale * ks;
    }
    pg[t] = page;
    float v = sc;
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if ((t & 31) == 0) red[t >> 5] = v;
    __syncthreads();
    const float mnew = fmaxf(mx, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = mnew == -INFINITY ? 0.f : mnew;
    const float alpha = expf(mx - base);
    w[t] = expf(sc - base);
    __syncthreads();
    acc *= alpha, l *= alpha;
    for (int i = 0; i < 128; ++i) {
      if (pg[i] < 0) continue;
      l += w[i];
      if (t < DH) {
        const E* row = vp + pg[i] * c.page_stride + ((int64_t)kv * ps + (p0 + i) % ps) * DH;
        acc = fmaf(w[i], to_float(row[t]), acc);
      }
    }
    mx = mnew;
    __syncthreads();
  }
  if (t < DH) out[m * out_stride + (int64_t)h * DH + t] = __float2half_rn(l == 0.f ? 0.f : acc / l * vs);
}

}  // namespace

size_t paged_attention_ws_bytes(int64_t, int64_t, int64_t, int64_t, int) { return 256; }

cudaError_t launch_paged_attention(const __half* q, int64_t q_stride, const int* pos, const int* seq,
                                   const tri_paged_cache& c, __half* out, int64_t out_stride, int64_t M,
                                   int64_t H, float scale, void*, int, cudaStream_t s) {
  const unsigned grid = (unsigned)(M * H);
  if (c.dtype == TRI_CACHE_E4M3) {
    if (c.head_dim == 128)
      paged_attn_simple_kernel<__nv_fp8_e4m3, 128><<<grid, 128, 0, s>>>(q, q_stride, pos, seq, c, out, out_stride,
                                                                         (int)H, scale);
    else
      paged_attn_simple_kernel<__nv_fp8_e4m3, 64><<<grid, 128, 0, s>>>(q, q_stride, pos, seq, c, out, out_stride,
                                                                        (int)H, scale);
  } else {
    if (c.head_dim == 128)
      paged_attn_simple_kernel<__half, 128><<<grid, 128, 0, s>>>(q, q_stride, pos, seq, c, out, out_stride, (int)H,
                                                                 scale);
    else
      paged_attn_simple_kernel<__half, 64><<<grid, 128, 0, s>>>(q, q_stride, pos, seq, c, out, out_stride, (int)H,
                                                                scale);
  }
  return cudaGetLastError();
}

}  // namespace tri

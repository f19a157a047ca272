// Attention of new tokens over a paged key/value cache:
//   out = sum_p w_p V_p / sum_p w_p,  w_p = exp(scale q . K_p - max),
// over the positions 0..pos of the row whose page is present.
//
// What bounds it: every key and value is read once for the G = H / heads query
// heads that share it, 4 G flops per element: HBM bandwidth.
//
//  * Work = tiles of 64 or 128 positions of one (row, key/value head), in the order
//    row, head, tile; every CTA takes an equal run of them, so ragged lengths
//    load the SMs alike and the host needs no length.  A run covers the end of
//    one (row, head), whole ones, and the start of another: whole ones are
//    written at once, the two open ends leave a (max, sum, output) partial in
//    the workspace, and paged_combine_kernel joins each split (row, head).
//  * Two producer warps, of K and of V, walk the run, look the pages up one tile
//    ahead and load them with TMA into a ring of stages (a box is one page's rows,
//    128 bytes of each, hardware-swizzled), and the row's queries with the first
//    tile.  Absent pages are not loaded.  A descriptor per stage says what the
//    tile is.
//  * Four consumer warps (per 8 query heads) take 16 or 32 positions of a tile each.  Scores are formed
//    transposed, S^T = K Q^T (mma.sync m16n8k16: positions are the 16 rows, up
//    to 8 query heads the columns, so that no row is wasted on heads that do not
//    exist), with a running reference and sum in fp32 per warp.  O^T += V^T P^T:
//    V^T comes from ldmatrix.trans, P^T from the S^T accumulators by movmatrix,
//    in two fp16 parts, so that the fp32 accumulation bounds the error.  e4m3
//    elements become fp16 (exactly) in registers; the K scale joins the softmax
//    scale, the V scale the output.
//
// A row's tiles are counted from position 0: one in an absent page costs its turn in the
// run, not its bytes.
//
// Measured (B200, 64 query heads on 8 of 128 unless said, graphs of calls, join included):
// 16 rows x 4096 positions in fp16 47.4 us (5.7 TB/s of K and V, 87 % of a copy's rate),
// 1 x 131072 88-89 us (92 %), 100 ragged rows to 6000 in e4m3 99-103 us (86 %), 9 ragged
// rows to 20000 with 16 heads on one 18.0 us (20 %: five tiles a CTA), 9 x 80000 of those
// 51-53 us (54 %), 1 x 37 4.9-5.2 us.  A reference that is raised only when it must be,
// instead of the exact maximum of every tile, took 9 x 80000 from 58.6 to 53.2 us when it
// came, a wait's first poll before its limit is looked at from 53.3 to 51.9.
#include <cuda.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "sm100_ptx.cuh"
#include "tri_internal.cuh"

namespace tri {
namespace {

using namespace ptx;

// A run of more tiles than this gives one-tile (row, head)s to single warps, which
// take its blocks one after another and need no merge.  With / without, 8 heads x 60
// positions in fp16: 300 rows (8 tiles a run) 18.5 / 22.4 us, 111 (3) 9.1 / 9.9, 74 (2)
// 7.6 / 8.0, 16 (1) 6.4 / 5.8, 1 row 5.7 / 5.0.
constexpr int kSoloRun = 1;
// Weights are held times 2^14, sums and outputs with them: the two fp16 parts then
// reach down to 2^-39 of the largest weight instead of 2^-25, below which a hundred
// thousand small weights would vanish from the output but not from their sum.
constexpr float kWeightShift = 14.f;
constexpr float kWeightMost = 15.9f;         // log2: above it a weight would near fp16's largest, 65504
constexpr float kNothing = -3e38f;           // the reference before any position: below every score
constexpr unsigned kProducerCode = 51, kConsumerCode = 52, kDrainCode = 53;

// HG: groups of 8 query heads per key/value head, 1 or 2
template <int DH, bool FP8, int HG>
struct Cfg {
  static constexpr int kWarps = 4 * HG;                       // consumer warps
  static constexpr int kThreads = 32 * (kWarps + 2);          // and two producer warps, of K and of V
  // Two CTAs per SM; one where 320 threads of 162-165 registers leave no other choice, three
  // where a position is 64 bytes and registers and stages fit.  (16 heads on one of 64,
  // 9 x 80000: two CTAs at 96 registers 36.3 us, one at 142 39.8, in fp16; 35.1 and 41.3
  // in e4m3.  12 heads of 64, 37 x 6000 in e4m3: three CTAs 63.7 us, two 70.3.)
  static constexpr int kCtasPerSm = HG == 2 && DH == 128 ? 1 : HG == 1 && DH == 64 && FP8 ? 3 : 2;
  static constexpr int kRow = DH * (FP8 ? 1 : 2);             // bytes of a position
  // A warp's chain of dependent steps per tile (scores, maximum, weights, output)
  // takes about 0.7 us whatever its width, so rows of at most 128 bytes come 128 to
  // a tile (two sets of 16 per warp); 256-byte ones, for which HBM is slower than
  // that chain, 64.
  static constexpr int kSets = kRow <= 128 ? 2 : 1;
  static constexpr int kTile = 64 * kSets;                    // positions per stage
  static constexpr int kTileShift = kSets == 2 ? 7 : 6;
  static constexpr int kBox = kRow < 128 ? kRow : 128;        // bytes of it in one box
  static constexpr int kParts = kRow / kBox;
  static constexpr int kKV = kTile * kRow;                    // bytes of a K (or V) tile
  static constexpr int kQRow = DH * 2 + 16;                   // padded: fragment reads hit distinct banks
  static constexpr int kQ = 8 * HG * kQRow;
  static constexpr int kMerge = HG * 2 * DH * 8 * 4;          // two warps' outputs of each group
  static constexpr int kRoom = (kCtasPerSm == 1 ? 224 : kCtasPerSm == 2 ? 113 : 75) * 1024 - kMerge - 2304;
  static constexpr int kStages = kRoom / (2 * kKV + kQ);       // 3 to 5
  static constexpr int kSmem = 1024 + kStages * (2 * kKV + kQ) + kMerge;
  static_assert(kStages >= 3, "a ring of three stages at least");
};

struct Desc {                 // what a stage holds
  int row, head;              // of the batch; key/value head
  int nval;                   // positions of the tile below the row's end
  int pages;                  // bit i: the tile's i-th page was loaded
  int flags;
};
constexpr int kFirst = 1, kLast = 2, kOpenLeft = 4, kOpenRight = 8, kSolo = 16;

struct Params {
  const __half* q;
  const int *pos, *seq, *table;
  const float *k_scale, *v_scale;
  __half* out;
  int4* recs;                 // {row * heads + head, first CTA, partials (0: not split), -}, one per
                              // (row, head) where there are no more of them than CTAs, else per CTA
  float2* ml;                 // [2 CTAs][8 HG] (max, sum)
  float4* part;               // [2 CTAs][DH/16][HG][32 lanes]
  unsigned* error;
  int64_t q_stride, out_stride, table_stride, M;
  int heads, G, page_shift, pages, seqs, max_len, ctas;
  unsigned polls;             // of a wait for a stage
  float scale;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// log2 of a weight (with the shift) from a score and the column's reference.  The product is
// rounded by itself, as the reference's was: the score that is the reference gives exactly 0
// however large it is, where a fused product would leave a rounding error (beyond 2^24:
// powers of two).  The shift is rounded down, so that none is above kWeightShift by rounding.
__device__ __forceinline__ float weight_shift(float mx) { return __fadd_rd(kWeightShift, -mx); }
__device__ __forceinline__ float log2_weight(float score, float c2, float shift) {
  return __fadd_rn(__fmul_rn(score, c2), shift);
}
// Two weights as two fp16 parts each, the lower the rest to 2^-20.6 of the weight and to
// 2^-39 of the largest (half a step of fp16's smallest numbers, see kWeightShift).  A
// weight of 0 is 0 in both.  The high part is taken a little short of the weight
// (2^-12 of it and 2^-24) so that above 2^-37 of the largest both parts are positive and an
// infinite value stays infinite: 0 times it would be NaN.  A NaN stays one.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, uint32_t& lo) {
  float x, y;
  asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
      "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(x), "=f"(y) : "f"(a), "f"(b), "f"(1.f - 1.f / 4096.f), "f"(-1.f / 16777216.f));
  asm("cvt.rz.relu.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const __half2 g = __floats2half2_rn(a - f.x, b - f.y);
  lo = *reinterpret_cast<const uint32_t*>(&g);
}
// four e4m3 codes as fp16: bytes 0, 1 and bytes 2, 3
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(four));
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;"
      ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy) : "memory");
}

// positions row m attends to, and whether it has any page table row
__device__ __forceinline__ int row_length(const Params& p, int64_t m, int& s) {
  s = p.seq ? p.seq[m] : (m < p.seqs ? (int)m : -1);
  const int L = p.pos[m];
  if (s < 0 || s >= p.seqs || L < 0) return 0;
  return L < p.max_len ? L + 1 : p.max_len;
}

// the runs: the first `rem` CTAs take base + 1 tiles
struct Runs {
  int64_t base, rem;
  __device__ Runs(int64_t W, int C) : base(W / C), rem(W % C) {}
  __device__ int64_t start(int c) const { return base * c + (c < rem ? c : rem); }
  __device__ int cta_of(int64_t w) const {
    const int64_t big = (base + 1) * rem;
    return (int)(w < big ? w / (base + 1) : rem + (w - big) / base);
  }
};

// a row's 16-byte chunk in a K or V tile, as the TMA swizzle places it
template <typename C>
__device__ __forceinline__ uint32_t tile_address(uint32_t base, int row, int chunk) {
  if constexpr (C::kBox == 128)
    return base + (uint32_t)((chunk >> 3) * C::kTile * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
  else
    return base + (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// a lane's four sums of a feature block: heads h0 and h0 + 1 of (x, z) and (y, w)
template <int DH, bool FP8>
__device__ __forceinline__ void store_out(__half* dst, int h0, int G, int f, int gid, float4 y, float i0, float i1) {
  const int f0 = f + (FP8 ? 2 * gid : gid), f1 = f + (FP8 ? 2 * gid + 1 : 8 + gid);
  if (h0 < G) {
    dst[h0 * DH + f0] = __float2half_rn(y.x * i0);
    dst[h0 * DH + f1] = __float2half_rn(y.z * i0);
  }
  if (h0 + 1 < G) {
    dst[(h0 + 1) * DH + f0] = __float2half_rn(y.y * i1);
    dst[(h0 + 1) * DH + f1] = __float2half_rn(y.w * i1);
  }
}

template <int DH, bool FP8, int HG>
__global__ void __launch_bounds__((Cfg<DH, FP8, HG>::kThreads), (Cfg<DH, FP8, HG>::kCtasPerSm))
paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Params p) {
  using C = Cfg<DH, FP8, HG>;
  constexpr int kWarps = C::kWarps, kThreads = C::kThreads, kTile = C::kTile;
  constexpr int kTileShift = C::kTileShift, kSets = C::kSets;
  extern __shared__ uint8_t raw_smem[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* qring = sm + C::kStages * 2 * C::kKV;
  float4* merge = reinterpret_cast<float4*>(qring + C::kStages * C::kQ);
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ Desc desc[C::kStages];
  __shared__ __align__(16) float2 wml[kWarps][8];
  __shared__ long long sums[kWarps + 2], s_first_offset;
  __shared__ int s_first_row;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto row_tiles = [](int len) { return (len + kTile - 1) >> kTileShift; };

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
  }
  if (warp >= kWarps && lane == 0) prefetch_tensormap(warp == kWarps ? &kmap : &vmap);
  griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's run: thread t sums the tiles of M / kThreads consecutive rows
  const int64_t chunk = (p.M + kThreads - 1) / kThreads, m_lo = tid * chunk;
  const int64_t m_hi = m_lo + chunk < p.M ? m_lo + chunk : p.M;
  long long mine = 0;
  for (int64_t m = m_lo; m < m_hi; ++m) {
    int s;
    mine += row_tiles(row_length(p, m, s));
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps + 2; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  const Runs runs(total * p.heads, gridDim.x);
  const int64_t w0 = runs.start(blockIdx.x), ntiles = runs.start(blockIdx.x + 1) - w0;
  if (mine > 0 && w0 >= before * p.heads && w0 < (before + mine) * p.heads) {
    int64_t m = m_lo;
    long long at = before;
    for (; m < m_hi - 1; ++m) {
      int s;
      const int t = row_tiles(row_length(p, m, s));
      if (w0 < (at + t) * p.heads) break;
      at += t;
    }
    s_first_row = (int)m;
    s_first_offset = w0 - at * p.heads;
  }
  __syncthreads();
  // rows with nothing to read take no tiles: their zeros are dealt out by row
  const bool by_seg = p.M * p.heads <= gridDim.x;               // see Params::recs
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    int s;
    if (row_length(p, m, s) > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(p.out + m * p.out_stride);
    for (int i = tid; i < p.heads * p.G * (DH / 8); i += kThreads) dst[i] = make_uint4(0, 0, 0, 0);
    if (by_seg)
      for (int i = tid; i < p.heads; i += kThreads) p.recs[m * p.heads + i] = make_int4(0, 0, 0, 0);
  }
  if (ntiles == 0) {
    if (!by_seg && tid == 0) p.recs[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  if (warp >= kWarps) {
    // ------------------------------------------------------------ producers
    const bool is_v = warp > kWarps;
    const uint64_t policy = policy_evict_first();
    const int shift = p.page_shift, rows = shift < kTileShift ? 1 << shift : kTile;   // of a box
    const int npg = kTile / rows, nbox = npg * C::kParts;
    const int pi = lane % npg, part = lane / npg;
    const uint32_t box_dst = (uint32_t)((is_v ? C::kKV : 0) + part * kTile * C::kBox + pi * rows * C::kBox);
    const int box_x = part * (C::kBox / (FP8 ? 1 : 2));
    int64_t m = s_first_row;
    int s, L = row_length(p, m, s), T = row_tiles(L);
    const int64_t off = s_first_offset;
    int h = (int)(off / T), t = (int)(off % T);
    // the next row's length, read a row ahead
    int s_next = -1, L_next = m + 1 < p.M ? row_length(p, m + 1, s_next) : 0;
    auto lookup = [&](int s_, int L_, int t_) -> int {     // this lane's page of a tile, -1: do not load
      const int64_t first = (int64_t)t_ * kTile + (int64_t)pi * rows;
      if (lane >= nbox || first >= L_) return -1;
      const int id = p.table[(int64_t)s_ * p.table_stride + (first >> shift)];
      return id < p.pages ? id : -1;
    };
    int id = lookup(s, L, t);
    int4 split_rec = make_int4(0, 0, 0, 0);
    int st = 0;
    uint32_t phase = 1;                                         // of `empty`; nothing to wait for in the first round
    int64_t i = 0;
    for (; i < ntiles && p.polls != 0; ++i, ++st) {             // 0: a test's, nothing is loaded
      if (st == C::kStages) st = 0, phase ^= 1;
      const int cm = (int)m, ch = h, ct = t, cT = T, cL = L, cid = id;
      // step on, and look the next tile's page up while this stage's slot frees
      if (++t == T) {
        t = 0;
        if (++h == p.heads) {
          h = 0;
          do {                                                  // the next row that has anything
            ++m, s = s_next, L = L_next;
            L_next = m + 1 < p.M ? row_length(p, m + 1, s_next) : 0;
          } while (L == 0 && m + 1 < p.M);
          T = row_tiles(L);
        }
      }
      if (i + 1 < ntiles) id = lookup(s, L, t);
      // a wait that runs out ends the loads: a stage that is not free is not armed again
      if (i >= C::kStages && !__all_sync(0xFFFFFFFFu, mbar_wait_after_poll(&empty[st], phase, p.polls))) {
        if (lane == 0) record_wait_failure(p.error, kProducerCode);
        break;
      }
      const bool first = i == 0 || ct == 0, last = i + 1 == ntiles || ct == cT - 1;
      const unsigned loaded = __ballot_sync(0xFFFFFFFFu, cid >= 0);
      if (lane == 0 && !is_v) {
        Desc d;
        d.row = cm, d.head = ch;
        const int64_t left = (int64_t)cL - (int64_t)ct * kTile;
        d.nval = left < 0 ? 0 : (left < kTile ? (int)left : kTile);
        d.pages = (int)(loaded & ((1u << npg) - 1));       // lanes 0.. hold K's first part of page 0..
        d.flags = (first ? kFirst : 0) | (last ? kLast : 0);
        if (last) {
          const bool open_l = i - ct < 0;                  // the (row, head) began before this run
          const bool open_r = ct != cT - 1;
          d.flags |= (open_l ? kOpenLeft : 0) | (open_r ? kOpenRight : 0);
        }
        if (ct == 0 && cT == 1 && ntiles > kSoloRun) d.flags |= kSolo;
        desc[st] = d;
        // the CTA that holds the first tile of a (row, head) says who joins it
        if (ct == 0) {
          const int64_t seg = (int64_t)cm * p.heads + ch, end = i + cT;
          const bool split = end > ntiles;
          const int4 rec = make_int4((int)seg, (int)blockIdx.x,
                                     split ? runs.cta_of(w0 + end - 1) - (int)blockIdx.x + 1 : 0, 0);
          if (by_seg) p.recs[seg] = rec;
          else if (split) split_rec = rec;
        }
      }
      if (lane == 0)
        mbar_arrive_expect_tx(&full[st],
                              (uint32_t)(__popc(loaded) * rows * C::kBox + (first && !is_v ? p.G * DH * 2 : 0)));
      __syncwarp();
      if (first && !is_v && lane < p.G)
        bulk_load(qring + st * C::kQ + lane * C::kQRow, p.q + (int64_t)cm * p.q_stride + ((int64_t)ch * p.G + lane) * DH,
                  DH * 2, &full[st]);
      if (cid >= 0) {
        const int in_page = shift > kTileShift ? (int)(((int64_t)ct * kTile) & ((1 << shift) - 1)) : 0;
        tma_load_3d(smem_u32(sm) + (uint32_t)(st * 2 * C::kKV) + box_dst, is_v ? &vmap : &kmap, box_x,
                    (ch << shift) + in_page, cid, &full[st], policy);
      }
    }
    if (lane == 0 && !is_v && !by_seg) p.recs[blockIdx.x] = split_rec;
    // every copy has landed before the CTA may leave
    for (int64_t j = i > C::kStages ? i - C::kStages : 0; j < i; ++j)
      if (!mbar_wait(&full[j % C::kStages], (uint32_t)(j / C::kStages) & 1, kWaitPolls) && lane == 0)
        record_wait_failure(p.error, kDrainCode);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int gid = lane >> 2, tig = lane & 3, quarter = warp & 3, group = warp >> 2;
  const int hb = 8 * group;                                     // the first of this warp's query heads
  const int page_shift = p.page_shift < kTileShift ? p.page_shift : kTileShift;
  // ldmatrix rows and 16-byte chunks: K (and e4m3 V): rows (lane & 7) + 8 (lane
  // >> 3 & 1), chunk + (lane >> 4); fp16 V transposed: rows (lane & 7) + 8 (lane
  // >> 4), chunk + (lane >> 3 & 1)
  const int r_a = (lane & 7) + 8 * ((lane >> 3) & 1), c_a = lane >> 4;
  const int r_t = (lane & 7) + 8 * (lane >> 4), c_t = (lane >> 3) & 1;
  auto address = [](uint32_t base, int row, int chunk) { return tile_address<C>(base, row, chunk); };
  uint32_t qf[DH / 16][2];
  float o[DH / 16][4];
  float mx[2], l[2];
  float c2 = 0.f;
  uint32_t phase = 0;
  int st = 0;
  int64_t i = 0;
  for (; i < ntiles; ++i, ++st) {
    if (st == C::kStages) st = 0, phase ^= 1;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_after_poll(&full[st], phase, p.polls))) break;
    const Desc d = desc[st];
    // a one-tile (row, head) in a longer run is one warp's, with no merge; its
    // neighbours are the other warps'
    const bool solo = d.flags & kSolo;
    if (solo && (int)(i & 3) != quarter) {
      __syncwarp();                                              // every lane has read desc[st]
      if (lane == 0) mbar_arrive(&empty[st]);
      continue;
    }
    const uint32_t kbase = smem_u32(sm) + (uint32_t)(st * 2 * C::kKV), vbase = kbase + C::kKV;
    if (d.flags & kFirst) {
      const uint32_t qb = smem_u32(qring + st * C::kQ);
      const bool real = hb + gid < p.G;
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        // fp16: features 2 tig, +1 and 8 + 2 tig, +1 of the step; e4m3: 4 tig .. 4 tig + 3,
        // the order in which a lane gets its four bytes of K
        const uint32_t a = qb + (uint32_t)((hb + gid) * C::kQRow + kk * 32 + (FP8 ? 8 : 4) * tig);
        qf[kk][0] = real ? lds32(a) : 0u;
        qf[kk][1] = real ? lds32(a + (FP8 ? 4 : 16)) : 0u;
      }
      mx[0] = mx[1] = kNothing;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int fb = 0; fb < DH / 16; ++fb) o[fb][0] = o[fb][1] = o[fb][2] = o[fb][3] = 0.f;
      c2 = p.scale * 1.4426950408889634f * (FP8 ? p.k_scale[d.head] : 1.f);
    }
    // blocks of 16 kSets positions: this warp's, or all; none past the row's end,
    // none where nothing was loaded
    const int blocks = d.pages == 0 ? 0 : (d.nval + 16 * kSets - 1) / (16 * kSets);
    const int blk_end = solo ? blocks : (quarter < blocks ? quarter + 1 : 0);
    for (int blk = solo ? 0 : quarter; blk < blk_end; ++blk) {
      const int r0 = 16 * kSets * blk;
      // ---- S^T = K Q^T
      float sc[kSets][4];
      if constexpr (kSets == 1 && !FP8) {                          // two chains of dependent MMAs
        float odd[4] = {};
        sc[0][0] = sc[0][1] = sc[0][2] = sc[0][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          uint32_t a[4];
          ldsm_x4(address(kbase, r0 + r_a, 2 * kk + c_a), a);
          mma_16816(kk & 1 ? odd : sc[0], a, qf[kk][0], qf[kk][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[0][e] += odd[e];
      } else {
#pragma unroll
        for (int u = 0; u < kSets; ++u) sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.f;
        if constexpr (FP8) {
#pragma unroll
          for (int kp = 0; kp < DH / 32; ++kp)
#pragma unroll
            for (int u = 0; u < kSets; ++u) {
              uint32_t r[4];
              ldsm_x4(address(kbase, r0 + r_a + 16 * u, 2 * kp + c_a), r);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t a[4];
                e4m3x4_to_half2(r[2 * k], a[0], a[2]);
                e4m3x4_to_half2(r[2 * k + 1], a[1], a[3]);
                mma_16816(sc[u], a, qf[2 * kp + k][0], qf[2 * kp + k][1]);
              }
            }
        } else {
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
            for (int u = 0; u < kSets; ++u) {
              uint32_t a[4];
              ldsm_x4(address(kbase, r0 + r_a + 16 * u, 2 * kk + c_a), a);
              mma_16816(sc[u], a, qf[kk][0], qf[kk][1]);
            }
        }
      }
      // ---- positions that do not count (behind the row's end, in absent pages): no
      // weight, and a weight of zero times a NaN would be NaN, so their V rows are
      // cleared in the stage before they are read
      if (d.nval != kTile || d.pages != (1 << (kTile >> page_shift)) - 1) {
        auto valid = [&](int r) { return r < d.nval && ((d.pages >> (r >> page_shift)) & 1); };
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
          const int set = r0 + 16 * u;
          const bool v0 = valid(set + gid), v1 = valid(set + gid + 8);
          if (!v0) sc[u][0] = sc[u][1] = -INFINITY;
          if (!v1) sc[u][2] = sc[u][3] = -INFINITY;
          const int r = set + (lane >> 1);                         // two lanes a row
          if (!valid(r))
#pragma unroll
            for (int c = 0; c < C::kRow / 32; ++c) {
              const uint32_t a = address(vbase, r, 2 * c + (lane & 1));
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
            }
        }
        fence_proxy_async();                                       // before TMA refills the stage
        __syncwarp();
      }
      // ---- running softmax.  A column's reference is a maximum of tiles before; it is
      // raised (the eight lanes of the column agree on the new one, sums and outputs
      // are scaled) only where a weight would leave fp16, rarely after the first tiles
      uint32_t ph[kSets][2], pl[kSets][2];
      float pr[kSets][4];
      float down[2] = {weight_shift(mx[0]), weight_shift(mx[1])};
      bool over = false;
#pragma unroll
      for (int u = 0; u < kSets; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          pr[u][k] = log2_weight(sc[u][k], c2, down[k & 1]);
          over |= pr[u][k] > kWeightMost;
        }
      if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(sc[0][e], sc[0][2 + e]);
#pragma unroll
          for (int u = 1; u < kSets; ++u) top = fmaxf(top, fmaxf(sc[u][e], sc[u][2 + e]));
          top = __fmul_rn(top, c2);
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
          top = fmaxf(mx[e], fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16)));
          const float alpha = ex2(mx[e] - top);
          mx[e] = top;
          l[e] *= alpha;
#pragma unroll
          for (int fb = 0; fb < DH / 16; ++fb) o[fb][e] *= alpha, o[fb][2 + e] *= alpha;
          down[e] = weight_shift(top);
        }
#pragma unroll
        for (int u = 0; u < kSets; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) pr[u][k] = log2_weight(sc[u][k], c2, down[k & 1]);
      }
#pragma unroll
      for (int u = 0; u < kSets; ++u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[u][k] = ex2(pr[u][k]);
        l[0] += pr[u][0] + pr[u][2];
        l[1] += pr[u][1] + pr[u][3];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t hi, lo;
          split_weights(pr[u][2 * r], pr[u][2 * r + 1], hi, lo);
          pl[u][r] = transpose8x8(lo);
          ph[u][r] = transpose8x8(hi);
        }
      }
      // ---- O^T += V^T P^T
      if constexpr (FP8) {
#pragma unroll
        for (int fp = 0; fp < DH / 32; ++fp)
#pragma unroll
          for (int u = 0; u < kSets; ++u) {
            uint32_t r[4];
            ldsm_x4_t(address(vbase, r0 + r_a + 16 * u, 2 * fp + c_a), r);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              // bytes: position 2 tig, features 2 gid and 2 gid + 1; position 2 tig + 1, the same
              uint32_t a[4];
              e4m3x4_to_half2(__byte_perm(r[2 * k], 0, 0x3120), a[0], a[1]);
              e4m3x4_to_half2(__byte_perm(r[2 * k + 1], 0, 0x3120), a[2], a[3]);
              mma_16816(o[2 * fp + k], a, ph[u][0], ph[u][1]);
              mma_16816(o[2 * fp + k], a, pl[u][0], pl[u][1]);
            }
          }
      } else {
#pragma unroll
        for (int fb = 0; fb < DH / 16; ++fb)
#pragma unroll
          for (int u = 0; u < kSets; ++u) {
            uint32_t a[4];
            ldsm_x4_t(address(vbase, r0 + r_t + 16 * u, 2 * fb + c_t), a);
            mma_16816(o[fb], a, ph[u][0], ph[u][1]);
            mma_16816(o[fb], a, pl[u][0], pl[u][1]);
          }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (!(d.flags & kLast)) continue;

    const float vs = FP8 ? p.v_scale[d.head] : 1.f;
    __half* dst = p.out + (int64_t)d.row * p.out_stride + (int64_t)d.head * p.G * DH;
    const int h0 = hb + 2 * tig;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 4);
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 8);
      l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 16);
    }
    if (solo) {
      const float i0 = l[0] == 0.f ? 0.f : vs / l[0], i1 = l[1] == 0.f ? 0.f : vs / l[1];
#pragma unroll
      for (int fb = 0; fb < DH / 16; ++fb)
        store_out<DH, FP8>(dst, h0, p.G, 16 * fb, gid, make_float4(o[fb][0], o[fb][1], o[fb][2], o[fb][3]), i0, i1);
      continue;
    }
    // ---- the four quarters' (max, sum, output) into one, in their order; each
    // group of four warps (8 query heads) by itself
    float lsum[2], mtop[2];
    if (gid == 0)
      *reinterpret_cast<float4*>(&wml[warp][2 * tig]) = make_float4(mx[0], l[0], mx[1], l[1]);
    named_bar_sync(1 + group, 128);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = wml[4 * group + k][2 * tig + e];
      mtop[e] = fmaxf(fmaxf(w[0].x, w[1].x), fmaxf(w[2].x, w[3].x));
      const float base = mtop[e];
      lsum[e] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) lsum[e] = fmaf(w[k].y, ex2(w[k].x - base), lsum[e]);
      const float f = ex2(mx[e] - base);
#pragma unroll
      for (int fb = 0; fb < DH / 16; ++fb) o[fb][e] *= f, o[fb][2 + e] *= f;
    }
    constexpr int kVec = DH / 16 * 32;                           // float4s of one warp's output
    float4* buf = merge + group * 2 * kVec;
    auto put = [&](float4* to) {
#pragma unroll
      for (int fb = 0; fb < DH / 16; ++fb) to[fb * 32 + lane] = make_float4(o[fb][0], o[fb][1], o[fb][2], o[fb][3]);
    };
    if (quarter >= 2) put(buf + (quarter - 2) * kVec);
    named_bar_sync(1 + group, 128);
    if (quarter < 2) {
#pragma unroll
      for (int fb = 0; fb < DH / 16; ++fb) {
        const float4 v = buf[quarter * kVec + fb * 32 + lane];
        o[fb][0] += v.x, o[fb][1] += v.y, o[fb][2] += v.z, o[fb][3] += v.w;
      }
      put(buf + quarter * kVec);
    }
    named_bar_sync(1 + group, 128);
    // every warp adds and stores a quarter of the features
    const bool open = d.flags & (kOpenLeft | kOpenRight);
    const int64_t slot = 2 * (int64_t)blockIdx.x + ((d.flags & kOpenLeft) ? 0 : 1);
    if (open && quarter == 0 && gid == 0)
      *reinterpret_cast<float4*>(&p.ml[slot * 8 * HG + h0]) = make_float4(mtop[0], lsum[0], mtop[1], lsum[1]);
    const float i0 = lsum[0] == 0.f ? 0.f : vs / lsum[0], i1 = lsum[1] == 0.f ? 0.f : vs / lsum[1];
#pragma unroll
    for (int b = 0; b < DH / 64; ++b) {
      const int fb = quarter * (DH / 64) + b;
      const float4 u = buf[fb * 32 + lane], v = buf[kVec + fb * 32 + lane];
      const float4 y = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
      if (open) p.part[slot * HG * kVec + (fb * HG + group) * 32 + lane] = y;
      else store_out<DH, FP8>(dst, h0, p.G, 16 * fb, gid, y, i0, i1);
    }
  }
  if (i == ntiles) return;
  // ---- the wait for tile i ran out.  What the stage says may be an older tile's, and the
  // other warps of the group may still get theirs: this one reads and stores nothing
  // more, but passes the barriers of the merges it has left, which it counts from the
  // rows' lengths as the producers do, so that no barrier waits for it.  Its part of their
  // sums is NaN, and so is what they make of it
  if (lane == 0) record_wait_failure(p.error, kConsumerCode);
  int64_t m = s_first_row;
  int s, T = row_tiles(row_length(p, m, s)), h = (int)(s_first_offset / T);
  for (int64_t at = -(s_first_offset % T);;) {                   // tiles at .. at + T - 1 of the run: a (row, head)
    const int64_t end = at + T;
    if ((end < ntiles ? end : ntiles) > i && !(T == 1 && ntiles > kSoloRun)) {
      if (lane < 8) wml[warp][lane] = make_float2(kNothing, NAN);
      for (int b = 0; b < 3; ++b) named_bar_sync(1 + group, 128);
    }
    if (end >= ntiles) return;
    at = end;
    if (++h == p.heads) {
      h = 0;
      do {                                                       // the next row that has anything
        if (++m == p.M) return;
        T = row_tiles(row_length(p, m, s));
      } while (T == 0);
    }
  }
}

// Joins the partials of each split (row, head), in CTA order.  CTA (x, y): the
// x-th record, float4s 32 y .. 32 y + 31 of the output, which belong to eight
// heads.  Warp w weighs the partials of one head and sums every 8th partial of the
// outputs (the first 32 are on their way while the weights are formed: the chain of
// dependent loads is what this kernel takes); the eight sums are added in warp
// order.
constexpr int kCombineThreads = 256;

template <int DH, bool FP8, int HG>
__global__ void __launch_bounds__(kCombineThreads)
paged_combine_kernel(const Params p) {
  extern __shared__ float wts[];                                 // [partials][8]
  __shared__ float inv[8];
  __shared__ float4 sums[8][32];
  constexpr int kVec = DH / 16 * HG * 32;
  griddep_wait();                                                // in every CTA: the grid ends after its predecessor
  const int4 rec = p.recs[blockIdx.x];
  const int J = rec.z;
  // 0: not split.  A record that no call wrote (a workspace that unordered calls share) is not followed.
  if (J <= 0 || rec.y < 0 || J > p.ctas - rec.y || rec.x < 0 || rec.x >= p.M * p.heads) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = rec.x / p.heads, head = rec.x % p.heads;
  const int vec = blockIdx.y * 32 + lane, fb = blockIdx.y / HG, nt = blockIdx.y % HG;
  auto slot = [&](int j) -> int64_t { return 2 * (int64_t)(rec.y + j) + (j == 0 ? 1 : 0); };
  float4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (warp + 8 * k < J) v[k] = p.part[slot(warp + 8 * k) * kVec + vec];
  {
    const float2* ml = p.ml + 8 * nt + warp;
    const float2 none = make_float2(-INFINITY, 0.f), first = lane < J ? ml[slot(lane) * 8 * HG] : none;
    float top = first.x;
    for (int j = lane + 32; j < J; j += 32) top = fmaxf(top, ml[slot(j) * 8 * HG].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int j = lane; j < J; j += 32) {
      const float2 u = j == lane ? first : ml[slot(j) * 8 * HG];
      const float w = ex2(u.x - base);
      wts[j * 8 + warp] = w;
      sum = fmaf(w, u.y, sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) inv[warp] = sum == 0.f ? 0.f : (FP8 ? p.v_scale[head] : 1.f) / sum;
  }
  __syncthreads();
  const int gid = lane >> 2, tig = lane & 3;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = warp; j0 < J; j0 += 32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + 8 * k;
      if (j >= J) break;
      const float2 w = *reinterpret_cast<const float2*>(&wts[j * 8 + 2 * tig]);
      acc.x = fmaf(w.x, v[k].x, acc.x), acc.y = fmaf(w.y, v[k].y, acc.y);
      acc.z = fmaf(w.x, v[k].z, acc.z), acc.w = fmaf(w.y, v[k].w, acc.w);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j0 + 32 + 8 * k < J) v[k] = p.part[slot(j0 + 32 + 8 * k) * kVec + vec];
  }
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    const float4 u = sums[w][lane];
    acc.x += u.x, acc.y += u.y, acc.z += u.z, acc.w += u.w;
  }
  store_out<DH, FP8>(p.out + (int64_t)row * p.out_stride + (int64_t)head * p.G * DH, 8 * nt + 2 * tig, p.G, 16 * fb,
                     gid, acc, inv[2 * tig], inv[2 * tig + 1]);
}

// The same join where splits have few parts: a warp per record and 32 float4s of the
// output, which takes the parts four at a time; no barrier, an eighth of the CTAs.
template <int DH, bool FP8, int HG>
__global__ void __launch_bounds__(32 * DH / 16 * HG)
paged_combine_few_kernel(const Params p) {
  constexpr int kVec = DH / 16 * HG * 32;
  griddep_wait();
  const int4 rec = p.recs[blockIdx.x];
  const int J = rec.z;
  if (J <= 0 || rec.y < 0 || J > p.ctas - rec.y || rec.x < 0 || rec.x >= p.M * p.heads) return;
  const int block = threadIdx.x >> 5, lane = threadIdx.x & 31, fb = block / HG, group = block % HG;
  const int row = rec.x / p.heads, head = rec.x % p.heads;
  auto slot = [&](int j) -> int64_t { return 2 * (int64_t)(rec.y + j) + (j == 0 ? 1 : 0); };
  // lane 8 k + e: (max, sum) of head e in the k-th of four parts
  auto stats = [&](int j0) {
    const int j = j0 + (lane >> 3);
    return j < J ? p.ml[slot(j) * 8 * HG + 8 * group + (lane & 7)] : make_float2(-INFINITY, 0.f);
  };
  auto parts = [&](int j0, float4 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = j0 + k < J ? p.part[slot(j0 + k) * kVec + block * 32 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 v[4];
  parts(0, v);
  float2 ml = stats(0);
  float top = ml.x;
  for (int j0 = 4; j0 < J; j0 += 4) top = fmaxf(top, stats(j0).x);
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
  const float base = top == -INFINITY ? 0.f : top;
  const int gid = lane >> 2, tig = lane & 3;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < J; j0 += 4) {
    if (j0 > 0) ml = stats(j0), parts(j0, v);
    const float w = ex2(ml.x - base);
    sum = fmaf(w, ml.y, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = __shfl_sync(0xFFFFFFFFu, w, 8 * k + 2 * tig), b = __shfl_sync(0xFFFFFFFFu, w, 8 * k + 2 * tig + 1);
      acc.x = fmaf(a, v[k].x, acc.x), acc.y = fmaf(b, v[k].y, acc.y);
      acc.z = fmaf(a, v[k].z, acc.z), acc.w = fmaf(b, v[k].w, acc.w);
    }
  }
  sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
  sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
  const float inv = sum == 0.f ? 0.f : (FP8 ? p.v_scale[head] : 1.f) / sum;
  const float i0 = __shfl_sync(0xFFFFFFFFu, inv, 2 * tig), i1 = __shfl_sync(0xFFFFFFFFu, inv, 2 * tig + 1);
  store_out<DH, FP8>(p.out + (int64_t)row * p.out_stride + (int64_t)head * p.G * DH, 8 * group + 2 * tig, p.G, 16 * fb,
                     gid, acc, i0, i1);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn_p() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return nullptr;
  }();
  return fn;
}

constexpr int kMaxCtasPerSm = 3;
// parts per (row, head), as CTAs over (row, head)s, up to which the small join is used: at 4.6 it took
// 11.8 us against 12.0 (8 rows x 1000 x 8 heads, both kernels), at 2.3 45.9 against 47.9 (16 x 4096), at
// 7.4 17.4 against 16.6 (5 x 4000), at 37 17.0 against 10.7 (1 x 4096)
constexpr int kFewParts = 6;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct Space {
  size_t ml, part, total;
};
Space space(int64_t ctas, int64_t hg, int64_t dh) {
  Space w;
  w.ml = up256((size_t)ctas * sizeof(int4));
  w.part = w.ml + up256((size_t)(2 * ctas * 8 * hg) * sizeof(float2));
  w.total = w.part + (size_t)(2 * ctas * 8 * hg * dh) * sizeof(float);
  return w;
}

template <int DH, bool FP8, int HG>
cudaError_t launch(Params p, const tri_paged_cache& c, void* ws, int sms, cudaStream_t s) {
  using K = Cfg<DH, FP8, HG>;
  auto enc = encode_fn_p();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap maps[2];
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[3] = {(cuuint64_t)DH, (cuuint64_t)(c.heads * c.page_size), (cuuint64_t)c.pages};
    const cuuint64_t strides[2] = {(cuuint64_t)K::kRow, (cuuint64_t)c.page_stride * (FP8 ? 1 : 2)};
    const cuuint32_t box[3] = {(cuuint32_t)(K::kBox / (FP8 ? 1 : 2)),
                               (cuuint32_t)(c.page_size < K::kTile ? c.page_size : K::kTile), 1};
    const cuuint32_t es[3] = {1, 1, 1};
    if (enc(&maps[i], FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, i ? c.v : c.k, dims,
            strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            K::kBox == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  cudaError_t e = wait_status_word(&p.error);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> ready[64] = {};                      // host threads may call at once
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(paged_attn_kernel<DH, FP8, HG>, cudaFuncAttributeMaxDynamicSharedMemorySize, K::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  // no more CTAs than tiles can exist
  const int64_t most = p.M * p.heads * (int64_t)((p.max_len + K::kTile - 1) / K::kTile);
  const int64_t ctas = most < (int64_t)K::kCtasPerSm * sms ? most : (int64_t)K::kCtasPerSm * sms;
  p.ctas = (int)ctas;
  const Space w = space(ctas, HG, DH);
  p.recs = static_cast<int4*>(ws);
  p.ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + w.ml);
  p.part = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + w.part);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = K::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<DH, FP8, HG>, maps[0], maps[1], p)) != cudaSuccess) return e;
  if (p.max_len <= K::kTile) return cudaSuccess;                 // one tile a row at most: nothing is split
  const int64_t segs = p.M * p.heads;
  if (ctas <= kFewParts * segs) {
    cfg.gridDim = dim3((unsigned)(segs < ctas ? segs : ctas));
    cfg.blockDim = dim3(32 * DH / 16 * HG);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_combine_few_kernel<DH, FP8, HG>, p);
  }
  cfg.gridDim = dim3((unsigned)(segs < ctas ? segs : ctas), DH / 16 * HG);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.dynamicSmemBytes = (size_t)ctas * 8 * sizeof(float);
  return cudaLaunchKernelEx(&cfg, paged_combine_kernel<DH, FP8, HG>, p);
}

}  // namespace

size_t paged_attention_ws_bytes(int64_t, int64_t H, int64_t heads, int64_t head_dim, int sms) {
  return up256(space((int64_t)kMaxCtasPerSm * sms, H / heads > 8 ? 2 : 1, head_dim).total);
}

cudaError_t launch_paged_attention(const __half* q, int64_t q_stride, const int* pos, const int* seq,
                                   const tri_paged_cache& c, __half* out, int64_t out_stride, int64_t M,
                                   int64_t H, float scale, void* ws, int sms, cudaStream_t s) {
  Params p = {};
  p.q = q, p.pos = pos, p.seq = seq, p.table = c.table, p.k_scale = c.k_scale, p.v_scale = c.v_scale, p.out = out;
  p.q_stride = q_stride, p.out_stride = out_stride, p.table_stride = c.table_stride, p.M = M;
  p.heads = (int)c.heads, p.G = (int)(H / c.heads), p.pages = (int)c.pages, p.seqs = (int)c.seqs;
  p.max_len = (int)(c.seq_pages * c.page_size), p.scale = scale, p.polls = wait_polls();
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  const bool fp8 = c.dtype == TRI_CACHE_E4M3, wide = p.G > 8;
  if (c.head_dim == 128) {
    if (fp8) return wide ? launch<128, true, 2>(p, c, ws, sms, s) : launch<128, true, 1>(p, c, ws, sms, s);
    return wide ? launch<128, false, 2>(p, c, ws, sms, s) : launch<128, false, 1>(p, c, ws, sms, s);
  }
  if (fp8) return wide ? launch<64, true, 2>(p, c, ws, sms, s) : launch<64, true, 1>(p, c, ws, sms, s);
  return wide ? launch<64, false, 2>(p, c, ws, sms, s) : launch<64, false, 1>(p, c, ws, sms, s);
}

}  // namespace tri

// The gated delta rule in chunks of 64 tokens on the tensor cores (bf16 rows).
//
// With G_i the sum of the chunk's log decays up to token i, e_ij = exp(G_i -
// G_j), w_i = exp(G_C - G_i) and S the state at the chunk's start:
//   L_ij = e_ij k_i.k_j (j < i),  T = (I + diag(beta) L)^-1,
//   R = V - diag(e^G) K S,  U = T diag(beta) R,
//   P_ij = scale e_ij q_i.k_j (j <= i),  O = scale diag(e^G) Q S + P U,
//   S+ = e^G_C S + K^T diag(w) U
// T and P need no state: one kernel forms them for all chunks at once
// (delta_prep_kernel). What is left is the walk over the chunks.
//
// The walk runs transposed: S^T = [d_v, d_k]. The d_v rows are independent, so a
// warp owns 16 of them for the whole sequence with S^T in fp32 registers, and
// the fragments of one product's result are the left operand of the next
// (S^T K^T -> R^T -> U^T -> U^T K): no exchange between warps, no shared memory
// round trip on the chain from chunk to chunk. That chain bounds the kernel
// (sequences x heads x d / 16 warps, each one chunk after another), which is why
// it uses the warp-level products: their latency is tens of cycles, against the
// round trips through TMEM that three dependent products of a tcgen05 form
// would add to every chunk (a tcgen05 walk with one head per SM was measured at
// 10,000 cycles a chunk; the conversions between its products took 1200 each).
// Measured on two sequences of 6000-8192 tokens, 16 / 32 heads, d = 128: prep 113 us,
// walk 340 us, 2.7 us or 5000 cycles a chunk, of which the walking warp's products
// are 2530 at the warp-level rate (m16n8k16 in 8 cycles) and its conversions the rest.
//
// Precision: products whose results enter the state take each fp32 factor as a
// bf16 and the bf16 of the rest (16 bits or more; k, q, v and dout are bf16
// already), 2 or 3 products accumulated in fp32. S, U and P are rounded to one
// bf16 only where the result is a bf16 output.
#pragma once

#include <type_traits>

#include "delta_common.cuh"
#include "sm100.cuh"

namespace infini {

constexpr int kDcTok = 64;  // tokens of a chunk
constexpr uint32_t kDcMat = kDcTok * kDcTok * 2;  // a 64 x 64 bf16 matrix, 128-byte rows, 16-byte pieces swizzled

// What the prep kernel leaves for each (chunk, value head).
struct DcRecord {
  static constexpr uint32_t kThi = 0, kTlo = kDcMat, kPhi = 2 * kDcMat, kPlo = 3 * kDcMat;
  static constexpr uint32_t kVec = 4 * kDcMat;  // e^G, w, beta (fp32), G (fp64)
  static constexpr uint32_t kVecBytes = kDcTok * (3 * 4 + 8);
  static constexpr uint32_t kBytes = kVec + kVecBytes;
};
static_assert(DcRecord::kBytes % 256 == 0, "records stay aligned");

__device__ __forceinline__ int64_t dc_slot(const SeqRange& r, int seq, int c) {
  return (int64_t)(r.first / kDcTok) + seq + c;
}

// ------------------------------------------------------------ warp products
__device__ __forceinline__ uint32_t dc_smem(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16-byte piece `c` of row `r` in a tile with rows of RB bytes (128 or 256), or
// (kDcBlocks) as TMA lays out 64 rows: blocks of 64 columns, 128-byte rows each.
constexpr int kDcBlocks = 1;
template <int RB>
__device__ __forceinline__ uint32_t dc_at(int r, int c) {
  if constexpr (RB == kDcBlocks)
    return (uint32_t)((c >> 3) * (kDcTok * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
  else
    return (uint32_t)(r * RB + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ void ldsm(uint32_t (&f)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&f)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stsm(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c[x] += (hi + lo) b for N (a multiple of 2) neighbouring 16 x 8 tiles whose right operands lie in b[x / 2]:
// first all hi, then all lo, so that no product waits for the one before it.
template <int N>
__device__ __forceinline__ void mma_parts(float (*c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                                          const uint32_t (&b)[N / 2][4]) {
#pragma unroll
  for (int x = 0; x < N; ++x) mma16(c[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
  for (int x = 0; x < N; ++x) mma16(c[x], lo, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
}
// Addresses of the four 8 x 8 blocks that a lane names, by what they become:
// the right operand (columns n .. n + 15, 16 of k) from rows = n, or (t) from
// rows = k; the left operand (rows m .. m + 15, 16 of k) from rows = m, or (t)
// from rows = k. `c` counts 16-byte pieces.
template <int RB>
__device__ __forceinline__ uint32_t right_at(int n, int c, int lane) {
  return dc_at<RB>(n + ((lane >> 4) << 3) + (lane & 7), c + ((lane >> 3) & 1));
}
template <int RB>
__device__ __forceinline__ uint32_t right_t_at(int k, int c, int lane) {
  return dc_at<RB>(k + (((lane >> 3) & 1) << 3) + (lane & 7), c + (lane >> 4));
}
template <int RB>
__device__ __forceinline__ uint32_t left_at(int m, int c, int lane) {
  return right_t_at<RB>(m, c, lane);
}
template <int RB>
__device__ __forceinline__ uint32_t left_t_at(int k, int c, int lane) {
  return right_at<RB>(k, c, lane);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float low_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// x = hi + lo with hi = bf16(x), lo = bf16(x - hi).
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2(x, y);
  lo = pack2(x - low_f(hi), y - high_f(hi));
}
// Two neighbouring result tiles (16 x 8 each) as a left operand (16 x 16).
__device__ __forceinline__ void as_left(const float (&t0)[4], const float (&t1)[4], uint32_t (&hi)[4],
                                        uint32_t (&lo)[4]) {
  split2(t0[0], t0[1], hi[0], lo[0]);
  split2(t0[2], t0[3], hi[1], lo[1]);
  split2(t1[0], t1[1], hi[2], lo[2]);
  split2(t1[2], t1[3], hi[3], lo[3]);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: zeros are written and nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// 64 rows of W elements from element `col` on, rows behind `valid` as zeros.
template <int W, int NT>
__device__ __forceinline__ void dc_load_rows(uint32_t dst, const RowsOf<const __nv_bfloat16>& x, int64_t row, int h,
                                             int col, int valid, int tid) {
  constexpr int P = W / 8;
  for (int i = tid; i < kDcTok * P; i += NT) {
    const int r = i / P, c = i % P;
    const bool real = r < valid;
    cp16(dst + dc_at<W * 2>(r, c), x.at(row + (real ? r : 0), h) + col + c * 8, real);
  }
}
template <int NT>
__device__ __forceinline__ void dc_load_flat(uint32_t dst, const uint8_t* src, uint32_t bytes, int tid) {
  for (uint32_t i = tid * 16; i < bytes; i += NT * 16) cp16(dst + i, src + i, true);
}

// ------------------------------------------------------------------- prep
// CTA = (chunk, key head): k_i.k_j and q_i.k_j once, kept as result fragments
// (warp w: rows 16 w ..), then T and P for each value head of the group; only
// the blocks of 16 x 16 on and below the diagonal exist. Decays between blocks
// are products of two exponentials, both of sums that run one way (e_ij =
// exp(G_i - G_b) exp(G_b - G_j), b the start of i's block): no overflow, and few
// exponentials. T by blocks: the diagonal ones by substitution in fp32 (a column
// per lane), then X21 = -T22 (N21 T11) over blocks of 16 and of 32, whose
// products run on the tensor cores with both factors in two parts (2^-16 of the
// off-diagonal blocks; T leaves in two parts anyway). These products are small
// and dependent, so the kernel lives on CTAs per SM. TINY (for gradients): a
// |beta| below 2^-110, 0 too, is taken as 2^-110 with beta's sign, so that beta's own
// gradient, a ratio over what beta scales, exists there and keeps its digits (what
// beta scales is kept as bf16, which ends at 2^-126). Such a token's dv counts as 0.
// Measured: 7100 chunks of (64 tokens, value head), two heads a CTA: 113 us.
constexpr float kDpTiny = 0x1p-110f;
constexpr int kDpThreads = 128;
constexpr int kDpSt = 17;  // row stride of a diagonal block
template <int D>
struct DpSmem {
  static constexpr uint32_t kRows = 2 * kDcTok * D * 2;
  // T's parts, Y's parts (32 x 32 in 128-byte rows), the diagonal blocks of N: in the place of K and Q.
  static constexpr uint32_t kT = 0, kY = 2 * kDcMat, kN = kY + 2 * 32 * 128, kMats = kN + 4 * 16 * kDpSt * 4;
  static constexpr uint32_t kSmall = kRows > kMats ? kRows : (kMats + 127) / 128 * 128;
  // G (fp64), beta, exp(G_i - G_b), exp(G_b - G_j)
  static constexpr uint32_t kTotal = kSmall + kDcTok * (8 + 4 + 4 + 4 * 4) + 128;
};

// An 8 x 8 block of bf16 pairs turned over: from rows to columns across the warp.
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c[x] += a b, both in two parts (without lo lo), for two tiles whose right operands are b[0..1] and b[2..3].
__device__ __forceinline__ void mma_both(float (&c0)[4], float (&c1)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                         const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
  mma16(c0, ah, bh[0], bh[1]);
  mma16(c1, ah, bh[2], bh[3]);
  mma16(c0, al, bh[0], bh[1]);
  mma16(c1, al, bh[2], bh[3]);
  mma16(c0, ah, bl[0], bl[1]);
  mma16(c1, ah, bl[2], bl[3]);
}
// Two result tiles (rows m .., columns 8 c ..) times `sign`, in two parts, into two tiles of 128-byte rows.
__device__ __forceinline__ void put_parts(uint32_t hi_tile, uint32_t lo_tile, int m, int c, int lane, const float (&t0)[4],
                                          const float (&t1)[4], float sign) {
  uint32_t hi[4], lo[4];
  split2(sign * t0[0], sign * t0[1], hi[0], lo[0]);
  split2(sign * t0[2], sign * t0[3], hi[1], lo[1]);
  split2(sign * t1[0], sign * t1[1], hi[2], lo[2]);
  split2(sign * t1[2], sign * t1[3], hi[3], lo[3]);
  const uint32_t at = left_at<128>(m, c, lane);
  stsm(hi_tile + at, hi[0], hi[1], hi[2], hi[3]);
  stsm(lo_tile + at, lo[0], lo[1], lo[2], lo[3]);
}

template <int D, bool TINY>
__global__ void __launch_bounds__(kDpThreads, 4)
delta_prep_kernel(RowsOf<const __nv_bfloat16> q, RowsOf<const __nv_bfloat16> k, RowsOf<const __nv_bfloat16> g,
                  RowsOf<const __nv_bfloat16> beta, SeqTable seqs, int Hv, int G, float scale,
                  uint8_t* __restrict__ records) {
  using M = DpSmem<D>;
  extern __shared__ __align__(1024) uint8_t dc_smem_raw[];
  uint8_t* mem = dc_smem_raw + ((128 - (dc_smem(dc_smem_raw) & 127)) & 127);
  double* Gd = reinterpret_cast<double*>(mem + M::kSmall);
  float* be = reinterpret_cast<float*>(Gd + kDcTok);
  float* in = be + kDcTok;   // exp(G_i - G_b)
  float* out = in + kDcTok;  // [4][64]: exp(G_b - G_j), j < 16 b
  const uint32_t sK = dc_smem(mem), sQ = sK + kDcTok * D * 2;
  const uint32_t Th = sK + M::kT, Tl = Th + kDcMat, Yh = sK + M::kY, Yl = Yh + 32 * 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, qd = lane & 3, hk = blockIdx.y;
  SlotTile t;
  if (!chunk_tile<kDcTok>(seqs, blockIdx.x, &t)) return;
  const int n = min(kDcTok, t.r.len - t.tile * kDcTok);
  const int64_t row0 = t.r.first + t.tile * kDcTok;
  dc_load_rows<D, kDpThreads>(sK, k, row0, hk, 0, n, tid);
  dc_load_rows<D, kDpThreads>(sQ, q, row0, hk, 0, n, tid);
  cp_commit();
  const bool found = tile_found<kDcTok>(seqs, t);
  cp_wait();
  if (!found) return;
  __syncthreads();
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int x = 0; x < 8; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) kk[x][y] = qk[x][y] = 0.f;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    uint32_t ak[4], aq[4];
    ldsm(ak, sK + left_at<D * 2>(16 * warp, 2 * s, lane));
    ldsm(aq, sQ + left_at<D * 2>(16 * warp, 2 * s, lane));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x > warp) continue;
      uint32_t b[4];
      ldsm(b, sK + right_at<D * 2>(16 * x, 2 * s, lane));
      mma16(kk[2 * x], ak, b[0], b[1]);
      mma16(kk[2 * x + 1], ak, b[2], b[3]);
      mma16(qk[2 * x], aq, b[0], b[1]);
      mma16(qk[2 * x + 1], aq, b[2], b[3]);
    }
  }
  for (int u = blockIdx.z; u < G; u += gridDim.z) {
    const int h = hk * G + u;
    uint8_t* rec = records + (dc_slot(t.r, t.seq, t.tile) * Hv + h) * (int64_t)DcRecord::kBytes;
    float* vec = reinterpret_cast<float*>(rec + DcRecord::kVec);
    __syncthreads();
    if (warp == 0) {  // sums of log decays in 64 bits; lane has tokens 2 lane, 2 lane + 1
      double x[2];
      float b[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 2 * lane + y;
        x[y] = i < n ? (double)delta_log(to_f32(*g.at(row0 + i, h))) : 0.0;
        b[y] = i < n ? to_f32(*beta.at(row0 + i, h)) : 0.f;
        if (TINY && fabsf(b[y]) < kDpTiny) b[y] = copysignf(kDpTiny, b[y]);
      }
      double sum = x[0] + x[1];
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane >= s) sum += y;
      }
      const double G2[2] = {sum - x[1], sum};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        Gd[2 * lane + y] = G2[y];
        be[2 * lane + y] = b[y];
      }
    }
    __syncthreads();
    {
      const int i = tid & 63;
      if (tid < kDcTok) {
        in[i] = expf((float)(Gd[i] - Gd[i & 48]));
        vec[i] = expf((float)Gd[i]);
        vec[2 * kDcTok + i] = be[i];
        out[1 * kDcTok + i] = i < 16 ? expf((float)(Gd[16] - Gd[i])) : 0.f;
      } else {
        vec[kDcTok + i] = expf((float)(Gd[kDcTok - 1] - Gd[i]));
        reinterpret_cast<double*>(vec + 3 * kDcTok)[i] = Gd[i];
        out[2 * kDcTok + i] = i < 32 ? expf((float)(Gd[32] - Gd[i])) : 0.f;
        out[3 * kDcTok + i] = i < 48 ? expf((float)(Gd[48] - Gd[i])) : 0.f;
      }
    }
    __syncthreads();
    // P, and N = diag(beta) L: its diagonal block to shared memory, the blocks
    // left of it stay as (two-part) left operands nl, 16 columns each.
    const float in0 = in[16 * warp + gr], in1 = in[16 * warp + gr + 8];
    const float be0 = be[16 * warp + gr], be1 = be[16 * warp + gr + 8];
    float* Nb = reinterpret_cast<float*>(mem + M::kN) + warp * 16 * kDpSt;
    uint32_t nh[3][4], nl[3][4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x > warp) continue;
      float nn[2][4];
#pragma unroll
      for (int z = 0; z < 2; ++z) {  // the block's two tiles of 8 columns
        const int tile = 2 * x + z;
        float e[4];
        if (x < warp) {
          const float2 o = *reinterpret_cast<const float2*>(out + warp * kDcTok + 8 * tile + 2 * qd);
          e[0] = in0 * o.x;
          e[1] = in0 * o.y;
          e[2] = in1 * o.x;
          e[3] = in1 * o.y;
        } else {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int i = 16 * warp + gr + 8 * (y >> 1), j = 8 * tile + 2 * qd + (y & 1);
            e[y] = j <= i ? expf((float)(Gd[i] - Gd[j])) : 0.f;
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // rows gr, gr + 8
          uint32_t hi, lo;
          split2(scale * e[2 * y] * qk[tile][2 * y], scale * e[2 * y + 1] * qk[tile][2 * y + 1], hi, lo);
          const uint32_t at = dc_at<128>(16 * warp + gr + 8 * y, tile) + qd * 4;
          *reinterpret_cast<uint32_t*>(rec + DcRecord::kPhi + at) = hi;
          if (TINY) *reinterpret_cast<uint32_t*>(rec + DcRecord::kPlo + at) = lo;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          nn[z][y] = (y >> 1 ? be1 : be0) * e[y] * kk[tile][y];
          if (x == warp) Nb[(gr + 8 * (y >> 1)) * kDpSt + 8 * z + 2 * qd + (y & 1)] = nn[z][y];
        }
      }
      if (x < 3 && x < warp) as_left(nn[0], nn[1], nh[x], nl[x]);
    }
    __syncwarp();
    if (lane < 16) {  // column `lane` of the warp's diagonal block of T
      float x[16];
      uint16_t* th = reinterpret_cast<uint16_t*>(mem + M::kT);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) {
          if (j & 1)
            s1 = fmaf(-Nb[i * kDpSt + j], x[j], s1);
          else
            s0 = fmaf(-Nb[i * kDpSt + j], x[j], s0);
        }
        x[i] = i < lane ? 0.f : s0 + s1;
        const uint32_t hi = pack2(x[i], 0.f), lo = pack2(x[i] - low_f(hi), 0.f);
        const uint32_t at = (dc_at<128>(16 * warp + i, 2 * warp + (lane >> 3)) >> 1) + (lane & 7);
        th[at] = (uint16_t)hi;
        th[kDcMat / 2 + at] = (uint16_t)lo;
      }
    }
    __syncthreads();
    if (warp & 1) {  // block (w, w - 1), w = 1, 3: X = -T_ww (N_w,w-1 T_w-1,w-1)
      float y0[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t bh[4], bl[4], ah[4], al[4];
      const int p = warp - 1;
      ldsm_t(bh, Th + right_t_at<128>(16 * p, 2 * p, lane));
      ldsm_t(bl, Tl + right_t_at<128>(16 * p, 2 * p, lane));
      if (warp == 1)
        mma_both(y0, y1, nh[0], nl[0], bh, bl);
      else
        mma_both(y0, y1, nh[2], nl[2], bh, bl);
      as_left(y0, y1, ah, al);  // rows of Y; turned over they are a right operand
      const uint32_t rh[4] = {turn(ah[0]), turn(ah[1]), turn(ah[2]), turn(ah[3])};
      const uint32_t rl[4] = {turn(al[0]), turn(al[1]), turn(al[2]), turn(al[3])};
      float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
      ldsm(ah, Th + left_at<128>(16 * warp, 2 * warp, lane));
      ldsm(al, Tl + left_at<128>(16 * warp, 2 * warp, lane));
      mma_both(x0, x1, ah, al, rh, rl);
      put_parts(Th, Tl, 16 * warp, 2 * p, lane, x0, x1, -1.f);
    }
    __syncthreads();
    if (warp >= 2) {  // Y = N21 T11, rows 16 (w - 2) .. of 32
      float y[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int z = 0; z < 4; ++z) y[x][z] = 0.f;
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int c = 0; c <= z; ++c) {
          uint32_t bh[4], bl[4];
          ldsm_t(bh, Th + right_t_at<128>(16 * z, 2 * c, lane));
          ldsm_t(bl, Tl + right_t_at<128>(16 * z, 2 * c, lane));
          mma_both(y[2 * c], y[2 * c + 1], nh[z], nl[z], bh, bl);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) put_parts(Yh, Yl, 16 * (warp - 2), 2 * c, lane, y[2 * c], y[2 * c + 1], 1.f);
    }
    __syncthreads();
    {  // X21 = -T22 Y: warps 0, 1 the first 16 rows, 2, 3 the others; 16 columns each
      const int m = 32 + 16 * (warp >> 1), c = 2 * (warp & 1);
      float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (z > (warp >> 1)) continue;
        uint32_t ah[4], al[4], bh[4], bl[4];
        ldsm(ah, Th + left_at<128>(m, 4 + 2 * z, lane));
        ldsm(al, Tl + left_at<128>(m, 4 + 2 * z, lane));
        ldsm_t(bh, Yh + right_t_at<128>(16 * z, c, lane));
        ldsm_t(bl, Yl + right_t_at<128>(16 * z, c, lane));
        mma_both(x0, x1, ah, al, bh, bl);
      }
      put_parts(Th, Tl, m, c, lane, x0, x1, -1.f);
    }
    __syncthreads();
    // T's parts leave as they lie, in pieces of 16 bytes; row i has 2 (i / 16) + 2.
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = 16 * x + (tid >> 3), c = tid & 7;
      if (c >= 2 * x + 2) continue;
      const uint32_t at = dc_at<128>(i, c);
      *reinterpret_cast<uint4*>(rec + DcRecord::kThi + at) = *reinterpret_cast<const uint4*>(mem + M::kT + at);
      *reinterpret_cast<uint4*>(rec + DcRecord::kTlo + at) = *reinterpret_cast<const uint4*>(mem + M::kT + kDcMat + at);
    }
  }
}

// ------------------------------------------------------------------- walk
__device__ __forceinline__ void dc_tma(uint32_t dst, const CUtensorMap* m, int x, int h, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(h), "r"(row), "r"(sm100::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void dc_bulk(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}
// 64 rows x D columns from column x on.
template <int D>
__device__ __forceinline__ void dc_tma_rows(uint32_t dst, const CUtensorMap* m, int x, int h, int row, uint64_t* bar) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) dc_tma(dst + b * kDcTok * 128, m, x + 64 * b, h, row, bar);
}
// Rows [n, 64) of such a tile to zero, by a warp (what lies behind a sequence may be anything).
template <int D>
__device__ __forceinline__ void dc_zero_rows(uint32_t tile, int n, int lane) {
  for (int i = n * 8 + lane; i < kDcTok * 8; i += 32)
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * kDcTok * 128 + i * 16), "r"(0) : "memory");
}
// Barriers of a walk: full[i & 1] of step i's copies (one arrival), tail for a
// last chunk that ends behind its sequence (its rows are zeroed before full).
struct DcBars {
  uint64_t *full, *tail;
};
__device__ __forceinline__ DcBars dc_bars_init(uint64_t* at) {
  if (threadIdx.x == 0) {
    for (int b = 0; b < 3; ++b) sm100::mbar_init(at + b, 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  return {at, at + 2};
}
// After a wait that gave up the walk runs on over what is there (its barriers
// have to be met by every warp); the status word has the error.
__device__ __forceinline__ void dc_wait(uint64_t* bar, int phase, uint32_t epoch) {
  sm100::mbar_wait(bar, phase & 1, epoch);
  __syncwarp();
}
// Before the CTA ends after such a wait: its own copies have landed.
__device__ __forceinline__ void dc_drain(const DcBars& b, uint32_t epoch) {
  if (threadIdx.x == 0 && *reinterpret_cast<volatile unsigned int*>(&g_abort_epoch) == epoch)
    for (int x = 0; x < 3; ++x) {
      sm100::mbar_drain(b.full + x, 0);
      sm100::mbar_drain(b.full + x, 1);
    }
}

// Warps 0-3 walk (16 rows of S^T each); warps 4-7 bring in the next chunk and,
// one chunk behind, do for the same rows what the chain does not wait for. A
// walking warp alone leaves the tensor core of its quarter of the SM idle half
// of the time (its own conversions and copies issue in between); its partner
// fills that. One barrier per chunk.
constexpr int kDwThreads = 256;
constexpr int kDwRows = 64;  // rows of S^T (values) of a CTA: 16 per warp

// What a walking warp hands to its partner, as operand or result fragments (16
// bytes a lane): S^T as bf16 left operands and U^T in fp32.
template <int D>
struct DwHand {
  static constexpr uint32_t kS = 0, kU = D / 16 * 512, kWarp = kU + 8 * 512, kBytes = 4 * kWarp;
};

// GRADS: keeps U (rows [T][Hv][D]) and S at each chunk's start ([slot][Hv], S^T
// as bf16 [d_v][d_k]) for the gradient instead of writing out.
template <int D, bool GRADS>
struct DwSmem {
  static constexpr uint32_t kRow = kDcTok * D * 2, kVal = kDcTok * kDwRows * 2, kVecBytes = 3 * kDcTok * 4;
  // Tiles that TMA swizzles (K, V, Q) start on 1024 bytes.
  static constexpr uint32_t kK = 0, kT = kK + 2 * kRow, kV = kT + 4 * kDcMat, kQ = kV + 2 * kVal,
                            kP = kQ + (GRADS ? 0 : 3 * kRow), kHand = kP + (GRADS ? 0 : 3 * kDcMat),
                            kOut = kHand + 2 * DwHand<D>::kBytes, kVec = kOut + kVal + (GRADS ? kDwRows * D * 2 : 0),
                            kBars = kVec + 3 * kVecBytes, kTotal = kBars + 64;
  static_assert(kTotal <= 232448, "walk kernel shared memory");
};

// 64 tokens x 16 values of fragments [8][4] (rows = values) to rows of `dst`, through this warp's columns of a tile.
template <typename AT>
__device__ __forceinline__ void dc_store_tokens(const float (*f)[4], uint32_t tile, int strip, int lane, int n, AT at) {
  __syncwarp();
#pragma unroll
  for (int x = 0; x < 8; x += 2)
    stsm_t(tile + right_at<128>(8 * x, 2 * strip, lane), pack2(f[x][0], f[x][1]), pack2(f[x][2], f[x][3]),
           pack2(f[x + 1][0], f[x + 1][1]), pack2(f[x + 1][2], f[x + 1][3]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = (lane >> 1) + 16 * i, pc = lane & 1;
    if (tok < n)
      *reinterpret_cast<uint4*>(at(tok) + pc * 8) =
          *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(tile + dc_at<128>(tok, 2 * strip + pc)));
  }
}
// A warp's 16 rows of S^T, handed over as left operands, to 16 rows of D bf16 in global memory.
template <int D>
__device__ __forceinline__ void dc_store_state(uint32_t hand, uint32_t st, int lane, __nv_bfloat16* dst) {
  constexpr int RB = D * 2, NK = D / 8;
  __syncwarp();
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint4 f = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(hand + kk * 512 + lane * 16));
    stsm(st + dc_at<RB>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)), f.x, f.y, f.z, f.w);
  }
  __syncwarp();
#pragma unroll
  for (int i = lane; i < 16 * NK; i += 32) {
    const int rr = i / NK, pc = i % NK;
    *reinterpret_cast<uint4*>(dst + rr * D + pc * 8) =
        *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(st + dc_at<RB>(rr, pc)));
  }
}
__device__ __forceinline__ void dc_hand(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, bool GRADS>
__global__ void __launch_bounds__(kDwThreads, 1)
delta_walk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                  const __grid_constant__ CUtensorMap tmV, const DeltaArgs<__nv_bfloat16> a,
                  const uint8_t* __restrict__ records, __nv_bfloat16* __restrict__ kept_S,
                  __nv_bfloat16* __restrict__ kept_U, uint32_t epoch) {
  using M = DwSmem<D, GRADS>;
  using X = DwHand<D>;
  constexpr int RB = D * 2, NK = D / 8;  // bytes of a row of the state; 8-wide column tiles of S^T
  constexpr int RK = kDcBlocks;          // K and Q
  extern __shared__ __align__(1024) uint8_t dc_smem_raw[];
  const uint32_t base = dc_smem(dc_smem_raw);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) flag_timeout();
    return;
  }
  const DcBars bars = dc_bars_init(reinterpret_cast<uint64_t*>(dc_smem_raw + M::kBars));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, qd = lane & 3, strip = warp & 3;
  const int h = blockIdx.y, seq = long_sequence(a.seq, blockIdx.z), hk = h / a.G, m0 = blockIdx.x * kDwRows + 16 * strip;  // first value
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t state = ((int64_t)seq * a.Hv + h) * D * D;
  int chunks = (r.len + kDcTok - 1) / kDcTok;
  auto vec_at = [&](int c) {
    return reinterpret_cast<const float*>(__cvta_shared_to_generic(base + M::kVec + (c % 3) * M::kVecBytes));
  };
  auto hand_at = [&](int c) { return base + M::kHand + (c & 1) * X::kBytes + strip * X::kWarp; };

  if (warp >= 4) {
    // One thread starts all copies of a chunk.
    auto load = [&](int c) {
      const int n = r.len - c * kDcTok, row = r.first + c * kDcTok;
      uint64_t* bar = n < kDcTok ? bars.tail : bars.full + (c & 1);
      if (threadIdx.x == kDwThreads / 2) {
        const uint8_t* rec = records + (dc_slot(r, seq, c) * a.Hv + h) * (int64_t)DcRecord::kBytes;
        sm100::mbar_arrive_expect_tx(bar, (GRADS ? 1 : 2) * M::kRow + M::kVal + (GRADS ? 2 : 3) * kDcMat + M::kVecBytes);
        dc_tma_rows<D>(base + M::kK + (c & 1) * M::kRow, &tmK, 0, hk, row, bar);
        dc_bulk(base + M::kT + (c & 1) * 2 * kDcMat, rec + DcRecord::kThi, 2 * kDcMat, bar);
        dc_tma_rows<kDwRows>(base + M::kV + (c & 1) * M::kVal, &tmV, blockIdx.x * kDwRows, h, row, bar);
        dc_bulk(base + M::kVec + (c % 3) * M::kVecBytes, rec + DcRecord::kVec, M::kVecBytes, bar);
        if (!GRADS) {
          dc_tma_rows<D>(base + M::kQ + (c % 3) * M::kRow, &tmQ, 0, hk, row, bar);
          dc_bulk(base + M::kP + (c % 3) * kDcMat, rec + DcRecord::kPhi, kDcMat, bar);
        }
      }
    };
    // The first warp sees to the rows behind the sequence.
    auto finish_load = [&](int c) {
      const int n = r.len - c * kDcTok;
      if (n >= kDcTok || warp != 4) return;
      dc_wait(bars.tail, 0, epoch);
      dc_zero_rows<D>(base + M::kK + (c & 1) * M::kRow, n, lane);
      dc_zero_rows<kDwRows>(base + M::kV + (c & 1) * M::kVal, n, lane);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(bars.full + (c & 1));
    };
    if (chunks > 0) load(0);
    const bool found = chunks_found<kDcTok>(SlotRounds(a.seq, seq), a.seq, r);
    if (chunks > 0) finish_load(0);
    __syncthreads();
    if (!found) {  // the copies land before the CTA ends
      dc_wait(bars.full, 0, epoch);
      return;
    }
    for (int c = 0; c < chunks; ++c) {  // the walkers are at chunk c, this warp finishes chunk c - 1
      if (c + 1 < chunks) load(c + 1);
      dc_wait(bars.full + (c & 1), c >> 1, epoch);
      for (int d = c - 1; d <= (c + 1 < chunks ? c - 1 : c); ++d) {
        if (d == c) __syncthreads();    // behind the last chunk: finish that one too
        if (d < 0) continue;
        const uint32_t hand = hand_at(d);
        const int n = min(kDcTok, r.len - d * kDcTok);
        const int64_t row = r.first + (int64_t)d * kDcTok;
        float U[8][4];
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<float4*>(U[x]) =
              *reinterpret_cast<const float4*>(__cvta_shared_to_generic(hand + X::kU + x * 512 + lane * 16));
        if constexpr (GRADS) {
          dc_store_state<D>(hand, base + M::kOut + M::kVal + strip * 16 * RB, lane,
                            kept_S + ((dc_slot(r, seq, d) * a.Hv + h) * D + m0) * D);
          dc_store_tokens(U, base + M::kOut, strip, lane, n,
                          [&](int tok) { return kept_U + ((row + tok) * a.Hv + h) * D + m0; });
        } else {
          // O^T = scale e^G (S^T Q^T) + U^T P^T: S and P rounded to bf16, U in two parts.
          const uint32_t sq = base + M::kQ + (d % 3) * M::kRow, sp = base + M::kP + (d % 3) * kDcMat;
          const float* vec = vec_at(d);
          float O[8][4];
#pragma unroll
          for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) O[x][y] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint4 f = *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(hand + kk * 512 + lane * 16));
            const uint32_t hi[4] = {f.x, f.y, f.z, f.w};
            uint32_t b[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) ldsm(b[x], sq + right_at<RK>(16 * x, 2 * kk, lane));
#pragma unroll
            for (int x = 0; x < 8; ++x) mma16(O[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
          }
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float2 eg = *reinterpret_cast<const float2*>(vec + 8 * x + 2 * qd);
            O[x][0] *= a.scale * eg.x;
            O[x][1] *= a.scale * eg.y;
            O[x][2] *= a.scale * eg.x;
            O[x][3] *= a.scale * eg.y;
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            uint32_t hi[4], lo[4], b[4][4];
            as_left(U[2 * kk], U[2 * kk + 1], hi, lo);
#pragma unroll
            for (int x = kk; x < 4; ++x) ldsm(b[x], sp + right_at<128>(16 * x, 2 * kk, lane));
#pragma unroll
            for (int x = 2 * kk; x < 8; ++x) mma16(O[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
            for (int x = 2 * kk; x < 8; ++x) mma16(O[x], lo, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
          }
          dc_store_tokens(O, base + M::kOut, strip, lane, n, [&](int tok) { return a.out.at(row + tok, h) + m0; });
        }
      }
      if (c + 1 < chunks) {
        finish_load(c + 1);
        __syncthreads();
      }
    }
    return;
  }

  // Result-fragment layout: S[t] holds rows m0 + gr (+ 8), columns (d_k) 8 t +
  // 2 qd (+ 1).
  float S[NK][4];
#pragma unroll
  for (int t = 0; t < NK; ++t)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      S[t][y] = a.S_in ? a.S_in[state + (int64_t)(8 * t + 2 * qd + (y & 1)) * D + m0 + gr + 8 * (y >> 1)] : 0.f;
  if (!chunks_found<kDcTok>(SlotRounds(a.seq, seq), a.seq, r)) chunks = 0;
  for (int c = 0; c < chunks; ++c) {
    __syncthreads();
    dc_wait(bars.full + (c & 1), c >> 1, epoch);
    const uint32_t sk = base + M::kK + (c & 1) * M::kRow, sT = base + M::kT + (c & 1) * 2 * kDcMat,
                   sv = base + M::kV + (c & 1) * M::kVal, hand = hand_at(c);
    const float* vec = vec_at(c);
    // S^T K^T over d_k.
    float R[8][4];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) R[x][y] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t hi[4], lo[4], b[4][4];
      as_left(S[2 * kk], S[2 * kk + 1], hi, lo);
      dc_hand(hand + kk * 512 + lane * 16, hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
      for (int x = 0; x < 4; ++x) ldsm(b[x], sk + right_at<RK>(16 * x, 2 * kk, lane));
      mma_parts<8>(R, hi, lo, b);
    }
    // R^T = V^T - (.) e^G, times beta for the solve.
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      uint32_t v[4];
      ldsm_t(v, sv + right_at<128>(8 * x, 2 * strip, lane));
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int tok = 8 * (x + y) + 2 * qd;
        const float2 eg = *reinterpret_cast<const float2*>(vec + tok);
        const float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDcTok + tok);
        float(&f)[4] = R[x + y];
        f[0] = be.x * fmaf(-eg.x, f[0], low_f(v[2 * y]));
        f[1] = be.y * fmaf(-eg.y, f[1], high_f(v[2 * y]));
        f[2] = be.x * fmaf(-eg.x, f[2], low_f(v[2 * y + 1]));
        f[3] = be.y * fmaf(-eg.y, f[3], high_f(v[2 * y + 1]));
      }
    }
    // U^T = (beta R)^T T^T; T is lower triangular.
    float U[8][4];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) U[x][y] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4], b[4][4];
      as_left(R[2 * kk], R[2 * kk + 1], hi, lo);
#pragma unroll
      for (int x = kk; x < 4; ++x) ldsm(b[x], sT + right_at<128>(16 * x, 2 * kk, lane));
#pragma unroll
      for (int x = 2 * kk; x < 8; ++x) mma16(U[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
      for (int x = 2 * kk; x < 8; ++x) mma16(U[x], lo, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
      for (int x = kk; x < 4; ++x) ldsm(b[x], sT + kDcMat + right_at<128>(16 * x, 2 * kk, lane));
#pragma unroll
      for (int x = 2 * kk; x < 8; ++x) mma16(U[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
      dc_hand(hand + X::kU + x * 512 + lane * 16, __float_as_uint(U[x][0]), __float_as_uint(U[x][1]),
              __float_as_uint(U[x][2]), __float_as_uint(U[x][3]));
    // S^T = e^G_C S^T + (w U)^T K
    const float whole = vec[kDcTok - 1];
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y) S[t][y] *= whole;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float t0[4], t1[4];
      const float2 w0 = *reinterpret_cast<const float2*>(vec + kDcTok + 16 * kk + 2 * qd);
      const float2 w1 = *reinterpret_cast<const float2*>(vec + kDcTok + 16 * kk + 8 + 2 * qd);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        t0[y] = U[2 * kk][y] * (y & 1 ? w0.y : w0.x);
        t1[y] = U[2 * kk + 1][y] * (y & 1 ? w1.y : w1.x);
      }
      uint32_t hi[4], lo[4];
      as_left(t0, t1, hi, lo);
#pragma unroll
      for (int t = 0; t < NK; t += 8) {
        uint32_t b[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ldsm_t(b[x], sk + right_t_at<RK>(16 * kk, t + 2 * x, lane));
        mma_parts<8>(S + t, hi, lo, b);
      }
    }
  }
  __syncthreads();  // the partners finish the last chunk behind this
  dc_drain(bars, epoch);
  if (a.S_out) {
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y)
        a.S_out[state + (int64_t)(8 * t + 2 * qd + (y & 1)) * D + m0 + gr + 8 * (y >> 1)] = S[t][y];
  }
}

// ------------------------------------------------------------- reverse walk
// From the last chunk to the first, 16 rows of dS^T a warp:
//   dU = P^T dO + diag(w) K dS+,  Z = T^T dU,  dV = diag(beta) Z,
//   dS = e^G_C dS+ + scale Q^T diag(e^G) dO - K^T diag(e^G beta) Z
// Warps 4-7 load the next chunk and write what the last one left: Z (rows
// [T][Hv][D]), dV, and dS+ of each chunk (dS^T as bf16 [d_v][d_k]). Measured on 8
// sequences of 128-2048, 8 / 16 heads, d = 128: 114 us (the forward walk there: 94
// us, 83 us where it keeps S and U instead of writing the output).
template <int D>
struct DrSmem {
  static constexpr uint32_t kRow = kDcTok * D * 2, kVal = kDcTok * kDwRows * 2, kVecBytes = 3 * kDcTok * 4;
  static constexpr uint32_t kK = 0, kQ = kK + 2 * kRow, kT = kQ + 2 * kRow, kP = kT + 4 * kDcMat, kO = kP + 4 * kDcMat,
                            kVec = kO + 2 * kVal, kZ = kVec + 3 * kVecBytes, kS = kZ + 2 * 4 * 8 * 512,
                            kOut = kS + 2 * kDwRows * D * 2, kBars = kOut + kVal, kTotal = kBars + 64;
  static_assert(kTotal <= 232448, "reverse kernel shared memory");
};

template <int D>
__global__ void __launch_bounds__(kDwThreads, 1)
delta_reverse_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmO, const DeltaGradArgs<__nv_bfloat16> a,
                     const uint8_t* __restrict__ records, __nv_bfloat16* __restrict__ kept_dS,
                     __nv_bfloat16* __restrict__ kept_Z, uint32_t epoch) {
  using M = DrSmem<D>;
  constexpr int RB = D * 2, NK = D / 8, RK = kDcBlocks;
  extern __shared__ __align__(1024) uint8_t dc_smem_raw[];
  const uint32_t base = dc_smem(dc_smem_raw);
  if ((base & 1023u) != 0) {
    if (threadIdx.x == 0) flag_timeout();
    return;
  }
  const DcBars bars = dc_bars_init(reinterpret_cast<uint64_t*>(dc_smem_raw + M::kBars));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, qd = lane & 3, strip = warp & 3;
  const int h = blockIdx.y, seq = long_sequence(a.seq, blockIdx.z), hk = h / a.G, m0 = blockIdx.x * kDwRows + 16 * strip;
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t state = ((int64_t)seq * a.Hv + h) * D * D;
  int chunks = (r.len + kDcTok - 1) / kDcTok;  // step i takes chunk chunks - 1 - i
  auto vec_at = [&](int i) {
    return reinterpret_cast<const float*>(__cvta_shared_to_generic(base + M::kVec + (i % 3) * M::kVecBytes));
  };
  auto z_at = [&](int i) { return base + M::kZ + ((i & 1) * 4 + strip) * 8 * 512; };
  auto state_at = [&](int i) { return base + M::kS + ((i & 1) * 4 + strip) * 16 * RB; };

  if (warp >= 4) {
    auto load = [&](int i) {
      const int c = chunks - 1 - i, n = r.len - c * kDcTok, row = r.first + c * kDcTok;
      uint64_t* bar = n < kDcTok ? bars.tail : bars.full + (i & 1);
      if (threadIdx.x == kDwThreads / 2) {
        const uint8_t* rec = records + (dc_slot(r, seq, c) * a.Hv + h) * (int64_t)DcRecord::kBytes;
        sm100::mbar_arrive_expect_tx(bar, 2 * M::kRow + M::kVal + 4 * kDcMat + M::kVecBytes);
        dc_tma_rows<D>(base + M::kK + (i & 1) * M::kRow, &tmK, 0, hk, row, bar);
        dc_bulk(base + M::kP + (i & 1) * 2 * kDcMat, rec + DcRecord::kPhi, 2 * kDcMat, bar);
        dc_tma_rows<kDwRows>(base + M::kO + (i & 1) * M::kVal, &tmO, blockIdx.x * kDwRows, h, row, bar);
        dc_tma_rows<D>(base + M::kQ + (i & 1) * M::kRow, &tmQ, 0, hk, row, bar);
        dc_bulk(base + M::kT + (i & 1) * 2 * kDcMat, rec + DcRecord::kThi, 2 * kDcMat, bar);
        dc_bulk(base + M::kVec + (i % 3) * M::kVecBytes, rec + DcRecord::kVec, M::kVecBytes, bar);
      }
    };
    auto finish_load = [&](int i) {  // step 0 has the chunk that may end behind the sequence
      const int n = r.len - (chunks - 1 - i) * kDcTok;
      if (n >= kDcTok || warp != 4) return;
      dc_wait(bars.tail, 0, epoch);
      dc_zero_rows<D>(base + M::kK + (i & 1) * M::kRow, n, lane);
      dc_zero_rows<D>(base + M::kQ + (i & 1) * M::kRow, n, lane);
      dc_zero_rows<kDwRows>(base + M::kO + (i & 1) * M::kVal, n, lane);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(bars.full + (i & 1));
    };
    auto finish = [&](int i) {
      const int c = chunks - 1 - i, n = min(kDcTok, r.len - c * kDcTok);
      const int64_t row = r.first + (int64_t)c * kDcTok;
      __nv_bfloat16* dst = kept_dS + ((dc_slot(r, seq, c) * a.Hv + h) * D + m0) * D;
#pragma unroll
      for (int x = lane; x < 16 * NK; x += 32) {
        const int rr = x / NK, pc = x % NK;
        *reinterpret_cast<uint4*>(dst + rr * D + pc * 8) =
            *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(state_at(i) + dc_at<RB>(rr, pc)));
      }
      float Z[8][4];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        *reinterpret_cast<float4*>(Z[x]) =
            *reinterpret_cast<const float4*>(__cvta_shared_to_generic(z_at(i) + x * 512 + lane * 16));
      dc_store_tokens(Z, base + M::kOut, strip, lane, n, [&](int tok) { return kept_Z + ((row + tok) * a.Hv + h) * D + m0; });
      const float* vec = vec_at(i);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDcTok + 8 * x + 2 * qd);
        if (fabsf(be.x) <= kDpTiny) be.x = 0.f;
        if (fabsf(be.y) <= kDpTiny) be.y = 0.f;
        Z[x][0] *= be.x;
        Z[x][1] *= be.y;
        Z[x][2] *= be.x;
        Z[x][3] *= be.y;
      }
      dc_store_tokens(Z, base + M::kOut, strip, lane, n, [&](int tok) { return a.dv.at(row + tok, h) + m0; });
    };
    if (chunks > 0) load(0);
    const bool found = chunks_found<kDcTok>(SlotRounds(a.seq, seq), a.seq, r);
    if (chunks > 0) finish_load(0);
    __syncthreads();
    if (!found) {  // the copies land before the CTA ends
      dc_wait(bars.full, 0, epoch);
      return;
    }
    for (int i = 0; i < chunks; ++i) {  // the walkers are at step i, this warp finishes step i - 1
      if (i + 1 < chunks) load(i + 1);
      dc_wait(bars.full + (i & 1), i >> 1, epoch);
      if (i > 0) finish(i - 1);
      __syncthreads();
    }
    if (chunks > 0) finish(chunks - 1);
    return;
  }

  float S[NK][4];  // dS^T
#pragma unroll
  for (int t = 0; t < NK; ++t)
#pragma unroll
    for (int y = 0; y < 4; ++y)
      S[t][y] = a.dS_out ? a.dS_out[state + (int64_t)(8 * t + 2 * qd + (y & 1)) * D + m0 + gr + 8 * (y >> 1)] : 0.f;
  if (!chunks_found<kDcTok>(SlotRounds(a.seq, seq), a.seq, r)) chunks = 0;
  for (int i = 0; i < chunks; ++i) {
    __syncthreads();
    dc_wait(bars.full + (i & 1), i >> 1, epoch);
    const uint32_t sk = base + M::kK + (i & 1) * M::kRow, sq = base + M::kQ + (i & 1) * M::kRow,
                   sT = base + M::kT + (i & 1) * 2 * kDcMat, sp = base + M::kP + (i & 1) * 2 * kDcMat,
                   so = base + M::kO + (i & 1) * M::kVal;
    const float* vec = vec_at(i);
    // dU^T = (dS+^T K^T) w + dO^T P
    float U[8][4];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) U[x][y] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t hi[4], lo[4], b[4][4];
      as_left(S[2 * kk], S[2 * kk + 1], hi, lo);
      stsm(state_at(i) + dc_at<RB>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)), hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
      for (int x = 0; x < 4; ++x) ldsm(b[x], sk + right_at<RK>(16 * x, 2 * kk, lane));
      mma_parts<8>(U, hi, lo, b);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float2 w = *reinterpret_cast<const float2*>(vec + kDcTok + 8 * x + 2 * qd);
      U[x][0] *= w.x;
      U[x][1] *= w.y;
      U[x][2] *= w.x;
      U[x][3] *= w.y;
    }
    const float whole = vec[kDcTok - 1];
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y) S[t][y] *= whole;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {  // tokens i = 16 kk ..: into dU (j <= i) and, times scale e^G, into dS
      uint32_t o[4];
      ldsm_t(o, so + left_t_at<128>(16 * kk, 2 * strip, lane));
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        uint32_t b[4][4];
#pragma unroll
        for (int x = 0; x <= kk; ++x) ldsm_t(b[x], sp + part * kDcMat + right_t_at<128>(16 * kk, 2 * x, lane));
#pragma unroll
        for (int x = 0; x < 2 * kk + 2; ++x) mma16(U[x], o, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
      }
      const float2 e0 = *reinterpret_cast<const float2*>(vec + 16 * kk + 2 * qd);
      const float2 e1 = *reinterpret_cast<const float2*>(vec + 16 * kk + 8 + 2 * qd);
      uint32_t hi[4], lo[4];
      split2(low_f(o[0]) * (a.scale * e0.x), high_f(o[0]) * (a.scale * e0.y), hi[0], lo[0]);
      split2(low_f(o[1]) * (a.scale * e0.x), high_f(o[1]) * (a.scale * e0.y), hi[1], lo[1]);
      split2(low_f(o[2]) * (a.scale * e1.x), high_f(o[2]) * (a.scale * e1.y), hi[2], lo[2]);
      split2(low_f(o[3]) * (a.scale * e1.x), high_f(o[3]) * (a.scale * e1.y), hi[3], lo[3]);
#pragma unroll
      for (int t = 0; t < NK; t += 8) {
        uint32_t b[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ldsm_t(b[x], sq + right_t_at<RK>(16 * kk, t + 2 * x, lane));
        mma_parts<8>(S + t, hi, lo, b);
      }
    }
    // Z^T = dU^T T
    float Z[8][4];
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) Z[x][y] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      as_left(U[2 * kk], U[2 * kk + 1], hi, lo);
      uint32_t b[4][4];
#pragma unroll
      for (int x = 0; x <= kk; ++x) ldsm_t(b[x], sT + right_t_at<128>(16 * kk, 2 * x, lane));
#pragma unroll
      for (int x = 0; x < 2 * kk + 2; ++x) mma16(Z[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
      for (int x = 0; x < 2 * kk + 2; ++x) mma16(Z[x], lo, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
#pragma unroll
      for (int x = 0; x <= kk; ++x) ldsm_t(b[x], sT + kDcMat + right_t_at<128>(16 * kk, 2 * x, lane));
#pragma unroll
      for (int x = 0; x < 2 * kk + 2; ++x) mma16(Z[x], hi, b[x / 2][2 * (x & 1)], b[x / 2][2 * (x & 1) + 1]);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      dc_hand(z_at(i) + x * 512 + lane * 16, __float_as_uint(Z[x][0]), __float_as_uint(Z[x][1]), __float_as_uint(Z[x][2]),
              __float_as_uint(Z[x][3]));
      const float2 be = *reinterpret_cast<const float2*>(vec + 2 * kDcTok + 8 * x + 2 * qd);
      U[x][0] = Z[x][0] * be.x;
      U[x][1] = Z[x][1] * be.y;
      U[x][2] = Z[x][2] * be.x;
      U[x][3] = Z[x][3] * be.y;
    }
    // dS^T -= (e^G beta Z)^T K
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const float2 e0 = *reinterpret_cast<const float2*>(vec + 16 * kk + 2 * qd);
      const float2 e1 = *reinterpret_cast<const float2*>(vec + 16 * kk + 8 + 2 * qd);
      float t0[4], t1[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        t0[y] = -U[2 * kk][y] * (y & 1 ? e0.y : e0.x);
        t1[y] = -U[2 * kk + 1][y] * (y & 1 ? e1.y : e1.x);
      }
      uint32_t hi[4], lo[4];
      as_left(t0, t1, hi, lo);
#pragma unroll
      for (int t = 0; t < NK; t += 8) {
        uint32_t b[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) ldsm_t(b[x], sk + right_t_at<RK>(16 * kk, t + 2 * x, lane));
        mma_parts<8>(S + t, hi, lo, b);
      }
    }
  }
  __syncthreads();  // the partners finish the last step behind this
  dc_drain(bars, epoch);
  if (a.dS_in) {
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
      for (int y = 0; y < 4; ++y)
        a.dS_in[state + (int64_t)(8 * t + 2 * qd + (y & 1)) * D + m0 + gr + 8 * (y >> 1)] = S[t][y];
  }
}

// ---------------------------------------------------------------- gradients
// All chunks at once, CTA = (chunk, key head), value head after value head of
// the group (dq and dk stay in registers, warp w has tokens 16 w ..):
//   M = dO U^T (j <= i), H = Z U^T, F_ij = beta_i e_ij H_ij (j < i), X_ij = scale e_ij M_ij
//   dq_i += scale e^G_i S dO_i + sum_j X_ij k_j
//   dk_i += sum_j X_ji q_j - e^G_i beta_i S Z_i + w_i dS+ u_i - sum_j (F_ij + F_ji) k_j
//   dbeta_i = H_ii / beta_i  (U = beta times what beta scales)
//   dg_t = sum_{i >= t} s_i + sum_{i >= t > j} N_ij + sum_{j < t} x_j + e^G_C <dS+, S>,
//   N_ij = X_ij q_i.k_j - F_ij k_i.k_j, s_i = q_i.(scale e^G_i S dO_i) - k_i.(e^G_i beta_i S Z_i),
//   x_j = k_j.(w_j dS+ u_j)
// Z, U, S and dS+ enter rounded to bf16, X and F too: all results are bf16.
// Measured on 8 sequences of 128-2048, 8 / 16 heads, d = 128 (2200 chunks and value
// heads): 165 us; a head's 112 KB of operands are loaded before its products start.
constexpr int kDgThreads = 512;
template <int D>
struct DgSmem {
  static constexpr uint32_t kRow = kDcTok * D * 2;
  static constexpr uint32_t kK = 0, kQ = kRow, kU = 2 * kRow, kZ = 3 * kRow, kO = 4 * kRow, kS = 5 * kRow,
                            kdS = kS + D * D * 2, kX = kdS + D * D * 2, kF = kX + kDcMat, kVec = kF + kDcMat,
                            kMore = kVec + DcRecord::kVecBytes, kTotal = kMore + (29 * kDcTok + 16) * 4 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kDgThreads, 1)
delta_grad_kernel(const DeltaGradArgs<__nv_bfloat16> a, const uint8_t* __restrict__ records,
                  const __nv_bfloat16* __restrict__ kept_S, const __nv_bfloat16* __restrict__ kept_dS,
                  const __nv_bfloat16* __restrict__ kept_U, const __nv_bfloat16* __restrict__ kept_Z) {
  using M = DgSmem<D>;
  constexpr int RB = D * 2, NK = D / 8;
  extern __shared__ __align__(1024) uint8_t dc_smem_raw[];
  const uint32_t s = (dc_smem(dc_smem_raw) + 1023u) & ~1023u;
  auto ptr = [&](uint32_t at) { return reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(s + at)); };
  const float* vec = reinterpret_cast<const float*>(ptr(M::kVec));
  const double* Gd = reinterpret_cast<const double*>(vec + 3 * kDcTok);
  float* cols = reinterpret_cast<float*>(ptr(M::kMore));  // [16][64] a warp's share of the sums over N
  float* si = cols + 16 * kDcTok;                         // [4][64], one for each quarter of d_k
  float* xi = si + 4 * kDcTok;
  float* in = xi + 4 * kDcTok;   // exp(G_i - G_b), b the start of i's block of 16
  float* out = in + kDcTok;      // [4][64]: exp(G_b - G_j), j < 16 b
  float* red = out + 4 * kDcTok;  // [16]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, qd = lane & 3, hk = blockIdx.y;
  const int block = warp & 3, part = warp >> 2, m0 = 16 * block;
  SlotTile t;
  if (!chunk_tile<kDcTok>(a.seq, blockIdx.x, &t)) return;
  const int n = min(kDcTok, t.r.len - t.tile * kDcTok);
  const int64_t row0 = t.r.first + t.tile * kDcTok, slot = dc_slot(t.r, t.seq, t.tile);
  const RowsOf<const __nv_bfloat16> ru{kept_U, (int64_t)a.Hv * D, D}, rz{kept_Z, (int64_t)a.Hv * D, D};

  constexpr int NC = NK / 4;  // tiles of 8 columns (d_k) of a warp
  float dq[NC][4], dk[NC][4];
#pragma unroll
  for (int x = 0; x < NC; ++x)
#pragma unroll
    for (int y = 0; y < 4; ++y) dq[x][y] = dk[x][y] = 0.f;
  dc_load_rows<D, kDgThreads>(s + M::kK, a.k, row0, hk, 0, n, tid);
  dc_load_rows<D, kDgThreads>(s + M::kQ, a.q, row0, hk, 0, n, tid);
  cp_commit();
  if (!tile_found<kDcTok>(a.seq, t)) {
    cp_wait();
    return;
  }
  for (int u = 0; u < a.G; ++u) {
    const int h = hk * a.G + u;
    const uint8_t* rec = records + (slot * a.Hv + h) * (int64_t)DcRecord::kBytes;
    if (u) __syncthreads();
    dc_load_rows<D, kDgThreads>(s + M::kU, ru, row0, h, 0, n, tid);
    dc_load_rows<D, kDgThreads>(s + M::kZ, rz, row0, h, 0, n, tid);
    dc_load_rows<D, kDgThreads>(s + M::kO, a.dout, row0, h, 0, n, tid);
    for (int i = tid; i < D * NK; i += kDgThreads) {
      const int64_t at = (slot * a.Hv + h) * D * D + i * 8;
      cp16(s + M::kS + dc_at<RB>(i / NK, i % NK), kept_S + at, true);
      cp16(s + M::kdS + dc_at<RB>(i / NK, i % NK), kept_dS + at, true);
    }
    dc_load_flat<kDgThreads>(s + M::kVec, rec + DcRecord::kVec, DcRecord::kVecBytes, tid);
    cp_commit();
    cp_wait();
    __syncthreads();
    // Decays between tokens as in the prep kernel.
    if (tid < 5 * kDcTok) {
      const int b = tid >> 6, i = tid & 63;
      if (b == 0)
        in[i] = expf((float)(Gd[i] - Gd[i & 48]));
      else if (b < 4)
        out[b * kDcTok + i] = i < 16 * b ? expf((float)(Gd[16 * b] - Gd[i])) : 0.f;
    }
    // <dS+, S> over the whole state (the same places of two tiles).
    float dot = 0.f;
    for (int i = tid; i < D * NK; i += kDgThreads) {
      const uint4 x = *reinterpret_cast<const uint4*>(ptr(M::kS + i * 16));
      const uint4 y = *reinterpret_cast<const uint4*>(ptr(M::kdS + i * 16));
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int z = 0; z < 4; ++z)
        dot = fmaf(low_f(xs[z]), low_f(ys[z]), fmaf(high_f(xs[z]), high_f(ys[z]), dot));
    }
    dot = warp_sum(dot);
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    const float eg0 = vec[m0 + gr], eg1 = vec[m0 + gr + 8];
    const float w0 = vec[kDcTok + m0 + gr], w1 = vec[kDcTok + m0 + gr + 8];
    const float be0 = vec[2 * kDcTok + m0 + gr], be1 = vec[2 * kDcTok + m0 + gr + 8];
    const float whole = vec[kDcTok - 1];
    {
      // Rows 16 b .. of M and q.k (parts 0, 2) or of H and k.k (parts 1, 3),
      // columns 0 - 31 (parts 0, 1) or 32 - 63, up to the block's last row: N =
      // X q.k - F k.k comes in four shares.
      const bool second = part & 1;
      const int j0 = 4 * (part >> 1);  // first tile of 8 columns
      float mm[4][4], kk[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) mm[x][y] = kk[x][y] = 0.f;
      const uint32_t left = s + (second ? M::kZ : M::kO), left2 = s + (second ? M::kK : M::kQ);
      if (j0 <= 2 * block) {
#pragma unroll
        for (int z = 0; z < D / 16; ++z) {
          uint32_t l[4], l2[4];
          ldsm(l, left + left_at<RB>(m0, 2 * z, lane));
          ldsm(l2, left2 + left_at<RB>(m0, 2 * z, lane));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (j0 + 2 * x > 2 * block) continue;
            uint32_t b[4];
            ldsm(b, s + M::kU + right_at<RB>(8 * j0 + 16 * x, 2 * z, lane));
            mma16(mm[2 * x], l, b[0], b[1]);
            mma16(mm[2 * x + 1], l, b[2], b[3]);
            ldsm(b, s + M::kK + right_at<RB>(8 * j0 + 16 * x, 2 * z, lane));
            mma16(kk[2 * x], l2, b[0], b[1]);
            mma16(kk[2 * x + 1], l2, b[2], b[3]);
          }
        }
      }
      // X or F as bf16 into shared memory, and this share of sum_{i >= t > j}
      // N_ij over the warp's rows for every t: prefix sums over a row's columns
      // (4 lanes have 2 of every 8 each), then sums over rows.
      const float in0 = in[m0 + gr], in1 = in[m0 + gr + 8];
      float pre[2] = {0.f, 0.f};  // over columns before the tile, rows gr and gr + 8
      float sum[16];              // t = 8 x + 2 qd (+ 1), over this thread's two rows
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int xl = x & 3;
        sum[2 * x] = sum[2 * x + 1] = 0.f;
        if ((x >> 2) == (part >> 1)) {
          if ((x >> 1) > block) continue;  // above the diagonal: nothing is read there either
          float nn[4], xx[4];
          if ((x >> 1) < block) {  // every column before every row
            const float2 o = *reinterpret_cast<const float2*>(out + block * kDcTok + 8 * x + 2 * qd);
            const float f0 = in0 * (second ? be0 : a.scale), f1 = in1 * (second ? be1 : a.scale);
            xx[0] = f0 * o.x * mm[xl][0];
            xx[1] = f0 * o.y * mm[xl][1];
            xx[2] = f1 * o.x * mm[xl][2];
            xx[3] = f1 * o.y * mm[xl][3];
#pragma unroll
            for (int y = 0; y < 4; ++y) nn[y] = (second ? -xx[y] : xx[y]) * kk[xl][y];
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int i = m0 + gr + 8 * (y >> 1), j = 8 * x + 2 * qd + (y & 1);
              const float e = j <= i ? __expf((float)(Gd[i] - Gd[j])) : 0.f, be = y >> 1 ? be1 : be0;
              xx[y] = second ? (j < i ? be * e * mm[xl][y] : 0.f) : j <= i ? a.scale * e * mm[xl][y] : 0.f;
              nn[y] = j < i ? (second ? -xx[y] : xx[y]) * kk[xl][y] : 0.f;
              if (second && j == i && i < n) *a.dbeta.at(row0 + i, h) = __float2bfloat16_rn(mm[xl][y] / be);
            }
          }
          const uint32_t to = second ? M::kF : M::kX;
          *reinterpret_cast<uint32_t*>(ptr(to + dc_at<128>(m0 + gr, x) + qd * 4)) = pack2(xx[0], xx[1]);
          *reinterpret_cast<uint32_t*>(ptr(to + dc_at<128>(m0 + gr + 8, x) + qd * 4)) = pack2(xx[2], xx[3]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // rows gr, gr + 8
            float inc = nn[2 * y] + nn[2 * y + 1];  // over the 4 lanes of the row
            float up = __shfl_up_sync(0xffffffffu, inc, 1, 4);
            if (qd >= 1) inc += up;
            up = __shfl_up_sync(0xffffffffu, inc, 2, 4);
            if (qd >= 2) inc += up;
            // Not as a difference: behind a strong decay what is in front of it is
            // far smaller than the column itself.
            up = __shfl_up_sync(0xffffffffu, inc, 1, 4);
            const float before = pre[y] + (qd ? up : 0.f);
            const int i = m0 + gr + 8 * y, tt = 8 * x + 2 * qd;
            if (i >= tt) sum[2 * x] += before;
            if (i >= tt + 1) sum[2 * x + 1] += before + nn[2 * y];
            pre[y] += __shfl_sync(0xffffffffu, inc, 3, 4);
          }
        } else if ((x >> 2) > (part >> 1) && (x >> 1) <= block) {  // behind this share's columns: all of them count
          const int i = m0 + gr, tt = 8 * x + 2 * qd;
          sum[2 * x] = (i >= tt ? pre[0] : 0.f) + (i + 8 >= tt ? pre[1] : 0.f);
          sum[2 * x + 1] = (i >= tt + 1 ? pre[0] : 0.f) + (i + 8 >= tt + 1 ? pre[1] : 0.f);
        }
      }
      // Sums over the 8 lanes with the same qd: halve the values kept at each step.
#pragma unroll
      for (int st = 0; st < 3; ++st) {
        const int keep = 8 >> st;
        const bool upper = lane & (16 >> st);
#pragma unroll
        for (int x = 0; x < keep; ++x) {
          const float give = upper ? sum[x] : sum[x + keep], mine = upper ? sum[x + keep] : sum[x];
          sum[x] = mine + __shfl_xor_sync(0xffffffffu, give, 16 >> st);
        }
      }
      // Lane bits 4, 3, 2 chose value 8 b4 + 4 b3 + 2 b2 (+ 1): tile of value / 2.
      const int x = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
      cols[warp * kDcTok + 8 * x + 2 * qd] = sum[0];
      cols[warp * kDcTok + 8 * x + 2 * qd + 1] = sum[1];
    }
    __syncthreads();
    // The state's terms: rows of dO, Z and U times S and dS+, one after the
    // other, each dotted with its own row of q or k on the way.
    float sdot[2] = {0.f, 0.f}, xdot[2] = {0.f, 0.f};
    const int c0 = part * NC;  // this warp's columns (d_k), in tiles of 8
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      const uint32_t from = which == 0 ? M::kO : which == 1 ? M::kZ : M::kU;
      const uint32_t st = which == 2 ? M::kdS : M::kS;
      const uint32_t own = which == 0 ? M::kQ : M::kK;
      const float f0 = which == 0 ? a.scale * eg0 : which == 1 ? -eg0 * be0 : w0;
      const float f1 = which == 0 ? a.scale * eg1 : which == 1 ? -eg1 * be1 : w1;
      float dots[2] = {0.f, 0.f};
      float c[NC][4];
#pragma unroll
      for (int x = 0; x < NC; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) c[x][y] = 0.f;
#pragma unroll
      for (int z = 0; z < D / 16; ++z) {
        uint32_t l[4];
        ldsm(l, s + from + left_at<RB>(m0, 2 * z, lane));
#pragma unroll
        for (int x = 0; x < NC; x += 2) {
          uint32_t b[4];
          ldsm_t(b, s + st + right_t_at<RB>(16 * z, c0 + x, lane));
          mma16(c[x], l, b[0], b[1]);
          mma16(c[x + 1], l, b[2], b[3]);
        }
      }
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        const uint32_t o0 = *reinterpret_cast<const uint32_t*>(ptr(own + dc_at<RB>(m0 + gr, c0 + x) + qd * 4));
        const uint32_t o1 = *reinterpret_cast<const uint32_t*>(ptr(own + dc_at<RB>(m0 + gr + 8, c0 + x) + qd * 4));
        c[x][0] *= f0;
        c[x][1] *= f0;
        c[x][2] *= f1;
        c[x][3] *= f1;
        dots[0] = fmaf(c[x][0], low_f(o0), fmaf(c[x][1], high_f(o0), dots[0]));
        dots[1] = fmaf(c[x][2], low_f(o1), fmaf(c[x][3], high_f(o1), dots[1]));
        float(&to)[4] = which == 0 ? dq[x] : dk[x];
#pragma unroll
        for (int y = 0; y < 4; ++y) to[y] += c[x][y];
      }
      float(&acc)[2] = which == 2 ? xdot : sdot;
      acc[0] += dots[0];
      acc[1] += dots[1];
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      sdot[y] += __shfl_xor_sync(0xffffffffu, sdot[y], 1);
      sdot[y] += __shfl_xor_sync(0xffffffffu, sdot[y], 2);
      xdot[y] += __shfl_xor_sync(0xffffffffu, xdot[y], 1);
      xdot[y] += __shfl_xor_sync(0xffffffffu, xdot[y], 2);
      if (qd == 0) {
        si[part * kDcTok + m0 + gr + 8 * y] = sdot[y];
        xi[part * kDcTok + m0 + gr + 8 * y] = xdot[y];
      }
    }
    // dq += X K (j <= i);  dk += X^T Q (i >= j) - F K - F^T K
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      uint32_t l[4];
      if (z <= block) {
        ldsm(l, s + M::kX + left_at<128>(m0, 2 * z, lane));
#pragma unroll
        for (int x = 0; x < NC; x += 2) {
          uint32_t b[4];
          ldsm_t(b, s + M::kK + right_t_at<RB>(16 * z, c0 + x, lane));
          mma16(dq[x], l, b[0], b[1]);
          mma16(dq[x + 1], l, b[2], b[3]);
        }
      }
      if (z >= block) {
        ldsm_t(l, s + M::kX + left_t_at<128>(16 * z, 2 * block, lane));
#pragma unroll
        for (int x = 0; x < NC; x += 2) {
          uint32_t b[4];
          ldsm_t(b, s + M::kQ + right_t_at<RB>(16 * z, c0 + x, lane));
          mma16(dk[x], l, b[0], b[1]);
          mma16(dk[x + 1], l, b[2], b[3]);
        }
      }
      // F and F^T meet only in the diagonal block, where one is +0 wherever the
      // other is not: their sum is the bitwise or.
      uint32_t f[4] = {0u, 0u, 0u, 0u};
      if (z <= block) ldsm(f, s + M::kF + left_at<128>(m0, 2 * z, lane));
      if (z >= block) {
        uint32_t ft[4];
        ldsm_t(ft, s + M::kF + left_t_at<128>(16 * z, 2 * block, lane));
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] |= ft[y];
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) f[y] ^= 0x80008000u;
#pragma unroll
      for (int x = 0; x < NC; x += 2) {
        uint32_t b[4];
        ldsm_t(b, s + M::kK + right_t_at<RB>(16 * z, c0 + x, lane));
        mma16(dk[x], f, b[0], b[1]);
        mma16(dk[x + 1], f, b[2], b[3]);
      }
    }
    __syncthreads();
    if (warp == 0) {  // dg; lane has tokens 2 lane, 2 lane + 1
      float all = warp_sum(lane < kDgThreads / 32 ? red[lane] : 0.f) * whole;
      float sv[2], xv[2], cv[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 2 * lane + y;
        sv[y] = xv[y] = cv[y] = 0.f;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          sv[y] += si[z * kDcTok + i];
          xv[y] += xi[z * kDcTok + i];
        }
#pragma unroll
        for (int z = 0; z < kDgThreads / 32; ++z) cv[y] += cols[z * kDcTok + i];
      }
      float down = sv[0] + sv[1], up = xv[0] + xv[1];  // from the end, from the start
#pragma unroll
      for (int st = 1; st < 32; st <<= 1) {
        const float d2 = __shfl_down_sync(0xffffffffu, down, st), u2 = __shfl_up_sync(0xffffffffu, up, st);
        if (lane + st < 32) down += d2;
        if (lane >= st) up += u2;
      }
      up = __shfl_up_sync(0xffffffffu, up, 1);
      if (lane == 0) up = 0.f;
      float rest = __shfl_down_sync(0xffffffffu, down, 1);
      if (lane == 31) rest = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = 2 * lane + y;
        const float v = all + cv[y] + (y ? sv[1] : sv[0] + sv[1]) + rest + up + (y ? xv[0] : 0.f);
        if (i < n) *a.dg.at(row0 + i, h) = __float2bfloat16_rn(v);
      }
    }
  }
  __syncthreads();
  // dq and dk as whole rows through the U and Z tiles.
#pragma unroll
  for (int x = 0; x < NC; x += 2) {
    const uint32_t at = dc_at<RB>(m0 + (lane & 7) + ((lane >> 3) & 1) * 8, part * NC + x + (lane >> 4));
    stsm(s + M::kU + at, pack2(dq[x][0], dq[x][1]), pack2(dq[x][2], dq[x][3]), pack2(dq[x + 1][0], dq[x + 1][1]),
         pack2(dq[x + 1][2], dq[x + 1][3]));
    stsm(s + M::kZ + at, pack2(dk[x][0], dk[x][1]), pack2(dk[x][2], dk[x][3]), pack2(dk[x + 1][0], dk[x + 1][1]),
         pack2(dk[x + 1][2], dk[x + 1][3]));
  }
  __syncthreads();
  for (int i = tid; i < n * NK; i += kDgThreads) {
    const int rr = i / NK, pc = i % NK;
    *reinterpret_cast<uint4*>(a.dq.at(row0 + rr, hk) + pc * 8) =
        *reinterpret_cast<const uint4*>(ptr(M::kU + dc_at<RB>(rr, pc)));
    *reinterpret_cast<uint4*>(a.dk.at(row0 + rr, hk) + pc * 8) =
        *reinterpret_cast<const uint4*>(ptr(M::kZ + dc_at<RB>(rr, pc)));
  }
}

}  // namespace infini

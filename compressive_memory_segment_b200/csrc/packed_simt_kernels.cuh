// Causal softmax attention over packed sequences with grouped heads on the CUDA
// cores: any type, any lengths. fp32 inputs run here.
//
//   x_ij = scale q_i . k_j for j <= i + nk - nq,  lse_i = log sum_j exp x_ij,
//   o_i = sum_j exp(x_ij - lse_i) v_j;  a row that sees no key has o = 0 and
//   lse = -inf, and no gradient.
//
// fp32 products on the CUDA cores bound these kernels (a 32 x 32 block of
// scores costs 32 x 32 x D multiply-adds against 3 x 32 x D elements
// read from L2), so both operands are held in shared memory as fp32 and each
// of the 128 threads forms 4 x 2 (forward, d = 64: 4 x 4) scores and 4 x D / 16 outputs
// from registers.
// Measured: 4 sequences of 100-700, 8 / 4 heads, d = 64, fp32: 57 us, 14 TFLOP/s;
// loads from shared memory (8 of 16 bytes for 64 multiply-adds of the scores) are
// what the busy SMs wait for. Gradients of 4 sequences of 205-700 (the forward 66 us
// in a graph, L2 flushed): 437 us, d = 128 508 us: 4 x 2 scores a thread, and a tile's
// loads with nothing else in flight.
#pragma once

#include <type_traits>

#include "packed_common.cuh"

namespace infini {

constexpr int kPsRows = 32;     // rows a CTA owns (64 and twice the threads: 116 us where 32 took 84)
constexpr int kPsCols = 32;     // streamed rows of the other side
constexpr int kPsThreads = 128;
constexpr int kPsPst = kPsCols + 4;

// c[4][N] = the 4 x N block of A B^T at rows 4 ty, columns tx, tx + 16, ..
template <int D, int ST, int N>
__device__ __forceinline__ void ps_scores(const float* __restrict__ A, const float* __restrict__ B, int ty, int tx,
                                          float (&c)[4][N]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int y = 0; y < N; ++y) c[i][y] = 0.f;
#pragma unroll 4
  for (int x = 0; x < D; x += 4) {
    float4 b[N];
#pragma unroll
    for (int y = 0; y < N; ++y) b[y] = *reinterpret_cast<const float4*>(B + (tx + 16 * y) * ST + x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = *reinterpret_cast<const float4*>(A + (4 * ty + i) * ST + x);
#pragma unroll
      for (int y = 0; y < N; ++y)
        c[i][y] = fmaf(a.x, b[y].x, fmaf(a.y, b[y].y, fmaf(a.z, b[y].z, fmaf(a.w, b[y].w, c[i][y]))));
    }
  }
}

// acc[4][D / 16] += P[rows 4 ty ..][COLS] B[COLS][D], columns 4 tx + 64 u.
template <int D, int ST, int COLS, int PST = COLS + 4>
__device__ __forceinline__ void ps_accumulate(const float* __restrict__ P, const float* __restrict__ B, int ty, int tx,
                                              float (&acc)[4][D / 16]) {
#pragma unroll 2
  for (int j = 0; j < COLS; j += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(P + (4 * ty + i) * PST + j);
#pragma unroll
    for (int z = 0; z < 4; ++z)
#pragma unroll
      for (int u = 0; u < D / 64; ++u) {
        const float4 b = *reinterpret_cast<const float4*>(B + (j + z) * ST + 4 * tx + 64 * u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][4 * u] = fmaf(p[i][z], b.x, acc[i][4 * u]);
          acc[i][4 * u + 1] = fmaf(p[i][z], b.y, acc[i][4 * u + 1]);
          acc[i][4 * u + 2] = fmaf(p[i][z], b.z, acc[i][4 * u + 2]);
          acc[i][4 * u + 3] = fmaf(p[i][z], b.w, acc[i][4 * u + 3]);
        }
      }
  }
}

// The streamed rows of the next tile, on their way through registers while the
// present tile is worked on (rows behind the sequence as zeros).
template <typename T, int D, int COLS>
struct PsAhead {
  static constexpr int VE = 16 / (int)sizeof(T), VPR = D / VE, PER = COLS * VPR / kPsThreads;
  static_assert(COLS * VPR % kPsThreads == 0, "vectors per thread");
  uint4 r[PER];
  __device__ __forceinline__ void issue(const RowsOf<const T>& x, int64_t t0, int h, int valid, int tid) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = tid + u * kPsThreads, row = i / VPR, c = i % VPR;
      r[u] = row < valid ? *reinterpret_cast<const uint4*>(x.at(t0 + row, h) + c * VE) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void store(float* dst, int tid) const {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = tid + u * kPsThreads, row = i / VPR, c = i % VPR;
      RowTile<T, D, D + 4, 1, VPR>::put(r[u], dst + row * (D + 4) + c * VE);
    }
  }
};

template <typename T>
__device__ __forceinline__ void store4(T* dst, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
  } else {
    __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<uint32_t*>(&x), *reinterpret_cast<uint32_t*>(&y));
  }
}

// Keys of a forward tile: with twice as many a row's maximum and sum close half
// as often and a load feeds more products (d = 64, the case above: 63 us with 32, 57
// with 64; 30 sequences of 64, where the last half tile counts, 15 and 17); at d = 128
// the registers of the next tile's rows leave no room for it. Three CTAs an SM at d =
// 64 (four, with the registers that leaves: 70 us), two at d = 128 (118 -> 102 us on
// the same lengths against the registers of three).
template <int D>
constexpr int ps_keys() {
  return D == 64 ? 64 : 32;
}
template <int D>
constexpr size_t ps_fwd_smem() {
  return (size_t)((kPsRows + 2 * ps_keys<D>()) * (D + 4) + kPsRows * (ps_keys<D>() + 4)) * 4;
}
template <int D>
constexpr size_t ps_bwd_smem() {
  return (size_t)((2 * kPsRows + 2 * kPsCols) * (D + 4) + 2 * kPsRows * kPsPst + 2 * kPsRows) * 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPsThreads, 3 - (D == 128)) packed_simt_fwd_kernel(const PackedArgs<T> a, int64_t slots) {
  constexpr int ST = D + 4, COLS = ps_keys<D>(), PST = COLS + 4;
  extern __shared__ __align__(16) float ps_smem[];
  float* sQ = ps_smem;
  float* sK = sQ + kPsRows * ST;
  float* sV = sK + COLS * ST;
  float* sP = sV + COLS * ST;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, h = (int)(blockIdx.x % (unsigned)a.Hq), hk = h / a.G;
  SlotTile t;
  if (!work_tile<kPsRows, true>(a.sq, a.sk, blockIdx.x / (unsigned)a.Hq, slots, &t)) return;
  const SeqRange kr = t.other;
  const int r0 = t.tile * kPsRows, rows = min(kPsRows, t.r.len - r0);
  const int shift = kr.len - t.r.len;                       // row i sees keys j <= i + shift
  const int seen = max(0, min(kr.len, r0 + rows + shift));  // keys the last row sees
  load_rows_f32<T, D, kPsRows, ST, kPsThreads>(sQ, a.q, t.r.first + r0, h, rows, tid);

  // Running maximum and sum of each of the thread's rows; the 16 threads of a
  // row hold the same values.
  float m[4], l[4], o[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int u = 0; u < D / 16; ++u) o[i][u] = 0.f;
  }
  PsAhead<T, D, COLS> nk, nv;
  if (seen > 0) {
    nk.issue(a.k, kr.first, hk, seen, tid);
    nv.issue(a.v, kr.first, hk, seen, tid);
  }
  for (int j0 = 0; j0 < seen; j0 += COLS) {
    __syncthreads();
    nk.store(sK, tid);
    nv.store(sV, tid);
    __syncthreads();
    if (j0 + COLS < seen) {
      nk.issue(a.k, kr.first + j0 + COLS, hk, seen - j0 - COLS, tid);
      nv.issue(a.v, kr.first + j0 + COLS, hk, seen - j0 - COLS, tid);
    }
    auto work = [&](auto columns) {  // on the tile's first 16 N keys
      constexpr int N = decltype(columns)::value;
      float c[4][N];
      ps_scores<D, ST, N>(sQ, sK, ty, tx, c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int last = min(kr.len - 1, r0 + 4 * ty + i + shift);
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < N; ++y) {
          c[i][y] = j0 + tx + 16 * y <= last ? c[i][y] * a.scale : -INFINITY;
          top = fmaxf(top, c[i][y]);
        }
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float mn = fmaxf(m[i], top);
        const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every p below is 0
        const float fix = expf(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < N; ++y) {
          const float p = expf(c[i][y] - base);
          sum += p;
          sP[(4 * ty + i) * PST + tx + 16 * y] = p;
        }
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        l[i] = l[i] * fix + sum;
        m[i] = mn;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) o[i][u] *= fix;
      }
      __syncwarp();  // rows 4 ty .. are written and read by one half warp
      ps_accumulate<D, ST, 16 * N, PST>(sP, sV, ty, tx, o);
    };
    if (COLS > 32 && seen - j0 <= 32)
      work(std::integral_constant<int, 2>{});
    else
      work(std::integral_constant<int, COLS / 16>{});
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
    const bool none = r0 + r + shift < 0;  // by its place: a maximum of -inf may be NaN scores'
    const float inv = none ? 0.f : 1.f / l[i];
    T* dst = a.out.at(t.r.first + r0 + r, h);
#pragma unroll
    for (int u = 0; u < D / 64; ++u)
      store4(dst + 4 * tx + 64 * u, o[i][4 * u] * inv, o[i][4 * u + 1] * inv, o[i][4 * u + 2] * inv,
             o[i][4 * u + 3] * inv);
    if (tx == 0 && a.lse)
      a.lse[(int64_t)h * a.sq.T + t.r.first + r0 + r] = none ? -INFINITY : m[i] + logf(l[i]);
  }
}

// delta_i = dout_i . out_i: 16 bytes of both a lane, D / 8 (bf16) or D / 4 lanes
// a row; reading the two bounds it.
template <typename T, int D>
__global__ void __launch_bounds__(256) packed_delta_kernel(const PackedGradArgs<T> a) {
  constexpr int VE = 16 / (int)sizeof(T), LPR = D / VE;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
  const int c = (int)(threadIdx.x % LPR) * VE;
  const bool real = i < (int64_t)a.sq.T * a.Hq;
  const int64_t t = real ? i / a.Hq : 0;
  const int h = real ? (int)(i % a.Hq) : 0;
  float x[VE], y[VE], s = 0.f;
  RowTile<T, D, D, 1, LPR>::put(*reinterpret_cast<const uint4*>(a.dout.at(t, h) + c), x);
  RowTile<T, D, D, 1, LPR>::put(*reinterpret_cast<const uint4*>(a.out.at(t, h) + c), y);
#pragma unroll
  for (int e = 0; e < VE; ++e) s = fmaf(x[e], y[e], s);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (real && c == 0) a.delta[(int64_t)h * a.sq.T + t] = s;
}

// dq (KEYS = false): the CTA owns 32 query rows (X = Q, Y = dout) and streams
// the keys and values it sees. dk, dv (KEYS = true): it owns 32 keys (X = K,
// Y = V) and streams the queries that see them, head after head of the group,
// so the sums over the group's heads have one order. With s = X a^T and
// e = Y b^T both form p = exp(s - lse), ds = p (e - delta) and accumulate
// ds a (and p b for dv).
template <typename T, int D, bool KEYS>
__global__ void __launch_bounds__(kPsThreads) packed_simt_bwd_kernel(const PackedGradArgs<T> a, int64_t slots) {
  constexpr int ST = D + 4;
  extern __shared__ __align__(16) float ps_smem[];
  float* sX = ps_smem;
  float* sY = sX + kPsRows * ST;
  float* sA = sY + kPsRows * ST;
  float* sB = sA + kPsCols * ST;
  float* sP = sB + kPsCols * ST;
  float* sD = sP + kPsRows * kPsPst;
  float* sL = sD + kPsRows * kPsPst;  // lse and delta of the query rows at hand
  float* sE = sL + kPsRows;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const unsigned heads = KEYS ? a.Hkv : a.Hq;
  const int head = (int)(blockIdx.x % heads);  // the output's
  SlotTile t;
  if (!work_tile<kPsRows, !KEYS>(KEYS ? a.sk : a.sq, KEYS ? a.sq : a.sk, blockIdx.x / heads, slots, &t)) return;
  const SeqRange other = t.other;
  const int nq = KEYS ? other.len : t.r.len, nk = KEYS ? t.r.len : other.len, shift = nk - nq;
  const int r0 = t.tile * kPsRows, rows = min(kPsRows, t.r.len - r0);
  const int hk = KEYS ? head : head / a.G;
  // The streamed range: keys 0 .. the last row's, or queries from the first
  // that sees key r0 on.
  const int c_begin = KEYS ? max(0, r0 - shift) : 0;
  const int c_end = KEYS ? nq : max(0, min(nk, r0 + rows + shift));

  float acc[4][D / 16], acc2[KEYS ? 4 : 1][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      acc[i][u] = 0.f;
      if (KEYS) acc2[KEYS ? i : 0][u] = 0.f;
    }
  const int h_first = KEYS ? hk * a.G : head, h_last = KEYS ? h_first + a.G : h_first + 1;
  for (int h = h_first; h < h_last; ++h) {
    const float* lse = a.lse + (int64_t)h * a.sq.T;
    const float* delta = a.delta + (int64_t)h * a.sq.T;
    __syncthreads();
    if (h == h_first) {
      load_rows_f32<T, D, kPsRows, ST, kPsThreads>(sX, KEYS ? a.k : a.q, t.r.first + r0, KEYS ? hk : h, rows, tid);
      load_rows_f32<T, D, kPsRows, ST, kPsThreads>(sY, KEYS ? a.v : a.dout, t.r.first + r0, KEYS ? hk : h, rows, tid);
      if (!KEYS && tid < kPsRows) {
        sL[tid] = tid < rows ? lse[t.r.first + r0 + tid] : 0.f;
        sE[tid] = tid < rows ? delta[t.r.first + r0 + tid] : 0.f;
      }
    }
    for (int c0 = c_begin; c0 < c_end; c0 += kPsCols) {
      __syncthreads();
      const int left = (KEYS ? nq : nk) - c0;
      load_rows_f32<T, D, kPsCols, ST, kPsThreads>(sA, KEYS ? a.q : a.k, other.first + c0, KEYS ? h : hk, left, tid);
      load_rows_f32<T, D, kPsCols, ST, kPsThreads>(sB, KEYS ? a.dout : a.v, other.first + c0, KEYS ? h : hk, left,
                                                   tid);
      if (KEYS && tid < kPsCols) {
        sL[tid] = tid < left ? lse[other.first + c0 + tid] : 0.f;
        sE[tid] = tid < left ? delta[other.first + c0 + tid] : 0.f;
      }
      __syncthreads();
      float s[4][2], e[4][2];
      ps_scores<D, ST, 2>(sX, sA, ty, tx, s);
      ps_scores<D, ST, 2>(sY, sB, ty, tx, e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int r = 4 * ty + i, c = tx + 16 * u;
          const int qi = KEYS ? c0 + c : r0 + r, kj = KEYS ? r0 + r : c0 + c;
          const bool ok = qi < nq && kj < nk && kj <= qi + shift;
          const float p = ok ? expf(s[i][u] * a.scale - sL[KEYS ? c : r]) : 0.f;
          sP[r * kPsPst + c] = p;
          sD[r * kPsPst + c] = ok ? p * (e[i][u] - sE[KEYS ? c : r]) : 0.f;
        }
      __syncwarp();
      ps_accumulate<D, ST, kPsCols>(sD, sA, ty, tx, acc);
      if constexpr (KEYS) ps_accumulate<D, ST, kPsCols>(sP, sB, ty, tx, acc2);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
    const int64_t row = t.r.first + r0 + r;
    T* d0 = KEYS ? a.dk.at(row, hk) : a.dq.at(row, head);
#pragma unroll
    for (int u = 0; u < D / 64; ++u) {
      store4(d0 + 4 * tx + 64 * u, acc[i][4 * u] * a.scale, acc[i][4 * u + 1] * a.scale, acc[i][4 * u + 2] * a.scale,
             acc[i][4 * u + 3] * a.scale);
      if constexpr (KEYS)
        store4(a.dv.at(row, hk) + 4 * tx + 64 * u, acc2[i][4 * u], acc2[i][4 * u + 1], acc2[i][4 * u + 2],
               acc2[i][4 * u + 3]);
    }
  }
}

}  // namespace infini

// Few queries against many keys (a token against its cache): every CTA takes
// one chunk of one sequence's keys for one key head and a handful of rows (the
// group's heads x the sequence's queries), keeps a running maximum and sum,
// and writes (m, l, o) of its chunk; a second kernel joins the chunks:
//   m = max m_c,  l = sum l_c exp(m_c - m),  o = sum o_c exp(m_c - m) / l.
// Reading K and V once bounds it: rows of one group share the reads.
#pragma once

#include "packed_common.cuh"
#include "packed_simt_kernels.cuh"

namespace infini {

constexpr int kSplitThreads = 128;
constexpr int kSplitRows = 4;  // rows (query, head of the group) of one CTA

struct SplitShape {
  int chunk;     // keys of one chunk; the last of the grid takes what is left
  int n_chunks;  // grid size along the keys
};

// (m, l, o[D]) of one row's chunk, rows numbered t * Hq + h.
__device__ __forceinline__ float* split_partial(float* part, const SplitShape& s, int64_t row, int c, int D) {
  return part + (row * s.n_chunks + c) * (D + 2);
}
__device__ __forceinline__ void split_chunk(const SplitShape& s, int c, int nk, int* begin, int* end) {
  *begin = min(nk, c * s.chunk);
  *end = c == s.n_chunks - 1 ? nk : min(nk, (c + 1) * s.chunk);
}

// 8 lanes hold one key, so a warp works on 4 keys and the CTA on 16 at a time;
// each group of 8 lanes keeps its own maximum, sum and output.
template <typename T, int D>
__global__ void __launch_bounds__(kSplitThreads) packed_split_kernel(const PackedArgs<T> a, SplitShape s,
                                                                     float* __restrict__ part) {
  constexpr int VE = 16 / (int)sizeof(T), NV = D / (8 * VE), PER = D / 8, GROUPS = kSplitThreads / 8;
  extern __shared__ __align__(16) float split_smem[];  // [GROUPS][kSplitRows][D + 2]
  const int seq = blockIdx.y / a.Hkv, hk = blockIdx.y % a.Hkv, lane8 = threadIdx.x & 7, group = threadIdx.x >> 3;
  const SeqRange qr = seq_range(a.sq, seq), kr = seq_range(a.sk, seq);
  const int shift = kr.len - qr.len, n_rows = qr.len * a.G;
  int begin, end;
  split_chunk(s, blockIdx.x, kr.len, &begin, &end);
  for (int row0 = blockIdx.z * kSplitRows; row0 < n_rows; row0 += gridDim.z * kSplitRows) {
    float q[kSplitRows][PER], o[kSplitRows][PER], m[kSplitRows], l[kSplitRows];
    int last[kSplitRows];
#pragma unroll
    for (int r = 0; r < kSplitRows; ++r) {
      const int row = row0 + r;
      const bool ok = row < n_rows;
      const int qi = ok ? row / a.G : 0, h = hk * a.G + (ok ? row % a.G : 0);
      last[r] = ok ? qi + shift : -1;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          q[r][v * VE + e] = ok ? to_f32(a.q.at(qr.first + qi, h)[(v * 8 + lane8) * VE + e]) * a.scale : 0.f;
          o[r][v * VE + e] = 0.f;
        }
    }
    for (int j = begin + group; j < end; j += GROUPS) {
      const T* kp = a.k.at(kr.first + j, hk) + lane8 * VE;
      const T* vp = a.v.at(kr.first + j, hk) + lane8 * VE;
      float x[kSplitRows], kv[VE];
#pragma unroll
      for (int r = 0; r < kSplitRows; ++r) x[r] = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        RowTile<T, D, D, 1, 1>::put(*reinterpret_cast<const uint4*>(kp + v * 8 * VE), kv);
#pragma unroll
        for (int r = 0; r < kSplitRows; ++r)
#pragma unroll
          for (int e = 0; e < VE; ++e) x[r] = fmaf(q[r][v * VE + e], kv[e], x[r]);
      }
      float p[kSplitRows];
#pragma unroll
      for (int r = 0; r < kSplitRows; ++r) {
#pragma unroll
        for (int w = 4; w > 0; w >>= 1) x[r] += __shfl_xor_sync(0xffu << (8 * (group & 3)), x[r], w);
        if (j > last[r]) x[r] = -INFINITY;
        const float mn = fmaxf(m[r], x[r]), base = mn == -INFINITY ? 0.f : mn;
        const float fix = expf(m[r] - base);
        p[r] = expf(x[r] - base);
        l[r] = l[r] * fix + p[r];
        m[r] = mn;
#pragma unroll
        for (int e = 0; e < PER; ++e) o[r][e] *= fix;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        RowTile<T, D, D, 1, 1>::put(*reinterpret_cast<const uint4*>(vp + v * 8 * VE), kv);
#pragma unroll
        for (int r = 0; r < kSplitRows; ++r)
#pragma unroll
          for (int e = 0; e < VE; ++e)
            // a key that the row does not see adds nothing, whatever its value
            if (j <= last[r]) o[r][v * VE + e] = fmaf(p[r], kv[e], o[r][v * VE + e]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSplitRows; ++r) {
      float* d = split_smem + (group * kSplitRows + r) * (D + 2);
      if (lane8 == 0) {
        d[0] = m[r];
        d[1] = l[r];
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VE; ++e) d[2 + (v * 8 + lane8) * VE + e] = o[r][v * VE + e];
    }
    __syncthreads();
    // Warp r joins row r's groups.
    const int r = threadIdx.x >> 5, lane = threadIdx.x & 31, row = row0 + r;
    if (row < n_rows) {
      float top = -INFINITY;
      for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, split_smem[(g * kSplitRows + r) * (D + 2)]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc[D / 32];
#pragma unroll
      for (int u = 0; u < D / 32; ++u) acc[u] = 0.f;
      for (int g = 0; g < GROUPS; ++g) {
        const float* d = split_smem + (g * kSplitRows + r) * (D + 2);
        const float w = expf(d[0] - base);
        sum += d[1] * w;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc[u] = fmaf(d[2 + lane + 32 * u], w, acc[u]);
      }
      const int64_t t = qr.first + row / a.G;
      const int h = hk * a.G + row % a.G;
      float* dst = split_partial(part, s, t * a.Hq + h, blockIdx.x, D);
      if (lane == 0) {
        dst[0] = top;
        dst[1] = sum;
      }
#pragma unroll
      for (int u = 0; u < D / 32; ++u) dst[2 + lane + 32 * u] = acc[u];
    }
  }
}

// One warp joins one row's chunks.
template <typename T, int D>
__global__ void __launch_bounds__(128) packed_split_join_kernel(const PackedArgs<T> a, SplitShape s,
                                                                const float* __restrict__ part) {
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const SeqRange qr = seq_range(a.sq, seq), kr = seq_range(a.sk, seq);
  // Chunks that hold keys; the rest of the grid wrote empty ones.
  const int n = min(s.n_chunks, (kr.len + s.chunk - 1) / s.chunk);
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); i < (int64_t)qr.len * a.Hq;
       i += (int64_t)gridDim.x * 4) {
    const int64_t t = qr.first + i / a.Hq;
    const int h = (int)(i % a.Hq);
    const float* src = part + (t * a.Hq + h) * s.n_chunks * (D + 2);
    float top = -INFINITY;
    for (int c = 0; c < n; ++c) top = fmaxf(top, src[(int64_t)c * (D + 2)]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int u = 0; u < D / 32; ++u) acc[u] = 0.f;
    for (int c = 0; c < n; ++c) {
      const float* d = src + (int64_t)c * (D + 2);
      const float w = expf(d[0] - base);
      sum += d[1] * w;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) acc[u] = fmaf(d[2 + lane + 32 * u], w, acc[u]);
    }
    const float inv = top == -INFINITY ? 0.f : 1.f / sum;
    T* dst = a.out.at(t, h);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) dst[lane + 32 * u] = from_f32<T>(acc[u] * inv);
    if (lane == 0 && a.lse) a.lse[(int64_t)h * a.sq.T + t] = top == -INFINITY ? -INFINITY : top + logf(sum);
  }
}

}  // namespace infini

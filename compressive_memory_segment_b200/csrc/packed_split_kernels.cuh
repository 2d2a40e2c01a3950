// Few queries against many keys (a token against its cache): every CTA takes
// one chunk of one sequence's keys for one key head and a handful of rows (the
// group's heads x the sequence's queries), keeps a running maximum and sum,
// and writes (m, l, o) of its chunk; a second kernel joins the chunks:
//   m = max m_c,  l = sum l_c exp(m_c - m),  o = sum o_c exp(m_c - m) / l.
// Reading K and V once bounds it: rows of one group share the reads. Measured: 48
// sequences of 300-8192 keys, 32 / 8 heads, d = 128, one query each, bf16: 133 us,
// 5.2 TB/s (0.80 of a plain copy); fp32, the kernel below: 580 us, 2.4 TB/s, each key
// loaded where it is used.
#pragma once

#include "packed_common.cuh"
#include "packed_simt_kernels.cuh"
#include "delta_chunk_kernels.cuh"  // the warp-level products and copies

namespace infini {

constexpr int kSplitThreads = 128;
constexpr int kSplitRows = 4;  // rows (query, head of the group) of one CTA

struct SplitShape {
  int chunk;     // keys of one chunk; the last of the grid takes what is left
  int n_chunks;  // chunks of a sequence, the fastest part of the grid's x (then key head, sequence)
};
// This CTA's place in the grid.
struct SplitPlace {
  int chunk, seq, head;
};
__device__ __forceinline__ SplitPlace split_place(const SplitShape& s, int Hkv) {
  const int u = (int)(blockIdx.x / (unsigned)s.n_chunks);
  return {(int)(blockIdx.x % (unsigned)s.n_chunks), u / Hkv, u % Hkv};
}

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
  const SplitPlace at = split_place(s, a.Hkv);
  const int seq = at.seq, hk = at.head, lane8 = threadIdx.x & 7, group = threadIdx.x >> 3;
  const SeqPair both = seq_pair(a.sq, a.sk, seq);
  const SeqRange qr = both.own, kr = both.other;
  const int shift = kr.len - qr.len, n_rows = qr.len * a.G;
  int begin, end;
  split_chunk(s, at.chunk, kr.len, &begin, &end);
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
      float* dst = split_partial(part, s, t * a.Hq + h, at.chunk, D);
      if (lane == 0) {
        dst[0] = top;
        dst[1] = sum;
      }
#pragma unroll
      for (int u = 0; u < D / 32; ++u) dst[2 + lane + 32 * u] = acc[u];
    }
  }
}

// The same for bf16 on the tensor cores. A CTA takes 16 rows (query, head of the
// group) of one key head and one chunk of its keys; tiles of 64 keys and values
// come through a ring of cp.async stages, so the loads of the next tiles are in
// flight under the current one (reading them is what bounds the kernel: each
// value once per 16 rows). Warp w has the tile's keys 16 w .. and its own running
// maximum, sum and [16, D] output in registers: scores are Q K^T over warp-level
// products (one m16n8k16 covers all rows of a group; the 128-row tiles of tcgen05
// would be empty but for these few), P goes from result to operand registers, and
// the four warps' parts are joined once at the end. V rows behind the sequence
// are zeroed by the copies (0 x NaN is NaN).
constexpr int kSmRows = 16, kSmTile = 64, kSmThreads = 128;
template <int D>
struct SplitMma {
  static constexpr uint32_t kTileBytes = kSmTile * D * 2, kStage = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr uint32_t kTotal = kStages * kStage + 1024;
};

template <int D>
__global__ void __launch_bounds__(kSmThreads)
packed_split_mma_kernel(const PackedArgs<__nv_bfloat16> a, SplitShape s, float* __restrict__ part) {
  using M = SplitMma<D>;
  constexpr int RB = D * 2, P = D / 8, ND = D / 8, KS = D / 16;
  extern __shared__ __align__(128) uint8_t sm_raw[];
  const uint32_t base = (dc_smem(sm_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, qd = lane & 3;
  const SplitPlace at = split_place(s, a.Hkv);
  const int seq = at.seq, hk = at.head;
  const SeqPair both = seq_pair(a.sq, a.sk, seq);
  const SeqRange qr = both.own, kr = both.other;
  const int shift = kr.len - qr.len, n_rows = qr.len * a.G;
  int begin, end;
  split_chunk(s, at.chunk, kr.len, &begin, &end);
  const int tiles = (end - begin + kSmTile - 1) / kSmTile;
  const float scale2 = a.scale * 1.4426950408889634f;
  auto load = [&](int t) {
    if (t < tiles) {
      const uint32_t dst = base + (t % M::kStages) * M::kStage;
      const int j0 = begin + t * kSmTile, valid = end - j0;
      for (int i = tid; i < kSmTile * P; i += kSmThreads) {
        const int r = i / P, c = i % P;
        const bool real = r < valid;
        const int64_t row = kr.first + j0 + (real ? r : 0);
        cp16(dst + dc_at<RB>(r, c), a.k.at(row, hk) + c * 8, real);
        cp16(dst + M::kTileBytes + dc_at<RB>(r, c), a.v.at(row, hk) + c * 8, real);
      }
    }
    cp_commit();  // one group a tile, empty behind the last
  };
  for (int row0 = blockIdx.z * kSmRows; row0 < n_rows; row0 += gridDim.z * kSmRows) {
    if (tiles > 0) {
#pragma unroll
      for (int t = 0; t < M::kStages - 1; ++t) load(t);
    }
    // Q as left operands, straight from global memory (rows gr and gr + 8).
    uint32_t q[KS][4];
    int last[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = row0 + gr + 8 * x;
      const bool ok = row < n_rows;
      const int qi = ok ? row / a.G : 0, h = hk * a.G + (ok ? row % a.G : 0);
      last[x] = ok ? min(end - 1, qi + shift) : -1;
      const __nv_bfloat16* src = a.q.at(qr.first + qi, h) + 2 * qd;
#pragma unroll
      for (int z = 0; z < KS; ++z) {
        q[z][x] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * z) : 0u;
        q[z][2 + x] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * z + 8) : 0u;
      }
    }
    float o[ND][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[x][y] = 0.f;
    for (int t = 0; t < tiles; ++t) {
      asm volatile("cp.async.wait_group %0;" ::"n"(M::kStages - 2) : "memory");
      __syncthreads();  // tile t is there for all; tile t - 1 is read by all
      load(t + M::kStages - 1);
      const uint32_t sk = base + (t % M::kStages) * M::kStage, sv = sk + M::kTileBytes;
      float c[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) c[x][y] = 0.f;
#pragma unroll
      for (int z = 0; z < KS; ++z) {
        uint32_t b[4];
        ldsm(b, sk + right_at<RB>(16 * warp, 2 * z, lane));
        mma16(c[0], q[z], b[0], b[1]);
        mma16(c[1], q[z], b[2], b[3]);
      }
      const int j0 = begin + t * kSmTile + 16 * warp + 2 * qd;
#pragma unroll
      for (int x = 0; x < 2; ++x) {  // rows gr, gr + 8
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float& v = c[n][2 * x + y];
            v = j0 + 8 * n + y <= last[x] ? v * scale2 : -INFINITY;
            top = fmaxf(top, v);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[x], top), from = mn == -INFINITY ? 0.f : mn;
        const float fix = exp2f(m[x] - from);
        m[x] = mn;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            c[n][2 * x + y] = exp2f(c[n][2 * x + y] - from);
            sum += c[n][2 * x + y];
          }
        l[x] = l[x] * fix + sum;  // of this lane's columns
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          o[n][2 * x] *= fix;
          o[n][2 * x + 1] *= fix;
        }
      }
      const uint32_t p[4] = {pack2(c[0][0], c[0][1]), pack2(c[0][2], c[0][3]), pack2(c[1][0], c[1][1]),
                             pack2(c[1][2], c[1][3])};
#pragma unroll
      for (int n = 0; n < ND; n += 2) {
        uint32_t b[4];
        ldsm_t(b, sv + right_t_at<RB>(16 * warp, n, lane));
        mma16(o[n], p, b[0], b[1]);
        mma16(o[n + 1], p, b[2], b[3]);
      }
    }
    cp_wait();
    __syncthreads();
    // Join the four warps: [4][16][D + 2] in the ring.
    float* sm = reinterpret_cast<float*>(__cvta_shared_to_generic(base));
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      float* d = sm + (warp * kSmRows + gr + 8 * x) * (D + 2);
      if (qd == 0) {
        d[0] = m[x];
        d[1] = l[x];
      }
#pragma unroll
      for (int n = 0; n < ND; ++n)
        *reinterpret_cast<float2*>(d + 2 + 8 * n + 2 * qd) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
    }
    __syncthreads();
    for (int rr = warp; rr < kSmRows && row0 + rr < n_rows; rr += 4) {
      const int row = row0 + rr;
      float mw[4], top = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        mw[w] = sm[(w * kSmRows + rr) * (D + 2)];
        top = fmaxf(top, mw[w]);
      }
      const float from = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc[D / 32];
#pragma unroll
      for (int u = 0; u < D / 32; ++u) acc[u] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float* d = sm + (w * kSmRows + rr) * (D + 2);
        const float f = exp2f(mw[w] - from);
        sum = fmaf(d[1], f, sum);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc[u] = fmaf(d[2 + lane + 32 * u], f, acc[u]);
      }
      const int64_t t = qr.first + row / a.G;
      const int h = hk * a.G + row % a.G;
      float* dst = split_partial(part, s, t * a.Hq + h, at.chunk, D);
      if (lane == 0) {
        dst[0] = top * 0.6931471805599453f;  // the join works in natural logs
        dst[1] = sum;
      }
#pragma unroll
      for (int u = 0; u < D / 32; ++u) dst[2 + lane + 32 * u] = acc[u];
    }
    __syncthreads();
  }
}

// One warp joins one row's chunks.
template <typename T, int D>
__global__ void __launch_bounds__(128) packed_split_join_kernel(const PackedArgs<T> a, SplitShape s,
                                                                const float* __restrict__ part) {
  const int seq = blockIdx.x, lane = threadIdx.x & 31;
  const SeqPair both = seq_pair(a.sq, a.sk, seq);
  const SeqRange qr = both.own, kr = both.other;
  // Chunks that hold keys; the rest of the grid wrote empty ones.
  const int n = min(s.n_chunks, (kr.len + s.chunk - 1) / s.chunk);
  for (int64_t i = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 5); i < (int64_t)qr.len * a.Hq;
       i += (int64_t)gridDim.y * 4) {
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
    const bool none = i / a.Hq + kr.len - qr.len < 0;  // by its place: a maximum of -inf may be NaN scores'
    const float inv = none ? 0.f : 1.f / sum;
    T* dst = a.out.at(t, h);
#pragma unroll
    for (int u = 0; u < D / 32; ++u) dst[lane + 32 * u] = from_f32<T>(acc[u] * inv);
    if (lane == 0 && a.lse) a.lse[(int64_t)h * a.sq.T + t] = none ? -INFINITY : top + logf(sum);
  }
}

}  // namespace infini

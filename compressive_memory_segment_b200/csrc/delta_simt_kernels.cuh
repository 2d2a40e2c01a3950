// The gated delta rule on the CUDA cores, fp32 arithmetic throughout: short
// forwards token by token, longer ones and the gradient in chunks, and the
// one-token step. fp32 inputs run here.
#pragma once

#include "delta_common.cuh"
#include "packed_simt_kernels.cuh"

namespace infini {

constexpr int kDsThreads = 256;
constexpr int kDsCols = 32;    // columns of S (values) of one forward CTA
// A forward over at most this many tokens is the recurrence, a longer one goes in
// chunks. Recurrence against chunks, bf16, d = 128, 16 heads: 48 tokens 20 / 25 us
// (1 sequence) and 365 / 444 (64), 64 tokens 25 / 25 and 471 / 453, 128 tokens
// 45 / 37 and 898 / 757.
constexpr int kDsRecurMost = 48;
constexpr int kDsBlock = 16;   // tokens staged at a time
constexpr int kDsChunk = 32;   // tokens of a chunk

// Rows of W elements from column `col` on, on their way through registers while
// the tokens before them are worked on (rows behind `valid` as zeros).
template <typename T, int ROWS, int W, int ST>
struct DsAhead {
  static constexpr int VE = 16 / (int)sizeof(T), VPR = W / VE, ALL = ROWS * VPR;
  static constexpr int PER = (ALL + kDsThreads - 1) / kDsThreads;
  uint4 r[PER];
  __device__ __forceinline__ void issue(const RowsOf<const T>& x, int64_t t0, int h, int col, int valid, int tid) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = tid + u * kDsThreads, row = i / VPR, c = i % VPR;
      r[u] = row < min(valid, ROWS) ? *reinterpret_cast<const uint4*>(x.at(t0 + row, h) + col + c * VE)
                                    : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void store(float* dst, int tid) const {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = tid + u * kDsThreads, row = i / VPR, c = i % VPR;
      if (ALL % kDsThreads == 0 || i < ALL) RowTile<T, W, ST, 1, VPR>::put(r[u], dst + row * ST + c * VE);
    }
  }
};

// Columns of S are independent, so a CTA walks the tokens with 32 of them. 8
// lanes share a column (D / 8 rows each, in registers); the two dot products
// over d_k close with three shuffles each. The chain of those and the reads of k and
// q bound it: 0.22 us a token (200 tokens, d = 64, fp32: 45 us; the chunks below 28
// and 7 to form them).
template <typename T, int D>
__device__ __forceinline__ void ds_recur(const DeltaArgs<T>& a, int strip) {
  constexpr int PER = D / 8;
  __shared__ __align__(16) float sQ[kDsBlock][D], sK[kDsBlock][D];
  __shared__ __align__(16) float sV[kDsBlock][kDsCols];
  __shared__ float sG[kDsBlock], sB[kDsBlock];
  const int tid = threadIdx.x, part = tid & 7, c = tid >> 3, col = strip * kDsCols + c;
  const int h = blockIdx.y, seq = blockIdx.z, hk = h / a.G;
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t base = ((int64_t)seq * a.Hv + h) * D * D;
  float S[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = (i >> 2) * 32 + part * 4 + (i & 3);
    S[i] = a.S_in ? a.S_in[base + (int64_t)row * D + col] : 0.f;
  }
  DsAhead<T, kDsBlock, D, D> rq, rk;
  DsAhead<T, kDsBlock, kDsCols, kDsCols> rv;
  float rg = 0.f, rb = 0.f;
  auto issue = [&](int t0) {
    rq.issue(a.q, r.first + t0, hk, 0, r.len - t0, tid);
    rk.issue(a.k, r.first + t0, hk, 0, r.len - t0, tid);
    rv.issue(a.v, r.first + t0, h, strip * kDsCols, r.len - t0, tid);
    if (tid < min(kDsBlock, r.len - t0)) {
      rg = to_f32(*a.g.at(r.first + t0 + tid, h));
      rb = to_f32(*a.beta.at(r.first + t0 + tid, h));
    }
  };
  if (r.len > 0) issue(0);
  for (int t0 = 0; t0 < r.len; t0 += kDsBlock) {
    __syncthreads();
    const int n = min(kDsBlock, r.len - t0);
    rq.store(&sQ[0][0], tid);
    rk.store(&sK[0][0], tid);
    rv.store(&sV[0][0], tid);
    if (tid < n) {
      sG[tid] = expf(delta_log(rg));
      sB[tid] = rb;
    }
    __syncthreads();
    if (t0 + kDsBlock < r.len) issue(t0 + kDsBlock);
    // The next token's operands are read while this one's sums close: the chain
    // from token to token is the decay, one dot product and one update.
    float k[PER], q[PER], kn[PER], qn[PER], decay = sG[0], beta = sB[0], v = sV[0][c];
    auto fetch = [&](int t, float(&kk)[PER], float(&qq)[PER]) {
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        *reinterpret_cast<float4*>(kk + i) = *reinterpret_cast<const float4*>(&sK[t][(i >> 2) * 32 + part * 4]);
        *reinterpret_cast<float4*>(qq + i) = *reinterpret_cast<const float4*>(&sQ[t][(i >> 2) * 32 + part * 4]);
      }
    };
    fetch(0, k, q);
    T* out = a.out.p ? a.out.at(r.first + t0, h) + col : nullptr;
    float y = 0.f;
    for (int t = 0; t < n; ++t) {
      const int tn = min(t + 1, kDsBlock - 1);
      fetch(tn, kn, qn);
      const float dn = sG[tn], bn = sB[tn], vn = sV[tn][c];
      float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        S[i] *= decay;
        S[i + 1] *= decay;
        x0 = fmaf(S[i], k[i], x0);
        x1 = fmaf(S[i + 1], k[i + 1], x1);
      }
      float x = x0 + x1;
#pragma unroll
      for (int s = 4; s > 0; s >>= 1) {  // the last token's output closes beside this one's x
        x += __shfl_xor_sync(0xffffffffu, x, s);
        y += __shfl_xor_sync(0xffffffffu, y, s);
      }
      if (t > 0 && part == 0 && out) out[(t - 1) * a.out.st] = from_f32<T>(a.scale * y);
      const float u = beta * (v - x);
#pragma unroll
      for (int i = 0; i < PER; i += 2) {
        S[i] = fmaf(k[i], u, S[i]);
        S[i + 1] = fmaf(k[i + 1], u, S[i + 1]);
        y0 = fmaf(S[i], q[i], y0);
        y1 = fmaf(S[i + 1], q[i + 1], y1);
      }
      y = y0 + y1;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        k[i] = kn[i];
        q[i] = qn[i];
      }
      decay = dn;
      beta = bn;
      v = vn;
    }
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) y += __shfl_xor_sync(0xffffffffu, y, s);
    if (part == 0 && out) out[(n - 1) * a.out.st] = from_f32<T>(a.scale * y);
  }
  if (a.S_out) {
#pragma unroll
    for (int i = 0; i < PER; ++i) a.S_out[base + (int64_t)((i >> 2) * 32 + part * 4 + (i & 3)) * D + col] = S[i];
  }
}
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_fwd_kernel(const DeltaArgs<T> a) {
  ds_recur<T, D>(a, blockIdx.x);
}

// Chunks of 32 tokens. With G_i the sum of the chunk's log decays up to i,
// e_ij = exp(G_i - G_j), w_i = exp(G_C - G_i), S and dS+ the state at the chunk's
// start and its end's gradient:
//   N_ij = beta_i e_ij k_i.k_j (j < i), T = (I + N)^-1, R = V - diag(e^G) K S,
//   U = T diag(beta) R, P_ij = scale e_ij q_i.k_j (j <= i)
//   O = scale diag(e^G) Q S + P U,  S+ = e^G_C S + K^T diag(w) U
//   dU = P^T dO + diag(w) K dS+,  Z = T^T dU,  dV = diag(beta) Z
//   dS = e^G_C dS+ + scale Q^T diag(e^G) dO - K^T diag(e^G beta) Z
//   M = dO U^T (j <= i), H = Z U^T (j < i), F_ij = beta_i H_ij e_ij
//   dq_i = scale (e^G_i S dO_i + sum_j e_ij M_ij k_j)
//   dk_j = scale sum_i e_ij M_ij q_i - e^G_j beta_j S Z_j + w_j dS+ u_j - sum_i (F_ij + F_ji) k_i
//   dbeta_i = Z_i.R_i - sum_j H_ij e_ij k_i.k_j
//   dg_t = sum_{i >= t} s_i + sum_{i >= t > j} Q_ij + sum_{j < t} x_j + e^G_C <dS+, S>,
//     s_i = q_i.(scale e^G_i S dO_i) - k_i.(e^G_i beta_i S Z_i), x_j = w_j k_j.(dS+ u_j),
//     Q_ij = P_ij M_ij - F_ij k_i.k_j: what passes over the decay of token t, and no more, so
//     that nothing has to cancel.
// Only S and dS run from chunk to chunk (32 columns of one a CTA); what needs
// neither is formed for all chunks at once before, the rest of the gradients for
// all chunks at once behind. Measured on 2 sequences of up to 200 tokens, 4 heads,
// d = 64, fp32: forward 7 + 28 us, gradients 7 + 38 + 22 us (734 us as one kernel).
constexpr int kDsSt = kDsChunk + 1;
// What the kernels need of a chunk: rows of Q and K, and what is formed of them
// once for all (a kernel over all chunks; `record`, in memory between the kernels):
// sums of decays, k.k, N, P, T, e^G, w, beta. The walk needs P and what is behind it.
template <int D>
struct DsChunk {
  static constexpr int C = kDsChunk, ST = D + 4;
  static constexpr int kRecord = 2 * C + 4 * C * kDsSt + 3 * C, kWalkFrom = 2 * C + 2 * C * kDsSt;
  static constexpr size_t kFloats = kRecord + 2 * C * ST;
  static_assert(kRecord % 4 == 0 && kWalkFrom % 4 == 0, "records move in 16-byte pieces");
  float *record, *sQ, *sK, *KK, *P, *N, *T, *eg, *w, *be;
  double* Gd;
  __device__ __forceinline__ float* carve(float* m) {
    record = m;
    Gd = reinterpret_cast<double*>(m);
    KK = m + 2 * C;
    N = KK + C * kDsSt;
    P = N + C * kDsSt;
    T = P + C * kDsSt;
    eg = T + C * kDsSt;
    w = eg + C;
    be = w + C;
    sQ = be + C;
    sK = sQ + C * ST;
    return sK + C * ST;
  }
  // 528 of these a chunk: the fast exponential, off by 2^-22 and 2^-23 |x| of a value that
  // is below 2^-20 where |x| passes 14 (results stay at 1e-7 to 3e-7 by norm).
  __device__ __forceinline__ float e(int i, int j) const { return __expf((float)(Gd[i] - Gd[j])); }

  template <typename X>
  __device__ __forceinline__ void form(const DeltaArgs<X>& a, int64_t row0, int n, int h, int hk, int tid) {
    load_rows_f32<X, D, C, ST, kDsThreads>(sQ, a.q, row0, hk, n, tid);
    load_rows_f32<X, D, C, ST, kDsThreads>(sK, a.k, row0, hk, n, tid);
    if (tid < 32) {  // sums of the log decays, in 64 bits
      double x = tid < n ? (double)delta_log(to_f32(*a.g.at(row0 + tid, h))) : 0.0;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, s);
        if (tid >= s) x += y;
      }
      Gd[tid] = x;
      const double last = __shfl_sync(0xffffffffu, x, 31);
      eg[tid] = expf((float)x);
      w[tid] = expf((float)(last - x));
      be[tid] = tid < n ? to_f32(*a.beta.at(row0 + tid, h)) : 0.f;
    }
    __syncthreads();
    {  // 2 x 2 elements of k.k and q.k a thread
      const int i = tid / 16 * 2, j = tid % 16 * 2;
      float kk[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, qk[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 ki[2], kj[2], qi[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          ki[y] = *reinterpret_cast<const float4*>(sK + (i + y) * ST + c);
          kj[y] = *reinterpret_cast<const float4*>(sK + (j + y) * ST + c);
          qi[y] = *reinterpret_cast<const float4*>(sQ + (i + y) * ST + c);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            kk[y][z] = fmaf(ki[y].x, kj[z].x, fmaf(ki[y].y, kj[z].y, fmaf(ki[y].z, kj[z].z, fmaf(ki[y].w, kj[z].w, kk[y][z]))));
            qk[y][z] = fmaf(qi[y].x, kj[z].x, fmaf(qi[y].y, kj[z].y, fmaf(qi[y].z, kj[z].z, fmaf(qi[y].w, kj[z].w, qk[y][z]))));
          }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int ii = i + y, jj = j + z;
          const float d = jj <= ii ? e(ii, jj) : 0.f;
          KK[ii * kDsSt + jj] = kk[y][z];
          P[ii * kDsSt + jj] = a.scale * d * qk[y][z];
          N[ii * kDsSt + jj] = jj < ii ? be[ii] * d * kk[y][z] : 0.f;
        }
    }
    __syncthreads();
    if (tid < C) {  // T, one column each, by forward substitution in registers
      float x[C];
#pragma unroll
      for (int i = 0; i < C; ++i) {
        float s0 = i == tid ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) {
          if (j & 1)
            s1 = fmaf(-N[i * kDsSt + j], x[j], s1);
          else
            s0 = fmaf(-N[i * kDsSt + j], x[j], s0);
        }
        x[i] = i < tid ? 0.f : s0 + s1;
        T[i * kDsSt + tid] = x[i];
      }
    }
    __syncthreads();
  }
};

// Grid (slots, Hv); records [slot][Hv], none for sequences of at most `most` tokens.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_form_kernel(const DeltaArgs<T> a, int most,
                                                                     float* __restrict__ records) {
  extern __shared__ __align__(16) float ds_smem[];
  DsChunk<D> ch;
  ch.carve(ds_smem);
  SlotTile t;
  if (!chunk_tile<kDsChunk>(a.seq, blockIdx.x, &t) || t.r.len <= most || !tile_found<kDsChunk>(a.seq, t)) return;
  const int h = blockIdx.y, c0 = t.tile * kDsChunk;
  ch.form(a, t.r.first + c0, min(kDsChunk, t.r.len - c0), h, h / a.G, threadIdx.x);
  float4* to = reinterpret_cast<float4*>(records + ((int64_t)blockIdx.x * a.Hv + h) * DsChunk<D>::kRecord);
  for (int i = threadIdx.x; i < DsChunk<D>::kRecord / 4; i += kDsThreads)
    to[i] = reinterpret_cast<const float4*>(ch.record)[i];
}

// The part of a record that the walks need, on its way through registers.
template <int D>
struct DsRecordAhead {
  static constexpr int FROM = DsChunk<D>::kWalkFrom, ALL = (DsChunk<D>::kRecord - FROM) / 4;
  static constexpr int PER = (ALL + kDsThreads - 1) / kDsThreads;
  float4 r[PER];
  __device__ __forceinline__ void issue(const float* __restrict__ records, int64_t which, int tid) {
    const float4* from = reinterpret_cast<const float4*>(records + which * DsChunk<D>::kRecord + FROM);
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (tid + u * kDsThreads < ALL) r[u] = from[tid + u * kDsThreads];
  }
  __device__ __forceinline__ void store(const DsChunk<D>& ch, int tid) const {
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (tid + u * kDsThreads < ALL) reinterpret_cast<float4*>(ch.record + FROM)[tid + u * kDsThreads] = r[u];
  }
};
// Products [32, K] x [K, 32 columns] of a walk. Loads from shared memory bound
// them, so a thread keeps 4 x 4 elements (rows 4 warp .., columns 4 (lane / 4) ..)
// for every fourth k (from lane % 4 on), and the four lanes' shares are added at
// the end, where each keeps one row: 4 warp + lane % 4. (With one row a thread and
// all k: 37 and 47 us for the two walks below, 28 and 38 this way.)
__device__ __forceinline__ void ds_axpy(float4& y, float f, const float4& x) {
  y = make_float4(fmaf(f, x.x, y.x), fmaf(f, x.y, y.y), fmaf(f, x.z, y.z), fmaf(f, x.w, y.w));
}
template <int K, typename FA, typename FB>
__device__ __forceinline__ void ds_share(float4 (&acc)[4], int lane, FA fa, FB fb) {
#pragma unroll 4
  for (int k = lane & 3; k < K; k += 4) {
    const float4 b = fb(k);
#pragma unroll
    for (int i = 0; i < 4; ++i) ds_axpy(acc[i], fa(i, k), b);
  }
}
__device__ __forceinline__ void ds_zero(float4 (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}
// This lane's half of two values plus the other lane's share of it, element by
// element (a choice between whole vectors would be one between addresses).
__device__ __forceinline__ float ds_halve(bool up, float low, float high, int lanes) {
  return (up ? high : low) + __shfl_xor_sync(0xffffffffu, up ? low : high, lanes);
}
__device__ __forceinline__ float4 ds_halve(bool up, const float4& l, const float4& h, int lanes) {
  return make_float4(ds_halve(up, l.x, h.x, lanes), ds_halve(up, l.y, h.y, lanes), ds_halve(up, l.z, h.z, lanes),
                     ds_halve(up, l.w, h.w, lanes));
}
__device__ __forceinline__ float4 ds_close(const float4 (&acc)[4], int lane) {
  const float4 x0 = ds_halve(lane & 2, acc[0], acc[2], 2), x1 = ds_halve(lane & 2, acc[1], acc[3], 2);
  return ds_halve(lane & 1, x0, x1, 1);
}

constexpr int kDsVs = kDsCols + 8;  // stride of a row of 32 columns: four rows' pieces of 8 banks each
template <int D>
constexpr size_t ds_chain_smem() {
  return (DsChunk<D>::kFloats + D * kDsVs + 2 * kDsChunk * kDsVs + 8) * 4;
}

// dS from the last chunk to the first, 32 of its columns a CTA; keeps Z (fp32,
// [T][Hv][D]) and each chunk's dS+ ([slot][Hv][D][D]), writes dV.
template <typename T, int D>
__device__ __forceinline__ void ds_chain(const DeltaGradArgs<T>& a, const float* __restrict__ records,
                                         float* __restrict__ kept_dS, float* __restrict__ kept_Z, int strip) {
  constexpr int C = kDsChunk, V = kDsCols, VS = kDsVs;
  extern __shared__ __align__(16) float ds_smem[];
  DsChunk<D> ch;
  float* dS = ch.carve(ds_smem);  // [D][VS]
  dS += (4 - ((dS - ds_smem) & 3)) & 3;
  float* sO = dS + D * VS;   // dout
  float* sZ = sO + C * VS;
  const int tid = threadIdx.x, h = blockIdx.y, seq = blockIdx.z, hk = h / a.G, col0 = strip * V;
  const SlotRounds rounds(a.seq, seq);
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t base = ((int64_t)seq * a.Hv + h) * D * D + col0;
  for (int i = tid; i < D * V; i += kDsThreads)
    dS[(i / V) * VS + i % V] = a.dS_out ? a.dS_out[base + (int64_t)(i / V) * D + i % V] : 0.f;
  const int lane = tid & 31, r0 = tid / 32 * 4, ti = r0 + (lane & 3), tj = lane >> 2;
  DsAhead<T, C, D, DsChunk<D>::ST> rq, rk;
  DsAhead<T, C, V, VS> ro;
  DsRecordAhead<D> rec;
  auto issue = [&](int c) {
    const int64_t row0 = r.first + (int64_t)c * C, slot = (int64_t)(r.first / C) + seq + c;
    rq.issue(a.q, row0, hk, 0, r.len - c * C, tid);
    rk.issue(a.k, row0, hk, 0, r.len - c * C, tid);
    ro.issue(a.dout, row0, h, col0, r.len - c * C, tid);
    rec.issue(records, slot * a.Hv + h, tid);
  };
  int chunks = (r.len + C - 1) / C;
  if (chunks > 0) issue(chunks - 1);
  if (!chunks_found<C>(rounds, a.seq, r)) chunks = 0;
  for (int c = chunks - 1; c >= 0; --c) {
    const int n = min(C, r.len - c * C);
    const int64_t row0 = r.first + (int64_t)c * C, slot = (int64_t)(r.first / C) + seq + c;
    __syncthreads();
    rq.store(ch.sQ, tid);
    rk.store(ch.sK, tid);
    ro.store(sO, tid);
    rec.store(ch, tid);
    float* keep = kept_dS + (slot * a.Hv + h) * D * D + col0;
    for (int i = tid; i < D * V; i += kDsThreads) keep[(int64_t)(i / V) * D + i % V] = dS[(i / V) * VS + i % V];
    __syncthreads();
    if (c > 0) issue(c - 1);
    const float whole = ch.eg[C - 1];
    auto columns = [&](const float* x) {
      return [=](int k) { return *reinterpret_cast<const float4*>(x + k * VS + 4 * tj); };
    };
    // dU = P^T dO + diag(w) K dS+
    float4 acc[4];
    ds_zero(acc);
    ds_share<D>(acc, lane, [&](int i, int k) { return ch.sK[(r0 + i) * DsChunk<D>::ST + k]; }, columns(dS));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = ch.w[r0 + i];
      acc[i] = make_float4(f * acc[i].x, f * acc[i].y, f * acc[i].z, f * acc[i].w);
    }
    ds_share<C>(acc, lane, [&](int i, int k) { return ch.P[k * kDsSt + r0 + i]; }, columns(sO));
    *reinterpret_cast<float4*>(sZ + ti * VS + 4 * tj) = ds_close(acc, lane);
    __syncthreads();
    ds_zero(acc);  // Z = T^T dU
    ds_share<C>(acc, lane, [&](int i, int k) { return ch.T[k * kDsSt + r0 + i]; }, columns(sZ));
    const float4 z = ds_close(acc, lane);
    __syncthreads();
    const float bi = ch.be[ti], es = ch.eg[ti] * bi;
    if (ti < n) {
      *reinterpret_cast<float4*>(kept_Z + ((row0 + ti) * a.Hv + h) * D + col0 + 4 * tj) = z;
      store4(a.dv.at(row0 + ti, h) + col0 + 4 * tj, bi * z.x, bi * z.y, bi * z.z, bi * z.w);
    }
    // Rows of the two products into dS, scaled: scale e^G dO and e^G beta Z.
    *reinterpret_cast<float4*>(sZ + ti * VS + 4 * tj) = make_float4(es * z.x, es * z.y, es * z.z, es * z.w);
    {
      const float f = a.scale * ch.eg[ti];
      float4 o = *reinterpret_cast<float4*>(sO + ti * VS + 4 * tj);
      *reinterpret_cast<float4*>(sO + ti * VS + 4 * tj) = make_float4(f * o.x, f * o.y, f * o.z, f * o.w);
    }
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < D / 32; ++rr) {
      const float* q = ch.sQ + 32 * rr + r0;
      const float* kk = ch.sK + 32 * rr + r0;
      ds_zero(acc);
      ds_share<C>(acc, lane, [&](int i, int t) { return q[t * DsChunk<D>::ST + i]; }, columns(sO));
      ds_share<C>(acc, lane, [&](int i, int t) { return -kk[t * DsChunk<D>::ST + i]; }, columns(sZ));
      float4 d = ds_close(acc, lane);
      float4* at = reinterpret_cast<float4*>(dS + (32 * rr + ti) * VS + 4 * tj);
      ds_axpy(d, whole, *at);
      *at = d;
    }
  }
  __syncthreads();
  if (a.dS_in)
    for (int i = tid; i < D * V; i += kDsThreads) a.dS_in[base + (int64_t)(i / V) * D + i % V] = dS[(i / V) * VS + i % V];
}

// S from the first chunk to the last, 32 of its columns a CTA.
// KEEP: for the gradients, S at each chunk's start ([slot][Hv][D][D]) in place of O.
template <typename T, int D, bool KEEP>
__device__ __forceinline__ void ds_walk(const DeltaArgs<T>& a, const float* __restrict__ records,
                                        float* __restrict__ kept, int strip) {
  constexpr int C = kDsChunk, V = kDsCols, VS = kDsVs, ST = DsChunk<D>::ST;
  extern __shared__ __align__(16) float ds_smem[];
  DsChunk<D> ch;
  float* S = ch.carve(ds_smem);  // [D][VS]
  float* sV = S + D * VS;        // V, then diag(w) U
  float* sU = sV + C * VS;       // diag(beta) R, then U
  const int tid = threadIdx.x, h = blockIdx.y, seq = blockIdx.z, hk = h / a.G, col0 = strip * V;
  const SlotRounds rounds(a.seq, seq);
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t base = ((int64_t)seq * a.Hv + h) * D * D + col0;
  for (int i = tid; i < D * V; i += kDsThreads)
    S[(i / V) * VS + i % V] = a.S_in ? a.S_in[base + (int64_t)(i / V) * D + i % V] : 0.f;
  const int lane = tid & 31, r0 = tid / 32 * 4, ti = r0 + (lane & 3), tj = lane >> 2;
  DsAhead<T, C, D, ST> rq, rk;
  DsAhead<T, C, V, VS> rv;
  DsRecordAhead<D> rec;
  auto issue = [&](int c) {
    const int64_t row0 = r.first + (int64_t)c * C, slot = (int64_t)(r.first / C) + seq + c;
    if (!KEEP) rq.issue(a.q, row0, hk, 0, r.len - c * C, tid);
    rk.issue(a.k, row0, hk, 0, r.len - c * C, tid);
    rv.issue(a.v, row0, h, col0, r.len - c * C, tid);
    rec.issue(records, slot * a.Hv + h, tid);
  };
  int chunks = (r.len + C - 1) / C;
  if (chunks > 0) issue(0);
  if (!chunks_found<C>(rounds, a.seq, r)) chunks = 0;
  for (int c = 0; c < chunks; ++c) {
    __syncthreads();
    if (!KEEP) rq.store(ch.sQ, tid);
    rk.store(ch.sK, tid);
    rv.store(sV, tid);
    rec.store(ch, tid);
    if (KEEP) {
      const int64_t slot = (int64_t)(r.first / C) + seq + c;
      float* keep = kept + (slot * a.Hv + h) * D * D + col0;
      for (int i = tid; i < D * V; i += kDsThreads) keep[(int64_t)(i / V) * D + i % V] = S[(i / V) * VS + i % V];
    }
    __syncthreads();
    if (c + 1 < chunks) issue(c + 1);
    const float eg = ch.eg[ti], be = ch.be[ti], wi = ch.w[ti], whole = ch.eg[C - 1];
    auto columns = [&](const float* x) {
      return [=](int k) { return *reinterpret_cast<const float4*>(x + k * VS + 4 * tj); };
    };
    float4 acc[4], o[4];
    ds_zero(acc);
    ds_share<D>(acc, lane, [&](int i, int k) { return ch.sK[(r0 + i) * ST + k]; }, columns(S));
    const float4 x = ds_close(acc, lane), v = *reinterpret_cast<const float4*>(sV + ti * VS + 4 * tj);
    *reinterpret_cast<float4*>(sU + ti * VS + 4 * tj) =
        make_float4(be * (v.x - eg * x.x), be * (v.y - eg * x.y), be * (v.z - eg * x.z), be * (v.w - eg * x.w));
    if (!KEEP) {
      ds_zero(o);
      ds_share<D>(o, lane, [&](int i, int k) { return ch.sQ[(r0 + i) * ST + k]; }, columns(S));
    }
    __syncthreads();
    ds_zero(acc);
    ds_share<C>(acc, lane, [&](int i, int k) { return ch.T[(r0 + i) * kDsSt + k]; }, columns(sU));
    const float4 u = ds_close(acc, lane);
    *reinterpret_cast<float4*>(sV + ti * VS + 4 * tj) = make_float4(wi * u.x, wi * u.y, wi * u.z, wi * u.w);
    __syncthreads();
    if (!KEEP) *reinterpret_cast<float4*>(sU + ti * VS + 4 * tj) = u;
#pragma unroll
    for (int rr = 0; rr < D / 32; ++rr) {
      const float* kk = ch.sK + 32 * rr + r0;
      ds_zero(acc);
      ds_share<C>(acc, lane, [&](int i, int t) { return kk[t * ST + i]; }, columns(sV));
      float4 d = ds_close(acc, lane);
      float4* at = reinterpret_cast<float4*>(S + (32 * rr + ti) * VS + 4 * tj);
      ds_axpy(d, whole, *at);
      *at = d;
    }
    if (!KEEP) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = a.scale * ch.eg[r0 + i];
        o[i] = make_float4(f * o[i].x, f * o[i].y, f * o[i].z, f * o[i].w);
      }
      ds_share<C>(o, lane, [&](int i, int k) { return ch.P[(r0 + i) * kDsSt + k]; }, columns(sU));
      const float4 y = ds_close(o, lane);
      const int t = c * C + ti;
      if (t < r.len) store4(a.out.at(r.first + t, h) + col0 + 4 * tj, y.x, y.y, y.z, y.w);
    }
  }
  __syncthreads();
  if (a.S_out)
    for (int i = tid; i < D * V; i += kDsThreads) a.S_out[base + (int64_t)(i / V) * D + i % V] = S[(i / V) * VS + i % V];
}

// A forward pass: each sequence by its length.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_walk_kernel(const DeltaArgs<T> a,
                                                                     const float* __restrict__ records) {
  if (seq_range(a.seq, blockIdx.z).len <= kDsRecurMost)
    ds_recur<T, D>(a, blockIdx.x);
  else
    ds_walk<T, D, false>(a, records, nullptr, blockIdx.x);
}

// The two walks of a backward pass side by side: S again, and dS. Neither needs
// the other, and one launch after the other would add their chains.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_walks_kernel(const DeltaArgs<T> f, const DeltaGradArgs<T> a,
                                                                      const float* __restrict__ records,
                                                                      float* __restrict__ kept,
                                                                      float* __restrict__ kept_dS,
                                                                      float* __restrict__ kept_Z) {
  const int strip = blockIdx.x % (D / kDsCols);
  if (blockIdx.x < D / kDsCols)
    ds_chain<T, D>(a, records, kept_dS, kept_Z, strip);
  else
    ds_walk<T, D, true>(f, records, kept, strip);
}

template <int D>
constexpr size_t ds_grad_smem() {
  return (DsChunk<D>::kFloats + 3 * kDsChunk * (D + 4) + kDsChunk * (D + 1) + D * (D + 1) + 2 * kDsChunk * kDsSt +
          2 * kDsChunk + 16) * 4;
}

// Everything else, CTA = (chunk, value head): the walks' products over 32 columns
// at a time, S and then dS+ in shared memory with rows of D + 1 (read along and
// across). dq and dk leave per value head (fp32, [T][Hv][D]); a further kernel
// adds the group.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_grad_kernel(const DeltaGradArgs<T> a,
                                                                     const float* __restrict__ records,
                                                                     const float* __restrict__ kept,
                                                                     const float* __restrict__ kept_dS,
                                                                     const float* __restrict__ kept_Z,
                                                                     float* __restrict__ dq_part,
                                                                     float* __restrict__ dk_part) {
  constexpr int C = kDsChunk, ST = D + 4, CS = kDsSt, SS = D + 1, NS = D / 32;
  extern __shared__ __align__(16) float ds_smem[];
  DsChunk<D> ch;
  float* sO = ch.carve(ds_smem);  // dout
  float* sR = sO + C * ST;        // V, then R
  float* sZ = sR + C * ST;
  float* sU = sZ + C * ST;        // [C][SS]
  float* sS = sU + C * SS;        // [D][SS]
  float* H = sS + D * SS;         // then F
  float* M = H + C * CS;          // then X = scale e M
  float* dG = M + C * CS;
  float* xs = dG + C;
  float* red = xs + C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, hk = h / a.G;
  const int r0 = 4 * warp, ti = r0 + (lane & 3), tj = lane >> 2;
  SlotTile t;
  if (!chunk_tile<C>(a.seq, blockIdx.x, &t) || !tile_found<C>(a.seq, t)) return;
  const int n = min(C, t.r.len - t.tile * C);
  const int64_t row0 = t.r.first + (int64_t)t.tile * C;
  const int64_t at = (((int64_t)(t.r.first / C) + t.seq + t.tile) * a.Hv + h) * D * D;
  const float* S = kept + at;
  const float* dS = kept_dS + at;
  load_rows_f32<T, D, C, ST, kDsThreads>(sR, a.v, row0, h, n, tid);
  load_rows_f32<T, D, C, ST, kDsThreads>(sO, a.dout, row0, h, n, tid);
  load_rows_f32<float, D, C, ST, kDsThreads>(sZ, RowsOf<const float>{kept_Z, (int64_t)a.Hv * D, D}, row0, h, n, tid);
  load_rows_f32<T, D, C, ST, kDsThreads>(ch.sQ, a.q, row0, hk, n, tid);
  load_rows_f32<T, D, C, ST, kDsThreads>(ch.sK, a.k, row0, hk, n, tid);
  const float4* rec = reinterpret_cast<const float4*>(records + ((int64_t)blockIdx.x * a.Hv + h) * DsChunk<D>::kRecord);
  for (int i = tid; i < DsChunk<D>::kRecord / 4; i += kDsThreads) reinterpret_cast<float4*>(ch.record)[i] = rec[i];
  auto put_state = [&](int i, const float4& x) {  // elements 4 i .. of a state
    float* to = sS + i / (D / 4) * SS + i % (D / 4) * 4;
    to[0] = x.x;
    to[1] = x.y;
    to[2] = x.z;
    to[3] = x.w;
  };
  for (int i = tid; i < D * D / 4; i += kDsThreads) put_state(i, reinterpret_cast<const float4*>(S)[i]);
  __syncthreads();
  const float* eg = ch.eg;
  const float* w = ch.w;
  const float* be = ch.be;
  const float whole = eg[C - 1];
  float4 acc[4];
  auto rows4 = [&](const float* x, int stride, int c) {  // four columns from c on of row k
    return [=](int k) {
      const float* y = x + k * stride + c + 4 * tj;
      return make_float4(y[0], y[1], y[2], y[3]);
    };
  };
  auto turned = [&](const float* x, int stride, int c) {  // element k of four rows from c on
    return [=](int k) {
      const float* y = x + (c + 4 * tj) * stride + k;
      return make_float4(y[0], y[stride], y[2 * stride], y[3 * stride]);
    };
  };
  auto left = [&](const float* x, int stride) { return [=](int i, int k) { return x[(r0 + i) * stride + k]; }; };
  auto left_turned = [&](const float* x, int stride) { return [=](int i, int k) { return x[k * stride + r0 + i]; }; };
#pragma unroll
  for (int c = 0; c < D; c += 32) {  // R
    ds_zero(acc);
    ds_share<D>(acc, lane, left(ch.sK, ST), rows4(sS, SS, c));
    float4 y = ds_close(acc, lane);
    float4* to = reinterpret_cast<float4*>(sR + ti * ST + c + 4 * tj);
    float4 x = *to;
    ds_axpy(x, -eg[ti], y);
    *to = x;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < D; c += 32) {  // U
    ds_zero(acc);
    ds_share<C>(acc, lane, [&](int i, int k) { return ch.T[(r0 + i) * CS + k] * be[k]; }, rows4(sR, ST, c));
    const float4 y = ds_close(acc, lane);
    float* to = sU + ti * SS + c + 4 * tj;
    to[0] = y.x;
    to[1] = y.y;
    to[2] = y.z;
    to[3] = y.w;
  }
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {  // H = Z U^T, M = dO U^T
    ds_zero(acc);
    ds_share<D>(acc, lane, left(which ? sO : sZ, ST), turned(sU, SS, 0));
    const float4 y = ds_close(acc, lane);
    float* to = (which ? M : H) + ti * CS + 4 * tj;
    to[0] = y.x;
    to[1] = y.y;
    to[2] = y.z;
    to[3] = y.w;
  }
  __syncthreads();
  // dbeta; each row's sums over Q's first columns (into T); F and X: one warp per token.
  for (int i = warp; i < C; i += kDsThreads / 32) {
    float x = 0.f;
    for (int k = lane; k < D; k += 32) x = fmaf(sZ[i * ST + k], sR[i * ST + k], x);
    const int j = lane;
    const float d = j <= i ? ch.e(i, j) : 0.f, hij = H[i * CS + j], m = M[i * CS + j];
    const float low = j < i ? hij * d * ch.KK[i * CS + j] : 0.f;
    x = warp_sum(x - low);
    float y = j < i ? ch.P[i * CS + j] * m - be[i] * low : 0.f;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const float z = __shfl_up_sync(0xffffffffu, y, s);
      if (lane >= s) y += z;
    }
    ch.T[i * CS + j + 1] = y;
    M[i * CS + j] = a.scale * d * m;
    H[i * CS + j] = j < i ? be[i] * d * hij : 0.f;
    if (lane == 0) {
      ch.T[i * CS] = 0.f;
      if (i < n) *a.dbeta.at(row0 + i, h) = from_f32<T>(x);
    }
  }
  __syncthreads();
  // One 32-column part of a term: rows scaled by f, dotted with their own rows of x.
  float sdot = 0.f, xdot = 0.f;
  auto term = [&](const float* l, int ls, int c, float f, const float* x, float& dot) {
    ds_zero(acc);
    ds_share<D>(acc, lane, left(l, ls), turned(sS, SS, c));
    float4 y = ds_close(acc, lane);
    y = make_float4(f * y.x, f * y.y, f * y.z, f * y.w);
    const float4 o = *reinterpret_cast<const float4*>(x + ti * ST + c + 4 * tj);
    dot = fmaf(y.x, o.x, fmaf(y.y, o.y, fmaf(y.z, o.z, fmaf(y.w, o.w, dot))));
    return y;
  };
  float4 dk[NS];
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    float4 y = term(sO, ST, c, a.scale * eg[ti], ch.sQ, sdot);
    ds_zero(acc);
    ds_share<C>(acc, lane, left(M, CS), rows4(ch.sK, ST, c));
    ds_axpy(y, 1.f, ds_close(acc, lane));
    if (ti < n) *reinterpret_cast<float4*>(dq_part + ((row0 + ti) * a.Hv + h) * D + c + 4 * tj) = y;
    dk[c / 32] = term(sZ, ST, c, -eg[ti] * be[ti], ch.sK, sdot);
  }
  __syncthreads();
  float both = 0.f;  // <dS+, S>
  for (int i = tid; i < D * D / 4; i += kDsThreads) {
    const float4 x = reinterpret_cast<const float4*>(S)[i], y = reinterpret_cast<const float4*>(dS)[i];
    both = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, both))));
    put_state(i, y);
  }
  both = warp_sum(both);
  if (lane == 0) red[warp] = both;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    ds_axpy(dk[c / 32], 1.f, term(sU, SS, c, w[ti], ch.sK, xdot));
    ds_zero(acc);
    ds_share<C>(acc, lane, left_turned(M, CS), rows4(ch.sQ, ST, c));
    ds_share<C>(acc, lane, [&](int i, int k) { return -(H[(r0 + i) * CS + k] + H[k * CS + r0 + i]); }, rows4(ch.sK, ST, c));
    ds_axpy(dk[c / 32], 1.f, ds_close(acc, lane));
    if (ti < n) *reinterpret_cast<float4*>(dk_part + ((row0 + ti) * a.Hv + h) * D + c + 4 * tj) = dk[c / 32];
  }
#pragma unroll
  for (int s = 4; s < 32; s <<= 1) {
    sdot += __shfl_xor_sync(0xffffffffu, sdot, s);
    xdot += __shfl_xor_sync(0xffffffffu, xdot, s);
  }
  if (tj == 0) {
    dG[ti] = sdot;
    xs[ti] = xdot;
  }
  __syncthreads();
  if (tid < 32) {
    float d = dG[tid], y = tid ? xs[tid - 1] : 0.f;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {  // from the end, and from the start
      const float d2 = __shfl_down_sync(0xffffffffu, d, s), y2 = __shfl_up_sync(0xffffffffu, y, s);
      if (tid + s < 32) d += d2;
      if (tid >= s) y += y2;
    }
    d += y + warp_sum(tid < kDsThreads / 32 ? whole * red[tid] : 0.f);
    for (int i = tid; i < C; ++i) d += ch.T[i * CS + tid];
    if (tid < n) *a.dg.at(row0 + tid, h) = from_f32<T>(d);
  }
}

// dq, dk of a key head: the sum over its value heads, in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_group_sum_kernel(const DeltaGradArgs<T> a,
                                                              const float* __restrict__ dq_part,
                                                              const float* __restrict__ dk_part) {
  SlotTile t;
  if (!chunk_tile<kDsChunk>(a.seq, blockIdx.x, &t) || !tile_found<kDsChunk>(a.seq, t)) return;
  const int r0 = t.tile * kDsChunk, n = min(kDsChunk, t.r.len - r0), hk = blockIdx.y;
  for (int i = threadIdx.x; i < n * (D / 4); i += 256) {
    const int64_t row = t.r.first + r0 + i / (D / 4);
    const int c = (i % (D / 4)) * 4;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float* src = (which ? dk_part : dq_part) + (row * a.Hv + (int64_t)hk * a.G) * D + c;
      float4 s = *reinterpret_cast<const float4*>(src);
      for (int g = 1; g < a.G; ++g) {
        const float4 y = *reinterpret_cast<const float4*>(src + (int64_t)g * D);
        s.x += y.x;
        s.y += y.y;
        s.z += y.z;
        s.w += y.w;
      }
      store4((which ? a.dk : a.dq).at(row, hk) + c, s.x, s.y, s.z, s.w);
    }
  }
}

// One token: S is read once into registers (16-byte loads, all in flight at
// once) and written once; reading and writing it bounds the step. Warps take
// rows of S, so both products over d_k close through shared memory. Measured: 64
// tokens, 16 / 32 heads, d = 128: 47 us, 5.7 TB/s (0.88 of a plain copy).
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_step_kernel(const DeltaArgs<T> a) {
  constexpr int LPR = D / 4, RPP = 256 / LPR, N = D / RPP;  // lanes of a row, rows a pass, passes
  __shared__ float sq[D], sk[D];
  __shared__ __align__(16) float part[RPP][D];
  const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y, hk = h / a.G, rr = tid / LPR, c = (tid % LPR) * 4;
  const int64_t base = ((int64_t)b * a.Hv + h) * D * D;
  float4 S[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    S[i] = *reinterpret_cast<const float4*>(a.S_in + base + (int64_t)(rr + i * RPP) * D + c);
  if (tid < D) {
    sq[tid] = to_f32(a.q.at(b, hk)[tid]) * a.scale;
    sk[tid] = to_f32(a.k.at(b, hk)[tid]);
  }
  const float decay = expf(delta_log(to_f32(*a.g.at(b, h)))), beta = to_f32(*a.beta.at(b, h));
  const T* vp = a.v.at(b, h) + c;
  const float v[4] = {to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3])};
  __syncthreads();
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = sk[rr + i * RPP];
    S[i].x *= decay;
    S[i].y *= decay;
    S[i].z *= decay;
    S[i].w *= decay;
    x.x = fmaf(S[i].x, k, x.x);
    x.y = fmaf(S[i].y, k, x.y);
    x.z = fmaf(S[i].z, k, x.z);
    x.w = fmaf(S[i].w, k, x.w);
  }
  *reinterpret_cast<float4*>(&part[rr][c]) = x;
  __syncthreads();
  x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPP; ++i) {
    const float4 y = *reinterpret_cast<const float4*>(&part[i][c]);
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  const float4 u = make_float4(beta * (v[0] - x.x), beta * (v[1] - x.y), beta * (v[2] - x.z), beta * (v[3] - x.w));
  x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = sk[rr + i * RPP], q = sq[rr + i * RPP];
    S[i].x = fmaf(k, u.x, S[i].x);
    S[i].y = fmaf(k, u.y, S[i].y);
    S[i].z = fmaf(k, u.z, S[i].z);
    S[i].w = fmaf(k, u.w, S[i].w);
    x.x = fmaf(S[i].x, q, x.x);
    x.y = fmaf(S[i].y, q, x.y);
    x.z = fmaf(S[i].z, q, x.z);
    x.w = fmaf(S[i].w, q, x.w);
    *reinterpret_cast<float4*>(a.S_out + base + (int64_t)(rr + i * RPP) * D + c) = S[i];
  }
  __syncthreads();
  *reinterpret_cast<float4*>(&part[rr][c]) = x;
  __syncthreads();
  if (rr == 0) {
#pragma unroll
    for (int i = 1; i < RPP; ++i) {
      const float4 y = *reinterpret_cast<const float4*>(&part[i][c]);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    store4(a.out.at(b, h) + c, x.x, x.y, x.z, x.w);
  }
}

}  // namespace infini

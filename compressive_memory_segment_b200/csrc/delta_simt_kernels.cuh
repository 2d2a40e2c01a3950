// The gated delta rule on the CUDA cores, fp32 arithmetic throughout: the
// recurrence token by token (forward), the chunked gradient, and the one-token
// step. fp32 inputs run here.
#pragma once

#include "delta_common.cuh"
#include "packed_simt_kernels.cuh"

namespace infini {

constexpr int kDsThreads = 256;
constexpr int kDsCols = 32;    // columns of S (values) of one forward CTA
constexpr int kDsBlock = 16;   // tokens staged at a time
constexpr int kDsChunk = 32;   // tokens of a gradient chunk; the forward keeps S at each start

// Columns of S are independent, so a CTA walks the tokens with 32 of them. 8
// lanes share a column (D / 8 rows each, in registers); the two dot products
// over d_k close with three shuffles each. The chain of those bounds it.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_fwd_kernel(const DeltaArgs<T> a, float* __restrict__ kept) {
  constexpr int PER = D / 8;
  __shared__ __align__(16) float sQ[kDsBlock][D], sK[kDsBlock][D];
  __shared__ float sV[kDsBlock][kDsCols], sG[kDsBlock], sB[kDsBlock];
  const int tid = threadIdx.x, part = tid & 7, c = tid >> 3, col = blockIdx.x * kDsCols + c;
  const int h = blockIdx.y, seq = blockIdx.z, hk = h / a.G;
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t base = ((int64_t)seq * a.Hv + h) * D * D;
  float S[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = (i >> 2) * 32 + part * 4 + (i & 3);
    S[i] = a.S_in ? a.S_in[base + (int64_t)row * D + col] : 0.f;
  }
  for (int t0 = 0; t0 < r.len; t0 += kDsBlock) {
    __syncthreads();
    const int n = min(kDsBlock, r.len - t0);
    load_rows_f32<T, D, kDsBlock, D, kDsThreads>(&sQ[0][0], a.q, r.first + t0, hk, n, tid);
    load_rows_f32<T, D, kDsBlock, D, kDsThreads>(&sK[0][0], a.k, r.first + t0, hk, n, tid);
    for (int i = tid; i < kDsBlock * kDsCols; i += kDsThreads) {
      const int t = i / kDsCols, x = i % kDsCols;
      sV[t][x] = t < n ? to_f32(a.v.at(r.first + t0 + t, h)[blockIdx.x * kDsCols + x]) : 0.f;
    }
    if (tid < n) {
      sG[tid] = expf(delta_log(to_f32(*a.g.at(r.first + t0 + tid, h))));
      sB[tid] = to_f32(*a.beta.at(r.first + t0 + tid, h));
    }
    __syncthreads();
    if (kept && t0 % kDsChunk == 0) {
      const int64_t slot = (int64_t)(r.first / kDsChunk) + seq + t0 / kDsChunk;
      float* dst = kept + (slot * a.Hv + h) * D * D;
#pragma unroll
      for (int i = 0; i < PER; ++i) dst[(int64_t)((i >> 2) * 32 + part * 4 + (i & 3)) * D + col] = S[i];
    }
    for (int t = 0; t < n; ++t) {
      float x = 0.f, y = 0.f;
      float k[PER];
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&sK[t][(i >> 2) * 32 + part * 4]);
        k[i] = w.x;
        k[i + 1] = w.y;
        k[i + 2] = w.z;
        k[i + 3] = w.w;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        S[i] *= sG[t];
        x = fmaf(S[i], k[i], x);
      }
#pragma unroll
      for (int s = 4; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
      const float u = sB[t] * (sV[t][c] - x);
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&sQ[t][(i >> 2) * 32 + part * 4]);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i + e] = fmaf(k[i + e], u, S[i + e]);
        y = fmaf(S[i], w.x, fmaf(S[i + 1], w.y, fmaf(S[i + 2], w.z, fmaf(S[i + 3], w.w, y))));
      }
#pragma unroll
      for (int s = 4; s > 0; s >>= 1) y += __shfl_xor_sync(0xffffffffu, y, s);
      if (part == 0 && a.out.p) a.out.at(r.first + t0 + t, h)[col] = from_f32<T>(a.scale * y);
    }
  }
  if (a.S_out) {
#pragma unroll
    for (int i = 0; i < PER; ++i) a.S_out[base + (int64_t)((i >> 2) * 32 + part * 4 + (i & 3)) * D + col] = S[i];
  }
}

// acc[4][4] = the 4 x 4 block (rows 4 ti, columns 4 tj) of sum_k fa(i, k) fb(k, j).
template <int K, typename FA, typename FB>
__device__ __forceinline__ void ds_mm(int ti, int tj, FA fa, FB fb, float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int k = 0; k < K; ++k) {
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fa(4 * ti + i, k);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fb(k, 4 * tj + j);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}

template <int D>
constexpr size_t ds_bwd_smem() {
  return (size_t)(D * (D + 4) + 6 * kDsChunk * (D + 4) + 5 * kDsChunk * (kDsChunk + 1) + 6 * kDsChunk + 8) * 4 +
         kDsChunk * 8;
}

// The gradient chunk by chunk from the last to the first, one CTA per
// (sequence, value head), dS in shared memory. With G_i the sum of the chunk's
// log decays up to i, e_ij = exp(G_i - G_j), w_i = exp(G_C - G_i), S and dS+
// the state at the chunk's start and its end's gradient:
//   A_ij = beta_i e_ij k_i.k_j (j < i), T = (I + A)^-1, R = V - diag(e^G) K S,
//   U = T diag(beta) R, P_ij = scale e_ij q_i.k_j (j <= i)
//   dU = P^T dO + diag(w) K dS+,  Z = T^T dU,  dV = diag(beta) Z
//   dS = e^G_C dS+ + scale Q^T diag(e^G) dO - K^T diag(e^G beta) Z
//   M = dO U^T (j <= i), H = Z U^T (j < i), F_ij = beta_i H_ij e_ij
//   dq_i = scale (e^G_i S dO_i + sum_j e_ij M_ij k_j)
//   dk_j = scale sum_i e_ij M_ij q_i - e^G_j beta_j S Z_j + w_j dS+ u_j - sum_i (F_ij + F_ji) k_i
//   dbeta_i = Z_i.R_i - sum_j H_ij e_ij k_i.k_j
//   dg_t = sum_{i >= t} s_i + sum_{i >= t > j} N_ij + sum_{j < t} x_j + e^G_C <dS+, S>,
//     s_i = q_i.(scale e^G_i S dO_i) - k_i.(e^G_i beta_i S Z_i), x_j = w_j k_j.(dS+ u_j),
//     N_ij = P_ij M_ij - F_ij k_i.k_j: what passes over the decay of token t, and no more, so
//     that nothing has to cancel.
// dq and dk leave per value head (fp32, [T][Hv][D]); a second kernel adds the group.
template <typename T, int D>
__global__ void __launch_bounds__(kDsThreads) delta_simt_bwd_kernel(const DeltaGradArgs<T> a,
                                                                    const float* __restrict__ kept,
                                                                    float* __restrict__ dq_part,
                                                                    float* __restrict__ dk_part) {
  constexpr int C = kDsChunk, ST = D + 4, CS = C + 1, TJ = D / 4;
  static_assert(C * D / 16 <= kDsThreads, "one 4 x 4 block of a [C, D] product per thread");
  extern __shared__ __align__(16) float ds_smem[];
  float* dS = ds_smem;            // [D][ST]
  float* sQ = dS + D * ST;
  float* sK = sQ + C * ST;
  float* sO = sK + C * ST;        // dout
  float* sR = sO + C * ST;        // V, then R, then scratch
  float* sU = sR + C * ST;
  float* sZ = sU + C * ST;
  float* KK = sZ + C * ST;        // k_i.k_j
  float* QK = KK + C * CS;
  float* Ti = QK + C * CS;        // T
  float* H = Ti + C * CS;
  float* M = H + C * CS;
  float* eg = M + C * CS;         // e^G
  float* w = eg + C;
  float* be = w + C;
  float* dG = be + C;
  float* xs = dG + C;
  float* red = xs + C;            // [C + 8]
  double* Gd = reinterpret_cast<double*>(red + C + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.x, seq = blockIdx.y, hk = h / a.G;
  const SeqRange r = seq_range(a.seq, seq);
  const int64_t base = ((int64_t)seq * a.Hv + h) * D * D;
  for (int i = tid; i < D * D; i += kDsThreads) dS[(i / D) * ST + i % D] = a.dS_out ? a.dS_out[base + i] : 0.f;
  const int ti = tid / TJ, tj = tid % TJ;    // 4 x 4 block of a [C, D] product
  const bool mine = ti < C / 4;
  const int si = tid / (C / 4), sj = tid % (C / 4);  // of a [C, C] product
  const bool smine = si < C / 4;
  auto e = [&](int i, int j) { return __expf((float)(Gd[i] - Gd[j])); };
  float acc[4][4];

  for (int c = (r.len + C - 1) / C - 1; c >= 0; --c) {
    const int t0 = c * C, n = min(C, r.len - t0);
    const int64_t row0 = r.first + t0;
    const float* S = kept + (((int64_t)(r.first / C) + seq + c) * a.Hv + h) * D * D;
    __syncthreads();
    load_rows_f32<T, D, C, ST, kDsThreads>(sQ, a.q, row0, hk, n, tid);
    load_rows_f32<T, D, C, ST, kDsThreads>(sK, a.k, row0, hk, n, tid);
    load_rows_f32<T, D, C, ST, kDsThreads>(sR, a.v, row0, h, n, tid);
    load_rows_f32<T, D, C, ST, kDsThreads>(sO, a.dout, row0, h, n, tid);
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
      xs[tid] = 0.f;
    }
    __syncthreads();
    const float whole = eg[C - 1];
    if (smine) {
      ds_mm<D>(si, sj, [&](int i, int k) { return sK[i * ST + k]; }, [&](int k, int j) { return sK[j * ST + k]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) KK[(4 * si + i) * CS + 4 * sj + j] = acc[i][j];
      ds_mm<D>(si, sj, [&](int i, int k) { return sQ[i * ST + k]; }, [&](int k, int j) { return sK[j * ST + k]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) QK[(4 * si + i) * CS + 4 * sj + j] = acc[i][j];
    }
    if (mine) {  // R
      ds_mm<D>(ti, tj, [&](int i, int k) { return sK[i * ST + k]; }, [&](int k, int j) { return S[k * D + j]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sR[(4 * ti + i) * ST + 4 * tj + j] -= eg[4 * ti + i] * acc[i][j];
    }
    __syncthreads();
    if (tid < C) {  // T, one column each, by forward substitution
      for (int i = 0; i < C; ++i) {
        float x = i == tid ? 1.f : 0.f;
        for (int j = tid; j < i; ++j) x -= be[i] * e(i, j) * KK[i * CS + j] * Ti[j * CS + tid];
        Ti[i * CS + tid] = i < tid ? 0.f : x;
      }
    }
    __syncthreads();
    if (mine) {
      ds_mm<C>(ti, tj, [&](int i, int k) { return Ti[i * CS + k] * be[k]; },
               [&](int k, int j) { return sR[k * ST + j]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sU[(4 * ti + i) * ST + 4 * tj + j] = acc[i][j];
      // dU
      ds_mm<C>(ti, tj, [&](int i, int k) { return k >= i ? a.scale * e(k, i) * QK[k * CS + i] : 0.f; },
               [&](int k, int j) { return sO[k * ST + j]; }, acc);
      float more[4][4];
      ds_mm<D>(ti, tj, [&](int i, int k) { return sK[i * ST + k]; }, [&](int k, int j) { return dS[k * ST + j]; }, more);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sZ[(4 * ti + i) * ST + 4 * tj + j] = fmaf(w[4 * ti + i], more[i][j], acc[i][j]);
    }
    __syncthreads();
    if (mine)
      ds_mm<C>(ti, tj, [&](int i, int k) { return Ti[k * CS + i]; }, [&](int k, int j) { return sZ[k * ST + j]; }, acc);
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * ti + i;
#pragma unroll
        for (int j = 0; j < 4; ++j) sZ[t * ST + 4 * tj + j] = acc[i][j];
        if (t < n)
          store4(a.dv.at(row0 + t, h) + 4 * tj, be[t] * acc[i][0], be[t] * acc[i][1], be[t] * acc[i][2],
                 be[t] * acc[i][3]);
      }
    }
    __syncthreads();
    if (smine) {
      ds_mm<D>(si, sj, [&](int i, int k) { return sZ[i * ST + k]; }, [&](int k, int j) { return sU[j * ST + k]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) H[(4 * si + i) * CS + 4 * sj + j] = acc[i][j];
      ds_mm<D>(si, sj, [&](int i, int k) { return sO[i * ST + k]; }, [&](int k, int j) { return sU[j * ST + k]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) M[(4 * si + i) * CS + 4 * sj + j] = acc[i][j];
    }
    __syncthreads();
    // dbeta, and each row's sums over N's first columns (into Ti): one warp per token.
    for (int t = warp; t < C; t += kDsThreads / 32) {
      float x = 0.f;
      for (int k = lane; k < D; k += 32) x = fmaf(sZ[t * ST + k], sR[t * ST + k], x);
      const int j = lane;
      const float low = j < t ? H[t * CS + j] * e(t, j) * KK[t * CS + j] : 0.f;
      x = warp_sum(x - low);
      float y = j < t ? a.scale * e(t, j) * QK[t * CS + j] * M[t * CS + j] - be[t] * low : 0.f;  // N_tj
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float z = __shfl_up_sync(0xffffffffu, y, s);
        if (lane >= s) y += z;
      }
      Ti[t * CS + j + 1] = y;
      if (lane == 0) {
        Ti[t * CS] = dG[t] = 0.f;
        if (t < n) *a.dbeta.at(row0 + t, h) = from_f32<T>(x);
      }
    }
    __syncthreads();
    // sR becomes scratch for the terms whose dot with q or k enters dG.
    auto term = [&](auto fa, auto fb, auto fs) {  // sR[i] = fs(i) sum_j fa(i, j) fb(j, .)
      if (mine) {
        ds_mm<D>(ti, tj, fa, fb, acc);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sR[(4 * ti + i) * ST + 4 * tj + j] = fs(4 * ti + i) * acc[i][j];
      }
      __syncthreads();
    };
    auto dots = [&](const float* other, float* to) {  // to_i += other_i . sR_i
      for (int t = warp; t < C; t += kDsThreads / 32) {
        float x = 0.f;
        for (int k = lane; k < D; k += 32) x = fmaf(other[t * ST + k], sR[t * ST + k], x);
        x = warp_sum(x);
        if (lane == 0) to[t] += x;
      }
    };
    // dq
    term([&](int i, int k) { return sO[i * ST + k]; }, [&](int k, int j) { return S[j * D + k]; },
         [&](int i) { return a.scale * eg[i]; });
    dots(sQ, dG);
    if (mine) {
      ds_mm<C>(ti, tj, [&](int i, int k) { return k <= i ? e(i, k) * M[i * CS + k] : 0.f; },
               [&](int k, int j) { return sK[k * ST + j]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * ti + i;
        if (t >= n) continue;
        const float* x = sR + t * ST + 4 * tj;
        *reinterpret_cast<float4*>(dq_part + ((row0 + t) * a.Hv + h) * D + 4 * tj) =
            make_float4(fmaf(a.scale, acc[i][0], x[0]), fmaf(a.scale, acc[i][1], x[1]),
                        fmaf(a.scale, acc[i][2], x[2]), fmaf(a.scale, acc[i][3], x[3]));
      }
    }
    __syncthreads();
    // dk
    float dk[4][4];
    term([&](int i, int k) { return sZ[i * ST + k]; }, [&](int k, int j) { return S[j * D + k]; },
         [&](int i) { return -eg[i] * be[i]; });
    dots(sK, dG);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dk[i][j] = sR[(4 * ti + i) * ST + 4 * tj + j];
    }
    __syncthreads();
    term([&](int i, int k) { return sU[i * ST + k]; }, [&](int k, int j) { return dS[j * ST + k]; },
         [&](int i) { return w[i]; });
    dots(sK, xs);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dk[i][j] += sR[(4 * ti + i) * ST + 4 * tj + j];
      ds_mm<C>(ti, tj, [&](int i, int k) { return k >= i ? a.scale * e(k, i) * M[k * CS + i] : 0.f; },
               [&](int k, int j) { return sQ[k * ST + j]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dk[i][j] += acc[i][j];
      ds_mm<C>(ti, tj,
               [&](int i, int k) {
                 return k < i ? be[i] * H[i * CS + k] * e(i, k) : k > i ? be[k] * H[k * CS + i] * e(k, i) : 0.f;
               },
               [&](int k, int j) { return sK[k * ST + j]; }, acc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 4 * ti + i;
        if (t < n)
          *reinterpret_cast<float4*>(dk_part + ((row0 + t) * a.Hv + h) * D + 4 * tj) =
              make_float4(dk[i][0] - acc[i][0], dk[i][1] - acc[i][1], dk[i][2] - acc[i][2], dk[i][3] - acc[i][3]);
      }
    }
    // <dS+, S>, then dS itself.
    float x = 0.f;
    for (int i = tid; i < D * D; i += kDsThreads) x = fmaf(dS[(i / D) * ST + i % D], S[i], x);
    x = warp_sum(x);
    if (lane == 0) red[warp] = x;
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
      for (int i = tid; i < C; ++i) d += Ti[i * CS + tid];
      if (tid < n) *a.dg.at(row0 + tid, h) = from_f32<T>(d);
    }
    for (int b = tid; b < (D / 4) * TJ; b += kDsThreads) {
      const int bi = b / TJ, bj = b % TJ;
      ds_mm<C>(bi, bj, [&](int i, int k) { return sQ[k * ST + i] * (a.scale * eg[k]); },
               [&](int k, int j) { return sO[k * ST + j]; }, acc);
      float less[4][4];
      ds_mm<C>(bi, bj, [&](int i, int k) { return sK[k * ST + i] * (eg[k] * be[k]); },
               [&](int k, int j) { return sZ[k * ST + j]; }, less);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float* d = dS + (4 * bi + i) * ST + 4 * bj + j;
          *d = fmaf(whole, *d, acc[i][j] - less[i][j]);
        }
    }
  }
  __syncthreads();
  if (a.dS_in)
    for (int i = tid; i < D * D; i += kDsThreads) a.dS_in[base + i] = dS[(i / D) * ST + i % D];
}

// dq, dk of a key head: the sum over its value heads, in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_group_sum_kernel(const DeltaGradArgs<T> a,
                                                              const float* __restrict__ dq_part,
                                                              const float* __restrict__ dk_part) {
  SlotTile t;
  if (!slot_tile<kDsChunk>(a.seq, blockIdx.x, &t)) return;
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
// rows of S, so both products over d_k close through shared memory.
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

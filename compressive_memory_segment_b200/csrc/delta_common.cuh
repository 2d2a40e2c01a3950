// The gated delta rule over packed sequences. Per sequence and value head (key
// head h / G), with a_t = exp(g_t) and a state S [d_k, d_v] in fp32:
//   S' = a_t S_{t-1};  u_t = beta_t (v_t - S'^T k_t);  S_t = S' + k_t u_t^T
//   o_t = scale S_t^T q_t
#pragma once

#include "packed_common.cuh"

namespace infini {

// A decay below e^-200 is 0 in fp32, so log decays are cut there: -inf (a
// reset) then keeps the sums of logs, which are held in 64 bits, usable. A NaN is
// no reset and stays one.
constexpr float kDeltaMinLog = -200.f;
__device__ __forceinline__ float delta_log(float g) { return g < kDeltaMinLog ? kDeltaMinLog : g; }

template <typename T>
struct DeltaArgs {
  RowsOf<const T> q, k, v, g, beta;  // g, beta: one element a row
  RowsOf<T> out;
  const float* S_in;  // [n_seq][Hv][d][d] or null (zero)
  float* S_out;       // null: not written
  SeqTable seq;
  int Hk, Hv, G;
  float scale;
};

template <typename T>
struct DeltaGradArgs {
  RowsOf<const T> q, k, v, g, beta, dout;
  RowsOf<T> dq, dk, dv, dg, dbeta;
  const float* S_in;
  const float* dS_out;  // null: zero
  float* dS_in;         // null: not written
  SeqTable seq;
  int Hk, Hv, G;
  float scale;
};

}  // namespace infini

// Packed sequences: arguments shared by the packed attention and delta-rule
// kernels, and the map from a grid slot to a (sequence, tile) pair.
//
// The lengths live on the device, so a grid is sized by what the host knows:
// tiles of R rows of sequence s take the slots off[s] / R + s .. (+ tile).
// ceil(len / R) <= off[s + 1] / R - off[s] / R + 1 makes these ranges disjoint,
// T / R + n_seq slots hold all of them, and off[s] / R + s rises with s, so a
// CTA finds its sequence by a search; slots between two ranges stay empty.
// Offsets and lengths are clamped to the tensors before any use: bad ones give
// rows that are not computed and a bit in the status word, never an access out
// of range.
#pragma once

#include "common.cuh"

namespace infini {

constexpr unsigned int kStatusOffsets = 4u;

// Rows (t, h) of d elements at p + t * st + h * sh (elements, 64-bit).
template <typename T>
struct RowsOf {
  T* p;
  int64_t st, sh;
  __device__ __forceinline__ T* at(int64_t t, int h) const { return p + t * st + h * sh; }
};

struct SeqTable {
  const int* off;  // [n_seq + 1]
  const int* len;  // [n_seq] or null: off[s + 1] - off[s]
  int n_seq;
  int T;           // rows of the tensors it indexes
};

struct SeqRange {
  int first, len;
};

__device__ __forceinline__ SeqRange seq_range(const SeqTable& t, int s) {
  const int a = t.off[s], b = t.off[s + 1];
  int n = t.len ? t.len[s] : b - a;
  const bool ok = a >= 0 && b >= a && b <= t.T && n >= 0 && n <= b - a;
  if (ok) return {a, n};
  atomicOr(&g_status, kStatusOffsets);
  return {0, 0};  // the whole sequence is left out
}

// The sequence whose slot range holds `slot`, or -1. Called by whole warps; a
// 32-way search, one round of loads for up to 32 sequences, two for 1024.
template <int R>
__device__ __forceinline__ int slot_sequence(const SeqTable& t, int64_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = t.n_seq;
  do {
    const int step = (n + 31) / 32;
    bool le = false;
    if (lane * step < n) {
      const int s = lo + lane * step;
      const int o = max(0, min(t.off[s], t.T));
      le = (int64_t)(o / R) + s <= slot;
    }
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  } while (n > 1);
  return lo;
}

struct SlotTile {
  int seq, tile;   // tile of R rows inside the sequence
  SeqRange r;
};

template <int R>
__device__ __forceinline__ bool slot_tile(const SeqTable& t, int64_t slot, SlotTile* out) {
  const int s = slot_sequence<R>(t, slot);
  if (s < 0) return false;
  const SeqRange r = seq_range(t, s);
  const int64_t tile = slot - ((int64_t)(r.first / R) + s);
  if (tile < 0 || tile * R >= r.len) return false;
  out->seq = s;
  out->tile = (int)tile;
  out->r = r;
  return true;
}

// The same tiles, most work first, for up to 32 sequences (more: by slot): a
// launch of few and unequal units ends with its longest one otherwise. A
// sequence of m tiles has one of work w for each w of 1 .. m (causal attention:
// the last query tile sees the most keys, the first key tile the most queries),
// so c(w) = sum_s max(0, m_s - w + 1) units have work w or more, and unit i has the
// largest w with c(w) > i. Called by whole warps.
template <int R, bool LAST_HEAVY>
__device__ __forceinline__ bool work_tile(const SeqTable& t, int64_t unit, int64_t units, SlotTile* out) {
  if (t.n_seq > 32) return slot_tile<R>(t, LAST_HEAVY ? units - 1 - unit : unit, out);
  const int lane = threadIdx.x & 31;
  SeqRange r{0, 0};
  if (lane < t.n_seq) r = seq_range(t, lane);
  __syncwarp();
  const int m = (r.len + R - 1) / R, i = (int)unit;
  auto count = [&](int w) { return __reduce_add_sync(0xffffffffu, max(0, m - w + 1)); };
  if (count(1) <= i) return false;
  int lo = 1, hi = __reduce_max_sync(0xffffffffu, m);  // count(lo) > i
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (count(mid) > i)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int s = __fns(__ballot_sync(0xffffffffu, m >= lo), 0, i - count(lo + 1) + 1);
  out->seq = s;
  out->r = {__shfl_sync(0xffffffffu, r.first, s), __shfl_sync(0xffffffffu, r.len, s)};
  out->tile = LAST_HEAVY ? lo - 1 : __shfl_sync(0xffffffffu, m, s) - lo;
  return true;
}

// The sequence of rank `rank` by length, longest first, for up to 32 sequences
// (more: the sequence `rank` itself). Called by whole warps.
__device__ __forceinline__ int long_sequence(const SeqTable& t, int rank) {
  if (t.n_seq > 32) return rank;
  const int lane = threadIdx.x & 31, len = lane < t.n_seq ? seq_range(t, lane).len : -1;
  __syncwarp();
  int longer = 0;
#pragma unroll
  for (int s = 0; s < 32; ++s) {
    const int other = __shfl_sync(0xffffffffu, len, s);
    longer += other > len || (other == len && s < lane);
  }
  return __ffs(__ballot_sync(0xffffffffu, longer == rank)) - 1;
}

inline int64_t slot_count(int64_t T, int64_t n_seq, int R) { return T / R + n_seq; }

template <typename T>
struct PackedArgs {
  RowsOf<const T> q, k, v;
  RowsOf<T> out;
  float* lse;  // [Hq][Tq] or null
  SeqTable sq, sk;
  int Hq, Hkv, G;
  float scale;
  bool by_work;  // tensor-core forward: units with most work first
};

template <typename T>
struct PackedGradArgs {
  RowsOf<const T> q, k, v, out, dout;
  RowsOf<T> dq, dk, dv;
  const float* lse;  // [Hq][Tq]
  float* delta;      // [Hq][Tq] scratch: sum_c dout out
  SeqTable sq, sk;
  int Hq, Hkv, G;
  float scale;
};

// One row of D elements as fp32 into shared memory, by `NT` threads; rows from
// `valid` on are zero (what lies behind a sequence may be anything).
template <typename T, int D, int ROWS, int ST, int NT>
__device__ __forceinline__ void load_rows_f32(float* __restrict__ dst, const RowsOf<const T>& x, int64_t t0, int h,
                                              int valid, int tid) {
  constexpr int VE = 16 / (int)sizeof(T);
  constexpr int VPR = D / VE;
  for (int i = tid; i < ROWS * VPR; i += NT) {
    const int r = i / VPR, c = i % VPR;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (r < valid) w = *reinterpret_cast<const uint4*>(x.at(t0 + r, h) + c * VE);
    RowTile<T, D, ST, 1, VPR>::put(w, dst + r * ST + c * VE);
  }
}

}  // namespace infini

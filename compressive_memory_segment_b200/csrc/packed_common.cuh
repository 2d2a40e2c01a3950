// Packed sequences: arguments shared by the packed attention and delta-rule
// kernels, and the map from a grid slot to a (sequence, tile) pair.
//
// The lengths live on the device, so a grid is sized by what the host knows:
// tiles of R rows of sequence s take the slots off[s] / R + s .. (+ tile).
// ceil(len / R) <= off[s + 1] / R - off[s] / R + 1 makes these ranges disjoint,
// T / R + n_seq slots hold all of them, and off[s] / R + s rises with s, so a
// CTA finds its sequence by a search; slots between two ranges stay empty.
// Offsets and lengths are checked against the tensors before any use: bad ones
// give rows that are not computed and a bit in the status word, never an access
// out of range.
#pragma once

#include <limits.h>

#include "common.cuh"

namespace infini {

constexpr unsigned int kStatusOffsets = 4u;

// Rows (t, h) of d elements at p + t * st + h * sh (elements, 64-bit). The debug
// build knows how many there are, and a row that does not exist is the first one
// instead. (Tiles that come by TMA need no check: it reads nothing behind a tensor.)
template <typename T>
struct RowsOf {
  T* p;
  int64_t st, sh;
#ifdef INFINI_DEBUG
  int64_t n = 0;  // 0: not known
  int heads = 0;
#endif
  __device__ __forceinline__ T* at(int64_t t, int h) const {
#ifdef INFINI_DEBUG
    if (n > 0 && !INFINI_CHECK(t >= 0 && t < n && h >= 0 && h < heads)) return p;
#endif
    return p + t * st + h * sh;
  }
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

// The rows of sequence s, or false where its entries are no range of the tensor.
__device__ __forceinline__ bool seq_peek(const SeqTable& t, int s, SeqRange* r) {
  const int a = t.off[s], b = t.off[s + 1], room = (int)((unsigned)b - (unsigned)a);
  const int n = t.len ? t.len[s] : room;
  *r = {a, n};
  return a >= 0 && b >= a && b <= t.T && n >= 0 && n <= room;
}
// The same, a bad sequence reported and left out whole.
__device__ __forceinline__ SeqRange seq_range(const SeqTable& t, int s) {
  SeqRange r;
  if (seq_peek(t, s, &r)) return r;
  atomicOr(&g_status, kStatusOffsets);
  return {0, 0};
}
// A sequence in two tables (queries and keys), left out where either has it bad.
struct SeqPair {
  SeqRange own, other;
};
__device__ __forceinline__ SeqPair seq_pair(const SeqTable& t, const SeqTable& o, int s) {
  SeqPair p;
  const bool own = seq_peek(t, s, &p.own), other = seq_peek(o, s, &p.other);
  if (own && other) return p;
  atomicOr(&g_status, kStatusOffsets);
  return {{0, 0}, {0, 0}};
}
// Where a search leads the CTAs to their sequences, a bad one may be met by none:
// this launch ahead of such a call, 2 us, looks at all of them. (Inside the kernels it
// cost registers: dk and dv 5-12 %, the rows' D 14 -> 18 us.)
static __global__ void __launch_bounds__(256) packed_report_kernel(const SeqTable t, const SeqTable o) {
  for (int64_t s = (int64_t)blockIdx.x * 256 + threadIdx.x; s < t.n_seq; s += (int64_t)gridDim.x * 256)
    seq_pair(t, o, (int)s);
}

// A search over the table takes rounds of 32 runs of 32^k sequences, one a lane.
// This is the shift of the first round.
__device__ __forceinline__ int search_shift(int n_seq) { return n_seq <= 32 ? 0 : (31 - __clz(n_seq - 1)) / 5 * 5; }
// A lane's key in a round: the first slot of the first sequence of its run, `at`, whose offset is `o`.
template <int R>
__device__ __forceinline__ int run_key(int n_seq, int at, int o) {
  return at < n_seq ? (int)((unsigned)o / R) + at : INT_MAX;
}

// The search where offsets out of range have been met: a run is stood for by the
// first of its sequences whose offset is in range. (Apart, and not in line: it is
// seldom needed, and the kernels' code should stay small.)
template <int R>
__device__ __noinline__ int slot_sequence_careful(const int* off, int n_seq, int T, int64_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  for (int shift = search_shift(n_seq); shift >= 0; shift -= 5) {
    int at = lo + (lane << shift);
    const int end = (int)min((int64_t)n_seq, (int64_t)at + (1 << shift));
    while (at < end && (unsigned)off[at] > (unsigned)T) ++at;
    const bool le = at < end && run_key<R>(n_seq, at, off[at]) <= slot;
    const unsigned found = __ballot_sync(0xffffffffu, le);
    if (found == 0u) return -1;
    lo += (31 - __clz(found)) << shift;
  }
  return lo;
}

// The sequence whose slot range holds `slot`, or -1: the last one that starts at
// or before it, offsets out of range left aside. Called by whole warps; one round
// of loads for up to 32 sequences, two for 1024.
template <int R>
__device__ __forceinline__ int slot_sequence(const SeqTable& t, int64_t slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  bool bad = false;
  for (int shift = search_shift(t.n_seq); shift >= 0; shift -= 5) {
    const int at = lo + (lane << shift), o = at < t.n_seq ? t.off[at] : 0;
    bad |= (unsigned)o > (unsigned)t.T;
    const unsigned found = __ballot_sync(0xffffffffu, run_key<R>(t.n_seq, at, o) <= slot);
    if (found == 0u) {
      lo = -1;
      break;
    }
    lo += (31 - __clz(found)) << shift;
  }
  return __any_sync(0xffffffffu, bad) ? slot_sequence_careful<R>(t.off, t.n_seq, t.T, slot) : lo;
}

struct SlotTile {
  int seq, tile;  // tile of R rows inside the sequence
  SeqRange r;
  SeqRange other;  // attention: the sequence's rows on the other side
};

template <int R>
__device__ __forceinline__ bool slot_tile(const SeqTable& t, const SeqTable& o, int64_t slot, SlotTile* out) {
  const int s = slot_sequence<R>(t, slot);
  if (s < 0) return false;
  const SeqPair p = seq_pair(t, o, s);
  const int64_t tile = slot - ((int64_t)(p.own.first / R) + s);
  if (tile < 0 || tile * R >= p.own.len) return false;
  *out = {s, (int)tile, p.own, p.other};
  return true;
}

// The delta rule's kernels find a chunk's records and states by its slot, some
// coming from the slot and some from the sequence: all of them take a sequence
// or none does. Where offsets decrease, slots of one sequence may lead to another;
// such a sequence is reported and left out like a bad one. What slot_sequence
// answers rises with the slot, so the first and the last slot tell. The rounds of
// their searches are known ahead where they lead to s, and so are their loads.
struct SlotRounds {
  static constexpr int ROUNDS = 4;  // the delta rule has at most 65535 sequences
  int s, v[ROUNDS];
  static __device__ __forceinline__ int run(int s, int shift) {
    return (s & ~((32 << shift) - 1)) + ((threadIdx.x & 31) << shift);
  }
  __device__ __forceinline__ SlotRounds(const SeqTable& t, int s_) : s(s_) {
    const int top = search_shift(t.n_seq);
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) v[k] = 5 * k <= top && run(s, 5 * k) < t.n_seq ? t.off[run(s, 5 * k)] : 0;
  }
  template <int R>
  __device__ __forceinline__ bool lead_to(const SeqTable& t, int64_t first, int64_t last) const {
    const int top = search_shift(t.n_seq);
    bool bad = false, ok = true;
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
      if (5 * k > top) break;
      bad |= (unsigned)v[k] > (unsigned)t.T;
      const int key = run_key<R>(t.n_seq, run(s, 5 * k), v[k]), c = (s >> 5 * k) & 31;
      const unsigned f = __ballot_sync(0xffffffffu, key <= first), l = __ballot_sync(0xffffffffu, key <= last);
      ok = ok && f >> c == 1u && l >> c == 1u;
    }
    if (__any_sync(0xffffffffu, bad))
      ok = slot_sequence_careful<R>(t.off, t.n_seq, t.T, first) == s &&
           slot_sequence_careful<R>(t.off, t.n_seq, t.T, last) == s;
    return ok;
  }
};
// For a CTA of sequence s (rounds.s, rows r): whether to take it. Loads that do no
// harm where it is left out go ahead of this.
template <int R>
__device__ __forceinline__ bool chunks_found(const SlotRounds& rounds, const SeqTable& t, const SeqRange& r) {
  const int64_t first = (int64_t)(r.first / R) + rounds.s;
  if (r.len == 0 || rounds.lead_to<R>(t, first, first + (r.len - 1) / R)) return true;
  atomicOr(&g_status, kStatusOffsets);
  return false;
}
// For a CTA that its slot leads to a tile: the tile, and whether to take it (a
// sequence of one tile needs no more).
template <int R>
__device__ __forceinline__ bool chunk_tile(const SeqTable& t, int64_t slot, SlotTile* out) {
  const int s = slot_sequence<R>(t, slot);
  if (s < 0) return false;
  const SeqRange r = seq_range(t, s);
  const int64_t tile = slot - ((int64_t)(r.first / R) + s);
  if (tile < 0 || tile * R >= r.len) return false;
  *out = {s, (int)tile, r, {0, 0}};
  return true;
}
template <int R>
__device__ __forceinline__ bool tile_found(const SeqTable& t, const SlotTile& x) {
  return x.r.len <= R || chunks_found<R>(SlotRounds(t, x.seq), t, x.r);
}

// The same tiles, most work first, for up to 32 sequences (more: by slot): a
// launch of few and unequal units ends with its longest one otherwise. A
// sequence of m tiles has one of work w for each w of 1 .. m (causal attention:
// the last query tile sees the most keys, the first key tile the most queries),
// so c(w) = sum_s max(0, m_s - w + 1) units have work w or more, and unit i has the
// largest w with c(w) > i. Called by whole warps.
template <int R, bool LAST_HEAVY>
__device__ __forceinline__ bool few_tile(const SeqTable& t, const SeqTable& o, int64_t unit, SlotTile* out) {
  const int lane = threadIdx.x & 31;
  SeqPair p{{0, 0}, {0, 0}};
  if (lane < t.n_seq) p = seq_pair(t, o, lane);
  __syncwarp();
  const int m = (p.own.len + R - 1) / R, i = (int)unit;
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
  out->r = {__shfl_sync(0xffffffffu, p.own.first, s), __shfl_sync(0xffffffffu, p.own.len, s)};
  out->other = {__shfl_sync(0xffffffffu, p.other.first, s), __shfl_sync(0xffffffffu, p.other.len, s)};
  out->tile = LAST_HEAVY ? lo - 1 : __shfl_sync(0xffffffffu, m, s) - lo;
  return true;
}

template <int R, bool LAST_HEAVY>
__device__ __forceinline__ bool work_tile(const SeqTable& t, const SeqTable& o, int64_t unit, int64_t units,
                                          SlotTile* out) {
  return t.n_seq > 32 ? slot_tile<R>(t, o, LAST_HEAVY ? units - 1 - unit : unit, out)
                      : few_tile<R, LAST_HEAVY>(t, o, unit, out);
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

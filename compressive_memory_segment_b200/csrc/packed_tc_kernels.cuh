// Causal softmax attention over packed sequences on the tensor cores (bf16, d =
// 64 or 128): forward.
//
// A CTA owns two neighbouring 128-row query tiles of one head and streams the
// 128-key tiles that they see. Per tile pair and key tile: S = Q K^T into TMEM,
// one thread per row takes its 128 scores, keeps the running maximum and sum,
// writes P = exp(S - m) as bf16 over S, and O += P V accumulates in TMEM. While
// one tile's softmax runs the tensor cores work on the other tile. The maximum
// that scales P moves only when a row's grows by more than 2^8 (P stays within
// bf16's and the sums within fp32's range), so O is rescaled a few times per
// row, by the thread that owns it.
//
// Per pair of tiles and keys (2 x 128 x 128) the tensor cores need 2048 cycles
// at d = 128, and the 32768 exponentials 2048 cycles of the SM's 16 per cycle.
// What bounds it are the products: both operands of Q K^T come from shared memory,
// at its full rate, while the next tiles arrive there, so that a tile's takes 720
// cycles instead of 512 (a part of the exponentials on the multiply-add pipes made
// the softmax shorter and the kernel slower, 523 -> 557 us). Measured: one sequence
// of 8192, 32 / 8 heads, d = 128: 524 us, 1.05 PFLOP/s (0.64 of the burst rate of a
// plain matrix product; 3530 cycles a pair of tiles, 2900 of them products); 16
// sequences of 64-2048, 16 heads: 219 us, 0.64 PFLOP/s, where a unit has a few
// tiles only and its first product and last output stand alone.
//
// Bytes behind a sequence belong to its neighbour: the scores there are
// replaced by -inf, and the rows of V in the sequence's last tile are zeroed in
// shared memory before the product (0 x NaN is NaN).
//
// warps 0-3, 4-7  softmax and epilogue of query tile 0, 1
// warp 8          MMA issuer (and TMEM owner);  warp 9  TMA producer
// TMEM: S0 | S1 at columns 0, 128 (P in the first 64 of each), O0 | O1 behind.
#pragma once

#include "packed_common.cuh"
#include "tc_kernels.cuh"

namespace infini {
namespace tc {

constexpr int kPkThreads = 320;
constexpr int kPkRows = 2 * kTile;

template <int D>
struct PkFwd {
  static constexpr uint32_t kBytes = D / 64 * kHalf;  // a 128 x D bf16 tile
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr uint32_t kSmem = (2 + kStages) * kBytes + 512;
  static constexpr uint32_t kColO = 256;
};

// Work stealing over the grid: a running CTA asks for the index of one that has
// not been launched, which then never is; so CTAs stay on their SM with their
// pipelines full, and the longest units (launched first) even out. The answer
// (16 bytes) is written to shared memory and counted on `bar`.
__device__ __forceinline__ void steal_request(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The stolen CTA's blockIdx.x, or -1 if none was left.
__device__ __forceinline__ int64_t steal_answer(const void* answer) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\tmov.u32 %0, 0;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %1, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "=r"(x), "=r"(got)
      : "r"(smem_u32(answer))
      : "memory");
  return got ? (int64_t)x : -1;
}
// One unit of a persistent attention kernel, as its producer warp hands it to
// the other roles: a tile of rows of one head of one sequence.
struct PkUnit {
  int head, tile, first, len, other_first, other_len, n0, n1;  // n0 < 0: no more units
};

// Box {64 of d, 1 head, rows} at (x, head, row); x is 0 or 64 (bf16).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, int32_t x, int32_t h, int32_t row,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(h), "r"(row), "r"(smem_u32(bar))
      : "memory");
}
// ROWS x D tile in 64-column blocks of ROWS x 128 bytes.
template <int D, int ROWS>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* m, int h, int row, uint64_t* bar) {
#pragma unroll
  for (int b = 0; b < D / 64; ++b) tma_load_3d(dst + b * ROWS * 128, m, b * 64, h, row, bar);
}
// Zeroes rows [from, ROWS) of such a tile (a whole warp).
template <int D, int ROWS>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
  for (int i = from * 8 + lane; i < ROWS * 8; i += 32)
#pragma unroll
    for (int b = 0; b < D / 64; ++b) *reinterpret_cast<uint4*>(tile + b * ROWS * 128 + i * 16) = make_uint4(0, 0, 0, 0);
}

// max over 128 scores
__device__ __forceinline__ float row_max(const uint32_t* s) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 128; c += 8)
#pragma unroll
    for (int t = 0; t < 4; ++t)
      m[t] = max3f(m[t], __uint_as_float(s[c + 2 * t]), __uint_as_float(s[c + 2 * t + 1]));
  return fmaxf(max3f(m[0], m[1], m[2]), m[3]);
}

template <int D>
__global__ void __launch_bounds__(kPkThreads, 1)
packed_tc_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PackedArgs<__nv_bfloat16> a, int64_t slots,
                     uint32_t epoch) {
  using C = PkFwd<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) flag_timeout();
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* ring = smem_raw + 2 * C::kBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + C::kStages * C::kBytes);
  uint64_t* q_full = bars;                       // [2]
  uint64_t* full = bars + 2;                     // [kStages]
  uint64_t* tail = full + C::kStages;            // a sequence's last tile of V has landed
  uint64_t* stolen = tail + 1;                   // the next CTA's index has come
  uint64_t* empty = stolen + 1;                  // [kStages]
  uint64_t* q_empty = empty + C::kStages;        // [2] the unit's last Q K^T of a query tile done
  uint64_t* s_full = q_empty + 2;                // [2]
  uint64_t* p_full = s_full + 2;                 // [2], one arrival per warp
  uint64_t* pv_done = p_full + 2;                // [2]
  uint64_t* unit_full = pv_done + 2;             // [2]
  uint64_t* unit_empty = unit_full + 2;          // [2] read by the softmax warps and the MMA warp
  uint64_t* drain = unit_empty + 2;
  constexpr int kBars = 17 + 2 * C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  PkUnit* units = reinterpret_cast<PkUnit*>(bars + kBars + 1);  // [2]
  uint8_t* answer = reinterpret_cast<uint8_t*>(bars) + 512 - 16;
  static_assert(kBars * 8 + 8 + 2 * sizeof(PkUnit) <= 512 - 16, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < kBars; ++b) mbar_init(&bars[b], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&p_full[b], 4);
      mbar_init(&unit_empty[b], 9);
    }
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  uint32_t armed = 0;  // producer: barriers with a copy in flight, by their index in bars

  if (warp == 9) {
    // ------------------------------------------------ producer: units, Q, then K and V of each tile in turn
    if (elect_one_lane()) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    int64_t block = blockIdx.x;
    const bool by_work = a.by_work && a.sq.n_seq <= 32;
    int g = 0, tails = 0, asked = 0, qn[2] = {0, 0};  // stages, cut tiles, requests, query tiles so far
    for (int k = 0; ok; ++k) {
      // The next unit that has rows; units[] is double buffered.
      PkUnit un;
      un.n0 = -1;
      while (block >= 0) {
        SlotTile t;
        const bool have = by_work ? few_tile<kPkRows, true>(a.sq, a.sk, block / a.Hq, &t)
                                  : slot_tile<kPkRows>(a.sq, a.sk, slots - 1 - block / a.Hq, &t);
        if (have) {
          const SeqRange kr = t.other;
          const int shift = kr.len - t.r.len;
          int n_kt[2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int r0 = t.tile * kPkRows + w * kTile, rows = min(kTile, t.r.len - r0);
            n_kt[w] = rows > 0 ? (max(0, min(kr.len, r0 + rows + shift)) + kTile - 1) / kTile : 0;
          }
          un = {(int)(block % a.Hq), t.tile, t.r.first, t.r.len, kr.first, kr.len, n_kt[0], n_kt[1]};
        }
        // Ask for the one after it; the answer is there by the time it is needed.
        if (elect_one_lane()) {
          mbar_arrive_expect_tx(stolen, 16);
          steal_request(answer, stolen);
        }
        __syncwarp();
        armed |= 1u << (stolen - bars);
        ++asked;
        if (have) break;
        if (!(ok = mbar_wait_warp(stolen, (asked - 1) & 1, epoch))) break;
        block = steal_answer(answer);
        fence_proxy_async_smem();  // the read before the next answer's write
        __syncwarp();
      }
      if (!ok) break;
      if (k >= 2 && !(ok = mbar_wait_warp(&unit_empty[k & 1], ((k >> 1) - 1) & 1, epoch))) break;
      if (lane == 0) {
        units[k & 1] = un;
        mbar_arrive(&unit_full[k & 1]);
      }
      __syncwarp();
      if (un.n0 < 0) break;
      const int n = max(un.n0, un.n1), hk = un.head / a.G;
      for (int w = 0; w < 2 && ok; ++w) {
        if ((w ? un.n1 : un.n0) == 0) continue;
        if (qn[w] > 0 && !(ok = mbar_wait_warp(&q_empty[w], (qn[w] - 1) & 1, epoch))) break;
        ++qn[w];
        armed |= 1u << w;
        if (elect_one_lane()) {
          mbar_arrive_expect_tx(&q_full[w], C::kBytes);
          load_rows<D, kTile>(sQ + w * C::kBytes, &tmQ, un.head, un.first + un.tile * kPkRows + w * kTile, &q_full[w]);
        }
        __syncwarp();
      }
      for (int i = 0; i < 2 * n && ok; ++i, ++g) {
        const int slot = g % C::kStages, use = g / C::kStages, j = i >> 1;
        if (use > 0 && !(ok = mbar_wait_warp(&empty[slot], (use - 1) & 1, epoch))) break;
        uint8_t* dst = ring + slot * C::kBytes;
        const int valid = un.other_len - j * kTile;
        if ((i & 1) && valid < kTile) {  // the sequence's last rows of V: zeros behind them
          armed |= 1u << (tail - bars);
          if (elect_one_lane()) {
            mbar_arrive_expect_tx(tail, C::kBytes);
            load_rows<D, kTile>(dst, &tmV, hk, un.other_first + j * kTile, tail);
          }
          __syncwarp();
          if (!(ok = mbar_wait_warp(tail, tails & 1, epoch))) break;
          ++tails;
          zero_rows<D, kTile>(dst, valid, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one_lane()) mbar_arrive(&full[slot]);
        } else {
          armed |= 1u << (2 + slot);
          if (elect_one_lane()) {
            mbar_arrive_expect_tx(&full[slot], C::kBytes);
            load_rows<D, kTile>(dst, (i & 1) ? &tmV : &tmK, hk, un.other_first + j * kTile, &full[slot]);
          }
        }
        __syncwarp();
      }
      if (!ok || !(ok = mbar_wait_warp(stolen, (asked - 1) & 1, epoch))) break;
      block = steal_answer(answer);
      fence_proxy_async_smem();
      __syncwarp();
    }
  } else if (warp == 8) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, false, false), id_pv = idesc_bf16_f32(128, D, false, true);
      const uint64_t q0 = desc_kmajor_sw128(smem_u32(sQ)), k0 = desc_kmajor_sw128(smem_u32(ring)),
                     v0 = desc_mnmajor_sw128(smem_u32(ring), kHalf);
      int g0 = 0, qn[2] = {0, 0}, pn[2] = {0, 0};  // first stage of the unit; query tiles and key tiles so far
      for (int k = 0; ok; ++k) {
        if (!(ok = mbar_wait(&unit_full[k & 1], (k >> 1) & 1, epoch))) break;
        const int n_kt[2] = {units[k & 1].n0, units[k & 1].n1};
        mbar_arrive(&unit_empty[k & 1]);
        if (n_kt[0] < 0) break;
        const int n = max(n_kt[0], n_kt[1]);
        // Stage g0 + i holds K of tile i / 2 (even i) or V (odd).
        auto qk = [&](int w, int j) {
          const int g = g0 + 2 * j, slot = g % C::kStages;
          if (!mbar_wait(&full[slot], (g / C::kStages) & 1, epoch)) return false;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + w * 128, q0 + ((w * C::kBytes) >> 4) + kmaj_step(kk),
                        k0 + ((slot * C::kBytes) >> 4) + kmaj_step(kk), id_qk, kk != 0);
          mma_commit(&s_full[w]);
          if (j == n_kt[w] - 1) mma_commit(&q_empty[w]);
          return true;
        };
        for (int w = 0; w < 2 && ok; ++w)
          if (n_kt[w] > 0) ok = mbar_wait(&q_full[w], qn[w]++ & 1, epoch) && qk(w, 0);
        if (ok && n > 0) mma_commit(&empty[g0 % C::kStages]);
        for (int j = 0; j < n && ok; ++j) {
          const int g = g0 + 2 * j + 1, slot = g % C::kStages;
          for (int w = 0; w < 2 && ok; ++w) {
            if (j >= n_kt[w]) continue;
            ok = mbar_wait(&full[slot], (g / C::kStages) & 1, epoch) && mbar_wait(&p_full[w], pn[w]++ & 1, epoch);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts(tmem + C::kColO + w * D, tmem + w * 128 + kk * 8,
                          v0 + ((slot * C::kBytes) >> 4) + mnmaj_step(kk), id_pv, (j | kk) != 0);
            mma_commit(&pv_done[w]);
            if (j + 1 < n_kt[w]) ok = qk(w, j + 1);
          }
          if (ok) {
            mma_commit(&empty[slot]);
            if (j + 1 < n) mma_commit(&empty[(g + 1) % C::kStages]);
          }
        }
        g0 += 2 * n;
      }
    }
  } else {
    // ------------------------------------------------ softmax: thread = row
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t ts = tmem + w * 128 + ((uint32_t)(quarter * 32) << 16);
    const uint32_t to = tmem + C::kColO + w * D + ((uint32_t)(quarter * 32) << 16);
    const float scale2 = a.scale * 1.4426950408889634f;
    int it = 0;  // key tiles so far
    for (int k = 0; ok; ++k) {
      if (!(ok = mbar_wait_warp(&unit_full[k & 1], (k >> 1) & 1, epoch))) break;
      const PkUnit un = units[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[k & 1]);
      if (un.n0 < 0) break;
      const int n = w ? un.n1 : un.n0, row0 = un.tile * kPkRows + w * kTile;
      const int row = row0 + r, shift = un.other_len - un.len, nk = un.other_len;
      const int last = min(nk - 1, row + shift);                    // last key this row sees
      const int first_masked = min(nk, row0 + shift + 1) / kTile;   // tile whose scores may need a mask
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++it) {
        if (!(ok = mbar_wait_warp(&s_full[w], it & 1, epoch))) break;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_ld32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_ld32(ts + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
        tmem_ld32(ts + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
        tmem_ld_wait_regs(s);
        if (j >= first_masked) {
          const int see = last - j * kTile;  // columns up to this one
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > see) s[c] = __float_as_uint(-INFINITY);
        }
        const float top = row_max(s) * scale2;
        const bool need = top > m + 8.f;  // also the first finite maximum: m is -inf until then
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? top : m;
          const float fix = mn == -INFINITY ? 1.f : ex2(m - mn);
          if (j > 0) {  // every P V so far is in O once the last one is done
            if (!(ok = mbar_wait_warp(&pv_done[w], (it - 1) & 1, epoch))) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < D; cb += 16) {
              uint32_t o[16];
              tmem_ld16(to + cb, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * fix);
              tmem_st16(to + cb, o);
            }
            tmem_st_wait();
          }
          l *= fix;
          m = mn;
        }
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: every p is 2^-inf = 0
        const uint64_t sc2 = f32x2(scale2, scale2), nm2 = f32x2(-base, -base);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
#pragma unroll
          for (int c = ch * 32; c < ch * 32 + 32; c += 2) exp2_pair(s, c, sc2, nm2, acc[(c >> 1) & 3]);
          tmem_st16(ts + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&s[ch * 16]));
        }
        l += sum_f32x2(acc);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      // Epilogue: O / l, each thread its row. The next unit's first P V, which
      // overwrites O, waits for this warp's next P.
      if (ok && n > 0 && (ok = mbar_wait_warp(&pv_done[w], (it - 1) & 1, epoch))) tc_fence_after();
      if (!ok) break;
      if (row0 < un.len) {
        // Whether the row sees a key goes by its place: its maximum is -inf for NaN scores too.
        const bool none = last < 0;
        const float inv = 1.f / l;
        const bool mine = row < un.len;
        __nv_bfloat16* dst = a.out.at(un.first + (mine ? row : 0), un.head);
#pragma unroll
        for (int cb = 0; cb < D; cb += 32) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(to + cb, o);
            tmem_ld_wait_regs(o);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0u;
          }
          if (mine) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t p[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                // a row that saw no key holds what P V = 0 left; it is 0 all the same
                const float lo = none ? 0.f : __uint_as_float(o[8 * x + 2 * y]) * inv;
                const float hi = none ? 0.f : __uint_as_float(o[8 * x + 2 * y + 1]) * inv;
                p[y] = pack_bf16x2(lo, hi);
              }
              *reinterpret_cast<uint4*>(dst + cb + 8 * x) = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
        }
        if (mine && a.lse)
          a.lse[(int64_t)un.head * a.sq.T + un.first + row] =
              none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        tc_fence_before();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*reinterpret_cast<volatile unsigned int*>(&g_abort_epoch) == epoch) {
    // Abort path: this CTA's own copies (one of an armed barrier's two
    // parities is complete) and MMAs finish before exit.
    if (warp == 9 && lane == 0)
      for (int b = 0; b < kBars; ++b)
        if (armed >> b & 1u) {
          mbar_drain(&bars[b], 0);
          mbar_drain(&bars[b], 1);
        }
    if (warp == 8 && lane == 0) {
      mma_commit(drain);
      mbar_drain(drain, 0);
    }
    __syncthreads();
  }
  if (warp == 8) tmem_dealloc(tmem, 512);
}

}  // namespace tc
}  // namespace infini

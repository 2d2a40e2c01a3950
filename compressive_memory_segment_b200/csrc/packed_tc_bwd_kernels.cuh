// Causal softmax attention over packed sequences on the tensor cores (bf16, d =
// 64 or 128): gradients.
//
// One kernel for both sides. A CTA keeps 128 rows X, Y and streams 64-row tiles
// A, B of the other side:
//   dq     (KEYS = false): X = Q, Y = dout of one head;   A = K, B = V
//   dk, dv (KEYS = true):  X = K, Y = V of one key head;  A = Q, B = dout, query
//          tile after query tile and head after head of the group
//   S = X A^T, E = Y B^T;  p = exp(scale S - lse), ds = p (E - D);
//   acc += ds A (dq or dk, scaled at the end), acc2 += p B (dv)
// Every sum has one order (no atomics); the price is that S and E are formed
// twice, once for each side: 7 products instead of 5.
//
// Two buffers of S and E in TMEM alternate between two groups of four warps
// (one thread per row), so the products of one tile run under the arithmetic of
// the other; p and ds go back to TMEM as bf16 over S and E and are the A operand
// of the accumulating products. A tile costs the tensor cores 768 (dq) or 1024
// cycles at d = 128 and the exponentials 512.
//
// Rows of A and B behind the sequence are zeroed in shared memory (they meet
// zeros of p and ds, and 0 x NaN is NaN).
//
// warps 0-3, 4-7  rows of even, odd tiles;  warp 8  MMA issuer;  warp 9  TMA producer
// TMEM at D = 128: S0 S1 E0 E1 (64 columns each), acc (D), acc2 (D).
#pragma once

#include "packed_tc_kernels.cuh"

namespace infini {
namespace tc {

constexpr int kPbThreads = 320;
constexpr int kPbCols = 64;  // rows of a streamed tile

template <int D>
struct PkBwd {
  static constexpr uint32_t kFix = D / 64 * kHalf;                // a 128 x D tile
  static constexpr uint32_t kTileA = D / 64 * kPbCols * 128;      // a 64 x D tile
  static constexpr uint32_t kStage = 2 * kTileA + 2 * kPbCols * 4;  // A | B | lse | D of 64 queries
  static constexpr int kStages = 4;
  static constexpr uint32_t kSmem = 2 * kFix + kStages * kStage + 256;
  static constexpr uint32_t kColE = 128, kColAcc = 256, kColAcc2 = 256 + D;
};

template <int D, bool KEYS>
__global__ void __launch_bounds__(kPbThreads, 1)
packed_tc_bwd_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY,
                     const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const PackedGradArgs<__nv_bfloat16> a, int64_t slots, uint32_t epoch) {
  using C = PkBwd<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) flag_timeout();
    return;
  }
  uint8_t* sX = smem_raw;
  uint8_t* sY = smem_raw + C::kFix;
  uint8_t* tiles = smem_raw + 2 * C::kFix;                          // [kStages][A | B]
  float* rows_ld = reinterpret_cast<float*>(tiles + C::kStages * 2 * C::kTileA);  // [kStages][lse | D][64]
  uint64_t* bars = reinterpret_cast<uint64_t*>(rows_ld + C::kStages * 2 * kPbCols);
  uint64_t* fix_full = bars;
  uint64_t* full = bars + 1;              // [kStages]
  uint64_t* empty = full + C::kStages;    // [kStages]
  uint64_t* s_full = empty + C::kStages;  // [2] S and E of a buffer done
  uint64_t* ds_full = s_full + 2;         // [2] p and ds written, one arrival per warp
  uint64_t* fin = ds_full + 2;            // every product done
  uint64_t* tail = fin + 1;               // [2] a tile that ends behind its sequence has landed
  uint64_t* drain = tail + 2;
  constexpr int kBars = 1 + 2 * C::kStages + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  static_assert(kBars * 8 + 8 <= 256, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned heads = KEYS ? a.Hkv : a.Hq;
  const int head = (int)(blockIdx.x % heads);  // the output's
  const int64_t place = blockIdx.x / heads;
  SlotTile t;
  if (!slot_tile<kTile>(KEYS ? a.sk : a.sq, KEYS ? place : slots - 1 - place, &t)) return;
  const SeqRange other = seq_range(KEYS ? a.sq : a.sk, t.seq);
  const int nq = KEYS ? other.len : t.r.len, nk = KEYS ? t.r.len : other.len, shift = nk - nq;
  const int r0 = t.tile * kTile, rows = min(kTile, t.r.len - r0);
  // Streamed rows: keys up to the last row's, or queries from the first that
  // sees key r0; whole tiles from a multiple of 64.
  const int first = KEYS ? min(nq, max(0, r0 - shift)) / kPbCols * kPbCols : 0;
  const int end = KEYS ? nq : max(0, min(nk, r0 + rows + shift));
  const int per_head = end > first ? (end - first + kPbCols - 1) / kPbCols : 0;
  const int n = per_head * (KEYS ? a.G : 1);
  const int limit = KEYS ? nq : nk;   // rows of the streamed side that exist

  if (threadIdx.x == 0) {
    for (int b = 0; b < kBars; ++b) mbar_init(&bars[b], &bars[b] == ds_full || &bars[b] == ds_full + 1 ? 4 : 1);
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
    // ------------------------------------------------ TMA producer
    if (n > 0) {
      const int row = t.r.first + r0;
      armed |= 1u;
      if (elect_one_lane()) {
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmY);
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        mbar_arrive_expect_tx(fix_full, 2 * C::kFix);
        load_rows<D, kTile>(sX, &tmX, head, row, fix_full);
        load_rows<D, kTile>(sY, &tmY, head, row, fix_full);
      }
      __syncwarp();
      int tails = 0;
      for (int i = 0; i < n && ok; ++i) {
        const int slot = i % C::kStages, use = i / C::kStages;
        const int g = KEYS ? i / per_head : 0, c0 = first + (i - g * per_head) * kPbCols;
        const int h = KEYS ? head * a.G + g : head / a.G;  // head of the streamed rows
        const int valid = limit - c0;
        float le[2], de[2];
        if (KEYS) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int q = c0 + lane + 32 * x;
            const int64_t at = (int64_t)h * a.sq.T + other.first + q;
            le[x] = q < nq ? a.lse[at] * 1.4426950408889634f : 0.f;
            de[x] = q < nq ? a.delta[at] : 0.f;
          }
        }
        if (use > 0 && !(ok = mbar_wait_warp(&empty[slot], (use - 1) & 1, epoch))) break;
        uint8_t* sa = tiles + slot * 2 * C::kTileA;
        const bool cut = valid < kPbCols;
        uint64_t* bar = cut ? tail + (tails & 1) : &full[slot];
        armed |= 1u << (bar - bars);
        if (KEYS) {
          float* ld = rows_ld + slot * 2 * kPbCols;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ld[lane + 32 * x] = le[x];
            ld[kPbCols + lane + 32 * x] = de[x];
          }
          __syncwarp();
        }
        if (elect_one_lane()) {
          mbar_arrive_expect_tx(bar, 2 * C::kTileA);
          load_rows<D, kPbCols>(sa, &tmA, h, other.first + c0, bar);
          load_rows<D, kPbCols>(sa + C::kTileA, &tmB, h, other.first + c0, bar);
        }
        __syncwarp();
        if (cut) {
          if (!(ok = mbar_wait_warp(bar, (tails >> 1) & 1, epoch))) break;
          ++tails;
          zero_rows<D, kPbCols>(sa, valid, lane);
          zero_rows<D, kPbCols>(sa + C::kTileA, valid, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (elect_one_lane()) mbar_arrive(&full[slot]);
          __syncwarp();
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(128, kPbCols, false, false), id_acc = idesc_bf16_f32(128, D, false, true);
      const uint64_t x0 = desc_kmajor_sw128(smem_u32(sX)), y0 = desc_kmajor_sw128(smem_u32(sY)),
                     t0 = desc_kmajor_sw128(smem_u32(tiles)),
                     m0 = desc_mnmajor_sw128(smem_u32(tiles), kPbCols * 128);
      auto stage = [&](int i) { return (uint32_t)((i % C::kStages) * 2 * C::kTileA) >> 4; };
      auto step64 = [](int kk) { return (uint32_t)((kk >> 2) * kPbCols * 128 + (kk & 3) * 32) >> 4; };
      auto scores = [&](int i) {
        if (!mbar_wait(&full[i % C::kStages], (i / C::kStages) & 1, epoch)) return false;
        const uint32_t b = i & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(tmem + b * 64, x0 + kmaj_step(kk), t0 + stage(i) + step64(kk), id_s, kk != 0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(tmem + C::kColE + b * 64, y0 + kmaj_step(kk), t0 + stage(i) + (C::kTileA >> 4) + step64(kk), id_s,
                      kk != 0);
        mma_commit(&s_full[b]);
        return true;
      };
      ok = mbar_wait(fix_full, 0, epoch) && scores(0) && (n < 2 || scores(1));
      for (int i = 0; i < n && ok; ++i) {
        const uint32_t b = i & 1;
        if (!(ok = mbar_wait(&ds_full[b], (i >> 1) & 1, epoch))) break;
        tc_fence_after();
        if (KEYS) {
#pragma unroll
          for (int kk = 0; kk < kPbCols / 16; ++kk)
            mma_bf16_ts(tmem + C::kColAcc2, tmem + b * 64 + kk * 8, m0 + stage(i) + (C::kTileA >> 4) + mnmaj_step(kk),
                        id_acc, (i | kk) != 0);
        }
#pragma unroll
        for (int kk = 0; kk < kPbCols / 16; ++kk)
          mma_bf16_ts(tmem + C::kColAcc, tmem + C::kColE + b * 64 + kk * 8, m0 + stage(i) + mnmaj_step(kk), id_acc,
                      (i | kk) != 0);
        mma_commit(&empty[i % C::kStages]);
        if (i + 2 < n) ok = scores(i + 2);
      }
      if (ok) mma_commit(fin);
    }
  } else {
    // ------------------------------------------------ thread = row of X
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + w * 64 + lanes, te = tmem + C::kColE + w * 64 + lanes;
    const float scale2 = a.scale * 1.4426950408889634f;
    float lse = 0.f, dlt = 0.f;
    if (!KEYS && r < rows) {
      const int64_t at = (int64_t)head * a.sq.T + t.r.first + r0 + r;
      lse = a.lse[at] * 1.4426950408889634f;
      dlt = a.delta[at];
    }
    for (int i = w; i < n; i += 2) {
      const int c0 = first + (KEYS ? i % per_head : i) * kPbCols;
      if (!(ok = mbar_wait_warp(&s_full[w], (i >> 1) & 1, epoch))) break;
      tc_fence_after();
      // Columns that row r takes part in: [lo, hi).
      const bool cut = KEYS ? c0 + shift < r0 + kTile - 1 || c0 + kPbCols > nq
                            : c0 + kPbCols - 1 > r0 + shift || c0 + kPbCols > nk;
      const int lo = KEYS ? r0 + r - shift - c0 : 0;
      const int hi = KEYS ? nq - c0 : min(nk, r0 + r + shift + 1) - c0;
      const float* ld = rows_ld + (i % C::kStages) * 2 * kPbCols;
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t s[32], e[32];
        tmem_ld32(ts + ch * 32, s);
        tmem_ld32(te + ch * 32, e);
        tmem_ld_wait_regs(s);
        tmem_ld_wait_regs(e);
        uint32_t pk[16], dk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          float p[4], d[4];
          float4 l4, d4;
          if (KEYS) {
            l4 = *reinterpret_cast<const float4*>(ld + ch * 32 + c);
            d4 = *reinterpret_cast<const float4*>(ld + kPbCols + ch * 32 + c);
          } else {
            l4 = make_float4(lse, lse, lse, lse);
            d4 = make_float4(dlt, dlt, dlt, dlt);
          }
          const float lv[4] = {l4.x, l4.y, l4.z, l4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            p[x] = ex2(fmaf(__uint_as_float(s[c + x]), scale2, -lv[x]));
            d[x] = p[x] * (__uint_as_float(e[c + x]) - dv[x]);
            if (cut) {
              const int col = ch * 32 + c + x;
              if (col < lo || col >= hi) p[x] = d[x] = 0.f;
            }
          }
          pk[c / 2] = pack_bf16x2(p[0], p[1]);
          pk[c / 2 + 1] = pack_bf16x2(p[2], p[3]);
          dk[c / 2] = pack_bf16x2(d[0], d[1]);
          dk[c / 2 + 1] = pack_bf16x2(d[2], d[3]);
        }
        // Column 16 ch of the buffer is read by now: 32 ch covers it.
        if (KEYS) tmem_st16(ts + ch * 16, pk);
        tmem_st16(te + ch * 16, dk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[w]);
    }
    // Epilogue: warps 0-3 write dk (or the first half of dq's columns), warps
    // 4-7 dv (or the second half), whole rows through shared memory.
    if (ok && n > 0 && (ok = mbar_wait_warp(fin, 0, epoch))) tc_fence_after();
    if (ok) {
      constexpr int W = KEYS ? D : D / 2, V = W / 8;  // columns of this thread, 16-byte pieces
      const uint32_t from = tmem + lanes + (KEYS ? (w ? C::kColAcc2 : C::kColAcc) : C::kColAcc + w * W);
      const float mul = KEYS && w ? 1.f : a.scale;
      uint8_t* stage = (KEYS ? (w ? sY : sX) : sX + w * 128 * W * 2) + quarter * 32 * W * 2;
#pragma unroll
      for (int cb = 0; cb < W; cb += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(from + cb, o);
          tmem_ld_wait_regs(o);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            p[y] = pack_bf16x2(__uint_as_float(o[8 * x + 2 * y]) * mul, __uint_as_float(o[8 * x + 2 * y + 1]) * mul);
          const int piece = cb / 8 + x;
          *reinterpret_cast<uint4*>(stage + lane * W * 2 + ((piece ^ (lane & (V < 8 ? V - 1 : 7))) * 16)) =
              make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
      __syncwarp();
      const RowsOf<__nv_bfloat16>& dst = KEYS ? (w ? a.dv : a.dk) : a.dq;
      for (int x = lane; x < 32 * V; x += 32) {
        const int rr = x / V, piece = x % V, row = quarter * 32 + rr;
        if (row < rows)
          *reinterpret_cast<uint4*>(dst.at(t.r.first + r0 + row, head) + (KEYS ? 0 : w * W) + piece * 8) =
              *reinterpret_cast<const uint4*>(stage + rr * W * 2 + ((piece ^ (rr & (V < 8 ? V - 1 : 7))) * 16));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*reinterpret_cast<volatile unsigned int*>(&g_abort_epoch) == epoch) {
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

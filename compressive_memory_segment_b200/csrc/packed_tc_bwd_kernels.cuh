// Causal softmax attention over packed sequences on the tensor cores (bf16, d =
// 64 or 128): gradients.
//
// One kernel for both sides. A CTA keeps 128 rows X, Y and streams 128-row tiles
// A, B of the other side:
//   dq     (KEYS = false): X = Q, Y = dout of one head;   A = K, B = V
//   dk, dv (KEYS = true):  X = K, Y = V of one key head;  A = Q, B = dout, query
//          tile after query tile and head after head of the group
//   S = X A^T, E = Y B^T;  p = exp(scale S - lse), ds = p (E - D);
//   acc += ds A (dq or dk, scaled at the end), acc2 += p B (dv)
// Every sum has one order (no atomics); the price is that S and E are formed
// twice, once for each side: 7 products instead of 5.
//
// 128 x 128 products: their operands come from shared memory at the rate that
// the tensor cores use them (64 cycles for 16 of k), while 64-column ones took
// the same 64 cycles for half the work. All 256 threads work on one tile (a row's
// two halves of the columns), and the two halves of their work alternate with the
// tensor cores':
//   dk, dv: exponentials of tile i under dk of i - 1 and E of i (1024 cycles at
//           d = 128), ds of tile i under dv of i and S of i + 1 (1024);
//   dq:     exponentials under dq of i - 1 and E of i, ds under S of i + 1 or i + 2
//           (dv has no accumulator here, so S has two buffers).
// Measured on 6 sequences of 200-2048, 16 / 4 heads, d = 128: dk, dv 152 us (about
// 3300 cycles a tile against 2048 of products: the exponentials' half waits for lse
// from shared memory that the products are reading), dq 117 us.
// p and ds go back to TMEM as bf16 over S and E and are the A operand of the
// accumulating products.
//
// dk, dv of a group of two or more heads: two CTAs (a cluster) share the heads,
// since one key tile's work (all its queries times all heads) would else be the
// kernel's tail. Each then hands the other one of its sums through distributed
// shared memory: the first CTA finishes dk, the second dv, in one order of adding.
//
// Rows of A and B behind the sequence are zeroed in shared memory (they meet
// zeros of p and ds, and 0 x NaN is NaN).
//
// warps 0-3, 4-7  columns 0-63, 64-127 of a tile;  warp 8  MMA issuer;  warp 9  TMA producer
// TMEM: S 0-127, E 128-255, acc 256 (D columns), then acc2 (D) or the second S.
#pragma once

#include "packed_tc_kernels.cuh"

namespace infini {
namespace tc {

constexpr int kPbThreads = 320;

template <int D>
struct PkBwd {
  static constexpr uint32_t kTileBytes = D / 64 * kHalf;             // a 128 x D tile
  static constexpr int kStages = 5;                                  // ring of tiles: A, B, A, B, ..
  static constexpr uint32_t kLd = 2 * kTile * 4;                     // lse | D of 128 queries, two of these
  static constexpr uint32_t kSmem = (2 + kStages) * kTileBytes + 2 * kLd + 256;
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr uint32_t kColE = 128, kColAcc = 256, kColAcc2 = 256 + D, kColS1 = 384;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// 16 bytes into the same place of another CTA's shared memory.
__device__ __forceinline__ void store_remote4(uint32_t at, uint32_t rank, const uint32_t* v) {
  uint32_t to;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// Announces bytes without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// A load from shared memory that stays where it is written.
__device__ __forceinline__ float4 ld4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(p)) : "memory");
  return v;
}

// 2^x for two x on the multiply-add pipes, beside the exponential unit (16 a
// cycle and SM; dk, dv 158 -> 152 us with a quarter of them here): x = n + f with n = round(x) by adding 1.5
// 2^23 (Cody and Waite's reduction), 2^f on [-1/2, 1/2] by the polynomial of degree
// 4 with the least relative error (Remez exchange; 2.7e-6 in fp32 arithmetic,
// against 2^-9 of the rounding of p and ds that follows), times 2^n. x is taken as
// at least -125. A NaN stays one: the bound and the last product keep it (adding n to
// the exponent of a NaN's bits would not).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void exp2_poly(uint64_t x2, float& e0, float& e1) {
  float x0, x1, r0, r1;
  unpack_f32x2(x2, x0, x1);
  x2 = f32x2(max_nan(x0, -125.f), max_nan(x1, -125.f));
  const uint64_t r2 = add_f32x2(x2, f32x2(12582912.f, 12582912.f));
  const uint64_t n2 = add_f32x2(r2, f32x2(-12582912.f, -12582912.f));
  const uint64_t f2 = fma_f32x2(n2, f32x2(-1.f, -1.f), x2);
  uint64_t p2 = f32x2(0.009570102207362652f, 0.009570102207362652f);
  p2 = fma_f32x2(p2, f2, f32x2(0.05591785907745361f, 0.05591785907745361f));
  p2 = fma_f32x2(p2, f2, f32x2(0.240247443318367f, 0.240247443318367f));
  p2 = fma_f32x2(p2, f2, f32x2(0.6931217908859253f, 0.6931217908859253f));
  p2 = fma_f32x2(p2, f2, f32x2(0.9999992847442627f, 0.9999992847442627f));
  unpack_f32x2(r2, r0, r1);
  // The low bits of r are n: 2^n by its exponent field.
  const float n0 = __uint_as_float((__float_as_uint(r0) << 23) + 0x3f800000u);
  const float n1 = __uint_as_float((__float_as_uint(r1) << 23) + 0x3f800000u);
  unpack_f32x2(fma_f32x2(p2, f32x2(n0, n1), f32x2(-0.f, -0.f)), e0, e1);
}
// Which pairs of a row's columns go there: 2 of 8.
__device__ __forceinline__ constexpr bool on_poly(int c) { return ((c >> 1) & 3) == 3; }

// PAIR (KEYS only): launched in clusters of two.
template <int D, bool KEYS, bool PAIR>
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
  uint8_t* sY = smem_raw + C::kTileBytes;
  uint8_t* tiles = smem_raw + 2 * C::kTileBytes;                                      // [kStages]
  float* rows_ld = reinterpret_cast<float*>(tiles + C::kStages * C::kTileBytes);  // [2][lse | D][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(rows_ld + 2 * 2 * kTile);
  uint64_t* fix_full = bars;
  uint64_t* full = bars + 1;              // [kStages]
  uint64_t* tail = full + C::kStages;     // the two tiles that end behind their sequence have landed
  uint64_t* empty = tail + 1;             // [kStages]
  uint64_t* s_full = empty + C::kStages;  // [2] S done (dk, dv: the first only)
  uint64_t* e_full = s_full + 2;          // E done
  uint64_t* p_ready = e_full + 1;         // p written (dk, dv), one arrival per warp
  uint64_t* d_ready = p_ready + 1;        // ds written
  uint64_t* fin = d_ready + 1;            // every product done
  uint64_t* drain = fin + 1;
  constexpr int kBars = 9 + 2 * C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  static_assert(kBars * 8 + 8 <= 256, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned heads = KEYS ? a.Hkv : a.Hq;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const unsigned unit = PAIR ? blockIdx.x / 2 : blockIdx.x;
  const int head_ = (int)(unit % heads);  // the output's
  const int64_t place = unit / heads;
  // Query heads of the group that this CTA takes.
  const int g_first = PAIR && rank ? (a.G + 1) / 2 : 0, g_n = !KEYS ? 1 : PAIR ? (rank ? a.G / 2 : (a.G + 1) / 2) : a.G;
  SlotTile t;
  // dk, dv: few and unequal units, most work first; dq has one for each head and
  // query tile, the later tiles of a sequence first (121 us by work, 118 so).
  if (!(KEYS ? work_tile<kTile, false>(a.sk, a.sq, place, slots, &t) : slot_tile<kTile>(a.sq, a.sk, slots - 1 - place, &t)))
    return;
  const SeqRange other = t.other;
  const int nq = KEYS ? other.len : t.r.len, nk = KEYS ? t.r.len : other.len, shift = nk - nq;
  const int r0 = t.tile * kTile, rows = min(kTile, t.r.len - r0);
  // Streamed rows: keys up to the last row's, or queries from the first that
  // sees key r0; whole tiles from a multiple of 128.
  const int first = KEYS ? min(nq, max(0, r0 - shift)) / kTile * kTile : 0;
  const int end = KEYS ? nq : max(0, min(nk, r0 + rows + shift));
  const int per_head = end > first ? (end - first + kTile - 1) / kTile : 0;
  const int n = per_head * g_n;
  const int limit = KEYS ? nq : nk;   // rows of the streamed side that exist

  if (threadIdx.x == 0) {
    for (int b = 0; b < kBars; ++b) mbar_init(&bars[b], &bars[b] == p_ready || &bars[b] == d_ready ? 8 : 1);
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
        mbar_arrive_expect_tx(fix_full, 2 * C::kTileBytes);
        load_rows<D, kTile>(sX, &tmX, head_, row, fix_full);
        load_rows<D, kTile>(sY, &tmY, head_, row, fix_full);
      }
      __syncwarp();
      int tails = 0;
      for (int i = 0; i < n && ok; ++i) {
        const int ga = 2 * i, gb = 2 * i + 1;
        const int g = KEYS ? i / per_head : 0, c0 = first + (i - g * per_head) * kTile;
        const int h = KEYS ? head_ * a.G + g_first + g : head_ / a.G;  // head of the streamed rows
        const int valid = limit - c0;
        float le[4], de[4];
        if (KEYS) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int q = c0 + lane + 32 * x;
            const int64_t at = (int64_t)h * a.sq.T + other.first + q;
            le[x] = q < nq ? a.lse[at] * 1.4426950408889634f : 0.f;
            de[x] = q < nq ? a.delta[at] : 0.f;
          }
        }
        const bool cut = valid < kTile;
        uint8_t* sa = tiles + ga % C::kStages * C::kTileBytes;
        uint8_t* sb = tiles + gb % C::kStages * C::kTileBytes;
        uint64_t *full_a = &full[ga % C::kStages], *full_b = &full[gb % C::kStages];
        if (ga >= C::kStages && !(ok = mbar_wait_warp(&empty[ga % C::kStages], (ga / C::kStages - 1) & 1, epoch))) break;
        armed |= 1u << ((cut ? tail : full_a) - bars);
        if (elect_one_lane()) {
          if (cut)
            mbar_arrive_expect_tx(tail, 2 * C::kTileBytes);
          else
            mbar_expect_tx(full_a, C::kTileBytes);  // the arrival follows lse and D
          load_rows<D, kTile>(sa, &tmA, h, other.first + c0, cut ? tail : full_a);
        }
        __syncwarp();
        if (gb >= C::kStages && !(ok = mbar_wait_warp(&empty[gb % C::kStages], (gb / C::kStages - 1) & 1, epoch))) break;
        if (!cut) armed |= 1u << (full_b - bars);
        if (elect_one_lane()) {
          if (!cut) mbar_arrive_expect_tx(full_b, C::kTileBytes);
          load_rows<D, kTile>(sb, &tmB, h, other.first + c0, cut ? tail : full_b);
        }
        __syncwarp();
        if (KEYS) {
          // Tile gb's place was A of i - 2 (five places), whose last product
          // came after the threads had read lse and D of i - 2.
          float* ld = rows_ld + (i & 1) * 2 * kTile;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            ld[lane + 32 * x] = le[x];
            ld[kTile + lane + 32 * x] = de[x];
          }
        }
        if (cut) {
          if (!(ok = mbar_wait_warp(tail, tails & 1, epoch))) break;
          ++tails;
          zero_rows<D, kTile>(sa, valid, lane);
          zero_rows<D, kTile>(sb, valid, lane);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (elect_one_lane()) {
          mbar_arrive(full_a);
          if (cut) mbar_arrive(full_b);
        }
        __syncwarp();
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false), id_acc = idesc_bf16_f32(128, D, false, true);
      const uint64_t x0 = desc_kmajor_sw128(smem_u32(sX)), y0 = desc_kmajor_sw128(smem_u32(sY)),
                     t0 = desc_kmajor_sw128(smem_u32(tiles)), m0 = desc_mnmajor_sw128(smem_u32(tiles), kHalf);
      auto place = [&](int g) { return (uint32_t)(g % C::kStages * C::kTileBytes) >> 4; };
      auto there = [&](int g) { return mbar_wait(&full[g % C::kStages], (g / C::kStages) & 1, epoch); };
      auto scores = [&](int i) {  // S of tile i
        if (!there(2 * i)) return false;
        const uint32_t col = !KEYS && (i & 1) ? C::kColS1 : 0;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(tmem + col, x0 + kmaj_step(kk), t0 + place(2 * i) + kmaj_step(kk), id_s, kk != 0);
        mma_commit(&s_full[KEYS ? 0 : i & 1]);
        return true;
      };
      auto grads = [&](int i) {  // E of tile i
        if (!there(2 * i + 1)) return false;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(tmem + C::kColE, y0 + kmaj_step(kk), t0 + place(2 * i + 1) + kmaj_step(kk), id_s, kk != 0);
        mma_commit(e_full);
        if (!KEYS) mma_commit(&empty[(2 * i + 1) % C::kStages]);  // V is done with
        return true;
      };
      ok = mbar_wait(fix_full, 0, epoch) && scores(0) && grads(0) && (KEYS || n < 2 || scores(1));
      for (int i = 0; i < n && ok; ++i) {
        if (KEYS) {
          if (!(ok = mbar_wait(p_ready, i & 1, epoch))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_bf16_ts(tmem + C::kColAcc2, tmem + packed_a_col(kk), m0 + place(2 * i + 1) + mnmaj_step(kk), id_acc,
                        (i | kk) != 0);
          mma_commit(&empty[(2 * i + 1) % C::kStages]);  // dout is done with
          if (i + 1 < n && !(ok = scores(i + 1))) break;
        }
        if (!(ok = mbar_wait(d_ready, i & 1, epoch))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_bf16_ts(tmem + C::kColAcc, tmem + C::kColE + packed_a_col(kk), m0 + place(2 * i) + mnmaj_step(kk), id_acc,
                      (i | kk) != 0);
        mma_commit(&empty[2 * i % C::kStages]);
        if (i + 1 < n) ok = grads(i + 1);
        if (ok && !KEYS && i + 2 < n) ok = scores(i + 2);
      }
      if (ok) mma_commit(fin);
    }
  } else {
    // ------------------------------------------------ thread = row of X, half of the columns
    const int w = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t te = tmem + C::kColE + w * 64 + lanes;
    const float scale2 = a.scale * 1.4426950408889634f;
    float lse = 0.f, dlt = 0.f;
    if (!KEYS && r < rows) {
      const int64_t at = (int64_t)head_ * a.sq.T + t.r.first + r0 + r;
      lse = a.lse[at] * 1.4426950408889634f;
      dlt = a.delta[at];
    }
    for (int i = 0; i < n; ++i) {
      const int c0 = first + (KEYS ? i % per_head : i) * kTile;
      const uint32_t ts = tmem + (!KEYS && (i & 1) ? C::kColS1 : 0) + w * 64 + lanes;
      // While the products read shared memory at its full rate a load from it
      // takes some 800 cycles: all of lse (and of D below) at once, ahead of the wait.
      const float* ld = rows_ld + (i & 1) * 2 * kTile + 64 * w;
      float4 row[KEYS ? 16 : 1];
      if (KEYS) {
        if (!(ok = mbar_wait_warp(&full[2 * i % C::kStages], (2 * i / C::kStages) & 1, epoch))) break;
#pragma unroll
        for (int c = 0; c < 16; ++c) row[KEYS ? c : 0] = ld4(ld + 4 * c);
      }
      if (!(ok = KEYS ? mbar_wait_warp(&s_full[0], i & 1, epoch) : mbar_wait_warp(&s_full[i & 1], (i >> 1) & 1, epoch)))
        break;
      tc_fence_after();
      // Columns that row r takes part in: [lo, hi) of this thread's 64.
      const bool cut = KEYS ? c0 + shift < r0 + kTile - 1 || c0 + kTile > nq
                            : c0 + kTile - 1 > r0 + shift || c0 + kTile > nk;
      const int lo = KEYS ? r0 + r - shift - c0 - 64 * w : 0;
      const int hi = (KEYS ? nq - c0 : min(nk, r0 + r + shift + 1) - c0) - 64 * w;
      uint32_t s[64];  // scores, then p
      tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      tmem_ld32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
      tmem_ld_wait_regs(s);
      const uint64_t sc2 = f32x2(scale2, scale2);
#pragma unroll
      for (int c = 0; c < 64; c += 2) {
        const float4 l4 = KEYS ? row[KEYS ? c / 4 : 0] : make_float4(lse, lse, lse, lse);
        const uint64_t x2 = fma_f32x2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2,
                                      c & 2 ? f32x2(-l4.z, -l4.w) : f32x2(-l4.x, -l4.y));
        float p0, p1;
        if (on_poly(c)) {
          exp2_poly(x2, p0, p1);
        } else {
          unpack_f32x2(x2, p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
        }
        s[c] = __float_as_uint(p0);
        s[c + 1] = __float_as_uint(p1);
      }
      if (cut) {  // (scores there may be anything)
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < lo || c >= hi) s[c] = 0u;
      }
      if (KEYS) {
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            pk[c] = pack_bf16x2(__uint_as_float(s[32 * ch + 2 * c]), __uint_as_float(s[32 * ch + 2 * c + 1]));
          tmem_st16(ts + 16 * ch, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
      if (KEYS) {
#pragma unroll
        for (int c = 0; c < 16; ++c) row[KEYS ? c : 0] = ld4(ld + kTile + 4 * c);
      }
      if (!(ok = mbar_wait_warp(e_full, i & 1, epoch))) break;
      tc_fence_after();
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t e[32], dk[16];
        tmem_ld32(te + 32 * ch, e);
        tmem_ld_wait_regs(e);
        if (cut) {  // E may be anything there
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (32 * ch + c < lo || 32 * ch + c >= hi) e[c] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 d4 = KEYS ? row[KEYS ? 8 * ch + c / 4 : 0] : make_float4(dlt, dlt, dlt, dlt);
          const float dv[4] = {d4.x, d4.y, d4.z, d4.w};
          float d[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            d[x] = __uint_as_float(s[32 * ch + c + x]) * (__uint_as_float(e[c + x]) - dv[x]);
          dk[c / 2] = pack_bf16x2(d[0], d[1]);
          dk[c / 2 + 1] = pack_bf16x2(d[2], d[3]);
        }
        // Column 16 ch of this half of E has been read by now: 32 ch covers it.
        tmem_st16(te + 16 * ch, dk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(d_ready);
    }
    if (ok && n > 0 && (ok = mbar_wait_warp(fin, 0, epoch))) tc_fence_after();
  }
  if constexpr (PAIR) {
    // The sums that the other CTA finishes go into its ring, [column / 4][row]
    // of 16 bytes; both rings are free behind the first barrier. Every thread of
    // both CTAs comes to both barriers, also after a wait that gave up.
    static_assert(KEYS && C::kStages * C::kTileBytes >= kTile * D * 4, "room for one sum");
    __syncwarp();
    cluster_sync_all();
    const int w = warp >> 2;
    if (warp < 8 && ok && w != (int)rank) {
      const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (w ? C::kColAcc2 : C::kColAcc);
      const uint32_t to = smem_u32(tiles) + ((warp & 3) * 32 + lane) * 16;
#pragma unroll
      for (int cb = 0; cb < D; cb += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(from + cb, o);
          tmem_ld_wait_regs(o);
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0u;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) store_remote4(to + (cb / 4 + x) * kTile * 16, rank ^ 1u, o + 4 * x);
      }
    }
    cluster_sync_all();
  }
  if (warp < 8 && ok && (!PAIR || (warp >> 2) == (int)rank)) {
    const int w = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // Warps 0-3 write dk (or the first half of dq's columns), warps 4-7 dv (or
    // the second half), whole rows through shared memory.
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
      if constexpr (PAIR) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float4 add = *reinterpret_cast<const float4*>(tiles + ((cb / 4 + x) * kTile + quarter * 32 + lane) * 16);
          o[4 * x] = __float_as_uint(__uint_as_float(o[4 * x]) + add.x);
          o[4 * x + 1] = __float_as_uint(__uint_as_float(o[4 * x + 1]) + add.y);
          o[4 * x + 2] = __float_as_uint(__uint_as_float(o[4 * x + 2]) + add.z);
          o[4 * x + 3] = __float_as_uint(__uint_as_float(o[4 * x + 3]) + add.w);
        }
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
        *reinterpret_cast<uint4*>(dst.at(t.r.first + r0 + row, head_) + (KEYS ? 0 : w * W) + piece * 8) =
            *reinterpret_cast<const uint4*>(stage + rr * W * 2 + ((piece ^ (rr & (V < 8 ? V - 1 : 7))) * 16));
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

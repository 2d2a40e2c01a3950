// Host side of include/infini_attn_packed.h: argument checks, workspace
// layouts, choice of path and launches. Included by infini_attn.cu, whose
// helpers (round_up, aligned16, overlap, allow_smem) it uses.
#pragma once

#include <cmath>

#include "../../include/infini_attn_packed.h"
#include "packed_common.cuh"
#include "packed_simt_kernels.cuh"
#include "packed_split_kernels.cuh"
#include "packed_tc_kernels.cuh"
#include "packed_tc_bwd_kernels.cuh"
#include "delta_common.cuh"
#include "delta_simt_kernels.cuh"
#include "delta_chunk_kernels.cuh"

namespace {

constexpr int64_t kMaxGridY = 65535;

// Size of a workspace that holds `bytes`: always above kWsAlign, which stands
// for a call that needs none (and may be given none).
size_t scratch(size_t bytes) { return round_up(bytes, kWsAlign) + kWsAlign; }

// What a call reads or writes: rows of a tensor, or a flat array (st = 0).
struct Region {
  const char* p;
  int64_t bytes;                 // from p to the end of the last element
  int64_t st, sh;                // steps of a token and of a head
  int64_t piece, heads, tokens;  // bytes of one row, spans of a token's heads and of a head's tokens
  bool written;
};

Region flat(const void* p, int64_t bytes, bool written) {
  return {static_cast<const char*>(p), p ? bytes : 0, 0, 0, 0, 0, 0, written};
}

// a lies in the first wa bytes of every `step` from its start, b in the first wb from its own: never the same ones.
bool apart(const Region& a, const Region& b, int64_t step, int64_t wa, int64_t wb) {
  if (wa > step || wb > step) return false;
  int64_t gap = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % step;
  if (gap < 0) gap += step;
  return gap >= wa && gap + wb <= step;
}

// Two regions share a byte. Views that interleave do not: by tokens ([T][n][H][d],
// the same step over the tokens), by heads ([H][n][T][d]) or row by row ([T][H][n][d]
// and [H][T][n][d], the larger steps multiples of a common smallest one).
bool share(const Region& a, const Region& b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  if (!overlap(a.p, (size_t)a.bytes, b.p, (size_t)b.bytes)) return false;
  if (a.st > 0 && b.st > 0) {
    if (a.st == b.st && apart(a, b, a.st, a.heads, b.heads)) return false;
    if (a.sh == b.sh && apart(a, b, a.sh, a.tokens, b.tokens)) return false;
    const int64_t m = std::min(a.st, a.sh);
    if (m == std::min(b.st, b.sh) && a.st % m == 0 && a.sh % m == 0 && b.st % m == 0 && b.sh % m == 0 &&
        apart(a, b, m, a.piece, b.piece))
      return false;
  }
  return true;
}

int check_alias(const Region* r, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((r[i].written || r[j].written) && share(r[i], r[j])) return INFINI_ERR_ALIAS;
  return INFINI_OK;
}

// Checked rows and how many there are.
struct Rows : infini_rows {
  int64_t n, heads;
};

// Checks rows [T][H][d] of elt-byte elements at a 16-byte granularity (d = 1:
// single elements) and appends their region. The stride of a dimension of size
// 1 is replaced by the packed one.
int take_rows(const infini_rows* x, int64_t T, int64_t H, int64_t d, int64_t elt, bool written, Rows* y, Region* reg) {
  if (!x) return INFINI_ERR_NULL;
  *y = {*x, T, H};
  if (T > 0 && !x->ptr) return INFINI_ERR_NULL;
  if (H == 1) y->stride_h = d;
  if (T <= 1) y->stride_t = H == 1 ? d : y->stride_h * H;
  constexpr int64_t kMost = int64_t(1) << 38;
  if (y->stride_h < 1 || y->stride_t < 1 || y->stride_h > kMost || y->stride_t > kMost) return INFINI_ERR_SHAPE;
  const int64_t grain = d == 1 ? 1 : 16 / elt;
  if (y->stride_h % grain || y->stride_t % grain) return INFINI_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(x->ptr) % (d == 1 ? (size_t)elt : 16u)) return INFINI_ERR_ALIGN;
  const int64_t width = (H - 1) * y->stride_h + d;
  // An extent that no address space holds would wrap in the sums below.
  if (T > 0 && ((__int128)(T - 1) * y->stride_t + width) * elt > ((__int128)1 << 48)) return INFINI_ERR_SIZE;
  if (written && T > 0) {  // its own rows may not overlap
    const bool token_major = y->stride_h >= d && y->stride_t >= width;
    const bool head_major = y->stride_t >= d && y->stride_h >= (T - 1) * y->stride_t + d;
    if (!token_major && !head_major) return INFINI_ERR_ALIAS;
  }
  reg->p = static_cast<const char*>(x->ptr);
  reg->bytes = T > 0 ? ((T - 1) * y->stride_t + width) * elt : 0;
  reg->st = y->stride_t * elt;
  reg->sh = y->stride_h * elt;
  reg->piece = d * elt;
  reg->heads = width * elt;
  reg->tokens = T > 0 ? ((T - 1) * y->stride_t + d) * elt : 0;
  reg->written = written;
  return INFINI_OK;
}

template <typename T>
infini::RowsOf<T> rows_of(const Rows& x) {
#ifdef INFINI_DEBUG
  return {static_cast<T*>(x.ptr), x.stride_t, x.stride_h, x.n, (int)x.heads};
#else
  return {static_cast<T*>(x.ptr), x.stride_t, x.stride_h};
#endif
}

// ------------------------------------------------------------------ attention
int check_packed(const infini_packed_shape* s) {
  if (!s) return INFINI_ERR_NULL;
  if (s->n_seq < 0 || s->Tq < 0 || s->Tk < 0 || s->Hq < 1 || s->Hkv < 1 || s->Hq % s->Hkv != 0 || s->max_q < 0 ||
      s->max_k < 0)
    return INFINI_ERR_SHAPE;
  if (s->d != 64 && s->d != 128) return INFINI_ERR_UNSUPPORTED;
  if (s->dtype != INFINI_F32 && s->dtype != INFINI_BF16) return INFINI_ERR_UNSUPPORTED;
  if (!std::isfinite(s->scale) || !(s->scale > 0.f)) return INFINI_ERR_UNSUPPORTED;
  // Rows and slots are 32-bit inside the kernels; one CTA for each (slot, head).
  if (s->Tq >= (int64_t(1) << 30) || s->Tk >= (int64_t(1) << 30) || s->n_seq >= (int64_t(1) << 24) ||
      s->Hq > kMaxGridY || s->Tq * s->Hq >= (int64_t(1) << 33))
    return INFINI_ERR_SIZE;
  if (infini::slot_count(s->Tq, s->n_seq, infini::kPsRows) * s->Hq >= (int64_t(1) << 31) ||
      infini::slot_count(s->Tk, s->n_seq, infini::kPsRows) * s->Hkv >= (int64_t(1) << 31))
    return INFINI_ERR_SIZE;
  return INFINI_OK;
}

bool packed_tc_covers(const infini_packed_shape* s) {
  // Two CTAs for each (slot, key head) at most, beyond what every path needs; a tensor map has rows.
  return s->dtype == INFINI_BF16 && s->Tk > 0 && s->Tq > 0 &&
         infini::slot_count(s->Tk, s->n_seq, infini::tc::kTile) * s->Hkv * 2 < (int64_t(1) << 31);
}

// The caller's longest sequence, cut to what the sizes allow: any figure may be given.
int64_t longest(int64_t n) { return std::max<int64_t>(1, std::min(n, int64_t(1) << 30)); }

// Chunks of keys: enough CTAs for about eight to an SM, none under 256 keys.
infini::SplitShape split_shape(const infini_packed_shape* s) {
  const int64_t rows = longest(s->max_q) * (s->Hq / s->Hkv);
  const int64_t per = s->dtype == INFINI_BF16 ? infini::kSmRows : infini::kSplitRows;
  const int64_t z = std::min<int64_t>(64, (rows + per - 1) / per);
  // (beyond the CTAs asked for one chunk holds all keys)
  const int64_t ctas = std::min<int64_t>(148 * 8, std::max<int64_t>(1, s->n_seq * s->Hkv) * z);
  const int64_t keys = longest(s->max_k);
  int64_t chunk = (keys * ctas + 148 * 8 - 1) / (148 * 8);
  chunk = std::max<int64_t>(256, (chunk + 63) / 64 * 64);
  chunk = std::min<int64_t>(chunk, int64_t(1) << 24);
  const int64_t n = std::min<int64_t>((keys + chunk - 1) / chunk, 4096);
  return {(int)chunk, (int)n};
}

// One CTA for each (chunk, sequence, key head); rows of a key head are counted in
// 32 bits, and a CTA's next rows, up to 64 x 16 further on, are too.
bool packed_split_fits(const infini_packed_shape* s) {
  return s->n_seq * s->Hkv * split_shape(s).n_chunks < (int64_t(1) << 31) &&
         s->Tq * (s->Hq / s->Hkv) < (int64_t(1) << 31) - 64 * infini::kSmRows;
}

// Few rows for each key head (queries times heads of the group) go to the split
// kernels, which read a key head's keys once for every 16 (fp32: 4) of its rows;
// the other paths read them once for every 256 (fp32: 32) rows of one query head,
// by as many CTAs. While the GPU is full a share of the split kernel's costs about as
// much as 0.8 (bf16, d = 128), 0.57 (bf16, d = 64) or 0.67 (fp32) of the others' CTA,
// and below that many CTAs the others leave SMs idle however many keys there are. us,
// split against tensor-core path (bf16) or CUDA cores (fp32), by sequences, query / key
// heads, d, queries, keys:
//   bf16  48, 32 / 8, 128, 1, 4096: 133 / 579;  16 queries 514 / 635;  64 queries 1977 / 654
//         256, 8 / 8, 64, 16, 16: 40 / 61;  32, 32: 70 / 61;  64, 512: 260 / 117
//         2000, 4 / 2, 64, 20, 20: 170 / 205;  256, 16 / 1, 128, 4, 512: 77 / 236
//         1, 32 / 8, 128, 1, 8192: 21 / 109;  16 queries 43 / 109;  64 queries 87 / 110
//   fp32  256, 32 / 8, 128, 1, 512: 369 / 2341;  4, 4: 121 / 212;  8, 8: 258 / 236;
//         16, 512: 5660 / 2405;  256, 8 / 8, 64, 64, 512: 2759 / 569
//         1, 32 / 8, 128, 16, 512: 24 / 59;  1, 8 / 8, 64, 64, 512: 22 / 34
constexpr int64_t kSplitMostRows = 64;
bool packed_few_rows(const infini_packed_shape* s) {
  const bool bf16 = s->dtype == INFINI_BF16;
  const int64_t rows = longest(s->max_q) * (s->Hq / s->Hkv);
  if (rows > kSplitMostRows || !packed_split_fits(s)) return false;
  const int64_t per = bf16 ? infini::kSmRows : infini::kSplitRows, other = bf16 ? infini::tc::kPkRows : infini::kPsRows;
  const int64_t shares = s->n_seq * s->Hkv * ((rows + per - 1) / per);
  const int64_t ctas = s->n_seq * s->Hq * ((longest(s->max_q) + other - 1) / other);
  return 4 * shares <= (!bf16 ? 6 : s->d == 64 ? 7 : 5) * std::max<int64_t>(148, ctas);
}
int packed_auto(const infini_packed_shape* s) {
  if (packed_few_rows(s)) return INFINI_PATH_SPLIT;
  return packed_tc_covers(s) ? (int)INFINI_PATH_TC : (int)INFINI_PATH_SIMT;
}

// The tensor-core forward takes its units by work, over all sequences, while
// their keys and values fit L2 (126 MB) with room to spare; beyond, by slots, so
// that neighbouring tiles of one sequence read its keys together. Called again and
// again on changing inputs, by slots / by work, MB of keys and values: 13 MB 83 / 69 us
// (6 sequences of up to 2048, 16 / 4 heads, d = 128), 50 MB 342 / 306 (4 of 8192, 8
// heads, d = 64), 61 MB 153 / 142 (16 of 2048, 16 / 8 heads), 78 MB 284 / 279 (16 of
// 2048, 32 / 16 heads, d = 64), 84 MB 109 / 105 (12 of 2048, 16 heads), 95 MB 92 / 92
// (20 of 1024, 16 heads), 105 MB 1378 / 1420 (6 of 8192, 32 / 8 heads), 129 MB 164 /
// 168 (12 of 2048, 16 heads), 142 MB 178 / 183 (30 of 2048, 8 heads), 164 MB 220 / 234
// (16 of 2048, 16 heads). The rows of the tensor count, not the lengths, which the
// host does not know.
bool packed_by_work(const infini_packed_shape* s) {
  return (size_t)s->Tk * s->Hkv * s->d * 4 <= ((size_t)96 << 20);
}

int packed_resolve(const infini_packed_shape* s, int path, bool backward) {
  if (path == INFINI_PATH_AUTO)
    return !backward ? packed_auto(s) : packed_tc_covers(s) ? (int)INFINI_PATH_TC : (int)INFINI_PATH_SIMT;
  if (path == INFINI_PATH_SIMT) return path;
  if (path == INFINI_PATH_TC && packed_tc_covers(s)) return path;
  if (path == INFINI_PATH_SPLIT && !backward && packed_split_fits(s)) return path;
  return INFINI_ERR_UNSUPPORTED;
}

size_t packed_ws(const infini_packed_shape* s, int path) {
  if (path != INFINI_PATH_SPLIT) return kWsAlign;
  const infini::SplitShape p = split_shape(s);
  return scratch((size_t)s->Tq * s->Hq * p.n_chunks * (s->d + 2) * 4);
}

// Rows [T][H][d] as a tensor map with boxes of 64 elements x 1 head x `rows`
// tokens, 128-byte swizzle; what lies behind the last token reads as zero.
template <typename T>
bool make_rows_map(CUtensorMap* m, const infini::RowsOf<T>& x, int64_t n, int64_t H, int64_t d, int rows) {
  auto enc = infini::tc::tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)n};
  cuuint64_t strides[2] = {(cuuint64_t)x.sh * 2, (cuuint64_t)x.st * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(x.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_packed_report(const infini::SeqTable& q, const infini::SeqTable& k, cudaStream_t st) {
  infini::packed_report_kernel<<<(unsigned)std::min<int64_t>(((int64_t)q.n_seq + 255) / 256, 148), 256, 0, st>>>(q, k);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <int D>
int launch_packed_tc_forward(const infini_packed_shape* s, const infini::PackedArgs<__nv_bfloat16>& a,
                             cudaStream_t st) {
  using namespace infini;
  CUtensorMap mq, mk, mv;
  if (!make_rows_map(&mq, a.q, s->Tq, s->Hq, D, tc::kTile) || !make_rows_map(&mk, a.k, s->Tk, s->Hkv, D, tc::kTile) ||
      !make_rows_map(&mv, a.v, s->Tk, s->Hkv, D, tc::kTile))
    return INFINI_ERR_CUDA;
  constexpr size_t smem = tc::PkFwd<D>::kSmem;
  if (allow_smem(tc::packed_tc_fwd_kernel<D>, smem) != cudaSuccess) return INFINI_ERR_CUDA;
  if (!a.by_work || s->n_seq > 32) {
    const int rc = launch_packed_report(a.sq, a.sk, st);
    if (rc != INFINI_OK) return rc;
  }
  const int64_t slots = slot_count(s->Tq, s->n_seq, tc::kPkRows);
  tc::packed_tc_fwd_kernel<D><<<(unsigned)(slots * s->Hq), tc::kPkThreads, smem, st>>>(mq, mk, mv, a, slots,
                                                                                     next_epoch());
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <typename T, int D>
int launch_packed_forward(const infini_packed_shape* s, const infini::PackedArgs<T>& a, int path, char* ws,
                          cudaStream_t st) {
  using namespace infini;
  if (path == INFINI_PATH_SPLIT) {
    const SplitShape p = split_shape(s);
    const int64_t rows = longest(s->max_q) * a.G;
    constexpr int per = sizeof(T) == 2 ? kSmRows : kSplitRows;
    const unsigned z = (unsigned)std::min<int64_t>(64, (rows + per - 1) / per);
    const dim3 grid((unsigned)(p.n_chunks * s->n_seq * s->Hkv), 1, z);
    float* part = reinterpret_cast<float*>(ws);
    if constexpr (sizeof(T) == 2) {
      constexpr size_t smem = SplitMma<D>::kTotal;
      if (allow_smem(packed_split_mma_kernel<D>, smem) != cudaSuccess) return INFINI_ERR_CUDA;
      packed_split_mma_kernel<D><<<grid, kSmThreads, smem, st>>>(a, p, part);
    } else {
      constexpr size_t smem = (size_t)(kSplitThreads / 8) * kSplitRows * (D + 2) * 4;
      packed_split_kernel<T, D><<<grid, kSplitThreads, smem, st>>>(a, p, part);
    }
    if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
    const unsigned jx = (unsigned)std::min<int64_t>(1024, (longest(s->max_q) * s->Hq + 3) / 4);
    packed_split_join_kernel<T, D><<<dim3((unsigned)s->n_seq, jx), 128, 0, st>>>(a, p, part);
    return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
  }
  if constexpr (sizeof(T) == 2)
    if (path == INFINI_PATH_TC) return launch_packed_tc_forward<D>(s, a, st);
  constexpr size_t smem = ps_fwd_smem<D>();
  if (allow_smem(packed_simt_fwd_kernel<T, D>, smem) != cudaSuccess) return INFINI_ERR_CUDA;
  if (s->n_seq > 32) {
    const int rc = launch_packed_report(a.sq, a.sk, st);
    if (rc != INFINI_OK) return rc;
  }
  const int64_t slots = slot_count(s->Tq, s->n_seq, kPsRows);
  packed_simt_fwd_kernel<T, D><<<(unsigned)(slots * s->Hq), kPsThreads, smem, st>>>(a, slots);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <int D>
int launch_packed_tc_backward(const infini_packed_shape* s, const infini::PackedGradArgs<__nv_bfloat16>& a,
                              cudaStream_t st) {
  using namespace infini;
  using K = tc::PkBwd<D>;
  CUtensorMap mq, mo, mk, mv;
  if (!make_rows_map(&mq, a.q, s->Tq, s->Hq, D, tc::kTile) || !make_rows_map(&mo, a.dout, s->Tq, s->Hq, D, tc::kTile) ||
      !make_rows_map(&mk, a.k, s->Tk, s->Hkv, D, tc::kTile) || !make_rows_map(&mv, a.v, s->Tk, s->Hkv, D, tc::kTile))
    return INFINI_ERR_CUDA;
  const uint32_t epoch = next_epoch();
  const int64_t nk = slot_count(s->Tk, s->n_seq, tc::kTile), nq = slot_count(s->Tq, s->n_seq, tc::kTile);
  if (allow_smem(tc::packed_tc_bwd_kernel<D, false, false>, K::kSmem) != cudaSuccess) return INFINI_ERR_CUDA;
  if (a.G > 1) {
    auto* fn = tc::packed_tc_bwd_kernel<D, true, true>;
    if (allow_smem(fn, K::kSmem) != cudaSuccess) return INFINI_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(nk * s->Hkv * 2));
    cfg.blockDim = dim3(tc::kPbThreads);
    cfg.dynamicSmemBytes = K::kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, mk, mv, mq, mo, a, nk, epoch) != cudaSuccess) return INFINI_ERR_CUDA;
  } else {
    auto* fn = tc::packed_tc_bwd_kernel<D, true, false>;
    if (allow_smem(fn, K::kSmem) != cudaSuccess) return INFINI_ERR_CUDA;
    fn<<<(unsigned)(nk * s->Hkv), tc::kPbThreads, K::kSmem, st>>>(mk, mv, mq, mo, a, nk, epoch);
    if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  }
  tc::packed_tc_bwd_kernel<D, false, false><<<(unsigned)(nq * s->Hq), tc::kPbThreads, K::kSmem, st>>>(mq, mo, mk, mv, a, nq,
                                                                                                     epoch);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <typename T, int D>
int launch_packed_backward(const infini_packed_shape* s, const infini::PackedGradArgs<T>& a, int path,
                           cudaStream_t st) {
  using namespace infini;
  const int64_t rows = s->Tq * s->Hq;
  if (rows > 0) {
    constexpr int per = 256 * (16 / (int)sizeof(T)) / D;  // rows of a CTA
    packed_delta_kernel<T, D><<<(unsigned)((rows + per - 1) / per), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  }
  if (s->n_seq > 32) {
    const int rc = launch_packed_report(a.sq, a.sk, st);
    if (rc != INFINI_OK) return rc;
  }
  if constexpr (sizeof(T) == 2)
    if (path == INFINI_PATH_TC) return launch_packed_tc_backward<D>(s, a, st);
  constexpr size_t smem = ps_bwd_smem<D>();
  if (allow_smem(packed_simt_bwd_kernel<T, D, false>, smem) != cudaSuccess ||
      allow_smem(packed_simt_bwd_kernel<T, D, true>, smem) != cudaSuccess)
    return INFINI_ERR_CUDA;
  const int64_t nq = slot_count(s->Tq, s->n_seq, kPsRows), nk = slot_count(s->Tk, s->n_seq, kPsRows);
  packed_simt_bwd_kernel<T, D, false><<<(unsigned)(nq * s->Hq), kPsThreads, smem, st>>>(a, nq);
  if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  packed_simt_bwd_kernel<T, D, true><<<(unsigned)(nk * s->Hkv), kPsThreads, smem, st>>>(a, nk);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

// ----------------------------------------------------------------- delta rule
int check_delta(const infini_delta_shape* s) {
  if (!s) return INFINI_ERR_NULL;
  if (s->n_seq < 0 || s->T < 0 || s->Hk < 1 || s->Hv < 1 || s->Hv % s->Hk != 0 || s->max_len < 0)
    return INFINI_ERR_SHAPE;
  if (s->d != 64 && s->d != 128) return INFINI_ERR_UNSUPPORTED;
  if (s->dtype != INFINI_F32 && s->dtype != INFINI_BF16) return INFINI_ERR_UNSUPPORTED;
  if (!std::isfinite(s->scale)) return INFINI_ERR_UNSUPPORTED;
  if (s->T >= (int64_t(1) << 30) || s->n_seq > kMaxGridY || s->Hv > kMaxGridY) return INFINI_ERR_SIZE;
  return INFINI_OK;
}

// A forward over at most 8 tokens a sequence takes the recurrence on the CUDA
// cores, where the chunked form would pay two launches and a 64-token chunk: bf16,
// d = 128, 16 heads, recurrence against chunks: 1 sequence 4.5 / 15 us (4 tokens),
// 5.8 / 15 (8), 14 / 15 (32); 64 sequences 82 / 103, 104 / 103, 258 / 105.
constexpr int64_t kDeltaFew = 8;
int delta_resolve(const infini_delta_shape* s, int path, bool few) {
  const bool tc = s->dtype == INFINI_BF16 && s->T > 0;  // a tensor map has rows
  if (path == INFINI_PATH_AUTO) return tc && !few ? (int)INFINI_PATH_TC : (int)INFINI_PATH_SIMT;
  if (path == INFINI_PATH_SIMT) return path;
  if (path == INFINI_PATH_TC && tc) return path;
  return INFINI_ERR_UNSUPPORTED;
}

// Records of the chunked path, one for each (chunk, value head).
size_t delta_records(const infini_delta_shape* s) {
  return (size_t)infini::slot_count(s->T, s->n_seq, infini::kDcTok) * s->Hv * infini::DcRecord::kBytes;
}
size_t delta_simt_records(const infini_delta_shape* s) {
  return (size_t)infini::slot_count(s->T, s->n_seq, infini::kDsChunk) * s->Hv * infini::DsChunk<64>::kRecord * 4;
}
size_t delta_fwd_ws(const infini_delta_shape* s, int path) {
  if (path == INFINI_PATH_TC) return scratch(delta_records(s));
  return s->max_len <= kDeltaFew ? kWsAlign : scratch(delta_simt_records(s));
}

struct DeltaBwdPlan {
  size_t off_kept, off_dq, off_dk, off_rec;  // CUDA cores: S at chunk starts, dq and dk per value head, records
  size_t off_S, off_dS, off_U, off_Z;   // chunked (behind the records): S, U; both: dS at chunk ends, Z
  size_t total;
};
DeltaBwdPlan delta_bwd_plan(const infini_delta_shape* s, int path) {
  DeltaBwdPlan p{};
  const size_t dd = (size_t)s->Hv * s->d * s->d, td = (size_t)s->T * s->Hv * s->d;
  if (path == INFINI_PATH_TC) {
    const size_t states = (size_t)infini::slot_count(s->T, s->n_seq, infini::kDcTok) * dd * 2;
    p.off_S = round_up(delta_records(s), kWsAlign);
    p.off_dS = round_up(p.off_S + states, kWsAlign);
    p.off_U = round_up(p.off_dS + states, kWsAlign);
    p.off_Z = round_up(p.off_U + td * 2, kWsAlign);
    p.total = scratch(p.off_Z + td * 2);
    return p;
  }
  p.off_kept = 0;
  const size_t states = (size_t)infini::slot_count(s->T, s->n_seq, infini::kDsChunk) * dd * 4;
  p.off_dS = round_up(states, kWsAlign);
  p.off_Z = round_up(p.off_dS + states, kWsAlign);
  p.off_dq = round_up(p.off_Z + td * 4, kWsAlign);
  p.off_dk = round_up(p.off_dq + td * 4, kWsAlign);
  p.off_rec = round_up(p.off_dk + td * 4, kWsAlign);
  p.total = scratch(p.off_rec + delta_simt_records(s));
  return p;
}

template <int D, bool GRADS>
int launch_delta_walk(const infini_delta_shape* s, const infini::DeltaArgs<__nv_bfloat16>& a, uint8_t* records,
                      __nv_bfloat16* kept_S, __nv_bfloat16* kept_U, cudaStream_t st) {
  using namespace infini;
  using M = DwSmem<D, GRADS>;
  if (allow_smem(delta_prep_kernel<D, GRADS>, DpSmem<D>::kTotal) != cudaSuccess ||
      allow_smem(delta_walk_kernel<D, GRADS>, M::kTotal) != cudaSuccess)
    return INFINI_ERR_CUDA;
  // A CTA takes all value heads of its key head (k.k and q.k once), or, where all
  // CTAs fit the GPU at once (four to an SM), one each: then the chain of one
  // head is what the launch lasts.
  const int64_t slots = slot_count(s->T, s->n_seq, kDcTok);
  const unsigned split = a.G <= 64 && slots * s->Hv <= 4 * 148 ? (unsigned)a.G : 1u;
  delta_prep_kernel<D, GRADS><<<dim3((unsigned)slots, (unsigned)s->Hk, split), kDpThreads, DpSmem<D>::kTotal, st>>>(a.q, a.k, a.g, a.beta, a.seq, a.Hv, a.G, a.scale, records);
  if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  CUtensorMap mk, mq, mv;
  if (!make_rows_map(&mk, a.k, s->T, s->Hk, D, kDcTok) || !make_rows_map(&mq, a.q, s->T, s->Hk, D, kDcTok) ||
      !make_rows_map(&mv, a.v, s->T, s->Hv, D, kDcTok))
    return INFINI_ERR_CUDA;
  delta_walk_kernel<D, GRADS><<<dim3(D / kDwRows, (unsigned)s->Hv, (unsigned)s->n_seq), kDwThreads, M::kTotal, st>>>(
      mk, mq, mv, a, records, kept_S, kept_U, next_epoch());
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <int D>
int launch_delta_tc_backward(const infini_delta_shape* s, const infini::DeltaGradArgs<__nv_bfloat16>& a, char* ws,
                             cudaStream_t st) {
  using namespace infini;
  const DeltaBwdPlan p = delta_bwd_plan(s, INFINI_PATH_TC);
  uint8_t* rec = reinterpret_cast<uint8_t*>(ws);
  auto* S = reinterpret_cast<__nv_bfloat16*>(ws + p.off_S);
  auto* dS = reinterpret_cast<__nv_bfloat16*>(ws + p.off_dS);
  auto* U = reinterpret_cast<__nv_bfloat16*>(ws + p.off_U);
  auto* Z = reinterpret_cast<__nv_bfloat16*>(ws + p.off_Z);
  DeltaArgs<__nv_bfloat16> f{a.q, a.k, a.v, a.g, a.beta, {nullptr, 0, 0}, a.S_in, nullptr, a.seq, a.Hk, a.Hv, a.G,
                             a.scale};
  int rc = launch_delta_walk<D, true>(s, f, rec, S, U, st);
  if (rc != INFINI_OK) return rc;
  if (allow_smem(delta_reverse_kernel<D>, DrSmem<D>::kTotal) != cudaSuccess ||
      allow_smem(delta_grad_kernel<D>, DgSmem<D>::kTotal) != cudaSuccess)
    return INFINI_ERR_CUDA;
  CUtensorMap mk, mq, mo;
  if (!make_rows_map(&mk, a.k, s->T, s->Hk, D, kDcTok) || !make_rows_map(&mq, a.q, s->T, s->Hk, D, kDcTok) ||
      !make_rows_map(&mo, a.dout, s->T, s->Hv, D, kDcTok))
    return INFINI_ERR_CUDA;
  delta_reverse_kernel<D><<<dim3(D / kDwRows, (unsigned)s->Hv, (unsigned)s->n_seq), kDwThreads, DrSmem<D>::kTotal, st>>>(
      mk, mq, mo, a, rec, dS, Z, next_epoch());
  if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  delta_grad_kernel<D><<<dim3((unsigned)slot_count(s->T, s->n_seq, kDcTok), (unsigned)s->Hk), kDgThreads,
                         DgSmem<D>::kTotal, st>>>(a, rec, S, dS, U, Z);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <typename T, int D>
int launch_delta_form(const infini_delta_shape* s, const infini::DeltaArgs<T>& a, int most, float* records,
                      cudaStream_t st) {
  using namespace infini;
  constexpr size_t form = DsChunk<D>::kFloats * 4;
  static_assert(DsChunk<D>::kRecord == DsChunk<64>::kRecord, "the plan's size of a record");
  if (allow_smem(delta_simt_form_kernel<T, D>, form) != cudaSuccess) return INFINI_ERR_CUDA;
  delta_simt_form_kernel<T, D><<<dim3((unsigned)slot_count(s->T, s->n_seq, kDsChunk), (unsigned)s->Hv), kDsThreads,
                                 form, st>>>(a, most, records);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <typename T, int D>
int launch_delta_forward(const infini_delta_shape* s, const infini::DeltaArgs<T>& a, float* records, cudaStream_t st) {
  using namespace infini;
  const dim3 strips(D / kDsCols, (unsigned)s->Hv, (unsigned)s->n_seq);
  if (s->max_len <= kDeltaFew) {
    delta_simt_fwd_kernel<T, D><<<strips, kDsThreads, 0, st>>>(a);
  } else {
    const int rc = launch_delta_form<T, D>(s, a, kDsRecurMost, records, st);
    if (rc != INFINI_OK) return rc;
    constexpr size_t walk = ds_chain_smem<D>();
    if (allow_smem(delta_simt_walk_kernel<T, D>, walk) != cudaSuccess) return INFINI_ERR_CUDA;
    delta_simt_walk_kernel<T, D><<<strips, kDsThreads, walk, st>>>(a, records);
  }
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

template <typename T, int D>
int launch_delta_backward(const infini_delta_shape* s, const infini::DeltaGradArgs<T>& a, char* ws, cudaStream_t st) {
  using namespace infini;
  const DeltaBwdPlan p = delta_bwd_plan(s, INFINI_PATH_SIMT);
  float* kept = reinterpret_cast<float*>(ws + p.off_kept);
  float* dq = reinterpret_cast<float*>(ws + p.off_dq);
  float* dk = reinterpret_cast<float*>(ws + p.off_dk);
  DeltaArgs<T> f{a.q, a.k, a.v, a.g, a.beta, {nullptr, 0, 0}, a.S_in, nullptr, a.seq, a.Hk, a.Hv, a.G, a.scale};
  float* dS = reinterpret_cast<float*>(ws + p.off_dS);
  float* Z = reinterpret_cast<float*>(ws + p.off_Z);
  float* rec = reinterpret_cast<float*>(ws + p.off_rec);
  const int rc = launch_delta_form<T, D>(s, f, 0, rec, st);
  if (rc != INFINI_OK) return rc;
  constexpr size_t chain = ds_chain_smem<D>(), grad = ds_grad_smem<D>();
  if (allow_smem(delta_simt_walks_kernel<T, D>, chain) != cudaSuccess ||
      allow_smem(delta_simt_grad_kernel<T, D>, grad) != cudaSuccess)
    return INFINI_ERR_CUDA;
  const dim3 all((unsigned)slot_count(s->T, s->n_seq, kDsChunk), (unsigned)s->Hv);
  delta_simt_walks_kernel<T, D><<<dim3(2 * D / kDsCols, (unsigned)s->Hv, (unsigned)s->n_seq), kDsThreads, chain, st>>>(
      f, a, rec, kept, dS, Z);
  if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  delta_simt_grad_kernel<T, D><<<all, kDsThreads, grad, st>>>(a, rec, kept, dS, Z, dq, dk);
  if (cudaGetLastError() != cudaSuccess) return INFINI_ERR_CUDA;
  delta_group_sum_kernel<T, D><<<dim3((unsigned)slot_count(s->T, s->n_seq, kDsChunk), (unsigned)s->Hk), 256, 0, st>>>(
      a, dq, dk);
  return cudaGetLastError() == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

// A call that needs no scratch memory gives kWsAlign as its size (0 stands for
// an error) and may be given none.
int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws && need <= kWsAlign) return INFINI_OK;
  if (!ws) return INFINI_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(ws) & (kWsAlign - 1)) != 0) return INFINI_ERR_ALIGN;
  return bytes < need ? INFINI_ERR_WORKSPACE : INFINI_OK;
}

#define INFINI_TRY(x)                    \
  do {                                   \
    const int rc_ = (x);                 \
    if (rc_ != INFINI_OK) return rc_;    \
  } while (0)

}  // namespace

extern "C" {

size_t infini_attn_packed_workspace_size(const infini_packed_shape* s, int path) {
  if (check_packed(s) != INFINI_OK) return 0;
  path = packed_resolve(s, path, false);
  return path < 0 ? 0 : packed_ws(s, path);
}

int infini_attn_packed_select_path(const infini_packed_shape* s) {
  INFINI_TRY(check_packed(s));
  return packed_resolve(s, INFINI_PATH_AUTO, false);
}

int infini_attn_packed_forward(const infini_packed_shape* s, const infini_rows* q, const infini_rows* k,
                               const infini_rows* v, const int32_t* q_off, const int32_t* k_off, const int32_t* q_len,
                               const int32_t* k_len, const infini_rows* out, float* lse, void* workspace,
                               size_t workspace_bytes, int path, infini_stream_t stream) {
  INFINI_TRY(check_packed(s));
  path = packed_resolve(s, path, false);
  if (path < 0) return path;
  const int64_t elt = s->dtype == INFINI_F32 ? 4 : 2, n = s->n_seq;
  Rows x[4];
  Region r[10];
  INFINI_TRY(take_rows(q, s->Tq, s->Hq, s->d, elt, false, &x[0], &r[0]));
  INFINI_TRY(take_rows(k, s->Tk, s->Hkv, s->d, elt, false, &x[1], &r[1]));
  INFINI_TRY(take_rows(v, s->Tk, s->Hkv, s->d, elt, false, &x[2], &r[2]));
  INFINI_TRY(take_rows(out, s->Tq, s->Hq, s->d, elt, true, &x[3], &r[3]));
  if (n > 0 && (!q_off || !k_off)) return INFINI_ERR_NULL;
  INFINI_TRY(check_workspace(workspace, workspace_bytes, packed_ws(s, path)));
  r[4] = flat(lse, s->Hq * s->Tq * 4, true);
  r[5] = flat(workspace, (int64_t)packed_ws(s, path), true);
  r[6] = flat(q_off, (n + 1) * 4, false);
  r[7] = flat(k_off, (n + 1) * 4, false);
  r[8] = flat(q_len, n * 4, false);
  r[9] = flat(k_len, n * 4, false);
  INFINI_TRY(check_alias(r, 10));
  if (n == 0 || s->Tq == 0) return INFINI_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    infini::PackedArgs<T> a{rows_of<const T>(x[0]), rows_of<const T>(x[1]), rows_of<const T>(x[2]), rows_of<T>(x[3]),
                            lse, {q_off, q_len, (int)n, (int)s->Tq}, {k_off, k_len, (int)n, (int)s->Tk},
                            (int)s->Hq, (int)s->Hkv, (int)(s->Hq / s->Hkv), s->scale, packed_by_work(s)};
    char* ws = static_cast<char*>(workspace);
    return s->d == 64 ? launch_packed_forward<T, 64>(s, a, path, ws, st)
                      : launch_packed_forward<T, 128>(s, a, path, ws, st);
  };
  return s->dtype == INFINI_F32 ? go(float{}) : go(__nv_bfloat16{});
}

size_t infini_attn_packed_backward_workspace_size(const infini_packed_shape* s) {
  if (check_packed(s) != INFINI_OK) return 0;
  return scratch((size_t)s->Hq * s->Tq * 4);
}

int infini_attn_packed_backward(const infini_packed_shape* s, const infini_rows* q, const infini_rows* k,
                                const infini_rows* v, const infini_rows* out, const float* lse,
                                const infini_rows* dout, const int32_t* q_off, const int32_t* k_off,
                                const int32_t* q_len, const int32_t* k_len, const infini_rows* dq,
                                const infini_rows* dk, const infini_rows* dv, void* workspace,
                                size_t workspace_bytes, int path, infini_stream_t stream) {
  INFINI_TRY(check_packed(s));
  path = packed_resolve(s, path, true);
  if (path < 0) return path;
  const int64_t elt = s->dtype == INFINI_F32 ? 4 : 2, n = s->n_seq;
  Rows x[8];
  Region r[14];
  const infini_rows* in[8] = {q, k, v, out, dout, dq, dk, dv};
  const bool keys[8] = {false, true, true, false, false, false, true, true};
  for (int i = 0; i < 8; ++i)
    INFINI_TRY(take_rows(in[i], keys[i] ? s->Tk : s->Tq, keys[i] ? s->Hkv : s->Hq, s->d, elt, i >= 5, &x[i], &r[i]));
  if (n > 0 && (!q_off || !k_off)) return INFINI_ERR_NULL;
  if (!lse && s->Tq > 0) return INFINI_ERR_NULL;
  const size_t need = infini_attn_packed_backward_workspace_size(s);
  INFINI_TRY(check_workspace(workspace, workspace_bytes, need));
  r[8] = flat(lse, s->Hq * s->Tq * 4, false);
  r[9] = flat(workspace, (int64_t)need, true);
  r[10] = flat(q_off, (n + 1) * 4, false);
  r[11] = flat(k_off, (n + 1) * 4, false);
  r[12] = flat(q_len, n * 4, false);
  r[13] = flat(k_len, n * 4, false);
  INFINI_TRY(check_alias(r, 14));
  if (n == 0) return INFINI_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    infini::PackedGradArgs<T> a{rows_of<const T>(x[0]), rows_of<const T>(x[1]), rows_of<const T>(x[2]),
                                rows_of<const T>(x[3]), rows_of<const T>(x[4]), rows_of<T>(x[5]), rows_of<T>(x[6]),
                                rows_of<T>(x[7]), lse, static_cast<float*>(workspace),
                                {q_off, q_len, (int)n, (int)s->Tq}, {k_off, k_len, (int)n, (int)s->Tk},
                                (int)s->Hq, (int)s->Hkv, (int)(s->Hq / s->Hkv), s->scale};
    return s->d == 64 ? launch_packed_backward<T, 64>(s, a, path, st) : launch_packed_backward<T, 128>(s, a, path, st);
  };
  return s->dtype == INFINI_F32 ? go(float{}) : go(__nv_bfloat16{});
}

size_t infini_attn_delta_workspace_size(const infini_delta_shape* s, int path) {
  if (check_delta(s) != INFINI_OK) return 0;
  path = delta_resolve(s, path, s->max_len <= kDeltaFew);
  return path < 0 ? 0 : delta_fwd_ws(s, path);
}

int infini_attn_delta_forward(const infini_delta_shape* s, const infini_rows* q, const infini_rows* k,
                              const infini_rows* v, const infini_rows* g, const infini_rows* beta, const int32_t* off,
                              const int32_t* len, const float* S_in, const infini_rows* out, float* S_out,
                              void* workspace, size_t workspace_bytes, int path, infini_stream_t stream) {
  INFINI_TRY(check_delta(s));
  path = delta_resolve(s, path, s->max_len <= kDeltaFew);
  if (path < 0) return path;
  const int64_t elt = s->dtype == INFINI_F32 ? 4 : 2, n = s->n_seq, states = n * s->Hv * s->d * s->d * 4;
  Rows x[6];
  Region r[11];
  const infini_rows* in[6] = {q, k, v, g, beta, out};
  for (int i = 0; i < 6; ++i)
    INFINI_TRY(take_rows(in[i], s->T, i < 2 ? s->Hk : s->Hv, i == 3 || i == 4 ? 1 : s->d, elt, i == 5, &x[i], &r[i]));
  if (n > 0 && !off) return INFINI_ERR_NULL;
  if (!aligned16(S_in) || !aligned16(S_out)) return INFINI_ERR_ALIGN;
  const size_t need = delta_fwd_ws(s, path);
  INFINI_TRY(check_workspace(workspace, workspace_bytes, need));
  r[6] = flat(S_in == S_out ? nullptr : S_in, states, false);
  r[7] = flat(S_out, states, true);
  r[8] = flat(workspace, (int64_t)need, true);
  r[9] = flat(off, (n + 1) * 4, false);
  r[10] = flat(len, n * 4, false);
  INFINI_TRY(check_alias(r, 11));
  if (n == 0) return INFINI_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    infini::DeltaArgs<T> a{rows_of<const T>(x[0]), rows_of<const T>(x[1]), rows_of<const T>(x[2]),
                           rows_of<const T>(x[3]), rows_of<const T>(x[4]), rows_of<T>(x[5]), S_in, S_out,
                           {off, len, (int)n, (int)s->T}, (int)s->Hk, (int)s->Hv, (int)(s->Hv / s->Hk), s->scale};
    if constexpr (sizeof(T) == 2)
      if (path == INFINI_PATH_TC) {
        uint8_t* rec = static_cast<uint8_t*>(workspace);
        return s->d == 64 ? launch_delta_walk<64, false>(s, a, rec, nullptr, nullptr, st)
                          : launch_delta_walk<128, false>(s, a, rec, nullptr, nullptr, st);
      }
    float* rec = static_cast<float*>(workspace);
    return s->d == 64 ? launch_delta_forward<T, 64>(s, a, rec, st) : launch_delta_forward<T, 128>(s, a, rec, st);
  };
  return s->dtype == INFINI_F32 ? go(float{}) : go(__nv_bfloat16{});
}

size_t infini_attn_delta_backward_workspace_size(const infini_delta_shape* s, int path) {
  if (check_delta(s) != INFINI_OK) return 0;
  path = delta_resolve(s, path, false);
  return path < 0 ? 0 : delta_bwd_plan(s, path).total;
}

int infini_attn_delta_backward(const infini_delta_shape* s, const infini_rows* q, const infini_rows* k,
                               const infini_rows* v, const infini_rows* g, const infini_rows* beta, const int32_t* off,
                               const int32_t* len, const float* S_in, const infini_rows* dout, const float* dS_out,
                               const infini_rows* dq, const infini_rows* dk, const infini_rows* dv,
                               const infini_rows* dg, const infini_rows* dbeta, float* dS_in, void* workspace,
                               size_t workspace_bytes, int path, infini_stream_t stream) {
  INFINI_TRY(check_delta(s));
  path = delta_resolve(s, path, false);
  if (path < 0) return path;
  const int64_t elt = s->dtype == INFINI_F32 ? 4 : 2, n = s->n_seq, states = n * s->Hv * s->d * s->d * 4;
  Rows x[11];
  Region r[17];
  const infini_rows* in[11] = {q, k, v, g, beta, dout, dq, dk, dv, dg, dbeta};
  const bool key[11] = {true, true, false, false, false, false, true, true, false, false, false};
  const bool one[11] = {false, false, false, true, true, false, false, false, false, true, true};
  for (int i = 0; i < 11; ++i)
    INFINI_TRY(take_rows(in[i], s->T, key[i] ? s->Hk : s->Hv, one[i] ? 1 : s->d, elt, i >= 6, &x[i], &r[i]));
  if (n > 0 && !off) return INFINI_ERR_NULL;
  if (!aligned16(S_in) || !aligned16(dS_out) || !aligned16(dS_in)) return INFINI_ERR_ALIGN;
  const size_t need = delta_bwd_plan(s, path).total;
  INFINI_TRY(check_workspace(workspace, workspace_bytes, need));
  r[11] = flat(S_in, states, false);
  r[12] = flat(dS_out == dS_in ? nullptr : dS_out, states, false);
  r[13] = flat(dS_in, states, true);
  r[14] = flat(workspace, (int64_t)need, true);
  r[15] = flat(off, (n + 1) * 4, false);
  r[16] = flat(len, n * 4, false);
  INFINI_TRY(check_alias(r, 17));
  if (n == 0) return INFINI_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    infini::DeltaGradArgs<T> a{rows_of<const T>(x[0]), rows_of<const T>(x[1]), rows_of<const T>(x[2]),
                               rows_of<const T>(x[3]), rows_of<const T>(x[4]), rows_of<const T>(x[5]),
                               rows_of<T>(x[6]), rows_of<T>(x[7]), rows_of<T>(x[8]), rows_of<T>(x[9]),
                               rows_of<T>(x[10]), S_in, dS_out, dS_in, {off, len, (int)n, (int)s->T},
                               (int)s->Hk, (int)s->Hv, (int)(s->Hv / s->Hk), s->scale};
    char* ws = static_cast<char*>(workspace);
    if constexpr (sizeof(T) == 2)
      if (path == INFINI_PATH_TC)
        return s->d == 64 ? launch_delta_tc_backward<64>(s, a, ws, st) : launch_delta_tc_backward<128>(s, a, ws, st);
    return s->d == 64 ? launch_delta_backward<T, 64>(s, a, ws, st) : launch_delta_backward<T, 128>(s, a, ws, st);
  };
  return s->dtype == INFINI_F32 ? go(float{}) : go(__nv_bfloat16{});
}

int infini_attn_delta_step(const infini_delta_shape* s, const infini_rows* q, const infini_rows* k,
                           const infini_rows* v, const infini_rows* g, const infini_rows* beta, const float* S_in,
                           const infini_rows* out, float* S_out, infini_stream_t stream) {
  INFINI_TRY(check_delta(s));
  if (s->T > kMaxGridY) return INFINI_ERR_SIZE;
  const int64_t elt = s->dtype == INFINI_F32 ? 4 : 2, states = s->T * s->Hv * s->d * s->d * 4;
  Rows x[6];
  Region r[8];
  const infini_rows* in[6] = {q, k, v, g, beta, out};
  for (int i = 0; i < 6; ++i)
    INFINI_TRY(take_rows(in[i], s->T, i < 2 ? s->Hk : s->Hv, i == 3 || i == 4 ? 1 : s->d, elt, i == 5, &x[i], &r[i]));
  if (s->T > 0 && (!S_in || !S_out)) return INFINI_ERR_NULL;
  if (!aligned16(S_in) || !aligned16(S_out)) return INFINI_ERR_ALIGN;
  r[6] = flat(S_in == S_out ? nullptr : S_in, states, false);
  r[7] = flat(S_out, states, true);
  INFINI_TRY(check_alias(r, 8));
  if (s->T == 0) return INFINI_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag) {
    using T = decltype(tag);
    infini::DeltaArgs<T> a{rows_of<const T>(x[0]), rows_of<const T>(x[1]), rows_of<const T>(x[2]),
                           rows_of<const T>(x[3]), rows_of<const T>(x[4]), rows_of<T>(x[5]), S_in, S_out,
                           {nullptr, nullptr, 0, 0}, (int)s->Hk, (int)s->Hv, (int)(s->Hv / s->Hk), s->scale};
    const dim3 grid((unsigned)s->Hv, (unsigned)s->T);
    if (s->d == 64)
      infini::delta_step_kernel<T, 64><<<grid, 256, 0, st>>>(a);
    else
      infini::delta_step_kernel<T, 128><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? (int)INFINI_OK : (int)INFINI_ERR_CUDA;
  };
  return s->dtype == INFINI_F32 ? go(float{}) : go(__nv_bfloat16{});
}

}  // extern "C"

// Paged K/V cache (sm_100a): writing new rows (E4M3 quantisation or a copy),
// reading selected rows back, and attention with few query rows per kv head
// over the pages -- one token per sequence over selected rows, or a short
// chunk of tokens over every row up to its own.
//
// Rows and scales: see paged.cuh.  The scale of one position and kv head is a
// power of two, 2^e with e the least integer such that max|x| <= 448 * 2^e:
// E4M3 has the same relative step at every magnitude, so a finer scale would
// gain no precision, and a power of two makes x * 2^-e, code * 2^e and the
// value's bf16 form exact; the rounding to a code is the only one.
//
// Few-row attention: softmax(scale q.K^T) V by one pass with a running
// maximum and sum.  It reads the cache once, 2 * row bytes per position for
// 4 * 128 * Hq flops, so it is bound by HBM; the 16-row side of the matrix
// instructions (mma.sync, 16 x 8) takes the cache's, the 8-column side the G
// query heads of the chunk's tokens, which share the kv head's rows.
//
//   paged_write_kernel       one warp per token (K and V)
//   paged_gather_kernel      one warp per selected row (K and V)
//   paged_attn_rows_kernel   units of (block of up to 24 query rows, tile of
//       positions, all kv heads), flattened over the batch and cut evenly
//       over one CTA per SM; partials of (max, sum, output)
//   paged_attn_rows_merge_kernel   folds them by the log-sum-exp rule
#include "paged.cuh"
#include "tc_common.cuh"

namespace sa {
namespace {

// ------------------------------------------------------------------- write

// A new row (Hkv * 128 bf16) in registers: half a warp holds one head, lane j
// of the half 8 values (16 bytes).
struct NewRow {
  uint4 v[4];
};
__device__ __forceinline__ void load_row(NewRow& r, const uint16_t* __restrict__ x, int Hkv) {
  const int lane = threadIdx.x & 31, half = lane >> 4, j = lane & 15;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int h = 2 * it + half;
    r.v[it] = h < Hkv ? __ldg(reinterpret_cast<const uint4*>(x + h * kPgD) + j) : make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest magnitude (bf16 bits) of each of half a warp's heads: magnitudes
// compare as integers, two at a time, and two heads share their shuffles.
// FINITE leaves infinities and NaN out.
template <bool FINITE>
__device__ __forceinline__ void head_maxima(const NewRow& r, int Hkv, uint32_t (&am)[4]) {
#pragma unroll
  for (int it = 0; it < 4; it += 2) {
    uint32_t m[2] = {0u, 0u};
    am[it] = am[it + 1] = 0u;
    if (2 * it >= Hkv) break;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint4& v = r.v[it + t];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x = w[i] & 0x7fff7fffu;
        if (FINITE) {
          if ((x & 0xffffu) >= 0x7f80u) x &= 0xffff0000u;
          if ((x >> 16) >= 0x7f80u) x &= 0x0000ffffu;
        }
        m[t] = max_u16x2(m[t], x);
      }
    }
    uint32_t both = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) both = max_u16x2(both, __shfl_xor_sync(0xffffffffu, both, o));
    am[it] = both & 0xffffu;
    am[it + 1] = both >> 16;
  }
}

// Codes of four bf16 values times inv (NaN: the NaN code).
__device__ __forceinline__ uint32_t e4m3_codes(uint32_t w0, uint32_t w1, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(bf_hi(w0) * inv), "f"(bf_lo(w0) * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(bf_hi(w1) * inv), "f"(bf_lo(w1) * inv));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// The cache row of a new row.
template <bool FP8>
__device__ __forceinline__ void write_row(const NewRow& r, uint8_t* __restrict__ row, int Hkv) {
  const int lane = threadIdx.x & 31, half = lane >> 4, j = lane & 15;
  if constexpr (!FP8) {
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int h = 2 * it + half;
      if (h < Hkv) reinterpret_cast<uint4*>(row + h * (2 * kPgD))[j] = r.v[it];
    }
    if (lane == 0) *reinterpret_cast<uint4*>(row + Hkv * (2 * kPgD)) = make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint32_t tail[2] = {0u, 0u};   // the scale bytes of heads 0-3 and 4-7
    uint32_t am[4];
    head_maxima<false>(r, Hkv, am);
    const bool odd = __any_sync(0xffffffffu, max(max(am[0], am[1]), max(am[2], am[3])) >= 0x7f80u);
    if (odd) head_maxima<true>(r, Hkv, am);   // rare: not all finite
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      if (2 * it >= Hkv) break;
      uint32_t w[4] = {r.v[it].x, r.v[it].y, r.v[it].z, r.v[it].w};
      // am = 2^(E - 127) * (1 + M / 128); 448 = 2^8 * 1.75, so the least e
      // with am <= 448 * 2^e is E - 135, or E - 134 when 1 + M / 128 > 1.75
      const int E = (int)(am[it] >> 7), M = (int)(am[it] & 0x7fu);
      int e = E - (M > 0x60 ? 134 : 135);
      e = min(max(e, -118), 119);   // 448 * 2^119 and 2^-9 * 2^-118 are bf16 values
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      if (odd) {   // E4M3 has no infinity
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((w[i] & 0x7fffu) == 0x7f80u) w[i] |= 0x0040u;
          if ((w[i] & 0x7fff0000u) == 0x7f800000u) w[i] |= 0x00400000u;
        }
      }
      const int h = 2 * it + half;
      if (h < Hkv) {
        reinterpret_cast<uint2*>(row + h * kPgD)[j] =
            make_uint2(e4m3_codes(w[0], w[1], inv), e4m3_codes(w[2], w[3], inv));
        tail[it >> 1] |= (uint32_t)(e + 127) << (16 * (it & 1) + 8 * half);
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) tail[t] |= __shfl_xor_sync(0xffffffffu, tail[t], 16);
    if (lane == 0) *reinterpret_cast<uint4*>(row + Hkv * kPgD) = make_uint4(tail[0], tail[1], 0u, 0u);
  }
}

// Bound by HBM: 512 bytes in and 258 (E4M3) or 512 out per token, kv head and
// cache.  A warp takes a token's K and V; its rows are on their way while the
// token's sequence, position and page are looked up (four dependent reads).
// 32,768 tokens, 8 kv heads: E4M3 33.8 us (6.0 TB/s; 39.5 with a check for
// infinities at every value and a head's shuffles of its own), bf16 43.1 us
// (6.2 TB/s).  Fewer registers, more warps: 42 us at 40 registers.
template <bool FP8>
__global__ void __launch_bounds__(256)
paged_write_kernel(const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new, long long k_stride,
                   long long v_stride, const int32_t* __restrict__ q_start, const int32_t* __restrict__ kv_len,
                   const int32_t* __restrict__ table, int B, int N, int max_pages, int num_pages, int page_shift,
                   int Hkv, uint8_t* __restrict__ kp, uint8_t* __restrict__ vp, int* dbg) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);   // token
  if (i >= N) return;
  NewRow k, v;
  load_row(k, k_new + (long long)i * k_stride, Hkv);
  load_row(v, v_new + (long long)i * v_stride, Hkv);
  const int b = seq_of_token(q_start, B, i);
  if (b < 0) return;      // in front of the first sequence or behind the last
  const int capacity = max_pages << page_shift;
  const SeqSpan s = seq_span(q_start, kv_len, b, N, capacity);
  const long long at = (long long)kv_len[b] - s.len + (i - s.begin);
  if (at < 0 || at >= capacity) return;   // kv_len does not count this token, or the table has no place for it
  const int pos = (int)at;
  const int pg = table[(long long)b * max_pages + (pos >> page_shift)];
  if (pg < 0 || pg >= num_pages) {   // no page: the token is dropped, no other page is touched
    if ((threadIdx.x & 31) == 0) paged_note(dbg, kDbgPage, pg, num_pages);
    return;
  }
  const long long slot = ((long long)pg << page_shift) + (pos & ((1 << page_shift) - 1));
  const long long off = slot * paged_row_bytes(FP8, Hkv);
  write_row<FP8>(k, kp + off, Hkv);
  write_row<FP8>(v, vp + off, Hkv);
}

// ------------------------------------------------------------------ gather

// Bound by HBM: a row's bytes in, Hkv * 256 + 16 out, K and V.  One warp per
// selected row, both caches' loads issued together; 16 lanes take a head, 8
// values each, so that stores are 512 bytes side by side.
template <bool FP8>
__global__ void __launch_bounds__(256)
paged_gather_kernel(const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, const int32_t* __restrict__ table,
                    const int32_t* __restrict__ idx, const int32_t* __restrict__ count, int max_pages, int num_pages,
                    int page_shift, int Hkv, int k, uint16_t* __restrict__ ko, uint16_t* __restrict__ vo, int* dbg) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, half = lane >> 4, j16 = lane & 15;
  const int b = blockIdx.y;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= k) return;
  const int c = count[b];
  int j = idx[(long long)b * k + r];   // (not used from the count on)
  uint4* dst[2] = {reinterpret_cast<uint4*>(ko + ((long long)b * k + r) * (Hkv * kPgD + 8)),
                   reinterpret_cast<uint4*>(vo + ((long long)b * k + r) * (Hkv * kPgD + 8))};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (lane < 2) dst[lane][Hkv * 16] = zero;
  if (r >= c) {
    for (int e = lane; e < Hkv * 16; e += 32) dst[0][e] = dst[1][e] = zero;
    return;
  }
  const int capacity = max_pages << page_shift;
  if (j < 0 || j >= capacity) {
    paged_note(dbg, kDbgPagedIndex, j, capacity);
    j = j < 0 ? 0 : capacity - 1;
  }
  const int pg = checked_page(table[(long long)b * max_pages + (j >> page_shift)], num_pages, dbg);
  const long long off =
      (((long long)pg << page_shift) + (j & ((1 << page_shift) - 1))) * paged_row_bytes(FP8, Hkv);
  const uint8_t* row[2] = {kp + off, vp + off};
  if constexpr (!FP8) {
    uint4 v[2][4];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int it = 0; it < 4; ++it)
        if (2 * it + half < Hkv) v[kv][it] = __ldg(reinterpret_cast<const uint4*>(row[kv]) + it * 32 + lane);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int it = 0; it < 4; ++it)
        if (2 * it + half < Hkv) dst[kv][it * 32 + lane] = v[kv][it];
  } else {
    uint2 v[2][4], tail[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      tail[kv] = __ldg(reinterpret_cast<const uint2*>(row[kv] + Hkv * kPgD));
#pragma unroll
      for (int it = 0; it < 4; ++it)
        if (2 * it + half < Hkv) v[kv][it] = __ldg(reinterpret_cast<const uint2*>(row[kv] + (2 * it + half) * kPgD) + j16);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int h = 2 * it + half;
        if (h < Hkv)
          dst[kv][h * 16 + j16] =
              e4m3x8_to_bf16x8(v[kv][it], e8m0_value(((it < 2 ? tail[kv].x : tail[kv].y) >> (8 * (h & 3))) & 0xffu));
      }
  }
}

// ------------------------------------------------------- few-row attention

constexpr int kRwConsumers = 8;
// The producer and the three warps beside it (which copy selected rows and are
// idle otherwise) leave registers to the consumers: 8 * 224 + 4 * 56 = 12 * 168
// (without: 121 us for one token of each of 8 x 32K E4M3 positions, 115 with).
constexpr int kRwThreads = (kRwConsumers + 4) * 32, kRwConsumerRegs = 224, kRwOtherRegs = 56;
constexpr int kRwMaxStages = 8;
// Query rows of a block, in eights: what the consumers' registers hold (drafts
// of 20 rows, 16 sequences, 8 kv heads: bf16 82 us in blocks of 16, 68 of 24;
// E4M3 65 and 78, as 24 rows spill beside two scales and references).
template <bool FP8>
constexpr int kRwRows = FP8 ? 16 : 24;
constexpr int kRwBarBytes = 256;       // mbarriers, abort word, plan, scan
static_assert((2 * kRwMaxStages + 2 + kRwThreads / 32) * 8 <= kRwBarBytes, "barrier block");
constexpr int kRwStageBytes = 222 * 1024;
constexpr int kRwMergeThreads = 256;
// Rows from which a warp folds one, not a CTA (us, whole call, E4M3, one token
// of each sequence, 32 heads, warp / CTA: 64 x 4K positions 121 / 127, 32 x 4K
// 78 / 80, 16 x 4K 53 / 51, 1M selected from 35 / 18).
constexpr int kRwMergeMany = 1024;
constexpr int kRwMergeMaxC = 1280;     // contributors of one (row block, head)

// Positions a consumer warp takes per step: codes are half the bytes, so twice
// as many for the same stage, with more independent products in flight (16:
// 184 us for one token of each of 8 x 32K positions, 8 kv heads).
template <bool FP8>
constexpr int kRwKeys = FP8 ? 32 : 16;

struct RowsPlan {
  int nrb, tb, RB;         // row blocks per sequence, tokens and rows of one
  int P;                   // items: B * nrb
  int wph, R;              // consumer warps per kv head, positions per tile
  int row_bytes, stages;
  int W;                   // CTAs
  bool by_item;            // merge: CTAs by row block and token, not by token (most tokens are not here)
};

// Tiles of R positions that hold n (n + R may pass 2^31).
__device__ __forceinline__ int tiles_of(int n, int R) { return (int)(((unsigned)n + (unsigned)R - 1u) / (unsigned)R); }

// Tiles of item p: the positions its last token attends to, or the selected
// rows of its sequence.
template <bool SPARSE>
__device__ __forceinline__ int item_keys(const PagedArgs& a, const RowsPlan& pl, int p) {
  if constexpr (SPARSE) {
    return min(max(a.count[p], 0), a.k);
  } else {
    const int b = p / pl.nrb, t0 = p % pl.nrb * pl.tb;
    const SeqSpan s = seq_span(a.q_start, a.kv_len, b, a.N, a.max_pages << a.page_shift);
    const int n = min(s.len, a.max_q);
    if (t0 >= n || s.len > a.many) return 0;
    return max(s.pos0 + min(t0 + pl.tb, n), 0);
  }
}
template <bool SPARSE>
__device__ __forceinline__ int item_tiles(const PagedArgs& a, const RowsPlan& pl, int p) {
  return tiles_of(item_keys<SPARSE>(a, pl, p), pl.R);
}

// Sum over the block of v (threads kThreads, a multiple of 32), and the sum
// over the threads before this one.  Every thread calls it.
template <int kThreads>
__device__ __forceinline__ long long block_scan(int v, long long& before, long long* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  long long base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += sh[w];
    total += sh[w];
  }
  before = base + x - v;
  return total;
}

// v, and the sum over the lanes before this one; returns the warp's.
__device__ __forceinline__ long long warp_scan(int v, long long& before) {
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += y;
  }
  before = x - v;
  return __shfl_sync(0xffffffffu, x, 31);
}

// floor(x / d), x >= 0, d > 0 (a division of 64 bits takes hundreds of clocks).
__device__ __forceinline__ long long floor_div(long long x, long long d) {
  return (unsigned long long)(x | d) >> 32 ? x / d : (long long)((unsigned)x / (unsigned)d);
}

// Query fragments (the 8-column side): row 8 n + gq of the block is token
// tok0 + row / G, head row % G of kv head g.  For bf16 keys the usual layout;
// for codes, fp16 with the reduction index permuted to what one ldmatrix of 16
// codes gives (lane t holds elements 4t .. 4t+3 of every 16), each row scaled
// by a power of two that brings its largest magnitude to [2^14, 2^15): exact
// for every element within 2^-31 of the largest, and undone in fp32 (`rowc`,
// for rows 8 n + 2 tg + {0, 1}).
template <bool FP8, int NB>
__device__ __forceinline__ void load_q_rows(uint32_t (&q)[NB][8][2], float (&rowc)[NB][2], const PagedArgs& a, int tok0,
                                            int ntok, int g, bool active) {
  const int lane = threadIdx.x & 31, gq = lane >> 2, tg = lane & 3;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = gq + 8 * nb;
    const bool on = active && r < ntok * a.G;
    const uint16_t* src = a.q + (long long)(tok0 + (on ? r / a.G : 0)) * a.q_stride +
                          ((active ? g : 0) * a.G + (on ? r % a.G : 0)) * kPgD;
    float f = a.qscale;
    if constexpr (!FP8) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        q[nb][kk][0] = on ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * tg)) : 0u;
        q[nb][kk][1] = on ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + 2 * tg)) : 0u;
      }
    } else {
      uint2 v[8];
      uint32_t am = 0u;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        v[kk] = on ? __ldg(reinterpret_cast<const uint2*>(src + kk * 16 + 4 * tg)) : make_uint2(0u, 0u);
        const uint32_t w[2] = {v[kk].x, v[kk].y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
          am = max(am, lo < 0x7f80u ? lo : 0u);
          am = max(am, hi < 0x7f80u ? hi : 0u);
        }
      }
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int e = min(max((int)(am >> 7) - 141, -100), 113);   // largest * 2^-e in [2^14, 2^15)
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      f *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        q[nb][kk][0] = pack_f16x2(bf_lo(v[kk].x) * inv, bf_hi(v[kk].x) * inv);
        q[nb][kk][1] = pack_f16x2(bf_lo(v[kk].y) * inv, bf_hi(v[kk].y) * inv);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) rowc[nb][e] = __shfl_sync(0xffffffffu, f, 8 * tg + 4 * e);
  }
}

// D = A(16x16, row) * B(16x8, col) + D, fp16 inputs
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Running state of one warp's 8 NB rows: output, its reference (base-2
// logarithm), the softmax's reference and sum.  For codes the output's
// reference mo bounds z + log2(scale of v), so the weights that multiply the
// codes stay within fp16; for bf16 one reference serves both.  A lane holds
// rows 8 n + 2 tg + {0, 1}; o[n][c][e]: row 8 n + 2 tg + (e & 1), element
// 16 c + 2 gq + (e >> 1) (codes) or 16 c + 8 (e >> 1) + gq.
template <int NB>
struct RowState {
  float o[NB][8][4];
  float m[NB][2], l[NB][2], mo[NB][2];   // l: this lane's part of the sum
};

template <int NB>
__device__ __forceinline__ void state_init(RowState<NB>& st) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[nb][i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) st.m[nb][e] = st.mo[nb][e] = -INFINITY, st.l[nb][e] = 0.f;
  }
}

// Zeroes the halves of a pair of 16-bit values whose bit in `keep` is clear.
__device__ __forceinline__ uint32_t keep_halves(uint32_t v, bool lo, bool hi) {
  return v & ((lo ? 0x0000ffffu : 0u) | (hi ? 0xffff0000u : 0u));
}
// Whether either half is infinite or NaN (exponent bits `ex` all ones).
__device__ __forceinline__ uint32_t clean_halves(uint32_t v, uint32_t ex, bool& bad) {
  const bool lo = (v & ex) == ex, hi = ((v >> 16) & ex) == ex;
  bad |= lo || hi;
  return keep_halves(v, !lo, !hi);
}

// A reference rises only when a logit exceeds it by more than 2^kRwLazy, so
// the output is seldom scaled.  fp16 weights are at most 2^(kRwLift + kRwLazy)
// = 2^15 and keep what is within 2^-33 of the largest weight of their row.
constexpr float kRwLift = 9.f, kRwLazy = 6.f;

// An 8 x 8 block of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// One step over a slice of a tile (KS positions): scores, running maximum and
// sum, output.  The keys, then the output's elements, are on the 16-row side
// of the products and the query rows on the 8-column side, so a converted key
// or value serves all NB blocks of 8 rows and few rows leave no product empty
// (E4M3, rows on the 16-row side: one token of each of 8 x 32K positions 97 us
// for 95, of 8 x 2048 selected ones 15.4 for 14.4).  No lane needs another's
// maximum until a reference rises.
// tK, tV: the slice's first row, this kv head; rb: bytes from row to row; sK,
// sV: the scale bytes of this head in the slice's first row.  Key rbase + i is
// seen by row r when it is <= lim[r] (-1: never).
// EDGE: some key of the slice is not seen by some row.  Then V rows that no
// row sees are zeroed, and infinities and NaN in V are taken out of the
// product and added to the rows that see them only.
template <bool FP8, bool EDGE, int NB>
__device__ __forceinline__ void row_step(RowState<NB>& st, const uint32_t (&q)[NB][8][2], const float (&rowc)[NB][2],
                                         const uint8_t* tK, const uint8_t* tV, int rb, const uint8_t* sK,
                                         const uint8_t* sV, int rbase, const int (&lim)[NB][2], int top) {
  constexpr int KS = kRwKeys<FP8>, KH = KS / 16;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tg = lane & 3, mtx = lane >> 3;
  float sc[NB][KH][4], sd[KH][4];   // (one block: two sums a score, for products in flight)
#pragma unroll
  for (int kh = 0; kh < KH; ++kh)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sd[kh][e] = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) sc[nb][kh][e] = 0.f;
    }
  const uint8_t* kr = tK + ((mtx & 1) * 8 + (lane & 7)) * rb + (mtx >> 1) * 16;
  float kscale[KH][2], vexp[KH][2];
  if constexpr (FP8) {
#pragma unroll
    for (int c = 0; c < 8; c += 2)
#pragma unroll
      for (int kh = 0; kh < KH; ++kh) {   // 16 keys x 32 codes
        uint32_t w[4];                    // keys 0-7 and 8-15 of chunk c, then of chunk c + 1
        ldmatrix_x4(w[0], w[1], w[2], w[3], kr + kh * 16 * rb + c * 16);
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(w[i], a[i >> 1][i & 1], a[i >> 1][2 + (i & 1)]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_f16_16816(sc[nb][kh], a[0], q[nb][c][0], q[nb][c][1]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma_f16_16816(NB == 1 ? sd[kh] : sc[nb][kh], a[1], q[nb][c + 1][0], q[nb][c + 1][1]);
      }
    // lane l converts the scales of key l; each lane takes those of its keys
    const float ks = e8m0_value(sK[lane * rb]), ve = e8m0_exponent(sV[lane * rb]);
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        kscale[kh][h] = __shfl_sync(0xffffffffu, ks, kh * 16 + h * 8 + gq);
        vexp[kh][h] = __shfl_sync(0xffffffffu, ve, kh * 16 + h * 8 + gq);
      }
  } else {
#pragma unroll
    for (int kk = 0; kk < 8; kk += 2) {
      uint32_t a[4], b[4];   // keys 0-7 and 8-15, first and last 8 of 16 elements
      ldmatrix_x4(a[0], a[1], a[2], a[3], kr + kk * 32);
      ldmatrix_x4(b[0], b[1], b[2], b[3], kr + kk * 32 + 32);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_bf16_16816(sc[nb][0], a, q[nb][kk][0], q[nb][kk][1]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        mma_bf16_16816(NB == 1 ? sd[0] : sc[nb][0], b, q[nb][kk + 1][0], q[nb][kk + 1][1]);
    }
  }
  // base-2 logits; masked ones are -inf whatever the product was
  float mx[NB][2], mv[NB][2];
  bool up = false;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int row = 0; row < 2; ++row) mx[nb][row] = mv[nb][row] = -INFINITY;
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = e & 1, h = e >> 1;
        float z = (NB == 1 ? sc[nb][kh][e] + sd[kh][e] : sc[nb][kh][e]) * rowc[nb][row];
        if constexpr (FP8) z *= kscale[kh][h];
        if (EDGE) z = rbase + kh * 16 + h * 8 + gq <= lim[nb][row] ? z : -INFINITY;
        sc[nb][kh][e] = z;
        mx[nb][row] = fmaxf(mx[nb][row], z);
        // (an exponent that is NaN makes the weight NaN, not the reference)
        if constexpr (FP8) mv[nb][row] = fmaxf(mv[nb][row], z + vexp[kh][h]);
      }
#pragma unroll
    for (int row = 0; row < 2; ++row) {
      up |= mx[nb][row] > st.m[nb][row] + kRwLazy;
      if constexpr (FP8) up |= mv[nb][row] > st.mo[nb][row] + kRwLazy;
    }
  }
  if (__any_sync(0xffffffffu, up)) {   // a reference rises
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float alpha[2];
#pragma unroll
      for (int row = 0; row < 2; ++row) {
        alpha[row] = 1.f;
        float v = mx[nb][row], u = mv[nb][row];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          if constexpr (FP8) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
        }
        if (v > st.m[nb][row] + kRwLazy) {
          alpha[row] = ex2(st.m[nb][row] - v);
          st.m[nb][row] = v;
          st.l[nb][row] *= alpha[row];
        }
        if constexpr (FP8) {   // the output's own reference
          alpha[row] = 1.f;
          if (u > st.mo[nb][row] + kRwLazy) {
            alpha[row] = ex2(st.mo[nb][row] - u);
            st.mo[nb][row] = u;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[nb][c][e] *= alpha[e & 1];
    }
  }
  uint32_t pb[NB][KH][2];   // weights of 8 keys x 8 rows, as the products want them
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float mu[2], mo[2];
#pragma unroll
    for (int row = 0; row < 2; ++row) {
      mu[row] = st.m[nb][row] == -INFINITY ? 0.f : st.m[nb][row];
      mo[row] = (st.mo[nb][row] == -INFINITY ? 0.f : st.mo[nb][row]) - kRwLift;
    }
#pragma unroll
    for (int kh = 0; kh < KH; ++kh)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float wt[2];
#pragma unroll
        for (int row = 0; row < 2; ++row) {
          const float z = sc[nb][kh][2 * h + row];
          wt[row] = ex2(z - mu[row]);
          st.l[nb][row] += wt[row];
          if constexpr (FP8) {
            float zo = z + vexp[kh][h];
            if (EDGE) zo = z == -INFINITY ? -INFINITY : zo;   // (a masked row's scale may be NaN)
            wt[row] = ex2(zo - mo[row]);
          }
        }
        pb[nb][kh][h] = transpose_8x8(FP8 ? pack_f16x2(wt[0], wt[1]) : pack_bf16x2(wt[0], wt[1]));
      }
  }
  bool bad = false;
#pragma unroll
  for (int kh = 0; kh < KH; ++kh) {
    // V fragment registers hold keys 2 tg, 2 tg + 1 and those + 8
    const int k0 = rbase + kh * 16 + 2 * tg;
    const uint8_t* vr = tV + (kh * 16 + (mtx & 1) * 8 + (lane & 7)) * rb + (mtx >> 1) * 16;
#pragma unroll
    for (int c = 0; c < 8; c += FP8 ? 2 : 1) {
      uint32_t w[4];
      ldmatrix_x4_trans(w[0], w[1], w[2], w[3], vr + c * (FP8 ? 16 : 32));
#pragma unroll
      for (int i = 0; i < (FP8 ? 2 : 1); ++i) {
        uint32_t b[4];   // keys 0-7 and 8-15 of even codes, then of odd ones (bf16: of 8 elements, then the next)
        if constexpr (FP8) {
          e4m3x4_to_f16x4(__byte_perm(w[2 * i], 0u, 0x3120), b[0], b[2]);
          e4m3x4_to_f16x4(__byte_perm(w[2 * i + 1], 0u, 0x3120), b[1], b[3]);
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) b[h] = w[h];
        }
        if (EDGE) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int kb = k0 + (h & 1) * 8;
            b[h] = clean_halves(keep_halves(b[h], kb <= top, kb + 1 <= top), FP8 ? 0x7c00u : 0x7f80u, bad);
          }
        }
        const uint32_t a[4] = {b[0], b[2], b[1], b[3]};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if constexpr (FP8) mma_f16_16816(st.o[nb][c + i], a, pb[nb][kh][0], pb[nb][kh][1]);
          else mma_bf16_16816(st.o[nb][c], a, pb[nb][kh][0], pb[nb][kh][1]);
        }
      }
    }
  }
  if (EDGE && __any_sync(0xffffffffu, bad)) {
    // rare: infinities and NaN of V reach the rows that see their key
    for (int i = 0; i < KS; ++i) {
      if (rbase + i > top) break;
      const uint8_t* row = tV + (size_t)i * rb;
#pragma unroll
      for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = 16 * c + (FP8 ? 2 * gq + (e >> 1) : 8 * (e >> 1) + gq);
          float x;
          if constexpr (FP8) x = (row[d] & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000u) : 0.f;
          else x = bf_lo(reinterpret_cast<const uint16_t*>(row)[d]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            if (!isfinite(x) && rbase + i <= lim[nb][e & 1]) st.o[nb][c][e] += x;
        }
    }
  }
}

template <bool FP8, bool SPARSE, int NB>
__global__ void __launch_bounds__(kRwThreads, 1)
paged_attn_rows_kernel(const PagedArgs a, const RowsPlan pl, float* __restrict__ part_o, float* __restrict__ part_ml,
                       int* __restrict__ err) {
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kRwMaxStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kRwMaxStages);
  int* sh_plan = const_cast<int*>(abort_flag) + 1;                            // first item and its first tile
  long long* sh_scan = reinterpret_cast<long long*>(empty + kRwMaxStages + 2);   // a word per warp
  unsigned char* ring = smem + kRwBarBytes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rb = pl.row_bytes, R = pl.R;
  const size_t stage_bytes = 2 * (size_t)R * rb;
  if (threadIdx.x == 0) {
    for (int s = 0; s < pl.stages; ++s) {
      tc::mbar_init(&full[s], SPARSE ? 4 : 1);   // the warps that copy
      tc::mbar_init(&empty[s], kRwConsumers);
    }
    *abort_flag = 0;
    tc::fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  // ---- the CTA's share [lo, hi) of all tiles, and where it starts
  const int capacity = a.max_pages << a.page_shift;
  int p, tile;
  long long left;
  if (pl.P <= 32) {   // every warp works it out by itself
    const int n = lane < pl.P ? item_tiles<SPARSE>(a, pl, lane) : 0;
    long long before;
    const long long U = warp_scan(n, before), Weff = U < pl.W ? U : pl.W;
    if ((long long)blockIdx.x >= Weff) return;   // fewer tiles than CTAs
    const long long lo = floor_div(blockIdx.x * U, Weff);
    left = floor_div((blockIdx.x + 1) * U, Weff) - lo;
    p = __ffs(__ballot_sync(0xffffffffu, before <= lo && lo < before + n)) - 1;
    tile = (int)(lo - __shfl_sync(0xffffffffu, before, p));
  } else {
    const int per = (pl.P + kRwThreads - 1) / kRwThreads;
    const int p0 = min((int)threadIdx.x * per, pl.P), p1 = min(p0 + per, pl.P);
    int mine = 0;
    for (int i = p0; i < p1; ++i) mine += item_tiles<SPARSE>(a, pl, i);
    long long before;
    const long long U = block_scan<kRwThreads>(mine, before, sh_scan), Weff = U < pl.W ? U : pl.W;
    if ((long long)blockIdx.x >= Weff) return;
    const long long lo = floor_div(blockIdx.x * U, Weff);
    left = floor_div((blockIdx.x + 1) * U, Weff) - lo;
    if (before <= lo && lo < before + mine) {
      long long at = before;
      for (int i = p0; i < p1; ++i) {
        const int n = per == 1 ? mine : item_tiles<SPARSE>(a, pl, i);
        if (lo < at + n) {
          sh_plan[0] = i;
          sh_plan[1] = (int)(lo - at);
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    p = sh_plan[0], tile = sh_plan[1];
  }

  if (warp >= kRwConsumers) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRwOtherRegs));
    // pages are copied by one warp, selected rows by four: a warp issues a copy
    // every 55 clocks or so (8 x 2048 rows, E4M3: 22.3 us by one, 15.3 by four)
    const int pw = warp - kRwConsumers;
    if (!SPARSE && pw > 0) return;
    uint32_t fill = 0;
    const int page_mask = (1 << a.page_shift) - 1;
    bool ok = true;
    for (; left > 0 && ok; ++p, tile = 0) {
      const int keys = item_keys<SPARSE>(a, pl, p);
      const int tiles = tiles_of(keys, R);
      const int last = (int)min((long long)tiles, tile + left);
      if (tile >= last) continue;
      left -= last - tile;
      const int b = SPARSE ? p : p / pl.nrb;
      const int32_t* trow = a.table + (long long)b * a.max_pages;
      // dense: table entries e0 + lane of the tiles ahead, 32 at a time, the
      // next 32 loading while these are used; sparse: the positions of the
      // tile after the next and the pages of the next are loading while a
      // tile's copies are issued
      int e0 = 0, pg = 0, pg_next = 0;
      const int e_last = SPARSE ? 0 : (keys - 1) >> a.page_shift;
      constexpr int NI = kRwKeys<FP8> / 8;   // copies per lane: a tile has at most 8 slices
      int jn[NI] = {}, pn[NI] = {}, jnn[NI] = {};
      const int32_t* irow = SPARSE ? a.idx + (long long)b * a.k : nullptr;
      // copy c of a tile: row c / 2, of K or V
      auto row_of = [&](int i) { return (lane * 4 + pw + 128 * i) >> 1; };
      auto load_idx = [&](int (&j)[NI], int t) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = row_of(i), at = t * R + r;
          if (r < R && at < keys) {
            int v = __ldg(irow + at);
            if (v < 0 || v >= capacity) {
              if ((pw & 1) == 0) paged_note(a.dbg, kDbgPagedIndex, v, capacity);
              v = v < 0 ? 0 : capacity - 1;
            }
            j[i] = v;
          }
        }
      };
      auto load_pages = [&](int (&g)[NI], const int (&j)[NI], int t) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = row_of(i);
          if (r < R && t * R + r < keys) g[i] = __ldg(trow + (j[i] >> a.page_shift));
        }
      };
      if constexpr (SPARSE) {
        load_idx(jn, tile);
        load_pages(pn, jn, tile);
        if (tile + 1 < last) load_idx(jnn, tile + 1);
      } else {
        e0 = tile * R >> a.page_shift;
        pg = e0 + lane <= e_last ? __ldg(trow + e0 + lane) : 0;
        pg_next = e0 + 32 + lane <= e_last ? __ldg(trow + e0 + 32 + lane) : 0;
      }
      for (int t = tile; t < last; ++t) {
        const int s = (int)(fill % (uint32_t)pl.stages);
        const uint32_t use = fill / (uint32_t)pl.stages;
        if (use > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(&empty[s], (use - 1) & 1u, abort_flag, err, 21))) {
          ok = false;
          break;
        }
        unsigned char* stK = ring + (size_t)s * stage_bytes;
        unsigned char* stV = stK + (size_t)R * rb;
        const int rows = min(R, keys - t * R);   // rows past the last key stay as they are (masked)
        const int mine = SPARSE ? (rows + 1 - (pw >> 1)) / 2 : 2 * rows;   // rows this warp copies
        if (lane == 0) tc::mbar_arrive_expect_tx(&full[s], (uint32_t)mine * (uint32_t)rb);
        __syncwarp();
        if constexpr (SPARSE) {
          int jc[NI], pc[NI];
#pragma unroll
          for (int i = 0; i < NI; ++i) jc[i] = jn[i], pc[i] = pn[i], jn[i] = jnn[i];
          if (t + 1 < last) load_pages(pn, jn, t + 1);
          if (t + 2 < last) load_idx(jnn, t + 2);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int r = row_of(i);
            if (r < rows) {
              const int page = checked_page(pc[i], a.num_pages, pw & 1 ? nullptr : a.dbg);
              const long long off = (((long long)page << a.page_shift) + (jc[i] & page_mask)) * rb;
              if (pw & 1) tc::bulk_load(stV + (size_t)r * rb, a.vp + off, (uint32_t)rb, &full[s]);
              else tc::bulk_load(stK + (size_t)r * rb, a.kp + off, (uint32_t)rb, &full[s]);
            }
          }
        } else {
          // the tile is one piece of a page, or several whole pages
          const int j0 = t * R;
          const int piece = min(R, page_mask + 1);
          const int first = j0 >> a.page_shift, pages = (R + page_mask) >> a.page_shift;
          if (first >= e0 + 32) {
            e0 += 32;
            pg = pg_next;
            pg_next = e0 + 32 + lane <= e_last ? __ldg(trow + e0 + 32 + lane) : 0;
          }
          // (a tile's pages never straddle the window: both are powers of two)
          const int mine_pg = __shfl_sync(0xffffffffu, pg, (first - e0 + (lane & 15)) & 31);
          const int pi = lane & 15;
          const int r0 = pi * piece;
          if (pi < pages && r0 < rows) {
            const int page = checked_page(mine_pg, a.num_pages, a.dbg);
            const int n = min(piece, rows - r0);
            const long long off = (((long long)page << a.page_shift) + ((j0 + r0) & page_mask)) * rb;
            if (lane < 16) tc::bulk_load(stK + (size_t)r0 * rb, a.kp + off, (uint32_t)(n * rb), &full[s]);
            else tc::bulk_load(stV + (size_t)r0 * rb, a.vp + off, (uint32_t)(n * rb), &full[s]);
          }
        }
        ++fill;
      }
    }
    // every copy this warp issued lands before the CTA exits
    for (int s = 0; s < pl.stages; ++s) {
      if ((uint32_t)s < fill) {
        const uint32_t last_use = (fill - 1 - (uint32_t)s) / (uint32_t)pl.stages;
        if (!tc::mbar_wait_drain(&full[s], last_use & 1u) && err) atomicCAS(err, 0, 22);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRwConsumerRegs));
  const int gq = lane >> 2, tg = lane & 3;
  const int hs = warp / pl.wph, rs = warp % pl.wph;
  const bool active = hs < a.Hkv;
  RowState<NB> st;
  uint32_t qa[NB][8][2];
  float rowc[NB][2];
  uint32_t fill = 0;
  bool ok = true;
  for (; left > 0 && ok; ++p, tile = 0) {
    const int keys = item_keys<SPARSE>(a, pl, p);
    const int tiles = tiles_of(keys, R);
    const int last = (int)min((long long)tiles, tile + left);
    if (tile >= last) continue;
    left -= last - tile;
    int tok0 = p, ntok = 1, lim[NB][2];
    if constexpr (SPARSE) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) lim[nb][0] = lim[nb][1] = keys - 1;
    } else {
      const int b = p / pl.nrb, t0 = p % pl.nrb * pl.tb;
      const SeqSpan s = seq_span(a.q_start, a.kv_len, b, a.N, capacity);
      tok0 = s.begin + t0;
      ntok = min(pl.tb, min(s.len, a.max_q) - t0);
#pragma unroll
      for (int r = 0; r < 2 * NB; ++r)
        lim[r >> 1][r & 1] = min(s.pos0 + t0 + (8 * (r >> 1) + 2 * tg + (r & 1)) / a.G, keys - 1);
    }
    const int low = SPARSE ? keys - 1 : keys - ntok;   // the least position a row of the block ends at
    state_init(st);
    load_q_rows<FP8, NB>(qa, rowc, a, tok0, ntok, hs, active);
    for (int t = tile; t < last; ++t) {
      const int s = (int)(fill % (uint32_t)pl.stages);
      if (!__all_sync(0xffffffffu,
                      tc::mbar_wait(&full[s], (fill / (uint32_t)pl.stages) & 1u, abort_flag, err, 23))) {
        ok = false;
        break;
      }
      const int rbase = t * R + rs * kRwKeys<FP8>;
      if (active && rbase < keys) {
        const uint8_t* tK = ring + (size_t)s * stage_bytes + (size_t)(rs * kRwKeys<FP8>) * rb;
        const uint8_t* tV = tK + (size_t)R * rb;
        const int tail = a.Hkv * kPgD + hs, off = hs * (FP8 ? kPgD : 2 * kPgD);
        if (rbase + kRwKeys<FP8> - 1 > low)
          row_step<FP8, true, NB>(st, qa, rowc, tK + off, tV + off, rb, tK + tail, tV + tail, rbase, lim, keys - 1);
        else
          row_step<FP8, false, NB>(st, qa, rowc, tK + off, tV + off, rb, tK + tail, tV + tail, rbase, lim, keys - 1);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty[s]);
      ++fill;
    }
    if (active && ok) {
      // CTA c's partial of item p sits in slot p + c: the CTAs that meet item
      // p + 1 start at or after the last one that meets p, so slots never collide
      const long long slot = ((long long)p + blockIdx.x) * pl.wph + rs;
      const long long base = (slot * a.Hkv + hs) * pl.RB;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * nb + 2 * tg + e;
          float l = st.l[nb][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          if (r >= ntok * a.G) continue;
          float* po = part_o + (base + r) * kPgD;
          if constexpr (FP8) {
            // outputs go to the softmax's own reference m
            const float f = st.mo[nb][e] == -INFINITY ? 0.f : exp2f(st.mo[nb][e] - st.m[nb][e] - kRwLift);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<float2*>(po + c * 16 + 2 * gq) =
                  make_float2(st.o[nb][c][e] * f, st.o[nb][c][2 + e] * f);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              po[c * 16 + gq] = st.o[nb][c][e];
              po[c * 16 + 8 + gq] = st.o[nb][c][2 + e];
            }
          }
          if (gq == 0) *reinterpret_cast<float2*>(part_ml + (base + r) * 2) = make_float2(st.m[nb][e], l);
        }
    }
  }
}

// A contributor's weight against the reference m.  One that saw nothing (m
// -inf, l 0, o 0) has none, one whose visible logits are all NaN (m -inf, l NaN)
// has 1.  No contributor is left out for a weight of 0: 0 times a NaN or an
// infinity is NaN, as it is in the products of one contributor.
__device__ __forceinline__ float merge_weight(float2 ml, float m) {
  return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : exp2f(ml.x - m);
}

// out = sum_x w_x o_x / L, w_x = 2^(m_x - M), L = sum_x w_x l_x, M = max_x m_x
// over the contributors x of a row's block.  MANY: one CTA per token and 8
// query heads, a warp each; otherwise one CTA per row.
template <bool SPARSE, bool MANY>
__global__ void __launch_bounds__(kRwMergeThreads, MANY ? 3 : 4)
paged_attn_rows_merge_kernel(const PagedArgs a, const RowsPlan pl, const float* __restrict__ part_o,
                             const float* __restrict__ part_ml, const int* __restrict__ err) {
  constexpr int kWarps = kRwMergeThreads / 32;
  constexpr int kPre = 8;
  __shared__ long long sh_scan[kWarps], sh_at;
  __shared__ int sh_item[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hb = MANY ? (a.Hq + kWarps - 1) / kWarps : a.Hq;
  const int h = MANY ? blockIdx.x % hb * kWarps + warp : blockIdx.x % hb;
  int tok = blockIdx.x / hb, p_by = -1, t_by = 0;
  if (!SPARSE && pl.by_item) {
    p_by = tok / pl.tb, t_by = tok % pl.tb;
    const SeqSpan s = seq_span(a.q_start, a.kv_len, p_by / pl.nrb, a.N, a.max_pages << a.page_shift);
    const int t = p_by % pl.nrb * pl.tb + t_by;
    if (t >= min(s.len, a.max_q) || s.len > a.many) {
      pdl_wait();
      return;
    }
    tok = s.begin + t;
  }
  // the token's item, the tiles before it and in all
  auto holds = [&](int i, int& t) {   // whether item i holds the token, as its t-th
    t = t_by;
    if (SPARSE || pl.by_item) return i == (SPARSE ? tok : p_by);
    const SeqSpan s = seq_span(a.q_start, a.kv_len, i / pl.nrb, a.N, a.max_pages << a.page_shift);
    const int t0 = i % pl.nrb * pl.tb;
    t = tok - s.begin - t0;
    if (s.len > a.many) return false;   // the tensor cores' sequence: its tokens have their results
    return t >= 0 && t < pl.tb && t + t0 < min(s.len, a.max_q);
  };
  int p = -1, n_p = 0, t_p = 0;
  long long U, base_u = 0;
  if (pl.P <= 32) {   // every warp works it out by itself
    const int n = lane < pl.P ? item_tiles<SPARSE>(a, pl, lane) : 0;
    int t;
    const uint32_t hit = __ballot_sync(0xffffffffu, lane < pl.P && holds(lane, t));
    long long before;
    U = warp_scan(n, before);
    if (hit) {
      p = __ffs(hit) - 1;
      n_p = __shfl_sync(0xffffffffu, n, p);
      t_p = __shfl_sync(0xffffffffu, t, p);
      base_u = __shfl_sync(0xffffffffu, before, p);
    }
  } else {
    if (tid == 0) sh_item[0] = -1;
    const int per = (pl.P + kRwMergeThreads - 1) / kRwMergeThreads;
    const int p0 = min(tid * per, pl.P), p1 = min(p0 + per, pl.P);
    int mine = 0, mine_at = 0;
    for (int i = p0; i < p1; ++i) {
      const int n = item_tiles<SPARSE>(a, pl, i);
      int t;
      if (holds(i, t)) p = i, n_p = n, t_p = t, mine_at = mine;
      mine += n;
    }
    long long before;
    U = block_scan<kRwMergeThreads>(mine, before, sh_scan);
    if (p >= 0) {
      sh_item[0] = p;
      sh_item[1] = n_p;
      sh_item[2] = t_p;
      sh_at = before + mine_at;
    }
    __syncthreads();
    p = sh_item[0], n_p = sh_item[1], t_p = sh_item[2];
    base_u = sh_at;
  }
  if (p < 0) {   // of no sequence, or beyond the bound
    pdl_wait();
    return;
  }
  const int hs = min(h, a.Hq - 1) / a.G, row = t_p * a.G + h % a.G;
  const long long Weff = U < pl.W ? U : pl.W;
  // the CTA that owns unit u: the largest c with floor(c U / W) <= u
  const long long first = n_p ? floor_div((base_u + 1) * Weff - 1, U) : 0;
  const long long last_c = n_p ? floor_div((base_u + n_p) * Weff - 1, U) : -1;
  const int C = (int)(last_c - first + 1) * pl.wph;
  const long long xstride = (long long)a.Hkv * pl.RB;   // entries between consecutive contributors
  const long long e0 = (((long long)p + first) * pl.wph * a.Hkv + hs) * pl.RB + row;
  const float* pml = part_ml + e0 * 2;
  const float* po = part_o + e0 * kPgD;
  const long long at = (long long)tok * a.Hq + h;
  if constexpr (MANY) {
    if (h >= a.Hq) return;
    pdl_wait();
    pdl_launch_dependents();
    const bool failed = *err != 0;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < C; x0 += 32) {
      const int nx = min(32, C - x0);
      const float* ox = po + x0 * xstride * kPgD;
      float4 pre[kPre];
#pragma unroll
      for (int i = 0; i < kPre; ++i)
        if (i < nx) pre[i] = __ldcg(reinterpret_cast<const float4*>(ox + i * xstride * kPgD) + lane);
      const float2 ml = lane < nx ? __ldcg(reinterpret_cast<const float2*>(pml + (x0 + lane) * xstride * 2))
                                  : make_float2(-INFINITY, 0.f);
      const float m = fmaxf(M, warp_max(ml.x));
      const float w = merge_weight(ml, m);
      const float f = merge_weight(make_float2(M, L), m);
      M = m;
      L = weighted_sum(L, f, warp_sum(__fmul_rn(ml.y, w)), 1.f);
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      auto fold = [&](float4 ov, int i) {
        const float wt = __shfl_sync(0xffffffffu, w, i);
        acc.x = fmaf(ov.x, wt, acc.x);
        acc.y = fmaf(ov.y, wt, acc.y);
        acc.z = fmaf(ov.z, wt, acc.z);
        acc.w = fmaf(ov.w, wt, acc.w);
      };
#pragma unroll
      for (int i = 0; i < kPre; ++i)
        if (i < nx) fold(pre[i], i);
#pragma unroll 4
      for (int i = kPre; i < nx; ++i)
        fold(__ldcg(reinterpret_cast<const float4*>(ox + i * xstride * kPgD) + lane), i);
    }
    const bool none = L == 0.f;   // nothing to attend to
    const float inv = failed ? __int_as_float(0x7fc00000) : (none ? 0.f : 1.f / L);
    reinterpret_cast<uint2*>(a.out + at * kPgD)[lane] =
        none && !failed ? make_uint2(0u, 0u)
                        : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse != nullptr)
      a.lse[at] = failed ? __int_as_float(0x7fc00000) : (none ? -INFINITY : (M + log2f(L)) * kPgLn2);
    return;
  }
  __shared__ float wts[kRwMergeMaxC];
  __shared__ alignas(16) float red[kWarps][kPgD];   // (stored 16 bytes at a time)
  __shared__ float rmax[kWarps], rsum[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const float2 ml0 = tid < C ? __ldcg(reinterpret_cast<const float2*>(pml + (long long)tid * xstride * 2))
                             : make_float2(-INFINITY, 0.f);
  float4 pre[kPre];
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const int x = warp + kWarps * i;
    pre[i] = x < C ? __ldcg(reinterpret_cast<const float4*>(po + (long long)x * xstride * kPgD) + lane)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int failed = *err;
  float mloc = ml0.x;
  for (int x = tid + kRwMergeThreads; x < C; x += kRwMergeThreads)
    mloc = fmaxf(mloc, __ldcg(pml + (long long)x * xstride * 2));
  mloc = warp_max(mloc);
  if (lane == 0) rmax[warp] = mloc;
  __syncthreads();
  float M = rmax[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, rmax[w]);
  float lloc = 0.f;
  if (tid < C) {
    const float wv = merge_weight(ml0, M);
    wts[tid] = wv;
    lloc = ml0.y * wv;
  }
  for (int x = tid + kRwMergeThreads; x < C; x += kRwMergeThreads) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(pml + (long long)x * xstride * 2));
    const float wv = merge_weight(ml, M);
    wts[x] = wv;
    lloc = weighted_sum(lloc, 1.f, ml.y, wv);
  }
  lloc = warp_sum(lloc);
  if (lane == 0) rsum[warp] = lloc;
  __syncthreads();
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) L += rsum[w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fold = [&](float4 ov, float wt) {
    acc.x = fmaf(ov.x, wt, acc.x);
    acc.y = fmaf(ov.y, wt, acc.y);
    acc.z = fmaf(ov.z, wt, acc.z);
    acc.w = fmaf(ov.w, wt, acc.w);
  };
#pragma unroll
  for (int i = 0; i < kPre; ++i) {
    const int x = warp + kWarps * i;
    if (x < C) fold(pre[i], wts[x]);
  }
#pragma unroll 4
  for (int x = warp + kWarps * kPre; x < C; x += kWarps)
    fold(__ldcg(reinterpret_cast<const float4*>(po + (long long)x * xstride * kPgD) + lane), wts[x]);
  *reinterpret_cast<float4*>(&red[warp][lane * 4]) = acc;
  __syncthreads();
  if (tid < kPgD) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) o += red[w][tid];
    const bool none = L == 0.f;   // nothing to attend to
    const float res = none ? 0.f : o / L;
    // a kernel that gave up leaves NaN, so the failure is visible
    a.out[at * kPgD + tid] = failed ? (uint16_t)0x7fc0 : (uint16_t)(pack_bf16x2(res, 0.f) & 0xffffu);
    if (tid == 0 && a.lse != nullptr)
      a.lse[at] = failed ? __int_as_float(0x7fc00000) : (none ? -INFINITY : (M + log2f(L)) * kPgLn2);
  }
}

RowsPlan rows_plan(int fp8, int B, int Hkv, int G, int max_q) {
  RowsPlan pl;
  const int most = (fp8 ? kRwRows<true> : kRwRows<false>) / G;
  pl.nrb = (max_q + most - 1) / most;
  pl.tb = (max_q + pl.nrb - 1) / pl.nrb;
  pl.RB = pl.tb * G;
  pl.P = B * pl.nrb;
  pl.wph = kRwConsumers / Hkv;   // 8, 4, 2 or 1 for Hkv <= 8: tiles and pages are powers of two, neither
  pl.R = (fp8 ? kRwKeys<true> : kRwKeys<false>) * pl.wph;   // straddles the other
  pl.row_bytes = paged_row_bytes(fp8, Hkv);
  pl.by_item = false;
  const int stage = 2 * pl.R * pl.row_bytes;
  pl.stages = kRwStageBytes / stage < kRwMaxStages ? kRwStageBytes / stage : kRwMaxStages;
  pl.W = device_sm_count();
  if (pl.W > kRwMergeMaxC / pl.wph) pl.W = kRwMergeMaxC / pl.wph;
  return pl;
}

size_t align256p(size_t x) { return (x + 255) & ~size_t(255); }
constexpr size_t kRwHead = 256;   // the kernel error word

size_t rows_slots(const RowsPlan& pl, int Hkv) { return (size_t)(pl.P + pl.W) * pl.wph * Hkv * pl.RB; }

template <bool FP8, bool SPARSE>
cudaError_t launch_rows(const PagedArgs& a, void* parts, int* err, cudaStream_t st) {
  RowsPlan pl = rows_plan(FP8, a.B, a.Hkv, a.G, SPARSE ? 1 : a.max_q);
  const size_t slots = rows_slots(pl, a.Hkv);
  char* p = static_cast<char*>(parts);
  float* po = reinterpret_cast<float*>(p);
  float* pml = reinterpret_cast<float*>(p + align256p(slots * kPgD * 4));
  const size_t smem = kRwBarBytes + (size_t)pl.stages * 2 * pl.R * pl.row_bytes;
  auto kern = pl.RB <= 8    ? paged_attn_rows_kernel<FP8, SPARSE, 1>
              : pl.RB <= 16 ? paged_attn_rows_kernel<FP8, SPARSE, 2>
                            // (one token: 16 rows at most)
                            : paged_attn_rows_kernel<FP8, SPARSE, FP8 || SPARSE ? 2 : 3>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3((unsigned)pl.W), dim3(kRwThreads), smem, st, a, pl, po, pml, err);
  if (e != cudaSuccess) return e;
  constexpr int kWarps = kRwMergeThreads / 32;
  const long long by_item = (long long)pl.P * pl.tb;
  pl.by_item = !SPARSE && by_item < a.N;
  const long long tokens = pl.by_item ? by_item : a.N;
  if (tokens * a.Hq >= kRwMergeMany)
    e = launch_pdl(paged_attn_rows_merge_kernel<SPARSE, true>,
                   dim3((unsigned)(tokens * ((a.Hq + kWarps - 1) / kWarps))), dim3(kRwMergeThreads), 0, st, a, pl, po,
                   pml, err);
  else
    e = launch_pdl(paged_attn_rows_merge_kernel<SPARSE, false>, dim3((unsigned)(tokens * a.Hq)),
                   dim3(kRwMergeThreads), 0, st, a, pl, po, pml, err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

#ifdef SA_DEBUG
__device__ int g_paged_dbg[4];
#endif

cudaError_t paged_dbg_record(int** rec) {
  *rec = nullptr;
#ifdef SA_DEBUG
  return cudaGetSymbolAddress(reinterpret_cast<void**>(rec), g_paged_dbg);
#else
  return cudaSuccess;
#endif
}

cudaError_t paged_dbg_read(int* host4, bool reset) {
#ifdef SA_DEBUG
  cudaError_t e = cudaMemcpyFromSymbol(host4, g_paged_dbg, 4 * sizeof(int));
  if (e == cudaSuccess && reset) {
    const int zero[4] = {0, 0, 0, 0};
    e = cudaMemcpyToSymbol(g_paged_dbg, zero, sizeof(zero));
  }
  return e;
#else
  (void)reset;
  for (int i = 0; i < 4; ++i) host4[i] = 0;
  return cudaSuccess;
#endif
}

size_t paged_rows_part_bytes(int fp8, int B, int Hkv, int G, int max_q) {
  const RowsPlan pl = rows_plan(fp8, B, Hkv, G, max_q);
  const size_t slots = rows_slots(pl, Hkv);
  return align256p(slots * kPgD * 4) + align256p(slots * 2 * 4);
}

size_t paged_rows_workspace_bytes(int fp8, int B, int Hkv, int G, int max_q) {
  return kRwHead + paged_rows_part_bytes(fp8, B, Hkv, G, max_q);
}

cudaError_t launch_paged_rows(const PagedArgs& a, int fp8, void* parts, int* err, cudaStream_t st) {
  if (a.N <= 0) return cudaSuccess;
  if (a.idx != nullptr)
    return fp8 ? launch_rows<true, true>(a, parts, err, st) : launch_rows<false, true>(a, parts, err, st);
  return fp8 ? launch_rows<true, false>(a, parts, err, st) : launch_rows<false, false>(a, parts, err, st);
}

cudaError_t launch_paged_rows(const PagedArgs& a, int fp8, void* ws, cudaStream_t st) {
  return launch_paged_rows(a, fp8, static_cast<char*>(ws) + kRwHead, static_cast<int*>(ws), st);
}

// Chunks of few query rows per kv head go to the row kernel, which reads the
// cache once per 16 or 24 rows; longer ones to the tensor cores, which read it once
// per 256.  Measured, us (row kernel / tensor cores; all of the batch alike):
//   E4M3, 8 kv heads x 4:  20 rows, 4 x 16K positions   76 / 209
//                          64 rows, 4 x 16K             133 / 209
//                          128 rows, 1 x 4K             37 / 55;  256 rows 55 / 53
//   bf16, 8 kv heads x 4:  20 rows, 4 x 16K             74 / 127
//                          48 rows, 4 x 16K             119 / 131;  64 rows 156 / 133
// (E4M3 rows are converted for the tensor cores first, so they wait longer.)
static bool use_rows(int fp8, int G, int max_q) { return (long long)max_q * G <= (fp8 ? 128 : 48); }

// In a batch with a long chunk, sequences with one block of rows at most
// (decoding ones, short drafts) go to the row kernel all the same: a tile of
// 128 rows would be all but empty, and E4M3 rows would be converted for it.
// Measured, us (with / without), 32 heads over 8, a chunk of 512 of 2K beside
// 16 x 4K: E4M3 129 / 244, bf16 129 / 147; beside 63 x 4K: 244 / 741, 254 / 422.
// Two launches more cost 6 to 10 us when there is no such sequence, so chunks
// of 128 rows at most, which tend to be of one kind, go together (16 drafts of
// 40 rows, bf16: 78 / 68).
static int few_tokens(int B, int G, int max_q) { return B > 1 && (long long)max_q * G > 128 ? 16 / G : 0; }

size_t paged_attn_workspace_bytes(int fp8, int B, int max_q, long long capacity, int Hkv, int G) {
  if (use_rows(fp8, G, max_q)) return paged_rows_workspace_bytes(fp8, B, Hkv, G, max_q);
  const int few = few_tokens(B, G, max_q);
  return paged_tc_workspace_bytes(fp8, B, Hkv, G, max_q, capacity) +
         (few ? paged_rows_part_bytes(fp8, B, Hkv, G, few) : 0);
}

cudaError_t launch_paged_attn(const PagedArgs& a, int fp8, void* ws, cudaStream_t st) {
  if (use_rows(fp8, a.G, a.max_q)) return launch_paged_rows(a, fp8, ws, st);
  PagedArgs part = a;
  part.few = few_tokens(a.B, a.G, a.max_q);
  cudaError_t e = launch_paged_tc(part, fp8, ws, st);
  if (e != cudaSuccess || part.few == 0) return e;
  part.max_q = part.many = part.few;
  const long long capacity = (long long)a.max_pages << a.page_shift;
  char* parts = static_cast<char*>(ws) + paged_tc_workspace_bytes(fp8, a.B, a.Hkv, a.G, a.max_q, capacity);
  return launch_paged_rows(part, fp8, parts, static_cast<int*>(ws), st);
}

cudaError_t launch_paged_write(const uint16_t* k_new, const uint16_t* v_new, long long k_stride, long long v_stride,
                               const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int B, int N,
                               int max_pages, int num_pages, int page_shift, int Hkv, int fp8, uint8_t* kp,
                               uint8_t* vp, int* dbg, cudaStream_t st) {
  if (N <= 0) return cudaSuccess;
  const dim3 grid((unsigned)((N + 7) / 8));
  const cudaError_t e =
      launch_pdl(fp8 ? paged_write_kernel<true> : paged_write_kernel<false>, grid, dim3(256), 0, st, k_new, v_new,
                 k_stride, v_stride, q_start, kv_len, table, B, N, max_pages, num_pages, page_shift, Hkv, kp, vp, dbg);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_paged_gather(const uint8_t* kp, const uint8_t* vp, const int32_t* table, const int32_t* idx,
                                const int32_t* count, int B, int max_pages, int num_pages, int page_shift, int Hkv,
                                int k, int fp8, uint16_t* ko, uint16_t* vo, int* dbg, cudaStream_t st) {
  if (B <= 0) return cudaSuccess;
  const dim3 grid((unsigned)((k + 7) / 8), (unsigned)B);
  const cudaError_t e = launch_pdl(fp8 ? paged_gather_kernel<true> : paged_gather_kernel<false>, grid, dim3(256), 0,
                                   st, kp, vp, table, idx, count, max_pages, num_pages, page_shift, Hkv, k, ko, vo,
                                   dbg);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace sa

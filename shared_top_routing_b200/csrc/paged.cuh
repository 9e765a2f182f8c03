// Paged K/V cache: what the kernels of paged.cu and paged_tc.cu share.
//
// A pool is [num_pages, page_size, row] bytes; a cache row is one position of
// a sequence, all kv heads, K and V in pools of their own:
//   bf16   Hkv * 128 bf16 values, 16 zero bytes
//   E4M3   Hkv * 128 codes, Hkv scale bytes (E8M0: 2^(byte - 127)), zeros to
//          16 bytes; value = code * 2^(byte - 127)
// The 16 bytes at the end make a row the layout a tile has in shared memory:
// rows 16 bytes apart modulo 128 keep ldmatrix free of bank conflicts, so a
// run of rows is one bulk copy, and the scales travel with their codes.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {

constexpr int kPgD = 128;                  // head_dim
constexpr int kPgPad = 16;                 // bytes at the end of a row
constexpr float kPgLog2e = 1.4426950408889634f;
constexpr float kPgLn2 = 0.6931471805599453f;

__host__ __device__ __forceinline__ int paged_row_bytes(int fp8, int Hkv) {
  return Hkv * kPgD * (fp8 ? 1 : 2) + kPgPad;
}

// Debug builds: codes of the paged calls' own debug record, which
// sa_debug_read merges with the library's.
constexpr int kDbgPage = 5;         // a block table's page outside the pool
constexpr int kDbgPagedIndex = 6;   // a selected position outside the block table
// The record's device address on the current device, and its copy (cleared
// when asked to); null and zeros in release builds.
cudaError_t paged_dbg_record(int** rec);
cudaError_t paged_dbg_read(int* host4, bool reset);

// Debug builds record a bad page or position (code, two details) in `rec`
// (the device debug record) and go on; release builds do nothing.
__device__ __forceinline__ void paged_note(int* rec, int code, int a, int b) {
#ifdef SA_DEBUG
  if (rec != nullptr) {
    if (atomicCAS(&rec[0], 0, code) == 0) {
      rec[1] = a;
      rec[2] = b;
    }
    atomicAdd(&rec[3], 1);
  }
#else
  (void)rec, (void)code, (void)a, (void)b;
#endif
}

// A page id of a block table, clamped into the pool (a bad one is a caller
// error: a wrong page is read, nothing faults).
__device__ __forceinline__ int checked_page(int pg, int num_pages, int* rec) {
  if (pg < 0 || pg >= num_pages) {
    paged_note(rec, kDbgPage, pg, num_pages);
    pg = pg < 0 ? 0 : num_pages - 1;
  }
  return pg;
}

// 2^(byte - 127) as fp32 (E8M0: 255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : (b == 0u ? 0x00400000u : b << 23));
}
// byte - 127 as fp32 (255: NaN).
__device__ __forceinline__ float e8m0_exponent(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : (float)(int)b - 127.f;
}

// Four E4M3 codes (low byte first) -> four fp16 values in two words, exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two fp16 values -> two bf16 values times `s` (each product rounded once).
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h, float s) {
  float a, b;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(h));
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b * s), "f"(a * s));
  return r;
}
// 2^x (results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// a f + b w, both products rounded before the sum: the same bits whichever
// part comes first.
__device__ __forceinline__ float weighted_sum(float a, float f, float b, float w) {
  return __fadd_rn(__fmul_rn(a, f), __fmul_rn(b, w));
}

// Eight E4M3 codes times `s` -> eight bf16 values.
__device__ __forceinline__ uint4 e4m3x8_to_bf16x8(uint2 c, float s) {
  uint32_t r[4];
  e4m3x4_to_f16x4(c.x, r[0], r[1]);
  e4m3x4_to_f16x4(c.y, r[2], r[3]);
  return make_uint4(f16x2_to_bf16x2(r[0], s), f16x2_to_bf16x2(r[1], s), f16x2_to_bf16x2(r[2], s),
                    f16x2_to_bf16x2(r[3], s));
}

// The queries of sequence b: packed tokens [begin, begin + len), token t at
// position pos0 + t of the kv cached positions.  Whatever q_start and kv_len
// hold, begin and begin + len stay within [0, N] and kv within the table.
struct SeqSpan {
  int begin, len, kv, pos0;
};
__device__ __forceinline__ SeqSpan seq_span(const int32_t* __restrict__ q_start, const int32_t* __restrict__ kv_len,
                                            int b, int N, int capacity) {
  SeqSpan s;
  const int a = q_start[b], e = q_start[b + 1], kv = kv_len[b];
  s.begin = min(max(a, 0), N);
  s.len = min(max(e, s.begin), N) - s.begin;
  s.kv = min(max(kv, 0), capacity);
  s.pos0 = s.kv - s.len;
  return s;
}

// The sequence that token i belongs to (all lanes of a warp ask for the same
// token), or -1: the count of sequences that end at or before i, then a check.
__device__ __forceinline__ int seq_of_token(const int32_t* __restrict__ q_start, int B, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;   // the sequence lies in [lo, hi]
  while (hi > lo) {     // 32 probes a round: the ends of evenly spaced sequences
    const int span = hi - lo, step = (span + 31) / 32;
    const int probe = lo + lane * step + step - 1;
    const bool past = probe < hi && q_start[probe + 1] <= i;
    const int n = __popc(__ballot_sync(0xffffffffu, past));
    lo += n * step;
    if (lo >= hi) { lo = hi; break; }
    hi = min(hi, lo + step - 1);
  }
  if (lo >= B || q_start[lo] > i || q_start[lo + 1] <= i) return -1;
  return lo;
}

// What a paged attention call is given.
struct PagedArgs {
  const uint16_t* q = nullptr;      // [N, Hq, 128] bf16, tokens q_stride elements apart
  long long q_stride = 0;
  const int32_t* q_start = nullptr; // dense: [B + 1]
  const int32_t* kv_len = nullptr;  // dense: [B]
  const int32_t* idx = nullptr;     // sparse: [B, k] positions; count [B]
  const int32_t* count = nullptr;
  const uint8_t* kp = nullptr;      // pools
  const uint8_t* vp = nullptr;
  const int32_t* table = nullptr;   // [B, max_pages]
  int B = 0, N = 0, max_q = 0, max_pages = 0, num_pages = 0, page_shift = 0;
  int Hq = 0, Hkv = 0, G = 0, k = 0;
  int few = 0, many = 0x7fffffff;   // sequences of more than few (tensor cores) and at most many (rows) new tokens
  float qscale = 0.f;               // softmax scale * log2(e)
  uint16_t* out = nullptr;          // [N, Hq, 128]
  float* lse = nullptr;             // [N, Hq] or null
  int* dbg = nullptr;               // debug builds: the device debug record
};

// Launchers (paged.cu).
cudaError_t launch_paged_write(const uint16_t* k_new, const uint16_t* v_new, long long k_stride, long long v_stride,
                               const int32_t* q_start, const int32_t* kv_len, const int32_t* table, int B, int N,
                               int max_pages, int num_pages, int page_shift, int Hkv, int fp8, uint8_t* kp,
                               uint8_t* vp, int* dbg, cudaStream_t st);
cudaError_t launch_paged_gather(const uint8_t* kp, const uint8_t* vp, const int32_t* table, const int32_t* idx,
                                const int32_t* count, int B, int max_pages, int num_pages, int page_shift, int Hkv,
                                int k, int fp8, uint16_t* ko, uint16_t* vo, int* dbg, cudaStream_t st);
// Attention of few query rows per kv head (idx set: one token per sequence
// over selected rows; else a chunk of at most max_q tokens per sequence).
// parts: partial results, paged_rows_part_bytes; err: the kernel error word.
size_t paged_rows_part_bytes(int fp8, int B, int Hkv, int G, int max_q);
size_t paged_rows_workspace_bytes(int fp8, int B, int Hkv, int G, int max_q);   // the head with the word, and the parts
cudaError_t launch_paged_rows(const PagedArgs& a, int fp8, void* parts, int* err, cudaStream_t st);
cudaError_t launch_paged_rows(const PagedArgs& a, int fp8, void* ws, cudaStream_t st);
// Attention of many query rows per kv head on the tensor cores (paged_tc.cu).
size_t paged_tc_workspace_bytes(int fp8, int B, int Hkv, int G, int max_q, long long capacity);
cudaError_t launch_paged_tc(const PagedArgs& a, int fp8, void* ws, cudaStream_t st);
// Chunk attention: picks the kernels for the chunks' lengths.
size_t paged_attn_workspace_bytes(int fp8, int B, int max_q, long long capacity, int Hkv, int G);
cudaError_t launch_paged_attn(const PagedArgs& a, int fp8, void* ws, cudaStream_t st);

}  // namespace sa

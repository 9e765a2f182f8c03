// Attention of a chunk of new tokens over the paged cache on the tensor cores
// (tcgen05, sm_100a): many query rows per kv head.
//
// Mathematics: out_t = sum_{j <= p_t} softmax_j(scale q_t.k_j) v_j, one pass
// over the keys in tiles of 128 with a reference m and a sum l per row:
// S = Q K^T, P = 2^((S - m) c), l += sum P, O += P V (c = scale * log2 e);
// when m rises, l and O are scaled by 2^((m_old - m) c).  m rises only when a
// tile's maximum exceeds it by more than 8 / c (the sums stay far inside fp32
// and P, at most 2^8, keeps its relative precision in bf16), so a tile takes
// one pass and O is hardly ever scaled.
//
// Rows: the G query heads of a kv head times 128 / G tokens share a 128-row
// tile (they read the same keys); an item is two such tiles, A and B, of one
// sequence and kv head, with the key tiles up to its last token.  An item with
// tokens for one tile only lets A take its even key tiles and B its odd ones,
// and joins them at the end.  A and B alternate: while one's scores go through
// the softmax, the tensor core works for the other.
//
// Work: one CTA per SM.  Whole items, sorted by length, are dealt out forth
// and back when that loads the CTAs about evenly (2048 tokens of a prompt, 32
// heads over 8: 66 us, 104 us when cut; 8192 more of 65536: 7.1 ms, 8.5 ms,
// the CTAs at work on a head reading the same keys at about the same time).
// Otherwise - few or uneven items - the key tiles of all items form one list
// that is cut evenly; an item cut in pieces is joined by paged_tc_merge_kernel.
//
// E4M3 caches are first written out in bf16 (exact) by paged_window_kernel, a
// window of sequences or heads at a time, contiguous: a row is converted once
// instead of once per query tile (codes converted beside the products:
// 434 TFLOP/s).
//
// Bound: 4 * 128 flops per (row, key) on the tensor core, and as many clocks
// for the exponentials (128 x 256 of them per key tile at 16 per clock and SM,
// against 2048 clocks of MMA).
//
// CTA of 512 threads:
//   warps 0-3, 4-7   softmax of tile A, of tile B: one thread per row
//   warp 8           K and V tiles by TMA, a page (or half of one) at a time
//   warp 9           MMA issue; S and O in TMEM, P over S as the A operand
//   warp 10          Q tiles by TMA
//   warps 12-15      V rows no token of the item sees are zeroed, infinities
//                    and NaN in rows only some see are taken out and added
//                    to those rows' results at the end
#include <cudaTypedefs.h>

#include <climits>
#include <cstddef>
#include <mutex>

#include "paged.cuh"
#include "tc_common.cuh"

namespace sa {
namespace {

using namespace tc;

constexpr int kTcThreads = 512;
constexpr int kTile = 128;                      // rows of a q tile, keys of a key tile
constexpr uint32_t kHalfBytes = kTile * 128;    // 64 elements of 128 rows
constexpr uint32_t kTileBytes = 2 * kHalfBytes; // 128 x 128 bf16
constexpr int kStages = 2;
constexpr int kSoftmaxRegs = 152, kOtherRegs = 104;   // 2 * 152 + 2 * 104 = 4 * 128 per warpgroup at launch
constexpr int kBadRing = 8;                     // items whose bad-row masks are kept
constexpr int kBadTiles = 3;                    // key tiles a token of an item may not see in full
constexpr int kDealItems = 1024, kDealSlack = 4;   // whole items: per kv head at most; key tiles over the even share
constexpr int kStageRow = 80;                   // bytes of a staged output row: 64 and a pad

// Sequences [b0, b0 + nb) and kv heads [h0, h0 + nh) of a call; for E4M3 their
// rows in bf16, [nb][cap][nh * 128] (K and V).
struct TcPlan {
  int tpt, tpi, nqb, P;   // tokens per tile and item, items per sequence at most, items per kv head
  int W;                  // CTAs
  int b0, nb, h0, nh;
  long long cap;
  const uint16_t* kw;
  const uint16_t* vw;
};

// Where a CTA is in the list: sequence b0 + b.
struct TcIter {
  int b, qb, kvh, j0;   // j0 < 0: whole items dealt in turn, this one's round ~j0
  long long left;
};

struct TcBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], v_clean[kStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  alignas(16) uint32_t bad[kBadRing][kBadTiles][4];   // V rows with infinities or NaN, by key (read 16 bytes a time)
  long long scan[kTcThreads / 32];
  int peak[kTcThreads / 32];
  uint16_t order[kDealItems];   // dealt items from the longest
  TcIter iter[kTcThreads / 32];   // each warp's place: kept here, not in registers over an item's tiles
  int plan[4];
  uint32_t tmem_base;
  int abort;
};
constexpr int kBarBytes = 4096;
static_assert(sizeof(TcBars) <= kBarBytes && offsetof(TcBars, bad) % 16 == 0 && offsetof(TcBars, scan) % 8 == 0,
              "barrier block");

constexpr size_t kTcSmem = 1024 + 2 * kTileBytes + 2 * kStages * kTileBytes + kBarBytes + 8 * 32 * kStageRow;
static_assert(kTcSmem <= 227 * 1024 && 2 * kDealItems * 4 <= 8 * 32 * kStageRow, "shared memory");

// What a CTA's first piece is, for the merge.
struct TcPiece {
  int b, qb, kvh, j0, j1, n, valid, pad;
};

// A piece of an item: sequence b, block qb of tpi tokens, kv head h0 + kvh,
// key tiles [j0, j1) of its n.
struct TcItem {
  int b, qb, kvh;
  int tok0, ntA, ntB;   // first token (packed), tokens of tile A and B
  int pos0, top;        // position of the first token, keys the last one sees
  int n, j0, j1;
  int cntA, cntB;       // key tiles of A and B
  bool split;           // B's rows are A's, over the odd key tiles
  // the i-th key tile of A (x = 0) or B
  __device__ __forceinline__ int tile_of(int x, int i) const { return split ? j0 + 2 * i + x : j0 + i; }
  // first key tile that some token does not see in full
  __device__ __forceinline__ int first_masked() const { return pos0 < 0 ? 0 : (pos0 + 1) / kTile; }
};

// Key tiles below position end, one at least (end + kTile may pass 2^31).
__device__ __forceinline__ int tiles_upto(int end) {
  return max(1, (int)(((unsigned)max(end, 0) + (unsigned)kTile - 1u) / (unsigned)kTile));
}

// Tokens of block qb, and the key tiles up to its last; 0 when it has none.
__device__ __forceinline__ int item_span(const PagedArgs& a, const TcPlan& pl, int b, int qb, SeqSpan& s, int& nt) {
  s = seq_span(a.q_start, a.kv_len, b, a.N, a.max_pages << a.page_shift);
  const int n = s.len > a.few ? min(s.len, a.max_q) : 0, t0 = qb * pl.tpi;
  nt = min(pl.tpi, n - t0);
  if (nt <= 0) return 0;
  return tiles_upto(s.pos0 + t0 + nt);
}

// Dealt items: CTA c's r-th, items from the longest to the shortest, kv heads
// innermost, every other round backwards.  -1: there is none.
__device__ __forceinline__ int dealt(const TcPlan& pl, int cta, int r) {
  const int i = r * pl.W + (r & 1 ? pl.W - 1 - cta : cta);
  return i < pl.P * pl.nh ? i : -1;
}

// ALL: called by a whole warp (the place is the warp's).
template <bool ALL>
__device__ __forceinline__ bool next_item(const PagedArgs& a, const TcPlan& pl, const uint16_t* order, TcIter& place,
                                          TcItem& it) {
  TcIter c = place;
  if (ALL) __syncwarp();
  SeqSpan s;
  int nt, n, b, qb, kvh;
  const bool deal = c.j0 < 0;
  do {
    if (deal) {
      const int i = dealt(pl, blockIdx.x, ~c.j0--);
      if (i < 0) return false;
      const int p = order[i / pl.nh];
      b = p / pl.nqb, qb = p % pl.nqb, kvh = i % pl.nh;
    } else {
      if (c.left <= 0 || c.kvh >= pl.nh) return false;
      b = c.b, qb = c.qb, kvh = c.kvh;
    }
    n = item_span(a, pl, pl.b0 + b, qb, s, nt);
    if (deal && n == 0) return false;   // (the empty ones are the last)
    if (!deal && (n == 0 || ++c.qb == pl.nqb)) {   // this sequence's last
      c.qb = 0;
      if (++c.b == pl.nb) c.b = 0, ++c.kvh;
    }
  } while (n == 0);
  it.j0 = 0, it.j1 = n;
  if (!deal) {
    it.j0 = c.j0;
    it.j1 = (int)min((long long)n, c.j0 + c.left);
    c.left -= it.j1 - it.j0;
    c.j0 = 0;
  }
  if (!ALL || (threadIdx.x & 31) == 0) place = c;
  if (ALL) __syncwarp();
  it.b = pl.b0 + b, it.qb = qb, it.kvh = kvh;
  it.tok0 = s.begin + qb * pl.tpi;
  it.pos0 = s.pos0 + qb * pl.tpi;
  it.ntA = min(nt, pl.tpt);
  it.ntB = nt - it.ntA;
  it.top = max(it.pos0 + nt, 0);
  it.n = n;
  it.split = it.ntB == 0;
  const int len = it.j1 - it.j0;
  if (it.split) {
    it.cntA = (len + 1) / 2;
    it.cntB = len / 2;
  } else {
    const int nA = tiles_upto(it.pos0 + it.ntA);
    it.cntA = max(0, min(it.j1, nA) - it.j0);
    it.cntB = len;
  }
  return true;
}

// ---- instruction wrappers -------------------------------------------------

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 in, fp32 accumulate.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations in one instruction (sm_100).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Waits for this thread's TMEM loads; ties the 32 registers a load fills to
// the wait, so that nothing reads them before it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}

// A row of 128 scores in TMEM -> 2^(s qs + nm) as packed bf16, their sum and
// the largest score; columns beyond `last` count as -inf when MASKED.
template <bool MASKED>
__device__ __forceinline__ void exp_tile(uint32_t tS, float qs, float nm, int last, uint32_t (&p)[64], float& mx,
                                         float& sum) {
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t s[2][32];
  tmem_ld32(tS, s[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    tmem_ld_wait32(s[q & 1]);
    if (q < 3) tmem_ld32(tS + 32 * (q + 1), s[(q + 1) & 1]);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float2 v = make_float2(__uint_as_float(s[q & 1][2 * e]), __uint_as_float(s[q & 1][2 * e + 1]));
      if (MASKED) {
        v.x = 32 * q + 2 * e <= last ? v.x : -INFINITY;
        v.y = 32 * q + 2 * e + 1 <= last ? v.y : -INFINITY;
      }
      m4[e & 3] = fmaxf(fmaxf(m4[e & 3], v.x), v.y);
      v = fma2(v, make_float2(qs, qs), make_float2(nm, nm));
      v.x = ex2(v.x);
      v.y = ex2(v.y);
      acc[e & 1] = add2(acc[e & 1], v);
      p[16 * q + e] = pack_bf16x2(v.x, v.y);
    }
  }
  mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
  acc[0] = add2(acc[0], acc[1]);
  sum = acc[0].x + acc[0].y;
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// True in one lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_lane() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// A wait of a whole warp: every lane gets one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err,
                                          int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, code));
}

// A position's row of 128 bf16 values of one kv head of V.
template <bool LINEAR>
__device__ __forceinline__ const uint16_t* v_row(const uint8_t* __restrict__ vp, const int32_t* __restrict__ trow,
                                                 int pos, int page_shift, int num_pages, int rb) {
  if constexpr (LINEAR) {
    return reinterpret_cast<const uint16_t*>(vp + (long long)pos * rb);
  } else {
    const int pg = checked_page(__ldg(trow + (pos >> page_shift)), num_pages, nullptr);
    return reinterpret_cast<const uint16_t*>(
        vp + (((long long)pg << page_shift) + (pos & ((1 << page_shift) - 1))) * rb);
  }
}

// Rare: adds the infinities and NaN of the flagged V rows a token sees to its
// finished row (bf16) or partial row (fp32), whichever is given.  vp: the
// kv head's values in the pool, or in the sequence's window (LINEAR).
template <bool LINEAR>
__device__ __noinline__ void add_bad_rows(const uint8_t* __restrict__ vp, const int32_t* __restrict__ trow, int rb,
                                          int page_shift, int num_pages, int first_masked, const uint32_t* bad,
                                          int limit, uint16_t* out, float* part) {
  for (int i = 0; i < kBadTiles * kTile; ++i) {
    const int key = first_masked * kTile + i;
    if (key > limit) break;
    if (!((bad[i >> 5] >> (i & 31)) & 1u)) continue;
    const uint16_t* row = v_row<LINEAR>(vp, trow, key, page_shift, num_pages, rb);
    for (int d = 0; d < kPgD; ++d) {
      const float v = bf_lo(row[d]);
      if (isfinite(v)) continue;
      if (out) out[d] = (uint16_t)(pack_bf16x2(bf_lo(out[d]) + v, 0.f) & 0xffffu);
      else part[d] += v;
    }
  }
}

// ------------------------------------------------------------------ softmax

// Writes 64 bytes of each of a warp's 32 rows: lane r holds row r's (w), `at`
// is its place in 64-byte units (-1: no such row).  Through shared memory, so
// that four lanes write a row's 64 bytes side by side.
__device__ __forceinline__ void store_rows(unsigned char* stage, const uint32_t* w, int at, unsigned char* dst) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *reinterpret_cast<uint4*>(stage + lane * kStageRow + e * 16) =
        make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = e * 8 + (lane >> 2);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kStageRow + (lane & 3) * 16);
    const int to = __shfl_sync(0xffffffffu, at, r);
    if (to >= 0) *reinterpret_cast<uint4*>(dst + (long long)to * 64 + (lane & 3) * 16) = v;
  }
}

template <bool LINEAR>
__device__ __forceinline__ void softmax_role(const int x, const PagedArgs& a, const TcPlan& pl, TcIter& c, TcBars& bars,
                                             volatile int* abort_flag, int* err, float* part_o, float* part_ml,
                                             float* scratch, unsigned char* stage, uint32_t tmem) {
  const int row = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lanes = (uint32_t)(row & ~31) << 16;
  const uint32_t tS = tmem + x * kTile + lanes, tO = tmem + 2 * kTile + x * kTile + lanes;
  const float qs = a.qscale, lazy = fminf(8.f / qs, 1e30f);
  const int tr = row / a.G;   // this row's token in the tile
  const bool fits = row < pl.tpt * a.G;
  uint32_t ns = 0, no = 0, items = 0;   // key tiles and pieces so far
  TcItem it;
  for (; next_item<true>(a, pl, bars.order, c, it); ++items) {
    const int cnt = x ? it.cntB : it.cntA;
    const int nt = x && !it.split ? it.ntB : it.ntA;
    const int t = (x && !it.split ? pl.tpt : 0) + tr;   // token within the item
    const bool rowok = fits && tr < nt;
    const int limit = it.pos0 + t;
    const bool any = __any_sync(0xffffffffu, rowok);
    const int wmin = __reduce_min_sync(0xffffffffu, rowok ? limit : INT_MAX);
    float m = -INFINITY, l = 0.f;   // reference (of the scores), sum
    bool ok = __all_sync(0xffffffffu, *abort_flag == 0);
    for (int i = 0; i < cnt; ++i, ++ns) {
      const int kb = it.tile_of(x, i) * kTile;
      ok = warp_wait(&bars.s_full[x], ns & 1u, abort_flag, err, 34) && ok;
      if (ok && any) {
        tc_fence_after();
        // one pass with the reference so far; only when the tile's maximum
        // exceeds it by more than 2^8 (and for the first tile) a second pass
        const int last = limit - kb;   // columns beyond it are masked
        const bool masked = kb + kTile - 1 > wmin;
        uint32_t p[64];
        float sum;
        while (true) {
          const float nm = m == -INFINITY ? 0.f : -m * qs;
          float mx;
          if (masked) exp_tile<true>(tS, qs, nm, last, p, mx, sum);
          else exp_tile<false>(tS, qs, nm, last, p, mx, sum);
          const bool up = mx > m + lazy;
          if (!__any_sync(0xffffffffu, up)) break;
          const float f = up ? ex2((m - mx) * qs) : 1.f;   // 0 when nothing was seen before
          if (up) m = mx;
          l *= f;
          if (i > 0) {   // (the products before are done: the scores came after them)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * q, o);
              tmem_ld_wait32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tO + 32 * q, o);
            }
          }
        }
        l += sum;
        tmem_st32(tS, p);   // P over the scores
        tmem_st32(tS + 32, p + 32);
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[x]);
    }
    if (cnt > 0) {
      ok = warp_wait(&bars.o_full[x], no & 1u, abort_flag, err, 35) && ok;
      ++no;
      tc_fence_after();
    }
    if (m != -INFINITY) m *= qs;   // base-2 logarithm from here on
    const bool direct = it.j0 == 0 && it.j1 == it.n;
    const bool join = it.split && it.cntB > 0;
    if (x && it.split) {
      if (join) {   // B's share goes to A through the CTA's scratch rows
        if (ok && any) {
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * q, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              store_rows(stage, o + 16 * e, row * 8 + 2 * q + e, reinterpret_cast<unsigned char*>(scratch));
          }
          *reinterpret_cast<float2*>(scratch + kTile * kPgD + row * 2) = make_float2(m, l);
        }
        tc_fence_before();
        named_sync(1, 256);
        named_sync(2, 256);
      }
      continue;
    }
    // (a half or a piece that saw a key counts whatever its weight: 0 times a
    // NaN or an infinity is NaN, as it is within one product)
    const bool sawA = cnt > 0 && (m != -INFINITY || l != 0.f);
    bool sawB = false;
    float fA = 1.f, fB = 0.f;
    const float* other = scratch + (size_t)row * kPgD;
    if (join) {
      named_sync(1, 256);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(scratch + kTile * kPgD + row * 2));
      const float mb = ml.x, M = fmaxf(m, mb);
      sawB = mb != -INFINITY || ml.y != 0.f;
      fA = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - M);
      fB = mb == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2(mb - M);
      l = weighted_sum(l, fA, ml.y, fB);
      m = M;
    }
    const int tok = it.tok0 + t, head = (pl.h0 + it.kvh) * a.G + row % a.G;
    const long long orow = (long long)tok * a.Hq + head;
    // the piece's slot: 0 continues an item of the CTAs before, 1 is continued by the next
    const long long slot = 2ll * blockIdx.x + (it.j0 > 0 ? 0 : 1);
    float* part = part_o + slot * 2 * kTile * kPgD;
    const int prow = x * kTile + row;
    if (direct) {
      const bool none = l == 0.f;
      const float inv = none ? 0.f : 1.f / l;
      fA *= inv;
      fB *= inv;
    }
    if (any) {
      // (the item's first row of this warp is the base: rows of a warp lie
      // within 32-bit distances of 64-byte units)
      const long long base = __shfl_sync(0xffffffffu, orow, 0);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * q, o);
        tmem_ld_wait32(o);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = __float_as_uint(!ok ? __uint_as_float(0x7fc00000u) : sawA ? __uint_as_float(o[e]) * fA : 0.f);
        if (sawB) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(other + 32 * q) + e);
            o[4 * e] = __float_as_uint(fmaf(v.x, fB, __uint_as_float(o[4 * e])));
            o[4 * e + 1] = __float_as_uint(fmaf(v.y, fB, __uint_as_float(o[4 * e + 1])));
            o[4 * e + 2] = __float_as_uint(fmaf(v.z, fB, __uint_as_float(o[4 * e + 2])));
            o[4 * e + 3] = __float_as_uint(fmaf(v.w, fB, __uint_as_float(o[4 * e + 3])));
          }
        }
        if (direct) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          store_rows(stage, w, rowok ? (int)(orow - base) * 4 + q : -1,
                     reinterpret_cast<unsigned char*>(a.out + base * kPgD));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            store_rows(stage, o + 16 * e, rowok ? prow * 8 + 2 * q + e : -1, reinterpret_cast<unsigned char*>(part));
        }
      }
    }
    __syncwarp();   // a row is written by four lanes of the warp, and read again below by its own
    if (rowok) {
      if (!direct)
        *reinterpret_cast<float2*>(part_ml + (slot * 2 * kTile + prow) * 2) = make_float2(m, l);
      else if (a.lse != nullptr)
        a.lse[orow] = !ok ? __uint_as_float(0x7fc00000u) : (l == 0.f ? -INFINITY : (m + log2f(l)) * kPgLn2);
      const uint32_t(*bad)[4] = bars.bad[items % kBadRing];
      uint32_t flagged = 0u;
#pragma unroll
      for (int e = 0; e < kBadTiles; ++e) {
        const uint4 w = *reinterpret_cast<const uint4*>(bad[e]);
        flagged |= w.x | w.y | w.z | w.w;
      }
      if (flagged && ok) {
        const uint8_t* vp = LINEAR ? reinterpret_cast<const uint8_t*>(
                                         pl.vw + ((long long)(it.b - pl.b0) * pl.cap * pl.nh + it.kvh) * kPgD)
                                   : a.vp + (pl.h0 + it.kvh) * (2 * kPgD);
        add_bad_rows<LINEAR>(vp, a.table + (long long)it.b * a.max_pages,
                             LINEAR ? pl.nh * (2 * kPgD) : paged_row_bytes(0, a.Hkv), a.page_shift, a.num_pages,
                             it.first_masked(), bad[0], limit, direct ? a.out + orow * kPgD : nullptr,
                             part + (long long)prow * kPgD);
      }
    }
    tc_fence_before();   // O is read before the next item's first product overwrites it
    if (join) named_sync(2, 256);
  }
}

// --------------------------------------------------------------------- MMA

// Operand descriptors (128-byte swizzle, 8-row groups 1024 bytes apart): low
// words hold the start address in 16-byte units and a constant offset, high
// words are constant.  Q and K run along the reduction index in a row; V's
// reduction index runs over the rows, its next 64 columns are kHalfBytes on.
constexpr uint32_t kDescLoK = (16u >> 4) << 16;
constexpr uint32_t kDescLoV = (kHalfBytes >> 4) << 16;
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }

// One elected lane walks the items, waits and issues.  Waits cost a few hundred
// clocks each on this path, during which the tensor core runs dry, so each
// tile is waited for once (by the first of A and B that uses it) and before
// the wait for P, and a product pair O += P V, S = Q K'^T is issued in one go.
__device__ __forceinline__ void mma_role(const PagedArgs& a, const TcPlan& pl, TcIter& c, TcBars& bars,
                                         volatile int* abort_flag, int* err, uint32_t sQ, uint32_t sK, uint32_t sV,
                                         const uint32_t tmem) {
  constexpr uint32_t kIdS = idesc_bf16_f32(kTile, kTile);
  constexpr uint32_t kIdO = kIdS | (1u << 16);   // V: the reduction index is the row
  const uint32_t q_lo = kDescLoK | (sQ >> 4), k_lo = kDescLoK | (sK >> 4), v_lo = kDescLoV | (sV >> 4);
  uint32_t seq0 = 0, nq[2] = {0, 0}, np[2] = {0, 0};
  uint32_t k_seen = 0, v_seen = 0;   // key tiles known to be in shared memory
  TcItem it = {};
  bool ok = true;
  auto need_k = [&](uint32_t seq) {
    for (; k_seen <= seq; ++k_seen)
      ok = ok && mbar_wait(&bars.k_full[k_seen % kStages], (k_seen / kStages) & 1u, abort_flag, err, 36);
  };
  auto need_v = [&](uint32_t seq) {
    for (; v_seen <= seq; ++v_seen)
      ok = ok && mbar_wait(&bars.v_clean[v_seen % kStages], (v_seen / kStages) & 1u, abort_flag, err, 38);
  };
  // scores of tile x against the key tile `seq`
  auto qk = [&](int x, uint32_t seq) {
    const uint32_t s = seq % kStages;
    const uint32_t ql = q_lo + x * (kTileBytes >> 4), kl = k_lo + s * (kTileBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const uint32_t off = (((uint32_t)ks >> 2) * kHalfBytes + ((uint32_t)ks & 3u) * 32u) >> 4;
      umma_bf16(tmem + x * kTile, desc_of(ql + off), desc_of(kl + off), kIdS, ks > 0);
    }
    umma_commit(&bars.s_full[x]);
    if (x || it.split) umma_commit(&bars.k_empty[s]);
  };
  while (ok && next_item<false>(a, pl, bars.order, c, it)) {
    const int cnt[2] = {it.cntA, it.cntB};
    const int most = max(cnt[0], cnt[1]);
    const uint32_t mul = it.split ? 2u : 1u;   // tile i of A is mul * i, of B one on when split
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (cnt[x] == 0) continue;
      const uint32_t seq = seq0 + (it.split ? x : 0);
      ok = ok && mbar_wait(&bars.q_full[x], nq[x] & 1u, abort_flag, err, 37);
      ++nq[x];
      need_k(seq);
      if (!ok) break;
      tc_fence_after();
      qk(x, seq);
      if (cnt[x] == 1) umma_commit(&bars.q_empty[x]);
    }
    for (int i = 0; i < most && ok; ++i) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (i >= cnt[x]) continue;
        const uint32_t seq = seq0 + mul * i + (it.split ? x : 0), s = seq % kStages;
        const bool end = i + 1 == cnt[x];
        need_v(seq);
        if (!end) need_k(seq + mul);
        ok = ok && mbar_wait(&bars.p_full[x], np[x] & 1u, abort_flag, err, 40);
        if (!ok) break;
        ++np[x];
        tc_fence_after();
        const uint32_t vl = v_lo + s * (kTileBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_bf16_ts(tmem + 2 * kTile + x * kTile, tmem + x * kTile + ks * 8, desc_of(vl + ks * (2048u >> 4)), kIdO,
                       i > 0 || ks > 0);
        if (x || it.split) umma_commit(&bars.v_empty[s]);
        if (!end) qk(x, seq + mul);
        else umma_commit(&bars.o_full[x]);
        if (i + 2 == cnt[x]) umma_commit(&bars.q_empty[x]);   // the queries' last product
      }
    }
    seq0 += (uint32_t)(it.j1 - it.j0);
  }
  // everything issued is done before TMEM is freed (an abort by another warp
  // may still come after this one's last look at the flag)
  umma_commit(&bars.drain);
  if (!mbar_wait_drain(&bars.drain, 0) && err) atomicCAS(err, 0, 41);
}

// ------------------------------------------------------------------- kernel

template <bool LINEAR>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const PagedArgs a, const TcPlan pl,
                     TcPiece* __restrict__ pieces, float* __restrict__ part_o, float* __restrict__ part_ml,
                     float* __restrict__ scratch, int* __restrict__ err) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* sQ = base;                                   // tiles A, B
  unsigned char* sK = sQ + 2 * kTileBytes;
  unsigned char* sV = sK + kStages * kTileBytes;
  TcBars& bars = *reinterpret_cast<TcBars*>(sV + kStages * kTileBytes);
  unsigned char* stage = sV + kStages * kTileBytes + kBarBytes;   // output rows, a part per softmax warp
  volatile int* abort_flag = &bars.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 4);
      mbar_init(&bars.o_full[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.v_clean[i], 4);
    }
    mbar_init(&bars.drain, 1);
    bars.abort = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share of the key tiles of all items, kv heads outermost
  SeqSpan sp;
  int nt;
  const int per = (pl.P + kTcThreads - 1) / kTcThreads;
  const int p0 = min((int)threadIdx.x * per, pl.P), p1 = min(p0 + per, pl.P);
  int mine = 0, longest = 0;
  int* spans = reinterpret_cast<int*>(stage);   // (in use from here to the roles)
  for (int p = p0; p < p1; ++p) {
    const int n = item_span(a, pl, pl.b0 + p / pl.nqb, p % pl.nqb, sp, nt);
    mine += n;
    longest = max(longest, n);
    if (pl.P <= kDealItems) spans[p] = n;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  long long before = 0, S = 0;
  {
    long long v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) bars.scan[warp] = v, bars.peak[warp] = longest;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
#pragma unroll
    for (int w = 0; w < kTcThreads / 32; ++w) {
      if (w < warp) before += bars.scan[w];
      S += bars.scan[w];
      longest = max(longest, bars.peak[w]);
    }
    before += v - mine;
  }
  const long long U = S * pl.nh, Weff = U < pl.W ? U : pl.W;
  const bool idle = (long long)blockIdx.x >= Weff;
  const long long lo = idle ? 0 : blockIdx.x * U / Weff, hi = idle ? 0 : (blockIdx.x + 1) * U / Weff;
  const long long r = idle ? 0 : lo % S;
  // Whole items dealt to the CTAs instead, when the longest share exceeds the
  // even one by little: partial results written and joined take the time of
  // about 5 key tiles.
  auto even = [&](int load) { return (long long)(load - kDealSlack) * pl.W <= U + U / 16; };
  bool deal = pl.P <= kDealItems && even(longest);
  if (deal) {
    int* sorted = spans + kDealItems;
    for (int p = p0; p < p1; ++p) {
      const int n = spans[p];
      int rank = 0;
#pragma unroll 8
      for (int o = 0; o < pl.P; ++o) rank += spans[o] > n || (spans[o] == n && o < p);
      bars.order[rank] = (uint16_t)p;
      sorted[rank] = n;
    }
    __syncthreads();
    int load = 0;
    if ((int)threadIdx.x < pl.W)
      for (int i, k = 0; (i = dealt(pl, threadIdx.x, k)) >= 0; ++k) load += sorted[i / pl.nh];
    load = __reduce_max_sync(0xffffffffu, load);
    if (lane == 0) bars.peak[warp] = load;
    __syncthreads();
    for (int w = 0; w < kTcThreads / 32; ++w) load = max(load, bars.peak[w]);
    deal = even(load);
  }
  if (!idle && before <= r && r < before + mine) {
    long long at = before;
    for (int p = p0; p < p1; ++p) {
      const int n = item_span(a, pl, pl.b0 + p / pl.nqb, p % pl.nqb, sp, nt);
      if (r < at + n) {
        bars.plan[0] = p / pl.nqb;
        bars.plan[1] = p % pl.nqb;
        bars.plan[2] = (int)(r - at);
        break;
      }
      at += n;
    }
  }
  if (threadIdx.x == 0 && *err != 0) bars.abort = 1;   // an earlier call failed: every output shows it
  __syncthreads();
  const uint32_t tmem = bars.tmem_base;
  TcIter c0;
  c0.b = idle ? 0 : bars.plan[0];
  c0.qb = idle ? 0 : bars.plan[1];
  c0.kvh = idle ? 0 : (int)(lo / S);
  c0.j0 = deal ? -1 : idle ? 0 : bars.plan[2];
  c0.left = hi - lo;
  TcIter& c = bars.iter[warp];
  if (lane == 0) c = c0;
  __syncwarp();
  if (threadIdx.x == 0) {
    TcPiece pc = {};
    TcIter c2 = c0;
    TcItem it;
    if (!deal && next_item<false>(a, pl, bars.order, c2, it)) pc = {it.b, it.qb, it.kvh, it.j0, it.j1, it.n, 1, 0};
    pieces[blockIdx.x] = pc;
  }
  float* my_scratch = scratch + (size_t)blockIdx.x * kTile * (kPgD + 2);

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<LINEAR>(warp >> 2, a, pl, c, bars, abort_flag, err, part_o, part_ml, my_scratch,
                         stage + warp * 32 * kStageRow, tmem);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------- K and V loads
      uint32_t seq = 0, issued[2] = {0, 0};
      const int page_rows = LINEAR ? kTile : 1 << a.page_shift, piece = min(kTile, page_rows);
      const int pieces_per_tile = kTile / piece;
      const uint32_t piece_bytes = (uint32_t)piece * 128u;   // of one half
      TcItem it;
      bool ok = true;
      while (ok && next_item<true>(a, pl, bars.order, c, it)) {
        const int32_t* trow = a.table + (long long)it.b * a.max_pages;
        const int e_last = !LINEAR && it.top > 0 ? (it.top - 1) >> a.page_shift : 0;
        int e0 = it.j0 * kTile >> a.page_shift;
        int pg = 0, pg_next = 0;
        if constexpr (!LINEAR) {
          pg = e0 + lane <= e_last ? __ldg(trow + e0 + lane) : 0;
          pg_next = e0 + 32 + lane <= e_last ? __ldg(trow + e0 + 32 + lane) : 0;
        }
        for (int j = it.j0; j < it.j1 && ok; ++j, ++seq) {
          // lane: piece (lane / 2) % 16 of the tile, half lane % 2
          const int pi = lane >> 1, half = lane & 1;
          int y, live, xc;
          if constexpr (LINEAR) {
            live = 1;
            y = (int)((it.b - pl.b0) * pl.cap) + j * kTile;
            xc = it.kvh * kPgD + half * 64;
          } else {
            const int first = j * kTile >> a.page_shift;
            if (first >= e0 + 32) {
              e0 += 32;
              pg = pg_next;
              pg_next = e0 + 32 + lane <= e_last ? __ldg(trow + e0 + 32 + lane) : 0;
            }
            const int page = __shfl_sync(0xffffffffu, pg, (first - e0 + pi) & 31);
            // pieces past the last key any token sees are not read
            live = min(pieces_per_tile, max(0, (it.top - j * kTile + piece - 1) / piece));
            y = pi < live ? (checked_page(page, a.num_pages, a.dbg) << a.page_shift) +
                                (j * kTile + pi * piece & (page_rows - 1))
                          : 0;
            xc = (pl.h0 + it.kvh) * kPgD + half * 64;
          }
          const bool on = pi < live;
          const uint32_t s = seq % kStages;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            uint64_t* full = kv ? &bars.v_full[s] : &bars.k_full[s];
            if (seq >= kStages && !warp_wait(kv ? &bars.v_empty[s] : &bars.k_empty[s], (seq / kStages - 1) & 1u,
                                             abort_flag, err, 31)) {
              ok = false;
              break;
            }
            unsigned char* dst = (kv ? sV : sK) + s * kTileBytes + half * kHalfBytes + pi * piece_bytes;
            if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)live * piece_bytes * 2u);
            __syncwarp();
            if (on) tma_load_2d(dst, kv ? &map_v : &map_k, full, xc, y);
            issued[kv] = seq + 1;
          }
        }
      }
      // every copy issued lands before the CTA exits, whoever gives up later
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        for (uint32_t i = issued[kv] > kStages ? issued[kv] - kStages : 0; i < issued[kv]; ++i)
          if (!mbar_wait_drain(kv ? &bars.v_full[i % kStages] : &bars.k_full[i % kStages], (i / kStages) & 1u) && err)
            atomicCAS(err, 0, 44);
    } else if (warp == 9) {
      if (elect_lane()) mma_role(a, pl, c, bars, abort_flag, err, smem_u32(sQ), smem_u32(sK), smem_u32(sV), tmem);
      __syncwarp();
    } else if (warp == 10) {
      // ------------------------------------------------------------ Q loads
      if (lane == 0) {
        uint32_t nq[2] = {0, 0};
        const uint32_t bytes = (uint32_t)(pl.tpt * a.G) * 256u;
        TcItem it;
        bool ok = true;
        while (ok && next_item<false>(a, pl, bars.order, c, it)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || (x ? it.cntB : it.cntA) == 0) continue;   // (a split item's rows go to both)
            if (nq[x] > 0 && !mbar_wait(&bars.q_empty[x], (nq[x] - 1) & 1u, abort_flag, err, 32)) {
              ok = false;
              continue;
            }
            ++nq[x];
            mbar_arrive_expect_tx(&bars.q_full[x], bytes);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sQ + x * kTileBytes + h * kHalfBytes, &map_q, &bars.q_full[x], h * 64,
                          (pl.h0 + it.kvh) * a.G, it.tok0 + (it.split ? 0 : x * pl.tpt));
          }
        }
        for (int x = 0; x < 2; ++x)   // (as for K and V)
          if (nq[x] > 0 && !mbar_wait_drain(&bars.q_full[x], (nq[x] - 1) & 1u) && err) atomicCAS(err, 0, 45);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ------------------------------------------------------- V cleaning
    // Every tile is handed on from here, cleaned or not: these warps never
    // fall behind a barrier's phases.
    const int t = threadIdx.x & 127;   // row of the tile
    const uint32_t sw = (uint32_t)(t & 7);
    uint32_t seq = 0, items = 0;
    TcItem it;
    bool ok = true;
    for (; next_item<true>(a, pl, bars.order, c, it); ++items) {   // (after an abort too: the barrier below takes all four warps)
      uint32_t(*bad)[4] = bars.bad[items % kBadRing];
      if (t < kBadTiles * 4) bad[t >> 2][t & 3] = 0u;
      named_sync(3, 128);
      const int first_masked = it.first_masked();
      for (int j = it.j0; j < it.j1 && ok; ++j, ++seq) {
        const uint32_t s = seq % kStages;
        ok = warp_wait(&bars.v_full[s], (seq / kStages) & 1u, abort_flag, err, 33);
        if (!ok) break;
        const int key = j * kTile + t;
        unsigned char* vrow = sV + s * kTileBytes + (uint32_t)t * 128u;
        bool flag = false;
        if (j < first_masked) {   // seen by all: handed on as it is
        } else if (key >= it.top) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<uint4*>(vrow + (e >> 3) * kHalfBytes + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        } else if (key > it.pos0) {
#pragma unroll 4
          for (int e = 0; e < 16; ++e) {
            uint4* p = reinterpret_cast<uint4*>(vrow + (e >> 3) * kHalfBytes + (((uint32_t)e & 7u) ^ sw) * 16);
            const uint4 v = *p;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool hit = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if ((w[u] & 0x7f80u) == 0x7f80u) w[u] &= 0xffff0000u, hit = true;
              if ((w[u] & 0x7f800000u) == 0x7f800000u) w[u] &= 0x0000ffffu, hit = true;
            }
            if (hit) {
              *p = make_uint4(w[0], w[1], w[2], w[3]);
              flag = true;
            }
          }
        }
        if (flag) atomicOr(&bad[j - first_masked][t >> 5], 1u << (t & 31));
        if (j >= first_masked) fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.v_clean[s]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// The rows of E4M3 sequences [b0, b0 + nb) and kv heads [h0, h0 + nh) in
// bf16: one warp per position (K and V), the positions of all sequences dealt
// to the warps in turn (warps starting anew in every sequence: 155 us for 32
// of 1024 positions, 8 kv heads).  Bound by HBM: 258 bytes in and 512 out per
// position, kv head and cache.
__global__ void __launch_bounds__(256)
paged_window_kernel(const PagedArgs a, const TcPlan pl, uint16_t* __restrict__ kw, uint16_t* __restrict__ vw) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = blockIdx.x * 8 + (threadIdx.x >> 5), warps = gridDim.x * 8;
  const int rb = paged_row_bytes(1, a.Hkv), page_mask = (1 << a.page_shift) - 1;
  int skip = 0;   // positions before this sequence's, modulo the warps
  for (int g = 0; g < pl.nb; g += 32) {
    int kv_of = 0;   // positions of sequence b0 + g + lane, if it is one of these
    if (g + lane < pl.nb) {
      const SeqSpan s = seq_span(a.q_start, a.kv_len, pl.b0 + g + lane, a.N, a.max_pages << a.page_shift);
      kv_of = s.len > a.few ? s.kv : 0;
    }
    for (int i = 0; i < min(32, pl.nb - g); ++i) {
      const int n = __shfl_sync(0xffffffffu, kv_of, i);
      const int first = warp - skip + (warp < skip ? warps : 0);
      skip = (skip + n % warps) % warps;
      const int32_t* trow = a.table + (long long)(pl.b0 + g + i) * a.max_pages;
      for (unsigned pos = first; pos < (unsigned)n; pos += warps) {
        const int pg = checked_page(__ldg(trow + (pos >> a.page_shift)), a.num_pages, a.dbg);
        const long long off = (((long long)pg << a.page_shift) + (pos & page_mask)) * rb;
        const long long to = ((long long)(g + i) * pl.cap + pos) * pl.nh * kPgD;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint8_t* row = (kv ? a.vp : a.kp) + off;
          uint16_t* dst = (kv ? vw : kw) + to;
#pragma unroll
          for (int it = 0; it < 4; ++it) {   // 16 lanes per head, 8 codes per lane
            const int h = 2 * it + (lane >> 4), j = lane & 15;
            if (h >= pl.nh) break;
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(row + (pl.h0 + h) * kPgD) + j);
            const float sc = e8m0_value(row[a.Hkv * kPgD + pl.h0 + h]);
            reinterpret_cast<uint4*>(dst + h * kPgD)[j] = e4m3x8_to_bf16x8(c, sc);
          }
        }
      }
    }
  }
}

// Joins the pieces of items that several CTAs share.  Block (c, g): the item
// that CTA c is the first to continue; rows g * 32 .. + 31, four per warp.
__global__ void __launch_bounds__(256)
paged_tc_merge_kernel(const PagedArgs a, const TcPlan pl, const TcPiece* __restrict__ pieces,
                      const float* __restrict__ part_o, const float* __restrict__ part_ml,
                      const int* __restrict__ err) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x + 1;
  const TcPiece me = pieces[c], prev = pieces[c - 1];
  if (!me.valid || me.j0 == 0) return;
  auto same = [&](const TcPiece& o) { return o.valid && o.b == me.b && o.qb == me.qb && o.kvh == me.kvh; };
  if (same(prev) && prev.j0 > 0) return;   // not the first to continue it
  SeqSpan s;
  int nt;
  item_span(a, pl, me.b, me.qb, s, nt);
  constexpr int kRows = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = blockIdx.y * 32 + warp * kRows;
  long long at[kRows];
  bool on[kRows], any = false;
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    const int x = (row0 + q) >> 7, rr = (row0 + q) & 127, t = x * pl.tpt + rr / a.G;
    on[q] = rr < pl.tpt * a.G && t < nt;
    any |= on[q];
    at[q] = (long long)(s.begin + me.qb * pl.tpi + t) * a.Hq + (pl.h0 + me.kvh) * a.G + rr % a.G;
  }
  if (!any) return;
  float M[kRows], L[kRows];
  float4 o[kRows];
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    M[q] = -INFINITY;
    L[q] = 0.f;
    o[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // the beginning (slot 1 of CTA c - 1), then slot 0 of CTAs c .. to the one that ends the item
  int end = 0;
  for (int i = 0; end < me.n; ++i) {
    const long long slot = i == 0 ? 2ll * (c - 1) + 1 : 2ll * (c - 1 + i);
    float2 ml[kRows];
    float4 v[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const long long r = slot * 2 * kTile + row0 + q;
      ml[q] = on[q] ? __ldcg(reinterpret_cast<const float2*>(part_ml + r * 2)) : make_float2(-INFINITY, 0.f);
      v[q] = on[q] ? __ldcg(reinterpret_cast<const float4*>(part_o + r * kPgD) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    end = i == 0 ? me.j0 : pieces[c - 1 + i].j1;
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if (ml[q].x == -INFINITY && ml[q].y == 0.f) continue;   // this piece saw nothing (a NaN sum counts)
      const float m = fmaxf(M[q], ml[q].x);
      const float f = M[q] == -INFINITY ? (L[q] == 0.f ? 0.f : 1.f) : exp2f(M[q] - m);
      const float w = ml[q].x == -INFINITY ? 1.f : exp2f(ml[q].x - m);
      M[q] = m;
      // (a weight of 0 leaves nothing out: 0 times a NaN is NaN)
      L[q] = weighted_sum(L[q], f, ml[q].y, w);
      auto fold = [&](float acc, float x) { return weighted_sum(acc, f, x, w); };
      o[q].x = fold(o[q].x, v[q].x);
      o[q].y = fold(o[q].y, v[q].y);
      o[q].z = fold(o[q].z, v[q].z);
      o[q].w = fold(o[q].w, v[q].w);
    }
  }
  const bool failed = *err != 0;
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    if (!on[q]) continue;
    const bool none = L[q] == 0.f;
    const float inv = failed ? __uint_as_float(0x7fc00000u) : (none ? 0.f : 1.f / L[q]);
    reinterpret_cast<uint2*>(a.out + at[q] * kPgD)[lane] =
        make_uint2(pack_bf16x2(o[q].x * inv, o[q].y * inv), pack_bf16x2(o[q].z * inv, o[q].w * inv));
    if (lane == 0 && a.lse != nullptr)
      a.lse[at[q]] = failed ? __uint_as_float(0x7fc00000u) : (none ? -INFINITY : (M[q] + log2f(L[q])) * kPgLn2);
  }
}

// Windows of an E4M3 call hold at most this much (or one kv head of one
// sequence).
constexpr long long kWindowBytes = 1ll << 30;

TcPlan tc_plan(int fp8, int B, int Hkv, int G, int max_q, long long capacity) {
  TcPlan pl = {};
  pl.tpt = kTile / G;
  pl.tpi = 2 * pl.tpt;
  pl.nqb = (max_q + pl.tpi - 1) / pl.tpi;
  pl.W = device_sm_count();
  pl.cap = (capacity + kTile - 1) / kTile * kTile;
  pl.nb = B;
  pl.nh = Hkv;
  if (fp8) {
    const long long one = pl.cap * 4 * kPgD;   // K and V of one kv head of one sequence
    if (one * Hkv > kWindowBytes) {
      pl.nb = 1;
      pl.nh = (int)(kWindowBytes / one < 1 ? 1 : kWindowBytes / one);
    } else if (one * Hkv * B > kWindowBytes) {
      pl.nb = (int)(kWindowBytes / (one * Hkv));
    }
  }
  pl.P = pl.nb * pl.nqb;
  return pl;
}

constexpr size_t kTcHead = 256;   // the kernel error word
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
size_t tc_part_o_bytes(const TcPlan& pl) { return (size_t)pl.W * 2 * 2 * kTile * kPgD * 4; }
size_t tc_part_ml_bytes(const TcPlan& pl) { return (size_t)pl.W * 2 * 2 * kTile * 2 * 4; }
size_t tc_scratch_bytes(const TcPlan& pl) { return up256((size_t)pl.W * kTile * (kPgD + 2) * 4); }
size_t tc_pieces_bytes(const TcPlan& pl) { return up256(pl.W * sizeof(TcPiece)); }
size_t tc_window_bytes(const TcPlan& pl) { return (size_t)pl.nb * pl.cap * pl.nh * kPgD * 2; }   // K or V

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// q [N][Hq][128]: box of 64 elements x G heads x tpt tokens.
bool make_q_map(CUtensorMap* m, const PagedArgs& a, int tpt) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kPgD, (cuuint64_t)a.Hq, (cuuint64_t)a.N};
  cuuint64_t strides[2] = {(cuuint64_t)kPgD * 2, (cuuint64_t)a.q_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)a.G, (cuuint32_t)tpt};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K or V as [rows][row elements] (a pool, or a window): box of 64 values x
// `box_rows` rows.
bool make_kv_map(CUtensorMap* m, const void* p, long long rows, int row_elems, int row_bytes, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)row_elems, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t paged_tc_workspace_bytes(int fp8, int B, int Hkv, int G, int max_q, long long capacity) {
  const TcPlan pl = tc_plan(fp8, B, Hkv, G, max_q, capacity);
  return kTcHead + tc_pieces_bytes(pl) + tc_part_o_bytes(pl) + tc_part_ml_bytes(pl) + tc_scratch_bytes(pl) +
         (fp8 ? 2 * up256(tc_window_bytes(pl)) : 0);
}

cudaError_t launch_paged_tc(const PagedArgs& a, int fp8, void* ws, cudaStream_t st) {
  TcPlan pl = tc_plan(fp8, a.B, a.Hkv, a.G, a.max_q, (long long)a.max_pages << a.page_shift);
  char* p = static_cast<char*>(ws);
  int* err = reinterpret_cast<int*>(p);
  p += kTcHead;
  TcPiece* pieces = reinterpret_cast<TcPiece*>(p);
  p += tc_pieces_bytes(pl);
  float* po = reinterpret_cast<float*>(p);
  p += tc_part_o_bytes(pl);
  float* pml = reinterpret_cast<float*>(p);
  p += tc_part_ml_bytes(pl);
  float* scratch = reinterpret_cast<float*>(p);
  p += tc_scratch_bytes(pl);
  uint16_t* kw = reinterpret_cast<uint16_t*>(p);
  uint16_t* vw = reinterpret_cast<uint16_t*>(p + up256(tc_window_bytes(pl)));
  if (fp8) pl.kw = kw, pl.vw = vw;
  auto kern = fp8 ? paged_attn_tc_kernel<true> : paged_attn_tc_kernel<false>;
  cudaError_t e = ensure_dynamic_smem((const void*)kern, kTcSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!make_q_map(&mq, a, pl.tpt)) return cudaErrorInvalidValue;
  const int nb = pl.nb, nh = pl.nh;
  for (pl.h0 = 0; pl.h0 < a.Hkv; pl.h0 += nh)
    for (pl.b0 = 0; pl.b0 < a.B; pl.b0 += nb) {
      pl.nh = nh < a.Hkv - pl.h0 ? nh : a.Hkv - pl.h0;
      pl.nb = nb < a.B - pl.b0 ? nb : a.B - pl.b0;
      pl.P = pl.nb * pl.nqb;
      const int rows = fp8 ? kTile : 1 << a.page_shift, box = rows < kTile ? rows : kTile;
      const long long n = fp8 ? pl.nb * pl.cap : (long long)a.num_pages << a.page_shift;
      const int rb = fp8 ? pl.nh * kPgD * 2 : paged_row_bytes(0, a.Hkv);
      if (!make_kv_map(&mk, fp8 ? (const void*)kw : a.kp, n, rb / 2, rb, box) ||
          !make_kv_map(&mv, fp8 ? (const void*)vw : a.vp, n, rb / 2, rb, box))
        return cudaErrorInvalidValue;
      if (fp8) {
        e = launch_pdl(paged_window_kernel, dim3((unsigned)(8 * pl.W)), dim3(256), 0, st, a, pl, kw, vw);
        if (e != cudaSuccess) return e;
      }
      e = launch_pdl(kern, dim3((unsigned)pl.W), dim3(kTcThreads), kTcSmem, st, mq, mk, mv, a, pl, pieces, po, pml,
                     scratch, err);
      if (e != cudaSuccess) return e;
      if (pl.W > 1) {
        e = launch_pdl(paged_tc_merge_kernel, dim3((unsigned)(pl.W - 1), 2 * kTile / 32), dim3(256), 0, st, a, pl,
                       pieces, po, pml, err);
        if (e != cudaSuccess) return e;
      }
    }
  return cudaGetLastError();
}

}  // namespace sa

// Sparse core attention over an 8-bit K/V cache: E4M3 codes with one fp32
// scale per block of tokens and KV head.
//
// For query row t, KV head g and its group of query heads, over the visible
// entries j of the row's token list:
//     s_hj = scale * k_scale_j * (q_h . code(K_j)),  p = softmax_j(s_h),
//     out_h = sum_j p_hj v_scale_j code(V_j)
//
// Both products run on the tensor cores straight from the codes as they lie
// in memory, without widening them:
//  * 128 gathered list entries are the M side of S^T = K q^T, so TMEM lane =
//    entry and each thread owns one entry and the scores of all query heads.
//  * A 16-bit query element is split into E4M3 terms hi + lo / 16 (+ lo2 / 256
//    for fp16) after scaling its head by a power of two to at most 448; the
//    terms are separate N columns, recombined in fp32.  E4M3 holds 4
//    significant bits, so two terms hold a bf16 element exactly and three an
//    fp16 one, down to an absolute 2^-22 of the head's largest element.
//  * The output is O^T = V^T P: the V rows stay [entry][feature] in shared
//    memory and are read as an M-major operand (M = 128 features, two
//    halves), P as an N-major one, so that a thread writes its heads' codes in
//    16-byte stores.  The products p_hj v_scale_j are split into four terms the
//    same way: 2^-16 relative, 2^-22 of the head's largest product, well below the
//    16-bit output's rounding.  Four, not three, because the reference below may
//    lag by 2^8.75; the N columns of 8 or 12 heads, a multiple of 16, have room for
//    them anyway.
//  * Sums over entries are fp32: of the probabilities in registers, of the
//    output in TMEM and, when the reference moves, in registers.
//
// Work is the list of (row, KV head, 128-entry tile) triples in order; every CTA
// takes an equal contiguous run of it (two CTAs per SM), so any batch fills the
// GPU to one tile.  A run may begin and end inside a row's list: such pieces go
// to the workspace and finish_fp8_kernel merges them.  Inside a CTA
//  * warps 4-7 look entries up (list, page table) and gather their K and V rows
//    with 16-byte cp.async into three 32 KB buffers that K and V tiles take in
//    turn.  (TMA gathers are no match here: measured 10.7 cycles a 128-byte row
//    and SM for tile::gather4 and 27 a row for row-wise bulk copies, against 64
//    bytes a cycle and SM, 19 TB/s out of L2, for cp.async);
//  * warp 8 issues the MMAs, whichever product has its operands: S runs up to
//    S_BUFS tiles ahead of the softmax;
//  * warps 9-11 split each new row's queries;
//  * warps 0-3 run the softmax (thread = entry, then feature).  What is split into
//    terms is 2^(s + log2 v_scale - R), R a reference by head for the products: the
//    v_scales may differ by any factor, and a large one where nothing attends does
//    not push the others' products below what the terms hold.  R moves only when a
//    tile exceeds it by more than the terms have room for: until then a tile needs
//    no reduction, only a vote, and its output product adds up in TMEM.  The sum of
//    the probabilities takes the same exponentials over v_scale.  (Exponentials of
//    its own, 2^(s - M) with a second reference: 234 us in place of 210 for 1,024 rows.)
//
// Measured on B200 (24 / 2 heads, 2,051 entries a row): 16 requests x 4 rows
// 26.9 us with the merge (108 MB of distinct rows, 110 MB of DRAM reads; 16.5 us at
// the copy rate), one row 9.1 us, 1,024 rows 210 us (2.15 GB gathered out of L2: 10.2
// TB/s).  The last is near what shared memory carries: of about 1,650
// cycles a tile and SM, 512 write the gathered rows (128 bytes a cycle) and 670
// feed the MMAs (16 of M128 N32..48 K32, 42 to 45 cycles each alone), so the gather
// moves as little else through it as it can: 8 lanes copy both halves of a row, so
// that one shuffle serves two copies (204 us in place of 217 with 16 lanes a row, then).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.cuh"
#include "sm100.cuh"

namespace qsa {
namespace attn8 {

constexpr int D = 256;
constexpr int TILE = 128;              // list entries per tile (UMMA M)
constexpr int SOFT = 128;              // softmax threads: entry (scores), feature (output)
constexpr int PROD = 128;              // gathering threads
constexpr int THREADS = SOFT + PROD + 128;   // the last warpgroup: MMA issue, queries
// Registers a thread: 384 threads twice on an SM leave 80 each at launch; the
// warpgroups then share them out (the same sum of 240).
constexpr int REGS_LAUNCH = 80, REGS_SOFT = 152, REGS_PROD = 48, REGS_REST = 40;
static_assert(REGS_SOFT + REGS_PROD + REGS_REST <= 3 * REGS_LAUNCH, "setmaxnreg would wait for ever");
// log2 of a product p v_scale relative to its reference: the largest is brought to [0, 1) when the references move, and
// they move again above PROD_MOST (2^8.75 = 430; E4M3's largest value is 448).  The terms end at 2^-22.  (References 2^4
// lower, for products held to 2^-26 of the largest, move more often: 1,024 rows 248 us in place of 229 then.)
constexpr float PROD_MOST = 8.75f;
// Probabilities are added up as 2^(s - R + U), U = log2 of the largest v_scale in the tiles that moved the references,
// minus V_DROP.  The entry that R is from adds at least 2^-V_DROP, and one whose v_scale is 2^-d of that largest at
// most 2^(PROD_MOST + d - V_DROP): for d up to 190 and 2^20 entries both are fp32 numbers.  A product below 2^-126 is 0,
// which stands for a probability below 2^(d - 126) of the sum: from d = V_DROP on, exponentials of their own.
constexpr float V_DROP = 90.f;
constexpr float V_ZERO = -150.f;       // stands for log2 of a v_scale of 0: nothing that a 16-bit output holds
constexpr int MAX_GROUP = 16;          // query heads per KV head
constexpr int PT = 4;                  // E4M3 terms of a probability
constexpr int BUFS = 3;
constexpr int HALF_BYTES = TILE * 128;       // 128 features of every entry
constexpr int BUF_BYTES = 2 * HALF_BYTES;
constexpr int QC_SLOTS = 8;            // rows whose head factors are held: the current one and S_BUFS ahead fit
constexpr int Q_WARPS = 3;
constexpr size_t SMEM_OF_TWO = 233472 / 2 - 1024;   // dynamic shared memory of a CTA when two share an SM

// Sizes of one instance: 16-bit type and query heads held per KV head.
template <bool F16, int HG>
struct Cfg {
  static constexpr int QT = F16 ? 3 : 2;                          // E4M3 terms of a query element
  static constexpr int QCOLS = QT * HG, QN = (QCOLS + 15) / 16 * 16, QROWS = (QCOLS + 7) / 8 * 8;
  static constexpr int PCOLS = PT * HG, PN = (PCOLS + 15) / 16 * 16;
  static constexpr int S_BUFS = F16 ? 3 : 4;                      // score tiles held in TMEM
  static constexpr uint32_t TMEM = S_BUFS * QN + 2 * PN <= 256 ? 256 : 512;   // columns; two CTAs share 512
  static constexpr int Q_BYTES = QROWS * D;
  static constexpr int P_BYTES = PN * TILE;
  static constexpr int BARS = 2 * BUFS + 2 * S_BUFS + 5;
  // Scales of four tiles in shared memory, copied with the K rows, where two CTAs an SM leave room for them;
  // elsewhere the softmax threads look their entries up themselves.
  static constexpr size_t REST = BUFS * BUF_BYTES + Q_BYTES + P_BYTES + BARS * 8 + 4 * 17 * 4 + QC_SLOTS * HG * 4 + 16;
  static constexpr int RING_TILES = 4;
  static constexpr bool RING = REST + RING_TILES * TILE * 8 <= SMEM_OF_TWO;
  static constexpr int RING_BYTES = RING ? RING_TILES * TILE * 8 : 0;
  static constexpr size_t SMEM = REST + RING_BYTES;
  static_assert(TMEM == 256 || SMEM > SMEM_OF_TWO, "two CTAs would wait for each other's TMEM");
  static constexpr int RESIDENT = SMEM <= SMEM_OF_TWO ? 2 : 1;   // CTAs per SM
};

// n / d for 0 <= n < 2^31 as a product and a shift.
struct FastDiv {
  uint32_t mul;
  int32_t shift;
};
inline FastDiv fast_div(uint32_t d) {
  int l = 0;
  while ((uint64_t(1) << l) < d) ++l;
  return FastDiv{(uint32_t)(((uint64_t(1) << (31 + l)) + d - 1) / d), 31 + l};
}
__device__ __forceinline__ int divide(int n, FastDiv f) { return (int)(((uint64_t)(uint32_t)n * f.mul) >> f.shift); }

struct Params {
  const uint16_t* q;          // [T, Hq, 256] bf16 or fp16
  int64_t q_st, q_sh;
  int32_t Hq, Hkv, group;
  const uint8_t* k;           // E4M3 codes [pages, page_size, Hkv, 256]
  const uint8_t* v;
  const float* k_scale;       // [pages, page_size / block_tokens, Hkv]
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size;
  FastDiv by_page, by_block;  // / page_size, / block_tokens
  // Strides of the cache in rows of `pitch` bytes, the greatest common divisor
  // of the byte strides: a row's place is a 32-bit number.
  uint32_t pitch;
  int32_t page_rows, token_rows, head_rows;
  int64_t sc_page_stride, sc_block_stride;                // elements
  const int32_t* page_table;
  int64_t pt_stride;
  int32_t max_pages;
  const int32_t* cu;
  const int32_t* seq_lens;
  int32_t R;
  const int32_t* tok;
  int64_t tok_stride;
  int32_t width;
  int64_t T;
  int32_t tiles;              // tiles of one (row, KV head) pair
  int32_t ctas;               // runs: each has `per` units, the first `more` of them one more
  int32_t unit, per, more;    // a unit is one tile, or the tiles of a pair (no run then ends inside one)
  float scale_log2;
  float* part_o;              // [2 ctas, group, 256] unnormalised outputs of pairs cut by a run's ends
  float* part_ml;             // [2 ctas, group, 2] reference score (log2 units), sum
  float* part_d;              // [2 ctas, group] the outputs are 2^d times what they are relative to the reference score
  float* part_s;              // [T, Hq, width] scores (log2 units), or null
  float* lse2;                // [T, Hq] log2 of the sum of 2^s (of pairs that no run cuts), or null
  const float* gate;
  uint16_t* out;
  int64_t out_st;
  float* lse;
  float* weights;             // [T, width], or null
  int64_t w_stride;
  // the second launch: CTAs that add probabilities up, then `places` (pairs or cuts, whatever is fewer) per 2 heads
  int32_t sums, places;
};

// First tile of run i.
__device__ __forceinline__ int run_begin(const Params& p, int i) { return (i * p.per + min(i, p.more)) * p.unit; }
// The run that holds tile u.
__device__ __forceinline__ int run_of(const Params& p, int u) {
  const int v = u / p.unit, longer = p.more * (p.per + 1);
  return v < longer ? v / (p.per + 1) : p.more + (v - longer) / p.per;
}

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Shared-memory descriptor of an unswizzled N-major operand: cores of 8 K
// rows of 16 bytes, k8_stride bytes from one to the next along K and
// mn16_stride along N.  (The swizzled M-major operand, 128 bytes of M per K
// row and 8 rows per 1024-byte atom, has the fields of umma_desc_sw128.)
__device__ __forceinline__ uint64_t desc_plain_mn(uint32_t saddr, uint32_t k8_stride, uint32_t mn16_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(k8_stride >> 4) << 16;    // next 8 K
  d |= static_cast<uint64_t>(mn16_stride >> 4) << 32;  // next 16 bytes of M / N
  d |= static_cast<uint64_t>(1u) << 46;
  return d;
}

// kind::f8f6f4, E4M3 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}

// 32 lanes x 8 consecutive columns: thread i gets lane (base + i).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  static_assert(N % 8 == 0, "columns");
#pragma unroll
  for (int i = 0; i < N; i += 8) tmem_ld8(taddr + i, v + i);
}

__device__ __forceinline__ float log2_fast(float x) {   // 2 ulp (2^-22 for 0.5 to 2); log2(0) = -infinity
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp; 2^-inf = 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^n, n whole and between -126 and 127 (further out: the nearest of them)
__device__ __forceinline__ float power_of_two(float n) {
  return __int_as_float(((int)fminf(fmaxf(n, -126.f), 127.f) + 127) << 23);
}

__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
// Arrives on bar once this thread's cp.async copies so far have landed; the
// barrier counts this arrival like any other.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Whether any of the `threads` threads at barrier `id` says so.
__device__ __forceinline__ bool barrier_any(uint32_t id, uint32_t threads, bool says) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(says ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<const uint64_t*>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Two fp32 -> two E4M3 codes (nearest even, saturating); the low byte is a.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// ... and back (exact: every E4M3 value is an fp16 value).
__device__ __forceinline__ float2 e4m3x2_value(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Largest value over the warp (NaN ignored).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t x) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

template <bool F16>
__device__ __forceinline__ uint16_t narrow(float x) {
  if (F16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// attn::row_request, with position -1 (nothing visible) for the rows in front of
// the first request's and behind the last one's: the requests may be a slice of
// the batch, and a batch may be padded.
__device__ __forceinline__ void row_position(const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                                             int R, int64_t t, int lane, int& r, int& pos, int& L) {
  const int64_t begin = __ldg(cu);                     // row_request counts on a request that begins at or before t
  attn::row_request(cu, seq_lens, R, max(t, begin), lane, r, pos, L);
  if (t < begin || t >= (int64_t)__ldg(cu + r + 1)) pos = -1;
}

// The entries of consecutive tiles, looked up in stages so that no load is
// waited for: a tile's list entry two tiles and its page one tile before use.
// Every lane follows entry `entry` of the tile.
struct Feed {
  int t, g, tile;             // row, KV head and tile of the stage that loads list entries
  int left;                   // tiles of the run it has not loaded yet
  const int32_t* pt;          // the row's page table; last token it sees
  int last;
  int entry, lane;
  int jA, lastA, gA;          // list entry loaded
  const int32_t* ptA;
  int jB, pageB, lastB, gB;   // page loaded

  __device__ __forceinline__ void row(const Params& p) {
    int r, pos, L;
    row_position(p.cu, p.seq_lens, p.R, t, lane, r, pos, L);
    pt = p.page_table + (int64_t)r * p.pt_stride;
    last = min(pos, L - 1);
  }
  __device__ __forceinline__ int list_entry(const Params& p) {
    const int e = tile * TILE + entry;
    return e < p.width ? __ldg(p.tok + (int64_t)t * p.tok_stride + e) : -1;
  }
  // `first`: the list entry where it is loaded already
  __device__ __forceinline__ void load_entry(const Params& p, bool loaded = false, int first = -1) {
    lastA = last;
    gA = g;
    ptA = pt;
    jA = loaded ? first : left > 0 ? list_entry(p) : -1;
    if (left <= 0) return;
    --left;
    if (++tile == p.tiles) {
      tile = 0;
      if (++g == p.Hkv) {
        g = 0;
        ++t;
        if (left > 0) row(p);
      }
    }
  }
  __device__ __forceinline__ void load_page(const Params& p) {
    gB = gA;
    lastB = lastA;
    jB = jA;
    pageB = -1;
    if (jB >= 0) {                                     // what the row may see is checked later: `last` may be in flight
      const int lp = divide(jB, p.by_page);
      if (lp < p.max_pages) pageB = __ldg(ptA + lp);
    }
  }
  __device__ __forceinline__ void start(const Params& p, int pair, int tile_, int n, int entry_, int lane_) {
    entry = entry_;
    lane = lane_;
    tile = tile_;
    t = pair / p.Hkv;
    g = pair - t * p.Hkv;
    left = n;
    const int first = list_entry(p);                   // on its way while the row is looked up
    row(p);
    load_entry(p, true, first);
    load_page(p);
    load_entry(p);
  }
  // the next tile's entry: its page and token (page < 0: not visible)
  __device__ __forceinline__ void next(const Params& p, int& page, int& j, int& kv_head) {
    kv_head = gB;
    j = jB;
    page = jB <= lastB && (int64_t)pageB < p.num_pages ? pageB : -1;
    load_page(p);
    load_entry(p);
  }
};

__device__ __forceinline__ int64_t scale_index(const Params& p, int page, int in_page, int g) {
  return (int64_t)page * p.sc_page_stride + (int64_t)divide(in_page, p.by_block) * p.sc_block_stride + g;
}

template <int N>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool F16, int HG>
__global__ void __launch_bounds__(THREADS, (Cfg<F16, HG>::RESIDENT)) attn_fp8_kernel(const Params p) {
  using C = Cfg<F16, HG>;
  constexpr int QT = C::QT, QN = C::QN, PN = C::PN, S_BUFS = C::S_BUFS;
  constexpr uint32_t Q_HALF = C::QROWS * 128;
  constexpr uint32_t IDESC_S = idesc_e4m3(TILE, QN, false, false);
  constexpr uint32_t IDESC_O = idesc_e4m3(128, PN, true, true);
  extern __shared__ __align__(1024) uint8_t smem8[];   // the swizzle repeats every 1024 bytes
  uint8_t* buf_s = smem8;
  uint8_t* q_s = buf_s + BUFS * BUF_BYTES;             // [half][QROWS][128 bytes], swizzled; row = term * HG + head
  uint8_t* p_s = q_s + C::Q_BYTES;                     // [16 columns][entry][16 bytes]; column = term * HG + head
  float* sc_s = reinterpret_cast<float*>(p_s + C::P_BYTES);   // [RING_TILES][K, V][TILE] scales, 0 for unseen entries
  uint64_t* bars = reinterpret_cast<uint64_t*>(p_s + C::P_BYTES + C::RING_BYTES);
  uint64_t *kv_full = bars, *kv_empty = kv_full + BUFS, *s_full = kv_empty + BUFS, *s_empty = s_full + S_BUFS,
           *p_full = s_empty + S_BUFS, *o_full = p_full + 1, *q_full = o_full + 1, *q_empty = q_full + 1,
           *drained = q_empty + 1;
  float* red_s = reinterpret_cast<float*>(bars + C::BARS);  // [4 warps][17]: tile maxima by head, v_scale
  float* qc_s = red_s + 4 * 17;                        // [QC_SLOTS][HG]: a head's power of two times scale * log2(e)
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(qc_s + QC_SLOTS * HG);
  volatile int* abort = reinterpret_cast<int*>(tmem_s + 1);
  volatile int* add_s = abort + 1;                     // whether the next output product adds to what TMEM holds

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // they wait for this grid's end
  const int u0 = run_begin(p, blockIdx.x), n = run_begin(p, blockIdx.x + 1) - u0;
  const int pair0 = u0 / p.tiles, tile0 = u0 - pair0 * p.tiles;

  if (warp == 8) tmem_alloc(tmem_s, C::TMEM);
  if (tid == 0) {
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&kv_full[i], PROD);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < S_BUFS; ++i) {
      mbar_init(&s_full[i], 2);
      mbar_init(&s_empty[i], SOFT);
    }
    mbar_init(p_full, SOFT);
    mbar_init(o_full, 1);
    mbar_init(q_full, Q_WARPS * 32);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
    *abort = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  const uint32_t tm_o = tmem + S_BUFS * QN;                 // two halves of PN columns
  // A wait that runs out sets *abort.  Gathering and issuing warps then leave; the softmax warps go on through
  // their tiles without waiting, so that their barrier is always met.
  auto gone = [&]() {
    record_device_error(QSA_DEVERR_WAIT_TIMEOUT);
    *abort = 1;
  };

  if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- gather
    if constexpr (C::RESIDENT > 1) regs_shrink<REGS_PROD>();
    const int w = warp - 4;
    const int u = lane & 7, row4 = lane >> 3;          // 8 lanes a row (16 bytes of each half), 4 rows an instruction
    Feed f;
    f.start(p, pair0, tile0, n, 32 * w + lane, lane);
    // rows of the warp's 32 entries into the next buffer.  K goes one tile ahead of V: it is consumed as soon as it
    // lands, V only after the softmax.
    int item = 0;
    auto gather = [&](const uint8_t* base, int row, int tile, int64_t scale_at) -> bool {
      const int b = item % BUFS;
      if (!__all_sync(0xffffffffu, mbar_wait(&kv_empty[b], (uint32_t)((item / BUFS) & 1) ^ 1, abort))) return false;
      const uint32_t dst = smem_addr(buf_s + b * BUF_BYTES) + (32 * w + row4) * 128;
      const uint8_t* src = base + u * 16;
      if (C::RING && scale_at >= 0) {                  // the tile's scales land with its K rows
        const uint32_t at = smem_addr(sc_s + tile % C::RING_TILES * 2 * TILE + 32 * w + lane);
        cp_async4(at, p.k_scale + scale_at, row >= 0);
        cp_async4(at + TILE * 4, p.v_scale + scale_at, row >= 0);
      }
      int rr[8];                                       // all the look-ups before the copies
#pragma unroll
      for (int i = 0; i < 8; ++i) rr[i] = __shfl_sync(0xffffffffu, row, 4 * i + row4);
      const bool full = __all_sync(0xffffffffu, row >= 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t to = dst + i * 512 + ((u ^ (4 * (i & 1) + row4)) << 4);
        const uint8_t* from = src + (uint64_t)(uint32_t)max(rr[i], 0) * p.pitch;
        if (full) {
          cp_async16_all(to, from);
          cp_async16_all(to + HALF_BYTES, from + 128);
        } else {
          attn::cp_async16(to, from, rr[i] >= 0);
          attn::cp_async16(to + HALF_BYTES, from + 128, rr[i] >= 0);
        }
      }
      cp_async_arrive(&kv_full[b]);
      ++item;
      return true;
    };
    int row_v = -1;                                    // the last tile's row, whose V is still to come
    float held_v = 0.f;                                // and its k_scale: V codes of a block that holds nothing may
                                                       // be NaN, which no probability of 0 would hide
    auto gather_v = [&](int tile) { return gather(p.v, held_v != 0.f ? row_v : -1, tile, -1); };
    bool ok = true;
    for (int k = 0; k < n; ++k) {
      int page, j, g;
      f.next(p, page, j, g);
      const int in_page = j - divide(j, p.by_page) * p.page_size;
      const int row = page < 0 ? -1 : page * p.page_rows + in_page * p.token_rows + g * p.head_rows;
      const int64_t at = row >= 0 ? scale_index(p, page, in_page, g) : 0;
      const float held = row >= 0 ? __ldg(p.k_scale + at) : 0.f;
      ok = gather(p.k, row, k, at) && (k == 0 || gather_v(k - 1));
      if (!ok) break;
      row_v = row;
      held_v = held;
    }
    if (!ok || !gather_v(n - 1)) gone();
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 8) {
    // (one instruction for the warpgroup: its warps part only behind it)
    if constexpr (C::RESIDENT > 1) regs_shrink<REGS_REST>();
    if (warp == 8) {
      // ---------------------------------------------------------------- MMA issue
      // The whole warp goes round, so that descriptors stay in uniform registers; one lane issues.
      const uint64_t q_desc = umma_desc_sw128(smem_addr(q_s));
      const uint64_t kv_desc = umma_desc_sw128(smem_addr(buf_s));
      const uint64_t p_desc = desc_plain_mn(smem_addr(p_s), 128, TILE * 16);
      int ks = 0, ko = 0;                                // next tile of either product
      // K of tile k is item 2 k - 1 (0 for the first), V is item 2 k + 2 (2 n - 1 for the last)
      auto k_item = [](int k) { return k == 0 ? 0 : 2 * k - 1; };
      auto v_item = [&](int k) { return k + 1 < n ? 2 * k + 2 : 2 * n - 1; };
      int sb = 0;                                        // score buffer of ks and its phase
      uint32_t sp = 0;
      int tile = tile0, nth = 0;                         // of S: tile in its pair, pairs begun
      bool fresh = true;
      uint64_t since = global_timer_ns();
      uint32_t idle = 0;
      while (ko < n) {
        bool did = false;
        const int ki = k_item(ks), kb = ki % BUFS, vi = v_item(ko), vb = vi % BUFS;
        const uint32_t kp = (uint32_t)(ki / BUFS) & 1, vp = (uint32_t)(vi / BUFS) & 1;
        if (ko < ks && __all_sync(0xffffffffu, mbar_test(p_full, (uint32_t)ko & 1) &&
                                                   mbar_test(&kv_full[vb], vp))) {
          fence_proxy_async_smem();                      // the cp.async writes, before the tensor core reads them
          tc_fence_after();
          const bool add = *add_s != 0;
          const uint64_t vd = kv_desc + (uint32_t)(vb * (BUF_BYTES >> 4));
          if (elect_one()) {
  #pragma unroll
            for (int hf = 0; hf < 2; ++hf)
  #pragma unroll
              for (int s = 0; s < 4; ++s)
                mma_e4m3(tm_o + hf * PN, vd + hf * (HALF_BYTES >> 4) + s * (32 * 128 >> 4), p_desc + s * (32 * 16 >> 4),
                         IDESC_O, add || s > 0);
            umma_commit(&kv_empty[vb]);
            umma_commit(o_full);
          }
          __syncwarp();
          ++ko;
          did = true;
        }
        if (ks < n && ks < ko + S_BUFS &&
            __all_sync(0xffffffffu, mbar_test(&kv_full[kb], kp) &&
                                        mbar_test(&s_empty[sb], sp ^ 1) &&
                                        (!fresh || mbar_test(q_full, (uint32_t)nth & 1)))) {
          fence_proxy_async_smem();
          tc_fence_after();
          const uint64_t kd = kv_desc + (uint32_t)(kb * (BUF_BYTES >> 4));
          const uint32_t d = tmem + (uint32_t)sb * QN;
          const bool last = tile + 1 == p.tiles;
          if (elect_one()) {
  #pragma unroll
            for (int s = 0; s < 8; ++s)
              mma_e4m3(d, kd + (s >> 2) * (HALF_BYTES >> 4) + (s & 3) * 2, q_desc + (s >> 2) * (Q_HALF >> 4) + (s & 3) * 2,
                       IDESC_S, s > 0);
            umma_commit(&kv_empty[kb]);
            mbar_arrive(&s_full[sb]);                  // hands on what q_full published (the head factors)
            umma_commit(&s_full[sb]);
            if (last) umma_commit(q_empty);
          }
          __syncwarp();
          fresh = last;
          tile = last ? 0 : tile + 1;
          nth += last ? 1 : 0;
          ++ks;
          if (++sb == S_BUFS) {
            sb = 0;
            sp ^= 1;
          }
          did = true;
        }
        if (did) {
          idle = 0;
        } else if ((++idle & 63u) == 0) {
          if (idle == 64) since = global_timer_ns();
          if (__any_sync(0xffffffffu, *abort != 0 || global_timer_ns() - since > QSA_WAIT_TIMEOUT_NS)) {
            gone();
            if (elect_one()) umma_commit(drained);       // what was issued still ends before TMEM is freed
            mbar_wait(drained, 0, nullptr);
            break;
          }
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- queries: warp w takes heads w, w + 3, ...
      const int w = warp - 9;
      const int pairs = (tile0 + n - 1) / p.tiles + 1;
      for (int nth = 0; nth < pairs; ++nth) {
        const int64_t t = (pair0 + nth) / p.Hkv;
        const int g = pair0 + nth - (int)t * p.Hkv;
        const uint16_t* q_row = p.q + t * p.q_st + (int64_t)g * p.group * p.q_sh + lane * 8;
        constexpr int PER = (HG + Q_WARPS - 1) / Q_WARPS;
        uint4 x4[PER];                                   // read before the wait; heads past the group are zero
  #pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = w + Q_WARPS * i;
          x4[i] = make_uint4(0, 0, 0, 0);
          if (h < p.group) x4[i] = __ldg(reinterpret_cast<const uint4*>(q_row + h * p.q_sh));
        }
        if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (uint32_t)(nth & 1) ^ 1, abort))) {
          gone();
          break;
        }
  #pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int h = w + Q_WARPS * i;
          if (h >= HG) break;
          const uint32_t w4[4] = {x4[i].x, x4[i].y, x4[i].z, x4[i].w};
          // the head's largest magnitude, as a 16-bit pattern (NaN and infinity sort above every number)
          uint32_t top2 = 0;
  #pragma unroll
          for (int k = 0; k < 4; ++k) top2 = __vmaxu2(top2, w4[k] & 0x7fff7fffu);
          const uint32_t top16 = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
          const bool bad = top16 >= (F16 ? 0x7c00u : 0x7f80u);
          // the power of two that brings it into [224, 448]: 448 = 1.75 * 2^8
          const uint32_t tb = __float_as_uint(widen2<F16>(top16).x);
          const int e = max((int)(tb >> 23) - 127 - 8 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
          const float2 inv = both(bad ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - e) << 23));
          float2 y[4];
  #pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = mul2(widen2<F16>(w4[k]), inv);
          const int un = lane >> 1;                      // 16-byte unit of the row
  #pragma unroll
          for (int q = 0; q < QT; ++q) {
            uint32_t code[4];
  #pragma unroll
            for (int k = 0; k < 4; ++k) {
              code[k] = e4m3x2(y[k].x, y[k].y);
              if (q + 1 < QT) y[k] = fma2(e4m3x2_value(code[k]), both(-16.f), mul2(y[k], both(16.f)));
            }
            const int nr = q * HG + h;
            uint8_t* dst = q_s + (un >> 3) * Q_HALF + nr * 128 + (((un & 7) ^ (nr & 7)) << 4) + (lane & 1) * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(code[0] | (code[1] << 16), code[2] | (code[3] << 16));
          }
          if (lane == 0)
            qc_s[(nth % QC_SLOTS) * HG + h] =
                h < p.group ? p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23) : 0.f;
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    if constexpr (C::RESIDENT > 1) regs_grow<REGS_SOFT>();
    const uint32_t tm_lane = (uint32_t)(warp * 32) << 16;
    Feed f;
    if constexpr (!C::RING) f.start(p, pair0, tile0, n, tid, lane);
    // heads 2 i, 2 i + 1: sums over this thread's entries; features tid and 128 + tid
    float2 l_run[HG / 2], o0[HG / 2], o1[HG / 2];
    // References, same in every thread and whole numbers, so that moving them rounds nothing however often they move:
    // of the products, by head (negated), and U.
    float2 nref[HG / 2];
    float vsum = 0.f;
    bool set = false;                                  // the references hold maxima: a tile had a visible entry
    bool add = false;                                  // TMEM holds output of this pair that o0, o1 lack
    int pair = pair0, tile = tile0, nth = 0;
    int sb = 0;                                        // score buffer and its phase
    uint32_t sp = 0;
    bool fresh = true;
    // scales of the next tile's entry: loaded one tile ahead
    float ks_nx = 0.f, vs_nx = 0.f;
    auto scales = [&]() {
      int page, j, g;
      f.next(p, page, j, g);
      ks_nx = vs_nx = 0.f;
      if (page >= 0) {
        const int64_t at = scale_index(p, page, j - divide(j, p.by_page) * p.page_size, g);
        ks_nx = __ldg(p.k_scale + at);
        vs_nx = __ldg(p.v_scale + at);
      }
    };
    if constexpr (!C::RING) scales();
    auto output_done = [&](int k) {                // tile k's product is in TMEM, its P free
      if (!mbar_wait(o_full, (uint32_t)k & 1, abort)) gone();
      tc_fence_after();
    };
    auto take_output = [&]() {                         // o += what TMEM holds
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float d[(C::PCOLS + 7) / 8 * 8];
        tmem_ld(tm_o + tm_lane + hf * PN, d);
        tmem_wait_ld();
        float2* o = hf == 0 ? o0 : o1;
#pragma unroll
        for (int i = 0; i < HG / 2; ++i) {
          float2 x = make_float2(d[2 * i], d[2 * i + 1]);
          x = fma2(make_float2(d[HG + 2 * i], d[HG + 2 * i + 1]), both(1.f / 16.f), x);
          x = fma2(make_float2(d[2 * HG + 2 * i], d[2 * HG + 2 * i + 1]), both(1.f / 256.f), x);
          x = fma2(make_float2(d[3 * HG + 2 * i], d[3 * HG + 2 * i + 1]), both(1.f / 4096.f), x);
          o[i] = add2(o[i], x);
        }
      }
    };
    for (int k = 0; k < n; ++k) {
      bool seen;
      float ks = ks_nx, vs = vs_nx;
      float lvs;                                       // log2 v_scale, to 2 ulp
      float2 x[HG / 2];                                // log2 of the products, relative to their references
      {
        if (!mbar_wait(&s_full[sb], sp, abort)) gone();
        tc_fence_after();
        if constexpr (C::RING) {
          const float* sc = sc_s + k % C::RING_TILES * 2 * TILE + tid;
          ks = sc[0];
          vs = sc[TILE];
        }
        // unseen entries come with scales of 0, and a k_scale of 0 marks a block that holds nothing
        seen = ks != 0.f;
        lvs = seen ? max_or_nan(log2_fast(vs), V_ZERO) : 0.f;
        if (fresh) {
#pragma unroll
          for (int i = 0; i < HG / 2; ++i) nref[i] = l_run[i] = o0[i] = o1[i] = make_float2(0.f, 0.f);
          add = set = false;
        }
        const float2* qc = reinterpret_cast<const float2*>(qc_s + (nth % QC_SLOTS) * HG);
        float d[(C::QCOLS + 7) / 8 * 8];
        tmem_ld(tmem + tm_lane + (uint32_t)sb * QN, d);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&s_empty[sb]);
        if (++sb == S_BUFS) {
          sb = 0;
          sp ^= 1;
        }
#pragma unroll
        for (int i = 0; i < HG / 2; ++i) {
          x[i] = fma2(make_float2(d[HG + 2 * i], d[HG + 2 * i + 1]), both(1.f / 16.f), make_float2(d[2 * i], d[2 * i + 1]));
          if (QT > 2)
            x[i] = fma2(make_float2(d[(QT - 1) * HG + 2 * i], d[(QT - 1) * HG + 2 * i + 1]), both(1.f / 256.f), x[i]);
          x[i] = fma2(x[i], mul2(qc[i], both(ks)), add2(nref[i], both(lvs)));
        }
        if (!__all_sync(0xffffffffu, seen)) {
#pragma unroll
          for (int i = 0; i < HG / 2; ++i)
            if (!seen) x[i] = make_float2(-INFINITY, -INFINITY);
        }
      }
      if (p.part_s) {
        const int e = tile * TILE + tid;
        if (e < p.width) {
          float* dst = p.part_s + (int64_t)pair * p.group * p.width + e;
#pragma unroll
          for (int i = 0; i < HG / 2; ++i) {
            const float2 at = add2(nref[i], both(lvs));
            if (2 * i < p.group) dst[(int64_t)(2 * i) * p.width] = x[i].x - at.x;
            if (2 * i + 1 < p.group) dst[(int64_t)(2 * i + 1) * p.width] = x[i].y - at.y;
          }
        }
      }
      float over = -INFINITY;
#pragma unroll
      for (int i = 0; i < HG / 2; ++i) {
        over = fmaxf(over, fmaxf(x[i].x, x[i].y));
      }
      if (barrier_any(1, SOFT, !set || over > PROD_MOST)) {
        // ---- new references: the tile's maxima where they are larger
        auto maximum = [&](const float* at) { return floorf(fmaxf(fmaxf(at[0], at[17]), fmaxf(at[34], at[51]))); };
        float mine = -INFINITY;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float wm = warp_max(h & 1 ? x[h / 2].y - nref[h / 2].y : x[h / 2].x - nref[h / 2].x);
          if (lane == h) mine = wm;
        }
        const float vm = warp_max(seen ? lvs : -INFINITY);
        if (lane == 16) mine = vm;
        if (lane <= 16) red_s[warp * 17 + lane] = mine;
        named_barrier_sync(2, SOFT);
        if (add) {
          output_done(k - 1);
          take_output();
          add = false;
        }
        const bool was_set = set;
        const float was = vsum, top = maximum(red_s + 16) - V_DROP;
        if (top > -INFINITY) {                         // something is visible
          vsum = set ? fmaxf(vsum, top) : top;
          set = true;
        }
#pragma unroll
        for (int i = 0; i < HG / 2; ++i) {
          float a[2], nr[2] = {nref[i].x, nref[i].y};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float r = maximum(red_s + 2 * i + e);
            if (was_set) r = fmaxf(r, -nr[e]);
            if (!(r > -INFINITY)) r = 0.f;             // nothing visible yet (or only NaN)
            a[e] = -nr[e] - r;
            nr[e] = -r;
          }
          nref[i] = make_float2(nr[0], nr[1]);
          x[i] = add2(x[i], make_float2(a[0], a[1]));
          if (was_set) {                               // (else there is nothing to rescale)
            const float2 alpha = make_float2(exp2_fast(a[0]), exp2_fast(a[1]));
            l_run[i] = mul2(l_run[i], make_float2(exp2_fast(a[0] + (vsum - was)), exp2_fast(a[1] + (vsum - was))));
            o0[i] = mul2(o0[i], alpha);
            o1[i] = mul2(o1[i], alpha);
          }
        }
        named_barrier_sync(2, SOFT);                   // red_s may be written again
      }
      float per_v = vsum - lvs;
      if (per_v > 0.f && seen) {                       // the v_scale is 2^-V_DROP of the largest: p by itself
#pragma unroll
        for (int i = 0; i < HG / 2; ++i)
          l_run[i] = add2(l_run[i], make_float2(exp2_fast(x[i].x + per_v), exp2_fast(x[i].y + per_v)));
        per_v = -INFINITY;
      }
      per_v = exp2_fast(per_v);                        // (a number for unseen entries too)
      if constexpr (!C::RING) scales();                // of tile k + 1
      // ---- P times v_scale as four E4M3 terms
      uint32_t w4[PN / 4];
#pragma unroll
      for (int i = 0; i < PN / 4; ++i) w4[i] = 0;
#pragma unroll
      for (int c = 0; c < HG / 4; ++c) {
        float2 y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          y[e] = make_float2(exp2_fast(x[2 * c + e].x), exp2_fast(x[2 * c + e].y));
          l_run[2 * c + e] = fma2(y[e], both(per_v), l_run[2 * c + e]);
        }
#pragma unroll
        for (int q = 0; q < PT; ++q) {
          const uint32_t c0 = e4m3x2(y[0].x, y[0].y), c1 = e4m3x2(y[1].x, y[1].y);
          w4[q * (HG / 4) + c] = c0 | (c1 << 16);
          if (q + 1 < PT) {
            y[0] = fma2(e4m3x2_value(c0), both(-16.f), mul2(y[0], both(16.f)));
            y[1] = fma2(e4m3x2_value(c1), both(-16.f), mul2(y[1], both(16.f)));
          }
        }
      }
      if (k > 0) output_done(k - 1);
#pragma unroll
      for (int i = 0; i < PN / 16; ++i)
        *reinterpret_cast<uint4*>(p_s + (i * TILE + tid) * 16) =
            make_uint4(w4[4 * i], w4[4 * i + 1], w4[4 * i + 2], w4[4 * i + 3]);
      if (tid == 0) *add_s = add ? 1 : 0;
      add = true;
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(p_full);

      fresh = ++tile == p.tiles;
      if (fresh || k + 1 == n) {
        // ---- end of the pair or of the run: output, or the piece for the merge
        const bool whole = fresh && k + 1 >= p.tiles;
        const int at = lane & 15;
        float mine = 0.f, ref = 0.f;                   // of head `at`
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          float l = h & 1 ? l_run[h / 2].y : l_run[h / 2].x;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          if (at == h) {
            mine = l;
            ref = h & 1 ? -nref[h / 2].y : -nref[h / 2].x;
          }
        }
        if (lane < 16) red_s[warp * 17 + lane] = mine;
        named_barrier_sync(2, SOFT);
        float l = red_s[at] + red_s[17 + at] + red_s[34 + at] + red_s[51 + at];
        // The sum as a number in [1, 2) and its reference score, so that pieces with other references compare; the
        // outputs are 2^more times what they are relative to that.
        const float e = l > 0.f && l < INFINITY ? (float)((int)(__float_as_uint(l) >> 23) - 127) : 0.f;
        const float mref = ref - vsum + e, more = e - vsum;
        l *= power_of_two(-e);
        named_barrier_sync(2, SOFT);
        const int64_t t = pair / p.Hkv;
        const int g = pair - (int)t * p.Hkv;
        output_done(k);                                // (the product ran under the sums above)
        take_output();
        if (whole) {
          float mul = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays NaN
          const int64_t hq = t * p.Hq + (int64_t)g * p.group;
          if (p.gate && at < p.group) mul *= 1.f / (1.f + expf(-p.gate[hq + at]));
          const float half = floorf(more * 0.5f);      // 2^-more in two factors: it may lie outside fp32's range
          const float unit = power_of_two(-half);
          mul *= power_of_two(half - more);
          uint16_t* out = p.out + t * p.out_st + (int64_t)g * p.group * D + tid;
#pragma unroll
          for (int h = 0; h < HG; ++h) {
            const float m = __shfl_sync(0xffffffffu, mul, h), u = __shfl_sync(0xffffffffu, unit, h);
            if (h < p.group) {
              out[h * D] = narrow<F16>((h & 1 ? o0[h / 2].y : o0[h / 2].x) * u * m);
              out[h * D + 128] = narrow<F16>((h & 1 ? o1[h / 2].y : o1[h / 2].x) * u * m);
            }
          }
          if (warp == 0 && lane < p.group) {
            const float l2 = l == 0.f ? -INFINITY : mref + log2f(l);
            if (p.lse) p.lse[hq + lane] = l2 * 0.69314718055994531f;
            if (p.lse2) p.lse2[hq + lane] = l2;
          }
        } else {
          // slot 2 i: the pair that run i begins with; 2 i + 1: the one it ends with
          const int64_t slot = 2 * (int64_t)blockIdx.x + (pair == pair0 ? 0 : 1);
          float* po = p.part_o + slot * p.group * D + tid;
#pragma unroll
          for (int h = 0; h < HG; ++h)
            if (h < p.group) {
              po[h * D] = h & 1 ? o0[h / 2].y : o0[h / 2].x;
              po[h * D + 128] = h & 1 ? o1[h / 2].y : o1[h / 2].x;
            }
          if (warp == 0 && lane < p.group) {
            p.part_ml[(slot * p.group + lane) * 2] = l == 0.f ? -INFINITY : mref;
            p.part_ml[(slot * p.group + lane) * 2 + 1] = l;
            p.part_d[slot * p.group + lane] = more;
          }
        }
      }
      if (fresh) {
        tile = 0;
        ++pair;
        ++nth;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, C::TMEM);
}

// What follows the attention, in one launch that waits for it.  Its first CTAs add
// the probabilities up over the query heads, 256 entries of a row each; the
// others merge the pieces of pairs cut by the end of a run, two features a thread
// and 2 heads a CTA.  The first work a cut pair's sums out of its pieces again,
// instead of waiting for the merge in a launch of their own.
constexpr int MERGE_HEADS = 2, MERGE_THREADS = MERGE_HEADS * D / 2;

// weights[t, e] = sum over query heads of 2^(s - lse2): one thread per entry, heads in order.
template <int BATCH>
__device__ __forceinline__ void add_probabilities(const Params& p, int block) {
  const int per_row = (p.width + MERGE_THREADS - 1) / MERGE_THREADS;
  const int t = block / per_row, e = (block - t * per_row) * MERGE_THREADS + (int)threadIdx.x, lane = threadIdx.x & 31;
  const bool in = e < p.width;
  float w = 0.f;
  for (int g = 0; g < p.Hkv; ++g) {
    const int pair = t * p.Hkv + g, begin = pair * p.tiles, end = begin + p.tiles;
    const float* s = p.part_s + (int64_t)pair * p.group * p.width + e;
    float x[MAX_GROUP];                                // on their way while the sums are worked out
#pragma unroll
    for (int h = 0; h < MAX_GROUP; ++h) x[h] = in && h < p.group ? s[(int64_t)h * p.width] : -INFINITY;
    const int first = run_of(p, begin);
    float l2 = 0.f;                                    // of head `lane`
    if (lane < p.group) {
      if (run_begin(p, first + 1) >= end) {
        l2 = p.lse2[(int64_t)pair * p.group + lane];
      } else {
        float M = -INFINITY, sum = 0.f;
        for (int i0 = first; i0 < p.ctas && run_begin(p, i0) < end; i0 += BATCH) {
          float2 ml[BATCH];
          float m = M;
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int run = i0 + i;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (run < p.ctas && run_begin(p, run) < end) {
              const int64_t slot = 2 * (int64_t)run + (run == first && run_begin(p, run) < begin ? 1 : 0);
              ml[i] = reinterpret_cast<const float2*>(p.part_ml)[slot * p.group + lane];
            }
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) m = fmaxf(m, ml[i].x);
          const float mr = m == -INFINITY ? 0.f : m;
          sum *= exp2f(M - mr);
          M = m;
#pragma unroll
          for (int i = 0; i < BATCH; ++i) sum = fmaf(exp2f(ml[i].x - mr), ml[i].y, sum);
        }
        l2 = sum == 0.f ? -INFINITY : M + log2f(sum);
      }
    }
#pragma unroll
    for (int h = 0; h < MAX_GROUP; ++h) {
      const float l = __shfl_sync(0xffffffffu, l2, h);
      w += x[h] == -INFINITY ? 0.f : exp2f(x[h] - l);
    }
  }
  if (in) p.weights[t * p.w_stride + e] = w;
}

template <bool F16, int BATCH>   // pieces loaded in one round trip
__global__ void __launch_bounds__(MERGE_THREADS) finish_fp8_kernel(const Params p) {
  const int block = (int)blockIdx.x - p.sums;
  if (block < 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    add_probabilities<BATCH>(p, (int)blockIdx.x);
    return;
  }
  const int heads = block / p.places, place = block - heads * p.places;
  const int hh = heads * MERGE_HEADS + threadIdx.x / (D / 2), f2 = threadIdx.x % (D / 2);
  int pair, begin, first;
  bool mine;
  if (p.places < p.ctas - 1) {                         // fewer pairs than cuts: a CTA per pair
    pair = place;
    begin = pair * p.tiles;
    first = run_of(p, begin);
    mine = run_begin(p, first + 1) < begin + p.tiles;
  } else {                                             // a CTA per cut, between runs `place` and place + 1
    first = place;
    const int at = run_begin(p, first + 1);
    pair = at / p.tiles;
    begin = pair * p.tiles;
    mine = at > begin && (first == 0 || run_begin(p, first) <= begin);   // inside a pair, and its first cut
  }
  int pieces = 2;
  while (first + pieces < p.ctas && run_begin(p, first + pieces) < begin + p.tiles) ++pieces;
  // the first piece ends run `first` (its second slot unless the run begins with this pair); the others begin theirs
  const int slot0 = 2 * first + (run_begin(p, first) >= begin ? 0 : 1);
  auto slot = [&](int i) { return (int64_t)(i == 0 ? slot0 : 2 * (first + i)) * p.group + hh; };
  asm volatile("griddepcontrol.wait;" ::: "memory");   // every CTA: the grid must not end before the attention does
  if (!mine || hh >= p.group) return;
  // (plain loads: the pieces are written while this grid is already launched)
  // Sums relative to the largest reference score M so far, outputs 2^P times those: P as large as every piece allows.
  float M = -INFINITY, P = 0.f, sum = 0.f;
  float2 acc = make_float2(0.f, 0.f);
  for (int i0 = 0; i0 < pieces; i0 += BATCH) {
    float2 ml[BATCH], o[BATCH];
    float pd[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      o[i] = make_float2(0.f, 0.f);
      pd[i] = 0.f;
      if (i0 + i < pieces) {
        ml[i] = *reinterpret_cast<const float2*>(p.part_ml + slot(i0 + i) * 2);
        pd[i] = p.part_d[slot(i0 + i)];
        o[i] = reinterpret_cast<const float2*>(p.part_o + slot(i0 + i) * D)[f2];
      }
    }
    float m = M;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) m = fmaxf(m, ml[i].x);
    if (m == -INFINITY) continue;                      // nothing visible so far
    const float a = M - m;                             // -infinity until something is
    float d = P - a;                                   // (infinity for pieces without anything visible)
#pragma unroll
    for (int i = 0; i < BATCH; ++i) d = fminf(d, pd[i] + (m - ml[i].x));
    const float e = exp2_fast(a + (d - P));            // at most 1, 0 in the first round
    sum *= exp2_fast(a);
    acc = make_float2(acc.x * e, acc.y * e);
    M = m;
    P = d;
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const float b = ml[i].x - m, w = exp2_fast(b + (d - pd[i]));
      sum = fmaf(exp2_fast(b), ml[i].y, sum);
      acc.x = fmaf(w, o[i].x, acc.x);
      acc.y = fmaf(w, o[i].y, acc.y);
    }
  }
  const int64_t t = pair / p.Hkv;
  const int h = (pair - (int)t * p.Hkv) * p.group + hh;
  float mul = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // a NaN sum stays NaN
  if (p.gate) mul *= 1.f / (1.f + expf(-p.gate[t * p.Hq + h]));
  const float half = floorf(0.5f * P);                 // 2^-P in two factors, as above
  const float unit = power_of_two(-half);
  mul *= power_of_two(half - P);
  reinterpret_cast<uint32_t*>(p.out + t * p.out_st + (int64_t)h * D)[f2] =
      (uint32_t)narrow<F16>(acc.x * unit * mul) | ((uint32_t)narrow<F16>(acc.y * unit * mul) << 16);
  if (f2 == 0) {
    const float l2 = sum == 0.f ? -INFINITY : M + log2f(sum);
    if (p.lse) p.lse[t * p.Hq + h] = l2 * 0.69314718055994531f;
  }
}

}  // namespace attn8
}  // namespace qsa

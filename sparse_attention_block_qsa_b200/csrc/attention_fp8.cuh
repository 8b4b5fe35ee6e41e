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
//    halves), P as an N-major one, so thread e writes its 16 heads of a term
//    as one 16-byte store.  P (times v_scale_j over the tile's largest
//    v_scale, so at most 1) is split into three terms the same way: 2^-12
//    relative, 2^-26 of the tile's largest, well below the 16-bit output's
//    rounding.
//  * Running maximum, sum and output are fp32 in registers (thread = feature
//    for the output); each tile's O^T is read back from TMEM and added.
//
// Work is the list of (row, KV head, 128-entry tile) triples in order; every CTA
// takes an equal contiguous run of it (two CTAs per SM), so any batch fills the
// GPU to one tile.  A run may begin and end inside a row's list: such pieces go
// to the workspace and combine_fp8_kernel merges them.  Inside a CTA
//  * warps 4-7 gather K and V rows with 16-byte cp.async through the page table
//    into three 32 KB buffers (K and V tiles in turn), two tiles ahead of the
//    look-ups' consumers, and split each new row's queries;
//  * warp 8 issues the MMAs, whichever product has its operands: S of tile u + 1
//    usually runs under the softmax of tile u;
//  * warps 0-3 run the softmax (thread = entry) and add up the output (thread =
//    feature); the output product of a tile is read one tile later.
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
constexpr int THREADS = SOFT + PROD + 128;   // the last warpgroup: one warp that issues MMAs
// Registers a thread: 384 threads twice on an SM leave 80 each at launch; the
// warpgroups then share them out as 136 + 56 + 48 (the same sum of 240).
constexpr int REGS_LAUNCH = 80, REGS_SOFT = 136, REGS_PROD = 56, REGS_MMA = 48;
static_assert(REGS_SOFT + REGS_PROD + REGS_MMA <= 3 * REGS_LAUNCH, "setmaxnreg would wait for ever");
constexpr int MAX_GROUP = 16;          // query heads per KV head
constexpr int PT = 3;                  // E4M3 terms of a probability
constexpr int BUFS = 3;
constexpr int HALF_BYTES = TILE * 128;       // 128 features of every entry
constexpr int BUF_BYTES = 2 * HALF_BYTES;
constexpr int QC_SLOTS = 4;            // rows whose head factors are held

// Sizes of one instance: 16-bit type and query heads held per KV head.
template <bool F16, int HG>
struct Cfg {
  static constexpr int QT = F16 ? 3 : 2;                          // E4M3 terms of a query element
  static constexpr int QCOLS = QT * HG, QN = (QCOLS + 15) / 16 * 16, QROWS = (QCOLS + 7) / 8 * 8;
  static constexpr int PCOLS = PT * HG, PN = (PCOLS + 15) / 16 * 16;
  static constexpr uint32_t TMEM = 2 * QN + 2 * PN <= 128 ? 128 : 256;
  static constexpr int Q_BYTES = QROWS * D;
  static constexpr int P_BYTES = PN * TILE;
  static constexpr size_t SMEM =
      BUFS * BUF_BYTES + Q_BYTES + P_BYTES + 15 * 8 + 2 * 4 * 17 * 4 + QC_SLOTS * MAX_GROUP * 4 + 16;
  static constexpr int RESIDENT = 2 * (SMEM + 1024) <= 233472 ? 2 : 1;   // CTAs per SM
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
  int64_t kv_page_stride, kv_row_stride, kv_head_stride;  // bytes
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
  int64_t total;              // tiles of all pairs
  int32_t ctas;               // runs
  float scale_log2;
  float* part_o;              // [2 ctas, group, 256] unnormalised outputs of pairs cut by a run's ends
  float* part_ml;             // [2 ctas, group, 2] maximum (log2 units), sum
  float* part_s;              // [T, Hkv, width, group] scores (log2 units), or null
  float* lse2;                // [T, Hq] log2 of the sum of 2^s, or null
  const float* gate;
  uint16_t* out;
  int64_t out_st;
  float* lse;
  float* weights;             // [T, width], or null
  int64_t w_stride;
};

// First tile of run i: the runs differ by at most one tile.
__device__ __forceinline__ int64_t run_begin(const Params& p, int64_t i) {
  const int64_t per = p.total / p.ctas, more = p.total % p.ctas;
  return i * per + (i < more ? i : more);
}
// The run that holds tile u.
__device__ __forceinline__ int64_t run_of(const Params& p, int64_t u) {
  const int64_t per = p.total / p.ctas, more = p.total % p.ctas;
  return u < more * (per + 1) ? u / (per + 1) : more + (u - more * (per + 1)) / per;
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

__device__ __forceinline__ float exp2_fast(float x) {   // 2 ulp; 2^-inf = 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Arrives on bar once this thread's cp.async copies so far have landed; the
// barrier counts this arrival like any other.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

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

// attn::row_request, with position -1 (nothing visible) for the rows behind
// the last request's: a batch may be padded.
__device__ __forceinline__ void row_position(const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                                             int R, int64_t t, int lane, int& r, int& pos, int& L) {
  attn::row_request(cu, seq_lens, R, t, lane, r, pos, L);
  if (t >= (int64_t)__ldg(cu + r + 1)) pos = -1;
}

// The entries of consecutive tiles, looked up in stages so that no load is
// waited for: a tile's list entry two tiles and its page one tile before use.
// Every lane follows entry `lane_entry` of the tile.
struct Feed {
  int64_t t;                  // row, KV head and tile of the stage that loads list entries
  int g, tile;
  int64_t left;               // tiles of the run it has not loaded yet
  const int32_t* pt;          // the row's page table; last token it sees
  int last;
  int jA, lastA, gA;          // list entry loaded
  const int32_t* ptA;
  int jB, pageB, gB;          // page loaded

  __device__ __forceinline__ void row(const Params& p, int lane) {
    int r, pos, L;
    row_position(p.cu, p.seq_lens, p.R, t, lane, r, pos, L);
    pt = p.page_table + (int64_t)r * p.pt_stride;
    last = min(pos, L - 1);
  }
  __device__ __forceinline__ void load_entry(const Params& p, int lane_entry, int lane) {
    jA = -1;
    lastA = last;
    gA = g;
    ptA = pt;
    if (left <= 0) return;
    --left;
    const int e = tile * TILE + lane_entry;
    if (e < p.width) jA = __ldg(p.tok + t * p.tok_stride + e);
    if (++tile == p.tiles) {
      tile = 0;
      if (++g == p.Hkv) {
        g = 0;
        ++t;
        if (left > 0) row(p, lane);
      }
    }
  }
  __device__ __forceinline__ void load_page(const Params& p) {
    jB = jA >= 0 && jA <= lastA ? jA : -1;
    gB = gA;
    pageB = -1;
    if (jB >= 0) {
      const int lp = divide(jB, p.by_page);
      if (lp < p.max_pages) pageB = __ldg(ptA + lp);
    }
  }
  __device__ __forceinline__ void start(const Params& p, int64_t u0, int64_t n, int lane_entry, int lane) {
    const int64_t pair = u0 / p.tiles;
    tile = (int)(u0 - pair * p.tiles);
    t = pair / p.Hkv;
    g = (int)(pair - t * p.Hkv);
    left = n;
    row(p, lane);
    load_entry(p, lane_entry, lane);
    load_page(p);
    load_entry(p, lane_entry, lane);
  }
  // the next tile's entry: its page and token (page < 0: not visible)
  __device__ __forceinline__ void next(const Params& p, int lane_entry, int lane, int& page, int& j, int& kv_head) {
    j = jB;
    kv_head = gB;
    page = jB >= 0 && (int64_t)pageB < p.num_pages ? pageB : -1;
    load_page(p);
    load_entry(p, lane_entry, lane);
  }
};

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
  constexpr int QT = C::QT, QN = C::QN, PN = C::PN;
  constexpr uint32_t Q_HALF = C::QROWS * 128;
  constexpr uint32_t IDESC_S = idesc_e4m3(TILE, QN, false, false);
  constexpr uint32_t IDESC_O = idesc_e4m3(128, PN, true, true);
  extern __shared__ __align__(1024) uint8_t smem8[];   // the swizzle repeats every 1024 bytes
  uint8_t* buf_s = smem8;
  uint8_t* q_s = buf_s + BUFS * BUF_BYTES;             // [half][QROWS][128 bytes], swizzled; row = term * HG + head
  uint8_t* p_s = q_s + C::Q_BYTES;                     // [16 columns][entry][16 bytes]; column = term * HG + head
  uint64_t* bars = reinterpret_cast<uint64_t*>(p_s + C::P_BYTES);
  uint64_t *kv_full = bars, *kv_empty = bars + 3, *s_full = bars + 6, *s_empty = bars + 8, *p_full = bars + 10,
           *o_full = bars + 11, *q_full = bars + 12, *q_empty = bars + 13, *drained = bars + 14;
  float* red_s = reinterpret_cast<float*>(bars + 15);  // [2][4 warps][17]: tile maxima by head, v_scale
  float* qc_s = red_s + 2 * 4 * 17;                    // [QC_SLOTS][16]: a head's power of two times scale * log2(e)
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(qc_s + QC_SLOTS * MAX_GROUP);
  int* abort_s = reinterpret_cast<int*>(tmem_s + 1);
  volatile int* abort = abort_s;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t u0 = run_begin(p, blockIdx.x), n = run_begin(p, (int64_t)blockIdx.x + 1) - u0;
  const int64_t pair0 = u0 / p.tiles;
  const int tile0 = (int)(u0 - pair0 * p.tiles);

  if (warp == 8) tmem_alloc(tmem_s, C::TMEM);
  if (tid == 0) {
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(&kv_full[i], PROD);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 2);
      mbar_init(&s_empty[i], SOFT);
    }
    mbar_init(p_full, SOFT);
    mbar_init(o_full, 1);
    mbar_init(q_full, PROD);
    mbar_init(q_empty, 1);
    mbar_init(drained, 1);
    fence_mbar_init();
    *abort_s = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  const uint32_t tm_o = tmem + 2 * QN;                 // two halves of PN columns
  // A wait that runs out sets *abort.  Gathering and issuing warps then leave; the softmax warps go on through
  // their tiles without waiting, so that their barrier is always met.
  auto gone = [&]() {
    record_device_error(QSA_DEVERR_WAIT_TIMEOUT);
    *abort = 1;
  };

  if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- gather
    if constexpr (C::RESIDENT > 1) regs_shrink<REGS_PROD>();
    const int w = warp - 4, entry = 32 * w + lane;
    const int u = lane & 15, row2 = lane >> 4;         // 16 lanes a row, two rows per instruction
    Feed f;
    f.start(p, u0, n, entry, lane);
    int64_t pair = pair0;
    int tile = tile0;
    bool ok = true;
    // rows of the warp's 32 entries into buffer item % BUFS
    auto gather = [&](const uint8_t* base, int64_t off, int64_t item) {
      const int b = (int)(item % BUFS);
      ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[b], (uint32_t)((item / BUFS) & 1) ^ 1, abort));
      if (!ok) return;
      const uint32_t dst = smem_addr(buf_s + b * BUF_BYTES) + (u >> 3) * HALF_BYTES + 32 * w * 128;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int nrow = 2 * i + row2;
        const int64_t o = __shfl_sync(0xffffffffu, off, nrow);
        attn::cp_async16(dst + nrow * 128 + (((u & 7) ^ (nrow & 7)) << 4), o >= 0 ? base + o + u * 16 : base, o >= 0);
      }
      cp_async_arrive(&kv_full[b]);
    };
    // queries of a pair: E4M3 terms; heads at or above the group are zero
    auto queries = [&](int64_t pr, int nth) {
      const int64_t t = pr / p.Hkv;
      const int g = (int)(pr - t * p.Hkv);
      uint4 x4[HG / 4];
#pragma unroll
      for (int i = 0; i < HG / 4; ++i) {
        const int h = w + 4 * i;
        x4[i] = make_uint4(0, 0, 0, 0);
        if (h < p.group)
          x4[i] = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_st + ((int64_t)g * p.group + h) * p.q_sh + lane * 8));
      }
      ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (uint32_t)(nth & 1) ^ 1, abort));
      if (!ok) return;
#pragma unroll
      for (int i = 0; i < HG / 4; ++i) {
        const int h = w + 4 * i;
        const uint32_t w4[4] = {x4[i].x, x4[i].y, x4[i].z, x4[i].w};
        float x[8];
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = widen2<F16>(w4[k]);
          x[2 * k] = v.x;
          x[2 * k + 1] = v.y;
          top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          bad = bad || !(fabsf(v.x) <= 3.4e38f) || !(fabsf(v.y) <= 3.4e38f);
        }
        top = warp_max(top);
        bad = __any_sync(0xffffffffu, bad);
        // the power of two that brings the largest element into [224, 448]: 448 = 1.75 * 2^8
        const uint32_t tb = __float_as_uint(top);
        int e = (int)(tb >> 23) - 127 - 8 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(e, -126);
        const float inv1 = __uint_as_float((uint32_t)(127 + (-e) / 2) << 23);       // 2^(-e) in two factors:
        const float inv2 = __uint_as_float((uint32_t)(127 + (-e) - (-e) / 2) << 23);  // one may leave fp32's range
        uint32_t term[QT][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) y[m] = bad ? __uint_as_float(0x7fc00000u) : x[4 * k + m] * inv1 * inv2;
#pragma unroll
          for (int q = 0; q < QT; ++q) {
            const uint32_t c0 = e4m3x2(y[0], y[1]), c1 = e4m3x2(y[2], y[3]);
            term[q][k] = c0 | (c1 << 16);
            const float2 f0 = e4m3x2_value(c0), f1 = e4m3x2_value(c1);
            y[0] = (y[0] - f0.x) * 16.f;
            y[1] = (y[1] - f0.y) * 16.f;
            y[2] = (y[2] - f1.x) * 16.f;
            y[3] = (y[3] - f1.y) * 16.f;
          }
        }
        const int un = lane >> 1;                      // 16-byte unit of the row
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          const int nr = q * HG + h;
          uint8_t* dst = q_s + (un >> 3) * Q_HALF + nr * 128 + (((un & 7) ^ (nr & 7)) << 4) + (lane & 1) * 8;
          *reinterpret_cast<uint2*>(dst) = make_uint2(term[q][0], term[q][1]);
        }
        if (lane == 0) qc_s[(nth % QC_SLOTS) * MAX_GROUP + h] = h < p.group ? ldexpf(p.scale_log2, e) : 0.f;
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    };
    int nth = 0;                                       // pairs begun
    for (int64_t k = 0; k < n && ok; ++k) {
      int page, j, g;
      f.next(p, entry, lane, page, j, g);
      const int64_t off = page < 0 ? -1
                                   : (int64_t)page * p.kv_page_stride +
                                         (int64_t)(j - divide(j, p.by_page) * p.page_size) * p.kv_row_stride +
                                         (int64_t)g * p.kv_head_stride;
      gather(p.k, off, 2 * k);
      if (ok && (k == 0 || tile == 0)) queries(pair, nth++);
      if (ok) gather(p.v, off, 2 * k + 1);
      if (++tile == p.tiles) {
        tile = 0;
        ++pair;
      }
    }
    if (!ok) gone();
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- MMA issue
    if constexpr (C::RESIDENT > 1) regs_shrink<REGS_MMA>();
    if (warp == 8 && lane == 0) {
      const uint64_t q_desc = umma_desc_sw128(smem_addr(q_s));
      const uint64_t p_desc = desc_plain_mn(smem_addr(p_s), 128, TILE * 16);
      int64_t ks = 0, ko = 0;                          // next tile of either product
      int tile = tile0, nth = 0;                       // of S: tile in its pair, pairs begun
      bool fresh = true;
      uint64_t since = global_timer_ns();
      uint32_t idle = 0;
      while (ko < n) {
        bool did = false;
        if (ks < n && ks <= ko + 1 && mbar_test(&kv_full[(2 * ks) % BUFS], (uint32_t)((2 * ks) / BUFS) & 1) &&
            mbar_test(&s_empty[ks & 1], (uint32_t)((ks >> 1) & 1) ^ 1) &&
            (!fresh || mbar_test(q_full, (uint32_t)nth & 1))) {
          fence_proxy_async_smem();                    // the cp.async writes, before the tensor core reads them
          tc_fence_after();
          const int b = (int)((2 * ks) % BUFS);
          const uint64_t kd = umma_desc_sw128(smem_addr(buf_s + b * BUF_BYTES));
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_e4m3(tmem + (uint32_t)(ks & 1) * QN, kd + (s >> 2) * (HALF_BYTES >> 4) + (s & 3) * 2,
                     q_desc + (s >> 2) * (Q_HALF >> 4) + (s & 3) * 2, IDESC_S, s > 0);
          umma_commit(&kv_empty[b]);
          mbar_arrive(&s_full[ks & 1]);                // hands on what q_full published (the head factors)
          umma_commit(&s_full[ks & 1]);
          fresh = ++tile == p.tiles;
          if (fresh) {
            umma_commit(q_empty);
            tile = 0;
            ++nth;
          }
          ++ks;
          did = true;
        }
        if (ko < ks && mbar_test(p_full, (uint32_t)ko & 1) &&
            mbar_test(&kv_full[(2 * ko + 1) % BUFS], (uint32_t)((2 * ko + 1) / BUFS) & 1)) {
          fence_proxy_async_smem();
          tc_fence_after();
          const int b = (int)((2 * ko + 1) % BUFS);
          const uint64_t vd = umma_desc_sw128(smem_addr(buf_s + b * BUF_BYTES));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_e4m3(tm_o + hf * PN, vd + hf * (HALF_BYTES >> 4) + s * (32 * 128 >> 4), p_desc + s * (32 * 16 >> 4),
                       IDESC_O, s > 0);
          umma_commit(&kv_empty[b]);
          umma_commit(o_full);
          ++ko;
          did = true;
        }
        if (did) {
          idle = 0;
        } else if ((++idle & 63u) == 0) {
          if (idle == 64) since = global_timer_ns();
          if (*abort || global_timer_ns() - since > QSA_WAIT_TIMEOUT_NS) {
            gone();
            umma_commit(drained);                      // what it issued still ends before TMEM is freed
            mbar_wait(drained, 0, nullptr);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    if constexpr (C::RESIDENT > 1) regs_grow<REGS_SOFT>();
    const uint32_t tm_lane = (uint32_t)(warp * 32) << 16;
    Feed f;
    f.start(p, u0, n, tid, lane);
    float l_run[HG], o0[HG], o1[HG];                   // l_run: this thread's entries; o: features tid, 128 + tid
    float m_lane = -INFINITY, a_prev = 0.f, ov_prev = 0.f, qc = 0.f;   // lane h: head h's maximum, last factor
    int64_t pair = pair0;
    int tile = tile0, nth = 0;
    bool fresh = true;
    // scales of the next tile's entry: loaded one tile ahead
    float ks_nx = 0.f, vs_nx = 0.f;
    bool seen_nx = false;
    auto scales = [&]() {
      int page, j, g;
      f.next(p, tid, lane, page, j, g);
      seen_nx = page >= 0;
      ks_nx = vs_nx = 0.f;
      if (seen_nx) {
        const int in_page = j - divide(j, p.by_page) * p.page_size;
        const int64_t at = (int64_t)page * p.sc_page_stride + (int64_t)divide(in_page, p.by_block) * p.sc_block_stride + g;
        ks_nx = __ldg(p.k_scale + at);
        vs_nx = __ldg(p.v_scale + at);
      }
    };
    scales();
    // o = o * a_prev + O^T of tile k
    auto add_output = [&](int64_t k) {
      if (!mbar_wait(o_full, (uint32_t)k & 1, abort)) gone();
      tc_fence_after();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float d[(C::PCOLS + 7) / 8 * 8];
        tmem_ld(tm_o + tm_lane + hf * PN, d);
        tmem_wait_ld();
        float* o = hf == 0 ? o0 : o1;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float x = fmaf(d[2 * HG + h], 1.f / 256.f, fmaf(d[HG + h], 1.f / 16.f, d[h]));
          o[h] = fmaf(o[h], __shfl_sync(0xffffffffu, a_prev, h), ov_prev * x);
        }
      }
    };
    for (int64_t k = 0; k < n; ++k) {
      const float ks = ks_nx, vs = vs_nx;
      const bool seen = seen_nx;
      if (fresh) {
        m_lane = -INFINITY;
#pragma unroll
        for (int h = 0; h < HG; ++h) l_run[h] = o0[h] = o1[h] = 0.f;
      }
      float x[HG];
      {
        if (!mbar_wait(&s_full[k & 1], (uint32_t)(k >> 1) & 1, abort)) gone();
        tc_fence_after();
        if (fresh) qc = (lane & 15) < HG ? qc_s[(nth % QC_SLOTS) * MAX_GROUP + (lane & 15)] : 0.f;
        float d[(C::QCOLS + 7) / 8 * 8];
        tmem_ld(tmem + tm_lane + (uint32_t)(k & 1) * QN, d);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&s_empty[k & 1]);
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          x[h] = fmaf(d[HG + h], 1.f / 16.f, d[h]);
          if (QT > 2) x[h] = fmaf(d[(QT - 1) * HG + h], 1.f / 256.f, x[h]);
          const float c = __shfl_sync(0xffffffffu, qc, h) * ks;
          x[h] = seen ? x[h] * c : -INFINITY;
        }
      }
      if (p.part_s) {
        const int e = tile * TILE + tid;
        if (e < p.width) {
          float* dst = p.part_s + (pair * p.width + e) * p.group;
#pragma unroll
          for (int h = 0; h < HG; ++h)
            if (h < p.group) dst[h] = x[h];
        }
      }
      scales();                                        // of tile k + 1
      // ---- maxima over the tile
      float* red = red_s + (k & 1) * 4 * 17;
      {
        float mine = -INFINITY;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float wm = warp_max(x[h]);
          if (lane == h) mine = wm;
        }
        const float vm = warp_max(vs);
        if (lane == 16) mine = vm;
        if (lane <= 16) red[warp * 17 + lane] = mine;
      }
      named_barrier_sync(1, SOFT);
      float a_lane, vref;
      {
        const int at = lane & 15;
        const float m = fmaxf(fmaxf(fmaxf(red[at], red[17 + at]), fmaxf(red[34 + at], red[51 + at])), m_lane);
        vref = fmaxf(fmaxf(red[16], red[33]), fmaxf(red[50], red[67]));
        a_lane = m == -INFINITY ? 0.f : exp2_fast(m_lane - m);
        m_lane = m;
      }
      const float mr = m_lane == -INFINITY ? 0.f : m_lane;   // nothing visible yet: every probability is 0
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        x[h] = exp2_fast(x[h] - __shfl_sync(0xffffffffu, mr, h));
        l_run[h] = fmaf(l_run[h], __shfl_sync(0xffffffffu, a_lane, h), x[h]);
      }
      // ---- the last tile's output, whose product also frees P
      if (!fresh) add_output(k - 1);
      a_prev = a_lane;
      ov_prev = vref * (1.f / 256.f);
      // ---- P times v_scale / vref, at most 256, as three E4M3 terms
      const float vn = vref > 0.f ? __fdividef(vs, vref) * 256.f : 0.f;
      uint32_t w4[PN / 4];
#pragma unroll
      for (int i = 0; i < PN / 4; ++i) w4[i] = 0;
#pragma unroll
      for (int c = 0; c < HG / 4; ++c) {
        float y[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) y[m] = x[4 * c + m] * vn;
#pragma unroll
        for (int q = 0; q < PT; ++q) {
          const uint32_t c0 = e4m3x2(y[0], y[1]), c1 = e4m3x2(y[2], y[3]);
          w4[q * (HG / 4) + c] = c0 | (c1 << 16);
          if (q + 1 < PT) {
            const float2 f0 = e4m3x2_value(c0), f1 = e4m3x2_value(c1);
            y[0] = (y[0] - f0.x) * 16.f;
            y[1] = (y[1] - f0.y) * 16.f;
            y[2] = (y[2] - f1.x) * 16.f;
            y[3] = (y[3] - f1.y) * 16.f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < PN / 16; ++i)
        *reinterpret_cast<uint4*>(p_s + (i * TILE + tid) * 16) =
            make_uint4(w4[4 * i], w4[4 * i + 1], w4[4 * i + 2], w4[4 * i + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(p_full);

      fresh = ++tile == p.tiles;
      if (fresh || k + 1 == n) {
        // ---- end of the pair or of the run: output, or the piece for the merge
        add_output(k);
        const bool whole = fresh && (k + 1 >= p.tiles);
        float* lsum = red_s + (k & 1) * 4 * 17;
        named_barrier_sync(1, SOFT);                   // every warp has read its maxima
        float mine = 0.f;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          float l = l_run[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          if (lane == h) mine = l;
        }
        if (lane < 16) lsum[warp * 17 + lane] = mine;
        named_barrier_sync(1, SOFT);
        const int at = lane & 15;
        const float l = lsum[at] + lsum[17 + at] + lsum[34 + at] + lsum[51 + at];
        const int64_t t = pair / p.Hkv;
        const int g = (int)(pair - t * p.Hkv);
        if (whole) {
          float mul = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN sum stays NaN
          const int64_t hq = t * p.Hq + (int64_t)g * p.group;
          if (p.gate && at < p.group) mul *= 1.f / (1.f + expf(-p.gate[hq + at]));
          uint16_t* out = p.out + t * p.out_st + (int64_t)g * p.group * D + tid;
#pragma unroll
          for (int h = 0; h < HG; ++h) {
            const float m = __shfl_sync(0xffffffffu, mul, h);
            if (h < p.group) {
              out[h * D] = narrow<F16>(o0[h] * m);
              out[h * D + 128] = narrow<F16>(o1[h] * m);
            }
          }
          if (warp == 0 && lane < p.group) {
            const float l2 = l == 0.f ? -INFINITY : m_lane + log2f(l);
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
              po[h * D] = o0[h];
              po[h * D + 128] = o1[h];
            }
          if (warp == 0 && lane < p.group) {
            p.part_ml[(slot * p.group + lane) * 2] = m_lane;
            p.part_ml[(slot * p.group + lane) * 2 + 1] = l;
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

// Merges the pieces of pairs cut by the end of a run: one warp per (cut, head).
// The warps of a pair's first cut merge all of its pieces.
template <bool F16>
__global__ void __launch_bounds__(256) combine_fp8_kernel(const Params p) {
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t cut = wid / p.group + 1;               // between runs cut - 1 and cut
  const int hh = (int)(wid % p.group);
  if (cut >= p.ctas) return;
  const int64_t at = run_begin(p, cut), pair = at / p.tiles, begin = pair * p.tiles;
  if (at == begin) return;                             // the runs part between two pairs
  const int64_t first = run_of(p, begin), last = run_of(p, begin + p.tiles - 1);
  if (cut != first + 1) return;
  float M = -INFINITY;
  for (int64_t i = first; i <= last; ++i) {
    const int64_t slot = 2 * i + (run_begin(p, i) >= begin || i > first ? 0 : 1);
    M = fmaxf(M, p.part_ml[(slot * p.group + hh) * 2]);
  }
  const float Mr = M == -INFINITY ? 0.f : M;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int64_t i = first; i <= last; ++i) {
    const int64_t slot = 2 * i + (run_begin(p, i) >= begin || i > first ? 0 : 1);
    const float w = exp2f(p.part_ml[(slot * p.group + hh) * 2] - Mr);
    sum = fmaf(w, p.part_ml[(slot * p.group + hh) * 2 + 1], sum);
    const float* po = p.part_o + (slot * p.group + hh) * D + lane * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, po[e], acc[e]);
  }
  const int64_t t = pair / p.Hkv;
  const int h = (int)(pair - t * p.Hkv) * p.group + hh;
  float mul = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // a NaN sum stays NaN
  if (p.gate) mul *= 1.f / (1.f + expf(-p.gate[t * p.Hq + h]));
  uint32_t w4[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w4[e] = (uint32_t)narrow<F16>(acc[2 * e] * mul) | ((uint32_t)narrow<F16>(acc[2 * e + 1] * mul) << 16);
  *reinterpret_cast<uint4*>(p.out + t * p.out_st + (int64_t)h * D + lane * 8) =
      make_uint4(w4[0], w4[1], w4[2], w4[3]);
  if (lane == 0) {
    const float l2 = sum == 0.f ? -INFINITY : M + log2f(sum);
    if (p.lse) p.lse[t * p.Hq + h] = l2 * 0.69314718055994531f;
    if (p.lse2) p.lse2[t * p.Hq + h] = l2;
  }
}

// weights[t, e] = sum over query heads of 2^(s - lse2): one thread per entry,
// heads in order.
__global__ void __launch_bounds__(256) weights_kernel(const Params p) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.T * p.width) return;
  const int64_t t = i / p.width;
  const int e = (int)(i % p.width);
  float w = 0.f;
  for (int g = 0; g < p.Hkv; ++g) {
    const float* s = p.part_s + ((t * p.Hkv + g) * p.width + e) * p.group;
    for (int h = 0; h < p.group; ++h) {
      const float x = s[h];
      if (x != -INFINITY) w += exp2f(x - p.lse2[t * p.Hq + g * p.group + h]);
    }
  }
  p.weights[t * p.w_stride + e] = w;
}

}  // namespace attn8
}  // namespace qsa

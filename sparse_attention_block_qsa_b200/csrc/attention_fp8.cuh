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
// One CTA per (row, KV head, split of the row's list); the rows are gathered
// with 16-byte cp.async through the page table into three 32 KB buffers that
// K and V tiles take in turn.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.cuh"
#include "sm100.cuh"

namespace qsa {
namespace attn8 {

constexpr int D = 256;
constexpr int TILE = 128;              // list entries per tile (UMMA M)
constexpr int THREADS = 128;           // thread = entry (scores), feature (output)
constexpr int NH = 16;                 // query heads per KV head, padded
constexpr int PT = 3;                  // E4M3 terms of a probability
constexpr int BUFS = 3;
constexpr int HALF_BYTES = TILE * 128;       // 128 features of every entry
constexpr int BUF_BYTES = 2 * HALF_BYTES;
constexpr int P_BYTES = PT * TILE * NH;
constexpr int RING = 2;                // tiles whose entry offsets are held

struct Params {
  const uint16_t* q;          // [T, Hq, 256] bf16 or fp16
  int64_t q_st, q_sh;
  int32_t Hq, Hkv, group;
  const uint8_t* k;           // E4M3 codes [pages, page_size, Hkv, 256]
  const uint8_t* v;
  const float* k_scale;       // [pages, page_size / block_tokens, Hkv]
  const float* v_scale;
  int64_t num_pages;
  int32_t page_size, block_tokens;
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
  int32_t splits, tiles_per_split;
  float scale_log2;
  float* part_o;              // [T, Hkv, splits, group, 256] unnormalised
  float* part_ml;             // [T, Hkv, splits, group, 2] maximum (log2 units), sum
  float* part_s;              // [T, Hkv, width, group] scores (log2 units), or null
  float* lse2;                // [T, Hq] log2 of the sum of 2^s, or null
  const float* gate;
  uint16_t* out;
  int64_t out_st;
  float* lse;
  float* weights;             // [T, width], or null
  int64_t w_stride;
};

template <int QT>
constexpr size_t smem_bytes() {
  return BUFS * BUF_BYTES + QT * NH * D + P_BYTES + RING * TILE * 8 + 4 * (NH + 4) * 4 + NH * 4 + 32;
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
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

// attn::row_request, with position -1 (nothing visible) for the rows behind
// the last request's: a batch may be padded.
__device__ __forceinline__ void row_position(const int32_t* __restrict__ cu, const int32_t* __restrict__ seq_lens,
                                             int R, int64_t t, int lane, int& r, int& pos, int& L) {
  attn::row_request(cu, seq_lens, R, t, lane, r, pos, L);
  if (t >= (int64_t)__ldg(cu + r + 1)) pos = -1;
}

template <bool F16>
__global__ void __launch_bounds__(THREADS, 2) attn_fp8_kernel(const Params p) {
  constexpr int QT = F16 ? 3 : 2;                   // E4M3 terms of a query element
  constexpr int QN = QT * NH;
  constexpr uint32_t S_COLS = QN, O_COLS = PT * NH;
  constexpr uint32_t TMEM_COLS = S_COLS + 2 * O_COLS <= 128 ? 128 : 256;
  constexpr uint32_t IDESC_S = idesc_e4m3(TILE, QN, false, false);
  constexpr uint32_t IDESC_O = idesc_e4m3(128, PT * NH, true, true);
  extern __shared__ __align__(1024) uint8_t smem8[];   // the swizzle repeats every 1024 bytes
  uint8_t* buf_s = smem8;
  uint8_t* q_s = buf_s + BUFS * BUF_BYTES;          // [half][QN][128 bytes], swizzled
  uint8_t* p_s = q_s + QN * D;                      // [term][entry][16 heads]
  int64_t* off_s = reinterpret_cast<int64_t*>(p_s + P_BYTES);          // [RING][TILE]
  float* red_s = reinterpret_cast<float*>(off_s + RING * TILE);         // [4 warps][NH + 4]
  float* qc_s = red_s + 4 * (NH + 4);               // per head: its power of two times scale * log2(e)
  uint64_t* bar = reinterpret_cast<uint64_t*>(qc_s + NH);               // S done, O done
  uint32_t* tmem_s = reinterpret_cast<uint32_t*>(bar + 2);
  int* abort_s = reinterpret_cast<int*>(tmem_s + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = (int)(blockIdx.x % p.splits);
  const int g = (int)((blockIdx.x / p.splits) % p.Hkv);
  const int64_t t = blockIdx.x / ((int64_t)p.splits * p.Hkv);

  if (warp == 0) tmem_alloc(tmem_s, TMEM_COLS);
  if (tid == 0) {
    mbar_init(&bar[0], 1);
    mbar_init(&bar[1], 1);
    fence_mbar_init();
    *abort_s = 0;
  }

  int r, pos, L;
  row_position(p.cu, p.seq_lens, p.R, t, lane, r, pos, L);

  const int e_begin = split * p.tiles_per_split * TILE;
  const int e_end = min(p.width, e_begin + p.tiles_per_split * TILE);
  const int ntiles = e_end > e_begin ? (e_end - e_begin + TILE - 1) / TILE : 0;
  const int32_t* tok_row = p.tok + t * p.tok_stride;
  const int32_t* pt_row = p.page_table + (int64_t)r * p.pt_stride;

  // Entry tid of tile c: list entry, then page, then pool offset.  The two
  // dependent loads run one and two tiles ahead of the offset.
  auto tok_of = [&](int c) -> int {
    const int e = e_begin + c * TILE + tid;
    int j = c < ntiles && e < e_end ? __ldg(tok_row + e) : -1;
    return j > pos || j >= L ? -1 : j;
  };
  auto page_of = [&](int j) -> int {
    if (j < 0) return -1;
    const int lp = j / p.page_size;
    const int page = lp < p.max_pages ? __ldg(pt_row + lp) : -1;
    return (int64_t)page < p.num_pages ? page : -1;
  };
  auto off_of = [&](int j, int page) -> int64_t {
    return page < 0 ? -1 : (int64_t)page * p.kv_page_stride + (int64_t)(j % p.page_size) * p.kv_row_stride +
                               (int64_t)g * p.kv_head_stride;
  };
  auto scale_at = [&](int j, int page) -> int64_t {
    return page < 0 ? -1 : (int64_t)page * p.sc_page_stride +
                               (int64_t)((j % p.page_size) / p.block_tokens) * p.sc_block_stride + g;
  };
  // gather the K or V rows of tile c into buffer b: 16 threads a row
  auto load_tile = [&](const uint8_t* base, int c, int b) {
    if (c < ntiles) {
      const uint32_t dst = smem_addr(buf_s + b * BUF_BYTES);
      const int u = tid & 15, n8 = tid >> 4;
      const uint32_t in_row = (uint32_t)((u >> 3) * HALF_BYTES + (((u & 7) ^ n8) << 4));
      const int64_t* off = off_s + (c % RING) * TILE;
#pragma unroll
      for (int i = 0; i < TILE / 8; ++i) {
        const int n = i * 8 + n8;
        const int64_t o = off[n];
        attn::cp_async16(dst + in_row + n * 128, o >= 0 ? base + o + u * 16 : base, o >= 0);
      }
    }
    attn::cp_async_commit();
  };

  // offsets of the first two tiles; state of the look-ups that run ahead
  int j_nx = tok_of(0), page_nx = page_of(j_nx);
  off_s[tid] = off_of(j_nx, page_nx);
  int64_t sc0 = scale_at(j_nx, page_nx), sc1;       // scale index of tiles c, c + 1
  j_nx = tok_of(1);
  page_nx = page_of(j_nx);
  off_s[TILE + tid] = off_of(j_nx, page_nx);
  sc1 = scale_at(j_nx, page_nx);
  j_nx = tok_of(2);
  page_nx = page_of(j_nx);                          // tile c + 2
  int j_nx2 = tok_of(3);                            // tile c + 3
  __syncthreads();
  load_tile(p.k, 0, 0);
  load_tile(p.v, 0, 1);
  load_tile(p.k, 1, 2);

  // ---- queries: E4M3 terms, heads >= group zero.  Warp w takes heads w, w + 4, ...
#pragma unroll
  for (int i = 0; i < NH / 4; ++i) {
    const int h = warp + 4 * i;
    uint4 raw4 = make_uint4(0, 0, 0, 0);
    if (h < p.group)
      raw4 = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_st + ((int64_t)g * p.group + h) * p.q_sh + lane * 8));
    float x[8];
    const uint32_t w4[4] = {raw4.x, raw4.y, raw4.z, raw4.w};
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = widen2<F16>(w4[k]);
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
      top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
      bad = bad || !(fabsf(f.x) <= 3.4e38f) || !(fabsf(f.y) <= 3.4e38f);
    }
    top = warp_max(top);
    bad = __any_sync(0xffffffffu, bad);
    // the power of two that brings the largest element into [224, 448]: 448 = 1.75 * 2^8
    const uint32_t tb = __float_as_uint(top);
    int e = (int)(tb >> 23) - 127 - 8 + ((tb & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    const float inv1 = __uint_as_float((uint32_t)(127 + (-e) / 2) << 23);       // 2^(-e) in two factors: it can
    const float inv2 = __uint_as_float((uint32_t)(127 + (-e) - (-e) / 2) << 23);  // exceed the fp32 range
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
    const int u = lane >> 1;                        // 16-byte unit of the row
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      const int n = q * NH + h;
      uint8_t* dst = q_s + (u >> 3) * (QN * 128) + n * 128 + (((u & 7) ^ (n & 7)) << 4) + (lane & 1) * 8;
      *reinterpret_cast<uint2*>(dst) = make_uint2(term[q][0], term[q][1]);
    }
    if (lane == 0) qc_s[h] = h < p.group ? ldexpf(p.scale_log2, e) : 0.f;
  }

  float m_run[NH], l_run[NH], o0[NH], o1[NH];       // l_run: this thread's entries; o: features tid, 128 + tid
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    m_run[h] = -INFINITY;
    l_run[h] = o0[h] = o1[h] = 0.f;
  }
  float ks = sc0 >= 0 ? __ldg(p.k_scale + sc0) : 0.f, vs = sc0 >= 0 ? __ldg(p.v_scale + sc0) : 0.f;
  bool seen = sc0 >= 0;

  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_s;
  const uint32_t tm_lane = tmem + ((uint32_t)(warp * 32) << 16);
  const uint64_t q_desc = umma_desc_sw128(smem_addr(q_s));
  const uint64_t p_desc = desc_plain_mn(smem_addr(p_s), 128, TILE * NH);
  volatile int* abort = abort_s;

  for (int c = 0; c < ntiles; ++c) {
    const uint32_t par = c & 1;
    // ---- S^T = K q^T
    attn::cp_async_wait<2>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (*abort) break;
    if (tid == 0) {
      tc_fence_after();
      const uint64_t kd = umma_desc_sw128(smem_addr(buf_s + ((2 * c) % BUFS) * BUF_BYTES));
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_e4m3(tmem, kd + (s >> 2) * (HALF_BYTES >> 4) + (s & 3) * 2,
                 q_desc + (s >> 2) * ((QN * 128) >> 4) + (s & 3) * 2, IDESC_S, s > 0);
      umma_commit(&bar[0]);
    }
    // while it runs: offsets of tile c + 2, and the look-ups behind them
    off_s[((c + 2) % RING) * TILE + tid] = off_of(j_nx, page_nx);
    const int64_t sc2 = scale_at(j_nx, page_nx);
    j_nx = j_nx2;
    page_nx = page_of(j_nx);
    j_nx2 = tok_of(c + 4);
    const float ks_nx = sc1 >= 0 ? __ldg(p.k_scale + sc1) : 0.f;
    const float vs_nx = sc1 >= 0 ? __ldg(p.v_scale + sc1) : 0.f;

    if (!mbar_wait(&bar[0], par, abort)) {
      record_device_error(QSA_DEVERR_WAIT_TIMEOUT);
      *abort_s = 1;
    }
    tc_fence_after();
    load_tile(p.v, c + 1, (2 * c) % BUFS);          // K of this tile is consumed

    float x[NH];
    {
      float a[NH], b[NH];
      tmem_ld16(tm_lane, a);
      tmem_ld16(tm_lane + NH, b);
      tmem_wait_ld();
#pragma unroll
      for (int h = 0; h < NH; ++h) x[h] = fmaf(b[h], 1.f / 16.f, a[h]);
      if (QT > 2) {
        tmem_ld16(tm_lane + 2 * NH, a);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < NH; ++h) x[h] = fmaf(a[h], 1.f / 256.f, x[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) x[h] = seen ? x[h] * (qc_s[h] * ks) : -INFINITY;
    if (p.part_s) {
      const int e = e_begin + c * TILE + tid;
      if (e < e_end) {
        float* dst = p.part_s + ((t * p.Hkv + g) * p.width + e) * p.group;
#pragma unroll
        for (int h = 0; h < NH; ++h)
          if (h < p.group) dst[h] = x[h];
      }
    }
    // ---- maxima over the tile
    const float vtop = warp_max(vs);
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float w = warp_max(x[h]);
      if (lane == h) red_s[warp * (NH + 4) + h] = w;
    }
    if (lane == NH) red_s[warp * (NH + 4) + NH] = vtop;
    __syncthreads();
    float alpha[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float m = m_run[h];
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, red_s[w * (NH + 4) + h]);
      const float mr = m == -INFINITY ? 0.f : m;   // nothing visible yet: every probability is 0
      alpha[h] = exp2f(m_run[h] - mr);
      x[h] = exp2f(x[h] - mr);
      m_run[h] = m;
      l_run[h] = fmaf(l_run[h], alpha[h], x[h]);
    }
    float vref = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) vref = fmaxf(vref, red_s[w * (NH + 4) + NH]);
    // ---- P times v_scale / vref, at most 256, as three E4M3 terms
    const float vn = vref > 0.f ? vs / vref * 256.f : 0.f;
#pragma unroll
    for (int h = 0; h < NH; ++h) x[h] *= vn;
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      uint32_t w4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t c0 = e4m3x2(x[4 * k], x[4 * k + 1]), c1 = e4m3x2(x[4 * k + 2], x[4 * k + 3]);
        w4[k] = c0 | (c1 << 16);
        if (q + 1 < PT) {
          const float2 f0 = e4m3x2_value(c0), f1 = e4m3x2_value(c1);
          x[4 * k] = (x[4 * k] - f0.x) * 16.f;
          x[4 * k + 1] = (x[4 * k + 1] - f0.y) * 16.f;
          x[4 * k + 2] = (x[4 * k + 2] - f1.x) * 16.f;
          x[4 * k + 3] = (x[4 * k + 3] - f1.y) * 16.f;
        }
      }
      *reinterpret_cast<uint4*>(p_s + (q * TILE + tid) * NH) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
    }
    // ---- O^T = V^T P
    attn::cp_async_wait<2>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (*abort) break;
    if (tid == 0) {
      tc_fence_after();
      const uint64_t vd = umma_desc_sw128(smem_addr(buf_s + ((2 * c + 1) % BUFS) * BUF_BYTES));
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_e4m3(tmem + S_COLS + hf * O_COLS, vd + hf * (HALF_BYTES >> 4) + s * (32 * 128 >> 4),
                   p_desc + s * (32 * NH >> 4), IDESC_O, s > 0);
      umma_commit(&bar[1]);
    }
    if (!mbar_wait(&bar[1], par, abort)) {
      record_device_error(QSA_DEVERR_WAIT_TIMEOUT);
      *abort_s = 1;
    }
    tc_fence_after();
    load_tile(p.k, c + 2, (2 * c + 1) % BUFS);      // V of this tile is consumed
    const float ov = vref * (1.f / 256.f);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float a[NH], b[NH], d[NH];
      const uint32_t at = tm_lane + S_COLS + hf * O_COLS;
      tmem_ld16(at, a);
      tmem_ld16(at + NH, b);
      tmem_ld16(at + 2 * NH, d);
      tmem_wait_ld();
      float* o = hf == 0 ? o0 : o1;
#pragma unroll
      for (int h = 0; h < NH; ++h)
        o[h] = fmaf(o[h], alpha[h], ov * fmaf(d[h], 1.f / 256.f, fmaf(b[h], 1.f / 16.f, a[h])));
    }
    seen = sc1 >= 0;
    ks = ks_nx;
    vs = vs_nx;
    sc1 = sc2;
  }
  attn::cp_async_wait<0>();

  // ---- the split's maximum, sum and unnormalised output
  __syncthreads();
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    float l = l_run[h];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == h) red_s[warp * (NH + 4) + h] = l;
  }
  tc_fence_before();
  __syncthreads();
  const int64_t base = (t * p.Hkv + g) * p.splits + split;
  float* po = p.part_o + base * p.group * D;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    if (h < p.group) {
      po[h * D + tid] = o0[h];
      po[h * D + 128 + tid] = o1[h];
      if (tid == h) {
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) l += red_s[w * (NH + 4) + h];
        p.part_ml[(base * p.group + h) * 2] = m_run[h];
        p.part_ml[(base * p.group + h) * 2 + 1] = l;
      }
    }
  }
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// One warp per (row, query head): merge the splits, gate, 16-bit output, LSE.
template <bool F16>
__global__ void __launch_bounds__(256) combine_fp8_kernel(const Params p) {
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= p.T * p.Hq) return;
  const int64_t t = wid / p.Hq;
  const int h = (int)(wid % p.Hq);
  const int g = h / p.group, hh = h % p.group;
  const int64_t base = (t * p.Hkv + g) * p.splits;
  float M = -INFINITY;
  for (int s = 0; s < p.splits; ++s) M = fmaxf(M, p.part_ml[((base + s) * p.group + hh) * 2]);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  const float Mr = M == -INFINITY ? 0.f : M;
  for (int s = 0; s < p.splits; ++s) {
    const float w = exp2f(p.part_ml[((base + s) * p.group + hh) * 2] - Mr);
    sum = fmaf(w, p.part_ml[((base + s) * p.group + hh) * 2 + 1], sum);
    const float* po = p.part_o + ((base + s) * p.group + hh) * D + lane * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, po[i], acc[i]);
  }
  float mul = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);   // a NaN sum stays NaN
  if (p.gate) mul *= 1.f / (1.f + expf(-p.gate[t * p.Hq + h]));
  uint32_t w4[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = acc[2 * i] * mul, b = acc[2 * i + 1] * mul;
    if (F16) {
      const __half2 v = __floats2half2_rn(a, b);
      w4[i] = *reinterpret_cast<const uint32_t*>(&v);
    } else {
      w4[i] = attn::pack_bf16(a, b);
    }
  }
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

// The 8-bit K/V cache around its attention: appending new tokens, adding
// attention weights up per cached token, dropping the lightest pages.
//
//  * append_kernel: one CTA per (scale block, KV head, K or V).  A block's
//    scale is the smallest power of two that holds its largest element
//    (amax <= 448 s), so the codes lose nothing to the scale, a grown scale
//    moves old codes by whole exponents (only what falls below E4M3's
//    normal range is rounded again), and attention reads back exact products.
//  * accumulate_kernel: one warp per 128 list entries of a row.  Weights are
//    counted in units of 2^-32 in 64-bit integers: the order of the atomics
//    cannot change the sums.
//  * page_weight_kernel, evict_kernel: one warp per logical page sums its
//    tokens; one CTA per request finds the lightest pages by a radix
//    selection over the 64-bit sums and writes the new table and the freed
//    pages in order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention_fp8.cuh"
#include "sm100.cuh"

namespace qsa {
namespace kv8 {

constexpr int D = 256;

// ---------------------------------------------------------------- append

constexpr int APPEND_WARPS = 4;

struct AppendParams {
  const uint16_t* x[2];       // new K, V rows [T, Hkv, 256]
  int64_t x_st[2], x_sh[2];
  uint8_t* cache[2];
  float* scale[2];
  int64_t num_pages;
  int32_t page_size, block_tokens;
  int64_t kv_page_stride, kv_row_stride, kv_head_stride;  // bytes
  int64_t sc_page_stride, sc_block_stride;                // elements
  int32_t Hkv;
  const int32_t* page_table;
  int64_t pt_stride;
  int32_t max_pages;
  const int32_t* cu;
  const int32_t* seq_lens;
  int32_t R;
  int64_t T;
  int64_t* token_weight;      // [num_pages, page_size] or null
};

// The smallest power of two s >= 2^-64 with top <= 448 s, as its exponent.
__device__ __forceinline__ int scale_exponent(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  return max(e, -64);
}

// x as 8 values; |x| of the finite ones
template <bool F16>
__device__ __forceinline__ void widen8(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = attn8::widen2<F16>(w[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ uint2 encode8(const float* x) {
  return make_uint2(attn8::e4m3x2(x[0], x[1]) | (attn8::e4m3x2(x[2], x[3]) << 16),
                    attn8::e4m3x2(x[4], x[5]) | (attn8::e4m3x2(x[6], x[7]) << 16));
}

// Slots of scale blocks: request r owns slots cu[r] / bt + 2 r onwards, which
// are enough (qlen rows touch at most qlen / bt + 2 blocks).
template <bool F16>
__global__ void __launch_bounds__(APPEND_WARPS * 32) append_kernel(const AppendParams p) {
  __shared__ float top_s[APPEND_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slot = blockIdx.x;
  const int h = blockIdx.y, which = blockIdx.z;
  const int bt = p.block_tokens;
  int lo = 0, hi = p.R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)(__ldg(p.cu + mid) / bt) + 2 * (int64_t)mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int first = __ldg(p.cu + lo), qlen = __ldg(p.cu + lo + 1) - first;
  const int L = __ldg(p.seq_lens + lo);
  if (qlen <= 0 || first < 0 || (int64_t)first + qlen > p.T) return;
  const int64_t p0 = (int64_t)L - qlen;             // position of the request's first new row
  const int64_t nth = slot - (first / bt + 2 * (int64_t)lo);
  // blocks do not cross pages: bt divides page_size
  const int64_t a = max(p0, (int64_t)0);
  const int64_t block0 = (a / bt + nth) * bt;       // first token of this block
  if (block0 >= L) return;
  const int64_t begin = max(block0, a);
  const int n_new = (int)(min(block0 + bt, (int64_t)L) - begin);
  const int n_old = (int)(begin - block0);
  const int64_t lp = block0 / p.page_size;
  const int page = lp < p.max_pages ? __ldg(p.page_table + (int64_t)lo * p.pt_stride + lp) : -1;
  if (page < 0 || page >= p.num_pages) return;      // no page: the tokens are dropped
  const int in_page = (int)(block0 - lp * p.page_size);
  const uint16_t* x = p.x[which] + (first + (begin - p0)) * p.x_st[which] + h * p.x_sh[which] + lane * 8;
  uint8_t* rows = p.cache[which] + page * p.kv_page_stride + in_page * p.kv_row_stride + h * p.kv_head_stride + lane * 8;
  float* sc = p.scale[which] + page * p.sc_page_stride + (in_page / bt) * p.sc_block_stride + h;

  float top = 0.f;
  for (int i = warp; i < n_new; i += APPEND_WARPS) {
    float f[8];
    widen8<F16>(__ldg(reinterpret_cast<const uint4*>(x + i * p.x_st[which])), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[k]) <= 3.4e38f ? fabsf(f[k]) : 0.f);
  }
  top = attn8::warp_max(top);
  if (lane == 0) top_s[warp] = top;
  const float before = n_old > 0 ? *sc : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < APPEND_WARPS; ++w) top = fmaxf(top, top_s[w]);
  const float s = fmaxf(before, __uint_as_float((uint32_t)(scale_exponent(top) + 127) << 23));
  if (threadIdx.x == 0 && s != before) *sc = s;
  if (n_old > 0 && s != before) {
    const float ratio = before / s;
    for (int i = warp; i < n_old; i += APPEND_WARPS) {
      uint2* at = reinterpret_cast<uint2*>(rows + i * p.kv_row_stride);
      const uint2 c = *at;
      float f[8];
      const float2 f0 = attn8::e4m3x2_value(c.x & 0xffffu), f1 = attn8::e4m3x2_value(c.x >> 16);
      const float2 f2 = attn8::e4m3x2_value(c.y & 0xffffu), f3 = attn8::e4m3x2_value(c.y >> 16);
      f[0] = f0.x * ratio; f[1] = f0.y * ratio; f[2] = f1.x * ratio; f[3] = f1.y * ratio;
      f[4] = f2.x * ratio; f[5] = f2.y * ratio; f[6] = f3.x * ratio; f[7] = f3.y * ratio;
      *at = encode8(f);
    }
  }
  for (int i = warp; i < n_new; i += APPEND_WARPS) {
    float f[8];
    widen8<F16>(__ldg(reinterpret_cast<const uint4*>(x + i * p.x_st[which])), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = f[k] / s;
    *reinterpret_cast<uint2*>(rows + (int64_t)(n_old + i) * p.kv_row_stride) = encode8(f);
  }
  if (p.token_weight && h == 0 && which == 0)
    for (int i = threadIdx.x; i < n_new; i += blockDim.x)
      p.token_weight[(int64_t)page * p.page_size + in_page + n_old + i] = 0;
}

// ---------------------------------------------------------------- accumulate

struct AccumulateParams {
  const float* weights;       // [T, width]
  int64_t w_stride;
  const int32_t* tok;
  int64_t tok_stride;
  int32_t width;
  int64_t T;
  int64_t num_pages;
  int32_t page_size;
  const int32_t* page_table;
  int64_t pt_stride;
  int32_t max_pages;
  const int32_t* cu;
  const int32_t* seq_lens;
  int32_t R;
  unsigned long long* token_weight;
  int32_t chunks;             // warps per row
};

constexpr int ACC_PER_WARP = 128;
constexpr float ACC_MOST = 1048576.f;   // one weight counts at most 2^20

__global__ void __launch_bounds__(256) accumulate_kernel(const AccumulateParams p) {
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= p.T * p.chunks) return;
  const int64_t t = wid / p.chunks;
  const int e0 = (int)(wid % p.chunks) * ACC_PER_WARP + lane;
  int j[ACC_PER_WARP / 32];
  float w[ACC_PER_WARP / 32];
#pragma unroll
  for (int i = 0; i < ACC_PER_WARP / 32; ++i) {
    const int e = e0 + 32 * i;
    j[i] = e < p.width ? __ldg(p.tok + t * p.tok_stride + e) : -1;
    w[i] = e < p.width ? __ldg(p.weights + t * p.w_stride + e) : 0.f;
  }
  int r, pos, L;
  attn8::row_position(p.cu, p.seq_lens, p.R, t, lane, r, pos, L);
  const int32_t* pt_row = p.page_table + (int64_t)r * p.pt_stride;
#pragma unroll
  for (int i = 0; i < ACC_PER_WARP / 32; ++i) {
    // NaN and weights at or below 0 add nothing
    if (j[i] < 0 || j[i] > pos || j[i] >= L || !(w[i] > 0.f)) continue;
    const int lp = j[i] / p.page_size;
    const int page = lp < p.max_pages ? __ldg(pt_row + lp) : -1;
    if (page < 0 || page >= p.num_pages) continue;
    const double units = (double)fminf(w[i], ACC_MOST) * 4294967296.0;
    atomicAdd(p.token_weight + (int64_t)page * p.page_size + (j[i] - lp * p.page_size),
              (unsigned long long)__double2ll_rn(units));
  }
}

// ---------------------------------------------------------------- eviction

struct EvictParams {
  const int64_t* token_weight;  // [num_pages, page_size]
  int64_t num_pages;
  int32_t page_size;
  const int32_t* page_table;
  int64_t pt_stride;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* keep;
  int32_t R;
  int32_t keep_first, keep_last;
  int32_t* table_out;
  int64_t out_stride;
  int32_t* freed;               // [R, max_pages]
  int64_t freed_stride;
  int32_t* counts;
  unsigned long long* key;      // workspace [R, max_pages]: page weight, ordered as an unsigned number
};

__device__ __forceinline__ int logical_pages(const EvictParams& p, int r) {
  const int L = __ldg(p.seq_lens + r);
  return L <= 0 ? 0 : (int)min((int64_t)p.max_pages, ((int64_t)L + p.page_size - 1) / p.page_size);
}

__global__ void __launch_bounds__(256) page_weight_kernel(const EvictParams p) {
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (int64_t)p.R * p.max_pages) return;
  const int r = (int)(wid / p.max_pages), lp = (int)(wid % p.max_pages);
  if (lp >= logical_pages(p, r)) return;
  const int page = __ldg(p.page_table + (int64_t)r * p.pt_stride + lp);
  if (page < 0 || page >= p.num_pages) return;
  unsigned long long sum = 0;
  const int64_t* w = p.token_weight + (int64_t)page * p.page_size;
  for (int i = lane; i < p.page_size; i += 32) sum += (unsigned long long)__ldg(reinterpret_cast<const long long*>(w + i));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) p.key[wid] = sum ^ (1ull << 63);
}

constexpr int EVICT_THREADS = 1024;

// Sum over the CTA of one int per thread, and the exclusive prefix.
__device__ __forceinline__ int block_prefix(int v, int* warp_s, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < EVICT_THREADS / 32; ++w) {
    const int y = warp_s[w];
    if (w < warp) before += y;
    total += y;
  }
  return before + inc - v;
}

__global__ void __launch_bounds__(EVICT_THREADS) evict_kernel(const EvictParams p) {
  __shared__ int warp_s[EVICT_THREADS / 32];
  __shared__ int hist[256];
  __shared__ unsigned long long prefix_s;
  __shared__ int want_s;
  const int r = blockIdx.x, tid = threadIdx.x;
  const int n = logical_pages(p, r);
  const int32_t* row = p.page_table + (int64_t)r * p.pt_stride;
  int32_t* out = p.table_out + (int64_t)r * p.out_stride;
  int32_t* freed = p.freed + (int64_t)r * p.freed_stride;
  const unsigned long long* key = p.key + (int64_t)r * p.max_pages;
  auto live = [&](int lp) { return lp < n && row[lp] >= 0 && row[lp] < p.num_pages; };
  auto held = [&](int lp) { return lp < p.keep_first || lp >= n - p.keep_last; };

  int n_held = 0, n_free = 0;
  for (int lp = tid; lp < n; lp += EVICT_THREADS)
    if (live(lp)) (held(lp) ? n_held : n_free)++;
  int all_held, all_free;
  block_prefix(n_held, warp_s, all_held);
  block_prefix(n_free, warp_s, all_free);
  const int quota = max(0, min(all_free, (int)__ldg(p.keep + r) - all_held));  // pages that may stay

  // the quota-th largest key: its value and how many equal to it stay
  unsigned long long prefix = 0, mask = 0;
  int want = quota;
  if (quota > 0 && quota < all_free) {
    for (int shift = 56; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int lp = tid; lp < n; lp += EVICT_THREADS)
        if (live(lp) && !held(lp) && (key[lp] & mask) == prefix) atomicAdd(&hist[(key[lp] >> shift) & 255], 1);
      __syncthreads();
      if (tid == 0) {
        int b = 255, left = want;
        while (b > 0 && hist[b] < left) left -= hist[b--];
        prefix_s = prefix | ((unsigned long long)b << shift);
        want_s = left;
      }
      __syncthreads();
      prefix = prefix_s;
      want = want_s;
      mask |= 255ull << shift;
    }
  }
  // in page order: the first `want` pages at the threshold stay, then the new table and the freed list
  int ties = 0, gone = 0;
  for (int base = 0; base < p.max_pages; base += EVICT_THREADS) {
    const int lp = base + tid;
    const int entry = lp < p.max_pages ? row[lp] : -1;
    const bool may = lp < p.max_pages && live(lp) && !held(lp);
    const unsigned long long k = may ? key[lp] : 0;
    const bool tie = may && quota > 0 && quota < all_free && k == prefix;
    int total;
    const int at = ties + block_prefix(tie ? 1 : 0, warp_s, total);
    ties += total;
    const bool stays = !may || quota >= all_free || (quota > 0 && (k > prefix || (tie && at < want)));
    const int to = gone + block_prefix(stays ? 0 : 1, warp_s, total);
    gone += total;
    if (lp < p.max_pages) {
      out[lp] = stays ? entry : -1;
      if (!stays) freed[to] = entry;
    }
  }
  for (int i = gone + tid; i < p.max_pages; i += EVICT_THREADS) freed[i] = -1;
  if (tid == 0) p.counts[r] = gone;
}

}  // namespace kv8
}  // namespace qsa

// The 8-bit K/V cache around its attention: appending new tokens, adding
// attention weights up per cached token, dropping the lightest pages.
//
//  * append_kernel: one CTA, or for small blocks one warp, per (scale block, KV head, K or V).  A block's
//    scale is the smallest power of two that holds its largest element
//    (amax <= 448 s), so the codes lose nothing to the scale, a grown scale
//    moves old codes by whole exponents (only what falls below E4M3's
//    normal range is rounded again), and attention reads back exact products.
//    Bound by the chain lengths -> rows and page -> scale (2.9 us for 16 tokens)
//    and, for many rows, by how many CTAs hide it: 8,192 rows 8.2 us (25 MB).
//  * accumulate_kernel: a warp per run of a row's list entries.  Weights are
//    counted in units of 2^-32 in 64-bit integers: the order of the atomics
//    cannot change the sums.  4.2 M entries take 13.6 us, whatever a warp holds:
//    the rate of 64-bit atomics (310 G/s).
//  * evict_kernel: one CTA per request.  Groups of lanes sum the tokens of a
//    logical page each, then the CTA finds the lightest pages by a radix
//    selection over the 64-bit sums and writes the new table and the freed pages
//    in order.  For long tables, which one SM would read too slowly, and many
//    requests page_weight_kernel sums the pages on the whole GPU first.
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

// (out of line: eight of them in every store would make the kernel's code slower to fetch than its data)
__device__ __noinline__ float quotient(float a, float b) { return a / b; }

// Slots of scale blocks: request r owns slots cu[r] / bt + 2 r onwards, which
// are enough (qlen rows touch at most qlen / bt + 2 blocks).  Up to HELD rows a
// warp stay in registers between the maximum and the quantisation; the rows of
// longer blocks (LONG) are read again, out of L1 or L2.  Little code matters: the
// kernel runs for a few microseconds, much of it while instructions are fetched.
template <bool F16, int WARPS, int HELD, bool LONG>   // warps a block: all of the CTA's or one
__global__ void __launch_bounds__(APPEND_WARPS * 32) append_kernel(const AppendParams p) {
  __shared__ float top_s[APPEND_WARPS];
  const int warp = WARPS == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slot = WARPS == 1 ? (int64_t)blockIdx.x * APPEND_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  const int h = blockIdx.y, which = blockIdx.z;
  const int bt = p.block_tokens;
  // the last request whose slots begin at or before this one, 32 candidates a round trip
  int r = 0, left = p.R;
  while (left > 1) {
    const int step = (left + 31) >> 5, i = r + lane * step;
    const bool le = i < r + left && (int64_t)(__ldg(p.cu + i) / bt) + 2 * (int64_t)i <= slot;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    r += k * step;
    left = min(step, left - k * step);
  }
  const int first = __ldg(p.cu + r), qlen = __ldg(p.cu + r + 1) - first;
  const int L = __ldg(p.seq_lens + r);
  if (qlen <= 0 || first < 0 || (int64_t)first + qlen > p.T) return;
  const int64_t p0 = (int64_t)L - qlen;             // position of the request's first new row
  const int64_t nth = slot - (first / bt + 2 * (int64_t)r);
  // blocks do not cross pages: bt divides page_size
  const int64_t a = max(p0, (int64_t)0);
  const int64_t block0 = (a / bt + nth) * bt;       // first token of this block
  if (nth < 0 || block0 >= L) return;               // nth < 0: rows in front of the first request's
  const int64_t begin = max(block0, a);
  const int n_new = (int)(min(block0 + bt, (int64_t)L) - begin);
  const int n_old = (int)(begin - block0);
  const int64_t x_st = p.x_st[which];
  const uint16_t* x = p.x[which] + (first + (begin - p0)) * x_st + h * p.x_sh[which] + lane * 8;
  constexpr int ROUND = HELD * WARPS;               // rows in flight at once
  auto load = [&](int from, uint4 (&to)[HELD]) {
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (from + i * WARPS < n_new) to[i] = __ldg(reinterpret_cast<const uint4*>(x + (from + i * WARPS) * x_st));
  };
  uint4 row[HELD];
  load(warp, row);
  const int lp = (int)block0 / p.page_size;
  const int page = lp < p.max_pages ? __ldg(p.page_table + (int64_t)r * p.pt_stride + lp) : -1;
  if (page < 0 || page >= p.num_pages) return;      // no page: the tokens are dropped
  const int in_page = (int)block0 - lp * p.page_size;
  uint8_t* rows = p.cache[which] + page * p.kv_page_stride + in_page * p.kv_row_stride + h * p.kv_head_stride + lane * 8;
  float* sc = p.scale[which] + page * p.sc_page_stride + (in_page / bt) * p.sc_block_stride + h;
  const float before = n_old > 0 ? *sc : 0.f;

  // largest finite magnitude, as a 16-bit pattern of its type
  uint32_t top = 0;
  auto measure = [&](uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = w[k] & 0x7fff7fffu;
      const uint32_t fin = __vcmpltu2(m, F16 ? 0x7c007c00u : 0x7f807f80u);
      top = __vmaxu2(top, m & fin);
    }
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (warp + i * WARPS < n_new) measure(row[i]);
  if (LONG) {
#pragma unroll 1
    for (int from = warp + ROUND; from < n_new; from += ROUND) {
      uint4 more[HELD];                               // read again below, out of L1 or L2
      load(from, more);
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (from + i * WARPS < n_new) measure(more[i]);
    }
  }
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  float amax = 0.f;
  if (WARPS == 1) {
    amax = attn8::widen2<F16>(top).x;
  } else {
    if (lane == 0) top_s[warp] = attn8::widen2<F16>(top).x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, top_s[w]);
  }
  const float s = fmaxf(before, __uint_as_float((uint32_t)(scale_exponent(amax) + 127) << 23));
  if (warp == 0 && lane == 0 && s != before) *sc = s;
  if (n_old > 0 && s != before) {
    const float ratio = before / s;
    for (int i = warp; i < n_old; i += WARPS) {
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
  // x / s: a power of two's reciprocal is exact; a scale of another writer's is divided by
  const uint32_t sb = __float_as_uint(s);
  const bool pow2 = (sb & 0x7fffffu) == 0 && sb > 0 && sb < 0x7e800000u;
  const float inv = 1.f / s;
  auto store = [&](int i, uint4 v) {
    float f[8];
    widen8<F16>(v, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = pow2 ? f[k] * inv : quotient(f[k], s);
    *reinterpret_cast<uint2*>(rows + (int64_t)(n_old + i) * p.kv_row_stride) = encode8(f);
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (warp + i * WARPS < n_new) store(warp + i * WARPS, row[i]);
  if (LONG) {
#pragma unroll 1
    for (int from = warp + ROUND; from < n_new; from += ROUND) {
      load(from, row);
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (from + i * WARPS < n_new) store(from + i * WARPS, row[i]);
    }
  }
  if (p.token_weight && h == 0 && which == 0)
    for (int i = 32 * warp + lane; i < n_new; i += 32 * WARPS)
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
  attn8::FastDiv by_page;
};

constexpr float ACC_MOST = 1048576.f;   // one weight counts at most 2^20

template <int PER>   // list entries a lane
__global__ void __launch_bounds__(256) accumulate_kernel(const AccumulateParams p) {
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= p.T * p.chunks) return;
  const int64_t t = wid / p.chunks;
  const int e0 = (int)(wid % p.chunks) * (32 * PER) + lane;
  int j[PER];
  float w[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + 32 * i;
    j[i] = e < p.width ? __ldg(p.tok + t * p.tok_stride + e) : -1;
    w[i] = e < p.width ? __ldg(p.weights + t * p.w_stride + e) : 0.f;
  }
  int r, pos, L;
  attn8::row_position(p.cu, p.seq_lens, p.R, t, lane, r, pos, L);
  const int32_t* pt_row = p.page_table + (int64_t)r * p.pt_stride;
  int page[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    // NaN and weights at or below 0 add nothing
    const bool adds = j[i] >= 0 && j[i] <= pos && j[i] < L && w[i] > 0.f;
    const int lp = adds ? attn8::divide(j[i], p.by_page) : 0;
    page[i] = adds && lp < p.max_pages ? __ldg(pt_row + lp) : -1;
    j[i] -= lp * p.page_size;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (page[i] < 0 || page[i] >= p.num_pages) continue;
    const double units = (double)fminf(w[i], ACC_MOST) * 4294967296.0;
    atomicAdd(p.token_weight + (int64_t)page[i] * p.page_size + j[i], (unsigned long long)__double2ll_rn(units));
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

// Token weights of WEIGH_EACH pages at a time, `lanes` lanes a page, two tokens a
// load where rows allow it.  Pages below 0 have none.  The sums over lanes are
// scattered on the way (each step halves what a lane holds, 18 shuffles instead
// of 80 at 32 lanes): put(b, sum) is called once for every page.
constexpr int WEIGH_EACH = 8;

template <bool PAIRS, typename Put>
__device__ __forceinline__ void weigh(const EvictParams& p, const int (&page)[WEIGH_EACH], int sub, int lanes, Put put) {
  unsigned long long v[WEIGH_EACH];
#pragma unroll
  for (int b = 0; b < WEIGH_EACH; ++b) v[b] = 0;
  constexpr int STEP = PAIRS ? 2 : 1;
  for (int e = STEP * sub; e < p.page_size; e += STEP * lanes) {
    ulonglong2 x[WEIGH_EACH];                          // all loads before the sums
#pragma unroll
    for (int b = 0; b < WEIGH_EACH; ++b) {
      const int64_t* w = p.token_weight + (int64_t)page[b] * p.page_size + e;
      x[b] = make_ulonglong2(0, 0);
      if (page[b] >= 0) {
        if (PAIRS) x[b] = __ldg(reinterpret_cast<const ulonglong2*>(w));
        else x[b].x = __ldg(reinterpret_cast<const unsigned long long*>(w));
      }
    }
#pragma unroll
    for (int b = 0; b < WEIGH_EACH; ++b) v[b] += x[b].x + x[b].y;
  }
  int first = 0, held = WEIGH_EACH, o = lanes >> 1;    // this lane holds pages first .. first + held - 1
#pragma unroll
  for (int half = WEIGH_EACH / 2; half >= 1; half >>= 1) {
    if (o > 0) {
      const bool upper = (sub & o) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const unsigned long long keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
      first += upper ? half : 0;
      held = half;
      o >>= 1;
    }
  }
  const int copies = o > 0 ? 2 * o : 1;                // lanes that end with the same page
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  if ((sub & (copies - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < WEIGH_EACH; ++i)
      if (i < held) put(first + i, v[i]);
  }
}

__device__ __forceinline__ int logical_pages(const EvictParams& p, int r) {
  const int L = __ldg(p.seq_lens + r);
  return L <= 0 ? 0 : (int)min((int64_t)p.max_pages, ((int64_t)L + p.page_size - 1) / p.page_size);
}

// Page weights into the workspace: every group of lanes takes WEIGH_EACH
// logical pages of one request, all in flight at once.
constexpr int WEIGH_THREADS = 128;

template <bool PAIRS>
__global__ void __launch_bounds__(WEIGH_THREADS) page_weight_kernel(const EvictParams p, int lanes) {
  __shared__ int page_s[WEIGH_THREADS * WEIGH_EACH];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int sub = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = WEIGH_THREADS / lanes;
  const int r = blockIdx.y, base = blockIdx.x * groups * WEIGH_EACH, n = logical_pages(p, r);
  if (base >= n) return;
  for (int i = threadIdx.x; i < groups * WEIGH_EACH; i += WEIGH_THREADS) {
    const int page = base + i < n ? __ldg(p.page_table + (int64_t)r * p.pt_stride + base + i) : -1;
    page_s[i] = page < p.num_pages ? page : -1;
  }
  __syncthreads();
  int page[WEIGH_EACH];
#pragma unroll
  for (int b = 0; b < WEIGH_EACH; ++b) page[b] = page_s[b * groups + group];
  unsigned long long* key = p.key + (int64_t)r * p.max_pages + base;
  weigh<PAIRS>(p, page, sub, lanes, [&](int b, unsigned long long sum) {
    if (page_s[b * groups + group] >= 0) key[b * groups + group] = sum ^ (1ull << 63);
  });
}

// Selection: a thread holds PER consecutive pages in registers (PER * THREADS
// >= max_pages) or, for longer tables (PER = 0), looks them up again in every
// pass.
constexpr int BINS = 512;                              // of a pass: 9 bits
constexpr int PASSES = 8;                              // the first and up to 61 open bits after it
enum Weights { FROM_WORKSPACE, HERE, HERE_IN_PAIRS };  // where the page weights come from

// Exclusive prefix over the CTA of one int per thread, and the total.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int* warp_s, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                                     // warp_s may still be read
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  constexpr int WARPS = THREADS / 32;
  int ws = lane < WARPS ? warp_s[lane] : 0, wi = ws;   // every warp scans the warp sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += y;
  }
  total = __shfl_sync(0xffffffffu, wi, 31);
  return __shfl_sync(0xffffffffu, wi - ws, warp) + inc - v;
}

template <int THREADS, int PER, Weights FORM>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_kernel(const EvictParams p, int lanes) {
  extern __shared__ unsigned long long key_s[];        // page weights summed here
  __shared__ int warp_s[THREADS / 32];
  __shared__ int hist_s[PASSES][BINS];
  __shared__ unsigned long long and_s, or_s;
  __shared__ int held_s, free_s, bin_s, left_s;
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = logical_pages(p, r);
  const int32_t* row = p.page_table + (int64_t)r * p.pt_stride;
  int32_t* out = p.table_out + (int64_t)r * p.out_stride;
  int32_t* freed = p.freed + (int64_t)r * p.freed_stride;
  const unsigned long long* keys = FORM == FROM_WORKSPACE ? p.key + (int64_t)r * p.max_pages : key_s;
  const int want_keep = max(0, __ldg(p.keep + r));
  auto is_live = [&](int lp, int entry) { return lp < n && entry >= 0 && entry < p.num_pages; };
  auto is_held = [&](int lp) { return lp < p.keep_first || lp >= n - p.keep_last; };

  constexpr int HOLD = PER > 0 ? PER : 1;
  int entry[HOLD];
  unsigned long long key[HOLD];
  bool may[HOLD];                                      // live and not held: may be dropped
  int n_held = 0, n_free = 0;
  if (PER > 0) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int lp = tid * HOLD + i;
      entry[i] = lp < p.max_pages ? row[lp] : -1;
      const bool live = is_live(lp, entry[i]);
      may[i] = live && !is_held(lp);
      n_held += live && !may[i];
      n_free += may[i];
    }
  } else {
    for (int lp = tid; lp < n; lp += THREADS)
      if (is_live(lp, row[lp])) (is_held(lp) ? n_held : n_free)++;
  }
  for (int i = tid; i < PASSES * BINS; i += THREADS) hist_s[i / BINS][i % BINS] = 0;
  if (FORM != FROM_WORKSPACE) {
    int* page_s = reinterpret_cast<int*>(key_s + HOLD * THREADS);
#pragma unroll
    for (int i = 0; i < HOLD; ++i) page_s[tid * HOLD + i] = may[i] ? entry[i] : -1;
    __syncthreads();
    const int sub = tid & (lanes - 1), group = tid / lanes, groups = THREADS / lanes;
    for (int base = 0; base < n; base += groups * WEIGH_EACH) {
      auto at = [&](int b) { return base + b * groups + group; };
      int page[WEIGH_EACH];
#pragma unroll
      for (int b = 0; b < WEIGH_EACH; ++b) page[b] = at(b) < n ? page_s[at(b)] : -1;
      weigh<FORM == HERE_IN_PAIRS>(p, page, sub, lanes, [&](int b, unsigned long long sum) {
        if (at(b) < n) key_s[at(b)] = sum ^ (1ull << 63);
      });
    }
  }
  if (tid == 0) {
    and_s = ~0ull;
    or_s = 0;
    held_s = free_s = 0;
  }
  __syncthreads();
  if (FORM == FROM_WORKSPACE) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (PER > 0) {
#pragma unroll
    for (int i = 0; i < HOLD; ++i) key[i] = may[i] ? keys[tid * HOLD + i] : 0;
  }
  // every droppable page's key, in no particular order
  auto each_key = [&](auto&& f) {
    if (PER > 0) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (may[i]) f(key[i]);
    } else {
      for (int lp = tid; lp < n; lp += THREADS)
        if (is_live(lp, row[lp]) && !is_held(lp)) f(keys[lp]);
    }
  };
  unsigned long long all_and = ~0ull, all_or = 0;
  each_key([&](unsigned long long k) {
    all_and &= k;
    all_or |= k;
  });
  n_held = __reduce_add_sync(0xffffffffu, n_held);
  n_free = __reduce_add_sync(0xffffffffu, n_free);
  const uint32_t and_lo = __reduce_and_sync(0xffffffffu, (uint32_t)all_and);
  const uint32_t and_hi = __reduce_and_sync(0xffffffffu, (uint32_t)(all_and >> 32));
  const uint32_t or_lo = __reduce_or_sync(0xffffffffu, (uint32_t)all_or);
  const uint32_t or_hi = __reduce_or_sync(0xffffffffu, (uint32_t)(all_or >> 32));
  if (lane == 0) {
    if (n_held) atomicAdd(&held_s, n_held);
    if (n_free) {
      atomicAdd(&free_s, n_free);
      atomicAnd(&and_s, ((unsigned long long)and_hi << 32) | and_lo);
      atomicOr(&or_s, ((unsigned long long)or_hi << 32) | or_lo);
    }
  }
  __syncthreads();
  const int all_free = free_s;
  const int quota = max(0, min(all_free, want_keep - held_s));     // droppable pages that stay
  const bool some = quota > 0 && quota < all_free;

  // The quota-th largest key: pages stay when key & mask > prefix, and the first `want` pages when they are equal.
  unsigned long long prefix = 0, mask = 0;
  int want = quota;
  bool whole = true;                                   // every page at the threshold stays
  if (some) {
    // leading bits in which all keys agree need no pass
    const unsigned long long differ = and_s ^ or_s;
    int top = differ ? 64 - __clzll((long long)differ) : 0;   // bits below `top` are open
    mask = top >= 64 ? 0 : ~0ull << top;
    prefix = and_s & mask;
    whole = top > 0;                                   // all keys equal: the first ones stay
    // Histogram of the keys that share the prefix, then the bin of the want-th largest (bin_s), how many of it stay.
    auto find = [&](int* hist, auto&& bin_of) {
      each_key([&](unsigned long long k) {
        if ((k & mask) == prefix) atomicAdd(&hist[bin_of(k)], 1);
      });
      __syncthreads();
      if (warp == 0) {
        // lane l sums bins 16 (31 - l) .. + 15, so that a prefix over lanes counts from the largest bin down
        const int b0 = BINS / 32 * (31 - lane);
        int sum = 0;
#pragma unroll
        for (int b = 0; b < BINS / 32; ++b) sum += hist[b0 + b];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (inc >= want && inc - sum < want) {         // the threshold's bin is among this lane's
          int left = want - (inc - sum), b = BINS / 32 - 1;
          while (b > 0 && hist[b0 + b] < left) left -= hist[b0 + b--];
          bin_s = b0 + b;
          left_s = left;
        }
      }
      __syncthreads();
      want = left_s;
      whole = hist[bin_s] == want;
      return bin_s;
    };
    // First by the highest bit that differs and the 3 below it: weights spread over many powers of two, and bins of
    // equal width would put most of them (and their atomics) in one.
    int pass = 0;
    if (top > 0) {
      const unsigned long long low = top >= 64 ? ~0ull : (1ull << top) - 1;
      const int b = find(hist_s[pass++], [&](unsigned long long k) {
        const unsigned long long v = k & low;
        const int m = 63 - __clzll((long long)(v | 1));
        return m < 3 ? (int)v : 8 * (m - 2) + (int)((v >> (m - 3)) & 7);
      });
      top = b < 8 ? 0 : b / 8 - 1;                     // bits still open: below m - 3, m = b / 8 + 2
      prefix |= b < 8 ? (unsigned long long)b : (unsigned long long)(8 + (b & 7)) << top;
      mask = ~0ull << top;
    }
    while (top > 0 && !whole) {
      const int bits = min(9, top), shift = top - bits;
      __syncthreads();                                 // bin_s and left_s are read
      const int b = find(hist_s[pass++], [&](unsigned long long k) { return (int)(k >> shift) & ((1 << bits) - 1); });
      prefix |= (unsigned long long)b << shift;
      mask |= ((1ull << bits) - 1) << shift;
      top = shift;
    }
  }
  if (PER > 0) {
    int rank = 0, total;
    if (!whole) {                                      // the tied pages' order decides
      int ties = 0;
#pragma unroll
      for (int i = 0; i < HOLD; ++i) ties += may[i] && (key[i] & mask) == prefix;
      rank = block_prefix<THREADS>(ties, warp_s, total);
    }
    bool stays[HOLD];
    int gone = 0;
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const unsigned long long k = key[i] & mask;
      const bool tie = may[i] && k == prefix;
      stays[i] = !may[i] || quota >= all_free || (some && (k > prefix || (tie && (whole || rank < want))));
      rank += tie;
      gone += !stays[i];
    }
    int at = block_prefix<THREADS>(gone, warp_s, total);
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int lp = tid * HOLD + i;
      if (lp >= p.max_pages) break;
      out[lp] = stays[i] ? entry[i] : -1;
      if (!stays[i]) freed[at++] = entry[i];
    }
    for (int i = total + tid; i < p.max_pages; i += THREADS) freed[i] = -1;
    if (tid == 0) p.counts[r] = total;
  } else {
    int ties = 0, gone = 0;
    for (int base = 0; base < p.max_pages; base += THREADS) {
      const int lp = base + tid;
      const int e = lp < p.max_pages ? row[lp] : -1;
      const bool drop = is_live(lp, e) && !is_held(lp);
      const unsigned long long k = drop ? keys[lp] & mask : 0;
      const bool tie = some && drop && k == prefix;
      int total;
      const int rank = ties + block_prefix<THREADS>(tie ? 1 : 0, warp_s, total);
      ties += total;
      const bool stays = !drop || quota >= all_free || (some && (k > prefix || (tie && rank < want)));
      const int to = gone + block_prefix<THREADS>(stays ? 0 : 1, warp_s, total);
      gone += total;
      if (lp < p.max_pages) {
        out[lp] = stays ? e : -1;
        if (!stays) freed[to] = e;
      }
    }
    for (int i = gone + tid; i < p.max_pages; i += THREADS) freed[i] = -1;
    if (tid == 0) p.counts[r] = gone;
  }
}

}  // namespace kv8
}  // namespace qsa

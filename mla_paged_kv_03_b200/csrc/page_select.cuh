// page_select.cuh -- sparse decode over whole pages of the dense cache: one
// int8 key per page, kept beside the cache, scores the pages for each query,
// and the attention then reads the best pages only.
//
// Page key: the mean m of the page's rows (576 dims, the rows the sequence
// has), scale = max|m| * (1/127) (1 for a zero mean), code = round(m / scale).
// Query codes: the same per head row of q.
// Score of page p for query (b, i): max over heads h of
//     (s_h * (q8_h . k8_p)) * scale_p
// The integer products are exact and below 2^24 (576 * 127^2), so every step
// is one fp32 operation with a defined order: equal inputs score equal, and the
// selection does not depend on how the sums are split.
// Selection: the page that ends the query's tokens is always taken, and the
// topk - 1 pages of highest score before it; of equal scores the lowest page.
// The taken pages in ascending order form a block table of their own, with the
// (possibly partial) last page at its end, over which the dense decode runs.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "combine_kernel.cuh"

namespace mla {

constexpr float kInv127 = 1.0f / 127.0f;

__device__ __forceinline__ float int8_scale(float amax) {
  const float s = amax * kInv127;
  return s > 0.f ? s : 1.f;
}

__device__ __forceinline__ int int8_code(float x, float scale) {
  const int c = __float2int_rn(x / scale);  // 0 for NaN
  return max(-127, min(127, c));
}

__device__ __forceinline__ uint32_t pack_int8x4(int a, int b, int c, int d) {
  return (a & 0xFF) | ((b & 0xFF) << 8) | ((c & 0xFF) << 16) | (static_cast<uint32_t>(d) << 24);
}

// ------------------------------------------------------------------ page keys

struct PageKeysParams {
  const __nv_bfloat16* kcache;  // [num_blocks, 64, 576]
  int num_blocks;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seqlens;
  int tail;          // the last `tail` pages of each sequence
  int8_t* keys;      // [num_blocks, 576]
  float* scales;     // [num_blocks]
};

constexpr int kKeyUnits = kD / 8;      // 16-byte units of a row
constexpr int kKeyRowGroups = 4;       // threads that share a unit, each every 4th row
constexpr int kKeyThreads = kKeyUnits * kKeyRowGroups;  // 288

// grid (tail, batch), one CTA per page.  The sums are formed in fp64, where 64
// bf16 values add exactly unless they lie 39 binades apart: the code does not
// depend on the order, and a mean next to a rounding border is decided by its
// value.  HBM bound: 73.7 kB read a page.
__global__ void __launch_bounds__(kKeyThreads) mla_page_keys_kernel(const PageKeysParams P) {
  __shared__ double s_sum[kKeyRowGroups][kD];
  __shared__ float s_max[kKeyThreads / 32];
  const int b = blockIdx.y;
  int L = P.seqlens[b];
  if (L > P.max_pages * kPage) {
    if (threadIdx.x == 0) ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x72);
    L = P.max_pages * kPage;
  }
  const int page = (L + kPage - 1) / kPage - P.tail + static_cast<int>(blockIdx.x);
  if (L <= 0 || page < 0) return;
  const int blk = clamp_block(P.block_table[static_cast<size_t>(b) * P.max_pages + page],
                              P.num_blocks);
  const int n = min(kPage, L - page * kPage);
  const int unit = threadIdx.x % kKeyUnits, group = threadIdx.x / kKeyUnits;
  const uint4* src = reinterpret_cast<const uint4*>(P.kcache + static_cast<size_t>(blk) * kPage * kD) +
                     unit;
  constexpr int kRowsPerThread = kPage / kKeyRowGroups;
  uint4 w[kRowsPerThread];
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const int row = group + kKeyRowGroups * i;
    w[i] = row < n ? __ldg(src + row * kKeyUnits) : make_uint4(0, 0, 0, 0);
  }
  double sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0;
#pragma unroll
  for (int i = 0; i < kRowsPerThread; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum[2 * e] += static_cast<double>(__uint_as_float(u[e] << 16));
      sum[2 * e + 1] += static_cast<double>(__uint_as_float(u[e] & 0xFFFF0000u));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s_sum[group][8 * unit + e] = sum[e];
  __syncthreads();
  float mean[2], amax = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int d = 2 * threadIdx.x + e;
    const double t = (s_sum[0][d] + s_sum[1][d]) + (s_sum[2][d] + s_sum[3][d]);
    mean[e] = static_cast<float>(t / static_cast<double>(n));
    amax = fmaxf(amax, fabsf(mean[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kKeyThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float scale = int8_scale(amax);
  char2 code;
  code.x = static_cast<signed char>(int8_code(mean[0], scale));
  code.y = static_cast<signed char>(int8_code(mean[1], scale));
  reinterpret_cast<char2*>(P.keys + static_cast<size_t>(blk) * kD)[threadIdx.x] = code;
  if (threadIdx.x == 0) P.scales[blk] = scale;
}

// ------------------------------------------------------------------ scores

struct PageSelectParams {
  const __nv_bfloat16* q;  // [pairs * h_q, 576]
  const int8_t* keys;
  const float* scales;
  int num_blocks;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seqlens;  // [batch]
  int s_q, h_q, causal;
  int topk;                // pages taken (at most)
  int width;               // pages of a taken table row: min(topk, max_pages)
  float* scores;           // [pairs, max_pages]
  int32_t* taken_table;    // [pairs, width] physical blocks
  int32_t* taken_lens;     // [pairs]
  int32_t* pages;          // [pairs, topk] logical pages, -1 behind them; or null
};

// Tokens that query `pair` sees (0 .. max_pages * 64).
__device__ __forceinline__ int tokens_seen(const PageSelectParams& P, int pair) {
  const int b = pair / P.s_q, i = pair - b * P.s_q;
  int L = P.seqlens[b];
  if (L > P.max_pages * kPage) {
    if (threadIdx.x == 0) ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x73);
    L = P.max_pages * kPage;
  }
  return max(0, P.causal ? L - P.s_q + 1 + i : L);
}

constexpr int kScorePages = 128;   // pages per CTA
constexpr int kScoreHeads = 64;    // head rows per pass
constexpr int kScoreThreads = 256;
constexpr int kScoreStride = kD + 16;  // bytes; an odd number of 16-byte units: no bank conflicts
constexpr int kScoreSmem = (kScorePages + kScoreHeads) * kScoreStride;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// grid (ceil(max_pages / 128), pairs).  A CTA quantises the pair's query rows
// (64 heads at a time), multiplies them with its pages' keys on the integer
// tensor cores (warp tile 32 heads x 32 pages) and keeps each page's maximum.
// The keys are 576 bytes a page, 1/128 of the rows they stand for, so the whole
// step is bound by its latency and the quantisation, not by bytes.
__global__ void __launch_bounds__(kScoreThreads, 2) mla_page_score_kernel(const PageSelectParams P) {
  extern __shared__ __align__(16) uint8_t s_buf[];
  __shared__ float s_qscale[kScoreHeads];
  __shared__ float s_best[2][kScorePages];  // [head half][page]
  ptx::grid_dep_launch();
  const int pair = blockIdx.y;
  const int page0 = blockIdx.x * kScorePages;
  const int seen = tokens_seen(P, pair);
  const int last = (seen + kPage - 1) / kPage - 1;
  // nothing to choose, or no page before the last one here
  if (last < P.topk || page0 >= last) return;
  uint8_t* s_keys = s_buf;
  uint8_t* s_q = s_buf + kScorePages * kScoreStride;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* table = P.block_table + static_cast<size_t>(pair / P.s_q) * P.max_pages;

  // the pages' keys: 36 16-byte units each
  for (int i = tid; i < kScorePages * (kD / 16); i += kScoreThreads) {
    const int p = i / (kD / 16), c = i - p * (kD / 16);
    uint8_t* dst = s_keys + p * kScoreStride + 16 * c;
    if (page0 + p < last) {
      const int blk = clamp_block(table[page0 + p], P.num_blocks);
      const int8_t* src = P.keys + static_cast<size_t>(blk) * kD + 16 * c;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src));
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
    }
  }
  asm volatile("cp.async.commit_group;");
  if (tid < kScorePages) s_best[0][tid] = s_best[1][tid] = -INFINITY;

  const int hh = warp >> 2;  // head half: rows 32 hh .. + 31
  const int pg = warp & 3;   // pages 32 pg .. + 31
  for (int h0 = 0; h0 < P.h_q; h0 += kScoreHeads) {
    __syncthreads();  // the previous pass is done with s_q
    for (int r = warp; r < kScoreHeads; r += kScoreThreads / 32) {
      uint8_t* dst = s_q + r * kScoreStride;
      if (h0 + r >= P.h_q) {
        for (int u = lane; u < kD / 8; u += 32)
          *reinterpret_cast<uint2*>(dst + 8 * u) = make_uint2(0, 0);
        continue;
      }
      const uint4* src = reinterpret_cast<const uint4*>(
          P.q + (static_cast<size_t>(pair) * P.h_q + h0 + r) * kD);
      float x[3][8];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int u = lane + 32 * j;
        const uint4 w = u < kD / 8 ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[j][2 * e] = __uint_as_float(v[e] << 16);
          x[j][2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(x[j][2 * e]), fabsf(x[j][2 * e + 1])));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = int8_scale(amax);
      if (lane == 0) s_qscale[r] = scale;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int u = lane + 32 * j;
        int c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = int8_code(x[j][e], scale);
        if (u < kD / 8)
          *reinterpret_cast<uint2*>(dst + 8 * u) =
              make_uint2(pack_int8x4(c[0], c[1], c[2], c[3]), pack_int8x4(c[4], c[5], c[6], c[7]));
      }
    }
    if (h0 == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    if (h0 + 32 * hh < P.h_q) {
      int acc[2][4][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][n][e] = 0;
      // ldmatrix rows: A tiles (16 heads x 32 bytes) and B tiles (16 pages x 32 bytes)
      const uint32_t a0 = ptx::smem_u32(s_q) + (32 * hh + (lane & 15)) * kScoreStride +
                          16 * (lane >> 4);
      const uint32_t b0 = ptx::smem_u32(s_keys) +
                          (32 * pg + (lane & 7) + 8 * (lane >> 4)) * kScoreStride +
                          16 * ((lane >> 3) & 1);
#pragma unroll
      for (int k = 0; k < kD / 32; ++k) {
        uint32_t a[2][4], bq[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) ldmatrix_x4(a[m], a0 + 16 * m * kScoreStride + 32 * k);
#pragma unroll
        for (int n = 0; n < 2; ++n) ldmatrix_x4(bq[n], b0 + 16 * n * kScoreStride + 32 * k);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < 4; ++n)
            mma_s8(acc[m][n], a[m], bq[n >> 1][2 * (n & 1)], bq[n >> 1][2 * (n & 1) + 1]);
      }
      // max over the warp's 32 heads of s_h * dot, per page
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = -INFINITY;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const int r = 32 * hh + 16 * m + 8 * hi + (lane >> 2);
              if (h0 + r < P.h_q)
                v = fmaxf(v, static_cast<float>(acc[m][n][2 * hi + e]) * s_qscale[r]);
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
          if (lane < 4) {
            float& best = s_best[hh][32 * pg + 8 * n + 2 * lane + e];
            best = fmaxf(best, v);
          }
        }
    }
  }
  __syncthreads();
  if (tid < kScorePages && page0 + tid < last) {
    const int blk = clamp_block(table[page0 + tid], P.num_blocks);
    // + 0: a product that underflows to -0 ties with 0
    P.scores[static_cast<size_t>(pair) * P.max_pages + page0 + tid] =
        fmaxf(s_best[0][tid], s_best[1][tid]) * P.scales[blk] + 0.f;
  }
}

// ------------------------------------------------------------------ selection

constexpr int kSelectThreads = 256;

// fp32 -> unsigned key of the same order.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// grid (pairs): one CTA finds the (topk - 1)-th highest score by a radix
// selection (four passes of eight bits), then takes the pages above it and the
// first of those equal to it, in page order.
__global__ void __launch_bounds__(kSelectThreads) mla_page_select_kernel(const PageSelectParams P) {
  __shared__ int s_hist[256];
  __shared__ int s_warp[kSelectThreads / 32][2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  ptx::grid_dep_wait();  // the scores are complete
  ptx::grid_dep_launch();
  const int pair = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seen = tokens_seen(P, pair);
  const int last = (seen + kPage - 1) / kPage - 1;  // -1: the query sees nothing
  const int32_t* table = P.block_table + static_cast<size_t>(pair / P.s_q) * P.max_pages;
  int32_t* out_table = P.taken_table + static_cast<size_t>(pair) * P.width;
  int32_t* out_pages = P.pages ? P.pages + static_cast<size_t>(pair) * P.topk : nullptr;
  auto take = [&](int at, int page) {
    out_table[at] = clamp_block(table[page], P.num_blocks);
    if (out_pages) out_pages[at] = page;
  };
  int count = last + 1;  // pages taken
  if (last < P.topk) {
    for (int p = tid; p <= last; p += kSelectThreads) take(p, p);
  } else {
    count = P.topk;
    const float* scores = P.scores + static_cast<size_t>(pair) * P.max_pages;
    uint32_t prefix = 0;
    int need = P.topk - 1;  // still to take among the pages that share `prefix`
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      s_hist[tid] = 0;
      __syncthreads();
      for (int p = tid; p < last; p += kSelectThreads) {
        const uint32_t key = order_key(scores[p]);
        if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&s_hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      // suffix sums: thread d holds the count of digits above 255 - d
      const int d = 255 - tid;
      const int mine = s_hist[d];
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_warp[warp][0] = x;
      __syncthreads();
      for (int w = 0; w < warp; ++w) x += s_warp[w][0];
      const int above = x - mine;
      if (above < need && need <= x) {  // exactly one digit
        s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
        s_need = need - above;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
    // prefix is the border's key (no border when only the last page is taken);
    // `need` pages of that key are taken
    int gt0 = 0, eq0 = 0;
    for (int base = 0; base < last; base += kSelectThreads) {
      const int p = base + tid;
      bool gt = false, eq = false;
      if (p < last && P.topk > 1) {
        const uint32_t key = order_key(scores[p]);
        gt = key > prefix;
        eq = key == prefix;
      }
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      __syncthreads();  // s_warp of the previous chunk was read
      if (lane == 0) {
        s_warp[warp][0] = __popc(bg);
        s_warp[warp][1] = __popc(be);
      }
      __syncthreads();
      const uint32_t below = (1u << lane) - 1u;
      int g = gt0 + __popc(bg & below), q = eq0 + __popc(be & below);
      for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w < warp) {
          g += s_warp[w][0];
          q += s_warp[w][1];
        }
        gt0 += s_warp[w][0];
        eq0 += s_warp[w][1];
      }
      if (gt || (eq && q < need)) take(g + min(q, need), p);
    }
    if (tid == 0) take(P.topk - 1, last);
  }
  if (out_pages)
    for (int p = count + tid; p < P.topk; p += kSelectThreads) out_pages[p] = -1;
  if (tid == 0) P.taken_lens[pair] = last < 0 ? 0 : (count - 1) * kPage + seen - last * kPage;
}

}  // namespace mla

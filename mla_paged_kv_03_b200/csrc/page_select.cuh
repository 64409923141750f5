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
#include "sparse_gather.cuh"

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

// ------------------------------------------------------------------ page keys

struct PageKeysParams {
  const __nv_bfloat16* kcache;  // [num_blocks, 64, 576]
  int num_blocks;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seqlens;
  int batch;
  int tail;          // the last `tail` pages of each sequence
  int8_t* keys;      // [num_blocks, 576]
  float* scales;     // [num_blocks]
};

constexpr int kKeyUnits = kD / 8;      // 16-byte units of a row
constexpr int kKeyRowGroups = 4;       // threads that share a unit, each every 4th row
constexpr int kKeyGroup = kKeyUnits * kKeyRowGroups;  // 288 threads sum a page: two dims each
constexpr int kKeyGroups = 2;                         // groups, with every second page
constexpr int kKeyThreads = kKeyGroups * kKeyGroup + 32;  // and a warp that fetches
constexpr int kKeyHalf = kPage / 2;    // rows of a stage
constexpr int kKeyStageBytes = kKeyHalf * kD * 2;  // 36864
// Partial sums of a group: [row group][pair of a unit's dims][unit] two doubles,
// a pair's units padded so that neither the stores (a thread per unit) nor the
// loads (a thread per pair) meet in a bank more than twice.
constexpr int kKeyPairStride = kKeyUnits + 4;
constexpr int kKeySumBytes = kKeyRowGroups * 4 * kKeyPairStride * 16;
constexpr int kKeySmem = kKeyGroups * (2 * kKeyStageBytes + kKeySumBytes);

// Untiled bulk copy of `bytes` (a multiple of 16) to this CTA's shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

// All of the threads of group g of the page key kernel have ok (uniform).
__device__ __forceinline__ bool key_group_and(int g, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(ok ? 1 : 0), "r"(1 + g), "n"(kKeyGroup)
      : "memory");
  return all != 0;
}

// The two bf16 values of a word as the high words of doubles, 2^896 times too
// small: exponent and fraction keep their bits, which are read in the wider
// format's place (exact for every finite value, subnormal ones too).
__device__ __forceinline__ double low_bf16_scaled(uint32_t w) {
  return __hiloint2double((static_cast<int>(w << 16) >> 3) & 0x8FFFFFFF, 0);
}
__device__ __forceinline__ double high_bf16_scaled(uint32_t w) {
  return __hiloint2double((static_cast<int>(w) >> 3) & 0x8FFFE000, 0);
}

// One CTA per SM goes over the (page, sequence) places tail * batch.  Two groups
// of 288 threads take every second page each, so that one group's reduction and
// waits lie behind the other's sums; a warp of its own looks up the pages and
// fetches them.  The rows of a page that the sequence has lie in one piece, which
// comes in by bulk copies of 32 rows.  The sums are formed in fp64, where 64 bf16
// values add exactly unless they lie 39 binades apart: the code does not depend
// on the order, and a mean next to a rounding border is decided by its value.
// Converting bf16 to fp64 at the conversion unit's rate (16 a clock per SM) costs
// more than the page's share of HBM time; placing the bits does not.
// HBM bound; 6144 pages (453 MB) on B200: 135 us with a CTA per page and
// conversions, 117 us with bulk copies, 86 us with bits placed, 76 us with two
// groups; the copies alone take 73 us.
__global__ void __launch_bounds__(kKeyThreads, 1) mla_page_keys_kernel(const PageKeysParams P) {
  extern __shared__ __align__(128) uint8_t s_buf[];
  __shared__ uint64_t s_full[kKeyGroups][2], s_empty[kKeyGroups];  // [group][half of the page]
  __shared__ uint32_t s_max[kKeyGroups][kKeyGroup / 32];
  __shared__ int s_blk[kKeyGroups], s_rows[kKeyGroups];  // the group's page; 0 rows: the end
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    for (int g = 0; g < kKeyGroups; ++g) {
      ptx::mbar_init(&s_full[g][0], 1);
      ptx::mbar_init(&s_full[g][1], 1);
      ptx::mbar_init(&s_empty[g], kKeyGroup / 32);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();

  if (tid >= kKeyGroups * kKeyGroup) {
    if (lane != 0) return;
    const long long items = static_cast<long long>(P.tail) * P.batch;
    long long item = blockIdx.x;
    for (int k = 0;; ++k) {  // page k of this CTA goes to group k % 2
      int rows = 0, blk = 0;
      for (; rows == 0 && item < items; item += gridDim.x) {
        const int b = static_cast<int>(item / P.tail);
        int L = P.seqlens[b];
        if (L > P.max_pages * kPage) {
          ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x72);
          L = P.max_pages * kPage;
        }
        const int page = (L + kPage - 1) / kPage - P.tail +
                         static_cast<int>(item - static_cast<long long>(b) * P.tail);
        if (L <= 0 || page < 0) continue;
        const int entry = P.block_table[static_cast<size_t>(b) * P.max_pages + page];
        if (entry < 0 || entry >= P.num_blocks) {  // no block: no key to write
          ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x7a);
          continue;
        }
        blk = entry;
        rows = min(kPage, L - page * kPage);
      }
      const int g = k % kKeyGroups, round = k / kKeyGroups;
      // the group is done with its last page (and so are the copies of it)
      if (!ptx::mbar_wait(&s_empty[g], (round & 1) ^ 1, 0x74)) {
        // give up, once the other group's copies have landed (bounded, too)
        if (k > 0) {
          const int o = (k - 1) % kKeyGroups, ro = (k - 1) / kKeyGroups;
          ptx::mbar_wait(&s_full[o][0], ro & 1, 0x75);
          ptx::mbar_wait(&s_full[o][1], ro & 1, 0x75);
        }
        return;
      }
      s_blk[g] = blk;
      s_rows[g] = rows;
      const __nv_bfloat16* src = P.kcache + static_cast<size_t>(blk) * kPage * kD;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = min(kKeyHalf, rows - h * kKeyHalf);
        if (n > 0) {
          ptx::mbar_arrive_expect_tx(&s_full[g][h], n * kD * 2);
          bulk_load(s_buf + (2 * g + h) * kKeyStageBytes, src + h * kKeyHalf * kD, n * kD * 2,
                    &s_full[g][h]);
        } else {
          ptx::mbar_arrive(&s_full[g][h]);
        }
      }
      // after the last page each group gets an end mark
      if (rows == 0 && k >= kKeyGroups - 1 && s_rows[(k + 1) % kKeyGroups] == 0) return;
    }
  }

  const int g = tid / kKeyGroup, t = tid - g * kKeyGroup, warp = t >> 5;
  const int unit = t % kKeyUnits, row_group = t / kKeyUnits;
  double2* s_sum = reinterpret_cast<double2*>(s_buf + 2 * kKeyGroups * kKeyStageBytes +
                                              g * kKeySumBytes);
  for (int round = 0;; ++round) {
    if (!key_group_and(g, ptx::mbar_wait(&s_full[g][0], round & 1, 0x76))) break;
    const int n = s_rows[g], blk = s_blk[g];
    if (n == 0) return;
    bool ok = true;
    double sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1) ok = ptx::mbar_wait(&s_full[g][1], round & 1, 0x77);
      const uint4* src = reinterpret_cast<const uint4*>(s_buf + (2 * g + h) * kKeyStageBytes) + unit;
#pragma unroll
      for (int i = 0; i < kKeyHalf / kKeyRowGroups; ++i) {
        const int row = row_group + kKeyRowGroups * i;
        if (h * kKeyHalf + row < n) {
          const uint4 w = src[row * kKeyUnits];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum[2 * e] += low_bf16_scaled(u[e]);
            sum[2 * e + 1] += high_bf16_scaled(u[e]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&s_empty[g]);  // the page was read: fetch the next
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s_sum[(row_group * 4 + e) * kKeyPairStride + unit] = make_double2(sum[2 * e], sum[2 * e + 1]);
    if (!key_group_and(g, ok)) break;
    // dims 2 t and 2 t + 1: pair t % 4 of unit t / 4
    double2 total = make_double2(0.0, 0.0);
#pragma unroll
    for (int r = 0; r < kKeyRowGroups; ++r) {
      const double2 v = s_sum[(r * 4 + (t & 3)) * kKeyPairStride + (t >> 2)];
      total.x += v.x;
      total.y += v.y;
    }
    const double inv = n == kPage ? 0x1p+896 / kPage : 0x1p+896;
    total.x *= inv;
    total.y *= inv;
    if (n != kPage) {
      total.x /= n;
      total.y /= n;
    }
    const float m0 = static_cast<float>(total.x), m1 = static_cast<float>(total.y);
    // magnitudes of floats order like their bits
    const uint32_t top = __reduce_max_sync(
        0xffffffffu, max(__float_as_uint(fabsf(m0)), __float_as_uint(fabsf(m1))));
    if (lane == 0) s_max[g][warp] = top;
    ptx::named_bar_sync(1 + g, kKeyGroup);
    const float scale = int8_scale(__uint_as_float(
        __reduce_max_sync(0xffffffffu, lane < kKeyGroup / 32 ? s_max[g][lane] : 0u)));
    char2 code;
    code.x = static_cast<signed char>(int8_code(m0, scale));
    code.y = static_cast<signed char>(int8_code(m1, scale));
    reinterpret_cast<char2*>(P.keys + static_cast<size_t>(blk) * kD)[t] = code;
    if (t == 0) P.scales[blk] = scale;
  }
  // a copy did not come in time: leave once those of this group have landed (bounded)
  for (int h = 0; h < 2; ++h)
    for (uint32_t parity = 0; parity < 2; ++parity) ptx::mbar_wait(&s_full[g][h], parity, 0x78);
}

// ------------------------------------------------------------------ selection

struct PageSelectParams {
  const __nv_bfloat16* q;  // [pairs * h_q, 576]
  const int8_t* keys;
  const float* scales;
  int num_blocks;
  const int32_t* block_table;
  int max_pages;
  const int32_t* seqlens;  // [batch]
  int pairs, s_q, h_q, causal;
  int topk;                // pages taken (at most)
  int width;               // pages of a taken table row: min(topk, max_pages)
  int tile;                // pages per step of a CTA: 64 or 128
  uint32_t* scores;        // [pairs, max_pages] order keys >= 1 (scores while heads are left)
  int32_t* taken_table;    // [pairs, width] physical blocks
  int32_t* taken_lens;     // [pairs]
  int32_t* pages;          // [pairs, topk] logical pages, -1 behind them; or null
  // the plan of the decode over the taken pages
  int num_parts;
  PlanParams plan;
  int32_t* metadata;
  int32_t* num_splits;
};

// Tokens that query `pair` sees (0 .. max_pages * 64).
__device__ __forceinline__ int tokens_seen(const PageSelectParams& P, int pair) {
  const int b = pair / P.s_q, i = pair - b * P.s_q;
  const int L = max(0, min(P.seqlens[b], P.max_pages * kPage));
  return max(0, P.causal ? L - P.s_q + 1 + i : L);
}

// Tokens of the pages taken for a query that sees `seen` tokens: known before
// the selection, since the last page is always among them.
__device__ __forceinline__ int taken_tokens(const PageSelectParams& P, int seen) {
  const int last = (seen + kPage - 1) / kPage - 1;
  return last < P.topk ? seen : (P.topk - 1) * kPage + seen - last * kPage;
}

constexpr int kSelThreads = 512;
constexpr int kSelTile = 128;    // pages per step of a CTA, at most: M of its products
constexpr int kSelHeads = 128;   // head rows per pass: N of its products, at most
constexpr int kSelPerThread = 8;     // order keys a thread of the selection holds, at most
constexpr int kSelMaxCluster = 8;
constexpr int kSelTmemCols = 128;

// Shared memory of an operand of R rows (pages or heads) of 576 bytes, K-major in
// the 64-byte swizzle: nine chunks of R x 64 bytes, in a row of which the 16-byte
// units change places by two bits of the row.  (Pieces of 64 bytes keep the
// stores to other CTAs few; without swizzle a row lies in pieces of 16.)
constexpr int kSelChunk = 64;
constexpr int kSelUnits = kD / 16;  // 36
__device__ __forceinline__ int sel_offset(int R, int row, int unit) {
  return (unit >> 2) * R * kSelChunk + row * kSelChunk + (((unit ^ (row >> 1)) & 3) << 4);
}
constexpr int kSelKeyBytes = kSelTile * kD;

// Head rows that a pass of `h_q` heads holds (N is a multiple of 16).
__host__ __device__ inline int select_rows(int h_q) {
  return h_q >= kSelHeads ? kSelHeads : (h_q + 15) / 16 * 16;
}
// Dynamic shared memory: the rows' codes and two tiles of keys, or the plan's
// prefix sums of pairs + 1 costs.
__host__ __device__ inline int select_smem(int h_q, int pairs) {
  const int a = select_rows(h_q) * kD + 2 * kSelKeyBytes + 1024;  // the base aligned
  const int b = (pairs + 1) * 4;
  return a > b ? a : b;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}

// fp32 -> unsigned key of the same order.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Eight codes by division, for scales whose reciprocal is not a normal number.
// Hardly ever taken: kept out of line and out of the instruction cache.
__device__ __noinline__ uint2 int8_codes8_by_division(float4 lo, float4 hi, float scale) {
  const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e >> 2] |= (int8_code(x[e], scale) & 0xFF) << (8 * (e & 3));
  return make_uint2(o[0], o[1]);
}

// int8_code of eight finite values, inv = 1/scale.  Adding 1.5 * 2^23 rounds the
// quotient to a whole number, ties to even, whose low byte is the code.
__device__ __forceinline__ uint2 int8_codes8(const float* x, float scale, float inv) {
  constexpr float kMagic = 12582912.f;
  uint32_t m[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    m[e] = __float_as_uint(__fadd_rn(div_by(x[e], scale, inv), kMagic));
  uint2 o;
  o.x = __byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410);
  return o;
}

// Selection by one CTA, thread t holding the keys of pages m t .. m t + m - 1
// (m = ceil(n / threads) <= kKeys).  The border is the highest T with at least
// `need` keys >= T, found two bits a round from the highest bit in which the
// keys differ, or the first T on the way with exactly `need`.  take(i, page,
// entry): the i-th page, in page order, of the keys above the border and the
// first of those equal to it, with the page's block table entry.
template <int kKeys, class Take>
__device__ __forceinline__ void select_block(const uint32_t* keys, const int32_t* table, int n,
                                             int need, Take take) {
  constexpr int kWarps = kSelThreads / 32;
  __shared__ uint32_t s_part[2][2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = (n + kSelThreads - 1) / kSelThreads;
  uint32_t key[kKeys];
  int entry[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {  // unconditional: all loads are in flight at once
    const int p = min(m * tid + k, n - 1);
    key[k] = __ldcg(keys + p);
    entry[k] = __ldg(table + p);
  }
  uint32_t top = 0, low = 0xffffffffu;
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    top = max(top, key[k]);
    low = min(low, key[k]);
    if (k >= m || m * tid + k >= n) key[k] = 0u;  // no page
  }
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    s_part[1][0][warp] = top;
    s_part[1][1][warp] = low;
  }
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, s_part[1][0][lane & (kWarps - 1)]);
  low = __reduce_min_sync(0xffffffffu, s_part[1][1][lane & (kWarps - 1)]);
  // keys >= border: n at the start, where the border holds the common bits
  int bit = top == low ? -1 : (31 - __clz(top ^ low)) | 1;  // the upper of two bits
  uint32_t border = bit < 0 ? top : bit == 31 ? 0u : top & ~((2u << bit) - 1u);
  int count = n;
#pragma unroll 1
  for (int round = 0; bit > 0 && count != need; bit -= 2, round ^= 1) {
    const uint32_t step = 1u << (bit - 1);
    uint32_t c = 0;  // three counts of at most 32 kKeys
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      c += (key[k] >= border + step ? 1u : 0u) + (key[k] >= border + 2 * step ? 1u << 10 : 0u) +
           (key[k] >= border + 3 * step ? 1u << 20 : 0u);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s_part[round][0][warp] = c;
    __syncthreads();  // the other half of s_part is written next
    c = lane < kWarps ? s_part[round][0][lane] : 0u;
    const uint32_t c12 = __reduce_add_sync(0xffffffffu, (c & 1023u) | (c >> 10 & 1023u) << 16);
    const int c3 = __reduce_add_sync(0xffffffffu, c >> 20);
    const int c1 = c12 & 0xFFFFu, c2 = c12 >> 16;
    const int up = c3 >= need ? 3 : c2 >= need ? 2 : c1 >= need ? 1 : 0;
    border += up * step;
    count = up == 3 ? c3 : up == 2 ? c2 : up == 1 ? c1 : count;
  }
  int mine = 0;  // keys above, and equal to, the border
#pragma unroll
  for (int k = 0; k < kKeys; ++k)
    mine += (key[k] > border ? 1 : 0) + (key[k] == border ? 1 << 16 : 0);
  int total;
  const int before = block_exclusive_scan<kSelThreads>(mine, &total);
  const int equal = need - (total & 0xFFFF);  // taken of those equal to the border
  int g = before & 0xFFFF, q = before >> 16;
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const bool gt = key[k] > border, eq = key[k] == border;
    if (gt || (eq && q < equal)) take(g + min(q, equal), m * tid + k, entry[k]);
    g += gt;
    q += eq;
  }
}

// grid (cluster, 1 + pairs).  Row 0 of the grid: one CTA plans the decode over
// the taken pages, whose lengths do not depend on the selection.  Row 1 + pair:
// a cluster of 1..8 CTAs scores the pair's pages and its first CTA selects.
//   - Each CTA quantises its share of the head rows (128 at a time) and stores
//     the codes to every CTA of the cluster through distributed shared memory.
//   - Tiles of 128 pages (64 where the cluster then takes all of them at once) go
//     round the CTAs.  A tile's keys (at most 74 kB) come in by
//     cp.async, the next tile's behind this one's products: 18 integer UMMAs of
//     128 pages x the heads.  A thread then holds a page's products with up to
//     32 heads; their maximum goes to the score array as an order key.
//   - The first CTA selects.
// The keys are 576 bytes a page, 1/128 of the rows they stand for: latency, not
// bytes, bounds this step, hence one launch for plan, scores and selection, and
// the query, the table and the length read side by side at its start.
// B200, 32 queries x 128 heads over 1024 pages: 75 us as three launches (scores by
// a CTA per 128 pages, each quantising all heads by division), 20 us as one
// cluster with mma.sync (its shared-memory reads took as long as its products),
// 13 us with tcgen05: 5 us until the codes are everywhere, 4 us for the tiles,
// 3 us for the selection.
__global__ void __launch_bounds__(kSelThreads, 1) mla_page_select_kernel(const PageSelectParams P) {
  extern __shared__ __align__(16) uint8_t s_buf[];
  __shared__ float s_qscale[kSelHeads];
  __shared__ float s_best[kSelHeads / 32][kSelTile];  // [32 heads][page]
  __shared__ uint64_t s_done;                         // the tile's products
  __shared__ uint32_t s_tmem;
  __shared__ int s_hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, nrank = gridDim.x;
  ptx::grid_dep_launch();  // the decode grid waits for this one's end
  if (blockIdx.y == 0) {
    if (rank == 0)
      plan_block<kSelThreads>([&](int pair) { return taken_tokens(P, tokens_seen(P, pair)); },
                              P.pairs, P.num_parts, P.plan, reinterpret_cast<int32_t*>(s_buf),
                              P.metadata, P.num_splits, nullptr, nullptr, 0);
    return;
  }
  const int pair = blockIdx.y - 1;
  const int32_t* table = P.block_table + static_cast<size_t>(pair / P.s_q) * P.max_pages;
  uint32_t* scores = P.scores + static_cast<size_t>(pair) * P.max_pages;
  // raw values of one head row: lane l holds the 16-byte units l, l + 32, l + 64
  auto load_row = [&](int h, uint4 (&w)[3]) {
    const uint4* src =
        reinterpret_cast<const uint4*>(P.q + (static_cast<size_t>(pair) * P.h_q + h) * kD);
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int u = lane + 32 * j;
      w[j] = u < kD / 8 ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
    }
  };
  const int row0 = rank + nrank * warp, row_step = nrank * (kSelThreads / 32);
  const int tile = P.tile;
  const int key_shift = tile == kSelTile ? 2 : 3;  // 4 or 8 threads load a page's key
  const int page_of_thread = tid >> key_shift;
  uint4 raw[3];
  int entry = 0;  // the table's entry of the first tile's page
  if (P.topk > 1 && P.topk < P.max_pages) {
    if (row0 < min(kSelHeads, P.h_q)) load_row(row0, raw);
    if (rank * tile + page_of_thread < P.max_pages) entry = table[rank * tile + page_of_thread];
  }
  const int seen = tokens_seen(P, pair);
  const int last = (seen + kPage - 1) / kPage - 1;  // -1: the query sees nothing
  const bool choose = last >= P.topk && P.topk > 1;  // alike in the whole cluster

  if (choose) {
    cluster_arrive();  // this CTA runs: the others may store to its shared memory
    const int q_rows = select_rows(P.h_q);
    // (swizzle atoms are 512 bytes; the offset is the same in every CTA)
    uint8_t* s_keys = s_buf + ((1024 - (ptx::smem_u32(s_buf) & 1023)) & 1023);
    uint8_t* s_q = s_keys + 2 * kSelKeyBytes;
    constexpr int kMmaWarp = kSelThreads / 32 - 1;  // the one with the fewest head rows
    if (warp == kMmaWarp) {
      if (lane == 0) {
        ptx::mbar_init(&s_done, 1);
        ptx::fence_mbar_init();
      }
      __syncwarp();
      ptx::tmem_alloc(&s_tmem, kSelTmemCols);
      ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();  // seen by all threads behind the cluster barrier below
    int done = 0;            // tiles multiplied
    const int tiles = (last + tile - 1) / tile;
    // a tile's keys, 36 units of 16 bytes each; blk: the table's entry
    auto load_tile = [&](int t, int buf, int blk) {
      if (t < tiles && t * tile + page_of_thread < last) {
        blk = clamp_block(blk, P.num_blocks);
        const int8_t* src = P.keys + static_cast<size_t>(blk) * kD;
        const uint32_t dst = ptx::smem_u32(s_keys) + buf * kSelKeyBytes;
        for (int u = tid & ((1 << key_shift) - 1); u < kSelUnits; u += 1 << key_shift)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           dst + sel_offset(kSelTile, page_of_thread, u)),
                       "l"(src + 16 * u)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto entry_of = [&](int t) {
      const int p = t * tile + page_of_thread;
      return t < tiles && p < last ? table[p] : 0;
    };
    for (int h0 = 0; h0 < P.h_q; h0 += kSelHeads) {
      if (h0 > 0) {
        entry = entry_of(rank);
        if (h0 + row0 < P.h_q && row0 < kSelHeads) load_row(h0 + row0, raw);
        cluster_arrive();  // the previous pass is done with the codes
      }
      // the key loads of half of the warps go ahead of their head rows, those of
      // the others behind their first: the rows' shuffles and stores wait in line
      // behind loads
      const bool keys_first = warp >= kSelThreads / 64;
      if (keys_first) load_tile(rank, 0, entry);
      bool stored = false;
      const int nh = min(kSelHeads, P.h_q - h0);
      for (int r = row0; r < nh; r += row_step) {
        const uint4 w[3] = {raw[0], raw[1], raw[2]};
        if (r + row_step < nh) load_row(h0 + r + row_step, raw);
        float x[3][8];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
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
        uint2 code[3];
        if (scale > 0x1p-100f && scale < 0x1p+100f) {
          const float inv = __frcp_rn(scale);
#pragma unroll
          for (int j = 0; j < 3; ++j) code[j] = int8_codes8(x[j], scale, inv);
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            code[j] = int8_codes8_by_division(make_float4(x[j][0], x[j][1], x[j][2], x[j][3]),
                                              make_float4(x[j][4], x[j][5], x[j][6], x[j][7]),
                                              scale);
        }
        if (!stored) {
          __syncwarp();
          cluster_wait();
          stored = true;
        }
        const uint32_t dst = ptx::smem_u32(s_q);
        for (int c = 0; c < nrank; ++c) {
          const uint32_t to = ptx::mapa_shared(dst, c);
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (const int v = lane + 32 * j; v < kD / 8)  // half a unit
              st_cluster_v2(to + sel_offset(q_rows, r, v >> 1) + 8 * (v & 1), code[j].x, code[j].y);
          if (lane == 0) st_cluster(ptx::mapa_shared(ptx::smem_u32(&s_qscale[r]), c), scale);
        }
        if (!keys_first && r == row0) load_tile(rank, 0, entry);
      }
      if (!stored) cluster_wait();
      if (!keys_first && row0 >= nh) load_tile(rank, 0, entry);
      entry = entry_of(rank + nrank);
      cluster_arrive();  // this warp's codes are stored
      cluster_wait();

      ptx::tc_fence_after();
      const uint32_t tmem = s_tmem;
      const int n16 = (nh + 15) / 16 * 16;  // rows past nh: whatever lies there, not looked at
      const bool final_pass = h0 + kSelHeads >= P.h_q;
      // the table's entry of the page whose score this thread finishes next
      int scale_entry = 0;
      if (tid < tile && rank * tile + tid < last) scale_entry = table[rank * tile + tid];
      for (int t = rank, i = 0; t < tiles; t += nrank, ++i) {
        load_tile(t + nrank, (i + 1) & 1, entry);
        entry = entry_of(t + 2 * nrank);
        const int p = t * tile + tid;
        float key_scale = 0.f, prev = -INFINITY;
        if (tid < tile && p < last) {
          key_scale = P.scales[clamp_block(scale_entry, P.num_blocks)];
          if (h0 > 0) prev = __uint_as_float(scores[p]);
        }
        const int pn = p + nrank * tile;
        if (tid < tile && pn < last) scale_entry = table[pn];
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        ptx::fence_proxy_async_smem();
        __syncthreads();  // the tile's keys are in shared memory
        if (warp == kMmaWarp) {
          ptx::tc_fence_after();
          if (ptx::elect_one_sync()) {
            // eight rows are 512 bytes; two steps of 32 bytes a chunk
            const uint64_t da = ptx::smem_desc(ptx::smem_u32(s_keys) + (i & 1) * kSelKeyBytes, 16,
                                               8 * kSelChunk, ptx::kLayoutSW64);
            const uint64_t db =
                ptx::smem_desc(ptx::smem_u32(s_q), 16, 8 * kSelChunk, ptx::kLayoutSW64);
            const uint32_t idesc = ptx::idesc_s8_s32(kSelTile, n16);
#pragma unroll 1
            for (int k = 0; k < kD / 32; ++k) {
              const int in = 2 * (k & 1), c = k >> 1;  // 32 bytes within chunk c
              ptx::umma_i8_ss(tmem, da + c * (kSelTile * kSelChunk / 16) + in,
                              db + c * (q_rows * kSelChunk / 16) + in, idesc, k ? 1u : 0u);
            }
            ptx::umma_commit(&s_done);
          }
          __syncwarp();
        }
        // (a wait that runs out is on record; the scores are then worthless)
        ptx::mbar_wait(&s_done, done & 1, 0x79);
        ++done;
        ptx::tc_fence_after();
        // the lane's page, heads 32 hg .. + 31: max of s_h * dot
        const int hg = warp >> 2, h_first = 32 * hg;
        if (h_first < nh && 32 * (warp & 3) < tile) {
          const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + h_first;
          float d[32];
          if (h_first + 32 <= n16) {
            ptx::tmem_ld32(at, d);
            ptx::tmem_ld_wait_regs(d);
          } else {
            ptx::tmem_ld16(at, d);
            ptx::tmem_ld_wait_regs16(d);
          }
          float v = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (h_first + c < nh)
              v = fmaxf(v, static_cast<float>(__float_as_int(d[c])) * s_qscale[h_first + c]);
          s_best[hg][32 * (warp & 3) + lane] = v;
        }
        ptx::tc_fence_before();
        __syncthreads();  // s_best is complete, the tile's buffer free
        if (tid < tile && p < last) {
          float v = prev;
#pragma unroll
          for (int g = 0; g < kSelHeads / 32; ++g)
            if (32 * g < nh) v = fmaxf(v, s_best[g][tid]);
          // + 0: a product that underflows to -0 ties with 0 (of one fma it would stay -0)
          scores[p] = final_pass
                          ? max(order_key(__fadd_rn(__fmul_rn(v, key_scale), 0.f)), 1u)
                          : __float_as_uint(v);
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    cluster_arrive();  // this CTA's scores are written
    if (warp == kMmaWarp) {
      ptx::tc_fence_after();
      ptx::tmem_dealloc(s_tmem, kSelTmemCols);
    }
    cluster_wait();
  }
  if (rank != 0) return;

  if (tid == 0 && P.seqlens[pair / P.s_q] > P.max_pages * kPage)
    ptx::set_error(MLA_DEVERR_BAD_INDEX, 0x73);
  int32_t* out_table = P.taken_table + static_cast<size_t>(pair) * P.width;
  int32_t* out_pages = P.pages ? P.pages + static_cast<size_t>(pair) * P.topk : nullptr;
  auto take = [&](int at, int page, int entry_of_page) {
    out_table[at] = clamp_block(entry_of_page, P.num_blocks);
    if (out_pages) out_pages[at] = page;
  };
  const int count = min(last + 1, P.topk);  // pages taken
  if (tid == 0) P.taken_lens[pair] = taken_tokens(P, seen);
  if (out_pages)
    for (int p = count + tid; p < P.topk; p += kSelThreads) out_pages[p] = -1;
  if (last < P.topk) {
    for (int p = tid; p <= last; p += kSelThreads) take(p, p, table[p]);
    return;
  }
  if (tid == 0) take(P.topk - 1, last, table[last]);
  if (!choose) return;
  int need = P.topk - 1;  // pages to take before the last one
  // two keys a thread up to 1024 pages (65536 tokens), eight up to 4096
  if (last <= 2 * kSelThreads)
    return select_block<2>(scores, table, last, need, take);
  if (last <= kSelPerThread * kSelThreads)
    return select_block<kSelPerThread>(scores, table, last, need, take);
  // more pages than the registers hold: radix selection of the border, four
  // passes of eight bits over the score array, then chunks in page order
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    for (int p = tid; p < last; p += kSelThreads) {
      const uint32_t key = __ldcg(scores + p);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&s_hist[(key >> shift) & 255u], 1);
    }
    __syncthreads();
    // thread d < 256: keys of the digits above and of digit 255 - d
    const int d = 255 - tid;
    const int mine = tid < 256 ? s_hist[d] : 0;
    int total;
    const int above = block_exclusive_scan<kSelThreads>(mine, &total);
    if (tid < 256 && above < need && need <= above + mine) {  // exactly one digit
      s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      s_need = need - above;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  int gt0 = 0, eq0 = 0;
  for (int base = 0; base < last; base += kSelThreads) {
    const uint32_t key = base + tid < last ? __ldcg(scores + base + tid) : 0u;
    const int gt = key > prefix, eq = key == prefix;
    int total;
    const int before = block_exclusive_scan<kSelThreads>(gt | (eq << 16), &total);
    const int g = gt0 + (before & 0xFFFF), q = eq0 + (before >> 16);
    if (gt || (eq && q < need)) take(g + min(q, need), base + tid, table[base + tid]);
    gt0 += total & 0xFFFF;
    eq0 += total >> 16;
  }
}

}  // namespace mla

// paged_common.cuh -- what the paged attention kernels share: the requests as the kernels see
// them, the split of a ragged batch over the blocks, and the numerics of codes and page scales.
//
// Split.  The work is a list of units (a tile of KV rows for one item; an item is a request, a KV
// head and, in the tile kernel, a tile of query rows).  Block c of n takes units c*U/n ..
// (c+1)*U/n - 1: equal shares whatever the lengths, each block computing its own bounds from the
// lengths on the device, so that nothing has to be known on the host and a captured launch can
// be replayed with other lengths.  A block that does not hold a whole item writes a partial
// result, "head" (the item began in an earlier block) or "tail" (it began here and does not end
// here); the merge kernel joins them.
//
// Numerics.  Codes are exact in fp16 and so is a query row after its exponent is taken out
// (2^e with the row's largest magnitude in [2^14, 2^15); components below 2^-28 of the largest
// lose bits, by at most 2^-40 of it), so the fp16 products of Q K^T are exact and summed in fp32:
// z2 = log2(e) * scale * q.k = S * kc * 2^e,  kc = scale2 * k_scale.
// A value page's scale goes into the exponent of the probabilities: P = 2^(z2 + lv - M + P_OFF)
// with lv = log2(v_scale) and M >= max(z2 + lv) - (15 - P_OFF) a running reference, rounded to
// fp16, and O = sum P * code in fp32 needs no further scale.  fp16 holds 11 bits down to 2^-14 and
// multiples of 2^-24 below: with P_OFF = 15, M the maximum itself, a row's weight keeps 11 bits
// down to 2^-29 of the largest and is zero below 2^-40 (a row that outweighs all others may have
// values of zero, so that the others make the output).  The row kernel pays nothing for that (245
// against 244 us for the grouped decode); where M may lag by 11 the tile kernel rescales O less
// often, and a reference that lags by up to 3 (2^-26, 2^-37) costs it 0.4 to 2 %.  Measured and
// left: P as two bf16 parts, which keeps 16 bits at any weight (prompts 579 -> 739 us, chunk of
// 2048 on 65536 rows 1150 -> 1385); in the row kernel the rows below 2^-14 times 2^28 in MMAs of
// their own (grouped decode 245 -> 266, drafts 79 -> 88).
// The softmax sum is l = sum 2^(z2 - m) with m = M - P_OFF - lvref, lvref the largest lv met so far:
// formed from the unrounded P of each group of 16 rows (never more than one page) times
// 2^(lvref - lv), and moved when M or lvref grow.  Since M <= max z2 + lvref its largest term is
// not far below 1.  lvref belongs to a query row: a page that the row does not see does not move
// it.  lv is not taken below lvref - 60 (a page of zeros has the scale 2^-126), and where lvref
// grows so far that l would pass 2^60, M is raised with it: the values of a page whose scale is
// below 2^-60 of the largest that the row sees count with 2^-60 of it or less, its rows' share of
// the sum stays right.
#pragma once

#include <cuda_fp16.h>

#include "hcl_common.cuh"
#include "hcl_internal.h"

namespace hcl {
namespace paged {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// P's largest magnitude is 2^P_OFF .. 2^15; M may lag its maximum by 15 - P_OFF.
constexpr float P_OFF_ROWS = 15.f, P_OFF_TILE = 12.f;
constexpr float LV_SPAN = 60.f;
constexpr float SCALE_MIN = 1.17549435e-38f;  // 2^-126
constexpr int ROWS_SMALL = 16;     // query rows (queries x heads of a KV head) of the row kernel
constexpr int ROWS_ITEM = 256;     // query rows of an item of the tile kernel
// A partial result: (m, M, l, -) of each row, then O of each row.
__host__ __device__ constexpr size_t part_floats(int rows, int d) { return rows * 4 + rows * (size_t)d; }

// n / d for 0 <= n < 2^31 by a multiplication: q = (n * mul >> 32 + n) >> shift.
struct FastDiv {
  uint32_t mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    shift = 0;
    while ((1u << shift) < d) shift++;
    mul = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return int((__umulhi(uint32_t(n), mul) + uint32_t(n)) >> shift);
  }
};

struct Params {
  PagedAttnArgs a;
  FastDiv by_G, by_m;
  int sh;            // log2(page)
  int G;             // query heads per KV head
  float scale2;      // scale * log2(e)
  int n_blocks;      // blocks that share the units
  float* part;       // partial results
  struct Meta* meta; // one per block
  long long limit;
};

// One request, bounds applied.
struct Req {
  int nq, c0;        // queries (0: nothing to do), row of the first
  int len;           // rows held
  int qs;            // position of the first query
};

// Row range [lo, hi) that query i of a request sees.
__device__ __forceinline__ int vis_hi(const Params& p, const Req& r, int i) {
  const long long n = (long long)r.qs + i + 1;  // positions up to the query's
  if (n <= 0) return 0;
  return min(r.len, p.by_m.div((int)min(n, 0x7FFFFFFFll)));
}
__device__ __forceinline__ int vis_lo(const Params& p, const Req& r, int i) {
  if (p.a.W == 0) return 0;
  const long long lo = (long long)r.qs + i - p.a.W + 1;
  return (int)max(0ll, min(lo, (long long)r.len));
}

__device__ __forceinline__ Req load_req(const Params& p, int b, bool say) {
  Req r;
  // (plain loads: a read-only one could be moved to before the wait for the kernel that wrote them)
  int c0 = p.a.cu_q[b], c1 = p.a.cu_q[b + 1], len = p.a.kv_len[b];
  r.qs = p.a.q_start[b];
  const long long room = (long long)p.a.max_pages << p.sh;
  int fault = 0;
  if (c0 < 0 || c1 < c0 || c1 > p.a.T || c1 - c0 > p.a.max_q) {
    fault = 1;
    c1 = c0;
  }
  if (len > room) {
    fault = 1;
    len = (int)room;
  }
  r.c0 = c0;
  r.nq = c1 - c0;
  r.len = max(len, 0);
  if (say && fault) report(p.a.status, HCL_ERR_DEVICE_FAULT);
  return r;
}

// This block's share of the units of n entries (requests, or tiles of requests): units(e) of
// entry e, each asked for by one thread, e ascending.  No more blocks take part than there are
// units.  Every thread of the block calls it (NT threads, a multiple of 32); s: scratch of
// NT / 32 + 4 words.
struct Share {
  long long u0, u1;  // units [u0, u1)
  long long tot;     // all units
  int nb;            // blocks that have any
  int e;             // the entry of u0
  long long rem;     // u0's place among that entry's units
};
// Sum of the threads' values before this thread, and of all.
template <int NT>
__device__ __forceinline__ long long block_prefix(long long mine, long long* s, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  long long off = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; w++) {
    const long long x = s[w];
    if (w < warp) off += x;
    tot += x;
  }
  *total = tot;
  return off + inc - mine;
}
template <int NT, typename F>
__device__ __forceinline__ Share find_share(int n, int block, int n_blocks, long long* s, F units) {
  const int tid = threadIdx.x, per = (n + NT - 1) / NT, e0 = min(n, tid * per), e1 = min(n, e0 + per);
  long long mine = 0;
  for (int e = e0; e < e1; e++) mine += units(e);
  Share r;
  long long at = block_prefix<NT>(mine, s, &r.tot);
  r.nb = (int)min((long long)n_blocks, r.tot);
  r.u0 = r.u1 = 0;
  if (block < r.nb) {
    r.u0 = r.tot * block / r.nb;
    r.u1 = r.tot * (block + 1) / r.nb;
    if (at <= r.u0 && r.u0 < at + mine) {
      for (int e = e0; e < e1; e++) {
        const long long u = units(e);
        if (r.u0 < at + u) {
          s[NT / 32] = e;
          s[NT / 32 + 1] = r.u0 - at;
          break;
        }
        at += u;
      }
    }
  }
  __syncthreads();
  r.e = (int)s[NT / 32];
  r.rem = s[NT / 32 + 1];
  return r;
}

// What the merge needs of a block: whether a request that an earlier block began ends in it
// (then that item's first unit, all units, request, KV head and first query row).
struct Meta {
  long long first, tot;
  int ends, b, g, row0;
  int nb, pad[3];
};
static_assert(sizeof(Meta) == 48, "Meta");

// log2 of a page scale (exact for powers of two), the scale not below 2^-126.
__device__ __forceinline__ float log2_scale(float s) {
  s = fmaxf(s, SCALE_MIN);
  const uint32_t u = __float_as_uint(s);
  return (u & 0x7FFFFFu) == 0 ? float(int(u >> 23) - 127) : log2f(s);
}

// The power of two that brings a row's largest magnitude into [2^14, 2^15): returns the factor
// 2^-e and sets back = 2^e.  Zero and non-finite rows keep their values.
__device__ __forceinline__ float row_factor(float amax, float* back) {
  const int ex = int(__float_as_uint(amax) >> 23);  // biased exponent
  if (!(amax > 0.f) || ex == 255) {
    *back = 1.f;
    return 1.f;
  }
  const int e = min(max(ex - 127 - 14, -126), 113);  // 2^e
  *back = __uint_as_float(uint32_t(e + 127) << 23);
  return __uint_as_float(uint32_t(127 - e) << 23);
}

// lvref grows by d: a row's sum moves to the new reference, and its M too where the sum would
// pass 2^60.
__device__ __forceinline__ void grow_lvref(float d, float& l, float& M) {
  if (!(l > 0.f) || M == -INFINITY) return;
  const float lg = float(int(__float_as_uint(l) >> 23) - 126);  // l < 2^lg
  const float add = fmaxf(0.f, lg + d - 60.f);
  l *= exp2f(d - add);
  M += add;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes -> fp16 (exact); NaN codes become NaN.
__device__ __forceinline__ uint32_t half2_of_codes(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// 0xFF in every byte of x that is a NaN code (0x7F with either sign).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// The final row from O (value units), l and m (log2 units): a factor for O, a second one for the
// product (both at once may be below fp32's numbers: 2^lvref over a sum of 2^P_OFF each) and the
// log-sum-exp.
// M: O's reference; the sink's logit in log2 units, or -inf.
template <bool ROWS>
__device__ __forceinline__ float finish_row(float m, float M, float l, float sink2, float* second, float* lse) {
  *second = 0.f;
  if (!(l > 0.f) && !(l != l)) {  // no row
    *lse = sink2 == -INFINITY ? -INFINITY : sink2 * LN2;
    return 0.f;
  }
  const float mm = fmaxf(m, sink2);
  const float lt = l * exp2f(m - mm) + (sink2 == -INFINITY ? 0.f : exp2f(sink2 - mm));
  *lse = (mm + log2f(lt)) * LN2;
  *second = exp2f(M - (ROWS ? P_OFF_ROWS : P_OFF_TILE) - mm);
  return 1.f / lt;
}

// Kernels for requests of up to ROWS_SMALL query rows (`rows`: the most that one of them can
// have), and of more; how many blocks each runs with, and the merge of the requests that it split.
hcl_status_t launch_rows(const Params& p, int rows, cudaStream_t st);
hcl_status_t launch_tiles(const Params& p, cudaStream_t st);
int rows_blocks(int d, bool shared);
constexpr int ROWS_BLOCKS_MOST = 3;  // of launch_rows, per SM
int tile_blocks();
hcl_status_t launch_merge(const Params& p, int rows, cudaStream_t st);
// Workspace of a kernel with n blocks and items of `rows` rows: the blocks' Meta, then two parts
// each.
constexpr size_t meta_bytes(int n) { return (size_t(n) * 48 + 127) / 128 * 128; }
constexpr size_t split_workspace(int n, int rows, int d) {
  return meta_bytes(n) + 2 * size_t(n) * part_floats(rows, d) * 4;
}
// Tensor map of a code plane as rows of d bytes, boxes of `rows` rows.
hcl_status_t code_map(CUtensorMap* m, const void* codes, const hcl_paged_kv_t& kv, int rows, bool swizzle);

}  // namespace paged
}  // namespace hcl

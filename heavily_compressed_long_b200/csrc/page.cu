// page.cu -- the paged 8-bit cache's page plan (block tables and slot maps from request
// lengths) and the write that quantises new rows into pages.
#include <cuda_fp16.h>

#include <algorithm>

#include "hcl_common.cuh"
#include "hcl_internal.h"

namespace hcl {
namespace {

// ---------------------------------------------------------------------------------------
// Page plan.  Three prefix sums over the requests (new rows, pages released, pages taken) and
// three expansions (released ids onto the free stack, free ids into the table, a slot per row).
//
// One block, or a cluster of 8, does all of it in one launch: every block computes the whole
// scan for itself in shared memory (a few loads per thread), then the expansions are spread over
// all threads, each finding its request by binary search.  The cluster barrier after the
// releases orders them before the takes (a released page may be taken again in the same step),
// and separates every read of the old lengths and table from the writes, so that the state is
// updated in place and a captured launch can be replayed.  Latency bound.

constexpr int PP_THREADS = 1024;
constexpr int PP_STATIC = 1024;  // its static shared memory takes less than this
constexpr int PP_SAT = (1 << 30) - 1;  // row counts saturate here (T <= 2^29)

struct PlanSum {
  int rows, back, need;
};
__device__ __forceinline__ PlanSum plan_add(PlanSum a, PlanSum b) {
  return {min(a.rows + b.rows, PP_SAT), a.back + b.back, a.need + b.need};
}

// largest i in [0, n) with off[i] <= x (off ascending, off[0] == 0)
__device__ __forceinline__ int find_request(const int* off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PP_THREADS, 1) page_plan_kernel(PagePlanArgs p, int sh) {
  extern __shared__ int pp_sm[];
  int* s_keep = pp_sm;               // [B]
  int* s_rows = s_keep + p.B;        // [B + 1] exclusive sums of the new rows
  int* s_back = s_rows + p.B + 1;    // [B + 1] of the released pages
  int* s_need = s_back + p.B + 1;    // [B + 1] of the taken pages
  __shared__ PlanSum s_warp[32];
  __shared__ int s_used;
  static_assert(sizeof(s_warp) + sizeof(s_used) <= PP_STATIC / 2, "PP_STATIC");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthr = blockDim.x;
  const int gid = blockIdx.x * nthr + tid, gsize = gridDim.x * nthr;
  const int pmask = p.page - 1;
  const bool lead = blockIdx.x == 0;
  pdl_enter();

  // the requests' counts; thread t takes requests t * per .. t * per + per - 1
  const int per = (p.B + nthr - 1) / nthr;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const long long room = (long long)p.max_pages * p.page;
  int fault = 0;
  PlanSum mine = {0, 0, 0};
  for (int b = b0; b < b1; b++) {
    int seq = p.seq_len[b], keep = p.keep[b], nw = p.new_len[b];
    if (seq < 0 || seq > room) { seq = seq < 0 ? 0 : (int)room; fault = HCL_ERR_DEVICE_FAULT; }
    if (keep < 0 || keep > seq) { keep = keep < 0 ? 0 : seq; fault = HCL_ERR_DEVICE_FAULT; }
    if (nw < 0) { nw = 0; fault = HCL_ERR_DEVICE_FAULT; }
    const int kept = (keep + pmask) >> sh, old = (int)(((long long)seq + pmask) >> sh);
    const int need = (long long)keep + nw <= room ? (int)(((long long)keep + nw + pmask) >> sh) - kept : 0;
    s_keep[b] = keep;
    // this thread's exclusive sums; its offset is added below
    s_rows[b] = mine.rows; s_back[b] = mine.back; s_need[b] = mine.need;
    mine = plan_add(mine, {min(nw, PP_SAT), old - kept, need});
  }
  // block scan of the threads' totals
  PlanSum inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    PlanSum u = {__shfl_up_sync(~0u, inc.rows, o), __shfl_up_sync(~0u, inc.back, o),
                 __shfl_up_sync(~0u, inc.need, o)};
    if (lane >= o) inc = plan_add(u, inc);
  }
  if (lane == 31) s_warp[warp] = inc;
  if (tid == 0) s_used = 0;
  __syncthreads();
  PlanSum off = {0, 0, 0}, tot = {0, 0, 0};
  for (int w = 0; w < (nthr >> 5); w++) {
    if (w == warp) off = tot;
    tot = plan_add(tot, s_warp[w]);
  }
  {
    PlanSum ex = {__shfl_up_sync(~0u, inc.rows, 1), __shfl_up_sync(~0u, inc.back, 1),
                  __shfl_up_sync(~0u, inc.need, 1)};
    if (lane == 0) ex = {0, 0, 0};
    off = plan_add(off, ex);
  }
  for (int b = b0; b < b1; b++) {
    s_rows[b] = min(s_rows[b] + off.rows, PP_SAT);
    s_back[b] += off.back;
    s_need[b] += off.need;
  }
  if (tid == 0) { s_rows[p.B] = tot.rows; s_back[p.B] = tot.back; s_need[p.B] = tot.need; }
  int nfree = *p.n_free;
  if (nfree < 0 || nfree > p.n_pages) { nfree = nfree < 0 ? 0 : p.n_pages; fault = HCL_ERR_DEVICE_FAULT; }
  const int top = (int)min((long long)nfree + tot.back, (long long)p.n_pages);  // free pages after the releases
  __syncthreads();

  // releases: the r-th released page goes to place top - 1 - r of the stack
  // (r is unsigned: the counts reach 2^31 - 1 where lengths that nothing holds are given back)
  for (uint32_t r = gid; r < (uint32_t)tot.back; r += gsize) {
    const int b = find_request(s_back, p.B, r);
    const int j = ((s_keep[b] + pmask) >> sh) + (r - s_back[b]);
    const int id = p.table[(size_t)b * p.max_pages + j];
    if (r < (uint32_t)top) p.free_list[top - 1 - r] = id;
    else fault = HCL_ERR_DEVICE_FAULT;
  }
  __syncwarp();
  if (gridDim.x > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
  } else {
    __syncthreads();
  }

  // A request gets its rows when they fit the table, end within T, and the free pages reach for
  // it and all before it.  (Where the row sums are saturated a request that needs pages shows no
  // rows; it ends beyond T.)
  auto admitted = [&](int b) {
    const int nw = s_rows[b + 1] - s_rows[b], need = s_need[b + 1] - s_need[b];
    if (nw == 0 && need == 0) return true;
    return (long long)s_keep[b] + nw <= room && s_rows[b + 1] <= p.T &&
           (need == 0 || s_need[b + 1] <= top);
  };

  // takes: the r-th taken page is place top - 1 - r of the stack
  for (uint32_t r = gid; r < (uint32_t)tot.need; r += gsize) {
    const int b = find_request(s_need, p.B, r);
    if (!admitted(b)) continue;
    const int j = ((s_keep[b] + pmask) >> sh) + (r - s_need[b]);
    p.table[(size_t)b * p.max_pages + j] = p.free_list[top - 1 - r];
  }
  // released entries that are not taken again
  for (uint32_t r = gid; r < (uint32_t)tot.back; r += gsize) {
    const int b = find_request(s_back, p.B, r);
    const int kept = (s_keep[b] + pmask) >> sh;
    const int got = admitted(b) ? s_need[b + 1] - s_need[b] : 0;
    if ((int)(r - s_back[b]) >= got) p.table[(size_t)b * p.max_pages + kept + (r - s_back[b])] = -1;
  }
  // a slot for every new row
  const int rows = min(s_rows[p.B], p.T);
  for (int t = gid; t < p.T; t += gsize) {
    int ps = -1, sl = -1;
    if (t < rows) {
      const int b = find_request(s_rows, p.B, t);
      ps = s_keep[b] + (t - s_rows[b]);
      if (admitted(b)) {
        const int j = ps >> sh, kept = (s_keep[b] + pmask) >> sh;
        const int id = j < kept ? p.table[(size_t)b * p.max_pages + j]
                                : p.free_list[top - 1 - (s_need[b] + j - kept)];
        if (id >= 0 && id < p.n_pages) sl = id * p.page + (ps & pmask);
        else fault = HCL_ERR_DEVICE_FAULT;
      }
    }
    p.pos[t] = ps;
    p.slot[t] = sl;
  }
  if (lead) {
    int used = 0;
    for (int b = tid; b < p.B; b += nthr) {
      const bool ok = admitted(b);
      if (ok) used = max(used, s_need[b + 1] > s_need[b] ? s_need[b + 1] : 0);
      else fault |= HCL_ERR_NO_PAGES;
      p.seq_len[b] = s_keep[b] + (ok ? s_rows[b + 1] - s_rows[b] : 0);
    }
    for (int b = tid; b <= p.B; b += nthr) p.cu_new[b] = min(s_rows[b], p.T);
    atomicMax(&s_used, used);
    __syncthreads();
    if (tid == 0) *p.n_free = top - s_used;
  }
  if (fault) report(p.status, fault);
}

// ---------------------------------------------------------------------------------------
// Write.  A run is a stretch of consecutive slots of one page; one block quantises one run of
// one KV head and plane (k or v) at a time: up to page x d bf16 values held in registers (one
// read), their largest finite magnitude reduced over the block, codes written as 8-byte pieces.
// Bound by HBM: 2 bytes read and 1 written per value.
//
// grid.x covers the rows in chunks of `chunk` rows; a block takes the runs that begin in its
// chunk.  Prompts have one run per page of rows, a decode step one per row: the chunk is the
// page when that gives blocks enough to fill the GPU, less otherwise, down to one row.

constexpr int PW_THREADS = 128;  // (65 us for 64 K rows x 8 heads x 2 planes; 256 threads 73, 512 103)

__device__ __forceinline__ uint32_t bf2_absmax(uint32_t a, uint32_t b) {  // b: sign bits clear; NaN loses
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7FFF7FFFu), "r"(b));
  return r;
}

// Least power of two s >= 2^-126 with amax / s <= 448 = 1.75 * 2^8 (amax finite, >= 0).
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = int(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased exponent of s
  return __uint_as_float(uint32_t(max(e, 1)) << 23);
}

template <int D, int NP>  // NP 8-value pieces a thread: page * D / 8 <= NP * PW_THREADS
__global__ void __launch_bounds__(PW_THREADS) paged_write_kernel(PagedWriteArgs p, int sh, int chunk) {
  constexpr int PIECES = D / 8;  // per row
  __shared__ int s_len;
  __shared__ uint32_t s_begin[4];
  __shared__ float s_max[2][PW_THREADS / 32];  // (by turns: one barrier a run)
  int turn = 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int plane = blockIdx.y / p.kv.Hkv, g = blockIdx.y % p.kv.Hkv;
  const int page = p.kv.page;
  pdl_enter();
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(plane ? p.src[1] : p.src[0]);
  const int64_t stride = plane ? p.stride[1] : p.stride[0];
  uint8_t* codes = static_cast<uint8_t*>(plane ? p.kv.v : p.kv.k);
  float* scales = plane ? p.kv.v_scale : p.kv.k_scale;

  const int t_lo = blockIdx.x * chunk, t_hi = min(p.T, t_lo + chunk);
  // which rows of the chunk begin a run
  {
    const int t = t_lo + tid;
    bool begins = false;
    if (tid < chunk && t < t_hi) {
      const int slot = p.slot[t];
      const int prev = t > 0 ? p.slot[t - 1] : -1;
      // A row behind another of its page goes on with that run.  Where it is not the next slot it
      // begins none (two blocks would set the page's scale at once): it is left out.
      const bool goes_on = slot >= 0 && prev >= 0 && (prev >> sh) == (slot >> sh);
      begins = slot >= 0 && !goes_on;
      bool fault = goes_on && slot != prev + 1;
      if (begins && (slot >> sh) >= p.kv.n_pages) {
        begins = false;
        fault = true;
      }
      if (fault) report(p.status, HCL_ERR_DEVICE_FAULT);
    }
    const uint32_t mask = __ballot_sync(~0u, begins);
    if (lane == 0 && warp < 4) s_begin[warp] = mask;
  }
  __syncthreads();
  for (int c = 0; c < t_hi - t_lo; c++) {
    const uint32_t mask = s_begin[c >> 5] >> (c & 31);
    if (mask == 0) { c |= 31; continue; }
    c += __ffs(mask) - 1;
    const int t0 = t_lo + c, slot = p.slot[t0], off = slot & (page - 1);
    // The run: rows t0 + i with slot + i, up to the page's end.  Its rows are loaded while its
    // length is checked: all that the page has room for, where the next row continues it.
    const int most = min(page - off, p.T - t0);
    const int guess = most > 1 && p.slot[t0 + 1] == slot + 1 ? most : 1;
    const size_t pg = (size_t)(slot >> sh) * p.kv.Hkv + g;
    const float was = off ? scales[pg] : 0.f;
    uint4 x[NP];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < NP; i++) {
      const int e = i * PW_THREADS + tid;
      x[i] = make_uint4(0, 0, 0, 0);
      if (e < guess * PIECES)
        x[i] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)(t0 + e / PIECES) * stride +
                                                    g * D + (e % PIECES) * 8));
    }
    int n = guess;
    if (guess > 1 && !__syncthreads_and(tid >= most || p.slot[t0 + tid] == slot + tid)) {
      if (tid == 0) s_len = most;
      __syncthreads();
      if (tid < most && p.slot[t0 + tid] != slot + tid) atomicMin(&s_len, tid);
      __syncthreads();
      n = s_len;
#pragma unroll
      for (int i = 0; i < NP; i++)
        if (i * PW_THREADS + tid >= n * PIECES) x[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NP; i++)
      am = bf2_absmax(x[i].x, bf2_absmax(x[i].y, bf2_absmax(x[i].z, bf2_absmax(x[i].w, am))));
    float amax = fmaxf(bfbits2f(uint16_t(am & 0xFFFF)), bfbits2f(uint16_t(am >> 16)));
    if (!(amax < INFINITY)) {  // an infinity among them: the largest finite one
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < NP; i++) {
        const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float lo = fabsf(__uint_as_float(w4[j] << 16));
          const float hi = fabsf(__uint_as_float(w4[j] & 0xFFFF0000u));
          if (lo < INFINITY) amax = fmaxf(amax, lo);
          if (hi < INFINITY) amax = fmaxf(amax, hi);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    turn ^= 1;
    if (lane == 0) s_max[turn][warp] = amax;
    __syncthreads();
    amax = s_max[turn][lane & (PW_THREADS / 32 - 1)];
#pragma unroll
    for (int o = PW_THREADS / 64; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    const float s = fmaxf(pow2_scale(amax), was);
    // x / s: exact as a product when s is a power of two (a scale that the caller set may not be)
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    const float r = 1.f / s;
    uint8_t* base = codes + pg * page * D;
#pragma unroll
    for (int i = 0; i < NP; i++) {
      const int e = i * PW_THREADS + tid;
      if (e < n * PIECES) {
        const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          float lo = __uint_as_float(w4[j] << 16), hi = __uint_as_float(w4[j] & 0xFFFF0000u);
          if (pow2) { lo *= r; hi *= r; }
          else { lo = __fdiv_rn(lo, s); hi = __fdiv_rn(hi, s); }
          c[j] = cvt_e4m3x2(lo, hi);
        }
        *reinterpret_cast<uint2*>(base + (size_t)off * D + (size_t)e * 8) =
            make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
    }
    if (off && s != was) {
      // the scale grew: the rows before the run move to it
      const float f = was / s;
      for (int e = tid; e < off * PIECES; e += PW_THREADS) {
        uint2* at = reinterpret_cast<uint2*>(base + (size_t)e * 8);
        const uint2 old = *at;
        const uint16_t h[4] = {uint16_t(old.x), uint16_t(old.x >> 16), uint16_t(old.y),
                               uint16_t(old.y >> 16)};
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint32_t v;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(v) : "h"(h[j]));
          const __half2 hv = *reinterpret_cast<__half2*>(&v);
          c[j] = cvt_e4m3x2(__low2float(hv) * f, __high2float(hv) * f);
        }
        *at = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
    }
    if (tid == 0) scales[pg] = s;
  }
}

template <int D, int NP>
hcl_status_t write_t(const PagedWriteArgs& a, int sh, int chunk, cudaStream_t st) {
  const dim3 grid((a.T + chunk - 1) / chunk, a.kv.Hkv * (a.kv.v ? 2 : 1));
  return check_cuda(launch_pdl(paged_write_kernel<D, NP>, grid, dim3(PW_THREADS), 0, st, 1, a, sh, chunk),
                    "paged write launch");
}

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

}  // namespace

hcl_status_t launch_page_plan(const PagePlanArgs& a, cudaStream_t st) {
  const int smem = (4 * a.B + 3) * 4;
  // (the 48 KB that a launch may have without asking count the kernel's static arrays too)
  if (smem > 48 * 1024 - PP_STATIC) {
    hcl_status_t e = set_kernel_attrs(reinterpret_cast<const void*>(page_plan_kernel), smem, false);
    if (e != HCL_OK) return e;
  }
  // One block for small steps, without the cluster's barrier; eight share the expansions of others.
  // (Device time with 1 / 8 blocks: 8 rows 4.6 / 5.0 us, 2048 rows 6.9 / 6.9, 4096 rows 9.3 / 6.4,
  // 65536 rows 80 / 17; two or four are never the fastest by more than 0.3 us.)
  const int blocks = std::max(a.T, a.B) <= 2048 ? 1 : 8;
  return check_cuda(launch_pdl(page_plan_kernel, dim3(blocks), dim3(PP_THREADS), (size_t)smem, st, blocks,
                               a, log2_of(a.page)),
                    "page plan launch");
}

hcl_status_t launch_paged_write(const PagedWriteArgs& a, cudaStream_t st) {
  const int sh = log2_of(a.kv.page);
  const long long planes = (long long)a.kv.Hkv * (a.kv.v ? 2 : 1);
  if (planes > 65535) return fail(HCL_ERR_UNSUPPORTED, "paged write: too many KV heads");
  int chunk = a.kv.page;
  while (chunk > 1 && (a.T + chunk - 1) / chunk * planes < 8ll * num_sms()) chunk >>= 1;
  const int np = std::max(1, a.kv.page * a.kv.d / 8 / PW_THREADS);
  if (a.kv.d == 128) {
    if (np == 2) return write_t<128, 2>(a, sh, chunk, st);
    if (np == 4) return write_t<128, 4>(a, sh, chunk, st);
    if (np == 8) return write_t<128, 8>(a, sh, chunk, st);
    return write_t<128, 16>(a, sh, chunk, st);
  }
  if (np == 1) return write_t<64, 1>(a, sh, chunk, st);
  if (np == 2) return write_t<64, 2>(a, sh, chunk, st);
  if (np == 4) return write_t<64, 4>(a, sh, chunk, st);
  return write_t<64, 8>(a, sh, chunk, st);
}

}  // namespace hcl

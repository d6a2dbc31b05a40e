// paged_rows.cu -- paged attention for requests with few query rows (queries x heads of one KV
// head <= 16): decode and short drafts.  One pass over the codes, bound by HBM.
//
// Block: one producer warp and four consumer warps; two or three blocks per SM.  A unit is 64 KV
// rows of one request and KV head.  The producer copies its codes with TMA (one box per page, or
// per 64 rows of a longer page) into a ring of swizzled stages and its page scales with 4-byte
// asynchronous copies that complete on the same mbarrier; page ids are read eight units at a time,
// eight ahead.  With at most 8 query rows consumer warps 0, 1 take the even units and 2, 3 the odd
// ones, each 32 rows; with 9 to 16 every unit goes to all four, warps 0, 1 with the first 8 query
// rows and 2, 3 with the others, so that every code is converted in two warps (device time of
// 4 requests on up to 512 entries, 16 heads: 13 us with each half on a unit of its own, 10.6 so).
// Each has its own running softmax, so warps never wait for one another inside an item:
//   S^T (16 KV rows x 8 query rows) by m16n8k16 fp16 MMAs: KV rows are the M of the MMA, so up to
//   8 query rows (a group of 8 heads) waste none of it.  The K fragments come from ldmatrix on
//   the codes (a 16-byte piece of a row is one k-step, its dimensions taken in the order that
//   gives each thread four neighbouring codes; Q is laid out alike) and a conversion to fp16;
//   O^T (16 dimensions x 8 query rows) += V^T P^T from transposed ldmatrix on pairs of codes (a
//   pair's even and odd dimensions are rows m and m + 8); P^T is S^T's layout transposed
//   (movmatrix).
// The bytes bound the kernel once the chain from load to store is covered.  32 requests of up to
// 32 K rows, 8 KV heads of 8 query heads (1.37 GB, 209 us at the copy rate): 300 us with query
// rows as M, 16 KV rows a warp and step; 265 us with 32 KV rows; 222 us in this form (device
// time).  A lvref for each query row costs 2.5 % of that though it is one number while all rows
// have seen all groups; formed for each row in every step it cost 7 %.
#include <algorithm>

#include "paged_common.cuh"

namespace hcl {
namespace paged {
namespace {

constexpr int NW = 4;                  // consumer warps
constexpr int THREADS = (NW + 1) * 32;
constexpr int TILE = 64;               // KV rows per unit
constexpr int NG = 2;                  // groups of 16 rows (never more than a page) per warp and unit
constexpr int WPT = TILE / (16 * NG);  // warps per unit
constexpr float P_OFF = P_OFF_ROWS, P_LAZY = 15.f - P_OFF;

// Blocks per SM: three where an even number of stages leaves the room.
constexpr int blocks_per_sm(int d, bool shared) { return d == 128 && !shared ? 2 : 3; }

// RH: query rows / 8 that the warps divide among them
template <int D, bool SHARED, int RH>
struct Cfg {
  static constexpr int ROWS = 8 * RH;
  static constexpr int BLOCKS = blocks_per_sm(D, SHARED);
  static constexpr int PLANE = TILE * D;
  static constexpr int STAGE = PLANE * (SHARED ? 1 : 2);
  static constexpr int RING = BLOCKS == 3 ? 49152 : 65536;
  static constexpr int STAGES = RING / STAGE < 8 ? RING / STAGE : 8;
  // A stage always belongs to the same consumer warps: a warp that waited on every other phase of
  // a barrier could take an old phase for the one it wants.
  static_assert(STAGES % (NW / WPT) == 0, "stages");
  static constexpr int PIECES = D / 16;  // 16-byte pieces of a row = k-steps
  static constexpr int PITCH = D + 4;    // floats of a row in the exchange
  static constexpr uint32_t SCALES = STAGES * STAGE;                    // [STAGES][2][4] floats
  static constexpr uint32_t MERGE = SCALES + STAGES * 32;               // [NW][8][PITCH] floats
  static constexpr uint32_t STATS = MERGE + NW * 8 * PITCH * 4;         // [NW][8][3] floats
  static constexpr uint32_t BAR = STATS + NW * 8 * 3 * 4;
  static constexpr uint32_t SCRATCH = BAR + 2 * STAGES * 8;             // find_share
  static constexpr uint32_t MISC = SCRATCH + (NW + 1 + 4) * 8;
  static constexpr uint32_t TOTAL = MISC + 16;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held in fragment layout.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Byte address of 16-byte piece `c` of row `r` in a swizzled plane (128-byte rows: 128B mode,
// 64-byte rows: 64B mode).
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// The request's KV tiles for this kernel: first tile, and how many (one at least, so that rows
// that see nothing are written too).  0 tiles: not a request of this kernel.
__device__ __forceinline__ int tiles_of(const Params& p, const Req& r, int* t0) {
  *t0 = 0;
  if (r.nq == 0 || r.nq * p.G > ROWS_SMALL) return 0;
  const int hi = vis_hi(p, r, r.nq - 1), lo = min(vis_lo(p, r, 0), hi);
  if (hi <= lo) return 1;
  *t0 = lo / TILE;
  return (hi + TILE - 1) / TILE - *t0;
}

// Walks a block's units item by item.
struct Walk {
  Req r;
  int b, g, t0, nt;  // request, KV head, the item's first tile and tile count
  int tile, count;   // this block's part of the item: tiles tile .. tile + count - 1 of the nt
  long long left;    // units of the block after this part
};
__device__ __forceinline__ void walk_set(const Params& p, Walk& w) {
  w.count = (int)min((long long)(w.nt - w.tile), w.left);
  w.left -= w.count;
}
__device__ __forceinline__ bool walk_first(const Params& p, const Share& s, Walk& w) {
  w.left = s.u1 - s.u0;
  if (w.left <= 0) return false;
  w.b = s.e;
  w.r = load_req(p, w.b, false);
  w.nt = tiles_of(p, w.r, &w.t0);
  w.g = (int)(s.rem / w.nt);
  w.tile = (int)(s.rem % w.nt);
  walk_set(p, w);
  return true;
}
__device__ __forceinline__ bool walk_next(const Params& p, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.g == p.a.kv.Hkv) {
    w.g = 0;
    do {
      w.r = load_req(p, ++w.b, false);
      w.nt = tiles_of(p, w.r, &w.t0);
    } while (w.nt == 0);
  }
  w.tile = 0;
  walk_set(p, w);
  return true;
}

template <int D, bool SHARED, int RH>
__global__ void __launch_bounds__(THREADS, (Cfg<D, SHARED, RH>::BLOCKS))
    paged_rows_kernel(const Params p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using C = Cfg<D, SHARED, RH>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);  // (an offset: the compiler still sees shared memory)
  float* s_scale = reinterpret_cast<float*>(sm + C::SCALES);
  float* s_merge = reinterpret_cast<float*>(sm + C::MERGE);
  float* s_stat = reinterpret_cast<float*>(sm + C::STATS);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::BAR);
  uint64_t* empty = full + C::STAGES;
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + C::MISC);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; i++) {
      mbar_init(&full[i], 1 + 32);
      mbar_init(&empty[i], WPT * RH);
    }
    *s_abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tk);
    if (!SHARED) prefetch_tmap(&tv);
  }
  pdl_enter();
  const Share share = find_share<THREADS>(p.a.B, blockIdx.x, p.n_blocks, reinterpret_cast<long long*>(sm + C::SCRATCH),
                                          [&](int b) {
                                            const Req r = load_req(p, b, blockIdx.x == 0);
                                            int t0;
                                            return (long long)tiles_of(p, r, &t0) * p.a.kv.Hkv;
                                          });
  Walk w = {};
  const bool any = walk_first(p, share, w);
  if (tid == 0) {
    Meta* m = p.meta + blockIdx.x;
    m->ends = any && w.tile > 0 && w.tile + w.count == w.nt;
    m->first = share.u0 - w.tile;
    m->tot = share.tot;
    m->nb = share.nb;
    m->b = w.b;
    m->g = w.g;
    m->row0 = 0;
  }
  if (!any) return;

  if (warp == NW) {
    // ------------------------------------------------------------------ producer
    const int box = min(p.a.kv.page, TILE);  // rows of a box
    uint32_t it = 0;
    bool fault = false, ok = true;
    // pages of the 32 groups from tile i of this part on; -2 behind the rows held
    auto pages_at = [&](int i) {
      const int t = (w.t0 + w.tile + i) * TILE + lane * 16;
      return i < w.count && t < w.r.len ? __ldg(p.a.table + (size_t)w.b * p.a.max_pages + (t >> p.sh)) : -2;
    };
    do {
      int ids = -2, ids_next = pages_at(0);
      for (int i = 0; i < w.count && ok; i++, it++) {
        if ((i & 7) == 0) {
          ids = ids_next;
          ids_next = pages_at(i + 8);
        }
        const int id = __shfl_sync(~0u, ids, (i & 7) * 4 + (lane & 3));
        const int st = it % C::STAGES;
        if (it >= C::STAGES)
          ok = __all_sync(~0u, mbar_wait(&empty[st], ((it / C::STAGES) & 1) ^ 1, p.limit, s_abort));
        if (!ok) break;
        const bool good = id >= 0 && id < p.a.kv.n_pages;
        if (!good && id != -2 && lane < 4) fault = true;
        const int row = (int)(((long long)id * p.a.kv.Hkv + w.g) << p.sh);  // the page's first code row
        const int t = (w.t0 + w.tile + i) * TILE + (lane & 3) * 16;
        float* sc = s_scale + st * 8;
        uint8_t* kp = sm + st * C::STAGE;
        const bool first = lane < 4 && (lane & (box / 16 - 1)) == 0;  // this lane's group begins a box
        const uint32_t boxes = __popc(__ballot_sync(~0u, first && good));
        if (lane < 4 && !good) sc[lane] = 0.f;  // no page: the group is left out
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], boxes * box * D * (SHARED ? 1 : 2));
        __syncwarp();
        if (first && good) {
          tma_load_2d(kp + lane * 16 * D, &tk, &full[st], 0, row + (t & (p.a.kv.page - 1)));
          if (!SHARED) tma_load_2d(kp + C::PLANE + lane * 16 * D, &tv, &full[st], 0, row + (t & (p.a.kv.page - 1)));
        }
        if (lane < 4 && good) {
          const size_t pg = (size_t)id * p.a.kv.Hkv + w.g;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sc + lane)),
                       "l"(p.a.kv.k_scale + pg) : "memory");
          if (!SHARED)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sc + 4 + lane)),
                         "l"(p.a.kv.v_scale + pg) : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[st])) : "memory");
      }
    } while (ok && walk_next(p, w));
    if (!ok) {
      *s_abort = 1;
      if (lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
    }
    // every copy has landed before the block's shared memory goes away
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; k < it; k++)
      if (!mbar_wait(&full[k % C::STAGES], (k / C::STAGES) & 1, p.limit, nullptr) && lane == 0)
        report(p.a.status, HCL_ERR_TIMEOUT);
    if (fault) report(p.a.status, HCL_ERR_DEVICE_FAULT);
    return;
  }

  // -------------------------------------------------------------------- consumers
  // r0: KV row (and + 8) of a score, even / odd dimension pair of an output, query row of a Q
  // fragment; this thread's query rows: row0 + 2 t4 + e, e < 2
  const int r0 = lane >> 2, t4 = lane & 3;
  const int row0 = RH == 2 ? 8 * (warp >> 1) : 0;
  uint32_t it = 0;
  bool ok = true;
  do {
    const int nrows = w.r.nq * p.G;
    // Q row row0 + r0 (row = query * G + head), dims 16c + 4 t4 .. + 3 of every piece
    uint32_t qf[C::PIECES][2];
    float back[2];
    int hi_r[2], lo_r[2];
    {
      const int row = row0 + r0;
      const bool valid = row < nrows;
      const int i = valid ? p.by_G.div(row) : 0, head = w.g * p.G + (valid ? row - i * p.G : 0);
      const uint2* src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.a.q) +
                                                        (int64_t)(w.r.c0 + i) * p.a.q_stride + head * D) + t4;
      uint2 x[C::PIECES];
      float am = 0.f;
#pragma unroll
      for (int c = 0; c < C::PIECES; c++) x[c] = valid ? __ldg(src + c * 4) : make_uint2(0, 0);
#pragma unroll
      for (int c = 0; c < C::PIECES; c++) {
        const uint32_t a[2] = {x[c].x, x[c].y};
#pragma unroll
        for (int k = 0; k < 2; k++)
          am = fmax3(am, fabsf(__uint_as_float(a[k] << 16)), fabsf(__uint_as_float(a[k] & 0xFFFF0000u)));
      }
      am = fmaxf(am, __shfl_xor_sync(~0u, am, 1));
      am = fmaxf(am, __shfl_xor_sync(~0u, am, 2));
      float bk;
      const float f = row_factor(am, &bk);
#pragma unroll
      for (int e = 0; e < 2; e++) back[e] = __shfl_sync(~0u, bk, (2 * t4 + e) * 4);
#pragma unroll
      for (int c = 0; c < C::PIECES; c++) {
        qf[c][0] = half2_of(__uint_as_float(x[c].x << 16) * f, __uint_as_float(x[c].x & 0xFFFF0000u) * f);
        qf[c][1] = half2_of(__uint_as_float(x[c].y << 16) * f, __uint_as_float(x[c].y & 0xFFFF0000u) * f);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; r++) {
      const int row = row0 + 2 * t4 + r;
      const bool valid = row < nrows;
      const int i = valid ? p.by_G.div(row) : 0;
      hi_r[r] = valid ? vis_hi(p, w.r, i) : 0;
      lo_r[r] = valid ? vis_lo(p, w.r, i) : 0;
    }
    // the rows that all queries see, and that any sees
    const int all_lo = vis_lo(p, w.r, w.r.nq - 1), all_hi = vis_hi(p, w.r, 0);
    const int any_lo = vis_lo(p, w.r, 0), any_hi = vis_hi(p, w.r, w.r.nq - 1);

    float o[C::PIECES][4];  // dims 16 c + 2 r0 (+ 1 for the last two), query row e = k & 1
#pragma unroll
    for (int c = 0; c < C::PIECES; c++)
#pragma unroll
      for (int k = 0; k < 4; k++) o[c][k] = 0.f;
    const int rows0 = (warp % WPT) * 16 * NG;  // this warp's rows of a tile
    float M[2], l[2], lvref[2];
    bool alike = true;  // lvref is one for all query rows of the warp
#pragma unroll
    for (int r = 0; r < 2; r++) {
      M[r] = lvref[r] = -INFINITY;
      l[r] = 0.f;
    }

    for (int i = 0; i < w.count; i++, it++) {
      if (RH == 1 && it % (NW / WPT) != warp / WPT) continue;
      const int st = it % C::STAGES;
      ok = mbar_wait(&full[st], (it / C::STAGES) & 1, p.limit, s_abort);
      ok = __all_sync(~0u, ok);
      if (!ok) break;
      const int j0 = (w.t0 + w.tile + i) * TILE + rows0;
      float ks[NG];
#pragma unroll
      for (int g = 0; g < NG; g++) ks[g] = s_scale[st * 8 + (rows0 >> 4) + g];
      if (j0 < any_hi && j0 + 16 * NG > any_lo) {
        const uint32_t kb = smem_u32(sm + st * C::STAGE) + rows0 * D;
        const uint32_t vb = kb + (SHARED ? 0 : C::PLANE);
        // rows (lane & 15) of a group, piece (lane >> 4) of two
        const int frow = lane & 15, fpiece = lane >> 4;
        // S^T: z[g][k]: KV row 16 g + r0 + 8 (k >> 1), query row e = k & 1
        float z[NG][4];
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
          for (int k = 0; k < 4; k++) z[g][k] = 0.f;
#pragma unroll
        for (int c = 0; c < C::PIECES; c += 2)
#pragma unroll
          for (int g = 0; g < NG; g++) {
            uint32_t r[4];
            ldsm4(kb + piece<D>(g * 16 + frow, c + fpiece), r);
#pragma unroll
            for (int u = 0; u < 2; u++) {
              const uint32_t a[4] = {half2_of_codes(uint16_t(r[2 * u])), half2_of_codes(uint16_t(r[2 * u + 1])),
                                     half2_of_codes(uint16_t(r[2 * u] >> 16)), half2_of_codes(uint16_t(r[2 * u + 1] >> 16))};
              mma16816(z[g], a, qf[c + u][0], qf[c + u][1]);
            }
          }
        uint32_t poison = 0;  // a bit for each of the KV rows
        static_assert(16 * NG <= 32, "poison");
        const bool edge = j0 < all_lo || j0 + 16 * NG > all_hi || !(ks[0] > 0.f) || !(ks[NG - 1] > 0.f);
        if (edge) {
          // some query row does not see some of these KV rows, or a group has no page
#pragma unroll
          for (int g = 0; g < NG; g++)
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const int j = j0 + g * 16 + r0 + 8 * (k >> 1), r = k & 1;
              if (j < lo_r[r] || j >= hi_r[r] || !(ks[g] > 0.f)) z[g][k] = -INFINITY;
            }
          // NaN codes among the values would reach the query rows that do not see them (0 * NaN),
          // and rows behind the last (or of no page) hold anything: below they are taken as 0, and
          // `poison` says which KV rows had one
          const uint8_t* vp = sm + st * C::STAGE + (SHARED ? 0 : C::PLANE) + rows0 * D;
#pragma unroll
          for (int g = 0; g < NG; g++)
#pragma unroll
            for (int i2 = 0; i2 < C::PIECES / 2; i2++) {
              const int e = i2 * 32 + lane;  // piece of the group
              const uint4 v = *reinterpret_cast<const uint4*>(vp + g * 16 * D + e * 16);
              if (ks[g] > 0.f && (nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w)))
                poison |= 1u << (g * 16 + e / C::PIECES);
            }
          poison = __reduce_or_sync(~0u, poison);
        }
        float lvg[NG], kc[NG], Mo[2];  // Mo: O's reference
#pragma unroll
        for (int g = 0; g < NG; g++) {
          lvg[g] = log2_scale(SHARED ? ks[g] : s_scale[st * 8 + 4 + (rows0 >> 4) + g]);
          kc[g] = fmaxf(ks[g], SCALE_MIN) * p.scale2;
        }
#pragma unroll
        for (int r = 0; r < 2; r++) Mo[r] = M[r];
        float al[2], e[NG][2][2];
        bool grew = false;
        // lvref of query row r grows by d: l lies over the row's eight lanes, whose M must move alike
        auto grow = [&](int r, float d) {
          float big = l[r];
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o2));
          const float was = M[r];
          if (d > 0.f) grow_lvref(d, big, M[r]);
          if (was != -INFINITY) l[r] *= exp2f(d - (M[r] - was));
        };
        // probabilities of query row r with lv and wl of the groups
        auto probabilities = [&](int r, const float (&lv)[NG], const float (&wl)[NG]) {
          float c[NG], mw = -INFINITY;  // largest z2 + lv
#pragma unroll
          for (int g = 0; g < NG; g++) {
            c[g] = fmaxf(kc[g] * back[r], SCALE_MIN);
            mw = fmaxf(mw, fmaf(fmaxf(z[g][r], z[g][2 + r]), c[g], lv[g]));
          }
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) mw = fmaxf(mw, __shfl_xor_sync(~0u, mw, o2));
          const float M2 = mw > M[r] + P_LAZY ? mw : M[r];
          al[r] = M2 == Mo[r] || Mo[r] == -INFINITY ? 1.f : ex2_ftz(Mo[r] - M2);
          const float ll = M[r] == Mo[r] ? al[r] : ex2_ftz(M[r] - M2);
          grew |= al[r] != 1.f;
          M[r] = M2;
          // rows without a reference yet have seen nothing: their z are all -inf
          const float Mu = M2 == -INFINITY ? 0.f : M2;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < NG; g++) {
#pragma unroll
            for (int k = 0; k < 2; k++) e[g][r][k] = ex2_ftz(fmaf(z[g][2 * k + r], c[g], lv[g] - Mu + P_OFF));
            sum = fmaf(e[g][r][0] + e[g][r][1], wl[g], sum);
          }
          l[r] = fmaf(l[r], ll, sum);
        };
        alike = alike && !edge;
        if (alike) {
          // every query row has seen every group so far: one lvref
          const float was = lvref[0];
          float ref = was, lv[NG], wl[NG];
#pragma unroll
          for (int g = 0; g < NG; g++) ref = fmaxf(ref, lvg[g]);
#pragma unroll
          for (int g = 0; g < NG; g++) {
            lv[g] = fmaxf(lvg[g], ref - LV_SPAN);
            wl[g] = ex2_ftz(ref - lv[g]);
          }
          lvref[0] = lvref[1] = ref;
          if (ref != was && was != -INFINITY) {
#pragma unroll
            for (int r = 0; r < 2; r++) grow(r, ref - was);
          }
#pragma unroll
          for (int r = 0; r < 2; r++) probabilities(r, lv, wl);
        } else {
#pragma unroll
          for (int r = 0; r < 2; r++) {
            const float was = lvref[r];
            float ref = was, lv[NG], wl[NG];
#pragma unroll
            for (int g = 0; g < NG; g++)
              if (!edge || (ks[g] > 0.f && j0 + g * 16 < hi_r[r] && j0 + g * 16 + 16 > lo_r[r])) ref = fmaxf(ref, lvg[g]);
#pragma unroll
            for (int g = 0; g < NG; g++) {
              lv[g] = fmaxf(lvg[g], ref - LV_SPAN);
              wl[g] = ex2_ftz(ref - lv[g]);
            }
            lvref[r] = ref;
            grow(r, was == -INFINITY ? 0.f : ref - was);
            probabilities(r, lv, wl);
            for (uint32_t b = poison; b; b &= b - 1) {
              const int j = j0 + __ffs(b) - 1;
              if (j >= lo_r[r] && j < hi_r[r]) l[r] = NAN;
            }
          }
        }
        uint32_t pb[NG][2];  // P^T fragments
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
          for (int k = 0; k < 2; k++) pb[g][k] = transpose8(half2_of(e[g][0][k], e[g][1][k]));
        if (__any_sync(~0u, grew)) {
#pragma unroll
          for (int c = 0; c < C::PIECES; c++)
#pragma unroll
            for (int k = 0; k < 4; k++) o[c][k] *= al[k & 1];
        }
        // O^T += V^T P^T: pieces c, c + 1 per ldmatrix
#pragma unroll
        for (int c = 0; c < C::PIECES; c += 2)
#pragma unroll
          for (int g = 0; g < NG; g++) {
            uint32_t r[4];
            ldsm4t(vb + piece<D>(g * 16 + frow, c + fpiece), r);
            if (edge) {
#pragma unroll
              for (int i2 = 0; i2 < 4; i2++) r[i2] &= ~nan_bytes(r[i2]);
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
              // bytes (row 2t dim 2n, row 2t dim 2n+1, row 2t+1 dim 2n, row 2t+1 dim 2n+1)
              const uint32_t x0 = __byte_perm(r[2 * u], 0, 0x3120), x1 = __byte_perm(r[2 * u + 1], 0, 0x3120);
              const uint32_t a[4] = {half2_of_codes(uint16_t(x0)), half2_of_codes(uint16_t(x0 >> 16)),
                                     half2_of_codes(uint16_t(x1)), half2_of_codes(uint16_t(x1 >> 16))};
              mma16816(o[c + u], a, pb[g][0], pb[g][1]);
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (!ok) {
      *s_abort = 1;
      if (lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
    }
    // join the warps: l's partial sums lie over the eight threads of a query row
#pragma unroll
    for (int r = 0; r < 2; r++) {
#pragma unroll
      for (int o2 = 4; o2 < 32; o2 <<= 1) l[r] += __shfl_xor_sync(~0u, l[r], o2);
      if (r0 == 0) {
        float* s3 = s_stat + (warp * 8 + 2 * t4 + r) * 3;
        s3[0] = M[r] == -INFINITY ? -INFINITY : M[r] - P_OFF - lvref[r]; s3[1] = M[r]; s3[2] = l[r];
      }
    }
    // O in its own reference; the readers weigh it
#pragma unroll
    for (int c = 0; c < C::PIECES; c++)
#pragma unroll
      for (int r = 0; r < 2; r++)
        *reinterpret_cast<float2*>(s_merge + (warp * 8 + 2 * t4 + r) * C::PITCH + c * 16 + 2 * r0) =
            make_float2(o[c][r], o[c][2 + r]);
    // (a warp whose wait ran out ends the block here, at the same item for all four)
    uint32_t gone;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(gone) : "r"(uint32_t(!ok)), "n"(NW * 32) : "memory");
    if (gone) break;
    {
      // all four warps: rows of D / 4 threads with four dimensions each
      const bool whole = w.count == w.nt;
      float* pp = p.part + (2 * (size_t)blockIdx.x + (w.tile == 0 ? 1 : 0)) * part_floats(ROWS_SMALL, D);
      constexpr int TPR = D / 4;
      const int col = (tid % TPR) * 4;
#pragma unroll
      for (int k = 0; k < C::ROWS * TPR / (NW * 32); k++) {
        const int row = tid / TPR + k * (NW * 32 / TPR);
        // the warps that had this row
        constexpr int NV = NW / RH;
        const int v0 = (RH == 2 ? (row >> 3) * NV : 0) * 8 + (row & 7);
        float mt = -INFINITY, Mt = -INFINITY, lt = 0.f;
#pragma unroll
        for (int v = 0; v < NV; v++) {
          const float* s3 = s_stat + (v0 + v * 8) * 3;
          mt = fmaxf(mt, s3[0]);
          Mt = fmaxf(Mt, s3[1]);
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < NV; v++) {
          const float* s3 = s_stat + (v0 + v * 8) * 3;
          lt += s3[0] == -INFINITY ? s3[2] : s3[2] * ex2_ftz(s3[0] - mt);
          const float f = s3[1] == -INFINITY ? 0.f : ex2_ftz(s3[1] - Mt);
          if (f != 0.f) {
            const float4 x = *reinterpret_cast<const float4*>(s_merge + (v0 + v * 8) * C::PITCH + col);
            a.x = fmaf(x.x, f, a.x); a.y = fmaf(x.y, f, a.y); a.z = fmaf(x.z, f, a.z); a.w = fmaf(x.w, f, a.w);
          }
        }
        if (row >= nrows) continue;
        if (whole) {
          const int i = p.by_G.div(row), head = w.g * p.G + row - i * p.G;
          const size_t orow = (size_t)(w.r.c0 + i) * p.a.H + head;
          float lse, f2;
          const float f = finish_row<true>(mt, Mt, lt, p.a.sink ? p.a.sink[head] * LOG2E : -INFINITY, &f2, &lse);
          a = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                       : make_float4(a.x * f * f2, a.y * f * f2, a.z * f * f2, a.w * f * f2);
          if (p.a.out32)
            *reinterpret_cast<float4*>(p.a.out32 + orow * D + col) = a;
          else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + orow * D + col) =
                make_uint2(bf16x2_of(a.x, a.y), bf16x2_of(a.z, a.w));
          if (col == 0 && p.a.lse) p.a.lse[orow] = lse;
        } else {
          *reinterpret_cast<float4*>(pp + ROWS_SMALL * 4 + row * D + col) = a;
          if (col == 0) *reinterpret_cast<float4*>(pp + row * 4) = make_float4(mt, Mt, lt, 0.f);
        }
      }
    }
    // the exchange is free again
    asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
  } while (walk_next(p, w));
}

template <int D, bool SHARED, int RH>
hcl_status_t launch_t(const Params& p, cudaStream_t st) {
  CUtensorMap tk, tv;
  const int box = std::min(p.a.kv.page, TILE);
  hcl_status_t e = code_map(&tk, p.a.kv.k, p.a.kv, box, true);
  if (e != HCL_OK) return e;
  tv = tk;
  if (!SHARED) {
    e = code_map(&tv, p.a.kv.v, p.a.kv, box, true);
    if (e != HCL_OK) return e;
  }
  using C = Cfg<D, SHARED, RH>;
  auto kern = paged_rows_kernel<D, SHARED, RH>;
  const int smem = (int)C::TOTAL + 1024;
  static_assert(C::BLOCKS * (C::TOTAL + 2048) <= 233472, "blocks per SM");
  e = set_kernel_attrs(reinterpret_cast<const void*>(kern), smem, false);
  if (e != HCL_OK) return e;
  return check_cuda(launch_pdl(kern, dim3(p.n_blocks), dim3(THREADS), (size_t)smem, st, 1, p, tk, tv),
                    "paged attention (rows) launch");
}

}  // namespace

int rows_blocks(int d, bool shared) {
  return std::min(1024, blocks_per_sm(d, shared) * num_sms());
}

hcl_status_t launch_rows(const Params& p, int rows, cudaStream_t st) {
  const bool d128 = p.a.kv.d == 128, v = p.a.kv.v != nullptr;
  if (rows <= 8) {
    if (d128) return v ? launch_t<128, false, 1>(p, st) : launch_t<128, true, 1>(p, st);
    return v ? launch_t<64, false, 1>(p, st) : launch_t<64, true, 1>(p, st);
  }
  if (d128) return v ? launch_t<128, false, 2>(p, st) : launch_t<128, true, 2>(p, st);
  return v ? launch_t<64, false, 2>(p, st) : launch_t<64, true, 2>(p, st);
}

hcl_status_t code_map(CUtensorMap* m, const void* codes, const hcl_paged_kv_t& kv, int rows, bool swizzle) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(HCL_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {(cuuint64_t)kv.d, (cuuint64_t)kv.n_pages * kv.Hkv * kv.page};
  const cuuint64_t strides[1] = {(cuuint64_t)kv.d};
  const cuuint32_t box[2] = {(cuuint32_t)kv.d, (cuuint32_t)rows};
  const cuuint32_t el[2] = {1, 1};
  const CUtensorMapSwizzle sw = !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : kv.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, el,
          CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(HCL_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  return HCL_OK;
}

}  // namespace paged
}  // namespace hcl

// paged_rows.cu -- paged attention for requests with few query rows (queries x heads of one KV
// head <= 16): decode and short drafts.  One pass over the codes, bound by HBM.
//
// Block: one producer warp and four consumer warps, two blocks per SM.  A unit is 64 KV rows of
// one request and KV head.  The producer copies its codes with TMA (one box per page, or per 64
// rows of a longer page) into a ring of swizzled stages and its page scales with 4-byte
// asynchronous copies that complete on the same mbarrier; page ids are read eight units at a time,
// eight ahead.  Consumer warps 0, 1 take the even units and 2, 3 the odd ones, each 32 rows and
// its own running softmax, so warps never wait for one another inside an item.  (With 16 rows of
// every unit to each warp the chain from load to store, not the bytes, set the pace: 300 us for
// 1.37 GB; with 32, 265 us; 64 gain nothing more.)
//   S (16 query rows x 32 KV rows) by m16n8k16 fp16 MMAs; the K fragments come from ldmatrix on
//   the codes (a 16-byte piece of a row is one k-step, its dimensions taken in the order that
//   gives each thread four neighbouring codes; Q is laid out alike) and a conversion to fp16;
//   O += P V the same way from transposed ldmatrix on pairs of codes (even and odd dimensions
//   make two n-tiles).
// The tensor cores run at a fraction of their rate here; the bytes bound the kernel.
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

template <int D, bool SHARED>
struct Cfg {
  static constexpr int PLANE = TILE * D;
  static constexpr int STAGE = PLANE * (SHARED ? 1 : 2);
  static constexpr int STAGES = D == 128 ? (SHARED ? 8 : 4) : 8;
  static constexpr int PIECES = D / 16;  // 16-byte pieces of a row = k-steps
  static constexpr uint32_t SCALES = STAGES * STAGE;                // [STAGES][2][4] floats
  static constexpr uint32_t MERGE = SCALES + STAGES * 32;           // [NW - 1][16][D] floats
  static constexpr uint32_t STATS = MERGE + (NW - 1) * 16 * D * 4;  // [NW][16][3] floats
  static constexpr uint32_t BAR = STATS + NW * 16 * 3 * 4;
  static constexpr uint32_t SCRATCH = BAR + 2 * STAGES * 8;         // find_share
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

template <int D, bool SHARED>
__global__ void __launch_bounds__(THREADS, 2)
    paged_rows_kernel(const Params p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using C = Cfg<D, SHARED>;
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
      mbar_init(&empty[i], WPT);
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
  const int r0 = lane >> 2, t4 = lane & 3;  // fragment row (and + 8), column group
  uint32_t it = 0;
  bool ok = true;
  do {
    // Q rows r0, r0 + 8 (row = query * G + head), dims 16c + 4 t4 .. + 3 of every piece
    const int nrows = w.r.nq * p.G;
    uint32_t qf[C::PIECES][4];
    float back[2];
    int hi_r[2], lo_r[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int row = r0 + 8 * h;
      const bool valid = row < nrows;
      const int i = valid ? p.by_G.div(row) : 0, head = w.g * p.G + (valid ? row - i * p.G : 0);
      hi_r[h] = valid ? vis_hi(p, w.r, i) : 0;
      lo_r[h] = valid ? vis_lo(p, w.r, i) : 0;
      const uint2* src = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.a.q) +
                                                        (int64_t)(w.r.c0 + i) * p.a.q_stride + head * D) + t4;
      uint2 x[C::PIECES];
      float am = 0.f;
#pragma unroll
      for (int c = 0; c < C::PIECES; c++) {
        x[c] = valid ? __ldg(src + c * 4) : make_uint2(0, 0);
        const uint32_t a[2] = {x[c].x, x[c].y};
#pragma unroll
        for (int k = 0; k < 2; k++)
          am = fmaxf(am, fmaxf(fabsf(__uint_as_float(a[k] << 16)), fabsf(__uint_as_float(a[k] & 0xFFFF0000u))));
      }
      am = fmaxf(am, __shfl_xor_sync(~0u, am, 1));
      am = fmaxf(am, __shfl_xor_sync(~0u, am, 2));
      const float f = row_factor(am, &back[h]);
#pragma unroll
      for (int c = 0; c < C::PIECES; c++) {
        qf[c][h] = half2_of(__uint_as_float(x[c].x << 16) * f, __uint_as_float(x[c].x & 0xFFFF0000u) * f);
        qf[c][2 + h] = half2_of(__uint_as_float(x[c].y << 16) * f, __uint_as_float(x[c].y & 0xFFFF0000u) * f);
      }
    }
    // the rows that all queries see, and that any sees
    const int all_lo = vis_lo(p, w.r, w.r.nq - 1), all_hi = vis_hi(p, w.r, 0);
    const int any_lo = vis_lo(p, w.r, 0), any_hi = vis_hi(p, w.r, w.r.nq - 1);

    float o[C::PIECES][8];  // [piece][row half][dims 4 t4 .. + 3]
#pragma unroll
    for (int c = 0; c < C::PIECES; c++)
#pragma unroll
      for (int k = 0; k < 8; k++) o[c][k] = 0.f;
    const int rows0 = (warp % WPT) * 16 * NG;  // this warp's rows of a tile
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lvref = -INFINITY;

    for (int i = 0; i < w.count; i++, it++) {
      if (it % (NW / WPT) != warp / WPT) continue;
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
        // S
        float s[2 * NG][4];  // [n-tile]
#pragma unroll
        for (int n = 0; n < 2 * NG; n++)
#pragma unroll
          for (int k = 0; k < 4; k++) s[n][k] = 0.f;
#pragma unroll
        for (int q = 0; q < C::PIECES / 4; q++)
#pragma unroll
          for (int n = 0; n < 2 * NG; n++) {
            uint32_t r[4];
            ldsm4(kb + piece<D>(n * 8 + (lane & 7), q * 4 + (lane >> 3)), r);
#pragma unroll
            for (int c = 0; c < 4; c++)
              mma16816(s[n], qf[q * 4 + c], half2_of_codes(uint16_t(r[c])), half2_of_codes(uint16_t(r[c] >> 16)));
          }
        float z[NG][2][4];  // [group][row half][columns 2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4]
#pragma unroll
        for (int g = 0; g < NG; g++)
#pragma unroll
          for (int h = 0; h < 2; h++)
#pragma unroll
            for (int k = 0; k < 4; k++)  // (a group without a page is left out)
              z[g][h][k] = ks[g] > 0.f ? s[2 * g + (k >> 1)][2 * h + (k & 1)] : -INFINITY;
        uint32_t poison = 0;  // a bit for each of the KV rows
        static_assert(16 * NG <= 32, "poison");
        if (j0 < all_lo || j0 + 16 * NG > all_hi || !(ks[0] > 0.f) || !(ks[NG - 1] > 0.f)) {
          // some row does not see some of these KV rows
#pragma unroll
          for (int g = 0; g < NG; g++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
              for (int k = 0; k < 4; k++) {
                const int j = j0 + g * 16 + (k >> 1) * 8 + 2 * t4 + (k & 1);
                if (j < lo_r[h] || j >= hi_r[h]) z[g][h][k] = -INFINITY;
              }
          // NaN codes among the values would reach the rows that do not see them (0 * NaN), and
          // rows behind the last (or of no page) hold anything: they become 0, and `poison` says
          // which KV rows had one
          __syncwarp();
          uint8_t* vp = sm + st * C::STAGE + (SHARED ? 0 : C::PLANE) + rows0 * D;
#pragma unroll
          for (int g = 0; g < NG; g++)
#pragma unroll
            for (int i = 0; i < C::PIECES / 2; i++) {
              const int e = i * 32 + lane;  // piece of the group
              uint4* at = reinterpret_cast<uint4*>(vp + g * 16 * D + e * 16);
              const uint4 v = *at;
              const uint4 n4 = make_uint4(nan_bytes(v.x), nan_bytes(v.y), nan_bytes(v.z), nan_bytes(v.w));
              if (n4.x | n4.y | n4.z | n4.w) {
                *at = make_uint4(v.x & ~n4.x, v.y & ~n4.y, v.z & ~n4.z, v.w & ~n4.w);
                if (ks[g] > 0.f) poison |= 1u << (g * 16 + e / C::PIECES);
              }
            }
          poison = __reduce_or_sync(~0u, poison);
          fence_proxy_async_smem();
          __syncwarp();
        }
        float lv[NG], wl[NG], kc[NG];
#pragma unroll
        for (int g = 0; g < NG; g++) {
          lv[g] = log2_scale(SHARED ? ks[g] : s_scale[st * 8 + 4 + (rows0 >> 4) + g]);
          if (ks[g] > 0.f) lvref = fmaxf(lvref, lv[g]);
          kc[g] = fmaxf(ks[g], SCALE_MIN) * p.scale2;
        }
#pragma unroll
        for (int g = 0; g < NG; g++) {
          lv[g] = ks[g] > 0.f ? fmaxf(lv[g], lvref - LV_SPAN) : lvref;
          wl[g] = ks[g] > 0.f ? ex2_ftz(lvref - lv[g]) : 0.f;
        }
        float al[2];
        uint32_t pf[NG][4];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float c[NG], mz = -INFINITY, mw = -INFINITY;  // largest z2, largest z2 + lv
#pragma unroll
          for (int g = 0; g < NG; g++) {
            c[g] = fmaxf(kc[g] * back[h], SCALE_MIN);
            const float x = fmax3(fmaxf(z[g][h][0], z[g][h][1]), z[g][h][2], z[g][h][3]) * c[g];
            mz = fmaxf(mz, x);
            mw = fmaxf(mw, x + lv[g]);
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            mz = fmaxf(mz, __shfl_xor_sync(~0u, mz, o));
            mw = fmaxf(mw, __shfl_xor_sync(~0u, mw, o));
          }
          const float m2 = fmaxf(m[h], mz);
          l[h] *= m[h] == m2 ? 1.f : ex2_ftz(m[h] - m2);
          m[h] = m2;
          const float M2 = mw > M[h] + P_LAZY ? mw : M[h];
          al[h] = M2 == M[h] || M[h] == -INFINITY ? 1.f : ex2_ftz(M[h] - M2);
          M[h] = M2;
          // rows without a reference yet have seen nothing: their z are all -inf
          const float Mu = M2 == -INFINITY ? 0.f : M2, mu = m2 == -INFINITY ? 0.f : m2;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < NG; g++) {
            float e[4];
#pragma unroll
            for (int k = 0; k < 4; k++) e[k] = ex2_ftz(fmaf(z[g][h][k], c[g], lv[g] - Mu + P_OFF));
            sum = fmaf((e[0] + e[1]) + (e[2] + e[3]), wl[g], sum);
            pf[g][h] = half2_of(e[0], e[1]);
            pf[g][2 + h] = half2_of(e[2], e[3]);
          }
          l[h] = fmaf(sum, lvref == -INFINITY ? 0.f : ex2_ftz(Mu - P_OFF - lvref - mu), l[h]);
          for (uint32_t b = poison; b; b &= b - 1) {
            const int j = j0 + __ffs(b) - 1;
            if (j >= lo_r[h] && j < hi_r[h]) l[h] = NAN;
          }
        }
        if (__any_sync(~0u, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int c = 0; c < C::PIECES; c++)
#pragma unroll
            for (int k = 0; k < 8; k++) o[c][k] *= al[k >> 2];
        }
        // O += P V: pieces c, c + 1 per ldmatrix
#pragma unroll
        for (int c = 0; c < C::PIECES; c += 2)
#pragma unroll
          for (int g = 0; g < NG; g++) {
            uint32_t r[4];
            ldsm4t(vb + piece<D>(g * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, c + (lane >> 4)), r);
#pragma unroll
            for (int u = 0; u < 2; u++) {
              // bytes (row 2t dim 2n, row 2t dim 2n+1, row 2t+1 dim 2n, row 2t+1 dim 2n+1)
              const uint32_t x0 = __byte_perm(r[2 * u], 0, 0x3120), x1 = __byte_perm(r[2 * u + 1], 0, 0x3120);
              float ev[4] = {o[c + u][0], o[c + u][2], o[c + u][4], o[c + u][6]};
              float od[4] = {o[c + u][1], o[c + u][3], o[c + u][5], o[c + u][7]};
              mma16816(ev, pf[g], half2_of_codes(uint16_t(x0)), half2_of_codes(uint16_t(x1)));
              mma16816(od, pf[g], half2_of_codes(uint16_t(x0 >> 16)), half2_of_codes(uint16_t(x1 >> 16)));
              o[c + u][0] = ev[0]; o[c + u][2] = ev[1]; o[c + u][4] = ev[2]; o[c + u][6] = ev[3];
              o[c + u][1] = od[0]; o[c + u][3] = od[1]; o[c + u][5] = od[2]; o[c + u][7] = od[3];
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
    // join the warps: l's partial sums lie over the four threads of a row
#pragma unroll
    for (int h = 0; h < 2; h++) {
      l[h] += __shfl_xor_sync(~0u, l[h], 1);
      l[h] += __shfl_xor_sync(~0u, l[h], 2);
      if (t4 == 0) {
        float* s3 = s_stat + (warp * 16 + r0 + 8 * h) * 3;
        s3[0] = m[h]; s3[1] = M[h]; s3[2] = l[h];
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
    float mt[2], Mt[2], lt[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      mt[h] = Mt[h] = -INFINITY;
      lt[h] = 0.f;
#pragma unroll
      for (int v = 0; v < NW; v++) {
        const float* s3 = s_stat + (v * 16 + r0 + 8 * h) * 3;
        mt[h] = fmaxf(mt[h], s3[0]);
        Mt[h] = fmaxf(Mt[h], s3[1]);
      }
#pragma unroll
      for (int v = 0; v < NW; v++) {
        const float* s3 = s_stat + (v * 16 + r0 + 8 * h) * 3;
        lt[h] += s3[0] == -INFINITY ? s3[2] : s3[2] * ex2_ftz(s3[0] - mt[h]);
      }
      const float f = M[h] == -INFINITY ? 0.f : ex2_ftz(M[h] - Mt[h]);
      if (f != 1.f) {
#pragma unroll
        for (int c = 0; c < C::PIECES; c++)
#pragma unroll
          for (int k = 0; k < 4; k++) o[c][4 * h + k] = f == 0.f ? 0.f : o[c][4 * h + k] * f;
      }
    }
    if (warp > 0) {
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int c = 0; c < C::PIECES; c++)
          *reinterpret_cast<float4*>(s_merge + ((warp - 1) * 16 + r0 + 8 * h) * D + ((c ^ (r0 & 7)) & (C::PIECES - 1)) * 16 + t4 * 4) =
              make_float4(o[c][4 * h], o[c][4 * h + 1], o[c][4 * h + 2], o[c][4 * h + 3]);
    }
    // (a warp whose wait ran out ends the block here, at the same item for all four)
    uint32_t gone;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(gone) : "r"(uint32_t(!ok)), "n"(NW * 32) : "memory");
    if (gone) break;
    if (warp == 0) {
      const bool whole = w.count == w.nt;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int row = r0 + 8 * h;
        const bool valid = row < nrows;
        const int i = valid ? p.by_G.div(row) : 0, head = w.g * p.G + (valid ? row - i * p.G : 0);
        const size_t orow = (size_t)(w.r.c0 + i) * p.a.H + head;
        float f = 1.f, lse = 0.f;
        float* pp = p.part + (2 * (size_t)blockIdx.x + (w.tile == 0 ? 1 : 0)) * part_floats(ROWS_SMALL, D);
        if (whole) {
          const float sink2 = p.a.sink && valid ? p.a.sink[head] * LOG2E : -INFINITY;
          f = finish_row(mt[h], Mt[h], lt[h], sink2, &lse);
        } else if (t4 == 0) {
          *reinterpret_cast<float4*>(pp + row * 4) = make_float4(mt[h], Mt[h], lt[h], 0.f);
        }
#pragma unroll
        for (int c = 0; c < C::PIECES; c++) {
          float4 a = make_float4(o[c][4 * h], o[c][4 * h + 1], o[c][4 * h + 2], o[c][4 * h + 3]);
#pragma unroll
          for (int v = 0; v < NW - 1; v++) {
            const float4 x = *reinterpret_cast<const float4*>(s_merge + (v * 16 + row) * D + ((c ^ (r0 & 7)) & (C::PIECES - 1)) * 16 + t4 * 4);
            a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
          }
          if (whole) {
            if (valid)
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.out) + orow * D + c * 16 + t4 * 4) =
                  f == 0.f ? make_uint2(0, 0)
                           : make_uint2(bf16x2_of(a.x * f, a.y * f), bf16x2_of(a.z * f, a.w * f));
          } else {
            *reinterpret_cast<float4*>(pp + 64 + row * D + c * 16 + t4 * 4) = a;
          }
        }
        if (whole && valid && t4 == 0 && p.a.lse) p.a.lse[orow] = lse;
      }
    }
  } while (walk_next(p, w));
}

template <int D, bool SHARED>
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
  auto kern = paged_rows_kernel<D, SHARED>;
  const int smem = (int)Cfg<D, SHARED>::TOTAL + 1024;
  static_assert(2 * (Cfg<D, SHARED>::TOTAL + 2048) <= 233472, "two blocks per SM");
  e = set_kernel_attrs(reinterpret_cast<const void*>(kern), smem, false);
  if (e != HCL_OK) return e;
  return check_cuda(launch_pdl(kern, dim3(p.n_blocks), dim3(THREADS), (size_t)smem, st, 1, p, tk, tv),
                    "paged attention (rows) launch");
}

}  // namespace

int rows_blocks() { return std::min(1024, 2 * num_sms()); }

hcl_status_t launch_rows(const Params& p, cudaStream_t st) {
  if (p.a.kv.d == 128) return p.a.kv.v ? launch_t<128, false>(p, st) : launch_t<128, true>(p, st);
  return p.a.kv.v ? launch_t<64, false>(p, st) : launch_t<64, true>(p, st);
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

// paged_tile.cu -- paged attention for requests with many query rows (queries x heads of one KV
// head > 16): prompts, chunks, and decode with many heads on one KV head.  tcgen05 tensor cores.
//
// One persistent block per SM.  An item is 256 query rows (two tiles of 128, the M of an MMA) of
// one request and KV head; a round is 64 KV rows.  Roles:
//   warps 0-3 / 4-7   softmax of tile 0 / 1: one thread per query row; they also write the output
//   warps 12, 15      issue the MMAs of tile 0, 1.  (The tensor pipe takes hardly more than the
//                     MMA it works on, so what one issuer spends on its barriers must pass under
//                     the other's MMAs.)  Each tile has two score buffers: S(r+1) is
//                     issued before PV(r), the first of an item before the item ahead has written
//                     its output, so a softmax group finds its next scores ready and
//                     waits for MMAs only where O has to be rescaled.  (With one buffer and
//                     rounds of 128, the chain softmax -> PV -> S -> softmax took 6100 clocks a
//                     round of which the tensor cores worked 2050.)
//   warp 13           one thread walks the block's items and describes them, up to four ahead
//   warp 14           loads: TMA boxes of E4M3 codes (a page, or 64 rows of a longer one) into
//                     a ring of staging units of 64 rows, and the round's page parameters
//   warps 8-11        widening: codes from the staging ring to fp16 tiles, 128-byte swizzle.
//                     The same layout serves K (K-major B operand of S = Q K^T) and V (MN-major
//                     B operand of O += P V); rows that are both key and value are widened once.
//                     (Loading the codes straight into the widening threads' registers spent
//                     more issue slots on addresses than on the conversion.)  They also bring an
//                     item's Q, under the last rounds of the item before it.  (By the softmax
//                     groups, between two items: 5000 to 8000 clocks in which no MMA ran.)
// P (fp16) is written over the first half of its S in tensor memory and read there as the A
// operand.  TMEM: S_0 / P_0 and S_1 / P_1 (two buffers of 64 columns each), O_0, O_1.
// An item of at most 128 rows (decode over many heads, a request's last rows) runs in single
// mode: both softmax groups work on the same rows, group t on the rounds of parity t with its
// own O, and join at the end, each reading both O's, so the pipeline keeps its two streams.
//
// Bound by the latency of a round's softmax: a warp takes 2400 clocks for its 64 columns (340 to
// find the scores, 500 to load them, 550 for the maximum, 850 to 1250 for the exponentials, the
// more where both groups' fall together), with 1300 of MMAs and 1024 of exponentials (256 x 64 at
// 16 a clock) under it.  Measured and left: exponentials against the old reference while the
// maximum is formed (chunk of 2048 on 65536: 1151 -> 1136 us, but prompts 589 -> 613), turns
// between the groups (prompts 589 -> 710), scores read twice in rolled halves (chunk 1285), rings
// of 4 or 2 tiles, two or four staging units (the same within 1 %).  Code that runs once an item
// is kept in loops: unrolled it waited for instructions (prompts 622 -> 588 us).
//   decode, 8 x 128 K rows x 128 heads on one KV head: 77 us (27 at the MMA rate)
//   chunk of 2048 x 16 heads on 65536 rows: 1160 us (653);  prompts, 4 x 4096 x 32 heads: 585 us (206)
#include <algorithm>

#include "paged_common.cuh"

namespace hcl {
namespace paged {
namespace {

constexpr float P_OFF = P_OFF_TILE, P_LAZY = 15.f - P_OFF;
constexpr int TILE = 64;       // KV rows per round
constexpr int ITEM = ROWS_ITEM;  // query rows per item
constexpr int THREADS = 16 * 32;
// What an item costs beyond its rounds (pipeline fill, output), in rounds: the blocks' shares count
// it, or those of a prompt's first tiles (few rounds, many items) take twice as long.  (Prompts of
// 4 x 4096 x 32 heads: 624 us with 5, 592 with 8, 579 with 11, 585 with 13, 642 with 16; chunks in a
// window of 128: 53 us with all of them.)
constexpr int ITEM_COST = 11;
constexpr int PRING = 16;      // rounds whose page parameters are kept
constexpr uint32_t O_COL = 256;

struct RoundPar {              // what the softmax needs of a round's pages (groups of 16 rows)
  float kc[4], lv[4], wl[4];   // scale2 * k_scale, log2(v_scale) not below lvref - LV_SPAN, 2^(lvref - lv)
  float lvg[4];                // log2(v_scale)
  uint32_t poison[4];          // edge rounds: rows with a NaN value, by widening warp (see look())
  uint32_t valid[2];           // rows whose page is in the cache
  float lvref, top;            // largest log2(v_scale) from the part's first round on, of this round
  uint32_t edge;               // some query row of the item does not see the round whole
  uint32_t pad[3];
};
static_assert(sizeof(RoundPar) % 16 == 0, "RoundPar");

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
// The MMA warp runs as one: all lanes take the same path (so that descriptors and addresses stay
// in uniform registers) and `lead`, true in one lane, predicates each instruction.  Issued from
// inside a one-lane branch the same MMAs took 75 to 108 clocks each, with 48 to 64 of work.
// Descriptors are given by their low words; the high words (swizzle, stride) are constants.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (SMEM_SWIZZLE_128B << 29);
// D (+)= A B, both from shared memory.
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                        uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(lead), "n"(DESC_HI)
      : "memory");
}
// D (+)= A B with A (packed fp16 pairs) read from tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                        uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(lead), "n"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void commit_lead(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// Barrier `id` over n threads; returns whether any of them passed true.
__device__ __forceinline__ bool bar_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(uint32_t(x)), "r"(id), "r"(n) : "memory");
  return r != 0;
}
// bits j with lo <= c0 + j < hi
__device__ __forceinline__ uint32_t range_mask(int c0, int lo, int hi) {
  const int a = max(lo - c0, 0), b = min(hi - c0, 32);
  if (a >= b) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// ---- the items -----------------------------------------------------------------------------

__device__ __forceinline__ int tiles_of(const Params& p, const Req& r) {
  const int rows = r.nq * p.G;
  return rows <= ROWS_SMALL ? 0 : (rows + ITEM - 1) / ITEM;
}
// Rounds of a tile: first KV row (a multiple of TILE) and how many (at least one).
__device__ __forceinline__ int rounds_of(const Params& p, const Req& r, int tile, int* j0) {
  const int i0 = p.by_G.div(tile * ITEM), i1 = p.by_G.div(min(r.nq * p.G, (tile + 1) * ITEM) - 1);
  const int hi = vis_hi(p, r, i1), lo = min(vis_lo(p, r, i0), hi);
  *j0 = 0;
  if (hi <= lo) return 1;
  *j0 = lo / TILE * TILE;
  return (hi - *j0 + TILE - 1) / TILE;
}

// Items in order: request, tile, KV head.
struct Walk {
  Req r;
  int b, g, tile, j0, nt;  // request, KV head, tile; its first KV row and rounds
  int rd, count;           // this block's rounds of the item: rd .. rd + count - 1 of nt
  long long left;
};
// The units of an item are ITEM_COST + rounds; `at`: this block's first of them.
__device__ __forceinline__ void walk_set(Walk& w, int at) {
  const int n = (int)min((long long)(ITEM_COST + w.nt - at), w.left);  // this block's units
  w.rd = max(0, at - ITEM_COST);
  w.count = max(0, at + n - ITEM_COST) - w.rd;
  w.left -= n;
}
__device__ __forceinline__ bool walk_first(const Params& p, const Share& s, int b, int tile, Walk& w) {
  w.left = s.u1 - s.u0;
  if (w.left <= 0) return false;
  w.b = b;
  w.tile = tile;
  w.r = load_req(p, b, false);
  w.nt = rounds_of(p, w.r, tile, &w.j0);
  w.g = (int)(s.rem / (ITEM_COST + w.nt));
  walk_set(w, (int)(s.rem % (ITEM_COST + w.nt)));
  return true;
}
__device__ __forceinline__ bool walk_next(const Params& p, Walk& w) {
  if (w.left <= 0) return false;
  if (++w.g == p.a.kv.Hkv) {
    w.g = 0;
    if (++w.tile == tiles_of(p, w.r)) {
      w.tile = 0;
      do w.r = load_req(p, ++w.b, false);
      while (tiles_of(p, w.r) == 0);
    }
    w.nt = rounds_of(p, w.r, w.tile, &w.j0);
  }
  walk_set(w, 0);
  return true;
}
// What the roles are told of an item, in shared memory, written by the walking warp.
struct Item {
  int count;               // rounds of this block's part; 0: no item more
  int rows;                // query rows (> 128: both tiles)
  int j0;                  // first KV row of the part
  int b, g;                // request, KV head
  int row0, c0;            // first query row within the request, the request's first row of q
  int qs, len;             // position of its first query, rows held
  int any_hi, all_lo, all_hi;  // some row sees KV rows below any_hi; all see [all_lo, all_hi)
  int whole, head;         // not split; the part begins inside the item (an earlier block has its front)
  int pad[2];
};
constexpr int IRING = 4;

template <int D, bool SHARED>
struct Cfg {
  static constexpr int PIECES = D / 16;               // 16-code pieces of a row
  static constexpr int RPP = 128 / PIECES;            // rows per pass of the widening threads
  static constexpr int RPW = RPP / 4;                 // of which each of their warps has RPW
  static constexpr int NU = 3;                        // staging units (a plane of a round each)
  static constexpr uint32_t QT = 128 * D * 2;         // bytes of a Q tile
  static constexpr uint32_t KT = TILE * D * 2;        // bytes of a K or V tile
  static constexpr uint32_t HALF = TILE * 128;        // its two halves of 64 dimensions
  static constexpr int NK = SHARED ? 6 : 3;           // K (or shared) tiles in the ring
  static constexpr int NV = NK;
  static constexpr uint32_t K = 2 * QT;
  static constexpr uint32_t V = SHARED ? K : K + NK * KT;
  static constexpr uint32_t STAGE = K + 6 * KT;
  static constexpr uint32_t OUT = STAGE + NU * TILE * D;              // [8 warps][32 rows][128 bytes]
  static constexpr uint32_t PAR = OUT + 8 * 4096;
  static constexpr uint32_t STAT = PAR + PRING * sizeof(RoundPar);    // [2][128][4] floats (single mode)
  static constexpr uint32_t BACK = STAT + 2 * 128 * 16;               // [ITEM] floats: the query rows' factors
  static constexpr uint32_t ITEMS = BACK + ITEM * 4;
  static constexpr uint32_t BAR = ITEMS + IRING * sizeof(Item);
  static constexpr int NBAR = 2 * NK + 2 * NV + 3 * 4 + 2 + 1 + 2 * IRING + 2 * NU;
  static constexpr uint32_t SCRATCH = BAR + NBAR * 8;
  static constexpr uint32_t MISC = SCRATCH + (16 + 4) * 8;
  static constexpr uint32_t TOTAL = MISC + 16;
};

template <int D, bool SHARED>
__global__ void __launch_bounds__(THREADS, 1)
    paged_tile_kernel(const Params p, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using C = Cfg<D, SHARED>;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);  // (an offset: the compiler still sees shared memory)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  RoundPar* par = reinterpret_cast<RoundPar*>(sm + C::PAR);
  // A wait names a phase by its parity, so every waiter of a barrier follows it phase by phase, or
  // knows by other means that the phase before the wanted one has completed and the one after it
  // cannot: hence a barrier for each buffer.
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + C::BAR);
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* v_full = k_empty + C::NK;
  uint64_t* v_empty = v_full + C::NV;
  uint64_t* s_full = v_empty + C::NV;        // [tile][buffer] S of a step in TMEM
  uint64_t* p_full = s_full + 4;             // [tile][buffer] P in TMEM, O rescaled
  uint64_t* o_done = s_full + 8;             // [tile][buffer] PV of a step completed
  uint64_t* q_full = s_full + 12;            // the item's Q tiles and their factors stand
  uint64_t* q_empty = s_full + 13;           // its scores are all computed, its factors read
  uint64_t* drain = s_full + 14;
  uint64_t* i_full = s_full + 15;            // [IRING] an item's description stands
  uint64_t* i_empty = i_full + IRING;        // [IRING] every role is done with it
  uint64_t* u_full = i_empty + IRING;        // [NU] a staging unit's codes landed, its round's parameters stand
  uint64_t* u_empty = u_full + C::NU;        // [NU] the widening warps have read it
  Item* items = reinterpret_cast<Item*>(sm + C::ITEMS);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + C::MISC);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + C::MISC + 4);
  if (tid == 0) {
    for (int i = 0; i < C::NK; i++) { mbar_init(&k_full[i], 128); mbar_init(&k_empty[i], 2); }
    for (int i = 0; i < C::NV; i++) { mbar_init(&v_full[i], 128); mbar_init(&v_empty[i], 2); }
    for (int i = 0; i < 4; i++) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 128); mbar_init(&o_done[i], 1); }
    mbar_init(q_full, 128);
    mbar_init(q_empty, 2 + 8);
    mbar_init(drain, 2);
    for (int i = 0; i < IRING; i++) { mbar_init(&i_full[i], 1); mbar_init(&i_empty[i], 4 + 8 + 2 + 1); }
    for (int i = 0; i < C::NU; i++) { mbar_init(&u_full[i], 1); mbar_init(&u_empty[i], 4); }
    *s_abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tk);
    if (!SHARED) prefetch_tmap(&tv);
  }
  if (warp == 12) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  pdl_enter();
  tc_fence_before();
  // Units are rounds and ITEM_COST an item; the entries that share them are all tiles of all requests, so that no
  // thread has a long prompt to itself.  s_first (in memory that Q will take): each request's
  // first tile.
  long long* scratch = reinterpret_cast<long long*>(sm + C::SCRATCH);
  int* s_first = reinterpret_cast<int*>(sm);
  const int per = (p.a.B + THREADS - 1) / THREADS;
  const int b_lo = min(p.a.B, tid * per), b_hi = min(p.a.B, b_lo + per);
  long long tiles = 0, all_tiles;
  for (int b = b_lo; b < b_hi; b++) tiles += tiles_of(p, load_req(p, b, blockIdx.x == 0));
  tiles = block_prefix<THREADS>(tiles, scratch, &all_tiles);
  for (int b = b_lo; b < b_hi; b++) {
    s_first[b] = (int)tiles;
    tiles += tiles_of(p, load_req(p, b, false));
  }
  __syncthreads();
  int at_b = -1, at_end = 0;  // the request of the thread's current tile, and the tile after its last
  Req at_r = {};
  auto tile_at = [&](int e) {  // request of tile e
    if (at_b < 0 || e >= at_end || e < s_first[at_b]) {
      int lo = 0, hi = p.a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_first[mid] <= e) lo = mid;
        else hi = mid;
      }
      at_b = lo;
      at_r = load_req(p, lo, false);
      at_end = s_first[lo] + tiles_of(p, at_r);
    }
    return at_b;
  };
  const Share share = find_share<THREADS>((int)all_tiles, blockIdx.x, p.n_blocks, scratch, [&](int e) {
    int j0;
    tile_at(e);
    return (long long)(ITEM_COST + rounds_of(p, at_r, e - s_first[at_b], &j0)) * p.a.kv.Hkv;
  });
  at_b = -1;
  const int b0 = share.u1 > share.u0 ? tile_at(share.e) : 0;
  const int tile0 = share.u1 > share.u0 ? share.e - s_first[b0] : 0;
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *s_tmem;
  const bool any = share.u1 > share.u0;
  if (!any && tid == 0) p.meta[blockIdx.x].ends = 0;

  // registers of the four warpgroups: 176 + 176 + 64 + 96 = 4 * 128
  if (any && warp >= 8 && warp < 12) {
    // ------------------------------------------------------------------ widening
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int ww = warp - 8, pc = lane % C::PIECES, pr = lane / C::PIECES;
    // this thread's place in a pass of a staging unit and of a tile; the two 64-dimension halves
    // take a piece's two 16-byte parts in opposite order: no bank conflict
    const int row0 = ww * C::RPW + pr;
    const uint32_t src0 = C::STAGE + row0 * D + pc * 16;
    const int c0 = (pc & 3) * 2, sw = row0 & 7;  // (RPP is a multiple of 8: every pass has the same row & 7)
    const uint32_t dst0 = (pc >> 2) * C::HALF + row0 * 128;
    const uint32_t first = dst0 + (((pc & 4 ? c0 + 1 : c0) ^ sw) << 4), second = dst0 + (((pc & 4 ? c0 : c0 + 1) ^ sw) << 4);
    bool ok = true;
    uint32_t rg = 0, u = 0;  // rounds, staging units so far
    // Q rows of an item, bf16, to their places in the Q tiles (rows behind the last: zeros)
    auto load_q = [&](const Item* im) {
      constexpr int LPR = D / 8, STEP = 128 / LPR;  // 16-byte pieces of a row, rows a pass (a multiple of 8)
      const int rows = im->rows, w0 = tid - 256, pq = w0 % LPR, r0 = w0 / LPR;
      const int qr = im->row0 + r0, qi = p.by_G.div(qr), dq = p.by_G.div(STEP), dh = STEP - dq * p.G;
      int h = qr - qi * p.G;  // the row's query moves by dq (+ 1), its head by dh (- G)
      const char* src = static_cast<const char*>(p.a.q) +
                        2 * ((im->c0 + qi) * p.a.q_stride + (im->g * p.G + h) * D + pq * 8);
      const int64_t step = 2 * (dq * p.a.q_stride + dh * D), wrap = 2 * (p.a.q_stride - p.G * D);
      uint32_t dst = smem_u32(sm) + (pq >> 3) * 16384 + r0 * 128 + (((pq & 7) ^ (r0 & 7)) << 4);
      for (int t = 0; t * 128 < rows; t++, dst += C::QT - 16384) {
#pragma unroll 4
        for (int k = 0; k < LPR; k++, dst += STEP * 128) {
          const bool in = t * 128 + k * STEP + r0 < rows;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(in ? src : p.a.q), "r"(in ? 16 : 0)
                       : "memory");
          src += step;
          h += dh;
          if (h >= p.G) {
            h -= p.G;
            src += wrap;
          }
        }
      }
    };
    // this thread's row of Q tile t to fp16 with its exponent taken out
    auto convert_q = [&](int t) {
      const int r = tid - 256;
      uint8_t* qrow = sm + t * C::QT + r * 128;
      auto at = [&](int e) { return reinterpret_cast<uint4*>(qrow + (e >> 3) * 16384 + (((e & 7) ^ (r & 7)) << 4)); };
      uint32_t top = 0;  // (of magnitudes, whose bits order as their values do; NaN above all)
#pragma unroll
      for (int e = 0; e < D / 8; e++) {
        const uint4 x = *at(e);
        top = __vmaxu2(__vmaxu2(top, __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu)),
                       __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
      }
      float back;
      const float f = row_factor(__uint_as_float(max(top & 0xFFFFu, top >> 16) << 16), &back);
      reinterpret_cast<float*>(sm + C::BACK)[t * 128 + r] = back;
#pragma unroll 1
      for (int e = 0; e < D / 8; e += 4) {
        uint4 x[4];
#pragma unroll
        for (int u = 0; u < 4; u++) x[u] = *at(e + u);
#pragma unroll
        for (int u = 0; u < 4; u++) {
          uint32_t a[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
          for (int k = 0; k < 4; k++)
            a[k] = half2_of(__uint_as_float(a[k] << 16) * f, __uint_as_float(a[k] & 0xFFFF0000u) * f);
          *at(e + u) = make_uint4(a[0], a[1], a[2], a[3]);
        }
      }
    };
    // one staging unit into `tile`
    auto widen = [&](uint8_t* tile, RoundPar* rp, bool mark) {
      constexpr int NQ = TILE / C::RPP;
      const uint32_t su = u % C::NU;
      ok = ok && mbar_wait(&u_full[su], (u / C::NU) & 1, p.limit, s_abort);
      const bool edge = rp->edge && mark;
      uint4 x[NQ];
#pragma unroll
      for (int q = 0; q < NQ; q++)
        x[q] = *reinterpret_cast<const uint4*>(sm + src0 + su * (TILE * D) + q * C::RPP * D);
      if (edge) {
        // Not every query row sees the whole round: NaN codes become 0 (0 * NaN would reach rows
        // that do not see them; rows behind the last hold anything) and are noted for the softmax
        uint32_t bad = 0;
#pragma unroll
        for (int q = 0; q < NQ; q++) {
          const uint4 n4 = make_uint4(nan_bytes(x[q].x), nan_bytes(x[q].y), nan_bytes(x[q].z), nan_bytes(x[q].w));
          const bool n = (n4.x | n4.y | n4.z | n4.w) != 0;
          if (n) x[q] = make_uint4(x[q].x & ~n4.x, x[q].y & ~n4.y, x[q].z & ~n4.z, x[q].w & ~n4.w);
          const uint32_t who = __ballot_sync(~0u, n);
#pragma unroll
          for (int r = 0; r < C::RPW; r++)
            if ((who >> (r * C::PIECES)) & ((1u << C::PIECES) - 1u)) bad |= 1u << (q * C::RPW + r);
        }
        if (lane == 0) rp->poison[ww] = bad;
      }
#pragma unroll
      for (int q = 0; q < NQ; q++) {
        const uint4 lo = make_uint4(half2_of_codes(uint16_t(x[q].x)), half2_of_codes(uint16_t(x[q].x >> 16)),
                                    half2_of_codes(uint16_t(x[q].y)), half2_of_codes(uint16_t(x[q].y >> 16)));
        const uint4 hi = make_uint4(half2_of_codes(uint16_t(x[q].z)), half2_of_codes(uint16_t(x[q].z >> 16)),
                                    half2_of_codes(uint16_t(x[q].w)), half2_of_codes(uint16_t(x[q].w >> 16)));
        *reinterpret_cast<uint4*>(tile + first + q * C::RPP * 128) = pc & 4 ? hi : lo;
        *reinterpret_cast<uint4*>(tile + second + q * C::RPP * 128) = pc & 4 ? lo : hi;
      }
      fence_proxy_async_smem();
      // The unit is released only behind the stores that needed its values: a load that was issued
      // before an arrival may still read after it, and find the next unit's bytes.
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[su]);
      u++;
    };
    for (uint32_t it = 0;; it++) {
      ok = ok && mbar_wait(&i_full[it % IRING], (it / IRING) & 1, p.limit, s_abort);
      ok = !bar_or(2, 128, !ok);  // the four warps go on, or end, together
      const Item* im = items + it % IRING;
      const int count = ok ? im->count : 0;
      if (count == 0) break;
      // The item's Q rows go to shared memory as they are, while its first round is widened, and
      // are turned to fp16 in place.
      if (it > 0) ok = mbar_wait(q_empty, (it - 1) & 1, p.limit, s_abort);
      ok = !bar_or(2, 128, !ok);
      if (!ok) break;
      const int rows = im->rows, qtiles = rows > 128 ? 2 : 1;
      load_q(im);
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[it % IRING]);
      for (int i = 0; i < count && ok; i++, rg++) {
        RoundPar* rp = par + rg % PRING;
        const uint32_t kb = rg % C::NK;
        if (rg >= C::NK) ok = mbar_wait(&(SHARED ? v_empty : k_empty)[kb], ((rg / C::NK) & 1) ^ 1, p.limit, s_abort);
        widen(sm + C::K + kb * C::KT, rp, SHARED);
        mbar_arrive(&k_full[kb]);
        if constexpr (!SHARED) {
          const uint32_t vb = rg % C::NV;
          if (rg >= C::NV) ok = ok && mbar_wait(&v_empty[vb], ((rg / C::NV) & 1) ^ 1, p.limit, s_abort);
          widen(sm + C::V + vb * C::KT, rp, true);
          mbar_arrive(&v_full[vb]);
        }
        if (i == 0) {  // (all four warps come here, whatever their waits said)
          asm volatile("cp.async.wait_all;" ::: "memory");
          asm volatile("bar.sync 5, 128;" ::: "memory");
#pragma unroll 1
          for (int t = 0; t < qtiles; t++) convert_q(t);
          fence_proxy_async_smem();
          mbar_arrive(q_full);
        }
      }
    }
    if (!ok) {
      *s_abort = 1;
      if (lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
    }
  } else if (any && warp >= 12) {
    // ------------------------------------------------------------------ MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 12 || warp == 15) {
      const int t = warp == 15;  // the tile
      const uint32_t lead = lane == 0;
      const uint32_t tb = __shfl_sync(~0u, tbase, 0) + t * 128;
      const uint32_t sbase = smem_u32(sm);
      const uint32_t dq = ((sbase & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t dk = (((sbase + C::K) & 0x3FFFFu) >> 4) | (1u << 16);
      const uint32_t dv = (((sbase + C::V) & 0x3FFFFu) >> 4) | ((C::HALF >> 4) << 16);
      constexpr uint32_t idS = idesc_f16(128, TILE), idPV = idesc_f16(128, D) | (1u << 16);
      // rg: rounds before this item; n: this tile's steps before this one
      uint32_t rg = 0, n = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity, p.limit, s_abort); };
      // Both issuers release a K or V tile; where one of them alone uses it, it does so twice.
      auto release = [&](uint64_t* bar, bool alone) {
        commit_lead(bar, lead);
        if (alone) commit_lead(bar, lead);
      };
      // scores of round R, this tile's step s, with the Q tile at aq; `last` of the item.  They go
      // where P of the step before the last was: its PV must have completed.
      auto issue_s = [&](uint32_t R, uint32_t s, uint32_t aq, bool alone, bool last) {
        const uint32_t kb = R % C::NK;
        if (s > 1) wait(&o_done[2 * t + (s & 1)], ((s - 2) >> 1) & 1);
        wait(&k_full[kb], (R / C::NK) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint32_t b0 = dk + kb * (C::KT >> 4), d = tb + (s & 1) * TILE;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks++)
          umma_ss(d, aq + ((ks >> 2) * (16384 >> 4) + (ks & 3) * 2), b0 + ((ks >> 2) * (C::HALF >> 4) + (ks & 3) * 2), idS,
                  ks > 0 ? 1u : 0u, lead);
        commit_lead(&s_full[2 * t + (s & 1)], lead);
        if (last) commit_lead(q_empty, lead);
        if (!SHARED) release(&k_empty[kb], alone);
      };
      for (uint32_t it = 0;; it++) {
        wait(&i_full[it % IRING], (it / IRING) & 1);
        ok = __all_sync(~0u, ok);
        const int count = ok ? __shfl_sync(~0u, items[it % IRING].count, 0) : 0;
        if (count == 0) break;
        const bool pair = __shfl_sync(~0u, items[it % IRING].rows, 0) > 128;
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[it % IRING]);
        // this tile's step k is round k (pair) or 2k + t (single)
        const int steps = pair ? count : (count + 1 - t) / 2;
        const uint32_t aq = pair && t ? dq + (C::QT >> 4) : dq, stride = pair ? 1 : 2;
        wait(q_full, it & 1);
        uint32_t R = rg + (pair ? 0 : t);
        if (steps > 0) issue_s(R, n, aq, !pair, steps == 1);
        else if (lane == 0) mbar_arrive(q_empty);
        for (int k = 0; k < steps && ok; k++, R += stride, n++) {
          if (k + 1 < steps) issue_s(R + stride, n + 1, aq, !pair, k + 2 == steps);
          const uint32_t vb = R % C::NV;
          if (!SHARED) wait(&v_full[vb], (R / C::NV) & 1);
          wait(&p_full[2 * t + (n & 1)], (n >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t b0 = dv + vb * (C::KT >> 4), a0 = tb + (n & 1) * TILE;
#pragma unroll
          for (int ks = 0; ks < TILE / 16; ks++)
            umma_ts(tb + O_COL, a0 + ks * 8, b0 + ks * (2048 >> 4), idPV, ks > 0 || k > 0 ? 1u : 0u, lead);
          commit_lead(&o_done[2 * t + (n & 1)], lead);
          release(&v_empty[vb], !pair);
        }
        rg += count;
      }
      if (!ok) {
        *s_abort = 1;
        if (lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
      }
      // every MMA issued has completed before TMEM may be freed
      commit_lead(drain, lead);
      if (!mbar_wait(drain, 0, p.limit, nullptr) && lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
      __syncwarp();
    }
    if (warp == 14) {
      // ---------------------------------------------------------------- loads
      const int box = min(p.a.kv.page, TILE), pmask = p.a.kv.page - 1, gr = lane & 3;
      const bool begins = lane < 4 && (gr & (box / 16 - 1)) == 0;  // this lane's 16-row group begins a box
      bool ok = true, fault = false;
      uint32_t rg = 0, u = 0;
      for (uint32_t it = 0; ok; it++) {
        ok = __all_sync(~0u, mbar_wait(&i_full[it % IRING], (it / IRING) & 1, p.limit, s_abort));
        const Item im = items[it % IRING];
        if (!ok || im.count == 0) break;
        const int32_t* trow = p.a.table + (size_t)im.b * p.a.max_pages;
        // the page of this lane's group in round i: -2 where no row is wanted
        auto page_at = [&](int i) {
          const int j = im.j0 + i * TILE + gr * 16;
          return i < im.count && j < im.any_hi ? __ldg(trow + (j >> p.sh)) : -2;
        };
        auto good_page = [&](int id) { return (uint32_t)id < (uint32_t)p.a.kv.n_pages; };
        auto scales = [&](int id, float* ks, float* vs) {
          *ks = *vs = 1.f;
          if (good_page(id)) {
            const size_t pg = (size_t)id * p.a.kv.Hkv + im.g;
            *ks = __ldg(p.a.kv.k_scale + pg);
            *vs = SHARED ? *ks : __ldg(p.a.kv.v_scale + pg);
          }
        };
        float lvref = -INFINITY, ks, vs, ks1, vs1;
        int id = page_at(0), id1 = page_at(1);  // ids two rounds ahead, scales one
        scales(id, &ks, &vs);
        for (int i = 0; i < im.count && ok; i++, rg++) {
          const int id2 = page_at(i + 2);
          scales(id1, &ks1, &vs1);
          const bool good = good_page(id);
          fault |= !good && id != -2;
          const int j0 = im.j0 + i * TILE;
          float lv = good ? log2_scale(vs) : -INFINITY, mx = lv;
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
          lvref = fmaxf(lvref, mx);
          const uint32_t gm = __ballot_sync(~0u, good) & 0xF;
          const uint32_t boxes = __ballot_sync(~0u, good && begins);
          const int row = (int)(((long long)id * p.a.kv.Hkv + im.g) << p.sh) + ((j0 + gr * 16) & pmask);
#pragma unroll
          for (int h = 0; h < (SHARED ? 1 : 2); h++, u++) {
            const uint32_t su = u % C::NU;
            if (u >= C::NU) ok = ok && __all_sync(~0u, mbar_wait(&u_empty[su], ((u / C::NU) & 1) ^ 1, p.limit, s_abort));
            if (!ok) break;
            if (h == 0) {
              RoundPar* rp = par + rg % PRING;
              if (lane < 4) {
                rp->lvg[lane] = good ? lv : 0.f;
                lv = fmaxf(lv, lvref - LV_SPAN);
                rp->kc[lane] = good ? fmaxf(ks, SCALE_MIN) * p.scale2 : 0.f;
                rp->lv[lane] = good ? lv : 0.f;
                rp->wl[lane] = good ? ex2_ftz(lvref - lv) : 0.f;
                if (lane < 2)
                  rp->valid[lane] =
                      ((gm >> (2 * lane)) & 1 ? 0xFFFFu : 0u) | ((gm >> (2 * lane + 1)) & 1 ? 0xFFFF0000u : 0u);
                if (lane == 0) {
                  rp->lvref = lvref;
                  rp->top = mx;
                  rp->edge = j0 < im.all_lo || j0 + TILE > im.all_hi || gm != 0xF;
                }
              }
              __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(&u_full[su], __popc(boxes) * box * D);
            __syncwarp();
            if (boxes >> lane & 1)
              tma_load_2d(sm + C::STAGE + su * (TILE * D) + gr * 16 * D, h == 0 ? &tk : &tv, &u_full[su], 0, row);
          }
          id = id1; id1 = id2; ks = ks1; vs = vs1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[it % IRING]);
      }
      if (!ok) {
        *s_abort = 1;
        if (lane == 0) report(p.a.status, HCL_ERR_TIMEOUT);
      }
      if (fault) report(p.a.status, HCL_ERR_DEVICE_FAULT);
      // every copy has landed before the block's shared memory goes away
      for (uint32_t k = u > C::NU ? u - C::NU : 0; k < u; k++)
        if (!mbar_wait(&u_full[k % C::NU], (k / C::NU) & 1, p.limit, nullptr) && lane == 0)
          report(p.a.status, HCL_ERR_TIMEOUT);
    }
    if (warp == 13 && lane == 0) {
      // ---------------------------------------------------------------- the items
      Walk w;
      bool more = walk_first(p, share, b0, tile0, w), ok = true;
      Meta* m = p.meta + blockIdx.x;
      // (parts are told apart by rounds: an item's first part is with the block of its first round)
      m->ends = w.rd > 0 && w.rd + w.count == w.nt;
      m->first = share.u0 - w.rd;
      m->tot = share.tot;
      m->nb = share.nb;
      m->b = w.b;
      m->g = w.g;
      m->row0 = w.tile * ITEM;
      for (uint32_t it = 0; ok; it++) {
        if (it >= IRING) ok = mbar_wait(&i_empty[it % IRING], ((it / IRING) & 1) ^ 1, p.limit, s_abort);
        if (!ok) break;
        while (more && w.count == 0) more = walk_next(p, w);  // shares that end before the first round
        Item im = {};
        if (more) {
          im.count = w.count;
          im.rows = min(ITEM, w.r.nq * p.G - w.tile * ITEM);
          im.j0 = w.j0 + w.rd * TILE;
          im.b = w.b;
          im.g = w.g;
          im.row0 = w.tile * ITEM;
          im.c0 = w.r.c0;
          im.qs = w.r.qs;
          im.len = w.r.len;
          const int i0 = p.by_G.div(im.row0), i1 = p.by_G.div(im.row0 + im.rows - 1);
          im.any_hi = vis_hi(p, w.r, i1);
          im.all_lo = vis_lo(p, w.r, i1);
          im.all_hi = vis_hi(p, w.r, i0);
          im.whole = w.count == w.nt;
          im.head = w.rd > 0;
        }
        items[it % IRING] = im;
        mbar_arrive(&i_full[it % IRING]);
        if (!more) break;
        more = walk_next(p, w);
      }
      if (!ok) {
        *s_abort = 1;
        report(p.a.status, HCL_ERR_TIMEOUT);
      }
    }
    __syncwarp();
  } else if (any && warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int t = warp >> 2, row = tid & 127;
    const uint32_t lq = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lq + t * 128, tO = tbase + lq + O_COL + t * 128;
    float* s_stat = reinterpret_cast<float*>(sm + C::STAT);
    uint32_t rg = 0, step = 0;
    bool ok = true;
    for (uint32_t it = 0;; it++) {
      const Item* im = items + it % IRING;
      ok = ok && mbar_wait(&i_full[it % IRING], (it / IRING) & 1, p.limit, s_abort);
      if (ok && im->count) ok = mbar_wait(q_full, it & 1, p.limit, s_abort);
      if (bar_or(3, 256, !ok)) { ok = false; break; }
      const int n = im->count, rows = im->rows, jfirst = im->j0;
      if (n == 0) break;
      const bool pair = rows > 128;
      const int irow = (pair ? t * 128 : 0) + row;  // row of the item
      const bool valid = irow < rows;
      int hi, lo;
      int head, orow;  // (T * H < 2^31)
      {
        const int qr = im->row0 + (valid ? irow : 0), qi = p.by_G.div(qr);
        const Req r = {0, im->c0, im->len, im->qs};
        hi = valid ? vis_hi(p, r, qi) : 0;
        lo = valid ? vis_lo(p, r, qi) : 0;
        head = im->g * p.G + qr - qi * p.G;
        orow = (r.c0 + qi) * p.a.H + head;
      }
      const float back = reinterpret_cast<const float*>(sm + C::BACK)[irow];
      const int steps = pair ? n : (n + 1 - t) / 2;
      float m, M = -INFINITY, l = 0.f, lvref = -INFINITY;
      bool sick = false;  // a NaN value in a row that this query sees
      auto look = [&](uint32_t R, int j0) {
        const RoundPar* rp = par + R % PRING;
        if (!rp->edge) return;
        // bit q * RPW + r of widening warp v's word: row q * RPP + v * RPW + r
#pragma unroll 1
        for (int v = 0; v < 4; v++)
          for (uint32_t bits = rp->poison[v]; bits; bits &= bits - 1) {
            const int e = __ffs(bits) - 1, r = (e / C::RPW) * C::RPP + v * C::RPW + e % C::RPW;
            sick |= j0 + r >= lo && j0 + r < hi && ((rp->valid[r >> 5] >> (r & 31)) & 1u);
          }
      };
      const int back2 = pair ? 1 : 2;  // rounds from one step to the next
      for (int k = 0; k < steps; k++) {
        const int rr = pair ? k : 2 * k + t;
        const uint32_t R = rg + rr, n = step + k;
        const int j0 = jfirst + rr * TILE;
        const uint32_t tSn = tS + (n & 1) * TILE;
        ok = mbar_wait(&s_full[2 * t + (n & 1)], (n >> 1) & 1, p.limit, s_abort);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
        // (these scores were issued behind PV of the step before the last: its marks stand)
        if (k > 1) look(R - 2 * back2, j0 - 2 * back2 * TILE);
        const RoundPar* rp = par + R % PRING;
        uint32_t sv[TILE];
#pragma unroll
        for (int q = 0; q < 4; q++) tmem_ld16(tSn + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&sv[16 * q]));
        const float4 kc4 = *reinterpret_cast<const float4*>(rp->kc), lv4 = *reinterpret_cast<const float4*>(rp->lv);
        const float4 wl4 = *reinterpret_cast<const float4*>(rp->wl);
        float lv[4] = {lv4.x, lv4.y, lv4.z, lv4.w}, wl[4] = {wl4.x, wl4.y, wl4.z, wl4.w};
        const float Mo = M;           // O's reference
        const uint32_t vb[2] = {range_mask(j0, lo, hi) & rp->valid[0], range_mask(j0 + 32, lo, hi) & rp->valid[1]};
        // lvref over the groups that this query row sees: the part's, unless rounds at an edge of
        // what the item sees left this row some of its groups out
        float ref = lvref;
        if (rp->edge) {
#pragma unroll
          for (int g = 0; g < 4; g++)
            if (vb[g >> 1] & (g & 1 ? 0xFFFF0000u : 0xFFFFu)) ref = fmaxf(ref, rp->lvg[g]);
        } else {
          ref = fmaxf(ref, rp->top);
        }
        if (ref != rp->lvref) {
#pragma unroll
          for (int g = 0; g < 4; g++) {
            lv[g] = fmaxf(rp->lvg[g], ref - LV_SPAN);
            wl[g] = ex2_ftz(ref - lv[g]);
          }
        }
        if (ref != lvref) {
          if (lvref != -INFINITY) grow_lvref(ref - lvref, l, M);
          lvref = ref;
        }
        const float kc[4] = {fmaxf(kc4.x * back, SCALE_MIN), fmaxf(kc4.y * back, SCALE_MIN),
                             fmaxf(kc4.z * back, SCALE_MIN), fmaxf(kc4.w * back, SCALE_MIN)};
        tmem_ld_wait();
        if ((vb[0] & vb[1]) != 0xFFFFFFFFu) {
#pragma unroll
          for (int j = 0; j < TILE; j++)
            if (!((vb[j >> 5] >> (j & 31)) & 1u)) sv[j] = 0xFF800000u;  // -inf
        }
        float mw = -INFINITY;  // largest z2 + lv
#pragma unroll
        for (int q = 0; q < 4; q++) {
          float sx = fmaxf(__uint_as_float(sv[16 * q]), __uint_as_float(sv[16 * q + 1]));
#pragma unroll
          for (int j = 2; j < 16; j += 2)
            sx = fmax3(sx, __uint_as_float(sv[16 * q + j]), __uint_as_float(sv[16 * q + j + 1]));
          mw = fmaxf(mw, fmaf(sx, kc[q], lv[q]));
        }
        const float M2 = mw > M + P_LAZY ? mw : M;
        const float al = M2 == Mo || Mo == -INFINITY ? 1.f : ex2_ftz(Mo - M2);
        const float ll = M == Mo ? al : ex2_ftz(M - M2);
        M = M2;
        if (__any_sync(0xffffffffu, al != 1.f)) {
          // rescale O, once PV of the last step is done with it (rows without a reference yet are
          // in their first step or have an O of zeros)
          if (k > 0) {
            ok = mbar_wait(&o_done[2 * t + ((n & 1) ^ 1)], ((n - 1) >> 1) & 1, p.limit, s_abort);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; c++) {
            uint32_t r[32];
#pragma unroll
            for (int q = 0; q < 2; q++) tmem_ld16(tO + 32 * c + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&r[16 * q]));
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j++) r[j] = __float_as_uint(__uint_as_float(r[j]) * al);
#pragma unroll
            for (int q = 0; q < 2; q++) tmem_st16(tO + 32 * c + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&r[16 * q]));
          }
        }
        const float Mu = M == -INFINITY ? 0.f : M;
        // P over the first half of its S, whose scores are in registers
        float lr = 0.f;
#pragma unroll
        for (int c = 0; c < 2; c++) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const int gq = 2 * c + q;
            const float add = lv[gq] - Mu + P_OFF;
            const unsigned long long c2 = f2_make(kc[gq], kc[gq]), a2 = f2_make(add, add);
            unsigned long long g = 0ull;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const int e = 16 * gq + j;
              const unsigned long long x = f2_fma(f2_make(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, a2);
              const float e0 = ex2_ftz(f2_lo(x)), e1 = ex2_ftz(f2_hi(x));
              g = f2_add(g, f2_make(e0, e1));
              pk[8 * q + (j >> 1)] = half2_of(e0, e1);
            }
            lr = fmaf(f2_lo(g) + f2_hi(g), wl[gq], lr);
          }
          tmem_st16(tSn + 16 * c, pk);
        }
        l = fmaf(l, ll, lr);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[2 * t + (n & 1)]);
        if (k == 0) {  // (behind the use of the factor)
          __syncwarp();
          if (lane == 0) mbar_arrive(q_empty);
        }
      }
      if (steps == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty);
      }
      if (ok && steps > 0) {
        const uint32_t n = step + steps - 1;
        ok = mbar_wait(&o_done[2 * t + (n & 1)], (n >> 1) & 1, p.limit, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        for (int k = max(0, steps - 2); ok && k < steps; k++) {
          const int rr = pair ? k : 2 * k + t;
          look(rg + rr, jfirst + rr * TILE);
        }
      }
      m = M - P_OFF - lvref;  // (-inf where nothing was seen)
      if (M == -INFINITY) m = -INFINITY;
      if (sick) l = NAN;
      if (!ok) {
        *s_abort = 1;
        report(p.a.status, HCL_ERR_TIMEOUT);
      }
      // Single mode: the groups join their results, each reading both O's (the same lanes of TMEM)
      // for its half of the dimensions.
      float fa = 1.f, fb = 0.f;  // factors of the (first) O and the other group's,
      float f2 = 1.f;            // and of their sum
      if (!pair) {
        *reinterpret_cast<float4*>(s_stat + (t * 128 + row) * 4) = make_float4(m, M, l, 0.f);
        tc_fence_before();
        if (bar_or(3, 256, !ok)) { ok = false; break; }
        tc_fence_after();
        const float4 s0 = *reinterpret_cast<const float4*>(s_stat + row * 4);
        const float4 s1 = *reinterpret_cast<const float4*>(s_stat + (128 + row) * 4);
        m = fmaxf(s0.x, s1.x);
        M = fmaxf(s0.y, s1.y);
        l = (s0.x == -INFINITY ? s0.z : s0.z * ex2_ftz(s0.x - m)) + (s1.x == -INFINITY ? s1.z : s1.z * ex2_ftz(s1.x - m));
        fa = s0.y == -INFINITY ? 0.f : ex2_ftz(s0.y - M);
        fb = s1.y == -INFINITY ? 0.f : ex2_ftz(s1.y - M);
      }
      if (!ok) continue;  // (to the barrier where the block's end is agreed)
      const bool whole = im->whole != 0;
      float* pp = p.part + (2 * (size_t)blockIdx.x + (im->head ? 0 : 1)) * part_floats(ITEM, D);
      if (whole) {
        float lse;
        const float f = finish_row<false>(m, M, l, p.a.sink && valid ? p.a.sink[head] * LOG2E : -INFINITY, &f2, &lse);
        fa *= f;
        fb *= f;
        if (valid && p.a.lse && (pair || t == 0)) p.a.lse[orow] = lse;
      } else if (pair || t == 0) {
        *reinterpret_cast<float4*>(pp + irow * 4) = make_float4(m, M, l, 0.f);
      }
      // 32 dimensions at a time, through shared memory, so that the warp writes whole pieces of rows.
      // (Loops that are not unrolled: this code runs once an item, and its fetch would take longer.)
      uint8_t* stage = sm + C::OUT + warp * 4096;
      uint8_t* mine = stage + lane * 128;
      const int r_in = lane >> 3, e_in = lane & 7, irow0 = irow - lane;
      const uint32_t o_at = pair ? tO : tO - t * 128;
      const int c_lo = pair ? 0 : t * 64, c_hi = pair ? D : min(D, t * 64 + 64);
#pragma unroll 1
      for (int c = c_lo; c < c_hi; c += 32) {
        float x[32];
#pragma unroll
        for (int q = 0; q < 2; q++)
          tmem_ld16(o_at + c + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(reinterpret_cast<uint32_t*>(&x[16 * q])));
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j++) x[j] = fa == 0.f ? 0.f : x[j] * fa;
        if (!pair) {
          uint32_t y[32];
#pragma unroll
          for (int q = 0; q < 2; q++) tmem_ld16(o_at + 128 + c + 16 * q, *reinterpret_cast<uint32_t(*)[16]>(&y[16 * q]));
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j++)
            if (fb != 0.f) x[j] = fmaf(__uint_as_float(y[j]), fb, x[j]);
        }
#pragma unroll
        for (int j = 0; j < 32; j++) x[j] *= f2;
        if (whole && !p.a.out32) {
          // bf16, 64 dimensions in the rows' 128 bytes: 8 pieces, four of them now
          const int half = (c >> 3) & 4;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; k++) h[k] = bf16x2_of(x[8 * e + 2 * k], x[8 * e + 2 * k + 1]);
            *reinterpret_cast<uint4*>(mine + (((half + e) ^ (lane & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
          if (half) {
            __syncwarp();
#pragma unroll 2
            for (int k = 0; k < 8; k++) {
              const int r = 4 * k + r_in;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((e_in ^ (r & 7)) << 4));
              const int to = __shfl_sync(~0u, orow, r);
              if (irow0 + r < rows)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + (size_t)to * D + c - 32 + e_in * 8) = v;
            }
          }
        } else {
          // fp32
#pragma unroll
          for (int e = 0; e < 8; e++)
            *reinterpret_cast<float4*>(mine + ((e ^ (lane & 7)) << 4)) =
                make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          __syncwarp();
#pragma unroll 2
          for (int k = 0; k < 8; k++) {
            const int r = 4 * k + r_in;
            const float4 v = *reinterpret_cast<const float4*>(stage + r * 128 + ((e_in ^ (r & 7)) << 4));
            const int to = __shfl_sync(~0u, orow, r);
            if (irow0 + r < rows)
              *reinterpret_cast<float4*>((whole ? p.a.out32 + (size_t)to * D : pp + ITEM * 4 + (size_t)(irow0 + r) * D) + c +
                                         e_in * 4) = v;
          }
        }
        __syncwarp();
      }
      // (single mode: a group's O is read by both)
      tc_fence_before();
      if (!pair) asm volatile("bar.sync 4, 256;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[it % IRING]);
      rg += n;
      step += steps;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool SHARED>
hcl_status_t launch_t(const Params& p, cudaStream_t st) {
  CUtensorMap tk, tv;
  const int box = std::min(p.a.kv.page, 64);
  hcl_status_t e = code_map(&tk, p.a.kv.k, p.a.kv, box, false);
  if (e != HCL_OK) return e;
  tv = tk;
  if (!SHARED) {
    e = code_map(&tv, p.a.kv.v, p.a.kv, box, false);
    if (e != HCL_OK) return e;
  }
  auto kern = paged_tile_kernel<D, SHARED>;
  const int smem = (int)Cfg<D, SHARED>::TOTAL + 1024;
  static_assert(Cfg<D, SHARED>::TOTAL + 1024 <= 232448, "shared memory");
  e = set_kernel_attrs(reinterpret_cast<const void*>(kern), smem, false);
  if (e != HCL_OK) return e;
  return check_cuda(launch_pdl(kern, dim3(p.n_blocks), dim3(THREADS), (size_t)smem, st, 1, p, tk, tv),
                    "paged attention (tiles) launch");
}

}  // namespace

int tile_blocks() { return std::min(1024, num_sms()); }

hcl_status_t launch_tiles(const Params& p, cudaStream_t st) {
  if (p.a.kv.d == 128) return p.a.kv.v ? launch_t<128, false>(p, st) : launch_t<128, true>(p, st);
  return p.a.kv.v ? launch_t<64, false>(p, st) : launch_t<64, true>(p, st);
}

}  // namespace paged
}  // namespace hcl

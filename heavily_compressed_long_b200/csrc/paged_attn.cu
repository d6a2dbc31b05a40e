// paged_attn.cu -- paged attention: which kernel takes which request, and the merge of requests
// that were split over blocks.
#include <algorithm>

#include "paged_common.cuh"

namespace hcl {
namespace paged {
namespace {

// Joins the partial results of the items that were split.  Block (c, y) takes the item that ends
// in block c of the attention kernel.  An item with few parts (prompts: two or three) gives each
// warp a row of its own; one with many (a long decode over all blocks) gives each row the whole
// block, its warps taking the parts in turn and adding up in a fixed order.
// a += f * part; a part that weighs nothing may hold anything.
template <int E>
__device__ __forceinline__ void add_part(float (&a)[E], const float* src, float f) {
  float x[E];
  if constexpr (E == 4) {
    const float4 v = *reinterpret_cast<const float4*>(src);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(src);
    x[0] = v.x; x[1] = v.y;
  }
#pragma unroll
  for (int e = 0; e < E; e++) a[e] = f == 0.f ? a[e] : fmaf(x[e], f, a[e]);
}

constexpr int MW = 8;
// Parts that a warp of its own joins: a lane holds each one's statistics.  (The whole block a row
// for every item: drafts 82 -> 103 us, window chunks 54 -> 81, prompts 585 -> 676, grouped decode
// 246 -> 250.)
constexpr int FEW = 32;
template <int D, int ROWS>
__global__ void __launch_bounds__(MW * 32) paged_merge_kernel(const Params p) {
  constexpr int E = D / 32;
  constexpr size_t PART = part_floats(ROWS, D);
  __shared__ float s_w[1024];
  __shared__ float s_red[MW][3];
  __shared__ float s_o[MW][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  pdl_enter();
  const Meta mt = p.meta[c];
  if (!mt.ends) return;
  const int b = mt.b, g = mt.g, row0 = mt.row0;
  // the item began in the last block whose first unit, tot * c0 / nb, is not behind mt.first
  const int c0 = (int)(((mt.first + 1) * mt.nb - 1) / mt.tot), n = c - c0 + 1;
  // the part of block c0 + k: the tail of the first, the head of the others
  auto part = [&](int k) { return p.part + (2 * (size_t)(c0 + k) + (k == 0 ? 1 : 0)) * PART; };
  const Req r = load_req(p, b, false);
  const int rows = min(ROWS, r.nq * p.G - row0);
  const bool few = n <= FEW;
  const int step = few ? gridDim.y * MW : gridDim.y;
  for (int row = few ? blockIdx.y * MW + warp : blockIdx.y; row < rows; row += step) {
    const int qi = p.by_G.div(row0 + row), head = g * p.G + row0 + row - qi * p.G;
    const size_t orow = (size_t)(r.c0 + qi) * p.a.H + head;
    const float sink2 = p.a.sink ? p.a.sink[head] * LOG2E : -INFINITY;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + orow * D;
    float m = -INFINITY, M = -INFINITY, l = 0.f, f2, lse;
    if (few) {
      float4 h = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
      if (lane < n) h = *reinterpret_cast<const float4*>(part(lane) + row * 4);
      m = h.x;
      M = h.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
      }
      l = h.x == -INFINITY ? h.z : h.z * ex2_ftz(h.x - m);
      const float f = h.y == -INFINITY ? 0.f : ex2_ftz(h.y - M);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      float a[E];
#pragma unroll
      for (int e = 0; e < E; e++) a[e] = 0.f;
#pragma unroll 4
      for (int k = 0; k < n; k++) add_part<E>(a, part(k) + ROWS * 4 + (size_t)row * D + lane * E, __shfl_sync(~0u, f, k));
      const float fo = finish_row<ROWS == ROWS_SMALL>(m, M, l, sink2, &f2, &lse);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 x = fo == 0.f ? make_float2(0.f, 0.f) : make_float2(a[e] * fo * f2, a[e + 1] * fo * f2);
        if (p.a.out32)
          *reinterpret_cast<float2*>(p.a.out32 + orow * D + lane * E + e) = x;
        else
          *reinterpret_cast<uint32_t*>(out + lane * E + e) = bf16x2_of(x.x, x.y);
      }
      if (lane == 0 && p.a.lse) p.a.lse[orow] = lse;
      continue;
    }
    for (int k = tid; k < n; k += MW * 32) {
      const float4 h = *reinterpret_cast<const float4*>(part(k) + row * 4);
      m = fmaxf(m, h.x);
      M = fmaxf(M, h.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
      M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    }
    if (lane == 0) { s_red[warp][0] = m; s_red[warp][1] = M; }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < MW; v++) { m = fmaxf(m, s_red[v][0]); M = fmaxf(M, s_red[v][1]); }
    for (int k = tid; k < n; k += MW * 32) {
      const float4 h = *reinterpret_cast<const float4*>(part(k) + row * 4);
      s_w[k] = h.y == -INFINITY ? 0.f : ex2_ftz(h.y - M);
      l += h.x == -INFINITY ? h.z : h.z * ex2_ftz(h.x - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    if (lane == 0) s_red[warp][2] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int v = 0; v < MW; v++) l += s_red[v][2];
    float a[E];
#pragma unroll
    for (int e = 0; e < E; e++) a[e] = 0.f;
#pragma unroll 4
    for (int k = warp; k < n; k += MW) add_part<E>(a, part(k) + ROWS * 4 + (size_t)row * D + lane * E, s_w[k]);
#pragma unroll
    for (int e = 0; e < E; e++) s_o[warp][lane * E + e] = a[e];
    __syncthreads();
    const float fo = finish_row<ROWS == ROWS_SMALL>(m, M, l, sink2, &f2, &lse);
    for (int e = tid; e < D; e += MW * 32) {
      float x = 0.f;
#pragma unroll
      for (int v = 0; v < MW; v++) x += s_o[v][e];
      x = fo == 0.f ? 0.f : x * fo * f2;
      if (p.a.out32)
        p.a.out32[orow * D + e] = x;
      else
        out[e] = __float2bfloat16(x);
    }
    if (tid == 0 && p.a.lse) p.a.lse[orow] = lse;
    __syncthreads();
  }
}

}  // namespace

hcl_status_t launch_merge(const Params& p, int rows, cudaStream_t st) {
  const bool small = rows == ROWS_SMALL;
  auto kern = p.a.kv.d == 128
                  ? (small ? paged_merge_kernel<128, ROWS_SMALL> : paged_merge_kernel<128, ROWS_ITEM>)
                  : (small ? paged_merge_kernel<64, ROWS_SMALL> : paged_merge_kernel<64, ROWS_ITEM>);
  return check_cuda(launch_pdl(kern, dim3(p.n_blocks, small ? 4 : 16), dim3(MW * 32), 0, st, 1, p),
                    "paged attention merge launch");
}

}  // namespace paged

size_t paged_attn_workspace_bytes(int T, int H, int Hkv, int d) {
  using namespace paged;
  if (T < 1 || H < 1 || Hkv < 1) return 0;
  const int G = H / Hkv;
  return (G <= ROWS_SMALL ? split_workspace(std::min(1024, ROWS_BLOCKS_MOST * num_sms()), ROWS_SMALL, d) : 0) +
         ((long long)T * G > ROWS_SMALL ? split_workspace(tile_blocks(), ROWS_ITEM, d) : 0);
}

// Each request goes by its own query rows to the row kernel or the tile kernel; a launch that no
// request can need (by H / Hkv and max_q) is left out.
hcl_status_t launch_paged_attn(const PagedAttnArgs& a, void* ws, cudaStream_t st) {
  using namespace paged;
  Params p;
  p.a = a;
  p.sh = a.kv.page == 16 ? 4 : a.kv.page == 32 ? 5 : a.kv.page == 64 ? 6 : 7;
  p.G = a.H / a.kv.Hkv;
  p.by_G = FastDiv(p.G);
  p.by_m = FastDiv(a.m);
  p.scale2 = a.scale * LOG2E;
  p.limit = wait_limit_cycles();
  uint8_t* at = static_cast<uint8_t*>(ws);
  if (p.G <= ROWS_SMALL) {
    // (small requests have up to 8 rows, unless the call's bounds let them have up to 16)
    const int rows = (int)std::min<long long>(ROWS_SMALL, (long long)std::min(a.max_q, a.T) * p.G);
    p.n_blocks = rows_blocks(a.kv.d, a.kv.v == nullptr);
    p.meta = reinterpret_cast<Meta*>(at);
    p.part = reinterpret_cast<float*>(at + meta_bytes(p.n_blocks));
    hcl_status_t e = launch_rows(p, rows, st);
    if (e == HCL_OK) e = launch_merge(p, ROWS_SMALL, st);
    if (e != HCL_OK) return e;
    at += split_workspace(std::min(1024, ROWS_BLOCKS_MOST * num_sms()), ROWS_SMALL, a.kv.d);
  }
  if ((long long)std::max(1, std::min(a.max_q, a.T)) * p.G <= ROWS_SMALL) return HCL_OK;
  p.n_blocks = tile_blocks();
  p.meta = reinterpret_cast<Meta*>(at);
  p.part = reinterpret_cast<float*>(at + meta_bytes(p.n_blocks));
  hcl_status_t e = launch_tiles(p, st);
  return e == HCL_OK ? launch_merge(p, ROWS_ITEM, st) : e;
}

}  // namespace hcl

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
constexpr int MW = 8;
constexpr int FEW = 16;
template <int D, int ROWS>
__global__ void __launch_bounds__(MW * 32) paged_merge_kernel(const Params p) {
  constexpr int E = D / 32;
  constexpr size_t PART = part_floats(ROWS, D);
  __shared__ float s_w[1024];
  __shared__ float s_red[MW][3];
  __shared__ float s_o[MW][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  pdl_enter();
  auto first_unit = [&](int k) { return reinterpret_cast<const long long*>(p.meta + 2 * k)[0]; };
  const int* mi = reinterpret_cast<const int*>(p.meta + 2 * c);
  if (!mi[6]) return;
  const long long first = reinterpret_cast<const long long*>(mi)[1];
  const int b = mi[4], g = mi[5], row0 = mi[7];
  // the item began in the last block whose first unit is not behind `first`
  int c0 = 0;
  for (int hi = c; hi - c0 > 1;) {
    const int mid = (c0 + hi) >> 1;
    if (first_unit(mid) <= first) c0 = mid;
    else hi = mid;
  }
  const int n = c - c0 + 1;
  // the part of block c0 + k: the tail of the first, the head of the others; blocks between
  // without a unit wrote none
  auto part = [&](int k) { return p.part + (2 * (size_t)(c0 + k) + (k == 0 ? 1 : 0)) * PART; };
  auto used = [&](int k) { return k == 0 || k == n - 1 || first_unit(c0 + k) < first_unit(c0 + k + 1); };
  const Req r = load_req(p, b, false);
  const int rows = min(ROWS, r.nq * p.G - row0);
  const bool few = n <= FEW;
  const int step = few ? gridDim.y * MW : gridDim.y;
  for (int row = few ? blockIdx.y * MW + warp : blockIdx.y; row < rows; row += step) {
    const int head = g * p.G + (row0 + row) % p.G;
    const size_t orow = (size_t)(r.c0 + (row0 + row) / p.G) * p.a.H + head;
    const float sink2 = p.a.sink ? p.a.sink[head] * LOG2E : -INFINITY;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + orow * D;
    float m = -INFINITY, M = -INFINITY, l = 0.f, lse;
    if (few) {
      float4 h = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
      if (lane < n && used(lane)) h = *reinterpret_cast<const float4*>(part(lane) + row * 4);
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
      for (int k = 0; k < n; k++) {
        const float fk = __shfl_sync(~0u, f, k);
        if (fk != 0.f) {
          const float* src = part(k) + ROWS * 4 + (size_t)row * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e++) a[e] = fmaf(src[e], fk, a[e]);
        }
      }
      const float fo = finish_row(m, M, l, sink2, &lse);
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + lane * E + e) = fo == 0.f ? 0u : bf16x2_of(a[e] * fo, a[e + 1] * fo);
      if (lane == 0 && p.a.lse) p.a.lse[orow] = lse;
      continue;
    }
    for (int k = tid; k < n; k += MW * 32)
      if (used(k)) {
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
      float f = 0.f;
      if (used(k)) {
        const float4 h = *reinterpret_cast<const float4*>(part(k) + row * 4);
        f = h.y == -INFINITY ? 0.f : ex2_ftz(h.y - M);
        l += h.x == -INFINITY ? h.z : h.z * ex2_ftz(h.x - m);
      }
      s_w[k] = f;
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
    for (int k = warp; k < n; k += MW) {
      const float f = s_w[k];
      if (f != 0.f) {
        const float* src = part(k) + ROWS * 4 + (size_t)row * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e++) a[e] = fmaf(src[e], f, a[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < E; e++) s_o[warp][lane * E + e] = a[e];
    __syncthreads();
    const float fo = finish_row(m, M, l, sink2, &lse);
    for (int e = tid; e < D; e += MW * 32) {
      float x = 0.f;
#pragma unroll
      for (int v = 0; v < MW; v++) x += s_o[v][e];
      out[e] = __float2bfloat16(fo == 0.f ? 0.f : x * fo);
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
  (void)T;
  if (Hkv < 1) return 0;
  return paged::tile_workspace(d) + (H / Hkv <= paged::ROWS_SMALL ? paged::rows_workspace(d) : 0);
}

// Each request goes by its own query rows to the row kernel or the tile kernel; a launch that no
// request can need (by H / Hkv and max_q) is left out.
hcl_status_t launch_paged_attn(const PagedAttnArgs& a, void* ws, cudaStream_t st) {
  using namespace paged;
  Params p;
  p.a = a;
  p.sh = a.kv.page == 16 ? 4 : a.kv.page == 32 ? 5 : a.kv.page == 64 ? 6 : 7;
  p.G = a.H / a.kv.Hkv;
  p.scale2 = a.scale * LOG2E;
  p.limit = wait_limit_cycles();
  uint8_t* at = static_cast<uint8_t*>(ws);
  if (p.G <= ROWS_SMALL) {
    p.n_blocks = rows_blocks();
    p.meta = reinterpret_cast<int4*>(at);
    p.part = reinterpret_cast<float*>(p.meta + 2 * p.n_blocks);
    hcl_status_t e = launch_rows(p, st);
    if (e == HCL_OK) e = launch_merge(p, ROWS_SMALL, st);
    if (e != HCL_OK) return e;
    at += rows_workspace(a.kv.d);
  }
  if ((long long)a.max_q * p.G <= ROWS_SMALL) return HCL_OK;
  p.n_blocks = tile_blocks();
  p.meta = reinterpret_cast<int4*>(at);
  p.part = reinterpret_cast<float*>(p.meta + 2 * p.n_blocks);
  hcl_status_t e = launch_tiles(p, st);
  return e == HCL_OK ? launch_merge(p, ROWS_ITEM, st) : e;
}

}  // namespace hcl

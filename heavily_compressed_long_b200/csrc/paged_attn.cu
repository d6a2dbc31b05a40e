// paged_attn.cu -- attention of a ragged batch over the paged 8-bit cache.
#include <algorithm>

#include "paged_common.cuh"

namespace hcl {
namespace {

using namespace paged;

constexpr int PA_WARPS = 8;

// One block per (query, query head): each warp takes every eighth visible row with an online
// softmax, lanes over the head's dimensions; the warps' partial results merge in shared memory.
template <int D>
__global__ void __launch_bounds__(PA_WARPS * 32) paged_attn_rows_kernel(Params p) {
  constexpr int E = D / 32;
  __shared__ float s_m[PA_WARPS], s_l[PA_WARPS], s_o[PA_WARPS][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x / p.a.H, h = blockIdx.x % p.a.H, g = h / p.G;
  pdl_enter();
  int lo_b = 0, hi_b = p.a.B;
  while (hi_b - lo_b > 1) {
    const int mid = (lo_b + hi_b) >> 1;
    if (p.a.cu_q[mid] <= t) lo_b = mid;
    else hi_b = mid;
  }
  const int b = lo_b, c0 = p.a.cu_q[b];
  if (t < c0 || t >= p.a.cu_q[b + 1]) return;
  if (p.a.cu_q[b + 1] - c0 > p.a.max_q) {
    if (tid == 0) report(p.a.status, HCL_ERR_DEVICE_FAULT);
    return;
  }
  if ((p.a.cu_q[b + 1] - c0) * p.G <= ROWS_SMALL) return;
  const long long pos = (long long)p.a.q_start[b] + (t - c0);
  const long long room = (long long)p.a.max_pages << p.sh;
  long long len = p.a.kv_len[b];
  if (len > room) {
    len = room;
    if (tid == 0) report(p.a.status, HCL_ERR_DEVICE_FAULT);
  }
  const int hi = (int)max(0ll, min(len, pos < 0 ? 0ll : (pos + 1) / p.a.m));
  const int lo = p.a.W > 0 ? (int)max(0ll, pos - p.a.W + 1) : 0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.a.q) + (int64_t)t * p.a.q_stride + h * D;
  float qv[E], o[E];
#pragma unroll
  for (int i = 0; i < E; i++) { qv[i] = bf2f(q[lane * E + i]); o[i] = 0.f; }
  const uint8_t* kc = static_cast<const uint8_t*>(p.a.kv.k);
  const uint8_t* vc = static_cast<const uint8_t*>(p.a.kv.v ? p.a.kv.v : p.a.kv.k);
  const float* vs = p.a.kv.v ? p.a.kv.v_scale : p.a.kv.k_scale;
  float m = -INFINITY, l = 0.f;
  for (int j = lo + warp; j < hi; j += PA_WARPS) {
    const int id = p.a.table[(size_t)b * p.a.max_pages + (j >> p.sh)];
    if (id < 0 || id >= p.a.kv.n_pages) {
      if (lane == 0) report(p.a.status, HCL_ERR_DEVICE_FAULT);
      continue;
    }
    const size_t pg = (size_t)id * p.a.kv.Hkv + g;
    const size_t at = ((pg << p.sh) + (j & (p.a.kv.page - 1))) * D + lane * E;
    float kx[E], vx[E];
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      uint32_t u;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(u) : "h"(*reinterpret_cast<const uint16_t*>(kc + at + i)));
      const __half2 kh = *reinterpret_cast<__half2*>(&u);
      kx[i] = __low2float(kh); kx[i + 1] = __high2float(kh);
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(u) : "h"(*reinterpret_cast<const uint16_t*>(vc + at + i)));
      const __half2 vh = *reinterpret_cast<__half2*>(&u);
      vx[i] = __low2float(vh); vx[i + 1] = __high2float(vh);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; i++) s = fmaf(qv[i], kx[i], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(~0u, s, w);
    const float z = s * (fmaxf(p.a.kv.k_scale[pg], 1.17549435e-38f) * p.scale2);
    const float m2 = fmaxf(m, z), al = m == -INFINITY ? 0.f : exp2f(m - m2), w = exp2f(z - m2);
    l = l * al + w;
    const float wv = w * fmaxf(vs[pg], 1.17549435e-38f);
#pragma unroll
    for (int i = 0; i < E; i++) o[i] = o[i] * al + wv * vx[i];
    m = m2;
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int i = 0; i < E; i++) s_o[warp][lane * E + i] = o[i];
  __syncthreads();
  float mt = -INFINITY, lt = 0.f;
  for (int w = 0; w < PA_WARPS; w++) mt = fmaxf(mt, s_m[w]);
  const float sink2 = p.a.sink ? p.a.sink[h] * LOG2E : -INFINITY;
  mt = fmaxf(mt, sink2);
  for (int w = 0; w < PA_WARPS; w++) lt += s_m[w] == -INFINITY ? 0.f : s_l[w] * exp2f(s_m[w] - mt);
  if (sink2 != -INFINITY) lt += exp2f(sink2 - mt);
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
  for (int i = tid; i < D; i += PA_WARPS * 32) {
    float acc = 0.f;
    for (int w = 0; w < PA_WARPS; w++) acc += s_m[w] == -INFINITY ? 0.f : s_o[w][i] * exp2f(s_m[w] - mt);
    static_cast<__nv_bfloat16*>(p.a.out)[((size_t)t * p.a.H + h) * D + i] = __float2bfloat16(acc * inv);
  }
  if (tid == 0 && p.a.lse)
    p.a.lse[(size_t)t * p.a.H + h] = lt > 0.f ? (mt + log2f(lt)) * LN2 : -INFINITY;
}

}  // namespace

size_t paged_attn_workspace_bytes(int, int, int, int d) { return rows_workspace(d); }

hcl_status_t launch_paged_attn(const PagedAttnArgs& a, void* ws, cudaStream_t st) {
  Params p;
  p.a = a;
  p.sh = a.kv.page == 16 ? 4 : a.kv.page == 32 ? 5 : a.kv.page == 64 ? 6 : 7;
  p.G = a.H / a.kv.Hkv;
  p.scale2 = a.scale * LOG2E;
  p.limit = wait_limit_cycles();
  p.n_blocks = rows_blocks();
  p.meta = static_cast<int4*>(ws);
  p.part = reinterpret_cast<float*>(p.meta + 2 * p.n_blocks);
  if (p.G <= ROWS_SMALL) {
    hcl_status_t e = launch_rows(p, st);
    if (e != HCL_OK) return e;
    e = launch_rows_merge(p, st);
    if (e != HCL_OK) return e;
  }
  if ((long long)p.a.max_q * p.G <= ROWS_SMALL) return HCL_OK;
  auto kern = a.kv.d == 128 ? paged_attn_rows_kernel<128> : paged_attn_rows_kernel<64>;
  return check_cuda(launch_pdl(kern, dim3((unsigned)((long long)a.T * a.H)), dim3(PA_WARPS * 32), 0, st, 1, p),
                    "paged attention launch");
}

}  // namespace hcl

// MQA attention of the last T tokens of each sequence over a paged cache
// (K = V = the full 512-wide row), over all rows or those of chosen blocks.
//
// One warp per query head walks the rows with a running maximum and sum; lane
// l holds dims [16l, 16l + 16) of the query and of the output.
#include <algorithm>

#include "paged.cuh"
#include "quant.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) paged_attn_kernel(const lidx_paged_attn_args a, int shift, uint32_t *status) {
  const int64_t head = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  if (head >= static_cast<int64_t>(a.B) * a.T * a.H) return;
  const int64_t bt = head / a.H;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt % a.T);
  bool cut;
  const int32_t seen = cut_len(__ldg(a.len + b), a.cache, cut) - (a.T - 1 - t);
  bool bounds = cut;
  float q[16], o[16];
  const uint4 *qs = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + head * 512 + 16 * lane);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint4 w = __ldg(qs + i);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
      q[8 * i + 2 * k] = bf16x2_lo(x[k]);
      q[8 * i + 2 * k + 1] = bf16x2_hi(x[k]);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; i++) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * 1.4426950408889634f;
  int nb = (max(seen, 0) + a.cache.page_rows - 1) >> shift;
  if (a.blocks) nb = a.n_sel ? min(max(__ldg(a.n_sel + bt), 0), a.n_blocks) : a.n_blocks;
  for (int i = 0; i < nb; i++) {
    const int j = a.blocks ? __ldg(a.blocks + bt * a.ld_blocks + i) : i;
    if (j < 0 || j >= a.cache.max_pages) {
      bounds |= j != -1;
      continue;
    }
    const int32_t r0 = j << shift, n = min(a.cache.page_rows, seen - r0);
    if (n <= 0) continue;
    const int32_t p0 = pool_row(a.cache, shift, b, r0);
    if (p0 < 0) {
      bounds = true;
      continue;
    }
    for (int r = 0; r < n; r++) {
      float x[16], lo[8], hi[8];
      load8(a.cache.rows, p0 + r, 2 * lane, lo);
      load8(a.cache.rows, p0 + r, 2 * lane + 1, hi);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        x[k] = lo[k];
        x[8 + k] = hi[k];
      }
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < 16; k++) s = fmaf(q[k], x[k], s);
      s = warp_sum(s) * c2;
      const float mn = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(s - mn);
      l = fmaf(l, f, p);
#pragma unroll
      for (int k = 0; k < 16; k++) o[k] = fmaf(o[k], f, p * x[k]);
      m = mn;
    }
  }
  const float il = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < 16; k++) o[k] *= il;
  uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + head * 512 + 16 * lane);
  dst[0] = pack8_bf16(o);
  dst[1] = pack8_bf16(o + 8);
  if (lane == 0 && a.lse) a.lse[head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  if (bounds && lane == 0) raise_status(status, LIDX_DEV_BOUNDS);
}

}  // namespace

bool paged_attn_supported(const lidx_paged_attn_args &) { return true; }
size_t paged_attn_workspace(const lidx_paged_attn_args &) { return LIDX_WS_HEADER; }
int paged_attn_launches(const lidx_paged_attn_args &) { return 1; }

cudaError_t launch_paged_attn(const lidx_paged_attn_args &a, void *ws, cudaStream_t st) {
  const int64_t heads = static_cast<int64_t>(a.B) * a.T * a.H;
  return launch_kernel(paged_attn_kernel, dim3(static_cast<unsigned>((heads + 3) / 4)), dim3(kThreads), 0, st,
                       (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.cache), static_cast<uint32_t *>(ws));
}

}  // namespace lidx

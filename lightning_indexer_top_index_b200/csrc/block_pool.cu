// Summaries of the blocks (pages) of a paged index-key cache: the mean key as
// 8-bit codes under one scale, for the block selection's cheap score.
//
// One CTA of four warps takes a block at a time: lane l of each warp sums dims
// [4l, 4l + 4) of every fourth row in 64 bits, the warps' sums meet in shared
// memory, and 128 threads finish one dim each.  The sums are in 64 bits so
// that a mean next to a code's border rounds as the formula says, whatever the
// order of its sum.  A fp32 value's bits moved into a double's fields without
// re-biasing the exponent are the value times 2^-896 (subnormals included), so
// a conversion is integer arithmetic on the fields and the factor is taken out
// of the sum at the end; infinities and NaNs are noticed by their largest bits.
#include <algorithm>

#include "paged.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;

// x * 2^-896 for finite x
__device__ __forceinline__ double scaled_double(uint32_t u) {
  return __hiloint2double(static_cast<int>((u & 0x80000000u) | ((u & 0x7FFFFFFFu) >> 3)), static_cast<int>(u << 29));
}

// dims [4l, 4l + 4) of pool row p
__device__ __forceinline__ void load4(const lidx_kv &kv, int64_t p, int l, float (&v)[4]) {
  if (kv.dtype == LIDX_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(kv.data) + p * kv.ld) + l);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    return;
  }
  if (kv.dtype == LIDX_BF16 || l >= 16) {
    const uint16_t *s = kv.dtype == LIDX_BF16 ? static_cast<const uint16_t *>(kv.data) + p * kv.ld + 4 * l
                                              : static_cast<const uint16_t *>(kv.rope) + p * kv.ld_rope + 4 * (l - 16);
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(s));
    v[0] = bf16x2_lo(w.x); v[1] = bf16x2_hi(w.x); v[2] = bf16x2_lo(w.y); v[3] = bf16x2_hi(w.y);
    return;
  }
  const uint8_t *data = static_cast<const uint8_t *>(kv.data) + p * kv.ld;
  uint32_t x[4];
  float s;
  if (kv.dtype == LIDX_E4M3) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(data) + l);
    s = e8m0_to_f32(__ldg(kv.scale + p * kv.ld_scale));
    x[0] = e4m3x2_to_bf16x2(w);
    x[1] = e4m3x2_to_bf16x2(w >> 16);
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint16_t *>(data) + l);
    s = e8m0_to_f32(__ldg(kv.scale + p * kv.ld_scale + l / 8));
    e2m1x8_to_bf16x2(w, x);
  }
  v[0] = bf16x2_lo(x[0]) * s; v[1] = bf16x2_hi(x[0]) * s;
  v[2] = bf16x2_lo(x[1]) * s; v[3] = bf16x2_hi(x[1]) * s;
}

__global__ void __launch_bounds__(kThreads) block_pool_kernel(const lidx_block_pool_args a, int shift,
                                                               uint32_t *status) {
  __shared__ double sums[kWarps][128];
  __shared__ double tops[kWarps];
  __shared__ uint32_t bits[kWarps];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  bool cut;
  const int32_t len = cut_len(__ldg(a.len + b), a.keys, cut);
  if (cut && blockIdx.x == 0 && tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
  const int32_t rows = a.keys.page_rows;
  const int32_t first = a.first ? max(__ldg(a.first + b), 0) : 0;
  const int64_t nb = (static_cast<int64_t>(len) + rows - 1) >> shift;
  for (int64_t j = (first >> shift) + static_cast<int64_t>(blockIdx.x); j < nb && first < len; j += gridDim.x) {
    const int32_t page = __ldg(a.keys.table + static_cast<int64_t>(b) * a.keys.ld_table + j);
    if (page < 0 || page >= a.keys.n_pages) {  // the same for the whole CTA
      if (tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
      continue;
    }
    const int count = static_cast<int>(min(static_cast<int64_t>(rows), len - (j << shift)));
    const int64_t p0 = static_cast<int64_t>(page) << shift;
    double s[4] = {0., 0., 0., 0.};
    uint32_t most = 0u;
    for (int r = warp; r < count; r += kWarps * kUnroll) {
      float v[kUnroll][4];
#pragma unroll
      for (int u = 0; u < kUnroll; u++) {
        if (r + u * kWarps < count) load4(a.keys.rows, p0 + r + u * kWarps, lane, v[u]);
        else v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; u++)
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const uint32_t x = __float_as_uint(v[u][k]);
          most = max(most, x & 0x7FFFFFFFu);
          s[k] += scaled_double(x);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; k++) sums[warp][4 * lane + k] = s[k];
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) bits[warp] = most;
    __syncthreads();
    const bool finite = max(max(bits[0], bits[1]), max(bits[2], bits[3])) < 0x7F800000u;
    const double factor = __hiloint2double(0x77F00000, 0);  // 2^896
    const double mean =
        finite ? ((sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid])) * factor / static_cast<double>(count) : 0.;
    double top = fabs(mean);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = fmax(fmax(tops[0], tops[1]), fmax(tops[2], tops[3]));
    const float scale = static_cast<float>(top / 127.);
    double code = scale > 0.f ? rint(mean / static_cast<double>(scale)) : 0.;
    code = fmin(fmax(code, -127.), 127.);
    a.codes[static_cast<int64_t>(page) * 128 + tid] = static_cast<int8_t>(static_cast<int>(code));
    if (tid == 0) {
      a.scale[page] = finite ? scale : __uint_as_float(0x7FC00000u);
      if (!finite) raise_status(status, LIDX_DEV_NAN);
    }
  }
}

}  // namespace

cudaError_t launch_block_pool(const lidx_block_pool_args &a, void *ws, cudaStream_t st) {
  // the lens are on the device: enough CTAs to fill the machine, each striding over its sequence's blocks
  const int per_seq = std::max(1, std::min(a.keys.max_pages, (16 * 148 + a.B - 1) / a.B));
  return launch_kernel(block_pool_kernel, dim3(per_seq, a.B), dim3(kThreads), 0, st,
                       (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.keys), static_cast<uint32_t *>(ws));
}

}  // namespace lidx

// Summaries of the blocks (pages) of a paged index-key cache: the mean key as
// 8-bit codes under one scale, for the block selection's cheap score.
//
// One CTA of four warps takes a block at a time.  A warp's loads are 16 bytes a
// lane of one plane: a row's RoPE dims (or a whole bf16 / fp32 row) take 8 (16,
// 32) lanes, its E4M3 codes 4, its E2M1 codes 4 of 8 bytes; the loads of 64 rows are
// dealt out to the warps and are all in flight before the first is used.  A
// lane sums its dims over its rows in 64 bits, the lanes that hold the same
// dims add up by halves (each step sends one half and keeps the other), the
// warps' sums meet in shared memory, and 128 threads finish one dim each.
//
// The sums are in 64 bits so that a mean next to a code's border rounds as the
// formula says, whatever the order of its sum.  Conversions would bound the
// kernel, so there are none: a value's bits moved into a double's fields
// without re-biasing the exponent are the value times a fixed power of two
// (subnormals included): 2^-896 for fp32 and bf16, 2^-1016 for E4M3 and
// 2^-1022 for E2M1, whose block scale then enters as the factor of a fused
// multiply-add.  Everything is summed as values times 2^-896.
#include <algorithm>

#include "paged.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// bits of a code's fields at the top of x (sign at bit 31) -> a double's upper word
template <int kShift, uint32_t kMask>
__device__ __forceinline__ double field_double(uint32_t x) {
  return __hiloint2double(static_cast<int>((static_cast<int32_t>(x) >> kShift) & kMask), 0);
}

// Dims of a lane's load of a plane, and its bytes (a bf16 plane is also the RoPE dims').
template <int kFmt>
struct Plane {
  static constexpr int kDims = kFmt == LIDX_F32 ? 4 : kFmt == LIDX_BF16 ? 8 : 16;
  static constexpr int kBytes = kFmt == LIDX_E2M1 ? 8 : 16;
};

// s += the dims in w, times their block's factor; `bad` notices what is not finite
template <int kFmt, int kDims>
__device__ __forceinline__ void accumulate(double (&s)[kDims], const uint4 &w, double factor, uint32_t &bad) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  if constexpr (kFmt == LIDX_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      bad = max(bad, x[i] & 0x7FFFFFFFu);
      s[i] += __hiloint2double(static_cast<int>((static_cast<int32_t>(x[i]) >> 3) & 0x8FFFFFFFu), static_cast<int>(x[i] << 29));
    }
  } else if constexpr (kFmt == LIDX_BF16) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      bad = __vmaxu2(bad, x[i] & 0x7FFF7FFFu);
      s[2 * i] += field_double<3, 0x8FFFFFFFu>(x[i] << 16);
      s[2 * i + 1] += field_double<3, 0x8FFFE000u>(x[i]);
    }
  } else if constexpr (kFmt == LIDX_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      bad |= ((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a code of NaN
#pragma unroll
      for (int k = 0; k < 4; k++) s[4 * i + k] = fma(field_double<7, 0x80FE0000u>(x[i] << (24 - 8 * k)), factor, s[4 * i + k]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
      for (int k = 0; k < 8; k++) s[8 * i + k] = fma(field_double<9, 0x80380000u>(x[i] << (28 - 4 * k)), factor, s[8 * i + k]);
  }
}

template <int kFmt>
__device__ __forceinline__ bool not_finite(uint32_t bad) {
  if (kFmt == LIDX_F32) return bad >= 0x7F800000u;
  if (kFmt == LIDX_BF16) return (bad & 0xFFFFu) >= 0x7F80u || (bad >> 16) >= 0x7F80u;
  return bad != 0u;
}

// One plane of a block: rows [0, count) of pool rows from p0 on, its dims' sums into sums[].
template <int kFmt, int kLanes>
__device__ __forceinline__ bool sum_plane(const uint8_t *base, int64_t pitch, const uint8_t *scales, int64_t ld_scale,
                                          int64_t p0, int count, double *sums) {
  using P = Plane<kFmt>;
  constexpr int kDims = P::kDims, kRowsPer = 32 / kLanes;   // rows of a load
  constexpr int kLoads = 64 / (kRowsPer * kWarps) > 0 ? 64 / (kRowsPer * kWarps) : 1;  // loads of a warp for 64 rows
  constexpr bool kScaled = kFmt == LIDX_E4M3 || kFmt == LIDX_E2M1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, piece = lane % kLanes;
  double s[kDims];
#pragma unroll
  for (int i = 0; i < kDims; i++) s[i] = 0.;
  uint32_t bad = 0u;
#pragma unroll 1
  for (int r0 = 0; r0 < count; r0 += kLoads * kWarps * kRowsPer) {
    uint4 w[kLoads];
    uint32_t sc[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int r = r0 + (i * kWarps + warp) * kRowsPer + lane / kLanes;
      w[i] = make_uint4(0, 0, 0, 0);
      sc[i] = 127u;
      if (r < count) {
        const uint8_t *src = base + (p0 + r) * pitch + piece * P::kBytes;
        if (P::kBytes == 16) {
          w[i] = fetch(reinterpret_cast<const uint4 *>(src));
        } else {
          const uint2 h = fetch(reinterpret_cast<const uint2 *>(src));
          w[i].x = h.x;
          w[i].y = h.y;
        }
        if (kFmt == LIDX_E4M3) sc[i] = fetch(scales + (p0 + r) * ld_scale);
        if (kFmt == LIDX_E2M1) sc[i] = fetch(scales + (p0 + r) * ld_scale + piece / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      double factor = 1.;
      if (kScaled) {
        // 2^(c - 127) * 2^1016 (E4M3) or 2^1022 (E2M1) * 2^-896: the exponent field of a double is c + 1016 or c + 1022
        factor = __hiloint2double(static_cast<int>((sc[i] + (kFmt == LIDX_E4M3 ? 1016u : 1022u)) << 20), 0);
        if (sc[i] == 0xFFu) bad |= 0x80u;
      }
      accumulate<kFmt>(s, w[i], factor, bad);
    }
  }
  // lanes with the same piece add up: each step sends one half of the dims and keeps the other
  int n = kDims, at = piece * kDims;
#pragma unroll
  for (int o = 16; o >= kLanes; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < kDims / 2; i++) {
        if (i < n) {
          const double send = up ? s[i] : s[n + i], keep = up ? s[n + i] : s[i];
          s[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
      }
      at += up ? n : 0;
    } else {
      s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
    }
  }
#pragma unroll
  for (int i = 0; i < kDims; i++)
    if (i < n) sums[at + i] = s[i];
  return not_finite<kFmt>(bad);
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads) block_pool_kernel(const lidx_block_pool_args a, int shift, uint32_t *status) {
  __shared__ double sums[kWarps][128];
  __shared__ double tops[kWarps];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  bool cut;
  const int32_t len = cut_len(fetch(a.len + b), a.keys, cut);
  if (cut && blockIdx.x == 0 && tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
  const int32_t rows = a.keys.page_rows;
  const int32_t first = a.first ? max(fetch(a.first + b), 0) : 0;
  const int32_t nb = static_cast<int32_t>((static_cast<int64_t>(len) + rows - 1) >> shift);
  const lidx_kv &kv = a.keys.rows;
  for (int64_t j = (first >> shift) + static_cast<int64_t>(blockIdx.x); j < nb && first < len; j += gridDim.x) {
    const int32_t page = fetch(a.keys.table + static_cast<int64_t>(b) * a.keys.ld_table + j);
    if (page < 0 || page >= a.keys.n_pages) {  // the same for the whole CTA
      if (tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
      continue;
    }
    const int count = static_cast<int>(min(static_cast<int64_t>(rows), len - (j << shift)));
    const int64_t p0 = static_cast<int64_t>(page) << shift;
    const uint8_t *data = static_cast<const uint8_t *>(kv.data);
    bool bad;
    if constexpr (kFmt == LIDX_F32 || kFmt == LIDX_BF16) {
      bad = sum_plane<kFmt, 128 / Plane<kFmt>::kDims>(data, kv.ld * (kFmt == LIDX_F32 ? 4 : 2), nullptr, 0, p0, count, sums[warp]);
    } else {
      bad = sum_plane<kFmt, 4>(data, kv.ld, kv.scale, kv.ld_scale, p0, count, sums[warp]);
      bad |= sum_plane<LIDX_BF16, 8>(static_cast<const uint8_t *>(kv.rope), 2 * kv.ld_rope, nullptr, 0, p0, count,
                                     sums[warp] + 64);
    }
    const bool finite = !__syncthreads_or(bad);
    const double unit = __hiloint2double(0x77F00000, 0);  // 2^896
    const double mean =
        finite ? ((sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid])) * unit / static_cast<double>(count) : 0.;
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
  const int per_seq = std::max(1, std::min(a.keys.max_pages, (8 * 148 + a.B - 1) / a.B));
  const dim3 grid(per_seq, a.B);
  auto kern = block_pool_kernel<LIDX_E2M1>;
  switch (a.keys.rows.dtype) {
    case LIDX_F32: kern = block_pool_kernel<LIDX_F32>; break;
    case LIDX_BF16: kern = block_pool_kernel<LIDX_BF16>; break;
    case LIDX_E4M3: kern = block_pool_kernel<LIDX_E4M3>; break;
  }
  return launch_kernel(kern, grid, dim3(kThreads), 0, st, (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.keys),
                       static_cast<uint32_t *>(ws));
}

}  // namespace lidx

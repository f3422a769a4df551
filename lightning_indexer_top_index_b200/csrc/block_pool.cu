// Summaries of the blocks (pages) of a paged index-key cache: the mean key as
// 8-bit codes under one scale, for the block selection's cheap score.
//
// A block is summed by a warp, or by the four warps of a CTA where there are
// few blocks.  A load is one plane's: four rows' RoPE dims, E4M3 or E2M1 codes
// (16, 8 or 4 bytes a lane), two bf16 rows or an fp32 one, with eight to
// sixteen loads in flight.  A lane sums its dims over its rows in 64 bits and
// the lanes that hold the same dims add up by halves (each step sends one half
// and keeps the other), which leaves every lane with four of the 128 dims.  The
// instructions bound the kernel, so a block's additions over lanes, its page
// lookup and its finish are done once by one warp where there are enough blocks:
// 4 x 125000 E4M3 rows take 20.6 us so against 28.4 with a CTA for each block
// (half of the time is the reading, at the copy rate).
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
// CTAs on an SM where a warp takes a block by itself: 4 x 125000 E4M3 rows took
// 24.9 us with the three that 160 registers allow, 20.8 with five, 22.6 with
// six, whose registers spill.
constexpr int kCtas = 5;
// From how many blocks on: 600 blocks of 64 E4M3 keys take 4.7 us with a CTA
// each and 5.6 with a warp, 1200 8.1 and 7.4, 2400 14.1 and 11.0.
constexpr int64_t kManyBlocks = 148 * 7;

// bits of a code's fields at the top of x (sign at bit 31) -> a double's upper word
template <int kShift, uint32_t kMask>
__device__ __forceinline__ double field_double(uint32_t x) {
  return __hiloint2double(static_cast<int>((static_cast<int32_t>(x) >> kShift) & kMask), 0);
}

// Dims of a lane's load of a plane, and its bytes (a bf16 plane is also the RoPE dims').
template <int kFmt>
struct Plane {
  static constexpr int kDims = kFmt == LIDX_F32 ? 4 : 8;
  static constexpr int kBytes = kFmt == LIDX_E2M1 ? 4 : kFmt == LIDX_E4M3 ? 8 : 16;
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
    for (int i = 0; i < 2; i++) {
      bad |= ((x[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a code of NaN
#pragma unroll
      for (int k = 0; k < 4; k++) s[4 * i + k] = fma(field_double<7, 0x80FE0000u>(x[i] << (24 - 8 * k)), factor, s[4 * i + k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; k++) s[k] = fma(field_double<9, 0x80380000u>(x[0] << (28 - 4 * k)), factor, s[k]);
  }
}

template <int kFmt>
__device__ __forceinline__ bool not_finite(uint32_t bad) {
  if (kFmt == LIDX_F32) return bad >= 0x7F800000u;
  if (kFmt == LIDX_BF16) return (bad & 0xFFFFu) >= 0x7F80u || (bad >> 16) >= 0x7F80u;
  return bad != 0u;
}

// One plane of a block: rows [0, count) of pool rows from p0 on, warp `member`
// of kTeam taking its share of them.  Leaves the lane with the sums of kOwn
// dims, from dim `at` of the plane on.
template <int kFmt, int kLanes, int kTeam, int kOwn>
__device__ __forceinline__ bool sum_plane(const uint8_t *base, int64_t pitch, const uint8_t *scales, int64_t ld_scale,
                                          int64_t p0, int count, int member, double (&own)[kOwn], int &at) {
  using P = Plane<kFmt>;
  constexpr int kDims = P::kDims, kRowsPer = 32 / kLanes;   // rows of a load
  constexpr int kMost = P::kBytes == 16 ? 8 : 16;           // loads in flight
  constexpr int kShare = 64 / (kRowsPer * kTeam);           // loads of a warp for 64 rows
  constexpr int kLoads = kShare < kMost ? kShare : kMost;
  constexpr bool kScaled = kFmt == LIDX_E4M3 || kFmt == LIDX_E2M1;
  static_assert(kOwn * 32 == kDims * kLanes, "the dims are dealt out over the lanes");
  const int lane = threadIdx.x & 31, piece = lane % kLanes;
  double s[kDims];
#pragma unroll
  for (int i = 0; i < kDims; i++) s[i] = 0.;
  uint32_t bad = 0u;
#pragma unroll 1
  for (int r0 = 0; r0 < count; r0 += kLoads * kTeam * kRowsPer) {
    uint4 w[kLoads];
    uint32_t sc[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int r = r0 + (i * kTeam + member) * kRowsPer + lane / kLanes;
      w[i] = make_uint4(0, 0, 0, 0);
      sc[i] = 127u;
      if (r < count) {
        const uint8_t *src = base + (p0 + r) * pitch + piece * P::kBytes;
        if (P::kBytes == 16) {
          w[i] = fetch(reinterpret_cast<const uint4 *>(src));
        } else if (P::kBytes == 8) {
          const uint2 h = fetch(reinterpret_cast<const uint2 *>(src));
          w[i].x = h.x;
          w[i].y = h.y;
        } else {
          w[i].x = fetch(reinterpret_cast<const uint32_t *>(src));
        }
        if (kFmt == LIDX_E4M3) sc[i] = fetch(scales + (p0 + r) * ld_scale);
        if (kFmt == LIDX_E2M1) sc[i] = fetch(scales + (p0 + r) * ld_scale + piece / 4);
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
  int n = kDims;
  at = piece * kDims;
#pragma unroll
  for (int o = 16; o >= kLanes; o >>= 1) {
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
  }
#pragma unroll
  for (int i = 0; i < kOwn; i++) own[i] = s[i];
  return not_finite<kFmt>(bad);
}

// fp32(top / 127), the quotient rounded to 64 bits first.  A product with 1/127
// is within two units in the last place of that quotient, so it rounds to the
// same fp32 unless a border between two of them is that near.
__device__ __forceinline__ float scale_of(double top) {
  double q = top * (1. / 127.);
  const int low = __double2loint(q) & 0x1FFFFFFF;
  if (abs(low - 0x10000000) < 8 || q < 0x1p-120) q = top / 127.;
  return static_cast<float>(q);
}

// rint(mean / scale).  With 1 / scale rounded to fp32 the quotient (at most 127
// and a rounding) is off by less than 2^-16, so it gives the same whole number
// unless it is that near to the middle between two.
__device__ __forceinline__ int code_of(double mean, float scale, float inv) {
  const double x = mean * static_cast<double>(inv);
  double code = rint(x);
  if (!(fabs(x - code) < 0.4999) || scale < 0x1p-100f || scale > 0x1p100f) code = scale > 0.f ? rint(mean / static_cast<double>(scale)) : 0.;
  return static_cast<int>(fmin(fmax(code, -127.), 127.));
}

template <int kFmt, int kTeam>
__global__ void __launch_bounds__(kThreads, kTeam > 1 ? 1 : kCtas) block_pool_kernel(const lidx_block_pool_args a, int shift, uint32_t *status) {
  __shared__ double sums[kTeam][128], tops[kTeam];
  static_assert(kTeam == 1 || kTeam == kWarps, "a warp, or the CTA");
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int member = kTeam > 1 ? warp : 0;
  pdl_trigger();
  pdl_wait();
  bool cut;
  const int32_t len = cut_len(fetch(a.len + b), a.keys, cut);
  if (cut && blockIdx.x == 0 && tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
  const int32_t rows = a.keys.page_rows;
  const int32_t first = a.first ? max(fetch(a.first + b), 0) : 0;
  if (first >= len) return;
  const int32_t nb = static_cast<int32_t>((static_cast<int64_t>(len) + rows - 1) >> shift);
  const lidx_kv &kv = a.keys.rows;
  const int64_t j0 = kTeam > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kWarps / kTeam);
  for (int64_t j = (first >> shift) + j0; j < nb; j += step) {
    const int32_t page = fetch(a.keys.table + static_cast<int64_t>(b) * a.keys.ld_table + j);
    if (page < 0 || page >= a.keys.n_pages) {  // the same for the whole team
      if (member == 0 && lane == 0) raise_status(status, LIDX_DEV_BOUNDS);
      continue;
    }
    const int count = static_cast<int>(min(static_cast<int64_t>(rows), len - (j << shift)));
    const int64_t p0 = static_cast<int64_t>(page) << shift;
    const uint8_t *data = static_cast<const uint8_t *>(kv.data);
    constexpr bool kQuant = kFmt == LIDX_E4M3 || kFmt == LIDX_E2M1;
    double own[4];  // dims at, at + 1, then at2, at2 + 1
    int at, at2;
    bool bad;
    if constexpr (kQuant) {
      double x[2], y[2];
      bad = sum_plane<kFmt, 8, kTeam>(data, kv.ld, kv.scale, kv.ld_scale, p0, count, member, x, at);
      bad |= sum_plane<LIDX_BF16, 8, kTeam>(static_cast<const uint8_t *>(kv.rope), 2 * kv.ld_rope, nullptr, 0, p0, count,
                                            member, y, at2);
      at2 += 64;
      own[0] = x[0];
      own[1] = x[1];
      own[2] = y[0];
      own[3] = y[1];
    } else {
      bad = sum_plane<kFmt, 128 / Plane<kFmt>::kDims, kTeam>(data, kv.ld * (kFmt == LIDX_F32 ? 4 : 2), nullptr, 0, p0,
                                                             count, member, own, at);
      at2 = at + 2;
    }
    // the lane's dims for the finish: all four, or, of a team, one for each of its threads
    constexpr int kMine = kTeam > 1 ? 1 : 4;
    double mean[kMine], top = 0.;
    bool finite;
    if constexpr (kTeam > 1) {
      sums[member][at] = own[0];
      sums[member][at + 1] = own[1];
      sums[member][at2] = own[2];
      sums[member][at2 + 1] = own[3];
      finite = !__syncthreads_or(bad);
      mean[0] = (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]);
    } else {
      finite = !__any_sync(0xFFFFFFFFu, bad);
#pragma unroll
      for (int k = 0; k < kMine; k++) mean[k] = own[k];
    }
    if (count & (count - 1)) {
#pragma unroll
      for (int k = 0; k < kMine; k++) mean[k] = mean[k] * 0x1p896 / static_cast<double>(count);
    } else {  // times 2^896 / count, exactly
      const double unit = __hiloint2double((0x3FF + 896 + 1 - __ffs(count)) << 20, 0);
#pragma unroll
      for (int k = 0; k < kMine; k++) mean[k] *= unit;
    }
#pragma unroll
    for (int k = 0; k < kMine; k++) {
      if (!finite) mean[k] = 0.;
      top = fmax(top, fabs(mean[k]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if constexpr (kTeam > 1) {
      if (lane == 0) tops[warp] = top;
      __syncthreads();  // (and the sums have been read)
      top = fmax(fmax(tops[0], tops[1]), fmax(tops[2], tops[3]));
    }
    const float scale = scale_of(top), inv = __frcp_rn(scale);
    int8_t *codes = a.codes + static_cast<int64_t>(page) * 128;
    if constexpr (kTeam > 1) {
      codes[tid] = static_cast<int8_t>(code_of(mean[0], scale, inv));
    } else {
      int code[4];
#pragma unroll
      for (int k = 0; k < 4; k++) code[k] = code_of(mean[k], scale, inv) & 0xFF;
      *reinterpret_cast<uint16_t *>(codes + at) = static_cast<uint16_t>(code[0] | (code[1] << 8));
      *reinterpret_cast<uint16_t *>(codes + at2) = static_cast<uint16_t>(code[2] | (code[3] << 8));
    }
    if (member == 0 && lane == 0) {
      a.scale[page] = finite ? scale : __uint_as_float(0x7FC00000u);
      if (!finite) raise_status(status, LIDX_DEV_NAN);
    }
  }
}

}  // namespace

cudaError_t launch_block_pool(const lidx_block_pool_args &a, void *ws, cudaStream_t st) {
  // The lens are on the device.  With `first` each sequence has a few blocks; without it up to as many as its table.
  // The CTAs fill the machine and stride over the blocks.
  const bool many = !a.first && static_cast<int64_t>(a.B) * a.keys.max_pages >= kManyBlocks;
  const int per_cta = many ? kWarps : 1;
  const int per_seq = std::max(1, std::min((a.keys.max_pages + per_cta - 1) / per_cta, ((many ? 4 * kCtas : 8) * 148 + a.B - 1) / a.B));
  const dim3 grid(per_seq, a.B);
  auto kern = many ? block_pool_kernel<LIDX_E2M1, 1> : block_pool_kernel<LIDX_E2M1, kWarps>;
  switch (a.keys.rows.dtype) {
    case LIDX_F32: kern = many ? block_pool_kernel<LIDX_F32, 1> : block_pool_kernel<LIDX_F32, kWarps>; break;
    case LIDX_BF16: kern = many ? block_pool_kernel<LIDX_BF16, 1> : block_pool_kernel<LIDX_BF16, kWarps>; break;
    case LIDX_E4M3: kern = many ? block_pool_kernel<LIDX_E4M3, 1> : block_pool_kernel<LIDX_E4M3, kWarps>; break;
  }
  return launch_kernel(kern, grid, dim3(kThreads), 0, st, (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.keys),
                       static_cast<uint32_t *>(ws));
}

}  // namespace lidx

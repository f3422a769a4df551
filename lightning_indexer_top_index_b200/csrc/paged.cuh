// Paged caches on the device: from a sequence's row to its pool row, and from
// stored rows to the values they stand for.
#pragma once

#include "kernels.cuh"

namespace lidx {

// A load of what the kernel before this one may have written (rows, tables,
// lens, queries).  An ordinary one, which stays behind pdl_wait: a read-only
// load (ld.global.nc) promises that nothing writes there while the kernel
// runs, and a programmatic dependent launch runs before its predecessor ends.
template <typename T>
__device__ __forceinline__ T fetch(const T *p) {
  return *p;
}

// Pool row of row r of sequence b, or -1 where the table has no page for it.
// r >= 0; shift = log2(page_rows).
__device__ __forceinline__ int32_t pool_row(const lidx_pages &c, int shift, int b, int32_t r) {
  const int32_t j = r >> shift;
  if (j >= c.max_pages) return -1;
  const int32_t page = fetch(c.table + static_cast<int64_t>(b) * c.ld_table + j);
  if (page < 0 || page >= c.n_pages) return -1;
  return (page << shift) | (r & (c.page_rows - 1));
}

// Rows of sequence b that exist: len cut to what the table can hold.
__device__ __forceinline__ int32_t cut_len(int32_t len, const lidx_pages &c, bool &cut) {
  const int32_t most = c.max_pages * c.page_rows;
  cut = len > most;
  return min(max(len, 0), most);
}

// E8M0 byte -> 2^(c-127) in both halves of a bf16 pair, exactly (c = 0 is the
// bf16 subnormal 2^-127; 255 is NaN).
__device__ __forceinline__ uint32_t e8m0_to_bf16x2(uint32_t c) {
  const uint32_t h = c == 0u ? 0x0040u : c == 0xFFu ? 0x7FC0u : c << 7;
  return h | (h << 16);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight E2M1 codes (the first in the low nibble) -> four bf16 pairs.  The
// magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 have the bf16 bytes
//   low 00 00 80 C0 00 40 80 C0   high 00 3F 3F 3F 40 40 40 40,
// which byte permutes look up with the codes themselves as selectors, four a
// time; the sign bits are permuted into the high bytes' top bits.
__device__ __forceinline__ void e2m1x8_to_bf16x2(uint32_t w, uint32_t (&o)[4]) {
  const uint32_t mag = w & 0x77777777u;
  const uint32_t even = (w << 4) & 0x80808080u, odd = w & 0x80808080u;  // signs of the low and the high nibbles
  const uint32_t lo0 = __byte_perm(0xC0800000u, 0xC0804000u, mag);
  const uint32_t lo1 = __byte_perm(0xC0800000u, 0xC0804000u, mag >> 16);
  const uint32_t hi0 = __byte_perm(0x3F3F3F00u, 0x40404040u, mag) | __byte_perm(even, odd, 0x5140);
  const uint32_t hi1 = __byte_perm(0x3F3F3F00u, 0x40404040u, mag >> 16) | __byte_perm(even, odd, 0x7362);
  o[0] = __byte_perm(lo0, hi0, 0x5140);
  o[1] = __byte_perm(lo0, hi0, 0x7362);
  o[2] = __byte_perm(lo1, hi1, 0x5140);
  o[3] = __byte_perm(lo1, hi1, 0x7362);
}

// Eight E2M1 codes times their block's scale 2^(c - 127) as four bf16 pairs,
// exactly.  The three magnitude bits of a code, put at bits 8..6 of a bf16, are
// its value times 2^-126 (0.5 is a bf16 subnormal there), so one product with
// 2^(126 + e) decodes and scales; scales above 2 take a second one.  A byte's two
// codes come to the two halves by a permute (their upper bytes by its sign mode,
// which gives zeros here), one product with 2^6 + 2^12 puts magnitude and sign
// bits in place, and a mask leaves only those: 19 instructions for eight values,
// half of them on the multiply pipe (the lookup above all runs on the integer
// pipe, which bounds the attention's loader).
struct E2m1Scale {
  uint32_t c, s1;
  bool two;  // with kWarp (a converged warp) the same in all lanes
  template <bool kWarp = true>
  __device__ __forceinline__ static E2m1Scale of(uint32_t code) {
    E2m1Scale s;
    s.c = code;
    s.s1 = (min(code, 128u) + 126u) * 0x00800080u;
    s.two = kWarp ? __any_sync(0xFFFFFFFFu, code > 128u) != 0 : code > 128u;
    return s;
  }
  __device__ __forceinline__ void expand(uint32_t w, uint32_t (&o)[4]) const {
    const uint32_t even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t y;
      asm("prmt.b32 %0, %1, %2, %3;" : "=r"(y) : "r"(even), "r"(odd), "r"(0xC480u + 0x1111u * i));
      o[i] = mul_bf16x2((y * 0x1040u) & 0x81C081C0u, s1);
    }
    if (two) {
      const uint32_t s2 = (c == 0xFFu ? 0x7FC0u : c > 128u ? (c - 1u) << 7 : 0x3F80u) * 0x00010001u;
#pragma unroll
      for (int i = 0; i < 4; i++) o[i] = mul_bf16x2(o[i], s2);
    }
  }
};

__device__ __forceinline__ float bf16x2_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16x2_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Dims [8t, 8t + 8) of a pool row: loaded first, made values (the exact
// products of code and scale, as fp32) later, so that many loads are in flight.
template <int kFmt>
struct Dims8 {
  uint4 w[kFmt == LIDX_F32 ? 2 : 1];
  uint32_t scale;
  bool codes;  // E4M3 or E2M1 codes, not 16- or 32-bit values

  __device__ __forceinline__ void load(const lidx_kv &kv, int64_t p, int t) {
    const int d0 = 8 * t, q = kv.dim - 64;
    codes = (kFmt == LIDX_E4M3 || kFmt == LIDX_E2M1) && d0 < q;
    if (kFmt == LIDX_F32) {
      const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const float *>(kv.data) + p * kv.ld + d0);
      w[0] = fetch(s);
      w[kFmt == LIDX_F32] = fetch(s + 1);
    } else if (!codes) {
      const uint16_t *s = kFmt == LIDX_BF16 ? static_cast<const uint16_t *>(kv.data) + p * kv.ld + d0
                                            : static_cast<const uint16_t *>(kv.rope) + p * kv.ld_rope + (d0 - q);
      w[0] = fetch(reinterpret_cast<const uint4 *>(s));
    } else {
      const uint8_t *data = static_cast<const uint8_t *>(kv.data) + p * kv.ld;
      if (kFmt == LIDX_E4M3) {
        const uint2 x = fetch(reinterpret_cast<const uint2 *>(data + d0));
        w[0].x = x.x;
        w[0].y = x.y;
      } else {
        w[0].x = fetch(reinterpret_cast<const uint32_t *>(data + d0 / 2));
      }
      scale = fetch(kv.scale + p * kv.ld_scale + d0 / (kFmt == LIDX_E4M3 ? 64 : 32));
    }
  }

  // as bf16, where the cache is not fp32: the exact products, rounded where the scale takes them out of its range
  __device__ __forceinline__ uint4 bf16() const {
    if (kFmt == LIDX_E4M3 && codes) {
      const uint32_t s = e8m0_to_bf16x2(scale);
      return make_uint4(mul_bf16x2(e4m3x2_to_bf16x2(w[0].x), s), mul_bf16x2(e4m3x2_to_bf16x2(w[0].x >> 16), s),
                        mul_bf16x2(e4m3x2_to_bf16x2(w[0].y), s), mul_bf16x2(e4m3x2_to_bf16x2(w[0].y >> 16), s));
    }
    if (kFmt == LIDX_E2M1 && codes) {
      uint32_t o[4];
      E2m1Scale::of<false>(scale).expand(w[0].x, o);
      return make_uint4(o[0], o[1], o[2], o[3]);
    }
    return w[0];
  }

  __device__ __forceinline__ void values(float (&v)[8]) const {
    if (kFmt == LIDX_F32) {
      const uint4 &y = w[kFmt == LIDX_F32];
      v[0] = __uint_as_float(w[0].x); v[1] = __uint_as_float(w[0].y);
      v[2] = __uint_as_float(w[0].z); v[3] = __uint_as_float(w[0].w);
      v[4] = __uint_as_float(y.x); v[5] = __uint_as_float(y.y);
      v[6] = __uint_as_float(y.z); v[7] = __uint_as_float(y.w);
      return;
    }
    uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
    float s = 1.f;
    if (codes) {
      if (kFmt == LIDX_E4M3) {
        x[3] = e4m3x2_to_bf16x2(x[1] >> 16);
        x[2] = e4m3x2_to_bf16x2(x[1]);
        x[1] = e4m3x2_to_bf16x2(x[0] >> 16);
        x[0] = e4m3x2_to_bf16x2(x[0]);
      } else {
        e2m1x8_to_bf16x2(w[0].x, x);
      }
      s = e8m0_to_f32(scale);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = bf16x2_lo(x[i]) * s;
      v[2 * i + 1] = bf16x2_hi(x[i]) * s;
    }
  }
};

}  // namespace lidx

// Shared pieces of the 8-bit (block-128) units: the format's arithmetic on the
// device, element access with any stride, buffer sizes and the quantisers' launchers.
//
// Format.  128 consecutive elements along the contracted axis share a scale
// S = 2^k, the smallest with k >= -126 and amax / S <= 448, amax taken over the
// block's finite elements; an element is E4M3FN(v / S), round to nearest even
// (v / S is exact: S is a power of two, and what underflows float32 is far
// below half of the smallest code).  NaN and infinities become the NaN code, so
// they reach exactly the results that contract over them.  The scale is kept as
// the E8M0 byte k + 127: the form in which gfx950's block-scaled MFMA takes it,
// so applying it costs no VALU work.
#pragma once

#include "asp_device.h"

namespace asp {

constexpr int kFp8Block = ASP_FP8_BLOCK;
constexpr uint32_t kFp8PadScale = 127;  // scale bytes of blocks past the last: 1.0

typedef int i32x8_t __attribute__((ext_vector_type(8)));

inline int64_t fp8_blocks(int64_t cols) { return (cols + kFp8Block - 1) / kFp8Block; }
inline int64_t fp8_pitch(int64_t cols) { return fp8_blocks(cols) * kFp8Block; }
inline size_t fp8_code_bytes(int64_t rows, int64_t cols) { return (size_t)rows * fp8_pitch(cols); }
inline size_t fp8_scale_bytes(int64_t rows, int64_t cols) {
  return (size_t)((fp8_blocks(cols) + 3) / 4) * rows * 4;
}
// a launch has fewer than 2^32 lanes
constexpr int64_t kMaxLanes = UINT32_MAX;
inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// ------------------------------------------------------------------- device

// max over the 16 lanes of a DPP row, in every lane (all lanes active)
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  return v;
}

// |v|'s bits, 0 for NaN and infinities: unsigned order is magnitude order
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// scale byte of a block whose largest finite magnitude has bits u: with
// amax = m 2^e, 1 <= m < 2, k = e - 8 while m <= 1.75 (448 = 1.75 * 2^8), else
// e - 7; zeros and subnormals fall to the smallest scale, 2^-126
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t u) {
  const int s = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(s, 1);
}

// 1 / S of a scale byte (1..247): exact
__device__ __forceinline__ float fp8_inverse(uint32_t byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}

// four values -> four codes (|v * inv| <= 448 for finite v: never saturates)
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float inv) {
  const float nan = __builtin_bit_cast(float, 0x7FC00000u);
  auto s = [&](float v) { return __builtin_fabsf(v) < __builtin_inff() ? v * inv : nan; };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(s(a), s(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(s(c), s(d), w, true);
  return (uint32_t)w;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) {
  return __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// 16 bytes at an address aligned to an element only: the memory takes any, and an
// aligned one costs the same as if it were known to be
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

// eight consecutive elements as they lie in memory
template <typename XT>
struct Raw {
  u32x4_t q[sizeof(XT) / 2];
};

// From element c of a row of `cols`; past its end r is not touched, its zeros stay.
// Where the row ends inside the eight, float32 is loaded element by element.  16-bit
// elements would have to be waited for to be paired: there the eight before the row's end
// are loaded, as every other lane does, and raw_settle puts them in place where they are
// used (element by element 16384 x 4094 took 298 us in the norms' backward, where 4096
// columns take 185; so 203.  The same in float32 costs registers: 640 x 3023 29 us for
// 24).  SHORT: a row of fewer than eight.
template <bool SHORT, typename XT>
__device__ __forceinline__ void raw_load(const XT* row, int c, int cols, Raw<XT>& r) {
  if (c >= cols) return;
  if constexpr (sizeof(XT) == 2 && !SHORT) {
    r.q[0] = *reinterpret_cast<const u32x4_e2*>(row + (uint32_t)min(c, cols - 8));
  } else if constexpr (sizeof(XT) == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = e < cols ? row[e] : 0u;
      r.q[0][e >> 1] = e & 1 ? r.q[0][e >> 1] | w << 16 : w;
    }
  } else {
    const XT* p = row + (uint32_t)c;
    const int left = cols - c;
    if (left >= 8) {
      r.q[0] = *reinterpret_cast<const u32x4_e4*>(p);
      r.q[1] = *reinterpret_cast<const u32x4_e4*>(p + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        r.q[e >> 2][e & 3] = e < left ? __builtin_bit_cast(uint32_t, p[e]) : 0u;
    }
  }
}

template <bool SHORT, typename XT>
__device__ __forceinline__ void raw_settle(int c, int cols, Raw<XT>& r) {
  if constexpr (sizeof(XT) == 2 && !SHORT) {
    const int over = -cols & 7;  // uniform: the elements before the row's last piece
    if (over == 0 || c + 8 <= cols) return;
    uint32_t w[5] = {r.q[0][0], r.q[0][1], r.q[0][2], r.q[0][3], 0u};
    auto move = [&](int n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = i + n < 4 ? w[i + n < 4 ? i + n : 4] : 0u;
    };
    if (over & 4) move(2);
    if (over & 2) move(1);
    if (over & 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_alignbit(w[i + 1], w[i], 16);
    r.q[0] = u32x4_t{w[0], w[1], w[2], w[3]};
  }
}

template <typename XT>
__device__ __forceinline__ void unpack(const Raw<XT>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t w = sizeof(XT) == 2 ? r.q[0][e >> 1] : r.q[(sizeof(XT) / 2 - 1) & (e >> 2)][e & 3];
    if constexpr (sizeof(XT) == 2)
      v[e] = e & 1 ? bf16_hi(w) : bf16_lo(w);
    else
      v[e] = __builtin_bit_cast(float, w);
  }
}

// both, for any row
template <typename XT>
__device__ __forceinline__ void raw_get(const XT* row, int c, int cols, Raw<XT>& r) {
  if (cols >= 8) {
    raw_load<false>(row, c, cols, r);
    raw_settle<false>(c, cols, r);
  } else {
    raw_load<true>(row, c, cols, r);
  }
}

// eight elements from element c of a row of `cols`, 0 past its end
template <typename XT>
__device__ __forceinline__ void load8(const XT* row, int c, int cols, float (&v)[8]) {
  Raw<XT> r = {};
  raw_get(row, c, cols, r);
  unpack(r, v);
}

// ------------------------------------------------------------- host helpers

inline int32_t check_io_dtype(int32_t dtype, const char* name) {
  if (dtype != ASP_F32 && dtype != ASP_BF16) return fail(ASP_ERR_ARG, "%s=%d", name, dtype);
  return ASP_OK;
}

// a caller's matrix: element-aligned, any row stride of at least `cols`
inline int32_t check_matrix(const void* p, int32_t dtype, int64_t cols, int64_t ld,
                            const char* name) {
  if (!p) return fail(ASP_ERR_ARG, "%s is NULL", name);
  if ((uintptr_t)p % (dtype == ASP_BF16 ? 2 : 4))
    return fail(ASP_ERR_ALIGN, "%s is not aligned to its elements", name);
  if (ld < cols || ld > INT32_MAX)
    return fail(ASP_ERR_SHAPE, "row stride %lld of %s outside [%lld, 2^31)", (long long)ld, name,
                (long long)cols);
  return ASP_OK;
}

// rows >= 0 and 1 <= cols <= 2^20 of a matrix in the 8-bit format
inline int32_t check_fp8_dims(int64_t rows, int64_t cols, const char* rn, const char* cn) {
  if (rows < 0 || rows > INT32_MAX)
    return fail(ASP_ERR_SHAPE, "%s=%lld outside [0, 2^31)", rn, (long long)rows);
  if (cols < 1 || cols > kMaxK)
    return fail(ASP_ERR_SHAPE, "%s=%lld outside [1, %lld]", cn, (long long)cols, (long long)kMaxK);
  return ASP_OK;
}

inline int32_t check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return ASP_OK;
  if (!ws) return fail(ASP_ERR_ARG, "workspace is NULL");
  if (((uintptr_t)ws & 255u) != 0) return fail(ASP_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (have < need) return fail(ASP_ERR_WORKSPACE, "workspace: %zu bytes, need %zu", have, need);
  return ASP_OK;
}

// ----------------------------------------------- launchers (arguments checked)

int32_t fp8_quantize_rows(const void* in, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                          uint8_t* codes, uint8_t* scales, hipStream_t st);

// One matrix for the tile quantiser: any of the row form, the transposed form
// and the column sums; square: one scale for each 128 x 128 tile.
struct Fp8TileJob {
  const void* in;
  int64_t rows, cols, ld;
  uint8_t *codes, *scales;      // row form, or NULL
  uint8_t *codes_t, *scales_t;  // transposed form, or NULL
  float* sums;                  // [ceil(rows / 128)][cols] partial column sums, or NULL
  int32_t dtype, square;
};
int32_t fp8_quantize_tiles(int n, const Fp8TileJob* jobs, hipStream_t st);

}  // namespace asp

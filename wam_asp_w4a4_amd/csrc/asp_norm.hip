// Gated norms around a transformer block, forward and backward:
//
//   p = post(y)                       none, RMS or layer norm, times post_w
//   h = alpha x + gate[g] p           the residual stream, held in x's type
//   n = (pre(h) w + b) (1 + scale[g]) + shift[g]
//
// pre and post: v r with v = h (RMS) or h - mean (layer), r = 1/sqrt(mean v^2 +
// eps).  The tables gate, scale and shift have one row for each sequence g of
// packed rows offsets[g] .. offsets[g + 1] - 1.  n leaves in float32, bf16 or the
// 8-bit block-128 format.  Statistics, sums and all intermediate values are
// float32; h is rounded to x's type before the second norm reads it, so that the
// backward, which reads h again, sees the same values.
//
// Everything is bound by memory: a row is read once, held in registers through
// both norms (a layer norm's variance is summed around its mean, not as a
// difference of squares), and written once.  A workgroup walks a strip of
// consecutive rows; the tables of the strip's sequence stay in registers (read anew
// for each row they cost more cache traffic than the row itself).  T threads share a
// row, 8 columns each (E = 2: 16, above 8192 columns): a thread's share of a row, its
// tables and its column sums are then few enough registers for four waves a SIMD.
// 16384 x 4096 bf16, RMS before a modulated layer norm: 116 us, 4.6 TB/s; to 8-bit codes
// 112 us, in float32 214 (5.0 TB/s).  The backward of two RMS norms 168 us (4.8 TB/s), and
// 15 us of column sums where a table's or weight's gradient is wanted.
#include "asp_fp8.h"

namespace asp {
namespace {

struct NormArgs {
  const void *x, *y;
  const float *post_w, *gate, *pre_w, *pre_b, *scale, *shift;
  const int32_t* offsets;
  void *h, *n;
  uint8_t* n_scales;
  int64_t ldx, ldy, ldh, ldn, ldt;
  float alpha, eps;
  int M, C, G, post, pre, n_dtype, rows;  // rows: of a strip
  int zero;  // bits: the first, the second output's rows of no sequence become zeros
  // backward
  const void *dh, *dn;
  void *dx, *dy;
  float* part;  // [strips + G][3][C]
  int64_t lddh, lddn, lddx, lddy;
};

// sum over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row16_sum(float v) {
  auto add = [](float a, auto ctrl) {
    return a + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                             0, __builtin_bit_cast(int, a), decltype(ctrl)::value,
                                             0xf, 0xf, false));
  };
  v = add(v, std::integral_constant<int, 0x128>{});
  v = add(v, std::integral_constant<int, 0x124>{});
  v = add(v, std::integral_constant<int, 0x122>{});
  return add(v, std::integral_constant<int, 0x121>{});
}

__device__ __forceinline__ float wave_sum(float v) {
  const int w = __builtin_bit_cast(int, row16_sum(v));
  auto lane = [&](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(w, l)); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// sums of N values over the workgroup, in every lane; `slot` alternates, so that
// the one barrier also separates a slot's reads from its next writes
constexpr int kMaxSums = 4;
typedef float SumsLds[2][kMaxSums][16];
template <int T, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], SumsLds& lds, int& slot) {
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = wave_sum(s[i]);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) lds[slot][i][wave] = s[i];
    __syncthreads();
    const int w = lane & 15;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = row16_sum(w < W ? lds[slot][i][w < W ? w : 0] : 0.0f);
    slot ^= 1;
  }
}

// the sequence of a row: the first g with offsets[g + 1] > row, G if there is none
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int G, int row) {
  int lo = 0, hi = G;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// a thread's columns of a row: E chunks of 8, chunk e at column 8 (e T + t)
template <typename XT, int E, int T, bool SHORT>
__device__ __forceinline__ void row_load(const void* p, int64_t row, int64_t ld, int C, int t,
                                         Raw<XT> (&r)[E]) {
  const XT* base = static_cast<const XT*>(p) + row * ld;  // uniform
#pragma unroll
  for (int e = 0; e < E; ++e) {
    raw_load<SHORT>(base, (e * T + t) * 8, C, r[e]);
  }
}

template <int E, int T, bool SHORT>
__device__ __forceinline__ void table(const float* p, int64_t at, int C, int t, float other,
                                      float (&v)[E][8]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e * T + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[e][k] = other;
    if (!p || c >= C) continue;
    Raw<float> r = {};
    raw_load<SHORT>(p + at, c, C, r);
    raw_settle<SHORT>(c, C, r);
    unpack(r, v[e]);
  }
}

// 8 values to element c of a row that ends after `left` more
__device__ __forceinline__ void store8(void* p, int64_t row, uint32_t c, bool bf16, int left,
                                       const float (&v)[8]) {
  if (bf16) {
    uint16_t* d = static_cast<uint16_t*>(p) + row + c;
    if (left >= 8) {
      *reinterpret_cast<u32x4_e2*>(d) = u32x4_t{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
                                                bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) d[k] = bf16_rne(v[k]);
    }
  } else {
    float* d = static_cast<float*>(p) + row + c;
    if (left >= 8) {
      auto bits = [&](int k) { return __builtin_bit_cast(uint32_t, v[k]); };
      *reinterpret_cast<u32x4_e4*>(d) = u32x4_t{bits(0), bits(1), bits(2), bits(3)};
      *reinterpret_cast<u32x4_e4*>(d + 4) = u32x4_t{bits(4), bits(5), bits(6), bits(7)};
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) d[k] = v[k];
    }
  }
}

// a row of no sequence becomes zeros
template <int E, int T>
__device__ __forceinline__ void zero_row(void* p, int64_t row, bool bf16, int C, int t) {
  const float v[8] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e * T + t) * 8;
    store8(p, row, c, bf16, C - c, v);
  }
}

// f(e, k) for each of a thread's columns
template <int E, typename F>
__device__ __forceinline__ void each(F&& f) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) f(e, k);
}

// v - mean; columns past C become 0
template <int E, int T>
__device__ __forceinline__ void centre(float (&v)[E][8], float mean, int C, int t) {
  each<E>([&](int e, int k) { v[e][k] = (e * T + t) * 8 + k < C ? v[e][k] - mean : 0.0f; });
}

// the row's one square root and division are IEEE ones: they cost nothing
__device__ __forceinline__ float inverse_deviation(float squares, int C, float eps) {
  return 1.0f / sqrtf(squares / (float)C + eps);
}

// v -> the normed row
template <int E, int T>
__device__ __forceinline__ void normalise(float (&v)[E][8], int kind, int C, float eps, int t,
                                          SumsLds& lds, int& slot) {
  float s[1];
  if (kind == ASP_NORM_LAYER) {
    s[0] = 0.0f;
    each<E>([&](int e, int k) { s[0] += v[e][k]; });
    row_sums<T, 1>(s, lds, slot);
    centre<E, T>(v, s[0] / (float)C, C, t);
  }
  s[0] = 0.0f;
  each<E>([&](int e, int k) { s[0] = __builtin_fmaf(v[e][k], v[e][k], s[0]); });
  row_sums<T, 1>(s, lds, slot);
  const float r = inverse_deviation(s[0], C, eps);
  each<E>([&](int e, int k) { v[e][k] *= r; });
}

template <typename XT, int T, int E, bool SHORT = false>
__global__ void __launch_bounds__(T) k_norm_gate(const NormArgs a) {
  __shared__ SumsLds lds;
  const int t = threadIdx.x;
  int slot = 0;
  const int64_t r0 = (int64_t)blockIdx.x * a.rows;
  const int64_t r1 = min(r0 + a.rows, (int64_t)a.M);
  const int pitch = (a.C + kFp8Block - 1) / kFp8Block * kFp8Block;
  float gp[E][8], pa[E][8], pc[E][8];
  Raw<XT> nx[E] = {}, ny[E] = {};
  auto fetch = [&](int64_t row) {
    row_load<XT, E, T, SHORT>(a.x, row, a.ldx, a.C, t, nx);
    if (a.y) row_load<XT, E, T, SHORT>(a.y, row, a.ldy, a.C, t, ny);
  };
  const int64_t first = a.offsets ? max(r0, (int64_t)a.offsets[0]) : r0;
  if (first < r1) fetch(first);
  int64_t row = first, end = 0;
  for (; row < r1; ++row) {
    if (row == first || row >= end) {
      int g = 0;
      if (a.offsets) {
        g = sequence_of(a.offsets, a.G, (int)row);
        if (g >= a.G) break;  // behind the last sequence
        end = a.offsets[g + 1];
      } else {
        end = a.M;
      }
      float u[E][8], w[E][8];
      // v gate post_w, and (v w + b) (1 + scale) + shift = v pa + pc
      table<E, T, SHORT>(a.gate, g * a.ldt, a.C, t, 1.0f, gp);
      table<E, T, SHORT>(a.post_w, 0, a.C, t, 1.0f, u);
      each<E>([&](int e, int k) { gp[e][k] *= u[e][k]; });
      table<E, T, SHORT>(a.pre_w, 0, a.C, t, 1.0f, pa);
      table<E, T, SHORT>(a.pre_b, 0, a.C, t, 0.0f, pc);
      table<E, T, SHORT>(a.scale, g * a.ldt, a.C, t, 0.0f, u);
      table<E, T, SHORT>(a.shift, g * a.ldt, a.C, t, 0.0f, w);
      each<E>([&](int e, int k) {
        pa[e][k] *= 1.0f + u[e][k];
        pc[e][k] = __builtin_fmaf(pc[e][k], 1.0f + u[e][k], w[e][k]);
      });
    }
    float v[E][8], p[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      raw_settle<SHORT>((e * T + t) * 8, a.C, nx[e]);
      raw_settle<SHORT>((e * T + t) * 8, a.C, ny[e]);
      unpack(nx[e], v[e]);
      unpack(ny[e], p[e]);
    }
    if (row + 1 < r1) fetch(row + 1);
    if (a.post != ASP_NORM_NONE) normalise<E, T>(p, a.post, a.C, a.eps, t, lds, slot);
    each<E>([&](int e, int k) {
      v[e][k] = a.y ? __builtin_fmaf(p[e][k], gp[e][k], a.alpha * v[e][k]) : a.alpha * v[e][k];
    });
    if constexpr (sizeof(XT) == 2)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const uint32_t w = bf16x2_rne(v[e][k], v[e][k + 1]);
          v[e][k] = bf16_lo(w);
          v[e][k + 1] = bf16_hi(w);
        }
    if (a.h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * T + t) * 8;
        store8(a.h, row * a.ldh, c, sizeof(XT) == 2, a.C - c, v[e]);
      }
    if (a.pre == ASP_NORM_NONE) continue;
    normalise<E, T>(v, a.pre, a.C, a.eps, t, lds, slot);
    each<E>([&](int e, int k) { v[e][k] = __builtin_fmaf(v[e][k], pa[e][k], pc[e][k]); });
    if (a.n_dtype != ASP_E4M3) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * T + t) * 8;
        store8(a.n, row * a.ldn, c, a.n_dtype == ASP_BF16, a.C - c, v[e]);
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {  // 16 lanes hold one block of 128
      const int c = (e * T + t) * 8;
      uint32_t u = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (c + k >= a.C) v[e][k] = 0.0f;  // pads the block
        u = max(u, finite_bits(v[e][k]));
      }
      const uint32_t s = fp8_scale_byte(row16_max(u));
      const float inv = fp8_inverse(s);
      if (c < pitch)
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(a.n) + row * pitch + c) =
            u32x2_t{fp8_pack4(v[e][0], v[e][1], v[e][2], v[e][3], inv),
                    fp8_pack4(v[e][4], v[e][5], v[e][6], v[e][7], inv)};
      if ((t & 15) == 0 && c < (pitch + 511) / 512 * 512)
        a.n_scales[((int64_t)(c >> 9) * a.M + row) * 4 + ((c >> 7) & 3)] =
            (uint8_t)(c < pitch ? s : kFp8PadScale);
    }
  }
  if (!a.zero) return;
  // the strip's rows in front of the first sequence, then those behind the last
  for (int64_t z = r0 < first ? r0 : row; z < r1; z = z + 1 == first ? max(row, first) : z + 1) {
    if (a.zero & 1) zero_row<E, T>(a.h, z * a.ldh, sizeof(XT) == 2, a.C, t);
    if (!(a.zero & 2)) continue;
    if (a.n_dtype != ASP_E4M3) {
      zero_row<E, T>(a.n, z * a.ldn, a.n_dtype == ASP_BF16, a.C, t);
      continue;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * T + t) * 8;
      if (c < pitch)
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(a.n) + z * pitch + c) = u32x2_t{0u, 0u};
      if ((t & 15) == 0 && c < (pitch + 511) / 512 * 512)
        a.n_scales[((int64_t)(c >> 9) * a.M + z) * 4 + ((c >> 7) & 3)] = (uint8_t)kFp8PadScale;
    }
  }
}

// Backward.  With m the mean that the pre norm takes off (0 for RMS), v = (h - m) r
// and g = dn w (1 + scale):
//   dh' = dh + r (g - [layer] mean g - v mean(g v)),   dx = alpha dh'
// and the same form through the post norm for dy from dh' gate post_w.  mean(g v)
// is r mean(g (h - m)), so the sums of h's and y's squares and of g and g (h - m)
// are taken together: three barriers a row (two without a layer norm).
//
// Every gradient of a table or weight follows from three column sums over each
// sequence's rows, S1 = sum dn, S2 = sum dn v, S3 = sum dh' q (q the normed y, or
// y): a strip keeps them in registers and writes them once for each sequence it
// touches, to slot strip + g (strips and sequences both advance along the rows,
// so no two pairs share one).  k_norm_sums adds the strips in order: the
// results do not depend on scheduling.
template <typename XT, typename NT, int T, int E, bool SHORT = false>
__global__ void __launch_bounds__(T, 4) k_norm_gate_back(const NormArgs a) {
  // the next row's loads in flight where a row is few enough registers (8192 x 8192 bf16,
  // layer norms: 193 against 226 us); in float32 they cost registers that other waves
  // need (16384 x 4096: 368 against 346 us)
  constexpr bool kAhead = E == 1 && sizeof(XT) == 2;
  __shared__ SumsLds lds;
  const int t = threadIdx.x;
  int slot = 0;
  const int strip = blockIdx.x;
  const int64_t r0 = (int64_t)strip * a.rows;
  const int64_t r1 = min(r0 + a.rows, (int64_t)a.M);
  const float rc = 1.0f / (float)a.C;
  const bool pre = a.pre != ASP_NORM_NONE, post = a.post != ASP_NORM_NONE;
  const bool prel = a.pre == ASP_NORM_LAYER, postl = a.post == ASP_NORM_LAYER;
  float gp[E][8], pa[E][8], s1[E][8], s2[E][8], s3[E][8];
  auto flush = [&](int g) {
    const int64_t at = (int64_t)(strip + g) * 3 * a.C;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t c = (uint32_t)(e * T + t) * 8u;
      store8(a.part, at, c, false, a.C - (int)c, s1[e]);
      store8(a.part, at + a.C, c, false, a.C - (int)c, s2[e]);
      store8(a.part, at + 2 * (int64_t)a.C, c, false, a.C - (int)c, s3[e]);
    }
  };
  // dh and y not given, and h and dn without a pre norm, stay 0
  Raw<XT> rd[E] = {}, ry[E] = {}, rh[E] = {};
  Raw<NT> rn[E] = {};
  auto fetch = [&](int64_t row) {
    if (a.dh) row_load<XT, E, T, SHORT>(a.dh, row, a.lddh, a.C, t, rd);
    if (a.y) row_load<XT, E, T, SHORT>(a.y, row, a.ldy, a.C, t, ry);
    if (pre) {
      row_load<XT, E, T, SHORT>(a.h, row, a.ldh, a.C, t, rh);
      row_load<NT, E, T, SHORT>(a.dn, row, a.lddn, a.C, t, rn);
    }
  };
  const int64_t first = a.offsets ? max(r0, (int64_t)a.offsets[0]) : r0;
  if constexpr (kAhead)
    if (first < r1) fetch(first);
  int g = -1;
  int64_t row = first, end = 0;
  for (; row < r1; ++row) {
    if (row == first || row >= end) {
      if (g >= 0 && a.part) flush(g);
      g = 0;
      if (a.offsets) {
        g = sequence_of(a.offsets, a.G, (int)row);
        if (g >= a.G) {
          g = -1;
          break;
        }
        end = a.offsets[g + 1];
      } else {
        end = a.M;
      }
      float u[E][8];
      table<E, T, SHORT>(a.gate, g * a.ldt, a.C, t, 1.0f, gp);
      table<E, T, SHORT>(a.post_w, 0, a.C, t, 1.0f, u);
      each<E>([&](int e, int k) { gp[e][k] *= u[e][k]; });
      table<E, T, SHORT>(a.pre_w, 0, a.C, t, 1.0f, pa);
      table<E, T, SHORT>(a.scale, g * a.ldt, a.C, t, 0.0f, u);
      each<E>([&](int e, int k) {
        pa[e][k] *= 1.0f + u[e][k];
        s1[e][k] = s2[e][k] = s3[e][k] = 0.0f;
      });
    }
    if constexpr (!kAhead) fetch(row);
    float d[E][8], v[E][8], n[E][8], q[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * T + t) * 8;
      raw_settle<SHORT>(c, a.C, rd[e]);
      raw_settle<SHORT>(c, a.C, ry[e]);
      raw_settle<SHORT>(c, a.C, rh[e]);
      raw_settle<SHORT>(c, a.C, rn[e]);
      unpack(rd[e], d[e]);
      unpack(ry[e], q[e]);
      unpack(rh[e], v[e]);
      unpack(rn[e], n[e]);
    }
    if (kAhead && row + 1 < r1) fetch(row + 1);
    if (prel || postl) {
      float s[2] = {0.0f, 0.0f};
      each<E>([&](int e, int k) {
        s[0] += v[e][k];
        s[1] += q[e][k];
      });
      row_sums<T, 2>(s, lds, slot);
      if (prel) centre<E, T>(v, s[0] * rc, a.C, t);
      if (postl) centre<E, T>(q, s[1] * rc, a.C, t);
    }
    // squares of h - m and y - m, and of g = dn pa its sum and product with h - m
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    each<E>([&](int e, int k) {
      const float gv = n[e][k] * pa[e][k];
      s[0] = __builtin_fmaf(v[e][k], v[e][k], s[0]);
      s[1] = __builtin_fmaf(q[e][k], q[e][k], s[1]);
      s[2] = __builtin_fmaf(gv, v[e][k], s[2]);
      s[3] += gv;
    });
    row_sums<T, 4>(s, lds, slot);
    if (pre) {
      const float r = inverse_deviation(s[0], a.C, a.eps);
      const float c1 = prel ? s[3] * rc : 0.0f, c2 = r * s[2] * rc;
      each<E>([&](int e, int k) {
        const float vv = v[e][k] * r;
        s1[e][k] += n[e][k];
        s2[e][k] = __builtin_fmaf(n[e][k], vv, s2[e][k]);
        d[e][k] += r * (__builtin_fmaf(n[e][k], pa[e][k], -c1) - vv * c2);
      });
    }
    if (a.dx)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * T + t) * 8;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = a.alpha * d[e][k];
        store8(a.dx, row * a.lddx, c, sizeof(XT) == 2, a.C - c, o);
      }
    if (!a.y) continue;
    float r = 1.0f;
    if (post) {
      r = inverse_deviation(s[1], a.C, a.eps);
      each<E>([&](int e, int k) { q[e][k] *= r; });
    }
    each<E>([&](int e, int k) {
      s3[e][k] = __builtin_fmaf(d[e][k], q[e][k], s3[e][k]);
      d[e][k] *= gp[e][k];
    });
    if (!a.dy) continue;
    if (post) {
      float z[2] = {0.0f, 0.0f};
      centre<E, T>(d, 0.0f, a.C, t);  // columns past C count as 0 in the sums
      each<E>([&](int e, int k) {
        z[0] += d[e][k];
        z[1] = __builtin_fmaf(d[e][k], q[e][k], z[1]);
      });
      row_sums<T, 2>(z, lds, slot);
      const float c1 = postl ? z[0] * rc : 0.0f, c2 = z[1] * rc;
      each<E>([&](int e, int k) { d[e][k] = r * (d[e][k] - c1 - q[e][k] * c2); });
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * T + t) * 8;
      store8(a.dy, row * a.lddy, c, sizeof(XT) == 2, a.C - c, d[e]);
    }
  }
  if (g >= 0 && a.part) flush(g);
  if (!a.zero) return;
  for (int64_t z = r0 < first ? r0 : row; z < r1; z = z + 1 == first ? max(row, first) : z + 1) {
    if (a.zero & 1) zero_row<E, T>(a.dx, z * a.lddx, sizeof(XT) == 2, a.C, t);
    if (a.zero & 2) zero_row<E, T>(a.dy, z * a.lddy, sizeof(XT) == 2, a.C, t);
  }
}

struct SumArgs {
  float* part;
  const float *post_w, *gate, *pre_w, *pre_b, *scale;
  const int32_t* offsets;
  float *d_post_w, *d_gate, *d_pre_w, *d_pre_b, *d_scale, *d_shift;
  int64_t ldt, ldd, slots;
  int M, C, G, rows;
};

// The strips' column sums of sequence blockIdx.y, for 16 columns a workgroup: 16
// threads of a column take its strips in turn, and the first adds them in order.
// Their sequence's table gradients are written here; for the weights, which sum
// over the sequences, S1 (1 + scale), S2 (1 + scale) and S3 gate go behind the
// strips' slots, or are the results themselves when there is one sequence.
__global__ void __launch_bounds__(256) k_norm_sums(const SumArgs a) {
  __shared__ float lds[3][16][17];
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4, g = blockIdx.y;
  const int c = blockIdx.x * 16 + col;
  const bool in = c < a.C;
  int64_t o0 = 0, o1 = a.M;
  if (a.offsets) {
    o0 = max(a.offsets[g], 0);
    o1 = min(a.offsets[g + 1], a.M);
  }
  float s[3] = {0.0f, 0.0f, 0.0f};
  if (in && o0 < o1) {
    const int64_t k1 = (o1 - 1) / a.rows;
    const float* p = a.part + (o0 / a.rows + lane + g) * 3 * a.C + c;
#pragma unroll 4
    for (int64_t k = o0 / a.rows + lane; k <= k1; k += 16) {
#pragma unroll
      for (int i = 0; i < 3; ++i) s[i] += p[(int64_t)i * a.C];
      p += (int64_t)48 * a.C;
    }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) lds[i][lane][col] = s[i];
  __syncthreads();
  if (lane != 0 || !in) return;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    s[i] = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s[i] += lds[i][k][col];
  }
  const float w = a.pre_w ? a.pre_w[c] : 1.0f, b = a.pre_b ? a.pre_b[c] : 0.0f;
  const float m = a.scale ? 1.0f + a.scale[g * a.ldt + c] : 1.0f;
  const float gt = a.gate ? a.gate[g * a.ldt + c] : 1.0f;
  const float pw = a.post_w ? a.post_w[c] : 1.0f;
  if (a.d_shift) a.d_shift[g * a.ldd + c] = s[0];
  if (a.d_scale) a.d_scale[g * a.ldd + c] = s[1] * w + s[0] * b;
  if (a.d_gate) a.d_gate[g * a.ldd + c] = s[2] * pw;
  if (a.G == 1) {
    if (a.d_pre_b) a.d_pre_b[c] = s[0] * m;
    if (a.d_pre_w) a.d_pre_w[c] = s[1] * m;
    if (a.d_post_w) a.d_post_w[c] = s[2] * gt;
  } else {
    float* d = a.part + (a.slots + g) * 3 * a.C + c;
    d[0] = s[0] * m;
    d[a.C] = s[1] * m;
    d[2 * (int64_t)a.C] = s[2] * gt;
  }
}

// the weights' gradients: the sequences' sums in order
__global__ void __launch_bounds__(64) k_norm_weight_sums(const SumArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= a.C) return;
  float s[3] = {0.0f, 0.0f, 0.0f};
  const float* p = a.part + a.slots * 3 * a.C + c;
#pragma unroll 4
  for (int g = 0; g < a.G; ++g) {
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i] += p[(int64_t)i * a.C];
    p += 3 * (int64_t)a.C;
  }
  if (a.d_pre_b) a.d_pre_b[c] = s[0];
  if (a.d_pre_w) a.d_pre_w[c] = s[1];
  if (a.d_post_w) a.d_post_w[c] = s[2];
}

// ----------------------------------------------------------------- host side

constexpr int kMaxNormC = 16384;

// threads of a row
int row_threads(int64_t C) {
  return C <= 512 ? 64 : C <= 1024 ? 128 : C <= 2048 ? 256 : C <= 4096 ? 512 : 1024;
}

// Rows of a strip: as many strips as four waves a SIMD make resident at once, so that
// all of them run from the first row to the last; one row each where there are fewer.
int strip_rows(int64_t M, int64_t C) {
  const int64_t s = 256 * 16 * 64 / row_threads(C);
  return M > s ? (int)((M + s - 1) / s) : 1;
}

// The backward's: two at least where the strips' column sums, 12 bytes a column, are
// what it waits for (a replayed call, float32: 2000 x 1024 38 -> 31 us, 4000 x 500 37 -> 31;
// below half a million columns the second row costs more: 256 x 1024 19 against 20.5).
int back_rows(int64_t M, int64_t C) {
  return M * C < (1 << 19) ? strip_rows(M, C) : std::max(strip_rows(M, C), 2);
}

int64_t strips(int64_t M, int64_t rows) { return (M + rows - 1) / rows; }

int32_t check_norm(int32_t dtype, int64_t M, int64_t C, int32_t post, int32_t pre, int32_t G,
                   const int32_t* offsets, int64_t ldt, float eps) {
  ASP_TRY(check_io_dtype(dtype, "dtype"));
  if (M < 0 || M > INT32_MAX) return fail(ASP_ERR_SHAPE, "M=%lld outside [0, 2^31)", (long long)M);
  if (C < 1 || C > kMaxNormC)
    return fail(ASP_ERR_SHAPE, "C=%lld outside [1, %d]", (long long)C, kMaxNormC);
  if (post < ASP_NORM_NONE || post > ASP_NORM_LAYER) return fail(ASP_ERR_ARG, "post=%d", post);
  if (pre < ASP_NORM_NONE || pre > ASP_NORM_LAYER) return fail(ASP_ERR_ARG, "pre=%d", pre);
  if (G < 1 || G > 65535) return fail(ASP_ERR_SHAPE, "G=%d outside [1, 65535]", G);
  if (!offsets && G != 1) return fail(ASP_ERR_ARG, "offsets is NULL with G=%d sequences", G);
  if (offsets && ((uintptr_t)offsets & 3)) return fail(ASP_ERR_ALIGN, "offsets is not 4-byte aligned");
  if (ldt < (G > 1 ? C : 0) || ldt > INT32_MAX)
    return fail(ASP_ERR_SHAPE, "table stride %lld", (long long)ldt);
  if (!(eps >= 0.0f) || eps > 1.0f) return fail(ASP_ERR_ARG, "eps=%g outside [0, 1]", eps);
  return ASP_OK;
}

int32_t check_vec(const float* p, const char* name) {
  return (uintptr_t)p & 3 ? fail(ASP_ERR_ALIGN, "%s is not aligned to its elements", name) : ASP_OK;
}

template <typename XT>
int32_t launch_norm(const NormArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)strips(a.M, a.rows));
  if (a.C < 8) k_norm_gate<XT, 64, 1, true><<<grid, 64, 0, st>>>(a);
  else if (a.C <= 512) k_norm_gate<XT, 64, 1><<<grid, 64, 0, st>>>(a);
  else if (a.C <= 1024) k_norm_gate<XT, 128, 1><<<grid, 128, 0, st>>>(a);
  else if (a.C <= 2048) k_norm_gate<XT, 256, 1><<<grid, 256, 0, st>>>(a);
  else if (a.C <= 4096) k_norm_gate<XT, 512, 1><<<grid, 512, 0, st>>>(a);
  else if (a.C <= 8192) k_norm_gate<XT, 1024, 1><<<grid, 1024, 0, st>>>(a);
  else k_norm_gate<XT, 1024, 2><<<grid, 1024, 0, st>>>(a);
  return launch_status("norm");
}

template <typename XT, typename NT>
int32_t launch_back(const NormArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)strips(a.M, a.rows));
  if (a.C < 8) k_norm_gate_back<XT, NT, 64, 1, true><<<grid, 64, 0, st>>>(a);
  else if (a.C <= 512) k_norm_gate_back<XT, NT, 64, 1><<<grid, 64, 0, st>>>(a);
  else if (a.C <= 1024) k_norm_gate_back<XT, NT, 128, 1><<<grid, 128, 0, st>>>(a);
  else if (a.C <= 2048) k_norm_gate_back<XT, NT, 256, 1><<<grid, 256, 0, st>>>(a);
  else if (a.C <= 4096) k_norm_gate_back<XT, NT, 512, 1><<<grid, 512, 0, st>>>(a);
  else if (a.C <= 8192) k_norm_gate_back<XT, NT, 1024, 1><<<grid, 1024, 0, st>>>(a);
  else k_norm_gate_back<XT, NT, 1024, 2><<<grid, 1024, 0, st>>>(a);
  return launch_status("norm backward");
}

}  // namespace
}  // namespace asp

using namespace asp;

extern "C" {

int32_t asp_norm_gate(const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t dtype,
                      int64_t M, int64_t C, float alpha, int32_t post, const float* post_w,
                      const float* gate, int32_t pre, const float* pre_w, const float* pre_b,
                      const float* scale, const float* shift, int64_t ldt, int32_t G,
                      const int32_t* offsets, float eps, void* h, int64_t ldh, void* n,
                      int32_t n_dtype, int64_t ldn, uint8_t* n_scales, int32_t zero,
                      void* stream) {
  clear_error();
  ASP_TRY(check_norm(dtype, M, C, post, pre, G, offsets, ldt, eps));
  if (!y && (post != ASP_NORM_NONE || gate))
    return fail(ASP_ERR_ARG, "a post norm or gate without y");
  if (pre == ASP_NORM_NONE && (pre_w || pre_b || scale || shift || n))
    return fail(ASP_ERR_ARG, "pre norm arguments without a pre norm");
  if (pre == ASP_NORM_NONE && !h) return fail(ASP_ERR_ARG, "neither h nor n is asked for");
  if (post == ASP_NORM_NONE && post_w) return fail(ASP_ERR_ARG, "post_w without a post norm");
  if (zero < 0 || zero > 3 || (M > 0 && ((zero & 1 && !h) || (zero & 2 && !n))))
    return fail(ASP_ERR_ARG, "zero=%d", zero);
  if (n_dtype != ASP_F32 && n_dtype != ASP_BF16 && n_dtype != ASP_E4M3)
    return fail(ASP_ERR_ARG, "n_dtype=%d", n_dtype);
  if (M == 0) return ASP_OK;
  ASP_TRY(check_matrix(x, dtype, C, ldx, "x"));
  if (y) ASP_TRY(check_matrix(y, dtype, C, ldy, "y"));
  if (h) ASP_TRY(check_matrix(h, dtype, C, ldh, "h"));
  if (pre != ASP_NORM_NONE) {
    if (n_dtype == ASP_E4M3) {
      ASP_TRY(check_ptr(n, "n", true));
      ASP_TRY(check_ptr(n_scales, "n_scales", true));
    } else {
      ASP_TRY(check_matrix(n, n_dtype, C, ldn, "n"));
    }
  }
  ASP_TRY(check_vec(post_w, "post_w"));
  ASP_TRY(check_vec(gate, "gate"));
  ASP_TRY(check_vec(pre_w, "pre_w"));
  ASP_TRY(check_vec(pre_b, "pre_b"));
  ASP_TRY(check_vec(scale, "scale"));
  ASP_TRY(check_vec(shift, "shift"));
  NormArgs a = {};
  a.x = x; a.y = y; a.post_w = post_w; a.gate = gate; a.pre_w = pre_w; a.pre_b = pre_b;
  a.scale = scale; a.shift = shift; a.offsets = offsets; a.h = h; a.n = n; a.n_scales = n_scales;
  a.ldx = ldx; a.ldy = ldy; a.ldh = ldh; a.ldn = ldn; a.ldt = ldt; a.alpha = alpha; a.eps = eps;
  a.M = (int)M; a.C = (int)C; a.G = G; a.post = post; a.pre = pre; a.n_dtype = n_dtype;
  a.rows = strip_rows(M, C);
  a.zero = zero;
  const hipStream_t st = (hipStream_t)stream;
  return dtype == ASP_BF16 ? launch_norm<uint16_t>(a, st) : launch_norm<float>(a, st);
}

int32_t asp_norm_gate_backward_workspace_bytes(int64_t M, int64_t C, int32_t G, size_t* bytes) {
  clear_error();
  ASP_TRY(check_norm(ASP_F32, M, C, 0, 0, 1, nullptr, 0, 0.0f));
  if (G < 1 || G > 65535) return fail(ASP_ERR_SHAPE, "G=%d outside [1, 65535]", G);
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  // a slot for each pair of a strip and a sequence that it touches, and the sequences' sums
  *bytes = up256((size_t)(strips(M, back_rows(M, C)) + G + (G > 1 ? G : 0)) * 3 * C * 4);
  return ASP_OK;
}

int32_t asp_norm_gate_backward(const void* dh, int64_t lddh, const void* dn, int64_t lddn,
                               int32_t dn_dtype, const void* h, int64_t ldh, const void* y,
                               int64_t ldy, int32_t dtype, int64_t M, int64_t C, float alpha,
                               int32_t post, const float* post_w, const float* gate, int32_t pre,
                               const float* pre_w, const float* pre_b, const float* scale,
                               int64_t ldt, int32_t G, const int32_t* offsets, float eps, void* dx,
                               int64_t lddx, void* dy, int64_t lddy, int32_t zero,
                               float* d_post_w, float* d_gate, float* d_pre_w, float* d_pre_b,
                               float* d_scale, float* d_shift, int64_t ldd, void* workspace,
                               size_t workspace_bytes, void* stream) {
  clear_error();
  ASP_TRY(check_norm(dtype, M, C, post, pre, G, offsets, ldt, eps));
  ASP_TRY(check_io_dtype(dn_dtype, "dn_dtype"));
  if (!y && (post != ASP_NORM_NONE || gate || dy || d_gate))
    return fail(ASP_ERR_ARG, "a post norm, gate or dy without y");
  if (post == ASP_NORM_NONE && (post_w || d_post_w))
    return fail(ASP_ERR_ARG, "post_w without a post norm");
  if (pre == ASP_NORM_NONE &&
      (dn || pre_w || pre_b || scale || d_pre_w || d_pre_b || d_scale || d_shift))
    return fail(ASP_ERR_ARG, "pre norm arguments without a pre norm");
  if (ldd < (G > 1 ? C : 0) || ldd > INT32_MAX)
    return fail(ASP_ERR_SHAPE, "table gradient stride %lld", (long long)ldd);
  if (zero < 0 || zero > 3 || (M > 0 && ((zero & 1 && !dx) || (zero & 2 && !dy))))
    return fail(ASP_ERR_ARG, "zero=%d", zero);
  const bool sums = d_post_w || d_gate || d_pre_w || d_pre_b || d_scale || d_shift;
  if (!sums && !dx && !dy) return ASP_OK;
  if (M > 0) {
    if (dh) ASP_TRY(check_matrix(dh, dtype, C, lddh, "dh"));
    if (y) ASP_TRY(check_matrix(y, dtype, C, ldy, "y"));
    if (dx) ASP_TRY(check_matrix(dx, dtype, C, lddx, "dx"));
    if (dy) ASP_TRY(check_matrix(dy, dtype, C, lddy, "dy"));
    if (pre != ASP_NORM_NONE) {
      ASP_TRY(check_matrix(h, dtype, C, ldh, "h"));
      ASP_TRY(check_matrix(dn, dn_dtype, C, lddn, "dn"));
    } else if (!dh) {
      return fail(ASP_ERR_ARG, "neither dh nor dn is given");
    }
  }
  const float* vecs[] = {post_w, gate, pre_w, pre_b, scale, d_post_w, d_gate, d_pre_w, d_pre_b,
                         d_scale, d_shift};
  for (const float* p : vecs) ASP_TRY(check_vec(p, "a table or its gradient"));
  size_t need = 0;
  if (sums) ASP_TRY(asp_norm_gate_backward_workspace_bytes(M, C, G, &need));
  ASP_TRY(check_workspace(workspace, workspace_bytes, need));
  const hipStream_t st = (hipStream_t)stream;
  NormArgs a = {};
  a.y = y; a.post_w = post_w; a.gate = gate; a.pre_w = pre_w; a.pre_b = pre_b; a.scale = scale;
  a.offsets = offsets; a.h = const_cast<void*>(h); a.ldy = ldy; a.ldh = ldh; a.ldt = ldt;
  a.alpha = alpha; a.eps = eps; a.M = (int)M; a.C = (int)C; a.G = G; a.post = post; a.pre = pre;
  a.dh = dh; a.dn = dn; a.dx = dx; a.dy = dy; a.lddh = lddh; a.lddn = lddn; a.lddx = lddx;
  a.lddy = lddy; a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.rows = back_rows(M, C);
  a.zero = zero;
  if (M > 0) {
    const bool n16 = dn_dtype == ASP_BF16;
    if (dtype == ASP_BF16)
      ASP_TRY((n16 ? launch_back<uint16_t, uint16_t>(a, st) : launch_back<uint16_t, float>(a, st)));
    else
      ASP_TRY((n16 ? launch_back<float, uint16_t>(a, st) : launch_back<float, float>(a, st)));
  }
  if (!sums) return ASP_OK;
  SumArgs k = {};
  k.part = static_cast<float*>(workspace);
  k.post_w = post_w; k.gate = gate; k.pre_w = pre_w; k.pre_b = pre_b; k.scale = scale;
  k.offsets = offsets; k.d_post_w = d_post_w; k.d_gate = d_gate; k.d_pre_w = d_pre_w;
  k.d_pre_b = d_pre_b; k.d_scale = d_scale; k.d_shift = d_shift; k.ldt = ldt; k.ldd = ldd;
  k.M = (int)M; k.C = (int)C; k.G = G; k.rows = a.rows; k.slots = strips(M, a.rows) + G;
  k_norm_sums<<<dim3((unsigned)((C + 15) / 16), (unsigned)G), 256, 0, st>>>(k);
  if (G > 1 && (d_pre_w || d_pre_b || d_post_w))
    k_norm_weight_sums<<<dim3((unsigned)((C + 63) / 64)), 64, 0, st>>>(k);
  return launch_status("norm column sums");
}

}  // extern "C"

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
// difference of squares), and written once.  A workgroup (or, up to 1024
// columns, a wave) walks a strip of consecutive rows, so that the tables stay
// in registers too: read anew for each row they would cost more cache traffic
// than the row itself.
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
  // backward
  const void *dh, *dn;
  void *dx, *dy;
  float* part;  // [strips + G][3][C]
  int64_t lddh, lddn, lddx, lddy;
};

// T: the lanes that share a row (64: one wave); E: 8-column chunks of a lane
constexpr int threads_of(int T) { return T < 256 ? 256 : T; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// sums of two values over the row's lanes, in every lane; `slot` alternates, so
// that one barrier separates a slot's reads from its next writes
template <int T>
__device__ __forceinline__ void row_sums(float& a, float& b, float (&lds)[2][2][16], int& slot) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      lds[slot][0][wave] = a;
      lds[slot][1][wave] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      a += lds[slot][0][w];
      b += lds[slot][1][w];
    }
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

template <int E, int T>
__device__ __forceinline__ void table(const float* p, int64_t at, int C, int t, float other,
                                      float (&v)[E][8]) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = (e * T + t) * 8 + k;
      v[e][k] = p && c < C ? p[at + c] : other;
    }
}

template <typename XT, int E, int T, bool VEC>
__device__ __forceinline__ void row_load(const void* p, int64_t row, int64_t ld, int C, int t,
                                         float (&v)[E][8]) {
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = (e * T + t) * 8;
    load8<VEC>(static_cast<const XT*>(p) + row * ld + c, C - c, v[e]);
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t at, bool bf16, int left, const float (&v)[8]) {
  if (left <= 0) return;
  if (bf16) {
    uint16_t* d = static_cast<uint16_t*>(p) + at;
    if constexpr (VEC) {
      *reinterpret_cast<u32x4_t*>(d) = u32x4_t{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]),
                                               bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) d[k] = bf16_rne(v[k]);
    }
  } else {
    float* d = static_cast<float*>(p) + at;
    if constexpr (VEC) {
      *reinterpret_cast<f32x4_t*>(d) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_t*>(d + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) d[k] = v[k];
    }
  }
}

// v - mean; columns past C become 0
template <int E, int T>
__device__ __forceinline__ void centre(float (&v)[E][8], float mean, int C, int t) {
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[e][k] = (e * T + t) * 8 + k < C ? v[e][k] - mean : 0.0f;
}

template <int E>
__device__ __forceinline__ float sum_of(const float (&v)[E][8]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[e][k];
  return s;
}

template <int E>
__device__ __forceinline__ float dot_of(const float (&a)[E][8], const float (&b)[E][8]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = __builtin_fmaf(a[e][k], b[e][k], s);
  return s;
}

// v -> the normed row; returns r.  (IEEE square root and division: the row's
// one r costs nothing.)
template <int E, int T>
__device__ __forceinline__ float normalise(float (&v)[E][8], int kind, int C, float eps, int t,
                                           float (&lds)[2][2][16], int& slot) {
  float s, unused = 0.0f;
  if (kind == ASP_NORM_LAYER) {
    s = sum_of<E>(v);
    row_sums<T>(s, unused, lds, slot);
    centre<E, T>(v, s / (float)C, C, t);
  }
  s = dot_of<E>(v, v);
  unused = 0.0f;
  row_sums<T>(s, unused, lds, slot);
  const float r = 1.0f / sqrtf(s / (float)C + eps);
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[e][k] *= r;
  return r;
}

template <typename XT, int T, int E, bool VEC>
__global__ void __launch_bounds__(threads_of(T)) k_norm_gate(const NormArgs a) {
  __shared__ float lds[2][2][16];
  const int t = threadIdx.x % T;
  int slot = 0;
  const int strip = blockIdx.x * (threads_of(T) / T) + threadIdx.x / T;
  const int64_t r0 = (int64_t)strip * a.rows;
  const int64_t r1 = min(r0 + a.rows, (int64_t)a.M);
  const int pitch = (a.C + kFp8Block - 1) / kFp8Block * kFp8Block;
  float gp[E][8], pa[E][8], pc[E][8];
  int64_t begin = 0, end = 0;
  for (int64_t row = r0; row < r1; ++row) {
    if (row == r0 || row >= end) {
      int g = 0;
      if (a.offsets) {
        g = sequence_of(a.offsets, a.G, (int)row);
        if (g >= a.G) break;  // behind the last sequence
        begin = a.offsets[g];
        end = a.offsets[g + 1];
      } else {
        end = a.M;
      }
      float u[E][8];
      table<E, T>(a.gate, g * a.ldt, a.C, t, 1.0f, gp);
      if (a.post != ASP_NORM_NONE) {
        table<E, T>(a.post_w, 0, a.C, t, 1.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) gp[e][k] *= u[e][k];
      }
      // (v w + b) (1 + scale) + shift = v pa + pc
      table<E, T>(a.pre_w, 0, a.C, t, 1.0f, pa);
      table<E, T>(a.pre_b, 0, a.C, t, 0.0f, pc);
      if (a.scale) {
        table<E, T>(a.scale, g * a.ldt, a.C, t, 0.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            pa[e][k] *= 1.0f + u[e][k];
            pc[e][k] *= 1.0f + u[e][k];
          }
      }
      if (a.shift) {
        table<E, T>(a.shift, g * a.ldt, a.C, t, 0.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) pc[e][k] += u[e][k];
      }
    }
    if (row < begin) continue;  // in front of the first sequence
    float v[E][8], p[E][8];
    row_load<XT, E, T, VEC>(a.x, row, a.ldx, a.C, t, v);
    if (a.y) row_load<XT, E, T, VEC>(a.y, row, a.ldy, a.C, t, p);
    if (a.y) {
      if (a.post != ASP_NORM_NONE) normalise<E, T>(p, a.post, a.C, a.eps, t, lds, slot);
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[e][k] = __builtin_fmaf(p[e][k], gp[e][k], a.alpha * v[e][k]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[e][k] *= a.alpha;
    }
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
        store8<VEC>(a.h, row * a.ldh + c, sizeof(XT) == 2, a.C - c, v[e]);
      }
    if (a.pre == ASP_NORM_NONE) continue;
    normalise<E, T>(v, a.pre, a.C, a.eps, t, lds, slot);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[e][k] = __builtin_fmaf(v[e][k], pa[e][k], pc[e][k]);
    if (a.n_dtype != ASP_E4M3) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * T + t) * 8;
        store8<VEC>(a.n, row * a.ldn + c, a.n_dtype == ASP_BF16, a.C - c, v[e]);
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {  // 16 lanes hold one block of 128
      const int c = (e * T + t) * 8;
      uint32_t u = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (c + k >= a.C) v[e][k] = 0.0f;  // pads the last block (pc may be anything there)
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
}

// Backward.  With v the normed h (deviation 1/r), g = dn w (1 + scale):
//   dh' = dh + r (g - [layer] mean g - v mean(g v)),   dx = alpha dh'
// and the same form through the post norm for dy from dh' gate post_w.  Every
// gradient of a table or weight follows from three column sums over each
// sequence's rows, S1 = sum dn, S2 = sum dn v, S3 = sum dh' q (q the normed y, or
// y): a strip keeps them in registers and writes them once for each sequence it
// touches, to slot strip + g (strips and sequences both advance along the rows,
// so no two pairs share one).  k_norm_sums adds the strips in order: the
// results do not depend on scheduling.
template <typename XT, typename NT, int T, int E, bool VEC>
__global__ void __launch_bounds__(threads_of(T)) k_norm_gate_back(const NormArgs a) {
  __shared__ float lds[2][2][16];
  const int t = threadIdx.x % T;
  int slot = 0;
  const int strip = blockIdx.x * (threads_of(T) / T) + threadIdx.x / T;
  const int64_t r0 = (int64_t)strip * a.rows;
  const int64_t r1 = min(r0 + a.rows, (int64_t)a.M);
  float s1[E][8], s2[E][8], s3[E][8];
  auto clear = [&]() {
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) s1[e][k] = s2[e][k] = s3[e][k] = 0.0f;
  };
  auto flush = [&](int g) {
    float* d = a.part + (int64_t)(strip + g) * 3 * a.C;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = (e * T + t) * 8 + k;
        if (c < a.C) {
          d[c] = s1[e][k];
          d[a.C + c] = s2[e][k];
          d[2 * (int64_t)a.C + c] = s3[e][k];
        }
      }
  };
  int g = -1;
  int64_t begin = 0, end = 0;
  clear();
  for (int64_t row = r0; row < r1; ++row) {
    if (row == r0 || row >= end) {
      if (g >= 0 && a.part) flush(g);
      clear();
      g = 0;
      if (a.offsets) {
        g = sequence_of(a.offsets, a.G, (int)row);
        if (g >= a.G) {
          g = -1;
          break;
        }
        begin = a.offsets[g];
        end = a.offsets[g + 1];
      } else {
        end = a.M;
      }
    }
    if (row < begin) continue;
    float d[E][8], v[E][8], n[E][8], q[E][8];
    if (a.dh) row_load<XT, E, T, VEC>(a.dh, row, a.lddh, a.C, t, d);
    if (a.y) row_load<XT, E, T, VEC>(a.y, row, a.ldy, a.C, t, q);
    if (!a.dh)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) d[e][k] = 0.0f;
    if (a.pre != ASP_NORM_NONE) {
      row_load<XT, E, T, VEC>(a.h, row, a.ldh, a.C, t, v);
      row_load<NT, E, T, VEC>(a.dn, row, a.lddn, a.C, t, n);
      const float r = normalise<E, T>(v, a.pre, a.C, a.eps, t, lds, slot);
      float u[E][8];
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s1[e][k] += n[e][k];
          s2[e][k] = __builtin_fmaf(n[e][k], v[e][k], s2[e][k]);
        }
      if (a.pre_w) {
        table<E, T>(a.pre_w, 0, a.C, t, 1.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) n[e][k] *= u[e][k];
      }
      if (a.scale) {
        table<E, T>(a.scale, g * a.ldt, a.C, t, 0.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) n[e][k] *= 1.0f + u[e][k];
      }
      float c1 = a.pre == ASP_NORM_LAYER ? sum_of<E>(n) : 0.0f, c2 = dot_of<E>(n, v);
      row_sums<T>(c1, c2, lds, slot);
      c1 /= (float)a.C;
      c2 /= (float)a.C;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) d[e][k] += r * (n[e][k] - c1 - v[e][k] * c2);
    }
    if (a.dx)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (e * T + t) * 8;
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = a.alpha * d[e][k];
        store8<VEC>(a.dx, row * a.lddx + c, sizeof(XT) == 2, a.C - c, o);
      }
    if (!a.y) continue;
    float r = 1.0f;
    if (a.post != ASP_NORM_NONE) r = normalise<E, T>(q, a.post, a.C, a.eps, t, lds, slot);
    float u[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) s3[e][k] = __builtin_fmaf(d[e][k], q[e][k], s3[e][k]);
    if (!a.dy) continue;
    if (a.gate) {
      table<E, T>(a.gate, g * a.ldt, a.C, t, 1.0f, u);
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) d[e][k] *= u[e][k];
    }
    if (a.post != ASP_NORM_NONE) {
      if (a.post_w) {
        table<E, T>(a.post_w, 0, a.C, t, 1.0f, u);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) d[e][k] *= u[e][k];
      }
      centre<E, T>(d, 0.0f, a.C, t);  // columns past C count as 0 in the sums
      float c1 = a.post == ASP_NORM_LAYER ? sum_of<E>(d) : 0.0f, c2 = dot_of<E>(d, q);
      row_sums<T>(c1, c2, lds, slot);
      c1 /= (float)a.C;
      c2 /= (float)a.C;
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) d[e][k] = r * (d[e][k] - c1 - q[e][k] * c2);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (e * T + t) * 8;
      store8<VEC>(a.dy, row * a.lddy + c, sizeof(XT) == 2, a.C - c, d[e]);
    }
  }
  if (g >= 0 && a.part) flush(g);
}

struct SumArgs {
  const float* part;
  const float *post_w, *gate, *pre_w, *pre_b, *scale;
  const int32_t* offsets;
  float *d_post_w, *d_gate, *d_pre_w, *d_pre_b, *d_scale, *d_shift;
  int64_t ldt, ldd;
  int M, C, G, rows, post;
};

// 16 columns a workgroup; 16 lanes of a column take its strips in turn
__global__ void __launch_bounds__(256) k_norm_sums(const SumArgs a) {
  __shared__ float lds[3][16][17];
  const int col = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  const bool in = c < a.C;
  float w1 = 0.0f, w2 = 0.0f, w3 = 0.0f;  // sums over the sequences (first 16 threads)
  for (int g = 0; g < a.G; ++g) {
    int64_t o0 = 0, o1 = a.M;
    if (a.offsets) {
      o0 = max(a.offsets[g], 0);
      o1 = min(a.offsets[g + 1], a.M);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (in && o0 < o1)
      for (int64_t k = o0 / a.rows + part; k <= (o1 - 1) / a.rows; k += 16) {
        const float* p = a.part + (k + g) * 3 * a.C + c;
#pragma unroll
        for (int i = 0; i < 3; ++i) s[i] += p[(int64_t)i * a.C];
      }
#pragma unroll
    for (int i = 0; i < 3; ++i) lds[i][part][col] = s[i];
    __syncthreads();
    if (part == 0 && in) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        s[i] = 0.0f;
        for (int k = 0; k < 16; ++k) s[i] += lds[i][k][col];
      }
      const float w = a.pre_w ? a.pre_w[c] : 1.0f, b = a.pre_b ? a.pre_b[c] : 0.0f;
      const float m = a.scale ? 1.0f + a.scale[g * a.ldt + c] : 1.0f;
      const float gt = a.gate ? a.gate[g * a.ldt + c] : 1.0f;
      const float pw = a.post != ASP_NORM_NONE && a.post_w ? a.post_w[c] : 1.0f;
      if (a.d_shift) a.d_shift[g * a.ldd + c] = s[0];
      if (a.d_scale) a.d_scale[g * a.ldd + c] = s[1] * w + s[0] * b;
      if (a.d_gate) a.d_gate[g * a.ldd + c] = s[2] * pw;
      w1 += s[0] * m;
      w2 += s[1] * m;
      w3 += s[2] * gt;
    }
    __syncthreads();
  }
  if (part != 0 || !in) return;
  if (a.d_pre_b) a.d_pre_b[c] = w1;
  if (a.d_pre_w) a.d_pre_w[c] = w2;
  if (a.d_post_w) a.d_post_w[c] = w3;
}

// ----------------------------------------------------------------- host side

constexpr int kMaxNormC = 16384;

int strips_wanted(int64_t C) { return C <= 1024 ? 4096 : 1024; }
int strip_rows(int64_t M, int64_t C) {
  const int64_t s = strips_wanted(C);
  return (int)((M + s - 1) / s);
}

int32_t check_norm(int32_t dtype, int64_t M, int64_t C, int32_t post, int32_t pre, int32_t G,
                   const int32_t* offsets, int64_t ldt, float eps) {
  ASP_TRY(check_io_dtype(dtype, "dtype"));
  if (M < 0 || M > INT32_MAX) return fail(ASP_ERR_SHAPE, "M=%lld outside [0, 2^31)", (long long)M);
  if (C < 1 || C > kMaxNormC)
    return fail(ASP_ERR_SHAPE, "C=%lld outside [1, %d]", (long long)C, kMaxNormC);
  if (post < ASP_NORM_NONE || post > ASP_NORM_LAYER) return fail(ASP_ERR_ARG, "post=%d", post);
  if (pre < ASP_NORM_NONE || pre > ASP_NORM_LAYER) return fail(ASP_ERR_ARG, "pre=%d", pre);
  if (G < 1 || G > 65536) return fail(ASP_ERR_SHAPE, "G=%d outside [1, 65536]", G);
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

template <typename XT, bool VEC>
int32_t launch_norm(const NormArgs& a, hipStream_t st) {
  const int64_t strips = (a.M + a.rows - 1) / a.rows;
  const dim3 one((unsigned)strips), four((unsigned)((strips + 3) / 4));
  if (a.C <= 512) k_norm_gate<XT, 64, 1, VEC><<<four, 256, 0, st>>>(a);
  else if (a.C <= 1024) k_norm_gate<XT, 64, 2, VEC><<<four, 256, 0, st>>>(a);
  else if (a.C <= 2048) k_norm_gate<XT, 256, 1, VEC><<<one, 256, 0, st>>>(a);
  else if (a.C <= 4096) k_norm_gate<XT, 256, 2, VEC><<<one, 256, 0, st>>>(a);
  else if (a.C <= 8192) k_norm_gate<XT, 512, 2, VEC><<<one, 512, 0, st>>>(a);
  else k_norm_gate<XT, 512, 4, VEC><<<one, 512, 0, st>>>(a);
  return launch_status("norm");
}

template <typename XT, typename NT, bool VEC>
int32_t launch_back(const NormArgs& a, hipStream_t st) {
  const int64_t strips = (a.M + a.rows - 1) / a.rows;
  const dim3 one((unsigned)strips), four((unsigned)((strips + 3) / 4));
  if (a.C <= 512) k_norm_gate_back<XT, NT, 64, 1, VEC><<<four, 256, 0, st>>>(a);
  else if (a.C <= 1024) k_norm_gate_back<XT, NT, 64, 2, VEC><<<four, 256, 0, st>>>(a);
  else if (a.C <= 2048) k_norm_gate_back<XT, NT, 256, 1, VEC><<<one, 256, 0, st>>>(a);
  else if (a.C <= 4096) k_norm_gate_back<XT, NT, 256, 2, VEC><<<one, 256, 0, st>>>(a);
  else if (a.C <= 8192) k_norm_gate_back<XT, NT, 512, 2, VEC><<<one, 512, 0, st>>>(a);
  else k_norm_gate_back<XT, NT, 512, 4, VEC><<<one, 512, 0, st>>>(a);
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
                      int32_t n_dtype, int64_t ldn, uint8_t* n_scales, void* stream) {
  clear_error();
  ASP_TRY(check_norm(dtype, M, C, post, pre, G, offsets, ldt, eps));
  if (!y && (post != ASP_NORM_NONE || gate))
    return fail(ASP_ERR_ARG, "a post norm or gate without y");
  if (pre == ASP_NORM_NONE && (pre_w || pre_b || scale || shift || n))
    return fail(ASP_ERR_ARG, "pre norm arguments without a pre norm");
  if (pre == ASP_NORM_NONE && !h) return fail(ASP_ERR_ARG, "neither h nor n is asked for");
  if (post == ASP_NORM_NONE && post_w) return fail(ASP_ERR_ARG, "post_w without a post norm");
  if (n_dtype != ASP_F32 && n_dtype != ASP_BF16 && n_dtype != ASP_E4M3)
    return fail(ASP_ERR_ARG, "n_dtype=%d", n_dtype);
  if (M == 0) return ASP_OK;
  ASP_TRY(check_matrix(x, dtype, C, ldx, "x"));
  if (y) ASP_TRY(check_matrix(y, dtype, C, ldy, "y"));
  if (h) ASP_TRY(check_matrix(h, dtype, C, ldh, "h"));
  bool vec = vec8_ok(x, dtype, C, ldx) && (!y || vec8_ok(y, dtype, C, ldy)) &&
             (!h || vec8_ok(h, dtype, C, ldh));
  if (pre != ASP_NORM_NONE) {
    if (n_dtype == ASP_E4M3) {
      ASP_TRY(check_ptr(n, "n", true));
      ASP_TRY(check_ptr(n_scales, "n_scales", true));
    } else {
      ASP_TRY(check_matrix(n, n_dtype, C, ldn, "n"));
      vec = vec && vec8_ok(n, n_dtype, C, ldn);
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
  const hipStream_t st = (hipStream_t)stream;
  if (dtype == ASP_BF16) return vec ? launch_norm<uint16_t, true>(a, st) : launch_norm<uint16_t, false>(a, st);
  return vec ? launch_norm<float, true>(a, st) : launch_norm<float, false>(a, st);
}

int32_t asp_norm_gate_backward_workspace_bytes(int64_t M, int64_t C, int32_t G, size_t* bytes) {
  clear_error();
  ASP_TRY(check_norm(ASP_F32, M, C, 0, 0, 1, nullptr, 0, 0.0f));
  if (G < 1 || G > 65536) return fail(ASP_ERR_SHAPE, "G=%d outside [1, 65536]", G);
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  const int64_t rows = M ? strip_rows(M, C) : 1;
  *bytes = up256((size_t)((M + rows - 1) / rows + G) * 3 * C * 4);
  return ASP_OK;
}

int32_t asp_norm_gate_backward(const void* dh, int64_t lddh, const void* dn, int64_t lddn,
                               int32_t dn_dtype, const void* h, int64_t ldh, const void* y,
                               int64_t ldy, int32_t dtype, int64_t M, int64_t C, float alpha,
                               int32_t post, const float* post_w, const float* gate, int32_t pre,
                               const float* pre_w, const float* pre_b, const float* scale,
                               int64_t ldt, int32_t G, const int32_t* offsets, float eps, void* dx,
                               int64_t lddx, void* dy, int64_t lddy, float* d_post_w,
                               float* d_gate, float* d_pre_w, float* d_pre_b, float* d_scale,
                               float* d_shift, int64_t ldd, void* workspace,
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
  const bool sums = d_post_w || d_gate || d_pre_w || d_pre_b || d_scale || d_shift;
  if (!sums && !dx && !dy) return ASP_OK;
  bool vec = true;
  if (M > 0) {
    auto mat = [&](const void* p, int32_t dt, int64_t ld, const char* name) -> int32_t {
      ASP_TRY(check_matrix(p, dt, C, ld, name));
      vec = vec && vec8_ok(p, dt, C, ld);
      return ASP_OK;
    };
    if (dh) ASP_TRY(mat(dh, dtype, lddh, "dh"));
    if (y) ASP_TRY(mat(y, dtype, ldy, "y"));
    if (dx) ASP_TRY(mat(dx, dtype, lddx, "dx"));
    if (dy) ASP_TRY(mat(dy, dtype, lddy, "dy"));
    if (pre != ASP_NORM_NONE) {
      ASP_TRY(mat(h, dtype, ldh, "h"));
      ASP_TRY(mat(dn, dn_dtype, lddn, "dn"));
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
  a.rows = M ? strip_rows(M, C) : 1;
  if (M > 0) {
    int32_t s;
    const bool n16 = dn_dtype == ASP_BF16;
    if (dtype == ASP_BF16)
      s = n16 ? (vec ? launch_back<uint16_t, uint16_t, true>(a, st) : launch_back<uint16_t, uint16_t, false>(a, st))
              : (vec ? launch_back<uint16_t, float, true>(a, st) : launch_back<uint16_t, float, false>(a, st));
    else
      s = n16 ? (vec ? launch_back<float, uint16_t, true>(a, st) : launch_back<float, uint16_t, false>(a, st))
              : (vec ? launch_back<float, float, true>(a, st) : launch_back<float, float, false>(a, st));
    ASP_TRY(s);
  }
  if (!sums) return ASP_OK;
  SumArgs k = {};
  k.part = static_cast<const float*>(workspace);
  k.post_w = post_w; k.gate = gate; k.pre_w = pre_w; k.pre_b = pre_b; k.scale = scale;
  k.offsets = offsets; k.d_post_w = d_post_w; k.d_gate = d_gate; k.d_pre_w = d_pre_w;
  k.d_pre_b = d_pre_b; k.d_scale = d_scale; k.d_shift = d_shift; k.ldt = ldt; k.ldd = ldd;
  k.M = (int)M; k.C = (int)C; k.G = G; k.rows = a.rows; k.post = post;
  k_norm_sums<<<dim3((unsigned)((C + 15) / 16)), 256, 0, st>>>(k);
  return launch_status("norm column sums");
}

}  // extern "C"

// Attention, forward: o = softmax(scale q k^T) v over packed sequences whose queries and
// keys differ in number, with shared key heads, masked keys, and keys and values in bf16,
// float32 or a 4-bit cache.  asp_attn.h has the layouts.
//
// One pass over the keys with the running maximum m and sum l of each query: scores
// s = k q^T of a tile of keys, p = 2^(c s - m) with c = scale log2(e), l += p, o += v^T p.
// When a tile's maximum exceeds m by more than 2^8, m is raised and l and o are scaled down;
// until then p stays below 2^8, which costs float32 sums nothing.  Scores, sums
// and o are float32.  bf16: p is rounded to bf16 for its product (as v is: half a step
// is 2^-9 of each p, with signs that average out over the keys).  A row without a key has
// l = 0: o is 0 and its logarithm -infinity.
#include "asp_attn.h"

namespace asp {
namespace {

constexpr float kRaise = 8.0f;

template <typename XT, bool Q4>
using Product = std::conditional_t<sizeof(XT) == 4, Full, std::conditional_t<Q4, Half, Bf16>>;

// A workgroup has WM x WK waves.  Its WM rows of waves have 32 NQ rows (a token's shared
// heads follow one another) each; its WK columns take every WK-th tile of 32 KT keys, and
// their results are joined in LDS at the end.  `splits` workgroups share a longer range of
// keys and are joined by k_attn_join.
template <typename XT, int DT, int NQ, int WM, int WK, int KT, bool Q4>
struct Forward {
  using P = Product<XT, Q4>;
  using R = Rows<P::ES, DT>;
  static constexpr int THREADS = 64 * WM * WK, BM = 32 * NQ * WM, BN = 32 * KT;
  static constexpr int TILE = BN * R::BYTES;                // K or V
  static constexpr int BUFFERS = Q4 ? 1 : 2;
  static constexpr int GROUP = 2 * TILE * BUFFERS;          // of one of the WK columns
  static constexpr int STATE = 4 * 64 * (16 * DT + 2) * NQ;  // a wave's o, m and l
  static constexpr int JOIN = (WK - 1) * WM * STATE;
  static constexpr int LDS = WK * GROUP > JOIN ? WK * GROUP : JOIN;
  static_assert(LDS <= 160 * 1024, "a CU has 160 KB of LDS");
};

// eight codes and their scale as 16-bit or 32-bit values
__device__ __forceinline__ u32x4_t decode_half(uint32_t w, _Float16 s) {
  return __builtin_bit_cast(u32x4_t, decode8(w, s));
}

template <typename XT, int DT, int NQ, int WM, int WK, int KT, bool Q4>
__global__ void __launch_bounds__((Forward<XT, DT, NQ, WM, WK, KT, Q4>::THREADS))
    k_attn(const AttnArgs a) {
  using F = Forward<XT, DT, NQ, WM, WK, KT, Q4>;
  using P = typename F::P;
  using R = typename F::R;
  constexpr int BM = F::BM, BN = F::BN, TILE = F::TILE;
  constexpr int QS = R::PIECES / 2;             // pieces of a query in each half of the wave
  __shared__ __attribute__((aligned(16))) uint8_t smem[F::LDS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wm = wave % WM, wk = wave / WM;
  const int64_t run = attn_run(blockIdx.x, gridDim.x, a.qo != nullptr);
  if (run >= (int64_t)a.slots * a.splits * a.Hk) return;
  // the later parts, which shorter sequences do not have, come last
  const int slot = (int)(run % a.slots), hk = (int)(run / a.slots % a.Hk);
  const int split = (int)(run / a.slots / a.Hk);
  const AttnSeq seq = attn_seq(a, a.qo, a.Tq, a.group, BM, slot);

  if (a.zero && a.qo && split == 0)
    attn_outside(a.qo, a.G, a.Tq, slot, a.slots, [&](int64_t t) {
      const int pieces = a.D * (int)sizeof(XT) / 16;
      for (int i = threadIdx.x; i < a.group * pieces; i += F::THREADS) {
        const int h = hk * a.group + i / pieces;
        if (a.zero & 1)
          *reinterpret_cast<u32x4_t*>(static_cast<XT*>(a.o) + t * a.ot + h * a.oh +
                                      i % pieces * (16 / sizeof(XT))) = u32x4_t{0, 0, 0, 0};
        if (a.zero & 2 && i % pieces == 0) a.lse[t * a.Hq + h] = kNegInf;
      }
    });
  const int64_t row0 = seq.tile * BM, rows = seq.rows * a.group;
  const int parts = attn_parts(a, seq.keys);
  if (!seq.any || row0 >= rows || split >= parts) return;

  // the lane's queries
  int64_t token[NQ];
  int head[NQ];
  bool valid[NQ];
  u32x4_t qf[NQ][QS];
  float c[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int64_t r = row0 + 32 * (wm * NQ + n) + l32;
    valid[n] = r < rows;
    const int64_t t = a.group == 1 ? r : r / a.group;
    token[n] = seq.q0 + t;
    head[n] = hk * a.group + (int)(r - t * a.group);
    c[n] = attn_factor(a.scale);
    const XT* q = static_cast<const XT*>(a.q) + token[n] * a.qt + head[n] * a.qh;
#pragma unroll
    for (int s = 0; s < QS; ++s) {
      const int d = (2 * s + half) * (16 / P::ES);
      qf[n][s] = valid[n] && d < a.D ? *reinterpret_cast<const u32x4_t*>(q + d) : u32x4_t{0, 0, 0, 0};
    }
    if constexpr (std::is_same_v<P, Half>) {
      // fp16 has eleven bits but a short range: the row is scaled by a power of two so that its
      // largest finite element is 2^13 to 2^14; what then falls below fp16's
      // normal range is 2^-27 of that, below what float32 sums keep
      uint32_t top = 0;
#pragma unroll
      for (int s = 0; s < QS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = max(top, max(finite_bits(bf16_lo(qf[n][s][e])), finite_bits(bf16_hi(qf[n][s][e]))));
      top = __builtin_bit_cast(uint32_t, both_halves(__builtin_bit_cast(float, top), [](float x, float y) {
                                return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, x),
                                                                     __builtin_bit_cast(uint32_t, y)));
                              }));
      const int e2 = min(127 + 13 - (int)(top >> 23), 126);  // 2^e2 times the row
      const float up = __builtin_bit_cast(float, (uint32_t)(127 + e2) << 23);
      c[n] = fmaxf(c[n] * __builtin_bit_cast(float, (uint32_t)(127 - e2) << 23), kLeast);
#pragma unroll
      for (int s = 0; s < QS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          qf[n][s][e] = P::pair(bf16_lo(qf[n][s][e]) * up, bf16_hi(qf[n][s][e]) * up);
    }
  }

  f32x16_t acc[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = kNegInf;
    l[n] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[n][dt][v] = 0.0f;
  }

  // this workgroup's tiles of keys; each of its WK columns makes `turns`
  const int64_t tiles = (seq.keys + BN - 1) / BN;
  const int64_t first = tiles * split / parts, last = tiles * (split + 1) / parts;
  const int turns = (int)((last - first + WK - 1) / WK);
  uint8_t* mine = smem + wk * F::GROUP;
  const int64_t base_row = seq.k0;
  auto key0 = [&](int t) { return (first + (int64_t)t * WK + wk) * BN; };
  // whether the lane's key of a tile counts; the tiles' 64 lanes together are one bit a key
  auto key_on = [&](int t) -> int {
    const int64_t at = key0(t) + lane;
    const bool on = lane < BN && t < turns && first + (int64_t)t * WK + wk < last && at < seq.keys;
    return on ? (a.mask ? a.mask[base_row + at] : 1) : 0;
  };

  // ---- copies of bf16 and float32 tiles
  constexpr int COPIES = TILE / 1024 / WM;  // a wave's of K, and as many of V
  static_assert(Q4 || TILE % (1024 * WM) == 0, "whole copies for each wave");
  int offk[Q4 ? 1 : COPIES], offv[Q4 ? 1 : COPIES];
  if constexpr (!Q4)
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int row = R::row_of(wm * COPIES + i, lane), d = R::piece_of(wm * COPIES + i, lane) * (16 / P::ES);
      offk[i] = d < a.D ? (row * (int)a.kt + d) * P::ES : kFar;
      offv[i] = d < a.D ? (row * (int)a.vt + d) * P::ES : kFar;
    }
  auto issue = [&](int t, uint64_t live) {
    if constexpr (!Q4) {
      uint8_t* to = mine + (t & 1) * 2 * TILE;
      const int64_t at = base_row + key0(t);
      const int64_t n = min((int64_t)BN, seq.keys - key0(t));  // rows of the tile; may be none
      const XT* kp = static_cast<const XT*>(a.k) + (n > 0 ? at * a.kt + hk * a.kh : 0);
      const XT* vp = static_cast<const XT*>(a.v) + (n > 0 ? at * a.vt + hk * a.vh : 0);
      const auto rk = attn_rows(kp, n > 0 ? ((n - 1) * a.kt + a.D) * P::ES : 0);
      const auto rv = attn_rows(vp, n > 0 ? ((n - 1) * a.vt + a.D) * P::ES : 0);
#pragma unroll
      for (int i = 0; i < COPIES; ++i) attn_copy(rk, offk[i], to + (wm * COPIES + i) * 1024);
      // a masked key's values would meet a weight of 0, and make NaN of NaN or infinity
#pragma unroll
      for (int i = 0; i < COPIES; ++i) {
        int off = offv[i];
        if (a.mask && !(live >> R::row_of(wm * COPIES + i, lane) & 1)) off = kFar;
        attn_copy(rv, off, to + TILE + (wm * COPIES + i) * 1024);
      }
    }
  };
  // ---- blocks of a 4-bit tile, through registers
  constexpr int BLOCKS = BN * DT * 2 / (64 * WM);  // a lane's of K, and as many of V
  static_assert(!Q4 || BN * DT * 2 % (64 * WM) == 0, "whole blocks for each lane");
  u32x2_t ck[Q4 ? BLOCKS : 1], cv[Q4 ? BLOCKS : 1];
  uint32_t sk[Q4 ? BLOCKS : 1], sv[Q4 ? BLOCKS : 1];
  auto fetch = [&](int t, uint64_t live) {
    if constexpr (Q4) {
#pragma unroll
      for (int i = 0; i < BLOCKS; ++i) {
        const int b = (i * WM + wm) * 64 + lane, row = b / (2 * DT), blk = b % (2 * DT);
        ck[i] = cv[i] = u32x2_t{0, 0};
        sk[i] = sv[i] = 0;
        if ((live >> row & 1) && 16 * blk < a.D) {
          const int64_t at = ((base_row + key0(t) + row) * a.Hk + hk) * (a.D / 16) + blk;
          ck[i] = *reinterpret_cast<const u32x2_t*>(a.kc + 8 * at);
          cv[i] = *reinterpret_cast<const u32x2_t*>(a.vc + 8 * at);
          sk[i] = a.ks[at];
          sv[i] = a.vs[at];
        }
      }
    }
  };
  auto unpack4 = [&]() {
    if constexpr (Q4) {
#pragma unroll
      for (int i = 0; i < BLOCKS; ++i) {
        const int b = (i * WM + wm) * 64 + lane, row = b / (2 * DT), blk = b % (2 * DT);
        auto put = [&](uint8_t* tile, u32x2_t w, uint32_t code) {
          const float s = __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
          uint8_t* to = tile + row * R::BYTES;
          const int z = R::swizzle(row & 15);
          if constexpr (P::ES == 2) {
            const _Float16 h = (_Float16)s;
            *reinterpret_cast<u32x4_t*>(to + 16 * ((2 * blk) ^ z)) = decode_half(w[0], h);
            *reinterpret_cast<u32x4_t*>(to + 16 * ((2 * blk + 1) ^ z)) = decode_half(w[1], h);
          } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              f32x4_t v;
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = e2m1_decode(w[p >> 1] >> (16 * (p & 1) + 4 * e) & 15u) * s;
              *reinterpret_cast<f32x4_t*>(to + 16 * ((4 * blk + p) ^ z)) = v;
            }
          }
        };
        put(mine, ck[i], sk[i]);
        put(mine + TILE, cv[i], sv[i]);
      }
    }
  };

  // a tile's mask is loaded two turns ahead and looked at when the tile before it has landed
  uint64_t live = __ballot(key_on(0) != 0), next;
  int on = key_on(1);
  issue(0, live);
  fetch(0, live);
  for (int t = 0; t < turns; ++t) {
    const uint8_t* tile = mine + (Q4 ? 0 : (t & 1) * 2 * TILE);
    if constexpr (Q4) {
      attn_settle<(WM > 1)>();  // the tile before is read
      unpack4();
      attn_settle<(WM > 1)>();
      next = __ballot(on != 0);
      on = key_on(t + 2);
      if (t + 1 < turns) fetch(t + 1, next);
    } else {
      attn_settle<(WM > 1)>();  // tile t is there, and the one before is read
      next = __ballot(on != 0);
      on = key_on(t + 2);
      if (t + 1 < turns) issue(t + 1, next);
    }
    if (live != 0) {
      f32x16_t s[NQ][KT];
#pragma unroll
      for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int v = 0; v < 16; ++v) s[n][k][v] = 0.0f;
#pragma unroll
        for (int i = 0; i < QS; ++i) {
          const u32x4_t kf = row_frag<P::ES, DT>(tile + 32 * k * R::BYTES, i, half, l32);
#pragma unroll
          for (int n = 0; n < NQ; ++n) piece_mfma<P>(kf, qf[n][i], s[n][k]);
        }
      }
      constexpr uint64_t ALL = BN == 64 ? ~0ull : (1ull << (BN & 63)) - 1;
      if (live != ALL)
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          const uint32_t bits = (uint32_t)(live >> (32 * k)) >> (4 * half);
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (!(bits >> (8 * (v >> 2) + (v & 3)) & 1))
#pragma unroll
              for (int n = 0; n < NQ; ++n) s[n][k][v] = kNegInf;
        }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float top = kNegInf;
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int v = 0; v < 16; ++v) top = fmaxf(top, s[n][k][v]);
        top = both_halves(top, [](float x, float y) { return fmaxf(x, y); }) * c[n];
        if (__any(top > m[n] + kRaise)) {
          const float up = fmaxf(m[n], top);
          const float f = up == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[n] - up);
          m[n] = up;
          l[n] *= f;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[n][dt][v] *= f;
        }
        const float off = m[n] == kNegInf ? 0.0f : m[n];
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            s[n][k][v] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][k][v], c[n], -off));
            l[n] += s[n][k][v];
          }
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          Weights<P> w;
          w.set(s[n][k]);
          columns_mfma<P, DT>(tile + TILE + 32 * k * R::BYTES, w, acc[n], lane);
        }
      }
    }
    live = next;
  }

#pragma unroll
  for (int n = 0; n < NQ; ++n) l[n] = both_halves(l[n], [](float x, float y) { return x + y; });
  if constexpr (WK > 1) {
    __syncthreads();  // the tiles are read
    float* at = reinterpret_cast<float*>(smem) + lane;
    constexpr int EACH = 16 * DT + 2;  // values of a lane for each of its NQ rows
    if (wk > 0) {
      float* to = at + ((wk - 1) * WM + wm) * NQ * EACH * 64;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int v = 0; v < 16; ++v) to[(n * EACH + 16 * dt + v) * 64] = acc[n][dt][v];
        to[(n * EACH + 16 * DT) * 64] = m[n];
        to[(n * EACH + 16 * DT + 1) * 64] = l[n];
      }
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int w = 0; w < WK - 1; ++w) {
      const float* from = at + (w * WM + wm) * NQ * EACH * 64;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float m2 = from[(n * EACH + 16 * DT) * 64], l2 = from[(n * EACH + 16 * DT + 1) * 64];
        const float up = fmaxf(m[n], m2), off = up == kNegInf ? 0.0f : up;
        const float f = __builtin_amdgcn_exp2f(m[n] - off), f2 = __builtin_amdgcn_exp2f(m2 - off);
        l[n] = l[n] * f + l2 * f2;
        m[n] = up;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            acc[n][dt][v] = __builtin_fmaf(acc[n][dt][v], f, from[(n * EACH + 16 * dt + v) * 64] * f2);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const bool none = l[n] == 0.0f;
    const float inv = none ? 0.0f : 1.0f / l[n];
    // the logarithm to base 2 of the row's sum
    const float lg = none ? kNegInf : m[n] + __builtin_amdgcn_logf(l[n]);
    const int64_t at = token[n] * a.Hq + head[n];
    if (!valid[n]) continue;
    if (parts > 1) {
      float* part = a.part + ((int64_t)split * a.Tq * a.Hq + at) * a.D;
      store_row<float, DT>(part, acc[n], inv, a.D, half);
      if (half == 0) a.part_l[(int64_t)split * a.Tq * a.Hq + at] = lg;
    } else {
      XT* o = static_cast<XT*>(a.o) + token[n] * a.ot + head[n] * a.oh;
      store_row<XT, DT>(o, acc[n], inv, a.D, half);
      if (half == 0 && a.lse) a.lse[at] = lg * kLn2;
    }
  }
}

// The splits' results of a query (at most 64), joined by their sums.  A wave has one query: its
// lanes find the splits' weights, then four groups of 16 lanes take every fourth split, 8
// elements a lane.
template <typename XT>
__global__ void __launch_bounds__(256) k_attn_join(const AttnArgs a) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), rows = a.Tq * a.Hq;
  if (row >= rows) return;
  const int lane = threadIdx.x & 63, mine = lane >> 4;
  const int64_t t = row / a.Hq;
  const int h = (int)(row - t * a.Hq), d = 8 * (lane & 15);
  if (a.qo && (t < attn_offset(a.qo, 0, a.Tq) || t >= attn_offset(a.qo, a.G, a.Tq))) return;
  const int parts = attn_parts(a, attn_keys(a, a.qo ? attn_owner(a.qo, a.G, t) : 0));
  if (parts == 1) return;
  const float l = lane < parts ? a.part_l[lane * rows + row] : kNegInf;
  float top = l;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
  const float off = top == kNegInf ? 0.0f : top;
  const float w = l == l ? __builtin_amdgcn_exp2f(l - off) : l;  // a NaN is the row's
  float sum = w;
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
  float v[8] = {};
  for (int s = mine; s < parts; s += 4) {
    const float ws = __shfl(w, s);
    if (d < a.D && ws != 0.0f) {
      const f32x4_t* p = reinterpret_cast<const f32x4_t*>(a.part + (s * rows + row) * a.D + d);
      const f32x4_t x = p[0], y = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __builtin_fmaf(x[e], ws, v[e]);
        v[4 + e] = __builtin_fmaf(y[e], ws, v[4 + e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] += __shfl_xor(v[e], 16);
    v[e] += __shfl_xor(v[e], 32);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (lane == 0 && a.lse) a.lse[row] = sum == 0.0f ? kNegInf : (off + __builtin_amdgcn_logf(sum)) * kLn2;
  if (mine || d >= a.D) return;
  XT* o = static_cast<XT*>(a.o) + t * a.ot + h * a.oh + d;
  if constexpr (sizeof(XT) == 2) {
    *reinterpret_cast<u32x4_t*>(o) = u32x4_t{bf16x2_rne(v[0] * inv, v[1] * inv), bf16x2_rne(v[2] * inv, v[3] * inv),
                                             bf16x2_rne(v[4] * inv, v[5] * inv), bf16x2_rne(v[6] * inv, v[7] * inv)};
  } else {
    *reinterpret_cast<f32x4_t*>(o) = f32x4_t{v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv};
    *reinterpret_cast<f32x4_t*>(o + 4) = f32x4_t{v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv};
  }
}

// -------------------------------------------------------------------- host

AttnPlan plan_of(int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hk, int32_t G, bool ragged) {
  return attn_plan(Tq * (Hq / Hk), Tk, Hk, G, ragged);
}

size_t part_bytes(const AttnPlan& p, int64_t Tq, int32_t Hq, int32_t D) {
  return p.splits > 1 ? up256((size_t)p.splits * Tq * Hq * (D + 1) * 4) : 0;
}

template <typename XT, int DT, int NQ, int WM, int WK, int KT, bool Q4>
int32_t launch(const AttnArgs& a, hipStream_t st) {
  using F = Forward<XT, DT, NQ, WM, WK, KT, Q4>;
  const int64_t blocks = attn_grid(a, a.qo != nullptr);
  ASP_TRY(check_attn_grid(blocks, F::THREADS));
  k_attn<XT, DT, NQ, WM, WK, KT, Q4><<<dim3((unsigned)blocks), F::THREADS, 0, st>>>(a);
  return launch_status("attention");
}

template <typename XT, int DT, bool Q4>
int32_t launch_form(const AttnArgs& a, bool wide, hipStream_t st) {
  // rows of 512 bytes: half the tile, and two columns of waves, for LDS's sake
  constexpr bool LONG = sizeof(XT) == 4 && DT == 4;
  return wide ? launch<XT, DT, 1, 4, 1, LONG ? 1 : 2, Q4>(a, st)
              : launch<XT, DT, 1, 1, LONG ? 2 : 4, 1, Q4>(a, st);
}

template <typename XT, bool Q4>
int32_t launch_attn(const AttnArgs& a, bool wide, hipStream_t st) {
  ASP_TRY((a.D <= 64 ? launch_form<XT, 2, Q4>(a, wide, st) : launch_form<XT, 4, Q4>(a, wide, st)));
  if (a.splits == 1) return ASP_OK;
  const int64_t blocks = (a.Tq * a.Hq + 3) / 4;
  ASP_TRY(check_attn_grid(blocks, 256));
  k_attn_join<XT><<<dim3((unsigned)blocks), 256, 0, st>>>(a);
  return launch_status("attention join");
}

int32_t run_attn(AttnArgs& a, int32_t dtype, bool q4, void* workspace, size_t workspace_bytes,
                 hipStream_t st) {
  const AttnPlan p = plan_of(a.Tq, a.Tk, a.Hq, a.Hk, a.G, a.qo != nullptr);
  const size_t need = part_bytes(p, a.Tq, a.Hq, a.D);
  if (need) ASP_TRY(check_ptr(workspace, "workspace", true));
  if (workspace_bytes < need)
    return fail(ASP_ERR_WORKSPACE, "the workspace holds %zu bytes, the call needs %zu",
                workspace_bytes, need);
  a.group = a.Hq / a.Hk;
  a.slots = p.slots;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.part = static_cast<float*>(workspace);
  a.part_l = a.part + (size_t)p.splits * a.Tq * a.Hq * a.D;
  if (dtype == ASP_BF16)
    return q4 ? launch_attn<uint16_t, true>(a, p.wide, st) : launch_attn<uint16_t, false>(a, p.wide, st);
  return q4 ? launch_attn<float, true>(a, p.wide, st) : launch_attn<float, false>(a, p.wide, st);
}

}  // namespace
}  // namespace asp

using namespace asp;

extern "C" {

int32_t asp_attention_workspace_bytes(int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t G, size_t* bytes) {
  clear_error();
  const int32_t some = 0;
  ASP_TRY(check_attn(ASP_F32, Tq, Tk, Hq, Hk, D, G, 1.0f, &some, &some, nullptr));
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  *bytes = part_bytes(plan_of(Tq, Tk, Hq, Hk, G, true), Tq, Hq, D);
  return ASP_OK;
}

int32_t asp_attention(const void* q, int64_t ldq, int64_t hsq, const void* k, int64_t ldk,
                      int64_t hsk, const void* v, int64_t ldv, int64_t hsv, int32_t dtype,
                      int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hk, int32_t D, float scale,
                      int32_t G, const int32_t* q_offsets, const int32_t* kv_offsets,
                      const int32_t* kv_lengths, const uint8_t* key_mask, void* o, int64_t ldo,
                      int64_t hso, float* lse, int32_t zero, void* workspace,
                      size_t workspace_bytes, void* stream) {
  clear_error();
  ASP_TRY(check_attn(dtype, Tq, Tk, Hq, Hk, D, G, scale, q_offsets, kv_offsets, kv_lengths));
  if (zero < 0 || zero > 3 || (Tq > 0 && zero & 2 && !lse)) return fail(ASP_ERR_ARG, "zero=%d", zero);
  if (Tq == 0) return ASP_OK;
  ASP_TRY(check_attn_rows(q, dtype, Tq, Hq, D, ldq, hsq, false, "q"));
  ASP_TRY(check_attn_rows(o, dtype, Tq, Hq, D, ldo, hso, true, "o"));
  if (Tk > 0) {
    ASP_TRY(check_attn_rows(k, dtype, Tk, Hk, D, ldk, hsk, false, "k"));
    ASP_TRY(check_attn_rows(v, dtype, Tk, Hk, D, ldv, hsv, false, "v"));
  }
  if ((uintptr_t)lse & 3) return fail(ASP_ERR_ALIGN, "lse is not 4-byte aligned");
  AttnArgs a = {};
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.qt = ldq; a.qh = hsq; a.kt = ldk; a.kh = hsk; a.vt = ldv; a.vh = hsv; a.ot = ldo; a.oh = hso;
  a.qo = q_offsets; a.ko = kv_offsets; a.kl = kv_lengths; a.mask = key_mask;
  a.Tq = Tq; a.Tk = Tk; a.Hq = Hq; a.Hk = Hk; a.D = D; a.G = G; a.zero = zero; a.scale = scale;
  return run_attn(a, dtype, false, workspace, workspace_bytes, (hipStream_t)stream);
}

int32_t asp_attention_cache(const void* q, int64_t ldq, int64_t hsq, int32_t dtype,
                            const uint8_t* k_codes, const uint8_t* k_scales,
                            const uint8_t* v_codes, const uint8_t* v_scales, int64_t Tq, int64_t Tk,
                            int32_t Hq, int32_t Hk, int32_t D, float scale, int32_t G,
                            const int32_t* q_offsets, const int32_t* kv_offsets,
                            const int32_t* kv_lengths, const uint8_t* key_mask, void* o,
                            int64_t ldo, int64_t hso, float* lse, int32_t zero, void* workspace,
                            size_t workspace_bytes, void* stream) {
  clear_error();
  ASP_TRY(check_attn(dtype, Tq, Tk, Hq, Hk, D, G, scale, q_offsets, kv_offsets, kv_lengths));
  if (D % 16) return fail(ASP_ERR_SHAPE, "D=%d of a cache is not a multiple of 16", D);
  if (zero < 0 || zero > 3 || (Tq > 0 && zero & 2 && !lse)) return fail(ASP_ERR_ARG, "zero=%d", zero);
  if (Tq == 0) return ASP_OK;
  ASP_TRY(check_attn_rows(q, dtype, Tq, Hq, D, ldq, hsq, false, "q"));
  ASP_TRY(check_attn_rows(o, dtype, Tq, Hq, D, ldo, hso, true, "o"));
  if (Tk > 0) {
    ASP_TRY(check_ptr(k_codes, "k_codes", true));
    ASP_TRY(check_ptr(k_scales, "k_scales", true));
    ASP_TRY(check_ptr(v_codes, "v_codes", true));
    ASP_TRY(check_ptr(v_scales, "v_scales", true));
  }
  if ((uintptr_t)lse & 3) return fail(ASP_ERR_ALIGN, "lse is not 4-byte aligned");
  AttnArgs a = {};
  a.q = q; a.kc = k_codes; a.ks = k_scales; a.vc = v_codes; a.vs = v_scales; a.o = o; a.lse = lse;
  a.qt = ldq; a.qh = hsq; a.ot = ldo; a.oh = hso;
  a.qo = q_offsets; a.ko = kv_offsets; a.kl = kv_lengths; a.mask = key_mask;
  a.Tq = Tq; a.Tk = Tk; a.Hq = Hq; a.Hk = Hk; a.D = D; a.G = G; a.zero = zero; a.scale = scale;
  return run_attn(a, dtype, true, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"

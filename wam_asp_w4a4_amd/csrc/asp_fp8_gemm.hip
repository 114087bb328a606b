// The 8-bit (block-128) matrix product y = A B^T (+ bias) on gfx950's
// block-scaled MFMA, and the linear layer's forward and backward built on it.
//
// The scaled MFMA multiplies E4M3 operands at twice the rate of 16-bit ones and
// applies an E8M0 scale to each 32 elements of an operand row; a block of 128
// hands it the same byte four times, so the scales are free and the float32
// accumulators need no promotion between blocks.
//
// Two arithmetics, chosen by y's type.  The 8-bit MFMA adds the products of each
// 8 consecutive elements in a window of 14 bits below the largest of them and
// cuts off what lies lower, toward zero; only the sums of those groups are
// float32 (measured on gfx950: beside a product 2^16 one of 2^3 of its group
// counts and one of 2^2 does not; across groups 24 bits hold).  y is then off by
// 1.5e-5 of its 2-norm for normal data and up to 7e-5 for heavy tails, at every K:
// a bf16 y, rounded to 2^-8 of each value, loses nothing by it.  A float32 y
// would, so its operands are decoded to bf16 (exact: four significant bits, and
// the conversion applies the power-of-two scale) and multiplied by the 16-bit
// MFMA, whose sums are float32 throughout.
#include "asp_fp8.h"

namespace asp {
namespace {

// 8 codes (two dwords) times a scale, as bf16
__device__ __forceinline__ bf16x8_t decode_bf16(int lo, int hi, float s) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, s, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, s, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, s, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, s, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// the scale of the low byte of w (1..254)
__device__ __forceinline__ float scale_f32(uint32_t w) {
  return __builtin_bit_cast(float, (w & 255u) << 23);
}

struct GemmK {
  const uint8_t *a, *as, *b, *bs;
  const float* bias;
  void* y;
  float* part;  // [slices][M][N] partial sums when slices > 1
  int64_t lda, ldb;  // code pitches: KB * 128
  int M, N, KB, y_bf16, slices, tiles_m, tiles_n;
  int whole, parts;  // of k_fp8_gemm_tail: the tiles computed whole, the parts of each other
};

// Bytes p .. p + n - 1 as a buffer, and the direct copy of 16 bytes a lane from it to
// LDS: lane l's bytes, at offset v + s, land at lds_base (uniform) + 16 l.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const uint8_t* p, int64_t n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)n, 0x00020000);
}
__device__ __forceinline__ void buffer_copy16(__amdgpu_buffer_rsrc_t r, int v, int s, void* lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_base, 16,
                                           v, s, 0, 0);
}
__device__ __forceinline__ void buffer_copy4(__amdgpu_buffer_rsrc_t r, int v, void* lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_base, 4,
                                           v, 0, 0, 0);
}

// XCD-aware tile order.  Workgroups go to the 8 XCDs (each with its own L2) in
// turn; each XCD takes one contiguous run of tiles (xcd_run), walked in bands of 4 tile
// rows (tile_at), so that the operand rows its workgroups share stay in its L2.
__device__ __forceinline__ int xcd_run(int id, int total) {
  const int xcd = id % 8;
  return xcd * (total / 8) + min(xcd, total % 8) + id / 8;
}
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = 4 * tiles_n, b = t / band, r = t % band;
  const int rows = min(4, tiles_m - 4 * b);
  tm = __builtin_amdgcn_readfirstlane(4 * b + r % rows);
  tn = __builtin_amdgcn_readfirstlane(r / rows);
}

// four consecutive results of one row, n .. n + 3 (bounds checked)
__device__ __forceinline__ void store4(const GemmK& g, int64_t m, int n, f32x4_t v, bool vec) {
  if (m >= g.M || n >= g.N) return;
  if (g.bias)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += n + e < g.N ? g.bias[n + e] : 0.0f;
  const int64_t at = m * g.N + n;
  if (g.y_bf16) {
    uint16_t* y = static_cast<uint16_t*>(g.y) + at;
    if (vec)
      *reinterpret_cast<u32x2_t*>(y) = u32x2_t{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) y[e] = bf16_rne(v[e]);
  } else {
    float* y = static_cast<float*>(g.y) + at;
    if (vec)
      *reinterpret_cast<f32x4_t*>(y) = v;
    else
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) y[e] = v[e];
  }
}

// The order of half a block for the scheduler: after each MFMA its share of the
// half's LDS reads and memory loads, so that no group of them holds the matrix unit
// up (its MFMAs start one after the other, and a wave issues in order).
template <int MFMAS, int READS, int LOADS, int M = 0>
__device__ __forceinline__ void order() {
  if constexpr (M < MFMAS) {
    constexpr int R = READS * (M + 1) / MFMAS - READS * M / MFMAS;
    constexpr int L = LOADS * (M + 1) / MFMAS - LOADS * M / MFMAS;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (R > 0) __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    if constexpr (L > 0) __builtin_amdgcn_sched_group_barrier(0x020, L, 0);
    order<MFMAS, READS, LOADS, M + 1>();
  }
}

// k_fp8_gemm: a workgroup of 2 x 2 waves owns a BM x BN tile of y, each wave TM x TN
// MFMA tiles of 32 x 32.  K goes by in stages of 64, straight from memory to LDS (16
// bytes a lane, no registers).  Copy j of a stage fills 16 rows of 64 bytes; slot s
// of it holds row s / 4, piece (s % 4) ^ (row / 4 % 4) of that row's four 16-byte
// pieces, so that the MFMA reads (32 rows at one piece index) fall in distinct banks.
// The order of the K elements inside a stage is the same for both operands, and
// the scale is the same for all of them, so it needs no care.  The operands are
// swapped (B's rows are the MFMA's rows): a lane then holds four consecutive
// columns of a row of y.
//
// While a stage is multiplied from registers, the next one's fragments are read
// from LDS, and NB - 1 more stages are on their way into the NB buffers: at 8192^3
// 436 us with three of them against 486 us with one of twice the size.  One barrier
// a stage: by then every wave has the stage's fragments in registers, so its buffer
// is free for the stage NB later, and every wave's copies of the next stage have
// landed.  The scales go the same way (the dword of a row's four blocks,
// for each block anew): loaded to registers, their wait would be one for every older
// copy, since loads are counted in order.
template <int TM, int TN>
struct Tile {
  static constexpr int BM = 64 * TM, BN = 64 * TN, SK = 64, NB = 4;
  static constexpr int STAGE = (BM + BN) * SK;
  static constexpr int SCALES = 4 * (BM + BN);  // bytes of a block's scales
  static constexpr int PITCH16 = 64 * TN + 16, PITCH32 = 128 * TN + 16;  // of a wave's result rows in LDS
  static constexpr int TP = TM > 1 ? TM / 2 : 1;  // tile rows of a float32 result at a time
  static constexpr int OUT16 = 32 * TM * PITCH16, OUT32 = 32 * TP * PITCH32;
  static constexpr int OUT = OUT16 > OUT32 ? OUT16 : OUT32;  // a wave's result region
  static constexpr int STAGING = NB * STAGE + NB / 2 * SCALES;
  static constexpr int LDS = STAGING > 4 * OUT ? STAGING : 4 * OUT;
};

template <int TM, int TN, bool WIDE>
__device__ __forceinline__ void gemm_tile(const GemmK& g, const int64_t m0, const int64_t n0,
                                          uint8_t* smem) {
  using T = Tile<TM, TN>;
  constexpr int BM = T::BM, BN = T::BN, SK = T::SK, NB = T::NB, STAGE = T::STAGE, SCALES = T::SCALES;
  constexpr int PITCH16 = T::PITCH16, PITCH32 = T::PITCH32, TP = T::TP, OUT = T::OUT;
  constexpr int CA = BM * SK / 4096, CB = BN * SK / 4096;  // a wave's copies of A and B for a stage
  constexpr int SC = (TM + TN + 3) / 4;                    // and of 64 rows' scales for a block
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  const int wm = wave >> 1, wn = wave & 1;
  // the tile's last rows; rows past them re-read the last one, their results are not stored
  const int mlast = (int)min((int64_t)BM, g.M - m0) - 1, nlast = (int)min((int64_t)BN, g.N - n0) - 1;
  // this slice's blocks of K
  const int kb0 = (int)((int64_t)g.KB * blockIdx.y / g.slices);
  const int kb1 = (int)((int64_t)g.KB * (blockIdx.y + 1) / g.slices);

  // The copies go through buffer descriptors that end with the tile's last row: one
  // 32-bit offset a copy (a tile's rows span less than 2^28 bytes) and the stage's
  // offset in a scalar.
  const __amdgpu_buffer_rsrc_t ra = descriptor(g.a + m0 * g.lda, (mlast + 1) * g.lda);
  const __amdgpu_buffer_rsrc_t rb = descriptor(g.b + n0 * g.ldb, (nlast + 1) * g.ldb);
  int offa[CA], offb[CB];
  auto source = [&](int copy, int last, int64_t ld) {
    const int row = 16 * copy + (lane >> 2);
    return min(row, last) * (int)ld + 16 * ((lane & 3) ^ (row >> 2 & 3));
  };
#pragma unroll
  for (int c = 0; c < CA; ++c) offa[c] = source(wave * CA + c, mlast, g.lda);
#pragma unroll
  for (int c = 0; c < CB; ++c) offb[c] = source(wave * CB + c, nlast, g.ldb);
  // copy c of stage s (half s % 2 of block s / 2) into buffer s % NB; past the last stage the
  // last again, which nobody reads, so that the loop has no branch
  auto copy = [&](int s, int c) {
    uint8_t* base = smem + (s & (NB - 1)) * STAGE;
    const int at = min(s, 2 * kb1 - 1) * SK;
    if (c < CA)
      buffer_copy16(ra, offa[c < CA ? c : 0], at, base + (wave * CA + c) * 1024);
    else
      buffer_copy16(rb, offb[c < CA ? 0 : c - CA], at, base + BM * SK + (wave * CB + c - CA) * 1024);
  };
  auto issue = [&](int s) {
#pragma unroll
    for (int c = 0; c < CA + CB; ++c) copy(s, c);
  };
  // block kb's scales into scale buffer kb % (NB / 2): copy i has 64 rows of A, then of B (where
  // the waves have more copies than there are, the first ones are made again)
  const uint8_t* scale_base[SC];
  int64_t scale_group[SC];
  int scale_bytes[SC], scale_off[SC];
#pragma unroll
  for (int c = 0; c < SC; ++c) {
    const int i = (wave * SC + c) % (TM + TN);
    const bool is_a = i < TM;
    scale_base[c] = is_a ? g.as + 4 * m0 : g.bs + 4 * n0;
    scale_group[c] = 4 * (int64_t)(is_a ? g.M : g.N);
    scale_bytes[c] = 4 * ((is_a ? mlast : nlast) + 1);
    scale_off[c] = 4 * min(64 * (i % TM) + lane, is_a ? mlast : nlast);
  }
  auto issue_scales = [&](int kb) {
    const int64_t grp = min(kb, kb1 - 1) >> 2;
    uint8_t* base = smem + NB * STAGE + (kb & (NB / 2 - 1)) * SCALES;
#pragma unroll
    for (int c = 0; c < SC; ++c)
      buffer_copy4(descriptor(scale_base[c] + grp * scale_group[c], scale_bytes[c]), scale_off[c],
                   base + 256 * ((wave * SC + c) % (TM + TN)));
  };
  uint32_t ca[TM], cb[TN], na[TM], nb[TN];
  auto read_scale = [&](int kb, int f) {
    const uint8_t* base = smem + NB * STAGE + (kb & (NB / 2 - 1)) * SCALES + (min(kb, kb1 - 1) & 3);
    if (f < TN)
      nb[f < TN ? f : 0] = base[4 * (BM + 32 * (wn * TN + f) + l32)];
    else
      na[f < TN ? 0 : f - TN] = base[4 * (32 * (wm * TM + f - TN) + l32)];
  };
  auto next_scales = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i) ca[i] = na[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) cb[j] = nb[j];
  };

  f32x16_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  const int key = l32 >> 2 & 3;
  const int lo = 16 * ((2 * half) ^ key), hi = 16 * ((2 * half + 1) ^ key);
  const int rowa = (32 * TM * wm + l32) * SK, rowb = (BM + 32 * TN * wn + l32) * SK;
  auto frag = [&](const uint8_t* p) {
    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p + lo);
    const u32x4_t b = *reinterpret_cast<const u32x4_t*>(p + hi);
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
                   (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  };
  i32x8_t fa[2][TM], fb[2][TN];
  // fragment f of stage s: the columns' first
  auto read = [&](int s, int set, int f) {
    const uint8_t* base = smem + (s & (NB - 1)) * STAGE;
    if (f < TN)
      fb[set][f < TN ? f : 0] = frag(base + rowb + 32 * SK * f);
    else
      fa[set][f < TN ? 0 : f - TN] = frag(base + rowa + 32 * SK * (f - TN));
  };
  auto multiply = [&](int set) {
    if constexpr (WIDE) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8_t wa[TM], wb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j)
          wb[j] = decode_bf16(fb[set][j][2 * s], fb[set][j][2 * s + 1], scale_f32(cb[j]));
#pragma unroll
        for (int i = 0; i < TM; ++i)
          wa[i] = decode_bf16(fa[set][i][2 * s], fa[set][i][2 * s + 1], scale_f32(ca[i]));
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fb[set][j], fa[set][i], acc[i][j], 0, 0, 0, (int)cb[j], 0, (int)ca[i]);
    }
  };
  // The copies behind stage s + 1's when the barrier of stage s is reached: those of
  // NB - 2 stages and of (NB - 2) / 2 blocks' scales (which go behind an even stage's).
  constexpr int FLIGHT = (NB - 2) * (CA + CB) + (NB - 2) / 2 * SC;
  static_assert(FLIGHT + CA + CB < 64, "the wait counts up to 63 loads");
  auto barrier = [&](auto flight) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(flight)::value) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  using Flight = std::integral_constant<int, FLIGHT>;
  constexpr int F = TM + TN;  // fragments of a stage, and as many copies
  static_assert(CA + CB == F, "a copy for each fragment");

  if (kb0 < kb1) {
    // in the order of the loop, which the waits count on
    issue_scales(kb0);
#pragma unroll
    for (int s = 0; s < NB; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      if (s >= 2 && s % 2 == 0) issue_scales(kb0 + s / 2);
      __builtin_amdgcn_sched_barrier(0);
      issue(2 * kb0 + s);
    }
    barrier(std::integral_constant<int, FLIGHT + CA + CB>{});
#pragma unroll
    for (int f = 0; f < F; ++f) {
      read(2 * kb0, 0, f);
      read_scale(kb0, f);
    }
    next_scales();
  }
  // In each half the reads and copies alternate, spread evenly over the MFMAs: the four
  // waves' copies keep the load path busy half the time, and none waits for it.
  for (int kb = kb0; kb < kb1; ++kb) {
    barrier(Flight{});
#pragma unroll
    for (int f = 0; f < F; ++f) {
      read(2 * kb + 1, 1, f);
      copy(2 * kb + NB, f);
    }
    issue_scales(kb + NB / 2);
    multiply(0);
    if constexpr (!WIDE) {
      order<TM * TN, 2 * F, F>();
      __builtin_amdgcn_sched_group_barrier(0x020, SC, 0);
    }
    barrier(Flight{});
#pragma unroll
    for (int f = 0; f < F; ++f) {
      read(2 * kb + 2, 0, f);
      read_scale(kb + 1, f);
      copy(2 * kb + NB + 1, f);
    }
    multiply(1);
    if constexpr (!WIDE) order<TM * TN, 3 * F, F>();
    next_scales();
  }
  // every copy has landed and every read is done: the buffers become the results' rows
  barrier(std::integral_constant<int, 0>{});

  // Accumulator element v of lane l: column 8 (v / 4) + 4 (l / 32) + v % 4 of row
  // l % 32 of y's 32 x 32 tile.  Each wave turns its part in its own region of LDS
  // (rows padded by 16 bytes against bank conflicts) and stores whole 16-byte pieces of
  // its rows.
  const bool split = g.slices > 1;
  const bool y16 = g.y_bf16 && !split;
  uint8_t* mine = smem + wave * OUT;
  const int64_t mw = m0 + 32 * TM * wm;
  const int nw = (int)n0 + 32 * TN * wn;
  // the four columns (j, v): their bias, and their values of tile row i
  auto bias_of = [&](int j, int v) {
    f32x4_t b = {0.0f, 0.0f, 0.0f, 0.0f};
    const int n = nw + 32 * j + 8 * v + 4 * half;
    if (g.bias && !split) {
      if (n + 4 <= g.N)
        b = __builtin_bit_cast(f32x4_t, (u32x4_t) * reinterpret_cast<const u32x4_e4*>(g.bias + n));
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < g.N) b[e] = g.bias[n + e];
    }
    return b;
  };
  auto values = [&](int i, int j, int v, f32x4_t b) {
    return f32x4_t{acc[i][j][4 * v] + b[0], acc[i][j][4 * v + 1] + b[1], acc[i][j][4 * v + 2] + b[2],
                   acc[i][j][4 * v + 3] + b[3]};
  };
  auto settle = [&]() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
  if (y16) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const f32x4_t b = bias_of(j, v);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const f32x4_t r = values(i, j, v, b);
          *reinterpret_cast<u32x2_t*>(mine + (32 * i + l32) * PITCH16 + 64 * j + 16 * v + 8 * half) =
              u32x2_t{bf16x2_rne(r[0], r[1]), bf16x2_rne(r[2], r[3])};
        }
      }
    settle();
    constexpr int PIECES = 4 * TN;  // of 8 values a row
    const int col = 8 * (lane % PIECES), left = g.N - nw - col;
#pragma unroll
    for (int r = 0; r < 32 * TM; r += 64 / PIECES) {
      const int row = r + lane / PIECES;
      if (mw + row >= g.M) continue;
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(mine + row * PITCH16 + 2 * col);
      uint16_t* y = static_cast<uint16_t*>(g.y) + (mw + row) * g.N + nw + col;
      if (left >= 8) {
        *reinterpret_cast<u32x4_e2*>(y) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < left) y[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      }
    }
    return;
  }
  float* out = split ? g.part + (int64_t)blockIdx.y * g.M * g.N : static_cast<float*>(g.y);
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += TP) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const f32x4_t b = bias_of(j, v);
#pragma unroll
        for (int i = 0; i < TP; ++i)
          *reinterpret_cast<f32x4_t*>(mine + (32 * i + l32) * PITCH32 + 128 * j + 32 * v + 16 * half) =
              values(i0 + i, j, v, b);
      }
    settle();
    constexpr int PIECES = 8 * TN;  // of 4 values a row
    const int col = 4 * (lane % PIECES), left = g.N - nw - col;
#pragma unroll
    for (int r = 0; r < 32 * TP; r += 64 / PIECES) {
      const int row = r + lane / PIECES;
      const int64_t m = mw + 32 * i0 + row;
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(mine + row * PITCH32 + 4 * col);
      if (m >= g.M) continue;
      float* y = out + m * g.N + nw + col;
      if (left >= 4) {
        *reinterpret_cast<u32x4_e4*>(y) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t b = w[e];
          if (e < left) y[e] = __builtin_bit_cast(float, b);
        }
      }
    }
    settle();
  }
}

// tile id of g's
template <int TM, int TN, bool WIDE>
__device__ __forceinline__ void gemm_tile_of(const GemmK& g, int id, uint8_t* smem) {
  int tm, tn;
  tile_at(xcd_run(id, g.tiles_m * g.tiles_n), g.tiles_m, g.tiles_n, tm, tn);
  gemm_tile<TM, TN, WIDE>(g, (int64_t)tm * 64 * TM, (int64_t)tn * 64 * TN, smem);
}

template <int TM, int TN, bool WIDE>
__global__ void __launch_bounds__(256, TM * TN > 4 ? 1 : 2) k_fp8_gemm(const GemmK g) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Tile<TM, TN>::LDS];
  gemm_tile_of<TM, TN, WIDE>(g, blockIdx.x, smem);
}

// 256 x 256 tiles, the last of them in parts: g.whole tiles (whole rounds of the CUs, or
// none), then each of the others as two of 256 x 128 or four of 128 x 128, a CU's work each.
// 4096 x 14336 x 4096 (3.5 rounds) 248 -> 238 us, 4352 x 4352 x 4096 (1.13) 103 -> 83;
// float32 results 421 -> 395 and 185 -> 141.
template <bool WIDE>
__global__ void __launch_bounds__(256, 1) k_fp8_gemm_tail(const GemmK g) {
  using T = Tile<4, 4>;
  static_assert(Tile<4, 2>::LDS <= T::LDS && Tile<2, 2>::LDS <= T::LDS, "one region for all");
  __shared__ __attribute__((aligned(16))) uint8_t smem[T::LDS];
  const int id = blockIdx.x;
  int tm, tn;
  if (id < g.whole) {
    tile_at(xcd_run(id, g.whole), g.tiles_m, g.tiles_n, tm, tn);
    gemm_tile<4, 4, WIDE>(g, (int64_t)tm * T::BM, (int64_t)tn * T::BN, smem);
    return;
  }
  const int t = xcd_run(id - g.whole, gridDim.x - g.whole);
  tile_at(g.whole + t / g.parts, g.tiles_m, g.tiles_n, tm, tn);
  const int part = __builtin_amdgcn_readfirstlane(t % g.parts);
  const int64_t m0 = (int64_t)tm * T::BM + 128 * (part >> 1);
  const int64_t n0 = (int64_t)tn * T::BN + 128 * (part & 1);
  if (m0 >= g.M || n0 >= g.N) return;
  if (g.parts == 2)
    gemm_tile<4, 2, WIDE>(g, m0, n0, smem);
  else
    gemm_tile<2, 2, WIDE>(g, m0, n0, smem);
}

// the slices' partial sums, added in slice order, plus bias
__global__ void __launch_bounds__(256) k_fp8_join(const GemmK g) {
  const int64_t n4 = (g.N + 3) / 4;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = t / n4;
  const int n = (int)(t % n4) * 4;
  if (m >= g.M) return;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool vec = g.N % 4 == 0;
  for (int k = 0; k < g.slices; ++k) {
    const float* p = g.part + ((int64_t)k * g.M + m) * g.N + n;
    if (vec) {
      s += *reinterpret_cast<const f32x4_t*>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < g.N) s[e] += p[e];
    }
  }
  store4(g, m, n, s, vec && ((uintptr_t)g.y & 15) == 0);
}

// k_fp8_mid: few tiles.  A workgroup owns a 32 x 32 tile of y, and its waves take
// every kMidWaves-th block of K, each through two slots of LDS of its own: whole
// rows of 128 bytes are copied (read straight into MFMA registers, 32 lines a load,
// the same bytes take the load path twice as long: 11.7 against 6.6 us at 256 x 1024 x
// 4096), and no wave waits for another until their partial tiles meet in LDS and are
// added in wave order.  Bound by the latency of a wave's chain of blocks.  (Tiles of
// 32 x 64 and 64 x 64 leave fewer workgroups: 8.2 and 10.5 us; eight waves: 6.7.)  Copy
// j of a fragment fills 8 rows; slot s of it holds row s / 8, piece (s % 8) ^ (row % 8)
// of that row's eight.
constexpr int kMidWaves = 4;

constexpr int kMidSlot = 8192 + 256;  // B's 32 rows, A's, and their scale dwords
constexpr int kMidLds = kMidWaves * 2 * kMidSlot;

template <bool WIDE>
__device__ __forceinline__ void mid_tile(const GemmK& g, int id, uint8_t* smem) {
  constexpr int LD = 36;                     // floats of a partial tile's row
  constexpr int SLOT = kMidSlot;
  constexpr int OPS = 9;                     // copies of a block
  static_assert(32 * LD * 4 <= 2 * SLOT, "a partial tile fits a wave's slots");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, l32 = lane & 31;
  int tm, tn;
  tile_at(xcd_run(id, g.tiles_m * g.tiles_n), g.tiles_m, g.tiles_n, tm, tn);
  const int64_t m0 = 32 * (int64_t)tm, n0 = 32 * (int64_t)tn;
  const int mlast = (int)min((int64_t)32, g.M - m0) - 1, nlast = (int)min((int64_t)32, g.N - n0) - 1;
  const __amdgpu_buffer_rsrc_t ra = descriptor(g.a + m0 * g.lda, (mlast + 1) * g.lda);
  const __amdgpu_buffer_rsrc_t rb = descriptor(g.b + n0 * g.ldb, (nlast + 1) * g.ldb);
  int offa[4], offb[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int row = 8 * c + (lane >> 3), piece = 16 * ((lane & 7) ^ (row & 7));
    offa[c] = min(row, mlast) * (int)g.lda + piece;
    offb[c] = min(row, nlast) * (int)g.ldb + piece;
  }
  // the scale dword of B's row l32 (lower lanes) or A's
  const uint8_t* sp = half ? g.as + 4 * (m0 + min(l32, mlast)) : g.bs + 4 * (n0 + min(l32, nlast));
  const int64_t sg = 4 * (int64_t)(half ? g.M : g.N);
  uint8_t* mine = smem + wave * 2 * SLOT;
  auto issue = [&](int kb, int slot) {
    uint8_t* base = mine + slot * SLOT;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      buffer_copy16(rb, offb[c], kb * kFp8Block, base + 1024 * c);
      buffer_copy16(ra, offa[c], kb * kFp8Block, base + 4096 + 1024 * c);
    }
    __builtin_amdgcn_global_load_lds(sp + (kb >> 2) * sg, base + 8192, 4, 0, 0);
  };
  f32x16_t acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
  auto piece = [&](const uint8_t* base, int p) {
    return *reinterpret_cast<const u32x4_t*>(base + 128 * l32 + 16 * (p ^ (l32 & 7)));
  };
  auto frag = [&](const uint8_t* base, int kk) {
    const u32x4_t a = piece(base, 4 * kk + 2 * half), b = piece(base, 4 * kk + 2 * half + 1);
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3],
                   (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
  };
  if (wave < g.KB) issue(wave, 0);
  int slot = 0;
  for (int kb = wave; kb < g.KB; kb += kMidWaves, slot ^= 1) {
    // the next block's slot was read to the end before this point
    if (kb + kMidWaves < g.KB) {
      issue(kb + kMidWaves, slot ^ 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(OPS) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const uint8_t* base = mine + slot * SLOT;
    const i32x8_t fb[2] = {frag(base, 0), frag(base, 1)};
    const i32x8_t fa[2] = {frag(base + 4096, 0), frag(base + 4096, 1)};
    const uint32_t cb = base[8192 + 4 * l32 + (kb & 3)], ca = base[8192 + 128 + 4 * l32 + (kb & 3)];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      if constexpr (WIDE) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              decode_bf16(fb[kk][2 * s], fb[kk][2 * s + 1], scale_f32(cb)),
              decode_bf16(fa[kk][2 * s], fa[kk][2 * s + 1], scale_f32(ca)), acc, 0, 0, 0);
      } else {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[kk], fa[kk], acc, 0, 0, 0, (int)cb,
                                                              0, (int)ca);
      }
    }
  }
  __syncthreads();  // every wave is done with its slots: they become the partial tiles
  // accumulator element v of lane l: column 8 (v / 4) + 4 (l / 32) + v % 4 of row l % 32
  auto part = [&](int w, int row, int col) {
    return reinterpret_cast<f32x4_t*>(smem + w * 2 * SLOT + (row * LD + col) * 4);
  };
#pragma unroll
  for (int v = 0; v < 4; ++v)
    *part(wave, l32, 8 * v + 4 * half) =
        f32x4_t{acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]};
  __syncthreads();
  static_assert(64 * kMidWaves == 256, "four columns of the tile for each thread");
  const int row = tid / 8, col = 4 * (tid % 8);
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kMidWaves; ++w) s += *part(w, row, col);
  store4(g, m0 + row, (int)n0 + col, s, g.N % 4 == 0 && ((uintptr_t)g.y & 15) == 0);
}

template <bool WIDE>
__global__ void __launch_bounds__(64 * kMidWaves) k_fp8_mid(const GemmK g) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kMidLds];
  mid_tile<WIDE>(g, blockIdx.x, smem);
}

// k_fp8_few: at most 16 rows of x.  Bound by the weight's bytes, so a workgroup
// owns 16 columns of y over all of K, its W waves taking every W-th block
// straight from memory into registers: lane l holds row l % 16 of each operand
// and, of the block's 128 elements, the 16 at 16 (l / 16) and the 16 at
// 64 + 16 (l / 16).  XT = uint8_t reads x's codes; otherwise x itself is read and
// quantised in registers, with the same arithmetic as the row quantiser: a row's
// block is in the four lanes l % 16 + 16 q, two shuffles find its maximum.
template <int W, typename XT, bool WIDE>
__global__ void __launch_bounds__(64 * W)
    k_fp8_few(const GemmK g, const XT* __restrict__ x, int64_t ldx, int K) {
  constexpr int U = 4;  // blocks of a wave in flight
  __shared__ float part[W][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane >> 4, l16 = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int64_t n = min(n0 + l16, g.N - 1);
  const int64_t m = min(l16, g.M - 1);
  const uint8_t* bp = g.b + n * g.ldb + 16 * q;
  f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave; k0 < g.KB; k0 += W * U) {
    u32x4_t b[U][2];
    uint32_t bsc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * W;
      if (kb >= g.KB) break;
      b[u][0] = *reinterpret_cast<const u32x4_t*>(bp + (int64_t)kb * kFp8Block);
      b[u][1] = *reinterpret_cast<const u32x4_t*>(bp + (int64_t)kb * kFp8Block + 64);
      bsc[u] = g.bs[((int64_t)(kb >> 2) * g.N + n) * 4 + (kb & 3)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * W;
      if (kb >= g.KB) break;
      i32x8_t fa;
      uint32_t asc;
      if constexpr (sizeof(XT) == 1) {
        const uint8_t* p = g.a + m * g.lda + (int64_t)kb * kFp8Block + 16 * q;
        const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(p);
        const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(p + 64);
        fa = i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                     (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
        asc = g.as[((int64_t)(kb >> 2) * g.M + m) * 4 + (kb & 3)];
      } else {
        float v[4][8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int at = kb * kFp8Block + 64 * (c >> 1) + 16 * q + 8 * (c & 1);
          load8(x + m * ldx, at, K, v[c]);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max(top, finite_bits(v[c][e]));
        }
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        asc = fp8_scale_byte(top);
        const float inv = fp8_inverse(asc);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          fa[2 * c] = (int)fp8_pack4(v[c][0], v[c][1], v[c][2], v[c][3], inv);
          fa[2 * c + 1] = (int)fp8_pack4(v[c][4], v[c][5], v[c][6], v[c][7], inv);
        }
      }
      const i32x8_t fb = {(int)b[u][0][0], (int)b[u][0][1], (int)b[u][0][2], (int)b[u][0][3],
                          (int)b[u][1][0], (int)b[u][1][1], (int)b[u][1][2], (int)b[u][1][3]};
      if constexpr (WIDE) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              decode_bf16(fb[2 * s], fb[2 * s + 1], scale_f32(bsc[u])),
              decode_bf16(fa[2 * s], fa[2 * s + 1], scale_f32(asc)), acc, 0, 0, 0);
      } else {
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, 0, 0, 0, (int)bsc[u], 0,
                                                              (int)asc);
      }
    }
  }
  // accumulator element v of lane l: column 4 (l / 16) + v of row l % 16
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][l16][4 * q + v] = acc[v];
  __syncthreads();
  const int row = tid >> 4, col = tid & 15;
  if (tid >= 256 || row >= g.M || n0 + col >= g.N) return;
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += part[w][row][col];
  if (g.bias) s += g.bias[n0 + col];
  const int64_t at = (int64_t)row * g.N + n0 + col;
  if (g.y_bf16)
    static_cast<uint16_t*>(g.y)[at] = bf16_rne(s);
  else
    static_cast<float*>(g.y)[at] = s;
}

// column sums from the tile quantiser's partials: 16 columns a workgroup, whose 16
// threads of a column take the row blocks in turn; the first adds them in order
struct ColSum {
  const float* part;  // [nrb][N]
  float* out;
  int nrb, N;
};
__device__ __forceinline__ void column_sums(const ColSum& c, int id, float (&lds)[16][17]) {
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4, n = id * 16 + col;
  float s = 0.0f;
  if (n < c.N)
#pragma unroll 4
    for (int r = lane; r < c.nrb; r += 16) s += c.part[(int64_t)r * c.N + n];
  lds[lane][col] = s;
  __syncthreads();
  if (lane != 0 || n >= c.N) return;
  s = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += lds[k][col];
  c.out[n] = s;
}
__global__ void __launch_bounds__(256) k_fp8_colsum(const ColSum c) {
  __shared__ float lds[16][17];
  column_sums(c, blockIdx.x, lds);
}

// k_fp8_back: the small products of a layer's backward and its column sums, in one
// launch: g[0]'s tiles (count[0] workgroups), g[1]'s, then the sums.  Each alone
// is a few microseconds of latency on part of the CUs: 256 x 1024 x 1024, the whole
// backward, 17.8 us with a launch for each, 13.5 so.
struct BackK {
  GemmK g[2];
  int count[2], mid[2];
  ColSum sums;
};
template <bool MID>
__global__ void __launch_bounds__(256, 2) k_fp8_back(const BackK b) {
  constexpr int TILE = Tile<1, 1>::LDS;
  __shared__ __attribute__((aligned(16))) uint8_t smem[MID && kMidLds > TILE ? kMidLds : TILE];
  int id = blockIdx.x;
  const int second = id >= b.count[0];
  if (second) id -= b.count[0];
  if (second && id >= b.count[1])
    return column_sums(b.sums, id - b.count[1], *reinterpret_cast<float(*)[16][17]>(smem));
  const GemmK& g = b.g[second];
  if (MID && b.mid[second]) {
    if (g.y_bf16) mid_tile<false>(g, id, smem);
    else mid_tile<true>(g, id, smem);
  } else {
    if (g.y_bf16) gemm_tile_of<1, 1, false>(g, id, smem);
    else gemm_tile_of<1, 1, true>(g, id, smem);
  }
}

// ----------------------------------------------------------------- host side

// y = A B^T + bias, from A's codes
struct Fp8Gemm {
  const uint8_t *a, *as, *b, *bs;
  int64_t M, N, K;  // K >= 0
  const float* bias;
  void* y;
  int32_t y_dtype;
  void* ws;
};

constexpr int kFewRows = 16;

constexpr int kCUs = 256;

enum Kernel { kTiles256, kTiles256Tail, kTiles128, kTiles64, kMid };

struct Plan {
  Kernel kernel;
  int slices;  // of K
};

// The parts of each 256-tile left over by whole rounds of the CUs (all tiles, if there is
// no whole round): as many as keep every part on a CU of its own.
int tail_parts(int64_t tiles) {
  const int64_t left = tiles % kCUs;
  if (left == 0) return 1;
  return left <= kCUs / 4 ? 4 : left <= kCUs / 2 ? 2 : 1;
}

// The kernel for more than kFewRows rows.  A larger tile reads fewer bytes for its
// products (256 x 256 reach 2560 TFLOP/s at 8192^3, 128 x 128, two a CU, 1780), but a tile
// is one CU's work.  The product alone, us, bf16 result (float32 result), by the number of
// tiles; the kernel of the rule first:
//  - 256-tiles beyond half a round of them, against 128-tiles: 256 of them, 4096 x 4096 x
//    4096 63 and 88 (112, 123), K = 512 21.4 and 23.3; 144 of them, 2304 x 4096 x 4096 50 and
//    57 (87, 85), where a short K would have been as fast in 128-tiles (K = 512: 18.8, 18.1).
//  - A quarter to half a round as one round of their 256 x 128 halves, against 128-tiles:
//    2048 x 4096 x 4096 41 and 44, 700 x 6000 x 4096 32 and 39, K = 2048 20.5 and 22.4.  A
//    shorter K gains nothing (K = 1024: 15.5 and 15.1) and a float32 result nothing at any
//    (64 and 65; K = 1024 22.5 and 20.6): they take 128-tiles.
//  - 128-tiles from three quarters of the CUs on, against 64-tiles: 195 of them, 1664 x 1920 x
//    4096 23 and 37 (32, 47), K = 512 8.1 and 9.2 (11.6, 11.4).  120 of them, on the rule's
//    other side: 64-tiles 20.8, 128-tiles 21.3 (26, 31), K = 512 6.5 and 7.5.  In between, once
//    64-tiles are more than two a CU, it depends on K: 169 of them, 64-tiles 8.1 and
//    128-tiles 7.8 at K = 512 (9.7, 11.2), 29.4 and 22.5 at K = 4096 (37, 32).
//  - Slices of a long K over fewer 128-tiles, whose float32 partial sums a second kernel
//    adds: as many as fill those three quarters, of 32 blocks at least.  1280 x 1280 (100
//    tiles), K = 8192 in two: 30 and 36 unsliced, 37 in 64-tiles (38, 51, 45); K = 32768 80
//    and 126 (110, 183).  512 x 1024 (32 tiles), K = 32768 in eight: 35 and 46 in k_fp8_mid
//    (44, 52).  K = 4096, which is not sliced: 64-tiles 19.8, two slices 21.4 (24.8, 26.1).
//    Below 16 tiles k_fp8_mid has the workgroups to do without (256 x 512 x 16384: 13.5,
//    eight slices 19).
//  - What is left is bound by latency.  Up to 768 tiles of 32 x 32 k_fp8_mid, against
//    64-tiles: 256 x 1024 x 4096 5.9 and 10.7 (7.2, 16.8), 512 x 1536 x 1024 6.4 and 5.8
//    (7.0, 7.6), K = 4096 12.6 and 13.0 (14.3, 17.7); more are 64-tiles: 1024 of them, 256 x
//    4096 x 1024, 6.0 and 7.3 (7.8, 8.6).
// `wide`, a float32 result, never changes the slices.
Plan plan(int64_t M, int64_t N, int64_t K, bool wide) {
  auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
  const int64_t KB = fp8_blocks(K);
  if (tiles(256) > kCUs / 2 ||
      (tiles(256) > kCUs / 4 && tiles(128) > kCUs && KB >= 16 && !wide))
    return {tail_parts(tiles(256)) > 1 ? kTiles256Tail : kTiles256, 1};
  if (tiles(128) >= 192) return {kTiles128, 1};
  for (int s = 2; s <= 16; s *= 2)
    if (KB / s >= 32 && tiles(128) * s >= 192 && tiles(128) >= 16) return {kTiles128, s};
  return {tiles(32) <= 768 ? kMid : kTiles64, 1};
}

GemmK kernel_args(const Fp8Gemm& g, int slices) {
  GemmK k = {};
  k.a = g.a; k.as = g.as; k.b = g.b; k.bs = g.bs;
  k.bias = g.bias; k.y = g.y; k.part = static_cast<float*>(g.ws);
  k.KB = (int)fp8_blocks(g.K);
  k.lda = k.ldb = fp8_pitch(g.K);
  k.M = (int)g.M; k.N = (int)g.N;
  k.y_bf16 = g.y_dtype == ASP_BF16;
  k.slices = slices;
  return k;
}

template <int TM, int TN, bool WIDE>
int32_t launch_tiles(GemmK k, hipStream_t st) {
  constexpr int64_t BM = 64 * TM, BN = 64 * TN;
  const int64_t tm = (k.M + BM - 1) / BM, tn = (k.N + BN - 1) / BN;
  if (tm * tn > kMaxLanes / 256) return fail(ASP_ERR_SHAPE, "output too large for one launch");
  k.tiles_m = (int)tm;
  k.tiles_n = (int)tn;
  k_fp8_gemm<TM, TN, WIDE><<<dim3((unsigned)(tm * tn), (unsigned)k.slices), 256, 0, st>>>(k);
  return launch_status("fp8 gemm");
}

template <bool WIDE>
int32_t launch_tail(GemmK k, hipStream_t st) {
  k.tiles_m = (k.M + 255) / 256;
  k.tiles_n = (k.N + 255) / 256;
  const int64_t tiles = (int64_t)k.tiles_m * k.tiles_n;
  if (tiles > kMaxLanes / 256 - kCUs) return fail(ASP_ERR_SHAPE, "output too large for one launch");
  const int64_t left = tiles % kCUs;
  k.whole = (int)(tiles - left);
  k.parts = tail_parts(tiles);
  k_fp8_gemm_tail<WIDE><<<dim3((unsigned)(k.whole + k.parts * left)), 256, 0, st>>>(k);
  return launch_status("fp8 gemm");
}

template <bool WIDE>
int32_t launch_mid(GemmK k, hipStream_t st) {
  const int64_t tm = (k.M + 31) / 32, tn = (k.N + 31) / 32;
  k.tiles_m = (int)tm;
  k.tiles_n = (int)tn;
  k_fp8_mid<WIDE><<<dim3((unsigned)(tm * tn)), 64 * kMidWaves, 0, st>>>(k);
  return launch_status("fp8 mid gemm");
}

// Waves over which k_fp8_few splits K, by its blocks (4, 8, 16 waves, M = 1, bf16, us): N =
// 1024, K = 512 4.2 4.2 4.2, 1024 5.3 4.8 4.9, 2048 8.0 6.6 5.9, 16384 46 32 27.  At N =
// 14336, 896 workgroups, fewer waves lose less or nothing (K = 1024 9.1 9.6 13.1, 4096 28.5
// 27.5 31.3): the rule is for the columns of one round of the CUs.
int few_waves(int KB) { return KB >= 16 ? 16 : KB >= 8 ? 8 : 4; }

template <typename XT, bool WIDE>
void launch_few_as(const GemmK& k, const XT* x, int64_t ldx, int64_t K, hipStream_t st) {
  const dim3 grid((unsigned)(((int64_t)k.N + 15) / 16));
  const int waves = few_waves(k.KB);
  if (waves == 16) k_fp8_few<16, XT, WIDE><<<grid, 1024, 0, st>>>(k, x, ldx, (int)K);
  else if (waves == 8) k_fp8_few<8, XT, WIDE><<<grid, 512, 0, st>>>(k, x, ldx, (int)K);
  else k_fp8_few<4, XT, WIDE><<<grid, 256, 0, st>>>(k, x, ldx, (int)K);
}

template <typename XT>
int32_t launch_few(const GemmK& k, const XT* x, int64_t ldx, int64_t K, hipStream_t st) {
  if (((int64_t)k.N + 15) / 16 > kMaxLanes / (64 * few_waves(k.KB)))
    return fail(ASP_ERR_SHAPE, "output too large for one launch");
  if (k.y_bf16) launch_few_as<XT, false>(k, x, ldx, K, st);
  else launch_few_as<XT, true>(k, x, ldx, K, st);
  return launch_status("fp8 few-row gemm");
}

// x itself is taken where M is small enough, and quantised inside
bool fp8_fuses(int64_t M) { return M <= kFewRows; }

size_t fp8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewRows) return 0;
  const Plan p = plan(M, N, K, false);
  return p.slices > 1 ? up256((size_t)p.slices * M * N * 4) : 0;
}

int32_t fp8_gemm_fused(const Fp8Gemm& g, const void* x, int32_t x_dtype, int64_t ldx,
                       hipStream_t st) {
  const GemmK k = kernel_args(g, 1);
  if (x_dtype == ASP_BF16)
    return launch_few(k, static_cast<const uint16_t*>(x), ldx, g.K, st);
  return launch_few(k, static_cast<const float*>(x), ldx, g.K, st);
}

template <bool WIDE>
int32_t launch_plan(const Plan& p, const GemmK& k, hipStream_t st) {
  switch (p.kernel) {
    case kTiles256: return launch_tiles<4, 4, WIDE>(k, st);
    case kTiles256Tail: return launch_tail<WIDE>(k, st);
    case kTiles128: return launch_tiles<2, 2, WIDE>(k, st);
    case kTiles64: return launch_tiles<1, 1, WIDE>(k, st);
    default: return launch_mid<WIDE>(k, st);
  }
}

int32_t fp8_gemm_impl(const Fp8Gemm& g, hipStream_t st) {
  if (g.M <= kFewRows)
    return launch_few(kernel_args(g, 1), g.a, 0, g.K, st);
  const Plan p = plan(g.M, g.N, g.K, g.y_dtype != ASP_BF16);
  const GemmK k = kernel_args(g, p.slices);
  ASP_TRY(k.y_bf16 ? launch_plan<false>(p, k, st) : launch_plan<true>(p, k, st));
  if (p.slices == 1) return ASP_OK;
  const int64_t blocks = (g.M * ((g.N + 3) / 4) + 255) / 256;
  k_fp8_join<<<dim3((unsigned)blocks), 256, 0, st>>>(k);
  return launch_status("fp8 join");
}

// Latency-bound products, which share a launch with others (k_fp8_back): the backward asks
// this of each by itself, so that a gradient's bits do not depend on which others are
// wanted.  Up to kFewRows rows too: k_fp8_few would be a launch beside the column sums'
// (dx and db of 16 x 14336 x 4096: 18.3 us, with it 24.7; 1 x 4096 x 1024: 10.1 and 11.6).
bool small(const Fp8Gemm& g) {
  const Plan p = plan(g.M, g.N, g.K, g.y_dtype != ASP_BF16);
  return p.slices == 1 && (p.kernel == kMid || p.kernel == kTiles64);
}

// up to two small products, and column sums where c.out is given
int32_t launch_back(int n, const Fp8Gemm* g, const ColSum& c, hipStream_t st) {
  BackK b = {};
  b.sums = c;
  int64_t blocks = c.out ? (c.N + 15) / 16 : 0;
  for (int i = 0; i < n; ++i) {
    GemmK& k = b.g[i] = kernel_args(g[i], 1);
    b.mid[i] = plan(g[i].M, g[i].N, g[i].K, !k.y_bf16).kernel == kMid;
    const int t = b.mid[i] ? 32 : 64;
    k.tiles_m = (k.M + t - 1) / t;
    k.tiles_n = (k.N + t - 1) / t;
    b.count[i] = k.tiles_m * k.tiles_n;
    blocks += b.count[i];
  }
  if (b.mid[0] || b.mid[1]) k_fp8_back<true><<<dim3((unsigned)blocks), 256, 0, st>>>(b);
  else k_fp8_back<false><<<dim3((unsigned)blocks), 256, 0, st>>>(b);
  return launch_status("fp8 backward");
}

int32_t check_gemm(int64_t M, int64_t N, int64_t K) {
  ASP_TRY(check_fp8_dims(M, K, "M", "K"));
  if (N < 1 || N > (1 << 30)) return fail(ASP_ERR_SHAPE, "N=%lld outside [1, 2^30]", (long long)N);
  return ASP_OK;
}

// the backward contracts over M and N too
int32_t check_backward(int64_t M, int64_t N, int64_t K) {
  ASP_TRY(check_gemm(M, N, K));
  if (M > kMaxK || N > kMaxK)
    return fail(ASP_ERR_SHAPE, "M=%lld, N=%lld: the backward takes at most %lld of each",
                (long long)M, (long long)N, (long long)kMaxK);
  return ASP_OK;
}

struct FwdWs {
  size_t codes, scales, gemm, total;
};
FwdWs forward_ws(int64_t M, int64_t N, int64_t K) {
  FwdWs L = {0, 0, 0, 0};
  if (fp8_fuses(M)) return L;
  L.scales = up256(fp8_code_bytes(M, K));
  L.gemm = L.scales + up256(fp8_scale_bytes(M, K));
  L.total = L.gemm + fp8_gemm_workspace(M, N, K);
  return L;
}

struct BwdWs {
  size_t dyc, dys, dytc, dyts, xtc, xts, sums, gemm, total;
};
BwdWs backward_ws(int64_t M, int64_t N, int64_t K) {
  BwdWs L;
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t here = at;
    at += up256(b);
    return here;
  };
  L.dyc = take(fp8_code_bytes(M, N));
  L.dys = take(fp8_scale_bytes(M, N));
  L.dytc = take(fp8_code_bytes(N, M));
  L.dyts = take(fp8_scale_bytes(N, M));
  L.xtc = take(fp8_code_bytes(K, M));
  L.xts = take(fp8_scale_bytes(K, M));
  L.sums = take((size_t)fp8_blocks(M) * N * 4);
  // one region: the two products run one after the other on one stream
  const size_t dx = fp8_gemm_workspace(M, K, N), dw = fp8_gemm_workspace(N, K, M);
  L.gemm = take(dx > dw ? dx : dw);
  L.total = at;
  return L;
}

}  // namespace
}  // namespace asp

using namespace asp;

extern "C" {

int32_t asp_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  clear_error();
  ASP_TRY(check_gemm(M, N, K));
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  *bytes = fp8_gemm_workspace(M, N, K);
  return ASP_OK;
}

int32_t asp_fp8_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                     const uint8_t* b_scales, int64_t M, int64_t N, int64_t K, const float* bias,
                     void* y, int32_t y_dtype, void* workspace, size_t workspace_bytes,
                     void* stream) {
  clear_error();
  ASP_TRY(check_gemm(M, N, K));
  ASP_TRY(check_io_dtype(y_dtype, "y_dtype"));
  if (M == 0) return ASP_OK;
  ASP_TRY(check_ptr(a_codes, "a_codes", true));
  ASP_TRY(check_ptr(a_scales, "a_scales", true));
  ASP_TRY(check_ptr(b_codes, "b_codes", true));
  ASP_TRY(check_ptr(b_scales, "b_scales", true));
  if (bias) ASP_TRY(check_matrix(bias, ASP_F32, 0, 0, "bias"));
  ASP_TRY(check_matrix(y, y_dtype, N, N, "y"));
  ASP_TRY(check_workspace(workspace, workspace_bytes, fp8_gemm_workspace(M, N, K)));
  const Fp8Gemm g = {a_codes, a_scales, b_codes, b_scales, M, N, K, bias, y, y_dtype, workspace};
  return fp8_gemm_impl(g, (hipStream_t)stream);
}

int32_t asp_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  clear_error();
  ASP_TRY(check_gemm(M, N, K));
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  *bytes = forward_ws(M, N, K).total;
  return ASP_OK;
}

int32_t asp_fp8_forward(const void* x, int32_t x_dtype, int64_t ldx, int64_t M, int64_t N,
                        int64_t K, const uint8_t* w_codes, const uint8_t* w_scales,
                        const float* bias, void* y, int32_t y_dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  clear_error();
  ASP_TRY(check_gemm(M, N, K));
  ASP_TRY(check_io_dtype(x_dtype, "x_dtype"));
  ASP_TRY(check_io_dtype(y_dtype, "y_dtype"));
  if (M == 0) return ASP_OK;
  ASP_TRY(check_matrix(x, x_dtype, K, ldx, "x"));
  ASP_TRY(check_ptr(w_codes, "w_codes", true));
  ASP_TRY(check_ptr(w_scales, "w_scales", true));
  if (bias) ASP_TRY(check_matrix(bias, ASP_F32, 0, 0, "bias"));
  ASP_TRY(check_matrix(y, y_dtype, N, N, "y"));
  const FwdWs L = forward_ws(M, N, K);
  ASP_TRY(check_workspace(workspace, workspace_bytes, L.total));
  const hipStream_t st = (hipStream_t)stream;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  Fp8Gemm g = {nullptr, nullptr, w_codes, w_scales, M, N, K, bias, y, y_dtype, nullptr};
  if (fp8_fuses(M)) return fp8_gemm_fused(g, x, x_dtype, ldx, st);
  g.a = base + L.codes;
  g.as = base + L.scales;
  g.ws = base + L.gemm;
  ASP_TRY(fp8_quantize_rows(x, x_dtype, M, K, ldx, base + L.codes, base + L.scales, st));
  return fp8_gemm_impl(g, st);
}

int32_t asp_fp8_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  clear_error();
  ASP_TRY(check_backward(M, N, K));
  if (!bytes) return fail(ASP_ERR_ARG, "null output pointer");
  *bytes = backward_ws(M, N, K).total;
  return ASP_OK;
}

int32_t asp_fp8_backward(const void* dy, int32_t dy_dtype, int64_t lddy, const void* x,
                         int32_t x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                         const uint8_t* wt_codes, const uint8_t* wt_scales, void* dx,
                         int32_t dx_dtype, void* dw, int32_t dw_dtype, float* db, void* workspace,
                         size_t workspace_bytes, void* stream) {
  clear_error();
  ASP_TRY(check_backward(M, N, K));
  ASP_TRY(check_io_dtype(dy_dtype, "dy_dtype"));
  if (dw) ASP_TRY(check_io_dtype(x_dtype, "x_dtype"));
  if (dx) ASP_TRY(check_io_dtype(dx_dtype, "dx_dtype"));
  if (dw) ASP_TRY(check_io_dtype(dw_dtype, "dw_dtype"));
  if (!dx && !dw && !db) return ASP_OK;
  if (M > 0) {
    ASP_TRY(check_matrix(dy, dy_dtype, N, lddy, "dy"));
    if (dw) ASP_TRY(check_matrix(x, x_dtype, K, ldx, "x"));
    if (dx) {
      ASP_TRY(check_ptr(wt_codes, "wt_codes", true));
      ASP_TRY(check_ptr(wt_scales, "wt_scales", true));
      ASP_TRY(check_matrix(dx, dx_dtype, K, K, "dx"));
    }
  }
  if (dw) ASP_TRY(check_matrix(dw, dw_dtype, K, K, "dw"));
  if (db) ASP_TRY(check_matrix(db, ASP_F32, 0, 0, "db"));
  const BwdWs L = backward_ws(M, N, K);
  ASP_TRY(check_workspace(workspace, workspace_bytes, L.total));
  const hipStream_t st = (hipStream_t)stream;
  uint8_t* base = static_cast<uint8_t*>(workspace);
  Fp8TileJob jobs[2] = {
      {dy, M, N, lddy, dx ? base + L.dyc : nullptr, base + L.dys, dw ? base + L.dytc : nullptr,
       base + L.dyts, db ? reinterpret_cast<float*>(base + L.sums) : nullptr, dy_dtype, 0},
      {x, M, K, ldx, nullptr, nullptr, base + L.xtc, base + L.xts, nullptr, x_dtype, 0}};
  ASP_TRY(fp8_quantize_tiles(dw ? 2 : 1, jobs, st));
  const ColSum sums = {reinterpret_cast<const float*>(base + L.sums), db, (int)fp8_blocks(M), (int)N};
  Fp8Gemm g[2];
  int n = 0;
  if (dx && M > 0)
    g[n++] = {base + L.dyc, base + L.dys, wt_codes, wt_scales, M, K, N, nullptr,
              dx, dx_dtype, base + L.gemm};
  if (dw)
    g[n++] = {base + L.dytc, base + L.dyts, base + L.xtc, base + L.xts, N, K, M, nullptr,
              dw, dw_dtype, base + L.gemm};
  Fp8Gemm joint[2], alone[2];
  int nj = 0, na = 0;
  for (int i = 0; i < n; ++i) (small(g[i]) ? joint[nj++] : alone[na++]) = g[i];
  if (nj > 0) {
    ASP_TRY(launch_back(nj, joint, sums, st));
  } else if (db) {
    k_fp8_colsum<<<dim3((unsigned)((N + 15) / 16)), 256, 0, st>>>(sums);
    ASP_TRY(launch_status("fp8 column sums"));
  }
  for (int i = 0; i < na; ++i) ASP_TRY(fp8_gemm_impl(alone[i], st));
  return ASP_OK;
}

}  // extern "C"

// Quantisers of the 8-bit (block-128) format and their C entry points.
//
// All are bound by memory: a bf16 matrix is read once (2 bytes an element) and
// its codes written once (1 byte).  4096 x 4096 bf16 rows 11 us (4.6 TB/s); 8192 x 4096
// dy and x, transposed codes of both and rows and column sums of dy, 53 us (4.4 TB/s); a
// 4096 x 14336 bf16 weight, both forms, 47 us (5.0 TB/s).
#include "asp_fp8.h"

namespace asp {
namespace {

// Row form.  One wave takes 512 consecutive elements of a row: 8 for each lane
// (16-byte loads in bf16), a block for each 16 lanes, whose maximum is four DPP
// rotations, and the four blocks' scale bytes make the one dword that the
// scale layout keeps together.
template <typename XT>
__global__ void __launch_bounds__(256)
    k_fp8_rows(const XT* __restrict__ x, int64_t rows, int cols, int64_t ld, int groups,
               uint8_t* __restrict__ codes, uint32_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t row = w / groups;
  const int g = (int)(w % groups);
  if (row >= rows) return;  // the whole wave leaves
  const int c0 = 512 * g + 8 * lane;
  const int pitch = (cols + kFp8Block - 1) / kFp8Block * kFp8Block;
  float v[8];
  load8(x + row * ld, c0, cols, v);
  uint32_t u = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) u = max(u, finite_bits(v[e]));
  const uint32_t s = fp8_scale_byte(row16_max(u));
  const float inv = fp8_inverse(s);
  if (c0 < pitch)
    *reinterpret_cast<u32x2_t*>(codes + row * pitch + c0) =
        u32x2_t{fp8_pack4(v[0], v[1], v[2], v[3], inv), fp8_pack4(v[4], v[5], v[6], v[7], inv)};
  const int byte = c0 < pitch ? (int)s : (int)kFp8PadScale;
  const uint32_t word = (uint32_t)__builtin_amdgcn_readlane(byte, 0) |
                        (uint32_t)__builtin_amdgcn_readlane(byte, 16) << 8 |
                        (uint32_t)__builtin_amdgcn_readlane(byte, 32) << 16 |
                        (uint32_t)__builtin_amdgcn_readlane(byte, 48) << 24;
  if (lane == 0) scales[(int64_t)g * rows + row] = word;
}

struct TileArgs {
  Fp8TileJob j[2];
  int tiles0;  // workgroups of the first job
};

// Tile form: a workgroup of 512 reads a 128 x 128 tile once and writes from it the
// row form, the transposed form and the tile's column sums.  Thread t holds columns
// 8 (t % 16) .. +7 of rows 4 (t / 16) .. +3, as they lie in memory: a row's 128
// columns are one DPP row of lanes, and a column's 4 rows make 4 consecutive bytes of
// the transposed codes, which turn through LDS (dword index XOR 2 (column / 8), so that
// a wave's writes spread over the banks).  Rows and columns past the matrix count
// as zeros: they pad the last block.  4 rows a thread keep the kernel below 80 VGPRs; a
// workgroup of 256 with 8 rows a thread took 12% longer.
constexpr int kTileWaves = 8;

template <typename XT>
__device__ __forceinline__ void tile_body(const Fp8TileJob& j, int tile,
                                          uint32_t (&cmax)[kTileWaves][128],
                                          float (&csum)[kTileWaves][128],
                                          uint8_t (&turn)[128 * 128]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 15, rg = tid >> 4;
  const int ncb = (int)((j.cols + 127) / 128);
  const int rb = tile / ncb, cb = tile % ncb;
  const int64_t r0 = (int64_t)rb * 128 + 4 * rg, c0 = (int64_t)cb * 128 + 8 * cg;
  const XT* x = static_cast<const XT*>(j.in) + r0 * j.ld;
  Raw<XT> raw[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < j.rows) {
      if (j.cols >= 8) raw_load<false>(x + i * j.ld, (int)c0, (int)j.cols, raw[i]);
      else raw_load<true>(x + i * j.ld, (int)c0, (int)j.cols, raw[i]);
    }
  if (j.cols >= 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) raw_settle<false>((int)c0, (int)j.cols, raw[i]);
  // magnitudes: per row (this thread's 8 columns) and per column (its 4 rows)
  uint32_t ru[4], cu[8];
  float cs[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cu[e] = 0;
    cs[e] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
    unpack(raw[i], v);
    ru[i] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = finite_bits(v[e]);
      ru[i] = max(ru[i], u);
      cu[e] = max(cu[e], u);
      cs[e] += v[e];
    }
    ru[i] = row16_max(ru[i]);
  }
  if (j.codes_t || j.sums || j.square) {
    // the column results of the wave's four row groups, then of the waves
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cu[e] = max(cu[e], (uint32_t)__shfl_xor((int)cu[e], 16));
      cu[e] = max(cu[e], (uint32_t)__shfl_xor((int)cu[e], 32));
      if (j.sums) {
        cs[e] += __shfl_xor(cs[e], 16);
        cs[e] += __shfl_xor(cs[e], 32);
      }
      if (lane < 16) {
        cmax[wave][8 * cg + e] = cu[e];
        csum[wave][8 * cg + e] = cs[e];
      }
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t u = 0;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) {
        u = max(u, cmax[w][tid]);
        s += csum[w][tid];
      }
      cmax[0][tid] = u;
      if (j.sums && (int64_t)cb * 128 + tid < j.cols)
        j.sums[rb * j.cols + (int64_t)cb * 128 + tid] = s;
    }
    __syncthreads();
    const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(&cmax[0][8 * cg]);
    const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(&cmax[0][8 * cg + 4]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cu[e] = lo[e];
      cu[4 + e] = hi[e];
    }
  }
  if (j.square) {  // one scale for the tile: a DPP row's lanes hold every column group
    uint32_t u = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) u = max(u, cu[e]);
    u = row16_max(u);
#pragma unroll
    for (int e = 0; e < 8; ++e) cu[e] = u;
#pragma unroll
    for (int i = 0; i < 4; ++i) ru[i] = u;
  }
  if (j.codes) {
    const int64_t pitch = (int64_t)ncb * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r0 + i >= j.rows) continue;
      const uint32_t s = fp8_scale_byte(ru[i]);
      const float inv = fp8_inverse(s);
      float v[8];
      unpack(raw[i], v);
      *reinterpret_cast<u32x2_t*>(j.codes + (r0 + i) * pitch + c0) =
          u32x2_t{fp8_pack4(v[0], v[1], v[2], v[3], inv), fp8_pack4(v[4], v[5], v[6], v[7], inv)};
      if (cg == 0) {
        uint8_t* d = j.scales + ((int64_t)(cb >> 2) * j.rows + r0 + i) * 4;
        d[cb & 3] = (uint8_t)s;
        if (cb == ncb - 1)  // the rest of the last group of four
          for (int b = (cb & 3) + 1; b < 4; ++b) d[b] = (uint8_t)kFp8PadScale;
      }
    }
  }
  if (!j.codes_t) return;
  const int nrb = (int)((j.rows + 127) / 128);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack(raw[i], v[i]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t s = fp8_scale_byte(cu[e]);
    const float inv = fp8_inverse(s);
    *reinterpret_cast<uint32_t*>(&turn[(8 * cg + e) * 128 + 4 * (rg ^ 2 * cg)]) =
        fp8_pack4(v[0][e], v[1][e], v[2][e], v[3][e], inv);
    if (rg == 0 && c0 + e < j.cols) {
      uint8_t* d = j.scales_t + ((int64_t)(rb >> 2) * j.cols + c0 + e) * 4;
      d[rb & 3] = (uint8_t)s;
      if (rb == nrb - 1)
        for (int b = (rb & 3) + 1; b < 4; ++b) d[b] = (uint8_t)kFp8PadScale;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = rg + 32 * i;  // 16 lanes write one column's 128 bytes
    const int64_t c = (int64_t)cb * 128 + col;
    if (c < j.cols)
      *reinterpret_cast<u32x2_t*>(j.codes_t + c * ((int64_t)nrb * 128) + (int64_t)rb * 128 + 8 * cg) =
          *reinterpret_cast<const u32x2_t*>(&turn[col * 128 + 8 * (cg ^ (col >> 3))]);
  }
}

__global__ void __launch_bounds__(64 * kTileWaves) k_fp8_tiles(const TileArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t cmax[kTileWaves][128];
  __shared__ float csum[kTileWaves][128];
  __shared__ __attribute__((aligned(16))) uint8_t turn[128 * 128];
  const bool second = (int)blockIdx.x >= a.tiles0;
  const Fp8TileJob& j = a.j[second ? 1 : 0];
  const int tile = (int)blockIdx.x - (second ? a.tiles0 : 0);
  if (j.dtype == ASP_BF16)
    tile_body<uint16_t>(j, tile, cmax, csum, turn);
  else
    tile_body<float>(j, tile, cmax, csum, turn);
}

// One lane for each 8 codes.  An E4M3 value times a power of two is exact in
// float32 and in bf16 (four significant bits) but where it leaves the type's
// range: below it the product rounds once, into the type's subnormals.  Its stores are
// an element each: 4096 x 14336 to bf16 72 us (2.4 TB/s).
template <typename YT>
__global__ void __launch_bounds__(256)
    k_fp8_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                     int64_t rows, int cols, YT* __restrict__ out) {
  const int pitch = (cols + kFp8Block - 1) / kFp8Block * kFp8Block;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = t / (pitch / 8);
  const int c0 = (int)(t % (pitch / 8)) * 8;
  if (row >= rows || c0 >= cols) return;
  const u32x2_t w = *reinterpret_cast<const u32x2_t*>(codes + row * pitch + c0);
  const uint32_t sb = scales[((int64_t)(c0 >> 9) * rows + row) * 4 + ((c0 >> 7) & 3)];
  // 2^(sb - 127) for every byte but the NaN one: 0 stands for 2^-127, a subnormal
  const float s = sb == 255u ? __builtin_nanf("")
                  : sb == 0u ? __builtin_bit_cast(float, 0x00400000u)
                             : __builtin_bit_cast(float, sb << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (c0 + e >= cols) break;
    const uint32_t c = (w[e >> 2] >> (8 * (e & 3))) & 255u;
    const float m = (c & 0x7Fu) == 0x7Fu ? __builtin_nanf("") : e4m3_decode(c & 0x7Fu);
    const float v = (c & 0x80u ? -m : m) * s;
    if constexpr (sizeof(YT) == 2)
      out[row * cols + c0 + e] = bf16_rne(v);
    else
      out[row * cols + c0 + e] = v;
  }
}

int32_t check_quant(const void* in, int32_t dtype, int64_t rows, int64_t cols, int64_t ld) {
  ASP_TRY(check_io_dtype(dtype, "dtype"));
  ASP_TRY(check_fp8_dims(rows, cols, "rows", "cols"));
  if (rows == 0) return ASP_OK;
  return check_matrix(in, dtype, cols, ld, "in");
}

}  // namespace

int32_t fp8_quantize_rows(const void* in, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                          uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const int groups = (int)((fp8_blocks(cols) + 3) / 4);
  const int64_t blocks = (rows * groups + 3) / 4;
  if (blocks > kMaxLanes / 256) return fail(ASP_ERR_SHAPE, "input too large for one launch");
  const dim3 grid((unsigned)blocks);
  uint32_t* sc = reinterpret_cast<uint32_t*>(scales);
  if (dtype == ASP_BF16)
    k_fp8_rows<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(in), rows, (int)cols, ld,
                                               groups, codes, sc);
  else
    k_fp8_rows<float><<<grid, 256, 0, st>>>(static_cast<const float*>(in), rows, (int)cols, ld,
                                            groups, codes, sc);
  return launch_status("fp8 row quantise");
}

int32_t fp8_quantize_tiles(int n, const Fp8TileJob* jobs, hipStream_t st) {
  TileArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    a.j[i] = jobs[i];
    const int64_t t = fp8_blocks(jobs[i].rows) * fp8_blocks(jobs[i].cols);
    total += t;
    if (total > kMaxLanes / (64 * kTileWaves)) return fail(ASP_ERR_SHAPE, "input too large for one launch");
  }
  if (total == 0) return ASP_OK;
  a.tiles0 = (int)(fp8_blocks(jobs[0].rows) * fp8_blocks(jobs[0].cols));
  k_fp8_tiles<<<dim3((unsigned)total), 64 * kTileWaves, 0, st>>>(a);
  return launch_status("fp8 tile quantise");
}

}  // namespace asp

using namespace asp;

extern "C" {

int32_t asp_fp8_sizes(int64_t rows, int64_t cols, size_t* code_bytes, size_t* scale_bytes) {
  clear_error();
  ASP_TRY(check_fp8_dims(rows, cols, "rows", "cols"));
  if (!code_bytes || !scale_bytes) return fail(ASP_ERR_ARG, "null output pointer");
  *code_bytes = fp8_code_bytes(rows, cols);
  *scale_bytes = fp8_scale_bytes(rows, cols);
  return ASP_OK;
}

int32_t asp_fp8_quantize(const void* in, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                         uint8_t* codes, uint8_t* scales, void* stream) {
  clear_error();
  ASP_TRY(check_quant(in, dtype, rows, cols, ld));
  if (rows == 0) return ASP_OK;
  ASP_TRY(check_ptr(codes, "codes", true));
  ASP_TRY(check_ptr(scales, "scales", true));
  return fp8_quantize_rows(in, dtype, rows, cols, ld, codes, scales, (hipStream_t)stream);
}

int32_t asp_fp8_quantize_t(const void* in, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                           uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  clear_error();
  ASP_TRY(check_quant(in, dtype, rows, cols, ld));
  if (rows > kMaxK) return fail(ASP_ERR_SHAPE, "rows=%lld above %lld", (long long)rows, (long long)kMaxK);
  if (rows == 0) return ASP_OK;
  ASP_TRY(check_ptr(codes_t, "codes_t", true));
  ASP_TRY(check_ptr(scales_t, "scales_t", true));
  const Fp8TileJob j = {in, rows, cols, ld, nullptr, nullptr, codes_t, scales_t, nullptr, dtype, 0};
  return fp8_quantize_tiles(1, &j, (hipStream_t)stream);
}

int32_t asp_fp8_quantize_weight(const void* w, int32_t dtype, int64_t N, int64_t K, int64_t ld,
                                uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                                uint8_t* scales_t, void* stream) {
  clear_error();
  ASP_TRY(check_io_dtype(dtype, "dtype"));
  ASP_TRY(check_fp8_dims(N, K, "N", "K"));
  if (N < 1 || N > kMaxK)
    return fail(ASP_ERR_SHAPE, "N=%lld outside [1, %lld]", (long long)N, (long long)kMaxK);
  ASP_TRY(check_matrix(w, dtype, K, ld, "w"));
  ASP_TRY(check_ptr(codes, "codes", true));
  ASP_TRY(check_ptr(scales, "scales", true));
  ASP_TRY(check_ptr(codes_t, "codes_t", scales_t != nullptr));
  ASP_TRY(check_ptr(scales_t, "scales_t", codes_t != nullptr));
  const Fp8TileJob j = {w, N, K, ld, codes, scales, codes_t, scales_t, nullptr, dtype, 1};
  return fp8_quantize_tiles(1, &j, (hipStream_t)stream);
}

int32_t asp_fp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                           void* out, int32_t dtype, void* stream) {
  clear_error();
  ASP_TRY(check_io_dtype(dtype, "dtype"));
  ASP_TRY(check_fp8_dims(rows, cols, "rows", "cols"));
  if (rows == 0) return ASP_OK;
  ASP_TRY(check_ptr(codes, "codes", true));
  ASP_TRY(check_ptr(scales, "scales", true));
  ASP_TRY(check_matrix(out, dtype, cols, cols, "out"));
  const int64_t blocks = (rows * (fp8_pitch(cols) / 8) + 255) / 256;
  if (blocks > kMaxLanes / 256) return fail(ASP_ERR_SHAPE, "input too large for one launch");
  const dim3 grid((unsigned)blocks);
  if (dtype == ASP_BF16)
    k_fp8_dequantize<uint16_t><<<grid, 256, 0, (hipStream_t)stream>>>(
        codes, scales, rows, (int)cols, static_cast<uint16_t*>(out));
  else
    k_fp8_dequantize<float><<<grid, 256, 0, (hipStream_t)stream>>>(codes, scales, rows, (int)cols,
                                                                  static_cast<float*>(out));
  return launch_status("fp8 dequantise");
}

}  // extern "C"

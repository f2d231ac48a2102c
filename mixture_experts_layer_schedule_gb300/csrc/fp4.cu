// fp4.cu -- microscaled 4-bit floating point: quantiser and read-back.
//
// A value is an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times the
// scale of its block of consecutive values of a row:
//   MXFP4 (OCP Microscaling v1.0): blocks of 32, E8M0 scale 2^(floor(log2 amax) - 2),
//         code = exponent + 127 (0 for a block whose amax has a zero exponent field);
//   NVFP4: blocks of 16, scale sb = E4M3(amax / (6 ts)), to nearest even and
//         at most 448, times one fp32 tensor scale ts.
// Codes are v / step rounded to nearest even (ties in the code), saturating at
// 6, with step = 2^(code - 127) or fl32(sb ts); a zero step gives zero codes. A
// block that holds an infinity or a NaN gets the NaN scale (0xFF, 0x7F) and
// zero codes, so whatever is computed from it is NaN.
//
// Codes are packed two to a byte, the even element in the low nibble. Scales
// are stored the way the tensor-memory copy (tcgen05.cp 32x128b, warpx4)
// places them for the product: 512-byte chunks of 128 rows x 4 scales, chunk
// (row block rb, scale quad kc) at (rb * KC + kc) * 512 with KC quads per row,
// and in it the scale of (row r, j-th of the quad) at byte
// (r % 32) * 16 + (r / 32 % 4) * 4 + j. Chunks are written whole: rows and
// blocks past the matrix get scale 0.
//
// Both kernels stream memory. A warp takes the four rows r, r + 32, r + 64,
// r + 96 of a 128-row block, 256 columns wide: every lane holds 8 consecutive
// values of each row (one 16-byte load), a block's amax is one or two shuffles,
// the codes leave as full 128-byte lines, and the four rows' scales of a quad
// form one 16-byte store. 16384 x 4096 bf16 values take 28.9 us (MXFP4: 134 MB
// in, 36 MB out, 5.9 TB/s) or 31.1 us (NVFP4, 5.5 TB/s: the arithmetic of its
// scales shows), and 26 us back (6.6 TB/s).
#include <algorithm>

#include "dense_common.cuh"
#include "fp4.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQCols = 256;  // columns per warp step

__device__ __forceinline__ void e2m1x8_to_f32(uint32_t codes, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(h[i], true);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

template <int ELT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[8]) {
  if constexpr (ELT == MOE_ELT_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    constexpr bool h = ELT == MOE_ELT_FP16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(pack2(f[0], f[1], h), pack2(f[2], f[3], h), pack2(f[4], f[5], h), pack2(f[6], f[7], h));
  }
}

// The four rows of a warp: r0 + 32 i; its columns: 256 from c0, 8 per lane.
struct WarpPlace {
  int64_t row0;   // first of the four rows
  int64_t col;    // this lane's first column
  int64_t chunk;  // byte offset of this lane group's 16-byte scale line
};

template <bool NV>
__device__ __forceinline__ WarpPlace place(int64_t x, int kc_count) {
  constexpr int kLanes = NV ? 8 : 16;  // lanes per scale quad
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rb = blockIdx.y >> 2;
  const int r = static_cast<int>(blockIdx.y & 3) * 8 + warp;  // row in 0..31 of the block
  const int64_t kc = x * (kQCols / (8 * kLanes)) + lane / kLanes;
  WarpPlace p;
  p.row0 = rb * 128 + r;
  p.col = x * kQCols + lane * 8;
  p.chunk = (rb * kc_count + kc) * 512 + r * 16;
  return p;
}

template <int ELT, bool NV>
__global__ void __launch_bounds__(kQThreads) fp4_quantize_kernel(const void* src, int64_t ld, int64_t rows,
                                                                 int64_t cols, int kc_count, NvScale sc, uint8_t* q,
                                                                 uint8_t* s) {
  constexpr int kLanes = NV ? 8 : 16, kBlock = NV ? 2 : 4;  // lanes per quad, per block
  constexpr int kWidth = 8 * kLanes;                        // columns of a quad
  __shared__ float2 tab[NV ? 128 : 1];
  if constexpr (NV) {
    if (threadIdx.x < 128) tab[threadIdx.x] = nv_step_entry(threadIdx.x, sc.ts);
    __syncthreads();
  }
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const WarpPlace p = place<NV>(blockIdx.x, kc_count);
  constexpr int kElt = ELT == MOE_ELT_FP32 ? 4 : 2;
  // Rows of this warp inside the matrix, and everything that advances by a fixed
  // amount per step.
  const int n_rows = static_cast<int>(min(static_cast<int64_t>(4), max(static_cast<int64_t>(0), (rows - p.row0 + 31) / 32)));
  const char* sp = static_cast<const char*>(src) + (p.row0 * ld + p.col) * kElt;
  uint8_t* qp = q + p.row0 * (cols / 2) + p.col / 2;
  uint8_t* scp = s + p.chunk;
  const int64_t s_row = 32 * ld * kElt, q_row = 16 * cols;
  const int n_cols = static_cast<int>(cols), jump = static_cast<int>(gridDim.x) * kQCols;
  const int end = kc_count * kWidth;  // columns with a scale
  Raw8<ELT> next[4];
  auto fetch = [&](int col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (col < n_cols && i < n_rows) {  // cols is a multiple of 32: whole blocks
        next[i] = load_raw8<ELT>(sp + i * s_row, 0);
      } else {
#pragma unroll
        for (uint32_t& w : next[i].w) w = 0u;
      }
    }
  };
  int col = static_cast<int>(p.col);
  fetch(col);
  for (int c0 = static_cast<int>(blockIdx.x) * kQCols; c0 < end; c0 += jump) {
    Raw8<ELT> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = next[i];
    sp += static_cast<int64_t>(jump) * kElt;
    if (c0 + jump < end) fetch(col + jump);  // the next step's loads fly under this one
    uint32_t line[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t codes;
      const uint32_t scale = quantize8<ELT, NV>(raw[i], sc, tab, codes);
      if (col < n_cols && i < n_rows) *reinterpret_cast<uint32_t*>(qp + i * q_row) = codes;
      line[i] = quad_word<kBlock>(scale, lane);
    }
    if (col < end && lane % kLanes == 0)
      *reinterpret_cast<uint4*>(scp) = make_uint4(line[0], line[1], line[2], line[3]);
    col += jump;
    qp += jump / 2;
    scp += static_cast<int64_t>(jump / kWidth) * 512;
  }
}

template <int ELT, bool NV>
__global__ void __launch_bounds__(kQThreads) fp4_dequantize_kernel(const uint8_t* q, const uint8_t* s, int64_t rows,
                                                                   int64_t cols, int kc_count, float ts, void* dst,
                                                                   int64_t ld) {
  constexpr int kBlock = NV ? 2 : 4;
  const WarpPlace p = place<NV>(blockIdx.x, kc_count);
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  if (p.col >= cols) return;
  const uint4 lv = *reinterpret_cast<const uint4*>(s + p.chunk);
  const uint32_t line[4] = {lv.x, lv.y, lv.z, lv.w};
  uint32_t codes[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes[i] = p.row0 + 32 * i < rows
                   ? *reinterpret_cast<const uint32_t*>(q + (p.row0 + 32 * i) * (cols / 2) + p.col / 2)
                   : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.row0 + 32 * i >= rows) break;
    const uint32_t sb = (line[i] >> (8 * ((lane / kBlock) & 3))) & 0xffu;
    float step;
    if constexpr (NV) step = e4m3_to_f32(sb) * ts;
    else if (sb == kNanE8m0) step = __uint_as_float(0x7fc00000u);
    else step = __uint_as_float(sb == 0 ? 0x00400000u : sb << 23);  // 2^(sb - 127)
    float f[8];
    e2m1x8_to_f32(codes[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= step;
    store8<ELT>(dst, (p.row0 + 32 * i) * ld + p.col, f);
  }
}

// Row pitch and alignment of a matrix of `elt` values: 16-byte rows.
bool matrix_ok(const void* p, int64_t ld, int64_t cols, int32_t elt) {
  return aligned(p, 16) && ld >= cols && ld % (elt == MOE_ELT_FP32 ? 4 : 8) == 0;
}

}  // namespace

int fp4_quads(int32_t format, int64_t cols) {
  const int64_t w = format == FP4_NV ? 64 : 128;
  return static_cast<int>((cols + w - 1) / w);
}

moe_status fp4_check(int32_t format, int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
  if (format != FP4_MX && format != FP4_NV) return MOE_ERR_UNSUPPORTED;
  // whole blocks and 16-byte code rows; row blocks fit the grid
  if (cols % 32 != 0 || cols > (1 << 24) || rows > 16383LL * 128) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool fp4_scale_ok(int32_t format, float ts) {
  if (format == FP4_MX) return ts == 1.0f;
  return ts >= 0x1p-60f && ts <= 0x1p60f;  // false for a NaN
}

moe_status launch_fp4_quantize(const void* src, int32_t elt, int64_t rows, int64_t cols, int64_t ld,
                               int32_t format, float ts, uint8_t* q, uint8_t* s, cudaStream_t st) {
  const int kc = fp4_quads(format, cols);
  const int64_t steps = (static_cast<int64_t>(kc) * (format == FP4_NV ? 64 : 128) + kQCols - 1) / kQCols;
  const int64_t row_groups = (rows + 127) / 128 * 4;
  // Up to about eight CTAs per SM; beyond, a CTA walks several column steps.
  const int64_t wide = std::max<int64_t>(1, (8LL * device_sms() + row_groups - 1) / row_groups);
  const dim3 grid(static_cast<unsigned>(std::min(steps, wide)), static_cast<unsigned>(row_groups));
  const NvScale sc = nv_scale(ts);
  const LaunchCfg c(grid, kQThreads, 0, 1, true, st);
  moe_status status = MOE_OK;
  auto go = [&](auto kernel) { status = launch_kernel(c, kernel, src, ld, rows, cols, kc, sc, q, s); };
  const bool nv = format == FP4_NV;
  if (elt == MOE_ELT_BF16) nv ? go(fp4_quantize_kernel<MOE_ELT_BF16, true>) : go(fp4_quantize_kernel<MOE_ELT_BF16, false>);
  else if (elt == MOE_ELT_FP16) nv ? go(fp4_quantize_kernel<MOE_ELT_FP16, true>) : go(fp4_quantize_kernel<MOE_ELT_FP16, false>);
  else nv ? go(fp4_quantize_kernel<MOE_ELT_FP32, true>) : go(fp4_quantize_kernel<MOE_ELT_FP32, false>);
  return status;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status fp4_scale_bytes(int32_t format, int64_t rows, int64_t cols, size_t* bytes) {
  const moe_status st = fp4_check(format, rows, cols);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = static_cast<size_t>((rows + 127) / 128) * fp4_quads(format, cols) * 512;
  return MOE_OK;
}

moe_status fp4_quantize(const void* src, int32_t elt, int64_t rows, int64_t cols, int64_t ld, int32_t format,
                        float tensor_scale, uint8_t* q, uint8_t* s, void* stream) {
  const moe_status st = fp4_check(format, rows, cols);
  if (st != MOE_OK) return st;
  if (elt < MOE_ELT_BF16 || elt > MOE_ELT_FP32) return MOE_ERR_UNSUPPORTED;
  if (!fp4_scale_ok(format, tensor_scale)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!matrix_ok(src, ld, cols, elt) || !aligned(q, 16) || !aligned(s, 16)) return MOE_ERR_INVALID_ARG;
  return launch_fp4_quantize(src, elt, rows, cols, ld, format, tensor_scale, q, s,
                             static_cast<cudaStream_t>(stream));
}

moe_status fp4_dequantize(const uint8_t* q, const uint8_t* s, int32_t format, float tensor_scale, int64_t rows,
                          int64_t cols, void* dst, int32_t elt, int64_t ld, void* stream) {
  const moe_status st = fp4_check(format, rows, cols);
  if (st != MOE_OK) return st;
  if (elt < MOE_ELT_BF16 || elt > MOE_ELT_FP32) return MOE_ERR_UNSUPPORTED;
  if (!fp4_scale_ok(format, tensor_scale)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!matrix_ok(dst, ld, cols, elt) || !aligned(q, 16) || !aligned(s, 16)) return MOE_ERR_INVALID_ARG;
  const int kc = fp4_quads(format, cols);
  const dim3 grid(static_cast<unsigned>((cols + kQCols - 1) / kQCols), static_cast<unsigned>((rows + 127) / 128 * 4));
  const LaunchCfg c(grid, kQThreads, 0, 1, true, static_cast<cudaStream_t>(stream));
  moe_status status = MOE_OK;
  auto go = [&](auto kernel) { status = launch_kernel(c, kernel, q, s, rows, cols, kc, tensor_scale, dst, ld); };
  const bool nv = format == FP4_NV;
  if (elt == MOE_ELT_BF16) nv ? go(fp4_dequantize_kernel<MOE_ELT_BF16, true>) : go(fp4_dequantize_kernel<MOE_ELT_BF16, false>);
  else if (elt == MOE_ELT_FP16) nv ? go(fp4_dequantize_kernel<MOE_ELT_FP16, true>) : go(fp4_dequantize_kernel<MOE_ELT_FP16, false>);
  else nv ? go(fp4_dequantize_kernel<MOE_ELT_FP32, true>) : go(fp4_dequantize_kernel<MOE_ELT_FP32, false>);
  return status;
}

}  // extern "C"

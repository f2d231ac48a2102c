// fp4.cuh -- what the 4-bit quantiser (fp4.cu) and products (fp4_gemm.cu) share:
// the quantisation of eight consecutive values by one lane.
#pragma once
#include "dense_common.cuh"

namespace moe {

constexpr uint32_t kNanE4m3 = 0x7f, kNanE8m0 = 0xff;

// Scale quads (chunks of 4 scales) of a row of `cols` values.
int fp4_quads(int32_t format, int64_t cols);
// Sizes the formats support.
moe_status fp4_check(int32_t format, int64_t rows, int64_t cols);
// Whether `ts` is a tensor scale of the format (MXFP4 has none: 1).
bool fp4_scale_ok(int32_t format, float ts);

moe_status launch_fp4_quantize(const void* src, int32_t elt, int64_t rows, int64_t cols, int64_t ld,
                               int32_t format, float ts, uint8_t* q, uint8_t* s, cudaStream_t st);

// NVFP4 constants of a tensor scale ts: 6 ts and its correctly rounded
// reciprocal.
struct NvScale {
  float ts, ts6, r6;
};
inline NvScale nv_scale(float ts) {
  const float ts6 = static_cast<float>(6.0 * static_cast<double>(ts));
  return NvScale{ts, ts6, static_cast<float>(1.0 / static_cast<double>(ts6))};
}

// Eight consecutive values of a row, as loaded. With ordinary loads: a kernel
// here is resident while its predecessor may still write them (it waits before
// it reads), and the read-only path (ld.global.nc, which `const __restrict__`
// invites too) is for memory that nothing writes during the kernel's lifetime;
// such loads may be moved above the wait.
template <int ELT>
struct Raw8 {
  uint32_t w[ELT == MOE_ELT_FP32 ? 8 : 4];
};

template <int ELT>
__device__ __forceinline__ Raw8<ELT> load_raw8(const void* base, int64_t at) {
  Raw8<ELT> r;
  if constexpr (ELT == MOE_ELT_FP32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + at);
    const uint4 a = p[0], b = p[1];
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  }
  return r;
}

template <int ELT>
__device__ __forceinline__ void raw8_values(const Raw8<ELT>& r, float (&f)[8]) {
  if constexpr (ELT == MOE_ELT_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2(r.w[i], ELT == MOE_ELT_FP16);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}

// Largest magnitude of a block held by LANES neighbouring lanes, as fp32 bits; a
// non-finite value gives at least the bits of infinity. Magnitudes compare as
// integers, two 16-bit ones at a time.
template <int ELT, int LANES>
__device__ __forceinline__ uint32_t block_top(const Raw8<ELT>& r) {
  uint32_t m;
  if constexpr (ELT == MOE_ELT_FP32) {
    m = r.w[0] & 0x7fffffffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, r.w[i] & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  } else {
    m = r.w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
#pragma unroll
    for (int o = 1; o < LANES; o *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m >> 16, m & 0xffffu);
    if constexpr (ELT == MOE_ELT_BF16) return m << 16;
    return m >= 0x7c00u ? 0x7f800000u : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
  }
}

// Eight fp32 values to eight E2M1 codes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"  // first source: upper nibble
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code)));
  return unpack2(h2, true).x;
}

// Entry `code` of the NVFP4 step table: fl32(scale ts) and its correctly rounded
// reciprocal (0 for a zero step). Threads 0 to 127 of a CTA fill tab[128].
__device__ __forceinline__ float2 nv_step_entry(uint32_t code, float ts) {
  const float step = code < kNanE4m3 ? e4m3_to_f32(code) * ts : 0.0f;
  return make_float2(step, step > 0.0f ? __frcp_rn(step) : 0.0f);
}

// The block's stored scale and this lane's eight codes.
//
// Every quotient must be the correctly rounded one, or a value that is an exact
// tie between two codes would round to either side. MXFP4 steps are powers of
// two and the product with the inverse is exact. For NVFP4 a product with the
// correctly rounded reciprocal r of the divisor d and one residual correction
// give it (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): q = v r, then q - r (q d - v); in this form a
// zero keeps its sign. All lanes of the warp take part.
template <int ELT, bool NV>
__device__ __forceinline__ uint32_t quantize8(const Raw8<ELT>& raw, const NvScale& sc, const float2* tab,
                                              uint32_t& codes) {
  const uint32_t top = block_top<ELT, NV ? 2 : 4>(raw);
  const bool bad = top >= 0x7f800000u;  // what a non-finite block computes below is dropped
  float f[8];
  raw8_values<ELT>(raw, f);
  if constexpr (NV) {
    const float amax = __uint_as_float(top);
    const float a = fminf(amax, 500.0f * sc.ts6);  // past the largest scale: keeps the quotient finite
    const float s = a * sc.r6;
    const uint32_t sb = e4m3x2(fmaf(-sc.r6, fmaf(s, sc.ts6, -a), s), 0.0f) & 0x7fu;
    const float2 st = tab[sb];
    const float lim = 8.0f * st.x;
    if (__any_sync(0xffffffffu, amax > lim)) {  // a saturated scale or a zero step: keep the quotients finite
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -lim), lim);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = f[i] * st.y;
      f[i] = fmaf(-st.y, fmaf(q, st.x, -f[i]), q);
    }
    codes = st.x > 0.0f && !bad ? e2m1x8(f) : 0u;
    return bad ? kNanE4m3 : sb;
  } else {
    const int biased = static_cast<int>(top >> 23);
    const int code = max(biased - 2, 0);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - code) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv;
    // a subnormal amax too: its products with 2^127 are exact
    codes = top > 0 && !bad ? e2m1x8(f) : 0u;
    return bad ? kNanE8m0 : static_cast<uint32_t>(code);
  }
}

// The scale bytes of a quad (four neighbouring blocks of LANES lanes each) as
// one word, in every lane of the group.
template <int LANES>
__device__ __forceinline__ uint32_t quad_word(uint32_t scale, int lane) {
  uint32_t w = scale << (8 * ((lane / LANES) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, LANES);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * LANES);
  return w;
}

}  // namespace moe

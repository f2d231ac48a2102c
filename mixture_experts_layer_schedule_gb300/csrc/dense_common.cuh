// dense_common.cuh -- pieces shared by the kernels of the dense gated
// feed-forward block (ffn.cu) and of the 4-bit formats (fp4.cu, fp4_gemm.cu):
// the 16-bit element types, the gated activation and its derivative, the tile
// order, tensor maps of pitched matrices, and launches that may start before
// the previous kernel of the stream has ended.
#pragma once
#include <cuda_fp16.h>

#include <algorithm>

#include "context_cache.h"
#include "moe_common.cuh"
#include "moe_internal.h"
#include "tma_map.h"

namespace moe {

// ---- 16-bit element types -----------------------------------------------------

// Two fp32 values to a word of two 16-bit elements, round to nearest even.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float2 unpack2(uint32_t v, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(bf16lo(v), bf16hi(v));
}

// tcgen05 kind::f16 instruction descriptor: idesc_bf16 with the element format
// of A (bits 7-9) and B (bits 10-12) set to 0 for fp16.
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool a_mn, bool b_mn, bool fp16) {
  const uint32_t d = idesc_bf16(M, N, a_mn, b_mn);
  return fp16 ? d & ~((1u << 7) | (1u << 10)) : d;
}

// The halves of a 128-byte-swizzle operand descriptor (sdesc_sw128 with 1024
// bytes between 8-row groups): the low word carries the address, so a stage's
// operands and K steps differ by a 32-bit addition. One thread issues every MMA;
// building each descriptor anew cost it about 160 cycles an MMA, more than the
// 128 that the tensor core takes for one.
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kSdescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t sdesc_of(uint32_t lo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kSdescHi));
  return d;
}

// The warps that issue copies and MMAs run their loops with all lanes, and one
// elected lane issues: these instructions take uniform registers, which the
// compiler can fill ahead of time only in code that the whole warp runs. Under
// `if (lane == 0)` each operand was moved over for each instruction (350 cycles
// for the four MMAs and the commit of a k-block, now 90 to 110; 280 a copy).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// This warp's index, known to the compiler to be the same in all lanes.
__device__ __forceinline__ int warp_index() { return __shfl_sync(~0u, static_cast<int>(threadIdx.x >> 5), 0); }

// The barrier before a cluster's CTAs leave: they wait for each other, but pass
// no data, so this thread's stores to global memory need not have arrived (a
// releasing arrive waits for them, most of a microsecond at the end of every
// launch). Reads of another CTA's partial sums are over when a thread arrives, by
// data dependence and not by the memory model: every value read goes into the
// operand of a store that the thread issues before the arrive (the asm's memory
// clobber keeps that order), and a store cannot issue before its operand is there.
// Code that reads another CTA's memory for anything else needs the releasing form.
__device__ __forceinline__ void cluster_leave() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// mbar_wait by a whole warp, with one answer: what follows is often an instruction
// of the whole warp (tensor-memory loads and stores, shuffles), also when a wait
// ends with the abort flag.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
  return __all_sync(~0u, mbar_wait(bar, parity, abort, err));
}

// ---- gated activation ----------------------------------------------------------

// h(g) = g * sigma(p(g)): silu for p = g, and the tanh form of gelu for
// p = 2 sqrt(2/pi) (g + 0.044715 g^3), since 1/2 (1 + tanh z) = sigma(2 z).
//
// sigma is 1 / (1 + 2^(-p log2 e)) with the approximate exponential and
// reciprocal instructions (PTX: relative error 2^-22 and one ulp) in their
// flush-to-zero forms, so the whole error stays near 2^-21 (1 + |p|), far below
// the 16-bit rounding of every output. The general forms (__expf, __fdividef)
// guard subnormal operands that cannot matter here (a sigma under 2^-126, or
// one indistinguishable from 1) with more instructions than the arithmetic has.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu1 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.044715f;

__device__ __forceinline__ float gate_sigma_exp2(float minus_p_log2e) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(minus_p_log2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
  return s;
}

__device__ __forceinline__ float gate_act(float g, bool gelu) {
  const float w = gelu ? fmaf(-kLog2e * kGelu1 * kGelu3 * g, g, -kLog2e * kGelu1) : -kLog2e;
  return g * gate_sigma_exp2(g * w);
}

// h and dh/dg = s + h (1 - s) p'. In p', g^2 is taken up to 1024: beyond, h (1 - s)
// is zero in fp32 and p' must only stay finite.
__device__ __forceinline__ void gate_act_grad(float g, bool gelu, float& h, float& dh) {
  if (gelu) {
    const float g2 = g * g;
    const float s = gate_sigma_exp2(g * fmaf(-kLog2e * kGelu1 * kGelu3, g2, -kLog2e * kGelu1));
    h = g * s;
    dh = fmaf(fmaf(-h, s, h), fmaf(3.0f * kGelu1 * kGelu3, fminf(g2, 1024.0f), kGelu1), s);
  } else {
    const float s = gate_sigma_exp2(-kLog2e * g);
    h = g * s;
    dh = fmaf(-h, s, h) + s;
  }
}

// ---- tile order ------------------------------------------------------------------

// Tile t of an m_tiles x n_tiles grid, in bands of 8 M tiles with M fastest, so
// that the tiles in flight at one time form a compact block that shares its
// operand panels through L2.
__device__ __forceinline__ void band_tile(int64_t t, int m_tiles, int n_tiles, int& mt, int& nt) {
  constexpr int kBand = 8;
  const int64_t per = static_cast<int64_t>(kBand) * n_tiles;
  const int b = static_cast<int>(t / per);
  const int r = static_cast<int>(t - b * per);
  const int rows = min(kBand, m_tiles - b * kBand);
  mt = b * kBand + r % rows;
  nt = r / rows;
}

// ---- launch overlap ----------------------------------------------------------------
// Every kernel of these files is launched with permission to become resident
// while the previous kernel of the stream still runs, so that its set-up (and,
// inside one call, its weight loads) hides there. The order is always: wait,
// then let the next one in. So when a kernel starts, everything before its
// predecessor has ended; only the predecessor itself may still run.

// Wait until the previous kernel has ended and its writes are visible. Every
// read of data that it may have written, and every write, comes after.
__device__ __forceinline__ void grid_dep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// Let a dependent launch with the overlap attribute become resident.
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ---- partial sums of a cluster ---------------------------------------------------

// Threads of a split kernel: producer, MMA issuer, and eight warps that move the
// partial sums (two per accumulator lane quadrant).
constexpr int kSplitThreads = 320;

// Accumulator columns [0, cols) to part[column][128] in shared memory (row =
// accumulator lane); cols a multiple of 16. Warps 2 to 9 share the work.
__device__ __forceinline__ void park_partials(uint32_t tmem, int cols, int warp, int lane, float* part) {
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  float* p = part + quad * 32 + lane;
  const int mid = (cols / 16 + 1) / 2 * 16;  // half 0: [0, mid), half 1: [mid, cols)
  const int c1 = half ? cols : mid;
  int c = half ? mid : 0;
  for (; c + 64 <= c1; c += 64) {
    uint32_t r[2][32];
    tmem_ld32(taddr + c, r[0]);
    tmem_ld32(taddr + c + 32, r[1]);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 64; ++i) p[(c + i) * 128] = __uint_as_float(r[i / 32][i % 32]);
  }
  for (; c + 32 <= c1; c += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) p[(c + i) * 128] = __uint_as_float(r[i]);
  }
  if (c < c1) {
    uint32_t r[16];
    tmem_ld16(taddr + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) p[(c + i) * 128] = __uint_as_float(r[i]);
  }
}

// Four neighbouring features' partial sums of the cluster's S CTAs (`off` past
// their addresses), all loads in flight at once, added in rank order. The lanes
// of a warp read neighbouring 16 bytes: with gaps between them the reads from
// other SMs, which bound this step, took up to twice as long.
template <int S>
__device__ __forceinline__ float4 cluster_sum4(const uint32_t (&base)[S], uint32_t off) {
  float4 v[S];
#pragma unroll
  for (int r = 0; r < S; ++r) {
    if constexpr (S == 1)  // this CTA alone
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                   : "r"(base[r] + off));
    else
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                   : "r"(base[r] + off));
  }
  float4 s = v[0];
#pragma unroll
  for (int r = 1; r < S; ++r) {
    s.x += v[r].x;
    s.y += v[r].y;
    s.z += v[r].z;
    s.w += v[r].w;
  }
  return s;
}

// The cluster addresses of `local` in its S CTAs.
template <int S>
__device__ __forceinline__ void cluster_bases(uint32_t local, uint32_t (&base)[S]) {
#pragma unroll
  for (int r = 0; r < S; ++r) {
    if constexpr (S == 1) base[r] = local;
    else asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[r]) : "r"(local), "r"(r));
  }
}

// f(integral constant S) for the cluster's size: one of plan_split's.
template <int S>
struct IntC {
  static constexpr int value = S;
};
// f(gelu, fp16) with both flags as integral constants (gelu only where ACT).
template <bool ACT, class F>
__device__ __forceinline__ void with_flags(bool gelu, bool fp16, F&& f) {
  if (ACT && gelu) {
    if (fp16) f(IntC<ACT>(), IntC<1>());
    else f(IntC<ACT>(), IntC<0>());
  } else {
    if (fp16) f(IntC<0>(), IntC<1>());
    else f(IntC<0>(), IntC<0>());
  }
}

template <class F>
__device__ __forceinline__ void for_splits(int splits, F&& f) {
  switch (splits) {
    case 1: f(IntC<1>()); break;
    case 2: f(IntC<2>()); break;
    case 3: f(IntC<3>()); break;
    case 4: f(IntC<4>()); break;
    default: f(IntC<8>()); break;
  }
}

// The token columns [first, last) of a tile's `valid` that CTA `rank` of the
// cluster finishes.
__device__ __forceinline__ void finish_range(int valid, int rank, int splits, int& first, int& last) {
  const int per = (valid + splits - 1) / splits;
  first = min(valid, rank * per);
  last = min(valid, first + per);
}

__device__ __forceinline__ uint2 pack4(const float4& v, bool fp16) {
  return make_uint2(pack2(v.x, v.y, fp16), pack2(v.z, v.w, fp16));
}

// Arrive on a barrier of the other CTA of a pair. What it announces are tensor
// memory accesses, completed by tcgen05.wait and ordered by the tcgen05 fence,
// so no cluster-wide release of this thread's other writes is asked for (that
// fence holds the warp for about 1000 cycles, measured on a GB300).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t cluster_bar_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar_addr) : "memory");
}

__device__ __forceinline__ bool wait_drain_bar(uint64_t* bar, uint32_t parity, int32_t* err) {
  int no_abort = 0;  // drain waits do not stop at the abort flag
  return mbar_wait(bar, parity, &no_abort, err);
}

// ---- host side -------------------------------------------------------------------

// 2-D view [outer][inner] with `pitch` elements between rows (inner contiguous).
// Box rows of at most 128 bytes with the 128-byte swizzle. Loads outside the
// view read zeros, stores outside it are dropped.
inline bool tma_map_pitched(CUtensorMap* m, const void* base, int64_t inner, int64_t outer,
                            int64_t pitch, int box_inner, int box_outer,
                            CUtensorMapDataType dtype, int elem,
                            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFnT fn = tma_encode_fn();
  if (!fn || inner <= 0 || outer <= 0) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch * elem)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The status of a runtime call. CUDA keeps an error for whoever asks next, which
// would be another call's launch check, so it is taken here.
inline moe_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  (void)cudaGetLastError();
  return MOE_ERR_CUDA;
}

inline bool aligned(const void* p, uintptr_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Whether two pitched 16-bit matrices [rows][cols] share an address range.
inline bool overlap(const void* a, int64_t lda, int64_t cols_a, const void* b, int64_t ldb, int64_t cols_b,
                    int64_t rows) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + 2 * ((rows - 1) * ldb + cols_b) && b0 < a0 + 2 * ((rows - 1) * lda + cols_a);
}

// SMs of the GPU (every GPU of a machine is the same part; asked once).
inline int device_sms() {
  static const int sms = [] {
    int dev = 0, n = 0;
    cuda_status(cudaGetDevice(&dev));
    cuda_status(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    return n > 0 ? n : 148;
  }();
  return sms;
}

// Raises a kernel's dynamic shared-memory limit, which holds in the current
// context only.
template <class K>
bool set_smem(K kernel, int bytes) {
  return cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) == MOE_OK;
}

// Microseconds of a split kernel's parts, fitted to a GB300 over 20 to 24 problem
// sizes (1 to 4096 tokens) with every tile size and cluster size: about 170 to 380
// launches for each kind of product, and 130 with weights from HBM for the dense
// ones. The model is off by 10 to 15% rms. Of the launch shapes of a problem, the
// one that it picks is 2 to 4% slower than the best on average, 15% at worst for the
// dense products (400 tokens, 4096 x 512) and 22% for the 4-bit ones (512 tokens, 1536
// wide, K = 4096). KB: a stage's kilobytes.
struct SplitCost {
  double w_kb;               // KB of weights and scales per k-block
  double alone;              // per k-block, one CTA on an SM (or 0.0083 per KB: 120 GB/s into it)
  double two, two_kb;        // per k-block, two CTAs on an SM: two + two_kb * KB
  double remote;             // per KB of partial sums read from other SMs
  double own;                // per 128 token columns that a CTA finishes
  double cluster, member;    // a cluster at all; each of its CTAs
  double round;              // launch, first loads, last stores
  double quantise;           // per k-block and token that the CTA quantises itself
  int sums;                  // accumulators per token column
};

// Shape of a split kernel's launch: tokens per tile (a multiple of `step`, the
// MMA's N) and CTAs of a cluster that share one tile's K (sizes that pack the
// SMs well, 8 only where the sums are small), for n tokens, w_tiles weight tiles and nkb k-blocks.
struct SplitPlan {
  int nt, splits;
  double us;
};
inline SplitPlan plan_split(int64_t n, int64_t w_tiles, int nkb, const SplitCost& c, int first, int last, int step) {
  const int sms = device_sms();
  SplitPlan best{first, 1, 1e30};
  for (int nt = first; nt <= last && (nt == first || nt - step < n); nt += step) {
    const int64_t tiles = w_tiles * ((n + nt - 1) / nt);
    const bool single = c.sums == 2 && nt > 64;  // tensor memory for one CTA per SM
    const int slots = single ? sms * 9 / 10 : 2 * sms;
    const int used = static_cast<int>(std::min<int64_t>(nt, n));
    const double kilobytes = c.w_kb + 0.128 * nt, qx = c.quantise * used;
    const double alone = std::max(c.alone, 0.0083 * kilobytes) + qx, two = c.two + c.two_kb * kilobytes + qx;
    for (const int s : {1, 2, 3, 4, 8}) {
      const int64_t ctas = tiles * s;
      if (s > nkb || (s == 8 && nt > 64) || (s > 1 && ctas > 2 * slots)) break;
      const double rounds = static_cast<double>((ctas + slots - 1) / slots);
      const int kbs = (nkb + s - 1) / s, mine = (used + s - 1) / s;
      const double kb = !single && ctas > sms ? rounds * two : (single ? rounds * alone : alone);
      const double us = kbs * kb + rounds * (c.round + c.member * s + (s > 1 ? c.cluster : 0.0) +
                                             c.sums * (c.own * mine / 128.0 + c.remote * (s - 1) * mine * 0.512));
      if (us < best.us) best = SplitPlan{nt, s, us};
    }
  }
  return best;
}

// Microseconds of a pair kernel's product: `start` for launch, first loads and
// last stores, `wave` and 0.28 per k-block (512 cycles of MMAs, the same for 64
// 16-bit values or 256 4-bit ones) for each wave of 256 x 256 tiles.
inline double pair_time(int64_t tiles, int nkb, double start, double wave) {
  const int64_t pairs = device_sms() / 2;
  return start + (wave + 0.28 * nkb) * static_cast<double>((tiles + pairs - 1) / pairs);
}

// Launch configuration with a cluster size and, with `overlap`, permission to
// become resident while the previous kernel of the stream still runs.
struct LaunchCfg {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  LaunchCfg(dim3 grid, int threads, int smem, int cluster, bool overlap, cudaStream_t s) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    int n = 0;
    if (cluster > 1) {
      at[n].id = cudaLaunchAttributeClusterDimension;
      at[n].val.clusterDim.x = cluster;
      at[n].val.clusterDim.y = 1;
      at[n].val.clusterDim.z = 1;
      ++n;
    }
    if (overlap) {
      at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[n].val.programmaticStreamSerializationAllowed = 1;
      ++n;
    }
    cfg.attrs = at;
    cfg.numAttrs = n;
  }
  LaunchCfg(const LaunchCfg&) = delete;
};

// Launches a kernel and counts it.
template <class K, class... A>
moe_status launch_kernel(const LaunchCfg& c, K kernel, const A&... args) {
  const moe_status st = cuda_status(cudaLaunchKernelEx(&c.cfg, kernel, args...));
  if (st == MOE_OK) note_launch();
  return st;
}

}  // namespace moe

// fp4_gemm.cu -- products with 4-bit weights on the block-scaled tensor cores.
//
//   linear  Y = dq(q(X)) dq(W)^T
//   gated   A = h(dq(q(X)) dq(Wg)^T) * (dq(q(X)) dq(Wu)^T)      h = silu or gelu
//
// X (bf16 or fp16) is quantised along K in the call (fp4.cu, tensor scale
// given), the weights were quantised once. tcgen05.mma multiplies the E2M1
// codes with the block scales (kind::mxf4, one E8M0 scale per 32 values, or
// kind::mxf4nvf4, one E4M3 scale per 16) and sums in fp32; the tensor scales
// multiply the sum, and the result is rounded once to 16 bits.
//
// A k-block is 256 values: 128 bytes of codes per row, moved by TMA with the
// 128-byte swizzle, and per 128 rows four (NVFP4) or two (MXFP4) scale chunks
// of 512 bytes, which go into tensor memory as 32 lanes (one per row of a
// quarter) replicated to the four lane quadrants. Every ring stage owns its
// scale columns, so a copy never meets a product that still reads.
//
//  * fp4_pair_kernel: SM pairs, 256 x 256 tiles with the tokens on M. The
//    accumulator takes 256 columns and the scales of five stages 240, so there
//    is one accumulator: the epilogue warps move it into registers at once and
//    release it before they store. 16384 x 4096, K = 1536 takes 47 us after a
//    quantiser of 10 (MXFP4, 4.4 PFLOP/s), gated 76 us (5.4 PFLOP/s). Of a tile's
//    5100 to 5400 cycles the MMAs take 3070; 1400 pass from its last product to
//    the next tile's first (accumulator to registers), and 600 waiting for the
//    ring to refill: an SM takes in about 47 bytes a cycle, and a k-block is 35
//    (MXFP4) or 38 KB. Measured and not kept: token rows resident over a row of
//    weight tiles (K <= 1536: 57.1 against 57.7 us, gated 84 against 86), sixteen
//    epilogue warps in the linear kernel (63.6 us), output by plain stores
//    (59.8 us).
//  * fp4_split_kernel: weight rows on M, 16 to 128 tokens on N, K split over
//    the CTAs of a cluster (see dense_split_kernel in ffn.cu). Tiles of up to 32
//    tokens quantise X themselves; for tiles of 64 or 128 a quantiser runs first, and
//    the weight tiles and scales are fetched while it does. The plan takes the former
//    for few tokens (up to 32 at 4096 x 1536, up to 10 at 4096 x 7168) and for more
//    where the weights are small. Bound by the latency of one launch: one token
//    through 4096 x 1536 (3.5 MB) in 3.2 us, gated 1536, K = 4096 (7.1 MB) in
//    4.1 us; 64 tokens through 7168 x 2048 in 6 us.
#include <algorithm>

#include "dense_common.cuh"
#include "fp4.cuh"

namespace moe {
namespace {

constexpr int kQK = 256;                 // values per k-block (128 bytes of codes)
constexpr int kTile = 128 * 128;         // 16 KB: 128 rows of codes
constexpr int kSfTile = 4 * 512;         // scale chunks of 128 rows of a k-block (NVFP4)
constexpr int kSfCols = 16;              // their tensor-memory columns

struct FMaps {
  CUtensorMap a, b0, b1;     // codes: tokens, weights (gate), up weights
  CUtensorMap sa, sb0, sb1;  // scale chunks of the same
  CUtensorMap o;             // output (fp4_pair_kernel)
};

struct FArgs {
  int32_t* err;
  int64_t tiles, rows;       // tiles of the launch; tokens
  int m_tiles, n_tiles;
  int nkb;                   // k-blocks
  int cols;                  // output features
  float alpha0, alpha1;      // product of the tensor scales (gate / up)
  int fp16, gelu;
  void* out;                 // fp4_split_kernel
  int64_t ldo;
  int splits;
  int nt;                    // tokens loaded per tile (multiple of 16)
  int t_tiles;               // token tiles
  const void* x;             // fp4_split_kernel that quantises X itself
  int64_t ldx;
  int k;
  NvScale xsc;
};

// Tensor map of scale chunks as [row block][quad][128 words].
bool sf_map(CUtensorMap* m, const uint8_t* s, int quads, int64_t rows, int box_quads) {
  EncodeTiledFnT fn = tma_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(quads), static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[2] = {512, static_cast<cuuint64_t>(quads) * 512};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_quads), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t*>(s), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool code_map(CUtensorMap* m, const uint8_t* q, int64_t k, int64_t rows, int box_rows) {
  return tma_map_pitched(m, q, k / 2, rows, k / 2, 128, box_rows, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1);
}

// ---- PTX used only here ---------------------------------------------------------

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, uint64_t* bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Descriptor of an unswizzled scale chunk: 32 rows of 16 bytes, 8-row groups
// 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sf(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;  // descriptor version for tcgen05
  return d;
}

// One scale chunk into four tensor-memory columns.
__device__ __forceinline__ void tmem_cp_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Instruction descriptor, kind::mxf4 / kind::mxf4nvf4: E2M1 A (bits 7-9) and B
// (bits 10-11), both K-major, K = 64; scale type E8M0 (bit 23) or E4M3; first
// scale byte of the 32-bit column for A (bits 29-30) and B (bits 4-5).
template <bool NV>
__host__ __device__ constexpr uint32_t idesc_f4(int M, int N, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (NV ? 0u : 1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24) | (id << 29);
}

#define FP4_MMA(GROUP, KIND, VEC)                                                          \
  asm volatile(                                                                            \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                     \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC        \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                   \
      "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                           \
      : "memory")

template <bool NV, bool PAIR>
__device__ __forceinline__ void umma_f4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t acc) {
  if constexpr (NV && PAIR) FP4_MMA("2", "mxf4nvf4", "4X");
  else if constexpr (NV) FP4_MMA("1", "mxf4nvf4", "4X");
  else if constexpr (PAIR) FP4_MMA("2", "mxf4", "2X");
  else FP4_MMA("1", "mxf4", "2X");
}

// Scale chunks of a k-block: NVFP4 one per K = 64 step (all four bytes of a
// column word), MXFP4 one per two steps (two bytes each).
template <bool NV>
struct Sf {
  static constexpr int quads = NV ? 4 : 2;
  static __device__ __forceinline__ int quad(int ks) { return NV ? ks : ks >> 1; }
  static __device__ __forceinline__ uint32_t id(int ks) { return NV ? 0u : 2u * (ks & 1); }
};

// ---------------------------------------------------------------------------
// SM pairs.
//
// The scales do not go through tcgen05.cp here: those copies run in the tensor
// pipe itself, about 47 cycles each (measured on a GB300, MMAs of a 256 x 256
// tile: 512 cycles per k-block alone, 747 with the 6 copies of MXFP4, 1077
// with the 12 of NVFP4). Four scale warps per CTA read the chunks from shared
// memory and write the same columns with tcgen05.st, each warp its own lane
// quadrant: 229 cycles per k-block beside the MMAs, which keep their 512.
constexpr int kFStages = 5;
constexpr int kFStageBytes = 2 * kTile;           // this CTA's A rows and its half of B
constexpr int kFSfBytes = 3 * kSfTile;            // scales: A rows, B rows 0-127, B rows 128-255
constexpr uint32_t kFSfCol = 256;                 // scale columns start after the accumulator
constexpr int kOutBytes = 2048;                    // a staged output block: 32 rows x 32 values
static_assert(kFSfCol + kFStages * 3 * kSfCols <= 512, "tensor memory");

// Warps: operand producer, MMA issuer, epilogue, four scale warps, scale
// producer. The gated epilogue takes 16 warps of 32 features (activation in
// registers after the release), the linear one 8 warps of 128 features (sixteen
// warps' stores hold up the ring's loads).
template <bool GATED>
struct F4Pair {
  static constexpr int epi_warps = GATED ? 16 : 8;
  static constexpr int scale_warp = 2 + epi_warps;
  static constexpr int threads = 32 * (scale_warp + 5);
  static constexpr int smem = kFStages * (kFStageBytes + kFSfBytes) + epi_warps * kOutBytes + 1024;
  static_assert(smem <= 227 * 1024, "shared memory");
};

// 16 or 8 registers of each lane to its row of consecutive tensor-memory columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 packed 16-bit values of each lane's row, staged with the 64-byte swizzle,
// to one TMA store at (x, y). Copies and stores share one engine: 4 KB blocks
// held up the ring's loads longer than these (16384 x 4096, K = 1536: 61.9
// against 57.7 us).
__device__ __forceinline__ void store_packed(const CUtensorMap* om, const uint32_t* w, int32_t x, int32_t y,
                                             int lane, uint8_t* buf) {
  if (lane == 0) bulk_wait_read<0>();  // the last store has read the buffer
  __syncwarp();
  const uint32_t row = smem_u32(buf) + lane * 64;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((j ^ ((lane >> 1) & 3)) << 4)), "r"(w[4 * j]),
                 "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                 : "memory");
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(om, buf, x, y);
    bulk_commit();
  }
}

template <bool NV, bool GATED>
__global__ void __launch_bounds__(F4Pair<GATED>::threads, 1)
    fp4_pair_kernel(const __grid_constant__ FMaps maps, const FArgs args) {
  using C = F4Pair<GATED>;
  extern __shared__ uint8_t smem_raw[];
  // full, sf_ready and tempty are used in the even CTA; sf_full, empty and
  // tfull in both
  __shared__ uint64_t full_bar[kFStages], empty_bar[kFStages], sf_full_bar[kFStages], sf_ready_bar[kFStages];
  __shared__ uint64_t tfull_bar, tempty_bar, drain_bar;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_ring = smem + kFStages * kFStageBytes;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank());
  const bool leader = crank == 0;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b0);
    tma_prefetch_desc(&maps.sa);
    tma_prefetch_desc(&maps.sb0);
    for (int s = 0; s < kFStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
      mbar_init(&sf_full_bar[s], 1);
      mbar_init(&sf_ready_bar[s], 8);  // one arrive per scale warp of both CTAs
    }
    mbar_init(&tfull_bar, 1);
    mbar_init(&tempty_bar, 2 * C::epi_warps);  // one arrive per epilogue warp of both CTAs
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abortp = &abort_flag;
  const int64_t first = blockIdx.x / 2, stride = gridDim.x / 2;
  constexpr int kQuads = Sf<NV>::quads;
  constexpr int kSfBytes = kQuads * 512;  // of 128 rows of a k-block
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0 || warp == C::scale_warp + 4) {
    // ---------------- TMA producers (both CTAs): operands, scales ----------------
    const bool codes = warp == 0, one = elect_one();
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
    bool ok = true;
    for (int64_t t = first; t < args.tiles && ok; t += stride) {
      int mt, nt;
      band_tile(t, args.m_tiles, args.n_tiles, mt, nt);
      for (int kb = 0; kb < args.nkb; ++kb) {
        if (!warp_wait(&empty_bar[stage], phase ^ 1u, abortp, args.err)) { ok = false; break; }
        if (codes && one) {
          uint8_t* sA = smem + stage * kFStageBytes;
          const uint32_t bar = cluster_addr(&full_bar[stage], 0);
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kFStageBytes);
          tma_load_2d_pair(sA, &maps.a, bar, kb * 128, mt * 256 + crank * 128);
          // gated: D columns [0, 128) are gate rows (even CTA's B), [128, 256) up rows
          if constexpr (GATED) tma_load_2d_pair(sA + kTile, crank ? &maps.b1 : &maps.b0, bar, kb * 128, nt * 128);
          else tma_load_2d_pair(sA + kTile, &maps.b0, bar, kb * 128, nt * 256 + crank * 128);
        } else if (one) {
          uint8_t* sS = sf_ring + stage * kFSfBytes;
          uint64_t* bar = &sf_full_bar[stage];
          const int quad = kb * kQuads;
          mbar_arrive_expect_tx(bar, 3 * kSfBytes);
          tma_load_3d(sS, &maps.sa, bar, 0, quad, mt * 2 + crank);
          tma_load_3d(sS + kSfTile, &maps.sb0, bar, 0, quad, GATED ? nt : nt * 2);
          tma_load_3d(sS + 2 * kSfTile, GATED ? &maps.sb1 : &maps.sb0, bar, 0, quad, GATED ? nt : nt * 2 + 1);
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kFStages) { stage = 0; phase ^= 1u; }
      }
    }
    // Every copy lands before the CTA ends (the even CTA's full barriers count
    // both CTAs' operand copies).
    for (int s = 0; s < kFStages; ++s)
      if (one && ((issued_mask >> s) & 1u) && (leader || !codes))
        wait_drain_bar(codes ? &full_bar[s] : &sf_full_bar[s], (issued_parity >> s) & 1u, args.err);
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer (even CTA) ----------------
      const bool one = elect_one();
      const uint32_t lo0 = sdesc_lo(smem_u32(smem), 16);
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int64_t t = first; t < args.tiles; t += stride) {
        if (!warp_wait(&tempty_bar, acc_phase ^ 1u, abortp, args.err)) break;
        tc_fence_after();
        for (int kb = 0; kb < args.nkb; ++kb) {
          if (!warp_wait(&full_bar[stage], phase, abortp, args.err) ||
              !warp_wait(&sf_ready_bar[stage], phase, abortp, args.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t lo = lo0 + stage * (kFStageBytes >> 4);
          const uint32_t sf_t = tmem_base + kFSfCol + stage * (3 * kSfCols);
          if (one) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint32_t st = sf_t + Sf<NV>::quad(ks) * 12;
              umma_f4<NV, true>(tmem_base, sdesc_of(lo + 2 * ks), sdesc_of(lo + (kTile >> 4) + 2 * ks),
                                idesc_f4<NV>(256, 256, Sf<NV>::id(ks)), st, st + 4, (kb > 0 || ks > 0) ? 1u : 0u);
            }
            umma_commit_pair_mc(&empty_bar[stage], 0x3);
          }
          __syncwarp();
          if (++stage == kFStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (one) umma_commit_pair_mc(&tfull_bar, 0x3);
        __syncwarp();
        acc_phase ^= 1u;
      }
      if (one) {
        umma_commit_pair(&drain_bar);
        wait_drain_bar(&drain_bar, 0, args.err);
      }
    }
  } else if (warp >= C::scale_warp) {
    // ---------------- scale warps (both CTAs) ----------------
    // Each stage's chunks to its columns, per quad 12: A, B rows 0-127, B rows
    // 128-255. The stage is refilled only after the products that read these
    // columns are done, so its arrival also frees them.
    const uint32_t quadrant = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = first; t < args.tiles && ok; t += stride) {
      for (int kb = 0; kb < args.nkb; ++kb) {
        if (!warp_wait(&sf_full_bar[stage], phase, abortp, args.err)) { ok = false; break; }
        tc_fence_after();
        const uint32_t src = smem_u32(sf_ring + stage * kFSfBytes) + lane * 16;
        const uint32_t dst = tmem_base + quadrant + kFSfCol + stage * (3 * kSfCols);
        uint32_t w[12 * kQuads];
#pragma unroll
        for (int c = 0; c < kQuads; ++c)
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            uint32_t* p = w + c * 12 + j * 4;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
                         : "r"(src + j * kSfTile + c * 512));
          }
        tmem_st16(dst, w);
        if constexpr (NV) {
          tmem_st16(dst + 16, w + 16);
          tmem_st16(dst + 32, w + 32);
        } else {
          tmem_st8(dst + 16, w + 16);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&sf_ready_bar[stage]);
          else mbar_arrive_peer(cluster_addr(&sf_ready_bar[stage], 0));
        }
        if (++stage == kFStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else {
    // ---------------- epilogue warps (both CTAs) ----------------
    const int quad = warp & 3, part = (warp - 2) >> 2;  // lane quadrant, share of the columns
    uint8_t* buf = sf_ring + kFStages * kFSfBytes + (warp - 2) * kOutBytes;
    uint32_t acc_phase = 0;
    for (int64_t t = first; t < args.tiles; t += stride) {
      int mt, nt;
      band_tile(t, args.m_tiles, args.n_tiles, mt, nt);
      if (!warp_wait(&tfull_bar, acc_phase, abortp, args.err)) break;
      tc_fence_after();
      acc_phase ^= 1u;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      const int32_t y = mt * 256 + crank * 128 + quad * 32;
      auto release = [&] {  // the next tile's products may start
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&tempty_bar);
          else mbar_arrive_peer(cluster_addr(&tempty_bar, 0));
        }
      };
      if constexpr (GATED) {
        // gate columns [32 part, +32) and the up columns of the same features
        uint32_t g[32], u[32], w[16];
        tmem_ld32(taddr + 32 * part, g);
        tmem_ld32(taddr + 128 + 32 * part, u);
        tmem_ld_wait();
        release();
        const int32_t x = nt * 128 + 32 * part;
        if (y >= args.rows || x >= args.cols) continue;  // the whole warp
        with_flags<true>(args.gelu != 0, args.fp16 != 0, [&](auto gelu, auto fp16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              e[h] = gate_act(__uint_as_float(g[2 * i + h]) * args.alpha0, decltype(gelu)::value != 0) *
                     (__uint_as_float(u[2 * i + h]) * args.alpha1);
            w[i] = pack2(e[0], e[1], decltype(fp16)::value != 0);
          }
        });
        store_packed(&maps.o, w, x, y, lane, buf);
      } else {
        uint32_t w[2][32];  // columns [128 part, +128), rounded as they are read
        with_flags<false>(false, args.fp16 != 0, [&](auto, auto fp16) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t r[2][32];
            tmem_ld32(taddr + 128 * part + 64 * b, r[0]);
            tmem_ld32(taddr + 128 * part + 64 * b + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              w[b][i] = pack2(__uint_as_float(r[i / 16][2 * (i % 16)]) * args.alpha0,
                              __uint_as_float(r[i / 16][2 * (i % 16) + 1]) * args.alpha0,
                              decltype(fp16)::value != 0);
          }
        });
        release();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int32_t x = nt * 256 + 128 * part + 32 * b;
          if (y < args.rows && x < args.cols) store_packed(&maps.o, w[b / 2] + 16 * (b & 1), x, y, lane, buf);
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncwarp();
  // Both CTAs are through: the even CTA's MMAs into this CTA's tensor memory have
  // retired, and nothing signals a CTA that may leave.
  cluster_leave();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Weight rows on M, NT tokens on N, K split over the CTAs of a cluster. A gated
// tile holds 128 gate rows and the 128 up rows of the same features, each with
// an accumulator of its own.
//
// Tensor memory: CTAs with at most 256 columns keep their shared memory between
// 77 and 113 KB (two per SM, never three), the others above 153 KB (alone on
// their SM among kernels of this library), so no allocation ever waits.
template <bool GATED, int NT>
struct F4Split {
  static constexpr int nw = GATED ? 2 : 1;
  static constexpr int code_bytes = nw * kTile + NT * 128;
  static constexpr int sf_bytes = (nw + 1) * kSfTile;
  static constexpr int stage_bytes = code_bytes + sf_bytes;
  static constexpr int stages = GATED ? (NT == 128 ? 3 : 2) : (NT <= 16 ? 5 : (NT == 32 ? 4 : 3));
  static constexpr int smem = stages * stage_bytes + 1024;
  static constexpr int acc_cols = nw * NT;
  static constexpr int sf_cols = (nw + 1) * kSfCols;
  static constexpr int need = acc_cols + stages * sf_cols;
  static constexpr uint32_t cols = need <= 256 ? 256 : 512;
  static_assert(need <= 512, "tensor memory");
  static_assert(cols == 256 ? (smem >= 77 * 1024 && smem <= 113 * 1024) : (smem >= 153 * 1024 && smem <= 227 * 1024),
                "co-resident CTAs fit tensor memory");
  static_assert(nw * NT * 128 * 4 <= stages * stage_bytes, "the partial sums fit the drained ring");
};

// As split_finish in ffn.cu: a thread keeps its four features and walks the
// tokens that this CTA of the cluster finishes.
template <bool GATED, int NT, int S>
__device__ __forceinline__ void f4_finish(const FArgs& a, uint32_t part, int rank, int tile, int tok0) {
  constexpr int kStep = kSplitThreads / 32;
  int c0, c1;
  finish_range(static_cast<int>(min(static_cast<int64_t>(a.nt), a.rows - tok0)), rank, S, c0, c1);
  const bool fp16 = a.fp16 != 0, gelu = a.gelu != 0;
  const int f = 4 * (static_cast<int>(threadIdx.x) % 32), col = tile * 128 + f;
  int c = c0 + static_cast<int>(threadIdx.x) / 32;
  if (col >= a.cols) return;  // columns come in whole vectors of 8
  uint32_t base[S];
  cluster_bases<S>(part + (c * 128 + f) * 4, base);
  uint16_t* p = static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(tok0) + c) * a.ldo + col;
  uint32_t off = 0;
#pragma unroll 2
  for (; c < c1; c += kStep, off += kStep * 512, p += kStep * a.ldo) {
    float4 d = cluster_sum4<S>(base, off);
    d = make_float4(d.x * a.alpha0, d.y * a.alpha0, d.z * a.alpha0, d.w * a.alpha0);
    if constexpr (GATED) {
      const float4 u = cluster_sum4<S>(base, off + NT * 512);
      d = make_float4(gate_act(d.x, gelu) * (u.x * a.alpha1), gate_act(d.y, gelu) * (u.y * a.alpha1),
                      gate_act(d.z, gelu) * (u.z * a.alpha1), gate_act(d.w, gelu) * (u.w * a.alpha1));
    }
    *reinterpret_cast<uint2*>(p) = pack4(d, fp16);
  }
}

// Quantises the n <= 32 rows of a token tile, 256 columns of X, into a stage: codes
// in the 128-byte swizzle of a K-major tile, scales in chunk order. Eight warps,
// a row each per step; rows past n stay as they are (they reach only
// accumulator columns that nobody reads).
template <int ELT, bool NV>
__device__ __forceinline__ void quantise_x(const FArgs& a, const Raw8<ELT> (&raw)[4], int n, int w, int lane,
                                           const float2* tab, uint8_t* codes, uint8_t* scales) {
  constexpr int kLanes = NV ? 8 : 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = w + 8 * i;
    if (r >= n) break;  // the whole warp
    uint32_t c;
    const uint32_t sw = quad_word<kLanes / 4>(quantize8<ELT, NV>(raw[i], a.xsc, tab, c), lane);
    *reinterpret_cast<uint32_t*>(codes + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) = c;
    if (lane % kLanes == 0) *reinterpret_cast<uint32_t*>(scales + (lane / kLanes) * 512 + r * 16) = sw;
  }
}

template <int ELT>
__device__ __forceinline__ void fetch_x(const FArgs& a, Raw8<ELT> (&raw)[4], int tok0, int n, int w, int col) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (w + 8 * i < n && col < a.k) raw[i] = load_raw8<ELT>(a.x, (static_cast<int64_t>(tok0) + w + 8 * i) * a.ldx + col);
    else raw[i] = Raw8<ELT>{};
  }
}

// QX: tiles of at most 32 tokens, which the CTA quantises itself (its own K
// range), so that one launch does everything: for a few tokens a launch of its
// own costs more than quantising them once per weight tile.
template <bool NV, bool GATED, int NT, bool QX>
__global__ void __launch_bounds__(kSplitThreads) fp4_split_kernel(const __grid_constant__ FMaps maps, const FArgs args) {
  using C = F4Split<GATED, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[C::stages], empty_bar[C::stages], tfull_bar;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int splits = args.splits;
  const int rank = static_cast<int>(blockIdx.x) % splits, unit = static_cast<int>(blockIdx.x) / splits;
  const int tile = unit / args.t_tiles, t_tile = unit % args.t_tiles, tok0 = t_tile * args.nt;
  const int kb0 = args.nkb * rank / splits, n_mine = args.nkb * (rank + 1) / splits - kb0;  // nkb <= 2^16
  constexpr int kSfBytes = Sf<NV>::quads * 512;
  // TMA bytes of a stage
  const uint32_t tx = C::nw * (kTile + kSfBytes) + (QX ? 0 : args.nt * 128 + kSfBytes);
  __shared__ float2 tab[QX && NV ? 128 : 1];
  if constexpr (QX && NV) {
    if (threadIdx.x >= 192) tab[threadIdx.x - 192] = nv_step_entry(threadIdx.x - 192, args.xsc.ts);
  }

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.b0);
    tma_prefetch_desc(&maps.sb0);
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(&full_bar[s], QX ? 9 : 1);  // the producer and, with QX, eight quantiser warps
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(&tfull_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_slot, C::cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_slot;
  volatile int* abortp = &abort_flag;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    const bool one = elect_one();
    auto load_w = [&](int i) {
      if (!one) return;
      const int s = i % C::stages, kb = kb0 + i;
      uint8_t* st = smem + s * C::stage_bytes;
      mbar_arrive_expect_tx(&full_bar[s], tx);
      tma_load_2d(st, &maps.b0, &full_bar[s], kb * 128, tile * 128);
      tma_load_3d(st + C::code_bytes, &maps.sb0, &full_bar[s], 0, kb * Sf<NV>::quads, tile);
      if constexpr (GATED) {
        tma_load_2d(st + kTile, &maps.b1, &full_bar[s], kb * 128, tile * 128);
        tma_load_3d(st + C::code_bytes + kSfTile, &maps.sb1, &full_bar[s], 0, kb * Sf<NV>::quads, tile);
      }
    };
    auto load_x = [&](int i) {
      if (QX || !one) return;
      const int s = i % C::stages, kb = kb0 + i;
      uint8_t* st = smem + s * C::stage_bytes;
      tma_load_2d(st + C::nw * kTile, &maps.a, &full_bar[s], kb * 128, tok0);
      // the 128-row scale chunk that holds this tile's tokens (whole 32-row quarters)
      tma_load_3d(st + C::code_bytes + C::nw * kSfTile, &maps.sa, &full_bar[s], 0, kb * Sf<NV>::quads, tok0 / 128);
    };
    const int ahead = min(n_mine, C::stages);
    if constexpr (QX) grid_dep_wait();
    for (int i = 0; i < ahead; ++i) load_w(i);  // without QX the previous kernel is the quantiser of X
    if constexpr (!QX) grid_dep_wait();
    grid_dep_launch();
    for (int i = 0; i < ahead; ++i) load_x(i);
    int done = ahead;
    for (int i = ahead; i < n_mine; ++i, ++done) {
      if (!warp_wait(&empty_bar[i % C::stages], ((i / C::stages) & 1) ^ 1, abortp, args.err)) break;
      load_w(i);
      load_x(i);
      __syncwarp();
    }
    for (int i = max(0, done - C::stages); i < done; ++i)  // every copy lands before the CTA ends
      if (one) wait_drain_bar(&full_bar[i % C::stages], (i / C::stages) & 1, args.err);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const bool one = elect_one();
    // column of the tile's first token in its 128-row scale chunk (QX: always 0)
    const uint32_t sfx_quarter = QX ? 0u : (tok0 % 128) / 32;
    const uint32_t lo0 = sdesc_lo(smem_u32(smem), 16);
    // As every role: the previous kernel first, so that the barriers' limit does
    // not run while that kernel does.
    grid_dep_wait();
    for (int i = 0; i < n_mine; ++i) {
      const int s = i % C::stages;
      if (!warp_wait(&full_bar[s], (i / C::stages) & 1, abortp, args.err)) break;
      tc_fence_after();
      const uint32_t lo = lo0 + s * (C::stage_bytes >> 4);
      const uint32_t sf = smem_u32(smem + s * C::stage_bytes + C::code_bytes);
      const uint32_t sf_t = tmem_base + C::acc_cols + s * C::sf_cols;
      if (one) {
#pragma unroll
        for (int c = 0; c < Sf<NV>::quads; ++c)
#pragma unroll
          for (int j = 0; j <= C::nw; ++j)
            tmem_cp_sf(sf_t + j * kSfCols + c * 4, sdesc_sf(sf + j * kSfTile + c * 512));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int c = Sf<NV>::quad(ks);
          const uint64_t xd = sdesc_of(lo + ((C::nw * kTile) >> 4) + 2 * ks);
          const uint32_t sfx = sf_t + C::nw * kSfCols + c * 4 + sfx_quarter;
#pragma unroll
          for (int j = 0; j < C::nw; ++j)
            umma_f4<NV, false>(tmem_base + j * NT, sdesc_of(lo + ((j * kTile) >> 4) + 2 * ks), xd,
                               idesc_f4<NV>(128, args.nt, Sf<NV>::id(ks)), sf_t + j * kSfCols + c * 4, sfx,
                               (i > 0 || ks > 0) ? 1u : 0u);
        }
        umma_commit(&empty_bar[s]);
      }
      __syncwarp();
    }
    if (one) {
      umma_commit(&tfull_bar);
      wait_drain_bar(&tfull_bar, 0, args.err);
    }
  } else {
    grid_dep_wait();
    if constexpr (QX) {
      // ---------------- quantiser of X ----------------
      auto run = [&](auto elt) {
        constexpr int ELT = decltype(elt)::value;
        const int n = static_cast<int>(min(static_cast<int64_t>(args.nt), args.rows - tok0)), w = warp - 2;
        Raw8<ELT> next[4];
        fetch_x(args, next, tok0, n, w, kb0 * kQK + lane * 8);
        for (int i = 0; i < n_mine; ++i) {
          const int s = i % C::stages;
          Raw8<ELT> raw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) raw[j] = next[j];
          if (i + 1 < n_mine) fetch_x(args, next, tok0, n, w, (kb0 + i + 1) * kQK + lane * 8);
          if (i >= C::stages && !warp_wait(&empty_bar[s], ((i / C::stages) & 1) ^ 1, abortp, args.err)) break;
          uint8_t* st = smem + s * C::stage_bytes;
          quantise_x<ELT, NV>(args, raw, n, w, lane, tab, st + C::nw * kTile,
                              st + C::code_bytes + C::nw * kSfTile);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_bar[s]);
        }
      };
      if (args.fp16) run(IntC<MOE_ELT_FP16>());
      else run(IntC<MOE_ELT_BF16>());
    }
    // ---------------- partial sums to shared memory ----------------
    __syncwarp();
    if (warp_wait(&tfull_bar, 0, abortp, args.err)) {
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem);  // [nw][NT][128]; the ring is drained
      for (int j = 0; j < C::nw; ++j)
        park_partials(tmem_base + j * NT, args.nt, warp, lane, part + j * NT * 128);
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync();  // every CTA's partial sums are in place, and out of tensor memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::cols);
  }
  if (!*abortp) {
    for_splits(splits, [&](auto n) {
      f4_finish<GATED, NT, decltype(n)::value>(args, smem_u32(smem), rank, tile, tok0);
    });
  }
  if (splits > 1) {
    __syncwarp();
    // No CTA leaves while its partial sums may still be read. The barrier is
    // relaxed; see cluster_leave for why that is enough here.
    cluster_leave();
  }
}

// ---------------------------------------------------------------------------
// Host side.

template <bool NV, bool GATED>
moe_status launch_pair(const FMaps& m, const FArgs& a, cudaStream_t s) {
  using C = F4Pair<GATED>;
  static ContextCache<int> cache;
  int most = 0;  // co-resident pairs on the current device
  const bool ok = cache.get(current_context_id, [](int& n) {
    if (!set_smem(fp4_pair_kernel<NV, GATED>, C::smem)) return false;
    LaunchCfg c(dim3(2), C::threads, C::smem, 2, false, nullptr);
    return cuda_status(cudaOccupancyMaxActiveClusters(&n, fp4_pair_kernel<NV, GATED>, &c.cfg)) == MOE_OK;
  }, most);
  if (!ok || most <= 0) return MOE_ERR_CUDA;
  LaunchCfg c(dim3(2 * static_cast<unsigned>(std::min<int64_t>(most, a.tiles))), C::threads, C::smem, 2, true, s);
  return launch_kernel(c, fp4_pair_kernel<NV, GATED>, m, a);
}

template <bool NV, bool GATED, int NT, bool QX>
moe_status launch_split_nt(const FMaps& m, FArgs a, int w_tiles, cudaStream_t s) {
  using C = F4Split<GATED, NT>;
  static ContextCache<bool> cache;
  bool raised;
  if (!cache.get(current_context_id, [](bool& v) { return v = set_smem(fp4_split_kernel<NV, GATED, NT, QX>, C::smem); }, raised))
    return MOE_ERR_CUDA;
  LaunchCfg c(dim3(static_cast<unsigned>(w_tiles * a.t_tiles * a.splits)), kSplitThreads, C::smem, a.splits, true, s);
  return launch_kernel(c, fp4_split_kernel<NV, GATED, NT, QX>, m, a);
}

struct F4Layout {
  size_t q, s, bytes;
};

moe_status f4_layout(const fp4_problem* p, F4Layout* L) {
  if (!p || !L) return MOE_ERR_INVALID_ARG;
  if (p->N <= 0) return MOE_ERR_INVALID_ARG;
  const moe_status st = fp4_check(p->format, p->M, p->K);
  if (st != MOE_OK) return st;
  if (p->elt != MOE_ELT_BF16 && p->elt != MOE_ELT_FP16) return MOE_ERR_UNSUPPORTED;
  if (p->act != FFN_SILU && p->act != FFN_GELU_TANH) return MOE_ERR_UNSUPPORTED;
  if (p->kernel < 0 || p->kernel > 2) return MOE_ERR_UNSUPPORTED;
  if (p->N % 8 != 0 || p->N > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  L->q = 256;  // after the error word
  L->s = L->q + align256(static_cast<size_t>(p->M) * (p->K / 2));
  L->bytes = L->s + align256(static_cast<size_t>((p->M + 127) / 128) * fp4_quads(p->format, p->K) * 512);
  return MOE_OK;
}

bool operand_ok(const fp4_operand* w, int32_t format) {
  return w && aligned(w->q, 16) && aligned(w->s, 16) && fp4_scale_ok(format, w->scale);
}

template <bool NV, bool GATED>
moe_status product(const fp4_problem* p, const F4Layout& L, const void* x, int64_t ldx, float x_scale,
                   const fp4_operand& w0, const fp4_operand* w1, void* y, int64_t ldy, void* ws, cudaStream_t s) {
  uint8_t *xq = at<uint8_t>(ws, L.q), *xs = at<uint8_t>(ws, L.s);
  const int quads = fp4_quads(p->format, p->K), bq = Sf<NV>::quads;
  FMaps m{};
  FArgs a{};
  a.err = static_cast<int32_t*>(ws);
  a.rows = p->M;
  a.nkb = static_cast<int>((p->K + kQK - 1) / kQK);
  a.cols = p->N;
  a.alpha0 = x_scale * w0.scale;
  a.alpha1 = GATED ? x_scale * w1->scale : 0.0f;
  a.fp16 = p->elt == MOE_ELT_FP16;
  a.gelu = p->act == FFN_GELU_TANH;
  a.m_tiles = static_cast<int>((p->M + 255) / 256);
  a.n_tiles = (p->N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
  a.tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
  // Tiles of up to 32 tokens quantise X themselves; tiles of 64 or 128 (halves or
  // whole chunks of X's scales) follow a quantiser launch, about a microsecond
  // beyond what they hide of it.
  const int w_tiles = (p->N + 127) / 128;
  SplitCost cost = GATED ? SplitCost{38.9, 0.113, 0.0, 0.0201, 0.034, 1.08, 0.33, 0.164, 2.50, 0.0196, 2}
                         : SplitCost{20.5, 0.295, 0.875, 0.0, 0.048, 1.47, 0.44, 0.067, 2.59, 0.0135, 1};
  SplitPlan sp = plan_split(p->M, w_tiles, a.nkb, cost, 16, 32, 16);
  cost.quantise = 0.0;
  SplitPlan big = plan_split(p->M, w_tiles, a.nkb, cost, 64, 128, 64);
  big.us += GATED ? 1.9 : 1.0;
  // A product that quantises X itself reads it while other CTAs already store Y.
  if (big.us < sp.us || overlap(x, ldx, p->K, y, ldy, p->N, p->M)) sp = big;
  const bool split = p->kernel ? p->kernel == 2 : sp.us <= pair_time(a.tiles, a.nkb, GATED ? 5.2 : 3.6, GATED ? 1.5 : 2.6);
  const int64_t t_tiles = (p->M + sp.nt - 1) / sp.nt;
  if (split && t_tiles * w_tiles * 8 > INT32_MAX) return MOE_ERR_UNSUPPORTED;  // grid x
  const bool own_x = split && sp.nt <= 32;  // the product quantises X itself
  if (!own_x && (!code_map(&m.a, xq, p->K, p->M, split ? sp.nt : 128) || !sf_map(&m.sa, xs, quads, p->M, bq)))
    return MOE_ERR_CUDA;
  if (!code_map(&m.b0, w0.q, p->K, p->N, 128) || !sf_map(&m.sb0, w0.s, quads, p->N, bq)) return MOE_ERR_CUDA;
  if (GATED && (!code_map(&m.b1, w1->q, p->K, p->N, 128) || !sf_map(&m.sb1, w1->s, quads, p->N, bq)))
    return MOE_ERR_CUDA;
  if (!split &&
      !tma_map_pitched(&m.o, y, p->N, p->M, ldy, 32, 32, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, CU_TENSOR_MAP_SWIZZLE_64B))
    return MOE_ERR_CUDA;
  if (!own_x) {
    const moe_status st = launch_fp4_quantize(x, p->elt, p->M, p->K, ldx, p->format, x_scale, xq, xs, s);
    if (st != MOE_OK) return st;
  }
  if (!split) return launch_pair<NV, GATED>(m, a, s);
  a.out = y;
  a.ldo = ldy;
  a.t_tiles = static_cast<int>(t_tiles);
  a.nt = sp.nt;
  a.splits = sp.splits;
  a.x = x;
  a.ldx = ldx;
  a.k = p->K;
  a.xsc = nv_scale(x_scale);
  if (sp.nt <= 16) return launch_split_nt<NV, GATED, 16, true>(m, a, w_tiles, s);
  if (sp.nt <= 32) return launch_split_nt<NV, GATED, 32, true>(m, a, w_tiles, s);
  if (sp.nt <= 64) return launch_split_nt<NV, GATED, 64, false>(m, a, w_tiles, s);
  return launch_split_nt<NV, GATED, 128, false>(m, a, w_tiles, s);
}

moe_status checked(const fp4_problem* p, const void* x, int64_t ldx, float x_scale, const fp4_operand* w0,
                   const fp4_operand* w1, bool gated, void* y, int64_t ldy, void* ws, void* stream) {
  F4Layout L;
  const moe_status st = f4_layout(p, &L);
  if (st != MOE_OK) return st;
  if (!aligned(ws, 256) || !operand_ok(w0, p->format) || (gated && !operand_ok(w1, p->format)) ||
      !fp4_scale_ok(p->format, x_scale))
    return MOE_ERR_INVALID_ARG;
  if (p->M == 0) return MOE_OK;
  if (!aligned(x, 16) || ldx < p->K || ldx % 8 != 0 || !aligned(y, 16) || ldy < p->N || ldy % 8 != 0)
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->format == FP4_NV)
    return gated ? product<true, true>(p, L, x, ldx, x_scale, *w0, w1, y, ldy, ws, s)
                 : product<true, false>(p, L, x, ldx, x_scale, *w0, w1, y, ldy, ws, s);
  return gated ? product<false, true>(p, L, x, ldx, x_scale, *w0, w1, y, ldy, ws, s)
               : product<false, false>(p, L, x, ldx, x_scale, *w0, w1, y, ldy, ws, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status fp4_workspace_bytes(const fp4_problem* p, size_t* bytes) {
  F4Layout L;
  const moe_status st = f4_layout(p, &L);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = L.bytes;
  return MOE_OK;
}

moe_status fp4_linear(const fp4_problem* p, const void* x, int64_t ldx, float x_scale, const fp4_operand* w,
                      void* y, int64_t ldy, void* ws, void* stream) {
  return checked(p, x, ldx, x_scale, w, nullptr, false, y, ldy, ws, stream);
}

moe_status fp4_gated_linear(const fp4_problem* p, const void* x, int64_t ldx, float x_scale,
                            const fp4_operand* w_gate, const fp4_operand* w_up, void* y, int64_t ldy, void* ws,
                            void* stream) {
  return checked(p, x, ldx, x_scale, w_gate, w_up, true, y, ldy, ws, stream);
}

moe_status fp4_get_device_error(const fp4_problem* p, const void* ws, int32_t* code_out, void* stream) {
  F4Layout L;
  const moe_status st = f4_layout(p, &L);
  if (st != MOE_OK) return st;
  if (!aligned(ws, 256) || !code_out) return MOE_ERR_INVALID_ARG;
  return cuda_status(
      cudaMemcpyAsync(code_out, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, static_cast<cudaStream_t>(stream)));
}

moe_status fp4_clear_device_error(const fp4_problem* p, void* ws, void* stream) {
  F4Layout L;
  const moe_status st = f4_layout(p, &L);
  if (st != MOE_OK) return st;
  if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(ws, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

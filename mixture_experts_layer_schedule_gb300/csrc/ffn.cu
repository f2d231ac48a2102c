// ffn.cu -- the dense gated feed-forward block: one gate/up/down set of weights
// applied to every token (a shared expert, or the dense layers beside routed
// ones), forward, forward without saved values, and backward.
//
//   G = X Wg^T, U = X Wu^T, A = h(G) * U, Y = A Wd^T       h = silu or gelu (tanh)
//   dA = dY Wd, dU = dA h(G), dG = dA U h'(G)
//   dX = dG Wg + dU Wu, dWd = dY^T A, dWg = dG^T X, dWu = dU^T X
//
// bf16 or fp16 operands, fp32 accumulation on the tensor cores (tcgen05). G, U,
// A, dG and dU are rounded to 16 bits where they become operands of the next
// product or saved values; h and h' are evaluated in fp32 from the fp32
// accumulator (forward) or the saved 16-bit G and U (backward).
//
// Two kernels cover the token counts:
//  * dense_pair_kernel: SM pairs (cta_group::2), 256 x 256 tiles with the tokens
//    on M, persistent, a ring of TMA stages, two accumulators so that an
//    epilogue runs under the next tile's products. For many tokens. Bound by the
//    tensor cores: 16384 tokens through 4096 x 1536 forward in 330 us (618 GFLOP,
//    1.87 PFLOP/s, what cuBLAS reaches in a burst; 375 us or 1.65 PFLOP/s in a
//    row, where the power cap holds the clock near 1.45 GHz), 8192 through 7168 x
//    2048 backward in 750 us (1443 GFLOP, 1.92 PFLOP/s; 850 us in a row).
//  * dense_split_kernel: the weight rows on M (128 per tile) and 16 to 128
//    tokens on N, so that a few tokens cost shared memory and tensor work in
//    proportion to the weights alone; K split over the CTAs of a cluster, whose
//    partial sums meet through distributed shared memory in rank order (no
//    atomics, the same sum in every run). For few tokens, where the time is
//    that of streaming the weights once, and of two dependent launches (about
//    2.5 us each from the first load to the last store): one token through
//    7168 x 2048 in 19 us (88 MB, 4.6 TB/s), through 4096 x 1536 in 11.8 us
//    (37.7 MB, 3.2 TB/s; 8.9 us when the weights are in L2), 77 tokens through
//    2048 x 1024 in 9.2 us, 1003 through 1000 x 680 in 14.3 us.
// Loads past an edge read zeros and stores past it are dropped, so N is any
// number >= 0 and H, I any multiples of 8 (16-byte row pitch).
#include <algorithm>

#include "dense_common.cuh"

namespace moe {
namespace {

enum DMode { D_GATED = 0, D_PLAIN = 1, D_DACT = 2, D_DX = 3, D_WGRAD = 4 };

template <int MODE>
struct DTraits {
  // dense_pair_kernel: operand A holds tokens (gradient rows for D_WGRAD)
  static constexpr bool a_mn = MODE == D_WGRAD;
  static constexpr bool b_mn = MODE == D_DACT || MODE == D_DX || MODE == D_WGRAD;
};
// dense_split_kernel: the weights, transposed in the data gradients
template <int MODE>
constexpr bool kSplitMn = MODE == D_DACT || MODE == D_DX;

struct DMaps {
  CUtensorMap a[3], b[3], o[3];
  CUtensorMap g, u;  // D_DACT: the saved G, U
};

struct DArgs {
  int32_t* err;
  int64_t tiles;            // all tiles of the launch
  int m_tiles[3], n_tiles[3];  // per problem (one problem but in D_WGRAD)
  int n_probs;
  int kb1, kb2;             // k-blocks of the two phases (D_DX), else kb1
  int64_t rows;             // output rows (tokens; weight rows in D_WGRAD per problem)
  int cols;                 // output columns
  int w_rows[3], w_cols[3];  // D_WGRAD: output extents per problem
  void* w_out[3];            // D_WGRAD with K split: the gradients
  int fp16, gelu, store_gu, out_f32;
  const void *g, *u;        // D_DACT: the saved G, U [rows, cols]
  void *o0, *o1, *o2;       // outputs stored from registers
  int64_t ldo;              // their row pitch (elements)
  int splits;               // CTAs (split kernel) or pairs (weight gradients) that share a tile's K
  int nt;                   // dense_split_kernel: tokens loaded per tile (multiple of 16)
  int t_tiles;              // dense_split_kernel: token tiles
  int early_w;              // dense_split_kernel: the previous kernel is one of the same call,
                            // so the weights are in place before it ends
};

// dense_split_kernel: weight rows, tokens.
struct SMaps {
  CUtensorMap a[2], b[2];
};

constexpr int kBK = 64;                    // k-block: 128 bytes of 16-bit values
constexpr int kHalfTile = 128 * kBK * 2;   // 16 KB: 128 rows of a k-block
constexpr int kThreads = 320;              // producer, MMA issuer, eight epilogue warps
constexpr int kOutBlock = 4096;            // a staged output block: 32 rows x 128 bytes

// ---------------------------------------------------------------------------
// SM pairs. Each CTA stages its 128 A rows and its half of the 256 B rows; the
// even CTA issues the MMAs of both.
constexpr int kPStageBytes = 2 * kHalfTile;

// Ring stages against staging for the epilogue warps: a second staged block per
// warp where the epilogue stores three outputs or also reads G and U.
template <int MODE>
struct PCfg {
  static constexpr int bufs = MODE == D_GATED || MODE == D_DACT ? 2 : 1;
  static constexpr int stages = bufs == 2 ? 5 : 6;
  static constexpr int smem = stages * kPStageBytes + 8 * bufs * kOutBlock + 1024;
  static_assert(smem <= 227 * 1024, "ring and staging within one CTA's shared memory");
};

struct DTile {
  int prob, mt, nt;
};

template <int MODE>
__device__ __forceinline__ DTile pair_tile(const DArgs& a, int64_t t) {
  DTile ti{0, 0, 0};
  if constexpr (MODE == D_WGRAD) {
    while (ti.prob < a.n_probs - 1) {
      const int64_t n = static_cast<int64_t>(a.m_tiles[ti.prob]) * a.n_tiles[ti.prob];
      if (t < n) break;
      t -= n;
      ++ti.prob;
    }
  }
  band_tile(t, a.m_tiles[ti.prob], a.n_tiles[ti.prob], ti.mt, ti.nt);
  return ti;
}

template <int MODE>
__device__ __forceinline__ void pair_loads(const DMaps& m, const DArgs& a, const DTile& ti, int kb,
                                           uint8_t* sA, uint32_t bar, int crank) {
  uint8_t* sB = sA + kHalfTile;
  const int m0 = ti.mt * 256 + crank * 128;  // this CTA's A rows
  if constexpr (MODE == D_GATED) {
    // D columns [0, 128) are gate rows, [128, 256) up rows of the same features
    tma_load_2d_pair(sA, &m.a[0], bar, kb * kBK, m0);
    tma_load_2d_pair(sB, &m.b[crank], bar, kb * kBK, ti.nt * 128);
  } else if constexpr (MODE == D_PLAIN) {
    tma_load_2d_pair(sA, &m.a[0], bar, kb * kBK, m0);
    tma_load_2d_pair(sB, &m.b[0], bar, kb * kBK, ti.nt * 256 + crank * 128);
  } else if constexpr (MODE == D_DACT || MODE == D_DX) {
    const int seg = (MODE == D_DX && kb >= a.kb1) ? 1 : 0;
    const int kk = seg ? kb - a.kb1 : kb;
    tma_load_2d_pair(sA, &m.a[seg], bar, kk * kBK, m0);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      tma_load_2d_pair(sB + c * (kHalfTile / 2), &m.b[seg], bar,
                       ti.nt * 256 + crank * 128 + c * 64, kk * kBK);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      tma_load_2d_pair(sA + c * (kHalfTile / 2), &m.a[ti.prob], bar, m0 + c * 64, kb * kBK);
#pragma unroll
    for (int c = 0; c < 2; ++c)
      tma_load_2d_pair(sB + c * (kHalfTile / 2), &m.b[ti.prob], bar,
                       ti.nt * 256 + crank * 128 + c * 64, kb * kBK);
  }
}

// 16-byte chunk `j` of this lane's row in a staged 32 x 128-byte block (the
// 128-byte swizzle spreads one warp store over all banks).
__device__ __forceinline__ void stage_chunk(uint32_t buf, int lane, int j, uint32_t a, uint32_t b,
                                            uint32_t c, uint32_t d) {
  const uint32_t addr = buf + lane * 128 + ((j ^ (lane & 7)) << 4);
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// One 32-row x 64-column block of 16-bit values (64 fp32 of each lane's row)
// through a staging buffer to one TMA store at (x, y).
template <int NB, bool FP16>
__device__ __forceinline__ void store_block16(const CUtensorMap* om, const float (&v)[64], int32_t x, int32_t y,
                                              int lane, uint8_t* bufs, uint32_t& n) {
  uint8_t* buf = bufs + (n++ % NB) * kOutBlock;
  if (lane == 0) bulk_wait_read<NB - 1>();  // the store that last used this buffer has read it
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    stage_chunk(smem_u32(buf), lane, j, pack2(v[8 * j], v[8 * j + 1], FP16),
                pack2(v[8 * j + 2], v[8 * j + 3], FP16), pack2(v[8 * j + 4], v[8 * j + 5], FP16),
                pack2(v[8 * j + 6], v[8 * j + 7], FP16));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(om, buf, x, y);
    bulk_commit();
  }
}

// The same for a 32-row x 32-column block of fp32 values.
__device__ __forceinline__ void store_block32(const CUtensorMap* om, const float* v, int32_t x,
                                              int32_t y, int lane, uint8_t* buf) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    stage_chunk(smem_u32(buf), lane, j, __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(om, buf, x, y);
    bulk_commit();
  }
}

__device__ __forceinline__ void acc_ld64(uint32_t taddr, float (&v)[64], bool any) {
  if (!any) {  // an empty sum (K = 0): the accumulator was never written
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = 0.0f;
    return;
  }
  uint32_t r0[32], r1[32];
  tmem_ld32(taddr, r0);
  tmem_ld32(taddr + 32, r1);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = __uint_as_float(r0[i]);
    v[32 + i] = __uint_as_float(r1[i]);
  }
}

// One warp's state across the tiles of its CTA: staged stores, and for D_DACT the
// two sets of staged G and U blocks (32 rows x 32 columns each, 64-byte rows
// with that swizzle) with the barriers that their loads complete on.
struct EpiState {
  uint8_t* bufs;
  uint64_t* in_bar;  // [2]
  uint32_t n;        // staged stores / blocks so far
  uint32_t fetched;  // D_DACT: blocks whose loads were issued
};

constexpr int kInBlock = 2048;

// D_DACT, block `n` of the warp's sequence at (x, y): fetch G and U into set n % 2
// once the stores of block n - 2 have left it (PENDING: stores of later blocks
// that may still be in flight).
template <int PENDING>
__device__ __forceinline__ void fetch_gu(const DMaps& m, EpiState& e, uint32_t n, int32_t x, int32_t y, int lane) {
  e.fetched = n + 1;
  if (lane == 0) {
    bulk_wait_read<PENDING>();
    uint8_t* set = e.bufs + (n & 1u) * (2 * kInBlock);
    uint64_t* bar = e.in_bar + (n & 1u);
    mbar_arrive_expect_tx(bar, 2 * kInBlock);
    tma_load_2d(set, &m.g, bar, x, y);
    tma_load_2d(set + kInBlock, &m.u, bar, x, y);
  }
}

// Blocks of 32 columns that a warp has in its half of tile ti (D_DACT).
__device__ __forceinline__ int dact_blocks(const DArgs& a, int32_t x0, int32_t y) {
  return y >= a.rows || x0 >= a.cols ? 0 : min(4, (a.cols - x0 + 31) / 32);
}

// Epilogue of one tile: each warp takes 32 rows (one per lane) and half of the
// 256 columns (gated: 64 gate columns and the 64 up columns of the same
// features). The activation and the element type are template flags: as run-time
// flags they added a third to the instructions per value, which bound the
// activation-gradient epilogue.
template <int MODE, bool GELU, bool FP16>
__device__ __forceinline__ void pair_epilogue(const DMaps& m, const DArgs& a, const DTile& ti,
                                              uint32_t tmem_acc, int quad, int half, int lane, int crank,
                                              EpiState& e, volatile int* abortp) {
  constexpr int NB = PCfg<MODE>::bufs;
  const uint32_t taddr = tmem_acc + (static_cast<uint32_t>(quad * 32) << 16);
  const int32_t y = ti.mt * 256 + crank * 128 + quad * 32;
  if constexpr (MODE == D_GATED) {
    const int32_t x = ti.nt * 128 + 64 * half;
    if (y >= a.rows || x >= a.cols) return;
    float g[64], u[64];
    acc_ld64(taddr + 64 * half, g, true);
    acc_ld64(taddr + 128 + 64 * half, u, true);
    if (a.store_gu) {
      store_block16<NB, FP16>(&m.o[0], g, x, y, lane, e.bufs, e.n);
      store_block16<NB, FP16>(&m.o[1], u, x, y, lane, e.bufs, e.n);
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) g[i] = gate_act(g[i], GELU) * u[i];
    store_block16<NB, FP16>(&m.o[2], g, x, y, lane, e.bufs, e.n);
  } else if constexpr (MODE == D_PLAIN || MODE == D_DX) {
    if (y >= a.rows) return;
    for (int c = 128 * half; c < 128 * half + 128; c += 64) {
      const int32_t x = ti.nt * 256 + c;
      if (x >= a.cols) break;
      float d[64];
      acc_ld64(taddr + c, d, true);
      store_block16<NB, FP16>(&m.o[0], d, x, y, lane, e.bufs, e.n);
    }
  } else if constexpr (MODE == D_DACT) {
    // dG and dU take the place of G and U in their set and leave by TMA stores:
    // about 4000 cycles a tile. Per-lane row accesses to global memory made it
    // 24000 (32 lines per load), longer than the products of K < 3000.
    const int32_t x0 = ti.nt * 256 + 128 * half;
    const int nb = dact_blocks(a, x0, y);
    for (int b = 0; b < nb; ++b) {
      const uint32_t n = e.n + b;
      if (b >= 1 && b + 1 < nb) fetch_gu<0>(m, e, n + 1, x0 + 32 * (b + 1), y, lane);
      uint32_t d[32];
      tmem_ld32(taddr + 128 * half + 32 * b, d);
      if (!warp_wait(e.in_bar + (n & 1u), (n >> 1) & 1u, abortp, a.err)) return;
      const uint32_t gp = smem_u32(e.bufs + (n & 1u) * (2 * kInBlock)) + lane * 64, up = gp + kInBlock;
      tmem_ld_wait();
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t at = (v ^ ((lane >> 1) & 3)) << 4;
        uint32_t gw[4], uw[4], og[4], ou[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(gw[0]), "=r"(gw[1]), "=r"(gw[2]), "=r"(gw[3])
                     : "r"(gp + at));
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(uw[0]), "=r"(uw[1]), "=r"(uw[2]), "=r"(uw[3])
                     : "r"(up + at));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 g = unpack2(gw[q], FP16), u = unpack2(uw[q], FP16);
          const float d0 = __uint_as_float(d[8 * v + 2 * q]);
          const float d1 = __uint_as_float(d[8 * v + 2 * q + 1]);
          float h0, s0, h1, s1;
          gate_act_grad(g.x, GELU, h0, s0);
          gate_act_grad(g.y, GELU, h1, s1);
          og[q] = pack2(d0 * u.x * s0, d1 * u.y * s1, FP16);
          ou[q] = pack2(d0 * h0, d1 * h1, FP16);
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(gp + at), "r"(og[0]), "r"(og[1]),
                     "r"(og[2]), "r"(og[3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(up + at), "r"(ou[0]), "r"(ou[1]),
                     "r"(ou[2]), "r"(ou[3])
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        uint8_t* set = e.bufs + (n & 1u) * (2 * kInBlock);
        tma_store_2d(&m.o[0], set, x0 + 32 * b, y);
        tma_store_2d(&m.o[1], set + kInBlock, x0 + 32 * b, y);
        bulk_commit();
      }
    }
    e.n += nb;
  } else {  // D_WGRAD
    const CUtensorMap* om = &m.o[ti.prob];
    if (y >= a.w_rows[ti.prob]) return;
    for (int c = 128 * half; c < 128 * half + 128; c += 64) {
      const int32_t x = ti.nt * 256 + c;
      if (x >= a.w_cols[ti.prob]) break;
      float d[64];
      acc_ld64(taddr + c, d, a.kb1 > 0);
      if (a.out_f32) {
        store_block32(om, d, x, y, lane, e.bufs);
        if (x + 32 < a.w_cols[ti.prob]) store_block32(om, d + 32, x + 32, y, lane, e.bufs);
      } else {
        store_block16<NB, FP16>(om, d, x, y, lane, e.bufs, e.n);
      }
    }
  }
}

// K-split weight gradients: a CTA's 128 x 256 partial sums in the drained ring,
// rows of 260 floats (16-byte stores of a warp then cover all banks).
constexpr int kPartLd = 260;
static_assert(128 * kPartLd * 4 <= PCfg<D_WGRAD>::stages * kPStageBytes, "the partial sums fit the drained ring");

__device__ __forceinline__ void park_rows(uint32_t tmem, int warp, int lane, float* part) {
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128 * half;
  float4* row = reinterpret_cast<float4*>(part + (quad * 32 + lane) * kPartLd + 128 * half);
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i)
      row[c / 4 + i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                   __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
  }
}

// Rows [128 q / S, 128 (q + 1) / S) of this CTA's 128, q its pair's place in the
// cluster: the S partial sums in pair order, rounded once.
__device__ __forceinline__ void finish_rows(const DArgs& a, const DTile& ti, uint32_t part, int q, int crank,
                                            int warp, int lane) {
  const int S = a.splits;
  for (int r = 128 * q / S + warp; r < 128 * (q + 1) / S; r += kThreads / 32) {
    const int y = ti.mt * 256 + crank * 128 + r;
    if (y >= a.w_rows[ti.prob]) break;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = 128 * j + 4 * lane, x = ti.nt * 256 + col;
      if (x >= a.w_cols[ti.prob]) continue;  // columns come in whole vectors of 8
      float4 v[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m < S) {
          uint32_t addr;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                       : "=r"(addr)
                       : "r"(part + (r * kPartLd + col) * 4), "r"(2 * m + crank));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[m].x), "=f"(v[m].y), "=f"(v[m].z), "=f"(v[m].w)
                       : "r"(addr));
        }
      }
      float4 d = v[0];
#pragma unroll
      for (int m = 1; m < 4; ++m)
        if (m < S) {
          d.x += v[m].x;
          d.y += v[m].y;
          d.z += v[m].z;
          d.w += v[m].w;
        }
      const int64_t o = static_cast<int64_t>(y) * a.w_cols[ti.prob] + x;
      if (a.out_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.w_out[ti.prob]) + o) = d;
      else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.w_out[ti.prob]) + o) = pack4(d, a.fp16 != 0);
    }
  }
}

// KSPLIT (weight gradients of few tiles and many tokens): a cluster of up to
// four pairs shares one tile's K, and its partial sums meet through distributed
// shared memory in pair order.
template <int MODE, bool KSPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    dense_pair_kernel(const __grid_constant__ DMaps maps, const DArgs args) {
  static_assert(!KSPLIT || MODE == D_WGRAD, "K is split in the weight gradients only");
  constexpr int kPStages = PCfg<MODE>::stages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kPStages], empty_bar[kPStages], tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint64_t in_bar[MODE == D_DACT ? 16 : 1];  // D_DACT: two per epilogue warp
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const uint32_t lead = cta & ~1u;  // the pair's even CTA
  const int crank = static_cast<int>(cta & 1u);
  const bool leader = crank == 0;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);

  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
    if constexpr (MODE == D_GATED) {
      tma_prefetch_desc(&maps.b[1]);
      tma_prefetch_desc(&maps.o[2]);
    } else {
      tma_prefetch_desc(&maps.o[0]);
    }
    if constexpr (MODE == D_DACT) {
      tma_prefetch_desc(&maps.g);
      tma_prefetch_desc(&maps.u);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], 16);  // one arrive per epilogue warp of both CTAs
    }
    mbar_init(&drain_bar, 1);
    if constexpr (MODE == D_DACT)
      for (int i = 0; i < 16; ++i) mbar_init(&in_bar[i], 1);
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
  const int nkb = args.kb1 + args.kb2;
  // Tiles of this pair (KSPLIT: one, shared by the cluster) and its k-blocks.
  const int64_t first = KSPLIT ? blockIdx.x / 2 / args.splits : blockIdx.x / 2;
  const int64_t stride = KSPLIT ? args.tiles : gridDim.x / 2;
  const int q = KSPLIT ? static_cast<int>(cta >> 1) : 0;
  const int kb0 = KSPLIT ? static_cast<int>(static_cast<int64_t>(nkb) * q / args.splits) : 0;
  const int kb1 = KSPLIT ? static_cast<int>(static_cast<int64_t>(nkb) * (q + 1) / args.splits) : nkb;
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
    bool ok = true;
    for (int64_t t = first; t < args.tiles && ok; t += stride) {
      const DTile ti = pair_tile<MODE>(args, t);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!warp_wait(&empty_bar[stage], phase ^ 1u, abortp, args.err)) { ok = false; break; }
        if (one) {
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kPStageBytes);
          pair_loads<MODE>(maps, args, ti, kb, smem + stage * kPStageBytes,
                           cluster_addr(&full_bar[stage], lead), crank);
        }
        __syncwarp();
        issued_mask |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kPStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (leader && one)  // the even CTA's full barriers count both CTAs' copies
      for (int s = 0; s < kPStages; ++s)
        if ((issued_mask >> s) & 1u) wait_drain_bar(&full_bar[s], (issued_parity >> s) & 1u, args.err);
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer (even CTA) ----------------
      const bool one = elect_one();
      const uint32_t idesc = idesc_16(256, 256, DTraits<MODE>::a_mn, DTraits<MODE>::b_mn, args.fp16 != 0);
      constexpr uint32_t kAStep = (DTraits<MODE>::a_mn ? 2048 : 32) >> 4, kBStep = (DTraits<MODE>::b_mn ? 2048 : 32) >> 4;
      const uint32_t a_lo0 = sdesc_lo(smem_u32(smem), DTraits<MODE>::a_mn ? kHalfTile / 2 : 16);
      const uint32_t b_lo0 = sdesc_lo(smem_u32(smem + kHalfTile), DTraits<MODE>::b_mn ? kHalfTile / 2 : 16);
      int stage = 0, acc = 0;
      uint32_t phase = 0, uses = 0;  // uses: bit b = parity of the tiles committed on accumulator b
      bool ok = true;
      for (int64_t t = first; t < args.tiles; t += stride) {
        if (!warp_wait(&tempty_bar[acc], ((uses >> acc) & 1u) ^ 1u, abortp, args.err)) break;
        tc_fence_after();
        const uint32_t dtmem = tmem_base + acc * 256;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!warp_wait(&full_bar[stage], phase, abortp, args.err)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_lo = a_lo0 + stage * (kPStageBytes >> 4), b_lo = b_lo0 + stage * (kPStageBytes >> 4);
          if (one) {
#pragma unroll
            for (int ks = 0; ks < kBK / 16; ++ks)
              umma_bf16_pair(dtmem, sdesc_of(a_lo + ks * kAStep), sdesc_of(b_lo + ks * kBStep), idesc,
                             (kb > kb0 || ks > 0) ? 1u : 0u);
            umma_commit_pair_mc(&empty_bar[stage], pair_mask);  // both CTAs may refill the stage
          }
          __syncwarp();
          if (++stage == kPStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (one) umma_commit_pair_mc(&tfull_bar[acc], pair_mask);
        __syncwarp();
        uses ^= 1u << acc;
        acc ^= 1;
      }
      if (one) {
        umma_commit_pair(&drain_bar);
        wait_drain_bar(&drain_bar, 0, args.err);
      }
    }
  } else {
    // ---------------- epilogue warps 2..9 (both CTAs) ----------------
    const int quad = warp & 3, half = (warp - 2) >> 2;
    EpiState e{smem + kPStages * kPStageBytes + (warp - 2) * PCfg<MODE>::bufs * kOutBlock,
               in_bar + (MODE == D_DACT ? 2 * (warp - 2) : 0), 0u, 0u};
    uint32_t uses = 0;
    int acc = 0;
    for (int64_t t = first; t < args.tiles; t += stride) {
      const DTile ti = pair_tile<MODE>(args, t);
      if constexpr (MODE == D_DACT) {  // the first two blocks of G and U fly under the products
        const int32_t x0 = ti.nt * 256 + 128 * half, y = ti.mt * 256 + crank * 128 + quad * 32;
        const int nb = dact_blocks(args, x0, y);
        if (nb > 0) fetch_gu<1>(maps, e, e.n, x0, y, lane);
        if (nb > 1) fetch_gu<0>(maps, e, e.n + 1, x0 + 32, y, lane);
      }
      if (!warp_wait(&tfull_bar[acc], (uses >> acc) & 1u, abortp, args.err)) break;
      tc_fence_after();
      if constexpr (KSPLIT) park_rows(tmem_base, warp, lane, reinterpret_cast<float*>(smem));
      else with_flags<MODE == D_GATED || MODE == D_DACT>(args.gelu != 0, args.fp16 != 0, [&](auto gelu, auto fp16) {
        pair_epilogue<MODE, decltype(gelu)::value != 0, decltype(fp16)::value != 0>(
            maps, args, ti, tmem_base + acc * 256, quad, half, lane, crank, e, abortp);
      });
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(&tempty_bar[acc]);
        else mbar_arrive_peer(cluster_addr(&tempty_bar[acc], lead));
      }
      uses ^= 1u << acc;
      acc ^= 1;
    }
    for (uint32_t n = e.n; n < e.fetched; ++n)  // left early: its loads land before the CTA ends
      wait_drain_bar(e.in_bar + (n & 1u), (n >> 1) & 1u, args.err);
    if (lane == 0) bulk_wait_all();
  }

  if constexpr (KSPLIT) {
    __syncwarp();
    cluster_sync();  // every CTA's partial sums are in place
    if (!*abortp) finish_rows(args, pair_tile<MODE>(args, first), smem_u32(smem), q, crank, warp, lane);
  }
  tc_fence_before();
  __syncwarp();
  // Both CTAs are through: the even CTA's MMAs into this CTA's tensor memory have
  // retired, and nothing signals a CTA that may leave, or (KSPLIT) reads its partial
  // sums: see cluster_leave.
  cluster_leave();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------------------
// Weight rows on M, NT tokens on N, K split over the CTAs of a cluster.
//
// Shared memory per CTA is kept between 77 and 113 KB: two CTAs fit one SM (the
// bytes in flight that stream the weights at full rate come from both) and
// never three, so the accumulators of co-resident CTAs (at most 256 columns
// each) always fit tensor memory and no allocation waits for another CTA.
template <int NT>
struct SplitCfg {
  static constexpr int stage_bytes = kHalfTile + NT * kBK * 2;
  static constexpr int stages = NT <= 32 ? 5 : (NT == 64 ? 4 : 3);
  static constexpr int smem = stages * stage_bytes + 1024;
  static constexpr uint32_t cols = NT < 32 ? 32 : NT;
  static_assert(smem >= 77 * 1024 && smem <= 113 * 1024, "two CTAs per SM, never three");
  static_assert(NT * 128 * 4 <= stages * stage_bytes, "the partial sums fit the drained ring");
};

// The weight rows of one k-block (16 KB); what they hold does not depend on the
// kernel before this one.
template <int MODE>
__device__ __forceinline__ void split_load_w(const SMaps& m, const DArgs& a, int tile, int kb,
                                             uint8_t* sW, uint64_t* bar) {
  if constexpr (MODE == D_GATED) {  // 64 gate rows, then the 64 up rows of the same features
    tma_load_2d(sW, &m.a[0], bar, kb * kBK, tile * 64);
    tma_load_2d(sW + kHalfTile / 2, &m.a[1], bar, kb * kBK, tile * 64);
  } else if constexpr (MODE == D_PLAIN) {
    tma_load_2d(sW, &m.a[0], bar, kb * kBK, tile * 128);
  } else {
    const int seg = (MODE == D_DX && kb >= a.kb1) ? 1 : 0;
    const int kk = seg ? kb - a.kb1 : kb;
#pragma unroll
    for (int c = 0; c < 2; ++c)
      tma_load_2d(sW + c * (kHalfTile / 2), &m.a[seg], bar, tile * 128 + c * 64, kk * kBK);
  }
}

template <int MODE>
__device__ __forceinline__ void split_load_x(const SMaps& m, const DArgs& a, int tok0, int kb,
                                             uint8_t* sX, uint64_t* bar) {
  const int seg = (MODE == D_DX && kb >= a.kb1) ? 1 : 0;
  tma_load_2d(sX, &m.b[seg], bar, (seg ? kb - a.kb1 : kb) * kBK, tok0);
}

// The token columns that this CTA of the cluster finishes: the partial sums, the
// mode's arithmetic, the stores. A thread keeps its four features and walks the
// tokens, so that all but the sums is one addition per pointer.
template <int MODE, int S>
__device__ __forceinline__ void split_finish(const DArgs& a, uint32_t part, int rank, int tile, int tok0) {
  constexpr int kFeat = MODE == D_GATED ? 64 : 128;  // features of the tile
  constexpr int kQuads = kFeat / 4, kStep = kSplitThreads / kQuads;
  static_assert(kSplitThreads % kQuads == 0, "a thread keeps its features");
  int c0, c1;
  finish_range(static_cast<int>(min(static_cast<int64_t>(a.nt), a.rows - tok0)), rank, S, c0, c1);
  const bool fp16 = a.fp16 != 0, gelu = a.gelu != 0;
  const int f = 4 * (static_cast<int>(threadIdx.x) % kQuads), col = tile * kFeat + f;
  int c = c0 + static_cast<int>(threadIdx.x) / kQuads;
  if (col >= a.cols) return;  // columns come in whole vectors of 8
  uint32_t base[S];
  cluster_bases<S>(part + (c * 128 + f) * 4, base);
  const int64_t o = (static_cast<int64_t>(tok0) + c) * a.ldo + col, step = kStep * a.ldo;
  uint16_t *p0 = static_cast<uint16_t*>(a.o0) + o, *p1 = static_cast<uint16_t*>(a.o1) + o;
  uint16_t* p2 = static_cast<uint16_t*>(a.o2) + o;
  const uint16_t *pg = static_cast<const uint16_t*>(a.g) + o, *pu = static_cast<const uint16_t*>(a.u) + o;
  uint32_t off = 0;
#pragma unroll 2
  for (; c < c1; c += kStep, off += kStep * 512) {
    uint2 gw, uw;
    if constexpr (MODE == D_DACT) {
      gw = *reinterpret_cast<const uint2*>(pg);
      uw = *reinterpret_cast<const uint2*>(pu);
      pg += step;
      pu += step;
    }
    const float4 d = cluster_sum4<S>(base, off);
    if constexpr (MODE == D_GATED) {
      const float4 u = cluster_sum4<S>(base, off + 256);
      if (a.store_gu) {
        *reinterpret_cast<uint2*>(p0) = pack4(d, fp16);
        *reinterpret_cast<uint2*>(p1) = pack4(u, fp16);
        p0 += step;
        p1 += step;
      }
      *reinterpret_cast<uint2*>(p2) =
          pack4(make_float4(gate_act(d.x, gelu) * u.x, gate_act(d.y, gelu) * u.y, gate_act(d.z, gelu) * u.z,
                            gate_act(d.w, gelu) * u.w),
                fp16);
      p2 += step;
    } else if constexpr (MODE == D_DACT) {
      const float2 g0 = unpack2(gw.x, fp16), g1 = unpack2(gw.y, fp16);
      const float2 u0 = unpack2(uw.x, fp16), u1 = unpack2(uw.y, fp16);
      float h[4], q[4];
      gate_act_grad(g0.x, gelu, h[0], q[0]);
      gate_act_grad(g0.y, gelu, h[1], q[1]);
      gate_act_grad(g1.x, gelu, h[2], q[2]);
      gate_act_grad(g1.y, gelu, h[3], q[3]);
      *reinterpret_cast<uint2*>(p0) =
          pack4(make_float4(d.x * u0.x * q[0], d.y * u0.y * q[1], d.z * u1.x * q[2], d.w * u1.y * q[3]), fp16);
      *reinterpret_cast<uint2*>(p1) = pack4(make_float4(d.x * h[0], d.y * h[1], d.z * h[2], d.w * h[3]), fp16);
      p0 += step;
      p1 += step;
    } else {
      *reinterpret_cast<uint2*>(p0) = pack4(d, fp16);
      p0 += step;
    }
  }
}

template <int MODE, int NT>
__global__ void __launch_bounds__(kSplitThreads)
    dense_split_kernel(const __grid_constant__ SMaps maps, const DArgs args) {
  using C = SplitCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[C::stages], empty_bar[C::stages], tfull_bar;
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int splits = args.splits;
  // rank fastest, then the token tiles of one weight tile (they read its rows
  // from L2 at the same time), then the weight tiles
  const int rank = static_cast<int>(blockIdx.x) % splits, unit = static_cast<int>(blockIdx.x) / splits;
  const int tile = unit / args.t_tiles, tok0 = unit % args.t_tiles * args.nt;
  const uint32_t tx = kHalfTile + args.nt * (kBK * 2);  // bytes of a stage
  const int nkb = args.kb1 + args.kb2;
  const int kb0 = nkb * rank / splits, n_mine = nkb * (rank + 1) / splits - kb0;  // nkb <= 2^19

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&maps.a[0]);
    tma_prefetch_desc(&maps.b[0]);
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(&full_bar[s], 1);
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
    // After another kernel of the same call, the first ring of weight tiles
    // goes out before that kernel's results are needed.
    const bool one = elect_one();
    if (!args.early_w) grid_dep_wait();
    const int ahead = min(n_mine, C::stages);
    for (int i = 0; one && i < ahead; ++i) {
      mbar_arrive_expect_tx(&full_bar[i], tx);
      split_load_w<MODE>(maps, args, tile, kb0 + i, smem + i * C::stage_bytes, &full_bar[i]);
    }
    grid_dep_wait();
    grid_dep_launch();
    for (int i = 0; one && i < ahead; ++i)
      split_load_x<MODE>(maps, args, tok0, kb0 + i, smem + i * C::stage_bytes + kHalfTile, &full_bar[i]);
    int done = ahead;
    for (int i = ahead; i < n_mine; ++i, ++done) {
      const int s = i % C::stages;
      if (!warp_wait(&empty_bar[s], ((i / C::stages) & 1) ^ 1, abortp, args.err)) break;
      if (one) {
        uint8_t* st = smem + s * C::stage_bytes;
        mbar_arrive_expect_tx(&full_bar[s], tx);
        split_load_w<MODE>(maps, args, tile, kb0 + i, st, &full_bar[s]);
        split_load_x<MODE>(maps, args, tok0, kb0 + i, st + kHalfTile, &full_bar[s]);
      }
      __syncwarp();
    }
    for (int i = max(0, done - C::stages); i < done; ++i)  // every copy lands before the CTA ends
      if (one) wait_drain_bar(&full_bar[i % C::stages], (i / C::stages) & 1, args.err);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const bool one = elect_one();
    const uint32_t idesc = idesc_16(128, args.nt, kSplitMn<MODE>, false, args.fp16 != 0);
    constexpr uint32_t kWStep = (kSplitMn<MODE> ? 2048 : 32) >> 4;
    const uint32_t w_lo0 = sdesc_lo(smem_u32(smem), kSplitMn<MODE> ? kHalfTile / 2 : 16);
    const uint32_t x_lo0 = sdesc_lo(smem_u32(smem + kHalfTile), 16);
    // Every role waits for the previous kernel before its first barrier: the
    // barriers' limit must not run while that kernel does.
    grid_dep_wait();
    for (int i = 0; i < n_mine; ++i) {
      const int s = i % C::stages;
      if (!warp_wait(&full_bar[s], (i / C::stages) & 1, abortp, args.err)) break;
      tc_fence_after();
      const uint32_t w_lo = w_lo0 + s * (C::stage_bytes >> 4), x_lo = x_lo0 + s * (C::stage_bytes >> 4);
      if (one) {
#pragma unroll
        for (int ks = 0; ks < kBK / 16; ++ks)
          umma_bf16(tmem_base, sdesc_of(w_lo + ks * kWStep), sdesc_of(x_lo + 2 * ks), idesc,
                    (i > 0 || ks > 0) ? 1u : 0u);
        umma_commit(&empty_bar[s]);
      }
      __syncwarp();
    }
    if (one) {
      umma_commit(&tfull_bar);
      wait_drain_bar(&tfull_bar, 0, args.err);
    }
  } else {
    // ---------------- partial sums to shared memory ----------------
    grid_dep_wait();
    if (warp_wait(&tfull_bar, 0, abortp, args.err)) {
      tc_fence_after();
      park_partials(tmem_base, args.nt, warp, lane, reinterpret_cast<float*>(smem));  // the ring is drained
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
      split_finish<MODE, decltype(n)::value>(args, smem_u32(smem), rank, tile, tok0);
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

// Co-resident clusters of 1 to 4 CTA pairs of the pair kernel.
struct PairClusters {
  int n[5];
};

// Those of `pairs` pairs on the current device; 0 if it cannot be told.
template <int MODE, bool KSPLIT>
int pair_clusters(int pairs) {
  static ContextCache<PairClusters> cache;
  PairClusters v{};
  const bool ok = cache.get(current_context_id, [](PairClusters& c) {
    if (!set_smem(dense_pair_kernel<MODE, KSPLIT>, PCfg<MODE>::smem)) return false;
    for (int p = 1; p <= (KSPLIT ? 4 : 1); ++p) {
      LaunchCfg l(dim3(2 * p), kThreads, PCfg<MODE>::smem, 2 * p, false, nullptr);
      if (cuda_status(cudaOccupancyMaxActiveClusters(&c.n[p], dense_pair_kernel<MODE, KSPLIT>, &l.cfg)) != MOE_OK) return false;
    }
    return true;
  }, v);
  return ok ? v.n[pairs] : 0;
}

template <int MODE>
moe_status launch_pair_tiles(const DMaps& m, const DArgs& a, cudaStream_t s) {
  if (a.tiles <= 0) return MOE_OK;
  const int most = pair_clusters<MODE, false>(1);
  if (most <= 0) return MOE_ERR_CUDA;
  LaunchCfg c(dim3(2 * static_cast<unsigned>(std::min<int64_t>(most, a.tiles))), kThreads, PCfg<MODE>::smem, 2, true, s);
  return launch_kernel(c, dense_pair_kernel<MODE, false>, m, a);
}

// The weight gradients with K split over the pairs of a cluster where that
// shortens the k-blocks one pair walks by more than the join costs (about eight
// k-blocks): few tiles and many tokens.
moe_status launch_wgrad(const DMaps& m, DArgs a, cudaStream_t s) {
  int64_t least = 0;
  for (int p = 1; p <= 4; ++p) {
    const int most = p == 1 ? pair_clusters<D_WGRAD, false>(1) : pair_clusters<D_WGRAD, true>(p);
    if (most <= 0) continue;
    const int64_t t = (a.tiles + most - 1) / most * ((a.kb1 + p - 1) / p) + (p > 1 ? 8 : 0);
    if (p == 1 || t < least) {
      a.splits = p;
      least = t;
    }
  }
  if (a.splits == 1) return launch_pair_tiles<D_WGRAD>(m, a, s);
  LaunchCfg c(dim3(static_cast<unsigned>(2 * a.splits * a.tiles)), kThreads, PCfg<D_WGRAD>::smem, 2 * a.splits, true, s);
  return launch_kernel(c, dense_pair_kernel<D_WGRAD, true>, m, a);
}

template <int MODE, int NT>
moe_status launch_split_nt(const SMaps& m, const DArgs& a, int w_tiles, cudaStream_t s) {
  static ContextCache<bool> cache;
  bool raised;
  if (!cache.get(current_context_id, [](bool& v) { return v = set_smem(dense_split_kernel<MODE, NT>, SplitCfg<NT>::smem); }, raised))
    return MOE_ERR_CUDA;
  LaunchCfg c(dim3(static_cast<unsigned>(w_tiles * a.t_tiles * a.splits)), kSplitThreads, SplitCfg<NT>::smem, a.splits, true, s);
  return launch_kernel(c, dense_split_kernel<MODE, NT>, m, a);
}

template <int MODE>
moe_status launch_split(const SMaps& m, DArgs a, const SplitPlan& sp, int w_tiles, cudaStream_t s) {
  const int64_t t_tiles = (a.rows + sp.nt - 1) / sp.nt;
  if (w_tiles * t_tiles * 8 > INT32_MAX) return MOE_ERR_UNSUPPORTED;  // grid x
  a.nt = sp.nt;
  a.t_tiles = static_cast<int>(t_tiles);
  a.splits = sp.splits;
  if (sp.nt <= 16) return launch_split_nt<MODE, 16>(m, a, w_tiles, s);
  if (sp.nt <= 32) return launch_split_nt<MODE, 32>(m, a, w_tiles, s);
  if (sp.nt <= 64) return launch_split_nt<MODE, 64>(m, a, w_tiles, s);
  return launch_split_nt<MODE, 128>(m, a, w_tiles, s);
}

bool map16(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int64_t pitch, int box_outer) {
  return tma_map_pitched(m, base, inner, outer, pitch, kBK, box_outer, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2);
}
bool map_out16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t pitch) {
  return tma_map_pitched(m, base, cols, rows, pitch, 64, 32, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2);
}
// 32 x 32 blocks of a dense matrix (64-byte rows).
bool map_block16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows) {
  return tma_map_pitched(m, base, cols, rows, cols, 32, 32, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                         CU_TENSOR_MAP_SWIZZLE_64B);
}
bool map_out32(CUtensorMap* m, const void* base, int64_t cols, int64_t rows) {
  return tma_map_pitched(m, base, cols, rows, cols, 32, 32, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4);
}

int blocks(int64_t n, int b) { return static_cast<int>((n + b - 1) / b); }

struct FfnLayout {
  int64_t N;
  int H, I;
  size_t dg, du, bytes;
};

moe_status ffn_layout(const ffn_problem* p, FfnLayout* L) {
  if (!p || !L) return MOE_ERR_INVALID_ARG;
  if (p->N < 0 || p->H <= 0 || p->I <= 0) return MOE_ERR_INVALID_ARG;
  if (p->elt != MOE_ELT_BF16 && p->elt != MOE_ELT_FP16) return MOE_ERR_UNSUPPORTED;
  if (p->act != FFN_SILU && p->act != FFN_GELU_TANH) return MOE_ERR_UNSUPPORTED;
  if (p->grad_elt != p->elt && p->grad_elt != MOE_ELT_FP32) return MOE_ERR_UNSUPPORTED;
  if (p->kernel < 0 || p->kernel > 2) return MOE_ERR_UNSUPPORTED;
  if (p->H % 8 != 0 || p->I % 8 != 0) return MOE_ERR_UNSUPPORTED;
  // tile coordinates and token indices are int32 on the device
  if (p->N > (1LL << 31) - 512 || p->H > (1 << 24) || p->I > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  L->N = p->N;
  L->H = p->H;
  L->I = p->I;
  const size_t one = align256(static_cast<size_t>(p->N) * p->I * 2);
  L->dg = 256;  // after the error word
  L->du = L->dg + one;
  L->bytes = L->du + one;
  return MOE_OK;
}

// A pitched 16-bit matrix of `cols` columns (16-byte rows).
inline bool mat(const void* p, int64_t ld, int64_t cols) { return aligned(p, 16) && ld >= cols && ld % 8 == 0; }

// The split kernel's launch for a product over nkb k-blocks with w_tiles weight
// tiles, and whether it serves the product against `pair_tiles` 256 x 256 tiles
// on SM pairs: the smaller of two expected times.
SplitPlan ffn_plan(const ffn_problem* p, int w_tiles, int64_t pair_tiles, int nkb, bool backward, bool* split) {
  // The backward's stages take two or more boxes of transposed weights each.
  constexpr SplitCost kForward{16.4, 0.189, 0.030, 0.0119, 0.032, 0.49, 0.157, 0.148, 2.57, 0.0, 1};
  constexpr SplitCost kBackward{16.4, 0.283, 0.195, 0.0077, 0.054, 1.45, 0.32, 0.1, 2.14, 0.0, 1};
  const SplitPlan sp = plan_split(p->N, w_tiles, nkb, backward ? kBackward : kForward, 16, 128, 16);
  *split = p->kernel ? p->kernel == 2 : sp.us <= pair_time(pair_tiles, nkb, 2.5, 1.75);
  return sp;
}

DArgs base_args(const ffn_problem* p, void* ws) {
  DArgs a{};
  a.err = static_cast<int32_t*>(ws);
  a.rows = p->N;
  a.fp16 = p->elt == MOE_ELT_FP16;
  a.gelu = p->act == FFN_GELU_TANH;
  a.n_probs = 1;
  a.splits = 1;
  return a;
}

moe_status run_gate_up(const ffn_problem* p, const void* x, int64_t ldx, const void* wg, const void* wu,
                       void* g, void* u, void* act, void* ws, cudaStream_t s) {
  DArgs a = base_args(p, ws);
  a.cols = p->I;
  a.kb1 = blocks(p->H, kBK);
  a.store_gu = g != nullptr;
  bool split;
  const SplitPlan sp = ffn_plan(p, blocks(p->I, 64), static_cast<int64_t>(blocks(p->N, 256)) * blocks(p->I, 128), a.kb1, false, &split);
  if (split) {
    SMaps m{};
    if (!map16(&m.a[0], wg, p->H, p->I, p->H, 64) || !map16(&m.a[1], wu, p->H, p->I, p->H, 64) ||
        !map16(&m.b[0], x, p->H, p->N, ldx, sp.nt))
      return MOE_ERR_CUDA;
    a.o0 = g;
    a.o1 = u;
    a.o2 = act;
    a.ldo = p->I;
    return launch_split<D_GATED>(m, a, sp, blocks(p->I, 64), s);
  }
  DMaps m{};
  if (!map16(&m.a[0], x, p->H, p->N, ldx, 128) || !map16(&m.b[0], wg, p->H, p->I, p->H, 128) ||
      !map16(&m.b[1], wu, p->H, p->I, p->H, 128) || !map_out16(&m.o[2], act, p->I, p->N, p->I))
    return MOE_ERR_CUDA;
  if (g && (!map_out16(&m.o[0], g, p->I, p->N, p->I) || !map_out16(&m.o[1], u, p->I, p->N, p->I)))
    return MOE_ERR_CUDA;
  a.m_tiles[0] = blocks(p->N, 256);
  a.n_tiles[0] = blocks(p->I, 128);
  a.tiles = static_cast<int64_t>(a.m_tiles[0]) * a.n_tiles[0];
  return launch_pair_tiles<D_GATED>(m, a, s);
}

moe_status run_down(const ffn_problem* p, const void* act, const void* wd, void* y, int64_t ldy,
                    void* ws, cudaStream_t s) {
  DArgs a = base_args(p, ws);
  a.cols = p->H;
  a.kb1 = blocks(p->I, kBK);
  bool split;
  const SplitPlan sp = ffn_plan(p, blocks(p->H, 128), static_cast<int64_t>(blocks(p->N, 256)) * blocks(p->H, 256), a.kb1, false, &split);
  if (split) {
    SMaps m{};
    a.early_w = 1;
    if (!map16(&m.a[0], wd, p->I, p->H, p->I, 128) || !map16(&m.b[0], act, p->I, p->N, p->I, sp.nt))
      return MOE_ERR_CUDA;
    a.o0 = y;
    a.ldo = ldy;
    return launch_split<D_PLAIN>(m, a, sp, blocks(p->H, 128), s);
  }
  DMaps m{};
  if (!map16(&m.a[0], act, p->I, p->N, p->I, 128) || !map16(&m.b[0], wd, p->I, p->H, p->I, 128) ||
      !map_out16(&m.o[0], y, p->H, p->N, ldy))
    return MOE_ERR_CUDA;
  a.m_tiles[0] = blocks(p->N, 256);
  a.n_tiles[0] = blocks(p->H, 256);
  a.tiles = static_cast<int64_t>(a.m_tiles[0]) * a.n_tiles[0];
  return launch_pair_tiles<D_PLAIN>(m, a, s);
}

moe_status run_dact(const ffn_problem* p, const void* dy, int64_t lddy, const void* wd, const void* g,
                    const void* u, void* dg, void* du, void* ws, cudaStream_t s) {
  DArgs a = base_args(p, ws);
  a.cols = p->I;
  a.kb1 = blocks(p->H, kBK);
  a.g = g;
  a.u = u;
  a.o0 = dg;
  a.o1 = du;
  a.ldo = p->I;
  bool split;
  const SplitPlan sp = ffn_plan(p, blocks(p->I, 128), static_cast<int64_t>(blocks(p->N, 256)) * blocks(p->I, 256), a.kb1, true, &split);
  if (split) {
    SMaps m{};
    if (!map16(&m.a[0], wd, p->I, p->H, p->I, kBK) || !map16(&m.b[0], dy, p->H, p->N, lddy, sp.nt))
      return MOE_ERR_CUDA;
    return launch_split<D_DACT>(m, a, sp, blocks(p->I, 128), s);
  }
  DMaps m{};
  if (!map16(&m.a[0], dy, p->H, p->N, lddy, 128) || !map16(&m.b[0], wd, p->I, p->H, p->I, kBK) ||
      !map_block16(&m.g, g, p->I, p->N) || !map_block16(&m.u, u, p->I, p->N) ||
      !map_block16(&m.o[0], dg, p->I, p->N) || !map_block16(&m.o[1], du, p->I, p->N))
    return MOE_ERR_CUDA;
  a.m_tiles[0] = blocks(p->N, 256);
  a.n_tiles[0] = blocks(p->I, 256);
  a.tiles = static_cast<int64_t>(a.m_tiles[0]) * a.n_tiles[0];
  return launch_pair_tiles<D_DACT>(m, a, s);
}

moe_status run_dx(const ffn_problem* p, const void* dg, const void* du, const void* wg, const void* wu,
                  void* dx, int64_t lddx, void* ws, cudaStream_t s) {
  DArgs a = base_args(p, ws);
  a.cols = p->H;
  a.kb1 = a.kb2 = blocks(p->I, kBK);
  bool split;
  const SplitPlan sp = ffn_plan(p, blocks(p->H, 128), static_cast<int64_t>(blocks(p->N, 256)) * blocks(p->H, 256), 2 * a.kb1, true, &split);
  if (split) {
    SMaps m{};
    a.early_w = 1;
    if (!map16(&m.a[0], wg, p->H, p->I, p->H, kBK) || !map16(&m.a[1], wu, p->H, p->I, p->H, kBK) ||
        !map16(&m.b[0], dg, p->I, p->N, p->I, sp.nt) || !map16(&m.b[1], du, p->I, p->N, p->I, sp.nt))
      return MOE_ERR_CUDA;
    a.o0 = dx;
    a.ldo = lddx;
    return launch_split<D_DX>(m, a, sp, blocks(p->H, 128), s);
  }
  DMaps m{};
  if (!map16(&m.a[0], dg, p->I, p->N, p->I, 128) || !map16(&m.a[1], du, p->I, p->N, p->I, 128) ||
      !map16(&m.b[0], wg, p->H, p->I, p->H, kBK) || !map16(&m.b[1], wu, p->H, p->I, p->H, kBK) ||
      !map_out16(&m.o[0], dx, p->H, p->N, lddx))
    return MOE_ERR_CUDA;
  a.m_tiles[0] = blocks(p->N, 256);
  a.n_tiles[0] = blocks(p->H, 256);
  a.tiles = static_cast<int64_t>(a.m_tiles[0]) * a.n_tiles[0];
  return launch_pair_tiles<D_DX>(m, a, s);
}

// The three weight gradients in one launch (K = tokens): together they fill
// the last wave of pairs better than one by one.
moe_status run_wgrad(const ffn_problem* p, const void* x, int64_t ldx, const void* act, const void* dy,
                     int64_t lddy, const void* dg, const void* du, void* dwg, void* dwu, void* dwd,
                     void* ws, cudaStream_t s) {
  DMaps m{};
  DArgs a = base_args(p, ws);
  a.n_probs = 3;
  a.kb1 = blocks(p->N, kBK);
  a.out_f32 = p->grad_elt == MOE_ELT_FP32;
  const int H = p->H, I = p->I;
  const int rows[3] = {I, I, H}, cols[3] = {H, H, I};
  void* out[3] = {dwg, dwu, dwd};
  if (p->N > 0 &&
      (!map16(&m.a[0], dg, I, p->N, I, kBK) || !map16(&m.a[1], du, I, p->N, I, kBK) ||
       !map16(&m.a[2], dy, H, p->N, lddy, kBK) || !map16(&m.b[0], x, H, p->N, ldx, kBK) ||
       !map16(&m.b[2], act, I, p->N, I, kBK)))
    return MOE_ERR_CUDA;
  m.b[1] = m.b[0];
  for (int i = 0; i < 3; ++i) {
    if (!(a.out_f32 ? map_out32(&m.o[i], out[i], cols[i], rows[i])
                    : map_out16(&m.o[i], out[i], cols[i], rows[i], cols[i])))
      return MOE_ERR_CUDA;
    a.w_out[i] = out[i];
    a.w_rows[i] = rows[i];
    a.w_cols[i] = cols[i];
    a.m_tiles[i] = blocks(rows[i], 256);
    a.n_tiles[i] = blocks(cols[i], 256);
    a.tiles += static_cast<int64_t>(a.m_tiles[i]) * a.n_tiles[i];
  }
  return launch_wgrad(m, a, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define FFN_TRY(expr)              \
  do {                             \
    moe_status st_ = (expr);       \
    if (st_ != MOE_OK) return st_; \
  } while (0)

extern "C" {

moe_status ffn_workspace_bytes(const ffn_problem* p, size_t* bytes) {
  FfnLayout L;
  FFN_TRY(ffn_layout(p, &L));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = L.bytes;
  return MOE_OK;
}

moe_status ffn_forward(const ffn_problem* p, const void* x, int64_t ldx, const void* w_gate,
                       const void* w_up, const void* w_down, void* g, void* u, void* act, void* y,
                       int64_t ldy, void* ws, void* stream) {
  FfnLayout L;
  FFN_TRY(ffn_layout(p, &L));
  if (!aligned(ws, 256) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16)) return MOE_ERR_INVALID_ARG;
  if ((g == nullptr) != (u == nullptr) || (g && !act)) return MOE_ERR_INVALID_ARG;
  if (L.N == 0) return MOE_OK;
  if (!mat(x, ldx, L.H) || !mat(y, ldy, L.H) || (g && (!aligned(g, 16) || !aligned(u, 16))) ||
      (act && !aligned(act, 16)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* a = act ? act : at<char>(ws, L.dg);
  FFN_TRY(run_gate_up(p, x, ldx, w_gate, w_up, g, u, a, ws, s));
  return run_down(p, a, w_down, y, ldy, ws, s);
}

moe_status ffn_backward(const ffn_problem* p, const void* x, int64_t ldx, const void* g, const void* u,
                        const void* act, const void* w_gate, const void* w_up, const void* w_down,
                        const void* dy, int64_t lddy, void* dx, int64_t lddx, void* dw_gate,
                        void* dw_up, void* dw_down, void* ws, void* stream) {
  FfnLayout L;
  FFN_TRY(ffn_layout(p, &L));
  if (!aligned(ws, 256) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(w_down, 16) || !aligned(dw_gate, 16) ||
      !aligned(dw_up, 16) || !aligned(dw_down, 16))
    return MOE_ERR_INVALID_ARG;
  if (L.N > 0 && (!mat(x, ldx, L.H) || !mat(dy, lddy, L.H) || !mat(dx, lddx, L.H) || !aligned(g, 16) ||
                  !aligned(u, 16) || !aligned(act, 16)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void *dg = at<char>(ws, L.dg), *du = at<char>(ws, L.du);
  auto wgrad = [&] { return run_wgrad(p, x, ldx, act, dy, lddy, dg, du, dw_gate, dw_up, dw_down, ws, s); };
  if (L.N == 0) return wgrad();
  FFN_TRY(run_dact(p, dy, lddy, w_down, g, u, dg, du, ws, s));
  // dX and the weight gradients need dG and dU and not each other. The latter read
  // x and dy: before dX where it is written over one of them (one object whose dx
  // is handed on as the next layer's dy).
  const bool late = overlap(dx, lddx, L.H, dy, lddy, L.H, L.N) || overlap(dx, lddx, L.H, x, ldx, L.H, L.N);
  if (late) FFN_TRY(wgrad());
  FFN_TRY(run_dx(p, dg, du, w_gate, w_up, dx, lddx, ws, s));
  return late ? MOE_OK : wgrad();
}

moe_status ffn_get_device_error(const ffn_problem* p, const void* ws, int32_t* code_out, void* stream) {
  FfnLayout L;
  FFN_TRY(ffn_layout(p, &L));
  if (!aligned(ws, 256) || !code_out) return MOE_ERR_INVALID_ARG;
  return cuda_status(
      cudaMemcpyAsync(code_out, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, static_cast<cudaStream_t>(stream)));
}

moe_status ffn_clear_device_error(const ffn_problem* p, void* ws, void* stream) {
  FfnLayout L;
  FFN_TRY(ffn_layout(p, &L));
  if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  return cuda_status(cudaMemsetAsync(ws, 0, sizeof(int32_t), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

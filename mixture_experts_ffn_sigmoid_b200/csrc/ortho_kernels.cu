// Newton-Schulz orthogonalisation of a stack of matrices, bare or as the Muon
// optimiser's update of momentum and weights: what follows the block's weight
// gradients (expert stacks [E][f][d]) in training.
//
// For every matrix U of the stack (transposed first if it has more rows than
// columns: m <= n below), with coefficients (a, b, c) per step:
//
//   X = U / (|U|_F + eps)
//   repeat:  A = X X^T,  B = a I + b A + c A^2,  X = B X
//
// Each step applies p(s) = a s + b s^3 + c s^5 to the singular values, which
// approach 1; the singular vectors stay. Muon: M = mu M + G, U = G + mu M
// (Nesterov) or M, W = (1 - lr decay) W - lr scale X.
//
// What bounds it: the tensor cores. A step is 2 m^2 n + 2 m^3 + 2 m^2 n
// operations; A and A^2 are symmetric, so the tiles above the diagonal are
// not computed but written from those below (where SMs would idle otherwise, they
// are computed): 3 m^2 n + m^3.
//
// Precision. The operands are fp16, accumulated in fp32 in TMEM, and rounded
// once per product. X starts with norm 1 and its singular values stay in a
// range that the host checks for the given coefficients, so fp16's range
// suffices where bf16's is not needed and its three more bits count: five
// steps end 1.2e-3 (2-norm) from fp64 for a spread spectrum, bf16 operands end
// 1e-2 from it. X, A and B are stored times 64, so that small entries (1e-4
// and below in wide matrices) stay above fp16's subnormals; powers of two cost
// nothing. a I is folded into B. The diagonal of B, near 0.7 where the values
// have converged, is its largest part, and over few rows its roundings do not
// average out: for m <= 128 what fp16 leaves of it is kept in fp32 and its
// product with X added by the epilogue (on chip A's as well). Without that,
// matrices of 8 to 20 rows ended up to 2.8e-3 from fp64, with it 1.2e-3 (in a
// fp64 simulation of the roundings, 150 random shapes of up to 100 x 2500).
//
// Kernels: one pass over U for its norm (and the momentum), one that writes X
// in fp16 (transposing through shared memory), then three GEMM launches a step
// of one persistent kernel on CTA pairs: 256 x 256 tiles by M = 256, N = 256
// cta_group::2 MMAs, each CTA staging 128 rows of P and 128 of Q (32 KB per 64
// of K, six stages), two accumulators in TMEM so that the epilogue of a tile
// runs under the next one's MMAs. Where such tiles would leave SMs idle, a CTA
// takes a tile of 128 x 128 by itself. X is the MN-major operand of B X, so it is
// stored once. The last step's epilogue writes the result or the weights.
//
// Measured, five steps: 8 x 2048 x 7168 as a Muon step in bf16 3.6 to 4.3 ms with
// the power cap (3.95 TFLOP: 0.92 to 1.1 PFLOP/s; launched one by one the products
// take 207, 76 and 366 us for A, B and X, the last one 401, at 1.31, 1.01 and 1.31
// PFLOP/s of the tiles they compute, the two first passes 318 us for their 2.1 GB:
// 3.6 ms in all); 2 x 14336 x 4096 6.9 to 7.4 ms (1.1 PFLOP/s). Middling matrices
// are bound by their 15 dependent products: 4 of 256 x 384 take 94 us, of which a
// product's loads, its way out of TMEM and the stores' way to the next one are
// 1.5 to 2 us each. One launch for all
// products with waits across the grid in between took longer (122 -> 147 us).
//
// Matrices of up to 128 x 512 (either way round) stay in shared memory from the
// first read to the last write: one launch, one CTA a matrix (ns_chip_kernel).
// Their products are too short for launches between them: 8 matrices of 256 x
// 128 took 97 us in 17 launches, 45 here (2.9 us a product: MMAs, the trip
// through registers and two barriers).
#include <cuda_fp16.h>

#include "umma_common.cuh"

namespace moe {
namespace {

constexpr int NS_BK = 64;
constexpr int NS_HALF = 128;                       // rows of a tile per CTA of the pair
constexpr int NS_OP_BYTES = NS_HALF * NS_BK * 2;   // one operand's share of a stage
constexpr int NS_STAGE_BYTES = 2 * NS_OP_BYTES;
constexpr int NS_STAGES = 6;
constexpr int NS_EPI_WARPS = 8;
constexpr int NS_THREADS = 32 * (2 + NS_EPI_WARPS);
constexpr int NS_TMEM_COLS = 512;
constexpr int NS_SMEM = 1024 + 1024 + NS_STAGES * NS_STAGE_BYTES;
constexpr float kNsScale = 64.0f;                  // X, A and B are stored times this

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// TMA into this CTA's shared memory, completing on the pair leader's barrier.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (M = 256 over the pair) (+)= P Q^T, fp16 operands.
__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void ns_load(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, uint32_t bar) {
  if (PAIR) {
    tma_load_3d_pair(dst, tm, c0, c1, c2, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  }
}
template <bool PAIR>
__device__ __forceinline__ void ns_commit(uint64_t* bar, uint16_t mask) {
  if (PAIR) umma_commit_pair(smem_u32(bar), mask);
  else umma_commit(smem_u32(bar));
}

enum NsMode { kNsGram = 0, kNsPoly = 1, kNsApply = 2, kNsLast = 3 };

struct NsGemmParams {
  int n_mat, m, n;          // X is [n_mat][m][n], m <= n
  int ld_x, ld_a;           // row pitches (elements, multiples of 8) of X and of A, B
  float a, b, c;            // kNsPoly
  const __half* a_in;       // kNsPoly: A, read again in the epilogue
  __half* out;              // kNsGram: A, kNsPoly: B, kNsApply: the next X
  const __half* x_in;       // kNsApply, kNsLast: X, read again where diag is set
  float* diag;              // what fp16 left of B's diagonal, [n_mat][m], or null
  int full;                 // kNsGram, kNsPoly: all tiles, none mirrored
  // kNsLast: the caller's matrices, [n_mat][rows][cols]; tall: out = X^T.
  int tall, rows, cols;
  __nv_bfloat16* o;         // result, or null:
  void* weight;             // W = keep W - step X
  int weight_f32;
  float keep, step;
  uint32_t* err;
  long long timeout_ns;
};

struct NsTile {
  int mat, i0, j0;          // first row and column of D
};

template <int MODE, int TILE>
__device__ __forceinline__ NsTile ns_tile(const NsGemmParams& p, int tile) {
  const int tm = ceil_div(p.m, TILE);
  NsTile t;
  if ((MODE == kNsGram || MODE == kNsPoly) && !p.full) {   // tiles on and below the diagonal
    const int per = tm * (tm + 1) / 2;
    t.mat = tile / per;
    const int r = tile - t.mat * per;
    int i = (int)((sqrtf(8.0f * r + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > r) --i;
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    t.i0 = i * TILE;
    t.j0 = (r - i * (i + 1) / 2) * TILE;
  } else {                                        // rows fastest: neighbours share X's columns
    const int per = tm * (MODE == kNsGram || MODE == kNsPoly ? tm : ceil_div(p.n, TILE));
    t.mat = tile / per;
    const int r = tile - t.mat * per;
    t.j0 = (r / tm) * TILE;
    t.i0 = (r % tm) * TILE;
  }
  return t;
}

__device__ __forceinline__ uint4 pack_half8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// v[at], without indexing registers.
template <int N>
__device__ __forceinline__ float ns_pick(const float (&v)[N], int at) {
  float x = v[0];
#pragma unroll
  for (int e = 1; e < N; ++e) x = e == at ? v[e] : x;
  return x;
}

// Eight columns of a row of the last product into the caller's matrices.
__device__ __forceinline__ void ns_store_last(const NsGemmParams& p, int mat, int i, int j, const float (&v)[8]) {
  const size_t base = (size_t)mat * p.rows * p.cols;
  const bool vec = !p.tall && p.cols % 8 == 0;
  const int nj = min(8, p.n - j);
  if (p.o) {
    if (vec) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.o + base + (size_t)i * p.cols + j) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < nj)
          p.o[base + (p.tall ? (size_t)(j + e) * p.cols + i : (size_t)i * p.cols + j + e)] = __float2bfloat16_rn(v[e]);
    }
    return;
  }
  if (p.weight_f32) {
    float* w = static_cast<float*>(p.weight) + base;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nj) {
        float& x = w[p.tall ? (size_t)(j + e) * p.cols + i : (size_t)i * p.cols + j + e];
        x = p.keep * x - p.step * v[e];
      }
    return;
  }
  __nv_bfloat16* w = static_cast<__nv_bfloat16*>(p.weight) + base;
  if (vec) {
    uint4* at = reinterpret_cast<uint4*>(w + (size_t)i * p.cols + j);
    const uint4 old = *at;
    const uint32_t in[4] = {old.x, old.y, old.z, old.w};
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float lo = __uint_as_float(in[e] << 16), hi = __uint_as_float(in[e] & 0xffff0000u);
      const __nv_bfloat162 h =
          __floats2bfloat162_rn(p.keep * lo - p.step * v[2 * e], p.keep * hi - p.step * v[2 * e + 1]);
      out[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *at = make_uint4(out[0], out[1], out[2], out[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < nj) {
      __nv_bfloat16& x = w[p.tall ? (size_t)(j + e) * p.cols + i : (size_t)i * p.cols + j + e];
      x = __float2bfloat16_rn(p.keep * __bfloat162float(x) - p.step * v[e]);
    }
}

// D = P Q^T (kNsGram: P = Q = X; kNsPoly: P = Q = A) or D = P Q with Q read
// MN-major (kNsApply, kNsLast: P = B, Q = X). PAIR: a CTA pair per tile of 256 x
// 256, else one CTA per tile of 128 x 128.
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(NS_THREADS, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const NsGemmParams p) {
  constexpr bool SYM = MODE == kNsGram || MODE == kNsPoly;
  constexpr int TILE = PAIR ? 2 * NS_HALF : NS_HALF;
  constexpr uint32_t CTAS = PAIR ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty_bar = full_bar + NS_STAGES;
  uint64_t* accf_bar = empty_bar + NS_STAGES;
  uint64_t* acce_bar = accf_bar + 2;
  uint64_t* drain_bar = acce_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  uint8_t* ring = smem + 1024;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const bool leader = rank == 0;

  // The next launch may take the SMs that this one leaves idle and set up there.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS_STAGES; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf_bar[i]), 1);
      mbar_init(smem_u32(&acce_bar[i]), CTAS * NS_EPI_WARPS);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0u;
    fence_mbar_init();
    tmap_prefetch(&tmP);
    tmap_prefetch(&tmQ);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), NS_TMEM_COLS);
    } else {
      tmem_alloc(smem_u32(tmem_slot), NS_TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();   // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // What the launch before wrote is read only from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int tm = ceil_div(p.m, TILE);
  const int per = SYM ? (p.full ? tm * tm : tm * (tm + 1) / 2) : tm * ceil_div(p.n, TILE);
  const int total = p.n_mat * per;
  const int group = blockIdx.x / CTAS, ngroups = gridDim.x / CTAS;
  const int nk = ceil_div(MODE == kNsGram ? p.n : p.m, NS_BK);

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    bool ok = true;
    for (int tile = group; tile < total && ok; tile += ngroups) {
      const NsTile t = ns_tile<MODE, TILE>(p, tile);
      const int pi = t.i0 + (int)rank * NS_HALF, qj = t.j0 + (int)rank * NS_HALF;
      for (int kb = 0; kb < nk; ++kb) {
        if (!wait_bounded(smem_u32(&empty_bar[stage]), phase ^ 1u, abort_flag, p.err, p.timeout_ns, true)) {
          ok = false;
          break;
        }
        const uint32_t fb_local = smem_u32(&full_bar[stage]);
        const uint32_t fb = PAIR ? map_to_cta(fb_local, 0) : fb_local;
        const uint32_t sp = smem_u32(ring + stage * NS_STAGE_BYTES), sq = sp + NS_OP_BYTES;
        if (leader) mbar_expect_tx(fb_local, CTAS * NS_STAGE_BYTES);   // both CTAs' copies
        ns_load<PAIR>(sp, &tmP, kb * NS_BK, pi, t.mat, fb);
        if (SYM) {
          ns_load<PAIR>(sq, &tmQ, kb * NS_BK, qj, t.mat, fb);
        } else {
          ns_load<PAIR>(sq, &tmQ, qj, kb * NS_BK, t.mat, fb);
          ns_load<PAIR>(sq + MN_BOX_BYTES, &tmQ, qj + 64, kb * NS_BK, t.mat, fb);
        }
        ++issued;
        if (++stage == NS_STAGES) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && leader) {
      // Giving up: the copies under way land before shared memory is freed.
      const uint32_t n = issued < NS_STAGES ? issued : NS_STAGES;
      for (uint32_t k = issued - n; k < issued; ++k)
        wait_bounded(smem_u32(&full_bar[k % NS_STAGES]), (k / NS_STAGES) & 1u, abort_flag, p.err, p.timeout_ns, false);
    }
  } else if (warp == 1 && lane == 0 && leader) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool issued = false, ok = true;
    // fp16 x fp16 -> fp32, M = N = TILE; bit 16: Q is MN-major.
    const uint32_t idesc = (1u << 4) | ((uint32_t)(TILE >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24) |
                           (SYM ? 0u : 1u << 16);
    for (int tile = group; tile < total && ok; tile += ngroups) {
      if (!wait_bounded(smem_u32(&acce_bar[acc]), acc_phase ^ 1u, abort_flag, p.err, p.timeout_ns, true)) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * TILE);
      for (int kb = 0; kb < nk; ++kb) {
        if (!wait_bounded(smem_u32(&full_bar[stage]), phase, abort_flag, p.err, p.timeout_ns, true)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sp = smem_u32(ring + stage * NS_STAGE_BYTES);
        const uint64_t pd = sw128_desc(sp);
        const uint64_t qd = SYM ? sw128_desc(sp + NS_OP_BYTES) : sw128_mn_desc(sp + NS_OP_BYTES);
#pragma unroll
        for (int kk = 0; kk < NS_BK / 16; ++kk) {
          const uint64_t kp = (uint64_t)((kk * 32) >> 4);             // 16 k further along a row
          const uint64_t kq = SYM ? kp : (uint64_t)((kk * 2 * 1024) >> 4);
          if (PAIR) umma_f16_pair(d, pd + kp, qd + kq, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          else umma_bf16(d, pd + kp, qd + kq, idesc, (kb > 0 || kk > 0) ? 1u : 0u);   // kind::f16: idesc says fp16
        }
        issued = true;
        ns_commit<PAIR>(&empty_bar[stage], 0x3);
        if (++stage == NS_STAGES) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      ns_commit<PAIR>(&accf_bar[acc], 0x3);
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (issued) {                 // every MMA completes before TMEM is freed
      ns_commit<PAIR>(drain_bar, 0x1);
      wait_bounded(smem_u32(drain_bar), 0u, abort_flag, p.err, p.timeout_ns, false);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, cbeg = ((warp - 2) >> 2) * (TILE / 2);   // TMEM lane quarter, column half
    const uint32_t acce0 = PAIR ? map_to_cta(smem_u32(&acce_bar[0]), 0) : smem_u32(&acce_bar[0]);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = group; tile < total; tile += ngroups) {
      const NsTile t = ns_tile<MODE, TILE>(p, tile);
      const int i = t.i0 + (int)rank * NS_HALF + q * 32 + lane;
      const int j0 = t.j0 + cbeg;
      const int ncol = SYM ? p.m : p.n;
      // One outcome for the warp, whose lanes load TMEM together.
      if (!__all_sync(0xffffffffu, wait_bounded(smem_u32(&accf_bar[acc]), acc_phase, abort_flag, p.err, p.timeout_ns, true)))
        break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * TILE + cbeg);
      for (int c0 = 0; c0 < TILE / 2 && j0 + c0 < ncol; c0 += 32) {
        uint32_t r[2][16];
        tmem_ld16x2_wait(taddr + c0, taddr + c0 + 16, r[0], r[1]);
        const int j = j0 + c0;
        const bool row_ok = i < p.m;
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e >> 4][e & 15]);
        if (MODE == kNsPoly) {
          const __half* ap = p.a_in + ((size_t)t.mat * p.m + i) * p.ld_a + j;
          uint4 av[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            av[k] = row_ok && j + 8 * k < ncol ? *reinterpret_cast<const uint4*>(ap + 8 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const __half2 h = reinterpret_cast<const __half2*>(av)[e >> 1];
            float x = p.b * ((e & 1) ? __high2float(h) : __low2float(h)) + (p.c / kNsScale) * v[e];
            if (j + e == i) x += p.a * kNsScale;
            v[e] = x;
          }
          if (p.diag && row_ok && i >= j && i < j + 32) {
            const float x = ns_pick(v, i - j);
            p.diag[(size_t)t.mat * p.m + i] = x - __half2float(__float2half_rn(x));
          }
        } else {
          if (!SYM && p.diag && row_ok) {
            const float rest = p.diag[(size_t)t.mat * p.m + i];
            const __half* xp = p.x_in + ((size_t)t.mat * p.m + i) * p.ld_x + j;
            uint4 xv[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              xv[k] = j + 8 * k < ncol ? *reinterpret_cast<const uint4*>(xp + 8 * k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const __half2 h = reinterpret_cast<const __half2*>(xv)[e >> 1];
              v[e] = fmaf(rest, (e & 1) ? __high2float(h) : __low2float(h), v[e]);
            }
          }
          const float f = MODE == kNsLast ? 1.0f / (kNsScale * kNsScale) : 1.0f / kNsScale;
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] *= f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!row_ok || j + 8 * k >= ncol) break;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = v[8 * k + e];
          if (MODE == kNsLast) {
            ns_store_last(p, t.mat, i, j + 8 * k, w);
          } else {   // a row's last eight may run into its padding
            const int ld = SYM ? p.ld_a : p.ld_x;
            *reinterpret_cast<uint4*>(p.out + ((size_t)t.mat * p.m + i) * ld + j + 8 * k) = pack_half8(w);
          }
        }
        if (SYM && !p.full && t.i0 != t.j0 && row_ok) {   // the tile above the diagonal: consecutive lanes, consecutive columns
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (j + e < ncol) p.out[((size_t)t.mat * p.m + j + e) * p.ld_a + i] = __float2half_rn(v[e]);
        }
        __syncwarp();             // the next TMEM load takes the whole warp
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(acce0 + (uint32_t)acc * 8u);
        else mbar_arrive(acce0 + (uint32_t)acc * 8u);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync_all();   // the peer's shared memory and TMEM stay live until here
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, NS_TMEM_COLS);
    else tmem_dealloc(tmem_base, NS_TMEM_COLS);
  }
}

// ------------------------------------------------------- norm and first X
constexpr int NS_NORM_THREADS = 256;
constexpr int NS_NORM_MAX = 256;                   // blocks a matrix

template <typename T> __device__ __forceinline__ void ns_load8(const T* p, float (&f)[8]);
template <> __device__ __forceinline__ void ns_load8<float>(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <> __device__ __forceinline__ void ns_load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Sum of squares of U per matrix and block (fp32), with the momentum updated
// on the way. A matrix is one run of size = rows * cols elements; `vec` where
// every eight of them are aligned. Block (0, 0) clears the error word.
template <typename T, bool MOM>
__global__ void __launch_bounds__(NS_NORM_THREADS) ns_norm_kernel(const T* __restrict__ g, float* __restrict__ mom,
                                                                  float mu, int nesterov, long long size, int vec,
                                                                  float* __restrict__ partial, uint32_t* err) {
  __shared__ float red[NS_NORM_THREADS / 32];
  if (err && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *err = 0u;
  const size_t base = (size_t)blockIdx.y * size;
  const long long step = (long long)gridDim.x * NS_NORM_THREADS;
  float s = 0.0f;
  auto one = [&](float gv, float* mp) {
    float u = gv;
    if (MOM) {
      const float m = fmaf(mu, *mp, gv);
      *mp = m;
      u = nesterov ? fmaf(mu, m, gv) : m;
    }
    s = fmaf(u, u, s);
  };
  if (vec) {
    for (long long i = ((long long)blockIdx.x * NS_NORM_THREADS + threadIdx.x); i < size / 8; i += step) {
      float f[8], m[8];
      ns_load8(g + base + i * 8, f);
      if (MOM) ns_load8(mom + base + i * 8, m);
#pragma unroll
      for (int e = 0; e < 8; ++e) one(f[e], &m[e]);
      if (MOM) {
        float4* mp = reinterpret_cast<float4*>(mom + base + i * 8);
        mp[0] = make_float4(m[0], m[1], m[2], m[3]);
        mp[1] = make_float4(m[4], m[5], m[6], m[7]);
      }
    }
  } else {
    for (long long i = (long long)blockIdx.x * NS_NORM_THREADS + threadIdx.x; i < size; i += step) {
      float m = MOM ? mom[base + i] : 0.0f;
      one(to_f32(g[base + i]), &m);
      if (MOM) mom[base + i] = m;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0f;
    for (int w = 0; w < NS_NORM_THREADS / 32; ++w) s += red[w];
    partial[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
  }
}

// X = 64 U / (|U| + eps) in fp16, [m][ld]; a block takes 64 x 64 elements of U.
template <typename T, bool MOM>
__global__ void __launch_bounds__(256) ns_init_kernel(const T* __restrict__ g, const float* __restrict__ mom, float mu,
                                                      int nesterov, int rows, int cols, int vec, int tall, float eps,
                                                      const float* __restrict__ partial, int n_partial, int col_tiles,
                                                      __half* __restrict__ x, int ld) {
  __shared__ float red[8];
  __shared__ __half tile[64][72];
  const int tid = threadIdx.x, mat = blockIdx.y;
  float s = 0.0f;
  for (int i = tid; i < n_partial; i += 256) s += partial[(size_t)mat * n_partial + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((tid & 31) == 0) red[tid >> 5] = s;
  __syncthreads();
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += red[w];
  const float scale = kNsScale / (sqrtf(s) + eps);
  const int r0 = (blockIdx.x / col_tiles) * 64, c0 = (blockIdx.x % col_tiles) * 64;
  const size_t base = (size_t)mat * rows * cols;
  __half* xm = x + (size_t)mat * (tall ? cols : rows) * ld;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = r0 + k * 32 + tid / 8, c = c0 + (tid % 8) * 8;
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (r < rows && c < cols) {
      const size_t at = base + (size_t)r * cols + c;
      if (vec) {
        if (!MOM || nesterov) ns_load8(g + at, f);
        if (MOM) {
          float m[8];
          ns_load8(mom + at, m);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = nesterov ? fmaf(mu, m[e], f[e]) : m[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < cols) {
            f[e] = to_f32(g[at + e]);
            if (MOM) f[e] = nesterov ? fmaf(mu, mom[at + e], f[e]) : mom[at + e];
          }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    const uint4 h = pack_half8(f);
    if (!tall) {
      if (r < rows && c < cols) *reinterpret_cast<uint4*>(xm + (size_t)r * ld + c) = h;
    } else {
      *reinterpret_cast<uint4*>(&tile[k * 32 + tid / 8][(tid % 8) * 8]) = h;
    }
  }
  if (!tall) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = k * 32 + tid / 8, r = (tid % 8) * 8;    // row c of X, eight of its columns
    if (c0 + c >= cols || r0 + r >= rows) continue;
    __align__(16) __half h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = tile[r + e][c];
    *reinterpret_cast<uint4*>(xm + (size_t)(c0 + c) * ld + r0 + r) = *reinterpret_cast<const uint4*>(h);
  }
}

// ------------------------------------------------- small matrices, on chip
constexpr int NSC_THREADS = 512;
constexpr int NSC_M = 128, NSC_N = 512;
constexpr int NSC_BLOCK = NSC_M * 128;             // 64 columns of 128 rows
constexpr int NSC_SMEM = 1024 + (NSC_N / 64 + 2 * (NSC_M / 64)) * NSC_BLOCK;

// Element (r, c) of a matrix in blocks of 64 columns x 128 rows, 128-byte
// swizzle: K-major as it stands, and MN-major with its columns as N.
__device__ __forceinline__ uint32_t nsc_at(int r, int c) {
  return (uint32_t)((c >> 6) * NSC_BLOCK + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) * 16) + (c & 7) * 2);
}
// MN-major operand whose 64-column groups are a block apart.
__device__ __forceinline__ uint64_t nsc_mn_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(NSC_BLOCK >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

struct NsChipParams {
  NsGemmParams g;
  const void* grad;
  float* mom;
  float mu, eps;
  int nesterov, steps, clear_err;
  float coeffs[3 * 64];
};

// One matrix per CTA: X [128][64 k] stays in shared memory, A and B beside it;
// each product's accumulator (128 rows, up to 512 columns of TMEM) goes through
// registers back into the operand it becomes. Thread 0 issues the MMAs, all 16
// warps move the results: lane quarter warp % 4, every fourth 32 columns.
template <typename T, bool MOM>
__global__ void __launch_bounds__(NSC_THREADS, 1) ns_chip_kernel(const __grid_constant__ NsChipParams cp) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float red[NSC_THREADS / 32];
  __shared__ __align__(16) float rest_a[NSC_M], rest_b[NSC_M];         // what fp16 left of the diagonals of A and B
  __shared__ uint64_t done_bar;
  __shared__ uint32_t tmem_slot, abort_word;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const NsGemmParams& p = cp.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mat = blockIdx.x;
  const int nb = ceil_div(p.n, 64);
  uint8_t *xs = smem, *as = smem + (NSC_N / 64) * NSC_BLOCK, *bs = as + (NSC_M / 64) * NSC_BLOCK;
  volatile uint32_t* abort_flag = &abort_word;
  if (tid == 0) {
    mbar_init(smem_u32(&done_bar), 1);
    abort_word = 0u;
    if (cp.clear_err && mat == 0) *p.err = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  if (tid < NSC_M) rest_a[tid] = 0.0f;
  for (int i = tid; i < (nb + 2 * (NSC_M / 64)) * (NSC_BLOCK / 16); i += NSC_THREADS)   // rows and columns past the matrix
    reinterpret_cast<uint4*>(i < nb * (NSC_BLOCK / 16) ? xs : as - nb * NSC_BLOCK)[i] = make_uint4(0, 0, 0, 0);

  // ------------------------------------------------------ norm, then X
  const size_t size = (size_t)p.rows * p.cols, base = (size_t)mat * size;
  const T* grad = static_cast<const T*>(cp.grad) + base;
  float* mom = MOM ? cp.mom + base : nullptr;
  const bool vec = p.cols % 8 == 0;
  const int per_row = ceil_div(p.cols, 8), groups = p.rows * per_row;
  // Eight columns of a row of U; `first`: the momentum moves on.
  auto load_u = [&](int i, bool first, float (&f)[8], int& r, int& c) {
    r = i / per_row;
    c = (i - r * per_row) * 8;
    const size_t at = (size_t)r * p.cols + c;
    const int n = min(8, p.cols - c);
    float m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = m[e] = 0.0f;
    if (vec) {
      ns_load8(grad + at, f);
      if (MOM) ns_load8(mom + at, m);
    } else {
      for (int e = 0; e < n; ++e) {
        f[e] = to_f32(grad[at + e]);
        if (MOM) m[e] = mom[at + e];
      }
    }
    if (MOM) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (first) m[e] = fmaf(cp.mu, m[e], f[e]);
        f[e] = cp.nesterov ? fmaf(cp.mu, m[e], f[e]) : m[e];
      }
      if (first) {
        if (vec) {
          reinterpret_cast<float4*>(mom + at)[0] = make_float4(m[0], m[1], m[2], m[3]);
          reinterpret_cast<float4*>(mom + at)[1] = make_float4(m[4], m[5], m[6], m[7]);
        } else {
          for (int e = 0; e < n; ++e) mom[at + e] = m[e];
        }
      }
    }
  };
  float s = 0.0f;
#pragma unroll 2
  for (int i = tid; i < groups; i += NSC_THREADS) {
    float f[8];
    int r, c;
    load_u(i, true, f, r, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(f[e], f[e], s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < NSC_THREADS / 32; ++w) s += red[w];
  const float scale = kNsScale / (sqrtf(s) + cp.eps);
#pragma unroll 2
  for (int i = tid; i < groups; i += NSC_THREADS) {      // each thread what it wrote itself
    float f[8];
    int r, c;
    load_u(i, false, f, r, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    if (p.tall) {
      for (int e = 0; e < 8 && c + e < p.cols; ++e)
        *reinterpret_cast<__half*>(xs + nsc_at(c + e, r)) = __float2half_rn(f[e]);
    } else {
      *reinterpret_cast<uint4*>(xs + nsc_at(r, c)) = pack_half8(f);
    }
  }

  // ---------------------------------------------------------- products
  const uint32_t xa = smem_u32(xs), aa = smem_u32(as), ba = smem_u32(bs);
  const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;
  const bool row_ok = row < p.m;
  const int k16 = ceil_div(p.m, 16);                     // steps of 16 along m
  uint32_t phase = 0;
  bool ok = true;
  uint32_t taddr = 0, tmem_base = 0;
  // Operands written by every thread -> the tensor core -> the accumulator.
  auto multiply = [&](auto issue) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem_base = tmem_slot;
    taddr = tmem_base + ((uint32_t)(q * 32) << 16);
    if (tid == 0) {
      issue();
      umma_commit(smem_u32(&done_bar));
    }
    ok = wait_bounded(smem_u32(&done_bar), phase, abort_flag, p.err, p.timeout_ns, true);
    phase ^= 1u;
    ok = __syncthreads_and(ok);
    tc_fence_after();
  };
  // fp16 operands, M = 128; the square products take N = 128.
  const uint32_t idesc0 = (1u << 4) | ((uint32_t)(NSC_M >> 4) << 24);
  const uint32_t idesc_sq = idesc0 | ((uint32_t)(NSC_M >> 3) << 17);
  for (int k = 0; k < cp.steps && ok; ++k) {
    const float ca = cp.coeffs[3 * k] * kNsScale, cb = cp.coeffs[3 * k + 1], cc = cp.coeffs[3 * k + 2] / kNsScale;
    multiply([&]() {                                     // A = X X^T
      for (int b = 0; b < nb; ++b)
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = sw128_desc(xa + b * NSC_BLOCK) + (uint64_t)((kk * 32) >> 4);
          umma_bf16(tmem_base, d, d, idesc_sq, b > 0 || kk > 0);
        }
    });
    if (!ok) break;
    for (int c0 = part * 32; c0 < p.m; c0 += 128) {
      uint32_t r[2][16];
      tmem_ld16x2_wait(taddr + c0, taddr + c0 + 16, r[0], r[1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[j >> 1][(j & 1) * 8 + e]) * (1.0f / kNsScale);
        if (c0 + 8 * j == (row & ~7)) {                  // the diagonal
          const float x = ns_pick(v, row & 7);
          rest_a[row] = x - __half2float(__float2half_rn(x));
        }
        *reinterpret_cast<uint4*>(as + nsc_at(row, c0 + 8 * j)) = pack_half8(v);
      }
    }
    multiply([&]() {                                     // B = a I + b A + c A^2
      for (int kk = 0; kk < k16; ++kk) {
        const uint64_t d = sw128_desc(aa + (kk >> 2) * NSC_BLOCK) + (uint64_t)(((kk & 3) * 32) >> 4);
        umma_bf16(tmem_base, d, d, idesc_sq, kk > 0);
      }
    });
    if (!ok) break;
    const float rest = rest_a[row], cr = fmaf(cc, rest, cb);
    for (int c0 = part * 32; c0 < p.m; c0 += 128) {
      uint32_t r[2][16];
      tmem_ld16x2_wait(taddr + c0, taddr + c0 + 16, r[0], r[1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 old = *reinterpret_cast<const uint4*>(as + nsc_at(row, c0 + 8 * j));
        const __half2* h = reinterpret_cast<const __half2*>(&old);
        // (A + D)^2 = A A + D A + A D + ..., D the diagonal's rest
        const float4 d0 = *reinterpret_cast<const float4*>(&rest_a[c0 + 8 * j]);
        const float4 d1 = *reinterpret_cast<const float4*>(&rest_a[c0 + 8 * j + 4]);
        const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = (e & 1) ? __high2float(h[e >> 1]) : __low2float(h[e >> 1]);
          v[e] = fmaf(fmaf(cc, d[e], cr), x, cc * __uint_as_float(r[j >> 1][(j & 1) * 8 + e]));
        }
        if (c0 + 8 * j == (row & ~7)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += e == (row & 7) ? fmaf(cb, rest, ca) : 0.0f;
          const float x = ns_pick(v, row & 7);
          rest_b[row] = x - __half2float(__float2half_rn(x));
        }
        *reinterpret_cast<uint4*>(bs + nsc_at(row, c0 + 8 * j)) = pack_half8(v);
      }
    }
    multiply([&]() {                                     // X = B X
      for (int j0 = 0; j0 < p.n; j0 += 256) {
        const int n = min(256, ceil_div(p.n - j0, 16) * 16);
        const uint32_t idesc = idesc0 | ((uint32_t)(n >> 3) << 17) | (1u << 16);   // X is MN-major
        for (int kk = 0; kk < k16; ++kk)
          umma_bf16(tmem_base + j0, sw128_desc(ba + (kk >> 2) * NSC_BLOCK) + (uint64_t)(((kk & 3) * 32) >> 4),
                    nsc_mn_desc(xa + (j0 >> 6) * NSC_BLOCK) + (uint64_t)((kk * 2 * 1024) >> 4), idesc, kk > 0);
      }
    });
    if (!ok) break;
    const bool last = k + 1 == cp.steps;
    const float more = row < p.m ? rest_b[row] : 0.0f;
    for (int c0 = part * 32; c0 < p.n; c0 += 128) {
      uint32_t r[2][16];
      tmem_ld16x2_wait(taddr + c0, taddr + c0 + 16, r[0], r[1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c0 + 8 * j >= p.n) break;
        float v[8];
        const float f = last ? 1.0f / (kNsScale * kNsScale) : 1.0f / kNsScale;
        const uint4 old = *reinterpret_cast<const uint4*>(xs + nsc_at(row, c0 + 8 * j));
#pragma unroll
        for (int e = 0; e < 8; ++e) {   // columns past n were not computed
          const __half2 h = reinterpret_cast<const __half2*>(&old)[e >> 1];
          const float x = (e & 1) ? __high2float(h) : __low2float(h);
          v[e] = fmaf(more, x, __uint_as_float(r[j >> 1][(j & 1) * 8 + e])) * f;
          if (c0 + 8 * j + 8 > p.n && c0 + 8 * j + e >= p.n) v[e] = 0.0f;
        }
        if (!last) *reinterpret_cast<uint4*>(xs + nsc_at(row, c0 + 8 * j)) = pack_half8(v);
        else if (row_ok) ns_store_last(p, mat, row, c0 + 8 * j, v);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// fp16 [outer][rows][cols] with a row pitch, 128-byte swizzle, box 64 x box_rows.
bool make_ns_tmap(CUtensorMap* tm, const void* base, long long cols, long long rows, long long outer, long long ld,
                  int box_rows) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), (cuuint64_t)(rows * ld * 2)};
  cuuint32_t box[3] = {(cuuint32_t)NS_BK, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
long long ns_tiles(const NsGemmParams& p, int tile) {
  const long long tm = ceil_div(p.m, tile);
  if (MODE == kNsGram || MODE == kNsPoly) return p.n_mat * (p.full ? tm * tm : tm * (tm + 1) / 2);
  return p.n_mat * tm * ceil_div(p.n, tile);
}

template <int MODE, bool PAIR>
cudaError_t launch_ns_tiles(const CUtensorMap& tp, const CUtensorMap& tq, NsGemmParams p, int num_sms,
                            cudaStream_t s) {
  const cudaError_t e = allow_max_smem<ns_gemm_kernel<MODE, PAIR>>();
  if (e != cudaSuccess) return e;
  constexpr int TILE = PAIR ? 2 * NS_HALF : NS_HALF;
  const int ctas = PAIR ? 2 : 1, slots = num_sms / ctas;
  long long tiles = ns_tiles<MODE>(p, TILE);
  if (MODE == kNsGram || MODE == kNsPoly) {
    // Where all tiles take no more rounds than those on and below the diagonal,
    // nothing is mirrored: the stores of a tile's transpose (2 bytes a lane) are
    // a quarter of a short product. 4 of 256 x 384 122 -> 94 us, 2 of 768 x 768
    // 163 -> 136.
    p.full = 1;
    const long long all = ns_tiles<MODE>(p, TILE);
    if (ceil_div_ll(all, slots) <= ceil_div_ll(tiles, slots)) tiles = all;
    else p.full = 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * (unsigned)(tiles < slots ? tiles : slots));
  cfg.blockDim = dim3(NS_THREADS);
  cfg.dynamicSmemBytes = NS_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, ns_gemm_kernel<MODE, PAIR>, tp, tq, p);
}

// One CTA per 128 x 128 tile where that takes less time, in rounds of tiles:
// such a round takes 0.6 of one of pairs (half the products, but twice the
// bytes an operation). Five steps, pairs alone -> single CTAs alone -> by this
// rule: 2 of 768 x 768 229 -> 162 -> 162 us, 3 of 1024 x 4096 402 -> 429 -> 358,
// 2048 x 7168 687 -> 782 -> 638, 5 of 2000 x 3500 2080 -> 2389 -> 1863, 4096 x
// 4096 1220 -> 2286 -> (pairs). (Squares with mirrored tiles everywhere.)
template <int MODE>
cudaError_t launch_ns_gemm(const CUtensorMap& tp, const CUtensorMap& tq, const NsGemmParams& p, int num_sms,
                           cudaStream_t s) {
  const long long pair = ceil_div_ll(ns_tiles<MODE>(p, 2 * NS_HALF), num_sms / 2);
  const long long one = ceil_div_ll(ns_tiles<MODE>(p, NS_HALF), num_sms);
  return 0.6 * one < pair ? launch_ns_tiles<MODE, false>(tp, tq, p, num_sms, s)
                        : launch_ns_tiles<MODE, true>(tp, tq, p, num_sms, s);
}

constexpr size_t kNsAlign = 256;
size_t ns_round(size_t v) { return (v + kNsAlign - 1) / kNsAlign * kNsAlign; }

struct NsPlan {
  int m, n, ld_x, ld_a;
  int batch;                // matrices worked on at once
  int norm_blocks;          // partial sums per matrix
  size_t err, partial, x0, x1, a, b, diag, total;
};

bool ns_on_chip(int m, int n) { return m <= NSC_M && n <= NSC_N; }

// A matrix is independent of the others; enough of them run together to give
// the smallest product (tiles of A) about eight rounds of tiles per CTA pair,
// and no more, so that the scratch stays small and near L2's size. Matrices that
// stay on chip have no scratch but the error word, and run all together.
NsPlan ns_plan(int n_mat, int rows, int cols, int num_sms) {
  NsPlan q = {};
  q.m = rows < cols ? rows : cols;
  q.n = rows < cols ? cols : rows;
  q.ld_x = (q.n + 7) / 8 * 8;
  q.ld_a = (q.m + 7) / 8 * 8;
  const long long t = ceil_div(q.m, 2 * NS_HALF), tiles = t * (t + 1) / 2;
  long long most = ceil_div_ll(8LL * (num_sms / 2), tiles);
  if (most > 32768) most = 32768;
  const bool chip = ns_on_chip(q.m, q.n);
  const long long rounds = chip ? 1 : ceil_div_ll(n_mat > 0 ? n_mat : 1, most);
  q.batch = (int)ceil_div_ll(n_mat > 0 ? n_mat : 1, rounds);
  const long long size = (long long)rows * cols, blocks = ceil_div_ll(size, NS_NORM_THREADS * 8 * 4);
  q.norm_blocks = (int)(blocks < NS_NORM_MAX ? blocks : NS_NORM_MAX);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += ns_round(bytes);
    return o;
  };
  q.err = take(kNsAlign);
  if (!chip) {
    q.partial = take((size_t)q.batch * q.norm_blocks * 4);
    q.x0 = take((size_t)q.batch * q.m * q.ld_x * 2);
    q.x1 = take((size_t)q.batch * q.m * q.ld_x * 2);
    q.a = take((size_t)q.batch * q.m * q.ld_a * 2);
    q.b = take((size_t)q.batch * q.m * q.ld_a * 2);
    q.diag = take(q.m <= NSC_M ? (size_t)q.batch * q.m * 4 : 0);
  }
  q.total = off;
  return q;
}

template <typename T, bool MOM>
cudaError_t launch_ns_chip(const NsChipParams& cp, cudaStream_t s) {
  const cudaError_t e = allow_max_smem<ns_chip_kernel<T, MOM>>();
  if (e != cudaSuccess) return e;
  ns_chip_kernel<T, MOM><<<cp.g.n_mat, NSC_THREADS, NSC_SMEM, s>>>(cp);
  return cudaGetLastError();
}

template <typename T, bool MOM>
cudaError_t ns_first_x(const OrthoParams& p, const NsPlan& q, int first, int count, char* ws, bool clear,
                       cudaStream_t s) {
  const long long size = (long long)p.rows * p.cols;
  const int col_tiles = ceil_div(p.cols, 64);
  // Running both passes over a few matrices at a time, so that the second finds
  // U in L2, took 60 us more on 8 x 2048 x 7168 with momentum: the launches'
  // ends cost more than the 700 MB saved.
  const T* g = static_cast<const T*>(p.g) + (size_t)first * size;
  float* mom = MOM ? p.momentum + (size_t)first * size : nullptr;
  float* partial = reinterpret_cast<float*>(ws + q.partial);
  ns_norm_kernel<T, MOM><<<dim3(q.norm_blocks, count), NS_NORM_THREADS, 0, s>>>(
      g, mom, p.mu, p.nesterov, size, size % 8 == 0, partial, clear ? reinterpret_cast<uint32_t*>(ws + q.err) : nullptr);
  ns_init_kernel<T, MOM><<<dim3((unsigned)(col_tiles * (long long)ceil_div(p.rows, 64)), count), 256, 0, s>>>(
      g, mom, p.mu, p.nesterov, p.rows, p.cols, p.cols % 8 == 0, p.rows > p.cols, p.eps, partial, q.norm_blocks,
      col_tiles, reinterpret_cast<__half*>(ws + q.x0), q.ld_x);
  return cudaGetLastError();
}

}  // namespace

size_t ortho_workspace_bytes(int n_mat, int rows, int cols, int num_sms) {
  return ns_plan(n_mat, rows, cols, num_sms).total;
}

cudaError_t launch_ortho(const OrthoParams& p, void* workspace, int num_sms, cudaStream_t s) {
  const NsPlan q = ns_plan(p.n, p.rows, p.cols, num_sms);
  char* ws = static_cast<char*>(workspace);
  __half* x[2] = {reinterpret_cast<__half*>(ws + q.x0), reinterpret_cast<__half*>(ws + q.x1)};
  __half *a = reinterpret_cast<__half*>(ws + q.a), *b = reinterpret_cast<__half*>(ws + q.b);
  CUtensorMap xk[2], xn[2], ak, bk;
  const bool chip = ns_on_chip(q.m, q.n);
  for (int i = 0; i < 2 && !chip; ++i)
    if (!make_ns_tmap(&xk[i], x[i], q.n, q.m, q.batch, q.ld_x, NS_HALF) ||
        !make_ns_tmap(&xn[i], x[i], q.n, q.m, q.batch, q.ld_x, NS_BK))
      return cudaErrorInvalidValue;
  if (!chip && (!make_ns_tmap(&ak, a, q.m, q.m, q.batch, q.ld_a, NS_HALF) ||
                !make_ns_tmap(&bk, b, q.m, q.m, q.batch, q.ld_a, NS_HALF)))
    return cudaErrorInvalidValue;
  const size_t size = (size_t)p.rows * p.cols;
  for (int first = 0; first < p.n; first += q.batch) {
    const int count = p.n - first < q.batch ? p.n - first : q.batch;
    const bool f32 = p.dtype == MOE_DTYPE_F32, mom = p.momentum != nullptr;
    NsGemmParams g = {};
    g.n_mat = count;
    g.m = q.m; g.n = q.n;
    g.ld_x = q.ld_x; g.ld_a = q.ld_a;
    g.a_in = a;
    g.diag = !chip && q.m <= NSC_M ? reinterpret_cast<float*>(ws + q.diag) : nullptr;
    g.tall = p.rows > p.cols;
    g.rows = p.rows; g.cols = p.cols;
    g.o = p.o ? static_cast<__nv_bfloat16*>(p.o) + first * size : nullptr;
    g.weight_f32 = p.weight_dtype == MOE_DTYPE_F32;
    g.weight = p.weight ? static_cast<char*>(p.weight) + first * size * (g.weight_f32 ? 4 : 2) : nullptr;
    g.keep = p.keep;
    g.step = p.step;
    g.err = reinterpret_cast<uint32_t*>(ws + q.err);
    g.timeout_ns = kDefaultTimeoutNs;
    if (chip) {
      NsChipParams cp = {};
      cp.g = g;
      cp.grad = static_cast<const char*>(p.g) + first * size * (f32 ? 4 : 2);
      cp.mom = mom ? p.momentum + first * size : nullptr;
      cp.mu = p.mu;
      cp.eps = p.eps;
      cp.nesterov = p.nesterov;
      cp.steps = p.steps;
      cp.clear_err = first == 0;
      for (int k = 0; k < 3 * p.steps; ++k) cp.coeffs[k] = p.coeffs[k];
      const cudaError_t e = f32 ? (mom ? launch_ns_chip<float, true>(cp, s) : launch_ns_chip<float, false>(cp, s))
                                : (mom ? launch_ns_chip<__nv_bfloat16, true>(cp, s)
                                       : launch_ns_chip<__nv_bfloat16, false>(cp, s));
      if (e != cudaSuccess) return e;
      continue;
    }
    cudaError_t e =
        f32 ? (mom ? ns_first_x<float, true>(p, q, first, count, ws, first == 0, s)
                   : ns_first_x<float, false>(p, q, first, count, ws, first == 0, s))
            : (mom ? ns_first_x<__nv_bfloat16, true>(p, q, first, count, ws, first == 0, s)
                   : ns_first_x<__nv_bfloat16, false>(p, q, first, count, ws, first == 0, s));
    if (e != cudaSuccess) return e;
    for (int k = 0; k < p.steps; ++k) {
      const int cur = k & 1;
      g.a = p.coeffs[3 * k]; g.b = p.coeffs[3 * k + 1]; g.c = p.coeffs[3 * k + 2];
      g.out = a;
      if ((e = launch_ns_gemm<kNsGram>(xk[cur], xk[cur], g, num_sms, s)) != cudaSuccess) return e;
      g.out = b;
      if ((e = launch_ns_gemm<kNsPoly>(ak, ak, g, num_sms, s)) != cudaSuccess) return e;
      g.out = x[cur ^ 1];
      g.x_in = x[cur];
      e = k + 1 < p.steps ? launch_ns_gemm<kNsApply>(bk, xn[cur], g, num_sms, s)
                          : launch_ns_gemm<kNsLast>(bk, xn[cur], g, num_sms, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace moe

// Expert FFNs of small batches on 4-bit weights with group scales, and the
// kernels that make and unmake such weights.
//
//   W[m][k] = scale[m][k / G] * (code[m][k] - zero[m][k / G])     code in 0..15
//
// Sparse MoE FFN (DeepSeek-V3 note), "How it works": the SwiGLU equation
// W2 (SiLU(W1 u) * W3 u) of every expert over its packed rows, the shared
// expert over all tokens.
//
// What bounds it: a decode batch gives an expert a handful of rows, so its
// weights cross HBM for a few operations each. Four bits and a bf16 scale per
// G make that 0.5 + 2/G bytes a weight (3/G with zero points), a quarter of
// bf16; unpacking them is what then fills the SM. The products are small
// enough for the register-operand tensor path (tcgen05 would want unpacked
// weights written back to shared memory first): one mma.sync m16n8k16 takes 16
// weight rows x 8 tokens, with fp16 operands, because a code needs no
// arithmetic to become one: the half 0x000c is the subnormal number c 2^-24,
// exactly, and 0x00c0 is 16 times that. A 32-bit word holds eight codes of
// consecutive k; it and itself shifted by 8, masked by 0x000f000f and
// 0x00f000f0, are four operand pairs: five instructions per eight weights (the
// 128 + code form of bf16 took seven and a subtraction, e4m3 operands twelve,
// as their products run as fp16 ones on sm_100a).
//
// Token rows as fp16: a row is scaled by the power of two that brings its
// largest magnitude into [2^14, 2^15), the k under the 0x00f0 masks by 1/16
// besides. fp16's eleven bits hold bf16's eight; only values below 2^-27 of
// the row's largest lose bits. The intermediate h goes from the first launch to
// the second in 16 bits a value with fp16's eleven significant ones (2^-11; bf16's
// eight made the result's error 1.4 times its own rounding, up to 1.6 times for
// narrow experts): as fp16 over the power of two that brings the largest of
// eight neighbours into [1, 2), and no magnitude to 2, so that bit 14 of a word
// stays free. The eight free bits hold that power. Values below 2^-14 of the
// largest of their eight lose bits (to 2^-25 of it). A CTA makes the rows in
// shared memory when it comes to a segment, with each group's sum, off which the
// zero points come: it is where the group's product starts from. The product
// takes its scale in fp32. No weight is rounded.
//
// Layout of the work: the tiles of all non-empty segments (16 rows of W1 and W3,
// or 32 rows of W2, with a pass's 8 or 16 of the segment's token rows) are dealt to
// the CTAs in contiguous runs of equal length, so a batch that touches few
// experts still uses every SM. Within a CTA a run is cut where the token rows
// change; the chunks (256 k) of each piece's tiles go to its 8 warps in equal
// contiguous shares. A tile that straddles warps is finished by the one that
// began it, the others leave their sums in shared memory: no barrier but the
// two around a piece. Each warp streams its chunks through a ring of its own,
// its first lane starts a tile by one TMA (128 bytes by 16 rows, 128-byte
// swizzle: the word reads then meet every bank once), across pieces, so weights
// flow all the time. What is left to the lanes per 1024 weights (32 k of two
// tiles) is 5 shared reads, 20 integer instructions and 4 products.
//
// Measured: 32 tokens, 128 experts of 768 x 2048, top 8, of which 72 are touched
// (176 MB of weights and rows): 58 to 61 us the two launches in one stream, 3.0
// TB/s, 46% of the copy rate. Nothing is full: gate/up alone takes 42 us with the
// issue slots at 51%, the integer pipe at 54%, the tensor pipe at 20% and DRAM at
// 35%; its warps, with one chunk each in flight, wait most for their own chains of
// unpacking and products. 1 token (19.5 MB): 16.9 us, most of it two launches'
// start and the first loads. 24 tokens, 32 experts of 2048 x 7168 and the shared
// one, groups of 64 with zero points (798 MB): 282 to 308 us, 2.7 TB/s: gate/up's
// token rows (115 KB) leave one CTA an SM, whose 8 warps issue in 46% of the
// cycles, and it reads 633 MB, as segments of more than eight rows stream their
// weights twice.
#include <cuda_fp16.h>

#include <type_traits>

#include "umma_common.cuh"

namespace moe {
namespace {

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = W4_WARPS * 32;
constexpr int W4_CHUNK = 256;                       // k of one ring stage
constexpr int W4_TILE_BYTES = 16 * W4_CHUNK / 2;    // 16 rows of codes
constexpr int W4_STAGE_BYTES = 2 * W4_TILE_BYTES;
constexpr int W4_STAGES = 2;

// A bounded wait by a whole warp, with one outcome for all its lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* err,
                                          long long timeout_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, err, timeout_ns, true));
}
// c = i + a b, and c += a b, fp16 operands.
__device__ __forceinline__ void mma_f16_from(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float i0,
                                              float i1, float i2, float i3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(i0), "f"(i1), "f"(i2), "f"(i3));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two floats as a pair of fp16.
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The intermediate's words: value j of eight neighbours has bit h_bit(j) of their
// exponent byte (a float's: 0 for none, 255 for an infinity or NaN) in its bit 14.
__device__ __forceinline__ int h_bit(int j) { return (j >> 1) + (j & 1) * 4; }
__device__ __forceinline__ uint32_t h_exponent(const uint4& v) {
  const uint32_t m = 0x40004000u;
  const uint32_t a = ((v.x & m) >> 14) | ((v.y & m) >> 13) | ((v.z & m) >> 12) | ((v.w & m) >> 11);
  return (a & 15u) | ((a >> 12) & 0xf0u);
}
__device__ __forceinline__ __half2 h_pair(uint32_t w) {   // the two values of a word pair, exponent bits off
  w &= 0xbfffbfffu;
  return *reinterpret_cast<const __half2*>(&w);
}
// 2^p as a pair of fp16, 0 below fp16's smallest.
__device__ __forceinline__ __half2 half2_power(int p) {
  const uint32_t h = p >= -14 ? (uint32_t)(p + 15) << 10 : p >= -24 ? 1u << (p + 24) : 0u;
  const uint32_t w = h * 0x10001u;
  return *reinterpret_cast<const __half2*>(&w);
}
// The four operand pairs of a word of codes: (c0, c4), 16 (c1, c5), (c2, c6), 16 (c3, c7).
__device__ __forceinline__ void unpack_w4(uint32_t w, uint32_t (&p)[4]) {
  p[0] = w & 0x000f000fu;
  p[1] = w & 0x00f000f0u;
  p[2] = (w >> 8) & 0x000f000fu;
  p[3] = (w >> 8) & 0x00f000f0u;
}

// What a CTA knows of the i-th non-empty segment: x = chunks up to its end, y =
// its expert (n_routed: the dense one), z = its first token row, w = its rows.
using W4Entry = int4;

// Shared memory of a CTA: rings | sums left by warps that did not begin a tile |
// token rows in fp16 [rows][x_stride] | -8 or -1 times the groups' sums [K /
// GROUP][8 NT] | the rows' factors [8 NT] | table.
struct W4Plan {
  int rows;                 // token rows of a pass, at most 8 NT
  int x_stride;             // bytes of a token row
  int red, x, xs, f, tab;   // offsets
};

struct W4Piece {            // a run of one segment's tiles with the same token rows
  const W4Operand* op;
  size_t row0;              // first weight row of the segment in its matrix
  int M, K, nch;            // chunks of a tile
  int t0, rows;             // token rows [t0, t0 + rows)
  int tile0, tiles;         // the run
  bool dense;
};

template <int MATS, int NT, int GROUP, bool ZERO>
__global__ void __launch_bounds__(W4_THREADS, 2)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                   const __grid_constant__ CUtensorMap tm0s, const __grid_constant__ CUtensorMap tm1s,
                   const W4GemmParams p, const W4Plan plan) {
  constexpr int RED = 2 * NT * 32;                        // float4s of one warp's sums
  constexpr int WROWS = MATS == 2 ? 16 : 32;              // weight rows of a tile
  constexpr int NG = W4_CHUNK / GROUP;                    // groups of a chunk: 2, 4 or 8
  constexpr int PER = GROUP / 32;                         // steps of 32 k in a group
  constexpr int SCW = NG / 2, ZW = NG > 4 ? 2 : 1;        // words of a row's scales and zero points in a chunk
  extern __shared__ uint8_t w4_raw[];
  uint8_t* w4_dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w4_raw) + 1023) & ~uintptr_t(1023));
  __shared__ int warp_n[W4_WARPS];
  __shared__ long long warp_u[W4_WARPS];
  __shared__ uint64_t full_bar[W4_WARPS][W4_STAGES];
  __shared__ uint32_t abort_word;
  __shared__ int bad_word;
  volatile uint32_t* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const uint8_t* ring = w4_dyn + (size_t)warp * W4_STAGES * W4_STAGE_BYTES;
  float4* red = reinterpret_cast<float4*>(w4_dyn + plan.red);
  uint8_t* xp = w4_dyn + plan.x;
  float* xsum = reinterpret_cast<float*>(w4_dyn + plan.xs);
  float2* xfac = reinterpret_cast<float2*>(w4_dyn + plan.f);
  W4Entry* tab = reinterpret_cast<W4Entry*>(w4_dyn + plan.tab);
  if (tid == 0) {
    for (int w = 0; w < W4_WARPS; ++w)
      for (int i = 0; i < W4_STAGES; ++i) mbar_init(smem_u32(&full_bar[w][i]), 1);
    abort_word = 0u;
    bad_word = 0;
    fence_mbar_init();
    tmap_prefetch(&tm0);
    if (MATS == 2) tmap_prefetch(&tm1);
  }

  // What the launches before wrote, the routing among it, gate/up reads only from
  // here on; down waits below, after its first weights.
  if (!p.wait_previous) asm volatile("griddepcontrol.wait;" ::: "memory");

  // -------------------------------------------------- the segments' table
  const int n_seg = p.n_routed + (p.dense_rows > 0 ? 1 : 0);
  int base_n = 0;
  long long base_u = 0;
  for (int s0 = 0; s0 < n_seg; s0 += W4_THREADS) {
    const int s = s0 + tid;
    int begin = 0, rows = 0;
    long long units = 0;
    if (s < n_seg) {
      int M = p.M_s, K = p.K_s;
      if (s < p.n_routed) {
        M = p.M;
        K = p.K;
        begin = min(max(p.offsets[s], 0), p.max_rows);
        rows = min(max(p.offsets[s + 1], 0), p.max_rows) - begin;   // below 0 (a bad table): no rows
      } else {
        rows = p.dense_rows;
      }
      if (rows > 0) units = (long long)ceil_div(M, WROWS) * ceil_div(K, W4_CHUNK) * ceil_div(rows, plan.rows);
    }
    const unsigned act = __ballot_sync(0xffffffffu, units > 0);
    long long inc = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) {
      warp_n[warp] = __popc(act);
      warp_u[warp] = inc;
    }
    __syncthreads();
    int n = base_n;
    long long u = base_u;
    for (int w = 0; w < W4_WARPS; ++w) {
      if (w < warp) {
        n += warp_n[w];
        u += warp_u[w];
      }
      base_n += warp_n[w];
      base_u += warp_u[w];
    }
    if (units > 0) {
      const int i = n + __popc(act & ((1u << lane) - 1u));
      tab[i] = make_int4((int)(u + inc), s, begin, rows);
    }
    __syncthreads();
  }
  // Down may start beside gate/up from here on: the routing that it reads too is
  // complete. (Down itself does not call the next launch in early: waiting CTAs
  // in its SMs cost the wide case 7%.)
  if (!p.wait_previous) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // A count past 32 bits comes from overlapping segments, a bad table: no work.
  const int n_act = base_n, total = base_u <= 0x7fffffffLL ? (int)base_u : 0;
  // A CTA's share of the chunks, moved down to where tiles begin: positions
  // are (segment, tile), a segment's tiles counted pass after pass.
  auto seg_chunks = [&](int s) { return ceil_div(s >= p.n_routed ? p.K_s : p.K, W4_CHUNK); };
  auto boundary = [&](int b, int& seg, int& tile) {
    const int at = (int)((long long)total * b / gridDim.x);
    int lo = 0, hi = n_act;                          // the first segment that ends past `at`
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at < tab[mid].x) hi = mid; else lo = mid + 1;
    }
    seg = lo;
    tile = lo < n_act ? (at - (lo ? tab[lo - 1].x : 0)) / seg_chunks(tab[lo].y) : 0;
  };
  int seg0, tile0, seg1, tile1;
  boundary(blockIdx.x, seg0, tile0);
  boundary(blockIdx.x + 1, seg1, tile1);
  // The piece that begins at (seg, tile), which move past it; false at the end.
  auto next_piece = [&](int& seg, int& tile, W4Piece& w) -> bool {
    if (seg > seg1 || (seg == seg1 && tile >= tile1)) return false;
    const W4Entry e = tab[seg];
    w.dense = e.y >= p.n_routed;
    w.op = w.dense ? p.w_s : p.w;
    w.M = w.dense ? p.M_s : p.M;
    w.K = w.dense ? p.K_s : p.K;
    w.nch = ceil_div(w.K, W4_CHUNK);
    w.row0 = w.dense ? 0 : (size_t)e.y * p.M;
    const int per = ceil_div(w.M, WROWS), pass = tile / per;
    int end = per * ceil_div(e.w, plan.rows);        // of the segment
    const int last = seg == seg1 ? tile1 : end;
    w.t0 = e.z + pass * plan.rows;
    w.rows = min(plan.rows, e.w - pass * plan.rows);
    w.tile0 = tile - pass * per;
    w.tiles = min(last, (pass + 1) * per) - tile;
    tile += w.tiles;
    if (tile >= end) {
      ++seg;
      tile = 0;
    }
    return true;
  };
  auto share = [&](const W4Piece& w, int k) { return (int)((long long)w.tiles * w.nch * k / W4_WARPS); };

  // ------------------------------------------------------- weight stream
  // The next chunk of this warp: the piece it is in, its tile and number, and
  // how many more the warp has there. All lanes keep count, the first one
  // starts the copies; each loads the scales of its rows, into registers.
  int pseg = seg0, ptile = tile0, pc = 0, pleft = 0, pm = 0;
  W4Piece pw = {};
  const uint16_t* psc[2] = {nullptr, nullptr};       // row g's scales
  const uint8_t* pz[2] = {nullptr, nullptr};         // and zero points, or null
  int pgroups = 0;
  // Scales (bf16 pairs) and zero points (bytes) of the last chunk started, rows
  // g and g + 8 of each tile.
  uint32_t sc_r[2][2][SCW] = {}, z_r[2][2][ZW] = {};
  auto open_tile = [&]() {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const W4Operand& op = pw.op[MATS == 2 ? a : 0];
      const size_t row = pw.row0 + pm + (MATS == 2 ? 0 : 16 * a) + g;   // M is a multiple of 32
      psc[a] = static_cast<const uint16_t*>(op.scale) + row * pgroups;
      if (ZERO) pz[a] = op.zero ? op.zero + row * pgroups : nullptr;
    }
  };
  const uint32_t ring_s = smem_u32(ring);
  auto issue = [&](int slot) {
    while (pleft == 0) {                             // the next piece in which the warp has a share
      if (!next_piece(pseg, ptile, pw)) return;
      const int from = share(pw, warp);
      pleft = share(pw, warp + 1) - from;
      pgroups = pw.K / GROUP;
      pm = (pw.tile0 + from / pw.nch) * WROWS;
      pc = from % pw.nch;
      if (pleft) open_tile();
    }
    if (lane == 0) {
      const uint32_t fb = smem_u32(&full_bar[warp][slot]), dst = ring_s + slot * W4_STAGE_BYTES;
      const int y = (int)pw.row0 + pm;
      mbar_expect_tx(fb, W4_STAGE_BYTES);            // k past the matrix's end: zero fill
      tma_load_2d(dst, pw.dense ? &tm0s : &tm0, pc * (W4_CHUNK / 2), y, fb);
      if (MATS == 2) tma_load_2d(dst + W4_TILE_BYTES, pw.dense ? &tm1s : &tm1, pc * (W4_CHUNK / 2), y, fb);
      else tma_load_2d(dst + W4_TILE_BYTES, pw.dense ? &tm0s : &tm0, pc * (W4_CHUNK / 2), y + 16, fb);
    }
    // A row's scales of a chunk are NG neighbours: one load, unless K ends
    // inside a chunk.
    const int g0 = pc * NG;
    const bool whole = pgroups % NG == 0;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint16_t* sc = psc[a] + h * 8 * pgroups;
        const uint8_t* z = ZERO && pz[a] ? pz[a] + h * 8 * pgroups : nullptr;
        uint32_t* to = sc_r[a][h];
        uint32_t* tz = z_r[a][h];
        if (whole) {
          if (NG == 2) to[0] = __ldg(reinterpret_cast<const uint32_t*>(sc + g0));
          if (NG == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(sc + g0));
            to[0] = v.x;
            to[SCW > 1 ? 1 : 0] = v.y;
          }
          if (NG == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(sc + g0));
            to[0] = v.x;
            to[SCW > 1 ? 1 : 0] = v.y;
            to[SCW > 2 ? 2 : 0] = v.z;
            to[SCW > 2 ? 3 : 0] = v.w;
          }
          if (ZERO) {
            if (!z) {
#pragma unroll
              for (int i = 0; i < ZW; ++i) tz[i] = 0x08080808u;
            } else if (NG == 2) {
              tz[0] = __ldg(reinterpret_cast<const uint16_t*>(z + g0));
            } else if (NG == 4) {
              tz[0] = __ldg(reinterpret_cast<const uint32_t*>(z + g0));
            } else {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(z + g0));
              tz[0] = v.x;
              tz[ZW - 1] = v.y;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < SCW; ++i) {
            const int i0 = min(g0 + 2 * i, pgroups - 1), i1 = min(g0 + 2 * i + 1, pgroups - 1);
            to[i] = (uint32_t)__ldg(sc + i0) | ((uint32_t)__ldg(sc + i1) << 16);
          }
          if (ZERO) {
#pragma unroll
            for (int i = 0; i < ZW; ++i) {
              tz[i] = 0;
#pragma unroll
              for (int e = 0; e < 4 && e < NG; ++e)
                tz[i] |= (z ? (uint32_t)__ldg(z + min(g0 + 4 * i + e, pgroups - 1)) : 8u) << (8 * e);
            }
          }
        }
      }
    --pleft;
    if (++pc == pw.nch) {
      pc = 0;
      pm += WROWS;
      if (pleft) open_tile();
    }
  };
  issue(0);

  if (p.check && blockIdx.x == gridDim.x - 1) {
    // The last CTA checks the caller's indices for all, before anything could
    // time out. Where no earlier kernel of the call could have left a code it
    // writes the error word outright, which saves a launch that clears it.
    bool bad = false;
    for (int s = tid; s < p.n_routed; s += W4_THREADS) {
      const int a = p.offsets[s], b = p.offsets[s + 1];
      bad |= a < 0 || b < a || b > p.max_rows;
    }
    if (p.gather)
      for (int r = tid; r < p.max_rows; r += W4_THREADS) bad |= p.gather[r] < 0 || p.gather[r] >= p.gather_rows;
    if (bad) bad_word = 1;
    __syncthreads();
    if (tid == 0) *p.err = (p.err_keep ? *p.err : 0u) | (bad_word ? kErrBadIndex : 0u);
  }
  if (p.wait_previous) asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------------------------------------- token rows
  // A row of a piece by one warp, or by 2 or 4 where there are few rows:
  // its largest magnitude (each of them), then its values, eight k a lane paired
  // as the codes are, and its groups' sums (each a share).
  auto stage_rows = [&](const W4Piece& sg) {
    const int team = sg.rows > W4_WARPS / 2 ? 1 : sg.rows > W4_WARPS / 4 ? 2 : 4;
    for (int r = warp / team; r < sg.rows; r += W4_WARPS / team) {
      size_t src = sg.t0 + r;
      if (!sg.dense && p.gather) {
        const int v = p.gather[sg.t0 + r];
        src = v >= 0 && v < p.gather_rows ? v : 0;
      }
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(sg.dense ? p.x_s : p.x) +
                                                        src * (size_t)sg.K);
      const int n8 = sg.K / 8;
      // The largest magnitude: of two bf16 a word (they order like their bits, NaN
      // above infinity), or its exponent, as the intermediate's words have it.
      uint32_t big = 0;
#pragma unroll 8
      for (int i = lane; i < n8; i += 32) {
        const uint4 v = row[i];
        if (MATS == 1)
          big = max(big, h_exponent(v));
        else
          big = __vmaxu2(__vmaxu2(big, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
      const uint32_t top = MATS == 1 ? big << 7 : max(big & 0xffffu, big >> 16);
      // 2^e top in [2^14, 2^15); e splits in two so that both factors are
      // normal numbers, as does the power that the sums are multiplied by.
      int e = MATS == 1 || top >= 0x0080u ? 14 - ((int)(top >> 7) - 127) : 140;
      if (top >= 0x7f80u) e = 0;
      const float f1 = __int_as_float((127 + e / 2) << 23), f2 = __int_as_float((127 + e - e / 2) << 23);
      const int b = 24 - e;
      if (lane == 0 && warp % team == 0)
        xfac[r] = make_float2(top >= 0x7f80u ? __int_as_float(0x7fc00000) : __int_as_float((127 + b / 2) << 23),
                              __int_as_float((127 + b - b / 2) << 23));
      uint8_t* to = xp + (size_t)r * plan.x_stride;
      const int n8_pad = sg.nch * (W4_CHUNK / 8);
#pragma unroll 2
      for (int i = (warp % team) * 32 + lane; i < n8_pad; i += 32 * team) {   // whole warps: n8_pad is a multiple of 32
        const uint4 v = i < n8 ? row[i] : make_uint4(0, 0, 0, 0);
        float sum = 0.0f;
        if (MATS == 1) {
          // fp16 already: a product with a power of two, rounded once where it
          // falls below fp16's normal numbers.
          const int up = 14 + (int)h_exponent(v) - (int)big;
          const __half2 f = half2_power(up), f16 = half2_power(up - 4);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = __half22float2(__hmul2(h_pair(w[j]), f));
            sum += x.x;
            sum += x.y;
          }
          const __half2 o[4] = {__hmul2(h_pair(__byte_perm(v.x, v.z, 0x5410)), f),
                                __hmul2(h_pair(__byte_perm(v.x, v.z, 0x7632)), f16),
                                __hmul2(h_pair(__byte_perm(v.y, v.w, 0x5410)), f),
                                __hmul2(h_pair(__byte_perm(v.y, v.w, 0x7632)), f16)};
          *reinterpret_cast<uint4*>(to + i * 16) = *reinterpret_cast<const uint4*>(o);
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float x[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16) * f1 * f2;
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * f1 * f2;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += x[j];
          *reinterpret_cast<uint4*>(to + i * 16) =
              make_uint4(half_pair(x[0], x[4]), half_pair(x[1] * 0.0625f, x[5] * 0.0625f), half_pair(x[2], x[6]),
                         half_pair(x[3] * 0.0625f, x[7] * 0.0625f));
        }
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (i % (GROUP / 8) == 0)
          xsum[(i / (GROUP / 8)) * (8 * NT) + r] = sum * (ZERO ? -1.0f / 16777216.0f : -8.0f / 16777216.0f);
      }
    }
  };

  // ------------------------------------------------------------- products
  uint32_t get[W4_CHUNK / 32];                       // word q of row g's piece s, pieces swapped by the swizzle
#pragma unroll
  for (int s = 0; s < W4_CHUNK / 32; ++s) get[s] = g * 128 + ((s ^ g) * 16) + q * 4;
  const uint8_t* xlane = xp + (size_t)(g & (min(plan.rows, 8) - 1)) * plan.x_stride + q * 16;
  int slot = 0, seg = seg0, tile = tile0;
  uint32_t phase = 0;
  bool ok = true;
  W4Piece sg;
  while (next_piece(seg, tile, sg)) {
    stage_rows(sg);                                  // the last piece's barrier has freed the old rows
    __syncthreads();
    const int from = share(sg, warp), to = share(sg, warp + 1);
    float acc[2][NT][4];
    // A finished tile: lane's rows g and g + 8, token columns 2 q and 2 q + 1.
    auto finish = [&](int m) {
      const size_t first = (size_t)sg.t0 * sg.M + m + g;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (MATS == 2) {
          // The activation, by eight neighbours (the lanes of one q): the largest
          // exponent, of magnitudes raised by 2^-11 so that none rounds up to 2.
          float v[4];
          uint32_t ex = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 fac = xfac[t * 8 + q * 2 + (i & 1)];
            const float v0 = acc[0][t][i] * fac.x * fac.y, v1 = acc[1][t][i] * fac.x * fac.y;
            v[i] = v0 / (1.0f + __expf(-v0)) * v1;
            ex |= ((__float_as_uint(v[i] * (1.0f + 0x1p-11f)) & 0x7fffffffu) >> 23) << (8 * i);
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) ex = __vmaxu4(ex, __shfl_xor_sync(0xffffffffu, ex, o));
          uint16_t* out = static_cast<uint16_t*>(sg.dense ? p.out_s : p.out) + first;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = t * 8 + q * 2 + (i & 1);
            if (n >= sg.rows) continue;
            const uint32_t e = (ex >> (8 * i)) & 255u;
            const float f = __uint_as_float(e >= 254u ? 0x00400000u : (254u - e) << 23);    // 2^(127 - e)
            const uint32_t w = __half_as_ushort(__float2half_rn(v[i] * f)) & 0xbfffu;
            out[(size_t)n * sg.M + (i >> 1) * 8] = (uint16_t)(w | ((e >> h_bit(g)) & 1u) << 14);
          }
        } else {
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(sg.dense ? p.out_s : p.out) + first;
#pragma unroll
          for (int i = 0; i < 4; ++i) {    // the result's one rounding
            const int n = t * 8 + q * 2 + (i & 1);
            if (n >= sg.rows) continue;
            const float2 fac = xfac[n];
            __nv_bfloat16* at = out + (size_t)n * sg.M + (i >> 1) * 8;
            at[0] = __float2bfloat16_rn(acc[0][t][i] * fac.x * fac.y);
            at[16] = __float2bfloat16_rn(acc[1][t][i] * fac.x * fac.y);
          }
        }
      }
    };
    int c = from % sg.nch, m = (sg.tile0 + from / sg.nch) * WROWS;
    bool began = c == 0;
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][t][i] = 0.0f;
    for (int k = from; k < to; ++k) {
      uint32_t sc[2][2][SCW], zp[2][2][ZW];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < SCW; ++i) sc[a][h][i] = sc_r[a][h][i];
#pragma unroll
          for (int i = 0; i < ZW; ++i) zp[a][h][i] = z_r[a][h][i] & 0x0f0f0f0fu;
        }
      if (ok) issue(slot ^ 1);
      ok = ok && warp_wait(smem_u32(&full_bar[warp][slot]), phase, abort_flag, p.err, p.timeout_ns);
      const uint8_t* st = ring + slot * W4_STAGE_BYTES;
      const uint8_t* xc = xlane + c * (2 * W4_CHUNK);
      const float* xsc = xsum + c * NG * (8 * NT) + q * 2;
      float grp[2][NT][4];
#pragma unroll
      for (int s = 0; s < W4_CHUNK / 32; ++s) {      // 32 codes of each row
        uint4 xb[NT];
        // Minus eight times a group's sum of activations (or minus once, where
        // there are zero points to multiply it): where its products start from.
        float2 xs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t > 0 && t * 8 >= sg.rows) break;
          xb[t] = *reinterpret_cast<const uint4*>(xc + (size_t)t * 8 * plan.x_stride + s * 64);
          if (s % PER == 0) xs[t] = *reinterpret_cast<const float2*>(xsc + (s / PER) * (8 * NT) + t * 8);
        }
        const int sub = s / PER;                     // the chunk's group that step s belongs to
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const uint8_t* w = st + a * W4_TILE_BYTES + get[s];
          uint32_t lo[4], hi[4];
          unpack_w4(*reinterpret_cast<const uint32_t*>(w), lo);
          unpack_w4(*reinterpret_cast<const uint32_t*>(w + 1024), hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
          float z0 = 1.0f, z1 = 1.0f;
          if (ZERO && s % PER == 0) {
            // 2^23 + zero point as a float, its last byte picked from the row's
            z0 = __uint_as_float(__byte_perm(zp[a][0][sub / 4], 0x4b000000u, 0x7440 + (sub & 3))) - 8388608.0f;
            z1 = __uint_as_float(__byte_perm(zp[a][1][sub / 4], 0x4b000000u, 0x7440 + (sub & 3))) - 8388608.0f;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t > 0 && t * 8 >= sg.rows) break;
            if (s % PER == 0) {
              if (ZERO) mma_f16_from(grp[a][t], a0, xb[t].x, xb[t].y, z0 * xs[t].x, z0 * xs[t].y, z1 * xs[t].x, z1 * xs[t].y);
              else mma_f16_from(grp[a][t], a0, xb[t].x, xb[t].y, xs[t].x, xs[t].y, xs[t].x, xs[t].y);
            } else {
              mma_f16(grp[a][t], a0, xb[t].x, xb[t].y);
            }
            mma_f16(grp[a][t], a1, xb[t].z, xb[t].w);
          }
          if ((s + 1) % PER == 0) {                  // the group's sum is whole
            const uint32_t w0 = sc[a][0][sub / 2], w1 = sc[a][1][sub / 2];
            const float s0 = __uint_as_float(sub & 1 ? w0 & 0xffff0000u : w0 << 16);
            const float s1 = __uint_as_float(sub & 1 ? w1 & 0xffff0000u : w1 << 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (t > 0 && t * 8 >= sg.rows) break;
              acc[a][t][0] = fmaf(s0, grp[a][t][0], acc[a][t][0]);
              acc[a][t][1] = fmaf(s0, grp[a][t][1], acc[a][t][1]);
              acc[a][t][2] = fmaf(s1, grp[a][t][2], acc[a][t][2]);
              acc[a][t][3] = fmaf(s1, grp[a][t][3], acc[a][t][3]);
            }
          }
        }
      }
      __syncwarp();                                  // every lane has read the stage
      slot ^= 1;
      if (slot == 0) phase ^= 1u;
      if (++c == sg.nch) {                           // the tile ends
        if (began) {
          finish(m);
        } else {
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int t = 0; t < NT; ++t)
              red[warp * RED + (a * NT + t) * 32 + lane] =
                  make_float4(acc[a][t][0], acc[a][t][1], acc[a][t][2], acc[a][t][3]);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[a][t][i] = 0.0f;
        c = 0;
        m += WROWS;
        began = true;
      }
    }
    const bool open = c > 0 && from < to;            // the share ends inside a tile
    if (open && !began) {                            // and began inside the same one
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          red[warp * RED + (a * NT + t) * 32 + lane] =
              make_float4(acc[a][t][0], acc[a][t][1], acc[a][t][2], acc[a][t][3]);
    }
    __syncthreads();                                 // left sums visible, token rows free
    if (open && began) {
      // The tile's other shares, in order: the warps whose shares begin before
      // its end.
      const int end = (to / sg.nch + 1) * sg.nch;
      for (int w = warp + 1; w < W4_WARPS && share(sg, w) < end; ++w) {
        if (share(sg, w) == share(sg, w + 1)) continue;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float4 v = red[w * RED + (a * NT + t) * 32 + lane];
            acc[a][t][0] += v.x;
            acc[a][t][1] += v.y;
            acc[a][t][2] += v.z;
            acc[a][t][3] += v.w;
          }
      }
      finish(m);
    }
    __syncthreads();                                 // left sums and factors free
  }
  // After a wait that ran out: the copies under way land (or have had two more
  // seconds) before shared memory is freed.
  if (!ok && lane == 0)
    for (int i = 0; i < W4_STAGES; ++i)
      wait_bounded(smem_u32(&full_bar[warp][slot ^ i]), phase ^ (slot + i >= W4_STAGES ? 1u : 0u), abort_flag, p.err,
                   p.timeout_ns, false);
}

// Codes [rows][K/2] as bytes, 128-byte swizzle, box 128 bytes x 16 rows.
bool make_w4_tmap(CUtensorMap* tm, const void* q, long long rows, int K) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {W4_CHUNK / 2, 16};
  cuuint32_t estr[2] = {1, 1};
  return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared memory of a CTA that has an SM alone, and of two that share one.
constexpr int W4_SMEM = 232000, W4_SMEM_HALF = 115000;

int w4_layout(const W4GemmParams& p, int nt, int rows, W4Plan& l) {
  const int K = p.n_routed > 0 && p.K > p.K_s ? p.K : (p.dense_rows > 0 && p.K_s > p.K ? p.K_s : p.K);
  const int pad = ceil_div(K, W4_CHUNK) * W4_CHUNK;
  int off = 0;
  auto take = [&](int bytes) {
    const int o = off;
    off += ceil_div(bytes, 128) * 128;
    return o;
  };
  l.rows = rows;
  l.x_stride = 2 * pad + 64;                // 64 past a multiple of 128: a pair of rows takes every bank once
  take(W4_WARPS * W4_STAGES * W4_STAGE_BYTES);
  l.red = take(W4_WARPS * 2 * nt * 512);
  l.x = take(rows * l.x_stride);
  l.xs = take(pad / p.group * 8 * nt * 4);
  l.f = take(8 * nt * 8);
  l.tab = take((p.n_routed + (p.dense_rows > 0 ? 1 : 0)) * (int)sizeof(W4Entry));
  return off + 1024;                        // the rings start on a multiple of 1024
}

struct W4Shape {
  W4Plan plan;
  int nt, ctas, smem;
};

// Eight token rows a pass, or sixteen where groups are of 128 and the segments'
// rows (their mean, by weights) are 64 at least; fewer where rows that wide do not
// fit in an SM's shared memory. Two CTAs an SM where their rows fit twice.
// A second tile of eight shares the unpacking of a weight, but its accumulators
// leave the warps less to hide latency with, and half of it idles behind a short
// segment. us, one tile and two, by rows of each expert:
//                       8         16         32         64         128
//  64 of 768 x 2048
//    G 128            60   73    87   85   144  135   264  243   504  463
//    G 64             62   84    91   96   152  154   281  276   538  526
//    G 32             67  103    99  116   167  189   309  342   595  655
//    G 32, zeros      83  158   126  173   214  286   401  523   777 1009
//  128 of 256 x 512, G 128
//                     27   32    34   37    51   48    85   73   148  126
//  8 of 1536 x 4096, G 128
//                     41   57    63   78    94  107   157  159   284  264
// Four tiles spill and took 1.3 to 2 times the time of one everywhere.
bool w4_shape(const W4GemmParams& p, W4Shape& s) {
  const double routed = p.n_routed * (double)p.M * p.K, shared = p.dense_rows > 0 ? (double)p.M_s * p.K_s : 0.0;
  const double weighted = (double)p.max_rows * p.M * p.K + shared * p.dense_rows;   // rows of a segment x its weights
  s.nt = p.group == 128 && weighted >= 64.0 * (routed + shared) ? 2 : 1;
  if (s.nt == 2 && w4_layout(p, 2, 16, s.plan) > W4_SMEM) s.nt = 1;
  int rows = 8 * s.nt;
  while (rows > 1 && w4_layout(p, s.nt, rows, s.plan) > W4_SMEM) rows /= 2;
  s.smem = w4_layout(p, s.nt, rows, s.plan);
  s.ctas = s.smem <= W4_SMEM_HALF ? 2 : 1;
  return s.smem <= W4_SMEM;
}

// ------------------------------------------------------ making the weights
// Eight weights a thread; a group is 4, 8 or 16 neighbouring threads.
template <typename T> __device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <> __device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&f)[8]);
template <> __device__ __forceinline__ void store8<float>(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// scale = (largest magnitude) * (1/7) with the codes centred on 8, or (max -
// min) * (1/15) with a zero point, the factors and products in fp32; it is
// rounded to bf16 before the codes are taken: the rounding costs no accuracy.
// A group of zeros gets scale 0; one that holds a value that is not finite
// gets a NaN scale, so that it shows (the extremes are taken so that a NaN
// wins).
//
// round(w / scale) without a division per weight. t = w times the reciprocal is
// off by less than 1e-5 (four units of 2^-24 of at most 16).
//  - bf16 weights: scale and w have 8 significant bits, so 2 w and (2 k + 1)
//    scale are multiples of one unit that is at least 2^-10 of scale where w is
//    near (k + 1/2) scale: t lies on a half or at least 2^-10 from it. Rounded
//    to a multiple of 2^-12 first, it rounds as the exact quotient does.
//  - fp32 weights: a thread that meets a t within 1e-4 of a half divides.
// Scales near the ends of fp32's range divide too. Adding 2^23 * 1.5 rounds to
// an integer in the mantissa, ties to even; the codes' word is summed from
// these bits as they are, modulo 2^32, what they have in common taken off at
// the end. Dividing every weight took three times as long as the kernel's
// bytes, testing every weight for a tie still 125 us at 16384 x 7168; this form
// takes 90 us there (295 MB, 3.3 TB/s): the instructions per weight bound it.
constexpr float kRoundMagic = 12582912.0f;
constexpr float kRound12 = 1.5f * 2048.0f;   // multiples of 2^-12
constexpr int W4_QUANT_AHEAD = 2;     // vectors a thread loads at once

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T, bool ZERO>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ w, long long n8, int lanes_log2,
                                                          uint32_t* __restrict__ q, __nv_bfloat16* __restrict__ scale,
                                                          uint8_t* __restrict__ zero) {
  constexpr bool BF16 = sizeof(T) == 2;
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long start = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int lanes = 1 << lanes_log2;
  // Whole warps stay together over the shuffles: n8 is a multiple of `lanes`,
  // a group's lanes are in or out of range together.
  for (long long i0 = start; i0 - (threadIdx.x & 31) < n8; i0 += W4_QUANT_AHEAD * stride) {
    float f[W4_QUANT_AHEAD][8];
#pragma unroll
    for (int k = 0; k < W4_QUANT_AHEAD; ++k) {
      if (i0 + k * stride < n8) load8(w + (i0 + k * stride) * 8, f[k]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) f[k][j] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < W4_QUANT_AHEAD; ++k) {
      const long long i = i0 + k * stride;
      float hi = 0.0f, neg = 0.0f;                     // largest value, or magnitude; largest of -w
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hi = max_nan(hi, ZERO ? f[k][j] : fabsf(f[k][j]));
        if (ZERO) neg = max_nan(neg, -f[k][j]);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        if (ZERO) neg = max_nan(neg, __shfl_xor_sync(0xffffffffu, neg, o));
      }
      const bool finite = hi < INFINITY && neg < INFINITY;
      const __nv_bfloat16 s16 = __float2bfloat16_rn(ZERO ? (hi + neg) * (1.0f / 15.0f) : hi * (1.0f / 7.0f));
      const float s = __bfloat162float(s16), step = s > 0.0f ? s : 1.0f, inv = __fdividef(1.0f, step);
      const float zf = ZERO ? fminf(fmaxf(rintf(neg / step), 0.0f), 15.0f) : 8.0f;
      const uint32_t z = (uint32_t)zf;
      // round(w / step) + z clamped to 0..15; without zero points |w / step| is
      // at most 7.03 and needs no clamp.
      uint32_t word = 0;
      bool divide = !(step > 1e-37f && step < 1e37f);
      float far = 0.0f;                                // the farthest from an integer
#pragma unroll
      for (int j = 7; j >= 0; --j) {
        float t = BF16 ? fmaf(f[k][j], inv, kRound12) - kRound12 : f[k][j] * inv;
        if (!BF16) far = fmaxf(far, fabsf(t - ((t + kRoundMagic) - kRoundMagic)));
        if (ZERO) t = fminf(fmaxf(t, -zf), 15.0f - zf);
        word = word * 16u + (uint32_t)__float_as_int(t + kRoundMagic);
      }
      // sum over j of 16^j (bits of 1.5 * 2^23, less z), modulo 2^32
      word += z * 0x11111111u - 0x4b400000u * 0x11111111u;
      if (!BF16) divide |= !(far <= 0.4999f);
      if (divide) {
        word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = fminf(fmaxf(rintf(f[k][j] / step) + zf, 0.0f), 15.0f);
          word |= (uint32_t)c << (4 * j);
        }
      }
      if (i < n8) {
        q[i] = word;
        if ((i & (lanes - 1)) == 0) {
          scale[i >> lanes_log2] = finite ? s16 : __ushort_as_bfloat16(0x7fc0);
          if (ZERO) zero[i >> lanes_log2] = (uint8_t)z;
        }
      }
    }
  }
}

// scale (code - zero) in fp32, rounded once to T; eight weights a thread. Bound
// by HBM: 16384 x 7168 into bf16 in 52 us (295 MB, 5.7 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const __nv_bfloat16* __restrict__ scale,
                                                            const uint8_t* __restrict__ zero, long long n8,
                                                            int lanes_log2, T* __restrict__ w) {
  const long long stride = (long long)gridDim.x * blockDim.x;
#pragma unroll 2
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const uint32_t word = __ldg(q + i);
    const float s = __bfloat162float(scale[i >> lanes_log2]);
    // 2^23 + code is a float whose last bits are the code.
    const float z = 8388608.0f + (float)(zero ? (zero[i >> lanes_log2] & 15) : 8);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = s * (__uint_as_float(((word >> (4 * j)) & 15u) | 0x4b000000u) - z);
    store8(w + i * 8, f);
  }
}

}  // namespace

cudaError_t launch_w4_gemm(const W4GemmParams& p, int num_sms, cudaStream_t s) {
  W4Shape shape;
  if (!w4_shape(p, shape)) return cudaErrorInvalidValue;
  const int slots = shape.ctas * num_sms;
  CUtensorMap tm[4];
  for (int a = 0; a < 2; ++a) {
    if (a < p.mats) {
      if (!make_w4_tmap(&tm[a], p.w[a].q, (long long)p.n_routed * p.M, p.K)) return cudaErrorInvalidValue;
      if (p.dense_rows > 0 && !make_w4_tmap(&tm[2 + a], p.w_s[a].q, p.M_s, p.K_s)) return cudaErrorInvalidValue;
    } else {
      tm[a] = tm[0];
    }
    if (a >= p.mats || p.dense_rows == 0) tm[2 + a] = p.dense_rows > 0 ? tm[2] : tm[a];
  }
  auto go = [&](auto tag) {
    constexpr auto kernel = decltype(tag)::value;
    const cudaError_t e = allow_max_smem<kernel>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(slots);
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = shape.smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tm[0], tm[1], tm[2], tm[3], p, shape.plan);
  };
  auto with = [&](auto mats, auto n, auto zero) {
    constexpr int M = decltype(mats)::value, N = decltype(n)::value;
    constexpr bool Z = decltype(zero)::value;
    if constexpr (N == 2)      // groups of 128 only
      return go(KernelTag<w4_gemm_kernel<M, N, 128, Z>>{});
    else
      return p.group == 128  ? go(KernelTag<w4_gemm_kernel<M, N, 128, Z>>{})
             : p.group == 64 ? go(KernelTag<w4_gemm_kernel<M, N, 64, Z>>{})
                             : go(KernelTag<w4_gemm_kernel<M, N, 32, Z>>{});
  };
  auto mats = [&](auto n, auto zero) {
    return p.mats == 2 ? with(std::integral_constant<int, 2>{}, n, zero)
                       : with(std::integral_constant<int, 1>{}, n, zero);
  };
  auto rows_of = [&](auto n) { return p.has_zero ? mats(n, std::true_type{}) : mats(n, std::false_type{}); };
  return shape.nt == 1 ? rows_of(std::integral_constant<int, 1>{}) : rows_of(std::integral_constant<int, 2>{});
}

cudaError_t launch_w4_quantize(int dtype, const void* w, long long n, int group, void* q, void* scale, void* zero,
                               int num_sms, cudaStream_t s) {
  const long long n8 = n / 8, blocks = ceil_div_ll(n8, 256);
  const int grid = (int)(blocks < 8LL * num_sms ? blocks : 8LL * num_sms);
  auto go = [&](auto kernel, auto* src) {
    kernel<<<grid, 256, 0, s>>>(src, n8, group == 32 ? 2 : group == 64 ? 3 : 4, static_cast<uint32_t*>(q), static_cast<__nv_bfloat16*>(scale),
                                static_cast<uint8_t*>(zero));
    return cudaGetLastError();
  };
  if (dtype == MOE_DTYPE_F32) {
    const float* src = static_cast<const float*>(w);
    return zero ? go(w4_quantize_kernel<float, true>, src) : go(w4_quantize_kernel<float, false>, src);
  }
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w);
  return zero ? go(w4_quantize_kernel<__nv_bfloat16, true>, src) : go(w4_quantize_kernel<__nv_bfloat16, false>, src);
}

cudaError_t launch_w4_dequantize(int dtype, const void* q, const void* scale, const void* zero, long long n, int group,
                                 void* w, int num_sms, cudaStream_t s) {
  const long long n8 = n / 8, blocks = ceil_div_ll(n8, 256);
  const int grid = (int)(blocks < 8LL * num_sms ? blocks : 8LL * num_sms);
  auto go = [&](auto kernel, auto* dst) {
    kernel<<<grid, 256, 0, s>>>(static_cast<const uint32_t*>(q), static_cast<const __nv_bfloat16*>(scale),
                                static_cast<const uint8_t*>(zero), n8, group == 32 ? 2 : group == 64 ? 3 : 4, dst);
    return cudaGetLastError();
  };
  if (dtype == MOE_DTYPE_F32) return go(w4_dequantize_kernel<float>, static_cast<float*>(w));
  return go(w4_dequantize_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16*>(w));
}

}  // namespace moe

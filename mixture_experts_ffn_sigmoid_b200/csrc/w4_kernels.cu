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
// bf16. The products are small enough for the legacy tensor path: one
// mma.sync m16n8k16 takes 16 weight rows x 8 tokens from registers, where the
// codes are unpacked; tcgen05 would want the unpacked weights written back to
// shared memory first, four times the bytes that HBM delivers.
//
// Unpacking: a 32-bit word holds eight codes c0..c7 of consecutive k. (w >> 4i)
// & 0x000f000f is the pair (ci, c(i+4)); OR-ed with 0x4300 it is the pair of
// bf16 numbers 128 + code. The products run over these, and the 128 + zero
// that is too much comes off each group's sum in fp32, sum_k x_k of the group
// being one more product with a matrix of ones (shared by every row): seven
// integer instructions per eight weights and no arithmetic on them. The group's
// fp32 sum then takes its scale. No weight is rounded; the sums run about 30
// times as large as the result, which costs five of fp32's 24 bits and stays
// far below the rounding of the bf16 output. The order of k inside a group is
// free as long as both operands agree: token rows are paired the same way
// (x_i, x_(i+4)), by byte permutes in gate/up; h is written in that order, so
// the down product needs none.
//
// Layout of the work: a CTA of 8 warps takes a contiguous run of units; a unit
// is 16 WM rows of W1 and W3 (32 WM rows of W2) of one expert times up to 8 NT
// of its token rows, its K split over WK = 8 / WM warps in chunks of 256, two
// 16-row tiles a warp, which share the token fragments. Each warp streams its
// chunks through a ring of cp.async stages of its own, across unit boundaries,
// so weights keep flowing while a unit's partial sums meet in shared memory.
// Units of the non-empty segments only are dealt, evenly, so a batch that
// touches few experts still uses every SM.
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = W4_WARPS * 32;
constexpr int W4_CHUNK = 256;                       // k of one ring stage
constexpr int W4_TILE_BYTES = 16 * W4_CHUNK / 2;    // 16 rows of codes
constexpr int W4_STAGE_BYTES = 2 * W4_TILE_BYTES;
constexpr int W4_STAGES = 2;

__device__ __forceinline__ uint32_t w4_smem(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, or zeros where !valid (nothing is read then).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// c = a b, and c += a b.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The four bf16 pairs (128 + ci, 128 + c(i+4)) of a word.
__device__ __forceinline__ void unpack_w4(uint32_t w, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
}

struct W4Seg {   // one segment's share of a unit
  const W4Operand* op;      // [MATS] matrices
  size_t row0;              // first weight row of the segment in its matrix
  int M, K;
  int t0, rows;             // token rows [t0, t0 + rows) of the pass
  bool dense;
};

// What a CTA knows of the i-th non-empty segment: x = units up to its end, y =
// its expert (n_routed: the dense one), z = its first token row, w = its rows.
using W4Entry = int4;

// MATS = 2: gate/up, the two tiles of a warp are the same rows of W1 and W3.
// MATS = 1: down, they are 16 rows of W2 and the 16 after them.
template <int MATS, int NT, int GROUP>
__global__ void __launch_bounds__(W4_THREADS, 2) w4_gemm_kernel(const W4GemmParams p, int WK) {
  constexpr int RED = 2 * NT * 32;                        // float4s of one warp's partial sums
  constexpr int WROWS = MATS == 2 ? 16 : 32;              // weight rows of a warp
  extern __shared__ __align__(128) uint8_t w4_dyn[];
  __shared__ int warp_n[W4_WARPS];
  __shared__ long long warp_u[W4_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int WM = W4_WARPS / WK, wk = warp % WK, wm = warp / WK;
  uint8_t* ring = w4_dyn + (size_t)warp * W4_STAGES * W4_STAGE_BYTES;
  float4* red = reinterpret_cast<float4*>(w4_dyn + (size_t)W4_WARPS * W4_STAGES * W4_STAGE_BYTES);
  W4Entry* tab = reinterpret_cast<W4Entry*>(red + W4_WARPS * RED);

  // -------------------------------------------------- the segments' table
  const int n_seg = p.n_routed + (p.dense_rows > 0 ? 1 : 0);
  const int unit_rows = WROWS * WM;
  int base_n = 0;
  long long base_u = 0;
  for (int s0 = 0; s0 < n_seg; s0 += W4_THREADS) {
    const int s = s0 + tid;
    int begin = 0, rows = 0;
    long long units = 0;
    if (s < n_seg) {
      int M = p.M_s;
      if (s < p.n_routed) {
        M = p.M;
        begin = min(max(p.offsets[s], 0), p.max_rows);
        rows = min(max(p.offsets[s + 1], 0), p.max_rows) - begin;   // below 0 (a bad table): no rows
      } else {
        rows = p.dense_rows;
      }
      if (rows > 0) units = (long long)ceil_div(M, unit_rows) * ceil_div(rows, 8 * NT);
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
  // A count past 32 bits comes from overlapping segments, a bad table: no work.
  const int n_act = base_n, total = base_u <= 0x7fffffffLL ? (int)base_u : 0;
  if (!p.wait_previous) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int u0 = (int)((long long)total * blockIdx.x / gridDim.x);
  const int u1 = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);

  // Unit -> segment, tile of weight rows, pass over its token rows. Passes run
  // innermost: the weights they share are still in L2.
  auto locate = [&](int u, int& hint, W4Seg& sg, int& m0) {
    while (u >= tab[hint].x) ++hint;
    const W4Entry e = tab[hint];
    const int s = e.y, begin = e.z, rows = e.w, passes = ceil_div(rows, 8 * NT);
    const int rel = u - (hint ? tab[hint - 1].x : 0);
    sg.dense = s >= p.n_routed;
    sg.op = sg.dense ? p.w_s : p.w;
    sg.M = sg.dense ? p.M_s : p.M;
    sg.K = sg.dense ? p.K_s : p.K;
    sg.row0 = sg.dense ? 0 : (size_t)s * p.M;
    const int pass = rel % passes;
    sg.t0 = begin + pass * 8 * NT;
    sg.rows = min(8 * NT, rows - pass * 8 * NT);
    m0 = (rel / passes) * unit_rows + wm * WROWS;
  };
  // The first segment by halving: later ones follow one by one.
  int first_seg = 0;
  if (u0 < u1) {
    int lo = 0, hi = n_act - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (u0 < tab[mid].x) hi = mid; else lo = mid + 1;
    }
    first_seg = lo;
  }

  // ------------------------------------------------------- weight stream
  constexpr int NG = W4_CHUNK / GROUP;               // groups of a chunk: 2, 4 or 8
  constexpr int PER = GROUP / 32;                    // steps of 32 k in a group
  constexpr int HELD = NG > 4 ? 2 : 1;               // scales of a row that a lane loads: 4 lanes share a row's
  int pu = u0, phint = first_seg, pc = 0, pn = 0, pK = 0, pgroups = 0;   // the next chunk: unit, index, count
  const uint8_t* pq[2] = {nullptr, nullptr};         // this lane's pieces of codes, per tile
  const uint16_t* psc[2] = {nullptr, nullptr};       // row g's scales
  const uint8_t* pz[2] = {nullptr, nullptr};         // and zero points, or null
  uint16_t sc_r[2][2][HELD];                         // scales of the chunk under way: rows g and g + 8
  uint8_t z_r[2][2][HELD];

  auto open_unit = [&]() {                           // pointers of unit pu
    W4Seg sg;
    int m0;
    locate(pu, phint, sg, m0);
    pK = sg.K;
    pn = ceil_div(sg.K, W4_CHUNK);
    pgroups = sg.K / GROUP;
    pc = wk;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const W4Operand& op = sg.op[MATS == 2 ? a : 0];
      // A tile past the matrix (M is a multiple of 32) reads the first one: its
      // products are not stored.
      int m = MATS == 2 ? m0 : m0 + 16 * a;
      if (m >= sg.M) m = 0;
      const size_t row = sg.row0 + m;
      pq[a] = op.q + (row + (lane >> 3)) * (size_t)(sg.K / 2) + (lane & 7) * 16 + pc * (W4_CHUNK / 2);
      psc[a] = static_cast<const uint16_t*>(op.scale) + (row + g) * pgroups;
      pz[a] = op.zero ? op.zero + (row + g) * pgroups : nullptr;
    }
  };
  // A tile in a stage: 128 bytes a row, its 16-byte pieces swapped about so
  // that these writes and the word reads below each take every bank once.
  const uint32_t ring_s = w4_smem(ring);
  uint32_t put[2];                                   // rows lane / 8 + 8 i, and + 4
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = (lane >> 3) + 4 * h;
    put[h] = r * 128 + (((lane & 7) ^ r) * 16);
  }
  // Start the next chunk of this warp's stream into stage `slot`: codes into
  // shared memory, scales into registers, both used one chunk later.
  auto issue = [&](int slot) {
    while (pu < u1 && pc >= pn) {
      if (++pu < u1) open_unit();
    }
    if (pu < u1) {
      const uint32_t dst = ring_s + slot * W4_STAGE_BYTES;
      const size_t row4 = (size_t)pK * 2;            // four rows of codes
      if ((pc + 1) * W4_CHUNK <= pK) {
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cp_async16_all(dst + a * W4_TILE_BYTES + (i >> 1) * 1024 + put[i & 1], pq[a] + i * row4);
      } else {                                       // K ends inside the chunk
        const bool in_k = pc * W4_CHUNK + (lane & 7) * 32 < pK;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cp_async16_zfill(dst + a * W4_TILE_BYTES + (i >> 1) * 1024 + put[i & 1], pq[a] + i * row4 - (in_k ? 0 : (lane & 7) * 16), in_k);
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        pq[a] += WK * (W4_CHUNK / 2);
#pragma unroll
        for (int e = 0; e < HELD; ++e) {
          const int gi = min(pc * NG + (q & (NG / HELD - 1)) * HELD + e, pgroups - 1);
          sc_r[a][0][e] = __ldg(psc[a] + gi);
          sc_r[a][1][e] = __ldg(psc[a] + gi + 8 * pgroups);
          z_r[a][0][e] = z_r[a][1][e] = 8;
          if (pz[a]) {
            z_r[a][0][e] = __ldg(pz[a] + gi);
            z_r[a][1][e] = __ldg(pz[a] + gi + 8 * pgroups);
          }
        }
      }
      pc += WK;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (pu < u1) open_unit();
  issue(0);
  if (p.wait_previous) asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------------------------------------- products
  const uint32_t ones[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
  const uint32_t get = g * 128 + q * 4;              // word q of row g's piece s: ^ (s ^ g) * 16
  int slot = 0, hint = first_seg;
  for (int u = u0; u < u1; ++u) {
    W4Seg sg;
    int m0;
    locate(u, hint, sg, m0);
    const uint4* xrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // Token columns past the segment's rows read its first row: a column of
      // the product takes nothing from its neighbours, and these are not stored.
      const int r = t * 8 + g < sg.rows ? t * 8 + g : 0;
      size_t src = sg.t0 + r;
      if (!sg.dense && p.gather) {
        const int v = p.gather[sg.t0 + r];
        src = v >= 0 && v < p.gather_rows ? v : 0;
      }
      xrow[t] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(sg.dense ? p.x_s : p.x) +
                                               src * (size_t)sg.K) + q;
    }
    float acc[2][NT][4];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][t][i] = 0.0f;
    const int nch = ceil_div(sg.K, W4_CHUNK);
    for (int c = wk; c < nch; c += WK) {
      uint32_t sc[2][HELD];                          // rows g and g + 8
      float off[2][HELD][2];                         // with zero points: -scale (128 + zero), exact
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int e = 0; e < HELD; ++e) {
          sc[a][e] = (uint32_t)sc_r[a][0][e] | ((uint32_t)sc_r[a][1][e] << 16);
          if (p.has_zero)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              off[a][e][h] = __uint_as_float((uint32_t)sc_r[a][h][e] << 16) * (-128.0f - (float)(z_r[a][h][e] & 15));
        }
      issue(slot ^ 1);
      const bool whole = (c + 1) * W4_CHUNK <= sg.K;
      auto load_x = [&](int t, int s) -> uint4 {     // eight k of a token row
        if (whole) return xrow[t][c * (W4_CHUNK / 8) + s * 4];
        return c * W4_CHUNK + s * 32 < sg.K ? xrow[t][c * (W4_CHUNK / 8) + s * 4] : make_uint4(0, 0, 0, 0);
      };
      constexpr int AHEAD = NT == 1 ? 4 : 1;         // steps whose token rows are fetched ahead
      uint4 xv[AHEAD];
      if (NT == 1)
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) xv[s] = load_x(0, s);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      const uint8_t* st = ring + slot * W4_STAGE_BYTES;
      float grp[2][NT][4], xs[NT][4];
#pragma unroll
      for (int s = 0; s < W4_CHUNK / 32; ++s) {      // 32 codes of each row
        uint32_t xb[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t > 0 && t * 8 >= sg.rows) break;
          const uint4 v = NT == 1 ? xv[s % AHEAD] : load_x(t, s);
          if (NT == 1 && s + AHEAD < W4_CHUNK / 32) xv[s % AHEAD] = load_x(0, s + AHEAD);
          if (MATS == 2) {
            xb[t][0] = __byte_perm(v.x, v.z, 0x5410);
            xb[t][1] = __byte_perm(v.x, v.z, 0x7632);
            xb[t][2] = __byte_perm(v.y, v.w, 0x5410);
            xb[t][3] = __byte_perm(v.y, v.w, 0x7632);
          } else {
            xb[t][0] = v.x; xb[t][1] = v.y; xb[t][2] = v.z; xb[t][3] = v.w;
          }
          if (s % PER == 0) mma_16816_first(xs[t], ones, xb[t][0], xb[t][1]);
          else mma_16816(xs[t], ones, xb[t][0], xb[t][1]);
          mma_16816(xs[t], ones, xb[t][2], xb[t][3]);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const uint8_t* w = st + a * W4_TILE_BYTES + (get ^ ((s ^ g) * 16));
          uint32_t lo[4], hi[4];
          unpack_w4(*reinterpret_cast<const uint32_t*>(w), lo);
          unpack_w4(*reinterpret_cast<const uint32_t*>(w + 1024), hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t > 0 && t * 8 >= sg.rows) break;
            if (s % PER == 0) mma_16816_first(grp[a][t], a0, xb[t][0], xb[t][1]);
            else mma_16816(grp[a][t], a0, xb[t][0], xb[t][1]);
            mma_16816(grp[a][t], a1, xb[t][2], xb[t][3]);
          }
          if ((s + 1) % PER == 0) {                  // the group's sum is whole: its scale, from the lane that has it
            const int sub = s / PER;
            const uint32_t ss = __shfl_sync(0xffffffffu, sc[a][sub % HELD], (lane & 28) | (sub / HELD));
            const float s0 = __uint_as_float(ss << 16), s1 = __uint_as_float(ss & 0xffff0000u);
            float o0 = -136.0f * s0, o1 = -136.0f * s1;
            if (p.has_zero) {
              o0 = __shfl_sync(0xffffffffu, off[a][sub % HELD][0], (lane & 28) | (sub / HELD));
              o1 = __shfl_sync(0xffffffffu, off[a][sub % HELD][1], (lane & 28) | (sub / HELD));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              if (t > 0 && t * 8 >= sg.rows) break;
              acc[a][t][0] = fmaf(s0, grp[a][t][0], fmaf(o0, xs[t][0], acc[a][t][0]));
              acc[a][t][1] = fmaf(s0, grp[a][t][1], fmaf(o0, xs[t][1], acc[a][t][1]));
              acc[a][t][2] = fmaf(s1, grp[a][t][2], fmaf(o1, xs[t][0], acc[a][t][2]));
              acc[a][t][3] = fmaf(s1, grp[a][t][3], fmaf(o1, xs[t][1], acc[a][t][3]));
            }
          }
        }
      }
      __syncwarp();                                  // every lane has read the stage
      slot ^= 1;
    }
    // ------------------------------------------- the K shares meet, epilogue
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        red[warp * RED + (a * NT + t) * 32 + lane] =
            make_float4(acc[a][t][0], acc[a][t][1], acc[a][t][2], acc[a][t][3]);
    __syncthreads();
    const int mu = m0 - wm * WROWS;                  // the unit's first weight row
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(sg.dense ? p.out_s : p.out);
    const float* redf = reinterpret_cast<const float*>(red);
    for (int i = tid; i < sg.rows * unit_rows; i += W4_THREADS) {
      const int n = i / unit_rows, m = i - n * unit_rows;
      if (mu + m >= sg.M) continue;
      const int r = m & 15, a = MATS == 1 ? (m >> 4) & 1 : 0, w0 = m / WROWS * WK;
      const int at = ((n >> 3) * 32 + (r & 7) * 4 + ((n & 7) >> 1)) * 4 + (r >> 3) * 2 + (n & 1);
      float v[2] = {0.0f, 0.0f};
      for (int w = 0; w < WK; ++w) {
        v[0] += redf[((w0 + w) * RED + a * NT * 32) * 4 + at];
        if (MATS == 2) v[1] += redf[((w0 + w) * RED + NT * 32) * 4 + at];
      }
      // One rounding, of the activation (gate/up) or of the result (down).
      const float o = MATS == 2 ? v[0] / (1.0f + __expf(-v[0])) * v[1] : v[0];
      int col = mu + m;
      if (MATS == 2) col = (col & ~7) | ((col & 3) * 2 + ((col >> 2) & 1));   // h in the down product's order of k
      out[(size_t)(sg.t0 + n) * sg.M + col] = __float2bfloat16_rn(o);
    }
    __syncthreads();
  }
  // CTA 0 checks the caller's indices for all. Where no earlier kernel of the
  // call could have left a code it writes the error word outright, which saves
  // a launch that clears it.
  if (p.err && blockIdx.x == 0) {
    int bad = 0;
    for (int s = tid; s < p.n_routed; s += W4_THREADS) {
      const int a = p.offsets[s], b = p.offsets[s + 1];
      bad |= a < 0 || b < a || b > p.max_rows;
    }
    if (p.gather)
      for (int r = tid; r < p.max_rows; r += W4_THREADS) bad |= p.gather[r] < 0 || p.gather[r] >= p.gather_rows;
    bad = __syncthreads_or(bad);
    if (tid == 0) *p.err = (p.err_keep ? *p.err : 0u) | (bad ? kErrBadIndex : 0u);
  }
}

template <int NT> int w4_smem_bytes(int n_seg) {
  return W4_WARPS * (W4_STAGES * W4_STAGE_BYTES + 2 * NT * 512) + n_seg * (int)sizeof(W4Entry);
}

// Experts that a batch is expected to touch under even routing.
double w4_touched(const W4GemmParams& p) {
  if (p.n_routed <= 0 || p.max_rows <= 0) return 0.0;
  return p.n_routed * (1.0 - pow(1.0 - 1.0 / p.n_routed, (double)p.max_rows));
}

// Token tiles of eight per unit. A segment with more rows takes its weights
// again for every 8 NT of them, a unit with more tiles does more products per
// weight: 1, 1.3 and 2.1 times the time of one tile, measured at d = 7168 with
// 8, 16 and 32 rows an expert. Routed segments vary about their mean.
int w4_token_tiles(const W4GemmParams& p) {
  const double act = w4_touched(p), cost[3] = {1.0, 1.3, 2.1};
  int best = 1;
  double least = 1e300;
  for (int i = 0; i < 3; ++i) {
    const int nt = 1 << i;
    double t = (double)p.M_s * p.K_s * ceil_div(p.dense_rows, 8 * nt);
    if (act > 0.0) {
      const double mean = p.max_rows / act, passes = (mean + sqrt(mean)) / (8.0 * nt);
      t += act * p.M * p.K * (passes > 1.0 ? passes : 1.0);
    }
    t *= cost[i];
    if (t < least) {
      least = t;
      best = nt;
    }
  }
  return best;
}

// Warps along K. A CTA's time is its units times a warp's chunks in each (and
// about half a chunk of joining the shares); the split that makes this
// smallest for the experts that the batch is expected to touch wins.
int w4_split(const W4GemmParams& p, int slots) {
  const double act = w4_touched(p);
  int best = 1;
  double least = 1e300;
  for (int wk = 1; wk <= W4_WARPS; wk *= 2) {
    const int rows = (p.mats == 2 ? 16 : 32) * (W4_WARPS / wk);
    const double units = act * ceil_div(p.M, rows) + (p.dense_rows > 0 ? ceil_div(p.M_s, rows) : 0);
    const int K = p.n_routed > 0 ? p.K : p.K_s;
    const double t = ceil(units / slots) * (ceil_div(ceil_div(K, W4_CHUNK), wk) + 0.5);
    if (t < least) {
      least = t;
      best = wk;
    }
  }
  return best;
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
// round(w / scale) is taken from w times the reciprocal, which is off by less
// than 1e-5 steps (four units of 2^-24 of at most 16); only where that lies
// within 1e-4 of a half, and for scales near the ends of fp32's range, does
// the thread divide. Adding 2^23 * 1.5 rounds to an integer in the mantissa,
// ties to even; 8 more is even and changes no tie. Dividing every weight took
// three times as long as the kernel's bytes.
constexpr float kRoundMagic = 12582912.0f;
constexpr int W4_QUANT_AHEAD = 2;   // vectors a thread loads at once

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T, bool ZERO>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ w, long long n8, int lanes_log2,
                                                          uint32_t* __restrict__ q, __nv_bfloat16* __restrict__ scale,
                                                          uint8_t* __restrict__ zero) {
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
      const int z = ZERO ? (int)fminf(fmaxf(rintf(neg / step), 0.0f), 15.0f) : 8;
      uint32_t word = 0;
      float far = 0.0f;                                // the farthest from an integer
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = f[k][j] * inv, m = t + kRoundMagic;
        far = fmaxf(far, fabsf(t - (m - kRoundMagic)));
        int c = __float_as_int(m) - __float_as_int(kRoundMagic) + z;
        if (ZERO) c = min(max(c, 0), 15);              // without: |t| <= 7.03, 1 to 15 as it is
        word |= (uint32_t)(c & 15) << (4 * j);
      }
      if (!(far <= 0.4999f) || !(step > 1e-37f && step < 1e37f)) {
        word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = fminf(fmaxf(rintf(f[k][j] / step) + (float)z, 0.0f), 15.0f);
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
  const int slots = 2 * num_sms;
  const int nt = w4_token_tiles(p);
  const int wk = w4_split(p, slots);
  const int n_seg = p.n_routed + (p.dense_rows > 0 ? 1 : 0);
  auto go = [&](auto tag, int smem) {
    constexpr auto kernel = decltype(tag)::value;
    const cudaError_t e = allow_max_smem<kernel>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(slots);
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.wait_previous ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, wk);
  };
  auto with = [&](auto mats, auto n) {
    constexpr int M = decltype(mats)::value, N = decltype(n)::value;
    const int smem = w4_smem_bytes<N>(n_seg);
    return p.group == 128  ? go(KernelTag<w4_gemm_kernel<M, N, 128>>{}, smem)
           : p.group == 64 ? go(KernelTag<w4_gemm_kernel<M, N, 64>>{}, smem)
                           : go(KernelTag<w4_gemm_kernel<M, N, 32>>{}, smem);
  };
  auto rows_of = [&](auto n) {
    return p.mats == 2 ? with(std::integral_constant<int, 2>{}, n) : with(std::integral_constant<int, 1>{}, n);
  };
  return nt == 1   ? rows_of(std::integral_constant<int, 1>{})
         : nt == 2 ? rows_of(std::integral_constant<int, 2>{})
                   : rows_of(std::integral_constant<int, 4>{});
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

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
// & 0x000f000f is the pair (ci, c(i+4)); OR-ed with 0x4300 it is bf16 128 +
// code, from which 128 + zero is subtracted exactly. The products therefore
// run over exact small integers; the scale is applied in fp32 to each group's
// accumulator, so no weight is ever rounded. The order of k inside a group is
// free as long as both operands agree: token rows are paired the same way
// (x_i, x_(i+4)).
//
// Layout of the work: a CTA of 8 warps takes a contiguous run of units; a unit
// is 16 WM weight rows of one expert (times up to 8 NT of its token rows), its
// K split over WK = 8 / WM warps in chunks of 128. Each warp streams its chunks
// through a ring of cp.async stages of its own, across unit boundaries, so
// weights keep flowing while a unit's partial sums meet in shared memory. Units
// of the non-empty segments only are dealt, evenly, so a batch that touches
// few experts still uses every SM.
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = W4_WARPS * 32;
// Ring stages: with 32 token rows a unit the partial sums take a stage's room.
template <int NT> constexpr int w4_stages() { return NT == 4 ? 3 : 4; }
constexpr int W4_CHUNK = 128;                       // k of one ring stage
constexpr int W4_MAT_BYTES = 16 * W4_CHUNK / 2;     // 16 rows of codes
constexpr int W4_SC_BYTES = 32 * 16;                // scales and zeros, 16 bytes a lane

__device__ __forceinline__ uint32_t w4_smem(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes, or zeros where !valid (nothing is read then).
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The four bf16 pairs (ci - z, c(i+4) - z), z128 = 128 + zero in both halves.
__device__ __forceinline__ void unpack_w4(uint32_t w, uint32_t z128, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                     *reinterpret_cast<const __nv_bfloat162*>(&z128));
    p[i] = *reinterpret_cast<const uint32_t*>(&d);
  }
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

template <int MATS, int NT>
__global__ void __launch_bounds__(W4_THREADS, 2) w4_gemm_kernel(const W4GemmParams p, int WK) {
  constexpr int W4_STAGES = w4_stages<NT>();
  constexpr int STAGE = MATS * W4_MAT_BYTES + W4_SC_BYTES;
  constexpr int RED = MATS * NT * 32;                     // float4s of one warp's partial sums
  extern __shared__ __align__(128) uint8_t w4_dyn[];
  __shared__ int warp_n[W4_WARPS];
  __shared__ long long warp_u[W4_WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int WM = W4_WARPS / WK, wk = warp % WK, wm = warp / WK;
  uint8_t* ring = w4_dyn + (size_t)warp * W4_STAGES * STAGE;
  float4* red = reinterpret_cast<float4*>(w4_dyn + (size_t)W4_WARPS * W4_STAGES * STAGE);
  W4Entry* tab = reinterpret_cast<W4Entry*>(red + W4_WARPS * RED);

  // -------------------------------------------------- the segments' table
  const int n_seg = p.n_routed + (p.dense_rows > 0 ? 1 : 0);
  const int unit_rows = 16 * WM;
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
    m0 = (rel / passes) * unit_rows + wm * 16;
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
  const int sub_n = W4_CHUNK / p.group;             // groups of a chunk: 1, 2 or 4
  int pu = u0, phint = first_seg, pm0 = 0, pc = wk;
  W4Seg ps = {};
  if (pu < u1) locate(pu, phint, ps, pm0);
  uint16_t sc_r[MATS][2];
  uint8_t z_r[MATS][2];
  int sc_slot = -1;                                  // stage that the loaded scales belong to
#pragma unroll
  for (int a = 0; a < MATS; ++a) sc_r[a][0] = sc_r[a][1] = z_r[a][0] = z_r[a][1] = 0;

  auto store_scales = [&]() {
    if (sc_slot < 0) return;
    uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < MATS; ++a) {
      v[a] = (uint32_t)sc_r[a][0] | ((uint32_t)sc_r[a][1] << 16);
      v[2 + a] = (uint32_t)z_r[a][0] | ((uint32_t)z_r[a][1] << 16);
    }
    *reinterpret_cast<uint4*>(ring + (size_t)sc_slot * STAGE + MATS * W4_MAT_BYTES + lane * 16) =
        make_uint4(v[0], v[1], v[2], v[3]);
    sc_slot = -1;
  };
  // Start the next chunk of this warp's stream into stage `slot`. Its scales
  // come by plain loads and are put into the stage at the next call, when
  // they have arrived.
  auto issue = [&](int slot) {
    store_scales();
    while (pu < u1 && pc >= ceil_div(ps.K, W4_CHUNK)) {
      if (++pu < u1) locate(pu, phint, ps, pm0);
      pc = wk;
    }
    if (pu < u1) {
      const int k0 = pc * W4_CHUNK, groups = ps.K / p.group;
      const uint32_t dst = w4_smem(ring + (size_t)slot * STAGE);
      const int gi = min(k0 / p.group + (q & (sub_n - 1)), groups - 1);
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        const W4Operand& op = ps.op[a];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = g + 8 * h;
          const bool row_ok = pm0 + r < ps.M;
          const size_t row = ps.row0 + (row_ok ? pm0 + r : 0);
          const bool ok = row_ok && k0 + q * 32 < ps.K;
          cp_async16_zfill(dst + a * W4_MAT_BYTES + r * 64 + ((q ^ ((r >> 1) & 3)) * 16),
                           op.q + row * (size_t)(ps.K / 2) + (ok ? (k0 + q * 32) / 2 : 0), ok);
          sc_r[a][h] = __ldg(static_cast<const uint16_t*>(op.scale) + row * groups + gi);
          z_r[a][h] = op.zero ? __ldg(op.zero + row * groups + gi) : (uint8_t)8;
        }
      }
      sc_slot = slot;
      pc += WK;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < W4_STAGES - 1; ++i) issue(i);
  if (p.wait_previous) asm volatile("griddepcontrol.wait;" ::: "memory");

  // ------------------------------------------------------------- products
  int slot = 0, hint = first_seg;
  for (int u = u0; u < u1; ++u) {
    W4Seg sg;
    int m0;
    locate(u, hint, sg, m0);
    const uint4* xrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = t * 8 + g;
      xrow[t] = nullptr;
      if (r < sg.rows) {
        size_t src = sg.t0 + r;
        if (!sg.dense && p.gather) {
          const int v = p.gather[sg.t0 + r];
          src = v >= 0 && v < p.gather_rows ? v : 0;
        }
        xrow[t] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(sg.dense ? p.x_s : p.x) +
                                                 src * (size_t)sg.K);
      }
    }
    float acc[MATS][NT][4];
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[a][t][i] = 0.0f;
    const int nch = ceil_div(sg.K, W4_CHUNK);
    for (int c = wk; c < nch; c += WK) {
      issue(slot == 0 ? W4_STAGES - 1 : slot - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(W4_STAGES - 1) : "memory");
      __syncwarp();
      const uint8_t* st = ring + (size_t)slot * STAGE;
      const uint4 sz = *reinterpret_cast<const uint4*>(st + MATS * W4_MAT_BYTES + lane * 16);
      const uint32_t szv[4] = {sz.x, sz.y, sz.z, sz.w};
      float grp[MATS][NT][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {                  // 32 codes of each row
        const int sub = s * sub_n / 4;               // the chunk's group they belong to
        const bool starts = (s * sub_n) % 4 == 0, ends = ((s + 1) * sub_n) % 4 == 0;
        uint32_t xb[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int k = c * W4_CHUNK + s * 32 + q * 8;
          const uint4 v = xrow[t] && k < sg.K ? *(xrow[t] + k / 8) : make_uint4(0, 0, 0, 0);
          xb[t][0] = __byte_perm(v.x, v.z, 0x5410);
          xb[t][1] = __byte_perm(v.x, v.z, 0x7632);
          xb[t][2] = __byte_perm(v.y, v.w, 0x5410);
          xb[t][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int a = 0; a < MATS; ++a) {
          const uint32_t zz = __shfl_sync(0xffffffffu, szv[2 + a], (lane & 28) | sub);
          const uint32_t z0 = ((zz & 15u) | 0x4300u) * 0x00010001u, z1 = (((zz >> 16) & 15u) | 0x4300u) * 0x00010001u;
          const uint8_t* w = st + a * W4_MAT_BYTES + g * 64 + ((s ^ ((g >> 1) & 3)) * 16) + q * 4;
          uint32_t lo[4], hi[4];
          unpack_w4(*reinterpret_cast<const uint32_t*>(w), z0, lo);
          unpack_w4(*reinterpret_cast<const uint32_t*>(w + 512), z1, hi);
          const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (t > 0 && t * 8 >= sg.rows) break;
            if (starts) grp[a][t][0] = grp[a][t][1] = grp[a][t][2] = grp[a][t][3] = 0.0f;
            mma_16816(grp[a][t], a0, xb[t][0], xb[t][1]);
            mma_16816(grp[a][t], a1, xb[t][2], xb[t][3]);
          }
          if (ends) {
            const uint32_t ss = __shfl_sync(0xffffffffu, szv[a], (lane & 28) | sub);
            const float s0 = __uint_as_float(ss << 16), s1 = __uint_as_float(ss & 0xffff0000u);
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
      if (++slot == W4_STAGES) slot = 0;
    }
    // ------------------------------------------- the K shares meet, epilogue
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        red[warp * RED + (a * NT + t) * 32 + lane] =
            make_float4(acc[a][t][0], acc[a][t][1], acc[a][t][2], acc[a][t][3]);
    __syncthreads();
    const int mu = m0 - wm * 16;                     // the unit's first weight row
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(sg.dense ? p.out_s : p.out);
    const float* redf = reinterpret_cast<const float*>(red);
    for (int i = tid; i < sg.rows * unit_rows; i += W4_THREADS) {
      const int n = i / unit_rows, m = i - n * unit_rows;
      if (mu + m >= sg.M) continue;
      const int r = m & 15;
      const int at = ((n >> 3) * 32 + (r & 7) * 4 + ((n & 7) >> 1)) * 4 + (r >> 3) * 2 + (n & 1);
      float v[MATS];
#pragma unroll
      for (int a = 0; a < MATS; ++a) {
        v[a] = 0.0f;
        for (int w = 0; w < WK; ++w) v[a] += redf[((m >> 4) * WK + w) * RED * 4 + a * NT * 128 + at];
      }
      // One rounding, of the activation (gate/up) or of the result (down).
      const float o = MATS == 2 ? v[0] / (1.0f + __expf(-v[0])) * v[MATS - 1] : v[0];
      out[(size_t)(sg.t0 + n) * sg.M + mu + m] = __float2bfloat16_rn(o);
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

template <int MATS, int NT> int w4_smem_bytes(int n_seg) {
  return W4_WARPS * (w4_stages<NT>() * (MATS * W4_MAT_BYTES + W4_SC_BYTES) + MATS * NT * 512) +
         n_seg * (int)sizeof(W4Entry);
}

// Warps along K. A CTA's time is its units times a warp's chunks in each (and
// about half a chunk of joining the shares); the split that makes this
// smallest for the experts that the batch is expected to touch wins.
int w4_split(const W4GemmParams& p, int slots) {
  double act = 0.0;
  if (p.n_routed > 0 && p.max_rows > 0)
    act = p.n_routed * (1.0 - pow(1.0 - 1.0 / p.n_routed, (double)p.max_rows));
  int best = 1;
  double least = 1e300;
  for (int wk = 1; wk <= W4_WARPS; wk *= 2) {
    const int rows = 16 * (W4_WARPS / wk);
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

// scale = (largest magnitude) / 7 with the codes centred on 8, or (max - min)
// / 15 with a zero point, rounded to bf16 before the codes are taken: the
// rounding costs no accuracy. A group of zeros gets scale 0; one that holds a
// value that is not finite gets a NaN scale, so that it shows.
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ w, long long n8, int lanes,
                                                          uint32_t* __restrict__ q, __nv_bfloat16* __restrict__ scale,
                                                          uint8_t* __restrict__ zero) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  const long long start = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  // Whole warps stay together over the shuffles: n8 is a multiple of `lanes`,
  // a group's lanes are in or out of range together.
  for (long long i = start; i - (threadIdx.x & 31) < n8; i += stride) {
    const bool on = i < n8;
    float f[8];
    if (on) load8(w + i * 8, f);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    float lo = 0.0f, hi = 0.0f;
    int odd = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, f[j]);
      hi = fmaxf(hi, f[j]);
      odd |= !isfinite(f[j]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      odd |= __shfl_xor_sync(0xffffffffu, odd, o);
    }
    const __nv_bfloat16 s16 = __float2bfloat16_rn(zero ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f);
    const float s = __bfloat162float(s16), step = s > 0.0f ? s : 1.0f;
    const float z = zero ? fminf(fmaxf(rintf(-lo / step), 0.0f), 15.0f) : 8.0f;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = fminf(fmaxf(rintf(f[j] / step) + z, 0.0f), 15.0f);
      word |= (uint32_t)c << (4 * j);
    }
    if (on) {
      q[i] = word;
      if (i % lanes == 0) {
        scale[i / lanes] = odd ? __ushort_as_bfloat16(0x7fc0) : s16;
        if (zero) zero[i / lanes] = (uint8_t)z;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const __nv_bfloat16* __restrict__ scale,
                                                            const uint8_t* __restrict__ zero, long long n8, int lanes,
                                                            T* __restrict__ w) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
    const uint32_t word = __ldg(q + i);
    const float s = __bfloat162float(scale[i / lanes]);
    const int z = zero ? (zero[i / lanes] & 15) : 8;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = s * (float)((int)((word >> (4 * j)) & 15u) - z);
    store8(w + i * 8, f);
  }
}

}  // namespace

cudaError_t launch_w4_gemm(const W4GemmParams& p, int num_sms, cudaStream_t s) {
  const int slots = 2 * num_sms;
  // Token rows a unit takes: its segments' mean, with room for the uneven
  // ones (more rows run as further passes over the unit's weights).
  const double mean = p.n_routed > 0 ? (double)p.max_rows / p.n_routed : 0.0;
  const double want = mean > 0.0 ? 2.0 * mean + 2.0 : 0.0;
  const double rows = want > p.dense_rows ? want : p.dense_rows;
  const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  const int wk = w4_split(p, slots);
  const int n_seg = p.n_routed + (p.dense_rows > 0 ? 1 : 0);
  auto go = [&](auto kernel, int smem) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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
  if (p.mats == 2)
    return nt == 1   ? go(w4_gemm_kernel<2, 1>, w4_smem_bytes<2, 1>(n_seg))
           : nt == 2 ? go(w4_gemm_kernel<2, 2>, w4_smem_bytes<2, 2>(n_seg))
                     : go(w4_gemm_kernel<2, 4>, w4_smem_bytes<2, 4>(n_seg));
  return nt == 1   ? go(w4_gemm_kernel<1, 1>, w4_smem_bytes<1, 1>(n_seg))
         : nt == 2 ? go(w4_gemm_kernel<1, 2>, w4_smem_bytes<1, 2>(n_seg))
                   : go(w4_gemm_kernel<1, 4>, w4_smem_bytes<1, 4>(n_seg));
}

cudaError_t launch_w4_quantize(int dtype, const void* w, long long n, int group, void* q, void* scale, void* zero,
                               int num_sms, cudaStream_t s) {
  const long long n8 = n / 8, blocks = ceil_div_ll(n8, 256);
  const int grid = (int)(blocks < 8LL * num_sms ? blocks : 8LL * num_sms);
  auto go = [&](auto kernel, auto* src) {
    kernel<<<grid, 256, 0, s>>>(src, n8, group / 8, static_cast<uint32_t*>(q), static_cast<__nv_bfloat16*>(scale),
                                static_cast<uint8_t*>(zero));
    return cudaGetLastError();
  };
  if (dtype == MOE_DTYPE_F32) return go(w4_quantize_kernel<float>, static_cast<const float*>(w));
  return go(w4_quantize_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16*>(w));
}

cudaError_t launch_w4_dequantize(int dtype, const void* q, const void* scale, const void* zero, long long n, int group,
                                 void* w, int num_sms, cudaStream_t s) {
  const long long n8 = n / 8, blocks = ceil_div_ll(n8, 256);
  const int grid = (int)(blocks < 8LL * num_sms ? blocks : 8LL * num_sms);
  auto go = [&](auto kernel, auto* dst) {
    kernel<<<grid, 256, 0, s>>>(static_cast<const uint32_t*>(q), static_cast<const __nv_bfloat16*>(scale),
                                static_cast<const uint8_t*>(zero), n8, group / 8, dst);
    return cudaGetLastError();
  };
  if (dtype == MOE_DTYPE_F32) return go(w4_dequantize_kernel<float>, static_cast<float*>(w));
  return go(w4_dequantize_kernel<__nv_bfloat16>, static_cast<__nv_bfloat16*>(w));
}

}  // namespace moe

// The RMS norms on both sides of a block, fused with its gate and residual
// scale, and their gradients.
//
// Sparse MoE FFN (DeepSeek-V3 note), eq. 12: the layer is a residual around
// the block, h'_t = u_t + MoE(u_t). In a model the block reads a normalised
// stream and may be normalised itself:
//
//   h' = alpha h + beta g . N(y; w_post)      N(v; w) = v r(v) . (w + w_offset)
//   u  = N(h'; w_pre)                         r(v) = (mean(v^2) + eps)^(-1/2)
//
// with y the block's output, g a gate row shared by `gate_tokens` consecutive
// tokens, and u the next block's input. Either norm and the gate may be absent.
//
// Backward, given du and the gradient dh' that arrives through the stream,
// with n = h' r(h'), z = y r(y), q = du . (w_pre + w_offset):
//
//   dH = dh' + r(h') (q - n mean(q n))        the whole gradient of h'
//   dh = alpha dH
//   p  = beta g . dH . (w_post + w_offset),   dy = r(y) (p - z mean(p z))
//   dw_pre  = sum_t du n
//   with S_j = sum of dH z over the tokens of gate row j:
//   dw_post = sum_j beta g_j S_j,   dg_j = beta (w_post + w_offset) S_j
//
// Both kernels are bound by HBM: forward 4 T d elements, backward 6 T d. A CTA
// owns whole rows, each thread the same 16-byte vectors of every row, so a row
// crosses HBM once in each direction. Rows arrive through a ring of cp.async
// stages in shared memory that is private to each thread (it reads only what
// it copied itself): loads run ahead without registers and without a barrier.
// Each row needs two sums over the block one after the other (y's, then the
// stream's; in the backward the stream's and y's squares, then the branch's);
// the second of one row and the first of the next share a barrier.
//
// Measured, bf16, T = 4096, d = 7168: forward 45 us (235 MB: 5.2 TB/s, 79% of
// the copy rate; 69% of the issue slots), backward 77 to 78 us (353 MB: 4.6 TB/s, 70%),
// 72 of them the rows, 5 the sums over runs (a row's four vectors a thread and the
// sums leave 14 warps an SM, which issue in 62% of the cycles). 4096 x 4096: 31
// and 54 us. Five vectors a thread spill: 4096 x 8192 takes 174 and 296 us, fp32
// 4096 x 4096 126 and 149. fp32, T = 1111, d = 1000: backward 16.4 us, 15.1 on the
// GPU, for 27 MB: 371 runs of three rows and the sums over them. 32 rows of 2048:
// 3.5 us on the GPU.
//
// Weight gradients: in the backward each CTA takes a contiguous run of rows
// and keeps fp32 sums (dw_pre's and the gate's in registers, dw_post's, which
// change with the gate row only, in shared memory); the runs' sums are added in run order by a
// second kernel, so results do not depend on timing. A gate row whose tokens
// all lie in one run is finished by that run; one that straddles runs goes
// through the run's head or tail slot (a run holds at most one of each).
#include "moe_internal.cuh"

namespace moe {
namespace {

// Two 16-byte vectors a thread up to 14 KB rows, then five. 448 threads leave 72
// registers each to two CTAs an SM; one CTA's get 128. Two vectors fit those (20
// bytes spilled in the bf16 forward), five do not: 0.6 KB a thread spilled in the
// bf16 forward, 1.1 in the backward, 0.2 in fp32.
constexpr int kNormMaxThreads = 448;
constexpr int kNormWideVpt = 5;
constexpr int kNormMaxStages = 4;
constexpr int kNormSmem = 216 * 1024;   // of an SM

template <typename T> __device__ __forceinline__ void unpack16(const uint4& v, float (&f)[Vec16<T>::N]);
template <> __device__ __forceinline__ void unpack16<float>(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T> __device__ __forceinline__ uint4 pack16(const float (&f)[Vec16<T>::N]);
template <> __device__ __forceinline__ uint4 pack16<float>(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <> __device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void cp_async16(uint4* dst, const uint4* src) {
  const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most `pending` (0 .. kNormMaxStages - 1) of this thread's newest groups are still in flight.
__device__ __forceinline__ void cp_async_wait(int pending) {
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

// Sums of four values over the block, the same bits in every thread. `buf`
// alternates between calls: the barrier of one call separates the reads of
// the call before it from the writes of the call after it. Within a warp the
// four are reduced together (each exchange halves the values a lane holds): 6
// shuffles instead of 20, and as many again over the warps' sums.
__device__ __forceinline__ void block_sum4(float (&v)[4], float* red, int& buf) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  auto fold = [&](float a0, float a1, float a2, float a3) -> float {   // lane's value index: bits 4 and 3
    const bool up = lane & 16, hi = lane & 8;
    const float b0 = (up ? a2 : a0) + __shfl_xor_sync(0xffffffffu, up ? a0 : a2, 16);
    const float b1 = (up ? a3 : a1) + __shfl_xor_sync(0xffffffffu, up ? a1 : a3, 16);
    float c = (hi ? b1 : b0) + __shfl_xor_sync(0xffffffffu, hi ? b0 : b1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
  };
  float c = fold(v[0], v[1], v[2], v[3]);
  if (nw > 1) {
    float* r = red + buf * (4 * 32);
    buf ^= 1;
    if ((lane & 7) == 0) r[(lane >> 3) * 32 + w] = c;   // value lane >> 3 of this warp
    __syncthreads();
    static_assert(kNormMaxThreads <= 16 * 32, "two sums a lane");
    const int i = lane & 7;
    c = (i < nw ? r[(lane >> 3) * 32 + i] : 0.0f) + (i + 8 < nw ? r[(lane >> 3) * 32 + i + 8] : 0.0f);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, c, i * 8);
}

// Ring of rows: `stages` slots of ARRAYS x VPT vectors per thread. Vectors past
// the row's end and arrays that are absent stay zero from the start, so that
// readers need no case of their own. Every call of fetch commits one group, so
// that a wait can count rows.
template <int ARRAYS, int VPT>
struct RowRing {
  uint4* base;
  int nt, nv, stages;
  __device__ __forceinline__ const uint4* slot(int st) const { return base + (size_t)st * ARRAYS * VPT * nt; }
  __device__ __forceinline__ uint4 get(const uint4* slot, int array, int j) const {
    return slot[(array * VPT + j) * nt];
  }
  __device__ __forceinline__ void clear(const uint4* const (&src)[ARRAYS]) const {
    for (int st = 0; st < stages; ++st)
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a)
          if (!src[a] || (int)threadIdx.x + j * nt >= nv)
            base[((size_t)st * ARRAYS * VPT + a * VPT + j) * nt] = make_uint4(0, 0, 0, 0);
  }
  // The row whose first vector of this thread is `off` vectors into each array.
  __device__ __forceinline__ void fetch(const uint4* const (&src)[ARRAYS], size_t off, bool on, int st) const {
    if (on) {
      uint4* to = base + (size_t)st * ARRAYS * VPT * nt;
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a)
        if (src[a]) {
          const uint4* from = src[a] + off;
#pragma unroll
          for (int j = 0; j < VPT; ++j)
            if ((int)threadIdx.x + j * nt < nv) cp_async16(to + (a * VPT + j) * nt, from + j * nt);
        }
    }
    cp_async_commit();
  }
};

// The branch's factor per column, beta g (w_post + offset), 1 for what is
// absent. The gate row comes in ahead (packed), w_post from the caches.
template <typename T, int VPT>
struct BranchWeight {
  static constexpr int N = Vec16<T>::N;
  const uint4* gate;        // or null
  const uint4* w_post;      // or null
  float beta, w_offset;
  int nt, nv;
  uint4 next[VPT];
  __device__ __forceinline__ int col(int j) const { return min((int)threadIdx.x + j * nt, nv - 1); }
  __device__ __forceinline__ void load(int row) {
    if (!gate) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j) next[j] = __ldg(gate + (size_t)row * nv + col(j));
  }
  __device__ __forceinline__ void post_weights(int j, float (&w)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 1.0f;
    if (w_post) {
      unpack16<T>(__ldg(w_post + col(j)), w);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] += w_offset;
    }
  }
  __device__ __forceinline__ void open(float (&out)[VPT][N]) const {   // of the row loaded last
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float w[N], g[N];
      post_weights(j, w);
      if (gate) unpack16<T>(next[j], g);
#pragma unroll
      for (int i = 0; i < N; ++i) out[j][i] = beta * w[i] * (gate ? g[i] : 1.0f);
    }
  }
};

template <typename T, int VPT>
__global__ void __launch_bounds__(kNormMaxThreads, 2) residual_norm_kernel(const NormParams p, int stages) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ uint4 ring_mem[];
  __shared__ float red[2 * 4 * 32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.d / N;
  const bool has_y = p.y != nullptr, post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const uint4* const src[2] = {static_cast<const uint4*>(p.h), static_cast<const uint4*>(p.y)};
  const RowRing<2, VPT> ring = {ring_mem + tid, nt, nv, stages};
  uint4* h_out = static_cast<uint4*>(p.h_out);
  uint4* u = static_cast<uint4*>(p.u);
  const float inv_d = 1.0f / (float)p.d;
  int buf = 0;

  // Row k of this CTA: rows are dealt in turn, so that CTAs work on neighbours.
  const int rows = p.T > (int)blockIdx.x ? (p.T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  // Offsets run along: of the row to fetch, of the row at hand.
  const size_t row_step = (size_t)gridDim.x * nv;
  size_t off_in = (size_t)blockIdx.x * nv + tid, off = off_in;
  auto fetch = [&](int k, int st) {
    ring.fetch(src, off_in, k < rows, st);
    off_in += row_step;
  };
  ring.clear(src);
  for (int k = 0; k < stages - 1; ++k) fetch(k, k);

  uint4 wpre[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    wpre[j] = pre ? __ldg(static_cast<const uint4*>(p.w_pre) + min(tid + j * nt, nv - 1)) : make_uint4(0, 0, 0, 0);
  BranchWeight<T, VPT> branch = {static_cast<const uint4*>(p.gate), static_cast<const uint4*>(p.w_post), p.beta,
                                 p.w_offset, nt, nv};
  float wbr[VPT][N];
  // The row's gate row and its place in it, and a step's part in each.
  int gate_row = (int)blockIdx.x / p.gate_tokens, in_gate = (int)blockIdx.x - gate_row * p.gate_tokens;
  const int gate_step = (int)gridDim.x / p.gate_tokens, in_step = (int)gridDim.x - gate_step * p.gate_tokens;
  if (rows > 0) {
    branch.load(gate_row);
    branch.open(wbr);
  }
  auto sum_y = [&](const uint4* slot) -> float {     // this thread's share of y's squares
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[N];
      unpack16<T>(ring.get(slot, 1, j), f);
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
    }
    return s;
  };
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};             // y's squares of the row to come, the stream's
  if (post && rows > 0) {
    cp_async_wait(stages - 2);
    s[0] = sum_y(ring.slot(0));
    block_sum4(s, red, buf);
  }
  int st = 0;
  for (int k = 0; k < rows; ++k) {
    const int next = st + 1 == stages ? 0 : st + 1;
    fetch(k + stages - 1, st == 0 ? stages - 1 : st - 1);
    cp_async_wait(stages - 1);
    const uint4* slot = ring.slot(st);
    float o[VPT][N], sh = 0.0f;
    const float ry = post ? rsqrtf(s[0] * inv_d + p.eps) : 1.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[N];
      unpack16<T>(ring.get(slot, 0, j), o[j]);
      unpack16<T>(ring.get(slot, 1, j), f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        o[j][i] = fmaf(ry, f[i] * wbr[j][i], p.alpha * o[j][i]);
        sh = fmaf(o[j][i], o[j][i], sh);
      }
      if (has_y && tid + j * nt < nv) h_out[off + j * nt] = pack16<T>(o[j]);
    }
    const bool more = k + 1 < rows;
    int next_gate = gate_row;
    if (more && p.gate) {
      next_gate += gate_step;
      in_gate += in_step;
      if (in_gate >= p.gate_tokens) {
        in_gate -= p.gate_tokens;
        ++next_gate;
      }
      if (next_gate != gate_row) branch.load(next_gate);
    }
    if (more && post) {
      cp_async_wait(stages - 2);
      s[0] = sum_y(ring.slot(next));
    }
    s[1] = sh;
    if (pre || (more && post)) block_sum4(s, red, buf);
    if (pre) {
      // The norm reads the stream in fp32, before the rounding that h_out
      // takes: u is rounded once.
      const float r = rsqrtf(s[1] * inv_d + p.eps), ro = r * p.w_offset;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float w[N];
        unpack16<T>(wpre[j], w);
#pragma unroll
        for (int i = 0; i < N; ++i) o[j][i] *= fmaf(r, w[i], ro);
        if (tid + j * nt < nv) u[off + j * nt] = pack16<T>(o[j]);
      }
    }
    off += row_step;
    if (next_gate != gate_row) {
      gate_row = next_gate;
      branch.open(wbr);
    }
    st = next;
  }
}

// Per run c: sums[0][c] dw_post, sums[1][c] dw_pre, sums[2][c] / sums[3][c]
// the head and tail slots of the gate's gradient, each [d] fp32. PIPE: the
// ring holds two rows at least, and a row's first sums are taken with the last
// of the row before; else (rows past 25 KB) they have a barrier of their own.
template <typename T, int VPT, bool PIPE>
__global__ void __launch_bounds__(kNormMaxThreads, 1)
    residual_norm_bwd_kernel(const NormBwdParams p, int stages, int rows_per_run) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ uint4 ring_mem[];
  __shared__ float red[2 * 4 * 32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.d / N;
  const bool has_y = p.y != nullptr, post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const uint4* const src[4] = {static_cast<const uint4*>(p.h_out), static_cast<const uint4*>(p.y),
                               static_cast<const uint4*>(p.du), static_cast<const uint4*>(p.dh_out)};
  const RowRing<4, VPT> ring = {ring_mem + tid, nt, nv, stages};
  const float inv_d = 1.0f / (float)p.d;
  int buf = 0;
  // T may be the largest int: nothing is added to a token's number before it is
  // known to stay below T.
  const int t0 = blockIdx.x * rows_per_run, t1 = t0 + min(p.T - t0, rows_per_run);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the reduction may line up
  const int gt = p.gate ? p.gate_tokens : p.T;   // without a gate: one group
  size_t off_in = (size_t)t0 * nv + tid, off = off_in;   // of the row to fetch, of the row at hand
  auto fetch = [&](bool on, int st) {
    ring.fetch(src, off_in, on, st);
    off_in += nv;
  };
  ring.clear(src);
  for (int i = 0; i < stages - 1; ++i) fetch(i < t1 - t0, i);

  float wpre[VPT][N], wbr[VPT][N];               // fp32, offsets and beta in
  float acc_pre[VPT][N], acc_s[VPT][N];
  // dw_post's sums move on only where a gate row closes: in shared memory,
  // behind the ring, each thread its own.
  float4* acc_post = reinterpret_cast<float4*>(ring_mem + (size_t)stages * 4 * VPT * nt) + tid;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    unpack16<T>(pre ? __ldg(static_cast<const uint4*>(p.w_pre) + min(tid + j * nt, nv - 1)) : make_uint4(0, 0, 0, 0),
                wpre[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      wpre[j][i] += p.w_offset;
      acc_pre[j][i] = acc_s[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) acc_post[(j * (N / 4) + i) * nt] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  BranchWeight<T, VPT> branch = {static_cast<const uint4*>(p.gate), static_cast<const uint4*>(p.w_post), p.beta,
                                 p.w_offset, nt, nv};
  int grp = t0 / gt, left = gt - (t0 - grp * gt);        // gate row, its tokens from this row on
  bool begins = left == gt;                              // whether it began in this run
  if (t0 < t1) {
    branch.load(grp);
    branch.open(wbr);
  }
  // This thread's shares of the sums of h'^2, q h', y^2.
  auto first_sums = [&](const uint4* slot, float (&s)[4]) {
    s[0] = s[1] = s[2] = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float f[N], q[N];
      unpack16<T>(ring.get(slot, 0, j), f);
      unpack16<T>(ring.get(slot, 2, j), q);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[0] = fmaf(f[i], f[i], s[0]);
        s[1] = fmaf(q[i] * wpre[j][i], f[i], s[1]);
      }
      unpack16<T>(ring.get(slot, 1, j), f);
#pragma unroll
      for (int i = 0; i < N; ++i) s[2] = fmaf(f[i], f[i], s[2]);
    }
  };

  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (PIPE && t0 < t1) {
    cp_async_wait(stages - 2);
    first_sums(ring.slot(0), s);
    block_sum4(s, red, buf);
  }
  int st = 0;
  for (int t = t0; t < t1; ++t) {
    fetch(stages - 1 < t1 - t, st == 0 ? stages - 1 : st - 1);
    cp_async_wait(stages - 1);
    const uint4* slot = ring.slot(st);
    const int next = st + 1 == stages ? 0 : st + 1;
    if (!PIPE) {
      first_sums(slot, s);
      s[3] = 0.0f;
      block_sum4(s, red, buf);
    }
    const float rh = pre ? rsqrtf(s[0] * inv_d + p.eps) : 0.0f, ry = post ? rsqrtf(s[2] * inv_d + p.eps) : 1.0f;
    // r mean(q n), formed so that nothing leaves fp32's range before the result
    // does: r^3 by itself is lost past an RMS of 1e13 and infinite below 1e-13.
    const float ch = rh * (rh * s[1] * inv_d);
    float dm[VPT][N], sy = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float dH[N], f[N], q[N];
      unpack16<T>(ring.get(slot, 3, j), dH);
      unpack16<T>(ring.get(slot, 0, j), f);
      unpack16<T>(ring.get(slot, 2, j), q);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc_pre[j][i] = fmaf(q[i] * rh, f[i], acc_pre[j][i]);
        dH[i] = fmaf(rh, fmaf(-ch, f[i], q[i] * wpre[j][i]), dH[i]);
      }
      if (p.dh && tid + j * nt < nv) {
        float a[N];
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = p.alpha * dH[i];
        static_cast<uint4*>(p.dh)[off + j * nt] = pack16<T>(a);
      }
      unpack16<T>(ring.get(slot, 1, j), f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc_s[j][i] = fmaf(dH[i], f[i] * ry, acc_s[j][i]);
        dm[j][i] = dH[i] * wbr[j][i];
        sy = fmaf(dm[j][i], f[i], sy);
      }
    }
    // The last row of its gate row, or of the run: its sums go out below.
    const bool ends = --left == 0 || t + 1 == p.T, close = ends || t + 1 == t1;
    if (close && t + 1 < t1) branch.load(grp + 1);
    const bool ahead = PIPE && t + 1 < t1;
    if (ahead) {
      cp_async_wait(stages - 2);
      first_sums(ring.slot(next), s);
    }
    s[3] = sy;
    if (ahead || post) block_sum4(s, red, buf);
    if (p.dy) {
      const float cy = post ? ry * (ry * s[3] * inv_d) : 0.0f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float f[N] = {}, o[N];
        if (post) unpack16<T>(ring.get(slot, 1, j), f);   // without a norm no y: it may be infinite
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = ry * fmaf(-cy, f[i], dm[j][i]);
        if (tid + j * nt < nv) static_cast<uint4*>(p.dy)[off + j * nt] = pack16<T>(o);
      }
    }
    if (has_y && close) {
      float* slot_f = nullptr;
      if (!(begins && ends)) slot_f = p.partial + ((size_t)(begins ? 3 : 2) * gridDim.x + blockIdx.x) * p.d;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float w[N], g[N], o[N];
        branch.post_weights(j, w);
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = 1.0f;
        if (p.gate) unpack16<T>(__ldg(static_cast<const uint4*>(p.gate) + (size_t)grp * nv + branch.col(j)), g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          o[i] = p.beta * acc_s[j][i];
          acc_s[j][i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          float4& a = acc_post[(j * (N / 4) + i / 4) * nt];
          a.x = fmaf(o[i], g[i], a.x);
          a.y = fmaf(o[i + 1], g[i + 1], a.y);
          a.z = fmaf(o[i + 2], g[i + 2], a.z);
          a.w = fmaf(o[i + 3], g[i + 3], a.w);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= w[i];
        if (p.dgate && tid + j * nt < nv) {
          if (slot_f) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
              *reinterpret_cast<float4*>(slot_f + (size_t)(tid + j * nt) * N + i) =
                  make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else {
            static_cast<uint4*>(p.dgate)[(size_t)grp * nv + tid + j * nt] = pack16<T>(o);
          }
        }
      }
      if (t + 1 < t1) branch.open(wbr);
    }
    if (left == 0) {
      ++grp;
      left = gt;
      begins = true;
    }
    off += nv;
    st = next;
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (tid + j * nt >= nv) continue;
    const size_t c = (size_t)(tid + j * nt) * N;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      if (p.dw_post)
        *reinterpret_cast<float4*>(p.partial + (size_t)blockIdx.x * p.d + c + i) =
            acc_post[(j * (N / 4) + i / 4) * nt];
      if (p.dw_pre)
        *reinterpret_cast<float4*>(p.partial + (size_t)(gridDim.x + blockIdx.x) * p.d + c + i) =
            make_float4(acc_pre[j][i], acc_pre[j][i + 1], acc_pre[j][i + 2], acc_pre[j][i + 3]);
    }
  }
}

// Adds the runs' sums in run order. blockIdx.y = 0: dw_post, 1: dw_pre, from 2
// on: a gate row that straddles runs, by its own number, or (`by_run`, where
// there are fewer runs than gate rows) by the run it begins in. 128
// columns, four a thread, by 16 slices of the runs per block.
template <typename T>
__global__ void __launch_bounds__(512) norm_reduce_kernel(const NormBwdParams p, int runs, int rows_per_run,
                                                          int by_run) {
  __shared__ float4 part[16][32];
  const int col = (blockIdx.x * 32 + threadIdx.x) * 4;    // d is a multiple of 4
  const int what = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the runs' sums
  T* out = nullptr;
  const float* first = nullptr;   // one row outside the sequence, added first
  const float* base = nullptr;
  int n = 0;
  if (what == 0) {
    out = static_cast<T*>(p.dw_post);
    base = p.partial;
    n = runs;
  } else if (what == 1) {
    out = static_cast<T*>(p.dw_pre);
    base = p.partial + (size_t)runs * p.d;
    n = runs;
  } else {
    // The gate row of the last token of a run is the only one that can begin
    // in it and go on.
    const long long gt = p.gate_tokens;
    const long long grp = by_run ? ((what - 2 + 1LL) * rows_per_run - 1) / gt : what - 2;
    const long long begin = grp * gt, end = min(begin + gt, (long long)p.T);
    const int c = (int)(begin / rows_per_run), last = (int)((end - 1) / rows_per_run);
    if (last == c || (by_run && c != what - 2)) return;
    out = static_cast<T*>(p.dgate) + (size_t)grp * p.d;
    first = p.partial + ((size_t)3 * runs + c) * p.d;
    base = p.partial + ((size_t)2 * runs + c + 1) * p.d;
    n = last - c;
  }
  if (!out) return;
  const int per = ceil_div(n, 16);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4 v) {
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  };
  if (col < p.d) {
    if (first && threadIdx.y == 0) add(*reinterpret_cast<const float4*>(first + col));
    const int i1 = min(n, (int)(threadIdx.y + 1) * per);
#pragma unroll 8
    for (int i = threadIdx.y * per; i < i1; ++i) add(*reinterpret_cast<const float4*>(base + (size_t)i * p.d + col));
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < p.d) {
    s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 16; ++i) add(part[i][threadIdx.x]);
    out[col] = from_f32<T>(s.x);
    out[col + 1] = from_f32<T>(s.y);
    out[col + 2] = from_f32<T>(s.z);
    out[col + 3] = from_f32<T>(s.w);
  }
}

struct NormShape {
  int vpt, threads, ctas_per_sm, stages, smem;
};
// One 16-byte vector a thread where 32 threads cover a row, else two, else
// five; CTAs fill `per_sm` threads an SM and share 216 KB of shared memory.
NormShape norm_shape(int dtype, int d, int arrays, int per_sm, int more) {   // more: bytes a thread and vector
  const int nv = d / (dtype == MOE_DTYPE_F32 ? 4 : 8);
  NormShape s;
  s.vpt = nv > 2 * kNormMaxThreads ? kNormWideVpt : nv > 32 ? 2 : 1;
  s.threads = ceil_div(ceil_div(nv, s.vpt), 32) * 32;
  s.ctas_per_sm = per_sm / s.threads;
  if (s.ctas_per_sm > 16) s.ctas_per_sm = 16;
  if (s.ctas_per_sm < 1) s.ctas_per_sm = 1;
  const int row = arrays * s.vpt * s.threads * 16;
  more *= s.vpt * s.threads;
  if (kNormSmem / s.ctas_per_sm - more < 2 * row) s.ctas_per_sm = 1;
  s.stages = (kNormSmem / s.ctas_per_sm - more) / row;
  if (s.stages > kNormMaxStages) s.stages = kNormMaxStages;
  if (s.stages < 1) s.stages = 1;
  s.smem = s.stages * row + more;
  return s;
}

}  // namespace

bool norm_width_supported(int dtype, int d) {
  return (long long)d * (dtype == MOE_DTYPE_F32 ? 4 : 2) <= 32768;
}

int norm_backward_runs(int dtype, int T, int d, int num_sms) {
  const long long n = (long long)norm_shape(dtype, d, 4, kNormMaxThreads, dtype == MOE_DTYPE_F32 ? 16 : 32).ctas_per_sm * num_sms;
  const long long per = ceil_div_ll(T, n < T ? n : T);
  return (int)ceil_div_ll(T, per);
}

cudaError_t launch_residual_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.dtype, p.d, 2, 2 * kNormMaxThreads, 0);
  const long long slots = (long long)sh.ctas_per_sm * num_sms;
  const int grid = (int)(slots < p.T ? slots : p.T);
  auto go = [&](auto tag) {
    constexpr auto kernel = decltype(tag)::value;
    const cudaError_t e = allow_max_smem<kernel>();
    if (e != cudaSuccess) return e;
    kernel<<<grid, sh.threads, sh.smem, s>>>(p, sh.stages);
    return cudaGetLastError();
  };
  auto with = [&](auto zero) {
    using T = decltype(zero);
    return sh.vpt == 1   ? go(KernelTag<residual_norm_kernel<T, 1>>{})
           : sh.vpt == 2 ? go(KernelTag<residual_norm_kernel<T, 2>>{})
                         : go(KernelTag<residual_norm_kernel<T, kNormWideVpt>>{});
  };
  return p.dtype == MOE_DTYPE_F32 ? with(float{}) : with(__nv_bfloat16{});
}

cudaError_t launch_residual_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.dtype, p.d, 4, kNormMaxThreads, p.dtype == MOE_DTYPE_F32 ? 16 : 32);
  const int runs = norm_backward_runs(p.dtype, p.T, p.d, num_sms);
  const int per = (int)ceil_div_ll(p.T, runs);
  auto go = [&](auto tag) {
    constexpr auto kernel = decltype(tag)::value;
    const cudaError_t e = allow_max_smem<kernel>();
    if (e != cudaSuccess) return e;
    kernel<<<runs, sh.threads, sh.smem, s>>>(p, sh.stages, per);
    return cudaGetLastError();
  };
  auto with = [&](auto zero) {
    using T = decltype(zero);
    return sh.vpt == 1       ? go(KernelTag<residual_norm_bwd_kernel<T, 1, true>>{})
           : sh.vpt == 2     ? go(KernelTag<residual_norm_bwd_kernel<T, 2, true>>{})
           : sh.stages >= 2  ? go(KernelTag<residual_norm_bwd_kernel<T, kNormWideVpt, true>>{})
                             : go(KernelTag<residual_norm_bwd_kernel<T, kNormWideVpt, false>>{});
  };
  const cudaError_t e = p.dtype == MOE_DTYPE_F32 ? with(float{}) : with(__nv_bfloat16{});
  if (e != cudaSuccess || !(p.dw_post || p.dw_pre || p.dgate)) return e;
  // No gate row straddles runs of whole gate rows.
  const int gates = (int)ceil_div_ll(p.T, p.gate_tokens), by_run = gates > runs - 1;
  const int straddle = !p.dgate || per % p.gate_tokens == 0 ? 0 : by_run ? runs - 1 : gates;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(p.d, 128), 2 + straddle);
  cfg.blockDim = dim3(32, 16);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return p.dtype == MOE_DTYPE_F32 ? cudaLaunchKernelEx(&cfg, norm_reduce_kernel<float>, p, runs, per, by_run)
                                  : cudaLaunchKernelEx(&cfg, norm_reduce_kernel<__nv_bfloat16>, p, runs, per, by_run);
}

}  // namespace moe

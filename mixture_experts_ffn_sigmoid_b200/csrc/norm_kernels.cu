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
// crosses HBM once in each direction and stays in registers over both of its
// reductions. Rows arrive through a ring of cp.async stages in shared memory
// that is private to each thread (it reads only what it copied itself): the
// loads of the next rows run on while a row's block reductions wait, without
// registers for them and without a barrier.
//
// Weight gradients: in the backward each CTA takes a contiguous run of rows
// and keeps fp32 sums in registers; the runs' sums are added in run order by a
// second kernel, so results do not depend on timing. A gate row whose tokens
// all lie in one run is finished by that run; one that straddles runs goes
// through the run's head or tail slot (a run holds at most one of each).
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxStages = 4;

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

// Sum of N values over the block, the same bits in every thread. `buf`
// alternates between calls: the barrier of one call separates the reads of
// the call before it from the writes of the call after it.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* red, int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return;
  float* r = red + buf * (3 * 32);
  buf ^= 1;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[i * 32 + w] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < nw ? r[i * 32 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kNormMaxThreads) residual_norm_kernel(const NormParams p, int stages) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ uint4 ring[];   // [stages][h, y][VPT][threads]
  __shared__ float red[2 * 3 * 32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.d / N;
  const bool has_y = p.y != nullptr, post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const uint4* h = static_cast<const uint4*>(p.h);
  const uint4* y = static_cast<const uint4*>(p.y);
  uint4* h_out = static_cast<uint4*>(p.h_out);
  uint4* u = static_cast<uint4*>(p.u);
  const float inv_d = 1.0f / (float)p.d;
  int buf = 0;

  uint4 wpost[VPT], wpre[VPT], gate[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * nt;
    wpost[j] = wpre[j] = gate[j] = make_uint4(0, 0, 0, 0);
    if (v < nv && post) wpost[j] = __ldg(static_cast<const uint4*>(p.w_post) + v);
    if (v < nv && pre) wpre[j] = __ldg(static_cast<const uint4*>(p.w_pre) + v);
  }
  int gate_row = -1;

  auto fetch = [&](int t, int st) {
    if (t < p.T) {
      uint4* slot = ring + (size_t)st * 2 * VPT * nt + tid;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * nt;
        if (v < nv) {
          cp_async16(slot + j * nt, h + (size_t)t * nv + v);
          if (has_y) cp_async16(slot + (VPT + j) * nt, y + (size_t)t * nv + v);
        }
      }
    }
    cp_async_commit();
  };
  // Rows are dealt in turn: consecutive CTAs work on neighbouring rows.
  for (int i = 0; i < stages - 1; ++i) fetch(blockIdx.x + i * gridDim.x, i);
  int st = 0;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const long long ahead = (long long)t + (long long)(stages - 1) * gridDim.x;
    fetch(ahead < p.T ? (int)ahead : p.T, st == 0 ? stages - 1 : st - 1);
    if (p.gate && t / p.gate_tokens != gate_row) {
      gate_row = t / p.gate_tokens;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < nv)
          gate[j] = __ldg(static_cast<const uint4*>(p.gate) + (size_t)gate_row * nv + tid + j * nt);
    }
    cp_async_wait(stages - 1);
    const uint4* slot = ring + (size_t)st * 2 * VPT * nt + tid;
    if (++st == stages) st = 0;
    float o[VPT][N], s[1] = {0.0f};
    uint4 yv[VPT];
    if (has_y) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) yv[j] = tid + j * nt < nv ? slot[(VPT + j) * nt] : make_uint4(0, 0, 0, 0);
      float ry = p.beta;
      if (post) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          float f[N];
          unpack16<T>(yv[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) s[0] = fmaf(f[i], f[i], s[0]);
        }
        block_sum(s, red, buf);
        ry *= rsqrtf(s[0] * inv_d + p.eps);
        s[0] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float f[N], w[N], g[N];
        unpack16<T>(tid + j * nt < nv ? slot[j * nt] : make_uint4(0, 0, 0, 0), o[j]);
        unpack16<T>(yv[j], f);
        unpack16<T>(wpost[j], w);
        unpack16<T>(gate[j], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float b = f[i] * ry;
          if (post) b *= w[i] + p.w_offset;
          if (p.gate) b *= g[i];
          o[j][i] = fmaf(p.alpha, o[j][i], b);
          s[0] = fmaf(o[j][i], o[j][i], s[0]);
        }
        if (tid + j * nt < nv) h_out[(size_t)t * nv + tid + j * nt] = pack16<T>(o[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        unpack16<T>(tid + j * nt < nv ? slot[j * nt] : make_uint4(0, 0, 0, 0), o[j]);
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] = fmaf(o[j][i], o[j][i], s[0]);
      }
    }
    if (pre) {
      // The norm reads the stream in fp32, before the rounding that h_out
      // takes: u is rounded once.
      block_sum(s, red, buf);
      const float r = rsqrtf(s[0] * inv_d + p.eps);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float w[N];
        unpack16<T>(wpre[j], w);
#pragma unroll
        for (int i = 0; i < N; ++i) o[j][i] *= r * (w[i] + p.w_offset);
        if (tid + j * nt < nv) u[(size_t)t * nv + tid + j * nt] = pack16<T>(o[j]);
      }
    }
  }
}

// Per run c: sums[0][c] dw_post, sums[1][c] dw_pre, sums[2][c] / sums[3][c]
// the head and tail slots of the gate's gradient, each [d] fp32.
template <typename T, int VPT>
__global__ void __launch_bounds__(kNormMaxThreads, 1)
    residual_norm_bwd_kernel(const NormBwdParams p, int stages, int rows_per_run) {
  constexpr int N = Vec16<T>::N;
  extern __shared__ uint4 ring[];   // [stages][h_out, y, du, dh_out][VPT][threads]
  __shared__ float red[2 * 3 * 32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.d / N;
  const bool has_y = p.y != nullptr, post = p.w_post != nullptr, pre = p.w_pre != nullptr;
  const uint4* src[4] = {static_cast<const uint4*>(p.h_out), static_cast<const uint4*>(p.y),
                         static_cast<const uint4*>(p.du), static_cast<const uint4*>(p.dh_out)};
  const float inv_d = 1.0f / (float)p.d;
  int buf = 0;
  const int t0 = blockIdx.x * rows_per_run, t1 = min(p.T, t0 + rows_per_run);
  const int gt = p.gate ? p.gate_tokens : p.T;   // without a gate: one group

  uint4 wpost[VPT], wpre[VPT], gate[VPT];
  float acc_post[VPT][N], acc_pre[VPT][N], acc_s[VPT][N];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * nt;
    wpost[j] = wpre[j] = gate[j] = make_uint4(0, 0, 0, 0);
    if (v < nv && post) wpost[j] = __ldg(static_cast<const uint4*>(p.w_post) + v);
    if (v < nv && pre) wpre[j] = __ldg(static_cast<const uint4*>(p.w_pre) + v);
#pragma unroll
    for (int i = 0; i < N; ++i) acc_post[j][i] = acc_pre[j][i] = acc_s[j][i] = 0.0f;
  }
  auto load_gate = [&](int row) {
    if (!p.gate) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (tid + j * nt < nv) gate[j] = __ldg(static_cast<const uint4*>(p.gate) + (size_t)row * nv + tid + j * nt);
  };
  auto fetch = [&](int t, int st) {
    if (t < t1) {
      uint4* slot = ring + (size_t)st * 4 * VPT * nt + tid;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * nt;
        if (v < nv) {
#pragma unroll
          for (int a = 0; a < 4; ++a)
            if (src[a]) cp_async16(slot + (a * VPT + j) * nt, src[a] + (size_t)t * nv + v);
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < stages - 1; ++i) fetch(t0 + i, i);
  if (t0 < t1) load_gate(t0 / gt);
  int st = 0;
  for (int t = t0; t < t1; ++t) {
    fetch(t + stages - 1 < t1 ? t + stages - 1 : t1, st == 0 ? stages - 1 : st - 1);
    cp_async_wait(stages - 1);
    const uint4* slot = ring + (size_t)st * 4 * VPT * nt + tid;
    if (++st == stages) st = 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // sums of h'^2, q h', y^2
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (pre || post) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (tid + j * nt >= nv) continue;
        float f[N], q[N], w[N];
        if (pre) {
          unpack16<T>(slot[j * nt], f);
          unpack16<T>(slot[(2 * VPT + j) * nt], q);
          unpack16<T>(wpre[j], w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            s[0] = fmaf(f[i], f[i], s[0]);
            s[1] = fmaf(q[i] * (w[i] + p.w_offset), f[i], s[1]);
          }
        }
        if (post) {
          unpack16<T>(slot[(VPT + j) * nt], f);
#pragma unroll
          for (int i = 0; i < N; ++i) s[2] = fmaf(f[i], f[i], s[2]);
        }
      }
      block_sum(s, red, buf);
    }
    const float rh = rsqrtf(s[0] * inv_d + p.eps), ry = post ? rsqrtf(s[2] * inv_d + p.eps) : 1.0f;
    const float ch = rh * rh * rh * s[1] * inv_d;
    float dm[VPT][N], sy[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool on = tid + j * nt < nv;
      float dH[N], f[N], w[N], g[N];
      unpack16<T>(on && src[3] ? slot[(3 * VPT + j) * nt] : zero, dH);
      if (pre) {
        float q[N];
        unpack16<T>(on ? slot[j * nt] : zero, f);
        unpack16<T>(on ? slot[(2 * VPT + j) * nt] : zero, q);
        unpack16<T>(wpre[j], w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          acc_pre[j][i] = fmaf(q[i], f[i] * rh, acc_pre[j][i]);
          dH[i] += rh * (q[i] * (w[i] + p.w_offset)) - ch * f[i];
        }
      }
      if (p.dh && on) {
        float a[N];
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = p.alpha * dH[i];
        static_cast<uint4*>(p.dh)[(size_t)t * nv + tid + j * nt] = pack16<T>(a);
      }
      if (has_y) {
        unpack16<T>(on ? slot[(VPT + j) * nt] : zero, f);
        unpack16<T>(wpost[j], w);
        unpack16<T>(gate[j], g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          acc_s[j][i] = fmaf(dH[i], f[i] * ry, acc_s[j][i]);
          float b = p.beta * dH[i];
          if (post) b *= w[i] + p.w_offset;
          if (p.gate) b *= g[i];
          dm[j][i] = b;
          sy[0] = fmaf(b, f[i], sy[0]);
        }
      }
    }
    if (has_y) {
      float cy = 0.0f;
      if (post) {
        block_sum(sy, red, buf);
        cy = ry * ry * ry * sy[0] * inv_d;
      }
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (tid + j * nt >= nv) continue;
        float f[N], o[N];
        unpack16<T>(slot[(VPT + j) * nt], f);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = ry * dm[j][i] - cy * f[i];
        if (p.dy) static_cast<uint4*>(p.dy)[(size_t)t * nv + tid + j * nt] = pack16<T>(o);
      }
      // The last row of its gate row, or of the run.
      const int grp = t / gt;
      const bool ends = (t + 1) % gt == 0 || t + 1 == p.T;
      if (ends || t + 1 == t1) {
        const bool begins = (long long)grp * gt >= t0;
        float* slot_f = nullptr;
        if (!(begins && ends)) slot_f = p.partial + ((size_t)(begins ? 3 : 2) * gridDim.x + blockIdx.x) * p.d;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          if (tid + j * nt >= nv) continue;
          float w[N], g[N], o[N];
          unpack16<T>(wpost[j], w);
          unpack16<T>(gate[j], g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float b = p.beta * acc_s[j][i];
            acc_post[j][i] = fmaf(b, p.gate ? g[i] : 1.0f, acc_post[j][i]);
            o[i] = post ? b * (w[i] + p.w_offset) : b;
            acc_s[j][i] = 0.0f;
          }
          if (p.dgate) {
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
        if (t + 1 < t1) load_gate(grp + 1);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (tid + j * nt >= nv) continue;
    const size_t c = (size_t)(tid + j * nt) * N;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      if (p.dw_post)
        *reinterpret_cast<float4*>(p.partial + (size_t)blockIdx.x * p.d + c + i) =
            make_float4(acc_post[j][i], acc_post[j][i + 1], acc_post[j][i + 2], acc_post[j][i + 3]);
      if (p.dw_pre)
        *reinterpret_cast<float4*>(p.partial + (size_t)(gridDim.x + blockIdx.x) * p.d + c + i) =
            make_float4(acc_pre[j][i], acc_pre[j][i + 1], acc_pre[j][i + 2], acc_pre[j][i + 3]);
    }
  }
}

// Adds the runs' sums in run order. blockIdx.y = 0: dw_post, 1: dw_pre, 2 + c:
// the gate row that begins in run c and goes on past its end. 32 columns by
// 16 slices of the runs per block.
template <typename T>
__global__ void __launch_bounds__(512) norm_reduce_kernel(const NormBwdParams p, int runs, int rows_per_run) {
  __shared__ float part[16][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  const int what = blockIdx.y;
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
  } else if (p.dgate) {
    const int c = what - 2;
    const long long t0 = (long long)c * rows_per_run, t1 = t0 + rows_per_run;   // t1 < T: c is not the last run
    const long long grp = (t1 - 1) / p.gate_tokens;
    if (t1 >= p.T || t1 / p.gate_tokens != grp || grp * p.gate_tokens < t0) return;
    const long long end = min((grp + 1) * (long long)p.gate_tokens, (long long)p.T);
    out = static_cast<T*>(p.dgate) + (size_t)grp * p.d;
    first = p.partial + ((size_t)3 * runs + c) * p.d;
    base = p.partial + ((size_t)2 * runs + c + 1) * p.d;
    n = (int)((end - 1) / rows_per_run) - c;
  }
  if (!out) return;
  const int per = ceil_div(n, 16);
  float s = 0.0f;
  if (col < p.d) {
    if (first && threadIdx.y == 0) s = first[col];
    const int i1 = min(n, (int)(threadIdx.y + 1) * per);
    for (int i = threadIdx.y * per; i < i1; ++i) s += base[(size_t)i * p.d + col];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < p.d) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[i][threadIdx.x];
    out[col] = from_f32<T>(s);
  }
}

struct NormShape {
  int vpt, threads, ctas_per_sm, stages, smem;
};
// A thread takes one 16-byte vector of a row, or two where 1024 threads do not
// cover it; CTAs per SM fill about 1024 threads, and share 200 KB of ring.
NormShape norm_shape(int dtype, int d, int arrays) {
  const int nv = d / (dtype == MOE_DTYPE_F32 ? 4 : 8);
  NormShape s;
  s.vpt = nv > kNormMaxThreads ? 2 : 1;
  s.threads = ceil_div(ceil_div(nv, s.vpt), 32) * 32;
  s.ctas_per_sm = kNormMaxThreads / s.threads;
  if (s.ctas_per_sm > 16) s.ctas_per_sm = 16;
  const int row = arrays * s.vpt * s.threads * 16;
  s.stages = 200 * 1024 / s.ctas_per_sm / row;
  if (s.stages > kNormMaxStages) s.stages = kNormMaxStages;
  if (s.stages < 1) s.stages = 1;
  s.smem = s.stages * row;
  return s;
}

template <typename K>
cudaError_t allow_smem(K kernel, int smem) {
  if (smem <= 32 * 1024) return cudaSuccess;   // with the static arrays below the default 48 KB
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace

bool norm_width_supported(int dtype, int d) {
  return (long long)d * (dtype == MOE_DTYPE_F32 ? 4 : 2) <= 2 * kNormMaxThreads * 16;
}

int norm_backward_runs(int dtype, int T, int d, int num_sms) {
  const long long n = (long long)norm_shape(dtype, d, 4).ctas_per_sm * num_sms;
  const int per = ceil_div(T, (int)(n < T ? n : T));
  return ceil_div(T, per);
}

cudaError_t launch_residual_norm(const NormParams& p, int num_sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.dtype, p.d, 2);
  const long long slots = (long long)sh.ctas_per_sm * num_sms;
  const int grid = (int)(slots < p.T ? slots : p.T);
  auto go = [&](auto kernel) {
    cudaError_t e = allow_smem(kernel, sh.smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, sh.threads, sh.smem, s>>>(p, sh.stages);
    return cudaGetLastError();
  };
  if (p.dtype == MOE_DTYPE_F32)
    return sh.vpt == 1 ? go(residual_norm_kernel<float, 1>) : go(residual_norm_kernel<float, 2>);
  return sh.vpt == 1 ? go(residual_norm_kernel<__nv_bfloat16, 1>) : go(residual_norm_kernel<__nv_bfloat16, 2>);
}

cudaError_t launch_residual_norm_backward(const NormBwdParams& p, int num_sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.dtype, p.d, 4);
  const int runs = norm_backward_runs(p.dtype, p.T, p.d, num_sms);
  const int per = ceil_div(p.T, runs);
  auto go = [&](auto kernel) {
    cudaError_t e = allow_smem(kernel, sh.smem);
    if (e != cudaSuccess) return e;
    kernel<<<runs, sh.threads, sh.smem, s>>>(p, sh.stages, per);
    return cudaGetLastError();
  };
  cudaError_t e;
  if (p.dtype == MOE_DTYPE_F32)
    e = sh.vpt == 1 ? go(residual_norm_bwd_kernel<float, 1>) : go(residual_norm_bwd_kernel<float, 2>);
  else
    e = sh.vpt == 1 ? go(residual_norm_bwd_kernel<__nv_bfloat16, 1>) : go(residual_norm_bwd_kernel<__nv_bfloat16, 2>);
  if (e != cudaSuccess || !(p.dw_post || p.dw_pre || p.dgate)) return e;
  const dim3 grid(ceil_div(p.d, 32), 2 + (p.dgate ? runs - 1 : 0));
  const dim3 block(32, 16);
  if (p.dtype == MOE_DTYPE_F32) norm_reduce_kernel<float><<<grid, block, 0, s>>>(p, runs, per);
  else norm_reduce_kernel<__nv_bfloat16><<<grid, block, 0, s>>>(p, runs, per);
  return cudaGetLastError();
}

}  // namespace moe

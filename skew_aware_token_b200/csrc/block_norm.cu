// The norms before and after the block, with its gate and residual scale, and their gradient.
//
//   n(v; w) = v * rms(v) * (w + w_offset),  rms(v) = rsqrt(mean(v^2) + eps)
//   h' = res_scale h + out_scale g n(y; w_post),   x = bf16(n(h'; w_next))
//
// One pass: a row lives in the registers of a group of warps (8 columns a thread and step),
// so h, y and the weights are read once and h' and x are written once; the two means are two
// reductions over the group.  Bound by HBM.
//
// The gradient needs six sums of a row, and by linearity one reduction for all of them: with
// q = dx (w_next + o), u = dh' + A q - B h', A = rms(h'), B = A^3 <q, h'> / d,
//   <u w_post, y> = <dh' w_post, y> + A <q w_post, y> - B <h' w_post, y>,
// so u itself is not needed before the reduction.  The weights' gradients are kept per column
// in registers over all rows of a CTA, written as one partial row per CTA, and added over
// the CTAs in a fixed order by a second kernel.
#include "train_common.cuh"

namespace moe {
namespace {

// Partial rows of the weight gradients (CTAs of the backward kernel): what the workspace
// holds, four per SM of a 148-SM GPU.
constexpr int kMaxPartials = 592;

struct NormArgs {
  int T, d8, W;  // rows, 8-column steps of a row, warps of a row's group
  float inv_d, eps, w_offset, res_scale, out_scale;
};

// Sum over the group of each of N values, on every thread.  `red` is one of the group's two
// buffers of N * 32 floats; a caller alternates them, so one barrier a reduction is enough.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int W, int group, int warp, int lane,
                                          float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (W == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < W ? red[i * 32 + lane] : 0.f);
}

template <class WT>
__device__ __forceinline__ void load_weight(const WT* w, int v, bool in, float offset,
                                            float* out) {
  if (w && in) {
    load8(w + v * 8, out);
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] += offset;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = 1.f;
  }
}

template <class HT, class WT, int V>
__global__ void __launch_bounds__(1024)
block_norm_kernel(const NormArgs a, const HT* h, const float* __restrict__ y,
                  const float* __restrict__ gate, const WT* __restrict__ w_post,
                  const WT* __restrict__ w_next, HT* h_out, __nv_bfloat16* __restrict__ x) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  float* red = smem + group * 64;
  float wp[V][8], wn[V][8];
  bool in[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = (u * a.W + warp) * 32 + lane;
    in[u] = v < a.d8;
    load_weight(w_post, v, in[u], a.w_offset, wp[u]);
    load_weight(w_next, v, in[u], a.w_offset, wn[u]);
  }
  for (int t = blockIdx.x * groups + group; t < a.T; t += gridDim.x * groups) {
    float hv[V][8], yv[V][8];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const long long at = ((long long)t * a.d8 + (u * a.W + warp) * 32 + lane) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) hv[u][j] = yv[u][j] = 0.f;
      if (in[u]) {
        load8(h + at, hv[u]);
        if (y) load8(y + at, yv[u]);
      }
    }
    if (y) {
      float scale = a.out_scale;
      if (gate) scale *= gate[t];
      if (w_post) {
        float s[1] = {0.f};
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] = fmaf(yv[u][j], yv[u][j], s[0]);
        group_sum(s, a.W, group, warp, lane, red);
        scale *= rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      }
#pragma unroll
      for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          hv[u][j] = fmaf(yv[u][j] * wp[u][j], scale, hv[u][j] * a.res_scale);
        if (in[u])
          store8(h_out + ((long long)t * a.d8 + (u * a.W + warp) * 32 + lane) * 8, hv[u]);
      }
    }
    if (w_next) {
      float s[1] = {0.f};
#pragma unroll
      for (int u = 0; u < V; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (in[u]) s[0] = fmaf(hv[u][j], hv[u][j], s[0]);
      group_sum(s, a.W, group, warp, lane, red + 32);
      const float r = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
      for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int j = 0; j < 8; ++j) hv[u][j] *= r * wn[u][j];
        if (in[u])
          store8(x + ((long long)t * a.d8 + (u * a.W + warp) * 32 + lane) * 8, hv[u]);
      }
    }
  }
}

// A thread owns 8 columns of every row of its group.
template <class HT, class WT>
__global__ void __launch_bounds__(1024)
block_norm_backward_kernel(const NormArgs a, const HT* __restrict__ h_out,
                           const float* __restrict__ y, const float* __restrict__ gate,
                           const WT* __restrict__ w_post, const WT* __restrict__ w_next,
                           const HT* dh_out, const float* __restrict__ dx, HT* dh,
                           float* __restrict__ dy, float* __restrict__ dgate,
                           float* __restrict__ partial) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  float* red = smem + group * (2 * 6 * 32);
  const int v = warp * 32 + lane;
  const bool in = v < a.d8;
  float wp[8], wn[8], gp[8], gn[8];
  load_weight(w_post, v, in, a.w_offset, wp);
  load_weight(w_next, v, in, a.w_offset, wn);
#pragma unroll
  for (int j = 0; j < 8; ++j) gp[j] = gn[j] = 0.f;
  int turn = 0;
  for (int t = blockIdx.x * groups + group; t < a.T; t += gridDim.x * groups, turn ^= 1) {
    const long long at = ((long long)t * a.d8 + v) * 8;
    float hv[8], yv[8], q[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) hv[j] = yv[j] = q[j] = u[j] = 0.f;
    if (in) {
      if (w_next) load8(h_out + at, hv);
      if (y) load8(y + at, yv);
      if (dh_out) load8(dh_out + at, u);
      if (w_next) load8(dx + at, q);
    }
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float qw = q[j] * wn[j], yw = yv[j] * wp[j];
      s[0] = fmaf(hv[j], hv[j], s[0]);
      s[1] = fmaf(qw, hv[j], s[1]);
      s[2] = fmaf(yv[j], yv[j], s[2]);
      s[3] = fmaf(u[j], yw, s[3]);
      s[4] = fmaf(qw, yw, s[4]);
      s[5] = fmaf(hv[j], yw, s[5]);
    }
    group_sum(s, a.W, group, warp, lane, red + turn * (6 * 32));
    float A = 0.f, B = 0.f;
    if (w_next) {
      A = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      B = A * A * A * s[1] * a.inv_d;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      gn[j] = fmaf(q[j] * hv[j], A, gn[j]);
      u[j] = fmaf(A, q[j] * wn[j], fmaf(-B, hv[j], u[j]));
    }
    if (y) {
      const float uy = fmaf(A, s[4], fmaf(-B, s[5], s[3]));
      const float ry = w_post ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 1.f;
      if (gate && threadIdx.x % (a.W * 32) == 0) dgate[t] = a.out_scale * ry * uy;
      const float scale = a.out_scale * (gate ? gate[t] : 1.f) * ry;
      const float back = w_post ? ry * ry * uy * a.inv_d : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gp[j] = fmaf(u[j] * yv[j], scale, gp[j]);
        yv[j] = scale * fmaf(u[j], wp[j], -yv[j] * back);
        u[j] *= a.res_scale;
      }
      if (in) store8(dy + at, yv);
    }
    if (in) store8(dh + at, u);
  }
  // the CTA's partial row: the groups' columns added in group order
  float* col = smem + groups * (2 * 6 * 32);
  for (int g = 0; g < groups; ++g) {
    if (groups > 1) __syncthreads();
    if (group == g && in) {
      if (g > 0) {
        float t8[8];
        load8(col + v * 8, t8);
#pragma unroll
        for (int j = 0; j < 8; ++j) gp[j] += t8[j];
        load8(col + (a.d8 + v) * 8, t8);
#pragma unroll
        for (int j = 0; j < 8; ++j) gn[j] += t8[j];
      }
      float* out = g == groups - 1 ? partial + (long long)blockIdx.x * 2 * a.d8 * 8 : col;
      store8(out + v * 8, gp);
      store8(out + (a.d8 + v) * 8, gn);
    }
  }
}

// dw = sum of `rows` partial rows, 32 columns a CTA, 8 rows at a time.
__global__ void __launch_bounds__(256)
norm_weight_grad_kernel(const float* __restrict__ partial, int rows, int d,
                        float* __restrict__ dw_post, float* __restrict__ dw_next) {
  __shared__ float part[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), lane_row = threadIdx.x >> 5;
  wait_for_predecessor();
  float s = 0.f;
  if (col < 2 * d)
    for (int r = lane_row; r < rows; r += 8) s += partial[(long long)r * 2 * d + col];
  part[lane_row][threadIdx.x & 31] = s;
  __syncthreads();
  if (lane_row == 0 && col < 2 * d) {
#pragma unroll
    for (int r = 1; r < 8; ++r) s += part[r][threadIdx.x & 31];
    if (col < d) {
      if (dw_post) dw_post[col] = s;
    } else if (dw_next) {
      dw_next[col - d] = s;
    }
  }
}

NormArgs make_args(const moe_cfg& c, const moet_norm& n, int V) {
  NormArgs a;
  a.T = c.T;
  a.d8 = c.d / 8;
  a.W = (a.d8 + 32 * V - 1) / (32 * V);
  a.inv_d = 1.f / (float)c.d;
  a.eps = n.eps;
  a.w_offset = n.w_offset;
  a.res_scale = n.res_scale;
  a.out_scale = n.out_scale;
  return a;
}
// row groups of a CTA: about 256 threads
int groups_of(int W) { return W >= 8 ? 1 : 8 / W; }

template <class HT, class WT, int V>
cudaError_t forward(const moe_cfg& c, const moet_norm& n, const void* h, const float* y,
                    const float* gate, const void* wp, const void* wn, void* h_out,
                    uint16_t* x, cudaStream_t st) {
  const NormArgs a = make_args(c, n, V);
  const int groups = groups_of(a.W), threads = groups * a.W * 32;
  const int want = (c.T + groups - 1) / groups, cap = num_sms() * (2048 / threads);
  block_norm_kernel<HT, WT, V><<<want < cap ? want : cap, threads, groups * 64 * 4, st>>>(
      a, static_cast<const HT*>(h), y, gate, static_cast<const WT*>(wp),
      static_cast<const WT*>(wn), static_cast<HT*>(h_out),
      reinterpret_cast<__nv_bfloat16*>(x));
  return cudaGetLastError();
}

template <class HT, class WT>
cudaError_t backward(const moe_cfg& c, const moet_norm& n, const void* h_out, const float* y,
                     const float* gate, const void* wp, const void* wn, const void* dh_out,
                     const float* dx, void* dh, float* dy, float* dgate, float* dw_post,
                     float* dw_next, void* ws, cudaStream_t st) {
  const NormArgs a = make_args(c, n, 1);
  const int groups = groups_of(a.W), threads = groups * a.W * 32;
  const size_t smem = (size_t)groups * 2 * 6 * 32 * 4 + (groups > 1 ? 2 * (size_t)c.d * 4 : 0);
  int grid = (c.T + groups - 1) / groups;
  const int cap = num_sms() * (2048 / threads);
  if (grid > cap) grid = cap;
  if (grid > kMaxPartials) grid = kMaxPartials;
  if (grid > 0) {
    block_norm_backward_kernel<HT, WT><<<grid, threads, smem, st>>>(
        a, static_cast<const HT*>(h_out), y, gate, static_cast<const WT*>(wp),
        static_cast<const WT*>(wn), static_cast<const HT*>(dh_out), dx, static_cast<HT*>(dh),
        dy, dgate, static_cast<float*>(ws));
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (!dw_post && !dw_next) return cudaSuccess;
  return launch_after(norm_weight_grad_kernel, dim3((2 * c.d + 31) / 32), dim3(256), 0, st,
                      static_cast<const float*>(ws), grid, c.d, dw_post, dw_next);
}

}  // namespace

size_t norm_bwd_workspace_bytes(const moe_cfg& c) {
  const size_t rows = c.T < kMaxPartials ? (c.T < 1 ? 1 : c.T) : kMaxPartials;
  return rows * 2 * c.d * sizeof(float);
}

cudaError_t launch_block_norm(const moe_cfg& c, const moet_norm& n, const void* h,
                              const float* y, const float* gate, const void* w_post,
                              const void* w_next, void* h_out, uint16_t* x, cudaStream_t st) {
  if (c.T == 0) return cudaSuccess;
  auto run = [&](auto ht, auto wt) {
    using HT = decltype(ht);
    using WT = decltype(wt);
    if (c.T < num_sms())
      return forward<HT, WT, 1>(c, n, h, y, gate, w_post, w_next, h_out, x, st);
    return forward<HT, WT, 2>(c, n, h, y, gate, w_post, w_next, h_out, x, st);
  };
  const bool hb = n.h_dtype == MOET_BF16, wb = n.w_dtype == MOET_BF16;
  if (hb) return wb ? run(__nv_bfloat16(), __nv_bfloat16()) : run(__nv_bfloat16(), 0.f);
  return wb ? run(0.f, __nv_bfloat16()) : run(0.f, 0.f);
}

cudaError_t launch_block_norm_backward(const moe_cfg& c, const moet_norm& n,
                                       const void* h_out, const float* y, const float* gate,
                                       const void* w_post, const void* w_next,
                                       const void* dh_out, const float* dx, void* dh,
                                       float* dy, float* dgate, float* dw_post,
                                       float* dw_next, void* ws, cudaStream_t st) {
  auto run = [&](auto ht, auto wt) {
    return backward<decltype(ht), decltype(wt)>(c, n, h_out, y, gate, w_post, w_next, dh_out,
                                                dx, dh, dy, dgate, dw_post, dw_next, ws, st);
  };
  const bool hb = n.h_dtype == MOET_BF16, wb = n.w_dtype == MOET_BF16;
  if (hb) return wb ? run(__nv_bfloat16(), __nv_bfloat16()) : run(__nv_bfloat16(), 0.f);
  return wb ? run(0.f, __nv_bfloat16()) : run(0.f, 0.f);
}

}  // namespace moe

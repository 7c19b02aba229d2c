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

constexpr int kFwdThreads = 512;  // of a CTA with several row groups

struct NormArgs {
  int T, d8, W;  // rows, 8-column steps of a row, warps of a row's group
  float inv_d, eps, w_offset, res_scale, out_scale;
  bool whole;  // the fp32 outputs lie on 32 bytes
};

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

// The 8 elements of a lane in its slots: one 16-byte unit of bf16 or two of fp32, units a CTA's
// width apart (consecutive lanes read consecutive 16 bytes).  A lane copies and reads its own
// slots, so no barrier guards them.  The copies go through L1, where the second half of an
// fp32 sector hits: past L1, or with the warp's copies rearranged to runs of 512 bytes, the
// 16384 x 7168 forward took 407 and 295 us for 286.
template <class T>
struct Slots {
  static constexpr int kUnits = sizeof(T) * 8 / 16;
  __device__ static void fill(uint32_t slot, uint32_t pitch, const T* src) {
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      copy_ahead16(slot + i * pitch, reinterpret_cast<const char*>(src) + 16 * i);
  }
  __device__ static void read(uint32_t slot, uint32_t pitch, float* v) {
    if constexpr (kUnits == 1) {
      bf16x8_to_f32(slot16(slot), v);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 a = slot16(slot + i * pitch);
        v[4 * i] = __uint_as_float(a.x), v[4 * i + 1] = __uint_as_float(a.y);
        v[4 * i + 2] = __uint_as_float(a.z), v[4 * i + 3] = __uint_as_float(a.w);
      }
    }
  }
};

// The sum over the group of one value, on every thread.  `red` is one of the group's buffers of
// 32 floats; a caller uses two in turn, so one barrier a sum is enough.
__device__ __forceinline__ float group_sum(float v, int W, int group, int warp, int lane,
                                           float* red) {
  v = warp_sum(v);
  if (W == 1) return v;
  if (lane == 0) red[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
  return warp_sum(lane < W ? red[lane] : 0.f);
}

// A thread owns 8 columns of every row of its group, and their weights.  The next row's
// columns are copied to the thread's slots as soon as this row's are in registers, so that
// memory works through both means of a row (two or three rows ahead gave nothing: they only
// take L1 from the copies).
template <class HT, class WT>
__global__ void __launch_bounds__(1024)
block_norm_kernel(const NormArgs a, const HT* h, const float* __restrict__ y,
                  const float* __restrict__ gate, const WT* __restrict__ w_post,
                  const WT* __restrict__ w_next, HT* h_out, __nv_bfloat16* __restrict__ x) {
  constexpr int HU = Slots<HT>::kUnits;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  const uint32_t pitch = blockDim.x * 16;
  const uint32_t slot_h = smem_addr(smem) + threadIdx.x * 16, slot_y = slot_h + HU * pitch;
  float* red = reinterpret_cast<float*>(smem + (HU + 2) * pitch) + group * 64;
  const int v = warp * 32 + lane;
  const bool in = v < a.d8;
  auto ahead = [&](int t) {
    if (t < a.T && in) {
      const long long at = ((long long)t * a.d8 + v) * 8;
      Slots<HT>::fill(slot_h, pitch, h + at);
      if (y) Slots<float>::fill(slot_y, pitch, y + at);
    }
    commit_copies();
  };
  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + group;
  ahead(t);
  float wp[8], wn[8];
  load_weight(w_post, v, in, a.w_offset, wp);
  load_weight(w_next, v, in, a.w_offset, wn);
  for (; t < a.T; t += step) {
    const long long at = ((long long)t * a.d8 + v) * 8;
    float scale = a.out_scale;
    if (gate) scale *= gate[t];
    float hv[8], yv[8];
    wait_copies<0>();
#pragma unroll
    for (int j = 0; j < 8; ++j) hv[j] = yv[j] = 0.f;
    if (in) {
      Slots<HT>::read(slot_h, pitch, hv);
      if (y) Slots<float>::read(slot_y, pitch, yv);
    }
    ahead(t + step);
    if (y) {
      if (w_post) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(yv[j], yv[j], s);
        s = group_sum(s, a.W, group, warp, lane, red);
        scale *= rsqrtf(fmaf(s, a.inv_d, a.eps));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) hv[j] = fmaf(yv[j] * wp[j], scale, hv[j] * a.res_scale);
      if (in) store8_if(a.whole, h_out + at, hv);
    }
    if (w_next) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(hv[j], hv[j], s);
      s = group_sum(s, a.W, group, warp, lane, red + 32);
      const float r = rsqrtf(fmaf(s, a.inv_d, a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) hv[j] *= r * wn[j];
      if (in) store8(x + at, hv);
    }
  }
}

// 8 elements of the stream as they are stored, so that a bf16 row takes half the registers
// while it waits for the row's sums.
template <class T>
struct Held;
template <>
struct Held<float> {
  float v[8];
  __device__ void read(uint32_t slot, uint32_t pitch) { Slots<float>::read(slot, pitch, v); }
  __device__ float operator[](int j) const { return v[j]; }
};
template <>
struct Held<__nv_bfloat16> {
  uint32_t w[4];
  __device__ void read(uint32_t slot, uint32_t pitch) {
    const uint4 a = slot16(slot);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ float operator[](int j) const {
    return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};

__device__ __forceinline__ void read4(uint32_t slot, float* v) {
  const uint4 a = slot16(slot);
  v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y);
  v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
}

// The six sums of a row over its group of W warps, on every thread.  `red`: 8 * 17 floats.
__device__ __forceinline__ void group_sum8(float (&v)[8], int W, int group, int warp, int lane,
                                           float* red) {
  float s = warp_sum8(v, lane);
  if (W > 1) {
    if ((lane & 3) == 0) red[(lane >> 2) * 17 + warp] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int w = (lane & 3) + 4 * i;
      if (w < W) s += red[(lane >> 2) * 17 + w];
    }
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, s, 4 * i);
}

constexpr int kBwdV = 2;                        // 8-column steps of a thread
constexpr int kBwdThreads = 512;
constexpr int kBwdRed = 2 * 8 * 17;             // floats of a group's two reduction buffers
template <class HT>
constexpr int bwd_units() {                     // 16-byte units of a thread: a row and weights
  return kBwdV * (2 * Slots<HT>::kUnits + 4 + 4);
}

// A thread owns 16 columns of every row of its group.  The next row's columns are copied to
// the thread's slots while this row is worked on (no thread reads another's slots).
template <class HT, class WT>
__global__ void __launch_bounds__(kBwdThreads)
block_norm_backward_kernel(const NormArgs a, const HT* __restrict__ h_out,
                           const float* __restrict__ y, const float* __restrict__ gate,
                           const WT* __restrict__ w_post, const WT* __restrict__ w_next,
                           const HT* dh_out, const float* __restrict__ dx, HT* dh,
                           float* __restrict__ dy, float* __restrict__ dgate,
                           float* __restrict__ partial) {
  constexpr int V = kBwdV, HU = Slots<HT>::kUnits;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  const uint32_t pitch = blockDim.x * 16;
  const uint32_t slots = smem_addr(smem) + threadIdx.x * 16;
  float* red = reinterpret_cast<float*>(smem + bwd_units<HT>() * pitch) + group * kBwdRed;
  // unit offsets: h', dh', y, dx, then the weights
  auto slot = [&](int unit) { return slots + (uint32_t)unit * pitch; };
  constexpr int kH = 0, kDh = V * HU, kY = 2 * V * HU, kDx = kY + 2 * V, kWp = kDx + 2 * V,
                kWn = kWp + 2 * V;
  bool in[V];
  float gp[V][8], gn[V][8];
  let_successor_start();  // it waits for this kernel's end; its launch need not
  float4* own = reinterpret_cast<float4*>(smem) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kWp; ++i) own[i * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    in[u] = (u * a.W + warp) * 32 + lane < a.d8;
#pragma unroll
    for (int j = 0; j < 8; ++j) gp[u][j] = gn[u][j] = 0.f;
  }
  auto ahead = [&](int t) {
    if (t < a.T) {
#pragma unroll
      for (int u = 0; u < V; ++u) {
        if (!in[u]) continue;
        const long long at = ((long long)t * a.d8 + (u * a.W + warp) * 32 + lane) * 8;
        if (w_next) Slots<HT>::fill(slot(kH + u * HU), pitch, h_out + at);
        if (dh_out) Slots<HT>::fill(slot(kDh + u * HU), pitch, dh_out + at);
        if (y) Slots<float>::fill(slot(kY + 2 * u), pitch, y + at);
        if (w_next) Slots<float>::fill(slot(kDx + 2 * u), pitch, dx + at);
      }
    }
    commit_copies();
  };
  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + group, turn = 0;
  ahead(t);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int v = (u * a.W + warp) * 32 + lane;
    float w[8];
    load_weight(w_post, v, in[u], a.w_offset, w);
    own[(kWp + 2 * u) * blockDim.x] = make_float4(w[0], w[1], w[2], w[3]);
    own[(kWp + 2 * u + 1) * blockDim.x] = make_float4(w[4], w[5], w[6], w[7]);
    load_weight(w_next, v, in[u], a.w_offset, w);
    own[(kWn + 2 * u) * blockDim.x] = make_float4(w[0], w[1], w[2], w[3]);
    own[(kWn + 2 * u + 1) * blockDim.x] = make_float4(w[4], w[5], w[6], w[7]);
  }
  for (; t < a.T; t += step, turn ^= 1) {
    Held<HT> hv[V], dv[V];
    float yv[V][8], q[V][8];
    const float gt = gate ? gate[t] : 1.f;
    wait_copies<0>();
#pragma unroll
    for (int u = 0; u < V; ++u) {
      hv[u].read(slot(kH + u * HU), pitch);
      dv[u].read(slot(kDh + u * HU), pitch);
      Slots<float>::read(slot(kY + 2 * u), pitch, yv[u]);
      Slots<float>::read(slot(kDx + 2 * u), pitch, q[u]);
    }
    ahead(t + step);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      float wp[4], wn[4];
      read4(slot(kWp + i), wp);
      read4(slot(kWn + i), wn);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int u = i / 2, j = 4 * (i % 2) + k;
        const float qw = q[u][j] * wn[k], yw = yv[u][j] * wp[k];
        const float hj = hv[u][j];
        s[0] = fmaf(hj, hj, s[0]);
        s[1] = fmaf(qw, hj, s[1]);
        s[2] = fmaf(yv[u][j], yv[u][j], s[2]);
        s[3] = fmaf(dv[u][j], yw, s[3]);
        s[4] = fmaf(qw, yw, s[4]);
        s[5] = fmaf(hj, yw, s[5]);
      }
    }
    group_sum8(s, a.W, group, warp, lane, red + turn * (kBwdRed / 2));
    float A = 0.f, B = 0.f;
    if (w_next) {
      A = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      B = A * A * A * s[1] * a.inv_d;
    }
    const float uy = fmaf(A, s[4], fmaf(-B, s[5], s[3]));
    const float ry = w_post ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 1.f;
    const float scale = a.out_scale * gt * ry;
    const float back = w_post ? ry * ry * uy * a.inv_d : 0.f;
    const float res = y ? a.res_scale : 1.f;
    if (gate && warp == 0 && lane == 0) dgate[t] = a.out_scale * ry * uy;
    float out[8];
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      const int u = i / 2;
      float wp[4], wn[4];
      read4(slot(kWp + i), wp);
      read4(slot(kWn + i), wn);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 4 * (i % 2) + k;
        const float hj = hv[u][j], qa = q[u][j] * A;
        gn[u][j] = fmaf(qa, hj, gn[u][j]);
        const float g = fmaf(qa, wn[k], fmaf(-B, hj, dv[u][j]));
        gp[u][j] = fmaf(g * scale, yv[u][j], gp[u][j]);
        yv[u][j] = scale * fmaf(g, wp[k], -yv[u][j] * back);
        out[j] = g * res;
      }
      if (i % 2 == 1 && in[u]) {
        const long long at = ((long long)t * a.d8 + (u * a.W + warp) * 32 + lane) * 8;
        if (y) store8_if(a.whole, dy + at, yv[u]);
        store8_if(a.whole, dh + at, out);
      }
    }
  }
  // the CTA's partial row: the groups' columns added in group order, in the slots' place
  float* col = reinterpret_cast<float*>(smem);
  if (groups > 1) __syncthreads();
  for (int g = 0; g < groups; ++g) {
    if (group == g) {
      float* out = g == groups - 1 ? partial + (long long)blockIdx.x * 2 * a.d8 * 8 : col;
#pragma unroll
      for (int u = 0; u < V; ++u) {
        const int v = (u * a.W + warp) * 32 + lane;
        if (!in[u]) continue;
        if (g > 0) {
          float t8[8];
          load8(col + v * 8, t8);
#pragma unroll
          for (int j = 0; j < 8; ++j) gp[u][j] += t8[j];
          load8(col + (a.d8 + v) * 8, t8);
#pragma unroll
          for (int j = 0; j < 8; ++j) gn[u][j] += t8[j];
        }
        store8(out + v * 8, gp[u]);
        store8(out + (a.d8 + v) * 8, gn[u]);
      }
    }
    if (groups > 1) __syncthreads();
  }
}

// dw = sum of `rows` partial rows: 32 columns a CTA, its warps take the rows in turn and are
// added in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32)
norm_weight_grad_kernel(const float* __restrict__ partial, int rows, int d,
                        float* __restrict__ dw_post, float* __restrict__ dw_next) {
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  wait_for_predecessor();
  float s = 0.f;
  if (col < 2 * d) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kSumWarps) s += partial[(long long)r * 2 * d + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < 2 * d) {
#pragma unroll
    for (int r = 1; r < kSumWarps; ++r) s += part[r][lane];
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
bool on_sectors(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 31u) return false;
  return true;
}

// Row groups of a CTA: as many as `threads` hold, but no more than it takes to give every SM
// rows.
int groups_of(int T, int W, int threads) {
  const int fit = threads / 32 / W, sms = num_sms(), rows = (T + sms - 1) / sms;
  const int n = fit < rows ? fit : rows;
  return n < 1 ? 1 : n;
}

template <class HT, class WT>
cudaError_t forward(const moe_cfg& c, const moet_norm& n, const void* h, const float* y,
                    const float* gate, const void* wp, const void* wn, void* h_out,
                    uint16_t* x, cudaStream_t st) {
  constexpr int kUnits = Slots<HT>::kUnits + 2;
  NormArgs a = make_args(c, n, 1);
  a.whole = on_sectors({h_out});
  const int groups = groups_of(c.T, a.W, kFwdThreads), threads = groups * a.W * 32;
  auto kernel = block_norm_kernel<HT, WT>;
  static OncePerDevice once;
  const cudaError_t err = once_per_device(once, [&](int&) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kUnits * 1024 * 16 + 16 * 64 * 4);
  });
  if (err != cudaSuccess) return err;
  const int want = (c.T + groups - 1) / groups, cap = num_sms() * (1024 / threads);
  kernel<<<want < cap ? want : cap, threads, kUnits * threads * 16 + groups * 64 * 4, st>>>(
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
  NormArgs a = make_args(c, n, kBwdV);
  a.whole = on_sectors({dh, dy});
  const int sms = num_sms();
  const int groups = groups_of(c.T, a.W, kBwdThreads), threads = groups * a.W * 32;
  const size_t smem = (size_t)bwd_units<HT>() * threads * 16 + (size_t)groups * kBwdRed * 4;
  auto kernel = block_norm_backward_kernel<HT, WT>;
  static OncePerDevice once;
  cudaError_t err = once_per_device(once, [&](int&) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bwd_units<HT>() * kBwdThreads * 16 + 16 * kBwdRed * 4);
  });
  if (err != cudaSuccess) return err;
  int grid = (c.T + groups - 1) / groups;
  const int cap = sms * (kBwdThreads / threads);
  if (grid > cap) grid = cap;
  if (grid > kMaxPartials) grid = kMaxPartials;
  if (grid > 0) {
    kernel<<<grid, threads, smem, st>>>(
        a, static_cast<const HT*>(h_out), y, gate, static_cast<const WT*>(wp),
        static_cast<const WT*>(wn), static_cast<const HT*>(dh_out), dx, static_cast<HT*>(dh),
        dy, dgate, static_cast<float*>(ws));
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (!dw_post && !dw_next) return cudaSuccess;
  return launch_after(norm_weight_grad_kernel, dim3((2 * c.d + 31) / 32),
                      dim3(kSumWarps * 32), 0, st, static_cast<const float*>(ws), grid, c.d,
                      dw_post, dw_next);
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
    return forward<HT, WT>(c, n, h, y, gate, w_post, w_next, h_out, x, st);
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

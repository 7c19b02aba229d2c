// The norms before and after the block, with its gate and residual scale, and their gradient.
//
//   n(v; w) = v * rms(v) * (w + w_offset),  rms(v) = rsqrt(mean(v^2) + eps)
//   h' = res_scale h + out_scale g n(y; w_post),   x = bf16(n(h'; w_next))
//
// One pass: a row lives in the registers of a group of warps (units of 4 columns, two a thread),
// so h, y and the weights are read once and h' and x are written once; the two means are two
// reductions over the group.  A persistent group copies its next row to shared memory while it
// works on this one.  Bound by HBM: 16384 x 7168 with an fp32 stream 262 us (1.64 GB, 6.3
// TB/s; a copy of as many bytes takes 251), 4096 x 2048 in bf16 17 us (12.8).  With fewer arrays a
// row's latency shows: on a bf16 stream of 16384 x 7168 the post-norm alone takes 160 us (143), the
// pre-norm alone, which copies the fewest bytes ahead, 113 us (72).
//
// The gradient needs six sums of a row, and by linearity one reduction for all of them: with
// q = dx (w_next + o), u = dh' + A q - B h', A = rms(h'), B = A^3 <q, h'> / d,
//   <u w_post, y> = <dh' w_post, y> + A <q w_post, y> - B <h' w_post, y>,
// so u itself is not needed before the reduction (nine shuffles for all six).  The weights'
// gradients are kept per column in registers over all rows of a CTA, written as one partial
// row per CTA, and added over the CTAs in a fixed order by a second kernel.  128 registers a
// thread without a spill: a few spilled ones in the row loop cost half of the rate.
// 16384 x 7168 in bf16 takes 355 us (2.11 GB, 6.0 TB/s; a copy of as many bytes 323), the post-norm's
// gradient alone 289 us (215), the pre-norm's 271 us (179): the arithmetic is the same whatever is
// absent.  What it waits for most are shared memory and the reduction's shuffles, then the
// operations' own latency.
#include "train_common.cuh"

namespace moe {
namespace {

// Partial rows of the weight gradients (CTAs of the backward kernel): what the workspace
// holds, four per SM of a 148-SM GPU.
constexpr int kMaxPartials = 592;

struct NormArgs {
  int T, d4, W;  // rows, 4-column units of a row, warps of a row's group
  float inv_d, eps, w_offset, res_scale, out_scale;
};

// ---- units of 4 columns: of bf16 8 bytes, of fp32 16.  Consecutive lanes take consecutive
// units, so every copy, load and store of a warp is one run of whole sectors ----
__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* v) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
template <class WT>
__device__ __forceinline__ void load_weight(const WT* w, int unit, bool in, float offset,
                                            float* out) {
  if (w && in) {
    load4(w + unit * 4, out);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] += offset;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = 1.f;
  }
}

// A unit's slot in shared memory, and the unit as it is stored (a bf16 one takes half the
// registers while it waits for its row's sums).  A lane copies and reads its own slots, so no
// barrier guards them; the copies go through L1 (past it they took a third longer).
template <class T>
struct Unit;
template <>
struct Unit<float> {
  static constexpr int kBytes = 16;
  float v[4];
  __device__ static void copy(uint32_t slot, const float* src) { copy_ahead16(slot, src); }
  __device__ static void clear(uint32_t slot) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(slot), "r"(0) : "memory");
  }
  __device__ void read(uint32_t slot) {
    const uint4 a = slot16(slot);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
  }
  __device__ float operator[](int j) const { return v[j]; }
};
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int kBytes = 8;
  uint32_t w[2];
  __device__ static void copy(uint32_t slot, const __nv_bfloat16* src) {
    copy_ahead8(slot, src);
  }
  __device__ static void clear(uint32_t slot) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(slot), "r"(0) : "memory");
  }
  __device__ void read(uint32_t slot) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(w[0]), "=r"(w[1])
                 : "r"(slot)
                 : "memory");
  }
  __device__ float operator[](int j) const {
    return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};

// The slots of one array: kUnits units a thread.
template <class T>
struct Array {
  uint32_t first, pitch;
  __device__ Array(uint32_t base, int threads)
      : first(base + threadIdx.x * Unit<T>::kBytes), pitch(threads * Unit<T>::kBytes) {}
  __device__ uint32_t slot(int i) const { return first + i * pitch; }
};

// Units of a thread, its columns of every row of its group.  Forward: 2, so that the weights
// stay in registers with 32 warps a row.  Backward: 4, since its reduction of six sums costs
// a thread the same whatever it holds.
constexpr int kFwdUnits = 2, kBwdUnits = 4;
constexpr int kThreads = 512;       // of a CTA with several row groups, or of the backward's
constexpr int kFwdRed = 2 * 32;     // floats of a group's reduction buffers
constexpr int kBwdRed = 2 * 8 * 17;

// The sum over the group of one value, on every thread.  `red` is one of the group's two
// buffers, which a caller alternates from sum to sum, whichever sums its rows take: a warp that
// writes a buffer again has passed the barrier of the sum between, which the others reach only
// when they have read this one.  So one barrier a sum is enough.
__device__ __forceinline__ float group_sum(float v, int W, int group, int warp, int lane,
                                           uint32_t red) {
  v = warp_sum(v);
  if (W == 1) return v;
  if (lane == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(red + warp * 4), "f"(v) : "memory");
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
  float s = 0.f;
  if (lane < W) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(red + lane * 4) : "memory");
  return warp_sum(s);
}

// The six sums of a row over its group of W warps, on every thread.  `red`: 8 * 17 floats.
__device__ __forceinline__ void group_sum8(float (&v)[8], int W, int group, int warp, int lane,
                                           float* red) {
  float s = warp_sums(v, lane);
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

// The next row's columns are copied to the thread's slots as soon as this row's are in
// registers, so that memory works through both means of a row (two or three rows ahead gave
// nothing: they only take L1 from the copies).
template <class HT, class WT>
__global__ void __launch_bounds__(1024)
block_norm_kernel(const NormArgs a, const HT* h, const float* __restrict__ y,
                  const float* __restrict__ gate, const WT* __restrict__ w_post,
                  const WT* __restrict__ w_next, HT* h_out, __nv_bfloat16* __restrict__ x) {
  constexpr int U = kFwdUnits;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  const Array<float> ys(smem_addr(smem), blockDim.x);
  const Array<HT> hs(smem_addr(smem) + U * 16 * blockDim.x, blockDim.x);
  uint32_t red = smem_addr(smem) + U * (16 + Unit<HT>::kBytes) * blockDim.x + group * kFwdRed * 4;
  const uint32_t both = 2 * red + kFwdRed * 2;  // two buffers: behind `red` comes both - red
  auto unit = [&](int i) { return (i * a.W + warp) * 32 + lane; };
  auto ahead = [&](int t) {
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const long long at = ((long long)t * a.d4 + unit(i)) * 4;
        if (unit(i) >= a.d4) continue;
        Unit<HT>::copy(hs.slot(i), h + at);
        if (y) Unit<float>::copy(ys.slot(i), y + at);
      }
    }
    commit_copies();
  };
  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + group;
  ahead(t);
  float wp[U][4], wn[U][4];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    load_weight(w_post, unit(i), unit(i) < a.d4, a.w_offset, wp[i]);
    load_weight(w_next, unit(i), unit(i) < a.d4, a.w_offset, wn[i]);
  }
  for (; t < a.T; t += step) {
    float scale = a.out_scale;
    if (gate) scale *= gate[t];
    Unit<HT> hu[U];
    Unit<float> yu[U];
    wait_copies<0>();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      hu[i].read(hs.slot(i));
      if (y) yu[i].read(ys.slot(i));
    }
    ahead(t + step);
    float hv[U][4];
    if (y) {
      if (w_post) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (unit(i) < a.d4) s = fmaf(yu[i][j], yu[i][j], s);
        s = group_sum(s, a.W, group, warp, lane, red);
        red = both - red;
        scale *= rsqrtf(fmaf(s, a.inv_d, a.eps));
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          hv[i][j] = fmaf(yu[i][j] * wp[i][j], scale, hu[i][j] * a.res_scale);
        if (unit(i) < a.d4) store4(h_out + ((long long)t * a.d4 + unit(i)) * 4, hv[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) hv[i][j] = hu[i][j];
    }
    if (w_next) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (unit(i) < a.d4) s = fmaf(hv[i][j], hv[i][j], s);
      s = group_sum(s, a.W, group, warp, lane, red);
      red = both - red;
      const float r = rsqrtf(fmaf(s, a.inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) hv[i][j] *= r * wn[i][j];
        if (unit(i) < a.d4) store4(x + ((long long)t * a.d4 + unit(i)) * 4, hv[i]);
      }
    }
  }
}

// Bytes of a thread's slots in the backward kernel: a row's units, then the weights'.
template <class HT>
constexpr int bwd_slot_bytes() {
  return kBwdUnits * (2 * Unit<HT>::kBytes + 4 * 16);
}

template <class HT, class WT>
__global__ void __launch_bounds__(kThreads)
block_norm_backward_kernel(const NormArgs a, const HT* __restrict__ h_out,
                           const float* __restrict__ y, const float* __restrict__ gate,
                           const WT* __restrict__ w_post, const WT* __restrict__ w_next,
                           const HT* dh_out, const float* __restrict__ dx, HT* dh,
                           float* __restrict__ dy, float* __restrict__ dgate,
                           float* __restrict__ partial) {
  constexpr int U = kBwdUnits;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / a.W, warp = (threadIdx.x >> 5) % a.W;
  const int groups = (blockDim.x >> 5) / a.W;
  const uint32_t base = smem_addr(smem), step16 = U * 16 * blockDim.x;
  const Array<float> ys(base, blockDim.x), qs(base + step16, blockDim.x);
  const Array<float> wps(base + 2 * step16, blockDim.x), wns(base + 3 * step16, blockDim.x);
  const uint32_t stream = base + 4 * step16;
  const Array<HT> hs(stream, blockDim.x),
      ds(stream + U * Unit<HT>::kBytes * blockDim.x, blockDim.x);
  float* red = reinterpret_cast<float*>(smem + bwd_slot_bytes<HT>() * blockDim.x) + group * kBwdRed;
  auto unit = [&](int i) { return (i * a.W + warp) * 32 + lane; };
  let_successor_start();  // it waits for this kernel's end; its launch need not
  // what no copy fills stays zero: absent arrays, columns behind the row
#pragma unroll
  for (int i = 0; i < U; ++i) {
    Unit<float>::clear(ys.slot(i));
    Unit<float>::clear(qs.slot(i));
    Unit<HT>::clear(hs.slot(i));
    Unit<HT>::clear(ds.slot(i));
  }
  auto ahead = [&](int t) {
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (unit(i) >= a.d4) continue;
        const long long at = ((long long)t * a.d4 + unit(i)) * 4;
        if (w_next) Unit<HT>::copy(hs.slot(i), h_out + at);
        if (dh_out) Unit<HT>::copy(ds.slot(i), dh_out + at);
        if (y) Unit<float>::copy(ys.slot(i), y + at);
        if (w_next) Unit<float>::copy(qs.slot(i), dx + at);
      }
    }
    commit_copies();
  };
  const int step = gridDim.x * groups;
  int t = blockIdx.x * groups + group, turn = 0;
  ahead(t);
  float gp[U][4], gn[U][4];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float w[4];
    load_weight(w_post, unit(i), unit(i) < a.d4, a.w_offset, w);
    reinterpret_cast<float4*>(smem)[2 * U * blockDim.x + i * blockDim.x + threadIdx.x] =
        make_float4(w[0], w[1], w[2], w[3]);
    load_weight(w_next, unit(i), unit(i) < a.d4, a.w_offset, w);
    reinterpret_cast<float4*>(smem)[3 * U * blockDim.x + i * blockDim.x + threadIdx.x] =
        make_float4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) gp[i][j] = gn[i][j] = 0.f;
  }
  for (; t < a.T; t += step, turn ^= 1) {
    Unit<HT> hu[U], du[U];
    Unit<float> yu[U], qu[U];
    const float gt = gate ? gate[t] : 1.f;
    wait_copies<0>();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      hu[i].read(hs.slot(i));
      du[i].read(ds.slot(i));
      yu[i].read(ys.slot(i));
      qu[i].read(qs.slot(i));
    }
    ahead(t + step);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      Unit<float> wp, wn;
      wp.read(wps.slot(i));
      wn.read(wns.slot(i));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float qw = qu[i][j] * wn[j], yw = yu[i][j] * wp[j], hj = hu[i][j];
        s[0] = fmaf(hj, hj, s[0]);
        s[1] = fmaf(qw, hj, s[1]);
        s[2] = fmaf(yu[i][j], yu[i][j], s[2]);
        s[3] = fmaf(du[i][j], yw, s[3]);
        s[4] = fmaf(qw, yw, s[4]);
        s[5] = fmaf(hj, yw, s[5]);
      }
    }
    group_sum8(s, a.W, group, warp, lane, red + turn * (kBwdRed / 2));
    float A = 0.f, B = 0.f;
    if (w_next) {
      A = rsqrtf(fmaf(s[0], a.inv_d, a.eps));
      // <q, h'> times A first: rms(h') |h'| is at most sqrt(d), while A^3 by itself leaves fp32
      // (rows of zeros with eps under 1e-25, rows of 1e13)
      B = A * (A * (A * s[1] * a.inv_d));
    }
    const float uy = fmaf(A, s[4], fmaf(-B, s[5], s[3]));
    const float ry = w_post ? rsqrtf(fmaf(s[2], a.inv_d, a.eps)) : 1.f;
    const float scale = a.out_scale * gt * ry;
    const float back = w_post ? ry * (ry * uy * a.inv_d) : 0.f;
    const float res = y ? a.res_scale : 1.f;
    if (gate && warp == 0 && lane == 0) dgate[t] = a.out_scale * ry * uy;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      Unit<float> wp, wn;
      wp.read(wps.slot(i));
      wn.read(wns.slot(i));
      float to_y[4], to_h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float hj = hu[i][j], qa = qu[i][j] * A;
        gn[i][j] = fmaf(qa, hj, gn[i][j]);
        const float g = fmaf(qa, wn[j], fmaf(-B, hj, du[i][j]));
        gp[i][j] = fmaf(g * scale, yu[i][j], gp[i][j]);
        to_y[j] = scale * fmaf(g, wp[j], -yu[i][j] * back);
        to_h[j] = g * res;
      }
      if (unit(i) < a.d4) {
        const long long at = ((long long)t * a.d4 + unit(i)) * 4;
        if (y) store4(dy + at, to_y);
        store4(dh + at, to_h);
      }
    }
  }
  // the CTA's partial row: the groups' columns added in group order, in the slots' place
  float* col = reinterpret_cast<float*>(smem);
  if (groups > 1) __syncthreads();
  for (int g = 0; g < groups; ++g) {
    if (group == g) {
      float* out = g == groups - 1 ? partial + (long long)blockIdx.x * 2 * a.d4 * 4 : col;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (unit(i) >= a.d4) continue;
        if (g > 0) {
          float t4[4];
          load4(col + unit(i) * 4, t4);
#pragma unroll
          for (int j = 0; j < 4; ++j) gp[i][j] += t4[j];
          load4(col + (a.d4 + unit(i)) * 4, t4);
#pragma unroll
          for (int j = 0; j < 4; ++j) gn[i][j] += t4[j];
        }
        store4(out + unit(i) * 4, gp[i]);
        store4(out + (a.d4 + unit(i)) * 4, gn[i]);
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

NormArgs make_args(const moe_cfg& c, const moet_norm& n, int units) {
  NormArgs a;
  a.T = c.T;
  a.d4 = c.d / 4;
  a.W = (a.d4 + 32 * units - 1) / (32 * units);
  a.inv_d = 1.f / (float)c.d;
  a.eps = n.eps;
  a.w_offset = n.w_offset;
  a.res_scale = n.res_scale;
  a.out_scale = n.out_scale;
  return a;
}

// Row groups of a CTA: as many as it holds, but no more than it takes to give every SM rows.
int groups_of(int T, int W) {
  const int fit = kThreads / 32 / W, sms = num_sms(), rows = (T + sms - 1) / sms;
  const int n = fit < rows ? fit : rows;
  return n < 1 ? 1 : n;
}

template <class HT, class WT>
cudaError_t forward(const moe_cfg& c, const moet_norm& n, const void* h, const float* y,
                    const float* gate, const void* wp, const void* wn, void* h_out,
                    uint16_t* x, cudaStream_t st) {
  constexpr int kSlots = kFwdUnits * (16 + Unit<HT>::kBytes);  // bytes a thread
  const NormArgs a = make_args(c, n, kFwdUnits);
  const int groups = groups_of(c.T, a.W), threads = groups * a.W * 32;
  auto kernel = block_norm_kernel<HT, WT>;
  static OncePerDevice once;
  const cudaError_t err = once_per_device(once, [&](int&) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSlots * 1024 + 16 * kFwdRed * 4);
  });
  if (err != cudaSuccess) return err;
  const int want = (c.T + groups - 1) / groups, cap = num_sms() * (1024 / threads);
  kernel<<<want < cap ? want : cap, threads, kSlots * threads + groups * kFwdRed * 4, st>>>(
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
  const NormArgs a = make_args(c, n, kBwdUnits);
  const int sms = num_sms(), groups = groups_of(c.T, a.W), threads = groups * a.W * 32;
  const size_t smem = (size_t)bwd_slot_bytes<HT>() * threads + (size_t)groups * kBwdRed * 4;
  auto kernel = block_norm_backward_kernel<HT, WT>;
  static OncePerDevice once;
  cudaError_t err = once_per_device(once, [&](int&) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bwd_slot_bytes<HT>() * kThreads + kThreads / 32 * kBwdRed * 4);
  });
  if (err != cudaSuccess) return err;
  int grid = (c.T + groups - 1) / groups;
  const int cap = sms * (kThreads / threads);
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

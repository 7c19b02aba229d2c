// AdamW over many tensors in one launch, with fp32 or 8-bit moments.
//
//   t = step + 1, g = grad * grad_scale, m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// The tensors' addresses travel in the launch's parameters, so a call needs neither a table in
// device memory nor a copy to one.  Tensors of one combination of types share a launch; a
// persistent grid walks their tiles of 2048 elements (a warp per block of 256: each lane
// holds elements 4 l .. 4 l + 3 of either half, so every load and store is a run of whole
// sectors) and finds a tile's tensor by bisection of the tile prefix.
//
// 8-bit moments hold a block of 256 elements as e4m3 with one fp32 scale: m itself, and the
// root r of v (whose range is half of v's in the exponent: e4m3's 2^18 of range for r is
// 2^36 for v).  The new largest |m| and r of a block are two warp reductions of the bit
// patterns (non-negative floats order as integers).  The moments' operations and the
// roundings to codes are the IEEE ones, each rounded by itself, so the stored states are
// reproducible outside this kernel bit for bit; the weight's quotient is the approximate one
// (2 ulp of fp32, below what the weight's own rounding does to it).
//
// Bound by HBM: 4 (p) + 4 (g) + 4 (m, v) bytes an element with bf16 weights and 8-bit states.
#include <cuda_fp8.h>

#include <cmath>

#include "train_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = MOET_ADAMW_BLOCK;
constexpr int kTile = kThreads / 32 * kBlock;  // elements of one CTA's turn
constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Tiny = 0.001953125f;  // 2^-9, the smallest code above 0
constexpr float kLeastTop = 1e-30f;        // blocks below it are stored as zeros

enum WeightKind { W_F32 = 0, W_BF16 = 1, W_BF16_MASTER = 2 };

struct Item {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  long long n;
  float wd;
};
// Three capacities of the parameter block, so that a few tensors do not pay for many; the
// largest stays under the 32764 bytes a launch can carry.
template <int CAP>
struct Batch {
  int32_t count;
  int32_t first_tile[CAP + 1];
  Item item[CAP];
};
constexpr int kCaps[3] = {8, 64, 400};
static_assert(sizeof(Batch<400>) <= 32000, "launch parameters");

struct Consts {
  float b1, b2, omb1, omb2, log_b1, log_b2, eps;
};

__device__ __forceinline__ void load4(const float* p, long long i, long long n, float* v) {
  if (i + 4 <= n) {
    const float4 a = *reinterpret_cast<const float4*>(p + i);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? p[i + j] : 0.f;
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, long long i, long long n,
                                      float* v) {
  if (i + 4 <= n) {
    const uint2 a = *reinterpret_cast<const uint2*>(p + i);
    v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + j < n ? __bfloat162float(p[i + j]) : 0.f;
  }
}
__device__ __forceinline__ uint32_t load4_codes(const uint8_t* p, long long i, long long n) {
  if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(p + i);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)p[i + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void decode4(uint32_t w, float* v) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w >> (16 * j)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x, v[2 * j + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t encode4(const float* v) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE,
                                               __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE,
                                               __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ void store4(float* p, long long i, long long n, const float* v) {
  if (i + 4 <= n) {
    *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = v[j];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, long long i, long long n,
                                       const float* v) {
  if (i + 4 <= n) {
    *reinterpret_cast<uint2*>(p + i) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = __float2bfloat16_rn(v[j]);
  }
}
__device__ __forceinline__ void store4_codes(uint8_t* p, long long i, long long n,
                                             uint32_t w) {
  if (i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p + i) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) p[i + j] = (uint8_t)(w >> (8 * j));
  }
}

// The largest of the lanes' non-negative values (NaN above infinity above all numbers).
__device__ __forceinline__ float warp_top(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

template <int W, bool GBF16, bool S8, int CAP>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ Batch<CAP> b, const Consts c, const float* lr_p,
             const float* grad_scale, int32_t* step, bool last_launch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float gs = grad_scale ? *grad_scale : 1.f;
  if (!isfinite(gs)) return;  // the same for every CTA: the step is left out as a whole
  const int t = step[0] + 1;
  const float lr = *lr_p;
  const float lr1 = lr / -expm1f((float)t * c.log_b1);
  const float inv2 = rsqrtf(-expm1f((float)t * c.log_b2));
  const int tiles = b.first_tile[b.count];

  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int lo = 0, hi = b.count - 1;  // the last tensor whose first tile is at or before this
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (b.first_tile[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    const Item& it = b.item[lo];
    const long long n = it.n;
    const long long block = (long long)(tile - b.first_tile[lo]) * (kThreads / 32) + warp;
    if (block * kBlock >= n) continue;
    const float decay = fmaf(-lr, it.wd, 1.f);
    long long at[2];
    float g[2][4], p[2][4], m[2][4], v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      at[h] = block * kBlock + h * (kBlock / 2) + lane * 4;
      if (GBF16) load4(static_cast<const __nv_bfloat16*>(it.g), at[h], n, g[h]);
      else load4(static_cast<const float*>(it.g), at[h], n, g[h]);
      if (W == W_F32) load4(static_cast<const float*>(it.p), at[h], n, p[h]);
      else if (W == W_BF16) load4(static_cast<const __nv_bfloat16*>(it.p), at[h], n, p[h]);
      else load4(it.master, at[h], n, p[h]);
      if (S8) {
        decode4(load4_codes(static_cast<const uint8_t*>(it.m), at[h], n), m[h]);
        decode4(load4_codes(static_cast<const uint8_t*>(it.v), at[h], n), v[h]);
      } else {
        load4(static_cast<const float*>(it.m), at[h], n, m[h]);
        load4(static_cast<const float*>(it.v), at[h], n, v[h]);
      }
    }
    float sm = 0.f, sv = 0.f, top_m = 0.f, top_r = 0.f;
    if (S8) {
      sm = it.m_scale[block];
      sv = it.v_scale[block];
    }
    float r[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float mo = m[h][j], vo = v[h][j];
        if (S8) {
          mo = __fmul_rn(mo, sm);
          vo = __fmul_rn(vo, sv);
          vo = __fmul_rn(vo, vo);
        }
        const float gr = grad_scale ? __fmul_rn(g[h][j], gs) : g[h][j];
        mo = __fadd_rn(__fmul_rn(mo, c.b1), __fmul_rn(gr, c.omb1));
        vo = __fadd_rn(__fmul_rn(vo, c.b2), __fmul_rn(__fmul_rn(gr, c.omb2), gr));
        const float root = __fsqrt_rn(vo);
        const float step_by = __fdividef(mo, fmaf(root, inv2, c.eps));
        p[h][j] = fmaf(-lr1, step_by, p[h][j] * decay);
        m[h][j] = mo;
        v[h][j] = vo;
        r[h][j] = root;
        if (S8) {
          // as bit patterns: a NaN stays the largest
          top_m = __uint_as_float(max(__float_as_uint(top_m), __float_as_uint(fabsf(mo))));
          top_r = __uint_as_float(max(__float_as_uint(top_r), __float_as_uint(root)));
        }
      }
    if (S8) {
      top_m = warp_top(top_m);
      top_r = warp_top(top_r);
      const bool some_m = !(top_m < kLeastTop), some_r = !(top_r < kLeastTop);
      const float im = some_m ? __fmul_rn(kE4m3Max, __frcp_rn(top_m)) : 0.f;
      const float ir = some_r ? __fmul_rn(kE4m3Max, __frcp_rn(top_r)) : 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[h][j] = __fmul_rn(m[h][j], im);
          const float code = __fmul_rn(r[h][j], ir);
          v[h][j] = r[h][j] > 0.f ? fmaxf(code, kE4m3Tiny) : code;
        }
      if (lane == 0) {
        it.m_scale[block] = some_m ? __fmul_rn(top_m, 1.f / kE4m3Max) : 0.f;
        it.v_scale[block] = some_r ? __fmul_rn(top_r, 1.f / kE4m3Max) : 0.f;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (W == W_F32) store4(static_cast<float*>(it.p), at[h], n, p[h]);
      else store4(static_cast<__nv_bfloat16*>(it.p), at[h], n, p[h]);
      if (W == W_BF16_MASTER) store4(it.master, at[h], n, p[h]);
      if (S8) {
        store4_codes(static_cast<uint8_t*>(it.m), at[h], n, encode4(m[h]));
        store4_codes(static_cast<uint8_t*>(it.v), at[h], n, encode4(v[h]));
      } else {
        store4(static_cast<float*>(it.m), at[h], n, m[h]);
        store4(static_cast<float*>(it.v), at[h], n, v[h]);
      }
    }
  }
  // The last CTA to end raises the step count: all have read it by then.  The ticket wraps
  // to 0 by itself, so nothing has to be cleared between calls.
  if (last_launch) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      const unsigned ticket =
          atomicInc(reinterpret_cast<unsigned*>(step + 1), gridDim.x - 1);
      if (ticket == gridDim.x - 1) step[0] = t;
    }
  }
}

template <int W, bool GBF16, bool S8, int CAP>
cudaError_t launch_batch(const moet_adamw_tensor* const* ts, int count, const Consts& c,
                         const float* lr, const float* gs, int32_t* step, bool last,
                         cudaStream_t st) {
  Batch<CAP> b;
  b.count = count;
  b.first_tile[0] = 0;
  for (int i = 0; i < count; ++i) {
    const moet_adamw_tensor& t = *ts[i];
    b.item[i] = {t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.master, t.n, t.weight_decay};
    b.first_tile[i + 1] = b.first_tile[i] + (int32_t)((t.n + kTile - 1) / kTile);
  }
  auto kernel = adamw_kernel<W, GBF16, S8, CAP>;
  static OncePerDevice once;
  int per_sm = 1;
  cudaError_t err = once_per_device(once, [&](int& v) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kernel, kThreads, 0);
  }, &per_sm);
  if (err != cudaSuccess) return err;
  const int cap = num_sms() * (per_sm > 0 ? per_sm : 1);
  const int tiles = b.first_tile[count];
  const int grid = tiles < 1 ? 1 : tiles < cap ? tiles : cap;
  kernel<<<grid, kThreads, 0, st>>>(b, c, lr, gs, step, last);
  return cudaGetLastError();
}

template <int W, bool GBF16, bool S8>
cudaError_t launch_kind(const moet_adamw_tensor* const* ts, int count, const Consts& c,
                        const float* lr, const float* gs, int32_t* step, bool last,
                        cudaStream_t st) {
  if (count <= kCaps[0]) return launch_batch<W, GBF16, S8, kCaps[0]>(ts, count, c, lr, gs, step, last, st);
  if (count <= kCaps[1]) return launch_batch<W, GBF16, S8, kCaps[1]>(ts, count, c, lr, gs, step, last, st);
  return launch_batch<W, GBF16, S8, kCaps[2]>(ts, count, c, lr, gs, step, last, st);
}

using LaunchKind = cudaError_t (*)(const moet_adamw_tensor* const*, int, const Consts&,
                                   const float*, const float*, int32_t*, bool, cudaStream_t);
constexpr int kKinds = 12;
const LaunchKind kLaunch[kKinds] = {
    launch_kind<W_F32, false, false>,         launch_kind<W_F32, false, true>,
    launch_kind<W_F32, true, false>,          launch_kind<W_F32, true, true>,
    launch_kind<W_BF16, false, false>,        launch_kind<W_BF16, false, true>,
    launch_kind<W_BF16, true, false>,         launch_kind<W_BF16, true, true>,
    launch_kind<W_BF16_MASTER, false, false>, launch_kind<W_BF16_MASTER, false, true>,
    launch_kind<W_BF16_MASTER, true, false>,  launch_kind<W_BF16_MASTER, true, true>,
};

int kind_of(const moet_adamw_tensor& t) {
  const int w = t.p_dtype == MOET_F32 ? W_F32 : t.master ? W_BF16_MASTER : W_BF16;
  return w * 4 + (t.g_dtype == MOET_BF16 ? 2 : 0) + (t.state_dtype == MOET_E4M3 ? 1 : 0);
}

}  // namespace

cudaError_t launch_adamw(const moet_adamw_tensor* tensors, int count, const moet_adamw& opt,
                         const float* lr, const float* grad_scale, int32_t* step,
                         cudaStream_t st) {
  const Consts c = {(float)opt.beta1,           (float)opt.beta2,
                    (float)(1.0 - opt.beta1),   (float)(1.0 - opt.beta2),
                    (float)std::log(opt.beta1), (float)std::log(opt.beta2),
                    (float)opt.eps};
  // the launches: runs of tensors of one kind, cut at the largest capacity and at 2^30 tiles
  // (a launch that raises the count goes last, with no tensors if there are none)
  const moet_adamw_tensor* run[kCaps[2]];
  const moet_adamw_tensor* pending[kCaps[2]];
  int n_pending = -1, pending_kind = 0;
  auto flush = [&](int kind, int n) -> cudaError_t {
    cudaError_t err = cudaSuccess;
    if (n_pending >= 0)
      err = kLaunch[pending_kind](pending, n_pending, c, lr, grad_scale, step, false, st);
    for (int i = 0; i < n; ++i) pending[i] = run[i];
    n_pending = n;
    pending_kind = kind;
    return err;
  };
  for (int kind = 0; kind < kKinds; ++kind) {
    int n = 0;
    long long tiles = 0;
    for (int i = 0; i < count; ++i) {
      if (tensors[i].n == 0 || kind_of(tensors[i]) != kind) continue;
      const long long more = (tensors[i].n + kTile - 1) / kTile;
      if (n == kCaps[2] || (n && tiles + more > (1LL << 30))) {
        const cudaError_t err = flush(kind, n);
        if (err != cudaSuccess) return err;
        n = 0;
        tiles = 0;
      }
      run[n++] = &tensors[i];
      tiles += more;
    }
    if (n) {
      const cudaError_t err = flush(kind, n);
      if (err != cudaSuccess) return err;
    }
  }
  return kLaunch[pending_kind](pending, n_pending < 0 ? 0 : n_pending, c, lr, grad_scale,
                               step, true, st);
}

}  // namespace moe

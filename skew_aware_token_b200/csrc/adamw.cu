// AdamW over many tensors in one launch, with fp32 or 8-bit moments.
//
//   t = step + 1, g = grad * grad_scale, m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
//
// The tensors' addresses travel in the launch's parameters, so a call needs neither a table in
// device memory nor a copy to one.  Tensors of one combination of types share a launch, whose
// CTAs take tiles of 2048 elements (a warp per block of 256) at the grid's stride; a CTA finds
// its first tile's tensor by bisection and steps on from there.
//
// 8-bit moments hold a block of 256 elements as e4m3 with one fp32 scale: m itself, and the
// root r of v (whose range is half of v's in the exponent: e4m3's 2^18 of range for r is
// 2^36 for v).  A block's largest |m| and v are two warp reductions of the bit patterns
// (non-negative floats order as integers).  The moments, the scales and the roundings to
// codes are those of IEEE operations, each rounded by itself, so the stored states are
// reproducible outside this kernel bit for bit; the weight's root and quotient are
// approximate ones (a few steps of fp32, below what the weight's own rounding does; a subnormal
// v has the root 0 unless eps is so small that this would show).
//
// Bound by HBM: fp32 states 200 us for 50 M fp32 weights with bf16 gradients (26 bytes each,
// 6.5 TB/s, a copy's rate).  With bf16 weights, fp32 gradients and 8-bit states 12 bytes an
// element carry 48 instructions: 403 M weights take 875 to 900 us at the clocks that the power
// limit leaves, 830 to 840 before they fall (4.86 GB: 741 us at a copy's rate).  The same accesses
// without the arithmetic take 810 to 830 us; the two blocks copied ahead hide most of it (one
// ahead: 942 us, none: 960).
// Streaming stores, wider or narrower CTAs, two or four blocks a warp at a time gave nothing or
// cost time.
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

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
// Three capacities of the parameter block, so that a few tensors do not pay for many: what is
// copied at a launch costs the host alone.  A call of 8 tensors takes 7.9 us with the first
// capacity, 9.0 with the second, 10.6 with the third, one of 100 tensors 15.8 with the second and
// 17.5 with the third (64 as the second: 60 tensors 12.3 for 13.0, 100 tensors 17.6).  The
// largest stays under the 32764 bytes a launch can carry.
template <int CAP>
struct Batch {
  int32_t count;
  int32_t first_tile[CAP + 1];
  Item item[CAP];
};
constexpr int kCaps[3] = {8, 128, 400};
static_assert(sizeof(Batch<400>) <= 32000, "launch parameters");

struct Consts {
  float b1, b2, omb1, omb2, log_b1, log_b2, eps, one;
  bool tiny_eps;  // next to eps the root of a subnormal v counts
};

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void decode8(uint32_t lo, uint32_t hi, float2 (&v)[4]) {
  const uint32_t w[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    v[i] = __half22float2(*reinterpret_cast<const __half2*>(&h));
  }
}

// A lane's 8 elements of a block, as 4 pairs.  With 8-bit states they are consecutive (8 codes
// in one access); with fp32 states two runs of 4, one in either half of the block, so that the
// accesses of 16 bytes stay consecutive over the lanes.
// FULL: the whole block lies inside the tensor (an 8-bit one then comes from the slots).
template <bool S8>
struct Lane {
  uint32_t at, n;  // the lane's first element, and the elements there are, from the tile's first
  __device__ Lane(int warp, int lane, uint32_t n)
      : at(warp * kBlock + lane * (S8 ? 8 : 4)), n(n) {}
  __device__ uint32_t index(int i) const { return at + (S8 || i < 4 ? i : kBlock / 2 + i - 4); }

  template <bool FULL>
  __device__ void load(const float* p, float2 (&v)[4]) const {
    if constexpr (FULL) {
      const float4 a = *reinterpret_cast<const float4*>(p + at);
      const float4 b = *reinterpret_cast<const float4*>(p + index(4));
      v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
      v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = make_float2(index(2 * i) < n ? p[index(2 * i)] : 0.f,
                           index(2 * i + 1) < n ? p[index(2 * i + 1)] : 0.f);
    }
  }
  template <bool FULL>
  __device__ void load(const __nv_bfloat16* p, float2 (&v)[4]) const {
    if constexpr (FULL) {
      const uint2 lo = *reinterpret_cast<const uint2*>(p + at);
      const uint2 hi = *reinterpret_cast<const uint2*>(p + index(4));
      const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = bf16_pair(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = make_float2(
            index(2 * i) < n ? __bfloat162float(p[index(2 * i)]) : 0.f,
            index(2 * i + 1) < n ? __bfloat162float(p[index(2 * i + 1)]) : 0.f);
    }
  }
  template <bool FULL>
  __device__ void load(const uint8_t* p, float2 (&v)[4]) const {
    static_assert(!FULL, "whole 8-bit blocks come from the slots");
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (index(i) < n) w[i / 4] |= (uint32_t)p[index(i)] << (8 * (i % 4));
    decode8(w[0], w[1], v);
  }
  template <bool FULL>
  __device__ void store(float* p, const float2 (&v)[4]) const {
    if constexpr (FULL) {
      *reinterpret_cast<float4*>(p + at) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      *reinterpret_cast<float4*>(p + index(4)) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (index(2 * i) < n) p[index(2 * i)] = v[i].x;
        if (index(2 * i + 1) < n) p[index(2 * i + 1)] = v[i].y;
      }
    }
  }
  template <bool FULL>
  __device__ void store(__nv_bfloat16* p, const float2 (&v)[4]) const {
    if constexpr (FULL) {
      const uint2 lo = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
      const uint2 hi = make_uint2(pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
      if constexpr (S8) {
        *reinterpret_cast<uint4*>(p + at) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        *reinterpret_cast<uint2*>(p + at) = lo;
        *reinterpret_cast<uint2*>(p + index(4)) = hi;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (index(2 * i) < n) p[index(2 * i)] = __float2bfloat16_rn(v[i].x);
        if (index(2 * i + 1) < n) p[index(2 * i + 1)] = __float2bfloat16_rn(v[i].y);
      }
    }
  }
  template <bool FULL>
  __device__ void store(uint8_t* p, const float2 (&v)[4]) const {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(v[2 * i], __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(v[2 * i + 1], __NV_SATFINITE, __NV_E4M3) << 16;
    if constexpr (FULL) {
      *reinterpret_cast<uint2*>(p + at) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (index(i) < n) p[index(i)] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }
};

// max(|a|, |b|, |c|), NaN if any is
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest of the lanes' non-negative values (NaN above infinity above all numbers).
__device__ __forceinline__ float warp_top(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}
__device__ __forceinline__ float least3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float near_root(float x) {  // 0 of a subnormal x
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float near_root_of_any(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations an instruction.
__device__ __forceinline__ unsigned long long bits2(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 pair(unsigned long long r) {
  float2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return pair(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return pair(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mulc(float2 a, float c) { return mul2(a, both(c)); }
// The sum of two rounded products, as a * one + b with a `one` that the compiler cannot see:
// it fuses a packed product and sum (even with .rn) into one rounding.
__device__ __forceinline__ float2 sum2(float2 a, float2 b, const Consts& c) {
  return fma2(a, both(c.one), b);
}

struct Step {
  float gs, lr, lr1, inv2;  // gradient scale, lr, lr / (1 - b1^t), (1 - b2^t)^-1/2
  bool scaled;
};

template <int W, bool GBF16, bool S8>
struct Types {
  using G = typename std::conditional<GBF16, __nv_bfloat16, float>::type;
  using P = typename std::conditional<W == W_F32, float, __nv_bfloat16>::type;
  using M = typename std::conditional<S8, uint8_t, float>::type;
  using Source = typename std::conditional<W == W_BF16, __nv_bfloat16, float>::type;
};

// One tile's part of a tensor: the addresses of its first element.  They are the same for
// the whole CTA, and a lane's place in the tile is 32 bits that stay, so that the accesses
// need no address arithmetic of the lanes.
template <int W, bool GBF16, bool S8>
struct Tile {
  using T = Types<W, GBF16, S8>;
  const typename T::G* g;
  typename T::P* p;
  float* master;
  typename T::M* m;
  typename T::M* v;
  float* m_scale;
  float* v_scale;
  float wd;
  uint32_t n;  // elements from here to the tensor's end, at most kTile (0: no tile)
  template <int CAP>
  __device__ Tile(const Batch<CAP>& b, int item, int tile) {
    n = 0;
    if (item >= b.count) return;
    const Item& it = b.item[item];
    const long long in = tile - b.first_tile[item], first = in * kTile;
    g = static_cast<const typename T::G*>(it.g) + first;
    p = static_cast<typename T::P*>(it.p) + first;
    if constexpr (W == W_BF16_MASTER) master = it.master + first;
    m = static_cast<typename T::M*>(it.m) + first;
    v = static_cast<typename T::M*>(it.v) + first;
    if constexpr (S8) {
      m_scale = it.m_scale + in * (kThreads / 32);
      v_scale = it.v_scale + in * (kThreads / 32);
    }
    wd = it.wd;
    n = (uint32_t)(it.n - first < kTile ? it.n - first : kTile);
  }
  __device__ const typename T::Source* weights() const {
    if constexpr (W == W_BF16_MASTER) return master;
    else return p;
  }
};

// Where a block's values come from: global memory,
template <int W, bool GBF16, bool S8, bool FULL>
struct Direct {
  const Tile<W, GBF16, S8>& tl;
  const Lane<S8> at;
  __device__ Direct(const Tile<W, GBF16, S8>& tl, int warp, int lane)
      : tl(tl), at(warp, lane, tl.n) {}
  __device__ void g(float2 (&x)[4]) const { at.template load<FULL>(tl.g, x); }
  __device__ void m(float2 (&x)[4]) const { at.template load<FULL>(tl.m, x); }
  __device__ void v(float2 (&x)[4]) const { at.template load<FULL>(tl.v, x); }
  __device__ void p(float2 (&x)[4]) const { at.template load<FULL>(tl.weights(), x); }
  __device__ float2 scales(int warp) const {
    return make_float2(tl.m_scale[warp], tl.v_scale[warp]);
  }
  __device__ void done() const {}
};

// One block of one tensor by one warp.
template <int W, bool GBF16, bool S8, bool FULL, class From>
__device__ __forceinline__ void step_block(const Tile<W, GBF16, S8>& tl, int warp, int lane,
                                           const Consts& c, const Step& st, From&& from) {
  const Lane<S8> at(warp, lane, tl.n);
  const float decay = fmaf(-st.lr, tl.wd, 1.f), by = -st.lr1;
  float2 m[4], v[4], r[4];  // r: the root to 2^-23 of itself, as the weights need it
  {
    float2 g[4];
    from.g(g);
    from.m(m);
    from.v(v);
    float2 scale = make_float2(0.f, 0.f);
    if constexpr (S8) scale = from.scales(warp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (S8) {
        m[i] = mulc(m[i], scale.x);
        v[i] = mulc(v[i], scale.y);
        v[i] = mul2(v[i], v[i]);
      }
      if (st.scaled) g[i] = mulc(g[i], st.gs);
      m[i] = sum2(mulc(m[i], c.b1), mulc(g[i], c.omb1), c);
      v[i] = sum2(mulc(v[i], c.b2), mul2(mulc(g[i], c.omb2), g[i]), c);
      r[i] = make_float2(near_root(v[i].x), near_root(v[i].y));
    }
    float2 p[4];
    from.p(p);
    from.done();
    if (c.tiny_eps) {  // behind the others: in their place the branch cost fp32 states 2 %
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = make_float2(near_root_of_any(v[i].x), near_root_of_any(v[i].y));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 den = fma2(r[i], both(st.inv2), both(c.eps));
      const float2 q = mul2(m[i], make_float2(reciprocal(den.x), reciprocal(den.y)));
      p[i] = fma2(q, both(by), mulc(p[i], decay));
    }
    at.template store<FULL>(tl.p, p);
    if constexpr (W == W_BF16_MASTER) at.template store<FULL>(tl.master, p);
  }
  if constexpr (S8) {
    float top_m = 0.f, top_v = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top_m = top3(m[i].x, m[i].y, top_m);
      top_v = top3(v[i].x, v[i].y, top_v);
    }
    top_m = warp_top(top_m);
    top_v = warp_top(top_v);  // the nearest root rises with v: the largest root is its
    // even lanes take the codes' factor of m, odd ones of r: one root and reciprocal a lane
    const float top = lane & 1 ? __fsqrt_rn(top_v) : top_m;
    const bool some = !(top < kLeastTop);
    const float inv = some ? __fmul_rn(kE4m3Max, __frcp_rn(top)) : 0.f;
    const float im = __shfl_sync(0xffffffffu, inv, 0), ir = __shfl_sync(0xffffffffu, inv, 1);
    uint32_t border = ~0u;
    float least = INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = mulc(m[i], im);
      r[i] = mulc(r[i], ir);
      // The code goes by the nearest root.  This one, and its product, are off by 4 steps at
      // most, which matters only next to a border between codes (half way in the last 20
      // bits, above the subnormal codes): 8 steps from one, or below 2^-6, it is done again.
      border = __vimin3_u32(border, (__float_as_uint(r[i].x) + 0x80008u) & 0xfffffu,
                            (__float_as_uint(r[i].y) + 0x80008u) & 0xfffffu);
      least = least3(r[i].x, r[i].y, least);
    }
    if ((border <= 16u || least < 0.015625f) && ir > 0.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = make_float2(__fmul_rn(__fsqrt_rn(v[i].x), ir),
                           __fmul_rn(__fsqrt_rn(v[i].y), ir));
        if (v[i].x > 0.f) r[i].x = fmaxf(r[i].x, kE4m3Tiny);
        if (v[i].y > 0.f) r[i].y = fmaxf(r[i].y, kE4m3Tiny);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
    if (lane < 2)
      (lane ? tl.v_scale : tl.m_scale)[warp] = some ? __fmul_rn(top, 1.f / kE4m3Max) : 0.f;
  }
  at.template store<FULL>(tl.m, m);
  at.template store<FULL>(tl.v, v);
}

// 16-byte slots of a thread, kThreads apart, of two blocks: their gradient, weights and codes.
template <int W, bool GBF16>
struct Ahead {
  static constexpr int kG = GBF16 ? 1 : 2, kP = W == W_BF16 ? 1 : 2;
  static constexpr int kPitch = 16 * kThreads, kBytes = (kG + kP + 1) * kPitch;
  uint32_t slot;         // of the block taken next; the one behind it is kBytes on or back
  float2 scales, after;  // theirs
  __device__ explicit Ahead(const char* smem) : slot(smem_addr(smem) + threadIdx.x * 16) {}
  __device__ float2 fill(const Tile<W, GBF16, true>& tl, int warp, int lane, uint32_t slot) const {
    const uint32_t at = warp * kBlock + lane * 8;
    const char* g = reinterpret_cast<const char*>(tl.g + at);
    const char* p = reinterpret_cast<const char*>(tl.weights() + at);
#pragma unroll
    for (int i = 0; i < kG; ++i) copy_ahead16(slot + i * kPitch, g + 16 * i);
#pragma unroll
    for (int i = 0; i < kP; ++i) copy_ahead16(slot + (kG + i) * kPitch, p + 16 * i);
    copy_ahead8(slot + (kG + kP) * kPitch, tl.m + at);
    copy_ahead8(slot + (kG + kP) * kPitch + 8, tl.v + at);
    return make_float2(tl.m_scale[warp], tl.v_scale[warp]);
  }
  __device__ uint2 codes(uint32_t byte) const {
    uint2 a;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(a.x), "=r"(a.y)
                 : "r"(slot + (kG + kP) * kPitch + byte)
                 : "memory");
    return a;
  }
  template <int UNITS>
  __device__ void read(int unit, float2 (&v)[4]) const {
    const uint4 a = slot16(slot + unit * kPitch);
    if constexpr (UNITS == 1) {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = bf16_pair(w[i]);
    } else {
      const uint4 b = slot16(slot + (unit + 1) * kPitch);
      v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
      v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
      v[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
      v[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
  }
};
// or the slots, which take the block after next as soon as they have been read.
template <int W, bool GBF16, int CAP>
struct Copied {
  Ahead<W, GBF16>& from;
  const Batch<CAP>& b;
  int next_item, next_tile, warp, lane;
  __device__ void g(float2 (&x)[4]) const { from.template read<Ahead<W, GBF16>::kG>(0, x); }
  __device__ void p(float2 (&x)[4]) const {
    from.template read<Ahead<W, GBF16>::kP>(Ahead<W, GBF16>::kG, x);
  }
  __device__ void m(float2 (&x)[4]) const {
    const uint2 a = from.codes(0);
    decode8(a.x, a.y, x);
  }
  __device__ void v(float2 (&x)[4]) const {
    const uint2 a = from.codes(8);
    decode8(a.x, a.y, x);
  }
  uint32_t stage;
  __device__ float2 scales(int) const { return from.scales; }
  __device__ void done() const {
    const Tile<W, GBF16, true> next(b, next_item, next_tile);
    from.scales = from.after;
    if (next.n == kTile) from.after = from.fill(next, warp, lane, from.slot);
    from.slot += stage;
    commit_copies();
  }
};

// CTAs of an SM: the registers that keep the row of operations without a spill (8-bit states
// 80 a thread, with masters more: 201 M weights 582 us at 2 CTAs, 632 with 4 bytes spilled at 3).
constexpr int ctas_per_sm(int w, bool s8) { return !s8 ? 4 : w == W_BF16_MASTER ? 2 : 3; }

template <int W, bool GBF16, bool S8, int CAP>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(W, S8))
adamw_kernel(const __grid_constant__ Batch<CAP> b, const __grid_constant__ Consts c,
             const float* lr_p, const float* grad_scale, int32_t* step, bool last_launch) {
  __shared__ __align__(16) char smem[S8 ? 2 * Ahead<W, GBF16>::kBytes : 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tiles = b.first_tile[b.count];
  int tile = blockIdx.x;
  int item = 0;  // of this tile: the last tensor that begins at or before it
  for (int hi = b.count - 1; item < hi;) {
    const int mid = (item + hi + 1) >> 1;
    if (b.first_tile[mid] <= tile) item = mid;
    else hi = mid - 1;
  }
  Ahead<W, GBF16> ahead(smem);
  // the tensor of the tile at or behind `from_item` (tiles only rise)
  auto item_of = [&](int t, int from_item) {
    if (t >= tiles) return b.count;
    while (b.first_tile[from_item + 1] <= t) ++from_item;
    return from_item;
  };
  const int stride = (int)gridDim.x;
  int next_item = S8 ? item_of(tile + stride, item) : 0;
  uint32_t stage = Ahead<W, GBF16>::kBytes;
  if constexpr (S8) {
    const Tile<W, GBF16, S8> tl(b, item, tile);
    if (tl.n == kTile) ahead.scales = ahead.fill(tl, warp, lane, ahead.slot);
    commit_copies();
    const Tile<W, GBF16, S8> nx(b, next_item, tile + stride);
    if (nx.n == kTile) ahead.after = ahead.fill(nx, warp, lane, ahead.slot + stage);
    commit_copies();
  }
  Step st;
  st.scaled = grad_scale != nullptr;
  st.gs = st.scaled ? *grad_scale : 1.f;
  const int t = step[0] + 1;
  st.lr = *lr_p;
  st.lr1 = st.lr / -expm1f((float)t * c.log_b1);
  st.inv2 = rsqrtf(-expm1f((float)t * c.log_b2));
  if (!isfinite(st.gs)) {  // the same for every CTA: the step is left out as a whole
    if constexpr (S8) wait_copies<0>();
    return;
  }

  while (tile < tiles) {
    const Tile<W, GBF16, S8> tl(b, item, tile);
    // a tensor's last tile: block by block, each lane looking after its own elements
    if constexpr (S8) {
      wait_copies<1>();
      const int then = tile + 2 * stride, then_item = item_of(then, next_item);
      const Copied<W, GBF16, CAP> copied = {ahead, b, then_item, then, warp, lane, stage};
      if (tl.n == kTile) {
        step_block<W, GBF16, S8, true>(tl, warp, lane, c, st, copied);
      } else {
        copied.done();
        if (warp * kBlock < tl.n)
          step_block<W, GBF16, S8, false>(tl, warp, lane, c, st,
                                          Direct<W, GBF16, S8, false>(tl, warp, lane));
      }
      stage = 0u - stage;
      item = next_item;
      next_item = then_item;
    } else if (tl.n == kTile) {
      step_block<W, GBF16, S8, true>(tl, warp, lane, c, st,
                                     Direct<W, GBF16, S8, true>(tl, warp, lane));
    } else if (warp * kBlock < tl.n) {
      step_block<W, GBF16, S8, false>(tl, warp, lane, c, st,
                                      Direct<W, GBF16, S8, false>(tl, warp, lane));
    }
    tile += stride;
    if constexpr (!S8) item = item_of(tile, item);
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
  // fp32 states: up to 16 CTAs one after another in an SM's slot, so that the SMs that memory
  // serves faster take more of the tiles (50 M weights: 197 us, 222 with one CTA a slot that
  // stays).  8-bit states: one that stays, since a CTA's start, with no block copied ahead,
  // costs more than that gives (402 M weights: 875 us, 937 with 2 a slot).
  const int per_slot = S8 ? 1 : 16;
  const int most = tiles < cap ? tiles : cap;
  const int turns = tiles / (cap * per_slot) > 1 ? tiles / (cap * per_slot) : 1;
  const int grid = tiles < 1 ? 1 : S8 ? most : (tiles + turns - 1) / turns;
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
  // The root of a subnormal v is below 2^-63, at most 2^-63 (1 - b2)^-1/2 in the denominator:
  // from 2^24 times that on, eps hides it, and the weights take the root that is 0 there (403 M
  // with 8-bit states 877 us, with the other one 909).
  const bool tiny_eps = opt.eps < std::ldexp(1.0, -39) / std::sqrt(1.0 - opt.beta2);
  const Consts c = {(float)opt.beta1,           (float)opt.beta2,
                    (float)(1.0 - opt.beta1),   (float)(1.0 - opt.beta2),
                    (float)std::log(opt.beta1), (float)std::log(opt.beta2),
                    (float)opt.eps,             1.f,
                    tiny_eps};
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

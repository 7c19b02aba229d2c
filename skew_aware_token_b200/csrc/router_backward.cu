// Gradient of the router's logits: through the gates (what the layer's output does with
// them) and through the balance and z losses.
//
//   dgates[t, j] = <dy[t], O[tok_row[t, j]]>
//   dlogits[t, e] = p_te (a_se - sum_i a_si p_ti + zc lse_t)          (counted tokens)
//                 + sum_{j: id_j = e} g_j (dgates_j - sum_i g_i dgates_i)
//
// A group of W warps takes a token: its threads hold the columns of dy and of the k expert
// rows (16-byte loads, all k rows of a column in flight together) and one stride of the
// experts; the k products and sum_i a_i p_i leave in one reduction, after which the group's
// threads write their experts.  Bound by HBM: k d 2 bytes of O rows and d 4 of dy a token.
// p = e^(x - lse) takes the lse that the forward stored: its rounding is a relative error of
// |lse| 2^-24 in p, which a second pass over the logits for their largest would not be worth.
// The losses' part alone: 16384 tokens of 256 experts 10.0 us (34 MB, 5.1 us), of 128 experts on
// 24 sequences 8.3 us (2.6), 256 tokens of 8 experts 2.3 us.
// The rows' indices are read a token ahead and the logits before the rows: with the index's
// and the logits' latency in front of the rows, 16384 tokens of 8 x 7168 took 550 us; without
// it 356 us (2.38 GB, 6.7 TB/s: the rate of a plain copy).
#include <type_traits>
#include "train_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

struct RouterArgs {
  int T, E, k, d8, n_seq;
  long long r_max;
};

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// W warps a token, kEpt experts a thread, at most K choices a token.  dy == NULL: the losses'
// part alone; dloss == NULL: the gates' part alone.
template <int W, int kEpt, int K>
__global__ void __launch_bounds__(kThreads)
router_backward_kernel(const RouterArgs a, const float* __restrict__ logits,
                       const int32_t* __restrict__ ids, const float* __restrict__ gates,
                       const float* __restrict__ dy, const uint4* __restrict__ o,
                       const int32_t* __restrict__ tok_row, const uint8_t* __restrict__ mask,
                       const int32_t* __restrict__ off, const int32_t* __restrict__ counts,
                       const int32_t* __restrict__ seq_info, const float* __restrict__ lse,
                       const float* __restrict__ dloss, float* __restrict__ dgates,
                       float* __restrict__ dlogits, int32_t* __restrict__ status) {
  constexpr int kGroups = kThreads / 32 / W;
  __shared__ float red[kGroups][2][K + 1][W];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / W, warp = (threadIdx.x >> 5) % W;
  const int tid = warp * 32 + lane;
  const int step = gridDim.x * kGroups;
  int t = blockIdx.x * kGroups + group;
  // lane j holds the row of the token's j-th choice, read a token ahead
  auto row_of = [&](int token) {
    return dy && lane < a.k && token < a.T ? __ldg(tok_row + (long long)token * a.k + lane) : 0;
  };
  int next_row = row_of(t);
  float b = 0.f, z = 0.f;
  if (dloss) {
    const int n = seq_info[a.n_seq], some = seq_info[a.n_seq + 1];
    b = some > 0 ? dloss[0] * (float)a.E / ((float)a.k * (float)some) : 0.f;
    z = n > 0 ? 2.f * dloss[1] / (float)n : 0.f;
  }
  bool bad = false;
  int turn = 0;
  for (; t < a.T; t += step, turn ^= 1) {
    int my_row = next_row;
    next_row = row_of(t + step);
    // what the end of the token needs, on its way while the rows are read
    float x[kEpt], l = 0.f, g = 0.f;
    int id = -1;
    bool on = false;
    if (dloss) {
      on = !mask || mask[t];
      l = lse[t];
#pragma unroll
      for (int i = 0; i < kEpt; ++i) {
        const int e = tid + i * 32 * W;
        x[i] = e < a.E ? __ldg(logits + (long long)t * a.E + e) : 0.f;
      }
    }
    float s[K];
#pragma unroll
    for (int j = 0; j < K; ++j) s[j] = 0.f;
    if (dy) {
      if (lane < a.k) {
        g = __ldg(gates + (long long)t * a.k + lane);
        id = __ldg(ids + (long long)t * a.k + lane);
        if (id < 0 || id >= a.E) bad = true;
        if (my_row < 0 || my_row >= a.r_max) {
          bad = true;
          my_row = -1;
        }
      } else {
        my_row = -1;
      }
      int row[K];
#pragma unroll
      for (int j = 0; j < K; ++j) row[j] = __shfl_sync(0xffffffffu, my_row, j);
      for (int v = tid; v < a.d8; v += 32 * W) {
        uint4 r[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
          r[j] = row[j] >= 0 ? ld_once(o + (long long)row[j] * a.d8 + v)
                             : make_uint4(0, 0, 0, 0);
        float g8[8];
        load8(dy + ((long long)t * a.d8 + v) * 8, g8);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          float f[8];
          bf16x8_to_f32(r[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[j] = fmaf(g8[i], f[i], s[j]);
        }
      }
    }
    // the losses' part: p and a of this thread's experts
    float p[kEpt], c[kEpt], dot = 0.f;
#pragma unroll
    for (int i = 0; i < kEpt; ++i) p[i] = c[i] = 0.f;
    if (on) {
      int seq = 0;
      if (off) {
        int hi = a.n_seq - 1;  // the last sequence that begins at or before t
        while (seq < hi) {
          const int mid = (seq + hi + 1) >> 1;
          if (off[mid] <= t) seq = mid;
          else hi = mid - 1;
        }
        on = t >= off[seq] && t < off[seq + 1];
      }
      if (on) {
        const float n_s = (float)seq_info[seq];
        const float scale = n_s > 0.f ? b / (n_s * n_s) : 0.f;
#pragma unroll
        for (int i = 0; i < kEpt; ++i) {
          const int e = tid + i * 32 * W;
          if (e < a.E) {
            p[i] = expf(x[i] - l);
            c[i] = scale * (float)counts[(long long)seq * a.E + e];
            dot = fmaf(p[i], c[i], dot);
          }
        }
      }
    }
    dot = warp_sum(dot);
    float sum = warp_sums(s, lane);  // lane l: product l / (32 / K)
    if (W > 1) {
      if (lane % (32 / K) == 0) red[group][turn][lane / (32 / K)][warp] = sum;
      if (lane == 0) red[group][turn][K][warp] = dot;
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
      sum = dot = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        dot += red[group][turn][K][w];
        if (lane < K) sum += red[group][turn][lane][w];
      }
    } else {
      sum = __shfl_sync(0xffffffffu, sum, lane * (32 / K) & 31);  // lane j: product j
    }
    float out[kEpt];
#pragma unroll
    for (int i = 0; i < kEpt; ++i) out[i] = on ? p[i] * (c[i] - dot + z * l) : 0.f;
    if (dy) {
      const float mean = warp_sum(lane < a.k ? g * sum : 0.f);
      const float add = g * (sum - mean);
      if (dgates && warp == 0 && lane < a.k) dgates[(long long)t * a.k + lane] = sum;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int e = __shfl_sync(0xffffffffu, id, j);
        const float to = __shfl_sync(0xffffffffu, add, j);
#pragma unroll
        for (int i = 0; i < kEpt; ++i)
          if (e == tid + i * 32 * W) out[i] += to;
      }
    }
#pragma unroll
    for (int i = 0; i < kEpt; ++i) {
      const int e = tid + i * 32 * W;
      if (e < a.E) dlogits[(long long)t * a.E + e] = out[i];
    }
  }
  if (bad) set_status(status, MOE_STATUS_BAD_ID);
}

}  // namespace

cudaError_t launch_router_backward(const moe_cfg& c, const float* logits, const int32_t* ids,
                                   const float* gates, const float* dy, const uint16_t* o,
                                   const int32_t* tok_row, const uint8_t* mask,
                                   const int32_t* seq_off, int n_seq, const int32_t* counts,
                                   const int32_t* seq_info, const float* lse,
                                   const float* dloss, float* dgates, float* dlogits,
                                   int32_t* status, cudaStream_t st) {
  if (c.T == 0) return cudaSuccess;
  RouterArgs a;
  a.T = c.T;
  a.E = c.E;
  a.k = c.k;
  a.d8 = dy ? c.d / 8 : 0;
  a.n_seq = n_seq;
  a.r_max = max_rows(c);
  auto run = [&](auto kernel, int W) {
    const int per_cta = kThreads / 32 / W;
    const int want = (c.T + per_cta - 1) / per_cta, cap = num_sms() * 8;
    kernel<<<want < cap ? want : cap, kThreads, 0, st>>>(
        a, logits, ids, gates, dy, reinterpret_cast<const uint4*>(o), tok_row, mask, seq_off,
        counts, seq_info, lse, dloss, dgates, dlogits, status);
    return cudaGetLastError();
  };
  auto choices = [&](auto w, auto ept) {
    constexpr int W = decltype(w)::value, kEpt = decltype(ept)::value;
    if (c.k <= 2 || !dy) return run(router_backward_kernel<W, kEpt, 2>, W);
    if (c.k <= 4) return run(router_backward_kernel<W, kEpt, 4>, W);
    return run(router_backward_kernel<W, kEpt, 8>, W);
  };
  auto warps = [&](auto w) {
    constexpr int W = decltype(w)::value;
    const int ept = (c.E + 32 * W - 1) / (32 * W);
    if constexpr (W <= 1)
      if (ept > 4) return choices(w, std::integral_constant<int, 8>());
    if constexpr (W <= 2)
      if (ept > 2) return choices(w, std::integral_constant<int, 4>());
    if constexpr (W <= 2)
      if (ept > 1) return choices(w, std::integral_constant<int, 2>());
    return choices(w, std::integral_constant<int, 1>());
  };
  // Warps a token, by the 16-byte loads that a token is (k rows of O, twice that of dy) and
  // the tokens there are.  Measured us, 1 | 2 | 8 warps a token: 16384 tokens of 8 x 2048
  // (2560 loads) 151 | 141 | 119, 4096 of them 41 | 42 | 34, 1 token of 8 x 7168 39 | 11 | 5;
  // below that the end of a token costs more than its rows and fewer warps share it: 16384 of
  // 8 x 1024 (1280) 80 | 77 | 95, of 2 x 4096 105 | 99 | 116, of 4 x 512 (384) 27 | 29 | 85, 4096
  // of them 6.9 | 8.4 | 21; with few tokens a second warp finds an idle SM: 2048 of 4 x 1024
  // 9.8 | 6.8 | 12.3, 1111 of 4 x 512 4.0 | 3.5 | 6.1.
  const int loads = a.d8 * (c.k + 2), sms = num_sms();
  if (loads >= 2560 || (loads && c.T < sms)) return warps(std::integral_constant<int, 8>());
  if (loads >= 1024 || c.T < sms * 16) return warps(std::integral_constant<int, 2>());
  return warps(std::integral_constant<int, 1>());
}

}  // namespace moe

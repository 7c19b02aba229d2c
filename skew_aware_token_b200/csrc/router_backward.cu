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

// W warps a token.  K8: k rows of O are read (k <= 8), else the losses' part alone.
template <int W>
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
  constexpr int kEpt = kMaxE / (32 * W);  // experts a thread
  __shared__ float red[kGroups][2][kMaxK + 1][W];
  const int lane = threadIdx.x & 31;
  const int group = (threadIdx.x >> 5) / W, warp = (threadIdx.x >> 5) % W;
  const int tid = warp * 32 + lane;
  float b = 0.f, z = 0.f;
  if (dloss) {
    const int n = seq_info[a.n_seq], some = seq_info[a.n_seq + 1];
    b = some > 0 ? dloss[0] * (float)a.E / ((float)a.k * (float)some) : 0.f;
    z = n > 0 ? 2.f * dloss[1] / (float)n : 0.f;
  }
  bool bad = false;
  int turn = 0;
  for (int t = blockIdx.x * kGroups + group; t < a.T; t += gridDim.x * kGroups, turn ^= 1) {
    // the losses' part: p and a of this thread's experts
    float p[kEpt], c[kEpt], zt = 0.f;
#pragma unroll
    for (int i = 0; i < kEpt; ++i) p[i] = c[i] = 0.f;
    float s[kMaxK + 1];
#pragma unroll
    for (int j = 0; j <= kMaxK; ++j) s[j] = 0.f;
    if (dloss) {
      int seq = 0;
      bool on = !mask || mask[t];
      if (off) {
        int lo = 0, hi = a.n_seq - 1;  // the last sequence that begins at or before t
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (off[mid] <= t) lo = mid;
          else hi = mid - 1;
        }
        seq = lo;
        on = on && t >= off[seq] && t < off[seq + 1];
      }
      if (on) {
        const float l = lse[t], n_s = (float)seq_info[seq];
        const float scale = b / (n_s * n_s);
        zt = z * l;
#pragma unroll
        for (int i = 0; i < kEpt; ++i) {
          const int e = tid + i * 32 * W;
          if (e < a.E) {
            p[i] = expf(logits[(long long)t * a.E + e] - l);
            c[i] = scale * (float)counts[(long long)seq * a.E + e];
            s[kMaxK] = fmaf(p[i], c[i], s[kMaxK]);
          }
        }
      }
    }
    if (dy) {
      int row[kMaxK];
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        row[j] = j < a.k ? __ldg(tok_row + (long long)t * a.k + j) : -1;
        if (j < a.k && (row[j] < 0 || row[j] >= a.r_max)) {
          bad = true;
          row[j] = -1;
        }
      }
      for (int v = tid; v < a.d8; v += 32 * W) {
        uint4 r[kMaxK];
#pragma unroll
        for (int j = 0; j < kMaxK; ++j)
          r[j] = row[j] >= 0 ? ld_once(o + (long long)row[j] * a.d8 + v)
                             : make_uint4(0, 0, 0, 0);
        float g8[8];
        load8(dy + ((long long)t * a.d8 + v) * 8, g8);
#pragma unroll
        for (int j = 0; j < kMaxK; ++j) {
          float f[8];
          bf16x8_to_f32(r[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[j] = fmaf(g8[i], f[i], s[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j <= kMaxK; ++j) s[j] = warp_sum(s[j]);
    if (W > 1) {
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j <= kMaxK; ++j) red[group][turn][j][warp] = s[j];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
#pragma unroll
      for (int j = 0; j <= kMaxK; ++j) {
        s[j] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s[j] += red[group][turn][j][w];
      }
    }
    float out[kEpt];
#pragma unroll
    for (int i = 0; i < kEpt; ++i) out[i] = p[i] * (c[i] - s[kMaxK] + zt);
    if (dy) {
      float g[kMaxK], mean = 0.f;
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        g[j] = j < a.k ? __ldg(gates + (long long)t * a.k + j) : 0.f;
        mean = fmaf(g[j], s[j], mean);
      }
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        if (j >= a.k) break;
        const int e = __ldg(ids + (long long)t * a.k + j);
        if (e < 0 || e >= a.E) bad = true;
#pragma unroll
        for (int i = 0; i < kEpt; ++i)
          if (e == tid + i * 32 * W) out[i] = fmaf(g[j], s[j] - mean, out[i]);
        if (dgates && tid == j) dgates[(long long)t * a.k + j] = s[j];
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
  if (a.d8 <= 64) return run(router_backward_kernel<1>, 1);
  if (a.d8 <= 256) return run(router_backward_kernel<4>, 4);
  return run(router_backward_kernel<8>, 8);
}

}  // namespace moe

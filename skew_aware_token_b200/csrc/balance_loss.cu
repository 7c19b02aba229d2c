// Balance loss, z loss and per-expert counts of the router over packed sequences.
//
//   balance = (1/S+) sum_s E / (k n_s^2) sum_e c_se (sum_t p_te),   z = (1/n) sum_t lse_t^2
//
// First kernel: a CTA takes a chunk of consecutive tokens and walks the sequences inside it.
// A warp holds a few token rows at a time (lane l: experts l, l + 32, ...), takes their
// maximum and sum of exponentials, and adds the rows' probabilities to its lanes' columns;
// a sequence's end adds the warps' columns in warp order into one partial row.  Chunk i's
// part of sequence s goes to row i + s: both only rise along the tokens, and one of them
// rises from each (chunk, sequence) pair that meets to the next, so no two share a row.
// Second kernel: a CTA per sequence and 32 experts adds that sequence's partial rows in chunk
// order; the last CTA to end adds the sequences' losses in order.  No atomics on values: the
// same bits on every run.  Bound by reading the logits once, for all but the largest layers
// by the two launches.
#include "train_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFinalThreads = 512;
constexpr int kFinalWarps = kFinalThreads / 32;
constexpr int kChunks = 512;    // chunks a batch is cut into, at most
constexpr int kMinChunk = 32;   // tokens of a chunk, at least

int chunk_tokens(int T) {
  const int c = (T + kChunks - 1) / kChunks;
  return c < kMinChunk ? kMinChunk : c;
}
int num_chunks(int T) { return T > 0 ? (T + chunk_tokens(T) - 1) / chunk_tokens(T) : 0; }

// The workspace: per partial row E column sums, E counts, then n and sum lse^2; per sequence
// and 32 experts a part of its loss; per sequence its sum lse^2; the ticket.
struct Workspace {
  float* psum;
  int32_t* count;
  int32_t* tokens;
  float* zsum;
  float* part;
  float* seq_z;
  uint32_t* ticket;
};
inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }
inline int slices(int E) { return (E + 31) / 32; }
size_t layout(const moe_cfg& c, int n_seq, void* base, Workspace* w) {
  const size_t rows = (size_t)num_chunks(c.T) + n_seq;
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* q = p + at;
    at += up256(bytes);
    return q;
  };
  Workspace v;
  v.psum = reinterpret_cast<float*>(take(rows * c.E * 4));
  v.count = reinterpret_cast<int32_t*>(take(rows * c.E * 4));
  v.tokens = reinterpret_cast<int32_t*>(take(rows * 4));
  v.zsum = reinterpret_cast<float*>(take(rows * 4));
  v.part = reinterpret_cast<float*>(take((size_t)n_seq * slices(c.E) * 4));
  v.seq_z = reinterpret_cast<float*>(take((size_t)n_seq * 4));
  v.ticket = reinterpret_cast<uint32_t*>(take(4));
  if (w) *w = v;
  return at;
}

// Sequence bounds, kept inside [0, T]; NULL: one sequence of all tokens.
__device__ __forceinline__ int seq_at(const int32_t* off, int s, int T) {
  if (!off) return s == 0 ? 0 : T;
  const int v = off[s];
  return v < 0 ? 0 : v > T ? T : v;
}

// The last sequence that begins at or before token t (0 when none does), by a warp that
// probes 32 bounds at a time: one latency for up to 32 sequences, two for up to 1024.
__device__ __forceinline__ int last_at_or_before(const int32_t* off, int n_seq, int t,
                                                 int lane) {
  int lo = 0, n = n_seq;  // the answer is one of the n sequences from lo on
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, i < n && off[lo + i] <= t);
    const int k = below ? 31 - __clz(below) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

template <int EPL, int TPW>
__global__ void __launch_bounds__(kThreads)
balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                       const uint8_t* __restrict__ mask, const int32_t* __restrict__ off,
                       int T, int E, int k, int n_seq, int chunk, Workspace w,
                       float* __restrict__ lse_out, int32_t* __restrict__ status) {
  __shared__ float s_p[kWarps][32 * EPL];
  __shared__ int32_t s_count[32 * EPL];
  __shared__ float s_z[kWarps];
  __shared__ int s_n[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int begin = blockIdx.x * chunk, end = min(T, begin + chunk);
  let_successor_start();  // it waits for this kernel's end; its launch need not
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0;
  for (int e = threadIdx.x; e < 32 * EPL; e += kThreads) s_count[e] = 0;
  bool bad_value = false, bad_id = false;
  if (off) {
    // every bound is looked at by one CTA
    for (int s = blockIdx.x * kThreads + threadIdx.x; s <= n_seq; s += gridDim.x * kThreads)
      if (off[s] < 0 || off[s] > T || (s > 0 && off[s] < off[s - 1]))
        set_status(status, MOET_STATUS_BAD_SEQ);
  }
  const int lo = off ? last_at_or_before(off, n_seq, begin, lane) : 0;
  int done = begin;  // tokens before it have their lse
  for (int s = lo; s < n_seq; ++s) {
    const int from = max(done, seq_at(off, s, T));
    if (from >= end) break;
    const int to = min(end, seq_at(off, s + 1, T));
    for (int t = done + threadIdx.x; t < from; t += kThreads) lse_out[t] = 0.f;
    done = from;
    if (to <= from) continue;
    done = to;
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    float z = 0.f;
    int n = 0;
    __syncthreads();  // the counts are cleared, the last sequence's sums are read
    for (int t0 = from + warp * TPW; t0 < to; t0 += kWarps * TPW) {
      // the rows, their masks and their choices at once: a masked row is read and not used
      float x[TPW][EPL], top[TPW], sum[TPW];
      bool on[TPW];
      int id[TPW];
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        const bool row = t0 + u < to;
        on[u] = row && (!mask || mask[t0 + u]);
        id[u] = row && lane < k ? __ldg(ids + (long long)(t0 + u) * k + lane) : 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const int e = lane + 32 * i;
          x[u][i] = row && e < E ? __ldg(logits + (long long)(t0 + u) * E + e) : -INFINITY;
        }
      }
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        top[u] = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (!on[u]) x[u][i] = -INFINITY;
          bad_value |= on[u] && lane + 32 * i < E && !isfinite(x[u][i]);
          top[u] = fmaxf(top[u], x[u][i]);
        }
      }
#pragma unroll
      for (int off2 = 16; off2 > 0; off2 >>= 1)
#pragma unroll
        for (int u = 0; u < TPW; ++u)
          top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], off2));
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        if (top[u] == -INFINITY) top[u] = 0.f;  // a row of nothing: exponentials of 0
        sum[u] = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          x[u][i] = expf(x[u][i] - top[u]);
          sum[u] += x[u][i];
        }
      }
#pragma unroll
      for (int off2 = 16; off2 > 0; off2 >>= 1)
#pragma unroll
        for (int u = 0; u < TPW; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], off2);
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        if (t0 + u >= to) continue;
        const float lse = on[u] ? top[u] + logf(sum[u]) : 0.f;
        if (lane == 0) lse_out[t0 + u] = lse;
        if (!on[u]) continue;
        const float inv = sum[u] > 0.f ? 1.f / sum[u] : 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = fmaf(x[u][i], inv, acc[i]);
        z = fmaf(lse, lse, z);
        ++n;
        if (lane < k) {
          if (id[u] >= 0 && id[u] < E) atomicAdd(&s_count[id[u]], 1);
          else bad_id = true;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) s_p[warp][lane + 32 * i] = acc[i];
    if (lane == 0) {
      s_z[warp] = z;
      s_n[warp] = n;
    }
    __syncthreads();
    const long long row = (long long)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) p += s_p[i][e];
      w.psum[row * E + e] = p;
      w.count[row * E + e] = s_count[e];
      s_count[e] = 0;
    }
    if (threadIdx.x == 0) {
      float zs = 0.f;
      int ns = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        zs += s_z[i];
        ns += s_n[i];
      }
      w.zsum[row] = zs;
      w.tokens[row] = ns;
    }
  }
  for (int t = done + threadIdx.x; t < end; t += kThreads) lse_out[t] = 0.f;
  if (bad_value) set_status(status, MOE_STATUS_NONFINITE);
  if (bad_id) set_status(status, MOE_STATUS_BAD_ID);
}

__global__ void __launch_bounds__(kFinalThreads)
balance_final_kernel(const int32_t* __restrict__ off, int T, int E, int k, int n_seq, int chunk,
                     int n_slices, Workspace w, float* __restrict__ losses,
                     int32_t* __restrict__ counts, float* __restrict__ probs,
                     int32_t* seq_info) {
  __shared__ float s_p[kFinalWarps][32];
  __shared__ int32_t s_c[kFinalWarps][32];
  __shared__ float s_z[kFinalWarps];
  __shared__ int32_t s_n[kFinalWarps];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_predecessor();
  for (long long unit = blockIdx.x; unit < (long long)n_seq * n_slices; unit += gridDim.x) {
    const int s = (int)(unit / n_slices), slice = (int)(unit % n_slices);
    const int from = seq_at(off, s, T), to = seq_at(off, s + 1, T);
    const int e = slice * 32 + lane;
    float p = 0.f, z = 0.f;
    int32_t c = 0, n = 0;
    if (to > from) {
      const int i0 = from / chunk, i1 = (to - 1) / chunk;
      if (e < E) {
#pragma unroll 8
        for (int i = i0 + warp; i <= i1; i += kFinalWarps) {
          const long long row = (long long)i + s;
          p += w.psum[row * E + e];
          c += w.count[row * E + e];
        }
      }
      for (int i = i0 + threadIdx.x; i <= i1; i += kFinalThreads) {
        n += w.tokens[(long long)i + s];
        z += w.zsum[(long long)i + s];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    z = warp_sum(z);
    __syncthreads();
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    if (lane == 0) {
      s_n[warp] = n;
      s_z[warp] = z;
    }
    __syncthreads();
    if (warp == 0) {
      n = 0;
      z = 0.f;
#pragma unroll
      for (int i = 0; i < kFinalWarps; ++i) {
        n += s_n[i];
        z += s_z[i];
        if (i > 0) {
          p += s_p[i][lane];
          c += s_c[i][lane];
        }
      }
      const float mean = n > 0 ? p / (float)n : 0.f;
      if (e < E) {
        probs[(long long)s * E + e] = mean;
        counts[(long long)s * E + e] = c;
      }
      const float dot = warp_sum(e < E ? mean * (float)c : 0.f);
      if (lane == 0) {
        w.part[unit] = n > 0 ? dot / (float)n : 0.f;
        if (slice == 0) {
          seq_info[s] = n;
          w.seq_z[s] = z;
        }
      }
    }
  }
  // the last CTA to end adds the sequences
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(w.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  __shared__ double d_b[kFinalWarps], d_z[kFinalWarps];
  __shared__ int32_t i_n[kFinalWarps], i_s[kFinalWarps];
  double b = 0., z = 0.;
  int32_t n = 0, some = 0;
  for (long long i = threadIdx.x; i < (long long)n_seq * n_slices; i += kFinalThreads)
    b += (double)__ldcg(w.part + i);
  for (int s = threadIdx.x; s < n_seq; s += kFinalThreads) {
    const int32_t ns = __ldcg(seq_info + s);
    z += (double)__ldcg(w.seq_z + s);
    n += ns;
    some += ns > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    b += __shfl_xor_sync(0xffffffffu, b, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
    some += __shfl_xor_sync(0xffffffffu, some, o);
  }
  if (lane == 0) {
    d_b[warp] = b;
    d_z[warp] = z;
    i_n[warp] = n;
    i_s[warp] = some;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kFinalWarps; ++i) {
      b += d_b[i];
      z += d_z[i];
      n += i_n[i];
      some += i_s[i];
    }
    losses[0] = some > 0 ? (float)(b * E / ((double)k * some)) : 0.f;
    losses[1] = n > 0 ? (float)(z / n) : 0.f;
    seq_info[n_seq] = n;
    seq_info[n_seq + 1] = some;
  }
}

template <int EPL>
void launch_partial(const moe_cfg& c, const float* logits, const int32_t* ids,
                    const uint8_t* mask, const int32_t* off, int n_seq, const Workspace& w,
                    float* lse, int32_t* status, cudaStream_t st) {
  constexpr int TPW = EPL <= 4 ? 4 : 2;
  balance_partial_kernel<EPL, TPW><<<num_chunks(c.T), kThreads, 0, st>>>(
      logits, ids, mask, off, c.T, c.E, c.k, n_seq, chunk_tokens(c.T), w, lse, status);
}

}  // namespace

size_t balance_workspace_bytes(const moe_cfg& c, int n_seq) {
  return layout(c, n_seq, nullptr, nullptr);
}

cudaError_t launch_balance_loss(const moe_cfg& c, const float* logits, const int32_t* ids,
                                const uint8_t* mask, const int32_t* seq_off, int n_seq,
                                float* losses, int32_t* counts, float* probs,
                                int32_t* seq_info, float* lse, void* ws, int32_t* status,
                                cudaStream_t st) {
  Workspace w;
  layout(c, n_seq, ws, &w);
  if (c.T == 0) {
    const cudaError_t err = cudaMemsetAsync(w.ticket, 0, 4, st);
    if (err != cudaSuccess) return err;
  } else {
    switch ((c.E + 31) / 32) {
      case 1: launch_partial<1>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 2: launch_partial<2>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 3: launch_partial<3>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 4: launch_partial<4>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 5: launch_partial<5>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 6: launch_partial<6>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      case 7: launch_partial<7>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
      default: launch_partial<8>(c, logits, ids, mask, seq_off, n_seq, w, lse, status, st); break;
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  const int n_slices = slices(c.E);
  const long long units = (long long)n_seq * n_slices;
  const long long cap = (long long)num_sms() * 8;
  return launch_after(balance_final_kernel, dim3((unsigned)(units < cap ? units : cap)),
                      dim3(kFinalThreads), 0, st, seq_off, c.T, c.E, c.k, n_seq,
                      chunk_tokens(c.T), n_slices, w, losses, counts, probs, seq_info);
}

}  // namespace moe

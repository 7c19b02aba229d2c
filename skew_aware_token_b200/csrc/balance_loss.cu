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
// Second kernel (the same one, behind a cluster barrier, for a small batch): a CTA per sequence
// and 32 experts adds that sequence's partial rows in chunk order; the last CTA to end adds
// the sequences' losses in order.  No atomics on values: the same bits on every run.  The
// traffic is the logits once (16384 x 256: 2.6 us of HBM); what bounds it are the two dependent
// kernels, each a chain of loads, sums and barriers: 12.6 us at that size, 12.3 us on 24 packed
// sequences of 128 experts.  The first waits for its loads (DRAM at 9 %, a third of the issue
// slots taken), the second at its barriers.
#include "train_common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFinalThreads = 512;
constexpr int kFinalWarps = kFinalThreads / 32;
constexpr int kChunks = 296;    // chunks a batch is cut into, at most (2 for each of 148 SMs)
constexpr int kMinChunk = 32;   // tokens of a chunk, at least

constexpr int kCluster = 8;     // CTAs that a small batch takes in one launch
// A batch is small while the cluster's chunks are the shortest ones (8 warps of up to 4 tokens
// at a time).  One launch against two, us: 256 tokens of 8, 64, 256 experts 6.2 | 7.0, 6.6 | 6.4,
// 6.8 | 7.9; 128 tokens 6.7 | 7.2, 6.5 | 7.2, 7.0 | 8.0; 288 tokens 7.8 | 6.7, 7.2 | 7.3,
// 8.2 | 7.4; 512 tokens 7.4 | 7.4, 7.3 | 7.2, 8.7 | 8.0.
constexpr int kSmallTokens = kCluster * kMinChunk;

int chunk_tokens(int T) {
  const int n = T <= kSmallTokens ? kCluster : kChunks;
  const int c = (T + n - 1) / n;
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

struct Batch {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* off;
  int T, E, k, n_seq, chunk, n_slices;
};
struct Results {
  float* losses;
  int32_t* counts;
  float* probs;
  int32_t* seq_info;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float exp2_near(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The partial rows of one chunk (the CTA's).
template <int EPL, int TPW>
__device__ __forceinline__ void chunk_sums(const Batch& b, const Workspace& w, const Results& r) {
  const float* __restrict__ logits = b.logits;
  const int32_t* __restrict__ ids = b.ids;
  const uint8_t* __restrict__ mask = b.mask;
  const int32_t* __restrict__ off = b.off;
  const int T = b.T, E = b.E, k = b.k, n_seq = b.n_seq, chunk = b.chunk;
  float* lse_out = r.lse;
  int32_t* status = r.status;
  __shared__ float s_p[kWarps][32 * EPL];
  __shared__ int32_t s_count[32 * EPL];
  __shared__ float s_z[kWarps];
  __shared__ int s_n[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int begin = blockIdx.x * chunk, end = min(T, begin + chunk);
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
    if (to <= from) {  // an empty one: past those like it at this token (any number of them)
      if (off) s = max(s, last_at_or_before(off, n_seq, from, lane) - 1);
      continue;
    }
    done = to;
    float acc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.f;
    float z = 0.f;  // of the tokens whose lane of a turn this is
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
        float zero = 0.f;  // NaN if a logit is not finite
        top[u] = x[u][0];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if (lane + 32 * i < E) zero = fmaf(x[u][i], 0.f, zero);
          if (i > 0) top[u] = fmaxf(top[u], x[u][i]);
        }
        bad_value |= on[u] && zero != 0.f;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top[u]) : "f"(top[u]));
      }
      // e^(x - top) = 2^((x - top) log2 e): the argument's rounding, 2^-24 of it, is a relative
      // error of p that falls as p does, under 2^-22 where p > 1/16
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        sum[u] = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          x[u][i] = exp2_near((x[u][i] - top[u]) * 1.44269504f);
          sum[u] += x[u][i];
        }
      }
#pragma unroll
      for (int off2 = 16; off2 > 0; off2 >>= 1)
#pragma unroll
        for (int u = 0; u < TPW; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], off2);
      // lane u: token u's lse
      float my_sum = 1.f, my_top = 0.f;
      bool my_on = false;
#pragma unroll
      for (int u = 0; u < TPW; ++u) {
        if (lane == u) {
          my_sum = sum[u];
          my_top = top[u];
          my_on = on[u];
        }
        if (!on[u]) continue;
        const float inv = __fdividef(1.f, sum[u]);
#pragma unroll
        for (int i = 0; i < EPL; ++i) acc[i] = fmaf(x[u][i], inv, acc[i]);
        ++n;
        if (lane < k) {
          if (id[u] >= 0 && id[u] < E) atomicAdd(&s_count[id[u]], 1);
          else bad_id = true;
        }
      }
      const float lse = my_on ? my_top + logf(my_sum) : 0.f;
      if (lane < TPW && t0 + lane < to) lse_out[t0 + lane] = lse;
      z = fmaf(lse, lse, z);
    }
    z = warp_sum(z);
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

// The units (a sequence's 32 experts) of this CTA: counts, mean probabilities, part of the loss.
template <int WARPS, bool WAIT>
__device__ __forceinline__ void sequence_sums(const Batch& b, const Workspace& w,
                                              const Results& out) {
  __shared__ float s_p[WARPS][32];
  __shared__ int32_t s_c[WARPS][32];
  __shared__ float s_z[WARPS];
  __shared__ int32_t s_n[WARPS];
  const int32_t* off = b.off;
  const int T = b.T, E = b.E, n_seq = b.n_seq, chunk = b.chunk, n_slices = b.n_slices;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool waited = !WAIT;
  for (long long unit = blockIdx.x; unit < (long long)n_seq * n_slices; unit += gridDim.x) {
    const int s = (int)(unit / n_slices), slice = (int)(unit % n_slices);
    const int from = seq_at(off, s, T), to = seq_at(off, s + 1, T);
    if (!waited) {  // the bounds are the caller's, what follows is the first kernel's
      wait_for_predecessor();
      waited = true;
    }
    const int e = slice * 32 + lane;
    float p = 0.f, z = 0.f;
    int32_t c = 0, n = 0;
    if (to > from) {
      const int i0 = from / chunk, i1 = (to - 1) / chunk;
      if (e < E) {
#pragma unroll 8
        for (int i = i0 + warp; i <= i1; i += WARPS) {
          const long long row = (long long)i + s;
          p += w.psum[row * E + e];
          c += w.count[row * E + e];
        }
      }
      for (int i = i0 + threadIdx.x; i <= i1; i += WARPS * 32) {
        n += w.tokens[(long long)i + s];
        z += w.zsum[(long long)i + s];
      }
    }
    n = __reduce_add_sync(0xffffffffu, n);
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
      for (int i = 0; i < WARPS; ++i) {
        n += s_n[i];
        z += s_z[i];
        if (i > 0) {
          p += s_p[i][lane];
          c += s_c[i][lane];
        }
      }
      const float mean = n > 0 ? p / (float)n : 0.f;
      if (e < E) {
        out.probs[(long long)s * E + e] = mean;
        out.counts[(long long)s * E + e] = c;
      }
      const float dot = warp_sum(e < E ? mean * (float)c : 0.f);
      if (lane == 0) {
        w.part[unit] = n > 0 ? dot / (float)n : 0.f;
        if (slice == 0) {
          out.seq_info[s] = n;
          w.seq_z[s] = z;
        }
      }
    }
  }
}

// The losses, from every sequence's parts in order (one CTA).
template <int WARPS>
__device__ __forceinline__ void batch_sums(const Batch& bt, const Workspace& w,
                                           const Results& out) {
  const int E = bt.E, k = bt.k, n_seq = bt.n_seq, n_slices = bt.n_slices;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ double d_b[WARPS], d_z[WARPS];
  __shared__ int32_t i_n[WARPS], i_s[WARPS];
  double b = 0., z = 0.;
  int32_t n = 0, some = 0;
  for (long long i = threadIdx.x; i < (long long)n_seq * n_slices; i += WARPS * 32)
    b += (double)__ldcg(w.part + i);
  for (int s = threadIdx.x; s < n_seq; s += WARPS * 32) {
    const int32_t ns = __ldcg(out.seq_info + s);
    z += (double)__ldcg(w.seq_z + s);
    n += ns;
    some += ns > 0;
  }
  auto warp_totals = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b += __shfl_xor_sync(0xffffffffu, b, o);
      z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    some = __reduce_add_sync(0xffffffffu, some);
  };
  warp_totals();
  if ((long long)n_seq * n_slices > 32) {  // else the first warp has it all
    if (lane == 0) {
      d_b[warp] = b;
      d_z[warp] = z;
      i_n[warp] = n;
      i_s[warp] = some;
    }
    __syncthreads();
    if (warp > 0) return;
    const bool in = lane < WARPS;
    b = in ? d_b[lane] : 0.;
    z = in ? d_z[lane] : 0.;
    n = in ? i_n[lane] : 0;
    some = in ? i_s[lane] : 0;
    warp_totals();
  }
  if (threadIdx.x == 0) {
    out.losses[0] = some > 0 ? (float)b * ((float)E / ((float)k * (float)some)) : 0.f;
    out.losses[1] = n > 0 ? (float)z / (float)n : 0.f;
    out.seq_info[n_seq] = n;
    out.seq_info[n_seq + 1] = some;
  }
}

template <int EPL, int TPW>
__global__ void __launch_bounds__(kThreads, 4)
balance_partial_kernel(const Batch b, const Workspace w, const Results r) {
  let_successor_start();  // it waits for this kernel's end; its launch need not
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.ticket = 0;
  chunk_sums<EPL, TPW>(b, w, r);
}

__global__ void __launch_bounds__(kFinalThreads)
balance_final_kernel(const Batch b, const Workspace w, const Results r) {
  __shared__ bool s_last;
  sequence_sums<kFinalWarps, true>(b, w, r);
  // the last CTA to end adds the sequences
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(w.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (s_last) batch_sums<kFinalWarps>(b, w, r);
}

// Both in one launch of one cluster: its barrier, which orders the CTAs' writes, stands
// between the steps.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int EPL, int TPW>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
balance_small_kernel(const Batch b, const Workspace w, const Results r) {
  chunk_sums<EPL, TPW>(b, w, r);
  __syncthreads();
  cluster_barrier();
  sequence_sums<kWarps, false>(b, w, r);
  __syncthreads();
  cluster_barrier();
  if (blockIdx.x == 0) batch_sums<kWarps>(b, w, r);
}

template <int EPL>
cudaError_t launch(const Batch& b, const Workspace& w, const Results& r, cudaStream_t st) {
  constexpr int TPW = EPL <= 2 ? 4 : 2;
  const long long units = (long long)b.n_seq * b.n_slices;
  // A small batch of few sequences takes one launch.
  if (b.T <= kSmallTokens && units <= kCluster * 4) {
    balance_small_kernel<EPL, TPW><<<kCluster, kThreads, 0, st>>>(b, w, r);
    return cudaGetLastError();
  }
  balance_partial_kernel<EPL, TPW><<<b.T ? num_chunks(b.T) : 1, kThreads, 0, st>>>(b, w, r);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const long long cap = (long long)num_sms() * 8;
  return launch_after(balance_final_kernel, dim3((unsigned)(units < cap ? units : cap)),
                      dim3(kFinalThreads), 0, st, b, w, r);
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
  const Batch b = {logits, ids,   mask,  seq_off,           c.T,
                   c.E,    c.k,   n_seq, chunk_tokens(c.T), slices(c.E)};
  const Results r = {losses, counts, probs, seq_info, lse, status};
  switch ((c.E + 31) / 32) {
    case 1: return launch<1>(b, w, r, st);
    case 2: return launch<2>(b, w, r, st);
    case 3: return launch<3>(b, w, r, st);
    case 4: return launch<4>(b, w, r, st);
    case 5: return launch<5>(b, w, r, st);
    case 6: return launch<6>(b, w, r, st);
    case 7: return launch<7>(b, w, r, st);
    default: return launch<8>(b, w, r, st);
  }
}

}  // namespace moe

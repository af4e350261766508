// Balance loss, z loss, per-expert counts and the gradient of the router's logits.
//
// With c[s,e] the number of valid tokens of sequence s that chose expert e, n_s its valid tokens
// and n all of them, the balance loss is a sum over tokens once c is known:
//   balance = sum_t a_s <c_s, p_t>,  a_s = alpha E / (k n n_s),  s = the token's sequence,
//   dl_t = p_t (a_s (c_s - <c_s, p_t>) + b lse_t),  b = 2 z_coef / n,
// so one pass over the logits gives loss and gradient.  Two launches: the counts (integers, in
// shared memory, one thread-block cluster per sequence), then that pass, whose blocks start while
// the counts are taken and whose last block joins the blocks' losses in a fixed order.
#include <algorithm>
#include <cmath>

#include "mok_vec.cuh"

namespace mok {

constexpr int kBalThreads = 256;
constexpr int kBalMaxBlocks = 1024;
constexpr int kBalBlocksPerSm = 3;
constexpr int kCountThreads = 512;

struct BalanceParams {
  const float* logits;
  const int32_t* topk_idx;
  const int32_t* seq_offsets;  // [S + 1] or NULL
  const uint8_t* mask;         // or NULL
  const float* grad;           // or NULL
  int32_t* counts;             // [S, E]
  int32_t* n_seq;              // [S], then the ticket of the pass's blocks
  float2* partial;             // [blocks] {sum a <c, p>, sum b lse^2}
  float* loss;
  float* dlogits;              // or NULL
  int* status;
  int64_t T;
  int S, E, k;
  float alpha, z_coef;
};

// First token of sequence s (s = S: the end of the last one), within [0, T].
__device__ __forceinline__ int64_t sequence_begin(const BalanceParams& p, int s) {
  if (!p.seq_offsets) return s ? p.T : 0;
  return min(max((int64_t)p.seq_offsets[s], (int64_t)0), p.T);
}

// The k experts of a token.  VEC: k is 4 or 8 and the rows are 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ void load_routes(const BalanceParams& p, int64_t t, int (&e)[kMaxK]) {
#pragma unroll
  for (int j = 0; j < kMaxK; j += 4) {
    if constexpr (VEC) {
      if (j < p.k) {
        const int4 q = *reinterpret_cast<const int4*>(p.topk_idx + t * p.k + j);
        e[j] = q.x;
        e[j + 1] = q.y;
        e[j + 2] = q.z;
        e[j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = j; i < j + 4; ++i)
        if (i < p.k) e[i] = p.topk_idx[t * p.k + i];
    }
  }
}

// One cluster of C blocks (C = 1: one block) per sequence; a thread takes a token at a time, two
// under way.  Every rank counts in its own shared memory, then adds up a C-th of the experts over
// all ranks.  Bound by latency: of the routes' loads, of shared-memory additions to the experts
// that many tokens choose, and of two cluster barriers.  The whole call at T = 16384, E = 384, k = 8
// with one sequence takes 30 / 21 / 16.5 / 14.3 us with C = 1 / 2 / 4 / 8, with 37 sequences 16.1 /
// 14.8 / 14.4 / 15.1, with 200 14.2 / 15.5 / 18.7 / 25.8; a thread per route instead of per token
// 16.1 us (one sequence, C = 8), 22 with a mask.
template <bool VEC>
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const __grid_constant__ BalanceParams p, int C) {
  __shared__ int hist[kMaxE + 1];  // the last one: valid tokens
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x / C, rank = C > 1 ? (int)cluster_ctarank() : 0;
  for (int e = threadIdx.x; e <= p.E; e += kCountThreads) hist[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.n_seq[p.S] = 0;
  const int64_t first = sequence_begin(p, s), end = sequence_begin(p, s + 1);
  __syncthreads();
  const int64_t step = (int64_t)C * kCountThreads;
  int own = 0;
  for (int64_t t = first + (int64_t)rank * kCountThreads + threadIdx.x; t < end; t += 2 * step) {
    int e[2][kMaxK];
    bool valid[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = t + i * step;
      valid[i] = at < end;
      if (valid[i]) {
        load_routes<VEC>(p, at, e[i]);
        if (p.mask) valid[i] = p.mask[at] != 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!valid[i]) continue;
      ++own;
#pragma unroll
      for (int j = 0; j < kMaxK; ++j) {
        if (j >= p.k) continue;
        if ((uint32_t)e[i][j] < (uint32_t)p.E) atomicAdd(&hist[e[i][j]], 1);
        else record_status(p.status, MOK_ERR_DEVICE_CHECK);
      }
    }
  }
  own = __reduce_add_sync(0xffffffffu, own);
  if ((threadIdx.x & 31) == 0 && own) atomicAdd(&hist[p.E], own);
  if (C > 1) cluster_sync();
  else __syncthreads();
  const int per = (p.E + 1 + C - 1) / C;
  for (int e = rank * per + threadIdx.x; e < min(p.E + 1, (rank + 1) * per); e += kCountThreads) {
    int n = 0;
    if (C > 1) {
      for (int q = 0; q < C; ++q) {
        int v;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(&hist[e]), (uint32_t)q)));
        n += v;
      }
    } else {
      n = hist[e];
    }
    if (e < p.E) p.counts[(int64_t)s * p.E + e] = n;
    else p.n_seq[s] = n;
  }
  if (C > 1) cluster_sync();  // the others read this block's counts until here
}

// Sequence of token t, or -1; a warp searches 32 of the S + 1 offsets at a time.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int64_t t, int lane) {
  if (!offsets) return 0;
  int lo = 0, hi = S + 1;  // the first offset above t is in [lo, hi]
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int at = min(lo + (lane + 1) * step - 1, hi - 1);
    const int below = __popc(__ballot_sync(0xffffffffu, offsets[at] <= t));
    lo = min(lo + below * step, hi);
    hi = min(lo + step, hi);
  }
  lo += __popc(__ballot_sync(0xffffffffu, lo + lane < hi && offsets[min(lo + lane, S)] <= t));
  return lo - 1 < S ? lo - 1 : -1;
}
// The offsets in shared memory, where they fit; the block synchronises before it reads them.
constexpr int kOffsets = 1024;
__device__ __forceinline__ const int32_t* near_offsets(const BalanceParams& p, int32_t* smem, int threads) {
  if (!p.seq_offsets || p.S >= kOffsets) return p.seq_offsets;
  for (int i = threadIdx.x; i <= p.S; i += threads) smem[i] = p.seq_offsets[i];
  return smem;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Losses and gradients of the tokens [t, end) of a warp (neighbours, so that the counts of their
// sequence stay in registers); the warp's {sum a <c, p>, sum b lse^2}, the same in all lanes.  Lane i holds the 4-element vectors i, i + 32, ... of a
// token's logits (EV of them); the next kRing tokens' come into a ring in shared memory by
// asynchronous copies, each lane's to where it reads them back itself.  exp(l - max) is
// 2^((l - max) log2 e), the difference first: l log2 e overflows for finite logits, and from 2e9 on
// its rounding alone is more than the exponential's range.
// ready() comes before the first use of counts and n_seq and returns the number of valid tokens;
// sequence(t, s) is the sequence of a token, or -1, s the one of a token before it, or -1.
constexpr float kLog2e = 1.4426950408889634f;
constexpr int ring_of(int ev) { return ev == 4 ? 2 : 3; }  // rows; at most 36 KB per block
template <int EV, class Ready, class Sequence>
__device__ __forceinline__ float2 balance_tokens(const BalanceParams& p, int64_t t, int64_t end, uint32_t ring,
                                                 Ready ready, Sequence sequence) {
  constexpr int kRing = ring_of(EV);
  const int lane = threadIdx.x & 31, nvec = p.E / 4;
  ring += 16 * lane;
  auto fetch = [&](int64_t row, int slot) {
    if (row < end) {
      const float4* src = reinterpret_cast<const float4*>(p.logits) + row * nvec + lane;
#pragma unroll
      for (int i = 0; i < EV; ++i)
        if (lane + 32 * i < nvec) copy16(ring + (slot * EV + i) * 512, src + 32 * i);
    }
    copies_end();
  };
  auto mask = [&](int64_t row) { return row < end && p.mask ? (uint32_t)p.mask[row] : 1u; };
#pragma unroll
  for (int k = 0; k < kRing; ++k) fetch(t + k, k);
  uint32_t mask_now = mask(t), mask_next = mask(t + 1);
  const float inv_n = 1.0f / (float)max(ready(), 1);
  const float g = p.grad ? *p.grad : 1.0f;
  const float a_all = p.alpha * (float)p.E / (float)p.k * inv_n, b_all = 2.0f * p.z_coef * inv_n;
  float2 sum = make_float2(0.0f, 0.0f);
  float2 c[2 * EV];
  float a = 0.0f;
  int s_held = -1, slot = 0;
  for (; t < end; ++t) {
    const int s = mask_now ? sequence(t, s_held) : -1;
    mask_now = mask_next;
    mask_next = mask(t + 2);
    float2 l[2 * EV];
    float top = -INFINITY;
    copies_wait<kRing - 1>();
#pragma unroll
    for (int i = 0; i < EV; ++i) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (lane + 32 * i < nvec) v = ld_shared_v4(ring + (slot * EV + i) * 512);
      l[2 * i] = make_float2(v.x, v.y);
      l[2 * i + 1] = make_float2(v.z, v.w);
      top = fmaxf(top, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
    }
    fetch(t + kRing, slot);  // the reads of this place come before in program order
    slot = slot + 1 == kRing ? 0 : slot + 1;
    if (s != s_held && s >= 0) {
      s_held = s;
      a = a_all / (float)p.n_seq[s];
      const int4* src = reinterpret_cast<const int4*>(p.counts) + (int64_t)s * nvec + lane;
#pragma unroll
      for (int i = 0; i < EV; ++i) {
        const int4 ci = lane + 32 * i < nvec ? src[32 * i] : make_int4(0, 0, 0, 0);
        c[2 * i] = make_float2((float)ci.x, (float)ci.y);
        c[2 * i + 1] = make_float2((float)ci.z, (float)ci.w);
      }
    }
    bool live = s >= 0;
    float q = 0.0f, inner = 0.0f, b = 0.0f;
    if (live) {
      top = warp_max(top);
      if (top == -INFINITY) top = 0.0f;
      float2 total2 = make_float2(0.0f, 0.0f), inner2 = total2;
#pragma unroll
      for (int i = 0; i < 2 * EV; ++i) {
        const float2 x = __fmul2_rn(__fadd2_rn(l[i], make_float2(-top, -top)), make_float2(kLog2e, kLog2e));
        l[i] = make_float2(exp2_approx(x.x), exp2_approx(x.y));
        total2 = __fadd2_rn(total2, l[i]);
        inner2 = __ffma2_rn(c[i], l[i], inner2);
      }
      float2 r = make_float2(total2.x + total2.y, inner2.x + inner2.y);
#pragma unroll
      for (int o = 16; o; o >>= 1)
        r = __fadd2_rn(r, make_float2(__shfl_xor_sync(0xffffffffu, r.x, o), __shfl_xor_sync(0xffffffffu, r.y, o)));
      live = r.x != 0.0f;  // nothing but -inf: no loss, no gradient (a NaN total stays live)
      if (live) {
        const float inv = 1.0f / r.x, lse = top + logf(r.x);
        inner = r.y * inv;
        b = b_all * lse;
        sum.x += a * inner;
        sum.y += b * lse;  // not lse^2 alone: it may overflow where the z loss does not, or is off
        q = g * inv;
      }
    }
    if (p.dlogits) {
      float4* dst = reinterpret_cast<float4*>(p.dlogits) + t * nvec + lane;
      const float2 q2 = make_float2(q, q), a2 = make_float2(a, a), b2 = make_float2(b, b), i2 = make_float2(-inner, -inner);
#pragma unroll
      for (int i = 0; i < EV; ++i) {
        if (lane + 32 * i < nvec) {
          float2 lo = make_float2(0.0f, 0.0f), hi = lo;
          if (live) {
            lo = __fmul2_rn(__fmul2_rn(l[2 * i], q2), __ffma2_rn(a2, __fadd2_rn(c[2 * i], i2), b2));
            hi = __fmul2_rn(__fmul2_rn(l[2 * i + 1], q2), __ffma2_rn(a2, __fadd2_rn(c[2 * i + 1], i2), b2));
          }
          dst[32 * i] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  }
  return sum;
}

// Sum over the block's warps, in order; in thread 0.
__device__ __forceinline__ float2 block_join(float2 v, float2* smem, int warps) {
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int w = 1; w < warps && threadIdx.x == 0; ++w) {
    v.x += smem[w].x;
    v.y += smem[w].y;
  }
  return v;
}
__device__ __forceinline__ void write_loss(const BalanceParams& p, float2 v) {
  p.loss[0] = v.x;
  p.loss[1] = 0.5f * v.y;  // b = 2 z_coef / n
}

// Valid tokens of all sequences (every thread of the block calls this).
__device__ __forceinline__ int valid_tokens(const BalanceParams& p, const int32_t* n_seq, int* smem, int threads) {
  if (!p.mask) return (int)max(sequence_begin(p, p.S) - sequence_begin(p, 0), (int64_t)0);
  int own = 0;
  for (int s = threadIdx.x; s < p.S; s += threads) own += n_seq[s];
  own = __reduce_add_sync(0xffffffffu, own);
  if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = own;
  __syncthreads();
  int n = 0;
  for (int w = 0; w < threads / 32; ++w) n += smem[w];
  return n;
}

// At T = 16384, E = 384, k = 8, 37 sequences (50.9 MB): 14.4 us with the counts, of 7.5 at the copy
// rate; at T = 65536 42 us of 30.  About 5 us go to the counts and the start; the pass itself (35 us
// at T = 65536, 5.8 TB/s) waits on the chain of a token's two reductions, exponentials and
// logarithm (380 instructions per token, 55% of the issue slots with 24 warps per SM).  Tokens
// strided over the warps cost 1.5 us more (the counts of a sequence are read again for every
// token), four blocks per SM 0.5, five 2.5.
template <int EV>
__global__ void __launch_bounds__(kBalThreads, kBalBlocksPerSm) balance_grad_kernel(const __grid_constant__ BalanceParams p) {
  constexpr int kWarps = kBalThreads / 32;
  __shared__ float2 smem[kWarps];
  __shared__ int total[kWarps];
  __shared__ int32_t own_offsets[kOffsets];
  __shared__ bool last;
  const int lane = threadIdx.x & 31;
  extern __shared__ __align__(16) uint8_t ring[];
  const int32_t* offsets = nullptr;
  auto ready = [&]() {
    offsets = near_offsets(p, own_offsets, kBalThreads);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are there
    __syncthreads();
    return valid_tokens(p, p.n_seq, total, kBalThreads);
  };
  const int64_t per = (p.T + (int64_t)gridDim.x * kWarps - 1) / ((int64_t)gridDim.x * kWarps);
  const int64_t first = per * ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5));
  float2 v = balance_tokens<EV>(p, first, min(first + per, p.T), smem_u32(ring) + (threadIdx.x >> 5) * (ring_of(EV) * EV * 512), ready,
                                [&](int64_t t, int s) {
                                  if (s >= 0 && (!offsets || t < offsets[s + 1])) return s;
                                  return sequence_of(offsets, p.S, t, lane);
                                });
  v = block_join(v, smem, kWarps);
  if (threadIdx.x == 0) {
    p.partial[blockIdx.x] = v;
    __threadfence();
    last = atomicAdd(p.n_seq + p.S, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  v = make_float2(0.0f, 0.0f);
  for (int i = threadIdx.x; i < gridDim.x; i += kBalThreads) {
    const float2 u = __ldcg(p.partial + i);
    v.x += u.x;
    v.y += u.y;
  }
  v = block_join(make_float2(warp_sum(v.x), warp_sum(v.y)), smem, kWarps);
  if (threadIdx.x == 0) write_loss(p, v);
}

static size_t balance_ws(int64_t S) {
  return 256 + (((size_t)S + 1) * sizeof(int32_t) + 255) / 256 * 256 + kBalMaxBlocks * sizeof(float2);
}

}  // namespace mok

extern "C" {

size_t mok_balance_loss_workspace_size(const mok_dims* dims, int64_t n_seqs) {
  using namespace mok;
  if (check_dims(dims) != MOK_OK || n_seqs < 1 || n_seqs > 0x7fffffffLL / dims->E) return 0;
  return balance_ws(n_seqs);
}

int mok_balance_loss(const mok_dims* dims, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, int64_t n_seqs, const uint8_t* token_mask,
                     float alpha, float z_coef, const float* grad, int32_t* counts, float* loss,
                     float* dlogits, void* ws, size_t ws_bytes, mok_stream_t stream) {
  using namespace mok;
  const int rc = check_dims(dims);
  if (rc != MOK_OK) return rc;
  if (n_seqs < 1 || (!seq_offsets && n_seqs != 1) || !std::isfinite(alpha) || !std::isfinite(z_coef))
    return MOK_ERR_INVALID_ARG;
  if (n_seqs > 0x7fffffffLL / dims->E) return MOK_ERR_UNSUPPORTED;
  if (!counts || !loss || !ws || (dims->T > 0 && (!logits || !topk_idx))) return MOK_ERR_INVALID_ARG;
  for (const void* q : {(const void*)logits, (const void*)counts, (const void*)dlogits, (const void*)ws})
    if (reinterpret_cast<uintptr_t>(q) & 15u) return MOK_ERR_UNSUPPORTED;
  for (const void* q : {(const void*)topk_idx, (const void*)seq_offsets, (const void*)grad, (const void*)loss})
    if (reinterpret_cast<uintptr_t>(q) & 3u) return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < balance_ws(n_seqs)) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws);
  BalanceParams p{};
  p.logits = logits;
  p.topk_idx = topk_idx;
  p.seq_offsets = seq_offsets;
  p.mask = token_mask;
  p.grad = grad;
  p.counts = counts;
  p.n_seq = reinterpret_cast<int32_t*>(w + 256);
  p.partial = reinterpret_cast<float2*>(w + balance_ws(n_seqs) - kBalMaxBlocks * sizeof(float2));
  p.loss = loss;
  p.dlogits = dlogits;
  p.status = static_cast<int*>(ws);
  p.T = dims->T;
  p.S = (int)n_seqs;
  p.E = dims->E;
  p.k = dims->k;
  p.alpha = alpha;
  p.z_coef = z_coef;
  const int ev = (p.E + 127) / 128;
  auto pick = [&](auto one, auto two, auto three, auto four) { return ev == 1 ? one : ev == 2 ? two : ev == 3 ? three : four; };
  // blocks of a sequence's cluster: a power of two up to 8 that leaves each about 100 tokens
  int C = 1;
  while (C < 8 && 2 * C * 96 * n_seqs <= p.T) C *= 2;
  const bool vec = p.k % 4 == 0 && (reinterpret_cast<uintptr_t>(topk_idx) & 15u) == 0;
  const auto count = vec ? balance_count_kernel<true> : balance_count_kernel<false>;
  cudaError_t e;
  prof_begin("balance_count", s);
  if (C > 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    cfg.gridDim = dim3((unsigned)(n_seqs * C));
    cfg.blockDim = dim3(kCountThreads);
    cfg.stream = s;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = C;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, count, p, C);
  } else {
    count<<<(unsigned)n_seqs, kCountThreads, 0, s>>>(p, 1);
    e = cudaGetLastError();
  }
  prof_end(s);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  // as many blocks as are resident together, and no more of them than give every warp its tokens
  const int64_t warps = kBalThreads / 32, most = std::min(kBalMaxBlocks, num_sms() * kBalBlocksPerSm);
  const int64_t turns = std::max<int64_t>(1, (p.T + warps * most - 1) / (warps * most));
  const int blocks = (int)std::max<int64_t>(1, (p.T + warps * turns - 1) / (warps * turns));
  prof_begin("balance_grad", s);
  e = launch_after_smem(kBalThreads / 32 * ring_of(ev) * ev * 512, pick(balance_grad_kernel<1>, balance_grad_kernel<2>, balance_grad_kernel<3>, balance_grad_kernel<4>),
                   blocks, kBalThreads, s, p);
  prof_end(s);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(2);
  return MOK_OK;
}

}  // extern "C"

// The norm after a branch with its gate, the scaled residual and the next norm in one pass, and the
// backward pass of it.
//
//   n = x rho1 post gate token_gate,  h = res_scale r + n,  v = h rho2 weight,
//   rho = 1 / sqrt(mean(row^2) + eps);
//   ds = rho2 (g - hhat mean(g hhat)) + dres,  g = dv weight,  dr = res_scale ds,
//   dx = rho1 tg (ds W - xhat mean(ds W xhat)),  W = post gate,  q = sum ds W xhat = dtoken_gate,
//   A = sum over rows of tg ds xhat:  dpost = A gate,  dgate = A post,  dweight = sum dv hhat.
//
// Both are bound by HBM and close to it by issue.  A block stays for many rows, which one thread fetches
// into a ring in shared memory by bulk copies (whole rows are contiguous) up to three rows ahead, and a
// row's sums are taken a row ahead where they do not wait for others.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mok_ring.cuh"

namespace mok {

constexpr int kSandwichMaxD = 32768;

struct SandwichParams {
  const void* x;         // bf16
  const void* residual;  // bf16 or fp32
  const void* post;
  const void* gate;          // or NULL
  const float* token_gate;   // or NULL
  const void* weight;        // or NULL: no next norm
  void* residual_out;
  void* y;                   // bf16, or NULL
  void* codes;               // or NULL
  uint8_t* scales;
  void* x_codes;             // or NULL, with the next three
  uint8_t* x_scales;
  void* h_codes;
  uint8_t* h_scales;
  int64_t T, rows;           // rows: T, or T padded to 128 (scale atoms)
  int d;
  float eps, inv_d, res_scale;
  int post_f32, gate_f32, weight_f32, atoms, depth;
  int fetched;               // rows that are fetched: T, or fewer in the self-test
  uint64_t budget;           // of a wait, ns
};

// Sums of two values over the row's threads, the same in all of them: a row is a block's, of at most 16
// warps, or a warp's (32 threads in x).  The first step of the tree leaves each half of a warp with one of
// the values.  `turn` alternates between calls: two buffers need one barrier per call.  smem is zero
// where there is no warp.
__device__ __forceinline__ void row_sums(float (&a)[2], float (&smem)[2][2][16], int turn) {
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const bool hi = lane & 16;
  float v = (hi ? a[1] : a[0]) + __shfl_xor_sync(kFull, hi ? a[0] : a[1], 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if (blockDim.x > 32) {
    if ((lane & 15) == 0) smem[turn][hi][threadIdx.x >> 5] = v;
    __syncthreads();
    v = smem[turn][hi][lane & 15];
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  }
  a[0] = __shfl_sync(kFull, v, 0);
  a[1] = __shfl_sync(kFull, v, 16);
}

// MXFP8 form of eight elements whose block of 32 lies in four neighbouring lanes.
__device__ __forceinline__ void quantise8(const Pairs& a, bool in, void* codes, int64_t at, uint8_t* scale, bool first) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(a.p[j].x), fabsf(a.p[j].y)));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int byte = mx_scale_byte(amax);
  if (!in) return;
  static_cast<uint2*>(codes)[at] = mx_codes8(a, byte);
  if (first) *scale = (uint8_t)byte;
}

// A ring of `depth` rows: each place has an mbarrier that the copies of its row complete.
struct RowRing {
  uint32_t base, place, bars;  // first place, bytes of one, first barrier
  int depth, slot;
  uint32_t phase;
  __device__ __forceinline__ uint32_t at(int ahead) const {  // place of the row `ahead` of the present one
    int k = slot + ahead;
    if (k >= depth) k -= depth;
    return base + k * place;
  }
  __device__ __forceinline__ uint32_t bar(int ahead) const {
    int k = slot + ahead;
    if (k >= depth) k -= depth;
    return bars + 8 * k;
  }
  __device__ __forceinline__ bool wait(int ahead, volatile int* abort, uint64_t budget) const {
    return mbar_wait(bar(ahead), slot + ahead >= depth ? phase ^ 1 : phase, nullptr, abort, budget);
  }
  __device__ __forceinline__ void next() {
    if (++slot == depth) {
      slot = 0;
      phase ^= 1;
    }
  }
};
template <bool F32>
__device__ __forceinline__ Pairs row_pairs(uint32_t at, int v) {  // vector v of a row in shared memory
  if constexpr (!F32) return pairs(unpack8(ring16(at + 16 * v)));
  Raw8<true> r;
  r.u[0] = ring16(at + 32 * v);
  r.u[1] = ring16(at + 32 * v + 16);
  return pairs(value8<true>(r));
}

// For the threads of a row where a wait ran out: `lost` is this thread's first row that it has not seen
// arrive, or kNoRow.  The rows from the first such row on become NaN in every output.  Copies that may still be
// under way write to shared memory, so the block does not end before they have landed (or the limit on
// waits has run out once more).
constexpr int kNoRow = 0x7fffffff;
template <bool F32>
__device__ __forceinline__ void lose_rows(const SandwichParams& p, uint32_t bars, int lost) {
  __shared__ int s_first;
  const int step = gridDim.x * blockDim.y, begin = blockIdx.x * blockDim.y + threadIdx.y, nvec = p.d >> 3;
  if (threadIdx.x == 0 && lost != kNoRow) {  // it fetches up to depth - 1 rows past the one that it has last seen
    const int n = (lost - begin) / step;
    for (int i = n; i < (n ? n + p.depth - 1 : p.depth) && begin + (int64_t)i * step < p.fetched; ++i) {
      int none = 0;
      mbar_wait(bars + 8 * (i % p.depth), (i / p.depth) & 1, nullptr, &none, p.budget);
    }
  }
  lost = __reduce_min_sync(0xffffffffu, lost);
  if (blockDim.x > 32) {
    if (threadIdx.x == 0) s_first = kNoRow;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) atomicMin(&s_first, lost);
    __syncthreads();
    lost = s_first;
  }
  Pairs a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a.p[j] = both(NAN);
  auto codes = [&](void* c, uint8_t* scales, int64_t at, int64_t s, int v) {
    static_cast<uint2*>(c)[at] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    if ((v & 3) == 0) scales[s] = 0;
  };
  for (int64_t t = lost; t < p.T; t += step) {
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
      const int64_t at = t * nvec + v;
      store_pairs<F32>(p.residual_out, at, a);
      if (p.y) store_pairs<false>(p.y, at, a);
      if (p.codes) {
        const int b = v >> 2;
        codes(p.codes, p.scales, at, p.atoms ? sf_atom_word(t >> 7, b >> 2, p.d / 128, t & 127) + (b & 3) : at >> 2, v);
      }
      if (p.x_codes) {
        codes(p.x_codes, p.x_scales, at, at >> 2, v);
        codes(p.h_codes, p.h_scales, at, at >> 2, v);
      }
    }
  }
}

// V vectors of eight per thread, MT threads at most.  Sum h^2 follows from sum x^2, which is taken beside
// the row before's sum h^2: one exchange and one barrier per row.  (Writing sum h^2 out in sums of the
// inputs, as the backward pass does with its sums, would lose rho2 where the branch cancels the residual.)
// At T = 16384, d = 7168 with a bf16 residual, codes and checkpoint (1.30 GB) 199 us, 98% of the copy
// rate, 562 instructions per warp and row; with rows by asynchronous copies of the threads' own vectors
// 234 us and 668, with scalar arithmetic and sums in every lane besides 257 and 845.
template <int V, bool F32, bool RING, int MT>
__global__ void __launch_bounds__(MT, V == 1 || MT <= 320 ? 2 : 1) sandwich_kernel(const __grid_constant__ SandwichParams p) {
  __shared__ float smem[2][2][16];
  __shared__ __align__(8) uint64_t bars[8][3];
  __shared__ int s_abort;
  extern __shared__ __align__(16) uint8_t ring[];
  const int nvec = p.d >> 3;
  const int step = gridDim.x * blockDim.y, T = (int)p.T;
  int t = blockIdx.x * blockDim.y + threadIdx.y;
  int64_t row = (int64_t)t * nvec;  // vectors before the row
  const int64_t row_step = (int64_t)step * nvec;
  constexpr int kRes = F32 ? 32 : 16;
  constexpr bool kHold = V <= 2;  // the weights in registers; else read where they are used
  RowRing q{smem_u32(ring) + threadIdx.y * p.depth * (16 + kRes) * nvec, (16u + kRes) * nvec, smem_u32(bars[threadIdx.y]), p.depth, 0, 0};
  int lost = kNoRow;
  bool in[V];
  Pairs W[kHold ? V : 1], w2[kHold ? V : 1];
  auto inner = [&](int v, bool ok) {  // post gate
    Vec8 a = load_weight(p.post, p.post_f32, v, ok);
    if (p.gate) {
      const Vec8 g = load_weight(p.gate, p.gate_f32, v, ok);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] *= g.v[j];
    }
    return pairs(a);
  };
  // the row `ahead` of the present one; every read of what is in its place has ended
  auto fetch = [&](int ahead) {
    if (RING && threadIdx.x == 0 && t + (int64_t)ahead * step < p.fetched && lost == kNoRow) {
      const int64_t from = row + ahead * row_step;
      const uint32_t at = ahead == q.depth ? q.at(0) : q.at(ahead), bar = ahead == q.depth ? q.bar(0) : q.bar(ahead);
      mbar_arrive_expect_tx(bar, q.place);
      bulk_load(at, static_cast<const uint4*>(p.x) + from, 16 * nvec, bar);
      bulk_load(at + 16 * nvec, static_cast<const char*>(p.residual) + kRes * from, kRes * nvec, bar);
    }
  };
  auto read_x = [&](int64_t from, int ahead, int v) {
    if constexpr (RING) return row_pairs<false>(q.at(ahead), v);
    else return pairs(load8<false>(p.x, from + v));
  };
  auto square_of = [&](int64_t from, int ahead) {  // this thread's share of sum x^2
    float2 ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        const Pairs a = read_x(from, ahead, threadIdx.x + i * blockDim.x);
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = __ffma2_rn(a.p[j], a.p[j], ss);
      }
    }
    return ss.x + ss.y;
  };
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = i < V - 1 || threadIdx.x + i * blockDim.x < nvec;  // only the last can be past the row
  if (RING && threadIdx.x == 0) {
    for (int k = 0; k < p.depth; ++k) mbar_init(q.bars + 8 * k, 1);
    if (threadIdx.y == 0) s_abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.y == 0)
    for (int i = threadIdx.x; i < 64; i += blockDim.x) (&smem[0][0][0])[i] = 0.0f;
  __syncthreads();
  for (int k = 0; k < p.depth; ++k) fetch(k);
  float gate = 1.0f, next_gate = 1.0f;
  if (p.token_gate && t < T) gate = p.token_gate[t];
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) {
    W[i] = inner(threadIdx.x + i * blockDim.x, in[i]);
    w2[i] = pairs(p.weight ? load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, in[i]) : Vec8{});
  }
  float sums[2] = {0.0f, 0.0f};
  if (t < T) {
    if constexpr (RING) lost = q.wait(0, &s_abort, p.budget) ? kNoRow : t;
    sums[1] = square_of(row, 0);
  }
  row_sums(sums, smem, 1);
  const float2 a2 = both(p.res_scale);
  for (int turn = 0; t < T; turn ^= 1) {
    const bool more = t + step < T;
    if (p.token_gate && more) next_gate = p.token_gate[t + step];
    const float2 rho1 = both(rsqrtf(fmaf(sums[1], p.inv_d, p.eps)) * gate);
    Pairs h[V];
    float2 ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Pairs x{};
      h[i] = Pairs{};
      if (in[i]) {
        x = read_x(row, 0, v);
        if constexpr (RING) h[i] = row_pairs<F32>(q.at(0) + 16 * nvec, v);
        else h[i] = pairs(load8<F32>(p.residual, row + v));
        const Pairs w = kHold ? W[kHold ? i : 0] : inner(v, true);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i].p[j] = __ffma2_rn(__fmul2_rn(x.p[j], rho1), w.p[j], __fmul2_rn(h[i].p[j], a2));
          ss = __ffma2_rn(h[i].p[j], h[i].p[j], ss);
        }
        store_pairs<F32>(p.residual_out, row + v, h[i]);
      }
      if (p.x_codes) {
        const int64_t s = (row + v) >> 2;
        quantise8(x, in[i], p.x_codes, row + v, p.x_scales + s, (v & 3) == 0);
        quantise8(h[i], in[i], p.h_codes, row + v, p.h_scales + s, (v & 3) == 0);
      }
    }
    sums[0] = ss.x + ss.y;
    sums[1] = 0.0f;
    if (more) {
      if constexpr (RING) lost = q.wait(1, &s_abort, p.budget) ? lost : min(lost, t + step);
      sums[1] = square_of(row + row_step, 1);
    }
    row_sums(sums, smem, turn);
    if (blockDim.x == 32) __syncwarp();
    fetch(q.depth);  // into this row's place
    if (p.weight) {
      const float2 rho2 = both(rsqrtf(fmaf(sums[0], p.inv_d, p.eps)));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const Pairs w = kHold ? w2[kHold ? i : 0] : pairs(load_weight(p.weight, p.weight_f32, v, in[i]));
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i].p[j] = __fmul2_rn(__fmul2_rn(h[i].p[j], rho2), w.p[j]);
        if (p.y && in[i]) store_pairs<false>(p.y, row + v, h[i]);
        if (p.codes) {
          const int b = v >> 2;
          const int64_t s = p.atoms ? sf_atom_word(t >> 7, b >> 2, p.d / 128, t & 127) + (b & 3) : (row + v) >> 2;
          quantise8(h[i], in[i], p.codes, row + v, p.scales + s, (v & 3) == 0);
        }
      }
    }
    gate = next_gate;
    t += step;
    row += row_step;
    q.next();
  }
  if (RING && (blockDim.x > 32 ? __syncthreads_or(lost != kNoRow) : __any_sync(0xffffffffu, lost != kNoRow)))
    lose_rows<F32>(p, q.bars, lost);
  for (int64_t r = t; r < p.rows; r += step)  // padding rows of the scale atoms
    for (int kb = threadIdx.x; kb < p.d / 128; kb += blockDim.x)
      *reinterpret_cast<uint32_t*>(p.scales + sf_atom_word(r >> 7, kb, p.d / 128, (int)(r & 127))) = 0;
}

struct SandwichBwdParams {
  const void* dy;          // bf16, or NULL (no next norm), with h and weight
  const void* h;           // bf16, fp32 or codes
  const uint8_t* h_scales;
  const void* x;           // bf16 or codes
  const uint8_t* x_scales;
  const void* dres;        // or NULL
  const void* post;
  const void* gate;        // or NULL
  const float* token_gate; // or NULL
  const void* weight;
  void* dx;
  void* dresidual;
  float* dtoken_gate;      // or NULL
  float* partial;          // [2][grid][d]: A, dweight
  int* status;
  int64_t T;
  int d;
  float eps, inv_d, res_scale;
  int post_f32, gate_f32, weight_f32, depth;
  int fetched;             // rows that are fetched: T, or fewer in the self-test
  uint64_t budget;         // of a wait for a row, ns
};

// NaN in every output of the rows t, t + gridDim.x, ... and in the block's sums over rows, each thread its
// columns of the backward pass.
template <bool F32>
__device__ __forceinline__ void lose_bwd_rows(const SandwichBwdParams& p, int64_t t, int threads) {
  const int nvec = p.d >> 3;
  Pairs a;
#pragma unroll
  for (int j = 0; j < 4; ++j) a.p[j] = both(NAN);
  for (; t < p.T; t += gridDim.x) {
    for (int v = threadIdx.x; v < nvec; v += threads) {
      store_pairs<F32>(p.dresidual, t * nvec + v, a);
      store_pairs<false>(p.dx, t * nvec + v, a);
    }
    if (p.dtoken_gate && threadIdx.x == 0) p.dtoken_gate[t] = NAN;
  }
  float* mine = p.partial + (int64_t)blockIdx.x * p.d;
  for (int v = threadIdx.x; v < nvec; v += threads) {
    store_pairs<true>(mine, v, a);
    if (p.dy) store_pairs<true>(mine + (int64_t)gridDim.x * p.d, v, a);
  }
}

// Six sums of a row (an array of eight, two of them empty) over the consumer warps.  In put_sums every step
// of the tree halves the number of values that a lane still has; the four lanes of value i then hold its
// sum over the warp.  get_sums joins up to 16 warps.  smem is zero where there is no warp.
__device__ __forceinline__ void put_sums(const float (&a)[8], float (&smem)[8][16], int warp) {
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  float b[4], c[2];
  const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (h16 ? a[i + 4] : a[i]) + __shfl_xor_sync(kFull, h16 ? a[i] : a[i + 4], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = (h8 ? b[i + 2] : b[i]) + __shfl_xor_sync(kFull, h8 ? b[i] : b[i + 2], 8);
  float v = (h4 ? c[1] : c[0]) + __shfl_xor_sync(kFull, h4 ? c[0] : c[1], 4);
  v += __shfl_xor_sync(kFull, v, 2);
  v += __shfl_xor_sync(kFull, v, 1);
  if ((lane & 3) == 0) smem[lane >> 2][warp] = v;
}
__device__ __forceinline__ void get_sums(float (&a)[6], float (&smem)[8][16]) {
  constexpr unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const float4 q = reinterpret_cast<const float4*>(smem[lane >> 2])[lane & 3];
  float v = (q.x + q.y) + (q.z + q.w);
  v += __shfl_xor_sync(kFull, v, 2);
  v += __shfl_xor_sync(kFull, v, 1);
#pragma unroll
  for (int i = 0; i < 6; ++i) a[i] = __shfl_sync(kFull, v, 4 * i);
}

// PACKED: x and h come as codes and scales.  The mean over ds W xhat, which dx needs, would follow from
// ds and so from the means before it; written out,
//   sum ds W x = rho2 (sum g W x + c2 sum h W x) + sum dres W x,  c2 = - rho2^2 mean(g h),
// it takes sums of the inputs alone, so that one pass over a row gives all six sums and one exchange
// serves it; a second pass gives ds, dx and what is summed over rows.  The first pass runs a row ahead:
// its exchange (an mbarrier that the warps arrive on) ends under the second pass of the row before.
// One more warp fetches rows as their places come free.
// Rows of fp32 without codes, of which only two may fit, take the second pass first, so that the next
// fetch has the first pass and the exchange to land.
// At T = 8192, d = 7168 with a gradient through the residual 117 us from bf16 rows (704 MB, 90% of the
// copy rate) and 122.5 from codes (591 MB, 72%: 780 instructions per warp and row, some 120 more, at 62% of
// the issue slots).  With q summed from ds, in a second exchange per row, 142 us from codes and more than
// that with the weights in registers, which x, h and ds then share with it (185).
template <int V, bool F32, bool PACKED, bool RING, int MT>
__global__ void __launch_bounds__(MT) sandwich_bwd_kernel(const __grid_constant__ SandwichBwdParams p) {
  __shared__ __align__(16) float smem[2][8][16];
  __shared__ __align__(8) uint64_t s_bars[7];  // full and empty, three each; the exchange
  __shared__ int s_abort, s_stuck;  // a wait for a row, for the exchange has run out
  __shared__ int s_lost;            // the first row that a thread has not seen arrive
  extern __shared__ __align__(16) uint8_t ring[];
  const int nvec = p.d >> 3, T = (int)p.T;
  const int threads = RING ? blockDim.x - 32 : blockDim.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int t = blockIdx.x;  // gridDim.x <= T
  int64_t row = (int64_t)t * nvec;  // vectors before the row
  const int64_t row_step = (int64_t)gridDim.x * nvec;
  constexpr bool kHold = V <= 3;  // the weights in registers; else they are read where they are used
  constexpr bool kLate = F32 && !PACKED;
  const bool next_norm = p.dy != nullptr, has_res = p.dres != nullptr;
  // planes of a place: dy, dres, h, x, and for codes the two tensors' scales
  constexpr int kRes = F32 ? 32 : 16, kH = PACKED ? 8 : kRes, kX = PACKED ? 8 : 16;
  const uint32_t scale_bytes = PACKED ? (nvec / 4 + 31) & ~15 : 0;
  const uint32_t res_at = next_norm ? 16 * nvec : 0, h_at = res_at + (has_res ? kRes * nvec : 0);
  const uint32_t x_at = h_at + (next_norm ? kH * nvec : 0), xs_at = x_at + kX * nvec, hs_at = xs_at + scale_bytes;
  const uint32_t place = hs_at + (next_norm ? scale_bytes : 0), base = smem_u32(ring);
  const uint32_t full = smem_u32(s_bars), empty = full + 24, exchange = full + 48;
  if (threadIdx.x == 0) {
    for (int k = 0; k < 3; ++k) {
      mbar_init(full + 8 * k, 1);
      mbar_init(empty + 8 * k, threads >> 5);
    }
    mbar_init(exchange, threads >> 5);
    s_abort = s_stuck = 0;
    s_lost = kNoRow;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < 256; i += blockDim.x) (&smem[0][0][0])[i] = 0.0f;
  __syncthreads();

  if (RING && (int)threadIdx.x >= threads) {
    // The producer.  A row's scales need not be whole 16 bytes: those around them are copied, up to the
    // last whole ones of the tensor; what is left at its end is stored before the arrival that others
    // wait for.  It stays until its last copies have landed (or the limit on waits has run out), also where
    // the others wait no longer.
    const int64_t scale_end = PACKED ? ((p.T * nvec) >> 2) & ~(int64_t)15 : 0;
    if (lane == 0) {
      int k = 0, n = 0;
      uint32_t phase = 1;  // a place's first wait ends at once
      for (; t < p.fetched; t += gridDim.x, row += row_step, ++n) {
        if (!mbar_wait(empty + 8 * k, phase, p.status, &s_abort, p.budget)) break;
        const uint32_t at = base + k * place, bar = full + 8 * k;
        const int64_t s0 = (row >> 2) & ~(int64_t)15, s1 = min((((row + nvec) >> 2) + 15) & ~(int64_t)15, scale_end);
        const uint32_t scales = PACKED && s1 > s0 ? (uint32_t)(s1 - s0) : 0;
        if constexpr (PACKED) {
          for (int64_t b = max(s0, scale_end); b < (row + nvec) >> 2; ++b) {
            const uint32_t to = at + (uint32_t)(b - s0);
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + xs_at), "r"((uint32_t)p.x_scales[b]) : "memory");
            if (next_norm) asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + hs_at), "r"((uint32_t)p.h_scales[b]) : "memory");
          }
        }
        mbar_arrive_expect_tx(bar, xs_at + (next_norm ? 2 : 1) * scales);
        if (next_norm) bulk_load(at, static_cast<const uint4*>(p.dy) + row, 16 * nvec, bar);
        if (has_res) bulk_load(at + res_at, static_cast<const char*>(p.dres) + kRes * row, kRes * nvec, bar);
        if (next_norm) bulk_load(at + h_at, static_cast<const char*>(p.h) + kH * row, kH * nvec, bar);
        bulk_load(at + x_at, static_cast<const char*>(p.x) + kX * row, kX * nvec, bar);
        if (scales) bulk_load(at + xs_at, p.x_scales + s0, scales, bar);
        if (scales && next_norm) bulk_load(at + hs_at, p.h_scales + s0, scales, bar);
        if (++k == p.depth) {
          k = 0;
          phase ^= 1;
        }
      }
      for (int i = max(0, n - p.depth); i < n; ++i) {
        int none = 0;
        mbar_wait(full + 8 * (i % p.depth), (i / p.depth) & 1, p.status, &none, p.budget);
      }
    }
    return;
  }

  bool in[V];
  Pairs A[V], dw[V], W[kHold ? V : 1], w2[kHold ? V : 1];
  auto inner = [&](int v, bool ok) {
    Vec8 a = load_weight(p.post, p.post_f32, v, ok);
    if (p.gate) {
      const Vec8 g = load_weight(p.gate, p.gate_f32, v, ok);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] *= g.v[j];
    }
    return pairs(a);
  };
  auto weight_of = [&](int i) {
    return kHold ? w2[kHold ? i : 0] : pairs(load_weight(p.weight, p.weight_f32, threadIdx.x + i * threads, true));
  };
  auto inner_of = [&](int i) { return kHold ? W[kHold ? i : 0] : inner(threadIdx.x + i * threads, true); };
  auto read_dy = [&](int64_t from, uint32_t at, int v) {
    if constexpr (RING) return row_pairs<false>(at, v);
    else return pairs(load8<false>(p.dy, from + v));
  };
  auto read_res = [&](int64_t from, uint32_t at, int v) {
    if constexpr (RING) return row_pairs<F32>(at + res_at, v);
    else return pairs(load8<F32>(p.dres, from + v));
  };
  auto unpacked = [&](int64_t from, uint32_t at, uint32_t scales_at, const void* rows, const uint8_t* scales, int v) {
    uint2 c;
    uint32_t byte;
    if constexpr (RING) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(c.x), "=r"(c.y) : "r"(at + 8 * v));
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(byte) : "r"(scales_at + ((uint32_t)(from >> 2) & 15) + (v >> 2)));
    } else {
      c = static_cast<const uint2*>(rows)[from + v];
      byte = scales[(from + v) >> 2];
    }
    const uint4 u = e4m3_halves(c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const float2 s = both(mx_scale(byte));
    Pairs r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.p[j] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&w[j])), s);
    return r;
  };
  auto read_h = [&](int64_t from, uint32_t at, int v) {
    if constexpr (PACKED) return unpacked(from, at + h_at, at + hs_at, p.h, p.h_scales, v);
    else if constexpr (RING) return row_pairs<F32>(at + h_at, v);
    else return pairs(load8<F32>(p.h, from + v));
  };
  auto read_x = [&](int64_t from, uint32_t at, int v) {
    if constexpr (PACKED) return unpacked(from, at + x_at, at + xs_at, p.x, p.x_scales, v);
    else if constexpr (RING) return row_pairs<false>(at + x_at, v);
    else return pairs(load8<false>(p.x, from + v));
  };
  // first pass: h h, g h, x x, g W x, h W x, dres W x
  auto first = [&](int64_t from, uint32_t at, int turn) {
    float2 s[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) s[k] = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        const int v = threadIdx.x + i * threads;
        const Pairs x = read_x(from, at, v), w = inner_of(i);
        Pairs wx;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[2] = __ffma2_rn(x.p[j], x.p[j], s[2]);
          wx.p[j] = __fmul2_rn(x.p[j], w.p[j]);
        }
        if (next_norm) {
          const Pairs h = read_h(from, at, v), dy = read_dy(from, at, v), u = weight_of(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 g = __fmul2_rn(dy.p[j], u.p[j]);
            s[0] = __ffma2_rn(h.p[j], h.p[j], s[0]);
            s[1] = __ffma2_rn(h.p[j], g, s[1]);
            s[3] = __ffma2_rn(g, wx.p[j], s[3]);
            s[4] = __ffma2_rn(h.p[j], wx.p[j], s[4]);
          }
        }
        if (has_res) {
          const Pairs r = read_res(from, at, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[5] = __ffma2_rn(r.p[j], wx.p[j], s[5]);
        }
      }
    }
    float a[8];
#pragma unroll
    for (int k = 0; k < 6; ++k) a[k] = s[k].x + s[k].y;
    a[6] = a[7] = 0.0f;
    put_sums(a, smem[turn], warp);
    __syncwarp();
    if (lane == 0) mbar_arrive(exchange);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = i < V - 1 || (int)threadIdx.x + i * threads < nvec;  // only the last can be past the row
#pragma unroll
    for (int j = 0; j < 4; ++j) A[i].p[j] = dw[i].p[j] = both(0.0f);
  }
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) {
    const int v = threadIdx.x + i * threads;
    W[i] = inner(v, in[i]);
    w2[i] = pairs(next_norm ? load_weight(p.weight, p.weight_f32, v, in[i]) : Vec8{});
  }
  float gate = p.token_gate ? p.token_gate[t] : 1.0f, next_gate = 1.0f;
  float sums[6];
  const float2 a2 = both(p.res_scale);
  uint32_t at = base, phase = 0;  // the row's place in the ring and its phase
  int k = 0, turn = 0;
  // Every warp arrives on the exchange once its wait for the row has ended, so that the wait for the
  // others runs out later than theirs and does not heed s_abort.
  if constexpr (RING)
    if (!mbar_wait(full, 0, p.status, &s_abort, p.budget)) atomicMin(&s_lost, t);
  first(row, at, 0);
  if (!mbar_wait(exchange, 0, p.status, &s_stuck, 2 * p.budget)) atomicMin(&s_lost, t);
  get_sums(sums, smem[0]);
  while (true) {
    const bool more = t + (int)gridDim.x < T;
    const int next_k = k + 1 == p.depth ? 0 : k + 1;
    const uint32_t next_phase = next_k ? phase : phase ^ 1, next_at = base + next_k * place;
    turn ^= 1;
    auto ahead = [&]() {
      if (!more) return;
      if (p.token_gate) next_gate = p.token_gate[t + gridDim.x];
      if constexpr (RING)
        if (!mbar_wait(full + 8 * next_k, next_phase, p.status, &s_abort, p.budget)) atomicMin(&s_lost, t + (int)gridDim.x);
      first(row + row_step, next_at, turn);
    };
    if constexpr (!kLate) ahead();
    const float rho1 = rsqrtf(fmaf(sums[2], p.inv_d, p.eps)), rho2 = rsqrtf(fmaf(sums[0], p.inv_d, p.eps));
    const float c2 = -sums[1] * p.inv_d * rho2 * rho2;  // - mean(g hhat) rho2
    const float q = fmaf(rho2, fmaf(c2, sums[4], sums[3]), sums[5]);
    const float2 r2 = both(rho2), cc2 = both(c2), rt = both(rho1 * gate), c1 = both(-q * p.inv_d * rho1 * rho1);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        const int v = threadIdx.x + i * threads;
        Pairs ds = has_res ? read_res(row, at, v) : Pairs{}, o;
        if (next_norm) {
          const Pairs h = read_h(row, at, v), dy = read_dy(row, at, v), u = weight_of(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i].p[j] = __ffma2_rn(dy.p[j], __fmul2_rn(h.p[j], r2), dw[i].p[j]);
            ds.p[j] = __ffma2_rn(__ffma2_rn(h.p[j], cc2, __fmul2_rn(dy.p[j], u.p[j])), r2, ds.p[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o.p[j] = __fmul2_rn(ds.p[j], a2);
        store_pairs<F32>(p.dresidual, row + v, o);
        const Pairs x = read_x(row, at, v), w = inner_of(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          A[i].p[j] = __ffma2_rn(__fmul2_rn(ds.p[j], x.p[j]), rt, A[i].p[j]);
          o.p[j] = __fmul2_rn(__ffma2_rn(x.p[j], c1, __fmul2_rn(ds.p[j], w.p[j])), rt);
        }
        store_pairs<false>(p.dx, row + v, o);
      }
    }
    if (p.dtoken_gate && threadIdx.x == 0) p.dtoken_gate[t] = rho1 * q;
    if constexpr (RING) {
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * k);
    }
    if constexpr (kLate) ahead();
    if (!more) break;
    t += gridDim.x;
    if (!mbar_wait(exchange, turn, p.status, &s_stuck, 2 * p.budget)) atomicMin(&s_lost, t);
    get_sums(sums, smem[turn]);
    gate = next_gate;
    row += row_step;
    k = next_k;
    phase = next_phase;
    at = next_at;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float* mine = p.partial + (int64_t)blockIdx.x * p.d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * threads;
    if (in[i]) {
      store_pairs<true>(mine, v, A[i]);
      if (next_norm) store_pairs<true>(mine + (int64_t)gridDim.x * p.d, v, dw[i]);
    }
  }
  asm volatile("barrier.cta.sync 1, %0;" ::"r"(threads) : "memory");  // the producer has no part in it
  if (s_lost != kNoRow) lose_bwd_rows<F32>(p, s_lost, threads);
}

// Sums the n partial rows of A (blockIdx.y == 0) and of dweight (1) in a fixed order.  A block takes 32
// columns: lane l of warp w adds the rows 4 w + l / 8, + 64, ... of the columns 4 (l % 8) .., then the
// four rows of a warp and the warps are joined.
constexpr int kSumWarps = 16;
struct SandwichSumParams {
  const float* partial;
  int n, d;
  const void* post;
  const void* gate;  // or NULL
  float* dpost;
  float* dgate;      // or NULL
  float* dweight;    // or NULL
  int post_f32, gate_f32;
};
__device__ __forceinline__ float4 weight4(const void* w, int f32, int c) {  // columns 4 c ..
  if (f32) return static_cast<const float4*>(w)[c];
  const uint2 u = static_cast<const uint2*>(w)[c];
  return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
}
__global__ void __launch_bounds__(32 * kSumWarps) sandwich_sum_kernel(const __grid_constant__ SandwichSumParams p) {
  __shared__ float4 smem[kSumWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 8 + (lane & 7);  // group of four columns
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first pass still runs
  const float* rows = p.partial + (int64_t)blockIdx.y * p.n * p.d;
  if (4 * c < p.d) {
#pragma unroll 8
    for (int r = 4 * warp + (lane >> 3); r < p.n; r += 4 * kSumWarps) {
      const float4 v = reinterpret_cast<const float4*>(rows + (int64_t)r * p.d)[c];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, o);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, o);
  }
  if (lane < 8) smem[warp][lane] = a;
  __syncthreads();
  if (warp != 0 || lane >= 8 || 4 * c >= p.d) return;
  for (int w = 1; w < kSumWarps; ++w) {
    const float4 v = smem[w][lane];
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  auto times = [](float4 u, float4 v) { return make_float4(u.x * v.x, u.y * v.y, u.z * v.z, u.w * v.w); };
  if (blockIdx.y == 1) {
    reinterpret_cast<float4*>(p.dweight)[c] = a;
  } else {
    reinterpret_cast<float4*>(p.dpost)[c] = p.gate ? times(a, weight4(p.gate, p.gate_f32, c)) : a;
    if (p.dgate) reinterpret_cast<float4*>(p.dgate)[c] = times(a, weight4(p.post, p.post_f32, c));
  }
}

// What mok_selftest_lost_rows asks of the next call of this host thread.
struct LostRows {
  int64_t first = -1;
  uint64_t budget = kWaitNs;
  int fetched(int64_t T) const { return (int)(first < 0 ? T : std::min(first, T)); }
};
static thread_local LostRows g_lost_rows;

static bool sandwich_sizes_ok(int64_t T, int d) {
  return T >= 0 && T <= 0x7fffffffLL / 8 && d > 0 && d <= kSandwichMaxD && d % 8 == 0;
}
static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool is4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool elem_ok(int type) { return type == MOK_T_BF16 || type == MOK_T_F32; }

// Vectors per thread, threads of a row, rows of a block, blocks per SM.
struct SandwichShape {
  int v, threads, rows, blocks;
};
constexpr int kSmemPerSm = 227 * 1024;  // for the blocks of an SM together
constexpr int kSmemOwn = 3 * 1024;      // of a block: reserved and static
constexpr int kPlainSmem = 40 * 1024;   // dynamic bytes that need no attribute
constexpr int kWideThreads = 512;       // of a block with two vectors per thread and more: 128 registers each
// Forward: one vector per thread up to 512 threads, of which 1024 fit an SM (64 registers): 2^25 elements
// with a bf16 residual at d = 4096 in 45 us, 61 with one block per SM, 40 at the copy rate.  With two
// vectors two blocks fit up to 320 threads (96 registers): T = 8192, d = 5120 58 us, 61 with one.
static SandwichShape sandwich_shape(int d) {
  SandwichShape n;
  const int nvec = d / 8;
  n.v = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 8;
  n.threads = ((nvec + n.v - 1) / n.v + 31) / 32 * 32;
  n.rows = n.threads == 32 ? 8 : 1;
  n.blocks = n.v == 1 ? std::max(1, std::min(1024 / (n.threads * n.rows), 8)) : n.v == 2 && n.threads <= 320 ? 2 : 1;
  return n;
}
// Backward: one warp more fetches (not for the widest rows, which have no ring).  A vector of a thread
// takes 32 registers across rows (two weights, two sums), so threads get 96 registers with one vector, 128
// with two, 168 with three, and with that warp a block has no more threads than those allow.  T = 8192 at
// d = 8192 130 us with three, 287 with four; at d = 7168 from codes 123 with two, 130 with three, 154 with
// one in 28 warps; 2^25 elements at d = 2048 76 us with two blocks per SM, 121 with one.
constexpr int kNarrowThreads = 512 + 32, kThreeThreads = 384;
static SandwichShape sandwich_bwd_shape(int d) {
  SandwichShape n;
  const int nvec = d / 8;
  n.v = nvec <= 512 ? 1 : nvec <= 2 * (kWideThreads - 32) ? 2 : nvec <= 3 * (kThreeThreads - 32) ? 3
      : nvec <= 4 * (kWideThreads - 32) ? 4 : 8;
  n.threads = ((nvec + n.v - 1) / n.v + 31) / 32 * 32;
  n.rows = 1;
  n.blocks = n.v == 1 ? std::max(1, std::min(65536 / 96 / (n.threads + 32), 8)) : 1;
  return n;
}
static int sandwich_bwd_grid(int sms, int64_t T, int d) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(T, (int64_t)sms * sandwich_bwd_shape(d).blocks));
}
// Places of the ring for the rows that a block has to take, three or (`two`) two; 0 where they do not fit and
// for the widest rows (they are then read from memory, the second time from L2).
static int ring_depth(int64_t turns, int blocks, int64_t bytes, int v, bool two) {
  if (v > 4) return 0;
  const int64_t room = kSmemPerSm / blocks - kSmemOwn;
  for (int depth = 3; depth >= (two ? 2 : 3); --depth)
    if (std::min<int64_t>(depth, turns) * bytes <= room) return (int)std::min<int64_t>(depth, turns);
  return 0;
}
template <class K>
static cudaError_t allow_smem(K k, int64_t smem) {
  if (smem <= kPlainSmem) return cudaSuccess;
  return cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm - kSmemOwn);
}

}  // namespace mok

extern "C" {

int mok_selftest_lost_rows(int64_t first, int64_t budget_ns) {
  if (first < -1 || budget_ns <= 0 || budget_ns > (int64_t)mok::kWaitNs) return MOK_ERR_INVALID_ARG;
  mok::g_lost_rows.first = first;
  mok::g_lost_rows.budget = first < 0 ? mok::kWaitNs : (uint64_t)budget_ns;
  return MOK_OK;
}

int mok_sandwich_norm(const mok_sandwich* a, int64_t T, int d, const void* x, const void* residual, void* residual_out,
                      void* y, void* codes, void* scales, int scale_layout, void* x_codes, void* x_scales,
                      void* h_codes, void* h_scales, mok_stream_t stream) {
  using namespace mok;
  if (!a) return MOK_ERR_INVALID_ARG;
  if (!sandwich_sizes_ok(T, d) || ((codes || x_codes) && d % 128)) return MOK_ERR_UNSUPPORTED;
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->res_scale)) return MOK_ERR_INVALID_ARG;
  if (!elem_ok(a->res_type) || !elem_ok(a->post_type) || !elem_ok(a->gate_type) || !elem_ok(a->weight_type) ||
      (scale_layout != MOK_SCALES_ROWS && scale_layout != MOK_SCALES_ATOMS))
    return MOK_ERR_INVALID_ARG;
  if (T > 0 && (!x || !residual || !residual_out || !a->post_weight || (codes != nullptr) != (scales != nullptr) ||
                (a->weight == nullptr) != (!y && !codes)))
    return MOK_ERR_INVALID_ARG;
  const bool save = x_codes || x_scales || h_codes || h_scales;
  if (T > 0 && save && (!x_codes || !x_scales || !h_codes || !h_scales)) return MOK_ERR_INVALID_ARG;
  for (const void* q : {x, residual, a->post_weight, a->gate, a->weight, (const void*)residual_out, (const void*)y,
                        (const void*)codes, (const void*)scales, (const void*)x_codes, (const void*)x_scales,
                        (const void*)h_codes, (const void*)h_scales})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  if (!is4(a->token_gate)) return MOK_ERR_UNSUPPORTED;
  set_last_launches(0);
  if (T == 0) return MOK_OK;
  const bool f32 = a->res_type == MOK_T_F32;
  SandwichParams p{x, residual, a->post_weight, a->gate, a->token_gate, a->weight, residual_out, y, codes,
                   static_cast<uint8_t*>(scales), x_codes, static_cast<uint8_t*>(x_scales), h_codes,
                   static_cast<uint8_t*>(h_scales), T, T, d, a->eps, 1.0f / (float)d, a->res_scale,
                   a->post_type == MOK_T_F32, a->gate_type == MOK_T_F32, a->weight_type == MOK_T_F32,
                   scale_layout == MOK_SCALES_ATOMS, 0, g_lost_rows.fetched(T), g_lost_rows.budget};
  g_lost_rows = LostRows();
  if (codes && p.atoms) p.rows = (T + 127) / 128 * 128;
  const int sms = num_sms();
  const SandwichShape n = sandwich_shape(d);
  const int64_t row_bytes = 2 * d * (f32 ? 3 : 2);
  const int64_t groups = (p.rows + n.rows - 1) / n.rows, most = (int64_t)sms * n.blocks;
  const int grid = (int)std::min<int64_t>(groups, most);
  p.depth = ring_depth((T + (int64_t)grid * n.rows - 1) / ((int64_t)grid * n.rows), n.blocks, n.rows * row_bytes, n.v, true);
  const int64_t smem = p.depth * n.rows * row_bytes;
  void (*k)(const SandwichParams) = nullptr;
  auto pick = [&](auto type, auto ring) {
    constexpr bool F = decltype(type)::value, R = decltype(ring)::value;
    k = n.v == 1 ? sandwich_kernel<1, F, R, 512> : n.v == 2 ? (n.threads <= 320 ? sandwich_kernel<2, F, R, 320> : sandwich_kernel<2, F, R, 512>)
        : n.v == 4 ? sandwich_kernel<4, F, R, 512> : sandwich_kernel<8, F, false, 512>;
  };
  if (f32 && p.depth) pick(std::true_type{}, std::true_type{});
  else if (f32) pick(std::true_type{}, std::false_type{});
  else if (p.depth) pick(std::false_type{}, std::true_type{});
  else pick(std::false_type{}, std::false_type{});
  if (allow_smem(k, smem) != cudaSuccess) return MOK_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_begin("sandwich_norm", s);
  k<<<grid, dim3(n.threads, n.rows), smem, s>>>(p);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(1);
  return MOK_OK;
}

size_t mok_sandwich_norm_workspace_size(int64_t T, int d) {
  using namespace mok;
  if (!sandwich_sizes_ok(T, d)) return 0;
  return 256 + 2 * sizeof(float) * (size_t)sandwich_bwd_grid(num_sms(), T, d) * d;
}

int mok_sandwich_norm_backward(const mok_sandwich* a, int64_t T, int d, const void* dy, const void* dres, const void* x,
                               const void* x_scales, const void* h, const void* h_scales, void* dx, void* dresidual,
                               float* dpost_weight, float* dgate, float* dtoken_gate, float* dweight, void* ws,
                               size_t ws_bytes, mok_stream_t stream) {
  using namespace mok;
  if (!a) return MOK_ERR_INVALID_ARG;
  const bool packed = x_scales != nullptr;
  if (!sandwich_sizes_ok(T, d) || (packed && d % 128)) return MOK_ERR_UNSUPPORTED;
  if (!(a->eps > 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->res_scale)) return MOK_ERR_INVALID_ARG;
  if (!elem_ok(a->res_type) || !elem_ok(a->post_type) || !elem_ok(a->gate_type) || !elem_ok(a->weight_type))
    return MOK_ERR_INVALID_ARG;
  if (!ws || !a->post_weight || !dpost_weight || (a->gate != nullptr) != (dgate != nullptr) ||
      (a->weight != nullptr) != (dweight != nullptr))
    return MOK_ERR_INVALID_ARG;
  if (T > 0 && (!x || !dx || !dresidual || (a->weight != nullptr) != (dy != nullptr) || (dy && !h) || (!dy && !dres) ||
                (dy && (h_scales != nullptr) != packed) || (a->token_gate != nullptr) != (dtoken_gate != nullptr)))
    return MOK_ERR_INVALID_ARG;
  for (const void* q : {dy, dres, x, x_scales, h, h_scales, a->post_weight, a->gate, a->weight, (const void*)dx,
                        (const void*)dresidual, (const void*)dpost_weight, (const void*)dgate, (const void*)dweight,
                        (const void*)ws})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  if (!is4(a->token_gate) || !is4(dtoken_gate)) return MOK_ERR_UNSUPPORTED;
  const int sms = num_sms(), grid = sandwich_bwd_grid(sms, T, d);
  if (ws_bytes < 256 + 2 * sizeof(float) * (size_t)grid * d) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    cudaError_t e = cudaSuccess;
    for (float* g : {dpost_weight, dgate, dweight})
      if (g && e == cudaSuccess) e = cudaMemsetAsync(g, 0, sizeof(float) * d, st);
    return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
  }
  const bool f32 = a->res_type == MOK_T_F32;
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  SandwichBwdParams p{dy, h, static_cast<const uint8_t*>(h_scales), x, static_cast<const uint8_t*>(x_scales), dres,
                      a->post_weight, a->gate, a->token_gate, a->weight, dx, dresidual, dtoken_gate, partial,
                      static_cast<int*>(ws), T, d, a->eps, 1.0f / (float)d, a->res_scale, a->post_type == MOK_T_F32,
                      a->gate_type == MOK_T_F32, a->weight_type == MOK_T_F32, 0, g_lost_rows.fetched(T), g_lost_rows.budget};
  g_lost_rows = LostRows();
  const SandwichShape n = sandwich_bwd_shape(d);
  const int64_t nvec = d / 8, res = f32 ? 32 : 16;
  const int64_t scales = packed ? (nvec / 4 + 31) / 16 * 16 : 0;  // as the kernel lays a place out
  const int64_t row_bytes = nvec * ((dy ? 16 : 0) + (dres ? res : 0) + (dy ? (packed ? 8 : res) : 0) + (packed ? 8 : 16)) + scales * (dy ? 2 : 1);
  p.depth = ring_depth((T + grid - 1) / grid, n.blocks, row_bytes, n.v, f32 && !packed);
  const int64_t smem = p.depth * row_bytes;
  void (*k)(const SandwichBwdParams) = nullptr;
  auto pick = [&](auto type, auto codes, auto ring) {
    constexpr bool F = decltype(type)::value, C = decltype(codes)::value, R = decltype(ring)::value;
    k = n.v == 1 ? sandwich_bwd_kernel<1, F, C, R, kNarrowThreads> : n.v == 2 ? sandwich_bwd_kernel<2, F, C, R, kWideThreads>
        : n.v == 3 ? sandwich_bwd_kernel<3, F, C, R, kThreeThreads> : n.v == 4 ? sandwich_bwd_kernel<4, F, C, R, kWideThreads>
        : sandwich_bwd_kernel<8, F, C, false, kWideThreads>;
  };
  auto pick2 = [&](auto type, auto codes) {
    if (p.depth) pick(type, codes, std::true_type{});
    else pick(type, codes, std::false_type{});
  };
  if (f32 && packed) pick2(std::true_type{}, std::true_type{});
  else if (f32) pick2(std::true_type{}, std::false_type{});
  else if (packed) pick2(std::false_type{}, std::true_type{});
  else pick2(std::false_type{}, std::false_type{});
  if (allow_smem(k, smem) != cudaSuccess) return MOK_ERR_CUDA;
  prof_begin("sandwich_bwd", st);
  k<<<grid, n.threads + (p.depth ? 32 : 0), smem, st>>>(p);
  prof_end(st);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  const SandwichSumParams sp{partial, grid, d, a->post_weight, a->gate, dpost_weight, dgate, dweight, p.post_f32, p.gate_f32};
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((d + 31) / 32), dweight ? 2u : 1u);
  c.blockDim = dim3(32 * kSumWarps);
  c.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  prof_begin("sandwich_sum", st);
  const cudaError_t e = cudaLaunchKernelEx(&c, sandwich_sum_kernel, sp);
  prof_end(st);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(2);
  return MOK_OK;
}

}  // extern "C"

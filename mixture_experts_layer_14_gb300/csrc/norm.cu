// RMS norm with the residual's addition and an optional MXFP8 output, and its backward pass.
//
//   h = x + residual,  rho = 1 / sqrt(mean(h^2) + eps),  v = h rho weight
//   ds = rho (g - xhat mean(g xhat)) + dres,  g = dy weight,  xhat = s rho;  dweight = sum dy xhat
//
// Both passes are bound by HBM, and a row's reduction is a barrier that nothing of the row passes.
// So blocks stay for many rows, and every thread keeps the next rows' vectors coming into a ring
// in shared memory by asynchronous copies while it works on the present row in registers: thread
// i of a row holds the 8-element vectors i, i + n, ... (contiguous 512 bytes per warp; four
// neighbouring lanes hold a 32-element MXFP8 block) and copies exactly what it reads back itself,
// so that waiting for its own copies is enough.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mok_ring.cuh"

namespace mok {

constexpr int kNormMaxD = 32768;

struct NormParams {
  const void* x;         // bf16
  const void* residual;  // or NULL
  const void* weight;
  void* y;               // bf16, or NULL
  void* residual_out;
  void* codes;           // or NULL
  uint8_t* scales;
  int64_t T, rows;       // rows: T, or T padded to 128 (scale atoms)
  int d;
  float eps;
  int weight_f32, atoms, depth;  // depth: rows in the ring
};

// Sum of two values over the row's threads, the same in all of them.  A row is a block's
// (blockDim.y == 1) or, up to 256 elements, a warp's.  `turn` alternates between calls: two
// buffers need one barrier per call.  The forward pass has one sum and passes 0 beside it: with the
// second one taken out it takes 165 us instead of 162 with scales in rows and 163 instead of 167 with
// scale atoms (T = 16384, d = 7168).
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (&smem)[2][32], int turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return make_float2(a, b);
  if (lane == 0) smem[turn][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 t = lane < warps ? smem[turn][lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(t.x), warp_sum(t.y));
}

// RES: 0 no residual, 1 bf16, 2 fp32.  V vectors per thread, MT threads at most.  At T = 16384,
// d = 7168 with a bf16 residual and MXFP8 output (1.06 GB) 156 us, 6.8 TB/s; a block per row without
// a ring 229 us.
template <int V, int RES, int MT>
__global__ void __launch_bounds__(MT) rms_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 smem[2][32];
  const int nvec = p.d >> 3;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kPlanes = 1 + (RES == 0 ? 0 : RES);  // of 16 bytes per vector
  const uint32_t place = kPlanes * 16 * nvec;        // bytes of a row
  const uint32_t base = smem_u32(ring) + threadIdx.y * p.depth * place;
  constexpr bool kHold = V < 4;  // the weight in registers; else read where it is used, from L1 or L2
  bool in[V];
  Vec8 w[kHold ? V : 1];
  auto fetch = [&](int64_t row, int slot) {
    if (row < p.T) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const uint32_t at = base + slot * place;
        copy8<false>(at, p.x, row * nvec, v, nvec);
        if constexpr (RES != 0) copy8<RES == 2>(at + 16 * nvec, p.residual, row * nvec, v, nvec);
      }
    }
    copies_end();
  };
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = threadIdx.x + i * blockDim.x < nvec;
  for (int k = 0; k < p.depth; ++k) fetch(t + k * step, k);
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) w[i] = load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, in[i]);
  int slot = 0;
  for (int turn = 0; t < p.T; t += step, turn ^= 1) {
    Vec8 h[V];
    float ss = 0.0f;
    if (p.depth == 2) copies_wait<1>();
    else copies_wait<0>();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const uint32_t at = base + slot * place;
      h[i] = value8<false>(in[i] ? ring8<false>(at, v, nvec) : zero8<false>());
      if constexpr (RES != 0) {
        const Vec8 a = value8<RES == 2>(in[i] ? ring8<RES == 2>(at + 16 * nvec, v, nvec) : zero8<RES == 2>());
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] += a.v[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[i].v[j], h[i].v[j], ss);
    }
    fetch(t + p.depth * step, slot);  // this thread's reads of the place come before in program order
    slot = slot + 1 == p.depth ? 0 : slot + 1;
    ss = row_sum(ss, 0.0f, smem, turn).x;
    const float rho = 1.0f / sqrtf(ss / (float)p.d + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (RES != 0 && in[i]) store8<RES == 2>(p.residual_out, t * nvec + v, h[i]);
      const Vec8 g = kHold ? w[kHold ? i : 0] : load_weight(p.weight, p.weight_f32, v, in[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i].v[j] = h[i].v[j] * rho * g.v[j];
      if (p.y && in[i]) store8<false>(p.y, t * nvec + v, h[i]);
      if (p.codes) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(h[i].v[j]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int s = mx_exponent(amax);
        const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
        if (in[i]) {
          uint2 q;
          q.x = e4m3x2(h[i].v[0] * inv, h[i].v[1] * inv) | (uint32_t)e4m3x2(h[i].v[2] * inv, h[i].v[3] * inv) << 16;
          q.y = e4m3x2(h[i].v[4] * inv, h[i].v[5] * inv) | (uint32_t)e4m3x2(h[i].v[6] * inv, h[i].v[7] * inv) << 16;
          static_cast<uint2*>(p.codes)[t * nvec + v] = q;
          if ((v & 3) == 0) {
            const int b = v >> 2;
            const int64_t at = p.atoms ? sf_atom_word(t >> 7, b >> 2, p.d / 128, (int)(t & 127)) + (b & 3)
                                       : t * (nvec >> 2) + b;
            p.scales[at] = (uint8_t)(s + 127);
          }
        }
      }
    }
  }
  for (; t < p.rows; t += step)  // padding rows of the scale atoms
    for (int kb = threadIdx.x; kb < p.d / 128; kb += blockDim.x)
      *reinterpret_cast<uint32_t*>(p.scales + sf_atom_word(t >> 7, kb, p.d / 128, (int)(t & 127))) = 0;
}

struct NormBwdParams {
  const void* dy;    // bf16
  const void* s;
  const void* dres;  // or NULL
  const void* weight;
  void* dx;          // bf16, or NULL
  void* dresidual;   // or NULL
  float* partial;    // [grid][d]
  int64_t T;
  int d;
  float eps;
  float inv_d;
  int weight_f32, depth, ring_res;  // ring_res: dres goes through the ring too
};

// DRES: a gradient arrives through the residual.  A block takes one row per turn and keeps its share
// of dweight in registers until its last row.  The two sums of a row and what needs them are a turn
// apart: in the turn that finishes row n the sums of row n + 1 begin, and the shuffles of both
// reductions run side by side, so that a turn has one barrier and little waiting.  Rows are read
// from the ring in both turns, which leaves registers for 1024 threads; without RING (rows of which
// two do not fit) from memory, the second time from L2.  At T = 8192, d = 7168 with bf16 rows and a
// gradient through the residual (470 MB) 78 us, 6.0 TB/s, of 69 at the copy rate: 54 rows per
// block, of which the first waits for memory and the last for its stores, and 250 instructions per
// warp and row (68% of the issue slots).  A block per row 128 us; two places in the ring instead of
// three 122 us; scalar arithmetic 88 us.
template <int V, bool F32, bool DRES, bool RING, int MT>
__global__ void __launch_bounds__(MT) rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
  __shared__ float2 smem[2][32];
  const int nvec = p.d >> 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t row_step = (int64_t)gridDim.x * nvec;  // vectors from a turn's row to the next one's
  const int64_t end = p.T * nvec;
  constexpr bool kHold = V < 4;  // the weight in registers; else read where it is used, from L1 or L2
  bool in[V];
  Pairs dw[V], w[kHold ? V : 1];
  auto weight = [&](int i) {
    return kHold ? w[kHold ? i : 0] : pairs(load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, true));
  };
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kPlanes = F32 ? 2 : 1;  // of 16 bytes per vector: one for dy, then s, then dres
  const uint32_t s_at = 16 * nvec, r_at = s_at + 16 * kPlanes * nvec;
  const uint32_t place = DRES && p.ring_res ? r_at + 16 * kPlanes * nvec : r_at;
  const uint32_t base = smem_u32(ring);
  const bool deep = p.depth == 3;
  // the row that begins at vector `row` into the place at `at`
  auto fetch = [&](int64_t row, uint32_t at) {
    if constexpr (!RING) return;
    if (row < end) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        copy8<false>(at, p.dy, row, v, nvec);
        copy8<F32>(at + s_at, p.s, row, v, nvec);
        if (DRES && p.ring_res) copy8<F32>(at + r_at, p.dres, row, v, nvec);
      }
    }
    copies_end();
  };
  auto landed = [&]() {  // all but the newest row (with two places: all)
    if constexpr (RING) {
      if (deep) copies_wait<1>();
      else copies_wait<0>();
    }
  };
  auto read = [&](int64_t row, uint32_t at, int v, Pairs* s, Pairs* dy) {
    if constexpr (RING) {
      *s = pairs(value8<F32>(ring8<F32>(at + s_at, v, nvec)));
      *dy = pairs(value8<false>(ring8<false>(at, v, nvec)));
    } else {
      *s = pairs(load8<F32>(p.s, row + v));
      *dy = pairs(load8<false>(p.dy, row + v));
    }
  };
  // this thread's share of sum s^2 and sum g s of a row
  auto sums_of = [&](int64_t row, uint32_t at) {
    float2 ss = both(0.0f), dot = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        Pairs a, b;
        const Pairs g = weight(i);
        read(row, at, threadIdx.x + i * blockDim.x, &a, &b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ss = __ffma2_rn(a.p[j], a.p[j], ss);
          dot = __ffma2_rn(a.p[j], __fmul2_rn(b.p[j], g.p[j]), dot);
        }
      }
    }
    return make_float2(ss.x + ss.y, dot.x + dot.y);
  };
  int64_t row = (int64_t)blockIdx.x * nvec;  // gridDim.x <= T
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = threadIdx.x + i * blockDim.x < nvec;
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i].p[j] = both(0.0f);
  }
  uint32_t at = base, last = base + (p.depth - 1) * place;  // this row's place; the one before it
  fetch(row, base);
  if (deep) fetch(row + row_step, base + place);
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) w[i] = pairs(load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, in[i]));
  landed();
  {
    const float2 own = sums_of(row, base);
    const float a = warp_sum(own.x), b = warp_sum(own.y);
    if (lane == 0) smem[0][warp] = make_float2(a, b);
  }
  __syncthreads();
  for (int turn = 0; row < end; row += row_step, turn ^= 1) {
    fetch(row + (deep ? 2 : 1) * row_step, last);
    landed();
    const uint32_t next = at + place == base + p.depth * place ? base : at + place;
    Raw8<F32> res = zero8<F32>();  // dres, if not in the ring: early where registers allow
    if (DRES && V == 1 && in[0] && !(RING && p.ring_res)) res = raw8<F32>(p.dres, row + threadIdx.x);
    float2 own = both(0.0f), sums = lane < warps ? smem[turn][lane] : both(0.0f);
    if (row + row_step < end) own = sums_of(row + row_step, next);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sums = __fadd2_rn(sums, make_float2(__shfl_xor_sync(0xffffffffu, sums.x, o), __shfl_xor_sync(0xffffffffu, sums.y, o)));
      own = __fadd2_rn(own, make_float2(__shfl_xor_sync(0xffffffffu, own.x, o), __shfl_xor_sync(0xffffffffu, own.y, o)));
    }
    if (lane == 0) smem[turn ^ 1][warp] = own;
    const float rho = rsqrtf(fmaf(sums.x, p.inv_d, p.eps));
    const float2 rho2 = both(rho), c = both(-sums.y * p.inv_d * rho * rho);  // - mean(g xhat) rho
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (in[i]) {
        Pairs a, b;
        read(row, at, v, &a, &b);
        Vec8 ds;
        Pairs r;
        const Pairs gw = weight(i);
        if constexpr (DRES)
          r = pairs(value8<F32>(RING && p.ring_res ? ring8<F32>(at + r_at, v, nvec)
                                   : V == 1                ? res
                                                           : raw8<F32>(p.dres, row + v)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dw[i].p[j] = __ffma2_rn(b.p[j], __fmul2_rn(a.p[j], rho2), dw[i].p[j]);
          const float2 g = __ffma2_rn(a.p[j], c, __fmul2_rn(b.p[j], gw.p[j]));
          const float2 q = DRES ? __ffma2_rn(g, rho2, r.p[j]) : __fmul2_rn(g, rho2);
          ds.v[2 * j] = q.x;
          ds.v[2 * j + 1] = q.y;
        }
        if (p.dx) store8<false>(p.dx, row + v, ds);
        if (p.dresidual) store8<F32>(p.dresidual, row + v, ds);
      }
    }
    last = at;
    at = next;
    __syncthreads();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (in[i]) {
      Vec8 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o.v[2 * j] = dw[i].p[j].x;
        o.v[2 * j + 1] = dw[i].p[j].y;
      }
      store8<true>(p.partial + (int64_t)blockIdx.x * p.d, v, o);
    }
  }
}

// dweight = sum over the n partial rows, in a fixed order.  A block takes 32 columns: lane l of warp
// w adds the rows 4 w + l / 8, + 64, ... of the columns 4 (l % 8) .., then the four rows of a warp
// and the warps are joined.
constexpr int kDwWarps = 16;
__global__ void __launch_bounds__(32 * kDwWarps) rms_norm_dweight_kernel(const float* partial, int n, int d,
                                                                         float* __restrict__ dweight) {
  __shared__ float4 smem[kDwWarps][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 8 + (lane & 7);  // group of four columns
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the first pass still runs
  if (4 * c < d) {
#pragma unroll 8
    for (int r = 4 * warp + (lane >> 3); r < n; r += 4 * kDwWarps) {
      const float4 v = reinterpret_cast<const float4*>(partial + (int64_t)r * d)[c];
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
  if (warp == 0 && lane < 8 && 4 * c < d) {
    for (int w = 1; w < kDwWarps; ++w) {
      const float4 v = smem[w][lane];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    reinterpret_cast<float4*>(dweight)[c] = a;
  }
}

static bool norm_sizes_ok(int64_t T, int d) {
  return T >= 0 && T <= 0x7fffffffLL / 8 && d > 0 && d <= kNormMaxD && d % 8 == 0;
}
// Vectors per thread (1, 2 or 4), threads of a row, rows of a block, blocks per SM and the ring's
// depth.  One vector per thread up to 1024 threads: at T = 16384, d = 7168 with MXFP8 output 160 us
// against 168 us with two (448 threads); blocks fill an SM's registers with 1024 threads.  More
// rows under way than the copies' latency needs cost bandwidth: forward, 2^26 elements, with one /
// two / three rows per block 84 / 93 / 96 us at d = 4096 (two blocks per SM, bf16; 79 at the copy
// rate) and 90 / 85 / 93 at d = 7168 (one).
struct NormShape {
  int v, threads, rows, blocks, depth;
};
constexpr int kSmemPerSm = 227 * 1024;             // for the blocks of an SM together
constexpr int kSmemOwn = 2048;                     // of a block: reserved and static
constexpr int kRingBytes = kSmemPerSm - kSmemOwn;  // most dynamic bytes of a block
constexpr int kPlainSmem = 40 * 1024;              // dynamic bytes that need no attribute
static NormShape norm_shape(int sms, int64_t T, int d, int row_bytes, bool warp_rows) {
  NormShape n;
  const int nvec = d / 8;
  n.v = nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : 4;
  n.threads = ((nvec + n.v - 1) / n.v + 31) / 32 * 32;
  n.rows = warp_rows && n.threads == 32 ? 8 : 1;
  n.blocks = std::max(1, std::min(1024 / (n.threads * n.rows), 8));
  n.depth = n.blocks > 1 || T <= (int64_t)sms * n.blocks * n.rows || 2 * row_bytes > kRingBytes ? 1 : 2;
  return n;
}
// Backward: two rows at least, three where they fit, or depth 0 where not even two do.  dres goes
// through the ring in bf16 where three rows with it fit; in fp32 it comes straight to registers
// (2^26 elements at d = 7168: 165 us against 198 through the ring, 158 at the copy rate).
static NormShape norm_bwd_shape(int sms, int64_t T, int d, bool f32, bool dres, int* row_bytes, int* ring_res) {
  const int plane = 2 * d, planes = f32 ? 2 : 1;
  NormShape n = norm_shape(sms, T, d, plane, false);
  const int room = kSmemPerSm / n.blocks - kSmemOwn;
  *ring_res = dres && !f32 && 9 * plane <= room;
  *row_bytes = plane * (1 + planes * (*ring_res ? 2 : 1));
  n.depth = std::min(3, room / *row_bytes);
  const int64_t turns = (T + (int64_t)sms * n.blocks - 1) / ((int64_t)sms * n.blocks);
  n.depth = n.depth < 2 ? 0 : (int)std::min<int64_t>(n.depth, turns + 1);
  return n;
}
// The same for every type, so that one workspace size serves them all.
static int norm_bwd_grid(int sms, int64_t T, int d) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(T, (int64_t)sms * norm_shape(sms, T, d, 2 * d, false).blocks));
}
static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace mok

extern "C" {

int mok_rms_norm(int64_t T, int d, float eps, const void* x, const void* residual, int res_type,
                 const void* weight, int weight_type, void* y, void* residual_out, void* codes,
                 void* scales, int scale_layout, mok_stream_t stream) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return MOK_ERR_UNSUPPORTED;
  if (codes && d % 128) return MOK_ERR_UNSUPPORTED;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MOK_ERR_INVALID_ARG;
  if ((res_type != MOK_T_BF16 && res_type != MOK_T_F32) || (weight_type != MOK_T_BF16 && weight_type != MOK_T_F32) ||
      (scale_layout != MOK_SCALES_ROWS && scale_layout != MOK_SCALES_ATOMS))
    return MOK_ERR_INVALID_ARG;
  if (T > 0 && (!x || !weight || (!y && !codes) || (codes && !scales))) return MOK_ERR_INVALID_ARG;
  if (T > 0 && (residual != nullptr) != (residual_out != nullptr)) return MOK_ERR_INVALID_ARG;
  for (const void* q : {x, residual, weight, (const void*)y, (const void*)residual_out, (const void*)codes, (const void*)scales})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  set_last_launches(0);
  if (T == 0) return MOK_OK;
  NormParams p{x, residual, weight, y, residual_out, codes, static_cast<uint8_t*>(scales), T, T, d, eps,
               weight_type == MOK_T_F32, scale_layout == MOK_SCALES_ATOMS, 1};
  if (codes && p.atoms) p.rows = (T + 127) / 128 * 128;
  const int row_bytes = 2 * d * (1 + (!residual ? 0 : res_type == MOK_T_F32 ? 2 : 1));
  const int sms = num_sms();
  const NormShape n = norm_shape(sms, T, d, row_bytes, true);
  p.depth = n.depth;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = (int)std::min<int64_t>((p.rows + n.rows - 1) / n.rows, (int64_t)sms * n.blocks);
  void (*k)(const NormParams) = nullptr;
  auto pick = [&](auto res) {
    constexpr int R = decltype(res)::value;
    k = n.v == 1 ? (n.threads * n.rows <= 256 ? rms_norm_kernel<1, R, 256> : rms_norm_kernel<1, R, 1024>)
        : n.v == 2 ? rms_norm_kernel<2, R, 1024> : rms_norm_kernel<4, R, 1024>;
  };
  if (!residual) pick(std::integral_constant<int, 0>{});
  else if (res_type == MOK_T_BF16) pick(std::integral_constant<int, 1>{});
  else pick(std::integral_constant<int, 2>{});
  const int smem = n.depth * n.rows * row_bytes;
  if (smem > kPlainSmem && cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    return MOK_ERR_CUDA;
  prof_begin("rms_norm", s);
  k<<<grid, dim3(n.threads, n.rows), smem, s>>>(p);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(1);
  return MOK_OK;
}

size_t mok_rms_norm_workspace_size(int64_t T, int d) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return 0;
  return 256 + sizeof(float) * (size_t)norm_bwd_grid(num_sms(), T, d) * d;
}

int mok_rms_norm_backward(int64_t T, int d, float eps, const void* dy, const void* s, int res_type,
                          const void* weight, int weight_type, const void* dres, void* dx,
                          void* dresidual, float* dweight, void* ws, size_t ws_bytes,
                          mok_stream_t stream) {
  using namespace mok;
  if (!norm_sizes_ok(T, d)) return MOK_ERR_UNSUPPORTED;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MOK_ERR_INVALID_ARG;
  if ((res_type != MOK_T_BF16 && res_type != MOK_T_F32) || (weight_type != MOK_T_BF16 && weight_type != MOK_T_F32))
    return MOK_ERR_INVALID_ARG;
  if (!dweight || !ws || (T > 0 && (!dy || !s || !weight || (!dx && !dresidual)))) return MOK_ERR_INVALID_ARG;
  for (const void* q : {dy, s, weight, dres, (const void*)dx, (const void*)dresidual, (const void*)dweight, (const void*)ws})
    if (!is16(q)) return MOK_ERR_UNSUPPORTED;
  const int sms = num_sms(), grid = norm_bwd_grid(sms, T, d);
  if (ws_bytes < 256 + sizeof(float) * (size_t)grid * d) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return cudaMemsetAsync(dweight, 0, sizeof(float) * d, st) == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  NormBwdParams p{dy, s, dres, weight, dx, dresidual, partial, T, d, eps, 1.0f / (float)d, weight_type == MOK_T_F32, 0, 0};
  int row_bytes;
  const bool f32 = res_type == MOK_T_F32;
  const NormShape n = norm_bwd_shape(sms, T, d, f32, dres != nullptr, &row_bytes, &p.ring_res);
  p.depth = n.depth;
  void (*k)(const NormBwdParams) = nullptr;
  auto pick = [&](auto type, auto has) {
    constexpr bool F = decltype(type)::value, R = decltype(has)::value;
    k = n.v == 1 ? (n.threads <= 256 ? rms_norm_bwd_kernel<1, F, R, true, 256> : rms_norm_bwd_kernel<1, F, R, true, 1024>)
        : n.v == 2 ? rms_norm_bwd_kernel<2, F, R, true, 1024>
        : n.depth ? rms_norm_bwd_kernel<4, F, R, true, 1024> : rms_norm_bwd_kernel<4, F, R, false, 1024>;
  };
  if (f32 && dres) pick(std::true_type{}, std::true_type{});
  else if (f32) pick(std::true_type{}, std::false_type{});
  else if (dres) pick(std::false_type{}, std::true_type{});
  else pick(std::false_type{}, std::false_type{});
  const int smem = n.depth * row_bytes;
  if (smem > kPlainSmem && cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess)
    return MOK_ERR_CUDA;
  prof_begin("rms_norm_bwd", st);
  k<<<grid, n.threads, smem, st>>>(p);
  prof_end(st);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  prof_begin("rms_norm_dweight", st);
  const cudaError_t e = launch_after(rms_norm_dweight_kernel, (d + 31) / 32, 32 * kDwWarps, st, (const float*)partial,
                                     grid, d, dweight);
  prof_end(st);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(2);
  return MOK_OK;
}

}  // extern "C"

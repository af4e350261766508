// The norm after a branch with its gate, the scaled residual and the next norm in one pass, and the
// backward pass of it.
//
//   n = x rho1 post gate token_gate,  h = res_scale r + n,  v = h rho2 weight,
//   rho = 1 / sqrt(mean(row^2) + eps);
//   ds = rho2 (g - hhat mean(g hhat)) + dres,  g = dv weight,  dr = res_scale ds,
//   dx = rho1 tg (ds W - xhat mean(ds W xhat)),  W = post gate,  q = sum ds W xhat = dtoken_gate,
//   A = sum over rows of tg ds xhat:  dpost = A gate,  dgate = A post,  dweight = sum dv hhat.
//
// Both are bound by HBM.  A block stays for many rows, which come through a ring in shared memory by
// asynchronous copies two rows ahead, and holds the present one in registers.  Each row needs two
// sums of which the second follows from the first; the first ones are taken a row ahead, so that
// both go through one exchange and one barrier per row.
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
};

// Sums of N values over the row's threads, the same in all of them: a row is a block's or a warp's
// (32 threads in x).  `turn` alternates between calls: two buffers need one barrier per call.
template <int N, int W>
__device__ __forceinline__ void row_sums(float (&a)[N], float (&smem)[2][W][N], int turn) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
  if (warps == 1) return;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) smem[turn][threadIdx.x >> 5][i] = a[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = lane < warps ? smem[turn][lane][i] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
}

// MXFP8 form of eight elements whose block of 32 lies in four neighbouring lanes.
__device__ __forceinline__ void quantise8(const Vec8& a, bool in, void* codes, int64_t at, uint8_t* scale, bool first) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(a.v[j]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int s = mx_exponent(amax);
  const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
  if (!in) return;
  uint2 q;
  q.x = e4m3x2(a.v[0] * inv, a.v[1] * inv) | (uint32_t)e4m3x2(a.v[2] * inv, a.v[3] * inv) << 16;
  q.y = e4m3x2(a.v[4] * inv, a.v[5] * inv) | (uint32_t)e4m3x2(a.v[6] * inv, a.v[7] * inv) << 16;
  static_cast<uint2*>(codes)[at] = q;
  if (first) *scale = (uint8_t)(s + 127);
}

// V vectors of eight per thread, MT threads at most.
template <int V, bool F32, bool RING, int MT>
__global__ void __launch_bounds__(MT) sandwich_kernel(const __grid_constant__ SandwichParams p) {
  __shared__ float smem[2][32][2];
  extern __shared__ __align__(16) uint8_t ring[];
  const int nvec = p.d >> 3;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  constexpr int kPlanes = 1 + (F32 ? 2 : 1);  // of 16 bytes per vector
  const uint32_t place = kPlanes * 16 * nvec;
  const uint32_t base = smem_u32(ring) + threadIdx.y * p.depth * place;
  constexpr bool kHold = V <= 2;  // the weights in registers; else read where they are used
  bool in[V];
  Vec8 W[kHold ? V : 1], w2[kHold ? V : 1];
  auto inner = [&](int v, bool ok) {  // post gate
    Vec8 a = load_weight(p.post, p.post_f32, v, ok);
    if (p.gate) {
      const Vec8 g = load_weight(p.gate, p.gate_f32, v, ok);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] *= g.v[j];
    }
    return a;
  };
  auto fetch = [&](int64_t row, uint32_t at) {
    if constexpr (!RING) return;
    if (row < p.T) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        copy8<false>(at, p.x, row * nvec, v, nvec);
        copy8<F32>(at + 16 * nvec, p.residual, row * nvec, v, nvec);
      }
    }
    copies_end();
  };
  auto read_x = [&](int64_t row, uint32_t at, int v) {
    if constexpr (RING) return value8<false>(ring8<false>(at, v, nvec));
    else return load8<false>(p.x, row * nvec + v);
  };
  auto read_r = [&](int64_t row, uint32_t at, int v) {
    if constexpr (RING) return value8<F32>(ring8<F32>(at + 16 * nvec, v, nvec));
    else return load8<F32>(p.residual, row * nvec + v);
  };
  auto square_of = [&](int64_t row, uint32_t at) {  // this thread's share of sum x^2
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        const Vec8 a = read_x(row, at, threadIdx.x + i * blockDim.x);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a.v[j], a.v[j], ss);
      }
    }
    return ss;
  };
#pragma unroll
  for (int i = 0; i < V; ++i) in[i] = threadIdx.x + i * blockDim.x < nvec;
  uint32_t at = base, last = base + (p.depth - 1) * place;  // this row's place, and the one before it
  fetch(t, base);
  fetch(t + step, base + place);
  float gate = 1.0f, next_gate = 1.0f;
  if (p.token_gate && t < p.T) gate = p.token_gate[t];
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) {
    W[i] = inner(threadIdx.x + i * blockDim.x, in[i]);
    w2[i] = p.weight ? load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, in[i]) : Vec8{};
  }
  if constexpr (RING) copies_wait<1>();
  float sums[2] = {0.0f, t < p.T ? square_of(t, base) : 0.0f};
  row_sums(sums, smem, 1);
  for (int turn = 0; t < p.T; t += step, turn ^= 1) {
    fetch(t + 2 * step, last);
    if constexpr (RING) copies_wait<1>();
    const uint32_t next = at + place == base + p.depth * place ? base : at + place;
    if (p.token_gate && t + step < p.T) next_gate = p.token_gate[t + step];
    const float rho1 = rsqrtf(fmaf(sums[1], p.inv_d, p.eps)) * gate;
    Vec8 h[V];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      Vec8 x{};
      h[i] = Vec8{};
      if (in[i]) {
        x = read_x(t, at, v);
        h[i] = read_r(t, at, v);
        const Vec8 w = kHold ? W[kHold ? i : 0] : inner(v, true);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i].v[j] = fmaf(x.v[j] * rho1, w.v[j], p.res_scale * h[i].v[j]);
          ss = fmaf(h[i].v[j], h[i].v[j], ss);
        }
        store8<F32>(p.residual_out, t * nvec + v, h[i]);
      }
      if (p.x_codes) {
        const int64_t s = t * (nvec >> 2) + (v >> 2);
        quantise8(x, in[i], p.x_codes, t * nvec + v, p.x_scales + s, (v & 3) == 0);
        quantise8(h[i], in[i], p.h_codes, t * nvec + v, p.h_scales + s, (v & 3) == 0);
      }
    }
    sums[0] = ss;
    sums[1] = t + step < p.T ? square_of(t + step, next) : 0.0f;
    row_sums(sums, smem, turn);
    if (p.weight) {
      const float rho2 = rsqrtf(fmaf(sums[0], p.inv_d, p.eps));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const Vec8 w = kHold ? w2[kHold ? i : 0] : load_weight(p.weight, p.weight_f32, v, in[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i].v[j] = h[i].v[j] * rho2 * w.v[j];
        if (p.y && in[i]) store8<false>(p.y, t * nvec + v, h[i]);
        if (p.codes) {
          const int b = v >> 2;
          const int64_t s = p.atoms ? sf_atom_word(t >> 7, b >> 2, p.d / 128, (int)(t & 127)) + (b & 3) : t * (nvec >> 2) + b;
          quantise8(h[i], in[i], p.codes, t * nvec + v, p.scales + s, (v & 3) == 0);
        }
      }
    }
    gate = next_gate;
    last = at;
    at = next;
  }
  for (; t < p.rows; t += step)  // padding rows of the scale atoms
    for (int kb = threadIdx.x; kb < p.d / 128; kb += blockDim.x)
      *reinterpret_cast<uint32_t*>(p.scales + sf_atom_word(t >> 7, kb, p.d / 128, (int)(t & 127))) = 0;
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
  int64_t T;
  int d;
  float eps, inv_d, res_scale;
  int post_f32, gate_f32, weight_f32, depth;
};

// PACKED: x and h come as codes and scales.
template <int V, bool F32, bool PACKED, bool RING, int MT>
__global__ void __launch_bounds__(MT) sandwich_bwd_kernel(const __grid_constant__ SandwichBwdParams p) {
  __shared__ float smem[2][32][4];
  extern __shared__ __align__(16) uint8_t ring[];
  const int nvec = p.d >> 3;
  const int64_t row_step = (int64_t)gridDim.x * nvec;  // vectors from a turn's row to the next one's
  const int64_t end = p.T * nvec;
  constexpr bool kHold = V <= 2;
  const bool next_norm = p.dy != nullptr, has_res = p.dres != nullptr;
  // planes of a place: dy, dres, h, x; codes with a word of scales (the vector's is one of its four bytes)
  constexpr int kRes = F32 ? 32 : 16, kH = PACKED ? 12 : kRes, kX = PACKED ? 12 : 16;
  const uint32_t res_at = next_norm ? 16 * nvec : 0, h_at = res_at + (has_res ? kRes * nvec : 0);
  const uint32_t x_at = h_at + (next_norm ? kH * nvec : 0), place = (x_at + kX * nvec + 15) & ~15u;
  const uint32_t base = smem_u32(ring);
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
    return kHold ? w2[kHold ? i : 0] : pairs(load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, true));
  };
  auto inner_of = [&](int i) { return kHold ? W[kHold ? i : 0] : inner(threadIdx.x + i * blockDim.x, true); };
  auto copy_packed = [&](uint32_t at, const void* codes, const uint8_t* scales, int64_t row, int v) {
    if (v >= nvec) return;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at + 8 * v), "l"(static_cast<const uint2*>(codes) + row + v) : "memory");
    // a row has nvec / 4 scales; nvec is a multiple of 16, so the four around the vector's are a word
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 8 * nvec + 4 * v), "l"(scales + (row >> 2) + (v >> 4) * 4) : "memory");
  };
  auto fetch = [&](int64_t row, uint32_t at) {
    if constexpr (!RING) return;
    if (row < end) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (next_norm) copy8<false>(at, p.dy, row, v, nvec);
        if (has_res) copy8<F32>(at + res_at, p.dres, row, v, nvec);
        if constexpr (PACKED) {
          if (next_norm) copy_packed(at + h_at, p.h, p.h_scales, row, v);
          copy_packed(at + x_at, p.x, p.x_scales, row, v);
        } else {
          if (next_norm) copy8<F32>(at + h_at, p.h, row, v, nvec);
          copy8<false>(at + x_at, p.x, row, v, nvec);
        }
      }
    }
    copies_end();
  };
  auto unpacked = [&](uint32_t at, const void* codes, const uint8_t* scales, int64_t row, int v) {
    uint2 q;
    uint32_t s;
    if constexpr (RING) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(at + 8 * v));
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s) : "r"(at + 8 * nvec + 4 * v));
      s = (s >> (2 * (v & 12))) & 255u;
    } else {
      q = static_cast<const uint2*>(codes)[row + v];
      s = scales[(row + v) >> 2];
    }
    return dequantise8(q, mx_scale(s));
  };
  auto read_dy = [&](int64_t row, uint32_t at, int v) {
    if constexpr (RING) return pairs(value8<false>(ring8<false>(at, v, nvec)));
    else return pairs(load8<false>(p.dy, row + v));
  };
  auto read_res = [&](int64_t row, uint32_t at, int v) {
    if constexpr (RING) return pairs(value8<F32>(ring8<F32>(at + res_at, v, nvec)));
    else return pairs(load8<F32>(p.dres, row + v));
  };
  auto read_h = [&](int64_t row, uint32_t at, int v) {
    if constexpr (PACKED) return pairs(unpacked(at + h_at, p.h, p.h_scales, row, v));
    else if constexpr (RING) return pairs(value8<F32>(ring8<F32>(at + h_at, v, nvec)));
    else return pairs(load8<F32>(p.h, row + v));
  };
  auto read_x = [&](int64_t row, uint32_t at, int v) {
    if constexpr (PACKED) return pairs(unpacked(at + x_at, p.x, p.x_scales, row, v));
    else if constexpr (RING) return pairs(value8<false>(ring8<false>(at + x_at, v, nvec)));
    else return pairs(load8<false>(p.x, row + v));
  };
  // this thread's share of a row's sum h^2, sum dy weight h, sum x^2
  auto sums_of = [&](int64_t row, uint32_t at, float& hh, float& dot, float& xx) {
    float2 a = both(0.0f), b = both(0.0f), c = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (in[i]) {
        const int v = threadIdx.x + i * blockDim.x;
        const Pairs x = read_x(row, at, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __ffma2_rn(x.p[j], x.p[j], c);
        if (next_norm) {
          const Pairs h = read_h(row, at, v), dy = read_dy(row, at, v), w = weight_of(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a = __ffma2_rn(h.p[j], h.p[j], a);
            b = __ffma2_rn(h.p[j], __fmul2_rn(dy.p[j], w.p[j]), b);
          }
        }
      }
    }
    hh = a.x + a.y;
    dot = b.x + b.y;
    xx = c.x + c.y;
  };
  int64_t row = (int64_t)blockIdx.x * nvec;  // gridDim.x <= T
#pragma unroll
  for (int i = 0; i < V; ++i) {
    in[i] = threadIdx.x + i * blockDim.x < nvec;
#pragma unroll
    for (int j = 0; j < 4; ++j) A[i].p[j] = dw[i].p[j] = both(0.0f);
  }
  uint32_t at = base, last = base + (p.depth - 1) * place;  // this row's place; the one before it
  fetch(row, base);
  fetch(row + row_step, base + place);
#pragma unroll
  for (int i = 0; i < (kHold ? V : 0); ++i) {
    W[i] = inner(threadIdx.x + i * blockDim.x, in[i]);
    w2[i] = pairs(next_norm ? load_weight(p.weight, p.weight_f32, threadIdx.x + i * blockDim.x, in[i]) : Vec8{});
  }
  if constexpr (RING) copies_wait<1>();
  int64_t t = blockIdx.x;
  float gate = p.token_gate ? p.token_gate[t] : 1.0f, next_gate = 1.0f;
  float sums[4];  // h^2, dy weight h, x^2 of the next row; ds W x of this one
  sums_of(row, base, sums[0], sums[1], sums[2]);
  sums[3] = 0.0f;
  row_sums(sums, smem, 1);
  for (int turn = 0; row < end; row += row_step, t += gridDim.x, turn ^= 1) {
    fetch(row + 2 * row_step, last);
    if constexpr (RING) copies_wait<1>();
    const uint32_t next = at + place == base + p.depth * place ? base : at + place;
    if (p.token_gate && row + row_step < end) next_gate = p.token_gate[t + gridDim.x];
    const float rho1 = rsqrtf(fmaf(sums[2], p.inv_d, p.eps)), rho2 = rsqrtf(fmaf(sums[0], p.inv_d, p.eps));
    const float2 r2 = both(rho2), c2 = both(-sums[1] * p.inv_d * rho2 * rho2);  // - mean(g hhat) rho2
    const float2 rt = both(rho1 * gate), a2 = both(p.res_scale);
    Pairs ds[V];
    float2 q = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (in[i]) {
        if (has_res) ds[i] = read_res(row, at, v);
        else ds[i] = pairs(Vec8{});
        if (next_norm) {
          const Pairs h = read_h(row, at, v), dy = read_dy(row, at, v), w = weight_of(i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i].p[j] = __ffma2_rn(dy.p[j], __fmul2_rn(h.p[j], r2), dw[i].p[j]);
            const float2 g = __ffma2_rn(h.p[j], c2, __fmul2_rn(dy.p[j], w.p[j]));
            ds[i].p[j] = __ffma2_rn(g, r2, ds[i].p[j]);
          }
        }
        const Pairs x = read_x(row, at, v), w = inner_of(i);
        Vec8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 dx = __fmul2_rn(ds[i].p[j], x.p[j]);
          A[i].p[j] = __ffma2_rn(dx, rt, A[i].p[j]);
          q = __ffma2_rn(dx, w.p[j], q);
          const float2 r = __fmul2_rn(ds[i].p[j], a2);
          o.v[2 * j] = r.x;
          o.v[2 * j + 1] = r.y;
        }
        store8<F32>(p.dresidual, row + v, o);
      }
    }
    sums[0] = sums[1] = sums[2] = 0.0f;
    if (row + row_step < end) sums_of(row + row_step, next, sums[0], sums[1], sums[2]);
    sums[3] = q.x + q.y;
    row_sums(sums, smem, turn);
    const float2 c1 = both(-sums[3] * p.inv_d * rho1 * rho1);  // - mean(ds W xhat) rho1
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (in[i]) {
        const Pairs x = read_x(row, at, v), w = inner_of(i);
        Vec8 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 r = __fmul2_rn(__ffma2_rn(x.p[j], c1, __fmul2_rn(ds[i].p[j], w.p[j])), rt);
          o.v[2 * j] = r.x;
          o.v[2 * j + 1] = r.y;
        }
        store8<false>(p.dx, row + v, o);
      }
    }
    if (p.dtoken_gate && threadIdx.x == 0) p.dtoken_gate[t] = rho1 * sums[3];
    gate = next_gate;
    last = at;
    at = next;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float* mine = p.partial + (int64_t)blockIdx.x * p.d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (in[i]) {
      Vec8 a, b;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a.v[2 * j] = A[i].p[j].x;
        a.v[2 * j + 1] = A[i].p[j].y;
        b.v[2 * j] = dw[i].p[j].x;
        b.v[2 * j + 1] = dw[i].p[j].y;
      }
      store8<true>(mine, v, a);
      if (next_norm) store8<true>(mine + (int64_t)gridDim.x * p.d, v, b);
    }
  }
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
constexpr int kSmemOwn = 3072;          // of a block: reserved and static
constexpr int kPlainSmem = 40 * 1024;   // dynamic bytes that need no attribute
static SandwichShape sandwich_shape(int d, bool warp_rows, int per_sm) {
  SandwichShape n;
  const int nvec = d / 8;
  n.v = nvec <= per_sm ? 1 : nvec <= 2 * per_sm ? 2 : nvec <= 4 * per_sm ? 4 : 8;
  n.threads = ((nvec + n.v - 1) / n.v + 31) / 32 * 32;
  n.rows = warp_rows && n.threads == 32 ? 8 : 1;
  n.blocks = std::max(1, std::min(per_sm / (n.threads * n.rows), 8));
  return n;
}
constexpr int kThreadsPerSm = 512;  // 128 registers each
static int sandwich_bwd_grid(int sms, int64_t T, int d) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(T, (int64_t)sms * sandwich_shape(d, false, kThreadsPerSm).blocks));
}
// Places of the ring for the rows that a block has to take, at most three; 0 where they do not fit and
// for the widest rows (rows are then read from memory, the second time from L2).
static int ring_depth(int64_t turns, int blocks, int64_t bytes, int v) {
  if (v > 4) return 0;
  const int depth = (int)std::min<int64_t>(3, turns);
  return depth * bytes <= kSmemPerSm / blocks - kSmemOwn ? depth : 0;
}
template <class K>
static cudaError_t allow_smem(K k, int64_t smem) {
  if (smem <= kPlainSmem) return cudaSuccess;
  return cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm - kSmemOwn);
}

}  // namespace mok

extern "C" {

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
                   scale_layout == MOK_SCALES_ATOMS, 0};
  if (codes && p.atoms) p.rows = (T + 127) / 128 * 128;
  const int sms = num_sms();
  const SandwichShape n = sandwich_shape(d, true, kThreadsPerSm);
  const int64_t row_bytes = 2 * d * (f32 ? 3 : 2);
  const int64_t groups = (p.rows + n.rows - 1) / n.rows, most = (int64_t)sms * n.blocks;
  const int grid = (int)std::min<int64_t>(groups, most);
  p.depth = ring_depth((T + (int64_t)grid * n.rows - 1) / ((int64_t)grid * n.rows), n.blocks, n.rows * row_bytes, n.v);
  const int64_t smem = p.depth * n.rows * row_bytes;
  void (*k)(const SandwichParams) = nullptr;
  auto pick = [&](auto type, auto ring) {
    constexpr bool F = decltype(type)::value, R = decltype(ring)::value;
    k = n.v == 1 ? sandwich_kernel<1, F, R, 512> : n.v == 2 ? sandwich_kernel<2, F, R, 512>
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
                      a->post_weight, a->gate, a->token_gate, a->weight, dx, dresidual, dtoken_gate, partial, T, d, a->eps,
                      1.0f / (float)d, a->res_scale, a->post_type == MOK_T_F32, a->gate_type == MOK_T_F32,
                      a->weight_type == MOK_T_F32, 0};
  const SandwichShape n = sandwich_shape(d, false, kThreadsPerSm);
  const int64_t nvec = d / 8, res = f32 ? 32 : 16;
  const int64_t row_bytes = (nvec * ((dy ? 16 : 0) + (dres ? res : 0) + (dy ? (packed ? 12 : res) : 0) + (packed ? 12 : 16)) + 15) / 16 * 16;
  p.depth = ring_depth((T + grid - 1) / grid, n.blocks, row_bytes, n.v);
  const int64_t smem = p.depth * row_bytes;
  void (*k)(const SandwichBwdParams) = nullptr;
  auto pick = [&](auto type, auto codes, auto ring) {
    constexpr bool F = decltype(type)::value, C = decltype(codes)::value, R = decltype(ring)::value;
    k = n.v == 1 ? sandwich_bwd_kernel<1, F, C, R, 512> : n.v == 2 ? sandwich_bwd_kernel<2, F, C, R, 512>
        : n.v == 4 ? sandwich_bwd_kernel<4, F, C, R, 512> : sandwich_bwd_kernel<8, F, C, false, 512>;
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
  k<<<grid, n.threads, smem, st>>>(p);
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

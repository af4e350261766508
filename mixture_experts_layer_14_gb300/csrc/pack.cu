// Activations in 8 bits and back: E4M3 codes and one UE8M0 scale per 32 consecutive elements (the rule
// of mok_mx.cuh), from bf16 or fp32; and the activations that a layer saves for its backward pass,
// all of them in one launch.
//
// Bound by HBM.  A lane takes 16 bytes of the wide side at a time (8 bf16 or 4 fp32 elements, so that 4
// or 8 lanes hold a block), which keeps every access of a warp contiguous, and has several vectors
// under way.  65536 x 2048 elements: bf16 to codes 59 us, codes to fp32 101, both at the copy rate.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mok_ring.cuh"

namespace mok {

constexpr int kPackThreads = 256;
constexpr int kPackSegments = 4;

struct PackParams {
  const void* wide_in[kPackSegments];  // packing: from; unpacking: NULL
  void* wide_out[kPackSegments];       // unpacking: to
  uint8_t* codes[kPackSegments];
  uint8_t* scales[kPackSegments];
  int64_t vectors[kPackSegments];      // of 16 wide bytes
  int64_t first_block[kPackSegments + 1];
  int segments;
  int K, atoms;                        // of the one segment whose scales are in atoms
};

template <bool F32>
constexpr int kPackElems = F32 ? 4 : 8;  // of a vector
template <bool F32>
constexpr int kPackUnroll = F32 ? 8 : 4;

__device__ __forceinline__ int segment_of(const PackParams& p) {
  int s = 0;
#pragma unroll
  for (int i = 1; i < kPackSegments; ++i) s += i < p.segments && (int64_t)blockIdx.x >= p.first_block[i];
  return s;
}

template <bool F32>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const __grid_constant__ PackParams p) {
  constexpr int N = kPackElems<F32>, U = kPackUnroll<F32>, L = 32 / N;  // elements, vectors, lanes of a block
  const int s = segment_of(p);
  const int64_t n = p.vectors[s], first = ((int64_t)blockIdx.x - p.first_block[s]) * (kPackThreads * U) + threadIdx.x;
  const uint4* src = static_cast<const uint4*>(p.wide_in[s]);
  uint4 u[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + i * kPackThreads;
    u[i] = v < n ? src[v] : make_uint4(0, 0, 0, 0);  // blocks are whole: their lanes agree
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + i * kPackThreads;
    float a[8] = {};
    if constexpr (F32) {
      a[0] = __uint_as_float(u[i].x); a[1] = __uint_as_float(u[i].y); a[2] = __uint_as_float(u[i].z); a[3] = __uint_as_float(u[i].w);
    } else {
      const Vec8 w = unpack8(u[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = w.v[j];
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) amax = fmaxf(amax, fabsf(a[j]));
#pragma unroll
    for (int o = 1; o < L; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = mx_exponent(amax);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    if (v >= n) continue;
    uint2 q;
    q.x = e4m3x2(a[0] * inv, a[1] * inv) | (uint32_t)e4m3x2(a[2] * inv, a[3] * inv) << 16;
    if constexpr (F32) {
      reinterpret_cast<uint32_t*>(p.codes[s])[v] = q.x;
    } else {
      q.y = e4m3x2(a[4] * inv, a[5] * inv) | (uint32_t)e4m3x2(a[6] * inv, a[7] * inv) << 16;
      reinterpret_cast<uint2*>(p.codes[s])[v] = q;
    }
    if (v % L == 0) p.scales[s][v / L] = (uint8_t)(e + 127);
  }
}

template <bool F32>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const __grid_constant__ PackParams p) {
  constexpr int N = kPackElems<F32>, U = kPackUnroll<F32>, L = 32 / N;
  const int s = segment_of(p);
  const int64_t n = p.vectors[s], first = ((int64_t)blockIdx.x - p.first_block[s]) * (kPackThreads * U) + threadIdx.x;
  uint2 q[U];
  uint32_t byte[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + i * kPackThreads;
    q[i] = make_uint2(0, 0);
    byte[i] = 0;
    if (v < n) {
      if constexpr (F32) q[i].x = reinterpret_cast<const uint32_t*>(p.codes[s])[v];
      else q[i] = reinterpret_cast<const uint2*>(p.codes[s])[v];
      int64_t at = v / L;
      if (p.atoms) {
        const int64_t row = v / (p.K / N);
        const int b = (int)(v - row * (p.K / N)) / L;
        at = sf_atom_word(row >> 7, b >> 2, p.K / 128, (int)(row & 127)) + (b & 3);
      }
      byte[i] = p.scales[s][at];
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t v = first + i * kPackThreads;
    const Vec8 w = dequantise8(q[i], byte[i] == 255 ? NAN : mx_scale(byte[i]));
    uint4 o = pack8(w);
    if constexpr (F32) o = make_uint4(__float_as_uint(w.v[0]), __float_as_uint(w.v[1]), __float_as_uint(w.v[2]), __float_as_uint(w.v[3]));
    if (v < n) static_cast<uint4*>(p.wide_out[s])[v] = o;
  }
}

// Gives the segments their blocks; the number of blocks.
static int64_t spread(PackParams& p, int unroll) {
  int64_t blocks = 0;
  for (int s = 0; s < p.segments; ++s) {
    p.first_block[s] = blocks;
    blocks += (p.vectors[s] + kPackThreads * unroll - 1) / (kPackThreads * unroll);
  }
  p.first_block[p.segments] = blocks;
  return blocks;
}
static cudaError_t launch_pack(PackParams& p, bool f32, bool pack, cudaStream_t s) {
  const int64_t blocks = spread(p, f32 ? kPackUnroll<true> : kPackUnroll<false>);
  if (blocks == 0) return cudaSuccess;
  void (*k)(const PackParams) = pack ? (f32 ? pack_kernel<true> : pack_kernel<false>) : (f32 ? unpack_kernel<true> : unpack_kernel<false>);
  prof_begin(pack ? "pack" : "unpack", s);
  k<<<(unsigned)blocks, kPackThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

cudaError_t launch_pack_segments(bool pack, bool f32, int segments, void* const* wide, uint8_t* const* codes,
                                 uint8_t* const* scales, const int64_t* elems, cudaStream_t s) {
  PackParams p{};
  for (int i = 0; i < segments; ++i) {
    if (elems[i] == 0) continue;
    const int j = p.segments++;
    p.wide_in[j] = p.wide_out[j] = wide[i];
    p.codes[j] = codes[i];
    p.scales[j] = scales[i];
    p.vectors[j] = elems[i] / (f32 ? kPackElems<true> : kPackElems<false>);
  }
  return launch_pack(p, f32, pack, s);
}

static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static int check_pack(int64_t rows, int K, const void* wide, int type, const void* codes, const void* scales) {
  if (type != MOK_T_BF16 && type != MOK_T_F32) return MOK_ERR_INVALID_ARG;
  if (rows < 0 || K <= 0 || K % 32 || rows > (int64_t(1) << 40) / K) return MOK_ERR_UNSUPPORTED;
  if (rows > 0 && (!wide || !codes || !scales)) return MOK_ERR_INVALID_ARG;
  return is16(wide) && is16(codes) && is16(scales) ? MOK_OK : MOK_ERR_UNSUPPORTED;
}

}  // namespace mok

extern "C" {

int mok_activation_pack(int64_t rows, int K, const void* src, int type, void* codes, void* scales, mok_stream_t stream) {
  using namespace mok;
  const int rc = check_pack(rows, K, src, type, codes, scales);
  if (rc != MOK_OK) return rc;
  const bool f32 = type == MOK_T_F32;
  PackParams p{};
  p.segments = 1;
  p.wide_in[0] = src;
  p.codes[0] = static_cast<uint8_t*>(codes);
  p.scales[0] = static_cast<uint8_t*>(scales);
  p.vectors[0] = rows * (K / (f32 ? kPackElems<true> : kPackElems<false>));
  set_last_launches(0);
  if (launch_pack(p, f32, true, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(rows > 0 ? 1 : 0);
  return MOK_OK;
}

int mok_activation_unpack(int64_t rows, int K, const void* codes, const void* scales, int scale_layout, void* dst, int type,
                          mok_stream_t stream) {
  using namespace mok;
  if (scale_layout != MOK_SCALES_ROWS && scale_layout != MOK_SCALES_ATOMS) return MOK_ERR_INVALID_ARG;
  const int rc = check_pack(rows, K, dst, type, codes, scales);
  if (rc != MOK_OK) return rc;
  if (scale_layout == MOK_SCALES_ATOMS && K % 128) return MOK_ERR_UNSUPPORTED;
  const bool f32 = type == MOK_T_F32;
  PackParams p{};
  p.segments = 1;
  p.wide_out[0] = dst;
  p.codes[0] = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scales[0] = static_cast<uint8_t*>(const_cast<void*>(scales));
  p.vectors[0] = rows * (K / (f32 ? kPackElems<true> : kPackElems<false>));
  p.K = K;
  p.atoms = scale_layout == MOK_SCALES_ATOMS;
  set_last_launches(0);
  if (launch_pack(p, f32, false, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(rows > 0 ? 1 : 0);
  return MOK_OK;
}

}  // extern "C"

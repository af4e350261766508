// Choice of the experts from router logits, and its backward pass.
//
//   s = softmax(l) or sigmoid(l);  c = s + b (the balance bias only ranks);  groups of neighbouring
//   experts by their largest c or the sum of their two largest;  top-k of c in the groups that stay;
//   w_j = scale s_j / sum s_i (or scale s_j).
//
// A warp takes a token, a lane a run of neighbouring experts of one group, so that among equal keys
// the first lane and slot hold the lowest index.  Which of two experts is chosen is decided as in
// exact arithmetic: keys are ranked in fp32, and where two that the choice depends on are nearer
// than fp32 can tell (about one token in a thousand) the few experts in question are ranked again
// in 64 bits.  Without a bias scores rise with the logits, which are ranked themselves.
#include <algorithm>
#include <cmath>

#include "mok_vec.cuh"

namespace mok {

constexpr int kSelectWarps = 4;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kMaxGroups = 32;

struct SelectParams {
  const float* logits;
  const float* bias;  // or NULL
  int32_t* topk_idx;
  float* topk_w;
  int* status;
  int64_t T;
  int E, k;
  int groups, kept, n;     // groups, how many stay, experts of one
  int lanes, log_lanes;    // of a group: a power of two
  int chunk;               // experts of a lane
  int softmax, top2, renorm;
  float scale;
};

// Order-preserving unsigned image of a float; 0 and 1 stay free below the image of -inf.
__device__ __forceinline__ unsigned ordered(float v) {
  const unsigned b = __float_as_uint(v + 0.0f);  // -0 ranks as 0
  return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr unsigned kAbsent = 0, kMasked = 1;  // no such expert, or its group is out; shut off
// Logits and biases from here on down (-inf, the lowest value of a type) shut an expert off; sums of
// two biases within +-1e30 stay finite.
constexpr float kShutOff = -1e30f;

// l - top for the exponent: 0 for the largest, whatever it is.
template <class F>
__device__ __forceinline__ F below(F l, F top) { return l == top ? F(0) : l - top; }

// 1 / (1 + e^-l), within 2^-20 of itself (expf and the quotient 2 ulp each, the sum half of one).
__device__ __forceinline__ float sigmoid_near(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }

// A token's keys in 64 bits.
struct ExactRow {
  const float* logits;  // of the token
  const float* bias;    // or NULL
  double top, sum;      // softmax: largest logit and sum of exp(l - top); sum 1 without a bias
  bool softmax;
};
__device__ __forceinline__ double exact_key(const ExactRow& r, int e, unsigned u) {
  if (u == kMasked) return -1e300;
  const double l = r.logits[e];
  const double s = r.softmax ? exp(below(l, r.top)) / r.sum : 1.0 / (1.0 + exp(-l));
  return r.bias ? s + (double)r.bias[e] : s;
}

// The k best experts of [lo, hi) in exact order among those with keys[e] >= threshold (k <= 8);
// lane j < k returns the j-th (index -1: there is none).  `list` holds hi - lo numbers.  The
// candidates are packed 24 to a round beside the best so far, so that the usual handful takes one
// evaluation in 64 bits.
__device__ __noinline__ int exact_best(const ExactRow& r, const unsigned* keys, int* list, int lo, int hi,
                                       unsigned threshold, int k, double* key_out) {
  const int lane = threadIdx.x & 31;
  int count = 0;
  for (int e0 = lo; e0 < hi; e0 += 32) {
    const int e = e0 + lane;
    const bool cand = e < hi && keys[e] >= threshold;
    const unsigned mask = __ballot_sync(kAll, cand);
    if (cand) list[count + __popc(mask & ((1u << lane) - 1u))] = e;
    count += __popc(mask);
  }
  __syncwarp();
  int idx = -1;
  double key = 0.0;
  for (int at = 0; at < count; at += 24) {
    if (lane >= 8) {
      idx = at + lane - 8 < count ? list[at + lane - 8] : -1;
      if (idx >= 0) key = exact_key(r, idx, keys[idx]);
    }
    int mine = -1;
    double mine_key = 0.0;
    for (int j = 0; j < k; ++j) {
      double bk = key;
      int bi = idx;
      for (int o = 16; o; o >>= 1) {
        const double ok = __shfl_xor_sync(kAll, bk, o);
        const int oi = __shfl_xor_sync(kAll, bi, o);
        const bool take = oi >= 0 && (bi < 0 || ok > bk || (ok == bk && oi < bi));
        if (take) { bk = ok; bi = oi; }
      }
      if (bi >= 0 && idx == bi) idx = -1;
      if (lane == j) { mine = bi; mine_key = bk; }
    }
    idx = lane < k ? mine : -1;
    key = mine_key;
  }
  __syncwarp();
  *key_out = key;
  return idx;
}

// Sum of exp(l - top) over a token's experts, in 64 bits.
__device__ __noinline__ double exact_sum(const float* row, int E, float top) {
  double z = 0.0;
  for (int e = threadIdx.x & 31; e < E; e += 32)
    if (row[e] > kShutOff) z += exp(below((double)row[e], (double)top));
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  return z;
}

// V: experts of a lane at most.  VEC: groups and runs are whole vectors of four.
template <int V, bool VEC>
__global__ void __launch_bounds__(32 * kSelectWarps) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ unsigned s_keys[kSelectWarps][kMaxE];  // only where fp32 cannot tell
  __shared__ int s_list[kSelectWarps][kMaxE];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelectWarps + warp;
  if (t >= p.T) return;
  const int group = lane >> p.log_lanes, sub = lane & (p.lanes - 1);
  const float* row = p.logits + t * p.E;
  const int first = group * p.n + sub * p.chunk;  // this lane's experts: first .. first + own - 1
  const int own = group < p.groups ? max(0, min(p.chunk, p.n - sub * p.chunk)) : 0;
  float l[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) { l[i] = -INFINITY; b[i] = 0.0f; }
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (i < own) {
        const float4 q = *reinterpret_cast<const float4*>(row + first + i);
        l[i] = q.x; l[i + 1] = q.y; l[i + 2] = q.z; l[i + 3] = q.w;
        if (p.bias) {
          const float4 a = *reinterpret_cast<const float4*>(p.bias + first + i);
          b[i] = a.x; b[i + 1] = a.y; b[i + 2] = a.z; b[i + 3] = a.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < own) {
        l[i] = row[first + i];
        if (p.bias) b[i] = p.bias[first + i];
      }
    }
  }
  // A logit that shuts its expert off becomes -inf, as does such a bias, which leaves the score.  NaN
  // (and a bias that is too large) does so too and is reported.
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bad |= l[i] != l[i] || !(b[i] < -kShutOff);
    if (!(l[i] > kShutOff)) l[i] = -INFINITY;
    if (!(fabsf(b[i]) < -kShutOff)) b[i] = -INFINITY;
  }
  if (__any_sync(kAll, bad) && lane == 0) record_status(p.status, MOK_ERR_DEVICE_CHECK);

  const bool scored = p.bias != nullptr || p.groups > 1;  // the choice depends on more than the logits' order
  float top = -INFINITY, sum = 1.0f, smax = 1.0f;
  if (p.softmax && (scored || !p.renorm)) {
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) a += l[i] > -INFINITY ? expf(below(l[i], top)) : 0.0f;
    sum = warp_sum(a);
  }
  unsigned u[V];
  float err = 0.0f;  // of a key, its last rounding apart
  if (!scored) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = i >= own ? kAbsent : l[i] > -INFINITY ? ordered(l[i]) : kMasked;
  } else {
    float c[V];
    float m = 0.0f;
    const float inv = p.softmax && p.bias ? 1.0f / sum : 1.0f;  // without a bias a common factor changes nothing
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = !(l[i] > -INFINITY) ? 0.0f : p.softmax ? expf(below(l[i], top)) * inv : sigmoid_near(l[i]);
      m = fmaxf(m, s);
      c[i] = l[i] > -INFINITY ? s + b[i] : -INFINITY;  // -inf: shut off
    }
    smax = warp_max(m);
    // softmax: expf 2 ulp, its argument D e^-D half ulps, the sum of at most 512 terms 37 half ulps
    err = smax * (p.softmax ? 0x1p-17f : 0x1p-20f) + 1e-37f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      u[i] = i >= own ? kAbsent : c[i] > -INFINITY ? ordered(p.bias ? c[i] : l[i]) : kMasked;
    if (p.groups > 1) {
      float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i < own) {
          t2 = fmaxf(t2, fminf(t1, c[i]));
          t1 = fmaxf(t1, c[i]);
        }
      }
      for (int o = 1; o < p.lanes; o <<= 1) {
        const float a1 = __shfl_xor_sync(kAll, t1, o), a2 = __shfl_xor_sync(kAll, t2, o);
        t2 = fmaxf(fmaxf(t2, a2), fminf(t1, a1));
        t1 = fmaxf(t1, a1);
      }
      const float score = p.top2 && t2 > -INFINITY ? t1 + t2 : t1;
      int rank = 0;
      float in = INFINITY, out = -INFINITY;  // lowest score that stays, highest that goes
      for (int g = 0; g < p.groups; ++g) {
        const float other = __shfl_sync(kAll, score, g << p.log_lanes);
        rank += other > score || (other == score && g < group);
      }
      bool stays = rank < p.kept;
      if (group < p.groups) {
        if (stays) in = score;
        else out = score;
      }
      in = -warp_max(-in);
      out = warp_max(out);
      // a group without experts (-inf) never comes near one that has some
      const float size = warp_max(t2 > -INFINITY ? fabsf(t1) + fabsf(t2) : t1 > -INFINITY ? fabsf(t1) : 0.0f);
      const float slack = 4.0f * err + 0x1p-21f * size;
      if (p.kept < p.groups && out > -INFINITY && !(in - out > slack)) {
        const ExactRow xr{row, p.bias, top, p.softmax && p.bias ? exact_sum(row, p.E, top) : 1.0, (bool)p.softmax};
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < own) s_keys[warp][first + i] = c[i] > -INFINITY ? ordered(c[i]) : kAbsent;
        __syncwarp();
        double mine = -1e300;  // exact score of this lane's group; far ones keep their fp32 score
        if (score > -INFINITY) mine = score;
        for (int g = 0; g < p.groups; ++g) {
          const float sc = __shfl_sync(kAll, score, g << p.log_lanes);
          const float second = __shfl_sync(kAll, p.top2 && t2 > -INFINITY ? t2 : t1, g << p.log_lanes);
          if (!(sc > -INFINITY) || sc - in > slack || out - sc > slack) continue;
          double key;
          const int e = exact_best(xr, s_keys[warp], s_list[warp], g * p.n, (g + 1) * p.n,
                                   ordered(second - 2.0f * err - 0x1p-22f * fabsf(second)), p.top2 ? 2 : 1, &key);
          const double k1 = __shfl_sync(kAll, key, 0), k2 = __shfl_sync(kAll, key, 1);
          const int e2 = __shfl_sync(kAll, e, 1);
          if (group == g) mine = p.top2 && e2 >= 0 ? k1 + k2 : k1;
        }
        rank = 0;
        for (int g = 0; g < p.groups; ++g) {
          const double other = __shfl_sync(kAll, mine, g << p.log_lanes);
          rank += other > mine || (other == mine && g < group);
        }
        stays = rank < p.kept;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!stays) u[i] = kAbsent;
    }
  }

  unsigned best = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) best = max(best, u[i]);
  int idx = 0;             // lane j < k: the j-th expert
  unsigned key = kMasked;  // and its key
  const int rounds = p.bias ? p.k + 1 : p.k;  // one more: the best of those that are not chosen
  unsigned gone = 0;       // this lane's slots that are taken
  for (int j = 0; j < rounds; ++j) {
    const unsigned m = __reduce_max_sync(kAll, best);
    const int w = __ffs(__ballot_sync(kAll, best == m)) - 1;
    int slot = 0;
    if (lane == w) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (u[i] == m && !(gone >> i & 1)) slot = i;
      gone |= 1u << slot;
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (!(gone >> i & 1)) best = max(best, u[i]);
    }
    const int e = __shfl_sync(kAll, first + slot, w);
    if (lane == j) { idx = e; key = m; }
  }
  if (p.bias) {
    // Neighbours in the order that are nearer than their errors, unless they are one and the same
    // number; such a pair at the border may have others as near behind it.
    const float a = unordered(key);
    const float last = __shfl_sync(kAll, a, p.k - 1);
    auto near = [&](float x, float y) { return !(x - y > 2.0f * err + 0x1p-23f * (fabsf(x) + fabsf(y))); };
    const unsigned next = __shfl_down_sync(kAll, key, 1);
    const int other = __shfl_down_sync(kAll, idx, 1);
    bool unsure = false, tie = false;
    if (lane < p.k && key > kMasked && next > kMasked && near(a, unordered(next))) {
      tie = row[idx] == row[other] && p.bias[idx] == p.bias[other];
      unsure = !tie;
    }
    if (__shfl_sync(kAll, (int)tie, p.k - 1)) {
      const int e = __shfl_sync(kAll, idx, p.k - 1);
      const float le = row[e], be = p.bias[e];
#pragma unroll
      for (int i = 0; i < V; ++i)
        unsure |= u[i] > kMasked && !(gone >> i & 1) && near(last, unordered(u[i])) && !(l[i] == le && b[i] == be);
    }
    if (__any_sync(kAll, unsure)) {
      const ExactRow xr{row, p.bias, top, p.softmax ? exact_sum(row, p.E, top) : 1.0, (bool)p.softmax};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < own) s_keys[warp][first + i] = u[i];
      __syncwarp();
      const bool all = __shfl_sync(kAll, key, p.k - 1) == kMasked;  // fewer than k are open
      double d;
      idx = exact_best(xr, s_keys[warp], s_list[warp], 0, p.E,
                       all ? kMasked : max(ordered(last - 2.0f * err - 0x1p-22f * fabsf(last)), kMasked), p.k, &d);
    }
  }
  // weights: lane j has its own logit
  const bool mine = lane < p.k;
  const float lj = mine ? row[idx] : -INFINITY;
  const bool on = mine && lj > kShutOff;
  float wj = 0.0f;
  if (p.renorm) {
    // both scores over their largest possible common factor, so that small ones do not vanish:
    // softmax e^(l - m); sigmoid e^(l - m) / (1 + e^l) for m = max l <= 0, else its value
    const float m = warp_max(on ? lj : -INFINITY);
    if (on) wj = p.softmax ? expf(below(lj, m)) : m <= 0.0f ? expf(below(lj, m)) / (1.0f + expf(lj)) : 1.0f / (1.0f + expf(-lj));
    const float total = warp_sum(wj);
    wj = total > 0.0f ? p.scale * (wj / total) : 0.0f;
  } else if (on) {
    wj = p.scale * (p.softmax ? expf(below(lj, top)) / sum : 1.0f / (1.0f + expf(-lj)));
  }
  if (mine) {
    p.topk_idx[t * p.k + lane] = idx;
    p.topk_w[t * p.k + lane] = wj;
  }
}

struct SelectBwdParams {
  const float* logits;
  const int32_t* topk_idx;
  const float* dw;         // [T, k], or NULL: sums of
  const float* partial;    // <a, h> per destination row and N tile, [R, ldp]
  const int32_t* inv_pos;  // destination row of every route
  int ldp;
  const float* aux;        // [T, E] or NULL
  float* dlogits;
  __nv_bfloat16* dl;       // [T, ldl] copy for the layer's GEMMs, or NULL
  int ldl;
  int* status;
  int64_t T;
  int E, k;
  int softmax, renorm;
  float scale;
};

constexpr int kSelectBwdWarps = 8;

// A warp takes a token: lane j < k the j-th chosen expert, whose gradient goes to its place of a
// row of zeros in shared memory; then every lane writes vectors of four.  With p_j = s_j / sum s_i
//   renormalised: dl_j = scale p_j (dw_j - sum p_i dw_i) (times 1 - s_j for sigmoid scores);
//   sigmoid:      dl_j = scale s_j (1 - s_j) dw_j;
//   softmax:      dl_e = scale s_e (dw of e - sum s_i dw_i), for every expert.
__global__ void __launch_bounds__(32 * kSelectBwdWarps) select_bwd_kernel(const __grid_constant__ SelectBwdParams p) {
  __shared__ float4 s_up[kSelectBwdWarps][kMaxE / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* up = reinterpret_cast<float*>(s_up[warp]);
  const int nvec = p.E / 4;
  for (int v = lane; v < nvec; v += 32) s_up[warp][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncwarp();
  const int64_t step = (int64_t)gridDim.x * kSelectBwdWarps;
  for (int64_t t = (int64_t)blockIdx.x * kSelectBwdWarps + warp; t < p.T; t += step) {
    const float* row = p.logits + t * p.E;
    int e = -1;
    float l = -INFINITY, dw = 0.0f;
    if (lane < p.k) {
      const int64_t r = t * p.k + lane;
      e = p.topk_idx[r];
      if (e < 0 || e >= p.E) {
        record_status(p.status, MOK_ERR_DEVICE_CHECK);
        e = -1;
      } else {
        l = row[e];
      }
      if (p.dw) {
        dw = p.dw[r];
      } else {
        const int pos = p.inv_pos[r];
        if (pos >= 0)
          for (int n = 0; n < p.ldp; ++n) dw += p.partial[(int64_t)pos * p.ldp + n];
      }
    }
    const bool on = l > kShutOff;  // not NaN either
    const bool dense = p.softmax && !p.renorm;
    float top = -INFINITY, sum = 1.0f;
    if (dense) {
      for (int v = lane; v < nvec; v += 32) {
        const float4 q = reinterpret_cast<const float4*>(row)[v];
        top = fmaxf(fmaxf(fmaxf(top, q.x), fmaxf(q.y, q.z)), q.w);  // fmaxf passes NaN by
      }
      top = warp_max(top);
      sum = 0.0f;
      for (int v = lane; v < nvec; v += 32) {
        const float4 q = reinterpret_cast<const float4*>(row)[v];
        for (float a : {q.x, q.y, q.z, q.w}) sum += a > kShutOff ? expf(below(a, top)) : 0.0f;
      }
      sum = warp_sum(sum);
    }
    float g = 0.0f, inner = 0.0f;
    if (dense) {
      const float s = on ? expf(below(l, top)) / sum : 0.0f;
      inner = warp_sum(on ? s * dw : 0.0f);
      g = on ? dw : 0.0f;
    } else if (p.renorm) {
      const float m = warp_max(on ? l : -INFINITY);
      float s = 0.0f;
      if (on) s = p.softmax ? expf(below(l, m)) : m <= 0.0f ? expf(below(l, m)) / (1.0f + expf(l)) : 1.0f / (1.0f + expf(-l));
      const float total = warp_sum(s);
      const float pj = total > 0.0f ? s / total : 0.0f;
      const float dot = warp_sum(on ? pj * dw : 0.0f);
      if (on) g = p.scale * pj * (dw - dot) * (p.softmax ? 1.0f : 1.0f / (1.0f + expf(l)));
    } else if (on) {
      g = p.scale * dw * (1.0f / (1.0f + expf(-l))) * (1.0f / (1.0f + expf(l)));
    }
    float total = 0.0f;  // routes that name one expert twice add up, in the routes' order
    for (int j = 0; j < p.k; ++j) {
      const int ej = __shfl_sync(kAll, e, j);
      const float gj = __shfl_sync(kAll, g, j);
      if (ej == e) total += gj;
    }
    if (e >= 0) up[e] = total;
    __syncwarp();
    const int end = p.dl ? p.ldl / 4 : nvec;
    for (int v = lane; v < end; v += 32) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (v < nvec) {
        a = s_up[warp][v];
        if (dense) {
          const float4 q = reinterpret_cast<const float4*>(row)[v];
          auto grad = [&](float x, float d) { return x > kShutOff ? p.scale * (expf(below(x, top)) / sum) * (d - inner) : 0.0f; };
          a = make_float4(grad(q.x, a.x), grad(q.y, a.y), grad(q.z, a.z), grad(q.w, a.w));
        }
        if (p.aux) {
          const float4 x = reinterpret_cast<const float4*>(p.aux + t * p.E)[v];
          a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        }
        reinterpret_cast<float4*>(p.dlogits + t * p.E)[v] = a;
      }
      if (p.dl) reinterpret_cast<uint2*>(p.dl + t * p.ldl)[v] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    }
    __syncwarp();
    if (e >= 0) up[e] = 0.0f;
    __syncwarp();
  }
}

int check_selection(const mok_dims* dims, const mok_selection* sel) {
  if (!sel) return MOK_ERR_INVALID_ARG;
  if ((sel->score != MOK_SCORE_SOFTMAX && sel->score != MOK_SCORE_SIGMOID) ||
      (sel->group_score != MOK_GROUP_MAX && sel->group_score != MOK_GROUP_TOP2) || !std::isfinite(sel->scale))
    return MOK_ERR_INVALID_ARG;
  if (sel->n_groups < 1 || sel->n_groups > kMaxGroups || dims->E % sel->n_groups || sel->topk_groups < 1 ||
      sel->topk_groups > sel->n_groups || dims->k > sel->topk_groups * (dims->E / sel->n_groups))
    return MOK_ERR_UNSUPPORTED;
  return MOK_OK;
}

cudaError_t launch_select_backward(const mok_dims* dims, const mok_selection* sel, const float* logits,
                                   const int32_t* topk_idx, const float* dw, const float* partial,
                                   const int32_t* inv_pos, int ldp, const float* aux, float* dlogits,
                                   void* dl_bf16, int* status, cudaStream_t s) {
  SelectBwdParams p{logits, topk_idx, dw, partial, inv_pos, ldp, aux, dlogits, static_cast<__nv_bfloat16*>(dl_bf16),
                    (dims->E + 63) & ~63, status, dims->T, dims->E, dims->k, sel->score == MOK_SCORE_SOFTMAX,
                    sel->renormalise != 0, sel->scale};
  const int64_t blocks = (dims->T + kSelectBwdWarps - 1) / kSelectBwdWarps;
  prof_begin("select_bwd", s);
  select_bwd_kernel<<<(int)std::min<int64_t>(blocks, (int64_t)num_sms() * 8), 32 * kSelectBwdWarps, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

static bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool is4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace mok

extern "C" {

int mok_select_experts(const mok_dims* dims, const mok_selection* sel, const float* logits, const float* sel_bias,
                       int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes, mok_stream_t stream) {
  using namespace mok;
  int rc = check_dims(dims);
  if (rc == MOK_OK) rc = check_selection(dims, sel);
  if (rc != MOK_OK) return rc;
  if (!ws || (dims->T > 0 && (!logits || !topk_idx || !topk_w))) return MOK_ERR_INVALID_ARG;
  if (!is16(logits) || !is16(sel_bias) || !is16(ws) || !is4(topk_idx) || !is4(topk_w)) return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < 256) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  if (dims->T == 0) return MOK_OK;
  SelectParams p{logits, sel_bias, topk_idx, topk_w, static_cast<int*>(ws), dims->T, dims->E, dims->k, sel->n_groups,
                 sel->topk_groups, dims->E / sel->n_groups, 1, 0, 0, sel->score == MOK_SCORE_SOFTMAX,
                 sel->group_score == MOK_GROUP_TOP2, sel->renormalise != 0, sel->scale};
  while (2 * p.lanes * p.groups <= 32) {
    p.lanes *= 2;
    ++p.log_lanes;
  }
  p.chunk = (p.n + p.lanes - 1) / p.lanes;  // at most 30: E <= 512
  const bool vec = p.n % 4 == 0;
  if (vec) p.chunk = (p.chunk + 3) / 4 * 4;
  void (*k)(const SelectParams) = nullptr;
  if (vec) k = p.chunk <= 4 ? select_kernel<4, true> : p.chunk <= 8 ? select_kernel<8, true> : p.chunk <= 12 ? select_kernel<12, true>
               : p.chunk <= 16 ? select_kernel<16, true> : select_kernel<32, true>;
  else k = p.chunk <= 8 ? select_kernel<8, false> : select_kernel<32, false>;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  prof_begin("select", s);
  k<<<(unsigned)((dims->T + kSelectWarps - 1) / kSelectWarps), 32 * kSelectWarps, 0, s>>>(p);
  prof_end(s);
  if (cudaGetLastError() != cudaSuccess) return MOK_ERR_CUDA;
  set_last_launches(1);
  return MOK_OK;
}

int mok_select_experts_backward(const mok_dims* dims, const mok_selection* sel, const float* logits,
                                const int32_t* topk_idx, const float* dtopk_w, const float* dlogits_aux,
                                float* dlogits, void* ws, size_t ws_bytes, mok_stream_t stream) {
  using namespace mok;
  int rc = check_dims(dims);
  if (rc == MOK_OK) rc = check_selection(dims, sel);
  if (rc != MOK_OK) return rc;
  if (!ws || (dims->T > 0 && (!logits || !topk_idx || !dtopk_w || !dlogits))) return MOK_ERR_INVALID_ARG;
  if (!is16(logits) || !is16(dlogits_aux) || !is16(dlogits) || !is16(ws) || !is4(topk_idx) || !is4(dtopk_w))
    return MOK_ERR_UNSUPPORTED;
  if (ws_bytes < 256) return MOK_ERR_WORKSPACE;
  set_last_launches(0);
  if (dims->T == 0) return MOK_OK;
  if (launch_select_backward(dims, sel, logits, topk_idx, dtopk_w, nullptr, nullptr, 0, dlogits_aux, dlogits, nullptr,
                             static_cast<int*>(ws), reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MOK_ERR_CUDA;
  set_last_launches(1);
  return MOK_OK;
}

}  // extern "C"

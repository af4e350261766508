// Choice of the experts from router logits, and its backward pass.
//
//   s = softmax(l) or sigmoid(l);  c = s + b (the balance bias only ranks);  groups of neighbouring
//   experts by their largest c or the sum of their two largest;  top-k of c in the groups that stay;
//   w_j = scale s_j / sum s_i (or scale s_j).
//
// A warp takes a token, a lane a run of neighbouring experts of one group, in ascending order.  The
// k-th largest of the lanes' own largest keys is a lower limit of the k-th key, which leaves about
// k + 2 candidates (their expected number, 32 (H(32) - H(32 - k)), is 9.1 for k = 8); these go
// to a lane each and are ranked by counting.  Which of two experts is chosen does not depend on fp32
// roundings: where two keys that the choice depends on are nearer than fp32 can tell (a few tokens
// in a thousand) the experts in question are ranked again in 64 bits, and keys that are equal there by their
// logits, with which scores rise (a sigmoid is 1 in 64 bits from 37 on).  Without a bias the logits are
// ranked themselves.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "mok_vec.cuh"

namespace mok {

constexpr int kSelectWarps = 2;
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
  int top2, renorm;
  float scale;
};

// Keys: kAbsent for a slot without an expert, or whose group is out; kMasked for one that is shut off.
constexpr float kAbsent = -INFINITY, kMasked = -FLT_MAX;
// Logits from here on down (-inf, the lowest value of a type) shut an expert off: it ranks last and weighs
// 0.  Biases from here on down only rank: the expert is the last choice, with its score.  Sums of two biases
// within +-1e30 stay finite.
constexpr float kShutOff = -1e30f;

__device__ __forceinline__ float warp_top(float v) {  // not NaN
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// l - top for the exponent: 0 for the largest, whatever it is.
template <class F>
__device__ __forceinline__ F below(F l, F top) { return l == top ? F(0) : l - top; }

// e^x from one product and ex2.approx (2 ulp; results below 2^-126 are 0): off by at most
// 2^-22 + 2^-23 |x| of itself.
__device__ __forceinline__ float exp_near(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.44269504f));
  return r;
}
__device__ __forceinline__ float reciprocal_near(float x) {  // 1 ulp; 0 above 2^126
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A token's row and what its scores need.
template <bool SOFTMAX, bool BIAS>
struct SelectRow {
  const float* logits;
  const float* bias;
  float top, inv;  // softmax: largest logit, 1 / sum of exp(l - top) (1 without a bias: a common factor)
  // Off by at most error() before the sum with the bias is rounded.
  __device__ __forceinline__ float score(float l) const {
    return SOFTMAX ? exp_near(below(l, top)) * inv : reciprocal_near(1.0f + exp_near(-l));
  }
  // The largest error of the row's scores: |x| e^-x < 0.37 for x > 0, so the errors are a multiple of
  // the largest score; for sigmoid scores of negative logits |x| reaches the largest logit's.  softmax:
  // the sum of at most 512 terms adds 37 roundings and the terms' own errors.
  __device__ __forceinline__ float error() const {
    return score(top) * (SOFTMAX ? 0x1p-17f : fmaf(0x1p-22f, fmaxf(-top, 0.0f), 0x1p-20f)) + 1e-37f;
  }
  __device__ __forceinline__ float bias_of(int e) const { return BIAS ? bias[e] : 0.0f; }
  // What experts are ranked by, and what groups are.
  __device__ __forceinline__ float key(float l, float b) const {
    if constexpr (!BIAS) return l > kShutOff ? l : kMasked;
    const float c = score(l) + b;
    return l > kShutOff && fabsf(b) < -kShutOff ? c : kMasked;
  }
  __device__ __forceinline__ float group_key(float l, float b) const {
    const float c = score(l) + b;
    return l > kShutOff && (!BIAS || fabsf(b) < -kShutOff) ? c : -INFINITY;
  }
};

// Key of expert e in 64 bits; sum: of exp(l - top), for softmax with a bias.
template <bool SOFTMAX, bool BIAS>
__device__ __forceinline__ double exact_key(const SelectRow<SOFTMAX, BIAS>& r, double sum, int e, float key) {
  if (key == kMasked) return -1e300;
  const double l = r.logits[e];
  const double s = SOFTMAX ? exp(below(l, (double)r.top)) / sum : 1.0 / (1.0 + exp(-l));
  return BIAS ? s + (double)r.bias[e] : s;
}
template <bool SOFTMAX, bool BIAS>
__device__ __noinline__ double exact_sum(SelectRow<SOFTMAX, BIAS> r, int E) {
  if (!SOFTMAX || !BIAS) return 1.0;
  double z = 0.0;
  for (int e = threadIdx.x & 31; e < E; e += 32)
    if (r.logits[e] > kShutOff) z += exp(below((double)r.logits[e], (double)r.top));
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  return z;
}

// The k best experts of [lo, hi) in exact order (64-bit key, logit, lower index) among those with keys[e] >=
// threshold (k <= 8); lane j < k returns the j-th (index -1: there is none).  `list` holds hi - lo numbers.
// Up to 32 are ranked by counting; more of them (many equal numbers) come 24 to a round beside the best
// so far.
template <bool SOFTMAX, bool BIAS>
__device__ __noinline__ int exact_best(SelectRow<SOFTMAX, BIAS> r, double sum, const float* keys, int* list, int lo, int hi,
                                       float threshold, int k, double* key_out) {
  const int lane = threadIdx.x & 31;
  int count = 0;
  for (int e0 = lo; e0 < hi; e0 += 32) {
    const int e = e0 + lane;
    const bool cand = e < hi && keys[e] > kAbsent && keys[e] >= threshold;
    const unsigned mask = __ballot_sync(kAll, cand);
    if (cand) list[count + __popc(mask & ((1u << lane) - 1u))] = e;
    count += __popc(mask);
  }
  __syncwarp();
  int idx = -1;
  double key = 0.0;
  // Of experts a and b with equal keys, whether a comes first.
  auto first = [&](int a, int b) {
    const float la = r.logits[a], lb = r.logits[b];
    return keys[a] != kMasked && la != lb ? la > lb : a < b;
  };
  if (count <= 32) {  // a lane each, in ascending order
    if (lane < count) {
      idx = list[lane];
      key = exact_key(r, sum, idx, keys[idx]);
    }
    int place = 0;
    for (int j = 0; j < count; ++j) {
      const double o = __shfl_sync(kAll, key, j);
      place += o > key || (o == key && j != lane && lane < count && first(list[j], idx));
    }
    __syncwarp();
    if (lane < count) list[place] = lane;
    __syncwarp();
    const int from = lane < min(k, count) ? list[lane] : -1;
    const int i = __shfl_sync(kAll, idx, max(from, 0));
    const double d = __shfl_sync(kAll, key, max(from, 0));
    __syncwarp();
    *key_out = d;
    return from < 0 ? -1 : i;
  }
  for (int at = 0; at < count; at += 24) {
    if (lane >= 8) {
      idx = at + lane - 8 < count ? list[at + lane - 8] : -1;
      if (idx >= 0) key = exact_key(r, sum, idx, keys[idx]);
    }
    int mine = -1;
    double mine_key = 0.0;
    for (int j = 0; j < k; ++j) {
      double bk = key;
      int bi = idx;
      for (int o = 16; o; o >>= 1) {
        const double ok = __shfl_xor_sync(kAll, bk, o);
        const int oi = __shfl_xor_sync(kAll, bi, o);
        const bool take = oi >= 0 && (bi < 0 || ok > bk || (ok == bk && first(oi, bi)));
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

// Whether this lane's group stays, where fp32 scores of one that stays and one that goes are within
// slack: groups farther than that from both keep their fp32 score, the others get exact ones.  Largest keys
// that are equal in 64 bits go by their logits, sums of two to the lower group.
template <bool SOFTMAX, bool BIAS>
__device__ __noinline__ bool exact_groups(SelectRow<SOFTMAX, BIAS> r, const SelectParams& p, float* keys, int* list, float err,
                                          float score, float second, float in, float out, float slack) {
  const int lane = threadIdx.x & 31, group = lane >> p.log_lanes;
  for (int e = lane; e < p.E; e += 32) keys[e] = r.group_key(r.logits[e], r.bias_of(e));
  const double sum = exact_sum(r, p.E);
  __syncwarp();
  double mine = score > -INFINITY ? (double)score : -1e300;
  float mine_l = 0.0f;
  for (int g = 0; g < p.groups; ++g) {
    const float sc = __shfl_sync(kAll, score, g << p.log_lanes), low = __shfl_sync(kAll, second, g << p.log_lanes);
    if (!(sc > -INFINITY) || sc - in > slack || out - sc > slack) continue;
    double key;
    const int e = exact_best(r, sum, keys, list, g * p.n, (g + 1) * p.n, low - 2.0f * err - 0x1p-22f * fabsf(low),
                             p.top2 ? 2 : 1, &key);
    const double k1 = __shfl_sync(kAll, key, 0), k2 = __shfl_sync(kAll, key, 1);
    const int e1 = __shfl_sync(kAll, e, 0), e2 = __shfl_sync(kAll, e, 1);
    if (group == g) {
      mine = p.top2 && e2 >= 0 ? k1 + k2 : k1;
      mine_l = p.top2 || e1 < 0 ? 0.0f : r.logits[e1];
    }
  }
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const double other = __shfl_sync(kAll, mine, g << p.log_lanes);
    const float other_l = __shfl_sync(kAll, mine_l, g << p.log_lanes);
    rank += other > mine || (other == mine && (other_l > mine_l || (other_l == mine_l && g < group)));
  }
  return rank < p.kept;
}

// Bound by latencies (64% of the issue slots): at T = 16384, E = 384, k = 8 with sigmoid scores and a bias
// 18.9 us (12.3 without a bias; 4 at the copy rate), E = 256 with 4 of 8 groups 20-24.  Most of a token's
// instructions do not depend on E, and 2 tokens in a warp share them but wait longer: 27 us where one
// took 23.6.  Ranking by rounds of a maximum over the warp 47 us.
// V: experts of a lane at most.  VEC: groups and runs are whole vectors of four.
template <int V, bool VEC, bool SOFTMAX, bool BIAS>
__global__ void __launch_bounds__(32 * kSelectWarps, V <= 16 ? 14 : 8) select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ __align__(16) float s_keys[kSelectWarps][kMaxE];
  __shared__ int s_list[kSelectWarps][kMaxE];
  __shared__ float s_key[kSelectWarps][kMaxK + 1];  // the chosen ones and the next, in order
  __shared__ int s_idx[kSelectWarps][kMaxK + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kSelectWarps + warp;
  if (t >= p.T) return;
  const int group = lane >> p.log_lanes, sub = lane & (p.lanes - 1);
  const float* row = p.logits + t * p.E;
  const int first = group * p.n + sub * p.chunk;  // this lane's experts: first .. first + own - 1
  const int own = group < p.groups ? max(0, min(p.chunk, p.n - sub * p.chunk)) : 0;
  float* keys = s_keys[warp];
  int* list = s_list[warp];
  float c[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) { c[i] = -INFINITY; b[i] = 0.0f; }
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (i < own) {
        const float4 q = *reinterpret_cast<const float4*>(row + first + i);
        c[i] = q.x; c[i + 1] = q.y; c[i + 2] = q.z; c[i + 3] = q.w;
        if constexpr (BIAS) {
          const float4 a = *reinterpret_cast<const float4*>(p.bias + first + i);
          b[i] = a.x; b[i + 1] = a.y; b[i + 2] = a.z; b[i + 3] = a.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < own) {
        c[i] = row[first + i];
        if (BIAS) b[i] = p.bias[first + i];
      }
    }
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) top = max_or_nan(top, c[i]);
  bool bad = top != top;
  if (bad) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, c[i]);  // passes NaN by
  }
  if (BIAS && t == 0) {  // the same for every token
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !(b[i] < -kShutOff);
  }
  if (__any_sync(kAll, bad) && lane == 0) record_status(p.status, MOK_ERR_DEVICE_CHECK);

  SelectRow<SOFTMAX, BIAS> r{row, p.bias, warp_top(top), 1.0f};
  float sum = 1.0f;
  if (SOFTMAX && (BIAS || !p.renorm)) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) a += c[i] > kShutOff ? exp_near(below(c[i], r.top)) : 0.0f;
    sum = warp_sum(a);
    if (BIAS) r.inv = 1.0f / sum;
  }
  const float err = r.error();
  bool stays = true;
  if (p.groups > 1) {
    float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float g = r.group_key(c[i], b[i]);  // -inf where there is no expert
      t2 = fmaxf(t2, fminf(t1, g));
      t1 = fmaxf(t1, g);
    }
    for (int o = 1; o < p.lanes; o <<= 1) {
      const float a1 = __shfl_xor_sync(kAll, t1, o), a2 = __shfl_xor_sync(kAll, t2, o);
      t2 = fmaxf(fmaxf(t2, a2), fminf(t1, a1));
      t1 = fmaxf(t1, a1);
    }
    const bool both = p.top2 && t2 > -INFINITY;
    const float score = both ? t1 + t2 : t1;
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float other = __shfl_sync(kAll, score, g << p.log_lanes);
      rank += other > score || (other == score && g < group);
    }
    stays = rank < p.kept;
    const bool real = group < p.groups;
    const float in = -warp_top(real && stays ? -score : -INFINITY);   // the lowest score that stays
    const float out = warp_top(real && !stays ? score : -INFINITY);   // the highest that goes
    if (out > -INFINITY) {
      const float size = warp_top(both ? fabsf(t1) + fabsf(t2) : t1 > -INFINITY ? fabsf(t1) : 0.0f);
      const float slack = 4.0f * err + 0x1p-21f * size;
      if (!(in - out > slack)) stays = exact_groups(r, p, keys, list, err, score, both ? t2 : t1, in, out, slack);
    }
  }
  float best = kAbsent;
  const int here = stays ? own : 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    c[i] = (VEC ? i / 4 * 4 : i) < here ? r.key(c[i], b[i]) : kAbsent;  // VEC: whole fours
    best = fmaxf(best, c[i]);
  }
  // The `want`-th largest of the lanes' largest keys (one more than k where the next one matters).  (The
  // least of the largest keys of 8 sets of lanes takes a tenth of the instructions and leaves 22
  // candidates: 21.9 us where this took 20.0.)
  const int want = BIAS ? p.k + 1 : p.k;
  float limit = kAbsent, left = best;
  for (int j = 0; j < want; ++j) {
    limit = warp_top(left);
    if (left == limit) left = kAbsent;  // equal ones together: the limit is then lower than it might be
  }
  if (limit == kAbsent && __popc(__ballot_sync(kAll, best > kAbsent)) >= want)  // or all of them: the least of the lanes' largest
    limit = -warp_top(best > kAbsent ? -best : kAbsent);
  // Candidates in ascending order: open experts with keys at the limit or above.  Beyond 32 of them, of
  // those at the limit only the first `want`, behind the others; fewer than k, shut off ones behind them.
  unsigned mine = 0;
  const float from = fmaxf(limit, kMasked / 2);  // below every open key
#pragma unroll
  for (int i = 0; i < V; ++i) mine |= (c[i] >= from ? 1u : 0u) << i;
  auto scan = [&](unsigned v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  unsigned upto = scan(__popc(mine));
  int n = (int)__shfl_sync(kAll, upto, 31);
  int at = (int)upto - __popc(mine);
  if ((n > 32 && limit > kMasked) || n < p.k) {
    const float rest = n < p.k ? kMasked : limit;
    unsigned equal = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) equal |= (c[i] == rest ? 1u : 0u) << i;
    mine &= ~equal;
    const unsigned two = __popc(mine) | __popc(equal) << 16;
    upto = scan(two);
    const unsigned all = __shfl_sync(kAll, upto, 31);
    const int more = (int)(all & 0xffff);
    at = (int)((upto - two) & 0xffff);
    n = more + min((int)(all >> 16), want);
    for (int q = more + (int)((upto - two) >> 16); equal && q < n; ++q, equal &= equal - 1) list[q] = first + __ffs(equal) - 1;
  }
  for (; mine; mine &= mine - 1) list[at++] = first + __ffs(mine) - 1;
  __syncwarp();
  // A lane per candidate: its key once more, then its place in the order: the number of larger ones, and
  // of equal ones before it.
  if (lane <= kMaxK) s_idx[warp][lane] = 0;
  for (int q = lane; q < (n + 3) / 4 * 4; q += 32)
    keys[q] = q < n ? r.key(row[list[q]], r.bias_of(list[q])) + 0.0f : kAbsent;  // one zero
  __syncwarp();
  for (int q = lane; q < n; q += 32) {
    const float key = keys[q];
    int place = 0;
    for (int j = 0; j < n; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(keys + j);
      place += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
    }
    if (n <= 32) {  // the lanes below n, once
      const unsigned here = n == 32 ? kAll : (1u << n) - 1u;
      place += __popc(__match_any_sync(here, __float_as_uint(key)) & ((1u << lane) - 1u));
    } else {
      for (int j = 0; j < q; ++j) place += keys[j] == key;
    }
    if (place < want) {
      s_key[warp][place] = key;
      s_idx[warp][place] = list[q];
    }
  }
  __syncwarp();
  int idx = lane < min(want, n) ? s_idx[warp][lane] : 0;  // n >= k
  const float key = lane < min(want, n) ? s_key[warp][lane] : kAbsent;
  if constexpr (BIAS) {
    // Neighbours in the order that are nearer than their errors, unless they are one and the same
    // number; such a pair at the border may have others as near behind it.
    const float last = __shfl_sync(kAll, key, p.k - 1);
    const int last_idx = __shfl_sync(kAll, idx, p.k - 1);
    auto near = [&](float x, float y) { return !(x - y > 2.0f * err + 0x1p-23f * (fabsf(x) + fabsf(y))); };
    const float next = __shfl_down_sync(kAll, key, 1);
    const int other = __shfl_down_sync(kAll, idx, 1);
    bool unsure = false, tie = false;
    if (lane < p.k && key > kMasked && next > kMasked && near(key, next)) {
      tie = row[idx] == row[other] && p.bias[idx] == p.bias[other];
      unsure = !tie;
    }
    if (__shfl_sync(kAll, (int)tie, p.k - 1)) {
#pragma unroll 1
      for (int e = first; e < first + own; ++e) {
        const float y = r.key(row[e], r.bias_of(e));
        unsure |= stays && y > kMasked && (y < last || (y == last && e > last_idx)) && near(last, y) &&
                  !(row[e] == row[last_idx] && p.bias[e] == p.bias[last_idx]);
      }
    }
    if (__any_sync(kAll, unsure)) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < own) keys[first + i] = c[i];
      const double total = exact_sum(r, p.E);
      __syncwarp();
      double d;
      // kMasked: fewer than k are open
      idx = exact_best(r, total, keys, list, 0, p.E,
                       last == kMasked ? kMasked : fmaxf(last - 2.0f * err - 0x1p-22f * fabsf(last), kMasked), p.k, &d);
      idx = max(idx, 0);
    }
  }
  // weights: lane j has its own logit
  const float lj = lane < p.k ? row[idx] : -INFINITY;
  const bool on = lj > kShutOff;
  float wj = 0.0f;
  if (p.renorm) {
    // both scores over their largest possible common factor, so that small ones do not vanish:
    // softmax e^(l - m); sigmoid e^(l - m) / (1 + e^l) for m = max l <= 0, else its value
    const float m = warp_top(on ? lj : -INFINITY);
    if (on) wj = SOFTMAX ? expf(below(lj, m)) : m <= 0.0f ? __fdividef(expf(below(lj, m)), 1.0f + expf(lj)) : __fdividef(1.0f, 1.0f + expf(-lj));
    const float total = warp_sum(wj);
    wj = total > 0.0f ? p.scale * __fdividef(wj, total) : 0.0f;
  } else if (on) {
    wj = p.scale * (SOFTMAX ? __fdividef(expf(below(lj, r.top)), sum) : __fdividef(1.0f, 1.0f + expf(-lj)));
  }
  if (lane < p.k) {
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
// row of zeros in shared memory; then every lane writes its up to four vectors of four.  With p_j = s_j / sum s_i
//   renormalised: dl_j = scale p_j (dw_j - sum p_i dw_i) (times 1 - s_j for sigmoid scores);
//   sigmoid:      dl_j = scale s_j (1 - s_j) dw_j;
//   softmax:      dl_e = scale s_e (dw of e - sum s_i dw_i), for every expert (DENSE).
// Bound by latency: the index, then its logit.  What does not depend on them is under way before.
template <bool DENSE>
__global__ void __launch_bounds__(32 * kSelectBwdWarps) select_bwd_kernel(const __grid_constant__ SelectBwdParams p) {
  __shared__ float4 s_up[kSelectBwdWarps][kMaxE / 4];
  constexpr int kVec = kMaxE / 128;
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
      if (p.dw) {
        dw = p.dw[r];
      } else {
        const int pos = p.inv_pos[r];
        if (pos >= 0)
          for (int n = 0; n < p.ldp; ++n) dw += p.partial[(int64_t)pos * p.ldp + n];
      }
    }
    float4 x[kVec], q[DENSE ? kVec : 1];  // aux; logits
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = lane + 32 * i;
      x[i] = p.aux && v < nvec ? reinterpret_cast<const float4*>(p.aux + t * p.E)[v] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if constexpr (DENSE)
        q[i] = v < nvec ? reinterpret_cast<const float4*>(row)[v] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
    if (lane < p.k) {
      if (e < 0 || e >= p.E) {
        record_status(p.status, MOK_ERR_DEVICE_CHECK);
        e = -1;
      } else {
        l = row[e];
      }
    }
    const bool on = l > kShutOff;  // not NaN either
    float top = -INFINITY, sum = 1.0f, g = 0.0f, inner = 0.0f;
    if constexpr (DENSE) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) top = fmaxf(fmaxf(fmaxf(top, q[i].x), fmaxf(q[i].y, q[i].z)), q[i].w);  // fmaxf passes NaN by
      top = warp_max(top);
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        for (float a : {q[i].x, q[i].y, q[i].z, q[i].w}) sum += a > kShutOff ? expf(below(a, top)) : 0.0f;
      sum = warp_sum(sum);
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
    const int end = p.dl ? p.ldl / 4 : nvec;  // at most 128
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = lane + 32 * i;
      if (v >= end) break;
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (v < nvec) {
        a = s_up[warp][v];
        if constexpr (DENSE) {
          auto grad = [&](float l, float d) { return l > kShutOff ? p.scale * (expf(below(l, top)) / sum) * (d - inner) : 0.0f; };
          a = make_float4(grad(q[i].x, a.x), grad(q[i].y, a.y), grad(q[i].z, a.z), grad(q[i].w, a.w));
        }
        a.x += x[i].x; a.y += x[i].y; a.z += x[i].z; a.w += x[i].w;
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
  auto k = p.softmax && !p.renorm ? select_bwd_kernel<true> : select_bwd_kernel<false>;
  k<<<(int)std::min<int64_t>(blocks, (int64_t)num_sms() * 8), 32 * kSelectBwdWarps, 0, s>>>(p);
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
                 sel->topk_groups, dims->E / sel->n_groups, 1, 0, 0,
                 sel->group_score == MOK_GROUP_TOP2, sel->renormalise != 0, sel->scale};
  while (2 * p.lanes * p.groups <= 32) {
    p.lanes *= 2;
    ++p.log_lanes;
  }
  p.chunk = (p.n + p.lanes - 1) / p.lanes;  // at most 30: E <= 512
  const bool vec = p.n % 4 == 0;
  if (vec) p.chunk = (p.chunk + 3) / 4 * 4;
  void (*k)(const SelectParams) = nullptr;
  auto pick = [&](auto softmax, auto bias) {
    constexpr bool S = decltype(softmax)::value, B = decltype(bias)::value;
    k = !vec ? select_kernel<32, false, S, B> : p.chunk <= 8 ? select_kernel<8, true, S, B> : p.chunk <= 12 ? select_kernel<12, true, S, B>
        : p.chunk <= 16 ? select_kernel<16, true, S, B> : select_kernel<32, true, S, B>;
  };
  if (sel->score == MOK_SCORE_SOFTMAX && sel_bias) pick(std::true_type{}, std::true_type{});
  else if (sel->score == MOK_SCORE_SOFTMAX) pick(std::true_type{}, std::false_type{});
  else if (sel_bias) pick(std::false_type{}, std::true_type{});
  else pick(std::false_type{}, std::false_type{});
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

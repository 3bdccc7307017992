// Expert router for gfx950: logits [T, E] -> the top-k experts of every token
// and their weights.
//
// ("DeepSeek-V4 W8A8 执行链从量化权重到 Ascend INT8 算子", §三: the expert runner
// is handed topk_ids and topk_weights; the router that makes them is not on the
// page, the definition below is this library's.)
//
//   score_e = 1 / (1 + exp(-l_e)), or exp(l_e - max l) / sum exp(l - max l)
//   key_e   = score_e + bias_e
//   An expert whose logit is NaN or -inf, or whose key is NaN or -inf, is out;
//   a logit of +inf counts as the largest float. With groups of E / n_group
//   consecutive experts, a group's mark is the sum of its two largest keys (the
//   key if only one is in, out if none is); the topk_group groups of largest
//   mark stay, lowest index first among equals. The top_k experts of largest
//   key, lowest index first among equals, are the result, in that order; slots
//   that no expert fills get id -1 and weight 0. weight = score, divided by the
//   sum of the k where asked (0 where that sum is 0), times a factor.
//
// Which of two close keys is larger decides an expert: the result is that of
// doubles (gate_exact), found with floats wherever they can tell (gate_fast).
#include <hip/hip_fp16.h>

#include "device_common.hpp"
#include "dpp_row.hpp"
#include "fp8b.hpp"
#include "launch.hpp"

namespace w8a8 {

constexpr double kOut = -__builtin_huge_val();  // key of an expert that is out

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (DT == 0) return reinterpret_cast<const float*>(p)[i];
  if (DT == 1) return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
  return __half2float(reinterpret_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ double shfl_xor_d(double v, int m) { return __shfl_xor(v, m, kWave); }

// v of another lane by DPP; lanes of rows outside ROWS keep their own
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const int lo = (int)(uint32_t)u, hi = (int)(uint32_t)(u >> 32);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xF, false);
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
}

__device__ __forceinline__ double readlane_d(double v, int l) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), l);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// maximum and sum over the wavefront, in every lane
__device__ __forceinline__ double wave_max_d(double v) {
  v = fmax(v, dpp_d<0xB1>(v));
  v = fmax(v, dpp_d<0x4E>(v));
  v = fmax(v, dpp_d<0x141>(v));
  v = fmax(v, dpp_d<0x140>(v));
  v = fmax(v, dpp_d<0x142, 0xA>(v));  // the ends of rows 0 and 2 into rows 1 and 3
  v = fmax(v, dpp_d<0x143, 0xC>(v));  // and of the first half into the second
  return readlane_d(v, 63);
}

__device__ __forceinline__ double wave_sum_d(double v) {
  v += dpp_d<0xB1>(v);
  v += dpp_d<0x4E>(v);
  v += dpp_d<0x141>(v);
  v += dpp_d<0x140>(v);
  return (readlane_d(v, 0) + readlane_d(v, 16)) + (readlane_d(v, 32) + readlane_d(v, 48));
}

__device__ __forceinline__ void merge2_d(double& a, double& b, double oa, double ob) {
  b = fmax(fmin(a, oa), fmax(b, ob));
  a = fmax(a, oa);
}

// The definition itself, in doubles, by one wavefront; lane l holds the experts
// P l + i. Every lane of the wavefront takes part. A launch lasts as long as its
// slowest wavefront and this code is cold when it runs, so it has no LDS latency in
// its loops and one copy of the exponential (unrolled and with shuffles, one such
// token added 10 us to a launch).
template <int DT, int P>
__device__ void gate_exact(const GateArgs& g, int64_t t, int lane) {
  const int E = g.E, e0 = lane * P;
  float l[P];
  bool in[P];
  double top = kOut;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    l[i] = e0 + i < E ? load_logit<DT>(g.logits, t * g.ld + e0 + i) : -__builtin_huge_valf();
    in[i] = l[i] > -__builtin_huge_valf();  // false for NaN
    l[i] = fminf(l[i], 3.402823466e38f);
    if (in[i]) top = fmax(top, (double)l[i]);
  }
  double score[P], key[P];
  const bool sigmoid = g.scoring == 1;
  if (!sigmoid) top = wave_max_d(top);
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) score[i] = 0.0;
#pragma nounroll
  for (int n = 0; n < P; ++n) {  // one copy of the exponential's code
    float x = l[0];
    bool ok = in[0];
#pragma unroll
    for (int i = 1; i < P; ++i) {
      x = n == i ? l[i] : x;
      ok = n == i ? in[i] : ok;
    }
    double v = exp(sigmoid ? -(double)x : (double)x - top);
    if (sigmoid) v = 1.0 / (1.0 + v);
    v = ok ? v : 0.0;
    sum += v;
#pragma unroll
    for (int i = 0; i < P; ++i) score[i] = n == i ? v : score[i];
  }
  if (!sigmoid) {
    sum = wave_sum_d(sum);
#pragma unroll
    for (int i = 0; i < P; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double k = g.bias && in[i] ? score[i] + (double)g.bias[e0 + i] : score[i];
    key[i] = in[i] && k > kOut ? k : kOut;
  }
  if (g.n_group > 1) {
    const int per = E / g.n_group;
    double mark = kOut;  // lane h: the mark of group h
    for (int h = 0; h < g.n_group; ++h) {
      double a = kOut, b = kOut;  // the group's two largest keys
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = e0 + i;
        if (e >= h * per && e < (h + 1) * per) {
          b = fmax(b, fmin(a, key[i]));
          a = fmax(a, key[i]);
        }
      }
      merge2_d(a, b, dpp_d<0xB1>(a), dpp_d<0xB1>(b));
      merge2_d(a, b, dpp_d<0x4E>(a), dpp_d<0x4E>(b));
      merge2_d(a, b, dpp_d<0x141>(a), dpp_d<0x141>(b));
      merge2_d(a, b, dpp_d<0x140>(a), dpp_d<0x140>(b));
      double x = readlane_d(a, 0), y = readlane_d(b, 0);  // the four rows of 16 lanes
#pragma unroll
      for (int q = 16; q < kWave; q += 16) merge2_d(x, y, readlane_d(a, q), readlane_d(b, q));
      if (lane == h) mark = y > kOut ? x + y : x;
    }
    int rank = 0;
    for (int h = 0; h < g.n_group; ++h) {
      const double o = readlane_d(mark, h);
      rank += o > mark || (o == mark && h < lane);
    }
    const uint64_t stays = __ballot(lane < g.n_group && rank < g.topk_group);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e0 + i < E && !((stays >> ((e0 + i) / per)) & 1)) key[i] = kOut;
  }
  int id = -1;        // lane j: the j-th expert
  double w = 0.0;
  double total = 0.0;
  for (int j = 0; j < g.top_k; ++j) {
    double m = key[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = fmax(m, key[i]);
    const double best = wave_max_d(m);
    if (!(best > kOut)) break;  // uniform: nothing is left
    int at = P - 1;  // this lane's lowest index of its maximum, and that one's score
    double s = score[P - 1];
#pragma unroll
    for (int i = P - 2; i >= 0; --i) {
      at = key[i] == m ? i : at;
      s = key[i] == m ? score[i] : s;
    }
    const int owner = __builtin_ctzll(__ballot(m == best));
    const int e = owner * P + __builtin_amdgcn_readlane(at, owner);
    const double bs = readlane_d(s, owner);
    at = lane == owner ? at : -1;
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = at == i ? kOut : key[i];
    if (lane == j) { id = e; w = bs; }
    total += bs;
  }
  if (lane < g.top_k) {
    if (g.renormalize) w = total > 0.0 ? w / total : 0.0;
    g.ids[t * g.top_k + lane] = id;
    g.weights[t * g.top_k + lane] = (float)(w * (double)g.scale);
  }
}

// ---------------------------------------------------------------------------
// Fast form: one wavefront per token, lane l holds the P consecutive experts
// P l + i, keys are floats. Where float rounding could change the choice the
// wavefront falls back to gate_exact: it does so if two keys that have to be told
// apart (neighbours among the k + 1 largest, unless equal logits and biases place
// them both inside the list; the last group that stays and the first that goes) are
// within 2^-20 or 2^-19 times (1 + |a| + |b|). With d the exponential's relative error, (1 + |x|) 2^-23 at most
// (one ulp, and the rounded argument):
// - a sigmoid is off by s (1 - s) d <= 0.48 2^-23, a rounding of 1 + e and an ulp of
//   the reciprocal, together less than 2^-22; keys by 2^-24 |key| more and marks
//   by twice that. Two of either are compared with 2^-20 (1 + |a| + |b|);
// - a softmax by s d <= 2^-23 and an ulp of the division, and all scores of a token
//   by the error of their sum, at most 2^-23 times 2.4 / s (its terms' d; s the
//   largest score) + 5 (its roundings, a tree of 10). Two sums of two scores
//   differ by less than 2^-19 for that; compared with 2^-19 (1 + |a| + |b|).
// What only two candidates decide is settled in place (sigmoid scores with a bias):
// two groups at the border by their marks in doubles, close neighbours among the
// selected and the runner-up by the doubles that their weights need anyway. What is
// left, a third group or a chain of close keys that leaves the list, falls back
// (a launch lasts as long as its slowest wavefront: with every close choice left to
// gate_exact, 2048 tokens took 15.8 us in a graph instead of 7.1, and 16384 took 5.9 more).
// Without a bias the order of keys is the order of logits, which are compared as
// they are, as far as doubles tell the keys of distinct logits apart (unsure_logit);
// a selected one 700 under the maximum (softmax) or under -700 (sigmoid), where
// doubles run out, falls back, and with a bias a softmax whose selected are all 600 under.
// The weights come from the selected logits alone, in doubles; only the sum of a
// softmax that is not renormalized is a float sum.
// ---------------------------------------------------------------------------
constexpr float kNearSigmoid = 0x1p-20f, kNearSoftmax = 0x1p-19f;

__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// a >= b: whether float rounding could have put two keys or marks in this order (NaN: yes)
__device__ __forceinline__ bool too_close(float a, float b, float near) {
  return !(a - b > near * (1.f + fabsf(a) + fabsf(b)));
}

// Whether doubles may give logit x the key of another logit, so that the lower index
// would win and not the larger logit. Sigmoids: logits d apart have scores at least
// d exp(-x) / 4 apart (x >= 0) or a share of d / 2 (x < 0). Distinct floats of magnitude
// 2^-16 and more are 2^-40 apart and more, from 8 on 2^-20, from 16 on 2^-19, so up to
// x = 20 scores are 2^-50 apart, eight steps of doubles under 1; from 23 on neighbours
// meet. Softmax: l - max, above -700 (below: see there), is rounded by 2^-44 at most,
// and so distinct floats of magnitude 2^-16 and more keep scores that differ by a share
// of 2^-41; those next to 0 may be absorbed.
__device__ __forceinline__ bool unsure_logit(float x, bool sigmoid) {
  return (sigmoid && x > 20.f) || fabsf(x) < 0x1p-16f;
}
// a > b, a unsure: whether doubles tell their keys apart all the same. Sigmoids of a and
// b = a - d differ by exp(-b) (1 - exp(-d)) / 2 at least (by 1/2 for b < 0), and 1 - exp(-d)
// is 3/4 min(d, 1/2) or more: past 2^-50 where the product passes 2^-48, twice what the two
// doubles are off by. 2^-30 next to 0 is 2^-32 in the scores. (Logits of deviation 7, 16384
// x 256, top 8: 9.4 us in a graph; told apart only across 19, 26.7.)
__device__ __forceinline__ bool keys_apart(float a, float b, bool sigmoid) {
  return sigmoid && a > 20.f ? exp_f(-b) * fminf(a - b, 0.5f) > 0x1p-48f : a - b > 0x1p-30f;
}

// Softmax scores run out of doubles under e^-708 of the maximum's. Where the selected
// are all at most e^-600 (chosen by the bias) their sum may be 0, and then so are the
// weights, or hold few bits of those 103 under the largest, which floats still have.
__device__ __forceinline__ bool scores_vanish(float largest, float top) { return largest - top < -600.f; }

// order-preserving map of finite floats and +inf to integers above 0 (0: out)
__device__ __forceinline__ uint32_t key_bits(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);  // -0 becomes +0: equal keys have equal bits
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ void merge2(float& a, float& b, float oa, float ob) {
  b = fmaxf(fminf(a, oa), fmaxf(b, ob));
  a = fmaxf(a, oa);
}

// the two largest of `seg` consecutive lanes (aligned, a power of two), in all of them
__device__ __forceinline__ void segment_top2(float& a, float& b, int seg) {
  if (seg >= 2) merge2(a, b, dpp_f<0xB1>(a), dpp_f<0xB1>(b));    // lanes l ^ 1
  if (seg >= 4) merge2(a, b, dpp_f<0x4E>(a), dpp_f<0x4E>(b));    // l ^ 2
  if (seg >= 8) merge2(a, b, dpp_f<0x141>(a), dpp_f<0x141>(b));  // the other quad of 8
  if (seg >= 16) merge2(a, b, dpp_f<0x140>(a), dpp_f<0x140>(b)); // the other half of 16
  if (seg >= 32) merge2(a, b, __shfl_xor(a, 16, kWave), __shfl_xor(b, 16, kWave));
  if (seg >= 64) merge2(a, b, __shfl_xor(a, 32, kWave), __shfl_xor(b, 32, kWave));
}

// A group's mark from its two largest keys: their sum, the one that is in, or out. Lost:
// both are in and the sum is below the floats; it then stands with the groups that are out.
// Which of those stay takes doubles, unless only marks clear of that range do.
__device__ __forceinline__ bool mark_lost(float mark, float b) {
  return b > -__builtin_huge_valf() && mark == -__builtin_huge_valf();
}
__device__ __forceinline__ bool mark_clear(float last_that_stays) { return last_that_stays > -1e38f; }

// sum of P floats (a power of two) with log2 P roundings
template <int P>
__device__ __forceinline__ float tree_sum(const float (&v)[P]) {
  float t[P];
#pragma unroll
  for (int i = 0; i < P; ++i) t[i] = v[i];
#pragma unroll
  for (int h = P / 2; h > 0; h >>= 1) {
#pragma unroll
    for (int i = 0; i < h; ++i) t[i] += t[i + h];
  }
  return t[0];
}

__device__ __forceinline__ float wave_sum_f(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  v += dpp_f<0x140>(v);
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

__device__ __forceinline__ float readlane_f(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// wave_max_u32 with one readlane: the DPP broadcasts of row ends carry the
// maximum to lane 63 (the scalar unit, shared by the CU's SIMDs, is what four
// readlanes and their maxima ran out of)
__device__ __forceinline__ uint32_t wave_max_last(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));  // row_bcast15 into rows 1, 3
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));  // row_bcast31 into rows 2, 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// the largest of the lanes' keys as a float; 0 if none is in
__device__ __forceinline__ float wave_top(uint32_t kb) {
  const uint32_t m = wave_max_u32(kb);
  return m ? key_value(m) : 0.f;
}

// logits of experts P lane .. P lane + P - 1 of token t (0 past the last)
template <int DT, int P>
__device__ __forceinline__ void load_logits(const GateArgs& g, int64_t t, int lane, float (&l)[P]) {
  const int e0 = lane * P;
  const int64_t at = t * g.ld + e0;
  if (P >= 4 && DT == 0 && g.vec) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      float4 v = {0.f, 0.f, 0.f, 0.f};
      if (e0 + i < g.E) v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(g.logits) + at + i);
      l[i] = v.x; l[i + 1] = v.y; l[i + 2] = v.z; l[i + 3] = v.w;
    }
  } else if (P >= 4 && DT != 0 && g.vec) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      uint2 v = {0u, 0u};
      if (e0 + i < g.E) v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(g.logits) + at + i);
      const uint32_t h[4] = {v.x & 0xFFFFu, v.x >> 16, v.y & 0xFFFFu, v.y >> 16};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        l[i + j] = DT == 1 ? bf16_to_f32(h[j]) : __half2float(__builtin_bit_cast(__half, (uint16_t)h[j]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = e0 + i < g.E ? load_logit<DT>(g.logits, at + i) : 0.f;
  }
}

// biases of experts e0 .. e0 + P - 1; 0 without one and past the last expert
template <int P>
__device__ __forceinline__ void load_bias(const GateArgs& g, int e0, float (&b)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) b[i] = 0.f;
  if (!g.bias) return;
  if (P >= 4 && g.bias_vec) {
#pragma unroll
    for (int i = 0; i + 4 <= P; i += 4) {
      if (e0 + i < g.E) {
        const float4 v = *reinterpret_cast<const float4*>(g.bias + e0 + i);
        b[i] = v.x; b[i + 1] = v.y; b[i + 2] = v.z; b[i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) b[i] = e0 + i < g.E ? g.bias[e0 + i] : 0.f;
  }
}

// Order of the k + 1 entries of a row of 16 lanes (lane j: expert id of double key
// `key`, weight w) by those keys, lowest index first among equals. The entries fill
// the row from lane 0; others stay where they are. Every lane takes part.
template <int N>
__device__ __forceinline__ void settle_step(int& rank, int id, double key, bool entry) {
  const double ok = dpp_d<0x120 + N>(key);
  const int oid = __builtin_amdgcn_update_dpp(0, id, 0x120 + N, 0xF, 0xF, false);
  const int oe = __builtin_amdgcn_update_dpp(0, (int)entry, 0x120 + N, 0xF, 0xF, false);
  rank += oe && (ok > key || (ok == key && oid < id));
}

__device__ __forceinline__ void settle_row(int& id, double& w, double key, int k, int lane) {
  const bool entry = (lane & 15) <= k && id >= 0;
  int rank = 0;
  settle_step<1>(rank, id, key, entry); settle_step<2>(rank, id, key, entry); settle_step<3>(rank, id, key, entry);
  settle_step<4>(rank, id, key, entry); settle_step<5>(rank, id, key, entry); settle_step<6>(rank, id, key, entry);
  settle_step<7>(rank, id, key, entry); settle_step<8>(rank, id, key, entry); settle_step<9>(rank, id, key, entry);
  settle_step<10>(rank, id, key, entry); settle_step<11>(rank, id, key, entry); settle_step<12>(rank, id, key, entry);
  settle_step<13>(rank, id, key, entry); settle_step<14>(rank, id, key, entry); settle_step<15>(rank, id, key, entry);
  const int to = 4 * (entry ? (lane & 48) + rank : lane);
  const uint64_t u = __builtin_bit_cast(uint64_t, w);
  id = __builtin_amdgcn_ds_permute(to, id);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_permute(to, (int)(uint32_t)u);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_ds_permute(to, (int)(uint32_t)(u >> 32));
  w = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// false: the choice is too close for floats
template <int DT, int P>
__device__ __forceinline__ bool gate_fast(const GateArgs& g, int64_t t, int lane) {
  const int E = g.E, k = g.top_k;
  const bool sigmoid = g.scoring == 1, biased = g.bias != nullptr;
  const float near = sigmoid ? kNearSigmoid : kNearSoftmax;
  float l[P];
  load_logits<DT, P>(g, t, lane, l);
  bool in[P];
  float top = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < P; ++i) {
    in[i] = lane * P + i < E && l[i] > -__builtin_huge_valf();  // false for NaN
    l[i] = fminf(l[i], 3.402823466e38f);
    if (in[i]) top = fmaxf(top, l[i]);
  }
  const bool need_scores = biased || g.n_group > 1 || (!sigmoid && !g.renormalize);
  float s[P];
  float total = 1.f;  // softmax: the sum of the exponentials
  if (need_scores) {
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = in[i] ? __builtin_amdgcn_rcpf(1.f + exp_f(-l[i])) : 0.f;
    } else {
      const uint32_t tb = wave_max_u32(top > -__builtin_huge_valf() ? key_bits(top) : 0u);
      top = tb ? key_value(tb) : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = in[i] ? exp_f(l[i] - top) : 0.f;
      total = wave_sum_f(tree_sum<P>(s));
      const float r = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] *= r;
    }
  }
  float bias[P];
  load_bias<P>(g, lane * P, bias);
  // keys as integers: logits without a bias, else scores + bias
  uint32_t u[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float key = l[i];
    bool ok = in[i];
    if (biased) {
      key = s[i] + bias[i];
      ok = ok && key > -__builtin_huge_valf();
    }
    u[i] = ok ? key_bits(key) : 0u;
  }
  bool close = false;
  if (g.n_group > 1) {
    const int per = E / g.n_group, seg = per / P;
    float a = -__builtin_huge_valf(), b = a;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float v = u[i] ? (biased ? key_value(u[i]) : s[i]) : -__builtin_huge_valf();
      b = fmaxf(b, fminf(a, v));
      a = fmaxf(a, v);
    }
    segment_top2(a, b, seg);
    const float mark = b > -__builtin_huge_valf() ? a + b : a;
    const int mine = lane / seg;
    int rank = 0;
    for (int h = 0; h < g.n_group; ++h) {
      const float o = readlane_f(mark, h * seg);
      rank += o > mark || (o == mark && h < mine);
    }
    const bool group = mine < g.n_group;
    if (g.topk_group < g.n_group) {
      // the last that stays and the first that goes
      const int last = __builtin_ctzll(__ballot(group && rank == g.topk_group - 1));
      const int next = __builtin_ctzll(__ballot(group && rank == g.topk_group));
      const float x = readlane_f(mark, last), y = readlane_f(mark, next);
      if (y > -__builtin_huge_valf()) close = too_close(x, y, near);
      if (close && sigmoid && biased) {  // uniform
        // their marks in doubles, if no third group is close to either
        const uint64_t before = __ballot(group && rank == g.topk_group - 2), past = __ballot(group && rank == g.topk_group + 1);
        const float px = before ? readlane_f(mark, __builtin_ctzll(before)) : 0.f;
        const float py = past ? readlane_f(mark, __builtin_ctzll(past)) : -__builtin_huge_valf();
        const bool pair = !(before && too_close(px, x, near)) && !(py > -__builtin_huge_valf() && too_close(y, py, near));
        if (pair) {  // uniform
          const bool border = group && (rank == g.topk_group - 1 || rank == g.topk_group);
          double first = kOut, second = kOut;
#pragma nounroll
          for (int n = 0; n < P; ++n) {
            uint32_t un = u[0];
            float ln = l[0];
#pragma unroll
            for (int i = 1; i < P; ++i) {
              un = n == i ? u[i] : un;
              ln = n == i ? l[i] : ln;
            }
            // keys that may be among the group's two largest
            const bool cand = border && un && !(key_value(un) < b - near * (1.f + 2.f * fabsf(b)));
            if (!__ballot(cand)) continue;
            const double v = 1.0 / (1.0 + exp(-(double)ln));
            if (cand) merge2_d(first, second, v + (double)g.bias[lane * P + n], kOut);
          }
          for (int d = 1; d < seg; d <<= 1) {
            const double o1 = shfl_xor_d(first, d), o2 = shfl_xor_d(second, d);
            merge2_d(first, second, o1, o2);
          }
          const double dm = second > kOut ? first + second : first;
          const double dx = readlane_d(dm, last), dy = readlane_d(dm, next);
          if (border && (dy > dx || (dy == dx && next < last))) rank = 2 * g.topk_group - 1 - rank;
          close = false;
        }
      }
      if (mark_lost(mark, b) && !mark_clear(x)) close = true;
    }
    if (!(group && rank < g.topk_group)) {
#pragma unroll
      for (int i = 0; i < P; ++i) u[i] = 0u;
    }
  }
  // top k (and the runner-up where keys are rounded): every step takes the
  // largest key of the wavefront, of the lowest lane and index among equals
  int id = -1;          // lane j: the j-th expert
  uint32_t kb = 0u;     // and its key
  // with a bias two more than asked, as far as there are lanes: the runner-up and the
  // one after it
  const int steps = biased ? min(k + 2, kWave) : k;
  for (int j = 0; j < steps; ++j) {
    uint32_t m = u[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = max(m, u[i]);
    const uint32_t best = wave_max_last(m);
    if (best == 0u) break;  // uniform: nothing is left
    int at = P - 1;  // this lane's lowest index of its maximum
#pragma unroll
    for (int i = P - 2; i >= 0; --i) at = u[i] == m ? i : at;
    const int owner = __builtin_ctzll(__ballot(m == best));
    const int e = owner * P + __builtin_amdgcn_readlane(at, owner);
    at = lane == owner ? at : -1;
#pragma unroll
    for (int i = 0; i < P; ++i) u[i] = at == i ? 0u : u[i];
    if (lane == j) {
      id = e;
      kb = best;
    }
  }
  const float sel = id >= 0 ? fminf(load_logit<DT>(g.logits, t * g.ld + id), 3.402823466e38f) : 0.f;
  const float bj = biased && id >= 0 ? g.bias[id] : 0.f;
  bool swap = false;  // lane j: too close to lane j + 1, other than equal inside the list
  if (biased) {
    const float v = key_value(kb);
    const int n = __shfl_down(id, 1, kWave);
    const float nv = __shfl_down(v, 1, kWave), nl = __shfl_down(sel, 1, kWave), nb = __shfl_down(bj, 1, kWave);
    if (lane <= k && lane + 1 < kWave && id >= 0 && n >= 0 && !(lane < k - 1 && nl == sel && nb == bj))
      swap = too_close(v, nv, near);
    if (k > 14 && (lane < k || k == kWave)) close = close || swap || k == kWave;  // past a row of lanes
    if (!sigmoid) {
      if (lane < k) close = close || swap;
      if (g.renormalize && scores_vanish(wave_top(lane < k && id >= 0 ? key_bits(sel) : 0u), top)) close = true;
    }
  } else {
    const float first = need_scores && !sigmoid ? top : readlane_f(sel, 0);
    const bool chosen = lane < k && id >= 0;
    if (chosen) close = close || (sigmoid ? sel < -700.f : sel - first < -700.f);
    const bool unsure = chosen && unsure_logit(sel, sigmoid);
    const uint64_t any = __ballot(unsure);
    if (any) {  // uniform
      const int n = __shfl_down(id, 1, kWave);
      const float nl = __shfl_down(sel, 1, kWave);
      if (unsure && lane < k - 1 && n >= 0 && nl != sel && !keys_apart(sel, nl, sigmoid)) close = true;
      if (any >> (k - 1) & 1) {  // the last of the list against what is left
        const float last = readlane_f(sel, k - 1);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float v = key_value(u[i]);
          if (u[i] && v != last && !keys_apart(last, v, sigmoid)) close = true;
        }
      }
    }
  }
  const uint64_t pairs = __ballot(swap);
  const bool order = biased && sigmoid && k <= 14 && (pairs & ((1ull << k) - 1)) != 0;  // uniform
  // close to the last of the list, which is close to one outside of it
  if (__ballot(close) || (order && (pairs >> (k - 1) & 3) == 3)) return false;
  double w = 0.0;
  if (sigmoid) {
    if (lane <= k && id >= 0) w = 1.0 / (1.0 + exp(-(double)sel));
    if (order) settle_row(id, w, w + (double)bj, k, lane);
    if (!(lane < k && id >= 0)) w = 0.0;
  } else {
    // renormalized: the largest selected logit stands for the maximum
    const bool mine = lane < k && id >= 0;
    const float ref = g.renormalize ? wave_top(mine ? key_bits(sel) : 0u) : top;
    if (mine) w = exp((double)sel - (double)ref);
  }
  if (g.renormalize) {
    double sum = w;
    for (int d = 1; d < k; d <<= 1) sum += shfl_xor_d(sum, d);  // lanes past k hold 0
    w = sum > 0.0 ? w / sum : 0.0;
  } else if (!sigmoid) {
    w = total > 0.f ? w / (double)total : 0.0;
  }
  if (lane < k) {
    g.ids[t * k + lane] = id;
    g.weights[t * k + lane] = (float)(w * (double)g.scale);
  }
  return true;
}

template <int DT, int P>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs g) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= g.T) return;
  if (!g.fast || !gate_fast<DT, P>(g, t, lane)) gate_exact<DT, P>(g, t, lane);  // uniform
}

// ---------------------------------------------------------------------------
// Many tokens: the fast form with four tokens a wavefront, 16 lanes each. Lane s
// of a token holds experts P s .. P s + P - 1 (E <= 16 P), their keys also in LDS, the
// maxima of its runs of four in registers: a step of the selection looks into one
// run of the lane that owns the maximum instead of at every key. Vector
// instructions (1476 a wavefront, 9.8 us at 16384 tokens) and the selection's
// dependent steps bound this kernel: 16384 x 256, sigmoid, 8 groups, bias, top 8
// take 14.2 to 14.5 us in a graph, the logits' bytes 4.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<0xB1>(v);
  v += dpp_f<0x4E>(v);
  v += dpp_f<0x141>(v);
  return v + dpp_f<0x140>(v);
}

__device__ __forceinline__ double row_max_d(double v) {
  v = fmax(v, dpp_d<0xB1>(v));
  v = fmax(v, dpp_d<0x4E>(v));
  v = fmax(v, dpp_d<0x141>(v));
  return fmax(v, dpp_d<0x140>(v));
}

__device__ __forceinline__ double row_sum_d(double v) {
  v += dpp_d<0xB1>(v);
  v += dpp_d<0x4E>(v);
  v += dpp_d<0x141>(v);
  return v + dpp_d<0x140>(v);
}

// rank += "the mark of the lane N to the right in the row is better", N a rotation
template <int N>
__device__ __forceinline__ void rank_step(int& rank, float mark, int group, int seg) {
  if (N % seg == 0) {  // uniform: one lane of every other group
    const float o = dpp_f<0x120 + N>(mark);
    const int og = __builtin_amdgcn_update_dpp(0, group, 0x120 + N, 0xF, 0xF, false);
    rank += o > mark || (o == mark && og < group);
  }
}

constexpr int kQuadWaves = 4;

template <int DT, int P>
__global__ __launch_bounds__(kQuadWaves * 64) void gate_quad_kernel(GateArgs g) {
  constexpr int kRuns = P / 4, kPitch = P + 4;  // keys of a lane in LDS, padded against bank conflicts
  __shared__ __attribute__((aligned(16))) uint32_t keys[kQuadWaves][64 * kPitch];
  const int lane = threadIdx.x & 63, sub = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = ((int64_t)blockIdx.x * kQuadWaves + wave) * 4;
  if (t0 >= g.T) return;
  const bool live = t0 + (lane >> 4) < g.T;
  const int64_t t = live ? t0 + (lane >> 4) : g.T - 1;
  const int E = g.E, k = g.top_k, e0 = sub * P;
  const bool sigmoid = g.scoring == 1, biased = g.bias != nullptr;
  const float near = sigmoid ? kNearSigmoid : kNearSoftmax;
  uint32_t* const mine = keys[wave] + lane * kPitch;

  float l[P];
  load_logits<DT, P>(g, t, sub, l);
  const float low = -__builtin_huge_valf();
  float top = low;
  uint32_t in = 0u;  // bit i: expert e0 + i takes part
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const bool ok = e0 + i < E && l[i] > low;  // false for NaN
    in |= ok ? 1u << i : 0u;
    l[i] = fminf(l[i], 3.402823466e38f);
    if (ok) top = fmaxf(top, l[i]);
  }
  const bool need_scores = biased || g.n_group > 1 || (!sigmoid && !g.renormalize);
  float total = 1.f, r = 1.f;
  if (need_scores && !sigmoid) {
    const uint32_t tb = row_max_u32(top > low ? key_bits(top) : 0u);
    top = tb ? key_value(tb) : 0.f;
    float part[P];
#pragma unroll
    for (int i = 0; i < P; ++i) part[i] = (in >> i) & 1 ? exp_f(l[i] - top) : 0.f;
    total = row_sum(tree_sum<P>(part));
    r = total > 0.f ? 1.f / total : 0.f;
  }
  float bias[P];
  load_bias<P>(g, e0, bias);
  // scores; keys as integers; the lane's two largest values for its group's mark
  uint32_t u[P];
  float a = low, b = low;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float v = l[i], key = l[i];
    bool ok = (in >> i) & 1;
    if (need_scores) v = sigmoid ? __builtin_amdgcn_rcpf(1.f + exp_f(-l[i])) : exp_f(l[i] - top) * r;
    if (biased) {
      v = v + bias[i];
      key = v;
      ok = ok && key > low;
    }
    u[i] = ok ? key_bits(key) : 0u;
    v = ok ? v : low;
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
  }
  bool close = false;
  if (g.n_group > 1) {
    const int seg = E / g.n_group / P;  // lanes of a group
    segment_top2(a, b, seg);
    const float mark = b > low ? a + b : a;
    const int group = sub / seg;
    int rank = 0;
    rank_step<1>(rank, mark, group, seg); rank_step<2>(rank, mark, group, seg); rank_step<3>(rank, mark, group, seg);
    rank_step<4>(rank, mark, group, seg); rank_step<5>(rank, mark, group, seg); rank_step<6>(rank, mark, group, seg);
    rank_step<7>(rank, mark, group, seg); rank_step<8>(rank, mark, group, seg); rank_step<9>(rank, mark, group, seg);
    rank_step<10>(rank, mark, group, seg); rank_step<11>(rank, mark, group, seg); rank_step<12>(rank, mark, group, seg);
    rank_step<13>(rank, mark, group, seg); rank_step<14>(rank, mark, group, seg); rank_step<15>(rank, mark, group, seg);
    const bool real = group < g.n_group;
    if (g.topk_group < g.n_group) {
      // the last group that stays and the first that goes
      const uint32_t xb = row_max_u32(real && rank == g.topk_group - 1 && mark > low ? key_bits(mark) : 0u);
      const uint32_t yb = row_max_u32(real && rank == g.topk_group && mark > low ? key_bits(mark) : 0u);
      const float x = key_value(xb), y = key_value(yb);
      if (yb) close = too_close(x, y, near);
      if (sigmoid && biased && __ballot(close)) {  // uniform
        // their marks in doubles, if no third group is close to either
        const uint32_t pb = row_max_u32(real && rank == g.topk_group - 2 && mark > low ? key_bits(mark) : 0u);
        const uint32_t nb = row_max_u32(real && rank == g.topk_group + 1 && mark > low ? key_bits(mark) : 0u);
        const float prev = key_value(pb), next = key_value(nb);
        const bool pair = close && !(pb && too_close(prev, x, near)) && !(nb && too_close(y, next, near));
        const bool border = pair && real && (rank == g.topk_group - 1 || rank == g.topk_group);
        // the keys that may be among the group's two largest
        const float from = b - near * (1.f + 2.f * fabsf(b));
        uint32_t cand = 0u;
#pragma unroll
        for (int i = 0; i < P; ++i) cand |= border && u[i] && !(key_value(u[i]) < from) ? 1u << i : 0u;
        double first = kOut, second = kOut;
        while (__ballot(cand != 0u)) {
          const int n = cand ? __builtin_ctz(cand) : 0;
          float x1 = l[0];
#pragma unroll
          for (int i = 1; i < P; ++i) x1 = n == i ? l[i] : x1;
          double v = 1.0 / (1.0 + exp(-(double)x1));
          if (cand) merge2_d(first, second, v + (double)g.bias[e0 + n], kOut);
          cand &= cand - 1u;  // 0 stays 0
        }
        for (int d = 1; d < seg; d <<= 1) {
          const double o1 = shfl_xor_d(first, d), o2 = shfl_xor_d(second, d);
          merge2_d(first, second, o1, o2);
        }
        const double dm = second > kOut ? first + second : first;
        const double dx = row_max_d(border && rank == g.topk_group - 1 ? dm : kOut);
        const double dy = row_max_d(border && rank == g.topk_group ? dm : kOut);
        const uint32_t gx = row_max_u32(border && rank == g.topk_group - 1 ? (uint32_t)group : 0u);
        const uint32_t gy = row_max_u32(border && rank == g.topk_group ? (uint32_t)group : 0u);
        if (border && (dy > dx || (dy == dx && gy < gx))) rank = 2 * g.topk_group - 1 - rank;
        close = close && !pair;
      }
      if (mark_lost(mark, b) && !mark_clear(x)) close = true;  // x NaN: fewer marks than groups that stay
    }
    const bool stays = real && rank < g.topk_group;
#pragma unroll
    for (int i = 0; i < P; ++i) u[i] = stays ? u[i] : 0u;
  }
  uint32_t run[kRuns];  // maxima of four
#pragma unroll
  for (int q = 0; q < kRuns; ++q) {
    *reinterpret_cast<uint4*>(mine + 4 * q) = uint4{u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]};
    run[q] = max(max(u[4 * q], u[4 * q + 1]), max(u[4 * q + 2], u[4 * q + 3]));
  }
  int id = -1;       // lane j of a token: its j-th expert
  uint32_t kb = 0u;  // and that one's key
  const int steps = biased ? k + 2 : k;  // at most 16: the runner-up and the one after it
  for (int j = 0; j < steps; ++j) {
    uint32_t m = run[0];
#pragma unroll
    for (int q = 1; q < kRuns; ++q) m = max(m, run[q]);
    const uint32_t best = row_max_u32(m);
    const uint32_t same = (uint32_t)(__ballot(m == best) >> (lane & 48)) & 0xFFFFu;
    const int owner = __builtin_ctz(same);
    int q = kRuns - 1;
#pragma unroll
    for (int i = kRuns - 2; i >= 0; --i) q = run[i] == m ? i : q;
    const uint4 v = *reinterpret_cast<const uint4*>(mine + 4 * q);
    const int i = v.x == m ? 0 : v.y == m ? 1 : v.z == m ? 2 : 3;
    const int e = __shfl(e0 + 4 * q + i, (lane & 48) | owner, kWave);
    if (sub == j && best != 0u) {
      id = e;
      kb = best;
    }
    if (sub == owner && best != 0u) {
      mine[4 * q + i] = 0u;
      const uint32_t left = max(max(i == 0 ? 0u : v.x, i == 1 ? 0u : v.y), max(i == 2 ? 0u : v.z, i == 3 ? 0u : v.w));
#pragma unroll
      for (int n = 0; n < kRuns; ++n) run[n] = n == q ? left : run[n];
    }
  }
  const float sel = id >= 0 ? fminf(load_logit<DT>(g.logits, t * g.ld + id), 3.402823466e38f) : 0.f;
  const float bj = biased && id >= 0 ? g.bias[id] : 0.f;
  const bool chosen = sub < k && id >= 0;
  bool swap = false;  // lane j: too close to lane j + 1 of the token, other than equal inside the list
  if (biased) {
    const float v = key_value(kb);
    const int n = __shfl_down(id, 1, 16);
    const float nv = __shfl_down(v, 1, 16), nl = __shfl_down(sel, 1, 16), nb = __shfl_down(bj, 1, 16);
    if (sub <= k && id >= 0 && n >= 0 && !(sub < k - 1 && nl == sel && nb == bj))
      swap = too_close(v, nv, near);
    if (!sigmoid && sub < k) close = close || swap;
  } else {
    const float first = need_scores && !sigmoid ? top : __shfl(sel, lane & 48, kWave);
    if (chosen) close = close || (sigmoid ? sel < -700.f : sel - first < -700.f);
    const bool unsure = chosen && unsure_logit(sel, sigmoid);
    const uint64_t any = __ballot(unsure);
    if (any) {  // uniform
      const int n = __shfl_down(id, 1, 16);
      const float nl = __shfl_down(sel, 1, 16);
      if (unsure && sub < k - 1 && n >= 0 && nl != sel && !keys_apart(sel, nl, sigmoid)) close = true;
      // the last of the list against what is left of the token
      const float last = __shfl(sel, (lane & 48) + k - 1, kWave);
      if (any >> ((lane & 48) + k - 1) & 1) {
        for (int i = 0; i < P; ++i) {
          const uint32_t left = mine[i];
          const float v = key_value(left);
          if (left && v != last && !keys_apart(last, v, sigmoid)) close = true;
        }
      }
    }
  }
  const uint64_t all = __ballot(swap);
  if (sigmoid && biased) {
    // close to the last of the list, which is close to one outside of it
    const uint32_t pairs = (uint32_t)(all >> (lane & 48)) & 0xFFFFu;
    close = close || (pairs >> (k - 1) & 3) == 3;
  }
  double w = 0.0;
  if (sigmoid) {
    if (sub <= k && id >= 0) w = 1.0 / (1.0 + exp(-(double)sel));
    if (biased && all) settle_row(id, w, w + (double)bj, k, lane);  // uniform
    if (!(sub < k && id >= 0)) w = 0.0;
  } else {
    const uint32_t tb = row_max_u32(chosen ? key_bits(sel) : 0u);
    const float ref = g.renormalize ? (tb ? key_value(tb) : 0.f) : top;
    if (biased && scores_vanish(ref, top)) close = true;
    if (chosen) w = exp((double)sel - (double)ref);
  }
  if (g.renormalize) {
    const double sum = row_sum_d(w);
    w = sum > 0.0 ? w / sum : 0.0;
  } else if (!sigmoid) {
    w = total > 0.f ? w / (double)total : 0.0;
  }
  const uint64_t again = __ballot(close && live);
  if (live && sub < k && ((again >> (lane & 48)) & 0xFFFFu) == 0u) {
    g.ids[t * k + sub] = id;
    g.weights[t * k + sub] = (float)(w * (double)g.scale);
  }
  // tokens too close for floats, one after the other (uniform)
  for (int q = 0; q < 4; ++q)
    if ((again >> (16 * q)) & 0xFFFFu) gate_exact<DT, (P * 16 + 63) / 64>(g, t0 + q, lane);
}

// From about here on (five wavefronts a SIMD) four tokens a wavefront beat one; us a
// call in a graph, 256 experts, one / four:
//                             sigmoid, 8 groups, bias, top 8   softmax, bf16, top 8
//                   1024 tokens    6.7 /  9.1                   4.5 / 6.0
//                   4096           8.4 /  9.5                   6.0 / 6.1
//                   5120          10.0 / 10.5                   6.7 / 6.7
//                   8192          13.0 / 10.6                   8.8 / 6.7
//                  16384          22.3 / 14.5                  14.6 / 8.8
constexpr int64_t kQuadTokens = 5120;

template <int DT>
static hipError_t launch_gate_dt(const GateArgs& args, hipStream_t stream) {
  GateArgs p = args;
  const int P = p.E <= 64 ? 1 : p.E <= 128 ? 2 : p.E <= 256 ? 4 : p.E <= 512 ? 8 : 16;
  const int per = p.E / p.n_group, seg = per / P;
  // groups have to be whole aligned runs of a power of two of lanes
  p.fast = p.n_group == 1 || (per % P == 0 && (seg & (seg - 1)) == 0);
  p.bias_vec = p.E % 4 == 0 && ((uintptr_t)p.bias & 15) == 0;
  p.vec = p.E % 4 == 0 && p.ld % 4 == 0 && ((uintptr_t)p.logits & (DT == 0 ? 15 : 7)) == 0;
  const int Q = p.E <= 64 ? 4 : p.E <= 128 ? 8 : 16, qseg = per / Q;
  if (p.T >= kQuadTokens && p.E <= 256 && p.top_k + (p.bias ? 2 : 0) <= 16 &&
      (p.n_group == 1 || (per % Q == 0 && (qseg & (qseg - 1)) == 0))) {
    auto fn = Q == 4 ? gate_quad_kernel<DT, 4> : Q == 8 ? gate_quad_kernel<DT, 8> : gate_quad_kernel<DT, 16>;
    hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(p.T, 4 * kQuadWaves)), dim3(kQuadWaves * 64), 0, stream, p);
    return hipGetLastError();
  }
  void (*fn)(GateArgs) = P == 1 ? gate_kernel<DT, 1> : P == 2 ? gate_kernel<DT, 2> : P == 4 ? gate_kernel<DT, 4>
                       : P == 8 ? gate_kernel<DT, 8> : gate_kernel<DT, 16>;
  hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(p.T, 4)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gate(const GateArgs& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  return p.dtype == 0 ? launch_gate_dt<0>(p, stream) : p.dtype == 1 ? launch_gate_dt<1>(p, stream)
                                                                    : launch_gate_dt<2>(p, stream);
}

}  // namespace w8a8

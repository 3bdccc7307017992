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
// Which of two close keys is larger decides an expert, so scores and keys are
// doubles here and the weights are rounded once.
#include <hip/hip_fp16.h>

#include "device_common.hpp"
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

// One wavefront per token; lane l holds experts l + 64 i.
template <int DT, int P>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs g) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= g.T) return;
  const int E = g.E;
  float l[P];
  bool in[P];
  float top = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < E ? load_logit<DT>(g.logits, t * g.ld + e) : -__builtin_huge_valf();
    in[i] = l[i] > -__builtin_huge_valf();  // false for NaN
    l[i] = fminf(l[i], 3.402823466e38f);
    if (in[i]) top = fmaxf(top, l[i]);
  }
  double score[P], key[P];
  if (g.scoring == 1) {
#pragma unroll
    for (int i = 0; i < P; ++i) score[i] = in[i] ? 1.0 / (1.0 + exp(-(double)l[i])) : 0.0;
  } else {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      score[i] = in[i] ? exp((double)l[i] - (double)top) : 0.0;
      sum += score[i];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += shfl_xor_d(sum, d);
#pragma unroll
    for (int i = 0; i < P; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double k = g.bias && in[i] ? score[i] + (double)g.bias[lane + 64 * i] : score[i];
    key[i] = in[i] && k > kOut ? k : kOut;
  }
  if (g.n_group > 1) {
    const int per = E / g.n_group;
    double mark = kOut;  // lane h: the mark of group h
    for (int h = 0; h < g.n_group; ++h) {
      double a = kOut, b = kOut;  // the group's two largest keys
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int e = lane + 64 * i;
        if (e >= h * per && e < (h + 1) * per) {
          b = fmax(b, fmin(a, key[i]));
          a = fmax(a, key[i]);
        }
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double oa = shfl_xor_d(a, d), ob = shfl_xor_d(b, d);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (lane == h) mark = b > kOut ? a + b : a;
    }
    int rank = 0;
    for (int h = 0; h < g.n_group; ++h) {
      const double o = __shfl(mark, h, kWave);
      rank += o > mark || (o == mark && h < lane);
    }
    const uint64_t stays = __ballot(lane < g.n_group && rank < g.topk_group);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((stays >> (e / per)) & 1)) key[i] = kOut;
    }
  }
  int id = -1;        // lane j: the j-th expert
  double w = 0.0;
  double total = 0.0;
  for (int j = 0; j < g.top_k; ++j) {
    double best = kOut;
    int be = 1 << 30;
    double bs = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (key[i] > best) { best = key[i]; be = lane + 64 * i; bs = score[i]; }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double ok = shfl_xor_d(best, d), os = shfl_xor_d(bs, d);
      const int oe = __shfl_xor(be, d, kWave);
      if (ok > best || (ok == best && oe < be)) { best = ok; be = oe; bs = os; }
    }
    if (!(best > kOut)) break;  // uniform: nothing is left
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (be == lane + 64 * i) key[i] = kOut;
    if (lane == j) { id = be; w = bs; }
    total += bs;
  }
  if (lane < g.top_k) {
    if (g.renormalize) w = total > 0.0 ? w / total : 0.0;
    g.ids[t * g.top_k + lane] = id;
    g.weights[t * g.top_k + lane] = (float)(w * (double)g.scale);
  }
}

template <int DT>
static hipError_t launch_gate_dt(const GateArgs& p, hipStream_t stream) {
  void (*fn)(GateArgs) = p.E <= 64 ? gate_kernel<DT, 1> : p.E <= 128 ? gate_kernel<DT, 2> : p.E <= 256 ? gate_kernel<DT, 4>
                       : p.E <= 512 ? gate_kernel<DT, 8> : gate_kernel<DT, 16>;
  hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(p.T, 4)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gate(const GateArgs& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  return p.dtype == 0 ? launch_gate_dt<0>(p, stream) : p.dtype == 1 ? launch_gate_dt<1>(p, stream)
                                                                    : launch_gate_dt<2>(p, stream);
}

}  // namespace w8a8

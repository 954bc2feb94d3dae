// route.cuh - expert routing in its general form, one warp per token.
//
//   s_e = softmax(l)_e over the live experts, or sigmoid(l_e)
//   c_e = fp32(s_e) + bias_e                           (what the choice goes by)
//   group score = c of the group's best live expert, or the sum of its two best
//   keep the topk_group best groups, pick k experts of them by c
//   w_j = s_j / sum of the picked s (renormalize) or s_j, times the scaling factor
//
// Scores are evaluated in double and rounded to fp32 once: the choice between
// two neighbours then depends on one rounding of a value that any machine
// reproduces to far below it, and never on the order of a sum. The weights are
// taken from the unrounded scores and rounded once at the end.
//
// An expert is dead for a token when its mask is 0, its logit is NaN or -inf,
// or its c is NaN or -inf (a bias of -inf switches an expert off). Dead
// experts are picked last, lowest index first, with weight 0: a row always
// gets k distinct experts, so that the slots of the layer's sort and the
// arrival counts of its stage 2 stay complete whatever the mask leaves.
//
// What bounds it: latency and instruction issue, not bytes (a 256-expert fp32
// row is 1 KB). The chain is load -> double exp -> (max, sum) -> group choice ->
// k rounds of arg-max. The rounds are kept short: c is mapped to an unsigned key
// with the same order and one round is a redux.max of the key and a redux.min
// of the index among the lanes that hold it, with each lane's best key kept
// between rounds. The exponential is the library's; its sum and quotient use a
// reciprocal by Newton's iteration, which needs no special cases for a divisor
// in [1, 512]. The scores of a softmax stay in shared memory for the weights.
// Measured: 32 tokens of 128 experts 3.4 us, 4096 of 256 in 8 groups 11.1 us (2000
// instructions a token at 68 % of the issue rate; with the exponential in fp32,
// 9.8 us).
#pragma once
#include "ptx_ext.cuh"
#include "router.cuh"

namespace moe {

// 1 / d for d in [1, 512]: two Newton steps from the single-precision
// reciprocal, 2^-23 -> 2^-46 -> the double's last place or two.
__device__ __forceinline__ double route_rcp(double d) {
  double y = static_cast<double>(__frcp_rn(static_cast<float>(d)));
  y = fma(y, fma(-d, y, 1.0), y);
  return fma(y, fma(-d, y, 1.0), y);
}

// sigmoid(l) = 1 / (1 + a) or a / (1 + a) with a = exp(-|l|) in (0, 1]
__device__ __forceinline__ double route_sigmoid(float l) {
  const double a = exp(-fabs(static_cast<double>(l)));
  const double r = route_rcp(1.0 + a);
  return l < 0.f ? a * r : r;
}

// Lanes that share a group in the group choice: 32 / (n_group rounded up to a
// power of two); the group's values lie `stride` words apart in shared memory,
// with stride % 32 == lanes so that the 32 lanes read 32 banks.
struct RouteGroups {
  int size, lanes, stride;
  uint32_t magic;  // expert e is in group e * magic >> 20: exact for e < 512, since magic exceeds 2^20 / size by
                   // less than 1 and e / 2^20 stays below 1 / size, the least distance to the next quotient
  RouteGroups() = default;
  __host__ RouteGroups(int E, int n_group) {
    int p = 1;
    while (p < n_group) p *= 2;
    size = E / n_group;
    lanes = 32 / p;
    stride = size + ((lanes - size) % 32 + 32) % 32;
    magic = ((1u << 20) + size - 1) / size;
  }
  __host__ __device__ int words(int n_group) const { return n_group * stride; }
};

struct RouteArgs {
  const void* logits;  // [T, E], rows ld apart
  size_t ld;
  int dtype;                 // MOE_DT_F32, MOE_DT_BF16 or MOE_DT_FP16
  const float* bias;         // [E] or nullptr
  const uint8_t* mask;       // [E], 0 = dead, or nullptr
  const int32_t* num_valid;  // rows from *num_valid on are padding, or nullptr
  int T, E, k, n_group, topk_group, group_max, renormalize;
  float rsf;
  int32_t* ids;  // [T, k]
  float* wts;    // [T, k]
  RouteGroups groups;
};

constexpr int kRouteWarps = 4;

// Order-preserving key of a float that is not NaN. -inf maps to kDeadKey,
// every larger value above it; 0 is left for experts that cannot be picked.
constexpr uint32_t kDeadKey = 0x007fffffu;
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 rank as equals
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float route_logit(const RouteArgs& a, size_t row, int e) {
  if (a.dtype == 4) return static_cast<const float*>(a.logits)[row + e];
  const unsigned short b = static_cast<const unsigned short*>(a.logits)[row + e];
  return a.dtype == 0 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}

// exp(l - mx) with the limit of equal infinities taken as 1.
__device__ __forceinline__ double route_exp(float l, float mx) {
  return l == mx ? 1.0 : exp(static_cast<double>(l) - static_cast<double>(mx));
}

template <int VPL, bool SOFTMAX>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a) {
  extern __shared__ float route_sm[];  // per warp: c by group (n_group > 1)
  __shared__ double p_sm[SOFTMAX ? kRouteWarps : 1][SOFTMAX ? 32 * VPL : 1];
  const int wib = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + wib;
  grid_dependents_launch();
  if (t >= a.T) return;
  grid_dependency_wait();
  const float NEG_INF = __int_as_float(0xff800000);
  const size_t row = static_cast<size_t>(t) * a.ld;

  // every load of the row's inputs first: they are in flight together (the bias moved down to its use: 4096 x 256 in
  // groups 11.5 against 11.3 us)
  float l[VPL], bias[VPL];
  float mx = NEG_INF;
  bool on[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    const bool in = e < a.E;
    l[i] = in ? route_logit(a, row, e) : NEG_INF;
    on[i] = !(in && a.mask) || a.mask[e] != 0;
    bias[i] = in && a.bias ? ld_global_here(a.bias + e) : 0.f;
  }
  const size_t out = static_cast<size_t>(t) * a.k + lane;
  if (a.num_valid && t >= *a.num_valid) {
    if (lane < a.k) {
      a.ids[out] = kNoExpert;
      a.wts[out] = 0.f;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (!on[i] || l[i] != l[i]) l[i] = NEG_INF;
    mx = fmaxf(mx, l[i]);
  }

  // c of this lane's experts e = lane + 32 i, then its key; positions past E
  // take no part (key 0)
  double inv_z = 1.0;
  float c[VPL];
  if (SOFTMAX) {
    mx = warp_max_f(mx);
    double p[VPL];
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = l[i] == NEG_INF ? 0.0 : route_exp(l[i], mx);
      p_sm[wib][lane + 32 * i] = p[i];
      z += p[i];
    }
    z = warp_sum_d(z);
    inv_z = z > 0.0 ? route_rcp(z) : 0.0;  // the largest term is 1
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = static_cast<float>(p[i] * inv_z);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = static_cast<float>(route_sigmoid(l[i]));
  }
  const RouteGroups& G = a.groups;
  float* c_sm = route_sm + wib * G.words(a.n_group);
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    if (e < a.E) {
      float v = a.bias ? __fadd_rn(c[i], bias[i]) : c[i];
      if (l[i] == NEG_INF || v != v) v = NEG_INF;
      key[i] = order_key(v);
      if (a.n_group > 1) {
        const int g = static_cast<int>(static_cast<uint32_t>(e) * G.magic >> 20);
        c_sm[e + g * (G.stride - G.size)] = v;
      }
    }
  }

  if (a.n_group > 1) {
    __syncwarp();
    // two best values of this lane's share of group g, merged over its lanes
    const int g = lane / G.lanes;
    const int sub = lane - g * G.lanes;
    float m1 = NEG_INF, m2 = NEG_INF;
    if (g < a.n_group) {
      for (int j = sub; j < G.size; j += G.lanes) {
        const float v = c_sm[g * G.stride + j];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    }
    for (int o = 1; o < G.lanes; o *= 2) {
      const float o1 = __shfl_xor_sync(0xffffffffu, m1, o);
      const float o2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
      m1 = fmaxf(m1, o1);
    }
    // a group with one live expert scores that expert alone; two whose sum lies below the fp32 range (biases of
    // its lowest value) still score above a group without one
    const float score = (a.group_max || m2 == NEG_INF) ? m1 : fmaxf(__fadd_rn(m1, m2), -3.402823466e38f);
    uint32_t gkey = (sub == 0 && g < a.n_group) ? order_key(score) : 0;
    uint32_t kept = 0;  // by group
    for (int r = 0; r < a.topk_group; ++r) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
      const int win = __ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1;  // lowest lane = lowest group
      if (lane == win) gkey = 0;
      kept |= 1u << (win / G.lanes);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      if (!((kept >> (static_cast<uint32_t>(e) * G.magic >> 20)) & 1u)) key[i] = 0;  // past E the key is 0 already
    }
  }

  // k rounds; lane j keeps the j-th pick. k1 / i1: this lane's best key and the
  // lowest slot that holds it. With eight slots or more also the next, k2 / i2:
  // such a lane looks through its slots again only when both are gone, which few
  // rows come to (4096 x 256: 11.3 against 12.2 us; 32 x 128, four slots, 3.5
  // against 3.4).
  constexpr bool kTwo = VPL >= 8;
  uint32_t k1, k2, taken = 0;
  int i1, i2;
  auto scan = [&]() {
    k1 = k2 = 0;
    i1 = i2 = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t v = (taken >> i) & 1u ? 0u : key[i];
      if (v > k1) {
        k2 = k1, i2 = i1;
        k1 = v, i1 = i;
      } else if (kTwo && v > k2) {
        k2 = v, i2 = i;
      }
    }
  };
  scan();
  bool second = kTwo;  // k2 / i2 hold the lane's next
  __syncwarp();        // p_sm
  int sel = 0;
  bool live = false;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, k1);
    const unsigned e = __reduce_min_sync(0xffffffffu, k1 == m ? static_cast<unsigned>(lane + 32 * i1) : 0xffffffffu);
    if (lane == j) {
      sel = static_cast<int>(e);
      live = m > kDeadKey;
    }
    if (lane == static_cast<int>(e & 31u)) {
      taken |= 1u << i1;
      if (second) {
        k1 = k2;
        i1 = i2;
        second = false;
      } else {
        scan();
        second = kTwo;
      }
    }
  }

  double p = 0.0;
  if (lane < a.k && live) {
    p = SOFTMAX ? p_sm[wib][sel] * inv_z : route_sigmoid(route_logit(a, row, sel));
  }
  if (a.renormalize) {
    const double sum = warp_sum_d(p);
    p = sum > 0.0 ? p / sum : 0.0;
  }
  if (lane < a.k) {
    a.ids[out] = sel;
    a.wts[out] = static_cast<float>(p * static_cast<double>(a.rsf));
  }
}

}  // namespace moe

// norm.cuh - residual add, RMS norm and quantisation in one pass.
//
//   z = x + residual                    (fp32)       residual_out = round(z)
//   y = z * rsqrt(mean(z^2) + eps) * gamma           (fp32)
//   y rounded once to x's type, and / or quantised from the unrounded y to the
//   layer's operand formats: e4m3 codes with one fp32 scale per row, or MXFP8
//   (e4m3 codes, one ue8m0 byte per 32 columns).
//
// The norm reads the unrounded z, so that y carries one rounding, not two.
//
// What bounds it: bytes. Every operand is read once and every output written
// once; a row stays in registers between the sum and the stores. TPR threads
// share a row, V 16-byte chunks (8 values) each; narrow rows are packed several
// to a block of 256 threads so that a block always has 256 threads' loads in
// flight. Measured at 4096 x 7168 with residual, 16-bit rows and MXFP8 codes: 41.1 to
// 41.6 us for 265 MB, 6.4 TB/s, the measured copy rate; to fp8 codes 46.6, two
// reductions.
#pragma once
#include "ptx_ext.cuh"
#include "quant.cuh"
#include "router.cuh"

namespace moe {

enum NormQuant : int { kNormPlain = 0, kNormFp8 = 1, kNormMx = 2 };

struct NormArgs {
  const void* x;         // [T, H] bf16 or fp16
  const void* residual;  // [T, H] or nullptr
  const void* gamma;     // [H]: x's type, or fp32 with gamma_f32
  int gamma_f32;
  float eps;
  int T, H;
  void* residual_out;  // [T, H] or nullptr
  void* y;             // [T, H] or nullptr
  uint8_t* codes;      // [T, H] (kNormFp8, kNormMx)
  float* scale;        // [T] (kNormFp8)
  uint8_t* sbytes;     // [T, H / 32] (kNormMx)
};

// Two rounded values in a word, low half first: the packing conversion (the
// conversions of single values run at an eighth of its rate).
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename TX>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  unpack2(v.x, TX(), f[0], f[1]);
  unpack2(v.y, TX(), f[2], f[3]);
  unpack2(v.z, TX(), f[4], f[5]);
  unpack2(v.w, TX(), f[6], f[7]);
}
template <typename TX>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1], TX()), pack2(f[2], f[3], TX()), pack2(f[4], f[5], TX()),
                    pack2(f[6], f[7], TX()));
}

// Sum or maximum over the TPR threads of a row. `sm`: one float per warp of
// the block; a second call in one kernel takes another array.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* sm) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    __syncthreads();
    const int w0 = warp / W * W;
    v = sm[w0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = MAX ? fmaxf(v, sm[w0 + w]) : v + sm[w0 + w];
  }
  return v;
}

// y / s rounded to nearest, from inv = 1 / s rounded to nearest: the estimate y * inv
// is within a unit of the last place, its remainder q s - y is exact in one fused
// operation, and q minus the remainder times inv, again fused, rounds as the
// quotient does (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). Needs a normal inv (s <= 2^120 here, 448 s being
// finite) and a remainder that does not underflow: a multiple of 2^-56 s or more for
// quotients from 2^-10 on, hence s >= 2^-90. Below 2^-10 the estimate's error cannot
// change the code, which is a zero of y's sign (the remainder of a zero keeps it).
__device__ __forceinline__ float row_quotient(float y, float s, float inv) {
  const float q = y * inv;
  return fmaf(-fmaf(q, s, -y), inv, q);
}

template <typename TX, int Q, int TPR, int V>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) k_rmsnorm(const NormArgs a) {
  constexpr int kThreads = TPR > 256 ? TPR : 256;
  __shared__ float sum_sm[kThreads / 32], max_sm[kThreads / 32];
  const int sub = threadIdx.x % TPR;
  const int t = blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  const bool row = t < a.T;  // the last block's spare rows only take part in its barriers
  const int nc = row ? a.H / 8 : 0;
  const size_t base = static_cast<size_t>(row ? t : 0) * a.H;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const TX*>(a.x) + base);
  const uint4* r = a.residual ? reinterpret_cast<const uint4*>(static_cast<const TX*>(a.residual) + base) : nullptr;

  // 16-bit gamma is fetched with the row, or, where four chunks per thread leave few
  // registers, while the sum is reduced (4096 x 7168 fp8: 46.9 against 51.3 us; 1792 x
  // 16384 MXFP8: 44.0 against 45.0; 4096 x 4096 plain: 21.8 against 23.0). Early is
  // better elsewhere (4096 x 7168 MXFP8 42.0 against 46.4; 4096 x 4096 fp8 24.5 against
  // 27.4, MXFP8 24.5 against 25.5; 1792 x 16384 fp8 49.9 against 61.5).
  constexpr bool kGammaLate = V == 4 && (Q == kNormPlain || TPR == (Q == kNormFp8 ? 256 : 512));
  auto gamma16 = [&](int c) {
    return !a.gamma_f32 && c < nc ? static_cast<const uint4*>(a.gamma)[c] : make_uint4(0, 0, 0, 0);
  };

  grid_dependents_launch();
  grid_dependency_wait();
  uint4 xv[V], rv[V], gv[V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int c = sub + u * TPR;
    xv[u] = c < nc ? x[c] : make_uint4(0, 0, 0, 0);
    rv[u] = r && c < nc ? r[c] : make_uint4(0, 0, 0, 0);
    if (!kGammaLate) gv[u] = gamma16(c);
  }
  float z[V][8];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int c = sub + u * TPR;
    unpack8<TX>(xv[u], z[u]);
    if (r) {
      float f[8];
      unpack8<TX>(rv[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[u][i] += f[i];
    }
    if (a.residual_out && c < nc)
      reinterpret_cast<uint4*>(static_cast<TX*>(a.residual_out) + base)[c] = pack8<TX>(z[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(z[u][i], z[u][i], ss);
  }
  if (kGammaLate) {
#pragma unroll
    for (int u = 0; u < V; ++u) gv[u] = gamma16(sub + u * TPR);
  }
  ss = row_reduce<TPR, false>(ss, sum_sm);
  const float rstd = rsqrtf(ss / static_cast<float>(a.H) + a.eps);

  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int c = sub + u * TPR;
    float g[8];
    if (a.gamma_f32) {
      const float4* gp = static_cast<const float4*>(a.gamma) + 2 * c;
      const float4 lo = c < nc ? *gp : make_float4(0, 0, 0, 0);
      const float4 hi = c < nc ? gp[1] : make_float4(0, 0, 0, 0);
      g[0] = lo.x, g[1] = lo.y, g[2] = lo.z, g[3] = lo.w;
      g[4] = hi.x, g[5] = hi.y, g[6] = hi.z, g[7] = hi.w;
    } else {
      unpack8<TX>(gv[u], g);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) z[u][i] = z[u][i] * rstd * g[i];
    if (a.y && c < nc) reinterpret_cast<uint4*>(static_cast<TX*>(a.y) + base)[c] = pack8<TX>(z[u]);
    if (Q != kNormPlain) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(z[u][i]));
      if (Q == kNormFp8) {
        amax = fmaxf(amax, m);
      } else {
        // 32 columns = the chunks of four consecutive lanes (H % 32 == 0: in or out together)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (c < nc) {
          const int X = mx_exponent_bits(m);
          const float f = pow2_neg(X);  // exact: a power of two in the normal range
          uint32_t q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) q[i] = cvt_e4m3x2(z[u][2 * i] * f, z[u][2 * i + 1] * f);
          reinterpret_cast<uint2*>(a.codes + base)[c] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
          if ((threadIdx.x & 3) == 0)
            a.sbytes[static_cast<size_t>(t) * (a.H / 32) + c / 4] = static_cast<uint8_t>(X + 127);
        }
      }
    }
  }
  if (Q == kNormFp8) {
    amax = row_reduce<TPR, true>(amax, max_sm);
    const float s = amax > 0.f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (row && sub == 0) a.scale[t] = s;
    // One division per row, and every quotient corrected by its remainder (row_quotient): dividing every value cost
    // 69 against 50 us at 4096 x 7168; the correction costs 0.4 us there (46.2 -> 46.6). Scales outside its range
    // divide: below 2^-90, and infinite.
    const float inv = __fdiv_rn(1.0f, s);
    const bool divide = !(s >= 0x1p-90f && s <= 3.402823466e38f);
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int c = sub + u * TPR;
      if (c < nc) {
        if (divide) {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[u][i] = __fdiv_rn(z[u][i], s);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) z[u][i] = row_quotient(z[u][i], s, inv);
        }
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = cvt_e4m3x2(z[u][2 * i], z[u][2 * i + 1]);
        reinterpret_cast<uint2*>(a.codes + base)[c] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
    }
  }
}

}  // namespace moe

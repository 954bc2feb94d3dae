// block_ops.cu - the library's translation unit: the layer (moe_b200.cu) and,
// here, the host side of the operators around it: moe_linear, moe_route and
// moe_rmsnorm_quantize (include/moe_b200.h). As there, every call checks its
// arguments before it launches anything and allocates nothing. One unit, so that
// all kernels share one device error word and the helpers of the layer's file.
#include "moe_b200.cu"

#include "linear.cuh"
#include "norm.cuh"
#include "route.cuh"

namespace {

inline bool is_16bit(int dtype) { return dtype == MOE_DT_BF16 || dtype == MOE_DT_FP16; }
inline bool is_float_dt(int dtype) { return is_16bit(dtype) || dtype == MOE_DT_F32; }
inline int float_size(int dtype) { return dtype == MOE_DT_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Launch that may start while the stream's previous kernel still drains (see
// grid_dependency_wait): the kernel waits for it on the device. `early` = false
// launches as usual (the kernel's wait then returns at once). `cluster`: CTAs
// per cluster, or 0. Measured back to back in a graph: linear 5.8 -> 4.8 us (one
// token, 2048 x 2048), 23.8 -> 23.1 us (fp8, 1024 x 5632 x 4096), norm 1.8 ->
// 1.4 us and routing 3.8 -> 3.3 us (32 tokens).
template <typename... P, typename... A>
moe_status_t launch_early(void (*kern)(P...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                          bool early, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = early;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = cluster ? 2 : 1;
  MOE_CK(cudaLaunchKernelEx(&cfg, kern, args...));
  return MOE_OK;
}

// make_map in a thread that may not have used CUDA before: the driver call behind it
// needs the device's context to be current, which a thread gets from its first
// runtime call that uses the device. One retry, so that other calls pay nothing.
moe_status_t make_map_any_thread(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base,
                                 const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const moe_status_t r = make_map(m, dt, rank, base, dims, strides, box);
  if (r == MOE_OK) return r;
  int dev = 0;
  MOE_CK(cudaGetDevice(&dev));
  MOE_CK(cudaSetDevice(dev));
  return make_map(m, dt, rank, base, dims, strides, box);
}

// An operand of the linear product, `rows` rows of K elements, ld elements
// apart: `m` as [atoms][rows][128 bytes] over the K atoms that K fills, read
// kLinAtoms atoms x box_rows rows at a time, and `tail` as the plain matrix,
// read one atom at a time (zeros past K). A map that no stage reads is a copy
// of the other.
moe_status_t make_linear_maps(CUtensorMap* m, CUtensorMap* tail, int dtype, const void* base, int rows, int K,
                              int64_t ld, int box_rows) {
  const int es = is_16bit(dtype) ? 2 : 1;
  const CUtensorMapDataType dt = dtype == MOE_DT_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : dtype == MOE_DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint32_t ke = static_cast<cuuint32_t>(moe::kTileKBytes / es);
  const cuuint64_t row = static_cast<cuuint64_t>(ld) * es;
  const bool whole = K >= static_cast<int>(ke) * moe::kLinAtoms;      // some stage is full
  const bool ragged = K % (static_cast<int>(ke) * moe::kLinAtoms) != 0;  // the last one is not
  if (ragged) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t st[1] = {row};
    const cuuint32_t box[2] = {ke, static_cast<cuuint32_t>(box_rows)};
    const moe_status_t r = make_map_any_thread(tail, dt, 2, base, dims, st, box);
    if (r != MOE_OK) return r;
  }
  if (whole) {
    const cuuint64_t dims[3] = {ke, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(K / ke)};
    const cuuint64_t st[2] = {row, moe::kTileKBytes};
    const cuuint32_t box[3] = {ke, static_cast<cuuint32_t>(box_rows), moe::kLinAtoms};
    const moe_status_t r = make_map_any_thread(m, dt, 3, base, dims, st, box);
    if (r != MOE_OK) return r;
  }
  if (!ragged) *tail = *m;
  if (!whole) *m = *tail;
  return MOE_OK;
}

// The widest access (16, 8, 4 or 2 bytes) that divides the address and the length
// of every row.
int row_unit(const void* base, size_t ld, int cols, int es) {
  const size_t all = reinterpret_cast<uintptr_t>(base) | (ld * es) | (static_cast<size_t>(cols) * es);
  return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

struct LinearCall {
  int dtype;
  const void *x, *w;
  int64_t ldx, ldw;
  int K;
  moe::LinearArgs g;
};

template <int BN, bool FP8, bool F32, bool PROMOTE>
moe_status_t launch_linear_split(const LinearCall& c, int S, cudaStream_t s) {
  using L = moe::SplitCfg<BN>;
  CUtensorMap tw, twt, tx, txt;
  moe_status_t r = make_linear_maps(&tw, &twt, c.dtype, c.w, c.g.N, c.K, c.ldw, moe::kTileM);
  if (r != MOE_OK) return r;
  r = make_linear_maps(&tx, &txt, c.dtype, c.x, c.g.T, c.K, c.ldx, BN);
  if (r != MOE_OK) return r;
  auto kern = moe::k_linear_split<BN, FP8, F32, PROMOTE>;
  static std::atomic<int> attr_set[64];
  r = set_smem_attr(kern, 227 * 1024, attr_set);
  if (r != MOE_OK) return r;
  const int ctas = (c.g.N - 1) / moe::kTileM * S + S;
  // one CTA per SM takes all of its shared memory for stages; more CTAs than
  // SMs share it two by two (N = 20000, K = 2048, one token: 16.7 against 21.2 us)
  const int n_stages = L::stages(ctas <= num_sms() ? 227 * 1024 : 113 * 1024);
  return launch_early(kern, ctas, moe::kSplitThreads, L::bytes(n_stages), S, true, s, tw, twt, tx, txt, c.g, S, n_stages);
}

template <bool FP8, bool PROMOTE, bool SPLIT, int U>
moe_status_t launch_linear_tile(const LinearCall& c, int tn, int split, cudaStream_t s) {
  using L = moe::TileCfg;
  CUtensorMap tx, txt, tw, twt;
  moe_status_t r = make_linear_maps(&tx, &txt, c.dtype, c.x, c.g.T, c.K, c.ldx, moe::kTileM);
  if (r != MOE_OK) return r;
  r = make_linear_maps(&tw, &twt, c.dtype, c.w, c.g.N, c.K, c.ldw, tn / 2);
  if (r != MOE_OK) return r;
  auto kern = moe::k_linear_tile<FP8, PROMOTE, SPLIT, U>;
  static std::atomic<int> attr_set[64];
  r = set_smem_attr(kern, 227 * 1024, attr_set);
  if (r != MOE_OK) return r;
  moe::LinearArgs g = c.g;
  g.tn = tn;
  g.n_tb = (g.T + 2 * moe::kTileM - 1) / (2 * moe::kTileM);
  g.n_nt = (g.N + tn - 1) / tn;
  const int64_t tiles = static_cast<int64_t>(g.n_tb) * g.n_nt;
  if (tiles > INT32_MAX / 16) return MOE_ERR_SHAPE;
  g.split = split;
  const int pairs = num_sms() / 2;
  const int ctas = static_cast<int>(SPLIT ? 2 * tiles * split : 2 * (tiles < pairs ? tiles : pairs));
  return launch_early(kern, ctas, moe::kTileThreads, L::bytes(tn), SPLIT ? 2 * split : 2, true, s,
                      tx, txt, tw, twt, g);
}

struct LinearPlan {
  int bn;     // k_linear_split: tokens per tile
  int split;  // CTAs (k_linear_split) or pairs (k_linear_tile) along K
  int tn;     // k_linear_tile: outputs per tile, or 0
};

template <bool FP8, bool PROMOTE>
moe_status_t launch_linear_pairs(LinearCall& c, const LinearPlan& p, cudaStream_t s) {
  moe::LinearArgs& g = c.g;
  const int os = float_size(g.out_dt);
  g.out_unit = row_unit(g.out, g.ldo, g.N, os);
  g.res_unit = g.residual ? row_unit(g.residual, g.ldr, g.N, os) : 16;
  if (p.split > 1) return launch_linear_tile<FP8, PROMOTE, true, 16>(c, p.tn, p.split, s);
  const int unit = g.out_unit < g.res_unit ? g.out_unit : g.res_unit;
  if (unit == 16) return launch_linear_tile<FP8, PROMOTE, false, 16>(c, p.tn, 1, s);
  if (unit == 8) return launch_linear_tile<FP8, PROMOTE, false, 8>(c, p.tn, 1, s);
  if constexpr (!PROMOTE) {  // fp32 rows are aligned to 4 bytes at least
    if (unit == 2) return launch_linear_tile<FP8, PROMOTE, false, 2>(c, p.tn, 1, s);
  }
  return launch_linear_tile<FP8, PROMOTE, false, 4>(c, p.tn, 1, s);
}

// Clusters of the pair kernel (2 * split CTAs, one per SM) that run at one time.
int resident_clusters(int split) {
  static std::atomic<int> cache[64][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  std::atomic<int>& slot = cache[dev][split / 2];
  int n = slot.load();
  if (n) return n;
  auto kern = moe::k_linear_tile<false, false, true, 16>;
  static std::atomic<int> attr_set[64];
  if (set_smem_attr(kern, 227 * 1024, attr_set) != MOE_OK) return 1;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(2 * split);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * split * num_sms()));
  cfg.blockDim = dim3(moe::kTileThreads);
  cfg.dynamicSmemBytes = 200 * 1024;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kern), &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();  // clear: no K split
    n = 1;
  }
  slot.store(n);
  return n;
}

// Which kernel and tiles. The times below are nanoseconds measured on B200;
// they only rank the choices.
LinearPlan plan_linear(int T, int N, int nk, bool f32_out) {
  LinearPlan p{};
  const int ns = (nk + moe::kLinAtoms - 1) / moe::kLinAtoms;  // stages along K
  if (T <= 64) {
    // Weights on the MMA's M side. The K split that still runs all CTAs at one
    // time streams the weights fastest (N = K = 2048, one token: 8.6, 7.2, 6.3
    // us for 1, 2, 4 CTAs per tile and 10.1 for 8, whose clusters no longer
    // fit; N = K = 7168: 21.7, 19.4, 23.4). fp32 results give each CTA a piece of
    // at most 14 atoms, as far as 8 CTAs go; past that a CTA takes several in turn.
    p.bn = T <= 16 ? 16 : T <= 32 ? 32 : 64;
    const int tiles = (N - 1) / moe::kTileM + 1;
    p.split = 1;
    for (int S = 2; S <= 8 && ns >= S; S *= 2) {
      const int fit = S == 8 ? num_sms() * 3 / 4 : num_sms();
      const bool precise = f32_out && (ns + p.split - 1) / p.split > moe::kSplitPieceStages;
      if (static_cast<int64_t>(tiles) * S <= fit || precise) p.split = S;
    }
    return p;
  }
  // Tokens on the M side, CTA pairs. ns per K atom and fixed time of a tile by
  // its width (T = 1024, N = 9 tn, K = 2048 and 8192): the narrow ones are
  // bound by the copies' round trip over the stages that fit, the widest by
  // the MMAs (512 clocks an atom at tn = 256).
  const int64_t tb = (T - 1) / 256 + 1;
  int64_t best = INT64_MAX;
  for (int tn = 256; tn >= 64; tn -= 32) {
    static const int atom_ns[7] = {145, 187, 200, 210, 280, 290, 308};
    const int64_t a = atom_ns[tn / 32 - 2];
    const int64_t tiles = tb * ((N - 1) / tn + 1);
    const int64_t fixed = 4500 + 12 * tn;
    if (!f32_out || tn <= moe::kPromoteTn) {
      const int64_t waves = (tiles - 1) / (num_sms() / 2) + 1;
      const int64_t cost = fixed + waves * nk * a;
      if (cost < best) best = cost, p.tn = tn, p.split = 1;
    }
    // K over 2 or 4 pairs of a cluster: one wave only, and for fp32 results at
    // most 14 atoms in each of a pair's two accumulations
    for (int S = 2; S <= 4; S *= 2) {
      if (ns < 4 * S || (f32_out && (ns + S - 1) / S > 14)) continue;
      if (tiles > resident_clusters(S)) continue;
      const int64_t cost = fixed + 3500 + 9 * tn + nk * a / S;  // plus the join
      if (cost < best) best = cost, p.tn = tn, p.split = S;
    }
  }
  return p;
}

template <bool FP8, bool F32, bool PROMOTE>
moe_status_t launch_linear_bn(const LinearCall& c, const LinearPlan& p, cudaStream_t s) {
  if (p.bn == 16) return launch_linear_split<16, FP8, F32, PROMOTE>(c, p.split, s);
  if (p.bn == 32) return launch_linear_split<32, FP8, F32, PROMOTE>(c, p.split, s);
  return launch_linear_split<64, FP8, F32, PROMOTE>(c, p.split, s);
}

template <bool FP8, bool F32>
moe_status_t launch_linear(LinearCall& c, cudaStream_t s) {
  const LinearPlan p = plan_linear(c.g.T, c.g.N, c.g.nk, F32);
  if (p.tn) return launch_linear_pairs<FP8, F32>(c, p, s);
  if constexpr (F32) {  // a CTA's share of K above one piece
    const int ns = (c.g.nk + moe::kLinAtoms - 1) / moe::kLinAtoms;
    if ((ns + p.split - 1) / p.split > moe::kSplitPieceStages) return launch_linear_bn<FP8, true, true>(c, p, s);
  }
  return launch_linear_bn<FP8, F32, false>(c, p, s);
}

template <int VPL>
moe_status_t launch_route(const moe::RouteArgs& a, bool softmax, cudaStream_t s) {
  const size_t smem = a.n_group > 1 ? moe::kRouteWarps * a.groups.words(a.n_group) * sizeof(float) : 0;
  const int blocks = (a.T - 1) / moe::kRouteWarps + 1;  // T goes up to 2^31 - 1
  // a grid that fills the SMs gains nothing from a successor's waiting blocks (4096 tokens: 12.2 against 13.0 us)
  return launch_early(softmax ? moe::k_route<VPL, true> : moe::k_route<VPL, false>, blocks, moe::kRouteWarps * 32, smem,
                      0, blocks <= 2 * num_sms(), s, a);
}

template <typename TX, int Q, int TPR, int V>
moe_status_t launch_rmsnorm(const moe::NormArgs& a, cudaStream_t s) {
  constexpr int threads = TPR > 256 ? TPR : 256;
  constexpr int rows = threads / TPR;
  return launch_early(moe::k_rmsnorm<TX, Q, TPR, V>, (a.T - 1) / rows + 1, threads, 0, 0, true, s, a);
}

// Threads per row and 16-byte chunks per thread, by the row's chunk count: one
// chunk per thread is the quickest row. Rows of 2049 to 4096 columns are cheaper
// with four chunks per thread when there are enough of them to fill the SMs
// (T = 4096: fp8 24.6 against 30.6 us, MXFP8 24.5 against 25.4, plain 21.8 against
// 25.0; T = 300: fp8 3.4 against 3.9 the other way round), and the two reductions
// of a wide fp8 row with half the warps (H = 7168, T = 4096: 46.9 against 61.1 us,
// T = 32: 2.6 against 2.8; MXFP8, with one, 42.4 against 41.7).
template <typename TX, int Q>
moe_status_t launch_rmsnorm_row(const moe::NormArgs& a, cudaStream_t s) {
  const int nc = a.H / 8;
  if (nc <= 32) return launch_rmsnorm<TX, Q, 32, 1>(a, s);
  if (nc <= 64) return launch_rmsnorm<TX, Q, 64, 1>(a, s);
  if (nc <= 128) return launch_rmsnorm<TX, Q, 128, 1>(a, s);
  if (nc <= 256) return launch_rmsnorm<TX, Q, 256, 1>(a, s);
  if (nc <= 512)
    return a.T >= 4 * num_sms() ? launch_rmsnorm<TX, Q, 128, 4>(a, s) : launch_rmsnorm<TX, Q, 512, 1>(a, s);
  if (nc <= 1024)
    return Q == moe::kNormFp8 ? launch_rmsnorm<TX, Q, 256, 4>(a, s) : launch_rmsnorm<TX, Q, 512, 2>(a, s);
  return launch_rmsnorm<TX, Q, 512, 4>(a, s);
}

template <typename TX>
moe_status_t launch_rmsnorm_quant(const moe::NormArgs& a, int q, cudaStream_t s) {
  if (q == moe::kNormFp8) return launch_rmsnorm_row<TX, moe::kNormFp8>(a, s);
  if (q == moe::kNormMx) return launch_rmsnorm_row<TX, moe::kNormMx>(a, s);
  return launch_rmsnorm_row<TX, moe::kNormPlain>(a, s);
}

}  // namespace

extern "C" {

moe_status_t moe_linear(int dtype, const void* x, int64_t ldx, const float* x_scale, const void* w, int64_t ldw,
                        const float* w_scale, int w_scale_rows, const void* bias, int bias_dtype, int act,
                        const void* residual, int64_t ldr, void* out, int out_dtype, int64_t ldo, int T, int N, int K,
                        moe_stream_t stream) {
  const bool fp8 = dtype == MOE_DT_FP8_E4M3;
  if (!is_16bit(dtype) && !fp8) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (!is_float_dt(out_dtype) || (bias && !is_float_dt(bias_dtype))) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || N < 1 || K < 1 || act < MOE_ACT_NONE || act > MOE_ACT_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !w || !out) return MOE_ERR_INVALID_ARG;
  if (fp8 ? (!x_scale || !w_scale || (w_scale_rows != 1 && w_scale_rows != N)) : (x_scale || w_scale))
    return MOE_ERR_INVALID_ARG;
  if (ldx < K || ldw < K || ldo < N || (residual && ldr < N)) return MOE_ERR_INVALID_ARG;
  const int es = fp8 ? 1 : 2;
  const int64_t row_max = int64_t{1} << 36;  // row strides the tensor maps and 64-bit offsets cover
  const int size_max = 1 << 30;              // and sizes whose tiles count in 32 bits, past the last one included
  if (T > size_max || N > size_max || K > size_max) return MOE_ERR_SHAPE;
  if (ldx > row_max || ldw > row_max || ldo > row_max || (residual && ldr > row_max)) return MOE_ERR_SHAPE;
  const int os = float_size(out_dtype);
  if (!aligned16(x) || !aligned16(w) || ldx * es % 16 != 0 || ldw * es % 16 != 0 || !aligned_to(out, os) ||
      (residual && !aligned_to(residual, os)) || (bias && !aligned_to(bias, float_size(bias_dtype))) ||
      !aligned_to(x_scale, 4) || !aligned_to(w_scale, 4))
    return MOE_ERR_ALIGNMENT;
  LinearCall c{};
  c.dtype = dtype;
  c.x = x;
  c.w = w;
  c.ldx = ldx;
  c.ldw = ldw;
  c.K = K;
  moe::LinearArgs& g = c.g;
  g.T = T;
  g.N = N;
  g.nk = static_cast<int>((static_cast<int64_t>(K) * es + moe::kTileKBytes - 1) / moe::kTileKBytes);
  g.nk_full = K / (moe::kTileKBytes / es);
  g.f16 = dtype == MOE_DT_FP16;
  g.x_scale = x_scale;
  g.w_scale = w_scale;
  g.w_scale_step = w_scale_rows == 1 ? 0 : 1;
  g.bias = bias;
  g.bias_dt = bias_dtype;
  g.act = act;
  g.residual = residual;
  g.ldr = static_cast<size_t>(ldr);
  g.out = out;
  g.ldo = static_cast<size_t>(ldo);
  g.out_dt = out_dtype;
  cudaStream_t s = as_stream(stream);
  if (out_dtype == MOE_DT_F32) return fp8 ? launch_linear<true, true>(c, s) : launch_linear<false, true>(c, s);
  return fp8 ? launch_linear<true, false>(c, s) : launch_linear<false, false>(c, s);
}

moe_status_t moe_route(const void* logits, int logits_dtype, int64_t ld, const float* bias,
                       const uint8_t* expert_mask, const int32_t* num_valid, int T, int E, int top_k, int score,
                       int n_group, int topk_group, int group_score, int renormalize, float routed_scaling_factor,
                       int32_t* topk_ids, float* topk_weights, moe_stream_t stream) {
  if (!is_float_dt(logits_dtype)) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || E < 1 || E > MOE_MAX_EXPERTS || top_k < 1 || top_k > E || top_k > MOE_MAX_TOPK)
    return MOE_ERR_INVALID_ARG;
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (group_score != MOE_GROUP_TOP2 && group_score != MOE_GROUP_MAX) return MOE_ERR_INVALID_ARG;
  if (n_group < 1 || n_group > 32 || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
      top_k > topk_group * (E / n_group))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights || ld < E) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(logits, float_size(logits_dtype)) || !aligned_to(bias, 4) || !aligned_to(num_valid, 4) ||
      !aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4))
    return MOE_ERR_ALIGNMENT;
  moe::RouteArgs a{logits, static_cast<size_t>(ld), logits_dtype, bias, expert_mask, num_valid, T, E, top_k,
                   n_group, topk_group, group_score == MOE_GROUP_MAX, renormalize, routed_scaling_factor, topk_ids,
                   topk_weights, moe::RouteGroups(E, n_group)};
  const bool softmax = score == MOE_SCORE_SOFTMAX;
  cudaStream_t s = as_stream(stream);
  if (E <= 32) return launch_route<1>(a, softmax, s);
  if (E <= 64) return launch_route<2>(a, softmax, s);
  if (E <= 128) return launch_route<4>(a, softmax, s);
  if (E <= 256) return launch_route<8>(a, softmax, s);
  return launch_route<16>(a, softmax, s);
}

moe_status_t moe_rmsnorm_quantize(int dtype, int quant, const void* x, const void* residual, const void* gamma,
                                  int gamma_dtype, float eps, int T, int H, void* residual_out, void* y, void* codes,
                                  void* scale, moe_stream_t stream) {
  if (!is_16bit(dtype) || (gamma_dtype != dtype && gamma_dtype != MOE_DT_F32)) return MOE_ERR_UNSUPPORTED_DTYPE;
  const bool fp8 = quant == MOE_DT_FP8_E4M3, mx = quant == MOE_DT_MXFP8_E4M3;
  if (quant != MOE_DT_NONE && !fp8 && !mx) return MOE_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || H < 1 || !(eps > 0.f)) return MOE_ERR_INVALID_ARG;
  if (H % (mx ? 32 : 8) != 0 || H > 16384) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !gamma || (!residual_out && !y && quant == MOE_DT_NONE)) return MOE_ERR_INVALID_ARG;
  if ((quant != MOE_DT_NONE) != (codes != nullptr) || (codes != nullptr) != (scale != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned_to(codes, 8) || (fp8 && !aligned_to(scale, 4)))
    return MOE_ERR_ALIGNMENT;
  moe::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.gamma_f32 = gamma_dtype == MOE_DT_F32;
  a.eps = eps;
  a.T = T;
  a.H = H;
  a.residual_out = residual_out;
  a.y = y;
  a.codes = static_cast<uint8_t*>(codes);
  if (fp8) a.scale = static_cast<float*>(scale);
  else a.sbytes = static_cast<uint8_t*>(scale);
  const int q = fp8 ? moe::kNormFp8 : mx ? moe::kNormMx : moe::kNormPlain;
  cudaStream_t s = as_stream(stream);
  return dtype == MOE_DT_BF16 ? launch_rmsnorm_quant<__nv_bfloat16>(a, q, s) : launch_rmsnorm_quant<__half>(a, q, s);
}

}  // extern "C"

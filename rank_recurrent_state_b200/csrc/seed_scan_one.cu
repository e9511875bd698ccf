// seed_scan_one.cu -- the scan for one or two tokens per sequence: a model served with
// dense states takes it every decode step.
//
// Bound by the states' bytes: a block holds the whole d_k x d_v state of one (sequence,
// head) in registers, read and written once in float4 rows (coalesced, streaming), and
// forms S^T k and S^T q together before the update, as the dense step does:
//     w = beta (v - S'^T k), S+ = S' + k w^T, o = S'^T q + (k . q) w
// One token of 16 sequences x 48 heads of 128 x 128: 20 us, 5.1 TB/s (the token-by-token
// kernel, whose accesses to the state are 32-byte pieces, 46 us).  Every token costs two
// block-wide barriers, so longer sequences go to the kernels without them.
#include "seed_scan.cuh"

namespace seed {

namespace {

template <int FORM, int DK, int DV, int NT>
__global__ void __launch_bounds__(NT) scan_one_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  constexpr int CQ = DV / 4, RG = NT / CQ, RPT = DK / RG;      // column quads, row groups, rows per thread
  static_assert(RPT >= 1 && RG * CQ == NT, "tile");
  __shared__ __align__(16) float s_k[DK], s_q[DK], s_al[KDA ? DK : 4];
  __shared__ __align__(16) float s_pk[RG][DV], s_pq[RG][DV];
  __shared__ float s_kq;
  const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H, hk = h / (p.H / p.HK);
  const SeqRange sr = seq_range(p, seq, h == 0 && tid == 0);
  const long long mat = (long long)blockIdx.x * DK * DV + 4 * cq;

  float4 S[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) S[r] = p.S0 != nullptr ? ld_stream4(p.S0 + mat + (long long)(rg + RG * r) * DV) : zero4();
  bool bad = false;
  for (int t = 0; t < sr.len; ++t) {
    const long long row = sr.first + t, at = (row * p.HK + hk) * DK;
    __syncthreads();
    for (int i = tid; i < DK; i += NT) {
      s_k[i] = act_ld(p.k, at + i, p.elem);
      s_q[i] = act_ld(p.q, at + i, p.elem);
      if constexpr (KDA) s_al[i] = p.alpha[(row * p.H + h) * DK + i];
    }
    const float g = KDA ? 1.f : p.alpha[row * p.H + h];
    const float be = p.beta[row * p.H + h];
    const float4 v = act_ld4(p.v, (row * p.H + h) * DV + 4 * cq, p.elem);
    __syncthreads();
    if (tid < 32) {
      float x = 0.f;
      for (int i = tid; i < DK; i += 32) x = fmaf(s_k[i], s_q[i], x);
      x = group_sum<32>(x);
      if (tid == 0) s_kq = x;
    }
    float4 pk = zero4(), pq = zero4();
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      const int i = rg + RG * r;
      const float d = KDA ? s_al[i] : g;
      S[r] = make_float4(d * S[r].x, d * S[r].y, d * S[r].z, d * S[r].w);
      if constexpr (!M2) pk = fma4(s_k[i], S[r], pk);
      pq = fma4(s_q[i], S[r], pq);
    }
    if constexpr (!M2) st4(&s_pk[rg][4 * cq], pk);
    st4(&s_pq[rg][4 * cq], pq);
    __syncthreads();
    float4 a = zero4(), b = zero4();
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      if constexpr (!M2) a = fma4(1.f, ld4(&s_pk[r][4 * cq]), a);
      b = fma4(1.f, ld4(&s_pq[r][4 * cq]), b);
    }
    const float4 w = make_float4(be * (v.x - a.x), be * (v.y - a.y), be * (v.z - a.z), be * (v.w - a.w));
#pragma unroll
    for (int r = 0; r < RPT; ++r) S[r] = fma4(s_k[rg + RG * r], w, S[r]);
    if (rg == 0) {
      const float4 o = fma4(s_kq, w, b);
      act_st4(p.o, (row * p.H + h) * DV + 4 * cq, o, p.elem);
      bad = bad || !(act_finite(o.x, p.elem) && act_finite(o.y, p.elem) && act_finite(o.z, p.elem) && act_finite(o.w, p.elem));
    }
  }
  if (p.S_out != nullptr) {
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      st_stream4(p.S_out + mat + (long long)(rg + RG * r) * DV, S[r]);
      bad = bad || !finite4(S[r]);
    }
  }
  if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
}

}  // namespace

int launch_scan_one(const ScanParams& p, int form, cudaStream_t st) {
#define SEED_ONE(F, K, V)                                                              \
  if (form == F && p.dk == K && p.dv == V) {                                           \
    constexpr int NT = K * V / 4 < 256 ? K * V / 4 : 256;                              \
    scan_one_kernel<F, K, V, NT><<<p.seqs * p.H, NT, 0, st>>>(p);                      \
    return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;                \
  }
#define SEED_ONE_D(F) \
  SEED_ONE(F, 16, 16) SEED_ONE(F, 32, 32) SEED_ONE(F, 64, 64) SEED_ONE(F, 128, 128) SEED_ONE(F, 128, 64) SEED_ONE(F, 64, 128)
  SEED_ONE_D(SEED_GDN)
  SEED_ONE_D(SEED_KDA)
  SEED_ONE_D(SEED_MAMBA2)
#undef SEED_ONE_D
#undef SEED_ONE
  return SEED_ERR_SHAPE;
}

}  // namespace seed

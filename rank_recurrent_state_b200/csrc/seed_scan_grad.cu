// seed_scan_grad.cu -- the gradients of one chunk of the dense scan from its states.
//
// For a chunk with the state S0 before it, the gradient dS of the state behind it,
// the written values w_i and their gradients dw_i (all from the two recurrences), and
// X_ij = do_i . w_j (j <= i), Y_ij = dw_i . w_j (j < i; zero for Mamba-2):
//     dq_i = B_i (S0 do_i) + sum_{j<=i} X_ij D_ij k_j
//     h_i  = B_i (S0 dw_i) + sum_{j<i}  Y_ij D_ij k_j            (= S'_i dw_i)
//     c_i  = D_Ci (dS w_i) + sum_{m>=i} X_mi D_mi q_m - sum_{m>i} beta_m Y_mi D_mi k_m
//     dk_i = c_i - beta_i h_i
//     dv_i = beta_i dw_i,   dbeta_i = v_i . dw_i - k_i . h_i
// per channel (summed over the channels where a head has one decay)
//     d log a_t = sum_{i>=t} (q_i dq_i - beta_i k_i h_i - k_i c_i)
//                 + B_C (S0 dS^T)_cc + sum_i k_i D_Ci (dS w_i)
// The last line is the derivative along log a: finite where a decay is zero.  Its terms
// that no decay touches (X_ii, and the last token's share of the state behind it) cancel
// within it; they are left out, so that what has no decay in it is exactly zero.
//
// One block per (chunk, head), all products in float32 FMA from shared memory; the
// decays run as products along the chunk, so zeros and per-channel decays need no case
// of their own.  Bound by FMA issue and shared-memory reads.
#include "seed_scan_pass.cuh"
#include "seed_scan_prep.cuh"

namespace seed {

namespace {

constexpr int kNT = 256;

template <int DK, int DV>
struct GradSmem {
  static constexpr int PK = DK + 4, PV = DV + 4;     // padded pitches (float4 rows, spread banks)
  static constexpr int CT = 16;                      // state columns per tile
  static constexpr int PT = CT + 4;
  static constexpr int PX = kChunk + 4;
  float q[kChunk * PK], k[kChunk * PK];
  union {
    struct { float d_o[kChunk * PV], w[kChunk * PV], dw[kChunk * PV]; } in;
    struct { float dq[kChunk * PK], h[kChunk * PK], c[kChunk * PK]; } out;
  };
  union {
    struct { float S0[DK * PT], dS[DK * PT]; } t;
    struct { float X[kChunk * PX], Y[kChunk * PX]; } xy;
  };
  float alpha[kChunk], beta[kChunk], kh[kChunk], xd[kChunk], val[8];
  float E[kNT];
  float red[8][kChunk][2];
};

// Sum over groups of G consecutive lanes (G = min(32, DK)); every lane gets it.
template <int G>
SEED_DEV float lanes_sum(float x) { return group_sum<G>(x); }

// The sums over the chunk, the outputs and the decays' gradients, from q, k, the state's
// products (sm.out), X and Y (sm.xy) in shared memory.  E: (S0 dS^T)_cc in thread c < DK.
template <int FORM, int DK, int NT, typename Sm>
SEED_DEV void grad_sums(const ScanParams& p, const ChunkAt& ck, int h, Sm& sm, float E) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  constexpr int PK = Sm::PK, PX = Sm::PX;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n = ck.n, hk = h / (p.H / p.HK);
  const float* al = p.alpha;
  // ---- sums over the chunk: a thread owns channel c and every NG-th block of 4 rows
  constexpr int NG = NT / DK;
  constexpr int LG = DK < 32 ? DK : 32;
  const int c = tid % DK, grp = tid / DK;
  const float* arow = KDA ? al + (ck.first * p.H + h) * DK + c : nullptr;
  const long long astep = (long long)p.H * DK;
  auto dec = [&](int i) -> float {     // decay of token i (1 behind the chunk's tokens)
    if constexpr (KDA) return i < n ? arow[i * astep] : 1.f;
    else return sm.alpha[i];
  };
  float Epart = 0.f;
  for (int i0 = 4 * grp; i0 < kChunk; i0 += 4 * NG) {
    // rows i0 .. i0+3 against columns j <= i0, then the few inside the block
    float sq[4] = {}, sh[4] = {};
    float f = 1.f;
#pragma unroll 4
    for (int j = i0; j >= 0; --j) {
      const float t = f * sm.k[j * PK + c];
      const float4 x = ld4(&sm.xy.X[j * PX + i0]);
      sq[0] = fmaf(x.x, t, sq[0]); sq[1] = fmaf(x.y, t, sq[1]);
      sq[2] = fmaf(x.z, t, sq[2]); sq[3] = fmaf(x.w, t, sq[3]);
      if constexpr (!M2) {
        const float4 y = ld4(&sm.xy.Y[j * PX + i0]);
        sh[0] = fmaf(y.x, t, sh[0]); sh[1] = fmaf(y.y, t, sh[1]);
        sh[2] = fmaf(y.z, t, sh[2]); sh[3] = fmaf(y.w, t, sh[3]);
      }
      f *= dec(j);
    }
    // f = B_i0; S0's part joins here
    const float d1 = dec(i0 + 1), d2 = dec(i0 + 2), d3 = dec(i0 + 3);
    const float fr[4] = {1.f, d1, d1 * d2, d1 * d2 * d3};
    float k4[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int at = (i0 + a) * PK + c;
      sq[a] = fr[a] * fmaf(f, sm.out.dq[at], sq[a]);
      if constexpr (!M2) sh[a] = fr[a] * fmaf(f, sm.out.h[at], sh[a]);
      k4[a] = sm.k[at];
    }
#pragma unroll
    for (int b = 1; b < 4; ++b) {      // column i0 + b, rows i0 + b .. i0 + 3
      float t = k4[b];
#pragma unroll
      for (int a = b; a < 4; ++a) {
        if (a > b) t *= a == 2 ? d2 : d3;
        sq[a] = fmaf(sm.xy.X[(i0 + b) * PX + i0 + a], t, sq[a]);
        if constexpr (!M2) sh[a] = fmaf(sm.xy.Y[(i0 + b) * PX + i0 + a], t, sh[a]);
      }
    }
    // columns i0 .. i0+3 against row i0+3, then four rows behind it at a time (their X and
    // Y are one float4 per column), then the few inside the block
    float sc[4] = {};
    f = 1.f;
    {
      const float tq = sm.q[(i0 + 3) * PK + c];
      const float tk = M2 ? 0.f : -sm.beta[i0 + 3] * sm.k[(i0 + 3) * PK + c];
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        sc[a] = sm.xy.X[(i0 + a) * PX + i0 + 3] * tq;
        if constexpr (!M2) sc[a] = fmaf(sm.xy.Y[(i0 + a) * PX + i0 + 3], tk, sc[a]);
      }
    }
#pragma unroll 1
    for (int m = i0 + 4; m < kChunk; m += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        x[a] = ld4(&sm.xy.X[(i0 + a) * PX + m]);
        if constexpr (!M2) y[a] = ld4(&sm.xy.Y[(i0 + a) * PX + m]);
      }
      const float4 be4 = ld4(&sm.beta[m]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f *= dec(m + e);
        const float tq = f * sm.q[(m + e) * PK + c];
        const float tk = M2 ? 0.f : -f * (&be4.x)[e] * sm.k[(m + e) * PK + c];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          sc[a] = fmaf((&x[a].x)[e], tq, sc[a]);
          if constexpr (!M2) sc[a] = fmaf((&y[a].x)[e], tk, sc[a]);
        }
      }
    }
    const float br[4] = {d1 * d2 * d3, d2 * d3, d3, 1.f};     // D between column i0 + a and row i0 + 3
    float vs[4], kh[4], last[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int at = (i0 + a) * PK + c;
      const float end = br[a] * f * sm.out.c[at];              // D_Ci (dS w_i)
      const bool crosses = i0 + a < n - 1;
      if (crosses) Epart = fmaf(k4[a], end, Epart);
      sc[a] = fmaf(br[a], sc[a], crosses ? end : 0.f);
      last[a] = crosses ? 0.f : end;
    }
#pragma unroll
    for (int b = 0; b < 3; ++b) {      // row i0 + b, columns i0 .. i0 + b
      float tq = sm.q[(i0 + b) * PK + c];
      float tk = M2 ? 0.f : -sm.beta[i0 + b] * k4[b];
#pragma unroll
      for (int a = b; a >= 0; --a) {
        if (a < b) {
          const float d = a == 0 ? d1 : d2;
          tq *= d;
          tk *= d;
        }
        sc[a] = fmaf(sm.xy.X[(i0 + a) * PX + i0 + b], tq, sc[a]);
        if constexpr (!M2) sc[a] = fmaf(sm.xy.Y[(i0 + a) * PX + i0 + b], tk, sc[a]);
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int i = i0 + a;
      const float be = sm.beta[i];
      const float qi = sm.q[i * PK + c];
      const float ci = fmaf(sm.xd[i], qi, sc[a]) + last[a];
      const float dk = M2 ? ci : fmaf(-be, sh[a], ci);
      const float dq = fmaf(sm.xd[i], k4[a], sq[a]);
      kh[a] = M2 ? 0.f : k4[a] * sh[a];
      vs[a] = qi * sq[a] - be * kh[a] - k4[a] * sc[a];
      if (i < n) {
        if (p.part != nullptr) {
          const long long at = ((ck.first + i) * p.H + h) * DK + c;
          p.part[at] = dq;
          p.part[p.tokens * p.H * DK + at] = dk;
        } else {
          const long long at = ((ck.first + i) * p.HK + hk) * DK + c;
          act_st(p.dq, at, dq, p.elem);
          act_st(p.dk_, at, dk, p.elem);
        }
      }
      if constexpr (!M2) kh[a] = lanes_sum<LG>(kh[a]);
      if constexpr (KDA) sm.out.dq[i * PK + c] = vs[a];      // this thread alone reads and writes that element
      else vs[a] = lanes_sum<LG>(vs[a]);
      if ((c & (LG - 1)) == 0) {
        sm.red[c / LG][i][0] = kh[a];
        sm.red[c / LG][i][1] = vs[a];
      }
    }
  }
  sm.E[tid] = Epart;
  __syncthreads();
  // ---- dbeta, and the suffix sums of the decays' gradients
  constexpr int NR = DK / LG;
  if (tid < kChunk && tid < n) {
    float x = 0.f;
    if constexpr (!M2) {
#pragma unroll
      for (int r = 0; r < NR; ++r) x += sm.red[r][tid][0];
    }
    p.dbeta[(ck.first + tid) * p.H + h] = sm.kh[tid] - x;
  }
  if (tid < (DK < 32 ? 32 : DK)) {     // whole warps: the sums below are warp-wide
    float e = 0.f;
    if (tid < DK) {
      float BC = 1.f;
#pragma unroll 16
      for (int i = 0; i < n; ++i) BC *= dec(i);
      e = BC * E;
#pragma unroll
      for (int g = 0; g < NG; ++g) e += sm.E[g * DK + tid];
    }
    if constexpr (KDA) {
      if (tid < DK) {
        for (int i = n - 1; i >= 0; --i) {
          e += sm.out.dq[i * PK + tid];
          p.dlog_alpha[((ck.first + i) * p.H + h) * DK + tid] = dec(i) == 0.f ? 0.f : e;
        }
      }
    } else {
      e = lanes_sum<LG>(e);
      if (tid < DK && (tid & (LG - 1)) == 0) sm.val[tid / LG] = e;
    }
  }
  if constexpr (!KDA) {
    __syncthreads();
    if (tid < 32) {
      // suffix sums of 64 row values, two per lane
      float e = 0.f;
#pragma unroll
      for (int r = 0; r < NR; ++r) e += sm.val[r];
      float hi = 0.f, lo = 0.f;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        lo += sm.red[r][2 * lane][1];
        hi += sm.red[r][2 * lane + 1][1];
      }
      float tot = lo + hi;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, tot, off);
        if (lane + off < 32) tot += x;
      }
      // an inclusive sum of pairs: the odd token leaves its even neighbour's value out
      float next = __shfl_down_sync(0xffffffffu, tot, 1);
      if (lane == 31) next = 0.f;
      if (2 * lane < n) p.dlog_alpha[(ck.first + 2 * lane) * p.H + h] = sm.alpha[2 * lane] == 0.f ? 0.f : e + tot;
      if (2 * lane + 1 < n)
        p.dlog_alpha[(ck.first + 2 * lane + 1) * p.H + h] = sm.alpha[2 * lane + 1] == 0.f ? 0.f : e + (hi + next);
    }
  }
}

template <int FORM, int DK, int DV>
__global__ void __launch_bounds__(kNT, 1) scan_grad_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = GradSmem<DK, DV>;
  constexpr int PK = Sm::PK, PV = Sm::PV, PT = Sm::PT, PX = Sm::PX, CT = Sm::CT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / p.H, h = blockIdx.x - slot * p.H;
  ChunkAt ck;
  if (!chunk_at(p, slot, &ck)) return;
  const int n = ck.n;
  const int hk = h / (p.H / p.HK);
  const long long mat = (long long)DK * DV;
  const float* S0 = p.chunk_S + ((long long)slot * p.H + h) * mat;
  const float* dS = p.chunk_dS + ((long long)slot * p.H + h) * mat;
  const float* al = p.alpha;

  // ---- inputs; rows behind the chunk's tokens are zero
  act_type(p.elem, [&](auto tag) {
    using E = decltype(tag);
#pragma unroll 4
    for (int e = tid; e < kChunk * DK / 4; e += kNT) {
      const int i = e / (DK / 4), c = 4 * (e % (DK / 4));
      float4 a = zero4(), b = zero4();
      if (i < n) {
        const long long at = ((ck.first + i) * p.HK + hk) * DK + c;
        a = fac_ld4(static_cast<const E*>(p.q) + at);
        b = fac_ld4(static_cast<const E*>(p.k) + at);
      }
      st4(&sm.q[i * PK + c], a);
      st4(&sm.k[i * PK + c], b);
    }
#pragma unroll 4
    for (int e = tid; e < kChunk * DV / 4; e += kNT) {
      const int i = e / (DV / 4), c = 4 * (e % (DV / 4));
      float4 a = zero4(), b = zero4(), d = zero4();
      if (i < n) {
        const long long at = ((ck.first + i) * p.H + h) * DV + c;
        a = fac_ld4(static_cast<const E*>(p.d_o) + at);
        b = ld4(p.w + at);
        d = ld4(p.dw + at);
      }
      st4(&sm.in.d_o[i * PV + c], a);
      st4(&sm.in.w[i * PV + c], b);
      st4(&sm.in.dw[i * PV + c], d);
    }
  });
  if (tid < kChunk) {
    sm.beta[tid] = tid < n ? p.beta[(ck.first + tid) * p.H + h] : 0.f;
    if constexpr (!KDA) sm.alpha[tid] = tid < n ? al[(ck.first + tid) * p.H + h] : 1.f;
  }
  __syncthreads();

  // ---- dv and v . dw, a warp per row
  for (int i = warp; i < n; i += kNT / 32) {
    const long long row = ((ck.first + i) * p.H + h) * DV;
    float x = 0.f;
    for (int c = lane; c < DV; c += 32) {
      const float d = sm.in.dw[i * PV + c];
      x = fmaf(act_ld(p.v, row + c, p.elem), d, x);
      act_st(p.dv_, row + c, sm.beta[i] * d, p.elem);
    }
    x = group_sum<32>(x);
    if (lane == 0) sm.kh[i] = x;
  }

  // ---- S0 do, S0 dw, dS w: thread tile of 4 rows x DK / 16 columns
  constexpr int NC = DK / 16;
  const int ty = tid >> 4, tx = tid & 15;
  float aq[4][NC] = {}, ah[4][NC] = {}, ac[4][NC] = {};
  float E = 0.f;         // thread c < DK: (S0 dS^T)_cc
  for (int j0 = 0; j0 < DV; j0 += CT) {
    __syncthreads();
    for (int e = tid; e < DK * CT / 4; e += kNT) {
      const int c = e / (CT / 4), jj = 4 * (e % (CT / 4));
      st4(&sm.t.S0[c * PT + jj], ld4(S0 + (long long)c * DV + j0 + jj));
      st4(&sm.t.dS[c * PT + jj], ld4(dS + (long long)c * DV + j0 + jj));
    }
    __syncthreads();
    if (tid < DK) {
#pragma unroll
      for (int jj = 0; jj < CT; jj += 4) E += dot4(ld4(&sm.t.S0[tid * PT + jj]), ld4(&sm.t.dS[tid * PT + jj]));
    }
#pragma unroll
    for (int jj = 0; jj < CT; jj += 4) {
      float4 xo[4], xd[4], xw[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int at = (ty + 16 * a) * PV + j0 + jj;
        xo[a] = ld4(&sm.in.d_o[at]);
        if constexpr (!M2) xd[a] = ld4(&sm.in.dw[at]);
        xw[a] = ld4(&sm.in.w[at]);
      }
#pragma unroll
      for (int b = 0; b < NC; ++b) {
        const float4 s = ld4(&sm.t.S0[(tx + 16 * b) * PT + jj]);
        const float4 g = ld4(&sm.t.dS[(tx + 16 * b) * PT + jj]);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          aq[a][b] += dot4(xo[a], s);
          if constexpr (!M2) ah[a][b] += dot4(xd[a], s);
          ac[a][b] += dot4(xw[a], g);
        }
      }
    }
  }
  __syncthreads();
  // ---- X and Y, kept as [column j][row i] (a row block of four is one float4)
  {
    float X[4][4] = {}, Y[4][4] = {};
    for (int jj = 0; jj < DV; jj += 4) {
      float4 xo[4], xd[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        xo[a] = ld4(&sm.in.d_o[(ty + 16 * a) * PV + jj]);
        if constexpr (!M2) xd[a] = ld4(&sm.in.dw[(ty + 16 * a) * PV + jj]);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float4 w = ld4(&sm.in.w[(tx + 16 * b) * PV + jj]);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          X[a][b] += dot4(xo[a], w);
          if constexpr (!M2) Y[a][b] += dot4(xd[a], w);
        }
      }
    }
    // (the state tiles X and Y overlay were last read before the barrier above)
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = ty + 16 * a, j = tx + 16 * b;
        sm.xy.X[j * PX + i] = j < i ? X[a][b] : 0.f;
        if (i == j) sm.xd[i] = X[a][b];
        if constexpr (!M2) sm.xy.Y[j * PX + i] = j < i ? Y[a][b] : 0.f;
      }
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < NC; ++b) {
      const int at = (ty + 16 * a) * PK + tx + 16 * b;
      sm.out.dq[at] = aq[a][b];
      if constexpr (!M2) sm.out.h[at] = ah[a][b];
      sm.out.c[at] = ac[a][b];
    }
  __syncthreads();

  grad_sums<FORM, DK, kNT>(p, ck, h, sm, E);
}

// The same with the products of the states, X and Y on the tensor cores (two-term fp16,
// seed_umma.cuh), for d_k, d_v in {64, 128}.  Operands are row-scaled K-major tiles along
// the value channels: OD = [do; dw], W = w, and S0, then dS in the same place:
//     S0 OD^T (key channel x 128 tokens), OD W^T (X and Y), dS W^T (key channel x 64 tokens)
// The results replace the tiles in shared memory; the sums over the chunk are as above.
// Measured: 1,430 chunks x heads of 128 x 128 bf16 460 us (all in float32 FMA: 900), now
// bound by the shared-memory reads of the sums over the chunk (67 % of their peak).
// threads of the tensor-core kernel: its loops over shared memory are bound by latency
constexpr int kGradThreads = 512;

template <int DK, int DV>
struct GradUmmaSmem {
  static constexpr int PK = DK + 4, PX = kChunk + 4;
  static constexpr int OD = DV * 256, W = DV * 128, SX = DV * 256;      // one term each
  union {
    struct {
      alignas(1024) unsigned char od[2 * OD], w[2 * W], sx[2 * SX];
    } tile;
    struct {
      alignas(1024) float q[kChunk * PK];
      float k[kChunk * PK];
      struct { float dq[kChunk * PK], h[kChunk * PK], c[kChunk * PK]; } out;
      struct { float X[kChunk * PX], Y[kChunk * PX]; } xy;
    };
  };
  float alpha[kChunk], beta[kChunk], kh[kChunk], xd[kChunk], val[8];
  float E[kGradThreads];
  float red[8][kChunk][2];
  float inv_od[128], inv_w[kChunk], inv_s[128], Epart[128];
  uint64_t done[2];
  uint32_t tmem;
  int dead;
};

template <int FORM, int DK, int DV, typename T>
__global__ void __launch_bounds__(kGradThreads, 1) scan_grad_umma_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = GradUmmaSmem<DK, DV>;
  constexpr int kNT = kGradThreads;
  constexpr int PK = Sm::PK, PX = Sm::PX;
  extern __shared__ unsigned char smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / p.H, h = blockIdx.x - slot * p.H;
  ChunkAt ck;
  if (!chunk_at(p, slot, &ck)) return;
  const int n = ck.n, hk = h / (p.H / p.HK);
  const long long mat = (long long)DK * DV;
  const float* S0 = p.chunk_S + ((long long)slot * p.H + h) * mat;
  const float* dS = p.chunk_dS + ((long long)slot * p.H + h) * mat;
  if (tid == 0) {
    mbar_init(&sm.done[0], 1);
    mbar_init(&sm.done[1], 1);
    fence_mbar_init();
    sm.dead = 0;
  }
  if (warp == 0) tmem_alloc(&sm.tmem, 256);

  // ---- operand tiles; a thread holds eight value channels of every RPI-th row
  constexpr int LPR = DV / 8, RPI = kNT / LPR, IT = kChunk / RPI;
  const int r0 = tid / LPR, c0 = 8 * (tid % LPR);
  const long long row = (ck.first + r0) * p.H + h, step = (long long)RPI * p.H;
  const int left = (n - r0 + RPI - 1) / RPI;
  if (tid < kChunk) {
    sm.beta[tid] = tid < n ? p.beta[(ck.first + tid) * p.H + h] : 0.f;
    if constexpr (!KDA) sm.alpha[tid] = tid < n ? p.alpha[(ck.first + tid) * p.H + h] : 1.f;
  }
  {
    float a[IT][8], b[IT][8], v[IT][8];
    act_ld8_rows(static_cast<const T*>(p.d_o) + row * DV + c0, step * DV, left, a);
    act_ld8_rows(p.dw + row * DV + c0, step * DV, left, b);
    act_ld8_rows(static_cast<const T*>(p.v) + row * DV + c0, step * DV, left, v);
    tile_rows<true, LPR, RPI, IT>(sm.tile.od, Sm::OD, 128, 0, sm.inv_od, a, r0, c0, nullptr, 0);
    tile_rows<true, LPR, RPI, IT>(sm.tile.od, Sm::OD, 128, kChunk, sm.inv_od + kChunk, b, r0, c0, nullptr, 0);
    act_ld8_rows(p.w + row * DV + c0, step * DV, left, a);
    tile_rows<true, LPR, RPI, IT>(sm.tile.w, Sm::W, kChunk, 0, sm.inv_w, a, r0, c0, nullptr, 0);
    // dv and v . dw
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int i = r0 + it * RPI;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x = fmaf(v[it][e], b[it][e], x);
#pragma unroll
      for (int off = LPR / 2; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (c0 == 0) sm.kh[i] = x;
      if (i < n) {
        const float be = p.beta[(ck.first + i) * p.H + h];
        const long long at = (row + it * step) * DV + c0;
        act_st4(p.dv_, at, make_float4(be * b[it][0], be * b[it][1], be * b[it][2], be * b[it][3]), p.elem);
        act_st4(p.dv_, at + 4, make_float4(be * b[it][4], be * b[it][5], be * b[it][6], be * b[it][7]), p.elem);
      }
    }
  }
  auto state_tile = [&](const float* M, bool second) {
#pragma unroll 1
    for (int x = 0; x < DK; x += kChunk) {
      float a[IT][8], b[IT][8];
      act_ld8_rows(M + (long long)(x + r0) * DV + c0, (long long)RPI * DV, IT, a);
      if (second) {
        act_ld8_rows(S0 + (long long)(x + r0) * DV + c0, (long long)RPI * DV, IT, b);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          float e = 0.f;
#pragma unroll
          for (int y = 0; y < 8; ++y) e = fmaf(a[it][y], b[it][y], e);
#pragma unroll
          for (int off = LPR / 2; off >= 1; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
          if (c0 == 0) sm.Epart[x + r0 + it * RPI] = e;
        }
      }
      tile_rows<true, LPR, RPI, IT>(sm.tile.sx, Sm::SX, 128, x, sm.inv_s + x, a, r0, c0, nullptr, 0);
    }
  };
  state_tile(S0, false);
  fence_proxy_async_smem();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tm = sm.tmem;
  constexpr uint32_t kSO = 0, kXY = 128, kSW = 192;      // accumulators' columns
  const auto step128 = [](int ks) { return (uint32_t)((ks >> 2) * 16384 + (ks & 3) * 32); };
  const auto step64 = [](int ks) { return (uint32_t)((ks >> 2) * 8192 + (ks & 3) * 32); };
  if (tid == 0) {
    const uint64_t od = umma_desc(smem_addr(sm.tile.od), 16), w = umma_desc(smem_addr(sm.tile.w), 16);
    const uint64_t sx = umma_desc(smem_addr(sm.tile.sx), 16);
    product_ss<DV / 16, umma_idesc(128, M2 ? 64 : 128, false)>(tm + kSO, sx, Sm::SX, step128, od, Sm::OD, step128);
    umma_commit(&sm.done[0]);
    product_ss<DV / 16, umma_idesc(128, 64, false)>(tm + kXY, od, Sm::OD, step128, w, Sm::W, step64);
    // (dS's tile takes S0's place; its product is issued below)
  }
  __syncwarp();
  pass_wait(&sm.done[0], 0, &sm.dead, p.status);
  const int j = 32 * (warp & 3) + lane, part = warp >> 2;      // this thread's lane, and its quarter of the columns
  const uint32_t lanes = tm + ((uint32_t)(32 * (warp & 3)) << 16);
  const float inv_s0 = sm.inv_s[j < DK ? j : 0];
  __syncthreads();
  state_tile(dS, true);
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    const uint64_t w = umma_desc(smem_addr(sm.tile.w), 16), sx = umma_desc(smem_addr(sm.tile.sx), 16);
    product_ss<DV / 16, umma_idesc(128, 64, false)>(tm + kSW, sx, Sm::SX, step128, w, Sm::W, step64);
    umma_commit(&sm.done[1]);
  }
  __syncwarp();
  pass_wait(&sm.done[1], 0, &sm.dead, p.status);
  tmem_fence_after();
  // ---- results and q, k into the tiles' place (the scales stay where they are)
  const float inv_ds = sm.inv_s[j < DK ? j : 0];
  const float E = tid < DK ? sm.Epart[tid] : 0.f;
  __syncthreads();
  {
    const int x = 16 * part;
    float a[16], b[16], c[16], y[16];
    tmem_ld16(lanes + kSO + x, a);
    if constexpr (!M2) tmem_ld16(lanes + kSO + 64 + x, b);
    tmem_ld16(lanes + kSW + x, c);
    tmem_ld16(lanes + kXY + x, y);
    tmem_wait_ld();
    if (j < DK) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int i = x + e;
        sm.out.dq[i * PK + j] = a[e] * (inv_s0 * sm.inv_od[i]);
        if constexpr (!M2) sm.out.h[i * PK + j] = b[e] * (inv_s0 * sm.inv_od[kChunk + i]);
        sm.out.c[i * PK + j] = c[e] * (inv_ds * sm.inv_w[i]);
      }
    }
    // lane i: X_i. for i < 64, Y_(i-64). behind
    const int i = j & 63;
    float* xy = j < kChunk ? sm.xy.X : sm.xy.Y;
    const float si = sm.inv_od[j];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float v = y[e] * (si * sm.inv_w[x + e]);
      xy[(x + e) * PX + i] = x + e < i ? v : 0.f;
      if (x + e == i && j < kChunk) sm.xd[i] = v;
    }
  }
  tmem_fence_before();
  {
    constexpr int LPK = DK / 8, RPK = kNT / LPK, ITK = kChunk / RPK;
    const int rk = tid / LPK, ck0 = 8 * (tid % LPK);
    float a[ITK][8], b[ITK][8];
    const long long at = ((ck.first + rk) * p.HK + hk) * DK + ck0, stp = (long long)RPK * p.HK * DK;
    act_ld8_rows(static_cast<const T*>(p.q) + at, stp, (n - rk + RPK - 1) / RPK, a);
    act_ld8_rows(static_cast<const T*>(p.k) + at, stp, (n - rk + RPK - 1) / RPK, b);
#pragma unroll
    for (int it = 0; it < ITK; ++it) {
      float* q = &sm.q[(rk + it * RPK) * PK + ck0];
      float* k = &sm.k[(rk + it * RPK) * PK + ck0];
      st4(q, make_float4(a[it][0], a[it][1], a[it][2], a[it][3]));
      st4(q + 4, make_float4(a[it][4], a[it][5], a[it][6], a[it][7]));
      st4(k, make_float4(b[it][0], b[it][1], b[it][2], b[it][3]));
      st4(k + 4, make_float4(b[it][4], b[it][5], b[it][6], b[it][7]));
    }
  }
  __syncthreads();
  if (warp == 0) {
    tmem_fence_after();
    tmem_free(tm, 256);
  }
  grad_sums<FORM, DK, kNT>(p, ck, h, sm, E);
}

__global__ void __launch_bounds__(256) scan_share_kernel(const ScanParams p) {
  const long long per = p.tokens * p.HK * (p.dk / 4);
  const int rep = p.H / p.HK;
  for (long long e = blockIdx.x * 256ll + threadIdx.x; e < 2 * per; e += gridDim.x * 256ll) {
    const int which = e >= per;
    const long long x = e - which * per;
    const int c = 4 * (int)(x % (p.dk / 4));
    const long long th = x / (p.dk / 4);                // token * HK + key head
    const long long t = th / p.HK;
    if (t < p.offsets[0] || t >= p.offsets[p.seqs]) continue;
    const float* src = p.part + which * p.tokens * p.H * p.dk + th * rep * p.dk + c;
    float4 s = zero4();
    for (int r = 0; r < rep; ++r) s = fma4(1.f, ld4(src + (long long)r * p.dk), s);
    act_st4(which ? p.dk_ : p.dq, th * p.dk + c, s, p.elem);
  }
}

template <int FORM, int DK, int DV>
int launch_grad_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  constexpr size_t bytes = sizeof(GradSmem<DK, DV>);
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_grad_kernel<FORM, DK, DV>), bytes, &dev)) return rc;
  const long long blocks = (long long)p.slots * p.H;
  if (blocks > 0x7fffffffLL) return SEED_ERR_SHAPE;
  scan_grad_kernel<FORM, DK, DV><<<(unsigned)blocks, kNT, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

template <int FORM, int DK, int DV, typename T>
int launch_grad_umma_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  constexpr size_t need = sizeof(GradUmmaSmem<DK, DV>) + 1024;
  constexpr size_t bytes = need < 116 * 1024 ? 116 * 1024 : need;      // one block per SM: tensor memory
  static_assert(bytes <= 227 * 1024, "shared memory");
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_grad_umma_kernel<FORM, DK, DV, T>), bytes, &dev)) return rc;
  scan_grad_umma_kernel<FORM, DK, DV, T><<<(unsigned)(p.slots * p.H), kGradThreads, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace

int launch_scan_grad(const ScanParams& p, int form, cudaStream_t st) {
  if (p.dk >= 64 && p.dv >= 64) {
    return with_factor_type_of(p.elem, [&](auto t) -> int {
      using T = decltype(t);
#define SEED_GRAD(F, K, V) \
  if (form == F && p.dk == K && p.dv == V) return launch_grad_umma_t<F, K, V, T>(p, st);
#define SEED_GRAD_D(F) SEED_GRAD(F, 64, 64) SEED_GRAD(F, 128, 128) SEED_GRAD(F, 128, 64) SEED_GRAD(F, 64, 128)
      SEED_GRAD_D(SEED_GDN)
      SEED_GRAD_D(SEED_KDA)
      SEED_GRAD_D(SEED_MAMBA2)
#undef SEED_GRAD_D
#undef SEED_GRAD
      return SEED_ERR_SHAPE;
    });
  }
#define SEED_GRAD(F, K, V) \
  if (form == F && p.dk == K && p.dv == V) return launch_grad_t<F, K, V>(p, st);
#define SEED_GRAD_D(F) SEED_GRAD(F, 16, 16) SEED_GRAD(F, 32, 32)
  SEED_GRAD_D(SEED_GDN)
  SEED_GRAD_D(SEED_KDA)
  SEED_GRAD_D(SEED_MAMBA2)
#undef SEED_GRAD_D
#undef SEED_GRAD
  return SEED_ERR_SHAPE;
}

int launch_scan_share(const ScanParams& p, cudaStream_t st) {
  const long long n = 2 * p.tokens * p.HK * (p.dk / 4);
  const long long blocks = (n + 255) / 256;
  scan_share_kernel<<<(unsigned)(blocks < 148 * 16 ? (blocks < 1 ? 1 : blocks) : 148 * 16), 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace seed

// seed_scan_step.cu -- the scan token by token: forward, and the reverse recurrence
// of the backward pass.
//
// The columns of S (one per value channel) evolve independently given k, a and beta,
// so a block owns 32 columns of one (sequence, head): four lanes per column, each
// with d_k / 4 rows in registers, in groups of four consecutive rows so that a
// token's k and q are read as float4 broadcasts.  A token costs three passes over
// the registers (S'^T k, the rank-one update, S+^T q) and two quad reductions; the
// chain from token to token is one quad reduction and two FMA passes long.  Tokens
// are staged kStage at a time, the next stage's loads in flight while one is used.
//
// Bound by latency per token for few heads (0.55 us a token at 48 heads of 128 x 128), by
// float32 FMA issue for many (7.4 us a token at 768 heads): used for the shapes and lengths
// the chunked kernels do not take.
#include "seed_scan.cuh"

namespace seed {

namespace {

constexpr int kStage = 8;     // tokens per stage
constexpr int kCols = 32;     // value columns per block
constexpr int kNT = 128;

// Staged inputs of kStage tokens.  x: v forward, do backward.
template <int FORM, int DK>
struct StepStage {
  float k[kStage][DK];
  float q[kStage][DK];
  float a[kStage][FORM == SEED_KDA ? DK : 4];
  float x[kStage][kCols];
  float b[kStage];
};

// Registers that carry the next stage from global to shared memory.
template <int FORM, int DK>
struct StepRegs {
  static constexpr int V4 = kStage * DK / 4;                 // float4 of k (and of q)
  static constexpr int PER = (V4 + kNT - 1) / kNT;
  float4 k[PER], q[PER], a[FORM == SEED_KDA ? PER : 1];
  float4 x;
  float a1, b1;

  // tokens t0 .. t0 + n - 1 of the sequence (n <= kStage), forward order
  SEED_DEV void load(const ScanParams& p, long long row0, int n, int h, int col0, const void* xs, int tid) {
    const int hk = h / (p.H / p.HK);
    act_type(p.elem, [&](auto tag) {
      using T = decltype(tag);
#pragma unroll
      for (int m = 0; m < PER; ++m) {
        const int e = tid + m * kNT;
        const int t = e / (DK / 4), c = 4 * (e % (DK / 4));
        if (e < V4 && t < n) {
          const long long at = ((row0 + t) * p.HK + hk) * DK + c;
          k[m] = fac_ld4(static_cast<const T*>(p.k) + at);
          q[m] = fac_ld4(static_cast<const T*>(p.q) + at);
          if constexpr (FORM == SEED_KDA) a[m] = ld4(p.alpha + ((row0 + t) * p.H + h) * DK + c);
        }
      }
      if (tid < kStage * kCols / 4) {
        const int t = tid / (kCols / 4), c = col0 + 4 * (tid % (kCols / 4));
        if (t < n && c < p.dv) x = fac_ld4(static_cast<const T*>(xs) + ((row0 + t) * p.H + h) * p.dv + c);
      }
    });
    if (tid < n) {
      const long long at = (row0 + tid) * p.H + h;
      b1 = p.beta[at];
      if constexpr (FORM != SEED_KDA) a1 = p.alpha[at];
    }
  }

  SEED_DEV void store(StepStage<FORM, DK>& s, int tid) const {
#pragma unroll
    for (int m = 0; m < PER; ++m) {
      const int e = tid + m * kNT;
      if (e < V4) {
        const int t = e / (DK / 4), c = 4 * (e % (DK / 4));
        st4(&s.k[t][c], k[m]);
        st4(&s.q[t][c], q[m]);
        if constexpr (FORM == SEED_KDA) st4(&s.a[t][c], a[m]);
      }
    }
    if (tid < kStage * kCols / 4) st4(&s.x[tid / (kCols / 4)][4 * (tid % (kCols / 4))], x);
    if (tid < kStage) {
      s.b[tid] = b1;
      if constexpr (FORM != SEED_KDA) s.a[tid][0] = a1;
    }
  }
};

SEED_DEV float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// Copy of a block's columns between registers and a row-major d_k x d_v matrix.
template <int DK>
SEED_DEV void cols_load(float (&S)[DK / 4], const float* M, int dv, int j, int r) {
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[4 * m + e] = M[(long long)(4 * (r + 4 * m) + e) * dv + j];
}
template <int DK>
SEED_DEV bool cols_store(const float (&S)[DK / 4], float* M, int dv, int j, int r) {
  bool ok = true;
#pragma unroll
  for (int m = 0; m < DK / 16; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      M[(long long)(4 * (r + 4 * m) + e) * dv + j] = S[4 * m + e];
      ok = ok && isfinite(S[4 * m + e]);
    }
  return ok;
}

// BACK = false: forward, tokens in order.  BACK = true: the reverse recurrence of
// G, the gradient of the state, tokens from last to first:
//     G += q do^T, dw = G^T k, G -= k (beta dw)^T (not Mamba-2), G <- Diag(a) G
template <int FORM, int DK, bool BACK>
__global__ void __launch_bounds__(kNT) scan_step_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA;
  __shared__ __align__(16) StepStage<FORM, DK> stage[2];
  __shared__ __align__(16) float s_o[kStage][kCols], s_w[kStage][kCols];

  const int tid = threadIdx.x;
  const int slices = (p.dv + kCols - 1) / kCols;
  const int sh = blockIdx.x / slices, slice = blockIdx.x - sh * slices;
  const int seq = sh / p.H, h = sh - (sh / p.H) * p.H;
  const int col0 = slice * kCols;
  const int jl = tid >> 2, r = tid & 3, j = col0 + jl;
  const bool on = j < p.dv;
  const SeqRange sr = seq_range(p, seq, h == 0 && slice == 0 && tid == 0);
  const long long mat = (long long)DK * p.dv;

  float S[DK / 4];
  const float* from = BACK ? p.dS_out : p.S0;
  if (from != nullptr && on) cols_load<DK>(S, from + sh * mat, p.dv, j, r);
  else {
#pragma unroll
    for (int e = 0; e < DK / 4; ++e) S[e] = 0.f;
  }

  const int nst = (sr.len + kStage - 1) / kStage;
  const void* xs = BACK ? p.d_o : p.v;
  StepRegs<FORM, DK> regs = {};
  auto first_of = [&](int i) { return (BACK ? nst - 1 - i : i) * kStage; };
  if (nst > 0) {
    regs.load(p, sr.first + first_of(0), min(kStage, sr.len - first_of(0)), h, col0, xs, tid);
    regs.store(stage[0], tid);
  }
  __syncthreads();
  bool bad = false;
  for (int i = 0; i < nst; ++i) {
    const int t0 = first_of(i), n = min(kStage, sr.len - t0);
    const StepStage<FORM, DK>& sg = stage[i & 1];
    if (i + 1 < nst) {
      const int t1 = first_of(i + 1);
      regs.load(p, sr.first + t1, min(kStage, sr.len - t1), h, col0, xs, tid);
    }
    for (int u = 0; u < n; ++u) {
      const int t = BACK ? n - 1 - u : u;
      const int pos = t0 + t;
      // the state before a chunk's first token, the gradient behind its last one
      if constexpr (!BACK) {
        if (p.chunk_S != nullptr && pos % kChunk == 0 && on)
          cols_store<DK>(S, p.chunk_S + ((long long)(sr.slot0 + pos / kChunk) * p.H + h) * mat, p.dv, j, r);
      } else {
        if ((pos % kChunk == kChunk - 1 || pos == sr.len - 1) && on)
          cols_store<DK>(S, p.chunk_dS + ((long long)(sr.slot0 + pos / kChunk) * p.H + h) * mat, p.dv, j, r);
      }
      const float be = sg.b[t], x = sg.x[t][jl];
      const float g = KDA ? 1.f : sg.a[t][0];
      float k[DK / 4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < DK / 16; ++m) {
        const int at = 4 * (r + 4 * m);
        const float4 kk = ld4(&sg.k[t][at]);
        k[4 * m] = kk.x; k[4 * m + 1] = kk.y; k[4 * m + 2] = kk.z; k[4 * m + 3] = kk.w;
        if constexpr (BACK) {
          const float4 qq = ld4(&sg.q[t][at]);
          S[4 * m] = fmaf(qq.x, x, S[4 * m]); S[4 * m + 1] = fmaf(qq.y, x, S[4 * m + 1]);
          S[4 * m + 2] = fmaf(qq.z, x, S[4 * m + 2]); S[4 * m + 3] = fmaf(qq.w, x, S[4 * m + 3]);
        } else if constexpr (KDA) {
          const float4 al = ld4(&sg.a[t][at]);
          S[4 * m] *= al.x; S[4 * m + 1] *= al.y; S[4 * m + 2] *= al.z; S[4 * m + 3] *= al.w;
        }
        if constexpr (BACK || FORM != SEED_MAMBA2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fmaf(k[4 * m + e], S[4 * m + e], acc[e]);
        }
      }
      float ks = 0.f;
      if constexpr (BACK || FORM != SEED_MAMBA2) ks = quad_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
      if constexpr (BACK) {
        const float dw = ks;
        const float e1 = FORM == SEED_MAMBA2 ? 0.f : -be * dw;
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
          float4 al = make_float4(g, g, g, g);
          if constexpr (KDA) al = ld4(&sg.a[t][4 * (r + 4 * m)]);
          S[4 * m] = al.x * fmaf(k[4 * m], e1, S[4 * m]);
          S[4 * m + 1] = al.y * fmaf(k[4 * m + 1], e1, S[4 * m + 1]);
          S[4 * m + 2] = al.z * fmaf(k[4 * m + 2], e1, S[4 * m + 2]);
          S[4 * m + 3] = al.w * fmaf(k[4 * m + 3], e1, S[4 * m + 3]);
        }
        if (r == 0) s_w[t][jl] = dw;
      } else {
        const float w = FORM == SEED_MAMBA2 ? be * x : be * (x - g * ks);
        float oa[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < DK / 16; ++m) {
          const float4 qq = ld4(&sg.q[t][4 * (r + 4 * m)]);
          const float qv[4] = {qq.x, qq.y, qq.z, qq.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[4 * m + e] = fmaf(k[4 * m + e], w, KDA ? S[4 * m + e] : g * S[4 * m + e]);
            oa[e] = fmaf(qv[e], S[4 * m + e], oa[e]);
          }
        }
        const float o = quad_sum((oa[0] + oa[1]) + (oa[2] + oa[3]));
        if (r == 0) {
          s_o[t][jl] = o;
          s_w[t][jl] = w;
        }
      }
    }
    __syncthreads();
    // this stage's results, rows of up to 32 columns
    if (tid < kStage * kCols / 4) {
      const int t = tid / (kCols / 4), c = 4 * (tid % (kCols / 4));
      if (t < n && col0 + c < p.dv) {
        const long long at = ((sr.first + t0 + t) * p.H + h) * p.dv + col0 + c;
        if constexpr (BACK) {
          st4(p.dw + at, ld4(&s_w[t][c]));
        } else {
          const float4 ov = ld4(&s_o[t][c]);
          if (p.o != nullptr) {
            act_st4(p.o, at, ov, p.elem);
            bad = bad || !(act_finite(ov.x, p.elem) && act_finite(ov.y, p.elem) && act_finite(ov.z, p.elem) &&
                           act_finite(ov.w, p.elem));
          }
          if (p.w != nullptr) st4(p.w + at, ld4(&s_w[t][c]));
        }
      }
    }
    if (i + 1 < nst) regs.store(stage[(i + 1) & 1], tid);
    __syncthreads();
  }
  float* to = BACK ? p.dS0 : p.S_out;
  if (to != nullptr && on) bad = !cols_store<DK>(S, to + sh * mat, p.dv, j, r) || bad;
  if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
}

template <bool BACK>
int launch_step(const ScanParams& p, int form, cudaStream_t st) {
  const long long blocks = (long long)p.seqs * p.H * ((p.dv + kCols - 1) / kCols);
  if (blocks > 0x7fffffffLL) return SEED_ERR_SHAPE;
#define SEED_STEP(F, K)                                                         \
  if (form == F && p.dk == K) {                                                 \
    scan_step_kernel<F, K, BACK><<<(unsigned)blocks, kNT, 0, st>>>(p);          \
    return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;         \
  }
#define SEED_STEP_K(F) SEED_STEP(F, 16) SEED_STEP(F, 32) SEED_STEP(F, 64) SEED_STEP(F, 128)
  SEED_STEP_K(SEED_GDN)
  SEED_STEP_K(SEED_KDA)
  SEED_STEP_K(SEED_MAMBA2)
#undef SEED_STEP_K
#undef SEED_STEP
  return SEED_ERR_SHAPE;
}

}  // namespace

int launch_scan_step(const ScanParams& p, int form, cudaStream_t st) { return launch_step<false>(p, form, st); }
int launch_scan_step_back(const ScanParams& p, int form, cudaStream_t st) { return launch_step<true>(p, form, st); }

}  // namespace seed

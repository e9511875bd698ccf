// seed_scan_prep.cu -- the two triangular matrices of every chunk of the dense scan,
// for the chunked passes (seed_scan_pass.cu).
//
// With D_ij the product of the decays behind token j up to i,
//     P_ij = sum_c q_i[c] k_j[c] D_ij[c]              (j <= i)
//     A_ij = beta_i sum_c k_i[c] k_j[c] D_ij[c]       (j < i),   T = (I + A)^-1
// so that within a chunk w = T (beta (v - (B k) S0)) and o = (B q) S0 + P w.
//
// Chunks are independent here, so one block per (chunk, key head) fills every SM while
// the passes, which run along the sequence, cannot.  The Gram matrices use the tensor
// cores in tf32: 16-bit inputs are exact in it (one product), float32 ones are split in
// two terms (three products, 2^-22).  One decay per head multiplies the Gram matrix
// afterwards, so the heads that share keys share it; decays per channel go into the
// operands, around the first token of each block of 16 rows (every factor a product of
// decays, so none overflows), and the 16 x 16 diagonal blocks are summed directly.
// T is inverted block by block, 16 -> 32 -> 64: T21 = -T22 A21 T11.
//
// Results go to scratch as the passes' shared-memory images (two-term fp16, 128-byte
// swizzle, one power-of-two scale per row), 32.5 KB per chunk and head.
#include "seed_scan.cuh"
#include "seed_umma.cuh"

namespace seed {

namespace {

constexpr int kNT = 256;
constexpr int PX = kChunk + 4;

template <bool KDA, int DK>
struct PrepSmem {
  static constexpr int PK = DK + 4;
  union {
    struct { float q[kChunk * PK], k[kChunk * PK], a[KDA ? kChunk * PK : 4]; } in;
    struct { float A[kChunk * PX], T[kChunk * PX], P[kChunk * PX], M[32 * 36]; } t;
  };
  float KK[kChunk * PX], QK[kChunk * PX];
  float mv[KDA ? 3 : 1][KDA ? DK : 4];
  float alpha[kChunk], beta[kChunk];
};

SEED_DEV float tf32_hi(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

SEED_DEV void mma_tf32(float (&c)[4], const float (&a)[4], const float (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
        "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}

// One 16 x 8 tile over DK channels: rows r0.. of X, rows n0.. of Y (times m per channel).
template <int DK, bool SPLIT>
SEED_DEV void gram_tile(float (&c)[4], const float* X, const float* Y, const float* m, int r0, int n0, int lane) {
  constexpr int PK = DK + 4;
  const int g = lane >> 2, t = lane & 3;
  c[0] = c[1] = c[2] = c[3] = 0.f;
  const float* x0 = X + (r0 + g) * PK + t;
  const float* x1 = x0 + 8 * PK;
  const float* y0 = Y + (n0 + g) * PK + t;
#pragma unroll 4
  for (int k = 0; k < DK; k += 8) {
    const float a[4] = {x0[k], x1[k], x0[k + 4], x1[k + 4]};
    float b[2] = {y0[k], y0[k + 4]};
    if (m != nullptr) {
      b[0] *= m[k + t];
      b[1] *= m[k + 4 + t];
    }
    if constexpr (SPLIT) {
      const float ah[4] = {tf32_hi(a[0]), tf32_hi(a[1]), tf32_hi(a[2]), tf32_hi(a[3])};
      const float al[4] = {a[0] - ah[0], a[1] - ah[1], a[2] - ah[2], a[3] - ah[3]};
      const float bh[2] = {tf32_hi(b[0]), tf32_hi(b[1])};
      const float bl[2] = {b[0] - bh[0], b[1] - bh[1]};
      mma_tf32(c, al, bh);
      mma_tf32(c, ah, bl);
      mma_tf32(c, ah, bh);
    } else {
      mma_tf32(c, a, b);
    }
  }
}

SEED_DEV void gram_store(const float (&c)[4], float* G, int r0, int n0, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2*>(&G[(r0 + g) * PX + n0 + 2 * t]) = make_float2(c[0], c[1]);
  *reinterpret_cast<float2*>(&G[(r0 + g + 8) * PX + n0 + 2 * t]) = make_float2(c[2], c[3]);
}

// The image of a 64 x 64 matrix (rows of 128 bytes, chunk ^= row % 8; hi, then lo) and
// its rows' inverse scales.  Four threads per row.
SEED_DEV void store_image(unsigned char* img, float* inv, const float* M, int tid) {
  const int i = tid >> 2, qd = tid & 3;
  float x[16], mx = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float4 v = ld4(&M[i * PX + 16 * qd + 4 * e]);
    x[4 * e] = v.x; x[4 * e + 1] = v.y; x[4 * e + 2] = v.z; x[4 * e + 3] = v.w;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(x[e]));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const float s = pow2_scale(mx);
  if (qd == 0) inv[i] = pow2_inverse(s);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 hi, lo;
    uint32_t* h = &hi.x;
    uint32_t* l = &lo.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(s * x[8 * half + 2 * e], s * x[8 * half + 2 * e + 1], h[e], l[e]);
    const int at = i * 128 + (((2 * qd + half) ^ (i & 7)) << 4);
    *reinterpret_cast<uint4*>(img + at) = hi;
    *reinterpret_cast<uint4*>(img + 8192 + at) = lo;
  }
}

// T = (I + A)^-1 of sm.t.A (strictly lower) into sm.t.T.
template <typename Sm>
SEED_DEV void invert(Sm& sm, int tid) {
  float* A = sm.t.A;
  float* T = sm.t.T;
  float* M = sm.t.M;
  for (int e = tid; e < kChunk * kChunk / 4; e += kNT) st4(&T[(e / 16) * PX + 4 * (e % 16)], zero4());
  __syncthreads();
  if (tid < 128) {      // a warp per diagonal block, a lane per column: forward substitution
    const int b = 16 * (tid >> 5), c = tid & 31;
    if (c < 16) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == c ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-A[(b + i) * PX + b + j], x[j], s);
        x[i] = s;
        T[(b + i) * PX + b + c] = s;
      }
    }
  }
  __syncthreads();
  {      // two 32 x 32 blocks, each from its 16 x 16 quarters
    const int b = 32 * (tid >> 7), e = tid & 127, i = e >> 3, c = 2 * (e & 7);
    float m0 = 0.f, m1 = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float a = A[(b + 16 + i) * PX + b + k];
      const float2 t = *reinterpret_cast<const float2*>(&T[(b + k) * PX + b + c]);
      m0 = fmaf(a, t.x, m0);
      m1 = fmaf(a, t.y, m1);
    }
    *reinterpret_cast<float2*>(&M[(b / 2 + i) * 36 + c]) = make_float2(m0, m1);
    __syncthreads();
    m0 = m1 = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float a = T[(b + 16 + i) * PX + b + 16 + k];
      const float2 t = *reinterpret_cast<const float2*>(&M[(b / 2 + k) * 36 + c]);
      m0 = fmaf(-a, t.x, m0);
      m1 = fmaf(-a, t.y, m1);
    }
    *reinterpret_cast<float2*>(&T[(b + 16 + i) * PX + b + c]) = make_float2(m0, m1);
  }
  __syncthreads();
  {      // the 64 x 64 block from its 32 x 32 quarters
    const int i = tid >> 3, c = 4 * (tid & 7);
    float4 m = zero4();
#pragma unroll
    for (int k = 0; k < 32; ++k) m = fma4(A[(32 + i) * PX + k], ld4(&T[k * PX + c]), m);
    st4(&M[i * 36 + c], m);
    __syncthreads();
    m = zero4();
#pragma unroll
    for (int k = 0; k < 32; ++k) m = fma4(-T[(32 + i) * PX + 32 + k], ld4(&M[k * 36 + c]), m);
    st4(&T[(32 + i) * PX + c], m);
  }
  __syncthreads();
}

template <int FORM, int DK, bool SPLIT>
__global__ void __launch_bounds__(kNT) scan_prep_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = PrepSmem<KDA, DK>;
  constexpr int PK = Sm::PK;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rep = p.H / p.HK;
  const int groups = KDA ? p.H : p.HK;      // blocks per chunk
  const int slot = blockIdx.x / groups, grp = blockIdx.x - slot * groups;
  ChunkAt ck;
  if (!chunk_at(p, slot, &ck)) return;
  const int n = ck.n;
  const int hk = KDA ? grp / rep : grp;

  act_type(p.elem, [&](auto tag) {
    using E = decltype(tag);
#pragma unroll
    for (int e = tid; e < kChunk * DK / 4; e += kNT) {
      const int i = e / (DK / 4), c = 4 * (e % (DK / 4));
      float4 q = zero4(), k = zero4(), a = make_float4(1.f, 1.f, 1.f, 1.f);
      if (i < n) {
        const long long at = ((ck.first + i) * p.HK + hk) * DK + c;
        q = fac_ld4(static_cast<const E*>(p.q) + at);
        k = fac_ld4(static_cast<const E*>(p.k) + at);
        if constexpr (KDA) a = ld4(p.alpha + ((ck.first + i) * p.H + grp) * DK + c);
      }
      st4(&sm.in.q[i * PK + c], q);
      st4(&sm.in.k[i * PK + c], k);
      if constexpr (KDA) st4(&sm.in.a[i * PK + c], a);
    }
  });
  __syncthreads();

  if constexpr (!KDA) {
    // 20 tiles of 16 x 8 on or below the diagonal for each matrix, five per warp
    const bool isq = warp < 4;
    if (isq || !M2) {
#pragma unroll 1
      for (int e = 0; e < 5; ++e) {
        const int x = 5 * (warp & 3) + e;
        const int I = x < 8 ? 3 : x < 10 ? 0 : x < 16 ? 2 : 1;
        const int nt = x < 8 ? x : x < 10 ? x - 8 : x < 16 ? x - 10 : x - 16;
        float c[4];
        gram_tile<DK, SPLIT>(c, isq ? sm.in.q : sm.in.k, sm.in.k, nullptr, 16 * I, 8 * nt, lane);
        gram_store(c, isq ? sm.QK : sm.KK, 16 * I, 8 * nt, lane);
      }
    }
  } else {
    // diagonal 16 x 16 blocks: a thread takes columns j and 15 - j of a block over a
    // quarter of the channels (four channels in turn per lane), the decay running with i
    if (tid < 128) {
      const int b = 16 * (tid >> 5), pr = (tid >> 2) & 7, part = tid & 3;
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        const int j = side ? 15 - pr : pr;
        float f[DK / 4];
#pragma unroll
        for (int x = 0; x < DK / 16; ++x) {
          const float4 v = ld4(&sm.in.k[(b + j) * PK + 16 * x + 4 * part]);
          f[4 * x] = v.x; f[4 * x + 1] = v.y; f[4 * x + 2] = v.z; f[4 * x + 3] = v.w;
        }
        for (int i = 0; i < 16; ++i) {
          float sq = 0.f, sk = 0.f;
          if (i >= j) {
#pragma unroll
            for (int x = 0; x < DK / 16; ++x) {
              const int at = (b + i) * PK + 16 * x + 4 * part;
              if (i > j) {
                const float4 a = ld4(&sm.in.a[at]);
                f[4 * x] *= a.x; f[4 * x + 1] *= a.y; f[4 * x + 2] *= a.z; f[4 * x + 3] *= a.w;
              }
              const float4 q = ld4(&sm.in.q[at]), k = ld4(&sm.in.k[at]);
              const float4 ff = make_float4(f[4 * x], f[4 * x + 1], f[4 * x + 2], f[4 * x + 3]);
              sq += dot4(q, ff);
              sk += dot4(k, ff);
            }
          }
          sq += __shfl_xor_sync(0xffffffffu, sq, 1);
          sq += __shfl_xor_sync(0xffffffffu, sq, 2);
          sk += __shfl_xor_sync(0xffffffffu, sk, 1);
          sk += __shfl_xor_sync(0xffffffffu, sk, 2);
          if (i >= j && part == 0) {
            sm.QK[(b + i) * PX + b + j] = sq;
            sm.KK[(b + i) * PX + b + j] = sk;
          }
        }
      }
    }
    __syncthreads();
    // operands around the blocks' first tokens: rows q_i F_i, k_i F_i with F_i the decays
    // behind the block's first token, columns k_j G_j with G_j those up to the next block's
    // first token (in the decays' place), and mv the products over whole blocks
    constexpr int NG = kNT / DK;             // threads per channel
    const int c = tid % DK, hf = tid / DK;
    float nxt[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) nxt[x] = x < 3 ? sm.in.a[16 * (x + 1) * PK + c] : 1.f;
    __syncthreads();
    for (int x = hf; x < 4; x += NG) {
      float a[16], k[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        a[i] = sm.in.a[(16 * x + i) * PK + c];
        k[i] = sm.in.k[(16 * x + i) * PK + c];
      }
      float f = 1.f, g = nxt[x];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i > 0) f *= a[i];
        sm.in.q[(16 * x + i) * PK + c] *= f;
        sm.in.k[(16 * x + i) * PK + c] = k[i] * f;
      }
      if (x == 1 || x == 2) sm.mv[x - 1][c] = f * nxt[x];
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        sm.in.a[(16 * x + i) * PK + c] = k[i] * g;
        g *= a[i];
      }
    }
    __syncthreads();
    if (tid < DK) sm.mv[2][tid] = sm.mv[0][tid] * sm.mv[1][tid];
    __syncthreads();
    // 24 tiles left of the diagonal blocks, three per warp
#pragma unroll 1
    for (int e = 0; e < 3; ++e) {
      const int x = 3 * warp + e;
      const bool isq = x < 12;
      const int y = isq ? x : x - 12;
      const int I = y < 2 ? 1 : y < 6 ? 2 : 3;
      const int nt = y < 2 ? y : y < 6 ? y - 2 : y - 6;
      const int J = nt / 2 + 1;              // the block behind the columns'
      const float* m = J == I ? nullptr : (J == 1 && I == 2) ? sm.mv[0] : J == 2 ? sm.mv[1] : sm.mv[2];
      float cc[4];
      gram_tile<DK, true>(cc, isq ? sm.in.q : sm.in.k, sm.in.a, m, 16 * I, 8 * nt, lane);
      gram_store(cc, isq ? sm.QK : sm.KK, 16 * I, 8 * nt, lane);
    }
  }
  __syncthreads();

  for (int r = 0; r < (KDA ? 1 : rep); ++r) {
    const int h = KDA ? grp : hk * rep + r;
    if (tid < kChunk) {
      const bool in = tid < n;
      sm.beta[tid] = in ? p.beta[(ck.first + tid) * p.H + h] : 0.f;
      if constexpr (!KDA) sm.alpha[tid] = in ? p.alpha[(ck.first + tid) * p.H + h] : 1.f;
    }
    __syncthreads();
    {      // a thread takes column j of a block of 16 rows, the decay running down
      const int j = tid & 63, i0 = 16 * (tid >> 6);
      float f = 1.f;
      if constexpr (!KDA) {
        for (int s = j + 1; s < i0; ++s) f *= sm.alpha[s];
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int i = i0 + x;
        if (!KDA && i > j) f *= sm.alpha[i];
        sm.t.P[i * PX + j] = i >= j ? f * sm.QK[i * PX + j] : 0.f;
        if constexpr (!M2) sm.t.A[i * PX + j] = i > j ? sm.beta[i] * f * sm.KK[i * PX + j] : 0.f;
      }
    }
    unsigned char* img = p.tri + ((long long)slot * p.H + h) * kTriBytes;
    float* inv = reinterpret_cast<float*>(img + 32768);
    if constexpr (!M2) {
      invert(sm, tid);                  // begins with a barrier
      store_image(img, inv, sm.t.T, tid);
    } else {
      __syncthreads();
    }
    store_image(img + 16384, inv + kChunk, sm.t.P, tid);
    __syncthreads();
  }
}

template <int FORM, int DK, bool SPLIT>
int launch_prep_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  constexpr size_t bytes = sizeof(PrepSmem<FORM == SEED_KDA, DK>);
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_prep_kernel<FORM, DK, SPLIT>), bytes, &dev)) return rc;
  const int blocks = p.slots * (FORM == SEED_KDA ? p.H : p.HK);
  scan_prep_kernel<FORM, DK, SPLIT><<<blocks, kNT, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

template <int FORM, int DK>
int launch_prep_k(const ScanParams& p, cudaStream_t st) {
  if constexpr (FORM != SEED_KDA) {      // per-channel decays make the operands float32 in any case
    if (p.elem != SEED_FACTORS_F32) return launch_prep_t<FORM, DK, false>(p, st);
  }
  return launch_prep_t<FORM, DK, true>(p, st);
}

}  // namespace

int launch_scan_prep(const ScanParams& p, int form, cudaStream_t st) {
  if (p.dk != 64 && p.dk != 128) return SEED_ERR_SHAPE;
  const bool big = p.dk == 128;
  switch (form) {
    case SEED_GDN: return big ? launch_prep_k<SEED_GDN, 128>(p, st) : launch_prep_k<SEED_GDN, 64>(p, st);
    case SEED_KDA: return big ? launch_prep_k<SEED_KDA, 128>(p, st) : launch_prep_k<SEED_KDA, 64>(p, st);
    case SEED_MAMBA2: return big ? launch_prep_k<SEED_MAMBA2, 128>(p, st) : launch_prep_k<SEED_MAMBA2, 64>(p, st);
  }
  return SEED_ERR_INVALID_ARG;
}

}  // namespace seed

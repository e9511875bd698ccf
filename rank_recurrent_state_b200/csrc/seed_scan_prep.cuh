// seed_scan_prep.cuh -- what the chunked passes of the dense scan need of every chunk.
//
// With D_ij the product of the decays behind token j up to i, B_i that since the chunk's
// start and E_i that behind token i to its end,
//     P_ij = sum_c q_i[c] k_j[c] D_ij[c]              (j <= i)
//     A_ij = beta_i sum_c k_i[c] k_j[c] D_ij[c]       (j < i),   T = (I + A)^-1
// so that within a chunk w = T (beta (v - (B k) S0)) and o = (B q) S0 + P w.  T, P, k and q
// go to scratch as the passes' shared-memory tiles: fp16 in the 128-byte swizzle, a
// power-of-two scale per row (seed_umma.cuh).  One decay per head leaves k and q as they
// are (the passes apply B_i and E_i to rows and columns), so the heads that share keys
// share their tiles, and 16-bit activations need one fp16 term (a row-scaled fp16 value
// holds bf16's 8 bits exactly down to 2^-14 of the row's scale and is off by at most 2^-25
// of it below).  Decays per channel go into the tiles: B k, B q and E k, two terms each.
//
// Chunks are independent here, so one block per (chunk, key head) -- per (chunk, head) for
// decays per channel -- fills every SM while the passes, which run along the sequence,
// cannot.  The Gram matrices use warp-level matrix products (16-bit activations as they
// are, float32 operands as two tf32 terms): 64 x 64 x d_k per chunk is too little to feed
// tensor memory.  T is inverted block by block, 16 -> 32 -> 64: T21 = -T22 A21 T11.
//
// Measured: 5,400 chunks x heads of 128 bf16 with a decay per head 191 us (two blocks per SM
// at 20,000 cycles each; shared-memory wavefronts 58 % of their peak, half of a block's time
// waits at barriers and for the first loads); 4,096 with decays per channel 616 us (one
// block per SM; the diagonal blocks take 13,000 of its 40,000 cycles).
#pragma once

#include "seed_scan.cuh"
#include "seed_umma.cuh"

namespace seed {

namespace {

// Threads per block: with decays per channel the shared memory has room for one block per SM.
__host__ __device__ constexpr int prep_threads(bool kda) { return kda ? 512 : 256; }
constexpr int PX = kChunk + 4;

// Element type of k and q in shared memory: 16-bit activations stay as they are; with
// decays per channel, or float32 activations, float32.
template <bool KDA, typename T>
using PrepT = typename std::conditional<KDA, float, T>::type;

template <bool KDA, int DK, typename Act>
struct PrepSmem {
  using S = PrepT<KDA, Act>;
  static constexpr int PK = DK + 16 / (int)sizeof(S);      // padded pitch: rows 4 banks apart
  union {
    struct { S q[kChunk * PK], k[kChunk * PK]; float a[KDA ? kChunk * PK : 4]; } in;
    struct { float A[kChunk * PX], T[kChunk * PX], P[kChunk * PX], M[32 * 36]; } t;
  };
  float KK[kChunk * PX], QK[kChunk * PX];
  float mv[KDA ? 3 : 1][KDA ? DK : 4];
  float alpha[kChunk], beta[kChunk], G[kChunk], B[kChunk], E[kChunk], blk[4];
  float invK[kChunk], invQ[kChunk], invE[kChunk];
};

SEED_DEV float tf32_hi(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

SEED_DEV void mma_tf32(float (&c)[4], const float (&a)[4], const float (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
        "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}
template <typename T>
SEED_DEV void mma_16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// One 16 x 8 tile over DK channels: rows r0.. of X, rows n0.. of Y (times m per channel).
template <int DK, typename S>
SEED_DEV void gram_tile(float (&c)[4], const S* X, const S* Y, const float* m, int r0, int n0, int lane) {
  constexpr int PK = DK + 16 / (int)sizeof(S);
  const int g = lane >> 2, t = lane & 3;
  c[0] = c[1] = c[2] = c[3] = 0.f;
  if constexpr (std::is_same<S, float>::value) {
    const float* x0 = X + (r0 + g) * PK + t;
    const float* x1 = x0 + 8 * PK;
    const float* y0 = Y + (n0 + g) * PK + t;
    // Accumulators round towards zero at every step: the small products have one of their
    // own, the others one for each quarter of the channels, added to nearest at the end.
    float lo[4] = {}, hi[4][4] = {};
#pragma unroll
    for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
    for (int k = k4 * (DK / 4); k < (k4 + 1) * (DK / 4); k += 8) {
      const float a[4] = {x0[k], x1[k], x0[k + 4], x1[k + 4]};
      float b[2] = {y0[k], y0[k + 4]};
      if (m != nullptr) {
        b[0] *= m[k + t];
        b[1] *= m[k + 4 + t];
      }
      const float ah[4] = {tf32_hi(a[0]), tf32_hi(a[1]), tf32_hi(a[2]), tf32_hi(a[3])};
      const float al[4] = {a[0] - ah[0], a[1] - ah[1], a[2] - ah[2], a[3] - ah[3]};
      const float bh[2] = {tf32_hi(b[0]), tf32_hi(b[1])};
      const float bl[2] = {b[0] - bh[0], b[1] - bh[1]};
      mma_tf32(lo, al, bh);
      mma_tf32(lo, ah, bl);
      mma_tf32(hi[k4], ah, bh);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = ((hi[0][e] + hi[1][e]) + (hi[2][e] + hi[3][e])) + lo[e];
  } else {
    const S* x0 = X + (r0 + g) * PK + 2 * t;
    const S* x1 = x0 + 8 * PK;
    const S* y0 = Y + (n0 + g) * PK + 2 * t;
    auto w = [](const S* p) { return *reinterpret_cast<const uint32_t*>(p); };
#pragma unroll
    for (int k = 0; k < DK; k += 16) {
      const uint32_t a[4] = {w(x0 + k), w(x1 + k), w(x0 + k + 8), w(x1 + k + 8)};
      const uint32_t b[2] = {w(y0 + k), w(y0 + k + 8)};
      mma_16<S>(c, a, b);
    }
  }
}

SEED_DEV void gram_store(const float (&c)[4], float* G, int r0, int n0, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2*>(&G[(r0 + g) * PX + n0 + 2 * t]) = make_float2(c[0], c[1]);
  *reinterpret_cast<float2*>(&G[(r0 + g + 8) * PX + n0 + 2 * t]) = make_float2(c[2], c[3]);
}

// A 16 x 8 tile of X Y over K terms, X [16][K] and Y [K][8] in shared memory, both as two
// tf32 terms; and its store, times f.
template <int K>
SEED_DEV void tile_product(float (&c)[4], const float* X, int px, const float* Y, int py, int lane) {
  const int g = lane >> 2, t = lane & 3;
  c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
  for (int k = 0; k < K; k += 8) {
    const float a[4] = {X[g * px + k + t], X[(g + 8) * px + k + t], X[g * px + k + t + 4], X[(g + 8) * px + k + t + 4]};
    const float b[2] = {Y[(k + t) * py + g], Y[(k + t + 4) * py + g]};
    const float ah[4] = {tf32_hi(a[0]), tf32_hi(a[1]), tf32_hi(a[2]), tf32_hi(a[3])};
    const float al[4] = {a[0] - ah[0], a[1] - ah[1], a[2] - ah[2], a[3] - ah[3]};
    const float bh[2] = {tf32_hi(b[0]), tf32_hi(b[1])};
    const float bl[2] = {b[0] - bh[0], b[1] - bh[1]};
    mma_tf32(c, al, bh);
    mma_tf32(c, ah, bl);
    mma_tf32(c, ah, bh);
  }
}
SEED_DEV void tile_store(const float (&c)[4], float* D, int pd, float f, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2*>(&D[g * pd + 2 * t]) = make_float2(f * c[0], f * c[1]);
  *reinterpret_cast<float2*>(&D[(g + 8) * pd + 2 * t]) = make_float2(f * c[2], f * c[3]);
}

// Eight values of row `row` of a tile whose panels of 64 channels hold `rows` rows, from
// channel c0 on, already scaled; two: the second term `lo` bytes behind.
template <bool TWO>
SEED_DEV void put8(unsigned char* tile, int lo, int rows, int row, int c0, const float (&x)[8]) {
  const int at = (c0 / 64) * rows * 128 + row * 128 + ((((c0 & 63) >> 3) ^ (row & 7)) << 4);
  uint4 h;
  if constexpr (TWO) {
    uint4 l;
    split2(x[0], x[1], h.x, l.x);
    split2(x[2], x[3], h.y, l.y);
    split2(x[4], x[5], h.z, l.z);
    split2(x[6], x[7], h.w, l.w);
    *reinterpret_cast<uint4*>(tile + lo + at) = l;
  } else {
    const __half2 t[4] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3]), __floats2half2_rn(x[4], x[5]),
                          __floats2half2_rn(x[6], x[7])};
    memcpy(&h, t, 16);
  }
  *reinterpret_cast<uint4*>(tile + at) = h;
}
// The largest of |x| over a row shared by LPR consecutive lanes.
template <int LPR>
SEED_DEV float row_max(const float (&x)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  return m;
}

// Rows r0, r0 + RPI, .. (times f, a matrix of the given pitch, if there is one), scaled,
// into a tile from its row `row0` on, and their inverse scales.
template <bool TWO, int LPR, int RPI, int IT>
SEED_DEV void tile_rows(unsigned char* tile, int lo, int rows, int row0, float* inv, const float (&x)[IT][8], int r0,
                        int c0, const float* f, int pitch) {
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int i = r0 + it * RPI;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[it][e];
    if (f != nullptr) {
      const float4 a = ld4(f + i * pitch + c0), b = ld4(f + i * pitch + c0 + 4);
      y[0] *= a.x; y[1] *= a.y; y[2] *= a.z; y[3] *= a.w;
      y[4] *= b.x; y[5] *= b.y; y[6] *= b.z; y[7] *= b.w;
    }
    const float s = pow2_scale(row_max<LPR>(y));
    if (c0 == 0) inv[i] = pow2_inverse(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= s;
    put8<TWO>(tile, lo, rows, row0 + i, c0, y);
  }
}

// The tile of a 64 x 64 matrix (two terms, 8192 bytes apart) and its rows' inverse scales.
SEED_DEV void store_square(unsigned char* img, float* inv, const float* M, int tid) {      // 256 threads
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = (tid >> 3) + 32 * half, c = 8 * (tid & 7);
    float x[8];
    const float4 a = ld4(&M[i * PX + c]), b = ld4(&M[i * PX + c + 4]);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    const float s = pow2_scale(row_max<8>(x));
    if (c == 0) inv[i] = pow2_inverse(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= s;
    put8<true>(img, 8192, kChunk, i, c, x);
  }
}

// T = (I + A)^-1 of sm.t.A (strictly lower) into sm.t.T, whose upper half is zero.
// Begins and ends with a barrier.
template <typename Sm>
SEED_DEV void invert(Sm& sm, int tid) {
  float* A = sm.t.A;
  float* T = sm.t.T;
  float* M = sm.t.M;
  __syncthreads();
  if ((tid & 31) < 8 && tid < 256) {      // eight columns of a diagonal block per warp: forward substitution
    const int b = 16 * (tid >> 6), c = (tid & 7) + 8 * ((tid >> 5) & 1);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s[2] = {i == c ? 1.f : 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        if (j < i) {
          const float4 a = ld4(&A[(b + i) * PX + b + j]);
          s[0] = fmaf(-a.x, x[j], s[0]);
          if (j + 1 < i) s[1] = fmaf(-a.y, x[j + 1], s[1]);
          if (j + 2 < i) s[0] = fmaf(-a.z, x[j + 2], s[0]);
          if (j + 3 < i) s[1] = fmaf(-a.w, x[j + 3], s[1]);
        }
      }
      x[i] = s[0] + s[1];
      T[(b + i) * PX + b + c] = x[i];
    }
  }
  __syncthreads();
  // The blocks left of the diagonal by warp-level matrix products, a 16 x 8 tile per warp:
  // M = A21 T11, T21 = -T22 M.  (In float32 FMA from shared memory these two products took
  // 2,500 of the 8,700 shared-memory wavefronts of a chunk and head.)
  const int warp = tid >> 5, lane = tid & 31;
  {      // two 32 x 32 blocks, each from its 16 x 16 quarters
    const int b = 32 * ((warp >> 1) & 1), n0 = 8 * (warp & 1);
    float c[4];
    if (warp < 4) {
      tile_product<16>(c, &A[(b + 16) * PX + b], PX, &T[b * PX + b + n0], PX, lane);
      tile_store(c, &M[(b / 2) * 36 + n0], 36, 1.f, lane);
    }
    __syncthreads();
    if (warp < 4) {
      tile_product<16>(c, &T[(b + 16) * PX + b + 16], PX, &M[(b / 2) * 36 + n0], 36, lane);
      tile_store(c, &T[(b + 16) * PX + b + n0], PX, -1.f, lane);
    }
  }
  __syncthreads();
  {      // the 64 x 64 block from its 32 x 32 quarters
    const int i0 = 16 * ((warp >> 2) & 1), n0 = 8 * (warp & 3);
    float c[4];
    if (warp < 8) {
      tile_product<32>(c, &A[(32 + i0) * PX], PX, &T[n0], PX, lane);
      tile_store(c, &M[i0 * 36 + n0], 36, 1.f, lane);
    }
    __syncthreads();
    if (warp < 8) {
      tile_product<32>(c, &T[(32 + i0) * PX + 32], PX, &M[n0], 36, lane);
      tile_store(c, &T[(32 + i0) * PX + n0], PX, -1.f, lane);
    }
  }
  __syncthreads();
}

template <int FORM, int DK, typename T>
__global__ void __launch_bounds__(prep_threads(FORM == SEED_KDA)) scan_prep_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  constexpr bool TWO = scan_two_terms(FORM, std::is_same<T, float>::value);
  constexpr int kNT = prep_threads(KDA);
  using Sm = PrepSmem<KDA, DK, T>;
  using S = typename Sm::S;
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
  unsigned char* kq = p.kq + (long long)blockIdx.x * kq_bytes(FORM, DK, TWO);
  constexpr int kTerm = DK * 256;      // one term of the k and q rows

  // ---- k and q; a thread holds eight channels of every RPI-th row
  constexpr int LPR = DK / 8, RPI = kNT / LPR, IT = kChunk / RPI;
  const int r0 = tid / LPR, c0 = 8 * (tid % LPR);
  float k[IT][8], q[IT][8];
  {
    const long long at = ((ck.first + r0) * p.HK + hk) * DK + c0, step = (long long)RPI * p.HK * DK;
    const int left = (n - r0 + RPI - 1) / RPI;
    act_ld8_rows(static_cast<const T*>(p.k) + at, step, left, k);
    act_ld8_rows(static_cast<const T*>(p.q) + at, step, left, q);
  }
  auto keep = [&](S* dst, int i, const float (&x)[8]) {
    S t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = fac_from_f<S>(x[e]);      // exact
    S* at = dst + i * PK + c0;
#pragma unroll
    for (int y = 0; y < 8 * (int)sizeof(S) / 16; ++y) {
      uint4 raw;
      memcpy(&raw, reinterpret_cast<const unsigned char*>(t) + 16 * y, 16);
      reinterpret_cast<uint4*>(at)[y] = raw;
    }
  };
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    keep(sm.in.k, r0 + it * RPI, k[it]);
    keep(sm.in.q, r0 + it * RPI, q[it]);
  }
  if constexpr (!KDA) {
    tile_rows<TWO, LPR, RPI, IT>(kq, kTerm, 2 * kChunk, 0, sm.invK, k, r0, c0, nullptr, 0);
    tile_rows<TWO, LPR, RPI, IT>(kq, kTerm, 2 * kChunk, kChunk, sm.invQ, q, r0, c0, nullptr, 0);
    __syncthreads();
    // 20 tiles of 16 x 8 on or below the diagonal for each matrix, five per warp
    const bool isq = warp < 4;
    if (isq || !M2) {
#pragma unroll 1
      for (int e = 0; e < 5; ++e) {
        const int x = 5 * (warp & 3) + e;
        const int I = x < 8 ? 3 : x < 10 ? 0 : x < 16 ? 2 : 1;
        const int nt = x < 8 ? x : x < 10 ? x - 8 : x < 16 ? x - 10 : x - 16;
        float c[4];
        gram_tile<DK>(c, isq ? sm.in.q : sm.in.k, sm.in.k, nullptr, 16 * I, 8 * nt, lane);
        gram_store(c, isq ? sm.QK : sm.KK, 16 * I, 8 * nt, lane);
      }
    }
  } else {
    // ---- decays per channel: a thread per channel runs through the chunk
    const float* arow = p.alpha + (ck.first * p.H + grp) * DK;
    const long long astep = (long long)p.H * DK;
    float* tri_end = reinterpret_cast<float*>(p.tri + ((long long)slot * p.H + grp) * kTriBytes + kTriEnd);
    for (int e = tid; e < kChunk * DK / 4; e += kNT) {
      const int i = e / (DK / 4), c = 4 * (e % (DK / 4));
      st4(&sm.in.a[i * PK + c], i < n ? ld4(arow + i * astep + c) : make_float4(1.f, 1.f, 1.f, 1.f));
    }
    __syncthreads();
    // diagonal 16 x 16 blocks, two warps each: a thread takes two columns over an eighth of
    // the channels (four channels in turn per lane), the decays running with row i
    if (warp < 8) {
      const int b = 16 * (warp >> 1), part = lane & 7, g = lane >> 3;
      const int col[2] = {(warp & 1) ? 7 - g : g, (warp & 1) ? 8 + g : 15 - g};
      float f[2][DK / 8] = {};
      float* out = (part & 4) ? sm.KK : sm.QK;
      const int out_col = b + ((part & 2) ? col[1] : col[0]);
#pragma unroll 2
      for (int i = 0; i < 16; ++i) {
        float v[4] = {};      // q with column 0, column 1, k with column 0, column 1
#pragma unroll
        for (int x = 0; x < DK / 32; ++x) {
          const int at = (b + i) * PK + 32 * x + 4 * part;
          const float4 a = ld4(&sm.in.a[at]), qq = ld4(&sm.in.q[at]), kk = ld4(&sm.in.k[at]);
          const float av[4] = {a.x, a.y, a.z, a.w}, qv[4] = {qq.x, qq.y, qq.z, qq.w}, kv[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const bool starts = i == col[y];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& ff = f[y][4 * x + e];
              ff = starts ? kv[e] : ff * av[e];      // zero above the diagonal
              v[y] = fmaf(qv[e], ff, v[y]);
              v[2 + y] = fmaf(kv[e], ff, v[2 + y]);
            }
          }
        }
        // four sums over eight lanes by halving: lane bits 4 and 2 pick the value
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float send = (part & 4) ? v[y] : v[2 + y], keep = (part & 4) ? v[2 + y] : v[y];
          v[y] = keep + __shfl_xor_sync(0xffffffffu, send, 4);
        }
        const float send = (part & 2) ? v[0] : v[1], keep = (part & 2) ? v[1] : v[0];
        float t = keep + __shfl_xor_sync(0xffffffffu, send, 2);
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        if (!(part & 1)) out[(b + i) * PX + out_col] = t;
      }
    }
    __syncthreads();
    // Per block of 16 tokens and channel, all as products from the decays: F_i behind the
    // block's first token up to i, G_j behind j up to the next block's first token.
    // Operands of the blocks left of the diagonal: q_i F_i, k_i F_i, and k_j G_j (in the
    // decays' place); mv: the products over whole blocks between them.
    constexpr int NG = kNT / DK;             // threads per channel
    const int c = tid % DK, hf = tid / DK;
    float nxt[5];                            // decays of the blocks' first tokens
#pragma unroll
    for (int x = 0; x < 5; ++x) nxt[x] = x < 4 ? sm.in.a[16 * x * PK + c] : 1.f;
    __syncthreads();
    for (int x = hf; x < 4; x += NG) {
      float a[16], kk[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        a[i] = sm.in.a[(16 * x + i) * PK + c];
        kk[i] = sm.in.k[(16 * x + i) * PK + c];
      }
      float f = 1.f, g = x == 0 ? nxt[1] : x == 1 ? nxt[2] : x == 2 ? nxt[3] : 1.f;
      const float behind = g;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i > 0) f *= a[i];
        sm.in.q[(16 * x + i) * PK + c] *= f;
        sm.in.k[(16 * x + i) * PK + c] = kk[i] * f;
      }
      if (x == 1 || x == 2) sm.mv[x - 1][c] = f * behind;
#pragma unroll
      for (int i = 15; i >= 0; --i) {
        sm.in.a[(16 * x + i) * PK + c] = kk[i] * g;
        g *= a[i];
      }
    }
    __syncthreads();
    if (tid < DK) sm.mv[2][tid] = sm.mv[0][tid] * sm.mv[1][tid];
    __syncthreads();
    // 24 tiles left of the diagonal blocks
#pragma unroll 1
    for (int x = warp; x < 24; x += kNT / 32) {
      const bool isq = x < 12;
      const int y = isq ? x : x - 12;
      const int I = y < 2 ? 1 : y < 6 ? 2 : 3;
      const int nt = y < 2 ? y : y < 6 ? y - 2 : y - 6;
      const int J = nt / 2 + 1;              // the block behind the columns'
      const float* m = J == I ? nullptr : (J == 1 && I == 2) ? sm.mv[0] : J == 2 ? sm.mv[1] : sm.mv[2];
      float cc[4];
      gram_tile<DK>(cc, isq ? sm.in.q : sm.in.k, sm.in.a, m, 16 * I, 8 * nt, lane);
      gram_store(cc, isq ? sm.QK : sm.KK, 16 * I, 8 * nt, lane);
    }
    __syncthreads();
    // B_i and E_i per channel in the operands' place, then the tiles
    float* Bm = sm.in.q;
    float* Em = sm.in.k;
    if (tid < 2 * DK) {
      const int cc = tid % DK;
      const bool fwd = tid < DK;
      float f = 1.f;
#pragma unroll 16
      for (int s = 0; s < kChunk; ++s) {
        const int i = fwd ? s : kChunk - 1 - s;
        const float av = i < n ? arow[i * astep + cc] : 1.f;
        if (fwd) {
          f *= av;
          Bm[i * PK + cc] = f;
        } else {
          Em[i * PK + cc] = f;
          f *= av;
        }
      }
      if (fwd) tri_end[cc] = f;
    }
    __syncthreads();
    tile_rows<TWO, LPR, RPI, IT>(kq, kTerm, 2 * kChunk, 0, sm.invK, k, r0, c0, Bm, PK);
    tile_rows<TWO, LPR, RPI, IT>(kq, kTerm, 2 * kChunk, kChunk, sm.invQ, q, r0, c0, Bm, PK);
    tile_rows<TWO, LPR, RPI, IT>(kq + 2 * kTerm, kTerm / 2, kChunk, 0, sm.invE, k, r0, c0, Em, PK);
  }
  __syncthreads();

  float be_next = 0.f, al_next = 1.f;      // token tid's, of the next head
  auto fetch = [&](int h) {
    if (tid < n) {
      be_next = p.beta[(ck.first + tid) * p.H + h];
      if constexpr (!KDA) al_next = p.alpha[(ck.first + tid) * p.H + h];
    }
  };
  fetch(KDA ? grp : hk * rep);
  for (int r = 0; r < (KDA ? 1 : rep); ++r) {
    const int h = KDA ? grp : hk * rep + r;
    unsigned char* tri = p.tri + ((long long)slot * p.H + h) * kTriBytes;
    float* vec = reinterpret_cast<float*>(tri + kTriVec);
    if (tid < kChunk) {
      sm.beta[tid] = be_next;
      vec[kVecBeta * kChunk + tid] = be_next;
      if constexpr (KDA) {
        vec[kVecK * kChunk + tid] = sm.invK[tid];
        vec[kVecQ * kChunk + tid] = sm.invQ[tid];
        vec[kVecE * kChunk + tid] = sm.invE[tid];
      } else {
        // products within blocks of 16 tokens: up to the token, and behind it
        sm.alpha[tid] = al_next;
        float f = al_next, g = al_next;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) {
          const float x = __shfl_up_sync(0xffffffffu, f, off, 16), y = __shfl_down_sync(0xffffffffu, g, off, 16);
          if ((tid & 15) >= off) f *= x;
          if ((tid & 15) + off < 16) g *= y;
        }
        g = __shfl_down_sync(0xffffffffu, g, 1, 16);
        sm.B[tid] = f;
        sm.G[tid] = (tid & 15) == 15 ? 1.f : g;
        if ((tid & 15) == 15) sm.blk[tid >> 4] = f;
      }
    }
    for (int e = tid; e < kChunk * kChunk / 4; e += kNT) st4(&sm.t.T[(e / 16) * PX + 4 * (e % 16)], zero4());
    if (!KDA && r + 1 < rep) fetch(h + 1);
    __syncthreads();
    if constexpr (!KDA) {
      if (tid < kChunk) {      // over the blocks
        const int b = tid >> 4;
        float f = sm.B[tid], g = sm.G[tid];
        for (int x = 0; x < b; ++x) f *= sm.blk[x];
        for (int x = b + 1; x < 4; ++x) g *= sm.blk[x];
        vec[kVecK * kChunk + tid] = f * sm.invK[tid];
        vec[kVecQ * kChunk + tid] = f * sm.invQ[tid];
        vec[kVecE * kChunk + tid] = g * sm.invK[tid];
        if (tid == kChunk - 1) *reinterpret_cast<float*>(tri + kTriEnd) = f;
      }
    }
    if (tid < 256) {      // a thread takes column j of a block of 16 rows, the decay running down
      const int j = tid & 63, ib = tid >> 6, jb = j >> 4;
      float f = 1.f;
      if constexpr (!KDA) {
        if (ib > jb) {
          f = sm.G[j];
          for (int x = jb + 1; x < ib; ++x) f *= sm.blk[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int i = 16 * ib + x;
        if (!KDA && i > j) f *= sm.alpha[i];
        sm.t.P[i * PX + j] = i >= j ? f * sm.QK[i * PX + j] : 0.f;
        if constexpr (!M2) sm.t.A[i * PX + j] = i > j ? sm.beta[i] * f * sm.KK[i * PX + j] : 0.f;
      }
    }
    if constexpr (!M2) {
      invert(sm, tid);
      if (tid < 256) store_square(tri, vec + kVecT * kChunk, sm.t.T, tid);
    } else {
      __syncthreads();
    }
    if (tid >= kNT - 256) store_square(tri + 16384, vec + kVecP * kChunk, sm.t.P, tid - (kNT - 256));
    __syncthreads();
  }
}

template <int FORM, int DK, typename T>
int launch_prep_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  constexpr size_t bytes = sizeof(PrepSmem<FORM == SEED_KDA, DK, T>);
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_prep_kernel<FORM, DK, T>), bytes, &dev)) return rc;
  const int blocks = p.slots * (FORM == SEED_KDA ? p.H : p.HK);
  scan_prep_kernel<FORM, DK, T><<<blocks, prep_threads(FORM == SEED_KDA), bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace

// The launcher for one activation type (instantiated by seed_scan_pass_*.cu).
template <typename T>
int launch_scan_prep_as(const ScanParams& p, int form, cudaStream_t st) {
  if (p.dk != 64 && p.dk != 128) return SEED_ERR_SHAPE;
  const bool big = p.dk == 128;
  switch (form) {
    case SEED_GDN: return big ? launch_prep_t<SEED_GDN, 128, T>(p, st) : launch_prep_t<SEED_GDN, 64, T>(p, st);
    case SEED_KDA: return big ? launch_prep_t<SEED_KDA, 128, T>(p, st) : launch_prep_t<SEED_KDA, 64, T>(p, st);
    case SEED_MAMBA2: return big ? launch_prep_t<SEED_MAMBA2, 128, T>(p, st) : launch_prep_t<SEED_MAMBA2, 64, T>(p, st);
  }
  return SEED_ERR_INVALID_ARG;
}

}  // namespace seed

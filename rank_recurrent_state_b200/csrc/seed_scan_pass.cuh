// seed_scan_pass.cuh -- the dense scan chunk by chunk on the tensor cores.
//
// One block per (sequence, head) walks its chunks of 64 tokens with S^T (value channel
// x key channel) in registers.  Per chunk, with T and P from seed_scan_prep.cu, Kb and Qb
// the keys and queries times the decays since the chunk's start and Ke the keys times
// the decays to its end:
//     r^T = beta (v^T - S^T Kb^T),  w^T = r^T T^T,  o^T = S^T Qb^T + w^T P^T
//     S^T <- S^T Diag(B_C) + w^T Ke
// Every product has M = 128 value channels (tensor-memory lanes; d_v = 64 leaves half of
// them unused).  The A operands (S^T, r^T, w^T) are made by the threads that own those
// lanes and go to tensor memory, so neither the state nor a transpose ever passes through
// shared memory; the B operands are shared-memory tiles, K-major for Kb, Qb, T and P,
// MN-major for Ke.  All products run in two-term fp16 (seed_umma.cuh).
//
// Warps 0-7 own the lanes (two warps per 32 lanes, half of the columns each), thread 0
// issues the products; warps 8-11 make the next chunk's tiles meanwhile, each tile as soon
// as the products that read it are done.  The chain per chunk is S -> r -> w -> S: three
// products of 128 x 64 x d_k, 128 x 64 x 64 and 128 x d_k x 64 (three fp16 products each)
// and the conversions between them; the outputs hang beside it.
//
// Waits are bounded: one that runs out raises SEED_FLAG_TIMEOUT, and every later wait of
// the block returns at once, so that it ends (with unspecified results).
#pragma once

#include "seed_scan.cuh"
#include "seed_umma.cuh"

namespace seed {

namespace {

constexpr int kLaneThreads = 256;
constexpr int kTileThreads = 128;
constexpr int kNT = kLaneThreads + kTileThreads;

// Tensor-memory columns (512 in all).
constexpr uint32_t kS = 0;          // S^T: 64 columns hi, 64 lo
constexpr uint32_t kKS = 128;       // S^T Kb^T (64); then w^T = r^T T^T
constexpr uint32_t kQS = 192;       // S^T Qb^T (64)
constexpr uint32_t kRW = 256;       // r^T, then w^T: 32 columns hi, 32 lo
constexpr uint32_t kPW = 320;       // w^T P^T (64)
constexpr uint32_t kUp = 384;       // w^T Ke (d_k)

enum { kBarK, kBarQ, kBarT, kBarH, kBarP,          // products done: tile free, accumulator ready
       kFullK, kFullQ, kFullT, kFullH, kFullP,     // tile in place
       kBarDone,                                   // the lanes are done with the chunk's vectors
       kBars };

template <int FORM, int DK>
struct PassSmem {
  static constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  static constexpr int TILE = DK * 128;      // one fp16 term of 64 x DK
  alignas(1024) unsigned char K[M2 ? 1024 : 2 * TILE];
  alignas(1024) unsigned char Q[2 * TILE];
  alignas(1024) unsigned char H[2 * TILE];
  alignas(1024) unsigned char T[M2 ? 1024 : 16384];
  alignas(1024) unsigned char P[16384];
  float dec[KDA ? 2 * kChunk * DK : 4];      // B_i[c], then the decays from i to the end
  // per chunk parity
  float invT[2][kChunk], invP[2][kChunk];
  float csK[2][kChunk], csQ[2][kChunk];      // what undoes Kb's and Qb's scales (one decay: and applies B_i)
  float beta[2][kChunk];
  float end[2][KDA ? DK : 4];                // B_C
  float invH[2];
  float alpha[kChunk], dB[kChunk], dE[kChunk];
  float red[4];
  float mx[2][kLaneThreads];
  uint64_t bar[kBars];
  uint32_t tmem;
  int dead;
};

// Bounded wait; after the block's first failure every wait returns at once.
SEED_DEV void pass_wait(uint64_t* bar, uint32_t phase, volatile int* dead, uint32_t* status) {
  if (mbar_test_wait(bar, phase)) return;
  if (*dead) return;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, phase)) {
    if (*dead) return;
    if (global_ns() - t0 > kWaitLimitNs) {
      *dead = 1;
      raise_flag(status, SEED_FLAG_TIMEOUT);
      return;
    }
  }
}

// Three products (hi hi, hi lo, lo hi) of an A operand in tensor memory (lo terms
// A_LO columns behind the hi ones) with a tile in shared memory (its descriptor; lo terms
// B_LO bytes behind).  KS steps of 16; step(ks): byte offset of a step in the tile.
template <int KS, uint32_t A_LO, uint32_t B_LO, uint32_t IDESC, typename Step>
SEED_DEV void product(uint32_t d, uint32_t a, uint64_t tile, Step step) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      umma_ts(d, a + (t == 2 ? A_LO : 0u) + 8 * ks, tile + (((t == 1 ? B_LO : 0u) + step(ks)) >> 4), IDESC,
              t + ks > 0);
  }
}

// T: activation type.  SAVE: the backward pass's recomputation, which writes w and the
// state before each chunk instead of o and S_out.  (Both are template parameters for the
// size of the loop's code: it is walked once per chunk, and from beyond the instruction
// caches every instruction costs several cycles.)
template <int FORM, int DK, int DV, typename T, bool SAVE>
__global__ void __launch_bounds__(kNT, 1) scan_pass_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = PassSmem<FORM, DK>;
  constexpr uint32_t TILE = Sm::TILE;
  extern __shared__ unsigned char smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H;
  const SeqRange sr = seq_range(p, seq, h == 0 && tid == 0);
  const int nch = (sr.len + kChunk - 1) / kChunk;
  const long long mat = (long long)DK * DV;
  const long long sh = blockIdx.x;

  if (nch == 0) {
    if (p.S_out != nullptr) {
      for (int e = tid; e < DK * DV / 4; e += kNT)
        st4(p.S_out + sh * mat + 4 * e, p.S0 ? ld4(p.S0 + sh * mat + 4 * e) : zero4());
    }
    return;
  }
  if (tid == 0) {
    for (int b = 0; b < kBars; ++b)
      mbar_init(&sm.bar[b], b == kFullK || b == kFullQ || b == kFullH ? kTileThreads : b == kBarDone ? kLaneThreads : 1);
    fence_mbar_init();
    sm.dead = 0;
  }
  if (warp == 0) tmem_alloc(&sm.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tm = sm.tmem;
  auto wait = [&](int b, int chunk) { pass_wait(&sm.bar[b], (uint32_t)chunk & 1u, &sm.dead, p.status); };

  if (tid >= kLaneThreads) {
    // ================================================================ tiles
    const int t = tid - kLaneThreads;
    const int hk = h / (p.H / p.HK);
    constexpr int LPR = DK / 8;               // threads per row, 8 channels each
    constexpr int RPI = kTileThreads / LPR;   // rows per turn
    constexpr int IT = kChunk / RPI;
    const int r0 = t / LPR, c0 = 8 * (t % LPR);
    auto tile_sync = [&] { named_sync(3, kTileThreads); };
    // 8 scaled values of row i into both terms of a tile
    auto put = [&](unsigned char* tile, int i, const float (&x)[8]) {
      uint4 hi, lo;
      split2(x[0], x[1], hi.x, lo.x);
      split2(x[2], x[3], hi.y, lo.y);
      split2(x[4], x[5], hi.z, lo.z);
      split2(x[6], x[7], hi.w, lo.w);
      const int at = (c0 / 64) * 8192 + i * 128 + ((((c0 & 63) >> 3) ^ (i & 7)) << 4);
      *reinterpret_cast<uint4*>(tile + at) = hi;
      *reinterpret_cast<uint4*>(tile + TILE + at) = lo;
    };
    auto row_max = [&](const float (&x)[8]) {
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
      return m;
    };
    for (int c = 0; c < nch; ++c) {
      const int par = c & 1;
      const long long first = sr.first + (long long)c * kChunk;
      const int n = min(kChunk, sr.len - c * kChunk);
      // this thread's values of q or k: rows r0, r0 + RPI, .., zeros behind the tokens
      auto load = [&](const void* src, float (&x)[IT][8]) {
        act_ld8_rows(static_cast<const T*>(src) + ((first + r0) * p.HK + hk) * DK + c0, (long long)RPI * p.HK * DK,
                     (n - r0 + RPI - 1) / RPI, x);
      };
      // decays of the chunk and the per-token vectors
      if (t < kChunk) {
        const long long at = (first + t) * p.H + h;
        sm.beta[par][t] = t < n ? p.beta[at] : 0.f;
        if constexpr (!KDA) sm.alpha[t] = t < n ? p.alpha[at] : 1.f;
      }
      if constexpr (KDA) {
        tile_sync();      // the last chunk's readers of dec
        if (t < DK) {
          float a[kChunk];
          const float* src = p.alpha + (first * p.H + h) * DK + t;
#pragma unroll
          for (int i = 0; i < kChunk; ++i) a[i] = i < n ? src[(long long)i * p.H * DK] : 1.f;
          float f = 1.f;
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            f *= a[i];
            sm.dec[i * DK + t] = f;
          }
          sm.end[par][t] = f;
          f = 1.f;
#pragma unroll
          for (int i = kChunk - 1; i >= 0; --i) {
            sm.dec[(kChunk + i) * DK + t] = f;
            f *= a[i];
          }
        }
        tile_sync();
      } else {
        tile_sync();
        if (t < 32) {      // prefix and suffix products of 64 decays, two per lane
          const float a0 = sm.alpha[2 * lane], a1 = sm.alpha[2 * lane + 1];
          float f = a0 * a1, g = f;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, f, off);
            const float y = __shfl_down_sync(0xffffffffu, g, off);
            if (lane >= off) f *= x;
            if (lane + off < 32) g *= y;
          }
          float before = __shfl_up_sync(0xffffffffu, f, 1);
          float behind = __shfl_down_sync(0xffffffffu, g, 1);
          if (lane == 0) before = 1.f;
          if (lane == 31) behind = 1.f;
          sm.dB[2 * lane] = before * a0;
          sm.dB[2 * lane + 1] = f;
          sm.dE[2 * lane] = a1 * behind;
          sm.dE[2 * lane + 1] = behind;
          if (lane == 31) sm.end[par][0] = f;
        }
        tile_sync();
      }
      const unsigned char* img = p.tri + ((long long)(sr.slot0 + c) * p.H + h) * kTriBytes;
      // row-scaled tiles: x (times the decays per channel) and what undoes the scale
#pragma unroll 1
      for (int which = M2 ? 1 : 0; which < 2; ++which) {      // Kb, then Qb
        if (SAVE && which == 1) break;
        unsigned char* tile = which ? sm.Q : sm.K;
        float* cs = which ? sm.csQ[par] : sm.csK[par];
        float x[IT][8];
        load(which ? p.q : p.k, x);
        if (c >= 1) wait(which ? kBarQ : kBarK, c - 1);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int i = r0 + it * RPI;
          if constexpr (KDA) {
            const float4 d0 = ld4(&sm.dec[i * DK + c0]), d1 = ld4(&sm.dec[i * DK + c0 + 4]);
            x[it][0] *= d0.x; x[it][1] *= d0.y; x[it][2] *= d0.z; x[it][3] *= d0.w;
            x[it][4] *= d1.x; x[it][5] *= d1.y; x[it][6] *= d1.z; x[it][7] *= d1.w;
          }
          float m = row_max(x[it]);
#pragma unroll
          for (int off = LPR / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          const float s = pow2_scale(m);
          if (c0 == 0) cs[i] = (KDA ? 1.f : sm.dB[i]) * pow2_inverse(s);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[it][e] *= s;
          put(tile, i, x[it]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.bar[which ? kFullQ : kFullK]);
      }
      if constexpr (!M2) {
        if (t == 0) {
          if (c >= 1) wait(kBarT, c - 1);
          mbar_arrive_expect_tx(&sm.bar[kFullT], 16384 + kChunk * 4);
          bulk_g2s(sm.T, img, 16384, &sm.bar[kFullT]);
          bulk_g2s(sm.invT[par], img + 32768, kChunk * 4, &sm.bar[kFullT]);
        }
        __syncwarp();
      }
      {      // keys times the decays to the chunk's end, one scale for the tile
        float x[IT][8], m = 0.f;
        load(p.k, x);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const int i = r0 + it * RPI;
          if constexpr (KDA) {
            const float* d = &sm.dec[(kChunk + i) * DK + c0];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[it][e] *= d[e];
          } else {
            const float d = sm.dE[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[it][e] *= d;
          }
          m = fmaxf(m, row_max(x[it]));
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) sm.red[t >> 5] = m;
        tile_sync();
        m = fmaxf(fmaxf(sm.red[0], sm.red[1]), fmaxf(sm.red[2], sm.red[3]));
        const float s = pow2_scale(m);
        if (t == 0) sm.invH[par] = pow2_inverse(s);
        if (c >= 1) wait(kBarH, c - 1);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[it][e] *= s;
          put(sm.H, r0 + it * RPI, x[it]);
        }
        fence_proxy_async_smem();
        // the vectors of chunk c - 1 make room for those of c + 1.  Waited for before this
        // chunk's last tile is handed over, so that no barrier runs two phases ahead of a wait.
        if (c >= 1) wait(kBarDone, c - 1);
        mbar_arrive(&sm.bar[kFullH]);
      }
      if (!SAVE && t == 0) {
        if (c >= 1) wait(kBarP, c - 1);
        mbar_arrive_expect_tx(&sm.bar[kFullP], 16384 + kChunk * 4);
        bulk_g2s(sm.P, img + 16384, 16384, &sm.bar[kFullP]);
        bulk_g2s(sm.invP[par], img + 32768 + kChunk * 4, kChunk * 4, &sm.bar[kFullP]);
      }
      __syncwarp();
    }
    if (t == 0 && sm.dead) {      // a wait ran out: let the copies in flight land all the same
      if (!M2) mbar_wait_bounded(&sm.bar[kFullT], (uint32_t)(nch - 1) & 1u, kWaitLimitNs);
      if (!SAVE) mbar_wait_bounded(&sm.bar[kFullP], (uint32_t)(nch - 1) & 1u, kWaitLimitNs);
    }
  } else {
    // ================================================================ lanes
    const int lg = warp & 3, half = warp >> 2;
    const int j = 32 * lg + lane;                      // value channel
    const bool on = j < DV;
    const uint32_t lanes = tm + ((uint32_t)(32 * lg) << 16);
    constexpr int NS = DK / 2;                         // state columns per thread
    const int cs0 = half * NS, t0 = half * 32;         // its first state column, its first token
    auto pair_sync = [&] { named_sync(4 + lg, 64); };  // the two warps of the same lanes
    auto lane_sync = [&] { named_sync(2, kLaneThreads); };
    auto pair_max = [&](float m, int which) {
      sm.mx[which][half * 128 + j] = m;
      pair_sync();
      return fmaxf(m, sm.mx[which][(half ^ 1) * 128 + j]);
    };
    // 32 values in registers as the A operand at kRW, scaled by s
    auto put_rw = [&](const float (&x)[32], float s) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) split2(s * x[2 * e], s * x[2 * e + 1], hi[e], lo[e]);
      tmem_st16(lanes + kRW + t0 / 2, hi);
      tmem_st16(lanes + kRW + 32 + t0 / 2, lo);
      tmem_wait_st();
      tmem_fence_before();
    };
    constexpr uint32_t kIdesc64 = umma_idesc(128, 64, false), kIdescUp = umma_idesc(128, DK, true);
    const auto rowstep = [](int ks) { return (uint32_t)((ks >> 2) * 8192 + (ks & 3) * 32); };
    const long long vstep = (long long)p.H * DV;       // from a token's values to the next one's
    float S[NS];
#pragma unroll
    for (int c = 0; c < NS; ++c) S[c] = on && p.S0 != nullptr ? p.S0[sh * mat + (long long)(cs0 + c) * DV + j] : 0.f;
    float nan = 0.f, top = 0.f;      // NaN once a result was not finite; the largest |o|
    float invS = 1.f, invW = 1.f;

    // one turn more than chunks: the last one only writes the last outputs
    for (int c = 0; c < nch + (SAVE ? 0 : 1); ++c) {
      const int par = c & 1;
      float m = 0.f;
      const float invS_before = invS;
      if (c < nch && !(SAVE && M2)) {
        // ---- S^T as an operand
#pragma unroll
        for (int x = 0; x < NS; ++x) m = fmaxf(m, fabsf(S[x]));
        m = pair_max(m, 0);
        const float sS = pow2_scale(m);
        invS = pow2_inverse(sS);
#pragma unroll
        for (int x = 0; x < NS / 32; ++x) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) split2(sS * S[32 * x + 2 * e], sS * S[32 * x + 2 * e + 1], hi[e], lo[e]);
          tmem_st16(lanes + kS + cs0 / 2 + 16 * x, hi);
          tmem_st16(lanes + kS + 64 + cs0 / 2 + 16 * x, lo);
        }
        tmem_wait_st();
        tmem_fence_before();
        // A thread waits for a tile before the barrier behind which the products that free
        // the tile are issued: every thread has seen the tile (and the vectors written with
        // it) before its barrier can move on.
        if constexpr (!M2) {
          wait(kFullK, c);
          lane_sync();
          if (tid == 0) {
            tmem_fence_after();
            product<DK / 16, 64, TILE, kIdesc64>(tm + kKS, tm + kS, umma_desc(smem_addr(sm.K), 16), rowstep);
            umma_commit(&sm.bar[kBarK]);
          }
        }
      }
      if constexpr (SAVE) {
        if (on) {
          float* dst = p.chunk_S + ((long long)(sr.slot0 + c) * p.H + h) * mat + (long long)cs0 * DV + j;
#pragma unroll
          for (int x = 0; x < NS; ++x) dst[x * DV] = S[x];
        }
      } else if (c > 0) {
        // ---- the last chunk's outputs, beside this one's S^T Kb^T
        const int before = par ^ 1, n = min(kChunk, sr.len - (c - 1) * kChunk);
        wait(kBarP, c - 1);
        tmem_fence_after();
#pragma unroll 1
        for (int x = t0; x < t0 + 32; x += 16) {
          float a[16], b[16];
          tmem_ld16(lanes + kQS + x, a);
          tmem_ld16(lanes + kPW + x, b);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 fq = ld4(&sm.csQ[before][x + e]), fp = ld4(&sm.invP[before][x + e]);
            a[e] = fmaf(a[e], invS_before * fq.x, b[e] * (invW * fp.x));
            a[e + 1] = fmaf(a[e + 1], invS_before * fq.y, b[e + 1] * (invW * fp.y));
            a[e + 2] = fmaf(a[e + 2], invS_before * fq.z, b[e + 2] * (invW * fp.z));
            a[e + 3] = fmaf(a[e + 3], invS_before * fq.w, b[e + 3] * (invW * fp.w));
          }
          if (on) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {      // (tokens behind the chunk's have q = 0 and rows of P of zeros)
              nan = fmaf(a[e], 0.f, nan);
              top = fmaxf(top, fabsf(a[e]));
            }
            act_st_rows(static_cast<T*>(p.o) + ((sr.first + (long long)(c - 1) * kChunk + x) * p.H + h) * DV + j, vstep,
                        n - x, a);
          }
        }
        tmem_fence_before();
      }
      if (c > 0) mbar_arrive(&sm.bar[kBarDone]);
      if (c == nch) break;
      const long long first = sr.first + (long long)c * kChunk;
      const int n = min(kChunk, sr.len - c * kChunk);
      if constexpr (!SAVE) {
        wait(kFullQ, c);
        lane_sync();
        if (tid == 0) {
          tmem_fence_after();
          product<DK / 16, 64, TILE, kIdesc64>(tm + kQS, tm + kS, umma_desc(smem_addr(sm.Q), 16), rowstep);
          umma_commit(&sm.bar[kBarQ]);
        }
      }
      // ---- r, w
      float x[32];
      act_ld_rows(static_cast<const T*>(p.v) + ((first + t0) * p.H + h) * DV + j, vstep, on ? n - t0 : 0, x);
      if constexpr (!M2) {
        wait(kBarK, c);
        tmem_fence_after();
        m = 0.f;
#pragma unroll
        for (int y = 0; y < 32; y += 16) {
          float a[16];
          tmem_ld16(lanes + kKS + t0 + y, a);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 fk = ld4(&sm.csK[par][t0 + y + e]), be = ld4(&sm.beta[par][t0 + y + e]);
            x[y + e] = be.x * fmaf(-a[e], invS * fk.x, x[y + e]);
            x[y + e + 1] = be.y * fmaf(-a[e + 1], invS * fk.y, x[y + e + 1]);
            x[y + e + 2] = be.z * fmaf(-a[e + 2], invS * fk.z, x[y + e + 2]);
            x[y + e + 3] = be.w * fmaf(-a[e + 3], invS * fk.w, x[y + e + 3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(x[e]));
        m = pair_max(m, 1);
        const float sR = pow2_scale(m), invR = pow2_inverse(sR);
        put_rw(x, sR);
        wait(kFullT, c);
        lane_sync();
        if (tid == 0) {
          tmem_fence_after();
          product<4, 32, 8192, kIdesc64>(tm + kKS, tm + kRW, umma_desc(smem_addr(sm.T), 16), rowstep);
          umma_commit(&sm.bar[kBarT]);
        }
        wait(kBarT, c);
        tmem_fence_after();
        tmem_ld16(lanes + kKS + t0, x);
        tmem_ld16(lanes + kKS + t0 + 16, x + 16);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 ft = ld4(&sm.invT[par][t0 + e]);
          x[e] *= invR * ft.x;
          x[e + 1] *= invR * ft.y;
          x[e + 2] *= invR * ft.z;
          x[e + 3] *= invR * ft.w;
        }
      } else {
        if constexpr (SAVE) wait(kFullH, c);      // the vectors come with the first tile
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 be = ld4(&sm.beta[par][t0 + e]);
          x[e] *= be.x;
          x[e + 1] *= be.y;
          x[e + 2] *= be.z;
          x[e + 3] *= be.w;
        }
      }
      if constexpr (SAVE) act_st_rows(p.w + ((first + t0) * p.H + h) * DV + j, vstep, on ? n - t0 : 0, x);
      m = 0.f;
#pragma unroll
      for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(x[e]));
      m = pair_max(m, 0);
      const float sW = pow2_scale(m);
      invW = pow2_inverse(sW);
      put_rw(x, sW);
      wait(kFullH, c);
      if constexpr (!SAVE) wait(kFullP, c);
      lane_sync();
      if (tid == 0) {
        tmem_fence_after();
        product<4, 32, TILE, kIdescUp>(tm + kUp, tm + kRW, umma_desc(smem_addr(sm.H), 8192),
                                       [](int ks) { return (uint32_t)(ks * 2048); });
        umma_commit(&sm.bar[kBarH]);
        if constexpr (!SAVE) {
          product<4, 32, 8192, kIdesc64>(tm + kPW, tm + kRW, umma_desc(smem_addr(sm.P), 16), rowstep);
          umma_commit(&sm.bar[kBarP]);
        }
      }
      // ---- S behind the chunk
      wait(kBarH, c);
      tmem_fence_after();
      const float up = invW * sm.invH[par], end = sm.end[par][0];
#pragma unroll
      for (int y = 0; y < NS; y += 16) {
        float a[16];
        tmem_ld16(lanes + kUp + cs0 + y, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) S[y + e] = fmaf(a[e], up, (KDA ? sm.end[par][cs0 + y + e] : end) * S[y + e]);
      }
      tmem_fence_before();
    }
    bool bad = !(nan == 0.f) || !act_finite(top, p.elem);
    if (!SAVE && p.S_out != nullptr && on) {
      float* dst = p.S_out + sh * mat + (long long)cs0 * DV + j;
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        dst[(long long)c * DV] = S[c];
        bad = bad || !isfinite(S[c]);
      }
    }
    if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
    // every product was waited for, and with it the copies it read
    tmem_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tmem_fence_after();
    tmem_free(tm, 512);
  }
}

template <int FORM, int DK, int DV, typename T, bool SAVE>
int launch_pass_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  // one block per SM (it holds all of the SM's tensor memory)
  constexpr size_t need = sizeof(PassSmem<FORM, DK>) + 1024;
  constexpr size_t bytes = need < 116 * 1024 ? 116 * 1024 : need;
  static_assert(bytes <= 227 * 1024, "shared memory");
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_pass_kernel<FORM, DK, DV, T, SAVE>), bytes, &dev))
    return rc;
  scan_pass_kernel<FORM, DK, DV, T, SAVE><<<p.seqs * p.H, kNT, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace

// The launcher for one activation type (instantiated by seed_scan_pass_*.cu).
template <typename T>
int launch_scan_pass_as(const ScanParams& p, int form, cudaStream_t st) {
#define SEED_PASS(F, K, V)                                                                       \
  if (form == F && p.dk == K && p.dv == V)                                                       \
    return p.chunk_S != nullptr ? launch_pass_t<F, K, V, T, true>(p, st) : launch_pass_t<F, K, V, T, false>(p, st);
#define SEED_PASS_D(F) SEED_PASS(F, 64, 64) SEED_PASS(F, 128, 128) SEED_PASS(F, 128, 64) SEED_PASS(F, 64, 128)
  SEED_PASS_D(SEED_GDN)
  SEED_PASS_D(SEED_KDA)
  SEED_PASS_D(SEED_MAMBA2)
#undef SEED_PASS_D
#undef SEED_PASS
  return SEED_ERR_SHAPE;
}

}  // namespace seed

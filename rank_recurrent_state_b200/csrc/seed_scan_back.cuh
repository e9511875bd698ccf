// seed_scan_back.cuh -- the reverse recurrence of the dense scan's backward pass, chunk by
// chunk on the tensor cores.
//
// The counterpart of seed_scan_pass.cuh, with the gradient of the state dS^T (value
// channel x key channel) in registers and the chunks from the last to the first; the
// tiles are the forward's.  With B_i the decays since the chunk's start, E_i those to its
// end and dS the gradient behind the chunk:
//     x^T  = dS^T (E k)^T + do^T P,   dw^T = x^T T   (Mamba-2: dw = x)
//     dS^T <- dS^T Diag(B_C) + (B do)^T q - (B beta dw)^T k
// It writes dw, and the gradient behind each chunk for the gradients of seed_scan_grad.cu.
// P and T are read along their other axis (MN-major), so the scales of their rows go into
// the A operand; the update is one product of K = 128 over the k and q rows.
//
// Warps 0-7 own the lanes, a thread of warp 8 issues the products, one of warp 9 copies.
// The chain per chunk is dS -> x -> dw -> dS; do^T P does not depend on it.  Waits are
// bounded as in the forward pass.  Measured: GDN, 6 documents of up to 1500 tokens x 16
// heads, 235 us (24 chunks in turn, 10 us each; token by token 826 us).  Bound by latency:
// two more conversions than the forward pass, and dw and dS stored a value at a time.
#pragma once

#include "seed_scan_pass.cuh"

namespace seed {

namespace {

constexpr int kBackThreads = kLaneThreads + 64;

// Tensor-memory columns.
constexpr uint32_t kBS = 0;         // dS^T (64 hi, 64 lo); then (-B beta dw, B do)^T (64 hi, 64 lo)
constexpr uint32_t kBE = 128;       // dS^T (E k)^T (64); then x^T T
constexpr uint32_t kBP = 192;       // do^T P (64)
constexpr uint32_t kBX = 256;       // do^T, then x^T (32 hi, 32 lo)
constexpr uint32_t kBU = 320;       // the update (d_k)

template <int FORM, int DK, int DV, typename T>
struct BackSmem {
  static constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  static constexpr bool TWO = scan_two_terms(FORM, std::is_same<T, float>::value);
  static constexpr int NKQ = KDA ? 1 : 2, NTP = TWO ? 1 : 2;      // chunks of tiles held
  static constexpr int TERM = DK * 256;
  static constexpr int KQ = (TWO ? 2 : 1) * TERM;
  alignas(1024) unsigned char kq[NKQ][KQ];
  alignas(1024) unsigned char ke[KDA ? TERM : 1024];
  alignas(1024) unsigned char tt[NTP][M2 ? 1024 : 16384];
  alignas(1024) unsigned char pp[NTP][16384];
  alignas(128) T d_o[kChunk * DV];
  struct Vec {
    alignas(128) float v[kVecs][kChunk];
    float end[128];
  } vec[3];
  float mx[3][kLaneThreads];
  uint64_t done_e, done_p, done_t, done_up;      // products done
  uint64_t op_s, op_p, op_x, op_u;               // operands stored (one arrival per lane warp)
  uint64_t full_kq[NKQ], full_ke, full_t[NTP], full_p[NTP], full_vec[3], full_o;      // copies done
  uint64_t free_copy;
  uint32_t tmem;
  int dead;
};

template <int FORM, int DK, int DV, typename T>
__global__ void __launch_bounds__(kBackThreads, 1) scan_back_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = BackSmem<FORM, DK, DV, T>;
  constexpr bool TWO = Sm::TWO;
  constexpr int NKQ = Sm::NKQ, NTP = Sm::NTP;
  constexpr uint32_t TERM = Sm::TERM;
  extern __shared__ unsigned char smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seq = blockIdx.x / p.H, h = blockIdx.x - seq * p.H;
  const SeqRange sr = seq_range(p, seq, h == 0 && tid == 0);
  const int nch = (sr.len + kChunk - 1) / kChunk;
  const long long mat = (long long)DK * DV;
  const long long sh = blockIdx.x;

  if (nch == 0) {
    if (p.dS0 != nullptr) {
      for (int e = tid; e < DK * DV / 4; e += kBackThreads)
        st4(p.dS0 + sh * mat + 4 * e, p.dS_out ? ld4(p.dS_out + sh * mat + 4 * e) : zero4());
    }
    return;
  }
  if (tid == 0) {
    mbar_init(&sm.done_e, 1);
    mbar_init(&sm.done_p, 1);
    mbar_init(&sm.done_t, 1);
    mbar_init(&sm.done_up, 1);
    mbar_init(&sm.op_s, kLaneThreads / 32);
    mbar_init(&sm.op_p, kLaneThreads / 32);
    mbar_init(&sm.op_x, kLaneThreads / 32);
    mbar_init(&sm.op_u, kLaneThreads / 32);
    for (int s = 0; s < NKQ; ++s) mbar_init(&sm.full_kq[s], 1);
    for (int s = 0; s < NTP; ++s) {
      mbar_init(&sm.full_t[s], 1);
      mbar_init(&sm.full_p[s], 1);
    }
    for (int s = 0; s < 3; ++s) mbar_init(&sm.full_vec[s], 1);
    mbar_init(&sm.full_ke, 1);
    mbar_init(&sm.full_o, 1);
    mbar_init(&sm.free_copy, 1);
    fence_mbar_init();
    sm.dead = 0;
  }
  if (warp == 0) tmem_alloc(&sm.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tm = sm.tmem;
  auto wait = [&](uint64_t* bar, int phase) { pass_wait(bar, (uint32_t)phase & 1u, &sm.dead, p.status); };
  const long long vstep = (long long)p.H * DV;
  // Turns it = 0 .. nch - 1 take chunk nch - 1 - it.  No barrier runs two phases ahead of a
  // thread that waits for it, for the reasons given in the forward pass.

  if (warp == 8) {
    // ================================================================ products
    if (lane == 0) {
      constexpr uint32_t kIdesc64 = umma_idesc(128, 64, false), kIdesc64t = umma_idesc(128, 64, true);
      constexpr uint32_t kIdescUp = umma_idesc(128, DK, true);
      const auto step_rows = [](int ks) { return (uint32_t)(ks * 2048); };
      for (int it = 0; it < nch; ++it) {
        const int kst = it % NKQ, kph = it / NKQ, tst = it % NTP, tph = it / NTP;
        wait(&sm.full_p[tst], tph);
        wait(&sm.op_p, it);
        tmem_fence_after();
        product<4, true, kIdesc64t>(tm + kBP, tm + kBX, 32, umma_desc(smem_addr(sm.pp[tst]), 8192), 8192, false, step_rows);
        umma_commit(&sm.done_p);
        if constexpr (KDA) wait(&sm.full_ke, it);
        wait(&sm.full_kq[kst], kph);
        wait(&sm.op_s, it);
        tmem_fence_after();
        if constexpr (KDA)
          product<DK / 16, true, kIdesc64>(tm + kBE, tm + kBS, 64, umma_desc(smem_addr(sm.ke), 16), TERM / 2, false,
                                           [](int ks) { return (uint32_t)((ks >> 2) * 8192 + (ks & 3) * 32); });
        else
          product<DK / 16, TWO, kIdesc64>(tm + kBE, tm + kBS, 64, umma_desc(smem_addr(sm.kq[kst]), 16), TERM, false,
                                          [](int ks) { return (uint32_t)((ks >> 2) * 16384 + (ks & 3) * 32); });
        umma_commit(&sm.done_e);
        if constexpr (!M2) {
          wait(&sm.full_t[tst], tph);
          wait(&sm.op_x, it);
          tmem_fence_after();
          product<4, true, kIdesc64t>(tm + kBE, tm + kBX, 32, umma_desc(smem_addr(sm.tt[tst]), 8192), 8192, false, step_rows);
          umma_commit(&sm.done_t);
        }
        if (it > 0) wait(&sm.free_copy, it - 1);
        wait(&sm.op_u, it);
        tmem_fence_after();
        const uint64_t tile = umma_desc(smem_addr(sm.kq[kst]), 16384);
        if constexpr (M2)      // the q rows alone
          product<4, TWO, kIdescUp>(tm + kBU, tm + kBS + 32, 64, tile + (8192 >> 4), TERM, false, step_rows);
        else
          product<8, TWO, kIdescUp>(tm + kBU, tm + kBS, 64, tile, TERM, false, step_rows);
        umma_commit(&sm.done_up);
      }
    }
  } else if (warp == 9) {
    // ================================================================ copies
    if (lane == 0) {
      const long long kq_head = KDA ? h : h / (p.H / p.HK), kq_heads = KDA ? p.H : p.HK;
      constexpr int KQB = kq_bytes(FORM, DK, TWO);
      auto slot = [&](int it) { return (long long)(sr.slot0 + nch - 1 - it); };
      auto tri = [&](int it) { return p.tri + (slot(it) * p.H + h) * kTriBytes; };
      auto kq = [&](int it) { return p.kq + (slot(it) * kq_heads + kq_head) * KQB; };
      auto copy = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(dst, src, bytes, bar);
      };
      auto copy_kq = [&](int it) {
        if (it < nch) copy(sm.kq[it % NKQ], kq(it), Sm::KQ, &sm.full_kq[it % NKQ]);
      };
      auto copy_ke = [&](int it) {
        if (KDA && it < nch) copy(sm.ke, kq(it) + 2 * TERM, TERM, &sm.full_ke);
      };
      auto copy_t = [&](int it) {
        if (!M2 && it < nch) copy(sm.tt[it % NTP], tri(it), 16384, &sm.full_t[it % NTP]);
      };
      auto copy_p = [&](int it) {
        if (it < nch) copy(sm.pp[it % NTP], tri(it) + 16384, 16384, &sm.full_p[it % NTP]);
      };
      auto copy_vec = [&](int it) {
        if (it < nch) copy(&sm.vec[it % 3], tri(it) + kTriVec, kVecBytes, &sm.full_vec[it % 3]);
      };
      auto copy_o = [&](int it) {      // the chunk's rows of do
        if (it >= nch) return;
        const int c = nch - 1 - it, n = min(kChunk, sr.len - c * kChunk);
        const T* src = static_cast<const T*>(p.d_o) + ((sr.first + (long long)c * kChunk) * p.H + h) * DV;
        mbar_arrive_expect_tx(&sm.full_o, n * DV * (int)sizeof(T));
#pragma unroll 4
        for (int i = 0; i < n; ++i, src += vstep) bulk_g2s(sm.d_o + i * DV, src, DV * sizeof(T), &sm.full_o);
      };
      for (int it = 0; it < 2; ++it) {
        copy_vec(it);
        if (it == 0) copy_o(it);
        if (it < NTP) copy_p(it);
        if (it == 0) copy_ke(it);
        if (it < NKQ) copy_kq(it);
        if (it < NTP) copy_t(it);
      }
      for (int it = 0; it < nch; ++it) {
        wait(&sm.op_u, it);      // the lanes have read do for the last time
        copy_o(it + 1);
        if constexpr (NTP == 1) {
          wait(&sm.done_p, it);
          copy_p(it + 1);
        }
        if constexpr (KDA) {
          wait(&sm.done_e, it);
          copy_ke(it + 1);
        }
        if constexpr (NTP == 1 && !M2) {
          wait(&sm.done_t, it);
          copy_t(it + 1);
        }
        wait(&sm.done_up, it);
        copy_kq(it + NKQ);
        if constexpr (NTP == 2) {
          copy_p(it + 2);
          copy_t(it + 2);
        }
        copy_vec(it + 2);
        mbar_arrive(&sm.free_copy);
      }
      if (sm.dead) {      // a wait ran out: let the copies in flight land all the same
        const int it = nch - 1;
        mbar_wait_bounded(&sm.full_kq[it % NKQ], (uint32_t)(it / NKQ) & 1u, kWaitLimitNs);
        mbar_wait_bounded(&sm.full_o, (uint32_t)it & 1u, kWaitLimitNs);
        mbar_wait_bounded(&sm.full_vec[it % 3], (uint32_t)(it / 3) & 1u, kWaitLimitNs);
      }
    }
  } else {
    // ================================================================ lanes
    const int lg = warp & 3, half = warp >> 2;
    const int j = 32 * lg + lane;                      // value channel
    const bool on = j < DV;
    const uint32_t lanes = tm + ((uint32_t)(32 * lg) << 16);
    constexpr int NS = DK / 2;                         // state columns per thread
    const int cs0 = half * NS, t0 = half * 32;         // its first state column, its first token
    auto pair_max = [&](int which, float a) {
      float* mx = sm.mx[which] + j;
      mx[half * 128] = a;
      named_sync(4 + lg, 64);
      return fmaxf(a, mx[(half ^ 1) * 128]);
    };
    auto abs_max = [](const float (&x)[32]) {
      float m[4] = {};
#pragma unroll
      for (int e = 0; e < 32; ++e) m[e & 3] = fmaxf(m[e & 3], fabsf(x[e]));
      return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    };
    // 32 tokens' values times f (per token) and s, as an A operand (second term lo columns behind)
    auto put = [&](uint32_t at, uint32_t lo_cols, const float (&x)[32], float s) {
#pragma unroll
      for (int g = 0; g < 32; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2_scaled(x[g + 2 * e], x[g + 2 * e + 1], s, hi[e], lo[e]);
        tmem_st8(lanes + at + (t0 + g) / 2, hi);
        tmem_st8(lanes + at + lo_cols + (t0 + g) / 2, lo);
      }
    };
    auto scale_by = [&](float (&y)[32], const float (&x)[32], const float* f) {
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 v = ld4(f + t0 + e);
        const float2 a = mul2(make_float2(x[e], x[e + 1]), make_float2(v.x, v.y));
        const float2 b = mul2(make_float2(x[e + 2], x[e + 3]), make_float2(v.z, v.w));
        y[e] = a.x; y[e + 1] = a.y; y[e + 2] = b.x; y[e + 3] = b.y;
      }
    };
    auto hand = [&](uint64_t* op) {
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(op);
    };
    float S[NS];
#pragma unroll
    for (int c = 0; c < NS; ++c)
      S[c] = on && p.dS_out != nullptr ? p.dS_out[sh * mat + (long long)(cs0 + c) * DV + j] : 0.f;

    for (int it = 0; it < nch; ++it) {
      const int c = nch - 1 - it;
      const long long first = sr.first + (long long)c * kChunk;
      const int n = min(kChunk, sr.len - c * kChunk);
      const typename Sm::Vec& vc = sm.vec[it % 3];
      float x[32], y[32];
      auto read_o = [&] {
        const T* src = sm.d_o + t0 * DV + j;
        const int left = on ? n - t0 : 0;      // (rows behind the tokens hold another chunk's)
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float v = fac_to_f(src[e * DV]);
          x[e] = e < left ? v : 0.f;
        }
      };
      // ---- do^T as the operand of do^T P
      wait(&sm.full_vec[it % 3], it / 3);
      wait(&sm.full_o, it);
      read_o();
      scale_by(y, x, vc.v[kVecP]);
      const float sP = pow2_scale(pair_max(0, abs_max(y)));
      put(kBX, 32, y, sP);
      hand(&sm.op_p);
      // ---- dS^T as the operand of dS^T (E k)^T
      float m[4] = {};
#pragma unroll
      for (int e = 0; e < NS; ++e) m[e & 3] = fmaxf(m[e & 3], fabsf(S[e]));
      const float sS = pow2_scale(pair_max(1, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]))));
#pragma unroll
      for (int g = 0; g < NS; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2_scaled(S[g + 2 * e], S[g + 2 * e + 1], sS, hi[e], lo[e]);
        tmem_st8(lanes + kBS + (cs0 + g) / 2, hi);
        tmem_st8(lanes + kBS + 64 + (cs0 + g) / 2, lo);
      }
      hand(&sm.op_s);
      if (on) {
        float* dst = p.chunk_dS + ((long long)(sr.slot0 + c) * p.H + h) * mat + (long long)cs0 * DV + j;
#pragma unroll
        for (int e = 0; e < NS; ++e) dst[e * DV] = S[e];
      }
      // ---- x
      wait(&sm.done_p, it);
      wait(&sm.done_e, it);
      tmem_fence_after();
      const float invP = pow2_inverse(sP), invS = pow2_inverse(sS);
#pragma unroll
      for (int g = 0; g < 32; g += 16) {
        float a[16], b[16];
        tmem_ld16(lanes + kBE + t0 + g, a);
        tmem_ld16(lanes + kBP + t0 + g, b);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 fe = ld4(&vc.v[kVecE][t0 + g + e]);
          y[g + e] = fmaf(a[e], invS * fe.x, b[e] * invP);
          y[g + e + 1] = fmaf(a[e + 1], invS * fe.y, b[e + 1] * invP);
          y[g + e + 2] = fmaf(a[e + 2], invS * fe.z, b[e + 2] * invP);
          y[g + e + 3] = fmaf(a[e + 3], invS * fe.w, b[e + 3] * invP);
        }
      }
      // ---- dw
      if constexpr (!M2) {
        scale_by(y, y, vc.v[kVecT]);
        const float sX = pow2_scale(pair_max(2, abs_max(y)));
        put(kBX, 32, y, sX);
        hand(&sm.op_x);
        wait(&sm.done_t, it);
        tmem_fence_after();
        tmem_ld16(lanes + kBE + t0, y);
        tmem_ld16(lanes + kBE + t0 + 16, y + 16);
        tmem_wait_ld();
        const float invX = pow2_inverse(sX);
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] *= invX;
      }
      act_st_rows(p.dw + ((first + t0) * p.H + h) * DV + j, vstep, on ? n - t0 : 0, y);
      // ---- the update
      read_o();
      scale_by(x, x, vc.v[kVecQ]);
      float mu = abs_max(x);
      if constexpr (!M2) {
        scale_by(y, y, vc.v[kVecK]);
        scale_by(y, y, vc.v[kVecBeta]);
        mu = fmaxf(mu, abs_max(y));
      }
      const float sU = pow2_scale(pair_max(0, mu));
      if constexpr (!M2) put(kBS, 64, y, -sU);
      put(kBS + 32, 64, x, sU);
      hand(&sm.op_u);
      wait(&sm.done_up, it);
      tmem_fence_after();
      const float invU = pow2_inverse(sU), end = vc.end[0];
#pragma unroll
      for (int z = 0; z < NS; z += 16) {
        float a[16];
        tmem_ld16(lanes + kBU + cs0 + z, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 d = KDA ? *reinterpret_cast<const float2*>(&vc.end[cs0 + z + e]) : make_float2(end, end);
          const float2 v = fma2(make_float2(a[e], a[e + 1]), make_float2(invU, invU), mul2(d, make_float2(S[z + e], S[z + e + 1])));
          S[z + e] = v.x;
          S[z + e + 1] = v.y;
        }
      }
      tmem_fence_before();
    }
    if (p.dS0 != nullptr && on) {
      float* dst = p.dS0 + sh * mat + (long long)cs0 * DV + j;
#pragma unroll
      for (int c = 0; c < NS; ++c) dst[(long long)c * DV] = S[c];
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 0) {
    tmem_fence_after();
    tmem_free(tm, 512);
  }
}

template <int FORM, int DK, int DV, typename T>
int launch_back_t(const ScanParams& p, cudaStream_t st) {
  static LaunchCache cache;
  // one block per SM (it holds all of the SM's tensor memory)
  constexpr size_t need = sizeof(BackSmem<FORM, DK, DV, T>) + 1024;
  constexpr size_t bytes = need < 116 * 1024 ? 116 * 1024 : need;
  static_assert(bytes <= 227 * 1024, "shared memory");
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_back_kernel<FORM, DK, DV, T>), bytes, &dev)) return rc;
  scan_back_kernel<FORM, DK, DV, T><<<p.seqs * p.H, kBackThreads, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace

// The launcher for one activation type (instantiated by seed_scan_pass_*.cu).
template <typename T>
int launch_scan_back_as(const ScanParams& p, int form, cudaStream_t st) {
#define SEED_BACK(F, K, V) \
  if (form == F && p.dk == K && p.dv == V) return launch_back_t<F, K, V, T>(p, st);
#define SEED_BACK_D(F) SEED_BACK(F, 64, 64) SEED_BACK(F, 128, 128) SEED_BACK(F, 128, 64) SEED_BACK(F, 64, 128)
  SEED_BACK_D(SEED_GDN)
  SEED_BACK_D(SEED_KDA)
  SEED_BACK_D(SEED_MAMBA2)
#undef SEED_BACK_D
#undef SEED_BACK
  return SEED_ERR_SHAPE;
}

}  // namespace seed

// seed_scan_pass.cuh -- the dense scan chunk by chunk on the tensor cores.
//
// One block per (sequence, head) walks its chunks of 64 tokens with S^T (value channel
// x key channel) in registers.  Per chunk, with T, P and the k and q tiles of
// seed_scan_prep.cuh, B_i the decays since the chunk's start, E_i those to its end:
//     r^T = beta (v^T - S^T (B k)^T),  w^T = r^T T^T,  o^T = S^T (B q)^T + w^T P^T
//     S^T <- S^T Diag(B_C) + (E w)^T k
// Every product has M = 128 value channels (tensor-memory lanes; d_v = 64 leaves half of
// them unused).  The A operands (S^T, r^T, w^T) are made by the threads that own those
// lanes and go to tensor memory, so neither the state nor a transpose ever passes through
// shared memory; the B operands are shared-memory tiles, K-major for k and q (one product
// of N = 128 for both: an A operand in tensor memory costs the same 64 cycles a step up
// to there), T and P, MN-major for k in the update.  All products run in two-term fp16
// (seed_umma.cuh); tiles of one term take two products instead of three.
//
// Warps 0-7 own the lanes (two warps per 32 lanes, half of the columns each).  Warps 8-11
// write the outputs, beside the next chunk's work.  Of warps 12-15, which give their
// registers to the others, one thread issues the products and one keeps the tiles coming
// (bulk copies, two chunks ahead where shared memory holds two).  The chain per chunk is
// S -> r -> w -> S, three products and the conversions between them; everything else
// hangs beside it.
//
// Measured: GDN, 4096 tokens x 48 heads of 128 x 128 bf16, 344 us = 5.4 us a chunk, of which
// the products take 1.7 us and the rest is the latency of the conversions between them
// (tensor pipe active 21 %, 0.4 instructions issued a cycle).  One block per SM is what
// tensor memory allows: the accumulators and operands above fill its 512 columns.  Tried
// and dropped: 16 lane warps with half of the columns each (424 us: the same instructions,
// and the outputs fall behind); thread 0 of the lanes issuing the products (384 us);
// stores and loads of single values of o and v (every one holds the load-store units for
// about eight cycles: 600 us).
//
// Waits are bounded: one that runs out raises SEED_FLAG_TIMEOUT, and every later wait of
// the block returns at once, so that it ends (with unspecified results).
#pragma once

#include "seed_scan.cuh"
#include "seed_umma.cuh"

namespace seed {

namespace {

constexpr int kLaneThreads = 256;
constexpr int kOutThreads = 128;
constexpr int kPassThreads = kLaneThreads + kOutThreads + 128;
// Registers per thread of the lanes, the outputs and the rest; the launch gives each of the
// 512 threads 128, and the shares stay within that: 2 x 160 + 144 + 48 = 4 x 128.
constexpr int kLaneRegs = 160, kOutRegs = 144, kRestRegs = 48;

// Tensor-memory columns (512 in all).
constexpr uint32_t kS = 0;          // S^T: 64 columns hi, 64 lo; behind the first product (E w)^T: 32 hi, 32 lo
constexpr uint32_t kKQ = 128;       // S^T (B k)^T (64), S^T (B q)^T (64); behind it w^T = r^T T^T in the first half
constexpr uint32_t kRW = 256;       // r^T, then w^T: 32 columns hi, 32 lo
constexpr uint32_t kUp = 320;       // (E w)^T k (d_k)
constexpr uint32_t kPW = 448;       // w^T P^T (64)

template <int FORM, int DK, int DV, typename T>
struct PassSmem {
  static constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  static constexpr bool TWO = scan_two_terms(FORM, std::is_same<T, float>::value);
  static constexpr int NKQ = KDA ? 1 : 2;               // chunks of k and q tiles held
  static constexpr int NTP = TWO ? 1 : 2;               // of T and P
  static constexpr int TERM = DK * 256;                 // one term of the k and q rows
  static constexpr int KQ = (TWO ? 2 : 1) * TERM;
  static constexpr int OROWS = 32;                      // tokens of outputs staged at a time
  alignas(1024) unsigned char kq[NKQ][KQ];
  alignas(1024) unsigned char ke[KDA ? TERM : 1024];    // E k (two terms), decays per channel only
  alignas(1024) unsigned char tt[NTP][M2 ? 1024 : 16384];
  alignas(1024) unsigned char pp[NTP][16384];
  alignas(128) T v[kChunk * DV];
  alignas(128) T o[OROWS * DV];
  struct Vec {
    alignas(128) float v[kVecs][kChunk];
    float end[128];
  } vec[3];
  float2 mx[3][kLaneThreads];     // the lanes' maxima: of S, of r, of w and E w
  float inv[2][2][128];           // per chunk parity and lane, for the outputs: S's and w's inverse scales
  // products done: accumulator ready, tiles free
  uint64_t done_kq, done_t, done_up, done_pw;
  // copies done
  uint64_t full_kq[NKQ], full_ke, full_t[NTP], full_p[NTP], full_vec[3], full_v;
  // the outputs have read an accumulator
  uint64_t free_q, free_pw;
  uint64_t free_copy;             // the copying thread has seen a chunk's last product
  // the lanes have stored an operand (one arrival per warp)
  uint64_t op_s, op_r, op_e, op_w;
  uint32_t tmem;
  int dead;
};
static_assert(kVecBytes == sizeof(float) * (kVecs * kChunk + 128), "one layout");

// Bounded wait; after the block's first failure every wait returns at once.  The clock is
// read on one try in 64: a try suspends the warp, but what stands between two of them takes
// issue slots from the warps at work.
SEED_DEV void pass_wait(uint64_t* bar, uint32_t phase, volatile int* dead, uint32_t* status) {
  uint64_t t0 = 0;
  for (int i = 1; !mbar_try_wait_for(bar, phase, 1000000u); ++i) {
    if ((i & 63) == 0) {
      if (*dead) return;
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        *dead = 1;
        raise_flag(status, SEED_FLAG_TIMEOUT);
        return;
      }
    }
  }
}

// The products of a two-term A operand in tensor memory (the second term a_lo columns
// behind) with a tile (its descriptor; a second term b_lo bytes behind): lo hi, for a tile
// of two terms hi lo, and hi hi last.  The accumulator rounds towards zero at every step,
// so the small products go first, while it is small (errors of 1.3e-6 of the result with
// hi hi first).  KS steps of 16, step(ks) bytes apart in the tile.
template <int KS, bool TWO, uint32_t IDESC, typename Step>
SEED_DEV void product(uint32_t d, uint32_t a, uint32_t a_lo, uint64_t tile, uint32_t b_lo, bool accumulate, Step step) {
  const uint64_t high = tile & 0xffffffff00000000ull;
  uint32_t low = (uint32_t)tile;
  asm volatile("" : "+r"(low));      // or every step's descriptor is kept in a register across the chunks
#pragma unroll
  for (int t = 0; t < (TWO ? 3 : 2); ++t) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      umma_ts(d, a + (t == 0 ? a_lo : 0u) + 8 * ks, high | (low + (((TWO && t == 1 ? b_lo : 0u) + step(ks)) >> 4)), IDESC,
              accumulate || t + ks > 0);
  }
}

// The same with both operands in shared memory, two terms each.
template <int KS, uint32_t IDESC, typename StepA, typename StepB>
SEED_DEV void product_ss(uint32_t d, uint64_t a, uint32_t a_lo, StepA step_a, uint64_t b, uint32_t b_lo, StepB step_b) {
#pragma unroll
  for (int t = 0; t < 3; ++t) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      umma_ss(d, a + (((t == 0 ? a_lo : 0u) + step_a(ks)) >> 4), b + (((t == 1 ? b_lo : 0u) + step_b(ks)) >> 4), IDESC,
              t + ks > 0);
  }
}

// T: activation type.  SAVE: the backward pass's recomputation, which writes w and the
// state before each chunk instead of o and S_out.  (Both are template parameters for the
// size of the loop's code: it is walked once per chunk, and from beyond the instruction
// caches every instruction costs several cycles.)
template <int FORM, int DK, int DV, typename T, bool SAVE>
__global__ void __launch_bounds__(kPassThreads, 1) scan_pass_kernel(const ScanParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  using Sm = PassSmem<FORM, DK, DV, T>;
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
    if (p.S_out != nullptr) {
      for (int e = tid; e < DK * DV / 4; e += kPassThreads)
        st4(p.S_out + sh * mat + 4 * e, p.S0 ? ld4(p.S0 + sh * mat + 4 * e) : zero4());
    }
    return;
  }
  if (tid == 0) {
    mbar_init(&sm.done_kq, 1);
    mbar_init(&sm.done_t, 1);
    mbar_init(&sm.done_up, 1);
    mbar_init(&sm.done_pw, 1);
    for (int s = 0; s < NKQ; ++s) mbar_init(&sm.full_kq[s], 1);
    for (int s = 0; s < NTP; ++s) {
      mbar_init(&sm.full_t[s], 1);
      mbar_init(&sm.full_p[s], 1);
    }
    mbar_init(&sm.full_ke, 1);
    mbar_init(&sm.full_v, 1);
    for (int s = 0; s < 3; ++s) mbar_init(&sm.full_vec[s], 1);
    mbar_init(&sm.free_q, kOutThreads / 32);
    mbar_init(&sm.free_pw, kOutThreads / 32);
    mbar_init(&sm.free_copy, 1);
    mbar_init(&sm.op_s, kLaneThreads / 32);
    mbar_init(&sm.op_r, kLaneThreads / 32);
    mbar_init(&sm.op_e, kLaneThreads / 32);
    mbar_init(&sm.op_w, kLaneThreads / 32);
    fence_mbar_init();
    sm.dead = 0;
  }
  if (warp == 0) tmem_alloc(&sm.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tm = sm.tmem;
  auto wait = [&](uint64_t* bar, int phase) { pass_wait(bar, (uint32_t)phase & 1u, &sm.dead, p.status); };
  const int lg = warp & 3;
  const int j = 32 * lg + lane;                      // value channel
  const bool on = j < DV;
  const uint32_t lanes = tm + ((uint32_t)(32 * lg) << 16);
  const long long vstep = (long long)p.H * DV;       // from a token's values to the next one's
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // No barrier runs two phases ahead of a thread that waits for it.  The products of a
  // chunk wait for the lanes' operands of that chunk, and the first and the last one for
  // the outputs of the chunk before (free_q, free_pw); lanes and outputs signal behind
  // their own waits.  The issuing thread is the only one that waits for operands, tiles
  // and the outputs.  The copying thread waits for done_pw (SAVE: done_up) of every chunk
  // and signals free_copy behind it, which the next chunk's last product waits for; what
  // has one stage it copies behind the product (for v: the operand) that frees it, which
  // cannot come round again before the copy.  The vectors come round every third chunk.

  if (warp >= 12) {
    // ================================================================ products, copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRestRegs));
    if (warp == 12 && lane == 0) {
      constexpr uint32_t kIdesc64 = umma_idesc(128, 64, false), kIdesc128 = umma_idesc(128, 128, false);
      constexpr uint32_t kIdescUp = umma_idesc(128, DK, true);
      constexpr int ROWS = KDA ? kChunk : 2 * kChunk;    // of the tile with the update's k
      const auto step_kq = [](int ks) { return (uint32_t)((ks >> 2) * 16384 + (ks & 3) * 32); };
      const auto step_sq = [](int ks) { return (uint32_t)(ks * 32); };
      const auto step_up = [](int ks) { return (uint32_t)(ks * 2048); };
      for (int c = 0; c < nch; ++c) {
        const int kst = c % NKQ, kph = c / NKQ, tst = c % NTP, tph = c / NTP;
        if constexpr (!(M2 && SAVE)) {
          wait(&sm.full_kq[kst], kph);
          if (!SAVE && c > 0) wait(&sm.free_q, c - 1);
          wait(&sm.op_s, c);
          tmem_fence_after();
          const uint64_t tile = umma_desc(smem_addr(sm.kq[kst]), 16);
          if constexpr (SAVE)
            product<DK / 16, TWO, kIdesc64>(tm + kKQ, tm + kS, 64, tile, TERM, false, step_kq);
          else if constexpr (M2)
            product<DK / 16, TWO, kIdesc64>(tm + kKQ + 64, tm + kS, 64, tile + (8192 >> 4), TERM, false, step_kq);
          else
            product<DK / 16, TWO, kIdesc128>(tm + kKQ, tm + kS, 64, tile, TERM, false, step_kq);
          umma_commit(&sm.done_kq);
        }
        if constexpr (!M2) {
          wait(&sm.full_t[tst], tph);
          wait(&sm.op_r, c);
          tmem_fence_after();
          product<4, true, kIdesc64>(tm + kKQ, tm + kRW, 32, umma_desc(smem_addr(sm.tt[tst]), 16), 8192, false, step_sq);
          umma_commit(&sm.done_t);
        }
        if constexpr (KDA) wait(&sm.full_ke, c);
        if constexpr (M2 && SAVE) wait(&sm.full_kq[kst], kph);
        if (SAVE && c > 0) wait(&sm.free_copy, c - 1);
        wait(&sm.op_e, c);
        tmem_fence_after();
        if constexpr (KDA)
          product<4, true, kIdescUp>(tm + kUp, tm + kS, 32, umma_desc(smem_addr(sm.ke), ROWS * 128), TERM / 2, false, step_up);
        else
          product<4, TWO, kIdescUp>(tm + kUp, tm + kS, 32, umma_desc(smem_addr(sm.kq[kst]), ROWS * 128), TERM, false, step_up);
        umma_commit(&sm.done_up);
        if constexpr (!SAVE) {
          wait(&sm.full_p[tst], tph);
          if (c > 0) {
            wait(&sm.free_pw, c - 1);
            wait(&sm.free_copy, c - 1);
          }
          wait(&sm.op_w, c);
          tmem_fence_after();
          product<4, true, kIdesc64>(tm + kPW, tm + kRW, 32, umma_desc(smem_addr(sm.pp[tst]), 16), 8192, false, step_sq);
          umma_commit(&sm.done_pw);
        }
      }
    } else if (warp == 13 && lane == 0) {
      const long long kq_head = KDA ? h : h / (p.H / p.HK), kq_heads = KDA ? p.H : p.HK;
      constexpr int KQB = kq_bytes(FORM, DK, TWO);
      auto tri = [&](int c) { return p.tri + ((long long)(sr.slot0 + c) * p.H + h) * kTriBytes; };
      auto kq = [&](int c) { return p.kq + ((sr.slot0 + c) * kq_heads + kq_head) * KQB; };
      auto copy = [&](void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, bytes);
        bulk_g2s(dst, src, bytes, bar);
      };
      auto copy_kq = [&](int c) {
        if (c < nch) copy(sm.kq[c % NKQ], kq(c), Sm::KQ, &sm.full_kq[c % NKQ]);
      };
      auto copy_ke = [&](int c) {
        if (KDA && c < nch) copy(sm.ke, kq(c) + 2 * TERM, TERM, &sm.full_ke);
      };
      auto copy_t = [&](int c) {
        if (!M2 && c < nch) copy(sm.tt[c % NTP], tri(c), 16384, &sm.full_t[c % NTP]);
      };
      auto copy_p = [&](int c) {
        if (!SAVE && c < nch) copy(sm.pp[c % NTP], tri(c) + 16384, 16384, &sm.full_p[c % NTP]);
      };
      auto copy_vec = [&](int c) {
        if (c < nch) copy(&sm.vec[c % 3], tri(c) + kTriVec, kVecBytes, &sm.full_vec[c % 3]);
      };
      auto copy_v = [&](int c) {      // the chunk's rows of v
        if (c >= nch) return;
        const int n = min(kChunk, sr.len - c * kChunk);
        const T* src = static_cast<const T*>(p.v) + ((sr.first + (long long)c * kChunk) * p.H + h) * DV;
        mbar_arrive_expect_tx(&sm.full_v, n * DV * (int)sizeof(T));
#pragma unroll 4
        for (int i = 0; i < n; ++i, src += vstep) bulk_g2s(sm.v + i * DV, src, DV * sizeof(T), &sm.full_v);
      };
      for (int c = 0; c < 2; ++c) {
        copy_vec(c);
        if (c < NKQ) copy_kq(c);
        if (c == 0) copy_v(c);
        if (c < NTP) copy_t(c);
        if (c == 0) copy_ke(c);
        if (c < NTP) copy_p(c);
      }
      for (int c = 0; c < nch; ++c) {
        if constexpr (NKQ == 1) {
          wait(&sm.done_kq, c);
          copy_kq(c + 1);
        }
        wait(M2 ? &sm.op_e : &sm.op_r, c);
        copy_v(c + 1);
        if constexpr (NTP == 1 && !M2) {
          wait(&sm.done_t, c);
          copy_t(c + 1);
        }
        if constexpr (KDA) {
          wait(&sm.done_up, c);
          copy_ke(c + 1);
        }
        wait(SAVE ? &sm.done_up : &sm.done_pw, c);
        if constexpr (NKQ == 2) copy_kq(c + 2);
        if constexpr (NTP == 2) copy_t(c + 2);
        copy_p(c + NTP);
        copy_vec(c + 2);
        mbar_arrive(&sm.free_copy);
      }
      if (sm.dead) {      // a wait ran out: let the copies in flight land all the same
        const int c = nch - 1;
        mbar_wait_bounded(&sm.full_kq[c % NKQ], (uint32_t)(c / NKQ) & 1u, kWaitLimitNs);
        mbar_wait_bounded(&sm.full_v, (uint32_t)c & 1u, kWaitLimitNs);
        mbar_wait_bounded(&sm.full_vec[c % 3], (uint32_t)(c / 3) & 1u, kWaitLimitNs);
      }
    }
  } else if (warp >= 8) {
    // ================================================================ outputs
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOutRegs));
    float nan = 0.f;      // NaN once a stored result was not finite
    for (int c = 0; !SAVE && c < nch; ++c) {
      const float(*vec)[kChunk] = sm.vec[c % 3].v;
      float o[kChunk];
      {
        const int n = min(kChunk, sr.len - c * kChunk);
        wait(&sm.done_kq, c);
        wait(&sm.full_vec[c % 3], c / 3);
        tmem_fence_after();
#pragma unroll
        for (int x = 0; x < kChunk; x += 16) tmem_ld16(lanes + kKQ + 64 + x, o + x);
        tmem_wait_ld();
        tmem_fence_before();
        const float invS = sm.inv[c & 1][0][j];
        warp_arrive(&sm.free_q);
#pragma unroll
        for (int x = 0; x < kChunk; x += 4) {
          const float4 f = ld4(&vec[kVecQ][x]);
          o[x] *= invS * f.x;
          o[x + 1] *= invS * f.y;
          o[x + 2] *= invS * f.z;
          o[x + 3] *= invS * f.w;
        }
        wait(&sm.done_pw, c);
        tmem_fence_after();
        const float invW = sm.inv[c & 1][1][j];
#pragma unroll
        for (int x = 0; x < kChunk; x += 16) {
          float b[16];
          tmem_ld16(lanes + kPW + x, b);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 f = ld4(&vec[kVecP][x + e]);
            o[x + e] = fmaf(b[e], invW * f.x, o[x + e]);
            o[x + e + 1] = fmaf(b[e + 1], invW * f.y, o[x + e + 1]);
            o[x + e + 2] = fmaf(b[e + 2], invW * f.z, o[x + e + 2]);
            o[x + e + 3] = fmaf(b[e + 3], invW * f.w, o[x + e + 3]);
          }
        }
        tmem_fence_before();
        warp_arrive(&sm.free_pw);
        // through shared memory, so that whole rows go out in one copy each (a store per
        // value and token would hold the load-store units for longer than the chunk takes)
        const int ot = tid - kLaneThreads;
#pragma unroll
        for (int x = 0; x < kChunk; x += Sm::OROWS) {
          if (ot < Sm::OROWS) bulk_wait_read();
          named_sync(3, kOutThreads);
          if (on) {
#pragma unroll
            for (int e = 0; e < Sm::OROWS; ++e) {      // (tokens behind the chunk's have rows of zeros)
              const T t = fac_from_f<T>(o[x + e]);
              sm.o[e * DV + j] = t;
              nan = fmaf(fac_to_f(t), 0.f, nan);
            }
          }
          fence_proxy_async_smem();
          named_sync(3, kOutThreads);
          if (ot < Sm::OROWS && x + ot < n) {
            bulk_s2g(static_cast<T*>(p.o) + ((sr.first + (long long)c * kChunk + x + ot) * p.H + h) * DV, sm.o + ot * DV,
                     DV * sizeof(T));
            bulk_commit();
          }
        }
      }
    }
    bulk_wait_read();
    if (!(nan == 0.f)) raise_flag(p.status, SEED_FLAG_NONFINITE);
  } else {
    // ================================================================ lanes
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLaneRegs));
    const int half = warp >> 2;
    constexpr int NS = DK / 2;                         // state columns per thread
    const int cs0 = half * NS, t0 = half * 32;         // its first state column, its first token
    // the larger of both warps' values for these lanes
    auto pair_max = [&](int which, float a, float b) {
      float2* mx = sm.mx[which] + j;
      mx[half * 128] = make_float2(a, b);
      named_sync(4 + lg, 64);
      const float2 o = mx[(half ^ 1) * 128];
      return make_float2(fmaxf(a, o.x), fmaxf(b, o.y));
    };
    // 32 values in registers as an A operand at `at` (second term 32 columns behind)
    auto put_rw = [&](uint32_t at, const float (&x)[32], float s) {
#pragma unroll
      for (int g = 0; g < 32; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split2_scaled(x[g + 2 * e], x[g + 2 * e + 1], s, hi[e], lo[e]);
        tmem_st8(lanes + at + (t0 + g) / 2, hi);
        tmem_st8(lanes + at + 32 + (t0 + g) / 2, lo);
      }
    };
    auto hand = [&](uint64_t* op) {      // an operand is stored, everything read before it is read
      tmem_wait_st();
      tmem_fence_before();
      warp_arrive(op);
    };
    float S[NS];
#pragma unroll
    for (int c = 0; c < NS; ++c) S[c] = on && p.S0 != nullptr ? p.S0[sh * mat + (long long)(cs0 + c) * DV + j] : 0.f;
    float invS = 1.f;

    for (int c = 0; c < nch; ++c) {
      const long long first = sr.first + (long long)c * kChunk;
      const int n = min(kChunk, sr.len - c * kChunk);
      const typename Sm::Vec& vc = sm.vec[c % 3];
      // ---- S^T as an operand, S^T (B k)^T and S^T (B q)^T
      if constexpr (!(M2 && SAVE)) {
        float m[4] = {};
#pragma unroll
        for (int x = 0; x < NS; ++x) m[x & 3] = fmaxf(m[x & 3], fabsf(S[x]));
        const float sS = pow2_scale(pair_max(0, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), 0.f).x);
        invS = pow2_inverse(sS);
        if (!SAVE && half == 0) sm.inv[c & 1][0][j] = invS;
#pragma unroll
        for (int x = 0; x < NS; x += 16) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split2_scaled(S[x + 2 * e], S[x + 2 * e + 1], sS, hi[e], lo[e]);
          tmem_st8(lanes + kS + (cs0 + x) / 2, hi);
          tmem_st8(lanes + kS + 64 + (cs0 + x) / 2, lo);
        }
        hand(&sm.op_s);
      }
      // ---- r, w
      float x[32];
      wait(&sm.full_v, c);
      {
        const T* src = sm.v + t0 * DV + j;
        const int left = on ? n - t0 : 0;      // (rows behind the tokens hold an earlier chunk's)
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float y = fac_to_f(src[e * DV]);
          x[e] = e < left ? y : 0.f;
        }
      }
      if constexpr (SAVE) {
        if (on) {
          float* dst = p.chunk_S + ((long long)(sr.slot0 + c) * p.H + h) * mat + (long long)cs0 * DV + j;
#pragma unroll
          for (int y = 0; y < NS; ++y) dst[y * DV] = S[y];
        }
      }
      wait(&sm.full_vec[c % 3], c / 3);
      float m = 0.f, me = 0.f;
      if constexpr (!M2) {
        wait(&sm.done_kq, c);
        tmem_fence_after();
#pragma unroll
        for (int y = 0; y < 32; y += 16) {
          float a[16];
          tmem_ld16(lanes + kKQ + t0 + y, a);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 fk = ld4(&vc.v[kVecK][t0 + y + e]), be = ld4(&vc.v[kVecBeta][t0 + y + e]);
            x[y + e] = be.x * fmaf(-a[e], invS * fk.x, x[y + e]);
            x[y + e + 1] = be.y * fmaf(-a[e + 1], invS * fk.y, x[y + e + 1]);
            x[y + e + 2] = be.z * fmaf(-a[e + 2], invS * fk.z, x[y + e + 2]);
            x[y + e + 3] = be.w * fmaf(-a[e + 3], invS * fk.w, x[y + e + 3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(x[e]));
        const float sR = pow2_scale(pair_max(1, m, 0.f).x), invR = pow2_inverse(sR);
        put_rw(kRW, x, sR);
        hand(&sm.op_r);
        wait(&sm.done_t, c);
        tmem_fence_after();
        tmem_ld16(lanes + kKQ + t0, x);
        tmem_ld16(lanes + kKQ + t0 + 16, x + 16);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 ft = ld4(&vc.v[kVecT][t0 + e]);
          x[e] *= invR * ft.x;
          x[e + 1] *= invR * ft.y;
          x[e + 2] *= invR * ft.z;
          x[e + 3] *= invR * ft.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 be = ld4(&vc.v[kVecBeta][t0 + e]);
          x[e] *= be.x;
          x[e + 1] *= be.y;
          x[e + 2] *= be.z;
          x[e + 3] *= be.w;
        }
        // Mamba-2 has no product between S and w: S's operand may still be in use
        if constexpr (!SAVE) wait(&sm.done_kq, c);
      }
      // ---- the state's update: E w times the k rows
      m = 0.f;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 fe = ld4(&vc.v[kVecE][t0 + e]);
        m = fmaxf(fmaxf(fmaxf(m, fabsf(x[e])), fmaxf(fabsf(x[e + 1]), fabsf(x[e + 2]))), fabsf(x[e + 3]));
        me = fmaxf(fmaxf(fmaxf(me, fabsf(x[e] * fe.x)), fmaxf(fabsf(x[e + 1] * fe.y), fabsf(x[e + 2] * fe.z))),
                   fabsf(x[e + 3] * fe.w));
      }
      const float2 mm = pair_max(2, m, me);
      const float sW = pow2_scale(mm.x), sE = pow2_scale(mm.y), invE = pow2_inverse(sE);
#pragma unroll
      for (int g = 0; g < 32; g += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 fe = ld4(&vc.v[kVecE][t0 + g + e]);
          const float2 a = mul2(mul2(make_float2(x[g + e], x[g + e + 1]), make_float2(fe.x, fe.y)), sE);
          const float2 b = mul2(mul2(make_float2(x[g + e + 2], x[g + e + 3]), make_float2(fe.z, fe.w)), sE);
          split2(a.x, a.y, hi[e / 2], lo[e / 2]);
          split2(b.x, b.y, hi[e / 2 + 1], lo[e / 2 + 1]);
        }
        tmem_st8(lanes + kS + (t0 + g) / 2, hi);
        tmem_st8(lanes + kS + 32 + (t0 + g) / 2, lo);
      }
      if (!SAVE && half == 0) sm.inv[c & 1][1][j] = pow2_inverse(sW);
      hand(&sm.op_e);
      // ---- w P^T for the outputs, beside it
      if constexpr (!SAVE) {
        put_rw(kRW, x, sW);
        hand(&sm.op_w);
      } else {
        act_st_rows(p.w + ((first + t0) * p.H + h) * DV + j, vstep, on ? n - t0 : 0, x);
      }
      // ---- S behind the chunk
      wait(&sm.done_up, c);
      tmem_fence_after();
      const float end = vc.end[0];
#pragma unroll
      for (int z = 0; z < NS; z += 16) {
        float a[16];
        tmem_ld16(lanes + kUp + cs0 + z, a);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 d = KDA ? *reinterpret_cast<const float2*>(&vc.end[cs0 + z + e]) : make_float2(end, end);
          const float2 y = fma2(make_float2(a[e], a[e + 1]), make_float2(invE, invE), mul2(d, make_float2(S[z + e], S[z + e + 1])));
          S[z + e] = y.x;
          S[z + e + 1] = y.y;
        }
      }
      tmem_fence_before();
    }
    if (!SAVE && p.S_out != nullptr && on) {
      float* dst = p.S_out + sh * mat + (long long)cs0 * DV + j;
      bool bad = false;
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        dst[(long long)c * DV] = S[c];
        bad = bad || !isfinite(S[c]);
      }
      if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
    }
  }
  // every product has been waited for, and with it the copies it read
  tmem_fence_before();
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
  constexpr size_t need = sizeof(PassSmem<FORM, DK, DV, T>) + 1024;
  constexpr size_t bytes = need < 116 * 1024 ? 116 * 1024 : need;
  static_assert(bytes <= 227 * 1024, "shared memory");
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(scan_pass_kernel<FORM, DK, DV, T, SAVE>), bytes, &dev))
    return rc;
  scan_pass_kernel<FORM, DK, DV, T, SAVE><<<p.seqs * p.H, kPassThreads, bytes, st>>>(p);
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

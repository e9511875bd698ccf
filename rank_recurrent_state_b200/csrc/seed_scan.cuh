// seed_scan.cuh -- what the kernels of the dense scan (seed_dense_scan and its
// backward pass) share: launch parameters, the chunk slots of packed ragged
// sequences, and loads and stores of the three activation types.
//
// Notation, per head and per sequence (seed.h): a = decay, S' = Diag(a) S,
// w = beta (v - S'^T k) (Mamba-2: beta v), S+ = S' + k w^T, o = S+^T q.  Inside a
// chunk of kChunk tokens that starts from state S0, with B_i the product of the
// decays up to token i and D_ij = B_i / B_j (formed as a product, never a quotient):
//     S_i = B_i S0 + sum_{j <= i} D_ij k_j w_j^T
#pragma once

#include "seed_common.cuh"

namespace seed {

constexpr int kChunk = 64;
// ---- Scratch of the chunked passes, as seed_scan_prep.cuh writes it.
// Per chunk and head: T and P (two fp16 terms of 64 x 64 each), then vectors of 64
// floats, then the product of the chunk's decays (one, or one per channel).
constexpr int kTriVec = 4 * 8192;
enum { kVecT, kVecP,      // what undoes the scales of T's and P's rows
       kVecK, kVecQ,      // the same for the k and q rows, times B_i where the tiles have no decay in them
       kVecE,             // for the k rows of the state's update, times E_i likewise
       kVecBeta, kVecs };
constexpr int kTriEnd = kTriVec + kVecs * kChunk * 4;
constexpr int kTriBytes = kTriEnd + 512;
constexpr int kVecBytes = kTriBytes - kTriVec;
// Per chunk and key head (decays per channel: per chunk and head): the k rows, then the q
// rows, in panels of 64 channels; a second fp16 term where one does not hold the values;
// with decays per channel the tile of E k behind them.
__host__ __device__ constexpr bool scan_two_terms(int form, bool f32) { return f32 || form == SEED_KDA; }
__host__ __device__ constexpr int kq_bytes(int form, int dk, bool two) {
  return (two ? 2 : 1) * dk * 256 + (form == SEED_KDA ? dk * 256 : 0);
}

struct ScanParams {
  const int32_t* offsets;
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  const float* S0;        // [seqs][H][dk][dv] or null (zeros)
  void* o;                // null: not written
  float* S_out;           // or null
  // backward
  const void* d_o;
  const float* dS_out;    // or null (zeros)
  void* dq;
  void* dk_;
  void* dv_;
  float* dlog_alpha;
  float* dbeta;
  float* dS0;             // or null
  // scratch (null where the call does not need them)
  float* w;               // [tokens][H][dv]: the written values
  float* dw;              // [tokens][H][dv]: their gradients
  float* chunk_S;         // [slots][H][dk][dv]: the state before each chunk
  float* chunk_dS;        // [slots][H][dk][dv]: the gradient of the state behind each chunk
  float* part;            // [2][tokens][H][dk]: dq and dk per value head where heads share keys
  unsigned char* tri;     // [slots][H][kTriBytes]
  unsigned char* kq;      // [slots][HK, KDA: H][kq_bytes]
  uint32_t* status;
  long long tokens;
  int seqs, H, HK, dk, dv, elem, slots;
};

// ------------------------------------------------------------------ activations
// elem is a seed_factors value; arithmetic is float32, stores round to nearest even.
SEED_DEV float4 act_ld4(const void* p, long long i, int elem) {
  if (elem == SEED_FACTORS_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  if (elem == SEED_FACTORS_F16) return fac_ld4(static_cast<const __half*>(p) + i);
  return fac_ld4(static_cast<const __nv_bfloat16*>(p) + i);
}
SEED_DEV float act_ld(const void* p, long long i, int elem) {
  if (elem == SEED_FACTORS_F32) return static_cast<const float*>(p)[i];
  if (elem == SEED_FACTORS_F16) return fac_to_f(static_cast<const __half*>(p)[i]);
  return fac_to_f(static_cast<const __nv_bfloat16*>(p)[i]);
}
SEED_DEV void act_st4(void* p, long long i, float4 x, int elem) {
  const float e[4] = {x.x, x.y, x.z, x.w};
  if (elem == SEED_FACTORS_F32) fac_st<float, 4>(static_cast<float*>(p) + i, e);
  else if (elem == SEED_FACTORS_F16) fac_st<__half, 4>(static_cast<__half*>(p) + i, e);
  else fac_st<__nv_bfloat16, 4>(static_cast<__nv_bfloat16*>(p) + i, e);
}
SEED_DEV void act_st(void* p, long long i, float x, int elem) {
  if (elem == SEED_FACTORS_F32) static_cast<float*>(p)[i] = x;
  else if (elem == SEED_FACTORS_F16) static_cast<__half*>(p)[i] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}
// f(T{}) with T the activation type: around loops of loads, which must not branch on
// elem between one load and the next (each would wait for the one before).
template <typename F>
SEED_DEV void act_type(int elem, F&& f) {
  if (elem == SEED_FACTORS_F32) f(float{});
  else if (elem == SEED_FACTORS_F16) f(__half{});
  else f(__nv_bfloat16{});
}
// N values `step` apart (zeros from the left-th on).  All loads are issued before the
// first conversion: a conversion under the loads' predicate becomes a branch per value,
// each waiting for its load (32 bf16 values of 48 heads: 20,000 cycles against 1,000).
template <typename T, int N>
SEED_DEV void act_ld_rows(const T* src, long long step, int left, float (&x)[N]) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int e = 0; e < N; ++e, src += step) {
      x[e] = 0.f;
      if (e < left) x[e] = *src;
    }
  } else {
    uint16_t raw[N];
#pragma unroll
    for (int e = 0; e < N; ++e, src += step) {
      raw[e] = 0;
      if (e < left) raw[e] = *reinterpret_cast<const uint16_t*>(src);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      T t;
      memcpy(&t, &raw[e], 2);
      x[e] = fac_to_f(t);
    }
  }
}
// The stores that go with it.
template <typename T, int N>
SEED_DEV void act_st_rows(T* dst, long long step, int left, const float (&x)[N]) {
  T t[N];
#pragma unroll
  for (int e = 0; e < N; ++e) t[e] = fac_from_f<T>(x[e]);
#pragma unroll
  for (int e = 0; e < N; ++e, dst += step)
    if (e < left) *dst = t[e];
}
// N groups of eight consecutive values, `step` elements apart.
template <typename T, int N>
SEED_DEV void act_ld8_rows(const T* src, long long step, int left, float (&x)[N][8]) {
  constexpr int Q = sizeof(T) / 2;      // 16-byte loads per group
  uint4 raw[N][Q];
#pragma unroll
  for (int e = 0; e < N; ++e)
#pragma unroll
    for (int y = 0; y < Q; ++y) {
      raw[e][y] = make_uint4(0, 0, 0, 0);
      if (e < left) raw[e][y] = reinterpret_cast<const uint4*>(src + e * step)[y];
    }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    T t[8];
    memcpy(t, raw[e], sizeof(t));
#pragma unroll
    for (int y = 0; y < 8; ++y) x[e][y] = fac_to_f(t[y]);
  }
}
// Whether x, once stored as elem, is finite.
SEED_DEV bool act_finite(float x, int elem) {
  return isfinite(elem == SEED_FACTORS_F16 ? fac_round<__half>(x)
                                           : elem == SEED_FACTORS_BF16 ? fac_round<__nv_bfloat16>(x) : x);
}

// ------------------------------------------------------------------ packed sequences
// Sequence s holds the rows offsets[s] .. offsets[s+1] of the packed arrays.  An
// entry outside [0, tokens], or behind its successor, makes the sequence empty
// (SEED_FLAG_BADINDEX): no row outside the arrays is ever touched.
struct SeqRange {
  long long first;
  int len;
  int slot0;     // first chunk slot
};
SEED_DEV SeqRange seq_range(const ScanParams& p, int s, bool raise) {
  const long long a = p.offsets[s], b = p.offsets[s + 1];
  if (a < 0 || b < a || b > p.tokens) {
    if (raise) raise_flag(p.status, SEED_FLAG_BADINDEX);
    return {0, 0, 0};
  }
  return {a, (int)(b - a), (int)(a / kChunk) + s};
}

// Chunk slots: chunk i of sequence s is slot offsets[s] / kChunk + s + i.  The slots
// of different sequences never meet (floor(b/C) - floor(a/C) + 1 >= ceil((b-a)/C)),
// all lie below tokens / kChunk + seqs, and the host needs no sequence length.
// Returns false for a slot that holds no chunk.
struct ChunkAt {
  int seq, index, n;      // n: tokens of the chunk
  long long first;        // its first row
  bool last;              // the sequence's last chunk
};
SEED_DEV bool chunk_at(const ScanParams& p, int slot, ChunkAt* c) {
  // whole warps: the last sequence whose first slot is not behind `slot`, 32 probes a step
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.seqs;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    bool in = at < n;
    if (in) {
      const int off = p.offsets[lo + at];
      in = (off < 0 ? 0 : off / kChunk) + lo + at <= slot;
    }
    const unsigned below = __ballot_sync(0xffffffffu, in);
    const int last = below ? 31 - __clz(below) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  const SeqRange r = seq_range(p, lo, false);
  const int i = slot - r.slot0;
  if (i < 0 || (long long)i * kChunk >= r.len) return false;
  c->seq = lo;
  c->index = i;
  c->n = min(kChunk, r.len - i * kChunk);
  c->first = r.first + (long long)i * kChunk;
  c->last = (i + 1) * (long long)kChunk >= r.len;
  return true;
}

// ------------------------------------------------------------------ launchers
// One or two tokens per sequence, forward only (seed_scan_one.cu).
int launch_scan_one(const ScanParams& p, int form, cudaStream_t st);
// Token-by-token kernels (seed_scan_step.cu).
int launch_scan_step(const ScanParams& p, int form, cudaStream_t st);
int launch_scan_step_back(const ScanParams& p, int form, cudaStream_t st);
// What the passes need of every chunk (seed_scan_prep.cuh), d_k in {64, 128}.
template <typename T>
int launch_scan_prep_as(const ScanParams& p, int form, cudaStream_t st);
// The chunked pass on the tensor cores for activations of type T (seed_scan_pass.cuh),
// d_k and d_v in {64, 128}; writes w and chunk_S instead of o and S_out where chunk_S is set.
template <typename T>
int launch_scan_pass_as(const ScanParams& p, int form, cudaStream_t st);
// The reverse recurrence on the tensor cores (seed_scan_back.cuh), behind launch_scan_prep_as.
template <typename T>
int launch_scan_back_as(const ScanParams& p, int form, cudaStream_t st);
// Gradients of each chunk from its states (seed_scan_grad.cu).
int launch_scan_grad(const ScanParams& p, int form, cudaStream_t st);
// Sum of dq and dk over the heads that share a key head.
int launch_scan_share(const ScanParams& p, cudaStream_t st);

}  // namespace seed

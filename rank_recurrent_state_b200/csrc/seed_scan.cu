// seed_scan.cu -- the dense scan and its backward pass: scratch layout and the order
// of the launches.  The scratch lies in the caller's workspace behind the status
// words and is written anew by every call.
#include "seed_scan.cuh"

namespace seed {

namespace {

constexpr size_t kScratch0 = 256;      // the status words come first

struct Carver {
  size_t at = kScratch0;
  unsigned char* base;
  template <typename T>
  T* take(long long n) {
    T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += ((size_t)n * sizeof(T) + 255) & ~(size_t)255;
    return p;
  }
};

// The chunked kernels take d_k and d_v of 64 and 128; sequences up to step_most tokens, and
// smaller heads, go token by token.  The chunked kernels cost a whole chunk however short
// it is, the token-by-token ones a fixed time per token and, once their blocks fill the
// SMs, work per token and head.  Measured (us, 128 x 128 bf16, forward; step / chunked): GDN 48
// heads 32 tokens 42 / 44, 48 tokens 51 / 44; 768 heads 8 tokens 101 / 134, 16 tokens 163 /
// 139.  KDA, whose chunks cost more to prepare: 48 heads 48 tokens 51 / 55, 64 tokens 61 /
// 56; 768 heads 16 tokens 171 / 244, 32 tokens 292 / 254.  (Backward: the same crossings.)
int step_most(const seed_scan_dims& d) {
  const bool many = (long long)d.seqs * d.heads >= 2 * 148, kda = d.form == SEED_KDA;
  return many ? (kda ? 24 : 10) : (kda ? 48 : 32);
}
bool chunked(const ScanParams& p, const seed_scan_dims& d) {
  return p.dk >= 64 && p.dv >= 64 && d.max_len > step_most(d);
}
// One or two tokens per sequence: the kernel that reads the states in whole rows (768 heads,
// one token 36 us against 64 token by token, two tokens 42 against 69, eight 110 against 101).
constexpr int kOneMost = 2;

// Assigns the scratch pointers (null base: only counts) and returns the bytes used.
size_t carve(ScanParams& p, const seed_scan_dims& d, bool backward, void* ws) {
  Carver c;
  c.base = static_cast<unsigned char*>(ws);
  if (chunked(p, d)) {
    const bool two = scan_two_terms(d.form, d.elem == SEED_FACTORS_F32);
    p.tri = c.take<unsigned char>((long long)p.slots * p.H * kTriBytes);
    p.kq = c.take<unsigned char>((long long)p.slots * (d.form == SEED_KDA ? p.H : p.HK) * kq_bytes(d.form, p.dk, two));
  }
  if (backward) {
    const long long rows = p.tokens * p.H, mats = (long long)p.slots * p.H * p.dk * p.dv;
    p.w = c.take<float>(rows * p.dv);
    p.dw = c.take<float>(rows * p.dv);
    p.chunk_S = c.take<float>(mats);
    p.chunk_dS = c.take<float>(mats);
    if (p.H != p.HK) p.part = c.take<float>(2 * rows * p.dk);
  }
  return c.at;
}

// Forward, or its recomputation: o, S_out, w and chunk_S where they are asked for.
int forward(const ScanParams& p, const seed_scan_dims& d, cudaStream_t st) {
  if (d.max_len <= kOneMost && d.tokens > 0 && p.chunk_S == nullptr) return launch_scan_one(p, d.form, st);
  if (!chunked(p, d)) return launch_scan_step(p, d.form, st);
  return with_factor_type_of(d.elem, [&](auto t) -> int {
    using T = decltype(t);
    if (d.tokens > 0) {
      if (const int rc = launch_scan_prep_as<T>(p, d.form, st)) return rc;
    }
    return launch_scan_pass_as<T>(p, d.form, st);
  });
}

ScanParams params_of(const seed_scan_dims& d) {
  ScanParams p{};
  p.tokens = d.tokens;
  p.seqs = d.seqs;
  p.H = d.heads;
  p.HK = d.k_heads;
  p.dk = d.d_k;
  p.dv = d.d_v;
  p.elem = d.elem;
  p.slots = (int)(d.tokens / kChunk) + d.seqs;
  return p;
}

}  // namespace

size_t scan_workspace_bytes(const seed_scan_dims& d, bool backward) {
  ScanParams p = params_of(d);
  return carve(p, d, backward, nullptr);
}

int launch_scan(const seed_scan_dims& d, const int32_t* offsets, const void* q, const void* k, const void* v,
                const float* alpha, const float* beta, const float* S0, void* o, float* S_out, void* ws,
                cudaStream_t st) {
  ScanParams p = params_of(d);
  carve(p, d, false, ws);
  p.offsets = offsets;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.S0 = S0;
  p.o = o;
  p.S_out = S_out;
  p.status = static_cast<uint32_t*>(ws);
  return forward(p, d, st);
}

int launch_scan_backward(const seed_scan_dims& d, const int32_t* offsets, const void* q, const void* k, const void* v,
                         const float* alpha, const float* beta, const void* d_o, const float* S0, const float* dS_out,
                         void* dq, void* dk, void* dv, float* dlog_alpha, float* dbeta, float* dS0, void* ws,
                         cudaStream_t st) {
  ScanParams p = params_of(d);
  carve(p, d, true, ws);
  p.offsets = offsets;
  p.q = q;
  p.k = k;
  p.v = v;
  p.alpha = alpha;
  p.beta = beta;
  p.S0 = S0;
  p.d_o = d_o;
  p.dS_out = dS_out;
  p.dq = dq;
  p.dk_ = dk;
  p.dv_ = dv;
  p.dlog_alpha = dlog_alpha;
  p.dbeta = dbeta;
  p.dS0 = dS0;
  p.status = static_cast<uint32_t*>(ws);
  int rc;
  if ((rc = forward(p, d, st))) return rc;                        // w and the state before each chunk
  // dw, the gradient behind each chunk, dS0
  if (chunked(p, d))
    rc = with_factor_type_of(d.elem, [&](auto t) -> int { return launch_scan_back_as<decltype(t)>(p, d.form, st); });
  else
    rc = launch_scan_step_back(p, d.form, st);
  if (rc) return rc;
  if (d.tokens == 0) return SEED_OK;
  if ((rc = launch_scan_grad(p, d.form, st))) return rc;
  return p.part ? launch_scan_share(p, st) : SEED_OK;
}

}  // namespace seed

// seed_tree.cu -- a tree of drafted tokens read against the stored state, and the
// commit of its accepted path.
//
// Node t of a request's tree continues its parent's state, the roots the stored one,
// S = a vbar^T + U V^T.  With B_t the product of the decays on the path to t and D_tj
// that behind its ancestor j, every node's state is
//     S_t = B_t S + sum_{j on the path to t, t included} D_tj k_j w_j^T
//     w_t = beta_t (v_t - read(B_t k_t) - sum_{ancestors j} (k_t . D_tj k_j) w_j)
//     o_t = read(B_t q_t) + sum_{j on the path, t included} (q_t . D_tj k_j) w_j
//     read(x) = S^T x = vbar (a . x) + V (U^T x)
// (Mamba-2: w_t = beta_t v_t).  So the stored columns are read once for all nodes,
// and no node's d_k x d_v state is ever formed.
//
// One block per (request, head).  Decays are products along a node's path to the root,
// never quotients (a zero decay is an ordinary value).  With one decay per head a thread
// walks the path of each node, and the dot products of all nodes' k and q with the stored
// columns, a and the nodes' k are one small product from shared memory.  With decays per
// channel a warp walks the path with the running decays in registers, which leaves
// k_t . D_tj k_j, q_t . D_tj k_j and the decayed k_t, q_t for the product with the columns.
// Then each thread owns a value channel and resolves the nodes in order.
//
// Measured: 3,072 trees of 16 nodes over 16-32 stored columns (GDN, 128 x 128 float32) 134
// us, their bytes 27 us; 1,024 trees of 32 nodes (KDA, bf16 factors) 171 us.  Bound by the
// latency of the phases, of which three blocks per SM overlap: the dot products take 14,000
// of a block's 45,000 cycles, the nodes in turn 16,000, the loads the first 10,000.
#include "seed_decode.cuh"
#include "seed_tma.cuh"

namespace seed {

namespace {

constexpr int kNT = 128;

struct TreeParams {
  const int32_t* parent;
  const float* q;
  const float* k;
  const float* v;
  const float* alpha;
  const float* beta;
  float* o;
  float* w;
  const float* a;
  const void* U;
  const void* V;
  const float* scale;
  const int32_t* ncols;
  const float* vbar;
  uint32_t* status;
  int B, L, H, layer, m, slen, N, dk, dv;
};

// Shared-memory layout (floats).  The stored V and the nodes' v are staged behind the rest
// where at least two blocks then still share an SM: read where they are needed, they cost
// the column phase a trip to memory every few columns (200 of 230 us of a batch of 3072
// trees of 16 nodes were spent waiting).
struct TreeSmem {
  int rows, xs, us, ys, kk, pp, vs, vv, total;      // offsets; rows = 2 N rounded up to a multiple of 16
  bool staged;
  __host__ __device__ TreeSmem(int N, int m, int dk, int dv, int elem_bytes) {
    rows = (2 * N + 15) & ~15;
    xs = 0;
    us = xs + rows * (dk + 8);
    const int u1 = ((m + 1 + 3) & ~3) * (dk + 8), w1 = N * dv;
    ys = us + (u1 > w1 ? u1 : w1);
    const int y1 = (m + 1) * rows, k1 = N * (dk + 8);
    kk = ys + (y1 > k1 ? y1 : k1);
    pp = kk + N * N;
    vs = (pp + N * N + 3) & ~3;
    vv = vs + (m * dv * elem_bytes + 15) / 16 * 4;
    total = vv + N * dv;
    staged = total * 4 <= 112 * 1024;
    if (!staged) total = vs;
  }
};

template <int FORM, int DK, int DV, typename TS>
__global__ void __launch_bounds__(kNT) decode_tree_kernel(const TreeParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  extern __shared__ __align__(16) float smf[];
  __shared__ int s_par[SEED_MAX_NODES];
  __shared__ __align__(16) float s_al[SEED_MAX_NODES], s_be[SEED_MAX_NODES], s_B[SEED_MAX_NODES], s_sc[SEED_MAX_COLS + 1];
  __shared__ unsigned long long s_anc[SEED_MAX_NODES];     // ancestors, the node itself left out
  constexpr int dk = DK, dv = DV, PK = DK + 8, E = DK < 32 ? 1 : DK / 32;
  const int N = p.N;
  const TreeSmem lay(N, p.m, dk, dv, sizeof(TS));
  float* xs = smf + lay.xs;      // rows t: k_t, rows rows/2 + t: q_t (KDA: decayed by B_t)
  float* us = smf + lay.us;      // true U columns, then a; later w
  float* ys = smf + lay.ys;      // KDA: the nodes' k; then [column][row]
  float* kk = smf + lay.kk;
  float* pp = smf + lay.pp;
  const int half = lay.rows / 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const long long unit = ((long long)b * p.L + p.layer) * p.H + h;
  const int c = p.ncols[unit];
  if (c < 0 || c > p.m) {
    if (tid == 0) raise_flag(p.status, SEED_FLAG_BADCOLS);
    return;
  }
  const float* vb = p.vbar + ((long long)p.layer * p.H + h) * dv;

  // ---- q and k, the stored columns and the nodes' v on their way
  const long long row = (long long)b * N * p.H + h;     // token t: row + t H
  constexpr int q4 = dk / 4;
  constexpr bool kRawU = !KDA && std::is_same<TS, float>::value;      // U's scales go to its dot products
  float* const kt_rows = KDA ? ys : xs;                 // [t][PK]: the nodes' k
  for (int e = tid; e < half * q4; e += kNT) {
    const int t = e / q4, i = 4 * (e % q4);
    const long long at = (row + (long long)t * p.H) * dk + i;
    if (t < N) {
      cp_async16(kt_rows + t * PK + i, p.k + at);
      cp_async16(xs + (half + t) * PK + i, p.q + at);
    } else {
      if (!KDA) st4(xs + t * PK + i, zero4());
      st4(xs + (half + t) * PK + i, zero4());
    }
  }
  if constexpr (kRawU) {
    const float* Ug = static_cast<const float*>(p.U) + unit * (long long)p.m * dk;
    for (int e = tid; e < c * q4; e += kNT) cp_async16(us + (e / q4) * PK + 4 * (e % q4), Ug + 4 * e);
  }
  const TS* Vg = static_cast<const TS*>(p.V) + unit * (long long)p.m * dv;
  TS* vs = reinterpret_cast<TS*>(smf + lay.vs);
  float* vv = smf + lay.vv;
  if (lay.staged) {
    constexpr int per = 16 / (int)sizeof(TS);
    for (int e = tid; e < c * dv / per; e += kNT) cp_async16(vs + e * per, Vg + e * per);
    for (int e = tid; e < N * dv / 4; e += kNT) {
      const int t = e / (dv / 4), i = 4 * (e % (dv / 4));
      cp_async16(vv + t * dv + i, p.v + (((long long)b * N + t) * p.H + h) * dv + i);
    }
  }
  cp_async_commit();

  // ---- the tree: s_par[t] = parent, or -2 for an unused node.  A node is used when
  // every step of its path goes to an earlier node and ends at -1.
  if (tid < N) s_par[tid] = p.parent[(long long)b * N + tid];
  __syncthreads();
  int par = -2;
  bool bad_tree = false;
  if (tid < N) {
    par = s_par[tid];
    if (par >= -1) {
      int u = tid;
      while (u >= 0) {
        const int up = s_par[u];
        if (up < -1 || up >= u) {
          bad_tree = true;
          break;
        }
        u = up;
      }
      if (bad_tree) par = -2;
    } else {
      par = -2;
    }
  }
  __syncthreads();
  if (tid < N) s_par[tid] = par;
  if (bad_tree && h == 0) raise_flag(p.status, SEED_FLAG_BADINDEX);
  __syncthreads();

  // ---- stored columns (true U) and a, beside them
  const TS* U = static_cast<const TS*>(p.U) + unit * (long long)p.m * dk;
  const float* sc = p.scale + unit * p.slen;
  if constexpr (!kRawU) {
#pragma unroll 8
    for (int e = tid; e < c * q4; e += kNT) {
      const int j = e / q4, i = 4 * (e % q4);
      float4 x = fac_ld4(U + (long long)j * dk + i);
      if constexpr (KDA) x = mul4(x, ld4(sc + i));
      st4(us + j * PK + i, x);
    }
  }
  if constexpr (!KDA) {
    for (int j = tid; j < c; j += kNT) s_sc[j] = sc[j];
    if (tid == 0) s_sc[c] = 1.f;      // a
  }
  for (int i = tid; i < dk; i += kNT) us[c * PK + i] = p.a[unit * dk + i];
  if (!KDA && tid < N) s_al[tid] = p.alpha[row + (long long)tid * p.H];
  if (tid < N) s_be[tid] = p.beta[row + (long long)tid * p.H];
  cp_async_wait<0>();
  __syncthreads();

  // ---- paths
  if constexpr (!KDA) {
    if (tid < half) {
      float f = 1.f;
      unsigned long long anc = 0;
      for (int j = tid < N && s_par[tid] >= -1 ? tid : -1; j >= 0; j = s_par[j]) {
        if (j != tid) anc |= 1ull << j;
        kk[tid * N + j] = pp[tid * N + j] = f;      // D_tj, times the dot products below
        f *= s_al[j];
      }
      s_B[tid] = f;
      if (tid < N) s_anc[tid] = anc;
    }
  }
  for (int t = KDA ? warp : half; t < half; t += kNT / 32) {
    float kt[E], qt[E], f[E];
    const bool used = t < N && s_par[t] >= -1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      kt[e] = used && i < dk ? ys[t * PK + i] : 0.f;
      qt[e] = used && i < dk ? xs[(half + t) * PK + i] : 0.f;      // (decayed in place below)
      f[e] = 1.f;
    }
    // four nodes of the path at a time: their eight dot products are summed over the warp
    // together
    unsigned long long anc = 0;
    int j = used ? t : -1;
    while (j >= 0) {
      float v[8] = {};
      int at[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        at[x] = j;
        if (j >= 0) {
          if (j != t) anc |= 1ull << j;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int i = lane + 32 * e;
            if (i < dk) {
              const float kj = f[e] * ys[j * PK + i];
              if constexpr (!M2) v[4 + x] = fmaf(kt[e], kj, v[4 + x]);
              v[x] = fmaf(qt[e], kj, v[x]);
              f[e] *= p.alpha[(row + (long long)j * p.H) * dk + i];
            }
          }
          j = s_par[j];
        }
      }
      const float tot = warp_xreduce<8>(v);      // value lane / 4
      const int which = lane >> 2, node = at[0] * ((which & 3) == 0) + at[1] * ((which & 3) == 1) +
                                          at[2] * ((which & 3) == 2) + at[3] * ((which & 3) == 3);
      if ((lane & 3) == 0 && node >= 0) {
        if (which < 4) pp[t * N + node] = tot;
        else if (!M2) kk[t * N + node] = tot;
      }
    }
    if (lane == 0 && t < N) s_anc[t] = anc;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      if (i < dk) {
        xs[t * PK + i] = f[e] * kt[e];
        xs[(half + t) * PK + i] = f[e] * qt[e];
      }
    }
  }
  __syncthreads();

  // ---- ys[j][row] = x_row . (column j); column c is a, and with one decay per head the
  // nodes' k follow.  Tiles of 4 rows (a quarter of the rows apart) x 4 columns, two lanes
  // along the channels each: eight lanes then read 128 bytes of different banks.
  const int rq = lay.rows / 4;
  const int cols = KDA ? c + 1 : c + 1 + N, ct = (cols + 3) / 4;
  for (int e0 = 0; e0 < rq * ct; e0 += kNT / 2) {
    const int e = e0 + tid / 2, part = tid & 1;
    const bool on = e < rq * ct;
    const int r0 = on ? e % rq : 0, j0 = on ? 4 * (e / rq) : 0;
    float acc[4][4] = {};
    if (on) {
      const float* xr = xs + r0 * PK + 4 * part;
      const float* ur = xs + 4 * part;
      int at[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int col = j0 + y < cols ? j0 + y : cols - 1;
        at[y] = col <= c ? lay.us - lay.xs + col * PK : (col - c - 1) * PK;
      }
#pragma unroll 4
      for (int i = 0; i < dk; i += 8) {
        float4 u[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) u[y] = ld4(ur + at[y] + i);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (M2 && r < 2) continue;          // Mamba-2 reads with q alone, rows from the half on
          const float4 x = ld4(xr + r * rq * PK + i);
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[r][y] += dot4(x, u[y]);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r][y] += __shfl_xor_sync(0xffffffffu, acc[r][y], 1);
      const int col = j0 + y;
      if (on && part == (y & 1) && col < cols) {
#pragma unroll
        for (int r = M2 ? 2 : 0; r < 4; ++r) {
          const int row_ = r0 + r * rq, t = r0 + (r & 1) * rq;      // (2 rq = half)
          if (col <= c) ys[col * lay.rows + row_] = KDA ? acc[r][y] : acc[r][y] * (s_B[t] * s_sc[col]);
          else if (t < N) (r < 2 ? kk : pp)[t * N + col - c - 1] *= acc[r][y];
        }
      }
    }
  }
  __syncthreads();

  // ---- value channels: a thread resolves its channel's w and o, nodes in order
  float* ws = us;
  bool bad = false;
  for (int col = tid; col < dv; col += kNT) {
    const TS* V = (lay.staged ? vs : Vg) + col;
    const float vbc = vb[col];
    for (int t0 = 0; t0 < N; t0 += 8) {
      float rk[8], rq[8], vt[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        vt[r] = 0.f;
        if (t0 + r < N) vt[r] = lay.staged ? vv[(t0 + r) * dv + col] : p.v[(row + (long long)(t0 + r) * p.H) * dv + col];
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        rk[r] = vbc * ys[c * lay.rows + t0 + r];
        rq[r] = vbc * ys[c * lay.rows + half + t0 + r];
      }
#pragma unroll 4
      for (int j = 0; j < c; ++j) {
        const float vj = fac_to_f(V[j * dv]);
        const float* y = ys + j * lay.rows + t0;
        if constexpr (!M2) {
          const float4 a0 = ld4(y), a1 = ld4(y + 4);
          rk[0] = fmaf(a0.x, vj, rk[0]); rk[1] = fmaf(a0.y, vj, rk[1]);
          rk[2] = fmaf(a0.z, vj, rk[2]); rk[3] = fmaf(a0.w, vj, rk[3]);
          rk[4] = fmaf(a1.x, vj, rk[4]); rk[5] = fmaf(a1.y, vj, rk[5]);
          rk[6] = fmaf(a1.z, vj, rk[6]); rk[7] = fmaf(a1.w, vj, rk[7]);
        }
        const float4 b0 = ld4(y + half), b1 = ld4(y + half + 4);
        rq[0] = fmaf(b0.x, vj, rq[0]); rq[1] = fmaf(b0.y, vj, rq[1]);
        rq[2] = fmaf(b0.z, vj, rq[2]); rq[3] = fmaf(b0.w, vj, rq[3]);
        rq[4] = fmaf(b1.x, vj, rq[4]); rq[5] = fmaf(b1.y, vj, rq[5]);
        rq[6] = fmaf(b1.z, vj, rq[6]); rq[7] = fmaf(b1.w, vj, rq[7]);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int t = t0 + r;
        if (t < N) {
          const long long rt = row + (long long)t * p.H;
          const bool used = s_par[t] >= -1;
          float w = 0.f, o = 0.f;
          if (used) {
            float x = vt[r];
            o = rq[r];
            if constexpr (!M2) x -= rk[r];
            // ancestors alone: another branch's values (NaN, say) never come in
            for (unsigned long long anc = s_anc[t]; anc; anc &= anc - 1) {
              const int j = __ffsll(anc) - 1;
              const float wj = ws[j * dv + col];
              if constexpr (!M2) x = fmaf(-kk[t * N + j], wj, x);
              o = fmaf(pp[t * N + j], wj, o);
            }
            w = s_be[t] * x;
            o = fmaf(pp[t * N + t], w, o);
            bad = bad || !(isfinite(w) && isfinite(o));
          }
          ws[t * dv + col] = w;
          p.w[rt * dv + col] = w;
          p.o[rt * dv + col] = o;
        }
      }
    }
  }
  if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
}

// ------------------------------------------------------------------ commit
// The accepted path's nodes as so many decode steps, without their read-outs: the sink
// coefficient's own recurrence a+ = a' + s k with s = beta (omega - a' . k), a' = the
// decayed a (Mamba-2: s = beta omega), the column pair (k, w - s vbar), the lazy scales.
struct CommitParams {
  const int32_t* parent;
  const int32_t* leaf;
  const float* k;
  const float* v;
  const float* alpha;
  const float* beta;
  const float* w;
  float* a;
  void* U;
  void* V;
  float* scale;
  int32_t* ncols;
  const float* vbar;
  uint32_t* status;
  int B, L, H, layer, m, slen, N, dk, dv;
};

template <int FORM, typename TS>
__global__ void __launch_bounds__(kNT) tree_commit_kernel(const CommitParams p) {
  constexpr bool KDA = FORM == SEED_KDA, M2 = FORM == SEED_MAMBA2;
  __shared__ int s_path[SEED_MAX_NODES], s_par[SEED_MAX_NODES];
  __shared__ float s_om[SEED_MAX_NODES], s_after[SEED_MAX_NODES + 1];
  __shared__ float s_red[2][kNT / 32];
  __shared__ int s_len;
  const int N = p.N, dk = p.dk, dv = p.dv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.H, h = blockIdx.x - b * p.H;
  const long long unit = ((long long)b * p.L + p.layer) * p.H + h;
  const int leaf = p.leaf[b];
  if (leaf < 0) return;
  const int c = p.ncols[unit];
  if (tid < N) s_par[tid] = p.parent[(long long)b * N + tid];
  __syncthreads();
  if (tid == 0) {
    int len = 0, u = leaf;
    bool ok = leaf < N;
    while (ok && u >= 0) {
      const int up = s_par[u];
      if (up < -1 || up >= u) ok = false;
      s_path[len++] = u;
      u = up;
    }
    uint32_t flag = 0;
    if (!ok) flag = SEED_FLAG_BADINDEX;
    else if (c < 0 || c > p.m) flag = SEED_FLAG_BADCOLS;
    else if (c + len > p.m) flag = SEED_FLAG_FULL;
    if (flag) raise_flag(p.status, flag);
    for (int i = 0; i < len / 2; ++i) {      // root first
      const int x = s_path[i];
      s_path[i] = s_path[len - 1 - i];
      s_path[len - 1 - i] = x;
    }
    s_len = flag ? 0 : len;
  }
  __syncthreads();
  const int len = s_len;
  if (len == 0) return;
  const long long row = (long long)b * N * p.H + h;
  const float* vb = p.vbar + ((long long)p.layer * p.H + h) * dv;
  float vv = 0.f;
  for (int e = lane; e < dv; e += 32) vv = fmaf(vb[e], vb[e], vv);
  vv = group_sum<32>(vv);
  if (!(vv > 0.f)) {
    if (tid == 0) raise_flag(p.status, SEED_FLAG_ZERO_VBAR);
    return;
  }
  for (int i = warp; i < len; i += kNT / 32) {
    const float* v = p.v + (row + (long long)s_path[i] * p.H) * dv;
    float x = 0.f;
    for (int e = lane; e < dv; e += 32) x = fmaf(v[e], vb[e], x);
    x = group_sum<32>(x);
    if (lane == 0) s_om[i] = x / vv;
  }
  if (!KDA && tid == 0) {
    float f = 1.f;
    for (int i = len - 1; i >= 0; --i) {      // s_after[i]: decay behind node i; [len] of the whole path
      s_after[i] = f;
      f *= p.alpha[row + (long long)s_path[i] * p.H];
    }
    s_after[len] = f;
  }
  __syncthreads();

  bool bad = false;
  const bool on = tid < dk;
  const float vbc = tid < dv ? vb[tid] : 0.f;      // d_k, d_v <= 128 threads
  float a = on ? p.a[unit * dk + tid] : 0.f;
  float P = KDA && on ? p.scale[unit * dk + tid] : 1.f;
  TS* U = static_cast<TS*>(p.U) + (unit * p.m + c) * (long long)dk;
  TS* V = static_cast<TS*>(p.V) + (unit * p.m + c) * (long long)dv;
  float k_next = 0.f, al_next = 1.f, be_next = 0.f, w_next = 0.f;      // the next node's values (w: channel tid)
  auto fetch = [&](int i) {
    const long long rt = row + (long long)s_path[i] * p.H;
    if (on) k_next = p.k[rt * dk + tid];
    if (!KDA || on) al_next = KDA ? p.alpha[rt * dk + tid] : p.alpha[rt];
    be_next = p.beta[rt];
    if (tid < dv) w_next = p.w[rt * dv + tid];
  };
  fetch(0);
  for (int i = 0; i < len; ++i) {
    const float k = k_next, al = al_next, be = be_next, w = w_next;
    if (i + 1 < len) fetch(i + 1);
    a *= al;
    float ka = 0.f;
    if constexpr (!M2) {
      ka = group_sum<32>(k * a);
      if (lane == 0) s_red[i & 1][warp] = ka;
      __syncthreads();          // the other half is written only behind the next one
      ka = 0.f;
#pragma unroll
      for (int x = 0; x < kNT / 32; ++x) ka += s_red[i & 1][x];
    }
    const float s = be * (s_om[i] - ka);
    a = fmaf(s, k, a);
    if (on) {
      float u = k;
      if constexpr (KDA) {
        P *= al;
        u = k / P;
      }
      bad = bad || !isfinite(fac_round<TS>(u));
      U[(long long)i * dk + tid] = fac_from_f<TS>(u);
    }
    if (tid < dv) {
      const float x = fmaf(-s, vbc, w);
      bad = bad || !isfinite(fac_round<TS>(x));
      V[(long long)i * dv + tid] = fac_from_f<TS>(x);
    }
  }
  if (on) {
    p.a[unit * dk + tid] = a;
    bad = bad || !isfinite(a);
    if constexpr (KDA) p.scale[unit * dk + tid] = P;
  }
  if constexpr (!KDA) {
    float* sc = p.scale + unit * p.slen;
    for (int j = tid; j < c + len; j += kNT) sc[j] = j < c ? s_after[len] * sc[j] : s_after[j - c];
  }
  if (tid == 0) p.ncols[unit] = c + len;
  if (bad) raise_flag(p.status, SEED_FLAG_NONFINITE);
}

template <int FORM, int DK, int DV, typename TS>
int launch_tree_t(const TreeParams& p, cudaStream_t st) {
  static LaunchCache cache;
  const size_t bytes = sizeof(float) * (size_t)TreeSmem(p.N, p.m, p.dk, p.dv, sizeof(TS)).total;
  constexpr size_t most = 220 * 1024;      // 64 nodes, 96 columns, d 128: 203 KB
  if (bytes > most) return SEED_ERR_SHAPE;
  int dev;
  if (int rc = cache.prepare(reinterpret_cast<const void*>(decode_tree_kernel<FORM, DK, DV, TS>), most, &dev)) return rc;
  decode_tree_kernel<FORM, DK, DV, TS><<<p.B * p.H, kNT, bytes, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

template <int FORM, typename TS>
int launch_commit_t(const CommitParams& p, cudaStream_t st) {
  tree_commit_kernel<FORM, TS><<<p.B * p.H, kNT, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SEED_OK : SEED_ERR_CUDA;
}

}  // namespace

int launch_decode_tree(const seed_dims& d, const seed_state& s, int layer, int n_nodes, const int32_t* parent,
                       const float* q, const float* k, const float* v, const float* alpha, const float* beta, float* o,
                       float* w, uint32_t* status, cudaStream_t st) {
  const TreeParams p{parent, q, k, v, alpha, beta, o, w, s.a, s.U, s.V, s.scale, s.ncols, s.vbar, status,
                     d.batch, d.layers, d.heads, layer, d.R + d.W, scale_len(d), n_nodes, d.d_k, d.d_v};
  return with_factor_type(d, [&](auto t) -> int {
    using TS = decltype(t);
#define SEED_TREE(F, K, V) \
  if (d.form == F && d.d_k == K && d.d_v == V) return launch_tree_t<F, K, V, TS>(p, st);
#define SEED_TREE_D(F) \
  SEED_TREE(F, 16, 16) SEED_TREE(F, 32, 32) SEED_TREE(F, 64, 64) SEED_TREE(F, 128, 128) SEED_TREE(F, 128, 64) SEED_TREE(F, 64, 128)
    SEED_TREE_D(SEED_GDN)
    SEED_TREE_D(SEED_KDA)
    SEED_TREE_D(SEED_MAMBA2)
#undef SEED_TREE_D
#undef SEED_TREE
    return SEED_ERR_SHAPE;
  });
}

int launch_tree_commit(const seed_dims& d, const seed_state& s, int layer, int n_nodes, const int32_t* parent,
                       const int32_t* leaf, const float* k, const float* v, const float* alpha, const float* beta,
                       const float* w, uint32_t* status, cudaStream_t st) {
  const CommitParams p{parent, leaf, k, v, alpha, beta, w, s.a, s.U, s.V, s.scale, s.ncols, s.vbar, status,
                       d.batch, d.layers, d.heads, layer, d.R + d.W, scale_len(d), n_nodes, d.d_k, d.d_v};
  return with_factor_type(d, [&](auto t) -> int {
    using TS = decltype(t);
    switch (d.form) {
      case SEED_GDN: return launch_commit_t<SEED_GDN, TS>(p, st);
      case SEED_KDA: return launch_commit_t<SEED_KDA, TS>(p, st);
      case SEED_MAMBA2: return launch_commit_t<SEED_MAMBA2, TS>(p, st);
    }
    return SEED_ERR_INVALID_ARG;
  });
}

}  // namespace seed

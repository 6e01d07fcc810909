// gdn_backward.cu -- gradients of the chunk form (C = 64 rows a chunk).
//
// Per (sequence, value head) and chunk, with entry state H, exit state H',
// cumulative gates G_r, D_rs = e^{G_r - G_s}, B = strictly lower (K K^T * D) and
// the strictly lower S = (I + B diag(beta))^-1 B:
//   X = V - e^G K H,  u = X - S (beta X),  H' = e^{G_C} H + (e^{G_C-G} K)^T (beta u).
// u_r is row r's delta (v_r - H^T k_r against its decayed state), so the chunk
// form and the token form share it.  With dH' the gradient of H':
//   Y = scale (Q K^T * D)^T dO + e^{G_C-G} K dH',  E = Y - S^T (beta Y),
//   dH = e^{G_C} dH' + scale (e^G Q)^T dO - (e^G K)^T (beta E).
// Neither scan needs the other, so both run side by side.  Then, per chunk,
//   dv = beta E,  dbeta = E . u,
//   P = scale (dO (beta u)^T) * D (with the diagonal),
//   N = -strictly lower ((beta E) (beta u)^T) * D,
//   dq = scale e^G (dO H^T) + P K,
//   dk = P^T Q + (N + N^T) K - e^G (beta E) H^T + e^{G_C-G} (beta u) dH'^T,
//   dg_r = <H', dH'> + sum_{s >= r} (q_s . dq_s - v_s . dv_s),
// the last because e^{G_r} enters only by scaling q_r up and v_r down.
//
// Gates reach the exponentials as differences of 64-bit cumulative sums, kept
// as two floats: a strong decay early in the chunk costs later rows nothing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int kBC = 64;         // rows of a chunk
constexpr int kScanCols = 32;   // state columns of a scan CTA
constexpr float kGateFloor = -1e4f;  // e^x is 0 in f32 far above it; keeps sums finite

// Where everything is in the workspace (element offsets are 64-bit).
struct BwdArgs {
  const uint16_t *q, *k, *v, *dout;
  const float *g, *beta;
  int qk_stride, v_stride, gb_stride;
  const int32_t* cu;
  int num_seqs, total_tokens, H_k, H_v;
  const float *h0, *dhT;
  uint16_t *dq, *dk, *dv;
  float *dg, *dbeta, *dh0;
  float scale;
  // workspace
  int32_t* cu_chunks;   // [num_seqs + 1]
  int32_t* chunk_seq;   // [max_chunks]
  int max_chunks;
  float2* G;            // [chunk][H_v][64] cumulative gates, high and low part
  float* S;             // [chunk][H_v][64][64]
  float* M;             // [chunk][H_v][64][64]  Q K^T * D, lower with the diagonal
  float* u;             // [chunk][H_v][64][D]
  float* E;             // [chunk][H_v][64][D]
  float* H;             // [chunk + sequence][H_v][D][D] entry states, then the final state
  float* dH;            // [chunk][H_v][D][D] gradient of the exit state
};

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
__device__ __forceinline__ float expdiff(float2 a, float2 b) {
  return expf((a.x - b.x) + (a.y - b.y));
}

// The rows of chunk i: sequence, first row, number of rows (0 where the row
// offsets are inconsistent).
struct ChunkRows {
  int seq, row0, rows;
};
__device__ __forceinline__ ChunkRows chunk_rows(const BwdArgs& a, int i) {
  ChunkRows c;
  c.seq = a.chunk_seq[i];
  const int lo = max(a.cu[c.seq], 0), hi = min(a.cu[c.seq + 1], a.total_tokens);
  c.row0 = lo + kBC * (i - a.cu_chunks[c.seq]);
  c.rows = max(0, min(kBC, hi - c.row0));
  return c;
}

// ---------------------------------------------------------------------------
// Prep: per (chunk, value head) G, M and S.
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) bwd_prep_kernel(BwdArgs a) {
  extern __shared__ float sm[];
  float* Ks = sm;                    // [64][D + 1]
  float* Qs = Ks + kBC * (D + 1);    // [64][D + 1]
  float* Bs = Qs + kBC * (D + 1);    // [64][65]
  float* Ss = Bs + kBC * 65;         // [64][65]
  __shared__ float2 Gs[kBC];
  __shared__ float bs[kBC];
  const int i = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (i >= a.cu_chunks[a.num_seqs]) return;
  const ChunkRows c = chunk_rows(a, i);
  const int hk = h / (a.H_v / a.H_k);
  const size_t unit = size_t(i) * a.H_v + h;
  for (int x = tid; x < kBC * D; x += 256) {
    const int r = x / D, j = x % D;
    const size_t at = size_t(c.row0 + r) * a.qk_stride + hk * D + j;
    Ks[r * (D + 1) + j] = r < c.rows ? bf16f(a.k[at]) : 0.f;
    Qs[r * (D + 1) + j] = r < c.rows ? bf16f(a.q[at]) : 0.f;
  }
  if (tid < kBC) bs[tid] = tid < c.rows ? a.beta[size_t(c.row0 + tid) * a.gb_stride + h] : 0.f;
  if (tid == 0) {
    double run = 0.0;
    for (int r = 0; r < kBC; ++r) {
      if (r < c.rows) {
        const float x = a.g[size_t(c.row0 + r) * a.gb_stride + h];
        run += x < kGateFloor ? kGateFloor : x;
      }
      const float hi = float(run);
      Gs[r] = make_float2(hi, float(run - double(hi)));
      a.G[unit * kBC + r] = Gs[r];
    }
  }
  __syncthreads();
  for (int x = tid; x < kBC * kBC; x += 256) {
    const int r = x / kBC, s = x % kBC;
    float kk = 0.f, qk = 0.f;
    if (s <= r) {
      for (int j = 0; j < D; ++j) {
        kk = fmaf(Ks[r * (D + 1) + j], Ks[s * (D + 1) + j], kk);
        qk = fmaf(Qs[r * (D + 1) + j], Ks[s * (D + 1) + j], qk);
      }
      const float e = expdiff(Gs[r], Gs[s]);
      kk *= e;
      qk *= e;
    }
    a.M[unit * kBC * kBC + x] = qk;
    Bs[r * 65 + s] = s < r ? kk : 0.f;
  }
  __syncthreads();
  // S = B - B diag(beta) S, row by row; thread = column
  if (tid < kBC) {
    const int j = tid;
    for (int r = 0; r < kBC; ++r) {
      float x = Bs[r * 65 + j];
      for (int s = 0; s < r; ++s) x = fmaf(-Bs[r * 65 + s] * bs[s], Ss[s * 65 + j], x);
      Ss[r * 65 + j] = x;
    }
  }
  __syncthreads();
  for (int x = tid; x < kBC * kBC; x += 256)
    a.S[unit * kBC * kBC + x] = Ss[(x / kBC) * 65 + x % kBC];
}

// ---------------------------------------------------------------------------
// Scans: one CTA per (sequence, value head, 32 state columns, direction).
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(128) bwd_scan_kernel(BwdArgs a) {
  extern __shared__ float sm[];
  float* Hs = sm;                      // [D][32]
  float* Ks = Hs + D * kScanCols;      // [64][D]
  float* Qs = Ks + kBC * D;            // [64][D]
  float* Xs = Qs + kBC * D;            // [64][32]
  float* Ss = Xs + kBC * kScanCols;    // [64][64]
  float* Ms = Ss + kBC * kBC;          // [64][64]
  float* Os = Ms + kBC * kBC;          // [64][32]
  __shared__ float eG[kBC], eT[kBC], bs[kBC], eCs;
  constexpr int SL = D / kScanCols;
  const int slice = blockIdx.x % SL, h = blockIdx.x / SL % a.H_v, b = blockIdx.x / SL / a.H_v;
  const bool back = blockIdx.y != 0;
  const int tid = threadIdx.x, j = tid % 32, w = tid / 32, col = slice * kScanCols + j;
  const int hk = h / (a.H_v / a.H_k);
  const int c0 = a.cu_chunks[b], n = a.cu_chunks[b + 1] - c0;
  const float* init = back ? a.dhT : a.h0;
  const size_t seq_state = (size_t(b) * a.H_v + h) * D * D;
  for (int x = w; x < D; x += 4)
    Hs[x * 32 + j] = init != nullptr ? init[seq_state + size_t(x) * D + col] : 0.f;
  for (int t = 0; t < n; ++t) {
    const int i = c0 + (back ? n - 1 - t : t);
    const ChunkRows c = chunk_rows(a, i);
    const size_t unit = size_t(i) * a.H_v + h;
    float* state = back ? a.dH + unit * D * D : a.H + (size_t(i + b) * a.H_v + h) * D * D;
    __syncthreads();
    for (int x = tid; x < kBC * D; x += 128) {
      const int r = x / D, d = x % D;
      const size_t at = size_t(c.row0 + r) * a.qk_stride + hk * D + d;
      Ks[x] = r < c.rows ? bf16f(a.k[at]) : 0.f;
      if (back) Qs[x] = r < c.rows ? bf16f(a.q[at]) : 0.f;
    }
    for (int x = tid; x < kBC * kBC; x += 128) {
      Ss[x] = a.S[unit * kBC * kBC + x];
      if (back) Ms[x] = a.M[unit * kBC * kBC + x];
    }
    if (back)
      for (int r = w; r < kBC; r += 4)
        Os[r * 32 + j] = r < c.rows
            ? a.scale * bf16f(a.dout[(size_t(c.row0 + r) * a.H_v + h) * D + col]) : 0.f;
    if (tid < kBC) {
      const float2 G = a.G[unit * kBC + tid], GC = a.G[unit * kBC + kBC - 1];
      eG[tid] = expf(G.x + G.y);
      eT[tid] = expdiff(GC, G);
      bs[tid] = tid < c.rows ? a.beta[size_t(c.row0 + tid) * a.gb_stride + h] : 0.f;
      if (tid == 0) eCs = expf(GC.x + GC.y);
    }
    for (int x = w; x < D; x += 4) state[size_t(x) * D + col] = Hs[x * 32 + j];
    __syncthreads();
    float y[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int r = w * 16 + m;
      float kh = 0.f;
      for (int d = 0; d < D; ++d) kh = fmaf(Ks[r * D + d], Hs[d * 32 + j], kh);
      if (!back) {
        const float vv = r < c.rows
            ? bf16f(a.v[size_t(c.row0 + r) * a.v_stride + h * D + col]) : 0.f;
        y[m] = vv - eG[r] * kh;
      } else {
        float acc = eT[r] * kh;
        for (int s = r; s < kBC; ++s) acc = fmaf(Ms[s * kBC + r], Os[s * 32 + j], acc);
        y[m] = acc;
      }
      Xs[r * 32 + j] = bs[r] * y[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int r = w * 16 + m;
      if (!back)
        for (int s = 0; s < r; ++s) y[m] = fmaf(-Ss[r * kBC + s], Xs[s * 32 + j], y[m]);
      else
        for (int s = r + 1; s < kBC; ++s) y[m] = fmaf(-Ss[s * kBC + r], Xs[s * 32 + j], y[m]);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const int r = w * 16 + m;
      (back ? a.E : a.u)[(unit * kBC + r) * D + col] = y[m];
      Xs[r * 32 + j] = bs[r] * y[m];
    }
    __syncthreads();
    for (int d = w; d < D; d += 4) {
      float acc = eCs * Hs[d * 32 + j];
      for (int r = 0; r < kBC; ++r) {
        if (!back)
          acc = fmaf(eT[r] * Ks[r * D + d], Xs[r * 32 + j], acc);
        else
          acc = fmaf(eG[r] * Qs[r * D + d], Os[r * 32 + j],
                     fmaf(-eG[r] * Ks[r * D + d], Xs[r * 32 + j], acc));
      }
      Hs[d * 32 + j] = acc;
    }
  }
  float* last = back ? (a.dh0 != nullptr ? a.dh0 + seq_state : nullptr)
                     : a.H + (size_t(c0 + n + b) * a.H_v + h) * D * D;
  if (last != nullptr)
    for (int x = w; x < D; x += 4) last[size_t(x) * D + col] = Hs[x * 32 + j];
}

// ---------------------------------------------------------------------------
// Grads: per (chunk, key head), the value heads of the group one after another.
// ---------------------------------------------------------------------------

// acc[4][NT] += A[64][K] B[N][K]^T, operands fetched element by element; thread
// (ty, tx) of 16 x 16 owns rows ty + 16 m and columns tx + 16 n.
template <int NT, class FA, class FB>
__device__ __forceinline__ void block_nt(float (&acc)[4][NT], int K, FA fa, FB fb, float* As,
                                         float* Bt) {
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  for (int k0 = 0; k0 < K; k0 += 32) {
    __syncthreads();
    for (int x = tid; x < 64 * 32; x += 256) As[(x / 32) * 33 + x % 32] = fa(x / 32, k0 + x % 32);
    for (int x = tid; x < 16 * NT * 32; x += 256)
      Bt[(x / 32) * 33 + x % 32] = fb(x / 32, k0 + x % 32);
    __syncthreads();
    for (int kk = 0; kk < 32; ++kk) {
      float av[4], bv[NT];
#pragma unroll
      for (int m = 0; m < 4; ++m) av[m] = As[(ty + 16 * m) * 33 + kk];
#pragma unroll
      for (int n = 0; n < NT; ++n) bv[n] = Bt[(tx + 16 * n) * 33 + kk];
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n] = fmaf(av[m], bv[n], acc[m][n]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(256) bwd_grads_kernel(BwdArgs a) {
  constexpr int NT = D / 16;
  extern __shared__ float sm[];
  float* As = sm;                 // [64][33]
  float* Bt = As + 64 * 33;       // [D][33]
  float* Ps = Bt + D * 33;        // [64][65]
  float* Ns = Ps + 64 * 65;       // [64][65]
  __shared__ float eG[kBC], eT[kBC], bs[kBC], dG[kBC];
  __shared__ float2 Gs[kBC];
  __shared__ float red[8];
  const int i = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  if (i >= a.cu_chunks[a.num_seqs]) return;
  const ChunkRows c = chunk_rows(a, i);
  const int vpg = a.H_v / a.H_k;
  auto Kf = [&](int r, int d) {
    return r < c.rows ? bf16f(a.k[size_t(c.row0 + r) * a.qk_stride + hk * D + d]) : 0.f;
  };
  auto Qf = [&](int r, int d) {
    return r < c.rows ? bf16f(a.q[size_t(c.row0 + r) * a.qk_stride + hk * D + d]) : 0.f;
  };
  float dqs[4][NT] = {}, dks[4][NT] = {};
  for (int h = hk * vpg; h < (hk + 1) * vpg; ++h) {
    const size_t unit = size_t(i) * a.H_v + h;
    const float* H = a.H + (size_t(i + c.seq) * a.H_v + h) * D * D;
    const float* H1 = H + size_t(a.H_v) * D * D;
    const float* dH = a.dH + unit * D * D;
    const float *u = a.u + unit * kBC * D, *E = a.E + unit * kBC * D;
    __syncthreads();
    if (tid < kBC) {
      Gs[tid] = a.G[unit * kBC + tid];
      const float2 GC = a.G[unit * kBC + kBC - 1];
      eG[tid] = expf(Gs[tid].x + Gs[tid].y);
      eT[tid] = expdiff(GC, Gs[tid]);
      bs[tid] = tid < c.rows ? a.beta[size_t(c.row0 + tid) * a.gb_stride + h] : 0.f;
    }
    __syncthreads();
    auto dOf = [&](int r, int d) {
      return r < c.rows ? bf16f(a.dout[(size_t(c.row0 + r) * a.H_v + h) * D + d]) : 0.f;
    };
    auto uf = [&](int r, int d) { return bs[r] * u[r * D + d]; };
    auto Ef = [&](int r, int d) { return bs[r] * E[r * D + d]; };
    {
      float p[4][4] = {}, nn[4][4] = {};
      block_nt<4>(p, D, dOf, uf, As, Bt);
      block_nt<4>(nn, D, Ef, uf, As, Bt);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int r = ty + 16 * m, s = tx + 16 * n;
          const float e = s <= r ? expdiff(Gs[r], Gs[s]) : 0.f;
          Ps[r * 65 + s] = a.scale * p[m][n] * e;
          Ns[r * 65 + s] = s < r ? -nn[m][n] * e : 0.f;
        }
    }
    float dq[4][NT] = {};
    block_nt<NT>(dq, D, dOf, [&](int x, int d) { return H[x * D + d]; }, As, Bt);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) dq[m][n] *= a.scale * eG[ty + 16 * m];
    block_nt<NT>(dq, kBC, [&](int r, int s) { return Ps[r * 65 + s]; },
                 [&](int x, int s) { return Kf(s, x); }, As, Bt);
    block_nt<NT>(dks, kBC, [&](int r, int s) { return Ps[s * 65 + r]; },
                 [&](int x, int s) { return Qf(s, x); }, As, Bt);
    block_nt<NT>(dks, kBC, [&](int r, int s) { return Ns[r * 65 + s] + Ns[s * 65 + r]; },
                 [&](int x, int s) { return Kf(s, x); }, As, Bt);
    block_nt<NT>(dks, D, [&](int r, int d) { return -eG[r] * Ef(r, d); },
                 [&](int x, int d) { return H[x * D + d]; }, As, Bt);
    block_nt<NT>(dks, D, [&](int r, int d) { return eT[r] * uf(r, d); },
                 [&](int x, int d) { return dH[x * D + d]; }, As, Bt);
    // dv, dbeta and dG: a row per warp at a time for the value columns
    for (int r = tid / 32; r < c.rows; r += 8) {
      float db = 0.f, vd = 0.f;
      for (int d = tid % 32; d < D; d += 32) {
        const float e = E[r * D + d], dv = bs[r] * e;
        db = fmaf(e, u[r * D + d], db);
        vd = fmaf(bf16f(a.v[size_t(c.row0 + r) * a.v_stride + h * D + d]), dv, vd);
        a.dv[(size_t(c.row0 + r) * a.H_v + h) * D + d] =
            __bfloat16_as_ushort(__float2bfloat16_rn(dv));
      }
      for (int off = 16; off > 0; off >>= 1) {
        db += __shfl_xor_sync(0xffffffffu, db, off);
        vd += __shfl_xor_sync(0xffffffffu, vd, off);
      }
      if (tid % 32 == 0) {
        a.dbeta[size_t(c.row0 + r) * a.H_v + h] = db;
        dG[r] = -vd;
      }
    }
    float hh = 0.f;
    for (int x = tid; x < D * D; x += 256) hh = fmaf(H1[x], dH[x], hh);
    for (int off = 16; off > 0; off >>= 1) hh += __shfl_xor_sync(0xffffffffu, hh, off);
    if (tid % 32 == 0) red[tid / 32] = hh;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int r = ty + 16 * m;
      float x = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x = fmaf(Qf(r, tx + 16 * n), dq[m][n], x);
        dqs[m][n] += dq[m][n];
      }
      for (int off = 8; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (tx == 0 && r < c.rows) dG[r] += x;
    }
    __syncthreads();
    if (tid == 0) {
      float run = 0.f;
      for (int w = 0; w < 8; ++w) run += red[w];
      for (int r = c.rows - 1; r >= 0; --r) {
        run += dG[r];
        a.dg[size_t(c.row0 + r) * a.H_v + h] = run;
      }
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = ty + 16 * m;
      if (r >= c.rows) continue;
      const size_t at = (size_t(c.row0 + r) * a.H_k + hk) * D + tx + 16 * n;
      a.dq[at] = __bfloat16_as_ushort(__float2bfloat16_rn(dqs[m][n]));
      a.dk[at] = __bfloat16_as_ushort(__float2bfloat16_rn(dks[m][n]));
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Lays the workspace out behind `base` (which may be null) and returns its size.
size_t layout(BwdArgs* a, char* base, int total_tokens, int num_seqs, int H_v, int D) {
  const size_t mc = size_t(total_tokens / kBC) + size_t(num_seqs);
  const size_t units = mc * H_v;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += up256(bytes);
    return p;
  };
  a->max_chunks = int(mc);
  a->cu_chunks = reinterpret_cast<int32_t*>(take((size_t(num_seqs) + 1) * 4));
  a->chunk_seq = reinterpret_cast<int32_t*>(take(mc * 4));
  a->G = reinterpret_cast<float2*>(take(units * kBC * 8));
  a->S = reinterpret_cast<float*>(take(units * kBC * kBC * 4));
  a->M = reinterpret_cast<float*>(take(units * kBC * kBC * 4));
  a->u = reinterpret_cast<float*>(take(units * kBC * D * 4));
  a->E = reinterpret_cast<float*>(take(units * kBC * D * 4));
  a->H = reinterpret_cast<float*>(take((mc + num_seqs) * size_t(H_v) * D * D * 4));
  a->dH = reinterpret_cast<float*>(take(units * D * D * 4));
  return at;
}

template <int D>
cudaError_t run(const BwdArgs& a, cudaStream_t s) {
  const int prep_smem = (2 * kBC * (D + 1) + 2 * kBC * 65) * 4;
  const int scan_smem = (D * kScanCols + 2 * kBC * D + 2 * kBC * kScanCols + 2 * kBC * kBC) * 4;
  const int grads_smem = (64 * 33 + D * 33 + 2 * 64 * 65) * 4;
  cudaError_t e;
  const auto kMax = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(bwd_prep_kernel<D>, kMax, prep_smem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(bwd_scan_kernel<D>, kMax, scan_smem)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(bwd_grads_kernel<D>, kMax, grads_smem)) != cudaSuccess) return e;
  bwd_prep_kernel<D><<<dim3(a.max_chunks, a.H_v), 256, prep_smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  bwd_scan_kernel<D><<<dim3(a.num_seqs * a.H_v * (D / kScanCols), 2), 128, scan_smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  bwd_grads_kernel<D><<<dim3(a.max_chunks, a.H_k), 256, grads_smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t backward_workspace_bytes(int total_tokens, int num_seqs, int H_v, int D) {
  BwdArgs a;
  return layout(&a, nullptr, total_tokens, num_seqs, H_v, D);
}

cudaError_t launch_backward(const BackwardCall& c, cudaStream_t s) {
  BwdArgs a;
  layout(&a, static_cast<char*>(c.workspace), c.total_tokens, c.num_seqs, c.H_v, c.D);
  a.q = c.q, a.k = c.k, a.v = c.v, a.dout = c.dout;
  a.g = c.g, a.beta = c.beta;
  a.qk_stride = c.qk_stride, a.v_stride = c.v_stride, a.gb_stride = c.gb_stride;
  a.cu = c.cu_seqlens;
  a.num_seqs = c.num_seqs, a.total_tokens = c.total_tokens, a.H_k = c.H_k, a.H_v = c.H_v;
  a.h0 = c.h0, a.dhT = c.dhT;
  a.dq = c.dq, a.dk = c.dk, a.dv = c.dv, a.dg = c.dg, a.dbeta = c.dbeta, a.dh0 = c.dh0;
  a.scale = c.scale;
  TablesCall t = {};
  t.cu_in = c.cu_seqlens;
  t.num_seqs = c.num_seqs;
  t.row_capacity = c.total_tokens;
  t.cu_chunks = a.cu_chunks;
  t.chunk_seq = a.chunk_seq;
  t.chunk_capacity = a.max_chunks;
  cudaError_t e = launch_tables(t, s);
  if (e != cudaSuccess) return e;
  return c.D == 128 ? run<128>(a, s) : run<64>(a, s);
}

}  // namespace gdn

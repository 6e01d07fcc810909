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
//   dg_r = e^{G_C} <H, dH'> + sum_{t >= r} a_t + sum_{s < r} b_s + sum_{s < r <= t} W_ts  with
//   a_t = e^{G_t} (scale q_t . H dO_t - k_t . H beta E_t),  b_s = e^{G_C-G_s} k_s . dH' beta u_s,
//   W_ts = P_ts q_t . k_s + N_ts k_t . k_s:
// what row r's gate decays is all that lies before it, H and the rows s < r, and it decays it for
// all behind, dH' and the rows t >= r.  Every term has the gate's own decay in it, so a strong one
// costs dg no accuracy.  (As sum_{s >= r} (q_s . dq_s - v_s . dv_s) + <H', dH'>, which needs no W, dg
// is the small rest of large terms where decays are strong.)
//
// Gates reach the exponentials as differences of 64-bit cumulative sums (in base
// 2: exp2f is the shorter function), kept as two floats: a strong decay early in
// the chunk costs later rows nothing.
//
// Arithmetic.  dg, dbeta and dh0 are f32, so everything they depend on is kept
// to f32 accuracy; a single bf16 or f16 operand would cost three digits.  Every
// product runs on the tensor cores in f16 with f32 sums, each f32 operand as
// two f16 limbs (hi = f16(x s), lo = f16(x s - hi)) under a power-of-two scale s
// that puts the largest value of what shares it in [2^14, 2^15): 22 bits, or
// 2^-40 of the largest value, whichever is coarser.  Only what enters the same sums
// shares one: a row, a column, a state (a head's entry state or its gradient).  A row
// of bf16 inputs is exact in one limb under its scale.  exact x f32 takes 2 MMAs, f32 x f32 takes 3
// (lo x lo is below the f32 rounding).  Where no scale would do (S, M, P and N, whose elements
// decays set apart along rows and columns, and what S is multiplied with) the limbs are bf16: three
// of them, f32's own 24 bits, six MMAs with another such operand; two for P and N, which reach only
// dq and dk, rounded to bf16 themselves (2^-17 of a row's terms against 2^-9 of the row).
//
// The scans and the gradients run on tcgen05; the first kernel, whose products are
// small and triangular, on warp-level MMAs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int kBC = 64;              // rows of a chunk
constexpr int kBlk = 8192;           // bytes of a [64 rows][64 columns] 16-bit tile block
constexpr float kGateFloor = -1e4f;  // e^x is 0 in f32 far above it; keeps sums finite

// Where everything is in the workspace.  16-bit tiles are blocks of 64 columns,
// rows of 128 bytes, 16-byte pieces XOR-swizzled by row (sw128_offset): a copy
// brings them into shared memory as the matrix loads want them.
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
  int32_t* cu_chunks;  // [num_seqs + 1]
  int32_t* chunk_seq;  // [max_chunks]
  int max_chunks;
  int sms;             // SMs of the device
  uint8_t* KQ;         // [chunk][H_k] f16 tiles of K, then of Q, a scale per row
  uint8_t* O;          // [chunk][H_v] f16 tile of dO, a scale per row
  uint8_t* GO;         // [chunk][H_v] scale e^G dO, high and low tile, a scale per column
  uint8_t* S;          // [chunk][H_v] -S, three limbs
  float* Y0;           // [chunk][H_v][64][D] scale (Q K^T * D)^T dO
  float* fac;          // [chunk][H_v][kFac]
  float* ff;           // [chunk][H_v][kFwdFac] factors for the forward scan
  float* fb;           // [chunk][H_v][kBackFac] ... and for the backward one
  float2* G;           // [chunk][H_v][64] cumulative gates / ln 2, high and low part
  float* u;            // [chunk][H_v][D / 32][64][32]
  float* E;            // [chunk][H_v][D / 32][64][32]
  float* H;            // [chunk][H_v][D / 16][D][16] entry states
  float* dH;           // [chunk][H_v][D / 16][D][16] gradient of the exit state
  float* Hmax;         // [chunk][H_v][2][8] largest |H| and |dH| of each scan warp's part
};

// Per-unit factors for the gradients: of each row e^G, e^{G_C - G}, beta, e^{G_b - G} with b
// the last row of its 16-row block, and scale times the inverse scale of dO's row; e^{G_C}.
enum { kFeG = 0, kFeT = kBC, kFbeta = 2 * kBC, kFend = 3 * kBC, kFo = 4 * kBC, kFeC = 5 * kBC };
constexpr int kFac = 5 * kBC + 4;

// For a scan: what scales the rows of its three products (kSx: the state times K^T; kSin:
// X or Y into the product with S; kSw: u or E into the product with K) and e^{G_C}.  The
// backward scan also has the inverse scales of GO's columns.
enum { kSx = 0, kSin = kBC, kSw = 2 * kBC, kSeC = 3 * kBC, kScol = kSeC + 4 };
constexpr int kFwdFac = kScol, kBackFac = kScol + 128;

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(uint32_t(x) << 16); }
__device__ __forceinline__ float expdiff(float2 a, float2 b) {
  return exp2f((a.x - b.x) + (a.y - b.y));
}
// The decay e^{G_r - G_s} for s <= r as two factors, e^{G_r - G_b} e^{G_b - G_s} with b the last row
// of column s's 16-row block, takes one exponential a row and block.  The first factor is above
// 1 where r comes before b, and the second one where gates rise from s to b, both far out of f32's
// range for gates that are steep enough: then each pair of rows takes an exponential of its own.
__device__ __forceinline__ bool steep(float2 Gr, float2 Gb) {
  const float x = Gr.x - Gb.x;
  return x > 60.f || x < -100.f;
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

// The same without the map, for up to 32 sequences, by a whole warp; *chunks gets the
// number of chunks.  `write`: this warp writes the map (chunk 0's warp the offsets), which
// holds what gdn_state_tables would write there.
constexpr int kFewSeqs = 32;
__device__ __forceinline__ ChunkRows map_chunk(const BwdArgs& a, int i, bool write, int* chunks) {
  const int lane = threadIdx.x & 31, n = a.num_seqs;
  int lo = 0, hi = 0;
  if (lane < n) lo = a.cu[lane], hi = a.cu[lane + 1];
  const int own = min(int((unsigned(max(hi - lo, 0)) + kBC - 1) / kBC), a.max_chunks + 1);
  int end = own;  // (32 times max_chunks stays below 2^31)
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += x;
  }
  const int first = end - own;
  *chunks = min(__shfl_sync(0xffffffffu, end, 31), a.max_chunks);
  ChunkRows c;
  c.seq = 31 - __clz(__ballot_sync(0xffffffffu, lane < n && first <= i));
  lo = max(__shfl_sync(0xffffffffu, lo, c.seq), 0);
  hi = min(__shfl_sync(0xffffffffu, hi, c.seq), a.total_tokens);
  c.row0 = lo + kBC * (i - __shfl_sync(0xffffffffu, first, c.seq));
  c.rows = max(0, min(kBC, hi - c.row0));
  if (write) {
    if (i == 0 && lane < n) a.cu_chunks[lane] = min(first, a.max_chunks);
    if (i == 0 && lane == 0) a.cu_chunks[n] = *chunks;
    if (i < *chunks && lane == 0) a.chunk_seq[i] = c.seq;
  }
  return c;
}

// ---------------------------------------------------------------------------
// Limbs, fragments, MMAs
// ---------------------------------------------------------------------------

// Power-of-two scale that brings `largest` (>= 0) into [2^14, 2^15), and its
// inverse.  Zero and what is below 2^-111 take the largest scale; infinity and
// NaN stay what they are through the split.
__device__ __forceinline__ float pow2_scale(float largest, float* inverse) {
  const uint32_t e = max(__float_as_uint(largest) >> 23, 16u);
  *inverse = __uint_as_float((e - 14u) << 23);
  return __uint_as_float((268u - e) << 23);
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// a and b as two limbs: hi = f16(x), lo = f16(x - hi).
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16(a, b);
  float x, y;  // x - hi with hi read as f16 (exact: it is below half a step of hi)
  asm("{\n\t.reg .b16 l, h, m;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "mov.b16 m, 0xBC00;\n\t"
      "fma.rn.f32.f16 %0, l, m, %3;\n\t"
      "fma.rn.f32.f16 %1, h, m, %4;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(hi), "f"(a), "f"(b));
  lo = pack_f16(x, y);
}

// a and b as N bf16 limbs, 8 bits each of any f32: no scale is needed.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int N>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&limb)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    limb[i] = pack_bf16(a, b);
    a -= __uint_as_float(limb[i] << 16), b -= __uint_as_float(limb[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void mma16_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                           uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += A B with a rounded sum: the MMA's own accumulation truncates, and over the
// steps of a long product the losses have one sign and add up.
__device__ __forceinline__ void add_mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  float p[4] = {};
  mma16_bf16(p, a, b0, b1);
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += p[e];
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Lane address of a 16 x 16 piece at (row, col) of a swizzled tile.  order_rc:
// the four 8 x 8 matrices run (0,0), (0,8), (8,0), (8,8) -- B fragments of two
// n-tiles from rows n, columns k (plain) -- else (0,0), (8,0), (0,8), (8,8):
// A fragments from rows m, columns k (plain), and B fragments of two n-tiles
// from rows k, columns n (transposed).  An A fragment from rows k, columns m
// (transposed) takes order_rc.
template <bool order_rc>
__device__ __forceinline__ uint32_t piece(uint32_t tile, int row, int col) {
  const int lane = threadIdx.x & 31, m = lane >> 3;
  const int r = row + (lane & 7) + (order_rc ? (m >> 1) * 8 : (m & 1) * 8);
  const int c = col + (order_rc ? (m & 1) * 8 : (m >> 1) * 8);
  return tile + (c >> 6) * kBlk + sw128_offset(r, (c & 63) * 2);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on = true) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// `bytes` (a multiple of 16 x threads) from global to shared memory.
template <int THREADS>
__device__ __forceinline__ void cp_async_block(uint32_t dst, const uint8_t* src, int bytes) {
  for (int x = threadIdx.x * 16; x < bytes; x += THREADS * 16) cp_async16(dst + x, src + x);
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
// The larger, NaN if either is (so that a NaN reaches the outputs).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------------------
// Prep: per (chunk, value head), what neither scan's state enters: the f16
// tiles of K, Q, dO and e^G dO, the gate factors, Y0 = scale M^T dO and S.
//
// A chunk's decays span any range, and what they make small can be all there is: where only
// the last row has an output gradient, E_s is e^{G_63 - G_s} times something of size 1.  So S
// and M, whose elements they set apart along rows and columns, have three bf16 limbs each,
// which need no scale, and so has what S is multiplied with.
//
// K K^T and Q K^T are one pass of MMAs each (exact operands).  With L_b the
// diagonal 16 x 16 blocks of B diag(beta), S by block rows:
//   S_bj = (I + L_b)^-1 (B_bj - sum over j <= c < b of B_bc (diag(beta) S)_cj).
// The four inverses are solved side by side in f32 on the CUDA cores (a thread a
// column); the block products are TF32 MMAs in two limbs each (22 bits).  Bound
// by latency and the writes; two CTAs an SM hide some of it (three spill).  160 us at 4576
// rows, 16 key and 48 value heads, d = 128: 0.41 GB written.
// ---------------------------------------------------------------------------

// 64 x D bf16 rows (row stride in elements) and the tiles that are made of them.
template <int D>
struct TileIn {
  uint4 x[D / 32];
  __device__ __forceinline__ void fetch(const uint16_t* src, size_t stride, int rows) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int p = threadIdx.x + 256 * i, r = p / (D / 8), c = p % (D / 8);
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) x[i] = *reinterpret_cast<const uint4*>(src + size_t(r) * stride + 8 * c);
    }
  }
  // As f16, each row times a power of two of its own, to global memory (NULL: not); the inverse
  // scales times f to inv[64].
  __device__ __forceinline__ void store(uint8_t* out, float f, float* inv) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int p = threadIdx.x + 256 * i, r = p / (D / 8), c = 8 * (p % (D / 8));
      uint32_t m = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                            __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
#pragma unroll
      for (int off = 1; off < D / 8; off <<= 1)  // the row's lanes
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
      float is;
      const float s = pow2_scale(__uint_as_float(max(m >> 16, m & 0xffffu) << 16), &is);
      if (c == 0) inv[r] = is * f;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = pack_f16(__uint_as_float(w[j] << 16) * s,
                        __uint_as_float(w[j] & 0xffff0000u) * s);
      const uint32_t at = (c >> 6) * kBlk + sw128_offset(r, (c & 63) * 2);
      if (out != nullptr) *reinterpret_cast<uint4*>(out + at) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
  // as it is, to shared memory
  __device__ __forceinline__ void store_raw(uint32_t tile) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int p = threadIdx.x + 256 * i, r = p / (D / 8), c = 8 * (p % (D / 8));
      st_shared_v4(tile + (c >> 6) * kBlk + sw128_offset(r, (c & 63) * 2), x[i].x, x[i].y, x[i].z,
                   x[i].w);
    }
  }
  // The largest finite |f[row] x| of each column into most[D], words that were zero.  (A NaN or
  // an infinity reaches its own column's results whatever its scale.)
  __device__ __forceinline__ void largest_of_columns(const float* f, uint32_t* most) const {
    uint32_t m[8] = {};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float fr = f[(threadIdx.x + 256 * i) / (D / 8)];
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = __float_as_uint(__uint_as_float(w[j] << 16) * fr) & 0x7fffffffu;
        const uint32_t b = __float_as_uint(__uint_as_float(w[j] & 0xffff0000u) * fr) & 0x7fffffffu;
        m[2 * j] = max(m[2 * j], a < 0x7f800000u ? a : 0u);
        m[2 * j + 1] = max(m[2 * j + 1], b < 0x7f800000u ? b : 0u);
      }
    }
    // the warp's rows: lanes D / 8 apart have the same columns
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int off = D / 8; off < 32; off <<= 1)
        m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], off));
      if ((threadIdx.x & 31) < D / 8) atomicMax(&most[8 * (threadIdx.x % (D / 8)) + j], m[j]);
    }
  }
  // f[row] x as two limb tiles, a scale per column.
  __device__ __forceinline__ void store_limbs(const float* f, const uint32_t* most,
                                              uint8_t* out) const {
    const int c = 8 * (threadIdx.x % (D / 8));
    float s[8], inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = pow2_scale(__uint_as_float(most[c + j]), &inv);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int r = (threadIdx.x + 256 * i) / (D / 8);
      const float fr = f[r];
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t h[4], l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        split_f16(__uint_as_float(w[j] << 16) * fr * s[2 * j],
                  __uint_as_float(w[j] & 0xffff0000u) * fr * s[2 * j + 1], h[j], l[j]);
      const uint32_t at = (c >> 6) * kBlk + sw128_offset(r, (c & 63) * 2);
      *reinterpret_cast<uint4*>(out + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(out + D / 64 * kBlk + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
  }
};

constexpr int kBT = 68;  // row length of the f32 squares (16-byte rows, 4 banks apart)

template <int D>
struct PrepSmem {
  static constexpr int kTile = D / 64 * kBlk;
  static constexpr int K = 0, Q = kTile;       // bf16 tiles; later dO; then from 0 on S's limbs
  static constexpr int M = 2 * kBlk;           // later, over Q: the three limbs of M
  static constexpr int B = 5 * kBlk;
  static constexpr int S = B + kBC * kBT * 4;
  static constexpr int T = S + kBC * kBT * 4;  // [4][16][20] the diagonal blocks' inverses
  static constexpr int kBytes = T + 4 * 16 * 20 * 4;
};

// x as two TF32 limbs: the upper 19 bits of x rounded (half away from zero), and the
// rest, of which the MMA reads the upper 19 bits.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma8_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// acc (16 x 16, two tiles) += A (16 x 16, row length la) diag(f) B (16 x 16, row length kBT),
// with `negate` minus it; f may be NULL (ones).  The low limbs' products have sums of
// their own: two short chains instead of a long one.
__device__ __forceinline__ void block_product(float (&acc)[2][4], const float* A, int la,
                                              const float* f, const float* Bm, bool negate) {
  const int lane = threadIdx.x & 31, g8 = lane >> 2, t = lane & 3;
  float low[2][4] = {};
#pragma unroll
  for (int k0 = 0; k0 < 16; k0 += 8) {
    float x[4] = {A[g8 * la + k0 + t], A[(g8 + 8) * la + k0 + t], A[g8 * la + k0 + t + 4],
                  A[(g8 + 8) * la + k0 + t + 4]};
    if (f != nullptr) x[0] *= f[k0 + t], x[1] *= f[k0 + t], x[2] *= f[k0 + t + 4], x[3] *= f[k0 + t + 4];
    uint32_t ah[4], al[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_tf32(negate ? -x[e] : x[e], ah[e], al[e]);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t h0, l0, h1, l1;
      split_tf32(Bm[(k0 + t) * kBT + 8 * n + g8], h0, l0);
      split_tf32(Bm[(k0 + t + 4) * kBT + 8 * n + g8], h1, l1);
      mma8_tf32(low[n], al, h0, h1);
      mma8_tf32(acc[n], ah, h0, h1);
      mma8_tf32(low[n], ah, l0, l1);
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] += low[n][e];
}

// The gates of head h: 64-bit sums, two rows per lane of one warp, into shared memory
// (gs: largest scale e^G) and the unit's factors.
struct GateRows {
  float2 G[kBC];
  float beta[kBC], eG[kBC];  // eG: scale e^G / scale of Q
  float end[kBC];            // e^{G_b - G}, b the last row of the 16-row block
};
__device__ __forceinline__ void make_gates(const BwdArgs& a, const ChunkRows& c, size_t unit, int h,
                                           const float* invk, const float* invq, GateRows* s) {
  const int lane = threadIdx.x & 31;
  float *fac = a.fac + unit * kFac, *ff = a.ff + unit * kFwdFac, *fb = a.fb + unit * kBackFac;
  double x[2];
  float bt[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * lane + e;
    float gv = 0.f;
    bt[e] = 0.f;
    if (r < c.rows) {
      gv = a.g[size_t(c.row0 + r) * a.gb_stride + h];
      bt[e] = a.beta[size_t(c.row0 + r) * a.gb_stride + h];
    }
    x[e] = (gv < kGateFloor ? kGateFloor : gv) * 1.4426950408889634;
    s->beta[r] = bt[e];
  }
  x[1] += x[0];
  double run = x[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, run, off);
    if (lane >= off) run += y;
  }
  const double total = __shfl_sync(0xffffffffu, run, 31);
  x[0] += run - x[1];
  x[1] = run;
  const double end = __shfl_sync(0xffffffffu, x[1], lane | 7);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * lane + e;
    const float hi = float(x[e]);
    const float2 G = make_float2(hi, float(x[e] - double(hi)));
    s->G[r] = G;
    a.G[unit * kBC + r] = G;
    const float eG = exp2f(G.x + G.y), eT = exp2f(float(total - x[e]));
    s->eG[r] = a.scale * eG * invq[r];
    s->end[r] = exp2f(float(end - x[e]));
    fac[kFend + r] = s->end[r];
    fac[kFeG + r] = eG;
    fac[kFeT + r] = eT;
    fac[kFbeta + r] = bt[e];
    ff[kSx + r] = -eG * invk[r];
    ff[kSin + r] = bt[e];
    ff[kSw + r] = bt[e] * eT * invk[r];
    fb[kSx + r] = eT * invk[r];
    fb[kSin + r] = bt[e];
    fb[kSw + r] = -bt[e] * eG * invk[r];
  }
  if (lane == 0) fac[kFeC] = ff[kSeC] = fb[kSeC] = exp2f(float(total));
}

template <int D>
__global__ void __launch_bounds__(256, 2) bwd_prep_kernel(BwdArgs a, int heads) {
  using L = PrepSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ GateRows gates[2];  // by the head's parity
  __shared__ float invk[kBC], invq[kBC];  // inverse scales of K's and Q's rows
  __shared__ uint32_t cols[D];   // by head: columns of scale e^G dO / scale of Q's row
  const int i = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_wait();
  grid_launch_next();
  ChunkRows c;
  if (a.num_seqs <= kFewSeqs) {
    int chunks;
    c = map_chunk(a, i, blockIdx.y == 0 && warp == 0, &chunks);
    if (i >= chunks) return;
  } else {
    if (i >= a.cu_chunks[a.num_seqs]) return;
    c = chunk_rows(a, i);
  }
  const int vpg = a.H_v / a.H_k, h0 = blockIdx.y * heads, hk = h0 / vpg;
  const uint32_t base = smem_u32(smem);
  const size_t unit0 = size_t(i) * a.H_v;
  auto dout = [&](int h) { return a.dout + (size_t(c.row0) * a.H_v + h) * D; };
  TileIn<D> ot;
  {
    TileIn<D> kt, qt;
    kt.fetch(a.k + size_t(c.row0) * a.qk_stride + hk * D, a.qk_stride, c.rows);
    qt.fetch(a.q + size_t(c.row0) * a.qk_stride + hk * D, a.qk_stride, c.rows);
    ot.fetch(dout(h0), size_t(a.H_v) * D, c.rows);
    uint8_t* kq = h0 % vpg == 0 ? a.KQ + (size_t(i) * a.H_k + hk) * 2 * L::kTile : nullptr;
    kt.store_raw(base + L::K);
    qt.store_raw(base + L::Q);
    kt.store(kq, 1.f, invk);
    qt.store(kq != nullptr ? kq + L::kTile : nullptr, 1.f, invq);
  }
  __syncthreads();
  if (warp == 7) make_gates(a, c, unit0 + h0, h0, invk, invq, &gates[h0 & 1]);
  // K K^T and Q K^T, for all the heads: warp = 16 rows, every other 16-column block up
  // to the diagonal
  const int rb = warp >> 1, par = warp & 1, g8 = lane >> 2, t2 = 2 * (lane & 3);
  float kk_[4][4] = {}, qk[4][4] = {};
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    uint32_t ak[4], aq[4];
    ldsm4(ak, piece<false>(base + L::K, 16 * rb, 16 * kk));
    ldsm4(aq, piece<false>(base + L::Q, 16 * rb, 16 * kk));
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * j + par <= rb) {
        uint32_t bv[4];
        ldsm4(bv, piece<true>(base + L::K, 16 * (2 * j + par), 16 * kk));
        add_mma16(kk_[2 * j], ak, bv[0], bv[1]);
        add_mma16(kk_[2 * j + 1], ak, bv[2], bv[3]);
        add_mma16(qk[2 * j], aq, bv[0], bv[1]);
        add_mma16(qk[2 * j + 1], aq, bv[2], bv[3]);
      }
  }
  float* B = reinterpret_cast<float*>(smem + L::B);
  float* S = reinterpret_cast<float*>(smem + L::S);
  float* T = reinterpret_cast<float*>(smem + L::T);
  for (int h = h0; h < h0 + heads; ++h) {
    const size_t unit = unit0 + h;
    const GateRows& gr = gates[h & 1];
    const float* bs = gr.beta;
    if (tid >= 128 && tid < 128 + D) cols[tid - 128] = 0;
    if (tid == 0) tma_store_wait_read<0>();  // the last head's S has left
    __syncthreads();  // the last head's (or K and Q's) shared memory is free
    // B and M
    ot.largest_of_columns(gr.eG, cols);
    float m_[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int s0 = 32 * (j >> 1) + 16 * par + 8 * (j & 1) + t2;
      if (2 * (j >> 1) + par <= rb) {
        const float2 Gb = gr.G[s0 | 15];  // the decay in two factors, see steep()
        const float2 f = *reinterpret_cast<const float2*>(&gr.end[s0]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int r = 16 * rb + g8 + (e >> 1) * 8;
          const float2 Gr = gr.G[r];
          float d0, d1;
          if (steep(Gr, Gb)) {
            d0 = s0 <= r ? expdiff(Gr, gr.G[s0]) : 0.f;
            d1 = s0 + 1 <= r ? expdiff(Gr, gr.G[s0 + 1]) : 0.f;
          } else {
            const float d = expdiff(Gr, Gb);
            d0 = s0 <= r ? d * f.x : 0.f;
            d1 = s0 + 1 <= r ? d * f.y : 0.f;
          }
          *reinterpret_cast<float2*>(&B[r * kBT + s0]) =
              make_float2(s0 < r ? kk_[j][e] * d0 : 0.f, s0 + 1 < r ? kk_[j][e + 1] * d1 : 0.f);
          m_[j][e] = s0 <= r ? qk[j][e] * d0 : 0.f;
          m_[j][e + 1] = s0 + 1 <= r ? qk[j][e + 1] * d1 : 0.f;
        }
      }
    }
    __syncthreads();  // B, the largest values
    // M, dO and scale e^G dO as tiles
    {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (2 * (j >> 1) + par <= rb)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            uint32_t limb[3];
            split_bf16(m_[j][e], m_[j][e + 1], limb);
            const uint32_t at = sw128_offset(16 * rb + g8 + (e >> 1) * 8,
                                             (32 * (j >> 1) + 16 * par + 8 * (j & 1) + t2) * 2);
#pragma unroll
            for (int x = 0; x < 3; ++x)
              *reinterpret_cast<uint32_t*>(smem + L::M + x * kBlk + at) = limb[x];
          }
      ot.store_raw(base);
      ot.store(a.O + unit * L::kTile, a.scale, a.fac + unit * kFac + kFo);
      ot.store_limbs(gr.eG, cols, a.GO + unit * 2 * L::kTile);
      if (tid < D) {
        float inv;
        pow2_scale(__uint_as_float(cols[tid]), &inv);
        a.fb[unit * kBackFac + kScol + tid] = inv;
      }
    }
    __syncthreads();  // M and dO
    if (h + 1 < h0 + heads) ot.fetch(dout(h + 1), size_t(a.H_v) * D, c.rows);
    if (warp < 4) {
      // The inverses of I + L_b: thread = (block, column), forward substitution
      if (tid < kBC) {
        const int b = tid >> 4, j = tid & 15;
        float x[16], t[16];  // beta times the column, and the column
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float* row = B + (16 * b + r) * kBT + 16 * b;
          float y0 = r == j ? 1.f : 0.f, y1 = 0.f;
#pragma unroll
          for (int q = 0; q < r; q += 4) {
            const float4 w = *reinterpret_cast<const float4*>(row + q);
            y0 = fmaf(-w.x, x[q], y0);
            if (q + 1 < r) y1 = fmaf(-w.y, x[q + 1], y1);
            if (q + 2 < r) y0 = fmaf(-w.z, x[q + 2], y0);
            if (q + 3 < r) y1 = fmaf(-w.w, x[q + 3], y1);
          }
          t[r] = y0 + y1;
          x[r] = t[r] * bs[16 * b + r];  // L_b's columns carry beta
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) T[(b * 16 + r) * 20 + j] = t[r];
      }
      named_sync(1, 128);
      // (I + L_b)^-1 B_bj in B's place: warp = block row b and, for the short rows, some
      // of the long ones' blocks
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        // warp 0: (0,0) (3,0) (2,0); 1: (1,0) (1,1) (3,1); 2: (2,1) (2,2); 3: (3,2) (3,3)
        const int code = warp == 0 ? 0x20'30'00 >> (8 * m) : warp == 1 ? 0x31'11'10 >> (8 * m)
                         : warp == 2 ? 0xff'22'21 >> (8 * m) : 0xff'33'32 >> (8 * m);
        const int b = (code >> 4) & 15, j = code & 15;
        if (b > 3) break;
        float* at = B + 16 * b * kBT + 16 * j;
        float acc[2][4] = {};
        block_product(acc, T + b * 16 * 20, 20, nullptr, at, false);
        __syncwarp();
        float* s_at = S + 16 * b * kBT + 16 * j;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int o = (g8 + (e >> 1) * 8) * kBT + 8 * n + t2;
            const float2 v = make_float2(acc[n][e], acc[n][e + 1]);
            *reinterpret_cast<float2*>(&at[o]) = v;
            if (b == j) *reinterpret_cast<float2*>(&s_at[o]) = v;  // S's diagonal blocks
          }
      }
      named_sync(1, 128);
      // Block column j = warp of S, downwards: nothing of another column enters it
      const int j = warp;
      for (int b = j + 1; b < 4; ++b) {
        float acc[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[n][e] = B[(16 * b + g8 + (e >> 1) * 8) * kBT + 16 * j + 8 * n + t2 + (e & 1)];
        for (int cc = j; cc < b; ++cc)
          block_product(acc, B + 16 * b * kBT + 16 * cc, kBT, bs + 16 * cc,
                        S + 16 * cc * kBT + 16 * j, true);
        float* out = S + 16 * b * kBT + 16 * j;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            *reinterpret_cast<float2*>(&out[(g8 + (e >> 1) * 8) * kBT + 8 * n + t2]) =
                make_float2(acc[n][e], acc[n][e + 1]);
        __syncwarp();
      }
    } else {
      // Meanwhile Y0 = scale M^T dO: warp = 16 rows s; k-steps from the diagonal
      const int mt = warp & 3;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        float y[4][4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk >= mt) {
            uint32_t am[3][4];
#pragma unroll
            for (int x = 0; x < 3; ++x)
              ldsm4t(am[x], piece<true>(base + L::M + x * kBlk, 16 * kk, 16 * mt));
#pragma unroll
            for (int np = 0; np < 2; ++np) {
              uint32_t bv[4];
              ldsm4t(bv, piece<false>(base, 16 * kk, c0 + 16 * np));
              float p0[4] = {}, p1[4] = {};
#pragma unroll
              for (int x = 2; x >= 0; --x) {
                mma16_bf16(p0, am[x], bv[0], bv[1]);
                mma16_bf16(p1, am[x], bv[2], bv[3]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) y[2 * np][e] += p0[e], y[2 * np + 1][e] += p1[e];
            }
          }
        float* out = a.Y0 + (unit * kBC + 16 * mt + g8) * D + c0 + t2;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            *reinterpret_cast<float2*>(out + (e >> 1) * 8 * D + 8 * n) =
                make_float2(y[n][e] * a.scale, y[n][e + 1] * a.scale);
      }
      if (warp == 7 && h + 1 < h0 + heads)
        make_gates(a, c, unit + 1, h + 1, invk, invq, &gates[(h + 1) & 1]);
    }
    __syncthreads();
    // -S as limbs: warp = 16 rows, half of the columns; zeros above the diagonal blocks
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int r = 16 * rb + g8 + 8 * (m & 1), s = 32 * par + 8 * (m >> 1) + t2;
      float2 v = make_float2(0.f, 0.f);
      if (2 * par + (m >> 2) <= rb) v = *reinterpret_cast<const float2*>(&S[r * kBT + s]);
      uint32_t limb[3];
      split_bf16(-v.x, -v.y, limb);
#pragma unroll
      for (int x = 0; x < 3; ++x)
        *reinterpret_cast<uint32_t*>(smem + x * kBlk + sw128_offset(r, 2 * s)) = limb[x];
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store_s2g(a.S + unit * 3 * kBlk, smem, 3 * kBlk);
      tma_store_commit();
    }
  }
  if (tid == 0) tma_store_wait_all<0>();
}

// ---------------------------------------------------------------------------
// Scans: one CTA per (sequence, value head, direction), both directions in one launch
// (the backward one first): 286 us at 4576 rows, 48 heads, 4.0 us a chunk.
//
// H^T [dv][dk] is held by 8 state warps, thread (dv, half of d_k), 64 f32
// registers at D = 128.  Per chunk three products, M = 128 (dv), A from tensor
// memory (the limbs that the state warps write), B the chunk's tiles:
//   1. H^T K^T -> X (or Y), 2. (beta X)^T S^T -> u (or S: E), 3. (f u)^T K -> H'.
// The limbs of products 1 and 3 are f16, a row's under one scale per half (its thread's own
// maximum, with the factors of the rows in it), so no warp waits for another one's maximum: the
// halves go to accumulators of their own, summed when they are read.  Product 2, whose results
// decays set apart, has three bf16 limbs on both sides.  The backward scan also has
// (scale e^G dO)^T Q, from tiles made before, between products 1 and 2.
//   warps 0-7: state; warp 8: loads (bulk copies into buffers freed by the
//   products that read them); warp 9: one thread issues the MMAs after the state
//   warps' barrier.
// Low limbs are multiplied first: the f32 accumulator then rounds against small
// sums while it holds them.  D = 64 runs the same code with half of the rows idle.
//
// Bound by the chain, about 7800 cycles a chunk: 16 + 24 + 8 MMAs (about 58 cycles each) take
// 2900 of them, what the state warps do between them (limbs of the state 800, X and its limbs
// 900, u or E and its limbs 900, their way out 600, the new state 450) and the hand-overs, three
// each way, the rest.  The state's way out (1400) runs beside the first two products.
// ---------------------------------------------------------------------------

constexpr int kScanThreads = 384;
// Registers after re-allocation: 256 x 232 + 128 x 40 is the launch's 384 x 168.
constexpr uint32_t kRegsScan = 232, kRegsFeed = 40;
constexpr int kScanSync = 288;  // the state warps and the issuer

__device__ uint32_t g_err_backward;

// Instruction descriptor as make_idesc_bf16, with f16 operands.
__host__ __device__ constexpr uint32_t make_idesc_f16(int M, int N, int a_mn, int b_mn) {
  return make_idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

enum { kTX0 = 0, kTX1 = 64, kTH0 = 128, kTH1 = 256, kTA = 384 };  // tensor memory columns
enum { bKF = 0, bKE = 2, bEF = 4, bQE, bYF, bYE, bSF, bSE, bX, bQ, bS, bH, bDrain, kBars };

template <int D, bool back>
struct ScanSmem {
  static constexpr int kTile = D / 64 * kBlk;
  static constexpr int K = 0;                      // two buffers
  static constexpr int S = 2 * kTile;              // -S, three limbs
  static constexpr int Y = S + 3 * kBlk;           // Y0 (f32) or V (bf16), [64][D]
  static constexpr int Q = Y + kBC * D * (back ? 4 : 2);
  static constexpr int GO = Q + (back ? kTile : 0);  // two limbs, M = 128 rows each
  // The state on its way out: its slices, 64 bytes apart from a multiple of all
  // banks, so that the two slices of a warp do not collide.  Every warp sends its own
  // part, two runs of kRun bytes, and then, from the first one's place, its part of u
  // or E (4 KB; D = 64 has a place of its own for that).
  static constexpr int kStep = D * 64 + 64, kRun = D / 2 * 64;
  static constexpr int St = GO + (back ? 2 * kTile + (D == 64 ? kBlk : 0) : 0);
  static constexpr int U = St + D / 16 * kStep;
  static constexpr int kFactors = back ? kBackFac : kFwdFac;
  static constexpr int Fac = U + (D == 64 ? 8 * 4096 : 0);  // two buffers
  static constexpr int Inv = Fac + 2 * kFactors * 4;   // [2][2][128] inverse row scales
  static constexpr int Bars = Inv + 4 * 128 * 4;
  static constexpr int kUsed = Bars + kBars * 8 + 16 + 1024;  // 1024: alignment of the base
  // More than half of an SM's: all of its tensor memory goes to one CTA.
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

// N floats times s as f16 limbs: hi to TMEM columns `hi`, lo to `lo` (N / 2 each).
template <int N>
__device__ __forceinline__ void limbs_to_tmem(const float (&x)[N], float s, uint32_t hi,
                                              uint32_t lo) {
  uint32_t h[N / 2], l[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 y = mul2(make_float2(x[2 * i], x[2 * i + 1]), both(s));
    split_f16(y.x, y.y, h[i], l[i]);
  }
  if constexpr (N == 64) {
    tmem_st32u(hi, h);
    tmem_st32u(lo, l);
  } else {
    tmem_st16u(hi, h);
    tmem_st16u(lo, l);
  }
  tmem_st_wait();
}

template <int N>
__device__ __forceinline__ float max_abs_of(const float (&x)[N]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int i = 0; i < N; i += 2) m0 = max_nan(m0, fabsf(x[i])), m1 = max_nan(m1, fabsf(x[i + 1]));
  return max_nan(m0, m1);
}

// The CTA `at` of one direction.
template <int D, bool back>
__device__ __forceinline__ void scan(const BwdArgs& a, int at) {
  using L = ScanSmem<D, back>;
  constexpr int NK = D / 2;   // d_k columns of a thread
  extern __shared__ uint8_t smem_raw[];
  __shared__ int seq_at;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::Bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* err = &g_err_backward;
  const int tid = threadIdx.x, warp = int(warp_id_sync()), lane = tid & 31;
  const int h = at % a.H_v, order = at / a.H_v, hk = h / (a.H_v / a.H_k);

  // Long sequences first: the order-th longest (for up to 64 of them).
  if (tid == 0) {
    seq_at = order;
    for (int b = 0; b < kBars; ++b) mbar_init(&bars[b], b == bYF && !back ? 32u : 1u);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  __syncthreads();
  grid_wait();
  grid_launch_next();
  if (a.num_seqs <= 64 && tid < a.num_seqs) {
    const int len = a.cu[tid + 1] - a.cu[tid];
    int rank = 0;
    for (int j = 0; j < a.num_seqs; ++j) {
      const int other = a.cu[j + 1] - a.cu[j];
      rank += other > len || (other == len && j < tid);
    }
    if (rank == order) seq_at = tid;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int b = seq_at;
  const int c0 = a.cu_chunks[b], n = a.cu_chunks[b + 1] - c0;
  auto chunk_of = [&](int t) { return c0 + (back ? n - 1 - t : t); };

  if (warp < 8) {
    setmaxnreg_inc<kRegsScan>();
    const int hh = warp >> 2, dv = 32 * (warp & 3) + lane;
    const bool on = D == 128 || dv < D;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);  // this warp's TMEM lanes
    float* inv_h = reinterpret_cast<float*>(smem + L::Inv);        // [2][128]
    float* inv_w = inv_h + 256;                                    // [2][128]
    const size_t head = (size_t(b) * a.H_v + h) * D * D;
    float st[NK];
    {
      const float* init = back ? a.dhT : a.h0;
#pragma unroll
      for (int i = 0; i < NK; ++i)
        st[i] = init != nullptr && on ? init[head + size_t(NK * hh + i) * D + dv] : 0.f;
    }
    // The warp's part of a state: its lanes' rows of two slices, d_k from NK hh.
    const int slice = 2 * (warp & 3);
    uint8_t* run = smem + L::St + slice * L::kStep + hh * L::kRun;
    float* out_st = reinterpret_cast<float*>(run + (lane >> 4) * L::kStep) + (lane & 15);
    // In two halves of the rows d_k, while products 1 and 2 run.
    auto send_state = [&](float* to, int half) {
      if (half == 0) {
        if (lane == 0) tma_store_wait_read<0>();  // what the warp sent last
        __syncwarp();
      }
      if (on) {
#pragma unroll
        for (int x = 0; x < NK / 2; ++x) out_st[(half * NK / 2 + x) * 16] = st[half * NK / 2 + x];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          float* p = to + slice * D * 16 + (hh * NK + half * NK / 2) * 16;
          const uint8_t* from = run + half * L::kRun / 2;
          bulk_store_s2g(p, from, L::kRun / 2);
          bulk_store_s2g(p + D * 16, from + L::kStep, L::kRun / 2);
          tma_store_commit();
        }
      }
    };
    bool ok = true;
    int t = 0;
    for (; t < n; ++t) {
      const int i = chunk_of(t);
      const size_t unit = size_t(i) * a.H_v + h;
      const float* fac = reinterpret_cast<const float*>(smem + L::Fac) + (t & 1) * L::kFactors;
      // 1. the state's limbs
      const float most = max_abs_of(st);
      {
        float inv;
        const float s = pow2_scale(most, &inv);
        inv_h[128 * hh + dv] = inv;
        limbs_to_tmem(st, s, tl + kTA + NK / 2 * hh, tl + kTA + 64 + NK / 2 * hh);
      }
      tc_fence_before();
      if (!named_all(1, kScanSync, ok)) break;
      {
        send_state((back ? a.dH : a.H) + unit * D * D, 0);
        const float wm = warp_max(on ? most : 0.f);
        if (lane == 0) a.Hmax[(unit * 2 + back) * 8 + warp] = wm;
      }
      // 2. X = V - e^G K H, or Y = Y0 + e^{G_C - G} K dH': rows 32 hh ..
      ok = mbar_wait(&bars[bKF + (t & 1)], (t >> 1) & 1, abort_flag, err, 1u) && ok;
      ok = mbar_wait(&bars[bYF], t & 1, abort_flag, err, 1u) && ok;
      ok = mbar_wait(&bars[bX], t & 1, abort_flag, err, 2u) && ok;
      tc_fence_after();
      float x[32];
      {
        float y0[32], y1[32];
        tmem_ld32(tl + kTX0 + 32 * hh, y0);
        tmem_ld32(tl + kTX1 + 32 * hh, y1);
        tmem_ld_wait();
        const float i0 = inv_h[dv], i1 = inv_h[128 + dv];
        const float* fr = fac + kSx + 32 * hh;
#pragma unroll
        for (int r = 0; r < 32; r += 2) {
          float2 f = *reinterpret_cast<const float2*>(fr + r), v = make_float2(0.f, 0.f);
          const int y = (32 * hh + r) * D + dv;
          if (back && on)
            v = make_float2(reinterpret_cast<const float*>(smem + L::Y)[y],
                            reinterpret_cast<const float*>(smem + L::Y)[y + D]);
          if (!back && on)
            v = make_float2(bf16f(reinterpret_cast<const uint16_t*>(smem + L::Y)[y]),
                            bf16f(reinterpret_cast<const uint16_t*>(smem + L::Y)[y + D]));
          const float2 kh = fma2(make_float2(y0[r], y0[r + 1]), both(i0),
                                 mul2(make_float2(y1[r], y1[r + 1]), both(i1)));
          const float2 d = fma2(f, kh, v);
          x[r] = d.x, x[r + 1] = d.y;
        }
      }
      {  // into the product with S, whose rows decays set apart: bf16 limbs
        uint32_t z[3][16];
#pragma unroll
        for (int r = 0; r < 32; r += 2) {
          const float2 d = mul2(make_float2(x[r], x[r + 1]),
                                *reinterpret_cast<const float2*>(fac + kSin + 32 * hh + r));
          uint32_t limb[3];
          split_bf16(d.x, d.y, limb);
#pragma unroll
          for (int l = 0; l < 3; ++l) z[l][r / 2] = limb[l];
        }
#pragma unroll
        for (int l = 0; l < 3; ++l) tmem_st16u(tl + kTA + 32 * l + 16 * hh, z[l]);
        tmem_st_wait();
      }
      tc_fence_before();
      if (!named_all(1, kScanSync, ok)) break;
      if (tid == 0) mbar_arrive(&bars[bYE]);
      send_state((back ? a.dH : a.H) + unit * D * D, 1);
      const float eC = fac[kSeC];
      if constexpr (back) {  // e^{G_C} dH' + (scale e^G dO)^T Q
        ok = mbar_wait(&bars[bQ], t & 1, abort_flag, err, 2u) && ok;
        tc_fence_after();
        const float f = fac[kScol + (D == 128 ? dv : dv & 63)];
#pragma unroll
        for (int p = 0; p < NK; p += 32) {
          float y[32];
          tmem_ld32(tl + kTH0 + NK * hh + p, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 d = fma2(both(eC), make_float2(st[p + e], st[p + e + 1]),
                                  mul2(make_float2(y[e], y[e + 1]), both(f)));
            st[p + e] = d.x, st[p + e + 1] = d.y;
          }
        }
      }
      // 3. u = X - (beta X) S^T, E = Y - (beta Y) S
      ok = mbar_wait(&bars[bS], t & 1, abort_flag, err, 2u) && ok;
      tc_fence_after();
      {
        float y0[32], y1[32];
        tmem_ld32(tl + kTX0 + 32 * hh, y0);
        tmem_ld32(tl + kTX1 + 32 * hh, y1);
        tmem_ld_wait();
#pragma unroll
        for (int r = 0; r < 32; r += 2) {
          const float2 d = add2(make_float2(x[r], x[r + 1]),
                                add2(make_float2(y0[r], y0[r + 1]), make_float2(y1[r], y1[r + 1])));
          x[r] = d.x, x[r + 1] = d.y;
        }
      }
      {
        float w[32], inv;
#pragma unroll
        for (int r = 0; r < 32; r += 2) {
          const float2 d = mul2(make_float2(x[r], x[r + 1]),
                                *reinterpret_cast<const float2*>(fac + kSw + 32 * hh + r));
          w[r] = d.x, w[r + 1] = d.y;
        }
        const float s = pow2_scale(max_abs_of(w), &inv);
        inv_w[128 * hh + dv] = inv;
        limbs_to_tmem(w, s, tl + kTA + 64 + 16 * hh, tl + kTA + 96 + 16 * hh);
      }
      tc_fence_before();
      if (!named_all(1, kScanSync, ok)) break;
      // 4. u or E out, while the product runs; the next state
      if (lane == 0) tma_store_wait_read<0>();
      __syncwarp();
      if (on) {
        uint8_t* place = D == 128 ? run : smem + L::U + warp * 4096;
        float* out = reinterpret_cast<float*>(place) + lane;
#pragma unroll
        for (int r = 0; r < 32; ++r) out[r * 32] = x[r];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          bulk_store_s2g((back ? a.E : a.u) + unit * kBC * D + (warp & 3) * kBC * 32 + hh * 32 * 32,
                         place, 4096);
          tma_store_commit();
        }
      }
      const float i0 = inv_w[dv], i1 = inv_w[128 + dv];
      ok = mbar_wait(&bars[bH], t & 1, abort_flag, err, 2u) && ok;
      tc_fence_after();
#pragma unroll
      for (int p = 0; p < NK; p += 32) {
        float y0[32], y1[32];
        tmem_ld32(tl + kTH0 + NK * hh + p, y0);
        tmem_ld32(tl + kTH1 + NK * hh + p, y1);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 d = make_float2(st[p + e], st[p + e + 1]);
          if (!back) d = mul2(d, both(eC));
          d = fma2(make_float2(y0[e], y0[e + 1]), both(i0),
                   fma2(make_float2(y1[e], y1[e + 1]), both(i1), d));
          st[p + e] = d.x, st[p + e + 1] = d.y;
        }
      }
    }
    if (lane == 0) tma_store_wait_all<0>();
    __syncwarp();
    if (back && on && a.dh0 != nullptr) {
#pragma unroll
      for (int x = 0; x < NK; ++x) a.dh0[head + size_t(NK * hh + x) * D + dv] = st[x];
    }
    tc_fence_before();
  } else {
   setmaxnreg_dec<kRegsFeed>();
   if (warp == 8) {
    // Loads, in the order in which the chain frees their buffers.
    const int seq_lo = max(a.cu[b], 0), seq_hi = min(a.cu[b + 1], a.total_tokens);
    bool ok = true;
    int tk = -1, te = -1, ty = -1, ts = -1;  // the last chunk of each kind that was issued
    for (int t = 0; t < n && ok; ++t) {
      const int i = chunk_of(t);
      const size_t unit = size_t(i) * a.H_v + h;
      const uint8_t* kq = a.KQ + (size_t(i) * a.H_k + hk) * 2 * L::kTile;
      if (t >= 2) ok = mbar_wait(&bars[bKE + (t & 1)], ((t >> 1) & 1) ^ 1, abort_flag, err, 4u);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[bKF + (t & 1)], L::kTile + L::kFactors * 4);
        bulk_load_g2s(smem + L::K + (t & 1) * L::kTile, kq, L::kTile, &bars[bKF + (t & 1)]);
        bulk_load_g2s(smem + L::Fac + (t & 1) * L::kFactors * 4,
                      (back ? a.fb : a.ff) + unit * L::kFactors, L::kFactors * 4,
                      &bars[bKF + (t & 1)]);
      }
      tk = t;
      if constexpr (back) {
        if (t >= 1) ok = mbar_wait(&bars[bQE], (t - 1) & 1, abort_flag, err, 4u);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[bEF], 3 * L::kTile);
          bulk_load_g2s(smem + L::Q, kq + L::kTile, L::kTile, &bars[bEF]);
          bulk_load_g2s(smem + L::GO, a.GO + unit * 2 * L::kTile, 2 * L::kTile, &bars[bEF]);
        }
        te = t;
      }
      if (t >= 1) ok = mbar_wait(&bars[bYE], (t - 1) & 1, abort_flag, err, 4u);
      if (!__all_sync(0xffffffffu, ok)) break;
      if constexpr (back) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars[bYF], kBC * D * 4);
          bulk_load_g2s(smem + L::Y, a.Y0 + unit * kBC * D, kBC * D * 4, &bars[bYF]);
        }
      } else {
        const int row0 = seq_lo + kBC * t, rows = max(0, min(kBC, seq_hi - row0));
        for (int y = lane; y < kBC * D / 8; y += 32) {
          const int r = y / (D / 8), p = y % (D / 8);
          const uint16_t* src = a.v + h * D + 8 * p;
          cp_async16(base + L::Y + y * 16, r < rows ? src + size_t(row0 + r) * a.v_stride : src,
                     r < rows);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&bars[bYF]))
                     : "memory");
      }
      ty = t;
      if (t >= 1) ok = mbar_wait(&bars[bSE], (t - 1) & 1, abort_flag, err, 4u);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[bSF], 3 * kBlk);
        bulk_load_g2s(smem + L::S, a.S + unit * 3 * kBlk, 3 * kBlk, &bars[bSF]);
      }
      ts = t;
    }
    // nothing may still be landing in shared memory at exit
    for (int t = tk - 1; t <= tk; ++t)
      if (t >= 0) mbar_wait(&bars[bKF + (t & 1)], (t >> 1) & 1, nullptr, err, 8u);
    if (te >= 0) mbar_wait(&bars[bEF], te & 1, nullptr, err, 8u);
    if (ty >= 0) mbar_wait(&bars[bYF], ty & 1, nullptr, err, 8u);
    if (ts >= 0) mbar_wait(&bars[bSF], ts & 1, nullptr, err, 8u);
    cp_async_wait<0>();
    __syncwarp();
   } else if (warp == 9) {
    const bool leader = lane == 0;
    const uint64_t kmaj = make_sdesc_sw128(0, 16, 1024);    // K-major operands
    const uint64_t mnmaj = make_sdesc_sw128(0, 8192, 1024);  // MN-major, 64-element blocks apart
    constexpr uint32_t id_x = make_idesc_f16(128, 64, 0, 0);
    constexpr uint32_t id_s = make_idesc_bf16(128, 64, 0, back ? 1 : 0);
    constexpr uint32_t id_h = make_idesc_f16(128, D, 0, 1);
    constexpr uint32_t id_q = make_idesc_f16(128, D, 1, 1);
    uint32_t b4 = base >> 4;
    for (int t = 0; t < n; ++t) {
      asm volatile("" : "+r"(b4));  // (descriptors are made where they are needed, not kept)
      const uint32_t k4 = b4 + ((L::K + (t & 1) * L::kTile) >> 4);
      bool ok = true;
      if (leader) ok = mbar_wait(&bars[bKF + (t & 1)], (t >> 1) & 1, abort_flag, err, 16u);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!named_all(1, kScanSync, ok)) break;
      if (leader) {
        tc_fence_after();
#pragma unroll
        for (int limb = 1; limb >= 0; --limb)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int half = kk / (D / 32);
            mma_bf16_ts(tmem + (half ? kTX1 : kTX0), tmem + kTA + 64 * limb + 8 * kk,
                        kmaj + (k4 + (kk >> 2) * (kBlk >> 4) + (kk & 3) * 2), id_x,
                        limb == 0 || kk % (D / 32) != 0);
          }
        mma_commit(&bars[bX]);
        if constexpr (back) {
          ok = mbar_wait(&bars[bEF], t & 1, abort_flag, err, 16u);
          if (ok) {
            tc_fence_after();
#pragma unroll
            for (int limb = 1; limb >= 0; --limb)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_bf16_ss(tmem + kTH0,
                            mnmaj + (b4 + ((L::GO + limb * L::kTile) >> 4) + 128 * kk),
                            mnmaj + (b4 + (L::Q >> 4) + 128 * kk), id_q,
                            limb == 0 || kk != 0);
          }
          mma_commit(&bars[bQ]);
          mma_commit(&bars[bQE]);
        }
        ok = mbar_wait(&bars[bSF], t & 1, abort_flag, err, 16u) && ok;
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!named_all(1, kScanSync, ok)) break;
      if (leader) {
        tc_fence_after();
        const uint32_t s4 = b4 + (L::S >> 4);
        // limb pairs from the smallest on, without those below 2^-24; the rows' halves apart
#pragma unroll
        for (int q = 0; q < 6; ++q)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int lx = q == 0 ? 2 : q == 2 || q == 3 ? 1 : 0, ls = q == 1 ? 2 : q == 2 || q == 4 ? 1 : 0;
            const uint32_t at = s4 + ls * (kBlk >> 4);
            mma_bf16_ts(tmem + (kk >> 1 ? kTX1 : kTX0), tmem + kTA + 32 * lx + 8 * kk,
                        back ? mnmaj + (at + 128 * kk) : kmaj + (at + 2 * kk), id_s,
                        q != 0 || (kk & 1) != 0);
          }
        mma_commit(&bars[bS]);
        mma_commit(&bars[bSE]);
      }
      __syncwarp();
      if (!named_all(1, kScanSync, true)) break;
      if (leader) {
        tc_fence_after();
#pragma unroll
        for (int limb = 1; limb >= 0; --limb)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(tmem + (kk >> 1 ? kTH1 : kTH0), tmem + kTA + 64 + 32 * limb + 8 * kk,
                        mnmaj + (k4 + 128 * kk), id_h, limb == 0 || (kk & 1) != 0);
        mma_commit(&bars[bH]);
        mma_commit(&bars[bKE + (t & 1)]);
      }
      __syncwarp();
    }
    if (leader) {  // every MMA this thread issued has completed
      mma_commit(&bars[bDrain]);
      mbar_wait(&bars[bDrain], 0, nullptr, err, 32u);
    }
    __syncwarp();
   }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
__global__ void __launch_bounds__(kScanThreads, 1) bwd_scan_kernel(BwdArgs a) {
  const int half = gridDim.x / 2;
  if (int(blockIdx.x) < half)
    scan<D, true>(a, blockIdx.x);
  else
    scan<D, false>(a, blockIdx.x - half);
}

cudaError_t take_err_backward(uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_err_backward, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_err_backward, &zero, sizeof(uint32_t));
}

// ---------------------------------------------------------------------------
// Grads: one CTA per (chunk, key head), the value heads of the group one after
// another, so that the shared dq and dk are summed in registers, in one order.  (A call
// of few chunks has a CTA per value head instead; the CTAs of a key head are a cluster
// and sum through each other's shared memory.)
//
// All products are transposed, M = 128 rows d_k (or, for P and N, the rows of dO
// above those of beta E), so that two of them share an MMA where they share an
// operand:
//   [Q; K] K^T, once
//   [P; N]       = [dO; beta E] (beta u)^T           K = d_v
//   [A1 | A2]    = H [dO; beta E]^T                  K = d_v, by halves, in turn with
//   A6           = dH' (beta u)^T                    K = d_v, by halves
//   A3           = P K,  A4 = P^T Q + N K + N^T K    K = 64
//   dq = scale e^G A1 + A3,  dk = A4 - e^G A2 + e^{G_C - G} A6.
// Row factors that differ within a product are applied to its result.
//   warps 0-7: rows u and E to tiles, the masks of P and N, the sums dq, dk and those of dg;
//   warps 8-11: states to limbs, in two slots, and <H, dH'>;
//   warp 12: one thread loads dO and issues the MMAs; warp 13: dg; warps 14, 15: Q and K.
// Between a head's products and sums the row warps stage the next head's rows, as soon as the
// products that read the last ones are done, so that the slots are free again early.
// 336 us at 4576 rows, 48 heads.  Bound by the latency of a head's steps, each of which waits for
// another group's (issue slots 36 % used, tensor pipe 15 %, barriers and loads the stalls).  The
// states' values come to the slots by bulk copies and become limbs in place: with loads through
// registers, two batches in flight, the call took 55 us more.
// ---------------------------------------------------------------------------

template <int D>
struct GradsSmem {
  static constexpr int kTile = D / 64 * kBlk;
  // Q and K as they are (bf16), for each 64 columns one over the other
  static constexpr int QK = 0, kQK = 2 * kBlk;
  // dO, beta E high and beta E low, likewise
  static constexpr int OE = D / 64 * kQK, kOE = 3 * kBlk;
  static constexpr int UH = OE + D / 64 * kOE, UL = UH + kTile;  // beta u, two limbs
  // Slots for 64 columns (d_v) of H and of dH', as they are (f32, slices of 16 columns), then
  // in the same place as limbs with 128 rows, high and low
  static constexpr int H = UL + kTile, kSlot = 4 * kBlk;
  // bf16 limbs of P and N
  static constexpr int PL = H + 2 * kSlot, NL = PL + kBlk, PH = NL + kBlk, NH = PH + kBlk;
  static constexpr int Fac = NH + kBlk;          // two buffers of the unit's factors
  static constexpr int G = Fac + 2 * kFac * 4;   // two buffers of the cumulative gates
  static constexpr int F = G + 2 * kBC * 8;      // floats from here
  static constexpr int kFloats = 4 * kBC + 12 * kBC + kBC + 40;
  static constexpr int Bars = F + kFloats * 4;
  static constexpr int kUsed = Bars + 16 * 8 + 16 + 1024;
  // More than half of an SM's: all of its tensor memory goes to one CTA.
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

constexpr int kGradsRows = 256, kGradsStates = 128, kGradsThreads = 512;
// Registers after re-allocation: 128 (2 x 176 + 112 + 48) is the launch's 512 x 128.
constexpr uint32_t kRegsRows = 176, kRegsStates = 112, kRegsIssue = 48;
enum { gO = 0, gQK, gU, gLand, gFull = gLand + 2, gFree = gFull + 2, gP = gFree + 2, gPN, gStates,
       gA34, gE, gDrain, kGradsBars };
enum { kTPN = 0, kTA1 = 64, kTA2 = 128, kTA3 = 192, kTA4 = 256, kTEL = 320, kTA6 = 384,
       kTQK = 448 };  // (kTEL: beta E's low limb in N)

// Sums over the warp's lanes of N values each: lane l gets that of value l / (32 / N).
template <int N>
__device__ __forceinline__ float sum_over_lanes(float (&x)[N]) {
  constexpr int step = 32 / N;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = N / 2; w >= 1; w >>= 1) {
    const bool up = lane & (step * w);
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float send = up ? x[k] : x[k + w];
      x[k] = (up ? x[k + w] : x[k]) + __shfl_xor_sync(0xffffffffu, send, step * w);
    }
  }
#pragma unroll
  for (int w = step / 2; w >= 1; w >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], w);
  return x[0];
}

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Quad q of 64 columns of a state (slice of 16 columns, d_k, quad): where its limbs are in the
// slot's tile.
template <int D>
__device__ __forceinline__ uint32_t quad_place(int q) {
  return sw128_offset((q >> 2) % D, (q / (4 * D) * 16 + (q & 3) * 4) * 2);
}

template <int D, bool split>
__global__ void __launch_bounds__(kGradsThreads, 1) bwd_grads_kernel(BwdArgs a) {
  using L = GradsSmem<D>;
  constexpr int J = D / 32;         // quads of a row per lane in the row pass
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::Bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kGradsBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* err = &g_err_backward;
  const int i = blockIdx.x, tid = threadIdx.x, warp = int(warp_id_sync()), lane = tid & 31;
  const int vpg = a.H_v / a.H_k, heads = split ? 1 : vpg;
  const int hk = split ? blockIdx.y / vpg : blockIdx.y, h0 = split ? blockIdx.y : hk * vpg;
  if (tid == 0) {
    for (int b = 0; b < kGradsBars; ++b)
      mbar_init(&bars[b], b == gQK ? 2 : b == gU || b == gP || b == gE ? kGradsRows / 32 : b == gFull || b == gFull + 1 ? kGradsStates / 32 : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  // Every CTA waits, those without a chunk too: this grid's end is the call's.
  grid_wait();
  if (i >= a.cu_chunks[a.num_seqs]) return;
  const ChunkRows c = chunk_rows(a, i);
  if (warp == 0) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  float* invU2 = reinterpret_cast<float*>(smem + L::F);  // [2][64], by the head's parity
  float* invE2 = invU2 + 2 * kBC;   // [2][64]
  // for dg, of the 32 rows d_k or t of each warp: a_t and b_s, W's sums over t with s before the
  // column; [2][32] W of P's and N's rows 32 .. summed over the columns before 32
  float *part_a = invE2 + 2 * kBC, *part_b = part_a + 4 * kBC, *part_w = part_b + 4 * kBC;
  float* row_w = part_w + 4 * kBC;
  // by the head's number: [4][8] <H, dH'>, [2][2] 1 / scale of H, dH'
  float* red = row_w + kBC;
  // this warp's part of a tile is written: the issuer may use it
  auto ready = [&](int b) {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[b]);
  };

  if (warp < 8) {
    setmaxnreg_inc<kRegsRows>();
    const int qd = warp & 3, ch = warp >> 2;  // TMEM lanes 32 qd .., 32 columns 32 ch ..
    const int dk = 32 * qd + lane;
    const bool on = D == 128 || dk < D;
    const uint32_t tl = tmem + (uint32_t(32 * qd) << 16) + 32 * ch;
    // factors and gates of head h, into the buffer of its parity
    auto load_head = [&](int h) {
      const size_t unit = size_t(i) * a.H_v + h;
      const int p = h & 1;
      if (tid < kFac / 4)
        cp_async16(base + L::Fac + p * kFac * 4 + tid * 16, a.fac + unit * kFac + tid * 4);
      else if (tid >= 128 && tid < 128 + kBC / 2)
        cp_async16(base + L::G + p * kBC * 8 + (tid - 128) * 16,
                   a.G + unit * kBC + (tid - 128) * 2);
      cp_async_commit();
    };
    float dqs[32] = {}, dks[32] = {};
    load_head(h0);
    // Head h's masks and the sums over d_v, the next head's rows, then h's other sums (while the
    // next head's P and N are multiplied).
    for (int h = h0 - 1; h < h0 + heads; ++h) {
      const bool on_head = h >= h0, more = h + 1 < h0 + heads;
      const uint32_t ph = (h - h0) & 1;
      const float* fac = reinterpret_cast<const float*>(smem + L::Fac) + (h & 1) * kFac;
      const float2* Gs = reinterpret_cast<const float2*>(smem + L::G) + (h & 1) * kBC;
      const float *invU = invU2 + kBC * (h & 1), *invE = invE2 + kBC * (h & 1);
      if (on_head) {
        // the rows' scales are there, the last head's factors and its parts of dg free
        named_sync(3, kGradsRows + 32);
        if (more) load_head(h + 1);
        // P and N: lanes 0-63 are rows of P, 64-127 of N
        float x[32];
        mbar_wait(&bars[gPN], ph, abort_flag, err, 64u);
        tc_fence_after();
        {
          float y[32];
          tmem_ld32(tl + kTPN, x);
          tmem_ld_wait();
          if (qd >= 2) {
            tmem_ld32(tl + kTEL, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] += y[k];
          }
        }
        {
          const bool isn = qd >= 2;
          const int pr = dk & 63, pb = pr >> 4;
          const float2 Gr = Gs[pr];
          const float fr = isn ? -invE[pr] : fac[kFo + pr];
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {  // 16-column blocks
            const int s0 = 32 * ch + 16 * cb, sb = s0 >> 4;
            const float2 Gb = Gs[s0 + 15];  // the decay in two factors, see steep()
            const float fe = pb < sb ? 0.f : fr * expdiff(Gr, Gb);
            const int last = pb > sb ? 16 : pb < sb ? 0 : pr - s0 + (isn ? 0 : 1);
            if (pb >= sb && steep(Gr, Gb)) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                x[16 * cb + k] = k < last
                    ? x[16 * cb + k] * invU[s0 + k] * (expdiff(Gr, Gs[s0 + k]) * fr) : 0.f;
            } else {
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                // (the decay's two factors first: either of them may be out of range with 1 / scale)
                const float4 e4 = *reinterpret_cast<const float4*>(fac + kFend + s0 + k);
                const float4 u4 = *reinterpret_cast<const float4*>(invU + s0 + k);
                float* y = x + 16 * cb + k;
                y[0] = k < last ? y[0] * u4.x * (fe * e4.x) : 0.f;
                y[1] = k + 1 < last ? y[1] * u4.y * (fe * e4.y) : 0.f;
                y[2] = k + 2 < last ? y[2] * u4.z * (fe * e4.z) : 0.f;
                y[3] = k + 3 < last ? y[3] * u4.w * (fe * e4.w) : 0.f;
              }
            }
          }
          // bf16 limbs: decays set the elements of a row as well as those of a column apart, and
          // the tiles are multiplied along both, so no scale would do
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4][2];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              split_bf16(x[8 * k + 2 * y], x[8 * k + 2 * y + 1], w[y]);
            const uint32_t at = base + sw128_offset(pr, 64 * ch + 16 * k);
            st_shared_v4(at + (isn ? L::NH : L::PH), w[0][0], w[1][0], w[2][0], w[3][0]);
            st_shared_v4(at + (isn ? L::NL : L::PL), w[0][1], w[1][1], w[2][1], w[3][1]);
          }
        }
        ready(gP);
        // W, and what of it crosses each row of this half: 0 where t comes before the columns
        if (ch <= (qd & 1)) {
#pragma unroll
          for (int cb = 0; cb < 2; ++cb) {
            float y[16];
            tmem_ld16(tl + kTQK + 16 * cb, y);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k)  // (P's diagonal crosses none)
              x[16 * cb + k] *= 32 * ch + 16 * cb + k == (dk & 63) ? 0.f : y[k];
          }
          float run = 0.f;
#pragma unroll
          for (int k = 0; k < 32; ++k) {  // of the columns before k, for t >= k
            const float w = x[k];
            x[k] = ch < (qd & 1) || k <= lane ? run : 0.f;
            run += w;
          }
          if (ch < (qd & 1)) row_w[32 * (qd >> 1) + lane] = run;
          part_w[qd * kBC + 32 * ch + lane] = sum_over_lanes(x);
        }
        // dq, dk and dg, what comes from the states: row d_k of this thread, 2 x 16 chunk rows
        mbar_wait(&bars[gStates], ph, abort_flag, err, 64u);
        tc_fence_after();
        const float ih = red[32 + 2 * (h & 1)], id = red[33 + 2 * (h & 1)];  // the states' scales
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) {
          float x0[16], x1[16], x2[16];
          const int s0 = 32 * ch + 16 * cb;
          tmem_ld16(tl + kTA1 + 16 * cb, x0);
          tmem_ld16(tl + kTA2 + 16 * cb, x1);
          tmem_ld16(tl + kTA6 + 16 * cb, x2);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int r = s0 + k;
            const float eg = fac[kFeG + r] * ih;
            const float dq = x0[k] * fac[kFo + r] * eg, dkh = x1[k] * invE[r] * eg;
            const float dkd = x2[k] * invU[r] * (fac[kFeT + r] * id);
            dqs[16 * cb + k] += dq;
            dks[16 * cb + k] += dkd - dkh;
            float qv = 0.f, kv = 0.f;
            if (on) {
              const uint8_t* at = smem + L::QK + (dk >> 6) * L::kQK + sw128_offset(r, (dk & 63) * 2);
              qv = bf16f(*reinterpret_cast<const uint16_t*>(at));
              kv = bf16f(*reinterpret_cast<const uint16_t*>(at + kBlk));
            }
            x0[k] = fmaf(qv, dq, -(kv * dkh));
            x1[k] = kv * dkd;
          }
          const float sa = sum_over_lanes(x0), sb = sum_over_lanes(x1);
          if ((lane & 1) == 0) {
            part_a[qd * kBC + s0 + (lane >> 1)] = sa;
            part_b[qd * kBC + s0 + (lane >> 1)] = sb;
          }
        }
        ready(gE);
        named_arrive(2, kGradsRows + 32);  // warp 13 sums dg
      }
      if (more) {
        const int n = h + 1;
        const size_t unit = size_t(i) * a.H_v + n;
        const float* fan = reinterpret_cast<const float*>(smem + L::Fac) + (n & 1) * kFac;
        // Rows 8 w .. 8 w + 7 in two halves, 8 lanes a row, 4 J columns a lane.
        const int l8 = lane & 7;
        float4 u[2][J], e[2][J];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int r = 8 * warp + 4 * m + (lane >> 3);
          const float* up = a.u + unit * kBC * D + r * 32 + 4 * l8;
          const float* ep = a.E + unit * kBC * D + r * 32 + 4 * l8;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            u[m][j] = __ldcg(reinterpret_cast<const float4*>(up + kBC * 32 * j));
            e[m][j] = __ldcg(reinterpret_cast<const float4*>(ep + kBC * 32 * j));
          }
        }
        if (tid == 0 && n + 1 < h0 + heads) {
          prefetch_l2(a.u + (unit + 1) * kBC * D, kBC * D * 4);
          prefetch_l2(a.E + (unit + 1) * kBC * D, kBC * D * 4);
        }
        cp_async_wait<0>();  // the factors
        named_sync(1, kGradsRows);  // ... are there, and every row warp is done with the last tiles
        // dv, dbeta, and the f16 tiles of u and E
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int r = 8 * warp + 4 * m + (lane >> 3);
          const float bt = fan[kFbeta + r];
          float db = 0.f, mu = 0.f, me = 0.f;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float4 &x = u[m][j], &y = e[m][j];
            db = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, db))));
            x.x *= bt, x.y *= bt, x.z *= bt, x.w *= bt;
            y.x *= bt, y.y *= bt, y.z *= bt, y.w *= bt;
            mu = max_nan(mu, max_nan(max_nan(fabsf(x.x), fabsf(x.y)), max_nan(fabsf(x.z), fabsf(x.w))));
            me = max_nan(me, max_nan(max_nan(fabsf(y.x), fabsf(y.y)), max_nan(fabsf(y.z), fabsf(y.w))));
          }
#pragma unroll
          for (int off = 1; off < 8; off <<= 1) {
            db += __shfl_xor_sync(0xffffffffu, db, off);
            mu = fmaxf(mu, __shfl_xor_sync(0xffffffffu, mu, off));
            me = fmaxf(me, __shfl_xor_sync(0xffffffffu, me, off));
          }
          float iu, ie;
          const float su = pow2_scale(mu, &iu), se = pow2_scale(me, &ie);
          if (l8 == 0) {
            if (r < c.rows) a.dbeta[size_t(c.row0 + r) * a.H_v + n] = db;
            invU2[kBC * (n & 1) + r] = iu, invE2[kBC * (n & 1) + r] = ie;
          }
          uint16_t* dv = a.dv + (size_t(c.row0 + r) * a.H_v + n) * D + 4 * l8;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const float4 x = u[m][j], y = e[m][j];
            if (r < c.rows)
              *reinterpret_cast<uint2*>(dv + 32 * j) =
                  make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
            const int col = 4 * l8 + 32 * j;
            const uint32_t at = (col >> 6) * kBlk + sw128_offset(r, (col & 63) * 2);
            uint32_t p0, p1, q0, q1;
            split_f16(x.x * su, x.y * su, p0, q0);
            split_f16(x.z * su, x.w * su, p1, q1);
            st_shared_v2(base + L::UH + at, p0, p1);
            st_shared_v2(base + L::UL + at, q0, q1);
            split_f16(y.x * se, y.y * se, p0, q0);
            split_f16(y.z * se, y.w * se, p1, q1);
            const uint32_t e_at = base + L::OE + (col >> 6) * (L::kOE - kBlk) + kBlk + at;
            st_shared_v2(e_at, p0, p1);
            st_shared_v2(e_at + kBlk, q0, q1);
          }
        }
        ready(gU);
      }
      if (!on_head) continue;
      // and what comes from the chunk's own rows
      mbar_wait(&bars[gA34], ph, abort_flag, err, 64u);
      tc_fence_after();
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float x0[16], x1[16];
        tmem_ld16(tl + kTA3 + 16 * cb, x0);
        tmem_ld16(tl + kTA4 + 16 * cb, x1);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) dqs[16 * cb + k] += x0[k], dks[16 * cb + k] += x1[k];
      }
    }
    if constexpr (split) {
      // One head a CTA, the key head's CTAs a cluster: each sums every vpg-th row of all of
      // them, in the heads' order.  (The states have been multiplied: their slots are free.)
      float* mine = reinterpret_cast<float*>(smem + L::H) + ch * D + dk;
      if (on) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          mine[4 * k * D] = dqs[k];
          mine[(4 * k + 2) * D] = dks[k];
        }
      }
      cluster_sync();
      for (int k = int(cluster_ctarank()); on && k < min(32, c.rows - 32 * ch); k += vpg) {
        float x = 0.f, y = 0.f;
        for (int w = 0; w < vpg; ++w) {
          const uint32_t from = mapa_shared(smem_u32(mine + 4 * k * D), w);
          x += ld_cluster_f32(from), y += ld_cluster_f32(from + 2 * D * 4);
        }
        const size_t at = (size_t(c.row0 + 32 * ch + k) * a.H_k + hk) * D + dk;
        a.dq[at] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        a.dk[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      }
      cluster_sync();  // the others have read
    } else if (on) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const int rr = 32 * ch + k;
        if (rr < c.rows) {
          const size_t at = (size_t(c.row0 + rr) * a.H_k + hk) * D + dk;
          a.dq[at] = __bfloat16_as_ushort(__float2bfloat16_rn(dqs[k]));
          a.dk[at] = __bfloat16_as_ushort(__float2bfloat16_rn(dks[k]));
        }
      }
    }
  } else if (warp < 12) {
    setmaxnreg_dec<kRegsStates>();
    const int t = tid - kGradsRows;
    // By halves of d_v: H's f32 values come to its slot by a bulk copy, those of dH' to the other,
    // and are turned into limbs there.  The next half's copy to a slot starts when that has been
    // multiplied.
    constexpr int kHalves = D / 64, kBytes = 64 * D * 4;
    constexpr int kQuads = kBytes / 16 / kGradsStates;  // 16 or 8 a thread
    const size_t unit = size_t(i) * a.H_v + h0;
    const uint32_t slot_h = base + L::H, slot_d = slot_h + L::kSlot;
    int loads[2] = {};
    auto load = [&](int p, int x) {  // the p-th half of the CTA's states H or dH'
      mbar_arrive_expect_tx(&bars[gLand + x], kBytes);
      bulk_load_g2s(smem + L::H + x * L::kSlot,
                    (x ? a.dH : a.H) + unit * D * D + size_t(p) * 64 * D, kBytes, &bars[gLand + x]);
      ++loads[x];
    };
    const float* hm = a.Hmax + unit * 16 + (lane & 15);
    float largest = *hm;  // lanes 0-7: |H| of a scan warp's part, 8-15: |dH|
    if (t == 0) load(0, 0), load(0, 1);
    int p = 0;
    const int halves = heads * kHalves;
    bool ok = true;
    for (int h = h0; h < h0 + heads; ++h, hm += 16) {
#pragma unroll
      for (int off = 1; off < 8; off <<= 1)
        largest = max_nan(largest, __shfl_xor_sync(0xffffffffu, largest, off));
      float ih, id;
      const float sh = pow2_scale(__shfl_sync(0xffffffffu, largest, 0), &ih);
      const float sd = pow2_scale(__shfl_sync(0xffffffffu, largest, 8), &id);
      if (h + 1 < h0 + heads) largest = hm[16];
      float hh = 0.f;
#pragma unroll 1
      for (int half = 0; half < kHalves; ++half, ++p) {
        if (t == 0 && p + 1 < halves) {  // the next half to L2
          prefetch_l2(a.H + unit * D * D + size_t(p + 1) * 64 * D, kBytes);
          prefetch_l2(a.dH + unit * D * D + size_t(p + 1) * 64 * D, kBytes);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t slot = x ? slot_d : slot_h;
          float4 v[kQuads];
          ok = mbar_wait(&bars[gLand + x], p & 1, abort_flag, err, 64u) && ok;
#pragma unroll
          for (int m = 0; m < kQuads; ++m)
            v[m] = *reinterpret_cast<const float4*>(smem + L::H + x * L::kSlot +
                                                    16 * (t + m * kGradsStates));
          if (x) {  // <H, dH'>, H from its limbs
#pragma unroll
            for (int m = 0; m < kQuads; ++m) {
              const uint32_t at = L::H + quad_place<D>(t + m * kGradsStates);
              const uint2 hi = *reinterpret_cast<const uint2*>(smem + at);
              const uint2 lo = *reinterpret_cast<const uint2*>(smem + at + 2 * kBlk);
              const float2 a0 = add2(unpack_f16(hi.x), unpack_f16(lo.x));
              const float2 a1 = add2(unpack_f16(hi.y), unpack_f16(lo.y));
              hh += fmaf(a0.x, v[m].x, a0.y * v[m].y) + fmaf(a1.x, v[m].z, a1.y * v[m].w);
            }
          }
          if (x) fence_proxy_async_smem();  // H's limbs have been read: before a copy comes there
          named_sync(4, kGradsStates);      // all have read
          if (x && t == 0 && p + 1 < halves && mbar_test_wait(&bars[gFree], p & 1)) load(p + 1, 0);
          const float s = x ? sd : sh;
#pragma unroll
          for (int m = 0; m < kQuads; ++m) {
            const uint32_t to = slot + quad_place<D>(t + m * kGradsStates);
            uint32_t p0, p1, q0, q1;
            split_f16(v[m].x * s, v[m].y * s, p0, q0);
            split_f16(v[m].z * s, v[m].w * s, p1, q1);
            st_shared_v2(to, p0, p1);
            st_shared_v2(to + 2 * kBlk, q0, q1);
          }
          if (x == 0 && half == 0 && t == 0) {
            // (The last head's states have been multiplied, so the rows' warps are done with the
            // head before it, whose scales were here.)
            red[32 + 2 * (h & 1)] = ih, red[33 + 2 * (h & 1)] = id;
          }
          if (x && half + 1 == kHalves) {
            hh = warp_sum(hh) * ih;
            if (lane == 0) red[8 * (h & 3) + warp - 8] = hh;
          }
          ready(gFull + x);
        }
        if (t == 0 && p + 1 < halves) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (loads[x] == p + 1) {
              ok = mbar_wait(&bars[gFree + x], p & 1, abort_flag, err, 64u) && ok;
              if (ok) load(p + 1, x);
            }
        }
        __syncwarp();
      }
    }
    if (t == 0)  // nothing may still be landing in shared memory at exit
      for (int x = 0; x < 2; ++x) mbar_wait(&bars[gLand + x], (loads[x] - 1) & 1, nullptr, err, 32u);
    if constexpr (split) cluster_sync(), cluster_sync();
  } else {
   setmaxnreg_dec<kRegsIssue>();
   if (warp == 12 && lane == 0) {
    // The issuer; it also loads each head's dO.
    // Descriptors: the high word is a constant, the low one an address and the (for the
    // K-major tiles unused) distance of 64-column blocks.
    // (In a cluster the address has the CTA's rank above its low 18 bits.)
    uint32_t b4 = (split ? base & 0x3ffffu : base) >> 4;
    constexpr uint32_t kKmaj = 1u << 16, kMnmaj = (uint32_t(L::kQK) >> 4) << 16;
    constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
    auto desc = [&](uint32_t low) { return uint64_t(kHigh) << 32 | low; };
    constexpr uint32_t id64 = make_idesc_f16(128, 64, 0, 0), id128 = make_idesc_f16(128, 128, 0, 0);
    constexpr uint32_t id_qk = make_idesc_bf16(128, 64, 0, 0);
    constexpr uint32_t id_a128 = make_idesc_bf16(128, 128, 1, 0);  // A MN-major
    constexpr uint32_t id_ab = make_idesc_bf16(128, 64, 1, 1);  // both MN-major
    auto load_o = [&](int h) {
      const uint8_t* src = a.O + (size_t(i) * a.H_v + h) * L::kTile;
      for (int x = 0; x < D / 64; ++x)
        bulk_load_g2s(smem + L::OE + x * L::kOE, src + x * kBlk, kBlk, &bars[gO]);
    };
    mbar_arrive_expect_tx(&bars[gO], L::kTile);
    load_o(h0);
    int loads = 1;
    constexpr uint32_t oe = L::OE, el = L::OE + 2 * kBlk, uh = L::UH, ul = L::UL;
    constexpr uint32_t tq = L::QK, tk = L::QK + kBlk;
    // descriptors: dO and beta E, Q and K, a slot (64 columns), 64 rows, and those along their columns
    auto out = [&](uint32_t tile, int kk) {
      return desc(b4 + (kKmaj | (tile + (kk >> 2) * L::kOE + (kk & 3) * 32) >> 4));
    };
    auto both_qk = [&](uint32_t tile, int kk) {
      return desc(b4 + (kKmaj | (tile + (kk >> 2) * L::kQK + (kk & 3) * 32) >> 4));
    };
    auto slot = [&](int x, int limb, int kk) {
      return desc(b4 + (kKmaj | (L::H + x * L::kSlot + limb * 2 * kBlk + (kk & 3) * 32) >> 4));
    };
    auto flat = [&](uint32_t tile, int kk) {
      return desc(b4 + (kKmaj | (tile + (kk >> 2) * kBlk + (kk & 3) * 32) >> 4));
    };
    auto rows = [&](uint32_t tile, int kk) { return desc(b4 + (kMnmaj | (tile + kk * 2048) >> 4)); };
    bool ok = true;
    int p = 0;  // halves of states
    ok = mbar_wait(&bars[gQK], 0, abort_flag, err, 128u);
    tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      mma_bf16_ss(tmem + kTQK, both_qk(tq, kk), both_qk(tk, kk), id_qk, kk != 0);
    for (int h = h0; h < h0 + heads && ok; ++h) {
      const uint32_t ph = (h - h0) & 1;
      asm volatile("" : "+r"(b4));  // (a hundred descriptors are made where they are needed, not kept)
      ok = mbar_wait(&bars[gO], ph, abort_flag, err, 128u) &&
           mbar_wait(&bars[gU], ph, abort_flag, err, 128u);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_ss(tmem + kTPN, out(oe, kk), flat(ul, kk), id64, kk != 0);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_ss(tmem + kTPN, out(oe, kk), flat(uh, kk), id64, 1u);
      // (rows 64 to 127 of this one: beta E's low limb)
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_ss(tmem + kTEL, out(oe + kBlk, kk), flat(uh, kk), id64, kk != 0);
      mma_commit(&bars[gPN]);
      // (the rows' warps have read the last head's sums)
      if (h > h0) ok = mbar_wait(&bars[gE], ph ^ 1, abort_flag, err, 128u);
      if (!ok) break;
#pragma unroll 1
      for (int k0 = 0; k0 < D / 16; k0 += 4, ++p) {  // by halves of d_v
        asm volatile("" : "+r"(b4));
        ok = mbar_wait(&bars[gFull], p & 1, abort_flag, err, 128u);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_ss(tmem + kTA1, slot(0, 1, kk), out(oe, k0 + kk), id128, k0 + kk != 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_ss(tmem + kTA2, slot(0, 0, kk), out(el, k0 + kk), id64, 1u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_ss(tmem + kTA1, slot(0, 0, kk), out(oe, k0 + kk), id128, 1u);
        mma_commit(&bars[gFree]);
        ok = mbar_wait(&bars[gFull + 1], p & 1, abort_flag, err, 128u);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < 3; ++x)  // low x high, high x low, high x high
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ss(tmem + kTA6, slot(1, x == 0, kk), flat(x == 1 ? ul : uh, k0 + kk), id64,
                        k0 + kk + x != 0);
        mma_commit(&bars[gFree + 1]);
      }
      if (!ok) break;
      mma_commit(&bars[gStates]);
      if (h + 1 < h0 + heads) {  // dO's last reader is done
        ok = mbar_wait(&bars[gStates], ph, abort_flag, err, 128u);
        if (!ok) break;
        mbar_arrive_expect_tx(&bars[gO], L::kTile);
        load_o(h + 1);
        ++loads;
      }
      ok = mbar_wait(&bars[gP], ph, abort_flag, err, 128u);
      if (!ok) break;
      tc_fence_after();
      // A limb of P and that of N are one tile of 128 rows, A3 and A4 side by side.
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ss(tmem + kTA3, rows(tk, kk), flat(L::PL, kk), id_a128, kk != 0);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16_ss(tmem + kTA3, rows(tk, kk), flat(L::PH, kk), id_a128, 1u);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          mma_bf16_ss(tmem + kTA4, rows(tq, kk), rows(x ? L::PH : L::PL, kk), id_ab, 1u);
          mma_bf16_ss(tmem + kTA4, rows(tk, kk), rows(x ? L::NH : L::NL, kk), id_ab, 1u);
        }
      mma_commit(&bars[gA34]);
    }
    mma_commit(&bars[gDrain]);
    mbar_wait(&bars[gDrain], 0, nullptr, err, 32u);
    mbar_wait(&bars[gO], (loads - 1) & 1, nullptr, err, 32u);
   } else if (warp >= 14) {  // Q and K
    const uint16_t* src = (warp == 14 ? a.q : a.k) + hk * D;
    const uint32_t to = base + L::QK + (warp == 14 ? 0 : kBlk);
    for (int y = lane; y < kBC * D / 8; y += 32) {
      const int r = y / (D / 8), col = 8 * (y % (D / 8));
      cp_async16(to + (col >> 6) * L::kQK + sw128_offset(r, (col & 63) * 2),
                 r < c.rows ? src + size_t(c.row0 + r) * a.qk_stride + col : src, r < c.rows);
    }
    cp_async_commit();
    cp_async_wait<0>();
    ready(gQK);
   } else if (warp == 13) {
    for (int h = h0; h < h0 + heads; ++h) {
      named_sync(3, kGradsRows + 32);
      named_sync(2, kGradsRows + 32);
      // Two rows a lane, 2 l and 2 l + 1: sums of a from the row on, of b before it, and of W; of
      // row_w, for the rows 32 .., from the row on.
      double up[2], down[2], far[2], own[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 2 * lane + k;
        float sa = 0.f, sb = 0.f, sw = 0.f;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) sa += part_a[w * kBC + r], sb += part_b[w * kBC + r];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (r < 32 || w & 1) sw += part_w[w * kBC + r];
        up[k] = sa, down[k] = sb, own[k] = sw;
        far[k] = r < 32 ? 0.0 : double(row_w[r - 32]) + double(row_w[r]);
      }
      double run_a = up[0] + up[1], run_f = far[0] + far[1], run_b = down[0] + down[1];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double wa = __shfl_down_sync(0xffffffffu, run_a, off);
        const double wf = __shfl_down_sync(0xffffffffu, run_f, off);
        const double wb = __shfl_up_sync(0xffffffffu, run_b, off);
        if (lane + off < 32) run_a += wa, run_f += wf;
        if (lane >= off) run_b += wb;
      }
      // (the sums before and behind the lane's rows as sums, not as differences: nothing cancels)
      double next_a = __shfl_down_sync(0xffffffffu, run_a, 1);
      double next_f = __shfl_down_sync(0xffffffffu, run_f, 1);
      double prev_b = __shfl_up_sync(0xffffffffu, run_b, 1);
      if (lane == 31) next_a = next_f = 0.0;
      if (lane == 0) prev_b = 0.0;
      const float* fac = reinterpret_cast<const float*>(smem + L::Fac) + (h & 1) * kFac;
      double hh = 0.0;
#pragma unroll
      for (int w = 0; w < kGradsStates / 32; ++w) hh += red[8 * (h & 3) + w];
      hh *= fac[kFeC];
      const double z[2] = {hh + (next_a + up[1] + up[0]) + prev_b + own[0] +
                               (lane < 16 ? 0.0 : next_f + far[1] + far[0]),
                           hh + (next_a + up[1]) + (prev_b + down[0]) + own[1] +
                               (lane < 16 ? 0.0 : next_f + far[1])};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 2 * lane + k;
        if (r < c.rows) a.dg[size_t(c.row0 + r) * a.H_v + h] = float(z[k]);
      }
    }
   }
   __syncwarp();
   if constexpr (split) cluster_sync(), cluster_sync();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------

namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Lays the workspace out behind `base` (which may be null) and returns its size.
size_t layout(BwdArgs* a, char* base, int total_tokens, int num_seqs, int H_k, int H_v, int D) {
  const size_t mc = size_t(total_tokens / kBC) + size_t(num_seqs);
  const size_t units = mc * H_v, tile = size_t(D) / 64 * kBlk;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at += up256(bytes);
    return p;
  };
  a->max_chunks = int(mc);
  a->cu_chunks = reinterpret_cast<int32_t*>(take((size_t(num_seqs) + 1) * 4));
  a->chunk_seq = reinterpret_cast<int32_t*>(take(mc * 4));
  a->KQ = reinterpret_cast<uint8_t*>(take(mc * H_k * 2 * tile));
  a->O = reinterpret_cast<uint8_t*>(take(units * tile));
  a->GO = reinterpret_cast<uint8_t*>(take(units * 2 * tile));
  a->S = reinterpret_cast<uint8_t*>(take(units * 3 * kBlk));
  a->Y0 = reinterpret_cast<float*>(take(units * kBC * D * 4));
  a->fac = reinterpret_cast<float*>(take(units * kFac * 4));
  a->ff = reinterpret_cast<float*>(take(units * kFwdFac * 4));
  a->fb = reinterpret_cast<float*>(take(units * kBackFac * 4));
  a->G = reinterpret_cast<float2*>(take(units * kBC * 8));
  a->u = reinterpret_cast<float*>(take(units * kBC * D * 4));
  a->E = reinterpret_cast<float*>(take(units * kBC * D * 4));
  a->H = reinterpret_cast<float*>(take(units * D * D * 4));
  a->dH = reinterpret_cast<float*>(take(units * D * D * 4));
  a->Hmax = reinterpret_cast<float*>(take(units * 2 * 8 * 4));
  return at;
}

template <int D>
cudaError_t run(const BwdArgs& a, cudaStream_t s) {
  constexpr int prep = PrepSmem<D>::kBytes, grads = GradsSmem<D>::kBytes;
  constexpr int scans = ScanSmem<D, true>::kBytes > ScanSmem<D, false>::kBytes
                            ? ScanSmem<D, true>::kBytes : ScanSmem<D, false>::kBytes;
  cudaError_t e;
  const auto kMax = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if ((e = cudaFuncSetAttribute(bwd_prep_kernel<D>, kMax, prep)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(bwd_scan_kernel<D>, kMax, scans)) != cudaSuccess) return e;
  // The value heads that share a key head in one CTA (their K K^T and Q K^T are made
  // once), unless that leaves SMs without a CTA: then every head has its own.
  const int vpg = a.H_v / a.H_k;
  const int heads = (long long)a.max_chunks * a.H_k >= 2 * a.sms ? vpg : 1;
  // Each kernel is launched while the one before it ends, and all of its CTAs wait for that
  // one's end themselves, before they read anything.
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attrs;
  cfg.numAttrs = a.num_seqs <= kFewSeqs ? 0 : 1;  // (the call's first kernel waits for all)
  cfg.gridDim = dim3(a.max_chunks, a.H_v / heads);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = prep;
  if ((e = cudaLaunchKernelEx(&cfg, bwd_prep_kernel<D>, a, heads)) != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2u * a.num_seqs * a.H_v);
  cfg.blockDim = dim3(kScanThreads);
  cfg.dynamicSmemBytes = scans;
  if ((e = cudaLaunchKernelEx(&cfg, bwd_scan_kernel<D>, a)) != cudaSuccess) return e;
  // Few chunks: one head a CTA, the key head's CTAs joined in clusters, while there is an SM for
  // each (one chunk of 48 heads in threes: 65.9 -> 48.0 us a call; 18 chunks of 6 heads: 118 -> 102;
  // at the rule's edge, where clusters of three leave SMs free and a second wave may come, 24 chunks
  // of 6 heads 163 -> 161, 12 of 12 heads 113.8 -> 113.0).
  const bool split = vpg > 1 && vpg <= 8 && (long long)a.max_chunks * a.H_v <= a.sms;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = attrs[1].val.clusterDim.z = 1;
  attrs[1].val.clusterDim.y = vpg;
  if (split) cfg.numAttrs = 2;
  cfg.gridDim = dim3(a.max_chunks, split ? a.H_v : a.H_k);
  cfg.blockDim = dim3(kGradsThreads);
  cfg.dynamicSmemBytes = grads;
  const auto last = split ? bwd_grads_kernel<D, true> : bwd_grads_kernel<D, false>;
  if ((e = cudaFuncSetAttribute(last, kMax, grads)) != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, last, a);
}

}  // namespace

size_t backward_workspace_bytes(int total_tokens, int num_seqs, int H_k, int H_v, int D) {
  BwdArgs a;
  return layout(&a, nullptr, total_tokens, num_seqs, H_k, H_v, D);
}

cudaError_t launch_backward(const BackwardCall& c, cudaStream_t s) {
  BwdArgs a;
  layout(&a, static_cast<char*>(c.workspace), c.total_tokens, c.num_seqs, c.H_k, c.H_v, c.D);
  a.q = c.q, a.k = c.k, a.v = c.v, a.dout = c.dout;
  a.g = c.g, a.beta = c.beta;
  a.qk_stride = c.qk_stride, a.v_stride = c.v_stride, a.gb_stride = c.gb_stride;
  a.cu = c.cu_seqlens;
  a.num_seqs = c.num_seqs, a.total_tokens = c.total_tokens, a.H_k = c.H_k, a.H_v = c.H_v;
  a.h0 = c.h0, a.dhT = c.dhT;
  a.dq = c.dq, a.dk = c.dk, a.dv = c.dv, a.dg = c.dg, a.dbeta = c.dbeta, a.dh0 = c.dh0;
  a.scale = c.scale;
  a.sms = sm_count();
  // Up to 32 sequences (a lane each): the first kernel finds its chunks itself, one launch less.
  if (c.num_seqs > kFewSeqs) {
    TablesCall t = {};
    t.cu_in = c.cu_seqlens;
    t.num_seqs = c.num_seqs;
    t.row_capacity = c.total_tokens;
    t.cu_chunks = a.cu_chunks;
    t.chunk_seq = a.chunk_seq;
    t.chunk_capacity = a.max_chunks;
    const cudaError_t e = launch_tables(t, s);
    if (e != cudaSuccess) return e;
  }
  return c.D == 128 ? run<128>(a, s) : run<64>(a, s);
}

}  // namespace gdn

// gdn_decode.cu -- the recurrent form of the gated delta rule: every sequence's
// state takes its new rows (none, one or a few) in place.
//
// For one row, with a = e^g and the state H = S^T [d_k][d_v] before it:
//   p = H^T k,  s = H^T q,  u = beta (v - a p),
//   o = scale (a s + (k.q) u),  H <- a H + k u^T.
// p, s and k.q come from one pass over H, so a row costs one reduction.
//
// Bound: HBM.  A row has 8 flops per state element against 8 bytes of it moved,
// so each state is read and written exactly once, and stays in registers over
// all rows of its sequence.  Columns of H never mix, so one CTA of 128 threads
// owns kCols = 32 columns of one (sequence, head): thread = (row group of D/16
// rows, column quad), every access a 16-byte one, 128 contiguous bytes per
// state row.  Small CTAs keep many loads in flight per SM and give 4 CTAs per
// head to a call with one sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr int kDecThreads = 128;
constexpr int kCols = 32;               // state columns of a CTA
constexpr int kQuads = kCols / 4;       // column quads
constexpr int kGroups = kDecThreads / kQuads;  // row groups (16)

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// One row's inputs as one thread needs them: k and q of its D / 16 state rows,
// v of its four columns, the two gates.
template <int D>
struct DecodeRow {
  uint32_t k[D / 32], q[D / 32];
  uint2 v;
  float g, beta;
  __device__ __forceinline__ void load(const uint16_t* kp, const uint16_t* qp,
                                       const uint16_t* vp, const float* gp, const float* bp) {
    if constexpr (D == 128) {
      *reinterpret_cast<uint4*>(k) = *reinterpret_cast<const uint4*>(kp);
      *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(qp);
    } else {
      *reinterpret_cast<uint2*>(k) = *reinterpret_cast<const uint2*>(kp);
      *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(qp);
    }
    v = *reinterpret_cast<const uint2*>(vp);
    g = *gp;
    beta = *bp;
  }
};

template <int D>
__global__ void __launch_bounds__(kDecThreads)
    decode_kernel(float* const* __restrict__ h_table, const uint16_t* __restrict__ q,
                  const uint16_t* __restrict__ k, int qk_stride,
                  const uint16_t* __restrict__ v, int v_stride, const float* __restrict__ g,
                  const float* __restrict__ beta, int gb_stride,
                  const int32_t* __restrict__ cu_seqlens, uint16_t* __restrict__ o,
                  int total_rows, int H_k, int H_v, float scale) {
  constexpr int RPT = D / kGroups;  // state rows per thread
  constexpr int SLICES = D / kCols;
  __shared__ float part[2][kDecThreads / 32][2 * kCols + 1];  // double-buffered over rows
  const int slice = blockIdx.x % SLICES;
  const int unit = blockIdx.x / SLICES;
  const int h = unit % H_v, b = unit / H_v;
  const int tid = threadIdx.x, quad = tid % kQuads, grp = tid / kQuads;
  const int warp = tid >> 5, lane = tid & 31;
  const int hk = h / (H_v / H_k);
  int row = b, end = b + 1;
  if (cu_seqlens != nullptr) {  // rows outside the call's are never touched
    row = max(cu_seqlens[b], 0);
    end = min(cu_seqlens[b + 1], total_rows);
  }
  if (row >= end) return;
  const int col = slice * kCols + quad * 4;
  uint16_t* orow = o + (size_t(row) * H_v + h) * D + col;
  float* base = h_table[b];
  if (base == nullptr) {  // padding sequence: zero outputs, no state
    for (; row < end; ++row, orow += size_t(H_v) * D)
      if (grp == 0) *reinterpret_cast<uint2*>(orow) = make_uint2(0u, 0u);
    return;
  }
  float* H = base + size_t(h) * D * D + size_t(grp * RPT) * D + col;
  float4 st[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) st[i] = *reinterpret_cast<const float4*>(H + i * D);

  const uint16_t* kp = k + size_t(row) * qk_stride + hk * D + grp * RPT;
  const uint16_t* qp = q + size_t(row) * qk_stride + hk * D + grp * RPT;
  const uint16_t* vp = v + size_t(row) * v_stride + h * D + col;
  const float* gp = g + size_t(row) * gb_stride + h;
  const float* bp = beta + size_t(row) * gb_stride + h;
  DecodeRow<D> cur;
  cur.load(kp, qp, vp, gp, bp);
  for (int buf = 0; row < end; ++row, buf ^= 1) {
    DecodeRow<D> next = cur;
    if (row + 1 < end) {
      kp += qk_stride, qp += qk_stride, vp += v_stride, gp += gb_stride, bp += gb_stride;
      next.load(kp, qp, vp, gp, bp);
    }
    float p[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f}, kq = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float ki = i & 1 ? bf16_hi(cur.k[i / 2]) : bf16_lo(cur.k[i / 2]);
      const float qi = i & 1 ? bf16_hi(cur.q[i / 2]) : bf16_lo(cur.q[i / 2]);
      p[0] = fmaf(st[i].x, ki, p[0]), s[0] = fmaf(st[i].x, qi, s[0]);
      p[1] = fmaf(st[i].y, ki, p[1]), s[1] = fmaf(st[i].y, qi, s[1]);
      p[2] = fmaf(st[i].z, ki, p[2]), s[2] = fmaf(st[i].z, qi, s[2]);
      p[3] = fmaf(st[i].w, ki, p[3]), s[3] = fmaf(st[i].w, qi, s[3]);
      kq = fmaf(ki, qi, kq);
    }
    // the warp's four row groups, then the four warps
#pragma unroll
    for (int off = kQuads; off < 32; off <<= 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        p[c] += __shfl_xor_sync(0xffffffffu, p[c], off);
        s[c] += __shfl_xor_sync(0xffffffffu, s[c], off);
      }
      kq += __shfl_xor_sync(0xffffffffu, kq, off);
    }
    if (lane < kQuads) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        part[buf][warp][4 * lane + c] = p[c];
        part[buf][warp][kCols + 4 * lane + c] = s[c];
      }
      if (lane == 0) part[buf][warp][2 * kCols] = kq;
    }
    // One barrier per row: the buffer written now is read again two rows on.
    __syncthreads();
    kq = 0.f;
#pragma unroll
    for (int w = 0; w < kDecThreads / 32; ++w) kq += part[buf][w][2 * kCols];
    const float a = expf(cur.g), vv[4] = {bf16_lo(cur.v.x), bf16_hi(cur.v.x), bf16_lo(cur.v.y),
                                          bf16_hi(cur.v.y)};
    float u[4], out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float pc = 0.f, sc = 0.f;
#pragma unroll
      for (int w = 0; w < kDecThreads / 32; ++w) {
        pc += part[buf][w][4 * quad + c];
        sc += part[buf][w][kCols + 4 * quad + c];
      }
      u[c] = cur.beta * (vv[c] - a * pc);
      out[c] = scale * fmaf(kq, u[c], a * sc);
    }
    if (grp == 0)
      *reinterpret_cast<uint2*>(orow) =
          make_uint2(pack_bf16x2(out[0], out[1]), pack_bf16x2(out[2], out[3]));
    orow += size_t(H_v) * D;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float ki = i & 1 ? bf16_hi(cur.k[i / 2]) : bf16_lo(cur.k[i / 2]);
      st[i].x = fmaf(ki, u[0], a * st[i].x);
      st[i].y = fmaf(ki, u[1], a * st[i].y);
      st[i].z = fmaf(ki, u[2], a * st[i].z);
      st[i].w = fmaf(ki, u[3], a * st[i].w);
    }
    cur = next;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) *reinterpret_cast<float4*>(H + i * D) = st[i];
}

cudaError_t launch_decode(float* const* h_table, const uint16_t* q, const uint16_t* k,
                          int qk_stride, const uint16_t* v, int v_stride, const float* g,
                          const float* beta, int gb_stride, const int32_t* cu_seqlens,
                          uint16_t* o, int batch, int total_rows, int H_k, int H_v, int D,
                          float scale, cudaStream_t s) {
  const unsigned grid = unsigned(batch) * unsigned(H_v) * unsigned(D / kCols);
  if (D == 128)
    decode_kernel<128><<<grid, kDecThreads, 0, s>>>(h_table, q, k, qk_stride, v, v_stride, g,
                                                    beta, gb_stride, cu_seqlens, o, total_rows,
                                                    H_k, H_v, scale);
  else
    decode_kernel<64><<<grid, kDecThreads, 0, s>>>(h_table, q, k, qk_stride, v, v_stride, g,
                                                   beta, gb_stride, cu_seqlens, o, total_rows,
                                                   H_k, H_v, scale);
  return cudaGetLastError();
}

}  // namespace gdn

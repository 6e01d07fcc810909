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
//
// Measured (48 heads, D = 128, one row each): 64 sequences 64 us a call (404 MB, 6.3 TB/s),
// 256 sequences 240 us (6.7 TB/s).  37 sequences of 0 to 6 rows (32 heads; 31 with rows, 132 MB)
// take 35 us, 34 of them the kernel: there issue slots are 55 % used and the stalls are those of
// the rows' reductions (shuffles and shared memory) before those of loads, so the arithmetic is
// packed, two f32 per instruction (44 us of the call before).
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

// Six CTAs an SM: with the compiler's own choice of registers (96, five CTAs) 64 x 48 heads
// took 66.9 us a call instead of 66.0 and 256 x 48 251 instead of 248, with eight CTAs (spills)
// 70 us the first; the rows of 37 x 32 heads take 34 us of kernel instead of 32.
template <int D>
__global__ void __launch_bounds__(kDecThreads, 6)
    decode_kernel(float* const* __restrict__ h_table, const uint16_t* __restrict__ q,
                  const uint16_t* __restrict__ k, int qk_stride,
                  const uint16_t* __restrict__ v, int v_stride, const float* __restrict__ g,
                  const float* __restrict__ beta, int gb_stride,
                  const int32_t* __restrict__ cu_seqlens, uint16_t* __restrict__ o,
                  int total_rows, int H_k, int H_v, float scale) {
  constexpr int RPT = D / kGroups;  // state rows per thread
  constexpr int SLICES = D / kCols;
  // double-buffered over rows
  __shared__ __align__(16) float part[2][kDecThreads / 32][2 * kCols];
  __shared__ __align__(16) float part_kq[2][kDecThreads / 32];
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
  float2 st[RPT][2];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const float4 x = *reinterpret_cast<const float4*>(H + i * D);
    st[i][0] = make_float2(x.x, x.y), st[i][1] = make_float2(x.z, x.w);
  }

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
    if (cur.g < -104.f) {  // e^g is 0: the state is forgotten, whatever it holds (0 times NaN is NaN)
#pragma unroll
      for (int i = 0; i < RPT; ++i) st[i][0] = st[i][1] = make_float2(0.f, 0.f);
    }
    float2 p0{}, p1{}, s0{}, s1{};  // of the thread's columns 0, 1 and 2, 3
    float kq = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float ki = i & 1 ? bf16_hi(cur.k[i / 2]) : bf16_lo(cur.k[i / 2]);
      const float qi = i & 1 ? bf16_hi(cur.q[i / 2]) : bf16_lo(cur.q[i / 2]);
      p0 = fma2(st[i][0], both(ki), p0), p1 = fma2(st[i][1], both(ki), p1);
      s0 = fma2(st[i][0], both(qi), s0), s1 = fma2(st[i][1], both(qi), s1);
      kq = fmaf(ki, qi, kq);
    }
    // The warp's four row groups, the values spread over them: upper half s, lower half p,
    // then two columns each.
    const bool up = lane & 16, right = lane & 8;
    float2 a0 = up ? s0 : p0, a1 = up ? s1 : p1;
    const float2 b0 = up ? p0 : s0, b1 = up ? p1 : s1;
    a0 = add2(a0, make_float2(__shfl_xor_sync(0xffffffffu, b0.x, 16),
                              __shfl_xor_sync(0xffffffffu, b0.y, 16)));
    a1 = add2(a1, make_float2(__shfl_xor_sync(0xffffffffu, b1.x, 16),
                              __shfl_xor_sync(0xffffffffu, b1.y, 16)));
    const float2 mine = right ? a1 : a0, other = right ? a0 : a1;
    *reinterpret_cast<float2*>(&part[buf][warp][(up ? kCols : 0) + 4 * quad + (right ? 2 : 0)]) =
        add2(mine, make_float2(__shfl_xor_sync(0xffffffffu, other.x, 8),
                               __shfl_xor_sync(0xffffffffu, other.y, 8)));
    kq += __shfl_xor_sync(0xffffffffu, kq, 8);
    kq += __shfl_xor_sync(0xffffffffu, kq, 16);
    if (lane == 0) part_kq[buf][warp] = kq;
    // One barrier per row: the buffer written now is read again two rows on.
    __syncthreads();
    const float4 kq4 = *reinterpret_cast<const float4*>(part_kq[buf]);
    kq = (kq4.x + kq4.y) + (kq4.z + kq4.w);
    p0 = p1 = s0 = s1 = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kDecThreads / 32; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(&part[buf][w][4 * quad]);
      const float4 y = *reinterpret_cast<const float4*>(&part[buf][w][kCols + 4 * quad]);
      p0 = add2(p0, make_float2(x.x, x.y)), p1 = add2(p1, make_float2(x.z, x.w));
      s0 = add2(s0, make_float2(y.x, y.y)), s1 = add2(s1, make_float2(y.z, y.w));
    }
    const float a = expf(cur.g);
    const float2 beta2 = both(cur.beta);
    const float2 u0 = mul2(beta2, fma2(both(-a), p0, make_float2(bf16_lo(cur.v.x), bf16_hi(cur.v.x))));
    const float2 u1 = mul2(beta2, fma2(both(-a), p1, make_float2(bf16_lo(cur.v.y), bf16_hi(cur.v.y))));
    if (grp == 0) {
      const float2 x = mul2(both(scale), fma2(both(kq), u0, mul2(both(a), s0)));
      const float2 y = mul2(both(scale), fma2(both(kq), u1, mul2(both(a), s1)));
      *reinterpret_cast<uint2*>(orow) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
    }
    orow += size_t(H_v) * D;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float ki = i & 1 ? bf16_hi(cur.k[i / 2]) : bf16_lo(cur.k[i / 2]);
      st[i][0] = fma2(both(ki), u0, mul2(both(a), st[i][0]));
      st[i][1] = fma2(both(ki), u1, mul2(both(a), st[i][1]));
    }
    cur = next;
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
    *reinterpret_cast<float4*>(H + i * D) =
        make_float4(st[i][0].x, st[i][0].y, st[i][1].x, st[i][1].y);
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

// Products with packed 4-bit layers and 8-bit activations, for few tokens.
//
//   Y[t][r] = sum over regions  sw[r][g] sx[t][c] (sum_k q[r][k] x[t][k] - z[r][g] sum_k x[t][k])
//
// with q the layer's codes (0..15), x the activations' codes (int8), sw and z
// the layer's scales and zero points, sx the activations' scales; a region is
// a run of columns inside one weight group and one block of 128 columns.  The
// inner sums are whole numbers and exact in int32; the scales multiply them
// in fp32, so a region brings one rounding of the scales' product and one of
// the sum.
//
// The contraction runs on mma.sync m16n8k32 (u8 x s8, int32 accumulation)
// with the weights' rows as M and the tokens as N = 8: at few tokens the pass
// is bound by reading the packed weights once, and what counts is how little
// work a word of eight codes costs.  Two ANDs and a shift give its even and
// odd codes as bytes, which are the k positions of one mma; the activations
// are permuted to match (two PRMT for eight of them, shared by all row
// tiles).  The zero points are not subtracted from the codes: an mma of ones
// gives sum_k x in the same registers as the products, for all row tiles.
//
// A CTA has 8 warps and 32 rows of each layer; warp w takes the 128-column
// chunks w, w + 8, ... and a sum over the warps through shared memory ends
// the tile, in a fixed order.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "act8.cuh"
#include "common.cuh"

namespace gptq {
namespace w4a8 {

namespace cg = cooperative_groups;

constexpr int OUT_F32 = 0, OUT_BF16 = 1, OUT_I8 = 2;  // == GPTQ_F32, GPTQ_BF16, GPTQ_I8
constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int WT = 2;           // 16-row tiles of each layer
constexpr int ROWS = 16 * WT;   // rows of each layer per CTA
constexpr int TOK = 8;          // tokens per CTA
constexpr int CLUSTER = 128 / ROWS;  // CTAs that share a block of 128 output columns

struct Layer {
  const uint32_t* qweight;
  const float* scales;
  const uint8_t* zeros;
};

struct Params {
  Layer layer[2];
  const int8_t* x;
  const float* xs;
  void* y;
  float* ys;           // scales of an 8-bit output
  int64_t ldx, ldy;
  int64_t n;
  int d_row, d_col;
  int group, n_groups;  // of the weights; group = d_col when there is one a row
  int xgroups;          // 1, or one per 128 columns
  int out;
};

__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t even_codes(uint32_t w) { return w & 0x0F0F0F0Fu; }
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) { return (w >> 4) & 0x0F0F0F0Fu; }

__device__ __forceinline__ float silu_times(float g, float u) {
  return g / (1.0f + expf(-g)) * u;
}

__device__ __forceinline__ void store_out(const Params& p, int64_t at, float v) {
  if (p.out == OUT_BF16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  else static_cast<float*>(p.y)[at] = v;
}

// RJ: runs of 32 columns in a region: 1, 2, or 4 (whole chunks).  With whole
// chunks the k order inside a chunk is free, and a lane reads 16 bytes of a
// row (columns 32 t .. 32 t + 31 for lane t of a quad); else word 4 j + t.
template <bool GATED, int RJ>
__global__ void __launch_bounds__(THREADS, 2) w4a8_rows_kernel(const Params p) {
  constexpr int NL = GATED ? 2 : 1;
  constexpr int NREG = 4 / RJ;
  __shared__ float red[WARPS][NL * WT][32][4];
  __shared__ uint32_t tops[TOK];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int words = p.d_col >> 3;
  const int nchunks = (p.d_col + 127) >> 7;
  const int row0 = blockIdx.x * ROWS;
  const int64_t tok0 = static_cast<int64_t>(blockIdx.y) * TOK;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(TOK), p.n - tok0));

  float acc[NL * WT][4];
#pragma unroll
  for (int i = 0; i < NL * WT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.0f;

  // rows past the layer are computed on its last row and never written;
  // tokens past the batch are zeros
  int prow[WT][2];
#pragma unroll
  for (int i = 0; i < WT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) prow[i][h] = min(row0 + 16 * i + g + 8 * h, p.d_row - 1);
  const int8_t* xrow = p.x + (tok0 + (g < ntok ? g : 0)) * p.ldx;
  const float* xs0 = p.xs + (tok0 + min(2 * t, ntok - 1)) * p.xgroups;
  const float* xs1 = p.xs + (tok0 + min(2 * t + 1, ntok - 1)) * p.xgroups;

  if (row0 < p.d_row) {
    for (int c = warp; c < nchunks; c += WARPS) {
      uint2 xv[4];
      uint32_t w[NL * WT][2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the run of 32 columns that the lane's word j lies in
        const bool in = 128 * c + 32 * (RJ == 4 ? t : j) < p.d_col;
        const int word = 16 * c + (RJ == 4 ? 4 * t + j : 4 * j + t);
        xv[j] = in && g < ntok ? *reinterpret_cast<const uint2*>(xrow + 8 * word) : make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < NL * WT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            w[i][h][j] = in ? __ldg(p.layer[i / WT].qweight +
                                    static_cast<size_t>(prow[i % WT][h]) * words + word)
                            : 0u;
      }
      const int cx = p.xgroups == 1 ? 0 : c;
      const float sx0 = __ldg(xs0 + cx), sx1 = __ldg(xs1 + cx);
#pragma unroll
      for (int m = 0; m < NREG; ++m) {
        if (128 * c + 32 * RJ * m >= p.d_col) break;
        const int gi = (128 * c + 32 * RJ * m) / p.group;
        int sums[4] = {0, 0, 0, 0};
        uint32_t b0[RJ], b1[RJ];
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          b0[j] = __byte_perm(xv[RJ * m + j].x, xv[RJ * m + j].y, 0x6420);
          b1[j] = __byte_perm(xv[RJ * m + j].x, xv[RJ * m + j].y, 0x7531);
          mma_u8s8(sums, 0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u, b0[j], b1[j]);
        }
#pragma unroll
        for (int i = 0; i < NL * WT; ++i) {
          int prod[4] = {0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < RJ; ++j) {
            const uint32_t vg = w[i][0][RJ * m + j], vh = w[i][1][RJ * m + j];
            mma_u8s8(prod, even_codes(vg), even_codes(vh), odd_codes(vg), odd_codes(vh), b0[j], b1[j]);
          }
          const Layer& L = p.layer[i / WT];
          const size_t og = static_cast<size_t>(prow[i % WT][0]) * p.n_groups + gi;
          const size_t oh = static_cast<size_t>(prow[i % WT][1]) * p.n_groups + gi;
          const float sg = __ldg(L.scales + og), sh = __ldg(L.scales + oh);
          const int zg = __ldg(L.zeros + og), zh = __ldg(L.zeros + oh);
          acc[i][0] = fmaf(sg * sx0, static_cast<float>(prod[0] - zg * sums[0]), acc[i][0]);
          acc[i][1] = fmaf(sg * sx1, static_cast<float>(prod[1] - zg * sums[1]), acc[i][1]);
          acc[i][2] = fmaf(sh * sx0, static_cast<float>(prod[2] - zh * sums[2]), acc[i][2]);
          acc[i][3] = fmaf(sh * sx1, static_cast<float>(prod[3] - zh * sums[3]), acc[i][3]);
        }
      }
    }
  }

  // Sum over the warps.  Element e of lane l of a fragment is row
  // (l >> 2) + 8 (e >> 1) of the 16-row tile, token 2 (l & 3) + (e & 1).
#pragma unroll
  for (int i = 0; i < NL * WT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][i][lane][e] = acc[i][e];
  __syncthreads();
  const int rl = threadIdx.x & 31, tk = threadIdx.x >> 5;  // one output each
  const int fl = (rl & 7) * 4 + (tk >> 1), fe = 2 * ((rl >> 3) & 1) + (tk & 1);
  float v[NL];
#pragma unroll
  for (int a = 0; a < NL; ++a) {
    v[a] = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v[a] += red[w][a * WT + (rl >> 4)][fl][fe];
  }
  const bool live = row0 + rl < p.d_row && tk < ntok;
  const float out = GATED ? silu_times(v[0], v[NL - 1]) : v[0];
  if (!GATED || p.out != OUT_I8) {
    if (live) store_out(p, (tok0 + tk) * p.ldy + row0 + rl, out);
    return;
  }
  if constexpr (GATED) {
    // 8-bit output: a warp has one token's 32 rows; the CTAs of the cluster
    // exchange their maxima over the block of 128 output columns
    cg::cluster_group cl = cg::this_cluster();
    uint32_t top = __reduce_max_sync(0xffffffffu, live ? act8::abs_bits(out) : 0u);
    if (rl == 0) tops[tk] = top;
    cl.sync();
    for (int r = 0; r < CLUSTER; ++r) top = max(top, *cl.map_shared_rank(&tops[tk], r));
    const act8::Quant q = act8::quant_of(top);
    if (live) {
      static_cast<int8_t*>(p.y)[(tok0 + tk) * p.ldy + row0 + rl] =
          static_cast<int8_t>(act8::code_or_zero(out, q));
      if (row0 % 128 == 0 && rl == 0)
        p.ys[(tok0 + tk) * ((p.d_row + 127) / 128) + row0 / 128] = q.scale;
    }
    cl.sync();  // no CTA leaves while another may still read its maxima
  }
}

}  // namespace w4a8
}  // namespace gptq

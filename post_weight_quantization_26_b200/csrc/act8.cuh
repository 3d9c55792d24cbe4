// Residual addition, root-mean-square norm and 8-bit output in one pass.
//
//   r = x + residual              (rounded once, to the residual's type, and stored)
//   y = r * rsqrt(mean_k r_k^2 + eps) * weight
//   s = max|y| / 127,  q = rint(y * (127 / max|y|))   per token, or per 128 columns
//
// The norm is taken of the stored r, so a later reader of the residual
// stream sees the values that the codes were made from.  Everything between
// the loads and the stores is fp32.  Of the sum of squares a thread adds its own
// share in order, 8 to 32 columns with the row in registers and d / 256 in the
// kernel for any width, and the threads' sums meet in a tree: a relative error of
// at most (d / 256 + 42) 2^-24.  Squares outside fp32's range are lost: a token of
// values near 2^64 / sqrt(d) and beyond gives scales 0, with eps 0 one below 2^-63
// loses accuracy.
//
// Maxima are taken over the bit patterns of |y| as unsigned integers: they
// order like the values, and every NaN lies above infinity, so a NaN is never
// lost.  A maximum that is not finite gives the scale NaN and codes 0, which a
// product turns into NaN for the token.  A maximum of zero gives scale 0.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace gptq {
namespace act8 {

constexpr int GROUP = 128;  // columns that share a scale, where a token has several

struct Params {
  const void* x;
  const void* res;      // nullptr: r = x and nothing is stored
  void* res_out;
  const float* weight;  // nullptr: 1
  int8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldo, ldq;
  int64_t n;
  int d, n_groups;      // n_groups 1 with per-token scales
  float eps;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float& o, float v) { o = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16& o, float v) { o = __float2bfloat16_rn(v); }

// Scale and the multiplier of a maximum (given by its bits).  Maxima below
// 2^-100 are lifted by 2^64 before the division, as 127 / max would overflow;
// y is multiplied by `lift` first (exact for powers of two).
struct Quant {
  float scale, inv, lift;
};
__device__ __forceinline__ Quant quant_of(uint32_t top_bits) {
  Quant q;
  const float top = __uint_as_float(top_bits);
  q.lift = 1.0f;
  if (top_bits >= 0x7f800000u) {
    q.scale = __uint_as_float(0x7fc00000u);
    q.inv = 0.0f;
  } else if (top == 0.0f) {
    q.scale = q.inv = 0.0f;
  } else {
    q.scale = top / 127.0f;
    if (top < 7.8886090522e-31f) q.lift = 18446744073709551616.0f;  // 2^-100, 2^64
    q.inv = 127.0f / (top * q.lift);
  }
  return q;
}

// rint(y * inv) as the low byte of the sum with 1.5 * 2^23: one rounding, to
// nearest even, at the units' place.
__device__ __forceinline__ uint32_t code_of(float y, const Quant& q) {
  return __float_as_uint(fmaf(y * q.lift, q.inv, 12582912.0f)) & 0xffu;
}
// The same with NaN and infinity in y mapped to code 0.
__device__ __forceinline__ uint32_t code_or_zero(float y, const Quant& q) {
  return q.inv == 0.0f ? 0u : code_of(y, q);
}

__device__ __forceinline__ uint32_t abs_bits(float y) { return __float_as_uint(y) & 0x7fffffffu; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum (or maximum of bits) over the block; every thread gets it.  `buf` has
// one word per warp and is free again after the next block-wide barrier (a loop
// takes two in turn).
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? buf[lane] : 0.0f);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* buf) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, lane < warps ? buf[lane] : 0u);
}

// Eight consecutive elements as fp32, 16 or 32 aligned bytes.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// Round v to the type, store it, and leave the rounded values in v.
__device__ __forceinline__ void store8(float* p, float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of eight values as two words.
__device__ __forceinline__ uint2 codes8(const float (&y)[8], const Quant& q) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(fmaf(y[i] * q.lift, q.inv, 12582912.0f));
  if (q.inv == 0.0f) return make_uint2(0u, 0u);
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// Eight elements as they are in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ float at(int j) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
    if (sizeof(T) == 4) return __uint_as_float(w[j]);
    return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
  }
};

// Aligned rows of whole vectors of eight: a block a token, NV vectors a thread
// in registers, so the pass reads and writes each byte once and is bound by
// HBM: 16384 x 8192 bf16 with residual, 939 MB, in 172 us, 5.5 TB/s.  A block
// takes rows blockIdx.x, + gridDim.x, ... and has the next row's loads on the way
// while it reduces and writes the current one (AHEAD; 205 us with a block a row).
// Rows of more than 8192 columns take more threads, and then the registers do not
// hold a second row.  Sixteen lanes
// hold a group of 128 columns.  res_out may be the memory of x or of the
// residual: a row is loaded whole before it is stored, and no row's loads reach
// into another's.
template <typename TX, typename TR, int NV, bool AHEAD>
__global__ void __launch_bounds__(AHEAD ? 1024 / NV : 1024) rmsnorm_quant8_kernel(const Params p) {
  __shared__ float sums[2][32];
  __shared__ uint32_t tops[2][32];
  const int nvec = p.d >> 3;
  Raw8<TX> rx[AHEAD ? NV : 1];
  Raw8<TR> rr[AHEAD ? NV : 1];
  auto fetch = [&](int64_t t, int i, Raw8<TX>& x, Raw8<TR>& r) {
    const int k = threadIdx.x + i * blockDim.x;
    if (k >= nvec) return;
    x.load(static_cast<const TX*>(p.x) + t * p.ldx + 8 * k);
    if (p.res) r.load(static_cast<const TR*>(p.res) + t * p.ldr + 8 * k);
  };
  int64_t t = blockIdx.x;
  if (AHEAD)
#pragma unroll
    for (int i = 0; i < NV; ++i) fetch(t, i, rx[i], rr[i]);
  for (int turn = 0; t < p.n; turn ^= 1) {
    float v[NV][8], r[8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = threadIdx.x + i * blockDim.x, b = AHEAD ? i : 0;
      if (!AHEAD) fetch(t, i, rx[0], rr[0]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = k < nvec ? rx[b].at(j) : 0.0f;
      if (p.res && k < nvec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += rr[b].at(j);
        store8(static_cast<TR*>(p.res_out) + t * p.ldo + 8 * k, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += v[i][j] * v[i][j];
    }
    const int64_t now = t;
    t += gridDim.x;
    if (AHEAD && t < p.n)
#pragma unroll
      for (int i = 0; i < NV; ++i) fetch(t, i, rx[i], rr[i]);
    sum = block_sum(sum, sums[turn]);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
    uint32_t top[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int k = threadIdx.x + i * blockDim.x;
      if (p.weight && k < nvec) {
        load8(p.weight + 8 * k, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
      }
      top[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top[i] = max(top[i], abs_bits(v[i][j]));
      if (k >= nvec) top[i] = 0;  // 0 * infinity
    }
    int8_t* codes = p.codes + now * p.ldq;
    if (p.n_groups == 1) {
#pragma unroll
      for (int i = 1; i < NV; ++i) top[0] = max(top[0], top[i]);
      const Quant q = quant_of(block_max(top[0], tops[turn]));
      if (threadIdx.x == 0) p.scales[now] = q.scale;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
        if (k < nvec) *reinterpret_cast<uint2*>(codes + 8 * k) = codes8(v[i], q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int o = 8; o; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
        const Quant q = quant_of(top[i]);
        if (k < nvec) {
          *reinterpret_cast<uint2*>(codes + 8 * k) = codes8(v[i], q);
          if ((k & 15) == 0) p.scales[now * p.n_groups + (k >> 4)] = q.scale;
        }
      }
    }
  }
}

// Any width, stride and alignment: one block a token, three passes that read
// r back from where it is (the caches), an element at a time: 4096 x 4095 bf16 with
// residual take 59 us, 2.0 TB/s (4096 columns, in registers: 24 us).  A warp owns whole groups of 128
// columns, four a lane, and each element is only ever touched by one thread,
// so res_out may be the memory of x or of the residual.
template <typename TX, typename TR>
__global__ void __launch_bounds__(256) rmsnorm_quant8_any_kernel(const Params p) {
  __shared__ float sums[8];
  __shared__ uint32_t tops[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + t * p.ldx;
  const TR* res = p.res ? static_cast<const TR*>(p.res) + t * p.ldr : nullptr;
  TR* out = p.res ? static_cast<TR*>(p.res_out) + t * p.ldo : nullptr;
  const int ngr = (p.d + GROUP - 1) / GROUP;

  float sum = 0.0f;
  for (int g = warp; g < ngr; g += 8)
    for (int j = 0; j < 4; ++j) {
      const int k = g * GROUP + j * 32 + lane;
      if (k < p.d) {
        float r = to_f(x[k]);
        if (res) {
          TR o;
          from_f(o, r + to_f(res[k]));
          out[k] = o;
          r = to_f(o);
        }
        sum += r * r;
      }
    }
  sum = block_sum(sum, sums);
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
  auto value = [&](int k) {
    const float r = res ? to_f(out[k]) : to_f(x[k]);
    return r * rstd * (p.weight ? p.weight[k] : 1.0f);
  };

  uint32_t top = 0;
  Quant q;
  if (p.n_groups == 1) {
    for (int g = warp; g < ngr; g += 8)
      for (int j = 0; j < 4; ++j) {
        const int k = g * GROUP + j * 32 + lane;
        if (k < p.d) top = max(top, abs_bits(value(k)));
      }
    q = quant_of(block_max(top, tops));
    if (threadIdx.x == 0) p.scales[t] = q.scale;
  }
  for (int g = warp; g < ngr; g += 8) {
    float y[4];
    top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = g * GROUP + j * 32 + lane;
      y[j] = k < p.d ? value(k) : 0.0f;
      top = max(top, abs_bits(y[j]));
    }
    if (p.n_groups != 1) {
      q = quant_of(__reduce_max_sync(0xffffffffu, top));
      if (lane == 0) p.scales[t * p.n_groups + g] = q.scale;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = g * GROUP + j * 32 + lane;
      if (k < p.d) p.codes[t * p.ldq + k] = static_cast<int8_t>(code_or_zero(y[j], q));
    }
  }
}

}  // namespace act8
}  // namespace gptq

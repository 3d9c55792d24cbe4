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
// with the weights' rows as M and the tokens as N = 8 (up to four times): at
// few tokens the pass is bound by reading the packed weights once, and what
// counts is bytes in flight and how little work a word of eight codes costs.
// Two ANDs and a shift give a word's even and odd codes as bytes, which are
// the k positions of one mma; the activations are permuted to match (two PRMT
// for eight of them, shared by both row tiles).  The zero points are not
// subtracted from the codes: an mma of ones gives sum_k x in the same
// registers as the products, for both row tiles.
//
// A CTA has two 16-row tiles: rows of one layer, or the same rows of gate and
// up.  A producer warp brings stages of eight 128-column chunks into a ring by
// tensor copies (the tiles' words in boxes of 128 B rows, two chunks each; the
// tokens' codes in one box where the row is whole chunks), and of each stage
// warp w computes chunk w.  A sum over the warps through shared memory ends
// the tile, in a fixed order.  Two CTAs share an SM, with 128 KB of weights on
// the way, and take tile after tile, so the copies never pause.  Scales and
// zero points come with the stages by asynchronous copies of 16 bytes; where
// groups or alignment do not allow that, they are loaded one chunk ahead.  One
// token of 22016 x 8192: gate and up 40 to 42 us with the staged scales (4600 to
// 4860 GB/s, 0.71 to 0.74 of the memory's rate), 45 us with loads; the same loop
// without scales or products, copies alone, 34 us.  What is left is the chain of a stage, about
// a wait, the reads, 12 mma and their folds, on 16 warps an SM.
#pragma once

#include <cuda_bf16.h>

#include "act8.cuh"
#include "common.cuh"

namespace gptq {
namespace w4a8 {

constexpr int OUT_F32 = 0, OUT_BF16 = 1, OUT_I8 = 2;  // == GPTQ_F32, GPTQ_BF16, GPTQ_I8
// Fault injection, here and in the tile kernel: the producer issues no loads, or
// a stage of its ring is never counted as read, so that a wait runs out.
constexpr int STALL_LOADS = 1, STALL_STAGES = 2;
constexpr int WARPS = 8;     // computing warps
constexpr int THREADS = WARPS * 32 + 32;  // and the producer warp
constexpr int CPS = WARPS;      // 128-column chunks per stage

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
  uint32_t gmagic;      // ceil(2^32 / group): umulhi(k, gmagic) == k / group for k, group <= 2^16
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

// 4 or 16 bytes into shared memory without passing through a register.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// NL: layers; RJ: runs of 32 columns in a region: 1, 2, or 4 (whole chunks);
// NT: groups of eight tokens; STAGED: scales come with the stages, for groups of
// 32 RJ columns in fours and aligned rows.  Derived: S, the ring's stages, as many
// as let MINB CTAs share an SM.
template <int NL_, int RJ_, int NT_, bool STAGED_>
struct Cfg {
  static constexpr int NL = NL_, RJ = RJ_, NT = NT_;
  static constexpr bool STAGED = STAGED_;
  static constexpr int ROWS = NL == 2 ? 16 : 32;  // rows of each layer per CTA
  static constexpr int W_BYTES = 32 * 128 * CPS / 2;  // both tiles' words of a stage
  static constexpr int X_BYTES = 8 * NT * 128;        // the tokens' codes of one chunk
  // a stage's scales: 32 rows' (pitch odd in 16-byte units, so that the reads of
  // eight rows are free of conflicts), their zero points, the tokens'
  static constexpr int NREG = 4 / RJ;                 // regions of a chunk
  static constexpr int SP = 4 * CPS * NREG + 16, ZP = CPS * NREG, XSP = 4 * CPS;
  static constexpr int SCALES_AT = W_BYTES + CPS * X_BYTES;
  static constexpr int STAGE_BYTES =
      (SCALES_AT + (STAGED ? 32 * SP + 32 * ZP + 8 * NT * XSP : 0) + 1023) / 1024 * 1024;
  static constexpr int MINB = 2;
  static constexpr int RED_BYTES = WARPS * NT * 32 * 16;  // the warps' sums of one 16-row tile
  static constexpr int S = (228 * 1024 / MINB - 1024 - RED_BYTES - 1280) / STAGE_BYTES;
  static constexpr int SMEM = S * STAGE_BYTES + RED_BYTES + 2 * S * 8 + 16 + 1024 /* alignment */;
  static_assert(S >= 2, "stages");
  static_assert((SMEM + 1024) * MINB <= 228 * 1024, "shared memory");
};

struct Launch {
  Params p;
  uint64_t wait_ns;
  int tiles;  // blocks of ROWS rows
  int whole;  // the tokens' map is 3-D: columns of a chunk, chunks, tokens
  int stall;  // a STALL_* (0 in normal use)
};

template <class C>
__global__ void __launch_bounds__(THREADS, C::MINB)
w4a8_rows_kernel(const __grid_constant__ CUtensorMap tmap_w0,
                 const __grid_constant__ CUtensorMap tmap_w1,
                 const __grid_constant__ CUtensorMap tmap_x, const Launch a) {
  constexpr int NL = C::NL, RJ = C::RJ, NT = C::NT, S = C::S, ROWS = C::ROWS;
  constexpr int NREG = 4 / RJ;
  const Params& p = a.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (ring - raw);
  float* red = reinterpret_cast<float*>(base + S * C::STAGE_BYTES);  // [warp][NT][32][4]
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + S * C::STAGE_BYTES + C::RED_BYTES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 2 * S);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, C::STAGED ? 33 : 1);  // the copies, and the producer's lanes'
      mbar_init(empty0 + 8u * s, WARPS + (a.stall == STALL_STAGES));
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmap_w0);
    if (NL == 2) tma_prefetch_desc(&tmap_w1);
    tma_prefetch_desc(&tmap_x);
  }
  // what follows on the stream may be launched, to wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __syncthreads();

  const int nchunks = (p.d_col + 127) >> 7;
  const int stages = (nchunks + CPS - 1) / CPS;
  const int ntok = static_cast<int>(p.n);
  const int g = lane >> 2, t = lane & 3;
  bool ok = true;
  uint32_t st = 0, ph = 0;

  if (warp == WARPS) {
    // ------------------------------------------------------------ producer
    uint32_t issued = 0;
    for (int tile = blockIdx.x; tile < a.tiles && ok && a.stall != STALL_LOADS; tile += gridDim.x) {
      const int row0 = tile * ROWS;
      for (int s = 0; s < stages; ++s) {
        ok = mbar_wait_bounded(empty0 + 8u * st, ph ^ 1u, abort_flag, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t fb = full0 + 8u * st, at = ring + st * C::STAGE_BYTES;
        const int c0 = s * CPS, nc = min(CPS, nchunks - c0), pairs = (nc + 1) / 2;
        if (lane == 0)
          mbar_arrive_expect_tx(fb, pairs * 4096 + (a.whole ? CPS : nc) * ntok * 128);
        __syncwarp();
        if (lane < pairs) {  // 32 rows of 128 B each, at 4 KB
          const int x = (c0 / 2 + lane) * 128;
          tma_load_2d(at + lane * 4096, &tmap_w0, fb, x, row0);
          if (NL == 2) tma_load_2d(at + lane * 4096 + 2048, &tmap_w1, fb, x, row0);
        }
        if (a.whole) {  // [token][chunk][128 B]
          if (lane == 8) tma_load_3d(at + C::W_BYTES, &tmap_x, fb, 0, c0, 0);
        } else if (lane >= 8 && lane < 8 + nc) {  // [chunk][token][128 B]
          tma_load_2d(at + C::W_BYTES + (lane - 8) * C::X_BYTES, &tmap_x, fb, (c0 + lane - 8) * 128, 0);
        }
        if (C::STAGED) {  // a lane a row, and a token; groups are counted in fours
          uint8_t* to = base + st * C::STAGE_BYTES + C::SCALES_AT;
          const int row = min(row0 + (NL == 2 ? lane & 15 : lane), p.d_row - 1);
          const Layer& L = p.layer[NL == 2 ? lane >> 4 : 0];
          const size_t first = static_cast<size_t>(row) * p.n_groups;
          const int g0 = c0 * NREG;
#pragma unroll
          for (int j = 0; j < CPS * NREG; j += 4)
            if (g0 + j < p.n_groups) {
              copy_async<16>(to + lane * C::SP + 4 * j, L.scales + first + g0 + j);
              copy_async<4>(to + 32 * C::SP + lane * C::ZP + j, L.zeros + first + g0 + j);
            }
          if (lane < ntok) {
            uint8_t* xt = to + 32 * (C::SP + C::ZP) + lane * C::XSP;
            const float* from = p.xs + static_cast<int64_t>(lane) * p.xgroups;
            if (p.xgroups == 1) copy_async<4>(xt, from);
            else
#pragma unroll
              for (int j = 0; j < CPS; j += 4)
                if (c0 + j < p.xgroups) copy_async<16>(xt + 4 * j, from + c0 + j);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(fb) : "memory");
        }
        __syncwarp();
        ++issued;
        if (++st == S) { st = 0; ph ^= 1u; }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // No copy may land in memory that is handed on.  Usually all have been read;
    // not so where this warp or a reader, at its own time, gave up.
    if (lane == 0) {
      int own = 0;
      for (uint32_t k = 0; k < S && k < issued; ++k) {
        const uint32_t i = issued - 1 - k;
        mbar_wait_bounded(full0 + 8u * (i % S), (i / S) & 1u, &own, a.wait_ns);
      }
    }
  } else {
    // ------------------------------------------------------------- compute
    float acc[2][NT][4];
    const float* sp[2][2];
    const uint8_t* zp[2][2];
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
      const int row0 = tile * ROWS;
      // rows past the layer take its last row's scales and are never written
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = min(row0 + (NL == 2 ? 0 : 16 * i) + g + 8 * h, p.d_row - 1);
          const Layer& L = p.layer[NL == 2 ? i : 0];
          sp[i][h] = L.scales + static_cast<size_t>(row) * p.n_groups;
          zp[i][h] = L.zeros + static_cast<size_t>(row) * p.n_groups;
        }
      struct Scales {
        float sx[NT][2], s[2][2][NREG];
        uint32_t z[2][2][NREG];
      };
      auto load = [&](int c, Scales& k) {
        const int cx = p.xgroups == 1 ? 0 : min(c, nchunks - 1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            k.sx[n][e] = __ldg(p.xs + static_cast<int64_t>(min(8 * n + 2 * t + e, ntok - 1)) * p.xgroups + cx);
#pragma unroll
        for (int m = 0; m < NREG; ++m) {
          const int gi =
              min(static_cast<int>(__umulhi(128 * c + 32 * RJ * m, p.gmagic)), p.n_groups - 1);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              k.s[i][h][m] = __ldg(sp[i][h] + gi);
              k.z[i][h][m] = __ldg(zp[i][h] + gi);
            }
        }
      };
      // One chunk; with whole chunks the scales of the warp's next one are on
      // the way meanwhile, into registers of their own: a copy would wait.
      auto chunk = [&](int c, int slot, Scales& k, Scales& knext) {
        if (!C::STAGED) {
          if (RJ == 4) load(c + WARPS, knext);
          else load(c, k);
        }
        if (__all_sync(0xffffffffu, ok) && c < nchunks) {
          if (C::STAGED) {
            const uint8_t* from = base + st * C::STAGE_BYTES + C::SCALES_AT;
#pragma unroll
            for (int m = 0; m < NREG; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int r = g + 8 * h + 16 * i, e = slot * NREG + m;
                  k.s[i][h][m] = *reinterpret_cast<const float*>(from + r * C::SP + 4 * e);
                  k.z[i][h][m] = from[32 * C::SP + r * C::ZP + e];
                }
            const float* xf = reinterpret_cast<const float*>(from + 32 * (C::SP + C::ZP)) +
                              (p.xgroups == 1 ? 0 : slot);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) k.sx[n][e] = xf[min(8 * n + 2 * t + e, ntok - 1) * CPS];
          }
          // 128-byte swizzle: 16-byte piece q of row r lies at q ^ (r & 7)
          const uint8_t* wt = base + st * C::STAGE_BYTES + (slot >> 1) * 4096 + g * 128;
          const int q0 = 4 * (slot & 1);
          const uint8_t* xt = base + st * C::STAGE_BYTES + C::W_BYTES +
                              (a.whole ? g * (CPS * 128) + slot * 128 : slot * C::X_BYTES + g * 128);
          const int xg = a.whole ? 8 * CPS * 128 : 1024, xr = a.whole ? slot & 7 : g;
          uint32_t w[2][2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* from = wt + (16 * i + 8 * h) * 128;
              if (RJ == 4) {  // words 4 t .. 4 t + 3: the k order inside a chunk is free
                const uint4 v = *reinterpret_cast<const uint4*>(from + (((q0 + t) ^ g) << 4));
                w[i][h][0] = v.x; w[i][h][1] = v.y; w[i][h][2] = v.z; w[i][h][3] = v.w;
              } else {  // word 4 j + t
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[i][h][j] = *reinterpret_cast<const uint32_t*>(from + (((q0 + j) ^ g) << 4) + 4 * t);
              }
            }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint2 x[4];  // the activations of the lane's words
            const uint8_t* from = xt + n * xg;
            if (RJ == 4) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(from + (((2 * t + j) ^ xr) << 4));
                x[2 * j] = make_uint2(v.x, v.y);
                x[2 * j + 1] = make_uint2(v.z, v.w);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[j] = *reinterpret_cast<const uint2*>(from + (((2 * j + (t >> 1)) ^ xr) << 4) + 8 * (t & 1));
            }
            uint32_t b0[4], b1[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              b0[j] = __byte_perm(x[j].x, x[j].y, 0x6420);
              b1[j] = __byte_perm(x[j].x, x[j].y, 0x7531);
            }
#pragma unroll
            for (int m = 0; m < NREG; ++m) {
              int sums[4] = {0, 0, 0, 0};
#pragma unroll
              for (int j = RJ * m; j < RJ * m + RJ; ++j)
                mma_u8s8(sums, 0x01010101u, 0x01010101u, 0x01010101u, 0x01010101u, b0[j], b1[j]);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                int prod[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = RJ * m; j < RJ * m + RJ; ++j)
                  mma_u8s8(prod, even_codes(w[i][0][j]), even_codes(w[i][1][j]), odd_codes(w[i][0][j]),
                           odd_codes(w[i][1][j]), b0[j], b1[j]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  acc[i][n][e] = fmaf(k.s[i][e >> 1][m] * k.sx[n][e & 1],
                                      static_cast<float>(prod[e] - static_cast<int>(k.z[i][e >> 1][m]) * sums[e]),
                                      acc[i][n][e]);
              }
            }
          }
        }
      };
      auto stage = [&](int s, Scales& k, Scales& knext) {
        if (s >= stages) return;
        ok = ok && mbar_wait_bounded(full0 + 8u * st, ph, abort_flag, a.wait_ns);
        chunk(s * CPS + warp, warp, k, knext);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(empty0 + 8u * st);
        if (++st == S) { st = 0; ph ^= 1u; }
      };
      Scales k0, k1;
      if (RJ == 4 && !C::STAGED) load(warp, k0);
      for (int s = 0; s < stages; s += 2) {
        stage(s, k0, k1);
        stage(s + 1, k1, k0);
      }

      // The sums over the warps, one 16-row tile at a time; a thread gets the
      // outputs tid, tid + 256, ... of 16 rows x 8 NT tokens.  Element e of lane
      // l of a fragment is row (l >> 2) + 8 (e >> 1) of its tile, token
      // 2 (l & 3) + (e & 1) of its group of eight.
      constexpr int OUTS = (16 * 8 * NT + 32 * WARPS - 1) / (32 * WARPS);
      float v[2][OUTS];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        named_bar(1, 32 * WARPS);  // the last sums have been read
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float4*>(red + ((warp * NT + n) * 32 + lane) * 4) =
              make_float4(acc[i][n][0], acc[i][n][1], acc[i][n][2], acc[i][n][3]);
        named_bar(1, 32 * WARPS);
#pragma unroll
        for (int j = 0; j < OUTS; ++j) {
          const int o = threadIdx.x + j * 32 * WARPS, rl = o & 15, tk = o >> 4;
          v[i][j] = 0.0f;
          if (tk < ntok)
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
              v[i][j] += red[((w * NT + (tk >> 3)) * 32 + (rl & 7) * 4 + ((tk & 7) >> 1)) * 4 +
                             2 * (rl >> 3) + (tk & 1)];
        }
      }
#pragma unroll
      for (int j = 0; j < OUTS; ++j) {
        const int o = threadIdx.x + j * 32 * WARPS, row = row0 + (o & 15), tk = o >> 4;
        if (tk >= ntok) continue;
        if (NL == 2) {
          if (row < p.d_row) store_out(p, tk * p.ldy + row, silu_times(v[0][j], v[1][j]));
        } else {
          if (row < p.d_row) store_out(p, tk * p.ldy + row, v[0][j]);
          if (row + 16 < p.d_row) store_out(p, tk * p.ldy + row + 16, v[1][j]);
        }
      }
    }
  }
}

// The 8-bit form of fp32 rows, a warp a token and block of 128 columns.  It
// stands behind the row kernel on the stream, whose CTAs hold 16 rows of a
// block each: clusters of eight that exchange their maxima have to lie within a
// GPC, where 33 fit on the GPU instead of 37 and a ninth of the places stays empty
// (with them one token through a gated pair of 22016 x 8192 took 61 us, without 44).
__global__ void __launch_bounds__(128) quant8_rows_kernel(const float* __restrict__ h, int64_t ldh,
                                                          int n, int d, int8_t* codes, int64_t ldq,
                                                          float* scales) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int blocks = (d + 127) / 128;
  const int lane = threadIdx.x & 31;
  const int at = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (at >= blocks * n) return;
  const int tk = at / blocks, col = (at % blocks) * 128 + 4 * lane;
  const float4 f = *reinterpret_cast<const float4*>(h + tk * ldh + col);  // rows are whole blocks
  const float v[4] = {f.x, f.y, f.z, f.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < d) top = max(top, act8::abs_bits(v[i]));
  const act8::Quant q = act8::quant_of(__reduce_max_sync(0xffffffffu, top));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col + i < d) codes[tk * ldq + col + i] = static_cast<int8_t>(act8::code_or_zero(v[i], q));
  if (lane == 0) scales[at] = q.scale;
}

}  // namespace w4a8
}  // namespace gptq

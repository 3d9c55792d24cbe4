// Products with packed 4-bit layers and 8-bit activations on the 5th-generation
// tensor cores, for more than a few tokens.  The mathematics is that of
// w4a8.cuh; here the zero points are subtracted from the codes on the way into
// shared memory, so a run's sum comes out of one contraction of signed bytes
// (kind::i8, int32 accumulators, exact).
//
// A tile is 128 rows of the layer (of both layers, for the gated pair) by TN
// tokens, the layer's rows on the M side.  Work goes in chunks of 128 columns,
// two to a stage:
//
//   TMA warp      the rows' words (128 B a row and stage) and the tokens' codes
//                 (two times 128 B), 128-byte swizzle, into a ring
//   unpack warps  a thread has a row: words of eight codes -> q - z as signed
//                 bytes in column order, into 128-byte-swizzled operand slots.
//                 Bytes 0x80 + q - z never borrow from their neighbour, so four
//                 codes cost an AND-OR, a subtraction, half of two PRMT, an XOR.
//                 Groups of four warps take the slots in turn
//   MMA warps     one thread issues tcgen05.mma, 32 columns each; a run (32, 64
//                 or 128 columns, or more where no scale changes) starts from
//                 zero in its own TMEM buffer
//   scale warp    row scales, zero points and token scales of the next four
//                 runs, copied to shared memory some sets ahead
//   epilogue      int32 -> fp32, times row scale and token scale, added to fp32
//                 registers while the next runs are in the tensor cores
//
// Every mbarrier wait is bounded, as in the Hessian kernel.
//
// Three shapes (Cfg).  SMALL and MID have one tile a cluster of up to 8 CTAs
// that split the chunks; their sums meet in shared memory of the cluster, in
// rank order, so the result does not vary.  BIG is persistent, without a split.
//
// What bounds it (measured): 4096 tokens through 8192 x 22016 (groups of 128)
// take 1.27 to 1.30 ms, 1.16 PFLOP/s, 0.70 of the bf16 rate that cuBLAS reaches.  The
// MMAs would take 512 clocks a chunk of 128 x 256 outputs; with nothing but
// copies, unpacking and MMAs a chunk takes 860 (one scale a row and a token, whose
// runs are folded once a tile: 0.82 ms), with the epilogue 1970: scaling
// each run's sums costs a conversion, a product and a fused add an output, 2050 of
// the chunk's 6160 warp instructions, with the issue slots 78% taken.  For
// one layer more epilogue warps in groups of their own, and spreading the token
// scales by an MMA with ones and 128-token tiles, were built and were slower.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "w4a8.cuh"

namespace gptq {
namespace w4a8t {

using w4a8::copy_async;
using w4a8::Params;

constexpr int BM = 128;  // layer rows per tile
constexpr int CH = 128;  // columns per chunk
constexpr int PACKED_BYTES = BM * CH;  // a stage's words: two chunks, 128 bytes a row
constexpr int SLOT_BYTES = BM * CH;
constexpr int SUM_PITCH = BM + 4;  // rows of a token's sums: spreads a warp's 8 rows x 4 tokens

// NL: layers; TN: tokens per tile; UW, EW: unpack and epilogue warps; S: ring
// stages; AS: operand slots of one layer and chunk; NS: sets of scales on the
// way or in use; MORE: registers of an epilogue thread.  Four more warps are the
// TMA warp, two MMA warps and the scale warp.
template <int NL_, int TN_, int UW_, int EW_, int S_, int AS_, int NS_, int MORE_, bool BIG_>
struct Cfg {
  static constexpr int NL = NL_, TN = TN_, UW = UW_, EW = EW_, S = S_, AS = AS_, NS = NS_;
  static constexpr bool BIG = BIG_;
  static constexpr int WARPS = UW + EW + 4;
  static constexpr int THREADS = WARPS * 32;
  // TMEM buffers: with 8 two MMA warps take turns at four runs a chunk, too (61
  // tokens, 4096 x 8192 in groups of 32: 29 us against 31 with 4)
  static constexpr int NU = 512 / TN < 8 ? 512 / TN : 8;
  static constexpr int TMEM_COLS = NU * TN < 32 ? 32 : NU * TN;
  static constexpr int NB = NU / NL;                 // of a layer
  static constexpr int COLS = TN / (EW / 4);         // columns (tokens) per epilogue warp
  // While it folds, half of the warps has gate, half has up, twice the columns
  // each, so that two chains of waits run beside each other and the reads of TMEM
  // run ahead (333 tokens, 11008 x 4096 in groups of 32: 245 us, together 336; 60
  // tokens, 22016 x 8192: 151 against 157; 2048 tokens: 1589 against 1620).  With
  // four warps or one layer, crews for every other run were slower (61 tokens, 4096
  // x 11008 in groups of 64: 27.0 us against 26.0).
  static constexpr int CREWS = NL == 2 && EW > 4 ? 2 : 1;
  static constexpr int FCOLS = CREWS * COLS;         // columns that a crew's warp folds
  static constexpr int X_BYTES = TN * CH;
  static constexpr int STAGE_BYTES = NL * PACKED_BYTES + 2 * X_BYTES;
  static constexpr int RING_BYTES = S * STAGE_BYTES;
  static constexpr int SUM_BYTES = BIG ? 0 : NL * TN * SUM_PITCH * 4;  // over the ring, at the end
  static constexpr int SX_BYTES = NS * 4 * TN * 4;       // sets of token scales, four a token
  static constexpr int SW_BYTES = NS * 4 * NL * BM * 4;  // of row scales, four a row
  static constexpr int Z_BYTES = NS * NL * BM * 4;       // of zero points, four in a word
  static constexpr int TOP_BYTES = BIG && NL == 2 ? 4 * TN * 4 : 0;
  static constexpr int TRADE_BYTES = BIG && CREWS == 2 ? EW * 1024 : 0;
  static constexpr int BARS = 2 * S + 2 * AS + 2 * NU + 2 * NS + 2;
  static constexpr int SMEM = RING_BYTES + AS * SLOT_BYTES + SX_BYTES + SW_BYTES + Z_BYTES + TOP_BYTES + TRADE_BYTES +
                              BARS * 8 + 16 + 1024 /* alignment */;
  static_assert(NB >= 1 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "TMEM");
  static_assert(SUM_BYTES <= RING_BYTES + AS * SLOT_BYTES, "the sums lie over the ring");
  // Where two MMA warps (and two groups of unpack warps) take the slots in turn, an
  // odd number of slots hands a slot from one to the other, and a wait by parity
  // takes a barrier that is a whole phase behind for its own.  MMA warps: a warp has
  // waited for the TMEM buffer of its chunk first, which is free when the chunk NB
  // before is folded; folds go in order, so with NB <= AS the slot's chunk before this
  // one is multiplied.  Unpack groups: the stage's words came after the MMAs of the
  // stage S before, and a warp's commit stands for its earlier MMAs, too; with S <= 3
  // those of 2 AS chunks before are among them.
  static_assert(AS % 2 == 0 || (NL == 1 && NB <= AS && AS == 3 && S <= 3), "slots by parity");
  static_assert(EW % 4 == 0 && UW % 4 == 0 && (FCOLS == 32 || FCOLS == 64), "warps");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // one CTA an SM, so no CTA of a cluster waits for TMEM that another holds
  static_assert(2 * SMEM > 228 * 1024, "one CTA");
  // the launch's registers, THREADS x LAUNCH, move between warpgroups
  static constexpr int LAUNCH = 65536 / THREADS / 8 * 8, MORE = MORE_,
                       FEWER = (THREADS * LAUNCH - EW * 32 * MORE) / ((UW + 4) * 32) / 8 * 8;
  static_assert((EW * MORE + (UW + 4) * FEWER) * 32 <= THREADS * LAUNCH && FEWER >= 40, "registers");
};

struct Tiled {
  Params p;
  int row_tiles, tok_tiles;
  int ksplit;        // CTAs of a cluster along the columns
  int runs;          // runs per chunk: 4 (32 columns), 2, or 1
  int yvec;          // eight rows of an output are aligned for one store
  int xvec, wvec;    // rows of token scales, and of row scales and zero points, allow vector loads
  uint64_t wait_ns;
  int stall;         // a w4a8::STALL_* (0 in normal use)
};

__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Four signed bytes q - z of one word's even or odd codes, still biased by 128.
__device__ __forceinline__ uint32_t biased(uint32_t codes, uint32_t z4) {
  return ((codes & 0x0F0F0F0Fu) | 0x80808080u) - z4;
}

// Eight codes of a word -> eight signed bytes in column order.
__device__ __forceinline__ uint2 unpack_word(uint32_t w, uint32_t z4) {
  const uint32_t lo = biased(w, z4), hi = biased(w >> 4, z4);
  return make_uint2(__byte_perm(lo, hi, 0x5140) ^ 0x80808080u,
                    __byte_perm(lo, hi, 0x7362) ^ 0x80808080u);
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 lanes x 32 columns of TMEM: register 4 b + 2 i + e of lane t has
// row t / 4 + 8 i, column 8 b + 2 (t % 4) + e.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// A thread's share of 32 rows x COLS tokens: rows lane / 4 + 8 i + 16 h, and
// of each eight tokens two: v[(h COLS / 8 + b) 2 + i] has the tokens 8 b +
// 2 (lane % 4) + {0, 1} of row (h, i).  With four rows a thread needs a quarter
// of the tokens' scales: one row a thread and all tokens read 128 B a warp and
// value from shared memory, 620 clocks a chunk of 128 x 256 outputs.
template <int COLS>
struct Share {
  uint64_t v[COLS / 2];
  __device__ __forceinline__ float at(int b, int h, int i, int e) const {
    const float2 f = unpack2(v[(h * (COLS / 8) + b) * 2 + i]);
    return e ? f.y : f.x;
  }
};

// Transpose 8 values of the 8 lanes with one lane % 4: lane / 4 = j gets value
// j of each, in the order of the lanes.
__device__ __forceinline__ void transpose8(float (&v)[8]) {
  const int j = (threadIdx.x >> 2) & 7;
#pragma unroll
  for (int s = 1; s < 8; s <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & s)) {
        const bool up = j & s;
        const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i | s], s << 2);
        if (up) v[i] = got;
        else v[i | s] = got;
      }
}

// Eight consecutive rows of a token, `left` of them inside the layer; vec: 16-
// byte (8-bit codes: 8-byte) stores are aligned.
__device__ __forceinline__ void store_rows8(const Params& p, int64_t at, const float (&v)[8],
                                            int left, bool vec, const act8::Quant& q) {
  if (vec && left >= 8) {
    if (p.out == w4a8::OUT_I8) {
      *reinterpret_cast<uint2*>(static_cast<int8_t*>(p.y) + at) = act8::codes8(v, q);
    } else if (p.out == w4a8::OUT_BF16) {
      float w[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
      act8::store8(static_cast<__nv_bfloat16*>(p.y) + at, w);
    } else {
      float w[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
      act8::store8(static_cast<float*>(p.y) + at, w);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= left) break;
    if (p.out == w4a8::OUT_I8)
      static_cast<int8_t*>(p.y)[at + i] = static_cast<int8_t>(act8::code_or_zero(v[i], q));
    else
      w4a8::store_out(p, at + i, v[i]);
  }
}

// 16 lanes x 16 columns: the same with two groups of eight columns.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// One run's sums, scaled and added; t0: the warp's lanes and first column in
// TMEM, sw: its four rows' scales, sx: the first token's scale; `read` is called
// when the last sums are in registers and the buffer may be written again (4096
// tokens, 8192 x 22016: 1340 us, against 1420 with the buffer kept to the end).
// TMEM is read in pieces of 16 lanes.  A warp of 64 tokens reads 16 columns at a
// time with the next piece on the way while it folds one (1295 us); one of 32
// tokens has few pieces and is faster with 32 columns at a time (61 tokens, 8192 x
// 8192 in groups of 32: 51.8 us against 53.0).  The conversion
// to fp32 is an instruction of half the adders' rate; the add of 1.5 * 2^23 and
// its subtraction would cost as much and more issue slots.
template <int COLS, class Read>
__device__ __forceinline__ void fold_run(Share<COLS>& acc, uint32_t t0, const float (&sw)[4],
                                         const float* sx, Read read) {
  const float* sxt = sx + 8 * (threadIdx.x & 3);  // four a token
  constexpr bool AHEAD = COLS == 64;
  constexpr int W = AHEAD ? 16 : 32, N = 2 * COLS / W;  // piece k: columns W (k / 2), lanes 16 (k % 2)
  uint32_t v[AHEAD ? 2 : 1][W / 2];
  uint64_t s[W / 8];
  auto load = [&](int k) {
    tmem_ld_16x256b(t0 + (static_cast<uint32_t>(16 * (k & 1)) << 16) + W * (k >> 1), v[AHEAD ? k & 1 : 0]);
  };
  if (AHEAD) load(0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int h = k & 1, c = W * (k >> 1);
    if (!AHEAD) load(k);
    if (h == 0)
#pragma unroll
      for (int b = 0; b < W / 8; ++b) s[b] = pack2(sxt[4 * (c + 8 * b)], sxt[4 * (c + 8 * b) + 4]);
    tmem_ld_wait();
    if (k == N - 1) read();
    else if (AHEAD) load(k + 1);
    const uint32_t(&w)[W / 2] = v[AHEAD ? k & 1 : 0];
#pragma unroll
    for (int b = 0; b < W / 8; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t f = pack2(__int2float_rn(static_cast<int>(w[4 * b + 2 * i])),
                                 __int2float_rn(static_cast<int>(w[4 * b + 2 * i + 1])));
        uint64_t& o = acc.v[(h * (COLS / 8) + c / 8 + b) * 2 + i];
        o = fma2(f, mul2(pack2(sw[2 * h + i], sw[2 * h + i]), s[b]), o);
      }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
w4a8_tiled_kernel(const __grid_constant__ CUtensorMap tmap_w0,
                  const __grid_constant__ CUtensorMap tmap_w1,
                  const __grid_constant__ CUtensorMap tmap_x, const Tiled a) {
  constexpr int NL = C::NL, TN = C::TN, S = C::S, AS = C::AS, NU = C::NU, NB = C::NB, NS = C::NS, EW = C::EW,
                UW = C::UW;
  constexpr uint32_t IDESC = (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(TN >> 3) << 17) |
                             (uint32_t(BM >> 4) << 24);  // s32 += s8 x s8, both K-major
  namespace cg = cooperative_groups;
  const Params& p = a.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (ring - raw);
  const uint32_t slots = ring + C::RING_BYTES;
  float* sx = reinterpret_cast<float*>(base + C::RING_BYTES + AS * SLOT_BYTES);
  float* swb = sx + C::SX_BYTES / 4;
  uint32_t* zb = reinterpret_cast<uint32_t*>(swb + C::SW_BYTES / 4);
  uint32_t* tops = zb + C::Z_BYTES / 4;
  uint64_t* trade = reinterpret_cast<uint64_t*>(tops + C::TOP_BYTES / 4);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(tops) + C::TOP_BYTES + C::TRADE_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * S, afull0 = empty0 + 8u * S,
                 aempty0 = afull0 + 8u * AS, tfull0 = aempty0 + 8u * AS,
                 tempty0 = tfull0 + 8u * NU, sfull0 = tempty0 + 8u * NU, sempty0 = sfull0 + 8u * C::NS,
                 drain = sempty0 + 8u * C::NS;

  // Each chunk's last run closes its TMEM buffer, or runs span chunks.  Where
  // they close, two MMA warps take the operand slots in turn, provided that
  // they use different buffers (their waits tell phases by parity alone):
  // each layer has its own.  For the slots themselves see Cfg.
  const bool every = p.xgroups != 1 || a.runs != 1 || p.group == CH;
  const bool turns = every && (NL == 2 || NU % (2 * a.runs) == 0);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool leader = elect_one();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 8 * NL + (turns ? 2 : 1) +  // unpacked, and multiplied
                                     (a.stall == w4a8::STALL_STAGES));
    }
    for (int s = 0; s < AS; ++s) {
      mbar_init(afull0 + 8u * s, 4);
      mbar_init(aempty0 + 8u * s, 1);
    }
    for (int u = 0; u < NU; ++u) {
      mbar_init(tfull0 + 8u * u, 1);
      mbar_init(tempty0 + 8u * u, EW / C::CREWS);
    }
    for (int u = 0; u < C::NS; ++u) {
      mbar_init(sfull0 + 8u * u, 64);  // the scale warp's lanes and their copies
      mbar_init(sempty0 + 8u * u, UW + EW);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 8u, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tmap_w0);
    if (NL == 2) tma_prefetch_desc(&tmap_w1);
    tma_prefetch_desc(&tmap_x);
  }
  if (warp == UW + EW + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int nchunks = (p.d_col + CH - 1) / CH;
  const int krank = C::BIG ? 0 : static_cast<int>(blockIdx.x) % a.ksplit;
  // shares of whole fours of chunks, so that sets of scales start aligned
  const int quads = (nchunks + 3) / 4;
  const int c0 = 4 * (quads * krank / a.ksplit);
  // an odd last chunk makes a pair with one of zeros, which the copies fill in
  const int c1 = min((nchunks + 1) / 2 * 2, 4 * (quads * (krank + 1) / a.ksplit));
  const int64_t tiles = static_cast<int64_t>(a.row_tiles) * a.tok_tiles;
  const int64_t tile0 = C::BIG ? blockIdx.x : blockIdx.x / a.ksplit;
  const int64_t tile_step = C::BIG ? gridDim.x : tiles;
  // a chunk's last run closes its TMEM buffer unless neither scale changes
  auto group_of = [&](int col) {
    return min(static_cast<int>(__umulhi(static_cast<uint32_t>(col), p.gmagic)), p.n_groups - 1);
  };
  auto closes = [&](int c) {
    return every || c == c1 - 1 || group_of((c + 1) * CH) != group_of(c * CH);
  };
  bool ok = true;
#define W4T_WAIT(bar, par) \
  (ok = ok && mbar_wait_bounded((bar), (par), abort_flag, a.wait_ns))
// The same with one answer for the warp, whose lanes leave loops by it and meet
// again inside them: where one lane gave up and another's wait came through, those
// that stay would wait for those that left.  (The other roles keep looping.)
#define W4T_WAIT_ALL(bar, par) \
  (ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded((bar), (par), abort_flag, a.wait_ns)))

#define W4T_FEWER() \
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::FEWER))
#define W4T_MORE() \
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::MORE))

  if (warp >= UW + EW) {
    W4T_FEWER();  // the whole warpgroup, at one place
    if (warp == UW + EW) {
      // ------------------------------------------------------------ TMA warp
      // The warp stays together and one thread issues, here and below.
      uint32_t st = 0, ph = 0, issued = 0;
      for (int64_t t = tile0; t < tiles && ok && a.stall != w4a8::STALL_LOADS; t += tile_step) {
        const int row = static_cast<int>(t / a.tok_tiles) * BM;
        const int tok = static_cast<int>(t % a.tok_tiles) * TN;
        for (int c = c0; c < c1; c += 2) {
          if (!W4T_WAIT_ALL(empty0 + 8u * st, ph ^ 1u)) break;
          const uint32_t fb = full0 + 8u * st, at = ring + st * C::STAGE_BYTES;
          if (leader) {
            mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
            tma_load_2d(at, &tmap_w0, fb, c * (CH / 2), row);
            if (NL == 2) tma_load_2d(at + PACKED_BYTES, &tmap_w1, fb, c * (CH / 2), row);
            tma_load_2d(at + NL * PACKED_BYTES, &tmap_x, fb, c * CH, tok);
            tma_load_2d(at + NL * PACKED_BYTES + C::X_BYTES, &tmap_x, fb, (c + 1) * CH, tok);
            ++issued;
          }
          __syncwarp();
          if (++st == S) { st = 0; ph ^= 1u; }
        }
      }
      // No copy may land in memory that is handed on.  Usually all have been read;
      // not so where this role or a reader, at its own time, gave up.
      if (leader) {
        int own = 0;
        for (uint32_t k = 0; k < S && k < issued; ++k) {
          const uint32_t i = issued - 1 - k;
          mbar_wait_bounded(full0 + 8u * (i % S), (i / S) & 1u, &own, a.wait_ns);
        }
      }
    } else if (warp <= UW + EW + 2) {
      // ----------------------------------------------------------- MMA warps
      const uint32_t mw = warp - (UW + EW + 1);
      const uint64_t DESC = smem_desc_sw128(0, 16, 1024);  // addresses are added
      uint32_t st = 0, k = 0, unit = 0;  // stage, slots and a layer's TMEM buffers so far
      bool open = false;                 // the current buffers hold a started run
      for (int64_t t = tile0; t < tiles && ok; t += tile_step) {
        for (int c = c0; c < c1 && ok; ++c) {
          const bool close = closes(c);
          // The tokens' codes came with the words that the unpack warps waited
          // for, so their arrival stands for both.
          const uint64_t xd = DESC + ((ring + st * C::STAGE_BYTES + NL * PACKED_BYTES +
                                       (c & 1) * C::X_BYTES) >> 4);
#pragma unroll
          for (int l = 0; l < NL; ++l, ++k) {
            if (turns ? (k & 1u) != mw : mw != 0) continue;
            const uint32_t slot = k % AS;
            const uint64_t ad = DESC + ((slots + slot * SLOT_BYTES) >> 4);
            // An even number of slots: a warp sees its slots' every phase, and waits here
            // (before the buffer; 2048 tokens gated, 22016 x 8192: 1608 us, after it
            // 1648).  Odd: the slot's parity means nothing before the buffer is free.
            if constexpr (AS % 2 == 0) W4T_WAIT_ALL(afull0 + 8u * slot, (k / AS) & 1u);
            // 32 columns are 32 bytes: 2 units of a descriptor's address
            if (a.runs == 1) {
              const uint32_t buf = l * NB + unit % NB, d = tmem_base + buf * TN;
              if (!open) W4T_WAIT_ALL(tempty0 + 8u * buf, ((unit / NB) & 1u) ^ 1u);
              if constexpr (AS % 2 != 0) W4T_WAIT_ALL(afull0 + 8u * slot, (k / AS) & 1u);
              tc_fence_after();
              if (ok && leader) {
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_i8_ss(d, ad + 2 * i, xd + 2 * i, IDESC, i != 0 || open);
                if (close) mma_commit(tfull0 + 8u * buf);
              }
            } else {
              if constexpr (AS % 2 != 0) W4T_WAIT_ALL(afull0 + 8u * slot, (k / AS) & 1u);
              for (int m = 0; m < a.runs; ++m) {
                const uint32_t u = unit + m, buf = l * NB + u % NB, d = tmem_base + buf * TN;
                W4T_WAIT_ALL(tempty0 + 8u * buf, ((u / NB) & 1u) ^ 1u);
                tc_fence_after();
                if (ok && leader) {
                  if (a.runs == 2) {
                    mma_i8_ss(d, ad + 4 * m, xd + 4 * m, IDESC, 0);
                    mma_i8_ss(d, ad + 4 * m + 2, xd + 4 * m + 2, IDESC, 1);
                  } else {
                    mma_i8_ss(d, ad + 2 * m, xd + 2 * m, IDESC, 0);
                  }
                  mma_commit(tfull0 + 8u * buf);
                }
              }
            }
            if (ok && leader) {
              mma_commit(aempty0 + 8u * slot);
              // after the warp's last slot of the stage
              if (turns ? NL == 1 || (c & 1) : (c & 1) && l == NL - 1) mma_commit(empty0 + 8u * st);
            }
            __syncwarp();
          }
          if ((c & 1) && ++st == S) st = 0;
          open = !close;
          if (close) unit += a.runs;
        }
      }
      // The tensor cores are done before TMEM and the operands' memory are freed,
      // whichever role gave up.
      if (leader) {
        int own = 0;
        mma_commit(drain + 8u * mw);
        mbar_wait_bounded(drain + 8u * mw, 0, &own, a.wait_ns);
      }
    } else {
      // ---------------------------------------------------------- scale warp
      // The scales and zero points of the next runs, in sets of four runs (4,
      // 2 or 1 chunks), and those chunks' token scales: a lane copies a row's
      // or token's four at once where they lie in 16 aligned bytes, straight
      // to shared memory and NS sets ahead, as row scales come from HBM.  (One
      // value at a time and line took more of the load unit than all else, 640
      // clocks a chunk of 128 x 256 outputs.)
      const int per_set = 4 / a.runs, step = CH / a.runs;
      uint32_t set = 0;
      for (int64_t t = tile0; t < tiles; t += tile_step) {
        const int row0 = static_cast<int>(t / a.tok_tiles) * BM;
        const int64_t tok0 = (t % a.tok_tiles) * TN;
        for (int cs = c0; cs < c1; cs += per_set, ++set) {
          const uint32_t at = set % NS;
          const int g[4] = {group_of(cs * CH), group_of(cs * CH + step), group_of(cs * CH + 2 * step),
                            group_of(cs * CH + 3 * step)};
          const bool xvec = a.xvec && (cs & 3) == 0 && cs + 4 <= p.xgroups;
          const bool wvec = a.wvec && (g[0] & 3) == 0 && g[3] == g[0] + 3;
          W4T_WAIT(sempty0 + 8u * at, ((set / NS) & 1u) ^ 1u);
          if (!ok) continue;
#pragma unroll 1
          for (int r = lane; r < TN; r += 32) {
            const float* from = p.xs + min(tok0 + r, p.n - 1) * p.xgroups;
            float* to = sx + (at * TN + r) * 4;
            if (xvec) {
              copy_async<16>(to, from + cs);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                copy_async<4>(to + j, from + (p.xgroups == 1 ? 0 : min(cs + j, nchunks - 1)));
            }
          }
#pragma unroll
          for (int l = 0; l < NL; ++l) {
            uint32_t z[BM / 32][4];
#pragma unroll
            for (int i = 0; i < BM / 32; ++i) {
              const int r = lane + 32 * i;
              const size_t first = static_cast<size_t>(min(row0 + r, p.d_row - 1)) * p.n_groups;
              const float* sf = p.layer[l].scales + first;
              const uint8_t* zf = p.layer[l].zeros + first;
              float* to = swb + ((at * NL + l) * BM + r) * 4;
              if (wvec) {
                copy_async<16>(to, sf + g[0]);
                copy_async<4>(zb + (at * NL + l) * BM + r, zf + g[0]);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  copy_async<4>(to + j, sf + g[j]);
                  z[i][j] = __ldg(zf + g[j]);
                }
              }
            }
            if (!wvec)
#pragma unroll
              for (int i = 0; i < BM / 32; ++i)
                zb[(at * NL + l) * BM + lane + 32 * i] =
                    z[i][0] | (z[i][1] << 8) | (z[i][2] << 16) | (z[i][3] << 24);
          }
          // the copies arrive when they are done, the lane for its own stores
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sfull0 + 8u * at)
                       : "memory");
          mbar_arrive(sfull0 + 8u * at);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp < UW) {
    // -------------------------------------------------------------- unpack
    W4T_FEWER();
    // Groups of four warps take the operand slots (a chunk of one layer) in
    // turn: a slot's way from barrier to barrier is a chain of latencies, and
    // one group at it was the pace of the whole kernel.
    constexpr uint32_t UG = UW / 4;
    const uint32_t group = warp >> 2;
    const int r = threadIdx.x & (BM - 1);  // row of the tile
    const uint32_t in_row = r * 128, out_row = r * 128;
    uint32_t k = 0, kc = 0, set = 0;  // slots, chunks and sets so far
    const int per_set = 4 / a.runs;
    for (int64_t t = tile0; t < tiles; t += tile_step) {
      for (int cs = c0; cs < c1; cs += per_set, ++set) {
        const uint32_t at = set % NS;
        W4T_WAIT(sfull0 + 8u * at, (set / NS) & 1u);
        uint32_t z[NL];  // four zero points of the row
#pragma unroll
        for (int l = 0; l < NL; ++l) z[l] = zb[(at * NL + l) * BM + r];
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(sempty0 + 8u * at);
        const int ce = min(cs + per_set, c1);
#pragma unroll 1
        for (int c = cs; c < ce; ++c, ++kc) {
          const uint32_t st = (kc >> 1) % S;
#pragma unroll
          for (int l = 0; l < NL; ++l, ++k) {
            if (k % UG != group) continue;
            const uint32_t slot = k % AS;
            W4T_WAIT(full0 + 8u * st, ((kc >> 1) / S) & 1u);
            const uint8_t* in = base + st * C::STAGE_BYTES + l * PACKED_BYTES + in_row;
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = *reinterpret_cast<const uint4*>(in + (((4 * (c & 1) + i) ^ (r & 7)) << 4));
            const uint32_t first = (c - cs) * a.runs;  // the chunk's first run in the set
            W4T_WAIT(aempty0 + 8u * slot, ((k / AS) & 1u) ^ 1u);
            uint8_t* out = base + C::RING_BYTES + slot * SLOT_BYTES + out_row;
            if (ok) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t zi = __byte_perm(z[l], 0, (first + (i * a.runs >> 2)) * 0x1111);
                const uint2 b0 = unpack_word(w[i].x, zi), b1 = unpack_word(w[i].y, zi);
                const uint2 b2 = unpack_word(w[i].z, zi), b3 = unpack_word(w[i].w, zi);
                *reinterpret_cast<uint4*>(out + (((2 * i) ^ (r & 7)) << 4)) =
                    make_uint4(b0.x, b0.y, b1.x, b1.y);
                *reinterpret_cast<uint4*>(out + (((2 * i + 1) ^ (r & 7)) << 4)) =
                    make_uint4(b2.x, b2.y, b3.x, b3.y);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) {
              mbar_arrive(afull0 + 8u * slot);
              mbar_arrive(empty0 + 8u * st);
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    W4T_MORE();
    const int e = threadIdx.x - UW * 32;
    const int quarter = warp & 3, half = (warp - UW) >> 2;  // of the rows, of the columns
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr int COLS = C::COLS;
    // while folding: the columns, and the first layer
    constexpr int FCOLS = C::FCOLS, FL = C::CREWS == 2 ? 1 : NL;
    const int fhalf = half / C::CREWS, mine = half % C::CREWS;
    const int per_set = 4 / a.runs;
    uint32_t unit = 0, set = 0;
    for (int64_t t = tile0; t < tiles; t += tile_step) {
      const int row0 = static_cast<int>(t / a.tok_tiles) * BM;
      const int64_t tok0 = (t % a.tok_tiles) * TN;
      const int row_t = quarter * 32 + (lane >> 2);  // + 8 i + 16 h
      Share<FCOLS> sum[FL];
#pragma unroll
      for (int l = 0; l < FL; ++l)
#pragma unroll
        for (int j = 0; j < FCOLS / 2; ++j) sum[l].v[j] = 0ull;
      for (int cs = c0; cs < c1; cs += per_set, ++set) {
        const uint32_t at = set % NS;
        W4T_WAIT(sfull0 + 8u * at, (set / NS) & 1u);
        const float* sxs = sx + (at * TN + fhalf * FCOLS) * 4;
        const float* sws = swb + ((at * NL + mine) * BM + row_t) * 4;
        const int ce = min(cs + per_set, c1);
#pragma unroll 1
        for (int c = cs; c < ce; ++c, ++sxs) {
          if (!closes(c)) continue;
#pragma unroll 1
          for (int m = 0; m < a.runs; ++m) {
#pragma unroll
            for (int l = 0; l < FL; ++l) {
              const uint32_t u = unit + m, buf = (mine + l) * NB + u % NB;
              const float* from = sws + l * BM * 4 + (c - cs) * a.runs + m;
              const float sw[4] = {from[0], from[32], from[64], from[96]};  // rows + 8 i + 16 h
              W4T_WAIT(tfull0 + 8u * buf, (u / NB) & 1u);
              __syncwarp();  // the loads are the whole warp's, also after a wait that gave up
              tc_fence_after();
              fold_run<FCOLS>(
                  sum[l], tmem_base + lanes + buf * TN + fhalf * FCOLS, sw, sxs, [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(tempty0 + 8u * buf);
                  });
            }
          }
          unit += a.runs;
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(sempty0 + 8u * at);
      }
      const int col_t = 2 * (lane & 3);
      if constexpr (C::BIG) {
        Share<COLS> acc[NL];
        if constexpr (C::CREWS == 2) {
          // Of 2 COLS columns the warp keeps those of its half and gets their other
          // layer's from the warp beside it, which lies in the same lanes, a quarter
          // of its registers at a time.
          uint64_t* to = trade + (warp - UW) * 128 + lane;
          const uint64_t* from = trade + ((warp - UW) ^ 4) * 128 + lane;
          const int bar = 2 + quarter + 4 * fhalf;
#pragma unroll
          for (int c = 0; c < COLS / 8; ++c) {  // eight columns: two registers for each 16 rows
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int low = ((j >> 1) * (FCOLS / 8) + c) * 2 + (j & 1), high = low + COLS / 4;
              to[32 * j] = mine ? sum[0].v[low] : sum[0].v[high];
            }
            named_bar(bar, 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int low = ((j >> 1) * (FCOLS / 8) + c) * 2 + (j & 1), high = low + COLS / 4;
              const int at = ((j >> 1) * (COLS / 8) + c) * 2 + (j & 1);
              const uint64_t own = mine ? sum[0].v[high] : sum[0].v[low], other = from[32 * j];
              acc[0].v[at] = mine ? other : own;
              acc[NL - 1].v[at] = mine ? own : other;
            }
            named_bar(bar, 64);
          }
        } else {
#pragma unroll
          for (int l = 0; l < NL; ++l)
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j) acc[l].v[j] = sum[l].v[j];
        }
        const bool codes = NL == 2 && p.out == w4a8::OUT_I8;
        if (NL == 2) {
#pragma unroll
          for (int j = 0; j < COLS / 2; ++j) {
            const float2 g = unpack2(acc[0].v[j]), u = unpack2(acc[NL - 1].v[j]);
            acc[0].v[j] = pack2(w4a8::silu_times(g.x, u.x), w4a8::silu_times(g.y, u.y));
          }
        }
        if (codes) {
          // maxima over the tile's 128 rows, through shared memory
#pragma unroll
          for (int q = 0; q < COLS / 8; ++q)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              uint32_t top = 0;
#pragma unroll
              for (int hi = 0; hi < 4; ++hi)
                if (row0 + row_t + 8 * hi < p.d_row)
                  top = max(top, act8::abs_bits(acc[0].at(q, hi >> 1, hi & 1, e2)));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              if (lane < 4) tops[quarter * TN + half * COLS + 8 * q + col_t + e2] = top;
            }
          named_bar(1, EW * 32);
          if (e < TN) {  // one thread a token: its scale, and what the rows multiply by
            const act8::Quant q = act8::quant_of(
                max(max(tops[e], tops[TN + e]), max(tops[2 * TN + e], tops[3 * TN + e])));
            tops[e] = __float_as_uint(q.inv);
            tops[TN + e] = __float_as_uint(q.lift);
            if (tok0 + e < p.n) p.ys[(tok0 + e) * ((p.d_row + 127) / 128) + row0 / BM] = q.scale;
          }
          named_bar(1, EW * 32);
        }
        // of each eight tokens the warp's lanes trade rows for (token, rows)
        // pairs: lane j of eight gets token j % 2 of its two, rows 8 (j / 2) ..
        const int j = (lane >> 2) & 7;
        const int64_t row = row0 + quarter * 32 + 8 * (j >> 1);
#pragma unroll
        for (int q = 0; q < COLS / 8; ++q) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = acc[0].at(q, k >> 2, (k >> 1) & 1, k & 1);
          transpose8(v);
          const int col = half * COLS + 8 * q + col_t + (j & 1);
          act8::Quant k{};
          if (codes) {
            k.inv = __uint_as_float(tops[col]);
            k.lift = __uint_as_float(tops[TN + col]);
          }
          if (tok0 + col < p.n)
            store_rows8(p, (tok0 + col) * p.ldy + row, v, static_cast<int>(p.d_row - row), a.yvec, k);
        }
        if (codes) named_bar(1, EW * 32);  // all have read before the next tile's maxima
      } else {
        // the sums, token-major, over the ring: every copy has been consumed
        named_bar(1, EW * 32);
        float* sums = reinterpret_cast<float*>(base);
#pragma unroll
        for (int l = 0; l < FL; ++l)
#pragma unroll
          for (int q = 0; q < FCOLS / 8; ++q)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              float* to =
                  sums + ((mine + l) * TN + fhalf * FCOLS + 8 * q + col_t + e2) * SUM_PITCH + row_t;
#pragma unroll
              for (int hi = 0; hi < 4; ++hi) to[8 * hi] = sum[l].at(q, hi >> 1, hi & 1, e2);
            }
      }
    }
  }
#undef W4T_WAIT
#undef W4T_WAIT_ALL
#undef W4T_FEWER
#undef W4T_MORE

  tc_fence_before();
  __syncthreads();
  if (warp == UW + EW + 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if constexpr (!C::BIG) {
    // The cluster's CTAs each finish a share of the tokens, a warp a token and
    // a lane four rows.  TMEM is free by now: no CTA holds it while it waits.
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    const int row0 = static_cast<int>(tile0 / a.tok_tiles) * BM;
    const int64_t tok0 = (tile0 % a.tok_tiles) * TN;
    const int ntok = static_cast<int>(min(static_cast<int64_t>(TN), p.n - tok0));
    float* sums = reinterpret_cast<float*>(base);
    for (int tk = krank + warp * a.ksplit; tk < ntok; tk += C::WARPS * a.ksplit) {
      float4 v[NL];
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        float* own = sums + (l * TN + tk) * SUM_PITCH + 4 * lane;
        v[l] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < a.ksplit; ++r) {
          const float4 o = *reinterpret_cast<const float4*>(cl.map_shared_rank(own, r));
          v[l].x += o.x; v[l].y += o.y; v[l].z += o.z; v[l].w += o.w;
        }
      }
      float h[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
      if (NL == 2) {
        h[0] = w4a8::silu_times(h[0], v[NL - 1].x);
        h[1] = w4a8::silu_times(h[1], v[NL - 1].y);
        h[2] = w4a8::silu_times(h[2], v[NL - 1].z);
        h[3] = w4a8::silu_times(h[3], v[NL - 1].w);
      }
      const int row = row0 + 4 * lane;
      const int64_t at = (tok0 + tk) * p.ldy + row;
      if (NL == 2 && p.out == w4a8::OUT_I8) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row + i < p.d_row) top = max(top, act8::abs_bits(h[i]));
        const act8::Quant q = act8::quant_of(__reduce_max_sync(0xffffffffu, top));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row + i < p.d_row)
            static_cast<int8_t*>(p.y)[at + i] = static_cast<int8_t>(act8::code_or_zero(h[i], q));
        if (lane == 0) p.ys[(tok0 + tk) * ((p.d_row + 127) / 128) + row0 / BM] = q.scale;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row + i < p.d_row) w4a8::store_out(p, at + i, h[i]);
      }
    }
    cl.sync();  // no CTA leaves while another may still read its sums
  }
}

}  // namespace w4a8t
}  // namespace gptq

// bcq_i8.cu -- the 8-bit integer product: rows to codes, and
//   y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k]   (the sum exact in int32).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "bcq.h"
#include "bcq_device.cuh"
#include "bcq_f32x2.cuh"
#include "bcq_launch.h"
#include "bcq_tcgen05.cuh"

namespace bcq {
namespace {

__device__ int g_i8_error = 0;

// ------------------------------------------------------------------ types

template <typename T>
struct Bits16;  // 16-bit floating types by their bits
template <>
struct Bits16<__half> {
  static constexpr uint32_t kInf = 0x7C00u;
  static __device__ __forceinline__ float to_float(uint32_t b) { return h2f((uint16_t)b); }
};
template <>
struct Bits16<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ float to_float(uint32_t b) { return __uint_as_float(b << 16); }
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ----------------------------------------------------------- rows to codes

// The code of x: 127 x / a to the nearest integer, x times 127 / a first;
// where that lies within 1e-4 of a half (its error is below 127 * 3 * 2^-24 <
// 3e-5) the quotient itself decides.  With the mantissas X and A (at most 11
// bits) the quotient is 127 X / A times a power of two that is at most 1, so
// one that is no half is at least 1 / (254 X) > 2^-19 of itself away from it,
// more than the division's rounding (2^-24): the rounded quotient is on the
// right side of the half.  127 X is exact, and so is a quotient that is a
// half.  Rows of very large or very small values are scaled by a power of two
// first, exactly, so that neither 127 x nor 127 / a leaves fp32.
struct RowScale {
  float pre, as, inv;  // power of two, a * pre, 127 / as
  bool any;            // finite and not all zeros
};

template <typename T>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  const float a = Bits16<T>::to_float(top);
  const float pre = a > 0x1p64f ? 0x1p-64f : a < 0x1p-64f ? 0x1p64f : 1.f;
  return {pre, a * pre, __fdiv_rn(127.f, a * pre), top != 0 && top < Bits16<T>::kInf};
}

// Codes of eight values (two a word), a byte each; rounding by adding 1.5 2^23
// (conversion instructions run at an eighth of the rate).
template <typename T>
__device__ __forceinline__ uint2 codes_of(const uint4& words, const RowScale& s) {
  constexpr float kMagic = 12582912.f;
  const uint32_t w[4] = {words.x, words.y, words.z, words.w};
  const uint64_t pre = pack_f32x2(s.pre, s.pre), inv = pack_f32x2(s.inv, s.inv), minus = pack_f32x2(-1.f, -1.f),
                 magic = pack_f32x2(kMagic, kMagic), no_magic = pack_f32x2(-kMagic, -kMagic);
  float up[8], off = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t x = pack_f32x2(Bits16<T>::to_float(w[e >> 1] & 0xFFFFu), Bits16<T>::to_float(w[e >> 1] >> 16));
    const uint64_t v = mul_f32x2(mul_f32x2(x, pre), inv), u = add_f32x2(v, magic);
    float a, b;
    unpack_f32x2(u, up[e], up[e + 1]);
    unpack_f32x2(fma_f32x2(add_f32x2(u, no_magic), minus, v), a, b);
    off = max3(off, fabsf(a), fabsf(b));
  }
  if (off > 0.4999f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = Bits16<T>::to_float((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * s.pre;
      if (fabsf(fmaf(up[e] - kMagic, -1.f, x * s.inv)) > 0.4999f) up[e] = __fdiv_rn(x * 127.f, s.as) + kMagic;
    }
  }
  auto four = [&](int e) {
    return prmt(prmt(__float_as_uint(up[e]), __float_as_uint(up[e + 1]), 0x0040),
                prmt(__float_as_uint(up[e + 2]), __float_as_uint(up[e + 3]), 0x0040), 0x5410);
  };
  return make_uint2(four(0), four(4));
}

__device__ __forceinline__ float4 lds_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void sts_cluster(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

// One block a row, which it holds in registers between the two looks at it
// (NV vectors of eight a thread): a row is read once.  |x| is compared by its
// bits, two at a time, which order like the values (an infinity or a NaN is
// the largest of all).  VEC: rows start on 16 bytes; else its values are loaded
// one by one, twice.
// Bound by the way of a block (load, two barriers, codes, store): 4096 x 4096 in
// 11.2 us (4.5 TB/s), 14336 x 4096 in 31 us (5.6 TB/s), a row of 4096 in 1.5 us.
template <typename T, int NV, bool VEC>
__global__ void __launch_bounds__(NV == 2 ? 256 : 1024, NV == 2 ? 8 : 1) quantize_i8_kernel(const uint16_t* __restrict__ x,
                                                           int64_t ldx, int K, int8_t* q,
                                                           int64_t ldq, float* scale) {
  __shared__ uint32_t s_max[32];
  grid_dependency_wait();
  launch_dependents();  // the product may fetch its weights meanwhile
  const int64_t m = blockIdx.x;
  const uint16_t* row = x + m * ldx;
  int8_t* to = q + m * ldq;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int vecs = VEC ? K / 8 : 0;
  uint4 v[NV];
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (tid + i * threads < vecs) v[i] = ldg_nc_v4(row + (int64_t)(tid + i * threads) * 8);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    top2 = __vmaxu2(top2, v[i].x & 0x7FFF7FFFu);
    top2 = __vmaxu2(top2, v[i].y & 0x7FFF7FFFu);
    top2 = __vmaxu2(top2, v[i].z & 0x7FFF7FFFu);
    top2 = __vmaxu2(top2, v[i].w & 0x7FFF7FFFu);
  }
  uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
  // eight values from k on, one by one, with zeros beyond the row
  auto eight = [&](int k) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) w[e >> 1] |= (uint32_t)row[k + e] << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  for (int k = (vecs + tid) * 8; k < K; k += threads * 8) {
    const uint4 x = eight(k);
    const uint32_t y = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    top = max(top, max(y & 0xFFFFu, y >> 16));
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((tid & 31) == 0) s_max[tid >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(0xFFFFFFFFu, (tid & 31) < threads / 32 ? s_max[tid & 31] : 0u);
  const RowScale rs = row_scale<T>(top);
  if (tid == 0)
    scale[m] = top < Bits16<T>::kInf ? __fdiv_rn(Bits16<T>::to_float(top), 127.f)
                                     : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (tid + i * threads >= vecs) continue;
    const uint2 out = rs.any ? codes_of<T>(v[i], rs) : make_uint2(0, 0);
    *reinterpret_cast<uint2*>(to + (int64_t)(tid + i * threads) * 8) = out;
  }
  for (int k = (vecs + tid) * 8; k < K; k += threads * 8) {
    const uint2 out = rs.any ? codes_of<T>(eight(k), rs) : make_uint2(0, 0);
    if (k + 8 <= K) {
      *reinterpret_cast<uint2*>(to + k) = out;
    } else {
      for (int e = 0; k + e < K; ++e) to[k + e] = (int8_t)((e < 4 ? out.x : out.y) >> (8 * (e & 3)));
    }
  }
}

// ------------------------------------------------------------- the product

// y^T in tiles of R <= 128 rows of w by BT <= 512 rows of x, in one instruction
// or (pairs) two of at most 256: the weight's rows
// are the tensor core's M (its lanes of tensor memory), the tokens its N, so a
// single token costs no more than the 16 columns that an instruction has at
// least, and y's rows are written along the lanes.  Both operands come in
// blocks of 128 columns of K through TMA (128-byte swizzle, zeros beyond the
// matrices' edges) into a ring of stages of G blocks, each operand from a warp
// of its own; tcgen05 (kind::i8) adds them into int32 accumulators in tensor
// memory, two sets of them, so that a tile's output is written while the next
// one is summed.  A wait and four instructions of few columns keep a warp for
// longer than the tensor core (about 450 cycles against 160), so up to four
// warps take stages in turn, each into an accumulator of its own; the output
// adds them up.  A ring slot always belongs to the same warp (the ring's depth
// is a multiple of theirs): a warp that took a slot's next round could wait
// for it before the round in progress is full, and a wait by parity would take
// the round before that one for it.  R needs no alignment: the tensor core reads
// 64 or 128 rows of the stage whatever they hold, and what they give for rows
// beyond R is not looked at.
//
// PAIR: two CTAs of a cluster share an instruction (cta_group::2, M = 256).
// Each holds R rows of w, half of the tile's rows of x, and the outputs of its
// own R rows, so a CTA fetches BT / 2 rows of x instead of BT.  The CTA of rank
// 0 issues for both; its `full` barriers count the copies of both, and
// consumed stages and finished sums are told to both.  Rows of w's
// blocks beyond R are zeros there, which cost the tensor core less power (333 x
// 28672 x 8192: 77.6 against 79.4 us).
//
// What bounds it.  Few rows: the weight's way from memory, and some 3 us until it
// flows (1 x 14336 x 4096 11.6 us, 16 x 4096 x 14336 12.6 us: 5 TB/s).  Many: at
// full clocks the tensor core, 87 % of its cycles (4096 x 14336 x 4096 in 165 us,
// 2.9 POP/s); kept up for longer, the board's power, which takes a quarter of the
// clock (205 us with the quantiser; 148 us with zeros for codes).  Between: a
// second round of tiles that is not full (333 x 28672 x 8192 in 76 us).
struct GemmParams {
  const float* sx;
  const float* sw;
  void* y;
  int64_t ldy;
  int M, N, K;
  int R, BT, rows;      // tile (PAIR: R rows for each CTA); rows the tensor core takes of w, 64 or 128
  int BS;               // rows of x of an instruction
  int BX;               // of those, what a CTA holds (BS, or half of it)
  int mt, tiles;        // tiles along M, in all
  int KB, G, KG;        // blocks of K, blocks a stage, stages' worth of K
  int stages;           // ring depth
  int bufs;             // sets of accumulators (1 or 2)
  int issuers;          // warps that issue MMAs, accumulators of a set (1, 2 or 4)
  int workers;          // CTAs, or pairs
  int tiles_each, tiles_more;  // tiles of every worker, workers that have one more
  uint32_t kg_step;     // 2^16 KG / workers: where a worker starts along K
  int overlap;          // the kernel before is the quantiser, which writes x's codes and nothing of w
  uint32_t a_block, b_block, b_off, bar_off, tmem_cols;
};

constexpr int kGemmThreads = 448;  // w, x, MMA, MMA, eight output warps, MMA, MMA
constexpr int kMaxGemmStages = 32;
constexpr uint32_t kKBlock = 128;
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s

// Where a CTA is on its way through its tiles and, within each, K.
struct GemmCursor {
  int tile, kg, left, slot;  // left: stages left of the tile
  uint32_t phase;            // of the ring slot
  __device__ __forceinline__ void start(int worker, int kg_first, int KG) {
    tile = worker;
    kg = kg_first;
    left = KG;
    slot = 0;
    phase = 0;
  }
  // returns whether the next stage belongs to another tile
  __device__ __forceinline__ bool step(int KG, int S, int workers) {
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
    if (++kg == KG) kg = 0;
    if (--left > 0) return false;
    left = KG;
    tile += workers;
    return true;
  }
};

// PAIR: see above; SUBS: instructions along the tile's rows of x (two in pairs
// only; loops over them would slow the issue of small tiles' copies); IMPATIENT:
// see bcq_debug_impatient (as an argument it costs 3 % of a long product).
template <typename TO, bool PAIR, int SUBS, bool IMPATIENT>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                   const GemmParams p) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // warp roles, waits and loops are uniform by construction, so that
  // descriptors and addresses stay in uniform registers (moved there for each
  // instruction, they cost 107 cycles an MMA against 39)
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = p.stages;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int worker = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x;
  const uint32_t full = sbase + p.bar_off, empty = full + 8u * S, accfull = empty + 8u * S,
                 accempty = accfull + 16u, drain = accempty + 16u, slot = drain + 32u,
                 failed = slot + 4u, sx_off = slot + 16u;
  if (warp <= 1 && lane == 0) tma_prefetch_map(warp == 0 ? &wmap : &xmap);
  if (warp == 0) {
    for (int i = lane; i < S; i += 32) {
      mbar_init(full + 8u * i, 2);
      mbar_init(empty + 8u * i, 1);
    }
    if (lane < 2) {
      mbar_init(accfull + 8u * lane, (uint32_t)p.issuers);
      mbar_init(accempty + 8u * lane, PAIR ? 16 : 8);
    }
    if (lane < 4) mbar_init(drain + 8u * lane, 1);
    if (lane == 0) sts_f32(failed, 0.f);
    fence_mbar_init();
  } else if (warp == 2) {
    if (PAIR) tmem_alloc_pair(slot, p.tmem_cols);
    else tmem_alloc(slot, p.tmem_cols);
  }
  if (PAIR) {
    // rows of w's blocks beyond R: zeros
    const uint32_t pad = (uint32_t)(128 - p.R) * 8;  // of 16 bytes, a block
    for (uint32_t i = threadIdx.x; i < pad * (uint32_t)(S * p.G); i += kGemmThreads) {
      const uint32_t block = i / pad;
      sts_zero16(sbase + block * p.a_block + (uint32_t)p.R * kKBlock + (i - block * pad) * 16);
    }
    fence_proxy_async_smem();
  }
  umma_fence_before();
  if (PAIR) {
    __syncthreads();
    cluster_sync();
  } else if (warp == 0) {
    // the weights' warp goes ahead: its first loads need nothing of the others
    asm volatile("bar.arrive 2, %0;" ::"n"(kGemmThreads) : "memory");
  } else {
    named_barrier_sync(2, kGemmThreads);
  }
  umma_fence_after();
  const uint32_t tmem = !PAIR && warp == 0 ? 0u : lds_u32v(slot);
  const int mine = p.tiles_each + (worker < p.tiles_more ? 1 : 0);
  const int total = mine * p.KG;
  // Stages of K in turn from a first one of this worker's own (the sum is exact in
  // any order): CTAs that read the same rows of x do not ask for the same lines
  // of L2 at the same time.
  const int kg_first = (int)(((uint32_t)worker * p.kg_step) >> 16);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, IMPATIENT ? mbar_wait_impatient(bar, parity) : mbar_wait_bounded(bar, parity, kWaitNs)) != 0;
  };
  // for what is in flight at the end
  auto end = [&](uint32_t bar, uint32_t parity) {
    return IMPATIENT ? mbar_look(bar, parity, 1000000) : mbar_wait_bounded(bar, parity, kWaitNs);
  };
  // A wait that ran out is recorded, and its warp does no more work; but it comes
  // to every barrier that other warps come to, and what it has in flight ends
  // before its CTA does.
  auto give_up = [&]() {
    if (lane != 0) return;
    record_error(&g_i8_error, BCQ_ERR_TIMEOUT);
    if (PAIR)
      for (uint32_t i = 0; i < 2; ++i) sts_cluster(map_rank(failed, i), 1u);
  };

  if (warp <= 1) {
    // ---------------------------------------------------------- the operands
    const bool one = elect_one(), is_w = warp == 0;
    const CUtensorMap* map = is_w ? &wmap : &xmap;
    const uint32_t block = is_w ? p.a_block : p.b_block, base = sbase + (is_w ? 0u : p.b_off);
    const uint32_t bytes = (uint32_t)(is_w ? p.R : SUBS * p.BX) * kKBlock * (PAIR ? 2u : 1u);  // of both CTAs
    // behind the quantiser the first weights need not wait for it
    if (!is_w || !p.overlap) grid_dependency_wait();
    if (!is_w) launch_dependents();  // (this CTA holds its tensor memory)
    GemmCursor c;
    c.start(worker, kg_first, p.KG);
    auto first_row = [&]() {
      const int nt = p.mt == 1 ? c.tile : c.tile / p.mt;
      return is_w ? (PAIR ? 2 * nt + rank : nt) * p.R : (c.tile - nt * p.mt) * p.BT + rank * p.BX;
    };
    int row = first_row(), issued = 0;  // copies' stages, the last S of them
    for (int i = 0; i < total; ++i) {
      if (i >= S && !wait(empty + 8u * c.slot, c.phase ^ 1u)) {
        give_up();
        break;
      }
      issued = min(S, i + 1);
      const int kb = c.kg * p.G, n = min(p.G, p.KB - kb);
      if (one) {
        const uint32_t bar = full + 8u * c.slot;
        uint32_t to = base + (uint32_t)(c.slot * p.G) * block;
        if (rank == 0) mbar_arrive_expect_tx(bar, bytes * (uint32_t)n);
        const uint32_t leader = PAIR ? map_rank(bar, 0) : bar;
        for (int j = 0; j < n; ++j, to += block) {
          const int k = (kb + j) * (int)kKBlock;
          if (PAIR) tma_load_2d_pair(to, map, k, row, leader);
          else tma_load_2d(to, map, k, row, bar);
          if (SUBS == 2 && !is_w)
            tma_load_2d_pair(to + (uint32_t)p.BX * kKBlock, map, k, row + p.BS, leader);
        }
      }
      if (c.step(p.KG, S, p.workers)) row = first_row();
    }
    // The copies end before the CTA does, whoever has given up (a pair's are all
    // told to rank 0, which the other CTA waits for): slots from c.slot on hold the
    // round before c's.
    bool there = rank == 0;
    for (int i = 0; i < issued && there; ++i)
      there = end(full + 8u * i, c.phase ^ (issued == S && i >= c.slot ? 1u : 0u));
  } else if (warp < 4 || warp >= 12) {
    // --------------------------------------------------------------- the sums
    const int issuer = warp < 4 ? warp - 2 : warp - 10;
    const bool one = elect_one();
    // kind::i8: int32 D, signed A and B, both K-major, N = BS, M = rows
    const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(p.BS >> 3) << 17) |
                           ((uint32_t)((PAIR ? 256 : p.rows) >> 4) << 24);
    const uint64_t ad0 = umma_desc_sw128(sbase), bd0 = umma_desc_sw128(sbase + p.b_off);
    const uint32_t a_units = p.a_block >> 4, b_units = p.b_block >> 4;  // never carry out of the address
    auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
      if (PAIR) umma_i8_ss_pair(d, a, b, id, acc);
      else umma_i8_ss(d, a, b, id, acc);
    };
    auto commit = [](uint32_t bar) {
      if (PAIR) umma_commit_pair(bar);
      else umma_commit(bar);
    };
    bool ok = true;
    GemmCursor c;
    c.start(worker, kg_first, p.KG);
    for (int t = 0; t < mine && ok && issuer < p.issuers && rank == 0; ++t) {
      const int buf = p.bufs == 2 ? t & 1 : 0, round = p.bufs == 2 ? t >> 1 : t;
      if (round > 0) ok = wait(accempty + 8u * buf, (uint32_t)(round - 1) & 1u);
      umma_fence_after();
      const uint32_t d = tmem + (uint32_t)((buf * p.issuers + issuer) * p.BT);
      uint32_t more = 0;  // whether the accumulator holds something
      for (int g = 0; g < p.KG && ok; ++g) {
        if ((c.slot & (p.issuers - 1)) == issuer) {
          ok = wait(full + 8u * c.slot, c.phase);
          if (!ok) break;
          umma_fence_after();
          const int kb = c.kg * p.G, n = min(p.G, p.KB - kb);
          uint64_t ad = ad0 + (uint32_t)(c.slot * p.G) * a_units, bd = bd0 + (uint32_t)(c.slot * p.G) * b_units;
          if (one) {
            for (int j = 0; j < n; ++j, ad += a_units, bd += b_units) {
              // 32-byte slices of K: all four, or those that hold some of it
              const int rest = p.K - (kb + j) * (int)kKBlock;
              mma(d, ad, bd, idesc, more);
              if (rest > 32) mma(d, ad + 2, bd + 2, idesc, 1u);
              if (rest > 64) mma(d, ad + 4, bd + 4, idesc, 1u);
              if (rest > 96) mma(d, ad + 6, bd + 6, idesc, 1u);
              if (SUBS == 2) {
                const uint64_t bs = bd + (uint32_t)p.BX * (kKBlock >> 4);
                const uint32_t ds = d + (uint32_t)p.BS;
                mma(ds, ad, bs, idesc, more);
                if (rest > 32) mma(ds, ad + 2, bs + 2, idesc, 1u);
                if (rest > 64) mma(ds, ad + 4, bs + 4, idesc, 1u);
                if (rest > 96) mma(ds, ad + 6, bs + 6, idesc, 1u);
              }
              more = 1;
            }
            commit(empty + 8u * c.slot);
          }
          more = 1;
        }
        c.step(p.KG, S, p.workers);
      }
      if (ok && one) commit(accfull + 8u * buf);
    }
    if (!ok) give_up();
    if (rank == 0 && issuer < p.issuers) {  // the products end before the CTA does
      if (one) {
        if (PAIR) umma_commit_pair_here(drain + 8u * issuer);
        else umma_commit(drain + 8u * issuer);
      }
      end(drain + 8u * issuer, 0);
    }
  } else {
    // ------------------------------------------------------------ the outputs
    // 64 rows lie in the first 16 lanes of each quarter, 128 in all 32
    // two warps a quarter, each half of the columns
    const int quarter = warp & 3, each = p.rows >> 2, half = (warp - 4) >> 2;
    const int split = ((p.BT >> 4) + 1) / 2 * 16;
    const int r = lane < each ? quarter * each + lane : 1 << 20;
    grid_dependency_wait();  // sx, and y's last use
    bool ok = true;
    for (int t = 0; t < mine; ++t) {
      const int tile = worker + t * p.workers;
      const int nt = p.mt == 1 ? tile : tile / p.mt;
      const int n = (PAIR ? 2 * nt + rank : nt) * p.R + r, m0 = (tile - nt * p.mt) * p.BT;
      const int buf = p.bufs == 2 ? t & 1 : 0, cols = min(p.BT, p.M - m0);
      const bool row = r < p.R && n < p.N;
      const float swn = row ? p.sw[n] : 0.f;
      // the tile's sx, fetched while it is summed; two buffers, and the barrier
      // of the next tile parts their uses
      const uint32_t sxs = sx_off + (uint32_t)(t & 1) * 2048u;
      for (int c = (int)threadIdx.x - 128; c < p.BT; c += 256)
        sts_f32(sxs + 4u * c, c < cols ? p.sx[m0 + c] : 0.f);
      named_barrier_sync(1, 256);
      if (ok && !(ok = wait(accfull + 8u * buf, (uint32_t)(p.bufs == 2 ? t >> 1 : t) & 1u))) give_up();
      if (!ok) continue;  // to the next tile's barrier
      umma_fence_after();
      if (quarter * each < p.R) {
        const int c_first = half * split, c_end = half ? cols : min(cols, split);
        TO* y = static_cast<TO*>(p.y) + ((int64_t)m0 + c_first) * p.ldy + n;
        const uint32_t acc = tmem + (uint32_t)(buf * p.issuers * p.BT) + ((uint32_t)(quarter * 32) << 16);
        for (int c = c_first; c < c_end; c += 16) {
          uint32_t v[16];
          tmem_ld16(acc + (uint32_t)c, v);
          float4 sx4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) sx4[j] = lds_f32x4(sxs + 4u * (c + 4 * j));
          tmem_wait_ld();
          for (int i = 1; i < p.issuers; ++i) {
            uint32_t w[16];
            tmem_ld16(acc + (uint32_t)(i * p.BT + c), w);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += w[j];
          }
          float f[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float4 q = sx4[j >> 2];
            f[j] = (float)(int)v[j] * ((j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w) * swn;
          }
          if (row && c + 16 <= c_end) {
#pragma unroll
            for (int j = 0; j < 16; ++j, y += p.ldy) store_out(y, f[j]);
          } else if (row) {
#pragma unroll
            for (int j = 0; j < 16; ++j, y += p.ldy)
              if (c + j < c_end) store_out(y, f[j]);
          }
        }
      }
      umma_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_cluster(map_rank(accempty + 8u * buf, 0));
        else mbar_arrive_cta(accempty + 8u * buf);
      }
    }
  }
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  if (PAIR) {
    cluster_sync();  // neither CTA leaves while the other uses its memory
    if (lds_u32v(failed)) {
      // copies of rank 1 that rank 0 no longer expected have a millisecond (they
      // take some microseconds)
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 1000000ull) {
      }
      cluster_sync();
    }
  }
  if (warp == 2) {
    umma_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, p.tmem_cols);
    else tmem_dealloc(tmem, p.tmem_cols);
  }
}

// -------------------------------------------------------------------- host

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t padded_k(int K) { return ((int64_t)K + 15) / 16 * 16; }

bool sizes_ok(int M, int K) { return M >= 0 && K >= 1 && K <= BCQ_I8_MAX_K; }

bool is16(int dtype) { return dtype == BCQ_F16 || dtype == BCQ_BF16; }

constexpr size_t kMaxSmem = 232448;                          // 227 KiB per CTA on sm_100

template <typename T>
cudaError_t launch_quantize_t(const uint16_t* x, int M, int K, int64_t ldx, int8_t* q, int64_t ldq,
                              float* scale, cudaStream_t st) {
  auto launch = [&](auto kernel, unsigned threads) {
    return launch_early(kernel, dim3((unsigned)M), threads, 0, st, x, ldx, K, q, ldq, scale);
  };
  if (!aligned(x, 16) || (ldx % 8 && M > 1)) return launch(quantize_i8_kernel<T, 1, false>, 256);
  // Many rows: fewer threads a row, more rows an SM and loads in flight; few rows:
  // more threads a row (us, few | many threads: 64 x 4096 2.6 | 2.0, 1024 x 4096
  // 4.8 | 4.0, 4096 x 4096 11.2 | 11.8, 14336 x 4096 31.1 | 34.4; 333 x 14336 6.5 |
  // 5.2, 1024 x 14336 11.5 | 12.7, 4096 x 14336 33.3 | 42.2).
  if (K <= 4096 && M < 3000) return launch(quantize_i8_kernel<T, 2, true>, 256);
  if (K <= 4096) return launch(quantize_i8_kernel<T, 4, true>, 128);
  if (K <= 16384 && M < 1024) return launch(quantize_i8_kernel<T, 4, true>, 512);
  if (K <= 16384) return launch(quantize_i8_kernel<T, 8, true>, 256);
  return launch(quantize_i8_kernel<T, 8, true>, 1024);
}

cudaError_t launch_quantize(const void* x, int dtype, int M, int K, int64_t ldx, int8_t* q,
                            int64_t ldq, float* scale, cudaStream_t st) {
  const uint16_t* p = static_cast<const uint16_t*>(x);
  return dtype == BCQ_F16 ? launch_quantize_t<__half>(p, M, K, ldx, q, ldq, scale, st)
                          : launch_quantize_t<__nv_bfloat16>(p, M, K, ldx, q, ldq, scale, st);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder (no link-time dependency on the driver library).
EncodeTiled encode_tiled() {
  static std::atomic<void*> found{nullptr};
  void* f = found.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return nullptr;
    found.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Codes [rows][K] in boxes of box_rows rows by 128 columns.
bool encode_codes(CUtensorMap* map, const int8_t* p, int64_t rows, int64_t K, int64_t ld,
                  uint32_t box_rows) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {kKBlock, box_rows}, step[2] = {1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t v, int64_t by) { return (v + by - 1) / by; }
int round_up(int64_t v, int to) { return (int)(ceil_div(v, to) * to); }

// The tile and the kernel (*kind: 0 single CTAs, 1 pairs, 2 pairs with two
// instructions along x's rows) that a model of one SM's time likes
// best.  A block of K takes the longest of: the tensor core (BT / 2 cycles for
// each of its four instructions), shared memory's reads by it (128 rows of w
// and those of x at 128 bytes a cycle), the operands' way from L2 (about 50
// bytes a cycle an SM), and, where w is read by one tile only, its share of
// the memory's rate (about 24 bytes a cycle an SM).  Rounds of tiles count
// whole; a tile's output costs about 15 cycles a column when nothing hides it,
// a pair's start some 1000 cycles.
// Measured (us: single CTAs | pairs | the model's choice of pairs with one or two
// instructions, where there is one): 64 x 14336 x 4096 12.5 | 13.9, 128 rows 17.6
// | 15.4, 256 rows 21.0 | 18.7, 512 rows 33.0 | 29.0 | 29.8, 333 x 28672 x 8192
// 95.9 | 90.5 | 77.4, 1024 x 4096 x 4096 17.1 | 17.4 | 17.3, 4096 x 14336 x 4096
// 181 | 164 | 165.
void plan_gemm(int M, int N, int K, int sms, GemmParams* p, size_t* smem, int* grid, int* kind) {
  const int KB = (K + (int)kKBlock - 1) / (int)kKBlock;
  double best = 0;
  for (int two = 0; two < 2; ++two) {
    const int workers = two ? sms / 2 : sms;
    for (int subs = 1; subs <= 1 + two; ++subs) {
      // every BS that is the least for its number of tiles, up to four more of them
      // than whole ones would be
      const int step = two ? 32 : 16, least_bs = subs == 2 ? 128 : two ? 64 : 16;
      for (int BS = std::min(256, round_up(ceil_div(M, subs), step)); BS >= least_bs; BS -= step) {
        const int BT = subs * BS;
        const int64_t mt = ceil_div(M, BT);
        if (BS != round_up(ceil_div(M, mt * subs), step) || mt > ceil_div(M, 256) + 4) continue;
        const int rows_most = two ? 256 : 128;
        const int64_t least = ceil_div(ceil_div(N, rows_most) * mt, workers);
        for (int64_t rounds = least; rounds <= least + 2; ++rounds) {
          const int64_t nt_most = std::max<int64_t>(1, rounds * workers / mt);
          int64_t rows = std::min<int64_t>(rows_most, std::max<int64_t>(8, ceil_div(N, nt_most)));
          if (two) rows = (rows + 1) / 2 * 2;
          const int R = (int)(two ? rows / 2 : rows);
          const int64_t nt = ceil_div(N, rows), tiles = nt * mt, whole = ceil_div(tiles, workers);
          const int BX = two ? BS / 2 : BS;
          const double core = 4.0 * subs * std::max(BS / 2.0, 32.0 + BX / 4.0);
          const double l2 = 128.0 * (R + subs * BX) / 50.0, dram = mt == 1 ? 128.0 * R / 24.0 : 0;
          // outputs that no other tile's sums hide: the last tile's, or all
          // where tensor memory has no room for a second set of accumulators
          const double out = 15.0 * BT * (2 * BT > 512 ? whole : 1);
          const double cost = whole * (KB * std::max(core, std::max(l2, dram)) + 20.0) + out + (two ? 1000.0 : 0.0);
          if (best == 0 || cost < best) {
            best = cost;
            p->R = std::min(R, N);
            p->BT = BT;
            *kind = two + subs - 1;
            p->BS = BS;
            p->BX = BX;
            p->mt = (int)mt;
            p->tiles = (int)tiles;
            p->workers = (int)std::min<int64_t>(workers, tiles);
          }
        }
      }
    }
  }
  const bool pair = *kind > 0;
  const int subs = *kind == 2 ? 2 : 1;
  p->KB = KB;
  p->bufs = p->tiles > p->workers && 2 * p->BT <= 512 ? 2 : 1;
  p->rows = p->R <= 64 && !pair ? 64 : 128;
  p->a_block = (uint32_t)(pair ? 128 : round_up(p->R, 8)) * kKBlock;
  p->b_block = (uint32_t)(subs * p->BX) * kKBlock;
  const uint32_t block = p->a_block + p->b_block;
  // about 24 KB a stage: a wait costs the MMA warp about 100 cycles, as long
  // as the four instructions of a small block of K take
  p->G = std::max(1, std::min({8, KB, (int)(24576 / block)}));
  p->KG = (KB + p->G - 1) / p->G;
  const size_t room = kMaxSmem - 1024 /* alignment */ - 16 * kMaxGemmStages - 96 - 4096 /* sx */;
  const uint32_t overrun = (uint32_t)p->rows * kKBlock;  // read of the last block of w, beyond R
  int S = (int)std::min<size_t>(kMaxGemmStages, room / (block * (uint32_t)p->G));
  while (S > 1 && (size_t)S * p->G * p->a_block + overrun > room) --S;
  // accumulators fit tensor memory, every issuer has a stage of every tile, and
  // the ring is a multiple of the issuers
  p->issuers = p->bufs * p->BT <= 128 ? 4 : p->bufs * p->BT <= 256 ? 2 : 1;
  while (p->issuers > p->KG || p->issuers > S) p->issuers /= 2;
  S -= S % p->issuers;
  p->stages = S;
  p->b_off = (uint32_t)(S * p->G) * p->a_block;
  p->bar_off = p->b_off + std::max((uint32_t)(S * p->G) * p->b_block, overrun);
  uint32_t cols = 32;
  while (cols < (uint32_t)(p->bufs * p->issuers * p->BT)) cols *= 2;
  p->tmem_cols = cols;
  *smem = 1024 + p->bar_off + 16 * (size_t)S + 96 + 4096;
  *grid = pair ? 2 * p->workers : p->workers;
  p->tiles_each = p->tiles / p->workers;
  p->tiles_more = p->tiles % p->workers;
  p->kg_step = ((uint32_t)p->KG << 16) / (uint32_t)p->workers;
}

// SMs of the current device, 0 if it cannot be asked.
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2)
    return 0;
  return n;
}

template <typename TO, bool PAIR, int SUBS, bool IMPATIENT = false>
cudaError_t launch_gemm_t(const CUtensorMap& wmap, const CUtensorMap& xmap, const GemmParams& p,
                          size_t smem, int grid, cudaStream_t st) {
  if constexpr (std::is_same_v<TO, __half> && !IMPATIENT)
    if (impatient()) return launch_gemm_t<TO, PAIR, SUBS, true>(wmap, xmap, p, smem, grid, st);
  const auto kernel = gemm_i8_kernel<TO, PAIR, SUBS, IMPATIENT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kernel, kMaxSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2] = {};
  int n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, kernel, wmap, xmap, p);
}

// overlap: the kernel before in the stream is the quantiser, whose codes and
// scales are waited for; it writes nothing of w.
cudaError_t launch_gemm(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w,
                        int64_t ldw, const float* sw, int M, int N, int K, void* y, int dtype,
                        int64_t ldy, bool overlap, cudaStream_t st) {
  const int sms = sm_count();
  if (sms == 0) return cudaErrorInvalidDevice;
  GemmParams p = {};
  p.sx = sx;
  p.sw = sw;
  p.y = y;
  p.ldy = ldy;
  p.M = M;
  p.N = N;
  p.K = K;
  p.overlap = overlap;
  size_t smem = 0;
  int grid = 0;
  int kind = 0;
  plan_gemm(M, N, K, sms, &p, &smem, &grid, &kind);
  CUtensorMap wmap, xmap;
  if (!encode_codes(&wmap, w, N, K, ldw, (uint32_t)p.R) ||
      !encode_codes(&xmap, x, M, K, ldx, (uint32_t)p.BX))
    return cudaErrorInvalidValue;
  auto launch = [&](auto* type) {
    using TO = std::remove_pointer_t<decltype(type)>;
    return kind == 2   ? launch_gemm_t<TO, true, 2>(wmap, xmap, p, smem, grid, st)
           : kind == 1 ? launch_gemm_t<TO, true, 1>(wmap, xmap, p, smem, grid, st)
                       : launch_gemm_t<TO, false, 1>(wmap, xmap, p, smem, grid, st);
  };
  if (dtype == BCQ_F32) return launch((float*)nullptr);
  if (dtype == BCQ_F16) return launch((__half*)nullptr);
  return launch((__nv_bfloat16*)nullptr);
}

// The weight's and the output's arguments, shared by bcq_gemm_i8 and bcq_linear_i8.
bcq_status check_product(const int8_t* w, int64_t ldw, const float* sw, int M, int N, int K,
                         const void* y, int dtype, int64_t ldy) {
  if (!w || !sw || !y) return BCQ_ERR_NULL;
  if (!sizes_ok(M, K) || N < 1 || ldw < K || ldy < N) return BCQ_ERR_SHAPE;
  if (!is16(dtype) && dtype != BCQ_F32) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(w, 16) || ldw % 16 || !aligned(sw, 4) || !aligned(y, dtype == BCQ_F32 ? 4 : 2))
    return BCQ_ERR_ALIGN;
  return BCQ_OK;
}

}  // namespace

cudaError_t read_and_clear_i8_error(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_i8_error, sizeof(int));
  if (e == cudaSuccess && *code != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_i8_error, &zero, sizeof(int));
  }
  return e;
}

}  // namespace bcq

using namespace bcq;

extern "C" {

bcq_status bcq_quantize_i8(const void* x, int dtype, int M, int K, int64_t ldx, int8_t* q,
                           int64_t ldq, float* scale, void* stream) {
  if (M == 0 && sizes_ok(M, K)) return BCQ_OK;
  if (!x || !q || !scale) return BCQ_ERR_NULL;
  if (!sizes_ok(M, K) || ldx < K || ldq < K) return BCQ_ERR_SHAPE;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(x, 2) || !aligned(q, 16) || ldq % 16 || !aligned(scale, 4)) return BCQ_ERR_ALIGN;
  return launch_quantize(x, dtype, M, K, ldx, q, ldq, scale, (cudaStream_t)stream) == cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

bcq_status bcq_gemm_i8(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w,
                       int64_t ldw, const float* sw, int M, int N, int K, void* y, int dtype,
                       int64_t ldy, void* stream) {
  if (M == 0 && sizes_ok(M, K) && N >= 1) return BCQ_OK;
  if (!x || !sx) return BCQ_ERR_NULL;
  const bcq_status s = check_product(w, ldw, sw, M, N, K, y, dtype, ldy);
  if (s != BCQ_OK) return s;
  if (ldx < K) return BCQ_ERR_SHAPE;
  if (!aligned(x, 16) || ldx % 16 || !aligned(sx, 4)) return BCQ_ERR_ALIGN;
  return launch_gemm(x, ldx, sx, w, ldw, sw, M, N, K, y, dtype, ldy, false, (cudaStream_t)stream) ==
                 cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

size_t bcq_linear_i8_workspace_bytes(int M, int K) {
  if (!sizes_ok(M, K)) return 0;
  return (size_t)M * (size_t)padded_k(K) + ((size_t)M * 4 + 15) / 16 * 16;
}

bcq_status bcq_linear_i8(const void* x, int dtype, int64_t ldx, const int8_t* w, int64_t ldw,
                         const float* sw, int M, int N, int K, void* y, int64_t ldy,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (M == 0 && sizes_ok(M, K) && N >= 1) return BCQ_OK;
  if (!x || !workspace) return BCQ_ERR_NULL;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  const bcq_status s = check_product(w, ldw, sw, M, N, K, y, dtype, ldy);
  if (s != BCQ_OK) return s;
  if (ldx < K) return BCQ_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(workspace, 16)) return BCQ_ERR_ALIGN;
  if (workspace_bytes < bcq_linear_i8_workspace_bytes(M, K)) return BCQ_ERR_NULL;
  const int64_t ldq = padded_k(K);
  int8_t* q = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(q + (size_t)M * (size_t)ldq);
  cudaStream_t st = (cudaStream_t)stream;
  if (launch_quantize(x, dtype, M, K, ldx, q, ldq, sx, st) != cudaSuccess) return BCQ_ERR_CUDA;
  return launch_gemm(q, ldq, sx, w, ldw, sw, M, N, K, y, dtype, ldy, true, st) == cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

}  // extern "C"

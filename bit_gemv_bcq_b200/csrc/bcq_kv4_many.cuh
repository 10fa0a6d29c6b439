// bcq_kv4_many.cuh -- attention of many rows over the 4-bit cache (prompts and
// their chunks), on the 5th-generation tensor core (included by bcq_kv4.cu
// only, whose parameters, spans and helpers it uses).
//
//   S = Q K^T,  P = exp2(S fs - m),  O += P V  for 128 rows of a key/value head
// (query heads that share it times rows of the call) a tile, two tiles a CTA
// (one where D = 256 leaves tensor memory for no more), and 64 positions a
// step.  Four warps for K and four for V turn the codes into fp16 operands in
// shared memory, once for both tiles: c from its bits (1024 + c or 1024 + 16 c, exactly), then a c +
// z with one rounding to fp16 (half a step, 2^-11).  That puts an error of up to
// 2^-11 of |scale| sum |q K| on a score; over many positions of like weight it
// averages out of lse, over few it does not.  So a block of rows one of which sees
// fewer than kFewSeen positions has K's in two parts (2^-22), which doubles the
// products and their operands; a block of a prompt's later rows, or of a longer
// sequence of the same call, has not (us, one part | two | the few-row kernel: 8
// prompts of 200 to 400 new tokens, 32 heads of 128 on 8, 48.0 | 52.0 | 147; windows
// of 256 over 4 x 1000 new tokens, 16 heads of 64 on 4, 34.3 | 36.5 | 60.0; 8 x 100
// rows over 400 positions, 16 heads of 256 on 4, 22.9 | 30.5 | 38.7).  One warp issues the
// products; four warps a tile do its softmax, a thread a row.  S has two
// buffers a tile, so that a step's scores are there when the softmax of the
// one before ends (steps of 128 positions leave tensor memory for one: the
// softmax then waits for two products a step, 5200 cycles for 128 positions).
// P replaces S in tensor memory, in fp16 (the second rounding of 2^-11); O
// stays there, and is scaled only when a row's maximum has risen by more than
// 2^8 over the one in use.  p is held times 2^7, so it is at most 2^15 and keeps
// its 11 bits down to 2^-21 of the row's largest; below, a position is off by
// 2^-32 of that at most.
// Queries are scaled by a power of two a row to the top of fp16's range.
// Within eight values of a vector both operands have the order 0 4 1 5 2 6 3 7,
// in which masks yield them; outputs are put right as they are written.
//
// A value of V that is no number must not reach rows that do not see its
// position (0 * NaN): such groups become zeros, and rows that see them are told
// by a mask to write NaN.
//
// What bounds it: the softmax of 2 x 128 rows, some 2300 cycles for 64 positions
// where the tensor core needs 1280 (the exponentials alone 1024 of the special-
// function units, the rest issue and the way to and from tensor memory), and the
// last CTAs, which see the most.  2 x 2048 new tokens over their prompts, 32
// heads of 128 on 8: 561 TFLOP/s; a chunk of 2048 that ends at 4096, 16 heads of 256
// on 4: 669 TFLOP/s (of 1642 that a dense bf16 product reaches).
#pragma once

#include "bcq_tcgen05.cuh"

namespace bcq {
namespace {

constexpr float kManyBits = 7.f;  // p is held times 2^7

template <int D>
struct ManyShape {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  static constexpr int kTokens = 64;                         // of a step
  // K's and V's operands share six tiles (four where D = 256): three buffers each,
  // or two of K's in two parts and two of V's.  (More shared memory leaves less
  // to L1: with nine tiles 2 x 2048 new tokens took 228 us, 220 with six.)
  static constexpr int kBufs = D == 256 ? 2 : 3;             // of K's, and of V's
  static constexpr int kKBufs2 = D == 256 ? 1 : 2;           // of K's in two parts
  static constexpr int kVBufs2 = 2;                          // of V's beside them
  static_assert(2 * kKBufs2 + kVBufs2 <= 2 * kBufs, "operands' tiles");
  static constexpr int kBlocks = D / 64;                     // 128-byte column blocks of a vector
  static constexpr uint32_t kQBlock = 128 * 128;             // bytes of 64 columns of 128 rows
  static constexpr uint32_t kQTile = kBlocks * kQBlock;
  static constexpr uint32_t kKvBlock = kTokens * 128;
  static constexpr uint32_t kKvTile = kBlocks * kKvBlock;
  static constexpr uint32_t kOffK = kTiles * kQTile;
  static constexpr uint32_t kOffBar = kOffK + 2 * kBufs * kKvTile;
  // a step's mask words: the positions without a page, and V's groups that are
  // no numbers.  A ring of eight: K's operands of step j + 8 come after the
  // scores of step j + 8 - kBufs, and so after the softmax of step j + 3 (V's
  // after the product of step j + 8 - kBufs); step j's words are read for the
  // last time as step j + 1 ends.
  static constexpr int kPieces = D / 32;                     // 16-byte pieces of a vector's codes
  static constexpr int kPasses = kTokens * kPieces / 128;    // pieces a thread and step
  static constexpr int kPerWarp = 32 / kPieces;              // positions a warp and pass
  static constexpr int kWords = kPasses * 4;
  static constexpr uint32_t kOffMask = kOffBar + 256;
  static constexpr uint32_t kOffOdd = kOffMask + 2 * 8 * kWords * 4;  // whether any mask word is not zero
  static constexpr uint32_t kSmem = 1024 + kOffOdd + 16;
  static constexpr int kOCol = 2 * kTiles * kTokens;         // tensor memory: S buffers, then O tiles
  // softmax, K's and V's codes, MMA.  Two tiles' 20 warps start with 96
  // registers a thread, 61440 in all, and share them anew by groups of four
  // warps: 2 * 128 * 128 (softmax) + 2 * 128 * 80 (codes) + 128 * 56 = 60416.
  static constexpr int kThreads = kTiles == 2 ? 640 : 416;
};

// A ring's slot and the round it is in.
struct RingAt {
  int slot = 0, round = 0;
  __device__ __forceinline__ void step(int slots) {
    if (++slot == slots) {
      slot = 0;
      ++round;
    }
  }
};

// Shared-memory descriptor, 128-byte swizzle: `lead` bytes between 64-element
// blocks of a contiguous M or N (1 where K is contiguous), `stride` bytes
// between groups of 8 rows.
__device__ __forceinline__ uint64_t umma_desc_blocks(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(stride >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void umma_f16_ss(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// One word of codes as eight fp16 values a c + z, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 word_values(uint32_t w, __half2 a, __half2 z) {
  const __half2 k1024 = __float2half2_rn(1024.f), k16 = __float2half2_rn(0.0625f),
                k64 = __float2half2_rn(-64.f);
  auto low = [&](uint32_t x) {   // 1024 + c
    const uint32_t h = (x & 0x000F000Fu) | 0x64006400u;
    return __hfma2(a, __hsub2(*reinterpret_cast<const __half2*>(&h), k1024), z);
  };
  auto high = [&](uint32_t x) {  // 1024 + 16 c
    const uint32_t h = (x & 0x00F000F0u) | 0x64006400u;
    return __hfma2(a, __hfma2(*reinterpret_cast<const __half2*>(&h), k16, k64), z);
  };
  const __half2 v[4] = {low(w), high(w), low(w >> 8), high(w >> 8)};
  return *reinterpret_cast<const uint4*>(v);
}

// The same, a c + z in fp32, as two fp16 parts.
__device__ __forceinline__ void word_parts(uint32_t w, float a, float z, uint4& first, uint4& second) {
  const uint64_t a2 = pack_f32x2(a, a), z2 = pack_f32x2(z, z), no_magic = pack_f32x2(-8388608.f, -8388608.f),
                 minus = pack_f32x2(-1.f, -1.f);
  const uint32_t low = w & 0x0F0F0F0Fu, high = (w >> 4) & 0x0F0F0F0Fu;
  auto two = [&](uint32_t x, uint32_t from, uint32_t& p, uint32_t& q) {  // bytes from and from + 2
    const float c0 = __uint_as_float(prmt(x, 0x4B000000u, 0x7440u + from));  // 2^23 + c
    const float c1 = __uint_as_float(prmt(x, 0x4B000000u, 0x7442u + from));
    const uint64_t v = fma_f32x2(a2, add_f32x2(pack_f32x2(c0, c1), no_magic), z2);
    float f0, f1;
    unpack_f32x2(v, f0, f1);
    p = pack_f16(f0, f1);
    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&p));
    unpack_f32x2(fma_f32x2(pack_f32x2(back.x, back.y), minus, v), f0, f1);
    q = pack_f16(f0, f1);
  };
  two(low, 0, first.x, second.x);
  two(high, 0, first.y, second.y);
  two(low, 1, first.z, second.z);
  two(high, 1, first.w, second.w);
}

__device__ __forceinline__ void sts_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Whether some row of a block sees fewer than kFewSeen positions: the first one
// sees the fewest under a causal mask, else the last one.
__device__ __forceinline__ bool few_seen(const AttentionParams& p, const Span& sp, int block) {
  auto seen = [&](int i) {
    const int pos = sp.pos0 + i;
    return (p.causal ? min(sp.len, pos + 1) : sp.len) - (p.window > 0 ? max(0, pos - p.window + 1) : 0);
  };
  const int i0 = p.group.quotient(block * p.rows), i1 = p.group.quotient((block + 1) * p.rows - 1);
  return min(seen(i0), seen(min(i1, sp.rows - 1))) < kFewSeen;
}

// IMPATIENT: see bcq_debug_impatient (as an argument it costs 3 %).
template <typename T, int D, bool IMPATIENT>
__global__ void __launch_bounds__(ManyShape<D>::kThreads, 1) kv4_many_kernel(const AttentionParams p) {
  using S = ManyShape<D>;
  constexpr int G = D / kKvGroup;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem_raw + (sbase - smem_u32(smem_raw)) + S::kOffMask);
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // the last blocks of rows see the most: theirs go first, of every sequence
  // and head
  const int pairs = p.at.heads * p.at.B, pair = (int)(blockIdx.x % (unsigned)pairs);
  const int block = p.row_blocks - 1 - (int)(blockIdx.x / (unsigned)pairs);
  const int b = p.by_heads.quotient(pair), kvh = pair - b * p.at.heads, part = blockIdx.y;
  grid_dependency_wait();
  const Span sp = span_of(p, b, block);
  if (part == 0 && block == 0 && kvh == 0 && threadIdx.x == 0) {
    if (rows_of(p.at, b).y > p.max_q) record_error(&g_kv4_error, BCQ_ERR_SHAPE);
    if (p.at.kv_len[b] != sp.len) record_error(&g_kv4_error, BCQ_ERR_PAGE);
  }
  if (part >= sp.parts) return;
  const bool two_parts = few_seen(p, sp, block);  // of K's operands
  const int k_bufs = two_parts ? S::kKBufs2 : S::kBufs, v_bufs = two_parts ? S::kVBufs2 : S::kBufs;
  const uint32_t k_step = two_parts ? 2 * S::kKvTile : S::kKvTile;  // a second part follows the first
  const uint32_t off_v = S::kOffK + (uint32_t)k_bufs * k_step;
  const int row0 = block * p.rows, row_n = min(p.rows, sp.rows * p.group.d - row0);
  const int begin = sp.begin + part * sp.chunk, end = min(sp.end, begin + sp.chunk);
  const int steps = end > begin ? (end - begin + S::kTokens - 1) / S::kTokens : 0;
  const int tiles = row_n > 128 ? 2 : 1;  // of this CTA

  // S, P and their tiles' barriers: [tile][buffer]
  const uint32_t bar = sbase + S::kOffBar;
  const uint32_t q_full = bar, k_full = bar + 8, k_empty = bar + 32, v_full = bar + 56,
                 v_empty = bar + 80, s_full = bar + 104, p_full = bar + 136, o_done = bar + 168,
                 drain = bar + 184, slot = bar + 192;
  constexpr int kCodeWarp0 = 4 * S::kTiles, kMmaWarp = kCodeWarp0 + 8;
  if (warp == kMmaWarp) {
    if (lane == 0) {
      mbar_init(q_full, (uint32_t)(4 * tiles));
      mbar_init(drain, 1);
      for (int i = 0; i < 3; ++i) {
        mbar_init(k_full + 8 * i, 4);
        mbar_init(k_empty + 8 * i, 1);
        mbar_init(v_full + 8 * i, 4);
        mbar_init(v_empty + 8 * i, 1);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(s_full + 8 * i, 1);
        mbar_init(p_full + 8 * i, 4);
      }
      for (int i = 0; i < 2; ++i) mbar_init(o_done + 8 * i, 1);
      sts_f32(sbase + S::kOffOdd, 0.f);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(slot, 512);
  }
  umma_fence_before();
  __syncthreads();
  umma_fence_after();
  const uint32_t tmem = lds_u32v(slot);
  constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s
  // A waiting thread that sleeps takes some 400 cycles to wake: look a while first.
  auto wait = [&](uint32_t at, int round) {
    if (IMPATIENT) return __all_sync(0xFFFFFFFFu, mbar_wait_impatient(at, (uint32_t)round & 1u)) != 0;
    bool there = false;
#pragma unroll 1
    for (int i = 0; i < 64 && !there; ++i) there = mbar_test(at, (uint32_t)round & 1u);
    return __all_sync(0xFFFFFFFFu, there || mbar_wait_bounded(at, (uint32_t)round & 1u, kWaitNs)) != 0;
  };
  // A warp whose wait ran out does no more work, but comes to every barrier that
  // other warps come to; the products in flight end before the CTA does.
  auto give_up = [&]() {
    if (lane == 0) record_error(&g_kv4_error, BCQ_ERR_TIMEOUT);
  };

  if (warp >= kMmaWarp) {
    if (S::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kMmaWarp) {
    // ------------------------------------------------------------ the products
    // (a choice within the loop keeps addresses out of the uniform registers, 4 %;
    // both parts' instructions written out one behind the other would not fit the
    // registers, 8 % where D = 256)
    auto products = [&](auto two_type) {
      constexpr bool kTwo = decltype(two_type)::value;
      constexpr uint32_t kStep = kTwo ? 2 * S::kKvTile : S::kKvTile;
      constexpr uint32_t kOffV = S::kOffK + (kTwo ? S::kKBufs2 : S::kBufs) * kStep;
      const bool one = elect_one();
      // fp16 A and B, fp32 D, M = 128; V has its values (N) contiguous
      constexpr uint32_t kIdS = (1u << 4) | ((uint32_t)(S::kTokens >> 3) << 17) | (8u << 24);
      constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
      const uint64_t qd = umma_desc_sw128(sbase), kd = umma_desc_sw128(sbase + S::kOffK);
      const uint64_t vd = umma_desc_blocks(sbase + kOffV, S::kKvBlock, 1024);
      bool ok = steps == 0 || wait(q_full, 0);
      RingAt ka, va;
      auto scores = [&](int j) {  // of step j, both tiles
        if (!(ok = wait(k_full + 8u * ka.slot, ka.round))) return;
        umma_fence_after();
        if (one) {
          for (int t = 0; t < tiles; ++t) {
#pragma unroll 1
            for (int part = 0; part < (kTwo ? 2 : 1); ++part) {
              const uint64_t k = kd + ((ka.slot * kStep + (uint32_t)part * S::kKvTile) >> 4);
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
                umma_f16_ss(tmem + (uint32_t)((2 * t + (j & 1)) * S::kTokens),
                            qd + (uint32_t)((t * S::kQTile + (c >> 2) * S::kQBlock + (c & 3) * 32) >> 4),
                            k + (uint32_t)(((c >> 2) * S::kKvBlock + (c & 3) * 32) >> 4), kIdS, c != 0 || part != 0);
            }
            umma_commit(s_full + 8u * (2 * t + (j & 1)));
          }
          umma_commit(k_empty + 8u * ka.slot);
        }
        ka.step(kTwo ? S::kKBufs2 : S::kBufs);
      };
      if (steps > 0 && ok) scores(0);
      for (int j = 0; j < steps && ok; ++j) {
        // the next scores go over the last step's weights, behind the product
        // that reads them
        if (j + 1 < steps) scores(j + 1);
        if (!ok || !(ok = wait(v_full + 8u * va.slot, va.round))) break;
        for (int t = 0; t < tiles; ++t) {
          const int s = 2 * t + (j & 1);
          if (!(ok = wait(p_full + 8u * s, j >> 1))) break;
          umma_fence_after();
          if (one) {
#pragma unroll
            for (int i = 0; i < S::kTokens / 16; ++i)
              umma_f16_ts(tmem + (uint32_t)(S::kOCol + t * D), tmem + (uint32_t)(s * S::kTokens + i * 8),
                          vd + (uint32_t)((va.slot * S::kKvTile + i * 2048) >> 4), kIdO, (j | i) != 0);
            umma_commit(o_done + 8u * t);
          }
        }
        if (ok && one) umma_commit(v_empty + 8u * va.slot);
        va.step(kTwo ? S::kVBufs2 : S::kBufs);
      }
      if (!ok) give_up();
      if (one) umma_commit(drain);
      mbar_wait_bounded(drain, 0, kWaitNs);
    };
    if (two_parts) products(std::true_type());
    else products(std::false_type());
    }
  } else if (warp >= kCodeWarp0) {
    // --------------------------------------------------------------- the codes
    if (S::kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const bool is_v = warp >= kCodeWarp0 + 4;
    const int w = (warp - kCodeWarp0) & 3;
    // eight lanes in turn store eight positions' same piece: all banks
    const int piece = lane / S::kPerWarp, sub = lane % S::kPerWarp;
    const uint8_t* code = (is_v ? p.v : p.k) + piece * 16;
    const __half2* param = (is_v ? p.v_param : p.k_param) + (piece >> 1);
    const uint32_t tiles_at = sbase + (is_v ? off_v : S::kOffK), full = is_v ? v_full : k_full,
                   empty = is_v ? v_empty : k_empty;
    uint32_t* mask = masks + (is_v ? 8 * S::kWords : 0);
    struct Piece {
      uint4 codes;
      uint32_t az;
      bool gone;  // a position that has no page
    };
    // The positions of a warp and pass lie in one page.  Lane l looks up pass l
    // % kPasses of step l / kPasses of the next 32 / kPasses: the vector of
    // their first position.
    constexpr int kAhead = 32 / S::kPasses;
    constexpr uint32_t kNone = 0xFFFFFFFEu, kGone = 0xFFFFFFFFu;  // beyond the end, without a page
    uint32_t vecs = kNone;
    auto look_up = [&](int j) {
      const int at = begin + (j + lane / S::kPasses) * S::kTokens +
                     (lane % S::kPasses * 4 + w) * S::kPerWarp;
      vecs = kNone;
      if (at < end && at + S::kPerWarp > sp.seen) {  // (a page in front of every row's window need not be there)
        const int64_t found = vector_at(p.at, b, at, kvh);
        vecs = (uint32_t)found;
        if (found < 0) record_error(&g_kv4_error, BCQ_ERR_PAGE);
      }
    };
    auto load = [&](Piece (&x)[S::kPasses], int j) {
      if (j % kAhead == 0) look_up(j);
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        uint32_t vec = __shfl_sync(0xFFFFFFFFu, vecs, j % kAhead * S::kPasses + i);
        const int at = begin + j * S::kTokens + (i * 4 + w) * S::kPerWarp + sub;
        x[i].codes = make_uint4(0, 0, 0, 0);
        x[i].az = 0;
        x[i].gone = vec == kGone;
        if (vec < kNone && at < end) {
          vec += (uint32_t)sub;
          x[i].codes = *reinterpret_cast<const uint4*>(code + (uint64_t)vec * (D / 2));
          x[i].az = *reinterpret_cast<const uint32_t*>(param + (uint64_t)vec * G);
        }
      }
    };
    uint32_t to[4];  // where this lane's four words go in a row of eight positions
#pragma unroll
    for (int e = 0; e < 4; ++e)
      to[e] = (uint32_t)((piece >> 1) * S::kKvBlock + (w * S::kPerWarp + sub) * 128) +
              ((uint32_t)(((piece & 1) * 4 + e) ^ ((w * S::kPerWarp + sub) & 7)) << 4);
    // into a tile (kTwo: K's in two parts); for V what is no number becomes zero.
    // The mask word of a pass: lanes of a position without a page (K), or of such
    // a group (V)
    auto store = [&](auto two_type, uint32_t tile, uint32_t* word_at, const Piece (&x)[S::kPasses]) {
      constexpr bool kTwo = decltype(two_type)::value;
#pragma unroll
      for (int i = 0; i < S::kPasses; ++i) {
        uint32_t az = x[i].az;
        const bool odd = odd_half2(az);
        const uint32_t word = __ballot_sync(0xFFFFFFFFu, is_v ? odd : x[i].gone);
        if (lane == 0) {
          word_at[i * 4 + w] = word;
          if (word) sts_f32(sbase + S::kOffOdd, 1.f);
        }
        if (is_v && odd) az = 0;
        const uint4 c = x[i].codes;
        const __half2 f = *reinterpret_cast<const __half2*>(&az);
        const uint32_t row = tile + (uint32_t)(i * 4 * S::kPerWarp * 128);
        if (kTwo) {
          const float2 az32 = __half22float2(f);
          uint4 rest = c;  // (a word after the other: all at once they would not fit the registers)
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            uint4 first, second;
            word_parts(rest.x, az32.x, az32.y, first, second);
            if (odd) second = make_uint4(0, 0, 0, 0);
            const uint32_t at = row + (to[0] ^ ((uint32_t)e << 4));
            sts_v4(at, first);
            sts_v4(at + S::kKvTile, second);
            rest = make_uint4(rest.y, rest.z, rest.w, rest.x);
          }
          continue;
        }
        const __half2 a = __low2half2(f), z = __high2half2(f);
        const uint4 v[4] = {word_values(c.x, a, z), word_values(c.y, a, z), word_values(c.z, a, z),
                            word_values(c.w, a, z)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sts_v4(row + to[e], v[e]);
      }
      fence_proxy_async_smem();
    };
    // a step's codes are asked for a step ahead
    bool ok = true;
    auto all_steps = [&](auto two_type) {
      RingAt at;
      Piece x[2][S::kPasses];
      auto one_step = [&](int j, Piece (&now)[S::kPasses], Piece (&next)[S::kPasses]) {
        load(next, j + 1);
        if (at.round > 0 && !(ok = wait(empty + 8u * at.slot, at.round - 1))) return;
        store(two_type, tiles_at + (uint32_t)at.slot * (is_v ? S::kKvTile : k_step), mask + (j & 7) * S::kWords, now);
        __syncwarp();
        if (lane == 0) mbar_arrive_cta(full + 8u * at.slot);
        at.step(is_v ? v_bufs : k_bufs);
      };
      load(x[0], 0);
      for (int j = 0; j < steps && ok; j += 2) {
        one_step(j, x[0], x[1]);
        if (ok && j + 1 < steps) one_step(j + 1, x[1], x[0]);
      }
    };
    // (a choice within the loop: 152 -> 193 us for 2048 rows of 256 over 4096)
    if (two_parts && !is_v) all_steps(std::true_type());
    else all_steps(std::false_type());
    if (!ok) give_up();
  } else {
    // -------------------------------------------------------------- the softmax
    if (S::kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    if (warp < 4 * tiles) {
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;  // tile, row of it
    const int row = t * 128 + r;
    const bool live = row < row_n;
    const int i = live ? p.group.quotient(row0 + row) : 0;
    const int h = live ? (kvh - i) * p.group.d + row0 + row : 0;
    const int64_t token = sp.first_row + i;
    const int pos = sp.pos0 + i;
    const int hi = live ? (p.causal ? min(end, pos + 1) : end) : 1 << 30;
    const int lo = live && p.window > 0 ? max(0, pos - p.window + 1) : 0;
    const int hi_all = min(end, __reduce_min_sync(0xFFFFFFFFu, hi)), lo_all = __reduce_max_sync(0xFFFFFFFFu, lo);
    float fs = 0.f, m = -INFINITY, l = 0.f;
    uint32_t poison = 0;  // groups of the output that a seen position makes NaN
    if (steps > 0) {
      // all of a row at once (half, where it is 512 bytes), and again from L1
      const uint16_t* src = p.q + token * p.ld_q + (int64_t)h * p.hd_q;
      constexpr int kBatch = D / 8 < 16 ? D / 8 : 16;
      uint4 raw[kBatch];
      auto fetch = [&](int c0) {
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          raw[c] = make_uint4(0, 0, 0, 0);
          if (live) raw[c] = *reinterpret_cast<const uint4*>(src + (c0 + c) * 8);
        }
      };
      uint32_t top2 = 0;  // |x| by its bits, two at a time
#pragma unroll
      for (int c0 = 0; c0 < D / 8; c0 += kBatch) {
        fetch(c0);
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
          top2 = __vmaxu2(__vmaxu2(__vmaxu2(top2, raw[c].x & 0x7FFF7FFFu), raw[c].y & 0x7FFF7FFFu),
                          __vmaxu2(raw[c].z & 0x7FFF7FFFu, raw[c].w & 0x7FFF7FFFu));
      }
      const float top = bits_to_float<T>(max(top2 & 0xFFFFu, top2 >> 16));  // not finite: power 0
      const int up = row_power(top);
      // (a row with an infinity or a NaN is NaN, also where all of its scores were -infinity)
      const float mul = !(top < INFINITY) ? __uint_as_float(0x7FC00000u)
                        : p.scale < 0.f ? -power_of_two(up) : p.scale == 0.f ? 0.f : power_of_two(up);
      fs = score_factor(p.scale, -up);
      const uint32_t to = sbase + (uint32_t)t * S::kQTile + (uint32_t)r * 128u;
#pragma unroll
      for (int c0 = 0; c0 < D / 8; c0 += kBatch) {
        if (D / 8 > kBatch) fetch(c0);
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
          const uint32_t x[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[e] = bits_to_float<T>((x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * mul;
          const int at8 = c0 + c;
          const uint32_t at = to + (uint32_t)(at8 >> 3) * S::kQBlock + (uint32_t)(((at8 & 7) ^ (r & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack_f16(f[0], f[4])),
                       "r"(pack_f16(f[1], f[5])), "r"(pack_f16(f[2], f[6])), "r"(pack_f16(f[3], f[7]))
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(q_full);
    }
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts0 = tmem + lanes + (uint32_t)(2 * t * S::kTokens), to = tmem + lanes + (uint32_t)(S::kOCol + t * D);
    // whether position `token` of a step's mask words is marked, for piece q
    auto marked = [&](const uint32_t* word, int token, int q) {
      const int at = token / S::kPerWarp;
      return (word[at] >> (q * S::kPerWarp + token % S::kPerWarp)) & 1u;
    };
    // Once something is odd (the words are rarely looked at): V's groups of step
    // j.  Its flag and its words are there once its product is (the scores of
    // step j + 1 say nothing of them: they are issued before V of step j is
    // waited for), so this stands behind o_done's round j and reads the flag anew.
    auto look_for_nan = [&](int j) {
      const uint32_t* word = masks + (8 + (j & 7)) * S::kWords;
      const uint32_t* gone = masks + (j & 7) * S::kWords;
      for (int k = 0; k < S::kTokens; ++k) {
        const int at = begin + j * S::kTokens + k;
        if (at < lo || at >= min(hi, end) || marked(gone, k, 0)) continue;
        for (int g = 0; g < G; ++g)
          if (marked(word, k, 2 * g)) poison |= 1u << g;
      }
    };
    // The two tiles' warps of a scheduler take turns at the exponentials, which
    // have a unit to themselves there: one's other work runs beside the other's.
    // (Left alone they go in step, and the unit stands idle for both.)  Barrier
    // 1 + 2 q + t is tile t's turn.
    const bool turns = tiles == 2;
    auto take_turn = [&]() {
      if (turns) named_barrier_sync(1 + 2 * (warp & 3) + t, 64);
    };
    auto give_turn = [&]() {
      if (turns) asm volatile("bar.arrive %0, 64;" ::"r"(1 + 2 * (warp & 3) + (t ^ 1)) : "memory");
    };
    if (steps > 0 && t == 1) give_turn();
    int taken = 0;
    bool ok = true, there = false;  // there: the next scores, seen ahead
    for (int j = 0; j < steps; ++j) {
      const uint32_t ts = ts0 + (uint32_t)((j & 1) * S::kTokens);
      if (!__all_sync(0xFFFFFFFFu, there) &&
          !(ok = wait(s_full + 8u * (2 * t + (j & 1)), j >> 1)))
        break;
      umma_fence_after();
      // shared memory answers slowly while the tensor core reads its operands
      // there: what is not needed at once is asked for ahead of the scores
      const uint32_t odd = lds_u32v(sbase + S::kOffOdd);
      uint32_t s[2][32];
      tmem_ld32(ts, s[0]);
      tmem_ld32(ts + 32, s[1]);
      tmem_wait_ld();
      const bool holes = __any_sync(0xFFFFFFFFu, odd != 0);
      const int j0 = begin + j * S::kTokens;
      const uint32_t* gone = masks + (j & 7) * S::kWords;
      if (holes || j0 < lo_all || j0 + S::kTokens > hi_all) {
#pragma unroll
        for (int k = 0; k < 64; ++k) {
          const int at = j0 + k;
          if (at < lo || at >= min(hi, end) || (holes && marked(gone, k, 0))) s[k >> 5][k & 31] = 0xFF800000u;
        }
      }
      float x4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < 64; k += 2)
        x4[(k >> 1) & 3] = max3(x4[(k >> 1) & 3], __uint_as_float(s[k >> 5][k & 31]),
                                __uint_as_float(s[k >> 5][(k & 31) + 1]));
      const float now = fmaxf(fmaxf(x4[0], x4[1]), fmaxf(x4[2], x4[3])) * fs;
      const bool moved = now > m + 8.f;  // the first finite maximum moves from -infinity
      bool behind = j == 0;  // the last step's product has been waited for
      if (__any_sync(0xFFFFFFFFu, moved)) {
        const float f = moved ? ex2(m - now) : 1.f;
        if (j > 0) {
          if (!(ok = wait(o_done + 8u * t, j - 1))) break;
          behind = true;
          umma_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(to + (uint32_t)c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(to + (uint32_t)c, o);
          }
        }
        if (moved) {
          l *= f;
          m = now;
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      const uint64_t fs2 = pack_f32x2(fs, fs), base2 = pack_f32x2(kManyBits - base, kManyBits - base);
      uint64_t sum2[2] = {0, 0};
      take_turn();
      ++taken;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float x, y;
          unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])),
                                 fs2, base2),
                       x, y);
          x = ex2(x);
          y = ex2(y);
          sum2[k & 1] = add_f32x2(sum2[k & 1], pack_f32x2(x, y));
          w[k] = pack_f16(x, y);
        }
        tmem_st16(ts + (uint32_t)(16 * c), w);  // over scores that this thread has read
      }
      give_turn();
      there = j + 1 < steps && mbar_test(s_full + 8u * (2 * t + ((j + 1) & 1)), (uint32_t)((j + 1) >> 1) & 1u);
      float sa, sb;
      unpack_f32x2(add_f32x2(sum2[0], sum2[1]), sa, sb);
      l += sa + sb;
      tmem_wait_st();
      umma_fence_before();
      // Each round of a barrier is waited for in turn, this one before the next can
      // end: a wait by parity would take a round that was passed over for one to
      // come.
      if (!behind && !(ok = wait(o_done + 8u * t, j - 1))) break;
      __syncwarp();
      if (lane == 0) mbar_arrive_cta(p_full + 8u * (2 * t + (j & 1)));
      if (j > 0 && __any_sync(0xFFFFFFFFu, lds_u32v(sbase + S::kOffOdd) != 0)) look_for_nan(j - 1);
    }
    for (; taken < steps; ++taken) {  // after a wait that ran out: the other tile's warp has its turns
      take_turn();
      give_turn();
    }
    if (steps > 0 && ok) {
      ok = wait(o_done + 8u * t, steps - 1);
      umma_fence_after();
      if (ok && lds_u32v(sbase + S::kOffOdd)) look_for_nan(steps - 1);
    }
    if (!ok) {
      give_up();
    } else {
      // ------------------------------------------------------------ the outputs
      const bool none = m == -INFINITY && l == 0.f, split = sp.parts > 1;
      constexpr float kPartScale = kWeightScale / 128.f;  // a part's weights are held as the few-row kernel's
      const float inv = none ? 0.f : split ? kPartScale : 1.f / l;
      const int64_t at = ((int64_t)part * p.T + token) * p.q_heads + h;
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        __syncwarp();
        if (steps > 0) {
          tmem_ld32(to + (uint32_t)c, o);
          tmem_wait_ld();
        }
        const bool bad = (poison >> (c / kKvGroup)) & 1u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = none ? 0.f : __uint_as_float(o[8 * e + k]) * inv;
            y[(k >> 1) + 4 * (k & 1)] = bad ? __uint_as_float(0x7FC00000u) : x;
          }
          if (!live) continue;
          if (split) {
            float4* to4 = reinterpret_cast<float4*>(p.part + at * D + c + 8 * e);
            to4[0] = make_float4(y[0], y[1], y[2], y[3]);
            to4[1] = make_float4(y[4], y[5], y[6], y[7]);
          } else {
            union {
              T v[8];
              uint4 q;
            } u;
#pragma unroll
            for (int k = 0; k < 8; ++k) u.v[k] = from_float<T>(y[k]);
            *reinterpret_cast<uint4*>(p.out + token * p.ld_o + (int64_t)h * p.hd_o + c + 8 * e) = u.q;
          }
        }
      }
      if (live && split) {
        float* ml = p.part + (int64_t)p.splits * p.T * p.q_heads * D + at * 2;
        ml[0] = m;
        ml[1] = l * kPartScale;
      } else if (live && p.lse) {
        p.lse[token * p.q_heads + h] = none ? -INFINITY : (m + log2f(l) - kManyBits) * 0.69314718055994531f;
      }
    }
  }
  }
  launch_dependents();
  __syncwarp();
  umma_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    umma_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace
}  // namespace bcq

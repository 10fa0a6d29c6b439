// bcq_kv4.cu -- the key/value cache in 4 bits: rows into the cache, rows out
// of it, and attention over it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bcq.h"
#include "bcq_device.cuh"
#include "bcq_f32x2.cuh"
#include "bcq_launch.h"

namespace bcq {
namespace {

__device__ int g_kv4_error = 0;

constexpr int kKvGroup = BCQ_KV4_GROUP;
constexpr float kKvRange = 60000.f;  // beyond it a group becomes NaN: a c + z stays below fp16's 65504

// ------------------------------------------------------------------ types

template <typename T>
__device__ __forceinline__ float bits_to_float(uint32_t b);
template <>
__device__ __forceinline__ float bits_to_float<__half>(uint32_t b) { return h2f((uint16_t)b); }
template <>
__device__ __forceinline__ float bits_to_float<__nv_bfloat16>(uint32_t b) {
  return __uint_as_float(b << 16);
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Division of 0 <= n < 2^31 by a number that the host knows, as a product (a
// division takes some 35 instructions): with s = ceil(log2 d) and m = ceil(2^(31
// + s) / d), n m / 2^(31 + s) exceeds n / d by less than n / 2^31 / d < 1 / d.
struct Divisor {
  int d;
  uint32_t m;
  int shift;  // s - 1
  __device__ __forceinline__ int quotient(int n) const {
    return d == 1 ? n : (int)(__umulhi((uint32_t)n, m) >> shift);
  }
};

// What a call knows of the cache's places.
struct Places {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  int table_width, B, pages, page_size, heads;
  int room;             // positions of a table row
  Divisor by_page;
};

// The sequence that row t belongs to: the last b with cu[b] <= t, or -1 when
// t is outside cu[0]..cu[B]-1.  Without cu, row t is sequence t's.
__device__ __forceinline__ int sequence_of(const Places& p, int t) {
  if (!p.cu) return t < p.B ? t : -1;
  if (t < p.cu[0] || t >= p.cu[p.B]) return -1;
  int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// First row and number of rows of sequence b.
__device__ __forceinline__ int2 rows_of(const Places& p, int b) {
  return p.cu ? make_int2(p.cu[b], p.cu[b + 1] - p.cu[b]) : make_int2(b, 1);
}

// The vector of position j of sequence b, head h, as an index into [pages]
// [heads][page_size]; -1 where the cache has none.  (A cache has fewer than
// 2^32 vectors: one takes 72 bytes or more.)
__device__ __forceinline__ int64_t vector_at(const Places& p, int b, int j, int h) {
  if (j < 0) return -1;
  if (j >= p.room) return -1;
  const int entry = p.by_page.quotient(j);
  const int page = p.table[(int64_t)b * p.table_width + entry];
  if (page < 0 || page >= p.pages) return -1;
  return (int64_t)((uint64_t)((uint32_t)page * (uint32_t)p.heads + (uint32_t)h) * (uint32_t)p.page_size) +
         (j - entry * p.page_size);
}

// --------------------------------------------------- rows in, rows out

constexpr int kRowThreads = 256;

// Where `rows` <= kRows rows from t0 on go, found by the whole block: place[i] = index of
// the vector of head 0 (the other heads' lie page_size apart), -1 for a
// position that the cache does not have, -2 for a row of no sequence.  Two
// loads one after the other: the sequences' first rows and lengths (up to 256
// of them, the usual case, kept in shared memory), then the table.
template <int kRows>
struct RowPlaces {
  int64_t place[kRows];
  int count[kRows];
  int cu[kRowThreads + 1], len[kRowThreads];
};
template <int kRows>
__device__ __forceinline__ void locate_rows(const Places& p, int t0, int T, int rows, RowPlaces<kRows>& s) {
  const int tid = threadIdx.x;
  const bool kept = p.B <= kRowThreads;
  if (p.cu) {
    if (tid < rows) s.count[tid] = 0;
    if (kept) {
      if (tid == 0) s.cu[0] = p.cu[0];
      if (tid < p.B) s.len[tid] = p.kv_len[tid];
    }
    __syncthreads();
    // row t's sequence: how many of cu[1..B] are not above t
    for (int b0 = 1; b0 <= p.B; b0 += kRowThreads) {
      const int end = b0 + tid <= p.B ? p.cu[b0 + tid] : INT32_MAX;
      if (kept && b0 + tid <= p.B) s.cu[b0 + tid] = end;
#pragma unroll 4
      for (int i = 0; i < rows; ++i) {
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, end <= t0 + i));
        if ((tid & 31) == 0 && n) atomicAdd(&s.count[i], n);
      }
    }
    __syncthreads();
  }
  if (tid < rows) {
    const int t = t0 + tid;
    int64_t at = -2;
    const int b = p.cu ? s.count[tid] : t;
    if (t < T && b < p.B && (!p.cu || t >= (kept ? s.cu[0] : p.cu[0]))) {
      int first = t, n = 1, len;
      if (p.cu && kept) {
        first = s.cu[b];
        n = s.cu[b + 1] - first;
        len = s.len[b];
      } else {
        const int2 rows = rows_of(p, b);
        first = rows.x;
        n = rows.y;
        len = p.kv_len[b];
      }
      at = vector_at(p, b, len - n + (t - first), 0);
    }
    if (at == -1) record_error(&g_kv4_error, BCQ_ERR_PAGE);
    s.place[tid] = at;
  }
  __syncthreads();
}

// Where a row has few words (few heads, small ones) a block's threads are shared
// out among `sets` of kRows rows each: as many as fit, a power of two.
constexpr int kMostSets = 16;  // a row has 16 words at least
__device__ __host__ __forceinline__ int row_sets(int items) {
  int sets = 1;
  while (2 * sets * items <= kRowThreads) sets *= 2;
  return sets;
}

struct AppendParams {
  Places at;
  const uint16_t* x[2];  // K, V
  int64_t ld[2], hd[2];
  uint8_t* code[2];
  __half2* param[2];
  int T;
};

template <typename T>
struct Pair16;  // two values of a 16-bit type
template <>
struct Pair16<__half> {
  using V = __half2;
};
template <>
struct Pair16<__nv_bfloat16> {
  using V = __nv_bfloat162;
};

// Rows in: z = fp16(lo), a = fp16((hi - lo) / 15), c = (x - z) / a of each group.
// A block takes kRows rows, whose values it asks for before it knows their
// places; eight lanes a group of 64, eight values a lane, one 32-bit word of
// codes.  Least and greatest come from packed 16-bit compares that keep a NaN.
// (hi - lo) / 15 is a product with fp32(1 / 15) and Markstein's correction by
// the remainder, which gives the correctly rounded quotient.  A code's quotient
// is taken in fp32 with an approximate reciprocal, clamped by the saturation of
// its fifteenth to 0..1, and rounded by adding 1.5 2^23; conversions, which
// run at an eighth of the rate, are left out, and four codes become 16 bits by
// fused multiply-adds.  Where a quotient lies within 1e-4 of a half (its error is
// below 16 * 6 * 2^-24 < 6e-6, and the difference's rounding adds less) the
// half decides in fp64, where x - z and (c + 1/2) a are exact.
// Bound by its instructions, some 200 for 256 values: 8 x 1024 rows of 8 heads
// of 128 take 15.1 us (43 MB, 2.8 TB/s), 64 rows 3.0 us (launch, and four loads
// one after the other).
template <typename T, int D, int kRows, bool SHARED>
__global__ void __launch_bounds__(kRowThreads, 4) kv4_append_kernel(const AppendParams p) {
  using V = typename Pair16<T>::V;
  constexpr int G = D / kKvGroup, kWords = D / 8;
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, halves to even
  __shared__ RowPlaces<SHARED ? kRows * kMostSets : kRows> places;
  const int heads = p.at.heads, items = 2 * heads * kWords;
  const int sets = SHARED ? row_sets(items) : 1, threads = kRowThreads / sets;  // of a set
  const int set = SHARED ? (int)threadIdx.x / threads : 0, first = (int)threadIdx.x - set * threads;
  const int b0 = (int)blockIdx.x * kRows * sets, t0 = b0 + set * kRows;
  uint4 raw[kRows];
  auto fetch = [&](int i) {
    const int kv = i >= heads * kWords, in = kv ? i - heads * kWords : i;
    // (chosen, not indexed: a param array with a thread's index is loaded by the lane)
    const int64_t ld = kv ? p.ld[1] : p.ld[0], hd = kv ? p.hd[1] : p.hd[0];
    const uint16_t* x = (kv ? p.x[1] : p.x[0]) + (int64_t)(in / kWords) * hd + in % kWords * 8 + t0 * ld;
#pragma unroll
    for (int j = 0; j < kRows; ++j, x += ld) {
      raw[j] = make_uint4(0, 0, 0, 0);
      if (t0 + j < p.T && i < items) raw[j] = ldg_nc_v4(x);
    }
  };
  grid_dependency_wait();
  launch_dependents();
  fetch(first);
  locate_rows(p.at, b0, p.T, kRows * sets, places);
  const int lane = threadIdx.x & 31;
  for (int i = first; SHARED ? i == first : i - lane < items; i += threads) {  // whole warps
    const int kv = i >= heads * kWords, in = kv ? i - heads * kWords : i;
    const int h = in / kWords, word = in % kWords;
    if (i != first) fetch(i);
    uint8_t* const code = (kv ? p.code[1] : p.code[0]) + word * 4;
    __half2* const param = (kv ? p.param[1] : p.param[0]) + word / 8;
    const int64_t to_head = (int64_t)h * p.at.page_size;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t place = places.place[set * kRows + j];
      if (!SHARED && place < 0) continue;  // for all of the block
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
      const V* v2 = reinterpret_cast<const V*>(w);
      const V lo2 = __hmin2_nan(__hmin2_nan(v2[0], v2[1]), __hmin2_nan(v2[2], v2[3]));
      const V hi2 = __hmax2_nan(__hmax2_nan(v2[0], v2[1]), __hmax2_nan(v2[2], v2[3]));
      V ends;  // (lo, -hi): the least of both
      ends.x = __hmin_nan(lo2.x, lo2.y);
      ends.y = __hneg(__hmax_nan(hi2.x, hi2.y));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) ends = __hmin2_nan(ends, __shfl_xor_sync(0xFFFFFFFFu, ends, o));
      const float lo = (float)ends.x, hi = -(float)ends.y;
      const bool ok = lo >= -kKvRange && hi <= kKvRange;  // false for a NaN
      const float d = __fsub_rn(hi, lo), r15 = 1.f / 15.f;
      const float q15 = __fmul_rn(d, r15);
      const __half a16 = __float2half_rn(__fmaf_rn(__fmaf_rn(q15, -15.f, d), r15, q15));
      const __half z16 = __float2half_rn(lo);
      const float a = __half2float(a16), z = __half2float(z16);
      uint32_t codes = 0;
      if (ok && a > 0.f) {
        const float inv = __fdividef(1.f, a * 15.f);
        float f[8], c[8], off = 0.f;
        const uint64_t minus_z = pack_f32x2(-z, -z), fifteen = pack_f32x2(15.f, 15.f), minus = pack_f32x2(-1.f, -1.f),
                       magic = pack_f32x2(kMagic, kMagic), no_magic = pack_f32x2(-kMagic, -kMagic);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          f[e] = bits_to_float<T>(w[e >> 1] & 0xFFFFu);
          f[e + 1] = bits_to_float<T>(w[e >> 1] >> 16);
          float x, y;
          unpack_f32x2(add_f32x2(pack_f32x2(f[e], f[e + 1]), minus_z), x, y);
          const uint64_t q = pack_f32x2(__saturatef(x * inv), __saturatef(y * inv));  // of 15
          const uint64_t r = add_f32x2(fma_f32x2(q, fifteen, magic), no_magic);
          unpack_f32x2(r, c[e], c[e + 1]);
          unpack_f32x2(fma_f32x2(q, fifteen, mul_f32x2(r, minus)), x, y);
          off = max3(off, fabsf(x), fabsf(y));
        }
        if (off > 0.4999f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = __saturatef((f[e] - z) * inv) * 15.f;
            if (fabsf(v - c[e]) > 0.4999f) {
              const float below = floorf(v);  // the half in question is below + 1/2
              const double x = (double)f[e] - (double)z, edge = ((double)below + 0.5) * (double)a;
              c[e] = below + (x > edge || (x == edge && ((int)below & 1)) ? 1.f : 0.f);
            }
          }
        }
        const float lo16 = fmaf(c[3], 4096.f, fmaf(c[2], 256.f, fmaf(c[1], 16.f, c[0])));
        const float hi16 = fmaf(c[7], 4096.f, fmaf(c[6], 256.f, fmaf(c[5], 16.f, c[4])));
        codes = prmt(__float_as_uint(lo16 + 8388608.f), __float_as_uint(hi16 + 8388608.f), 0x5410);
      }
      if (i >= items || place < 0) continue;
      const int64_t vec = place + to_head;
      *reinterpret_cast<uint32_t*>(code + vec * (D / 2)) = codes;
      if (word % 8 == 0) {
        const __half nan = __ushort_as_half(0x7E00);
        param[vec * G] = ok ? __halves2half2(a16, z16) : __halves2half2(nan, nan);
      }
    }
  }
}

struct ReadParams {
  Places at;
  const uint8_t* code[2];
  const __half2* param[2];
  void* y[2];
  int T;
};

// Rows out: a c + z.  Eight values (one word of codes) a thread and row, its
// four rows' loads in flight together.  Bound by memory from some thousand rows
// on: 8 x 1024 rows of 8 heads of 128 as fp16 8.2 us (43 MB, 5.2 TB/s), 64 rows
// 2.7 us.
template <typename TO, int D, int kRows, bool SHARED>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const ReadParams p) {
  constexpr int G = D / kKvGroup, kWords = D / 8;
  __shared__ RowPlaces<SHARED ? kRows * kMostSets : kRows> places;
  const int heads = p.at.heads, items = 2 * heads * kWords;
  const int sets = SHARED ? row_sets(items) : 1, threads = kRowThreads / sets;  // of a set
  const int set = SHARED ? (int)threadIdx.x / threads : 0, first = (int)threadIdx.x - set * threads;
  const int b0 = (int)blockIdx.x * kRows * sets, t0 = b0 + set * kRows;
  const int64_t* place = places.place + set * kRows;
  grid_dependency_wait();
  launch_dependents();
  locate_rows(p.at, b0, p.T, kRows * sets, places);
  for (int i = first; i < items; i += threads) {
    const int kv = i >= heads * kWords;
    const int in = kv ? i - heads * kWords : i;
    const int h = in / kWords, word = in % kWords;
    const uint8_t* const code = (kv ? p.code[1] : p.code[0]) + 4 * word;
    const __half2* const param = (kv ? p.param[1] : p.param[0]) + word / 8;
    const int64_t to_head = (int64_t)h * p.at.page_size;
    uint32_t codes[kRows];
    __half2 az[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      codes[j] = 0;
      az[j] = __floats2half2_rn(0.f, 0.f);
      if (place[j] >= 0) {
        const int64_t vec = place[j] + to_head;
        codes[j] = *reinterpret_cast<const uint32_t*>(code + vec * (D / 2));
        az[j] = param[vec * G];
      }
    }
    TO* y = static_cast<TO*>(kv ? p.y[1] : p.y[0]) + ((int64_t)t0 * heads + h) * D + 8 * word;
#pragma unroll
    for (int j = 0; j < kRows; ++j, y += (int64_t)heads * D) {
      if (place[j] == -2) continue;
      const float2 f = __half22float2(az[j]);
      union {
        TO v[8];
        uint4 q[8 * sizeof(TO) / 16];
      } out;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // 2^23 + c by its bits, instead of a conversion
        const float c = __uint_as_float(0x4B000000u | ((codes[j] >> (4 * e)) & 15u)) - 8388608.f;
        out.v[e] = from_float<TO>(fmaf(c, f.x, f.y));
      }
#pragma unroll
      for (int e = 0; e < (int)(8 * sizeof(TO) / 16); ++e) reinterpret_cast<uint4*>(y)[e] = out.q[e];
    }
  }
}

// --------------------------------------------------------------- attention

// Attention of few rows a key/value head: decode steps, drafts, short chunks.
//
// A warp takes 32 positions at a time, the codes as they lie in the cache.  A
// nibble masked out of a word is the fp16 subnormal c 2^-24 (the high one of a
// byte c 2^-20), which the tensor core multiplies exactly, so a code becomes
// an operand by one AND, without a conversion, a scale or an offset: those are
// applied to the results (for V, whole bytes low + 16 high stand in for the
// high codes, one operation less; their sums' difference from the low codes'
// over 16 is the high codes' sum),
//   q . K_t = sum_g  a_tg (sum_{d in g} q_d c_td) + z_tg (sum_{d in g} q_d)
//   out_d   = sum_t (p_t a_tg) c_td + sum_t p_t z_tg,
// a few operations a position instead of one a value; the two sums with the
// offsets are one more instruction of the tensor core each (the sums of q as
// two fp16 parts, so to 2^-22).  Both products have the codes as the first
// operand of mma.m16n8k16 (16 positions, or 16 values of a vector; one 32-bit
// word of codes fills the four registers) and 8 rows as the second, so 8 rows
// of a key/value head (the query heads that share it, times the rows of the
// call) fill an instruction.  Queries are scaled by a power of two to the top
// of fp16's range.  p and p a are rounded to fp16 (half a step, 2^-11, each).
// So that neither falls among fp16's subnormals, whose step does not shrink with
// them: the maximum in use follows a row's own only when that has risen by more
// than 2^4, and p is held times 2^9, so it is at most 2^13 and keeps its 11 bits
// down to 2^-23 of the row's largest; and a is taken times a power of two that a
// warp has for each group, which brings the largest a among its positions so far
// to 1/2 .. 2 (p a' is below 2^15 then, and keeps its bits where a is not below
// 2^-13 of that largest; further down it is off by 2^-24 of the largest at most).
// The power follows a larger a as the maximum in use follows a score, with one
// look a stage, and is taken out of the sums at the end.  Scores, sums and outputs
// are fp32.
//
// A scale or offset of V that is no number must not reach rows that do not see
// its position (0 * NaN): where some row does not see all positions such
// values become zeros, and the rows that see them are told to write NaN.
//
// The codes' way: cp.async into a ring of three stages a warp (nobody else
// reads them, so no barrier but the warp's own), 16-byte pieces placed so that
// the fragment loads have no bank conflicts.  A long sequence is split over
// CTAs, whose partial results a second kernel joins in order.
//
// What bounds it: with all SMs busy the ALU pipe (masks and permutes of codes,
// some 55 %, beside 90 % of the memory's rate in the steady state) -- a row over
// 524288 positions takes 120 us (5.0 TB/s), 64 rows over up to 8192 each, ragged,
// 86.6 us (3.8 TB/s); below that a CTA's start (page table, then codes, some 3
// us) and the joining kernel: 131072 positions 38.5 us, 4001 positions 8.0 us.
// The looks at V's scales and their powers are 2 to 4 % of that.  (A second product
// with what the rounding of p a leaves, the codes' operands being there, would
// bring fp16 outputs of decode steps from 5.8e-4 of their norm to 3.1e-4, an
// output's own rounding being 2.1e-4, and take 2 to 11 % more: 64 rows 95.1 us.)
// Four CTAs of four warps an SM hide one another's loads: the registers of a
// thread (128) leave no more, and three stages of 32 positions a warp are what
// shared memory has room for.
struct AttentionParams {
  Places at;
  const uint8_t* k;
  const __half2* k_param;
  const uint8_t* v;
  const __half2* v_param;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t ld_q, hd_q, ld_o, hd_o;
  int T, q_heads, max_q, causal, window;
  float scale;
  Divisor group;   // query heads a key/value head
  Divisor by_blocks, by_heads, by_rows;  // row_blocks, the cache's heads, rows
  int rows;        // rows (of a key/value head) a CTA
  int row_blocks;  // CTAs along max_q * group rows
  int splits;      // most CTAs along the positions
  int chunk;       // positions of one, at least
  float* part;     // [splits][T][q_heads][D], then (max, sum) [splits][T][q_heads]
};

// The positions that a block of rows sees, and how they are split.
struct Span {
  int first_row, rows;   // of the sequence in the call
  int len;               // tokens in the cache, within the table
  int pos0;              // position of the sequence's first row
  int seen, end;         // positions seen by some row of the block
  int begin;             // seen, down to a multiple of 32
  int chunk, parts;      // positions a part, parts
};

__device__ __forceinline__ Span span_of(const AttentionParams& p, int b, int block) {
  Span s;
  const int2 r = rows_of(p.at, b);
  s.first_row = r.x;
  s.rows = r.x < 0 ? 0 : min(min(r.y, p.max_q), p.T - r.x);
  const int len = p.at.kv_len[b];
  s.len = min(max(len, 0), p.at.room);
  s.pos0 = len - r.y;
  const int i0 = p.group.quotient(block * p.rows);                          // first and last row
  const int i1 = min(s.rows - 1, p.group.quotient((block + 1) * p.rows - 1));  // (of the sequence)
  s.end = p.causal ? min(s.len, s.pos0 + i1 + 1) : s.len;
  s.seen = p.window > 0 ? max(0, s.pos0 + i0 - p.window + 1) : 0;
  s.begin = s.seen & ~31;
  const int n = s.end - s.begin;
  if (i0 >= s.rows || n <= 0) {
    s.parts = i0 < s.rows ? 1 : 0;  // rows that see nothing are still written
    s.chunk = 0;
    s.end = s.begin;
    return s;
  }
  if (n <= p.chunk) {
    s.chunk = p.chunk;
    s.parts = 1;
    return s;
  }
  const int even = (n + p.splits - 1) / p.splits;
  s.chunk = max(p.chunk, (even + 127) & ~127);
  s.parts = (n + s.chunk - 1) / s.chunk;
  return s;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16, fp16) x B (16 x 8, fp16).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same into a fresh D.
__device__ __forceinline__ void mma16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Transpose of an 8 x 8 matrix of 16-bit values, two a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float half_low(uint32_t bits) { return h2f((uint16_t)bits); }
__device__ __forceinline__ uint32_t mul_half2(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Halves that are no finite numbers, as zeros.
__device__ __forceinline__ uint32_t finite_half2(uint32_t x) {
  if ((x & 0x7C00u) == 0x7C00u) x &= 0xFFFF0000u;
  if ((x & 0x7C000000u) == 0x7C000000u) x &= 0x0000FFFFu;
  return x;
}
__device__ __forceinline__ bool odd_half2(uint32_t x) {
  return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds_u32v(addr);
  } else if constexpr (N == 2) {
    const uint2 v = lds_v2u(addr);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = lds_v4(addr);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// 2^n for -126 <= n <= 127.
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }
// The power that brings a row whose largest magnitude is `top` to the top of
// fp16's range: 2^14 <= top 2^n < 2^15 (n at most 126; 0 for no finite top).
__device__ __forceinline__ int row_power(float top) {
  if (!(top > 0.f && top < INFINITY)) return 0;
  return min(126, 141 - (int)(__float_as_uint(top) >> 23));
}
// What makes such a row's products scores in powers of two: |scale| log2(e)
// 2^n.  Never zero, so that a hidden score stays at -infinity.
__device__ __forceinline__ float score_factor(float scale, int n) {
  if (scale == 0.f) return 1.f;  // the row itself is taken times zero
  const int h = n / 2;
  return fmaxf(fabsf(scale) * 1.4426950408889634f * power_of_two(h) * power_of_two(n - h), 1e-37f);
}

constexpr int kFewWarps = 4;    // of a CTA
constexpr int kFewStages = 3;   // of a warp's ring
constexpr int kFewTokens = 32;  // of a stage
constexpr float kWeightBits = 9.f;    // p is held times 2^9
constexpr float kWeightScale = 512.f;
constexpr float kLazyBits = 4.f;      // how far a row's maximum may rise over the one in use
constexpr int kFewSeen = 512;         // below so many positions the many-row kernel has keys in two parts
constexpr uint32_t kFirstPower = 30u << 10;  // 2^15, of V's scales, by the bits of an fp16

template <int D>
struct FewShape {
  static constexpr int kGroups = D / kKvGroup;
  static constexpr int kRow = D / 2;                         // bytes of a vector's codes
  static constexpr int kPieces = kRow / 16;                  // 16-byte pieces of it
  static constexpr uint32_t kCodes = 16 * kRow;              // of 16 positions, K or V
  static constexpr uint32_t kParam = 16 * kGroups * 4;
  static constexpr uint32_t kHalf = 2 * kCodes + 2 * kParam; // 16 positions: K, V, their params
  static constexpr uint32_t kStage = 2 * kHalf;
  static constexpr uint32_t kRing = kFewStages * kStage;     // of a warp
  // where piece `piece` of row `row` of 16 lies: four rows in turn take four
  // different 32-byte parts of the banks
  static __device__ __forceinline__ uint32_t place(int row, int piece) {
    const int f = kGroups == 1 ? 0 : kGroups == 2 ? (row >> 1) & 1 : row & 3;
    return (uint32_t)(row * kRow + ((piece ^ (f << 1)) << 4));
  }
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kFewWarps * 32, NT == 1 && D <= 128 ? 4 : 2) kv4_few_kernel(const AttentionParams p) {
  using S = FewShape<D>;
  constexpr int G = S::kGroups;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const int pair = p.by_blocks.quotient((int)blockIdx.x), block = (int)blockIdx.x - pair * p.row_blocks;
  const int b = p.by_heads.quotient(pair), kvh = pair - b * p.at.heads, part = blockIdx.y;
  grid_dependency_wait();
  const Span sp = span_of(p, b, block);
  if (part == 0 && block == 0 && kvh == 0 && threadIdx.x == 0) {
    if (rows_of(p.at, b).y > p.max_q) record_error(&g_kv4_error, BCQ_ERR_SHAPE);
    if (p.at.kv_len[b] != sp.len) record_error(&g_kv4_error, BCQ_ERR_PAGE);
  }
  if (part >= sp.parts) return;
  const int row0 = block * p.rows;                       // of the key/value head's rows
  const int row_n = min(p.rows, sp.rows * p.group.d - row0);

  // the queries are asked for before the cache is
  uint4 raw_q[NT][G][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 8 + r, i = p.group.quotient(row);
    const uint16_t* src = p.q + (int64_t)(sp.first_row + i) * p.ld_q +
                          (int64_t)((kvh - i) * p.group.d + row) * p.hd_q;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        raw_q[nt][g][w] = make_uint4(0, 0, 0, 0);
        if (nt * 8 + r < row_n) raw_q[nt][g][w] = ldg_nc_v4(src + g * kKvGroup + (2 * c + w) * 8);
      }
  }

  // ---- the positions
  const int begin = sp.begin + part * sp.chunk, end = min(sp.end, begin + sp.chunk);
  const int stages = (end - begin + kFewTokens - 1) / kFewTokens;
  const int mine = stages > warp ? (stages - warp + kFewWarps - 1) / kFewWarps : 0;
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * S::kRing;
  uint32_t vecs = 0xFFFFFFFFu;  // lane l: first vector of half l & 1 of stage (l >> 1) of the next 16
  auto look_up = [&](int s) {   // page table entries of stages s .. s + 15
    const int j = begin + ((s + (lane >> 1)) * kFewWarps + warp) * kFewTokens + (lane & 1) * 16;
    vecs = 0xFFFFFFFFu;
    if (j < end && j + 16 > sp.seen) {  // (a page in front of every row's window need not be there)
      const int64_t vec = vector_at(p.at, b, j, kvh);
      if (vec >= 0) vecs = (uint32_t)vec;
      else record_error(&g_kv4_error, BCQ_ERR_PAGE);
    }
  };
  // this lane's pieces of 16 positions, from and to (V's rows in the order 0, 2,
  // 4, 6, 1, 3, 5, 7, and so the next 8); of the params, K's or V's
  uint32_t k_to[S::kPieces / 2], v_to[S::kPieces / 2];
#pragma unroll
  for (int i = 0; i < S::kPieces / 2; ++i) {
    const int id = i * 32 + lane, row = id / S::kPieces, piece = id % S::kPieces;
    k_to[i] = S::place(row, piece);
    v_to[i] = S::kCodes + S::place((row & 8) | ((row & 1) << 2) | ((row >> 1) & 3), piece);
  }
  const bool is_vp = lane >= 4 * G;
  const uint32_t p_to = 2 * S::kCodes + (is_vp ? S::kParam : 0u) + (uint32_t)(lane & (4 * G - 1)) * 16u;
  const uint8_t* k_from = p.k + lane * 16;
  const uint8_t* v_from = p.v + lane * 16;
  const uint8_t* p_from =
      reinterpret_cast<const uint8_t*>(is_vp ? p.v_param : p.k_param) + (lane & (4 * G - 1)) * 16;
  int fill = 0;      // the ring's next stage
  uint32_t bad = 0;  // two bits a stage of the ring: halves that have no page
  auto fetch = [&](int s) {
    if (s < mine) {
      if ((s & 15) == 0) look_up(s);
      const int slot = fill;
      fill = fill + 1 == kFewStages ? 0 : fill + 1;
      const uint32_t to = ring + (uint32_t)slot * S::kStage;
      bad &= ~(3u << (2 * slot));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t vec = __shfl_sync(0xFFFFFFFFu, vecs, 2 * (s & 15) + half);
        if (vec == 0xFFFFFFFFu) {
          bad |= 1u << (2 * slot + half);
          continue;
        }
        const uint8_t* k = k_from + (uint64_t)vec * S::kRow;
        const uint8_t* v = v_from + (uint64_t)vec * S::kRow;
        const uint32_t at = to + (uint32_t)half * S::kHalf;
#pragma unroll
        for (int i = 0; i < S::kPieces / 2; ++i) {
          cp_async16(at + k_to[i], k + i * 512);
          cp_async16(at + v_to[i], v + i * 512);
        }
        if (lane < 8 * G) {
          cp_async16(at + p_to, p_from + (uint64_t)vec * (G * 4));
        }
      }
    }
    cp_async_commit();
  };
  // the first stages are on their way while the queries are made ready
  for (int s = 0; s < kFewStages - 1; ++s) fetch(s);

  // ---- queries: lane (r, c) holds row r's values that its codes will meet
  uint32_t qf[NT][G][2][4];
  uint32_t qz[NT];  // sums over the groups, as two fp16 parts, over 2^7
  float fs[NT][2];
  int hi[NT][2], lo[NT][2];
  int hi_all = sp.end, lo_all = sp.begin;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = nt * 8 + r;
    const bool live = row < row_n;
    const int i = live ? p.group.quotient(row0 + row) : 0;
    float f[G][2][8];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 raw = raw_q[nt][g][w];
        const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[g][w][e] = bits_to_float<T>((words[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
          top = fmaxf(top, fabsf(f[g][w][e]));
        }
      }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int up = row_power(top);
    const float mul = p.scale < 0.f ? -power_of_two(up) : p.scale == 0.f ? 0.f : power_of_two(up);
    const float back = score_factor(p.scale, 24 - up);
    float sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sum[g] = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float* x = f[g][w];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= mul;
          sum[g] += x[e];
        }
        // code order in a word: values (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16
        qf[nt][g][w][0] = pack_f16(x[0], x[4]);
        qf[nt][g][w][1] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
        qf[nt][g][w][2] = pack_f16(x[2], x[6]);
        qf[nt][g][w][3] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
      }
      sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 2);
      sum[g] *= 0x1p-7f;
    }
    // K index 2c, 2c + 1 of the offsets' instruction: the groups' first parts
    // in turn, then their second ones
    {
      float first[G], second[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        first[g] = __half2float(__float2half_rn(sum[g]));
        second[g] = sum[g] - first[g];
      }
      if constexpr (G == 1) qz[nt] = c == 0 ? pack_f16(first[0], second[0]) : 0u;
      if constexpr (G == 2)
        qz[nt] = c == 0 ? pack_f16(first[0], first[1]) : c == 1 ? pack_f16(second[0], second[1]) : 0u;
      if constexpr (G == 4)
        qz[nt] = c == 0   ? pack_f16(first[0], first[1])
                 : c == 1 ? pack_f16(first[2], first[3])
                 : c == 2 ? pack_f16(second[0], second[1])
                          : pack_f16(second[2], second[3]);
    }
    const int pos = sp.pos0 + i;
    const int top_pos = live ? (p.causal ? min(sp.len, pos + 1) : sp.len) : 1 << 30;
    const int low_pos = live && p.window > 0 ? max(0, pos - p.window + 1) : 0;
    // the results have rows 2c and 2c + 1 in a lane
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int from = (2 * c + e) * 4;
      fs[nt][e] = __shfl_sync(0xFFFFFFFFu, back, from);
      hi[nt][e] = __shfl_sync(0xFFFFFFFFu, top_pos, from);
      lo[nt][e] = __shfl_sync(0xFFFFFFFFu, low_pos, from);
    }
    hi_all = min(hi_all, (int)__reduce_min_sync(0xFFFFFFFFu, top_pos));
    lo_all = max(lo_all, (int)__reduce_max_sync(0xFFFFFFFFu, low_pos));
  }

  // where this lane's pieces lie in 16 positions: K's words 2c and 2c + 1 of
  // position r, V's word r of position 2c, K's params of position r and V's of
  // position 2c.  The others' places differ by whole rows (S::place repeats
  // every four).
  uint32_t k_at[G], v_at[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    k_at[g] = S::place(r, 2 * g + (c >> 1)) + (uint32_t)(c & 1) * 8u;
    v_at[g] = S::kCodes + S::place(c, 2 * g + (r >> 2)) + (uint32_t)(r & 3) * 4u;
  }
  const uint32_t kp_at = 2 * S::kCodes + (uint32_t)(r * G * 4);
  const uint32_t vp_at = 2 * S::kCodes + S::kParam + (uint32_t)(2 * c * G * 4);

  // nb: what is added to a score for p's exponent, kWeightBits - m
  float o[NT][G][4][4] = {}, zo[NT][4] = {}, m[NT][2], nb[NT][2] = {}, l[NT][2] = {};
  uint32_t power[G];  // what V's scales are taken times, by an fp16's bits: (s + 15) 2^10 is 2^s
#pragma unroll
  for (int g = 0; g < G; ++g) power[g] = kFirstPower;
  const uint32_t own_at = 2 * S::kCodes + S::kParam + (uint32_t)((lane >> 4) * S::kHalf + (lane & 15) * G * 4);
  uint32_t poison = 0;  // bit (nt * 2 + e) * G + g: that row's group is NaN
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY;

  // One stage: 32 positions from j0.  WHOLE: every row sees all of them.
  auto stage = [&](auto whole_type, uint32_t at0, int j0, uint32_t gone) {
    constexpr bool WHOLE = decltype(whole_type)::value;
    uint32_t own_a[G];  // V's scales of one position a lane
    lds_words<G>(at0 + own_at, own_a);
    // scores u[..]: positions r and r + 8 of each half, rows 2c and 2c + 1
    float u[2][NT][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t at = at0 + (uint32_t)half * S::kHalf;
      float acc[NT][G][4];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // words 2c and 2c + 1 of the group, of positions r and r + 8
        const uint2 wa = lds_v2u(at + k_at[g]);
        const uint2 wb = lds_v2u(at + k_at[g] + 8 * S::kRow);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t x = w ? wa.y : wa.x, y = w ? wb.y : wb.x;
          const uint32_t x2 = x >> 8, y2 = y >> 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (w == 0)
              mma16816_new(acc[nt][g], x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u,
                           y & 0x00F000F0u, qf[nt][g][w][0], qf[nt][g][w][1]);
            else
              mma16816(acc[nt][g], x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u,
                       y & 0x00F000F0u, qf[nt][g][w][0], qf[nt][g][w][1]);
            mma16816(acc[nt][g], x2 & 0x000F000Fu, y2 & 0x000F000Fu, x2 & 0x00F000F0u,
                     y2 & 0x00F000F0u, qf[nt][g][w][2], qf[nt][g][w][3]);
          }
        }
      }
      // (a, z) of the groups, of positions r and r + 8
      uint32_t az[2][G];
#pragma unroll
      for (int e = 0; e < 2; ++e) lds_words<G>(at + kp_at + (uint32_t)(8 * e * G * 4), az[e]);
      // the offsets, two groups a lane
      uint32_t z2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (G == 1) z2[e] = prmt(az[e][0], az[e][0], 0x3232);
        if constexpr (G == 2) z2[e] = prmt(az[e][0], az[e][1], 0x7632);
        if constexpr (G == 4)
          z2[e] = (c & 1) ? prmt(az[e][2], az[e][3], 0x7632) : prmt(az[e][0], az[e][1], 0x7632);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float t[4];
        mma16816_new(t, z2[0], z2[1], 0u, 0u, qz[nt], 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = t[e] * 0x1p-17f;
#pragma unroll
          for (int g = 0; g < G; ++g) x = fmaf(half_low(az[e >> 1][g]), acc[nt][g][e], x);
          u[half][nt][e] = x;
        }
      }
    }

    uint32_t seen = 0xFFFFFFFFu;  // bit half * 4 NT + nt * 4 + e
    if (!WHOLE) {
      seen = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + half * 16 + r + (e >> 1) * 8;
            const bool ok = j < min(hi[nt][e & 1], end) && j >= lo[nt][e & 1] && !((gone >> half) & 1u);
            if (ok) seen |= 1u << (half * 4 * NT + nt * 4 + e);
            else u[half][nt][e] = -INFINITY;
          }
    }

    // the powers in use for V's scales
    const bool own_seen = WHOLE || (j0 + lane >= sp.seen && j0 + lane < end && !((gone >> (lane >> 4)) & 1u));
    uint32_t most = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      own_a[g] &= 0x7FFFu;
      if (!own_seen || own_a[g] >= 0x7C00u) own_a[g] = 0;
      most = max(most, own_a[g] + power[g]);
    }
    const bool over = most > 31u << 10;  // a 2^s > 2

    // the maximum in use (a factor fs >= 0 makes u the score)
    float top[NT][2];
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[nt][e] = fmaxf(fmaxf(u[0][nt][e], u[0][nt][e + 2]), fmaxf(u[1][nt][e], u[1][nt][e + 2]));
        moved |= top[nt][e] * fs[nt][e] > m[nt][e] + kLazyBits;
      }
    if (__any_sync(0xFFFFFFFFu, moved || over)) {
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[nt][e];
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 16));
            const float now = fmaxf(m[nt][e], t * fs[nt][e]);
            const float fix = now == -INFINITY ? 1.f : ex2(m[nt][e] - now);
            m[nt][e] = now;
            nb[nt][e] = now == -INFINITY ? 0.f : kWeightBits - now;
            l[nt][e] *= fix;
            zo[nt][e] *= fix;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                o[nt][g][j][e] *= fix;
                o[nt][g][j][e + 2] *= fix;
              }
          }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t a = __reduce_max_sync(0xFFFFFFFFu, own_a[g]);
        if (a + power[g] <= 31u << 10) continue;
        // a 2^s from 1/2 on (below 4 for a scale beyond 2^15, which has no smaller power)
        const uint32_t now = max(1u << 10, (29u << 10) - min(a & 0x7C00u, 28u << 10));
        const float fix = power_of_two((int)(now >> 10) - (int)(power[g] >> 10));
        power[g] = now;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][g][j][e] *= fix;
      }
    }

    // weights, and the second product
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t at = at0 + (uint32_t)half * S::kHalf;
      const uint32_t pa = at + 2 * S::kCodes + S::kParam;
      uint32_t b0[NT], b1[NT];  // p of positions 2c, 2c + 1, and 2c + 8, 2c + 9, of row r
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = ex2(fmaf(u[half][nt][e], fs[nt][e & 1], nb[nt][e & 1]));
        l[nt][0] += w[0] + w[2];
        l[nt][1] += w[1] + w[3];
        b0[nt] = transpose8x8(pack_f16(w[0], w[1]));
        b1[nt] = transpose8x8(pack_f16(w[2], w[3]));
      }
      // (a, z) of positions 2c, 2c + 1, 2c + 8, 2c + 9
      uint32_t az[4][G];
#pragma unroll
      for (int k = 0; k < 4; ++k) lds_words<G>(at + vp_at + (uint32_t)(((k & 1) + 8 * (k >> 1)) * G * 4), az[k]);
      if (!WHOLE) {
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = j0 + half * 16 + 2 * c + (k & 1) + 8 * (k >> 1);
          const bool in = j >= sp.seen && j < end && !((gone >> half) & 1u);  // by some row
#pragma unroll
          for (int g = 0; g < G; ++g) {
            odd |= odd_half2(az[k][g]);
            az[k][g] = in ? finite_half2(az[k][g]) : 0u;
          }
        }
        if (__any_sync(0xFFFFFFFFu, odd)) {
#pragma unroll
          for (int e8 = 0; e8 < 2; ++e8) {
            uint32_t own[G];
            lds_words<G>(pa + (uint32_t)((r + 8 * e8) * G * 4), own);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (odd_half2(own[g]) && ((seen >> (half * 4 * NT + nt * 4 + 2 * e8 + e)) & 1u))
                    poison |= 1u << ((nt * 2 + e) * G + g);
          }
        }
      }
      // row g < G of the offsets' instruction: the group's z
      uint32_t za = 0, zb = 0;
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (r == g) {
          za = prmt(az[0][g], az[1][g], 0x7632);
          zb = prmt(az[2][g], az[3][g], 0x7632);
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma16816(zo[nt], za, 0u, zb, 0u, b0[nt], b1[nt]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t by = power[g] | power[g] << 16;
        const uint32_t a01 = mul_half2(prmt(az[0][g], az[1][g], 0x5410), by),
                       a23 = mul_half2(prmt(az[2][g], az[3][g], 0x5410), by);
        // word r of the group, of positions 2c, 2c + 1, 2c + 8, 2c + 9
        const uint32_t va = at + v_at[g];
        const uint32_t v0 = lds_u32v(va), v1 = lds_u32v(va + 4 * S::kRow);
        const uint32_t v2 = lds_u32v(va + 8 * S::kRow), v3 = lds_u32v(va + 12 * S::kRow);
        uint32_t p0[NT], p1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          p0[nt] = mul_half2(b0[nt], a01);
          p1[nt] = mul_half2(b1[nt], a23);
        }
#pragma unroll
        for (int j = 0; j < 4; j += 2) {  // byte j: values 8r + 2j and 8r + 2j + 1
          const uint32_t x = prmt(v0, v1, j == 0 ? 0x5410 : 0x7632);  // bytes j, j + 1 of each
          const uint32_t y = prmt(v2, v3, j == 0 ? 0x5410 : 0x7632);
          const uint32_t x0 = x & 0x00FF00FFu, y0 = y & 0x00FF00FFu;
          const uint32_t x1 = prmt(x, 0u, 0x4341), y1 = prmt(y, 0u, 0x4341);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[nt][g][j], x & 0x000F000Fu, x0, y & 0x000F000Fu, y0, p0[nt], p1[nt]);
            mma16816(o[nt][g][j + 1], x1 & 0x000F000Fu, x1, y1 & 0x000F000Fu, y1, p0[nt], p1[nt]);
          }
        }
      }
    }
  };

  for (int s = 0, slot = 0; s < mine; ++s) {
    cp_async_wait<kFewStages - 2>();
    __syncwarp();
    fetch(s + kFewStages - 1);
    const uint32_t at0 = ring + (uint32_t)slot * S::kStage;
    const int j0 = begin + (s * kFewWarps + warp) * kFewTokens;
    const uint32_t gone = (bad >> (2 * slot)) & 3u;
    if (j0 >= lo_all && j0 + kFewTokens <= min(hi_all, end) && gone == 0)
      stage(std::true_type(), at0, j0, 0u);
    else
      stage(std::false_type(), at0, j0, gone);
    if (++slot == kFewStages) slot = 0;
  }
  launch_dependents();  // the joining kernel may be set up
  cp_async_wait<0>();
  __syncthreads();  // the rings are free: they take the warps' results

  // ---- join the warps: [warp][row][D] and (max, sum) behind them
  constexpr int kRows = 8 * NT;
  float* so = reinterpret_cast<float*>(smem);
  float* sm = so + kFewWarps * kRows * D;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int step = 4; step < 32; step *= 2) {
        l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], step);
        poison |= __shfl_xor_sync(0xFFFFFFFFu, poison, step);
      }
      float z[G];  // the offsets' sum of group g lies with the lanes of r = g
#pragma unroll
      for (int g = 0; g < G; ++g) {
        z[g] = __shfl_sync(0xFFFFFFFFu, zo[nt][e], g * 4 + c);
        if ((poison >> ((nt * 2 + e) * G + g)) & 1u) z[g] = __uint_as_float(0x7FC00000u);
      }
      const int row = warp * kRows + nt * 8 + 2 * c + e;
      if (r == 0) {
        sm[2 * row] = m[nt][e];
        sm[2 * row + 1] = l[nt][e];
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float back = power_of_two(39 - (int)(power[g] >> 10));  // 2^(24 - s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float2*>(so + row * D + g * kKvGroup + 8 * r + 2 * j) =
              make_float2(fmaf(o[nt][g][j][e], back, z[g]),
                          fmaf(o[nt][g][j][e + 2] - o[nt][g][j][e], back * 0.0625f, z[g]));
      }
    }
  __syncthreads();
  for (int id = threadIdx.x; id < row_n * (D / 4); id += kFewWarps * 32) {
    const int row = id / (D / 4), d = id % (D / 4) * 4;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, sm[2 * (w * kRows + row)]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      const float mw = sm[2 * (w * kRows + row)];
      const float lw = sm[2 * (w * kRows + row) + 1];
      if (mw == -INFINITY && lw == 0.f) continue;  // this warp saw nothing of the row
      const float f = ex2(mw - top);
      sum = fmaf(lw, f, sum);
      const float4 y = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + d);
      x.x = fmaf(y.x, f, x.x);
      x.y = fmaf(y.y, f, x.y);
      x.z = fmaf(y.z, f, x.z);
      x.w = fmaf(y.w, f, x.w);
    }
    const int i = p.group.quotient(row0 + row), h = (kvh - i) * p.group.d + row0 + row;
    const int64_t t = sp.first_row + i;
    if (sp.parts > 1) {
      const int64_t at = ((int64_t)part * p.T + t) * p.q_heads + h;
      *reinterpret_cast<float4*>(p.part + at * D + d) = x;
      if (d == 0) {
        float* ml = p.part + (int64_t)p.splits * p.T * p.q_heads * D + at * 2;
        ml[0] = top;
        ml[1] = sum;
      }
      continue;
    }
    const bool none = top == -INFINITY && sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const T y[4] = {from_float<T>(x.x * inv), from_float<T>(x.y * inv), from_float<T>(x.z * inv),
                    from_float<T>(x.w * inv)};
    *reinterpret_cast<uint2*>(p.out + t * p.ld_o + (int64_t)h * p.hd_o + d) =
        *reinterpret_cast<const uint2*>(y);
    if (p.lse && d == 0)
      p.lse[t * p.q_heads + h] =
          none ? -INFINITY : (top + log2f(sum) - kWeightBits) * 0.69314718055994531f;
  }
}

// Joins the parts of the rows that were split, in the same order whenever it
// runs: a CTA a row and head.  Every part's (max, sum) at once first, which
// give its weight; then D / 4 threads a part, 512 / D parts at a time, whose
// loads wait for nothing.  Two rounds of loads from L2 bound it: some 2.5 us for
// a row's 32 heads and 30 to 80 parts, of which the setting up goes on while the
// parts are still computed.
constexpr int kMostParts = 512;

template <typename T, int D>
__global__ void __launch_bounds__(128) kv4_join_kernel(const AttentionParams p) {
  constexpr int kLanes = D / 4, kSets = 128 / kLanes;
  __shared__ float weight[kMostParts];
  __shared__ float4 so[kSets][kLanes];
  __shared__ float red[2][4];
  const int64_t id = blockIdx.x;
  const int t = (int)((uint32_t)id / (uint32_t)p.q_heads), h = (int)((uint32_t)id % (uint32_t)p.q_heads);
  const int tid = threadIdx.x, set = tid / kLanes, lane = tid % kLanes;
  // Row offsets and lengths are read ahead of the wait: the kernel whose parts are
  // joined writes neither, and lets this one start only behind its own wait, when
  // whatever wrote them has ended.
  const int b = sequence_of(p.at, t);
  Span sp = {};
  if (b >= 0)
    sp = span_of(p, b, p.by_rows.quotient((t - rows_of(p.at, b).x) * p.group.d + h - p.group.quotient(h) * p.group.d));
  grid_dependency_wait();  // every CTA: this kernel must not end before the one that it joins
  launch_dependents();
  if (b < 0 || sp.parts <= 1 || t - sp.first_row >= sp.rows) return;
  const int64_t step = (int64_t)p.T * p.q_heads;
  const float* ml = p.part + (int64_t)p.splits * step * D + id * 2;
  const float* src = p.part + id * D + lane * 4;
  // the first parts' values are asked for before the weights are known
  constexpr int kAhead = 4;
  float4 y[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (set + k * kSets < sp.parts) y[k] = *reinterpret_cast<const float4*>(src + (set + k * kSets) * step * D);
  float2 own[kMostParts / 128];
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMostParts / 128; ++k) {
    own[k] = make_float2(-INFINITY, 0.f);
    if (tid + 128 * k < sp.parts) own[k] = *reinterpret_cast<const float2*>(ml + (tid + 128 * k) * step * 2);
    top = fmaxf(top, own[k].x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((tid & 31) == 0) red[0][tid >> 5] = top;
  __syncthreads();
  top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kMostParts / 128; ++k) {
    const bool nothing = own[k].x == -INFINITY && own[k].y == 0.f;
    const float w = nothing ? 0.f : ex2(own[k].x - top);
    if (tid + 128 * k < sp.parts) weight[tid + 128 * k] = w;
    if (!nothing) sum = fmaf(own[k].y, w, sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((tid & 31) == 0) red[1][tid >> 5] = sum;
  __syncthreads();
  sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& v, int i) {
    const float w = weight[i];
    x.x = fmaf(v.x, w, x.x);
    x.y = fmaf(v.y, w, x.y);
    x.z = fmaf(v.z, w, x.z);
    x.w = fmaf(v.w, w, x.w);
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (set + k * kSets < sp.parts) add(y[k], set + k * kSets);
#pragma unroll 8
  for (int i = set + kAhead * kSets; i < sp.parts; i += kSets)
    add(*reinterpret_cast<const float4*>(src + i * step * D), i);
  so[set][lane] = x;
  __syncthreads();
  if (set != 0) return;
#pragma unroll
  for (int i = 1; i < kSets; ++i) {
    x.x += so[i][lane].x;
    x.y += so[i][lane].y;
    x.z += so[i][lane].z;
    x.w += so[i][lane].w;
  }
  const bool none = top == -INFINITY && sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  const T out[4] = {from_float<T>(x.x * inv), from_float<T>(x.y * inv), from_float<T>(x.z * inv),
                    from_float<T>(x.w * inv)};
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.ld_o + (int64_t)h * p.hd_o + lane * 4) =
      *reinterpret_cast<const uint2*>(out);
  if (p.lse && tid == 0)
    p.lse[id] = none ? -INFINITY : (top + log2f(sum) - kWeightBits) * 0.69314718055994531f;
}

}  // namespace
}  // namespace bcq

#include "bcq_kv4_many.cuh"

namespace bcq {
namespace {

// -------------------------------------------------------------------- host

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is16(int dtype) { return dtype == BCQ_F16 || dtype == BCQ_BF16; }

bool cache_sizes_ok(const bcq_kv4* c) {
  return c->pages >= 1 && c->heads >= 1 && c->page_size >= 16 && c->page_size % 16 == 0;
}

// Positions of a sequence; twice as many are still counted in an int.
constexpr int kMostPositions = 1 << 30;

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

bcq_status check_cache(const bcq_kv4* c, int T, const int32_t* table, int table_width,
                       const int32_t* kv_len, const int32_t* cu, int B) {
  if (!c || !c->k || !c->k_param || !c->v || !c->v_param || !table || !kv_len)
    return BCQ_ERR_NULL;
  if (!cache_sizes_ok(c) || T < 0 || B < 1 || table_width < 1 ||
      (int64_t)table_width * c->page_size > kMostPositions || (!cu && T != B) ||
      (double)c->pages * c->heads * c->page_size >= 4294967294.0 /* vectors are numbered in 32 bits */)
    return BCQ_ERR_SHAPE;
  if (!head_dim_ok(c->head_dim)) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->k_param, 16) || !aligned(c->v, 16) ||
      !aligned(c->v_param, 16) || !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(cu, 4))
    return BCQ_ERR_ALIGN;
  return BCQ_OK;
}

// Rows [T][heads][D] of a 16-bit type, strided.
bcq_status check_rows(const void* x, int64_t ld, int64_t hd, int dtype) {
  if (!x) return BCQ_ERR_NULL;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  if (ld < 0 || hd < 0) return BCQ_ERR_SHAPE;
  return !aligned(x, 16) || ld % 8 || hd % 8 ? BCQ_ERR_ALIGN : BCQ_OK;
}

Divisor divisor(int d) {
  int s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {d, s == 0 ? 0u : (uint32_t)((((uint64_t)1 << (31 + s)) + (uint64_t)d - 1) / (uint64_t)d), s - 1};
}

Places places_of(const bcq_kv4* c, const int32_t* table, int table_width, const int32_t* kv_len,
                 const int32_t* cu, int B) {
  return {table,    kv_len,       cu,       table_width,
          B,        c->pages,     c->page_size, c->heads,
          table_width * c->page_size, divisor(c->page_size)};
}

// How the rows of a call, in or out, are shared out: one row a block up to T =
// `one`, else four, whose places are found and whose loads are in flight together;
// from `side_by_side` rows on several fours in a block, where a row has no more
// than `words` words (and a block so that it holds them).
//
// In (us, one | four rows a block): up to 592 rows all blocks of one row fit the
// SMs at once, and a row waits for fewer loads (512 rows of 1, 8 heads of 128 and
// 32 of 64: 3.2 | 3.8, 3.7 | 4.3, 5.2 | 6.1; 640 of the first two 4.5 | 4.1, 5.0 | 4.6,
// 768 of the third 6.7 | 6.7).  Rows of four turns of the block's loop or more go on
// to twice as many (32 heads of 128: 768 rows 10.2 | 10.9, 1024 11.2 | 11.1, 2048
// 19.8 | 16.3; of 256: 1024 rows 18.7 | 19.1, 2048 37.6 | 30.8).
// Out: 384 rows of 8 heads of 128, 32 of 64 and 32 of 128 2.9 | 2.8, 3.4 | 3.4, 4.4 |
// 4.6, 512 rows 3.1 | 2.8, 3.6 | 3.4, 5.0 | 4.6.
// Side by side (us, four rows | sets of four), in: 2048 rows of 2 heads of 64 or
// 128 4.1 | 5.8, 4.4 | 4.8, 4096 rows 7.0 | 5.9, 6.9 | 5.6, of 8 heads of 64 7.6 | 6.5.
// Out: 8192 rows of 2 heads of 64 or 128 5.1 | 4.8, 5.4 | 6.0, 12288 rows 6.9 | 5.5, 7.5 |
// 6.3, of 8 heads of 64 8.9 | 9.4, 65536 rows 42.2 | 43.9.
struct RowsRule {
  int one, side_by_side, words;
};
RowsRule rows_in_rule(int words) { return {words >= 4 * kRowThreads ? 1184 : 592, 4096, kRowThreads / 2}; }
RowsRule rows_out_rule() { return {444, 10240, kRowThreads / 4}; }

// f(D, rows a block, whether side by side, blocks), the first three as compile-time
// numbers; words: of a row's K and V.
template <typename F>
void by_shape(int D, int words, int T, const RowsRule& rule, const F& f) {
  auto rows = [&](auto d) {
    if (T <= rule.one) f(d, std::integral_constant<int, 1>(), std::false_type(), T);
    else if (words > rule.words || T < rule.side_by_side) f(d, std::integral_constant<int, 4>(), std::false_type(), (T + 3) / 4);
    else f(d, std::integral_constant<int, 4>(), std::true_type(), (T + 4 * row_sets(words) - 1) / (4 * row_sets(words)));
  };
  if (D == 64) rows(std::integral_constant<int, 64>());
  else if (D == 128) rows(std::integral_constant<int, 128>());
  else rows(std::integral_constant<int, 256>());
}

// How a call's rows and positions are shared out: the kernel (nt: row groups of
// eight a CTA of the few-row kernel; 0 the many-row kernel, -1 the same where all
// rows see few positions), rows of a CTA, and parts of the positions.
struct AttentionPlan {
  int nt, rows, row_blocks, splits, chunk;
};

// How many parts the positions are cut into, by a model of the time (us, which is
// returned) on the 148 SMs of a B200, on which its numbers were fitted (a constant:
// the workspace's size must not depend on the device that is current when it is
// asked for).  `each` CTAs fit an SM; a CTA takes `start`, and `per` a position
// (beside each - 1 others); splitting at all takes `join`, and some a part.  While
// all CTAs run at once the fullest SM decides, and fewer than `each` on it run
// faster, though not in proportion; beyond that CTAs start as others end: the
// whole work's share and `tail` of a CTA.  Of max_kv `there` is thought to be
// there on average, and half a part more.
struct PartsModel {
  int each;
  float there, per, start, join, join_part, tail;
};
constexpr int kSms = 148;
float plan_parts(AttentionPlan* f, int64_t units, int max_kv, const PartsModel& m) {
  static const float kPace[5] = {0, 0.49f, 0.63f, 0.8f, 1.0f};
  const float room = (float)kSms * (float)m.each, mean = m.there * (float)max_kv;
  float best = 0;
  const uint32_t kv = (uint32_t)max_kv;
  uint32_t chunk = ((kv + kMostParts - 1) / kMostParts + 127) & ~127u;
  for (bool more = true; more; chunk += std::max(128u, (chunk / 8) & ~127u)) {
    const uint32_t parts = (kv + chunk - 1) / chunk;
    const float length = (float)std::min(chunk, kv) * m.per, all = (float)parts;
    const float ctas = (float)units * std::min(all, m.there * all + 0.5f);
    float cost;
    if (ctas <= room) {
      const int fullest = ((int)ctas + kSms - 1) / kSms;
      cost = length * kPace[std::min(4, fullest * 4 / m.each)] + m.start;
    } else {
      cost = std::max(length * kPace[m.each == 1 ? 4 : 1] + m.start,
                      ((float)units * mean * m.per + ctas * m.start) / room + m.tail * (length + m.start));
    }
    cost += parts > 1 ? m.join + m.join_part * all : 0.f;
    if (best == 0 || cost < best) {
      best = cost;
      f->splits = (int)parts;
      f->chunk = (int)std::min(chunk, (uint32_t)kMostPositions);
    }
    more = parts > 1 && length * kPace[1] < best;  // longer ones cost more
  }
  return best;
}

// The few-row kernel passes over the positions once for every 16 rows (8 where
// there are no more, or D = 256: 13.0 us in one pass for 16 rows and 8 x 2000
// positions, 15.0 in two), four CTAs an SM (two where rows or values are many),
// with exact products of queries and codes; the many-row kernel once for every
// 256 (128 where D = 256), with keys rounded to fp16, or, in the blocks of rows that
// see few positions, in two parts, which takes 1.05 to 1.15 times as long (1.2 to 1.35
// where D = 256 leaves room for one set of them).  Calls that the second kernel is not thought to
// save a seventh stay with the first.
//
// The models' numbers are fitted to 68 calls of the first (1 to 256 sequences,
// 300 to 262144 positions, heads of 64 to 256) and 60 of the second, each over 10
// to 20 parts: 2 and 1 % on average above the best part of each call, 3 % above
// the better kernel's.  Measured (us, few | many): 64 rows over 4000 positions,
// 8 heads of 128, 14.3 | 14.4, over 8 x 2000 21.8 | 25.1, 32 x 1000 41.0 | 42.0; 128
// rows 19.9 | 17.3, 27.8 | 29.8, 70.6 | 43.5; 512 rows 46.7 | 32.5, 97.1 | 58.3, 231 |
// 97.
AttentionPlan plan_attention(const bcq_kv4* c, int q_heads, int B, int max_q, int max_kv, int window) {
  const int D = c->head_dim, group = q_heads / c->heads;
  const int64_t rows = (int64_t)max_q * group;
  auto plan = [&](int nt, int block_rows, AttentionPlan* f) {
    f->nt = nt;
    f->rows = block_rows;
    f->row_blocks = (int)std::min<int64_t>((rows + block_rows - 1) / block_rows, INT32_MAX);
    const int64_t units = (int64_t)f->row_blocks * c->heads * B;
    // what a block of rows sees at most
    const int seen = window == 0 ? max_kv
                                 : (int)std::min<int64_t>(max_kv, (int64_t)window + block_rows / group + 32);
    const bool ragged = B > 1 && seen == max_kv;
    if (nt > 0) {
      const float per = D == 64 ? 0.0072f : D == 128 ? 0.0125f : 0.0143f;
      return plan_parts(f, units, seen, {nt == 1 && D <= 128 ? 4 : 2, ragged ? 0.75f : 1.f, per, 2.75f, 2.f, 0.037f, 0.126f}) + 1.f;
    }
    const bool two = D != 256 && rows > 128;  // tiles
    const float per = (D == 64 ? (two ? 0.0209f : 0.0114f) : D == 128 ? (two ? 0.0254f : 0.0144f) : 0.023f) *
                      (nt == 0 ? 1.f : D == 256 ? 1.3f : 1.1f);
    const float out = 1e-6f * (float)B * (float)rows * (float)c->heads * (float)D;  // written and read for each part
    return plan_parts(f, units, seen, {1, ragged ? 0.6f : 1.f, per, 6.f, 5.3f, 1.87f * out, 0.66f});
  };
  const int nt = rows <= 8 || D == 256 ? 1 : 2;
  AttentionPlan few, many;
  const float few_time = plan(nt, 8 * nt, &few);
  if (rows <= 16) return few;
  const bool few_seen = max_kv < kFewSeen || (window != 0 && window < kFewSeen);
  return plan(few_seen ? -1 : 0, D == 256 ? 128 : 256, &many) < 0.85f * few_time ? many : few;
}

template <typename T, int D, int NT>
cudaError_t launch_few_t(const AttentionParams& p, cudaStream_t st) {
  constexpr int smem = (int)(kFewWarps * FewShape<D>::kRing);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kv4_few_kernel<T, D, NT>, smem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)p.row_blocks * p.at.heads * p.at.B), (unsigned)p.splits);
  return launch_early(kv4_few_kernel<T, D, NT>, grid, kFewWarps * 32, smem, st, p);
}

template <typename T, int D, bool IMPATIENT = false>
cudaError_t launch_many_t(const AttentionParams& p, cudaStream_t st) {
  using S = ManyShape<D>;
  if constexpr (std::is_same_v<T, __half> && D == 128 && !IMPATIENT)
    if (impatient()) return launch_many_t<T, D, true>(p, st);
  const auto kernel = kv4_many_kernel<T, D, IMPATIENT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kernel, S::kSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((int64_t)p.row_blocks * p.at.heads * p.at.B), (unsigned)p.splits);
  return launch_early(kernel, grid, S::kThreads, S::kSmem, st, p);
}

template <typename T, int D>
cudaError_t launch_join_t(const AttentionParams& p, cudaStream_t st) {
  return launch_early(kv4_join_kernel<T, D>, dim3((unsigned)((int64_t)p.T * p.q_heads)), 128, 0, st, p);
}

template <typename T, int D>
cudaError_t launch_attention_t(const AttentionParams& p, int nt, cudaStream_t st) {
  cudaError_t e;
  if (nt <= 0) e = launch_many_t<T, D>(p, st);
  else if constexpr (D == 256) e = launch_few_t<T, D, 1>(p, st);
  else e = nt == 1 ? launch_few_t<T, D, 1>(p, st) : launch_few_t<T, D, 2>(p, st);
  return e == cudaSuccess && p.splits > 1 ? launch_join_t<T, D>(p, st) : e;
}

template <typename T>
cudaError_t launch_attention(const AttentionParams& p, int D, int nt, cudaStream_t st) {
  if (D == 256) return launch_attention_t<T, 256>(p, nt, st);
  return D == 128 ? launch_attention_t<T, 128>(p, nt, st) : launch_attention_t<T, 64>(p, nt, st);
}

}  // namespace

cudaError_t read_and_clear_kv4_error(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_kv4_error, sizeof(int));
  if (e == cudaSuccess && *code != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_error, &zero, sizeof(int));
  }
  return e;
}

}  // namespace bcq

using namespace bcq;

extern "C" {

bcq_status bcq_kv4_append(const bcq_kv4* cache, const void* k, int64_t ld_k, int64_t hd_k,
                          const void* v, int64_t ld_v, int64_t hd_v, int dtype, int T,
                          const int32_t* table, int table_width, const int32_t* kv_len,
                          const int32_t* cu, int B, void* stream) {
  bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK || T == 0) return s;
  if ((s = check_rows(k, ld_k, hd_k, dtype)) != BCQ_OK) return s;
  if ((s = check_rows(v, ld_v, hd_v, dtype)) != BCQ_OK) return s;
  const AppendParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                          {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v)},
                          {ld_k, ld_v},
                          {hd_k, hd_v},
                          {cache->k, cache->v},
                          {reinterpret_cast<__half2*>(cache->k_param),
                           reinterpret_cast<__half2*>(cache->v_param)},
                          T};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  const int words = 2 * cache->heads * (cache->head_dim / 8);
  by_shape(cache->head_dim, words, T, rows_in_rule(words), [&](auto d, auto rows, auto shared, int count) {
    constexpr int D = decltype(d)::value, kRows = decltype(rows)::value;
    constexpr bool kShared = decltype(shared)::value;
    const unsigned blocks = (unsigned)count;
    if (dtype == BCQ_F16) e = launch_early(kv4_append_kernel<__half, D, kRows, kShared>, blocks, kRowThreads, 0, st, p);
    else e = launch_early(kv4_append_kernel<__nv_bfloat16, D, kRows, kShared>, blocks, kRowThreads, 0, st, p);
  });
  return e == cudaSuccess ? BCQ_OK : BCQ_ERR_CUDA;
}

bcq_status bcq_kv4_read(const bcq_kv4* cache, void* k, void* v, int dtype, int T,
                        const int32_t* table, int table_width, const int32_t* kv_len,
                        const int32_t* cu, int B, void* stream) {
  const bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK || T == 0) return s;
  if (!k || !v) return BCQ_ERR_NULL;
  if (!is16(dtype) && dtype != BCQ_F32) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16)) return BCQ_ERR_ALIGN;
  const ReadParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                        {cache->k, cache->v},
                        {reinterpret_cast<const __half2*>(cache->k_param),
                         reinterpret_cast<const __half2*>(cache->v_param)},
                        {k, v},
                        T};
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  const int words = 2 * cache->heads * (cache->head_dim / 8);
  by_shape(cache->head_dim, words, T, rows_out_rule(), [&](auto d, auto rows, auto shared, int count) {
    constexpr int D = decltype(d)::value, kRows = decltype(rows)::value;
    constexpr bool kShared = decltype(shared)::value;
    const unsigned blocks = (unsigned)count;
    if (dtype == BCQ_F16) e = launch_early(kv4_read_kernel<__half, D, kRows, kShared>, blocks, kRowThreads, 0, st, p);
    else if (dtype == BCQ_BF16) e = launch_early(kv4_read_kernel<__nv_bfloat16, D, kRows, kShared>, blocks, kRowThreads, 0, st, p);
    else e = launch_early(kv4_read_kernel<float, D, kRows, kShared>, blocks, kRowThreads, 0, st, p);
  });
  return e == cudaSuccess ? BCQ_OK : BCQ_ERR_CUDA;
}

size_t bcq_kv4_attention_workspace_bytes(const bcq_kv4* cache, int T, int q_heads, int B,
                                         int max_q, int max_kv, int window) {
  if (!cache || !cache_sizes_ok(cache) || !head_dim_ok(cache->head_dim) || T < 0 || B < 1 ||
      max_q < 1 || max_kv < 1 || window < 0 || q_heads < 1 || q_heads % cache->heads)
    return 0;
  const AttentionPlan f = plan_attention(cache, q_heads, B, max_q, max_kv, window);
  if (f.splits == 1) return 0;
  return (size_t)f.splits * (size_t)T * (size_t)q_heads * (size_t)(cache->head_dim + 2) * 4;
}

bcq_status bcq_kv4_attention(const bcq_kv4* cache, const void* q, int64_t ld_q, int64_t hd_q,
                             int dtype, int T, int q_heads, const int32_t* table,
                             int table_width, const int32_t* kv_len, const int32_t* cu, int B,
                             int max_q, int max_kv, int causal, int window, float scale,
                             void* out, int64_t ld_o, int64_t hd_o, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || q_heads / cache->heads > 128 || max_q < 1 ||
      max_kv < 1 || window < 0 || !std::isfinite(scale))
    return BCQ_ERR_SHAPE;
  if (T == 0) return BCQ_OK;
  if ((s = check_rows(q, ld_q, hd_q, dtype)) != BCQ_OK) return s;
  if ((s = check_rows(out, ld_o, hd_o, dtype)) != BCQ_OK) return s;
  // rows of out that share memory would be written by several threads
  const int64_t D = cache->head_dim;
  if ((T > 1 && ld_o < D) || (q_heads > 1 && hd_o < D) ||
      (T > 1 && q_heads > 1 && ld_o < (q_heads - 1) * hd_o + D && hd_o < (T - 1) * ld_o + D))
    return BCQ_ERR_SHAPE;
  if (lse && !aligned(lse, 4)) return BCQ_ERR_ALIGN;
  const size_t need = bcq_kv4_attention_workspace_bytes(cache, T, q_heads, B, max_q, max_kv, window);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return BCQ_ERR_NULL;
    if (!aligned(workspace, 16)) return BCQ_ERR_ALIGN;
  }
  AttentionParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                       cache->k,
                       reinterpret_cast<const __half2*>(cache->k_param),
                       cache->v,
                       reinterpret_cast<const __half2*>(cache->v_param),
                       static_cast<const uint16_t*>(q),
                       static_cast<uint16_t*>(out),
                       lse,
                       ld_q,
                       hd_q,
                       ld_o,
                       hd_o,
                       T,
                       q_heads,
                       max_q,
                       causal,
                       std::min(window, kMostPositions),  // a wider one hides nothing either
                       scale};
  const AttentionPlan f = plan_attention(cache, q_heads, B, max_q, max_kv, window);
  p.group = divisor(q_heads / cache->heads);
  p.by_blocks = divisor(f.row_blocks);
  p.by_heads = divisor(cache->heads);
  p.by_rows = divisor(f.rows);
  p.rows = f.rows;
  p.row_blocks = f.row_blocks;
  p.splits = f.splits;
  p.chunk = f.chunk;
  p.part = static_cast<float*>(workspace);
  if ((int64_t)f.row_blocks * cache->heads * B > INT32_MAX || (int64_t)T * q_heads > INT32_MAX ||
      (int64_t)max_q * (q_heads / cache->heads) > INT32_MAX - 512)
    return BCQ_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == BCQ_F16 ? launch_attention<__half>(p, cache->head_dim, f.nt, st)
                                         : launch_attention<__nv_bfloat16>(p, cache->head_dim, f.nt, st);
  return e == cudaSuccess ? BCQ_OK : BCQ_ERR_CUDA;
}

}  // extern "C"

// tt_cache_kernels.hip -- keys and values of a paged cache: written, and
// attended to (declared in include/tt_step.h).
#include "tt_lanes.h"
#include "tt_step_kernels.h"

#include <algorithm>
#include <type_traits>

namespace tt {
namespace {

constexpr int64_t MAX_ITEMS = 0xFFFFFFFF;  // threads that a launch may have in a dimension of its grid

__host__ __device__ inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// N words at any address.
template <int N>
struct Words {
  typedef uint32_t type __attribute__((ext_vector_type(N), aligned(1)));
};
template <>
struct Words<1> {
  typedef uint32_t type __attribute__((aligned(1)));
};

// Division of numbers below 2^31 by one from 1 to 2^20: with s = ceil(log2 d) the factor is above 2^(31+s) / d by at
// most 1, which adds less than a / 2^31 of a d-th to a / d.
struct Division {
  uint32_t divisor, factor, shift;
};
Division division(int64_t d) {
  uint32_t s = 0;
  while (((int64_t)1 << s) < d) ++s;
  return {(uint32_t)d, (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)d + 1), 31 + s};
}
__device__ inline uint32_t quotient(uint32_t a, Division d) { return (uint32_t)(((uint64_t)a * d.factor) >> d.shift); }

// ------------------------------------------------------------------- writing

constexpr int WR_THREADS = 256;

template <class T>
struct Eight {
  typedef T type __attribute__((ext_vector_type(8), aligned(alignof(T))));
};

// A quotient by s, of which r is the rounded reciprocal, rounded as a division would: the product is put right by its remainder (Markstein's
// theorem), which holds while neither leaves the normal range.  Where r is not used it is 0.
__device__ inline float quotient(float x, float s, float r) {
  const float q = x * r, y = fmaf(fmaf(-q, s, x), r, q);
  return __builtin_isfpclass(q, 0x108) ? y : q;  // of normal numbers; zeros keep their sign, infinities and NaN what they are
}
// The reciprocal where quotients that are then taken into 2^-10 .. 448 may go by it.
__device__ inline float reciprocal_of(float s) {
  const float a = fabsf(s);
  return a > 0x1p-60f && a < 0x1p60f ? 1.0f / s : 0.0f;
}

// Eight elements, divided by their scale, in the cache's type.
template <class I, class O>
__device__ inline void put_eight(typename Eight<I>::type x, const float* scale, int64_t head, O* to) {
  if constexpr (std::is_same<O, uint8_t>::value) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = (float)x[k];
    if (scale) {
      const float s = scale[head], r = reciprocal_of(s);
      if (r != 0.0f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = quotient(f[k], s, r);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] /= s;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float y = __builtin_amdgcn_fmed3f(f[k], -448.0f, 448.0f);
      f[k] = f[k] != f[k] ? f[k] : y;  // NaN stays
    }
    typename Words<2>::type w;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int low = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
      w[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], low, true);
    }
    *reinterpret_cast<typename Words<2>::type*>(to) = w;
  } else {
    typename Eight<O>::type y;
    if (scale) {
      const float s = scale[head];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = (O)((float)x[k] / s);
    } else if constexpr (std::is_same<I, O>::value) {
      y = x;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = (O)x[k];
    }
    *reinterpret_cast<typename Eight<O>::type*>(to) = y;
  }
}

// Each thread moves eight keys and the eight values beside them, of `total` of the tokens from `first` on: both loads are on their way
// before the slot is known to be there.  Eight elements are 16 bytes of bfloat16, and of 8 bits what one lane can store at once.
// Bound by memory: 48,000 tokens of 8 heads of 128 elements, bfloat16 to e4m3, take 60 us for 292 MB (4.9 TB/s, what a
// large copy reaches; with divisions in place of the corrected products 69); 8 tokens 2.3 us, the launch and two dependent reads.
template <class I, class O>
__global__ __launch_bounds__(WR_THREADS) void k_write(tt_write_args a, Division by_token, Division by_head, Division by_block, int64_t first, uint32_t total) {
  const uint32_t at = blockIdx.x * WR_THREADS + threadIdx.x;
  if (at >= total) return;
  const uint32_t nth = quotient(at, by_token), rest = at - nth * by_token.divisor, head = quotient(rest, by_head), d = (rest - head * by_head.divisor) * 8;
  const int64_t token = first + nth, slot = a.slots[token];
  typedef typename Eight<I>::type In;
  const In k = *reinterpret_cast<const In*>(static_cast<const I*>(a.keys) + token * a.key_stride + head * a.key_head_stride + d);
  const In v = *reinterpret_cast<const In*>(static_cast<const I*>(a.values) + token * a.value_stride + head * a.value_head_stride + d);
  if (slot < 0) return;
  const tt_paged_cache& c = a.cache;
  const int64_t block = slot <= 0x7FFFFFFF ? quotient((uint32_t)slot, by_block) : slot / c.block_size;
  const int64_t place = slot - block * c.block_size;
  if (block >= c.blocks) return;
  put_eight<I, O>(k, c.key_scale, head,
                  static_cast<O*>(c.keys) + block * c.key_block_stride + place * c.key_place_stride + head * c.key_head_stride + d);
  put_eight<I, O>(v, c.value_scale, head,
                  static_cast<O*>(c.values) + block * c.value_block_stride + place * c.value_place_stride + head * c.value_head_stride + d);
}

// ----------------------------------------------------------------- attention
//
// Products go by 16x16x32 matrix instructions, whose lane l holds row (of the first operand) or column (of the second)
// l % 16 and of the 32 that are summed over those of group g = l / 16, eight of them; of the result it holds column l % 16
// and rows 4 g .. 4 g + 3.  What is summed over may come in any order that both operands share.
//
//   scores:  keys [16 tokens x 32 d] times queries [32 d x 16 heads]: lane (c, g) loads 16 bytes of token c's key, and gets
//            the scores of head c with tokens 4 g + r.
//   output:  values [16 d x 32 tokens] times weights [32 tokens x 16 heads], over the tokens that the lane's scores are
//            of, 4 g + r of two tiles of 16: the weights need no exchange.  Lane (c, g) loads the same d of its eight
//            tokens, D / 16 of them from c * D / 16 on, and product j takes every j-th: one byte permutation per pair.
//
// Keys and values so go from memory to registers without LDS, each read once.  With sixteen rows of a product for the heads that
// share a head of keys, most of which stand empty for few of them, the products are never what bounds it.
//
// Each wavefront has one tile's keys and values in registers and the next one's loads on their way while it computes.  Two or three wavefronts a
// SIMD then keep 30 KB and more of a CU in flight.  What it measured:
//   64 requests of up to 32,000 tokens, 64 heads on 8 of 128 elements, bfloat16   903 us for 5.13 GB: 5.7 TB/s, memory
//   33 requests of up to 8,000, 16 heads on 4 of 256                              128 us for 663 MB: 5.2 TB/s, memory
//   9 requests of up to 9,000, 28 heads on 4 of 128, float16                      27.5 us for 104 MB
//   one request of 4,000, 32 heads on 8 of 128                                    10.9 us for 16 MB, a tile or two a wavefront
//   2 requests of 400,001, 16 heads on one of 128, e4m3                           46.0 us for 205 MB: 4.4 TB/s; three wavefronts a SIMD (49-54 us)
//     and tiles of 64 tokens (52) were slower
//   301 queries of 40 rows, 12 heads of 64, a window of 1,024, capped, float16    40.2 us for 165 MB, in bundles
// What all of these but the first have beside their bytes at 5.6 TB/s is the same 8 to 11 us: the way to the first tile (lengths, sums over them, table, addresses,
// keys, each waiting for the one before) and the end.  Vector operations keep a SIMD busy for 12 to 14 percent of the first three's time, and
// matrix operations for 3 to 6; with e4m3, which is widened, 25 and 7.

constexpr int AT_THREADS = 256;
constexpr int AT_WAVES = AT_THREADS / WAVE;
constexpr int AT_TILE = 32;                  // tokens of a wavefront at a time
constexpr int AT_UNIT = AT_TILE * AT_WAVES;  // tokens of a workgroup at a time
constexpr int AT_HEADS = 16;                 // query heads of a workgroup
constexpr int AT_QUERIES = 512;              // most queries of a call whose tokens are dealt out

int padded(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// How a call is cut up.  An item is a query, or a bundle of queries of the same row.
struct AttendShape {
  int group, parts, rows;  // query heads of a head of keys; workgroups that they take; rows of a product that are in use
  int bundle;              // most queries of an item
  int64_t lanes;           // heads of keys times parts
  int workers;             // workgroups that the tokens of each lane are dealt out to; 0: one for each query
};

// Tokens are dealt out where a workgroup for each query would not fill the card a few times over: 256 CUs take three workgroups each
// of heads of up to 64 elements, two of 128, one of 256 (that is what their registers leave room for).  On 8 heads of keys of 128
// elements 64 requests of 2,000 to 32,000 tokens take 905 us dealt out and 1,121 by a workgroup each, which wait for the longest;
// 256 of 300 to 4,000 tokens 477 and 488; 500 of up to 2,000 482 and 470.
// Where there are more queries than the table has rows, some go by the same row, and those that a product has room for are attended to together.
// In a table with rows to spare the host cannot tell whether queries share one, and they go one by one.
AttendShape attend_shape(int64_t queries, int64_t heads, int64_t cache_heads, int64_t dim, int64_t table_rows, bool by_rows) {
  AttendShape s;
  s.group = (int)(heads / cache_heads);
  s.parts = (int)div_up(s.group, AT_HEADS);
  s.lanes = cache_heads * s.parts;
  const int groups = padded(dim) == 256 ? 256 : padded(dim) == 64 ? 768 : 512;
  const bool shared = by_rows && queries > table_rows && queries <= AT_QUERIES && s.group <= AT_HEADS / 2;
  const bool deal = shared || (queries <= AT_QUERIES && queries * s.lanes <= 2048);
  s.workers = deal ? (int)std::max((int64_t)1, groups / s.lanes) : 0;
  s.bundle = shared ? AT_HEADS / s.group : 1;
  s.rows = std::min(s.group, AT_HEADS) * s.bundle;
  return s;
}

// A workspace: two pieces of output for every worker of every lane, their maxima and sums, and for each item and lane its first piece and
// how many it has (one: it was put out at once); with bundles also the items, their first units, the queries in their order
// and each query's place among them.
struct Item {
  int32_t row, members, first;  // of the ordered queries
  uint32_t from, upto;
};
struct AttendSpace {
  float* piece;
  float* statistic;
  int2* pieces;
  int64_t* start;
  Item* item;
  int32_t* order;
  int32_t* place;  // item * AT_HEADS + which of its queries
  int64_t bytes;
};
AttendSpace attend_space(const AttendShape& s, int64_t queries, int64_t dim, void* at) {
  AttendSpace w{};
  if (!s.workers) return w;
  const bool joined = s.workers > 1;  // one worker puts everything out at once
  const int64_t pieces = joined ? 2 * s.workers * s.lanes * s.rows : 0, ends = joined ? queries * s.lanes : 0;
  w.piece = static_cast<float*>(at);
  w.statistic = w.piece + pieces * padded(dim);
  w.pieces = reinterpret_cast<int2*>(w.statistic + 2 * pieces);
  w.start = reinterpret_cast<int64_t*>(w.pieces + ends);
  w.bytes = pieces * (padded(dim) + 2) * 4 + ends * 8;
  if (s.bundle > 1) {
    w.item = reinterpret_cast<Item*>(w.start + AT_QUERIES + 1);
    w.order = reinterpret_cast<int32_t*>(w.item + AT_QUERIES);
    w.place = w.order + AT_QUERIES;
    w.bytes += (AT_QUERIES + 1) * 8 + AT_QUERIES * (int64_t)(sizeof(Item) + 8);
  }
  return w;
}

// Which tokens of which row a query sees.
struct Seen {
  int32_t row;
  uint32_t from, upto;
};
__device__ inline Seen seen(const tt_attend_args& a, int64_t i) {
  Seen s;
  const int64_t row = a.rows ? a.rows[i] : i, most = a.width * a.cache.block_size;
  int64_t n = min((int64_t)a.lengths[i], most);
  if (n < 0 || row < 0 || row >= a.table_rows || a.cache.blocks == 0) n = 0;
  s.row = n ? (int32_t)row : 0;
  s.upto = (uint32_t)n;
  s.from = a.window > 0 && n > a.window ? (uint32_t)(n - a.window) : 0;
  return s;
}

template <class T>
__device__ inline f32x4 product(u32x4 x, u32x4 y, f32x4 z) {
  if constexpr (std::is_same<T, _Float16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), z, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), z, 0, 0, 0);
}

// Two e4m3 (bytes 0 and 1, or 2 and 3) in 16 bits each, which hold them exactly.
template <class T, bool HIGH>
__device__ inline uint32_t widened(uint32_t w) {
  if constexpr (std::is_same<T, _Float16>::value)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HIGH));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

template <class T>
__device__ inline uint32_t two(float x, float y) {
  typedef T pair __attribute__((ext_vector_type(2)));
  const pair p = {(T)x, (T)y};
  return __builtin_bit_cast(uint32_t, p);
}
template <class T>
__device__ inline float one_of(uint32_t w, int k) {
  typedef T pair __attribute__((ext_vector_type(2)));
  return (float)__builtin_bit_cast(pair, w)[k];
}

// 1 for each element of a word that is infinite or NaN: those whose exponent is all ones carry into the bit above; of e4m3 all ones but the sign.
template <class T, bool EIGHT>
__device__ inline uint32_t not_finite(uint32_t w) {
  if constexpr (EIGHT) return ((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u;
  else return ((w & 0x7FFF7FFFu) + (std::is_same<T, _Float16>::value ? 0x04000400u : 0x00800080u)) >> 15 & 0x00010001u;
}

__device__ inline float over_groups(float x, bool sum) {
  const float y = __shfl_xor(x, 16), z = sum ? x + y : fmaxf(x, y), u = __shfl_xor(z, 32);
  return sum ? z + u : fmaxf(z, u);
}

__device__ inline float across_groups_max(float x) {
  const float y = fmaxf(x, __uint_as_float(across<16>(__float_as_uint(x))));
  return fmaxf(y, __uint_as_float(across<32>(__float_as_uint(y))));
}

constexpr uint32_t ALL = 0xFFFFFFFFu;

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.693147180559945309417f;

// 1 - 2 / (1 + e^2y), off by 2^-23 or so; below 1/4, where that would be many steps, the series up to y^9, whose next term is 2^-27 of it.
__device__ inline float tanh_of(float y) {
  const float p = y * y, near = y * fmaf(p, fmaf(p, fmaf(p, fmaf(p, 62.0f / 2835, -17.0f / 315), 2.0f / 15), -1.0f / 3), 1.0f);
  return fabsf(y) < 0.25f ? near : 1.0f - 2.0f / (1.0f + __builtin_amdgcn_exp2f(y * (2 * LOG2E)));
}

// One workgroup: a lane's heads, for some tokens of a query after the other.
template <class T, bool EIGHT, int D, bool WHOLE>
struct Attend {
  static constexpr int SIZE = EIGHT ? 1 : 2;
  static constexpr int STEPS = D / 32;             // products of a score
  static constexpr int PER = 16 / SIZE;            // elements of a load of keys
  static constexpr int LOADS = D / (4 * PER);      // of a token's key, by its four lanes
  static constexpr int MINE = D / 16;              // values of a token that a lane loads
  static constexpr int VWORDS = MINE * SIZE / 4;
  static constexpr bool HALF = std::is_same<T, _Float16>::value;
  static constexpr int ROW = D + 4;                // of the output in LDS, so that 16 heads lie in other banks

  struct Shared {
    float out[AT_WAVES][AT_HEADS][ROW];
    float top[AT_WAVES][AT_HEADS], sum[AT_WAVES][AT_HEADS], total[AT_HEADS];
    int64_t key_at[AT_WAVES][AT_TILE], value_at[AT_WAVES][AT_TILE];
  };

  const tt_attend_args& a;
  const AttendShape& shape;
  const AttendSpace& space;
  Division by_block;
  Shared& s;
  int lane, wave, c, g;
  int64_t head;  // of keys
  int part;      // which of its query heads

  // The query and the head of it that row r of a product stands for.
  __device__ __forceinline__ int64_t query_of(int64_t i, const Item& q, int r) const { return shape.bundle > 1 ? space.order[q.first + r / shape.group] : i; }
  __device__ __forceinline__ int64_t head_of(int r) const { return head * shape.group + part * AT_HEADS + (shape.bundle > 1 ? r % shape.group : r); }

  // Tokens from `from` up to `end` of item i; slot: where the piece goes, negative: it is the whole output.
  __device__ __forceinline__ void run(int64_t i, const Item& q, uint32_t from, uint32_t end, int64_t slot) {
    const tt_paged_cache& cache = a.cache;
    const uint32_t dim = (uint32_t)cache.dim;
    const int here = shape.bundle > 1 ? q.members * shape.group : min(AT_HEADS, shape.group - part * AT_HEADS);
    // what the lane's own query sees, of several; all of them see the tokens between
    uint32_t own_from = 0, own_upto = ALL, all_from = 0, all_upto = ALL;
    const int64_t own = c < here ? query_of(i, q, c) : 0;
    if (shape.bundle > 1) {
      const Seen mine = seen(a, own);
      own_from = mine.from, own_upto = mine.upto;
      all_upto = seen(a, space.order[q.first]).upto, all_from = seen(a, space.order[q.first + q.members - 1]).from;
    }
    u32x4 query[STEPS];
    const T* row = static_cast<const T*>(a.query) + own * a.query_stride + (c < here ? head_of(c) : 0) * a.query_head_stride;
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      const uint32_t d = EIGHT ? k / 2 * 64 + g * 16 + k % 2 * 8 : k * 32 + g * 8;
      query[k] = 0;
      if (c < here && (WHOLE || d < dim)) query[k] = *reinterpret_cast<const typename Words<4>::type*>(row + d);
    }
    float before = (float)a.scale * (cache.key_scale ? cache.key_scale[head] : 1.0f), after = 0;
    const bool capped = a.softcap > 0;
    if (capped) before /= (float)a.softcap, after = (float)a.softcap * LOG2E;
    else before *= LOG2E;

    const int32_t* table = a.table + (int64_t)q.row * a.table_stride;
    const char* keys = static_cast<const char*>(cache.keys) + head * cache.key_head_stride * SIZE;
    const char* values = static_cast<const char*>(cache.values) + head * cache.value_head_stride * SIZE;
    uint32_t base = from + wave * AT_TILE;

    // A tile's blocks, its addresses in LDS, then its keys and values.
    auto entry_of = [&](uint32_t at) {
      const uint32_t t = at + lane;
      return lane < AT_TILE && t < end ? table[quotient(t, by_block)] : -1;
    };
    auto addresses = [&](int32_t entry, uint32_t at) -> uint32_t {
      const uint32_t t = at + lane;
      const bool there = entry >= 0 && entry < cache.blocks;
      const int64_t block = there ? entry : 0, place = there ? t - quotient(t, by_block) * by_block.divisor : 0;
      if (lane < AT_TILE) {
        s.key_at[wave][lane] = (block * cache.key_block_stride + place * cache.key_place_stride) * SIZE;
        s.value_at[wave][lane] = (block * cache.value_block_stride + place * cache.value_place_stride) * SIZE;
      }
      return (uint32_t)__ballot(there);
    };
    u32x4 key[2][LOADS];
    auto load_keys = [&] {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const char* at = keys + s.key_at[wave][t * 16 + c];
#pragma unroll
        for (int k = 0; k < LOADS; ++k) {
          const uint32_t d = k * 4 * PER + g * PER;
          if (WHOLE) {
            key[t][k] = *reinterpret_cast<const typename Words<4>::type*>(at + d * SIZE);
          } else if (!EIGHT) {  // past the head: its first elements again, against zeros of the query
            key[t][k] = *reinterpret_cast<const typename Words<4>::type*>(at + (d < dim ? d : 0) * SIZE);
            if (d >= dim) key[t][k] = 0;
          } else {
            const auto low = *reinterpret_cast<const typename Words<2>::type*>(at + (d < dim ? d : 0));
            const auto high = *reinterpret_cast<const typename Words<2>::type*>(at + (d + 8 < dim ? d + 8 : 0));
            key[t][k][0] = d < dim ? low[0] : 0, key[t][k][1] = d < dim ? low[1] : 0;
            key[t][k][2] = d + 8 < dim ? high[0] : 0, key[t][k][3] = d + 8 < dim ? high[1] : 0;
          }
        }
      }
    };
    uint32_t value[8][VWORDS];
    auto load_values = [&] {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const char* at = values + s.value_at[wave][k / 4 * 16 + g * 4 + k % 4];
        constexpr int N = VWORDS < 4 ? VWORDS : 4;
#pragma unroll
        for (int w = 0; w < VWORDS; w += N) {
          // past the head: its first elements again, for outputs that are not stored
          uint32_t d = c * MINE + w * 4 / SIZE;
          if constexpr (!WHOLE && N * 4 / SIZE > 8) {  // 16 elements, of which the head may have 8
            const auto low = *reinterpret_cast<const typename Words<2>::type*>(at + (d < dim ? d : 0));
            const auto high = *reinterpret_cast<const typename Words<2>::type*>(at + (d + 8 < dim ? d + 8 : 0));
            value[k][w] = low[0], value[k][w + 1] = low[1], value[k][w + 2] = high[0], value[k][w + 3] = high[1];
          } else {
            if (!WHOLE && d >= dim) d = 0;
            const auto x = *reinterpret_cast<const typename Words<N>::type*>(at + d * SIZE);
            if constexpr (N == 1) {
              value[k][w] = x;
            } else {
#pragma unroll
              for (int n = 0; n < N; ++n) value[k][w + n] = x[n];
            }
          }
        }
      }
    };

    // Columns j and j + 1 of the lane's values, each word of them as `f` has it, for a product over its eight tokens.
    auto columns = [&](int j, auto f, u32x4& even, u32x4& odd) {
      uint32_t pair[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (EIGHT) pair[k] = j % 4 ? widened<T, true>(f(value[k][j / 4])) : widened<T, false>(f(value[k][j / 4]));
        else pair[k] = f(value[k][j / 2]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        even[k] = __builtin_amdgcn_perm(pair[2 * k + 1], pair[2 * k], 0x05040100);
        odd[k] = __builtin_amdgcn_perm(pair[2 * k + 1], pair[2 * k], 0x07060302);
      }
    };

    f32x4 out[MINE];
#pragma unroll
    for (int j = 0; j < MINE; ++j) out[j] = 0;
    float top = -__builtin_inff(), sum = 0;
    [[maybe_unused]] float peak = top;  // the largest score, where the reference may be below it

    int32_t entry = entry_of(base);
    uint32_t there = addresses(entry, base);
    entry = entry_of(base + AT_UNIT);
    if (base < end) {
      load_keys();
      load_values();
    }
    // Without branches: tokens that are not there are read from the cache's first place, and past the last tile nothing else is.
    while (base < end) {
      const uint32_t there_next = addresses(entry, base + AT_UNIT);
      entry = entry_of(base + 2 * AT_UNIT);
      const bool edge = __any(base < all_from || base + AT_TILE > all_upto);  // some queries of a bundle do not see all of the tile
      float x[8];
      {
        f32x4 score[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          score[t] = 0;
#pragma unroll
          for (int k = 0; k < STEPS; ++k) {
            u32x4 w;
            if constexpr (EIGHT) {
              const uint32_t lo = key[t][k / 2][k % 2 * 2], hi = key[t][k / 2][k % 2 * 2 + 1];
              w = u32x4{widened<T, false>(lo), widened<T, true>(lo), widened<T, false>(hi), widened<T, true>(hi)};
            } else {
              w = key[t][k];
            }
            score[t] = product<T>(w, query[k], score[t]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = score[k / 4][k % 4] * before;
          if (capped) x[k] = tanh_of(x[k]) * after;
        }
        if (there != 0xFFFFFFFFu) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!(there >> (k / 4 * 16 + g * 4 + k % 4) & 1)) {
              x[k] = -__builtin_inff();
#pragma unroll
              for (int w = 0; w < VWORDS; ++w) value[k][w] = 0;  // a weight of zero does not take out NaN
            }
        }
        if (edge) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t t = base + k / 4 * 16 + g * 4 + k % 4;
            if (t < own_from || t >= own_upto) x[k] = -__builtin_inff();
          }
          // Infinities and NaN among the values must not reach queries that do not see them, and would by their weights of
          // zero: a product of ones tells which outputs see some, and they are taken out.
          uint32_t some = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int w = 0; w < VWORDS; ++w) some |= not_finite<T, EIGHT>(value[k][w]);
          if (__any(some != 0)) {
            u32x4 seeing;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t t = base + k / 2 * 16 + g * 4 + k % 2 * 2;
              seeing[k] = two<T>(t >= own_from && t < own_upto ? 1.0f : 0.0f, t + 1 >= own_from && t + 1 < own_upto ? 1.0f : 0.0f);
            }
            const uint32_t one = EIGHT ? 0x38 : two<T>(1.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < MINE; j += 2) {
              u32x4 even, odd;
              columns(j, [&](uint32_t w) { return not_finite<T, EIGHT>(w) * one; }, even, odd);
              const f32x4 low = product<T>(even, seeing, f32x4{0, 0, 0, 0}), high = product<T>(odd, seeing, f32x4{0, 0, 0, 0});
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                out[j][r] = low[r] > 0 ? __builtin_nanf("") : out[j][r];
                out[j + 1][r] = high[r] > 0 ? __builtin_nanf("") : out[j + 1][r];
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int w = 0; w < VWORDS; ++w) value[k][w] &= ~(not_finite<T, EIGHT>(value[k][w]) * (EIGHT ? 0xFFu : 0xFFFFu));
          }
        }
      }
      // what follows is kept behind the loads, and the products behind the weights: moved ahead they take half as many registers again
      __builtin_amdgcn_sched_barrier(0);
      load_keys();
      __builtin_amdgcn_sched_barrier(0);
      {
        // weights go by a reference that is moved where a tile's largest score is far from it, which most tiles' are not: by a maximum that may be 8 too low,
        // so that they stay below 2^8
        float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if constexpr (HALF) {
          // Terms of float16 end at 2^-24, whatever the sum that they go into. So the reference goes down with the scores too: a tile's largest
          // weight is 2^15 at most and 2^-3 at least, what its others lose is 2^-22 of that.  (Below 2^-48 of all a tile may have fewer bits, for the sums to stay
          // in range.)
          most = across_groups_max(most);
          peak = fmaxf(peak, most);
          const float to = fmaxf(most, peak - 48.0f) - 7.0f;
          const bool move = to > top + 8.0f || (to < top - 10.0f && most > -__builtin_inff());
          if (__any(move)) {
            const float by = move ? __builtin_amdgcn_exp2f(top - to) : 1.0f;
            top = move ? to : top;
            sum *= by;
#pragma unroll
            for (int j = 0; j < MINE; ++j) out[j] *= by;
          }
        } else if (__any(most > top + 8.0f)) {
          most = fmaxf(over_groups(most, false), top);
          const float by = most == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(top - most);
          top = most;
          sum *= by;
#pragma unroll
          for (int j = 0; j < MINE; ++j) out[j] *= by;
        }
        const float less = top == -__builtin_inff() ? 0.0f : top;
        // weights in two terms of 16 bits each, together good for 16 bits of mantissa (float16: 22, down to 2^-25): rounded to one they
        // would cost as much as the output's own rounding
        u32x4 weight, rest;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = __builtin_amdgcn_exp2f(x[k] - less);
          sum += x[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          weight[k] = two<T>(x[2 * k], x[2 * k + 1]);
          rest[k] = two<T>(x[2 * k] - one_of<T>(weight[k], 0), x[2 * k + 1] - one_of<T>(weight[k], 1));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < MINE; j += 2) {
          u32x4 even, odd;
          columns(j, [](uint32_t w) { return w; }, even, odd);
          out[j] = product<T>(even, weight, out[j]);
          out[j] = product<T>(even, rest, out[j]);
          out[j + 1] = product<T>(odd, weight, out[j + 1]);
          out[j + 1] = product<T>(odd, rest, out[j + 1]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      load_values();
      there = there_next;
      base += AT_UNIT;
    }

    // the wavefronts' parts together
    sum = over_groups(sum, true);
    if constexpr (HALF) {
      if (peak > -__builtin_inff()) sum *= __builtin_amdgcn_exp2f(top - peak);
      if (g == 0) s.top[wave][c] = peak, s.sum[wave][c] = sum;
    } else {
      if (g == 0) s.top[wave][c] = top, s.sum[wave][c] = sum;
    }
    __syncthreads();
    float all = s.top[0][c], total = 0;
#pragma unroll
    for (int w = 1; w < AT_WAVES; ++w) all = fmaxf(all, s.top[w][c]);
    const float less = all == -__builtin_inff() ? 0.0f : all;
#pragma unroll
    for (int w = 0; w < AT_WAVES; ++w) total += s.sum[w][c] * __builtin_amdgcn_exp2f(s.top[w][c] - less);
    const float by = __builtin_amdgcn_exp2f(top - less);
    if (c < here) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < MINE; j += 4)
          *reinterpret_cast<f32x4*>(&s.out[wave][c][(g * 4 + r) * MINE + j]) =
              f32x4{out[j][r], out[j + 1][r], out[j + 2][r], out[j + 3][r]} * by;
    }
    const int64_t unit = head * shape.parts + part;
    if (wave == 0 && g == 0 && c < here) {
      if (slot < 0) {
        if (a.lse) a.lse[own * a.lse_stride + head_of(c)] = total == 0 ? -__builtin_inff() : (all + __log2f(total)) * LN2;
      } else {
        float* to = space.statistic + ((slot * shape.lanes + unit) * shape.rows + c) * 2;
        to[0] = all, to[1] = total;
      }
      s.total[c] = total;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < here * (D / 8); e += AT_THREADS) {
      const int row = e / (D / 8), d = e % (D / 8) * 8;
      f32x4 y[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < AT_WAVES; ++w)
#pragma unroll
        for (int k = 0; k < 2; ++k) y[k] += *reinterpret_cast<const f32x4*>(&s.out[w][row][d + 4 * k]);
      if (slot < 0) {
        if (!WHOLE && d >= (int)dim) continue;
        const float of = s.total[row], scale = (cache.value_scale ? cache.value_scale[head] : 1.0f) / of;
        typename Eight<T>::type z;
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = (T)(of == 0 ? 0.0f : y[k / 4][k % 4] * scale);
        *reinterpret_cast<typename Eight<T>::type*>(static_cast<T*>(a.out) + query_of(i, q, row) * a.out_stride +
                                                    head_of(row) * a.out_head_stride + d) = z;
      } else {
        float* to = space.piece + ((slot * shape.lanes + unit) * shape.rows + row) * D + d;
#pragma unroll
        for (int k = 0; k < 2; ++k) *reinterpret_cast<f32x4*>(to + 4 * k) = y[k];
      }
    }
    __syncthreads();  // before the next query's parts
  }
};

// Units that an item's tokens take; one that sees nothing has one too, to put out its zeros.
__device__ inline int64_t units_of(uint32_t from, uint32_t upto) { return max((upto - from + AT_UNIT - 1) / AT_UNIT, 1u); }

// Sums over the workgroup, with the sum of all.
template <int N>
__device__ inline int64_t group_sums(int64_t v, int64_t* of_wave, int64_t& all) {
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  int64_t upto = (int64_t)sums_upto((u64)v);
  __syncthreads();
  if (lane == WAVE - 1) of_wave[wave] = upto;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < N / WAVE; ++w) {
    if (w == wave) upto += all;
    all += of_wave[w];
  }
  return upto;
}

constexpr int BU_THREADS = AT_QUERIES;

// Puts the queries of a call in the order of rows and, within a row, of their last tokens, and those of a row that see some of the same tokens into bundles: so
// no bundle reads more tokens than its queries do one by one.  By one workgroup, a query a thread, which is why a call may have at
// most as many.  A chain of 45 exchanges and three sums: 7.3 us for 301 queries of 40 rows.  A call of these, which see 1,024 tokens of 12
// heads each, takes 51 us with bundles, 108 without.
__global__ __launch_bounds__(BU_THREADS) void k_bundle(tt_attend_args a, AttendShape shape, AttendSpace space) {
  __shared__ u64 s_key[BU_THREADS];
  __shared__ int64_t s_wave[BU_THREADS / WAVE];
  __shared__ int32_t s_first[BU_THREADS + 1];
  __shared__ Seen s_seen[BU_THREADS];
  const int tid = threadIdx.x, n = (int)a.queries;
  u64 key = 0;  // the largest first, so inverted
  if (tid < n) {
    s_seen[tid] = seen(a, tid);
    // rows are fewer than queries, so below 2^9
    key = ~(((u64)s_seen[tid].row << 32 | s_seen[tid].upto) << 9 | (u64)tid);
  }
#pragma unroll 1
  for (int run = 2; run / 2 < n; run *= 2) {
#pragma unroll 1
    for (int apart = run / 2; apart >= WAVE; apart /= 2) {
      __syncthreads();
      s_key[tid] = key;
      __syncthreads();
      const u64 other = s_key[tid ^ apart];
      key = (!(tid & apart) == !(tid & run)) == (other > key) ? other : key;
    }
    key = exchanged_in_wave(key, tid, run);
  }
  key = ~key;
  __syncthreads();
  s_key[tid] = key;
  __syncthreads();
  const int i = (int)(key & (BU_THREADS - 1));
  const Seen own = tid < n ? s_seen[i] : Seen{0, 0, 0};
  bool first = tid < n;
  if (tid > 0 && tid < n) {
    const Seen before = s_seen[s_key[tid - 1] & (BU_THREADS - 1)];
    first = before.row != own.row || own.from > before.upto;
  }
  // where the run of queries that this one is of starts: the number of starts, and each start's place
  int64_t all;
  const int64_t runs = group_sums<BU_THREADS>(first, s_wave, all);
  if (first) s_first[runs - 1] = tid;
  __syncthreads();
  const int nth = tid < n ? tid - s_first[runs - 1] : 1;
  const bool opens = tid < n && nth % shape.bundle == 0;
  int64_t items;
  const int64_t item = group_sums<BU_THREADS>(opens, s_wave, items) - 1;
  __syncthreads();
  if (opens) s_first[item] = tid;
  if (tid == 0) s_first[items] = n;
  __syncthreads();
  if (tid < n) {
    space.order[tid] = i;
    space.place[i] = (int32_t)item * AT_HEADS + tid - s_first[item];
  }
  Item mine{0, 0, 0, 0, 0};
  if (tid < items) {
    mine.first = s_first[tid], mine.members = s_first[tid + 1] - mine.first;
    const Seen from = s_seen[s_key[mine.first] & (BU_THREADS - 1)], upto = s_seen[s_key[mine.first + mine.members - 1] & (BU_THREADS - 1)];
    mine.row = from.row, mine.from = from.from, mine.upto = upto.upto;
    space.item[tid] = mine;
  }
  const int64_t units = tid < items ? units_of(mine.from, mine.upto) : 0;
  int64_t sum;
  const int64_t upto = group_sums<BU_THREADS>(units, s_wave, sum);
  space.start[tid] = upto - units;  // past the last item: all units
  if (tid == 0) space.start[BU_THREADS] = sum;
}

// Workgroups of the same lane share out the units of all items evenly, so that short and long requests do not wait for
// each other; where the cut goes through an item its pieces are joined by k_join.  As many workgroups as the card holds at once: each
// sums up the items by itself, which costs it less than a launch that does so would.
template <class T, bool EIGHT, int D, bool WHOLE>
__global__ __launch_bounds__(AT_THREADS, D == 256 ? 1 : D == 64 ? 3 : 2) void k_attend(tt_attend_args a, AttendShape shape, AttendSpace space,
                                                                                   Division by_block, int64_t first) {
  typedef Attend<T, EIGHT, D, WHOLE> Work;
  __shared__ typename Work::Shared s;
  __shared__ int64_t s_start[AT_QUERIES + 1], s_wave[AT_WAVES];
  __shared__ Seen s_seen[AT_QUERIES];
  const int64_t id = first + blockIdx.x, unit = id % shape.lanes;
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  Work work{a, shape, space, by_block, s, lane, wave, lane % 16, lane / 16, unit / shape.parts, (int)(unit % shape.parts)};
  if (!shape.workers) {
    const int64_t i = id / shape.lanes;
    const Seen q = seen(a, i);
    work.run(i, Item{q.row, 1, 0, q.from, q.upto}, q.from, q.upto, -1);
    return;
  }
  constexpr int MANY = AT_QUERIES / AT_THREADS;
  const int n = (int)a.queries;
  if (shape.bundle > 1) {
    for (int k = tid; k <= AT_QUERIES; k += AT_THREADS) s_start[k] = space.start[k];
  } else {
    const int per = (n + AT_THREADS - 1) / AT_THREADS;
    Seen q[MANY];
    int64_t units = 0, all;
#pragma unroll
    for (int k = 0; k < MANY; ++k) {
      const int i = tid * per + k;
      if (k < per && i < n) q[k] = seen(a, i);
    }
#pragma unroll
    for (int k = 0; k < MANY; ++k)
      if (k < per && tid * per + k < n) units += units_of(q[k].from, q[k].upto);
    int64_t at = group_sums<AT_THREADS>(units, s_wave, all) - units;
#pragma unroll
    for (int k = 0; k < MANY; ++k) {
      const int i = tid * per + k;
      if (k < per && i < n) {
        s_start[i] = at, s_seen[i] = q[k];
        at += units_of(q[k].from, q[k].upto);
      }
    }
    if (tid == 0) s_start[n] = all;
  }
  __syncthreads();
  const int worker = (int)(id / shape.lanes);
  // past the last item there are no units; each worker has one at least, so an item's pieces have workers in a row
  const int64_t all = s_start[shape.bundle > 1 ? AT_QUERIES : n], sharers = min((int64_t)shape.workers, all);
  if (worker >= sharers) return;
  const int64_t upto = all * (worker + 1) / sharers;
  int64_t at = all * worker / sharers;
  int lo = 0, hi = n;  // the last item that starts at `at` or before, and has units
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (s_start[mid] <= at) lo = mid;
    else hi = mid;
  }
  for (int nth = 0; at < upto; ++nth, ++lo) {
    const int64_t begin = s_start[lo], end = s_start[lo + 1], stop = min(end, upto);
    const int slot = 2 * worker + (nth > 0);
    const bool whole = at == begin && stop == end;
    // the worker of its last unit: the first one whose share reaches the item's end
    if (tid == 0 && at == begin && shape.workers > 1) space.pieces[lo * shape.lanes + unit] = int2{slot, (int)((end * sharers + all - 1) / all) - worker};
    const Item q = shape.bundle > 1 ? space.item[lo] : Item{s_seen[lo].row, 1, 0, s_seen[lo].from, s_seen[lo].upto};
    work.run(lo, q, q.from + (uint32_t)(at - begin) * AT_UNIT, stop == end ? q.upto : q.from + (uint32_t)(stop - begin) * AT_UNIT,
             whole ? -1 : slot);
    at = stop;
  }
}

// The pieces of a query head together, by THREADS of a workgroup: the first one, and the first one of each worker after its own.  `across`
// threads go by the elements, four each, of `split` workgroups a head; the others by the pieces, each with a maximum of its own. Bound by
// the launch and two dependent reads: 5 us for a few heads, 6.7 for 32 heads of up to 256 pieces, 5.6 for 4,096.
template <class T, int THREADS>
__global__ __launch_bounds__(AT_THREADS) void k_join(tt_attend_args a, AttendShape shape, AttendSpace space, int wide, int split) {
  __shared__ f32x4 s_out[AT_THREADS];
  __shared__ float s_top[AT_THREADS], s_sum[AT_THREADS];
  constexpr int HEADS = AT_THREADS / THREADS;
  const int at_block = threadIdx.x / THREADS * THREADS, tid = threadIdx.x - at_block;
  const int64_t id = (int64_t)(blockIdx.x / split) * HEADS + threadIdx.x / THREADS, i = id / a.heads;
  const int h = (int)(id % a.heads), kv = h / shape.group, nth = h % shape.group;
  const int64_t unit = (int64_t)kv * shape.parts + nth / AT_HEADS;
  const bool here = i < a.queries;
  const int32_t place = shape.bundle > 1 ? (here ? space.place[i] : 0) : (int32_t)(i * AT_HEADS);
  const int64_t row = place % AT_HEADS * shape.group + nth % AT_HEADS;
  const int2 of = here ? space.pieces[place / AT_HEADS * shape.lanes + unit] : int2{0, 1};
  const bool cut = of.y > 1;
  const int before = of.x / 2, across = wide / 4 / split, side = THREADS / across;
  const int d = (blockIdx.x % split * across + tid % across) * 4;
  float top = -__builtin_inff(), sum = 0;
  f32x4 y = 0;
#pragma unroll 4
  for (int k = cut ? tid / across : of.y; k < of.y; k += side) {
    const int64_t at = ((k ? 2 * (before + k) : of.x) * shape.lanes + unit) * shape.rows + row;
    const float m = space.statistic[at * 2], l = space.statistic[at * 2 + 1];
    const f32x4 x = *reinterpret_cast<const f32x4*>(space.piece + at * wide + d);
    const float most = fmaxf(top, m), less = most == -__builtin_inff() ? 0.0f : most;
    const float old = __builtin_amdgcn_exp2f(top - less), by = __builtin_amdgcn_exp2f(m - less);
    y = y * old + x * by, sum = sum * old + l * by, top = most;
  }
  s_out[threadIdx.x] = y, s_top[threadIdx.x] = top, s_sum[threadIdx.x] = sum;
  __syncthreads();
  if (tid >= across || !cut) return;
  float most = top;
  for (int k = 1; k < side; ++k) most = fmaxf(most, s_top[at_block + k * across + tid]);
  const float less = most == -__builtin_inff() ? 0.0f : most;
  sum = 0, y = 0;
  for (int k = 0; k < side; ++k) {
    const int at = at_block + k * across + tid;
    const float by = __builtin_amdgcn_exp2f(s_top[at] - less);
    y += s_out[at] * by, sum += s_sum[at] * by;
  }
  if (tid == 0 && blockIdx.x % split == 0 && a.lse) a.lse[i * a.lse_stride + h] = sum == 0 ? -__builtin_inff() : (most + __log2f(sum)) * LN2;
  if (d >= a.cache.dim) return;
  const float scale = (a.cache.value_scale ? a.cache.value_scale[kv] : 1.0f) / sum;
  T* to = static_cast<T*>(a.out) + i * a.out_stride + h * a.out_head_stride + d;
#pragma unroll
  for (int k = 0; k < 4; ++k) to[k] = (T)(sum == 0 ? 0.0f : y[k] * scale);
}

template <class T, bool EIGHT, int D, bool WHOLE>
void enqueue_attend(const tt_attend_args& a, const AttendShape& shape, const AttendSpace& space, hipStream_t st) {
  const Division by_block = division(a.cache.block_size);
  const int64_t groups = shape.lanes * (shape.workers ? shape.workers : a.queries), most = MAX_ITEMS / AT_THREADS;
  for (int64_t at = 0; at < groups; at += most)
    hipLaunchKernelGGL((k_attend<T, EIGHT, D, WHOLE>), dim3((uint32_t)std::min(most, groups - at)), dim3(AT_THREADS), 0, st, a,
                       shape, space, by_block, at);
}

template <class T, bool EIGHT>
void enqueue_attend(const tt_attend_args& a, const AttendShape& shape, const AttendSpace& space, hipStream_t st) {
  switch (a.cache.dim) {
    case 64: return enqueue_attend<T, EIGHT, 64, true>(a, shape, space, st);
    case 128: return enqueue_attend<T, EIGHT, 128, true>(a, shape, space, st);
    case 256: return enqueue_attend<T, EIGHT, 256, true>(a, shape, space, st);
  }
  if (a.cache.dim < 64) return enqueue_attend<T, EIGHT, 64, false>(a, shape, space, st);
  if (a.cache.dim < 128) return enqueue_attend<T, EIGHT, 128, false>(a, shape, space, st);
  return enqueue_attend<T, EIGHT, 256, false>(a, shape, space, st);
}

template <class I, class O>
void enqueue_write(const tt_write_args& a, hipStream_t st) {
  const int64_t per_head = a.cache.dim / 8, per_token = a.cache.heads * per_head, most = 0x7FFFFFFF / per_token;  // tokens of a launch
  for (int64_t at = 0; at < a.tokens; at += most) {
    const uint32_t total = (uint32_t)(std::min(most, a.tokens - at) * per_token);
    hipLaunchKernelGGL((k_write<I, O>), dim3((uint32_t)div_up(total, WR_THREADS)), dim3(WR_THREADS), 0, st, a, division(per_token), division(per_head),
                       division(a.cache.block_size), at, total);
  }
}

template <class I>
void enqueue_write(const tt_write_args& a, hipStream_t st) {
  if (a.cache.type == TT_E4M3) enqueue_write<I, uint8_t>(a, st);
  else if (a.cache.type == TT_F16) enqueue_write<I, _Float16>(a, st);
  else enqueue_write<I, __bf16>(a, st);
}

}  // namespace

hipError_t launch_write(const tt_write_args& a, hipStream_t st) {
  if (a.in_type == TT_F32) enqueue_write<float>(a, st);
  else if (a.in_type == TT_F16 && a.cache.type == TT_E4M3) enqueue_write<_Float16, uint8_t>(a, st);
  else if (a.in_type == TT_F16) enqueue_write<_Float16, _Float16>(a, st);
  else if (a.cache.type == TT_E4M3) enqueue_write<__bf16, uint8_t>(a, st);
  else enqueue_write<__bf16, __bf16>(a, st);
  return hipGetLastError();
}

int64_t attend_workspace(int64_t queries, int64_t heads, int64_t cache_heads, int64_t dim) {
  // of the calls of these sizes the one that needs most
  int64_t bytes = 0;
  for (bool shared : {false, true})
    bytes = std::max(bytes, attend_space(attend_shape(queries, heads, cache_heads, dim, shared ? 0 : queries, shared), queries, dim, nullptr).bytes);
  return bytes;
}

hipError_t launch_attend(const tt_attend_args& a, hipStream_t st) {
  const bool eight = a.cache.type == TT_E4M3, half = a.type == TT_F16;
  const AttendShape shape = attend_shape(a.queries, a.heads, a.cache.heads, a.cache.dim, a.table_rows, a.rows != nullptr);
  const AttendSpace space = attend_space(shape, a.queries, a.cache.dim, a.workspace);
  if (shape.bundle > 1) hipLaunchKernelGGL(k_bundle, dim3(1), dim3(BU_THREADS), 0, st, a, shape, space);
  if (half && eight) enqueue_attend<_Float16, true>(a, shape, space, st);
  else if (half) enqueue_attend<_Float16, false>(a, shape, space, st);
  else if (eight) enqueue_attend<__bf16, true>(a, shape, space, st);
  else enqueue_attend<__bf16, false>(a, shape, space, st);
  if (shape.workers > 1) {
    // few heads are joined by several workgroups each: 32 heads of 256 pieces take 10 us with one
    const int64_t heads = a.queries * a.heads;
    const int split = heads <= 128 ? padded(a.cache.dim) / 32 : 1;
    // many by a wavefront each: 3,612 take 5.1 us so and 8.8 with a workgroup each, calls with 1,600 14.6 and 15.4, with 512 28.2 and 27.1
    const bool many = heads >= 1024;
    auto* k = many ? (half ? k_join<_Float16, WAVE> : k_join<__bf16, WAVE>) : (half ? k_join<_Float16, AT_THREADS> : k_join<__bf16, AT_THREADS>);
    const int64_t groups = many ? div_up(heads, AT_THREADS / WAVE) : heads * split;
    hipLaunchKernelGGL(k, dim3((uint32_t)groups), dim3(AT_THREADS), 0, st, a, shape, space, padded(a.cache.dim), many ? 1 : split);
  }
  return hipGetLastError();
}

}  // namespace tt

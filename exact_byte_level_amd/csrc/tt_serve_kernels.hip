// tt_serve_kernels.hip -- block tables, token sets, grammar masks and the
// shaping of logits (declared in include/tt_serve.h).
#include "tt_serve_kernels.h"

#include <algorithm>
#include <type_traits>

namespace tt {
namespace {

constexpr int WAVE = 64;
constexpr int64_t MAX_ITEMS = 0xFFFFFFFF;  // threads that a launch may have in a dimension of its grid

__host__ __device__ inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline uint32_t div_up32(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

// ---------------------------------------------------------------- block tables

constexpr int BT_THREADS = 256;
constexpr int BT_WAVES = BT_THREADS / WAVE;
constexpr int BT_MANY = 4;                       // rows, places or blocks of a thread that are on their way together
constexpr int BT_PART = BT_THREADS * BT_MANY;    // rows, places or blocks of a workgroup at a time

// Data errors, as bits; the lowest one set is reported.
constexpr uint32_t BAD_OFFSETS = 1, BAD_FREE = 2, BAD_SIZE = 4, BAD_NONE_LEFT = 8;

__device__ inline int64_t fault_code(uint32_t bad) {
  if (bad & BAD_OFFSETS) return TT_EOFFSETS;
  if (bad & BAD_FREE) return TT_EINVAL;
  if (bad & BAD_SIZE) return TT_ETOOBIG;
  return TT_ENOBLOCKS;
}

// v plus what the lanes `CTRL` says (of the rows of 16 in ROWS) hold of it.
template <int CTRL, int ROWS>
__device__ inline uint32_t plus_lanes(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}

// Inclusive sums over the lanes of a row of 16, and of a wavefront: lane
// shifts by 1, 2, 4, 8, then the last lanes of rows 0 and 2, then of row 1.
__device__ inline uint32_t row_sums(uint32_t v) {
  v = plus_lanes<0x111, 0xf>(v);
  v = plus_lanes<0x112, 0xf>(v);
  v = plus_lanes<0x114, 0xf>(v);
  return plus_lanes<0x118, 0xf>(v);
}
__device__ inline uint32_t wave_sums(uint32_t v) {
  return plus_lanes<0x143, 0xc>(plus_lanes<0x142, 0xa>(row_sums(v)));
}

// Inclusive sums of K values over the workgroup (modulo 2^32), with their totals.
template <int K>
__device__ inline void block_sums(uint32_t (&v)[K], uint32_t (&total)[K], uint32_t (*lds)[BT_WAVES]) {
  static_assert(BT_WAVES <= 16, "the wavefronts' totals fit a row of lanes");
  const int lane = threadIdx.x % WAVE, w = threadIdx.x / WAVE;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sums(v[k]);
  if (lane == WAVE - 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) lds[k][w] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const uint32_t all = row_sums(lane < BT_WAVES ? lds[k][lane] : 0);
    total[k] = (uint32_t)__builtin_amdgcn_readlane((int)all, BT_WAVES - 1);
    const int before = __builtin_amdgcn_readfirstlane(w) - 1;
    v[k] += before >= 0 ? (uint32_t)__builtin_amdgcn_readlane((int)all, max(before, 0)) : 0;
  }
}

// Sums of blocks, which may pass 32 bits, go as two: of 22 bits each, and of
// the rest, up to 2^40 (more than any free list has) from a thread.
constexpr int LOW = 22;
static_assert(BT_THREADS << LOW <= 1u << 31 && (int64_t)BT_THREADS << (40 - LOW) <= 1u << 31, "both sums fit 32 bits");
__device__ inline int64_t capped(int64_t v) { return min(v, (int64_t)1 << 40); }
__device__ inline uint32_t low(int64_t v) { return (uint32_t)v & ((1u << LOW) - 1); }
__device__ inline uint32_t high(int64_t v) { return (uint32_t)(v >> LOW); }
__device__ inline int64_t joined(uint32_t lo, uint32_t hi) { return (int64_t)lo + ((int64_t)hi << LOW); }

// For each t: the last of ROWS rows that starts at or before it.
template <int ROWS>
__device__ inline void last_rows(const uint32_t* start, const uint32_t (&t)[BT_MANY], int (&row)[BT_MANY]) {
#pragma unroll
  for (int k = 0; k < BT_MANY; ++k) row[k] = 0;
#pragma unroll
  for (int d = ROWS / 2; d > 0; d >>= 1)
#pragma unroll
    for (int k = 0; k < BT_MANY; ++k)
      if (start[row[k] + d] <= t[k]) row[k] += d;
}

// One row of a plan: as given, where its new tokens start, how many they
// are, the blocks it has and the ones it needs.
struct RowPlan {
  int32_t length;
  int64_t from, upto;  // its places
  uint32_t start, held, need;
  int64_t count;
};

template <bool SINGLE>
__device__ inline RowPlan row_loads(const tt_plan_args& a, int64_t r) {
  RowPlan p;
  p.length = a.lengths[r];
  p.from = SINGLE ? r : a.offsets[r];
  p.upto = SINGLE ? r + 1 : a.offsets[r + 1];
  return p;
}

template <bool SINGLE>
__device__ inline void row_plan(const tt_plan_args& a, RowPlan& p, uint32_t& bad) {
  const int64_t start = p.length > 0 ? p.length : 0;
  p.count = SINGLE ? p.length >= 0 : p.upto - p.from;
  p.start = (uint32_t)start;
  p.held = p.need = 0;
  if (p.count < 0) {
    bad |= BAD_OFFSETS;
    p.count = 0;
  }
  const int64_t room = a.width * a.block_size - start;  // width * block_size < 2^31
  if (p.count > room) {
    bad |= BAD_SIZE;
    p.count = 0;
    return;
  }
  const uint32_t bs = (uint32_t)a.block_size;
  p.held = div_up32(p.start, bs);
  p.need = div_up32(p.start + (uint32_t)p.count, bs) - p.held;
}

__device__ inline void put_place(const tt_plan_args& a, int64_t t, int64_t slot, int32_t position, int32_t row) {
  a.slots[t] = slot;
  if (a.positions) a.positions[t] = position;
  if (a.row_of) a.row_of[t] = row;
}

// The places of the new tokens, and the blocks they need.
//
// Exclusive sums of the rows' needs say which entries of the free list a row
// takes.  Every workgroup sums up all rows by itself (a few KB from L2), so that
// one launch is enough and no workgroup waits for another one's sums; up to
// 256 rows each thread reads one row, once.  Then it fills its part of the places,
// four to a thread with their row searches and look-ups on their way together.
// One to 256 rows with a token each take 3.0 us, which is the launch and three
// dependent reads; 1,500 rows with 48,000 tokens 6.9 us; 64 rows with two million
// 12.4 us, 2.7 TB/s of the 16 bytes written for a token (a fill of as many bytes
// takes 8.5 us).  Past 256 rows two loops go by 256 rows at a time, a round trip each: the
// walk to the rows of a part, and the finisher's, whose stores may be what it loads next.  4,000 rows with a token each
// take 9.1 us by place and 15.6 us by offsets; in place, where the finisher has a launch of its own, 14.7 and 21.3 us.
// `finisher`: the workgroup that writes the lengths and counts; it may be one without places.
template <bool SINGLE>
__global__ __launch_bounds__(BT_THREADS) void k_plan(tt_plan_args a, int64_t per_block, int finisher) {
  __shared__ uint32_t s_sums[2][5][BT_WAVES];
  __shared__ uint32_t s_bad;
  __shared__ uint32_t s_off[BT_THREADS + 1], s_start[BT_THREADS], s_held[BT_THREADS], s_base[BT_THREADS];
  const int tid = threadIdx.x;
  const int64_t t0 = min((int64_t)blockIdx.x * per_block, a.places);
  const int64_t t1 = min(t0 + per_block, a.places);
  const bool few = a.rows <= BT_THREADS;
  const int64_t n_free = *a.n_free, last = SINGLE ? a.rows : a.offsets[a.rows], first = SINGLE ? 0 : a.offsets[0];
  if (tid == 0) s_bad = 0;
  // all blocks needed; those of the rows that end at or before t0, and how many rows that are; tokens
  int64_t all = 0;
  uint32_t before = 0, rows_before = 0, count = 0, bad = 0, unused = 0;
  RowPlan mine{-1, 0, 0, 0, 0, 0, 0};
  for (int64_t base = 0; base < a.rows; base += BT_PART) {
    RowPlan p[BT_MANY];
#pragma unroll
    for (int k = 0; k < BT_MANY; ++k)
      if (base + k * BT_THREADS < a.rows) p[k] = row_loads<SINGLE>(a, min(base + k * BT_THREADS + tid, a.rows - 1));
#pragma unroll
    for (int k = 0; k < BT_MANY; ++k)
      if (base + k * BT_THREADS + tid < a.rows) {
        row_plan<SINGLE>(a, p[k], bad);
        const bool past = p[k].upto <= t0;
        all += p[k].need;
        before += past ? p[k].need : 0;
        rows_before += past;
        count += (uint32_t)p[k].count;
        mine = p[k];  // the only one, of few rows
      }
  }
  if (first != 0) bad |= BAD_OFFSETS;
  if (last > a.places) bad |= BAD_SIZE;
  if (n_free < 0 || n_free > a.free_cap) bad |= BAD_FREE;
  __syncthreads();
  if (bad) atomicOr(&s_bad, bad);
  all = capped(all);
  uint32_t v[5] = {low(all), high(all), before, rows_before, count}, total[5];
  block_sums(v, total, s_sums[1]);
  bad = s_bad;
  const int64_t needed = joined(total[0], total[1]), tokens = SINGLE ? (int64_t)total[4] : last;
  if (needed > n_free) bad |= BAD_NONE_LEFT;
  const int64_t end = min(t1, bad ? 0 : last);  // of the places that may hold a token
  const uint32_t bs = (uint32_t)a.block_size;
  uint32_t carry = few ? 0 : total[2];
  int turn = 0;
  for (int64_t c0 = few ? 0 : total[3]; t0 < end && c0 < a.rows; c0 += BT_THREADS, ++turn) {
    const int64_t r = c0 + tid;
    RowPlan p{-1, 0, 0, 0, 0, 0, 0};
    uint32_t base;
    if (few) {  // a thread has had one row: its sum is there
      p = mine;
      base = (uint32_t)joined(v[0], v[1]) - p.need;
    } else {
      if (r < a.rows) {
        p = row_loads<SINGLE>(a, r);
        row_plan<SINGLE>(a, p, unused);
      }
      uint32_t s[1] = {p.need}, chunk[1];
      block_sums(s, chunk, s_sums[turn & 1]);
      base = carry + s[0] - p.need;
      carry += chunk[0];
    }
    if (SINGLE) {  // place r is row r's
      if (r >= t0 && r < end) {
        const uint32_t blk = p.start / bs, in = p.start - blk * bs;
        int32_t id = -1;
        if (p.need) a.table[r * a.table_stride + blk] = id = a.free_blocks[n_free - 1 - (int64_t)base];
        else if (p.length >= 0) id = a.table[r * a.table_stride + blk];
        const bool live = p.length >= 0;
        put_place(a, r, live && id >= 0 ? (int64_t)id * bs + in : -1, live ? (int32_t)p.start : -1, live ? (int32_t)r : -1);
      }
      if (c0 + BT_THREADS >= end) break;
      continue;
    }
    s_off[tid] = (uint32_t)(r < a.rows ? p.from : last);
    if (tid == BT_THREADS - 1) s_off[BT_THREADS] = (uint32_t)(r < a.rows ? p.upto : last);
    s_start[tid] = p.start;
    s_held[tid] = p.held;
    s_base[tid] = base;
    __syncthreads();
    const uint32_t lo = max((uint32_t)t0, s_off[0]), hi = min((uint32_t)end, s_off[BT_THREADS]);
    for (uint32_t t = lo; t < hi; t += BT_PART) {
      uint32_t at[BT_MANY], in[BT_MANY];
      int i[BT_MANY];
      int32_t id[BT_MANY];
#pragma unroll
      for (int k = 0; k < BT_MANY; ++k) at[k] = min(t + k * BT_THREADS + tid, hi - 1);
      last_rows<BT_THREADS>(s_off, at, i);
      int32_t* entry[BT_MANY];  // of a new block that starts here
#pragma unroll
      for (int k = 0; k < BT_MANY; ++k) {
        const uint32_t place = s_start[i[k]] + (at[k] - s_off[i[k]]), blk = place / bs, held = s_held[i[k]];
        in[k] = place - blk * bs;
        int32_t* own = a.table + (c0 + i[k]) * a.table_stride + blk;
        const int32_t* from = blk >= held ? a.free_blocks + (n_free - 1 - (int64_t)(s_base[i[k]] + (blk - held))) : own;
        id[k] = *from;
        entry[k] = blk >= held && in[k] == 0 ? own : nullptr;
      }
#pragma unroll
      for (int k = 0; k < BT_MANY; ++k) {
        if (t + k * BT_THREADS + tid >= hi) break;
        if (entry[k]) *entry[k] = id[k];
        put_place(a, at[k], id[k] >= 0 ? (int64_t)id[k] * bs + in[k] : -1,
                  (int32_t)(s_start[i[k]] + (at[k] - s_off[i[k]])), (int32_t)(c0 + i[k]));
      }
    }
    if (hi >= end) break;
    __syncthreads();
  }
  for (int64_t t = max(t0, bad ? 0 : last) + tid; t < t1; t += BT_THREADS) put_place(a, t, -1, -1, -1);
  if ((int)blockIdx.x != finisher) return;
  __syncthreads();  // out_lengths may be lengths, which every thread has read by now
  for (int64_t r = tid; r < a.rows; r += BT_THREADS) {
    if (!few) {
      mine = row_loads<SINGLE>(a, r);
      row_plan<SINGLE>(a, mine, unused);
    }
    a.out_lengths[r] = bad || mine.count == 0 ? mine.length : (int32_t)(mine.start + (uint32_t)mine.count);
  }
  if (tid == 0) {
    *a.out_n_free = (int32_t)(bad ? n_free : n_free - needed);
    *a.out_n = bad ? fault_code(bad) : tokens;
  }
}

// The blocks that the thread's rows of the BT_PART from c0 on give back, and the rows' lengths afterwards.
__device__ inline void row_releases(const ReleaseArgs& a, int64_t c0, uint32_t (&m)[BT_MANY], int32_t (&length)[BT_MANY],
                                    uint32_t& bad) {
  bool done[BT_MANY];
#pragma unroll
  for (int k = 0; k < BT_MANY; ++k) {
    const int64_t r = c0 + BT_MANY * threadIdx.x + k, at = min(r, a.rows - 1);
    length[k] = a.lengths[at];
    done[k] = a.done[at] != 0 && r < a.rows;
  }
#pragma unroll
  for (int k = 0; k < BT_MANY; ++k) {
    m[k] = 0;
    if (!done[k] || length[k] < 0) continue;
    m[k] = div_up32((uint32_t)length[k], (uint32_t)a.block_size);
    if (m[k] > a.width) {
      bad |= BAD_SIZE;
      m[k] = 0;
    }
    length[k] = -1;
  }
}

// The blocks that come back, moved to the free list.  As in k_plan each
// workgroup sums up all rows (1,024 at a time, since the rows' sums have to be
// there before a part can begin), then copies its part.  16 rows take 3.9 us, 660,000
// blocks of 512 rows out of 1,024 7.7 us, of which the copy itself is about one: a workgroup has two or three turns of
// search, read and write.  4,000 rows take 15.4 us, in place, with a second launch to finish, 17.3 us.
__global__ __launch_bounds__(BT_THREADS) void k_release(ReleaseArgs a, bool fill, int finisher) {
  __shared__ uint32_t s_sums[2][2][BT_WAVES];
  __shared__ uint32_t s_bad;
  __shared__ __attribute__((aligned(16))) uint32_t s_base[BT_PART];
  const int tid = threadIdx.x;
  const bool few = a.rows <= BT_PART;
  if (tid == 0) s_bad = 0;
  const int64_t n_free = *a.n_free;
  int64_t all = 0;
  uint32_t bad = 0, unused = 0, m[BT_MANY] = {};
  int32_t length[BT_MANY] = {};
  for (int64_t c0 = 0; c0 < a.rows; c0 += BT_PART) {
    row_releases(a, c0, m, length, bad);
    all += (int64_t)m[0] + m[1] + m[2] + m[3];
  }
  if (n_free < 0 || n_free > a.free_cap) bad |= BAD_FREE;
  __syncthreads();
  if (bad) atomicOr(&s_bad, bad);
  all = capped(all);
  uint32_t v[2] = {low(all), high(all)}, sums[2];
  block_sums(v, sums, s_sums[1]);
  bad = s_bad;
  const int64_t total = joined(sums[0], sums[1]);
  if (!(bad & BAD_FREE) && n_free + total > a.free_cap) bad |= BAD_SIZE;
  if (fill && !bad) {
    const int64_t per = div_up(total, gridDim.x);
    const int64_t o0 = min((int64_t)blockIdx.x * per, total), o1 = min(o0 + per, total);
    int64_t carry = 0;
    int turn = 0;
    for (int64_t c0 = 0; c0 < a.rows && carry < o1; c0 += BT_PART, ++turn) {
      uint32_t chunk = (uint32_t)total, base;
      if (few) {
        base = (uint32_t)(joined(v[0], v[1]) - all);
      } else {
        row_releases(a, c0, m, length, unused);
        const uint32_t sum = m[0] + m[1] + m[2] + m[3];
        uint32_t s[1] = {sum}, all_of[1];
        block_sums(s, all_of, s_sums[turn & 1]);
        base = s[0] - sum;
        chunk = all_of[0];
      }
#pragma unroll
      for (int k = 0; k < BT_MANY; ++k) {
        s_base[BT_MANY * tid + k] = base;
        base += m[k];
      }
      __syncthreads();
      const uint32_t lo = (uint32_t)(max(o0, carry) - carry), hi = (uint32_t)min(o1 - carry, (int64_t)chunk);
      for (uint32_t t = lo; t < hi; t += BT_PART) {
        uint32_t at[BT_MANY];
        int i[BT_MANY];
        int32_t id[BT_MANY];
#pragma unroll
        for (int k = 0; k < BT_MANY; ++k) at[k] = min(t + k * BT_THREADS + tid, hi - 1);
        last_rows<BT_PART>(s_base, at, i);
#pragma unroll
        for (int k = 0; k < BT_MANY; ++k) id[k] = a.table[(c0 + i[k]) * a.table_stride + (at[k] - s_base[i[k]])];
#pragma unroll
        for (int k = 0; k < BT_MANY; ++k)
          if (t + k * BT_THREADS + tid < hi) a.free_blocks[n_free + carry + at[k]] = id[k];
      }
      carry += chunk;
      __syncthreads();
    }
  }
  if ((int)blockIdx.x != finisher) return;
  __syncthreads();  // out_lengths may be lengths, which every thread has read by now
  for (int64_t c0 = 0; c0 < a.rows; c0 += BT_PART) {
    if (!few) row_releases(a, c0, m, length, unused);
#pragma unroll
    for (int k = 0; k < BT_MANY; ++k) {
      const int64_t r = c0 + BT_MANY * tid + k;
      if (r < a.rows) a.out_lengths[r] = bad ? a.lengths[r] : length[k];
    }
  }
  if (tid == 0) {
    *a.out_n_free = (int32_t)(bad ? n_free : n_free + total);
    *a.out_n = bad ? fault_code(bad) : total;
  }
}

// ---------------------------------------------------------------- token sets

constexpr int TB_THREADS = 1024;
constexpr int TB_WORDS = 16384;  // words of a set that a workgroup holds in LDS
constexpr int TB_BATCH = 8192;   // ids that a workgroup has on their way at a time, eight for a thread
constexpr int64_t TB_SPLIT = 65536;  // ids from which on they may be dealt out in equal parts
constexpr int64_t TB_LONG = 12288;   // and ids of a text, on average

typedef uint32_t Ids4 __attribute__((ext_vector_type(4), aligned(4)));  // from any id on

// Ids of texts repeat: a bit that is there costs a read, which lanes share, and
// no atomic, which they would queue for.
__device__ inline void put_bit(uint32_t id, uint32_t v0, uint32_t v1, uint32_t* set) {
  if (id < v0 || id >= v1) return;
  uint32_t* w = &set[(id - v0) >> 5];
  if (!(*w >> (id & 31) & 1)) atomicOr(w, 1u << (id & 31));
}

// The ids [lo, hi) that are in [v0, v1), as bits of `set` from id v0 on.  The
// next ids are loaded before these are looked at; the last loads reach back,
// since a bit may be set twice.
__device__ inline void gather_bits(const int32_t* ids, int64_t lo, int64_t hi, uint32_t v0, uint32_t v1, uint32_t* set) {
  auto put = [&](uint32_t id) { put_bit(id, v0, v1, set); };
  if (hi - lo < 4) {
    if (lo + threadIdx.x < hi) put((uint32_t)ids[lo + threadIdx.x]);
    return;
  }
  auto load = [&](int64_t i) { return *reinterpret_cast<const Ids4*>(ids + min(i, hi - 4)); };
  Ids4 x = load(lo + 4 * threadIdx.x), y = load(lo + TB_BATCH / 2 + 4 * threadIdx.x);
  for (int64_t base = lo; base < hi; base += TB_BATCH) {
    const Ids4 a = x, b = y;
    if (base + TB_BATCH < hi) {
      x = load(base + TB_BATCH + 4 * threadIdx.x);
      y = load(base + TB_BATCH + TB_BATCH / 2 + 4 * threadIdx.x);
    }
    if (base + 4 * threadIdx.x < hi) {
#pragma unroll
      for (int k = 0; k < 4; ++k) put(a[k]);
    }
    if (base + TB_BATCH / 2 + 4 * threadIdx.x < hi) {
#pragma unroll
      for (int k = 0; k < 4; ++k) put(b[k]);
    }
  }
}

__device__ inline int64_t bound(const int64_t* offsets, int64_t r, int64_t n) {
  return min(max(offsets[r], (int64_t)0), n);
}

// The set of a text by one workgroup (or by several, each for a part of the
// vocabulary, where LDS does not hold all of it): no atomics on memory.  One
// text of 2,500 ids takes 2.7 us, a launch and two dependent reads.
__global__ __launch_bounds__(TB_THREADS) void k_token_bits(const int32_t* ids, int64_t n, const int64_t* offsets,
                                                           int64_t vocab, int32_t* bits, int64_t stride, int tiles,
                                                           bool add) {
  extern __shared__ uint32_t set[];
  const int64_t r = blockIdx.x / tiles, words = div_up(vocab, 32);
  const int64_t w0 = (int64_t)(blockIdx.x % tiles) * TB_WORDS;
  const int here = (int)min((int64_t)TB_WORDS, words - w0);
  const int64_t lo = offsets ? bound(offsets, r, n) : 0, hi = offsets ? bound(offsets, r + 1, n) : n;
  for (int i = threadIdx.x; i < here; i += TB_THREADS) set[i] = 0;
  __syncthreads();
  gather_bits(ids, lo, hi, (uint32_t)(w0 * 32), (uint32_t)min(vocab, (w0 + here) * 32), set);
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(bits) + r * stride + w0;
  for (int i = threadIdx.x; i < here; i += TB_THREADS) out[i] = add ? out[i] | set[i] : set[i];
}

// Many ids: they are dealt out in equal parts, whatever texts they belong to.
// A workgroup gathers what its part has of a text in LDS and joins it to the
// text's set, cleared before, by atomics (a joint of sets is the same in any
// order).  Where its part of a text is short, one wavefront sets the bits one by
// one.  Ids and bounds are loaded together, and the ids stay in registers for all
// texts of the part.  64 texts of two million ids (8 MB) take 11 us and the clearing
// 1 to 4: a part's loads, its LDS atomics and the atomics on memory follow each other, and
// there is one part for a CU.  Two words to an atomic on memory is no faster.
// `first`: the id that the launch's first part begins with.
__global__ __launch_bounds__(TB_THREADS) void k_token_bits_split(const int32_t* ids, int64_t n, const int64_t* offsets,
                                                                 int64_t rows, int64_t vocab, int32_t* bits,
                                                                 int64_t stride, int64_t first) {
  extern __shared__ uint32_t set[];
  // texts that reach into the part, of the 1,024 at hand, and their ids in it
  __shared__ int s_row[TB_THREADS];
  __shared__ int s_lo[TB_THREADS], s_hi[TB_THREADS];
  __shared__ int s_rows;
  const int tid = threadIdx.x, words = (int)div_up(vocab, 32);
  const int64_t t0 = first + (int64_t)blockIdx.x * TB_BATCH, t1 = min(t0 + TB_BATCH, n);
  const bool in_lds = words <= TB_WORDS;
  const int least = max(words / 4, WAVE);  // ids that are worth a set in LDS
  // n is more than a part: the last part's loads reach back
  const int64_t x_at = min(t0 + 4 * tid, n - 4), y_at = min(t0 + TB_BATCH / 2 + 4 * tid, n - 4);
  const Ids4 x = *reinterpret_cast<const Ids4*>(ids + x_at), y = *reinterpret_cast<const Ids4*>(ids + y_at);
  const int x_from = (int)(x_at - t0), y_from = (int)(y_at - t0);  // negative where they reach back
  if (in_lds)
    for (int i = tid; i < words; i += TB_THREADS) set[i] = 0;
  for (int64_t base = 0; base < rows; base += TB_THREADS) {
    if (tid == 0) s_rows = 0;
    __syncthreads();
    const int64_t mine = base + tid;
    if (mine < rows) {
      const int64_t lo = max(offsets ? bound(offsets, mine, n) : 0, t0);
      const int64_t hi = min(offsets ? bound(offsets, mine + 1, n) : n, t1);
      if (lo < hi) {
        const int j = atomicAdd(&s_rows, 1);
        s_row[j] = tid;
        s_lo[j] = (int)(lo - t0);
        s_hi[j] = (int)(hi - t0);
      }
    }
    __syncthreads();
    const int count = s_rows;
    for (int j = 0; j < count; ++j) {
      const int lo = s_lo[j], hi = s_hi[j];
      uint32_t* out = reinterpret_cast<uint32_t*>(bits) + (base + s_row[j]) * stride;
      if (!in_lds || hi - lo < least) {
        if (j % (TB_THREADS / WAVE) != tid / WAVE) continue;
        for (int i = lo + tid % WAVE; i < hi; i += WAVE) {
          const uint32_t id = (uint32_t)ids[t0 + i];
          if (id < (uint32_t)vocab) atomicOr(&out[id >> 5], 1u << (id & 31));
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (x_from + k >= lo && x_from + k < hi) put_bit(x[k], 0, (uint32_t)vocab, set);
        if (y_from + k >= lo && y_from + k < hi) put_bit(y[k], 0, (uint32_t)vocab, set);
      }
      __syncthreads();
      for (int i = tid; i < words; i += TB_THREADS)
        if (const uint32_t w = set[i]) {
          atomicOr(&out[i], w);
          set[i] = 0;
        }
      __syncthreads();
    }
    __syncthreads();
  }
}

__global__ void k_clear_bits(int32_t* bits, int64_t rows, int64_t words, int64_t stride) {
  const int64_t r = blockIdx.y, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t row = r; row < rows; row += gridDim.y)
    if (i < words) bits[row * stride + i] = 0;
}

// ------------------------------------------------------------------- grammars

constexpr int GR_THREADS = 256;

// The bytes of a token, kept inside the strings whatever its offsets say.
__device__ inline void token_span(const tt_grammar& g, int64_t v, int64_t& at, int& len) {
  const int64_t a = g.string_offsets[v], b = g.string_offsets[v + 1];
  at = min(max(a, (int64_t)0), g.n_bytes);
  len = (int)(min(max(b, at), g.n_bytes) - at);
}

// The sets of few states: a thread walks one token from one state, which ends at
// the first dead byte.  One state and 100,257 tokens take 3.0 us, a launch and
// some dependent reads from L2; 340 us for 1,024 states.
__global__ __launch_bounds__(GR_THREADS) void k_grammar_bits(tt_grammar g, const int32_t* states, int64_t vocab,
                                                             int32_t* bits, int64_t stride, int tiles) {
  __shared__ uint8_t cls[256];
  for (int i = threadIdx.x; i < 256; i += GR_THREADS) cls[i] = (uint8_t)min((int)g.classes[i], (int)g.n_classes - 1);
  __syncthreads();
  const int64_t r = blockIdx.x / tiles;
  const int64_t v = (int64_t)(blockIdx.x % tiles) * GR_THREADS + threadIdx.x;
  const int32_t q0 = states[r];
  const uint32_t n = (uint32_t)g.n_states, nc = (uint32_t)g.n_classes;
  bool ok = false;
  if (v < vocab) {
    if (q0 == TT_STATE_FREE) {
      ok = true;
    } else if ((uint32_t)q0 < n) {
      if (v == g.end_id) {
        ok = g.accept[q0] != 0;
      } else if (v < g.n_tokens) {
        int64_t at;
        int len;
        token_span(g, v, at, len);
        uint32_t q = (uint32_t)q0;
        for (int k = 0; k < len && q < n; ++k) q = (uint32_t)(int32_t)g.next[q * nc + cls[g.strings[at + k]]];
        ok = len > 0 && q < n;
      }
    }
  }
  const uint64_t m = __ballot(ok);
  const int lane = threadIdx.x % WAVE;
  const int64_t word = v / 32;
  if (lane % 32 == 0 && word < div_up(vocab, 32)) bits[r * stride + word] = (int32_t)(uint32_t)(m >> lane);
}

// The sets of many states at a time.  A workgroup takes 2,048 tokens, puts them
// in order of the classes of their first two bytes, and keeps the byte classes of
// two tokens in each thread's registers, so that the 64 tokens of a wavefront mostly
// begin alike.  Then, 64 states at a time, a lane looks for each state at what the
// tokens begin with: in most states of a grammar few bytes are possible, and those
// that none of the 64 tokens begins with are done.  So are the states from which all
// further bytes of all 64 lead back to it (the inside of a text), by two sets of classes.
// What is left is walked, each lane from its own next state.
//
// 1,024 states and 100,257 tokens take 51-55 us (k_grammar_bits 340).  About 10 us are the
// loading and ordering of the tokens; then wavefronts with many walks (runs of
// spaces, mixed beginnings), each a chain of reads of LDS, keep the others of
// their workgroup waiting, which is what bounds it.  Walking two or four states together
// in a lane is slower (63 and 69 us where one took 58), and so is skipping bytes that lead
// back to a state by their classes (84 us where stepping takes 51).
constexpr int GM_THREADS = 1024;
constexpr int GM_CHUNKS = 2;                       // tokens of a thread
constexpr int GM_TOKENS = GM_THREADS * GM_CHUNKS;  // of a workgroup
constexpr int GM_WORDS = GM_TOKENS / 32;
constexpr int GM_KEYS = 512;                       // by which a workgroup's tokens are ordered
constexpr int GM_KEEP = 16;                        // bytes of a token that are kept as classes
constexpr int64_t GM_LDS = 156 * 1024;              // at most, beside 2.3 KB that are always there

typedef uint32_t Bytes16 __attribute__((ext_vector_type(4)));
typedef uint32_t Bytes16Any __attribute__((ext_vector_type(4), aligned(1)));  // at any address

// A token as its thread keeps it.
struct KeptToken {
  uint32_t c[GM_KEEP / 4];  // classes of its first bytes
  uint64_t later;           // set of the classes of all bytes but the first, if there are at most 64 classes
  int at, len;              // its bytes; len 0: none or not to be walked
  int place;                // in the workgroup's tokens
};

// Classes that lead from a state to itself, and to any state.
struct StateSets {
  uint64_t self, live;
};

__device__ inline uint64_t wave_or(uint64_t v) {
  for (int d = WAVE / 2; d > 0; d >>= 1) v |= __shfl_xor((unsigned long long)v, d);
  return v;
}

// The state after the bytes K .. GM_KEEP - 1 of each lane's token.
template <int K>
__device__ inline uint32_t walk(const int16_t* next, uint32_t n, uint32_t nc, const KeptToken& t, uint32_t s, bool go) {
  if constexpr (K < GM_KEEP) {
    const bool on = go && K < t.len && s < n;
    if (!__any(on)) return s;
    if (on) s = (uint32_t)(int32_t)next[s * nc + (t.c[K / 4] >> (8 * (K % 4)) & 255)];
    return walk<K + 1>(next, n, nc, t, s, go);
  }
  return s;
}

template <bool IN_LDS>
__global__ __launch_bounds__(GM_THREADS) void k_grammar_many(tt_grammar g, const int32_t* states, int64_t rows,
                                                             int64_t vocab, int32_t* bits, int64_t stride, int tiles,
                                                             int64_t per_block, int batch, bool sets) {
  // [batch][GM_WORDS] the sets at hand (first, the tokens' order); [n] the states' sets, if `sets`; the automaton
  extern __shared__ __attribute__((aligned(16))) uint32_t s_bits[];
  __shared__ uint8_t cls[256];
  __shared__ uint32_t s_first[GM_KEYS + 1];  // tokens by their first class and three bits of the second
  const int tid = threadIdx.x, lane = tid % WAVE;
  const uint32_t n = (uint32_t)g.n_states, nc = (uint32_t)g.n_classes;
  StateSets* s_sets = reinterpret_cast<StateSets*>(s_bits + batch * GM_WORDS);
  int16_t* s_next = reinterpret_cast<int16_t*>(s_sets + (sets ? n : 0));
  const int16_t* next = IN_LDS ? s_next : g.next;
  // the tokens in order; those that are not walked are left out
  const int64_t v0 = (int64_t)(blockIdx.x % tiles) * GM_TOKENS;
  uint16_t* order = reinterpret_cast<uint16_t*>(s_bits);
  int first[GM_CHUNKS], then[GM_CHUNKS], nth[GM_CHUNKS];
#pragma unroll
  for (int j = 0; j < GM_CHUNKS; ++j) {
    const int64_t v = v0 + j * GM_THREADS + tid;
    int64_t at = 0;
    int len = 0;
    if (v < g.n_tokens && v < vocab && v != g.end_id) token_span(g, v, at, len);
    first[j] = len > 0 ? g.strings[at] : -1;
    then[j] = len > 1 ? g.strings[at + 1] : -1;
  }
  for (int i = tid; i < 256; i += GM_THREADS) cls[i] = (uint8_t)min((int)g.classes[i], (int)nc - 1);
  if (tid <= GM_KEYS) s_first[tid] = 0;
  if (IN_LDS) {
    const uint32_t whole = n * nc / 8;
#pragma unroll 4
    for (uint32_t i = tid; i < whole; i += GM_THREADS)
      reinterpret_cast<Bytes16*>(s_next)[i] = reinterpret_cast<const Bytes16Any*>(g.next)[i];
    for (uint32_t i = 8 * whole + tid; i < n * nc; i += GM_THREADS) s_next[i] = g.next[i];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < GM_CHUNKS; ++j)
    if (first[j] >= 0) {
      first[j] = sets ? cls[first[j]] * 8 + (then[j] >= 0 ? cls[then[j]] & 7 : 0) : cls[first[j]];
      nth[j] = (int)atomicAdd(&s_first[first[j] + 1], 1u);
    }
  if (sets)
    for (uint32_t q = tid; q < n; q += GM_THREADS) {
      StateSets m{0, 0};
      for (uint32_t k = 0; k < nc; ++k) {
        const uint32_t to = (uint32_t)(int32_t)next[q * nc + k];
        m.self |= (uint64_t)(to == q) << k;
        m.live |= (uint64_t)(to < n) << k;
      }
      s_sets[q] = m;
    }
  __syncthreads();
  if (tid < WAVE) {  // inclusive sums of the counts by one wavefront, eight to a lane
    constexpr int EACH = GM_KEYS / WAVE;
    uint32_t c[EACH], sum = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) c[k] = sum += s_first[1 + EACH * lane + k];
    const uint32_t before = wave_sums(sum) - sum;
#pragma unroll
    for (int k = 0; k < EACH; ++k) s_first[1 + EACH * lane + k] = before + c[k];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < GM_CHUNKS; ++j)
    if (first[j] >= 0) order[s_first[first[j]] + nth[j]] = (uint16_t)(j * GM_THREADS + tid);
  __syncthreads();
  const int walked = (int)s_first[GM_KEYS];
  KeptToken t[GM_CHUNKS];
  bool alike[GM_CHUNKS], single[GM_CHUNKS];
  int lead[GM_CHUNKS];
  uint64_t second[GM_CHUNKS], later[GM_CHUNKS];
#pragma unroll
  for (int j = 0; j < GM_CHUNKS; ++j) {
    // a wavefront's chunks are 16 apart, so that the long runs of one class are shared out
    const int i = (j * (GM_THREADS / WAVE) + tid / WAVE) * WAVE + lane;
    t[j] = KeptToken{};
    if (i < walked) {
      t[j].place = order[i];
      int64_t at;
      token_span(g, v0 + t[j].place, at, t[j].len);
      t[j].at = (int)at;
    }
    Bytes16 b = 0;
    if (t[j].len > 0) {
      if ((int64_t)t[j].at + GM_KEEP <= g.n_bytes) {  // strings may be 2^31 - 1 bytes long
        b = *reinterpret_cast<const Bytes16Any*>(g.strings + t[j].at);
      } else {  // at the end of the strings
        for (int k = 0; k < min(t[j].len, GM_KEEP); ++k) b[k / 4] |= (uint32_t)g.strings[t[j].at + k] << (8 * (k % 4));
      }
    }
#pragma unroll
    for (int k = 0; k < GM_KEEP; ++k) {
      if (!__any(k < t[j].len)) continue;
      const uint32_t c = cls[b[k / 4] >> (8 * (k % 4)) & 255];
      t[j].c[k / 4] |= c << (8 * (k % 4));
      if (k && k < t[j].len) t[j].later |= 1ull << (c & 63);
    }
    for (int k = GM_KEEP; k < t[j].len; ++k) t[j].later |= 1ull << (cls[g.strings[t[j].at + k]] & 63);
    // what the 64 tokens have in common: their first class, if it is one, and the sets of their other ones
    const uint64_t some = __ballot(t[j].len > 0);
    lead[j] = some ? __builtin_ctzll(some) : 0;
    const uint32_t c0 = (uint32_t)__builtin_amdgcn_readlane((int)(t[j].c[0] & 255), lead[j]);
    alike[j] = sets && some && __ballot(t[j].len > 0 && (t[j].c[0] & 255) != c0) == 0;
    single[j] = __any(t[j].len == 1);
    second[j] = wave_or(t[j].len > 1 ? 1ull << (t[j].c[0] >> 8 & 63) : 0);
    later[j] = wave_or(t[j].later);
  }

  const int64_t r0 = blockIdx.x / tiles * per_block, r1 = min(r0 + per_block, rows);
  const int64_t word0 = v0 / 32, words = min(div_up(vocab, 32) - word0, (int64_t)GM_WORDS);
  const int end = g.end_id >= v0 && g.end_id < min(v0 + GM_TOKENS, vocab) ? (int)(g.end_id - v0) : -1;
  for (int64_t r = r0; r < r1; r += batch) {
    const int batch_rows = (int)min((int64_t)batch, r1 - r);
    __syncthreads();  // the order is read, or the sets before are written
    for (int i = tid; i < batch_rows * GM_WORDS; i += GM_THREADS) s_bits[i] = 0;
    __syncthreads();
    for (int r64 = 0; r64 < batch_rows; r64 += WAVE) {
      const int count = min(WAVE, batch_rows - r64);
      uint32_t* sets_of = s_bits + r64 * GM_WORDS;
      const int32_t q_lane = lane < count ? states[r + r64 + lane] : TT_STATE_DEAD;
      const bool good = (uint32_t)q_lane < n;
      const uint64_t possible = sets && good ? s_sets[q_lane].live : 0;
      uint64_t free = __ballot(q_lane == TT_STATE_FREE);
      for (; free && tid < WAVE; free &= free - 1) {
        static_assert(GM_WORDS == WAVE, "a lane for each word");
        const int64_t rest = vocab - (word0 + lane) * 32;
        sets_of[__builtin_ctzll(free) * GM_WORDS + lane] = rest >= 32 ? 0xFFFFFFFFu : rest > 0 ? (1u << rest) - 1u : 0u;
      }
      if (end >= 0 && tid < count && good && g.accept[q_lane])
        atomicOr(&sets_of[tid * GM_WORDS + (end >> 5)], 1u << (end & 31));
#pragma unroll
      for (int j = 0; j < GM_CHUNKS; ++j) {
        // the states that each token's first byte leaves alive
        uint64_t mine = 0, all = 0;
        if (alike[j]) {
          // of them, those that all tokens stay in, and those that some token's second byte leaves alive
          const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)(t[j].c[0] & 255), lead[j]);
          const uint32_t q = good ? (uint32_t)(int32_t)next[(uint32_t)q_lane * nc + c] : n;
          const StateSets m = s_sets[q < n ? q : 0];
          const bool whole = q < n && (later[j] & ~m.self) == 0;
          all = __ballot(whole);
          const uint64_t some = __ballot(q < n && !whole && (single[j] || (m.live & second[j])));
          if (t[j].len > 0) mine = some;
        } else {
          for (uint64_t left = __ballot(t[j].len > 0); left;) {
            const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)(t[j].c[0] & 255), __builtin_ctzll(left));
            const bool same = t[j].len > 0 && (t[j].c[0] & 255) == c;
            bool live = possible >> (c & 63) & 1;
            if (!sets) live = good && (uint32_t)(int32_t)next[(uint32_t)q_lane * nc + c] < n;
            const uint64_t states_of = __ballot(live);
            if (same) mine = states_of;
            left &= ~__ballot(same);
          }
        }
        const int word = t[j].place >> 5;
        const uint32_t bit = 1u << (t[j].place & 31);
        for (; all; all &= all - 1)
          if (t[j].len > 0) atomicOr(&sets_of[__builtin_ctzll(all) * GM_WORDS + word], bit);
        while (__any(mine != 0)) {  // each lane walks from its own next state
          const bool on = mine != 0;
          const int i = on ? __builtin_ctzll(mine) : 0;
          mine &= mine - 1;
          const uint32_t q0 = (uint32_t)__shfl(q_lane, i);
          uint32_t q = n;
          if (on) q = (uint32_t)(int32_t)next[q0 * nc + (t[j].c[0] & 255)];
          bool go = q < n && t[j].len > 1;
          if (sets && go && (t[j].later & ~s_sets[q].self) == 0) go = false;  // every further byte stays in it
          q = walk<1>(next, n, nc, t[j], q, go);
          for (int k = GM_KEEP; go && k < t[j].len && q < n; ++k)
            q = (uint32_t)(int32_t)next[q * nc + cls[g.strings[t[j].at + k]]];
          if (q < n) atomicOr(&sets_of[i * GM_WORDS + word], bit);
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < batch_rows * GM_WORDS; i += GM_THREADS) {
      const int row = i / GM_WORDS, w = i % GM_WORDS;
      if (w < words) bits[(r + row) * stride + word0 + w] = (int32_t)s_bits[i];
    }
  }
}

// A thread walks one token.  Two dependent reads from L2 a byte, its class and the next state: 256 tokens of one byte take
// 3.8 us a call, which is the launch, 256 of 37 bytes 9.2 us.
__global__ void k_grammar_advance(tt_grammar g, const int32_t* states, const int32_t* tokens, int64_t rows,
                                  int32_t* out) {
  const int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  const int32_t q0 = states[r], t = tokens[r];
  const uint32_t n = (uint32_t)g.n_states, nc = (uint32_t)g.n_classes;
  int32_t q = q0;
  if (t >= 0 && q0 != TT_STATE_FREE) {
    q = TT_STATE_DEAD;
    if ((uint32_t)q0 < n && t != g.end_id && t < g.n_tokens) {
      int64_t at;
      int len;
      token_span(g, t, at, len);
      uint32_t s = len > 0 ? (uint32_t)q0 : n;
      for (int k = 0; k < len && s < n; ++k)
        s = (uint32_t)(int32_t)g.next[s * nc + min((uint32_t)g.classes[g.strings[at + k]], nc - 1)];
      if (s < n) q = (int32_t)s;
    }
  }
  out[r] = q;
}

// --------------------------------------------------------------------- logits

constexpr int SH_VEC = 8;    // tokens of a load: one byte of a token set
constexpr int SH_BATCH = 8;  // generated tokens that a thread has on their way at a time

// A vector that may start at any element.
template <class T>
struct Pack {
  typedef T type __attribute__((ext_vector_type(SH_VEC), aligned(sizeof(T))));
};

// Bit k of bits ? a : b, in two instructions (written as a select it becomes four).
__device__ inline float pick(uint32_t bits, int k, float a, float b) {
  const int m = __builtin_amdgcn_sbfe((int)bits, k, 1);
  float d;
  asm("v_bfi_b32 %0, %1, %2, %3" : "=v"(d) : "v"(m), "v"(a), "v"(b));
  return d;
}

// Whether quotients by d may go by its reciprocal.
__device__ inline bool has_reciprocal(float d) { return fabsf(d) >= 0x1p-20f && fabsf(d) <= 0x1p100f; }

// Quotients of eight values, as exact as divisions: the product with the reciprocal, put right by its remainder's share, where that
// is exact (a multiple of 2^-47 of the value) and no finite value has an infinite product.  Values outside the bounds, a
// zero among them, whose sign would be lost, are divided; infinities, which have no remainder, are only passed over.
__device__ inline void quotients(const float (&x)[SH_VEC], float d, float reciprocal, bool by_reciprocal, float (&y)[SH_VEC]) {
  constexpr float LEAST = 0x1p-100f, MOST = 0x1p100f;
  float lo = fabsf(x[0]), hi = lo;
#pragma unroll
  for (int k = 1; k < SH_VEC; ++k) {
    lo = fminf(lo, fabsf(x[k]));
    hi = fmaxf(hi, fabsf(x[k]));
  }
  if (by_reciprocal && lo >= LEAST && hi <= MOST) {
#pragma unroll
    for (int k = 0; k < SH_VEC; ++k) {
      const float q = x[k] * reciprocal;
      y[k] = fmaf(fmaf(-q, d, x[k]), reciprocal, q);
    }
    return;
  }
  hi = 0.0f;
#pragma unroll
  for (int k = 0; k < SH_VEC; ++k) hi = fmaxf(hi, fabsf(fmaf(x[k], 0.0f, x[k])));  // NaN, which max passes over, for an infinity
  if (by_reciprocal && lo >= LEAST && hi <= MOST) {
#pragma unroll
    for (int k = 0; k < SH_VEC; ++k) {
      const float q = x[k] * reciprocal, fixed = fmaf(fmaf(-q, d, x[k]), reciprocal, q);
      y[k] = fabsf(q) < __builtin_inff() ? fixed : q;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < SH_VEC; ++k) y[k] = x[k] / d;
}

// Element i of a row, by a 32-bit offset (rows are shorter than 2^32 bytes).
template <class T>
__device__ inline T* from(T* row, uint32_t i) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(row) + (uint32_t)(i * sizeof(T)));
}

// A workgroup shapes one tile of a row: N * SH_VEC tokens a thread.  The
// tile's logits and set bytes are loaded first; while they arrive the
// generated tokens that fall into the tile are counted in LDS, each workgroup
// of a row reading the whole (short) list.  A tile that a bias entry names then
// uses the same words again to find each token's last entry; the others skip that.
// A tile has a workgroup of its own: its stores need not be waited for, as those
// of a loop over tiles have to be (116 us instead of 97 for the bare copy).
// 256 x 262,144 float32 take 99 us, 5.6 TB/s of what has to be read and written
// (a library copy of the logits alone 100 us): bound by memory.  16-bit logits come
// near the vector instructions, 25 for a token: 256 x 262,144 bfloat16 to float32 84 us,
// 4.9 TB/s, to bfloat16 59 us, 4.8 TB/s.  61 x 100,257 float16 take 12 us, where all tiles are resident at
// once and the list, the biases and the barriers between them add 4 us to the copy's 8.
template <class I, class O, int T, int N>
__global__ __launch_bounds__(T, 6) void k_shape(tt_shape_args a, int tiles, int64_t first_row) {
  constexpr int TOKENS = T * SH_VEC * N;  // of a tile
  __shared__ __attribute__((aligned(16))) uint32_t s_word[TOKENS];
  __shared__ int s_hit[2];  // some entry names a token of the tile; some generated token is in it
  const int64_t r = first_row + blockIdx.x / tiles;
  const int tid = threadIdx.x;
  const uint32_t vocab = (uint32_t)a.vocab, v0 = blockIdx.x % tiles * (uint32_t)TOKENS;
  const uint32_t here = min((uint32_t)TOKENS, vocab - v0);

  // Vectors that would leave the row are loaded from its end and put right
  // where they are used.  Without a set, bytes of the row itself are loaded in
  // its place, which costs less than a branch.
  typedef typename Pack<I>::type Vec;
  const I* row = static_cast<const I*>(a.logits) + r * a.logits_stride;
  const uint8_t* seen = a.seen ? reinterpret_cast<const uint8_t*>(a.seen + r * a.seen_stride)
                               : reinterpret_cast<const uint8_t*>(row);
  Vec x[N];
  uint32_t sb[N], ab[N], byte[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t v = v0 + (uint32_t)(j * T + tid) * SH_VEC;
    byte[j] = min(v, vocab - 1) >> 3;
    x[j] = 0;
    if (vocab >= SH_VEC) x[j] = *reinterpret_cast<const Vec*>(from(row, min(v, vocab - SH_VEC)));
    sb[j] = seen[byte[j]];
  }
  // the row's parameters: all loads before the first use, so that they wait once
  const int64_t entry_at = a.bias_offsets ? a.bias_offsets[r] : 0, entry_to = a.bias_offsets ? a.bias_offsets[r + 1] : 0;
  const int n_gen_at = a.n_generated ? a.n_generated[r] : 0x7FFFFFFF;
  const int set = a.allowed_rows ? a.allowed_rows[r] : (int)r;
  const float rho = a.repetition ? a.repetition[r] : 1.0f;
  const float phi = a.frequency ? a.frequency[r] : 0.0f;
  const float pi = a.presence ? a.presence[r] : 0.0f;
  const float temp = a.temperature ? a.temperature[r] : 0.0f;
  const int n_gen = a.generated ? min(max(n_gen_at, 0), (int)a.generated_cap) : 0;
  const int64_t b0 = min(max(entry_at, (int64_t)0), a.n_bias);
  const int n_bias = (int)(min(max(entry_to, b0), a.n_bias) - b0);
  const bool masked = a.allowed && set != TT_STATE_FREE;
  const bool none = masked && (set < 0 || set >= a.allowed_count);  // nothing is allowed
  const uint8_t* allowed = masked && !none ? reinterpret_cast<const uint8_t*>(a.allowed + set * a.allowed_stride)
                                           : reinterpret_cast<const uint8_t*>(row);
#pragma unroll
  for (int j = 0; j < N; ++j) ab[j] = allowed[byte[j]];

  // the first generated tokens and entries, on their way with the logits
  const int32_t* gen = a.generated + r * a.generated_stride;
  uint32_t ids[SH_BATCH], first = 0;
  auto take = [&](int base) {
#pragma unroll
    for (int k = 0; k < SH_BATCH; ++k)
      if (base + k * T < n_gen) ids[k] = (uint32_t)gen[min(base + k * T + tid, n_gen - 1)];
  };
  if (n_gen > 0) take(0);
  if (n_bias > 0) first = (uint32_t)a.bias_ids[b0 + min(tid, n_bias - 1)];
#pragma unroll
  for (int j = 0; j < 2 * N; ++j) reinterpret_cast<uint4*>(s_word)[j * T + tid] = make_uint4(0, 0, 0, 0);
  if (tid < 2) s_hit[tid] = 0;
  __syncthreads();

  for (int base = 0; base < n_gen; base += SH_BATCH * T) {
    if (base) take(base);
#pragma unroll
    for (int k = 0; k < SH_BATCH; ++k)
      if (base + k * T < n_gen && base + k * T + tid < n_gen && ids[k] - v0 < here) {
        atomicAdd(&s_word[ids[k] - v0], 1u);
        s_hit[1] = 1;
      }
  }
  for (int i = tid; i < n_bias; i += T) {
    const uint32_t t = (i < T ? first : (uint32_t)a.bias_ids[b0 + i]) - v0;
    if (t < here) s_hit[0] = 1;
  }
  __syncthreads();
  const bool biased = s_hit[0] != 0, counted = s_hit[1] != 0;
  uint32_t n[N][SH_VEC];
  float add[N][SH_VEC];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (counted) {
      const uint4* w = reinterpret_cast<const uint4*>(s_word) + 2 * (j * T + tid);
      lo = w[0];
      hi = w[1];
    }
    n[j][0] = lo.x, n[j][1] = lo.y, n[j][2] = lo.z, n[j][3] = lo.w, n[j][4] = hi.x, n[j][5] = hi.y, n[j][6] = hi.z, n[j][7] = hi.w;
#pragma unroll
    for (int k = 0; k < SH_VEC; ++k) add[j][k] = 0.0f;
  }
  if (biased) {  // the words again, now for the last entry that names each token
#pragma unroll
    for (int j = 0; j < N; ++j) {  // each thread the ones that it has read: others may not have theirs yet
      uint4* w = reinterpret_cast<uint4*>(s_word) + 2 * (j * T + tid);
      w[0] = w[1] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int i = tid; i < n_bias; i += T) {
      const uint32_t t = (i < T ? first : (uint32_t)a.bias_ids[b0 + i]) - v0;
      if (t < here) atomicMax(&s_word[t], (uint32_t)i + 1u);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) {
        const uint32_t w = s_word[(j * T + tid) * SH_VEC + k];
        if (w) add[j][k] = a.bias_values[b0 + w - 1];
      }
  }

  // Quotients by rho and by the temperature go by the reciprocal.  Where the result stays in 32 bits they are put right by the
  // remainder, and vectors with a value that this does not serve are divided; where it has 16 they are mere products, each off
  // by up to 2^-23 of the value at hand (a division 2^-24), before the one rounding to 16.
  const float inv_rho = 1.0f / rho, inv_temp = 1.0f / temp;
  const bool plain_rho = !has_reciprocal(rho), plain_temp = temp > 0.0f && !has_reciprocal(temp);
  const float scale = temp > 0.0f && !plain_temp ? inv_temp : 1.0f;
  const float lowest = -__builtin_inff();
  O* dst = static_cast<O*>(a.out) + r * a.out_stride + v0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t i = (uint32_t)(j * T + tid) * SH_VEC;
    if (here < TOKENS && i + SH_VEC > here) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k)
        if (i + k < here) x[j][k] = *from(row, v0 + i + k);
    }
    uint32_t was = a.seen ? sb[j] : 0u;
    const uint32_t may = none ? 0u : masked ? ab[j] : 255u;
    float f[SH_VEC];
#pragma unroll
    for (int k = 0; k < SH_VEC; ++k) f[k] = (float)x[j][k];
    const uint32_t* c = n[j];
    const bool some = (c[0] | c[1] | c[2] | c[3] | c[4] | c[5] | c[6] | c[7]) != 0;
    if (some) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) was |= (c[k] != 0) << k;
    }
    if (sizeof(O) == 4 && was) {
      float y[SH_VEC];
      quotients(f, rho, inv_rho, !plain_rho, y);
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] = pick(was, k, f[k] > 0.0f ? y[k] : f[k] * rho, f[k]);
    }
    if (sizeof(O) == 2 && was && !plain_rho) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] = pick(was, k, f[k] * (f[k] > 0.0f ? inv_rho : rho), f[k]);
    }
    if (sizeof(O) == 2 && was && plain_rho) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] = pick(was, k, f[k] > 0.0f ? f[k] / rho : f[k] * rho, f[k]);
    }
    if (some) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k)
        if (c[k]) f[k] = f[k] - phi * (float)c[k] - pi;
    }
    if (biased) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] += add[j][k];
    }
    if (sizeof(O) == 4 && temp > 0.0f) {
      float y[SH_VEC];
      quotients(f, temp, inv_temp, !plain_temp, y);
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] = y[k];
    }
    if (sizeof(O) == 2 && plain_temp) {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k) f[k] /= temp;
    }
    typename Pack<O>::type y;
#pragma unroll
    for (int k = 0; k < SH_VEC; ++k) y[k] = (O)pick(may, k, sizeof(O) == 4 ? f[k] : f[k] * scale, lowest);
    if (i + SH_VEC <= here) {
      *reinterpret_cast<typename Pack<O>::type*>(from(dst, i)) = y;
    } else {
#pragma unroll
      for (int k = 0; k < SH_VEC; ++k)
        if (i + k < here) *from(dst, i + k) = y[k];
    }
  }
}

template <class I, class O, int T, int N>
void enqueue_tiles(const tt_shape_args& a, hipStream_t st) {
  const int64_t tiles = div_up(a.vocab, T * SH_VEC * N);
  const int64_t most = MAX_ITEMS / T / tiles;  // rows of a launch
  for (int64_t r = 0; r < a.rows; r += most)
    hipLaunchKernelGGL((k_shape<I, O, T, N>), dim3((uint32_t)(std::min(most, a.rows - r) * tiles)), dim3(T), 0, st, a,
                       (int)tiles, r);
}

// Tiles of 4,096 tokens once they fill the card, since every tile reads the
// list of generated tokens: 250 rows of 260,003 bfloat16 with lists of up to
// 16,000 take 85 us, with tiles of 2,048 110 us.  Fewer go by 2,048, which
// spreads a row over twice the CUs: one row of 50,256 takes 4.4 us.
template <class I, class O>
void enqueue_shape(const tt_shape_args& a, hipStream_t st) {
  if (a.rows * div_up(a.vocab, 4096) >= 1024) enqueue_tiles<I, O, 256, 2>(a, st);
  else enqueue_tiles<I, O, 256, 1>(a, st);
}

}  // namespace

// In the launchers min and max are std's: HIP's own take ints on the host.

// What is written where it was read has to wait until every workgroup has
// read it: it gets a launch of its own.  Otherwise one more workgroup, without
// places, writes lengths and counts beside the others.
hipError_t launch_plan(const tt_plan_args& a, hipStream_t st) {
  const int64_t per = div_up(div_up(a.places, 1024), BT_PART) * BT_PART;  // at most 1,024 parts: each sums up all rows
  const int parts = a.places > 0 ? (int)div_up(a.places, per) : 1;
  auto* k = a.offsets ? k_plan<false> : k_plan<true>;
  if (parts == 1) {
    hipLaunchKernelGGL(k, dim3(1), dim3(BT_THREADS), 0, st, a, per, 0);
  } else if (a.out_lengths != a.lengths && a.out_n_free != a.n_free) {
    hipLaunchKernelGGL(k, dim3((uint32_t)parts + 1), dim3(BT_THREADS), 0, st, a, per, parts);
  } else {
    hipLaunchKernelGGL(k, dim3((uint32_t)parts), dim3(BT_THREADS), 0, st, a, per, -1);
    hipLaunchKernelGGL(k, dim3(1), dim3(BT_THREADS), 0, st, a, (int64_t)0, 0);
  }
  return hipGetLastError();
}

hipError_t launch_release(const ReleaseArgs& a, hipStream_t st) {
  // the blocks that come back are counted on the device: a part for every 8,192 entries of the table, at most 512
  int64_t parts = a.rows * a.width / 8192 + 1;
  if (parts > 512) parts = 512;
  if (parts == 1) {
    hipLaunchKernelGGL(k_release, dim3(1), dim3(BT_THREADS), 0, st, a, true, 0);
  } else if (a.out_lengths != a.lengths && a.out_n_free != a.n_free) {
    hipLaunchKernelGGL(k_release, dim3((uint32_t)parts), dim3(BT_THREADS), 0, st, a, true, (int)parts - 1);
  } else {
    hipLaunchKernelGGL(k_release, dim3((uint32_t)parts), dim3(BT_THREADS), 0, st, a, true, -1);
    hipLaunchKernelGGL(k_release, dim3(1), dim3(BT_THREADS), 0, st, a, false, 0);
  }
  return hipGetLastError();
}

hipError_t launch_token_bits(const int32_t* ids, int64_t n, const int64_t* offsets, int64_t rows, int64_t vocab,
                             int32_t* bits, int64_t stride, bool add, hipStream_t st) {
  const int64_t words = div_up(vocab, 32), tiles = div_up(words, TB_WORDS);
  const size_t lds = (size_t)(words < TB_WORDS ? words : TB_WORDS) * 4;
  // One workgroup for a text while texts are short or many: 30 texts of 200,000 ids in all take 7.7 us (dealt out
  // 11 us), 250 texts of two million 8.5 us (12 us).  Fewer and longer ones are dealt out: 64 texts of two
  // million ids take 12.6 us (one workgroup each 21 us), one text of two million 12 us (216 us).
  if (n < TB_SPLIT || n < TB_LONG * rows) {
    const int64_t most = MAX_ITEMS / TB_THREADS / tiles;  // texts of a launch
    for (int64_t r = 0; r < rows; r += most)
      hipLaunchKernelGGL(k_token_bits, dim3((uint32_t)(std::min(most, rows - r) * tiles)), dim3(TB_THREADS), lds, st, ids, n,
                         offsets ? offsets + r : nullptr, vocab, bits + r * stride, stride, (int)tiles, add);
    return hipGetLastError();
  }
  if (!add)
    hipLaunchKernelGGL(k_clear_bits, dim3((uint32_t)div_up(words, 256), (uint32_t)std::min(rows, (int64_t)32768)), dim3(256),
                       0, st, bits, rows, words, stride);
  const int64_t most = MAX_ITEMS / TB_THREADS * TB_BATCH;  // ids of a launch
  for (int64_t t = 0; t < n; t += most)
    hipLaunchKernelGGL(k_token_bits_split, dim3((uint32_t)div_up(std::min(most, n - t), TB_BATCH)), dim3(TB_THREADS), lds, st, ids,
                       n, offsets, rows, vocab, bits, stride, t);
  return hipGetLastError();
}

hipError_t launch_grammar_bits(const tt_grammar& g, const int32_t* states, int64_t rows, int32_t* bits,
                               int64_t stride, int64_t vocab, hipStream_t st) {
  // The sets of many states have LDS hold the classes' sets of all states, where there are at most 64 classes and 8,960 states, and
  // the automaton where it fits beside them, which is read from L2 otherwise.  With the classes' sets 64 rows are no slower
  // than by k_grammar_bits; without them a wavefront's tokens are tried one class at a time, which pays from about 128 rows
  // on: 10,000 states of 35 classes take 36 us for 64 rows (k_grammar_bits 27), 37 us for 300 (100) and 0.81 ms for all
  // (3.2); 2,000 states of 151 classes 101 us for 128 rows (77) and 0.58 ms for all (1.2).
  const int64_t least = WAVE * GM_WORDS * 4, table = 2 * g.n_states * g.n_classes;
  const bool sets = g.n_classes <= 64 && 16 * g.n_states + least <= GM_LDS;
  if (rows >= (sets ? WAVE : 2 * WAVE)) {
    // a workgroup for every CU, each with 64 states at least; as many sets at a time as LDS holds beside the rest
    const int64_t tiles = div_up(vocab, GM_TOKENS);
    const int64_t parts = std::min(div_up(rows, WAVE), std::max((int64_t)1, (int64_t)256 / tiles)), per = div_up(rows, parts);
    const int64_t self = sets ? 16 * g.n_states : 0;
    const bool in_lds = table + self + least <= GM_LDS;
    const int64_t fixed = self + (in_lds ? table : 0), room = (GM_LDS - fixed) / least * WAVE;
    const int64_t batch = std::min(room, div_up(per, WAVE) * WAVE);
    auto* k = in_lds ? k_grammar_many<true> : k_grammar_many<false>;
    hipLaunchKernelGGL(k, dim3((uint32_t)(tiles * div_up(rows, per))), dim3(GM_THREADS),
                       (size_t)(fixed + batch * GM_WORDS * 4), st, g, states, rows, vocab, bits, stride, (int)tiles, per,
                       (int)batch, sets);
    return hipGetLastError();
  }
  const int64_t tiles = div_up(vocab, GR_THREADS);
  hipLaunchKernelGGL(k_grammar_bits, dim3((uint32_t)(rows * tiles)), dim3(GR_THREADS), 0, st, g, states, vocab, bits,
                     stride, (int)tiles);
  return hipGetLastError();
}

hipError_t launch_grammar_advance(const tt_grammar& g, const int32_t* states, const int32_t* tokens, int64_t rows,
                                  int32_t* out, hipStream_t st) {
  hipLaunchKernelGGL(k_grammar_advance, dim3((uint32_t)div_up(rows, 64)), dim3(64), 0, st, g, states, tokens, rows,
                     out);
  return hipGetLastError();
}

hipError_t launch_shape(const tt_shape_args& a, hipStream_t st) {
  const bool wide = a.out_type == TT_F32;
  if (a.in_type == TT_F32) enqueue_shape<float, float>(a, st);
  else if (a.in_type == TT_F16 && wide) enqueue_shape<_Float16, float>(a, st);
  else if (a.in_type == TT_F16) enqueue_shape<_Float16, _Float16>(a, st);
  else if (wide) enqueue_shape<__bf16, float>(a, st);
  else enqueue_shape<__bf16, __bf16>(a, st);
  return hipGetLastError();
}

}  // namespace tt

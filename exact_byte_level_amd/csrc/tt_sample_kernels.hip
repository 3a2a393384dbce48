// tt_sample_kernels.hip -- the choice of the next token (declared in include/tt_step.h).
#include "tt_lanes.h"
#include "tt_step_kernels.h"

#include <algorithm>
#include <type_traits>

namespace tt {
namespace {

// ------------------------------------------------------------------- numbers
//
// A token is drawn where a running sum of up to 2^24 weights passes a random number, so weights and sums are held in 64
// bits: in 32 bits about one draw in a thousand from a flat distribution would be another token's.

// The order of logits as whole numbers; NaN below everything, the zeros alike.
__device__ inline uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x != x ? 0u : (u >> 31 ? ~u : u | 0x80000000u);
}
__device__ inline float logit_of(uint32_t order) { return __uint_as_float(order >> 31 ? order & 0x7FFFFFFFu : ~order); }
constexpr uint32_t NOTHING = 0x007FFFFFu;  // the order of -infinity
constexpr uint32_t ALL = 0xFFFFFFFFu;

// 2^t for t from -1010 to 0: the nearest whole number apart, which a large number added leaves in its lowest bits, 1 + f p(f) on
// -1/2 .. 1/2 with p through the 9 Chebyshev nodes, off by less than 4e-14 of the value and exact at 0; the whole number goes to the exponent.
__device__ inline double power_of_two(double t) {
  constexpr double LARGE = 6755399441055744.0;  // 1.5 * 2^52
  const double n = t + LARGE, f = t - (n - LARGE);
  double y = 1.0203121113055101e-07;
  y = fma(y, f, 1.3255224878933224e-06);
  y = fma(y, f, 1.5252686846120593e-05);
  y = fma(y, f, 0.00015403455852451632);
  y = fma(y, f, 0.0013333558179043103);
  y = fma(y, f, 0.0096181291594025619);
  y = fma(y, f, 0.055504108664760424);
  y = fma(y, f, 0.24022650695812989);
  y = fma(y, f, 0.69314718055994529);
  y = fma(y, f, 1.0);
  return __hiloint2double(__double2hiint(y) + (int)((uint32_t)__double2loint(n) << 20), __double2loint(y));
}

// Weights of a row: e^((x - top) / temperature); below 2^-1000 they count as zero.
struct Weigher {
  float most;    // top as it was
  float lowest;  // the logit that weighs 2^-1000, as far as 32 bits tell
  double top, by;  // by = log2 e / temperature
  __device__ Weigher(float most_, float temperature) : most(most_), top(most_), by(1.4426950408889634 / (double)temperature) {
    lowest = (float)(top - 1000.0 / by);
  }
  // log2 of the weight; NaN where there is none
  __device__ double exponent(float x) const { return ((double)x - top) * by; }
  // (top itself apart, for an infinite one and for temperatures at which nothing else weighs; NaN weighs nothing.  Rounded to 32 bits, `lowest`
  // may lie many powers off where a step of the logits is as large as the temperature, so the exponent itself is compared)
  __device__ double operator()(float x) const {
    const double t = exponent(x), y = power_of_two(t);
    return x == most ? 1.0 : t >= -1000.0 ? y : 0.0;
  }
  // Where the lowest is a number well below the top, sums that the top is in do not tell 2^-1000 from zero; and where it is not so far below that
  // its power leaves the range, the smaller logits may be taken for it.
  __device__ bool clear() const {
    const double t = exponent(lowest);
    return t < -900.0 && t >= -1010.0;
  }
  __device__ double roughly(float x) const { return power_of_two(exponent(fmaxf(x, lowest))); }
  // log2 of the weight, 0 down to -2^25.
  __device__ float depth(float x) const {
    const double t = exponent(x);
    return x == most ? 0.0f : t >= -1000.0 ? (float)t : -33554432.0f;
  }
};

// What is asked of a row.
struct Limits {
  float temperature, top_p, min_p, uniform;
  int64_t top_k;                    // 0: none
  bool single, by_mass, by_weight;  // the first token alone; top_p limits; min_p limits
  __device__ __forceinline__ bool limited() const { return top_k || by_mass || by_weight; }
  // The weight of the whole row is asked for: the nucleus is a share of it, or the draw goes by it.  After top_k it is a share of what that leaves.
  __device__ __forceinline__ bool summed() const { return !single && !top_k && (by_mass || !by_weight); }
};
__device__ inline Limits limits_of(const tt_sample_args& a, int64_t r) {
  Limits l;
  const float u = a.uniform[r];
  l.temperature = a.temperature ? a.temperature[r] : 1.0f;
  l.top_p = a.top_p ? a.top_p[r] : 1.0f;
  l.min_p = a.min_p ? a.min_p[r] : 0.0f;
  const int k = a.top_k ? a.top_k[r] : 0;
  l.top_k = k > 0 && k < a.vocab ? k : 0;
  l.uniform = u >= 1.0f ? 0x1.fffffep-1f : u > 0.0f ? u : 0.0f;  // NaN is 0
  l.by_mass = l.top_p < 1.0f;
  l.by_weight = l.min_p > 0.0f;
  l.single = !(l.temperature > 0.0f) || k == 1 || l.top_p <= 0.0f || l.min_p > 1.0f;
  return l;
}

// ------------------------------------------------------------ parts of a row
//
// A wavefront takes up to 2,048 logits into registers: their maximum, the sum of their weights by it, and, where the row has
// limits, a list of its largest ones, all that are not below a bar of its own.  What is above the highest of
// the bars is in the lists, so rows need not be read again whose likely tokens are spread over the ids.  Where they lie beside each
// other, the parts that have them raise the highest bar, and less is above it: of 20 rows of 128,256 normal logits (sigma 2) that fall by
// ln(id + 10) some 10 tokens, and top_k 50 goes over all of them again.

constexpr int PT_STEP = WAVE * 8;
constexpr int PT_LIST = 64;
constexpr int PT_THREADS = 256;
constexpr int64_t PT_BATCH = 65536;  // parts of a launch
constexpr int WD_SLOTS = 256;        // most rows of a launch that are gone over again by many workgroups
constexpr int WD_BINS = 2048;
constexpr int WD_SEGMENT = 4;        // parts of a workgroup: 256 x 262,144 take 110 us, with 8 or 2 114; 61 x 100,257 49, with 8 53

struct Part {
  double sum;
  double kept;     // of rows gone over again: the weight of what is kept for certain
  float most;
  uint32_t bar;    // the order down to which all tokens are listed
  uint32_t count;  // of the list; above PT_LIST: it would have had more
  uint32_t high;   // a higher bar, which a few of the tokens listed are not below
};
struct Listed {
  uint32_t order, id;
};
struct Slot {
  int64_t row;
  u64 mass[WD_BINS];
};
// What is known of a row that is not done.
struct Row {
  double whole;    // what all tokens weigh, if that is asked for
  float most;      // the largest logit
  uint32_t state;  // DONE, LEFT, or its slot
  uint32_t last;   // with a slot: the bin that the nucleus ends in
  uint32_t none;
};
struct Space {
  uint32_t* slots_taken;
  Row* rows;
  Part* parts;
  Listed* lists;
  Slot* slots;  // nullptr: rows are gone over again by a workgroup each
  uint32_t slot_count;
  int64_t per_row, bytes;
  uint32_t size;  // tokens of a part
};
constexpr uint32_t DONE = 0xFFFFFFFFu, LEFT = 0xFFFFFFFEu;

template <class T>
struct Eight {
  typedef T type __attribute__((ext_vector_type(8), aligned(alignof(T))));
};

// Q * 512 tokens a part, each read once.  By a wavefront alone: parts need nothing of each other.  Most of a call's wavefronts are there at once, so
// all load first and weigh then, and one hides little of the other.  What bounds it are the weights: one and its sum are 16 operations in 64 bits, at
// a bit more than half the rate of those in 32.  192 x 100,256 bfloat16 without limits take 21.8 us, of which reading is 7
// (38.5 MB at 5.6 TB/s); 256 x 262,144 float32, a third of whose rows are summed up, 54, of which reading is 48, and 64 if all are.
template <class T, int Q>
__global__ __launch_bounds__(PT_THREADS) void k_sample_parts(tt_sample_args a, Space space) {
  constexpr int MINE = Q * 8;
  const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int64_t id = (int64_t)blockIdx.x * (PT_THREADS / WAVE) + wave, r = id / space.per_row;
  if (id == 0 && lane == 0) *space.slots_taken = 0;
  if (r >= a.rows) return;
  const uint32_t vocab = (uint32_t)a.vocab, first = (uint32_t)(id - r * space.per_row) * (Q * PT_STEP);
  const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
  float x[MINE];
  if (first + Q * PT_STEP <= vocab) {
    typename Eight<T>::type v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = *reinterpret_cast<const typename Eight<T>::type*>(row + first + q * PT_STEP + lane * 8);
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[q * 8 + k] = (float)v[q][k];
  } else {
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const uint32_t v = first + i / 8 * PT_STEP + lane * 8 + i % 8;
      x[i] = v < vocab ? (float)row[v] : -__builtin_inff();
    }
  }
  const Limits limits = limits_of(a, r);
  float mine = -__builtin_inff();  // the maximum passes over NaN
#pragma unroll
  for (int i = 0; i < MINE; ++i) mine = fmaxf(mine, x[i]);
  const uint32_t own = order_of(mine);
  const uint32_t top = max_of_lanes(own);
  Part part{0, 0, logit_of(top), NOTHING + 1, 0, NOTHING + 1};
  if (top > NOTHING && !limits.single) {
    if (limits.summed()) {
      const Weigher w(part.most, limits.temperature);
      double sum = 0;
      if (w.clear()) {
#pragma unroll
        for (int i = 0; i < MINE; ++i) sum += w.roughly(x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < MINE; ++i) sum += w(x[i]);
      }
      part.sum = sum_of_lanes(sum);
    }
    if (limits.limited()) {
      // A bar is the n-th largest of the lanes' maxima, n halved where the list would not hold what is not below it.  The high one leaves 300
      // to 400 tokens of a row; the other one, for where top_k may be more than that, about 64 ln 2 = 44 of a part, or half of that where the
      // lists of a row would be too many.
      auto largest = [&](int among) {
        uint32_t bar = 0;
        for (uint32_t bit = 1u << 31; bit; bit >>= 1)
          if (__popcll(__ballot(own >= (bar | bit))) >= among) bar |= bit;
        return max(bar, NOTHING + 1);
      };
      const int few = min((int)(300 / space.per_row) + 6, WAVE / 2);
      const bool many = limits.top_k > 128;
      uint32_t bar = 0, count = 0, counts = 0, in = 0;  // in: a bit for each token of the lane
      for (int among = !many ? few : space.per_row > 128 ? WAVE / 4 : WAVE / 2; among; among /= 2) {
        bar = largest(among);
        const float from = logit_of(bar);
        in = 0;
#pragma unroll
        for (int i = MINE - 1; i >= 0; --i) in = in + in + (uint32_t)(x[i] >= from);
        // counts of the steps, a byte each, which hold what a list does: eight tokens of a lane, the lanes, the steps
        counts = in - (in >> 1 & 0x55555555u);
        counts = (counts & 0x33333333u) + (counts >> 2 & 0x33333333u);
        counts = (counts + (counts >> 4)) & 0x0F0F0F0Fu;
        count = sum_of_lanes((uint32_t)__popc(in));
        if (count <= PT_LIST) break;
      }
      if (count > PT_LIST) bar = ALL, count = 0;
      part.bar = bar, part.count = count, part.high = many ? max(largest(few), bar) : bar;
      if (count) {
        const uint32_t upto = sums_upto(counts), all = of_lane(upto, WAVE - 1);
        // where the lane's tokens of each step go, a byte each again
        const uint32_t at = upto - counts + (all << 8) + (all << 16) + (all << 24);
        Listed* to = space.lists + id * PT_LIST;
        for (uint32_t left = in; left; left &= left - 1) {  // a few; registers have no numbers, so they are read again
          const uint32_t i = __builtin_ctz(left), q = i / 8;
          const uint32_t place = (at >> (8 * q) & 255) + __popc(in & ((1u << i) - 1) & ~((1u << (8 * q)) - 1));
          const uint32_t v = first + q * PT_STEP + lane * 8 + i % 8;
          to[place] = Listed{order_of((float)row[v]), v};
        }
      }
    }
  }
  if (lane == 0) space.parts[id] = part;
}

// -------------------------------------------------------------- a workgroup
//
// The draw from the lists is a chain of sums over a workgroup with little to do in between, which eight wavefronts get through
// sooner than sixteen (one row of 50,256 24.4 us instead of 25.6, 61 of 100,257 48.9 instead of 49.9); going over a row again takes sixteen.

constexpr int DR_THREADS = 512;
constexpr int RS_THREADS = 1024;
constexpr int SA_PARTS = 256;   // of a row whose lists are put together
constexpr int SA_LIST = 4096;   // tokens of the lists that are above all bars
constexpr int SA_BINS = 256;
constexpr int SA_TILES = 1024;  // that a row is summed up in

// What a wavefront has found.
struct Hit {
  u64 before;
  uint32_t thread, kind;
};

struct SampleShared {
  union {
    u64 key[RS_THREADS];
    u64 depth[WD_BINS];
    double tile[SA_TILES];
    uint32_t ties[SA_TILES];
  };
  double weight[SA_LIST];
  uint32_t order[SA_LIST], id[SA_LIST];
  uint32_t start[SA_PARTS];
  u64 digit[SA_BINS];
  u64 of_wave[RS_THREADS / WAVE];
  Hit hit[RS_THREADS / WAVE];
  u64 above, of;
  uint32_t found, place;
};

__device__ inline u64 bits(double v) { return (u64)__double_as_longlong(v); }
__device__ inline u64 bits(u64 v) { return v; }
__device__ inline u64 bits(uint32_t v) { return v; }
template <class V>
__device__ inline V value(u64 v) {
  if constexpr (std::is_same<V, double>::value) return __longlong_as_double((long long)v);
  else return (V)v;
}

// The N threads of a workgroup and what they share.
template <int N>
struct Group {
  static constexpr int THREADS = N, WAVES = N / WAVE;
  SampleShared& s;
  int tid, lane, wave;

  // The sum of x over the workgroup, and over the threads before this one and up to it, the one of a thread being the other's of the next.
  template <class V>
  __device__ __forceinline__ V sum(V x, V& before, V& upto) {
    upto = sums_upto(x);
    before = from_lanes<0x138, 0xf>(upto);  // of the lane before
    __syncthreads();
    if (lane == WAVE - 1) s.of_wave[wave] = bits(upto);
    __syncthreads();
    V total = lane < WAVES ? value<V>(s.of_wave[lane]) : 0;  // of the wavefronts up to the lane's
    total += from_lanes<0x111, 0xf>(total);
    total += from_lanes<0x112, 0xf>(total);
    total += from_lanes<0x114, 0xf>(total);
    total += from_lanes<0x118, 0xf>(total);
    const V base = wave ? of_lane(total, wave - 1) : 0, here = of_lane(total, wave);
    before += base, upto = lane == WAVE - 1 ? here : upto + base;
    return of_lane(total, WAVES - 1);
  }
  template <class V>
  __device__ __forceinline__ V sum(V x) {
    V before, upto;
    return sum(x, before, upto);
  }
  // The largest x and y.
  __device__ __forceinline__ void most(uint32_t& x, uint32_t& y) {
    x = max_of_lanes(x), y = max_of_lanes(y);
    __syncthreads();
    if (lane == 0) s.of_wave[wave] = (u64)x << 32 | y;
    __syncthreads();
    const u64 v = lane < WAVES ? s.of_wave[lane] : 0;
    x = max_of_lanes((uint32_t)(v >> 32)), y = max_of_lanes((uint32_t)v);
  }

  // The first thread with an x above 0 at which the running sum of x satisfies enough(sum, sum of all), which 0 does not; the last one with an
  // x above 0 if none does, since sums that are rounded may stay just below.  `before`: the sum of the threads before it.  Nor need rounded sums rise: a thread
  // without anything may have one that is a step above that of the thread before it, so what it has itself is asked too.
  // Each wavefront writes down its own such thread; that happens behind the barriers of a sum, so it cannot meet the reads of the search before.
  template <class V, class F>
  __device__ __forceinline__ uint32_t first(V x, F enough, V& before, V& all) {
    V at, upto;
    all = sum(x, at, upto);
    const u64 some = __ballot(x > 0), reached = __ballot(x > 0 && enough(upto, all));
    if (lane == (reached ? __builtin_ctzll(reached) : some ? 63 - __builtin_clzll(some) : 0))
      s.hit[wave] = Hit{bits(at), (uint32_t)tid, reached ? 2u : some ? 1u : 0u};
    __syncthreads();
    const Hit hit = lane < WAVES ? s.hit[lane] : Hit{0, 0, 0};
    const u64 found = __ballot(hit.kind == 2), other = __ballot(hit.kind == 1);
    const int of = found ? __builtin_ctzll(found) : other ? 63 - __builtin_clzll(other) : 0;
    before = value<V>(of_lane(hit.before, of));
    return of_lane(hit.thread, of);
  }
};

// Where the logits come from: a row in memory, or the tokens listed with their weights.  each: f(order, weight, place), the weight to be
// called for, for the tokens of the thread in any order; in_row: for those of its share of the places from `from` up to `end`,
// in order, as long as f returns true.
template <class T>
struct RowSource {
  // logits of 16 bits leave the lowest bits of their order alike
  static constexpr bool LISTED = false;
  static constexpr int LOW = std::is_same<T, float>::value ? 0 : std::is_same<T, _Float16>::value ? 13 : 16;
  const T* row;
  uint32_t size;
  // Eight from `place` on; -infinity from `end` on.
  __device__ void eight(uint32_t place, uint32_t end, float (&x)[8]) const {
    if (place + 8 <= end) {
      const auto v = *reinterpret_cast<const typename Eight<T>::type*>(row + place);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = (float)v[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = place + k < end ? (float)row[place + k] : -__builtin_inff();
    }
  }
  template <int N, class F>
  __device__ __forceinline__ void each(const Weigher& w, F f) const {
#pragma unroll 1
    for (uint32_t i = threadIdx.x * 8; i < size; i += N * 8) {
      float x[8];
      eight(i, size, x);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + k < size) f(order_of(x[k]), [&] { return w(x[k]); }, i + k);
    }
  }
  template <int N, class F>
  __device__ __forceinline__ void in_row(const Weigher& w, uint32_t from, uint32_t end, F f) const {
    const uint32_t per = (end - from + N - 1) / N, own = from + threadIdx.x * per, stop = min(own + per, end);
    bool more = true;
#pragma unroll 1
    for (uint32_t at = own; at < stop && more; at += 8) {
      float x[8];
      eight(at, stop, x);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at + k < stop && more) more = f(order_of(x[k]), [&] { return w(x[k]); }, at + k);
    }
  }
};
template <class T>
struct ListSource {
  static constexpr bool LISTED = true;
  static constexpr int LOW = RowSource<T>::LOW;
  const SampleShared& s;
  uint32_t size;
  template <int N, class F>
  __device__ __forceinline__ void each(const Weigher&, F f) const {
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < size; i += N) f(s.order[i], [&] { return s.weight[i]; }, i);
  }
  template <int N, class F>
  __device__ __forceinline__ void in_row(const Weigher&, uint32_t, uint32_t, F f) const {
    const uint32_t per = (size + N - 1) / N, own = threadIdx.x * per, stop = min(own + per, size);
#pragma unroll 1
    for (uint32_t i = own; i < stop; ++i)
      if (!f(s.order[i], [&] { return s.weight[i]; }, i)) break;
  }
};

// The place from `from` up to `end` at which the running sum of f(order, weight, place), `before` at first, gets above goal(sum of these), the last one
// with a sum if it does not, and its f; by the workgroup.
template <class V, class Source, class Threads, class F, class G>
__device__ __forceinline__ uint32_t locate(const Source& source, const Weigher& w, Threads& g, uint32_t from, uint32_t end, V before, F f, G goal, V& mine,
                                           V& all) {
  constexpr int N = Threads::THREADS;
  V sum = 0, at;
  source.template in_row<N>(w, from, end, [&](uint32_t o, auto weight, uint32_t place) {
    sum += f(o, weight, place);
    return true;
  });
  const uint32_t thread = g.first(sum, [&](V upto, V total) { return before + upto > goal(total); }, at, all);
  if (thread == (uint32_t)g.tid) {
    V run = before + at, of = 0;
    uint32_t found = from;
    source.template in_row<N>(w, from, end, [&](uint32_t o, auto weight, uint32_t place) {
      const V x = f(o, weight, place);
      run += x;
      if (x > 0) found = place, of = x;
      return !(x > 0 && run > goal(all));
    });
    g.s.place = found, g.s.of = bits(of);
  }
  __syncthreads();
  mine = value<V>(g.s.of);
  return g.s.place;
}

// Sums of weights in 64 bits of fixed point, which are the same in any order.  A value from 0 to 2^62, rounded at its lowest bits.
__device__ inline u64 fixed(double x) {
  const double high = __builtin_floor(x * 0x1p-32), low = fma(high, -0x1p32, x);
  return (u64)(uint32_t)high << 32 | (uint32_t)low;
}
// This is 1.
__device__ inline double one_of(uint32_t tokens) { return __builtin_ldexp(1.0, 62 - (32 - __builtin_clz(tokens))); }

// What is kept of a source of logits: orders above `least`, and those at it up to the place `until`, of a weight of min_p or more.
struct Kept {
  uint32_t least, until;
  double min_p;
  template <class W>
  __device__ __forceinline__ double of(uint32_t order, W weight, uint32_t place) const {
    if (order < least || (order == least && place > until)) return 0.0;
    const double y = weight();
    return y < min_p ? 0.0 : y;
  }
};

// A source of logits that a workgroup passes over for every question.
template <class Source, class Threads>
struct Sampler {
  static constexpr int N = Threads::THREADS;
  const Source& source;
  const Weigher& w;
  Threads& g;
  SampleShared& s;
  uint32_t most;  // the largest order

  // What the tokens weigh whose order `take` takes.
  template <class F>
  __device__ __forceinline__ double sum(F take) {
    double sum = 0;
    source.template each<N>(w, [&](uint32_t o, auto weight, uint32_t) {
      if (take(o)) sum += weight();
    });
    return g.sum(sum);
  }

  // The order at which, from the largest down to `least`, as many tokens (or, by mass, as much weight) as `target` are reached,
  // by digits of 8 bits, each from the first bit on that tells the candidates apart.  `above` receives how many (how much) there are above it,
  // `there` how many (how much) at it.
  __device__ __forceinline__ uint32_t reach(bool mass, uint32_t least, double target, double& above, double& there) {
    const double one = mass ? one_of(source.size) : 1.0, unit = 1 / one;
    uint32_t largest = most, smallest = least;  // of the orders that it may be
    above = 0;
#pragma unroll 1
    while (true) {
      const uint32_t apart = largest ^ smallest;
      const int top = max(apart ? 32 - __builtin_clz(apart) : 0, Source::LOW), width = min(8, top - Source::LOW), shift = top - width;
      const uint32_t prefix = top < 32 ? largest >> top : 0;
      __syncthreads();
      if (g.tid < SA_BINS) s.digit[g.tid] = 0;
      __syncthreads();
      source.template each<N>(w, [&](uint32_t o, auto weight, uint32_t) {
        if (o >= least && (top == 32 || o >> top == prefix))
          atomicAdd(&s.digit[o >> shift & ((1u << width) - 1)], mass ? fixed(weight() * one) : (u64)1);
      });
      __syncthreads();
      const u64 x = g.tid < SA_BINS ? s.digit[SA_BINS - 1 - g.tid] : 0;  // from the largest down
      u64 before, all;
      const uint32_t digit = SA_BINS - 1 - g.first(x, [&](u64 upto, u64) { return upto && above + (double)upto * unit >= target; }, before, all);
      above += (double)before * unit;
      there = (double)s.digit[digit] * unit;
      const uint32_t found = prefix << width | digit;
      // the largest and the smallest that are left; the rest of the digits that they share is skipped
      largest = 0;
      uint32_t inverse = 0;
      source.template each<N>(w, [&](uint32_t o, auto, uint32_t) {
        if (o >= least && o >> shift == found) largest = max(largest, o), inverse = max(inverse, ~o);
      });
      g.most(largest, inverse);
      smallest = ~inverse;
      if (!inverse) return most;  // nothing weighs anything
      if (largest == smallest || !width) return largest;
    }
  }

  // The first place at which the running sum of f(order, weight, place) is above goal(sum of all); mine: its f.
  template <class V, class F, class G>
  __device__ __forceinline__ uint32_t find(V* tiles, F f, G goal, V& mine, V& all) {
    if constexpr (Source::LISTED) {
      return locate(source, w, g, 0, source.size, (V)0, f, goal, mine, all);
    } else {
      static_assert(N == SA_TILES, "a tile for each thread");
      const uint32_t size = (source.size + SA_TILES - 1) / SA_TILES, per = (size + WAVE - 1) / WAVE * WAVE;  // of a tile
      __syncthreads();
#pragma unroll 1
      for (uint32_t t = g.wave; t < SA_TILES; t += N / WAVE) {
        V sum = 0;
#pragma unroll 1
        for (uint32_t i = t * per + g.lane; i < min((t + 1) * per, source.size); i += WAVE) {
          const float x = (float)source.row[i];
          sum += f(order_of(x), [&] { return w(x); }, i);
        }
        sum = sum_of_lanes(sum);
        if (g.lane == 0) tiles[t] = sum;
      }
      __syncthreads();
      const V x = tiles[g.tid];
      V before, some;
      const uint32_t t = g.first(x, [&](V upto, V total) { return upto > goal(total); }, before, all);
      const V least = goal(all);
      return locate(source, w, g, t * per, min((t + 1) * per, source.size), before, f, [&](V) { return least; }, mine, some);
    }
  }

  // The last place kept of those of order `least`, if the first `ties` of them are.
  __device__ __forceinline__ uint32_t until(uint32_t least, double ties) {
    const uint32_t goal = (uint32_t)__builtin_fmin(ties, 4e9) - 1;
    uint32_t one, all;
    const uint32_t place = find(s.ties, [&](uint32_t o, auto, uint32_t) { return (uint32_t)(o == least); }, [&](uint32_t) { return goal; }, one, all);
    return goal < all ? place : ALL;
  }

  // The token drawn, as its place, and what it and all that are kept weigh.  `by_mass`, if it is not negative: what the nucleus has
  // to weigh, or, of the tokens that top_k leaves, what share of them.
  __device__ __forceinline__ Kept kept(const Limits& l, double by_mass) {
    uint32_t least = NOTHING + 1;
    double ties = -1;  // of those at `least` so many are kept; all of them if negative
#pragma unroll 1
    for (int mass = 0; mass < 2; ++mass) {  // the same code for both limits
      if (!(mass ? by_mass >= 0 : l.top_k != 0)) continue;
      double target = mass ? by_mass : (double)l.top_k, above, there;
      if (mass && l.top_k)
        target *= sum([&](uint32_t o) { return o > least || (ties < 0 && o == least); }) + (ties > 0 ? ties * w(logit_of(least)) : 0.0);
      const uint32_t last = reach(mass, mass ? least : NOTHING, target, above, there);
      if (!mass) {
        if (last > NOTHING) least = last, ties = target - above < there ? target - above : -1;
        continue;
      }
      above = sum([&](uint32_t o) { return o > last; });
      const double one = w(logit_of(last)), needed = __builtin_fmax(__builtin_ceil((target - above) / one), 1.0);
      // all of them, where their weight says for certain how many they are
      const bool every = one * one_of(source.size) > 0x1p28 && needed >= __builtin_rint(there / one);
      if (last == least && ties >= 0) ties = __builtin_fmin(ties, needed);
      else ties = every ? -1 : needed;
      least = last;
    }
    return Kept{least, ties >= 0 ? until(least, ties) : ALL, l.by_weight ? (double)l.min_p : 0.0};
  }
  __device__ __forceinline__ uint32_t draw(const Limits& l, double by_mass, double& mine, double& all) {
    const Kept k = kept(l, by_mass);
    return find(s.tile, [&](uint32_t o, auto weight, uint32_t place) { return k.of(o, weight, place); }, [&](double total) { return (double)l.uniform * total; },
                mine, all);
  }
};

// Puts out a row's token.
__device__ inline void put_token(const tt_sample_args& a, int64_t r, uint32_t token, double mine, double all) {
  a.tokens[r] = (int32_t)token;
  if (a.logprobs) a.logprobs[r] = token == ALL ? -__builtin_inff() : (float)log(mine / all);
}

// The tokens that the parts' lists hold from the order `bar` on, in the order of ids, to s.order and s.id; how many there are, which may be
// more than there is room for: then none are taken.  s.start[p]: where those of part p begin.
template <class Threads>
__device__ __forceinline__ uint32_t gather(Threads& g, const Part* parts, const Listed* lists, int n, uint32_t bar) {
  constexpr int WAVES = Threads::WAVES, MANY = 128 / WAVES;  // lists of a wavefront that are on their way together
  SampleShared& s = g.s;
  __syncthreads();
  if (g.tid < SA_PARTS) s.start[g.tid] = 0;
  __syncthreads();
  Listed entry[MANY];
  uint32_t count[MANY], start, upto, size = 0;
  // the same loop counts what there is, and then takes it
#pragma unroll 1
  for (int take = 0; take < 2; ++take) {
#pragma unroll 1
    for (int from = g.wave; from < n; from += MANY * WAVES) {
      if (!take || n > MANY * WAVES) {
#pragma unroll
        for (int k = 0; k < MANY; ++k) {
          const int p = min(from + k * WAVES, n - 1);
          entry[k] = lists[(int64_t)p * PT_LIST + g.lane];  // past the count there is anything
          count[k] = from + k * WAVES < n ? parts[p].count : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < MANY; ++k) {
        const bool here = g.lane < (int)count[k] && entry[k].order >= bar;
        const u64 in = __ballot(here);
        if (!take) {
          if (g.lane == 0 && in) s.start[from + k * WAVES] = __popcll(in);
        } else if (here) {
          const uint32_t to = s.start[from + k * WAVES] + __popcll(in & (((u64)1 << g.lane) - 1));
          s.order[to] = entry[k].order, s.id[to] = entry[k].id;
        }
      }
    }
    __syncthreads();
    if (take) break;
    size = g.sum(g.tid < SA_PARTS ? s.start[g.tid] : 0, start, upto);
    if (g.tid < SA_PARTS) s.start[g.tid] = start;
    __syncthreads();
    if (size > SA_LIST) break;
  }
  return size;
}

// The weights of a list.
template <class Threads>
__device__ __forceinline__ void weigh(Threads& g, uint32_t size, const Weigher& w) {
#pragma unroll 1
  for (uint32_t i = g.tid; i < size; i += Threads::THREADS) g.s.weight[i] = w(logit_of(g.s.order[i]));
  __syncthreads();
}

// All tokens of a row that is short enough, as a list.
template <class Threads, class T>
__device__ __forceinline__ uint32_t gather_row(Threads& g, const RowSource<T>& row) {
  __syncthreads();
  for (uint32_t i = g.tid; i < row.size; i += Threads::THREADS) g.s.order[i] = order_of((float)row.row[i]), g.s.id[i] = i;
  __syncthreads();
  return row.size;
}

// The keys of the workgroup's threads, the largest first; `size` of them are not 0.
template <class Threads>
__device__ __forceinline__ u64 sorted(Threads& g, u64 key, uint32_t size) {
  SampleShared& s = g.s;
#pragma unroll 1
  for (int run = 2; run < 2 * Threads::THREADS; run *= 2) {
    if (run / 2 >= (int)size) break;  // what is not 0 is sorted
#pragma unroll 1
    for (int apart = run / 2; apart >= WAVE; apart /= 2) {
      __syncthreads();
      s.key[g.tid] = key;
      __syncthreads();
      const u64 other = s.key[g.tid ^ apart];
      key = (!(g.tid & apart) == !(g.tid & run)) == (other > key) ? other : key;
    }
    key = exchanged_in_wave(key, g.tid, run);
  }
  return key;
}

// What is kept of a list of at most as many tokens as threads, a token a thread.
struct Picked {
  bool decided;
  double weight;  // of the thread's token, 0 if it is not kept
  u64 last;       // the key of the last one kept: its order, and the inverse of its place
};

// `bar`: the order that the list goes down to, all tokens being there if nothing is below; `above`: what tokens before the list weigh, all of
// them kept; `whole`: what all tokens of the row weigh.  The list is shorter than the workgroup.
template <class Threads>
__device__ __forceinline__ Picked pick(Threads& g, uint32_t size, uint32_t top_k, const Limits& l, const Weigher& w, uint32_t bar, double above, double whole) {
  SampleShared& s = g.s;
  const uint32_t tid = g.tid;
  const bool here = tid < size, complete = bar <= NOTHING + 1;
  const uint32_t own = here ? s.order[tid] : tid == size ? bar : 0;
  const double weight = w(logit_of(own));
  s.weight[tid] = weight;
  const u64 key = here ? (u64)own << 32 | ~tid : 0;  // the larger the earlier
  const u64 nth = sorted(g, key, size);
  __syncthreads();
  const bool light = l.by_weight && s.weight[size] < (double)l.min_p;  // what is below the bar
  double before, upto;
  g.sum(nth ? s.weight[~(uint32_t)nth] : 0.0, before, upto);
  before += above, upto += above;
  const bool limit = top_k && top_k <= size;
  const uint32_t most = limit ? top_k : size;
  if (tid == most - 1) s.above = bits(upto), s.found = tid;
  __syncthreads();
  const double of = value<double>(s.above);  // what the first `most` weigh
  const double target = (double)l.top_p * (limit || (complete && top_k) ? of : whole);
  const bool known = complete || limit || !top_k;  // what the nucleus is a share of
  const bool by_mass = l.by_mass && known && (complete || of >= target * (limit ? 1 : 1 + 1e-12));
  if (by_mass && upto >= target && (tid == 0 || before < target)) atomicMin(&s.found, tid);
  __syncthreads();
  if (tid == s.found) s.of = nth;
  __syncthreads();
  Picked p;
  p.last = s.of;
  p.decided = l.by_mass ? by_mass || (known && light) : complete || limit || light;
  p.weight = here && key >= p.last && weight >= (l.by_weight ? (double)l.min_p : 0.0) ? weight : 0.0;
  return p;
}

// Of a list of `size` tokens those that top_k may leave, all of its last order among them, with `bar` that order: how many there are. They
// stay in the order of ids, which a few tokens a thread one behind the other keep.
template <class Source, class Threads>
__device__ __forceinline__ uint32_t shortened(const Source& source, Threads& g, const Weigher& w, uint32_t most, uint32_t top_k, uint32_t& bar) {
  constexpr int MINE = SA_LIST / Threads::THREADS;
  SampleShared& s = g.s;
  double above, there;
  Sampler<Source, Threads> list{source, w, g, s, most};
  const uint32_t last = list.reach(false, bar > NOTHING + 1 ? bar : 0, top_k, above, there);
  uint32_t order[MINE], id[MINE], count = 0, before, upto;
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const uint32_t i = g.tid * MINE + k;
    order[k] = i < source.size ? s.order[i] : 0, id[k] = i < source.size ? s.id[i] : 0;
    count += i < source.size && order[k] >= last;
  }
  const uint32_t size = g.sum(count, before, upto);
#pragma unroll
  for (int k = 0; k < MINE; ++k)
    if (g.tid * MINE + k < source.size && order[k] >= last) s.order[before] = order[k], s.id[before++] = id[k];
  __syncthreads();
  bar = last;
  return size;
}

// A row by a workgroup, from its parts.  Without limits the part that the random number falls into is read again; with limits
// the tokens above all high bars, if they are few, are sorted, which answers everything that is asked of them; if the last one kept is not
// among them the row is left to be gone over again.  Bound by its chain of dependent steps: the bars, the lists, 45 exchanges, three
// sums, 13 us for a row of 50,256, 15 for 256 rows of 262,144 at once; the radix selection that it took the place of was 40.
template <class T>
__global__ __launch_bounds__(DR_THREADS) void k_sample(tt_sample_args a, Space space) {
  __shared__ SampleShared s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const Part* parts = space.parts + r * space.per_row;
  const Limits l = limits_of(a, r);
  const int n = (int)space.per_row, per = (n + DR_THREADS - 1) / DR_THREADS;  // parts of a thread, one behind the other
  const RowSource<T> row{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab};
  Group<DR_THREADS> g{s, tid, tid % WAVE, tid / WAVE};

  uint32_t top = 0, high = NOTHING + 1;  // the largest order and the highest of the high bars
  for (int p = tid * per; p < min((tid + 1) * per, n); ++p) top = max(top, order_of(parts[p].most)), high = max(high, parts[p].high);
  g.most(top, high);
  if (tid == 0) space.rows[r].state = DONE;
  if (top <= NOTHING) {
    if (tid == 0) put_token(a, r, ALL, 0, 1);
    return;
  }
  double mine = 1, all = 1, whole = 0, some;
  uint32_t token;
  const Weigher w(logit_of(top), l.temperature);
  auto weight_of = [&](int p) { return parts[p].sum > 0 ? parts[p].sum * w(parts[p].most) : 0.0; };
  if (l.summed())
    for (int p = tid * per; p < min((tid + 1) * per, n); ++p) whole += weight_of(p);
  if (l.single || !l.limited()) {
    uint32_t p = 0;
    double goal = 0, before = 0;
    if (l.single) {  // the first part that has it
      uint32_t first = 0;
      for (int q = tid; q < n; q += DR_THREADS)
        if (order_of(parts[q].most) == top) first = max(first, ~(uint32_t)q);
      uint32_t none = 0;
      g.most(first, none);
      p = ~first;
    } else {
      const uint32_t thread = g.first(whole, [&](double upto, double total) { return upto > (double)l.uniform * total; }, before, all);
      goal = (double)l.uniform * all;
      double upto = before;
      for (uint32_t q = thread * per; q < min((thread + 1) * per, (uint32_t)n); ++q) {
        const double y = weight_of(q);
        if (!(y > 0)) continue;
        p = q, before = upto, upto += y;
        if (upto > goal) break;
      }
    }
    const uint32_t from = p * space.size;
    const RowSource<T> part{row.row + from, min(space.size, row.size - from)};
    gather_row(g, part);
    if (l.single) {
      for (uint32_t i = tid; i < part.size; i += DR_THREADS) s.weight[i] = s.order[i] == top ? 1.0 : 0.0;
      __syncthreads();
    } else {
      weigh(g, part.size, w);
    }
    const ListSource<T> list{s, part.size};
    token = from + locate(list, w, g, 0, part.size, before, [&](uint32_t, auto weight, uint32_t) { return weight(); }, [&](double) { return goal; }, mine, some);
    if (tid == 0) put_token(a, r, token, mine, all);
    return;
  }
  whole = g.sum(whole);
  uint32_t size = ALL;
  if (row.size < DR_THREADS) size = gather_row(g, row), high = NOTHING + 1;
  else if (n <= SA_PARTS && high != ALL) size = gather(g, parts, space.lists + r * space.per_row * PT_LIST, n, high);
  if (size < DR_THREADS) {
    const Picked some = pick(g, size, (uint32_t)l.top_k, l, w, high, 0, whole);
    if (some.decided) {
      double before;
      const uint32_t thread = g.first(some.weight, [&](double sum, double total) { return sum > (double)l.uniform * total; }, before, all);
      if ((uint32_t)tid == thread) put_token(a, r, s.id[tid], some.weight, all);
      return;
    }
  }
  __syncthreads();
  if (tid == 0) {
    s.found = ALL;
    if (space.slots && !l.top_k) s.found = atomicAdd(space.slots_taken, 1u);
    space.rows[r] = Row{whole, logit_of(top), s.found < space.slot_count ? s.found : LEFT, WD_BINS, 0};
    if (s.found < space.slot_count) space.slots[s.found].row = r;
  }
  __syncthreads();
  if (s.found < space.slot_count)
    for (int i = tid; i < WD_BINS; i += DR_THREADS) space.slots[s.found].mass[i] = 0;
}

// ------------------------------------------- rows that have to be gone over again
//
// Where the nucleus goes below the bars, weights are summed by depth (32 bins to a halving), which gives the bin that it ends in;
// then each part sums up what is above that bin and lists what is in it.

// The bin of a token.
__device__ inline uint32_t bin_of(const Weigher& w, float x) { return min((uint32_t)(w.depth(x) * -32.0f), (uint32_t)WD_BINS - 1); }

// The weight of the places from `at` up to `end` into bins of LDS, by a workgroup.
template <class T>
__device__ __forceinline__ void add_to_bins(const RowSource<T>& row, uint32_t at, uint32_t end, int threads, const Weigher& w, double one, u64* bin) {
  for (uint32_t i = at + threadIdx.x * 8; i < end; i += threads * 8) {
    float x[8];
    row.eight(i, end, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double y = w(x[k]);
      if (y > 0) atomicAdd(&bin[bin_of(w, x[k])], fixed(y * one));
    }
  }
}

// A part of such a row, by a wavefront: kept, and sum, are what weighs above bin `last`; of the bin the tokens are listed.
template <class T>
__device__ __forceinline__ void part_above(const RowSource<T>& row, const Space& space, int64_t id, uint32_t p, const Weigher& w, uint32_t last,
                                           double min_p) {
  const int lane = threadIdx.x % WAVE;
  const uint32_t first = p * space.size, end = min(first + space.size, row.size);
  double sum = 0, kept = 0;
  uint32_t count = 0;
  Listed* to = space.lists + id * PT_LIST;
  for (uint32_t step = first; step < end; step += PT_STEP) {
    float x[8];
    const uint32_t at = step + lane * 8;
    row.eight(at, end, x);
    uint32_t in = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const double y = w(x[k]);
      const uint32_t b = bin_of(w, x[k]);
      if (y > 0 && b < last) sum += y, kept += y < min_p ? 0.0 : y;
      in |= (uint32_t)(y > 0 && b == last) << k;
    }
    if (!__ballot(in != 0)) continue;
    const uint32_t mine = __popc(in), upto = sums_upto(mine);
    uint32_t place = count + upto - mine;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (in >> k & 1) {
        if (place < PT_LIST) to[place] = Listed{order_of(x[k]), at + k};
        ++place;
      }
    count += of_lane(upto, WAVE - 1);
  }
  sum = sum_of_lanes(sum), kept = sum_of_lanes(kept);
  if (lane == 0) {
    Part& part = space.parts[id];
    part.sum = sum, part.kept = kept, part.count = count;
  }
}

// The last bin of the nucleus, by a workgroup of WD_BINS / N threads.
template <int N>
__device__ __forceinline__ uint32_t last_bin(const u64* bin, double target, u64* of_wave, uint32_t* found) {
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  u64 x[N], mine = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) mine += x[k] = bin[N * tid + k];
  const u64 upto = sums_upto(mine);
  __syncthreads();  // what is shared may still be read
  if (tid == 0) *found = 0;
  if (lane == WAVE - 1) of_wave[wave] = upto;
  __syncthreads();
  u64 run = upto - mine;
  for (int k = 0; k < wave; ++k) run += of_wave[k];
  uint32_t less = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) run += x[k], less += !((double)run >= target);
  less = sum_of_lanes(less);
  if (lane == 0 && less) atomicAdd(found, less);
  __syncthreads();
  const uint32_t last = *found;
  __syncthreads();
  return min(last, (uint32_t)WD_BINS - 1);
}

// The rows in slots: the bins of their weights.  Each segment is summed up in LDS first.  Bound by the weights and by LDS atomics, 64 bits
// each: 12.4 us for those of 256 rows of 262,144 tokens that need it, which come from the larger cache in good part.
template <class T>
__global__ __launch_bounds__(PT_THREADS) void k_sample_bins(tt_sample_args a, Space space) {
  __shared__ u64 s_bin[WD_BINS];
  const uint32_t slots = min(*space.slots_taken, space.slot_count), across = (uint32_t)((space.per_row + WD_SEGMENT - 1) / WD_SEGMENT);
  for (uint32_t item = blockIdx.x; item < slots * across; item += gridDim.x) {
    Slot& slot = space.slots[item / across];
    const int64_t r = slot.row;
    const Limits l = limits_of(a, r);
    if (!l.by_mass) continue;
    const RowSource<T> row{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab};
    const Weigher w(space.rows[r].most, l.temperature);
    const uint32_t from = item % across * WD_SEGMENT * space.size;
    for (int i = threadIdx.x; i < WD_BINS; i += PT_THREADS) s_bin[i] = 0;
    __syncthreads();
    add_to_bins(row, from, min(from + WD_SEGMENT * space.size, row.size), PT_THREADS, w, one_of((uint32_t)a.vocab), s_bin);
    __syncthreads();
    for (int i = threadIdx.x; i < WD_BINS; i += PT_THREADS)
      if (s_bin[i]) atomicAdd(&slot.mass[i], s_bin[i]);
    __syncthreads();
  }
}

// Their parts.
template <class T>
__global__ __launch_bounds__(PT_THREADS) void k_sample_above(tt_sample_args a, Space space) {
  __shared__ u64 s_wave[PT_THREADS / WAVE];
  __shared__ uint32_t s_found;
  const uint32_t slots = min(*space.slots_taken, space.slot_count), across = (uint32_t)((space.per_row + WD_SEGMENT - 1) / WD_SEGMENT);
  for (uint32_t item = blockIdx.x; item < slots * across; item += gridDim.x) {
    const Slot& slot = space.slots[item / across];
    const int64_t r = slot.row;
    const Limits l = limits_of(a, r);
    const RowSource<T> row{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab};
    const Weigher w(space.rows[r].most, l.temperature);
    const double target = (double)l.top_p * space.rows[r].whole * one_of((uint32_t)a.vocab);
    const uint32_t last = l.by_mass ? last_bin<WD_BINS / PT_THREADS>(slot.mass, target, s_wave, &s_found) : WD_BINS;
    if (item % across == 0 && threadIdx.x == 0) space.rows[r].last = last;
    const uint32_t stop = min((item % across + 1) * WD_SEGMENT, (uint32_t)space.per_row);
    for (uint32_t p = item % across * WD_SEGMENT + threadIdx.x / WAVE; p < stop; p += PT_THREADS / WAVE)
      part_above(row, space, r * space.per_row + p, p, w, last, l.by_weight ? (double)l.min_p : 0.0);
  }
}

// The tokens of rows that are left, or whose parts know what is above their last bin: the bin's tokens are put in order, the part
// is found, and the token in it.  A workgroup a row, since what each needs is little: a row whose bin is known takes 10 to 20 us, one
// whose top_k is beyond what its lists have above the highest bar, or that has more tokens of one logit than these hold, several passes
// over it: a call of one row of 262,144 takes 380 to 550 us then, of 256 rows 440 to 1,000.
template <class T>
__global__ __launch_bounds__(RS_THREADS) void k_sample_rest(tt_sample_args a, Space space) {
  __shared__ SampleShared s;
  const int64_t r = blockIdx.x;
  const Row known = space.rows[r];
  const uint32_t state = known.state;
  if (state == DONE) return;
  const int tid = threadIdx.x, n = (int)space.per_row;
  const Limits l = limits_of(a, r);
  const RowSource<T> row{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab};
  Group<RS_THREADS> g{s, tid, tid % WAVE, tid / WAVE};
  const Part* parts = space.parts + r * space.per_row;
  const float most = known.most;
  const Weigher w(most, l.temperature);
  const double whole = known.whole, target = (double)l.top_p * whole, min_p = l.by_weight ? (double)l.min_p : 0.0;
  double mine = 0, all = 0;
  uint32_t token, last = WD_BINS, size = 0;
  // of rows that slots are for, those that found none go the same way as the others: which ones these are must not change a sum
  if (state == LEFT && n <= SA_PARTS && (l.top_k || !space.slots)) {
    uint32_t bar = NOTHING + 1, none = 0;
    for (int p = tid; p < n; p += RS_THREADS) bar = max(bar, parts[p].bar);
    g.most(bar, none);
    if (row.size <= SA_LIST) size = gather_row(g, row), bar = NOTHING + 1;
    else size = bar == ALL ? ALL : gather(g, parts, space.lists + r * space.per_row * PT_LIST, n, bar);
    if (size >= RS_THREADS && size <= SA_LIST && l.top_k && l.top_k <= size) size = shortened(ListSource<T>{s, size}, g, w, order_of(most), (uint32_t)l.top_k, bar);
    if (size < RS_THREADS) {
      const Picked some = pick(g, size, (uint32_t)l.top_k, l, w, bar, 0, whole);
      if (some.decided) {
        double before;
        const uint32_t thread = g.first(some.weight, [&](double sum, double total) { return sum > (double)l.uniform * total; }, before, all);
        if ((uint32_t)tid == thread) put_token(a, r, s.id[tid], some.weight, all);
        return;
      }
    } else if (size <= SA_LIST) {
      weigh(g, size, w);
      const ListSource<T> listed{s, size};
      Sampler<ListSource<T>, Group<RS_THREADS>> list{listed, w, g, s, order_of(most)};
      double by_mass = !l.by_mass ? -1 : l.top_k ? (double)l.top_p : target;
      bool decided = true;
      if (bar > NOTHING + 1) {
        // tokens below the bar are not there: none of them may be kept, or be needed for a sum
        const bool light = l.by_weight && w(logit_of(bar)) < min_p;
        if (l.top_k && size < l.top_k) {
          decided = light && !l.by_mass;
        } else if (l.by_mass && !l.top_k) {
          if (!(list.sum([](uint32_t) { return true; }) >= by_mass * (1 + 1e-12))) {
            decided = light;  // the nucleus goes below the bar, what min_p leaves does not
            by_mass = -1;
          }
        } else if (!l.top_k) {
          decided = light;
        }
      }
      if (decided) {
        token = s.id[list.draw(l, by_mass, mine, all)];
        if (tid == 0) put_token(a, r, token, mine, all);
        return;
      }
    }
    size = 0;
  }
  bool again = l.top_k || n > SA_PARTS;
  if (!again) {
    if (l.by_mass) {
      last = known.last;
      if (state == LEFT) {
        const double one = one_of((uint32_t)a.vocab);
        __syncthreads();
        for (int i = tid; i < WD_BINS; i += RS_THREADS) s.depth[i] = 0;
        __syncthreads();
        add_to_bins(row, 0, row.size, RS_THREADS, w, one, s.depth);
        __syncthreads();
        last = last_bin<WD_BINS / RS_THREADS>(s.depth, target * one, s.of_wave, &s.found);
      }
    }
    if (state == LEFT)
      for (int p = g.wave; p < n; p += g.WAVES) part_above(row, space, r * space.per_row + p, p, w, last, min_p);
    __syncthreads();  // a workgroup sees what it has written itself
    uint32_t longest = tid < n ? parts[tid].count : 0, none = 0;
    g.most(longest, none);
    again = longest > PT_LIST;  // too many tokens of the same depth
    if (!again) size = gather(g, parts, space.lists + r * space.per_row * PT_LIST, n, 0);
    again = again || size > SA_LIST;
  }
  if (again) {
    Sampler<RowSource<T>, Group<RS_THREADS>> whole_row{row, w, g, s, order_of(most)};
    token = whole_row.draw(l, !l.by_mass ? -1 : l.top_k ? (double)l.top_p : target, mine, all);
  } else {
    Kept kept{0, ALL, min_p};
    uint32_t until = ALL;  // as an id
    double sum = 0, before, some;
    if (tid < n) sum = parts[tid].kept;
    if (size) {
      const double above = g.sum(tid < n ? parts[tid].sum : 0.0);
      if (size < RS_THREADS) {
        const Picked some = pick(g, size, 0, l, w, 0, above, whole);
        kept.least = (uint32_t)(some.last >> 32), kept.until = ~(uint32_t)some.last;
      } else {
        weigh(g, size, w);
        const ListSource<T> in_bin{s, size};
        uint32_t largest = 0, none = 0;
        for (uint32_t i = tid; i < size; i += RS_THREADS) largest = max(largest, s.order[i]);
        g.most(largest, none);
        Sampler<ListSource<T>, Group<RS_THREADS>> list{in_bin, w, g, s, largest};
        kept = list.kept(l, __builtin_fmax(target - above, 0.0));
      }
      if (kept.until < size) until = s.id[kept.until];
      if (tid < n) {
        const uint32_t end = s.start[tid] + parts[tid].count;
#pragma unroll 1
        for (uint32_t k = s.start[tid]; k < end; ++k) sum += kept.of(s.order[k], [&] { return s.weight[k]; }, k);
      }
    }
    const uint32_t p = g.first(sum, [&](double upto, double total) { return upto > (double)l.uniform * total; }, before, all);
    const double goal = (double)l.uniform * all;
    token = locate(row, w, g, p * space.size, min((p + 1) * space.size, row.size), before,
                   [&](uint32_t o, auto weight, uint32_t id) {
                     const uint32_t b = bin_of(w, logit_of(o));
                     if (b > last || (b == last && (o < kept.least || (o == kept.least && id > until)))) return 0.0;
                     const double y = weight();
                     return y < min_p ? 0.0 : y;
                   },
                   [&](double) { return goal; }, mine, some);
  }
  if (tid == 0) put_token(a, r, token, mine, all);
}

// Steps of 512 tokens that a part has.  Calls of 2^23 logits and more fill the card with parts of 2,048, whose lists are few.  Below that
// smaller ones leave each wavefront less to do, as long as a row has at most 128 of them (more lists than that take longer to
// put together): of 1,024 tokens for 61 x 100,257 float16 with all limits 49 us instead of 54.5, for 60 x 60,000 without any 12.8 instead
// of 13.8; below 2^20 logits of 512 for one row of 50,256 24.4 instead of 31.5.
uint32_t part_steps(int64_t rows, int64_t vocab) {
  if (rows * vocab >= (int64_t)1 << 23 || vocab > 256 * PT_STEP) return 4;
  return rows * vocab < (int64_t)1 << 20 && vocab <= 128 * PT_STEP ? 1 : 2;
}

Space space_of(int64_t rows, int64_t vocab, void* at) {
  Space s{};
  s.size = part_steps(rows, vocab) * PT_STEP;
  s.per_row = std::max((vocab + s.size - 1) / s.size, (int64_t)1);
  const int64_t batch = std::min(rows, std::max(PT_BATCH / s.per_row, (int64_t)1)), parts = batch * s.per_row;
  // Many workgroups go over a row again, as many rows as there are slots, where it is too long to be listed whole: 61 x 100,257 with all
  // limits take 49 us so and 113 by one each, 256 x 262,144 110 and 256, a row of 50,256 with a wide nucleus 29 and 42; where no row is
  // left the launches cost 5.
  const bool wide = vocab > SA_LIST && s.per_row <= SA_PARTS;
  s.slots_taken = static_cast<uint32_t*>(at);
  s.rows = reinterpret_cast<Row*>(static_cast<char*>(at) + 16);
  s.parts = reinterpret_cast<Part*>(s.rows + batch);
  s.lists = reinterpret_cast<Listed*>(s.parts + parts);
  s.bytes = 16 + batch * (int64_t)sizeof(Row) + parts * (int64_t)(sizeof(Part) + PT_LIST * sizeof(Listed));
  if (wide) {
    s.slots = reinterpret_cast<Slot*>(s.lists + parts * PT_LIST);
    s.slot_count = (uint32_t)std::min(batch, (int64_t)WD_SLOTS);
    s.bytes += s.slot_count * (int64_t)sizeof(Slot);
  }
  return s;
}

template <class T>
void enqueue_sample(const tt_sample_args& a, hipStream_t st) {
  const Space space = space_of(a.rows, a.vocab, a.workspace);
  const int64_t batch = std::min(a.rows, std::max(PT_BATCH / space.per_row, (int64_t)1));
  for (int64_t r = 0; r < a.rows; r += batch) {
    tt_sample_args some = a;
    some.rows = std::min(batch, a.rows - r);
    some.logits = static_cast<const T*>(a.logits) + r * a.logits_stride;
    some.uniform += r, some.tokens += r;
    for (auto* p : {&some.temperature, &some.top_p, &some.min_p})
      if (*p) *p += r;
    if (some.top_k) some.top_k += r;
    if (some.logprobs) some.logprobs += r;
    constexpr int64_t waves = PT_THREADS / WAVE;
    auto* k = space.size == PT_STEP ? k_sample_parts<T, 1> : space.size == 2 * PT_STEP ? k_sample_parts<T, 2> : k_sample_parts<T, 4>;
    hipLaunchKernelGGL(k, dim3((uint32_t)((some.rows * space.per_row + waves - 1) / waves)), dim3(PT_THREADS), 0, st, some, space);
    hipLaunchKernelGGL(k_sample<T>, dim3((uint32_t)some.rows), dim3(DR_THREADS), 0, st, some, space);
    if (!a.top_k && !a.top_p && !a.min_p) continue;  // no row is left
    if (space.slots && (a.top_p || a.min_p)) {
      const int64_t items = std::min(some.rows, (int64_t)space.slot_count) * ((space.per_row + WD_SEGMENT - 1) / WD_SEGMENT);
      const dim3 grid((uint32_t)std::min(items, (int64_t)1024));
      hipLaunchKernelGGL(k_sample_bins<T>, grid, dim3(PT_THREADS), 0, st, some, space);
      hipLaunchKernelGGL(k_sample_above<T>, grid, dim3(PT_THREADS), 0, st, some, space);
    }
    hipLaunchKernelGGL(k_sample_rest<T>, dim3((uint32_t)some.rows), dim3(RS_THREADS), 0, st, some, space);
  }
}

}  // namespace

int64_t sample_workspace(int64_t rows, int64_t vocab) { return space_of(rows, vocab, nullptr).bytes; }

hipError_t launch_sample(const tt_sample_args& a, hipStream_t st) {
  if (a.type == TT_F32) enqueue_sample<float>(a, st);
  else if (a.type == TT_F16) enqueue_sample<_Float16>(a, st);
  else enqueue_sample<__bf16>(a, st);
  return hipGetLastError();
}

}  // namespace tt

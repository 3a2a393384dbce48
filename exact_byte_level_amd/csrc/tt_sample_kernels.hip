// tt_sample_kernels.hip -- the choice of the next token (declared in include/tt_step.h).
#include "tt_step_kernels.h"

#include <algorithm>
#include <type_traits>

namespace tt {
namespace {

constexpr int WAVE = 64;

typedef unsigned long long u64;

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

// 2^t for t from -1100 to 0: the nearest whole number apart, 1 + f p(f) on -1/2 .. 1/2 with p through the 9 Chebyshev
// nodes, off by less than 4e-14 of the value and exact at 0.
__device__ inline double power_of_two(double t) {
  const double n = __builtin_rint(t), f = t - n;
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
  return __builtin_ldexp(y, (int)n);
}

// Weights of a row: e^((x - top) / temperature).
struct Weigher {
  double top, by;  // by = log2 e / temperature
  bool endless;    // top is +infinity: everything below weighs nothing
  __device__ Weigher(float most, float temperature)
      : top(most), by(1.4426950408889634 / (double)temperature), endless(most == __builtin_inff()) {}
  __device__ double operator()(float x) const {
    // NaN, which -infinity gives where the temperature is infinite, becomes a weight of zero
    const double w = power_of_two(__builtin_fmax(((double)x - top) * by, -1100.0));
    return endless ? (x == __builtin_inff() ? 1.0 : 0.0) : w;
  }
};

// What is asked of a row.
struct Limits {
  float temperature, top_p, min_p, uniform;
  int64_t top_k;                     // 0: none
  bool single, by_mass, by_weight;   // the first token alone; top_p limits; min_p limits
  __device__ bool limited() const { return top_k || by_mass || by_weight; }
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
// A wavefront takes 2,048 logits into registers: their maximum, the sum of their weights by it, and, where the row has
// limits, a list of its largest ones, all that are not below a bar of its own.  What is above the highest of
// the bars is in the lists, so most rows need not be read again.

constexpr int PT_TOKENS = 2048;  // of a part
constexpr int PT_MINE = PT_TOKENS / WAVE;
constexpr int PT_LIST = 64;
constexpr int PT_THREADS = 256;
constexpr int64_t PT_BATCH = 65536;  // parts of a launch

struct Part {
  double sum;
  float most;
  uint32_t bar;    // the order down to which all tokens are listed
  uint32_t count;  // of the list
  uint32_t unused;
};
struct Listed {
  uint32_t order, id;
};

template <class T>
struct Eight {
  typedef T type __attribute__((ext_vector_type(8), aligned(alignof(T))));
};

template <class T>
__global__ __launch_bounds__(PT_THREADS) void k_sample_parts(tt_sample_args a, Part* parts, Listed* lists, int64_t per_row) {
  const int lane = threadIdx.x % WAVE;
  const int64_t id = (int64_t)blockIdx.x * (PT_THREADS / WAVE) + threadIdx.x / WAVE, r = id / per_row;
  if (r >= a.rows) return;
  const uint32_t vocab = (uint32_t)a.vocab, first = (uint32_t)(id - r * per_row) * PT_TOKENS;
  const T* row = static_cast<const T*>(a.logits) + r * a.logits_stride;
  float x[PT_MINE];
  if (first + PT_TOKENS <= vocab) {
    typename Eight<T>::type v[PT_MINE / 8];
#pragma unroll
    for (int q = 0; q < PT_MINE / 8; ++q) v[q] = *reinterpret_cast<const typename Eight<T>::type*>(row + first + q * 512 + lane * 8);
#pragma unroll
    for (int q = 0; q < PT_MINE / 8; ++q)
#pragma unroll
      for (int k = 0; k < 8; ++k) x[q * 8 + k] = (float)v[q][k];
  } else {
#pragma unroll
    for (int i = 0; i < PT_MINE; ++i) {
      const uint32_t v = first + i / 8 * 512 + lane * 8 + i % 8;
      x[i] = v < vocab ? (float)row[v] : -__builtin_inff();
    }
  }
  const Limits limits = limits_of(a, r);
  float mine = -__builtin_inff();  // the maximum passes over NaN
#pragma unroll
  for (int i = 0; i < PT_MINE; ++i) mine = fmaxf(mine, x[i]);
  float most = mine;
#pragma unroll
  for (int d = 1; d < WAVE; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
  Part part{0, most, NOTHING + 1, 0, 0};
  if (most > -__builtin_inff() && !limits.single) {
    const Weigher w(most, limits.temperature);
    double sum = 0;
#pragma unroll
    for (int i = 0; i < PT_MINE; ++i) sum += w(x[i]);
#pragma unroll
    for (int d = 1; d < WAVE; d *= 2) sum += __shfl_xor(sum, d);
    part.sum = sum;
    if (limits.limited()) {
      // The bar is the 32nd largest of the lanes' maxima, which about 64 ln 2 = 44 tokens are not below; of the largest
      // 16, 8, 4, 2, 1 where the list would not hold them.
      const uint32_t at_most = order_of(mine);
      uint32_t bar = 0, count = 0;
      for (int among = WAVE / 2; among; among /= 2) {
        bar = 0;
        for (uint32_t bit = 1u << 31; bit; bit >>= 1)
          if (__popcll(__ballot(at_most >= (bar | bit))) >= among) bar |= bit;
        bar = max(bar, NOTHING + 1);
        count = 0;
#pragma unroll
        for (int i = 0; i < PT_MINE; ++i) count += __popcll(__ballot(order_of(x[i]) >= bar));
        if (count <= PT_LIST) break;
        count = PT_LIST + 1;
      }
      if (count > PT_LIST) bar = 0xFFFFFFFFu, count = 0;
      part.bar = bar, part.count = count;
      if (count) {
        // places by ids: eight tokens of a lane, the lanes, the four steps; sums of at most 64 fit a byte each
        uint32_t counts = 0;
#pragma unroll
        for (int i = 0; i < PT_MINE; ++i) counts += (uint32_t)(order_of(x[i]) >= bar) << (i / 8 * 8);
        uint32_t upto = counts;
#pragma unroll
        for (int d = 1; d < WAVE; d *= 2) {
          const uint32_t other = __shfl_up(upto, d);
          if (lane >= d) upto += other;
        }
        const uint32_t all = __shfl(upto, WAVE - 1);
        uint32_t step = 0;
        Listed* to = lists + id * PT_LIST;
#pragma unroll
        for (int q = 0; q < PT_MINE / 8; ++q) {
          uint32_t at = step + ((upto - counts) >> (8 * q) & 255);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (order_of(x[q * 8 + k]) >= bar) to[at++] = Listed{order_of(x[q * 8 + k]), first + q * 512 + lane * 8 + k};
          step += all >> (8 * q) & 255;
        }
      }
    }
  }
  if (lane == 0) parts[id] = part;
}

// ---------------------------------------------------------- a row by a workgroup

constexpr int SA_THREADS = 1024;
constexpr int SA_WAVES = SA_THREADS / WAVE;
constexpr int SA_TILES = 1024;     // parts that a row is summed up in
constexpr int SA_STEP = WAVE * 8;  // tokens of a wavefront at a time
constexpr int SA_BINS = 2048;
constexpr int SA_LIST = 8192;      // tokens of the lists that are above all bars

struct SampleShared {
  union {
    u64 bin[SA_BINS];
    double tile[SA_TILES];
    uint32_t ties[SA_TILES];
  };
  double sum[SA_WAVES];
  u64 best[SA_WAVES];
  double above;
  uint32_t found, last, token;
  uint32_t order[SA_LIST], id[SA_LIST];
};

// Where the logits come from: a row in memory, or the tokens listed.  eight(at, end, f) calls f(logit, place, k) for the places
// from `at` on, eight at most.
template <class T>
struct RowSource {
  const T* row;
  uint32_t size;
  template <class F>
  __device__ void eight(uint32_t at, uint32_t end, F f) const {
    if (at + 8 <= end) {
      const auto x = *reinterpret_cast<const typename Eight<T>::type*>(row + at);
#pragma unroll
      for (int k = 0; k < 8; ++k) f((float)x[k], at + k, k);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (at + k < end) f((float)row[at + k], at + k, k);
    }
  }
};
struct ListSource {
  const uint32_t* order;
  uint32_t size;
  template <class F>
  __device__ void eight(uint32_t at, uint32_t end, F f) const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (at + k < end) f(logit_of(order[at + k]), at + k, k);
  }
};

template <class Source>
struct Sampler {
  const Source& source;
  SampleShared& s;
  int tid, lane, wave;

  // f(logit, place) for every token that the thread has.
  template <class F>
  __device__ void each(F f) {
    for (uint32_t at = tid * 8; at < source.size; at += SA_THREADS * 8) source.eight(at, source.size, f);
  }

  __device__ double sum_of(double x) {
#pragma unroll
    for (int d = 1; d < WAVE; d *= 2) x += __shfl_xor(x, d);
    if (lane == 0) s.sum[wave] = x;
    __syncthreads();
    x = 0;
    for (int w = 0; w < SA_WAVES; ++w) x += s.sum[w];
    __syncthreads();
    return x;
  }

  template <class V>
  __device__ V sums_upto(V x) {
#pragma unroll
    for (int d = 1; d < WAVE; d *= 2) {
      const V other = __shfl_up(x, d);
      if (lane >= d) x += other;
    }
    return x;
  }

  // The order at which, from the largest down to `least`, as many tokens (or as much weight) as `target` are reached,
  // digit by digit of 11, 11 and 10 bits; `above` receives how many (how much) there are above it.
  template <bool MASS>
  __device__ uint32_t reach(const Weigher& w, uint32_t least, double target, double scale, double& above) {
    const double unit = MASS ? 1 / scale : 1.0;
    uint32_t prefix = 0;
    above = 0;
    for (int shift = 21;; shift = shift == 21 ? 10 : 0) {
      const int bits = shift ? 11 : 10;
      for (int i = tid; i < SA_BINS; i += SA_THREADS) s.bin[i] = 0;
      if (tid == 0) s.found = s.last = 0;
      __syncthreads();
      each([&](float x, uint32_t, int) {
        const uint32_t o = order_of(x);
        if (o < least || (shift < 21 && o >> (shift + bits) != prefix)) return;
        // weights are summed in 64 bits of fixed point: in any order the same
        atomicAdd(&s.bin[o >> shift & ((1u << bits) - 1)], MASS ? (u64)__builtin_rint(w(x) * scale) : (u64)1);
      });
      __syncthreads();
      // bins from the largest down, two a thread
      const u64 mine[2] = {s.bin[SA_BINS - 1 - 2 * tid], s.bin[SA_BINS - 2 - 2 * tid]};
      const u64 upto = sums_upto(mine[0] + mine[1]);
      if (lane == WAVE - 1) s.best[wave] = upto;
      __syncthreads();
      u64 sum[3] = {upto - mine[0] - mine[1]};
      for (int k = 0; k < wave; ++k) sum[0] += s.best[k];
      sum[1] = sum[0] + mine[0], sum[2] = sum[1] + mine[1];
      uint32_t less = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        less += above + (double)sum[k + 1] * unit < target;
        if (mine[k]) atomicMax(&s.last, (uint32_t)(2 * tid + k));
      }
      if (less) atomicAdd(&s.found, less);
      __syncthreads();
      const uint32_t found = min(s.found, s.last);  // sums that are rounded may end just below the target
      if (found / 2 == (uint32_t)tid) s.above = above + (double)(found % 2 ? sum[1] : sum[0]) * unit;
      __syncthreads();
      above = s.above;
      prefix = prefix << bits | (SA_BINS - 1 - found);
      __syncthreads();
      if (!shift) return prefix;
    }
  }

  // Parts of the row, whole numbers of wavefronts' steps, one behind the other.
  __device__ uint32_t tile_size() const { return (source.size + SA_TILES * SA_STEP - 1) / (SA_TILES * SA_STEP) * SA_STEP; }

  // Tile t's sum of f(logit, id), put into `to`.
  template <class V, class F>
  __device__ void tile_sums(V* to, F f) {
    const uint32_t size = tile_size(), tiles = (source.size + size - 1) / size;
    for (uint32_t t = wave; t < SA_TILES; t += SA_WAVES) {
      V sum = 0;
      if (t < tiles) {
        const uint32_t end = min((t + 1) * size, source.size);
        for (uint32_t at = t * size + lane * 8; at < end; at += SA_STEP) source.eight(at, end, [&](float x, uint32_t id, int) { sum += f(x, id); });
#pragma unroll
        for (int d = 1; d < WAVE; d *= 2) sum += __shfl_xor(sum, d);
      }
      if (lane == 0) to[t] = sum;
    }
    __syncthreads();
  }

  // The first tile at which the running sum of the tiles' sums `of` passes goal(all of them), and the sum before it; the last
  // tile with a sum if none does.
  template <class V, class G>
  __device__ uint32_t passing(const V* of, G goal, V& before, V& total) {
    V* sums = reinterpret_cast<V*>(s.sum);
    const V mine = of[tid], upto = sums_upto(mine);
    if (lane == WAVE - 1) sums[wave] = upto;
    if (tid == 0) s.found = s.last = 0;
    __syncthreads();
    V sum = upto;
    total = 0;
    for (int k = 0; k < SA_WAVES; ++k) {
      if (k < wave) sum += sums[k];
      total += sums[k];
    }
    if (!(sum > goal(total))) atomicAdd(&s.found, 1u);
    if (mine > 0) atomicMax(&s.last, (uint32_t)tid);
    __syncthreads();
    const uint32_t found = min(s.found, s.last);
    if ((uint32_t)tid == found) reinterpret_cast<V*>(&s.above)[0] = sum - mine;
    __syncthreads();
    before = reinterpret_cast<V*>(&s.above)[0];
    __syncthreads();
    return found;
  }

  // The first token of tile t at which `before` and the running sum of f are above `goal`, the last one with a
  // weight if none is; by one wavefront.
  template <class V, class F>
  __device__ uint32_t token_passing(uint32_t t, V before, V goal, F f, V& mine, uint32_t size) {
    const uint32_t end = min((t + 1) * size, source.size);
    uint32_t last = t * size;
    mine = 0;
    for (uint32_t at = t * size; at < end; at += SA_STEP) {
      V x[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = 0;
      if (at + lane * 8 < end) source.eight(at + lane * 8, end, [&](float l, uint32_t id, int k) { x[k] = f(l, id); });
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += x[k];
      const V upto = sums_upto(sum);
      V run = before + (upto - sum);
      uint32_t hit = 8, some = 8;
      V of = 0, of_some = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        run += x[k];
        if (x[k] > 0) {
          some = k, of_some = x[k];
          if (hit == 8 && run > goal) hit = k, of = x[k];
        }
      }
      const u64 hits = __ballot(hit < 8), somes = __ballot(some < 8);
      if (hits) {
        const int l = __builtin_ctzll(hits);
        mine = __shfl(of, l);
        return at + l * 8 + __shfl(hit, l);
      }
      if (somes) {
        const int l = 63 - __builtin_clzll(somes);
        mine = __shfl(of_some, l);
        last = at + l * 8 + __shfl(some, l);
      }
      before += __shfl(upto, WAVE - 1);
    }
    return last;
  }

  // The token drawn, as its place, and what it and all that are kept weigh.  `sum`: what the tokens that top_k leaves weigh if it does
  // not limit.
  __device__ uint32_t draw(const Limits& l, const Weigher& w, double sum, double& mine, double& all) {
    // kept: orders above `least`, and of those at it the first `ties` (all of them if negative)
    uint32_t least = NOTHING + 1;
    double ties = -1, above;
    if (l.top_k) {
      const uint32_t o = reach<false>(w, 0, (double)l.top_k, 1.0, above);
      if (o > NOTHING) least = o, ties = (double)l.top_k - above;
      if (l.by_mass) {
        sum = 0;
        each([&](float x, uint32_t, int) { sum += order_of(x) > least || (ties < 0 && order_of(x) == least) ? w(x) : 0.0; });
        sum = sum_of(sum) + (ties > 0 ? ties * w(logit_of(least)) : 0.0);
      }
    }
    if (l.by_mass) {
      const double target = (double)l.top_p * sum, scale = __builtin_ldexp(1.0, 62 - (32 - __builtin_clz(source.size)));
      const uint32_t o = reach<true>(w, least, target, scale, above);
      above = 0;
      each([&](float x, uint32_t, int) { above += order_of(x) > o ? w(x) : 0.0; });
      above = sum_of(above);
      const double needed = __builtin_fmax(__builtin_ceil((target - above) / w(logit_of(o))), 1.0);
      ties = o == least && ties >= 0 ? __builtin_fmin(ties, needed) : needed;
      least = o;
    }
    uint32_t until = 0xFFFFFFFFu;  // the last place kept of those at `least`
    if (ties >= 0) {
      auto tie = [&](float x, uint32_t) { return (uint32_t)(order_of(x) == least); };
      tile_sums(s.ties, tie);
      const uint32_t goal = (uint32_t)__builtin_fmin(ties, 4e9) - 1;
      uint32_t before, total, one;
      const uint32_t tile = passing(s.ties, [&](uint32_t) { return goal; }, before, total);
      if (goal < total) until = token_passing(tile, before, goal, tie, one, tile_size());
      __syncthreads();
    }
    auto weight = [&](float x, uint32_t place) {
      const uint32_t o = order_of(x);
      if (o < least || (o == least && place > until)) return 0.0;
      const double y = w(x);
      return l.by_weight && y < (double)l.min_p ? 0.0 : y;
    };
    tile_sums(s.tile, weight);
    double before;
    const uint32_t tile = passing(s.tile, [&](double total) { return (double)l.uniform * total; }, before, all);
    const uint32_t token = token_passing(tile, before, (double)l.uniform * all, weight, mine, tile_size());
    __syncthreads();
    return token;
  }
};

// A row by a workgroup, from its parts.  Without limits the part that the random number falls into is read again; with limits
// the tokens listed decide if the last one kept is above all bars; else the row is passed over for every question.
template <class T>
__global__ __launch_bounds__(SA_THREADS) void k_sample(tt_sample_args a, const Part* parts, const Listed* lists, int64_t per_row) {
  __shared__ SampleShared s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % WAVE, wave = tid / WAVE;
  parts += r * per_row;
  lists += r * per_row * PT_LIST;
  const Limits l = limits_of(a, r);
  const int n = (int)per_row;
  const RowSource<T> whole{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab};
  Sampler<RowSource<T>> row{whole, s, tid, lane, wave};

  // the largest logit, and its first part
  u64 best = 0;
  uint32_t bar = NOTHING + 1;
  for (int p = tid; p < n; p += SA_THREADS) {
    best = max(best, (u64)order_of(parts[p].most) << 32 | ~(uint32_t)p);
    bar = max(bar, parts[p].bar);
  }
#pragma unroll
  for (int d = 1; d < WAVE; d *= 2) {
    best = max(best, __shfl_xor(best, d));
    bar = max(bar, __shfl_xor(bar, d));
  }
  if (lane == 0) s.best[wave] = best, s.ties[wave] = bar;
  __syncthreads();
  for (int w = 0; w < SA_WAVES; ++w) best = max(best, s.best[w]), bar = max(bar, s.ties[w]);
  __syncthreads();
  const float most = logit_of((uint32_t)(best >> 32));
  if (best >> 32 <= NOTHING) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logprobs) a.logprobs[r] = -__builtin_inff();
    }
    return;
  }
  if (l.single) {
    const uint32_t first = ~(uint32_t)best * PT_TOKENS, end = min(first + PT_TOKENS, whole.size);
    if (tid == 0) s.token = 0xFFFFFFFFu;
    __syncthreads();
    for (uint32_t v = first + tid; v < end; v += SA_THREADS)
      if (order_of((float)whole.row[v]) == best >> 32) atomicMin(&s.token, v);
    __syncthreads();
    if (tid == 0) {
      a.tokens[r] = (int32_t)s.token;
      if (a.logprobs) a.logprobs[r] = 0.0f;
    }
    return;
  }
  const Weigher w(most, l.temperature);
  auto weight_of = [&](int p) { return p < n && parts[p].sum > 0 ? parts[p].sum * w(parts[p].most) : 0.0; };
  double mine = 0, all = 0;
  uint32_t token;
  if (!l.limited() && n <= SA_TILES) {
    s.tile[tid] = weight_of(tid);
    __syncthreads();
    double before;
    const uint32_t part = row.passing(s.tile, [&](double sum) { return (double)l.uniform * sum; }, before, all);
    const RowSource<T> some{whole.row, min((part + 1) * (uint32_t)PT_TOKENS, whole.size)};
    Sampler<RowSource<T>> last{some, s, tid, lane, wave};
    token = last.token_passing(part, before, (double)l.uniform * all, [&](float x, uint32_t) { return w(x); }, mine, PT_TOKENS);
  } else {
    double sum = 0;
    for (int p = tid; p < n; p += SA_THREADS) sum += weight_of(p);
    sum = row.sum_of(sum);
    // what the lists hold above the bar, in the order of ids
    bool listed = l.limited() && n <= SA_TILES && bar != 0xFFFFFFFFu;
    uint32_t size = 0;
    if (listed) {
      for (int p = wave; p < SA_TILES; p += SA_WAVES) {
        const bool in = p < n && lane < (int)parts[p].count && lists[(int64_t)p * PT_LIST + lane].order >= bar;
        const uint32_t count = __popcll(__ballot(in));
        if (lane == 0) s.ties[p] = count;
      }
      __syncthreads();
      const uint32_t count = s.ties[tid], upto = row.sums_upto(count);
      if (lane == WAVE - 1) s.best[wave] = upto;
      __syncthreads();
      uint32_t at = upto - count;
      for (int k = 0; k < SA_WAVES; ++k) {
        if (k < wave) at += (uint32_t)s.best[k];
        size += (uint32_t)s.best[k];
      }
      s.ties[tid] = at;
      __syncthreads();
      listed = size <= SA_LIST;
      if (listed) {
        for (int p = wave; p < n; p += SA_WAVES) {
          const Listed entry = lane < (int)parts[p].count ? lists[(int64_t)p * PT_LIST + lane] : Listed{0, 0};
          const u64 in = __ballot(entry.order >= bar);
          const uint32_t to = s.ties[p] + __popcll(in & (((u64)1 << lane) - 1));
          if (entry.order >= bar) s.order[to] = entry.order, s.id[to] = entry.id;
        }
      }
      __syncthreads();
    }
    const ListSource top{s.order, size};
    Sampler<ListSource> short_list{top, s, tid, lane, wave};
    if (listed && bar > NOTHING + 1) {
      // tokens below the bar are not listed: none of them may be kept, or be needed for a sum
      const bool light = l.by_weight && w(logit_of(bar)) < (double)l.min_p;
      if (l.top_k && size < l.top_k) {
        listed = light && !l.by_mass;
      } else if (l.by_mass && !l.top_k) {
        double there = 0;
        short_list.each([&](float x, uint32_t, int) { there += w(x); });
        listed = short_list.sum_of(there) >= (double)l.top_p * sum * (1 + 1e-12);
      } else if (!l.top_k) {
        listed = light;
      }
    }
    if (listed) token = s.id[short_list.draw(l, w, sum, mine, all)];
    else token = row.draw(l, w, sum, mine, all);
  }
  if (tid == 0) {
    a.tokens[r] = (int32_t)token;
    if (a.logprobs) a.logprobs[r] = (float)log(mine / all);
  }
}

int64_t parts_of(int64_t vocab) { return std::max((vocab + PT_TOKENS - 1) / PT_TOKENS, (int64_t)1); }
int64_t batch_of(int64_t rows, int64_t vocab) { return std::min(rows, std::max(PT_BATCH / parts_of(vocab), (int64_t)1)); }

template <class T>
void enqueue_sample(const tt_sample_args& a, hipStream_t st) {
  const int64_t per_row = parts_of(a.vocab), batch = batch_of(a.rows, a.vocab);
  Part* parts = static_cast<Part*>(a.workspace);
  Listed* lists = reinterpret_cast<Listed*>(parts + batch * per_row);
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
    hipLaunchKernelGGL(k_sample_parts<T>, dim3((uint32_t)((some.rows * per_row + waves - 1) / waves)), dim3(PT_THREADS), 0, st, some, parts,
                       lists, per_row);
    hipLaunchKernelGGL(k_sample<T>, dim3((uint32_t)some.rows), dim3(SA_THREADS), 0, st, some, parts, lists, per_row);
  }
}

}  // namespace

int64_t sample_workspace(int64_t rows, int64_t vocab) {
  return batch_of(rows, vocab) * parts_of(vocab) * (int64_t)(sizeof(Part) + PT_LIST * sizeof(Listed));
}

hipError_t launch_sample(const tt_sample_args& a, hipStream_t st) {
  if (a.type == TT_F32) enqueue_sample<float>(a, st);
  else if (a.type == TT_F16) enqueue_sample<_Float16>(a, st);
  else enqueue_sample<__bf16>(a, st);
  return hipGetLastError();
}

}  // namespace tt

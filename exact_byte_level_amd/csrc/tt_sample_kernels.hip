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

// ---------------------------------------------------------- a row by a workgroup

constexpr int SA_THREADS = 1024;
constexpr int SA_WAVES = SA_THREADS / WAVE;
constexpr int SA_TILES = 1024;  // parts that a row is summed up in
constexpr int SA_STEP = WAVE * 8;  // tokens of a wavefront at a time
constexpr int SA_BINS = 2048;

template <class T>
struct Eight {
  typedef T type __attribute__((ext_vector_type(8), aligned(alignof(T))));
};

struct SampleShared {
  union {
    u64 bin[SA_BINS];
    double tile[SA_TILES];
    uint32_t ties[SA_TILES];
  };
  double sum[SA_WAVES];
  u64 best[SA_WAVES];
  double above;
  uint32_t found, last;
};

template <class T>
struct RowSampler {
  const T* row;
  uint32_t vocab;
  SampleShared& s;
  int tid, lane, wave;

  // f(logit, id) for every token that the thread has, eight at a time.
  template <class F>
  __device__ void each(F f) {
    for (uint32_t at = tid * 8; at < vocab; at += SA_THREADS * 8) eight(at, vocab, f);
  }
  template <class F>
  __device__ void eight(uint32_t at, uint32_t end, F f) {
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

  // The largest logit's order and its first token, as order and the inverted id.
  __device__ u64 best() {
    u64 most = 0;
    each([&](float x, uint32_t id, int) { most = max(most, (u64)order_of(x) << 32 | ~id); });
#pragma unroll
    for (int d = 1; d < WAVE; d *= 2) most = max(most, __shfl_xor(most, d));
    if (lane == 0) s.best[wave] = most;
    __syncthreads();
    for (int w = 0; w < SA_WAVES; ++w) most = max(most, s.best[w]);
    __syncthreads();
    return most;
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
  __device__ uint32_t tile_size() const { return (vocab + SA_TILES * SA_STEP - 1) / (SA_TILES * SA_STEP) * SA_STEP; }

  // Tile t's sum of f(logit, id), put into `to`.
  template <class V, class F>
  __device__ void tile_sums(V* to, F f) {
    const uint32_t size = tile_size(), tiles = (vocab + size - 1) / size;
    for (uint32_t t = wave; t < SA_TILES; t += SA_WAVES) {
      V sum = 0;
      if (t < tiles) {
        const uint32_t end = min((t + 1) * size, vocab);
        for (uint32_t at = t * size + lane * 8; at < end; at += SA_STEP) eight(at, end, [&](float x, uint32_t id, int) { sum += f(x, id); });
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
  __device__ uint32_t token_passing(uint32_t t, V before, V goal, F f, V& mine) {
    const uint32_t size = tile_size(), end = min((t + 1) * size, vocab);
    uint32_t last = t * size;
    mine = 0;
    for (uint32_t at = t * size; at < end; at += SA_STEP) {
      V x[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = 0;
      if (at + lane * 8 < end) eight(at + lane * 8, end, [&](float l, uint32_t id, int k) { x[k] = f(l, id); });
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
};

// A row by a workgroup, passing over it for every question: where the top tokens end, what they weigh, where the nucleus ends,
// which token.
template <class T>
__global__ __launch_bounds__(SA_THREADS) void k_sample(tt_sample_args a) {
  __shared__ SampleShared s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  RowSampler<T> row{static_cast<const T*>(a.logits) + r * a.logits_stride, (uint32_t)a.vocab, s, tid, tid % WAVE, tid / WAVE};
  const float temperature = a.temperature ? a.temperature[r] : 1.0f, given = a.uniform[r];
  const float top_p = a.top_p ? a.top_p[r] : 1.0f, min_p = a.min_p ? a.min_p[r] : 0.0f;
  const int top_k = a.top_k ? a.top_k[r] : 0;
  const float uniform = given >= 1.0f ? 0x1.fffffep-1f : given > 0.0f ? given : 0.0f;
  const u64 best = row.best();
  const uint32_t most = (uint32_t)(best >> 32);
  if (most <= NOTHING) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logprobs) a.logprobs[r] = -__builtin_inff();
    }
    return;
  }
  if (!(temperature > 0.0f) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {  // the first token alone
    if (tid == 0) {
      a.tokens[r] = (int32_t)~(uint32_t)best;
      if (a.logprobs) a.logprobs[r] = 0.0f;
    }
    return;
  }
  const Weigher w(logit_of(most), temperature);
  // kept: orders above `least`, and of those at it the first `ties` (all of them if negative)
  uint32_t least = NOTHING + 1;
  double ties = -1, above;
  if (top_k > 0 && top_k < (int64_t)row.vocab) {
    const uint32_t o = row.template reach<false>(w, 0, top_k, 1.0, above);
    if (o > NOTHING) least = o, ties = top_k - above;
  }
  if (top_p < 1.0f) {
    const double sum = row.sum_of([&] {
      double sum = 0;
      row.each([&](float x, uint32_t, int) { sum += order_of(x) > least || (ties < 0 && order_of(x) == least) ? w(x) : 0.0; });
      return sum;
    }());
    const double target = (double)top_p * (sum + (ties > 0 ? ties * w(logit_of(least)) : 0.0));
    const double scale = __builtin_ldexp(1.0, 62 - (32 - __builtin_clz(row.vocab)));
    const uint32_t o = row.template reach<true>(w, least, target, scale, above);
    above = row.sum_of([&] {
      double sum = 0;
      row.each([&](float x, uint32_t, int) { sum += order_of(x) > o ? w(x) : 0.0; });
      return sum;
    }());
    const double needed = __builtin_fmax(__builtin_ceil((target - above) / w(logit_of(o))), 1.0);
    ties = o == least && ties >= 0 ? __builtin_fmin(ties, needed) : needed;
    least = o;
  }
  uint32_t until = 0xFFFFFFFFu;  // the last token kept of those at `least`
  if (ties >= 0) {
    row.tile_sums(s.ties, [&](float x, uint32_t) { return (uint32_t)(order_of(x) == least); });
    const uint32_t goal = (uint32_t)__builtin_fmin(ties, 4e9) - 1;
    uint32_t before, all;
    const uint32_t tile = row.passing(s.ties, [&](uint32_t) { return goal; }, before, all);
    if (goal < all) {
      uint32_t one;
      until = row.token_passing(tile, before, goal, [&](float x, uint32_t) { return (uint32_t)(order_of(x) == least); }, one);
    }
    __syncthreads();
  }
  auto weight = [&](float x, uint32_t id) {
    const uint32_t o = order_of(x);
    if (o < least || (o == least && id > until)) return 0.0;
    const double y = w(x);
    return min_p > 0.0f && y < (double)min_p ? 0.0 : y;
  };
  row.tile_sums(s.tile, weight);
  double before, all, mine;
  const uint32_t tile = row.passing(s.tile, [&](double sum) { return (double)uniform * sum; }, before, all);
  if (row.wave == 0) {
    const uint32_t token = row.token_passing(tile, before, (double)uniform * all, weight, mine);
    if (tid == 0) {
      a.tokens[r] = (int32_t)token;
      if (a.logprobs) a.logprobs[r] = (float)log(mine / all);
    }
  }
}

}  // namespace

int64_t sample_workspace(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const tt_sample_args& a, hipStream_t st) {
  auto* k = a.type == TT_F32 ? k_sample<float> : a.type == TT_F16 ? k_sample<_Float16> : k_sample<__bf16>;
  constexpr int64_t most = 0xFFFFFFFF / SA_THREADS;
  for (int64_t r = 0; r < a.rows; r += most) {
    tt_sample_args part = a;
    part.logits = static_cast<const char*>(a.logits) + r * a.logits_stride * (a.type == TT_F32 ? 4 : 2);
    part.uniform += r, part.tokens += r;
    for (auto* p : {&part.temperature, &part.top_p, &part.min_p})
      if (*p) *p += r;
    if (part.top_k) part.top_k += r;
    if (part.logprobs) part.logprobs += r;
    hipLaunchKernelGGL(k, dim3((uint32_t)std::min(most, a.rows - r)), dim3(SA_THREADS), 0, st, part);
  }
  return hipGetLastError();
}

}  // namespace tt

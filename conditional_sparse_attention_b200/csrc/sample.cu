// A token per row of logits from a given uniform number: temperature, top-k, top-p and min-p.
//
// One cluster of up to 8 CTAs works on a row.  The row is read from HBM once, into the shared memory of
// its cluster (a contiguous segment per CTA), and every later pass runs from there.
//
//   1. the maximum (and for a greedy row its lowest index)
//   2. one pass for the mass of all weights (where top-p or an unfiltered draw needs it), and for a
//      histogram of every eighth value over the distance d = (max - l) / T
//   3. with a filter on: the distance within which the sample tells of some 700 values; those values (at
//      most 1024) go to CTA 0 in index order, which finds the cut by count and by mass (16 thresholds a
//      round, one a warp), drops by min-p and draws, while the other CTAs leave
//   4. where those do not reach the cut (flat or wide filters): a histogram over d in 1024 bins of 1/32,
//      counts and masses, gives the bin of the cut, whose values CTA 0 sorts; a fuller bin is cut again
//      by the bits of the values, and one of equal values by their index
//   5. without a list: the masses of the survivors, a prefix over warps and CTAs, and the element at
//      u * mass
//
// Weights e^-d are computed in fp64 (table of 2^(j/64) and a Taylor polynomial of degree 4, relative
// error below 5e-14) and held as whole multiples of 2^-43 of the largest weight: sums of whole numbers do not
// depend on their order, so neither atomics nor the cluster's shape can change a token.  A row of
// ODA_MAX_VOCAB = 2^18 weights sums to at most 2^61.
//
// Bound: HBM for the row, then the fp64 pipe (some 12 operations a weight at 64 lanes a clock and SM)
// and, for few rows, the latency of the cluster's barriers.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace oda {
namespace {

constexpr int kT = 512;                  // threads of a CTA
constexpr int kWarps = kT / 32;
constexpr int kMaxC = 8;                 // CTAs of a cluster
constexpr int kBins = 1024;
constexpr int kList = 1024;
constexpr int kSeg = 5120;               // values of a CTA above which the cluster grows
constexpr int kFrac = 43;                // weights are multiples of 2^-43
constexpr int kCoarse = 128;              // bins of 1/8 of the sampled histogram
constexpr int kWant = 700;               // listed values aimed at
constexpr float kNear = 6.f;             // distance from which on a total mass is summed in fp32

struct SampleParams {
  const float* logits;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* prob;
  int64_t row_stride;
  int vocab, seg;                        // seg: values of a CTA, a multiple of 4
};

struct Exchange {
  unsigned long long a, b;
  uint32_t c, d;
};

struct Shared {
  double pow64[64];                      // 2^(j/64)
  uint32_t coarse[kCoarse];
  Exchange ex[2];
  unsigned long long w64[kWarps];
  uint32_t w32[kWarps];
  uint32_t wk[kWarps];
  Exchange found;
  uint32_t n_list;
};

// (ln 2 / 64)^i / i!: 2^(r/64) = sum of these times r^i; |r| <= 1/2, so the next term is below 4e-14
constexpr double kL = 0.69314718055994530942 / 64.0;
constexpr double kC2 = kL * kL / 2, kC3 = kL * kL * kL / 6, kC4 = kL * kL * kL * kL / 24;

// Weight e^((l - max)/T) of logit l, and as a whole multiple of 2^-kFrac; s = 64 log2(e) / T.  No branch, so
// that the weights of a loop run abreast; -inf gives 0.
__device__ __forceinline__ unsigned long long weight(const Shared& sm, float l, double max, double s, double* w) {
  const double y0 = ((double)l - max) * s;              // <= 0, -inf, or NaN (0 * inf: the maximum itself)
  const bool in = !(y0 <= -64.0 * (kFrac + 1)) && l > -INFINITY;   // below half a step the weight is 0
  const double y = in && y0 == y0 ? y0 : 0.0;
  const double t = y + 6755399441055744.0;              // 1.5 * 2^52: rounds to a whole number, in the low bits
  const double r = y - (t - 6755399441055744.0);
  const int k = (int)__double_as_longlong(t);
  double e = fma(fma(fma(fma(kC4, r, kC3), r, kC2), r, kL), r, 1.0) * sm.pow64[k & 63];
  e = __longlong_as_double(__double_as_longlong(e) + ((long long)(k >> 6) << 52));
  *w = in ? e : 0.0;
  // e * 2^kFrac <= 2^kFrac: adding 2^52 leaves its nearest whole number in the low bits
  const unsigned long long W = (unsigned long long)__double_as_longlong(fma(e, (double)(1ll << kFrac), 4503599627370496.0)) -
                               0x4330000000000000ull;
  return in ? W : 0ull;
}

__device__ __forceinline__ uint32_t key_of(float x) {   // order-preserving
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kMasked = 0x007fffffu;               // key of -inf

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <class T>
__device__ __forceinline__ T warp_scan(T v, int lane) { // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Sorts the first m of a CTA's list ascending (what fills it up to a power of two goes behind).  Not
// inlined, like all that a row runs once: the kernel's time for few rows is its instruction fetch.
__device__ __noinline__ void sort_list(unsigned long long* list, int m) {
  const int tid = threadIdx.x;
  int p2 = 2;
  while (p2 < m) p2 <<= 1;
  for (int i = m + tid; i < p2; i += kT) list[i] = ~0ull;
#pragma unroll 1
  for (int k = 2; k <= p2; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < p2 / 2; i += kT) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const unsigned long long u = list[a], v = list[b];
        if ((u > v) == ((a & k) == 0)) list[a] = v, list[b] = u;
      }
    }
  __syncthreads();
}

// Masses of list entries 2 tid and 2 tid + 1 of m (0 below mpd or behind m), of all before them, and of all;
// an entry's key is its inverted high word (`high`) or its low word.
struct Scan {
  unsigned long long before, w0, w1, all;
};
__device__ __noinline__ Scan scan_list(Shared& sm, const unsigned long long* list, int m, bool high, double mpd,
                                       double dmax, double s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned long long W[2];
#pragma unroll 1
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    unsigned long long w = 0;
    if (i < m) {
      double x;
      w = weight(sm, of_key(high ? ~(uint32_t)(list[i] >> 32) : (uint32_t)list[i]), dmax, s, &x);
      if (x < mpd) w = 0;
    }
    if (j) W[1] = w;
    else W[0] = w;
  }
  const unsigned long long ws = warp_scan(W[0] + W[1], lane);
  __syncthreads();
  if (lane == 31) sm.w64[warp] = ws;
  __syncthreads();
  const unsigned long long v = lane < kWarps ? sm.w64[lane] : 0ull;
  return {ws - (W[0] + W[1]) + warp_sum(lane < warp ? v : 0ull), W[0], W[1], warp_sum(v)};
}

// The elements kept so far: key > cut, or key == cut and place <= at.
struct Cut {
  uint32_t key;
  int at;
};

  // CTA 0: the last element of the shortest prefix (largest first, ties by place) of the m listed values
  // whose count or mass is >= target, and the mass of that prefix.  Every round, each warp takes one
  // of 16 thresholds of the range that is left.
  struct CutMass {
  Cut cut;
  unsigned long long mass;
};
__device__ __noinline__ CutMass cut_list(Shared& sm, const uint32_t* key, int m, bool by_count, unsigned long long target) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t* place = key + kList;
    const unsigned long long* W = reinterpret_cast<const unsigned long long*>(key + 2 * kList);
    uint32_t a = 0xffffffffu, b = 0;
    for (int i = lane; i < m; i += 32) a = min(a, key[i]), b = max(b, key[i]);
    uint32_t lo = __reduce_min_sync(0xffffffffu, a), hi = __reduce_max_sync(0xffffffffu, b) + 1u;
    // sum(key >= lo) reaches the target, sum(key >= hi) does not
#pragma unroll 1
    while (hi - lo > 1u) {
      const uint32_t step = (uint32_t)(((unsigned long long)(hi - lo) + kWarps) / (kWarps + 1));
      const uint32_t mine = lo + step * (uint32_t)(warp + 1);
      unsigned long long f = 0;
#pragma unroll 4
      for (int i = lane; i < m; i += 32)
        if (key[i] >= mine) f += by_count ? 1ull : W[i];
      f = warp_sum(f);
      __syncthreads();
      if (lane == 0) sm.w32[warp] = mine < hi && mine > lo && f >= target;
      __syncthreads();
      const uint32_t ok = __ballot_sync(0xffffffffu, lane < kWarps && sm.w32[lane]);
      const int n_ok = __popc(ok);       // thresholds rise with the warp: the first n_ok hold
      const uint32_t base = lo;
      lo = base + step * (uint32_t)n_ok;
      hi = min(hi, base + step * (uint32_t)(n_ok + 1));
    }
    // values equal to lo, in index order: how many of them, and the last one's place (every warp by itself)
    unsigned long long above = 0, mass = 0, one = 0;
    for (int i = lane; i < m; i += 32) {
      if (key[i] > lo) above += by_count ? 1ull : W[i], mass += W[i];
      if (key[i] == lo) one = W[i];
    }
    above = warp_sum(above);
    mass = warp_sum(mass);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) one = max(one, __shfl_xor_sync(0xffffffffu, one, o));
    const unsigned long long need = max(1ull, by_count ? target - above : (target - above + one - 1) / max(1ull, one));
    unsigned long long seen = 0;
    int at = 0x7fffffff;
    for (int i0 = 0; i0 < m; i0 += 32) {
      const uint32_t here = __ballot_sync(0xffffffffu, i0 + lane < m && key[i0 + lane] == lo);
      if (seen + __popc(here) >= need) {
        const bool it = ((here >> lane) & 1u) && seen + __popc(here & ((1u << lane) - 1u)) + 1 == need;
        at = (int)place[i0 + __ffs((int)__ballot_sync(0xffffffffu, it)) - 1];
        break;
      }
      seen += __popc(here);
    }
    return {{lo, at}, mass + need * one};
  }

struct Row {                             // a CTA's view of its row
  Shared& sm;
  float* x;                              // its segment
  uint32_t* cnt;                         // [kBins]
  uint32_t* lo;                          // [kBins] mass, low and high words
  uint32_t* hi;
  unsigned long long* list;              // [kList] (~key, place)
  int e0, n;                             // place of x[0] in the row; values here
  int C, rank, tid, lane, warp;
  int turn;                              // of the exchange buffers
  int per;                               // values of a warp's contiguous part
  float lmax;
  float inv_t;
  double s, dmax;                        // 64 log2(e) / T, the maximum

  __device__ Exchange& remote(int r, int t) { return cg::this_cluster().map_shared_rank(&sm, r)->ex[t]; }

  // Every CTA's thread 0 gives `mine`; returns after all CTAs' values can be read with remote(r, t).
  __device__ int exchange(const Exchange& mine) {
    const int t = turn;
    turn ^= 1;
    if (tid == 0) sm.ex[t] = mine;
    cg::this_cluster().sync();
    return t;
  }

  // The CTAs' values, one lane each (0 beyond the cluster's size): field by field, then sums or maxima.
  __device__ unsigned long long sum_a(int t) { return warp_sum(lane < C ? remote(lane, t).a : 0ull); }
  __device__ uint32_t sum_c(int t) { return __reduce_add_sync(0xffffffffu, lane < C ? remote(lane, t).c : 0u); }

  __device__ float distance(float l) const { return (lmax - l) * inv_t; }

  // Mass of this warp's values: all in fp64, or, `rough`, those beyond kNear in fp32 (in a fixed order).
  // The rough one serves as top-p's total: beyond kNear a weight is below 2^-8.6, and the relative error
  // of their sum (2^-22 a weight, averaged over thousands) is far below what moves a cut.
  __device__ unsigned long long warp_mass(bool rough) const {
    const int a = min(n, warp * per), e = min(n, a + per);
    unsigned long long m = 0;
    double w;
    if (!rough) {
#pragma unroll 4
      for (int i = a + lane; i < e; i += 32) m += weight(sm, x[i], dmax, s, &w);
    } else {
      const float c = inv_t * 1.4426950408889634f;
      float far = 0.f;
#pragma unroll 4
      for (int i = a + lane; i < e; i += 32) {
        const float l = x[i];
        if (distance(l) < kNear) m += weight(sm, l, dmax, s, &w);
        else far += exp2f((l - lmax) * c);
      }
      if (far == far) m += (unsigned long long)__double2ll_rn((double)far * (double)(1ll << kFrac));
    }
    return warp_sum(m);
  }

  // Histogram of every eighth 32 values into the CTA's coarse bins.
  __device__ void sample_distances() {
    const int a = min(n, warp * per), e = min(n, a + per);
#pragma unroll 1
    for (int i = a + lane; i < e; i += 256) {
      const float d = distance(x[i]);
      if (d < kCoarse * 0.125f) atomicAdd(&sm.coarse[(int)(d * 8.f)], 1u);
    }
  }

  __device__ int bin0(float l) const { return min(kBins - 1, (int)((lmax - l) * inv_t * 32.f)); }

  __device__ void add(int b, float l, bool mass) {
    atomicAdd(&cnt[b], 1u);
    if (!mass) return;
    double w;
    const unsigned long long W = weight(sm, l, dmax, s, &w);
    const uint32_t low = (uint32_t)W, high = (uint32_t)(W >> 32);
    if (W == 0) return;
    const uint32_t old = atomicAdd(&lo[b], low);
    const uint32_t up = high + (old + low < old ? 1u : 0u);
    if (up) atomicAdd(&hi[b], up);
  }

  // Histogram of the unmasked values: by bin0, or of keys in [kmin, kmax] by (kmax - key) >> shift.
  __device__ __noinline__ void histogram(bool first, uint32_t kmin, uint32_t kmax, int shift, bool mass) {
    __syncthreads();
    for (int i = tid; i < kBins; i += kT) cnt[i] = lo[i] = hi[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kT) {
      const float l = x[i];
      const uint32_t k = key_of(l);
      if (k == kMasked) continue;
      if (first) add(bin0(l), l, mass);
      else if (k >= kmin && k <= kmax) add((int)((kmax - k) >> shift), l, mass);
    }
    cg::this_cluster().sync();
  }

  // First bin at which the running count (by_count) or mass, on top of (ca, ma), reaches `target`.
  struct Hit {
    unsigned long long mass_above;
    uint32_t count_above, bin, count;    // values above the bin, and in it
  };
  __device__ __noinline__ Hit cross(bool by_count, unsigned long long target, uint32_t ca, unsigned long long ma) {
    // this CTA's share of the bins, summed over the cluster
    const int nb = kBins / C, each = (nb + kT - 1) / kT;
    const int b0 = rank * nb + tid * each;
    uint32_t c[2] = {0, 0};
    unsigned long long m[2] = {0, 0};
    if (tid * each < nb)
      for (int j = 0; j < each; ++j)
#pragma unroll
        for (int r = 0; r < kMaxC; ++r) {
          if (r >= C) continue;
          auto cl = cg::this_cluster();
          c[j] += cl.map_shared_rank(cnt, r)[b0 + j];
          m[j] += (unsigned long long)cl.map_shared_rank(lo, r)[b0 + j] +
                  ((unsigned long long)cl.map_shared_rank(hi, r)[b0 + j] << 32);
        }
    const uint32_t cs = warp_scan(c[0] + c[1], lane);
    const unsigned long long ms = warp_scan(m[0] + m[1], lane);
    __syncthreads();
    if (lane == 31) {
      sm.w32[warp] = cs;
      sm.w64[warp] = ms;
    }
    __syncthreads();
    uint32_t cb = cs - (c[0] + c[1]), ct = 0;
    unsigned long long mb = ms - (m[0] + m[1]), mt = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) cb += sm.w32[w], mb += sm.w64[w];
      ct += sm.w32[w], mt += sm.w64[w];
    }
    int t = exchange({mt, 0, ct, 0});
    cb += ca;
    mb += ma;
    for (int r = 0; r < rank; ++r) cb += remote(r, t).c, mb += remote(r, t).a;
    if (tid == 0) sm.found = {};
    __syncthreads();
    for (int j = 0; j < each; ++j) {
      const bool before = by_count ? cb < target : mb < target;
      const bool after = by_count ? cb + c[j] >= target : mb + m[j] >= target;
      if (before && after) sm.found = {mb, (unsigned long long)c[j], cb, (uint32_t)(b0 + j) + 1u};
      cb += c[j];
      mb += m[j];
    }
    __syncthreads();
    t = exchange(sm.found);
    Hit h = {0, 0, 0, 0};
    for (int r = 0; r < C; ++r) {
      const Exchange e = remote(r, t);
      if (e.d) h = {e.a, e.c, e.d - 1u, (uint32_t)e.b};
    }
    return h;
  }

  // Place of the m-th (from 1) value with key k, in index order.
  __device__ __noinline__ int nth_equal(uint32_t k, uint32_t m) {
    const int a = min(n, warp * per), e = min(n, a + per);
    uint32_t c = 0;
    for (int i = a + lane; i < e; i += 32) c += key_of(x[i]) == k;
    c = warp_sum(c);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = c;
    if (tid == 0) sm.found = {};
    __syncthreads();
    uint32_t before = 0, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm.w32[w];
      total += sm.w32[w];
    }
    int t = exchange({0, 0, total, 0});
    for (int r = 0; r < rank; ++r) before += remote(r, t).c;
    if (before < m && m <= before + c)
      for (int i = a; i < e; i += 32) {
        const uint32_t here = __ballot_sync(0xffffffffu, i + lane < e && key_of(x[i + lane]) == k);
        if (before + __popc(here) >= m) {
          if (lane == 0) sm.found = {0, 0, (uint32_t)(e0 + i + (int)__fns(here, 0, (int)(m - before))), 1};
          break;
        }
        before += __popc(here);
      }
    __syncthreads();
    t = exchange(sm.found);
    int at = 0;
    for (int r = 0; r < C; ++r)
      if (remote(r, t).d) at = (int)remote(r, t).c;
    return at;
  }

  // Number and mass of this warp's values nearer than `far`.
  __device__ uint32_t near_count(float far, unsigned long long* mass) const {
    const int a = min(n, warp * per), e = min(n, a + per);
    uint32_t c = 0;
    unsigned long long m = 0;
#pragma unroll 4
    for (int i = a + lane; i < e; i += 32) {
      const float l = x[i];
      if (distance(l) < far) {
        double w;
        ++c;
        m += weight(sm, l, dmax, s, &w);
      }
    }
    *mass = warp_sum(m);
    return __reduce_add_sync(0xffffffffu, c);
  }

  // This warp's `c` values nearer than `far` to place `at` on of CTA 0's key and place arrays, in index order.
  __device__ void gather(float far, uint32_t at, uint32_t c) {
    uint32_t* key = cg::this_cluster().map_shared_rank(cnt, 0);
    uint32_t* place = key + kList;
    const int a = min(n, warp * per), e = min(n, a + per);
    const uint32_t stop = at + c;
#pragma unroll 1
    for (int i0 = a; i0 < e && at < stop; i0 += 32) {
      const int i = i0 + lane;
      const float l = i < e ? x[i] : -INFINITY;
      const bool in = i < e && distance(l) < far;
      const uint32_t here = __ballot_sync(0xffffffffu, in);
      const uint32_t to = at + __popc(here & ((1u << lane) - 1u));
      if (in && to < (uint32_t)kList) key[to] = key_of(l), place[to] = (uint32_t)(e0 + i);
      at += __popc(here);
    }
  }

  // CTA 0 draws from the m listed values, which hold every cut (`mass`: top-p's total without top-k).
  __device__ void draw_list(int m, int kk, float tp, float mp, unsigned long long mass, float u, int* token, float* prob) {
    const bool by_p = tp < 1.f;
    const uint32_t* key = cnt;
    const uint32_t* place = cnt + kList;
    unsigned long long* W = reinterpret_cast<unsigned long long*>(cnt + 2 * kList);
    const double mpd = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
    uint32_t drop = 0;                     // bit j: this thread's j-th value is below min_p
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * tid + j;
      if (i < m) {
        double w;
        const unsigned long long v = weight(sm, of_key(key[i]), dmax, s, &w);
        W[i] = v;
        if (w < mpd) drop |= 1u << j;
      }
    }
    __syncthreads();
    Cut cut = {0, 0x7fffffff};
    if (kk > 0) {
      const CutMass c = cut_list(sm, cnt, m, true, (unsigned long long)kk);
      cut = c.cut;
      mass = c.mass;
    }
    if (by_p) {
      const double want = tp > 0.f ? ceil((double)tp * (double)mass) : 1.0;
      const unsigned long long target = max(1ull, min((unsigned long long)want, mass));
      cut = cut_list(sm, cnt, m, false, target).cut;
    }
    // the survivors' masses in index order
    unsigned long long w0 = 0, w1 = 0;
    {
      const int i = 2 * tid;
      if (i < m && !(drop & 1) && (key[i] > cut.key || (key[i] == cut.key && (int)place[i] <= cut.at))) w0 = W[i];
      if (i + 1 < m && !(drop & 2) && (key[i + 1] > cut.key || (key[i + 1] == cut.key && (int)place[i + 1] <= cut.at)))
        w1 = W[i + 1];
    }
    const unsigned long long ws = warp_scan(w0 + w1, lane);
    __syncthreads();
    if (lane == 31) sm.w64[warp] = ws;
    __syncthreads();
    const unsigned long long v = lane < kWarps ? sm.w64[lane] : 0ull;
    const unsigned long long before = ws - (w0 + w1) + warp_sum(lane < warp ? v : 0ull), total = warp_sum(v);
    const unsigned long long want = min((unsigned long long)((double)u * (double)total), total - 1);
    if (before <= want && want < before + w0 + w1) {
      const bool second = want >= before + w0;
      *token = (int)place[2 * tid + (second ? 1 : 0)];
      *prob = (float)((double)(second ? w1 : w0) / (double)total);
    }
  }

  // The shortest prefix (largest first, ties by place) of count >= target or mass >= target; its last
  // element, and its mass (0 where masses are not kept).  fresh: the level-0 histogram is in place.
  __device__ __noinline__ Cut search(bool by_count, unsigned long long target, bool mass, bool& fresh, unsigned long long* total) {
    if (!fresh) histogram(true, 0, 0, 0, mass);
    fresh = true;
    Hit h = cross(by_count, target, 0, 0);
    uint32_t kmin = 0, kmax = 0;
    bool level0 = true;
    int shift = 0;
    uint32_t top = 0;                    // kmax of the level that h.bin belongs to
    while (true) {
      // the bin's elements: bin0 == h.bin, or (top - key) >> shift == h.bin
      if (h.count <= kList) break;
      uint32_t a = 0xffffffffu, b = 0;
      for (int i = tid; i < n; i += kT) {
        const uint32_t k = key_of(x[i]);
        if (k == kMasked) continue;
        const bool in = level0 ? bin0(x[i]) == (int)h.bin : (k >= kmin && k <= top && ((top - k) >> shift) == h.bin);
        if (in) a = min(a, k), b = max(b, k);
      }
      a = __reduce_min_sync(0xffffffffu, a);
      b = __reduce_max_sync(0xffffffffu, b);
      __syncthreads();
      if (lane == 0) sm.w32[warp] = a, sm.wk[warp] = b;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) a = min(a, sm.w32[w]), b = max(b, sm.wk[w]);
      const int t = exchange({0, 0, a, b});
      for (int r = 0; r < C; ++r) a = min(a, remote(r, t).c), b = max(b, remote(r, t).d);
      kmin = a;
      kmax = b;
      if (kmin == kmax) {                // equal values: cut by index
        double w;
        const unsigned long long W = weight(sm, of_key(kmin), dmax, s, &w);
        unsigned long long m = by_count ? target - h.count_above : (target - h.mass_above + W - 1) / (W ? W : 1);
        m = max(1ull, min(m, (unsigned long long)h.count));
        *total = h.mass_above + m * W;
        return {kmin, nth_equal(kmin, (uint32_t)m)};
      }
      level0 = false;
      top = kmax;
      shift = 0;
      while (((kmax - kmin) >> shift) >= (uint32_t)kBins) ++shift;
      fresh = false;
      histogram(false, kmin, kmax, shift, mass);
      h = cross(by_count, target, h.count_above, h.mass_above);
    }
    // gather into CTA 0
    if (tid == 0) sm.n_list = 0;
    cg::this_cluster().sync();
    {
      Shared* s0 = cg::this_cluster().map_shared_rank(&sm, 0);
      unsigned long long* l0 = cg::this_cluster().map_shared_rank(list, 0);
      for (int i = tid; i < n; i += kT) {
        const uint32_t k = key_of(x[i]);
        if (k == kMasked) continue;
        const bool in = level0 ? bin0(x[i]) == (int)h.bin : (k >= kmin && k <= top && ((top - k) >> shift) == h.bin);
        if (in) {
          const uint32_t at = atomicAdd(&s0->n_list, 1u);
          if (at < (uint32_t)kList) l0[at] = ((unsigned long long)~k << 32) | (uint32_t)(e0 + i);
        }
      }
    }
    cg::this_cluster().sync();
    if (rank == 0) {
      const int m = min((int)sm.n_list, kList);
      sort_list(list, m);
      // running mass and count over the sorted list
      if (tid == 0) sm.found = {};
      const Scan sc = scan_list(sm, list, mass ? m : 0, true, 0.0, dmax, s);
      const unsigned long long W[2] = {sc.w0, sc.w1};
      unsigned long long before = h.mass_above + sc.before;
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * tid + j;
        if (i < m) {
          const bool hit = by_count ? h.count_above + (unsigned long long)i + 1 == target
                                    : before < target && before + W[j] >= target;
          if (hit) sm.found = {before + W[j], list[i], 0, 1};
        }
        before += W[j];
      }
      __syncthreads();
    }
    const int t = exchange(sm.found);
    const Exchange e = remote(0, t);
    *total = e.a;
    return {~(uint32_t)(e.b >> 32), (int)(uint32_t)e.b};
  }
};

// A row whose cut the list does not reach, or without a filter: from the masses of all values.
__device__ __noinline__ void general(const SampleParams& p, Row R, int row, int mis, int kk, float tp, float mp, float u,
                                     unsigned long long mass, unsigned long long mine) {
  Shared& sm = R.sm;
  float* const x = R.x;
  const int n = R.n, e0 = R.e0, tid = R.tid, lane = R.lane, warp = R.warp, rank = R.rank, C = R.C, per = R.per;
  const bool by_k = kk > 0 && kk < p.vocab, by_p = tp < 1.f, plain = !by_k && !by_p && !(mp > 0.f);
  int t;
  // ---- top-k, then top-p: the last element kept
  Cut cut = {0, 0x7fffffff};
  bool fresh = false;
  unsigned long long unused;
  if (by_k || by_p) {
    R.histogram(true, 0, 0, 0, by_p);
    fresh = true;
    uint32_t c = 0;
    unsigned long long m = 0;
    for (int i = tid; i < kBins; i += kT) {
      c += R.cnt[i];
      m += (unsigned long long)R.lo[i] + ((unsigned long long)R.hi[i] << 32);
    }
    c = __reduce_add_sync(0xffffffffu, c);
    m = warp_sum(m);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = c, sm.w64[warp] = m;
    __syncthreads();
    c = 0;
    m = 0;
    for (int w = 0; w < kWarps; ++w) c += sm.w32[w], m += sm.w64[w];
    t = R.exchange({m, 0, c, 0});
    c = R.sum_c(t);
    mass = R.sum_a(t);
    // (fewer values than top_k: all stay)
    if (by_k && (uint32_t)kk < c) cut = R.search(true, (unsigned long long)kk, by_p, fresh, by_p ? &mass : &unused);
  }
  if (by_p) {
    const double want = tp > 0.f ? ceil((double)tp * (double)mass) : 1.0;
    const unsigned long long target = max(1ull, min((unsigned long long)want, mass));
    cut = R.search(false, target, true, fresh, &unused);
  }
  // ---- masses of the survivors, warp by warp in index order
  const double mpd = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
  auto kept = [&](int i) -> unsigned long long {
    const float l = x[i];
    const uint32_t k = key_of(l);
    if (k < cut.key || k == kMasked || (k == cut.key && e0 + i > cut.at)) return 0;
    double w;
    const unsigned long long W = weight(sm, l, R.dmax, R.s, &w);
    return w >= mpd ? W : 0ull;
  };
  const int a = min(n, warp * per), e = min(n, a + per);
  unsigned long long m = mine;           // without a filter the first pass has it
  if (!plain) {
    m = 0;
#pragma unroll 4
    for (int i = a + lane; i < e; i += 32) m += kept(i);
    m = warp_sum(m);
  }
  __syncthreads();
  if (lane == 0) sm.w64[warp] = m;
  __syncthreads();
  unsigned long long before = 0, here = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.w64[w];
    here += sm.w64[w];
  }
  t = R.exchange({here, 0, 0, 0});
  const unsigned long long theirs = lane < C ? R.remote(lane, t).a : 0ull;
  before += warp_sum(lane < rank ? theirs : 0ull);
  const unsigned long long total = warp_sum(theirs);
  const unsigned long long want = min((unsigned long long)((double)u * (double)total), total - 1);
  if (before <= want && want < before + m) {             // one warp of the cluster
    // contiguous parts of the warp's values, one for each lane
    const int part = per / 32, a2 = min(e, a + lane * part), e2 = min(e, a2 + part);
    unsigned long long w = 0;
    for (int i = a2; i < e2; ++i) w += kept(i);
    unsigned long long run = before + warp_scan(w, lane) - w;
    if (run <= want && want < run + w)
      for (int i = a2; i < e2; ++i) {
        const unsigned long long W = kept(i);
        if (want < run + W) {
          p.token[row] = e0 + i - mis;
          if (p.prob) p.prob[row] = (float)((double)W / (double)total);
          break;
        }
        run += W;
      }
  }
  cg::this_cluster().sync();             // no CTA leaves while another may read its shared memory
}

__global__ void __launch_bounds__(kT, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sm;
  auto cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* x = reinterpret_cast<float*>(dyn);
  uint32_t* cnt = reinterpret_cast<uint32_t*>(x + p.seg);
  if (tid < 64) sm.pow64[tid] = exp2((double)tid / 64.0);
  if (tid < kCoarse) sm.coarse[tid] = 0;

  // ---- the row into shared memory.  Places are counted from the 16-byte boundary at or below
  // the row's first value, so all inner loads are 16 bytes wide.
  const float* src = p.logits + (int64_t)row * p.row_stride;
  const int mis = (int)((reinterpret_cast<uintptr_t>(src) >> 2) & 3);
  const int e0 = rank * p.seg, e1 = min(e0 + p.seg, p.vocab + mis);   // places mis .. vocab + mis - 1 are values
  const int n = max(0, e1 - e0);
  uint32_t best = kMasked;               // as an ordered key
  auto take = [&](float l) {
    l = l == l ? l + 0.f : -INFINITY;    // NaN is masked; -0 counts as 0
    best = max(best, key_of(l));
    return l;
  };
  const float* at0 = src - mis;
#pragma unroll 5
  for (int i = 4 * tid; i < n; i += 4 * kT) {
    const int e = e0 + i;
    float4 v;
    if (e >= mis && e + 4 <= p.vocab + mis) {
      v = __ldcs(reinterpret_cast<const float4*>(at0 + e));
    } else {
      float t[4];
      for (int j = 0; j < 4; ++j) t[j] = (e + j >= mis && e + j < p.vocab + mis) ? at0[e + j] : -INFINITY;
      v = make_float4(t[0], t[1], t[2], t[3]);
    }
    v.x = take(v.x);
    v.y = take(v.y);
    v.z = take(v.z);
    v.w = take(v.w);
    *reinterpret_cast<float4*>(x + i) = v;
  }
  // ---- the maximum
  best = __reduce_max_sync(0xffffffffu, best);
  if (lane == 0) sm.w32[warp] = best;
  __syncthreads();
  best = __reduce_max_sync(0xffffffffu, lane < kWarps ? sm.w32[lane] : 0u);
  const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  Row R = {sm, x, cnt, cnt + kBins, cnt + 2 * kBins, reinterpret_cast<unsigned long long*>(cnt + 3 * kBins),
           e0, n, C, rank, tid, lane, warp, 0, per, 0.f, 1.f, 0.0, 0.0};
  int t = R.exchange({0, 0, best, 0});
  best = __reduce_max_sync(0xffffffffu, lane < C ? R.remote(lane, t).c : 0u);
  // ---- settings
  const float T = p.temperature ? p.temperature[row] : 1.f;
  const int kk = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  float u = p.u[row];
  u = u >= 0.f ? fminf(u, 1.f) : 0.f;
  const bool none = best == kMasked;
  if (none || !(T > 0.f)) {              // the same for the whole cluster
    uint32_t at = 0xffffffffu;           // the lowest place of the maximum
    if (!none)
      for (int i = tid; i < n && at == 0xffffffffu; i += kT)
        if (key_of(x[i]) == best) at = (uint32_t)(e0 + i);
    at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = at;
    __syncthreads();
    at = __reduce_min_sync(0xffffffffu, lane < kWarps ? sm.w32[lane] : 0xffffffffu);
    t = R.exchange({0, 0, at, 0});
    at = __reduce_min_sync(0xffffffffu, lane < C ? R.remote(lane, t).c : 0xffffffffu);
    if (rank == 0 && tid == 0) {
      p.token[row] = none ? -1 : (int)at - mis;
      if (p.prob) p.prob[row] = none ? 0.f : 1.f;
    }
    cluster.sync();                      // the exchange above may still be read
    return;
  }
  R.lmax = of_key(best);
  if (R.lmax == INFINITY) {              // only +inf counts, with equal weights
    __syncthreads();
    for (int i = tid; i < n; i += kT) x[i] = x[i] == INFINITY ? 0.f : -INFINITY;
    R.lmax = 0.f;
    __syncthreads();
  }
  R.inv_t = 1.f / T;
  R.dmax = (double)R.lmax;
  R.s = 92.332482616893656769 / (double)T;              // 64 log2(e) / T
  const bool by_k = kk > 0 && kk < p.vocab, by_p = tp < 1.f, by_m = mp > 0.f;
  const bool plain = !by_k && !by_p && !by_m, total = plain || (by_p && !by_k);
  unsigned long long mass = 0;
  const unsigned long long mine = total ? R.warp_mass(!plain) : 0ull;
  if (!plain) {
    // ---- a distance that holds a list's worth of values, from the sample
    R.sample_distances();
    __syncthreads();
    if (lane == 0) sm.w64[warp] = mine;
    __syncthreads();
    t = R.exchange({warp_sum(lane < kWarps ? sm.w64[lane] : 0ull), 0, 0, 0});
    mass = R.sum_a(t);
    uint32_t c4[4] = {0, 0, 0, 0};       // bins 4 lane .. 4 lane + 3
#pragma unroll
    for (int r = 0; r < kMaxC; ++r)
      if (r < C) {
        const uint4 v = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(sm.coarse, r) + 4 * lane);
        c4[0] += v.x, c4[1] += v.y, c4[2] += v.z, c4[3] += v.w;
      }
    uint32_t run = warp_scan(c4[0] + c4[1] + c4[2] + c4[3], lane) - (c4[0] + c4[1] + c4[2] + c4[3]);
    int bins = 0;                        // bins whose running number stays within the list
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      run += c4[j];
      bins += run * 8u <= (uint32_t)kWant;
    }
    bins = __reduce_add_sync(0xffffffffu, bins);
    // rows that fit the list whole need no distance
    const float far = p.vocab <= kList ? INFINITY : (float)max(bins, 1) * 0.125f;
    // ---- their exact number and mass, and where each warp's begin
    unsigned long long near_mass;
    const uint32_t c = R.near_count(far, &near_mass);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = c, sm.w64[warp] = near_mass;
    __syncthreads();
    const uint32_t cw = lane < kWarps ? sm.w32[lane] : 0u;
    const int t2 = R.exchange({warp_sum(lane < kWarps ? sm.w64[lane] : 0ull), 0, __reduce_add_sync(0xffffffffu, cw), 0});
    const uint32_t theirs = lane < C ? R.remote(lane, t2).c : 0u;
    const uint32_t m = __reduce_add_sync(0xffffffffu, theirs);
    near_mass = R.sum_a(t2);
    if (p.vocab <= kList) mass = near_mass;
    // does the list hold the cut?  (min-p alone: 2^-20 covers the rounding of the distances)
    bool ok = m > 0 && m <= (uint32_t)kList;
    if (by_k) ok = ok && m >= (uint32_t)kk;
    else if (by_p) ok = ok && (double)near_mass >= ceil((double)tp * (double)mass);
    else ok = ok && -logf(fminf(mp, 1.f)) * (1.f + 0x1p-20f) + 0x1p-20f < far;
    if (ok) {
      R.gather(far, __reduce_add_sync(0xffffffffu, lane < rank ? theirs : 0u) + __reduce_add_sync(0xffffffffu, lane < warp ? cw : 0u), c);
      cluster.sync();                    // CTA 0 has the list; nothing else of the others is read any more
      if (rank != 0) return;
      int token = -1;
      float prob = 0.f;
      R.draw_list((int)m, by_k ? kk : 0, tp, mp, mass, u, &token, &prob);
      if (token >= 0) {
        p.token[row] = token - mis;
        if (p.prob) p.prob[row] = prob;
      }
      return;
    }
  }
  general(p, R, row, mis, kk, tp, mp, u, mass, mine);
}

int sample_smem(int seg) { return seg * 4 + 3 * kBins * 4 + kList * 8; }

}  // namespace

oda_status prepare_sample_kernel() {
  const int most = (ODA_MAX_VOCAB + 3 + kMaxC - 1) / kMaxC + 3;
  return check_cuda(cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         sample_smem(most / 4 * 4 + 4)),
                    "cudaFuncSetAttribute(sample)");
}

oda_status launch_sample(oda_ctx* ctx, int n_rows, int vocab, int64_t row_stride, const float* logits,
                         const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                         const float* u, int32_t* token, float* prob, cudaStream_t stream) {
  if (!logits || !u || !token) return set_error(ODA_ERR_INVALID_ARG, "sample: null pointer argument");
  if (n_rows < 1 || n_rows > 65535) return set_error(ODA_ERR_INVALID_ARG, "sample: n_rows must be 1..65535");
  if (vocab < 1 || vocab > ODA_MAX_VOCAB)
    return set_error(ODA_ERR_INVALID_ARG, "sample: vocab must be 1..%d", ODA_MAX_VOCAB);
  if (row_stride < vocab || row_stride > (int64_t(1) << 40))
    return set_error(ODA_ERR_INVALID_ARG, "sample: row_stride must be at least vocab");
  const void* al[] = {logits, temperature, top_k, top_p, min_p, u, token, prob};
  for (const void* q : al)
    if (reinterpret_cast<uintptr_t>(q) & 3) return set_error(ODA_ERR_INVALID_ARG, "sample: buffers must be 4-byte aligned");
  ctx->prev_attention = false;
  SampleParams p = {logits, temperature, top_k, top_p, min_p, u, token, prob, row_stride, vocab, 0};
  const int places = vocab + 3;          // the row may start up to 3 places behind a 16-byte boundary
  int C = 1;
  while (C < kMaxC && (places + C - 1) / C > kSeg) C *= 2;
  p.seg = ((places + C - 1) / C + 3) / 4 * 4;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(n_rows * C));
  lc.blockDim = dim3(kT);
  lc.dynamicSmemBytes = sample_smem(p.seg);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&lc, sample_kernel, p), "sample launch");
}

}  // namespace oda

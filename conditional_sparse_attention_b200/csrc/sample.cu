// A token per row of logits from a given uniform number: temperature, top-k, top-p and min-p.
//
// One cluster of up to 8 CTAs works on a row.  The row is read from HBM once, into the shared memory of
// its cluster (a contiguous segment per CTA), and every later pass runs from there.
//
//   1. maximum (and its lowest index, the greedy answer)
//   2. where top-k or top-p is on: a histogram over d = (max - l) / T in 1024 bins of 1/32 (counts, and
//      masses where top-p is on) gives the bin in which the k-th value, or the p-th part of the mass,
//      lies.  Its elements, if at most 1024, are sorted by CTA 0, which finds the exact last element; a
//      fuller bin is cut again by the bits of the values, and one of equal values by their index.
//   3. the masses of the survivors, a prefix over warps and CTAs, and the element at u * mass.
//
// Weights e^-d are computed in fp64 (table of 2^(j/32) and a Taylor polynomial of degree 5, relative
// error below 1e-14) and held as whole multiples of 2^-43 of the largest weight: sums of whole numbers do not
// depend on their order, so neither atomics nor the cluster's shape can change a token.  A row of
// ODA_MAX_VOCAB = 2^18 weights sums to at most 2^61.
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
  double pow32[32];                      // 2^(j/32)
  Exchange ex[2];
  unsigned long long w64[kWarps];
  uint32_t w32[kWarps];
  uint32_t wk[kWarps];
  Exchange found;
  uint32_t n_list;
};

// (1/i!) (ln 2 / 32)^i: 2^(r/32) = sum of these times r^i
constexpr double kL = 0.69314718055994530942 / 32.0;
constexpr double kC1 = kL, kC2 = kL * kL / 2, kC3 = kL * kL * kL / 6, kC4 = kL * kL * kL * kL / 24,
                 kC5 = kL * kL * kL * kL * kL / 120;

// Weight of logit l as a multiple of 2^-kFrac: e^((l - max)/T); s = 32 log2(e) / T; *w the weight itself.
__device__ __forceinline__ unsigned long long weight(const Shared& sm, float l, double max, double s, double* w) {
  const double y = ((double)l - max) * s;               // <= 0
  if (!(y > -32.0 * (kFrac + 2))) {                      // below half a step (also -inf)
    *w = 0.0;
    return 0;
  }
  const double n = rint(y), r = y - n;
  const int k = (int)n;
  const double e = fma(fma(fma(fma(fma(kC5, r, kC4), r, kC3), r, kC2), r, kC1), r, 1.0) * sm.pow32[k & 31];
  *w = __longlong_as_double(__double_as_longlong(e) + ((long long)(k >> 5) << 52));
  return (unsigned long long)__double2ll_rn(__longlong_as_double(__double_as_longlong(e) + ((long long)((k >> 5) + kFrac) << 52)));
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

// The elements kept so far: key > cut, or key == cut and place <= at.
struct Cut {
  uint32_t key;
  int at;
};

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
  double s, dmax;                        // 32 log2(e) / T, the maximum

  __device__ Exchange& remote(int r, int t) { return cg::this_cluster().map_shared_rank(&sm, r)->ex[t]; }

  // Every CTA's thread 0 gives `mine`; returns after all CTAs' values can be read with remote(r, t).
  __device__ int exchange(const Exchange& mine) {
    const int t = turn;
    turn ^= 1;
    if (tid == 0) sm.ex[t] = mine;
    cg::this_cluster().sync();
    return t;
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
  __device__ void histogram(bool first, uint32_t kmin, uint32_t kmax, int shift, bool mass) {
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
  __device__ Hit cross(bool by_count, unsigned long long target, uint32_t ca, unsigned long long ma) {
    // this CTA's share of the bins, summed over the cluster
    const int nb = kBins / C, each = (nb + kT - 1) / kT;
    const int b0 = rank * nb + tid * each;
    uint32_t c[2] = {0, 0};
    unsigned long long m[2] = {0, 0};
    if (tid * each < nb)
      for (int j = 0; j < each; ++j)
        for (int r = 0; r < C; ++r) {
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
    if (tid == 0) sm.found = {0, 0, 0, 0};
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
  __device__ int nth_equal(uint32_t k, uint32_t m) {
    const int a = min(n, warp * per), e = min(n, a + per);
    uint32_t c = 0;
    for (int i = a + lane; i < e; i += 32) c += key_of(x[i]) == k;
    c = warp_sum(c);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = c;
    if (tid == 0) sm.found = {0, 0, 0, 0};
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

  // The shortest prefix (largest first, ties by place) of count >= target or mass >= target; its last
  // element, and its mass (0 where masses are not kept).  fresh: the level-0 histogram is in place.
  __device__ Cut search(bool by_count, unsigned long long target, bool mass, bool& fresh, unsigned long long* total) {
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
      int p2 = 2;
      while (p2 < m) p2 <<= 1;
      for (int i = m + tid; i < p2; i += kT) list[i] = ~0ull;
      for (int k = 2; k <= p2; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
          __syncthreads();
          for (int i = tid; i < p2 / 2; i += kT) {
            const int a = 2 * i - (i & (j - 1)), b = a + j;
            const unsigned long long u = list[a], v = list[b];
            if ((u > v) == ((a & k) == 0)) list[a] = v, list[b] = u;
          }
        }
      __syncthreads();
      // running mass and count over the sorted list, two values a thread
      unsigned long long W[2] = {0, 0};
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * tid + j;
        double w;
        if (mass && i < m) W[j] = weight(sm, of_key(~(uint32_t)(list[i] >> 32)), dmax, s, &w);
      }
      const unsigned long long ws = warp_scan(W[0] + W[1], lane);
      if (lane == 31) sm.w64[warp] = ws;
      if (tid == 0) sm.found = {0, 0, 0, 0};
      __syncthreads();
      unsigned long long before = h.mass_above + ws - (W[0] + W[1]);
      for (int w = 0; w < warp; ++w) before += sm.w64[w];
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

__global__ void __launch_bounds__(kT, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sm;
  auto cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* x = reinterpret_cast<float*>(dyn);
  uint32_t* cnt = reinterpret_cast<uint32_t*>(x + p.seg);
  if (tid < 32) sm.pow32[tid] = exp2((double)tid / 32.0);

  // ---- the row into shared memory.  Places are counted from the 16-byte boundary at or below
  // the row's first value, so all inner loads are 16 bytes wide.
  const float* src = p.logits + (int64_t)row * p.row_stride;
  const int mis = (int)((reinterpret_cast<uintptr_t>(src) >> 2) & 3);
  const int e0 = rank * p.seg, e1 = min(e0 + p.seg, p.vocab + mis);   // places mis .. vocab + mis - 1 are values
  const int n = max(0, e1 - e0);
  float best = -INFINITY;
  int best_at = 0x7fffffff;
  auto take = [&](float l, int e) {
    l = l == l ? l + 0.f : -INFINITY;    // NaN is masked; -0 counts as 0
    if (l > best || (l == best && e < best_at)) best = l, best_at = e;
    return l;
  };
  const float* at0 = src - mis;
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
    v.x = take(v.x, e);
    v.y = take(v.y, e + 1);
    v.z = take(v.z, e + 2);
    v.w = take(v.w, e + 3);
    *reinterpret_cast<float4*>(x + i) = v;
  }
  // ---- the maximum and its lowest place
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float l = __shfl_xor_sync(0xffffffffu, best, o);
    const int e = __shfl_xor_sync(0xffffffffu, best_at, o);
    if (l > best || (l == best && e < best_at)) best = l, best_at = e;
  }
  if (lane == 0) sm.w32[warp] = __float_as_uint(best), sm.wk[warp] = (uint32_t)best_at;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) {
    const float l = __uint_as_float(sm.w32[w]);
    const int e = (int)sm.wk[w];
    if (l > best || (l == best && e < best_at)) best = l, best_at = e;
  }
  const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  Row R = {sm, x, cnt, cnt + kBins, cnt + 2 * kBins, reinterpret_cast<unsigned long long*>(cnt + 3 * kBins),
           e0, n, C, rank, tid, lane, warp, 0, per, 0.f, 1.f, 0.0, 0.0};
  int t = R.exchange({0, 0, __float_as_uint(best), (uint32_t)best_at});
  for (int r = 0; r < C; ++r) {
    const float l = __uint_as_float(R.remote(r, t).c);
    const int e = (int)R.remote(r, t).d;
    if (l > best || (l == best && e < best_at)) best = l, best_at = e;
  }
  // ---- settings
  const float T = p.temperature ? p.temperature[row] : 1.f;
  const int kk = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  const bool none = best == -INFINITY;
  if (none || !(T > 0.f)) {              // the same for the whole cluster
    if (rank == 0 && tid == 0) {
      p.token[row] = none ? -1 : best_at - mis;
      if (p.prob) p.prob[row] = none ? 0.f : 1.f;
    }
    cluster.sync();                      // the exchange above may still be read
    return;
  }
  if (best == INFINITY) {                // only +inf counts, with equal weights
    __syncthreads();
    for (int i = tid; i < n; i += kT) x[i] = x[i] == INFINITY ? 0.f : -INFINITY;
    best = 0.f;
    __syncthreads();
  }
  R.lmax = best;
  R.inv_t = 1.f / T;
  R.dmax = (double)best;
  R.s = 46.166241308446828384 / (double)T;              // 32 log2(e) / T
  // ---- top-k, then top-p: the last element kept
  Cut cut = {0, 0x7fffffff};
  const bool by_p = tp < 1.f;
  bool fresh = false;
  unsigned long long mass = 0;
  bool have_mass = false;
  if (kk > 0 && kk < p.vocab) {
    R.histogram(true, 0, 0, 0, by_p);
    fresh = true;
    // fewer values than top_k: all stay
    uint32_t c = 0;
    for (int i = tid; i < kBins; i += kT) c += cnt[i];
    c = warp_sum(c);
    __syncthreads();
    if (lane == 0) sm.w32[warp] = c;
    __syncthreads();
    c = 0;
    for (int w = 0; w < kWarps; ++w) c += sm.w32[w];
    t = R.exchange({0, 0, c, 0});
    c = 0;
    for (int r = 0; r < C; ++r) c += R.remote(r, t).c;
    if ((uint32_t)kk < c) {
      cut = R.search(true, (unsigned long long)kk, by_p, fresh, &mass);
      have_mass = by_p;
    }
  }
  if (by_p) {
    if (!fresh) R.histogram(true, 0, 0, 0, true);
    fresh = true;
    if (!have_mass) {
      unsigned long long m = 0;
      for (int i = tid; i < kBins; i += kT) m += (unsigned long long)R.lo[i] + ((unsigned long long)R.hi[i] << 32);
      m = warp_sum(m);
      __syncthreads();
      if (lane == 0) sm.w64[warp] = m;
      __syncthreads();
      m = 0;
      for (int w = 0; w < kWarps; ++w) m += sm.w64[w];
      t = R.exchange({m, 0, 0, 0});
      mass = 0;
      for (int r = 0; r < C; ++r) mass += R.remote(r, t).a;
    }
    const double want = tp > 0.f ? ceil((double)tp * (double)mass) : 1.0;
    const unsigned long long target = max(1ull, min((unsigned long long)want, mass));
    cut = R.search(false, target, true, fresh, &mass);
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
  unsigned long long m = 0;
  for (int i = a + lane; i < e; i += 32) m += kept(i);
  m = warp_sum(m);
  __syncthreads();
  if (lane == 0) sm.w64[warp] = m;
  __syncthreads();
  unsigned long long before = 0, here = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.w64[w];
    here += sm.w64[w];
  }
  t = R.exchange({here, 0, 0, 0});
  for (int r = 0; r < C; ++r) {
    if (r < rank) before += R.remote(r, t).a;
    total += R.remote(r, t).a;
  }
  float u = p.u[row];
  u = u >= 0.f ? fminf(u, 1.f) : 0.f;
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
  cluster.sync();                        // no CTA leaves while another may read its shared memory
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

// A token per row of logits from a given uniform number: temperature, top-k, top-p and min-p.
//
// One cluster of up to 8 CTAs works on a row.  The row is read from HBM once, into the shared memory of
// its cluster (a contiguous segment per CTA), and every later pass runs from there.
//
//   1. the maximum (and for a greedy row its lowest index)
//   2. for top-k and top-p a histogram over the distance d = (max - l) / T, in 512 bins of 1/32
//      (for a top-k that lies farther, of 1/2, of 8 and of 128)
//   3. it tells closely how far the cut lies (a bin's weights differ by 3%).  Exact counts and masses within
//      two distances around that (again with others where they miss it) leave a window of at most 1024
//      values, which go to CTA 0 in index order; it finds the last one kept (by 8 bits of the values at a
//      time, or in pairs).  Where the window begins at the maximum CTA 0 drops by min-p and draws, and the
//      others leave.
//   4. else the masses of the survivors, a prefix over warps and CTAs, and the element at u * mass
//   5. where no window is found (many equal values, masked or extreme rows, top-p of a large top-k): a
//      histogram over d in 1024 bins of 1/32, counts and masses, gives the bin of the cut, whose values
//      CTA 0 sorts; a fuller bin is cut again by the bits of the values, and one of equal values by
//      their index
//
// Weights e^-d are computed in fp64 (table of 2^(j/64) and a Taylor polynomial of degree 4, relative
// error below 5e-14) and held as whole multiples of 2^-43 of the largest weight: sums of whole numbers do not
// depend on their order, so neither atomics nor the cluster's shape can change a draw.  (Only step 3's
// masses beyond d = 3 are fp32 sums, each in a fixed order.)  A row of ODA_MAX_VOCAB = 2^18 weights sums to
// at most 2^61.
//
// Bound: latency.  A row of 152k values is 0.6 MB, 0.1 us of HBM, and its phases wait for one another: some
// 4500 clocks for the row, 2000 for the maximum, 12000 for step 2, 7000 for a pass of step 3, 2500 to 9000 for
// CTA 0's part, 13000 for step 4 (where every value survives, the fp64 pipe: some 11 operations a weight at 64
// lanes a clock and SM).  Two CTAs an SM overlap theirs.  Measured at 151936 values, settings mixed, data not
// in L2: one row 18 to 25 us, 32 rows 40 us, 256 rows 190 to 197 us (0.8 TB/s); greedy 256 rows 70 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "tc5.cuh"

namespace cg = cooperative_groups;

namespace oda {
namespace {

constexpr int kT = 512;                  // threads of a CTA
constexpr int kWarps = kT / 32;
constexpr int kMaxC = 8;                 // CTAs of a cluster
constexpr int kBins = 1024;
constexpr int kList = 1024;
constexpr int kBatch = 5;               // 16-byte loads of a thread in flight
constexpr int kShort = 192;              // listed values that are compared in pairs
constexpr int kSeg = 5120;               // values of a CTA above which the cluster grows
constexpr int kFrac = 43;                // weights are multiples of 2^-43
constexpr int kCoarse = 512;              // bins of the histogram that aims
constexpr float kCoarseBins = 32.f;       // bins to a distance of 1, first
constexpr int kWant = 900;               // values aimed at in a window
constexpr int kNone = -2;                // in a token's place: the row has none
constexpr float kNear = 3.f;             // distance from which on masses that place a cut are summed in fp32

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
  int32_t* err;
};

struct alignas(16) Exchange {
  unsigned long long a, b;
  uint32_t c, d;
  unsigned long long m;
};
static_assert(sizeof(Exchange) == 32, "two 16-byte stores");

struct Shared {
  double pow64[64];                      // 2^(j/64)
  alignas(16) uint32_t coarse[kCoarse];  // values by distance
  float wbeyond[kWarps];                 // each warp's mass behind the last bin
  alignas(16) Exchange ex[2][kMaxC];     // what each CTA told this one, in two buffers used in turn
  alignas(8) uint64_t told[2];           // and the barriers that count its bytes
  unsigned long long w64[kWarps];
  uint32_t w32[kWarps];
  uint32_t wk[kWarps];
  Exchange wx[kWarps];
  Exchange found;
  float temperature, top_p, min_p, u;    // the row's settings
  int top_k;
  uint32_t n_list;
  uint32_t around[2];                    // values around the aim, and nearer than the window's far side
  unsigned long long list_mass;
};

// (ln 2 / 64)^i / i!: 2^(r/64) = sum of these times r^i; |r| <= 1/2, so the next term is below 4e-14
constexpr double kL = 0.69314718055994530942 / 64.0;
constexpr double kC2 = kL * kL / 2, kC3 = kL * kL * kL / 6, kC4 = kL * kL * kL * kL / 24;

// Weight e^((l - max)/T) of logit l, and as a whole multiple of 2^-kFrac; s = 64 log2(e) / T.  No branch, so
// that the weights of a loop run abreast; -inf gives 0.
__device__ __forceinline__ unsigned long long weight(const Shared& sm, float l, double max, double s, double* w) {
  const double y0 = ((double)l - max) * s;              // <= 0 (s is finite for every T > 0); -inf or NaN for l = -inf
  // |y0| < 64 (kFrac + 1) = 2816 by its high word: below half a step the weight is 0
  static_assert(kFrac == 43, "the word below is -2816's");
  const bool in = (uint32_t)__double2hiint(y0) < 0xc0a60000u && l > -INFINITY;
  const double y = in ? y0 : 0.0;
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

// Sum over a warp of values whose sum is below 2^62: three whole-warp reductions of 21 bits and the rest
// (a tenth of the time of ten shuffles).
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x1fffffu);
  const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 21) & 0x1fffffu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 42));
  return ((unsigned long long)hi << 42) + ((unsigned long long)mid << 21) + lo;
}
__device__ __forceinline__ float warp_sum(float v) {
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

// CTA 0: the last element of the shortest prefix (largest first, ties by place) of the m listed values (key,
// place and mass arrays) whose count or mass is >= target, and the mass of that prefix: by 8 bits of the
// keys' range at a time, then by index among equals.  Every thread has two of the values.
struct CutMass {
  Cut cut;
  unsigned long long mass;
};
__device__ __noinline__ CutMass cut_list(Shared& sm, const uint32_t* key, int m, bool by_count, unsigned long long target) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t* place = key + kList;
  const unsigned long long* W = reinterpret_cast<const unsigned long long*>(key + 2 * kList);
  uint32_t* lo = const_cast<uint32_t*>(key) + 4 * kList;         // [256] low and [256] high words
  uint32_t* hi = lo + 256;
  const int i = 2 * tid;
  const bool in0 = i < m, in1 = i + 1 < m;
  const uint32_t k0 = in0 ? key[i] : 0u, k1 = in1 ? key[i + 1] : 0u;
  const unsigned long long w0 = in0 ? W[i] : 0ull, w1 = in1 ? W[i + 1] : 0ull;
  uint32_t top = __reduce_max_sync(0xffffffffu, max(k0, k1));
  uint32_t bot = __reduce_min_sync(0xffffffffu, min(in0 ? k0 : 0xffffffffu, in1 ? k1 : 0xffffffffu));
  __syncthreads();
  if (lane == 0) sm.w32[warp] = top, sm.wk[warp] = bot;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, lane < kWarps ? sm.w32[lane] : 0u);
  bot = __reduce_min_sync(0xffffffffu, lane < kWarps ? sm.wk[lane] : 0xffffffffu);
  unsigned long long above = 0;          // count or mass of the keys above `top`
  int shift = 0;
  while (((top - bot) >> shift) >= 256u) shift += 8;
#pragma unroll 1
  while (true) {
    lo[tid] = 0;                         // both arrays: kT = 512
    __syncthreads();
    auto put = [&](uint32_t k, unsigned long long w, bool in) {
      if (!in || k > top || k < bot) return;
      const uint32_t b = (top - k) >> shift;
      if (by_count) {
        atomicAdd(&lo[b], 1u);
      } else {
        const uint32_t low = (uint32_t)w, old = atomicAdd(&lo[b], low);
        const uint32_t up = (uint32_t)(w >> 32) + (old + low < old ? 1u : 0u);
        if (up) atomicAdd(&hi[b], up);
      }
    };
    put(k0, w0, in0);
    put(k1, w1, in1);
    __syncthreads();
    // each of 8 warps scans 32 bins; the bin where the running sum reaches the target
    const unsigned long long v = tid < 256 ? (unsigned long long)lo[tid] + ((unsigned long long)hi[tid] << 32) : 0ull;
    unsigned long long run = warp_scan(v, lane);
    if (lane == 31) sm.w64[warp] = run;
    __syncthreads();
    run += above + warp_sum(lane < warp ? sm.w64[lane] : 0ull);
    if (tid < 256 && run - v < target && run >= target) sm.found = {run - v, v, (uint32_t)tid, 0};
    __syncthreads();
    const Exchange f = sm.found;
    above = f.a;
    top -= f.c << shift;
    const uint32_t width = (1u << shift) - 1u;
    bot = max(bot, top > width ? top - width : 0u);        // (a bin may reach below key 0: values near the type's lowest)
    if (shift == 0) break;
    shift -= 8;
  }
  // values equal to `top`: of those the first `need` in index order; and the mass above them
  unsigned long long mass = (k0 > top ? w0 : 0ull) + (k1 > top ? w1 : 0ull);
  unsigned long long one = in0 && k0 == top ? w0 : in1 && k1 == top ? w1 : 0ull;
  const bool e0 = in0 && k0 == top, e1 = in1 && k1 == top;
  const uint32_t b0 = __ballot_sync(0xffffffffu, e0), b1 = __ballot_sync(0xffffffffu, e1);
  mass = warp_sum(mass);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) one = max(one, __shfl_xor_sync(0xffffffffu, one, o));
  __syncthreads();
  if (lane == 0) sm.wx[warp] = {mass, one, (uint32_t)(__popc(b0) + __popc(b1)), 0};
  __syncthreads();
  const Exchange v = lane < kWarps ? sm.wx[lane] : Exchange{};
  mass = warp_sum(v.a);
  one = v.b;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) one = max(one, __shfl_xor_sync(0xffffffffu, one, o));
  const uint32_t need = (uint32_t)max(1ull, by_count ? target - above : (target - above + one - 1) / max(1ull, one));
  const uint32_t low = (1u << lane) - 1u;
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v.c : 0u) + __popc(b0 & low) + __popc(b1 & low);
  if (e0 && before + 1 == need) sm.found.d = place[i];
  if (e1 && before + e0 + 1 == need) sm.found.d = place[i + 1];
  __syncthreads();
  return {{top, (int)sm.found.d}, mass + need * one};
}

// 16 bytes into another CTA's shared memory, counted on a barrier there.
__device__ __forceinline__ void store_async16(uint32_t to, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
               ::"r"(to), "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar) : "memory");
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
  int turn;                              // exchanges so far
  int per;                               // values of a warp's contiguous part
  float half_max, inv_half;              // max / 2 and 2 / T
  double s, dmax;                        // 64 log2(e) / T, the maximum
  int32_t* err;

  __device__ const Exchange& remote(int r, int t) const { return sm.ex[t][r]; }

  // Every CTA's thread 0 has `mine`; returns the buffer t in which remote(r, t) is CTA r's.  The values
  // are pushed into every CTA's shared memory, which counts their bytes: one way through the cluster
  // instead of a barrier and the way there and back.  A CTA that is one exchange ahead writes the other
  // buffer; it cannot be two ahead, since that needs this one's values of the exchange between.
  __device__ int exchange(const Exchange& mine) {
    const int t = turn & 1, parity = (turn >> 1) & 1;
    ++turn;
    if (warp == 0) {
      const unsigned long long va = __shfl_sync(0xffffffffu, mine.a, 0), vb = __shfl_sync(0xffffffffu, mine.b, 0);
      const unsigned long long vm = __shfl_sync(0xffffffffu, mine.m, 0);
      const uint32_t vc = __shfl_sync(0xffffffffu, mine.c, 0), vd = __shfl_sync(0xffffffffu, mine.d, 0);
      if (lane == 0) mbar_arrive_expect_tx(&sm.told[t], (uint32_t)(C * sizeof(Exchange)));
      if (lane < C) {
        const uint32_t to = mapa_shared(smem_u32(&sm.ex[t][rank]), (uint32_t)lane);
        const uint32_t bar = mapa_shared(smem_u32(&sm.told[t]), (uint32_t)lane);
        store_async16(to, bar, (uint32_t)va, (uint32_t)(va >> 32), (uint32_t)vb, (uint32_t)(vb >> 32));
        store_async16(to + 16, bar, vc, vd, (uint32_t)vm, (uint32_t)(vm >> 32));
      }
    }
    // (a wait that gave up is reported; the row's token is then undefined)
    if (!mbar_wait_bounded(&sm.told[t], parity, 2000000000ull)) atomicOr(err, ODA_DEVERR_WAIT_TIMEOUT);
    return t;
  }

  // The CTAs' values, one lane each (0 beyond the cluster's size): field by field, then sums or maxima.
  __device__ unsigned long long sum_a(int t) { return warp_sum(lane < C ? remote(lane, t).a : 0ull); }
  __device__ uint32_t sum_c(int t) { return __reduce_add_sync(0xffffffffu, lane < C ? remote(lane, t).c : 0u); }

  // (max - l) / T, never below 0; by halves, whose difference cannot overflow.  NaN where 2 / T is infinite, or 0 for
  // l = -inf.
  __device__ float distance(float l) const { return fmaf(l, -0.5f, half_max) * inv_half; }

  // Four values 32 apart (-inf behind e).  Weights are made four abreast, since one alone is a chain of a
  // dozen fp64 operations.
  __device__ void load4(int i, int e, float* l) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) l[j] = i + 32 * j < e ? x[i + 32 * j] : -INFINITY;
  }
  // The same of four neighbours, for passes without an order (i a multiple of 4; x is filled up to one with -inf).
  __device__ void load4v(int i, int e, float* l) const {
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (i < e) v = *reinterpret_cast<const float4*>(x + i);
    l[0] = v.x, l[1] = v.y, l[2] = v.z, l[3] = v.w;
  }
  // The CTA's values by distance, `bins` to a distance of 1, and the mass of those behind the last bin.
  __device__ void distances(float bins) {
    const int a = min(n, warp * per), e = min(n, a + per);
    float beyond = 0.f;
#pragma unroll 1
    for (int i = a + 4 * lane; i - 4 * lane < e; i += 128) {
      float l[4];
      load4v(i, e, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = distance(l[j]), b = d * bins;
        if (b < (float)kCoarse) atomicAdd(&sm.coarse[(int)b], 1u);
        else beyond += exp2_approx(d * -1.4426950408889634f);
      }
    }
    beyond = warp_sum(beyond);
    if (lane == 0) sm.wbeyond[warp] = beyond;
  }

  __device__ int bin0(float l) const { return min(kBins - 1, (int)(distance(l) * 32.f)); }

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
    c = __reduce_add_sync(0xffffffffu, c);
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

  // Numbers, and where asked masses, of all values nearer than d1 and than d2 (>= d1), over the cluster: a, c
  // and b, d of the result; m the mass of all.  (Each warp's stay in sm.wx, each CTA's in buffer *t.)
  // These masses place a cut: those beyond kNear are summed in fp32, in a fixed order.  A weight there is off by at
  // most (4.2 d + 4) 2^-24 of itself (2 / T, the difference, the distance, log2(e) and the exponent round once each,
  // the exponential 2^-22), a lane's sum of n / 512 of them by half as many 2^-24.  What all of them share in it, as
  // 2 / T's rounding, moves the cut by (mass up to d = 3) (1 - top_p), at most 1/4, of it.  Measured over 38000 rows
  // of up to 262144 values, most of them with half their mass at distances 9..13.5: 1.5e-7 of the mass.  A draw's own
  // masses are exact.
  __device__ Exchange within(float d1, float d2, bool mass, int* t) {
    const int a = min(n, warp * per), e = min(n, a + per);
    Exchange v = {};
    float f1 = 0.f, f2 = 0.f, f = 0.f;
#pragma unroll 1
    for (int i = a + 4 * lane; i - 4 * lane < e; i += 128) {
      float l[4], d[4];
      bool close = false;
      load4v(i, e, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = distance(l[j]);
        v.c += d[j] < d1;
        v.d += d[j] < d2;
        close |= d[j] < kNear;
      }
      if (!mass) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float w = exp2_approx(d[j] * -1.4426950408889634f);
        if (!(d[j] >= kNear)) w = 0.f;
        f += w;
        if (d[j] < d1) f1 += w;
        if (d[j] < d2) f2 += w;
      }
      if (__any_sync(0xffffffffu, close)) {
        unsigned long long W[4];
        double w;
#pragma unroll
        for (int j = 0; j < 4; ++j) W[j] = weight(sm, l[j], dmax, s, &w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!(d[j] < kNear)) continue;
          v.m += W[j];
          if (d[j] < d1) v.a += W[j];
          if (d[j] < d2) v.b += W[j];
        }
      }
    }
    const double one = (double)(1ll << kFrac);
    v = {warp_sum(v.a + (unsigned long long)__double2ll_rn((double)f1 * one)),
         warp_sum(v.b + (unsigned long long)__double2ll_rn((double)f2 * one)), __reduce_add_sync(0xffffffffu, v.c),
         __reduce_add_sync(0xffffffffu, v.d), warp_sum(v.m + (unsigned long long)__double2ll_rn((double)f * one))};
    __syncthreads();
    if (lane == 0) sm.wx[warp] = v;
    __syncthreads();
    if (warp == 0) {
      v = lane < kWarps ? sm.wx[lane] : Exchange{};
      v = {warp_sum(v.a), warp_sum(v.b), __reduce_add_sync(0xffffffffu, v.c), __reduce_add_sync(0xffffffffu, v.d), warp_sum(v.m)};
    }
    *t = exchange(v);
    v = lane < C ? remote(lane, *t) : Exchange{};
    return {warp_sum(v.a), warp_sum(v.b), __reduce_add_sync(0xffffffffu, v.c), __reduce_add_sync(0xffffffffu, v.d), warp_sum(v.m)};
  }

  // Number of this warp's values in [near, far).
  __device__ uint32_t window_count(float near, float far) const {
    const int a = min(n, warp * per), e = min(n, a + per);
    uint32_t c = 0;
#pragma unroll 4
    for (int i = a + lane; i < e; i += 32) {
      const float d = distance(x[i]);
      c += d >= near && d < far;
    }
    return __reduce_add_sync(0xffffffffu, c);
  }

  // This warp's `c` values in [near, far) to place `at` on of CTA 0's key and place arrays, in index order.
  __device__ void gather(float near, float far, uint32_t at, uint32_t c) {
    uint32_t* key = cg::this_cluster().map_shared_rank(cnt, 0);
    uint32_t* place = key + kList;
    const int a = min(n, warp * per), e = min(n, a + per);
    const uint32_t stop = at + c;
    for (int i = a + lane; i - lane < e && at < stop; i += 128) {
      float l[4];
      uint32_t here[4];
      load4(i, e, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = distance(l[j]);
        here[j] = __ballot_sync(0xffffffffu, d >= near && d < far && i + 32 * j < e);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t to = at + __popc(here[j] & ((1u << lane) - 1u));
        if (((here[j] >> lane) & 1u) && to < (uint32_t)kList) key[to] = key_of(l[j]), place[to] = (uint32_t)(e0 + i + 32 * j);
        at += __popc(here[j]);
      }
    }
  }

  // CTA 0: the masses of the m listed values, and in sm.list_mass their sum; bit j of the result: this thread's
  // j-th is below `mpd`.
  __device__ uint32_t list_weights(int m, double mpd) {
    unsigned long long* W = reinterpret_cast<unsigned long long*>(cnt + 2 * kList);
    uint32_t drop = 0;
    unsigned long long all = 0;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      const int i = 2 * tid + j;
      if (i < m) {
        double w;
        const unsigned long long v = weight(sm, of_key(cnt[i]), dmax, s, &w);
        W[i] = v;
        all += v;
        if (w < mpd) drop |= 1u << j;
      }
    }
    all = warp_sum(all);
    __syncthreads();
    if (lane == 0) sm.w64[warp] = all;
    __syncthreads();
    all = warp_sum(lane < kWarps ? sm.w64[lane] : 0ull);
    if (tid == 0) sm.list_mass = all;
    __syncthreads();
    return drop;
  }

  // The same draw for a short list, a thread a value: every thread sums what lies above its own (a list of
  // 2: 9600 -> 2700 clocks, one of 150: 8200 -> 7200).
  __device__ void draw_short(int m, bool whole, int kk, float tp, float mp, unsigned long long mass, float u, int* token,
                             float* prob) {
    const uint32_t* key = cnt;
    unsigned long long* W = reinterpret_cast<unsigned long long*>(cnt + 2 * kList);
    const uint32_t own = tid < m ? key[tid] : 0u;
    unsigned long long w = 0;
    double x = 0.0;
    if (tid < m) w = weight(sm, of_key(own), dmax, s, &x);
    if (tid < (m + 3) / 4 * 4) W[tid] = w, cnt[tid] = own;   // (key 0: in front of nothing)
    __syncthreads();
    unsigned long long above = 0;        // mass and number of the values in front, largest first, ties by place
    uint32_t number = 0;
    if (32 * warp < m) {
#pragma unroll 1
      for (int j = 0; j < m; j += 4) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(key + j);
        const ulonglong2 w01 = *reinterpret_cast<const ulonglong2*>(W + j), w23 = *reinterpret_cast<const ulonglong2*>(W + j + 2);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        const unsigned long long v[4] = {w01.x, w01.y, w23.x, w23.y};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool front = k[q] >= (j + q < tid ? own : own + 1u);
          above += front ? v[q] : 0ull;  // (no branch: all lanes differ)
          number += front ? 1u : 0u;
        }
      }
    }
    bool keep = tid < m && (kk <= 0 || number < (uint32_t)kk);
    auto sum = [&](unsigned long long v, unsigned long long* before) {
      const unsigned long long run = warp_scan(v, lane);
      __syncthreads();
      if (lane == 31) sm.w64[warp] = run;
      __syncthreads();
      const unsigned long long each = lane < kWarps ? sm.w64[lane] : 0ull;
      *before = run - v + warp_sum(lane < warp ? each : 0ull);
      return warp_sum(each);
    };
    unsigned long long before;
    if (tp < 1.f) {
      if (whole || kk > 0) mass = sum(keep ? w : 0ull, &before);
      const double want = tp > 0.f ? ceil((double)tp * (double)mass) : 1.0;
      keep = keep && above < max(1ull, min((unsigned long long)want, mass));
    }
    if (mp > 0.f) keep = keep && x >= fmin((double)mp, 1.0);
    const unsigned long long total = sum(keep ? w : 0ull, &before);
    if (total == 0) {
      if (tid == 0) *token = kNone;
      return;
    }
    const unsigned long long want = min((unsigned long long)((double)u * (double)total), total - 1);
    if (keep && before <= want && want < before + w) {
      *token = (int)cnt[kList + tid];
      *prob = (float)((double)w / (double)total);
    }
  }

  // CTA 0 draws from the m listed values, which hold every cut (`mass`: top-p's total without top-k; `whole`: they
  // are the row's all).  One thread gets the token's place; where nothing is left, thread 0 gets kNone.
  __device__ void draw_list(int m, bool whole, int kk, float tp, float mp, unsigned long long mass, float u, int* token,
                            float* prob) {
    if (m <= kShort) return draw_short(m, whole, kk, tp, mp, mass, u, token, prob);
    const bool by_p = tp < 1.f;
    const uint32_t* key = cnt;
    const uint32_t* place = cnt + kList;
    const unsigned long long* W = reinterpret_cast<const unsigned long long*>(cnt + 2 * kList);
    const uint32_t drop = list_weights(m, mp > 0.f ? fmin((double)mp, 1.0) : 0.0);
    if (whole) mass = sm.list_mass;
    Cut cut = {0, 0x7fffffff};
    if (kk > 0) {
      const CutMass c = cut_list(sm, cnt, m, true, (unsigned long long)kk);
      cut = c.cut;
      mass = c.mass;
    }
    if (by_p) {
      const double want = tp > 0.f ? ceil((double)tp * (double)mass) : 1.0;
      const unsigned long long target = max(1ull, min((unsigned long long)want, mass));
      cut = cut_list(sm, cnt, m, false, min(target, sm.list_mass)).cut;   // (the list's own mass is exact)
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
    if (total == 0) {
      if (tid == 0) *token = kNone;
      return;
    }
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

// The last element kept by top-k, then top-p, of any row.
__device__ __noinline__ Cut general(Row R, int vocab, int kk, float tp, int* turn) {
  Shared& sm = R.sm;
  const int tid = R.tid, lane = R.lane, warp = R.warp;
  const bool by_k = kk > 0 && kk < vocab, by_p = tp < 1.f;
  unsigned long long mass = 0;
  int t;
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
  *turn = R.turn;
  return cut;
}

// The CTA's values times a power of two.
__device__ __noinline__ void scale_row(float* x, int n, float by) {
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kT) x[i] *= by;
  __syncthreads();
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
  if (tid == 0) {
    mbar_init(&sm.told[0], 1);
    mbar_init(&sm.told[1], 1);
    fence_mbar_init();
  }
  cluster_arrive();                      // waited for before the first exchange
  if (tid == kT - 1) {                   // (the settings on their way while the row comes)
    sm.temperature = p.temperature ? p.temperature[row] : 1.f;
    sm.top_k = p.top_k ? p.top_k[row] : 0;
    sm.top_p = p.top_p ? p.top_p[row] : 1.f;
    sm.min_p = p.min_p ? p.min_p[row] : 0.f;
    sm.u = p.u[row];
  }
  if (tid < 64) sm.pow64[tid] = exp2((double)tid / 64.0);
  sm.coarse[tid] = 0;                    // kCoarse = kT
  if (tid < 2) sm.around[tid] = 0;

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
  // kBatch loads of a thread in flight together, the two ends of the row apart
#pragma unroll 1
  for (int i0 = 4 * tid; i0 < n; i0 += kBatch * 4 * kT) {
    float4 v[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + q * 4 * kT, e = e0 + i;
      if (i < n && e >= mis && e + 4 <= p.vocab + mis) v[q] = __ldcs(reinterpret_cast<const float4*>(at0 + e));
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = i0 + q * 4 * kT, e = e0 + i;
      if (i >= n) break;
      if (e < mis || e + 4 > p.vocab + mis) {
        float t[4];
        for (int j = 0; j < 4; ++j) t[j] = (e + j >= mis && e + j < p.vocab + mis) ? at0[e + j] : -INFINITY;
        v[q] = make_float4(t[0], t[1], t[2], t[3]);
      }
      v[q].x = take(v[q].x);
      v[q].y = take(v[q].y);
      v[q].z = take(v[q].z);
      v[q].w = take(v[q].w);
      *reinterpret_cast<float4*>(x + i) = v[q];
    }
  }
  // ---- the maximum
  best = __reduce_max_sync(0xffffffffu, best);
  if (lane == 0) sm.w32[warp] = best;
  __syncthreads();
  best = __reduce_max_sync(0xffffffffu, lane < kWarps ? sm.w32[lane] : 0u);
  const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  Row R = {sm, x, cnt, cnt + kBins, cnt + 2 * kBins, reinterpret_cast<unsigned long long*>(cnt + 3 * kBins),
           e0, n, C, rank, tid, lane, warp, 0, per, 0.f, 2.f, 0.0, 0.0, p.err};
  cluster_wait();                        // every CTA's barriers are there
  int t = R.exchange({0, 0, best, 0});
  best = __reduce_max_sync(0xffffffffu, lane < C ? R.remote(lane, t).c : 0u);
  // ---- settings
  float T = sm.temperature;
  const float tp = sm.top_p, mp = sm.min_p;
  const int kk = sm.top_k;
  float u = sm.u;
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
    return;
  }
  float lmax = of_key(best);
  if (lmax == INFINITY) {              // only +inf counts, with equal weights
    __syncthreads();
    for (int i = tid; i < n; i += kT) x[i] = x[i] == INFINITY ? 0.f : -INFINITY;
    lmax = 0.f;
    __syncthreads();
  }
  if (T < 0x1p-100f && fabsf(lmax) < 0x1p60f) {
    // Halves of values of such a temperature's size lose bits: logits and temperature times 2^60, which no weight
    // depends on.  (What becomes -inf by that lies 2^160 T behind the maximum; beyond 2^60 every difference does.)
    scale_row(x, n, 0x1p60f);
    lmax *= 0x1p60f;
    T *= 0x1p60f;
  }
  R.half_max = 0.5f * lmax;
  R.inv_half = 2.f / T;
  R.dmax = (double)lmax;
  R.s = 92.332482616893656769 / (double)T;              // 64 log2(e) / T
  const bool by_k = kk > 0 && kk < p.vocab, by_p = tp < 1.f, by_m = mp > 0.f;
  Cut cut = {0, 0x7fffffff};
  if (by_k || by_p) {
    // ---- top-k's count or top-p's mass
    unsigned long long mass = 0;
    const bool by_mass = !by_k;
    // ---- how far that is, to a few values, and a distance on both sides of it.  A bin a thread.
    float d1, d2, bins = kCoarseBins;
#pragma unroll 1
    while (true) {
      R.distances(bins);
      cluster.sync();
      uint32_t c = 0;
#pragma unroll
      for (int r = 0; r < kMaxC; ++r)
        if (r < C) c += cluster.map_shared_rank(sm.coarse, r)[tid];
      float beyond = 0.f;
      for (int w = lane; w < C * kWarps; w += 32) beyond += cluster.map_shared_rank(sm.wbeyond, w / kWarps)[w % kWarps];
      beyond = warp_sum(beyond);
      // a bin's values at the weight of its middle, top-k: at 1
      const float wb = (float)c * (by_mass ? exp2_approx(-1.4426950408889634f / kCoarseBins * ((float)tid + 0.5f)) : 1.f);
      const float run = warp_scan(wb, lane);
      __syncthreads();
      if (lane == 31) sm.wx[warp].a = (unsigned long long)__float_as_uint(run);
      __syncthreads();
      const float part = lane < kWarps ? __uint_as_float((uint32_t)sm.wx[lane].a) : 0.f;
      // from the far end, where the weights are small: how much lies behind the cut, and in this bin and behind
      const float all = warp_sum(part), from = all - warp_sum(lane < warp ? part : 0.f) - run + wb;
      // top-k that reaches behind the last bin (a low temperature): again with wider ones
      if (by_k && all < (float)kk && bins > 0.1f) {
        cluster.sync();
        sm.coarse[tid] = 0;
        __syncthreads();
        bins *= 1.f / 16.f;
        continue;
      }
      const float behind = by_mass ? (1.f - tp) * (all + beyond) - beyond : all - (float)kk;
      const float at = warp_sum(from - wb > behind ? 1.f : from > behind && wb > 0.f ? (from - behind) / wb : 0.f);
      if (lane == 0) sm.wx[warp].c = __float_as_uint(at);
      __syncthreads();
      const float mid = warp_sum(lane < kWarps ? __uint_as_float(sm.wx[lane].c) : 0.f);           // in bins
      // the values in the three bins around it, and half a window's width; the values nearer than its far end
      const uint32_t three = __reduce_add_sync(0xffffffffu, fabsf((float)tid + 0.5f - mid) < 1.5f ? c : 0u);
      if (lane == 0 && three) atomicAdd(&sm.around[0], three);
      __syncthreads();
      const float half = fminf(fmaxf(bins, 2.f), (float)(kWant / 2) * 3.f / (float)max(1u, sm.around[0]));
      const uint32_t below = __reduce_add_sync(0xffffffffu, (float)tid < mid + half ? c : 0u);
      if (lane == 0 && below) atomicAdd(&sm.around[1], below);
      __syncthreads();
      const float step = __uint_as_float(0x7f000000u - __float_as_uint(bins));           // 1 / bins, a power of two
      d1 = sm.around[1] <= (uint32_t)kList ? 0.f : fmaxf(0.f, mid - half) * step;
      d2 = (mid + half) * step;
      if (p.vocab <= kList) d1 = 0.f, d2 = INFINITY;
      break;
    }
    // ---- a window of at most kList values that holds the cut
    float near = 0.f, far = INFINITY;    // fewer than the target lie nearer than `near`, enough nearer than `far`
    unsigned long long near_m = 0, far_m = 0;
    uint32_t near_c = 0, far_c = 0xffffffffu;
    unsigned long long target = (unsigned long long)kk;
    bool ok = false;
    int at_near = 0, at_far = 0;         // where the window's sides are from: 1, 2: the last distances tried
#pragma unroll 1
    for (int turn = 0; turn < 20 && !(by_k && by_p && turn > 1); ++turn) {
      const Exchange v = R.within(d1, d2, by_mass, &t);
      if (by_mass) {
        mass = v.m;
        target = max(1ull, min(tp > 0.f ? (unsigned long long)ceil((double)tp * (double)mass) : 1ull, mass));
      }
      at_near = at_near ? 3 : 0;
      at_far = 3;
      const bool one = by_mass ? v.a >= target : v.c >= target, two = by_mass ? v.b >= target : v.d >= target;
      if (one) {
        far = d1, far_c = v.c, far_m = v.a, at_far = 1;
      } else {
        near = d1, near_c = v.c, near_m = v.a, at_near = 1;
        if (two) far = d2, far_c = v.d, far_m = v.b, at_far = 2;
        else near = d2, near_c = v.d, near_m = v.b, at_near = 2;
      }
      // (a window from the maximum on saves the pass over the survivors)
      if (far_c <= (uint32_t)kList) near = 0.f, near_c = 0, near_m = 0, at_near = 0;
      ok = far_c != 0xffffffffu && far_c - near_c <= (uint32_t)kList;
      if (ok) break;
      if (far_c == 0xffffffffu) {        // none far enough yet
        if (turn >= 8 || near == INFINITY) break;
        d1 = near + 0.125f * (float)(1 << turn);
        d2 = d1 + 0.25f * (float)(1 << turn);
      } else {
        // on from the distances just tried, by the density between them; else where a straight line
        // between the two sides meets the target
        const float span = far - near;
        const double v1 = by_mass ? (double)v.a : (double)v.c, v2 = by_mass ? (double)v.b : (double)v.d;
        float mid = d1 + (d2 - d1) * (float)(((double)target - v1) / (v2 - v1));
        float half = (d2 - d1) * (float)(kWant / 2) / (float)(v.d - v.c);
        if (!(v2 > v1 && v.d > v.c && mid > near && mid < far && half < 0.25f * span)) {
          const double n0 = by_mass ? (double)near_m : (double)near_c, n1 = by_mass ? (double)far_m : (double)far_c;
          mid = near + span * (float)(((double)target - n0) / (n1 - n0));
          half = span * fmaxf(0.05f, fminf(0.25f, (kWant / 2) / (float)(far_c - near_c)));
        }
        d1 = mid - half > near ? mid - half : near + span * 0.01f;
        d2 = mid + half < far ? mid + half : far - span * 0.01f;
        if (!(d1 > near && d2 < far && d1 <= d2)) break;      // the distances are used up: equal values
      }
    }
    if (by_k && by_p) ok = ok && near_c == 0;                 // top-p has to lie in the window too
    if (ok) {
      // every warp's and every CTA's number of them: known from the last pass, or counted
      uint32_t cw, theirs;
      if (at_near < 3 && at_far < 3) {
        const Exchange w = lane < kWarps ? sm.wx[lane] : Exchange{}, r = lane < C ? R.remote(lane, t) : Exchange{};
        cw = (at_far == 1 ? w.c : w.d) - (at_near == 0 ? 0u : at_near == 1 ? w.c : w.d);
        theirs = (at_far == 1 ? r.c : r.d) - (at_near == 0 ? 0u : at_near == 1 ? r.c : r.d);
      } else {
        const uint32_t c1 = R.window_count(near, far);
        __syncthreads();
        if (lane == 0) sm.w32[warp] = c1;
        __syncthreads();
        cw = lane < kWarps ? sm.w32[lane] : 0u;
        t = R.exchange({0, 0, __reduce_add_sync(0xffffffffu, cw), 0});
        theirs = lane < C ? R.remote(lane, t).c : 0u;
      }
      const uint32_t c = __shfl_sync(0xffffffffu, cw, warp);
      const int m = (int)__reduce_add_sync(0xffffffffu, theirs);
      R.gather(near, far, __reduce_add_sync(0xffffffffu, lane < rank ? theirs : 0u) + __reduce_add_sync(0xffffffffu, lane < warp ? cw : 0u), c);
      cluster.sync();
      if (near_c == 0) {
        // CTA 0 has every candidate; nothing of the other CTAs is read any more
        if (rank != 0) return;
        int token = -1;
        float prob = 0.f;
        R.draw_list(m, p.vocab <= kList, by_k ? kk : 0, tp, mp, mass, u, &token, &prob);
        if (token != -1) {               // this thread's to write
          p.token[row] = token == kNone ? -1 : token - mis;
          if (p.prob) p.prob[row] = prob;
        }
        return;
      }
      Exchange got = {};
      if (rank == 0) {
        R.list_weights(m, 0.0);
        const CutMass r = cut_list(sm, R.cnt, m, by_k, by_mass ? min(target - near_m, sm.list_mass) : target - near_c);
        got = {0, 0, r.cut.key, (uint32_t)r.cut.at};
      }
      t = R.exchange(got);
      cut = {R.remote(0, t).c, (int)R.remote(0, t).d};
    } else {
      int turns;
      cut = general(R, p.vocab, kk, tp, &turns);
      R.turn = turns;
    }
  }
  // ---- masses of the survivors, warp by warp in index order
  const double mpd = by_m ? fmin((double)mp, 1.0) : 0.0;
  // (a distance that min-p cannot reach; 2^-20 covers the rounding of the distances)
  const float far = by_m ? -logf(fminf(mp, 1.f)) * (1.f + 0x1p-20f) + 0x1p-20f : INFINITY;
  const int a = min(n, warp * per), e = min(n, a + per);
  const bool cuts = cut.key > kMasked;  // else every unmasked value stays
  const float edge = cuts ? of_key(cut.key) : -INFINITY;
  const int edge_at = cuts ? cut.at : -1;
  // 4 values 32 apart from i on that the cut (and, but for roundings, min-p) keeps, else -inf
  auto kept4 = [&](int i, int to, float* l) {
    R.load4(i, to, l);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bool in = l[j] > edge || (l[j] == edge && e0 + i + 32 * j <= edge_at);
      if (by_m) in = in && !(R.distance(l[j]) > far);
      if (!in) l[j] = -INFINITY;
    }
  };
  auto masses4 = [&](const float* l, unsigned long long* W) {
    double w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) W[j] = weight(sm, l[j], R.dmax, R.s, &w[j]);
    if (by_m) {
#pragma unroll
      for (int j = 0; j < 4; ++j) W[j] = w[j] >= mpd ? W[j] : 0ull;
    }
  };
  unsigned long long m = 0, W[4];
  float l[4];
  if (!cuts && !by_m) {
#pragma unroll 1
    for (int i = a + 4 * lane; i - 4 * lane < e; i += 128) {
      double w;
      R.load4v(i, e, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) W[j] = weight(sm, l[j], R.dmax, R.s, &w);
      m += (W[0] + W[1]) + (W[2] + W[3]);
    }
  } else {
    // few are kept: closed up in 256 places of the warp's own, and weighed 128 at a time
    __syncthreads();                     // (CTA 0's list lay there)
    float* buf = reinterpret_cast<float*>(cnt) + 256 * warp;
    uint32_t fill = 0;
#pragma unroll 1
    for (int i = a + lane; true; i += 128) {
      const bool more = i - lane < e;
      if (more) {
        kept4(i, e, l);
        if (!__any_sync(0xffffffffu, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) > -INFINITY)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t in = __ballot_sync(0xffffffffu, l[j] > -INFINITY);
          if (l[j] > -INFINITY) buf[fill + __popc(in & ((1u << lane) - 1u))] = l[j];
          fill += __popc(in);
        }
        if (fill < 128) continue;
      }
      __syncwarp();
      const uint32_t from = fill > 128 ? fill - 128 : 0;     // (behind the last, fill < 128)
#pragma unroll
      for (int j = 0; j < 4; ++j) l[j] = from + 32 * j + lane < fill ? buf[from + 32 * j + lane] : -INFINITY;
      masses4(l, W);
      m += (W[0] + W[1]) + (W[2] + W[3]);
      fill = from;
      __syncwarp();
      if (!more) break;
    }
  }
  m = warp_sum(m);
  __syncthreads();
  if (lane == 0) sm.w64[warp] = m;
  __syncthreads();
  const unsigned long long here = warp_sum(lane < kWarps ? sm.w64[lane] : 0ull);
  t = R.exchange({here, 0, 0, 0});
  const unsigned long long theirs = lane < C ? R.remote(lane, t).a : 0ull;
  unsigned long long before = warp_sum(lane < rank ? theirs : 0ull);
  const unsigned long long total = warp_sum(theirs);
  if (total == 0) {                      // the same for the whole cluster
    if (rank == 0 && tid == 0) {
      p.token[row] = -1;
      if (p.prob) p.prob[row] = 0.f;
    }
    return;
  }
  const unsigned long long want = min((unsigned long long)((double)u * (double)total), total - 1);
  if (want < before || want >= before + here) return;    // the draw is another CTA's
  // ---- the element: the warp's part that holds it, which all warps share out, then the share
  auto part = [&]() {                    // index of the warp's mass that holds it; before: all in front
    const unsigned long long mass = lane < kWarps ? sm.w64[lane] : 0ull, upto = before + warp_scan(mass, lane);
    const int at = __ffs((int)__ballot_sync(0xffffffffu, want < upto)) - 1;
    before = __shfl_sync(0xffffffffu, upto - mass, at);
    return at;
  };
  const int a1 = min(n, part() * per), e1w = min(n, a1 + per), per2 = (per / kWarps + 31) / 32 * 32;
  const int a2 = min(e1w, a1 + warp * per2), e2 = min(e1w, a2 + per2);
  m = 0;
#pragma unroll 1
  for (int i = a2 + lane; i - lane < e2; i += 128) {
    kept4(i, e2, l);
    masses4(l, W);
    m += (W[0] + W[1]) + (W[2] + W[3]);
  }
  m = warp_sum(m);
  __syncthreads();
  if (lane == 0) sm.w64[warp] = m;
  __syncthreads();
  if (part() != warp) return;
#pragma unroll 1
  for (int i = a2 + lane; i - lane < e2; i += 128) {
    kept4(i, e2, l);
    masses4(l, W);
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const unsigned long long upto = before + warp_scan(W[0], lane);
      if (upto - W[0] <= want && want < upto) {
        p.token[row] = e0 + i + 32 * j - mis;
        if (p.prob) p.prob[row] = (float)((double)W[0] / (double)total);
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
      W[0] = W[1], W[1] = W[2], W[2] = W[3];
    }
  }
}

int sample_smem(int seg) { return seg * 4 + 3 * kBins * 4 + kList * 8; }
static_assert(4 * kList * 4 + 2 * 256 * 4 <= 3 * kBins * 4 + kList * 8 && kT == 512, "the list and its bins lie over the histogram and its list");

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
  SampleParams p = {logits, temperature, top_k, top_p, min_p, u, token, prob, row_stride, vocab, 0, ctx->err};
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

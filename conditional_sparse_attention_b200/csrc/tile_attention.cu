// Attention of many query rows per KV head on the fifth-generation tensor cores: whole prompts
// (packed sequences, full or local set) and trees of drafted tokens over the paged cache.
//
// Mathematics: for a query row q with visible set S, o = sum_{j in S} p_j v_j / sum_{j in S} p_j with
// p_j = 2^(c (q.k_j - m)), c = log2(e) / sqrt(128), m a running reference that is at least the running
// maximum less 8 / c, so 2^8 bounds p and the reference moves (and O is rescaled) only where the
// maximum has grown by more than that.
//
// One CTA works on two "slots" of 128 query rows that share the KV head and its K/V tiles of 128
// positions.  A slot's rows are (token, head of the group) pairs, 128 / g tokens x g heads, so a KV tile
// is read once for all heads of its group and a short prompt or a small tree still fills the rows.
// Where only slot 0 has tokens, slot 1 takes every second KV tile of the same rows and the two partial
// results are joined through tensor memory at the end: the two slots always alternate on the tensor
// cores, one computing weights while the other's products run.
//
//   warps 0-7, 8-15: two threads per row of slot 0 / 1, one for each 64 columns of a tile: scores from
//                    TMEM, weights back to TMEM as bf16
//   warp 16:         issues the products S = Q K^T and O += P V (M = N = 128, 16-deep steps)
//   warps 17, 19:    bring Q and K, and V, by TMA (a ring of 5 stages of 32 KB, in the order of use)
//   warp 18:         plans the CTA's units of work, two ahead
//
// TMEM: S0 | S1 | O0 | O1, 128 columns each; the weights of columns 0..63 and 64..127 overwrite columns
// 0..31 and 64..95 of S_i, so that each thread's weights lie over its own scores.
// Every wait is bounded; a wait that gives up sets ODA_DEVERR_WAIT_TIMEOUT and ends the CTA (the row
// threads, which meet in pairs, go on without waiting to the end of their unit).
//
// Bounds and measurements (B200; copies at 6548 GB/s, library products at 1624 TFLOP/s):
//   prompts: the matrix products and, as long, the exponentials of a step, each waiting for the other; in
//     repeated calls the power cap (the same time with any share of the exponentials on the FMA pipe).  One
//     prompt of 8192, 32/8 heads, full set: 435 to 475 us alone, 500 to 528 repeated (1040 to 1100 TFLOP/s, 64 to 68%);
//     local set (4 + 2048): 260 us alone, 263 to 281 repeated (the tiles at the window's two
//     ends and the sinks' tile are partly masked: 18 tiles for 16).  One token: 7.3 us; 512 tokens, 16/8 heads: 14.4 us.
//   trees: the cache's bytes while a KV head has few rows (32 sequences of 2000..32768, 16 nodes, 16/8 heads: 387 us
//     alone, 6.1 TB/s, 393 to 441 repeated), then the products and the power of both (4 of 131072, 64 nodes, 32/8
//     heads: 514 us alone, 582 to 654 repeated).  A chain of 5 over 4096 positions: 20 us, of which the join is 5.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "tc5.cuh"

namespace oda {
namespace {

constexpr int kTile = 128;              // query rows of a slot; positions of a KV tile
constexpr int kStages = 5;
constexpr int kStageBytes = kTile * 256;
constexpr int kHalf = kTile * 128;      // bytes of one 64-value half of a tile
constexpr int kThreads = 640;           // 96 registers a thread at launch, then 4 x 104 and 64 by warpgroup
constexpr int kRegs = 96, kRegsRow = 104, kRegsOther = 64;
static_assert(4 * kRegsRow + kRegsOther == 5 * kRegs, "the split has to add up to the launch");
constexpr int kWarpMma = 16, kWarpLoad = 17, kWarpPlan = 18, kWarpLoadV = 19;
constexpr int kAhead = 2;               // units planned ahead
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kGrow = 8.0f;           // log2 of the growth that moves a row's reference
constexpr uint32_t kColS = 0, kColO = 256;
constexpr int kPoly = 4;                  // one pair of weights in 4 is made on the FMA pipe

struct TileParams {
  const int32_t* cu;
  __nv_bfloat16* out;
  int32_t* err;
  int64_t n_rows;
  int n_seqs, Hq, Hkv, g, nt;           // nt = tokens of a slot
  int nq;                               // tree: nodes of a copy of Q, a divisor of nt
  int local, sinks, window;
  float c;                              // log2(e) / sqrt(128)
  // tree
  const int32_t* page_table;
  const int32_t* pos;
  const int32_t* flag;
  const int32_t* parent;
  int64_t n_pages;
  int max_pages;
  float* part_o;                        // [2 grid][256][128]
  float* part_ml;                       // [2 grid][256][2]
  uint32_t* plan;                       // [n_seqs + 1] tiles before each sequence
};

// A CTA's unit of work: up to two slots of one KV head against a run of KV tiles.
struct Job {
  int b, h;            // sequence, KV head
  int row0;            // packed row of the sequence's first token or node
  int len;             // its tokens or nodes
  int tok0;            // first token of slot 0
  int n0, n1;          // valid tokens of each slot
  int first, sink;     // KV tile of step s: s == 0 && sink ? 0 : first + s - sink
  int steps0, steps1;  // steps of each slot (dual: of the job)
  int total;
  int dual;
  int cached;          // tree: cached positions; prompt: unused
  int node_tile;       // tree: the KV tile that holds the nodes; prompt: -1
  int direct;          // result complete: write out, else a partial
  int part;            // partial slot
};
struct Smem {
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_ready[2][2], o_full[2];
  uint64_t m_ready, m_done;
  uint64_t job_full[kAhead], job_empty[kAhead];
  float pair[2][kTile];                 // what the two threads of a row tell each other
  float join_m[kTile];                  // slot 1's references where the slots are joined (sums: in pair)
  Job jobs[kAhead];
  uint32_t tmem;
  uint32_t pref[ODA_MAX_BATCH + 1];     // prompt: blocks of each sequence; tree: tiles before it
};
constexpr int kTileBytes = (2 + kStages) * kStageBytes;   // Q slots, then K and V stages
// A V tile in shared memory, one half of 64 dims behind the other.  Prompts: halves of 128 positions.  Trees: a
// page's 16 positions, both halves, one page behind the other, so that a page comes in one copy.  (K tiles, whose
// 8-row groups have to lie evenly, are halves of 128 positions in both.)
template <bool TREE>
constexpr int kVHalf = TREE ? 2048 : kHalf;
template <bool TREE>
constexpr int kV16 = TREE ? 4096 : 2048;  // bytes from 16 positions to the next
constexpr int kDynBytes = kTileBytes + sizeof(Smem);
static_assert(kDynBytes <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ int kv_tile(const Job& j, int s) { return (j.sink && s == 0) ? 0 : j.first + s - j.sink; }
// Place of a step's K and V tile in the job's order of use: K0 | V0 K1 | V1 K2 ..., and where the slots
// alternate on the tiles of one, whose products with V come two steps later, K0 | K1 | V0 K2 | V1 K3 ...
__device__ __forceinline__ uint32_t order_k(const Job& j, int s) { return j.dual && s > 0 ? 2 * s - 1 : 2 * s; }
__device__ __forceinline__ uint32_t order_v(const Job& j, int s) { return j.dual && s < j.total - 1 ? 2 * s + 2 : 2 * s + 1; }
__device__ __forceinline__ int slot_steps(const Job& j, int i) { return j.dual ? (j.total + 1 - i) >> 1 : i ? j.steps1 : j.steps0; }

__device__ __forceinline__ int seq_len(const TileParams& p, int b, int most, bool report) {
  const int a = p.cu[b], e = p.cu[b + 1];
  if (a < 0 || e < a || (int64_t)e > p.n_rows || e - a > most) {
    if (report) atomicOr(p.err, ODA_DEVERR_ROW_RANGE);
    return 0;
  }
  return e - a;
}

// Prompt work: block j of a sequence is its tokens [2 nt j, 2 nt (j + 1)); units are (block, KV head),
// ordered by falling block index over all sequences (the longest rows first), KV heads innermost.
// pref holds every sequence's block count.  Called by a whole warp.  (Loops are kept rolled: a CTA
// runs this code before its first copy, at the pace of its instruction fetch.)
__device__ __forceinline__ uint32_t blocks_from(const Smem& sm, int n_seqs, uint32_t j, int lane) {
  uint32_t s = 0;
#pragma unroll 1
  for (int b = lane; b < n_seqs; b += 32) s += sm.pref[b] > j ? sm.pref[b] - j : 0u;
  return __reduce_add_sync(0xffffffffu, s);
}

__device__ __forceinline__ bool prompt_job(const TileParams& p, const Smem& sm, uint32_t id, uint32_t total, uint32_t most,
                                           int lane, Job& jb) {
  const uint32_t rank = id / (uint32_t)p.Hkv;
  if (rank >= total) return false;
  // the block index: blocks_from(lo) > rank >= blocks_from(hi) = behind
  uint32_t lo = 0, hi = most, behind = 0;
  if (p.n_seqs == 1) {
    lo = total - 1 - rank;
    behind = rank;
  } else {
#pragma unroll 1
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) >> 1, f = blocks_from(sm, p.n_seqs, mid, lane);
      if (f > rank) lo = mid;
      else hi = mid, behind = f;
    }
  }
  uint32_t k = rank - behind;            // the k-th of the sequences that have this block
  int b = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
    const uint32_t here = __ballot_sync(0xffffffffu, b0 + lane < p.n_seqs && sm.pref[b0 + lane] > lo);
    const uint32_t cnt = __popc(here);
    if (k < cnt) {
      const bool it = ((here >> lane) & 1u) && __popc(here & ((1u << lane) - 1u)) == (int)k;
      b = b0 + __ffs((int)__ballot_sync(0xffffffffu, it)) - 1;
      break;
    }
    k -= cnt;
  }
  jb.b = b;
  jb.h = (int)(id % (uint32_t)p.Hkv);
  jb.row0 = p.cu[b];
  jb.len = p.cu[b + 1] - jb.row0;
  jb.tok0 = (int)lo * 2 * p.nt;
  jb.n0 = min(p.nt, jb.len - jb.tok0);
  jb.n1 = max(0, min(p.nt, jb.len - jb.tok0 - p.nt));
  jb.first = 0;
  if (p.local && jb.tok0 >= p.window) jb.first = (jb.tok0 - p.window + 1) / kTile;
  jb.sink = (p.local && p.sinks > 0 && jb.first > 0) ? 1 : 0;
  jb.steps0 = (jb.tok0 + jb.n0 - 1) / kTile - jb.first + 1 + jb.sink;
  jb.steps1 = jb.n1 > 0 ? (jb.tok0 + p.nt + jb.n1 - 1) / kTile - jb.first + 1 + jb.sink : 0;
  jb.total = max(jb.steps0, jb.steps1);
  jb.dual = jb.n1 == 0 && jb.total > 1;
  jb.node_tile = -1;
  jb.cached = 0;
  jb.direct = 1;
  jb.part = 0;
  return true;
}

// Tree work: sequence b has M = ceil(nodes / 2 nt) units per KV head, each of `tiles` KV tiles
// (the cached positions', then one for the nodes).  All tiles of all units, in the order
// (sequence, KV head, unit), are cut into equal runs, one for each CTA; `at` walks this CTA's run.
__device__ __forceinline__ bool tree_job(const TileParams& p, const Smem& sm, uint32_t& at, uint32_t begin,
                                         uint32_t end, Job& jb) {
  if (at >= end) return false;
  int lo = 0, hi = p.n_seqs;             // pref[lo] <= at < pref[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sm.pref[mid] <= at) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  jb.b = b;
  jb.row0 = p.cu[b];
  jb.len = p.cu[b + 1] - jb.row0;
  jb.cached = p.pos[b] - 1;
  const uint32_t tiles = (uint32_t)((jb.cached + kTile - 1) / kTile + 1);
  const uint32_t M = (uint32_t)((jb.len + 2 * p.nt - 1) / (2 * p.nt));
  const uint32_t rel = at - sm.pref[b];
  const uint32_t u = rel / tiles, j0 = rel - u * tiles;
  const uint32_t j1 = min(tiles, j0 + (end - at));
  jb.h = (int)(u / M);
  jb.tok0 = (int)(u % M) * 2 * p.nt;
  jb.n0 = min(p.nt, jb.len - jb.tok0);
  jb.n1 = max(0, min(p.nt, jb.len - jb.tok0 - p.nt));
  jb.first = (int)j0;
  jb.sink = 0;
  jb.total = (int)(j1 - j0);
  jb.steps0 = jb.total;
  jb.steps1 = jb.n1 > 0 ? jb.total : 0;
  jb.dual = jb.n1 == 0 && jb.total > 1;
  jb.node_tile = (int)tiles - 1;
  jb.direct = j0 == 0 && j1 == tiles;
  jb.part = 2 * (int)blockIdx.x + (at == begin ? 0 : 1);
  at += j1 - j0;
  return true;
}

// Walks the CTA's units; the planning warp's.
template <bool TREE>
struct Walk {
  uint32_t at = 0, begin = 0, end = 0;   // tree: the CTA's run of tiles
  uint32_t total = 0, most = 0, turn = 0;  // prompt: blocks of all sequences, and of the longest
  __device__ Walk(const TileParams& p, const Smem& sm, int lane) {
    if (TREE) {
      const uint32_t W = sm.pref[p.n_seqs];
      const uint32_t share = (W + gridDim.x - 1) / gridDim.x;
      begin = min(W, share * blockIdx.x);
      end = min(W, begin + share);
      at = begin;
    } else {
#pragma unroll 1
      for (int b = lane; b < p.n_seqs; b += 32) {
        total += sm.pref[b];
        most = max(most, sm.pref[b]);
      }
      total = __reduce_add_sync(0xffffffffu, total);
      most = __reduce_max_sync(0xffffffffu, most);
    }
  }
  __device__ bool next(const TileParams& p, const Smem& sm, int lane, Job& j) {
    if (TREE) return tree_job(p, sm, at, begin, end, j);
    // the units fall in cost: odd turns go the other way round the CTAs, so that none gets the
    // longest of every turn
    const uint32_t id = turn * gridDim.x + ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    ++turn;
    return prompt_job(p, sm, id, total, most, lane, j);
  }
};

// Low `n` bits (n may be <= 0 or >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Nodes that node `i` of a tree of at most 64 sees: its ancestors and itself.
__device__ __forceinline__ uint64_t ancestors(const int32_t* parent, int i, int32_t* err) {
  uint64_t m = 0;
  while (true) {
    m |= 1ull << i;
    const int up = parent[i];
    if (up < -1 || up >= i) {
      atomicOr(err, ODA_DEVERR_ROW_RANGE);
      break;
    }
    if (up < 0) break;
    i = up;                              // falls at every turn: at most 64 turns
  }
  return m;
}

__device__ __forceinline__ void pin16(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}
// Keeps what reads registers loaded from TMEM behind the wait for that load.
__device__ __forceinline__ void pin32(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// N = 16 or 32 columns of TMEM, arrived.
template <int N>
__device__ __forceinline__ void load_cols(uint32_t* v, uint32_t at) {
  if constexpr (N == 16) tmem_ld16(v, at);
  else tmem_ld32(v, at);
  tmem_wait_ld();
  if constexpr (N == 16) pin16(v);
  else pin32(v);
}

// 2^x of a pair on the FMA pipe: x = n + f with n whole and |f| <= 1/2, 2^f by the cubic of least
// relative error on that range (7.5e-5, fitted by reweighted least squares; the weights are then
// rounded to bf16, 3.9e-3), times 2^n made of its exponent's bits.  x is held at -127 from below, where those are 0:
// a masked column's weight is 0, like the exponential unit's.
__device__ __forceinline__ void exp2_pair(uint64_t x2, float& a, float& b) {
  f32x2_split(x2, a, b);
  x2 = f32x2(fmaxf(a, -127.f), fmaxf(b, -127.f));
  const float kRound = 12583039.f;       // 1.5 * 2^23 + 127: adding it leaves n + 127 in the low bits
  const uint64_t t2 = add_f32x2(x2, f32x2(kRound, kRound));
  const uint64_t n2 = add_f32x2(t2, f32x2(-kRound, -kRound));
  const uint64_t f2 = fma_f32x2(n2, f32x2(-1.f, -1.f), x2);
  uint64_t y2 = fma_f32x2(f2, f32x2(0.05517132f, 0.05517132f), f32x2(0.24261054f, 0.24261054f));
  y2 = fma_f32x2(y2, f2, f32x2(0.69326099f, 0.69326099f));
  y2 = fma_f32x2(y2, f2, f32x2(0.99992811f, 0.99992811f));
  float ta, tb;
  f32x2_split(t2, ta, tb);
  y2 = mul_f32x2(y2, f32x2(__uint_as_float(__float_as_uint(ta) << 23), __uint_as_float(__float_as_uint(tb) << 23)));
  f32x2_split(y2, a, b);
}

// Weights 2^(c v - mc) of 32 columns as bf16 pairs, which take the scores' registers, and their sums
// (unrounded) added to s0, s1.  The exponential unit makes 16 a clock and SM, 2048 clocks for the two
// slots' tiles, as long as the tile's products: one pair in kPoly goes to the FMA pipe.
__device__ __forceinline__ void weights(uint32_t* v, uint64_t c2, uint64_t mc2, uint64_t& s0, uint64_t& s1) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t x2 = fma_f32x2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, mc2);
    float a, b;
    if (e % kPoly == kPoly - 1) {
      exp2_pair(x2, a, b);
    } else {
      f32x2_split(x2, a, b);
      a = exp2_approx(a);
      b = exp2_approx(b);
    }
    if (e & 1) s1 = add_f32x2(s1, f32x2(a, b));
    else s0 = add_f32x2(s0, f32x2(a, b));
    v[e] = cvt_bf16x2(a, b);
  }
}

// The two warps that share 32 rows meet: plainly, or with the OR of a predicate.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_or(int id, bool x) {
  uint32_t y;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.or.pred q, %1, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(y) : "r"(id), "r"((uint32_t)x) : "memory");
  return y != 0;
}

// Masked ones of 32 scores to -inf.
__device__ __forceinline__ void mask32(uint32_t* v, uint32_t seen) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (!((seen >> e) & 1u)) v[e] = 0xff800000u;
}

// Writes one line of N 16-byte chunks (N = 2 or 4; 4 N registers) per lane, line `line` of L of row `row` of dst
// (row < 0: none), N lanes to a line: an N x N transpose of chunks among each N lanes, then 32 / N whole
// lines a store.  A lane writing its own line would touch 32 lines in every store.
template <int N, int L>
__device__ __forceinline__ void store_lines(uint32_t* v, uint4* dst, int row, int line, int lane) {
#pragma unroll
  for (int bit = 1; bit < N; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (c & bit) continue;             // chunks c and c | bit: one of them goes to the partner lane
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t give = up ? v[4 * c + w] : v[4 * (c | bit) + w];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, bit);
        if (up) v[4 * c + w] = got;
        else v[4 * (c | bit) + w] = got;
      }
    }
  }
  // now chunk j of this lane is chunk (lane mod N) of the line of the j-th of its N lanes
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int to = __shfl_sync(0xffffffffu, row, (lane & ~(N - 1)) + j);
    if (to >= 0) dst[(int64_t)to * (L * N) + line * N + (lane & (N - 1))] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  }
}

template <bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
tile_attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mkn,
                      const __grid_constant__ CUtensorMap mvn, const TileParams p) {
  extern __shared__ __align__(1024) uint8_t dyn[];
  Smem& sm = *reinterpret_cast<Smem*>(dyn + kTileBytes);
  uint8_t* sq = dyn;                                    // two slots of Q
  uint8_t* skv = dyn + 2 * kStageBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_ready[i][0], 4);
      mbar_init(&sm.p_ready[i][1], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.m_ready, 8);
    mbar_init(&sm.m_done, 8);
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&sm.job_full[i], 1);
      mbar_init(&sm.job_empty[i], 19);
    }
    fence_mbar_init();
  }
  if (warp == kWarpMma) tmem_alloc(&sm.tmem, 512);
  if (TREE) {
    // tiles before each sequence: one warp, 32 sequences at a time
    if (warp == kWarpLoad) {
      uint32_t run = 0;
      for (int b0 = 0; b0 < p.n_seqs; b0 += 32) {
        const int b = b0 + lane;
        uint32_t w = 0;
        if (b < p.n_seqs && (!p.flag || p.flag[b] != 0)) {
          const int n = seq_len(p, b, ODA_MAX_TREE, blockIdx.x == 0);
          const int t = p.pos[b];
          const bool ok = t >= 1 && (int64_t)(t - 1) <= (int64_t)p.max_pages * 16;
          if (!ok && blockIdx.x == 0) atomicOr(p.err, ODA_DEVERR_POS_RANGE);
          if (ok && n > 0)
            w = (uint32_t)((t - 1 + kTile - 1) / kTile + 1) * (uint32_t)((n + 2 * p.nt - 1) / (2 * p.nt)) * (uint32_t)p.Hkv;
        }
        uint32_t inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (b < p.n_seqs) sm.pref[b] = run + inc - w;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) sm.pref[p.n_seqs] = run;
      __syncwarp();
      if (blockIdx.x == 0)
        for (int b = lane; b <= p.n_seqs; b += 32) p.plan[b] = sm.pref[b];
    }
  } else {
    for (int b = tid; b < p.n_seqs; b += kThreads)
      sm.pref[b] = (uint32_t)((seq_len(p, b, 0x7fffffff, blockIdx.x == 0) + 2 * p.nt - 1) / (2 * p.nt));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  // Every role walks the planned units: waits for one, reads it where it lies, gives it back.
  uint32_t turn = 0;
  auto next_job = [&]() {                // false at the end, or where the wait gave up (ok)
    if (ok) ok = mbar_wait_bounded(&sm.job_full[turn % kAhead], (turn / kAhead) & 1, kWaitNs);
    return ok && sm.jobs[turn % kAhead].total > 0;
  };
  auto done_job = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.job_empty[turn % kAhead]);
    ++turn;
  };

  if (warp >= kWarpMma) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kWarpPlan) {
    Walk<TREE> walk(p, sm, lane);
    Job jb;
    for (uint32_t n = 0; ok; ++n) {
      const bool more = walk.next(p, sm, lane, jb);
      if (!more) jb.total = 0;
      const uint32_t at = n % kAhead;
      if (n >= kAhead) ok = mbar_wait_bounded(&sm.job_empty[at], (n / kAhead - 1) & 1, kWaitNs);
      if (ok && lane == 0) {
        sm.jobs[at] = jb;
        mbar_arrive(&sm.job_full[at]);
      }
      __syncwarp();
      if (!more) break;
    }
  } else if (warp == kWarpLoad || warp == kWarpLoadV) {
    // ------------------------------------------------------------------ loads
    const int w = warp == kWarpLoadV;    // K or V tiles
    uint32_t gs = 0, jobs = 0;           // KV tiles (K, V counted apart: 2 gs) and jobs so far
    const int pg = (lane >> 1) & 7, hf = lane & 1;      // tree: lanes 0-15 bring 8 pages x 2 halves
    while (next_job()) {
      const Job& jb = sm.jobs[turn % kAhead];
      // the page-table entries are read a tile ahead of the copies that wait for them
      auto entry = [&](int t) {
        const int at = t * 8 + pg;
        return t < jb.node_tile && at * 16 < jb.cached ? p.page_table[(size_t)jb.b * p.max_pages + at] : -1;
      };
      int phys = TREE ? entry(jb.first) : 0;
      if (w == 0) {
        if (jobs > 0) ok = mbar_wait_bounded(&sm.q_empty, (jobs - 1) & 1, kWaitNs);
        if (!ok) break;
        const int slots = jb.n1 > 0 ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(&sm.q_full, (uint32_t)(slots * 2 * 128 * p.g * p.nt));
        if (TREE) {
          // A copy a lane (4 nt / nq <= 32 of them): nq nodes' half rows.  Those behind the tree's last node come
          // from behind the last row, as zeros: rows of zeros cost the tensor cores less power, and the
          // power cap holds the clock (32 sequences, 16 nodes, on a GPU at its cap: 464 -> 440 us).
          __syncwarp();
          const int each = p.nt / p.nq, i = lane / (2 * each), part = (lane >> 1) % each, tok = jb.tok0 + i * p.nt + part * p.nq;
          if (i < slots)
            tma_load_3d(sq + i * kStageBytes + (lane & 1) * kHalf + part * p.nq * p.g * 128, &mq, (lane & 1) * 64, jb.h * p.g,
                        tok < jb.len ? jb.row0 + tok : (int)p.n_rows, &sm.q_full);
        } else if (lane == 0) {
          for (int i = 0; i < slots; ++i)
            for (int h2 = 0; h2 < 2; ++h2)
              tma_load_3d(sq + i * kStageBytes + h2 * kHalf, &mq, h2 * 64, jb.h * p.g, jb.row0 + jb.tok0 + i * p.nt,
                          &sm.q_full);
        }
      }
      ++jobs;
      for (int s = 0; s < jb.total; ++s) {
        const int t = kv_tile(jb, s);
        const int page = phys;
        if (TREE) phys = entry(t + 1);
        const uint32_t n = 2 * gs + (w ? order_v(jb, s) : order_k(jb, s)), st = n % kStages;
        if (n >= kStages) ok = mbar_wait_bounded(&sm.kv_empty[st], (n / kStages - 1) & 1, kWaitNs);
        if (!ok) break;
        uint8_t* dst = skv + st * kStageBytes;
        if (!TREE) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.kv_full[st], kStageBytes);
            for (int h2 = 0; h2 < 2; ++h2)
              tma_load_3d(dst + h2 * kHalf, w ? &mv : &mk, h2 * 64, jb.h, jb.row0 + t * kTile, &sm.kv_full[st]);
          }
        } else if (t == jb.node_tile) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&sm.kv_full[st], ODA_MAX_TREE * 256);
            if (w)
              for (int i = 0; i < ODA_MAX_TREE / 16; ++i)
                tma_load_4d(dst + i * kV16<TREE>, &mvn, 0, jb.row0 + 16 * i, 0, jb.h, &sm.kv_full[st]);
            else
              for (int h2 = 0; h2 < 2; ++h2) tma_load_3d(dst + h2 * kHalf, &mkn, h2 * 64, jb.h, jb.row0, &sm.kv_full[st]);
          }
        } else {
          const int pages = min(8, (jb.cached - t * kTile + 15) / 16);
          if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full[st], (uint32_t)(pages * 4096));
          __syncwarp();
          if (lane < 2 * pages && (w == 0 || hf == 0)) {
            int64_t row = ((int64_t)page * p.Hkv + jb.h) * 16;
            if (page < 0 || page >= p.n_pages) {
              atomicOr(p.err, ODA_DEVERR_PAGE_RANGE);
              row = p.n_pages * p.Hkv * 16;             // past the pool: the copy fills zeros
            }
            if (w) tma_load_3d(dst + pg * kV16<TREE>, &mv, 0, (int32_t)row, 0, &sm.kv_full[st]);
            else tma_load_2d(dst + hf * kHalf + pg * 2048, &mk, hf * 64, (int32_t)row, &sm.kv_full[st]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      gs += jb.total;
      done_job();
    }
    if (!ok) {
      // gave up: let the copies in flight (microseconds) land before the CTA ends
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {
      }
    }
  } else if (warp == kWarpMma) {
    // --------------------------------------------------------------- products
    // One thread for both slots in turn, which keeps them half a period apart: with a warp for each
    // the slots fall into step, and the tensor cores idle while both make weights.  What it runs between
    // two products lies on the path from weights to scores, at some 8 clocks an instruction: one
    // thread alone (no votes), running stage and phase numbers, descriptors made once.
    if (elect_one()) {
      constexpr uint32_t kIdS = mma_idesc_bf16(128, 128, false), kIdO = mma_idesc_bf16(128, 128, true);
      const uint64_t dq = smem_desc(smem_u32(sq), 16, 1024), dk = smem_desc(smem_u32(skv), 16, 1024);
      const uint64_t dv = smem_desc(smem_u32(skv), kVHalf<TREE>, 1024);
      constexpr uint32_t kV = kV16<TREE> >> 4;
      constexpr uint32_t kStep = kStageBytes >> 4;  // of a descriptor's address
      uint32_t st = 0, ph = 0;                      // stage and phase of the next tile in the order of use
      uint32_t np0 = 0, np1 = 0, jobs = 0;          // parity of each slot's weights consumed; of the jobs
      // O_i += P_i V: the first 64 weights of every row, then the others; nk = 16-row steps of the tile
      auto pv = [&](int i, uint32_t& np, uint32_t at, bool acc, int nk) {
        const uint32_t tS = tmem + kColS + i * 128, tO = tmem + kColO + i * 128;
        const uint64_t bv = dv + at * kStep;
        ok = mbar_wait_bounded(&sm.p_ready[i][0], np, kWaitNs);
        if (!ok) return;
        tc_fence_after();
        if (nk == 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16_ts(tO, tS + k * 8, bv + k * kV, kIdO, acc || k > 0);
        } else {
#pragma unroll 1
          for (int k = 0; k < min(nk, 4); ++k) mma_f16_ts(tO, tS + k * 8, bv + k * kV, kIdO, acc || k > 0);
        }
        ok = mbar_wait_bounded(&sm.p_ready[i][1], np, kWaitNs);
        np ^= 1;
        if (!ok) return;
        tc_fence_after();
        if (nk == 8) {
#pragma unroll
          for (int k = 4; k < 8; ++k) mma_f16_ts(tO, tS + 32 + k * 8, bv + k * kV, kIdO, true);
        } else {
#pragma unroll 1
          for (int k = 4; k < nk; ++k) mma_f16_ts(tO, tS + 32 + k * 8, bv + k * kV, kIdO, true);
        }
      };
      // S_i = Q K^T of the tile's first 16 nk positions
      auto qk = [&](int i, uint64_t aq, uint32_t at, int nk) {
        const uint64_t bk = dk + at * kStep;
        const uint32_t id = kIdS - ((uint32_t)(8 - nk) << 18);               // N = 16 nk
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t off = (k >> 2) * (kHalf >> 4) + (k & 3) * 2;
          mma_f16_ss(tmem + kColS + i * 128, aq + off, bk + off, id, k > 0);
        }
        mma_commit(&sm.s_full[i]);
      };
      auto next = [&] {
        if (++st == kStages) st = 0, ph ^= 1;
      };
      while (next_job()) {
        const Job& jb = sm.jobs[turn % kAhead];
        const int total = jb.total, steps0 = jb.steps0, steps1 = jb.steps1;
        const bool dual = jb.dual != 0;
        // valid rows of the last V tile and of the one before it
        const int ends = jb.first + total - jb.sink;                // behind the last tile
        const int valid1 = TREE ? (ends > jb.node_tile ? jb.len : jb.cached - (ends - 1) * kTile) : jb.len - (ends - 1) * kTile;
        const int valid2 = TREE ? jb.cached - (ends - 2) * kTile : kTile;
        const int nk1 = min(8, (valid1 + 15) >> 4), nk2 = min(8, (valid2 + 15) >> 4);
        const uint64_t aq1 = dq + (dual ? 0 : kStep);
        ok = mbar_wait_bounded(&sm.q_full, jobs, kWaitNs);
        jobs ^= 1;
        const int lag = dual ? 2 : 1, end = total + lag;
        // steps at which both slots have a product of each kind and whole tiles
        const int even0 = !TREE && jb.sink ? 2 : 1, even1 = dual ? 0 : min(min(steps0, steps1), total) - 1;
        // Prompts: 16-position steps of a slot's last tile up to its last token, and of the sinks' tile 1.  The other
        // scores are whatever lies there, and masked.  (8191 tokens, local set: 271 -> 267 us; 8 short prompts: 15.4 ->
        // 14.7 us.)
        const int nkq0 = TREE ? 8 : min(8, (jb.tok0 + jb.n0 - (jb.first + steps0 - 1 - jb.sink) * kTile + 15) >> 4);
        const int nkq1 = TREE || steps1 == 0 ? 8 : min(8, (jb.tok0 + p.nt + jb.n1 - (jb.first + steps1 - 1 - jb.sink) * kTile + 15) >> 4);
        auto steps_of = [&](int i, int t) {              // of slot i in step t
          if (TREE) return 8;
          if (t == 0 && jb.sink) return 1;
          if (dual) return t == total - 1 ? nkq0 : 8;
          return t == (i ? steps1 : steps0) - 1 ? (i ? nkq1 : nkq0) : 8;
        };
        for (int s = 0; s < end && ok; ++s) {
          if (s >= even0 && s < even1) {
            const uint32_t vs = st;
            ok = mbar_wait_bounded(&sm.kv_full[st], ph, kWaitNs);
            if (ok) pv(0, np0, vs, s > 1, 8);
            next();
            if (ok) ok = mbar_wait_bounded(&sm.kv_full[st], ph, kWaitNs);
            if (!ok) break;
            qk(0, dq, st, 8);
            pv(1, np1, vs, s > 1, 8);
            if (!ok) break;
            qk(1, aq1, st, 8);
            mma_commit(&sm.kv_empty[vs]);
            mma_commit(&sm.kv_empty[st]);
            next();
            continue;
          }
          const int sp = s - lag;
          const bool hasV = sp >= 0, hasK = s < total;
          const int nk = sp == total - 1 ? nk1 : sp == total - 2 ? nk2 : 8;
          uint32_t vs = 0, ks = 0, kph = 0;
          bool kwait = hasK;
          if (hasV) {
            vs = st;
            ok = mbar_wait_bounded(&sm.kv_full[st], ph, kWaitNs);
            next();
          }
          if (hasK) {
            ks = st;
            kph = ph;
            next();
          }
#pragma unroll 1
          for (int i = 0; i < 2 && ok; ++i) {
            const int steps = i ? steps1 : steps0;
            const bool turn_i = (s & 1) == i;
            if (hasV && (dual ? turn_i : sp < steps)) {
              uint32_t np = i ? np1 : np0;
              pv(i, np, vs, dual ? sp >= 2 : sp > 0, min(nk, steps_of(i, sp)));
              if (i) np1 = np;
              else np0 = np;
              if (!ok) break;
              if (dual ? s >= total : s >= steps) mma_commit(&sm.o_full[i]);   // the slot's last
            }
            if (hasK && (dual ? turn_i : s < steps)) {
              if (kwait) ok = mbar_wait_bounded(&sm.kv_full[ks], kph, kWaitNs);
              kwait = false;
              if (ok) qk(i, i ? aq1 : dq, ks, steps_of(i, s));
            }
          }
          if (!ok) break;
          if (hasV) mma_commit(&sm.kv_empty[vs]);
          if (hasK) mma_commit(&sm.kv_empty[ks]);
          if (s == total - 1) mma_commit(&sm.q_empty);
        }
        if (!ok) break;
        mbar_arrive(&sm.job_empty[turn % kAhead]);
        ++turn;
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
      // gave up: let the products in flight (microseconds) finish before TMEM is freed
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {
      }
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRow));
    // ---------------------------------------------------------------- weights
    const int i = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
    const int meet = 1 + i * 4 + (warp & 3);     // barrier of the two warps of these rows
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + kColS + i * 128 + half * 64;
    const uint32_t tO = tmem + lane_base + kColO + i * 128 + half * 64;
    const int tok = r / p.g;
    uint32_t ns = 0, no = 0, duals = 0;          // scores, results and joins of this slot so far
    uint32_t gs = 0;                             // KV tiles of the jobs before
    while (true) {
      const bool more = next_job();
      if (pair_or(meet, !ok) || !more) break;    // both warps of a pair go on, or neither
      const Job& jb = sm.jobs[turn % kAhead];
      const int mine = jb.dual ? 0 : i;          // slot whose rows these are
      const int place = jb.tok0 + mine * p.nt + tok;
      const bool row_ok = tok < (mine ? jb.n1 : jb.n0);
      // a warp without rows (small trees) only keeps the barriers' counts; its rows of P are whatever lies
      // there, and its rows of O are never read (32 sequences, 16 nodes: 494 -> 456 us; prompts, which rarely
      // have such warps, lose 3% to the registers it takes)
      const bool idle = TREE && !__any_sync(0xffffffffu, row_ok);
      uint64_t anc = 0;
      if (TREE && row_ok && jb.first + jb.total > jb.node_tile) anc = ancestors(p.parent + jb.row0, place, p.err);
      const int cnt = slot_steps(jb, i);
      // Rows behind the sequence in its last V tiles hold another one's values or old ones: their
      // weights are 0, and 0 * NaN must not reach the sums.  Steps of 16 such rows are left out of the
      // product; the rows of the last step are cleared here (by both slots: the same zeros).
      auto clear_behind = [&](int t0, int x) {
        const int valid = TREE ? (t0 >= jb.node_tile * kTile ? jb.len : jb.cached - t0) : jb.len - t0;
        if (valid >= kTile || !(valid & 15)) return;
        const uint32_t n = 2 * gs + order_v(jb, jb.dual ? 2 * x + i : x), st = n % kStages;
        if (ok) ok = mbar_wait_bounded(&sm.kv_full[st], (n / kStages) & 1, kWaitNs);
        const int rows = 16 - (valid & 15);
        for (int z = half * kTile + r; z < rows * 16; z += 2 * kTile) {
          const int row = valid + (z >> 4), ch = z & 15;
          const int at = TREE ? (row >> 4) * kV16<TREE> + (row & 15) * 128 : row * 128;
          *reinterpret_cast<uint4*>(skv + st * kStageBytes + (ch >> 3) * kVHalf<TREE> + at + (ch & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      };
      float m = -INFINITY, l = 0.f;
      for (int x = 0; x < cnt; ++x) {
        if (idle) {
          if (ok) ok = mbar_wait_bounded(&sm.s_full[i], ns & 1, kWaitNs);
          ++ns;
          clear_behind(kv_tile(jb, jb.dual ? 2 * x + i : x) * kTile, x);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[i][half]);
          continue;
        }
        // ---- which of this thread's columns the row sees
        const int t0 = kv_tile(jb, jb.dual ? 2 * x + i : x) * kTile, c0 = t0 + half * 64;
        uint32_t mw0, mw1;
        if (TREE) {
          if (t0 >= jb.node_tile * kTile) {
            mw0 = half ? 0u : (uint32_t)anc;
            mw1 = half ? 0u : (uint32_t)(anc >> 32);
          } else {
            mw0 = low_bits(jb.cached - c0);
            mw1 = low_bits(jb.cached - c0 - 32);
          }
        } else {
          mw0 = low_bits(place + 1 - c0);
          mw1 = low_bits(place + 1 - c0 - 32);
          if (p.local) {
            mw0 &= ~low_bits(place - p.window + 1 - c0) | low_bits(p.sinks - c0);
            mw1 &= ~low_bits(place - p.window + 1 - c0 - 32) | low_bits(p.sinks - c0 - 32);
          }
        }
        const bool masked = __any_sync(0xffffffffu, (mw0 & mw1) != 0xffffffffu);
        if (ok) ok = mbar_wait_bounded(&sm.s_full[i], ns & 1, kWaitNs);
        ++ns;
        tc_fence_after();
        // ---- the maximum
        uint32_t v[64];
        tmem_ld32(v, tS);
        tmem_ld32(v + 32, tS + 32);
        tmem_wait_ld();
        pin32(v);
        pin32(v + 32);
        if (masked) {
          mask32(v, mw0);
          mask32(v + 32, mw1);
        }
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          top0 = max3(top0, __uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]));
          top1 = max3(top1, __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
        }
        const float top = max3(top0, top1, top1);
        // also the first finite value (m = -inf), and a NaN that the row sees, which stays the reference
        const bool grow = row_ok && !(top * p.c <= m * p.c + kGrow);
        if (pair_or(meet, grow)) {
          if (half) sm.pair[i][r] = top;
          pair_sync(meet);
          if (!half) {
            const float nm = max3(m, top, sm.pair[i][r]);
            sm.pair[i][r] = nm < INFINITY ? nm : NAN;    // +inf has no finite weight beside it
          }
          pair_sync(meet);
          const float nm = sm.pair[i][r];
          const float al = m == nm ? 1.f : exp2_approx((m - nm) * p.c);
          m = nm;
          l *= al;
          if (x > 0) {
            // these scores were issued after the slot's previous product, so that one is in O
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t w[16];
              tmem_ld16(w, tO + 16 * q);
              tmem_wait_ld();
              pin16(w);
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * al);
              tmem_st16(tO + 16 * q, w);
            }
          }
        }
        clear_behind(t0, x);
        // ---- weights
        const float mc = m == -INFINITY ? 0.f : m * p.c;
        const uint64_t c2 = f32x2(p.c, p.c), mc2 = f32x2(-mc, -mc);
        uint64_t s0 = f32x2(l, 0.f), s1 = f32x2(0.f, 0.f);
        weights(v, c2, mc2, s0, s1);
        tmem_st16(tS, v);
        weights(v + 32, c2, mc2, s0, s1);
        tmem_st16(tS + 16, v + 32);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[i][half]);
        float a, b;
        f32x2_split(add_f32x2(s0, s1), a, b);
        l = a + b;
      }
      // ---- the slot's result
      if (cnt > 0) {
        if (ok) ok = mbar_wait_bounded(&sm.o_full[i], no & 1, kWaitNs);
        ++no;
        tc_fence_after();
        if (!idle) {
          if (half) sm.pair[i][r] = l;
          pair_sync(meet);
          if (!half) sm.pair[i][r] += l;
          pair_sync(meet);
          l = sm.pair[i][r];
        }
      }
      float a0 = 1.f, a1 = 0.f;                  // factors of O0 and O1
      if (jb.dual) {
        if (i == 1) {
          if (!half) sm.join_m[r] = m;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.m_ready);
          if (ok) ok = mbar_wait_bounded(&sm.m_done, duals & 1, kWaitNs);
          ++duals;
          tc_fence_after();
          gs += jb.total;
          done_job();
          continue;
        }
        if (ok) ok = mbar_wait_bounded(&sm.m_ready, duals & 1, kWaitNs);
        ++duals;
        tc_fence_after();
        const float m1 = sm.join_m[r], nm = fmaxf(m, m1);
        a0 = m == nm ? 1.f : exp2_approx((m - nm) * p.c);
        a1 = m1 == nm ? 1.f : exp2_approx((m1 - nm) * p.c);
        m = nm;
        l = l * a0 + sm.pair[1][r] * a1;
      }
      if (cnt > 0 && !idle) {
        if (jb.direct) {
          const float inv = m > -INFINITY ? __fdividef(1.f, l) : NAN;   // (every score -inf: no weights)
          a0 *= inv;
          a1 *= inv;
        }
        // Prompts: 32 columns at a time, 64-byte lines.  Trees: 16, lines of 32 bytes of bf16 or 64 of a fp32
        // partial; a CTA has few units, so it meets this code cold, and half of it is fetched sooner (a tree of 5
        // over 4096: 21.7 -> 20.0 us; prompts lose 0.4 us of 9).
        constexpr int kCols = TREE ? 16 : 32, kLines = 128 / kCols;
        const int at = !row_ok ? -1 : jb.direct ? (jb.row0 + place) * p.Hq + jb.h * p.g + (r - tok * p.g)
                                                : jb.part * 256 + mine * 128 + r;
        if (row_ok && !jb.direct && !half) reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(m, l);
#pragma unroll 1
        for (int q = 0; q < kLines / 2; ++q) {
          uint32_t o[kCols];
          load_cols<kCols>(o, tO + kCols * q);
#pragma unroll
          for (int e = 0; e < kCols; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a0);
          if (jb.dual) {
            uint32_t o1[kCols];
            load_cols<kCols>(o1, tO + 128 + kCols * q);
#pragma unroll
            for (int e = 0; e < kCols; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(o1[e]) * a1);
          }
          const int line = half * (kLines / 2) + q;
          if (!TREE || jb.direct) {
#pragma unroll
            for (int e = 0; e < kCols / 2; ++e) o[e] = cvt_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            store_lines<kCols / 8, kLines>(o, reinterpret_cast<uint4*>(p.out), at, line, lane);
          } else {
            store_lines<kCols / 4, kLines>(o, reinterpret_cast<uint4*>(p.part_o), at, line, lane);
          }
        }
        tc_fence_before();
      }
      if (jb.dual) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.m_done);
      }
      gs += jb.total;
      done_job();
    }
  }
  if (!ok && lane == 0) atomicOr(p.err, ODA_DEVERR_WAIT_TIMEOUT);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// Joins the partial results of the units that several CTAs shared: a warp per (node, query head), blockIdx =
// (node, group of 4 heads).
__global__ void __launch_bounds__(128) tree_join_kernel(const TileParams p, uint32_t grid) {
  grid_dependency_wait();
  const int row = blockIdx.x, lane = threadIdx.x & 31;
  int b = -1;                            // the sequence of this row, if it has tiles
#pragma unroll 1
  for (int b0 = 0; b0 < p.n_seqs && b < 0; b0 += 32) {
    const int x = b0 + lane;
    const uint32_t here = __ballot_sync(0xffffffffu, x < p.n_seqs && p.cu[x] <= row && row < p.cu[x + 1] &&
                                                         p.plan[x] != p.plan[x + 1]);
    if (here) b = b0 + __ffs((int)here) - 1;
  }
  if (b < 0) return;
  const uint32_t before = p.plan[b], W = p.plan[p.n_seqs];
  const int first = p.cu[b], len = p.cu[b + 1] - first, node = row - first, cached = p.pos[b] - 1;
  const uint32_t share = (W + grid - 1) / grid;
  const uint32_t tiles = (uint32_t)((cached + kTile - 1) / kTile + 1);
  const uint32_t M = (uint32_t)((len + 2 * p.nt - 1) / (2 * p.nt)), unit = (uint32_t)(node / (2 * p.nt));
  const int in = node % (2 * p.nt), r0 = (in / p.nt) * 128 + (in % p.nt) * p.g;
  {
    const int head = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (head >= p.Hq) return;
    const uint32_t h = (uint32_t)(head / p.g), us = before + (h * M + unit) * tiles, ue = us + tiles;
    const uint32_t c0 = us / share, c1 = (ue - 1) / share;
    if (c0 == c1) return;                                // one CTA had it all and wrote it
    const int r = r0 + head - (int)h * p.g;
    // partial of CTA c: its first unit's, or its last one's; a lane has the statistics of each 32nd
    auto part = [&](uint32_t c) { return (size_t)(us > c * share ? 2 * c + 1 : 2 * c) * 256 + r; };
    float m = -INFINITY;
    float2 ml = make_float2(-INFINITY, 0.f);
#pragma unroll 1
    for (uint32_t c = c0 + lane; c <= c1; c += 32) {
      ml = reinterpret_cast<const float2*>(p.part_ml)[part(c)];
      m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t c = c0; c <= c1; c += 32) {
      if (c1 - c0 >= 32) ml = c + lane <= c1 ? reinterpret_cast<const float2*>(p.part_ml)[part(c + lane)] : make_float2(-INFINITY, 0.f);
      const float w = ml.x == m ? 1.f : exp2_approx((ml.x - m) * p.c);
      l += w * ml.y;
      const int n = (int)min(32u, c1 - c + 1);
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const float4 o = reinterpret_cast<const float4*>(p.part_o)[part(c + j) * 32 + lane];
        acc.x += wj * o.x;
        acc.y += wj * o.y;
        acc.z += wj * o.z;
        acc.w += wj * o.w;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = m > -INFINITY ? __fdividef(1.f, l) : NAN;
    uint2 w;
    w.x = cvt_bf16x2(acc.x * inv, acc.y * inv);
    w.y = cvt_bf16x2(acc.z * inv, acc.w * inv);
    reinterpret_cast<uint2*>(p.out)[((size_t)row * p.Hq + head) * 32 + lane] = w;
  }
}

oda_status encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
  EncodeFn enc = get_encode();
  if (!enc) return set_error(ODA_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims,
                         strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return set_error(ODA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ODA_OK;
}

// Packed rows [n_rows][heads][128] with a row stride in elements: boxes of 64 values x `heads_box`
// heads x `rows_box` rows, which land in shared memory as rows of (row, head).
oda_status encode_rows(CUtensorMap* m, const void* ptr, int64_t n_rows, int heads, int64_t stride,
                       int heads_box, int rows_box) {
  const cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)n_rows};
  const cuuint64_t st[2] = {256, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box};
  return encode(m, ptr, 3, dims, st, box);
}

bool aligned16(const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15) == 0; }

}  // namespace

size_t tile_part_rows(int n_sms) { return (size_t)2 * n_sms * 256; }

oda_status prepare_tile_attention() {
  // the kernel moves registers between its warpgroups: the launch has to bring as many
  const void* f[2] = {reinterpret_cast<const void*>(tile_attention_kernel<false>),
                      reinterpret_cast<const void*>(tile_attention_kernel<true>)};
  for (const void* k : f) {
    cudaFuncAttributes fa;
    const oda_status a = check_cuda(cudaFuncGetAttributes(&fa, k), "cudaFuncGetAttributes(tile attention)");
    if (a != ODA_OK) return a;
    if (fa.numRegs < kRegs)
      return set_error(ODA_ERR_UNSUPPORTED, "tile attention: built with %d registers a thread", fa.numRegs);
  }
  oda_status st = check_cuda(cudaFuncSetAttribute(tile_attention_kernel<false>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes),
                             "cudaFuncSetAttribute(prompt attention)");
  if (st == ODA_OK)
    st = check_cuda(cudaFuncSetAttribute(tile_attention_kernel<true>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes),
                    "cudaFuncSetAttribute(tree attention)");
  return st;
}

oda_status launch_prompt(oda_ctx* ctx, int n_seqs, int64_t n_rows, const int32_t* cu_rows, const void* q,
                         const void* k, const void* v, int64_t q_stride, int64_t kv_stride, void* out, int local,
                         cudaStream_t stream) {
  const oda_config& cf = ctx->cfg;
  if (!cu_rows || !q || !k || !v || !out) return set_error(ODA_ERR_INVALID_ARG, "prompt: null pointer argument");
  if (n_seqs < 1 || n_seqs > ODA_MAX_BATCH)
    return set_error(ODA_ERR_INVALID_ARG, "prompt: n_seqs must be 1..%d", ODA_MAX_BATCH);
  if (n_rows < 1 || n_rows > INT32_MAX / cf.n_q_heads)
    return set_error(ODA_ERR_INVALID_ARG, "prompt: n_rows out of range (%lld)", (long long)n_rows);
  if (q_stride < (int64_t)cf.n_q_heads * 128 || kv_stride < (int64_t)cf.n_kv_heads * 128 || (q_stride & 7) ||
      (kv_stride & 7) || q_stride > (int64_t(1) << 32) || kv_stride > (int64_t(1) << 32))
    return set_error(ODA_ERR_INVALID_ARG, "prompt: row strides must cover the heads and be multiples of 8");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return set_error(ODA_ERR_INVALID_ARG, "prompt: q, k, v and out must be 16-byte aligned");
  ctx->prev_attention = false;
  TileParams p = {};
  p.cu = cu_rows;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = ctx->err;
  p.n_rows = n_rows;
  p.n_seqs = n_seqs;
  p.Hq = cf.n_q_heads;
  p.Hkv = cf.n_kv_heads;
  p.g = ctx->g;
  p.nt = kTile / ctx->g;
  p.local = local;
  p.sinks = cf.sinks;
  p.window = cf.window;
  p.c = (float)(1.4426950408889634 / std::sqrt(128.0));
  CUtensorMap mq, mk, mv;
  oda_status st = encode_rows(&mq, q, n_rows, cf.n_q_heads, q_stride, p.g, p.nt);
  if (st == ODA_OK) st = encode_rows(&mk, k, n_rows, cf.n_kv_heads, kv_stride, 1, kTile);
  if (st == ODA_OK) st = encode_rows(&mv, v, n_rows, cf.n_kv_heads, kv_stride, 1, kTile);
  if (st != ODA_OK) return st;
  const int64_t most = (n_rows / (2 * p.nt) + n_seqs) * cf.n_kv_heads;
  const int grid = (int)std::min<int64_t>(ctx->n_sms, most);
  tile_attention_kernel<false><<<grid, kThreads, kDynBytes, stream>>>(mq, mk, mv, mk, mv, p);
  return check_cuda(cudaGetLastError(), "prompt attention launch");
}

oda_status launch_tree(oda_ctx* ctx, const oda_kv_layer* layer, const int32_t* page_table, const int32_t* pos,
                       const int32_t* flag, int64_t n_rows, const int32_t* cu_rows, const int32_t* parent,
                       const void* q, const void* k_new, const void* v_new, void* out, cudaStream_t stream) {
  const oda_config& cf = ctx->cfg;
  if (!layer || !layer->k || !layer->v || !page_table || !pos || !cu_rows || !parent || !q || !k_new || !v_new || !out)
    return set_error(ODA_ERR_INVALID_ARG, "tree: null pointer argument");
  if (layer->n_pages <= 0 || layer->n_pages >= INT32_MAX / (cf.n_kv_heads * (int64_t)16))
    return set_error(ODA_ERR_INVALID_ARG, "tree: n_pages out of range (%lld)", (long long)layer->n_pages);
  if (n_rows < 1 || n_rows > (int64_t)cf.batch * ODA_MAX_TREE)
    return set_error(ODA_ERR_INVALID_ARG, "tree: n_rows must be 1..batch * %d", ODA_MAX_TREE);
  if (!aligned16(layer->k) || !aligned16(layer->v) || !aligned16(q) || !aligned16(k_new) || !aligned16(v_new) ||
      !aligned16(out))
    return set_error(ODA_ERR_INVALID_ARG, "tree: pools, q, k_new, v_new and out must be 16-byte aligned");
  TileParams p = {};
  p.nt = kTile / ctx->g;
  p.nq = p.nt % 16 ? p.nt : 16;
  const int64_t units = (ODA_MAX_TREE + 2 * p.nt - 1) / (2 * p.nt);
  if ((int64_t)cf.batch * cf.n_kv_heads * units * ((cf.max_pages + 7) / 8 + 1) > (int64_t)INT32_MAX)
    return set_error(ODA_ERR_UNSUPPORTED, "tree: batch * KV heads * max_pages beyond the tile count");
  ctx->prev_attention = false;
  p.cu = cu_rows;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = ctx->err;
  p.n_rows = n_rows;
  p.n_seqs = cf.batch;
  p.Hq = cf.n_q_heads;
  p.Hkv = cf.n_kv_heads;
  p.g = ctx->g;
  p.c = (float)(1.4426950408889634 / std::sqrt(128.0));
  p.page_table = page_table;
  p.pos = pos;
  p.flag = flag;
  p.parent = parent;
  p.n_pages = layer->n_pages;
  p.max_pages = cf.max_pages;
  p.part_o = ctx->tile_part_o;
  p.part_ml = ctx->tile_part_ml;
  p.plan = ctx->tile_plan;
  CUtensorMap mq, mk, mv, mkn, mvn;
  const cuuint64_t pool = (cuuint64_t)layer->n_pages * cf.n_kv_heads * 16;
  const cuuint64_t kd[2] = {128, pool}, ks[1] = {256}, vd[3] = {64, pool, 2}, vs[2] = {256, 128};
  const cuuint32_t kb[2] = {64, 16}, vb[3] = {64, 16, 2};
  oda_status st = encode(&mk, layer->k, 2, kd, ks, kb);
  if (st == ODA_OK) st = encode(&mv, layer->v, 3, vd, vs, vb);
  if (st == ODA_OK) st = encode_rows(&mq, q, n_rows, cf.n_q_heads, (int64_t)cf.n_q_heads * 128, p.g, p.nq);
  if (st == ODA_OK) st = encode_rows(&mkn, k_new, n_rows, cf.n_kv_heads, (int64_t)cf.n_kv_heads * 128, 1, ODA_MAX_TREE);
  const cuuint64_t nd[4] = {64, (cuuint64_t)n_rows, 2, (cuuint64_t)cf.n_kv_heads};
  const cuuint64_t ns[3] = {(cuuint64_t)cf.n_kv_heads * 256, 128, 256};
  const cuuint32_t nb[4] = {64, 16, 2, 1};
  if (st == ODA_OK) st = encode(&mvn, v_new, 4, nd, ns, nb);
  if (st != ODA_OK) return st;
  const int grid = ctx->n_sms;
  tile_attention_kernel<true><<<grid, kThreads, kDynBytes, stream>>>(mq, mk, mv, mkn, mvn, p);
  st = check_cuda(cudaGetLastError(), "tree attention launch");
  if (st != ODA_OK) return st;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)n_rows, (unsigned)((cf.n_q_heads + 3) / 4));
  lc.blockDim = dim3(128);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&lc, tree_join_kernel, p, (uint32_t)grid), "tree join launch");
}

}  // namespace oda

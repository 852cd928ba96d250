// Transactional commit of the chosen branch, and snapshot / restore of recurrent state.
//
// Method: "On-Demand Attention：让语言模型按需读取完整历史" (method notes) §2.3: the current K,V
// of every layer are staged and only the chosen branch's update is written to the full cache
// (and with it to the local view, which here is an index set over the same cache); the
// committed hidden state comes from the same branch (eq. h_t = h^{b_t}_t, C_t = C_{t-1} ||
// dC^{b_t}_t).  Hybrid backbones snapshot conv and recurrent state before the local pass and
// restore the pre-step state before the full retry.
//
// bf16 pages: pure data movement, 16-byte copies, bit-exact.  fp8 pages: each committed token
// row is quantised (e4m3 codes, one fp32 scale per row) into its page block; the same routine
// packs a whole bf16 cache into fp8 blocks.  The commit grid is (layers x sequences);
// the last CTA of each sequence (completion counter, no waiting) takes the hidden state and
// advances the position, after every layer of that sequence has read it.
#include "internal.h"
#include "ptx.cuh"

namespace oda {
namespace {

constexpr int kPageTok = 16;

// fp8 page block of one (page, KV head): K codes [16 tokens][128] with chunk k of token j at
// chunk position k ^ (j & 7); V codes transposed [128 dims][16 slots], slot s holding token
// 2*(s/4) + (s&1) + 8*((s>>1)&1); K scales fp32 [16]; V scales fp32 [16] (4224 bytes).
constexpr int kF8Block = 4224;
constexpr int kF8V = 2048;
constexpr int kF8SK = 4096;
constexpr int kF8SV = 4160;

__device__ __forceinline__ int v8_slot(int j) { return 4 * ((j & 7) >> 1) + ((j >> 3) << 1) + (j & 1); }

// Quantises one 128-value bf16 row (this lane: values 4*lane .. 4*lane + 3, given as two bf16
// pairs) to e4m3 codes with one fp32 scale: s = max|x| / 448 (1 for an all-zero row),
// code = round-to-nearest-even(x / s) with saturation at +-448; both divisions in fp32 with
// IEEE rounding.  Returns the four codes (value 4*lane + i in byte i); *scale gets s.
__device__ __forceinline__ uint32_t quantize_row_e4m3(uint32_t w01, uint32_t w23, int lane, float* scale) {
  const float x0 = bf16_lo_to_f32(w01), x1 = bf16_hi_to_f32(w01);
  const float x2 = bf16_lo_to_f32(w23), x3 = bf16_hi_to_f32(w23);
  float amax = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), fmaxf(fabsf(x2), fabsf(x3)));
  // (the bits of values >= 0 are in their order; a lane of NaN alone counts as 0)
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, amax == amax ? __float_as_uint(amax) : 0u));
  float s = 1.0f, q0, q1, q2, q3;
  if (amax >= 0x1p-80f && amax <= 0x1p100f) {
    // The same roundings by a reciprocal (Markstein): r = RN(1 / b), q = RN(a r), RN(q + r (a - q b)) is RN(a / b)
    // where a - q b is exact.  Here it is for every quotient of 2^-11 or more (s >= 2^-89, so its products with
    // a quotient's last place reach down to 2^-145); a smaller one is a code of 0 however it is rounded.  (Its sign
    // is a's, as a division's: from a = -0 the correction makes +0.)
    auto quotient = [](float a, float by, float r) {
      const float q = a * r;
      return copysignf(fmaf(r, fmaf(-q, by, a), q), a);
    };
    s = quotient(amax, 448.0f, 1.0f / 448.0f);
    const float r = __frcp_rn(s);
    q0 = quotient(x0, s, r), q1 = quotient(x1, s, r), q2 = quotient(x2, s, r), q3 = quotient(x3, s, r);
  } else {
    if (amax > 0.f) s = __fdiv_rn(amax, 448.0f);
    q0 = __fdiv_rn(x0, s), q1 = __fdiv_rn(x1, s), q2 = __fdiv_rn(x2, s), q3 = __fdiv_rn(x3, s);
  }
  *scale = s;
  return f32x2_to_e4m3x2(q0, q1) | (f32x2_to_e4m3x2(q2, q3) << 16);
}

// Writes a quantised token row (K if which == 0, else V) into slot j of a block.
__device__ __forceinline__ void store_row_e4m3(uint8_t* blk, int which, int j, uint32_t codes,
                                               float scale, int lane) {
  if (which == 0) {
    const int k = lane >> 2;   // 16-dim chunk of values 4*lane .. 4*lane + 3
    *reinterpret_cast<uint32_t*>(blk + 128 * j + 16 * (k ^ (j & 7)) + 4 * (lane & 3)) = codes;
    if (lane == 0) *reinterpret_cast<float*>(blk + kF8SK + 4 * j) = scale;
  } else {
    const int sl = v8_slot(j);
#pragma unroll
    for (int i = 0; i < 4; ++i) blk[kF8V + 16 * (4 * lane + i) + sl] = (uint8_t)(codes >> (8 * i));
    if (lane == 0) *reinterpret_cast<float*>(blk + kF8SV + 4 * j) = scale;
  }
}

struct CommitParams {
  void* k[ODA_MAX_LAYERS];
  void* v[ODA_MAX_LAYERS];
  int64_t n_pages[ODA_MAX_LAYERS];
  const int32_t* page_table;
  int32_t* pos;
  const int32_t* flag;
  const uint4* ks[2];     // staging [L][B][Hkv][128] bf16 as 16-byte words; [0] local, [1] full
  const uint4* vs[2];
  const float4* h[2];
  float4* h_prev;
  int32_t* cnt;           // [B]
  int32_t* err;
  int L, B, Hkv, max_pages, D4;
};

template <int F>
__global__ void __launch_bounds__(256) commit_kernel(const CommitParams p) {
  const int l = blockIdx.x, b = blockIdx.y;
  const int t = p.pos[b];
  const int br = p.flag[b] != 0 ? 1 : 0;
  __shared__ int s_last;
  const bool pos_ok = t >= 1 && (int64_t)t <= (int64_t)p.max_pages * kPageTok;
  if (pos_ok) {
    const int lp = (t - 1) / kPageTok, slot = (t - 1) % kPageTok;
    const int phys = p.page_table[(size_t)b * p.max_pages + lp];
    if (phys >= 0 && (int64_t)phys < p.n_pages[l]) {
      const int words = p.Hkv * 16;  // 16-byte words per token of one layer (K or V)
      const size_t src0 = ((size_t)l * p.B + b) * words;
      if constexpr (F == 0) {
        for (int i = threadIdx.x; i < 2 * words; i += blockDim.x) {
          const int which = i >= words;     // 0: K, 1: V
          const int w = i - which * words;
          const int h = w >> 4, c = w & 15;
          const uint4 val = which ? p.vs[br][src0 + w] : p.ks[br][src0 + w];
          uint4* pool = reinterpret_cast<uint4*>(which ? p.v[l] : p.k[l]);
          pool[(((size_t)phys * p.Hkv + h) * kPageTok + slot) * 16 + c] = val;
        }
      } else {
        // one warp per (head, K or V) row: quantise and write into the page block
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int row = warp; row < 2 * p.Hkv; row += blockDim.x >> 5) {
          const int which = row / p.Hkv, h = row - which * p.Hkv;
          const uint2 wv = reinterpret_cast<const uint2*>(which ? p.vs[br] : p.ks[br])[(src0 + h * 16) * 2 + lane];
          float sc;
          const uint32_t codes = quantize_row_e4m3(wv.x, wv.y, lane, &sc);
          uint8_t* blk = static_cast<uint8_t*>(p.k[l]) + ((size_t)phys * p.Hkv + h) * kF8Block;
          store_row_e4m3(blk, which, slot, codes, sc, lane);
        }
      }
    } else if (threadIdx.x == 0) {
      atomicOr(p.err, ODA_DEVERR_PAGE_RANGE);
    }
  } else if (threadIdx.x == 0 && l == 0) {
    atomicOr(p.err, ODA_DEVERR_POS_RANGE);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = (atomicAdd(&p.cnt[b], 1) == p.L - 1);
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (pos_ok) {
    for (int i = threadIdx.x; i < p.D4; i += blockDim.x) p.h_prev[(size_t)b * p.D4 + i] = p.h[br][(size_t)b * p.D4 + i];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (pos_ok) p.pos[b] = t + 1;
    p.cnt[b] = 0;
  }
}

struct AppendParams {
  void* k[ODA_MAX_LAYERS];
  void* v[ODA_MAX_LAYERS];
  int64_t n_pages[ODA_MAX_LAYERS];
  const int32_t* page_table;
  const int32_t* pos;
  const int32_t* cu;
  const int32_t* rows;
  const uint4* ks;        // staging [L][n_stage][Hkv][128] bf16 as 16-byte words
  const uint4* vs;
  const float4* h;
  float4* h_prev;
  int32_t* pos_next;
  int32_t* err;
  int64_t n_rows, n_stage;
  int B, Hkv, max_pages, D4;
};

__device__ __forceinline__ bool append_bounds(const AppendParams& p, int b, int* a, int* e) {
  *a = p.cu[b];
  *e = p.cu[b + 1];
  return *a >= 0 && *e >= *a && (int64_t)*e <= p.n_rows;
}

// A run: the appended rows of one sequence that go to one page.
struct AppendRun {
  int cnt;       // rows (0: nothing to write)
  int row0;      // first packed row
  int slot0;     // its slot in the page
  int phys;
};

// The id-th run of the call, by a whole warp.  Sequence b's rows take the places pos - 1 .. of its
// cache, so its runs are the pages that these places touch; sequences with bad bounds have none.
__device__ __forceinline__ AppendRun append_run(const AppendParams& p, int id, int lane, bool report) {
  AppendRun r = {0, 0, 0, 0};
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int a = 0, e = 0, first = 0, runs = 0;
    if (b < p.B && append_bounds(p, b, &a, &e) && e > a) {
      first = p.pos[b];
      // (a position below 1 is one run, which reports it)
      runs = first >= 1 ? (int)(((int64_t)((first - 1) & 15) + (e - a) + 15) >> 4) : 1;
    }
    int inc = runs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, id >= before + inc - runs && id < before + inc);
    if (here) {
      const int src = __ffs((int)here) - 1;
      a = __shfl_sync(0xffffffffu, a, src);
      e = __shfl_sync(0xffffffffu, e, src);
      first = __shfl_sync(0xffffffffu, first, src);
      const int k = id - before - __shfl_sync(0xffffffffu, inc - runs, src);
      const int64_t page = (int64_t)((first - 1) >> 4) + k;
      if (first < 1 || page >= p.max_pages) {
        if (report && lane == 0) atomicOr(p.err, ODA_DEVERR_POS_RANGE);
        return r;
      }
      const int off = (first - 1) & 15;                  // places before the first row in its page
      const int lo = max(0, 16 * k - off), hi = (int)min((int64_t)(e - a), (int64_t)16 * (k + 1) - off);
      r.cnt = hi - lo;
      r.row0 = a + lo;
      r.slot0 = (off + lo) & 15;
      r.phys = p.page_table[(size_t)(b0 + src) * p.max_pages + page];
      return r;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// One CTA writes a run of one layer (blockIdx.y).  Rows of 256 bytes per head that are neighbours in the
// page, so bf16 pages take whole lines, and an fp8 page's transposed V is written whole.
// Bound, bf16: the copy (two prompts of 900..2100 into 28 layers, 871 MB: 150 us, 5.8 TB/s, 89% of the measured
// copy).  fp8, few rows: latency and instructions, a CTA's lookups and then some 150 instructions a warp and row;
// accepted paths of 32 sequences into 36 layers, 27 MB: 27 us (22.7 with L2 warm; 28 with a V page's bytes written
// one by one and IEEE divisions).  Slower: a warp a run, layer and head without barriers, several layers a
// CTA, CTAs of 128 or 512 threads, 48 registers for a fifth CTA an SM.
template <int F>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  __shared__ AppendRun run;
  __shared__ int src[kPageTok];          // staging rows (< 0: none)
  __shared__ bool part;                  // some slots of the page are left as they are
  const int l = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    AppendRun r = append_run(p, blockIdx.x, lane, l == 0);
    if (r.cnt > 0 && (r.phys < 0 || (int64_t)r.phys >= p.n_pages[l])) {
      if (lane == 0) atomicOr(p.err, ODA_DEVERR_PAGE_RANGE);
      r.cnt = 0;
    }
    if (lane == 0) run = r;
    if (lane < r.cnt) {
      const int64_t x = p.rows ? p.rows[r.row0 + lane] : r.row0 + lane;
      const bool ok = x >= 0 && x < p.n_stage;
      if (!ok && l == 0) atomicOr(p.err, ODA_DEVERR_ROW_RANGE);
      src[lane] = ok ? (int)x : -1;
    }
    __syncwarp();
    if (lane == 0) part = false;
    __syncwarp();
    if (r.cnt < kPageTok ? lane == 0 : lane < kPageTok && src[lane] < 0) part = true;
  }
  __syncthreads();
  const AppendRun r = run;
  if (r.cnt == 0) return;
  const int words = p.Hkv * 16;          // 16-byte words per row of K or V
  if constexpr (F == 0) {
    // consecutive threads take a head's consecutive rows: the destination is contiguous
    const int per = r.cnt * 16, all = 2 * p.Hkv * per;
#pragma unroll 4
    for (int x = threadIdx.x; x < all; x += 256) {
      const int head = x / per, y = x - head * per;      // K heads, then V heads
      const int which = head >= p.Hkv, h = head - which * p.Hkv, j = y >> 4, c = y & 15;
      const int from = src[j];
      if (from < 0) continue;
      const uint4 val = __ldcs((which ? p.vs : p.ks) + ((size_t)l * p.n_stage + from) * words + h * 16 + c);
      uint4* pool = reinterpret_cast<uint4*>(which ? p.v[l] : p.k[l]);
      pool[(((size_t)r.phys * p.Hkv + h) * kPageTok + r.slot0 + j) * 16 + c] = val;
    }
  } else {
    for (int y = warp; y < 2 * p.Hkv; y += 8) {
      const int which = y >= p.Hkv, h = y - which * p.Hkv;
      const uint2* rows = reinterpret_cast<const uint2*>(which ? p.vs : p.ks) + ((size_t)l * p.n_stage * words + h * 16) * 2;
      uint8_t* blk = static_cast<uint8_t*>(p.k[l]) + ((size_t)r.phys * p.Hkv + h) * kF8Block;
      // K: this lane has dims 4 lane .. + 3.  V: dims lane, 32 + lane, 64 + lane, 96 + lane, each with its 16 slots,
      // one byte each, in v: the transposed rows that it writes whole, 512 bytes a store.  Where the run fills
      // only part of the page they are read first (no other warp of the call writes this page's V).
      uint32_t v[16];
      uint4* line = reinterpret_cast<uint4*>(blk + kF8V) + lane;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint4 old = which && part ? line[32 * d] : make_uint4(0, 0, 0, 0);
        v[4 * d] = old.x, v[4 * d + 1] = old.y, v[4 * d + 2] = old.z, v[4 * d + 3] = old.w;
      }
#pragma unroll 1
      for (int j0 = 0; j0 < r.cnt; j0 += 4) {
        uint2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int from = j0 + j < r.cnt ? src[j0 + j] : -1;
          if (from < 0) continue;
          const uint2* row = rows + (size_t)from * words * 2;
          if (which == 0) {
            w[j] = __ldcs(row + lane);
          } else {
            const unsigned short* x = reinterpret_cast<const unsigned short*>(row) + lane;
            w[j].x = (uint32_t)__ldcs(x) | (uint32_t)__ldcs(x + 32) << 16;
            w[j].y = (uint32_t)__ldcs(x + 64) | (uint32_t)__ldcs(x + 96) << 16;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j0 + j >= r.cnt || src[j0 + j] < 0) continue;
          const int slot = r.slot0 + j0 + j;
          float sc;
          const uint32_t codes = quantize_row_e4m3(w[j].x, w[j].y, lane, &sc);
          if (which == 0) {
            store_row_e4m3(blk, 0, slot, codes, sc, lane);
          } else {
            const int sl = v8_slot(slot), at = 4 * (sl & 3);
            // byte d of the codes to byte sl mod 4 of word sl / 4 of dim d
            const uint32_t keep = 0x3210u & ~(0xfu << at);
            auto put = [&](int q) {
#pragma unroll
              for (int d = 0; d < 4; ++d) v[4 * d + q] = __byte_perm(v[4 * d + q], codes, keep | (uint32_t)(4 + d) << at);
            };
            if ((sl >> 2) == 0) put(0);
            else if ((sl >> 2) == 1) put(1);
            else if ((sl >> 2) == 2) put(2);
            else put(3);
            if (lane == 0) *reinterpret_cast<float*>(blk + kF8SV + 4 * slot) = sc;
          }
        }
      }
      if (which == 0) continue;
#pragma unroll
      for (int d = 0; d < 4; ++d) line[32 * d] = make_uint4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
    }
  }
}

// After every row is written: the hidden state of each sequence's last row, and its next position.
__global__ void __launch_bounds__(256) append_finish_kernel(const AppendParams p) {
  grid_dependency_wait();
  const int b = blockIdx.x;
  int a, e;
  const bool ok = append_bounds(p, b, &a, &e);
  const int t = p.pos[b];
  if (threadIdx.x == 0 && !ok) atomicOr(p.err, ODA_DEVERR_ROW_RANGE);
  if (!ok || t < 1) {
    __syncthreads();
    if (threadIdx.x == 0 && p.pos_next) p.pos_next[b] = t;
    return;
  }
  if (p.h_prev && e > a) {
    const int64_t src = p.rows ? p.rows[e - 1] : e - 1;
    if (src >= 0 && src < p.n_stage)
      for (int i = threadIdx.x; i < p.D4; i += blockDim.x) p.h_prev[(size_t)b * p.D4 + i] = p.h[(size_t)src * p.D4 + i];
  }
  __syncthreads();                // every thread has read pos[b], which pos_next may be
  if (threadIdx.x == 0 && p.pos_next) p.pos_next[b] = t + (e - a);
}

// dst[b] <- src[b] for every sequence (flag == nullptr) or the flagged ones; blockIdx.y = b.
__global__ void state_copy_kernel(const float4* src, float4* dst, size_t per_seq4,
                                  const int32_t* flag) {
  const int b = blockIdx.y;
  if (flag && flag[b] == 0) return;
  const float4* s = src + (size_t)b * per_seq4;
  float4* d = dst + (size_t)b * per_seq4;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < per_seq4;
       i += (size_t)gridDim.x * blockDim.x)
    d[i] = s[i];
}

// Packs bf16 pools [n_pages][Hkv][16][128] (K and V) into fp8 page blocks; one CTA of 8 warps
// per (page, KV head) block, one warp per token row of K or V (32 rows).
__global__ void __launch_bounds__(256) kv8_pack_kernel(const uint2* k, const uint2* v, uint8_t* dst) {
  const size_t blkid = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* blk = dst + blkid * kF8Block;
  for (int row = warp; row < 2 * kPageTok; row += 8) {
    const int which = row >> 4, j = row & 15;
    const uint2 w = (which ? v : k)[(blkid * kPageTok + j) * 32 + lane];
    float sc;
    const uint32_t codes = quantize_row_e4m3(w.x, w.y, lane, &sc);
    store_row_e4m3(blk, which, j, codes, sc, lane);
  }
}

}  // namespace

oda_status launch_kv8_pack(const oda_kv_layer* src, const oda_kv8_layer* dst, int32_t n_kv_heads,
                           cudaStream_t stream) {
  if (!src || !dst || !src->k || !src->v || !dst->kv)
    return set_error(ODA_ERR_INVALID_ARG, "kv8_pack: null pointer argument");
  if (n_kv_heads < 1 || src->n_pages < 1 || src->n_pages != dst->n_pages ||
      src->n_pages * (int64_t)n_kv_heads > INT32_MAX)
    return set_error(ODA_ERR_INVALID_ARG, "kv8_pack: page counts differ or out of range");
  if ((reinterpret_cast<uintptr_t>(src->k) | reinterpret_cast<uintptr_t>(src->v) |
       reinterpret_cast<uintptr_t>(dst->kv)) & 15)
    return set_error(ODA_ERR_INVALID_ARG, "kv8_pack: pools must be 16-byte aligned");
  const int64_t blocks = src->n_pages * n_kv_heads;
  kv8_pack_kernel<<<(unsigned)blocks, 256, 0, stream>>>(static_cast<const uint2*>(src->k),
                                                         static_cast<const uint2*>(src->v),
                                                         static_cast<uint8_t*>(dst->kv));
  return check_cuda(cudaGetLastError(), "kv8_pack launch");
}

oda_status launch_commit(oda_ctx* ctx, const KvPool* layers, int32_t n_layers,
                         const int32_t* page_table, int32_t* pos, const int32_t* flag,
                         const void* ksl, const void* vsl, const void* ksf, const void* vsf,
                         const float* h_local, const float* h_full, float* h_prev,
                         cudaStream_t stream) {
  const oda_config& cf = ctx->cfg;
  if (!layers || n_layers < 1 || n_layers > ODA_MAX_LAYERS)
    return set_error(ODA_ERR_INVALID_ARG, "commit: n_layers must be 1..%d", ODA_MAX_LAYERS);
  const int F = layers[0].fmt;
  if (!page_table || !pos || !flag || !ksl || !vsl || !ksf || !vsf || !h_local || !h_full || !h_prev)
    return set_error(ODA_ERR_INVALID_ARG, "commit: null pointer argument");
  const void* al[] = {ksl, vsl, ksf, vsf, h_local, h_full, h_prev};
  for (const void* q : al)
    if (reinterpret_cast<uintptr_t>(q) & 15)
      return set_error(ODA_ERR_INVALID_ARG, "commit: staging and hidden buffers must be 16-byte aligned");
  CommitParams p;
  for (int l = 0; l < n_layers; ++l) {
    if (layers[l].fmt != F || !layers[l].k || (F == 0 && !layers[l].v) || layers[l].n_pages <= 0 ||
        ((reinterpret_cast<uintptr_t>(layers[l].k) | reinterpret_cast<uintptr_t>(layers[l].v)) & 15))
      return set_error(ODA_ERR_INVALID_ARG, "commit: bad KV pool of layer %d", l);
    p.k[l] = const_cast<void*>(layers[l].k);
    p.v[l] = const_cast<void*>(layers[l].v);
    p.n_pages[l] = layers[l].n_pages;
  }
  p.page_table = page_table;
  p.pos = pos;
  p.flag = flag;
  p.ks[0] = static_cast<const uint4*>(ksl);
  p.vs[0] = static_cast<const uint4*>(vsl);
  p.ks[1] = static_cast<const uint4*>(ksf);
  p.vs[1] = static_cast<const uint4*>(vsf);
  p.h[0] = reinterpret_cast<const float4*>(h_local);
  p.h[1] = reinterpret_cast<const float4*>(h_full);
  p.h_prev = reinterpret_cast<float4*>(h_prev);
  p.cnt = ctx->glue_cnt + cf.batch;  // commit's own counters
  p.err = ctx->err;
  p.L = n_layers;
  p.B = cf.batch;
  p.Hkv = cf.n_kv_heads;
  p.max_pages = cf.max_pages;
  p.D4 = cf.head_in_dim / 4;
  if (F == 0)
    commit_kernel<0><<<dim3(n_layers, cf.batch), 256, 0, stream>>>(p);
  else
    commit_kernel<1><<<dim3(n_layers, cf.batch), 256, 0, stream>>>(p);
  return check_cuda(cudaGetLastError(), "commit launch");
}

oda_status launch_append(oda_ctx* ctx, const KvPool* layers, int32_t n_layers, const int32_t* page_table,
                         const int32_t* pos, int64_t n_rows, int64_t n_stage, const int32_t* cu_rows,
                         const int32_t* rows, const void* k_stage, const void* v_stage, const float* h_stage,
                         float* h_prev, int32_t* pos_next, cudaStream_t stream) {
  const oda_config& cf = ctx->cfg;
  const int F = layers[0].fmt;
  if (!page_table || !pos || !cu_rows || !k_stage || !v_stage)
    return set_error(ODA_ERR_INVALID_ARG, "append: null pointer argument");
  if ((h_stage == nullptr) != (h_prev == nullptr))
    return set_error(ODA_ERR_INVALID_ARG, "append: h_stage and h_prev go together");
  if (n_rows < 0 || n_rows > INT32_MAX || n_stage < 1 || n_stage > INT32_MAX || (!rows && n_rows > n_stage))
    return set_error(ODA_ERR_INVALID_ARG, "append: n_rows or n_stage out of range");
  const void* al[] = {k_stage, v_stage, h_stage, h_prev};
  for (const void* q : al)
    if (reinterpret_cast<uintptr_t>(q) & 15)
      return set_error(ODA_ERR_INVALID_ARG, "append: staging and hidden buffers must be 16-byte aligned");
  AppendParams p;
  for (int l = 0; l < n_layers; ++l) {
    if (!layers[l].k || (F == 0 && !layers[l].v) || layers[l].n_pages <= 0 ||
        ((reinterpret_cast<uintptr_t>(layers[l].k) | reinterpret_cast<uintptr_t>(layers[l].v)) & 15))
      return set_error(ODA_ERR_INVALID_ARG, "append: bad KV pool of layer %d", l);
    p.k[l] = const_cast<void*>(layers[l].k);
    p.v[l] = const_cast<void*>(layers[l].v);
    p.n_pages[l] = layers[l].n_pages;
  }
  p.page_table = page_table;
  p.pos = pos;
  p.cu = cu_rows;
  p.rows = rows;
  p.ks = static_cast<const uint4*>(k_stage);
  p.vs = static_cast<const uint4*>(v_stage);
  p.h = reinterpret_cast<const float4*>(h_stage);
  p.h_prev = reinterpret_cast<float4*>(h_prev);
  p.pos_next = pos_next;
  p.err = ctx->err;
  p.n_rows = n_rows;
  p.n_stage = n_stage;
  p.B = cf.batch;
  p.Hkv = cf.n_kv_heads;
  p.max_pages = cf.max_pages;
  p.D4 = cf.head_in_dim / 4;
  ctx->prev_attention = false;
  oda_status st = ODA_OK;
  if (n_rows > 0) {
    // runs: a sequence of n rows touches at most n / 16 + 2 pages
    const int64_t runs = n_rows / kPageTok + 2 * std::min<int64_t>(n_rows, cf.batch);
    const dim3 grid((unsigned)runs, n_layers);
    if (F == 0)
      append_kernel<0><<<grid, 256, 0, stream>>>(p);
    else
      append_kernel<1><<<grid, 256, 0, stream>>>(p);
    st = check_cuda(cudaGetLastError(), "append launch");
    if (st != ODA_OK) return st;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(cf.batch);
  lc.blockDim = dim3(256);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return check_cuda(cudaLaunchKernelEx(&lc, append_finish_kernel, p), "append finish launch");
}

oda_status launch_state_copy(const oda_state* src, const oda_state* dst, int B,
                             const int32_t* flag, cudaStream_t stream) {
  if (!src || !dst || !src->rec || !dst->rec || !src->conv || !dst->conv)
    return set_error(ODA_ERR_INVALID_ARG, "state copy: null pointer argument");
  if (src->n_layers != dst->n_layers || src->heads != dst->heads || src->dk != dst->dk ||
      src->dv != dst->dv || src->conv_taps != dst->conv_taps || src->conv_width != dst->conv_width)
    return set_error(ODA_ERR_INVALID_ARG, "state copy: shapes differ");
  if (src->n_layers < 1 || src->heads < 1 || src->dk < 1 || src->dv < 1 || src->conv_taps < 0 ||
      src->conv_width < 0)
    return set_error(ODA_ERR_INVALID_ARG, "state copy: bad shape");
  const size_t rec = (size_t)src->n_layers * src->heads * src->dk * src->dv;
  const size_t conv = (size_t)src->n_layers * src->conv_taps * src->conv_width;
  if ((rec & 3) || (conv & 3))
    return set_error(ODA_ERR_UNSUPPORTED, "state copy: per-sequence sizes must be multiples of 4 floats");
  const void* al[] = {src->rec, dst->rec, src->conv, dst->conv};
  for (const void* q : al)
    if (reinterpret_cast<uintptr_t>(q) & 15)
      return set_error(ODA_ERR_INVALID_ARG, "state copy: buffers must be 16-byte aligned");
  const int blocks_rec = (int)std::min<size_t>(1024, (rec / 4 + 255) / 256);
  state_copy_kernel<<<dim3(blocks_rec, B), 256, 0, stream>>>(
      reinterpret_cast<const float4*>(src->rec), reinterpret_cast<float4*>(dst->rec), rec / 4, flag);
  oda_status st = check_cuda(cudaGetLastError(), "state copy launch");
  if (st != ODA_OK || conv == 0) return st;
  const int blocks_conv = (int)std::min<size_t>(1024, (conv / 4 + 255) / 256);
  state_copy_kernel<<<dim3(blocks_conv, B), 256, 0, stream>>>(
      reinterpret_cast<const float4*>(src->conv), reinterpret_cast<float4*>(dst->conv), conv / 4, flag);
  return check_cuda(cudaGetLastError(), "state copy launch");
}

}  // namespace oda

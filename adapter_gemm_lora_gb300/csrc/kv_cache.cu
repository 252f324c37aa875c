// KV rows into pages, and eviction from the KV cache by accumulated attention weight.
//
// Both work on device page tables [n_req][max_len][layers][2] (K page, V page per cached token and
// layer), so neither needs the host between steps.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <string>

#include "tc_ptx.h"

namespace {

// ---- page writes -------------------------------------------------------------------------------
// One warp per (row, K or V): the page ids are read through the table and checked, then the row's
// 2 H bytes are copied 16 bytes a lane.  HBM-bound: every row is read once and written once; 11,300
// prompt rows at H = 4096 take 57.2 us, 6.5 TB/s (0.97 of the copy rate).  One row per request of a
// decode step is a launch: 256 rows at H = 5120 take 5 us a call, most of it on the host.
constexpr int kWriteThreads = 256;
constexpr int kWriteBatch = 4;                             // 16-byte reads a lane has in flight

// The inputs are not marked read-only: this kernel may start while the one that writes them still
// runs (it waits before it reads), which read-only loads do not allow.
__global__ void __launch_bounds__(kWriteThreads)
kv_write_kernel(uint16_t* pool, int64_t num_pages, int32_t H, int32_t n_rows, const int32_t* row_req,
                const int32_t* row_pos, const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride,
                int32_t n_req, const int2* table, int32_t max_len, int32_t layers, int32_t layer, int32_t* err) {
  pdl_wait_then_release();
  const int64_t item = (int64_t)blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= 2 * (int64_t)n_rows) return;
  const int64_t t = item >> 1;
  const int half = (int)(item & 1);
  const int32_t r = row_req[t], j = row_pos[t];
  if (r == -1) return;
  if (r < -1 || r >= n_req || j < 0 || j >= max_len) {
    if (lane == 0) flag_error(err, LORA_DEV_BAD_SEGMENT);
    return;
  }
  const int2 pg = table[((int64_t)r * max_len + j) * layers + layer];
  if (pg.x < 0 || pg.x >= num_pages || pg.y < 0 || pg.y >= num_pages) {
    if (lane == 0) flag_error(err, LORA_DEV_BAD_PAGE);
    return;
  }
  const int32_t page = half ? pg.y : pg.x;
  const uint4* src = reinterpret_cast<const uint4*>(half ? v + t * v_stride : k + t * k_stride);
  uint4* dst = reinterpret_cast<uint4*>(pool + (int64_t)page * H);
  const int n = H / 8;
  for (int i0 = lane; i0 < n; i0 += 32 * kWriteBatch) {
    uint4 x[kWriteBatch];
#pragma unroll
    for (int b = 0; b < kWriteBatch; ++b)
      if (i0 + 32 * b < n) x[b] = src[i0 + 32 * b];
#pragma unroll
    for (int b = 0; b < kWriteBatch; ++b)
      if (i0 + 32 * b < n) dst[i0 + 32 * b] = x[b];
  }
}

// Many short rows: a warp per row leaves most of its lanes idle and pays three dependent reads (row,
// table, row's data) for a few bytes.  Here L = 8, 16 or 32 lanes copy a row and a warp takes 128 / L
// tokens: one lane per token reads its page ids while the first loads of k and v are under way, and
// each lane has kWritePacked 16-byte loads in flight.  160 MB in and out, us with a warp per row and
// here: H = 64 290 / 59.6, 128 153 / 55.4, 256 87.7 / 51.1, 512 58.6 / 50.1 (0.83 to 0.96 of the copy
// rate); 768 52.5 / 50.1, but 10,368 rows of it 7.5 / 9.7, and 1,024 49.2 / 51.9.  Rows that fit the
// SMs' warps once are quicker with a warp each: 64 rows of H = 64 2.2 / 2.9, 960 of 512 2.6 / 3.8; at
// 6,208 rows of 320 both take 4.2.
constexpr int kWritePacked = 8;
constexpr int kWritePackedMaxH = 512;
template <int L>
__global__ void __launch_bounds__(kWriteThreads)
kv_write_packed_kernel(uint16_t* pool, int64_t num_pages, int32_t H, int32_t n_rows, const int32_t* row_req,
                       const int32_t* row_pos, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                       int64_t v_stride, int32_t n_req, const int2* table, int32_t max_len, int32_t layers,
                       int32_t layer, int32_t* err) {
  constexpr int kRows = 32 / L;                            // rows (a token's K or V) at a time
  constexpr int kTokens = kRows * kWritePacked / 2;
  static_assert(kTokens <= 32, "a lane reads one token's entry");
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5)) * kTokens;
  if (t0 >= n_rows) return;
  int32_t r = -1, j = 0;
  if (lane < kTokens && t0 + lane < n_rows) {
    r = row_req[t0 + lane];
    j = row_pos[t0 + lane];
  }
  bool live = r != -1;
  if (live && (r < 0 || r >= n_req || j < 0 || j >= max_len)) {
    flag_error(err, LORA_DEV_BAD_SEGMENT);
    live = false;
  }
  int2 pg = make_int2(-1, -1);
  if (live) pg = table[((int64_t)r * max_len + j) * layers + layer];
  const unsigned lives = __ballot_sync(0xffffffffu, live);
  const int n = H / 8, col = lane % L, half = (lane / L) & 1;
  // Row b of this lane: token (b * kRows + lane / L) / 2; with one row at a time K and V take turns.
  bool first = true;
  for (int i = col; i - col < n; i += L) {
    uint4 x[kWritePacked];
#pragma unroll
    for (int b = 0; b < kWritePacked; ++b) {
      const int row = b * kRows + lane / L;
      const bool is_v = kRows == 1 ? (b & 1) : half;
      const int64_t t = t0 + (row >> 1);
      const uint16_t* src = is_v ? v + t * v_stride : k + t * k_stride;
      if (i < n && ((lives >> (row >> 1)) & 1)) x[b] = reinterpret_cast<const uint4*>(src)[i];
    }
    if (first && live && (pg.x < 0 || pg.x >= num_pages || pg.y < 0 || pg.y >= num_pages)) {
      flag_error(err, LORA_DEV_BAD_PAGE);
      pg = make_int2(-1, -1);
    }
    first = false;
#pragma unroll
    for (int b = 0; b < kWritePacked; ++b) {
      const int row = b * kRows + lane / L;
      const int32_t px = __shfl_sync(0xffffffffu, pg.x, row >> 1), py = __shfl_sync(0xffffffffu, pg.y, row >> 1);
      const int32_t page = (kRows == 1 ? (b & 1) : half) ? py : px;
      if (i < n && page >= 0) reinterpret_cast<uint4*>(pool + (int64_t)page * H)[i] = x[b];
    }
  }
}

// ---- page table and slot maps from token counts ----------------------------------------------------
// A block of rows per CTA, and with a new table a block of its positions per further CTA.  Every CTA sums
// the counts itself (a thread adds up n_req / 256 requests, one scan over the threads), so the call is one
// launch; a row's request is then found by bisection over the threads and a walk over that thread's
// requests.  Pages are moved a layer's K and V (8 bytes) a thread, or two layers' (16) where the layers are even and
// the arrays aligned.  64 prompts of 500 to 2,048 tokens, 40 layers, into a new table: 71 MB in 13.9 us.
// DRAM moves 28 MB of it (the pages read) and L2 keeps the rest; DRAM is 24 % busy, L2 29 %, so neither rate bounds it but
// the chain of a CTA: the counts first, then its entries, in 1.8 rounds.  Four entries in flight and four CTAs an SM;
// eight entries and two CTAs 16.4 us, and with the registers of four 14.3.
constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 4;                            // entries a thread has in flight
constexpr int kAppendEntries = 4 * kAppendBatch * kAppendThreads;   // entries that a CTA writes, about
constexpr int kAppendMaxRows = 1024;                       // rows a CTA takes, at most

struct AppendArgs {
  int32_t n_req;
  const int32_t* count;
  const int32_t* old_len;
  const void* pages;
  int32_t row_cap;
  void* table;
  int32_t max_len, layers;       // layers: entries of a token
  int32_t* new_len;
  int32_t* row_start;
  int32_t* row_req;
  int32_t* row_pos;
  int32_t rows_per_cta, row_ctas;
  uint64_t layers_inv;           // 2^40 / layers, rounded up: (e * layers_inv) >> 40 = e / layers for a CTA's entries (one row: 0)
  int32_t* err;
};

__device__ __forceinline__ int32_t append_old(const AppendArgs& a, int r) {
  return a.old_len ? min(max(a.old_len[r], 0), a.max_len) : 0;
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const AppendArgs a) {
  __shared__ int64_t before[kAppendThreads];               // rows of the requests of the threads before
  __shared__ int64_t warp_sum[kAppendThreads / 32];
  __shared__ int32_t req_s[kAppendMaxRows], pos_s[kAppendMaxRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait_then_release();
  const int per = (a.n_req + kAppendThreads - 1) / kAppendThreads;
  const int r0 = (int)min((int64_t)a.n_req, (int64_t)tid * per), r1 = min(a.n_req, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += max(a.count[r], 0);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t start = incl - mine;
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) start += w < warp ? warp_sum[w] : 0;
  before[tid] = start;
  __syncthreads();

  if (blockIdx.x == 0) {                                   // lengths and row starts
    for (int r = r0; r < r1; ++r) {
      const int32_t c = a.count[r], old = append_old(a, r);
      const int64_t room = min((int64_t)max(c, 0), max((int64_t)a.row_cap - start, (int64_t)0));   // rows that the arrays hold
      if (c < 0 || (a.old_len && a.old_len[r] != old) || old + (int64_t)max(c, 0) > a.max_len || room < c)
        flag_error(a.err, LORA_DEV_BAD_SEGMENT);
      a.new_len[r] = (int32_t)min((int64_t)a.max_len, old + room);
      a.row_start[r] = (int32_t)min((int64_t)a.row_cap, start);
      start += max(c, 0);
    }
    if (tid == kAppendThreads - 1) a.row_start[a.n_req] = (int32_t)min((int64_t)a.row_cap, start);
  }

  if ((int)blockIdx.x < a.row_ctas) {
    const int64_t t0 = (int64_t)blockIdx.x * a.rows_per_cta;
    const int n = (int)min((int64_t)a.rows_per_cta, a.row_cap - t0);
    for (int i = tid; i < n; i += kAppendThreads) {
      const int64_t t = t0 + i;
      int lo = 0;                                          // the last thread whose requests start at or before t
#pragma unroll
      for (int step = kAppendThreads / 2; step > 0; step >>= 1)
        if (before[lo + step] <= t) lo += step;
      int64_t s = before[lo];
      int r = min((int64_t)a.n_req, (int64_t)lo * per);
      const int end = min(a.n_req, r + per);
      int32_t req = -1, pos = 0;
      for (; r < end; ++r) {
        const int32_t c = max(a.count[r], 0);
        if (t < s + c) {
          const int64_t p = append_old(a, r) + (t - s);
          if (p < a.max_len) {
            req = r;
            pos = (int32_t)p;
          }
          break;
        }
        s += c;
      }
      req_s[i] = req;
      pos_s[i] = pos;
      a.row_req[t] = req;
      a.row_pos[t] = pos;
    }
    __syncthreads();
    const int entries = n * a.layers;
    const T* from = static_cast<const T*>(a.pages) + t0 * a.layers;
    T* table = static_cast<T*>(a.table);
    for (int e0 = tid; e0 < entries; e0 += kAppendBatch * kAppendThreads) {
      T v[kAppendBatch];
#pragma unroll
      for (int b = 0; b < kAppendBatch; ++b)
        if (e0 + b * kAppendThreads < entries) v[b] = from[e0 + b * kAppendThreads];
#pragma unroll
      for (int b = 0; b < kAppendBatch; ++b) {
        const int e = e0 + b * kAppendThreads;
        if (e >= entries) break;
        const int i = (int)(e * a.layers_inv >> 40);
        if (req_s[i] >= 0) table[((int64_t)req_s[i] * a.max_len + pos_s[i]) * a.layers + e - i * a.layers] = v[b];
      }
    }
    return;
  }
  // a new table: -1 behind every request's tokens
  const int64_t j0 = (int64_t)(blockIdx.x - a.row_ctas) * a.rows_per_cta, all = (int64_t)a.n_req * a.max_len;
  const int n = (int)min((int64_t)a.rows_per_cta, all - j0);
  for (int i = tid; i < n; i += kAppendThreads) {
    const int r = (int)((j0 + i) / a.max_len), c = r / per;
    int64_t s = before[c];
    for (int x = c * per; x < r; ++x) s += max(a.count[x], 0);
    const int64_t held = min((int64_t)max(a.count[r], 0), max((int64_t)a.row_cap - s, (int64_t)0));
    req_s[i] = (j0 + i) - (int64_t)r * a.max_len >= held;
  }
  __syncthreads();
  const int entries = n * a.layers;
  T* to = static_cast<T*>(a.table) + j0 * a.layers, none;
  memset(&none, 0xff, sizeof(T));
#pragma unroll 4
  for (int e = tid; e < entries; e += kAppendThreads)
    if (req_s[(int)(e * a.layers_inv >> 40)]) to[e] = none;
}

// ---- eviction ------------------------------------------------------------------------------------
// Sort key of a weight: ascending with the value, -0 = +0, NaN = -infinity.  Keys of weights lie in
// [0x007FFFFF, 0xFF800000]: outside are a token that stays in any case and one that is not there.
constexpr uint32_t kKeyStays = 0xFFFFFFFFu, kKeyAbsent = 0u;
__device__ __forceinline__ uint32_t weight_key(float w) {
  const int32_t b = __float_as_int(fmaxf(w, -INFINITY) + 0.f);       // fmaxf drops a NaN, + 0 a minus sign of 0
  return (uint32_t)(b ^ ((b >> 31) | INT32_MIN));
}

// Per row (one request at one layer) the keys that stay are found by radix selection, digit by digit
// from the top: a histogram of the digit over the keys that still match the digits chosen so far, and
// the bin that holds the need-th largest key.  It ends with the first bin that is wanted whole: for
// weights that differ, after the second digit or the third.  Digits of 10 bits: of 12 bits a cluster
// would need two, but reading the other CTAs' 4,096 bins took 32 layers of 131,071 tokens from 38 to
// 100 us.
constexpr int kEvictBits = 10, kEvictBins = 1 << kEvictBits;
struct EvictArgs {
  int32_t n_req;
  const int2* table;
  const int32_t* seq_len;
  int32_t max_len, layers;
  const float* weight;
  int32_t budget, recent;
  int32_t* keep;
  int32_t* new_len;
  int2* table_out;
  float* weight_out;
  int32_t max_len_out;
  int32_t* err;
};

// What stays of one (request, layer) row, before any key is looked at.
struct EvictRow {
  int64_t row;                   // layer * n_req + request
  int r, layer, n, n_keep;
  int old;                       // tokens that compete; the newer ones stay
  int need;                      // of them stay
  uint32_t cut;                  // keys above it stay, and the first `ties` of those equal to it
  int ties;
};
__device__ __forceinline__ EvictRow evict_row(const EvictArgs& a, int id, bool report) {
  EvictRow e;
  e.layer = id % a.layers;
  e.r = id / a.layers;
  e.row = (int64_t)e.layer * a.n_req + e.r;
  e.n = a.seq_len[e.r];
  if (e.n < 0 || e.n > a.max_len) {
    if (report) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    e.n = e.n < 0 ? 0 : a.max_len;
  }
  e.n_keep = min(e.n, a.budget);
  e.old = e.n - min(e.n, a.recent);
  e.need = e.n_keep - (e.n - e.old);
  e.cut = e.need >= e.old ? kKeyAbsent : kKeyStays - 1;    // all of them, or none
  e.ties = 0;
  return e;
}
constexpr int kEvictWarps = 16;                            // of a CTA
constexpr int kEvictThreads = 32 * kEvictWarps;
constexpr int kEvictMaxCluster = 8;

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {   // p in CTA `rank` of the cluster
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ int2 cluster_load2(uint32_t addr) {
  int2 v;
  asm volatile("ld.relaxed.cluster.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// One row per CTA, or with kCluster per cluster of `n_cta` CTAs, of which every one adds up all CTAs'
// histograms (integer sums: the order does not matter), which also tell it how many keys the CTAs
// before it keep.  Every warp takes a contiguous part of the row, the keys of 32 K weights held in
// registers (longer parts are read again in every pass), so the kept tokens are numbered with one
// exchange of counts.  Their positions go to a list in shared memory first, and the outputs are
// written from there, 32 neighbours at a time.
// A row is a chain of dependent steps (length, weights, two or three digits, counts, pages), so time
// goes with the chain's length times the rows per SM: the passes are free of branches within
// kEvictBatch chunks of 32 weights, whose steps overlap.
constexpr int kEvictBatch = 4;

template <int K, bool kCluster>
__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_kernel(const EvictArgs a, int32_t n_cta) {
  static_assert(K % kEvictBatch == 0, "whole batches");
  constexpr int kHists = kCluster ? 2 : 1, kPer = kEvictBins / kEvictThreads;   // bins a thread adds up
  static_assert(kPer == 2, "the CTAs' histograms are read two bins at a time");
  // Shared memory: a histogram, of a cluster two in turn (the other CTAs may still read the one
  // before); the kept list of each warp.
  extern __shared__ __align__(16) int smem_evict[];
  __shared__ int warp_gt[kEvictWarps], warp_eq[kEvictWarps];
  __shared__ int found_s[3];                               // the wanted bin, keys above it, keys in it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* hist = smem_evict;
  for (int i = tid; i < kEvictBins * kHists / 4; i += kEvictThreads)
    reinterpret_cast<int4*>(smem_evict)[i] = make_int4(0, 0, 0, 0);
  pdl_wait_then_release();
  const int rank = kCluster ? (int)cluster_rank() : 0;
  const int id = kCluster ? blockIdx.x / n_cta : blockIdx.x;
  const bool live = id < a.n_req * a.layers;               // always: the test saves registers (16 x 32 rows of 16,384 117 -> 112 us)
  EvictRow e{};
  if (live) e = evict_row(a, id, tid == 0 && rank == 0);
  // this CTA's slice of the row, and this warp's part of it (multiples of 32)
  const int per_cta = ((e.n + n_cta - 1) / n_cta + 31) & ~31;
  const int c0 = (int)min((int64_t)e.n, (int64_t)rank * per_cta), c1 = min(e.n, c0 + per_cta);
  const int per_warp = ((c1 - c0 + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
  const bool held = per_warp <= 32 * K;                    // the part stays in registers
  uint32_t key[K];
  const auto load = [&](int j0) {
    const float* w = a.weight + e.row * a.max_len;
#pragma unroll
    for (int b = 0; b < K; ++b)
      key[b] = j0 + 32 * b + lane < w1 ? __float_as_uint(w[j0 + 32 * b + lane]) : 0u;
#pragma unroll
    for (int b = 0; b < K; ++b) {
      const int j = j0 + 32 * b + lane;
      const uint32_t k = weight_key(__uint_as_float(key[b]));
      key[b] = j >= w1 ? kKeyAbsent : j >= e.old ? kKeyStays : k;
    }
  };
  if (held) load(w0);
  __syncthreads();
  // kept and tied keys of the row before this CTA's slice: all tokens, or the newer ones, or what the
  // digits say
  int pos = e.need >= e.old ? c0 : max(0, c0 - e.old), tied = 0;
  const bool select = live && e.need > 0 && e.need < e.old;
  if (select) {
    uint32_t prefix = 0, mask = 0;
    int need = e.need;
    for (int d = 0, bits = 32; bits > 0; ++d) {
      const int nb = min(kEvictBits, bits);
      bits -= nb;
      const uint32_t digit = (1u << nb) - 1;
      for (int j0 = w0; j0 < w1; j0 += 32 * K) {
        if (!held) load(j0);
#pragma unroll
        for (int b0 = 0; b0 < K; b0 += kEvictBatch) {
          if (j0 + 32 * b0 >= w1) break;
#pragma unroll
          for (int b = b0; b < b0 + kEvictBatch; ++b) {
            const uint32_t k = key[b];
            const bool in = d == 0 ? k - 1 < kKeyStays - 1 : (k & mask) == prefix;     // the marks match no later prefix
            if (in) atomicAdd(&hist[digit - ((k >> bits) & digit)], 1);                // largest first
          }
        }
      }
      // every thread adds up kPer neighbouring bins, and the row's threads find the one they lie in
      int v[kPer];
      if (kCluster) {
        cluster_sync_all();
        v[0] = v[1] = 0;
        for (int c = 0; c < n_cta; ++c) {
          const int2 x = cluster_load2(cluster_addr(hist + 2 * tid, c));
          v[0] += x.x;
          v[1] += x.y;
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = hist[tid * kPer + i];
      }
      int mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine += v[i];
      const int incl = warp_scan(mine, lane);
      if (lane == 31) warp_gt[warp] = incl;
      __syncthreads();
      int above = incl - mine;
#pragma unroll
      for (int i = 0; i < kEvictWarps; ++i) above += i < warp ? warp_gt[i] : 0;
      if (above < need && above + mine >= need) {          // one thread
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (above < need && above + v[i] >= need) {
            found_s[0] = tid * kPer + i;
            found_s[1] = above;
            found_s[2] = v[i];
          }
          above += v[i];
        }
      }
      if (!kCluster) {                                     // this thread's bins have been read by itself alone
#pragma unroll
        for (int i = 0; i < kPer; ++i) hist[tid * kPer + i] = 0;
      }
      __syncthreads();
      const int bin = found_s[0];
      need -= found_s[1];
      const bool whole = found_s[2] == need;               // the whole bin stays
      prefix |= (digit - (uint32_t)bin) << bits;
      mask |= digit << bits;
      e.cut = whole ? prefix - 1 : prefix;
      e.ties = whole ? 0 : need;
      if (kCluster) {
        // of the CTAs before this one: the keys above the bin, and those in it
        int gt = 0, in = 0;
        if (2 * tid <= bin)
          for (int c = 0; c < rank; ++c) {
            const int2 x = cluster_load2(cluster_addr(hist + 2 * tid, c));
            gt += (2 * tid < bin ? x.x : 0) + (2 * tid + 1 < bin ? x.y : 0);
            in += 2 * tid == bin ? x.x : 2 * tid + 1 == bin ? x.y : 0;
          }
        gt = __reduce_add_sync(0xffffffffu, gt);
        in = __reduce_add_sync(0xffffffffu, in);
        if (lane == 0) {
          warp_gt[warp] = gt;
          warp_eq[warp] = in;
        }
        __syncthreads();
        tied = 0;
#pragma unroll
        for (int i = 0; i < kEvictWarps; ++i) {
          pos += warp_gt[i];
          tied += warp_eq[i];
        }
        if (whole) pos += tied;
        // the other histogram: every CTA had read it when it came to this digit's barrier
        hist = smem_evict + ((d & 1) ^ 1) * kEvictBins;
        if (!whole && bits > 0 && d > 0)
          for (int i = tid; i < kEvictBins / 4; i += kEvictThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
      }
      if (whole) break;
    }
    if (kCluster) cluster_arrive();                        // this CTA reads no other's shared memory any more
  }

  // what each warp keeps: keys above the cut, and keys equal to it
  int gt = 0, eq = 0;
  for (int j0 = w0; j0 < w1; j0 += 32 * K) {
    if (!held) load(j0);
#pragma unroll
    for (int b0 = 0; b0 < K; b0 += kEvictBatch) {
      if (j0 + 32 * b0 >= w1) break;
#pragma unroll
      for (int b = b0; b < b0 + kEvictBatch; ++b) {
        gt += key[b] > e.cut;
        eq += key[b] == e.cut;
      }
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  __syncthreads();                                         // warp_gt's sums have been read
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  // kept and tied of the row before this warp's part
#pragma unroll
  for (int i = 0; i < kEvictWarps; ++i) {
    pos += i < warp ? warp_gt[i] : 0;
    tied += i < warp ? warp_eq[i] : 0;
  }
  pos += min(tied, e.ties);
  const uint32_t below = (1u << lane) - 1;
  for (int j0 = w0; j0 < w1; j0 += 32 * K) {
    if (!held) load(j0);
    int* list = smem_evict + kHists * kEvictBins + warp * 32 * K;
    int n_kept = 0;
#pragma unroll
    for (int b0 = 0; b0 < K; b0 += kEvictBatch) {
      if (j0 + 32 * b0 >= w1) break;
      bool stay[kEvictBatch];
#pragma unroll
      for (int b = 0; b < kEvictBatch; ++b) stay[b] = key[b0 + b] > e.cut;
      if (e.ties > 0) {
#pragma unroll
        for (int b = 0; b < kEvictBatch; ++b) {
          const bool q = key[b0 + b] == e.cut;
          const uint32_t mq = __ballot_sync(0xffffffffu, q);
          stay[b] = stay[b] || (q && tied + __popc(mq & below) < e.ties);
          tied += __popc(mq);
        }
      }
#pragma unroll
      for (int b = 0; b < kEvictBatch; ++b) {
        const uint32_t ms = __ballot_sync(0xffffffffu, stay[b]);
        if (stay[b]) list[n_kept + __popc(ms & below)] = j0 + 32 * (b0 + b) + lane;
        n_kept += __popc(ms);
      }
    }
    __syncwarp();
    {
      const float* w = a.weight + e.row * a.max_len;
      const int2* t_in = a.table + (int64_t)e.r * a.max_len * a.layers + e.layer;
      int32_t* keep = a.keep + e.row * a.budget + pos;
      float* w_out = a.weight_out + e.row * a.max_len_out + pos;
      int2* t_out = a.table_out + ((int64_t)e.r * a.max_len_out + pos) * a.layers + e.layer;
      constexpr int kBatch = 4;                            // reads a thread has in flight
      const int n_out = min(n_kept, e.n_keep - pos);       // equal; no write passes the row whatever the counts say
      for (int i0 = lane; i0 < n_out; i0 += 32 * kBatch) {
        int j[kBatch];
        float x[kBatch];
        int2 pages[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) j[b] = list[min(i0 + 32 * b, n_out - 1)];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          x[b] = w[j[b]];
          pages[b] = t_in[(int64_t)j[b] * a.layers];
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + 32 * b;
          if (i >= n_out) break;
          keep[i] = j[b];
          w_out[i] = x[b];
          t_out[(int64_t)i * a.layers] = pages[b];
        }
      }
    }
    pos += n_kept;
    __syncwarp();
  }
  const int step = n_cta * kEvictThreads, first = e.n_keep + rank * kEvictThreads + tid;
  int32_t* keep = a.keep + e.row * a.budget;
  float* w_out = a.weight_out + e.row * a.max_len_out;
  int2* t_out = a.table_out + (int64_t)e.r * a.max_len_out * a.layers + e.layer;
  for (int i = first; i < a.budget; i += step) keep[i] = -1;
  for (int i = first; i < a.max_len_out; i += step) {
    w_out[i] = 0.f;
    t_out[(int64_t)i * a.layers] = make_int2(-1, -1);
  }
  if (e.layer == 0 && rank == 0 && tid == 0) a.new_len[e.r] = e.n_keep;
  if (kCluster && select) cluster_wait();                  // and no other reads this one's
}

// Many short rows: four a CTA, four warps each.  Layers of one request are neighbours, and the page
// table [token][layer] is compacted for the four together, so that four lanes write a 32-byte sector of
// which a row by itself would write 8 bytes at a time.  The keys stay in shared memory: the first
// digit is counted while they come in, a warp's kept positions take the place of the keys it has read,
// and one exchange of counts numbers them.  64 requests x 40 layers of 500 to 2,048 tokens to 1,024:
// 31 us (a CTA per row 73); with the keys in registers, whose passes are unrolled to the longest row,
// 39; three CTAs per SM with 40 registers 34, two or three rows a CTA 33 and 32.
constexpr int kShortRow = 4096;                            // four rows a CTA up to this length
constexpr int kShortRows = 4, kShortThreads = 128 * kShortRows;
constexpr int kEvictLoads = 8;                             // weights a lane has on their way

__global__ void __launch_bounds__(kShortThreads, 2) kv_evict_rows_kernel(const EvictArgs a, int32_t cap) {
  constexpr int kRows = kShortRows, kRowWarps = 4, n_thr = 32 * kRowWarps, kPer = kEvictBins / n_thr;
  extern __shared__ __align__(16) int smem_evict[];
  __shared__ int warp_sum[kRows * kRowWarps], found_s[kRows][3];
  __shared__ int out_s[kRows][kRowWarps], part_s[kRows], keep_s[kRows];   // outputs before a warp's, its part's length
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = warp / kRowWarps, part = warp % kRowWarps, rtid = part * 32 + lane;
  int* hist = smem_evict + slot * kEvictBins;
  int* keys = smem_evict + kRows * kEvictBins + slot * cap;
  for (int i = tid; i < kEvictBins * kRows / 4; i += kShortThreads)
    reinterpret_cast<int4*>(smem_evict)[i] = make_int4(0, 0, 0, 0);
  const auto row_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "n"(n_thr) : "memory"); };
  pdl_wait_then_release();
  const int rows = a.n_req * a.layers, id = blockIdx.x * kRows + slot;
  const bool live = id < rows;                             // the last CTA may have rows to spare
  EvictRow e{};
  if (live) e = evict_row(a, id, rtid == 0);
  const int per_warp = ((e.n + kRowWarps - 1) / kRowWarps + 31) & ~31;
  const int w0 = min(e.n, part * per_warp), w1 = min(e.n, w0 + per_warp);
  const bool select = live && e.need > 0 && e.need < e.old;
  const float* w = a.weight + e.row * a.max_len;
  __syncthreads();
  for (int j0 = w0 + lane; j0 - lane < w1; j0 += 32 * kEvictLoads) {
    float x[kEvictLoads];
#pragma unroll
    for (int b = 0; b < kEvictLoads; ++b) x[b] = j0 + 32 * b < w1 ? w[j0 + 32 * b] : 0.f;
#pragma unroll
    for (int b = 0; b < kEvictLoads; ++b) {
      const int j = j0 + 32 * b;
      if (j >= w1) continue;
      const uint32_t k = j >= e.old ? kKeyStays : weight_key(x[b]);
      keys[j] = (int)k;
      if (select && k != kKeyStays) atomicAdd(&hist[kEvictBins - 1 - (k >> (32 - kEvictBits))], 1);   // largest first
    }
  }
  const auto key = [&](int j) { return j < w1 ? (uint32_t)keys[j] : kKeyAbsent; };
  if (select) {
    uint32_t prefix = 0, mask = 0;
    int need = e.need;
    for (int d = 0, bits = 32; bits > 0; ++d) {
      const int nb = min(kEvictBits, bits);
      bits -= nb;
      const uint32_t digit = (1u << nb) - 1;
      if (d > 0) {
        for (int j0 = w0 + lane; j0 - lane < w1; j0 += 32 * kEvictBatch) {
          uint32_t k[kEvictBatch];
#pragma unroll
          for (int b = 0; b < kEvictBatch; ++b) k[b] = key(j0 + 32 * b);
#pragma unroll
          for (int b = 0; b < kEvictBatch; ++b)
            if ((k[b] & mask) == prefix) atomicAdd(&hist[digit - ((k[b] >> bits) & digit)], 1);   // the marks match no prefix
        }
      }
      row_sync();
      // every thread adds up kPer neighbouring bins, and the row's threads find the one they lie in
      int v[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; i += 4) {
        int4* bins = reinterpret_cast<int4*>(hist + rtid * kPer + i);
        const int4 x = *bins;
        *bins = make_int4(0, 0, 0, 0);
        v[i] = x.x;
        v[i + 1] = x.y;
        v[i + 2] = x.z;
        v[i + 3] = x.w;
        mine += x.x + x.y + x.z + x.w;
      }
      const int incl = warp_scan(mine, lane);
      if (lane == 31) warp_sum[warp] = incl;
      row_sync();
      int above = incl - mine;
#pragma unroll
      for (int i = 0; i < kRowWarps; ++i) above += i < part ? warp_sum[slot * kRowWarps + i] : 0;
      if (above < need && above + mine >= need) {          // one thread
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (above < need && above + v[i] >= need) {
            found_s[slot][0] = rtid * kPer + i;
            found_s[slot][1] = above;
            found_s[slot][2] = v[i];
          }
          above += v[i];
        }
      }
      row_sync();
      need -= found_s[slot][1];
      const bool whole = found_s[slot][2] == need;         // the whole bin stays
      prefix |= (digit - (uint32_t)found_s[slot][0]) << bits;
      mask |= digit << bits;
      e.cut = whole ? prefix - 1 : prefix;
      e.ties = whole ? 0 : need;
      if (whole) break;
    }
  }
  int tied = 0;                                            // keys equal to the cut before this warp's part
  if (e.ties > 0) {
    int eq = 0;
    for (int j = w0 + lane; j < w1; j += 32) eq += (uint32_t)keys[j] == e.cut;
    eq = __reduce_add_sync(0xffffffffu, eq);
    row_sync();                                            // warp_sum has been read
    if (lane == 0) warp_sum[warp] = eq;
    row_sync();
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) tied += i < part ? warp_sum[slot * kRowWarps + i] : 0;
  }
  // the kept positions, in place of the keys this warp has read
  const uint32_t below = (1u << lane) - 1;
  int* list = keys + w0;
  int n_kept = 0;
  for (int j0 = w0 + lane; j0 - lane < w1; j0 += 32 * kEvictBatch) {
    uint32_t k[kEvictBatch];
#pragma unroll
    for (int b = 0; b < kEvictBatch; ++b) k[b] = key(j0 + 32 * b);
    __syncwarp();
#pragma unroll
    for (int b = 0; b < kEvictBatch; ++b) {
      bool stay = k[b] > e.cut;
      if (e.ties > 0) {
        const bool q = k[b] == e.cut;
        const uint32_t mq = __ballot_sync(0xffffffffu, q);
        stay = stay || (q && tied + __popc(mq & below) < e.ties);
        tied += __popc(mq);
      }
      const uint32_t ms = __ballot_sync(0xffffffffu, stay);
      if (stay) list[n_kept + __popc(ms & below)] = j0 + 32 * b;
      n_kept += __popc(ms);
    }
    __syncwarp();
  }
  row_sync();                                              // warp_sum has been read
  if (lane == 0) warp_sum[warp] = n_kept;
  row_sync();
  int pos = 0;
#pragma unroll
  for (int i = 0; i < kRowWarps; ++i) pos += i < part ? warp_sum[slot * kRowWarps + i] : 0;
  if (lane == 0) out_s[slot][part] = pos;
  if (rtid == 0) {
    part_s[slot] = per_warp;
    keep_s[slot] = e.n_keep;
  }
  __syncthreads();
  if (live) {
    int32_t* keep = a.keep + e.row * a.budget;
    float* w_out = a.weight_out + e.row * a.max_len_out;
    const int n_out = min(n_kept, e.n_keep - pos);         // equal; no write passes the row whatever the counts say
    for (int i0 = lane; i0 < n_out; i0 += 32 * kEvictBatch) {
      int j[kEvictBatch];
      float x[kEvictBatch];
#pragma unroll
      for (int b = 0; b < kEvictBatch; ++b) j[b] = list[min(i0 + 32 * b, n_out - 1)];
#pragma unroll
      for (int b = 0; b < kEvictBatch; ++b) x[b] = w[j[b]];
#pragma unroll
      for (int b = 0; b < kEvictBatch; ++b) {
        if (i0 + 32 * b >= n_out) break;
        keep[pos + i0 + 32 * b] = j[b];
        w_out[pos + i0 + 32 * b] = x[b];
      }
    }
    for (int i = e.n_keep + rtid; i < a.budget; i += n_thr) keep[i] = -1;
    for (int i = e.n_keep + rtid; i < a.max_len_out; i += n_thr) w_out[i] = 0.f;
    if (e.layer == 0 && rtid == 0) a.new_len[e.r] = e.n_keep;
  }

  // the page table of the CTA's rows: thread = (position, row), rows fastest
  const int trow = tid % kRows, tid_row = blockIdx.x * kRows + trow;
  if (tid_row >= rows) return;
  const int layer = tid_row % a.layers, r = tid_row / a.layers, n_keep = keep_s[trow], per = part_s[trow];
  const int o1 = out_s[trow][1], o2 = out_s[trow][2], o3 = out_s[trow][3];
  const int2* t_in = a.table + (int64_t)r * a.max_len * a.layers + layer;
  int2* t_out = a.table_out + (int64_t)r * a.max_len_out * a.layers + layer;
  const int* kept = smem_evict + kRows * kEvictBins + trow * cap;
  constexpr int kStep = kShortThreads / kRows, kBatch = 8; // positions a pass of the CTA covers, reads in flight
  for (int i0 = tid / kRows; i0 < n_keep; i0 += kStep * kBatch) {
    int2 pages[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = min(i0 + kStep * b, n_keep - 1);
      const int p = (i >= o1) + (i >= o2) + (i >= o3);     // the warp that kept it
      const int j = kept[p * per + i - (p == 0 ? 0 : p == 1 ? o1 : p == 2 ? o2 : o3)];
      pages[b] = t_in[(int64_t)j * a.layers];
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i0 + kStep * b >= n_keep) break;
      t_out[(int64_t)(i0 + kStep * b) * a.layers] = pages[b];
    }
  }
  for (int i = n_keep + tid / kRows; i < a.max_len_out; i += kStep) t_out[(int64_t)i * a.layers] = make_int2(-1, -1);
}

int launch_evict_rows(const lora_pool* p, const EvictArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.n_req * a.layers;
  const int cap = (a.max_len + 31) & ~31;
  static DeviceFlags flags;
  const int rc = ensure_smem_attr(flags, &kv_evict_rows_kernel, kShortRows * (kEvictBins + kShortRow) * (int)sizeof(int), "lora_kv_evict");
  if (rc != LORA_OK) return rc;
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e = launch_pdl(!p->prof_on, kv_evict_rows_kernel, dim3((unsigned)((rows + kShortRows - 1) / kShortRows)), dim3(kShortThreads),
                                   kShortRows * (size_t)(kEvictBins + cap) * sizeof(int), st, a, (int32_t)cap);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_evict launch");
}

template <int K, bool kCluster>
int launch_evict(const lora_pool* p, const EvictArgs& a, int n_cta, cudaStream_t st) {
  const int64_t rows = (int64_t)a.n_req * a.layers;
  constexpr int smem = ((kCluster ? 2 : 1) * kEvictBins + kEvictWarps * 32 * K) * (int)sizeof(int);
  static DeviceFlags flags;
  const int rc = ensure_smem_attr(flags, &kv_evict_kernel<K, kCluster>, smem, "lora_kv_evict");
  if (rc != LORA_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kCluster ? rows * n_cta : rows));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p->prof_on ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = n_cta;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_evict_kernel<K, kCluster>, a, (int32_t)n_cta);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_evict launch");
}

template <bool kCluster>
int launch_evict_k(const lora_pool* p, const EvictArgs& a, int n_cta, cudaStream_t st) {
  const int64_t per_cta = (((int64_t)a.max_len + n_cta - 1) / n_cta + 31) / 32 * 32;
  const int64_t chunks = ((per_cta + kEvictWarps - 1) / kEvictWarps + 31) / 32;      // of a warp, at most
  return chunks <= 4    ? launch_evict<4, kCluster>(p, a, n_cta, st)
         : chunks <= 8  ? launch_evict<8, kCluster>(p, a, n_cta, st)
         : chunks <= 12 ? launch_evict<12, kCluster>(p, a, n_cta, st)
         : chunks <= 16 ? launch_evict<16, kCluster>(p, a, n_cta, st)
         : chunks <= 20 ? launch_evict<20, kCluster>(p, a, n_cta, st)
         : chunks <= 24 ? launch_evict<24, kCluster>(p, a, n_cta, st)
                        : launch_evict<32, kCluster>(p, a, n_cta, st);
}

}  // namespace

extern "C" int lora_kv_write(lora_pool* p, int32_t n_rows, const int32_t* row_req, const int32_t* row_pos, const void* k,
                             const void* v, int64_t k_stride, int64_t v_stride, int32_t n_req,
                             const int32_t* table_dev, int32_t max_len, int32_t layers, int32_t layer,
                             lora_stream_t stream) {
  if (!p || n_rows < 0 || n_req < 0 || max_len < 0 || layers < 1 || layer < 0 || layer >= layers)
    return lora_fail(LORA_EINVAL, "lora_kv_write: bad arguments");
  if (n_rows > 0 && (!row_req || !row_pos || !k || !v || !table_dev))
    return lora_fail(LORA_EINVAL, "lora_kv_write: null pointer");
  if (k_stride == 0) k_stride = p->H;
  if (v_stride == 0) v_stride = p->H;
  if (k_stride < p->H || v_stride < p->H || ((k_stride | v_stride) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_write: row strides must be multiples of 8 and at least H");
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_write: k and v must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(table_dev) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_write: the table must be 8-byte aligned");
  if (((reinterpret_cast<uintptr_t>(row_req) | reinterpret_cast<uintptr_t>(row_pos)) & 3) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_write: row_req and row_pos must be 4-byte aligned");
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_kv_write: planning pool has no device state");
  if (n_rows == 0) return LORA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope prof(p, LORA_KIND_KV, st);
  const auto launch = [&](auto* kernel, int64_t warps) {
    const int per = kWriteThreads / 32;
    return launch_pdl(!p->prof_on, kernel, dim3((unsigned)((warps + per - 1) / per)), dim3(kWriteThreads), 0, st,
                      static_cast<uint16_t*>(p->pool_dev), p->num_pages, p->H, n_rows, row_req, row_pos,
                      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride, n_req,
                      reinterpret_cast<const int2*>(table_dev), max_len, layers, layer, p->d_err);
  };
  const int64_t rows = n_rows;
  const bool packed = p->H <= kWritePackedMaxH && 2 * rows > 64 * (int64_t)device_sm_count();
  const cudaError_t e = !packed       ? launch(kv_write_kernel, 2 * rows)
                        : p->H <= 64  ? launch(kv_write_packed_kernel<8>, (rows + 15) / 16)
                        : p->H <= 128 ? launch(kv_write_packed_kernel<16>, (rows + 7) / 8)
                                      : launch(kv_write_packed_kernel<32>, (rows + 3) / 4);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_write launch");
}

extern "C" int lora_kv_evict(lora_pool* p, int32_t n_req, const int32_t* table_dev, const int32_t* seq_len_dev,
                             int32_t max_len, int32_t layers, const float* weight_dev, int32_t budget, int32_t recent,
                             int32_t* keep_dev, int32_t* new_len_dev, int32_t* table_out, float* weight_out,
                             int32_t max_len_out, lora_stream_t stream) {
  if (!p || n_req < 0 || max_len < 1 || layers < 1) return lora_fail(LORA_EINVAL, "lora_kv_evict: bad arguments");
  if (budget < 1 || recent < 0 || recent > budget)
    return lora_fail(LORA_EINVAL, "lora_kv_evict: budget must be at least 1 and recent within [0, budget]");
  if (max_len > (1 << 30) || max_len_out > (1 << 30) || budget > (1 << 30))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: max_len, max_len_out and budget are at most 2^30");
  if (max_len_out < std::min(budget, max_len))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: max_len_out is below min(budget, max_len)");
  if (n_req > 0 && (!table_dev || !seq_len_dev || !weight_dev || !keep_dev || !new_len_dev || !table_out ||
                    !weight_out))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: null pointer");
  if (((reinterpret_cast<uintptr_t>(table_dev) | reinterpret_cast<uintptr_t>(table_out)) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_evict: tables must be 8-byte aligned");
  if (((reinterpret_cast<uintptr_t>(seq_len_dev) | reinterpret_cast<uintptr_t>(weight_dev) |
        reinterpret_cast<uintptr_t>(keep_dev) | reinterpret_cast<uintptr_t>(new_len_dev) |
        reinterpret_cast<uintptr_t>(weight_out)) & 3) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_evict: lengths, weights and positions must be 4-byte aligned");
  if (n_req > 0 && (table_dev == table_out || weight_dev == weight_out || seq_len_dev == new_len_dev))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: outputs must not be the inputs");
  if ((int64_t)n_req * layers > (1 << 30)) return lora_fail(LORA_EINVAL, "lora_kv_evict: too many (request, layer) rows");
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_kv_evict: planning pool has no device state");
  if (n_req == 0) return LORA_OK;
  EvictArgs a{};
  a.n_req = n_req;
  a.table = reinterpret_cast<const int2*>(table_dev);
  a.seq_len = seq_len_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.weight = weight_dev;
  a.budget = budget;
  a.recent = recent;
  a.keep = keep_dev;
  a.new_len = new_len_dev;
  a.table_out = reinterpret_cast<int2*>(table_out);
  a.weight_out = weight_out;
  a.max_len_out = max_len_out;
  a.err = p->d_err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)n_req * layers;
  const int sms = device_sm_count();
  // Four rows a CTA where there are enough to fill the SMs (2,560 rows of up to 2,048 tokens 31 us, a
  // CTA each 73; 40 rows 16.4, a CTA each 12.7).
  if (max_len <= kShortRow && rows >= 4 * (int64_t)sms) return launch_evict_rows(p, a, st);
  // Few rows or long ones.  A CTA's registers hold 16,384 weights; beyond that, and as long as all
  // CTAs run at once and slices stay above 2,048 tokens, a cluster per row (one row of 100,000 tokens
  // 20 us with 8 CTAs, 31 with 4; 32 rows of 131,071 37 us with 8, 45 with 4, 60 with 16).
  int n_cta = 1;
  while (n_cta < kEvictMaxCluster && max_len / (2 * n_cta) >= 2048 &&
         (max_len / n_cta > 16384 || rows * n_cta <= 2 * (int64_t)sms) && rows * n_cta * 2 <= INT32_MAX)
    n_cta *= 2;
  return n_cta > 1 ? launch_evict_k<true>(p, a, n_cta, st)
                   : launch_evict_k<false>(p, a, 1, st);
}

extern "C" int lora_kv_append(lora_pool* p, int32_t n_req, const int32_t* count, const int32_t* old_len,
                              const int32_t* pages, int32_t row_cap, int32_t* table_dev, int32_t max_len, int32_t layers,
                              int32_t* new_len, int32_t* row_start, int32_t* row_req, int32_t* row_pos,
                              lora_stream_t stream) {
  if (!p || n_req < 0 || row_cap < 0 || max_len < 1 || layers < 1) return lora_fail(LORA_EINVAL, "lora_kv_append: bad arguments");
  if (n_req > 65535) return lora_fail(LORA_EINVAL, "lora_kv_append: at most 65535 requests per call");
  if (max_len > (1 << 30)) return lora_fail(LORA_EINVAL, "lora_kv_append: max_len is at most 2^30");
  if (layers > (1 << 20)) return lora_fail(LORA_EINVAL, "lora_kv_append: at most 2^20 layers");
  if (!row_start || (n_req > 0 && (!count || !table_dev || !new_len)) || (row_cap > 0 && (!pages || !row_req || !row_pos)))
    return lora_fail(LORA_EINVAL, "lora_kv_append: null pointer");
  if (((reinterpret_cast<uintptr_t>(table_dev) | reinterpret_cast<uintptr_t>(pages)) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_append: table and pages must be 8-byte aligned");
  if (((reinterpret_cast<uintptr_t>(count) | reinterpret_cast<uintptr_t>(old_len) | reinterpret_cast<uintptr_t>(new_len) |
        reinterpret_cast<uintptr_t>(row_start) | reinterpret_cast<uintptr_t>(row_req) |
        reinterpret_cast<uintptr_t>(row_pos)) & 3) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_append: counts, lengths and rows must be 4-byte aligned");
  const struct {
    const void* at;
    double bytes;                                          // may pass 64 bits
    bool out;
  } arrays[] = {{count, 4. * n_req, false}, {old_len, 4. * n_req, false}, {pages, 8. * row_cap * layers, false},
                {table_dev, 8. * n_req * max_len * layers, true}, {new_len, 4. * n_req, true}, {row_start, 4. * (n_req + 1.), true},
                {row_req, 4. * row_cap, true}, {row_pos, 4. * row_cap, true}};
  AppendArgs a{};
  a.n_req = n_req;
  a.count = count;
  a.old_len = old_len;
  // Two layers at a time (64 prompts of 500 to 2,048 tokens, 40 layers 13.9 us; 39 layers, one at a time, 16.5).
  const bool wide = layers % 2 == 0 && ((reinterpret_cast<uintptr_t>(table_dev) | reinterpret_cast<uintptr_t>(pages)) & 15) == 0;
  if (wide) layers /= 2;
  a.pages = pages;
  a.row_cap = row_cap;
  a.table = table_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.new_len = new_len;
  a.row_start = row_start;
  a.row_req = row_req;
  a.row_pos = row_pos;
  a.rows_per_cta = std::min(std::max(kAppendEntries / layers, 1), kAppendMaxRows);
  a.layers_inv = a.rows_per_cta > 1 ? (((uint64_t)1 << 40) + layers - 1) / layers : 0;
  const int64_t rest = old_len ? 0 : ((int64_t)n_req * max_len + a.rows_per_cta - 1) / a.rows_per_cta;
  a.row_ctas = (int32_t)std::max(((int64_t)row_cap + a.rows_per_cta - 1) / a.rows_per_cta, (int64_t)1);
  if (a.row_ctas + rest > INT32_MAX) return lora_fail(LORA_EINVAL, "lora_kv_append: the table is too large for one call");
  for (const auto& x : arrays)                             // CTAs read counts, lengths and pages while others write
    for (const auto& y : arrays)
      if (x.out && &x != &y && x.at && y.at && x.bytes > 0 && y.bytes > 0 &&
          (x.at <= y.at ? (double)(static_cast<const char*>(y.at) - static_cast<const char*>(x.at)) < x.bytes
                        : (double)(static_cast<const char*>(x.at) - static_cast<const char*>(y.at)) < y.bytes))
        return lora_fail(LORA_EINVAL, "lora_kv_append: outputs must not overlap the inputs or one another");
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_kv_append: planning pool has no device state");
  a.err = p->d_err;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e = launch_pdl(!p->prof_on, wide ? kv_append_kernel<int4> : kv_append_kernel<int2>,
                                   dim3((unsigned)(a.row_ctas + rest)), dim3(kAppendThreads), 0, st, a);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_append launch");
}

// Attention of many query rows per sequence: causal over packed prompts, and of trees of drafted tokens
// over the paged KV cache.
//
// Per query head h (KV head h / G, G = n_heads / n_kv_heads, width D) and row i, over the tokens j it sees:
//     s_j = q_{i,h} . k_j / sqrt(D),  lse = log sum_j exp(s_j),  out_{i,h} = sum_j exp(s_j - lse) v_j
// Softmax in base 2: scores carry log2(e) / sqrt(D).
//
// One kernel for both.  A CTA per SM takes items one after another: 128 query rows (tokens or nodes times the group's
// heads) in each of two tiles (one at D = 256), over blocks of 128 tokens of one KV head.  Per tile and block
//     S = Q K^T (tcgen05, Q and K in shared memory, S in TMEM), P = 2^(S - m - 24) as bf16 in the same columns,
//     O += P V (P from TMEM, V in shared memory, O in TMEM for the whole item), l += sum P in fp32,
// so scores and weights never leave the SM.  Warps have roles that hand over by mbarriers: one finds the items, one
// thread issues the MMAs, one warp (tree: four, that gather) keeps a ring of K and V slots filled, a thread per row does
// the softmax and the outputs, with registers taken from the others.  The two tiles alternate: one's products run
// under the other's softmax.
//
// Masks.  A prompt's blocks below the diagonal and a tree's before the first node are seen whole.  In the others the
// softmax threads put -infinity into TMEM first, and infinities and NaN of V, whose products with weights of 0 would be
// NaN, are cleared in shared memory by a warp of its own; the outputs get back those that their row sees.
//
// Weights enter the V product as one bf16 term, off by half a step, 2^-8, at most; the weights' sum takes them unrounded
// in fp32.  Against 64 bits outputs are off by 0.0019 to 0.0024 of their size, their own rounding included (plain fp32
// form, rounded once: 0.0015 to 0.0017).  A second term, 2^-15 in all, is half as many MMAs again and three more
// operations a pair of weights in the softmax, which lies on a tile's chain whatever bounds the call: prompts 103 -> 167
// us (16 of 305 to 1,024 tokens), 1,440 -> 2,124 (16,384 tokens), 65 -> 104 (33 of 40 to 515), 195 -> 262 (D = 256), and trees that
// read pages at HBM's rate 193 -> 223 (64 requests of up to 2,047 tokens) and 319 -> 362 (131,072), of shared heads 135 -> 178.
//
// What bounds it, on one GB300 (MMA 1,952 TFLOP/s, copies 6,763 GB/s as measured):
//   prompts of 16,384 tokens, 32 heads of 128       1,470 us  1,495 TFLOP/s, 0.77 of the burst, 0.87 of the sustained rate
//   7 prompts of 386 to 5,000, 8 KV heads x 4 of 128  299 us  1,357 TFLOP/s: a block takes 3,000 cycles, its MMAs 2,048; a
//                                                             tile's scores wait for its own weights' product
//   2 of 3,926 and 4,097, 8 KV heads x 2 of 256       198 us  1,332 TFLOP/s: likewise, one tile with two score buffers
//   16 of 305 to 1,024, 32 heads of 128               105 us  3.5 TB/s of the inputs and outputs: items of 1 to 8 blocks,
//                                                             of which an item's start and end take 5,000 cycles
//   33 of 40 to 515, 32 KV heads x 2 of 64             67 us  2.5 TB/s: likewise
//   trees of 32 nodes, 64 requests of up to 2,047 tokens, 32 heads of 128   191 us  6.0 TB/s, 0.88 of the copy rate
//   one of 64 nodes, 131,072 tokens, 32 heads of 128                        315 us  6.8 TB/s, 1.00
//   48 nodes, 7 requests of 500 to 33,333 tokens, 8 KV heads x 4 of 128     136 us  4.7 TB/s, 0.69; tensor pipe 0.57 busy
// Pages are gathered by TMA, 256 bytes of each, four a copy (131,072 tokens with 16-byte cp.async instead: 503 us against
// 346 at that step; 4 warps, since a copy takes 50 cycles to issue).
// The CTA's warps share the instruction cache and an item of a short prompt runs through most of the code, so code size
// is time: 80 KB -> 54 KB took 10 to 17 % off short sequences.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "tc_ptx.h"

namespace {

constexpr int kRowsMaxGroup = 16;                   // query heads per KV head
constexpr int kBlock = 128;                         // tokens of K and V at a time
constexpr int kTileRows = 128;                      // query rows of a tile
// Weights are 2^(s - m - kShift), where m is at most kSlack below the largest score so far: any m gives the
// same softmax, and the sums of up to 2^(kShift - kSlack) weights times V stay within the range of V.  With
// the slack a tile's sums are rescaled in few of its blocks.
constexpr float kShift = 24.f, kSlack = 6.f;
// Scores are scaled, and m and the shift taken off, by one fma.  Its product is exact and m times the scale is not: where
// that is off by more than the exponent holds, from 2^31 on, every weight of a row would be 0 or infinite.  A block with
// rows whose m is past kFar has it taken off their scores in TMEM first, which is exact for those that matter (33 short
// prompts 65.9 -> 66.7 us, in registers 66.8 to 69.0: more code).
constexpr float kFar = 1 << 20;
__device__ __forceinline__ bool far(float m) { return fabsf(m) > kFar && fabsf(m) < INFINITY; }

struct RowsArgs {
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  int32_t n_req, n_rows, n_heads, n_kv, group;
  int32_t few;                                      // the CTAs plan for themselves
  int32_t npt;                                      // tokens (or nodes) of a tile: kTileRows / group
  uint32_t group_inv;                               // 2^16 / group, rounded up: (r * group_inv) >> 16 = r / group for a tile's rows
  const int32_t* start;                             // caller's row starts
  int32_t* bounds;                                  // workspace: the same, ascending within [0, n_rows]
  float scale_log2;
  int32_t* err;
  // prompt
  const uint16_t* v;
  int64_t v_stride;
  int32_t* n_items;                                 // workspace: work items per KV head, and they: (sequence, tile pair)
  int2* items;
  int32_t* seq_items;                               // workspace: items that begin with a sequence
  int32_t pack;                                     // short sequences share items
  int32_t heads_at;                                 // KV heads whose items run at the same time
  int32_t tickets;                                  // 0: a fixed share of the items a CTA; else CTAs of the grid, taken by those that run
  // tree
  const uint16_t* pool;
  int64_t num_pages;
  int32_t H;
  const int2* table;
  const int32_t* seq_len;
  int32_t max_len, layers, layer;
  const uint64_t* mask;
  int64_t* prefix;                                  // workspace: [n_req + 1] units of the requests before, per KV head
  int4* ws_start;                                   // [parts] (head, request, pair, last part) of a segment cut behind this part
  float2* ws_ml;                                    // [2 parts][slot_rows] m and l of a partial
  float* ws_acc;                                    // [2 parts][slot_rows][D]
  int32_t parts, slot_rows;
};

// Exclusive sum over the block's threads, and the total.
template <typename T>
__device__ __forceinline__ T block_exclusive(T v, T* part, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  T before = 0;
  total = 0;
  for (int w = 0; w < n; ++w) {
    before += w < warp ? part[w] : 0;
    total += part[w];
  }
  return before + incl - v;
}

// Exclusive maximum likewise (INT32_MIN before the first).
__device__ __forceinline__ int32_t block_exclusive_max(int32_t v, int32_t* part, int32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  int32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = max(incl, x);
  }
  int32_t before = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) before = INT32_MIN;
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  total = INT32_MIN;
  for (int w = 0; w < n; ++w) {
    if (w < warp) before = max(before, part[w]);
    total = max(total, part[w]);
  }
  return before;
}

// Row starts as the running maximum of the caller's, clamped into [0, n_rows]: sequences never overlap.
constexpr int kPlanThreads = 1024;
__device__ void plan_bounds(const RowsArgs& a) {
  __shared__ int32_t part[kPlanThreads / 32];
  int32_t before = INT32_MIN, total;
  for (int i0 = 0; i0 <= a.n_req; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int32_t x = i <= a.n_req ? a.start[i] : INT32_MIN;
    const int32_t m = max(max(x, before), block_exclusive_max(x, part, total));
    before = max(before, total);
    if (i <= a.n_req) {
      const int32_t b = min(max(m, 0), a.n_rows);
      if (b != x) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
      a.bounds[i] = b;
    }
  }
  __syncthreads();
}

// Items that begin with the sequence of rows [first, end), of per rows each.  Packed, sequences that lie in one window
// of as many rows share an item, which the first of them begins; before: the start of the last sequence with rows ahead
// of this one, if any.  An item's sequences are neighbours in q, k and v, so it is loaded like one sequence's, and each
// row is shown the tokens of its own.
__device__ __forceinline__ int prompt_items(bool pack, int per, int before, int first, int end) {
  const int window = pack ? first / per * per : 0;
  if (end <= first || (pack && end <= window + per && before >= window)) return 0;
  return (end - first + per - 1) / per;
}

// The prompts' work items, the longest first: item (s, L) is the L-th tile pair of sequence s, and it reads
// about L + 1 times as much as the first.  Counting sort by L; the order within one L does not matter.
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const RowsArgs a, int32_t per_item, int32_t levels) {
  extern __shared__ int32_t cursor[];                      // [levels]
  __shared__ int32_t part[kPlanThreads / 32];
  const int tid = threadIdx.x;
  for (int i = tid; i < levels; i += kPlanThreads) cursor[i] = 0;
  pdl_wait_then_release();
  plan_bounds(a);
  int32_t before = INT32_MIN, last;
  for (int s0 = 0; s0 < a.n_req; s0 += kPlanThreads) {
    const int s = s0 + tid, first = a.bounds[min(s, a.n_req)], end = a.bounds[min(s + 1, a.n_req)];
    const int32_t ahead = max(before, block_exclusive_max(end > first ? first : INT32_MIN, part, last));
    before = max(before, last);
    if (s >= a.n_req) continue;
    const int n = prompt_items(a.pack, per_item, ahead, first, end);
    a.seq_items[s] = n;
    if (n > 0) atomicAdd(&cursor[n - 1], 1);
  }
  __syncthreads();
  // from the top level down: sequences with this level, then items above it
  const int per = (levels + kPlanThreads - 1) / kPlanThreads, hi = levels - tid * per, lo = max(hi - per, 0);
  int32_t mine = 0, total;
  for (int L = hi - 1; L >= lo; --L) mine += cursor[L];
  int32_t run = block_exclusive<int32_t>(mine, part, total);
  int32_t items = 0;
  for (int L = hi - 1; L >= lo; --L) {
    run += cursor[L];
    cursor[L] = run;
    items += run;
  }
  int32_t at = block_exclusive<int32_t>(items, part, total);
  for (int L = hi - 1; L >= lo; --L) {
    const int32_t n = cursor[L];
    cursor[L] = at;
    at += n;
  }
  if (tid == 0) *a.n_items = total;
  __syncthreads();
  const int warp = tid >> 5, lane = tid & 31;
  for (int s = warp; s < a.n_req; s += kPlanThreads / 32) {
    const int n = a.seq_items[s];
    for (int L = lane; L < n; L += 32) a.items[atomicAdd(&cursor[L], 1)] = make_int2(s, L);
  }
}

// Of a tree request: its nodes that count, its cached tokens, and its units (blocks of tokens times tile groups).
struct TreeReq {
  int row0, nodes, len, base, blocks, groups;
};
template <int RT>
__device__ __forceinline__ TreeReq tree_request(const RowsArgs& a, int row0, int row1, int length) {
  TreeReq q;
  q.row0 = row0;
  q.nodes = min(row1 - row0, LORA_MAX_TREE);
  q.len = min(max(length, 0), a.max_len);
  q.base = max(q.len - q.nodes, 0);
  q.blocks = max((q.len + kBlock - 1) / kBlock, 1);
  q.groups = RT == 1 && a.npt >= LORA_MAX_TREE ? (q.nodes > 0 ? 1 : 0) : (q.nodes + RT * a.npt - 1) / (RT * a.npt);
  return q;
}
__device__ __forceinline__ bool tree_request_bad(const RowsArgs& a, int rows, int length) {
  return length < 0 || length > a.max_len || rows > LORA_MAX_TREE || rows > length;
}

template <int RT>
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const RowsArgs a) {
  __shared__ int64_t part[kPlanThreads / 32];
  pdl_wait_then_release();
  plan_bounds(a);
  int64_t before = 0;
  for (int r0 = 0; r0 < a.n_req; r0 += kPlanThreads) {
    const int r = r0 + threadIdx.x;
    int64_t units = 0, total;
    if (r < a.n_req) {
      const int row0 = a.bounds[r], row1 = a.bounds[r + 1], length = a.seq_len[r];
      if (tree_request_bad(a, row1 - row0, length)) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
      const TreeReq q = tree_request<RT>(a, row0, row1, length);
      units = (int64_t)q.blocks * q.groups;
    }
    const int64_t at = before + block_exclusive<int64_t>(units, part, total);
    if (r < a.n_req) a.prefix[r] = at;
    before += total;
  }
  if (threadIdx.x == 0) a.prefix[a.n_req] = before;
}

// ---- the kernel ----------------------------------------------------------------------------------
// An item is two tiles of query rows that work side by side (one tile at D = 256): rows of one KV head, which share
// its K and V blocks, or with kPair the same rows of two neighbouring KV heads.  A pair is taken where one tile holds a
// whole tree of 64 nodes (G <= 2), so that the second would be empty: 64 requests of 128 to 2,048 tokens, 32 heads of 128
// 215 -> 193 us (one request of 705 tokens, 4 heads of 64 10.5 -> 11.4).
template <int D_, bool kTree_, bool kPair_ = false, bool kPack_ = false>
struct Geo {
  static constexpr int D = D_;
  static constexpr bool kTree = kTree_;
  static constexpr bool kPair = kPair_;
  static constexpr bool kPack = kPack_;                    // prompt: short sequences share items
  static constexpr int NT = D == 256 ? 1 : 2;              // tiles of an item
  static constexpr int RT = kPair ? 1 : NT;                // of the rows of one head
  static constexpr int HT = kPair ? NT : 1;                // heads
  static_assert(!kPair || NT == 2, "a pair has two tiles");
  static constexpr int NB = 3 - NT;                        // score buffers of a tile
  static constexpr int DS = D < 128 ? D : 128;             // features of a ring slot
  static constexpr int PD = D / DS;                        // slots of a block of K or of V
  static constexpr int PANELS = DS / 64;                   // 128-byte wide panels of a slot
  static constexpr uint32_t kPanel = kBlock * 128;
  static constexpr uint32_t kSlot = PANELS * kPanel;
  static constexpr uint32_t kQTile = kTileRows * D * 2;
  static constexpr int NS = D == 64 ? 10 : 5;              // slots
  static constexpr int kSoftWarps = 4 * NT;
  static constexpr int kMmaWarp = kSoftWarps;
  static constexpr int kPlanWarp = kSoftWarps + 1;         // finds the items; tree: loads Q
  static constexpr int kLoadWarp = kSoftWarps + (kTree ? 4 : 2);        // prompt: one warp that loads Q, K and V; tree: four that gather K and V
  static constexpr int kLoadWarps = kTree ? 4 : 1;
  static constexpr int kScanWarp = kSoftWarps + (kTree ? 2 : 3);
  static constexpr int kScanWarps = kTree ? 2 : 1;
  static constexpr int kThreads = 32 * (kSoftWarps + (kTree ? 8 : 4));       // whole warpgroups: they trade registers
  // Registers a thread: a softmax thread holds a row of scores (without the trade 16 prompts 151 -> 177 us).  Launch 128
  // or 168 (D = 256: 168 or 232).
  static constexpr int kSoftRegs = NT == 1 ? 232 : kTree ? 192 : 208;
  static constexpr int kOtherRegs = NT == 1 ? (kTree ? 136 : 232) : kTree ? 64 : 88;
  static constexpr uint32_t kData = NT * kQTile + NS * kSlot;
  // barriers: full and empty per slot, landed and clean per guarded V slot in turn; Q full and empty; scores and
  // weights (two halves) per buffer; sums full and drained per tile; products
  static constexpr int kItems = 4;                         // items handed out at a time
  static constexpr int kTakers = kSoftWarps + 1 + kScanWarps + kLoadWarps;      // warps that take every item
  static constexpr int kBars = 4 * NS + 2 + 2 + 4 + 4 + 1 + 2 * kItems + 1;
  static constexpr int kWordsRing = 8;                     // blocks whose token masks are kept
  static constexpr uint32_t kTmemO = 256;                  // scores in columns [0, 256), sums behind them
};

__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// Four rows of a tensor map whose box is one row high, one behind another in shared memory; rows outside the tensor
// are zero.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int4 rows, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Read once: the last to stay in L2 (D = 256 at 4,097 tokens 201 -> 199 us).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b64 pol;\n\tcreatepolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], pol;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// mbar_wait in fewer instructions, for the kernel has some thirty waits and its warps share the instruction cache: it
// counts polls instead of cycles, 3 KB less code and 1 to 2 % of the time of short prompts.  A poll of a phase that does
// not end takes 22 to 8,000 cycles, so the limit lies between 50 ms and 20 s; what is waited for takes microseconds,
// and some 3 ms at most where a tile's outputs get infinities back.
constexpr uint32_t kWaitPolls = 1u << 22;
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}
// A wait that lasts as long as an item does: of a tree, whose items have up to 2^23 blocks, for as long as the CTA's
// products go on (an item of 12 million tokens takes some 150 ms).  Its code costs trees of shared heads 1.5 %: 131.8 -> 133.8 us.
template <bool kTree>
__device__ __forceinline__ bool wait_item(uint32_t bar, uint32_t parity, const volatile uint32_t* blocks) {
  if (!kTree) return wait_for(bar, parity);
  uint32_t seen;
  do {
    seen = *blocks;
    if (wait_for(bar, parity)) return true;
  } while (seen != *blocks);
  return false;
}
// Takes a CTA of the grid that has not been launched out of it, in place of the hardware: 16 bytes into shared memory
// say whether there was one, and which.  Not to be asked again after a no.
__device__ __forceinline__ void try_cancel(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst), "r"(bar) : "memory");
}
__device__ __forceinline__ int cancelled(uint32_t src) {   // the CTA's index, or -1
  int x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "mov.s32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}" : "=r"(x) : "r"(src) : "memory");
  return x;
}
// One thread of the warp, the same every time.  The compiler knows that a branch on it leaves one thread and keeps
// descriptors in uniform registers: eight MMAs issue in 80 cycles, behind a branch on the lane's number in 490.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {      // NaN counts as missing
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two fp32 values in one register pair: x * s + b, and sums.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// v[e] of lane j becomes v[j] of lane e, for every four lanes.
__device__ __forceinline__ void transpose_4x4(uint4 (&v)[4], int lane) {
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e & s) continue;
      const uint4 x = v[e], y = v[e | s];
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, up ? x.x : y.x, s);
      got.y = __shfl_xor_sync(0xffffffffu, up ? x.y : y.y, s);
      got.z = __shfl_xor_sync(0xffffffffu, up ? x.z : y.z, s);
      got.w = __shfl_xor_sync(0xffffffffu, up ? x.w : y.w, s);
      v[e] = make_uint4(up ? got.x : x.x, up ? got.y : x.y, up ? got.z : x.z, up ? got.w : x.w);
      v[e | s] = make_uint4(up ? y.x : got.x, up ? y.y : got.y, up ? y.z : got.z, up ? y.w : got.w);
    }
  }
}
// A bf16 pair's halves with an exponent of all ones (infinity, NaN): 0x8000 and 0x80000000.
__device__ __forceinline__ uint32_t non_finite2(uint32_t u) { return ((u & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t u, uint32_t bad) {
  return u & ~((bad & 0x8000u ? 0xFFFFu : 0u) | (bad & 0x80000000u ? 0xFFFF0000u : 0u));
}
// 16 bytes of V in shared memory: whether they hold an infinity or NaN, and those bytes without them.
__device__ __forceinline__ bool non_finite16(uint32_t addr) {
  const uint4 x = lds128(addr);
  return (non_finite2(x.x) | non_finite2(x.y) | non_finite2(x.z) | non_finite2(x.w)) != 0;
}
__device__ __forceinline__ void clean16(uint32_t addr) {
  uint4 x = lds128(addr);
  x.x = finite_or_zero(x.x, non_finite2(x.x));
  x.y = finite_or_zero(x.y, non_finite2(x.y));
  x.z = finite_or_zero(x.z, non_finite2(x.z));
  x.w = finite_or_zero(x.w, non_finite2(x.w));
  sts128(addr, x);
}

// Of 32 tokens those from the first to the last, a bit each; either may lie outside.
__device__ __forceinline__ uint32_t prompt_sees(int first, int last) {
  const uint32_t v = last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u;
  return first <= 0 ? v : first >= 32 ? 0u : v & (0xffffffffu << first);
}

// What a CTA works on at a time: the rows of a tile pair of one sequence and KV head, over some blocks of its tokens.
struct Item {
  int head;                      // KV head
  int req;
  int row0, pos0, count;         // first row of the item, that row's token (prompt) or node (tree), rows' tokens or nodes left from it on
  int b0, b1;                    // blocks of tokens
  int guard;                     // first block in which some row does not see every token
  // tree
  int len, base;                 // cached tokens (prompt: sequences), the first node's position
  int slot;                      // partial, or -1: the item has all blocks
  int nb0, nb1;                  // blocks of the tiles, 0: no rows
};

// Shared memory behind the tiles of Q and the ring.
constexpr int kFew = 127;                                  // sequences that a CTA plans for itself, at most
template <typename G>
struct Tail {
  uint64_t bars[G::kBars];
  uint32_t words[G::kWordsRing][4];      // a block's tokens that have data, a bit each
  int32_t first_bad;                     // this CTA's first item with V cleared of infinities
  uint32_t bad[8][G::kScanWarps][2][4];  // which tokens' of its guarded blocks, an item's in turn: 64 nodes, 128 tokens,
                                         // or 256 from a multiple of 256 on lie in two blocks
  uint32_t tmem;
  uint32_t blocks;                       // tree: blocks whose products are issued
  uint32_t guard_slot[G::NS];            // where guarded V slots lie, in turn
  Item items[G::kItems];
  int32_t bounds[kFew + 1];              // few sequences: their row starts, and
  int32_t units[kFew + 1];               // items (prompt) or units of the requests before (tree)
  alignas(16) int32_t ids[4][32];        // tree: a loading warp's pages; prompt: the answer of try_cancel
};
template <typename G>
constexpr uint32_t smem_bytes() { return G::kData + sizeof(Tail<G>); }

// The items of a CTA, one after another, found by one warp.  Up to kFew sequences it looks at the caller's starts and
// lengths itself; beyond, a kernel before this one has listed the items (prompt) or added up the units (tree).  With that
// kernel always: 4 prompts of 4 to 9 tokens 6.5 -> 13.0 us, one tree behind 705 tokens 11.5 -> 15.4, 127 prompts of 40 tokens
// 36.1 -> 41.7, 33 of 40 to 515 66.9 -> 71.4; every CTA reads the starts, so the limit is four of them a lane.
template <typename G>
struct Walk {
  int32_t* bounds_s;             // few: Tail's
  int32_t* units_s;
  int w, step, all;              // prompt: turn (or the ticket's next item), CTAs, items of a head
  uint32_t ticket, bar_ticket, asked;      // tickets: their place and barrier in shared memory, how many so far
  bool failed;
  int top;                       // prompt, few: the highest level
  int64_t u, u1, per_head;       // tree: units left are [u, u1)

  __device__ __forceinline__ Walk(const RowsArgs& a, int32_t* bounds, int32_t* units) : bounds_s(bounds), units_s(units) {
    const int lane = threadIdx.x & 31, heads = (a.n_kv + G::HT - 1) / G::HT;
    int total = 0, most = 0;
    if (a.few) {
      bool bad = false;
      int32_t carry = INT32_MIN;
#pragma unroll 1
      for (int r0 = 0; r0 <= a.n_req; r0 += 32) {          // the running maximum, as plan_bounds
        const int r = r0 + lane;
        const int32_t x = a.start[min(r, a.n_req)];
        int32_t m = max(x, carry);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t y = __shfl_up_sync(0xffffffffu, m, o);
          if (lane >= o) m = max(m, y);
        }
        carry = __shfl_sync(0xffffffffu, m, 31);
        const int32_t b = min(max(m, 0), a.n_rows);
        if (r <= a.n_req) {
          bad |= b != x;
          bounds_s[r] = b;
        }
      }
      __syncwarp();
      int ahead = INT32_MIN;                               // prompt: the start of the last sequence with rows so far
#pragma unroll 1
      for (int r0 = 0; r0 < a.n_req; r0 += 32) {
        const int r = min(r0 + lane, a.n_req - 1);
        const bool live = r0 + lane < a.n_req;
        const int row0 = bounds_s[r], row1 = bounds_s[r + 1];
        int n = 0;
        if (G::kTree) {
          const int length = a.seq_len[r];
          bad |= tree_request_bad(a, row1 - row0, length);
          const TreeReq q = tree_request<G::RT>(a, row0, row1, length);
          if (live) n = q.blocks * q.groups;
          int incl = n;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          if (live) units_s[r] = total + incl - n;
          total += __shfl_sync(0xffffffffu, incl, 31);
        } else {
          int before = INT32_MIN;
          if (G::kPack) {
            int m = row1 > row0 ? row0 : INT32_MIN;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int y = __shfl_up_sync(0xffffffffu, m, o);
              if (lane >= o) m = max(m, y);
            }
            before = __shfl_up_sync(0xffffffffu, m, 1);
            before = lane == 0 ? ahead : max(ahead, before);
            ahead = max(ahead, __shfl_sync(0xffffffffu, m, 31));
          }
          if (live) n = prompt_items(G::kPack, G::RT * a.npt, before, row0, row1);
          if (live) units_s[r] = n;
          total += __reduce_add_sync(0xffffffffu, n);
          most = max(most, (int)__reduce_max_sync(0xffffffffu, n));
        }
      }
      __syncwarp();
      if (bad && blockIdx.x == 0) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    }
    if (G::kTree) {
      per_head = a.few ? total : a.prefix[a.n_req];
      const int64_t units = per_head * heads, parts = min((int64_t)a.parts, units), p = blockIdx.x;
      u = p < parts ? p * units / parts : 0;
      u1 = p < parts ? (p + 1) * units / parts : 0;
    } else {
      w = a.tickets ? (int)blockIdx.x : 0;
      asked = 0;
      failed = false;
      step = gridDim.x;
      top = most - 1;
      all = a.few ? total : *a.n_items;
    }
  }
  // The part that holds unit x of all heads.
  __device__ __forceinline__ int part_of(const RowsArgs& a, int64_t x) const {
    const int64_t total = per_head * ((a.n_kv + G::HT - 1) / G::HT);
    return (int)(((x + 1) * min((int64_t)a.parts, total) - 1) / total);
  }
  // All lanes of a warp take part.
  __device__ __forceinline__ bool next(const RowsArgs& a, Item& it) {
    const int lane = threadIdx.x & 31;
    if (G::kTree) {
      if (u >= u1) return false;
      const int head = (int)(u / per_head);
      const int64_t x = u - head * per_head;
      int lo = 0;                                          // the request: prefix[lo] <= x < prefix[lo + 1]
      if (a.few) {
#pragma unroll 1
        for (int r0 = 0; r0 < a.n_req; r0 += 32) lo += __popc(__ballot_sync(0xffffffffu, r0 + lane < a.n_req && units_s[min(r0 + lane, kFew)] <= x));
        --lo;
      } else {
        int hi = a.n_req;                                  // 32 places a turn
#pragma unroll 1
        while (hi - lo > 1) {
          const int stride = (hi - lo + 31) / 32, at = lo + lane * stride;
          const unsigned in = __ballot_sync(0xffffffffu, at < hi && a.prefix[min(at, hi)] <= x);
          lo += (31 - __clz(in)) * stride;
          hi = min(hi, lo + stride);
        }
      }
      const int32_t* bounds = a.few ? bounds_s : a.bounds;
      const TreeReq q = tree_request<G::RT>(a, bounds[lo], bounds[lo + 1], a.seq_len[lo]);
      const int64_t y = x - (a.few ? units_s[lo] : a.prefix[lo]);
      it.req = lo;
      const int group = (int)y / q.blocks;                 // a request has fewer than 2^31 units
      it.head = head * G::HT;
      it.b0 = (int)y - group * q.blocks;
      it.b1 = (int)min((int64_t)q.blocks, it.b0 + (u1 - u));
      it.pos0 = group * G::RT * a.npt;
      it.row0 = q.row0 + it.pos0;
      it.count = q.nodes - it.pos0;
      it.len = q.len;
      it.base = q.base;
      it.guard = q.base / kBlock;
      it.slot = it.b0 == 0 && it.b1 == q.blocks ? -1 : 2 * (int)blockIdx.x + (it.b0 == 0 ? 1 : 0);
      // cut behind this part: the join goes on to the part of its last unit
      if (lane == 0 && it.slot >= 0 && it.b0 == 0)
        a.ws_start[blockIdx.x] = make_int4(it.head, it.row0, min(it.count, G::RT * a.npt), part_of(a, u + q.blocks - 1));
      u += it.b1 - it.b0;
      return true;
    }
    // Some heads at a time (their K and V stay in L2), of these the longest items of all sequences first.
    int x = w;
    if (a.tickets == 0) {                                  // there and back over the CTAs: none has the longer item of every turn
      x = w * step + ((w & 1) ? step - 1 - (int)blockIdx.x : (int)blockIdx.x);
      if (x >= all * a.n_kv) return false;
      ++w;
    } else {
      while (x >= all * a.n_kv) {                          // none (left) of this ticket
        if (lane == 0) {
          fence_proxy_async_shared();
          mbar_arrive_expect_tx(bar_ticket, 16);
          try_cancel(ticket, bar_ticket);
        }
        __syncwarp();
        const bool got = __all_sync(0xffffffffu, wait_for(bar_ticket, asked++ & 1));
        x = got ? cancelled(ticket) : -1;
        __syncwarp();
        failed = !got;
        if (x < 0) return false;
      }
      w = x + a.tickets;                                   // the item behind the last ticket's
    }
    const int turn = x / (all * a.heads_at), in = x - turn * all * a.heads_at, now = min(a.heads_at, a.n_kv - turn * a.heads_at);
    const int place = in / now;
    int first = 0, end = 0, tile = 0;
    it.head = turn * a.heads_at + in - place * now;
    if (a.few) {
      // The longest first: the lowest level with `place` or fewer items above it; the k-th sequence that has it.
      const auto above = [&](int L) {
        int n = 0;
#pragma unroll 1
        for (int r = lane; r < a.n_req; r += 32) n += max(units_s[r] - 1 - L, 0);
        return __reduce_add_sync(0xffffffffu, n);
      };
      int lo = 0, level = top;
#pragma unroll 1
      while (lo < level) {
        const int mid = (lo + level) / 2;
        if (above(mid) <= place) level = mid;
        else lo = mid + 1;
      }
      int k = place - above(level), s = 0;
#pragma unroll 1
      for (int r0 = 0; r0 < a.n_req; r0 += 32) {
        unsigned has = __ballot_sync(0xffffffffu, r0 + lane < a.n_req && units_s[min(r0 + lane, kFew)] > level);
        const int c = __popc(has);
        if (k < c) {
#pragma unroll 1
          for (; k > 0; --k) has &= has - 1;
          s = r0 + __ffs(has) - 1;
          break;
        }
        k -= c;
      }
      first = bounds_s[s];
      end = bounds_s[s + 1];
      tile = level;
      it.req = s;
    } else {
      const int2 e = a.items[place];
      first = a.bounds[e.x];
      end = a.bounds[e.x + 1];
      it.req = e.x;
      tile = e.y;
    }
    const int per = G::RT * a.npt, window_end = first / per * per + per;
    it.len = 1;
    if (G::kPack && end <= window_end) {                     // with the sequences behind it that end in its window
      const int32_t* bounds = a.few ? bounds_s : a.bounds;
      int lo = it.req + 1, hi = a.n_req;                   // 32 places a turn, bounds[lo] <= window_end
#pragma unroll 1
      while (lo < hi) {
        const int stride = (hi - lo) / 32 + 1, at = lo + lane * stride;
        const unsigned in = __ballot_sync(0xffffffffu, at <= hi && bounds[min(at, hi)] <= window_end);
        lo += (31 - __clz(in)) * stride;
        hi = min(hi, lo + stride - 1);
      }
      end = bounds[lo];
      it.len = lo - it.req;
    }
    it.pos0 = tile * per;
    it.row0 = first + it.pos0;
    it.count = end - first - it.pos0;
    it.b0 = 0;
    it.b1 = (it.pos0 + min(it.count, per) + kBlock - 1) / kBlock;
    it.guard = it.pos0 / kBlock;
    it.slot = -1;
    it.base = 0;
    return true;
  }
  // Of tile t of an item: its KV head, its first row from the item's, its rows' tokens (nodes), its blocks from b0 on.
  static __device__ __forceinline__ int head(const Item& it, int t) { return it.head + (G::kPair ? t : 0); }
  static __device__ __forceinline__ int offset(const RowsArgs& a, int t) { return G::kPair ? 0 : t * a.npt; }
  static __device__ __forceinline__ int count(const RowsArgs& a, const Item& it, int t) {
    if (G::kPair && it.head + t >= a.n_kv) return 0;
    return min(it.count - offset(a, t), a.npt);
  }
  static __device__ __forceinline__ int blocks(const RowsArgs& a, const Item& it, int t) {
    const int n = count(a, it, t);
    if (n <= 0) return 0;
    return G::kTree ? it.b1 - it.b0 : (it.pos0 + offset(a, t) + n + kBlock - 1) / kBlock;
  }
};

// Where a role stands in the ring.
template <int NS>
struct Ring {
  uint32_t at, phase;
  __device__ __forceinline__ void next() {
    if (++at == NS) {
      at = 0;
      phase ^= 1;
    }
  }
  template <int N>
  __device__ __forceinline__ void skip() {
#pragma unroll
    for (int i = 0; i < N; ++i) next();
  }
};

// The order of the ring's loads and their use, a block of K or V at a time (PD slots):
//   two tiles of one head  K0 V0 K1 V1 ...
//   one tile, two buffers  K0 K1 V0 K2 V1 ...
//   two heads a, b         K0a K0b V0a K1a V0b K1b ...
// Step s of the 2 n of an item's n blocks: whether V, and which block.
template <typename G>
__device__ __forceinline__ bool step_of(int s, int n, int& i) {
  const bool is_v = G::NB == 1 ? s & 1 : s > 0 && (!(s & 1) || s == 2 * n - 1);
  i = G::NB == 1 ? s / 2 : is_v ? (s == 2 * n - 1 ? n - 1 : s / 2 - 1) : (s + 1) / 2;
  return is_v;
}
template <typename G>
__global__ void __launch_bounds__(G::kThreads, 1)
rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ RowsArgs a) {
  constexpr int D = G::D, NT = G::NT, NB = G::NB, PD = G::PD, NS = G::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  if ((base & 1023u) != 0) {                               // the tiles' layout counts on it
    if (threadIdx.x == 0) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    return;
  }
  Tail<G>& tail = *reinterpret_cast<Tail<G>*>(smem_raw + G::kData);
  const uint32_t s_q = base, s_ring = base + NT * G::kQTile, s_bar = smem_u32(tail.bars);
  const uint32_t bar_full = s_bar, bar_empty = bar_full + 8 * NS, bar_clean = bar_empty + 8 * NS;
  const uint32_t bar_landed = bar_clean + 8 * NS;
  const uint32_t bar_qfull = bar_landed + 8 * NS, bar_qempty = bar_qfull + 8, bar_scores = bar_qempty + 8;
  const uint32_t bar_weights = bar_scores + 16, bar_sums = bar_weights + 32, bar_drained = bar_sums + 16;
  const uint32_t bar_product = bar_drained + 16, bar_item = bar_product + 8, bar_taken = bar_item + 8 * G::kItems;
  const uint32_t bar_ticket = bar_taken + 8 * G::kItems;
  volatile uint32_t* words = &tail.words[0][0];
  volatile int* first_bad = &tail.first_bad;
  volatile uint32_t* guard_slot = tail.guard_slot;
  volatile uint32_t* blocks = &tail.blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_full + 8 * s, G::kLoadWarps);
      mbar_init(bar_empty + 8 * s, 1);
      mbar_init(bar_clean + 8 * s, G::kScanWarps);
      mbar_init(bar_landed + 8 * s, G::kLoadWarps);
    }
    mbar_init(bar_qfull, 1);
    mbar_init(bar_qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_scores + 8 * i, 1);
      mbar_init(bar_weights + 16 * i, 4);
      mbar_init(bar_weights + 16 * i + 8, 4);
      mbar_init(bar_sums + 8 * i, 1);
      mbar_init(bar_drained + 8 * i, 4);
    }
    mbar_init(bar_product, 1);
    mbar_init(bar_ticket, 1);
    for (int i = 0; i < G::kItems; ++i) {
      mbar_init(bar_item + 8 * i, 1);
      mbar_init(bar_taken + 8 * i, G::kTakers);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *first_bad = INT32_MAX;
    *blocks = 0;
  }
  pdl_wait_then_release();                                 // TMEM is taken after it: an earlier kernel may still need its own
  if (warp == G::kMmaWarp) {
    tmem_alloc(smem_u32(&tail.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tail.tmem;
  Item it = {};
  bool ok = true;
  // The n-th item, as the planning warp found it; false behind the last one.  early: by a warp that may have nothing to
  // do in the items before it.
  constexpr std::true_type kEarly{};
  constexpr std::false_type kInTurn{};
  const auto read_item = [&](int n, Item& x, auto early) {
    const int at = n % G::kItems;
    if (!__all_sync(0xffffffffu, wait_item<G::kTree && early.value>(bar_item + 8 * at, (uint32_t)(n / G::kItems) & 1u, blocks))) return false;
    x = tail.items[at];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_taken + 8 * at);
    return true;
  };
  const auto take = [&](int n, auto early) {
    ok = read_item(n, it, early);
    return ok && it.req >= 0;
  };
  // Q of the item `it`, the n-th, by one thread.
  const auto load_q = [&](int n) {
    if (!wait_item<G::kTree>(bar_qempty, (n & 1) ^ 1, blocks)) return false;
    const bool two = it.nb1 > 0;
    const uint32_t bytes = (uint32_t)(a.npt * a.group * 128 * (D / 64));
    mbar_arrive_expect_tx(bar_qfull, two ? 2 * bytes : bytes);
#pragma unroll 1
    for (int t = 0; t < (two ? 2 : 1); ++t)
      for (int p = 0; p < D / 64; ++p)
        tma_load_3d(s_q + t * G::kQTile + p * G::kPanel, &tm_q, 64 * p, Walk<G>::head(it, t) * a.group,
                    it.row0 + Walk<G>::offset(a, t), bar_qfull);
    return true;
  };

  if (warp < G::kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSoftRegs));
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
  }
  if (warp < G::kSoftWarps) {
    // ---- softmax: a thread per row ----
    const int t = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int tok = (int)(row * a.group_inv >> 16), g = row - tok * a.group;
    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2);
    uint32_t use[2] = {0, 0}, items_t = 0, products = 0, blocks_done = 0;
    Item nxt;
    take(0, kInTurn);
    for (int n_item = 0; ok && it.req >= 0; ++n_item, it = nxt) {
      const int nb = t == 0 ? it.nb0 : it.nb1, nb_all = it.b1 - it.b0;
      if (nb == 0) {
        blocks_done += nb_all;
        ok = read_item(n_item + 1, nxt, kEarly);
        continue;
      }
      const int left = Walk<G>::count(a, it, t), row0 = it.row0 + Walk<G>::offset(a, t);
      const int pos0 = it.pos0 + Walk<G>::offset(a, t);    // left: tokens (nodes) of the tile
      const bool live = tok < left;
      const int pos = pos0 + min(tok, left - 1);
      uint64_t mask = 0;
      if (G::kTree) mask = a.mask[row0 + min(tok, left - 1)];
      int from = 0;                                        // prompt: the first token of the row's sequence
      if (G::kPack && it.len > 1) {
        const int32_t* bounds = a.few ? tail.bounds : a.bounds;
        int lo = it.req, hi = it.req + it.len;
#pragma unroll 1
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (bounds[mid] <= row0 - pos0 + pos) lo = mid;
          else hi = mid;
        }
        from = bounds[lo] - (row0 - pos0);
        __syncwarp();
      }
      float m = -INFINITY, l = 0.f;                        // m: of the scores as they come, before their scale
      for (int i = 0; i < nb; ++i) {
        const int x = NB == 1 ? t : (i & 1);
        const uint32_t scores = tmem + (uint32_t)(x * 128) + lane_off;
        if (!__all_sync(0xffffffffu, wait_for(bar_scores + 8 * x, use[x] & 1))) {
          ok = false;
          break;
        }
        ++use[x];
        tc_fence_after();
        // Blocks of which a row does not see every token: what it does not see becomes -infinity, in place, so that the
        // code of the other blocks serves them too.
        const int j0 = (it.b0 + i) * kBlock;
        bool some = !G::kTree && (it.b0 + i >= pos0 / kBlock || (G::kPack && it.len > 1));
        if (G::kTree) {
          bool all = j0 + kBlock <= it.base;
#pragma unroll
          for (int c = 0; c < 4; ++c) all = all && words[((blocks_done + i) % G::kWordsRing) * 4 + c] == 0xffffffffu;
          some = !all;
        }
        if (some) {                                        // the same for all lanes
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v, u[32];
            if (G::kTree) {
              const int d = j0 + 32 * c - it.base;
              v = words[((blocks_done + i) % G::kWordsRing) * 4 + c];
              if (d + 32 > 0) v &= d >= 64 ? 0u : d >= 0 ? (uint32_t)(mask >> d) : ((uint32_t)mask << -d) | ((1u << -d) - 1u);
            } else {
              v = prompt_sees(from - j0 - 32 * c, pos - j0 - 32 * c);
            }
            if (!__any_sync(0xffffffffu, v != 0xffffffffu)) continue;
            tmem_ld_32x32b_x32(scores + 32 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((v >> e) & 1)) u[e] = 0xff800000u;
            tmem_st_32x32b_x32(scores + 32 * c, u);
          }
          tmem_st_wait();
        }
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(scores + 32 * c, s[c]);
        tmem_ld_wait();
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 2) top[(c / 2) & 3] = max3(top[(c / 2) & 3], s[c / 32][c % 32], s[c / 32][c % 32 + 1]);
        const float bm = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool grow = (bm - m) * a.scale_log2 > kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? bm : m, c = grow ? ex2((m - mn) * a.scale_log2) : 1.f;
          l *= c;
          m = mn;
          if (i > 0) {
            if (NB == 2 && !__all_sync(0xffffffffu, wait_for(bar_product, (products + i - 1) & 1))) {
              ok = false;
              break;
            }
            const uint32_t sums = tmem + G::kTmemO + (uint32_t)(t * D) + lane_off;
            const uint64_t c2 = pack2(c, c);
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(sums + d, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint64_t y = mul2((uint64_t)o[e] | ((uint64_t)o[e + 1] << 32), c2);
                o[e] = (uint32_t)y;
                o[e + 1] = (uint32_t)(y >> 32);
              }
              tmem_st_32x32b_x32(sums + d, o);
            }
          }
        }
        if (__any_sync(0xffffffffu, far(m))) {
          const float less = far(m) ? -m : 0.f;
          const uint64_t less2 = pack2(less, less);
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t u[32];
            tmem_ld_32x32b_x32(scores + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const uint64_t y = add2((uint64_t)u[e] | ((uint64_t)u[e + 1] << 32), less2);
              u[e] = (uint32_t)y;
              u[e + 1] = (uint32_t)(y >> 32);
            }
            tmem_st_32x32b_x32(scores + c, u);
          }
          tmem_st_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(scores + 32 * c, s[c]);
          tmem_ld_wait();
        }
        const float shift = m == -INFINITY || far(m) ? -kShift : fmaf(-m, a.scale_log2, -kShift);
        const uint64_t shift2 = pack2(shift, shift);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int e = 64 * half + 2 * c;
            const uint64_t y = fma2((uint64_t)s[e / 32][e % 32] | ((uint64_t)s[e / 32][e % 32 + 1] << 32), scale2, shift2);
            const float p0 = ex2(lo2(y)), p1 = ex2(hi2(y));
            sum[c & 1] = add2(sum[c & 1], pack2(p0, p1));
            p[c] = pack_bf16(p0, p1);
          }
          tmem_st_32x32b_x32(scores + 32 * half, p);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_weights + 16 * x + 8 * half);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += lo2(sum[0]) + hi2(sum[0]);
      }
      if (!ok) break;
      products += nb;
      blocks_done += nb_all;
      // ---- the tile's outputs ----
      const bool part = G::kTree && it.slot >= 0;
      const int64_t orow = row0 + tok;
      const int kv = Walk<G>::head(it, t), head = kv * a.group + g;
      const int64_t prow = (int64_t)it.slot * a.slot_rows + t * (a.slot_rows / NT) + row;
      const float inv = 1.f / l;
      const uint32_t sums = tmem + G::kTmemO + (uint32_t)(t * D) + lane_off;
      // Of a finished tile four lanes exchange their 16-byte pieces, so that each store covers 64 bytes of eight
      // rows: with a row a lane a store touches 32 rows, half a sector each.  dst: this lane's place in its four rows.
      uint16_t* dst[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = (row & ~3) + e, tok_r = (int)(r * a.group_inv >> 16);
        dst[e] = tok_r < left ? a.out + (int64_t)(row0 + tok_r) * a.out_stride + (int64_t)(kv * a.group + r - tok_r * a.group) * D + 8 * (lane & 3)
                              : nullptr;
      }
      if (!read_item(n_item + 1, nxt, kInTurn) || !__all_sync(0xffffffffu, wait_for(bar_sums + 8 * t, items_t & 1))) {
        ok = false;
        break;
      }
      ++items_t;
      tc_fence_after();
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        __syncwarp();
        tmem_ld_32x32b_x32(sums + d, o);
        tmem_ld_wait();
        if (part) {
          if (!live) continue;
          uint4* to = reinterpret_cast<uint4*>(a.ws_acc + prow * D + d);
#pragma unroll
          for (int e = 0; e < 8; ++e) to[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else {
          uint4 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              u[f] = pack_bf16(__uint_as_float(o[8 * e + 2 * f]) * inv, __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
            v[e] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          transpose_4x4(v, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (dst[e]) *reinterpret_cast<uint4*>(dst[e] + d) = v[e];
        }
      }
      // A row without weight is 0, whatever weights of 0 made of V (33 short prompts 65.5 us; by selects on the way out 65.8).
      const bool none = live && !part && l == 0.f;
      if (__any_sync(0xffffffffu, none)) {
        __syncwarp();                                      // the row's pieces were stored by four lanes
#pragma unroll 1
        for (int d = 0; d < D && none; d += 8) *reinterpret_cast<uint4*>(a.out + orow * a.out_stride + (int64_t)head * D + d) = uint4{};
      }
      if (live && part) a.ws_ml[prow] = make_float2(m * a.scale_log2, l);
      if (live && !part && a.lse)
        a.lse[orow * a.n_heads + head] = l == 0.f ? -INFINITY : (fmaf(m, a.scale_log2, kShift) + log2f(l)) * 0.6931471805599453f;
      if (n_item >= *first_bad && it.guard < it.b1) {
        // Infinities and NaN of V in the blocks that not every row sees whole were left out of the products: the rows
        // that see them get them here.  Products with such blocks came after the scan of this item; an item without one
        // (of a tree cut before its nodes) has no words of its own, and nothing orders the scan's before it.
        __syncwarp();
        const int first = max(it.b0, it.guard);
        const volatile uint32_t* bad_words = &tail.bad[n_item % 8][0][0][0];
        const auto seen = [&](int c) {                     // of 32 tokens those with any that the row sees
          uint32_t v = bad_words[c];
          if (G::kScanWarps == 2) v |= bad_words[8 + c];
          const int j0 = first * kBlock + 32 * c;
          if (G::kTree) {
            const int d = j0 - it.base;
            if (d + 32 > 0) v &= d >= 64 ? 0u : d >= 0 ? (uint32_t)(mask >> d) : ((uint32_t)mask << -d) | ((1u << -d) - 1u);
          } else {
            v &= prompt_sees(from - j0, pos - j0);
          }
          return v;
        };
        uint32_t any = 0;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) any |= seen(c);
#pragma unroll 1
        for (int d = 0; d < D && live && any && l != 0.f; d += 8) {
          float c[8] = {};
#pragma unroll 1
          for (int at = 0; at < 8; ++at) {
#pragma unroll 1
            for (uint32_t v = seen(at); v; v &= v - 1) {
              const int j = first * kBlock + 32 * at + __ffs(v) - 1;
              const uint16_t* at_v;
              if (G::kTree) {
                const int2 pg = a.table[((int64_t)it.req * a.max_len + j) * a.layers + a.layer];
                if (pg.x < 0 || pg.x >= a.num_pages || pg.y < 0 || pg.y >= a.num_pages) continue;
                at_v = a.pool + (int64_t)pg.y * a.H + kv * D + d;
              } else {
                at_v = a.v + (row0 - pos0 + j) * a.v_stride + kv * D + d;
              }
              const uint4 x = *reinterpret_cast<const uint4*>(at_v);
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = non_finite2(u[e]);
                if (bad & 0x8000u) c[2 * e] += __uint_as_float(u[e] << 16);
                if (bad & 0x80000000u) c[2 * e + 1] += __uint_as_float(u[e] & 0xffff0000u);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (c[e] == 0.f) continue;
            if (part) {
              a.ws_acc[prow * D + d + e] += c[e];
            } else {
              uint16_t* y = a.out + orow * a.out_stride + (int64_t)head * D + d + e;
              *y = f32_to_bf16_rn(__uint_as_float((uint32_t)*y << 16) + c[e]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_drained + 8 * t);
    }
  } else if (warp == G::kMmaWarp) {
    // ---- products: one thread issues ----
    constexpr uint32_t kIdescS = make_idesc_bf16(kTileRows, kBlock);
    constexpr uint32_t kIdescO = make_idesc_bf16(kTileRows, G::DS) | (1u << 16);        // B (V) is MN-major
    uint32_t used = 0, items_t = 0, guarded = 0;           // bit x: phases of buffer x, tile x; V slots that were scanned so far
    Ring<NS> ring{0, 0};
    // Operands' descriptors: the low words move, the high ones (strides, version, swizzle) do not.
    const uint32_t lo_q = (uint32_t)sw128_kmajor_desc(s_q), lo_ring = (s_ring & 0x3FFFFu) >> 4;
    constexpr uint32_t kLdK = 1u << 16, kLdV = (G::kPanel >> 4) << 16;   // leading-dimension offsets
    const uint32_t kHiK = (uint32_t)(sw128_kmajor_desc(0) >> 32), kHiV = (uint32_t)(sw128_mnmajor_desc(0, G::kPanel, 1024) >> 32);
    const auto desc = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
    if (elect_one()) {
      // What is needed of an item is read while the one before it still runs.
      struct Mine {
        int n, guard, nb0, nb1;                            // blocks, the first guarded one; n < 0: behind the last item
      };
      const auto read = [&](int k, Mine& x) {
        const int at = k % G::kItems;
        if (!wait_for(bar_item + 8 * at, (uint32_t)(k / G::kItems) & 1u)) return false;
        const Item& y = tail.items[at];
        x = Mine{y.req < 0 ? -1 : y.b1 - y.b0, y.guard - y.b0, y.nb0, y.nb1};
        mbar_arrive(bar_taken + 8 * at);
        return true;
      };
      Mine cur, nxt;
      ok = read(0, cur);
      // Scores buffer x = Q_t K^T, K in the ring from r on.
      const auto issue_scores = [&](int t, int x, Ring<NS> r) {
#pragma unroll
        for (int p = 0; p < PD; ++p, r.next()) {
          if (!wait_for(bar_full + 8 * r.at, r.phase)) return false;
          tc_fence_after();
          const uint32_t qd = lo_q + (((uint32_t)t * G::kQTile + (uint32_t)p * G::PANELS * G::kPanel) >> 4);
          const uint32_t kd = (lo_ring | kLdK) + r.at * (G::kSlot >> 4);
#pragma unroll
          for (int k = 0; k < G::DS / 16; ++k) {
            const uint32_t off = ((k / 4) * G::kPanel + (k % 4) * 32) >> 4;
            mma_bf16_ss(tmem + x * 128, desc(qd + off, kHiK), desc(kd + off, kHiK), kIdescS, p > 0 || k > 0);
          }
        }
        mma_commit(bar_scores + 8 * x);
        return true;
      };
      // Sums of tile t += weights buffer x times V, V in the ring from r on.
      const auto issue_product = [&](int t, int x, Ring<NS> r, bool guard, bool add) {
#pragma unroll
        for (int p = 0; p < PD; ++p, r.next()) {
          const uint32_t n_th = guarded + p;               // of the V slots that are scanned: landed and cleared of infinities
          if (!(guard ? wait_for(bar_clean + 8 * (n_th % NS), (n_th / NS) & 1) : wait_for(bar_full + 8 * r.at, r.phase)))
            return false;
          const uint32_t vd = (lo_ring | kLdV) + r.at * (G::kSlot >> 4);
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k) {
            if (p == 0 && k % 4 == 0) {                    // half of the weights
              if (!wait_for(bar_weights + 16 * x + 2 * k, (used >> x) & 1)) return false;
              tc_fence_after();
            }
            mma_bf16_ts(tmem + G::kTmemO + t * D + p * G::DS, tmem + x * 128 + k * 8, desc(vd + ((k * 2048) >> 4), kHiV), kIdescO, add || k > 0);
          }
        }
        used ^= 1u << x;
        return true;
      };
      const auto release = [&](Ring<NS> r) {
#pragma unroll
        for (int p = 0; p < PD; ++p, r.next()) mma_commit(bar_empty + 8 * r.at);
      };
      constexpr bool kOwn = G::kPair || NB == 2;           // no two tiles share a block
      for (int n_item = 0; ok && cur.n >= 0; ++n_item, cur = nxt) {
        const int n = cur.n;
        ok = wait_for(bar_qfull, n_item & 1);
        tc_fence_after();
        // Scores are NB blocks ahead of the products.
#pragma unroll 1
        for (int i = -NB; i < n && ok; ++i) {
          const bool guard = i >= cur.guard;
          if (i + 1 == n) ok = read(n_item + 1, nxt);
          Ring<NS> next = ring;                            // where the scores' K lies
          if (i >= 0) next.template skip<PD>();
#pragma unroll 1
          for (int t = 0; t < NT && ok; ++t) {
            const int x = NB == 1 ? t : (i & 1);
            const int nb = t == 0 ? cur.nb0 : cur.nb1;
            if (i >= nb) continue;
            if (i >= 0) {
              if (i == 0) {
                ok = wait_for(bar_drained + 8 * t, ((items_t >> t) & 1) ^ 1);
                items_t ^= 1u << t;
              }
              ok = ok && issue_product(t, x, ring, guard, i > 0);
              if (!ok) continue;
              if (kOwn) {
                release(ring);
                ring.template skip<PD>();
                if (guard) guarded += PD;
              }
              if (NB == 2) mma_commit(bar_product);
              if (i + 1 == nb) mma_commit(bar_sums + 8 * t);
            }
            if (i + NB < nb) {
              ok = issue_scores(t, x, kOwn ? ring : next);
              if (ok && kOwn) {
                release(ring);
                ring.template skip<PD>();
              }
            }
          }
          if (!ok) break;
          if (!kOwn) {
            if (i >= 0) {
              release(ring);
              ring = next;
              if (guard) guarded += PD;
            }
            if (i + NB < n) {
              release(ring);
              ring.template skip<PD>();
            }
          }
          if (i + NB + 1 == n) mma_commit(bar_qempty);
          if (G::kTree) ++*blocks;
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  } else if (warp == G::kPlanWarp) {
    // ---- the items; of trees Q ----
    Walk<G> walk(a, tail.bounds, tail.units);
    walk.ticket = smem_u32(tail.ids);
    walk.bar_ticket = bar_ticket;
    if (G::kTree && lane == 0) a.ws_start[blockIdx.x] = make_int4(-1, 0, 0, 0);
    for (int n_item = 0; ok; ++n_item) {
      if (!G::kTree && a.tickets && n_item >= 2) {         // no earlier: it might run sooner elsewhere
        const int at = (n_item - 2) % G::kItems;
        ok = __all_sync(0xffffffffu, wait_for(bar_taken + 8 * at, (uint32_t)((n_item - 2) / G::kItems) & 1u));
        if (!ok) break;
      }
      const bool more = walk.next(a, it);
      if (!G::kTree && walk.failed) ok = false;
      if (!more) it.req = -1;
      it.nb0 = Walk<G>::blocks(a, it, 0);
      it.nb1 = NT == 2 ? Walk<G>::blocks(a, it, 1) : 0;
      if (elect_one()) {
        const int at = n_item % G::kItems;
        ok = wait_for(bar_taken + 8 * at, ((uint32_t)(n_item / G::kItems) & 1u) ^ 1u);
        if (ok) {
          tail.items[at] = it;
          mbar_arrive(bar_item + 8 * at);
        }
        if (G::kTree && more) {
          ok = ok && load_q(n_item);
          if (!ok && n_item > 0) (void)wait_for(bar_qfull, (n_item - 1) & 1);    // a copy may be in flight: the CTA may leave
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!more) break;
    }
  } else if (!G::kTree && warp == G::kLoadWarp) {
    // ---- prompt: TMA loads ----
    Ring<NS> ring{0, 1};                                   // phase: of the slot's release
    uint32_t guarded = 0;
    int issued = 0;
    for (int n_item = 0; ok && take(n_item, kInTurn); ++n_item) {
      if (elect_one()) {
        const auto load = [&](bool is_v, int i) {
          const CUtensorMap* map = is_v ? &tm_v : &tm_k;
#pragma unroll
          for (int p = 0; p < PD; ++p, ring.next(), ++issued) {
            ok = ok && wait_for(bar_empty + 8 * ring.at, ring.phase);
            if (!ok) return;
            uint32_t bar = bar_full + 8 * ring.at;
            if (is_v && it.b0 + i >= it.guard) {   // goes through the scan: the slot's own phase ends at once
              guard_slot[guarded % NS] = ring.at;
              mbar_arrive(bar);
              bar = bar_landed + 8 * (guarded++ % NS);
            }
            mbar_arrive_expect_tx(bar, G::kSlot);
            for (int c = 0; c < G::PANELS; ++c)
              tma_load_2d_plain(s_ring + ring.at * G::kSlot + c * G::kPanel, map, it.head * D + p * G::DS + 64 * c,
                                it.row0 - it.pos0 + (it.b0 + i) * kBlock, bar);
          }
        };
        const int n = it.b1 - it.b0;
#pragma unroll 1
        for (int s = 0; s < 2 * n && ok; ++s) {            // K0 may land while the item before still has its Q
          int i;
          const bool is_v = step_of<G>(s, n, i);
          load(is_v, i);
          if (s == 0) ok = ok && load_q(n_item);
        }
        if (!ok) {                                         // wait for the copies in flight: the CTA may leave
#pragma unroll 1
          for (int q = issued > NS ? issued - NS : 0; q < issued; ++q) (void)wait_for(bar_full + 8 * (q % NS), (uint32_t)(q / NS) & 1u);
#pragma unroll 1
          for (uint32_t c = guarded > NS ? guarded - NS : 0; c < guarded; ++c)
            (void)wait_for(bar_landed + 8 * (c % NS), (c / NS) & 1);
          if (n_item > 0) (void)wait_for(bar_qfull, (n_item - 1) & 1);
          (void)wait_for(bar_qfull, n_item & 1);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp >= G::kScanWarp && warp < G::kScanWarp + G::kScanWarps) {
    // ---- V blocks of which a row does not see every token are cleared of infinities and NaN, whose
    // products with the weights 0 would be NaN; the tile's outputs get those that a row does see ----
    const int w = warp - G::kScanWarp;
    uint32_t guarded = 0;
    for (int n_item = 0; ok && take(n_item, kEarly); ++n_item) {
      const int n = it.b1 - it.b0, tiles = G::kPair && it.nb1 > 0 ? 2 : 1;
      const int slots = (n - max(it.guard - it.b0, 0)) * PD * tiles;
      uint32_t* bad_words = &tail.bad[n_item % 8][w][0][0];
      __syncwarp();
      if (lane < 8) bad_words[lane] = 0;                   // eight items ago: its outputs are written
      __syncwarp();
#pragma unroll 1
      for (int k = 0; k < slots && ok; ++k) {
          ok = __all_sync(0xffffffffu, wait_item<G::kTree>(bar_landed + 8 * (guarded % NS), (guarded / NS) & 1, blocks));
          if (!ok) break;
          const uint32_t s = guard_slot[guarded % NS];
          const uint32_t off = w * (G::kSlot / G::kScanWarps), at = s_ring + s * G::kSlot + off + lane * 16;
          bool bad = false;
#pragma unroll 4
          for (uint32_t o = 0; o < G::kSlot / G::kScanWarps; o += 512) bad |= non_finite16(at + o);
          if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
            for (uint32_t o = 0; o < G::kSlot / G::kScanWarps; o += 512) {     // four tokens, 128 bytes of each
              const unsigned in = __ballot_sync(0xffffffffu, non_finite16(at + o));
              if (in == 0) continue;
              clean16(at + o);
              if (lane == 0) {
                const uint32_t token = (off + o) % G::kPanel / 128;
                bad_words[4 * (k / (PD * tiles)) + token / 32] |=
                    ((in & 0xffu ? 1u : 0u) | (in & 0xff00u ? 2u : 0u) | (in & 0xff0000u ? 4u : 0u) | (in & 0xff000000u ? 8u : 0u)) << (token % 32);
              }
            }
            if (lane == 0) atomicMin(const_cast<int*>(first_bad), n_item);
            __threadfence_block();
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_clean + 8 * (guarded % NS));
          ++guarded;
      }
    }
  } else if (G::kTree && warp >= G::kLoadWarp) {
    // ---- tree: rows of K and V from their pages, gathered four at a time by TMA, each warp 32 of a block's tokens ----
    const int w = warp - G::kLoadWarp;
    int32_t* ids = tail.ids[w];                            // K or V pages of a block; -1 (zeros): no data
    Ring<NS> ring{0, 1};                                   // phase: of the slot's release
    uint32_t guarded = 0;
    int blocks_done = 0, issued = 0;
    for (int n_item = 0; ok && take(n_item, kInTurn); ++n_item) {
      const int n = it.b1 - it.b0;
      const auto entry = [&](int i) {                      // this lane's token of block i
        const int j = (it.b0 + i) * kBlock + 32 * w + lane;
        return i < n && j < it.len ? a.table[((int64_t)it.req * a.max_len + j) * a.layers + a.layer] : make_int2(-1, -1);
      };
      const auto checked = [&](int2 e, int i) {
        if (e.x >= 0 && e.x < a.num_pages && e.y >= 0 && e.y < a.num_pages) return e;
        if (i < n && (it.b0 + i) * kBlock + 32 * w + lane < it.len) flag_error(a.err, LORA_DEV_BAD_PAGE);
        return make_int2(-1, -1);
      };
      const auto load = [&](int2 e, bool is_v, int i, int t) {
        __syncwarp();
        ids[lane] = is_v ? e.y : e.x;
        const unsigned has = __ballot_sync(0xffffffffu, e.x >= 0);
        __syncwarp();
#pragma unroll
        for (int p = 0; p < PD; ++p, ring.next()) {
          const uint32_t s = ring.at;
          ok = __all_sync(0xffffffffu, wait_for(bar_empty + 8 * s, ring.phase));
          if (!ok) return;
          const bool guard = is_v && it.b0 + i >= it.guard;
          if (elect_one()) {
            if (!is_v && p == 0 && t == 0) words[((blocks_done + i) % G::kWordsRing) * 4 + w] = has;
            uint32_t bar = bar_full + 8 * s;
            if (guard) {                                   // goes through the scan: the slot's own phase ends at once
              guard_slot[guarded % NS] = s;
              mbar_arrive(bar);
              bar = bar_landed + 8 * (guarded % NS);
            }
            mbar_arrive_expect_tx(bar, 32 * G::DS * 2);
            const uint32_t dst = s_ring + s * G::kSlot + w * 32 * 128;
            const int x = Walk<G>::head(it, t) * D + p * G::DS;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const int4 rows = *reinterpret_cast<const int4*>(ids + 4 * g);
#pragma unroll
              for (int c = 0; c < G::PANELS; ++c) tma_gather4(dst + c * G::kPanel + g * 512, &tm_k, x + 64 * c, rows, bar);
            }
          }
          guarded += guard;
          ++issued;
        }
      };
      int2 e0 = checked(entry(0), 0), e1 = entry(1);
      const int tiles = G::kPair && it.nb1 > 0 ? 2 : 1;
#pragma unroll 1
      for (int s = 0; s < 2 * n && ok; ++s) {
        int i;
        const bool is_v = step_of<G>(s, n, i);
        int2 e2 = e1;
        if (is_v) {                                        // entries are read two blocks ahead
          e2 = entry(i + 2);
          if (NB == 1) e1 = checked(e1, i + 1);
        } else if (NB == 2 && i > 0) {
          e1 = checked(e1, i);
        }
        if (!G::kPair) {
          load(is_v || i == 0 || NB == 1 ? e0 : e1, is_v, i, 0);
          if (is_v) {
            e0 = e1;
            e1 = e2;
          }
        } else if (s == 0) {
#pragma unroll 1
          for (int t = 0; t < tiles && ok; ++t) load(e0, false, 0, t);
        } else if (is_v) {                                 // V_i of a head, then its K of the next block
#pragma unroll 1
          for (int u = 0; u < 2 * tiles && ok; ++u)
            if (!(u & 1) || i + 1 < n) load(u & 1 ? e1 : e0, !(u & 1), i + (u & 1), u >> 1);
          e0 = e1;
          e1 = e2;
        }
      }
      blocks_done += n;
    }
    if (!ok && lane == 0) {                                // wait for the copies in flight: the CTA may leave
#pragma unroll 1
      for (int q = issued > NS ? issued - NS : 0; q < issued; ++q) (void)wait_for(bar_full + 8 * (q % NS), (uint32_t)(q / NS) & 1u);
#pragma unroll 1
      for (uint32_t c = guarded > NS ? guarded - NS : 0; c < guarded; ++c)
        (void)wait_for(bar_landed + 8 * (c % NS), (c / NS) & 1);
    }
  }
  if (!ok && lane == 0) flag_error(a.err, LORA_DEV_WAIT_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == G::kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---- joining a segment's partials ------------------------------------------------------------------
// Segments that lie in several parts: blocks (p, y) take the one that begins in part p and goes on behind it, a
// warp per row.  m = max m_i, l = sum l_i 2^(m_i - m), out = sum o_i 2^(m_i - m) / l, in the parts' order.
// A part far below the others has the factor 0 and its sums are multiplied by it all the same: an infinity or NaN of V there
// gives NaN, as it does within a part, wherever the request is cut.
// The latency of its loads bounds it: 16 blocks a part and four parts in flight took 131,072 tokens from 323 to 319 us, 8 blocks
// 321, 24 blocks 320 (and a small call from 10.5 to 11.6).
constexpr int kJoinWarps = 8, kJoinBlocks = 16, kJoinBatch = 4;     // warps of a block, blocks of a part, parts that a warp has in flight
template <typename G>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int D = G::D, E = D / 32;
  pdl_wait_then_release();
  const int p = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 rec = a.ws_start[p];                          // head, first row, nodes, last part
  if (rec.x < 0) return;
  const int rows = rec.z * a.group, heads = min(G::HT, a.n_kv - rec.x);
#pragma unroll 1
  for (int x = blockIdx.y * kJoinWarps + warp; x < rows * heads; x += gridDim.y * kJoinWarps) {
    const int h = x / rows, r = x - h * rows, node = r / a.group, g = r - node * a.group;
    const int t = G::kPair ? h : node / a.npt;
    const int64_t at = t * (a.slot_rows / G::NT) + (G::kPair ? node : node - t * a.npt) * a.group + g;
    const auto slot = [&](int i) { return (2 * (int64_t)i + (i == p ? 1 : 0)) * a.slot_rows + at; };
    float2 ml = make_float2(-INFINITY, 0.f);               // of 32 parts, a lane each
    if (p + lane <= rec.w) ml = a.ws_ml[slot(p + lane)];
    float m = ml.x;
#pragma unroll 1
    for (int i = p + 32 + lane; i <= rec.w; i += 32) m = fmaxf(m, a.ws_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int i0 = p; i0 <= rec.w; i0 += 32) {
      if (i0 > p) {
        ml = make_float2(-INFINITY, 0.f);
        if (i0 + lane <= rec.w) ml = a.ws_ml[slot(i0 + lane)];
      }
      const float c_own = ex2(ml.x - ms);
      const int n = min(32, rec.w - i0 + 1);
#pragma unroll 1
      for (int b0 = 0; b0 < n; b0 += kJoinBatch) {
        float c[kJoinBatch];
        float2 v[kJoinBatch][E / 2];
#pragma unroll
        for (int b = 0; b < kJoinBatch; ++b) {
          c[b] = __shfl_sync(0xffffffffu, c_own, b0 + b);  // 0 behind the last part
          l = fmaf(__shfl_sync(0xffffffffu, ml.y, b0 + b), c[b], l);
          const float2* src = reinterpret_cast<const float2*>(a.ws_acc + slot(i0 + b0 + b) * D + lane * E);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) v[b][e] = b0 + b < n ? src[e] : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int b = 0; b < kJoinBatch; ++b)
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            acc[2 * e] = fmaf(v[b][e].x, c[b], acc[2 * e]);
            acc[2 * e + 1] = fmaf(v[b][e].y, c[b], acc[2 * e + 1]);
          }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = rec.y + node;
    const int head = (rec.x + h) * a.group + g;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * a.out_stride + (int64_t)head * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = l == 0.f ? 0u : pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    if (a.lse && lane == 0) a.lse[row * a.n_heads + head] = l == 0.f ? -INFINITY : (m + kShift + log2f(l)) * 0.6931471805599453f;
  }
}

// ---- host side -------------------------------------------------------------------------------------
int check_heads(const std::string& fn, const lora_pool* p, int32_t n_req, int32_t n_heads, int32_t n_kv) {
  if (!p || n_req < 0 || n_heads < 1 || n_kv < 1) return lora_fail(LORA_EINVAL, fn + ": bad arguments");
  if (n_req > 65535) return lora_fail(LORA_EINVAL, fn + ": at most 65535 sequences per call");
  if (n_heads % n_kv != 0 || n_heads / n_kv > kRowsMaxGroup)
    return lora_fail(LORA_EINVAL, fn + ": n_heads must be 1 to 16 times n_kv_heads");
  if (p->H % n_kv != 0) return lora_fail(LORA_EINVAL, fn + ": H is not a multiple of n_kv_heads");
  const int D = p->H / n_kv;
  if (D != 64 && D != 128 && D != 256) return lora_fail(LORA_EINVAL, fn + ": head width must be 64, 128 or 256");
  return LORA_OK;
}

constexpr int64_t kMaxStride = (int64_t)1 << 32;    // elements between rows
int check_rows(const std::string& fn, std::initializer_list<std::pair<int64_t*, int64_t>> strides,
               std::initializer_list<const void*> rows) {
  for (const auto& s : strides) {
    if (*s.first == 0) *s.first = s.second;
    if (*s.first < s.second || *s.first > kMaxStride || (*s.first & 7) != 0)
      return lora_fail(LORA_EINVAL, fn + ": row strides must be multiples of 8, at least a row and at most 2^32");
  }
  for (const void* r : rows)
    if ((reinterpret_cast<uintptr_t>(r) & 15) != 0) return lora_fail(LORA_EINVAL, fn + ": q, k, v and out must be 16-byte aligned");
  return LORA_OK;
}

int check_workspace(const std::string& fn, const void* ws, int64_t bytes, int64_t need) {
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return lora_fail(LORA_EINVAL, fn + ": workspace must be 256-byte aligned");
  if (bytes < need)
    return lora_fail(LORA_EINVAL, fn + ": workspace has " + std::to_string(bytes) + " bytes, needs " + std::to_string(need));
  return LORA_OK;
}


int encode_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box) {
  auto fn = get_encode_fn();
  if (!fn) return lora_fail(LORA_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return lora_fail(LORA_ECUDA, "cuTensorMapEncodeTiled failed with code " + std::to_string((int)r));
  return LORA_OK;
}
// Query rows [row][head][feature]: a box is 64 features of one KV head's query heads of a tile's tokens.
int encode_q(CUtensorMap* map, const void* q, int D, int n_heads, int64_t n_rows, int64_t stride, int group, int npt) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)n_heads, (cuuint64_t)n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)npt};
  return encode_map(map, q, 3, dims, strides, box);
}
int encode_kv(CUtensorMap* map, const void* k, int H, int64_t n_rows, int64_t stride) {
  const cuuint64_t dims[2] = {(cuuint64_t)H, (cuuint64_t)n_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kBlock};
  return encode_map(map, k, 2, dims, strides, box);
}

// Pages of the pool, one row of 64 features a box: what TMA gathers.
int encode_pages(CUtensorMap* map, const void* pool, int H, int64_t num_pages) {
  const cuuint64_t dims[2] = {(cuuint64_t)H, (cuuint64_t)num_pages};
  const cuuint64_t strides[1] = {(cuuint64_t)H * 2};
  const cuuint32_t box[2] = {64, 1};
  return encode_map(map, pool, 2, dims, strides, box);
}

constexpr int64_t kKvInL2 = 96 << 20;
constexpr int64_t kShortRows = 1280 * 256;          // mean length times rows of an item
int tiles_of(int D) { return D == 256 ? 1 : 2; }

// Workspaces; every array starts on a 256-byte boundary.
struct PromptLayout {
  size_t bounds, n_items, items, seq_items, total;
  int32_t per_item, levels;
};
PromptLayout prompt_layout(int D, int32_t n_seq, int32_t n_rows, int32_t group) {
  PromptLayout L{};
  L.per_item = tiles_of(D) * (kTileRows / group);
  L.levels = (n_rows + L.per_item - 1) / L.per_item;
  size_t off = 0;
  L.bounds = off;   off = align256(off + ((size_t)n_seq + 1) * 4);
  L.n_items = off;  off = align256(off + 4);
  L.items = off;    off = align256(off + ((size_t)n_rows / L.per_item + n_seq) * sizeof(int2));
  L.seq_items = off; off = align256(off + (size_t)n_seq * 4);
  L.total = off;
  return L;
}
struct TreeLayout {
  size_t bounds, prefix, start, ml, acc, total;
  int32_t parts, slot_rows;
};
TreeLayout tree_layout(int D, int32_t n_req, int32_t group) {
  TreeLayout L{};
  L.parts = device_sm_count();
  const bool one = kTileRows / group >= LORA_MAX_TREE;     // a request's nodes fit a tile: two heads side by side
  L.slot_rows = one ? tiles_of(D) * LORA_MAX_TREE * group : tiles_of(D) * kTileRows;
  const size_t slots = 2 * (size_t)L.parts * L.slot_rows;
  size_t off = 0;
  L.bounds = off;  off = align256(off + ((size_t)n_req + 1) * 4);
  L.prefix = off;  off = align256(off + ((size_t)n_req + 1) * 8);
  L.start = off;   off = align256(off + (size_t)L.parts * sizeof(int4));
  L.ml = off;      off = align256(off + slots * sizeof(float2));
  L.acc = off;     off = align256(off + slots * D * 4);
  L.total = off;
  return L;
}

// The softmax warps take registers that the others give back: a kernel that was compiled to fewer than both hold would
// wait for them for ever.
template <typename G>
int check_registers(const char* what) {
  static const int regs = [] {
    cudaFuncAttributes attr{};
    return cudaFuncGetAttributes(&attr, rows_kernel<G>) == cudaSuccess ? attr.numRegs : 0;
  }();
  constexpr int kWarps = G::kThreads / 32, kNeed = G::kSoftWarps * G::kSoftRegs + (kWarps - G::kSoftWarps) * G::kOtherRegs;
  if (regs * kWarps < kNeed)
    return lora_fail(LORA_ECUDA, std::string(what) + ": the kernel has " + std::to_string(regs) + " registers a thread, its warps trade " +
                                     std::to_string((kNeed + kWarps - 1) / kWarps));
  return LORA_OK;
}

template <typename G>
int launch_rows(const lora_pool* p, const RowsArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                int ctas, const char* what, cudaStream_t st) {
  static DeviceFlags flags;
  int rc = ensure_smem_attr(flags, &rows_kernel<G>, (int)smem_bytes<G>(), what);
  if (rc == LORA_OK) rc = check_registers<G>(what);
  if (rc != LORA_OK) return rc;
  ProfScope prof(p, LORA_KIND_ATTENTION, st);
  const cudaError_t e = launch_pdl(!p->prof_on, rows_kernel<G>, dim3(ctas), dim3(G::kThreads), smem_bytes<G>(), st, q, k, v, a);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, what);
}

template <int D>
int launch_prompt_rows(const lora_pool* p, const RowsArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                       int ctas, const char* what, cudaStream_t st) {
  return a.pack ? launch_rows<Geo<D, false, false, true>>(p, a, q, k, v, ctas, what, st)
                : launch_rows<Geo<D, false>>(p, a, q, k, v, ctas, what, st);
}

int launch_prompt(const lora_pool* p, const RowsArgs& a, const PromptLayout& L, const CUtensorMap& q, const CUtensorMap& k,
                  const CUtensorMap& v, cudaStream_t st) {
  const char* what = "lora_attention_prompt launch";
  if (!a.few) {
    ProfScope prof(p, LORA_KIND_ATTENTION, st);
    const cudaError_t e = launch_pdl(!p->prof_on, prompt_plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)L.levels * 4, st, a,
                                     L.per_item, L.levels);
    if (e != cudaSuccess) return lora_cuda_fail(e, what);
  }
  const int64_t most = ((int64_t)a.n_rows / L.per_item + a.n_req) * a.n_kv;
  const int ctas = a.tickets ? a.tickets : (int)std::min<int64_t>(device_sm_count(), most);
  switch (p->H / a.n_kv) {
    case 64: return launch_prompt_rows<64>(p, a, q, k, v, ctas, what, st);
    case 128: return launch_prompt_rows<128>(p, a, q, k, v, ctas, what, st);
    default: return launch_prompt_rows<256>(p, a, q, k, v, ctas, what, st);
  }
}

template <typename G>
int launch_tree(const lora_pool* p, const RowsArgs& a, const CUtensorMap& q, const CUtensorMap& pages, cudaStream_t st) {
  const char* what = "lora_attention_tree launch";
  if (!a.few) {
    ProfScope prof(p, LORA_KIND_ATTENTION, st);
    const cudaError_t e = launch_pdl(!p->prof_on, tree_plan_kernel<G::RT>, dim3(1), dim3(kPlanThreads), 0, st, a);
    if (e != cudaSuccess) return lora_cuda_fail(e, what);
  }
  const int rc = launch_rows<G>(p, a, q, pages, pages, a.parts, what, st);
  if (rc != LORA_OK || a.max_len <= kBlock) return rc;     // a single block is never cut
  ProfScope prof(p, LORA_KIND_ATTENTION, st);
  const cudaError_t e = launch_pdl(!p->prof_on, tree_join_kernel<G>, dim3(a.parts, kJoinBlocks), dim3(32 * kJoinWarps), 0, st, a);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, what);
}

}  // namespace

extern "C" int64_t lora_attention_prompt_size(const lora_pool* p, int32_t n_seq, int32_t n_rows, int32_t n_heads,
                                              int32_t n_kv_heads) {
  const std::string fn = "lora_attention_prompt_size";
  const int rc = check_heads(fn, p, n_seq, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (n_rows < 0 || n_rows > LORA_MAX_TOKENS)
    return lora_fail(LORA_EINVAL, fn + ": n_rows must lie in [0, " + std::to_string(LORA_MAX_TOKENS) + "]");
  return (int64_t)prompt_layout(p->H / n_kv_heads, n_seq, n_rows, n_heads / n_kv_heads).total;
}

extern "C" int lora_attention_prompt(lora_pool* p, int32_t n_seq, const int32_t* seq_start, int32_t n_rows, const void* q,
                                     int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                     void* out, int64_t out_stride, int32_t n_heads, int32_t n_kv_heads, float* lse,
                                     void* workspace, int64_t workspace_bytes, lora_stream_t stream) {
  const std::string fn = "lora_attention_prompt";
  int rc = check_heads(fn, p, n_seq, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (n_rows < 0 || n_rows > LORA_MAX_TOKENS)
    return lora_fail(LORA_EINVAL, fn + ": n_rows must lie in [0, " + std::to_string(LORA_MAX_TOKENS) + "]");
  const bool some = n_seq > 0 && n_rows > 0;
  if (some && (!seq_start || !q || !k || !v || !out || !workspace)) return lora_fail(LORA_EINVAL, fn + ": null pointer");
  const int64_t width = (int64_t)n_heads * (p->H / n_kv_heads);
  rc = check_rows(fn, {{&q_stride, width}, {&out_stride, width}, {&k_stride, p->H}, {&v_stride, p->H}}, {q, k, v, out});
  if (rc != LORA_OK) return rc;
  if (some && (out == q || out == k || out == v)) return lora_fail(LORA_EINVAL, fn + ": out must not alias q, k or v");
  if (((reinterpret_cast<uintptr_t>(seq_start) | reinterpret_cast<uintptr_t>(lse)) & 3) != 0)
    return lora_fail(LORA_EINVAL, fn + ": starts and lse must be 4-byte aligned");
  const int D = p->H / n_kv_heads, group = n_heads / n_kv_heads;
  const PromptLayout L = prompt_layout(D, n_seq, n_rows, group);
  rc = check_workspace(fn, workspace, workspace_bytes, some ? (int64_t)L.total : 0);
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, fn + ": planning pool has no device state");
  if (!some) return LORA_OK;
  CUtensorMap tm_q, tm_k, tm_v;
  rc = encode_q(&tm_q, q, D, n_heads, n_rows, q_stride, group, kTileRows / group);
  if (rc == LORA_OK) rc = encode_kv(&tm_k, k, p->H, n_rows, k_stride);
  if (rc == LORA_OK) rc = encode_kv(&tm_v, v, p->H, n_rows, v_stride);
  if (rc != LORA_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  RowsArgs a{};
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.n_req = n_seq;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.n_kv = n_kv_heads;
  a.group = group;
  a.npt = kTileRows / group;
  a.group_inv = (65536 + group - 1) / group;
  a.start = seq_start;
  a.bounds = reinterpret_cast<int32_t*>(ws + L.bounds);
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)D);
  a.err = p->d_err;
  a.few = n_seq <= kFew;
  a.v = static_cast<const uint16_t*>(v);
  a.v_stride = v_stride;
  a.n_items = reinterpret_cast<int32_t*>(ws + L.n_items);
  a.items = reinterpret_cast<int2*>(ws + L.items);
  a.seq_items = reinterpret_cast<int32_t*>(ws + L.seq_items);
  // Sequences of two thirds of an item or less share items, unless each has an SM to itself: 127 prompts of 5 tokens, 8 KV
  // heads x 4 of 128 25.9 -> 11.5 us, 86 of 16, 16 heads of 256 45.1 -> 17.7; of 40 tokens of an item's 64 34.7 -> 34.9.
  // The code for it would cost longer ones 4 % (33 of 40 to 515 tokens 64.0 -> 66.7).
  a.pack = (int64_t)n_seq * n_kv_heads > device_sm_count() && n_rows / n_seq * 3 <= 2 * L.per_item;
  // A ticket per full item, the CTAs of the grid: those that run take the others' in turn, so that each has its share
  // by time.  Against a fixed share 0 to 10 % less (24,000 tokens of 32 heads of 128 in 4 prompts 324 -> 314 us).  Not
  // where the sequences are shorter than an item, of which a ticket would be several, nor for two rounds of items.
  const int64_t tickets = (int64_t)n_rows / L.per_item * n_kv_heads, kv_bytes = (int64_t)n_rows * p->H * 4;
  a.heads_at = n_kv_heads;
  if ((a.pack || n_rows / n_seq >= L.per_item) && tickets >= 2 * device_sm_count()) {
    a.tickets = (int32_t)tickets;
    // K and V beyond what L2 keeps, in sequences so short that reading them takes the time: about 48 MB of heads at a
    // time (30 prompts of 400 to 1,200 tokens, 32 heads of 128 242 -> 218 us, 16 of 256 306 -> 208; 7 of 1,700 tokens
    // 167 -> 170, which the rule leaves alone).
    if (kv_bytes > kKvInL2 && (int64_t)n_rows / n_seq * L.per_item < kShortRows)
      a.heads_at = (int)std::max<int64_t>(n_kv_heads / ((2 * kv_bytes + kKvInL2 - 1) / kKvInL2), 1);
  }
  return launch_prompt(p, a, L, tm_q, tm_k, tm_v, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int64_t lora_attention_tree_size(const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads,
                                            int32_t n_kv_heads) {
  const std::string fn = "lora_attention_tree_size";
  const int rc = check_heads(fn, p, n_req, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (max_len < 1 || max_len > (1 << 30)) return lora_fail(LORA_EINVAL, fn + ": max_len must lie in [1, 2^30]");
  if (p->planning) return lora_fail(LORA_EINVAL, fn + ": planning pool has no device state");
  return (int64_t)tree_layout(p->H / n_kv_heads, n_req, n_heads / n_kv_heads).total;
}

extern "C" int lora_attention_tree(lora_pool* p, int32_t n_req, const int32_t* table_dev, const int32_t* seq_len_dev,
                                   int32_t max_len, int32_t layers, int32_t layer, const int32_t* node_start,
                                   int32_t n_rows, const uint64_t* mask, const void* q, int64_t q_stride, void* out,
                                   int64_t out_stride, int32_t n_heads, int32_t n_kv_heads, float* lse, void* workspace,
                                   int64_t workspace_bytes, lora_stream_t stream) {
  const std::string fn = "lora_attention_tree";
  int rc = check_heads(fn, p, n_req, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (max_len < 1 || max_len > (1 << 30)) return lora_fail(LORA_EINVAL, fn + ": max_len must lie in [1, 2^30]");
  if (layers < 1 || layer < 0 || layer >= layers) return lora_fail(LORA_EINVAL, fn + ": layer outside [0, layers)");
  if (n_rows < 0) return lora_fail(LORA_EINVAL, fn + ": bad arguments");
  const bool some = n_req > 0 && n_rows > 0;
  if (some && (!table_dev || !seq_len_dev || !node_start || !mask || !q || !out || !workspace))
    return lora_fail(LORA_EINVAL, fn + ": null pointer");
  const int64_t width = (int64_t)n_heads * (p->H / n_kv_heads);
  rc = check_rows(fn, {{&q_stride, width}, {&out_stride, width}}, {q, out});
  if (rc != LORA_OK) return rc;
  if (some && out == q) return lora_fail(LORA_EINVAL, fn + ": out must not alias q");
  if (((reinterpret_cast<uintptr_t>(table_dev) | reinterpret_cast<uintptr_t>(mask)) & 7) != 0)
    return lora_fail(LORA_EINVAL, fn + ": table and mask must be 8-byte aligned");
  if (((reinterpret_cast<uintptr_t>(seq_len_dev) | reinterpret_cast<uintptr_t>(node_start) | reinterpret_cast<uintptr_t>(lse)) & 3) != 0)
    return lora_fail(LORA_EINVAL, fn + ": lengths, starts and lse must be 4-byte aligned");
  const int D = p->H / n_kv_heads, group = n_heads / n_kv_heads;
  const TreeLayout L = tree_layout(D, n_req, group);
  rc = check_workspace(fn, workspace, workspace_bytes, some ? (int64_t)L.total : 0);
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, fn + ": planning pool has no device state");
  if (!some) return LORA_OK;
  CUtensorMap tm_q, tm_pages;
  rc = encode_pages(&tm_pages, p->pool_dev, p->H, p->num_pages);
  if (rc == LORA_OK) rc = encode_q(&tm_q, q, D, n_heads, n_rows, q_stride, group, kTileRows / group);
  if (rc != LORA_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  RowsArgs a{};
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.n_req = n_req;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.n_kv = n_kv_heads;
  a.group = group;
  a.npt = kTileRows / group;
  a.group_inv = (65536 + group - 1) / group;
  a.start = node_start;
  a.bounds = reinterpret_cast<int32_t*>(ws + L.bounds);
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)D);
  a.err = p->d_err;
  a.pool = static_cast<const uint16_t*>(p->pool_dev);
  a.num_pages = p->num_pages;
  a.H = p->H;
  a.table = reinterpret_cast<const int2*>(table_dev);
  a.seq_len = seq_len_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.layer = layer;
  a.mask = mask;
  // units of all requests in 32 bits: at most 8 groups of tiles each
  a.few = n_req <= kFew && (int64_t)n_req * ((max_len + kBlock - 1) / kBlock + 1) * 8 <= INT32_MAX;
  a.prefix = reinterpret_cast<int64_t*>(ws + L.prefix);
  a.ws_start = reinterpret_cast<int4*>(ws + L.start);
  a.ws_ml = reinterpret_cast<float2*>(ws + L.ml);
  a.ws_acc = reinterpret_cast<float*>(ws + L.acc);
  a.parts = L.parts;
  a.slot_rows = L.slot_rows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool one = a.npt >= LORA_MAX_TREE;                 // as tree_layout
  switch (D) {
    case 64: return one ? launch_tree<Geo<64, true, true>>(p, a, tm_q, tm_pages, st) : launch_tree<Geo<64, true>>(p, a, tm_q, tm_pages, st);
    case 128: return one ? launch_tree<Geo<128, true, true>>(p, a, tm_q, tm_pages, st) : launch_tree<Geo<128, true>>(p, a, tm_q, tm_pages, st);
    default: return launch_tree<Geo<256, true>>(p, a, tm_q, tm_pages, st);
  }
}

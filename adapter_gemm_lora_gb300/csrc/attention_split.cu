// Paged decode attention split over the cache's length, with the tokens' attention weights.
//
// Per request and query head h (KV head h / G, G = n_heads / n_kv_heads, width D):
//     s_j = q_h . K_j / sqrt(D),  lse = log sum_j exp(s_j),  out_h = sum_j exp(s_j - lse) V_j
//     weight_out[j] = weight_in[j] + sum_h exp(s_{h,j} - lse_h)
// Softmax in base 2: scores carry log2(e) / sqrt(D).
//
// HBM-bound: every cached token's K and V rows (2 x 2 H bytes) are read once, against 4 H G flops.
// One GB300, a call: 256 requests of 128 to 2,048 tokens at H = 5120 826 us (7.1 TB/s, 1.06 of the copy
// rate: reads alone pass what a copy reaches), one request of 131,072 tokens at H = 4096 307 us (7.0
// TB/s), 64 requests with weights 179 us (0.94), 33 requests of up to 515 tokens 18.8 us (0.45: 3 us to
// the first data, 3 us of join).
//
// Split.  The tokens of all requests, in units of one ring stage (or one turn of the warps), form one sequence that is cut
// into P equal ranges; a CTA takes one range for one group of KV heads.  A request inside one range
// is finished there; one that spans ranges leaves a partial (m, l, sum exp2(s - m) V) per range,
// and the second kernel joins them: m = max m_i, l = sum l_i 2^(m_i - m), out likewise.  So the
// work per CTA does not depend on how the lengths are spread, and no result on who finishes first.
//
// Weights need the final lse, so the first kernel stores the scores (4 bytes per query head and
// token, against 4 D of K and V per KV head) and the second turns them into weights, each token's
// sum over the heads in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "tc_ptx.h"

namespace {

constexpr int kSplitMaxGroup = 16;                  // query heads per KV head
constexpr int kWarps = 4;                           // consumer warps
// A bulk copy costs its warp about 66 cycles to issue, whatever its size (with several producers on an
// SM still 33 each), so slices below 1 KB need two producer warps (one for K, one for V) to keep up:
// 160,000 tokens in 512-byte slices (four heads of 64) take 324 us with one and 214 us with two.  From
// 1 KB one is enough for a long request (316 us with one, 321 with two), but a request that one CTA
// takes whole waits for the issue: 61 tokens 7.8 us with one, 6.3 with two.
constexpr int kSmallSlice = 1024;
// Rows of up to 384 bytes have no producer: the consumer warps load K and V rows from their pages
// straight into MMA fragments, since a copy's cost does not fall with its size.  64 x 10,000 tokens,
// 1 query head per KV head, us by copies / direct: one head of 64 88 / 34.9 (one of 128 92 / 58.5),
// two of 64 93 / 58.9, three 107 / 94; but four 107 / 131, and at D = 128 two 106 / 106, four 196 / 204
// (eight heads of 64 197 / 311).  Short calls: 8 x 2,000 tokens of one head of 64 11.7 / 8.3.
constexpr int kDirectSlice = 384;
constexpr int64_t kTogetherBytes = 384 << 20;       // the cache's size, by max_len
constexpr int threads_of(int producers) { return 32 * (kWarps + producers); }
constexpr int kCtasPerSm = 2;
constexpr int kTile = 16;                           // tokens a warp takes at a time
constexpr int kTerms = 3;                           // bf16 terms of a weight in the V product
constexpr int kMaxTiles = 2;                        // 16-token tiles per stage, at most
constexpr int kStageBytes = 32 * 1024;              // K and V of a stage, at most
constexpr int kMaxStages = 8;
constexpr int kMaxSmem = (228 * 1024 / kCtasPerSm - 1024) & ~1023;   // a CTA's share, 1 KB of it reserved
constexpr int kStaticSmem = 1024;                   // barriers and stage records
constexpr int kFewWarps = 4, kManyWarps = 8;        // of a block of the join
constexpr int kJoinMany = 32;                       // partials per request from which a join is spread wider
constexpr int kWarpHeads = 8;                       // up to so many heads a warp adds its tokens' weights alone
constexpr int kJoinUnit = 64;                       // tokens whose weights a block takes at a time

// How a call is cut: fixed by the shapes, the same for the size query and the launch.
struct SplitPlan {
  int32_t D, group, n_kv;
  int32_t n_groups, heads;       // groups of KV heads, KV heads per group
  int32_t octets;                // warps per head by its query heads, 8 each
  int32_t head_slots;            // heads taken side by side: one a slot, or two (D = 64)
  int32_t sharers;               // warps that share a head's tokens
  int32_t tile_sharers;          // of them, those that take a stage's tiles in turn; the rest take turns at stages
  int32_t tiles;                 // 16-token tiles per stage
  int32_t stages;
  int32_t parts;                 // ranges the token sequence is cut into
  bool whole;                    // one range per request: nothing to join
  bool direct;                   // the consumers read the rows themselves
  bool pair, meet;               // direct: a warp has both KV heads of 64; the heads' warps wait for one another
  int32_t row_bytes, stage_bytes, smem;
};

struct SplitArgs {
  const uint16_t* pool;
  int64_t num_pages;
  int32_t H, n_req;
  const int32_t* table;
  const int32_t* seq_len;
  int32_t max_len, layers, layer;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  int32_t n_heads;
  float* lse;                          // caller's, nullable, natural log
  const float* weight_in;
  float* weight_out;
  int64_t weight_stride;
  float scale_log2;
  SplitPlan plan;
  float* ws_lse;                       // [n_req][n_heads], base 2: requests inside one range
  int2* ws_range;                      // [n_req] first and last range of a request
  int4* ws_start;                      // [parts] a range's first request, its token there, that request's ranges
  float2* ws_ml;                       // [2 parts][n_heads] m and l of a partial
  float* ws_acc;                       // [2 parts][n_heads][D]
  float* ws_scores;                    // [n_req][n_heads][score_stride], base 2; NULL without weights
  int64_t score_stride;
  int32_t* err;
};

// A range leaves at most two partials: slot 2 p for a request that began in an earlier range,
// slot 2 p + 1 for one that begins here and goes on.
__device__ __forceinline__ int64_t partial_slot(int p, bool starts) { return 2 * (int64_t)p + (starts ? 1 : 0); }

__device__ __forceinline__ int request_length(const SplitArgs& a, int r) {
  const int n = a.seq_len[r];
  return n < 0 ? 0 : n > a.max_len ? a.max_len : n;
}

__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A tile's V products are summed from zero, the smallest term first, and then added in fp32: MMAs cut
// their sums instead of rounding them, and the cuts of an accumulator that runs through a long request add
// up.  Outputs that are not the exact ones' rounding, one request of 131,072 tokens 0.7 % -> 0.02 % (0.3 %
// with fp32 products and sums), 256 of 128 to 2,048 0.2 % -> 0.02 %.  At most 4 % slower (16 query heads on
// 8 KV heads of 64, 64 x 10,000 tokens 254 -> 264 us), one KV head of 64, 64 x 40,000 tokens 141 -> 123.
constexpr int kBlocks = 4;                          // of 16 features, summed beside one another
__device__ __forceinline__ void add_tile(float (&acc)[4], const float (&sum)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] += sum[e];
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {        // toward zero
  uint32_t y;
  asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two weights as bf16 terms, without loss: each term but the last is the largest bf16 strictly below what
// is left, so 24 bits are used up in three, and no term of a weight above 2^-100 is zero or negative.  The
// terms' products with an infinite V are then that infinity, where a zero or negative term would add NaN.
// Two rounded terms hold 16 bits, which shows where V's terms cancel.  The third makes four MMAs of three:
// nothing where HBM bounds (256 x 128 to 2,048 tokens, H = 5120 831 / 834 us), most with 16 query heads on
// 8 KV heads of 64 (64 x 10,000 tokens 237 / 250 us).
__device__ __forceinline__ void weight_terms(float p0, float p1, uint32_t (&term)[kTerms]) {
  constexpr float kBelow = 1.f - 1.f / (1 << 24);          // x kBelow: the next smaller fp32
#pragma unroll
  for (int k = 0; k + 1 < kTerms; ++k) {
    term[k] = pack_bf16_down(p0 * kBelow, p1 * kBelow);
    p0 -= bf16_lo(term[k]);
    p1 -= bf16_hi(term[k]);
  }
  term[kTerms - 1] = pack_bf16(p0, p1);
}

// What turns the sum of weights x V into their mean; 0 for a row without weight.
__device__ __forceinline__ float normalizer(float l) { return l == 0.f ? 0.f : 1.f / l; }

enum : int32_t { kFirst = 1, kLast = 2, kStarts = 4, kEnds = 8 };

// One stage's tokens: which request, where, and which of them have data.
struct StageInfo {
  int32_t req, tok, n, flags;
  int32_t next;                  // on a request's last stage here: the request that follows, or -1
  uint16_t mask[kMaxTiles];      // per tile: bit i = token i has data
};

// Where a range begins in the sequence of all requests' units, and of its first request the length
// and the first and last range.
struct RangeStart {
  int32_t req, tok, units, n, p0, p1;
};

// Prefix sum over the warp's lanes.
__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The range [p U / P, (p + 1) U / P) of the U units of all requests (one unit: `st` tokens), with
// P = min(parts, U).  Up to 128 requests every warp finds it alone, four requests a lane; beyond, the
// block's warps sum the units of 128 requests at a time into `sums`, and every warp searches those.
// Units fit in 32 bits (checked by the host).
__device__ RangeStart find_range(const SplitArgs& a, int p, int parts, int st, int32_t* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_sums = (a.n_req + 127) / 128;
  int len[4], units[4], mine = 0, total = 0;               // requests 128 t + 4 lane ..
  const auto look = [&](int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 128 * t + 4 * lane + i;
      const int n = r < a.n_req ? a.seq_len[r] : 0;
      if (n < 0 || n > a.max_len) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
      len[i] = n < 0 ? 0 : n > a.max_len ? a.max_len : n;
    }
    mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      units[i] = (int)(((unsigned)len[i] + (unsigned)st - 1) / (unsigned)st);
      mine += units[i];
    }
  };
  if (n_sums == 1) {
    look(0);
    total = __reduce_add_sync(0xffffffffu, mine);
  } else {
    for (int t = warp; t < n_sums; t += blockDim.x >> 5) {
      look(t);
      const int u = __reduce_add_sync(0xffffffffu, mine);
      if (lane == 0) sums[t] = u;
    }
    __syncthreads();
    for (int t = lane; t < n_sums; t += 32) total += sums[t];
    total = __reduce_add_sync(0xffffffffu, total);
  }
  // No range between two used ones is empty (the join reads a partial of each): P = min(P, U).
  const int P = max(min(parts, total), 1);
  const int q0 = min(p, P), q1 = min(p + 1, P);
  const int u0 = (int)((long long)q0 * total / P), u1 = (int)((long long)q1 * total / P);
  if (u1 == u0) return RangeStart{0, 0, 0, 0, 0, 0};
  int before = 0, t = 0;                                   // units of the requests looked at so far
  if (n_sums > 1) {
    for (int t0 = 0; t0 < n_sums; t0 += 32) {              // the block of 128 requests that holds u0
      const int s = t0 + lane < n_sums ? sums[t0 + lane] : 0;
      const int incl = warp_inclusive(s, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > u0);
      if (hit) {
        const int k = __ffs(hit) - 1;
        t = t0 + k;
        before += __shfl_sync(0xffffffffu, incl - s, k);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    look(t);
  }
  const int incl = warp_inclusive(mine, lane);
  const int k = __ffs(__ballot_sync(0xffffffffu, before + incl > u0)) - 1;      // the lane, then its request
  before += __shfl_sync(0xffffffffu, incl - mine, k);
  RangeStart rs{128 * t + 4 * k, 0, u1 - u0, 0, 0, 0};
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = __shfl_sync(0xffffffffu, units[i], k), n = __shfl_sync(0xffffffffu, len[i], k);
    if (!found && before + u > u0) {
      rs.req += i;
      rs.tok = (u0 - before) * st;
      rs.n = n;
      // the range that holds unit x is the largest i with i U / P <= x, i.e. i U < (x + 1) P
      rs.p0 = (int)((((long long)before + 1) * P - 1) / total);
      rs.p1 = (int)((((long long)before + u) * P - 1) / total);
      found = true;
    }
    before += u;
  }
  return rs;
}

// Walks a range one unit at a time.
struct UnitWalk {
  int32_t req, tok, n, left;
  bool first;
};
__device__ __forceinline__ void walk_begin(const SplitArgs& a, UnitWalk& w) {   // skip to a request with tokens
  while (w.left > 0 && w.tok >= w.n) {
    ++w.req;
    w.tok = 0;
    w.n = request_length(a, w.req);
  }
}

// One CTA per (group of KV heads, range).  NP producer warps fill a ring of stages: per stage and
// token the group's slice of the K row and of the V row (heads x D contiguous bf16) by
// cp.async.bulk, all against the stage's one mbarrier; page ids are read one stage ahead.  A
// consumer warp owns up to 8 query heads of one KV head, or of two of 64, and the stages' 16-token
// tiles, shared out between the warps of the head where there are several.
//
// Per tile the products run on m16n8k16 MMAs with the tokens (or the features) as the 16 rows and
// the warp's query heads as the 8 columns: S^T = K q^T, then acc^T += V^T P^T.  A decode
// step has at most 16 query rows per KV head, far below the 64 or 128 rows of a tcgen05 tile, and
// every K and V byte is used once, so the tensor work is small; this layout leaves 1/8 instead of
// 1/16 of the MMA in use at one query head, and the running maximum, sum and rescaling of a column
// stay in the lanes that hold the column in both products.  P^T is the transpose of S^T's
// fragment (movmatrix) as three bf16 terms, so the weights reach the product with all their fp32 bits.
// Direct (NP = 0): no ring and no producer.  A lane loads 16 bytes (8 features) of its token's row at a
// time, and the products take the features in that order: K's registers are the first product's
// fragments as they come (q is read in the same order), V's are transposed (movmatrix) into the
// second's.  Page ids are two tiles ahead of the products and rows one, so a warp has 8 KB on its way;
// with half of that (one tile of 64 features) one KV head of 64 took 41 us instead of 34.9.
// A tile's K and V fragments are all in registers before its softmax starts (at D = 256 the second
// half of V follows it), and the stage is given back then: the chain of a tile (products, shuffles,
// exponentials) holds up no copy.
// Four consumer warps and two CTAs per SM, three stages of 32 KB each: one CTA of eight warps and
// 64 KB stages measured the same.  The producer is what has to be lean, since one warp prepares every
// copy: with a loop over up to eight tiles, seven of them unused, the batch above took 1,203 us, with
// the tile count fixed at compile time 840 us; without the consumers' arithmetic 826 us.
// More than 8 query heads per KV head take two warps a head, each with 8 of them and its own read of
// the head's K and V from shared memory: 4 x 40,000 tokens with 16 query heads per KV head take, join
// included, 116 us at D = 128 and 115 at 256 at H = 1024 (0.84 of the copy rate; 8 query heads 106 us), and
// 221 and 208 us at H = 2048, where one warp with two column tiles, whose accumulators spilled, took 260
// and 437.
template <int D, int TILES, int NP, int HW>
__global__ void __launch_bounds__(threads_of(NP), kCtasPerSm) attention_split_kernel(const __grid_constant__ SplitArgs a) {
  constexpr int KS = D / 16;
  constexpr int VR = KS < 8 ? KS : 8;                      // V fragments held over the softmax
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * kWarps];
  __shared__ StageInfo info[kMaxStages];
  const SplitPlan& pl = a.plan;
  const int tile_sharers = pl.tile_sharers;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g0 = blockIdx.x % pl.n_groups, p = blockIdx.x / pl.n_groups;
  const int h0 = g0 * pl.heads, n_act = min(pl.heads, pl.n_kv - h0);
  constexpr bool kDirect = NP == 0;
  constexpr bool kPair = kDirect && HW * TILES * D < 256 && HW == 2;   // direct, two KV heads of 64 a warp
  const int st = kDirect ? kTile * pl.tiles : kTile * TILES;
  const int S = pl.stages;
  const uint32_t ring = smem_u32(smem), RB = pl.row_bytes;
  const uint32_t bar_full = smem_u32(bars), bar_empty = bar_full + 8 * kMaxStages;
  const uint32_t bar_ready = bar_empty + 8 * kMaxStages, bar_done = bar_ready + 8 * kWarps;
  float* merge = reinterpret_cast<float*>(smem + (size_t)S * pl.stage_bytes);   // [head warps][8][D + 2]
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full + 8 * s, NP > 0 ? NP : 1);
      mbar_init(bar_empty + 8 * s, min(pl.head_slots, n_act) * pl.octets * pl.sharers);
    }
    for (int h = 0; h < kWarps; ++h) {
      mbar_init(bar_ready + 8 * h, 1);
      mbar_init(bar_done + 8 * h, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait_then_release();
  RangeStart rs{};
  if (pl.whole) {
    const int n = a.seq_len[p];
    if (threadIdx.x == 0 && (n < 0 || n > a.max_len)) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    rs.req = p;
    rs.tok = 0;
    rs.n = n < 0 ? 0 : min(n, a.max_len);
    rs.units = (int32_t)(((unsigned)rs.n + st - 1) / st);
  } else {
    rs = find_range(a, p, pl.parts, st, reinterpret_cast<int32_t*>(merge));
  }
  __syncthreads();                                         // barriers set up; the sums lie where heads merge
  if (g0 == 0 && threadIdx.x == 0) a.ws_start[p] = make_int4(rs.req, rs.units > 0 ? rs.tok : 0, rs.p0, rs.p1);

  const auto zero_empty = [&] {                            // requests without a token get zeros
    for (int r = p; r < a.n_req; r += pl.parts) {
      if (a.seq_len[r] > 0) continue;
      uint16_t* row = a.out + r * a.out_stride + (int64_t)h0 * pl.group * D;
      for (int i = lane; i < n_act * pl.group * D / 8; i += 32) reinterpret_cast<uint4*>(row)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int i = lane; i < n_act * pl.group; i += 32) a.lse[(int64_t)r * a.n_heads + h0 * pl.group + i] = -INFINITY;
    }
  };
  if (kDirect) {
    if (warp == kWarps - 1) zero_empty();
  } else if (warp >= kWarps) {
    // ---- producers: each finds every unit's valid tokens; with two, one copies K and one V ----
    const int role = warp - kWarps;
    const uint32_t bytes = (uint32_t)n_act * D * 2;
    const int half = lane >> 4, ti = lane & 15;            // lanes 0..15: K pages, 16..31: V pages
    const uint32_t dst0 = ring + (uint32_t)(half * TILES * kTile + ti) * RB;
    const uint16_t* rows = a.pool + h0 * D;
    const int64_t unit_step = (int64_t)st * a.layers * 2;
    UnitWalk w{rs.req, rs.tok, rs.n, rs.units, true};
    const auto entry = [&](const UnitWalk& u) {            // this lane's table entry of a unit's first tile
      return a.table + ((((int64_t)u.req * a.max_len + u.tok + ti) * a.layers) + a.layer) * 2 + half;
    };
    const int32_t* tab = entry(w);
    int32_t ids[TILES];
    const auto fetch = [&](const UnitWalk& u) {
#pragma unroll
      for (int c = 0; c < TILES; ++c)
        ids[c] = u.tok + kTile * c + ti < u.n ? tab[(int64_t)c * kTile * a.layers * 2] : -1;
    };
    if (w.left > 0) fetch(w);
    bool ok = true;
    int it = 0, s = 0;
    uint32_t phase = 1;                                    // of the ring's first round: nothing to wait for
    while (w.left > 0) {
      const UnitWalk cur = w;
      int32_t page[TILES];
#pragma unroll
      for (int c = 0; c < TILES; ++c) page[c] = ids[c];
      // the next unit, and its page ids while this one waits for its stage
      w.tok += st;
      --w.left;
      tab += unit_step;
      const bool ends = w.tok >= w.n;
      const bool last = ends || w.left == 0;
      w.first = ends;
      if (w.left > 0) {
        if (ends) {
          walk_begin(a, w);
          tab = entry(w);
        }
        fetch(w);
      }
      uint32_t mask[TILES];
      int n_valid = 0;
#pragma unroll
      for (int c = 0; c < TILES; ++c) {
        const bool good = page[c] >= 0 && page[c] < a.num_pages;
        const uint32_t b = __ballot_sync(0xffffffffu, good);
        mask[c] = b & (b >> 16) & 0xFFFFu;
        n_valid += __popc(mask[c]);
        if (!good && cur.tok + kTile * c + ti < cur.n) flag_error(a.err, LORA_DEV_BAD_PAGE);   // token skipped
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar_empty + 8 * s, phase));
      if (!ok) break;
      if (lane == 0) {
        if (role == 0) {
          StageInfo& f = info[s];
          f.req = cur.req;
          f.tok = cur.tok;
          f.n = cur.n;
          const int begun = cur.req == rs.req ? rs.tok : 0;  // the segment's first token
          f.flags = (cur.first ? kFirst : 0) | (last ? kLast : 0) | (begun == 0 ? kStarts : 0) | (ends ? kEnds : 0);
          f.next = w.left > 0 ? w.req : -1;
#pragma unroll
          for (int c = 0; c < TILES; ++c) f.mask[c] = (uint16_t)mask[c];
        }
        mbar_arrive_expect_tx(bar_full + 8 * s, 2 / (NP > 0 ? NP : 1) * bytes * n_valid);
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < TILES; ++c)
        if (((mask[c] >> ti) & 1u) && (NP == 1 || half == role))
          bulk_g2s(dst0 + (uint32_t)s * pl.stage_bytes + (uint32_t)(c * kTile) * RB, rows + (int64_t)page[c] * a.H, bytes,
                   bar_full + 8 * s);
      ++it;
      if (++s == S) {
        s = 0;
        phase ^= 1;
      }
    }
    if (!ok) {
      if (lane == 0) flag_error(a.err, LORA_DEV_WAIT_TIMEOUT);
      // the copies already issued land before this CTA's shared memory is released
      for (int c = it > S ? it - S : 0; c < it; ++c) (void)mbar_wait(bar_full + 8 * (c % S), (c / S) & 1);
    }
    if (role == 0) zero_empty();
    return;
  }

  // ---- consumers ----
  const int head_warps = pl.head_slots * pl.octets, hw = warp % head_warps, share = warp / head_warps;
  const int hh = hw / pl.octets, octet = hw % pl.octets;
  if (share >= pl.sharers || hh >= n_act || rs.units == 0) return;
  // HW = 2: two KV heads, hh and hh + head_slots, or (direct, not kPair) one with up to 16 query heads.
  const int n_mine = kDirect ? HW : HW == 1 || hh + pl.head_slots >= n_act ? 1 : 2;
  const int g = lane >> 2, t = lane & 3;
  const auto n_query = [&](int u) { return min(8, pl.group - 8 * (kDirect && !kPair ? octet + u : octet)); };
  const auto head_of = [&](int u) {
    return kDirect && !kPair ? (h0 + hh) * pl.group + 8 * (octet + u) : (h0 + hh + u * pl.head_slots) * pl.group + 8 * octet;
  };
  uint32_t qf[HW][KS][2];
  float acc[HW][KS][4], m[HW][2], l[HW][2];
  // The features that a lane holds: of a fragment's row g (+ 8 where hi), and of columns 2t and 2t + 1.
  const auto row_of = [&](int ks, int hi) {
    return kDirect ? 32 * (ks / 2) + 8 * (g / 2) + (g & 1) + 4 * (ks & 1) + 2 * hi : 16 * ks + g + 8 * hi;
  };
  const auto pair_of = [&](int ks, int hi) {
    return kDirect ? 32 * (ks / 2) + 8 * t + 4 * (ks & 1) + 2 * hi : 16 * ks + 2 * t + 8 * hi;
  };
  const auto load_q = [&](int req) {
#pragma unroll
    for (int u = 0; u < HW; ++u) {
      const bool has = u < n_mine && g < n_query(u);
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q + req * a.q_stride + (int64_t)(head_of(u) + g) * D);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[u][ks][0] = has ? qp[pair_of(ks, 0) / 2] : 0u;
        qf[u][ks][1] = has ? qp[pair_of(ks, 1) / 2] : 0u;
      }
    }
  };
  const auto begin_segment = [&] {
#pragma unroll
    for (int u = 0; u < HW; ++u) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) acc[u][ks][0] = acc[u][ks][1] = acc[u][ks][2] = acc[u][ks][3] = 0.f;
      m[u][0] = m[u][1] = -INFINITY;
      l[u][0] = l[u][1] = 0.f;
    }
  };
  // lane addresses of the fragments within a tile
  const uint32_t k_lane = (uint32_t)(lane & 15) * RB + (uint32_t)(hh * D + (lane >> 4) * 8) * 2;
  const uint32_t v_lane = (uint32_t)(TILES * kTile + (lane & 7) + (lane >> 4) * 8) * RB +
                          (uint32_t)(hh * D + ((lane >> 3) & 1) * 8) * 2;
  const uint32_t head_step = (uint32_t)(pl.head_slots * D * 2);
  const int turns = pl.sharers / tile_sharers, turn = share / tile_sharers;
  // Scores of NT tiles into weights 2^(s - m), transposed for the V product, in terms.
  constexpr int NT = kDirect ? TILES : 1;
  const auto tile_weights = [&](int u, int req, int j0, int n, uint32_t mask, float (&sc)[NT][4],
                                const float (&odd)[NT][4], uint32_t (&pt)[NT][kTerms][2]) {
    const int G = n_query(u);
    float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sc[i][e] = (mask >> (16 * i + g + (e & 2) * 4)) & 1u ? (sc[i][e] + odd[i][e]) * a.scale_log2 : -INFINITY;
      if (a.ws_scores && (i == 0 || j0 + i * kTile < n)) {
        float* dst = a.ws_scores + ((int64_t)req * a.n_heads + head_of(u) + 2 * t) * a.score_stride + j0 + i * kTile + g;
        if (2 * t < G) {
          dst[0] = sc[i][0];
          dst[8] = sc[i][2];
        }
        if (2 * t + 1 < G) {
          dst[a.score_stride] = sc[i][1];
          dst[a.score_stride + 8] = sc[i][3];
        }
      }
      x[0] = fmaxf(x[0], fmaxf(sc[i][0], sc[i][2]));
      x[1] = fmaxf(x[1], fmaxf(sc[i][1], sc[i][3]));
    }
    // A vote first: the maximum's shuffles and the rescaling follow only where a score passes it.  No weight
    // is above 1: a maximum that lags by up to 2^8 saves 4 % with 16 query heads on 8 KV heads of 64 (64 x
    // 10,000 tokens 260 -> 249 us), costs 13 % at three (64 x 40,000 tokens 371 -> 426) and lets sums
    // overflow for V above 2^119.
    if (__any_sync(0xffffffffu, x[0] > m[u][0] || x[1] > m[u][1])) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) x[k] = fmaxf(x[k], __shfl_xor_sync(0xffffffffu, x[k], o));
      float c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mn = fmaxf(m[u][k], x[k]);
        c[k] = mn == -INFINITY ? 0.f : exp2f(m[u][k] - mn);   // no score above -infinity yet: nothing to keep
        l[u][k] *= c[k];
        m[u][k] = mn;
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        acc[u][ks][0] *= c[0];
        acc[u][ks][1] *= c[1];
        acc[u][ks][2] *= c[0];
        acc[u][ks][3] *= c[1];
      }
    }
    const float ms[2] = {m[u][0] == -INFINITY ? 0.f : m[u][0], m[u][1] == -INFINITY ? 0.f : m[u][1]};   // every weight 0 there
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sc[i][k] = exp2f(sc[i][k] - ms[k]);
        sc[i][2 + k] = exp2f(sc[i][2 + k] - ms[k]);
        l[u][k] += sc[i][k] + sc[i][2 + k];
      }
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        uint32_t term[kTerms];
        weight_terms(sc[i][2 * hi], sc[i][2 * hi + 1], term);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) pt[i][k][hi] = transpose_8x8(term[k]);
      }
    }
  };
  int seg = 0;                                             // segments finished: the phase of the merge barriers
  load_q(rs.req);                                          // on its way beside the first stages
  bool broken = false;                                     // a wait ran out
  int next_s = 0, next_turn = 0;
  uint32_t phase = 0;
  // Direct: a warp takes NT neighbouring tiles of a unit; the page ids of its tokens (one a lane) are
  // read two units ahead and their rows one unit ahead.
  constexpr int KH = D / 32, KI = kPair ? 2 * KH : kDirect ? KH : 1;
  uint4 kn[2 * NT][KI], vn[2 * NT][KI];                    // [token g + 8 ..][features 32 i + 8 t ..]
  UnitWalk wi{rs.req, rs.tok, rs.n, rs.units, true}, wc = wi;   // of the page ids, of the products
  uint32_t mask_next = 0;
  int2 id = make_int2(-1, -1);
  bool no_token = true;
  const auto read_ids = [&] {
    id = make_int2(-1, -1);
    no_token = true;
    if (wi.left == 0) return;
    const int j = wi.tok + share * NT * kTile + lane;
    if (lane < NT * kTile && j < wi.n) {
      no_token = false;
      id = reinterpret_cast<const int2*>(a.table)[((int64_t)wi.req * a.max_len + j) * a.layers + a.layer];
    }
    wi.tok += st;
    --wi.left;
    walk_begin(a, wi);
  };
  const auto read_rows = [&] {
    const bool good = id.x >= 0 && id.x < a.num_pages && id.y >= 0 && id.y < a.num_pages;
    if (!good && !no_token) flag_error(a.err, LORA_DEV_BAD_PAGE);   // token skipped
    mask_next = __ballot_sync(0xffffffffu, good);
    const uint16_t* rows = a.pool + (h0 + hh) * D + 8 * t;
#pragma unroll
    for (int h = 0; h < 2 * NT; ++h) {
      const int pk = __shfl_sync(0xffffffffu, id.x, g + 8 * h), pv = __shfl_sync(0xffffffffu, id.y, g + 8 * h);
      const bool has = (mask_next >> (g + 8 * h)) & 1u;
      const uint4* kp = reinterpret_cast<const uint4*>(rows + (int64_t)pk * a.H);
      const uint4* vp = reinterpret_cast<const uint4*>(rows + (int64_t)pv * a.H);
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        kn[h][i] = has ? kp[4 * i] : make_uint4(0, 0, 0, 0);
        vn[h][i] = has ? vp[4 * i] : make_uint4(0, 0, 0, 0);
      }
    }
  };
  if (kDirect) {
    read_ids();
    read_rows();
    read_ids();
  }
  for (int left = rs.units; left > 0; --left) {
    const int s = next_s;
    int req, n, flags, tok, next;
    if constexpr (kDirect) {
      const uint32_t mask = mask_next;
      uint4 kc[2 * NT][KI], vc[2 * NT][KI];
#pragma unroll
      for (int h = 0; h < 2 * NT; ++h)
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          kc[h][i] = kn[h][i];
          vc[h][i] = vn[h][i];
        }
      if (pl.meet) asm volatile("bar.sync %0, %1;" ::"r"(1 + share), "r"(32 * head_warps) : "memory");
      read_rows();
      read_ids();
      req = wc.req;
      n = wc.n;
      tok = wc.tok;
      const bool first = wc.first, ends = wc.tok + st >= wc.n;
      wc.tok += st;
      --wc.left;
      wc.first = ends;
      walk_begin(a, wc);
      const int begun = req == rs.req ? rs.tok : 0;        // the segment's first token
      flags = (first ? kFirst : 0) | (ends || wc.left == 0 ? kLast : 0) | (begun == 0 ? kStarts : 0) | (ends ? kEnds : 0);
      next = wc.left > 0 ? wc.req : -1;
      if (first) begin_segment();
      const int j0 = tok + share * NT * kTile;
      if (j0 < n) {
        uint32_t pt[HW][NT][kTerms][2];
#pragma unroll
        for (int u = 0; u < HW; ++u) {
          float sc[NT][4], odd[NT][4];
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[b][i] = odd[b][i] = 0.f;
#pragma unroll
          for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int i = 0; i < KH; ++i) {
              const int c = kPair ? KH * u + i : i;
              const uint4 &x = kc[2 * b][c], &y = kc[2 * b + 1][c];
              const uint32_t k0[4] = {x.x, y.x, x.y, y.y}, k1[4] = {x.z, y.z, x.w, y.w};
              mma_16x8x16(sc[b], k0, qf[u][2 * i][0], qf[u][2 * i][1]);
              mma_16x8x16(odd[b], k1, qf[u][2 * i + 1][0], qf[u][2 * i + 1][1]);
            }
          tile_weights(u, req, j0, n, mask, sc, odd, pt[u]);
        }
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int i = 0; i < KI; ++i) {
            const uint4 &x = vc[2 * b][i], &y = vc[2 * b + 1][i];
            const uint32_t v0[4] = {transpose_8x8(x.x), transpose_8x8(x.y), transpose_8x8(y.x), transpose_8x8(y.y)};
            const uint32_t v1[4] = {transpose_8x8(x.z), transpose_8x8(x.w), transpose_8x8(y.z), transpose_8x8(y.w)};
#pragma unroll
            for (int u = 0; u < HW; ++u) {
              if (kPair && u != i / KH) continue;
              const int ks = 2 * (i % KH);
              float sum[2][4] = {};
#pragma unroll
              for (int k = kTerms - 1; k >= 0; --k) {
                mma_16x8x16(sum[0], v0, pt[u][b][k][0], pt[u][b][k][1]);
                mma_16x8x16(sum[1], v1, pt[u][b][k][0], pt[u][b][k][1]);
              }
              add_tile(acc[u][ks], sum[0]);
              add_tile(acc[u][ks + 1], sum[1]);
            }
          }
      }
    } else {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * s, phase))) {
        if (lane == 0) flag_error(a.err, LORA_DEV_WAIT_TIMEOUT);
        return;
      }
      if (++next_s == S) {
        next_s = 0;
        phase ^= 1;
      }
      const bool mine = next_turn == turn;
      if (++next_turn == turns) next_turn = 0;
      req = info[s].req;
      n = info[s].n;
      flags = info[s].flags;
      tok = info[s].tok;
      next = info[s].next;
      __syncwarp();
      if (flags & kFirst) begin_segment();
      if (!mine && lane == 0) mbar_arrive(bar_empty + 8 * s);
      for (int tile = mine ? share % tile_sharers : TILES; tile < TILES; tile += tile_sharers) {
        const int j0 = tok + tile * kTile;
        const bool final_tile = tile + tile_sharers >= TILES;
        if (j0 >= n) {
          if (final_tile) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
          }
          continue;
        }
        const uint32_t mask = info[s].mask[tile];
#pragma unroll
        for (int u = 0; u < HW; ++u) {
          if (u >= n_mine) break;
          const bool release = final_tile && u + 1 == n_mine;
          const uint32_t base = ring + (uint32_t)s * pl.stage_bytes + (uint32_t)(tile * kTile) * RB + u * head_step;
          float sc[NT][4], odd[NT][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[0][i] = odd[0][i] = 0.f;
#pragma unroll
          for (int k0 = 0; k0 < KS; k0 += 4) {
            uint32_t kf[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ldmatrix_x4(kf[k], base + k_lane + (k0 + k) * 32);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_16x8x16(k & 1 ? odd[0] : sc[0], kf[k], qf[u][k0 + k][0], qf[u][k0 + k][1]);
          }
          uint32_t vf[VR][4];
#pragma unroll
          for (int k = 0; k < VR; ++k) ldmatrix_x4_trans(vf[k], base + v_lane + k * 32);
          if (VR == KS && release) {                         // everything of the stage is in registers
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
          }
          uint32_t pt[NT][kTerms][2];
          tile_weights(u, req, j0, n, mask, sc, odd, pt);
          // V of a token without data is whatever the stage held before: its bits are cleared.
          const bool partial = mask != 0xFFFFu;
          const uint32_t b0 = mask >> (2 * t), b1 = mask >> (2 * t + 8);
          const uint32_t and0 = ((b0 & 1u) ? 0xFFFFu : 0u) | ((b0 & 2u) ? 0xFFFF0000u : 0u);
          const uint32_t and1 = ((b1 & 1u) ? 0xFFFFu : 0u) | ((b1 & 2u) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int k0 = 0; k0 < KS; k0 += VR) {
            if (k0 > 0) {
#pragma unroll
              for (int k = 0; k < VR; ++k) ldmatrix_x4_trans(vf[k], base + v_lane + (k0 + k) * 32);
            }
            if (partial) {
#pragma unroll
              for (int k = 0; k < VR; ++k) {
                vf[k][0] &= and0;
                vf[k][1] &= and0;
                vf[k][2] &= and1;
                vf[k][3] &= and1;
              }
            }
#pragma unroll
            for (int k1 = 0; k1 < VR; k1 += kBlocks) {
              float sum[kBlocks][4] = {};
#pragma unroll
              for (int i = kTerms - 1; i >= 0; --i)
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) mma_16x8x16(sum[k], vf[k1 + k], pt[0][i][0], pt[0][i][1]);
#pragma unroll
              for (int k = 0; k < kBlocks; ++k) add_tile(acc[u][k0 + k1 + k], sum[k]);
            }
          }
          if (VR < KS && release) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_empty + 8 * s);
          }
        }
      }
    }
    if (!(flags & kLast)) continue;

    // ---- the segment's end: sum l over the token lanes, join the warps that share the head ----
    if (next >= 0) load_q(next);                           // on its way while this segment is finished
#pragma unroll
    for (int u = 0; u < HW; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[u][k] += __shfl_xor_sync(0xffffffffu, l[u][k], 4);
        l[u][k] += __shfl_xor_sync(0xffffffffu, l[u][k], 8);
        l[u][k] += __shfl_xor_sync(0xffffffffu, l[u][k], 16);
      }
    if ((kDirect || HW == 1) && pl.sharers > 1) {
      constexpr int kMerged = HW * 8 * (D + 2);            // [HW][8][D + 2]: acc, m, l
      // Share 0 adds the other warps' parts in order.  One buffer per head, used by its warps in turn:
      // warp `share` writes it once the warp before (or, for the first, the last of the previous segment)
      // has been added.  Direct, where shared memory is free, every warp has its own.
      for (int o = 1; o < pl.sharers && !broken; ++o) {
        const uint32_t ready = bar_ready + 8 * (o * head_warps + hw);
        float* merged = merge + (size_t)(kDirect ? (o - 1) * head_warps + hw : hw) * kMerged;
        if (share == o) {
          const int before = kDirect ? o : o > 1 ? o - 1 : pl.sharers - 1;
          const uint32_t parity = kDirect || o == 1 ? (seg & 1) ^ 1 : seg & 1;
          if (!__all_sync(0xffffffffu, mbar_wait(bar_done + 8 * (before * head_warps + hw), parity))) {
            if (lane == 0) flag_error(a.err, LORA_DEV_WAIT_TIMEOUT);
            broken = true;
            break;
          }
#pragma unroll
          for (int uk = 0; uk < 2 * HW; ++uk) {
            const int u = uk / 2, k = uk & 1, qi = 2 * t + k;
            float* mb = merged + (size_t)u * 8 * (D + 2);
            if (qi >= n_query(u)) continue;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              mb[qi * (D + 2) + ks * 16 + g] = acc[u][ks][k];
              mb[qi * (D + 2) + ks * 16 + g + 8] = acc[u][ks][2 + k];
            }
            if (g == 0) {
              mb[qi * (D + 2) + D] = m[u][k];
              mb[qi * (D + 2) + D + 1] = l[u][k];
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(ready);
        } else if (share == 0) {
          if (!__all_sync(0xffffffffu, mbar_wait(ready, seg & 1))) {
            if (lane == 0) flag_error(a.err, LORA_DEV_WAIT_TIMEOUT);
            broken = true;
            break;
          }
#pragma unroll
          for (int uk = 0; uk < 2 * HW; ++uk) {
            const int u = uk / 2, k = uk & 1, qi = 2 * t + k;
            float* mb = merged + (size_t)u * 8 * (D + 2);
            if (qi >= n_query(u)) continue;
            const float om = mb[qi * (D + 2) + D], ol = mb[qi * (D + 2) + D + 1];
            const float mn = fmaxf(m[u][k], om), ms = mn == -INFINITY ? 0.f : mn;
            const float c0 = exp2f(m[u][k] - ms), c1 = exp2f(om - ms);
            m[u][k] = mn;
            l[u][k] = l[u][k] * c0 + ol * c1;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              acc[u][ks][k] = acc[u][ks][k] * c0 + mb[qi * (D + 2) + ks * 16 + g] * c1;
              acc[u][ks][2 + k] = acc[u][ks][2 + k] * c0 + mb[qi * (D + 2) + ks * 16 + g + 8] * c1;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_done + 8 * (o * head_warps + hw));
        }
      }
      ++seg;
      if (broken && !kDirect) return;                      // direct: the other warps wait at a barrier
      if (share != 0 || broken) continue;
    }
    const bool starts = flags & kStarts, ends = flags & kEnds;
    if (g0 == 0 && hw == 0 && lane == 0) {
      if (starts) a.ws_range[req].x = p;
      if (ends) a.ws_range[req].y = p;
    }
#pragma unroll
    for (int u = 0; u < HW; ++u) {
      if (u >= n_mine) break;
      const int head0 = head_of(u), G = n_query(u);
      if (starts && ends) {
        const float i0 = normalizer(l[u][0]), i1 = normalizer(l[u][1]);
        uint16_t* row = a.out + req * a.out_stride + (int64_t)(head0 + g) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t lo = transpose_8x8(pack_bf16(acc[u][ks][0] * i0, acc[u][ks][1] * i1));
          const uint32_t hi = transpose_8x8(pack_bf16(acc[u][ks][2] * i0, acc[u][ks][3] * i1));
          if (g < G) {
            *reinterpret_cast<uint32_t*>(row + pair_of(ks, 0)) = lo;
            *reinterpret_cast<uint32_t*>(row + pair_of(ks, 1)) = hi;
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int qi = 2 * t + k;
          if (g == 0 && qi < G) {
            const float z = l[u][k] == 0.f ? -INFINITY : m[u][k] + log2f(l[u][k]);
            a.ws_lse[(int64_t)req * a.n_heads + head0 + qi] = z;
            if (a.lse) a.lse[(int64_t)req * a.n_heads + head0 + qi] = z * 0.6931471805599453f;
          }
        }
      } else {
        const int64_t slot = partial_slot(p, starts) * a.n_heads + head0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int qi = 2 * t + k;
          if (qi >= G) continue;
          float* dst = a.ws_acc + (slot + qi) * D;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            dst[row_of(ks, 0)] = acc[u][ks][k];
            dst[row_of(ks, 1)] = acc[u][ks][2 + k];
          }
          if (g == 0) a.ws_ml[slot + qi] = make_float2(m[u][k], l[u][k]);
        }
      }
    }
  }
}

constexpr int kJoinBatch = 4;                              // partials whose loads are in flight together

// Adds partials i = p0 + first, + step, ... <= p1 of (request, head) to (m, l, acc); a lane holds
// every 32nd feature.
template <int D>
__device__ __forceinline__ void join_partials(const SplitArgs& a, int p0, int p1, int first, int step, int h, int lane,
                                              float& m, float& l, float (&acc)[D / 32]) {
  constexpr int E = D / 32;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i0 = p0 + first; i0 <= p1; i0 += kJoinBatch * step) {
    float x[kJoinBatch][E];
    float2 ml[kJoinBatch];
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const int i = min(i0 + b * step, p1);
      const int64_t slot = partial_slot(i, i == p0) * a.n_heads + h;
      ml[b] = a.ws_ml[slot];
      if (i0 + b * step > p1) ml[b] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[b][e] = i0 + b * step <= p1 ? a.ws_acc[slot * D + e * 32 + lane] : 0.f;
    }
    float mn = m;
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) mn = fmaxf(mn, ml[b].x);
    const float ms = mn == -INFINITY ? 0.f : mn, c = exp2f(m - ms);
    m = mn;
    l *= c;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= c;
#pragma unroll
    for (int b = 0; b < kJoinBatch; ++b) {
      const float f = exp2f(ml[b].x - ms);
      l = fmaf(ml[b].y, f, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(x[b][e], f, acc[e]);
    }
  }
}

// The same of 32 features, d0 + lane, for many partials: 16 of them at a time, a lane with the m and l
// of one and all the lane's loads in flight together.
template <int D>
__device__ __forceinline__ void join_many(const SplitArgs& a, int p0, int p1, int first, int step, int h, int d0, int lane,
                                          float& m, float& l, float& acc) {
  m = -INFINITY;
  l = acc = 0.f;
  for (int i0 = p0 + first; i0 <= p1; i0 += 16 * step) {
    const int mine = i0 + (lane & 15) * step;
    const float2 ml = mine <= p1 ? a.ws_ml[partial_slot(mine, mine == p0) * a.n_heads + h] : make_float2(-INFINITY, 0.f);
    float x[16];
#pragma unroll
    for (int b = 0; b < 16; ++b) {
      const int i = i0 + b * step;
      x[b] = i <= p1 ? a.ws_acc[(partial_slot(i, i == p0) * a.n_heads + h) * D + d0 + lane] : 0.f;
    }
    float mn = ml.x;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mn = fmaxf(mn, m);
    const float ms = mn == -INFINITY ? 0.f : mn, c = exp2f(m - ms), f = exp2f(ml.x - ms);
    m = mn;
    float add = ml.y * f;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
    l = fmaf(l, c, add);
    acc *= c;
#pragma unroll
    for (int b = 0; b < 16; ++b) acc = fmaf(x[b], __shfl_sync(0xffffffffu, f, b), acc);
  }
}

__device__ __forceinline__ void store_lse(const SplitArgs& a, int r, int h, float m, float l) {
  if (a.lse) a.lse[(int64_t)r * a.n_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Joins the requests that span ranges, and turns scores into weights: latency-bound, 4.5 us for a
// join alone, 10 us with the weights of 68,000 tokens x 32 heads (17 MB of scores read).
// Join: a request that spans ranges p0..p1 is the one in whose middle each of p0 + 1..p1 begins, so
// those ranges' blocks find it at once and share its query heads: up to JW partials a warp per head,
// beyond that a block per head, from kJoinMany on (JW = kManyWarps) a block per 32 features of one.
// Weights: the blocks cut the tokens of all requests anew into equal ranges.  Per request a block
// gathers the heads' lse (of a split request from its partials); then a lane of every warp takes two
// of 64 tokens, warp w every JW-th head, and the warps' sums are added in warp order.  With few heads
// every warp has tokens of its own instead and nothing to wait for: 64 requests of 8,000 to 15,625
// tokens of one head of 64 57 -> 48 us with the attention, but 32 heads of 128 46.6 -> 50.8.
// Registers are held to what lets 40 (or 32) warps share an SM, also with the split kernel's last blocks:
// at 60 instead of 48 one request of 8 KV heads of 128 with 4 query heads each took 15.2 us, not 11.9.
template <int D, int JW>
__global__ void __launch_bounds__(32 * JW, (JW == kFewWarps && D < 256 ? 40 : 32) / JW)
attention_join_kernel(const __grid_constant__ SplitArgs a, int32_t subs) {
  extern __shared__ float dyn[];                           // with weights: [n_heads] lse, the sums of find_range
  __shared__ float part[JW][D + 2];
  __shared__ __align__(8) float sums[2 * JW * kJoinUnit];
  constexpr int E = D / 32;
  pdl_wait_then_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!a.plan.whole) {
    const int p = blockIdx.x / subs, sub = blockIdx.x % subs;
    const int4 w = a.ws_start[p];
    if (w.y > 0) {
      const int r = w.x;
      const int2 range = make_int2(w.z, w.w);
      const bool wide = range.y - range.x >= JW;
      const int block = (p - range.x - 1) * subs + sub, blocks = (range.y - range.x) * subs;
      uint16_t* row = a.out + r * a.out_stride;
      if (JW > kFewWarps && range.y - range.x >= kJoinMany) {
        for (int item = block; item < a.n_heads * E; item += blocks) {
          const int h = item / E, d0 = item % E * 32;
          float m, l, acc;
          join_many<D>(a, range.x, range.y, warp, JW, h, d0, lane, m, l, acc);
          __syncthreads();
          part[warp][lane] = acc;
          if (lane == 0) {
            part[warp][D] = m;
            part[warp][D + 1] = l;
          }
          __syncthreads();
          if (warp == 0) {
            float M = -INFINITY, L = 0.f, x = 0.f;
#pragma unroll
            for (int v = 0; v < JW; ++v) M = fmaxf(M, part[v][D]);
            const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int v = 0; v < JW; ++v) {
              const float c = exp2f(part[v][D] - ms);
              L = fmaf(part[v][D + 1], c, L);
              x = fmaf(part[v][lane], c, x);
            }
            row[(int64_t)h * D + d0 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(x * normalizer(L)));
            if (d0 == 0 && lane == 0) store_lse(a, r, h, M, L);
          }
        }
      } else if (wide) {
        for (int h = block; h < a.n_heads; h += blocks) {
          float m, l, acc[E];
          join_partials<D>(a, range.x, range.y, warp, JW, h, lane, m, l, acc);
          __syncthreads();
#pragma unroll
          for (int e = 0; e < E; ++e) part[warp][e * 32 + lane] = acc[e];
          if (lane == 0) {
            part[warp][D] = m;
            part[warp][D + 1] = l;
          }
          __syncthreads();
          float M = -INFINITY, L = 0.f, c[JW];
#pragma unroll
          for (int v = 0; v < JW; ++v) M = fmaxf(M, part[v][D]);
          const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int v = 0; v < JW; ++v) {
            c[v] = exp2f(part[v][D] - ms);
            L = fmaf(part[v][D + 1], c[v], L);
          }
          const float inv = normalizer(L);
          for (int d = threadIdx.x; d < D; d += 32 * JW) {
            float x = 0.f;
#pragma unroll
            for (int v = 0; v < JW; ++v) x = fmaf(part[v][d], c[v], x);
            row[(int64_t)h * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(x * inv));
          }
          if (threadIdx.x == 0) store_lse(a, r, h, M, L);
        }
      } else {
        for (int h = block * JW + warp; h < a.n_heads; h += blocks * JW) {
          float m, l, acc[E];
          join_partials<D>(a, range.x, range.y, 0, 1, h, lane, m, l, acc);
          const float inv = normalizer(l);
#pragma unroll
          for (int e = 0; e < E; ++e)
            row[(int64_t)h * D + e * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
          if (lane == 0) store_lse(a, r, h, m, l);
        }
      }
    }
  }
  if (!a.weight_out) return;

  float* lse_s = dyn;
  const RangeStart rs = find_range(a, blockIdx.x, gridDim.x, kJoinUnit, reinterpret_cast<int32_t*>(dyn + a.n_heads));
  int r = rs.req, tok = rs.tok;
  for (int left = rs.units; left > 0;) {
    const int n = request_length(a, r);
    if (tok >= n) {
      ++r;
      tok = 0;
      continue;
    }
    const int units = min(left, (int)(((int64_t)n - tok + kJoinUnit - 1) / kJoinUnit));
    const int2 range = a.ws_range[r];
    __syncthreads();                                       // lse_s and part are done with
    if (range.x == range.y) {
      for (int h = threadIdx.x; h < a.n_heads; h += 32 * JW) {
        const float z = a.ws_lse[(int64_t)r * a.n_heads + h];
        lse_s[h] = z == -INFINITY ? INFINITY : z;          // a row without weight: 2^(s - inf) = 0
      }
    } else {
      // up to 32 heads, a lane each, the partials over the warps and over what lanes are left
      const int side = JW == kFewWarps || a.n_heads > 16 ? 32 : a.n_heads > 8 ? 16 : a.n_heads > 4 ? 8 : 4;
      const int rows = JW * (32 / side);
      for (int h0 = 0; h0 < a.n_heads; h0 += 32) {
        const int h = min(h0 + lane % side, a.n_heads - 1);
        float M = -INFINITY, L = 0.f;
        for (int i0 = range.x + warp * (32 / side) + lane / side; i0 <= range.y; i0 += 8 * rows) {
          float2 ml[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const int i = i0 + b * rows;
            ml[b] = i <= range.y ? a.ws_ml[partial_slot(i, i == range.x) * a.n_heads + h] : make_float2(-INFINITY, 0.f);
          }
          float mn = M;
#pragma unroll
          for (int b = 0; b < 8; ++b) mn = fmaxf(mn, ml[b].x);
          const float ms = mn == -INFINITY ? 0.f : mn;
          L *= exp2f(M - ms);
          M = mn;
#pragma unroll
          for (int b = 0; b < 8; ++b) L = fmaf(ml[b].y, exp2f(ml[b].x - ms), L);
        }
        for (int o = side; o < 32; o <<= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, M, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
          const float mn = fmaxf(M, m2), ms = mn == -INFINITY ? 0.f : mn;
          L = L * exp2f(M - ms) + l2 * exp2f(m2 - ms);
          M = mn;
        }
        __syncthreads();
        part[warp][2 * lane] = M;
        part[warp][2 * lane + 1] = L;
        __syncthreads();
        if (warp == 0 && h0 + lane < a.n_heads) {
          float m = -INFINITY, l = 0.f;
#pragma unroll
          for (int v = 0; v < JW; ++v) m = fmaxf(m, part[v][2 * lane]);
          const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int v = 0; v < JW; ++v) l = fmaf(part[v][2 * lane + 1], exp2f(part[v][2 * lane] - ms), l);
          lse_s[h] = l == 0.f ? INFINITY : m + log2f(l);
        }
      }
    }
    __syncthreads();
    // two neighbouring tokens a lane; a score row is padded to whole tiles, so the pair is there
    const float* row = a.ws_scores + (int64_t)r * a.n_heads * a.score_stride;
    if (a.n_heads <= kWarpHeads) {                         // a warp takes all heads of its tokens
      for (int u = warp; u < units; u += JW) {
        const int64_t j = tok + (int64_t)u * kJoinUnit + 2 * lane;
        if (j >= n) continue;
        const int64_t at = r * a.weight_stride + j;
        const bool two = j + 1 < n;
        float x0 = 0.f, x1 = 0.f;
        const float w0 = a.weight_in ? a.weight_in[at] : 0.f, w1 = a.weight_in && two ? a.weight_in[at + 1] : 0.f;
#pragma unroll 8
        for (int h = 0; h < a.n_heads; ++h) {
          const float2 v = *reinterpret_cast<const float2*>(row + j + h * a.score_stride);
          x0 += exp2f(v.x - lse_s[h]);
          x1 += exp2f(v.y - lse_s[h]);
        }
        a.weight_out[at] = w0 + x0;
        if (two) a.weight_out[at + 1] = w1 + x1;
      }
    } else {
    for (int u = 0; u < units; ++u) {
      const int64_t j = tok + (int64_t)u * kJoinUnit + 2 * lane;
      float x0 = 0.f, x1 = 0.f;
      if (j < n) {
        const float* sc = row + j;
#pragma unroll 8
        for (int h = warp; h < a.n_heads; h += JW) {
          const float2 v = *reinterpret_cast<const float2*>(sc + h * a.score_stride);
          x0 += exp2f(v.x - lse_s[h]);
          x1 += exp2f(v.y - lse_s[h]);
        }
      }
      float* sum = sums + (u & 1) * JW * kJoinUnit;                // two buffers: one barrier a turn
      sum[warp * kJoinUnit + 2 * lane] = x0;
      sum[warp * kJoinUnit + 2 * lane + 1] = x1;
      __syncthreads();
      const int64_t jt = tok + (int64_t)u * kJoinUnit + threadIdx.x;
      if (threadIdx.x < kJoinUnit && jt < n) {
        float x = 0.f;
#pragma unroll
        for (int v = 0; v < JW; ++v) x += sum[v * kJoinUnit + threadIdx.x];
        const int64_t at = r * a.weight_stride + jt;
        a.weight_out[at] = (a.weight_in ? a.weight_in[at] : 0.f) + x;
      }
    }
    }
    left -= units;
    tok = (int)min((int64_t)n, tok + (int64_t)units * kJoinUnit);
  }
}

struct SplitLayout {
  size_t lse, range, start, ml, acc, scores, total;
  int64_t score_stride;
};

SplitLayout split_layout(const SplitPlan& pl, int32_t n_req, int32_t max_len, int32_t n_heads, bool weights) {
  SplitLayout L{};
  const size_t slots = pl.whole ? 0 : 2 * (size_t)pl.parts;
  L.score_stride = ((int64_t)max_len + kTile - 1) / kTile * kTile;
  size_t off = 0;
  L.lse = off;     off = align256(off + (size_t)n_req * n_heads * 4);
  L.range = off;   off = align256(off + (size_t)n_req * sizeof(int2));
  L.start = off;   off = align256(off + (size_t)pl.parts * sizeof(int4));
  L.ml = off;      off = align256(off + slots * n_heads * sizeof(float2));
  L.acc = off;     off = align256(off + slots * n_heads * pl.D * 4);
  L.scores = off;  off = align256(off + (weights ? (size_t)n_req * n_heads * L.score_stride * 4 : 0));
  L.total = off;
  return L;
}

SplitPlan split_plan(int32_t H, int32_t n_req, int32_t max_len, int32_t n_heads, int32_t n_kv) {
  SplitPlan pl{};
  pl.n_kv = n_kv;
  pl.D = H / n_kv;
  pl.group = n_heads / n_kv;
  // Direct: a warp has one KV head, with all its query heads at D = 64 and 8 of them at D = 128.
  // Else a warp has 8 query heads of one KV head, or of two of 64 (so that a slice stays 1 KB); head
  // groups as even as they can be, a stage's K and V within kStageBytes at 16 tokens; with fewer heads
  // than warps some warps share a head's tokens and the stage has more of them.
  pl.direct = pl.D <= 128 && H * 2 <= kDirectSlice;
  // In a large cache it pays to read the heads of a token together: two heads of 64 by one warp, else by
  // warps that wait for one another.  64 requests, us without / with, one query head per KV head: two
  // heads of 64, 1 GB 251 / 171 (the warps waiting: 216), 512 MB 101 / 90.8, 256 MB 49.7 / 50.1, 2 MB
  // 4.0 / 5.6; three heads, 1 GB 246 / 201, 128 MB 31.5 / 32.8.
  const bool together = pl.direct && (int64_t)n_req * max_len * 4 * H >= kTogetherBytes;
  pl.pair = together && pl.D == 64 && n_kv == 2 && pl.group <= 8;
  pl.octets = pl.direct && pl.D == 64 ? 1 : (pl.group + 7) / 8;
  const int slots = kWarps / pl.octets, room_heads = std::max(1, kStageBytes / (4 * kTile * pl.D));
  const int most = std::min(pl.D == 64 && !pl.direct ? 2 * slots : slots, room_heads);
  pl.n_groups = (n_kv + most - 1) / most;
  pl.heads = (n_kv + pl.n_groups - 1) / pl.n_groups;
  pl.head_slots = pl.pair ? 1 : std::min(pl.heads, slots);
  pl.meet = together && pl.head_slots > 1;
  const int room = kStageBytes / (4 * kTile * pl.heads * pl.D);
  pl.sharers = slots / pl.head_slots;                      // a power of two where it is not 1, as is room then
  pl.tile_sharers = std::min(pl.sharers, room);
  pl.tiles = std::min(room / pl.tile_sharers, kMaxTiles / pl.tile_sharers) * pl.tile_sharers;
  if (pl.direct) pl.tiles = pl.sharers * (pl.pair ? 1 : 128 / pl.D);     // a unit: so many tiles per warp
  pl.row_bytes = pl.heads * pl.D * 2 + 16;                 // + 16: ldmatrix's 8 rows on 8 bank groups
  pl.stage_bytes = pl.direct ? 0 : 2 * kTile * pl.tiles * pl.row_bytes;
  // behind the ring: the sums of find_range (4 bytes per 128 requests), later the merged heads
  const int buffers = pl.sharers == 1 ? 0 : (pl.direct ? pl.sharers - 1 : 1) * pl.heads * ((pl.group + 7) / 8);
  const int merge = buffers * 8 * (pl.D + 2) * 4;
  const int tail = std::max(merge, (n_req + 127) / 128 * 4);
  pl.stages = pl.direct ? 0 : std::min(kMaxStages, (kMaxSmem - kStaticSmem - tail) / pl.stage_bytes);
  pl.smem = pl.stages * pl.stage_bytes + tail;
  const int sms = device_sm_count() * kCtasPerSm;
  // One CTA per request and head group, and no join, where a request is at most four tiles and all
  // CTAs run in two rounds.  H = 4096, one GB300, us a call, whole requests / ranges: 1 request of 13
  // tokens 3.7 / 6.8, of 61 6.3 / 7.0, of 125 9.8 / 7.2; 64 requests (512 CTAs) of 61 13.6 / 16.4; 256
  // requests (2,048 CTAs) of 13 24.6 / 18.1, of 61 59 / 47.
  pl.whole = max_len <= 4 * kTile && (int64_t)n_req * pl.n_groups <= 2 * sms;
  if (pl.whole) {
    pl.parts = n_req;
  } else {
    // As many CTAs as run at once; where the head groups do not divide them, up to 4 rounds (32 groups,
    // H = 16384: 60,000 tokens 587 us in one round of 288 CTAs, 567 in two of 304; 16 requests of 500
    // tokens 84.6 and 87.2).
    double best = 0;
    for (int k = 1; k <= 4; ++k) {
      const int parts = k * sms / pl.n_groups;
      const double used = (double)parts * pl.n_groups / (k * sms);
      if (used > best + 0.02) {
        best = used;
        pl.parts = parts;
      }
    }
    pl.parts = std::max(pl.parts, 1);
  }
  return pl;
}

// Shape checks shared by the size query and the call; 0 or an error code.
int check_shape(const char* fn, const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads, int32_t n_kv) {
  const auto fail = [fn](const char* what) { return lora_fail(LORA_EINVAL, std::string(fn) + what); };
  if (!p || n_req < 0 || max_len < 1 || n_heads < 1 || n_kv < 1) return fail(": bad arguments");
  if (n_req > 65535) return fail(": at most 65535 requests per call");
  if (max_len > (1 << 30)) return fail(": max_len is at most 2^30");   // positions are 32-bit, units pass the end
  if (n_req * (((int64_t)max_len + kTile - 1) / kTile) > INT32_MAX) return fail(": n_req x max_len is at most 16 x 2^31");
  if (n_heads % n_kv != 0 || n_heads / n_kv > kSplitMaxGroup)
    return fail(": n_heads must be 1 to 16 times n_kv_heads");
  if (p->H % n_kv != 0) return fail(": H is not a multiple of n_kv_heads");
  const int D = p->H / n_kv;
  if (D != 64 && D != 128 && D != 256) return fail(": head width must be 64, 128 or 256");
  return LORA_OK;
}

template <int D, int TILES, int NP, int HW>
int launch_split(const lora_pool* p, const SplitArgs& a, cudaStream_t st) {
  static DeviceFlags flags;
  const int rc = ensure_smem_attr(flags, &attention_split_kernel<D, TILES, NP, HW>, kMaxSmem - kStaticSmem, "lora_attention_split");
  if (rc != LORA_OK) return rc;
  ProfScope prof(p, LORA_KIND_ATTENTION, st);
  const cudaError_t e = launch_pdl(!p->prof_on, attention_split_kernel<D, TILES, NP, HW>, dim3(a.plan.parts * a.plan.n_groups),
                                   dim3(threads_of(NP)), a.plan.smem, st, a);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_attention_split launch");
}

// The kernel of a shape: split_plan gives these tile counts, and the slices that take two producers.
int launch_split_any(const lora_pool* p, const SplitArgs& a, cudaStream_t st) {
  const SplitPlan& pl = a.plan;
  const bool two = pl.whole || pl.heads * pl.D * 2 < kSmallSlice, pairs = pl.heads > pl.head_slots;
  if (pl.direct && pl.D == 128) return launch_split<128, 1, 0, 1>(p, a, st);
  if (pl.pair) return launch_split<64, 1, 0, 2>(p, a, st);
  if (pl.direct) return pl.group > 8 ? launch_split<64, 2, 0, 2>(p, a, st) : launch_split<64, 2, 0, 1>(p, a, st);
  switch (pl.D * 16 + pl.tiles) {
    case 64 * 16 + 1: return two ? launch_split<64, 1, 2, 2>(p, a, st) : launch_split<64, 1, 1, 2>(p, a, st);
    case 64 * 16 + 2: return pairs ? launch_split<64, 2, 2, 2>(p, a, st) : launch_split<64, 2, 2, 1>(p, a, st);
    case 128 * 16 + 1: return two ? launch_split<128, 1, 2, 1>(p, a, st) : launch_split<128, 1, 1, 1>(p, a, st);
    case 128 * 16 + 2: return launch_split<128, 2, 2, 1>(p, a, st);
    case 256 * 16 + 1: return two ? launch_split<256, 1, 2, 1>(p, a, st) : launch_split<256, 1, 1, 1>(p, a, st);
    case 256 * 16 + 2: return launch_split<256, 2, 2, 1>(p, a, st);
  }
  return lora_fail(LORA_EINVAL, "lora_attention_split: no kernel for this geometry");
}

template <int D, int JW>
int launch_join(const lora_pool* p, const SplitArgs& a, cudaStream_t st) {
  const int subs = std::max(1, 32 / JW * device_sm_count() / a.plan.parts);   // 32 warps per SM
  const size_t smem = a.weight_out ? (size_t)(a.n_heads + (a.n_req + 127) / 128) * 4 : 0;
  ProfScope prof(p, LORA_KIND_ATTENTION, st);
  const cudaError_t e = launch_pdl(!p->prof_on, attention_join_kernel<D, JW>, dim3(a.plan.parts * subs), dim3(32 * JW),
                                   smem, st, a, subs);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_attention_split launch");
}

template <int D>
int launch_join_any(const lora_pool* p, const SplitArgs& a, cudaStream_t st) {
  // Few heads with many partials each leave most blocks of four warps without a head, so a block of
  // eight warps takes 32 features of a head.  One GB300, 8 MB of K and V, us a call by few / many warps:
  // one request (304 partials a head) of 1 head of 64 17.7 / 11.2, of 2 KV heads of 256 with 16 query
  // heads each 23.8 / 15.7; 4 requests (76) of 1 head, 32 MB, 16.4 / 14.9.  With more heads the blocks
  // are busy: one request (152) of 128 heads of 128 11.4 / 13.6, with weights 20.3 / 24.9.
  const int64_t per = std::max(kJoinMany, 8 * a.n_heads);
  const bool many = !a.plan.whole && a.plan.parts >= per * a.n_req;
  return many ? launch_join<D, kManyWarps>(p, a, st) : launch_join<D, kFewWarps>(p, a, st);
}

}  // namespace

extern "C" int64_t lora_attention_split_size(const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads,
                                             int32_t n_kv_heads, int32_t with_weights) {
  const int rc = check_shape("lora_attention_split_size", p, n_req, max_len, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_attention_split_size: planning pool has no device state");
  const SplitPlan pl = split_plan(p->H, n_req, max_len, n_heads, n_kv_heads);
  return (int64_t)split_layout(pl, n_req, max_len, n_heads, with_weights != 0).total;
}

extern "C" int lora_attention_split(lora_pool* p, int32_t n_req, const int32_t* table_dev, const int32_t* seq_len_dev,
                                    int32_t max_len, int32_t layers, int32_t layer, const void* q, int64_t q_stride,
                                    void* out, int64_t out_stride, int32_t n_heads, int32_t n_kv_heads, float* lse,
                                    const float* weight_in, float* weight_out, int64_t weight_stride, void* workspace,
                                    int64_t workspace_bytes, lora_stream_t stream) {
  const int rc = check_shape("lora_attention_split", p, n_req, max_len, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (layers < 1 || layer < 0 || layer >= layers)
    return lora_fail(LORA_EINVAL, "lora_attention_split: layer outside [0, layers)");
  if (weight_in && !weight_out) return lora_fail(LORA_EINVAL, "lora_attention_split: weight_in without weight_out");
  if (n_req > 0 && (!table_dev || !seq_len_dev || !q || !out || !workspace))
    return lora_fail(LORA_EINVAL, "lora_attention_split: null pointer");
  const int64_t width = (int64_t)n_heads * (p->H / n_kv_heads);
  if (q_stride == 0) q_stride = width;
  if (out_stride == 0) out_stride = width;
  if (weight_stride == 0) weight_stride = max_len;
  if (q_stride < width || out_stride < width || ((q_stride | out_stride) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: row strides must be multiples of 8 and at least a row");
  if (weight_stride < max_len) return lora_fail(LORA_EINVAL, "lora_attention_split: weight_stride is below max_len");
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: q and out must be 16-byte aligned");
  if (n_req > 0 && q == out) return lora_fail(LORA_EINVAL, "lora_attention_split: out must not alias q");
  if ((reinterpret_cast<uintptr_t>(table_dev) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: the table must be 8-byte aligned");
  if (((reinterpret_cast<uintptr_t>(seq_len_dev) | reinterpret_cast<uintptr_t>(lse) |
        reinterpret_cast<uintptr_t>(weight_in) | reinterpret_cast<uintptr_t>(weight_out)) & 3) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: lengths, lse and weights must be 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: workspace must be 256-byte aligned");
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_attention_split: planning pool has no device state");
  if (n_req == 0) return LORA_OK;
  const SplitPlan pl = split_plan(p->H, n_req, max_len, n_heads, n_kv_heads);
  const SplitLayout L = split_layout(pl, n_req, max_len, n_heads, weight_out != nullptr);
  if (workspace_bytes < (int64_t)L.total)
    return lora_fail(LORA_EINVAL, "lora_attention_split: workspace has " + std::to_string(workspace_bytes) +
                                      " bytes, needs " + std::to_string(L.total));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  SplitArgs a{};
  a.pool = static_cast<const uint16_t*>(p->pool_dev);
  a.num_pages = p->num_pages;
  a.H = p->H;
  a.n_req = n_req;
  a.table = table_dev;
  a.seq_len = seq_len_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.layer = layer;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.n_heads = n_heads;
  a.lse = lse;
  a.weight_in = weight_in;
  a.weight_out = weight_out;
  a.weight_stride = weight_stride;
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)pl.D);   // log2(e) / sqrt(D)
  a.plan = pl;
  char* ws = static_cast<char*>(workspace);
  a.ws_lse = reinterpret_cast<float*>(ws + L.lse);
  a.ws_range = reinterpret_cast<int2*>(ws + L.range);
  a.ws_start = reinterpret_cast<int4*>(ws + L.start);
  a.ws_ml = reinterpret_cast<float2*>(ws + L.ml);
  a.ws_acc = reinterpret_cast<float*>(ws + L.acc);
  a.ws_scores = weight_out ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  a.score_stride = L.score_stride;
  a.err = p->d_err;
  const int rc2 = launch_split_any(p, a, st);
  if (rc2 != LORA_OK || (pl.whole && !weight_out)) return rc2;
  return pl.D == 64    ? launch_join_any<64>(p, a, st)
         : pl.D == 128 ? launch_join_any<128>(p, a, st)
                       : launch_join_any<256>(p, a, st);
}

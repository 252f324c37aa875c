// KV rows into pages, and eviction from the KV cache by accumulated attention weight.
//
// Both work on device page tables [n_req][max_len][layers][2] (K page, V page per cached token and
// layer), so neither needs the host between steps.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "tc_ptx.h"

namespace {

// ---- page writes -------------------------------------------------------------------------------
// One warp per (row, K or V): the page id is read through the table and checked, then the row's
// 2 H bytes are copied 16 bytes a lane.  HBM-bound: every row is read once and written once.
constexpr int kWriteThreads = 256;

__global__ void __launch_bounds__(kWriteThreads)
kv_write_kernel(uint16_t* __restrict__ pool, int64_t num_pages, int32_t H, int32_t n_rows,
                const int32_t* __restrict__ row_req, const int32_t* __restrict__ row_pos,
                const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t k_stride, int64_t v_stride,
                int32_t n_req, const int2* __restrict__ table, int32_t max_len, int32_t layers, int32_t layer,
                int32_t* err) {
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
  for (int i = lane; i < H / 8; i += 32) dst[i] = src[i];
}

// ---- eviction ------------------------------------------------------------------------------------
// Sort key of a weight: ascending with the value, -0 = +0, NaN = -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The keys that stay are found by radix selection, digit by digit from the top: a histogram of the
// digit over the keys that still match the digits chosen so far, and the bin that holds the
// need-th largest key.  11 + 11 + 10 bits: the first digit (sign, exponent, two bits of the
// fraction) already spreads weights of like size over many bins, and selection ends with the first
// digit whose bin is wanted whole, which for weights that differ is the second.
constexpr int kEvictMaxThreads = 512;
constexpr int kEvictMaxWarps = kEvictMaxThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictDigits = 3;
constexpr int kEvictMaxCluster = 8;
__device__ __forceinline__ int digit_shift(int d) { return d == 0 ? 21 : d == 1 ? 10 : 0; }

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
__device__ __forceinline__ void cluster_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t addr, int v) {
  asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

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

// One cluster of `n_cta` CTAs (one CTA where rows are short or many) per (request, layer), layers
// next to each other so that the table's 32-byte sectors, which hold four layers, are shared in L2.
// Every CTA takes a contiguous slice of the row, every warp a contiguous part of that, so the kept
// tokens are numbered with one exchange of counts: warps count what they keep, and then write from
// their offset, 32 tokens a step.  Several CTAs add their histograms' filled bins into each other's
// shared memory (integer sums: the order does not matter).
// Latency-bound: a row is a chain of dependent steps (length, weights, digits, counts, pages), so
// what counts is how many rows an SM holds, and for few long rows how many CTAs share one.
template <bool kCluster>
__global__ void __launch_bounds__(kEvictMaxThreads) kv_evict_kernel(const EvictArgs a, int32_t n_cta) {
  extern __shared__ int hist[];                            // [kEvictBins] mine; of a cluster then [digits][bins] all CTAs'
  __shared__ int warp_sum[kEvictMaxWarps];
  __shared__ int found[3];                                 // the wanted bin, keys above it, keys in it
  __shared__ int warp_gt[kEvictMaxWarps], warp_eq[kEvictMaxWarps];
  __shared__ int cta_gt[kEvictMaxCluster], cta_eq[kEvictMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_thr = blockDim.x, n_warp = n_thr >> 5;
  for (int i = tid; i < kEvictBins * (kCluster ? 1 + kEvictDigits : 1); i += n_thr) hist[i] = 0;
  pdl_wait_then_release();
  const int rank = kCluster ? (int)cluster_rank() : 0;
  const int id = kCluster ? blockIdx.x / n_cta : blockIdx.x;
  const int layer = id % a.layers, r = id / a.layers;
  int n = a.seq_len[r];
  if (n < 0 || n > a.max_len) {
    if (tid == 0) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    n = n < 0 ? 0 : a.max_len;
  }
  const int n_keep = min(n, a.budget);
  const int old = n - min(n, a.recent);                    // tokens that compete; the newer ones stay
  const int64_t row = (int64_t)layer * a.n_req + r;
  const float* w = a.weight + row * a.max_len;
  int need = n_keep - (n - old);                           // of the old ones stay
  // this CTA's slice of the row, and this warp's part of it (multiples of 32)
  const int per_cta = ((n + n_cta - 1) / n_cta + 31) & ~31;
  const int c0 = (int)min((int64_t)n, (int64_t)rank * per_cta), c1 = min(n, c0 + per_cta);
  const int per_warp = ((c1 - c0 + n_warp - 1) / n_warp + 31) & ~31;
  const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);

  uint32_t cut = 0;                                        // keys above it stay, and `ties` of those equal to it
  int ties = 0;
  const bool select = need > 0 && need < old;
  if (need >= old) {
    ties = old;                                            // every old key is >= 0: all stay
  } else if (!select) {
    cut = 0xFFFFFFFFu;                                     // none does
  }
  __syncthreads();
  if (kCluster) cluster_sync_all();                        // every CTA's histograms are clear
  if (select) {
    const int s0 = min(c0, old), s1 = min(c1, old);
    uint32_t prefix = 0, mask = 0;
    for (int d = 0; d < kEvictDigits; ++d) {
      const int shift = digit_shift(d);
      const uint32_t digit = d == 2 ? 1023u : 2047u;
#pragma unroll 4
      for (int j = s0 + tid; j < s1; j += n_thr) {
        const uint32_t key = weight_key(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1);
      }
      __syncthreads();
      const int* all = hist;
      if (kCluster) {
        int* sum = hist + kEvictBins * (1 + d);
        for (int i = tid; i < kEvictBins; i += n_thr) {
          const int v = hist[i];
          if (v == 0) continue;
          hist[i] = 0;
          for (int c = 0; c < n_cta; ++c) cluster_add(cluster_addr(sum + i, c), v);
        }
        cluster_sync_all();
        all = sum;
      }
      // bins from the top: thread t holds the bins [B - (t + 1) per, B - t per)
      const int per = kEvictBins / n_thr;
      int mine = 0;
      for (int i = 0; i < per; ++i) mine += all[kEvictBins - 1 - tid * per - i];
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      int above = incl - mine;
      for (int i = 0; i < warp; ++i) above += warp_sum[i];
      if (above < need && above + mine >= need) {          // one thread: the need-th largest key is in its bins
        int b = kEvictBins - 1 - tid * per;
        while (above + all[b] < need) above += all[b--];
        found[0] = b;
        found[1] = above;
        found[2] = all[b];
      }
      __syncthreads();
      need -= found[1];
      prefix |= (uint32_t)found[0] << shift;
      mask |= digit << shift;
      cut = prefix;
      ties = need;
      if (found[2] == need) {                              // the whole bin stays
        cut = prefix - 1;                                  // not 0: a key below it is left out
        ties = 0;
        break;
      }
      if (!kCluster && d + 1 < kEvictDigits) {
        for (int i = tid; i < kEvictBins; i += n_thr) hist[i] = 0;
        __syncthreads();
      }
    }
  }

  // what each warp keeps: keys above the cut (and the newer tokens), and keys equal to it
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < w1 && j < old ? weight_key(w[j]) : 0u;
    gt += j < w1 && (j >= old || key > cut);
    eq += j < w1 && j < old && key == cut;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  int gt_before = 0, eq_before = 0;                        // of the row, before this warp's part
  if (kCluster) {
    if (tid < n_cta) {
      int g = 0, e = 0;
      for (int i = 0; i < n_warp; ++i) {
        g += warp_gt[i];
        e += warp_eq[i];
      }
      cluster_store(cluster_addr(cta_gt + rank, tid), g);
      cluster_store(cluster_addr(cta_eq + rank, tid), e);
    }
    cluster_sync_all();
    for (int i = 0; i < rank; ++i) {
      gt_before += cta_gt[i];
      eq_before += cta_eq[i];
    }
  }
  for (int i = 0; i < warp; ++i) {
    gt_before += warp_gt[i];
    eq_before += warp_eq[i];
  }
  int pos = gt_before + min(eq_before, ties);
  int32_t* keep = a.keep + row * a.budget;
  float* w_out = a.weight_out + row * a.max_len_out;
  int2* t_out = a.table_out + (int64_t)r * a.max_len_out * a.layers + layer;
  const int2* t_in = a.table + (int64_t)r * a.max_len * a.layers + layer;
#pragma unroll 4
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const float x = j < w1 ? w[j] : 0.f;
    const uint32_t key = weight_key(x);
    const bool e = j < w1 && j < old && key == cut;
    const uint32_t me = __ballot_sync(0xffffffffu, e);
    const uint32_t below = (1u << lane) - 1;
    const bool stay = j < w1 && (j >= old || key > cut || (e && eq_before + __popc(me & below) < ties));
    const uint32_t ms = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const int i = pos + __popc(ms & below);
      keep[i] = j;
      w_out[i] = x;
      t_out[(int64_t)i * a.layers] = t_in[(int64_t)j * a.layers];
    }
    pos += __popc(ms);
    eq_before += __popc(me);
  }
  const int step = n_cta * n_thr, first = n_keep + rank * n_thr + tid;
  for (int i = first; i < a.budget; i += step) keep[i] = -1;
  for (int i = first; i < a.max_len_out; i += step) {
    w_out[i] = 0.f;
    t_out[(int64_t)i * a.layers] = make_int2(-1, -1);
  }
  if (layer == 0 && rank == 0 && tid == 0) a.new_len[r] = n_keep;
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
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_kv_write: planning pool has no device state");
  if (n_rows == 0) return LORA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t items = 2 * (int64_t)n_rows;
  const unsigned grid = (unsigned)((items + kWriteThreads / 32 - 1) / (kWriteThreads / 32));
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e =
      launch_pdl(!p->prof_on, kv_write_kernel, dim3(grid), dim3(kWriteThreads), 0, st,
                 static_cast<uint16_t*>(p->pool_dev), p->num_pages, p->H, n_rows, row_req, row_pos,
                 static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride, v_stride, n_req,
                 reinterpret_cast<const int2*>(table_dev), max_len, layers, layer, p->d_err);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_write launch");
}

extern "C" int lora_kv_evict(lora_pool* p, int32_t n_req, const int32_t* table_dev, const int32_t* seq_len_dev,
                             int32_t max_len, int32_t layers, const float* weight_dev, int32_t budget, int32_t recent,
                             int32_t* keep_dev, int32_t* new_len_dev, int32_t* table_out, float* weight_out,
                             int32_t max_len_out, lora_stream_t stream) {
  if (!p || n_req < 0 || max_len < 1 || layers < 1) return lora_fail(LORA_EINVAL, "lora_kv_evict: bad arguments");
  if (budget < 1 || recent < 0 || recent > budget)
    return lora_fail(LORA_EINVAL, "lora_kv_evict: budget must be at least 1 and recent within [0, budget]");
  if (max_len > (1 << 30) || max_len_out > (1 << 30))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: max_len and max_len_out are at most 2^30");
  if (max_len_out < std::min(budget, max_len))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: max_len_out is below min(budget, max_len)");
  if (n_req > 0 && (!table_dev || !seq_len_dev || !weight_dev || !keep_dev || !new_len_dev || !table_out ||
                    !weight_out))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: null pointer");
  if (((reinterpret_cast<uintptr_t>(table_dev) | reinterpret_cast<uintptr_t>(table_out)) & 7) != 0)
    return lora_fail(LORA_EINVAL, "lora_kv_evict: tables must be 8-byte aligned");
  if (n_req > 0 && (table_dev == table_out || weight_dev == weight_out || seq_len_dev == new_len_dev))
    return lora_fail(LORA_EINVAL, "lora_kv_evict: outputs must not be the inputs");
  if ((int64_t)n_req * layers > INT32_MAX) return lora_fail(LORA_EINVAL, "lora_kv_evict: too many (request, layer) rows");
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
  // A cluster per row while its slices stay above 2,048 tokens and all CTAs run at once.
  const int64_t rows = (int64_t)n_req * layers;
  int n_cta = 1;
  while (n_cta < kEvictMaxCluster && max_len / (2 * n_cta) >= 2048 && rows * n_cta * 2 <= 4 * (int64_t)device_sm_count())
    n_cta *= 2;
  if (rows * n_cta > INT32_MAX) return lora_fail(LORA_EINVAL, "lora_kv_evict: too many (request, layer) rows");
  const int threads = max_len > 4096 ? kEvictMaxThreads : 256;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * n_cta));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kEvictBins * sizeof(int) * (n_cta > 1 ? 1 + kEvictDigits : 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p->prof_on ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = n_cta;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n_cta > 1 ? 2 : 1;
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e = n_cta > 1 ? cudaLaunchKernelEx(&cfg, kv_evict_kernel<true>, a, n_cta)
                                  : cudaLaunchKernelEx(&cfg, kv_evict_kernel<false>, a, n_cta);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_evict launch");
}

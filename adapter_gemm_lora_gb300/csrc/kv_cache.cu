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

constexpr int kEvictThreads = 256;

__device__ __forceinline__ int block_sum(int v, int* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  int s = 0;
  for (int i = 0; i < kEvictThreads / 32; ++i) s += buf[i];
  return s;
}

// One CTA per (layer, request).  The smallest key that stays is found bit by bit; keys above it
// stay, and of the keys equal to it the first few; the kept positions are then numbered by a
// running block scan.
__global__ void __launch_bounds__(kEvictThreads)
kv_evict_kernel(int32_t n_req, const int2* __restrict__ table, const int32_t* __restrict__ seq_len, int32_t max_len,
                int32_t layers, const float* __restrict__ weight, int32_t budget, int32_t recent,
                int32_t* __restrict__ keep, int32_t* __restrict__ new_len, int2* __restrict__ table_out,
                float* __restrict__ weight_out, int32_t max_len_out, int32_t* err) {
  __shared__ int buf[kEvictThreads / 32];
  __shared__ int scan[2][kEvictThreads / 32];
  pdl_wait_then_release();
  const int layer = blockIdx.x % layers, r = blockIdx.x / layers;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = seq_len[r];
  if (n < 0 || n > max_len) {
    if (tid == 0) flag_error(err, LORA_DEV_BAD_SEGMENT);
    n = n < 0 ? 0 : max_len;
  }
  const int n_keep = min(n, budget);
  const int old = n - min(n, recent);          // tokens that compete; the rest stay
  const int need = n_keep - (n - old);         // of them stay
  const float* w = weight + ((int64_t)layer * n_req + r) * max_len;
  uint32_t cut = 0;                            // the need-th largest key
  if (need > 0 && need < old)
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = cut | (1u << bit);
      int c = 0;
      for (int j = tid; j < old; j += kEvictThreads) c += weight_key(w[j]) >= cand;
      if (block_sum(c, buf) >= need) cut = cand;
    }
  int above = 0;
  for (int j = tid; j < old; j += kEvictThreads) above += weight_key(w[j]) > cut;
  above = block_sum(above, buf);
  int ties = need - above;                     // of the keys equal to the cut, the first `ties` stay
  const bool all = need >= old;
  const int64_t row = (int64_t)layer * n_req + r;
  int kept = 0, tied = 0;
  for (int j0 = 0; j0 < n; j0 += kEvictThreads) {
    const int j = j0 + tid;
    float x = 0.f;
    bool gt = false, eq = false;
    if (j < n) {
      x = w[j];
      if (j >= old || all) {
        gt = true;
      } else if (need > 0) {
        const uint32_t key = weight_key(x);
        gt = key > cut;
        eq = key == cut;
      }
    }
    const uint32_t me = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) scan[0][warp] = __popc(me);
    __syncthreads();
    int eq_before = tied, eq_all = 0;
    for (int i = 0; i < kEvictThreads / 32; ++i) {
      if (i < warp) eq_before += scan[0][i];
      eq_all += scan[0][i];
    }
    eq_before += __popc(me & ((1u << lane) - 1));
    const bool stay = gt || (eq && eq_before < ties);
    const uint32_t ms = __ballot_sync(0xffffffffu, stay);
    if (lane == 0) scan[1][warp] = __popc(ms);
    __syncthreads();
    int pos = kept, st_all = 0;
    for (int i = 0; i < kEvictThreads / 32; ++i) {
      if (i < warp) pos += scan[1][i];
      st_all += scan[1][i];
    }
    pos += __popc(ms & ((1u << lane) - 1));
    if (stay) {
      keep[row * budget + pos] = j;
      weight_out[row * max_len_out + pos] = x;
      table_out[((int64_t)r * max_len_out + pos) * layers + layer] = table[((int64_t)r * max_len + j) * layers + layer];
    }
    kept += st_all;
    tied += eq_all;
  }
  for (int i = n_keep + tid; i < budget; i += kEvictThreads) keep[row * budget + i] = -1;
  for (int i = n_keep + tid; i < max_len_out; i += kEvictThreads) {
    weight_out[row * max_len_out + i] = 0.f;
    table_out[((int64_t)r * max_len_out + i) * layers + layer] = make_int2(-1, -1);
  }
  if (layer == 0 && tid == 0) new_len[r] = n_keep;
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
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  ProfScope prof(p, LORA_KIND_KV, st);
  const cudaError_t e =
      launch_pdl(!p->prof_on, kv_evict_kernel, dim3((unsigned)(n_req * layers)), dim3(kEvictThreads), 0, st, n_req,
                 reinterpret_cast<const int2*>(table_dev), seq_len_dev, max_len, layers, weight_dev, budget, recent,
                 keep_dev, new_len_dev, reinterpret_cast<int2*>(table_out), weight_out, max_len_out, p->d_err);
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_kv_evict launch");
}

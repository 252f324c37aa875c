// Paged decode attention split over the cache's length, with the tokens' attention weights.
//
// Per request and query head h (KV head h / G, G = n_heads / n_kv_heads, width D):
//     s_j = q_h . K_j / sqrt(D),  lse = log sum_j exp(s_j),  out_h = sum_j exp(s_j - lse) V_j
//     weight_out[j] = weight_in[j] + sum_h exp(s_{h,j} - lse_h)
// Softmax in base 2: scores carry log2(e) / sqrt(D).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "tc_ptx.h"

namespace {

constexpr int kSplitMaxGroup = 16;     // query heads per KV head

struct SplitArgs {
  const uint16_t* pool;
  int64_t num_pages;
  int32_t H, n_req;
  const int2* table;
  const int32_t* seq_len;
  int32_t max_len, layers, layer;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  int64_t out_stride;
  int32_t n_heads, group;
  float* lse;                          // caller's, nullable, natural log
  const float* weight_in;
  float* weight_out;
  int64_t weight_stride;
  float scale_log2;
  float* ws_lse;                       // [n_req][n_heads], base 2
  float* ws_scores;                    // [n_req][n_heads][max_len rounded up to 16], base 2; NULL without weights
  int64_t score_stride;
  int32_t* err;
};

__device__ __forceinline__ int request_length(const SplitArgs& a, int r, bool report) {
  int n = a.seq_len[r];
  if (n < 0 || n > a.max_len) {
    if (report) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    n = n < 0 ? 0 : a.max_len;
  }
  return n;
}

// One CTA per (query head, request): each of four warps takes every fourth token with its own
// running maximum, sum and accumulator; the four join in shared memory.
template <int D>
__global__ void __launch_bounds__(128) attention_split_kernel(const SplitArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm_m[4], sm_l[4], sm_acc[4][D];
  pdl_wait_then_release();
  const int h = blockIdx.x, r = blockIdx.y, kvh = h / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = request_length(a, r, threadIdx.x == 0);
  float qv[E], acc[E];
  for (int e = 0; e < E; ++e) {
    qv[e] = __uint_as_float((uint32_t)a.q[r * a.q_stride + (int64_t)h * D + lane + 32 * e] << 16);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += 4) {
    const int2 pg = a.table[((int64_t)r * a.max_len + j) * a.layers + a.layer];
    const bool ok = pg.x >= 0 && pg.x < a.num_pages && pg.y >= 0 && pg.y < a.num_pages;
    float s = -INFINITY;
    if (ok) {
      const uint16_t* k = a.pool + (int64_t)pg.x * a.H + kvh * D;
      s = 0.f;
      for (int e = 0; e < E; ++e) s = fmaf(qv[e], __uint_as_float((uint32_t)k[lane + 32 * e] << 16), s);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s);
      if (mn != -INFINITY || s != s) {
        const float c = exp2f(m - mn), p = exp2f(s - mn);
        const uint16_t* v = a.pool + (int64_t)pg.y * a.H + kvh * D;
        l = l * c + p;
        for (int e = 0; e < E; ++e)
          acc[e] = fmaf(p, __uint_as_float((uint32_t)v[lane + 32 * e] << 16), acc[e] * c);
        m = mn;
      }
    } else if (lane == 0) {
      flag_error(a.err, LORA_DEV_BAD_PAGE);
    }
    if (a.ws_scores && lane == 0) a.ws_scores[((int64_t)r * a.n_heads + h) * a.score_stride + j] = s;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) sm_acc[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w]);
  float c[4];
  for (int w = 0; w < 4; ++w) {
    c[w] = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - M);
    L += sm_l[w] * c[w];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w) o += sm_acc[w][d] * c[w];
    a.out[r * a.out_stride + (int64_t)h * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(L != 0.f ? o / L : 0.f));
  }
  if (threadIdx.x == 0) {
    const float lse2 = L != 0.f ? M + log2f(L) : -INFINITY;
    a.ws_lse[(int64_t)r * a.n_heads + h] = lse2;
    if (a.lse) a.lse[(int64_t)r * a.n_heads + h] = lse2 * 0.6931471805599453f;
  }
}

__global__ void __launch_bounds__(256) attention_weights_kernel(const SplitArgs a) {
  pdl_wait_then_release();
  const int r = blockIdx.y, n = request_length(a, r, false);
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= n) return;
  float w = 0.f;
  for (int h = 0; h < a.n_heads; ++h) {
    const float z = a.ws_lse[(int64_t)r * a.n_heads + h];
    if (z != -INFINITY) w += exp2f(a.ws_scores[((int64_t)r * a.n_heads + h) * a.score_stride + j] - z);
  }
  a.weight_out[r * a.weight_stride + j] = (a.weight_in ? a.weight_in[r * a.weight_stride + j] : 0.f) + w;
}

struct SplitLayout {
  size_t lse, scores, total;
  int64_t score_stride;
};

SplitLayout split_layout(int32_t n_req, int32_t max_len, int32_t n_heads, bool weights) {
  SplitLayout L{};
  L.score_stride = ((int64_t)max_len + 15) / 16 * 16;
  size_t off = 0;
  L.lse = off;     off = align256(off + (size_t)n_req * n_heads * 4);
  L.scores = off;  off = align256(off + (weights ? (size_t)n_req * n_heads * L.score_stride * 4 : 0));
  L.total = off;
  return L;
}

// Shape checks shared by the size query and the call; 0 or an error code.
int check_shape(const char* fn, const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads, int32_t n_kv) {
  const std::string f(fn);
  if (!p || n_req < 0 || max_len < 1 || n_heads < 1 || n_kv < 1) return lora_fail(LORA_EINVAL, f + ": bad arguments");
  if (n_req > 65535) return lora_fail(LORA_EINVAL, f + ": at most 65535 requests per call");
  if (n_heads % n_kv != 0 || n_heads / n_kv > kSplitMaxGroup)
    return lora_fail(LORA_EINVAL, f + ": n_heads must be 1 to 16 times n_kv_heads");
  if (p->H % n_kv != 0) return lora_fail(LORA_EINVAL, f + ": H is not a multiple of n_kv_heads");
  const int D = p->H / n_kv;
  if (D != 64 && D != 128 && D != 256) return lora_fail(LORA_EINVAL, f + ": head width must be 64, 128 or 256");
  return LORA_OK;
}

}  // namespace

extern "C" int64_t lora_attention_split_size(const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads,
                                             int32_t n_kv_heads, int32_t with_weights) {
  const int rc = check_shape("lora_attention_split_size", p, n_req, max_len, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_attention_split_size: planning pool has no device state");
  return (int64_t)split_layout(n_req, max_len, n_heads, with_weights != 0).total;
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
  if (((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(weight_in) | reinterpret_cast<uintptr_t>(weight_out)) & 3) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: lse and weights must be 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return lora_fail(LORA_EINVAL, "lora_attention_split: workspace must be 256-byte aligned");
  if (p->planning) return lora_fail(LORA_EINVAL, "lora_attention_split: planning pool has no device state");
  if (n_req == 0) return LORA_OK;
  const SplitLayout L = split_layout(n_req, max_len, n_heads, weight_out != nullptr);
  if (workspace_bytes < (int64_t)L.total)
    return lora_fail(LORA_EINVAL, "lora_attention_split: workspace has " + std::to_string(workspace_bytes) +
                                      " bytes, needs " + std::to_string(L.total));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int D = p->H / n_kv_heads;
  SplitArgs a{};
  a.pool = static_cast<const uint16_t*>(p->pool_dev);
  a.num_pages = p->num_pages;
  a.H = p->H;
  a.n_req = n_req;
  a.table = reinterpret_cast<const int2*>(table_dev);
  a.seq_len = seq_len_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.layer = layer;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.n_heads = n_heads;
  a.group = n_heads / n_kv_heads;
  a.lse = lse;
  a.weight_in = weight_in;
  a.weight_out = weight_out;
  a.weight_stride = weight_stride;
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)D);
  char* ws = static_cast<char*>(workspace);
  a.ws_lse = reinterpret_cast<float*>(ws + L.lse);
  a.ws_scores = weight_out ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  a.score_stride = L.score_stride;
  a.err = p->d_err;
  const dim3 grid(n_heads, n_req);
  cudaError_t e;
  {
    ProfScope prof(p, LORA_KIND_ATTENTION, st);
    if (D == 64) e = launch_pdl(!p->prof_on, attention_split_kernel<64>, grid, dim3(128), 0, st, a);
    else if (D == 128) e = launch_pdl(!p->prof_on, attention_split_kernel<128>, grid, dim3(128), 0, st, a);
    else e = launch_pdl(!p->prof_on, attention_split_kernel<256>, grid, dim3(128), 0, st, a);
  }
  if (e == cudaSuccess && weight_out) {
    ProfScope prof(p, LORA_KIND_ATTENTION, st);
    e = launch_pdl(!p->prof_on, attention_weights_kernel, dim3((unsigned)((max_len + 255) / 256), n_req), dim3(256), 0,
                   st, a);
  }
  return e == cudaSuccess ? LORA_OK : lora_cuda_fail(e, "lora_attention_split launch");
}

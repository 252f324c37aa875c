// Attention of many query rows per sequence: causal over packed prompts, and of trees of drafted tokens
// over the paged KV cache.
//
// Per query head h (KV head h / G, G = n_heads / n_kv_heads, width D) and row i, over the tokens j it sees:
//     s_j = q_{i,h} . k_j / sqrt(D),  lse = log sum_j exp(s_j),  out_{i,h} = sum_j exp(s_j - lse) v_j
// Softmax in base 2: scores carry log2(e) / sqrt(D).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "tc_ptx.h"

namespace {

constexpr int kRowsMaxGroup = 16;                   // query heads per KV head
// Weights are 2^(s - m - kShift), m the largest score: the sums of up to 2^24 weights times V stay within the
// range of V.
constexpr float kShift = 24.f;

struct RowsArgs {
  const uint16_t* q;
  int64_t q_stride;
  const uint16_t* k;                                // prompt: rows; tree: unused
  int64_t k_stride;
  const uint16_t* v;
  int64_t v_stride;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  int32_t n_req, n_rows, n_heads, n_kv;
  const int32_t* start;                             // caller's row starts
  int32_t* bounds;                                  // workspace: the same, ascending within [0, n_rows]
  // tree
  const uint16_t* pool;
  int64_t num_pages;
  int32_t H;
  const int2* table;
  const int32_t* seq_len;
  int32_t max_len, layers, layer;
  const uint64_t* mask;
  float scale_log2;
  int32_t* err;
};

// Row starts as the running maximum of the caller's, clamped into [0, n_rows]: sequences never overlap.
__global__ void __launch_bounds__(1024) rows_bounds_kernel(const RowsArgs a) {
  __shared__ int32_t part[32];
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t before = 0;
  for (int i0 = 0; i0 <= a.n_req; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int32_t x = i <= a.n_req ? a.start[i] : 0;
    int32_t m = x;
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, m, o);
      if (lane >= o) m = max(m, y);
    }
    if (lane == 31) part[warp] = m;
    __syncthreads();
    for (int w = 0; w < warp; ++w) m = max(m, part[w]);
    m = max(m, before);
    int32_t all = before;
    for (int w = 0; w < 32; ++w) all = max(all, part[w]);
    before = all;
    const int32_t b = min(max(m, 0), a.n_rows);
    if (i <= a.n_req) {
      if (b != x) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
      a.bounds[i] = b;
    }
    __syncthreads();
  }
}

// One warp per (row, query head), a running maximum and sum over the tokens one by one.
template <int D, bool kTree>
__global__ void __launch_bounds__(128) rows_simple_kernel(const RowsArgs a) {
  constexpr int E = D / 32;
  pdl_wait_then_release();
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t row = item / a.n_heads;
  const int h = (int)(item % a.n_heads), kvh = h / (a.n_heads / a.n_kv);
  if (row >= a.n_rows) return;
  int lo = 0, hi = a.n_req;                         // the request whose rows hold this one: bounds[lo] <= row < bounds[lo + 1]
  if (row < a.bounds[0] || row >= a.bounds[a.n_req]) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.bounds[mid] <= row) lo = mid; else hi = mid;
  }
  const int first = a.bounds[lo], node = (int)row - first;
  int n = node + 1, base = 0;
  uint64_t mask = ~0ull;
  if (kTree) {
    const int raw = a.seq_len[lo], len = min(max(raw, 0), a.max_len), m = a.bounds[lo + 1] - first;
    if (raw != len || m > LORA_MAX_TREE || m > len) {
      if (lane == 0) flag_error(a.err, LORA_DEV_BAD_SEGMENT);
    }
    if (node >= LORA_MAX_TREE) return;
    n = len;
    base = max(len - min(m, LORA_MAX_TREE), 0);
    mask = a.mask[row];
  }
  float q[E], acc[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.q[row * a.q_stride + (int64_t)h * D + e * 32 + lane] << 16);
    acc[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const uint16_t *k, *v;
    if (kTree) {
      const int2 pg = a.table[((int64_t)lo * a.max_len + j) * a.layers + a.layer];
      if (pg.x < 0 || pg.x >= a.num_pages || pg.y < 0 || pg.y >= a.num_pages) {
        if (lane == 0) flag_error(a.err, LORA_DEV_BAD_PAGE);
        continue;
      }
      if (j >= base && !((mask >> (j - base)) & 1)) continue;
      k = a.pool + (int64_t)pg.x * a.H + kvh * D;
      v = a.pool + (int64_t)pg.y * a.H + kvh * D;
    } else {
      k = a.k + (first + j) * a.k_stride + kvh * D;
      v = a.v + (first + j) * a.v_stride + kvh * D;
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], __uint_as_float((uint32_t)k[e * 32 + lane] << 16), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn, c = m == mn ? 1.f : exp2f(m - ms), p = exp2f(s - ms - kShift);
    m = mn;
    l = l * c + p;
    for (int e = 0; e < E; ++e) {
      const float x = __uint_as_float((uint32_t)v[e * 32 + lane] << 16);
      acc[e] = (c == 1.f ? acc[e] : acc[e] * c) + (p == 0.f ? 0.f : p * x);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int e = 0; e < E; ++e) a.out[row * a.out_stride + (int64_t)h * D + e * 32 + lane] = f32_to_bf16_rn(acc[e] * inv);
  if (a.lse && lane == 0) a.lse[row * a.n_heads + h] = l == 0.f ? -INFINITY : (m + kShift + log2f(l)) * 0.6931471805599453f;
}

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

int64_t prompt_bytes(int32_t n_seq) { return (int64_t)align256(((size_t)n_seq + 1) * 4); }
int64_t tree_bytes(int32_t n_req) { return (int64_t)align256(((size_t)n_req + 1) * 4); }

template <bool kTree>
int launch_rows(const lora_pool* p, const RowsArgs& a, const char* what, cudaStream_t st) {
  const int D = p->H / a.n_kv;
  cudaError_t e;
  {
    ProfScope prof(p, LORA_KIND_ATTENTION, st);
    e = launch_pdl(!p->prof_on, rows_bounds_kernel, dim3(1), dim3(1024), 0, st, a);
  }
  if (e != cudaSuccess) return lora_cuda_fail(e, what);
  ProfScope prof(p, LORA_KIND_ATTENTION, st);
  const dim3 grid((unsigned)(((int64_t)a.n_rows * a.n_heads + 3) / 4));
  e = D == 64    ? launch_pdl(!p->prof_on, rows_simple_kernel<64, kTree>, grid, dim3(128), 0, st, a)
      : D == 128 ? launch_pdl(!p->prof_on, rows_simple_kernel<128, kTree>, grid, dim3(128), 0, st, a)
                 : launch_pdl(!p->prof_on, rows_simple_kernel<256, kTree>, grid, dim3(128), 0, st, a);
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
  return prompt_bytes(n_seq);
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
  rc = check_workspace(fn, workspace, some ? workspace_bytes : prompt_bytes(n_seq), prompt_bytes(n_seq));
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, fn + ": planning pool has no device state");
  if (!some) return LORA_OK;
  RowsArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.k = static_cast<const uint16_t*>(k);
  a.k_stride = k_stride;
  a.v = static_cast<const uint16_t*>(v);
  a.v_stride = v_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.n_req = n_seq;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.n_kv = n_kv_heads;
  a.start = seq_start;
  a.bounds = static_cast<int32_t*>(workspace);
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)(p->H / n_kv_heads));
  a.err = p->d_err;
  return launch_rows<false>(p, a, "lora_attention_prompt launch", reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int64_t lora_attention_tree_size(const lora_pool* p, int32_t n_req, int32_t max_len, int32_t n_heads,
                                            int32_t n_kv_heads) {
  const std::string fn = "lora_attention_tree_size";
  const int rc = check_heads(fn, p, n_req, n_heads, n_kv_heads);
  if (rc != LORA_OK) return rc;
  if (max_len < 1 || max_len > (1 << 30)) return lora_fail(LORA_EINVAL, fn + ": max_len must lie in [1, 2^30]");
  return tree_bytes(n_req);
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
  rc = check_workspace(fn, workspace, some ? workspace_bytes : tree_bytes(n_req), tree_bytes(n_req));
  if (rc != LORA_OK) return rc;
  if (p->planning) return lora_fail(LORA_EINVAL, fn + ": planning pool has no device state");
  if (!some) return LORA_OK;
  RowsArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.n_req = n_req;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.n_kv = n_kv_heads;
  a.start = node_start;
  a.bounds = static_cast<int32_t*>(workspace);
  a.pool = static_cast<const uint16_t*>(p->pool_dev);
  a.num_pages = p->num_pages;
  a.H = p->H;
  a.table = reinterpret_cast<const int2*>(table_dev);
  a.seq_len = seq_len_dev;
  a.max_len = max_len;
  a.layers = layers;
  a.layer = layer;
  a.mask = mask;
  a.scale_log2 = 1.4426950408889634f / std::sqrt((float)(p->H / n_kv_heads));
  a.err = p->d_err;
  return launch_rows<true>(p, a, "lora_attention_tree launch", reinterpret_cast<cudaStream_t>(stream));
}

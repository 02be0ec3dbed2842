// Attention of a chunk of new tokens over a paged cache
// (ws_paged_attention in include/ws.h gives the formulas).
#include "ws_paged.cuh"

namespace {

struct AttnP {
  ws_paged_cache c;
  ws_attention_args a;
  int G;                                   // query heads per KV head
};

struct Req {
  int slot, row0, c, L;                    // cache slot, first row, chunk length, visible positions
};
__device__ __forceinline__ Req request(const AttnP& p, int i) {
  Req r;
  r.slot = p.a.req_ids ? p.a.req_ids[i] : i;
  r.row0 = p.a.cu_q[i];
  const int end = min(p.a.cu_q[i + 1], p.a.total_q);
  r.c = r.row0 >= 0 ? min(max(end - r.row0, 0), p.a.max_q) : 0;
  r.L = 0;
  if (r.slot >= 0 && r.slot < p.c.n_slots)
    r.L = (int)min((long long)min(max(p.a.kv_len[r.slot], 0), p.a.max_kv), (long long)p.c.table_stride * p.c.page_size);
  return r;
}
// Positions 0 .. limit - 1 are visible to row t of the chunk.
__device__ __forceinline__ int row_limit(const AttnP& p, const Req& r, int t) {
  return p.a.causal ? max(0, min(r.L, r.L - r.c + t + 1)) : r.L;
}

// One warp per (row, query head), two dims per lane.
template <typename T>
__global__ void simple_attn(const AttnP p) {
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.y, u = blockIdx.z, t = warp;
  const Req r = request(p, i);
  if (t >= r.c) return;
  const int row = r.row0 + t, lim = row_limit(p, r, t), h = u / p.G;
  const T* q = (const T*)p.a.q + (size_t)row * p.a.q_stride + (size_t)u * WS_DH;
  const float q0 = to_f(q[lane]), q1 = to_f(q[lane + 32]);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int j = 0; j < lim; ++j) {
    const int page = paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, j);
    if (page < 0) continue;
    const size_t off = paged_off(p.c, page, h, j);
    const T *k = (const T*)p.c.k + off, *v = (const T*)p.c.v + off;
    float s = q0 * to_f(k[lane]) + q1 * to_f(k[lane + 32]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.a.scale;
    const float mn = fmaxf(m, s), f = m == mn ? 1.f : expf(m - mn), e = s == mn ? 1.f : expf(s - mn);
    l = l * f + e; o0 = o0 * f + e * to_f(v[lane]); o1 = o1 * f + e * to_f(v[lane + 32]);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* out = (T*)p.a.out + (size_t)row * p.a.out_stride + (size_t)u * WS_DH;
  out[lane] = from_f<T>(o0 * inv);
  out[lane + 32] = from_f<T>(o1 * inv);
  if (p.a.lse && lane == 0) p.a.lse[(size_t)row * p.a.n_heads + u] = l > 0.f ? m + logf(l) : -INFINITY;
}

// One warp per (slot, KV head, position): the weights of every row and head.
template <typename T>
__global__ void simple_mass(const AttnP p, const float* lse) {
  const int j = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.y, h = blockIdx.z;
  const Req r = request(p, i);
  if (j >= r.L) return;
  const int page = paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, j);
  if (page < 0) return;
  const T* k = (const T*)p.c.k + paged_off(p.c, page, h, j);
  const float k0 = to_f(k[lane]), k1 = to_f(k[lane + 32]);
  float sum = 0.f;
  for (int t = 0; t < r.c; ++t) {
    if (j >= row_limit(p, r, t)) continue;
    for (int g = 0; g < p.G; ++g) {
      const int u = h * p.G + g;
      const T* q = (const T*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride + (size_t)u * WS_DH;
      float s = to_f(q[lane]) * k0 + to_f(q[lane + 32]) * k1;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      sum += expf(s * p.a.scale - lse[(size_t)(r.row0 + t) * p.a.n_heads + u]);
    }
  }
  if (lane == 0) p.a.mass[((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride + j] += sum;
}

const char* check_attn(const ws_paged_cache* c, const ws_attention_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0 || a->n_req > 65535) return "n_req must be 0..65535";
  if (a->total_q < 0 || a->max_q < 0 || a->max_kv < 0) return "negative size";
  if (a->n_heads < 1 || a->n_heads % c->n_kv_heads || a->n_heads > 65535)
    return "n_heads must be a multiple of n_kv_heads, at most 65535";
  if (a->causal != 0 && a->causal != 1) return "causal must be 0 or 1";
  if (!isfinite(a->scale)) return "scale must be finite";
  if (a->n_req == 0 || a->total_q == 0) return nullptr;
  if (!a->kv_len || !a->cu_q || !a->q || !a->out) return "null kv_len, cu_q, q or out";
  const int64_t unit = c->dtype == WS_BF16 ? 8 : 4;
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) & 15 || a->q_stride % unit ||
      a->out_stride % unit)
    return "rows of q and out must be 16-byte aligned";
  if (a->q_stride < (int64_t)a->n_heads * WS_DH || a->out_stride < (int64_t)a->n_heads * WS_DH)
    return "q_stride and out_stride must be >= 64 * n_heads";
  if (a->mass && a->mass_stride < a->max_kv) return "mass_stride must be >= max_kv";
  if (!a->req_ids && a->n_req > c->n_slots) return "more requests than slots";
  return nullptr;
}

template <typename T>
cudaError_t run_simple(const AttnP& p, float* lse, cudaStream_t s) {
  AttnP q = p;
  q.a.lse = lse;
  if (p.a.max_q > 0)
    simple_attn<T><<<dim3((p.a.max_q + 3) / 4, p.a.n_req, p.a.n_heads), 128, 0, s>>>(q);
  if (p.a.mass && p.a.max_kv > 0)
    simple_mass<T><<<dim3((p.a.max_kv + 3) / 4, p.a.n_req, p.c.n_kv_heads), 128, 0, s>>>(q, lse);
  ws_count_launches(2);
  return cudaGetLastError();
}

}  // namespace

extern "C" size_t ws_paged_attention_workspace(const ws_paged_cache* cache, const ws_attention_args* args) {
  if (check_attn(cache, args)) return 0;
  return args->mass && !args->lse ? (size_t)args->total_q * args->n_heads * 4 : 0;
}

extern "C" int ws_paged_attention(const ws_paged_cache* cache, const ws_attention_args* args, void* workspace,
                                  size_t workspace_bytes, ws_stream stream) {
  if (const char* e = check_attn(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0 || args->total_q == 0 || args->max_q == 0) return WS_OK;
  const size_t need = ws_paged_attention_workspace(cache, args);
  if (need && !workspace) return paged_fail(WS_EINVAL, "null workspace");
  if (need > workspace_bytes) return paged_fail(WS_ENOSPACE, "workspace smaller than ws_paged_attention_workspace()");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  AttnP p;
  p.c = *cache;
  p.a = *args;
  p.G = args->n_heads / cache->n_kv_heads;
  float* lse = args->lse ? args->lse : (float*)workspace;
  const cudaError_t e = cache->dtype == WS_BF16 ? run_simple<bf16>(p, lse, (cudaStream_t)stream)
                                                : run_simple<float>(p, lse, (cudaStream_t)stream);
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

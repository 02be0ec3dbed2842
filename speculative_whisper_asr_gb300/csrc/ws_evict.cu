// Eviction from a paged cache by accumulated attention weight
// (ws_cache_evict in include/ws.h gives the rule).
#include "ws_paged.cuh"

namespace {

struct EvictP {
  ws_paged_cache c;
  ws_evict_args a;
  const int32_t* tout;
  int tout_stride;
  int in_place;
  int32_t* idx;                            // [n_req][heads][keep] kept positions, ascending
  int32_t* len;                            // [n_req] kv_len before the call
};

constexpr int NT = 1024;

// Order of a position: protected first, then the mass as an unsigned integer
// (masses are >= 0 here, so their bits are ordered).
__device__ __forceinline__ uint32_t evict_key(const EvictP& p, const float* mass, int L, int j) {
  if (j < p.a.sink || j >= L - p.a.recent) return 0xFFFFFFFFu;
  return __float_as_uint(fmaxf(mass[j], 0.f)) & 0x7FFFFFFFu;
}

// One CTA per (request, head): the kept positions.
__global__ void __launch_bounds__(NT) evict_select(const EvictP p) {
  __shared__ int hist[256];
  __shared__ int s_warp[NT / 32];
  __shared__ int s_prefix, s_need;
  const int i = blockIdx.x, h = blockIdx.y, H = p.c.n_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  int L = 0;
  if (slot >= 0 && slot < p.c.n_slots)
    L = (int)min((long long)min(max(p.a.kv_len[slot], 0), p.a.max_kv), (long long)p.c.table_stride * p.c.page_size);
  if (h == 0 && tid == 0) p.len[i] = L;
  const int keep = min(L, p.a.keep);
  int32_t* idx = p.idx + ((size_t)i * H + h) * p.a.keep;
  if (keep == L) {
    for (int j = tid; j < L; j += NT) idx[j] = j;
    return;
  }
  const float* mass = p.a.mass + ((size_t)slot * H + h) * p.a.mass_stride;
  // the keep-th largest key, 8 bits at a time
  uint32_t prefix = 0;
  int need = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int b = tid; b < 256; b += NT) hist[b] = 0;
    __syncthreads();
    for (int j = tid; j < L; j += NT) {
      const uint32_t k = evict_key(p, mass, L, j);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int b = 255, left = need;
      for (; b > 0 && hist[b] < left; --b) left -= hist[b];
      s_prefix = (int)(prefix | ((uint32_t)b << shift));
      s_need = left;
    }
    __syncthreads();
    prefix = (uint32_t)s_prefix;
    need = s_need;
    __syncthreads();
  }
  // positions above the threshold, and the first `need` that equal it
  int base = 0, eq_base = 0;
  for (int j0 = 0; j0 < L; j0 += NT) {
    const int j = j0 + tid;
    const uint32_t k = j < L ? evict_key(p, mass, L, j) : 0u;
    const bool eq = j < L && k == prefix;
    const unsigned be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[warp] = __popc(be);
    __syncthreads();
    int before = eq_base, all = 0;
    for (int w = 0; w < NT / 32; ++w) { if (w < warp) before += s_warp[w]; all += s_warp[w]; }
    before += __popc(be & ((1u << lane) - 1u));
    eq_base += all;
    __syncthreads();
    const bool on = j < L && (k > prefix || (eq && before < need));
    const unsigned bo = __ballot_sync(0xffffffffu, on);
    if (lane == 0) s_warp[warp] = __popc(bo);
    __syncthreads();
    int at = base;
    all = 0;
    for (int w = 0; w < NT / 32; ++w) { if (w < warp) at += s_warp[w]; all += s_warp[w]; }
    at += __popc(bo & ((1u << lane) - 1u));
    if (on) idx[at] = j;
    base += all;
    __syncthreads();
  }
}

// One CTA per (request, head); in order, so that a place is read before
// anything is written over it.
template <typename T>
__global__ void __launch_bounds__(NT) evict_move(const EvictP p) {
  const int i = blockIdx.x, h = blockIdx.y, H = p.c.n_kv_heads;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  const int L = p.len[i], keep = min(L, p.a.keep);
  if (slot < 0 || slot >= p.c.n_slots) return;
  if (h == 0 && threadIdx.x == 0) p.a.kv_len_out[slot] = keep;
  const int32_t* idx = p.idx + ((size_t)i * H + h) * p.a.keep;
  constexpr int V = WS_DH * sizeof(T) / 16;     // 16-byte pieces of a row
  const int sub = threadIdx.x % V, r = threadIdx.x / V;
  const float* mass = p.a.mass + ((size_t)slot * H + h) * p.a.mass_stride;
  for (int j0 = 0; j0 < keep; j0 += NT / V) {
    const int j = j0 + r;
    const int src = j < keep ? idx[j] : 0;
    const int ps = j < keep ? paged_page(p.c, p.c.page_table, p.c.table_stride, slot, src) : -1;
    const int pd = j < keep ? paged_page(p.c, p.tout, p.tout_stride, slot, j) : -1;
    uint4 k, v;
    float m = 0.f;
    int pos = 0;
    const bool go = ps >= 0 && pd >= 0;
    if (go) {
      k = reinterpret_cast<const uint4*>((const T*)p.c.k + paged_off(p.c, ps, h, src))[sub];
      v = reinterpret_cast<const uint4*>((const T*)p.c.v + paged_off(p.c, ps, h, src))[sub];
    }
    if (j < keep && sub == 0) {
      m = mass[src];
      pos = p.a.pos ? p.a.pos[((size_t)slot * H + h) * p.a.pos_stride + src] : src;
    }
    __syncthreads();
    if (go) {
      reinterpret_cast<uint4*>((T*)p.c.k + paged_off(p.c, pd, h, j))[sub] = k;
      reinterpret_cast<uint4*>((T*)p.c.v + paged_off(p.c, pd, h, j))[sub] = v;
    }
    if (j < keep && sub == 0) {
      if (p.a.mass_out) p.a.mass_out[((size_t)slot * H + h) * p.a.mass_out_stride + j] = m;
      if (p.a.pos_out) p.a.pos_out[((size_t)slot * H + h) * p.a.pos_out_stride + j] = pos;
    }
    __syncthreads();
  }
}

const char* check_evict(const ws_paged_cache* c, const ws_evict_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0) return "n_req must be >= 0";
  if (a->max_kv < 1 || a->keep < 1 || a->keep > a->max_kv) return "keep must be 1..max_kv";
  if (a->sink < 0 || a->recent < 0 || (long long)a->sink + a->recent > a->keep)
    return "sink and recent must be >= 0 and sink + recent <= keep";
  if (a->n_req == 0) return nullptr;
  if (!a->kv_len || !a->kv_len_out || !a->mass) return "null kv_len, kv_len_out or mass";
  if (a->mass_stride < a->max_kv) return "mass_stride must be >= max_kv";
  if (a->mass_out && a->mass_out_stride < a->keep) return "mass_out_stride must be >= keep";
  if (a->mass_out == a->mass && a->mass_out_stride != a->mass_stride) return "in place, the mass strides must be equal";
  if (a->pos && a->pos_stride < a->max_kv) return "pos_stride must be >= max_kv";
  if (a->pos_out && a->pos_out_stride < a->keep) return "pos_out_stride must be >= keep";
  if (a->pos_out && a->pos_out == a->pos && a->pos_out_stride != a->pos_stride)
    return "in place, the pos strides must be equal";
  const bool in_place = !a->page_table_out || a->page_table_out == c->page_table;
  if (!in_place && a->table_out_stride < 1) return "table_out_stride must be >= 1";
  if (!in_place && (long long)a->table_out_stride * c->page_size < a->keep)
    return "page_table_out lists fewer than keep positions";
  if (!a->req_ids && a->n_req > c->n_slots) return "more requests than slots";
  return nullptr;
}

size_t evict_bytes(const ws_paged_cache* c, const ws_evict_args* a) {
  return (((size_t)a->n_req * 4 + 255) / 256 + ((size_t)a->n_req * c->n_kv_heads * a->keep * 4 + 255) / 256) * 256;
}

}  // namespace

extern "C" size_t ws_cache_evict_workspace(const ws_paged_cache* cache, const ws_evict_args* args) {
  if (check_evict(cache, args) || args->n_req == 0) return 0;
  return evict_bytes(cache, args);
}

extern "C" int ws_cache_evict(const ws_paged_cache* cache, const ws_evict_args* args, void* workspace,
                              size_t workspace_bytes, ws_stream stream) {
  if (const char* e = check_evict(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0) return WS_OK;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return paged_fail(WS_EINVAL, "workspace must be 16-byte aligned and not null");
  if (evict_bytes(cache, args) > workspace_bytes)
    return paged_fail(WS_ENOSPACE, "workspace smaller than ws_cache_evict_workspace()");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  EvictP p;
  p.c = *cache;
  p.a = *args;
  p.in_place = !args->page_table_out || args->page_table_out == cache->page_table;
  p.tout = p.in_place ? cache->page_table : args->page_table_out;
  p.tout_stride = p.in_place ? cache->table_stride : args->table_out_stride;
  p.len = (int32_t*)workspace;
  p.idx = (int32_t*)((char*)workspace + ((size_t)args->n_req * 4 + 255) / 256 * 256);
  cudaStream_t s = (cudaStream_t)stream;
  const dim3 grid(args->n_req, cache->n_kv_heads);
  evict_select<<<grid, NT, 0, s>>>(p);
  if (cache->dtype == WS_BF16) evict_move<bf16><<<grid, NT, 0, s>>>(p);
  else evict_move<float><<<grid, NT, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("cache eviction launch: ") + cudaGetErrorString(e));
  ws_count_launches(2);
  return WS_OK;
}

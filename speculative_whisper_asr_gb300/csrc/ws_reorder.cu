// Reordering the paged caches of beams by their parents (ws_cache_reorder in
// include/ws.h).  Full pages change hands in the page table; of the page that
// is being filled, the parent's tokens are copied.  Parents form no order (two
// beams may exchange places), and the copy is in place: a thread owns 16
// bytes of one token for all beams of a request, reads what each beam
// receives and then writes, so nothing needs a buffer or a second launch.
#include <string>

#include "ws_paged.cuh"

namespace {

constexpr int RO_NT = 128;
constexpr int RO_BEAMS = 16;

struct ReorderP {
  ws_paged_cache c;
  ws_reorder_args a;
  int ppr_log;                             // log2 of the 16-byte pieces of a token's keys or values
};

// NB: beams at most.
template <int NB>
__global__ void __launch_bounds__(RO_NT) reorder_kernel(const ReorderP p) {
  __shared__ int s_page[RO_BEAMS], s_slot[RO_BEAMS], s_par[RO_BEAMS], s_any;
  const int tid = threadIdx.x, i = blockIdx.y, B = p.a.beams;
  if (tid == 0) s_any = 0;
  __syncthreads();
  // the request's length is its first beam's; a beam of a bad slot stays out of it
  const int slot0 = p.a.req_ids ? p.a.req_ids[(size_t)i * B] : i * B;
  const int L = slot0 >= 0 && slot0 < p.c.n_slots ? max(p.a.kv_len[slot0], 0) : 0;
  const int full = min(L / p.c.page_size, p.c.table_stride), rest = full < p.c.table_stride ? L % p.c.page_size : 0;
  if (tid < B) {
    const int slot = p.a.req_ids ? p.a.req_ids[(size_t)i * B + tid] : i * B + tid;
    const bool ok = slot >= 0 && slot < p.c.n_slots;
    int par = p.a.parent[(size_t)i * B + tid];
    if (par < 0 || par >= B) par = tid;
    s_slot[tid] = ok ? slot : -1;
    s_page[tid] = ok && rest ? paged_page(p.c, p.c.page_table, p.c.table_stride, slot, full * p.c.page_size) : -1;
    s_par[tid] = par;
    if (par != tid) s_any = 1;
  }
  __syncthreads();
  if (!s_any) return;
  const int heads = p.c.n_kv_heads, lane0 = blockIdx.x * RO_NT + tid, step = gridDim.x * RO_NT;
  const int es = p.c.dtype == WS_F32 ? 4 : p.c.dtype == WS_BF16 ? 2 : 1;
  auto moves = [&](int b) { return b < B && s_par[b] != b && s_page[b] >= 0 && s_page[s_par[b]] >= 0; };
  // 16-byte pieces, head by head of keys and of values
  const long long per = (long long)rest << p.ppr_log, all = 2 * heads * per;
  for (long long x = lane0; x < all; x += step) {
    const int row = per == (int)per && all < (1ll << 31) ? (int)((uint32_t)x / (uint32_t)per) : (int)(x / per), y = (int)(x - row * per);
    const bool v = row >= heads;
    char* base = (char*)(v ? p.c.v : p.c.k) + ((size_t)(v ? row - heads : row) * (size_t)p.c.head_stride +
                                               (size_t)(y >> p.ppr_log) * (size_t)p.c.token_stride) * es +
                 (size_t)(y & ((1 << p.ppr_log) - 1)) * 16;
    uint4 r[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (moves(b)) r[b] = *reinterpret_cast<const uint4*>(base + (size_t)s_page[s_par[b]] * (size_t)p.c.page_stride * es);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (moves(b)) *reinterpret_cast<uint4*>(base + (size_t)s_page[b] * (size_t)p.c.page_stride * es) = r[b];
  }
  if (p.c.dtype == WS_E4M3) {
    const int blocks = (rest + p.c.scale_block - 1) / p.c.scale_block;
    for (long long x = lane0; x < 2ll * heads * blocks; x += step) {
      const int row = (int)(x / blocks);
      const bool v = row >= heads;
      uint8_t* sc = (v ? p.c.v_scale : p.c.k_scale) + (size_t)(v ? row - heads : row) * (size_t)p.c.scale_head_stride + (x - (long long)row * blocks);
      uint8_t r[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (moves(b)) r[b] = sc[(size_t)s_page[s_par[b]] * (size_t)p.c.scale_page_stride];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (moves(b)) sc[(size_t)s_page[b] * (size_t)p.c.scale_page_stride] = r[b];
    }
  }
  if (!p.a.page_table) return;
  // ---- the page table's rows, as far as pages are full
  for (int x = lane0; x < full; x += step) {
    int r[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b < B && s_slot[s_par[b]] >= 0) r[b] = p.a.page_table[(size_t)s_slot[s_par[b]] * p.c.table_stride + x];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b < B && s_par[b] != b && s_slot[b] >= 0 && s_slot[s_par[b]] >= 0)
        p.a.page_table[(size_t)s_slot[b] * p.c.table_stride + x] = r[b];
  }
}

const char* check_reorder(const ws_paged_cache* c, const ws_reorder_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0 || a->n_req > 65535) return "n_req must be 0..65535";
  if (a->beams < 1 || a->beams > RO_BEAMS) return "beams must be 1..16";
  if (c->page_size > 1 << 26) return "page_size must be at most 2^26";
  if (a->n_req == 0) return nullptr;
  if (!a->kv_len || !a->parent) return "null kv_len or parent";
  if (a->page_table && a->page_table != c->page_table) return "page_table must be the cache's own, or null";
  if (!a->req_ids && (long long)a->n_req * a->beams > c->n_slots) return "more beams than slots";
  return nullptr;
}

template <int NB>
void launch(const ReorderP& p, dim3 grid, cudaStream_t s) {
  reorder_kernel<NB><<<grid, RO_NT, 0, s>>>(p);
  ws_count_launches(1);
}

}  // namespace

extern "C" int ws_cache_reorder(const ws_paged_cache* cache, const ws_reorder_args* args, ws_stream stream) {
  if (const char* e = check_reorder(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0 || args->beams == 1) return WS_OK;
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  ReorderP p = {};
  p.c = paged_copy(*cache);
  p.a = *args;
  p.ppr_log = cache->dtype == WS_F32 ? 4 : cache->dtype == WS_BF16 ? 3 : 2;
  // 32 CTAs per SM in all, each with as much of a request as comes out: a CTA's
  // look at lengths, parents and pages is a chain of latencies (a CTA per head:
  // 96 requests x 5 beams x 80 heads 93 us, in this form 45).  At 46 / 65 / 131
  // registers (4 / 8 / 16 beams) 10 / 7 / 3 of them run on an SM at a time; two
  // rounds of those take 46 us for the 45, 59 for 57 (40 x 12 beams x 80 heads)
  // and 35 for 38 (96 x 12 x 20 heads), 64 per SM 48, 67 and 46.
  const long long pieces = ((long long)cache->page_size << p.ppr_log) * 2 * cache->n_kv_heads;
  const dim3 grid((unsigned)min((pieces + RO_NT - 1) / RO_NT, max(1ll, 32ll * SMS / args->n_req)), (unsigned)args->n_req);
  const cudaStream_t s = (cudaStream_t)stream;
  if (args->beams <= 4) launch<4>(p, grid, s);
  else if (args->beams <= 8) launch<8>(p, grid, s);
  else launch<16>(p, grid, s);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("cache reorder launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

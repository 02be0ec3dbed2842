// Eviction from a paged cache by accumulated attention weight
// (ws_cache_evict in include/ws.h gives the rule).
//
// evict_select finds, per (request, KV head), the keep-th largest key by four
// 8-bit histogram passes over keys held in shared memory, then writes the
// kept positions in ascending order.  A cluster of up to 8 CTAs shares a
// (request, head), so that few long caches still fill the machine: the
// histograms and counts meet through distributed shared memory.  All counts
// are integers, so their order does not matter.
//
// evict_move copies the kept rows.  Its floor is HBM: every kept key and value
// is read and written once.  To fresh pages, all rows move at once.
//
// evict_compact moves them in place.  A destination is never behind its
// source, so a CTA goes through the rows in order, a batch read before the
// batch is written; the parallelism comes from cutting the rows into parts,
// which never mix.
//
// 96 requests x 20 heads, up to 1500 positions cut to 512 (514 MB): selection
// 19 us, move 82 us (6.1 TB/s), in place 95; 8 requests x 8 heads, up to
// 65,536 cut to 16,384 (560 MB): 25 and 89 us, in place 120.  Selecting inside
// the moving kernel took 136 and 250 us: a CTA's histogram passes leave the
// memory idle.
#include "ws_paged.cuh"

namespace {

struct EvictP {
  ws_paged_cache c;
  ws_evict_args a;
  const int32_t* tout;
  int tout_stride;
  int32_t* idx;                            // [n_req][heads][keep] kept positions, ascending
  int32_t* len;                            // [n_req] kv_len before the call
  int cs;                                  // CTAs per (request, head) in evict_select
  int cached;                              // keys kept in shared memory per CTA (0: read again each pass)
  int ordered;                             // masses or labels move in place: one CTA takes a slot and head's in order
};

constexpr int MAX_CS = 8;

// Order of a position: protected first, then the mass as an unsigned integer
// (masses are >= 0 here, so their bits are ordered).
__device__ __forceinline__ uint32_t evict_key(const EvictP& p, const float* mass, int L, int j) {
  if (j < p.a.sink || j >= L - p.a.recent) return 0xFFFFFFFFu;
  return __float_as_uint(fmaxf(mass[j], 0.f)) & 0x7FFFFFFFu;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int remote_int(const int* local, uint32_t rank) {
  uint32_t addr;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Sum over the cluster's CTAs: all loads are in flight together (a loop that
// adds one at a time waits a round trip for each: 80 of the 84 us that 8
// caches of 65,536 positions took).
__device__ __forceinline__ int cluster_total(const int* local, int cs) {
  int v[MAX_CS];
#pragma unroll
  for (int r = 0; r < MAX_CS; ++r) v[r] = r < cs ? remote_int(local, (uint32_t)r) : 0;
  int s = 0;
#pragma unroll
  for (int r = 0; r < MAX_CS; ++r) s += v[r];
  return s;
}

// grid (cs, heads, requests), cluster (cs, 1, 1)
template <int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 6 : 2) evict_select(const EvictP p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) int hist[2][256];
  __shared__ __align__(16) int total[256];
  __shared__ int counts[2];                // keys of this CTA above the threshold, and equal to it
  __shared__ int wgt[NT / 32], weq[NT / 32];
  __shared__ int s_bin, s_left;
  pdl_trigger();
  const int i = blockIdx.z, h = blockIdx.y, H = p.c.n_kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cs = p.cs;
  const uint32_t rank = cs > 1 ? cluster_rank() : 0u;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  int L = 0;
  if (slot >= 0 && slot < p.c.n_slots)
    L = (int)min((long long)min(max(p.a.kv_len[slot], 0), p.a.max_kv), (long long)p.c.table_stride * p.c.page_size);
  if (h == 0 && rank == 0 && tid == 0) p.len[i] = L;
  const int keep = min(L, p.a.keep);
  int32_t* idx = p.idx + ((size_t)i * H + h) * p.a.keep;
  if (keep == L) {                         // the whole cluster leaves
    for (int j = rank * NT + tid; j < L; j += cs * NT) idx[j] = j;
    return;
  }
  const float* mass = p.a.mass + ((size_t)slot * H + h) * p.a.mass_stride;
  // this CTA's positions, and each warp's part of them (whole steps of 32)
  const int seg = (L + cs - 1) / cs, lo = min(L, (int)rank * seg), hi = min(L, lo + seg), n = hi - lo;
  const bool cached = p.cached > 0;
  auto key = [&](int x) { return cached ? keys[x] : evict_key(p, mass, L, lo + x); };
  if (cached) {
#pragma unroll 4
    for (int x = tid; x < n; x += NT) keys[x] = evict_key(p, mass, L, lo + x);
  }
  for (int b = tid; b < 512; b += NT) hist[b >> 8][b & 255] = 0;
  __syncthreads();
  // ---- the keep-th largest key, 8 bits at a time
  uint32_t prefix = 0;
  int need = keep;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass, buf = pass & 1;
#pragma unroll 4
    for (int x = tid; x < n; x += NT) {
      const uint32_t k = key(x);
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[buf][(k >> shift) & 255], 1);
    }
    if (cs > 1) cluster_sync(); else __syncthreads();
    if (cs > 1) {
      if (tid < 256) total[tid] = cluster_total(&hist[buf][tid], cs);
      __syncthreads();
    }
    // warp 0 takes the bins from the top: lane x bins 255 - 8 x .. 248 - 8 x
    if (warp == 0) {
      const int4* bins = reinterpret_cast<const int4*>((cs > 1 ? total : hist[buf]) + 8 * (31 - lane));
      const int4 low = bins[0], high = bins[1];
      const int c[8] = {high.w, high.z, high.y, high.x, low.w, low.z, low.y, low.x};
      const int sum = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
      int incl = sum;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
      }
      int before = incl - sum;
      if (before < need && incl >= need) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (before < need && before + c[q] >= need) { s_bin = 255 - 8 * lane - q; s_left = need - before; }
          before += c[q];
        }
      }
    }
    for (int b = tid; b < 256; b += NT) hist[buf ^ 1][b] = 0;   // read by nobody since the last barrier
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    need = s_left;
    if (cs > 1) cluster_sync(); else __syncthreads();           // the histograms are read everywhere
  }
  // ---- keys above the threshold, and the first `need` that equal it, in order
  const int wlen = (((n + NT / 32 - 1) / (NT / 32)) + 31) & ~31;
  const int wb = min(n, warp * wlen), we = min(n, wb + wlen);
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int x = wb + lane; x < we; x += 32) {
    const uint32_t k = key(x);
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, s);
    eq += __shfl_xor_sync(0xffffffffu, eq, s);
  }
  if (lane == 0) { wgt[warp] = gt; weq[warp] = eq; }
  __syncthreads();
  if (tid == 0) {
    int a = 0, b = 0;
    for (int w = 0; w < NT / 32; ++w) {
      const int x = wgt[w], y = weq[w];
      wgt[w] = a; weq[w] = b;
      a += x; b += y;
    }
    counts[0] = a; counts[1] = b;
  }
  int g0 = 0, e0 = 0;                      // in the CTAs before this one
  if (cs > 1) {
    cluster_sync();
#pragma unroll
    for (int r = 0; r < MAX_CS; ++r)
      if (r < (int)rank) { g0 += remote_int(&counts[0], (uint32_t)r); e0 += remote_int(&counts[1], (uint32_t)r); }
    cluster_sync();                        // nobody leaves while its counts are read
  } else {
    __syncthreads();
  }
  g0 += wgt[warp];
  e0 += weq[warp];
  for (int x0 = wb; x0 < we; x0 += 32) {
    const int x = x0 + lane;
    const uint32_t k = x < we ? key(x) : 0u;
    const bool is_eq = x < we && k == prefix, is_gt = x < we && k > prefix;
    const unsigned be = __ballot_sync(0xffffffffu, is_eq), bg = __ballot_sync(0xffffffffu, is_gt);
    const unsigned below = (1u << lane) - 1u;
    const int e = e0 + __popc(be & below);
    // kept before this one: all above the threshold, and the equal ones among the first `need`
    if (is_gt || (is_eq && e < need)) idx[g0 + __popc(bg & below) + min(e, need)] = lo + x;
    g0 += __popc(bg);
    e0 += __popc(be);
  }
}

// The row of a kept position in the source pages and its new row, as offsets
// in 16-byte units (-1: a bad page, nothing moves).
struct Move { long long src, dst; };
template <typename T>
__device__ __forceinline__ Move move_of(const EvictP& p, int slot, int h, int src, int dst) {
  const int ps = paged_page(p.c, p.c.page_table, p.c.table_stride, slot, src);
  const int pd = paged_page(p.c, p.tout, p.tout_stride, slot, dst);
  Move m;
  m.src = m.dst = -1;
  if (ps >= 0 && pd >= 0) {
    m.src = (long long)(paged_off(p.c, ps, h, src) * sizeof(T) / 16);
    m.dst = (long long)(paged_off(p.c, pd, h, dst) * sizeof(T) / 16);
  }
  return m;
}

// To fresh pages: one CTA per ROWS kept positions.
constexpr int MV_NT = 256;
template <typename T>
__global__ void __launch_bounds__(MV_NT) evict_move(const EvictP p) {
  constexpr int V = WS_DH * sizeof(T) / 16;     // 16-byte pieces of a row
  constexpr int U = 8;                          // copies in flight per thread
  constexpr int ROWS = U * MV_NT / (2 * V);
  __shared__ Move mv[ROWS];
  const int h = blockIdx.y, i = blockIdx.z, H = p.c.n_kv_heads, j0 = blockIdx.x * ROWS;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  pdl_wait();
  if (slot < 0 || slot >= p.c.n_slots) return;
  const int keep = min(p.len[i], p.a.keep), n = min(ROWS, keep - j0);
  if (h == 0 && j0 == 0 && threadIdx.x == 0) p.a.kv_len_out[slot] = keep;
  if (n <= 0) return;
  const int32_t* idx = p.idx + ((size_t)i * H + h) * p.a.keep + j0;
  const size_t unit = (size_t)slot * H + h;
  if (p.ordered && j0 == 0)
    for (int b = 0; b < keep; b += MV_NT) {
      const int j = b + threadIdx.x, src = j < keep ? idx[j] : 0;
      const float m = j < keep ? p.a.mass[unit * p.a.mass_stride + src] : 0.f;
      const int q = j < keep && p.a.pos ? p.a.pos[unit * p.a.pos_stride + src] : src;
      __syncthreads();                          // the batch is read before any of it is written
      if (j < keep && p.a.mass_out) p.a.mass_out[unit * p.a.mass_out_stride + j] = m;
      if (j < keep && p.a.pos_out) p.a.pos_out[unit * p.a.pos_out_stride + j] = q;
    }
  for (int x = threadIdx.x; x < n; x += MV_NT) {
    const int src = idx[x];
    mv[x] = move_of<T>(p, slot, h, src, j0 + x);
    if (p.ordered) continue;
    if (p.a.mass_out) p.a.mass_out[unit * p.a.mass_out_stride + j0 + x] = p.a.mass[unit * p.a.mass_stride + src];
    if (p.a.pos_out) p.a.pos_out[unit * p.a.pos_out_stride + j0 + x] = p.a.pos ? p.a.pos[unit * p.a.pos_stride + src] : src;
  }
  __syncthreads();
  const uint4 *k = (const uint4*)p.c.k, *v = (const uint4*)p.c.v;
  uint4 reg[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int x = u * MV_NT + threadIdx.x, row = x / (2 * V), piece = x % (2 * V);
    if (row < n && mv[row].src >= 0) reg[u] = __ldcs((piece < V ? k : v) + mv[row].src + piece % V);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int x = u * MV_NT + threadIdx.x, row = x / (2 * V), piece = x % (2 * V);
    if (row < n && mv[row].src >= 0) ((uint4*)(piece < V ? p.c.k : p.c.v))[mv[row].dst + piece % V] = reg[u];
  }
}

// In place: one CTA per (request, head, keys or values, part of the row: P
// pieces of 16 bytes).  A batch of rows is read before any of it is written;
// the next batch's places are looked up while the loads are in flight.
constexpr int CP_NT = 512;
template <typename T, int P>
__global__ void __launch_bounds__(CP_NT) evict_compact(const EvictP p) {
  constexpr int PARTS = WS_DH * sizeof(T) / (16 * P), U = 4, STEP = CP_NT / P * U, M = (STEP + CP_NT - 1) / CP_NT;
  __shared__ Move mv[2][STEP];
  const int h = blockIdx.y, i = blockIdx.z, H = p.c.n_kv_heads;
  const int col = blockIdx.x % PARTS, which = blockIdx.x / PARTS, tid = threadIdx.x;
  const int slot = p.a.req_ids ? p.a.req_ids[i] : i;
  pdl_wait();
  if (slot < 0 || slot >= p.c.n_slots) return;
  const int keep = min(p.len[i], p.a.keep);
  if (h == 0 && blockIdx.x == 0 && tid == 0) p.a.kv_len_out[slot] = keep;
  const int32_t* idx = p.idx + ((size_t)i * H + h) * p.a.keep;
  const size_t unit = (size_t)slot * H + h;
  uint4* base = (uint4*)(which ? p.c.v : p.c.k) + P * col + tid % P;
  const bool marks = blockIdx.x == 0;           // this CTA also moves the masses and labels
  int from[M];                                  // sources of the rows this thread looks up
  auto look_up = [&](int j0, Move* m) {
#pragma unroll
    for (int q = 0; q < M; ++q) {
      const int x = q * CP_NT + tid, j = j0 + x;
      if (x >= STEP) continue;
      from[q] = j < keep ? idx[j] : -1;
      Move w;
      w.src = w.dst = -1;
      if (j < keep && from[q] != j) w = move_of<T>(p, slot, h, from[q], j);
      m[x] = w;
    }
  };
  look_up(0, mv[0]);
  __syncthreads();
  for (int j0 = 0, buf = 0; j0 < keep; j0 += STEP, buf ^= 1) {
    uint4 reg[U];
    long long dst[U];
    float ms[M];
    int ps[M];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Move m = mv[buf][u * (CP_NT / P) + tid / P];
      dst[u] = m.src >= 0 ? m.dst : -1;
      if (m.src >= 0) reg[u] = base[m.src];
    }
    bool on[M];
#pragma unroll
    for (int q = 0; q < M; ++q) {
      on[q] = marks && q * CP_NT + tid < STEP && from[q] >= 0;
      if (!on[q]) continue;
      ms[q] = p.a.mass[unit * p.a.mass_stride + from[q]];
      ps[q] = p.a.pos ? p.a.pos[unit * p.a.pos_stride + from[q]] : from[q];
    }
    look_up(j0 + STEP, mv[buf ^ 1]);
    __syncthreads();                            // the batch is read before any of it is written
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) base[dst[u]] = reg[u];
#pragma unroll
    for (int q = 0; q < M; ++q) {
      if (!on[q]) continue;
      const int j = j0 + q * CP_NT + tid;
      if (p.a.mass_out) p.a.mass_out[unit * p.a.mass_out_stride + j] = ms[q];
      if (p.a.pos_out) p.a.pos_out[unit * p.a.pos_out_stride + j] = ps[q];
    }
    // a later batch reads positions behind all of this one's destinations,
    // and a part of the rows is read and written by this CTA alone
  }
}

const char* check_evict(const ws_paged_cache* c, const ws_evict_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0 || a->n_req > 65535) return "n_req must be 0..65535";
  if (a->max_kv > (1 << 30)) return "max_kv must be at most 2^30";
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

// CTAs per (request, head): as many as run at once (two per SM), each with
// 1,024 keys at least (whole eviction, 8 heads x 65,536 positions: 2 requests
// 171 us with one CTA each, 60 so; 8 requests 237 and 134); the keys stay in
// shared memory where they fit.
template <int NT>
cudaError_t select(EvictP& p, cudaStream_t s) {
  const long long units = (long long)p.a.n_req * p.c.n_kv_heads;
  p.cs = 1;
  while (p.cs < MAX_CS && 2 * units * p.cs <= 304 && p.a.max_kv / (2 * p.cs) >= 1024) p.cs *= 2;
  const int seg = (p.a.max_kv + p.cs - 1) / p.cs;
  p.cached = seg <= 48 * 1024 ? seg : 0;
  cudaError_t e = cudaFuncSetAttribute(evict_select<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 48 * 1024 * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(p.cs, p.c.n_kv_heads, p.a.n_req);
  c.blockDim = dim3(NT);
  c.dynamicSmemBytes = (size_t)p.cached * 4;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cs; at[0].val.clusterDim.y = 1; at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, evict_select<NT>, (const EvictP)p);
  if (e == cudaSuccess) ws_count_launches(1);
  return e;
}

template <typename T, int P>
cudaError_t compact(const EvictP& p, cudaStream_t s) {
  return launch_after(evict_compact<T, P>, dim3(2 * WS_DH * sizeof(T) / (16 * P), p.c.n_kv_heads, p.a.n_req), CP_NT, 0, s, p);
}

template <typename T>
cudaError_t move(const EvictP& p, bool in_place, cudaStream_t s) {
  constexpr int V = WS_DH * sizeof(T) / 16, ROWS = 8 * MV_NT / (2 * V);
  // 128 bytes of a row per CTA, or 64 where that gives too few CTAs (96 x 20
  // heads cut from 1500 to 512 115 and 127 us; 8 x 8 heads from 65,536 to
  // 16,384 183 and 147, with 32 bytes 193 and 200)
  if (in_place) return 2ll * p.a.n_req * p.c.n_kv_heads >= 4 * 152 ? compact<T, 8>(p, s) : compact<T, 4>(p, s);
  return launch_after(evict_move<T>, dim3((p.a.keep + ROWS - 1) / ROWS, p.c.n_kv_heads, p.a.n_req), MV_NT, 0, s, p);
}

}  // namespace

size_t cache_evict_workspace(const ws_paged_cache& cache, const ws_evict_args& args) { return evict_bytes(&cache, &args); }

cudaError_t launch_cache_evict(const ws_paged_cache& cache, const ws_evict_args& args, void* workspace, cudaStream_t s) {
  EvictP p = {};
  p.c = paged_copy(cache);
  p.a = args;
  const bool in_place = !args.page_table_out || args.page_table_out == cache.page_table;
  p.tout = in_place ? cache.page_table : args.page_table_out;
  p.tout_stride = in_place ? cache.table_stride : args.table_out_stride;
  p.len = (int32_t*)workspace;
  p.idx = (int32_t*)((char*)workspace + ((size_t)args.n_req * 4 + 255) / 256 * 256);
  p.ordered = args.mass_out == args.mass || (args.pos && args.pos_out == args.pos);
  // threads of a selecting CTA, 256 against 512 (whole eviction, 20 heads): 64
  // requests x 4096 positions 101 and 115 us, 32 x 8192 80 and 75 us, 8 x 8192
  // 42 and 37 us
  cudaError_t e = args.max_kv <= 4096 ? select<256>(p, s) : select<512>(p, s);
  if (e != cudaSuccess) return e;
  return cache.dtype == WS_BF16 ? move<bf16>(p, in_place, s) : move<float>(p, in_place, s);
}

extern "C" size_t ws_cache_evict_workspace(const ws_paged_cache* cache, const ws_evict_args* args) {
  if (check_evict(cache, args) || args->n_req == 0 || cache->dtype == WS_E4M3) return 0;
  return evict_bytes(cache, args);
}

extern "C" int ws_cache_evict(const ws_paged_cache* cache, const ws_evict_args* args, void* workspace,
                              size_t workspace_bytes, ws_stream stream) {
  if (const char* e = check_evict(cache, args)) return paged_fail(WS_EINVAL, e);
  if (cache->dtype == WS_E4M3) return paged_fail(WS_EUNSUPPORTED, "positions of a cache in 8 bits cannot leave their block's scale");
  if (args->n_req == 0) return WS_OK;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return paged_fail(WS_EINVAL, "workspace must be 16-byte aligned and not null");
  if (evict_bytes(cache, args) > workspace_bytes)
    return paged_fail(WS_ENOSPACE, "workspace smaller than ws_cache_evict_workspace()");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  const cudaError_t e = launch_cache_evict(*cache, *args, workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("cache eviction launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

// Shared by the kernels of ws_paged_attention.
#pragma once
#include "ws_paged.cuh"
#include "ws_tc.cuh"

// How key tiles of TK positions lie in the pages.  A tile is either one box
// of at most TK tokens of one page (page_size >= TK, or one that does not
// divide TK: `tpp` tiles per page) or, with small pages that divide TK,
// `ppt` whole pages.  Either way a tile's positions are consecutive.
struct TileGeo {
  int box;                                 // tokens per copy
  int tpp;                                 // tiles per page (0: several pages per tile)
  int ppt_log;                             // log2 pages per tile, page_log: log2 page_size
  int page_log;
  int pieces;                              // > 1: what is called a page here is one of so many pieces of a page
};
// `split`: pages that neither divide a tile nor hold whole ones may be taken in
// pieces that do (their largest power of two), else a page's last tile is
// short.  Many copies of eight keys cost up to a third, so those only where
// short tiles would be less than three quarters full.
inline TileGeo tile_geo(int page_size, int tk, bool split = false) {
  TileGeo g = {};
  const int piece = page_size & -page_size;
  if (split && page_size % tk && tk % page_size &&
      (piece >= 16 || (piece == 8 && page_size < (page_size + tk - 1) / tk * (tk / 4 * 3)))) {
    g.pieces = page_size / piece;
    page_size = piece;
  }
  if (page_size < tk && tk % page_size == 0 && page_size >= 8) {
    g.box = page_size;
    while ((1 << g.page_log) < page_size) ++g.page_log;
    while ((page_size << g.ppt_log) < tk) ++g.ppt_log;
  } else {
    g.box = page_size < tk ? page_size : tk;
    g.tpp = (page_size + tk - 1) / tk;
  }
  return g;
}
// Tiles that hold L positions (an upper bound grows with L).
__host__ __device__ __forceinline__ int tile_count(const TileGeo& g, int page_size, int tk, int L) {
  if (g.tpp == 0) return (L + tk - 1) / tk;
  return L / page_size * g.tpp + (L % page_size + tk - 1) / tk;
}
// Tiles that end at or before position L.
__device__ __forceinline__ int tile_whole(const TileGeo& g, int page_size, int tk, int L) {
  if (g.tpp == 0) return L / tk;
  const int rest = L % page_size;
  return L / page_size * g.tpp + rest / tk;
}

// A factor of scores, kept from 0 and infinity: times -inf or 0 they would be NaN.
__device__ __forceinline__ float score_factor(float f) { return fminf(fmaxf(f, 1.17549435e-38f), 3e38f); }

__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A warp's walk over every step-th tile from t0 on: position of the tile and
// the page(s) of its keys.
struct TileWalk {
  int t, pi, sub, step;
  __device__ __forceinline__ void start(const TileGeo& g, int t0, int st) {
    t = t0; step = st;
    if (g.tpp) { pi = t0 / g.tpp; sub = t0 - pi * g.tpp; }
  }
  __device__ __forceinline__ void next(const TileGeo& g) {
    t += step;
    if (g.tpp) { sub += step; while (sub >= g.tpp) { sub -= g.tpp; ++pi; } }
  }
  // first position of the tile, keys it may hold, and for key j its table entry
  __device__ __forceinline__ int base(const TileGeo& g, int ps, int tk) const { return g.tpp ? pi * ps + sub * tk : t * tk; }
  __device__ __forceinline__ int room(const TileGeo& g, int ps, int tk) const { return g.tpp ? min(tk, ps - sub * tk) : tk; }
  __device__ __forceinline__ int entry(const TileGeo& g, int j) const { return g.tpp ? pi : (t << g.ppt_log) + (j >> g.page_log); }
};

struct AttnP {
  ws_paged_cache c;
  ws_attention_args a;
  int pad_H;                               // > 0: request i has rows i * pad_H .., chunk_len[i] of them in use (cu_q is not read)
  const int32_t* chunk_len;
  int G;                                   // query heads per KV head
  float sl;                                // |scale| * log2(e): scores in log2 units (1 when scale is 0)
  uint32_t q_and, q_xor;                   // applied to bf16 query pairs: the sign of scale, or all zero
  int nsplit;                              // key splits per row tile
  int tps;                                 // key tiles per split
  TileGeo geo;
  float2* part_ml;                         // split partials: (max in log2 units, sum) [unit row][nsplit] ...
  float* part_o;                           // ... and values [unit row][nsplit][64], unit row = (i * Hkv + h) * max_q * G + r * G + g
  float* lse;                              // [total_q][n_heads], or null
  int row_tiles;                           // row tiles per (request, KV head)
  float* nl;                               // tcgen05 path with mass: -lse * log2(e) of every row tile's rows
                                           // [n_req][Hkv][row_tiles][128], 16-byte aligned; else null
  uint32_t block_mul;                      // 8 bits: 2^32 / scale_block, rounded up (0: scale_block is 1)
  unsigned long long* next_item;           // with nl: counter of the weight pass's work items, cleared by fa_kernel
};

struct Req {
  int slot, row0, c, L;                    // cache slot, first row, chunk length, visible positions
};
__device__ __forceinline__ Req request(const AttnP& p, int i) {
  Req r;
  r.slot = p.a.req_ids ? p.a.req_ids[i] : i;
  if (p.pad_H) {
    r.row0 = i * p.pad_H;
    r.c = min(max(p.chunk_len[i], 0), p.pad_H);
  } else {
    r.row0 = p.a.cu_q[i];
    const int end = min(p.a.cu_q[i + 1], p.a.total_q);
    r.c = r.row0 >= 0 ? min(max(end - r.row0, 0), p.a.max_q) : 0;
  }
  r.L = 0;
  if (r.slot >= 0 && r.slot < p.c.n_slots)
    r.L = (int)min((long long)min(max(p.a.kv_len[r.slot], 0), p.a.max_kv), (long long)p.c.table_stride * p.c.page_size);
  return r;
}
// Positions 0 .. limit - 1 are visible to row t of the chunk.
__device__ __forceinline__ int row_limit(const AttnP& p, const Req& r, int t) {
  return p.a.causal ? max(0, min(r.L, r.L - r.c + t + 1)) : r.L;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Values that are not finite where some row of the CTA does not see them: the
// row's weight is 0 there, but 0 * inf is not.  They are taken out of the tile
// and noted as the first position of a +inf, a -inf and a NaN in each element;
// the rows that see it get it back at the end (their weight is above 0).
struct Odd { int first[3][WS_DH]; int any; };      // `any` starts at 0, the rest with the first find
__device__ __forceinline__ float with_odd(const Odd& odd, float o, int limit, int d) {
  if (limit > odd.first[2][d]) o = NAN;
  if (limit > odd.first[0][d]) o += INFINITY;
  if (limit > odd.first[1][d]) o -= INFINITY;
  return o;
}
// Notes and clears such values of a tile.
template <int ROWS>
__device__ __forceinline__ void note_odd(Odd& odd, uint8_t* tile, int base, int lane) {
  if (!odd.any) {
    for (int x = lane; x < 3 * WS_DH; x += 32) odd.first[0][x] = 0x7FFFFFFF;
    __syncwarp();
  }
  uint4* at = reinterpret_cast<uint4*>(tile) + lane;
  for (int q = 0; q < ROWS / 4; ++q) {
    const int x = 32 * q + lane, row = x >> 3, d = ((x & 7) ^ (row & 7)) * 8;
    unsigned short* e = reinterpret_cast<unsigned short*>(at + 32 * q);
    for (int k = 0; k < 8; ++k) {
      const unsigned short b = e[k];
      if ((b & 0x7F80u) != 0x7F80u) continue;
      atomicMin(&odd.first[b & 0x7Fu ? 2 : b >> 15][d + k], base + row);
      e[k] = 0;
    }
  }
  __syncwarp();
  if (lane == 0) odd.any = 1;
}
template <int ROWS>
__device__ __noinline__ void call_note_odd(Odd& odd, uint8_t* tile, int base, int lane) {
  note_odd<ROWS>(odd, tile, base, lane);
}
// A warp looks through the ROWS rows (ROWS / 4 pieces of 16 bytes per lane) of
// a value tile of 128-byte rows, 128-byte swizzle, first position `base`; true
// if something was cleared.  CALL: the rare part outside the caller's code (not
// where setmaxnreg has limited the warp's registers: a called function does not
// know the limit).
template <int ROWS, int STEP, bool CALL>
__device__ __forceinline__ bool take_out_odd(Odd& odd, uint8_t* tile, int base, int lane) {
  constexpr int N = ROWS / 4;              // STEP of them in flight
  const uint4* at = reinterpret_cast<const uint4*>(tile) + lane;
  uint32_t found = 0;                      // bit 31 or 15 of a pair's exponent + 1: all ones
#pragma unroll
  for (int q = 0; q < N; q += STEP) {
    uint4 v[STEP];
#pragma unroll
    for (int k = 0; k < STEP; ++k) v[k] = at[32 * (q + k)];
#pragma unroll
    for (int k = 0; k < STEP; ++k)
      found |= ((v[k].x & 0x7FFF7FFFu) + 0x00800080u) | ((v[k].y & 0x7FFF7FFFu) + 0x00800080u) |
               ((v[k].z & 0x7FFF7FFFu) + 0x00800080u) | ((v[k].w & 0x7FFF7FFFu) + 0x00800080u);
  }
  if (!__any_sync(0xffffffffu, (found & 0x80008000u) != 0u)) return false;
  if (CALL) call_note_odd<ROWS>(odd, tile, base, lane);
  else note_odd<ROWS>(odd, tile, base, lane);
  return true;
}
constexpr float LN2 = 0.69314718055994531f, LOG2E = 1.4426950408889634f;

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int t, int h, int p) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(tc::smem_u32(dst)), "l"((uint64_t)map), "r"(x), "r"(t), "r"(h), "r"(p), "r"(tc::smem_u32(bar))
      : "memory");
}

// Long chunks on tcgen05 (ws_pattn_fa.cu): tiles of G * (128 / G) rows (whole
// chunk rows) against tiles of FA_KEYS keys.  Rows of unsplit calls go to
// out / lse, those of split calls to the partials.
constexpr int FA_ROWS = 128, FA_KEYS = 128;
cudaError_t launch_fa(const AttnP& p, bool two_heads, cudaStream_t s);
cudaError_t launch_fa_mass(const AttnP& p, cudaStream_t s);

// The fp32 model (ws_pattn_f32.cu): row tiles of 32 or 64 rows and key tiles of
// F32_KEYS positions; up to 16 rows per KV head in f32_rows_kernel.
constexpr int F32_KEYS = 64;
cudaError_t launch_f32(const AttnP& p, int rpt, cudaStream_t s);
struct F32Rows { int ctas, keys; bool join; };   // CTAs per (request, KV head), positions each, joined by a cluster
F32Rows f32_rows_plan(long long units, int max_kv, bool mass);
F32Rows f32_block_plan(int max_kv);                // a context's block: by max_kv (at most 8,192) alone
cudaError_t launch_f32_rows(const AttnP& p, const F32Rows& f, cudaStream_t s);
cudaError_t launch_f32_mass(const AttnP& p, int rpt, cudaStream_t s);

// Caches in 8 bits (ws_pattn_q8.cu): row tiles of 8 * nt rows that stream the cache.
constexpr int Q8_TK = 32;                          // keys per tile
cudaError_t launch_q8(const AttnP& p, int nt, cudaStream_t s);

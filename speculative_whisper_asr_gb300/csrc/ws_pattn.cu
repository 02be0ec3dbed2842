// Attention of a chunk of new tokens over a paged cache
// (ws_paged_attention in include/ws.h gives the formulas).
#include <type_traits>

#include "ws_attn_mma.cuh"
#include "ws_pattn.cuh"

namespace {

// ------------------------------------------------------------------ bf16, few rows: stream the cache once
// The rows of a (request, KV head) — chunk rows x the query heads that share
// the KV head — are cut into row tiles of 8 * NT.  One CTA takes a row tile
// and a range of key tiles; its four warps take every fourth tile of 32 keys
// through private rings of three TMA slots each (K and V, 128-byte swizzle),
// so no warp waits for another until the end.  HBM bounds the kernel, so the
// instruction count per byte matters: the products are taken transposed,
//   S^T = K Q^T    (16 keys x 8 rows per mma m16n8k16),
//   O^T = V^T P^T  (16 dims x 8 rows),
// which puts 8 rows, not 16, into an instruction.  S^T leaves the tensor core
// with keys along lanes; movmatrix turns the bf16 weights into the second
// product's operand.  Scores stay raw; p = 2^(s * sl - m * sl) with one FMA
// and one exponential.  The reference m of a row moves only when a score
// exceeds it by more than 2^8 (p <= 256), which a vote detects, so the
// common tile needs no reduction across lanes; rows that did not exceed it
// keep their reference, so a row's bits do not depend on the tile's other
// rows.  Statistics and sums are fp32.  Up to 8 rows the weights enter the
// value product as bf16 hi + lo (2^-16 relative), which the copy rate hides;
// with more rows as one bf16 value (2^-8 relative at most, the output's own
// step: hi + lo costs 7% at 9 rows, 94 -> 101 us for 96 requests x 20 heads),
// except for a context's blocks (HILO), whose rows have to come out the same
// bits in a block of any height.
//
// With STASH the raw scores stay in tensor memory, which this kernel has no
// other use for: each of the four warps owns a lane quarter and parks a
// tile's score fragment in its next 8 NT columns (256 columns per CTA, 512
// for NT = 4: 4096 / 2048 / 2048 keys).  Once the rows' log-sum-exp is known
// (the CTA has the whole cache: no splits) each warp reads its fragments
// back and adds its positions' weights, so the mass costs neither a second
// read of the keys nor shared memory that the rings need.  Measured at 96
// requests x 20 heads x 9 rows over 375-1500 positions (480 MB): a second
// pass over the keys 176 us, scores in shared memory 126 us, so 90 us (5.3
// TB/s; 77 us, 6.2 TB/s, without weights).  One row of 32 heads on 8 over 16
// caches of up to 65,536 positions (1.36 GB): 202 us, 6.7 TB/s, the rate of a
// plain copy.  One row of one request, 20 heads x 448 positions: 7 us, the
// latency of the chain of loads.
constexpr int SP_TK = 32;                  // keys per tile
constexpr int SP_W = 4;                    // warps
constexpr int SP_NS = 3;                   // ring slots per warp
constexpr int SP_KB = SP_TK * WS_DH * 2;   // bytes of a K or V tile
constexpr int SP_SMEM = SP_W * SP_NS * 2 * SP_KB + 1024;
constexpr int SP_OP = WS_DH + 4;           // row pitch of the CTA's merge area, which reuses the rings
static_assert(SP_W * 32 * (SP_OP + 2) * 4 <= SP_W * SP_NS * 2 * SP_KB, "the merge area fits the rings");
constexpr int sp_cols(int nt) { return nt == 4 ? 512 : 256; }                  // tensor memory columns
constexpr int sp_stash_tiles(int nt) { return sp_cols(nt) / (8 * nt); }        // tiles per warp
constexpr float SP_HOLD = 8.0f;

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

struct SpMeta { uint32_t valid; int base; };   // keys of a tile that count; its first position

// Query fragments of 8 * NT rows (B operand): rows r0 + 8 nt + lane / 4.
template <int NT>
__device__ __forceinline__ void sp_load_q(const AttnP& p, const Req& r, int h, int r0, int R, uint32_t qf[4][NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rho = r0 + 8 * nt + g;
    const bool on = rho < R;
    const int t = on ? rho / p.G : 0;
    const bf16* q = (const bf16*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride + (size_t)(h * p.G + (on ? rho - t * p.G : 0)) * WS_DH;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t v = on ? __ldg(reinterpret_cast<const unsigned int*>(q + 16 * s + 8 * e + 2 * c)) : 0u;
        qf[s][nt][e] = on ? (v & p.q_and) ^ p.q_xor : 0u;
      }
  }
}

// N consecutive tensor memory columns of the warp's lane quarter.
template <int N>
__device__ __forceinline__ void tm_st(uint32_t addr, const float* v) {
#pragma unroll
  for (int q = 0; q < N; q += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr + q),
                 "r"(__float_as_uint(v[q])), "r"(__float_as_uint(v[q + 1])), "r"(__float_as_uint(v[q + 2])),
                 "r"(__float_as_uint(v[q + 3])), "r"(__float_as_uint(v[q + 4])), "r"(__float_as_uint(v[q + 5])),
                 "r"(__float_as_uint(v[q + 6])), "r"(__float_as_uint(v[q + 7])) : "memory");
}
template <int N>
__device__ __forceinline__ void tm_ld(uint32_t addr, float* v) {
#pragma unroll
  for (int q = 0; q < N; q += 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr + q));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[q + e] = __uint_as_float(r[e]);
  }
}

// The values that the warps took out, back into their partials of the rows that see them.
template <int ROWS>
__device__ __noinline__ void give_back_odd(const AttnP& p, const Req& r, const Odd* odd, float* so, int r0, int R) {
  for (int x = threadIdx.x; x < SP_W * ROWS * WS_DH; x += SP_W * 32) {
    const int k = x / (ROWS * WS_DH), row = x / WS_DH % ROWS, d = x % WS_DH;
    if (r0 + row >= R || !odd[k].any) continue;
    float* o = so + (k * ROWS + row) * SP_OP + d;
    *o = with_odd(odd[k], *o, row_limit(p, r, (r0 + row) / p.G), d);
  }
  __syncthreads();
}

// MIX: causal chunks of more than one row, where values that are not finite
// are kept from the rows that do not see them.  The look at the last tiles
// costs 5% (96 requests x 20 heads: 32 rows over 375-1500 positions 112 -> 118
// us, 9 rows over 112-448 54 -> 57), which the other calls need not pay.
template <int NT, bool STASH, bool HILO, bool MIX>
__global__ void __launch_bounds__(SP_W * 32, NT == 4 ? 1 : 2)
split_kernel(const AttnP p, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  constexpr int MT = SP_TK / 16;           // key steps of 16
  constexpr uint32_t ALL = 0xffffffffu;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t full[SP_W][SP_NS];
  __shared__ SpMeta meta[SP_W][SP_NS];
  __shared__ Odd odd[MIX ? SP_W : 1];      // each warp's own
  __shared__ float row_lse[8 * NT];
  __shared__ uint32_t s_tmem;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int rt = blockIdx.x / p.nsplit, split = blockIdx.x - rt * p.nsplit, h = blockIdx.y, i = blockIdx.z;
  // a dependent kernel may take tensor memory and then wait for this one: with
  // STASH it may start only once every CTA here has its own
  if (!STASH) pdl_trigger();
  // the first tiles' pages are asked for together with the lengths: the
  // entries exist whatever the lengths turn out to be
  const int slot0 = p.a.req_ids ? p.a.req_ids[i] : i;
  const int32_t* table = p.c.page_table + (size_t)min(max(slot0, 0), p.c.n_slots - 1) * p.c.table_stride;
  TileWalk w;
  auto page_of = [&]() -> int {             // table entry of this lane's key in the walk's tile, -1: none
    const int e = w.entry(p.geo, lane);
    return e < p.c.table_stride ? __ldg(table + e) : -1;
  };
  w.start(p.geo, split * p.tps + warp, SP_W);
  int page0[SP_NS];
#pragma unroll
  for (int s = 0; s < SP_NS; ++s) { page0[s] = page_of(); w.next(p.geo); }
  const Req r = request(p, i);
  const int R = r.c * p.G, r0 = rt * 8 * NT;
  if (r0 >= R) return;
  if (lane == 0)
    for (int s = 0; s < SP_NS; ++s) tc::mbar_init(&full[warp][s], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();
  if (STASH && warp == 0) tc::tmem_alloc(&s_tmem, sp_cols(NT));
  // positions that some row of this tile sees, and those that all see
  const int last = min(R, r0 + 8 * NT) - 1;
  const int Lmax = row_limit(p, r, last / p.G), Lmin = row_limit(p, r, r0 / p.G);
  const int nt_all = tile_count(p.geo, p.c.page_size, SP_TK, Lmax);
  const int tb = min(nt_all, split * p.tps), te = min(nt_all, tb + p.tps);
  const int n_my = max(0, (te - tb - warp + SP_W - 1) / SP_W);
  uint8_t* ring = sm + warp * (SP_NS * 2 * SP_KB);
  auto issue = [&](int slot, int page) {
    const int base = w.base(p.geo, p.c.page_size, SP_TK);
    const bool ok = page >= 0 && page < p.c.n_pages && lane < w.room(p.geo, p.c.page_size, SP_TK) && base + lane < Lmax;
    const uint32_t valid = __ballot_sync(0xffffffffu, ok);
    const bool go = ok && (p.geo.tpp ? (valid & ((1u << lane) - 1u)) == 0u : (lane & (p.geo.box - 1)) == 0);
    const unsigned boxes = __ballot_sync(0xffffffffu, go);
    if (lane == 0) {
      meta[warp][slot].valid = valid;
      meta[warp][slot].base = base;
      tc::mbar_expect_tx(&full[warp][slot], (uint32_t)__popc(boxes) * 2u * (uint32_t)p.geo.box * 128u);
    }
    __syncwarp();
    if (go) {
      uint8_t* dst = ring + slot * (2 * SP_KB) + (p.geo.tpp ? 0 : lane * 128);
      const int tok = p.geo.tpp ? w.sub * SP_TK : 0;
      tma_load_4d(dst, &mk, &full[warp][slot], 0, tok, h, page);
      tma_load_4d(dst + SP_KB, &mv, &full[warp][slot], 0, tok, h, page);
    }
  };
  w.start(p.geo, split * p.tps + warp, SP_W);
#pragma unroll
  for (int s = 0; s < SP_NS; ++s)
    if (s < n_my) { issue(s, page0[s]); w.next(p.geo); }

  uint32_t qf[4][NT][2];
  sp_load_q<NT>(p, r, h, r0, R, qf);
  int lim[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[nt][e] = row_limit(p, r, min(r0 + 8 * nt + 2 * c + e, R - 1) / p.G);
  float o[4][NT][4], m[NT][2], msl[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) { m[nt][e] = -INFINITY; msl[nt][e] = 0.f; l[nt][e] = 0.f; }
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][nt][e] = 0.f;
  }
  const bool mixed = MIX && Lmin < Lmax;    // some row does not see all of the tile's positions
  if (MIX && lane == 0) odd[warp].any = 0;
  const float sl = p.sl, hold = fminf(SP_HOLD / sl, 1e30f);
  uint32_t tmem = 0;                        // this warp's columns
  if (STASH) {
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    pdl_trigger();
    tmem = s_tmem + ((uint32_t)warp << 21);
  }
  bool dead = false;
  // One tile.  The last ones, which some row does not see all of, have a copy
  // of the code to themselves (96 x 32 causal rows 118 us; 120 with their look
  // at the values inside the usual loop).
  auto tile = [&](int it, auto last_tiles) -> bool {
    const int slot = it % SP_NS;
    const bool more = it + SP_NS < n_my;
    const int page_next = more ? page_of() : -1;      // in flight while this tile is computed
    if (!tc::mbar_wait(&full[warp][slot], (uint32_t)((it / SP_NS) & 1))) { dead = true; return false; }
    const SpMeta mt_ = meta[warp][slot];
    uint8_t* Kt = ring + slot * (2 * SP_KB);
    uint8_t* Vt = Kt + SP_KB;
    if (mt_.valid != ALL) {
      // rows that do not count may hold anything: 0 * inf would reach the sums
      if (!((mt_.valid >> lane) & 1u)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(Vt + lane * 128 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot's next copy
      __syncwarp();
    }
    if (decltype(last_tiles)::value && take_out_odd<SP_TK, 2, true>(odd[warp], Vt, mt_.base, lane)) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the slot's next copy
      __syncwarp();
    }
    const uint32_t kb = tc::smem_u32(Kt), vb = tc::smem_u32(Vt);
    float sc[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[mt][nt][0] = sc[mt][nt][1] = sc[mt][nt][2] = sc[mt][nt][3] = 0.f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a[4];
        const int mtx = lane >> 3, key = 16 * mt + ((mtx & 1) << 3) + (lane & 7);
        ldsm_x4(kb + kv_off<true>(key, 2 * s + (mtx >> 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(sc[mt][nt], a, qf[s][nt][0], qf[s][nt][1]);
      }
    }
    if (mt_.valid != ALL || mt_.base + SP_TK > Lmin) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int j = 16 * mt + 8 * e2 + g;
          const bool ok = (mt_.valid >> j) & 1u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!ok || mt_.base + j >= lim[nt][e]) sc[mt][nt][2 * e2 + e] = -INFINITY;
        }
    }
    if (STASH) tm_st<8 * NT>(tmem + (uint32_t)(it * 8 * NT), &sc[0][0][0]);
    // ---- does a score pass its row's reference by more than 2^8?
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float t4 = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
        grow |= t4 > m[nt][e] + hold;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t4 = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][2 + e]), fmaxf(sc[1][nt][e], sc[1][nt][2 + e]));
          t4 = fmaxf(t4, __shfl_xor_sync(0xffffffffu, t4, 4));
          t4 = fmaxf(t4, __shfl_xor_sync(0xffffffffu, t4, 8));
          t4 = fmaxf(t4, __shfl_xor_sync(0xffffffffu, t4, 16));
          const float mn = t4 > m[nt][e] + hold ? t4 : m[nt][e];
          const float f = m[nt][e] > -INFINITY ? ex2((m[nt][e] - mn) * sl) : 0.f;
          m[nt][e] = mn;
          msl[nt][e] = mn > -INFINITY ? mn * sl : 0.f;
          l[nt][e] *= f;
#pragma unroll
          for (int d = 0; d < 4; ++d) { o[d][nt][e] *= f; o[d][nt][2 + e] *= f; }
        }
    }
    uint32_t pf[MT][NT][2], pg[MT][NT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const float p0 = ex2(fmaf(sc[mt][nt][2 * e2], sl, -msl[nt][0]));
          const float p1 = ex2(fmaf(sc[mt][nt][2 * e2 + 1], sl, -msl[nt][1]));
          l[nt][0] += p0;
          l[nt][1] += p1;
          const uint32_t hi = pack_bf16(p0, p1);
          const float2 hf = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi));
          pf[mt][nt][e2] = movm(hi);
          if (HILO) pg[mt][nt][e2] = movm(pack_bf16(p0 - hf.x, p1 - hf.y));
        }
#pragma unroll
    for (int ks = 0; ks < MT; ++ks)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t a[4];
        const int mtx = lane >> 3, key = 16 * ks + ((mtx >> 1) << 3) + (lane & 7);
        ldsm_x4_t(vb + kv_off<true>(key, 2 * d + (mtx & 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16_16816(o[d][nt], a, pf[ks][nt][0], pf[ks][nt][1]);
          if (HILO) mma_bf16_16816(o[d][nt], a, pg[ks][nt][0], pg[ks][nt][1]);
        }
      }
    __syncwarp();                           // every lane has read the slot
    if (more) { issue(slot, page_next); w.next(p.geo); }
    return true;
  };
  int it = 0;
  if (MIX) {
    // this warp's tiles that end at or before Lmin
    const int whole = mixed ? tile_whole(p.geo, p.c.page_size, SP_TK, Lmin) : n_my * SP_W;
    const int n_whole = min(n_my, max(0, (whole - tb - warp + SP_W - 1) / SP_W));
    while (it < n_whole && tile(it, std::false_type())) ++it;
    while (!dead && it < n_my && tile(it, std::true_type())) ++it;
  } else {
    while (it < n_my && tile(it, std::false_type())) ++it;
  }
  // ---- the four warps' partials meet in shared memory
  __syncthreads();
  constexpr int OP = SP_OP;
  float* so = reinterpret_cast<float*>(sm); // [warp][8 NT][OP]
  float* sml = so + SP_W * 8 * NT * OP;     // [warp][8 NT][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[nt][e];
      s += __shfl_xor_sync(0xffffffffu, s, 4);
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      const int row = 8 * nt + 2 * c + e;
      float* dst = so + (warp * 8 * NT + row) * OP;
#pragma unroll
      for (int d = 0; d < 4; ++d) { dst[16 * d + g] = o[d][nt][e]; dst[16 * d + 8 + g] = o[d][nt][2 + e]; }
      if (g == 0) {
        sml[(warp * 8 * NT + row) * 2] = dead ? NAN : m[nt][e];
        sml[(warp * 8 * NT + row) * 2 + 1] = dead ? NAN : s;
      }
    }
  __syncthreads();
  if (MIX && (odd[0].any | odd[1].any | odd[2].any | odd[3].any)) give_back_odd<8 * NT>(p, r, odd, so, r0, R);
  for (int x = threadIdx.x; x < 8 * NT * 16; x += SP_W * 32) {
    const int row = x >> 4, d4 = x & 15, rho = r0 + row;
    if (rho >= R) continue;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < SP_W; ++k) M = fmaxf(M, sml[(k * 8 * NT + row) * 2]);
    float sum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int k = 0; k < SP_W; ++k) {
      const float mk_ = sml[(k * 8 * NT + row) * 2];
      const float f = mk_ == -INFINITY ? 0.f : ex2((mk_ - M) * sl);
      const float4 v = *reinterpret_cast<const float4*>(so + (k * 8 * NT + row) * OP + 4 * d4);
      sum = fmaf(f, sml[(k * 8 * NT + row) * 2 + 1], sum);
      a0 = fmaf(f, v.x, a0); a1 = fmaf(f, v.y, a1); a2 = fmaf(f, v.z, a2); a3 = fmaf(f, v.w, a3);
    }
    if (p.nsplit > 1) {
      const size_t at = (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit + split;
      *reinterpret_cast<float4*>(p.part_o + at * WS_DH + 4 * d4) = make_float4(a0, a1, a2, a3);
      if (d4 == 0) p.part_ml[at] = make_float2(M == -INFINITY ? M : M * sl, sum);
      continue;
    }
    const int t = rho / p.G, u = h * p.G + rho - t * p.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (STASH && d4 == 0) row_lse[row] = sum == 0.f ? INFINITY : M * sl + lg2(sum);
    bf16* out = (bf16*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u * WS_DH + 4 * d4;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(a0 * inv, a1 * inv), pack_bf16(a2 * inv, a3 * inv));
    if (p.lse && d4 == 0) p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u] = sum == 0.f ? -INFINITY : (M * sl + lg2(sum)) * LN2;
  }
  if (STASH) {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    __syncthreads();
    float nl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) nl[nt][e] = r0 + 8 * nt + 2 * c + e < R ? row_lse[8 * nt + 2 * c + e] : INFINITY;
    // a row whose log-sum-exp is NaN adds NaN where it sees, and nothing elsewhere
    bool nan = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) nan |= nl[nt][0] != nl[nt][0] || nl[nt][1] != nl[nt][1];
    nan = __any_sync(ALL, nan);
    float* mass = p.a.mass + ((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride;
    // a quad ends up with the sums of four keys per step of 32; its lane c
    // adds key 8 c + g.  The position is this thread's alone, so the atomic
    // (which does not wait for the old value) has nothing to race with.
    w.start(p.geo, tb + warp, SP_W);
    constexpr int U = NT == 4 ? 1 : 2;      // tiles at once: one's latencies under the other's
    auto add_weights = [&](auto nan_row) {
      constexpr bool NAN_ROW = decltype(nan_row)::value;
      for (int it = 0; it < n_my; it += U) {
        float sv[U][MT][NT][4];
#pragma unroll
        for (int k = 0; k < U; ++k) tm_ld<8 * NT>(tmem + (uint32_t)(min(it + k, n_my - 1) * 8 * NT), &sv[k][0][0][0]);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        float part[U][4];
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int q = 0; q < 4; ++q) {       // keys 8 q + g
            float s = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float x = sv[k][q >> 1][nt][2 * (q & 1) + e], y = ex2(fmaf(x, sl, -nl[nt][e]));
                s += NAN_ROW && x == -INFINITY ? 0.f : y;
              }
            part[k][q] = s;
          }
        // a quad's four lanes hold parts of four keys: two exchanges leave each
        // lane with the whole sum of one
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float a0 = (c & 2 ? part[k][2] : part[k][0]) + __shfl_xor_sync(0xffffffffu, c & 2 ? part[k][0] : part[k][2], 2);
          const float a1 = (c & 2 ? part[k][3] : part[k][1]) + __shfl_xor_sync(0xffffffffu, c & 2 ? part[k][1] : part[k][3], 2);
          const float sum = (c & 1 ? a1 : a0) + __shfl_xor_sync(0xffffffffu, c & 1 ? a0 : a1, 1);
          const int j = 8 * c + g, pos = w.base(p.geo, p.c.page_size, SP_TK) + j;
          if (it + k < n_my && j < w.room(p.geo, p.c.page_size, SP_TK) && pos < Lmax) atomicAdd(mass + pos, sum);
          w.next(p.geo);
        }
      }
    };
    if (nan) add_weights(std::true_type());
    else add_weights(std::false_type());
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(s_tmem, sp_cols(NT));
  }
  // a wait that ran out leaves copies in flight: see them land before the memory is given back
  if (dead)
    for (int s = 0; s < SP_NS; ++s) { tc::mbar_wait(&full[warp][s], 0); tc::mbar_wait(&full[warp][s], 1); }
}

// Joins the key splits of a row: one warp per row, splits in order.
template <typename T>
__global__ void __launch_bounds__(128) combine_kernel(const AttnP p) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, i = blockIdx.z;
  const int rho = blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_trigger();
  const Req r = request(p, i);
  pdl_wait();
  if (rho >= r.c * p.G) return;
  const size_t at = (((size_t)i * p.c.n_kv_heads + h) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit;
  float M = -INFINITY;
  for (int s = lane; s < p.nsplit; s += 32) M = fmaxf(M, p.part_ml[at + s].x);
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  float sum = 0.f, a0 = 0.f, a1 = 0.f;
  for (int s = 0; s < p.nsplit; ++s) {
    const float2 ml = p.part_ml[at + s];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    const float2 v = *reinterpret_cast<const float2*>(p.part_o + (at + s) * WS_DH + 2 * lane);
    sum = fmaf(f, ml.y, sum);
    a0 = fmaf(f, v.x, a0);
    a1 = fmaf(f, v.y, a1);
  }
  const int t = rho / p.G, u = h * p.G + rho - t * p.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = (T*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u * WS_DH + 2 * lane;
  out[0] = from_f<T>(a0 * inv);
  out[1] = from_f<T>(a1 * inv);
  if (lane != 0) return;
  const float x = sum == 0.f ? -INFINITY : M + lg2(sum);
  if (p.lse) p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u] = x * LN2;
  if (p.nl) {
    const int TR = p.G * (FA_ROWS / p.G), rt = rho / TR;
    p.nl[(((size_t)i * p.c.n_kv_heads + h) * p.row_tiles + rt) * FA_ROWS + rho - rt * TR] = x == -INFINITY ? x : -x;
  }
}

// ------------------------------------------------------------------ bf16: accumulated weights
// With every row's log-sum-exp known, a second look at the keys: a warp holds
// 32 keys as matrix operands in registers and walks over all rows, eight at
// a time, adding 2^(s * sl - lse * log2 e) per key.  A position belongs to
// one warp, so the sum has a fixed order and needs no atomics.  A dot
// product does not care which dim stands at which k of the instruction, so
// lane c of a quad takes dims 16 c .. 16 c + 15 of its key and of its query
// row: two 16-byte loads each, whole lines per warp.
__device__ __forceinline__ void mass_load(const bf16* row, int c, uint32_t f[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + 16 * c)), b = __ldg(reinterpret_cast<const uint4*>(row + 16 * c) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__global__ void __launch_bounds__(128) mass_kernel(const AttnP p) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y, i = blockIdx.z;
  const Req r = request(p, i);
  const int k0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 32;
  if (k0 >= r.L || r.c == 0) {             // waits all the same: this grid's end has to follow the rows' kernels'
    pdl_wait();
    return;
  }
  uint32_t ka[2][2][8];                    // [16-key step][key g or g + 8][2 * step of 16 dims + half]
  uint32_t valid = 0;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int pos = k0 + 16 * mt + 8 * e + g;
      const int page = pos < r.L ? paged_page(p.c, p.c.page_table, p.c.table_stride, r.slot, pos) : -1;
#pragma unroll
      for (int q = 0; q < 8; ++q) ka[mt][e][q] = 0u;
      if (page >= 0) {
        valid |= 1u << (2 * mt + e);
        mass_load((const bf16*)p.c.k + paged_off(p.c, page, h, pos), c, ka[mt][e]);
      }
    }
  const int R = r.c * p.G;
  pdl_wait();                              // the log-sum-exps
  float sum[2][2] = {};
  // rows before the first that sees position k0 add nothing
  const int first = p.a.causal ? max(0, k0 - (r.L - r.c)) * p.G : 0;
  for (int r0 = first; r0 < R; r0 += 8) {
    uint32_t qf[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) qf[q] = 0u;
    if (r0 + g < R) {
      const int t = (r0 + g) / p.G;
      mass_load((const bf16*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride + (size_t)(h * p.G + r0 + g - t * p.G) * WS_DH, c, qf);
#pragma unroll
      for (int q = 0; q < 8; ++q) qf[q] = (qf[q] & p.q_and) ^ p.q_xor;
    }
    float nl[2];
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rho = r0 + 2 * c + e;
      const bool on = rho < R;
      const int t = on ? rho / p.G : 0;
      const float x = on ? p.lse[(size_t)(r.row0 + t) * p.a.n_heads + h * p.G + rho - t * p.G] : -INFINITY;
      lim[e] = on && x != -INFINITY ? row_limit(p, r, t) : 0;
      nl[e] = x * LOG2E;
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t a[4] = {ka[mt][0][2 * s], ka[mt][1][2 * s], ka[mt][0][2 * s + 1], ka[mt][1][2 * s + 1]};
        mma_bf16_16816(sc, a, qf[2 * s], qf[2 * s + 1]);
      }
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (k0 + 16 * mt + 8 * e2 + g < lim[e]) sum[mt][e2] += ex2(fmaf(sc[2 * e2 + e], p.sl, -nl[e]));
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = sum[mt][e];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (c == 0 && ((valid >> (2 * mt + e)) & 1u))
        p.a.mass[((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride + k0 + 16 * mt + 8 * e + g] += s;
    }
}

// ------------------------------------------------------------------ host
const char* check_attn(const ws_paged_cache* c, const ws_attention_args* a) {
  if (const char* e = check_paged_cache(c)) return e;
  if (!a) return "null arguments";
  if (a->n_req < 0 || a->n_req > 65535) return "n_req must be 0..65535";
  if (a->total_q < 0 || a->max_q < 0 || a->max_kv < 0) return "negative size";
  if (a->n_heads < 1 || a->n_heads % c->n_kv_heads || a->n_heads > 65535)
    return "n_heads must be a multiple of n_kv_heads, at most 65535";
  if ((long long)a->max_q * (a->n_heads / c->n_kv_heads) > (1ll << 28) || a->max_kv > (1 << 30))
    return "max_q times the heads that share a KV head must be at most 2^28, max_kv at most 2^30";
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
  if (a->q_stride >= (int64_t)1 << 37 || a->out_stride >= (int64_t)1 << 37) return "q_stride or out_stride too large";
  if (a->mass && a->mass_stride < a->max_kv) return "mass_stride must be >= max_kv";
  if (!a->req_ids && a->n_req > c->n_slots) return "more requests than slots";
  return nullptr;
}

// The launch shape and the workspace of a call: a function of the host sizes.
struct Plan {
  F32Rows rows = {};                       // fp32, up to 16 rows
  int rpt = 0;                             // fp32: row tiles of 16 * rpt rows (0: up to 16 rows, f32_rows_kernel)
  bool fa = false;                         // tcgen05 row tiles instead of streaming ones
  int nt = 1;                              // streaming row tile: 8 * nt rows
  int row_tiles = 1, nsplit = 1, tps = 1;
  bool stash = false;                      // the streaming kernel adds the mass itself
  TileGeo geo;
  bool parts = false;                      // the first kernel leaves partials to be joined
  size_t lse = 0, ml = 0, o = 0, nl = 0, next = 0, bytes = 0;
};
constexpr int SMS = 152, SLOTS = 2 * SMS;  // two streaming CTAs on each of 152 SMs

// `block`: the rows of a context's verify blocks (at most 16 per KV head).  A
// row has to come out the same bits in blocks of any height and beside any
// number of requests, so its keys are cut by the host bound max_kv alone (the
// context passes its max_frames): into one part (bf16), or the parts of one
// cluster (fp32).
constexpr int BLOCK_ROWS = 16;
Plan make_plan(const ws_paged_cache& c, const ws_attention_args& a, bool block = false) {
  Plan q;
  const long long R = (long long)a.max_q * (a.n_heads / c.n_kv_heads);
  auto take = [&](size_t n) { const size_t at = q.bytes; q.bytes += (n + 255) / 256 * 256; return at; };
  auto partials = [&](long long R_) {
    if (q.nsplit <= 1 && c.dtype == WS_BF16) return;
    q.parts = true;
    const size_t rows = (size_t)a.n_req * c.n_kv_heads * R_ * q.nsplit;
    q.ml = take(rows * 8);
    q.o = take(rows * WS_DH * 4);
  };
  if (c.dtype != WS_BF16) {
    q.geo = tile_geo(c.page_size, F32_KEYS);
    // 64 requests x 6 heads over 112-448 positions: 16 rows 62 us as rows, 17
    // rows 73 us in tiles of 32 and 87 in tiles of 64, 48 rows 106 and 90
    q.rpt = R <= 16 ? 0 : R <= 32 ? 2 : 4;
    if (!q.rpt) {
      q.rows = block ? f32_block_plan(a.max_kv)
                     : f32_rows_plan((long long)a.n_req * c.n_kv_heads, a.max_kv, a.mass != nullptr);
      if (q.rows.join) return q;
      q.nsplit = q.rows.ctas;
    }
    if (a.mass && !a.lse) q.lse = take((size_t)a.total_q * a.n_heads * 4);
    if (!q.rpt) { partials(R); return q; }
    q.row_tiles = (int)((R + 16 * q.rpt - 1) / (16 * q.rpt));
    const int tiles = max(1, (a.max_kv + F32_KEYS - 1) / F32_KEYS);
    const long long units = (long long)a.n_req * c.n_kv_heads * q.row_tiles;
    // enough CTAs for two rounds of two per SM
    const int want = (int)min((2ll * SLOTS + units - 1) / units, (long long)tiles);
    q.tps = (tiles + want - 1) / want;
    q.nsplit = (tiles + q.tps - 1) / q.tps;
    if (q.nsplit > 1) partials(R);
    return q;
  }
  const int G = a.n_heads / c.n_kv_heads;
  // Row tiles of 128 rows on tcgen05 or of 32 that stream the cache: 96
  // requests x 20 heads over 375-1500 positions take 152 us on tcgen05 at 48
  // rows (156 at 128) and 104 / 111 / 119 / 146 / 164 / 185 us streaming at
  // 17 / 32 / 33 / 40 / 48 / 64 rows (with the weights 300 against 179 / 188
  // / 259 / 302 / 335 / 387); 4 requests over 4-16 thousand positions 84
  // against 76 / 78 / 81 / 87 / 99 / 104 us.
  if (R > 40 && G <= FA_ROWS && a.scale > 0.f) {
    q.fa = true;
    q.row_tiles = (a.max_q + FA_ROWS / G - 1) / (FA_ROWS / G);
    q.geo = tile_geo(c.page_size, FA_KEYS);
    const int tiles = max(1, tile_count(q.geo, c.page_size, FA_KEYS, a.max_kv));
    const long long units = (long long)a.n_req * c.n_kv_heads * ((q.row_tiles + 1) / 2);
    // One round of CTAs (two per SM with one row tile each, else one), none
    // shorter than four key tiles: a single request fills the round (a CTA
    // more than the round costs another: 64 rows over 65,536 positions 140 us
    // with 16 splits of 20 heads, 97 with 15), several requests' lengths
    // differ and leave CTAs without keys, so one split more (4 requests over
    // 4-16 thousand positions 101 us without it, 83 with it).
    const long long round = (q.row_tiles == 1 ? 2ll : 1ll) * SMS / units + (a.n_req > 1 ? 1 : 0);
    const int want = (int)max(1ll, min(round, (long long)(tiles / 4)));
    q.tps = (tiles + want - 1) / want;
    q.nsplit = (tiles + q.tps - 1) / q.tps;
    partials(R);
    if (a.mass) {
      q.nl = take((size_t)a.n_req * c.n_kv_heads * q.row_tiles * FA_ROWS * 4);
      q.next = take(8);
    }
    return q;
  }
  if (a.mass && !a.lse) q.lse = take((size_t)a.total_q * a.n_heads * 4);
  // the smallest row tile that holds all rows (16 rows of 96 requests: 90 us,
  // 103 in a tile of 32; 8 rows 88 in either)
  q.nt = R <= 8 ? 1 : R <= 16 ? 2 : 4;
  q.row_tiles = (int)((R + 8 * q.nt - 1) / (8 * q.nt));
  const long long units = (long long)a.n_req * c.n_kv_heads * q.row_tiles;
  q.geo = tile_geo(c.page_size, SP_TK);
  const int tiles = max(1, tile_count(q.geo, c.page_size, SP_TK, a.max_kv));
  // Enough CTAs for about four rounds of the machine, none shorter than 512
  // keys.  With weights, one CTA keeps all scores where they fit, unless that
  // leaves most SMs idle: 20 heads x 9 rows x 2048 positions of 1 / 4 / 16
  // requests 32 / 33 / 60 us in one CTA each, 27 / 43 / 92 us split and with
  // the second pass over the keys.
  const bool fits = a.mass && q.row_tiles == 1 && tiles <= SP_W * sp_stash_tiles(q.nt);
  const int want = block || (fits && units >= SMS / 2)
                       ? 1
                       : (int)min((4ll * SLOTS + units - 1) / units, (long long)max(1, a.max_kv / 512));
  q.tps = (tiles + want - 1) / want;
  q.nsplit = (tiles + q.tps - 1) / q.tps;
  q.stash = fits && q.nsplit == 1;
  partials(R);
  return q;
}

template <int NT, bool STASH, bool HILO = NT == 1, bool MIX = false>
cudaError_t run_split(const AttnP& p, const Plan& q, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(split_kernel<NT, STASH, HILO, MIX>, cudaFuncAttributeMaxDynamicSharedMemorySize, SP_SMEM);
  if (e != cudaSuccess) return e;
  split_kernel<NT, STASH, HILO, MIX><<<dim3(q.row_tiles * q.nsplit, p.c.n_kv_heads, p.a.n_req), SP_W * 32, SP_SMEM, s>>>(
      p, reinterpret_cast<const CUtensorMap&>(mk), reinterpret_cast<const CUtensorMap&>(mv));
  ws_count_launches(1);
  return cudaGetLastError();
}

template <bool MIX>
cudaError_t run_tiles(const AttnP& p, const Plan& q, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  if (q.nt == 1) return q.stash ? run_split<1, true, true, MIX>(p, q, mk, mv, s) : run_split<1, false, true, MIX>(p, q, mk, mv, s);
  if (q.nt == 2) return q.stash ? run_split<2, true, false, MIX>(p, q, mk, mv, s) : run_split<2, false, false, MIX>(p, q, mk, mv, s);
  return q.stash ? run_split<4, true, false, MIX>(p, q, mk, mv, s) : run_split<4, false, false, MIX>(p, q, mk, mv, s);
}

cudaError_t run_streaming(const AttnP& p, const Plan& q, cudaStream_t s) {
  TcMap mk, mv;
  if (!tc_encode_paged(&mk, p.c.k, p.c, (uint32_t)q.geo.box) || !tc_encode_paged(&mv, p.c.v, p.c, (uint32_t)q.geo.box))
    return cudaErrorInvalidValue;
  if (p.pad_H) {                           // a context's block: all rows see all
    if (q.nt == 1) return q.stash ? run_split<1, true>(p, q, mk, mv, s) : run_split<1, false>(p, q, mk, mv, s);
    return q.stash ? run_split<2, true, true>(p, q, mk, mv, s) : run_split<2, false, true>(p, q, mk, mv, s);
  }
  return p.a.causal && p.a.max_q > 1 ? run_tiles<true>(p, q, mk, mv, s) : run_tiles<false>(p, q, mk, mv, s);
}

template <typename T>
cudaError_t combine(const AttnP& p, cudaStream_t s) {
  return launch_after(combine_kernel<T>, dim3((unsigned)(((long long)p.a.max_q * p.G + 3) / 4), p.c.n_kv_heads, p.a.n_req), 128,
                      0, s, p);
}

cudaError_t run_bf16(const AttnP& p, const Plan& q, cudaStream_t s) {
  cudaError_t e = q.fa ? launch_fa(p, s) : run_streaming(p, q, s);
  if (e == cudaSuccess && q.parts) e = combine<bf16>(p, s);
  if (e != cudaSuccess || !p.a.mass || p.a.max_kv == 0 || q.stash) return e;
  if (q.fa) return launch_fa_mass(p, s);
  return launch_after(mass_kernel, dim3((p.a.max_kv + 127) / 128, p.c.n_kv_heads, p.a.n_req), 128, 0, s, p);
}

cudaError_t run_f32(const AttnP& p, const Plan& q, cudaStream_t s) {
  cudaError_t e = q.rpt ? launch_f32(p, q.rpt, s) : launch_f32_rows(p, q.rows, s);
  if (e == cudaSuccess && q.parts) e = combine<float>(p, s);
  if (e != cudaSuccess || !p.a.mass || p.a.max_kv == 0 || q.rows.join) return e;
  return launch_f32_mass(p, q.rpt, s);
}

cudaError_t run(const ws_paged_cache& cache, const ws_attention_args& args, int pad_H, const int32_t* chunk_len,
                const Plan& q, char* ws, cudaStream_t s) {
  AttnP p = {};
  p.c = cache;
  p.a = args;
  p.pad_H = pad_H;
  p.chunk_len = chunk_len;
  p.G = args.n_heads / cache.n_kv_heads;
  p.sl = args.scale == 0.f ? 1.f : fabsf(args.scale) * LOG2E;
  p.q_and = args.scale == 0.f ? 0u : 0xffffffffu;
  p.q_xor = args.scale < 0.f ? 0x80008000u : 0u;
  p.nsplit = q.nsplit; p.tps = q.tps; p.geo = q.geo;
  p.lse = args.lse ? args.lse : args.mass && !q.fa && !q.rows.join ? (float*)(ws + q.lse) : nullptr;
  p.row_tiles = q.row_tiles;
  if (q.fa && args.mass) { p.nl = (float*)(ws + q.nl); p.next_item = (unsigned long long*)(ws + q.next); }
  if (q.parts) { p.part_ml = (float2*)(ws + q.ml); p.part_o = (float*)(ws + q.o); }
  return cache.dtype == WS_BF16 ? run_bf16(p, q, s) : run_f32(p, q, s);
}

}  // namespace

size_t block_attention_workspace(const ws_paged_cache& cache, const ws_attention_args& args) {
  return make_plan(cache, args, true).bytes;
}
cudaError_t launch_block_attention(const ws_paged_cache& cache, const ws_attention_args& args, int H,
                                   const int32_t* block_len, void* workspace, cudaStream_t s) {
  if ((long long)args.max_q * (args.n_heads / cache.n_kv_heads) > BLOCK_ROWS) return cudaErrorInvalidValue;
  return run(cache, args, H, block_len, make_plan(cache, args, true), (char*)workspace, s);
}

extern "C" size_t ws_paged_attention_workspace(const ws_paged_cache* cache, const ws_attention_args* args) {
  if (check_attn(cache, args) || args->n_req == 0 || args->total_q == 0 || args->max_q == 0) return 0;
  return make_plan(*cache, *args).bytes;
}

extern "C" int ws_paged_attention(const ws_paged_cache* cache, const ws_attention_args* args, void* workspace,
                                  size_t workspace_bytes, ws_stream stream) {
  if (const char* e = check_attn(cache, args)) return paged_fail(WS_EINVAL, e);
  if (args->n_req == 0 || args->total_q == 0 || args->max_q == 0) return WS_OK;
  const Plan q = make_plan(*cache, *args);
  if (q.bytes && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return paged_fail(WS_EINVAL, "workspace must be 16-byte aligned and not null");
  if (q.bytes > workspace_bytes) return paged_fail(WS_ENOSPACE, "workspace smaller than ws_paged_attention_workspace()");
  // key splits, row tiles and the weight passes read q after the first rows are stored
  const int64_t es = cache->dtype == WS_BF16 ? 2 : 4;
  if (rows_overlap(args->q, args->q_stride * es, args->out, args->out_stride * es, args->total_q,
                   (int64_t)args->n_heads * WS_DH * es))
    return paged_fail(WS_EINVAL, "out must not share elements with q");
  if (cudaError_t prior = cudaPeekAtLastError(); prior != cudaSuccess)
    return paged_fail(WS_ECUDA, std::string("a CUDA error was pending before this call: ") + cudaGetErrorString(prior));
  const cudaError_t e = run(*cache, *args, 0, nullptr, q, (char*)workspace, (cudaStream_t)stream);
  if (e != cudaSuccess) return paged_fail(WS_ECUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
  return WS_OK;
}

// ws_paged_attention for long chunks of the bf16 model, on tcgen05.
//
// fa_kernel.  One CTA per (request, KV head, W row tiles of up to 128 rows)
// and key range.  Rows are chunk rows x the query heads that share the KV
// head, so a box of the query map is a row tile.  W = 2, or, where a request
// has one row tile, W = 1 with half of the CTA's means, so that two CTAs
// share an SM and one's first copies and last rows lie under the other's
// tiles (96 requests x 20 heads x 128 rows over 375-1500 positions: 187 ->
// 156 us; with more row tiles W = 2 copies the keys half as often: 219 us
// against 306 for 4 x 2048 rows).  Row tiles A and B share every key tile of
// 128 keys:
//   warps 0, 2   producers: Q once and the K tiles; the V tiles (page by page)
//   warp 3       clears value rows that do not count, and values that are not
//                finite where some row does not see them
//   warp 1       MMA issuer: S = Q K^T (128 x 128, both from shared memory),
//                O += P V with P from tensor memory and V as it lies in the
//                pages (the "N-major" operand form: no transpose)
//   warps 4..7   softmax of A, warps 8..11 of B: one thread per row
// Tensor memory (256 columns per row tile): S, P and O have columns of their
// own, so the next S is computed as soon as the softmax has S in registers.
// The row's reference is the maximum of its first tile; it moves, and O is
// rescaled in tensor memory, only when a tile's weights pass 2^60.  With head
// width 64 a score costs 256 FLOP and one exponential, so the exponentials
// bound the kernel as much as the tensor core does; scaling and sums are
// packed pairs (f32x2).  P V (64 columns wide) takes the tensor core as long
// as Q K^T (128 wide).  4 requests x 20 heads x 2048 rows over up to 8192
// positions (198 GFLOP): 209 us, 0.95 PFLOP/s of the measured 1.92; tensor
// pipe 52% busy, exponential pipe 44%.
//
// fa_mass_kernel.  The weights summed per key, once every row's log-sum-exp
// is known: S^T = K Q^T puts a key into each thread, which adds
// 2^(s * sl - lse * log2 e) over the rows of a tile in order, without a
// reduction across threads.  A second pass over the scores (99 GFLOP more)
// and as many exponentials again: 160 us for the call above, exponential
// pipe 55% busy.
#include "ws_pattn.cuh"

namespace {

constexpr int TILE = FA_KEYS * WS_DH * 2;          // 16 KB: a Q, K or V tile
// What the cache holds: bf16; 8 bits whose scales hold for whole groups of 16
// positions; or 8 bits with other blocks.
enum { MODE_BF16 = 0, MODE_GROUPS = 1, MODE_ANY = 2 };
constexpr int CONV = 4;                            // 8 bits: converter warps
template <int W, int MODE = MODE_BF16>
struct FaShape {                                   // a CTA with W row tiles; 3 - W run on an SM
  static constexpr int STAGES = 2 * W;             // key stages
  static constexpr bool Q8 = MODE != MODE_BF16;
  // K producer, MMA, V producer, V cleaner | converters | softmax A | softmax B
  static constexpr int THREADS = 128 + (Q8 ? 128 : 0) + 128 * W;
  static constexpr int AHEAD = 3;                  // 8 bits: tiles of codes in shared memory, TILE bytes each
  static constexpr int SMEM = W * TILE + STAGES * 2 * TILE + (Q8 ? AHEAD * TILE : 0) + 1024;
  static constexpr uint32_t COLS = 256 * W;        // tensor memory
};
constexpr uint32_t IDESC_S = tc::idesc_bf16(128, 128);
constexpr uint32_t IDESC_PV = tc::idesc_bf16(128, 64) | (1u << 16);   // B (V) is N-major
constexpr uint32_t F16_FOR_BF16 = ~((1u << 7) | (1u << 10));          // descriptors' types of A and B
constexpr float MOST = 1152921504606846976.0f;     // 2^60: largest sum of a tile's weights before a row's reference moves
struct Meta { uint32_t valid[4]; int base; int full; };

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(tc::smem_u32(dst)), "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// Bounded wait that also gives up once another role has.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > tc::WAIT_BUDGET) { *abort = 1; return false; }
  }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait(bar, parity, abort);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p;
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
      ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Operand whose rows of 128 bytes (128-byte swizzle) run along K: 64 N
// elements per row, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_nmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(1024 >> 4) << 16;                // between groups of 64 N elements (there is one)
  d |= (uint64_t)(1024 >> 4) << 32;                // between groups of 8 K rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void tm_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void tm_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// A warp's look-up of one key tile: where its pages are and which keys count.
struct TileInfo {
  int page;                                        // this lane's page to copy, or -1
  int tok, base, dst;                              // first token in it, the tile's first position, byte offset of the copy
  uint32_t valid[4];
  bool clean;                                      // every row that the copies write counts, or is a zero behind a page's end
};
// PIECES: pages may be taken in pieces.
template <bool PIECES>
__device__ __forceinline__ int tile_entry(const AttnP& p, int t, int lane) {
  const int e = p.geo.tpp ? t / p.geo.tpp : (t << p.geo.ppt_log) + lane;
  return PIECES && p.geo.pieces > 1 ? e / p.geo.pieces : e;
}
template <bool PIECES = false>
__device__ __forceinline__ int tile_page(const AttnP& p, const int32_t* table, int t, int lane) {
  const int e = tile_entry<PIECES>(p, t, lane);
  return (p.geo.tpp || lane < (1 << p.geo.ppt_log)) && e < p.c.table_stride ? __ldg(table + e) : -1;
}
template <bool PIECES = false>
__device__ __forceinline__ TileInfo tile_info(const AttnP& p, int t, int page, int limit, int lane) {
  TileInfo f;
  const bool ok = page >= 0 && page < p.c.n_pages;
  if (p.geo.tpp) {
    const int pi = t / p.geo.tpp, sub = t - pi * p.geo.tpp, room = min(FA_KEYS, p.c.page_size - sub * FA_KEYS);
    f.tok = sub * FA_KEYS;
    f.base = pi * p.c.page_size + f.tok;
    f.dst = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      f.valid[q] = __ballot_sync(0xffffffffu, ok && 32 * q + lane < room && f.base + 32 * q + lane < limit);
    f.page = lane == 0 && ok && f.base < limit ? page : -1;
    f.clean = ok && f.base + room <= limit;        // one page: the same in every lane
  } else {
    const int ps = 1 << p.geo.page_log;
    f.tok = PIECES && p.geo.pieces > 1 ? ((t << p.geo.ppt_log) + lane) % p.geo.pieces * ps : 0;
    f.base = t * FA_KEYS;
    f.dst = lane * ps * 128;
    const uint32_t okm = __ballot_sync(0xffffffffu, ok && f.base + lane * ps < limit);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int j = 32 * q + lane;
      f.valid[q] = __ballot_sync(0xffffffffu, ((okm >> (j >> p.geo.page_log)) & 1u) && f.base + j < limit);
    }
    f.page = (okm >> lane) & 1u ? page : -1;
    f.clean = (f.valid[0] & f.valid[1] & f.valid[2] & f.valid[3]) == 0xffffffffu;
  }
  return f;
}

// The request whose visible length has rank z among the call's, the longest
// first (its own index where there are more than 128 requests): CTAs start in
// order, so the short ones end up filling the last round.  All threads call.
__device__ __forceinline__ int longest_first(const AttnP& p, int z) {
  __shared__ int len[128];
  __shared__ int s_req;
  const int n = p.a.n_req, x = threadIdx.x;
  if (n > 128 || n == 1) return z;
  if (x < n) len[x] = request(p, x).L;
  __syncthreads();
  if (x < n) {
    int rank = 0;
    for (int y = 0; y < n; ++y) rank += len[y] > len[x] || (len[y] == len[x] && y < x);
    if (rank == z) s_req = x;
  }
  __syncthreads();
  return s_req;
}

template <int W>
struct Bars {
  uint64_t q_full[W], full[FaShape<W>::STAGES], empty[FaShape<W>::STAGES], raw[FaShape<W>::STAGES], raw_free[FaShape<W>::STAGES], s_full[W], s_free[W],
      p_full[W], pv_done[W];
};

// Two e4m3 codes times f (a power of two, twice) as bf16: exact, NaN included.
__device__ __forceinline__ uint32_t widen_pair(uint16_t two, __nv_bfloat162 f) {
  uint32_t r;
  asm("{.reg .b32 h;\n\t.reg .b16 a, b;\n\t.reg .f32 x, y;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %1;\n\tmov.b32 {a, b}, h;\n\tcvt.f32.f16 x, a;\n\tcvt.f32.f16 y, b;\n\t"
      "cvt.rn.bf16x2.f32 %0, y, x;}" : "=r"(r) : "h"(two));
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&r), f);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 scale_pair(uint32_t byte) {      // 2^(byte - 127)
  const uint32_t u = byte ? byte << 7 : 0x0040u, two = u | u << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&two);
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }   // bit 7 of a byte: NaN
// 16 codes as fp16, in two 16-byte chunks.
__device__ __forceinline__ void halves16(const uint4& w, uint4& lo, uint4& hi) {
  auto four = [](uint32_t c, uint32_t& a, uint32_t& b) {
    asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
        : "=r"(a), "=r"(b) : "r"(c));
  };
  four(w.x, lo.x, lo.y);
  four(w.y, lo.z, lo.w);
  four(w.z, hi.x, hi.y);
  four(w.w, hi.z, hi.w);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 codes as bf16, with the scale of byte s, in two 16-byte chunks.
__device__ __forceinline__ void widen16(const uint4& w, uint32_t s, uint4& lo, uint4& hi) {
  const __nv_bfloat162 f = scale_pair(s);
  auto four = [f](uint32_t c, uint32_t& a, uint32_t& b) {
    a = widen_pair((uint16_t)c, f);
    b = widen_pair((uint16_t)(c >> 16), f);
  };
  four(w.x, lo.x, lo.y);
  four(w.y, lo.z, lo.w);
  four(w.z, hi.x, hi.y);
  four(w.w, hi.z, hi.w);
}

// A cache in 8 bits: warps 0 and 2 copy codes and scales of keys and of values,
// AHEAD tiles at once, and a warpgroup of converters (warps 4..7) writes the
// stages from them, rows that do not count as zeros; values that are not finite
// and that not every row sees are noted and left out at once, so there is
// nothing to clean.
// (Codes loaded into the converters' registers, or by copies of their own, cost
// a memory latency per tile: a warp's fence before its stores may be read
// waits for whatever it has asked for; 4 x 2048 rows 368 and 590 us.)  W = 2
// also for one row tile: two CTAs of W = 1 leave two warps each and room for
// one tile of codes (96 requests x 20 heads x 128 rows 262 us, 4 x 64 rows over
// 4-16 thousand positions 142 for 91).
//
// MODE_GROUPS: keys become fp16 (one conversion for two codes), and so do the
// queries, each row with a power of two of its own (ws_pattn_q8.cu); a group of
// 16 keys with one scale costs the softmax a factor.  Values become bf16 with
// their scales in them (ten instructions for four codes), because the weights
// have to be bf16: in fp16 their reference moves at 2^15, which some row of a
// warp does in most tiles (348 us).  MODE_ANY: keys like values, which any
// blocks of scales allow.
// The call above in 8 bits, pages and blocks of 16: 285-289 us, 0.69 PFLOP/s;
// blocks of 8 in pages of 64 277, in pages of 16 345.  Without the conversions'
// arithmetic it would take 245: they share the schedulers' issue slots with
// the softmax.
// HEADS: A and B are the only row tiles of two heads, whose key tiles take
// turns in the stages (96 requests x 20 heads x 128 rows 186 us for 227).
template <int W, int MODE, bool HEADS>
__global__ void __launch_bounds__(FaShape<W, MODE>::THREADS, 3 - W)
fa_kernel(const AttnP p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv) {
  using Shape = FaShape<W, MODE>;
  constexpr bool Q8 = MODE != MODE_BF16, GROUPS = MODE == MODE_GROUPS;
  constexpr uint32_t ID_S = GROUPS ? IDESC_S & F16_FOR_BF16 : IDESC_S;
  constexpr int NST = Shape::STAGES, THREADS = Shape::THREADS;
  constexpr uint32_t TM_S = 0, TM_P = 128 * W, TM_O = 192 * W;   // + 128 w, + 64 w, + 64 w
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) Bars<W> B;
  __shared__ Meta meta[NST];
  __shared__ Odd odds[HEADS ? 2 : 1];
  Odd& odd = odds[0];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  constexpr int AHEAD = Shape::AHEAD;
  __shared__ uint8_t s_scale[2][Q8 ? AHEAD : 1][GROUPS ? 8 : FA_KEYS];     // scale bytes of the rows' (groups') keys, and values
  __shared__ __align__(16) float s_ks[GROUPS ? NST : 1][8];                // scales of the groups' keys
  __shared__ Meta raw_meta[Q8 ? AHEAD : 1];        // of the codes
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  if (p.next_item && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *p.next_item = 0ull;
  const int groups = (p.row_tiles + W - 1) / W;
  const int pair = groups - 1 - blockIdx.x / p.nsplit, split = blockIdx.x % p.nsplit;   // the longest rows first
  const int h = HEADS ? 2 * blockIdx.y : blockIdx.y, i = longest_first(p, blockIdx.z);
  const int two = HEADS && h + 1 < p.c.n_kv_heads;         // log2 of the heads
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const Req r = request(p, i);
  const int R = r.c * p.G, RB = FA_ROWS / p.G, TR = RB * p.G;
  const int rho0 = HEADS ? 0 : pair * W * TR;
  if (rho0 >= R) return;
  // key tiles of each row tile within this split
  int n[W], lo;
  {
    const int ps = p.c.page_size;
    lo = split * p.tps;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int first = rho0 + (HEADS ? 0 : w * TR), last = min(R, first + TR) - 1;
      const int nt = last >= first && (!HEADS || w <= two) ? tile_count(p.geo, ps, FA_KEYS, row_limit(p, r, last / p.G)) : 0;
      n[w] = max(0, min(nt, lo + p.tps) - lo);
    }
  }
  const int nmax = max(n[0], n[W - 1]);
  const int items = nmax << two;                   // key tiles of the CTA: tile j of A is item j << two, that of B the next
  volatile int* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int b = 0; b < NST; ++b) {
      tc::mbar_init(&B.full[b], Q8 ? CONV : 2);
      tc::mbar_init(&B.empty[b], 1);
      tc::mbar_init(&B.raw[b], Q8 ? 4 : 1);
      tc::mbar_init(&B.raw_free[b], CONV);
    }
    for (Odd& o : odds) o.any = 0;
    for (int w = 0; w < W; ++w) {
      tc::mbar_init(&B.q_full[w], GROUPS ? 4 : 1); tc::mbar_init(&B.s_full[w], 1); tc::mbar_init(&B.s_free[w], 4);
      tc::mbar_init(&B.p_full[w], 4); tc::mbar_init(&B.pv_done[w], 1);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (Q8)
    for (Odd& o : odds)
      for (int x = threadIdx.x; x < 3 * WS_DH; x += THREADS) o.first[0][x] = 0x7FFFFFFF;
  if (warp == 1) tc::tmem_alloc(&s_tmem, Shape::COLS);
  uint8_t* sQ = sm;
  auto sK = [&](int b) { return sm + W * TILE + b * 2 * TILE; };
  auto sV = [&](int b) { return sm + (W + 1) * TILE + b * 2 * TILE; };
  if (!Q8 && p.geo.tpp && p.geo.box < FA_KEYS)     // value rows that no copy writes
    for (int x = threadIdx.x; x < NST * TILE / 16; x += THREADS)
      reinterpret_cast<uint4*>(sV(x / (TILE / 16)))[x % (TILE / 16)] = make_uint4(0u, 0u, 0u, 0u);
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  pdl_trigger();                                   // only now: a dependent kernel takes tensor memory too
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);

  // Value tiles that go straight to the MMA: all rows that the copies write
  // count, and every row of the CTA sees them all.  The others are cleaned
  // first: values behind the cache's length or of skipped pages may hold
  // anything, and of those that only later rows see, elements that are not
  // finite are taken out (0 * inf would reach the rows before) and come back
  // in the epilogue for the rows that see them.
  const int all_see = row_limit(p, r, rho0 / p.G);
  auto direct = [&](const TileInfo& f) { return f.clean && (all_see >= r.L || f.base + FA_KEYS <= all_see); };
  // ---- a cache in 8 bits: warps 0 (keys) and 2 (values), and the converters
  auto codes = [&](int slot) { return sm + (W + 2 * NST) * TILE + slot * TILE; };        // keys, and TILE / 2 on values
  auto copy_codes = [&](bool values) {
    const int32_t* table = p.c.page_table + (size_t)min(max(r.slot, 0), p.c.n_slots - 1) * p.c.table_stride;
    const uint8_t* scales = values ? p.c.v_scale : p.c.k_scale;
    int page = tile_page<true>(p, table, lo, lane), issued = 0;
    uint32_t sb[4] = {};                           // scale bytes of the tile asked for last
    auto keep_scales = [&](int slot) {
#pragma unroll
      for (int q = 0; q < (GROUPS ? 1 : 4); ++q)
        if (!GROUPS || lane < 8) s_scale[values][slot][32 * q + lane] = (uint8_t)sb[q];
      __syncwarp();
      if (lane == 0) arrive(&B.raw[slot]);
    };
    for (int j = 0; j < items; ++j) {
      const int slot = j % AHEAD, hj = h + (j & two);
      const TileInfo f = tile_info<true>(p, lo + (j >> two), page, r.L, lane);
      if (j + 1 < items) page = tile_page<true>(p, table, lo + ((j + 1) >> two), lane);
      if (j >= AHEAD && !wait_warp(&B.raw_free[slot], (uint32_t)((j / AHEAD - 1) & 1), abort)) break;
      const bool go = f.page >= 0;
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, go)) * (uint32_t)p.geo.box * 64u;
      if (lane == 0) {
        if (!values) {
#pragma unroll
          for (int q = 0; q < 4; ++q) raw_meta[slot].valid[q] = f.valid[q];
          raw_meta[slot].base = f.base;
        }
        tc::mbar_expect_tx(&B.raw[slot], bytes);
      }
      __syncwarp();
      if (go)
        tma_load_4d(codes(slot) + (values ? TILE / 2 : 0) + f.dst / 2, values ? &mv : &mk, &B.raw[slot], 0, f.tok, hj, f.page);
      ++issued;
      // the last tile's scales have arrived by now; this one's are stored with the next
      if (j > 0) keep_scales((j - 1) % AHEAD);
#pragma unroll
      for (int q = 0; q < (GROUPS ? 1 : 4); ++q) {
        const int x = GROUPS ? 16 * (lane & 7) : 32 * q + lane;    // the row whose scale it is
        const int from = p.geo.tpp ? 0 : x >> p.geo.page_log;      // the lane that copies it
        const int pg = __shfl_sync(0xffffffffu, f.page, from), tok0 = __shfl_sync(0xffffffffu, f.tok, from);
        uint32_t valid = f.valid[GROUPS ? 0 : q];
        if (GROUPS) valid = x < 32 ? f.valid[0] : x < 64 ? f.valid[1] : x < 96 ? f.valid[2] : f.valid[3];
        sb[q] = GROUPS && !values ? 127u : 0u;     // of keys that do not count, whose scores are -inf: any but 0
        if ((valid >> (x & 31)) & 1u) {
          const uint32_t tok = (uint32_t)(tok0 + (p.geo.tpp ? x : x & ((1 << p.geo.page_log) - 1)));
          uint32_t b = p.block_mul ? __umulhi(tok, p.block_mul) : tok;     // tok / scale_block, or one more
          b -= b * (uint32_t)p.c.scale_block > tok;
          sb[q] = __ldg(scales + (size_t)hj * (size_t)p.c.scale_head_stride + (uint64_t)(uint32_t)pg * (uint32_t)p.c.scale_page_stride + b);
        }
      }
    }
    if (issued) keep_scales((issued - 1) % AHEAD);
    if (*abort && lane == 0)                       // see the copies in flight land
      for (int j = max(0, issued - AHEAD); j < issued; ++j) tc::mbar_wait(&B.raw[j % AHEAD], (uint32_t)((j / AHEAD) & 1));
  };
  auto convert = [&](int ci) {
    constexpr int NC = CONV, NG = 16 / NC;         // groups of eight rows of a warp
    for (int j = 0; j < items; ++j) {
      const int s = j % NST, slot = j % AHEAD;
      if (j >= NST && !wait_warp(&B.empty[s], (uint32_t)((j / NST - 1) & 1), abort)) break;
      if (!wait_warp(&B.raw[slot], (uint32_t)((j / AHEAD) & 1), abort)) break;
      tc::mbar_try_wait(&B.raw[slot], (uint32_t)((j / AHEAD) & 1));        // every lane sees the copies, not lane 0 alone
      const int base = raw_meta[slot].base;
      const uint32_t* valid = raw_meta[slot].valid;
      const bool all = (valid[0] & valid[1] & valid[2] & valid[3]) == 0xffffffffu, seen = base + FA_KEYS <= all_see;
      if (ci == 0) {
        if (lane < 4) meta[s].valid[lane] = raw_meta[slot].valid[lane];
        if (lane == 0) { meta[s].base = base; meta[s].full = all; }
        if (GROUPS && lane < 8) s_ks[s][lane] = scale_of(s_scale[0][slot][lane]);
      }
#pragma unroll 1                               // unrolled, it overflows the instruction cache (4 x 2048 rows: 404 us)
      for (int q = 0; q < NG; ++q) {
        const int x = 8 * (ci + NC * q) + (lane >> 2);             // this lane's row, and 16 bytes of it
        const uint8_t* src = codes(slot) + x * WS_DH + (((lane & 3) ^ ((x >> 1) & 3)) << 4);
        uint4 kw = *reinterpret_cast<const uint4*>(src), vw = *reinterpret_cast<const uint4*>(src + TILE / 2);
        if (!all && !((valid[x >> 5] >> (x & 31)) & 1u)) kw = vw = make_uint4(0u, 0u, 0u, 0u);
        uint4 klo, khi, vlo, vhi;
        const uint32_t v_byte = s_scale[1][slot][GROUPS ? x >> 4 : x];
        widen16(vw, v_byte, vlo, vhi);
        if (GROUPS) halves16(kw, klo, khi);
        else widen16(kw, s_scale[0][slot][x], klo, khi);
        const uint32_t at = (uint32_t)(x * 128 + (((2 * (lane & 3)) ^ (x & 7)) << 4)), at2 = at ^ 16u;
        *reinterpret_cast<uint4*>(sK(s) + at) = klo;
        *reinterpret_cast<uint4*>(sK(s) + at2) = khi;
        *reinterpret_cast<uint4*>(sV(s) + at) = vlo;
        *reinterpret_cast<uint4*>(sV(s) + at2) = vhi;
        // values that are not finite and that not every row sees: noted, and zero to the product.  NaN codes, and what
        // passes fp32, 2^(code's exponent - 7 + byte - 127) of at least 2^128.
        if (!seen && (v_byte >= 262u - 15u || ((nan_codes(vw.x) | nan_codes(vw.y) | nan_codes(vw.z) | nan_codes(vw.w)) & 0x80808080u))) {
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const uint32_t code = src[TILE / 2 + e];
            const bool nan = (code & 0x7Fu) == 0x7Fu;
            if (!(nan || (code >> 3 & 15u) + v_byte >= 262u) || base + x < all_see) continue;
            *reinterpret_cast<uint16_t*>(sV(s) + (e < 8 ? at : at2) + 2u * (e & 7)) = 0u;
            atomicMin(&odds[j & two].first[nan ? 2 : code >> 7][16 * (lane & 3) + e], base + x);
            odds[j & two].any = 1;
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        arrive(&B.full[s]);
        arrive(&B.raw_free[slot]);
      }
    }
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (Q8 && warp != 1) {
    if (!GROUPS && warp == 0 && lane == 0) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (n[w]) {
          tc::mbar_expect_tx(&B.q_full[w], (uint32_t)TR * 128u);
          tma_load_3d(sQ + w * TILE, &mq, &B.q_full[w], 0, (HEADS ? h + w : h) * p.G, r.row0 + (HEADS ? 0 : pair * W * RB + w * RB));
        }
    }
    __syncwarp();
    if (warp != 3) copy_codes(warp == 2);
  } else if (!Q8 && (warp == 0 || warp == 2)) {
    // ---- producers: Q and K, and V.  Two warps, because small pages make
    // many copies of a tile and one warp's copies are issued one by one.
    const bool values = warp == 2;
    if (!values && lane == 0) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (n[w]) {
          tc::mbar_expect_tx(&B.q_full[w], (uint32_t)TR * 128u);
          tma_load_3d(sQ + w * TILE, &mq, &B.q_full[w], 0, h * p.G, r.row0 + pair * W * RB + w * RB);
        }
    }
    const int32_t* table = p.c.page_table + (size_t)min(max(r.slot, 0), p.c.n_slots - 1) * p.c.table_stride;
    int page = tile_page(p, table, lo, lane), issued = 0;
    uint32_t raw = 0, phase = 0;                   // by stage: the last tile went to the cleaner; its barrier's parity
    for (int j = 0; j < nmax; ++j) {
      const int s = j % NST;
      const TileInfo f = tile_info(p, lo + j, page, r.L, lane);
      if (j + 1 < nmax) page = tile_page(p, table, lo + j + 1, lane);
      if (j >= NST && !wait_warp(&B.empty[s], (uint32_t)((j / NST - 1) & 1), abort)) break;
      const bool go = f.page >= 0;
      const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, go)) * (uint32_t)p.geo.box * 128u;
      const bool dirty = values && !direct(f);
      uint64_t* bar = dirty ? &B.raw[s] : &B.full[s];
      if (lane == 0) {
        if (!values) {
#pragma unroll
          for (int q = 0; q < 4; ++q) meta[s].valid[q] = f.valid[q];
          meta[s].base = f.base;
          meta[s].full = (f.valid[0] & f.valid[1] & f.valid[2] & f.valid[3]) == 0xffffffffu;
        }
        tc::mbar_expect_tx(bar, bytes);
      }
      __syncwarp();
      if (go) tma_load_4d((values ? sV(s) : sK(s)) + f.dst, values ? &mv : &mk, bar, 0, f.tok, h, f.page);
      ++issued;
      raw = dirty ? raw | 1u << s : raw & ~(1u << s);
      if (dirty) phase ^= 1u << s;
    }
    if (*abort && lane == 0)                       // see the copies in flight land
      for (int j = max(0, issued - NST); j < issued; ++j) {
        const int s = j % NST;
        if ((raw >> s) & 1u) tc::mbar_wait(&B.raw[s], ~(phase >> s) & 1u);
        else tc::mbar_wait(&B.full[s], (uint32_t)((j / NST) & 1));
      }
  } else if (!Q8 && warp == 3) {
    // ---- cleaner
    const int32_t* table = p.c.page_table + (size_t)min(max(r.slot, 0), p.c.n_slots - 1) * p.c.table_stride;
    int page = tile_page(p, table, lo, lane);
    uint32_t phase = 0;
    for (int j = 0; j < nmax; ++j) {
      const int s = j % NST;
      const TileInfo f = tile_info(p, lo + j, page, r.L, lane);
      if (j + 1 < nmax) page = tile_page(p, table, lo + j + 1, lane);
      if (direct(f)) continue;
      if (!wait_warp(&B.raw[s], (phase >> s) & 1u, abort)) break;
      tc::mbar_try_wait(&B.raw[s], (phase >> s) & 1u);         // every lane sees the copy, not lane 0 alone
      phase ^= 1u << s;
      if (!f.clean) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!((f.valid[q] >> lane) & 1u))
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4*>(sV(s) + (32 * q + lane) * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      if (all_see < r.L && f.base + FA_KEYS > all_see) take_out_odd<FA_KEYS, 8, false>(odd, sV(s), f.base, lane);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(&B.full[s]);
    }
  } else if (warp == 1) {
    // ---- MMA issuer: the whole warp walks along, so that descriptors stay
    // in uniform registers; one elected lane issues
    const uint32_t lead = elect_one();
    const uint64_t qd0 = tc::sdesc_sw128(tc::smem_u32(sQ)), kd0 = tc::sdesc_sw128(tc::smem_u32(sK(0))),
                   vd0 = sdesc_nmajor(tc::smem_u32(sV(0)));
    auto qk = [&](int w, int j) -> bool {
      const int it = HEADS ? (j << two) + w : j, s = it % NST;
      if ((HEADS || w == 0 || j >= n[0]) && !wait(&B.full[s], (uint32_t)((it / NST) & 1), abort)) return false;
      if (j > 0 && !wait(&B.s_free[w], (uint32_t)((j - 1) & 1), abort)) return false;
      tc::tc_fence_after();
      if (lead) {
        const uint64_t qd = qd0 + (uint64_t)(w * (TILE >> 4)), kd = kd0 + (uint64_t)(s * (2 * TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < WS_DH / 16; ++kk)
          tc::umma_bf16(tmem + TM_S + 128u * w, qd + (uint64_t)(kk * 2), kd + (uint64_t)(kk * 2), ID_S, kk ? 1u : 0u);
        tc::umma_commit(&B.s_full[w]);
      }
      __syncwarp();
      return true;
    };
    auto pv = [&](int w, int j) -> bool {
      const int s = (HEADS ? (j << two) + w : j) % NST;
      if (!wait(&B.p_full[w], (uint32_t)(j & 1), abort)) return false;
      tc::tc_fence_after();
      if (lead) {
        const uint64_t vd = vd0 + (uint64_t)(s * (2 * TILE >> 4));
#pragma unroll
        for (int kk = 0; kk < FA_KEYS / 16; ++kk)
          umma_ts(tmem + TM_O + 64u * w, tmem + TM_P + 64u * w + 8u * kk, vd + (uint64_t)(kk * 128), IDESC_PV,
                  (j | kk) ? 1u : 0u);
        tc::umma_commit(&B.pv_done[w]);
        if (HEADS || w == W - 1 || j >= n[W - 1]) tc::umma_commit(&B.empty[s]);     // the stage's last reader
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    int sc[W] = {}, pc[W] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
      if (ok && n[w]) { ok = wait(&B.q_full[w], 0, abort) && qk(w, 0); sc[w] = ok; }
    for (int j = 0; j < nmax && ok; ++j)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (ok && j + 1 < n[w]) { ok = qk(w, j + 1); sc[w] += ok; }
        if (ok && j < n[w]) { ok = pv(w, j); pc[w] += ok; }
      }
    if (*abort && lane == 0)                       // nothing may be in flight when the CTA ends
      for (int w = 0; w < W; ++w) {
        if (n[w]) tc::mbar_wait(&B.q_full[w], 0);
        if (sc[w]) tc::mbar_wait(&B.s_full[w], (uint32_t)((sc[w] - 1) & 1));
        if (pc[w]) tc::mbar_wait(&B.pv_done[w], (uint32_t)((pc[w] - 1) & 1));
      }
    __syncwarp();
  }
  } else if (Q8 && warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    convert(warp - 4);
  } else {
    // ---- softmax: thread = row
    if (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");        // 128 a thread at launch: 4 * 128 = 2 * 72 + 2 * 184
    else if (W == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");     // 168 a thread at launch
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");            // 128
    const int w = (warp >> 2) - (Q8 ? 2 : 1), quarter = warp & 3, x = quarter * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tS = tl + TM_S + 128u * w, tP = tl + TM_P + 64u * w, tO = tl + TM_O + 64u * w;
    const int first = rho0 + (HEADS ? 0 : w * TR), rho = first + x, hw = HEADS ? h + w : h;
    const bool on = x < TR && rho < R && (!HEADS || w <= two);
    const int t = on ? rho / p.G : 0;
    const int lim = on ? row_limit(p, r, t) : 0, lim_all = first < R ? row_limit(p, r, first / p.G) : 0;
    const int nw = n[w];
    float sl = p.sl;
    if (GROUPS && nw > 0) {                        // this row's query as fp16, its largest element in 1 .. 2
      const bf16* q = (const bf16*)p.a.q + (size_t)(r.row0 + t) * p.a.q_stride + (size_t)(hw * p.G + (on ? rho - t * p.G : 0)) * WS_DH;
      uint4 v[8];
      float most = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        v[c] = on ? __ldg(reinterpret_cast<const uint4*>(q) + c) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = fmaxf(most, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
      }
      const int e2 = most >= 1.17549435e-38f && most < INFINITY ? min((int)(__float_as_uint(most) >> 23) - 127, 126) : 0;
      const float f = __uint_as_float((uint32_t)(127 - e2) << 23);
      sl = score_factor(sl * __uint_as_float((uint32_t)(127 + e2) << 23));
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack_f16(__uint_as_float(u[e] << 16) * f, __uint_as_float(u[e] & 0xFFFF0000u) * f);
        *reinterpret_cast<uint4*>(sQ + w * TILE + x * 128 + ((c ^ (x & 7)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) arrive(&B.q_full[w]);
    }
    const float2 sl2 = make_float2(sl, sl);
    float m = -INFINITY, msl = 0.f, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nw; ++j) {
      if (!wait_warp(&B.s_full[w], (uint32_t)(j & 1), abort)) { ok = false; break; }
      tc::tc_fence_after();
      float sv[FA_KEYS];
#pragma unroll
      for (int q = 0; q < 8; ++q) tm_ld16(tS + 16 * q, sv + 16 * q);
      const int stage = (HEADS ? (j << two) + w : j) % NST;
      const Meta& mt = meta[stage];
      const int base = mt.base;
      const bool dense = mt.full && base + FA_KEYS <= lim_all;
      ld_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&B.s_free[w]);
      if (!dense) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (mt.valid[q] == 0xffffffffu && base + 32 * q + 32 <= lim_all) continue;
          const int room = lim - base - 32 * q;    // columns of this word below the row's limit
          const uint32_t see = mt.valid[q] & (room >= 32 ? 0xffffffffu : room <= 0 ? 0u : (1u << room) - 1u);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1u)) sv[32 * q + e] = -INFINITY;
        }
      }
      // P and O are free once the previous product has finished
      if (j > 0 && !wait_warp(&B.pv_done[w], (uint32_t)((j - 1) & 1), abort)) { ok = false; break; }
      const float* ks = s_ks[GROUPS ? stage : 0];
      float2 sum2[2];
      float slk[8];                                // of the groups
#pragma unroll
      for (int g = 0; g < 8; ++g) slk[g] = GROUPS ? score_factor(sl * ks[g]) : sl;
      auto weigh = [&]() {
        const float2 nm2 = make_float2(-msl, -msl);
        sum2[0] = sum2[1] = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float s1 = slk[2 * q + (e >> 3)];
            float2 y = __ffma2_rn(make_float2(sv[32 * q + 2 * e], sv[32 * q + 2 * e + 1]), GROUPS ? make_float2(s1, s1) : sl2, nm2);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            sum2[e & 1] = __fadd2_rn(sum2[e & 1], y);
            u[e] = pack_bf(y.x, y.y);
          }
          tm_st16(tP + 16 * q, u);
        }
        return (sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y);
      };
      // The weights go by the reference at hand.  A floating sum does not mind
      // large weights, so the maximum is looked for only where a row has no
      // reference yet or its sum grew past 2^60 (the scores are still in
      // registers then).  Lanes without a row have no say: theirs are other
      // requests' rows, rows behind the last chunk, or shared memory that no
      // copy writes (rows TR .. 127), and a row's bits may not depend on them.
      float tile = 0.f;
      auto look = [&]() {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < FA_KEYS; e += 8)
          if (GROUPS) {
            const float top = max3(max3(sv[e], sv[e + 1], sv[e + 2]), max3(sv[e + 3], sv[e + 4], sv[e + 5]), fmaxf(sv[e + 6], sv[e + 7]));
            mx[e / 8 & 3] = fmaxf(mx[e / 8 & 3], top * ks[e / 16]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], sv[e + 2 * q], sv[e + 2 * q + 1]);
          }
        const float mn = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]));
        const float f = m > -INFINITY ? ex2((m - mn) * sl) : (mn > -INFINITY ? 0.f : 1.f);
        m = mn;
        msl = mn > -INFINITY ? mn * sl : 0.f;
        l *= f;
        if (j > 0) {
          st_wait();                               // the first weights are stored before the second ones are
          tc::tc_fence_after();
#pragma unroll(Q8 ? 1 : 4)
          for (int d = 0; d < 4; ++d) {
            float o[16];
            uint32_t v[16];
            tm_ld16(tO + 16 * d, o);
            ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(o[e] * f);
            tm_st16(tO + 16 * d, v);
          }
        }
      };
      auto passed = [&]() { return __any_sync(0xffffffffu, on && (m == -INFINITY || !(tile < MOST))) != 0; };
      if (j > 0) tile = weigh();
      if (j == 0 || passed()) {
        look();
        tile = weigh();
      }
      l += tile;
      st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(&B.p_full[w]);
    }
    if (ok && nw > 0) ok = wait_warp(&B.pv_done[w], (uint32_t)((nw - 1) & 1), abort);
    tc::tc_fence_after();
    const bool any_odd = nw > 0 && *(volatile int*)&odds[HEADS ? w : 0].any != 0;
    if (p.nsplit > 1) {
      const size_t at = on ? (((size_t)i * p.c.n_kv_heads + hw) * ((size_t)p.a.max_q * p.G) + rho) * p.nsplit + split : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float o[16];
        if (nw > 0) { tm_ld16(tO + 16 * q, o); ld_wait(); }
        if (any_odd)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = with_odd(odds[HEADS ? w : 0], o[e], lim, 16 * q + e);
        if (on)
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(p.part_o + at * WS_DH + 16 * q + e) =
                nw > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (on) p.part_ml[at] = make_float2(m == -INFINITY ? m : msl, ok ? l : NAN);
    } else {
      const float inv = !ok ? NAN : l == 0.f ? 0.f : 1.f / l;
      const int u_ = hw * p.G + (on ? rho - t * p.G : 0);
      bf16* out = (bf16*)p.a.out + (size_t)(r.row0 + t) * p.a.out_stride + (size_t)u_ * WS_DH;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float o[16];
        if (nw > 0) { tm_ld16(tO + 16 * q, o); ld_wait(); }
        if (any_odd)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = with_odd(odds[HEADS ? w : 0], o[e], lim, 16 * q + e);
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = nw > 0 ? pack_bf(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
        // a row that sees nothing inside a tile that does has P = 0, l = 0
        if (on) {
          reinterpret_cast<uint4*>(out + 16 * q)[0] = make_uint4(u[0], u[1], u[2], u[3]);
          reinterpret_cast<uint4*>(out + 16 * q)[1] = make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
      if (on && p.nl)
        p.nl[(((size_t)i * p.c.n_kv_heads + h) * p.row_tiles + pair * W + w) * FA_ROWS + x] =
            !ok ? NAN : l == 0.f ? -INFINITY : -(msl + lg2(l));
      if (on && p.lse)
        p.lse[(size_t)(r.row0 + t) * p.a.n_heads + u_] = !ok ? NAN : l == 0.f ? -INFINITY : (msl + lg2(l)) * LN2;
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, Shape::COLS);
}

// ------------------------------------------------------------------ accumulated weights
// Work items are key tiles of (request, KV head), drawn from a counter (a
// fixed share per CTA left the last one 25% behind); two CTAs per SM (256
// tensor memory columns each: S twice).  The
// producer runs up to MST row tiles ahead, across items, so that the next
// item's lengths, pages and keys arrive under the current one's sums: a CTA
// per item spent a third of its time on its first tile.  Two groups of four
// warps take alternate row tiles, one S buffer each: a scheduler then has four
// warps to choose from while exponentials are under way.
constexpr int MST = 4;                             // row tile stages
constexpr int MTHREADS = 320;                      // producer, MMA, two groups of four summing warps
constexpr int MASS_SMEM = 2 * TILE + MST * TILE + 1024;

struct MassItem {
  uint32_t valid[4];
  int base, nt;                                    // first position; row tiles (-1: no more items)
  int q_lo, R, c, L;                               // first row tile; rows, chunk length, cache length
  float* mass;
};
struct MassBars { uint64_t k_full[2], k_empty[2], q_full[MST], empty[MST], s_full[2], s_free[2], t_full[2]; };

__global__ void __launch_bounds__(MTHREADS, 2)
fa_mass_kernel(const AttnP p, int tiles, long long items, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk) {
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) MassBars B;
  __shared__ MassItem item[2];
  __shared__ __align__(16) float nlse[MST][FA_ROWS];   // -lse * log2(e) of a tile's rows
  __shared__ float half[2][FA_KEYS];                   // the second group's sums of an item
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int RB = FA_ROWS / p.G, TR = RB * p.G;
  volatile int* abort = &s_abort;
  if (threadIdx.x == 0) {
    for (int b = 0; b < MST; ++b) { tc::mbar_init(&B.q_full[b], 1); tc::mbar_init(&B.empty[b], 4); }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&B.k_full[b], 1); tc::mbar_init(&B.k_empty[b], 4);
      tc::mbar_init(&B.s_full[b], 1); tc::mbar_init(&B.s_free[b], 4);
      tc::mbar_init(&B.t_full[b], 4);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();                                      // the log-sum-exps and the counter; no tensor memory is held meanwhile
  if (warp == 1) tc::tmem_alloc(&s_tmem, 256);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  auto sK = [&](int b) { return sm + b * TILE; };
  auto sQ = [&](int b) { return sm + 2 * TILE + b * TILE; };

  if (warp == 0) {
    // ---- producer: key tiles, and row tiles with their log-sum-exps
    int n = 0, g = 0;                              // items and row tiles handed over
    auto draw = [&]() {                            // the next item nobody has
      long long x = 0;
      if (lane == 0) x = (long long)atomicAdd(p.next_item, 1ull) + gridDim.x;
      return __shfl_sync(0xffffffffu, x, 0);
    };
    long long it = blockIdx.x;
    auto where = [&](long long x, int& kt, int& h, int& i) {
      const long long u = x / tiles;
      kt = (int)(x - u * tiles); i = (int)(u / p.c.n_kv_heads); h = (int)(u - (long long)i * p.c.n_kv_heads);
    };
    bool ok = true;
    int kt = 0, h = 0, i = 0;
    Req r = {};
    if (it < items) { where(it, kt, h, i); r = request(p, i); }
    while (it < items && ok) {
      // the next item's lengths are asked for now
      const long long it2 = draw();
      int kt2 = 0, h2 = 0, i2 = 0;
      Req r2 = {};
      if (it2 < items) { where(it2, kt2, h2, i2); r2 = request(p, i2); }
      const int R = r.c * p.G, nq = (R + TR - 1) / TR;
      const int base0 = p.geo.tpp ? kt / p.geo.tpp * p.c.page_size + kt % p.geo.tpp * FA_KEYS : kt * FA_KEYS;
      // row tiles before the first row that sees position base0 add nothing
      const int q_lo = p.a.causal ? max(0, base0 - (r.L - r.c)) / RB : 0;
      const int nt = kt < tile_count(p.geo, p.c.page_size, FA_KEYS, r.L) ? max(0, nq - q_lo) : 0;
      if (nt > 0) {
        const int kb = n & 1;
        const int32_t* table = p.c.page_table + (size_t)max(r.slot, 0) * p.c.table_stride;
        const TileInfo f = tile_info(p, kt, tile_page(p, table, kt, lane), r.L, lane);
        const float* nl = p.nl + ((size_t)i * p.c.n_kv_heads + h) * p.row_tiles * FA_ROWS;
        if (n >= 2 && !wait_warp(&B.k_empty[kb], (uint32_t)((n / 2 - 1) & 1), abort)) { ok = false; break; }
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, f.page >= 0)) * (uint32_t)p.geo.box * 128u;
        if (lane == 0) {
          MassItem& m = item[kb];
#pragma unroll
          for (int q = 0; q < 4; ++q) m.valid[q] = f.valid[q];
          m.base = f.base; m.nt = nt; m.q_lo = q_lo; m.R = R; m.c = r.c; m.L = r.L;
          m.mass = p.a.mass + ((size_t)r.slot * p.c.n_kv_heads + h) * p.a.mass_stride;
          tc::mbar_expect_tx(&B.k_full[kb], bytes);
        }
        __syncwarp();
        if (f.page >= 0) tma_load_4d(sK(kb) + f.dst, &mk, &B.k_full[kb], 0, f.tok, h, f.page);
        ++n;
        for (int j = 0; j < nt; ++j, ++g) {
          const int s = g % MST;
          if (g >= MST && !wait_warp(&B.empty[s], (uint32_t)((g / MST - 1) & 1), abort)) { ok = false; break; }
          if (lane == 0) {
            tc::mbar_expect_tx(&B.q_full[s], (uint32_t)TR * 128u + FA_ROWS * 4u);
            tma_load_3d(sQ(s), &mq, &B.q_full[s], 0, h * p.G, r.row0 + (q_lo + j) * RB);
            tc::bulk_g2s(nlse[s], nl + (size_t)(q_lo + j) * FA_ROWS, FA_ROWS * 4, &B.q_full[s]);
          }
        }
      }
      it = it2; kt = kt2; h = h2; i = i2; r = r2;
    }
    if (ok && (n < 2 || wait_warp(&B.k_empty[n & 1], (uint32_t)((n / 2 - 1) & 1), abort)) && lane == 0) {
      item[n & 1].nt = -1;
      arrive(&B.k_full[n & 1]);
    }
    if (*abort && lane == 0) {                     // see the copies in flight land
      for (int x = max(0, n - 2); x < n; ++x) tc::mbar_wait(&B.k_full[x & 1], (uint32_t)((x / 2) & 1));
      for (int x = max(0, g - MST); x < g; ++x) tc::mbar_wait(&B.q_full[x % MST], (uint32_t)((x / MST) & 1));
    }
  } else if (warp == 1) {
    const uint32_t lead = elect_one();
    const uint64_t kd0 = tc::sdesc_sw128(tc::smem_u32(sK(0))), qd0 = tc::sdesc_sw128(tc::smem_u32(sQ(0)));
    int g = 0, used[2] = {0, 0};                   // row tiles so far, and of each S buffer
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int kb = n & 1;
      if (!wait(&B.k_full[kb], (uint32_t)((n / 2) & 1), abort)) break;
      const int nt = item[kb].nt;
      if (nt < 0) break;
      for (int j = 0; j < nt; ++j) {
        const int s = g % MST, b = j & 1;          // an item's even tiles go to the first group, odd ones to the second
        ok = wait(&B.q_full[s], (uint32_t)((g / MST) & 1), abort) &&
             (used[b] == 0 || wait(&B.s_free[b], (uint32_t)((used[b] - 1) & 1), abort));
        if (!ok) break;
        ++used[b];
        tc::tc_fence_after();
        if (lead) {
          const uint64_t kd = kd0 + (uint64_t)(kb * (TILE >> 4)), qd = qd0 + (uint64_t)(s * (TILE >> 4));
#pragma unroll
          for (int kk = 0; kk < WS_DH / 16; ++kk)
            tc::umma_bf16(tmem + 128u * b, kd + (uint64_t)(kk * 2), qd + (uint64_t)(kk * 2), IDESC_S, kk ? 1u : 0u);
          tc::umma_commit(&B.s_full[b]);
        }
        __syncwarp();
        ++g;
      }
    }
    if (*abort && lane == 0)
      for (int b = 0; b < 2; ++b)
        if (used[b] > 0) tc::mbar_wait(&B.s_full[b], (uint32_t)((used[b] - 1) & 1));
    __syncwarp();
  } else {
    // ---- sums: thread = key
    const int quarter = warp & 3, group = warp >= 6 ? 1 : 0;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + 128u * group;
    const float2 sl2 = make_float2(p.sl, p.sl);
    bool ok = true;
    int g = 0, used = 0;
    for (int n = 0; ok; ++n) {
      const int kb = n & 1;
      if (!wait_warp(&B.k_full[kb], (uint32_t)((n / 2) & 1), abort)) break;
      const MassItem& m = item[kb];
      const int nt = m.nt;
      if (nt < 0) break;
      const int pos = m.base + quarter * 32 + lane, R = m.R, q_lo = m.q_lo;
      const int first = p.a.causal ? max(0, pos - (m.L - m.c)) * p.G : 0;      // first row that sees this key
      float* mass = m.mass + pos;
      const bool on = (m.valid[quarter] >> lane) & 1u;
      float2 total = make_float2(0.f, 0.f);
      for (int j = 0; j < nt; ++j, ++g) {
        if ((j & 1) != group) continue;
        const int s = g % MST, rho = (q_lo + j) * TR;
        if (!wait_warp(&B.s_full[group], (uint32_t)(used & 1), abort)) { ok = false; break; }
        ++used;
        tc::tc_fence_after();
        const int cmin = first - rho, cmax = min(TR, R - rho);                 // columns that see this key
        const bool whole = __all_sync(0xffffffffu, cmin <= 0 && cmax == FA_ROWS);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float sv[32];
          tm_ld32(tl + 32 * q, sv);
          ld_wait();
          if (q == 3) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(&B.s_free[group]);
          }
          const float4* nl = reinterpret_cast<const float4*>(nlse[s] + 32 * q);
          // in a tile that is not whole, the 32 columns may still be, or may be out of every lane's range
          const bool all = whole || __all_sync(0xffffffffu, cmin <= 32 * q && cmax >= 32 * q + 32);
          if (!all && __all_sync(0xffffffffu, cmin >= 32 * q + 32 || cmax <= 32 * q)) continue;
          if (all) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 n4 = nl[e];
              float2 a = __ffma2_rn(make_float2(sv[4 * e], sv[4 * e + 1]), sl2, make_float2(n4.x, n4.y));
              float2 c = __ffma2_rn(make_float2(sv[4 * e + 2], sv[4 * e + 3]), sl2, make_float2(n4.z, n4.w));
              a.x = ex2(a.x); a.y = ex2(a.y);
              c.x = ex2(c.x); c.y = ex2(c.y);
              total = __fadd2_rn(total, __fadd2_rn(a, c));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = nlse[s][32 * q + e], y = ex2(fmaf(sv[e], p.sl, x));
              if (32 * q + e >= cmin && 32 * q + e < cmax && x != -INFINITY) total.x += y;
            }
          }
        }
        __syncwarp();
        if (lane == 0) arrive(&B.empty[s]);        // the tile's S is computed and its log-sum-exps are read
      }
      // the second group's part of the sum, then the first's on top
      const float part = ok ? total.x + total.y : NAN;
      if (group == 1) {
        half[kb][quarter * 32 + lane] = part;
        __syncwarp();
        if (lane == 0) arrive(&B.t_full[kb]);
      } else {
        if (!wait_warp(&B.t_full[kb], (uint32_t)((n / 2) & 1), abort)) break;
        // the position is this thread's alone: the atomic has nothing to race with
        if (on) atomicAdd(mass, part + half[kb][quarter * 32 + lane]);
        __syncwarp();
        if (lane == 0) arrive(&B.k_empty[kb]);     // the item's keys, description and sums are read
      }
    }
    tc::tc_fence_before();
  }
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, 256);
}

template <int W, int MODE, bool HEADS = false>
cudaError_t run_fa(const AttnP& p, const TcMap& mq, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  using Shape = FaShape<W, MODE>;
  constexpr auto kernel = fa_kernel<W, MODE, HEADS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::SMEM);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.row_tiles + W - 1) / W * p.nsplit, HEADS ? (p.c.n_kv_heads + 1) / 2 : p.c.n_kv_heads, p.a.n_req);
  kernel<<<grid, Shape::THREADS, Shape::SMEM, s>>>(p, reinterpret_cast<const CUtensorMap&>(mq),
                                                   reinterpret_cast<const CUtensorMap&>(mk),
                                                   reinterpret_cast<const CUtensorMap&>(mv));
  ws_count_launches(1);
  return cudaGetLastError();
}
template <int MODE>
cudaError_t run_q8(const AttnP& p, bool two_heads, const TcMap& mq, const TcMap& mk, const TcMap& mv, cudaStream_t s) {
  return two_heads ? run_fa<2, MODE, true>(p, mq, mk, mv, s) : run_fa<2, MODE>(p, mq, mk, mv, s);
}

}  // namespace

cudaError_t launch_fa(const AttnP& p, bool two_heads, cudaStream_t s) {
  TcMap mq, mk, mv;
  if (!tc_encode_heads(&mq, p.a.q, p.a.q_stride, (uint64_t)p.a.total_q, (uint32_t)p.a.n_heads, (uint32_t)p.G,
                       (uint32_t)(FA_ROWS / p.G)))
    return cudaErrorInvalidValue;
  if (!tc_encode_paged(&mk, p.c.k, p.c, (uint32_t)p.geo.box) || !tc_encode_paged(&mv, p.c.v, p.c, (uint32_t)p.geo.box))
    return cudaErrorInvalidValue;
  if (p.c.dtype == WS_E4M3)
    return p.c.scale_block % 16 == 0 ? run_q8<MODE_GROUPS>(p, two_heads, mq, mk, mv, s) : run_q8<MODE_ANY>(p, two_heads, mq, mk, mv, s);
  return p.row_tiles == 1 ? run_fa<1, MODE_BF16>(p, mq, mk, mv, s) : run_fa<2, MODE_BF16>(p, mq, mk, mv, s);
}

cudaError_t launch_fa_mass(const AttnP& p, cudaStream_t s) {
  TcMap mq, mk;
  if (!tc_encode_heads(&mq, p.a.q, p.a.q_stride, (uint64_t)p.a.total_q, (uint32_t)p.a.n_heads, (uint32_t)p.G,
                       (uint32_t)(FA_ROWS / p.G)) ||
      !tc_encode_paged(&mk, p.c.k, p.c, (uint32_t)p.geo.box))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(fa_mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MASS_SMEM);
  if (e != cudaSuccess) return e;
  const int tiles = tile_count(p.geo, p.c.page_size, FA_KEYS, p.a.max_kv);
  const long long items = (long long)tiles * p.c.n_kv_heads * p.a.n_req;
  if (items == 0) return cudaSuccess;
  return launch_after(fa_mass_kernel, dim3((unsigned)(items < 2 * 152 ? items : 2 * 152)), MTHREADS, MASS_SMEM, s, p, tiles,
                      items, reinterpret_cast<const CUtensorMap&>(mq), reinterpret_cast<const CUtensorMap&>(mk));
}
